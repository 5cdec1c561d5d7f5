"""Argument checks of the key/value cache's entry points: no GPU, nothing is launched or dereferenced."""
import ctypes

import pytest
import torch

import block_scaled_fp4_amax_b200 as fp4
from block_scaled_fp4_amax_b200 import build as fp4build

FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)
EINVAL, EUNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def L():
    fp4build.build()
    return fp4.lib()


def cache_args(a):
    return [a["kq"], a["ks"], a["vq"], a["vs"], a["pages"], a["page"], a["heads"], a["dim"]]


COMMON = dict(kq=FAKE, ks=FAKE, vq=FAKE, vs=FAKE, pages=10, page=16, heads=2, dim=128, fmt=1, block=16, kg=FAKE, vg=FAKE,
              table=FAKE, stride=4, cols=4, seqs=3)


def append(L, **kw):
    a = dict(COMMON, k=FAKE, v=FAKE, dtype=1, tokens=5, ks_=256, kh=128, vs_=256, vh=128, slots=FAKE, mode=0, **{})
    a.update(kw)
    return L.fp4_kv_append(a["k"], a["v"], a["dtype"], a["tokens"], a["ks_"], a["kh"], a["vs_"], a["vh"], a["slots"], a["fmt"],
                           a["block"], a["mode"], a["kg"], a["vg"], *cache_args(a), None)


def read(L, **kw):
    a = dict(COMMON, cu=FAKE, starts=None, total=7, dtype=1, ko=FAKE, vo=FAKE)
    a.update(kw)
    return L.fp4_kv_read(*cache_args(a), a["fmt"], a["block"], a["kg"], a["vg"], a["table"], a["stride"], a["cols"], a["seqs"],
                         a["cu"], a["starts"], a["total"], a["dtype"], a["ko"], a["vo"], None)


def attend(L, **kw):
    a = dict(COMMON, q=FAKE, dtype=1, total=3, qs=1024, qh=128, hq=8, cu=None, max_q=1, lens=FAKE, scale=0.1, causal=1, window=0,
             out=FAKE, lse=None, ws=FAKE, ws_bytes=None)
    a.update(kw)
    need = L.fp4_workspace_size(fp4.OP_KV_ATTENTION, 3, 8) if a["ws_bytes"] is None else a["ws_bytes"]
    return L.fp4_kv_attention(a["q"], a["dtype"], a["total"], a["qs"], a["qh"], a["hq"], *cache_args(a), a["fmt"], a["block"],
                              a["kg"], a["vg"], a["table"], a["stride"], a["cols"], a["seqs"], a["cu"], a["max_q"], a["lens"],
                              a["scale"], a["causal"], a["window"], a["out"], a["lse"], a["ws"], need, None)


@pytest.mark.parametrize("call", [append, read, attend])
@pytest.mark.parametrize("kw,status", [
    (dict(fmt=2), EUNSUPPORTED), (dict(fmt=5), EINVAL), (dict(block=32), EINVAL), (dict(fmt=0, block=16), EINVAL),
    (dict(dim=96), EUNSUPPORTED), (dict(dim=256), EUNSUPPORTED), (dict(page=8), EINVAL), (dict(page=48), EINVAL),
    (dict(page=2048), EINVAL), (dict(heads=0), EINVAL), (dict(heads=1025, hq=1025), EINVAL), (dict(pages=0), EINVAL), (dict(pages=2 ** 31), EINVAL),
    (dict(pages=2 ** 30, page=1024, heads=64, hq=64), EUNSUPPORTED),
    (dict(kq=None), EINVAL), (dict(vs=None), EINVAL), (dict(ks=ODD), EINVAL), (dict(kg=None), EINVAL), (dict(vg=None), EINVAL)])
def test_cache_refusals(L, call, kw, status):
    if call is not attend:
        kw = {k: v for k, v in kw.items() if k != "hq"}
    assert call(L, **kw) == status
    assert L.fp4_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), EINVAL), (dict(mode=3), EINVAL), (dict(mode=2), EUNSUPPORTED), (dict(fmt=0, block=32, mode=1), EUNSUPPORTED),
    (dict(tokens=-1), EINVAL), (dict(k=None), EINVAL), (dict(v=ctypes.c_void_p(0x10010)), EINVAL), (dict(ks_=136), EINVAL),
    (dict(vh=-128), EINVAL), (dict(slots=None), EINVAL), (dict(slots=ctypes.c_void_p(0x10004)), EINVAL),
    (dict(tokens=2 ** 40), EUNSUPPORTED)])
def test_append_refusals(L, kw, status):
    assert append(L, **kw) == status


@pytest.mark.parametrize("kw", [
    dict(dtype=3), dict(total=-1), dict(total=2 ** 31), dict(cu=None), dict(ko=None), dict(vo=ctypes.c_void_p(0x10010)),
    dict(table=None), dict(stride=3), dict(seqs=-1), dict(cols=-1)])
def test_read_refusals(L, kw):
    assert read(L, **kw) == EINVAL


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=0), EUNSUPPORTED), (dict(hq=7), EINVAL), (dict(hq=0), EINVAL), (dict(hq=8192), EINVAL), (dict(total=-1), EINVAL),
    (dict(total=2 ** 25), EINVAL), (dict(total=4), EINVAL), (dict(max_q=0), EINVAL), (dict(scale=float("nan")), EINVAL),
    (dict(scale=float("inf")), EINVAL), (dict(window=-1), EINVAL), (dict(q=None), EINVAL), (dict(q=ODD), EINVAL),
    (dict(qs=1020), EINVAL), (dict(qh=-128), EINVAL), (dict(lens=None), EINVAL), (dict(out=None), EINVAL), (dict(out=ODD), EINVAL),
    (dict(seqs=40000, total=40000), EUNSUPPORTED),
    (dict(page=1024, cols=2 ** 21, stride=2 ** 21), EUNSUPPORTED), (dict(cu=FAKE, max_q=2 ** 30), EUNSUPPORTED),
    (dict(cu=FAKE, max_q=2 ** 28, heads=1, hq=1, seqs=3000, total=2 ** 24), EUNSUPPORTED), (dict(ws=None), EINVAL), (dict(ws=ODD), EINVAL), (dict(ws_bytes=0), EINVAL), (dict(table=None), EINVAL), (dict(stride=1), EINVAL)])
def test_attention_refusals(L, kw, status):
    assert attend(L, **kw) == status


def test_nothing_to_do(L):
    assert append(L, tokens=0, k=None, v=None, slots=None) == 0
    assert read(L, total=0, ko=None) == 0 and read(L, seqs=0) == 0
    assert attend(L, total=0) == 0 and attend(L, seqs=0, total=5) == 0


def test_binding_refuses():
    c = fp4.fp4_kv_alloc(2, 1, 16, 64, device="cpu")
    assert [tuple(t.shape) for t in c] == [(2, 1, 16, 32), (2, 1, 16, 4)] * 2
    assert [t.shape[3] for t in fp4.fp4_kv_alloc(1, 1, 16, 64, fp4.MXFP4, device="cpu")] == [32, 2, 32, 2]
    k = torch.zeros(3, 1, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):  # no CPU path
        fp4.fp4_kv_append(k, k, c, i)
    with pytest.raises(ValueError):
        fp4.fp4_kv_read(c, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 0)
    with pytest.raises(ValueError):
        fp4.fp4_kv_attention(k, c, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
