"""GPU tests of the paged 4-bit key/value cache: bytes against the oracle, reads against its
dequantiser, attention against the formula in 64 bits (tests/kv.py derives the bounds)."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_amax_b200 as fp4
import oracle as O
from kv import FORMATS, Cache, attention64, block_of, check, quantise, run_and_check

pytestmark = pytest.mark.gpu

SENTINEL = 0xA5


def sentinel_cache(pages, heads, page, dim, fmt, device):
    return tuple(t.fill_(SENTINEL) for t in fp4.fp4_kv_alloc(pages, heads, page, dim, fmt, device=device))


def scales_for(fmt, device, k=0.0021, v=0.0016):
    if fmt == fp4.MXFP4:
        return {}
    return {n: torch.tensor([g], dtype=torch.float32, device=device) for n, g in (("k_global", k), ("v_global", v))}


# ---------------------------------------------------------------------------------------------
# append

@pytest.mark.parametrize("fmt,four_six", [("nvfp4", False), ("nvfp4", True), ("mxfp4", False)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,heads,dim,page,layout", [
    (1, 8, 128, 16, "dense"), (1, 1, 64, 16, "fused"), (37, 3, 64, 32, "fused"), (50, 2, 128, 64, "head_major"),
    (129, 5, 128, 128, "dense"), (7, 1, 128, 1024, "dense")])
def test_append_bytes(cuda, fmt, four_six, dtype, tokens, heads, dim, page, layout):
    rng = np.random.default_rng(tokens + dim)
    f = FORMATS[fmt]
    pages = -(-tokens // page) + 3
    cache = sentinel_cache(pages, heads, page, dim, f, cuda)
    # outlier channels, exact zeros and lattice points (ties, equal four-over-six errors)
    x = rng.standard_normal((2, tokens, heads, dim)) * (1 + 30 * (rng.random(dim) < 0.02))
    x[:, ::3] = rng.integers(-48, 49, size=x[:, ::3].shape) / 8
    x[:, :, :, 3] = 0
    wide = torch.from_numpy(x.astype(np.float32)).to(dtype)
    if layout == "fused":
        both = torch.zeros(tokens, 4 * heads, dim, dtype=dtype)
        both[:, heads:2 * heads], both[:, 3 * heads:] = wide[0], wide[1]
        both = both.to(cuda)
        k, v = both[:, heads:2 * heads], both[:, 3 * heads:]
    elif layout == "head_major":
        k, v = (w.transpose(0, 1).contiguous().to(cuda).transpose(0, 1) for w in wide)
    else:
        k, v = wide[0].to(cuda), wide[1].to(cuda)
    slots = rng.permutation(pages * page)[:tokens].astype(np.int64)
    slots[1::5] = -1 - slots[1::5]          # skipped rows
    if tokens > 8:
        slots[6] = pages * page             # one past the end: skipped too
    sc = scales_for(f, cuda)
    fp4.fp4_kv_append(k, v, cache, torch.from_numpy(slots).to(cuda), f, four_six=four_six, **sc)
    torch.cuda.synchronize()
    for which, g in ((0, 0.0021), (1, 0.0016)):
        want_q = np.full((pages, heads, page, dim // 2), SENTINEL, np.uint8)
        want_s = np.full((pages, heads, page, dim // block_of(f)), SENTINEL, np.uint8)
        q, s = quantise(wide[which].float().numpy(), f, g, four_six)
        live = (slots >= 0) & (slots < pages * page)
        want_q[slots[live] // page, :, slots[live] % page] = q[live]
        want_s[slots[live] // page, :, slots[live] % page] = s[live]
        assert np.array_equal(cache[2 * which].cpu().numpy(), want_q)
        assert np.array_equal(cache[2 * which + 1].cpu().numpy(), want_s)


def test_append_mx_exponent_range(cuda):
    """Block maxima beyond the cache's exponents: the exponent is clamped to -23..13, the codes are
    those of that exponent."""
    exps = [-140, -126, -40, -25, -24, -22, -21, -20, 0, 14, 15, 16, 17, 40, 120]
    rng = np.random.default_rng(3)
    x = np.zeros((len(exps), 1, 64), dtype=np.float32)
    for i, e in enumerate(exps):
        x[i, 0] = np.ldexp(rng.uniform(-1, 1, 64), e).astype(np.float32)
    x[2, 0, 32:] = 0
    t = torch.from_numpy(x).to(cuda)
    cache = fp4.fp4_kv_alloc(1, 1, 16, 64, fp4.MXFP4, device=cuda)
    fp4.fp4_kv_append(t, t, cache, torch.arange(len(exps), device=cuda), fp4.MXFP4)
    q, s = cache[0].cpu().numpy()[0, 0], cache[1].cpu().numpy()[0, 0]
    for i in range(len(exps)):
        for blk in range(2):
            xb = x[i, 0, 32 * blk:32 * blk + 32]
            e = min(max(O.mx_exponent(float(np.abs(xb).max())), -23), 13)
            codes = O.mx_encode_block(xb, e)[0]
            assert s[i, blk] == e + 127
            packed = np.asarray(codes[0::2]) | (np.asarray(codes[1::2]) << 4)
            assert np.array_equal(q[i, 16 * blk:16 * blk + 16], packed)


def test_append_nothing(cuda):
    cache = sentinel_cache(1, 2, 16, 64, fp4.NVFP4, cuda)
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=cuda)
    fp4.fp4_kv_append(e, e, cache, torch.empty(0, dtype=torch.int64, device=cuda), **scales_for(fp4.NVFP4, cuda))
    assert all(bool((t == SENTINEL).all()) for t in cache)


# ---------------------------------------------------------------------------------------------
# read

@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,heads,dim,page", [([1], 1, 64, 16), ([517], 8, 128, 16), ([33, 0, 100, 1, 64], 3, 64, 32),
                                                 ([200, 129], 2, 128, 128)])
def test_read_values(cuda, fmt, dtype, lens, heads, dim, page):
    c = Cache(lens, heads, dim, page, FORMATS[fmt])
    starts = [min(3, n) for n in lens]
    rows = [n - s for n, s in zip(lens, starts)]
    cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    total = int(cu[-1])
    pad = 5
    outs = tuple(torch.full((total + pad, heads, dim), 7.0, dtype=dtype, device=cuda) for _ in range(2))
    fp4.fp4_kv_read(c.arrays, c.table, torch.from_numpy(cu).to(cuda), total + pad, c.fmt,
                    starts=torch.tensor(starts, dtype=torch.int32, device=cuda), out=outs, **c.scales)
    for which, g in ((0, c.k_global), (1, c.v_global)):
        assert bool((outs[which][total:] == 7.0).all())
        at = 0
        for b, n in enumerate(lens):
            t = np.arange(starts[b], n)
            pg = c.table_np[b, t // page]
            q, s = (c.arrays_np[2 * which + i][pg, :, t % page] for i in (0, 1))
            if len(t):
                want = O.dequantize(q.reshape(-1, dim // 2), s.reshape(len(t) * heads, -1), c.fmt, np.float32(g)).reshape(len(t), heads, dim)
                assert torch.equal(outs[which][at:at + len(t)].cpu(), torch.from_numpy(want).to(dtype))
            at += len(t)


def test_read_every_scale_byte(cuda):
    """All 256 scale bytes: the values fp4_dequantize gives (NaN where it gives NaN)."""
    for fmt in (fp4.NVFP4, fp4.MXFP4):
        nb = 64 // block_of(fmt)
        cache = fp4.fp4_kv_alloc(256 // nb, 1, 16, 64, fmt, device=cuda)
        sb = torch.arange(256, dtype=torch.uint8).view(-1, nb)
        cache[0][:, 0, 0] = torch.arange(32, dtype=torch.uint8).mul(0x37).to(cuda)
        cache[1][:, 0, 0] = sb.to(cuda)
        rows = cache[0].shape[0]
        table = torch.arange(rows, dtype=torch.int32, device=cuda)[:, None]
        sc = scales_for(fmt, cuda)
        k, _ = fp4.fp4_kv_read(cache, table, torch.arange(rows + 1, dtype=torch.int32, device=cuda), rows, fmt,
                               out_dtype=torch.float32, **sc)
        want = fp4.fp4_dequantize(cache[0][:, 0, 0].contiguous(), cache[1][:, 0, 0].contiguous(), fmt, sc.get("k_global"))
        assert torch.equal(k[:, 0].view(torch.int32), want.view(torch.int32)) or \
            torch.equal(torch.nan_to_num(k[:, 0], nan=1e30), torch.nan_to_num(want, nan=1e30))


def test_read_missing_pages_and_ranges(cuda):
    c = Cache([70], 2, 64, 16, fp4.NVFP4)
    table = c.table.clone()
    table[0, 1], table[0, 3] = -1, 10 ** 6
    cu = torch.tensor([0, 90], dtype=torch.int32, device=cuda)
    k, v = fp4.fp4_kv_read(c.arrays, table, cu, 90, starts=torch.tensor([-4], dtype=torch.int32, device=cuda),
                           out_dtype=torch.float32, **c.scales)
    want, _ = fp4.fp4_kv_read(c.arrays, c.table, torch.tensor([0, 70], dtype=torch.int32, device=cuda), 70,
                              out_dtype=torch.float32, **c.scales)
    t = np.arange(-4, 86)
    zero = (t < 0) | (t >= 80) | ((t >= 16) & (t < 32)) | ((t >= 48) & (t < 64))
    kk = k.cpu().numpy()
    assert (kk[zero] == 0).all() and (v.cpu().numpy()[zero] == 0).all()
    seen = ~zero & (t < 70)
    assert np.array_equal(kk[seen], want.cpu().numpy()[t[seen]])


def test_read_many_sequences(cuda):
    """More sequences than a block keeps offsets of, empty ones among them."""
    lens = [(7 * i) % 5 for i in range(1500)]
    c = Cache(lens, 1, 64, 16, fp4.MXFP4, seed=1)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=cuda)
    k, v = fp4.fp4_kv_read(c.arrays, c.table, cu, sum(lens), fp4.MXFP4, out_dtype=torch.float32)
    assert np.array_equal(k.cpu().numpy(), np.concatenate(c.k64)) and np.array_equal(v.cpu().numpy(), np.concatenate(c.v64))


# ---------------------------------------------------------------------------------------------
# attention

@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [1, 3, 8, 16])
@pytest.mark.parametrize("lens,page", [([1], 16), ([15, 16, 17], 16), ([300, 1, 0, 129], 32), ([64, 65, 1000], 64)])
def test_decode(cuda, fmt, dim, group, lens, page):
    c = Cache(lens, 2, dim, page, FORMATS[fmt], seed=group)
    run_and_check(c, [1] * len(lens), group, uniform=True)


@pytest.mark.parametrize("heads,group,lens", [(1, 8, [9000]), (8, 1, [40] * 70), (3, 7, [2500, 100, 1, 700]), (1, 1, [5000]),
                                              (2, 32, [1500]), (1, 71, [333, 20])])
def test_decode_splits(cuda, heads, group, lens):
    """One long sequence over many blocks, many short ones in few, ragged mixes."""
    c = Cache(lens, heads, 128, 64, fp4.NVFP4, seed=5)
    run_and_check(c, [1] * len(lens), group, strided=True)


@pytest.mark.parametrize("window", [1, 7, 64, 130, 5000])
@pytest.mark.parametrize("causal", [True, False])
def test_window(cuda, window, causal):
    c = Cache([700, 64, 33, 129], 2, 64, 16, fp4.MXFP4, seed=2)
    run_and_check(c, [1, 5, 33, 12], 4, causal=causal, window=window)


@pytest.mark.parametrize("fmt,dim,page", [("nvfp4", 128, 32), ("mxfp4", 64, 16), ("mxfp4", 128, 256), ("nvfp4", 64, 64)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("queries,lens,group", [
    ([2, 5, 1, 8], [100, 5, 77, 900], 4), ([17, 40], [300, 40], 1), ([129, 64, 1, 0], [129, 500, 200, 3], 5),
    ([257], [700], 8), ([31, 130], [31, 130], 16)])
def test_several_queries(cuda, fmt, dim, page, causal, queries, lens, group):
    c = Cache(lens, 2, dim, page, FORMATS[fmt], seed=9)
    run_and_check(c, queries, group, causal=causal, strided=True, pad_rows=3)


def test_long_prompt_rows(cuda):
    """A prompt longer than any tile, checked on every row."""
    c = Cache([1500], 1, 128, 64, fp4.NVFP4, seed=4)
    run_and_check(c, [1500], 2)
    run_and_check(c, [600], 3, window=200)


def test_more_queries_than_keys(cuda):
    """Queries before the first key see nothing: zeros and -inf."""
    c = Cache([5, 0, 40], 2, 64, 16, fp4.NVFP4)
    out, lse = run_and_check(c, [9, 3, 70], 4)
    assert bool((out[:4] == 0).all()) and bool(torch.isneginf(lse[:4]).all())
    assert bool((out[9:12] == 0).all()) and bool(torch.isneginf(lse[9:12]).all())


@pytest.mark.parametrize("queries", [1, 3, 40])
def test_missing_pages_are_not_seen(cuda, queries):
    """Entries outside the cache hold no tokens, wherever they sit; a sequence of nothing else is empty."""
    c = Cache([200, 90, 64], 2, 64, 16, fp4.NVFP4, seed=3)
    gone = [np.zeros(n, dtype=bool) for n in c.lens]
    table = c.table.clone()
    for b, p, bad in ((0, 0, -1), (0, 5, 10 ** 6), (0, 12, -7), (1, 5, -1), *((2, p, -1) for p in range(4))):
        table[b, p] = bad
        gone[b][16 * p:16 * p + 16] = True
    c.table = table
    out, lse = run_and_check(c, [queries] * 3, 4, gone=gone)
    assert bool((out[2 * queries:] == 0).all()) and bool(torch.isneginf(lse[2 * queries:]).all())


@pytest.mark.parametrize("queries", [1, 40])
def test_lengths_beyond_the_table(cuda, queries):
    """lens past the table's pages count as the table's; negative as none."""
    c = Cache([64, 64], 1, 64, 16, fp4.NVFP4, extra_cols=0)
    c.lens_t = torch.tensor([10 ** 6, -3], dtype=torch.int32, device="cuda")
    c.lens = [64, 0]
    c.k64[1], c.v64[1] = c.k64[1][:0], c.v64[1][:0]
    run_and_check(c, [queries] * 2, 4)


@pytest.mark.parametrize("queries", [1, 48])
@pytest.mark.parametrize("spread", [1e-6, 40.0])
def test_extreme_scores(cuda, queries, spread):
    """Almost uniform weights, and weights of almost one key (scores of thousands)."""
    c = Cache([777], 1, 128, 16, fp4.NVFP4, seed=6)
    run_and_check(c, [queries], 8, q_spread=spread)


@pytest.mark.parametrize("queries", [1, 48])
def test_query_range(cuda, queries):
    """Queries of very large and very small magnitude, within a row too: bf16 far outside fp16's range."""
    c = Cache([200], 1, 64, 16, fp4.NVFP4, seed=8)
    g = torch.Generator().manual_seed(1)
    q = torch.randn(queries, 4, 64, generator=g)
    q = q * torch.tensor([2.0 ** 100, 2.0 ** -100, 1.0, 1.0])[None, :, None]
    q[:, 2, ::2] *= 2.0 ** -20
    q = q.to(torch.bfloat16)
    for h, scale in ((0, 2.0 ** -103), (1, 2.0 ** 97), (2, 0.125), (3, -0.125)):
        out, lse = fp4.fp4_kv_attention(q[:, h:h + 1].to(cuda), c.arrays, c.table, c.lens_t, max_q=queries, scale=scale,
                                        want_lse=True, **c.scales)
        ref = attention64(q[:, h:h + 1].double().numpy(), c.k64[0], c.v64[0], scale, True, 0)
        check(out, lse, ref, 200, 64, np.abs(c.v64[0]).max())


@pytest.mark.parametrize("queries", [1, 48])
def test_zero_queries_and_zero_scale(cuda, queries):
    c = Cache([100], 1, 64, 16, fp4.MXFP4)
    run_and_check(c, [queries], 2, q_spread=0.0)
    run_and_check(c, [queries], 2, scale=0.0)


@pytest.mark.parametrize("queries", [1, 40, 90])
def test_nan_scale_bytes(cuda, queries):
    """The scale byte of a key as NaN: NaN in the rows that see the token and in no other.  Of a value
    block: as zero."""
    c = Cache([100, 100], 1, 64, 16, fp4.NVFP4)
    q = torch.randn(2 * queries, 4, 64, device=cuda).to(torch.bfloat16)
    sees = torch.arange(100 - queries, 100, device=cuda) >= 37

    def run(which, byte):
        arrays = [a.clone() for a in c.arrays]
        arrays[which][int(c.table_np[0, 2]), 0, 5, 1] = byte   # token 37 of sequence 0
        return fp4.fp4_kv_attention(q, arrays, c.table, c.lens_t, max_q=queries, want_lse=True, **c.scales)

    out, lse = run(1, 0x7F)
    assert bool(torch.isnan(out[:queries].float())[sees].all()) and bool(torch.isnan(lse[:queries][sees]).all())
    good, good_lse = run(1, 0x30)
    assert torch.equal(out[queries:], good[queries:]) and torch.equal(lse[queries:], good_lse[queries:])
    assert torch.equal(out[:queries][~sees], good[:queries][~sees])
    out, lse = run(3, 0x7F)
    good, good_lse = run(3, 0x00)
    assert torch.equal(out, good) and torch.equal(lse, good_lse)


def test_max_q_bounds_the_work(cuda):
    """Queries beyond max_q of a sequence are not computed; their rows stay."""
    c = Cache([50, 60], 1, 64, 16, fp4.NVFP4)
    q = torch.randn(9, 2, 64, device=cuda).to(torch.bfloat16)
    cu = torch.tensor([0, 6, 9], dtype=torch.int32, device=cuda)
    full, _ = fp4.fp4_kv_attention(q, c.arrays, c.table, c.lens_t, cu_q=cu, max_q=6, **c.scales)
    out = torch.full_like(full, 7.0)
    fp4.fp4_kv_attention(q, c.arrays, c.table, c.lens_t, cu_q=cu, max_q=4, out=out, **c.scales)
    assert bool((out[4:6] == 7.0).all()) and torch.equal(out[:4], full[:4]) and torch.equal(out[6:], full[6:])


# ---------------------------------------------------------------------------------------------
# the operators together, streams, graphs

def test_serving_loop(cuda):
    """A prompt in two chunks, then single tokens, each step append + attention, against the formula on
    what the cache reads back."""
    heads, group, dim, page, seqs = 2, 4, 64, 16, 3
    rng = torch.Generator(device=cuda).manual_seed(0)
    cache = sentinel_cache(40, heads, page, dim, fp4.NVFP4, cuda)
    table = torch.randperm(36, generator=rng, device=cuda).to(torch.int32).view(seqs, 12)
    sc = scales_for(fp4.NVFP4, cuda)
    lens = [0] * seqs
    for new in ([30, 1, 47], [50, 20, 3], [1, 1, 1], [1, 1, 1], [4, 1, 2]):
        total = sum(new)
        qkv = torch.randn(total, (group + 2) * heads, dim, generator=rng, device=cuda).to(torch.bfloat16)
        seq = np.repeat(np.arange(seqs), new)
        token = np.concatenate([np.arange(n, n + m) for n, m in zip(lens, new)])
        slots = table.cpu().numpy()[seq, token // page].astype(np.int64) * page + token % page
        fp4.fp4_kv_append(qkv[:, group * heads:(group + 1) * heads], qkv[:, (group + 1) * heads:], cache,
                          torch.from_numpy(slots).to(cuda), **sc)
        lens = [n + m for n, m in zip(lens, new)]
        cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=cuda)
        lt = torch.tensor(lens, dtype=torch.int32, device=cuda)
        out, lse = fp4.fp4_kv_attention(qkv[:, :group * heads], cache, table, lt, cu_q=cu, max_q=max(new), want_lse=True, **sc)
        ck = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=cuda)
        k, v = fp4.fp4_kv_read(cache, table, ck, sum(lens), out_dtype=torch.float32, **sc)
        at = ak = 0
        for n, m in zip(lens, new):
            kk, vv = k[ak:ak + n].cpu().double().numpy(), v[ak:ak + n].cpu().double().numpy()
            ref = attention64(qkv[at:at + m, :group * heads].cpu().double().numpy(), kk, vv, dim ** -0.5, True, 0)
            check(out[at:at + m], lse[at:at + m], ref, n, dim, np.abs(vv).max())
            at, ak = at + m, ak + n


def _decode_case(cuda, seed, lens, page=16):
    c = Cache(lens, 2, 128, page, fp4.NVFP4, seed=seed)
    q = torch.randn(len(lens), 8, 128, device=cuda, generator=torch.Generator(device=cuda).manual_seed(seed)).to(torch.bfloat16)
    return c, q


def test_other_stream_and_repeatability(cuda):
    c, q = _decode_case(cuda, 1, [3000, 17, 900])
    want, lse = fp4.fp4_kv_attention(q, c.arrays, c.table, c.lens_t, want_lse=True, **c.scales)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        out, l2 = fp4.fp4_kv_attention(q, c.arrays, c.table, c.lens_t, want_lse=True, stream=side, **c.scales)
        side.synchronize()
        assert torch.equal(out, want) and torch.equal(l2, lse)


def test_graphs_replay_with_new_lengths(cuda):
    """Two captured decode steps, replayed at once on two streams with lengths changed after capture."""
    cases = [_decode_case(cuda, s, [2000, 64, 700]) for s in (1, 2)]
    graphs, outs = [], []
    for c, q in cases:
        fp4.fp4_kv_attention(q, c.arrays, c.table, c.lens_t, **c.scales)
    torch.cuda.synchronize()
    for c, q in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fp4.fp4_kv_attention(q, c.arrays, c.table, c.lens_t, **c.scales)[0])
        graphs.append(g)
    new = [1500, 3, 699]
    for c, _ in cases:
        c.lens_t.copy_(torch.tensor(new, dtype=torch.int32))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (c, q), out in zip(cases, outs):
        want, _ = fp4.fp4_kv_attention(q, c.arrays, c.table, c.lens_t, **c.scales)
        assert torch.equal(out, want)


def test_offsets_beyond_32_bits(cuda):
    """A cache of more than 2^32 bytes an array: pages at both ends give the same rows."""
    heads, page, dim = 8, 1024, 128
    pages = (2 ** 32) // (heads * page * (dim // 2)) + 2
    cache = tuple(torch.empty((pages, heads, page, n), dtype=torch.uint8, device=cuda) for n in (64, 8, 64, 8))
    sc = scales_for(fp4.NVFP4, cuda)
    x = torch.randn(2, 20, heads, dim, device=cuda).to(torch.bfloat16)
    tables = {}
    for name, p in (("low", 0), ("high", pages - 1)):
        slots = torch.arange(20, device=cuda) + p * page
        fp4.fp4_kv_append(x[0], x[1], cache, slots, **sc)
        tables[name] = torch.tensor([[p]], dtype=torch.int32, device=cuda)
    q = torch.randn(20, 16, dim, device=cuda).to(torch.bfloat16)
    n = torch.tensor([20], dtype=torch.int32, device=cuda)
    cu = torch.tensor([0, 20], dtype=torch.int32, device=cuda)
    for m in (1, 20):
        a, b = (fp4.fp4_kv_attention(q[:m], cache, t, n, max_q=m, **sc)[0] for t in tables.values())
        assert torch.equal(a, b) and bool(torch.isfinite(a.float()).all())
    a, b = (fp4.fp4_kv_read(cache, t, cu, 20, **sc)[0] for t in tables.values())
    assert torch.equal(a, b)
    want, _ = quantise(x[0].float().cpu().numpy(), fp4.NVFP4, 0.0021)
    assert np.array_equal(cache[0][pages - 1, :, :20].transpose(0, 1).cpu().numpy(), want)


# ---------------------------------------------------------------------------------------------
# calls at the edges of the kernels' rules

@pytest.mark.parametrize("queries,group,heads,length", [
    (16, 1, 2, 300), (17, 1, 2, 300), (6, 4, 1, 1000), (8, 4, 1, 129), (33, 1, 1, 5000), (16, 8, 1, 6000),   # rows 16 .. 128
    (43, 3, 2, 400), (64, 4, 1, 200), (257, 1, 1, 260), (40, 13, 1, 3000)])                                  # and past
def test_row_counts(cuda, queries, group, heads, length):
    """Rows a head on both sides of every kernel's limit, one to many splits of the keys."""
    for fmt, dim in ((fp4.NVFP4, 128), (fp4.MXFP4, 64)):
        c = Cache([length], heads, dim, 16, fmt, seed=queries)
        run_and_check(c, [queries], group)
        run_and_check(c, [queries], group, window=length // 3 + 1)


@pytest.mark.parametrize("queries", [1, 4, 40])
def test_sequences_without_queries_or_keys(cuda, queries):
    c = Cache([300, 0, 77, 500, 12, 0], 2, 64, 16, fp4.NVFP4, seed=2)
    run_and_check(c, [queries, 1, 0, queries, 0, 0], 4)
    run_and_check(c, [0, 0, 0, queries, 0, 0], 4)


@pytest.mark.parametrize("seqs,heads,long", [(90, 8, 3000), (300, 2, 700), (300, 1, 2000), (600, 1, 90)])
def test_many_sequences(cuda, seqs, heads, long):
    """More units than resident blocks, and more sequences than one schedule holds."""
    lens = [long] + [(37 * i) % 60 for i in range(1, seqs)]
    c = Cache(lens, heads, 64, 16, fp4.NVFP4, seed=3)
    run_and_check(c, [1] * seqs, 2)


def test_many_sequences_of_many_rows(cuda):
    lens = [150 + (37 * i) % 60 for i in range(70)]
    c = Cache(lens, 1, 64, 16, fp4.MXFP4, seed=3)
    run_and_check(c, [20 + i % 30 for i in range(70)], 2)


@pytest.mark.parametrize("queries", [1, 12, 48])
def test_layouts(cuda, queries):
    """Head-major queries, a block table that is a slice of a wider one, one head of many."""
    c = Cache([130, 61], 2, 128, 16, fp4.NVFP4, seed=5)
    q = torch.randn(2 * queries, 8, 128, device=cuda).to(torch.bfloat16)
    want, lse = fp4.fp4_kv_attention(q, c.arrays, c.table, c.lens_t, max_q=queries, want_lse=True, **c.scales)
    head_major = q.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.full((2, c.table.shape[1] + 7), -1, dtype=torch.int32, device=cuda)
    wide[:, :c.table.shape[1]] = c.table
    out, l2 = fp4.fp4_kv_attention(head_major, c.arrays, wide[:, :c.table.shape[1]], c.lens_t, max_q=queries, want_lse=True,
                                   workspace=torch.full((fp4.workspace_size(fp4.OP_KV_ATTENTION),), 0xFF, dtype=torch.uint8, device=cuda),
                                   **c.scales)
    assert torch.equal(out, want) and torch.equal(l2, lse)


def test_mx_scale_bytes_outside_the_cache_range(cuda):
    """Bytes 0..103 count as 104 in attention, 141..255 as 140."""
    c = Cache([40], 1, 64, 16, fp4.MXFP4)
    q = torch.randn(1, 4, 64, device=cuda).to(torch.bfloat16)
    for which in (1, 3):
        got = []
        for byte in (0, 104, 140, 200, 255):
            arrays = [a.clone() for a in c.arrays]
            arrays[which][int(c.table_np[0, 1]), 0, 3, 0] = byte
            got.append(torch.cat([fp4.fp4_kv_attention(q.expand(m, 4, 64).contiguous(), arrays, c.table, c.lens_t, fp4.MXFP4, max_q=m)[0] for m in (1, 40)]))
        assert torch.equal(got[0], got[1]) and torch.equal(got[2], got[3]) and torch.equal(got[2], got[4])


def test_two_calls_at_once(cuda):
    """Two streams, each with calls of its own (workspaces of the binding's making)."""
    cases = [_decode_case(cuda, s, [2500, 64, 700]) for s in (3, 4)]
    want = [fp4.fp4_kv_attention(q, c.arrays, c.table, c.lens_t, **c.scales)[0] for c, q in cases]
    prompts = [torch.randn(3 * 50, 8, 128, device=cuda).to(torch.bfloat16) for _ in cases]
    pwant = [fp4.fp4_kv_attention(q, c.arrays, c.table, c.lens_t, max_q=50, **c.scales)[0] for (c, _), q in zip(cases, prompts)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got, pgot = [], []
    for _ in range(4):
        for s, (c, q), pq in zip(streams, cases, prompts):
            got.append(fp4.fp4_kv_attention(q, c.arrays, c.table, c.lens_t, stream=s, **c.scales)[0])
            pgot.append(fp4.fp4_kv_attention(pq, c.arrays, c.table, c.lens_t, max_q=50, stream=s, **c.scales)[0])
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(got, pgot)):
        assert torch.equal(a, want[i % 2]) and torch.equal(b, pwant[i % 2])


def test_prompt_graph_and_append_in_it(cuda):
    """A captured step of append and attention, single tokens and a chunk, replayed on new inputs."""
    sc = scales_for(fp4.NVFP4, cuda)
    cache = sentinel_cache(20, 2, 16, 128, fp4.NVFP4, cuda)
    table = torch.arange(20, dtype=torch.int32, device=cuda).view(2, 10)
    for new in (1, 24):
        qkv = torch.zeros(2 * new, 12, 128, dtype=torch.bfloat16, device=cuda)
        slots = torch.zeros(2 * new, dtype=torch.int64, device=cuda)
        lens = torch.zeros(2, dtype=torch.int32, device=cuda)

        def step():
            fp4.fp4_kv_append(qkv[:, 8:10], qkv[:, 10:], cache, slots, **sc)
            return fp4.fp4_kv_attention(qkv[:, :8], cache, table, lens, max_q=new, **sc)[0]

        def fill(past):
            qkv.copy_(torch.randn(2 * new, 12, 128, device=cuda))
            pos = torch.arange(past, past + new, device=cuda)
            slots.copy_(torch.cat([table[b].long()[pos // 16] * 16 + pos % 16 for b in range(2)]))
            lens.fill_(past + new)

        fill(0)
        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        for past in (0, new, 2 * new):
            fill(past)
            g.replay()
            torch.cuda.synchronize()
            got = out.clone()
            assert torch.equal(step(), got)


def test_wait_limit_reports_and_recovers(cuda):
    """A limit of 0 ns makes the many-row kernel's first unfinished wait give up: the status word says so,
    the call returns, and the next call is right."""
    c = Cache([700], 1, 128, 16, fp4.NVFP4)
    q = torch.randn(300, 4, 128, device=cuda).to(torch.bfloat16)
    ws = torch.zeros(fp4.workspace_size(fp4.OP_KV_ATTENTION), dtype=torch.uint8, device=cuda)
    old = fp4.set_gemm_wait_limit(0)
    try:
        fp4.fp4_kv_attention(q, c.arrays, c.table, c.lens_t, max_q=300, workspace=ws, **c.scales)
        torch.cuda.synchronize()
    finally:
        fp4.set_gemm_wait_limit(old)
    assert int(ws[:4].view(torch.int32)) != 0
    want, _ = fp4.fp4_kv_attention(q, c.arrays, c.table, c.lens_t, max_q=300, workspace=ws, **c.scales)
    assert int(ws[:4].view(torch.int32)) == 0
    run_and_check(c, [300], 4)
    assert bool(torch.isfinite(want.float()).all())


def test_binding_refusals(cuda):
    c = Cache([40], 2, 64, 16, fp4.NVFP4)
    q = torch.randn(1, 4, 64, device=cuda).to(torch.bfloat16)
    k = torch.randn(3, 2, 64, device=cuda).to(torch.bfloat16)
    slots = torch.arange(3, device=cuda)

    def attend(**kw):
        a = dict(q=q, cache=c.arrays, table=c.table, lens=c.lens_t, **c.scales)
        a.update(kw)
        return fp4.fp4_kv_attention(a.pop("q"), a.pop("cache"), a.pop("table"), a.pop("lens"), **a)

    for err, kw in [(TypeError, dict(q=q.half())), (fp4.Fp4Error, dict(q=q.float())), (ValueError, dict(q=q[..., :32])),
                    (ValueError, dict(q=q.cpu())), (ValueError, dict(q=q.expand(2, 1, 4, 64))), (fp4.Fp4Error, dict(q=q[:, :3])),
                    (ValueError, dict(table=c.table.long())), (ValueError, dict(table=c.table[:, ::2])), (ValueError, dict(lens=c.lens_t.cpu())),
                    (ValueError, dict(lens=c.lens_t.long())), (ValueError, dict(cu_q=c.lens_t, max_q=1)),
                    (ValueError, dict(cu_q=torch.tensor([0, 1], dtype=torch.int32, device=cuda))), (fp4.Fp4Error, dict(max_q=2)),
                    (fp4.Fp4Error, dict(scale=float("nan"))), (ValueError, dict(out=torch.empty_like(q).float())),
                    (fp4.Fp4Error, dict(workspace=torch.empty(16, dtype=torch.uint8, device=cuda))), (fp4.Fp4Error, dict(k_global=None)),
                    (ValueError, dict(k_global=torch.ones(2, device=cuda))), (ValueError, dict(cache=c.arrays[:3] + (c.arrays[3][:1],))),
                    (ValueError, dict(fmt=fp4.MXFP4)), (fp4.Fp4Error, dict(fmt=fp4.IF4)), (TypeError, dict(window=1.5)),
                    (ValueError, dict(max_q=2 ** 40)), (TypeError, dict(lens=[40]))]:
        with pytest.raises(err):
            attend(**kw)
    for err, args in [(ValueError, (k, k.float(), c.arrays, slots)), (ValueError, (k, k[:2], c.arrays, slots)), (TypeError, (k.half(), k.half(), c.arrays, slots)),
                      (ValueError, (k, k, c.arrays, slots.int())), (ValueError, (k, k, c.arrays, slots[:2])), (ValueError, (k[:, :1], k[:, :1], c.arrays, slots)),
                      (ValueError, (k.transpose(1, 2).contiguous().transpose(1, 2), k, c.arrays, slots))]:
        with pytest.raises(err):
            fp4.fp4_kv_append(*args, **c.scales)
    with pytest.raises(fp4.Fp4Error):   # rows that start off a 32-byte boundary
        odd = torch.randn(3, 2 * 64 + 4, device=cuda).to(torch.bfloat16)[:, 4:].unflatten(1, (2, 64))
        fp4.fp4_kv_append(odd, k, c.arrays, slots, **c.scales)
    cu = torch.tensor([0, 40], dtype=torch.int32, device=cuda)
    for err, kw in [(ValueError, dict(cu=cu.long())), (ValueError, dict(starts=cu)), (TypeError, dict(out_dtype=torch.float16)),
                    (ValueError, dict(out=(torch.empty(40, 2, 64, device=cuda),) * 1 + (torch.empty(39, 2, 64, device=cuda),)))]:
        a = dict(cu=cu)
        a.update(kw)
        with pytest.raises(err):
            fp4.fp4_kv_read(c.arrays, c.table, a.pop("cu"), 40, **a, **c.scales)


# Rows, steps and units of the many-row kernel: two row tiles or one, keys split over blocks or not.
@pytest.mark.parametrize("queries,length", [(300, 700), (300, 6000), (20, 700), (20, 6000)])
def test_a_lost_wait_shows_in_the_output(cuda, queries, length):
    """Without a workspace of the caller's nobody can read the status word: rows of a block that gave up are
    NaN, all others right.  With one, its status word says so, and the next call on it is right."""
    c = Cache([length], 1, 128, 16, fp4.NVFP4)
    q = torch.randn(queries, 4, 128, device=cuda).to(torch.bfloat16)
    call = lambda **kw: fp4.fp4_kv_attention(q, c.arrays, c.table, c.lens_t, max_q=queries, want_lse=True, **kw, **c.scales)  # noqa: E731
    want, want_lse = call()
    ws = torch.zeros(fp4.workspace_size(fp4.OP_KV_ATTENTION), dtype=torch.uint8, device=cuda)
    got = []
    torch.cuda.synchronize()
    old = fp4.set_gemm_wait_limit(0)
    try:
        for kw in (dict(), dict(workspace=ws)):
            got.append(call(out=torch.full_like(want, 7.0), **kw))
            torch.cuda.synchronize()
    finally:
        fp4.set_gemm_wait_limit(old)
    assert int(ws[:4].view(torch.int32)) != 0
    for out, lse in got:
        right = (out == want).all(-1) & (lse == want_lse)
        lost = out.isnan().all(-1) & lse.isnan()
        assert bool(lost.any()) and bool((right | lost).all())
    run_and_check(c, [queries], 4, workspace=ws)
    assert int(ws[:4].view(torch.int32)) == 0


@pytest.mark.parametrize("group", [2, 12, 20, 32])
def test_units_cut_in_two_schedules(cuda, group):
    """More than 256 sequences, more units than blocks and a wide table: long units at both ends of both
    schedules are cut, and joined from the records of each block."""
    lens = [(37 * i) % 60 for i in range(300)]
    for b in (0, 75, 149, 150, 220, 299):
        lens[b] = 2500 - 3 * b
    c = Cache(lens, 3, 64, 16, fp4.MXFP4, seed=4)
    run_and_check(c, [1] * 300, group)


@pytest.mark.parametrize("queries", [1, 40])
def test_many_heads(cuda, queries):
    c = Cache([150, 20, 0], 40, 64, 16, fp4.NVFP4, seed=6)
    run_and_check(c, [queries] * 3, 1, strided=True)


@pytest.mark.parametrize("queries", [1, 40])
def test_value_scale_bytes_with_a_sign(cuda, queries):
    """fp4_kv_append writes no scale byte with its sign bit set: attention counts one of a value block as
    zero, one of a key block has its sign."""
    c = Cache([40], 1, 64, 16, fp4.NVFP4)
    q = torch.randn(queries, 4, 64, device=cuda).to(torch.bfloat16)
    at = int(c.table_np[0, 1]), 0, 3, 0

    def run(which, change):
        arrays = [a.clone() for a in c.arrays]
        change(arrays[which], arrays[which - 1])
        return fp4.fp4_kv_attention(q, arrays, c.table, c.lens_t, max_q=queries, **c.scales)[0]

    sign = lambda s, _: s.__setitem__(at, s[at] | 0x80)               # noqa: E731
    zero = lambda s, _: s.__setitem__(at, 0)                          # noqa: E731
    flip = lambda _, n: n[at[:3]][:8].bitwise_xor_(0x88)              # noqa: E731
    assert torch.equal(run(3, sign), run(3, zero))
    assert torch.equal(run(1, sign), run(1, flip))


@pytest.mark.parametrize("queries", [1, 48])
def test_queries_near_the_smallest_numbers(cuda, queries):
    """Rows that no power of two of fp32 brings to fp16's upper end, subnormals among them: exact all the same."""
    c = Cache([200], 1, 64, 16, fp4.NVFP4, seed=8)
    q = (torch.randn(queries, 4, 64, generator=torch.Generator().manual_seed(2)) * 2.0 ** -124).to(torch.bfloat16)
    out, lse = fp4.fp4_kv_attention(q.to(cuda), c.arrays, c.table, c.lens_t, max_q=queries, scale=2.0 ** 122, want_lse=True, **c.scales)
    ref = attention64(q.double().numpy(), c.k64[0], c.v64[0], 2.0 ** 122, True, 0)
    check(out, lse, ref, 200, 64, np.abs(c.v64[0]).max())


@pytest.mark.parametrize("queries", [1, 48])
@pytest.mark.parametrize("size,scale", [(2.0 ** 120, 2.0 ** -122), (2.0 ** -126, 1.75 * 2.0 ** 127)])
def test_scales_of_very_large_and_small_queries(cuda, queries, size, scale):
    """Scales whose product with the base's logarithm or the keys' scale alone leaves fp32's normal numbers."""
    c = Cache([200], 1, 64, 16, fp4.NVFP4, seed=8)
    q = (torch.randn(queries, 4, 64, generator=torch.Generator().manual_seed(2)) * size).to(torch.bfloat16)
    q[queries // 2, 1] = 0
    out, lse = fp4.fp4_kv_attention(q.to(cuda), c.arrays, c.table, c.lens_t, max_q=queries, scale=scale, want_lse=True, **c.scales)
    ref = attention64(q.double().numpy(), c.k64[0], c.v64[0], scale, True, 0)
    check(out, lse, ref, 200, 64, np.abs(c.v64[0]).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_mx_maxima_at_powers_of_two(cuda, dtype):
    """Block maxima that are powers of two, and the numbers next to them: the oracle's bytes."""
    rng = np.random.default_rng(5)
    exps = np.arange(-20, 14)
    x = rng.uniform(-0.9, 0.9, (len(exps), 3, 64)).astype(np.float32)
    step = np.float32(torch.finfo(dtype).eps)
    x[:, 0, ::32], x[:, 1, ::32], x[:, 2, ::32] = 1, 1 - step / 2, -1 - step
    t = torch.from_numpy(np.ldexp(x, exps[:, None, None]).astype(np.float32)).to(dtype)
    assert torch.equal(t[:, :, 0].double(), torch.from_numpy(np.ldexp(x[:, :, 0].astype(np.float64), exps[:, None])))
    cache = fp4.fp4_kv_alloc(3, 3, 16, 64, fp4.MXFP4, device=cuda)
    fp4.fp4_kv_append(t.to(cuda), t.to(cuda), cache, torch.arange(len(exps), device=cuda), fp4.MXFP4)
    q, s = quantise(t.float().numpy(), fp4.MXFP4, 1.0)
    for got, want in zip(cache, (q, s, q, s)):
        assert np.array_equal(got.transpose(1, 2).reshape(48, 3, -1)[:len(exps)].cpu().numpy(), want)
