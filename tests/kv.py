"""Helpers of the key/value cache tests: caches built on the host from the oracle's bytes, and the
attention formula in 64 bits."""
from __future__ import annotations

import numpy as np
import torch

import block_scaled_fp4_amax_b200 as fp4
import oracle as O

FORMATS = {"nvfp4": fp4.NVFP4, "mxfp4": fp4.MXFP4}


def block_of(fmt):
    return 16 if fmt == fp4.NVFP4 else 32


def quantise(x, fmt, s_g, four_six=False):
    """x [..., D] fp32 (MXFP4: block maxima inside the cache's exponent range) -> oracle bytes."""
    d = x.shape[-1]
    flat = np.ascontiguousarray(x.reshape(-1, d), dtype=np.float32)
    if fmt == fp4.NVFP4:
        q, s, _, _ = O.nvfp4_quantize(flat, four_six=four_six, global_in=s_g)
    else:
        q, s, _ = O.mx_quantize(flat)
    return q.reshape(*x.shape[:-1], d // 2), s.reshape(*x.shape[:-1], d // block_of(fmt))


def values64(q, s, fmt, s_g):
    d = 2 * q.shape[-1]
    v = O.dequantize_f64(q.reshape(-1, d // 2), s.reshape(-1, s.shape[-1]), fmt, s_g)
    return np.asarray(v, dtype=np.float64).reshape(*q.shape[:-1], d)


class Cache:
    """A paged cache of random tokens: pages in shuffled order, a block table padded with -1, every byte
    that no token owns set to `stale` (0xFF reads as NaN)."""

    def __init__(self, lens, heads, dim, page, fmt, seed=0, extra_pages=2, extra_cols=1, stale=0xFF, spread=1.0, device="cuda"):
        rng = np.random.default_rng(seed)
        self.fmt, self.page, self.heads, self.dim, self.lens = fmt, page, heads, dim, list(lens)
        used = [-(-n // page) for n in lens]
        pages = sum(used) + extra_pages
        order = rng.permutation(pages)
        cols = max(used + [0]) + extra_cols
        table = np.full((len(lens), cols), -1, dtype=np.int32)
        nb = dim // block_of(fmt)
        arrays = [np.full((pages, heads, page, n), stale, dtype=np.uint8) for n in (dim // 2, nb, dim // 2, nb)]
        self.k_global, self.v_global = (0.0021, 0.0016) if fmt == fp4.NVFP4 else (1.0, 1.0)
        self.k64, self.v64 = [], []
        at = 0
        for b, n in enumerate(lens):
            table[b, :used[b]] = order[at:at + used[b]]
            at += used[b]
            for which, (g, dense) in enumerate(((self.k_global, self.k64), (self.v_global, self.v64))):
                x = (rng.standard_normal((n, heads, dim)) * spread * (1 + which)).astype(np.float32)
                q, s = quantise(x, fmt, g) if n else (np.zeros((0, heads, dim // 2), np.uint8), np.zeros((0, heads, nb), np.uint8))
                t = np.arange(n)
                pg, off = table[b, t // page], t % page
                arrays[2 * which][pg, :, off] = q
                arrays[2 * which + 1][pg, :, off] = s
                dense.append(values64(q, s, fmt, g) if n else np.zeros((0, heads, dim)))
        self.table_np, self.arrays_np = table, arrays
        self.table = torch.from_numpy(table).to(device)
        self.arrays = tuple(torch.from_numpy(a).to(device) for a in arrays)
        self.lens_t = torch.tensor(self.lens, dtype=torch.int32, device=device)
        self.scales = {}
        if fmt == fp4.NVFP4:
            self.scales = {n: torch.tensor([g], dtype=torch.float32, device=device)
                           for n, g in (("k_global", self.k_global), ("v_global", self.v_global))}
            # the fp32 scale is what the cache's values stand for
            f = np.float64(np.float32(self.k_global)), np.float64(np.float32(self.v_global))
            self.k64 = [k * (f[0] / self.k_global) for k in self.k64]
            self.v64 = [v * (f[1] / self.v_global) for v in self.v64]


def attention64(q, k, v, scale, causal, window, gone=None):
    """One sequence: q [m, Hq, D], k, v [n, H, D] in fp64 -> out, lse, and per row the quantities the
    error bound needs: A = sum p |v| per channel and the largest sum |q k| of a visible key.  `gone`:
    bool [n], keys without a page."""
    m, hq, d = q.shape
    n, h = k.shape[:2]
    g = hq // h
    out, lse = np.zeros((m, hq, d)), np.full((m, hq), -np.inf)
    A, sabs = np.zeros((m, hq, d)), np.zeros((m, hq))
    pos = np.arange(n - m, n)[:, None]
    j = np.arange(n)[None]
    keep = np.ones((m, n), dtype=bool)
    if causal:
        keep &= j <= pos
    if window:
        keep &= j > pos - window
    if gone is not None:
        keep &= ~gone[None]
    any_key = keep.any(1)
    if n == 0 or not any_key.any():
        return out, lse, A, sabs
    for x in range(hq):
        kk, vv = k[:, x // g], v[:, x // g]
        s = np.where(keep, q[:, x] @ kk.T * scale, -np.inf)
        top = np.where(any_key, s.max(1, initial=-np.inf), 0.0)[:, None]
        p = np.exp(s - top)
        tot = p.sum(1, keepdims=True)
        with np.errstate(divide="ignore", invalid="ignore"):
            lse[:, x] = (top + np.log(tot))[:, 0]
            out[:, x] = np.where(any_key[:, None], p @ vv / tot, 0.0)
            A[:, x] = np.where(any_key[:, None], p @ np.abs(vv) / tot, 0.0)
        sabs[:, x] = np.where(keep, np.abs(q[:, x]) @ np.abs(kk).T, 0.0).max(1) * abs(scale)
    return out, lse, A, sabs


def check(out, lse, ref, n, dim, vmax):
    """The error a row may have, from the roundings the documentation names.
    Scores: dim products summed in fp32, each partial sum off by 2^-23 of the sum of magnitudes
    (tensor cores may truncate), and a few further roundings: ds = (dim + 8) 2^-23 sum |q k| scale.
    Weights: e^ds, 2^-11 from fp16, 2^-22 from the exponential.  A row's largest weight is written as at
    least 2^7, so a weight below 2^-21 of it is an fp16 subnormal, off by half their step: 2^-24 / 2 /
    2^7 = 2^-32 of the largest, which is at most the sum of all: n 2^-32 of the largest |v| for n
    keys.  Sums over n keys: (n + 16) 2^-23.  Output: bf16, 2^-8."""
    o64, l64, A, sabs = ref
    ds = (dim + 8) * 2.0 ** -23 * sabs
    o = out.float().cpu().numpy().astype(np.float64)
    bound = 2.0 ** -8 * np.abs(o64) + A * (2.0 ** -11 + 2 * ds[..., None] + (n + 16) * 2.0 ** -23) * (1 + 2.0 ** -8) \
        + n * 2.0 ** -32 * vmax
    err = np.abs(o - o64)
    assert np.isfinite(o).all()
    assert (err <= bound).all(), f"{(err > bound).sum()} of {err.size} outside; worst ratio {np.nanmax(err / np.maximum(bound, 1e-300)):.3f}"
    if lse is not None:
        got = lse.cpu().numpy().astype(np.float64)
        empty = np.isneginf(l64)
        assert np.array_equal(np.isneginf(got), empty)
        lb = 2 * ds + (n + 16) * 2.0 ** -23 + 2.0 ** -22 * np.abs(np.where(empty, 0, l64))
        le = np.abs(np.where(empty, 0, got) - np.where(empty, 0, l64))
        assert (le <= lb).all(), f"lse: worst ratio {np.max(le / np.maximum(lb, 1e-300)):.3f}"


def run_and_check(c: Cache, queries, group, causal=True, window=0, scale=None, seed=1, uniform=False, q_spread=1.0,
                  strided=False, pad_rows=0, gone=None, device="cuda", **kw):
    """fp4_kv_attention over the cache against the formula, sequence by sequence."""
    rng = np.random.default_rng(seed)
    hq, total = c.heads * group, sum(queries)
    scale = c.dim ** -0.5 if scale is None else scale
    wide = torch.from_numpy((rng.standard_normal((total + pad_rows, hq + 2 * c.heads, c.dim)) * q_spread).astype(np.float32)).to(torch.bfloat16)
    wide = wide.to(device)
    q = wide[:, c.heads:c.heads + hq]
    if not strided:
        q = q.contiguous()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(queries)]), dtype=torch.int32, device=device)
    out = torch.full((total + pad_rows, hq, c.dim), 7.0, dtype=torch.bfloat16, device=device)
    _, lse = fp4.fp4_kv_attention(q, c.arrays, c.table, c.lens_t, c.fmt, cu_q=None if uniform else cu, max_q=max(queries),
                                  scale=scale, causal=causal, window=window, want_lse=True, out=out, **c.scales, **kw)
    torch.cuda.synchronize()
    assert bool((out[total:] == 7.0).all())
    qd = q.cpu().double().numpy()
    at = 0
    for b, m in enumerate(queries):
        n = c.lens[b]
        ref = attention64(qd[at:at + m], c.k64[b], c.v64[b], scale, causal, window, None if gone is None else gone[b])
        check(out[at:at + m], lse[at:at + m], ref, n, c.dim, np.abs(c.v64[b]).max(initial=0.0))
        at += m
    return out, lse
