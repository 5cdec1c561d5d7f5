"""The 4-bit key/value cache: cases to measure, plain forms and 64-bit values.

Three operators: writing keys and values into a paged cache as they are quantised (followed by the
read of what was written, so that the outputs are the values the cache stands for), reading a cache
back, and attention over it.  `run` computes them in elementary torch operations where `own` is
false, and calls the library where it is true.
"""
import functools
import math
import operator

import numpy as np
import torch

own = False

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one new token for each of 64 sequences, keys and values sliced out of a fused projection
        dict(name="write_step_64", op="write", seqs=64, new=1, past=900, heads=8, dim=128, page=16, fmt="nvfp4",
             four_six=False, dtype="bf16", fused=True),
        # prompt chunks of four sequences under four-over-six
        dict(name="write_chunk_4x2048", op="write", seqs=4, new=2048, past=77, heads=8, dim=128, page=64, fmt="nvfp4",
             four_six=True, dtype="bf16", fused=True),
        # fp32 keys and values of a small model, MXFP4
        dict(name="write_f32_mx_3x1365", op="write", seqs=3, new=1365, past=5, heads=4, dim=64, page=32, fmt="mxfp4",
             four_six=False, dtype="f32", fused=False),
        # a short shared prefix brought back for a prefill in bf16
        dict(name="read_1x517", op="read", seqs=1, length=517, heads=8, dim=128, page=16, fmt="nvfp4", dtype="bf16"),
        # a batch of long caches moved out in fp32
        dict(name="read_mx_16x8192", op="read", seqs=16, length=8192, heads=8, dim=128, page=64, fmt="mxfp4", dtype="f32"),
        # one chat just begun: latency
        dict(name="decode_1x300", op="attend", seqs=1, q_len=1, length=300, q_heads=32, heads=8, dim=128, page=16,
             fmt="nvfp4", causal=True, window=0),
        # a full serving batch of ragged lengths
        dict(name="decode_64x8192", op="attend", seqs=64, q_len=1, length=8192, q_heads=64, heads=8, dim=128, page=64,
             fmt="nvfp4", causal=True, window=0),
        # one very long document
        dict(name="decode_1x131072", op="attend", seqs=1, q_len=1, length=131072, q_heads=64, heads=8, dim=128, page=64,
             fmt="nvfp4", causal=True, window=0),
        # sliding-window layers of a small model, an odd group of query heads
        dict(name="decode_mx_window_48x4099", op="attend", seqs=48, q_len=1, length=4099, q_heads=28, heads=4, dim=64,
             page=16, fmt="mxfp4", causal=True, window=1024),
        # verification of drafted tokens
        dict(name="verify_16x5x6001", op="attend", seqs=16, q_len=5, length=6001, q_heads=32, heads=8, dim=128, page=32,
             fmt="nvfp4", causal=True, window=0),
        # a chunk of two prompts after a long past
        dict(name="chunk_2x1024x16384", op="attend", seqs=2, q_len=1024, length=16384, q_heads=64, heads=8, dim=128,
             page=64, fmt="nvfp4", causal=True, window=0),
        # a whole prompt
        dict(name="prompt_1x8192", op="attend", seqs=1, q_len=8192, length=8192, q_heads=32, heads=8, dim=128, page=64,
             fmt="nvfp4", causal=True, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    fmt = rng.choice(["nvfp4", "nvfp4", "mxfp4"])
    dim = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    heads = rng.choice([1, 2, 4, 8])
    op = rng.choice(["write", "read", "attend", "attend", "attend"])
    if op == "write":
        seqs = _log(rng, 1, 96)
        return dict(op="write", seqs=seqs, new=_log(rng, 1, max(1, 8192 // seqs)), past=rng.randrange(0, 2000), heads=heads,
                    dim=dim, page=page, fmt=fmt, four_six=fmt == "nvfp4" and rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), fused=rng.random() < 0.5)
    if op == "read":
        seqs = _log(rng, 1, 64)
        return dict(op="read", seqs=seqs, length=_log(rng, 1, 100000 // seqs), heads=heads, dim=dim, page=page, fmt=fmt,
                    dtype=rng.choice(["bf16", "f32"]))
    group = rng.choice([1, 2, 4, 5, 7, 8, 16])
    kind = rng.choice(["decode", "decode", "verify", "chunk"])
    if kind == "decode":
        seqs = _log(rng, 1, 128)
        q_len, length = 1, _log(rng, 1, min(131072, 400000 // seqs))
    elif kind == "verify":
        seqs = _log(rng, 1, 48)
        q_len = rng.randrange(2, 9)
        length = q_len + _log(rng, 1, 200000 // seqs)
    else:
        seqs = rng.randrange(1, 5)
        heads = min(heads, max(1, 64 // group))
        q_len = _log(rng, 17, 8192)
        length = q_len + (_log(rng, 1, 16384) if rng.random() < 0.7 else 0)
        pairs = 1.3e9 / (heads * group)  # scores a query head: bounds the plain form's memory
        q_len = max(17, min(q_len, int(pairs / length)))
        seqs = max(1, min(seqs, int(pairs / (q_len * length))))
    return dict(op="attend", seqs=seqs, q_len=q_len, length=length, q_heads=heads * group, heads=heads, dim=dim, page=page,
                fmt=fmt, causal=rng.random() < 0.8, window=rng.choice([0, 0, 0, _log(rng, 1, length)]))


# -------------------------------------------------------------------------------------------------
# Sizes that follow from a case alone.

def _lengths(case):
    """Ragged lengths: the first sequence has the full one, the others down to about half of it."""
    n = case["length"]
    return [n - (i * 7919) % (n // 2 + 1) if i else n for i in range(case["seqs"])]


def _new(case):
    """New tokens a sequence (write): ragged in the same way."""
    n = case["new"]
    return [n - (i * 613) % (n // 2 + 1) if i else n for i in range(case["seqs"])]


def _queries(case):
    n = case["q_len"]
    return [min(n - (i * 331) % (n // 2 + 1) if i else n, length) for i, length in enumerate(_lengths(case))]


def _block(case):
    return 16 if case["fmt"] == "nvfp4" else 32


def _row_bytes(case):
    """Bytes of one token and head of one of the two caches."""
    return case["dim"] // 2 + case["dim"] // _block(case)


def _visible(case):
    """Pairs of query and key (of one head) that the mask leaves, and keys that some query sees."""
    pairs = keys = 0
    w = case["window"]
    for q, n in zip(_queries(case), _lengths(case)):
        pos = np.arange(n - q, n)
        hi = pos if case["causal"] else np.full(q, n - 1)
        lo = np.maximum(0, pos - w + 1) if w else np.zeros(q, dtype=np.int64)
        pairs += int(np.maximum(0, hi - lo + 1).sum())
        keys += int(hi.max() - lo.min() + 1) if q else 0
    return pairs, keys


def work(case):
    if case["op"] == "write":
        rows = 2 * sum(_new(case)) * case["heads"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": rows * (case["dim"] * size + 2 * _row_bytes(case) + 2 * case["dim"]) + 8 * sum(_new(case)), "flops": 0}
    if case["op"] == "read":
        rows = 2 * sum(_lengths(case)) * case["heads"]
        return {"bytes": rows * (_row_bytes(case) + case["dim"] * (2 if case["dtype"] == "bf16" else 4)), "flops": 0}
    pairs, keys = _visible(case)
    tokens = sum(_queries(case)) * case["q_heads"]
    return {"bytes": 2 * keys * case["heads"] * _row_bytes(case) + tokens * (4 * case["dim"] + 4),
            "flops": 4 * pairs * case["q_heads"] * case["dim"]}


# -------------------------------------------------------------------------------------------------
# Plain forms.

def _power(e):
    """2^e in fp32 for whole numbers e of -126..127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _encode(y):
    """E2M1 codes (0..15) of fp32 values, nearest with ties to the even code, saturating."""
    a = y.abs()
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return c.to(torch.uint8) | (torch.signbit(y).to(torch.uint8) << 3)


@functools.cache
def _lattice(device):
    return torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=torch.float32, device=device)


def _values(codes, device):
    return _lattice(device)[codes.long()]


def _nv_candidate(x, s_g, target):
    """x [..., D/16, 16] fp32: E4M3 scale bytes, codes and squared errors (summed in element order)."""
    inv = 1.0 / (target * s_g)
    d8 = (x.abs().amax(-1) * inv).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = d8.float()
    r = torch.where(d == 0, torch.zeros_like(d), 1.0 / (d * s_g))
    codes = _encode(x * r[..., None])
    err = x - (_values(codes, x.device) * d[..., None]) * s_g
    return d8.view(torch.uint8), codes, functools.reduce(operator.add, (err * err).unbind(-1))


def _quantise(x, fmt, s_g, four_six):
    """x [..., D] fp32 -> (packed nibbles [..., D/2], scale bytes [..., D/B])."""
    if fmt == "nvfp4":
        xb = x.unflatten(-1, (-1, 16))
        scales, codes, sse = _nv_candidate(xb, s_g, 6.0)
        if four_six:
            scales4, codes4, sse4 = _nv_candidate(xb, s_g, 4.0)
            take = sse4 < sse
            scales, codes = torch.where(take, scales4, scales), torch.where(take[..., None], codes4, codes)
    else:
        xb = x.unflatten(-1, (-1, 32))
        amax = xb.abs().amax(-1)
        e = torch.where(amax == 0, torch.zeros_like(amax), torch.frexp(amax)[1].float() - 3).clamp(-23, 13)
        codes = _encode(xb * _power(-e)[..., None])
        scales = (e + 127).to(torch.uint8)
    codes = codes.flatten(-2)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), scales


def _dequantise(q, scales, fmt, s_g):
    """Packed nibbles [..., D/2] and scale bytes [..., D/B] -> fp32 [..., D]."""
    v = _values(torch.stack([q & 15, q >> 4], -1).flatten(-2), q.device)
    if fmt == "nvfp4":
        return ((v.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float()[..., None]) * s_g).flatten(-2)
    return (v.unflatten(-1, (-1, 32)) * _power(scales.int() - 127)[..., None]).flatten(-2)


def _plain_write(s):
    pages, heads, page, _ = s["cache"][0].shape
    at, off = s["slots"] // page, s["slots"] % page
    out = []
    for x, q, sc, g in ((s["k"], s["cache"][0], s["cache"][1], s["k_global"]), (s["v"], s["cache"][2], s["cache"][3], s["v_global"])):
        packed, scales = _quantise(x.float(), s["fmt"], g, s["four_six"])
        q[at, :, off] = packed
        sc[at, :, off] = scales
        out.append(_dequantise(q[at, :, off], sc[at, :, off], s["fmt"], g).to(torch.bfloat16))
    return {"k": out[0], "v": out[1]}


def _plain_read(s):
    page = s["cache"][0].shape[2]
    at, off = s["table"][s["row_seq"], s["row_token"] // page].long(), s["row_token"] % page
    k = _dequantise(s["cache"][0][at, :, off], s["cache"][1][at, :, off], s["fmt"], s["k_global"])
    v = _dequantise(s["cache"][2][at, :, off], s["cache"][3][at, :, off], s["fmt"], s["v_global"])
    return {"k": k.to(s["dtype"]), "v": v.to(s["dtype"])}


def _plain_attend(s):
    table, lens, cu = s["table"].long(), s["lens"].long(), s["cu_q"].long()
    seqs, q_max = lens.numel(), s["q_max"]
    kv_heads, group, dim = s["cache"][0].shape[1], s["q"].shape[1] // s["cache"][0].shape[1], s["q"].shape[2]

    def dense(q, sc, g):  # [seqs, kv heads, tokens, dim]
        x = _dequantise(q[table], sc[table], s["fmt"], g)
        return x.transpose(1, 2).reshape(seqs, kv_heads, -1, dim)

    n_q = cu[1:] - cu[:-1]
    i = torch.arange(q_max, device=table.device)
    rows = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)                     # [seqs, q_max]
    q = s["q"][rows].float().unflatten(2, (kv_heads, group)).permute(0, 2, 3, 1, 4).reshape(seqs, kv_heads, group * q_max, dim)
    k = dense(s["cache"][0], s["cache"][1], s["k_global"])
    scores = (q @ k.transpose(-1, -2)) * s["scale"]
    del k
    j = torch.arange(scores.shape[-1], device=table.device)
    pos = (lens - n_q)[:, None] + i                                               # [seqs, q_max]
    keep = (j < lens[:, None, None]).expand(seqs, q_max, -1)
    if s["causal"]:
        keep = keep & (j <= pos[..., None])
    if s["window"]:
        keep = keep & (j > pos[..., None] - s["window"])
    keep = keep[:, None, None]
    scores = scores.view(seqs, kv_heads, group, q_max, -1).masked_fill_(~keep, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = dense(s["cache"][2], s["cache"][3], s["v_global"])
    o = (p.view(seqs, kv_heads, group * q_max, -1) @ v).view(seqs, kv_heads, group, q_max, dim)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = top + total.log()
    live = (i < n_q[:, None]).flatten().nonzero().flatten()
    o = o.permute(0, 3, 1, 2, 4).reshape(seqs * q_max, kv_heads * group, dim)[live]
    lse = lse[..., 0].permute(0, 3, 1, 2).reshape(seqs * q_max, kv_heads * group)[live]
    return {"out": o.to(torch.bfloat16), "lse": lse}


# -------------------------------------------------------------------------------------------------
# What a program has in hand.

def _numbers(gen, shape, device, spread=1.0):
    """Projections: normal values whose channels differ in size, a few of them much larger."""
    x = torch.randn(shape, generator=gen, device=device)
    c = torch.rand(shape[-2:], generator=gen, device=device)
    return x * (spread * (0.5 + c + 6.0 * (c > 0.98)))


def _fresh_cache(case, pages, device):
    shape = (pages, case["heads"], case["page"])
    mk = lambda n: torch.zeros(shape + (n,), dtype=torch.uint8, device=device)  # noqa: E731
    half, nb = case["dim"] // 2, case["dim"] // _block(case)
    return [mk(half), mk(nb), mk(half), mk(nb)]


def _table(gen, counts, page, device):
    """A block table over pages in random order, unused entries -1; pages in all."""
    used = [-(-n // page) for n in counts]
    pages = sum(used)
    order = torch.randperm(pages, generator=gen, device=device).to(torch.int32)
    table = torch.full((len(counts), max(used)), -1, dtype=torch.int32, device=device)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages


def _globals(case, k_amax, v_amax, device):
    m = 256.0 if case.get("four_six") else 448.0
    return tuple(torch.tensor([a / (6 * m)], dtype=torch.float32, device=device) for a in (k_amax, v_amax))


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device).manual_seed(seed)
    heads, dim, page, fmt = case["heads"], case["dim"], case["page"], case["fmt"]
    s = {"op": case["op"], "fmt": fmt, "four_six": bool(case.get("four_six"))}
    if case["op"] == "write":
        new = _new(case)
        past = [case["past"] + 3 * i for i in range(case["seqs"])]
        total = sum(new)
        table, pages = _table(gen, [p + n for p, n in zip(past, new)], page, device)
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        if case["fused"]:  # [tokens, 2 query heads a key head, keys, values]
            qkv = _numbers(gen, (total, 4 * heads, dim), device).to(dtype)
            s["k"], s["v"] = qkv[:, 2 * heads:3 * heads], qkv[:, 3 * heads:]
        else:
            s["k"], s["v"] = (_numbers(gen, (total, heads, dim), device).to(dtype) for _ in range(2))
        seq = torch.repeat_interleave(torch.arange(case["seqs"], device=device), torch.tensor(new, device=device))
        starts = torch.tensor(past, device=device)
        cu = torch.tensor([0] + list(np.cumsum(new)), device=device)
        token = torch.arange(total, device=device) - cu[seq] + starts[seq]
        s["slots"] = table[seq, token // page].long() * page + token % page
        s["table"], s["starts"], s["cu"] = table, starts.to(torch.int32), cu.to(torch.int32)
        s["cache"] = _fresh_cache(case, pages, device)
        s["k_global"], s["v_global"] = _globals(case, 32.0, 32.0, device)
        return s
    lens = _lengths(case)
    table, pages = _table(gen, lens, page, device)
    s["k_global"], s["v_global"] = _globals(case, 40.0, 40.0, device)
    s["cache"] = _fresh_cache(case, pages, device)
    step = max(1, (1 << 25) // (heads * page * dim))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        for q, sc, g in ((0, 1, s["k_global"]), (2, 3, s["v_global"])):
            x = _numbers(gen, (n, page, heads, dim), device).transpose(1, 2)
            s["cache"][q][a:a + n], s["cache"][sc][a:a + n] = _quantise(x, fmt, g, False)
    s["table"] = table
    if case["op"] == "read":
        s["dtype"] = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["starts"] = torch.zeros(len(lens), dtype=torch.int32, device=device)
        s["cu"] = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=device)
        s["row_seq"] = torch.repeat_interleave(torch.arange(len(lens), device=device), torch.tensor(lens, device=device))
        s["row_token"] = torch.arange(sum(lens), device=device) - s["cu"].long()[s["row_seq"]]
        return s
    queries = _queries(case)
    s["q"] = _numbers(gen, (sum(queries), case["q_heads"], dim), device, 0.7).to(torch.bfloat16)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=device)
    s["cu_q"] = torch.tensor([0] + list(np.cumsum(queries)), dtype=torch.int32, device=device)
    s["q_max"], s["scale"] = max(queries), dim ** -0.5
    s["causal"], s["window"] = case["causal"], case["window"]
    return s


def run(state):
    s = state
    if not own:
        return {"write": _plain_write, "read": _plain_read, "attend": _plain_attend}[s["op"]](s)
    import block_scaled_fp4_amax_b200 as fp4
    fmt = fp4.NVFP4 if s["fmt"] == "nvfp4" else fp4.MXFP4
    scales = dict(k_global=s["k_global"], v_global=s["v_global"]) if s["fmt"] == "nvfp4" else {}
    if s["op"] == "write":
        fp4.fp4_kv_append(s["k"], s["v"], s["cache"], s["slots"], fmt, four_six=s["four_six"], **scales)
        k, v = fp4.fp4_kv_read(s["cache"], s["table"], s["cu"], s["k"].shape[0], fmt, starts=s["starts"],
                               out_dtype=torch.bfloat16, **scales)
        return {"k": k, "v": v}
    if s["op"] == "read":
        k, v = fp4.fp4_kv_read(s["cache"], s["table"], s["cu"], s["row_seq"].numel(), fmt, starts=s["starts"],
                               out_dtype=s["dtype"], **scales)
        return {"k": k, "v": v}
    out, lse = fp4.fp4_kv_attention(s["q"], s["cache"], s["table"], s["lens"], fmt, cu_q=s["cu_q"], max_q=s["q_max"],
                                    scale=s["scale"], causal=s["causal"], window=s["window"], want_lse=True, **scales)
    return {"out": out, "lse": lse}


# -------------------------------------------------------------------------------------------------
# The definition in 64 bits: the encoder's 32-bit rounding steps are part of the format, so they are
# taken as 64-bit operations rounded to fp32 one by one; everything else stays in 64 bits.

def _f32(x):
    return x.float().double()


def _two_to(e):
    """2^e in fp64 for whole numbers e, from the exponent field."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _nearest(x, points):
    """Index of the nearest of the ascending `points`; a tie goes to the even index."""
    p = torch.tensor(points, dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(p, x.contiguous()).clamp(1, len(points) - 1)
    lo = hi - 1
    up, down = p[hi] - x, x - p[lo]
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def _e4m3_points():
    return [m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127]


def _exact_quantised(x, fmt, s_g, four_six):
    """The value that the cache holds for each of the fp64 values x [..., D], in 64 bits."""
    size = 16 if fmt == "nvfp4" else 32
    xb = x.reshape(-1, size)
    amax = xb.abs().amax(1, keepdim=True)
    points = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)

    def code(y):
        return points[_nearest(y.abs().clamp(max=6.0), _E2M1)] * torch.where(torch.signbit(y), -1.0, 1.0)

    if fmt != "nvfp4":
        e = torch.where(amax > 0, torch.floor(torch.log2(amax)), torch.full_like(amax, 2.0)) - 2
        unit = _two_to(e.clamp(-23, 13))
        return (code(xb / unit) * unit).reshape(x.shape)
    e4m3 = torch.tensor(_e4m3_points(), dtype=torch.float64, device=x.device)

    def candidate(t):
        d = e4m3[_nearest(_f32(amax * _f32(1.0 / _f32(t * s_g))).clamp(max=448.0), _e4m3_points())]
        back = torch.where(d > 0, _f32(1.0 / _f32(d * s_g).clamp(min=1e-300)), torch.zeros_like(d))
        c = code(_f32(xb * back)) * d
        total = torch.zeros(len(xb), dtype=torch.float64, device=x.device)
        for i in range(size):
            err = _f32(xb[:, i] - _f32(c[:, i] * s_g))
            total = _f32(total + _f32(err * err))
        return c * s_g, total

    best, err = candidate(6.0)
    if four_six:
        other, err4 = candidate(4.0)
        best = torch.where((err4 < err)[:, None], other, best)
    return best.reshape(x.shape)


def _exact_cached(q, scales, fmt, s_g):
    """Packed bytes -> fp64 values, from the bit fields."""
    nib = torch.stack([q & 15, q >> 4], -1).flatten(-2).to(torch.int32)
    exp, man = (nib >> 1) & 3, (nib & 1).double()
    v = torch.where(exp == 0, 0.5 * man, (1 + 0.5 * man) * _two_to(exp - 1)) * (1.0 - 2.0 * (nib >> 3).double())
    b = scales.to(torch.int32)
    if fmt == "nvfp4":
        exp, man = (b >> 3) & 15, (b & 7).double()
        d = torch.where(exp == 0, man * 2.0 ** -9, (8 + man) * _two_to(exp - 10)) * s_g.double()
        return (v.unflatten(-1, (-1, 16)) * d[..., None]).flatten(-2)
    return (v.unflatten(-1, (-1, 32)) * _two_to(b - 127)[..., None]).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    fmt = s["fmt"]
    if s["op"] == "write":
        return {"k": _exact_quantised(s["k"].double(), fmt, s["k_global"].double(), s["four_six"]),
                "v": _exact_quantised(s["v"].double(), fmt, s["v_global"].double(), s["four_six"])}
    kq, ks, vq, vs = s["cache"]
    page, lens, cu = case["page"], _lengths(case), [0]
    out = {"k": [], "v": []} if s["op"] == "read" else {"out": [], "lse": []}
    for b, n in enumerate(lens):
        at = s["table"][b, : -(-n // page)].long()
        k = _exact_cached(kq[at], ks[at], fmt, s["k_global"]).transpose(0, 1).flatten(1, 2)[:, :n]  # [heads, n, dim]
        v = _exact_cached(vq[at], vs[at], fmt, s["v_global"]).transpose(0, 1).flatten(1, 2)[:, :n]
        if s["op"] == "read":
            out["k"].append(k.transpose(0, 1))
            out["v"].append(v.transpose(0, 1))
            continue
        m = _queries(case)[b]
        cu.append(cu[-1] + m)
        q = s["q"][cu[-2]:cu[-1]].double()                                        # [m, q heads, dim]
        group = q.shape[1] // k.shape[0]
        pos = torch.arange(n - m, n, device=q.device)[:, None]
        j = torch.arange(n, device=q.device)[None]
        hide = torch.zeros(m, n, dtype=torch.bool, device=q.device)
        if s["causal"]:
            hide |= j > pos
        if s["window"]:
            hide |= j <= pos - s["window"]
        o, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float64, device=q.device)
        for h in range(q.shape[1]):
            z = (q[:, h] @ k[h // group].T) * s["scale"]
            z.masked_fill_(hide, -math.inf)
            lse[:, h] = torch.logsumexp(z, -1)
            w = torch.exp(z - lse[:, h, None])
            o[:, h] = torch.where(torch.isfinite(lse[:, h, None]), w @ v[h // group], torch.zeros_like(o[:, h]))
        out["out"].append(o)
        out["lse"].append(lse)
    return {name: torch.cat(parts) for name, parts in out.items()}
