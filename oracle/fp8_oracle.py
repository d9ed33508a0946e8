"""fp64 CPU definition of the FP8 block-scaled cache, of attention over it and
of the query/key norm with the rotary rotation.

Plain numpy written from the formulas, one sequence, block and head at a time;
it shares no code with the CUDA path and is test infrastructure only.
"""

import numpy as np

BLOCK = 16
MIN_EXP, MAX_EXP = -60, 60
BF16_MAX = 3.3895313892515355e38


def e4m3(x):
    """Nearest E4M3 value (ties to even, saturating at +-448) of finite x."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(np.where(x == 0, 1.0, x))           # |x| in [2^(e-1), 2^e)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)     # four significant bits, 2^-9 below 2^-6
    return np.clip(np.rint(x / step) * step, -448.0, 448.0)


def e4m3_bytes(v):
    """Codes of E4M3 values (uint8)."""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    _, e = np.frexp(np.where(a == 0, 1.0, a))
    e = np.maximum(e - 1, -6)
    m = np.ldexp(a, 3 - e).astype(np.int64)              # 8 .. 15, below 8 for subnormals
    code = np.where(m >= 8, ((e + 7) << 3) + (m - 8), m)
    return (code | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def e4m3_values(codes):
    c = np.asarray(codes).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, np.ldexp(m.astype(np.float64), -9), np.ldexp(8.0 + m, e - 10))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


def exponent(amax):
    """Smallest k in [MIN_EXP, MAX_EXP] with amax <= 448 * 2^k."""
    k = MIN_EXP
    while k < MAX_EXP and amax > 448.0 * 2.0 ** k:
        k += 1
    return k


def stored_exponent(scale):
    """Exponent of a stored scale; None for one that no write stores."""
    s = float(scale)
    if np.isfinite(s) and s > 0:
        m, e = np.frexp(s)
        if m == 0.5 and MIN_EXP <= e - 1 <= MAX_EXP:
            return int(e - 1)
    return None


def write(x, block_table, seq_lens, start, codes, scale):
    """Write x [T, H, D] (fp64 of bf16 values) into codes [NB, 16, H, D] (uint8)
    and scale [NB, H] in place."""
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), 0.0, np.clip(x, -BF16_MAX, BF16_MAX))
    heads = x.shape[1]
    for i in range(len(seq_lens)):
        n, length = int(start[i + 1] - start[i]), int(seq_lens[i])
        p0 = length - n
        for b in range(p0 // BLOCK, -(-length // BLOCK)) if n else ():
            lo, hi = max(p0, b * BLOCK), min(length, (b + 1) * BLOCK)
            blk, r0, r1 = int(block_table[i, b]), lo - b * BLOCK, hi - b * BLOCK
            if not 0 <= blk < codes.shape[0]:
                continue  # no block: its rows are skipped
            rows = x[start[i] + lo - p0:start[i] + hi - p0]
            for h in range(heads):
                k = exponent(np.abs(rows[:, h]).max())
                old = stored_exponent(scale[blk, h])
                if r0 > 0 and old is not None:
                    k = max(k, old)
                    if k > old:
                        codes[blk, :r0, h] = e4m3_bytes(e4m3(np.ldexp(e4m3_values(codes[blk, :r0, h]), old - k)))
                codes[blk, r0:r1, h] = e4m3_bytes(e4m3(np.ldexp(rows[:, h], -k)))
                scale[blk, h] = 2.0 ** k


def read(block_table, length, i, codes, scale, head):
    """Positions [0, length) of sequence i, one head: [length, D] in fp64."""
    p = np.arange(length)
    blk = block_table[i, p // BLOCK].astype(np.int64)
    return e4m3_values(codes[blk, p % BLOCK, head]) * scale[blk, head].astype(np.float64)[:, None]


def attention(q, caches, block_table, seq_lens, start, softmax_scale, causal, window=0, num_blocks=None):
    """(out, bound) for q [T, Hq, D] over caches (k codes, v codes, k scale, v
    scale).  bound is what the kernels' roundings can add to each output before
    the final one to bf16:
      - a weight times its V scale is rounded to f16, half a step 2^-11 of it,
        or, where it is subnormal, 2^-24 of the largest: half the spacing is 2^-25,
        and the largest is above 1/2, not 1, as exponents are taken relative to a
        whole number at or above the greatest; at most itself;
      - a score is an fp32 sum of D products of f16 and E4M3 values and one
        fma: at most (D + 4) 2^-24 sum |q k| in it, with the f16 spacing
        2^-24 max|q| of small query elements; the exponent's error moves weight
        and denominator alike, twice the error, and exp2 adds 2^-21;
      - the fp32 sums over the keys: n 2^-24 of sum p |v| at the very most,
        a few 2^-24 in the pairwise order that kernels use; n is capped at 64.
    """
    kc, vc, ks, vs = caches
    q = np.asarray(q, np.float64)
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    hkv, d = kc.shape[2], kc.shape[3]
    group = q.shape[1] // hkv
    nb = kc.shape[0] if num_blocks is None else num_blocks
    for i in range(len(seq_lens)):
        a, b, length = int(start[i]), int(start[i + 1]), int(seq_lens[i])
        n = b - a
        if n == 0 or length == 0:
            continue
        p = np.arange(length)
        blk = block_table[i, p // BLOCK].astype(np.int64)
        usable = (blk >= 0) & (blk < nb)
        safe = np.where(usable, blk, 0)
        pos = length - n + np.arange(n)
        seen = np.broadcast_to(usable[None], (n, length)).copy()
        if causal:
            seen &= p[None] <= pos[:, None]
        if window:
            seen &= p[None] > pos[:, None] - window
        for h in range(hkv):
            k = e4m3_values(kc[safe, p % BLOCK, h]) * ks[safe, h].astype(np.float64)[:, None]
            v = e4m3_values(vc[safe, p % BLOCK, h]) * vs[safe, h].astype(np.float64)[:, None]
            any_seen = seen.any(0)
            k[~any_seen], v[~any_seen] = 0.0, 0.0
            for j in range(group):
                x = q[a:b, h * group + j]
                s = np.where(seen, x @ k.T * softmax_scale, -np.inf)
                top = s.max(1, keepdims=True)
                w = np.where(seen, np.exp(s - np.where(np.isfinite(top), top, 0.0)), 0.0)
                tot = w.sum(1, keepdims=True)
                w = w / np.where(tot == 0, 1.0, tot)
                out[a:b, h * group + j] = w @ v
                size = np.where(seen, np.abs(x) @ np.abs(k).T, 0.0)
                small = np.abs(x).max(1, keepdims=True) * np.abs(k).sum(1)[None]
                ds = abs(softmax_scale) * 2.0 ** -24 * ((d + 4) * size + np.where(seen, small, 0.0))
                rel = 2.0 ** -21 + 64 * 2.0 ** -24 + 2 * ds.max(1, keepdims=True)
                scale_v = vs[safe, h].astype(np.float64)[None]
                part = np.where(seen, w * np.where(usable, scale_v, 0.0), 0.0)  # weights as the MMA holds them ...
                most = part.max(1, keepdims=True)
                u = part / np.where(most == 0, 1.0, most)                       # ... in units of the largest
                err = np.minimum(u, np.maximum(2.0 ** -11 * u, 2.0 ** -24)) * most
                code = np.abs(v) / np.where(any_seen & usable, vs[safe, h].astype(np.float64), 1.0)[:, None]
                bound[a:b, h * group + j] = rel * (w @ np.abs(v)) + err @ code
    return out, bound


def norm_rope(x, w, eps, cos_sin, positions, interleaved):
    """y [T, H, D] in fp64; w, cos_sin may be None."""
    y = np.asarray(x, np.float64).copy()
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    if cos_sin is not None and cos_sin.shape[1]:
        half = cos_sin.shape[1] // 2
        table = np.asarray(cos_sin, np.float64)[positions]
        cos, sin = table[:, None, :half], table[:, None, half:]
        i = np.arange(half)
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        u, v = y[..., lo].copy(), y[..., hi].copy()
        y[..., lo] = u * cos - v * sin
        y[..., hi] = v * cos + u * sin
    return y
