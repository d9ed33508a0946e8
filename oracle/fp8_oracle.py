"""fp64 CPU definition of the FP8 block-scaled cache, of attention over it, of the
weights that positions receive and eviction by them, and of the query/key norm
with the rotary rotation.

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


def norm_rope_axes(x, w, eps, cos_sin, positions, pair_axis, interleaved):
    """norm_rope with positions [axes, T] and the axis of every pair: pair by pair."""
    y = norm_rope(x, w, eps, None, None, interleaved)
    half = cos_sin.shape[1] // 2
    table = np.asarray(cos_sin, np.float64)
    for i, a in enumerate(pair_axis):
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        cos, sin = table[positions[a], i][:, None], table[positions[a], half + i][:, None]
        u, v = y[..., lo].copy(), y[..., hi].copy()
        y[..., lo] = u * cos - v * sin
        y[..., hi] = v * cos + u * sin
    return y


def _scores(q, codes, scale, table, length, n, i, h, group, softmax_scale, num_blocks):
    """Causal scores [n, group, length] of sequence i's queries (q [n, Hq, D]) against kv head h, -inf where hidden or
    without a block, and sums of |q k| and of max|q| |k| over the head."""
    p = np.arange(length)
    blk = table[i, p // BLOCK].astype(np.int64)
    usable = (blk >= 0) & (blk < num_blocks)
    safe = np.where(usable, blk, 0)
    k = e4m3_values(codes[safe, p % BLOCK, h]) * scale[safe, h].astype(np.float64)[:, None]
    k[~usable] = 0.0
    x = q[:, h * group:(h + 1) * group]
    seen = usable[None] & (p[None] <= (length - n + np.arange(n))[:, None])
    s = np.einsum("ngd,kd->ngk", x, k) * softmax_scale
    s = np.where(seen[:, None], s, -np.inf)
    size = np.einsum("ngd,kd->ngk", np.abs(x), np.abs(k))
    small = np.abs(x).max(2)[:, :, None] * np.abs(k).sum(1)[None, None]
    return s, size, small


def score_error(size, small, d, softmax_scale):
    """What the kernels' arithmetic can be off in a score: an fp32 sum of D exact products and a final product or fma,
    and the f16 spacing 2^-24 max|q| of query elements far below their row's largest."""
    return abs(softmax_scale) * 2.0 ** -24 * ((d + 4) * size + small)


def log_sum_exp(q, codes, scale, table, lens, start, softmax_scale, num_blocks=None):
    """(lse, bound) [T, Hq] of causal attention; -inf for a row that sees no key.  bound: the scores' errors, exp2 and
    the fp32 sums (n 2^-24 at most, 64 of them as in attention) move the sum by a share, the logarithm's own step and
    the maximum that is added are 2^-22 of the result and of the largest score."""
    q = np.asarray(q, np.float64)
    nb = codes.shape[0] if num_blocks is None else num_blocks
    hkv, d = codes.shape[2], codes.shape[3]
    group = q.shape[1] // hkv
    lse, bound = np.full(q.shape[:2], -np.inf), np.zeros(q.shape[:2])
    for i in range(len(lens)):
        a, b = int(start[i]), int(start[i + 1])
        for h in range(hkv) if b > a else ():
            s, size, small = _scores(q[a:b], codes, scale, table, int(lens[i]), b - a, i, h, group, softmax_scale, nb)
            top = s.max(2, keepdims=True)
            safe = np.where(np.isfinite(top), top, 0.0)
            with np.errstate(divide="ignore"):
                lse[a:b, h * group:(h + 1) * group] = (safe + np.log(np.exp(s - safe).sum(2, keepdims=True)))[..., 0]
            err = np.where(np.isfinite(s), score_error(size, small, d, softmax_scale), 0.0).max(2)
            bound[a:b, h * group:(h + 1) * group] = err + 2.0 ** -20 + 64 * 2.0 ** -24 + 2.0 ** -22 * (
                np.abs(safe[..., 0]) + np.abs(np.where(np.isfinite(top[..., 0]), lse[a:b, h * group:(h + 1) * group], 0.0)))
    return lse, bound


def mass(q, lse, codes, scale, table, lens, start, softmax_scale, m, num_blocks=None):
    """(mass, bound) [S, Hkv, positions] after a call on m.  A weight's exponent is off by the score's error and by the
    rounding of lse log2 e and of the sum, 2^-23 (|s| + |lse|); exp2 adds 2^-21; the sum over the rows n 2^-24."""
    q, lse = np.asarray(q, np.float64), np.asarray(lse, np.float64)
    nb = codes.shape[0] if num_blocks is None else num_blocks
    hkv, d = codes.shape[2], codes.shape[3]
    group = q.shape[1] // hkv
    m, bound = np.array(m, np.float64), np.zeros(m.shape)
    for i in range(len(lens)):
        a, b, length = int(start[i]), int(start[i + 1]), int(lens[i])
        n = b - a
        if n == 0:
            continue
        m[i, :, length - n:length] = 0.0
        for h in range(hkv):
            s, size, small = _scores(q[a:b], codes, scale, table, length, n, i, h, group, softmax_scale, nb)
            l = lse[a:b, h * group:(h + 1) * group, None]
            fine = np.isfinite(l)
            l = np.where(fine, l, 0.0)
            w = np.where(fine, np.exp(s - l), 0.0)
            err = score_error(size, small, d, softmax_scale) + 2.0 ** -23 * (np.where(np.isfinite(s), np.abs(s), 0) + np.abs(l))
            got = w.sum((0, 1))
            m[i, h, :length] += got
            bound[i, h, :length] = (w * (np.expm1(err) + 2.0 ** -21)).sum((0, 1)) + (n * group + 2) * 2.0 ** -24 * got
            bound[i, h, :length] += 2.0 ** -24 * np.abs(m[i, h, :length])
    return m, bound


def keep(m, length, budget, recent):
    """The positions that stay of a sequence for one kv head, ascending: the last `recent`, and of the others those of
    the largest mass, equal ones from the lowest position on, NaN below everything."""
    if length <= budget:
        return np.arange(length)
    x = np.where(np.isnan(m[:length - recent]), -np.inf, np.asarray(m[:length - recent], np.float64))
    nan = np.isnan(m[:length - recent])
    order = sorted(range(length - recent), key=lambda p: (nan[p], -x[p], p))
    return np.array(sorted(order[:budget - recent] + list(range(length - recent, length))), np.int64)


def evict(caches, m, table, lens, budget, recent, into, m_out, kept):
    """Moves what stays of every sequence in the numpy arrays given; returns the new lengths."""
    before = [np.array(x) for x in caches]
    m = np.array(m)
    new = []
    for i, length in enumerate(int(x) for x in lens):
        new.append(min(length, budget))
        for h in range(caches[0].shape[2]):
            idx = keep(m[i, h], length, budget, recent)
            n = len(idx)
            kept[i, h, :n], m_out[i, h, :n] = idx, m[i, h, idx]
            for b in range(-(-n // BLOCK)):
                rows = idx[b * BLOCK:(b + 1) * BLOCK]
                to = int(into[i, b])
                src = table[i, rows // BLOCK].astype(np.int64)
                if (rows == b * BLOCK + np.arange(len(rows))).all() and (src == to).all() or not 0 <= to < caches[0].shape[0]:
                    continue
                for codes, scale, old_codes, old_scale in ((caches[0], caches[2], before[0], before[2]),
                                                           (caches[1], caches[3], before[1], before[3])):
                    x = np.zeros((len(rows), codes.shape[3]))
                    for r, (s, p) in enumerate(zip(src, rows)):
                        if 0 <= s < codes.shape[0] and stored_exponent(old_scale[s, h]) is not None:
                            x[r] = e4m3_values(old_codes[s, p % BLOCK, h]) * float(old_scale[s, h])
                    k = exponent(np.abs(x).max())
                    codes[to, :len(rows), h] = e4m3_bytes(e4m3(np.ldexp(x, -k)))
                    scale[to, h] = 2.0 ** k
    return np.array(new, np.int32)
