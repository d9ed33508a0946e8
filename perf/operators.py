"""Cases, plain forms and 64-bit definitions of the operators around the FP8 block-scaled KV cache.

Four operators, as a serving step runs them one after the other:

  norm_rope  RMS norm of every query and key head vector, then the rotary position rotation
  write      K and V of new tokens quantised into a paged E4M3 cache with one power-of-two
             scale per (block of 16 tokens, kv head)
  attend     causal, windowed or cross attention of queries over that cache
  read       positions of the cache back as bf16

Cache: codes float8_e4m3fn [blocks][16][kv heads][head size], scales float32 [blocks][kv heads];
a code c of a block with scale s stands for c * s.
"""

import math
import random

import torch

own = False

BLOCK = 16
HEAD_SIZES = (64, 96, 128, 192, 256)
E4M3_MAX = 448.0
MIN_EXP, MAX_EXP = -60, 60      # a block's scale is 2^k with k in this range
INPUT_MAX = E4M3_MAX * 2.0 ** MAX_EXP
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _attend(name, kind, q_heads, kv_heads, head_size, seqs, q_lo, q_hi, kv_lo, kv_hi, decodes=0, window=0, shape_seed=1):
    c = {"op": "attend", "kind": kind, "q_heads": q_heads, "kv_heads": kv_heads, "head_size": head_size, "seqs": seqs,
         "q_lo": q_lo, "q_hi": q_hi, "kv_lo": kv_lo, "kv_hi": kv_hi, "decodes": decodes, "window": window,
         "shape_seed": shape_seed}
    return dict(c, name=name) if name else c


def _cache(name, op, kv_heads, head_size, seqs, n_lo, n_hi, past_hi, shape_seed=1):
    c = {"op": op, "kv_heads": kv_heads, "head_size": head_size, "seqs": seqs, "n_lo": n_lo, "n_hi": n_hi,
         "past_hi": past_hi, "shape_seed": shape_seed}
    return dict(c, name=name) if name else c


def _norm(name, q_heads, kv_heads, head_size, rot, tokens, interleaved, shape_seed=1):
    c = {"op": "norm_rope", "q_heads": q_heads, "kv_heads": kv_heads, "head_size": head_size, "rot": rot,
         "tokens": tokens, "interleaved": interleaved, "shape_seed": shape_seed}
    return dict(c, name=name) if name else c


def listed():
    return [
        # two short sequences with four new tokens each: the smallest call, all latency
        _attend("attend tiny", "append", 4, 4, 128, 2, 4, 4, 97, 128),
        # one step of a batch of conversations of many lengths, four query heads per kv head
        _attend("attend decode gqa", "append", 32, 8, 128, 64, 1, 1, 512, 8192),
        # one step over long documents
        _attend("attend decode long", "append", 32, 8, 128, 32, 1, 1, 32768, 32768),
        # prompts of several users at once
        _attend("attend prefill", "prompt", 32, 8, 128, 8, 0, 0, 512, 2048),
        # short prompts that arrive while other sequences decode, head size that is no power of two
        _attend("attend mixed", "prompt", 16, 4, 192, 4, 0, 0, 200, 400, decodes=28),
        # decoder tokens over an encoder's states of another length, one query head per kv head
        _attend("attend cross", "cross", 16, 16, 64, 8, 1, 448, 1, 1500),
        # one new token of each of 64 sequences
        _cache("write decode", "write", 8, 128, 64, 1, 1, 8192),
        # prompts written in one go
        _cache("write prompts", "write", 8, 128, 32, 2048, 2048, 0),
        # a short ragged prefix, every head its own kv head
        _cache("read ragged", "read", 32, 96, 5, 1, 200, 300),
        # whole histories handed to another consumer
        _cache("read histories", "read", 8, 128, 32, 1500, 2500, 0),
        # one token of each of 64 sequences
        _norm("norm_rope decode", 32, 8, 128, 128, 64, False),
        # a large chunk of prompt tokens
        _norm("norm_rope prompts", 32, 8, 128, 128, 16384, False),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("attend", "attend", "attend", "write", "read", "norm_rope"))
    d = rng.choice(HEAD_SIZES)
    hkv = _log(rng, 1, 32)
    seed = rng.randrange(1 << 30)
    if op == "attend":
        group = rng.choice((1, 1, 2, 3, 4, 5, 7, 8, 12, 16))
        hkv = max(1, min(hkv, 64 // group))
        kind = rng.choice(("append", "append", "prompt", "cross"))
        if kind == "append":
            q = rng.choice((1, 1, 1, 2, 3, 5))
            hi = _log(rng, q, 32768)
            seqs = _log(rng, 1, 256)
            while seqs > 1 and seqs * hi * hkv * d > 2 ** 29:
                seqs //= 2
            window = rng.choice((0, 0, 0, _log(rng, 1, hi)))
            return _attend("", kind, hkv * group, hkv, d, seqs, 1, q, max(q, rng.randint(1, hi)), hi, window=window,
                           shape_seed=seed)
        hi = _log(rng, 16, 2048)
        seqs = _log(rng, 1, 16)
        decodes = rng.choice((0, 0, _log(rng, 1, 16))) if kind == "prompt" else 0
        while seqs > 1 and (seqs + decodes) * hi * max(hi, 2048 if decodes else 0) * hkv * group > 2 ** 30:
            seqs //= 2
            decodes //= 2
        if kind == "prompt":
            return _attend("", kind, hkv * group, hkv, d, seqs, 0, 0, rng.randint(1, hi), hi,
                           decodes=decodes, window=rng.choice((0, 0, _log(rng, 1, hi))),
                           shape_seed=seed)
        return _attend("", kind, hkv * group, hkv, d, seqs, 1, _log(rng, 1, hi), rng.randint(1, hi), hi, shape_seed=seed)
    if op == "norm_rope":
        group = rng.choice((1, 2, 4, 5, 8))
        tokens = _log(rng, 1, 16384)
        while tokens > 1 and tokens * hkv * (group + 1) * d > 16384 * 40 * 128:
            tokens //= 2
        return _norm("", hkv * group, hkv, d, rng.choice((d, d, d // 2, 16 * rng.randint(1, d // 16))), tokens,
                     rng.random() < 0.3, shape_seed=seed)
    hi = _log(rng, 1, 4096)
    seqs = _log(rng, 1, 256)
    while seqs > 1 and seqs * hi * hkv * d > 2 ** 26:
        seqs //= 2
    while hi > 1 and seqs * hi * hkv * d > 2 ** 26:
        hi //= 2
    return _cache("", op, hkv, d, seqs, rng.randint(1, hi), hi, _log(rng, 1, 4096), shape_seed=seed)


def _lengths(case):
    """(new or query tokens, length in the cache) of every sequence."""
    r = random.Random(case["shape_seed"])
    if case["op"] in ("write", "read"):
        n = [r.randint(case["n_lo"], case["n_hi"]) for _ in range(case["seqs"])]
        return [(x, x + r.randint(0, case["past_hi"])) for x in n]
    got = []
    for _ in range(case["seqs"]):
        kv = r.randint(case["kv_lo"], case["kv_hi"])
        q = r.randint(case["q_lo"], case["q_hi"]) if case["kind"] != "prompt" else kv
        got.append((min(q, kv) if case["kind"] == "append" else q, kv))
    got += [(1, r.randint(1, 2048)) for _ in range(case["decodes"])]
    r.shuffle(got)
    return got


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _exponent(amax):
    """Smallest k with amax <= 448 * 2^k, in [MIN_EXP, MAX_EXP], as int32 (amax: float32)."""
    m, e = torch.frexp(amax)  # amax = m * 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    k = e - 9 + (m > 0.875).to(e.dtype)
    return torch.where(amax > 0, k, torch.full_like(k, MIN_EXP)).clamp(MIN_EXP, MAX_EXP)


def _two_to(k):
    """2^k exactly, from its bits (pow rounds); k outside [-126, 127] counts as the nearer end."""
    return ((k.to(torch.int32).clamp(-126, 127) + 127) << 23).view(torch.float32)


def _codes(x):
    """The bytes of the nearest E4M3 values."""
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def _values(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _history(g, blocks, kv_heads, d, gain):
    """Codes and scales of `blocks` blocks of normal values."""
    codes = torch.empty((blocks, BLOCK, kv_heads, d), dtype=torch.uint8, device="cuda")
    scale = torch.empty((blocks, kv_heads), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // (BLOCK * kv_heads * d))
    for b in range(0, blocks, step):
        n = min(step, blocks - b)
        x = torch.randn((n, BLOCK, kv_heads, d), generator=g, device="cuda") * gain
        s = _two_to(_exponent(x.abs().amax((1, 3))))
        codes[b:b + n] = _codes(x / s[:, None, :, None])
        scale[b:b + n] = s
    return codes.view(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    d, hkv = case["head_size"], case["kv_heads"]
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    if case["op"] == "norm_rope":
        t, hq = case["tokens"], case["q_heads"]
        # one projection's output holds q, k and v of a token side by side
        qkv = torch.randn((t, (hq + 2 * hkv) * d), generator=g, device="cuda").to(torch.bfloat16)
        r = random.Random(seed)
        far = 32768
        rot = case["rot"]
        angle = torch.arange(far, device="cuda", dtype=torch.float64)[:, None] * (
            10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot))
        return {"case": case, "q": qkv[:, :hq * d].view(t, hq, d), "k": qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d),
                "positions": torch.randint(0, far, (t,), generator=g, device="cuda") if t <= 256 else
                torch.arange(t, device="cuda") + r.randint(0, far - t),
                "cos_sin": torch.cat([angle.cos(), angle.sin()], 1).float(),
                "q_weight": (torch.rand(d, generator=g, device="cuda") + 0.5).to(torch.bfloat16),
                "k_weight": (torch.rand(d, generator=g, device="cuda") + 0.5).to(torch.bfloat16),
                "q_out": torch.empty((t, hq, d), **bf16), "k_out": torch.empty((t, hkv, d), **bf16),
                "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    lens = _lengths(case)
    need = [-(-kv // BLOCK) for _, kv in lens]
    blocks = sum(need) + 8
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor([0] + need, device="cuda").cumsum(0)[:-1]
    col = torch.arange(max(need), device="cuda")
    held = col[None] < torch.tensor(need, device="cuda")[:, None]
    table = torch.where(held, order[(first[:, None] + col[None]).clamp(max=blocks - 1)], torch.full_like(order[:1], -1))
    gain = torch.exp(0.5 * torch.randn((hkv, d), generator=g, device="cuda"))  # some channels are larger than others
    k_cache, k_scale = _history(g, blocks, hkv, d, gain)
    v_cache, v_scale = _history(g, blocks, hkv, d, 1.0)
    start = torch.tensor([0] + [n for n, _ in lens], device="cuda").cumsum(0).to(torch.int32)
    t = sum(n for n, _ in lens)
    s = {"case": case, "block_table": table.contiguous(), "k_cache": k_cache, "v_cache": v_cache, "k_scale": k_scale,
         "v_scale": v_scale, "seq_lens": torch.tensor([kv for _, kv in lens], dtype=torch.int32, device="cuda"),
         "start_loc": start, "tokens": t, "max_n": max(n for n, _ in lens), "max_len": max(kv for _, kv in lens),
         "status": torch.zeros(1, dtype=torch.int32, device="cuda"), "workspace": None}
    if case["op"] == "write":
        kv = torch.randn((t, 2 * hkv * d), generator=g, device="cuda")
        kv[:, :hkv * d] *= gain.reshape(-1)
        kv = kv.to(torch.bfloat16)
        s |= {"k": kv[:, :hkv * d].view(t, hkv, d), "v": kv[:, hkv * d:].view(t, hkv, d)}
    elif case["op"] == "read":
        s |= {"k": torch.empty((t, hkv, d), **bf16), "v": torch.empty((t, hkv, d), **bf16)}
    else:
        hq = case["q_heads"]
        s |= {"q": torch.randn((t, hq, d), generator=g, device="cuda").to(torch.bfloat16),
              "out": torch.empty((t, hq, d), **bf16), "scale": 1.0 / math.sqrt(d), "causal": case["kind"] != "cross"}
    return s


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"norm_rope": _plain_norm_rope, "write": _plain_write, "read": _plain_read, "attend": _plain_attend}[op](state)


def _own(s, op):
    import int4_token_head_gb300 as kv

    if op == "norm_rope":
        kv.qk_norm_rope(s["q"], s["k"], s["positions"], s["cos_sin"], s["q_weight"], s["k_weight"], EPS, s["q_out"],
                        s["k_out"], interleaved=s["case"]["interleaved"], dev_status=s["status"])
        return s["q_out"], s["k_out"]
    cache = s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    if op == "write":
        kv.write_fp8(s["k"], s["v"], s["block_table"], s["seq_lens"], s["start_loc"], s["max_n"], *cache,
                     dev_status=s["status"])
        return cache
    if op == "read":
        kv.read_fp8(*cache, s["block_table"], s["seq_lens"], s["start_loc"], s["max_n"], s["k"], s["v"],
                    dev_status=s["status"])
        return s["k"], s["v"]
    if s["workspace"] is None:
        c = s["case"]
        size = kv.attention_workspace_size(len(s["seq_lens"]), s["tokens"], c["q_heads"], c["kv_heads"], c["head_size"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    kv.attention_fp8(s["q"], *cache, s["block_table"], s["seq_lens"], s["start_loc"], s["max_n"], s["max_len"],
                     s["scale"], s["causal"], s["out"], s["workspace"], dev_status=s["status"],
                     sliding_window=s["case"]["window"])
    return s["out"]


def _plain_norm_rope(s):
    rot = s["case"]["rot"]
    table = s["cos_sin"][s["positions"]]
    cos, sin = table[:, None, :rot // 2], table[:, None, rot // 2:]

    def one(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        r, rest = x[..., :rot], x[..., rot:]
        if s["case"]["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = r[..., :rot // 2], r[..., rot // 2:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([r, rest], -1).to(torch.bfloat16)

    return one(s["q"], s["q_weight"]), one(s["k"], s["k_weight"])


def _slots(s):
    """(sequence, position, block, row) of every token of the call."""
    start = s["start_loc"].long()
    t = torch.arange(s["tokens"], device=start.device)
    seq = torch.searchsorted(start, t, right=True) - 1
    pos = s["seq_lens"].long()[seq] - (start[seq + 1] - start[seq]) + t - start[seq]
    return seq, pos, s["block_table"].long()[seq, pos // BLOCK], pos % BLOCK


def _plain_write(s):
    _, pos, block, row = _slots(s)
    start = s["start_loc"].long()
    n = start[1:] - start[:-1]
    p0 = s["seq_lens"].long() - n
    # the block that holds a sequence's first new position may hold earlier ones: their codes follow its scale
    at = s["block_table"].long().gather(1, (p0 // BLOCK)[:, None])[:, 0].clamp(min=0)
    kept = torch.arange(BLOCK, device=p0.device)[None] < (p0 % BLOCK)[:, None]
    count = torch.zeros(s["k_scale"].shape[0], dtype=torch.int64, device=p0.device)
    written = count.index_add(0, block, torch.ones_like(row)) > 0
    fresh = count.index_add(0, block, (row == 0).long()) > 0
    for x, codes, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        x = x.float().clamp(-INPUT_MAX, INPUT_MAX)
        amax = torch.zeros_like(scale).index_reduce(0, block, x.abs().amax(-1), "amax")
        old = torch.frexp(scale)[1] - 1
        k = torch.maximum(_exponent(amax), torch.where(fresh[:, None], torch.full_like(old, MIN_EXP), old))
        k = torch.where(written[:, None], k, old)
        codes = codes.view(torch.uint8)
        had = codes[at]
        moved = _codes(_values(had) * _two_to(old[at] - k[at])[:, None, :, None])
        codes[at] = torch.where(kept[:, :, None, None], moved, had)
        codes[block, row] = _codes(x * _two_to(-k[block])[:, :, None])
        scale.copy_(_two_to(k))
    return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _plain_read(s):
    _, _, block, row = _slots(s)
    return tuple((_values(codes.view(torch.uint8)[block, row]) * scale[block][:, :, None]).to(torch.bfloat16)
                 for codes, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))


def _plain_attend(s):
    c = s["case"]
    hq, hkv, d = c["q_heads"], c["kv_heads"], c["head_size"]
    group = hq // hkv
    start, length = s["start_loc"].long(), s["seq_lens"].long()
    n = start[1:] - start[:-1]
    table = s["block_table"].long().clamp(min=0)
    key = torch.arange(table.shape[1] * BLOCK, device=table.device)
    here = key[None] < length[:, None]                                                  # [S, L]

    def held(codes, scale):
        x = _values(codes.view(torch.uint8)[table]) * scale[table][:, :, None, :, None]
        x = torch.where(here[:, :, None, None], x.flatten(1, 2), torch.zeros((), device=x.device))
        return x.permute(0, 2, 1, 3)                                                     # [S, Hkv, L, d]

    j = torch.arange(s["max_n"], device=table.device)
    at = (start[:-1, None] + j[None]).clamp(max=s["tokens"] - 1)
    q = s["q"].float()[at].view(len(n), s["max_n"], hkv, group, d).permute(0, 2, 1, 3, 4)  # [S, Hkv, Q, G, d]
    scores = (q.flatten(2, 3) @ held(s["k_cache"], s["k_scale"]).transpose(2, 3)) * s["scale"]
    pos = (length - n)[:, None] + j[None]                                                # [S, Q]
    seen = here[:, None, :].expand(-1, s["max_n"], -1)
    if s["causal"]:
        seen = seen & (key[None, None] <= pos[:, :, None])
    if c["window"]:
        seen = seen & (key[None, None] > pos[:, :, None] - c["window"])
    seen = seen[:, None, :, None].expand(-1, 1, -1, group, -1).flatten(2, 3)             # [S, 1, Q G, L]
    scores = torch.where(seen, scores, torch.full((), -math.inf, device=q.device))
    top = scores.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(scores - top)
    o = (p @ held(s["v_cache"], s["v_scale"])) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.view(len(n), hkv, s["max_n"], group, d).permute(0, 2, 1, 3, 4).reshape(len(n), s["max_n"], hq, d)
    t = torch.arange(s["tokens"], device=table.device)
    seq = torch.searchsorted(start, t, right=True) - 1
    return o[seq, t - start[seq]].to(torch.bfloat16)


# ---------------------------------------------------------------------------
# bytes and operations that a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    d, hkv = case["head_size"], case["kv_heads"]
    if case["op"] == "norm_rope":
        t, h = case["tokens"], case["q_heads"] + hkv
        return {"bytes": t * (h * d * 4 + 8 + case["rot"] * 4), "flops": t * h * (4 * d + 3 * case["rot"])}
    lens = _lengths(case)
    t = sum(n for n, _ in lens)
    if case["op"] in ("write", "read"):
        touched = sum((kv - 1) // BLOCK - (kv - n) // BLOCK + 1 for n, kv in lens)
        return {"bytes": 2 * hkv * (t * d * 3 + touched * 8) + touched * 4 + 12 * len(lens), "flops": 2 * hkv * t * d * 2}
    hq, w = case["q_heads"], case["window"]
    keys = pairs = 0
    for q, kv in lens:
        if case["kind"] == "cross":
            keys, pairs = keys + kv, pairs + q * kv
            continue
        first = max(0, kv - q - w + 1) if w else 0
        keys += kv - first
        pairs += sum(min(p + 1, w) if w else p + 1 for p in range(kv - q, kv))
    blocks = -(-keys // BLOCK)
    return {"bytes": keys * hkv * 2 * d + blocks * (8 * hkv + 4) + t * hq * d * 4 + 12 * len(lens),
            "flops": 4 * d * hq * pairs}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
_POWERS = [2.0 ** e for e in range(-160, 161)]  # exact: pow on the GPU rounds


def _power(e):
    return torch.tensor(_POWERS, dtype=torch.float64, device=e.device)[e.long() + 160]


def _e4m3(x):
    """The nearest value with four significant bits and exponents -6 .. 8 (steps of 2^-9 below), ties to even."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -40)))
    step = _power(torch.clamp(e, -6.0, 20.0) - 3.0)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        rot, half = case["rot"], case["rot"] // 2
        both = []
        for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
            x = x.double()
            y = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
            i = torch.arange(half, device="cuda")
            lo, hi = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
            turn = torch.complex(s["cos_sin"][s["positions"], :half].double(), s["cos_sin"][s["positions"], half:].double())
            z = torch.complex(y[..., lo], y[..., hi]) * turn[:, None]
            y[..., lo], y[..., hi] = z.real.clone(), z.imag.clone()
            both.append(y)
        return tuple(both)
    lens = _lengths(case)
    tables = s["block_table"].cpu()
    d, hkv = case["head_size"], case["kv_heads"]
    if case["op"] == "write":
        out = []
        for x, codes, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
            codes, scale, x = codes.double(), scale.double(), x.double()
            t = 0
            for (n, kv), table in zip(lens, tables):
                p0, ids = kv - n, table[: -(-kv // BLOCK)].cuda()
                b0 = p0 // BLOCK
                ids = ids[b0:]
                r0 = p0 - b0 * BLOCK
                rows = torch.zeros((len(ids) * BLOCK, hkv, d), dtype=torch.float64, device="cuda")
                rows[r0:r0 + n] = x[t:t + n]
                live = rows.view(len(ids), BLOCK, hkv, d)
                top = live.abs().amax((1, 3))
                k = torch.ceil(torch.log2(top.clamp(min=2.0 ** -200) / 448.0))
                k = k.clamp(MIN_EXP - 1, MAX_EXP)
                k = torch.where(448.0 * _power(k - 1) >= top, k - 1, k)  # log2 may round across a whole number
                k = torch.where(448.0 * _power(k) < top, k + 1, k).clamp(MIN_EXP, MAX_EXP)
                if r0:
                    was = scale[ids[0]].clone()
                    k[0] = torch.maximum(k[0], torch.log2(was).round())
                    codes[ids[0], :r0] = _e4m3(codes[ids[0], :r0] * (was / _power(k[0]))[None, :, None])
                scale[ids] = _power(k)
                new = _e4m3(live / _power(k)[:, None, :, None]).flatten(0, 1)
                flat = ids.long().repeat_interleave(BLOCK) * BLOCK + torch.arange(BLOCK, device="cuda").repeat(len(ids))
                codes.view(-1, hkv, d)[flat[r0:r0 + n]] = new[r0:r0 + n]
                t += n
            out.append((codes, scale))
        return out[0][0], out[1][0], out[0][1], out[1][1]

    def whole(codes, scale, table, kv):
        ids = table[: -(-kv // BLOCK)].long().cuda()
        return (_values(codes.view(torch.uint8)[ids]).double() * scale[ids].double()[:, None, :, None]).flatten(0, 1)[:kv]

    if case["op"] == "read":
        parts = [[whole(codes, scale, table, kv)[kv - n:] for (n, kv), table in zip(lens, tables)]
                 for codes, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"]))]
        return tuple(torch.cat(p) for p in parts)
    group = case["q_heads"] // hkv
    out, t = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda"), 0
    for (n, kv), table in zip(lens, tables):
        k = whole(s["k_cache"], s["k_scale"], table, kv).repeat_interleave(group, 1)
        v = whole(s["v_cache"], s["v_scale"], table, kv).repeat_interleave(group, 1)
        a = torch.einsum("qhd,khd->hqk", s["q"][t:t + n].double(), k) / math.sqrt(d)
        gap = torch.arange(kv - n, kv, device="cuda")[:, None] - torch.arange(kv, device="cuda")[None]
        if case["kind"] != "cross":
            a.masked_fill_(gap < 0, -math.inf)
        if case["window"]:
            a.masked_fill_(gap >= case["window"], -math.inf)
        out[t:t + n] = torch.einsum("hqk,khd->qhd", torch.softmax(a, -1), v)
        t += n
    return out
