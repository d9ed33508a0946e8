"""Cases, plain forms and 64-bit definitions of the operators for prompts with images and shared prefixes on the FP8 KV cache.

Four operators, as a serving step runs them:

  rope   RMS norm of every query and key head vector, then the rotary rotation by positions with several
         axes (time, height, width): every pair of elements takes its angle from the axis that owns it
  share  causal attention of a batch whose groups of sequences have their first positions in common; also the
         logarithm of every row's denominator
  mass   the attention weight that every position has received, added up over the calls
  evict  the heaviest positions and the last ones stay, moved to the front of a sequence's blocks

Cache: codes float8_e4m3fn [blocks][16][kv heads][head size], scales float32 [blocks][kv heads];
a code c of a block with scale s stands for c * s.  Mass: float32 [sequences][kv heads][positions].
"""

import math
import random

import torch

own = False

BLOCK = 16
HEAD_SIZES = (64, 96, 128, 192, 256)
MIN_EXP, MAX_EXP = -60, 60      # a block's scale is 2^k with k in this range
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _named(name, c):
    return dict(c, name=name) if name else c


def _rope(name, q_heads, kv_heads, head_size, rot, tokens, sections, turns, interleaved=False, shape_seed=1):
    """sections: rotation pairs of each axis, as text; turns: the axes take pairs in turn, not one after the other."""
    return _named(name, {"op": "rope", "q_heads": q_heads, "kv_heads": kv_heads, "head_size": head_size, "rot": rot,
                         "tokens": tokens, "sections": sections, "turns": turns, "interleaved": interleaved,
                         "shape_seed": shape_seed})


def _share(name, q_heads, kv_heads, head_size, groups, members, prefix, own_lo, own_hi, q_lo, q_hi, shape_seed=1):
    return _named(name, {"op": "share", "q_heads": q_heads, "kv_heads": kv_heads, "head_size": head_size,
                         "groups": groups, "members": members, "prefix": prefix, "own_lo": own_lo, "own_hi": own_hi,
                         "q_lo": q_lo, "q_hi": q_hi, "shape_seed": shape_seed})


def _mass(name, q_heads, kv_heads, head_size, seqs, q_lo, q_hi, kv_lo, kv_hi, prompt=False, shape_seed=1):
    return _named(name, {"op": "mass", "q_heads": q_heads, "kv_heads": kv_heads, "head_size": head_size, "seqs": seqs,
                         "q_lo": q_lo, "q_hi": q_hi, "kv_lo": kv_lo, "kv_hi": kv_hi, "prompt": prompt,
                         "shape_seed": shape_seed})


def _evict(name, kv_heads, head_size, seqs, kv_lo, kv_hi, budget, recent, in_place, shape_seed=1):
    return _named(name, {"op": "evict", "kv_heads": kv_heads, "head_size": head_size, "seqs": seqs, "kv_lo": kv_lo,
                         "kv_hi": kv_hi, "budget": budget, "recent": recent, "in_place": in_place,
                         "shape_seed": shape_seed})


def listed():
    return [
        # one token of each of 64 sequences, three axes one after the other
        _rope("rope decode", 32, 8, 128, 128, 64, "16 24 24", False),
        # a long video prompt, three axes in turn
        _rope("rope video", 32, 8, 128, 128, 16384, "24 20 20", True),
        # an image encoder's patches: height and width, one query head per key head
        _rope("rope image", 16, 16, 64, 64, 4225, "16 16", False),
        # two short sequences with a few blocks in common: the smallest call, all latency
        _share("share tiny", 4, 4, 128, 1, 2, 64, 33, 64, 1, 4),
        # many answers to one prompt, one token of each
        _share("share samples", 32, 8, 128, 1, 64, 8192, 1, 512, 1, 1),
        # four long documents, eight conversations about each
        _share("share documents", 32, 8, 128, 4, 8, 32768, 16, 1024, 1, 1),
        # short questions to one long prefix, head size that is no power of two
        _share("share questions", 16, 4, 192, 1, 16, 16384, 8, 48, 8, 48),
        # one step of a batch of conversations of many lengths
        _mass("mass decode gqa", 32, 8, 128, 64, 1, 1, 512, 8192),
        # one step over long documents
        _mass("mass decode long", 32, 8, 128, 32, 1, 1, 32768, 32768),
        # prompts of several users at once
        _mass("mass prompts", 32, 8, 128, 8, 0, 0, 512, 2048, prompt=True),
        # prompts that leave their blocks to others: what is kept goes to blocks of its own
        _evict("evict prompts", 8, 128, 32, 6000, 8192, 2048, 256, False),
        # a few conversations a little over their budget, in their own blocks
        _evict("evict overflow", 8, 128, 4, 1025, 1152, 1024, 64, True),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "share", "share", "mass", "mass", "evict"))
    d = rng.choice(HEAD_SIZES)
    hkv = _log(rng, 1, 32)
    seed = rng.randrange(1 << 30)
    if op == "rope":
        group = rng.choice((1, 2, 4, 5, 8))
        tokens = _log(rng, 1, 16384)
        while tokens > 1 and tokens * hkv * (group + 1) * d > 16384 * 40 * 128:
            tokens //= 2
        rot = rng.choice((d, d, d // 2, 16 * rng.randint(1, d // 16)))
        cuts = sorted(rng.randint(0, rot // 2) for _ in range(rng.randint(1, 3)))
        sections = [b - a for a, b in zip([0] + cuts, cuts + [rot // 2])]
        return _rope("", hkv * group, hkv, d, rot, tokens, " ".join(map(str, sections)), rng.random() < 0.5,
                     rng.random() < 0.3, shape_seed=seed)
    if op == "evict":
        hi = _log(rng, 2, 32768)
        seqs = _log(rng, 1, 128)
        while seqs > 1 and seqs * hi * hkv * d > 32 * 8192 * 8 * 128:
            seqs //= 2
        while hi > 2 and seqs * hi * hkv * d > 32 * 8192 * 8 * 128:
            hi //= 2
        budget = _log(rng, 1, hi)
        return _evict("", hkv, d, seqs, rng.randint(1, hi), hi, budget, rng.randint(0, budget), rng.random() < 0.5,
                      shape_seed=seed)
    group = rng.choice((1, 1, 2, 3, 4, 5, 7, 8, 12, 16))
    hkv = max(1, min(hkv, 64 // group))
    if op == "share":
        groups, members = _log(rng, 1, 8), _log(rng, 1, 64)
        prefix = _log(rng, 1, 32768)
        q = rng.choice((1, 1, 1, 2, 5, _log(rng, 1, 64)))
        own_hi = _log(rng, q, 1024)
        while groups > 1 and groups * prefix * hkv * d > 2 ** 27:
            groups //= 2
        while members > 1 and (groups * members * (prefix + own_hi) * hkv * d > 2 ** 30 or
                               groups * members * q * (prefix + own_hi) * hkv * group > 2 ** 28):
            members //= 2
        while prefix > 1 and groups * members * q * (prefix + own_hi) * hkv * group > 2 ** 28:
            prefix //= 2
        return _share("", hkv * group, hkv, d, groups, members, prefix, rng.randint(1, own_hi), own_hi, 1, q,
                      shape_seed=seed)
    if rng.random() < 0.6:
        q = rng.choice((1, 1, 1, 2, 3, 5))
        hi = _log(rng, q, 32768)
        seqs = _log(rng, 1, 256)
        while seqs > 1 and seqs * hi * hkv * d > 2 ** 29:
            seqs //= 2
        return _mass("", hkv * group, hkv, d, seqs, 1, q, max(q, rng.randint(1, hi)), hi, shape_seed=seed)
    hi = _log(rng, 16, 2048)
    seqs = _log(rng, 1, 16)
    while seqs > 1 and seqs * hi * hi * hkv * group > 2 ** 29:
        seqs //= 2
    if rng.random() < 0.5:
        return _mass("", hkv * group, hkv, d, seqs, 0, 0, rng.randint(1, hi), hi, prompt=True, shape_seed=seed)
    lo = rng.randint(1, hi)
    return _mass("", hkv * group, hkv, d, seqs, 1, _log(rng, 1, lo), lo, hi, shape_seed=seed)


def _lengths(case):
    """(query tokens, length in the cache) of every sequence."""
    r = random.Random(case["shape_seed"])
    if case["op"] == "share":
        got = []
        for _ in range(case["groups"] * case["members"]):
            after = r.randint(case["own_lo"], case["own_hi"])
            got.append((min(after, r.randint(case["q_lo"], case["q_hi"])), case["prefix"] + after))
        return got
    got = []
    for _ in range(case["seqs"]):
        kv = r.randint(case["kv_lo"], case["kv_hi"])
        if case["op"] == "evict":
            got.append((0, kv))
        else:
            got.append((kv if case["prompt"] else min(kv, r.randint(case["q_lo"], case["q_hi"])), kv))
    return got


def _pair_axes(case):
    """The axis of every rotation pair, from the sections."""
    left = [int(x) for x in case["sections"].split()]
    if not case["turns"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    got = []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                got.append(a)
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


def _grid_positions(g, tokens, axes, far, r):
    """Positions as a prompt with frames has them: time, then rows, then columns of a frame."""
    w = max(1, int(math.isqrt(max(1, tokens // 16))))
    t = torch.arange(tokens, device="cuda")
    grid = [t // (w * w), t // w % w, t % w]
    if axes <= 2:
        grid = grid[1:] if axes == 2 else [t]
    start = r.randint(0, far - tokens)
    pos = torch.stack([(grid[a] if a < len(grid) else t) + start for a in range(axes)])
    if tokens <= 256:  # single tokens of conversations that are at different places
        pos = torch.randint(0, far, (axes, tokens), generator=g, device="cuda")
    return pos


def prepare(case, seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    d, hkv = case["head_size"], case["kv_heads"]
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if case["op"] == "rope":
        t, hq, rot = case["tokens"], case["q_heads"], case["rot"]
        qkv = torch.randn((t, (hq + 2 * hkv) * d), generator=g, device="cuda").to(torch.bfloat16)
        far = 32768
        angle = torch.arange(far, device="cuda", dtype=torch.float64)[:, None] * (
            10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot))
        axis = _pair_axes(case)
        return {"case": case, "q": qkv[:, :hq * d].view(t, hq, d), "k": qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d),
                "positions": _grid_positions(g, t, len(case["sections"].split()), far, random.Random(seed)),
                "cos_sin": torch.cat([angle.cos(), angle.sin()], 1).float(),
                "pair_axis": bytes(axis), "axis": torch.tensor(axis, device="cuda"),
                "q_weight": (torch.rand(d, generator=g, device="cuda") + 0.5).to(torch.bfloat16),
                "k_weight": (torch.rand(d, generator=g, device="cuda") + 0.5).to(torch.bfloat16),
                "q_out": torch.empty((t, hq, d), **bf16), "k_out": torch.empty((t, hkv, d), **bf16), "status": status}
    lens = _lengths(case)
    shared = case["prefix"] // BLOCK if case["op"] == "share" else 0  # blocks that a group has in common
    need = [-(-kv // BLOCK) for _, kv in lens]
    width = max(need)
    spare = sum(-(-min(case["budget"], kv) // BLOCK) for _, kv in lens) if case["op"] == "evict" else 8
    blocks = sum(n - shared for n in need) + shared * case.get("groups", 0) + spare
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    n_own = torch.tensor([n - shared for n in need], device="cuda")
    col = torch.arange(width, device="cuda")
    first = n_own.cumsum(0) - n_own + shared * case.get("groups", 0)
    at = first[:, None] + col[None] - shared
    if shared:
        group = torch.arange(len(lens), device="cuda") // case["members"]
        at = torch.where(col[None] < shared, group[:, None] * shared + col[None], at)
    held = col[None] < torch.tensor(need, device="cuda")[:, None]
    table = torch.where(held, order[at.clamp(0, blocks - 1)], torch.full_like(order[:1], -1)).contiguous()
    gain = torch.exp(0.5 * torch.randn((hkv, d), generator=g, device="cuda"))  # some channels are larger than others
    k_cache, k_scale = _history(g, blocks, hkv, d, gain)
    s = {"case": case, "block_table": table, "k_cache": k_cache, "k_scale": k_scale,
         "seq_lens": torch.tensor([kv for _, kv in lens], dtype=torch.int32, device="cuda"),
         "max_len": max(kv for _, kv in lens), "status": status, "workspace": None}
    if case["op"] != "mass":
        s["v_cache"], s["v_scale"] = _history(g, blocks, hkv, d, 1.0)
    start = torch.tensor([0] + [n for n, _ in lens], device="cuda").cumsum(0).to(torch.int32)
    t = sum(n for n, _ in lens)
    s |= {"start_loc": start, "tokens": t, "max_n": max(n for n, _ in lens), "scale": 1.0 / math.sqrt(d)}
    room = width * BLOCK
    if case["op"] != "share":
        # heavy positions are few, the first ones among them; some have received nothing at all
        m = torch.exp(2.0 * torch.randn((len(lens), hkv, room), generator=g, device="cuda"))
        m[:, :, :4] *= 100.0
        m *= torch.rand(m.shape, generator=g, device="cuda") > 0.01
        s["mass"] = m * (16.0 / room) if case["op"] == "mass" else m  # what some calls before have left
    if case["op"] == "evict":
        top = torch.tensor([-(-min(case["budget"], kv) // BLOCK) for _, kv in lens], device="cuda")
        into = table
        if not case["in_place"]:
            at = blocks - spare + (top.cumsum(0) - top)[:, None] + col[None]
            into = torch.where(col[None] < top[:, None], order[at.clamp(0, blocks - 1)],
                               torch.full_like(order[:1], -1)).contiguous()
        s |= {"into": into, "mass_out": torch.zeros_like(s["mass"]),
              "new_lens": torch.zeros(len(lens), dtype=torch.int32, device="cuda"),
              "kept": torch.full((len(lens), hkv, case["budget"]), -1, dtype=torch.int32, device="cuda")}
        return s
    hq = case["q_heads"]
    s["q"] = torch.randn((t, hq, d), generator=g, device="cuda").to(torch.bfloat16)
    if case["op"] == "share":
        m = case["members"]
        s |= {"out": torch.empty((t, hq, d), **bf16), "lse": torch.empty((t, hq), dtype=torch.float32, device="cuda"),
              "group_start": torch.arange(case["groups"] + 1, dtype=torch.int32, device="cuda") * m,
              "prefix_lens": torch.full((case["groups"],), case["prefix"], dtype=torch.int32, device="cuda"),
              "max_group": max(sum(n for n, _ in lens[i * m:i * m + m]) for i in range(case["groups"]))}
    else:
        s["lse"] = _rows_to_tokens(s, _log_sum_exp(_scores(s))[..., None])[..., 0].contiguous()
    return s


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"rope": _plain_rope, "share": _plain_share, "mass": _plain_mass, "evict": _plain_evict}[op](state)


def _own(s, op):
    import int4_token_head_gb300 as kv

    c = s["case"]
    if op == "rope":
        kv.qk_norm_rope_axes(s["q"], s["k"], s["positions"], s["cos_sin"], s["pair_axis"], s["q_weight"], s["k_weight"],
                             EPS, s["q_out"], s["k_out"], interleaved=c["interleaved"], dev_status=s["status"])
        return s["q_out"], s["k_out"]
    if op == "evict":
        kv.evict_fp8(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["mass"], s["block_table"], s["seq_lens"],
                     c["budget"], c["recent"], s["into"], s["mass_out"], s["new_lens"], s["kept"],
                     dev_status=s["status"])
        return _evicted(s)
    if op == "mass":
        kv.attention_mass_fp8(s["q"], s["lse"], s["k_cache"], s["k_scale"], s["block_table"], s["seq_lens"],
                              s["start_loc"], s["max_n"], s["max_len"], s["scale"], s["mass"], dev_status=s["status"])
        return s["mass"]
    if s["workspace"] is None:
        size = kv.attention_shared_workspace_size(len(s["seq_lens"]), c["groups"], s["tokens"], c["q_heads"],
                                                  c["kv_heads"], c["head_size"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    kv.attention_fp8_shared(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"],
                            s["seq_lens"], s["start_loc"], s["max_n"], s["max_len"], s["group_start"], s["prefix_lens"],
                            s["max_group"], s["scale"], s["out"], s["workspace"], lse=s["lse"],
                            dev_status=s["status"])
    return s["out"], s["lse"]


def _plain_rope(s):
    rot = s["case"]["rot"]
    pair = torch.arange(rot // 2, device="cuda")
    at = s["positions"].t()[:, s["axis"]]                                # [tokens, pairs]
    cos, sin = s["cos_sin"][at, pair][:, None], s["cos_sin"][at, pair + rot // 2][:, None]

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


def _held(s, codes, scale):
    """Every sequence's keys or values [S, kv heads, positions, d], zeros behind its end."""
    table = s["block_table"].long().clamp(min=0)
    x = _values(codes.view(torch.uint8)[table]) * scale[table][:, :, None, :, None]
    here = torch.arange(table.shape[1] * BLOCK, device=table.device)[None] < s["seq_lens"][:, None]
    return torch.where(here[:, :, None, None], x.flatten(1, 2), torch.zeros((), device=x.device)).permute(0, 2, 1, 3)


def _scores(s):
    """softmax_scale q . k of every sequence's query rows [S, kv heads, query tokens x group, positions]; -inf where
    a row does not see a position."""
    c = s["case"]
    hkv, group = c["kv_heads"], c["q_heads"] // c["kv_heads"]
    start, length = s["start_loc"].long(), s["seq_lens"].long()
    n = start[1:] - start[:-1]
    j = torch.arange(s["max_n"], device=start.device)
    at = (start[:-1, None] + j[None]).clamp(max=s["tokens"] - 1)
    q = s["q"].float()[at].view(len(n), s["max_n"], hkv, group, c["head_size"]).permute(0, 2, 1, 3, 4)
    scores = (q.flatten(2, 3) @ _held(s, s["k_cache"], s["k_scale"]).transpose(2, 3)) * s["scale"]
    key = torch.arange(scores.shape[3], device=start.device)
    pos = (length - n)[:, None] + j[None]
    seen = (key[None, None] <= pos[:, :, None]) & (key[None, None] < length[:, None, None]) & (j[None] < n[:, None])[:, :, None]
    seen = seen[:, None, :, None].expand(-1, 1, -1, group, -1).flatten(2, 3)
    return scores.masked_fill_(~seen, -math.inf)


def _log_sum_exp(scores):
    top = scores.amax(-1, keepdim=True).clamp(min=-3e38)
    return top[..., 0] + torch.log(torch.exp(scores - top).sum(-1))


def _rows_to_tokens(s, x):
    """[S, kv heads, query tokens x group, ...] as [tokens, q heads, ...]."""
    hkv, group = s["case"]["kv_heads"], s["case"]["q_heads"] // s["case"]["kv_heads"]
    x = x.unflatten(2, (s["max_n"], group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    t = torch.arange(s["tokens"], device=x.device)
    start = s["start_loc"].long()
    seq = torch.searchsorted(start, t, right=True) - 1
    return x[seq, t - start[seq]]


def _plain_share(s):
    scores = _scores(s)
    lse = _log_sum_exp(scores)
    p = torch.exp(scores - lse.clamp(min=-3e38)[..., None])
    o = p @ _held(s, s["v_cache"], s["v_scale"])
    return _rows_to_tokens(s, o).to(torch.bfloat16), _rows_to_tokens(s, lse[..., None])[..., 0]


def _plain_mass(s):
    group = s["case"]["q_heads"] // s["case"]["kv_heads"]
    start, length = s["start_loc"].long(), s["seq_lens"].long()
    n = start[1:] - start[:-1]
    j = torch.arange(s["max_n"], device=start.device)
    at = (start[:-1, None] + j[None]).clamp(max=s["tokens"] - 1)
    lse = s["lse"][at].unflatten(2, (-1, group)).permute(0, 2, 1, 3).flatten(2, 3)     # [S, kv heads, rows]
    got = torch.exp(_scores(s) - lse[..., None]).sum(2)                                # [S, kv heads, positions]
    key = torch.arange(got.shape[2], device=start.device)
    here, before = key[None] < length[:, None], key[None] < (length - n)[:, None]
    m = s["mass"]
    m.copy_(torch.where(here[:, None], torch.where(before[:, None], m, torch.zeros_like(m)) + got, m))
    return m


def _evicted(s):
    return (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["mass_out"], s["new_lens"], s["kept"])


def _plain_evict(s):
    c = s["case"]
    budget, length, m = c["budget"], s["seq_lens"].long(), s["mass"]
    key = torch.arange(m.shape[2], device=m.device)
    last = key[None] >= (length - c["recent"])[:, None]
    here = key[None] < length[:, None]
    weight = torch.where(last[:, None], torch.full_like(m, math.inf), m)
    weight = torch.where(here[:, None], weight, torch.full_like(m, -math.inf))
    order = torch.sort(weight, dim=2, descending=True, stable=True).indices[:, :, :budget]
    n = length.clamp(max=budget)
    j = torch.arange(order.shape[2], device=m.device)
    valid = (j[None] < n[:, None])[:, None].expand_as(order)
    idx = torch.sort(torch.where(valid, order, torch.full_like(order, 1 << 40)), dim=2).values
    src = torch.where(valid, idx, torch.zeros_like(idx))
    seq, head = torch.arange(len(n), device=m.device)[:, None, None], torch.arange(m.shape[1], device=m.device)[None, :, None]
    s["mass_out"][:, :, :len(j)] = torch.where(valid, m.gather(2, src), s["mass_out"][:, :, :len(j)])
    s["kept"][:, :, :len(j)] = torch.where(valid, idx, s["kept"][:, :, :len(j)].long()).to(torch.int32)
    s["new_lens"].copy_(n)
    table, into = s["block_table"].long(), s["into"].long()
    blk = table[seq, src // BLOCK].clamp(min=0)
    pad = -len(j) % BLOCK
    moves = torch.nn.functional.pad(valid & (idx != j), (0, pad)).unflatten(2, (-1, BLOCK)).any(3)   # [S, H, blocks]
    live = torch.nn.functional.pad(valid, (0, pad)).unflatten(2, (-1, BLOCK)).any(3)
    to = into[:, :live.shape[2]].clamp(min=0)
    write = live & (moves | (to != table[:, :live.shape[2]])[:, None])
    row = valid & write.repeat_interleave(BLOCK, 2)[:, :, :len(j)]
    ws, wh, wj = row.nonzero(as_tuple=True)
    bs, bh, bj = write.nonzero(as_tuple=True)
    for codes, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
        codes = codes.view(torch.uint8)
        x = _values(codes[blk, src % BLOCK, head]) * scale[blk, head][..., None]          # [S, H, budget, d]
        x = torch.where(valid[..., None], x, torch.zeros((), device=x.device))
        top = torch.nn.functional.pad(x.abs().amax(3), (0, pad)).unflatten(2, (-1, BLOCK)).amax(3)
        k = _exponent(top)
        new = _codes(x * _two_to(-k).repeat_interleave(BLOCK, 2)[:, :, :len(j), None])
        codes[to[ws, wj // BLOCK], wj % BLOCK, wh] = new[ws, wh, wj]
        scale[to[bs, bj], bh] = _two_to(k)[bs, bh, bj]
    return _evicted(s)


# ---------------------------------------------------------------------------
# bytes and operations that a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    d, hkv = case["head_size"], case["kv_heads"]
    if case["op"] == "rope":
        t, h = case["tokens"], case["q_heads"] + hkv
        return {"bytes": t * (h * d * 4 + 8 * len(case["sections"].split()) + case["rot"] * 4),
                "flops": t * h * (4 * d + 3 * case["rot"])}
    lens = _lengths(case)
    if case["op"] == "evict":
        n = [min(kv, case["budget"]) for _, kv in lens]
        blocks = sum(-(-x // BLOCK) for x in n)
        total = hkv * (sum(kv for _, kv in lens) * 4 + sum(n) * (4 * d + 8) + blocks * 16)
        return {"bytes": total, "flops": hkv * sum(n) * d * 2}
    hq = case["q_heads"]
    t = sum(n for n, _ in lens)
    pairs = sum(n * kv - n * (n - 1) // 2 for n, kv in lens)
    if case["op"] == "mass":
        keys = sum(kv for _, kv in lens)
        return {"bytes": hkv * (keys * (d + 8) + sum(-(-kv // BLOCK) for _, kv in lens) * 4) + t * hq * (2 * d + 4),
                "flops": 2 * d * hq * pairs}
    prefix = case["prefix"] // BLOCK * BLOCK
    keys = sum(kv - prefix for _, kv in lens) + prefix * case["groups"]
    return {"bytes": keys * hkv * 2 * d + -(-keys // BLOCK) * (8 * hkv + 4) + t * hq * (4 * d + 4),
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


def _whole(codes, scale, row, kv):
    ids = row[: -(-kv // BLOCK)].long().cuda()
    return (_values(codes.view(torch.uint8)[ids]).double() * scale[ids].double()[:, None, :, None]).flatten(0, 1)[:kv]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        rot, half = case["rot"], case["rot"] // 2
        axis, both = _pair_axes(case), []
        for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
            x = x.double()
            y = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
            for i, a in enumerate(axis):
                lo, hi = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
                row = s["cos_sin"][s["positions"][a]].double()
                turn = torch.complex(row[:, i], row[:, i + half])
                z = torch.complex(y[..., lo], y[..., hi]) * turn[:, None]
                y[..., lo], y[..., hi] = z.real.clone(), z.imag.clone()
            both.append(y)
        return tuple(both)
    lens, tables = _lengths(case), s["block_table"].cpu()
    if case["op"] == "evict":
        return _exact_evict(case, s, lens, tables)
    group = case["q_heads"] // case["kv_heads"]
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    m, t = s["mass"].double() if case["op"] == "mass" else None, 0
    for i, ((n, kv), row) in enumerate(zip(lens, tables)):
        k = _whole(s["k_cache"], s["k_scale"], row, kv).repeat_interleave(group, 1)
        a = torch.einsum("qhd,khd->hqk", s["q"][t:t + n].double(), k) / math.sqrt(case["head_size"])
        gap = torch.arange(kv - n, kv, device="cuda")[:, None] - torch.arange(kv, device="cuda")[None]
        a.masked_fill_(gap < 0, -math.inf)
        if case["op"] == "mass":
            w = torch.exp(a - s["lse"][t:t + n].double().t()[:, :, None])
            m[i, :, kv - n:kv] = 0.0
            m[i, :, :kv] += w.view(-1, group, n, kv).sum((1, 2))
        else:
            v = _whole(s["v_cache"], s["v_scale"], row, kv).repeat_interleave(group, 1)
            lse[t:t + n] = torch.logsumexp(a, -1).t()
            out[t:t + n] = torch.einsum("hqk,khd->qhd", torch.softmax(a, -1), v)
        t += n
    return m if case["op"] == "mass" else (out, lse)


def _exact_evict(case, s, lens, tables):
    hkv, d, into = case["kv_heads"], case["head_size"], s["into"].cpu()
    mass, kept = s["mass_out"].double(), s["kept"].long()
    codes = {x: s[x + "_cache"].double() for x in "kv"}
    scale = {x: s[x + "_scale"].double() for x in "kv"}
    plan = []
    for i, (_, kv) in enumerate(lens):  # what is kept, before anything moves
        n, last = min(kv, case["budget"]), max(0, kv - case["recent"])
        take = n - (kv - last)
        rows = s["mass"][i].double()
        best = torch.argsort(-rows[:, :last], dim=1, stable=True)[:, :take]
        tail = torch.arange(last, kv, device="cuda").expand(hkv, -1)
        idx = torch.cat([best, tail], 1).sort(1).values
        mass[i, :, :n], kept[i, :, :n] = rows.gather(1, idx), idx
        got = {x: _whole(s[x + "_cache"], s[x + "_scale"], tables[i], kv) for x in "kv"}
        at = idx.t()[:, :, None].expand(-1, -1, d)
        plan.append((n, idx, {x: got[x].gather(0, at) for x in "kv"}))
    for i, (n, idx, got) in enumerate(plan):
        home = torch.arange(n, device="cuda")
        ids = into[i, : -(-n // BLOCK)].long().cuda()
        same = ids == tables[i, : -(-n // BLOCK)].long().cuda()
        stays = (idx == home).cpu()
        stays = torch.stack([stays[:, b * BLOCK:(b + 1) * BLOCK].all(1) for b in range(len(ids))], 1).cuda()  # [H, blocks]
        free = ~(stays & same)
        for x in "kv":
            y = torch.zeros((len(ids) * BLOCK, hkv, d), dtype=torch.float64, device="cuda")
            y[:n] = got[x]
            y = y.view(len(ids), BLOCK, hkv, d)
            top = y.abs().amax((1, 3))
            k = torch.ceil(torch.log2(top.clamp(min=2.0 ** -200) / 448.0)).clamp(MIN_EXP - 1, MAX_EXP)
            k = torch.where(448.0 * _power(k - 1) >= top, k - 1, k)  # log2 may round across a whole number
            k = torch.where(448.0 * _power(k) < top, k + 1, k).clamp(MIN_EXP, MAX_EXP)
            new = _e4m3(y / _power(k)[:, None, :, None])
            live = (torch.arange(len(ids) * BLOCK, device="cuda") < n).view(-1, BLOCK)
            put = live[:, :, None] & free.t()[:, None]
            codes[x][ids] = torch.where(put[..., None], new, codes[x][ids])
            scale[x][ids] = torch.where(free.t(), _power(k), scale[x][ids])
    lens = torch.tensor([n for n, _, _ in plan], dtype=torch.int32, device="cuda")
    return codes["k"], codes["v"], scale["k"], scale["v"], mass, lens, kept.to(torch.int32)
