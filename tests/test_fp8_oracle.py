"""Pins of the FP8 oracle (oracle/fp8_oracle.py) and the host-side refusals of
the FP8 entry points and kv_qk_norm_rope, through the C ABI and the binding.
No test here needs a GPU: every library call stops at validation."""

import ctypes

import numpy as np
import pytest
import torch

import int4_token_head_gb300 as kv
from int4_token_head_gb300 import _lib
from oracle import fp8_oracle as F

HEADS = [64, 96, 128, 192, 256]


# ---------------------------------------------------------------------------
# oracle
# ---------------------------------------------------------------------------
def test_e4m3_codes_round_trip_and_match_torch():
    codes = np.arange(256, dtype=np.uint8)
    ours = F.e4m3_values(codes)
    theirs = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(ours), np.isnan(theirs)) and np.isnan(ours).sum() == 2
    fine = ~np.isnan(ours)
    assert np.array_equal(ours[fine], theirs[fine])
    assert np.array_equal(F.e4m3_bytes(ours[fine]), codes[fine])


def test_e4m3_rounding_matches_torch_on_every_bf16_value_in_range():
    bits = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16)
    x = bits.view(torch.bfloat16)
    x = x[x.float().abs() <= 448].float()
    got = F.e4m3(x.double().numpy())
    assert np.array_equal(got, x.to(torch.float8_e4m3fn).double().numpy())


def test_exponent_is_the_smallest_that_holds_the_value():
    assert F.exponent(0.0) == -60
    assert F.exponent(448.0) == 0 and F.exponent(np.nextafter(448.0, 1e9)) == 1
    assert F.exponent(1.75) == -8 and F.exponent(1.76) == -7
    assert F.exponent(1e38) == 60


def test_write_hand_worked_growth():
    """Row 0 holds 1.75 (scale 2^-8, code 448); row 1 brings 7.5 (scale 2^-5),
    so row 0's code becomes 448 / 8 = 56."""
    codes, scale = np.full((2, 16, 1, 64), 0xFF, np.uint8), np.full((2, 1), np.nan, np.float32)
    x = np.zeros((1, 1, 64))
    x[0, 0, 3] = 1.75
    F.write(x, np.array([[1]]), [1], [0, 1], codes, scale)
    assert scale[1, 0] == 2.0 ** -8 and F.e4m3_values(codes[1, 0, 0, 3]) == 448
    x[0, 0, 3] = 7.5
    F.write(x, np.array([[1]]), [2], [0, 1], codes, scale)
    assert scale[1, 0] == 2.0 ** -5
    assert F.e4m3_values(codes[1, 0, 0, 3]) == 56 and F.e4m3_values(codes[1, 1, 0, 3]) == 240
    assert (codes[0] == 0xFF).all() and (codes[1, 2:] == 0xFF).all()
    assert np.array_equal(F.read(np.array([[1]]), 2, 0, codes, scale, 0)[:, 3], [1.75, 7.5])


def test_token_by_token_equals_at_once_but_for_subnormal_codes():
    g = np.random.default_rng(3)
    x = torch.from_numpy(g.standard_normal((40, 2, 64)) * np.exp(g.uniform(-2, 2, (40, 1, 1)))).to(torch.bfloat16)
    x = x.double().numpy()
    table = np.array([[2, 0, 1]])
    once = np.zeros((3, 16, 2, 64), np.uint8), np.zeros((3, 2), np.float32)
    F.write(x, table, [40], [0, 40], *once)
    step = np.zeros((3, 16, 2, 64), np.uint8), np.zeros((3, 2), np.float32)
    for t in range(40):
        F.write(x[t:t + 1], table, [t + 1], [0, 1], *step)
    assert np.array_equal(once[1], step[1])
    a, b = F.e4m3_values(once[0]), F.e4m3_values(step[0])
    off = a != b
    assert (np.abs(a[off]) < 2.0 ** -6 + 2.0 ** -9).all() and np.abs(a - b).max() <= 2.0 ** -9


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 5), (False, 0), (False, 3)])
def test_attention_against_literal_loops(causal, window):
    g = np.random.default_rng(5)
    hkv, group, d = 2, 3, 64
    table, lens, start = np.array([[3, 1], [0, 2]]), [21, 9], [0, 4, 6]
    kc, vc = (F.e4m3_bytes(F.e4m3(g.standard_normal((4, 16, hkv, d)) * 20)) for _ in range(2))
    ks, vs = (2.0 ** g.integers(-6, -3, (4, hkv)).astype(np.float32) for _ in range(2))
    q = g.standard_normal((6, hkv * group, d))
    got, bound = F.attention(q, (kc, vc, ks, vs), table, lens, start, 0.3, causal, window)
    for i in range(2):
        for t in range(start[i], start[i + 1]):
            pos = lens[i] - (start[i + 1] - start[i]) + t - start[i]
            for hq in range(hkv * group):
                w, o = [], []
                for p in range(lens[i]):
                    if (causal and p > pos) or (window and p <= pos - window):
                        continue
                    b, r, h = table[i, p // 16], p % 16, hq // group
                    kk = F.e4m3_values(kc[b, r, h]) * float(ks[b, h])
                    w.append(np.exp(0.3 * float(q[t, hq] @ kk)))
                    o.append(F.e4m3_values(vc[b, r, h]) * float(vs[b, h]))
                want = np.sum([a * b for a, b in zip(w, o)], 0) / np.sum(w)
                assert np.allclose(got[t, hq], want, rtol=1e-10, atol=1e-12)
    # weights sum to one and each is off by 2^-11 of itself and little more
    assert (bound > 0).all() and bound.max() < 2.0 ** -10 * np.abs(F.e4m3_values(vc)).max() * float(vs.max())


def test_norm_rope_is_a_rotation_of_the_normed_vector():
    g = np.random.default_rng(6)
    x = g.standard_normal((5, 3, 64))
    angle = g.uniform(-3, 3, (9, 16))
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    pos = np.array([8, 0, 3, 3, 5])
    for inter in (False, True):
        y = F.norm_rope(x, np.ones(64), 0.0, table, pos, inter)
        assert np.allclose((y * y).mean(-1), 1.0)
        back = F.norm_rope(y, None, 0.0, np.concatenate([np.cos(angle), -np.sin(angle)], 1), pos, inter)
        assert np.allclose(back, x / np.sqrt((x * x).mean(-1, keepdims=True)))


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10008)   # 8-byte aligned only
ODDER = ctypes.c_void_p(0x10002)
OK, NULL, HEAD, HEADCNT, BS, ALIGN, WS, SIZE, ROT = 0, 1, 2, 3, 4, 5, 6, 7, 10


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def _cache_call(lib, name, **kw):
    a = dict(k=FAKE, ks=1024, v=FAKE, vs=1024, bt=FAKE, mb=8, sl=FAKE, st=FAKE, ns=2, nt=8, ml=4, kc=FAKE, vc=FAKE,
             ksc=FAKE, vsc=FAKE, nb=4, bs=16, hkv=8, d=128, status=None, stream=None)
    a.update(kw)
    cache = [a[x] for x in ("kc", "vc", "ksc", "vsc")]
    seqs = [a[x] for x in ("bt", "mb", "sl", "st", "ns", "nt", "ml")]
    toks = [a[x] for x in ("k", "ks", "v", "vs")]
    tail = [a[x] for x in ("nb", "bs", "hkv", "d", "status", "stream")]
    if name == "kv_fp8_write":
        return lib.kv_fp8_write(*toks, *seqs, *cache, *tail)
    return lib.kv_fp8_read(*cache, *seqs, *toks, *tail)


@pytest.mark.parametrize("name", ["kv_fp8_write", "kv_fp8_read"])
@pytest.mark.parametrize("kw,code", [
    (dict(ns=0), OK), (dict(nt=0), OK), (dict(nt=0, k=None, v=None), OK),
    (dict(nt=-1), SIZE), (dict(ns=-1), SIZE), (dict(ml=-1), SIZE), (dict(mb=-1), SIZE), (dict(nb=-1), SIZE),
    (dict(mb=1 << 27), SIZE), (dict(nt=1 << 30, hkv=8), SIZE),
    (dict(hkv=0), HEADCNT), (dict(d=80), HEAD), (dict(d=0), HEAD), (dict(bs=32), BS),
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(kc=None), NULL), (dict(vsc=None), NULL), (dict(bt=None), NULL),
    (dict(sl=None), NULL), (dict(st=None), NULL),
    (dict(k=ODD), ALIGN), (dict(v=ODD), ALIGN), (dict(kc=ODD), ALIGN), (dict(ks=1025), ALIGN), (dict(vs=-8), ALIGN),
    (dict(ksc=ODDER), ALIGN), (dict(bt=ODDER), ALIGN), (dict(status=ODDER), ALIGN),
])
def test_cache_call_refusals(lib, name, kw, code):
    assert _cache_call(lib, name, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(ns=0), OK), (dict(nt=0), OK), (dict(nt=-1), SIZE), (dict(mq=-1), SIZE), (dict(ms=-1), SIZE),
    (dict(win=-1), SIZE), (dict(hq=30), HEADCNT), (dict(hq=8 * 65), HEADCNT), (dict(hkv=0), HEADCNT),
    (dict(d=100), HEAD), (dict(bs=8), BS), (dict(q=None), NULL), (dict(out=None), NULL), (dict(kc=None), NULL),
    (dict(ksc=None), NULL), (dict(ws=None), WS), (dict(wsb=1024), WS), (dict(q=ODD), ALIGN), (dict(out=ODD), ALIGN),
    (dict(os=4097), ALIGN), (dict(ws=ctypes.c_void_p(0x10010)), ALIGN), (dict(sl=ODDER), ALIGN),
])
def test_attention_refusals(lib, kw, code):
    a = dict(q=FAKE, qs=4096, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, bt=FAKE, mb=8, sl=FAKE, st=FAKE, ns=2, nt=8, mq=4,
             ms=128, hq=32, hkv=8, d=128, bs=16, nb=16, sc=0.1, causal=1, win=0, out=FAKE, os=4096, ws=FAKE,
             wsb=1 << 40, status=None, stream=None)
    a.update(kw)
    assert lib.kv_fp8_attention(*a.values()) == code


@pytest.mark.parametrize("kw,code", [
    (dict(nt=0), OK), (dict(nt=0, q=None), OK), (dict(nt=-1), SIZE), (dict(eps=-1.0), SIZE),
    (dict(eps=float("nan")), SIZE), (dict(mp=-1), SIZE), (dict(hq=0), HEADCNT), (dict(hkv=0), HEADCNT),
    (dict(d=72), HEAD), (dict(rot=24), ROT), (dict(rot=144), ROT), (dict(rot=-16), ROT), (dict(q=None), NULL),
    (dict(ko=None), NULL), (dict(qw=None), NULL), (dict(kw_=None), NULL), (dict(pos=None), NULL), (dict(cs=None), NULL),
    (dict(q=ODD), ALIGN), (dict(ko=ODD), ALIGN), (dict(qw=ODD), ALIGN), (dict(cs=ODD), ALIGN),
    (dict(pos=ctypes.c_void_p(0x10004)), ALIGN), (dict(ks=1028), ALIGN), (dict(nt=1 << 30), SIZE),
])
def test_norm_rope_refusals(lib, kw, code):
    a = dict(q=FAKE, qs=4096, k=FAKE, ks=1024, nt=4, hq=32, hkv=8, d=128, qw=FAKE, kw_=FAKE, eps=1e-6, pos=FAKE,
             cs=FAKE, mp=64, rot=128, inter=0, qo=FAKE, qos=4096, ko=FAKE, kos=1024, status=None, stream=None)
    a.update(kw)
    assert lib.kv_qk_norm_rope(*a.values()) == code


def _cpu(hkv=2, d=64, seqs=2, t=3):
    bf = torch.bfloat16
    return dict(k=torch.zeros(t, hkv, d, dtype=bf), v=torch.zeros(t, hkv, d, dtype=bf),
                bt=torch.zeros(seqs, 2, dtype=torch.int32), sl=torch.ones(seqs, dtype=torch.int32),
                st=torch.zeros(seqs + 1, dtype=torch.int32), kc=torch.zeros(4, 16, hkv, d, dtype=torch.uint8),
                vc=torch.zeros(4, 16, hkv, d, dtype=torch.uint8), ks=torch.ones(4, hkv), vs=torch.ones(4, hkv))


def test_binding_refuses_bad_tensors():
    def write(**kw):
        a = _cpu()
        a.update(kw)
        kv.write_fp8(a["k"], a["v"], a["bt"], a["sl"], a["st"], 2, a["kc"], a["vc"], a["ks"], a["vs"])

    c = _cpu()
    for kw, what in [
        (dict(), "CUDA device"), (dict(k=c["k"].float()), "bfloat16"), (dict(k=c["k"][:, :1]), "k must be"),
        (dict(v=c["v"][:2]), "disagree"), (dict(kc=c["kc"].to(torch.int8)), "float8"),
        (dict(vc=c["vc"][:3]), "caches must be"), (dict(ks=torch.ones(4, 16, 2)), "scale caches"),
        (dict(vs=torch.ones(4, 2).double()), "scale caches"), (dict(bt=c["bt"].long()), "block_table"),
        (dict(bt=c["bt"][:1]), "metadata"), (dict(sl=c["sl"].long()), "int32"), (dict(st=c["st"][:2]), "metadata"),
        (dict(kc=c["kc"].transpose(1, 2).contiguous().transpose(1, 2)), "contiguous"),
    ]:
        with pytest.raises(ValueError, match=what):
            write(**kw)
    a = _cpu()
    with pytest.raises(ValueError, match="CUDA device"):
        kv.read_fp8(a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["sl"], a["st"], 2, a["k"], a["v"])
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    ws = torch.zeros(16, dtype=torch.uint8)
    for qq, out, w, what in [(q, q, ws, "CUDA device"), (q, q[:2], ws, "out must have"), (q[0], q, ws, "q must be"),
                             (q, q, ws.int(), "workspace"), (q, q.float(), ws, "bfloat16")]:
        with pytest.raises(ValueError, match=what):
            kv.attention_fp8(qq, a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["sl"], a["st"], 2, 16, 0.1, True, out, w)
    pos, cs, w = torch.zeros(3, dtype=torch.int64), torch.zeros(8, 64), torch.ones(64, dtype=torch.bfloat16)
    k = a["k"]
    for args, what in [((q, k, pos, cs, w, w, 0.0, q, k), "CUDA device"), ((q, k, pos, cs, w, None, 0.0, q, k), "both"),
                       ((q, k, None, cs, w, w, 0.0, q, k), "both"), ((q, k, pos.int(), cs, w, w, 0.0, q, k), "int64"),
                       ((q, k, pos, cs.double(), w, w, 0.0, q, k), "float32"),
                       ((q, k, pos, cs, w[:32], w, 0.0, q, k), "weights"), ((q, k[:2], pos, cs, w, w, 0.0, q, k), "disagree"),
                       ((q, k, pos, cs, w, w, 0.0, k, k), "q_out")]:
        with pytest.raises(ValueError, match=what):
            kv.qk_norm_rope(*args)


def test_paged_cache_refuses_slot_writes_for_fp8():
    from int4_token_head_gb300 import synthetic
    from int4_token_head_gb300.paged import PagedKV
    pk = PagedKV(synthetic.custom_workload(4, 2, 64, [(1, 20)]), device="cpu", fmt="fp8")
    assert pk.k_cache.dtype == torch.float8_e4m3fn and tuple(pk.k_scale.shape) == (pk.w.num_blocks, 2)
    with pytest.raises(ValueError, match="write_tokens"):
        pk.write(None, None, None)
    with pytest.raises(ValueError, match="unknown cache format"):
        PagedKV(pk.w, device="cpu", fmt="fp16")


# ---------------------------------------------------------------------------
# workspaces
# ---------------------------------------------------------------------------
def _int4_workspace(seqs, tokens, hq, hkv, d):
    """The INT4 attention's parts, each rounded up to 256 bytes: schedule, rotated
    queries, eight columns per (sequence, kv head) and for each of 4096 warps."""
    items = (tokens // max(1, 64 // (hq // hkv)) + seqs) * hkv
    columns = 8 * seqs * hkv
    parts = (256, 16 * seqs, 8 * (seqs + 1), 16 * items, 8 * items, 2 * tokens * hq * d, 4 * columns * d, 8 * columns,
             4 * 4096 * 8 * d, 8 * 4096 * 8)
    return sum(-(-x // 256) * 256 for x in parts)


@pytest.mark.parametrize("sizes", [(1, 1, 32, 8, 128), (64, 64, 16, 8, 256), (8, 9000, 32, 8, 128), (300, 300, 12, 1, 96),
                                   (1, 1, 1, 1, 64), (3, 70, 64, 1, 192)])
def test_int4_callers_do_not_pay_for_the_fp8_workspace(lib, sizes):
    assert lib.kv_int4_attention_workspace_size(*sizes) == _int4_workspace(*sizes)
    for fmt in ("int4", "int8"):
        assert kv.attention_workspace_size(*sizes, fmt=fmt) == _int4_workspace(*sizes)
    best = lib.kv_fp8_attention_workspace_size(*sizes)
    assert kv.attention_workspace_size(*sizes, fmt="fp8") == best > 0
    assert kv.attention_workspace_size(*sizes) == max(best, _int4_workspace(*sizes))


def test_workspace_sizes_refuse_what_no_call_takes(lib):
    assert lib.kv_fp8_attention_workspace_size(4, 4, 32, 7, 128) == 0
    assert lib.kv_fp8_attention_workspace_size(4, 4, 32, 8, 100) == 0
    assert lib.kv_fp8_attention_workspace_size(-1, 4, 32, 8, 128) == 0
    assert kv.attention_workspace_size(4, -4, 32, 8, 128) == 0
    with pytest.raises(ValueError, match="format"):
        kv.attention_workspace_size(4, 4, 32, 8, 128, fmt="fp4")


def test_paged_caches_hold_their_own_workspace():
    from int4_token_head_gb300 import synthetic
    from int4_token_head_gb300.paged import PagedKV
    w = synthetic.custom_workload(4, 2, 64, [(1, 20), (3, 9)])
    for fmt in ("int4", "int8", "fp8"):
        assert PagedKV(w, device="cpu", fmt=fmt).workspace.numel() == kv.attention_workspace_size(2, 4, 4, 2, 64, fmt=fmt)


@pytest.mark.parametrize("big", [1 << 31, (1 << 32) + 5, -(1 << 31) - 1])
def test_binding_refuses_counts_beyond_32_bits(big):
    """They would reach the library without their upper bits."""
    a = _cpu()
    cache, seqs = [a[x] for x in ("kc", "vc", "ks", "vs")], [a[x] for x in ("bt", "sl", "st")]
    q, ws = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="max_len must fit"):
        kv.write_fp8(a["k"], a["v"], *seqs, big, *cache)
    with pytest.raises(ValueError, match="max_len must fit"):
        kv.read_fp8(*cache, *seqs, big, a["k"], a["v"])
    for name, counts, window in (("max_query_len", (big, 16), 0), ("max_seq_len", (2, big), 0), ("sliding_window", (2, 16), big)):
        with pytest.raises(ValueError, match=f"{name} must fit"):
            kv.attention_fp8(q, *cache, *seqs, *counts, 0.1, True, q, ws, sliding_window=window)
    with pytest.raises(ValueError, match="CUDA device"):  # any whole number will do
        kv.write_fp8(a["k"], a["v"], *seqs, np.int64(2), *cache)
