"""Pins of the oracle's axes, masses and evictions, and the host-side refusals of
kv_qk_norm_rope_axes, kv_fp8_attention_shared, kv_fp8_attention_mass and
kv_fp8_evict (no GPU: everything is refused, or a no-op, before a launch)."""

import ctypes
import math

import numpy as np
import pytest
import torch

import int4_token_head_gb300 as kv
from int4_token_head_gb300 import _lib
from oracle import fp8_oracle as F

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first
FAKE2 = ctypes.c_void_p(0x20000)
ODD = ctypes.c_void_p(0x10008)   # 8-byte aligned only
ODDER = ctypes.c_void_p(0x10002)
OK, NULL, HEAD, HEADCNT, BS, ALIGN, WS, SIZE, ROT = 0, 1, 2, 3, 4, 5, 6, 7, 10


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


# ---------------------------------------------------------------------------
# the oracle
# ---------------------------------------------------------------------------
def test_rope_axes_lays_the_pairs_out():
    assert kv.rope_axes((2, 1, 3)) == bytes([0, 0, 1, 2, 2, 2])
    assert kv.rope_axes((4, 2, 2), turns=True) == bytes([0, 1, 2, 0, 1, 2, 0, 0])
    assert kv.rope_axes((0, 2, 1), turns=True) == bytes([1, 2, 1])
    assert kv.rope_axes(()) == kv.rope_axes((), turns=True) == b""
    for turns in (False, True):
        pairs = kv.rope_axes((24, 20, 20), turns)
        assert [pairs.count(a) for a in range(3)] == [24, 20, 20]
    assert kv.rope_axes((24, 20, 20), True)[-4:] == bytes(4)
    with pytest.raises(ValueError, match="negative"):
        kv.rope_axes((3, -1))


@pytest.mark.parametrize("inter", [False, True])
def test_oracle_axes_turn_every_pair_by_its_axis(inter):
    g = np.random.default_rng(3)
    x, angle = g.standard_normal((4, 2, 64)), g.uniform(-3, 3, (9, 16))
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    pos, pairs = g.integers(0, 9, (3, 4)), kv.rope_axes((6, 5, 5), turns=True)
    y = F.norm_rope_axes(x, None, 0.0, table, pos, pairs, inter)
    for t in range(4):
        for i in range(16):
            lo, hi = (2 * i, 2 * i + 1) if inter else (i, i + 16)
            z = (x[t, :, lo] + 1j * x[t, :, hi]) * np.exp(1j * angle[pos[pairs[i], t], i])
            assert np.allclose(y[t, :, lo], z.real) and np.allclose(y[t, :, hi], z.imag)
    assert (y[..., 32:] == x[..., 32:]).all()
    w = g.uniform(0.5, 2, 64)
    assert np.array_equal(F.norm_rope_axes(x, w, 1e-3, table, pos[[1] * 3], pairs, inter),
                          F.norm_rope(x, w, 1e-3, table, pos[1], inter))


def _cache(d=64, hkv=2, blocks=6, seed=0):
    g = np.random.default_rng(seed)
    codes = F.e4m3_bytes(F.e4m3(g.uniform(-300, 300, (blocks, 16, hkv, d))))
    return codes, np.ldexp(1.0, g.integers(-9, -6, (blocks, hkv))).astype(np.float32)


def test_oracle_masses_and_denominators_follow_the_formula():
    codes, scale = _cache()
    table = np.array([[2, 0], [5, 9]], np.int32)  # 9: no such block
    lens, start, sm = [20, 18], [0, 3, 5], 0.05
    q = np.random.default_rng(1).standard_normal((5, 4, 64))
    lse, bound = F.log_sum_exp(q, codes, scale, table, lens, start, sm)
    m0 = np.random.default_rng(2).uniform(0, 1, (2, 2, 24))
    skip = lse.copy()
    skip[1, 2] = math.inf
    got, err = F.mass(q, skip, codes, scale, table, lens, start, sm, m0)
    want = m0.copy()
    for i, (a, b) in enumerate(((0, 3), (3, 5))):
        for h in range(2):
            for p in range(lens[i]):
                own = p >= lens[i] - (b - a)
                total = 0.0 if own else m0[i, h, p]
                blk = table[i, p // 16]
                for t in range(a, b):
                    if p > lens[i] - (b - a) + t - a or blk >= 6:
                        continue
                    key = F.e4m3_values(codes[blk, p % 16, h]) * scale[blk, h]
                    for hq in (2 * h, 2 * h + 1):
                        if np.isfinite(skip[t, hq]):
                            total += math.exp(sm * (q[t, hq] @ key) - skip[t, hq])
                want[i, h, p] = total
    assert np.allclose(got, want, rtol=1e-12) and (got[:, :, 20:] == m0[:, :, 20:]).all()
    assert (bound > 0).all() and (bound < 1e-4).all() and (err[0, :, :20] > 0).all()
    for t, n in ((0, 18), (2, 20)):  # a row's weights add up to one
        s = [sm * (q[t, 3] @ (F.e4m3_values(codes[table[0, p // 16], p % 16, 1]) * scale[table[0, p // 16], 1]))
             for p in range(n)]
        assert math.isclose(sum(math.exp(x - lse[t, 3]) for x in s), 1.0, rel_tol=1e-12)
    alone, _ = F.log_sum_exp(q[:1], codes, scale, np.array([[9]]), [1], [0, 1], sm)
    assert (alone == -np.inf).all()


def test_oracle_keeps_the_heaviest_and_the_last():
    m = np.array([3.0, 1.0, 2.0, 2.0, math.nan, 0.0, 9.0, 9.0])
    assert F.keep(m, 8, 8, 0).tolist() == list(range(8))
    assert F.keep(m, 8, 5, 2).tolist() == [0, 2, 3, 6, 7]
    assert F.keep(m, 8, 4, 2).tolist() == [0, 2, 6, 7]           # of equal ones the first
    assert F.keep(m, 6, 5, 0).tolist() == [0, 1, 2, 3, 5]        # NaN goes first
    assert F.keep(m, 6, 1, 1).tolist() == [5]
    assert F.keep(np.array([math.nan, -math.inf, math.inf, -0.0, 0.0]), 5, 3, 0).tolist() == [2, 3, 4]


def test_oracle_eviction_moves_rows():
    codes, scale = _cache(blocks=5)
    caches = [codes, codes[::-1].copy(), scale, scale[::-1].copy()]
    before = [x.copy() for x in caches]
    table, into = np.array([[1, 3], [0, 0]], np.int32), np.array([[4], [2]], np.int32)
    m = np.zeros((2, 2, 32))
    m[0, 0, [3, 18, 19]], m[0, 1, [0, 1, 2]] = 1.0, 1.0
    out, kept = np.full((2, 2, 5), -7.0), np.full((2, 2, 5), -7)
    new = F.evict(caches, m, table, [22, 2], 5, 2, into, out, kept)
    assert new.tolist() == [5, 2]
    assert kept[0].tolist() == [[3, 18, 19, 20, 21], [0, 1, 2, 20, 21]]
    assert kept[1].tolist() == [[0, 1, -7, -7, -7]] * 2 and (out[1, :, 2:] == -7).all()
    assert out[0].tolist() == [[1, 1, 1, 0, 0]] * 2
    for j, p in enumerate((3, 18, 19, 20, 21)):
        src = (1, 3)[p // 16]
        for c in (0, 1):
            old = F.e4m3_values(before[c][src, p % 16, 0]) * before[c + 2][src, 0]
            have = F.e4m3_values(caches[c][4, j, 0]) * caches[c + 2][4, 0]
            assert np.abs(have - old).max() <= 2.0 ** -4 * np.abs(old).max()
    assert (caches[0][4, 5:] == before[0][4, 5:]).all() and (caches[0][[1, 3, 0]] == before[0][[1, 3, 0]]).all()


# ---------------------------------------------------------------------------
# refusals of the library
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kw,code", [
    (dict(nt=0), OK), (dict(nt=0, q=None, pa=None), OK), (dict(nt=-1), SIZE), (dict(eps=-1.0), SIZE),
    (dict(eps=float("nan")), SIZE), (dict(mp=-1), SIZE), (dict(hq=0), HEADCNT), (dict(hkv=-1), HEADCNT),
    (dict(d=72), HEAD), (dict(rot=24), ROT), (dict(rot=144), ROT), (dict(rot=-16), ROT), (dict(rot=1 << 30), ROT),
    (dict(axes=0), ROT), (dict(axes=5), ROT), (dict(axes=-1), ROT), (dict(axes=2), ROT), (dict(pas=-1), SIZE),
    (dict(pa=None), NULL), (dict(pa=bytes([3]) + bytes(63)), ROT), (dict(pa=bytes(63) + b"\xff"), ROT),
    (dict(rot=0, pa=None, pos=None, cs=None, nt=0), OK), (dict(q=None), NULL), (dict(ko=None), NULL), (dict(qw=None), NULL),
    (dict(kw_=None), NULL), (dict(pos=None), NULL), (dict(cs=None), NULL), (dict(q=ODD), ALIGN), (dict(ko=ODD), ALIGN),
    (dict(kw_=ODD), ALIGN), (dict(cs=ODD), ALIGN), (dict(pos=ctypes.c_void_p(0x10004)), ALIGN), (dict(qos=4100), ALIGN),
    (dict(status=ODDER), ALIGN), (dict(nt=1 << 30), SIZE),
])
def test_norm_rope_axes_refusals(lib, kw, code):
    a = dict(q=FAKE, qs=4096, k=FAKE, ks=1024, nt=4, hq=32, hkv=8, d=128, qw=FAKE, kw_=FAKE, eps=1e-6, pos=FAKE, pas=4,
             axes=3, pa=kv.rope_axes((24, 20, 20)), cs=FAKE, mp=64, rot=128, inter=0, qo=FAKE, qos=4096, ko=FAKE, kos=1024,
             status=None, stream=None)
    a.update(kw)
    assert lib.kv_qk_norm_rope_axes(*a.values()) == code


@pytest.mark.parametrize("kw,code", [
    (dict(ns=0), OK), (dict(nt=0), OK), (dict(nt=0, q=None, gs=None), OK), (dict(nt=-1), SIZE), (dict(ns=-1), SIZE),
    (dict(mq=-1), SIZE), (dict(ms=-1), SIZE), (dict(mb=-1), SIZE), (dict(mb=1 << 27), SIZE), (dict(ng=-1), SIZE),
    (dict(ng=1025), SIZE), (dict(mg=-1), SIZE), (dict(nb=0), SIZE), (dict(nb=-1), SIZE), (dict(nb=1 << 27), SIZE),
    (dict(qs=4088), SIZE), (dict(os=0), SIZE), (dict(ls=31), SIZE), (dict(nt=1 << 26), SIZE), (dict(hq=30), HEADCNT),
    (dict(hq=8 * 65), HEADCNT), (dict(hkv=0), HEADCNT), (dict(d=100), HEAD), (dict(bs=8), BS), (dict(q=None), NULL),
    (dict(out=None), NULL), (dict(kc=None), NULL), (dict(vsc=None), NULL), (dict(st=None), NULL), (dict(gs=None), NULL),
    (dict(pl=None), NULL), (dict(ws=None), WS), (dict(wsb=1024), WS), (dict(q=ODD), ALIGN), (dict(out=ODD), ALIGN),
    (dict(vc=ODD), ALIGN), (dict(qs=4097), ALIGN), (dict(os=4100), ALIGN), (dict(ws=ctypes.c_void_p(0x10010)), ALIGN),
    (dict(sl=ODDER), ALIGN), (dict(gs=ODDER), ALIGN), (dict(pl=ODDER), ALIGN), (dict(lse=ODDER), ALIGN),
    (dict(status=ODDER), ALIGN),
])
def test_shared_attention_refusals(lib, kw, code):
    a = dict(q=FAKE, qs=4096, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, bt=FAKE, mb=8, sl=FAKE, st=FAKE, ns=4, nt=8, mq=4,
             ms=128, gs=FAKE, pl=FAKE, ng=2, mg=8, hq=32, hkv=8, d=128, bs=16, nb=16, sc=0.1, out=FAKE, os=4096, lse=FAKE,
             ls=32, ws=FAKE, wsb=1 << 40, status=None, stream=None)
    a.update(kw)
    assert lib.kv_fp8_attention_shared(*a.values()) == code


@pytest.mark.parametrize("kw,code", [
    (dict(ns=0), OK), (dict(nt=0), OK), (dict(nt=0, q=None, lse=None, mass=None), OK), (dict(nt=-1), SIZE),
    (dict(mq=-1), SIZE), (dict(ms=-1), SIZE), (dict(ml=-1), SIZE), (dict(nb=-1), SIZE), (dict(mb=1 << 27), SIZE),
    (dict(ls=-1), SIZE), (dict(mss=-1), SIZE), (dict(mhs=-1), SIZE), (dict(hq=30), HEADCNT), (dict(hq=8 * 65), HEADCNT),
    (dict(hkv=0), HEADCNT), (dict(d=32), HEAD), (dict(bs=32), BS), (dict(q=None), NULL), (dict(lse=None), NULL),
    (dict(kc=None), NULL), (dict(ksc=None), NULL), (dict(bt=None), NULL), (dict(mass=None), NULL), (dict(q=ODD), ALIGN),
    (dict(qs=4097), ALIGN), (dict(kc=ODD), ALIGN), (dict(lse=ODDER), ALIGN), (dict(mass=ODDER), ALIGN),
    (dict(status=ODDER), ALIGN),
    (dict(mhs=127), SIZE), (dict(mss=1023), SIZE), (dict(mss=0), SIZE), (dict(mss=128, mhs=128), SIZE),
    (dict(mss=128, mhs=255), SIZE), (dict(nt=1 << 26), SIZE),
])
def test_mass_refusals(lib, kw, code):
    a = dict(q=FAKE, qs=4096, lse=FAKE, ls=32, kc=FAKE, ksc=FAKE, bt=FAKE, mb=8, sl=FAKE, st=FAKE, ns=2, nt=8, mq=4, ms=128,
             hq=32, hkv=8, d=128, bs=16, nb=16, sc=0.1, mass=FAKE, mss=1024, mhs=128, ml=128, status=None, stream=None)
    a.update(kw)
    assert lib.kv_fp8_attention_mass(*a.values()) == code


@pytest.mark.parametrize("kw,code", [
    (dict(ns=0), OK), (dict(ns=0, mass=None, kept=None), OK), (dict(ns=-1), SIZE), (dict(bud=0), SIZE), (dict(bud=-3), SIZE),
    (dict(rec=-1), SIZE), (dict(rec=65), SIZE), (dict(ml=-1), SIZE), (dict(mb=-1), SIZE), (dict(dmb=-1), SIZE),
    (dict(dmb=3), SIZE), (dict(nb=-1), SIZE), (dict(hkv=0), HEADCNT), (dict(d=80), HEAD), (dict(bs=32), BS),
    (dict(mss=-1), SIZE), (dict(ohs=-1), SIZE), (dict(kc=None), NULL), (dict(vsc=None), NULL), (dict(mass=None), NULL),
    (dict(bt=None), NULL), (dict(sl=None), NULL), (dict(dbt=None), NULL), (dict(mo=None), NULL), (dict(nl=None), NULL),
    (dict(kept=None), NULL), (dict(vc=ODD), ALIGN), (dict(mass=ODDER), ALIGN), (dict(mo=ODDER), ALIGN),
    (dict(kept=ODDER), ALIGN), (dict(dbt=ODDER), ALIGN), (dict(nl=ODDER), ALIGN), (dict(status=ODDER), ALIGN),
    (dict(nl=FAKE), SIZE), (dict(ohs=63), SIZE), (dict(oss=511), SIZE), (dict(oss=64, ohs=64), SIZE), (dict(mo=FAKE), SIZE),
    (dict(ns=1 << 23, mss=1 << 40), SIZE),
])
def test_evict_refusals(lib, kw, code):
    a = dict(kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, nb=16, bs=16, hkv=8, d=128, mass=FAKE, mss=1024, mhs=128, ml=128, bt=FAKE,
             mb=8, sl=FAKE, ns=2, bud=64, rec=16, dbt=FAKE, dmb=4, mo=FAKE2, oss=512, ohs=64, nl=FAKE2, kept=FAKE,
             status=None, stream=None)
    a.update(kw)
    assert lib.kv_fp8_evict(*a.values()) == code


def test_a_destination_holds_what_can_be_kept(lib):
    """No more blocks than the budget, the masses or the table allow (a call of no sequences launches nothing)."""
    for ml, mb, bud, need in ((128, 8, 64, 4), (128, 8, 65, 5), (128, 8, 500, 8), (40, 8, 500, 3), (128, 2, 500, 2), (0, 8, 5, 0)):
        for dmb in (need, need - 1):
            got = lib.kv_fp8_evict(FAKE, FAKE, FAKE, FAKE, 16, 16, 8, 128, FAKE, 1024, 128, ml, FAKE, mb, FAKE, 0, bud, 1,
                                   FAKE, dmb, FAKE2, 512, 64, FAKE2, FAKE, None, None)
            assert got == (OK if dmb == need else SIZE)


def test_lengths_whose_loops_would_leave_32_bits_are_refused(lib):
    """Masses and evictions of sequences of up to 2^31 - 2^16 positions, by the smallest bound of their lengths (calls
    of no sequences launch nothing)."""
    top, wide = (1 << 31) - 1, (1 << 27) - 1
    for ml, mb, ms, ok in ((top, wide, top, False), (top - (1 << 16) + 1, wide, top, True), (top - (1 << 16) + 2, wide, top, False),
                           (top, wide - (1 << 12) + 1, top, True), (top, wide - (1 << 12) + 2, top, False), (1000, wide, top, True)):
        assert lib.kv_fp8_evict(FAKE, FAKE, FAKE, FAKE, 16, 16, 8, 128, FAKE, ml, ml, ml, FAKE, mb, FAKE, 0, 64, 1, FAKE, 4,
                                FAKE2, 64, 64, FAKE2, FAKE, None, None) == (OK if ok else SIZE)
    for ml, mb, ms, ok in ((top, wide, top, False), (top, wide, top - (1 << 16) + 1, True), (top, wide, top - (1 << 16) + 2, False),
                           (top, 1000, top, True), (5, wide, top, True)):
        assert lib.kv_fp8_attention_mass(FAKE, 4096, FAKE, 32, FAKE, FAKE, FAKE, mb, FAKE, FAKE, 0, 8, 4, ms, 32, 8, 128, 16,
                                         16, 0.1, FAKE, ml, ml, ml, None, None) == (OK if ok else SIZE)


def test_shared_workspace_sizes(lib):
    size = lib.kv_fp8_attention_shared_workspace_size
    assert size(4, 2, 4, 32, 8, 128) == kv.attention_shared_workspace_size(4, 2, 4, 32, 8, 128) > 0
    assert size(0, 0, 0, 32, 8, 128) > 0
    for bad in ((4, 2, 4, 32, 7, 128), (4, 2, 4, 32, 8, 100), (-1, 2, 4, 32, 8, 128), (4, -1, 4, 32, 8, 128),
                (4, 2, -4, 32, 8, 128), (4, 2, 4, 0, 8, 128), (4, 2, 4, 32, 0, 128)):
        assert size(*bad) == 0, bad
    with pytest.raises(ValueError, match="sizes"):
        kv.attention_shared_workspace_size(4, 2, 4, 32, 7, 128)
    with pytest.raises(ValueError, match="32 bits"):
        kv.attention_shared_workspace_size(1 << 40, 2, 4, 32, 8, 128)


# ---------------------------------------------------------------------------
# refusals of the binding
# ---------------------------------------------------------------------------
def _cpu(hkv=2, d=64, seqs=2, t=3):
    bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
    return dict(q=torch.zeros(t, 4, d, dtype=bf), lse=torch.zeros(t, 4), bt=torch.zeros(seqs, 2, dtype=i32),
                sl=torch.ones(seqs, dtype=i32), st=torch.zeros(seqs + 1, dtype=i32),
                kc=torch.zeros(4, 16, hkv, d, dtype=u8), vc=torch.zeros(4, 16, hkv, d, dtype=u8), ks=torch.ones(4, hkv),
                vs=torch.ones(4, hkv), mass=torch.zeros(seqs, hkv, 32), gs=torch.zeros(2, dtype=i32),
                pl=torch.zeros(1, dtype=i32), ws=torch.zeros(64, dtype=u8), dbt=torch.zeros(seqs, 1, dtype=i32),
                mo=torch.zeros(seqs, hkv, 8), nl=torch.zeros(seqs, dtype=i32), kept=torch.zeros(seqs, hkv, 8, dtype=i32),
                out=torch.zeros(t, 4, d, dtype=bf))


def _shared(**kw):
    a = {**_cpu(), "mq": 2, "ms": 32, "mg": 3, **kw}
    kv.attention_fp8_shared(*(a[x] for x in ("q", "kc", "vc", "ks", "vs", "bt", "sl", "st", "mq", "ms", "gs", "pl", "mg")), 0.1,
                            a["out"], a["ws"], a["lse"])


def _mass(**kw):
    a = {**_cpu(), "mq": 2, "ms": 32, **kw}
    kv.attention_mass_fp8(*(a[x] for x in ("q", "lse", "kc", "ks", "bt", "sl", "st", "mq", "ms")), 0.1, a["mass"])


def _evict(**kw):
    a = {**_cpu(), "bud": 8, "rec": 2, **kw}
    kv.evict_fp8(*(a[x] for x in ("kc", "vc", "ks", "vs", "mass", "bt", "sl", "bud", "rec", "dbt", "mo", "nl", "kept")))


C = _cpu()
LENS = torch.ones(2, dtype=torch.int32)


@pytest.mark.parametrize("call,kw,what", [
    (_shared, dict(), "CUDA device"), (_shared, dict(lse=None), "CUDA device"), (_shared, dict(q=C["q"].float()), "bfloat16"),
    (_shared, dict(out=C["out"][:2]), "out must have"), (_shared, dict(q=C["q"][0]), "q must be"),
    (_shared, dict(kc=C["kc"].to(torch.int8)), "float8"), (_shared, dict(vs=C["vs"].double()), "scale caches"),
    (_shared, dict(bt=C["bt"].long()), "block_table"), (_shared, dict(sl=C["sl"][:1]), "metadata"),
    (_shared, dict(pl=C["pl"].long()), "prefix_lens"), (_shared, dict(pl=C["pl"][None]), "prefix_lens"),
    (_shared, dict(gs=C["gs"][:1]), "group_start"), (_shared, dict(gs=C["gs"].float()), "group_start"),
    (_shared, dict(ws=C["ws"].int()), "workspace"), (_shared, dict(lse=C["lse"].double()), "lse"),
    (_shared, dict(lse=C["lse"][:, :3]), "lse"), (_shared, dict(lse=C["lse"].T.contiguous().T), "lse"),
    (_shared, dict(mq=1 << 31), "max_query_len must fit"), (_shared, dict(ms=1 << 32), "max_seq_len must fit"),
    (_shared, dict(mg=-(1 << 31) - 1), "max_group_tokens must fit"),
    (_mass, dict(), "CUDA device"), (_mass, dict(q=C["q"].float()), "bfloat16"), (_mass, dict(q=C["q"][0]), "q must be"),
    (_mass, dict(lse=C["lse"][:2]), "lse"), (_mass, dict(lse=C["lse"].half()), "lse"),
    (_mass, dict(kc=C["kc"][0]), "caches must be"), (_mass, dict(ks=C["ks"][:3]), "scale caches"),
    (_mass, dict(st=C["st"][:2]), "metadata"), (_mass, dict(mass=C["mass"].double()), "mass must be"),
    (_mass, dict(mass=C["mass"][:1]), "mass must be"), (_mass, dict(mass=C["mass"][0]), "mass must be"),
    (_mass, dict(mass=C["mass"].transpose(1, 2).contiguous().transpose(1, 2)), "contiguous"),
    (_mass, dict(mq=1 << 31), "max_query_len must fit"), (_mass, dict(ms=1 << 31), "max_seq_len must fit"),
    (_evict, dict(), "CUDA device"), (_evict, dict(vc=C["vc"][:3]), "caches must be"),
    (_evict, dict(kc=C["kc"].transpose(1, 2).contiguous().transpose(1, 2)), "contiguous"),
    (_evict, dict(bt=C["bt"].long()), "block_table"), (_evict, dict(dbt=C["dbt"].long()), "dst_block_table"),
    (_evict, dict(dbt=C["dbt"][:1]), "disagree"), (_evict, dict(sl=C["sl"].long()), "seq_lens"),
    (_evict, dict(nl=C["nl"][:1]), "new_lens"), (_evict, dict(sl=LENS, nl=LENS), "must not be seq_lens"),
    (_evict, dict(kept=C["kept"].long()), "kept"), (_evict, dict(kept=C["kept"][..., :7]), "kept"),
    (_evict, dict(bud=9), "kept"), (_evict, dict(mo=C["mo"][..., :7]), "room"), (_evict, dict(mo=C["mo"].half()), "mass_out"),
    (_evict, dict(mass=C["mass"][:, :1]), "mass must be"), (_evict, dict(bud=1 << 31), "budget must fit"),
    (_evict, dict(rec=1 << 31), "recent must fit"),
])
def test_binding_refusals(call, kw, what):
    with pytest.raises(ValueError, match=what):
        call(**kw)


def test_norm_rope_axes_binding_refusals():
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    pos, cs, w = torch.zeros(2, 3, dtype=torch.int64), torch.zeros(8, 64), torch.ones(64, dtype=torch.bfloat16)
    pairs = kv.rope_axes((16, 16))
    for args, what in [((q, k, pos, cs, pairs, w, w, 0.0, q, k), "CUDA device"), ((q, k, pos, cs, pairs, w, None, 0.0, q, k), "both"),
                       ((q, k, pos[0], cs, pairs, w, w, 0.0, q, k), "int64"), ((q, k, pos.int(), cs, pairs, w, w, 0.0, q, k), "int64"),
                       ((q, k, pos[:, :2], cs, pairs, w, w, 0.0, q, k), "int64"),
                       ((q, k, pos.T.contiguous().T, cs, pairs, w, w, 0.0, q, k), "contiguous along"),
                       ((q, k, pos, cs, pairs[1:], w, w, 0.0, q, k), "32 pairs"), ((q, k, pos, cs, b"", w, w, 0.0, q, k), "32 pairs"),
                       ((q, k, pos, cs.double(), pairs, w, w, 0.0, q, k), "float32"),
                       ((q, k, pos, cs, pairs, w[:32], w, 0.0, q, k), "weights"),
                       ((q, k[:2], pos, cs, pairs, w, w, 0.0, q, k), "disagree"),
                       ((q, k, pos, cs, pairs, w, w, 0.0, k, k), "q_out")]:
        with pytest.raises(ValueError, match=what):
            kv.qk_norm_rope_axes(*args)


@pytest.mark.parametrize("pairs,what", [
    (32, "as bytes"), (1 << 40, "as bytes"), (np.int64(32), "as bytes"), (torch.tensor(32), "as bytes"), (torch.tensor([32]), "32 pairs"),
    (np.array(32), "as bytes"), (None, "as bytes"), ("0" * 32, "as bytes"), ([0] * 31 + [256], "as bytes"), ([-1] * 32, "as bytes"),
    ([0.0] * 32, "as bytes"), ([0] * 31, "32 pairs"), (True, "as bytes"),
    # axes that are taken: the next refusal is the tensors'
    ([0, 1] * 16, "CUDA device"), (bytearray(32), "CUDA device"), (np.zeros(32, np.int64), "CUDA device"),
    (torch.zeros(32, dtype=torch.int32), "CUDA device"), (tuple(kv.rope_axes((16, 16))), "CUDA device"),
])
def test_pair_axes_that_are_no_list_are_refused(pairs, what):
    """An integer would otherwise be as many pairs of axis 0."""
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match=what):
        kv.qk_norm_rope_axes(q, k, torch.zeros(2, 3, dtype=torch.int64), torch.zeros(8, 64), pairs, None, None, 0.0, q, k)


@pytest.mark.parametrize("code,words", [
    (ROT, ["rot_dim", "16", "head_size", "axes 1 to 4", "pair's axis"]),
    (SIZE, ["negative", "overflows", "budget", "recent", "eps", "group", "overlap", "destination", "output is an input"]),
])
def test_status_strings_name_every_reason(lib, code, words):
    text = _lib.status_string(code)
    assert all(w in text for w in words), text


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_small_shared_workspace_holds_its_slots_once(lib, d):
    """Slots of 8192 decode warps and rows of 40960 pieces, each of d values and two numbers; the rest is small.  Without
    groups: slots of 4096."""
    size, row = lib.kv_fp8_attention_shared_workspace_size, (d + 2) * 4
    for groups, warps in ((1, 8192), (0, 4096)):
        least = (warps * 8 + 40960) * row
        assert least <= size(1, groups, 1, 1, 1, d) < least + (1 << 19)
    # direct slots of 32 columns, once: 400 sequences and 8 groups of 8 kv heads
    small = size(1, 1, 1, 1, 1, d)
    assert size(400, 8, 400, 32, 8, d) < small + (408 * 8 * 32 + 2 * 400 * 32) * row + (1 << 19)
