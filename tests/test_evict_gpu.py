"""kv_fp8_evict against the oracle: positions, masses, codes and scales bit for bit."""

import numpy as np
import pytest
import torch

import int4_token_head_gb300 as kv
from int4_token_head_gb300 import _lib
from oracle import fp8_oracle as F
from test_fp8_gpu import Batch, HEADS, _assert_caches

pytestmark = pytest.mark.gpu


def _masses(b, seed=0, ties=False):
    g = np.random.default_rng(seed)
    m = np.exp(3 * g.standard_normal((len(b.seqs), b.hkv, b.table.shape[1] * 16))).astype(np.float32)
    return np.round(m).astype(np.float32) if ties else m


def _batch(lens, hkv, d, seed=0, spare=3, extra_width=1):
    """Written rows whose magnitudes differ by powers of two from row to row."""
    b = Batch([(0, length) for length in lens], hkv, d, seed=seed, spare=spare, extra_width=extra_width)
    g = np.random.default_rng(seed + 1)
    full = np.concatenate([[0], np.cumsum(b.lens)])
    for codes, scale in ((b.kc, b.ks), (b.vc, b.vs)):
        x = g.standard_normal((int(full[-1]), hkv, d)) * np.exp2(g.integers(-9, 10, (int(full[-1]), hkv, 1)))
        F.write(torch.from_numpy(x).to(torch.bfloat16).double().numpy(), b.table, b.lens, full, codes, scale)
    return b


def _other_blocks(b, budget):
    """A table of blocks that no sequence reads, behind the others."""
    need = [-(-min(budget, int(n)) // 16) for n in b.lens]
    into = np.full((len(b.lens), max(-(-min(budget, b.table.shape[1] * 16) // 16), 1)), -1, np.int32)
    at = b.nb
    for i, n in enumerate(need):
        into[i, :n] = np.arange(at, at + n)[::-1]
        at += n
    more = at - b.nb
    b.kc, b.vc = (np.concatenate([x, np.full((more, *x.shape[1:]), 0xFF, np.uint8)]) for x in (b.kc, b.vc))
    b.ks, b.vs = (np.concatenate([x, np.full((more, b.hkv), np.nan, np.float32)]) for x in (b.ks, b.vs))
    b.nb = at
    return into


def _run(b, mass, budget, recent, into=None, own_mass=True, table=None, lens=None, **kw):
    """The call on copies; (caches, mass_out, new_lens, kept) on the device."""
    dev = b.device()
    t, l, _ = b.meta()
    t = t if table is None else torch.from_numpy(table).cuda()
    l = l if lens is None else torch.from_numpy(lens).cuda()
    m = torch.from_numpy(mass.copy()).cuda()
    out = m if own_mass else torch.full_like(m, -7.0)
    new = torch.full_like(l, -7)
    kept = torch.full((len(b.lens), b.hkv, budget), -7, dtype=torch.int32, device="cuda")
    kv.evict_fp8(*dev, m, t, l, budget, recent, t if into is None else torch.from_numpy(into).cuda(), out, new, kept,
                 dev_status=b.status, **kw)
    return dev, out, new, kept


def _check(b, mass, budget, recent, into=None, own_mass=True):
    got = _run(b, mass, budget, recent, into, own_mass)
    out = mass.copy() if own_mass else np.full_like(mass, -7.0)
    kept = np.full((len(b.lens), b.hkv, budget), -7, np.int32)
    caches = [x.copy() for x in b.host()]
    new = F.evict(caches, mass, b.table, b.lens, budget, recent, b.table if into is None else into, out, kept)
    assert b.status.item() == 0
    assert np.array_equal(got[2].cpu().numpy(), new)
    assert np.array_equal(got[3].cpu().numpy(), kept)
    assert np.array_equal(got[1].cpu().numpy().view(np.int32), out.view(np.int32))
    _assert_caches(got[0], caches)


LENS = [0, 1, 16, 17, 33, 100, 40, 260, 41]


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("hkv", [1, 3])
@pytest.mark.parametrize("budget,recent", [(40, 8), (40, 0), (40, 40), (1, 0), (1, 1), (17, 16), (400, 5)])
@pytest.mark.parametrize("in_place", [True, False])
def test_short_sequences(d, hkv, budget, recent, in_place):
    b = _batch(LENS, hkv, d, seed=budget + recent)
    into = None if in_place else _other_blocks(b, budget)
    _check(b, _masses(b, budget), budget, recent, into, own_mass=in_place)


@pytest.mark.parametrize("d", [64, 128, 192])
@pytest.mark.parametrize("lens,budget,recent", [([3000], 1500, 100), ([2500, 3100, 900], 1000, 0), ([5000], 129, 64)])
@pytest.mark.parametrize("in_place", [True, False])
def test_long_sequences(d, lens, budget, recent, in_place):
    """Several chunks, one CTA or a cluster of them per task."""
    b = _batch(lens, 2, d)
    into = None if in_place else _other_blocks(b, budget)
    _check(b, _masses(b), budget, recent, into, own_mass=not in_place)


def test_masses_beyond_the_shared_memory():
    lens = [50000, 43000, 100]
    b = _batch(lens, 1, 64)
    m = _masses(b, ties=True)
    _check(b, m, 3000, 17)
    _check(b, m, 45000, 0)


@pytest.mark.parametrize("kind", ["equal", "zeros", "ties", "rising", "falling", "special"])
def test_orders_and_ties(kind):
    b = _batch([300, 1100], 2, 64)
    m = _masses(b, ties=True)
    p = np.arange(m.shape[2], dtype=np.float32)
    if kind == "equal":
        m[:] = 0.25
    elif kind == "zeros":
        m[:] = np.where(p % 3 == 0, np.float32(-0.0), np.float32(0.0))
    elif kind == "rising":
        m[:] = p
    elif kind == "falling":
        m[:] = -p  # negative values order too
    elif kind == "special":
        m[:, :, 3::7], m[:, :, 5::11], m[:, :, 2::13], m[:, :, 1::9] = np.nan, np.inf, -np.inf, np.float32(1e-42)
        m[:, :, 8::17] = -np.float32(np.nan)
    for budget, recent in ((200, 30), (64, 0), (299, 298)):
        _check(b, m, budget, recent)


def test_every_block_scale_and_subnormal_codes():
    """Rows of all scales in one block: codes shift into subnormals and away."""
    b = _batch([600], 1, 64)
    g = np.random.default_rng(4)
    b.ks[:] = np.exp2(g.integers(-60, 61, b.ks.shape)).astype(np.float32)
    b.vs[:] = np.exp2(g.integers(-8, 9, b.vs.shape)).astype(np.float32)
    b.kc[:], b.vc[:] = (np.where((c := g.integers(0, 256, b.kc.shape)) & 0x7F == 0x7F, 0x40, c).astype(np.uint8)
                        for _ in range(2))
    b.vc[:, :, :, :] = np.where(g.random(b.vc.shape) < 0.9, b.vc & 0x87, b.vc)  # many subnormal codes
    b.vc[b.table[0, 3]] = 0
    _check(b, _masses(b), 300, 20)


def test_a_token_over_the_budget_step_by_step():
    """In place, one position more than the budget: what lies before the first that goes is untouched."""
    b = _batch([129, 129, 128], 2, 128)
    m = _masses(b)
    m[0, :, :100] += 1e6
    _check(b, m, 128, 16)


def test_bad_blocks_scales_and_sequences():
    b = _batch([100, 90, 120, 60], 2, 64)
    m = _masses(b)
    table = b.table.copy()
    table[0, 2] = b.nb
    b.ks[b.table[1, 1], 0] = np.float32(0.75)    # no scale that a write stores
    lens = b.lens.copy()
    lens[2] = b.table.shape[1] * 16 + 1
    lens[3] = -5
    got = _run(b, m, 48, 10, table=table, lens=lens)
    assert b.status.item() == _lib.DEV_BAD_BLOCK | _lib.DEV_BAD_SEQ
    out, kept = m.copy(), np.full((4, 2, 48), -7, np.int32)
    caches = [x.copy() for x in b.host()]
    new = F.evict(caches, m[:2], table[:2], lens[:2], 48, 10, table[:2], out, kept)
    assert np.array_equal(got[2].cpu().numpy(), np.concatenate([new, lens[2:]]))
    assert np.array_equal(got[3].cpu().numpy(), kept) and np.array_equal(got[1].cpu().numpy(), out)
    _assert_caches(got[0], caches)


def test_a_destination_that_is_no_block():
    b = _batch([100], 2, 64)
    into = _other_blocks(b, 48)
    into[0, 1] = b.nb + 7
    m = _masses(b)
    got = _run(b, m, 48, 10, into)
    assert b.status.item() == _lib.DEV_BAD_BLOCK
    caches = [x.copy() for x in b.host()]
    F.evict(caches, m, b.table, b.lens, 48, 10, into, m.copy(), np.zeros((1, 2, 48), np.int32))
    _assert_caches(got[0], caches)


def test_a_copy_of_the_table_and_views_of_the_masses():
    b = _batch([300, 77, 500], 2, 96)
    m = _masses(b)
    _check(b, m, 100, 20, into=b.table.copy())
    wide = torch.full((2, 3, m.shape[2] + 5), -3.0, device="cuda")  # heads outside
    view = wide.transpose(0, 1)[:, :, 3:3 + m.shape[2]]
    view.copy_(torch.from_numpy(m))
    want = _run(b, m, 100, 20)
    dev, meta = b.device(), b.meta()
    new, kept = torch.empty_like(meta[1]), torch.full_like(want[3], -7)
    kv.evict_fp8(*dev, view, meta[0], meta[1], 100, 20, meta[0], view, new, kept, dev_status=b.status)
    assert torch.equal(view, want[1]) and torch.equal(kept, want[3]) and torch.equal(new, want[2])
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(dev, want[0]))
    assert (wide[:, :, :3] == -3).all() and (wide[:, :, 3 + m.shape[2]:] == -3).all()


def test_offsets_past_32_bits():
    hkv, d = 32, 256
    nb = (1 << 31) // (16 * hkv * d) + 60
    b = _batch([300, 77], hkv, d, spare=0)
    big = [torch.zeros(nb, 16, hkv, d, dtype=torch.uint8, device="cuda") for _ in range(2)] + [
        torch.ones(nb, hkv, device="cuda") for _ in range(2)]
    far = nb - b.nb
    for x, y in zip(big, b.host()):
        x[far:] = torch.from_numpy(y).cuda()
    m = _masses(b)
    want = _run(b, m, 64, 8)
    table, lens, _ = b.meta()
    table[table >= 0] += far
    mm, new, kept = torch.from_numpy(m).cuda(), torch.empty_like(lens), torch.empty_like(want[3])
    kv.evict_fp8(*big, mm, table, lens, 64, 8, table, mm, new, kept, dev_status=b.status)
    assert torch.equal(kept, want[3])
    for x, y in zip(big, want[0]):
        assert torch.equal(x[far:].view(torch.uint8), y.view(torch.uint8))


def test_repeats_streams_graphs_and_ctypes(monkeypatch):
    b = _batch([900, 300, 1500], 4, 128)
    m = _masses(b)

    def same(x, y):
        return all(torch.equal(a.view(torch.uint8), c.view(torch.uint8)) for a, c in zip((*x[0], *x[1:]), (*y[0], *y[1:])))

    want = _run(b, m, 256, 32)
    assert same(_run(b, m, 256, 32), want)
    assert same(_run(b, m, 256, 32, stream=torch.cuda.current_stream()), want)
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):
        got = _run(b, m, 256, 32)
    other.synchronize()
    assert same(got, want)
    dev, (table, lens, _) = b.device(), b.meta()
    mm, new = torch.from_numpy(m.copy()).cuda(), torch.full_like(lens, -7)
    kept = torch.full_like(want[3], -7)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.evict_fp8(*dev, mm, table, lens, 256, 32, table, mm, new, kept, dev_status=b.status)
    graph.replay()
    assert same((dev, mm, new, kept), want)
    monkeypatch.setattr(_lib, "_fp8", _lib._Calls)
    assert same(_run(b, m, 256, 32), want)
    assert b.status.item() == 0
