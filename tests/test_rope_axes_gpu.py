"""kv_qk_norm_rope_axes against the fp64 oracle: positions with several axes."""

import numpy as np
import pytest
import torch

import int4_token_head_gb300 as kv
from int4_token_head_gb300 import _lib
from oracle import fp8_oracle as F

pytestmark = pytest.mark.gpu
HEADS = [64, 96, 128, 192, 256]


def _inputs(t, hq, hkv, d, rot, axes, seed=0):
    g = np.random.default_rng(seed)
    angle = g.uniform(-4, 4, (50, rot // 2))
    table = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1)).float()
    pos = torch.from_numpy(g.integers(0, 50, (axes, t)))
    q, k = (torch.from_numpy(g.standard_normal((t, h, d)) * s).to(torch.bfloat16) for h, s in ((hq, 1.0), (hkv, 3.0)))
    w = [torch.from_numpy(g.uniform(0.5, 1.5, d)).to(torch.bfloat16) for _ in range(2)]
    return q, k, pos, table, w


def _check(got, x, w, eps, table, pos, axes, inter):
    """The bound of the norm and rotation: fp32 sums of d squares, rsqrt, the rotation's two products, bf16's half step."""
    d, half = x.shape[-1], table.shape[1] // 2
    ref = F.norm_rope_axes(x.double().numpy(), None if w is None else w.double().numpy(), eps, table.double().numpy(),
                           pos.numpy(), axes, inter)
    y = np.abs(F.norm_rope(x.double().numpy(), None if w is None else w.double().numpy(), eps, None, None, inter))
    size, c = np.abs(ref), np.abs(table.double().numpy())
    for i, a in enumerate(axes):
        lo, hi = (2 * i, 2 * i + 1) if inter else (i, i + half)
        co, si = c[pos[a].numpy(), i][:, None], c[pos[a].numpy(), half + i][:, None]
        size[..., lo], size[..., hi] = y[..., lo] * co + y[..., hi] * si, y[..., hi] * co + y[..., lo] * si
    tol = 2.0 ** -8 * np.abs(ref) + (d / 2 + 12) * 2.0 ** -24 * size * 1.01 + 1e-38
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= tol).all(), (err / tol).max()


def _run(q, k, pos, table, axes, w, eps=1e-6, inter=False, **kw):
    qo, ko = torch.empty_like(q, device="cuda"), torch.empty_like(k, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = [None if x is None else x.cuda() for x in w]
    kv.qk_norm_rope_axes(q.cuda(), k.cuda(), pos.cuda(), table.cuda(), axes, *w, eps, qo, ko, interleaved=inter,
                         dev_status=status, **kw)
    assert status.item() == 0
    return qo, ko


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("turns", [False, True])
@pytest.mark.parametrize("t,hq,hkv,axes", [(1, 1, 1, 3), (5, 8, 2, 2), (67, 5, 5, 4), (3, 40, 8, 1)])
def test_sections(d, inter, turns, t, hq, hkv, axes):
    g = np.random.default_rng(d + t)
    for rot in sorted({16, d // 2 // 16 * 16, d}):
        cuts = np.sort(g.integers(0, rot // 2 + 1, axes - 1))
        sections = np.diff(np.concatenate([[0], cuts, [rot // 2]]))  # odd ones, empty ones
        pairs = kv.rope_axes(sections, turns)
        q, k, pos, table, w = _inputs(t, hq, hkv, d, rot, axes, seed=d + rot)
        qo, ko = _run(q, k, pos, table, pairs, w, inter=inter)
        _check(qo, q, w[0], 1e-6, table, pos, pairs, inter)
        _check(ko, k, w[1], 1e-6, table, pos, pairs, inter)


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("inter", [False, True])
def test_any_owner_of_every_pair(d, inter):
    """Axes drawn pair by pair; without a norm."""
    pairs = bytes(np.random.default_rng(d).integers(0, 4, d // 2).tolist())
    q, k, pos, table, _ = _inputs(23, 6, 2, d, d, 4)
    qo, ko = _run(q, k, pos, table, pairs, [None, None], 0.0, inter)
    _check(qo, q, None, 0.0, table, pos, pairs, inter)
    _check(ko, k, None, 0.0, table, pos, pairs, inter)


@pytest.mark.parametrize("d", HEADS)
def test_equal_axes_are_one_position(d):
    """The same bits as qk_norm_rope, with a row of positions for all axes too."""
    q, k, pos, table, w = _inputs(33, 8, 2, d, d, 1)
    want = torch.empty_like(q, device="cuda"), torch.empty_like(k, device="cuda")
    kv.qk_norm_rope(q.cuda(), k.cuda(), pos[0].cuda(), table.cuda(), w[0].cuda(), w[1].cuda(), 1e-6, *want)
    pairs = kv.rope_axes((d // 2 - 9, 4, 5), turns=True)
    for p in (pos.expand(3, -1).contiguous().cuda(), pos.cuda().expand(3, -1)):
        got = _run(q, k, p, table, pairs, w)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_in_place_strided_and_without_rotation():
    d, t, hq, hkv = 96, 19, 6, 2
    q, k, pos, table, w = _inputs(t, hq, hkv, d, 32, 3)
    pairs = kv.rope_axes((5, 6, 5))
    want = _run(q, k, pos, table, pairs, w)
    fused = torch.full((t, (hq + hkv) * d + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    fq, fk = fused[:, 8:8 + hq * d].view(t, hq, d), fused[:, 8 + hq * d:8 + (hq + hkv) * d].view(t, hkv, d)
    fq.copy_(q)
    fk.copy_(k)
    wide = torch.full((3, t + 5), -1)
    wide[:, 2:2 + t] = pos
    kv.qk_norm_rope_axes(fq, fk, wide.cuda()[:, 2:2 + t], table.cuda(), pairs, w[0].cuda(), w[1].cuda(), 1e-6, fq, fk)
    assert torch.equal(fq, want[0]) and torch.equal(fk, want[1])
    assert (fused[:, :8] == 7).all() and (fused[:, 8 + (hq + hkv) * d:] == 7).all()
    none = torch.empty(50, 0)
    kv.qk_norm_rope_axes(q.cuda(), k.cuda(), pos.cuda(), none.cuda(), b"", w[0].cuda(), w[1].cuda(), 1e-6, fq, fk)
    norm = torch.empty_like(want[0]), torch.empty_like(want[1])
    kv.qk_norm_rope(q.cuda(), k.cuda(), None, None, w[0].cuda(), w[1].cuda(), 1e-6, *norm)
    assert torch.equal(fq, norm[0]) and torch.equal(fk, norm[1])


@pytest.mark.parametrize("axis", [0, 1, 2])
def test_a_bad_position_along_any_axis_leaves_its_rows(axis):
    q, k, pos, table, w = _inputs(8, 20, 4, 128, 128, 3)
    pairs = kv.rope_axes((24, 20, 20), turns=True)
    want = _run(q, k, pos, table, pairs, w)
    pos[axis, 2], pos[axis, 5] = 50, -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo, ko = (torch.full_like(x, 7.0, device="cuda") for x in (q, k))
    kv.qk_norm_rope_axes(q.cuda(), k.cuda(), pos.cuda(), table.cuda(), pairs, w[0].cuda(), w[1].cuda(), 1e-6, qo, ko,
                         dev_status=status)
    assert status.item() == _lib.DEV_BAD_POS
    for got, ref in ((qo, want[0]), (ko, want[1])):
        for t in range(8):
            assert (got[t] == 7).all() if t in (2, 5) else torch.equal(got[t], ref[t])


@pytest.mark.parametrize("d", HEADS)
def test_many_tokens_have_the_bits_of_few(d):
    """Above 32 tokens per SM a warp takes all heads of a token; in place, with bad positions among them."""
    t, hq, hkv = 32 * torch.cuda.get_device_properties(0).multi_processor_count + 7, 7, 6
    q, k, pos, table, w = _inputs(t, hq, hkv, d, d // 2, 3)
    pairs = kv.rope_axes((d // 8, d // 16, d // 16), turns=True)
    pos[1, 11::97] = 50
    args = [x.cuda() for x in (q, k, pos, table)]
    dw = [x.cuda() for x in w]
    want = [x.clone() for x in args[:2]]
    for i in range(0, t, 700):
        rows = slice(i, min(t, i + 700))
        kv.qk_norm_rope_axes(args[0][rows], args[1][rows], args[2][:, rows], args[3], pairs, *dw, 1e-6,
                             want[0][rows], want[1][rows])
    kv.qk_norm_rope_axes(*args, pairs, *dw, 1e-6, args[0], args[1])
    assert torch.equal(args[0], want[0]) and torch.equal(args[1], want[1])
    assert torch.equal(args[0][11::97].cpu(), q[11::97])
    some = slice(4000, 4040)
    _check(args[0][some].cpu()[:10], q[some][:10], w[0], 1e-6, table, pos[:, some][:, :10], pairs, False)


def test_streams_graph_and_ctypes_give_the_same_bits(monkeypatch):
    q, k, pos, table, w = _inputs(40, 8, 2, 128, 64, 3)
    pairs = kv.rope_axes((12, 10, 10))
    want = _run(q, k, pos, table, pairs, w)
    other = torch.cuda.Stream()
    assert all(torch.equal(a, b) for a, b in zip(_run(q, k, pos, table, pairs, w, stream=torch.cuda.current_stream()), want))
    with torch.cuda.stream(other):
        got = _run(q, k, pos, table, pairs, w)
    other.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    args = [x.cuda() for x in (q, k, pos, table)]
    dw, outs = [x.cuda() for x in w], [torch.empty_like(args[0]), torch.empty_like(args[1])]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # pair_axis is read during the call, its bytes may go
        kv.qk_norm_rope_axes(*args, bytes(bytearray(pairs)), *dw, 1e-6, *outs)
    args[2].copy_(pos.flip(1))
    graph.replay()
    flipped = _run(q, k, pos.flip(1), table, pairs, w)
    assert all(torch.equal(a, b) for a, b in zip(outs, flipped))
    monkeypatch.setattr(_lib, "_fp8", _lib._Calls)
    assert all(torch.equal(a, b) for a, b in zip(_run(q, k, pos, table, list(pairs), w), want))
