"""kv_fp8_attention_mass against the fp64 oracle, to the bound that the oracle
derives from fp32 scores, exponentials and sums."""

import numpy as np
import pytest
import torch

import int4_token_head_gb300 as kv
from int4_token_head_gb300 import _lib
from oracle import fp8_oracle as F
from test_fp8_gpu import Batch, HEADS, _bf16

pytestmark = pytest.mark.gpu


def _inputs(b, hq, scale=None, q_gain=1.0, seed=3, lse=None):
    q = _bf16((b.tokens, hq, b.d), seed, q_gain)
    scale = b.d ** -0.5 if scale is None else scale
    if lse is None:
        lse = F.log_sum_exp(q.double().numpy(), b.kc, b.ks, b.table, b.lens, b.start, scale)[0]
    g = np.random.default_rng(seed)
    mass = g.uniform(0, 1e-3, (len(b.seqs), b.hkv, b.table.shape[1] * 16)).astype(np.float32)
    return q, torch.from_numpy(lse).float(), mass, scale


def _call(b, q, lse, mass, scale, meta=None, max_q=None, **kw):
    m = torch.from_numpy(mass.copy()).cuda()
    kc, _, ks, _ = b.device()
    kv.attention_mass_fp8(q.cuda(), lse.cuda(), kc, ks, *(meta or b.meta()), b.max_len if max_q is None else max_q,
                          int(b.lens.max()), scale, m, dev_status=b.status, **kw)
    return m


def _check(got, b, q, lse, mass, scale, num_blocks=None, table=None):
    want, bound = F.mass(q.double().numpy(), lse.double().numpy(), b.kc, b.ks, b.table if table is None else table, b.lens,
                         b.start, scale, mass, num_blocks)
    got = got.cpu().numpy()
    for i, length in enumerate(b.lens):
        assert np.array_equal(got[i, :, length:], mass[i, :, length:])  # behind the sequence: left alone
    err = np.abs(got.astype(np.float64) - want)
    assert (err <= bound + 1e-37).all(), ((err / (bound + 1e-37)).max(), np.argwhere(~(err <= bound + 1e-37))[:4])


def _all(seqs, hq, hkv, d, **kw):
    b = Batch(seqs, hkv, d, seed=d + hq).fill(2, kw.pop("k_gain", 1.0))
    x = _inputs(b, hq, **kw)
    _check(_call(b, *x), b, *x)
    assert b.status.item() == 0


DECODE = [(1, 1), (1, 16), (1, 17), (0, 30), (1, 300), (1, 31), (1, 48), (1, 700)]


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (6, 2), (8, 1), (5, 1), (32, 8), (9, 9), (24, 2), (64, 1)])
def test_single_tokens(d, hq, hkv):
    _all(DECODE, hq, hkv, d)


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (7, 1), (12, 3)])
@pytest.mark.parametrize("seqs", [[(2, 2), (5, 40), (3, 3)], [(33, 33), (1, 200), (17, 150), (64, 64)],
                                  [(200, 200), (0, 5), (70, 333)]])
def test_several_tokens_and_prompts(d, hq, hkv, seqs):
    _all(seqs, hq, hkv, d)


@pytest.mark.parametrize("d", HEADS)
def test_a_long_prompt(d):
    """Many tiles of query rows, and a chunk of a prompt behind a history."""
    _all([(530, 530), (300, 900)], 4, 1, d)


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("hq,hkv", [(3, 3), (5, 1), (24, 2), (33, 1), (64, 1)])
def test_many_rows_of_odd_groups(d, hq, hkv):
    """Groups that do not divide a tile of query rows; sequences with few rows beside them."""
    _all([(40, 40), (1, 300), (129, 270), (0, 9), (2, 140)], hq, hkv, d)


def test_many_sequences_with_many_rows():
    """The orders of work: by distance from the end, one after the other, in windows of sequences."""
    g = np.random.default_rng(5)
    _all([(int(n), int(n + g.integers(0, 200))) for n in g.integers(30, 60, 100)], 2, 2, 64)
    _all([(int(n), int(n + g.integers(0, 200))) for n in g.integers(30, 60, 200)], 2, 2, 64)
    _all([(int(n), int(n)) for n in g.integers(30, 40, 1100)], 1, 1, 64)


def test_a_chunk_behind_a_very_long_history():
    _all([(40, 140000), (70, 3000)], 1, 1, 64)


@pytest.mark.parametrize("d", HEADS)
def test_one_query_row_for_every_token(d):
    """Queries that no tensor map holds."""
    b = Batch([(50, 70), (1, 40), (90, 200)], 2, d).fill()
    q, _, mass, scale = _inputs(b, 4)
    q = q[:1].expand(b.tokens, -1, -1)
    lse = torch.from_numpy(F.log_sum_exp(q.double().numpy(), b.kc, b.ks, b.table, b.lens, b.start, scale)[0]).float()
    m = torch.from_numpy(mass.copy()).cuda()
    kc, _, ks, _ = b.device()
    kv.attention_mass_fp8(q[:1].cuda().expand(b.tokens, -1, -1), lse.cuda(), kc, ks, *b.meta(), b.max_len, 200, scale, m,
                          dev_status=b.status)
    _check(m, b, q, lse, mass, scale)


@pytest.mark.parametrize("d", [64, 128])
def test_nan_queries_of_one_sequence_stay_in_its_masses(d):
    b = Batch([(40, 60), (33, 90), (1, 20)], 2, d).fill()
    q, lse, mass, scale = _inputs(b, 4)
    want = _call(b, q, lse, mass, scale)
    q[40:73] = float("nan")
    got = _call(b, q, lse, mass, scale)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2]) and torch.isnan(got[1, :, :90]).all()


def test_sharp_and_flat_scores():
    _all([(1, 400), (40, 100)], 8, 2, 128, q_gain=12.0)
    _all([(1, 400), (40, 100)], 8, 2, 128, q_gain=1e-3)
    _all([(1, 400), (40, 100)], 8, 2, 128, scale=-0.1)
    _all([(1, 400), (40, 100)], 8, 2, 128, scale=0.0)
    _all([(1, 400), (40, 100)], 8, 2, 64, k_gain=2.0 ** 40, scale=2.0 ** -43)


@pytest.mark.parametrize("d", [64, 128])
def test_rows_without_a_denominator_add_nothing(d):
    b = Batch([(3, 50), (20, 20)], 2, d).fill()
    q, lse, mass, scale = _inputs(b, 4)
    lse[1], lse[5, 2], lse[7] = float("-inf"), float("inf"), float("-inf")
    _check(_call(b, q, lse, mass, scale), b, q, lse, mass, scale)


def test_lse_far_from_zero():
    """Every logit at +-300: weights come from differences."""
    for sign in (1.0, -1.0):
        b = Batch([(2, 90)], 1, 64)
        full = np.concatenate([[0], np.cumsum(b.lens)])
        x = np.ones((90, 1, 64)) * 8
        x[:, :, 1] += np.random.default_rng(0).integers(-2, 3, (90, 1))
        F.write(x, b.table, b.lens, full, b.kc, b.ks)
        q = (torch.ones(2, 1, 64) * sign).to(torch.bfloat16)
        lse = F.log_sum_exp(q.double().numpy(), b.kc, b.ks, b.table, b.lens, b.start, 0.6)[0]
        assert abs(lse).min() > 250
        x = q, torch.from_numpy(lse).float(), np.zeros((1, 1, b.table.shape[1] * 16), np.float32), 0.6
        _check(_call(b, *x), b, *x)


def test_weights_of_a_prompt_sum_to_its_rows():
    """Every row's weights sum to one, so a head's masses sum to its rows."""
    b = Batch([(250, 250), (1, 77)], 2, 128).fill()
    q, lse, mass, scale = _inputs(b, 8)
    got = _call(b, q, lse, np.zeros_like(mass), scale).double().cpu().numpy()
    assert np.allclose(got[0].sum(1), 250 * 4, rtol=1e-5) and np.allclose(got[1].sum(1), 4, rtol=1e-5)


@pytest.mark.parametrize("seqs", [[(1, 70), (1, 40), (1, 100)], [(30, 70), (1, 40), (90, 100)]])
def test_bad_blocks_sequences_and_metadata(seqs):
    b = Batch(seqs, 2, 64).fill()
    q, lse, mass, scale = _inputs(b, 4)
    table = b.table.copy()
    table[0, 1], table[2, 0] = -1, b.nb
    lse = torch.from_numpy(F.log_sum_exp(q.double().numpy(), b.kc, b.ks, table, b.lens, b.start, scale)[0]).float()
    meta = [torch.from_numpy(x).cuda() for x in (table, b.lens, b.start)]
    _check(_call(b, q, lse, mass, scale, meta=meta), b, q, lse, mass, scale, table=table)
    assert b.status.item() == _lib.DEV_BAD_BLOCK
    b.status.zero_()
    lens = b.lens.copy()
    lens[1] = 0                                  # shorter than its queries
    meta[1] = torch.from_numpy(lens).cuda()
    got = _call(b, q, lse, mass, scale, meta=meta)
    assert b.status.item() == _lib.DEV_BAD_SEQ | _lib.DEV_BAD_BLOCK
    assert np.array_equal(got[1].cpu().numpy(), mass[1])
    b.status.zero_()
    narrow = mass[:, :, :64].copy()              # less room than two of the sequences have positions
    got = _call(b, q, lse, narrow, scale, meta=b.meta())
    assert b.status.item() == _lib.DEV_BAD_SEQ
    assert np.array_equal(got[0].cpu().numpy(), narrow[0]) and not np.array_equal(got[1].cpu().numpy(), narrow[1])
    if max(n for n, _ in seqs) > 1:
        b.status.zero_()
        got = _call(b, q, lse, mass, scale, max_q=1)
        assert b.status.item() == _lib.DEV_BAD_SEQ and np.array_equal(got[2].cpu().numpy(), mass[2])


def test_strides_shared_blocks_and_nan_codes_behind_the_end():
    """Views with the heads outside, queries inside a wider row; two sequences
    over the same blocks; rows behind a sequence hold NaN codes (Batch leaves them)."""
    b = Batch([(1, 90), (3, 90)], 2, 96).fill()
    b.table[1] = b.table[0]
    q, lse, mass, scale = _inputs(b, 6)
    want = _call(b, q, lse, mass, scale)
    _check(want, b, q, lse, mass, scale)
    wide = torch.full((b.tokens, 6 * 96 + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    vq = wide[:, 8:8 + 6 * 96].view(-1, 6, 96)
    vq.copy_(q)
    big = torch.full((b.tokens, 9), 5.0, device="cuda")
    big[:, 1:7] = lse.cuda()
    room = torch.full((2, 2, mass.shape[2] + 3), 9.0, device="cuda")  # [heads, sequences, positions]
    m = room.transpose(0, 1)[:, :, 1:1 + mass.shape[2]]
    m.copy_(torch.from_numpy(mass))
    kc, _, ks, _ = b.device()
    kv.attention_mass_fp8(vq, big[:, 1:7], kc, ks, *b.meta(), 3, 90, scale, m, dev_status=b.status)
    assert torch.equal(m, want) and b.status.item() == 0
    assert (room[:, :, 0] == 9).all() and (room[:, :, 1 + mass.shape[2]:] == 9).all()
    with pytest.raises(kv.KvInt4Error):
        kv.attention_mass_fp8(vq, big[:, 1:7], kc, ks, *b.meta(), 3, 90, scale, m[:1].expand(2, -1, -1))


def test_long_caches_past_32_bits():
    hkv, d = 32, 256
    nb = (1 << 31) // (16 * hkv * d) + 40
    b = Batch([(1, 50), (20, 40)], hkv, d, spare=0).fill()
    kc = torch.empty(nb, 16, hkv, d, dtype=torch.uint8, device="cuda")
    ks = torch.ones(nb, hkv, device="cuda")
    far = nb - b.nb
    kc[far:], ks[far:] = torch.from_numpy(b.kc).cuda(), torch.from_numpy(b.ks).cuda()
    table, lens, start = b.meta()
    table[table >= 0] += far
    q, lse, mass, scale = _inputs(b, hkv)
    m = torch.from_numpy(mass.copy()).cuda()
    kv.attention_mass_fp8(q.cuda(), lse.cuda(), kc, ks, table, lens, start, 20, 50, scale, m, dev_status=b.status)
    _check(m, b, q, lse, mass, scale)


@pytest.mark.parametrize("seqs", [[(1, 700), (1, 65), (1, 300)], [(200, 500), (1, 65), (90, 300)]])
def test_repeats_streams_graphs_and_ctypes(monkeypatch, seqs):
    b = Batch(seqs, 4, 128).fill()
    q, lse, mass, scale = _inputs(b, 16)
    want = _call(b, q, lse, mass, scale)
    assert torch.equal(_call(b, q, lse, mass, scale), want)
    assert torch.equal(_call(b, q, lse, mass, scale, stream=torch.cuda.current_stream()), want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs += [_call(b, q, lse, mass, scale) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    kc, _, ks, _ = b.device()
    args = [q.cuda(), lse.cuda(), kc, ks, *b.meta(), b.max_len, 700, scale]
    m = torch.from_numpy(mass.copy()).cuda()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.attention_mass_fp8(*args, m, dev_status=b.status)
    graph.replay()
    assert torch.equal(m, want)
    args[5].sub_(3)  # other lengths, the same graph
    graph.replay()
    again = want.clone()
    kv.attention_mass_fp8(*args, again, dev_status=b.status)
    assert torch.equal(m, again)
    monkeypatch.setattr(_lib, "_fp8", _lib._Calls)
    assert torch.equal(_call(b, q, lse, mass, scale), want)


def test_keys_farther_from_the_queries_than_32_bits_of_rows():
    """64 rows to a token and 2^25 positions before the queries: distances times rows leave 32 bits.  The history
    repeats four blocks, so that a position has the mass of its place among their 64."""
    period, history = 64, (1 << 25) + 4096
    b = Batch([(2, 2 * period + 2)], 1, 64).fill()
    b.table[0, 4:8] = b.table[0, :4]
    q, lse, mass, scale = _inputs(b, 64, lse=np.full((2, 64), 3.0))
    mass[:] = 0
    want, bound = F.mass(q.double().numpy(), lse.double().numpy(), b.kc, b.ks, b.table, b.lens, b.start, scale, mass)
    table = torch.from_numpy(np.concatenate([np.tile(b.table[0, :4], history // period), b.table[0, 8:9]])[None]).cuda()
    kc, _, ks, _ = b.device()
    m = torch.zeros(1, 1, history + 16, device="cuda")
    kv.attention_mass_fp8(q.cuda(), lse.cuda(), kc, ks, table, torch.tensor([history + 2], dtype=torch.int32, device="cuda"),
                          b.meta()[2], 2, history + 2, scale, m, dev_status=b.status)
    got = m[0, 0].double().cpu().numpy()
    assert (np.abs(got[:history].reshape(-1, period) - want[0, 0, :period]) <= bound[0, 0, :period]).all()
    assert (np.abs(got[history:history + 2] - want[0, 0, 2 * period:2 * period + 2]) <= bound[0, 0, 2 * period:2 * period + 2]).all()
    assert (got[history + 2:] == 0).all() and b.status.item() == 0
