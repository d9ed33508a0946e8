"""kv_fp8_attention_shared against the fp64 oracle: outputs to the bound of
kv_fp8_attention, log-sum-exps to the bound that the oracle derives."""

import numpy as np
import pytest
import torch

import int4_token_head_gb300 as kv
from int4_token_head_gb300 import _lib
from oracle import fp8_oracle as F
from test_fp8_gpu import Batch, HEADS, _assert_attention, _bf16

pytestmark = pytest.mark.gpu
WIDE = 700  # table entries behind the sequences: too long a table for the one-launch path, which shares nothing


class Shared:
    """groups: [(prefix, [(query tokens, positions behind the prefix)])]; prefix 0 for sequences in no group of
    several.  The members' first prefix // 16 blocks are the first member's."""

    def __init__(self, groups, hkv, d, seed=0, wide=WIDE, k_gain=1.0, v_gain=1.0):
        seqs = [(q, prefix + own) for prefix, members in groups for q, own in members]
        self.b = b = Batch(seqs, hkv, d, seed=seed, extra_width=wide).fill(seed + 1, k_gain, v_gain)
        self.group_start = np.concatenate([[0], np.cumsum([len(m) for _, m in groups])]).astype(np.int32)
        self.prefix = np.array([p for p, _ in groups], np.int32)
        for g, p in enumerate(self.prefix):
            at = self.group_start[g]
            for i in range(at, self.group_start[g + 1]):
                b.table[i, :p // 16] = b.table[at, :p // 16]
        tokens = [int(b.start[self.group_start[g + 1]] - b.start[self.group_start[g]]) for g in range(len(groups))]
        self.max_group = max(tokens)

    def call(self, q, hq, scale=None, lse=True, out=None, group_start=None, prefix=None, max_group=None, dev=None,
             meta=None, max_q=None, ws=None, **kw):
        b = self.b
        gs = torch.from_numpy(self.group_start if group_start is None else np.asarray(group_start, np.int32)).cuda()
        pl = torch.from_numpy(self.prefix if prefix is None else np.asarray(prefix, np.int32)).cuda()
        if ws is None:
            ws = torch.empty(kv.attention_shared_workspace_size(len(b.seqs), len(pl), q.shape[0], hq, b.hkv, b.d),
                             dtype=torch.uint8, device="cuda").fill_(0xFF)
        if out is None:
            out = torch.full((q.shape[0], hq, b.d), float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full((q.shape[0], hq), float("nan"), device="cuda") if lse is True else lse
        kv.attention_fp8_shared(q.cuda(), *(dev or b.device()), *(meta or b.meta()), b.max_len if max_q is None else max_q,
                                1 << 30, gs, pl, self.max_group if max_group is None else max_group,
                                b.d ** -0.5 if scale is None else scale, out, ws, lse=lse, dev_status=b.status, **kw)
        return out, lse

    def check(self, got, q, scale=None, rows=slice(None), table=None):
        b = self.b
        scale = b.d ** -0.5 if scale is None else scale
        table = b.table if table is None else table
        ref, bound = F.attention(q.double().numpy(), b.host(), table, b.lens, b.start, scale, True)
        _assert_attention(got[0][rows], ref[rows], bound[rows])
        lse, err = F.log_sum_exp(q.double().numpy(), b.kc, b.ks, table, b.lens, b.start, scale)
        have = got[1].double().cpu().numpy()[rows]
        lse, err = lse[rows], err[rows]
        fine = np.isfinite(lse)
        assert np.array_equal(have[~fine], lse[~fine])
        assert (np.abs(have - lse)[fine] <= err[fine]).all(), (np.abs(have - lse)[fine] / err[fine]).max()


def _check(groups, hq, hkv, d, q_gain=1.0, scale=None, **kw):
    s = Shared(groups, hkv, d, seed=d + hq, **kw)
    q = _bf16((s.b.tokens, hq, d), 5, q_gain)
    got = s.call(q, hq, scale)
    s.check(got, q, scale)
    assert s.b.status.item() == 0
    return s, q, got


DECODE = [(320, [(1, 1), (1, 40), (1, 17)]), (48, [(1, 3), (1, 500)]), (0, [(1, 77), (1, 200)]), (1000, [(1, 9)] * 2)]


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (8, 1), (5, 1), (12, 4), (9, 9), (32, 1), (64, 1)])
def test_single_tokens(d, hq, hkv):
    """Prefixes on the decode kernel (up to 32 rows of a group) and, with more q heads per kv head, in tiles."""
    _check(DECODE, hq, hkv, d)


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("hq,hkv", [(2, 2), (16, 4), (7, 1)])
def test_many_sequences_over_one_prefix(d, hq, hkv):
    """A group's rows in prefill tiles, the ends on the decode kernel beside them."""
    g = np.random.default_rng(d)
    _check([(720, [(1, int(n)) for n in g.integers(1, 90, 34)])], hq, hkv, d)


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (6, 1)])
def test_several_tokens_and_prompts(d, hq, hkv):
    """Queries of one to many tokens: ends in prefill tiles too, a long prompt in no group, one in a group that
    therefore shares nothing, a group of one."""
    _check([(640, [(5, 9), (1, 1), (20, 33), (0, 12), (30, 30)]), (0, [(300, 300)]), (160, [(2, 2), (280, 280)]),
            (96, [(3, 50)]), (1600, [(17, 17), (4, 60), (1, 2)])], hq, hkv, d)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prefix_of_any_length(d):
    """Lengths that end inside a block, in the first block, or reach into the queries: whole blocks before all of
    them are shared, results are the same."""
    for prefix in (15, 16, 17, 333, 350):
        s = Shared([(prefix, [(3, 20), (1, 1), (2, 5)])], 2, d, seed=prefix)
        q = _bf16((s.b.tokens, 8, d), 5)
        s.check(s.call(q, 8), q)
        p = prefix // 16 * 16
        s.check(s.call(q, 8, prefix=[p // 2]), q)
        s.check(s.call(q, 8, prefix=[-5]), q)
    # one sequence's queries begin inside the prefix: all members' blocks must be shared for that
    s = Shared([(320, [(30, 10), (1, 40)])], 2, d)
    q = _bf16((s.b.tokens, 8, d), 6)
    s.check(s.call(q, 8), q)
    assert s.b.status.item() == 0


@pytest.mark.parametrize("d", HEADS)
def test_short_batches_and_no_groups(d):
    """The one-launch path, and batches without groups on every path, with their log-sum-exp."""
    s, q, got = _check([(64, [(4, 33), (4, 64)])], 4, 4, d, wide=1)
    s.check(s.call(q, 4, group_start=[0], prefix=[]), q)
    for hq, seqs in ((4, [(1, 100), (1, 7000)]), (8, [(40, 300), (1, 900), (7, 7)])):
        s = Shared([(0, seqs)], 2, d)
        q = _bf16((s.b.tokens, hq, d), 5)
        s.check(s.call(q, hq, group_start=[0], prefix=[]), q)


def test_many_groups():
    g = np.random.default_rng(2)
    groups = [(int(g.integers(0, 8)) * 16, [(int(q), int(q + g.integers(0, 30))) for q in g.integers(0, 3, g.integers(1, 4))])
              for _ in range(600)]
    _check(groups, 4, 2, 64, wide=WIDE)


def test_more_rows_than_the_workspace_shares():
    """64 q heads: 2048 query tokens; the groups behind them are worked on whole."""
    _check([(64, [(1, 2)] * 1000), (64, [(3, 4)] * 300), (64, [(1, 1)] * 700), (32, [(1, 2), (1, 3)])], 64, 1, 64)


def test_sharp_scores_extreme_scales_and_signs():
    group = [(480, [(1, 30), (1, 1), (2, 9)] * 6), (32, [(1, 20), (1, 30)])]
    _check(group, 8, 2, 128, q_gain=12.0)
    _check(group, 8, 2, 128, q_gain=0.0)
    _check(group, 8, 2, 128, scale=-0.2)
    _check(group, 8, 2, 64, k_gain=2.0 ** 40, scale=2.0 ** -43)
    _check(group, 8, 2, 64, v_gain=2.0 ** -50)


@pytest.mark.parametrize("members", [[(1, 20), (1, 33)], [(1, 20), (1, 3)] * 20, [(20, 20), (33, 40)]])
def test_bad_blocks_and_sequences(members):
    s = Shared([(480, members)], 2, 64)
    b = s.b
    q = _bf16((b.tokens, 8, 64), 5)
    b.table[:, 3] = -1                        # in the prefix: hidden from all
    b.table[1, 31] = b.nb                     # the second sequence's own, if it has that many
    got = s.call(q, 8)
    s.check(got, q)
    assert b.status.item() == _lib.DEV_BAD_BLOCK
    b.table[:, :30] = -1                      # nothing of the prefix is usable
    s.check(s.call(q, 8), q)
    b.table[:] = -1                           # nothing at all: zeros
    out, lse = s.call(q, 8)
    assert (out == 0).all() and (lse == float("-inf")).all()


def test_bad_metadata_shares_nothing_or_skips():
    s = Shared([(320, [(1, 20), (1, 33), (2, 8)]), (160, [(1, 9), (1, 50)])], 2, 64)
    b = s.b
    q = _bf16((b.tokens, 8, 64), 5)
    for gs in ([0, 4, 3], [0, 3, 6], [-1, 3, 5]):
        b.status.zero_()
        s.check(s.call(q, 8, group_start=gs), q)
        assert b.status.item() == _lib.DEV_BAD_SEQ
    b.status.zero_()
    for gs in ([0, 3, 3], [1, 3, 4], [3, 3, 5], [0, 0, 0]):   # groups that leave sequences out
        s.check(s.call(q, 8, group_start=gs, prefix=[320, 160] if gs[1] != 4 else [320, 0]), q)
    s.check(s.call(q, 8, max_group=1), q)                     # no group is that small
    s.check(s.call(q, 8, max_group=1 << 20), q)
    assert b.status.item() == 0
    lens = b.lens.copy()
    lens[1] = 0                                               # a member without its own query
    meta = [torch.from_numpy(x).cuda() for x in (b.table, lens, b.start)]
    got = s.call(q, 8, meta=meta)
    assert b.status.item() == _lib.DEV_BAD_SEQ
    rows = np.array([0, 2, 3, 4, 5])
    s.check(got, q, rows=rows)
    assert torch.isnan(got[0][1]).all() and torch.isnan(got[1][1]).all()


def test_strides_padding_and_no_lse():
    s = Shared([(640, [(1, 20), (3, 33)] * 7), (0, [(50, 80)])], 2, 96)
    b, hq = s.b, 6
    q = _bf16((b.tokens, hq, 96), 5)
    want = s.call(q, hq)
    s.check(want, q)
    t, pad = b.tokens, 3
    wide = [torch.full((t + pad, hq * 96 + 24), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    vq, vo = (x[:, 8:8 + hq * 96].view(-1, hq, 96) for x in wide)
    vq[:t].copy_(q)
    big = torch.full((t + pad, hq + 3), 5.0, device="cuda")
    out, lse = s.call(vq, hq, out=vo, lse=big[:, 1:1 + hq])
    assert torch.equal(vo[:t], want[0]) and torch.equal(lse[:t], want[1])
    assert (wide[1][:, :8] == 3).all() and (wide[1][:, 8 + hq * 96:] == 3).all() and (wide[1][t:] == 3).all()
    assert (big[:, 0] == 5).all() and (big[:, 1 + hq:] == 5).all() and (big[t:] == 5).all()
    assert torch.equal(s.call(q, hq, lse=None)[0], want[0])
    ws = torch.empty(kv.attention_shared_workspace_size(len(b.seqs), 2, t, hq, 2, 96) + 4096, dtype=torch.uint8,
                     device="cuda").fill_(0xA5)
    assert torch.equal(s.call(q, hq, ws=ws[:-4096])[0], want[0]) and (ws[-4096:] == 0xA5).all()
    with pytest.raises(kv.KvInt4Error, match="workspace"):
        s.call(q, hq, ws=ws[:-4352])


@pytest.mark.parametrize("members", [[(1, 30)] * 50, [(1, 30), (9, 9)] * 12, [(1, 5)] * 3])
def test_repeats_streams_graphs_and_ctypes(monkeypatch, members):
    s = Shared([(3000, members), (0, [(1, 700)])], 4, 128)
    b, hq = s.b, 16
    q = _bf16((b.tokens, hq, 128), 5)

    def same(x, y):
        return torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])

    want = s.call(q, hq)
    s.check(want, q)
    for _ in range(3):
        assert same(s.call(q, hq), want)
    assert same(s.call(q, hq, stream=torch.cuda.current_stream()), want)
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for st in streams:
        with torch.cuda.stream(st):
            outs += [s.call(q, hq) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(same(o, want) for o in outs)
    dev, meta = b.device(), b.meta()
    gs, pl = torch.from_numpy(s.group_start).cuda(), torch.from_numpy(s.prefix).cuda()
    ws = torch.empty(kv.attention_shared_workspace_size(len(b.seqs), 2, b.tokens, hq, 4, 128), dtype=torch.uint8, device="cuda")
    out, lse, dq = torch.empty_like(want[0]), torch.empty_like(want[1]), q.cuda()

    def step():
        kv.attention_fp8_shared(dq, *dev, *meta, b.max_len, 1 << 30, gs, pl, s.max_group, 128 ** -0.5, out, ws, lse=lse,
                                dev_status=b.status)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    graph.replay()
    assert same((out, lse), want)
    for new_prefix, cut in (([1600, 0], 0), ([0, 0], 3), ([3000, 0], 3)):  # other sharing, other lengths
        pl.copy_(torch.tensor(new_prefix, dtype=torch.int32))
        meta[1].copy_(torch.from_numpy(b.lens - np.where(b.lens - 1 > 3010 + cut, cut, 0).astype(np.int32)))
        graph.replay()
        got = out.clone(), lse.clone()
        step()
        assert same(got, (out, lse))
    monkeypatch.setattr(_lib, "_fp8", _lib._Calls)
    assert same(s.call(q, hq), want)
    assert b.status.item() == 0


def test_offsets_past_32_bits():
    hkv, d = 32, 256
    nb = (1 << 31) // (16 * hkv * d) + 140
    s = Shared([(320, [(1, 20), (2, 33)] * 3)], hkv, d, wide=WIDE)
    b = s.b
    big = [torch.zeros(nb, 16, hkv, d, dtype=torch.uint8, device="cuda") for _ in range(2)] + [
        torch.ones(nb, hkv, device="cuda") for _ in range(2)]
    far = nb - b.nb
    for x, y in zip(big, b.host()):
        x[far:] = torch.from_numpy(y).cuda()
    table, lens, start = b.meta()
    table[table >= 0] += far
    q = _bf16((b.tokens, hkv, d), 2)
    s.check(s.call(q, hkv, dev=big, meta=(table, lens, start)), q)


@pytest.mark.parametrize("d", [64, 128])
def test_prefixes_written_just_before_and_masses_after(d):
    """The operators together: a shared prompt written, answered, its masses taken and its sequences shortened."""
    hq, hkv, prefix = 8, 2, 640
    s = Shared([(prefix, [(3, 40), (1, 9), (2, 25)] * 2)], hkv, d, wide=40)
    b = s.b
    dev, meta = b.device(), b.meta()
    q = _bf16((b.tokens, hq, d), 5)
    k, v = _bf16((b.tokens, hkv, d), 6), _bf16((b.tokens, hkv, d), 7)
    cos_sin = torch.rand(64, d)
    pos = torch.randint(0, 64, (3, b.tokens))
    axes = kv.rope_axes((d // 2 - 20, 12, 8), turns=True)
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    kv.qk_norm_rope_axes(qd, kd, pos.cuda(), cos_sin.cuda(), axes, None, None, 0.0, qd, kd, dev_status=b.status)
    q, k = qd.cpu(), kd.cpu()
    kv.write_fp8(kd, vd, *meta, 3, *dev, dev_status=b.status)
    for x, codes, scale in ((k, b.kc, b.ks), (v, b.vc, b.vs)):
        F.write(x.double().numpy(), b.table, b.lens, b.start, codes, scale)
    got = s.call(qd, hq, dev=dev, meta=meta)
    s.check(got, q)
    room = 700
    mass = torch.full((len(b.seqs), hkv, room), 0.5, device="cuda")
    kv.attention_mass_fp8(qd, got[1], dev[0], dev[2], *meta, 3, room, d ** -0.5, mass, dev_status=b.status)
    m, bound = F.mass(q.double().numpy(), got[1].double().cpu().numpy(), b.kc, b.ks, b.table, b.lens, b.start, d ** -0.5,
                      np.full(tuple(mass.shape), 0.5))
    assert (np.abs(mass.double().cpu().numpy() - m) <= bound + 1e-37).all()
    # every sequence keeps 100 positions in blocks of its own
    budget, n = 100, len(b.seqs)
    into = torch.arange(n * 7, dtype=torch.int32).view(n, 7).cuda() + b.nb
    more = [torch.cat([x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x,
                       torch.zeros(n * 7, *x.shape[1:], dtype=torch.uint8 if x.dim() == 4 else torch.float32, device="cuda")])
            for x in dev]
    new, kept = torch.empty_like(meta[1]), torch.empty(n, hkv, budget, dtype=torch.int32, device="cuda")
    host_mass, host_kept = mass.cpu().numpy().copy(), np.zeros((n, hkv, budget), np.int32)
    caches = [x.cpu().numpy() for x in more]
    before = host_mass.copy()
    kv.evict_fp8(*more, mass, meta[0], meta[1], budget, 16, into, mass, new, kept, dev_status=b.status)
    lens = F.evict(caches, before, b.table, b.lens, budget, 16, into.cpu().numpy(), host_mass, host_kept)
    assert np.array_equal(kept.cpu().numpy(), host_kept) and np.array_equal(new.cpu().numpy(), lens)
    assert np.array_equal(mass.cpu().numpy(), host_mass)
    for x, y in zip(more, caches):
        assert np.array_equal(x.cpu().numpy().view(np.uint8), y.view(np.uint8))
    # the next step attends what is left
    b.kc, b.vc, b.ks, b.vs = caches
    b.table, b.lens = into.cpu().numpy(), lens
    out = torch.empty(b.tokens, hq, d, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(kv.attention_workspace_size(n, b.tokens, hq, hkv, d), dtype=torch.uint8, device="cuda")
    kv.attention_fp8(qd, *more, into, new, meta[2], 3, 100, d ** -0.5, True, out, ws, dev_status=b.status)
    ref, bound = F.attention(q.double().numpy(), b.host(), b.table, b.lens, b.start, d ** -0.5, True)
    _assert_attention(out, ref, bound)
    assert b.status.item() == 0


@pytest.mark.parametrize("hq", [2, 8, 32, 64])
def test_groups_that_do_not_ascend_are_reported_by_every_path(hq):
    """Short batches in one launch (tables without room to spare) read the groups for the status alone, the first
    sequences may be empty or unusable."""
    for wide in (1, WIDE):
        for seqs in ([(1, 20), (1, 33), (1, 8), (1, 50)], [(0, 20), (1, 33), (1, 8), (1, 50)]):
            s = Shared([(0, seqs)], 2, 64, wide=wide)
            b = s.b
            q = _bf16((b.tokens, hq, 64), 5)
            groups = np.arange(0, 400) // 100  # more entries than a CTA has threads
            for gs, bad in (([0, 3, 2], True), ([0, 2, 5], True), ([-1, 2, 4], True), (groups[::-1], True), ([0, 2, 4], False),
                            (groups, False), ([4, 4], False), ([0], False)):
                b.status.zero_()
                s.check(s.call(q, hq, group_start=gs, prefix=[0] * (len(gs) - 1)), q)
                assert b.status.item() == (_lib.DEV_BAD_SEQ if bad else 0), (wide, gs)
            lens = b.lens.copy()
            lens[0] = -1 if seqs[0][0] else 20
            b.status.zero_()
            s.call(q, hq, group_start=[0, 3, 2], prefix=[0, 0], meta=[torch.from_numpy(x).cuda() for x in (b.table, lens, b.start)])
            assert b.status.item() == _lib.DEV_BAD_SEQ


def _bounded(s, q, hq, max_seq_len, group_start=None, prefix=None):
    """Shared.call with a bound of the lengths."""
    b, scale = s.b, s.b.d ** -0.5
    gs = torch.tensor(s.group_start if group_start is None else group_start, dtype=torch.int32, device="cuda")
    pl = torch.tensor(s.prefix if prefix is None else prefix, dtype=torch.int32, device="cuda")
    ws = torch.empty(kv.attention_shared_workspace_size(len(b.seqs), len(pl), q.shape[0], hq, b.hkv, b.d), dtype=torch.uint8,
                     device="cuda").fill_(0xFF)
    out = torch.full((q.shape[0], hq, b.d), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((q.shape[0], hq), float("nan"), device="cuda")
    kv.attention_fp8_shared(q.cuda(), *b.device(), *b.meta(), b.max_len, max_seq_len, gs, pl, s.max_group, scale, out, ws, lse=lse,
                            dev_status=b.status)
    return out, lse


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (7, 1)])
def test_bounds_under_which_no_tile_is_split(d, hq, hkv):
    """Tiles in batches whose longest sequence rules splits out on the host.  Up to 256 positions no bound splits
    them: the same bits."""
    g = np.random.default_rng(d)
    ends = [(1, int(n)) for n in g.integers(1, 50, 34)]
    most = 1000 if d <= 128 else 500
    for groups, same in (([(192, ends), (0, [(40, 60), (1, 200)])], True),
                         ([(most - 100, ends[:20] + [(9, 20), (30, 90)]), (0, [(most // 2, most // 2)]), (64, [(1, 5)] * 40)], False)):
        s = Shared(groups, hkv, d, seed=d)
        q = _bf16((s.b.tokens, hq, d), 5)
        want = _bounded(s, q, hq, int(s.b.lens.max()))
        s.check(want, q)
        loose = _bounded(s, q, hq, 1 << 30)
        s.check(loose, q)
        assert not same or (torch.equal(want[0], loose[0]) and torch.equal(want[1], loose[1]))
        s.check(_bounded(s, q, hq, int(s.b.lens.max()), [0], []), q)
        assert s.b.status.item() == 0


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("hq", [2, 4, 16, 64])
def test_one_launch_by_the_bound_of_the_lengths(d, hq):
    """Tables with room to spare, lengths that fit the one-launch path, or just not."""
    for groups in ([(64, [(1, 33), (1, 64)])], [(0, [(1, 1)])], [(160, [(1, 9)] * 3), (0, [(1, 31)])]):
        s = Shared(groups, 2, d, seed=hq, wide=WIDE)
        q = _bf16((s.b.tokens, hq, d), 5)
        for bound in (int(s.b.lens.max()), 512, 4096):
            s.check(_bounded(s, q, hq, bound), q)
        assert s.b.status.item() == 0


@pytest.mark.parametrize("d", HEADS)
def test_more_sequences_over_a_longer_prefix(d):
    g = np.random.default_rng(d)
    _check([(2400, [(1, int(n)) for n in g.integers(1, 90, 40)])], 8, 2, d)


@pytest.mark.parametrize("d", [64, 192])
def test_more_pieces_than_a_warp_has_lanes(d):
    """One kv head's tile of 34 rows over 20480 positions is 40 pieces (80 at head size 192), and with 1284 sequences
    a row is merged by one warp: in two rounds or more."""
    prefix, members, others = 20480, 34, 1250
    g = np.random.default_rng(d)
    own = [int(n) for n in g.integers(1, 40, members)]
    short = [int(n) for n in g.integers(1, 20, others)]
    b = Batch([(0, prefix)] + [(1, n) for n in own + short], 1, d, seed=d).fill(2)
    table = np.full((members + others, prefix // 16 + 4), -1, np.int32)
    for i, n in enumerate(own + short):
        at = prefix // 16 if i < members else 0
        table[i, :at] = b.table[0, :at]
        table[i, at:at + -(-n // 16)] = b.table[1 + i, :-(-n // 16)]
    b.table, b.seqs, b.start = table, b.seqs[1:], b.start[1:]
    b.lens = np.array([prefix + n for n in own] + short, np.int32)
    s = Shared.__new__(Shared)
    s.b, s.group_start, s.prefix, s.max_group = b, np.array([0, members], np.int32), np.array([prefix], np.int32), members
    q = _bf16((b.tokens, 1, d), 5, 3.0)
    s.check(s.call(q, 1), q)
    assert b.status.item() == 0


def test_one_launch_captured_with_groups_that_change(monkeypatch):
    s = Shared([(64, [(1, 33), (1, 64), (1, 5)])], 4, 128, wide=1)
    b, hq = s.b, 16
    q = _bf16((b.tokens, hq, 128), 5)
    want = s.call(q, hq)
    s.check(want, q)
    dev, meta, dq = b.device(), b.meta(), q.cuda()
    gs, pl = (torch.from_numpy(x).cuda() for x in (s.group_start, s.prefix))
    ws = torch.empty(kv.attention_shared_workspace_size(3, 1, b.tokens, hq, 4, 128), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.attention_fp8_shared(dq, *dev, *meta, 1, b.table.shape[1] * 16, gs, pl, 3, 128 ** -0.5, out, ws, lse=lse, dev_status=b.status)
    for groups, status in (([0, 3], 0), ([1, 4], _lib.DEV_BAD_SEQ), ([2, 2], 0), ([3, 1], _lib.DEV_BAD_SEQ)):
        gs.copy_(torch.tensor(groups, dtype=torch.int32))
        b.status.zero_()
        out.zero_(), lse.zero_()
        graph.replay()
        s.check((out, lse), q)
        assert b.status.item() == status
    monkeypatch.setattr(_lib, "_fp8", _lib._Calls)
    b.status.zero_()
    s.check(s.call(q, hq, group_start=[0, 4]), q)
    assert b.status.item() == _lib.DEV_BAD_SEQ
