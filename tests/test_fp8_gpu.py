"""The FP8 block-scaled cache (kv_fp8_write, kv_fp8_read, kv_fp8_attention) and
kv_qk_norm_rope against the fp64 oracle.

Codes and scales are compared bit for bit, reads too.  Attention is held to
the bound that the oracle derives from the kernels' roundings (f16 weights,
fp32 sums) plus half a step of the bf16 output, 2^-8 of the value; the norm
likewise with fp32 arithmetic before its rounding."""

import math

import numpy as np
import pytest
import torch

import int4_token_head_gb300 as kv
from int4_token_head_gb300 import _lib, synthetic
from int4_token_head_gb300.paged import PagedKV
from oracle import fp8_oracle as F

pytestmark = pytest.mark.gpu
HEADS = [64, 96, 128, 192, 256]
SENT_SCALE = 0x7FC00A5A


class Batch:
    """Sequences (n, length) over a shuffled block table, with sentinel caches
    (codes 0xFF are E4M3 NaN, scales a NaN payload) on host and device."""

    def __init__(self, seqs, hkv, d, seed=0, spare=3, extra_width=1):
        self.seqs, self.hkv, self.d = seqs, hkv, d
        need = [-(-length // 16) for _, length in seqs]
        self.nb = sum(need) + spare
        perm = np.random.default_rng(seed).permutation(self.nb)
        self.table = np.full((len(seqs), max(need + [0]) + extra_width), -1, np.int32)
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = perm[at:at + n]
            at += n
        self.lens = np.array([length for _, length in seqs], np.int32)
        self.start = np.concatenate([[0], np.cumsum([n for n, _ in seqs])]).astype(np.int32)
        self.tokens = int(self.start[-1])
        self.max_len = max(n for n, _ in seqs)
        self.kc, self.vc = (np.full((self.nb, 16, hkv, d), 0xFF, np.uint8) for _ in range(2))
        self.ks, self.vs = (np.full((self.nb, hkv), SENT_SCALE, np.int32).view(np.float32) for _ in range(2))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def host(self):
        return self.kc, self.vc, self.ks, self.vs

    def device(self):
        k, v, ks, vs = (torch.from_numpy(x.copy()).cuda() for x in self.host())
        return k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), ks, vs

    def meta(self):
        return [torch.from_numpy(x).cuda() for x in (self.table, self.lens, self.start)]

    def fill(self, seed=1, k_gain=1.0, v_gain=1.0):
        """Every position of every sequence written by the oracle."""
        g = np.random.default_rng(seed)
        full = np.concatenate([[0], np.cumsum(self.lens)])
        for codes, scale, gain in ((self.kc, self.ks, k_gain), (self.vc, self.vs, v_gain)):
            x = torch.from_numpy(g.standard_normal((int(full[-1]), self.hkv, self.d)) * gain).to(torch.bfloat16)
            F.write(x.double().numpy(), self.table, self.lens, full, codes, scale)
        return self


def _bf16(shape, seed, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * gain).to(torch.bfloat16)


def _assert_caches(got, want):
    for a, b, name in zip(got, want, ["k codes", "v codes", "k scale", "v scale"]):
        a = a.view(torch.uint8).cpu().numpy() if a.dtype == torch.float8_e4m3fn else a.cpu().numpy().view(np.int32)
        b = b if b.dtype == np.uint8 else b.view(np.int32)
        assert np.array_equal(a, b), (name, np.argwhere(a != b)[:5])


def _write_both(b, k, v, dev, max_len=None):
    kv.write_fp8(k.cuda(), v.cuda(), *b.meta(), b.max_len if max_len is None else max_len, *dev, dev_status=b.status)
    torch.cuda.synchronize()
    F.write(k.double().numpy(), b.table, b.lens, b.start, b.kc, b.ks)
    F.write(v.double().numpy(), b.table, b.lens, b.start, b.vc, b.vs)


# ---------------------------------------------------------------------------
# write
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_write_prompts_bit_exact(d, hkv):
    seqs = [(33, 33), (1, 1), (16, 16), (0, 0), (15, 15), (47, 47), (17, 17)]
    b = Batch(seqs, hkv, d, seed=d + hkv)
    dev = b.device()
    k = _bf16((b.tokens, hkv, d), 3 * d + hkv) * torch.exp(torch.empty(b.tokens, hkv, 1).uniform_(-6, 6)).to(torch.bfloat16)
    v = _bf16((b.tokens, hkv, d), 5 * d + hkv, 0.01)
    k[5] = 0
    _write_both(b, k, v, dev)
    _assert_caches(dev, b.host())
    assert b.status.item() == 0


@pytest.mark.parametrize("d,hkv", [(64, 2), (96, 5), (128, 8), (192, 1), (256, 4)])
@pytest.mark.parametrize("n", [1, 3, 20])
def test_write_appends_follow_grown_scales(d, hkv, n):
    """Growing values: every append moves the codes that its block held."""
    lens = [0, 7, 15, 16, 30]
    b = Batch([(0, 96)] * len(lens), hkv, d, seed=d)  # blocks for 30 + 3 * 20 positions
    b.lens[:] = lens
    b.fill(seed=2, k_gain=1e-3, v_gain=0.05)
    dev = b.device()
    for step in range(3):
        b.lens += n
        b.start = (np.arange(len(lens) + 1) * n).astype(np.int32)
        b.tokens = len(lens) * n
        gain = 4.0 ** (step - 1)
        _write_both(b, _bf16((b.tokens, hkv, d), 10 + step, 0.01 * gain), _bf16((b.tokens, hkv, d), 20 + step, gain), dev, n)
        _assert_caches(dev, b.host())
    assert b.status.item() == 0


def test_write_scale_over_all_magnitudes():
    """Single-value rows: the scale is the smallest power of two that holds the
    value, for all bf16 mantissas over exponents beyond both ends of the range."""
    exps = [-133, -126, -70, -61, -53, -52, -51, -20, -1, 0, 8, 9, 40, 68, 69, 70, 127]
    vals = [(1 + m / 128) * 2.0 ** e * (-1) ** m for e in exps for m in range(0, 128, 1)]
    d, hkv = 64, 4
    n = len(vals) // hkv
    b = Batch([(1, 1)] * n, hkv, d, spare=0, extra_width=0)
    dev = b.device()
    k = torch.zeros(n, hkv, d, dtype=torch.float64)
    for i, x in enumerate(vals):
        k[i // hkv, i % hkv, (7 * i) % d] = x
    k = k.to(torch.bfloat16)
    _write_both(b, k, k.flip(0), dev)
    _assert_caches(dev, b.host())


def test_write_ties_and_subnormal_codes():
    d = 128
    b = Batch([(4, 4)], 1, d)
    dev = b.device()
    k = torch.zeros(4, 1, d, dtype=torch.float64)
    k[0, 0, 0] = 448.0                                         # scale 1
    k[1, 0, :64] = (16 + torch.arange(64) * 0.5) / 16          # ties between neighbours of four bits
    k[1, 0, 64:] = -(1 + torch.arange(64) * 2.0 ** -5)
    k[2, 0, :] = torch.arange(d) * 2.0 ** -11                  # subnormal codes and their ties
    k[3, 0, :] = -torch.arange(d) * 2.0 ** -12
    k = k.to(torch.bfloat16)
    _write_both(b, k, k.flip(2), dev)
    _assert_caches(dev, b.host())


def test_write_non_finite_values_are_stored_finite_and_reported():
    d, hkv = 96, 2
    b = Batch([(20, 20)], hkv, d)
    dev = b.device()
    k = _bf16((20, hkv, d), 1)
    k[3, 0, 5], k[4, 0, 6], k[17, 1, 0] = float("inf"), float("nan"), float("-inf")
    v = _bf16((20, hkv, d), 2)
    _write_both(b, k, v, dev)
    assert b.status.item() == _lib.DEV_NONFINITE
    _assert_caches(dev, b.host())
    assert np.isfinite(F.e4m3_values(b.kc[b.table[0, :1]])).all()


def test_write_begins_a_block_whatever_was_in_it():
    """Row 0 drops the old scale; a block that no call began counts as scale 2^-60."""
    d, hkv = 64, 1
    b = Batch([(16, 16), (1, 5)], hkv, d)
    b.ks[b.table[0, 0]], b.vs[b.table[0, 0]] = 2.0 ** 50, 2.0 ** 50
    b.kc[b.table[1, 0]], b.vc[b.table[1, 0]] = 0x38, 0x38
    b.ks[b.table[1, 0]], b.vs[b.table[1, 0]] = [0.75], [-1.0]
    dev = b.device()
    _write_both(b, _bf16((17, hkv, d), 1), _bf16((17, hkv, d), 2), dev)
    _assert_caches(dev, b.host())
    assert b.ks[b.table[0, 0], 0] < 1


def test_write_strided_inputs_padding_and_bad_metadata():
    d, hkv = 128, 3
    seqs = [(4, 20), (1, 3), (2, 40), (3, 9)]
    b = Batch(seqs, hkv, d)
    dev = b.device()
    pad = 5
    qkv = _bf16((b.tokens + pad, 7 * hkv * d + 8), 4).cuda()
    k = qkv[:, 8:8 + hkv * d].view(-1, hkv, d)[:b.tokens + pad]
    v = qkv[:, 8 + hkv * d:8 + 2 * hkv * d].view(-1, hkv, d)
    table, lens, start = b.meta()
    lens[3] = 2                       # shorter than its tokens
    table[2, 2] = b.nb                # the third sequence's last block does not exist
    kv.write_fp8(k, v, table, lens, start, 4, *dev, dev_status=b.status)
    torch.cuda.synchronize()
    assert b.status.item() == _lib.DEV_BAD_SEQ | _lib.DEV_BAD_BLOCK
    keep = b.start.copy()
    keep[4] = keep[3]                 # the oracle writes the first two and the third's nothing
    x = {"k": k.cpu().double().numpy(), "v": v.cpu().double().numpy()}
    for name, codes, scale in (("k", b.kc, b.ks), ("v", b.vc, b.vs)):
        F.write(x[name][:5], b.table[:2], b.lens[:2], b.start[:3], codes, scale)
    _assert_caches(dev, b.host())
    # a count above max_len is refused too, and nothing is written
    b.status.zero_()
    before = [t.clone() for t in dev]
    kv.write_fp8(k, v, *b.meta(), 0, *dev, dev_status=b.status)
    torch.cuda.synchronize()
    assert b.status.item() == _lib.DEV_BAD_SEQ
    for a, c in zip(dev, before):
        assert torch.equal(a.view(torch.uint8), c.view(torch.uint8))


def test_write_many_sequences_search():
    """Unit search over thousands of sequences, empty ones among them."""
    g = np.random.default_rng(8)
    seqs = []
    for _ in range(2500):
        n = int(g.choice([0, 0, 1, 1, 2, 15, 16, 17, 18, 33]))
        seqs.append((n, n + int(g.integers(0, 40))))
    b = Batch(seqs, 1, 64)
    b.fill()
    dev = b.device()
    _write_both(b, _bf16((b.tokens, 1, 64), 1, 3.0), _bf16((b.tokens, 1, 64), 2, 3.0), dev)
    _assert_caches(dev, b.host())
    assert b.status.item() == 0


# ---------------------------------------------------------------------------
# the calls
# ---------------------------------------------------------------------------
def test_call_module_and_ctypes_agree(monkeypatch):
    """The call module makes the calls; without it the same ones go through
    ctypes, as they do on an explicit stream.  A stream that is current is used."""
    assert _lib._calls() is not _lib._Calls
    q0 = _bf16((5, 4, 64), 1)
    b = Batch([(1, 30), (4, 50)], 2, 64).fill()
    cos_sin = torch.rand(64, 32)
    pos = torch.tensor([29, 46, 47, 48, 49])

    def run(stream=None):
        dev = b.device()
        q, k, v = q0.cuda(), q0[:, :2].cuda(), q0[:, 2:].contiguous().cuda()
        kv.qk_norm_rope(q, k, pos.cuda(), cos_sin.cuda(), None, None, 1e-6, q, k, dev_status=b.status, stream=stream)
        kv.write_fp8(k, v, *b.meta(), 4, *dev, dev_status=b.status, stream=stream)
        out = _attend(b, q, dev, 4, stream=stream)
        back = torch.empty_like(v), torch.empty_like(v)
        kv.read_fp8(*dev, *b.meta(), 4, *back, dev_status=b.status, stream=stream)
        return (q, k, out, *back, *(x.view(torch.uint8) for x in dev))

    want = run()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        got = run()
    other.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    assert all(torch.equal(x, y) for x, y in zip(want, run(torch.cuda.current_stream())))
    monkeypatch.setattr(_lib, "_fp8", _lib._Calls)
    assert all(torch.equal(x, y) for x, y in zip(want, run()))
    assert b.status.item() == 0


# ---------------------------------------------------------------------------
# read
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("hkv", [1, 5])
def test_read_bit_exact_and_rows_behind_untouched(d, hkv):
    seqs = [(33, 50), (1, 1), (0, 12), (1, 100), (16, 32), (7, 7)]
    b = Batch(seqs, hkv, d).fill(k_gain=5.0)
    pad, wide = 4, (hkv + 1) * d + 8
    out = [torch.full((b.tokens + pad, wide), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k, v = (o[:, 8:8 + hkv * d].view(-1, hkv, d) for o in out)
    kv.read_fp8(*b.device(), *b.meta(), b.max_len, k, v, dev_status=b.status)
    torch.cuda.synchronize()
    assert b.status.item() == 0
    for got, whole, codes, scale in ((k, out[0], b.kc, b.ks), (v, out[1], b.vc, b.vs)):
        for i, (n, length) in enumerate(seqs):
            for h in range(hkv):
                want = F.read(b.table, length, i, codes, scale, h)[length - n:]
                assert np.array_equal(got[b.start[i]:b.start[i + 1], h].double().cpu().numpy(), want)
        assert (whole[b.tokens:] == 7).all() and (whole[:, :8] == 7).all() and (whole[:, 8 + hkv * d:] == 7).all()


def test_read_bad_blocks_are_zeros():
    b = Batch([(40, 40), (3, 3)], 2, 64).fill()
    table, lens, start = b.meta()
    table[0, 1] = -1
    k, v = (torch.full((43, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kv.read_fp8(*b.device(), table, lens, start, 40, k, v, dev_status=b.status)
    assert b.status.item() == _lib.DEV_BAD_BLOCK
    assert (k[16:32] == 0).all() and (v[16:32] == 0).all()
    assert np.array_equal(v[40:, 1].double().cpu().numpy(), F.read(b.table, 3, 1, b.vc, b.vs, 1))


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def _attend(b, q, dev, hq, causal=True, window=0, scale=None, out=None, meta=None, max_q=None, stream=None):
    ws = torch.empty(kv.attention_workspace_size(len(b.seqs), q.shape[0], hq, b.hkv, b.d), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)  # its contents need no initialisation
    if out is None:
        out = torch.full((q.shape[0], hq, b.d), float("nan"), dtype=torch.bfloat16, device="cuda")
    kv.attention_fp8(q, *dev, *(meta or b.meta()), b.max_len if max_q is None else max_q, int(b.lens.max()),
                     b.d ** -0.5 if scale is None else scale, causal, out, ws, dev_status=b.status,
                     sliding_window=window, stream=stream)
    return out


def _assert_attention(got, ref, bound):
    got = got.double().cpu().numpy()
    err = np.abs(got - ref)
    tol = 2.0 ** -8 * np.abs(ref) + bound + 1e-30
    assert (err <= tol).all(), (np.argwhere(~(err <= tol))[:4], np.nanmax(err / tol), np.isnan(got).sum())


def _check(seqs, hq, hkv, d, causal=True, window=0, seed=0, k_gain=1.0, v_gain=1.0, q_gain=1.0, scale=None):
    b = Batch(seqs, hkv, d, seed=seed).fill(seed + 1, k_gain, v_gain)
    q = _bf16((b.tokens, hq, d), seed + 2, q_gain)
    out = _attend(b, q.cuda(), b.device(), hq, causal, window, scale)
    ref, bound = F.attention(q.double().numpy(), b.host(), b.table, b.lens, b.start, scale or d ** -0.5, causal, window)
    _assert_attention(out, ref, bound)
    assert b.status.item() == 0


DECODE = [(1, 1), (1, 16), (1, 17), (1, 100), (1, 333), (1, 31), (1, 48)]


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (4, 1), (6, 2), (8, 1), (5, 1), (32, 8), (24, 12), (9, 9)])
def test_decode(d, hq, hkv):
    _check(DECODE, hq, hkv, d, seed=d + hq)


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("hq,hkv,ql", [(2, 2, 4), (2, 1, 2), (4, 4, 8), (3, 3, 3), (8, 4, 3), (7, 7, 2)])
def test_decode_several_tokens(d, hq, hkv, ql):
    _check([(ql, 60), (1, 9), (0, 20), (ql, ql), (0, 0), (ql, 130)], hq, hkv, d, seed=d + ql)


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (16, 1), (10, 2), (7, 1), (64, 1), (3, 1)])
def test_prefill(d, hq, hkv):
    _check([(70, 70), (17, 200), (1, 40), (33, 33), (9, 9), (130, 150), (0, 3)], hq, hkv, d, seed=d + hq)


@pytest.mark.parametrize("d", HEADS)
def test_prefill_many_tiles_per_cta(d):
    """More tiles than SMs, so that every CTA goes through several, short and
    long ones after another, and rows without keys between them; run again and
    again for the same bits."""
    seqs = [(n, n) for n in (300, 290, 17, 310, 300, 5, 280, 300, 290, 40, 300, 310, 300, 260, 300, 290, 300, 33, 300, 310)]
    b = Batch(seqs, 8, d, seed=d).fill(3)
    q = _bf16((b.tokens, 16, d), 4)
    dev, meta = b.device(), b.meta()
    out = _attend(b, q.cuda(), dev, 16, meta=meta)
    for _ in range(20):
        assert torch.equal(_attend(b, q.cuda(), dev, 16, meta=meta), out)
    ref, bound = F.attention(q.double().numpy(), b.host(), b.table, b.lens, b.start, d ** -0.5, True)
    _assert_attention(out, ref, bound)
    # cross attention, a third of the sequences without keys
    seqs = [(200, (0, 400, 90)[i % 3]) for i in range(30)]
    b = Batch(seqs, 8, d, seed=d).fill(5)
    q = _bf16((b.tokens, 16, d), 6)
    out = _attend(b, q.cuda(), b.device(), 16, causal=False)
    ref, bound = F.attention(q.double().numpy(), b.host(), b.table, b.lens, b.start, d ** -0.5, False)
    _assert_attention(out, ref, bound)
    assert b.status.item() == 0


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("hq,hkv,seqs", [
    (12, 1, [(1, 700), (1, 1), (0, 9), (1, 33)]),                # 12 columns, one launch
    (32, 1, [(1, 40), (1, 900)]),
    (48, 3, [(1, n) for n in (2600, 17, 900, 16)]),              # 16 columns, the balanced split and its merge
    (16, 2, [(2, 2900), (4, 4), (3, 300), (1, 600), (0, 3)]),    # 8 to 32 columns side by side
    (28, 4, [(3, 700), (1, 3000), (3, 3), (2, 250)]),
    (8, 8, [(27, 1000), (9, 100), (1, 1)]),                      # up to 27 tokens
    (24, 3, [(1, 100 + 7 * i) for i in range(40)] + [(4, 500), (3, 900)]),  # room for 16 columns, not for 32
])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 50)])
def test_decode_many_columns(d, hq, hkv, seqs, causal, window):
    _check(seqs, hq, hkv, d, causal=causal, window=window, seed=d + hq)


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("hq,hkv,seqs", [
    (16, 1, [(3, 5000)]),                                              # one tile, every piece of one step or two
    (24, 2, [(7, 3000), (1, 9), (2, 2500), (30, 2100), (0, 5), (9, 9)]),  # pieces beside whole tiles and decodes
    (8, 8, [(200, 1999), (260, 2200)]),                                # several tiles a sequence, rows of unlike limits
])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 700)])
def test_prefill_split_over_keys(d, hq, hkv, seqs, causal, window):
    _check(seqs, hq, hkv, d, causal=causal, window=window, seed=d + hq)


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("n", [300, 1100])
def test_prefill_of_many_sequences(d, n):
    """More prompts than the schedule's threads, and more tiles than it looks at
    for splits, beside decodes."""
    seqs = [(1, 20 + i % 60) if i % 7 == 0 else (33 + i % 9, 42 + i % 50) for i in range(n)]
    _check(seqs, 1, 1, d, seed=n)


@pytest.mark.parametrize("d", HEADS)
def test_captured_splits_follow_the_lengths(d):
    """Graphs of a call whose tiles are split and of one that decodes many columns,
    in one workspace, replayed in turn after the lengths changed on the device."""
    graphs, calls = [], []
    ws = None
    for seqs, hq, hkv in (([(50, 3000), (40, 4000), (1, 30)], 4, 2), ([(3, 3000), (1, 700), (2, 2)], 16, 2)):
        b = Batch(seqs, hkv, d).fill(2)
        q = _bf16((b.tokens, hq, d), 3)
        dev, (table, lens, start) = b.device(), b.meta()
        out = torch.empty(b.tokens, hq, d, dtype=torch.bfloat16, device="cuda")
        if ws is None:
            ws = torch.empty(kv.attention_workspace_size(3, 120, 16, 2, d), dtype=torch.uint8, device="cuda")
        qc = q.cuda()

        def call(qc=qc, dev=dev, table=table, lens=lens, start=start, b=b, out=out):
            kv.attention_fp8(qc, *dev, table, lens, start, b.max_len, int(b.lens.max()), d ** -0.5, True, out, ws,
                             dev_status=b.status)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
        calls.append((b, q, lens, out, call))  # with every tensor that the graph reads
    for step in range(3):
        for g, (b, q, lens, out, _) in zip(graphs, calls):
            now = np.maximum(b.lens - 700 * step, np.diff(b.start)).astype(np.int32)
            lens.copy_(torch.from_numpy(now))
            out.fill_(float("nan"))
            g.replay()
            ref, bound = F.attention(q.double().numpy(), b.host(), b.table, now, b.start, d ** -0.5, True)
            _assert_attention(out, ref, bound)
            assert b.status.item() == 0


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 60)])
def test_prefill_of_broadcast_queries(d, causal, window):
    """One row as every token's queries (stride 0), which no tensor map holds:
    prefill without copies by the tensor memory accelerator."""
    b = Batch([(70, 90), (100, 1500), (40, 2600), (1, 200), (0, 7), (50, 50)] + [(64, 0)] * (not causal), 2, d).fill(1)
    row = _bf16((1, 6, d), 2)
    out = _attend(b, row.cuda().expand(b.tokens, 6, d), b.device(), 6, causal, window)
    q = row.double().numpy().repeat(b.tokens, 0)
    ref, bound = F.attention(q, b.host(), b.table, b.lens, b.start, d ** -0.5, causal, window)
    _assert_attention(out, ref, bound)


@pytest.mark.parametrize("d", HEADS)
def test_prefill_split_repeats_bits_and_skips_bad_blocks(d):
    b = Batch([(40, 3500), (5, 4100)], 2, d).fill(1)
    q = _bf16((b.tokens, 10, d), 2).cuda()
    dev = b.device()
    first = _attend(b, q, dev, 10)
    for _ in range(10):
        assert torch.equal(_attend(b, q, dev, 10), first)
    assert b.status.item() == 0
    # every block of the first sequence's keys but the last three is unusable:
    # whole pieces without a key
    table, lens, start = b.meta()
    table[0, :216] = -1
    out = _attend(b, q, dev, 10, meta=(table, lens, start))
    ref, bound = F.attention(q.double().cpu().numpy(), b.host(), table.cpu().numpy(), b.lens, b.start, d ** -0.5, True)
    _assert_attention(out, ref, bound)
    assert b.status.item() == _lib.DEV_BAD_BLOCK


@pytest.mark.parametrize("d", HEADS)
def test_prefill_rising_scores(d):
    """Keys that grow along the sequence: the running maximum moves in every step,
    by little and by more than the weights can hold."""
    b = Batch([(200, 900), (60, 700)], 2, d)
    g = np.random.default_rng(2)
    for i, (_, length) in enumerate(b.seqs):
        for codes, scale, rising in ((b.kc, b.ks, True), (b.vc, b.vs, False)):
            x = g.standard_normal((length, 2, d))
            if rising:
                x *= np.exp2(np.linspace(-4, 5, length))[:, None, None]
            x = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
            F.write(x, b.table[i:i + 1], [length], [0, length], codes, scale)
    q = _bf16((b.tokens, 8, d), 7)
    for causal in (True, False):
        out = _attend(b, q.cuda(), b.device(), 8, causal=causal)
        ref, bound = F.attention(q.double().numpy(), b.host(), b.table, b.lens, b.start, d ** -0.5, causal)
        _assert_attention(out, ref, bound)


@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("window", [1, 5, 16, 33, 1000])
def test_windows(d, window):
    _check([(1, 100), (1, 7), (40, 90), (2, 64), (3, 3)], 4, 2, d, window=window, seed=window)
    _check([(1, 100), (1, 7), (2, 64)], 2, 2, d, window=window, seed=window)
    _check([(1, 100), (7, 64), (2, 64)], 4, 1, d, causal=False, window=window, seed=window)


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 2), (16, 1)])
def test_cross_attention_of_another_length(d, hq, hkv):
    """Queries over keys that do not hold them: more queries than keys, none."""
    _check([(50, 3), (1, 0), (300, 64), (2, 1), (1, 200), (20, 0), (5, 17), (4, 150)], hq, hkv, d, causal=False, seed=d)
    _check([(1, 0), (2, 1), (1, 200), (1, 0)], hq, hkv, d, causal=False, seed=d)
    _check([(1, 0), (2, 0)], hq, hkv, d, causal=False, seed=d)


def test_long_decode_splits_and_merges():
    """One sequence over every CTA; a short one beside it."""
    for hq, hkv, d in ((8, 2, 128), (4, 4, 96), (8, 1, 256), (1, 1, 64), (32, 8, 128)):
        _check([(1, 9000), (1, 5)], hq, hkv, d, seed=d)


def test_extreme_scales():
    """Queries, keys and values far from one: the weights hold any V scale."""
    for k_gain, v_gain, q_gain in ((1e-6, 1e12, 1e6), (1e9, 1e-15, 1e-9), (1.0, 2.0 ** 60, 1.0), (3e-3, 1e-12, 300.0)):
        for seqs in ([(1, 200), (1, 33)], [(40, 100)]):
            _check(seqs, 4, 2, 128, k_gain=k_gain, v_gain=v_gain, q_gain=q_gain)
            _check(seqs, 2, 1, 256, k_gain=k_gain, v_gain=v_gain, q_gain=q_gain)


def test_blocks_of_very_different_v_scales():
    """Zero V blocks (scale 2^-60) beside large ones, at sharp and flat scores."""
    for seqs in ([(1, 160), (1, 90)], [(30, 160)]):
        b = Batch(seqs, 2, 128).fill(3)
        for i in range(0, b.nb, 3):
            b.vc[i], b.vs[i] = 0, 2.0 ** -60
        b.vs[1::3] *= 2.0 ** 20
        q = _bf16((b.tokens, 8, 128), 5, 4.0)
        out = _attend(b, q.cuda(), b.device(), 8)
        ref, bound = F.attention(q.double().numpy(), b.host(), b.table, b.lens, b.start, 128 ** -0.5, True)
        _assert_attention(out, ref, bound)


def test_sharp_scores_and_zero_queries():
    b = Batch([(1, 120), (20, 64)], 2, 64).fill(4, k_gain=30.0)
    q = _bf16((b.tokens, 4, 64), 6, 30.0)
    q[0, 1] = 0
    q[5, 2] = 0
    q[6, 3, :32] *= 1e-5
    out = _attend(b, q.cuda(), b.device(), 4)
    ref, bound = F.attention(q.double().numpy(), b.host(), b.table, b.lens, b.start, 64 ** -0.5, True)
    _assert_attention(out, ref, bound)


@pytest.mark.parametrize("d", HEADS)
def test_bad_blocks_are_masked_and_bad_sequences_skipped(d):
    b = Batch([(1, 100), (20, 60), (1, 40), (1, 16), (18, 30)], 2, d).fill()
    table, lens, start = b.meta()
    table[0, 2], table[1, 1], table[3, 0], table[4, 0] = -1, b.nb + 7, 1 << 30, -5
    lens[2] = 10 ** 6
    q = _bf16((b.tokens, 4, d), 3)
    out = torch.full((b.tokens + 3, 4, d), 7.0, dtype=torch.bfloat16, device="cuda")
    _attend(b, torch.cat([q, q[:3]]).cuda(), b.device(), 4, meta=(table, lens, start), out=out)
    assert b.status.item() == _lib.DEV_BAD_BLOCK | _lib.DEV_BAD_SEQ
    t2 = table.cpu().numpy()
    ref, bound = F.attention(q.double().numpy(), b.host(), t2, b.lens, b.start, d ** -0.5, True)
    keep = np.ones(b.tokens, bool)
    keep[b.start[2]:b.start[3]] = False
    _assert_attention(out[:b.tokens][torch.from_numpy(keep)], ref[keep], bound[keep])
    assert (out[b.start[2]:b.start[3]] == 7).all() and (out[b.tokens:] == 7).all()
    assert (out[b.start[3]] == 0).all()  # its only block is unusable
    assert (out[b.start[4]:b.start[4] + 4] == 0).all()  # rows that see the unusable block alone


def test_more_queries_than_max_query_len_is_a_bad_sequence():
    b = Batch([(1, 40), (3, 30)], 2, 64).fill()
    out = _attend(b, _bf16((4, 4, 64), 1).cuda(), b.device(), 4, max_q=1)
    assert b.status.item() == _lib.DEV_BAD_SEQ
    assert torch.isnan(out[1:]).all() and torch.isfinite(out[0]).all()


@pytest.mark.parametrize("d", HEADS)
def test_strided_views_give_the_same_bits(d):
    b = Batch([(1, 70), (30, 90), (3, 33)], 2, d).fill()
    hq = 8
    q = _bf16((b.tokens, hq, d), 9).cuda()
    want = _attend(b, q, b.device(), hq)
    wide_q = torch.zeros(b.tokens, hq * d + 24, dtype=torch.bfloat16, device="cuda")
    wide_o = torch.full((b.tokens, hq * d + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    wide_q[:, 8:8 + hq * d] = q.view(b.tokens, -1)
    _attend(b, wide_q[:, 8:8 + hq * d].view(-1, hq, d), b.device(), hq, out=wide_o[:, 8:8 + hq * d].view(-1, hq, d))
    assert torch.equal(wide_o[:, 8:8 + hq * d].reshape(b.tokens, hq, d), want)
    assert (wide_o[:, :8] == 7).all() and (wide_o[:, 8 + hq * d:] == 7).all()


def test_nan_queries_stay_in_their_rows():
    for seqs in ([(1, 40), (1, 70)], [(30, 60), (1, 33)]):
        b = Batch(seqs, 2, 128).fill()
        q = _bf16((b.tokens, 8, 128), 1)
        clean = _attend(b, q.cuda(), b.device(), 8)
        q[0, 3, 7], q[-1, 0, 0] = float("nan"), float("inf")
        out = _attend(b, q.cuda(), b.device(), 8)
        assert torch.isnan(out[0, 3]).all() and torch.isnan(out[-1, 0]).all()
        out[0, 3], out[-1, 0] = clean[0, 3], clean[-1, 0]
        assert torch.equal(out, clean)


def test_offsets_past_32_bits():
    """Blocks beyond 2^31 code bytes."""
    hkv, d = 32, 256
    nb = (1 << 31) // (16 * hkv * d) + 40
    b = Batch([(1, 50), (20, 40)], hkv, d, spare=0)
    b.fill()
    kc, vc = (torch.empty(nb, 16, hkv, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(nb, hkv, device="cuda") for _ in range(2))
    far = nb - b.nb
    for big, small in zip((kc, vc, ks, vs), b.host()):
        big[far:] = torch.from_numpy(small).cuda()
    table, lens, start = b.meta()
    table[table >= 0] += far
    dev = (kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn), ks, vs)
    q = _bf16((b.tokens, hkv, d), 2)
    out = _attend(b, q.cuda(), dev, hkv, meta=(table, lens, start))
    ref, bound = F.attention(q.double().numpy(), b.host(), b.table, b.lens, b.start, d ** -0.5, True)
    _assert_attention(out, ref, bound)
    k, v = _bf16((b.tokens, hkv, d), 3), _bf16((b.tokens, hkv, d), 4)
    kv.write_fp8(k.cuda(), v.cuda(), table, lens, start, 20, *dev, dev_status=b.status)
    F.write(k.double().numpy(), b.table, b.lens, b.start, b.kc, b.ks)
    assert np.array_equal(kc[far:].cpu().numpy(), b.kc)
    ko, vo = torch.empty_like(k, device="cuda"), torch.empty_like(v, device="cuda")
    kv.read_fp8(*dev, table, lens, start, 20, ko, vo, dev_status=b.status)
    want = F.read(b.table, 40, 1, b.kc, b.ks, hkv - 1)[20:]
    assert np.array_equal(ko[1:, hkv - 1].double().cpu().numpy(), want)
    assert b.status.item() == 0


def test_two_streams_and_a_replayed_graph():
    """Two calls at once with their own workspaces, then a captured step
    replayed over new inputs in the same buffers."""
    b = Batch([(1, 700), (1, 65), (20, 90), (1, 300)], 4, 128).fill()
    q = _bf16((b.tokens, 16, 128), 1).cuda()
    dev, meta = b.device(), b.meta()
    want = _attend(b, q, dev, 16, meta=meta)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append([_attend(b, q, dev, 16, meta=meta) for _ in range(5)])
    torch.cuda.synchronize()
    for per in outs:
        for o in per:
            assert torch.equal(o, want)
    ws = torch.empty(kv.attention_workspace_size(4, b.tokens, 16, 4, 128), dtype=torch.uint8, device="cuda")
    out, kk, vv = torch.empty_like(q), *(torch.empty(b.tokens, 4, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    buf_q = q.clone()
    new_k, new_v = (_bf16((b.tokens, 4, 128), s).cuda() for s in (5, 6))

    def step():
        kv.write_fp8(new_k, new_v, *meta, b.max_len, *dev, dev_status=b.status)
        kv.attention_fp8(buf_q, *dev, *meta, b.max_len, 700, 0.1, True, out, ws, dev_status=b.status)
        kv.read_fp8(*dev, *meta, b.max_len, kk, vv, dev_status=b.status)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (7, 8):
        buf_q.copy_(_bf16((b.tokens, 16, 128), seed))
        new_k.copy_(_bf16((b.tokens, 4, 128), seed + 10, 2.0))
        meta[1].copy_(torch.from_numpy(b.lens - (seed - 7)))
        state = [t.clone() for t in dev]
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, kk, vv, *dev)]
        for t, s in zip(dev, state):
            t.copy_(s)
        step()
        torch.cuda.synchronize()
        for a, c in zip(got, (out, kk, vv, *dev)):
            assert torch.equal(a.view(torch.uint8), c.view(torch.uint8))
    assert b.status.item() == 0


def test_repeated_calls_give_the_same_bits():
    b = Batch([(1, 5000), (1, 77), (40, 300), (3, 1000)], 2, 128).fill()
    q = _bf16((b.tokens, 8, 128), 1).cuda()
    dev, meta = b.device(), b.meta()
    want = _attend(b, q, dev, 8, meta=meta)
    for _ in range(10):
        assert torch.equal(_attend(b, q, dev, 8, meta=meta), want)


# ---------------------------------------------------------------------------
# norm and rotary rotation
# ---------------------------------------------------------------------------
def _norm_inputs(t, hq, hkv, d, rot, seed=0):
    g = np.random.default_rng(seed)
    angle = g.uniform(-100, 100, (50, rot // 2))
    cs = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1)).float()
    w = [torch.from_numpy(g.uniform(0.5, 1.5, d)).to(torch.bfloat16) for _ in range(2)]
    return _bf16((t, hq, d), seed + 1), _bf16((t, hkv, d), seed + 2, 3.0), torch.from_numpy(g.integers(0, 50, t)), cs, w


def _norm_check(got, x, w, eps, cs, pos, inter):
    """fp32: the sum of squares D 2^-24, rsqrt 2^-22, the products and the
    rotation's two terms a few 2^-24 each; then bf16's half step."""
    d = x.shape[-1]
    wn = None if w is None else w.double().numpy()
    ref = F.norm_rope(x.double().numpy(), wn, eps, None if cs is None else cs.double().numpy(), pos.numpy(), inter)
    y = np.abs(F.norm_rope(x.double().numpy(), wn, eps, None, None, False))
    size = np.abs(ref)
    if cs is not None and cs.shape[1]:  # |a cos| + |b sin| of each rotated element
        c = np.abs(cs.double().numpy())
        half = cs.shape[1] // 2
        i = np.arange(half)
        lo, hi = (2 * i, 2 * i + 1) if inter else (i, i + half)
        co, si = c[pos.numpy()][:, None, :half], c[pos.numpy()][:, None, half:]
        size[..., lo], size[..., hi] = y[..., lo] * co + y[..., hi] * si, y[..., hi] * co + y[..., lo] * si
    tol = 2.0 ** -8 * np.abs(ref) + (d / 2 + 12) * 2.0 ** -24 * size * 1.01 + 1e-38
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("t,hq,hkv", [(1, 1, 1), (3, 8, 2), (67, 5, 5), (2, 40, 8)])
def test_norm_rope(d, inter, t, hq, hkv):
    for rot in sorted({16, 32, d // 2 // 16 * 16, d - 16, d}):
        q, k, pos, cs, w = _norm_inputs(t, hq, hkv, d, rot, seed=d + rot)
        q[0, 0] = 0
        qo, ko = torch.empty_like(q, device="cuda"), torch.empty_like(k, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        kv.qk_norm_rope(q.cuda(), k.cuda(), pos.cuda(), cs.cuda(), w[0].cuda(), w[1].cuda(), 1e-6, qo, ko,
                        interleaved=inter, dev_status=status)
        assert status.item() == 0
        _norm_check(qo, q, w[0], 1e-6, cs, pos, inter)
        _norm_check(ko, k, w[1], 1e-6, cs, pos, inter)


@pytest.mark.parametrize("d", [64, 96, 192])
def test_norm_rope_in_place_strided_and_parts(d):
    t, hq, hkv, rot = 19, 6, 2, 32
    q, k, pos, cs, w = _norm_inputs(t, hq, hkv, d, rot)
    fused = torch.full((t, (hq + 2 * hkv) * d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    fq, fk = fused[:, 8:8 + hq * d].view(t, hq, d), fused[:, 8 + hq * d:8 + (hq + hkv) * d].view(t, hkv, d)
    fq.copy_(q)
    fk.copy_(k)
    dw = [x.cuda() for x in w]
    qo, ko = torch.empty_like(q, device="cuda"), torch.empty_like(k, device="cuda")
    kv.qk_norm_rope(fq, fk, pos.cuda(), cs.cuda(), *dw, 1e-5, qo, ko)
    kv.qk_norm_rope(fq, fk, pos.cuda(), cs.cuda(), *dw, 1e-5, fq, fk)  # in place
    assert torch.equal(fq, qo) and torch.equal(fk, ko)
    assert (fused[:, :8] == 7).all() and (fused[:, 8 + (hq + hkv) * d:] == 7).all()
    _norm_check(qo, q, w[0], 1e-5, cs, pos, False)
    kv.qk_norm_rope(q.cuda(), k.cuda(), None, None, *dw, 1e-5, qo, ko)  # the norm alone
    _norm_check(ko, k, w[1], 1e-5, None, pos, False)
    kv.qk_norm_rope(q.cuda(), k.cuda(), pos.cuda(), cs.cuda(), None, None, 0.0, qo, ko)  # the rotation alone
    _norm_check(qo, q, None, 0.0, cs, pos, False)


def test_norm_rope_bad_position_leaves_its_rows():
    q, k, pos, cs, w = _norm_inputs(8, 4, 2, 64, 64)
    pos[2], pos[5] = 50, -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo, ko = (torch.full_like(x, 7.0, device="cuda") for x in (q, k))
    kv.qk_norm_rope(q.cuda(), k.cuda(), pos.cuda(), cs.cuda(), w[0].cuda(), w[1].cuda(), 1e-6, qo, ko, dev_status=status)
    assert status.item() == _lib.DEV_BAD_POS
    bad = torch.tensor([2, 5])
    assert (qo[bad] == 7).all() and (ko[bad] == 7).all()
    keep = torch.tensor([0, 1, 3, 4, 6, 7])
    _norm_check(qo[keep], q[keep], w[0], 1e-6, cs, pos[keep], False)


# ---------------------------------------------------------------------------
# the operators together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("hq,hkv,d,rot", [(8, 2, 128, 128), (4, 4, 96, 64), (6, 1, 192, 192), (16, 4, 64, 32)])
def test_a_prompt_and_its_decode_steps(hq, hkv, d, rot):
    """norm_rope -> write -> attend for a prompt step and decode steps, then the
    whole history read back; each stage is held to the oracle on the stage's own
    inputs, codes and scales bit for bit over all steps."""
    prompts = [37, 5, 64]
    b = Batch([(n, n + 6) for n in prompts], hkv, d)
    dev = b.device()
    g = np.random.default_rng(1)
    angle = np.arange(128)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    cs = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1)).float()
    w = [torch.from_numpy(g.uniform(0.5, 1.5, d)).to(torch.bfloat16) for _ in range(2)]
    lens = np.zeros(3, np.int32)
    for step, counts in enumerate([prompts, [1, 1, 1], [2, 0, 1], [1, 3, 1], [1, 1, 1]]):
        lens = lens + np.array(counts, np.int32)
        b.lens, b.start = lens, np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        b.tokens, b.max_len = int(b.start[-1]), max(counts)
        pos = torch.from_numpy(np.concatenate([np.arange(lens[i] - counts[i], lens[i]) for i in range(3)]))
        qkv = _bf16((b.tokens, (hq + 2 * hkv) * d), 30 + step, 2.0)
        fused = qkv.cuda()
        q, k, v = (x.view(b.tokens, -1, d) for x in (fused[:, :hq * d], fused[:, hq * d:(hq + hkv) * d], fused[:, (hq + hkv) * d:]))
        kv.qk_norm_rope(q, k, pos.cuda(), cs.cuda(), w[0].cuda(), w[1].cuda(), 1e-6, q, k, dev_status=b.status)
        _norm_check(k, qkv[:, hq * d:(hq + hkv) * d].reshape(b.tokens, hkv, d), w[1], 1e-6, cs, pos, False)
        kv.write_fp8(k, v, *b.meta(), b.max_len, *dev, dev_status=b.status)
        F.write(k.double().cpu().numpy(), b.table, b.lens, b.start, b.kc, b.ks)
        F.write(v.double().cpu().numpy(), b.table, b.lens, b.start, b.vc, b.vs)
        _assert_caches(dev, b.host())
        out = _attend(b, q, dev, hq)
        ref, bound = F.attention(q.double().cpu().numpy(), b.host(), b.table, b.lens, b.start, d ** -0.5, True)
        _assert_attention(out, ref, bound)
    b.start = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    k, v = (torch.empty(int(b.start[-1]), hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kv.read_fp8(*dev, *b.meta(), int(lens.max()), k, v, dev_status=b.status)
    for i in range(3):
        assert np.array_equal(v[b.start[i]:b.start[i + 1], 0].double().cpu().numpy(), F.read(b.table, lens[i], i, b.vc, b.vs, 0))
    assert b.status.item() == 0


@pytest.mark.parametrize("name", ["tiny", "mixed"])
def test_paged_cache_step(name):
    """PagedKV(fmt="fp8") on the synthetic workloads, sampled rows against the oracle."""
    over = dict(prefills=2, decodes=5, prefill_range=(100, 200), decode_range=(100, 900)) if name == "mixed" else {}
    w = synthetic.make_workload(name, **over)
    pk = PagedKV(w, fmt="fp8")
    pk.populate_history(gen_device="cpu", chunk_tokens=300)
    q, k, v, slots = pk.step_inputs(gen_device="cpu")
    out = torch.empty_like(q)
    pk.step(q, k, v, slots, out)
    kk, vv = torch.empty_like(k), torch.empty_like(v)
    pk.read_tokens(kk, vv)
    assert pk.status.item() == 0
    host = [t.view(torch.uint8).cpu().numpy() if t.dtype == torch.float8_e4m3fn else t.cpu().numpy()
            for t in (pk.k_cache, pk.v_cache, pk.k_scale, pk.v_scale)]
    ref, bound = F.attention(q.double().cpu().numpy(), host, w.block_table.numpy(), w.seq_lens.numpy(),
                             w.query_start_loc.numpy(), pk.softmax_scale, True)
    _assert_attention(out, ref, bound)
    want = (np.full(host[0].shape, 0xFF, np.uint8), np.full(host[2].shape, np.nan, np.float32))
    for s in range(w.num_seqs):
        ql, n = w.seqs[s]
        x = w.seq_kv(s, "cpu")[1].double().numpy()
        row = w.block_table[s:s + 1].numpy()
        if n > ql:
            F.write(x[:n - ql], row, [n - ql], [0, n - ql], *want)
        F.write(x[n - ql:], row, [n], [0, ql], *want)
    assert np.array_equal(host[1], want[0]) and np.array_equal(host[3], want[1], equal_nan=True)
    assert math.isfinite(float(vv.float().abs().max())) and (vv.float() - v.float()).abs().max() < 0.3


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("seqs", [[(1, 40), (1, 9)], [(40, 90), (7, 7)]])
def test_one_query_row_for_every_token(d, seqs):
    """q may repeat one row (token stride 0)."""
    b = Batch(seqs, 2, d).fill()
    q = _bf16((1, 4, d), 1).expand(b.tokens, 4, d)
    out = _attend(b, q.cuda()[:1].expand(b.tokens, 4, d), b.device(), 4)
    ref, bound = F.attention(q.double().numpy(), b.host(), b.table, b.lens, b.start, d ** -0.5, True)
    _assert_attention(out, ref, bound)


@pytest.mark.parametrize("d", HEADS)
def test_negative_and_zero_softmax_scale(d):
    for scale in (-0.3, 0.0):
        for seqs in ([(1, 70), (1, 9)], [(40, 90), (7, 7)]):
            b = Batch(seqs, 2, d).fill()
            q = _bf16((b.tokens, 4, d), 1)
            out = _attend(b, q.cuda(), b.device(), 4, scale=scale)
            ref, bound = F.attention(q.double().numpy(), b.host(), b.table, b.lens, b.start, scale, True)
            _assert_attention(out, ref, bound)


# ---------------------------------------------------------------------------
# logits far from zero
# ---------------------------------------------------------------------------
def _far(seqs, hkv, group, d, logit, seed=0, v_gain=1.0):
    """A filled batch and its queries whose scores all lie near `logit`: a common
    first element of the queries, and of the keys with its sign."""
    b = Batch(seqs, hkv, d, seed=seed)
    g = np.random.default_rng(seed + 1)
    full = np.concatenate([[0], np.cumsum(b.lens)])
    size = (abs(logit) * d ** 0.5) ** 0.5
    for codes, scale, gain in ((b.kc, b.ks, 1.0), (b.vc, b.vs, v_gain)):
        x = g.standard_normal((int(full[-1]), hkv, d)) * gain
        if codes is b.kc:
            x[..., 0] = math.copysign(size, logit)
        x = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
        F.write(x, b.table, b.lens, full, codes, scale)
    q = _bf16((b.tokens, hkv * group, d), seed + 2)
    q[..., 0] = size
    return b, q


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("group", [1, 2])
@pytest.mark.parametrize("window", [1, 20, 100])
@pytest.mark.parametrize("logit,v_gain", [(-100, 1.0), (-300, 1.0), (-60, 2.0 ** -50), (300, 1.0)])
def test_windows_where_every_logit_is_far_from_zero(d, group, window, logit, v_gain):
    """Softmax does not depend on a common offset: rows of a tile whose window
    starts behind the tile's first keys, prefill and decode alike."""
    for seqs, causal in (([(300, 300), (5, 260), (1, 200), (140, 500)], True), ([(280, 300), (1, 90)], False)):
        b, q = _far(seqs, 2, group, d, logit, seed=window, v_gain=v_gain)
        out = _attend(b, q.cuda(), b.device(), 2 * group, causal=causal, window=window)
        ref, bound = F.attention(q.double().numpy(), b.host(), b.table, b.lens, b.start, d ** -0.5, causal, window)
        _assert_attention(out, ref, bound)
        assert b.status.item() == 0


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("bad", [8, 17])
@pytest.mark.parametrize("logit", [-100, -300])
def test_first_blocks_unusable_where_every_logit_is_far_from_zero(d, bad, logit):
    """The rows' first usable keys come a step or more after the tile's first."""
    b, q = _far([(250, 400), (40, 300), (1, 350)], 2, 2, d, logit)
    table, lens, start = b.meta()
    table[:, :bad] = -1
    for causal in (True, False):
        out = _attend(b, q.cuda(), b.device(), 4, causal=causal, meta=(table, lens, start))
        ref, bound = F.attention(q.double().numpy(), b.host(), table.cpu().numpy(), b.lens, b.start, d ** -0.5, causal)
        _assert_attention(out, ref, bound)
    assert b.status.item() == _lib.DEV_BAD_BLOCK


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 4, 2 ** 30])
def test_windows_wider_than_any_sequence(d, window):
    """The largest windows hide nothing, of queries before the first key neither."""
    for seqs, hq, hkv in (([(9, 4), (2, 30), (1, 0)], 2, 2),               # one launch
                          ([(5, 1), (8, 3000), (7, 0), (3, 2)], 8, 2),     # planned decode of many columns
                          ([(300, 5), (40, 200), (20, 0), (1, 1)], 4, 2),  # prefill
                          ([(33, 2900), (70, 3)], 4, 2)):                  # tiles split over their keys
        _check(seqs, hq, hkv, d, causal=False, window=window, seed=d)
    _check([(30, 60), (1, 90), (7, 7)], 4, 2, d, window=window, seed=d)


# ---------------------------------------------------------------------------
# decode beside prefill
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("d", HEADS)
def test_decode_beside_prefill_sees_what_was_written_just_before(d):
    """Mixed calls whose queries, keys, values, table, lengths and schedule change
    from call to call in the same memory, nothing waited for in between, eager
    and replayed: the bits of a call that had the GPU to itself."""
    hq, hkv = 8, 2
    shapes = [[(1, 400), (90, 200), (1, 90), (1, 700), (40, 300)], [(60, 60), (1, 30), (1, 900), (70, 500), (1, 64)],
              [(1, 16), (1, 17), (128, 150), (3, 800), (1, 333)]]
    tokens = max(sum(n for n, _ in seqs) for seqs in shapes)
    batches = [Batch(seqs, hkv, d, seed=i).fill(i + 1) for i, seqs in enumerate(shapes)]
    nb, width = max(b.nb for b in batches), max(b.table.shape[1] for b in batches)

    def padded(b, seed):
        """One shape for all: spare blocks, table columns and tokens behind."""
        codes = [np.concatenate([x, np.full((nb - b.nb, *x.shape[1:]), 0xFF, np.uint8)]) for x in (b.kc, b.vc)]
        scales = [np.concatenate([x, np.full((nb - b.nb, hkv), np.nan, np.float32)]) for x in (b.ks, b.vs)]
        table = np.pad(b.table, ((0, 0), (0, width - b.table.shape[1])), constant_values=-1)
        return [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in (*codes, *scales, table, b.lens, b.start)] + [
            _bf16((tokens, hq, d), seed).cuda()]

    inputs = [padded(b, 10 + i) for i, b in enumerate(batches)]
    live = [x.clone() for x in inputs[0]]
    out = torch.empty(tokens, hq, d, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(kv.attention_workspace_size(5, tokens, hq, hkv, d), dtype=torch.uint8, device="cuda")
    new = [(_bf16((tokens, hkv, d), 20 + i).cuda(), _bf16((tokens, hkv, d), 30 + i).cuda()) for i in range(3)]
    new_k, new_v = (x.clone() for x in new[0])

    def step():
        kc, vc, ks, vs, table, lens, start, q = live
        kv.write_fp8(new_k, new_v, table, lens, start, 128, kc, vc, ks, vs, dev_status=status)
        kv.attention_fp8(q, kc, vc, ks, vs, table, lens, start, 128, 900, d ** -0.5, True, out, ws, dev_status=status)

    def load(i):
        for x, y in zip((*live, new_k, new_v), (*inputs[i], *new[i])):
            x.copy_(y)

    want = []
    for i in range(3):
        load(i)
        torch.cuda.synchronize()
        ws.fill_(0xFF)
        step()
        torch.cuda.synchronize()
        want.append(out[:batches[i].tokens].clone())
        assert torch.isfinite(want[i]).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for run in (step, graph.replay):
        got = []
        for n in range(12):
            load(n % 3)
            run()
            got.append(out[:batches[n % 3].tokens].clone())
        for n, x in enumerate(got):
            assert torch.equal(x, want[n % 3])
    assert status.item() == 0


# ---------------------------------------------------------------------------
# V scales at both ends of their range
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("hq,hkv,seqs,broadcast", [
    (4, 2, [(1, 200), (1, 90), (1, 700)], False),                # one launch
    (4, 4, [(1, 3000), (1, 300)], False),                        # planned decode: four blocks at once,
    (4, 1, [(1, 9000), (1, 300)], False),                        # two, one, and warps of columns
    (8, 1, [(1, 9000), (1, 40)], False),
    (16, 2, [(3, 3000), (1, 700), (2, 60)], False),
    (4, 2, [(100, 300), (300, 300), (40, 90), (1, 500)], False),  # prefill beside decode
    (8, 2, [(33, 2900), (5, 700)], False),                       # tiles split over their keys
    (4, 2, [(60, 260), (9, 2900)], True),                        # queries without a tensor map
])
@pytest.mark.parametrize("gap", [0, 8, 20, -30])
def test_v_scales_at_both_ends_of_their_range(d, hq, hkv, seqs, broadcast, gap):
    """One block of scale 2^60 among blocks of 2^-60, its scores `gap` binary
    orders above the others': their output does not show beside its, their
    share of the denominator does."""
    for where in (0.0, 0.5, 1.0):  # the block's place: first seen, later, in another piece
        b = Batch(seqs, hkv, d, seed=d).fill(4)
        g = np.random.default_rng(7)
        for i, (_, length) in enumerate(seqs):
            at = round(where * ((length - 1) // 16))
            x = g.standard_normal((length, hkv, d)) * 0.05
            x[:, :, 0] = 0.0
            x[16 * at:16 * at + 16, :, 0] = gap * math.log(2)
            x = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
            F.write(x, b.table[i:i + 1], [length], [0, length], b.kc, b.ks)
            held = b.table[i, :-(-length // 16)]
            b.vs[held] = 2.0 ** -60
            b.vs[held[at]] = 2.0 ** 60
        q = _bf16((1 if broadcast else b.tokens, hq, d), 5)
        q[..., 0] = d ** 0.5
        full = q.expand(b.tokens, hq, d)
        out = _attend(b, q.cuda().expand(b.tokens, hq, d), b.device(), hq)
        ref, bound = F.attention(full.double().numpy(), b.host(), b.table, b.lens, b.start, d ** -0.5, True)
        _assert_attention(out, ref, bound)
        assert b.status.item() == 0


# ---------------------------------------------------------------------------
# the smaller workspace
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("hq,hkv,seqs", [
    (4, 2, [(1, 300), (1, 40)]),                                  # one launch
    (8, 2, [(1, 6000), (1, 17), (2, 700)]),
    (16, 1, [(1, 3000), (3, 500), (1, 3)]),                       # 16 and 48 columns
    (8, 8, [(200, 1999), (260, 2200)]),                           # tiles that would be split
    (24, 2, [(7, 3000), (1, 9), (30, 2100), (0, 5), (9, 9)]),
    (2, 2, [(1, 20)] + [(0, 0)] * 40),                            # mostly sequences without queries
])
def test_attention_in_the_workspace_of_int4(d, hq, hkv, seqs):
    """kv_int4_attention_workspace_size bytes are enough: whole tiles, eight
    columns; nothing is touched behind them."""
    b = Batch(seqs, hkv, d, seed=d).fill(2)
    q = _bf16((b.tokens, hq, d), 3)
    sizes = len(seqs), b.tokens, hq, hkv, d
    least, best = (kv.attention_workspace_size(*sizes, fmt=f) for f in ("int4", "fp8"))
    assert least < best
    ref, bound = F.attention(q.double().numpy(), b.host(), b.table, b.lens, b.start, d ** -0.5, True)
    for size in (least, best - 256, best):
        whole = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        out = torch.full((b.tokens, hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        kv.attention_fp8(q.cuda(), *b.device(), *b.meta(), b.max_len, int(b.lens.max()), d ** -0.5, True, out,
                         whole[:size], dev_status=b.status)
        _assert_attention(out, ref, bound)
        assert (whole[size:] == 0xA5).all() and b.status.item() == 0
    with pytest.raises(kv.KvInt4Error, match="workspace"):
        kv.attention_fp8(q.cuda(), *b.device(), *b.meta(), b.max_len, int(b.lens.max()), d ** -0.5, True, out,
                         whole[:1024], dev_status=b.status)


# ---------------------------------------------------------------------------
# the two bindings' checks
# ---------------------------------------------------------------------------
def _changed(x):
    """What a call may not take in place of the tensor x, and some that it may."""
    yield "cpu", x.cpu()
    yield "type", x.to(torch.float64) if x.dtype != torch.float64 else x.float()
    yield "half", x.to(torch.float16)
    yield "int64", x.to(torch.int64)
    yield "bytes", x.to(torch.int32).to(torch.uint8)
    yield "another row", torch.cat([x, x[:1] if x.shape[0] else x.new_zeros(1, *x.shape[1:])])
    yield "less of the last dimension", x[..., :-1]
    yield "a dimension more", x[None]
    yield "flat", x.reshape(-1)
    yield "every other element", torch.stack([x, x], -1).flatten(-2)[..., ::2]
    yield "turned", x.transpose(0, -1).contiguous().transpose(0, -1)
    yield "wide rows", torch.cat([x, x], -1)[..., :x.shape[-1]]
    yield "none", None


@pytest.mark.parametrize("op", ["write", "read", "attention", "norm"])
def test_both_bindings_refuse_the_same_calls(monkeypatch, op):
    """Every argument changed in turn, in calls without tokens (nothing is
    launched): through the call module and through ctypes the same outcome."""
    assert _lib._calls() is not _lib._Calls
    d, cuda = 64, dict(device="cuda")
    cache = [torch.zeros(4, 16, 2, d, dtype=torch.uint8, **cuda).view(torch.float8_e4m3fn) for _ in range(2)] + [
        torch.ones(4, 2, **cuda) for _ in range(2)]
    seqs = [torch.zeros(3, 5, dtype=torch.int32, **cuda), torch.zeros(3, dtype=torch.int32, **cuda),
            torch.zeros(4, dtype=torch.int32, **cuda)]
    kv_rows = [torch.zeros(0, 2, d, dtype=torch.bfloat16, **cuda) for _ in range(2)]
    q_rows = [torch.zeros(0, 4, d, dtype=torch.bfloat16, **cuda) for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, **cuda)
    w = torch.ones(d, dtype=torch.bfloat16, **cuda)
    f, args = {
        "write": (kv.write_fp8, [*kv_rows, *seqs, 3, *cache, status]),
        "read": (kv.read_fp8, [*cache, *seqs, 3, *kv_rows, status]),
        "attention": (kv.attention_fp8, [q_rows[0], *cache, *seqs, 3, 64, 0.1, True, q_rows[1],
                                         torch.zeros(64, dtype=torch.uint8, **cuda), status]),
        "norm": (kv.qk_norm_rope, [q_rows[0], kv_rows[0], torch.zeros(0, dtype=torch.int64, **cuda), torch.ones(8, 32, **cuda),
                                   w, w.clone(), 1e-6, q_rows[1], kv_rows[1], False, status]),
    }[op]

    def outcome(args):
        try:
            return f(*args)
        except Exception as e:
            return type(e), str(e)

    module, refused = _lib._calls(), 0
    assert outcome(args) is None
    for i, x in enumerate(args):
        for what, y in _changed(x) if torch.is_tensor(x) else [("text", "3"), ("none", None), ("half", 0.5), ("large", 1 << 40)]:
            call = [*args[:i], y, *args[i + 1:]]
            monkeypatch.setattr(_lib, "_fp8", module)
            first = outcome(call)
            monkeypatch.setattr(_lib, "_fp8", _lib._Calls)
            assert outcome(call) == first, (i, what)
            refused += first is not None
    assert refused > 5 * len(args)


@pytest.mark.parametrize("d", HEADS)
@pytest.mark.parametrize("gain,eps", [(2.0 ** 70, 1e-6), (2.0 ** 120, 1e-6), (2.0 ** 120, 0.0), (2.0 ** -70, 0.0),
                                      (2.0 ** -110, 0.0), (2.0 ** -70, 2.0 ** -140), (2.0 ** -60, 2.0 ** -120)])
def test_norm_of_vectors_whose_squares_leave_fp32(d, gain, eps):
    """Beside ordinary vectors and one of zeros in the same warp."""
    q, k, pos, cs, w = _norm_inputs(9, 6, 2, d, 32, seed=d)
    far = torch.ones(9, 6, 1, dtype=torch.bool)
    far[::2, 1::3] = False
    q = torch.where(far, (q.double() * gain).to(torch.bfloat16), q)
    k = (k.double() * gain).to(torch.bfloat16)
    if eps > 0:
        q[1, 0] = 0
    qo, ko = torch.empty_like(q, device="cuda"), torch.empty_like(k, device="cuda")
    kv.qk_norm_rope(q.cuda(), k.cuda(), pos.cuda(), cs.cuda(), w[0].cuda(), w[1].cuda(), eps, qo, ko)
    _norm_check(qo, q, w[0], eps, cs, pos, False)
    _norm_check(ko, k, w[1], eps, cs, pos, False)
