"""GPU parity of the attention over the paged cache against the fp64 oracle.

Tolerance, from the arithmetic: a score is an fp32 sum of D products whose
query factor carries 22 bits, scaled and brought to base two; its error is
taken as (4 sqrt(D) + 16) * 2^-24 of scale * sum |q k| (the roundings of the
sum add up like a random walk), and twice that is the relative error of a
weight.  The weighted sum over n tokens adds (sqrt(n) + 64) * 2^-24.  Both act
on sum w |v| / sum w."""
import math

import numpy as np
import pytest

import bit_gemv_amd as rf
from _gpu import announce, device, empty, host, to_dev, torch
from oracle import attention as oa

pytestmark = pytest.mark.gpu

F16, I8 = rf.KV_F16, rf.KV_I8


class Setup:
    """A cache whose sequences hold given lengths, everything else poisoned."""

    def __init__(self, fmt, lens, T, H, Hkv, D, P, seed=0, q_gain=1.5, extra=0):
        rng = np.random.default_rng(seed)
        i8 = fmt == I8
        B = len(lens)
        need = [max(0, -(-n // P)) for n in lens]
        width = max(max(need), 1) + extra
        pages = sum(need) + 2
        order = rng.permutation(pages)
        table = np.full((B, width), -1, np.int32)
        dt = np.int8 if i8 else np.float16
        poison = 127 if i8 else np.nan
        kk, vv = (np.full((pages, P, Hkv, D), poison, dt) for _ in range(2))
        ks, vs = (np.full((pages, P, Hkv, D // 32), np.nan, np.float32) for _ in range(2))
        self.k, self.v = [], []                              # per sequence, the values held
        at = 0
        for b, n in enumerate(lens):
            n = max(n, 0)
            x = rng.standard_normal((2, n, Hkv, D)).astype(np.float32)
            x[0] *= np.exp(0.5 * rng.standard_normal((Hkv, D))).astype(np.float32)
            held = []
            for y, full, sc in ((x[0], kk, ks), (x[1], vv, vs)):
                held.append(oa.held(y, i8) if n else np.zeros((0, Hkv, D)))
                if i8 and n:
                    q, d = oa.quantize_heads(y)
                elif n:
                    q = y.astype(np.float16)
                for j in range(need[b]):
                    m = min(P, n - j * P)
                    full[order[at + j], :m] = q[j * P:j * P + m]
                    if i8:
                        sc[order[at + j], :m] = d[j * P:j * P + m]
            table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            self.k.append(held[0])
            self.v.append(held[1])
        self.q = (q_gain * rng.standard_normal((B, T, H, D))).astype(np.float32)
        self.fmt, self.lens, self.T, self.H, self.D = fmt, list(lens), T, H, D
        self.B, self.P, self.table = B, P, table
        self.scale = float(np.float32(D ** -0.5))
        scales = (to_dev(oa.eights_in_memory(ks)), to_dev(oa.eights_in_memory(vs))) if i8 else (None, None)
        self.cache = rf.KvCache(to_dev(oa.keys_in_memory(kk)), to_dev(oa.eights_in_memory(vv)),
                                *scales, to_dev(table))

    def reference(self, window=0, rows=None):
        y, mag, tol = (np.zeros(self.q.shape) for _ in range(3))
        for b, n in enumerate(self.lens):
            for t in range(self.T):
                pos = n - self.T + t
                if rows is not None and (b, t) not in rows:
                    continue
                y[b, t], mag[b, t], big = oa.attention(self.q[b, t], self.k[b], self.v[b], pos,
                                                       self.scale, window)
                seen = max(1, min(pos + 1, window or pos + 1))
                rel = 2 * big * (4 * math.sqrt(self.D) + 16) + math.sqrt(seen) + 64
                tol[b, t] = mag[b, t] * (rel * 2.0 ** -24)[:, None]
        return y, tol

    def run(self, window=0, q=None, y=None, ws=None, lens=None, err=None, stream=None):
        y = empty(self.q.shape, torch.float32).fill_(-11.0) if y is None else y
        torch.cuda.synchronize()
        rf.rfp2_paged_attn(self.cache, to_dev(self.q) if q is None else q, self.B, self.T, self.H,
                           to_dev(np.asarray(self.lens, np.int32)) if lens is None else lens,
                           self.scale, y, window=window, err=err, workspace=ws, stream=stream)
        torch.cuda.synchronize()                             # the call may be on a stream of its own
        return y


def assert_close(got, ref, tol, what=""):
    got = got.astype(np.float64)
    assert not np.isnan(got).any(), (what, "NaN", np.argwhere(np.isnan(got))[:4])
    err = np.abs(got - ref)
    bad = ~(err <= tol + 1e-37)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4], err[bad][:4], tol[bad][:4])


CASES = [  # lens, new tokens, H, Hkv, D, P, window
    ([1], 1, 1, 1, 32, 8, 0),
    ([0], 1, 4, 2, 64, 16, 0),
    ([2, 0, 1, 33, 32, 31], 1, 8, 2, 64, 16, 0),
    ([77], 1, 8, 8, 64, 16, 0),
    ([1000], 1, 32, 8, 128, 64, 0),
    ([4097, 5], 1, 16, 2, 128, 64, 0),
    ([129, 257, 64, 63, 65, 500, 1, 300], 1, 7, 1, 96, 8, 0),
    ([700, 90], 1, 16, 1, 256, 32, 0),
    ([515], 1, 40, 2, 192, 256, 0),                          # 20 query heads to a key head
    ([260, 31], 1, 33, 1, 32, 128, 0),                       # 33 of them
    ([3, 900, 0, 2, 128], 5, 8, 2, 128, 64, 0),              # new tokens before the start
    ([400, 8, 7], 8, 64, 8, 128, 16, 0),
    ([333], 8, 48, 2, 64, 32, 0),                            # 192 rows to a key head
    ([600, 40, 1], 1, 8, 1, 256, 16, 100),
    ([600, 40, 1, 0], 4, 6, 3, 160, 16, 33),
    ([1000, 64], 2, 4, 4, 224, 64, 1),                       # sees itself only
    ([3000], 1, 4, 1, 128, 4096, 5000),                      # a window wider than the sequence
]


@pytest.mark.parametrize("fmt", [F16, I8])
@pytest.mark.parametrize("lens,T,H,Hkv,D,P,window", CASES)
def test_attention(fmt, lens, T, H, Hkv, D, P, window):
    announce("paged_attn", fmt, lens, T, H, Hkv, D, P, window)
    s = Setup(fmt, lens, T, H, Hkv, D, P, seed=len(lens) * D + T)
    err = torch.zeros(1, dtype=torch.int32, device=device())
    y = s.run(window, err=err)
    assert int(host(err)[0]) == 0
    assert_close(host(y), *s.reference(window))
    assert torch.equal(s.run(window), y)                     # the same bits again


@pytest.mark.parametrize("fmt", [F16, I8])
def test_long_sequence(fmt):
    """Split over the length and joined; two heads of the oracle's."""
    announce("paged_attn long", fmt)
    s = Setup(fmt, [20011], 1, 4, 2, 64, 32, seed=5)
    assert_close(host(s.run()), *s.reference())


@pytest.mark.parametrize("fmt", [F16, I8])
def test_many_sequences(fmt):
    """More (sequence, head) pairs than workgroups, one token to a few pages each."""
    announce("paged_attn many", fmt)
    rng = np.random.default_rng(9)
    lens = rng.integers(0, 90, 700).tolist()
    s = Setup(fmt, lens, 1, 4, 4, 32, 16, seed=6)
    assert_close(host(s.run()), *s.reference())


@pytest.mark.parametrize("fmt", [F16, I8])
@pytest.mark.parametrize("gain", [0.0, 1e-6, 30.0, 3e4])
def test_flat_and_peaked_weights(fmt, gain):
    """Scores from nothing to thousands: the running maximum jumps, most weights vanish."""
    announce("paged_attn gain", fmt, gain)
    s = Setup(fmt, [900, 65], 1, 8, 2, 64, 16, seed=7, q_gain=gain)
    assert_close(host(s.run()), *s.reference())


def test_rising_scores_and_uneven_value_scales():
    """Every token scores higher than the one before, values differ by 2^40 between
    tokens and blocks: sums are rescaled all along."""
    announce("paged_attn rising")
    n, D = 600, 64
    s = Setup(I8, [n], 1, 2, 1, D, 16, seed=8)
    rng = np.random.default_rng(8)
    k = np.zeros((n, 1, D), np.float32)
    k[:, 0, :] = (np.arange(n) / 50.0)[:, None] * np.sign(s.q[0, 0, 0])[None, :]
    v = (rng.standard_normal((n, 1, D)) * np.exp2(rng.integers(-20, 20, (n, 1, 2))).repeat(32, -1)).astype(np.float32)
    seq, pos = to_dev(np.zeros(n, np.int32)), to_dev(np.arange(n, dtype=np.int32))
    s.table[0] = np.arange(s.table.shape[1])
    s.cache.page_table.copy_(to_dev(s.table))
    rf.rfp2_kv_write(s.cache, to_dev(k), to_dev(v), n, seq, pos)
    s.k, s.v = [oa.held(k, True)], [oa.held(v, True)]
    assert_close(host(s.run()), *s.reference())


def test_half_subnormals_and_large_values():
    announce("paged_attn subnormals")
    n, D = 100, 32
    s = Setup(F16, [n], 1, 2, 1, D, 16, seed=10)
    rng = np.random.default_rng(10)
    v = rng.standard_normal((n, 1, D)).astype(np.float32)
    v[..., :16] *= 2e-6                                       # below half's normal range
    v[..., 16:] *= 1e4
    k = (3e-6 * rng.standard_normal((n, 1, D))).astype(np.float32)
    s.q = (1e6 * rng.standard_normal(s.q.shape)).astype(np.float32)
    seq, pos = to_dev(np.zeros(n, np.int32)), to_dev(np.arange(n, dtype=np.int32))
    s.table[0] = np.arange(s.table.shape[1])
    s.cache.page_table.copy_(to_dev(s.table))
    rf.rfp2_kv_write(s.cache, to_dev(k), to_dev(v), n, seq, pos)
    s.k, s.v = [oa.held(k, False)], [oa.held(v, False)]
    assert_close(host(s.run()), *s.reference())


@pytest.mark.parametrize("fmt", [F16, I8])
def test_non_finite_inputs_stay_in_their_rows(fmt):
    announce("paged_attn non-finite", fmt)
    s = Setup(fmt, [200, 90], 1, 8, 2, 64, 16, seed=11)
    ref, tol = s.reference()
    s.q[0, 0, 5, 3] = np.nan
    s.q[1, 0, 2, 0] = np.inf
    got = host(s.run())
    bad = np.zeros(got.shape, bool)
    bad[0, 0, 5] = bad[1, 0, 2] = True
    assert np.isnan(got[bad]).all()
    assert_close(got[~bad], ref[~bad], tol[~bad])
    # a NaN held in a visible value, and in a visible key
    s = Setup(fmt, [200, 90], 1, 8, 2, 64, 16, seed=11)
    x = np.zeros((2, 2, 64), np.float32)
    x[0, 0, 1] = np.nan                                       # head 0 of the token's keys
    x[1, 1, 40] = np.nan                                      # head 1 of the token's values
    rf.rfp2_kv_write(s.cache, to_dev(x[0:1]), to_dev(x[1:2]), 1, to_dev(np.array([0], np.int32)),
                     to_dev(np.array([150], np.int32)))
    got = host(s.run())
    assert np.isnan(got[0, 0, :4]).all()
    w = np.isnan(got[0, 0, 4:])
    assert (w[:, 32:].all() and not w[:, :32].any()) if fmt == I8 else \
        (w[:, 40].all() and w.sum() == 4)
    assert_close(got[1], ref[1], tol[1])


@pytest.mark.parametrize("fmt", [F16, I8])
@pytest.mark.parametrize("D", [64, 96])
def test_hidden_non_finite_values_stay_hidden(fmt, D):
    """NaN and infinities in values that some rows do not see: a later new token's, and a
    token's that has left the window.  Rows that do see them get them."""
    announce("paged_attn hidden non-finite", fmt, D)
    s = Setup(fmt, [150, 200], 4, 4, 2, D, 16, seed=16)
    window = 30
    ref, tol = s.reference(window)
    kinds = [np.nan, np.inf, -np.inf]
    for at, first_blind, kind in ((147, 0, 0), (116, 1, 1), (148, 0, 2)):
        v = np.ones((1, 2, D), np.float32)
        v[0, :, 5] = kinds[kind]                              # value 5 of both heads
        k = s.k[0][at:at + 1].astype(np.float32)
        one = to_dev(np.array([at], np.int32))
        rf.rfp2_kv_write(s.cache, to_dev(k), to_dev(v), 1, to_dev(np.zeros(1, np.int32)), one)
        got = host(s.run(window))
        for t in range(4):
            pos = 146 + t
            sees = pos - window < at <= pos
            lost = slice(0, 32) if fmt == I8 else slice(5, 6)  # int8: the block's scale is NaN
            if sees:
                assert not np.isfinite(got[0, t, :, lost]).any(), (at, t)
                if fmt == F16 and kind:
                    assert (got[0, t, :, 5] == kinds[kind]).all(), (at, t)
            else:
                assert np.isfinite(got[0, t]).all(), (at, t)
        # the other sequence, and the values of the first that nothing touched, hold
        assert_close(got[1], ref[1], tol[1], at)
        clean = np.ones((1, 2, D), np.float32)
        rf.rfp2_kv_write(s.cache, to_dev(k), to_dev(clean), 1, to_dev(np.zeros(1, np.int32)), one)


@pytest.mark.parametrize("fmt", [F16, I8])
def test_bad_lengths_and_pages(fmt):
    announce("paged_attn bad pages", fmt)
    s = Setup(fmt, [100, 100, 100, 100], 1, 4, 2, 64, 16, seed=12)
    ref, tol = s.reference()
    table = s.table.copy()
    table[1, 3] = -1                                          # a visible page that is none
    table[2, 2] = 1 << 30
    s.cache.page_table.copy_(to_dev(table))
    err = torch.zeros(1, dtype=torch.int32, device=device())
    lens = to_dev(np.array([100, 100, 100, 16 * table.shape[1] + 1], np.int32))
    got = host(s.run(lens=lens, err=err))
    assert int(host(err)[0]) == 1
    assert np.isnan(got[1:]).all()
    assert_close(got[0], ref[0], tol[0])
    assert np.isnan(host(s.run(lens=lens))[1:]).all()         # without err: as loud
    # a page out of the window's sight does not matter; a negative length is empty
    err.zero_()
    lens = to_dev(np.array([100, 100, 100, -3], np.int32))
    got = host(s.run(window=40, lens=lens, err=err))
    ref, tol = s.reference(40)
    assert int(host(err)[0]) == 1 and np.isnan(got[1]).all() and not got[3].any()
    assert_close(got[[0, 2]], ref[[0, 2]], tol[[0, 2]])


@pytest.mark.parametrize("fmt", [F16, I8])
def test_rows_apart_streams_and_shared_workspace(fmt):
    announce("paged_attn strides", fmt)
    s = Setup(fmt, [300, 45, 0], 2, 8, 2, 64, 16, seed=13)
    ref, tol = s.reference()
    wide = torch.full((3, 2, 8 * 64 + 24), np.nan, device=device())
    wide[..., :512] = to_dev(s.q).view(3, 2, 512)
    ws = torch.empty(rf.rfp2_paged_attn_workspace_bytes(s.cache, 3, 2, 8), dtype=torch.uint8,
                     device=device()).fill_(0xFF)
    st = torch.cuda.Stream()
    y = s.run(q=wide[..., :512], ws=ws, stream=st)
    assert_close(host(y), ref, tol)
    y2 = s.run(q=wide.view(6, -1), ws=ws, stream=st)          # rows of a wider matrix
    assert torch.equal(y, y2)
    with pytest.raises(ValueError):
        s.run(stream=st)                                      # a stream of its own, no workspace
    with pytest.raises(rf.Rfp2Error):
        s.run(ws=ws[:-256])


@pytest.mark.parametrize("fmt", [F16, I8])
def test_graph_replays_follow_the_lengths(fmt):
    """Captured once; replayed with longer sequences, eager work in between."""
    announce("paged_attn graph", fmt)
    s = Setup(fmt, [700, 200], 1, 8, 2, 64, 16, seed=14)
    q, lens = to_dev(s.q), to_dev(np.array([1, 1], np.int32))
    y = empty(s.q.shape, torch.float32)
    ws = torch.empty(rf.rfp2_paged_attn_workspace_bytes(s.cache, 2, 1, 8), dtype=torch.uint8,
                     device=device())
    st = torch.cuda.Stream()
    s.run(q=q, y=y, ws=ws, lens=lens, stream=st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        rf.rfp2_paged_attn(s.cache, q, 2, 1, 8, lens, s.scale, y, workspace=ws, stream=st)
    k, v = s.k, s.v
    for n in ([1, 0], [33, 200], [700, 1], [64, 64], [699, 199]):
        lens.copy_(to_dev(np.array(n, np.int32)))
        y.fill_(-1.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        s.lens, s.k, s.v = n, [a[:m] for a, m in zip(k, n)], [a[:m] for a, m in zip(v, n)]
        assert_close(host(y), *s.reference(), what=n)
        assert torch.equal(s.run(q=q), y)


@pytest.mark.parametrize("fmt", [F16, I8])
def test_cache_beyond_32_bits(fmt):
    """More than 2^32 values in the cache, the sequence's pages at its end."""
    H, D, P, n = 8, 256, 1024, 1500
    pages = (1 << 32) // (H * D * P) + 2
    announce("paged_attn far offsets", fmt, pages)
    s = Setup(fmt, [n], 1, 8, 8, D, 16, seed=15)
    c = rf.KvCache.allocate(fmt, pages, P, H, D,
                            to_dev(np.array([[pages - 1, pages - 2]], np.int32)))
    rng = np.random.default_rng(15)
    k, v = rng.standard_normal((2, n, H, D)).astype(np.float32)
    seq, pos = to_dev(np.zeros(n, np.int32)), to_dev(np.arange(n, dtype=np.int32))
    rf.rfp2_kv_write(c, to_dev(k), to_dev(v), n, seq, pos)
    s.cache, s.k, s.v = c, [oa.held(k, fmt == I8)], [oa.held(v, fmt == I8)]
    assert_close(host(s.run()), *s.reference())
