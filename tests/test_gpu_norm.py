"""GPU parity of the norms and of the experts' weighted sum against the fp64 oracle: one
rounding of fp64 arithmetic, codes and scales bit for bit those of rfp2_quantize_acts."""
import numpy as np
import pytest

import bit_gemv_amd as rf
from _gpu import announce, device, empty, host, to_dev, torch
from _layer import assert_codes, assert_rounded
from oracle import feed_forward as ff

pytestmark = pytest.mark.gpu
EPS = 1e-5


def rows_apart(x, gap, fill=np.nan):
    """x as the first columns of a wider tensor whose rest holds `fill`."""
    wide = torch.full((x.shape[0], x[0].size + gap), fill, device=device())
    wide[:, :x[0].size] = to_dev(x.reshape(x.shape[0], -1))
    return wide


# T, H, D, columns between the rows: every count of lanes a head, one to many heads
HEADS = [(1, 1, 4, 0), (1, 40, 128, 0), (3, 5, 8, 4), (7, 3, 20, 8), (33, 8, 64, 64), (5, 2, 96, 0),
         (130, 48, 128, 256), (2, 17, 256, 0), (9, 3, 260, 12), (4, 2, 516, 0), (6, 1, 1024, 0),
         (1, 300, 32, 0), (2049, 3, 64, 0), (3, 1, 1000, 4), (600, 40, 128, 1024)]


@pytest.mark.parametrize("T,H,D,gap", HEADS)
def test_heads(T, H, D, gap):
    announce("rms_norm", T, H, D, gap)
    rng = np.random.default_rng(T * 7 + D)
    x = (rng.standard_normal((T, H, D)) * np.exp(rng.standard_normal((T, H, 1)))).astype(np.float32)
    gain = (1 + 0.3 * rng.standard_normal(D)).astype(np.float32)
    ref = ff.rms_norm(x, gain, EPS)
    wide, out = rows_apart(x, gap), torch.full((T, H * D + gap), -7.0, device=device())
    rf.rfp2_rms_norm(wide, T, H, D, to_dev(gain), EPS, out)
    got = host(out)
    assert_rounded(got[:, :H * D].reshape(T, H, D), ref)
    assert (got[:, H * D:] == -7.0).all()
    keep = wide.clone()
    rf.rfp2_rms_norm(wide, T, H, D, to_dev(gain), EPS, wide)          # in place
    assert torch.equal(wide[:, :H * D], out[:, :H * D])
    assert torch.equal(torch.nan_to_num(wide[:, H * D:]), torch.nan_to_num(keep[:, H * D:]))


# rows and widths: odd counts, one value group, widths that end inside a workgroup's reach, wide ones
ROWS = [(1, 32), (9, 256), (3, 288), (5, 512), (4, 544), (1, 4096), (3, 64), (2, 96), (5, 2048), (7, 5120), (33, 1056), (2, 16384), (1, 32768),
        (3, 34816), (2, 100000), (600, 4096), (1100, 160), (513, 8192)]


def stream_inputs(T, K, seed):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((T, K)) * np.exp(rng.standard_normal(K))).astype(np.float32)
    return rng, x, (1 + 0.3 * rng.standard_normal(K)).astype(np.float32)


def codes(y):
    """q, d of rfp2_quantize_acts on fp32 GPU rows."""
    M, K = y.shape
    q, d = empty((M, K), torch.int8), empty((M, K // 32), torch.float32)
    rf.rfp2_quantize_acts(y.contiguous(), M, K, q, d)
    return q, d


@pytest.mark.parametrize("T,K", ROWS)
def test_add_norm(T, K):
    announce("add_rms_norm", T, K)
    rng, x, gain = stream_inputs(T, K, T + K)
    a = rng.standard_normal((T, K)).astype(np.float32)
    href = ff.add(x, a)
    yref = ff.rms_norm(href, gain, EPS)
    xg, ag, gg = rows_apart(x, 8), rows_apart(a, 32), to_dev(gain)
    h, y = (torch.full((T, K + 4), -7.0, device=device()) for _ in range(2))
    q, d = torch.full((T + 1, K), 99, dtype=torch.int8, device=device()), torch.full((T + 1, K // 32), -7.0, device=device())
    rf.rfp2_add_rms_norm(xg, ag, T, K, gg, EPS, h, y, q, d)
    assert np.array_equal(host(h)[:, :K], href) and (host(h)[:, K:] == -7.0).all()
    assert_rounded(host(y)[:, :K], yref)
    assert (host(y)[:, K:] == -7.0).all()
    assert_codes(host(q)[:T], host(d)[:T], yref)
    assert (host(q)[T] == 99).all() and (host(d)[T] == -7.0).all()
    q2, d2 = codes(y[:, :K])
    assert torch.equal(q[:T], q2) and torch.equal(d[:T], d2)
    # every subset of the outputs, and the stream in place, give the same bits
    for want in ("h y", "y", "q", "h q", "y q"):
        h3, y3 = torch.zeros(T, K, device=device()), torch.zeros(T, K, device=device())
        q3, d3 = torch.zeros_like(q2), torch.zeros_like(d2)
        rf.rfp2_add_rms_norm(xg, ag, T, K, gg, EPS, h3 if "h" in want else None,
                             y3 if "y" in want else None, *((q3, d3) if "q" in want else (None, None)))
        assert torch.equal(h3, h[:, :K]) if "h" in want else not h3.any()
        assert torch.equal(y3, y[:, :K]) if "y" in want else not y3.any()
        assert torch.equal(q3, q2) and torch.equal(d3, d2) if "q" in want else not q3.any() and not d3.any()
    for over in ("x", "add", "both", "swapped"):
        xs, as_ = xg.clone(), ag.clone()
        ho, yo = {"x": (xs, None), "add": (as_, None), "both": (xs, as_), "swapped": (as_, xs)}[over]
        q4, d4 = torch.empty_like(q2), torch.empty_like(d2)
        rf.rfp2_add_rms_norm(xs, as_, T, K, gg, EPS, ho, yo, q4, d4)
        assert torch.equal(ho[:, :K], h[:, :K]) and torch.equal(q4, q2) and torch.equal(d4, d2), over
        assert yo is None or torch.equal(yo[:, :K], y[:, :K])
    for over in (0, 1):                                            # y over a source, no stream
        rows = [xg.clone(), ag.clone()]
        rf.rfp2_add_rms_norm(*rows, T, K, gg, EPS, None, rows[over])
        assert torch.equal(rows[over][:, :K], y[:, :K])


@pytest.mark.parametrize("T,K", [(1, 32), (4, 4096), (3, 33024), (520, 2048)])
def test_norm_alone(T, K):
    announce("norm without an addition", T, K)
    _, x, gain = stream_inputs(T, K, 3 * T + K)
    ref = ff.rms_norm(x, gain, EPS)
    xg, q, d = to_dev(x), empty((T, K), torch.int8), empty((T, K // 32), torch.float32)
    rf.rfp2_add_rms_norm(xg, None, T, K, to_dev(gain), EPS, None, None, q, d)
    assert_codes(host(q), host(d), ref)
    rf.rfp2_add_rms_norm(xg, None, T, K, to_dev(gain), EPS, None, xg)      # in place
    assert_rounded(host(xg), ref)
    q2, d2 = codes(xg)
    assert torch.equal(q, q2) and torch.equal(d, d2)


@pytest.mark.parametrize("T,K", [(2, 4), (3, 36), (5, 1028), (1, 60000), (700, 132)])
def test_norm_of_widths_without_codes(T, K):
    announce("norm, K no multiple of 32", T, K)
    rng, x, gain = stream_inputs(T, K, 5 * T + K)
    a = rng.standard_normal((T, K)).astype(np.float32)
    h, y = empty((T, K), torch.float32), empty((T, K), torch.float32)
    rf.rfp2_add_rms_norm(to_dev(x), to_dev(a), T, K, to_dev(gain), EPS, h, y)
    assert np.array_equal(host(h), ff.add(x, a))
    assert_rounded(host(y), ff.rms_norm(ff.add(x, a), gain, EPS))
    w, r = rng.random((T, 3)).astype(np.float32), rng.standard_normal((T, 3, K)).astype(np.float32)
    rf.rfp2_moe_combine(to_dev(x), to_dev(r), to_dev(w), T, 3, K, h, to_dev(gain), EPS, y)
    ref = ff.combine(x, r, w)
    assert_rounded(host(h), ref, np.abs(x) + (np.abs(w)[..., None] * np.abs(r)).sum(1))
    assert_rounded(host(y), ff.rms_norm(host(h), gain, EPS))


COMBINE = [(1, 8, 4096), (1, 1, 32), (3, 2, 96), (5, 6, 2048), (7, 10, 5120), (2, 3, 33024), (1, 64, 160),
           (300, 4, 1024), (600, 8, 256), (520, 3, 4096), (1, 7, 16384), (9, 16, 1056)]


@pytest.mark.parametrize("T,k,K", COMBINE)
def test_combine(T, k, K):
    announce("moe_combine", T, k, K)
    rng, x, gain = stream_inputs(T, K, T + 11 * k + K)
    r = rng.standard_normal((T, k, K)).astype(np.float32)
    w = rng.random((T, k)).astype(np.float32)
    w[0, k - 1] = 0.0
    size = np.abs(x) + (w[..., None] * np.abs(r)).sum(1)
    xg, rg, wg, gg = rows_apart(x, 12), to_dev(r), to_dev(w), to_dev(gain)
    h = torch.full((T, K + 4), -7.0, device=device())
    y, q, d = empty((T, K), torch.float32), empty((T, K), torch.int8), empty((T, K // 32), torch.float32)
    rf.rfp2_moe_combine(xg, rg, wg, T, k, K, h, gg, EPS, y, q, d)
    assert_rounded(host(h)[:, :K], ff.combine(x, r, w), size)
    assert (host(h)[:, K:] == -7.0).all()
    yref = ff.rms_norm(host(h)[:, :K], gain, EPS)
    assert_rounded(host(y), yref)
    assert_codes(host(q), host(d), yref)
    q2, d2 = codes(y)
    assert torch.equal(q, q2) and torch.equal(d, d2)
    # without the norm, without h, without a stream, in place
    h3, q3, d3 = empty((T, K), torch.float32), torch.zeros_like(q), torch.zeros_like(d)
    rf.rfp2_moe_combine(xg, rg, wg, T, k, K, h3)
    assert torch.equal(h3, h[:, :K])
    rf.rfp2_moe_combine(xg, rg, wg, T, k, K, None, gg, EPS, None, q3, d3)
    assert torch.equal(q3, q) and torch.equal(d3, d)
    over = rows_apart(x, 12)
    rf.rfp2_moe_combine(over, rg, wg, T, k, K, over)
    assert torch.equal(over[:, :K], h[:, :K])
    rf.rfp2_moe_combine(None, rg, wg, T, k, K, h3)
    assert_rounded(host(h3), ff.combine(None, r, w), size)
    rf.rfp2_moe_combine(xg, rg, wg, T, k, K, xg, gg, EPS, None, q3, d3)
    assert torch.equal(xg[:, :K], h[:, :K]) and torch.equal(q3, q) and torch.equal(d3, d)
    yx = rows_apart(x, 12)
    rf.rfp2_moe_combine(yx, rg, wg, T, k, K, h3, gg, EPS, yx)
    assert torch.equal(yx[:, :K], y) and torch.equal(h3, h[:, :K])


@pytest.mark.parametrize("T,K", [(4, 4096), (600, 4096), (4, 33024)])
def test_infinities_nan_and_zeros(T, K):
    """By the formula: an infinite value makes its place NaN (infinity times 0) and the row's
    others 0, a NaN the whole row NaN; the codes of such blocks are 0 with a NaN scale.  A row
    of zeros stays zeros; values whose squares leave fp32 do not overflow."""
    announce("norm of infinities", T, K)
    rng, x, gain = stream_inputs(T, K, 9)
    x[0, 5] = np.inf
    x[1, 40] = np.nan
    x[2] = 0.0
    x[3] = 1e30 * rng.standard_normal(K).astype(np.float32)
    y, q, d = empty((T, K), torch.float32), empty((T, K), torch.int8), empty((T, K // 32), torch.float32)
    for call in ("norm", "combine"):
        if call == "norm":
            rf.rfp2_add_rms_norm(to_dev(x), None, T, K, to_dev(gain), EPS, None, y, q, d)
        else:
            rf.rfp2_moe_combine(None, to_dev(x), torch.ones(T, 1, device=device()), T, 1, K, None,
                                to_dev(gain), EPS, y, q, d)
        yh, qh, dh = host(y), host(q), host(d)
        assert np.isnan(yh[0, 5]) and not np.delete(yh[0], 5).any() and np.isnan(yh[1]).all()
        assert np.isnan(dh[0, 0]) and not dh[0, 1:].any() and np.isnan(dh[1]).all() and not qh[:2].any()
        assert not yh[2].any() and not qh[2].any() and not dh[2].any()
        assert_rounded(yh[3:], ff.rms_norm(x[3:], gain, EPS))


def test_sizes_of_the_smallest_numbers():
    """Rows of subnormal values: eps holds the root, the codes are those of the quantizer."""
    announce("norm of subnormals")
    T, K = 3, 256
    rng = np.random.default_rng(4)
    x = (rng.standard_normal((T, K)) * np.array([[1e-42], [1e-38], [1e-20]])).astype(np.float32)
    gain = np.ones(K, dtype=np.float32)
    y = empty((T, K), torch.float32)
    q, d = empty((T, K), torch.int8), empty((T, K // 32), torch.float32)
    rf.rfp2_add_rms_norm(to_dev(x), None, T, K, to_dev(gain), 1e-30, None, y, q, d)
    assert_rounded(host(y), ff.rms_norm(x, gain, 1e-30))
    q2, d2 = codes(y)
    assert torch.equal(q, q2) and torch.equal(d, d2)


def test_two_calls_in_a_row_and_another_stream():
    announce("norm on another stream")
    T, K = 64, 4096
    rng, x, gain = stream_inputs(T, K, 12)
    a, gg = to_dev(rng.standard_normal((T, K)).astype(np.float32)), to_dev(gain)
    xg = to_dev(x)
    one, two = xg.clone(), xg.clone()
    q, d = empty((T, K), torch.int8), empty((T, K // 32), torch.float32)
    for _ in range(3):
        rf.rfp2_add_rms_norm(one, a, T, K, gg, EPS, one, None, q, d)
    q2, d2 = torch.empty_like(q), torch.empty_like(d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        rf.rfp2_add_rms_norm(two, a, T, K, gg, EPS, two, None, q2, d2, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(one, two) and torch.equal(q, q2) and torch.equal(d, d2)


def test_refused_on_the_gpu():
    x, g = torch.zeros(4, 64, device=device()), torch.ones(64, device=device())
    with pytest.raises(rf.Rfp2Error):
        rf.rfp2_add_rms_norm(x, None, 4, 64, g, EPS, x, x)                    # h without an addition
    with pytest.raises(ValueError):
        rf.rfp2_add_rms_norm(x, x[:3], 4, 64, g, EPS, None, x)                # too few rows
    with pytest.raises(ValueError):
        rf.rfp2_moe_combine(x, x, x, 4, 2, 64, x)                             # too few experts' rows
    with pytest.raises(TypeError):
        rf.rfp2_rms_norm(x.half(), 4, 1, 64, g, EPS, x)
    with pytest.raises(rf.Rfp2Error):
        rf.rfp2_rms_norm(x[:1].expand(4, 64), 4, 1, 64, g, EPS, x)            # rows on top of each other


def test_tensors_of_other_shapes():
    """What holds the call's values in another shape, or more of them, is taken as before:
    weights flat, outputs longer than the call."""
    announce("norm, other shapes")
    T, k, K = 3, 2, 64
    rng, x, gain = stream_inputs(T, K, 6)
    r, w = rng.standard_normal((T, k, K)).astype(np.float32), rng.random((T, k)).astype(np.float32)
    h, h2 = empty((T, K), torch.float32), empty((T + 2, K), torch.float32)
    q, d = empty((T, K), torch.int8), empty((T, K // 32), torch.float32)
    q2, d2 = empty((T + 1, K // 4, 4), torch.int8), empty((64,), torch.float32)
    rf.rfp2_moe_combine(to_dev(x), to_dev(r), to_dev(w), T, k, K, h, to_dev(gain), EPS, None, q, d)
    rf.rfp2_moe_combine(to_dev(x).view(T, 2, K // 2), to_dev(r).view(-1), to_dev(w).view(-1), T, k, K, h2,
                        to_dev(np.concatenate([gain, gain])), EPS, None, q2, d2)
    assert torch.equal(h, h2[:T]) and torch.equal(q.view(-1), q2.view(-1)[:T * K])
    assert torch.equal(d.view(-1), d2[:T * K // 32])
    with pytest.raises(ValueError):
        rf.rfp2_moe_combine(to_dev(x), to_dev(r), to_dev(w), T, k, K, h, to_dev(gain)[:32], EPS, None, q, d)
    with pytest.raises(ValueError):
        rf.rfp2_moe_combine(to_dev(x), to_dev(r).transpose(0, 1), to_dev(w), T, k, K, h)
    with pytest.raises(TypeError):
        rf.rfp2_moe_combine(to_dev(x), to_dev(r), to_dev(w).double(), T, k, K, h)
    with pytest.raises(TypeError):
        rf.rfp2_moe_combine(to_dev(x), r, to_dev(w), T, k, K, h)
    with pytest.raises(ValueError):
        rf.rfp2_moe_combine(to_dev(x), to_dev(r), torch.from_numpy(w), T, k, K, h)
