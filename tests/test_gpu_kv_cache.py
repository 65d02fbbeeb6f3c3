"""GPU parity of the key/value cache: what is written, bit for bit, in the
documented memory layout, and what is read back."""
import numpy as np
import pytest

import bit_gemv_amd as rf
from _gpu import announce, device, empty, host, to_dev, torch
from oracle import attention as oa

pytestmark = pytest.mark.gpu

SENTINEL = {rf.KV_F16: -77.0, rf.KV_I8: -128}       # no code is -128


def make_cache(fmt, pages, P, H, D, table):
    c = rf.KvCache.allocate(fmt, pages, P, H, D, to_dev(np.asarray(table, np.int32)))
    for t in (c.k, c.v):
        t.fill_(SENTINEL[fmt])
    if fmt == rf.KV_I8:
        c.k_scale.fill_(-3.0)
        c.v_scale.fill_(-3.0)
    return c


def expected(fmt, pages, P, H, D, table, k, v, seq, pos):
    """The cache's memory after the writes, from the oracle's arrays of tokens."""
    i8 = fmt == rf.KV_I8
    dt = np.int8 if i8 else np.float16
    kk, vv = (np.full((pages, P, H, D), SENTINEL[fmt], dt) for _ in range(2))
    ks, vs = (np.full((pages, P, H, D // 32), -3.0, np.float32) for _ in range(2))
    table = np.asarray(table)
    for t in range(len(seq)):
        if pos[t] < 0 or not 0 <= seq[t] < len(table) or pos[t] // P >= table.shape[1]:
            continue
        page = table[seq[t], pos[t] // P]
        if not 0 <= page < pages:
            continue
        r = pos[t] % P
        for x, full, sc in ((k, kk, ks), (v, vv, vs)):
            if i8:
                q, d = oa.quantize_heads(x[t:t + 1])
                full[page, r], sc[page, r] = q[0], d[0]
            else:
                full[page, r] = x[t].astype(np.float16)
    return oa.keys_in_memory(kk), oa.eights_in_memory(vv), oa.eights_in_memory(ks), \
        oa.eights_in_memory(vs)


def same_bits(a, b):
    return np.array_equal(np.ascontiguousarray(a).view(np.uint8), np.ascontiguousarray(b).view(np.uint8))


def assert_cache(c, ref):
    k, v, ks, vs = ref
    assert same_bits(host(c.k), k) and same_bits(host(c.v), v)
    if c.format == rf.KV_I8:
        assert same_bits(host(c.k_scale), ks) and same_bits(host(c.v_scale), vs)


def tokens(T, H, D, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((2, T, H, D)).astype(np.float32)
    x[0, 0, 0, :32] = 0.0                                     # an all-zero block
    x[1, 0, 0, :32] = np.arange(32, dtype=np.float32) - 15.5  # codes that end in a half
    x[1, 0, 0, 31] = 127.0
    return x[0], x[1]


CASES = [  # T, H, D, P, first position, sequences
    (1, 1, 32, 8, 0, 1), (1, 8, 128, 64, 4095, 1), (5, 2, 96, 16, 3, 5), (48, 8, 128, 64, 11, 48),
    (77, 3, 64, 8, 5, 1), (77, 1, 256, 32, 30, 1), (200, 2, 160, 128, 0, 2), (129, 4, 224, 16, 7, 3),
    # eight tokens a workgroup: starting inside a group of the cache, ending inside one, and
    # tokens that do not lie together
    (2051, 2, 64, 16, 5, 1), (2048, 1, 256, 64, 0, 1), (2100, 3, 96, 8, 3, 3), (2049, 1, 32, 128, 127, 1),
    (600, 2, 128, 64, 3, 1),
]


@pytest.mark.parametrize("fmt", [rf.KV_F16, rf.KV_I8])
@pytest.mark.parametrize("T,H,D,P,first,seqs", CASES)
def test_write_and_read_back(fmt, T, H, D, P, first, seqs):
    announce("kv_write/read", fmt, T, H, D, P, first, seqs)
    rng = np.random.default_rng(T + D)
    k, v = tokens(T, H, D, T * D)
    seq = (np.arange(T) * seqs // T).astype(np.int32)
    pos = np.concatenate([first + np.arange(n) for n in np.bincount(seq, minlength=seqs)]).astype(np.int32)
    width = int(pos.max()) // P + 1
    pages = seqs * width + 2
    table = rng.permutation(pages)[:seqs * width].reshape(seqs, width)
    order = rng.permutation(T) if seqs > 1 else np.arange(T)   # tokens in any order
    k, v, seq, pos = k[order], v[order], seq[order], pos[order]
    c = make_cache(fmt, pages, P, H, D, table)
    err = torch.zeros(1, dtype=torch.int32, device=device())
    # rows of a wider matrix: values first, then keys
    wide = to_dev(np.concatenate([v.reshape(T, -1), np.zeros((T, 4), np.float32),
                                  k.reshape(T, -1)], 1))
    sg, pg = to_dev(seq), to_dev(pos)
    rf.rfp2_kv_write(c, wide[:, H * D + 4:], wide[:, :H * D], T, sg, pg, err)
    ref = expected(fmt, pages, P, H, D, table, k, v, seq, pos)
    assert_cache(c, ref)
    out = torch.full((2, T, H * D + 4), -9.0, device=device())
    rf.rfp2_kv_read(c, T, sg, pg, out[0], out[1], err)
    got = host(out)
    assert (got[..., H * D:] == -9.0).all() and int(host(err)[0]) == 0
    for g, x in ((got[0], k), (got[1], v)):
        # one product code * scale, rounded once
        held = oa.held(x, fmt == rf.KV_I8)
        assert np.array_equal(g[:, :H * D].reshape(T, H, D), held.astype(np.float32))


@pytest.mark.parametrize("fmt", [rf.KV_F16, rf.KV_I8])
@pytest.mark.parametrize("T", [37, 2057])
@pytest.mark.parametrize("rot,inter", [(64, False), (64, True), (38, False), (38, True), (2, True), (62, False)])
def test_fused_equals_the_separate_calls(fmt, rot, inter, T):
    announce("rope_kv_write", fmt, rot, inter, T)
    Hq, H, D, P = 6, 2, 64, 16
    pages = -(-(T + 5) // P) + 4
    rng = np.random.default_rng(rot)
    qkv = to_dev(rng.standard_normal((T, (Hq + 2 * H) * D)).astype(np.float32))
    q, k, v = qkv.split([Hq * D, H * D, H * D], 1)
    table = rng.permutation(pages)[:pages - 4].reshape(1, -1)
    seq, pos = np.zeros(T, np.int32), (5 + np.arange(T)).astype(np.int32)
    seq[3] = 1                      # outside the cache: not stored, q rotated all the same
    pos[4] = -2                     # padding
    sg, pg = to_dev(seq), to_dev(pos)
    f = to_dev(oa.rope_freqs(rot, 10000.0))
    style = rf.ROPE_INTERLEAVED if inter else rf.ROPE_HALF
    a, b, e = (make_cache(fmt, pages, P, H, D, table) for _ in range(3))
    e1, e2 = (torch.zeros(1, dtype=torch.int32, device=device()) for _ in range(2))
    q1, q2, k2 = empty((T, Hq * D), torch.float32), empty((T, Hq, D), torch.float32), empty((T, H * D), torch.float32)
    rf.rfp2_rope_kv_write(a, q, k, v, T, Hq, sg, pg, f, rot, style, 1.1, q1, e1)
    rf.rfp2_rope(q, T, Hq, D, pg, f, rot, style, 1.1, q2)
    rf.rfp2_rope(k, T, H, D, pg, f, rot, style, 1.1, k2)
    rf.rfp2_kv_write(b, k2, v, T, sg, pg, e2)
    rf.rfp2_rope_kv_write(e, None, k, v, T, 0, sg, pg, f, rot, style, 1.1, None)
    assert torch.equal(q1.view(T, Hq, D).view(torch.int32), q2.view(torch.int32))
    for x, y, z in ((a.k, b.k, e.k), (a.v, b.v, e.v), (a.k_scale, b.k_scale, e.k_scale),
                    (a.v_scale, b.v_scale, e.v_scale)):
        if x is not None:
            assert same_bits(host(x), host(y)) and same_bits(host(x), host(z))
    assert int(host(e1)[0]) == int(host(e2)[0]) == 1
    ref = expected(fmt, pages, P, H, D, table, host(k2).reshape(T, H, D),
                   host(v.contiguous()).reshape(T, H, D), seq, pos)
    assert_cache(a, ref)


@pytest.mark.parametrize("fmt", [rf.KV_F16, rf.KV_I8])
def test_what_lies_outside_the_cache(fmt):
    announce("kv out of range", fmt)
    H, D, P = 2, 64, 8
    table = [[2, 0, 9, -1], [1, -5, 3, 1 << 30]]     # 4 pages: 9, -1, -5, 2^30 are none
    seq = np.array([0, 1, 0, 0, 1, 2, -1, 0, 1, 1, 0], np.int32)
    pos = np.array([0, 16, 17, 24, 8, 0, 0, 32, 31, 3, -1], np.int32)
    good = np.array([1, 1, 0, 0, 0, 0, 0, 0, 0, 1, 0], bool)
    T = len(seq)
    k, v = tokens(T, H, D, 1)
    c = make_cache(fmt, 4, P, H, D, table)
    sg, pg = to_dev(seq), to_dev(pos)
    kg, vg = to_dev(k), to_dev(v)
    rf.rfp2_kv_write(c, kg, vg, T, sg, pg)           # without err: still refused, silently
    assert_cache(c, expected(fmt, 4, P, H, D, table, k, v, seq, pos))
    err = torch.zeros(1, dtype=torch.int32, device=device())
    ko, vo = empty((T, H, D), torch.float32), empty((T, H, D), torch.float32)
    rf.rfp2_kv_read(c, T, sg, pg, ko, vo, err)
    assert int(host(err)[0]) == 1
    err.zero_()
    rf.rfp2_kv_write(c, kg, vg, T, sg, pg, err)
    assert int(host(err)[0]) == 1
    for x, o in ((k, host(ko)), (v, host(vo))):
        assert np.array_equal(o[good], oa.held(x[good], fmt == rf.KV_I8).astype(np.float32))
        assert np.isnan(o[~good & (pos >= 0)]).all() and (o[pos < 0] == 0).all()


def test_blocks_with_infinities_are_loud():
    announce("kv non-finite")
    c8, c16 = (make_cache(f, 1, 8, 1, 64, [[0]]) for f in (rf.KV_I8, rf.KV_F16))
    x = np.ones((1, 1, 64), np.float32)
    x[0, 0, 5], x[0, 0, 40] = np.nan, 1e6
    z = to_dev(np.zeros(1, np.int32))
    for c in (c8, c16):
        ko, vo = empty((1, 1, 64), torch.float32), empty((1, 1, 64), torch.float32)
        rf.rfp2_kv_write(c, to_dev(x), to_dev(x), 1, z, z)
        rf.rfp2_kv_read(c, 1, z, z, ko, vo)
        for o in (host(ko)[0, 0], host(vo)[0, 0]):
            if c is c8:
                assert np.isnan(o[:32]).all() and o[40] == np.float32(np.float32(1e6 / 127) * np.float32(127))
            else:
                assert np.isnan(o[5]) and np.isposinf(o[40]) and o[0] == 1.0


@pytest.mark.parametrize("fmt", [rf.KV_F16, rf.KV_I8])
def test_offsets_beyond_32_bits(fmt):
    """A cache of more than 2^32 values: the last pages, and page 0 untouched."""
    H, D, P = 8, 256, 1024
    pages = (1 << 32) // (H * D * P) + 2
    announce("kv far offsets", fmt, pages)
    table = [[pages - 1, 1, pages - 2]]
    c = rf.KvCache.allocate(fmt, pages, P, H, D, to_dev(np.asarray(table, np.int32)))
    pos = np.array([P - 1, P, 3 * P - 1], np.int32)
    k, v = tokens(3, H, D, 3)
    sg, pg = to_dev(np.zeros(3, np.int32)), to_dev(pos)
    rf.rfp2_kv_write(c, to_dev(k), to_dev(v), 3, sg, pg)
    ko, vo = empty((3, H, D), torch.float32), empty((3, H, D), torch.float32)
    rf.rfp2_kv_read(c, 3, sg, pg, ko, vo)
    for x, o in ((k, host(ko)), (v, host(vo))):
        assert np.array_equal(o, oa.held(x, fmt == rf.KV_I8).astype(np.float32))
    assert int((c.k[0] != 0).sum()) == 0 and int((c.v[0] != 0).sum()) == 0
