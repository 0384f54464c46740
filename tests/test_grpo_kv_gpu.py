"""GPU: NVFP4 cache rows written and read raggedly, and decode attention over shared prefixes, against 64-bit definitions."""
import numpy as np
import pytest
import torch

import synth
from tests import _grpo as G
from tests import _parity as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import nvfp4_quantized_rl_gb300 as m
    m.lib()
    return m


def rows(T, Hkv, D, dtype, seed, extra=0, at=0):
    """Packed rows as the middle of longer ones: (device tensor [T, Hkv, D], host bits or fp32)."""
    x = (synth.rng(seed, T, Hkv, D).standard_normal((T, Hkv + extra, D)) * 2).astype(np.float32)
    if dtype == "bf16":
        x = synth.bf16_bits(x)
        return P.dev_bf16(x)[:, at:at + Hkv], np.ascontiguousarray(x[:, at:at + Hkv])
    return P.dev(x)[:, at:at + Hkv], np.ascontiguousarray(x[:, at:at + Hkv])


def caches(B, L, H, D, fill=0):
    return tuple(torch.full((B, L, H, D // w), fill, dtype=torch.uint8, device="cuda") for w in (2, 16, 2, 16))


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def one(v):
    return torch.tensor([v], dtype=torch.float32, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H,D,Lmax,extra", [(1, 1, 1, 16, 1, 0), (1, 37, 4, 128, 64, 28), (3, 300, 8, 128, 200, 8),
                                                (5, 999, 3, 80, 400, 0), (2, 65, 1, 64, 20, 3), (4, 50, 2, 48, 33, 1)])
def test_append_and_read_are_exact(nv, dtype, B, T, H, D, Lmax, extra):
    offsets = G.ragged(B, T, T)
    T = int(offsets[-1]) + 3  # three rows behind the last sequence
    pos = synth.rng(3, B, T).integers(0, 9, B).astype(np.int32)
    k, kh = rows(T, H, D, dtype, 1, extra, extra)
    v, vh = rows(T, H, D, dtype, 2, extra, 0)
    gk, gv = np.float32(0.003), np.float32(1e-4)
    c = caches(B, Lmax, H, D, 0x11)
    nv.nvfp4_kv_append_ragged(k, v, ints(offsets), ints(pos), one(gk), one(gv), *c)
    want = [np.full((B, Lmax, H, D // w), 0x11, np.uint8) for w in (2, 16, 2, 16)]
    enc = G.encode(kh, gk) + G.encode(vh, gv)
    where = G.packed_to_cache(offsets, pos, T, Lmax)
    for t, at in enumerate(where):
        if at is not None and at[1] is not None:
            for w, e in zip(want, enc):
                w[at] = e[t]
    for got, w in zip(c, want):
        assert np.array_equal(got.cpu().numpy(), w)
    for out in ("bf16", "f32"):
        dt = torch.bfloat16 if out == "bf16" else torch.float32
        wide = [torch.full((T, H + extra, D), 7.0, dtype=dt, device="cuda") for _ in range(2)]
        ko, vo = (x[:, extra:] for x in wide)
        nv.nvfp4_kv_read(c[0], c[1], one(gk), c[2], c[3], one(gv), ints(offsets), ints(pos), k=ko, v=vo)
        for x, y, (a, b, g) in ((wide[0], ko, (0, 1, gk)), (wide[1], vo, (2, 3, gv))):
            assert torch.all(x[:, :extra] == 7.0)
            got = P.host_bits(y.contiguous()) if out == "bf16" else y.cpu().numpy()
            dec = G.values(want[a], want[b], g, out)
            seven = 0x40E0 if out == "bf16" else 7.0
            for t, at in enumerate(where):
                expect = np.full((H, D), seven) if at is None else np.zeros((H, D)) if at[1] is None else dec[at]
                assert np.array_equal(got[t], expect.astype(got.dtype)), (t, at)
    # tensors made by the call
    k2, v2 = nv.nvfp4_kv_read(c[0], c[1], one(gk), c[2], c[3], one(gv), ints(offsets), None, T)
    assert k2.shape == (T, H, D) and v2.dtype == torch.bfloat16


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("g", [0.0, -1.0, float("nan"), 1e-30, 1e-38, 3e-42, 1.0, 1e4])
def test_append_at_scales_off_the_rows_range(nv, dtype, g):
    """Saturation, zero scales, tiny scales; subnormal and zero elements, a lone large one."""
    T, H, D = 40, 2, 64
    x = (synth.rng(5, T).standard_normal((T, H, D)) * 10.0 ** synth.rng(6, T).integers(-30, 5, (T, H, 1))).astype(np.float32)
    x[0] = 0.0
    x[1, 0, 3] = -1e-40
    x[2, 1] = 0.0
    x[2, 1, 17] = 3e4
    x[3, 0] = -0.0
    h = synth.bf16_bits(x) if dtype == "bf16" else x
    d = P.dev_bf16(h) if dtype == "bf16" else P.dev(h)
    c = caches(1, T, H, D)
    nv.nvfp4_kv_append_ragged(d, d, ints([0, T]), None, one(g), one(g), *c)
    ref = G.encode(h, np.float32(g if g > 0 else 0.0))
    for got, want in zip(c, ref + ref):
        assert np.array_equal(got.cpu().numpy()[0], want)


def test_append_matches_the_one_token_append(nv):
    B, H, D = 3, 4, 128
    k, _ = rows(B, H, D, "bf16", 8)
    v, _ = rows(B, H, D, "bf16", 9)
    pos = ints([4, 0, 6])
    a, b = caches(B, 7, H, D), caches(B, 7, H, D)
    nv.nvfp4_kv_append(k, v, pos, one(0.002), one(0.001), *a)
    nv.nvfp4_kv_append_ragged(k, v, ints([0, 1, 2, 3]), pos, one(0.002), one(0.001), *b)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


@pytest.mark.parametrize("g", [0.002, 1e-36, 50.0])
def test_append_of_infinities_and_nans_matches_the_one_token_append(nv, g):
    B, H, D = 6, 2, 64
    x = synth.rng(10).standard_normal((B, H, D)).astype(np.float32)
    for b, bad in enumerate((np.inf, -np.inf, np.nan, -np.nan, 3.3e38)):
        x[b, 1, 16 * (b % 4) + 3 * b] = bad
    x[2, 0, :20] = np.nan
    k = P.dev_bf16(synth.bf16_bits(x))
    want, pos = caches(B, 1, H, D), ints([0] * B)
    nv.nvfp4_kv_append(k, k, pos, one(g), one(g), *want)
    for rows_ in (k, k.float()):
        got = caches(B, 1, H, D)
        nv.nvfp4_kv_append_ragged(rows_, rows_, ints(range(B + 1)), None, one(g), one(g), *got)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_append_with_many_empty_sequences_and_odd_offsets(nv):
    """Offsets that fall or leave the range, and places outside the cache: no fault, and nothing outside the rows."""
    B, T, H, D = 2000, 64, 1, 32
    off = np.zeros(B + 1, np.int32)
    off[1500:] = T
    k, kh = rows(T, H, D, "bf16", 10)
    c = caches(B, 8, H, D)
    nv.nvfp4_kv_append_ragged(k, k, ints(off), None, one(0.002), one(0.002), *c)
    want = G.encode(kh, np.float32(0.002))
    assert np.array_equal(c[0][1499, :8].cpu().numpy(), want[0][:8])
    assert int(c[0][:1499].max()) == 0 and int(c[0][1500:].max()) == 0
    for off in ([0, 60, 5], [-5, 200, 64], [70, 80, 90], [64, 0, 64], [-2**31, 2**31 - 1, 0]):
        for pos in ([0, 0], [-2**31, 2**31 - 1], [-60, 7]):
            c = caches(2, 8, H, D)
            nv.nvfp4_kv_append_ragged(k, k, ints(off), ints(pos), one(0.002), one(0.002), *c)
            nv.nvfp4_kv_read(c[0], c[1], one(0.002), c[2], c[3], one(0.002), ints(off), ints(pos), T)
    torch.cuda.synchronize()


# ---- attention ------------------------------------------------------------------------------------------------


def attend(nv, q, pre, own, plens, groups, lens, scale, **kw):
    """q host bits; pre, own: (k cache, v cache) of G.cache with one g each for K and V."""
    dev = lambda c: (P.dev(c[0]), P.dev(c[1]))  # noqa: E731
    own_args = (*dev(own[0]), *dev(own[1]), ints(lens)) if own else (None,) * 5
    qd = kw.pop("qd", None)
    return nv.nvfp4_kv_prefix_attention(P.dev_bf16(q) if qd is None else qd, *dev(pre[0]), *dev(pre[1]), ints(plens),
                                        ints(groups), *own_args, one(pre[0][2]), one(pre[1][2]), scale, **kw)


def setup(P_, B, Hq, Hkv, Lp, Lmax, seed, qscale=1.0):
    pre = (G.cache(P_, Lp, Hkv, seed), G.cache(P_, Lp, Hkv, seed + 1, spread=0.5))
    own = None
    if Lmax:
        own = tuple((*G.cache(B, Lmax, Hkv, seed + 2 + i, spread=1.0 - 0.5 * i)[:2], pre[i][2]) for i in range(2))
    q = synth.bf16_bits((synth.rng(seed, 9).standard_normal((B, Hq, 128)) * qscale).astype(np.float32))
    return q, pre, own


def check(nv, q, pre, own, plens, groups, lens, scale, **kw):
    got = attend(nv, q, pre, own, plens, groups, lens, scale, **kw)
    torch.cuda.synchronize()
    vals = lambda c: c and tuple(G.values(*x).astype(np.float64) for x in c)  # noqa: E731
    want, tol = G.attention(P.bf16_f64(q), vals(pre), vals(own), plens, groups, lens, scale)
    G.close(P.bf16_f64(P.host_bits(got)), want, tol, "attention")
    return got


@pytest.mark.parametrize("Hq,Hkv", [(7, 1), (4, 4), (16, 1), (28, 4), (10, 2), (6, 6), (24, 2), (1, 1)])
@pytest.mark.parametrize("groups,Lp,Lmax", [([0, 1], 1, 1), ([0, 8], 129, 5), ([0, 3, 3, 9], 257, 70), ([2, 5, 11], 64, 0)])
def test_prefix_attention(nv, Hq, Hkv, groups, Lp, Lmax):
    """Heads of each kind; groups of one, empty ones, sequences before and behind all groups; lengths around a tile."""
    Pn, B = len(groups) - 1, groups[-1] + (2 if len(groups) > 2 else 0)
    q, pre, own = setup(Pn, B, Hq, Hkv, Lp, Lmax, 11)
    r = synth.rng(4, Hq, Lp, Lmax)
    plens = [Lp] + [int(x) for x in r.integers(0, Lp + 1, Pn - 1)]
    lens = [int(x) for x in r.integers(0, Lmax + 1, B)]
    check(nv, q, pre, own, plens, groups, lens, 1 / np.sqrt(128))


@pytest.mark.parametrize("L", [1, 15, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 640])
def test_prefix_lengths(nv, L):
    q, pre, own = setup(2, 5, 14, 2, L, 3, 20 + L)
    check(nv, q, pre, own, [L, max(0, L - 1)], [0, 3, 5], [3, 0, 1, 2, 0], 0.09)


def test_lengths_are_clamped_and_empty_rows_are_zero(nv):
    q, pre, own = setup(3, 7, 8, 2, 40, 6, 31)
    plens, lens = [0, 1000, -4], [0, 6, 99, -3, 0, 0, 2]
    got = check(nv, q, pre, own, plens, [0, 2, 4, 6], lens, 0.1)
    assert torch.all(got[0] == 0) and torch.all(got[4:6] == 0)
    got = check(nv, q, pre, None, [0, 40, 0], [0, 2, 4, 6], None, 0.1)
    assert torch.all(got[4:] == 0)


@pytest.mark.parametrize("qscale,scale", [(1e-20, 0.09), (40.0, 0.09), (1e18, 1e-19), (1.0, 0.0), (1.0, -0.3), (300.0, 0.09)])
def test_sharp_flat_and_far_scores(nv, qscale, scale):
    q, pre, own = setup(2, 6, 14, 2, 300, 40, 41, qscale)
    q[3, 2] = 0
    check(nv, q, pre, own, [300, 171], [0, 4, 6], [40, 7, 0, 22, 1, 9], scale)


def test_rising_scores(nv):
    """The running maximum grows at every tile, by more and less than a power of two's slack."""
    H, L = 1, 1500
    q = np.ones((9, 4, 128), np.float32)
    k = np.ones((1, L, H, 128), np.float32) * (np.arange(L) / 160.0)[None, :, None, None].astype(np.float32)
    v = synth.rng(1, 2).standard_normal((1, L, H, 128)).astype(np.float32)
    for steps in (k, k[:, ::-1].copy(), np.where((np.arange(L) % 256 < 3)[None, :, None, None], k, -k).astype(np.float32)):
        pre = tuple((*G.encode(synth.bf16_bits(x), g), g) for x, g in ((steps, np.float32(0.004)), (v, np.float32(0.002))))
        check(nv, synth.bf16_bits(q), pre, None, [L], [0, 9], None, 0.09)


def test_a_group_larger_than_a_tile_and_a_long_prefix(nv):
    """45 sequences of seven heads over 9000 tokens: several row tiles, many spans."""
    q, pre, own = setup(1, 45, 7, 1, 9000, 130, 51, 2.0)
    lens = [int(x) for x in synth.rng(7, 7).integers(0, 131, 45)]
    check(nv, q, pre, own, [8999], [0, 45], lens, 1 / np.sqrt(128))


def test_many_groups(nv):
    Pn = 70
    groups = np.concatenate([[0], np.cumsum(synth.rng(8, 8).integers(0, 4, Pn))]).astype(np.int32)
    B = int(groups[-1]) + 1
    q, pre, own = setup(Pn, B, 4, 2, 50, 9, 61)
    r = synth.rng(9, 9)
    check(nv, q, pre, own, r.integers(0, 51, Pn), groups, r.integers(0, 10, B), 0.1)


def test_equals_decode_attention_on_joined_caches(nv):
    """The same tokens as one cache per sequence: both within the tolerance of the same numbers."""
    q, pre, own = setup(1, 4, 28, 4, 200, 56, 71)
    lens = [56, 1, 0, 30]
    got = check(nv, q, pre, own, [200], [0, 4], lens, 0.088)
    j = [[np.concatenate([np.repeat(pre[i][c], 4, 0), own[i][c]], 1) for c in range(2)] for i in range(2)]
    for b, n in enumerate(lens):
        for i in range(2):
            for c in range(2):
                j[i][c][b, 200:200 + n] = own[i][c][b, :n]
    ref = nv.nvfp4_kv_decode_attention(P.dev_bf16(q), P.dev(j[0][0]), P.dev(j[0][1]), one(pre[0][2]), P.dev(j[1][0]),
                                       P.dev(j[1][1]), one(pre[1][2]), ints([200 + n for n in lens]), 0.088)
    assert float((got.float() - ref.float()).abs().max()) <= 0.02


def test_queries_inside_fused_rows_and_given_outputs(nv):
    q, pre, own = setup(2, 6, 8, 2, 90, 12, 81)
    wide = torch.randn(6, 12, 128, device="cuda").bfloat16()
    wide[:, 1:9] = P.dev_bf16(q)
    args = ([90, 33], [0, 4, 6], [12, 0, 3, 4, 5, 6], 0.1)
    a = check(nv, q, pre, own, *args)
    out = torch.empty(6, 8, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(nv.workspace_bytes(nv.OP_KV_PREFIX_ATTENTION, 6, 2, 12, 4, 2), dtype=torch.uint8, device="cuda").fill_(255)
    b = attend(nv, q, pre, own, *args, qd=wide[:, 1:9], out=out, workspace=ws)
    assert b is out and torch.equal(a, b)


def test_offsets_that_fall_do_not_fault(nv):
    q, pre, own = setup(2, 6, 8, 2, 90, 12, 91)
    for groups in ([6, 0, 6], [0, 9, 2], [-7, 100, 3], [5, 5, 5], [2**31 - 1, -2**31, 4]):
        attend(nv, q, pre, own, [90, 33], groups, [12, 0, 3, 4, 5, 6], 0.1)
        attend(nv, q, pre, None, [90, 33], groups, None, 0.1)
    torch.cuda.synchronize()


def test_rows_past_32_bits_of_bytes(nv):
    """The third of three caches of 4.5 million rows of 8 heads lies 4.6 GB behind the first."""
    P_, L, H, Hq, T = 3, 4_500_000, 8, 16, 300
    c = tuple(torch.empty(P_, L, H, 128 // w, dtype=torch.uint8, device="cuda") for w in (2, 16, 2, 16))
    k, kh = rows(T, H, 128, "bf16", 91)
    v, vh = rows(T, H, 128, "bf16", 92)
    gk, gv = np.float32(0.002), np.float32(0.003)
    off = ints([0, 0, 0, T])
    enc = G.encode(kh, gk) + G.encode(vh, gv)
    vals = [G.values(enc[0], enc[1], gk), G.values(enc[2], enc[3], gv)]
    for place, there in ((0, T), (L - 50, 50)):  # the second ends behind the cache
        pos = ints([0, 0, place])
        nv.nvfp4_kv_append_ragged(k, v, off, pos, one(gk), one(gv), *c)
        for got, e in zip(c, enc):
            assert np.array_equal(got[2, place:place + there].cpu().numpy(), e[:there])
        for got, want in zip(nv.nvfp4_kv_read(c[0], c[1], one(gk), c[2], c[3], one(gv), off, pos, T, torch.float32), vals):
            assert np.array_equal(got[:there].cpu().numpy(), want[:there]) and not got[there:].any()
    q = synth.bf16_bits(synth.rng(93).standard_normal((P_, Hq, 128)).astype(np.float32))
    n = [0, 0, T]
    got = nv.nvfp4_kv_prefix_attention(P.dev_bf16(q), *c, ints(n), ints([0, 1, 2, 3]), *c, ints(n), one(gk), one(gv), 0.09)
    x = [np.concatenate([np.zeros((2,) + t.shape), t[None]]).astype(np.float64) for t in vals]
    want, tol = G.attention(P.dev_bf16(q).double().cpu().numpy(), x, x, n, [0, 1, 2, 3], n,
                            G.f32(0.09))
    G.close(got.double().cpu().numpy(), want, tol, "out")


def test_equal_bits_on_streams_and_in_graphs(nv):
    """Repeated, on a side stream, captured and replayed on other contents and lengths: the bits of plain calls."""
    q, pre, own = setup(2, 20, 14, 2, 700, 100, 101)
    r = synth.rng(10, 10)
    lens = r.integers(0, 101, 20)
    dev = [P.dev(x) for c in (*pre, *own) for x in c[:2]]
    pl, gr, ln, gk, gv = ints([700, 350]), ints([0, 12, 20]), ints(lens), one(pre[0][2]), one(pre[1][2])
    qd = P.dev_bf16(q)

    def call(**kw):
        return nv.nvfp4_kv_prefix_attention(qd, dev[0], dev[1], dev[2], dev[3], pl, gr, dev[4], dev[5], dev[6], dev[7], ln,
                                            gk, gv, 0.1, **kw)
    a = call()
    assert torch.equal(a, call())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = call(stream=s)
    s.synchronize()
    assert torch.equal(a, b)
    out = torch.zeros_like(a)
    ws = torch.empty(nv.workspace_bytes(nv.OP_KV_PREFIX_ATTENTION, 20, 2, 100, 7, 2), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out=out, workspace=ws)
    for plens, scale_q in (([700, 350], 1.0), ([3, 700], 0.5), ([0, 0], 2.0), ([129, 640], 1.0)):
        pl.copy_(ints(plens))
        qd.copy_(P.dev_bf16(q) * scale_q)
        ln.copy_(ints(r.integers(0, 101, 20)))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, call())


def test_status_word_is_clean(nv):
    torch.cuda.synchronize()
    assert nv.device_status(clear=True) == (0, 0)
