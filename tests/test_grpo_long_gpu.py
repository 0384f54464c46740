"""GPU: the group-sampling operators at sizes where a warp takes several steps of tokens, a CTA several passes over its rows,
a span of an own cache several groups of tokens, and the join its second form."""
import numpy as np
import pytest
import torch

import synth
from tests import _grpo as G
from tests import _parity as P
from tests.test_grpo_kv_gpu import caches, check, ints, one, rows, setup
from tests.test_grpo_loss_gpu import check_policy, tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import nvfp4_quantized_rl_gb300 as m
    m.lib()
    return m


def packed(n, few, seed, ahead):
    """Offsets of sequences over about n tokens behind `ahead` of no sequence: a few long ones, or thousands of short, long
    and empty ones with runs of a hundred empty ones among them."""
    r = synth.rng(seed, n)
    if few:
        size = (np.array([0.45, 0.2, 0.35]) * (n - ahead)).astype(np.int64)
    else:
        size = r.choice([0, 0, 0, 1, 2, 5, 30, 400, 3000], 4 * n // 300)
        size = size[:np.searchsorted(np.cumsum(size), n - ahead)]
        for at in (0, len(size) // 3, len(size) // 2, len(size) - 100):
            size[at:at + 100] = 0
    return (ahead + np.concatenate([[0], np.cumsum(size)])).astype(np.int32)


@pytest.mark.parametrize("n", [700_001, 2_000_003])
@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("per_token", [True, False])
@pytest.mark.parametrize("with_ref", [True, False])
def test_policy_loss_of_several_steps_to_a_warp(nv, n, few, per_token, with_ref):
    offsets = packed(n, few, 201, 1000 if few else 70_001)
    old, logp, ref = tokens(n, 202)
    r = synth.rng(203, n)
    adv = r.standard_normal(n if per_token else len(offsets) - 1).astype(np.float32)
    kw = dict(ref=ref, kl=0.04) if with_ref else dict()
    check_policy(nv, logp, old, adv, offsets, per_token=per_token, mode=0 if few else 1, mask=r.random(n) < 0.8,
                 weights=(0.5 + r.random(n)).astype(np.float32), dual=3.0, dloss=-0.75, **kw)


def places(offsets, pos, T, Lmax):
    """(sequence or -1, place or -1) of every packed row."""
    t = np.arange(T)
    b = np.searchsorted(offsets, t, side="right") - 1
    b[(b < 0) | (b >= len(offsets) - 1)] = -1
    at = t - offsets[b] + pos[b]
    return b, np.where((b >= 0) & (at >= 0) & (at < Lmax), at, -1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,B,H,D,Lmax,extra", [(6007, 300, 3, 48, 60, 2), (160_001, 700, 1, 16, 500, 1), (200_003, 5, 1, 32, 70_000, 0)])
def test_append_and_read_of_many_rows(nv, dtype, T, B, H, D, Lmax, extra):
    """CTAs with more than eight rows, and with more than one pass of 256: bytes and values exact."""
    offsets = G.ragged(B, T, T - 30) + 11  # eleven rows ahead of the first sequence, some behind the last
    pos = synth.rng(204, T).integers(-5, 9, B).astype(np.int32)
    k, kh = rows(T, H, D, dtype, 205, extra, extra)
    v, vh = rows(T, H, D, dtype, 206, extra, 0)
    gk, gv = np.float32(0.003), np.float32(1e-4)
    c = caches(B, Lmax, H, D, 0x11)
    nv.nvfp4_kv_append_ragged(k, v, ints(offsets), ints(pos), one(gk), one(gv), *c)
    want = [np.full((B, Lmax, H, D // w), 0x11, np.uint8) for w in (2, 16, 2, 16)]
    b, at = places(offsets, pos, T, Lmax)
    there = at >= 0
    for w, e in zip(want, G.encode(kh, gk) + G.encode(vh, gv)):
        w[b[there], at[there]] = e[there]
    for got, w in zip(c, want):
        assert np.array_equal(got.cpu().numpy(), w)
    for out, dt, seven in (("bf16", torch.bfloat16, 0x40E0), ("f32", torch.float32, 7.0)):
        ko, vo = (torch.full((T, H + extra, D), 7.0, dtype=dt, device="cuda")[:, extra:] for _ in range(2))
        nv.nvfp4_kv_read(c[0], c[1], one(gk), c[2], c[3], one(gv), ints(offsets), ints(pos), k=ko, v=vo)
        for y, (i, j, g) in ((ko, (0, 1, gk)), (vo, (2, 3, gv))):
            got = P.host_bits(y.contiguous()) if out == "bf16" else y.cpu().numpy()
            expect = np.full((T, H, D), seven, got.dtype)
            expect[b >= 0] = 0
            expect[there] = G.values(want[i][b[there], at[there]], want[j][b[there], at[there]], g, out)
            assert np.array_equal(got, expect)


def test_attention_of_more_rows_than_the_join_holds_at_once(nv):
    """2660 (sequence, head) rows; groups of one tile and of two; sequences of no group."""
    groups = [1, 25, 25, 60, 61, 92]
    q, pre, own = setup(5, 95, 28, 4, 130, 20, 211)
    r = synth.rng(212)
    check(nv, q, pre, own, [130, 5, 129, 64, 1], groups, r.integers(0, 21, 95), 1 / np.sqrt(128))


@pytest.mark.parametrize("Hq,Hkv", [(16, 8), (32, 16), (24, 24), (48, 12)])
def test_attention_of_many_kv_heads_side_by_side(nv, Hq, Hkv):
    """Eight (or four) KV heads side by side, one set of them and several, behind prefixes of several blocks."""
    q, pre, own = setup(3, 14, Hq, Hkv, 500, 70, 221)
    check(nv, q, pre, own, [500, 129, 385], [0, 6, 7, 13], synth.rng(222).integers(0, 71, 14), 1 / np.sqrt(128))


def test_own_caches_of_many_groups_to_a_span(nv):
    """82000 tokens in 256 spans: six groups of 64 to a warp, whose maximum grows on the way; shorter ones beside. Heads for
    one and for two of the kernel's column tiles."""
    q, pre, own = setup(1, 5, 12, 1, 300, 82_000, 231, 6.0)
    for heads in (5, 12):
        check(nv, np.ascontiguousarray(q[:, :heads]), pre, own, [300], [0, 3], [82_000, 16_385, 0, 50_001, 70_000], 1 / np.sqrt(128))


@pytest.mark.parametrize("Hq,Hkv", [(28, 4), (24, 2)])
def test_decode_attention_of_joined_caches_has_the_same_numbers(nv, Hq, Hkv):
    """The same tokens as one cache per sequence: both calls within the tolerance of the definition."""
    q, pre, own = setup(1, 4, Hq, Hkv, 200, 56, 241, 2.0)
    lens = [56, 1, 0, 30]
    check(nv, q, pre, own, [200], [0, 4], lens, 0.088)
    j = [[np.concatenate([np.repeat(pre[i][c], 4, 0), own[i][c]], 1) for c in range(2)] for i in range(2)]
    joined = [200 + n for n in lens]
    out = nv.nvfp4_kv_decode_attention(P.dev_bf16(q), P.dev(j[0][0]), P.dev(j[0][1]), one(pre[0][2]), P.dev(j[1][0]),
                                       P.dev(j[1][1]), one(pre[1][2]), ints(joined), 0.088)
    vals = tuple(G.values(*j[i], pre[i][2]).astype(np.float64) for i in range(2))
    want, tol = G.attention(P.bf16_f64(q), None, vals, [], [0], joined, 0.088)
    G.close(P.bf16_f64(P.host_bits(out)), want, tol, "decode attention")
