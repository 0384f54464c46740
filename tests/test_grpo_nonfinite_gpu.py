"""GPU: decode attention with queries that hold a NaN or an infinity, with heads far apart in size and with scales of any sign:
a bad head's row is NaN and stays alone (an infinite element makes every score an infinity or a NaN, of which there is no
softmax). The policy loss with NaN where it has no part."""
import numpy as np
import pytest
import torch

from tests import _grpo as G
from tests import _parity as P
from tests.test_grpo_kv_gpu import attend, ints, one, setup
from tests.test_grpo_loss_gpu import check_policy, run_policy, tokens

pytestmark = pytest.mark.gpu

BF16 = {"nan": 0x7FC1, "-nan": 0xFFC1, "inf": 0x7F80, "-inf": 0xFF80}


@pytest.fixture(scope="module")
def nv():
    import nvfp4_quantized_rl_gb300 as m
    m.lib()
    return m


def values(c):
    return c and tuple(G.values(*x).astype(np.float64) for x in c)


def definition(q, pre, own, plens, groups, lens, scale):
    with np.errstate(invalid="ignore", over="ignore"):
        return G.attention(P.bf16_f64(q), values(pre), values(own), plens, groups, lens, scale)


def decode(nv, q, own, lens, scale):
    k, v = own
    out = nv.nvfp4_kv_decode_attention(P.dev_bf16(q), P.dev(k[0]), P.dev(k[1]), one(k[2]), P.dev(v[0]), P.dev(v[1]), one(v[2]),
                                       ints(lens), scale)
    torch.cuda.synchronize()
    return P.bf16_f64(P.host_bits(out))


def spoil(q, where, bad):
    for b, h, d in where:
        q[b, h, d] = BF16[bad]
    return q


# (sequence, head, element): in the middle of a KV head's heads, and in the last one's last element
WHERE = [(1, 1, 5), (3, 6, 127), (4, 0, 64)]


def others(shape, where):
    m = np.ones(shape, bool)
    for b, h, _ in where:
        m[b, h] = False
    return m


@pytest.mark.parametrize("bad", sorted(BF16))
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (14, 1), (7, 7)])
@pytest.mark.parametrize("parts", ["both", "prefix", "own"])
def test_heads_beside_a_bad_one_keep_their_values(nv, bad, Hq, Hkv, parts):
    q, pre, own = setup(2, 6, Hq, Hkv, 200, 150 if parts != "prefix" else 0, 111, 2.0)
    plens = [0, 0] if parts == "own" else [200, 131]
    lens = [150, 149, 1, 70, 64, 0]
    spoil(q, WHERE, bad)
    args = (q, pre, own, plens, [0, 4, 6], lens if own else None, 0.09)
    want, tol = definition(*args)
    got = P.bf16_f64(P.host_bits(attend(nv, *args)))
    m = others((6, Hq), WHERE)
    G.close(got[m], want[m], tol[m], "the other heads")


@pytest.mark.parametrize("bad", sorted(BF16))
@pytest.mark.parametrize("Hq,Hkv,B", [(8, 2, 6), (14, 1, 6), (8, 2, 160)])
def test_decode_heads_beside_a_bad_one_keep_their_values(nv, bad, Hq, Hkv, B):
    """With several spans to a sequence and (160 sequences) with one."""
    q, _, own = setup(1, B, Hq, Hkv, 1, 150, 121, 2.0)
    lens = [150, 149, 1, 70, 64, 0] + [33] * (B - 6)
    spoil(q, WHERE, bad)
    want, tol = definition(q, None, own, [], [0], lens, 0.09)
    m = others((B, Hq), WHERE)
    G.close(decode(nv, q, own, lens, 0.09)[m], want[m], tol[m], "the other heads")


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (14, 1)])
def test_heads_far_apart_in_size(nv, Hq, Hkv):
    """A head 2^40 times as large as the others of its KV head: theirs keep every digit."""
    q, pre, own = setup(2, 6, Hq, Hkv, 200, 150, 131, 2.0)
    big = P.bf16_f64(q[:, 2]) * 2.0 ** 40  # a power of two: exact in bf16
    q[:, 2] = (big.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    lens = [150, 149, 1, 70, 64, 0]
    m = others((6, Hq), [(b, 2, 0) for b in range(6)])
    for plens in ([200, 131], [0, 0]):
        args = (q, pre, own, plens, [0, 4, 6], lens, 0.09)
        want, tol = definition(*args)
        got = P.bf16_f64(P.host_bits(attend(nv, *args)))
        G.close(got[m], want[m], tol[m], "the other heads")
    want, tol = definition(q, None, own, [], [0], lens, 0.09)
    G.close(decode(nv, q, own, lens, 0.09)[m], want[m], tol[m], "the other heads of a decode step")


@pytest.mark.parametrize("bad", sorted(BF16))
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (14, 1), (7, 7)])
@pytest.mark.parametrize("parts", ["both", "prefix", "own"])
def test_a_bad_head_is_nan_where_it_attends(nv, bad, Hq, Hkv, parts):
    """And 0 where there is nothing to attend to (the last sequence of the group without a prefix)."""
    q, pre, own = setup(2, 6, Hq, Hkv, 200, 150 if parts != "prefix" else 0, 141, 2.0)
    plens = [0, 0] if parts == "own" else [200, 0]
    lens = [150, 149, 1, 70, 64, 0]
    where = WHERE[:2] + [(5, 0, 0)]
    spoil(q, where, bad)
    args = (q, pre, own, plens, [0, 4, 6], lens if own else None, 0.09)
    want, tol = definition(*args)
    got = P.bf16_f64(P.host_bits(attend(nv, *args)))
    assert np.isnan(got[1, 1]).all() and np.isnan(got[3, 6]).all() and not got[5].any()
    G.close(got, want, tol, "attention")


@pytest.mark.parametrize("bad", sorted(BF16))
@pytest.mark.parametrize("Hq,Hkv,B", [(8, 2, 6), (14, 1, 6), (8, 2, 160)])
def test_a_bad_head_of_a_decode_step_is_nan_where_it_attends(nv, bad, Hq, Hkv, B):
    q, _, own = setup(1, B, Hq, Hkv, 1, 150, 151, 2.0)
    lens = [150, 149, 1, 70, 64, 0] + [33] * (B - 6)
    where = WHERE[:2] + [(5, 0, 0)]
    spoil(q, where, bad)
    want, tol = definition(q, None, own, [], [0], lens, 0.09)
    got = decode(nv, q, own, lens, 0.09)
    assert np.isnan(got[1, 1]).all() and np.isnan(got[3, 6]).all() and not got[5].any()
    G.close(got, want, tol, "decode")


@pytest.mark.parametrize("gk", [-0.0021, 0.0, -0.0, float("nan")])
@pytest.mark.parametrize("scale", [0.09, -0.09])
def test_key_scales_of_any_sign(nv, gk, scale):
    """A negative gk turns the scores' signs, 0 makes all weights equal, and a NaN leaves nothing but NaN."""
    q, pre, own = setup(2, 6, 8, 2, 200, 150, 161, 2.0)
    pre = ((*pre[0][:2], np.float32(gk)), pre[1])
    own = ((*own[0][:2], np.float32(gk)), own[1])
    for plens, lens in (([200, 131], [150, 149, 1, 70, 0, 0]), ([0, 0], [150, 149, 1, 70, 64, 0]), ([200, 0], [0] * 6)):
        args = (q, pre, own, plens, [0, 4, 6], lens, scale)
        want, tol = definition(*args)
        got = P.bf16_f64(P.host_bits(attend(nv, *args)))
        G.close(got, want, tol, "attention")
    want, tol = definition(q, None, own, [], [0], lens, scale)
    G.close(decode(nv, q, own, lens, scale), want, tol, "decode")


@pytest.mark.parametrize("bad", sorted(BF16))
def test_a_bad_first_row_stays_out_of_the_rows_that_fill_a_tile(nv, bad):
    """The batch's first head is bad, and every tile has rows without a sequence."""
    q, pre, own = setup(3, 9, 14, 2, 300, 40, 175, 2.0)
    spoil(q, [(0, 0, 0)], bad)
    args = (q, pre, own, [300, 200, 77], [0, 1, 4, 9], [40, 0, 3, 5, 40, 1, 0, 2, 9], 0.09)
    want, tol = definition(*args)
    got = P.bf16_f64(P.host_bits(attend(nv, *args)))
    assert np.isnan(got[0, 0]).all()
    G.close(got, want, tol, "attention")


def test_policy_nan_without_a_part_in_the_loss(nv):
    """An advantage of 0 leaves r and w out of the loss, a kl_coef of 0 the reference: they show in the statistics alone."""
    old, logp, ref = tokens(60, 171)
    adv, off = np.array([0.5, 0.0, -1.0], np.float32), np.array([0, 20, 40, 60], np.int32)
    w = np.ones(60, np.float32)
    w[22], logp[25], old[31] = np.nan, np.nan, np.nan
    got = check_policy(nv, logp, old, adv, off, weights=w)
    assert np.isfinite(got["loss"][0]) and np.isnan(got["stats"][4:6]).all() and not got["dlogp"][20:40].any()
    old, logp, ref = tokens(60, 172)
    ref[7] = np.nan
    with_ref, without = (run_policy(nv, logp, old, adv, off, ref=r) for r in (ref, None))
    assert np.isnan(with_ref["stats"][2]) and np.array_equal(with_ref["loss"], without["loss"])
    assert np.array_equal(with_ref["dlogp"], without["dlogp"])


def test_policy_norm_on_the_device(nv):
    """A sum of norm 1 whose gradient is scaled by a count that only the device knows: the token mean's gradient."""
    old, logp, ref = tokens(700, 173)
    off, adv = np.array([0, 300, 700], np.int32), np.array([0.7, -1.3], np.float32)
    want = G.policy(logp, old, adv, off, ref=ref, kl=0.1)
    args = [P.dev(x) for x in (logp, old, adv, off)]
    terms = dict(logp_ref=P.dev(ref), kl_coef=0.1)
    coef = nv.policy_loss(*args, mode=nv.LOSS_SUM, norm=1.0, **terms)[2]
    count = torch.full((1,), 700.0, device="cuda")
    grad = nv.policy_loss_backward(*args, coef, 1 / count, **terms)
    G.close(grad.cpu().numpy(), want["dlogp"], want["tol"]["dlogp"], "dlogp")
