"""GPU: the policy and preference losses and their gradients against 64-bit definitions and differences."""
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


def dev(a):
    return None if a is None else P.dev(a)


def tokens(n, seed, spread=0.2):
    r = synth.rng(seed, n)
    old = np.log(np.maximum(1e-6, r.random(n))).astype(np.float32)
    return old, (old + spread * r.standard_normal(n)).astype(np.float32), (old + spread * r.standard_normal(n)).astype(np.float32)


def run_policy(nv, logp, old, adv, offsets, ref=None, weights=None, mask=None, low=0.2, high=0.2, dual=0.0, kl=0.0,
               mode=0, norm=1.0, per_token=False, dloss=None):
    m = None if mask is None else P.dev(mask)
    terms = dict(logp_ref=dev(ref), weights=dev(weights), mask=m, eps_low=low, eps_high=high, dual_clip=dual, kl_coef=kl,
                 adv_per_token=per_token)
    lp, lo, ad, of = dev(logp), dev(old), dev(adv), dev(offsets)
    loss, stats, coef = nv.policy_loss(lp, lo, ad, of, mode=mode, norm=norm, **terms)
    dl = None if dloss is None else torch.tensor([dloss], device="cuda")
    grad = nv.policy_loss_backward(lp, lo, ad, of, coef, dl, **terms)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in dict(loss=loss, stats=stats, coef=coef, dlogp=grad).items()}


def check_policy(nv, logp, old, adv, offsets, dloss=None, **kw):
    got = run_policy(nv, logp, old, adv, offsets, dloss=dloss, **kw)
    want = G.policy(logp, old, adv, offsets, dloss=1.0 if dloss is None else G.f32(dloss), **kw)
    for k in ("loss", "stats", "coef", "dlogp"):
        G.close(got[k], want[k], want["tol"][k], k)
    return got


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("parts,total", [(1, 1), (1, 255), (1, 256), (1, 257), (3, 700), (40, None), (513, 30000), (7, 100000)])
def test_policy_loss(nv, mode, parts, total):
    offsets = G.ragged(parts, 3, total)
    n = int(offsets[-1]) + 5  # tokens behind the last sequence
    old, logp, ref = tokens(n, 4)
    r = synth.rng(5, n)
    adv = r.standard_normal(parts).astype(np.float32)
    check_policy(nv, logp, old, adv, offsets, mode=mode, norm=777.0)
    check_policy(nv, logp, old, r.standard_normal(n).astype(np.float32), offsets, ref=ref, kl=0.04, mode=mode, norm=3.5,
                 per_token=True, dloss=-0.25)
    check_policy(nv, logp, old, adv, offsets, ref=ref, kl=0.5, weights=(0.5 + r.random(n)).astype(np.float32),
                 mask=(r.random(n) < 0.8), low=0.1, high=0.28, dual=3.0, mode=mode, norm=100.0, dloss=2.0)


def test_policy_tokens_at_the_bounds(nv):
    """Ratios at a bound and one step to either side, for each of the bounds: clipping is decided without a rounding."""
    low, high, dual = 0.2, 0.28, 3.0
    bounds = [np.log1p(-G.f32(low)), np.log1p(G.f32(high)), np.log(dual)]
    logp, old = [], []
    for t in bounds:
        for base in (-0.7, -3.3, -1e-3, 0.0, -17.25):
            b = np.float32(base)
            x = np.float32(float(b) + t)
            for y in (x, np.nextafter(x, np.float32(9)), np.nextafter(x, np.float32(-99))):
                logp.append(y)
                old.append(b)
    logp, old = np.repeat(np.array(logp, np.float32), 2), np.repeat(np.array(old, np.float32), 2)
    adv = np.tile(np.array([1.5, -0.7], np.float32), len(logp) // 2)
    offsets = np.array([0, len(logp)], np.int32)
    check_policy(nv, logp, old, adv, offsets, low=low, high=high, dual=dual, per_token=True)


def test_policy_masked_tokens_are_not_looked_at(nv):
    offsets = np.array([0, 300, 300, 700], np.int32)
    n = 710
    old, logp, ref = tokens(n, 14)
    w, adv = np.ones(n, np.float32), synth.rng(15).standard_normal(n).astype(np.float32)
    mask = synth.rng(16).random(n) < 0.7
    mask[300:310] = False
    clean = run_policy(nv, logp, old, adv, offsets, ref=ref, weights=w, mask=mask, kl=0.1, per_token=True, mode=1)
    for i, x in enumerate((logp, old, ref, w, adv)):
        x[~mask] = [np.nan, -np.inf, np.inf, np.nan, np.inf][i]
        x[700:] = np.nan
    spoiled = run_policy(nv, logp, old, adv, offsets, ref=ref, weights=w, mask=mask, kl=0.1, per_token=True, mode=1)
    for k in clean:
        assert np.array_equal(clean[k], spoiled[k]), k
    assert np.all(spoiled["dlogp"][~mask] == 0) and np.all(spoiled["dlogp"][700:] == 0)
    bytes_ = np.where(mask, 200, 0).astype(np.uint8)  # any byte but 0 counts
    assert np.array_equal(run_policy(nv, logp, old, adv, offsets, ref=ref, weights=w, mask=bytes_, kl=0.1, per_token=True,
                                     mode=1)["dlogp"], clean["dlogp"])


def test_policy_without_tokens(nv):
    e = np.zeros(0, np.float32)
    for mode in (0, 1, 2):
        got = run_policy(nv, e, e, np.ones(3, np.float32), np.zeros(4, np.int32), mode=mode)
        assert got["loss"][0] == 0 and np.all(got["stats"] == 0) and got["dlogp"].size == 0
        got = run_policy(nv, e, e, e, np.zeros(1, np.int32), mode=mode)
        assert got["loss"][0] == 0
        old, logp, _ = tokens(50, 1)
        got = run_policy(nv, logp, old, np.ones(2, np.float32), np.array([0, 20, 50], np.int32), mask=np.zeros(50, bool),
                         mode=mode)
        assert got["loss"][0] == 0 and np.all(got["stats"] == 0) and np.all(got["dlogp"] == 0)
        assert np.all(np.isfinite(got["coef"]))


def test_policy_extremes(nv):
    """Ratios that overflow or vanish, advantages of 0, infinite log-probs, NaN in a counted token."""
    old = np.array([-100, 0, -200, -1, -1, -300], np.float32)
    logp = np.array([0, -150, 0, -np.inf, -1, 0], np.float32)
    adv = np.array([1, 1, 0, -1, 0, 2], np.float32)
    off = np.array([0, 6], np.int32)
    got = run_policy(nv, logp, old, adv, off, per_token=True, mode=2, norm=1.0)
    # terms: -1.2, -e^-150 -> 0, 0, (clip at 0.8) 0.8, 0, -2.4
    G.close(got["loss"], [-1.2 + 0.8 - 2.4], 1e-6, "loss")
    G.close(got["dlogp"], [0, 0, 0, 0, 0, 0], 1e-60 + 2.0 ** -120, "dlogp")
    got = run_policy(nv, logp[:1], old[:1], np.array([-1], np.float32), np.array([0, 1], np.int32), dual=3.0)
    assert got["loss"][0] == 3.0 and got["dlogp"][0] == 0
    got = run_policy(nv, logp[:1], old[:1], np.array([-1], np.float32), np.array([0, 1], np.int32))
    assert got["loss"][0] == np.inf
    logp[4] = np.nan
    got = run_policy(nv, logp, old, np.ones(6, np.float32), off, per_token=True)
    assert np.isnan(got["loss"][0]) and np.isnan(got["dlogp"][4]) and np.all(np.isfinite(got["dlogp"][:3]))


def test_policy_ratios_over_the_whole_range(nv):
    """e^d and 1 - e^x wherever fp32 holds them, through the gradients of tokens that are not clipped."""
    d = np.concatenate([np.linspace(-95, 88.7, 30011), np.linspace(-1, 1, 20011), [-0.5, 0.5, np.nextafter(0.5, 0), 0.0]]).astype(np.float32)
    n = len(d)
    zero, off = np.zeros(n, np.float32), np.array([0, n], np.int32)
    adv = np.where(d < 0, 1, -1).astype(np.float32)
    for kw in (dict(), dict(ref=zero, kl=1.0)):
        for logp in (d, -d):
            a = adv if not kw else zero
            got = run_policy(nv, logp, zero, a if logp is d else -a, off, mode=2, norm=1.0, per_token=True, low=0.999, high=3e38, **kw)
            want = G.policy(logp, zero, a if logp is d else -a, off, mode=2, norm=1.0, per_token=True, low=0.999, high=3e38, **kw)
            # what lies beyond the largest fp32 (from d = 88.7229 on; no d here is within its tolerance of that) is infinite in fp32
            top = float(np.finfo(np.float32).max)
            exact = np.where(np.abs(want["dlogp"]) > top, np.copysign(np.inf, want["dlogp"]), want["dlogp"])
            G.close(got["dlogp"], exact, want["tol"]["dlogp"], "dlogp")


def test_policy_gradient_against_differences(nv):
    """Central differences of the 64-bit loss."""
    offsets = np.array([0, 7, 7, 20], np.int32)
    n = 20
    old, logp, ref = tokens(n, 21, 0.15)
    adv = np.array([0.7, 5.0, -1.1], np.float32)
    w = (0.5 + synth.rng(22).random(n)).astype(np.float32)
    kw = dict(ref=ref, weights=w, kl=0.3, low=0.2, high=0.28, dual=3.0, mode=1)
    got = run_policy(nv, logp, old, adv, offsets, **kw)["dlogp"]
    lp64 = logp.astype(np.float64)
    for i in range(n):
        h, l = lp64.copy(), lp64.copy()
        h[i] += 1e-6
        l[i] -= 1e-6
        d = (G.policy(h, old, adv, offsets, **kw)["loss"][0] - G.policy(l, old, adv, offsets, **kw)["loss"][0]) / 2e-6
        assert abs(got[i] - d) <= 1e-6 * (1 + abs(d)), i


@pytest.mark.parametrize("mean", [False, True])
@pytest.mark.parametrize("pairs,total", [(1, 2), (1, 600), (5, None), (33, 10007), (300, 4000), (2, 200000)])
def test_preference_loss(nv, pairs, total, mean):
    offsets = G.ragged(2 * pairs, 31, total)
    n = int(offsets[-1]) + 2
    ref, logp, _ = tokens(n, 32)
    r = synth.rng(33, n)
    mask = r.random(n) < 0.7
    dl = r.standard_normal(pairs).astype(np.float32)
    for kw in (dict(), dict(ref=ref, mask=mask, margin=0.3, smoothing=0.1), dict(ref=ref, beta=2.5), dict(mask=mask, smoothing=0.4)):
        off = dev(offsets)
        m = None if kw.get("mask") is None else P.dev(mask)
        loss, rew, coef = nv.preference_loss(dev(logp), off, dev(kw.get("ref")), m, kw.get("beta", 0.1), kw.get("margin", 0.0),
                                             kw.get("smoothing", 0.0), mean)
        for d in (dl, None):
            grad = nv.preference_loss_backward(off, coef, dev(d), n, mask=m)
            torch.cuda.synchronize()
            want = G.preference(logp, offsets, mean=mean, dloss=d, **kw)
            for k, v in dict(loss=loss, rewards=rew, coef=coef, dlogp=grad).items():
                G.close(v.cpu().numpy(), want[k], want["tol"][k], k)


def test_preference_extremes(nv):
    """Margins far to either side, empty responses, masked garbage, infinities and NaN."""
    off = np.array([0, 1, 2, 3, 4, 4, 5, 6, 7, 8, 9, 9, 9], np.int32)
    logp = np.array([0, -5000, -5000, 0, -1, 0, -np.inf, np.nan, -1], np.float32)
    loss, rew, coef = (t.cpu().numpy() for t in nv.preference_loss(dev(logp), dev(off), beta=1.0))
    assert np.array_equal(loss[:2], [0, 5000]) and abs(loss[2] - np.log1p(np.exp(-1.0))) < 1e-6
    assert loss[3] == 0 and np.isnan(loss[4]) and abs(loss[5] - np.log(2)) < 1e-6
    assert np.array_equal(coef[:4], [0, 0, -1, 1]) and rew[7] == -np.inf
    mask = np.isfinite(logp)
    m, got = P.dev(mask), nv.preference_loss(dev(logp), dev(off), mask=P.dev(mask), beta=1.0, smoothing=0.25)
    assert np.all(np.isfinite(got[0].cpu().numpy()))
    grad = nv.preference_loss_backward(dev(off), got[2], None, 9, mask=m).cpu().numpy()
    assert np.all(grad[~mask] == 0) and np.all(np.isfinite(grad))


def test_preference_gradient_against_differences(nv):
    off = np.array([0, 4, 9, 11, 16], np.int32)
    ref, logp, _ = tokens(16, 41, 0.5)
    for mean in (False, True):
        kw = dict(ref=ref, beta=0.7, margin=0.2, smoothing=0.1, mean=mean)
        coef = nv.preference_loss(dev(logp), dev(off), dev(ref), None, 0.7, 0.2, 0.1, mean)[2]
        got = nv.preference_loss_backward(dev(off), coef, None, 16).cpu().numpy()
        lp = logp.astype(np.float64)
        for i in range(16):
            h, l = lp.copy(), lp.copy()
            h[i] += 1e-6
            l[i] -= 1e-6
            d = (G.preference(h, off, **kw)["loss"].sum() - G.preference(l, off, **kw)["loss"].sum()) / 2e-6
            assert abs(got[i] - d) <= 1e-6 * (1 + abs(d)), i


def test_offsets_that_fall_do_not_fault(nv):
    n = 3000
    old, logp, ref = tokens(n, 51)
    for off in ([0, 2000, 50, 3000], [-9, 5000, 7, 8], [3000, 0, 3000, 0], [2**31 - 1, -2**31, 0, 2**31 - 1], [5000, 6000, 7000, 8000]):
        o = dev(np.array(off, np.int32))
        _, _, coef = nv.policy_loss(dev(logp), dev(old), dev(np.ones(3, np.float32)), o)
        nv.policy_loss_backward(dev(logp), dev(old), dev(np.ones(3, np.float32)), o, coef)
        o = dev(np.array(off[:3], np.int32))
        _, _, coef = nv.preference_loss(dev(logp), o)
        nv.preference_loss_backward(o, coef, None, n)
    torch.cuda.synchronize()


def test_unaligned_views_streams_and_graphs(nv):
    """Arrays that start at any element; a side stream; a captured step replayed on other contents; equal bits."""
    offsets = G.ragged(60, 61, 9000)
    n = int(offsets[-1])
    old, logp, ref = tokens(n + 3, 62)
    mask = synth.rng(63).random(n + 3) < 0.6
    big = {k: dev(v) for k, v in dict(lp=logp, lo=old, rf=ref).items()}
    bm, off, adv = P.dev(mask), dev(offsets), dev(synth.rng(64).standard_normal(60).astype(np.float32))

    def step(shift, **kw):
        lp, lo, rf = (big[k][shift:shift + n] for k in ("lp", "lo", "rf"))
        terms = dict(logp_ref=rf, mask=bm[shift:shift + n], kl_coef=0.1, dual_clip=2.0)
        loss, stats, coef = nv.policy_loss(lp, lo, adv, off, mode=nv.LOSS_SEQ_MEAN, **terms, **kw)
        g = nv.policy_loss_backward(lp, lo, adv, off, coef, **terms, **{k: v for k, v in kw.items() if k == "stream"})
        pl, rw, pc = nv.preference_loss(lp, off, rf, bm[shift:shift + n], **kw)
        return loss, stats, g, pl, nv.preference_loss_backward(off, pc, None, n, mask=bm[shift:shift + n], **kw)

    for shift in (0, 1, 3):
        got = step(shift)
        want = G.policy(logp[shift:shift + n], old[shift:shift + n], adv.cpu().numpy(), offsets, ref=ref[shift:shift + n],
                        mask=mask[shift:shift + n], kl=0.1, dual=2.0, mode=1)
        G.close(got[1].cpu().numpy(), want["stats"], want["tol"]["stats"], "stats")
        G.close(got[2].cpu().numpy(), want["dlogp"], want["tol"]["dlogp"], "dlogp")
    a = step(1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = step(1, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = step(1)
    for f in (1.0, 0.5, 0.97):
        big["lp"].mul_(f)
        adv.neg_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(c, step(1)))


def test_given_outputs_count_as_modified(nv):
    old, logp, _ = tokens(100, 71)
    off = dev(np.array([0, 60, 100], np.int32))
    ws = torch.empty(nv.workspace_bytes(nv.OP_POLICY_LOSS, 100, 2, 0), dtype=torch.uint8, device="cuda").fill_(255)
    outs = [torch.empty(k, device="cuda") for k in (1, 8, 2, 100)]
    v = [t._version for t in outs]
    got = nv.policy_loss(dev(logp), dev(old), dev(np.ones(2, np.float32)), off, loss=outs[0], stats=outs[1], coef=outs[2],
                         workspace=ws)
    g = nv.policy_loss_backward(dev(logp), dev(old), dev(np.ones(2, np.float32)), off, outs[2], out=outs[3])
    assert got[0] is outs[0] and g is outs[3] and all(t._version > w for t, w in zip(outs, v))


def test_no_weight_on_the_divergence_leaves_it_out(nv):
    """kl_coef 0 with a reference far off (e^x overflows): the gradient and the loss do not see it."""
    old = np.array([-1, -2, -300], np.float32)
    ref = np.array([-1.5, -1, 0], np.float32)
    adv, off = np.array([0.5], np.float32), np.array([0, 3], np.int32)
    a, b = (run_policy(nv, old, old, adv, off, ref=r) for r in (ref, None))
    assert a["stats"][2] == np.inf and np.array_equal(a["loss"], b["loss"]) and np.array_equal(a["dlogp"], b["dlogp"])
