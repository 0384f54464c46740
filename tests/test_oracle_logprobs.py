"""Pins of the oracle's token log-probs and top-k distillation (CPU only): closed forms, torch in 64 bits,
central differences of the losses, invariances of the definitions; and planted mistakes that they catch."""
import math
import os
import tempfile

import numpy as np
import pytest
import torch

import oracle
import synth
from tests import _logits as G

SRC = os.path.join(os.path.dirname(oracle.__file__), "nvfp4_oracle.cpp")


def test_uniform_row_closed_form():
    x = np.full((1, 37), 2.5, np.float32)
    logp, h, lse, ids, top = oracle.token_logprobs(x, [11], 1.5, 4)
    assert logp[0] == pytest.approx(-math.log(37), rel=1e-13) and h[0] == pytest.approx(math.log(37), rel=1e-13)
    assert lse[0] == pytest.approx(3.75 + math.log(37), rel=1e-13)
    assert ids[0].tolist() == [0, 1, 2, 3]  # equal logits: the lower column first
    assert np.allclose(top, -math.log(37), rtol=1e-13)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_matches_torch_in_float64(dtype, scale):
    M, V, k = 5, 301, 17
    x = G.make(M, V, dtype, 3)
    z = torch.from_numpy(G.values(x)) * float(np.float32(scale))
    tok = np.array([0, 300, 17, 299, 1], np.int32)
    logp, h, lse, ids, top = oracle.token_logprobs(x, tok, scale, k)
    lp = torch.log_softmax(z, 1)
    assert np.allclose(logp, lp[torch.arange(M), torch.from_numpy(tok).long()], rtol=1e-12)
    assert np.allclose(h, torch.distributions.Categorical(logits=z).entropy(), rtol=1e-12)
    assert np.allclose(lse, torch.logsumexp(z, 1), rtol=1e-12)
    order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
    assert np.array_equal(ids, order.numpy()) and np.allclose(top, lp.gather(1, order), rtol=1e-12)


def test_a_large_common_offset_changes_nothing_but_lse():
    x = np.full((1, 300), -(2.0 ** 60), np.float32)
    logp, h, lse, _, _ = oracle.token_logprobs(x, [7], 1.0)
    assert logp[0] == pytest.approx(-math.log(300), rel=1e-13) and h[0] == pytest.approx(math.log(300), rel=1e-13)
    assert lse[0] == -(2.0 ** 60)


def test_masks_padding_and_bad_rows():
    x = G.make(6, 40, "f32", 1)
    x[0, 3:] = -np.inf                       # three columns left
    x[1, :] = np.finfo(np.float32).min       # none
    x[2, 5] = np.nan
    x[3, 7] = np.inf
    x[4, 0] = -2.0 ** 100                    # masked at the bound itself
    tok = [2, 0, 0, 0, 0, -100]
    logp, h, lse, ids, top = oracle.token_logprobs(x, tok, 1.0, 5)
    ref = torch.log_softmax(torch.from_numpy(x[0, :3].astype(np.float64)), 0)
    assert logp[0] == pytest.approx(float(ref[2]), rel=1e-12)
    assert sorted(ids[0][:3].tolist()) == [0, 1, 2] and ids[0][3:].tolist() == [-1, -1]
    assert lse[1] == logp[1] == -np.inf and h[1] == 0.0 and ids[1].tolist() == [-1] * 5
    for m in (2, 3):
        assert np.isnan([logp[m], h[m], lse[m]]).all() and np.isnan(top[m]).all() and (ids[m] == -1).all()
    assert logp[4] == -np.inf and np.isfinite(h[4])
    assert logp[5] == h[5] == lse[5] == 0.0 and (ids[5] == -1).all() and (top[5] == -np.inf).all()


def test_columns_behind_V_do_not_count():
    x = G.make(3, 50, "bf16", 9)
    a = oracle.token_logprobs(x, [1, 2, 44], 1.0, 3, V=45)
    b = oracle.token_logprobs(np.ascontiguousarray(x[:, :45]), [1, 2, 44], 1.0, 3)
    assert all(np.array_equal(p, q) for p, q in zip(a, b))
    assert oracle.token_logprobs(x, [45, 0, 0], 1.0, V=45)[0][0] == 0.0  # a token behind V is ignored


def _differences(f, x, step=2.0 ** -7):
    """Central differences of a scalar function of fp32 logits; steps that fp32 holds exactly."""
    d = np.zeros(x.shape)
    for i in np.ndindex(*x.shape):
        if x[i] <= G.MASKED:
            continue
        hi, lo = x.copy(), x.copy()
        hi[i] += np.float32(step)
        lo[i] -= np.float32(step)
        d[i] = (f(hi) - f(lo)) / (float(hi[i]) - float(lo[i]))
    return d


@pytest.mark.parametrize("terms", ["logp", "entropy", "both"])
def test_logprob_gradient_against_differences(terms):
    x = np.round(G.make(3, 11, "f32", 4) * 64) / 64
    x[1, 2] = -np.inf
    tok, s = [4, 0, -1], 0.75
    dl = np.array([0.5, -1.25, 2.0], np.float32) if terms != "entropy" else None
    dh = np.array([0.25, 1.0, -3.0], np.float32) if terms != "logp" else None

    def f(v):
        logp, h, *_ = oracle.token_logprobs(v, tok, s)
        return float((logp * dl).sum() if dl is not None else 0.0) + float((h * dh).sum() if dh is not None else 0.0)
    g = oracle.token_logprobs_grad(x, tok, s, dl, dh)
    # the differences are off by step^2 / 6 times a third derivative of order |d| s^3
    assert np.allclose(g, _differences(f, x), atol=2e-4) and np.all(g[2] == 0.0) and g[1, 2] == 0.0


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("twice", [False, True])
def test_distill_gradient_against_differences(tail, twice):
    x = np.round(G.make(4, 13, "f32", 6) * 64) / 64
    ids, l = G.teacher(4, 5, 13, 7, mass=0.8)
    if twice:
        ids[:, 3] = ids[:, 1]
    ids[2, 1:] = -1
    ids[3, :] = -1
    s, dloss = 1.25, np.array([1.0, -0.5, 2.0, 3.0], np.float32)
    g = oracle.topk_distill_grad(x, ids, l, s, tail, dloss)
    d = _differences(lambda v: float((oracle.topk_distill(v, ids, l, s, tail)[0] * dloss).sum()), x)
    assert np.allclose(g, d, atol=5e-4) and np.all(g[3] == 0.0)


def test_distill_closed_forms():
    x = G.make(4, 30, "f32", 2)
    z = torch.from_numpy(x.astype(np.float64))
    lp = torch.log_softmax(z, 1)
    # a teacher that lists every column with the student's own log-probs: no divergence
    ids = np.tile(np.arange(30, dtype=np.int32), (4, 1))
    for tail in (False, True):
        loss, lse, rest = oracle.topk_distill(x, ids, lp.numpy().astype(np.float32), 1.0, tail)
        assert np.all(np.abs(loss) < 1e-6) and np.all(rest == -np.inf)
        assert np.allclose(lse, torch.logsumexp(z, 1), rtol=1e-12)
    # normalized: a shift of the teacher's values changes nothing; KL from torch
    ids, l = G.teacher(4, 6, 30, 3)
    a = oracle.topk_distill(x, ids, l, 1.0, False)[0]
    assert np.allclose(a, oracle.topk_distill(x, ids, l + np.float32(4.0), 1.0, False)[0], rtol=1e-5)
    lq = torch.log_softmax(torch.from_numpy(l.astype(np.float64)), 1)
    ref = (lq.exp() * (lq - lp.gather(1, torch.from_numpy(ids).long()))).sum(1)
    assert np.allclose(a, ref, rtol=1e-12)
    # tail: the bucket as one more class
    b, _, rest = oracle.topk_distill(x, ids, l, 1.0, True)
    t = torch.from_numpy(ids).long()
    q = torch.from_numpy(l.astype(np.float64)).exp()
    p0 = 1.0 - lp.gather(1, t).exp().sum(1)
    q0 = 1.0 - q.sum(1)
    ref = (q * (q.log() - lp.gather(1, t))).sum(1) + q0 * (q0 / p0).log()
    assert np.allclose(b, ref, rtol=1e-9)
    assert np.allclose(rest, torch.logsumexp(z.scatter(1, t, -torch.inf), 1), rtol=1e-12)


def test_distill_edges():
    x = G.make(6, 9, "f32", 8)
    ids, l = G.teacher(6, 3, 9, 9)
    x[0, ids[0, 0]] = -np.inf            # a listed column masked in the student
    ids[1, :] = [-1, 9, -7]              # no entry
    l[2, :] = -np.inf                    # no teacher mass
    x[3, :] = -np.inf                    # no student mass
    x[4, 0] = np.nan
    x[5, [j for j in range(9) if j not in ids[5]]] = -np.inf  # no unlisted mass
    for tail in (False, True):
        loss, lse, rest = oracle.topk_distill(x, ids, l, 1.0, tail)
        g = oracle.topk_distill_grad(x, ids, l, 1.0, tail, np.ones(6, np.float32))
        assert loss[0] == np.inf and np.isfinite(g[0]).all()
        assert loss[1] == lse[1] == 0.0 and np.all(g[1] == 0)
        if tail:
            assert loss[2] == pytest.approx(-(rest[2] - lse[2]), rel=1e-12)  # q_0 = 1
        else:
            assert loss[2] == lse[2] == 0.0 and np.all(g[2] == 0)
        assert loss[3] == np.inf and lse[3] == -np.inf and np.all(g[3] == 0)
        assert np.isnan(loss[4]) and np.isnan(g[4]).all()
        assert np.isfinite(loss[5]) and rest[5] == -np.inf and np.isfinite(g[5]).all()


def test_a_column_listed_twice_is_one_column_with_both_shares():
    x = G.make(2, 20, "f32", 5)
    once = np.array([[3, 7]] * 2, np.int32)
    twice = np.array([[3, 7, 3]] * 2, np.int32)
    l1 = np.log(np.array([[0.5, 0.2]] * 2)).astype(np.float32)
    l2 = np.log(np.array([[0.3, 0.2, 0.2]] * 2)).astype(np.float32)
    for tail in (False, True):
        g1 = oracle.topk_distill_grad(x, once, l1, 1.0, tail, np.ones(2, np.float32))
        g2 = oracle.topk_distill_grad(x, twice, l2, 1.0, tail, np.ones(2, np.float32))
        assert np.allclose(g1, g2, atol=1e-7)
        assert np.array_equal(oracle.topk_distill(x, once, l1, 1.0, tail)[2], oracle.topk_distill(x, twice, l2, 1.0, tail)[2])


MUTANTS = {
    "scale_dropped": ("-INFINITY : scale * v;", "-INFINITY : v;"),
    "mask_missed": ("r.z[j] = v <= -bound ?", "r.z[j] = false ?"),
    "entropy_sign": ("h -= std::exp(log_p(r, j))", "h += std::exp(log_p(r, j))"),
    "tie_to_the_higher": ("if (best < 0 || v > load_elem(x, dtype, m * ld + best)) best = j;",
                          "if (best < 0 || v >= load_elem(x, dtype, m * ld + best)) best = j;"),
    "entropy_gradient_without_H": ("(dl + dh * (lp + h))", "(dl + dh * lp)"),
    "token_gradient_dropped": ("if (dlogp && j == tokens[m]) d[j] += dl;", ""),
    "gradient_scale_dropped": ("      d[j] *= scale;\n", ""),
    "tail_mass_kept_listed": ("if (!in[j]) s += std::exp(r.z[j] - top);", "s += std::exp(r.z[j] - top);"),
    "bucket_dropped": ("if (tail && !(sum >= 1.0)) t.q0 = 1.0 - sum;", ""),
    "bucket_gradient_at_listed": ("(listed[j] >= 0.0 ? listed[j] : share)", "(std::max(listed[j], 0.0) + share)"),
    "duplicate_overwrites": ("listed[t.col[i]] += t.q[i];", "listed[t.col[i]] = t.q[i];"),
    "reverse_divergence": ("sum += t.q[i] * (t.lq[i] - log_p(r, t.col[i]));",
                           "sum += std::exp(log_p(r, t.col[i])) * (log_p(r, t.col[i]) - t.lq[i]);"),
}


@pytest.mark.parametrize("name", sorted(MUTANTS))
def test_mutant_is_caught(name, monkeypatch):
    text = open(SRC).read()
    old, new = MUTANTS[name]
    assert text.count(old) >= 1, f"mutation site for {name} not found"
    with tempfile.TemporaryDirectory() as tmp:
        src = os.path.join(tmp, name + ".cpp")
        with open(src, "w") as f:
            f.write(text.replace(old, new, 1))
        L = oracle.lib(oracle.build(force=True, src=src, out=os.path.join(tmp, "lib" + name + ".so")))
    for fn in ("token_logprobs", "token_logprobs_grad", "topk_distill", "topk_distill_grad"):
        real = getattr(oracle, fn)
        monkeypatch.setattr(oracle, fn, lambda *a, _r=real, **k: _r(*a, **{**k, "L": L}))
    with pytest.raises(AssertionError):
        test_uniform_row_closed_form()
        test_matches_torch_in_float64("f32", 0.7)
        test_masks_padding_and_bad_rows()
        test_logprob_gradient_against_differences("both")
        test_distill_closed_forms()
        test_distill_edges()
        test_distill_gradient_against_differences(True, True)
