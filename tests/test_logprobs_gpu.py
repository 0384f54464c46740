"""The logits operators on the GPU against the oracle's 64-bit definitions (tolerances derived in _logits.py)."""
import numpy as np
import pytest
import torch

import oracle
import synth
from tests import _logits as G
from tests import _parity as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    from nvfp4_quantized_rl_gb300 import _build
    _build.build()
    import nvfp4_quantized_rl_gb300 as m
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def dev(x, V=None, shift=0):
    """Logits on the GPU, `shift` elements into their storage, as a view of the first V columns."""
    t = P.dev_bf16(x) if x.dtype == np.uint16 else P.dev(x)
    if shift:
        flat = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")
        flat[shift:] = t.reshape(-1)
        t = flat[shift:].view(t.shape)
    return t[:, :V] if V else t


def f64(t):
    return None if t is None else t.cpu().double().numpy()


def check_forward(nv, x, V, tok, scale, k, dtype, shift=0, what=""):
    """One call against the oracle; returns the GPU tensors."""
    lo, h0, lse0, ids0, top0 = oracle.token_logprobs(x, tok, scale, k, V=V)
    xd = dev(x, V, shift)
    logp, h, lse, ids, top = nv.token_logprobs(xd, P.dev(np.asarray(tok, np.int32)), scale, k=k)
    torch.cuda.synchronize()
    xv = x[:, :V]
    t_lse, S, ED, zmax, ln_s = G.row_tolerances(xv, scale, np.nan_to_num(lse0, neginf=0.0), np.nan_to_num(h0))
    t_lse, S, ED, ln_s, zm = (np.nan_to_num(v, nan=0.0, posinf=0.0, neginf=0.0) for v in (t_lse, S, ED, ln_s, zmax))
    G.close(f64(lse), lse0, t_lse, f"{what} lse")
    G.close(f64(h), h0, S * (1 + 3 * ED) + 8 * G.U * (ED + ln_s), f"{what} entropy")
    with np.errstate(invalid="ignore"):
        far = np.abs(np.nan_to_num(lo + lse0 - zmax, nan=0.0, posinf=0.0, neginf=0.0))
        G.close(f64(logp), lo, S + 8 * G.U * (far + ln_s), f"{what} logp")
        if k:
            assert np.array_equal(ids.cpu().numpy(), ids0), f"{what} top ids"
            far = np.abs(np.nan_to_num(top0 + (lse0 - zmax)[:, None], nan=0.0, posinf=0.0, neginf=0.0))
            G.close(f64(top), top0, (S + 8 * G.U * ln_s)[:, None] + 8 * G.U * far, f"{what} top logp")
        else:
            assert ids is None and top is None
    return xd, logp, h, lse, ids, top


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,V,k,scale,pad,shift", [
    (1, 1, 1, 1.0, 0, 0), (1, 7, 7, 1.0, 0, 0), (3, 8, 3, 0.7, 0, 1), (5, 33, 0, 1.25, 0, 3), (2, 1000, 20, 1.0, 24, 0),
    (4, 5003, 64, 0.5, 0, 0), (3, 8192, 128, 1.0, 1, 5), (1, 20001, 256, 2.0, 0, 7), (130, 1537, 5, 1.0, 0, 0),
    (333, 257, 33, 1.0, 7, 2), (20, 16385, 1, 1.0, 0, 0), (640, 2049, 2, 0.9, 3, 0), (1300, 301, 5, 1.0, 0, 1),
    (1301, 1500, 32, 1.0, 4, 0), (1000, 77, 0, 1.0, 0, 0), (950, 3003, 96, 0.6, 0, 0)])
def test_logprobs_match_the_oracle(nv, dtype, M, V, k, scale, pad, shift):
    x = G.make(M, V, dtype, 11, ld=V + pad)
    r = synth.rng(5, M, V)
    tok = r.integers(0, V, M).astype(np.int32)
    tok[r.random(M) < 0.2] = -100
    tok[r.random(M) < 0.05] = V  # in the padding, or behind the row
    check_forward(nv, x, V, tok, scale, k, dtype, shift, f"{M}x{V} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [9, 300, 4999, 40000])
def test_masks_and_bad_rows(nv, dtype, V):
    x = G.make(9, V, dtype, 21)
    low = -3.3895313892515355e38 if dtype == "bf16" else float(np.finfo(np.float32).min)
    G.set_value(x, (0, slice(2, None)), -np.inf)        # two columns left
    G.set_value(x, (1, slice(None)), -np.inf)           # none
    G.set_value(x, (2, slice(None)), low)               # none, by the type's lowest value
    G.set_value(x, (3, V // 2), np.nan)
    G.set_value(x, (4, V - 1), np.inf)
    G.set_value(x, (5, slice(None, V - 1)), low)        # the last column alone
    G.set_value(x, (6, V // 3), 2.0 ** 101)             # too large
    G.set_value(x, (7, slice(0, V, 2)), -2.0 ** 100)    # masked at the bound
    G.set_value(x, (8, 0), np.nan)
    tok = np.array([1, 0, 3, 0, 0, V - 1, 2, 0, -1], np.int32)
    check_forward(nv, x, V, tok, 1.0, min(V, 12), dtype, what=f"masks {V} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,k,times", [(300, 256, 1), (5000, 1, 1), (5000, 256, 1), (70001, 40, 1), (70001, 256, 1),
                                       (3001, 40, 80), (3001, 1, 150), (3001, 32, 150), (12001, 20, 40)])
def test_top_alternatives_of_hard_rows(nv, dtype, V, k, times):
    """One CTA or a cluster to a row, and (`times` over) the narrower CTAs of many rows."""
    r = synth.rng(31, V, k)
    up = np.arange(V, dtype=np.float32) / V * 20 - 10
    rows = [up, up[::-1], np.zeros(V), np.where(r.random(V) < 0.5, 1.0, 0.0),  # rising, falling, constant, two values
            np.where(np.arange(V) >= V - k - 3, 5.0, -1.0),                     # all of them at the end
            np.where(np.arange(V) % 37 == 5, up, -np.inf),                      # few left
            np.where(r.random(V) < 0.5, 0.0, -0.0),                             # the two zeros are one value
            -np.abs(r.standard_normal(V)) - 2.0 ** 60,
            np.where((np.arange(V) > 4) & (np.arange(V) < V // 2), -np.inf, r.standard_normal(V))]  # a share nearly empty
    x = np.stack(rows).astype(np.float32)
    x = np.tile(_bits(x) if dtype == "bf16" else x, (times, 1))
    check_forward(nv, x, V, np.arange(9 * times, dtype=np.int32) % V, 1.0, k, dtype, what=f"hard {V} {k} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,V,k", [(3, 30000, 20), (3, 30000, 130), (700, 9000, 64), (700, 1100, 256)])
def test_top_alternatives_below_zero(nv, dtype, M, V, k):
    """Negative logits only: the list's bounds fall between values, and round away from zero."""
    r = synth.rng(33, V, k)
    x = (-np.abs(r.standard_normal((M, V))) * 4 - 3 * r.random((M, 1))).astype(np.float32)
    rows = np.arange(M) % V
    check_forward(nv, _bits(x) if dtype == "bf16" else x, V, rows.astype(np.int32), 1.0, k, dtype, what=f"{V} {k}")


def _bits(x):
    """bf16 bits of fp32 values that may be infinite."""
    b = synth.bf16_bits(np.where(np.isfinite(x), x, 0.0))
    return np.where(np.isfinite(x), b, np.ascontiguousarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def test_only_what_is_asked_for(nv):
    x = dev(G.make(4, 1000, "bf16", 3))
    tok = torch.tensor([1, 2, 3, -1], dtype=torch.int32, device="cuda")
    full = nv.token_logprobs(x, tok, k=4)
    logp, h, lse, ids, top = nv.token_logprobs(x, tok, entropy=False)
    assert h is None and ids is None and top is None and torch.equal(logp, full[0]) and torch.equal(lse, full[2])
    logp, h, lse, ids, top = nv.token_logprobs(x, k=4)  # no tokens: every row counts
    assert logp is None and torch.equal(ids[:3], full[3][:3]) and torch.equal(h[:3], full[1][:3]) and h[3] > 0
    assert nv.token_logprobs(x[:0], tok[:0], k=2)[3].shape == (0, 2)
    with pytest.raises(nv.Nvfp4rlError):
        nv.token_logprobs(x, tok, scale=-1.0)
    with pytest.raises(ValueError):
        nv.token_logprobs(x, tok.long())


def check_backward(nv, x, V, tok, scale, dtype, dl, dh, shift=0, out=None, what=""):
    xd = dev(x, V, shift)
    td = P.dev(np.asarray(tok, np.int32))
    _, h, lse, _, _ = nv.token_logprobs(xd, td, scale)
    up = lambda a: None if a is None else P.dev(a)  # noqa: E731
    out = xd if out == "inplace" else out
    got = nv.token_logprobs_backward(xd, td, lse, up(dl), scale, entropy=h if dh is not None else None,
                                     dentropy=up(dh), out=out)
    torch.cuda.synchronize()
    ref = oracle.token_logprobs_grad(x, tok, scale, dl, dh, V=V)
    _, h0, lse0, _, _ = oracle.token_logprobs(x, tok, scale, V=V)
    xv = x[:, :V]
    with np.errstate(invalid="ignore"):
        t_lse = np.nan_to_num(G.row_tolerances(xv, scale, np.nan_to_num(lse0, neginf=0.0), np.nan_to_num(h0))[0])
    h0, l0 = np.nan_to_num(h0), np.nan_to_num(lse0, neginf=0.0)
    zero = np.zeros(len(tok))
    dl_, dh_ = np.abs(dl if dl is not None else zero), np.abs(dh if dh is not None else zero)
    spike = np.zeros(ref.shape)
    for m, t in enumerate(tok):
        if 0 <= t < V:
            spike[m, t] = dl_[m]
    t = G.grad_tolerance(xv, scale, l0, h0, t_lse, dtype, np.nan_to_num(ref), dl_, dh_, spike)
    G.close(f64(got), ref, t, f"{what} dlogits")
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("terms", ["logp", "entropy", "both"])
@pytest.mark.parametrize("M,V,scale,pad,shift", [(1, 1, 1.0, 0, 0), (3, 7, 1.0, 0, 1), (5, 64, 0.7, 8, 0), (2, 5003, 1.25, 0, 3),
                                                 (70, 1025, 1.0, 5, 0), (1, 40003, 1.0, 0, 0), (300, 130, 2.0, 0, 0)])
def test_logprobs_backward_matches_the_oracle(nv, dtype, terms, M, V, scale, pad, shift):
    x = G.make(M, V, dtype, 41, ld=V + pad)
    r = synth.rng(6, M, V)
    tok = r.integers(0, V, M).astype(np.int32)
    tok[r.random(M) < 0.2] = -100
    dl = r.standard_normal(M).astype(np.float32) if terms != "entropy" else None
    dh = r.standard_normal(M).astype(np.float32) if terms != "logp" else None
    if M > 2:  # a row whose gradients are 0
        for d in (dl, dh):
            if d is not None:
                d[1] = 0.0
    check_backward(nv, x, V, tok, scale, dtype, dl, dh, shift, what=f"{M}x{V} {dtype} {terms}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient_of_masked_and_bad_rows(nv, dtype):
    V = 3001
    x = G.make(6, V, dtype, 51)
    G.set_value(x, (0, slice(2, None)), -np.inf)
    G.set_value(x, (1, slice(None)), -np.inf)
    G.set_value(x, (2, 5), np.nan)
    G.set_value(x, (3, slice(0, V, 3)), -np.inf)
    G.set_value(x, (4, slice(0, V, 3)), -2.0 ** 100)
    tok = np.array([1, 0, 3, 4, 0, 7], np.int32)  # row 4's token is masked
    one = np.ones(6, np.float32)
    check_backward(nv, x, V, tok, 1.0, dtype, one, 0.5 * one, what=f"masked {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,pad,ldd,off", [(257, 0, 257, 0), (257, 7, 257, 0), (257, 0, 300, 3), (4096, 64, 4097, 1),
                                           (9001, 3, 9001, 5), (9001, 0, 9008, 2), (5, 3, 6, 1)])
def test_gradient_places(nv, dtype, V, pad, ldd, off):
    """Rows of the logits and of the gradient that start at different alignments; what lies between rows stays."""
    M = 5
    x = G.make(M, V, dtype, 61, ld=V + pad)
    r = synth.rng(7, V, ldd)
    tok = r.integers(0, V, M).astype(np.int32)
    tok[2] = -1
    dl, dh = r.standard_normal((2, M)).astype(np.float32)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    buf = torch.full((M * ldd + off + 8,), 7.0, dtype=t, device="cuda")
    out = buf[off:off + M * ldd].view(M, ldd)[:, :V]
    got = check_backward(nv, x, V, tok, 1.0, dtype, dl, dh, out=out, what=f"places {V} {ldd} {dtype}")
    assert got.data_ptr() == out.data_ptr()
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep[off:off + M * ldd].view(M, ldd)[:, :V] = False
    assert torch.all(buf[keep] == 7.0)
    apart = check_backward(nv, x, V, tok, 1.0, dtype, dl, dh, what="apart")
    assert torch.equal(apart, out)  # the same bits wherever it lies
    inplace = check_backward(nv, x, V, tok, 1.0, dtype, dl, dh, out="inplace", what="in place")
    assert torch.equal(inplace, out)


def teacher_case(M, V, k, dtype, seed, twice=False, pad_entries=0, ld=None, mass=0.9):
    x = G.make(M, V, dtype, seed, ld=ld)
    ids, l = G.teacher(M, k, V, seed + 1, mass=mass, pad=pad_entries)
    if k > V:
        l -= np.float32(np.log(k / V))
    if twice and k > 2:
        ids[:, k // 2] = ids[:, 0]
        ids[:, k - 1] = ids[:, 0]
    return x, ids, l


def check_distill(nv, x, V, ids, l, scale, tail, dtype, dloss, shift=0, out=None, what=""):
    xd, idd, ld = dev(x, V, shift), P.dev(ids), P.dev(l)
    loss, lse, rest = nv.topk_distill(xd, idd, ld, scale, tail=tail)
    torch.cuda.synchronize()
    loss0, lse0, rest0 = oracle.topk_distill(x, ids, l, scale, tail, V=V)
    xv = x[:, :V]
    s = float(np.float32(scale))
    M, k = ids.shape
    with np.errstate(all="ignore"):
        h0 = oracle.token_logprobs(x, None, scale, V=V)[1]
        t_lse, S, ED, zmax, ln_s = (np.nan_to_num(v, nan=0.0, posinf=0.0, neginf=0.0) for v in G.row_tolerances(
            xv, scale, np.nan_to_num(lse0, neginf=0.0), np.nan_to_num(h0)))
        valid = (ids >= 0) & (ids < V)
        z = np.take_along_axis(G.values(xv) * s, np.where(valid, ids, 0), 1)
        lq = np.where(valid, l.astype(np.float64), -np.inf)
        if not tail:
            top = np.max(lq, 1, keepdims=True)
            lq = lq - top - np.log(np.exp(lq - top).sum(1, keepdims=True))
        q = np.nan_to_num(np.exp(lq))
        lp = z - lse0[:, None]
        t_lp = S[:, None] + 8 * G.U * (np.abs(np.nan_to_num(z - zmax[:, None], neginf=0.0)) + ln_s[:, None])
        # q: the exponent's rounding (l - top, ln total: 3u each) and expf, a sum of up to 256 terms, a division
        e_q = G.U * (4 * np.abs(np.nan_to_num(lq, neginf=0.0)) + 24)
        term = np.abs(np.nan_to_num(lq - lp, posinf=0.0, neginf=0.0))
        t_loss = (q * (term * (e_q + 4 * G.U) + t_lp + e_q)).sum(1) + k * G.U * (q * term).sum(1)
        if tail:
            # q_0 = -expm1(l_max) - the others: each to 16 u of its size; d(term)/dq_0 = ln(q_0 / p_0) + 1
            q0 = np.maximum(0.0, 1.0 - q.sum(1))
            qmax = q.max(1)
            d0 = (16 + k) * G.U * ((1 - qmax) + (q.sum(1) - qmax)) + 4 * G.U * qmax * np.abs(np.log(np.maximum(qmax, 1e-30)))
            lp0 = rest0 - lse0
            far = np.abs(np.nan_to_num(np.log(np.maximum(q0, 1e-30)) - lp0, posinf=0.0, neginf=0.0))
            t_tail = S + t_lse + 8 * G.U * np.abs(np.nan_to_num(lp0, neginf=0.0))
            # the unlisted sum's own terms: D relative to the row's maximum may be large where p_0 is small
            t_tail = t_tail + 3 * G.U * np.abs(np.nan_to_num(lp0, neginf=0.0))
            t_loss = t_loss + d0 * (far + 1) + q0 * (2 * t_tail + 8 * G.U * far)
            z_all = np.where(np.isfinite(G.values(xv)), G.values(xv) * s, 0.0)
            t_rest = t_lse + t_tail + 8 * G.U * (np.abs(np.nan_to_num(rest0, neginf=0.0)) + np.abs(z_all).max(1))
            G.close(f64(rest), rest0, t_rest, f"{what} lse_tail")
        else:
            assert rest is None
        G.close(f64(lse), lse0, 2 * t_lse, f"{what} lse")
        G.close(f64(loss), loss0, np.nan_to_num(t_loss) * 1.05 + 1e-12, f"{what} loss")
    out = xd if isinstance(out, str) else out
    got = nv.topk_distill_backward(xd, idd, ld, lse, P.dev(dloss), scale, tail=tail, lse_tail=rest, out=out)
    torch.cuda.synchronize()
    ref = oracle.topk_distill_grad(x, ids, l, scale, tail, dloss, V=V)
    d = np.abs(dloss.astype(np.float64))
    spike = np.zeros((M, V))
    for m in range(M):
        for i in range(k):
            if valid[m, i]:
                spike[m, ids[m, i]] += q[m, i] * d[m] * (1 + np.max(e_q[m]) / G.U / 16)
    weight = d * (1 + q.sum(1))
    tol = np.nan_to_num(2 * t_lse)
    if tail:
        # unlisted columns go by lse_tail: p (Q - q_0 / p_0) = exp(z - lse_tail) (Q p_0 - q_0)
        p0 = np.exp(np.nan_to_num(lp0, neginf=-np.inf))
        share = np.nan_to_num(np.exp(G.values(xv) * s - np.where(np.isfinite(rest0), rest0, np.inf)[:, None]))
        lift = share * (d * (np.nan_to_num(d0) * 2 + p0 * (t_rest + t_lse + 16 * G.U)
                             + np.abs(p0 - q0) * (t_rest + G.U * 64)))[:, None] * s
        lift = lift + share * (d * np.abs(p0 - q0))[:, None] * s * G.U * 3 * np.abs(z_all)
    else:
        lift = 0.0
    t = G.grad_tolerance(xv, scale, np.nan_to_num(lse0, neginf=0.0), np.zeros(M), tol, dtype, np.nan_to_num(ref), weight,
                         np.zeros(M), spike)
    G.close(f64(got), ref, t + lift, f"{what} dlogits")
    return loss, lse, rest, got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("M,V,k,scale,pad,shift,twice", [
    (1, 1, 1, 1.0, 0, 0, False), (2, 7, 7, 1.0, 0, 1, False), (3, 8, 3, 0.7, 5, 0, True), (4, 33, 40, 1.0, 0, 0, False),
    (5, 1000, 20, 1.25, 0, 3, False), (2, 5003, 64, 1.0, 0, 0, True), (130, 1537, 5, 0.5, 7, 0, False),
    (3, 20001, 256, 1.0, 0, 0, True), (20, 4097, 100, 1.0, 1, 0, False), (400, 300, 33, 1.0, 0, 0, True),
    (1000, 203, 20, 1.0, 5, 1, True), (930, 1111, 64, 0.8, 0, 0, False), (500, 700, 128, 1.0, 0, 0, True)])
def test_distill_matches_the_oracle(nv, dtype, tail, M, V, k, scale, pad, shift, twice):
    x, ids, l = teacher_case(M, V, k, dtype, 71, twice, pad_entries=min(3, k - 1), ld=V + pad)
    if M > 2:
        ids[1, :] = -1                       # no teacher
        ids[2, k // 2] = V + pad             # an entry behind the row
    dloss = synth.rng(8, M, V).standard_normal(M).astype(np.float32)
    if M > 3:
        dloss[3] = 0.0
    check_distill(nv, x, V, ids, l, scale, tail, dtype, dloss, shift, what=f"{M}x{V} k={k} tail={tail} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_edges(nv, dtype, tail):
    M, V, k = 8, 3001, 6
    x, ids, l = teacher_case(M, V, k, dtype, 81)
    G.set_value(x, (0, int(ids[0, 0])), -np.inf)     # a listed column masked in the student
    l[1, :] = -np.inf                                # no teacher mass
    l[2, 2] = -np.inf                                # an entry without mass
    G.set_value(x, (3, slice(None)), -np.inf)        # no student mass
    G.set_value(x, (4, V - 1), np.nan)
    keep = ids[5].copy()
    v = x[5, keep].copy()
    G.set_value(x, (5, slice(None)), -np.inf)        # unlisted columns all masked
    x[5, keep] = v
    G.set_value(x, (6, int(ids[6, 1])), 90.0)        # the listed ones hold nearly all of p: p_0 ~ e^-80
    l[7, :] = np.log(1.0 / k)                        # q_0 = 0 but for rounding
    dloss = np.ones(M, np.float32)
    rows = [m for m in range(M) if not (tail and m == 7)]
    check_distill(nv, x[rows], V, ids[rows], l[rows], 1.0, tail, dtype, dloss[rows], what=f"edges {tail} {dtype}")
    # 1 - sum q may round to either side of 0: the loss has to be finite, and near the one without a bucket
    loss = nv.topk_distill(dev(x[7:]), P.dev(ids[7:]), P.dev(l[7:]), tail=tail)[0]
    assert abs(float(loss) - oracle.topk_distill(x[7:], ids[7:], l[7:], 1.0, False)[0][0]) < 1e-4
    l[0, 1] = np.nan
    loss = nv.topk_distill(dev(x[:1]), P.dev(ids[:1]), P.dev(l[:1]), tail=tail)[0]
    assert torch.isnan(loss).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_distill_gradient_places(nv, dtype):
    M, V, k = 4, 2051, 30
    x, ids, l = teacher_case(M, V, k, dtype, 91, twice=True, ld=V + 5)
    dloss = np.array([1.0, -2.0, 0.5, 3.0], np.float32)
    apart = check_distill(nv, x, V, ids, l, 1.0, True, dtype, dloss, what="apart")[3]
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    buf = torch.full((M, V + 3), 7.0, dtype=t, device="cuda")
    out = buf[:, 1:V + 1]
    check_distill(nv, x, V, ids, l, 1.0, True, dtype, dloss, out=out, what="strided")
    assert torch.equal(out, apart) and torch.all(buf[:, 0] == 7.0) and torch.all(buf[:, V + 1:] == 7.0)
    inplace = check_distill(nv, x, V, ids, l, 1.0, True, dtype, dloss, out="inplace", what="in place")[3]
    assert torch.equal(inplace, apart)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_subnormal_logits(nv, dtype):
    """Values below the smallest normal one are values: they order the alternatives, and give the uniform p."""
    V = 4000
    r = synth.rng(121)
    bits = r.integers(1, 0x80 if dtype == "bf16" else 0x7FFFFF, (2, V))
    bits = np.where(r.random((2, V)) < 0.5, bits, bits | (0x8000 if dtype == "bf16" else 0x80000000))
    x = bits.astype(np.uint16) if dtype == "bf16" else bits.astype(np.uint32).view(np.float32)
    check_forward(nv, x, V, np.array([5, 6], np.int32), 1.0, 50, dtype, what=f"subnormal {dtype}")
    check_forward(nv, np.tile(x, (700, 1)), V, np.arange(1400, dtype=np.int32), 1.0, 20, dtype, what=f"subnormal {dtype}")


def test_many_tiny_rows(nv):
    """Two hundred thousand rows of five columns (router logits' kind)."""
    M, V = 200003, 5
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(M, V, generator=g, device="cuda").bfloat16()
    tok = torch.randint(-1, V, (M,), generator=g, device="cuda").int()
    logp, h, lse, ids, top = nv.token_logprobs(x, tok, k=2)
    lp = torch.log_softmax(x.double(), 1)
    live = tok >= 0
    safe = tok.long().clamp_min(0)[:, None]
    # (3 E[D] + 4 + V / 64 + 64) u + 8 u (|z| + ln 5) with |z| < 8, D < 16
    tol = 300 * G.U
    assert torch.all((logp.double() - torch.where(live, lp.gather(1, safe)[:, 0], 0.0)).abs() < tol)
    order = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :2]
    assert torch.equal(ids.long(), torch.where(live[:, None], order, -1))
    one = torch.ones(M, device="cuda")
    d = nv.token_logprobs_backward(x, tok, lse, one).double()
    ref = torch.where(live[:, None], torch.zeros_like(lp).scatter_(1, safe, 1.0) - lp.exp(), 0.0)
    assert torch.all((d - ref).abs() <= ref.abs() * 2.0 ** -8 + tol)
    loss, lse2, rest = nv.topk_distill(x, ids, top, tail=True)  # a teacher that is the student
    assert torch.all(loss.abs() < 10 * tol)
    dd = nv.topk_distill_backward(x, ids, top, lse2, one, tail=True, lse_tail=rest)
    assert torch.all(dd.double().abs() < 20 * tol)


def test_offsets_beyond_32_bits(nv):
    """2.4 billion logits: the last rows lie behind element 2^31 (and 4 GB)."""
    M, V = 16000, 151665
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(M, V, dtype=torch.bfloat16, device="cuda")
    for a in range(0, M, 2000):
        x[a:a + 2000] = torch.randn(2000, V, generator=g, device="cuda").mul_(3.0)
    tok = torch.randint(0, V, (M,), generator=g, device="cuda").int()
    logp, h, lse, ids, top = nv.token_logprobs(x, tok, k=3)
    rows = torch.tensor([0, 1, 14159, 14160, 14161, M - 2, M - 1], device="cuda")
    z = x[rows].double()
    lp = torch.log_softmax(z, 1)
    assert torch.allclose(lse[rows].double(), torch.logsumexp(z, 1), rtol=0, atol=2e-4)
    assert torch.allclose(logp[rows].double(), lp.gather(1, tok[rows].long()[:, None])[:, 0], rtol=0, atol=2e-4)
    order = torch.sort(x[rows].float(), dim=1, descending=True, stable=True).indices[:, :3]
    assert torch.equal(ids[rows].long(), order)
    dl = torch.randn(M, generator=g, device="cuda")
    d = nv.token_logprobs_backward(x, tok, lse, dl, out=x)
    ref = -dl[rows].double()[:, None] * lp.exp()
    ref.scatter_add_(1, tok[rows].long()[:, None], dl[rows].double()[:, None])
    # p off by 2e-4 relative at most (the lse's bound above), then half an ulp of bf16
    assert torch.all((d[rows].double() - ref).abs() <= ref.abs() * (2.0 ** -8 + 4e-4) + 1e-7 * dl[rows].abs()[:, None])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_vocabulary(nv, dtype):
    """More columns than one block of step maxima and one bit map hold, in rows with one CTA each (64 bits by torch)."""
    M, V, k = 160, 400003, 70
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(4)
    x = (torch.randn(M, V, generator=g, device="cuda") * 2).to(t)
    ramp = torch.linspace(-9, 9, V, device="cuda").to(t)
    x[1] = 1.5
    x[2] = ramp
    x[3] = (torch.rand(V, generator=g, device="cuda") < 0.5).to(t)
    x[4, :350000] = -torch.inf
    x[5, :-3] = torch.finfo(t).min
    x[6] = ramp.flip(0)
    x[7] = -5 - torch.rand(V, generator=g, device="cuda").to(t)
    x[8, 390000:] = 3.0                      # ties for the last places, in the last block
    tok = torch.randint(0, V, (M,), generator=g, device="cuda").int()
    tok[5] = V - 1
    logp, h, lse, ids, top = nv.token_logprobs(x, tok, k=k)
    rows = torch.arange(12, device="cuda")
    f = x[rows].double()
    z = torch.where(f <= G.MASKED, -torch.inf, f)
    lp = torch.log_softmax(z, 1)
    order = torch.sort(f, dim=1, descending=True, stable=True).indices[:, :k]
    want = torch.where(z.gather(1, order) > -torch.inf, order, -1)
    assert torch.equal(ids[rows].long(), want)
    ref_lse = torch.logsumexp(z, 1)
    ref_h = -(lp.exp() * torch.where(lp == -torch.inf, 0.0, lp)).sum(1)
    # S of _logits.py with V / 512 additions in a chain, E[D] <= ln V
    tol = (3 * 13 + 4 + V / 512 + 64) * G.U + 8 * G.U * (ref_lse.abs() + 13)
    assert torch.all((lse[rows].double() - ref_lse).abs() <= tol)
    assert torch.all((h[rows].double() - ref_h).abs() <= tol * (1 + 3 * 13))
    got, ref = logp[rows].double(), lp.gather(1, tok[rows].long()[:, None])[:, 0]
    fin = torch.isfinite(ref)
    assert torch.equal(fin, torch.isfinite(got)) and torch.all(((got - ref).abs() <= tol + 8 * G.U * ref.abs())[fin])
    # the bit map's borders: vectors of 8 or 4 columns around 2^18, the first and the last column
    edge = torch.tensor([0, 1, 262139, 262142, 262143, 262144, 262145, 262150, V - 2, V - 1], device="cuda")
    tid = edge.expand(M, -1).int().contiguous()
    tl = torch.log_softmax(torch.randn(M, 11, generator=g, device="cuda"), 1)[:, :10].contiguous()
    live = torch.tensor([0, 3, 7, 9, 10, 11], device="cuda")  # rows whose listed columns are all unmasked
    loss, lse2, rest = nv.topk_distill(x, tid, tl, tail=True)
    lp, q = lp[live], tl[live].double().exp()
    q0 = 1 - q.sum(1)
    ref_rest = torch.logsumexp(z[live].scatter(1, edge.expand(6, -1), -torch.inf), 1)
    ref = (q * (tl[live].double() - lp[:, edge])).sum(1) + q0 * (q0.log() - (ref_rest - ref_lse[live]))
    assert torch.all((rest[live].double() - ref_rest).abs() <= tol[live])
    assert torch.all((loss[live].double() - ref).abs() <= 2 * tol[live] + 64 * G.U * (1 + ref.abs()))
    d = nv.topk_distill_backward(x, tid, tl, lse2, torch.ones(M, device="cuda"), tail=True, lse_tail=rest)[live].double()
    p0 = (ref_rest - ref_lse[live]).exp()
    ref = lp.exp() * (1 - q0 / p0)[:, None]
    ref[:, edge] = lp[:, edge].exp() - q
    half = 2.0 ** -8 if dtype == "bf16" else G.U
    assert torch.all((d - ref).abs() <= ref.abs() * half + lp.exp() * (4 * tol[live] + 64 * G.U)[:, None] * (1 + q0 / p0)[:, None]
                     + 32 * G.U * ((ref != 0) * q.max()))


def test_stream_argument(nv):
    x = dev(G.make(12, 9001, "bf16", 5))
    tok = torch.arange(12, dtype=torch.int32, device="cuda")
    _, ids, l = teacher_case(12, 9001, 5, "bf16", 17)
    ids, l = P.dev(ids), P.dev(l)
    one = torch.ones(12, device="cuda")

    def all_four(s):
        a = nv.token_logprobs(x, tok, k=4, stream=s)
        b = nv.topk_distill(x, ids, l, stream=s)
        return [*a, *b[:2], nv.token_logprobs_backward(x, tok, a[2], one, stream=s),
                nv.topk_distill_backward(x, ids, l, b[1], one, stream=s)]
    want = all_four(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = all_four(s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))


def test_same_bits_on_every_call_and_stream(nv):
    x = dev(G.make(40, 30011, "bf16", 5))
    tok = torch.arange(40, dtype=torch.int32, device="cuda")
    _, ids, l = teacher_case(40, 30011, 50, "bf16", 17, twice=True)
    ids, l = P.dev(ids), P.dev(l)
    dl = torch.randn(40, device="cuda")
    torch.cuda.synchronize()

    def all_four():
        a = nv.token_logprobs(x, tok, k=20)
        b = nv.topk_distill(x, ids, l, tail=True)
        return [*a, *b, nv.token_logprobs_backward(x, tok, a[2], dl, entropy=a[1], dentropy=dl),
                nv.topk_distill_backward(x, ids, l, b[1], dl, tail=True, lse_tail=b[2])]
    first = all_four()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(6):  # calls on two streams at once
        with torch.cuda.stream(streams[i % 2]):
            outs.append(all_four())
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(p, q) for p, q in zip(first, o))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = all_four()
    for t in kept:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, kept))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [2.0 ** -20, 1e-3, 300.0, 2.0 ** 20])
def test_scales_at_the_ends(nv, dtype, scale):
    """The tolerances grow with |z| and |lse|, which fp32 holds to half an ulp; the order of the alternatives is the logits'."""
    M, V = 4, 2500
    x = G.make(M, V, dtype, 101)
    tok = np.array([3, 2499, -1, 7], np.int32)
    check_forward(nv, x, V, tok, scale, 40, dtype, what=f"scale {scale} {dtype}")
    one = np.ones(M, np.float32)
    if scale < 1000.0:  # above, lse itself is off by more than a nat
        check_backward(nv, x, V, tok, scale, dtype, one, None, what=f"scale {scale} {dtype}")


def test_a_graph_replays_on_new_contents(nv):
    """A captured step, in place and over few rows (clusters) and many, reads what lies in its tensors at replay time."""
    for M, V, k in ((3, 20001, 20), (700, 3001, 33)):
        x, ids, l = teacher_case(M, V, k, "bf16", 111)
        x = dev(x)
        tok = torch.arange(M, dtype=torch.int32, device="cuda")
        ids, l, one = P.dev(ids), P.dev(l), torch.ones(M, device="cuda")
        logits = x.clone()

        def step():
            a = nv.token_logprobs(logits, tok, k=k)
            b = nv.topk_distill(logits, ids, l, tail=True)
            d = nv.topk_distill_backward(logits, ids, l, b[1], one, tail=True, lse_tail=b[2])
            return [*a, *b, d, nv.token_logprobs_backward(logits, tok, a[2], one, entropy=a[1], dentropy=one, out=logits)]
        step()
        torch.cuda.synchronize()
        logits.copy_(x)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kept = step()
        for seed in (1, 2):
            new = dev(G.make(M, V, "bf16", seed))
            tok.copy_(torch.randint(-1, V, (M,), device="cuda").int())
            logits.copy_(new)
            g.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in kept]
            logits.copy_(new)
            want = step()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_policy_step_from_linear_to_gradient(nv):
    """The run they are made for: logits of the same tokens from the W4A16 rollout head and from the bf16 trainer
    head, log-probs of both, AIS weights, and the gradient of the weighted policy objective to the trainer's logits;
    then the teacher's top alternatives distilled into the student."""
    M, N, K, V = 48, 1024, 512, 1000  # 1000 columns of the 1024 are the vocabulary
    W = synth.weight_bf16(N, K, 0.08, 3, 1)
    xh = synth.activation_bf16(M, K, 4, 1)
    codes, scales, g = nv.nvfp4_quantize(P.dev_bf16(W))
    hidden = P.dev_bf16(xh)
    z_roll = nv.nvfp4_lora_linear(hidden, codes, scales, g)
    z_train = (hidden.float() @ P.dev_bf16(W).float().t()).bfloat16()
    r = synth.rng(12)
    tok = r.integers(0, V, M).astype(np.int32)
    tok[::7] = -100
    adv = r.standard_normal(M).astype(np.float32)
    td = P.dev(tok)
    lp_r = nv.token_logprobs(z_roll[:, :V], td, entropy=False)[0]
    lp_t, h, lse, ids, top = nv.token_logprobs(z_train[:, :V], td, k=8)
    live = torch.from_numpy(tok >= 0).cuda()
    stats, w = nv.ais_mixing(lp_r[live].contiguous(), lp_t[live].contiguous(), P.dev(adv)[live].contiguous(), 2.0, 0.05,
                             0.5, 1.0)
    dl = torch.zeros(M, device="cuda")
    dl[live] = -w * P.dev(adv)[live] / int(live.sum())
    d = nv.token_logprobs_backward(z_train[:, :V], td, lse, dl)
    torch.cuda.synchronize()
    bits_r, bits_t = P.host_bits(z_roll), P.host_bits(z_train)
    o_r = oracle.token_logprobs(bits_r, tok, 1.0, V=V)[0]
    o_t = oracle.token_logprobs(bits_t, tok, 1.0, 8, V=V)
    on = tok >= 0
    # the per-row bound of _logits.py at |z|, D <= 60, V = 1000: (3 * 60 + 4 + 80 + 8 * 120) u < 8e-5
    assert np.abs(f64(lp_r) - o_r).max() < 8e-5 and np.abs(f64(lp_t) - o_t[0]).max() < 8e-5
    assert np.array_equal(ids.cpu().numpy(), o_t[3])
    ost, ow = oracle.ais(o_r[on], o_t[0][on], adv[on], 2.0, 0.05, 0.5, 1.0)
    # a weight min(exp(d), C) moves by at most C |error of d| = 2 * 1.6e-4, alpha by as much over delta
    assert np.abs(f64(w) - ow).max() < 2 * 1.6e-4 * (1 + 1 / 0.05)
    ref = oracle.token_logprobs_grad(bits_t, tok, 1.0, dl.cpu().numpy(), None, V=V)
    assert np.all(np.abs(f64(d) - ref) <= np.abs(ref) * (2.0 ** -8 + 2e-4) + 1e-6 * np.abs(dl.cpu().numpy())[:, None])
    # distillation: the trainer's alternatives as the teacher of the rollout head
    loss, lse_s, rest = nv.topk_distill(z_roll[:, :V], ids, top, tail=True)
    gd = nv.topk_distill_backward(z_roll[:, :V], ids, top, lse_s, torch.ones(M, device="cuda"), tail=True, lse_tail=rest)
    torch.cuda.synchronize()
    o_l = oracle.topk_distill(bits_r, ids.cpu().numpy(), top.cpu().numpy(), 1.0, True, V=V)[0]
    assert np.all(f64(loss)[on] >= -1e-4) and np.abs(f64(loss) - o_l).max() < 1e-3 and np.all(f64(loss)[~on] == 0)
    o_g = oracle.topk_distill_grad(bits_r, ids.cpu().numpy(), top.cpu().numpy(), 1.0, True, np.ones(M, np.float32), V=V)
    assert np.abs(f64(gd) - o_g).max() < 4e-3  # half an ulp of bf16 at 1 and the bound above


# ---- logits far from 0: offsets, and masks that are large finite numbers ----

def relative(x, scale, V):
    """From 64-bit scores relative to each row's maximum (z itself would lose them): ln p, entropy, ln s, E[D]."""
    d = G.values(x[:, :V])
    d = (d - d.max(1, keepdims=True)) * float(np.float32(scale))
    s = np.exp(d).sum(1)
    lp = d - np.log(s)[:, None]
    D = np.where(np.isfinite(d), -d, 0.0)
    p = np.exp(lp)
    ED = (p * D).sum(1)
    return lp, np.log(s) + ED, np.log(s), ED


def far_rows(M, V, dtype, fill, seed):
    """Rows that are `fill` but for: nothing; a few ordinary columns; the last column; all but one ordinary; differing
    fills; an ordinary row moved by fill (fp32 keeps little or nothing of it)."""
    x = G.make(M, V, "f32", seed)
    keep = x.copy()
    r = synth.rng(seed, M, 3)
    x[:] = fill
    for m in range(1, M):
        kind = m % 6
        if kind == 1:
            c = r.choice(V, size=5, replace=False)
            x[m, c] = keep[m, c]
        elif kind == 2:
            x[m, -1] = keep[m, -1]
        elif kind == 3:
            x[m] = keep[m]
            x[m, r.integers(V)] = fill
        elif kind == 4:
            x[m] = fill * (1.0 + 0.5 * r.random(V))
        elif kind == 5:
            x[m] = fill + keep[m]
    x = x.astype(np.float32)
    return synth.bf16_bits(x) if dtype == "bf16" else x


FILLS = [-1e4, -1e7, -1e9, -1e10, -1e30, 1e10, 3e29]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fill", FILLS)
@pytest.mark.parametrize("M,V", [(7, 5003), (7, 40000), (700, 1501)])
def test_forward_far_from_zero(nv, dtype, fill, M, V):
    for scale in (1.0, 0.7):
        x = far_rows(M, V, dtype, fill, 71)
        lp, h, ln_s, ED = relative(x, scale, V)
        tok = np.argmax(G.values(x), axis=1).astype(np.int32)
        tok[::2] = (np.arange(M)[::2] * 7919) % V
        S = (3 * ED + 4 + V / 64 + 64) * G.U  # as in _logits.py; scores beyond 2^24 are rounded once more, 2 u D
        S += 2 * G.U * ED
        xd, td = dev(x), P.dev(tok)
        for k in (0, 5, 40):
            logp, hd, lse, ids, top = nv.token_logprobs(xd, td, scale, k=k)
            at = lp[np.arange(M), tok]
            far = np.abs(at + ln_s)
            G.close(f64(logp), at, S + 10 * G.U * (far + ln_s), f"logp k={k}")
            G.close(f64(hd), h, S * (1 + 3 * ED) + 8 * G.U * (ED + ln_s), f"entropy k={k}")
            z = G.values(x).max(1) * float(np.float32(scale))
            G.close(f64(lse), z + ln_s, S + 8 * G.U * (np.abs(z) + ln_s), f"lse k={k}")
            if k:
                order = np.argsort(-G.values(x), axis=1, kind="stable")[:, :k]
                assert np.array_equal(ids.cpu().numpy(), order)
                want = np.take_along_axis(lp, order, 1)
                G.close(f64(top), want, S[:, None] + 10 * G.U * (np.abs(want + ln_s[:, None]) + ln_s[:, None]), "top")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fill", FILLS)
@pytest.mark.parametrize("tail", [False, True])
def test_distill_far_from_zero(nv, dtype, fill, tail):
    M, V, k = 37, 3001, 9
    x = far_rows(M, V, dtype, fill, 72)
    ids, t = G.teacher(M, k, V, 73)
    ids[::3, 0] = np.argmax(G.values(x), axis=1)[::3]
    ids[::3, 1:] = (ids[::3, :1] + 1 + np.arange(k - 1)) % V
    lp, _, ln_s, ED = relative(x, 1.0, V)
    li = np.take_along_axis(lp, ids.astype(np.int64), 1)
    lq = t.astype(np.float64)
    if not tail:
        lq = lq - np.log(np.exp(lq).sum(1, keepdims=True))
    q = np.exp(lq)
    ref = (q * (lq - li)).sum(1)
    size = (q * (np.abs(lq) + np.abs(li))).sum(1)
    S = (5 * np.log(V) + 4 + V / 64 + 64) * G.U  # E[D] = entropy - ln s, of the row as of its unlisted columns, is below ln V
    if tail:
        un = lp.copy()
        np.put_along_axis(un, ids.astype(np.int64), -np.inf, 1)
        top = un.max(1)
        rest = top + np.log(np.exp(un - top[:, None]).sum(1))  # ln p_0
        q0 = 1 - q.sum(1)
        ref += q0 * (np.log(q0) - rest)
        size += q0 * (np.abs(np.log(q0)) + np.abs(rest))
    loss, lse, lse_tail = nv.topk_distill(dev(x), P.dev(ids), P.dev(t), tail=tail)
    # each term q (ln q - ln p): ln q by (8 |ln q| + 40) u, ln p by S and 10 u |ln p|, the sum of k + 1 terms by (k + 8) u;
    # q_0, by the errors of k + 1 exponentials and their sum, (k + 12) u absolute
    extra = (k + 12) * G.U * np.abs(np.log(q0) - rest) if tail else 0.0
    G.close(f64(loss), ref, 2 * S + (k + 60) * G.U * (size + 1) + extra, "loss")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fill", FILLS)
@pytest.mark.parametrize("shift", [0, 3])
def test_gradients_far_from_zero(nv, dtype, fill, shift):
    """Masks far below ordinary logits, rows that are far as a whole (one largest logit, equal ones, ordinary ones moved),
    and far buckets of unlisted columns. A row's gradients add up to 0."""
    M, V, k = 8, 2049, 5
    x = G.make(M, V, "f32", 74)
    low = -abs(fill)
    x[1, ::2] = low
    x[2] = fill * (1.5 if fill < 0 else 0.5)
    x[2, 77] = fill
    x[3] = low
    x[3, [77, 1024, 1028, 5, 2000]] = [1.0, 2.0, 0.5, -1.0, 3.0]
    x[4] = np.where(np.arange(V) % 3 == 0, -np.inf, fill * (1.5 if fill < 0 else 0.5))
    x[4, 78] = fill
    x[6] = fill
    x[7] += np.float32(fill)
    x = synth.bf16_bits(x) if dtype == "bf16" else x
    scale = 1.25
    lp, h, ln_s, ED = relative(x, scale, V)
    p = np.exp(lp)
    ln = np.where(p > 0, lp, 0.0)
    tok = np.array([5, 1, 77, 1026, 5, 0, 9, 11], np.int32)
    dl = np.linspace(-1.0, 1.5, M).astype(np.float32)
    dh = np.linspace(0.5, -0.7, M).astype(np.float32)
    xd, td = dev(x, shift=shift), P.dev(tok)
    _, hd, lse, _, _ = nv.token_logprobs(xd, td, scale)
    hit = np.zeros((M, V))
    hit[np.arange(M), tok] = 1.0

    def p_error(ref_lse, lp):
        """Of p taken from ref_lse, relative: its rounding and that of |z| <= |lse| + |ln p| (3 u each, 8 u for lse's own
        sums), or up to 2^12; past it the sums are formed anew, which leaves what the forward call has."""
        S = (3 * ED + 4 + V / 64 + 64) * G.U
        far = np.abs(ref_lse) > 2.0 ** 12
        return S[:, None] + G.U * (6 * np.abs(lp) + 40 + np.where(far, 0.0, 14 * np.abs(np.where(far, 0.0, ref_lse)))[:, None])

    e = p_error(f64(lse), ln)
    for g_h in (None, dh):
        kw = dict(entropy=hd, dentropy=None if g_h is None else P.dev(g_h))
        got = nv.token_logprobs_backward(xd, td, lse, P.dev(dl), scale, **kw)
        in_place = xd.clone()
        nv.token_logprobs_backward(in_place, td, lse, P.dev(dl), scale, out=in_place, **kw)
        assert torch.equal(got, in_place)
        got = f64(got.float())
        ref = dl[:, None] * (hit - p) - (0.0 if g_h is None else g_h[:, None] * p * (ln + h[:, None]))
        part = np.abs(dl)[:, None] + np.abs(dh)[:, None] * (np.abs(ln) + h[:, None] + 1)
        tol = 4 * e * p * part + 16 * G.U * hit + 2.0 ** -120
        G.close(got, ref * scale, tol * scale + G.half_ulp(ref * scale, dtype), f"dlogits entropy {g_h is not None}")
    ids = np.stack([np.array([77, 1024, 1028, 5, 2000], np.int32)] * M)
    t = np.log(np.array([0.4, 0.2, 0.1, 0.1, 0.05], np.float32))[None].repeat(M, 0)
    q = np.zeros((M, V))
    np.put_along_axis(q, ids.astype(np.int64), np.exp(t.astype(np.float64)), 1)
    for tail in (False, True):
        loss, l2, lt = nv.topk_distill(xd, P.dev(ids), P.dev(t), scale, tail=tail)
        in_place = xd.clone()
        assert in_place.stride() == xd.stride()
        got = nv.topk_distill_backward(xd, P.dev(ids), P.dev(t), l2, P.dev(dl), scale, tail=tail, lse_tail=lt)
        nv.topk_distill_backward(in_place, P.dev(ids), P.dev(t), l2, P.dev(dl), scale, tail=tail, lse_tail=lt, out=in_place)
        assert torch.equal(got, in_place)
        got = f64(got.float())
        b, Q = np.zeros_like(p), q.sum(1, keepdims=True)
        if tail:
            un = np.where(q > 0, -np.inf, lp)
            top = un.max(1, keepdims=True)
            there = np.isfinite(top)
            b = np.where(there, np.exp(un - np.where(there, top, 0.0)), 0.0)
            b /= np.where(there, b.sum(1, keepdims=True), 1.0)  # the bucket's own softmax
            Q = np.where(there, 1.0, Q)
            ref = dl[:, None] * (Q * p - q - np.where(there, 1 - q.sum(1, keepdims=True), 0.0) * b)
            e = np.maximum(e, p_error(f64(lt), np.where(b > 0, np.log(np.maximum(b, 1e-300)), 0.0)))
        else:
            ref = dl[:, None] * (p - q / Q)
        tol = 4 * e * (p + b) + 60 * G.U * (p + q + b) + 2.0 ** -120
        G.close(got, ref * scale, tol * scale * np.abs(dl)[:, None] + G.half_ulp(ref * scale, dtype), f"distill tail {tail}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scales_at_the_ends_of_their_range(nv, dtype):
    """2^20 and 2^-20 with masked columns and logits of either bound: nothing turns into NaN."""
    M, V = 5, 6007
    x = G.make(M, V, "f32", 75)
    x[:, 1::7] = -np.inf
    x[1] *= 2.0 ** -18
    x[2] = -(2.0 ** 99)
    x[2, -1] = 2.0 ** 99
    x[3, :4000] = -(2.0 ** 99)
    x = synth.bf16_bits(x) if dtype == "bf16" else x
    tok = np.full(M, 6006, np.int32)
    one = np.ones(M, np.float32)
    for scale in (2.0 ** 20, 2.0 ** -20):
        lp, h, ln_s, ED = relative(x, scale, V)
        logp, hd, lse, _, _ = nv.token_logprobs(dev(x), P.dev(tok), scale, k=3)
        S = (5 * ED + 4 + V / 64 + 64) * G.U
        G.close(f64(hd), h, S * (1 + 3 * ED) + 8 * G.U * (ED + ln_s), "entropy")
        G.close(f64(logp), lp[:, -1], S + 10 * G.U * (np.abs(lp[:, -1] + ln_s) + ln_s), "logp")
        for dh in (0.5, 1000.0):
            got = nv.token_logprobs_backward(dev(x), P.dev(tok), lse, P.dev(one), scale, entropy=hd, dentropy=P.dev(one * dh))
            got = f64(got.float())
            assert np.all(np.isfinite(got))
            assert np.all(got[:, 1::7][G.values(x)[:, 1::7] == -np.inf] == 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,V", [(2, 60000), (40, 90001), (700, 30001), (2500, 9001)])
def test_alternatives_of_a_row_with_a_nan_behind_its_largest_logits(nv, dtype, M, V):
    """The NaN comes after the thread has seen logits far above all it sees later; many candidates are listed."""
    x = G.make(M, V, "f32", 76)
    r = synth.rng(77, M, V)
    for m in range(0, M, 2):
        x[m, :V // 8] = (1e3 * 10.0 ** (30 * r.random(V // 8)) * np.where(r.random(V // 8) < 0.5, 1, -1)).clip(-1e30, 1e30)
        x[m, V // 2 + 11 * m % (V // 3)::97] = np.nan
    x = synth.bf16_bits(x) if dtype == "bf16" else x
    for k in (1, 20, 64, 200):
        logp, h, lse, ids, top = nv.token_logprobs(dev(x), P.dev(np.arange(M, dtype=np.int32)), k=k)
        torch.cuda.synchronize()
        for t in (logp, h, lse, top):
            assert bool(torch.isnan(t[::2]).all()) and not bool(torch.isnan(t[1::2]).any())
        assert bool((ids[::2] == -1).all())
        order = np.argsort(-G.values(x[1::2]), axis=1, kind="stable")[:, :k]
        assert np.array_equal(ids[1::2].cpu().numpy(), order)
