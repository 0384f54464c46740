"""The logits operators on long rows, against 64-bit definitions."""
import numpy as np
import pytest
import torch

from tests import _logits as G
from tests import _parity as P
from tests.test_logprobs_gpu import _bits, dev, f64, nv, relative  # noqa: F401  (nv: the fixture)

pytestmark = pytest.mark.gpu


def far_and_long(V):
    """fp32 rows whose lse is past 2^12, of terms that a plain chain of additions drifts with: all but one column (or
    three) at one value, and an ordinary row moved."""
    x = np.full((3, V), -6000.0, np.float32)
    x[0, V // 3] = -5999.0
    x[1, [5, V // 2, V - 1]] = -5999.75
    x[2] = G.make(1, V, "f32", 131)[0] - np.float32(8000.0)
    return x


# The widths of a row's CTA: 256 threads without a list, 64, 128, 256 by the list's length.
@pytest.mark.parametrize("V", [152064, (1 << 22) - 3])
@pytest.mark.parametrize("form", ["logp", "entropy", "k20", "k20 tail", "k100", "k200 tail"])
def test_gradient_of_long_far_rows(nv, form, V):
    """A far row's sum is good to (4 E[D] + 30) u whatever its length: its terms to (4 D + 4) u (x - max, c, their product,
    the exponential), groups of 8 in turn 8 u, the compensated sum of the groups 2 u, the tree over 32 lanes and up to 8
    warps 13 u, 1 / s and its product with a term 3 u. p is good to that and its own term's (4 D + 4) u."""
    x = far_and_long(V)
    M = len(x)
    lp, h, ln_s, ED = relative(x, 1.0, V)
    p = np.exp(lp)
    S = ((4 * ED + 30) * G.U)[:, None]
    D = -(lp + ln_s[:, None])
    e = S + (4 * D + 4) * G.U
    lse = G.values(x).max(1) + ln_s
    dl = np.array([1.0, -0.75, 2.0], np.float32)
    w = np.abs(dl.astype(np.float64))[:, None]
    xd, lsed = dev(x), P.dev(lse.astype(np.float32))
    if not form.startswith("k"):
        tok = np.array([V // 3, 1, V - 2], np.int32)
        hit = np.zeros((M, V))
        hit[np.arange(M), tok] = 1.0
        dh = np.array([0.5, 1.0, -0.25], np.float32) if form == "entropy" else None
        kw = {} if dh is None else dict(entropy=P.dev(h.astype(np.float32)), dentropy=P.dev(dh))
        got = nv.token_logprobs_backward(xd, P.dev(tok), lsed, P.dev(dl), **kw)
        ref = dl[:, None] * (hit - p)
        tol = w * p * e
        if dh is not None:
            # ln p + H: ln s by S and 2 u of itself, the score by 2 u D, H and the sum by 2 u of their parts
            part = S + 4 * G.U * (np.abs(lp) + ln_s[:, None] + h[:, None])
            ref = ref - dh[:, None] * p * (lp + h[:, None])
            tol = tol + np.abs(dh)[:, None] * p * (e * np.abs(lp + h[:, None]) + part)
        tol = tol + 4 * G.U * w * hit
    else:
        k, tail = int(form.split()[0][1:]), form.endswith("tail")
        ids, t = G.teacher(M, k, V, 132)
        ids[:, 1] = V // 3
        at = ids.astype(np.int64)
        lq = t.astype(np.float64)
        if not tail:
            lq = lq - np.log(np.exp(lq).sum(1, keepdims=True))
        q = np.zeros((M, V))
        np.put_along_axis(q, at, np.exp(lq), 1)
        rest, b, q0 = None, 0.0, np.zeros(M)
        if tail:
            un = lp.copy()
            np.put_along_axis(un, at, -np.inf, 1)
            top = un.max(1)
            ln_p0 = top + np.log(np.exp(un - top[:, None]).sum(1))
            q0 = 1 - q.sum(1)
            b = np.exp(un - ln_p0[:, None])
            rest = P.dev((lse + ln_p0).astype(np.float32))
        got = nv.topk_distill_backward(xd, P.dev(ids), P.dev(t), lsed, P.dev(dl), tail=tail, lse_tail=rest)
        ref = dl[:, None] * (p - q - q0[:, None] * b)
        # q by its exponential and the list's sums (4 |ln q| + k + 24) u, q_0 by the k + 1 exponentials' (k + 16) u. The
        # bucket's sum holds the listed terms until they are taken out: below twice its size here.
        e_q = (4 * np.abs(lq).max() + k + 24) * G.U
        tol = w * (p * (e + (k + 16) * G.U * tail) + q * e_q)
        if tail:
            tol = tol + w * b * (q0[:, None] * (2 * e + S) + (k + 16) * G.U)
    torch.cuda.synchronize()
    # the result's own additions and its rounding: 4 u of their parts
    tol = tol + 4 * G.U * (np.abs(ref) + w * p)
    G.close(f64(got), ref, tol * 1.02 + 2.0 ** -120, f"dlogits {form} {V}")


def test_tensors_given_as_outputs_count_as_modified(nv):
    """A graph that saved the logits must not go on with the gradient in their place."""
    V, k = 1000, 4
    leaf = torch.randn(6, 1024, device="cuda", requires_grad=True)
    tok = torch.arange(6, dtype=torch.int32, device="cuda")
    one = torch.ones(6, device="cuda")
    for write in ("token", "distill"):
        for view in (lambda t: t, lambda t: t[:, :V], lambda t: t.detach()[:, :V]):
            logits = leaf * 2.0
            penalty = logits.square().sum()  # saves the logits
            x = view(logits)
            _, _, lse, ids, top = nv.token_logprobs(x, tok, k=k)
            torch.autograd.grad(penalty, leaf, retain_graph=True)  # the forward call changes nothing
            if write == "token":
                nv.token_logprobs_backward(x, tok, lse, one, out=x)
            else:
                nv.topk_distill_backward(x, ids, top, lse, one, out=x)
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                torch.autograd.grad(penalty, leaf)
    f32 = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    x = leaf.detach()
    outs = dict(logp=f32(6), h=f32(6), lse=f32(6), top_ids=torch.empty(6, k, dtype=torch.int32, device="cuda"), top_logp=f32(6, k))
    nv.token_logprobs(x, tok, k=k, **outs)
    assert [t._version for t in outs.values()] == [1] * 5
    nv.token_logprobs(x, tok, entropy=False, **outs)  # writes neither the entropies nor the lists
    assert [t._version for t in outs.values()] == [2, 1, 2, 1, 1]
    loss, rest = f32(6), f32(6)
    nv.topk_distill(x, outs["top_ids"], outs["top_logp"], loss=loss, lse=outs["lse"], lse_tail=rest)
    assert (loss._version, outs["lse"]._version, rest._version) == (1, 3, 0)
    nv.topk_distill(x, outs["top_ids"], outs["top_logp"], tail=True, loss=loss, lse_tail=rest)
    assert (loss._version, rest._version) == (2, 1)
    with torch.inference_mode():  # tensors without versions
        y = torch.randn(6, V, device="cuda")
        lse = nv.token_logprobs(y, tok, lse=f32(6))[2]
        nv.token_logprobs_backward(y, tok, lse, one, out=y)
    nv.token_logprobs_backward(y, tok, lse, one, out=y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1000.0, 2.0 ** 15, 2.0 ** 20])
def test_gradients_at_large_scales(nv, dtype, scale):
    """Scores of thousands to millions: tied and neighbouring largest logits, equal rows, masked columns, and rows on
    either side of |lse| = 2^12, against softmaxes formed from differences to the maximum in 64 bits."""
    M, V = 7, 2500
    x = G.make(M, V, "f32", 134)
    x[1, [3, 70, 71]] = 13.0
    x[2, 100:108] = 13.0 - 2.0 ** -20 * np.arange(8)  # neighbours in fp32: a score apart at 2^20; equal in bf16
    x[3] = 0.25
    x[4, ::2] = -np.inf
    x[5] *= np.float32(2.0 ** -10)
    x[6] -= np.float32(20.0)
    if dtype == "bf16":
        x = _bits(x)
    lp, h, ln_s, ED = relative(x, scale, V)
    p = np.exp(lp)
    ln = np.where(p > 0, lp, 0.0)
    best = np.argmax(G.values(x), axis=1)
    tok = best.astype(np.int32)
    tok[2] = 103
    tok[::3] = 9
    dl = np.linspace(-1.0, 1.5, M).astype(np.float32)
    dh = np.linspace(0.5, -0.7, M).astype(np.float32)
    hit = np.zeros((M, V))
    hit[np.arange(M), tok] = 1.0
    xd, td = dev(x), P.dev(tok)
    _, hd, lse, _, _ = nv.token_logprobs(xd, td, scale)

    def p_error(ref_lse, lp):
        """Of p, relative: the sums' S, and 6 u |ln p| + 40 u of its own score and exponential; taken from a 32-bit lse
        (up to 2^12) also 14 u |lse|: its rounding and those of lse log2 e and of z = lse + ln p."""
        S = (3 * ED + 4 + V / 64 + 64) * G.U
        near = np.where(np.abs(ref_lse) > 2.0 ** 12, 0.0, np.abs(ref_lse))
        return S[:, None] + G.U * (6 * np.abs(lp) + 40 + 14 * near[:, None])

    e = p_error(f64(lse), ln)
    for g_h in (None, dh):
        kw = {} if g_h is None else dict(entropy=hd, dentropy=P.dev(g_h))
        got = f64(nv.token_logprobs_backward(xd, td, lse, P.dev(dl), scale, **kw).float())
        ref = dl[:, None] * (hit - p) - (0.0 if g_h is None else g_h[:, None] * p * (ln + h[:, None]))
        part = np.abs(dl)[:, None] + np.abs(dh)[:, None] * (np.abs(ln) + h[:, None] + 1)
        tol = 4 * e * p * part + 16 * G.U * hit + 2.0 ** -120
        G.close(got, ref * scale, tol * scale + G.half_ulp(ref * scale, dtype), f"dlogits entropy {g_h is not None}")
    k = 12
    ids, t = G.teacher(M, k, V, 135)
    ids[1::2, 0] = best[1::2]
    ids[1::2, 1:] = (best[1::2, None] + 1 + np.arange(k - 1)) % V
    at = ids.astype(np.int64)
    q = np.zeros((M, V))
    np.put_along_axis(q, at, np.exp(t.astype(np.float64)), 1)
    for tail in (False, True):
        _, l2, lt = nv.topk_distill(xd, P.dev(ids), P.dev(t), scale, tail=tail)
        got = nv.topk_distill_backward(xd, P.dev(ids), P.dev(t), l2, P.dev(dl), scale, tail=tail, lse_tail=lt)
        got = f64(got.float())
        b, Q, e2 = np.zeros_like(p), q.sum(1, keepdims=True), e
        if tail:
            un = G.values(x) * float(np.float32(scale))
            np.put_along_axis(un, at, -np.inf, 1)
            un -= un.max(1, keepdims=True)
            b = np.exp(un)
            b /= b.sum(1, keepdims=True)  # the bucket's own softmax
            ref = dl[:, None] * (p - q - (1 - Q) * b)
            e2 = np.maximum(e, p_error(f64(lt), np.where(b > 0, np.log(np.maximum(b, 1e-300)), 0.0)))
        else:
            ref = dl[:, None] * (p - q / Q)
        tol = 4 * e2 * (p + b) + 60 * G.U * (p + q + b) + 2.0 ** -120
        G.close(got, ref * scale, tol * scale * np.abs(dl)[:, None] + G.half_ulp(ref * scale, dtype), f"distill tail {tail}")


def hard_rows(M, V, t, seed):
    """Ordinary logits, and among the first rows: a constant, rising and falling ramps, two values, masks up to far into the
    row and up to the last three columns, negative values, ties for the last places at the row's end."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(M, V, generator=g, device="cuda") * 2).to(t)
    ramp = torch.linspace(-9, 9, V, device="cuda").to(t)
    x[1] = 1.5
    x[2] = ramp
    x[3] = (torch.rand(V, generator=g, device="cuda") < 0.5).to(t)
    x[4, :V * 7 // 8] = -torch.inf
    x[5, :-3] = torch.finfo(t).min
    x[6] = ramp.flip(0)
    x[7] = -5 - torch.rand(V, generator=g, device="cuda").to(t)
    x[8, V - V // 40:] = 3.0
    return x, torch.randint(0, V, (M,), generator=g, device="cuda").int()


def exact_rows(x):
    """ln p, lse and entropy in 64 bits."""
    f = x.double()
    z = torch.where(f <= G.MASKED, -torch.inf, f)
    lse = torch.logsumexp(z, 1)
    lp = z - lse[:, None]
    return z, lp, lse, -(lp.exp() * torch.where(lp == -torch.inf, 0.0, lp)).sum(1)


@pytest.mark.parametrize("dtype,M,V,ks", [
    ("f32", 610, 100003, (1, 20, 96)),            # CTAs of 128 threads: a block of steps is 81920 columns
    ("bf16", 610, 200003, (1, 20, 96)),           # 163840
    ("f32", 9, (1 << 22) - 3, (5, 70, 256)),      # clusters of 8 CTAs: four blocks in each share
    ("bf16", 9, (1 << 22) - 3, (5, 70, 256))])    # two
def test_alternatives_over_several_blocks(nv, dtype, M, V, ks):
    """Rows whose step maxima fill more than one block, in narrow CTAs and in clusters."""
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    x, tok = hard_rows(M, V, t, 141)
    tok[5] = V - 1
    n = min(M, 12)
    z, lp, ref_lse, ref_h = exact_rows(x[:n])
    order = torch.sort(x[:n].float(), dim=1, descending=True, stable=True).indices[:, :max(ks)]
    # S of _logits.py with V / 256 additions in a chain at most, E[D] <= ln V < 16
    tol = (3 * 16 + 4 + V / 256 + 64) * G.U + 8 * G.U * (ref_lse.abs() + 16)
    for k in ks:
        logp, h, lse, ids, top = nv.token_logprobs(x, tok, k=k)
        at = order[:, :k]
        there = z.gather(1, at) > -torch.inf
        assert torch.equal(ids[:n].long(), torch.where(there, at, -1))
        assert torch.all((lse[:n].double() - ref_lse).abs() <= tol)
        assert torch.all((h[:n].double() - ref_h).abs() <= tol * (1 + 3 * 16))
        want = torch.where(there, lp.gather(1, at), -torch.inf)
        got = top[:n].double()
        assert torch.equal(there, torch.isfinite(got))
        assert torch.all(((got - want).abs() <= tol[:, None] + 8 * G.U * want.abs())[there])
        got, want = logp[:n].double(), lp.gather(1, tok[:n].long()[:, None])[:, 0]
        fin = torch.isfinite(want)
        assert torch.equal(fin, torch.isfinite(got)) and torch.all(((got - want).abs() <= tol + 8 * G.U * want.abs())[fin])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_distill_with_several_maps_to_a_share(nv, dtype):
    """Clusters of 8 CTAs, each with more columns than its bit map of the listed ones holds: columns listed at the borders
    of the shares and of the maps within them (256000 columns of bf16, 261120 of fp32)."""
    M, V = 5, (1 << 22) - 3
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(151)
    x = (torch.randn(M, V, generator=g, device="cuda") * 2).to(t)
    share, per_map = 524288, 256000 if dtype == "bf16" else 261120
    edges = {0, 1, V - 2, V - 1}
    for r in (0, 1, 4, 7):
        for m in range(3):
            at = r * share + m * per_map
            edges |= {c for c in (at - 9, at - 8, at - 4, at - 1, at, at + 1, at + 7, at + 8) if 0 <= c < V}
    cols = torch.tensor(sorted(edges), device="cuda")
    k = len(cols)
    x[1, cols] = 12.0  # the listed columns hold most of p: the bucket's sum must not see them
    ids = cols.expand(M, -1).int().contiguous()
    tl = torch.log_softmax(torch.randn(M, k + 1, generator=g, device="cuda"), 1)[:, :k].contiguous()
    z, lp, ref_lse, _ = exact_rows(x)
    q = tl.double().exp()
    q0 = 1 - q.sum(1)
    ref_rest = torch.logsumexp(z.index_fill(1, cols, -torch.inf), 1)
    # S of _logits.py with V / 256 additions in a chain at most, E[D] <= ln V < 16, of the row as of its unlisted columns
    tol = (3 * 16 + 4 + V / 256 + 64) * G.U + 8 * G.U * (ref_lse.abs() + 16)
    loss, lse, rest = nv.topk_distill(x, ids, tl, tail=True)
    assert torch.all((lse.double() - ref_lse).abs() <= 2 * tol) and torch.all((rest.double() - ref_rest).abs() <= tol)
    at = lp[:, cols]
    ref = (q * (tl.double() - at)).sum(1) + q0 * (q0.log() - (ref_rest - ref_lse))
    size = (q * (tl.double().abs() + at.abs())).sum(1) + (q0.log().abs() + (ref_rest - ref_lse).abs())
    # ln p and ln p_0 by the sums' tol; every other part by (k + 60) u, as of its size
    assert torch.all((loss.double() - ref).abs() <= 3 * tol + (k + 60) * G.U * (size + 1))
    loss, lse, rest = nv.topk_distill(x, ids, tl)
    total = torch.logsumexp(tl.double(), 1, keepdim=True)
    ref = ((tl.double() - total).exp() * (tl.double() - total - at)).sum(1)
    assert rest is None and torch.all((lse.double() - ref_lse).abs() <= 2 * tol)
    assert torch.all((loss.double() - ref).abs() <= 2 * tol + (k + 60) * G.U * (size + 1))
