"""Definitions in 64 bits and tolerances for the tests of the cache's ragged write and read, the shared-prefix attention
and the losses.

Tolerances, from the kernels' arithmetic, with u = 2^-24 (half an ulp of fp32, relative):
  * Cache bytes are exact. A value read back is one fp32 product of an exact code x scale with g, then one rounding to
    bf16: also exact, given the same two steps.
  * Attention: scores are sums of 128 exact products in fp32; with every addition off by at most 2u of the running
    sum of magnitudes (an aligned tensor-core addition may cut instead of round), a score is off by at most
    ds = scale 130 2u sum |q k|, and so is its exponential, relative. ex2 and its fp32 argument: 4u + 4u |s - max| log2 e.
    P enters the second product rounded to f16 (2^-11 relative; below 2^-14 of the step's reference by at most
    2^-25 absolute, times the number of tokens). Sums over up to N tokens in fp32: 2 N u at most. Numerator and
    denominator have these errors each; the result is off by that times A = sum p |v|, then half a bf16 step (2^-8).
  * Policy loss: e^d (2^t within 2^-22 = 4u, one fma) and two products: 8u of a term, e^x - x - 1: 16u and 4u |x| e^|x| / k of it
    (x is rounded once); a step's sums: 13 additions; the rest (pairs, a division, the last fma): 5u. A gradient the
    same without sums; 1 - e^x is off by 4u of itself and u |x| e^x.
  * Preference loss: s_b in pairs (2^-40 of the magnitudes), h by dh = 3u (|beta s| + |margin|); a loss by dh + 10u (loss + 1),
    a slope by (dh + 12u) of its parts.
"""
import numpy as np

import oracle
import synth

U = 2.0 ** -24
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def encode(x, g):
    """(codes, scales) of rows [..., D] as bf16 bits or fp32, by the oracle."""
    if x.dtype == np.uint16:
        return oracle.kv_quantize(x, g)
    L = oracle.lib()
    x = np.ascontiguousarray(x, np.float32)
    D = x.shape[-1]
    codes, scales = np.zeros(x.shape[:-1] + (D // 2,), np.uint8), np.zeros(x.shape[:-1] + (D // 16,), np.uint8)
    if x.size:
        L.oracle_quantize_rows(oracle._ptr(x), oracle.F32, D, 0, x.size // D, float(np.float32(g)), oracle._ptr(codes),
                               oracle._ptr(scales))
    return codes, scales


def exact_products(codes, scales):
    """Code x scale of cache rows, exactly, as float64 [..., D]."""
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1,)).astype(np.int64)
    v = GRID[nib & 7] * np.where(nib & 8, -1.0, 1.0)
    b = scales.astype(np.int64)
    e, m = b >> 3, (b & 7).astype(np.float64)
    s = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    return v * np.repeat(s, 16, axis=-1)


def values(codes, scales, g, dtype="f32"):
    """What a read gives: fp32, or bf16 bits."""
    v = exact_products(codes, scales).astype(np.float32) * np.float32(g)
    return synth.bf16_bits(v) if dtype == "bf16" else v


def packed_to_cache(offsets, pos, T, Lmax):
    """Cache row (b, place) of every packed row, or None (no sequence), or (b, None) (outside the cache)."""
    at = []
    for t in range(T):
        b = [i for i in range(len(offsets) - 1) if offsets[i] <= t < offsets[i + 1]]
        if not b:
            at.append(None)
            continue
        p = t - offsets[b[0]] + (0 if pos is None else pos[b[0]])
        at.append((b[0], int(p) if 0 <= p < Lmax else None))
    return at


def cache(B, L, Hkv, seed, D=128, spread=1.0):
    """A cache of encoded normal rows: (codes, scales, g)."""
    x = (synth.rng(seed, B, L, Hkv).standard_normal((B, L, Hkv, D)) * spread).astype(np.float32)
    g = np.float32(max(1e-30, np.abs(x).max() if x.size else 1.0) / 2688)
    return encode(synth.bf16_bits(x), g) + (g,)


def attention(q, prefix, own, plens, groups, lens, scale):
    """(out, tolerance) in 64 bits. q [B, Hq, 128]; prefix, own: (k, v) values [P, Lp, Hkv, 128], [B, L, Hkv, 128] (or None)."""
    B, Hq, D = q.shape
    Hkv = (prefix or own)[0].shape[2]
    r = Hq // Hkv
    out, tol = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    for b in range(B):
        ks, vs = [], []
        for p in range(len(groups) - 1):
            if groups[p] <= b < groups[p + 1]:
                L = min(max(int(plens[p]), 0), prefix[0].shape[1])
                ks.append(prefix[0][p, :L])
                vs.append(prefix[1][p, :L])
        if own is not None:
            L = min(max(int(lens[b]), 0), own[0].shape[1])
            ks.append(own[0][b, :L])
            vs.append(own[1][b, :L])
        k = np.concatenate(ks) if ks else np.zeros((0, Hkv, D))
        v = np.concatenate(vs) if vs else np.zeros((0, Hkv, D))
        if len(k) == 0:
            continue
        N = len(k)
        for h in range(Hq):
            kh, vh = k[:, h // r], v[:, h // r]
            s = scale * (kh @ q[b, h])
            mags = abs(scale) * (np.abs(kh) @ np.abs(q[b, h]))
            top = s.max()
            p = np.exp(s - top)
            z = p.sum()
            p /= z
            out[b, h] = p @ vh
            e = 130 * 2 * U * mags + (4 + 4 * (top - s) * 1.4427) * U + 130 * 2 * U * mags[np.argmax(s)]
            A = p @ np.abs(vh)
            err = (p * e) @ np.abs(vh) + A * ((p * e).sum() + 2.0 ** -11 + 4 * N * U) + N * 2.0 ** -25 / z * np.abs(vh).max()
            tol[b, h] = err + np.abs(out[b, h]) * 2.0 ** -8 + 2.0 ** -133
    return out, tol


def f32(v):
    return float(np.float32(v))


def policy(logp, old, adv, offsets, ref=None, weights=None, mask=None, low=0.2, high=0.2, dual=0.0, kl=0.0, mode=0,
           norm=1.0, per_token=False, dloss=1.0):
    """Dict of loss, stats, dlogp in 64 bits, and their tolerances under 'tol'."""
    n, B = len(logp), len(offsets) - 1
    low, high, dual, kl, norm = f32(low), f32(high), f32(dual), f32(kl), f32(norm)
    seq = np.full(n, -1)
    for b in range(B):
        seq[offsets[b]:offsets[b + 1]] = b
    live = (seq >= 0) & (True if mask is None else mask != 0)
    i = np.nonzero(live)[0]
    s = seq[i]
    lp = logp[i].astype(np.float64)
    d = lp - old[i].astype(np.float64)
    A = (adv[i] if per_token else adv[s]).astype(np.float64)
    w = np.ones(len(i)) if weights is None else weights[i].astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        r = np.exp(d)
        over, under, far = (A > 0) & (r > 1 + high), (A < 0) & (r < 1 - low), (A < 0) & (dual > 0) & (r > dual)
        used = np.where(far, dual, np.where(over, 1 + high, np.where(under, 1 - low, r)))
        l = np.where(A == 0, 0.0, -w * used * A)
        stop = over | under | far
        g_pol = np.where(stop, 0.0, l)
        x = np.zeros(len(i)) if ref is None else ref[i].astype(np.float64) - lp
        k = np.expm1(x) - x
        g_kl = -kl * np.expm1(x)
    count = np.bincount(s, minlength=B).astype(np.float64)[:B] if B else np.zeros(0)
    tokens, there = count.sum(), float((count > 0).sum())
    if mode == 0:
        coef = np.full(B, 1 / max(tokens, 1))
    elif mode == 1:
        coef = 1 / (np.maximum(count, 1) * max(there, 1))
    else:
        coef = np.full(B, 1 / norm)
    c = coef[s]
    grad = np.zeros(n)
    grad[i] = dloss * c * (g_pol + g_kl)
    pol, div = (c * l).sum(), (c * k).sum()
    m = max(tokens, 1)
    drift = np.expm1(d) - d
    stats = np.array([pol + kl * div, pol, div, stop.sum() / m, drift.sum() / m, r.sum() / m, tokens, there])
    ek = 16 * k + 4 * np.abs(x) * np.exp(np.abs(x))
    t_pol, t_div = U * (26 * c * np.abs(l)).sum(), U * (c * (ek + 18 * k)).sum()
    t_loss = t_pol + kl * t_div + 2 * U * abs(stats[0])
    t_drift = U * (34 * drift + 4 * np.abs(d) * np.exp(np.abs(d))).sum() / m
    t_stats = np.array([t_loss, t_pol, t_div, 4 * U * stats[3], t_drift, 26 * U * stats[5], U * tokens, 0.0]) + 2.0 ** -120
    t_grad = np.zeros(n)
    t_grad[i] = abs(dloss) * c * U * (14 * np.abs(g_pol) + kl * (8 * np.abs(np.expm1(x)) + 2 * np.abs(x) * np.exp(x)))
    return {"loss": stats[:1], "stats": stats, "dlogp": grad, "coef": coef,
            "tol": {"loss": t_stats[:1], "stats": t_stats, "dlogp": t_grad + 6 * U * np.abs(grad) + 2.0 ** -120,
                    "coef": 4 * U * coef}}


def preference(logp, offsets, ref=None, mask=None, beta=0.1, margin=0.0, smoothing=0.0, mean=False, dloss=None):
    n, seqs = len(logp), len(offsets) - 1
    beta, margin, eps = f32(beta), f32(margin), f32(smoothing)
    total, size, count = np.zeros(seqs), np.zeros(seqs), np.zeros(seqs)
    for b in range(seqs):
        t = np.arange(offsets[b], offsets[b + 1])
        t = t[mask[t] != 0] if mask is not None else t
        x = logp[t].astype(np.float64) - (0.0 if ref is None else ref[t].astype(np.float64))
        total[b], size[b], count[b] = x.sum(), np.abs(x).sum(), len(t)
    share = 1 / np.maximum(count, 1) if mean else np.ones(seqs)
    reward = beta * total * share
    with np.errstate(over="ignore", invalid="ignore"):
        h = reward[::2] - reward[1::2] - margin
        dh = 3 * U * (np.abs(reward[::2] - reward[1::2]) + abs(margin)) + 2.0 ** -40 * beta * ((size * share)[::2] + (size * share)[1::2])
        lose, win = np.logaddexp(0, -h), np.logaddexp(0, h)
        up, down = 1 / (1 + np.exp(-h)), 1 / (1 + np.exp(h))
        loss = (1 - eps) * lose + (eps * win if eps > 0 else 0.0)
        slope = -(1 - eps) * down + eps * up
        coef = beta * np.stack([slope, -slope], 1).reshape(-1) * share
        t_coef = beta * np.repeat((dh + 12 * U) * ((1 - eps) * down + eps * up), 2) * share + 2.0 ** -120
    dl = np.ones(seqs // 2) if dloss is None else dloss.astype(np.float64)
    grad, t_grad = np.zeros(n), np.zeros(n)
    for b in range(seqs):
        t = np.arange(offsets[b], offsets[b + 1])
        t = t[mask[t] != 0] if mask is not None else t
        grad[t], t_grad[t] = coef[b] * dl[b // 2], abs(dl[b // 2]) * (t_coef[b] + U * abs(coef[b]))
    return {"loss": loss, "rewards": reward, "coef": coef, "dlogp": grad,
            "tol": {"loss": dh + 10 * U * (loss + 1), "rewards": 4 * U * np.abs(reward) + 2.0 ** -40 * beta * size * share,
                    "coef": t_coef, "dlogp": t_grad}}


def close(got, want, tol, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, what
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    inf = ~fine & ~np.isnan(want)
    assert np.array_equal(got[inf], want[inf]), f"{what}: infinities in other places"
    err = np.abs(got[fine] - want[fine]) - np.broadcast_to(tol, want.shape)[fine]
    assert err.size == 0 or err.max() <= 0, f"{what}: {int((err > 0).sum())} of {err.size} outside, worst by {err.max()!r}"


def ragged(parts, seed, total=None, empty=0.2):
    """Offsets of `parts` sequences, some of them empty."""
    r = synth.rng(seed, parts)
    n = r.integers(1, 40, parts) if total is None else np.maximum(1, (r.dirichlet(np.ones(parts)) * total).astype(int))
    n[r.random(parts) < empty] = 0
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
