"""Inputs and tolerances of the tests of the logits operators (token log-probs, top-k distillation).

Tolerances, from the kernels' arithmetic, with u = 2^-24 (half an ulp of fp32, relative):
  * A term exp(z_j - z_max) is ex2 of t = fma(x, c, -R), c = fl(scale fl(log2 e)): c is off by 2u relative, the fma
    by u, so t by 3u |t| (R = fl(max c) shifts every term alike), and ex2.approx by 2 ulp = 4u. With
    |t| ln 2 = z_max - z_j =: D_j the term is off by (3 D_j + 4) u relative, and the sum, weighted by the
    terms, by (3 E[D] + 4) u, E[D] = sum p_j D_j = entropy + z_max - lse. Adding up to V terms costs at
    most u per addition of a thread's chain and of the tree: a chain has at most V / 64 + 64 terms here
    (64 threads or more per row). Merging threads of different maxima is one more term of the same kind.
    S = (3 E[D] + 4 + V / 64 + 64) u bounds the relative error of sum exp.
  * lse = fma(R, ln 2, ln s): S + u (2 |z_max| + 4 |lse| + 2 |ln s|) <= S + 8 u (|z_max| + |lse|).
  * logp = t ln 2 - ln s: S + u (6 |D_t| + 2 |ln s| + |logp|) <= S + 8 u (|D_t| + ln s).
  * entropy = ln s - ln 2 (w / s), w = sum e t: w's error is at most (2 S + 4u) E[D] relative to s, so
    S (1 + 3 E[D]) + 8 u (E[D] + ln s).
  * gradients: p_j = ex2(x c - lse log2 e) is off by e_j = u (3 |z_j| + 3 |lse| + 8) + tol(lse) relative; a
    term p_j (alpha + beta (ln p_j + H)) by that times its parts' sizes plus the errors of ln p_j and of H;
    then half an ulp of the output's type. Below 2^-126 ex2 gives 0.
"""
import numpy as np

import synth

U = 2.0 ** -24
MASKED = -(2.0 ** 100)


def values(bits):
    """Logits [M, V] as float64, masked ones -inf."""
    x = synth.bf16_to_f32(bits) if bits.dtype == np.uint16 else bits
    x = x.astype(np.float64)
    return np.where(x <= MASKED, -np.inf, x)


def make(M, V, dtype, seed, spread=2.0, ld=None):
    """Logits of a language model's kind: a broad bulk and a few likely columns. bf16 bits or fp32 [M, ld]."""
    r = synth.rng(seed, M, V)
    x = (r.standard_normal((M, ld or V)) * spread - 1.0).astype(np.float32)
    n = min(V, 12)
    for m in range(M):
        x[m, r.choice(V, size=n, replace=False)] = (3.0 + 9.0 * r.random(n)).astype(np.float32)
    return synth.bf16_bits(x) if dtype == "bf16" else x


def set_value(x, idx, v):
    """x[idx] = v for bf16 bits or fp32 (v: -inf, NaN, or any float that bf16 holds)."""
    if x.dtype == np.uint16:
        x[idx] = np.float32(v).view(np.uint32) >> 16
    else:
        x[idx] = np.float32(v)


def teacher(M, k, V, seed, mass=0.9, pad=0):
    """ids [M, k] (all different within a row) and log-probs that hold `mass` of 1; the last `pad` entries of every
    second row are not there (-1)."""
    r = synth.rng(seed, M, k, 5)
    ids = np.stack([r.permutation(V)[:k] if k <= V else np.arange(k) % V for _ in range(M)]).astype(np.int32)
    raw = np.sort(r.standard_normal((M, k)) * 2.0, axis=1)[:, ::-1]
    l = (raw - np.log(np.exp(raw).sum(1, keepdims=True)) + np.log(mass)).astype(np.float32)
    if pad:
        ids[::2, k - pad:] = -1
    return ids, l


def row_tolerances(x, scale, lse, h):
    """(tol of lse, S, E[D], z_max, ln s) per row, from the definitions above."""
    z = values(x) * float(np.float32(scale))
    with np.errstate(invalid="ignore"):
        zmax = np.max(z, axis=1)
        ED = np.maximum(h + zmax - lse, 0.0)
        ln_s = np.maximum(lse - zmax, 0.0)
    V = x.shape[1]
    S = (3 * ED + 4 + V / 64 + 64) * U
    return S + 8 * U * (np.abs(zmax) + np.abs(lse)), S, ED, zmax, ln_s


def close(got, ref, tol, what):
    """got [..] within tol of ref where ref is finite, equal to it elsewhere (NaN with NaN)."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    tol = np.broadcast_to(tol, ref.shape)
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN in other places"
    inf = ~fine & ~np.isnan(ref)
    assert np.array_equal(got[inf], ref[inf]), f"{what}: infinities in other places"
    err = np.abs(got[fine] - ref[fine]) - tol[fine]
    assert np.all(err <= 0), f"{what}: {int((err > 0).sum())} of {err.size} outside, worst by {err.max()!r}"


def half_ulp(ref, dtype):
    """Half a step of the output's type at ref, relative 2^-9 (bf16: eps / 2 = 2^-8 at most) or 2^-24."""
    return np.abs(ref) * (2.0 ** -8 if dtype == "bf16" else U) + 2.0 ** -133


def grad_tolerance(x, scale, lse, h, tol_lse, dtype, ref, weight, slope, spike=0.0):
    """weight, slope [M]: |alpha| and |beta| of p (alpha + beta (ln p + H)), the latter 0 without an entropy term;
    spike [M, V]: the size of what is added at single columns (its own error and the addition's: 16 u)."""
    z = values(x) * float(np.float32(scale))
    with np.errstate(invalid="ignore", over="ignore"):
        lp = z - lse[:, None]
        p = np.where(z == -np.inf, 0.0, np.exp(lp))
        e = U * (3 * np.abs(z) + 3 * np.abs(lse)[:, None] + 8) + tol_lse[:, None]
        tol_h = tol_lse * (1 + 3 * h) + 8 * U * (np.abs(lse) + h)
        part = weight[:, None] + slope[:, None] * (np.abs(lp) + h[:, None])
        t = p * (e * part * 2 + slope[:, None] * (tol_h[:, None] + 4 * U * (np.abs(lp) + h[:, None])))
    s = float(np.float32(scale))
    t = np.where(z == -np.inf, 0.0, t) + (weight + 200 * slope)[:, None] * 2.0 ** -126
    return t * s * 1.01 + half_ulp(ref, dtype) + 4 * U * np.abs(ref) + 16 * U * s * spike
