"""The operators of a GRPO step around the NVFP4 KV cache and the log-probs as measured cases: inputs, plain forms
and the library's calls.

  kv_write    prompts' keys and values (rows of a fused projection, or apart) written into an NVFP4 cache at the given
              tensor scale, and the written rows read back as the values that the cache holds
  kv_read     rows of an NVFP4 cache as bf16 or fp32
  attention   one decode step of sequences that share prefixes: softmax(scale q K^T) V over the group's prefix cache
              and the sequence's own cache together
  policy      a clipped policy loss with a KL term over packed responses, and its gradient to the log-probs
  preference  a loss of paired log ratios over packed responses, and its gradient to the log-probs

A cache row of D elements is D/2 bytes of E2M1 codes (low nibble first) and D/16 E4M3 scale bytes, one to 16 elements,
under one fp32 scale g for all: value = E2M1 * E4M3 * g.
"""
import math
import random

import torch

own = False

NEG = float("-inf")
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one prompt's keys and values, a part of the fused projection's rows, at prefill (latency)
        {"name": "kv_write_one", "op": "kv_write", "B": 1, "T": 37, "Hkv": 4, "D": 128, "dtype": "bf16",
         "fused": 36, "shift": 0},
        # a chunk of eight prompts behind what their caches hold already
        {"name": "kv_write_prefill", "op": "kv_write", "B": 8, "T": 65536, "Hkv": 8, "D": 128, "dtype": "bf16",
         "fused": 56, "shift": 300},
        # sixteen long prefixes read back for an attention in bf16
        {"name": "kv_read_prefixes", "op": "kv_read", "B": 16, "T": 131072, "Hkv": 8, "D": 128, "dtype": "bf16",
         "shift": 0},
        # another head size and an odd number of heads, in fp32
        {"name": "kv_read_odd_f32", "op": "kv_read", "B": 5, "T": 4999, "Hkv": 3, "D": 80, "dtype": "f32", "shift": 77},
        # a decode step of one group of eight samples of a short prompt, the first tokens (latency)
        {"name": "attend_group", "op": "attention", "P": 1, "B": 8, "Hq": 28, "Hkv": 4, "prefix": 511, "own": 3,
         "loose": 0},
        # four prompts, sixteen samples each, in the middle of their responses
        {"name": "attend_64", "op": "attention", "P": 4, "B": 64, "Hq": 28, "Hkv": 4, "prefix": 4096, "own": 700,
         "loose": 0},
        # sixteen long prompts (documents), sixteen samples each
        {"name": "attend_256", "op": "attention", "P": 16, "B": 256, "Hq": 40, "Hkv": 8, "prefix": 16384, "own": 500,
         "loose": 0},
        # as many KV heads as query heads, groups of odd sizes, sequences without a prefix
        {"name": "attend_odd", "op": "attention", "P": 3, "B": 23, "Hq": 6, "Hkv": 6, "prefix": 3001, "own": 333,
         "loose": 2},
        # eight responses to one prompt, each sequence's mean (latency)
        {"name": "policy_group", "op": "policy", "B": 8, "n": 1843, "mode": 1, "ref": True, "weights": False,
         "mask": False, "per_token": False, "kl": 0.04, "low": 0.2, "high": 0.2, "dual": 0.0},
        # 64 prompts x 8 responses, the mean over all tokens, rectified weights, a mask, a reference policy
        {"name": "policy_4m", "op": "policy", "B": 512, "n": 4194304, "mode": 0, "ref": True, "weights": True,
         "mask": True, "per_token": False, "kl": 0.001, "low": 0.2, "high": 0.28, "dual": 3.0},
        # 33 pairs of short answers without a reference model, lengths normalised
        {"name": "preference_33", "op": "preference", "B": 33, "n": 10007, "ref": False, "mask": True, "mean": True,
         "beta": 2.0, "margin": 0.5, "smooth": 0.0},
        # a large batch of pairs against a reference model
        {"name": "preference_1024", "op": "preference", "B": 1024, "n": 2097152, "ref": True, "mask": True,
         "mean": False, "beta": 0.1, "margin": 0.0, "smooth": 0.1},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["kv_write", "kv_read", "attention", "attention", "policy", "preference"])
    if op in ("kv_write", "kv_read"):
        Hkv, D, dtype = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 80, 128, 128, 128]), rng.choice(["bf16", "bf16", "f32"])
        case = {"op": op, "B": rng.choice([1, 2, 3, 5, 8, 16]), "T": _log(rng, 17, 50000 if dtype == "bf16" else 30000),
                "Hkv": Hkv, "D": D, "dtype": dtype, "shift": rng.choice([0, 0, 1, 63, 300])}
        if op == "kv_write":
            case["fused"] = rng.choice([0, 4 * Hkv, 2 * Hkv + 5])
        return case
    if op == "attention":
        Hkv, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        P, per = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 5, 8, 16, 24])
        most = min(16384, 120000000 // (P * per * Hkv * group))  # no more products than the largest listed case
        return {"op": op, "P": P, "B": P * per, "Hq": Hkv * group, "Hkv": Hkv, "prefix": _log(rng, 1, most),
                "own": _log(rng, 1, 600), "loose": rng.choice([0, 0, 1])}
    if op == "policy":
        B = _log(rng, 1, 512)
        return {"op": op, "B": B, "n": B * _log(rng, 3, 8000), "mode": rng.choice([0, 1, 2]), "ref": rng.random() < 0.6,
                "weights": rng.random() < 0.5, "mask": rng.random() < 0.5, "per_token": rng.random() < 0.3,
                "kl": rng.choice([0.0, 0.001, 0.04]), "low": rng.choice([0.1, 0.2]), "high": rng.choice([0.2, 0.28]),
                "dual": rng.choice([0.0, 3.0])}
    B = _log(rng, 1, 1024)
    return {"op": op, "B": B, "n": 2 * B * _log(rng, 2, 1000), "ref": rng.random() < 0.7, "mask": rng.random() < 0.6,
            "mean": rng.random() < 0.3, "beta": rng.choice([0.1, 0.3, 2.0]), "margin": rng.choice([0.0, 0.5]),
            "smooth": rng.choice([0.0, 0.1])}


# ---- what a case's sequences look like: the same whatever the seed ---------------------------------


def _shares(total, parts, sigma, key):
    """`total` tokens over `parts` sequences, their lengths log-normal (zero among them)."""
    rng = random.Random(key)
    w = [math.exp(rng.gauss(0.0, sigma)) for _ in range(parts)]
    edges, run = [0], 0.0
    for x in w:
        run += x
        edges.append(min(total, int(total * run / sum(w))))
    edges[-1] = total
    return edges


def _lengths(mean, parts, cap, key):
    rng = random.Random(key)
    return [min(cap, max(0, int(mean * math.exp(rng.gauss(0.0, 0.5) - 0.125)))) for _ in range(parts)]


def _groups(case):
    """Sequences [offsets[p], offsets[p + 1]) share prefix p; the last `loose` ones share none. Groups of equal sizes,
    or, where sequences are loose, of odd ones."""
    P, B, loose = case["P"], case["B"], case["loose"]
    B = max(0, B - loose)
    if not loose:
        return [p * B // P for p in range(P + 1)]
    return _shares(B, P, 0.8, f"groups {P} {B}")


def _attention_lengths(case):
    P, B = case["P"], case["B"]
    prefix = _lengths(case["prefix"], P, case["prefix"], f"prefix {P} {case['prefix']}")
    prefix[0] = case["prefix"]
    return prefix, _lengths(case["own"], B, 2 * case["own"], f"own {B} {case['own']}")


# ---- inputs ------------------------------------------------------------------------------------------


def _cache_rows(shape, Hkv, D, spread, gen):
    """Random rows of a real cache: encodings of normal rows with a few strong channels, drawn from a pool."""
    dev = "cuda"
    chan = torch.exp(0.4 * torch.randn(Hkv, 1, D, generator=gen, device=dev))
    pool = torch.randn(Hkv, 2048, D, generator=gen, device=dev) * chan * spread
    g = (pool.abs().max() / 2688.0).reshape(1).contiguous()
    codes, scales = _encode(pool.reshape(-1, D), g)
    n = shape[0] * shape[1]
    out = (torch.empty(n, Hkv, D // 2, dtype=torch.uint8, device=dev),
           torch.empty(n, Hkv, D // 16, dtype=torch.uint8, device=dev))
    base = (torch.arange(Hkv, device=dev) * 2048)[None]
    for a in range(0, n, 1 << 16):
        m = min(1 << 16, n - a)
        at = base + torch.randint(0, 2048, (m, Hkv), generator=gen, device=dev)
        out[0][a:a + m] = codes[at]
        out[1][a:a + m] = scales[at]
    return out[0].view(*shape, Hkv, D // 2), out[1].view(*shape, Hkv, D // 16), g


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    st = {"case": dict(case)}
    dev_ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    randn = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    op = case["op"]
    if op in ("kv_write", "kv_read"):
        B, T, Hkv, D = case["B"], case["T"], case["Hkv"], case["D"]
        edges = _shares(T, B, 0.4, f"tokens {T} {B}")
        longest = max(b - a for a, b in zip(edges, edges[1:]))
        st.update(edges=edges, offsets=dev_ints(edges), Lmax=longest + case["shift"] + 5,
                  pos=dev_ints([case["shift"]] * B))
        if op == "kv_read":
            st["kc"], st["ks"], st["gk"] = _cache_rows((B, st["Lmax"]), Hkv, D, 1.0, gen)
            st["vc"], st["vs"], st["gv"] = _cache_rows((B, st["Lmax"]), Hkv, D, 0.5, gen)
            return st
        dt = TYPES[case["dtype"]]
        if case["fused"]:  # [queries | keys | values] of a token in one row
            rows = torch.empty(T, case["fused"], D, dtype=dt, device=dev)
            for a in range(0, T, 8192):
                rows[a:a + 8192] = randn(min(8192, T - a), case["fused"], D).to(dt)
            st["k"], st["v"] = rows[:, -2 * Hkv:-Hkv], rows[:, -Hkv:]
        else:
            st["k"], st["v"] = randn(T, Hkv, D).to(dt), randn(T, Hkv, D).to(dt)
        st["k"].mul_(torch.exp(0.4 * randn(Hkv, D)).to(dt))
        # calibrated scales of the layer
        st["gk"], st["gv"] = (torch.full((1,), s / 2688.0, device=dev) for s in (16.0, 4.5))
        for n, w in (("kc", 2), ("ks", 16), ("vc", 2), ("vs", 16)):
            st[n] = torch.zeros(B, st["Lmax"], Hkv, D // w, dtype=torch.uint8, device=dev)
        return st
    if op == "attention":
        P, B, Hq, Hkv = case["P"], case["B"], case["Hq"], case["Hkv"]
        prefix, lens = _attention_lengths(case)
        groups = _groups(case)
        st.update(prefix=prefix, lens=lens, groups=groups, prefix_lens=dev_ints(prefix), own_lens=dev_ints(lens),
                  offsets=dev_ints(groups), scale=1.0 / math.sqrt(128.0))
        st["q"] = (randn(B, Hq, 128) * 1.5).to(torch.bfloat16)
        st["pkc"], st["pks"], st["gk"] = _cache_rows((P, case["prefix"]), Hkv, 128, 1.0, gen)
        st["pvc"], st["pvs"], st["gv"] = _cache_rows((P, case["prefix"]), Hkv, 128, 0.5, gen)
        st["kc"], st["ks"], _ = _cache_rows((B, 2 * case["own"]), Hkv, 128, 1.0, gen)
        st["vc"], st["vs"], _ = _cache_rows((B, 2 * case["own"]), Hkv, 128, 0.5, gen)
        return st
    n, B = case["n"], case["B"]
    rand = lambda *s: torch.rand(*s, generator=gen, device=dev)  # noqa: E731
    seqs = B if op == "policy" else 2 * B
    edges = _shares(n, seqs, 0.6, f"responses {n} {seqs}")
    st.update(edges=edges, offsets=dev_ints(edges))
    st["seq"] = torch.repeat_interleave(torch.arange(seqs, device=dev), dev_ints(edges).diff().long(), output_size=n)
    # a sampled token's log-prob: often near 0, now and then far below
    base = torch.log(rand(n).clamp_min(1e-6)) * rand(n) ** 2
    st["logp"] = (base + 0.1 * randn(n)).clamp_max(0.0)
    if case["mask"]:
        st["mask"] = rand(n) < 0.9
        if op == "policy":  # what a masked position holds is not looked at
            st["logp"] = torch.where(st["mask"] | (rand(n) < 0.5), st["logp"], NEG)
    if case["ref"]:
        st["ref"] = (base + 0.1 * randn(n)).clamp_max(0.0)
    if op == "policy":
        st["old"] = base
        if case["weights"]:
            st["weights"] = 0.5 + rand(n)
        st["adv"] = randn(n if case["per_token"] else B)
        st["dloss"] = torch.full((1,), 0.5, device=dev)  # one of two micro-batches
    else:
        st["dloss"] = torch.full((B,), 1.0 / B, device=dev)
    return st


# ---- the plain forms -----------------------------------------------------------------------------------


def _e4m3_table(dev):
    """The 127 values of the non-negative E4M3 bytes, in fp64."""
    b = torch.arange(127, device=dev)
    e, m = (b >> 3).double(), (b & 7).double()
    return torch.where(e == 0, m * 2.0 ** -9, (1.0 + m / 8.0) * torch.exp2(e - 7.0))


def _nearest(t, table):
    """Index of the nearest entry of a rising table, ties to the even index, in 64 bits."""
    mids = (table[1:] + table[:-1]) / 2
    i = torch.bucketize(t, mids)  # how many midpoints lie below t
    tie = (i < len(mids)) & (t == mids[i.clamp_max(len(mids) - 1)])
    return torch.where(tie & (i % 2 == 1), i + 1, i)


def _encode(x, g):
    """Rows [n, D] -> codes [n, D/2], scale bytes [n, D/16] under the scale g."""
    n, D = x.shape
    blocks = x.double().reshape(n, D // 16, 16)
    g = g.double()
    table = _e4m3_table(x.device)
    byte = _nearest(blocks.abs().amax(2) / (6.0 * g), table)
    d = (table[byte] * g)[..., None]
    a = torch.where(d > 0, blocks.abs() / torch.where(d > 0, d, 1.0), 0.0)
    code = _nearest(a, torch.tensor(GRID, dtype=torch.float64, device=x.device))
    code = (code + torch.where(torch.signbit(blocks), 8, 0)).reshape(n, D).to(torch.uint8)
    return code[:, ::2] | (code[:, 1::2] << 4), byte.to(torch.uint8)


def _decode(codes, scales, g):
    """Codes [..., D/2], scale bytes [..., D/16] -> values [..., D] in fp32, rounded once."""
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    s = _e4m3_table(codes.device).float()[scales.long().clamp_max(126)]
    v = grid[nib.long()].unflatten(-1, (-1, 16)) * s[..., None]  # exact: six significant bits
    return (v * g).flatten(-2)


def _ragged(st, cache, g, cols, dt):
    """The cached rows of every sequence's tokens as [T, Hkv, D]."""
    case, parts = st["case"], []
    codes, scales = cache
    for b, (a, e) in enumerate(zip(st["edges"], st["edges"][1:])):
        rows = slice(case["shift"], case["shift"] + e - a)
        for c in range(rows.start, rows.stop, 16384):
            r = slice(c, min(c + 16384, rows.stop))
            parts.append(_decode(codes[b, r], scales[b, r], g).to(dt))
    return torch.cat(parts) if parts else torch.empty(0, case["Hkv"], cols, dtype=dt, device=codes.device)


def _kv_read(st):
    dt, D = TYPES[st["case"]["dtype"]], st["case"]["D"]
    return {"k": _ragged(st, (st["kc"], st["ks"]), st["gk"], D, dt),
            "v": _ragged(st, (st["vc"], st["vs"]), st["gv"], D, dt)}


def _kv_write(st):
    Hkv, D, shift = st["case"]["Hkv"], st["case"]["D"], st["case"]["shift"]
    for x, codes, scales, g in ((st["k"], st["kc"], st["ks"], st["gk"]), (st["v"], st["vc"], st["vs"], st["gv"])):
        for b, (a, e) in enumerate(zip(st["edges"], st["edges"][1:])):
            for c in range(a, e, 8192):
                m = min(8192, e - c)
                q, s = _encode(x[c:c + m].reshape(m * Hkv, D), g)
                at = shift + c - a
                codes[b, at:at + m] = q.view(m, Hkv, D // 2)
                scales[b, at:at + m] = s.view(m, Hkv, D // 16)
    return _kv_read(st)


def _attention(st):
    case = st["case"]
    B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
    r = Hq // Hkv
    q = st["q"].float().view(B, Hkv, r, 128) * st["scale"]
    top = torch.full((B, Hkv, r, 1), NEG, device=q.device)
    total, acc = torch.zeros_like(top), torch.zeros(B, Hkv, r, 128, device=q.device)

    def add(rows, s, values):
        """Scores s [m, Hkv, r, L] and values [Hkv, L, 128] or [m, Hkv, L, 128] into the rows' running softmax."""
        if s.shape[-1] == 0:
            return
        m = torch.maximum(top[rows], s.amax(-1, keepdim=True))
        ref = torch.where(m == NEG, 0.0, m)
        p, keep = torch.exp(s - ref), torch.exp(top[rows] - ref)
        total[rows] = total[rows] * keep + p.sum(-1, keepdim=True)
        if values.dim() == 3:
            new = torch.matmul(p.transpose(0, 1).flatten(1, 2), values).unflatten(1, (-1, r)).transpose(0, 1)
        else:
            new = torch.matmul(p, values)
        acc[rows] = acc[rows] * keep + new
        top[rows] = m

    for p, (a, e) in enumerate(zip(st["groups"], st["groups"][1:])):
        if e == a:
            continue
        rows = slice(a, e)
        for c in range(0, st["prefix"][p], 8192):
            at = slice(c, min(c + 8192, st["prefix"][p]))
            k = _decode(st["pkc"][p, at], st["pks"][p, at], st["gk"]).transpose(0, 1)
            v = _decode(st["pvc"][p, at], st["pvs"][p, at], st["gv"]).transpose(0, 1)
            s = torch.matmul(q[rows].transpose(0, 1).flatten(1, 2), k.transpose(1, 2))
            add(rows, s.unflatten(1, (-1, r)).transpose(0, 1), v)
    longest = max(st["lens"])
    for a in range(0, B, 32):
        rows = slice(a, min(a + 32, B))
        k = _decode(st["kc"][rows, :longest], st["ks"][rows, :longest], st["gk"]).transpose(1, 2)
        v = _decode(st["vc"][rows, :longest], st["vs"][rows, :longest], st["gv"]).transpose(1, 2)
        s = torch.matmul(q[rows], k.transpose(2, 3))
        out = torch.arange(longest, device=q.device) >= st["own_lens"][rows, None, None, None]
        add(rows, s.masked_fill(out, NEG), v)
    o = torch.where(total > 0, acc / torch.where(total > 0, total, 1.0), 0.0)
    return {"out": o.view(B, Hq, 128).to(torch.bfloat16)}


def _bounds(case):
    """The bounds of the ratio, from the fp32 numbers that a call takes."""
    f = lambda v: torch.tensor(v, dtype=torch.float32).item()  # noqa: E731
    return 1.0 - f(case["low"]), 1.0 + f(case["high"]), f(case["dual"]), f(case["kl"])


def _policy(st):
    """In 64 bits up to the sums: a ratio next to a bound, and e^x - x - 1 of small x, need them."""
    case = st["case"]
    lo, hi, dual, kl = _bounds(case)
    B, n, seq = case["B"], case["n"], st["seq"]
    live = st["mask"] if case["mask"] else torch.ones(n, dtype=torch.bool, device=seq.device)
    m = live.double()
    lp = torch.where(live, st["logp"], 0.0).double()
    d = lp - torch.where(live, st["old"], 0.0).double()
    adv = (st["adv"] if case["per_token"] else st["adv"][seq]).double()
    w = st["weights"].double() if case["weights"] else 1.0
    r = torch.exp(d)
    full, cut = r * adv, r.clamp(lo, hi) * adv
    gain = torch.minimum(full, cut)
    free = full <= cut
    clipped = full > cut
    if dual:
        capped = (adv < 0) & (gain < dual * adv)
        gain = torch.where(capped, dual * adv, gain)
        free, clipped = free & ~capped, clipped | capped
    part, grad = -w * gain, torch.where(free, -w * full, 0.0)
    if case["ref"]:
        x = torch.where(live, st["ref"], 0.0).double() - lp
        k3 = torch.exp(x) - x - 1.0
        grad = grad + kl * (1.0 - torch.exp(x))
    else:
        k3 = torch.zeros_like(d)
    tokens = m.sum()
    per = torch.zeros(B, dtype=torch.float64, device=seq.device).index_add_(0, seq, m)
    there = (per > 0).sum()
    if case["mode"] == 0:
        coef = (1.0 / tokens.clamp_min(1.0)).expand(B)
    elif case["mode"] == 1:
        coef = 1.0 / (per.clamp_min(1.0) * there.clamp_min(1))
    else:
        coef = torch.full((B,), 1.0 / n, dtype=torch.float64, device=seq.device)
    c = m * coef[seq]
    mean = lambda v: (m * v).sum() / tokens.clamp_min(1.0)  # noqa: E731
    pol, div = (c * part).sum(), (c * k3).sum()
    loss = pol + kl * div if case["ref"] else pol
    stats = torch.stack([loss, pol, div, mean(clipped.double()), mean(r - 1.0 - d), mean(r), tokens, there.double()])
    return {"loss": loss.reshape(1).float(), "stats": stats.float(), "dlogp": (st["dloss"].double() * c * grad).float()}


def _preference(st):
    case = st["case"]
    B, n, seq = case["B"], case["n"], st["seq"]
    f = lambda v: torch.tensor(v, dtype=torch.float32).item()  # noqa: E731
    beta, margin, smooth = f(case["beta"]), f(case["margin"]), f(case["smooth"])
    m = st["mask"].double() if case["mask"] else torch.ones(n, dtype=torch.float64, device=seq.device)
    x = st["logp"].double() - (st["ref"].double() if case["ref"] else 0.0)
    zeros = torch.zeros(2 * B, dtype=torch.float64, device=seq.device)
    total, count = zeros.index_add(0, seq, m * x), zeros.index_add(0, seq, m)
    share = 1.0 / count.clamp_min(1.0) if case["mean"] else torch.ones_like(count)
    reward = beta * total * share
    h = reward[::2] - reward[1::2] - margin
    soft = lambda t: t.clamp_min(0.0) + torch.log1p(torch.exp(-t.abs()))  # noqa: E731  ln(1 + e^t)
    loss = (1.0 - smooth) * soft(-h) + smooth * soft(h)
    slope = 1.0 / (1.0 + torch.exp(-h)) - (1.0 - smooth)
    coef = beta * torch.stack([slope, -slope], 1).flatten() * share
    grad = m * (coef * st["dloss"].double().repeat_interleave(2))[seq]
    return {"loss": loss.float(), "rewards": reward.float(), "dlogp": grad.float()}


PLAIN = {"kv_write": _kv_write, "kv_read": _kv_read, "attention": _attention, "policy": _policy,
         "preference": _preference}


def _calls(st):
    """The library's calls on the same state."""
    import nvfp4_quantized_rl_gb300 as nv
    case, op = st["case"], st["case"]["op"]
    if op in ("kv_write", "kv_read"):
        if op == "kv_write":
            nv.nvfp4_kv_append_ragged(st["k"], st["v"], st["offsets"], st["pos"], st["gk"], st["gv"], st["kc"],
                                      st["ks"], st["vc"], st["vs"])
        k, v = nv.nvfp4_kv_read(st["kc"], st["ks"], st["gk"], st["vc"], st["vs"], st["gv"], st["offsets"], st["pos"],
                                case["T"], dtype=TYPES[case["dtype"]])
        return {"k": k, "v": v}
    if op == "attention":
        return {"out": nv.nvfp4_kv_prefix_attention(
            st["q"], st["pkc"], st["pks"], st["pvc"], st["pvs"], st["prefix_lens"], st["offsets"], st["kc"], st["ks"],
            st["vc"], st["vs"], st["own_lens"], st["gk"], st["gv"], st["scale"])}
    if op == "policy":
        terms = dict(logp_ref=st.get("ref"), weights=st.get("weights"), mask=st.get("mask"), eps_low=case["low"],
                     eps_high=case["high"], dual_clip=case["dual"], kl_coef=case["kl"],
                     adv_per_token=case["per_token"])
        loss, stats, coef = nv.policy_loss(st["logp"], st["old"], st["adv"], st["offsets"], mode=case["mode"],
                                           norm=float(case["n"]), **terms)
        dlogp = nv.policy_loss_backward(st["logp"], st["old"], st["adv"], st["offsets"], coef, st["dloss"], **terms)
        return {"loss": loss, "stats": stats, "dlogp": dlogp}
    loss, rewards, coef = nv.preference_loss(st["logp"], st["offsets"], logp_ref=st.get("ref"), mask=st.get("mask"),
                                             beta=case["beta"], margin=case["margin"], smoothing=case["smooth"],
                                             mean=case["mean"])
    return {"loss": loss, "rewards": rewards,
            "dlogp": nv.preference_loss_backward(st["offsets"], coef, st["dloss"], case["n"], mask=st.get("mask"))}


def run(state):
    if own:
        return _calls(state)
    return PLAIN[state["case"]["op"]](state)


def work(case):
    op = case["op"]
    if op in ("kv_write", "kv_read"):
        elements = 2 * case["T"] * case["Hkv"] * case["D"]
        b = 2 if case["dtype"] == "bf16" else 4
        if op == "kv_read":
            return {"bytes": elements * (b + 9 / 16), "flops": elements * 2}
        return {"bytes": elements * (2 * b + 9 / 16), "flops": elements * 5}  # rows in, cache and values out
    if op == "attention":
        prefix, lens = _attention_lengths(case)
        groups = _groups(case)
        sizes = [b - a for a, b in zip(groups, groups[1:])]
        read = sum(l for l, s in zip(prefix, sizes) if s) + sum(lens)
        pairs = sum(l * s for l, s in zip(prefix, sizes)) + sum(lens)
        return {"bytes": read * case["Hkv"] * 144 + 4 * case["B"] * case["Hq"] * 128,
                "flops": 4 * 128 * case["Hq"] * pairs}
    n = case["n"]
    if op == "policy":
        arrays = 2 + case["ref"] + case["weights"] + case["per_token"]
        return {"bytes": n * (4 * arrays + case["mask"] + 4) + 12 * case["B"], "flops": n * 30}
    return {"bytes": n * (4 * (1 + case["ref"]) + case["mask"] + 4) + 24 * case["B"], "flops": n * 6}


# ---- the definitions in 64 bits --------------------------------------------------------------------------


def _round_to(a, least, digits, most):
    """|a| to a binary float of `digits` bits behind the leading one, exponents from `least`, ties to even."""
    e = torch.frexp(a.clamp_min(2.0 ** -200)).exponent.double() - 1.0
    step = torch.exp2(torch.clamp_min(e, least) - digits)
    return (torch.round(a / step) * step).clamp_max(most)


def _values(st, which):
    """What a write of these rows leaves in the cache, block by block."""
    x, g = st[which].double(), st["g" + which].double()
    T, H, D = x.shape
    x = x.reshape(T, H, D // 16, 16)
    s = _round_to(x.abs().amax(-1, keepdim=True) / (6.0 * g), -6.0, 3.0, 448.0) * g
    near = _round_to((x / torch.where(s == 0, 1.0, s)).abs(), 0.0, 1.0, 6.0)
    return (torch.where(s == 0, 0.0, near * s) * torch.sign(x)).reshape(T, H, D)


def _held(codes, scales, g):
    """Values of cache rows: sign, two exponent bits and one of mantissa; four and three of the scales."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    e, m = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e == 0, m / 2, torch.ldexp(1.0 + m / 2, e - 1)) * (1.0 - 2.0 * (c >> 3).double())
    b = scales.long()
    e, m = b >> 3, (b & 7).double()
    s = torch.where(e == 0, torch.ldexp(m, torch.full_like(e, -9)), torch.ldexp(1.0 + m / 8, e - 7))
    return v * s.repeat_interleave(16, -1) * g.double()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "kv_write":
        return {"k": _values(st, "k"), "v": _values(st, "v")}
    if op == "kv_read":
        seq = torch.searchsorted(st["offsets"][1:].long(), torch.arange(case["T"], device="cuda"), right=True)
        row = torch.arange(case["T"], device="cuda") - st["offsets"].long()[seq] + case["shift"]
        out = {}
        for n in "kv":
            out[n] = torch.cat([_held(st[n + "c"][s, r], st[n + "s"][s, r], st["g" + n])
                                for s, r in zip(seq.split(8192), row.split(8192))])
        return out
    if op == "attention":
        outs, group, r = [], -1, case["Hq"] // case["Hkv"]
        of = {b: p for p, (a, e) in enumerate(zip(st["groups"], st["groups"][1:])) for b in range(a, e)}
        for b in range(case["B"]):
            if of.get(b) != group:
                group, k0, v0 = of.get(b), None, None
                if group is not None:
                    L = st["prefix"][group]
                    k0 = _held(st["pkc"][group, :L], st["pks"][group, :L], st["gk"])
                    v0 = _held(st["pvc"][group, :L], st["pvs"][group, :L], st["gv"])
            L = st["lens"][b]
            k, v = _held(st["kc"][b, :L], st["ks"][b, :L], st["gk"]), _held(st["vc"][b, :L], st["vs"][b, :L], st["gv"])
            if k0 is not None:
                k, v = torch.cat([k0, k]), torch.cat([v0, v])
            if len(k) == 0:
                outs.append(torch.zeros(case["Hq"], 128, dtype=torch.float64, device="cuda"))
                continue
            q = st["q"][b].double().view(case["Hkv"], r, 128)
            p = torch.softmax(torch.bmm(q, k.permute(1, 2, 0)) * st["scale"], -1)
            outs.append(torch.bmm(p, v.transpose(0, 1)).flatten(0, 1))
        return {"out": torch.stack(outs)}
    # sequence by sequence, from differences of running sums over the counted tokens
    keep = st["mask"] if case["mask"] else torch.ones(case["n"], dtype=torch.bool, device="cuda")
    idx = keep.nonzero()[:, 0]
    off = st["offsets"].long()
    ends = torch.searchsorted(idx, off)
    seq = st["seq"][idx]
    counts = ends.diff().double()

    def by_sequence(v):
        run = torch.cat([torch.zeros(1, dtype=torch.float64, device="cuda"), v.cumsum(0)])
        return run[ends[1:]] - run[ends[:-1]]
    dlogp = torch.zeros(case["n"], dtype=torch.float64, device="cuda")
    lp = st["logp"][idx].double()
    f32 = lambda v: torch.tensor(v, dtype=torch.float32).double().item()  # noqa: E731
    if op == "preference":
        ratio = lp - st["ref"][idx].double() if case["ref"] else lp
        length = counts.clamp_min(1.0) if case["mean"] else torch.ones_like(counts)
        reward = f32(case["beta"]) * by_sequence(ratio) / length
        pairs = reward.view(-1, 2)
        h = pairs[:, 0] - pairs[:, 1] - f32(case["margin"])
        eps = f32(case["smooth"])
        ls = torch.nn.functional.logsigmoid
        loss = -(1 - eps) * ls(h) - eps * ls(-h)
        dh = (eps * torch.sigmoid(h) - (1 - eps) * torch.sigmoid(-h)) * st["dloss"].double()
        each = torch.stack([dh, -dh], 1).view(-1) * f32(case["beta"]) / length
        dlogp[idx] = each[seq]
        return {"loss": loss, "rewards": reward, "dlogp": dlogp}
    low, high, dual, kl = f32(case["low"]), f32(case["high"]), f32(case["dual"]), f32(case["kl"])
    d = lp - st["old"][idx].double()
    A = (st["adv"][idx] if case["per_token"] else st["adv"][seq]).double()
    w = st["weights"][idx].double() if case["weights"] else torch.ones_like(d)
    ratio = d.exp()
    # clipping acts above the upper bound where the advantage is positive, below the lower one where it is negative
    over = (A > 0) & (ratio > 1 + high)
    under = (A < 0) & (ratio < 1 - low)
    used = torch.where(over, 1 + high, torch.where(under, 1 - low, ratio))
    stop = over | under
    if dual:
        far = (A < 0) & (ratio > dual)
        used, stop = torch.where(far, dual, used), stop | far
    policy = -w * used * A
    slope = torch.where(stop, 0.0, policy)
    div = torch.zeros_like(d)
    if case["ref"]:
        x = st["ref"][idx].double() - lp
        div = torch.expm1(x) - x
        slope = slope - kl * torch.expm1(x)
    tokens, there = counts.sum(), (counts > 0).sum().double()
    if case["mode"] == 0:
        coef = torch.ones_like(counts) / tokens.clamp_min(1)
    elif case["mode"] == 1:
        coef = torch.where(counts > 0, 1 / (counts.clamp_min(1) * there.clamp_min(1)), 0.0)
    else:
        coef = torch.ones_like(counts) / case["n"]
    pol, klv = (coef * by_sequence(policy)).sum(), (coef * by_sequence(div)).sum()
    loss = pol + (kl * klv if case["ref"] else 0.0)
    dlogp[idx] = st["dloss"].double() * coef[seq] * slope
    mean = lambda v: v.sum() / tokens.clamp_min(1)  # noqa: E731
    stats = torch.stack([loss, pol, klv, mean(stop.double()), mean(torch.expm1(d) - d), mean(ratio), tokens, there])
    return {"loss": loss.reshape(1), "stats": stats, "dlogp": dlogp}
