"""The log-probability and distillation operators as measured cases: inputs, plain forms and the library's calls.

The four operators work on logits x [M, V] (bf16 or fp32, V contiguous, rows `ld` elements apart) with z = scale x and
p = softmax(z). A logit at or below -2^100 is masked (p = 0).
  logprobs            a given token's log-prob, the entropy and the log-sum-exp of each row, and its k largest logits
                      (ties to the lower index) as (id, log-prob); a row whose token is outside [0, V) is ignored
  logprobs_backward   the gradient of sum(dlogp logp) + sum(dentropy entropy) to the logits
  distill             KL(q || p) against a teacher's k listed log-probs: q normalised over the list, or with everything
                      unlisted as one more bucket (tail)
  distill_backward    the gradient of sum(dloss loss) to the logits
"""
import math

import torch

own = False

MASKED = -(2.0 ** 100)
NEG = float("-inf")
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decode step of one sequence: the sampled token's log-prob and 20 alternatives (latency)
        {"name": "rollout_one", "op": "logprobs", "M": 1, "V": 152064, "ld": 152064, "dtype": "bf16", "k": 20,
         "entropy": True, "scale": 1.0, "pad": 0.0},
        # a decode step of the 64-sequence rollout batch, sampled at temperature 0.8
        {"name": "rollout_64", "op": "logprobs", "M": 64, "V": 152064, "ld": 152064, "dtype": "bf16", "k": 5,
         "entropy": True, "scale": 1.25, "pad": 0.0},
        # the trainer's log-probs of a packed batch of 8192 tokens (no alternatives)
        {"name": "train_8192", "op": "logprobs", "M": 8192, "V": 152064, "ld": 152064, "dtype": "bf16", "k": 0,
         "entropy": True, "scale": 1.0, "pad": 0.0},
        # a teacher's 64 top log-probs per position, the vocabulary's odd real size inside its padded rows
        {"name": "teacher_top64", "op": "logprobs", "M": 2048, "V": 151665, "ld": 152064, "dtype": "bf16", "k": 64,
         "entropy": False, "scale": 1.0, "pad": 0.0},
        # the policy gradient with an entropy bonus over a padded batch (an eighth of it prompt tokens)
        {"name": "train_backward_4096", "op": "logprobs_backward", "M": 4096, "V": 152064, "ld": 152064,
         "dtype": "bf16", "entropy": True, "scale": 1.0, "pad": 0.125},
        # fp32 logits of an odd vocabulary: every row starts at another alignment
        {"name": "odd_backward_f32", "op": "logprobs_backward", "M": 257, "V": 50257, "ld": 50257, "dtype": "f32",
         "entropy": False, "scale": 0.7, "pad": 0.0},
        # a few tokens
        {"name": "few_backward", "op": "logprobs_backward", "M": 8, "V": 32000, "ld": 32000, "dtype": "bf16",
         "entropy": True, "scale": 1.0, "pad": 0.0},
        # a small distillation batch in fp32, teacher renormalised over its list
        {"name": "distill_16_f32", "op": "distill", "M": 16, "V": 32000, "ld": 32000, "dtype": "f32", "k": 32,
         "tail": False, "scale": 1.0, "pad": 0.0},
        # a distillation step at full vocabulary with the tail bucket
        {"name": "distill_4096", "op": "distill", "M": 4096, "V": 152064, "ld": 152064, "dtype": "bf16", "k": 64,
         "tail": True, "scale": 1.0, "pad": 0.0},
        {"name": "distill_backward_4096", "op": "distill_backward", "M": 4096, "V": 152064, "ld": 152064,
         "dtype": "bf16", "k": 64, "tail": True, "scale": 1.0, "pad": 0.0},
        # fp32, odd vocabulary, long lists, a softened student, a quarter of the rows without a teacher
        {"name": "distill_odd_backward_f32", "op": "distill_backward", "M": 100, "V": 128257, "ld": 128257,
         "dtype": "f32", "k": 128, "tail": False, "scale": 0.5, "pad": 0.25},
    ]


def draw(rng):
    op = rng.choice(["logprobs", "logprobs_backward", "distill", "distill_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    V = int(round(math.exp(rng.uniform(math.log(1000), math.log(152064)))))
    V = min(152064, max(1000, V | 1 if rng.random() < 0.5 else (V + 127) // 128 * 128))
    most = 4096 if dtype == "bf16" else 2048
    M = max(1, min(most, int(math.exp(rng.uniform(0.0, math.log(most + 0.5))))))
    case = {"op": op, "M": M, "V": V, "ld": V if rng.random() < 0.6 else V + rng.randrange(1, 200), "dtype": dtype,
            "scale": rng.choice([1.0, 1.0, 0.5, 0.7, 1.25, 2.0]), "pad": rng.choice([0.0, 0.0, 0.1, 0.25])}
    if op == "logprobs":
        case.update(k=rng.choice([0, 1, 2, 5, 8, 20, 33, 64, 100, 128]), entropy=rng.random() < 0.6)
    elif op == "logprobs_backward":
        case.update(entropy=rng.random() < 0.6)
    if op.startswith("logprobs"):
        case["masked"] = rng.choice([0.0, 0.0, 0.0, 0.95])
    else:
        case.update(k=rng.choice([1, 4, 10, 20, 32, 50, 64, 100, 128]), tail=rng.random() < 0.5)
    return case


def _ignored(case):
    return int(case["M"] * case["pad"])


def prepare(case, seed):
    M, V, ld, dev = case["M"], case["V"], case["ld"], "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    rand = lambda *s: torch.rand(*s, generator=g, device=dev)  # noqa: E731
    randint = lambda n, *s: (rand(*s).double() * n).long().clamp_(0, n - 1)  # noqa: E731
    dt = TYPES[case["dtype"]]
    # a language model's logits: a broad bulk, and 40 likely tokens that stand out of it
    buf = torch.empty(M, ld, dtype=dt, device=dev)
    for a in range(0, M, 1024):
        part = torch.randn(min(1024, M - a), ld, generator=g, device=dev) * 2.0 - 1.0
        buf[a:a + 1024] = part.to(dt)
    x = buf[:, :V]
    step = V // 131
    hot = (randint(V, M, 1) + torch.arange(40, device=dev) * 3 * step) % V  # 40 different columns of a row
    if case.get("masked"):  # constrained decoding: most of the vocabulary is not allowed
        for a in range(0, M, 1024):
            x[a:a + 1024].masked_fill_(rand(min(1024, M - a), V) < case["masked"], NEG)
    x.scatter_(1, hot, (6.0 + 10.0 * rand(M, 40) ** 2).to(dt))
    st = {"case": dict(case), "x": x, "scale": float(case["scale"])}
    skip = torch.zeros(M, dtype=torch.bool, device=dev)
    skip[torch.randperm(M, generator=g, device=dev)[:_ignored(case)]] = True
    if case["op"].startswith("logprobs"):
        tok = torch.where(rand(M) < (1.0 if case.get("masked") else 0.8), hot.gather(1, randint(40, M, 1))[:, 0], randint(V, M))
        st["tokens"] = tok.masked_fill(skip, -100).to(torch.int32)
    else:
        k = case["k"]
        # the teacher lists likely tokens of the student's and others, all different within a row
        ids = (hot[:, :1] + torch.arange(k, device=dev) * step) % V
        st["ids"] = ids.masked_fill(skip[:, None], -1).to(torch.int32)
        raw = torch.sort(torch.randn(M, k + 1, generator=g, device=dev).double() * 2.0, dim=1, descending=True).values
        st["teacher_logp"] = (raw - raw.logsumexp(1, keepdim=True))[:, :k].float().contiguous()
    if case["op"].endswith("backward"):
        # what a training step has from its forward call, and the gradient that arrives
        st["grad"] = torch.randn(M, generator=g, device=dev) / M
        lse, ent, tail = (torch.zeros(M, device=dev) for _ in range(3))
        for a in range(0, M, 512):
            z = x[a:a + 512].double() * st["scale"]
            lz = z.logsumexp(1)
            lse[a:a + 512] = lz.float()
            if case.get("entropy"):
                ent[a:a + 512] = (lz - (torch.exp(z - lz[:, None]) * z.clamp_min(MASKED)).sum(1)).float()
            if case.get("tail"):
                tail[a:a + 512] = z.scatter(1, ids[a:a + 512], NEG).logsumexp(1).float()
        st["lse"] = lse.masked_fill(skip, 0.0)
        if case.get("entropy"):
            st["entropy"] = ent.masked_fill(skip, 0.0)
            st["dentropy"] = torch.randn(M, generator=g, device=dev) * (0.01 / M)
        if case.get("tail"):
            st["lse_tail"] = tail.masked_fill(skip, 0.0)
    return st


# ---- the plain forms ------------------------------------------------------------------------------


def _z(x, scale):
    """scale x in fp32, masked logits at -inf."""
    f = x.float()
    return torch.where(f <= MASKED, NEG, f * scale)


def _lse(z):
    top = z.max(1).values
    ref = torch.where(top == NEG, 0.0, top)
    return ref + torch.log(torch.exp(z - ref[:, None]).sum(1))


def _logprobs(st):
    x, k, V = st["x"], st["case"]["k"], st["case"]["V"]
    tok = st["tokens"].long()
    live = (tok >= 0) & (tok < V)
    z = _z(x, st["scale"])
    lse = _lse(z)
    logp = z.gather(1, torch.where(live, tok, 0)[:, None])[:, 0] - lse
    out = {"logp": torch.where(live, logp, 0.0), "lse": torch.where(live, lse, 0.0)}
    if st["case"]["entropy"]:
        lp = z - lse[:, None]
        h = -torch.where(lp == NEG, 0.0, torch.exp(lp) * lp).sum(1)
        out["entropy"] = torch.where(live, h, 0.0)
    if k:
        v, i = torch.sort(x.float(), dim=1, descending=True, stable=True)
        i, lp = i[:, :k], v[:, :k] * st["scale"] - lse[:, None]
        there = (v[:, :k] > MASKED) & live[:, None]
        out["top_ids"] = torch.where(there, i, -1).to(torch.int32)
        out["top_logp"] = torch.where(there, lp, NEG)
    return out


def _logprobs_backward(st):
    x, V = st["x"], st["case"]["V"]
    tok = st["tokens"].long()
    live = (tok >= 0) & (tok < V)
    lp = _z(x, st["scale"]) - st["lse"][:, None]
    p = torch.exp(lp)
    dlogp = torch.where(live, st["grad"], 0.0)
    d = -dlogp[:, None] * p
    if st["case"]["entropy"]:
        dh = torch.where(live, st["dentropy"], 0.0)
        d = d - dh[:, None] * torch.where(p == 0, 0.0, p * (lp + st["entropy"][:, None]))
    d.scatter_add_(1, torch.where(live, tok, 0)[:, None], dlogp[:, None])
    return {"dlogits": (d * st["scale"]).to(x.dtype)}


def _teacher(st):
    """Listed ids (0 where there is none), which of them count, and q, its log, and the bucket's mass."""
    V = st["case"]["V"]
    ids = st["ids"].long()
    valid = (ids >= 0) & (ids < V)
    lq = torch.where(valid, st["teacher_logp"], NEG)
    if not st["case"]["tail"]:
        total = _lse(lq)
        lq = lq - torch.where(total == NEG, 0.0, total)[:, None]
    q = torch.exp(lq)
    # 1 - sum q, in 64 bits: what is left of 1 may be little
    rest = (1.0 - torch.exp(lq.double()).sum(1)).clamp_min(0.0).float() if st["case"]["tail"] else torch.zeros_like(q[:, 0])
    return torch.where(valid, ids, 0), valid, q, lq, rest


def _distill(st):
    tail = st["case"]["tail"]
    ids, valid, q, lq, q0 = _teacher(st)
    live = valid.any(1)
    z = _z(st["x"], st["scale"])
    lse = _lse(z)
    lp = z.gather(1, ids) - lse[:, None]
    loss = torch.where(q > 0, q * (lq - lp), 0.0).sum(1)
    out = {"lse": torch.where(live, lse, 0.0)}
    if tail:
        # an entry that does not count masks nothing: it goes to a column behind the last
        wide = torch.cat([z, torch.full_like(z[:, :1], NEG)], 1)
        rest = _lse(wide.scatter(1, torch.where(valid, ids, z.shape[1]), NEG))
        term = q0 * (torch.log(q0) - (rest - lse))
        loss = loss + torch.where((q0 > 0) & (rest > NEG), term, 0.0)
        out["lse_tail"] = torch.where(live, rest, 0.0)
    out["loss"] = torch.where(live, loss, 0.0)
    return out


def _distill_backward(st):
    tail = st["case"]["tail"]
    ids, valid, q, lq, q0 = _teacher(st)
    z = _z(st["x"], st["scale"])
    dloss = torch.where(valid.any(1), st["grad"], 0.0)
    p = torch.exp(z - st["lse"][:, None])
    d = q.sum(1, keepdim=True) * p
    if tail:
        q0 = torch.where(st["lse_tail"] == NEG, 0.0, q0)
        mass = (q.sum(1) + q0)[:, None]
        # unlisted: Q p - q0 p / p0 with p / p0 = exp(z - lse_tail)
        share = torch.where(z == NEG, 0.0, torch.exp(z - st["lse_tail"][:, None]))
        d = mass * p - q0[:, None] * share
        listed_d = mass * p.gather(1, ids)
        d.scatter_(1, ids, torch.where(valid, listed_d, d.gather(1, ids)))
    d.scatter_add_(1, ids, torch.where(valid, -q, 0.0))
    return {"dlogits": (d * dloss[:, None] * st["scale"]).to(st["x"].dtype)}


PLAIN = {"logprobs": _logprobs, "logprobs_backward": _logprobs_backward, "distill": _distill,
         "distill_backward": _distill_backward}


def _calls(st):
    """The library's calls on the same state."""
    import nvfp4_quantized_rl_gb300 as nv
    case, op = st["case"], st["case"]["op"]
    if op == "logprobs":
        logp, h, lse, ids, top = nv.token_logprobs(st["x"], st["tokens"], st["scale"], k=case["k"],
                                                   entropy=case["entropy"])
        out = {"logp": logp, "lse": lse}
        if case["entropy"]:
            out["entropy"] = h
        if case["k"]:
            out.update(top_ids=ids, top_logp=top)
        return out
    if op == "logprobs_backward":
        return {"dlogits": nv.token_logprobs_backward(st["x"], st["tokens"], st["lse"], st["grad"], st["scale"],
                                                      entropy=st.get("entropy"), dentropy=st.get("dentropy"))}
    if op == "distill":
        loss, lse, rest = nv.topk_distill(st["x"], st["ids"], st["teacher_logp"], st["scale"], tail=case["tail"])
        return {"lse": lse, "loss": loss, "lse_tail": rest} if case["tail"] else {"lse": lse, "loss": loss}
    return {"dlogits": nv.topk_distill_backward(st["x"], st["ids"], st["teacher_logp"], st["lse"], st["grad"],
                                                st["scale"], tail=case["tail"], lse_tail=st.get("lse_tail"))}


def run(state):
    if own:
        return _calls(state)
    return PLAIN[state["case"]["op"]](state)


def work(case):
    """Each logit of a row that counts read once, every output written once."""
    M, V, b = case["M"], case["V"], 2 if case["dtype"] == "bf16" else 4
    live = M - _ignored(case)
    bytes_, flops = live * V * b, live * V * 3  # scale, exp, sum
    if case["op"] == "logprobs":
        bytes_ += M * (4 + 4 + 4 + (4 if case["entropy"] else 0) + 8 * case["k"])
        flops += live * V * 2 if case["entropy"] else 0
    elif case["op"] == "logprobs_backward":
        bytes_ += M * V * b + M * (12 + (8 if case["entropy"] else 0))
        flops += live * V * (3 if case["entropy"] else 1)
    elif case["op"] == "distill":
        bytes_ += M * (8 * case["k"] + 8 + (4 if case["tail"] else 0))
    else:
        bytes_ += M * V * b + M * (8 * case["k"] + 8 + (4 if case["tail"] else 0))
        flops += live * V
    return {"bytes": bytes_, "flops": flops}


# ---- the definitions in 64 bits, row by row in blocks ------------------------------------------------


def exact(case, seed):
    st = prepare(case, seed)
    parts = []
    for a in range(0, case["M"], 256):
        parts.append(_exact_rows(case, {n: v[a:a + 256] if torch.is_tensor(v) else v for n, v in st.items()}))
    return {n: torch.cat([p[n] for p in parts]) for n in parts[0]}


def _exact_rows(case, st):
    V, op, scale = case["V"], case["op"], st["scale"]
    x = st["x"].double()
    z = (x * scale).masked_fill(x <= MASKED, NEG)
    m = len(x)
    rows = torch.arange(m, device=x.device)
    if op == "logprobs":
        t = st["tokens"].long()
        skip = (t < 0) | (t >= V)
        lse = torch.logsumexp(z, 1)
        lp = z - lse[:, None]
        out = {"logp": lp[rows, t.masked_fill(skip, 0)].masked_fill(skip, 0.0), "lse": lse.masked_fill(skip, 0.0)}
        if case["entropy"]:
            out["entropy"] = (-(lp.exp() * lp).nan_to_num(0.0).sum(1)).masked_fill(skip, 0.0)
        if case["k"]:
            # largest first, ties to the lower column: the order of (value, -column)
            order = torch.argsort(x, dim=1, descending=True, stable=True)[:, :case["k"]]
            gone = (x.gather(1, order) <= MASKED) | skip[:, None]
            out["top_ids"] = order.masked_fill(gone, -1).int()
            out["top_logp"] = lp.gather(1, order).masked_fill(gone, NEG)
        return out
    # the backward passes take lse (and the entropy, the tail's lse) as the forward call left them, in fp32
    if op == "logprobs_backward":
        t = st["tokens"].long()
        skip = (t < 0) | (t >= V)
        lp = z - st["lse"].double()[:, None]
        dl = st["grad"].double().masked_fill(skip, 0.0)
        one = torch.zeros_like(z)
        one[rows, t.masked_fill(skip, 0)] = 1.0
        d = dl[:, None] * (one - lp.exp())
        if case["entropy"]:
            dh = st["dentropy"].double().masked_fill(skip, 0.0)
            d -= dh[:, None] * (lp.exp() * (lp + st["entropy"].double()[:, None])).nan_to_num(0.0)
        return {"dlogits": d * scale}
    ids = st["ids"].long()
    skip = ~((ids >= 0) & (ids < V)).any(1)  # here a row counts whole or not at all
    ids = ids.masked_fill(skip[:, None], 0)
    lq = st["teacher_logp"].double()
    if not case["tail"]:
        lq = lq - lq.logsumexp(1, keepdim=True)
    q = lq.exp()
    q0 = (1.0 - q.sum(1)).clamp_min(0.0) if case["tail"] else torch.zeros_like(q[:, 0])
    if op == "distill":
        lse = torch.logsumexp(z, 1)
        loss = (q * (lq - (z.gather(1, ids) - lse[:, None]))).sum(1)
        out = {"lse": lse.masked_fill(skip, 0.0)}
        if case["tail"]:
            rest = torch.logsumexp(z.scatter(1, ids, NEG), 1)
            loss = loss + (torch.xlogy(q0, q0) - q0 * (rest - lse))
            out["lse_tail"] = rest.masked_fill(skip, 0.0)
        out["loss"] = loss.masked_fill(skip, 0.0)
        return out
    p = (z - st["lse"].double()[:, None]).exp()
    mass = q.sum(1) + q0
    d = mass[:, None] * p
    if case["tail"]:
        unlisted = torch.ones_like(z).scatter(1, ids, 0.0)
        d -= unlisted * q0[:, None] * (z - st["lse_tail"].double()[:, None]).exp()
    target = torch.zeros_like(z).scatter_add(1, ids, q)
    dl = st["grad"].double().masked_fill(skip, 0.0)
    return {"dlogits": (d - target) * dl[:, None] * scale}
