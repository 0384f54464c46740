"""GPU: a step of group-relative policy optimisation through the operators together: prompts into the prefix caches, decode
steps for the samples behind them, log-probs, rectifying weights, the policy loss back to the logits, a preference loss over
the same responses; the same step captured and replayed, and captured steps that share a workspace."""
import numpy as np
import pytest
import torch

import synth
from tests import _grpo as G
from tests import _parity as P

pytestmark = pytest.mark.gpu

HQ, HKV, D, V, STEPS = 8, 2, 128, 96, 5
PROMPTS = [37, 150]           # tokens
GROUPS = [0, 3, 6]            # samples of each
B, LP, LMAX = GROUPS[-1], 160, 16
SCALE = 0.08


@pytest.fixture(scope="module")
def nv():
    import nvfp4_quantized_rl_gb300 as m
    m.lib()
    return m


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def inputs(seed):
    r = synth.rng(seed)
    bf = lambda *s: P.dev_bf16(synth.bf16_bits(r.standard_normal(s).astype(np.float32)))
    T = sum(PROMPTS)
    return {"pk": bf(T, HKV, D), "pv": bf(T, HKV, D), "q": bf(STEPS, B, HQ, D), "k": bf(STEPS, B, HKV, D),
            "v": bf(STEPS, B, HKV, D), "w": P.dev((r.standard_normal((HQ * D, V)) / 8).astype(np.float32)),
            "adv": P.dev(r.standard_normal(B).astype(np.float32)),
            "drift": P.dev((0.3 * r.standard_normal(B * STEPS)).astype(np.float32))}


class Step:
    def __init__(self, nv):
        self.nv = nv
        cache = lambda n, L: tuple(torch.zeros(n, L, HKV, D // w, dtype=torch.uint8, device="cuda") for w in (2, 16, 2, 16))
        self.pre, self.own = cache(len(PROMPTS), LP), cache(B, LMAX)
        self.g = torch.tensor([4.5 / 2688], device="cuda")
        self.offsets, self.plens, self.groups = ints([0] + list(np.cumsum(PROMPTS))), ints(PROMPTS), ints(GROUPS)
        self.places = [ints([t] * B) for t in range(STEPS + 1)]
        self.responses = ints([STEPS * b for b in range(B + 1)])

    def attend(self, q, lens):
        pk, ps, pv, pvs = self.pre
        k, s, v, vs = self.own
        return self.nv.nvfp4_kv_prefix_attention(q, pk, ps, pv, pvs, self.plens, self.groups, k, s, v, vs, lens, self.g, self.g,
                                                 SCALE)

    def __call__(self, x, between=lambda: None):
        nv = self.nv
        nv.nvfp4_kv_append_ragged(x["pk"], x["pv"], self.offsets, None, self.g, self.g, *self.pre)
        outs, logits, tokens, old = [], [], [], []
        for t in range(STEPS):
            between()
            nv.nvfp4_kv_append(x["k"][t], x["v"][t], self.places[t], self.g, self.g, *self.own)
            between()
            o = self.attend(x["q"][t], self.places[t + 1])
            between()
            z = o.view(B, HQ * D).float() @ x["w"]
            _, _, _, ids, _ = nv.token_logprobs(z, k=2)
            tok = ids[:, 1].contiguous()  # the runner-up, so that gradients are not small
            lp = nv.token_logprobs(z, tok, entropy=False)[0]
            for seen, new in zip((outs, logits, tokens, old), (o, z, tok, lp)):
                seen.append(new)
        pack = lambda seen: torch.stack(seen, 1).reshape((B * STEPS,) + seen[0].shape[1:]).contiguous()  # a sample's steps in a row
        z, tok, old = pack(logits), pack(tokens), pack(old)
        logp, _, lse, _, _ = nv.token_logprobs(z, tok, entropy=False)
        logp_old, ref = old + x["drift"], old - 0.5 * x["drift"]
        _, weights = nv.ais_mixing(logp_old, logp, torch.repeat_interleave(x["adv"], STEPS), 2.0, 1e-6, 1.0, 1.0)
        terms = dict(logp_ref=ref, weights=weights, kl_coef=0.05, dual_clip=3.0)
        loss, stats, coef = nv.policy_loss(logp, logp_old, x["adv"], self.responses, mode=nv.LOSS_SEQ_MEAN, **terms)
        dlogp = nv.policy_loss_backward(logp, logp_old, x["adv"], self.responses, coef, **terms)
        dz = nv.token_logprobs_backward(z, tok, lse, dlogp)
        pairs, rewards, pcoef = nv.preference_loss(logp, self.responses, ref, beta=0.3, mean=True)
        pgrad = nv.preference_loss_backward(self.responses, pcoef, None, B * STEPS)
        return dict(outs=torch.stack(outs), z=z, tok=tok, logp=logp, lse=lse, old=logp_old, ref=ref, weights=weights, loss=loss,
                    stats=stats, dlogp=dlogp, dz=dz, pairs=pairs, rewards=rewards, pgrad=pgrad)


def bits(r):
    torch.cuda.synchronize()
    return {k: v.clone() for k, v in r.items()}


def test_a_step_against_the_definitions(nv):
    step, x = Step(nv), inputs(1)
    got = bits(step(x))
    host = {k: v.cpu().numpy() for k, v in got.items() if v.dtype != torch.bfloat16}
    # every decode step, from the rows that the caches hold
    whole = lambda n, L: ints([L * b for b in range(n + 1)])
    read = lambda c, n, L: [t.cpu().numpy().astype(np.float64).reshape(n, L, HKV, D) for t in nv.nvfp4_kv_read(
        c[0], c[1], step.g, c[2], c[3], step.g, whole(n, L), tokens=n * L, dtype=torch.float32)]
    pre, own = read(step.pre, len(PROMPTS), LP), read(step.own, B, LMAX)
    for t in range(STEPS):
        want, tol = G.attention(x["q"][t].double().cpu().numpy(), pre, own, PROMPTS, GROUPS, [t + 1] * B, G.f32(SCALE))
        G.close(got["outs"][t].double().cpu().numpy(), want, tol, f"attention, step {t}")
    # the losses, from the log-probs that the step had
    off = np.arange(B + 1, dtype=np.int32) * STEPS
    want = G.policy(host["logp"], host["old"], x["adv"].cpu().numpy(), off, ref=host["ref"], weights=host["weights"], dual=3.0,
                    kl=0.05, mode=1)
    for k in ("loss", "stats", "dlogp"):
        G.close(host[k], want[k], want["tol"][k], k)
    pref = G.preference(host["logp"], off, ref=host["ref"], beta=0.3, mean=True)
    for k, name in (("pairs", "loss"), ("rewards", "rewards"), ("pgrad", "dlogp")):
        G.close(host[k], pref[name], pref["tol"][name], k)
    # back to the logits: dlogp (one-hot - softmax); an exponential of l - lse is off by its argument's rounding (u |l - lse|, the
    # lse by 4u (1 + |lse|)) and by 4u
    z = host["z"].astype(np.float64)
    lse = np.logaddexp.reduce(z, axis=1)[:, None]
    p = np.exp(z - lse)
    hot = np.eye(V)[host["tok"]]
    dl = want["dlogp"][:, None]
    tol = want["tol"]["dlogp"][:, None] * np.abs(hot - p) + np.abs(dl) * G.U * (
        p * (6 + 4 * (1 + np.abs(lse)) + 2 * np.abs(z - lse)) + 4 * np.abs(hot - p)) + 2.0 ** -120
    G.close(host["dz"], dl * (hot - p), tol, "gradient of the logits")
    assert np.abs(host["dz"]).max() > 1e-4


def test_a_step_needs_no_waiting_and_replays(nv):
    """Kernel behind kernel equals a wait after each; captured and replayed on other prompts, rows and advantages; on a side
    stream: the same bits."""
    step, x = Step(nv), inputs(2)
    want = bits(step(x, torch.cuda.synchronize))
    for _ in range(20):
        got = step(x)
        assert all(torch.equal(got[k], want[k]) for k in want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step(x)
    s.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x)
    for seed in (3, 4, 3):
        for k, v in inputs(seed).items():
            x[k].copy_(v)
        for c in step.pre + step.own:
            c.zero_()
        graph.replay()
        replayed = bits(out)
        eager = bits(step(x))
        assert all(torch.equal(replayed[k], eager[k]) for k in eager)


def test_graphs_that_share_a_workspace(nv):
    """Two captured calls of each operator with one workspace of any contents, replayed by turns on one stream."""
    r = synth.rng(7)
    Hq, Hkv, n = 12, 4, 20000
    g = torch.tensor([3.0 / 2688], device="cuda")
    states = []
    for seed, (P_, Bq) in ((11, (2, 9)), (12, (5, 30))):
        pre = tuple(P.dev(a) for a in G.cache(P_, 300, Hkv, seed)[:2] + G.cache(P_, 300, Hkv, seed + 1)[:2])
        own = tuple(P.dev(a) for a in G.cache(Bq, 90, Hkv, seed + 2)[:2] + G.cache(Bq, 90, Hkv, seed + 3)[:2])
        q = P.dev_bf16(synth.bf16_bits(r.standard_normal((Bq, Hq, 128)).astype(np.float32)))
        groups = ints([Bq * i // P_ for i in range(P_ + 1)])
        logp = P.dev((-r.random(n)).astype(np.float32))
        off = G.ragged(2 * Bq, seed, n)
        states.append(dict(pre=pre, own=own, q=q, groups=groups, plens=ints(r.integers(0, 301, P_)), lens=ints(r.integers(0, 91, Bq)),
                           logp=logp, old=logp + 0.1, off=P.dev(off), adv=P.dev(r.standard_normal(2 * Bq).astype(np.float32))))
    need = max(max(nv.workspace_bytes(nv.OP_KV_PREFIX_ATTENTION, len(s["lens"]), Hkv, 90, Hq // Hkv, len(s["plens"])) for s in states),
               nv.workspace_bytes(nv.OP_POLICY_LOSS, 20000, 60, 0), nv.workspace_bytes(nv.OP_PREFERENCE_LOSS, 20000, 30, 0))
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")

    def call(s, **kw):
        a = nv.nvfp4_kv_prefix_attention(s["q"], *s["pre"], s["plens"], s["groups"], *s["own"], s["lens"], g, g, 0.09, **kw)
        b = nv.policy_loss(s["logp"], s["old"], s["adv"], s["off"], **kw)
        c = nv.preference_loss(s["logp"], s["off"], **kw)
        return (a,) + b + c

    want = [call(s) for s in states]
    graphs = []
    for s in states:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call(s, workspace=ws)
        graphs.append((graph, out))
    for turn in (0, 1, 1, 0, 1, 0):
        graphs[turn][0].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(graphs[turn][1], want[turn])), turn
        ws.fill_(0xFF)


def test_two_steps_at_once(nv):
    """Two steps on two streams, each with caches of its own, side by side: the bits of one after the other."""
    steps = [(Step(nv), inputs(5)), (Step(nv), inputs(6))]
    want = [bits(step(x)) for step, x in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(10):
        got = []
        for s, (step, x) in zip(streams, steps):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(step(x))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(g[k], w[k]) for k in w)


def test_many_decode_steps_without_waiting(nv):
    """Each step appends a row next to rows that the last one read and lengthens the caches in place: kernel behind kernel equals
    a wait after each."""
    steps, seqs, rows = 300, 40, 320
    r = synth.rng(8)
    bf = lambda *s: P.dev_bf16(synth.bf16_bits(r.standard_normal(s).astype(np.float32)))
    q, k, v = bf(steps, seqs, 4, D), bf(steps, seqs, 1, D), bf(steps, seqs, 1, D)
    pre = tuple(P.dev(a) for a in G.cache(2, 200, 1, 81)[:2] + G.cache(2, 200, 1, 82)[:2])
    g = torch.tensor([4.5 / 2688], device="cuda")
    groups, plens = ints([0, 11, seqs]), ints([200, 77])

    def run(between):
        own = tuple(torch.zeros(seqs, rows, 1, D // w, dtype=torch.uint8, device="cuda") for w in (2, 16, 2, 16))
        pos, lens, outs = ints([0] * seqs), ints([0] * seqs), []
        for t in range(steps):
            nv.nvfp4_kv_append(k[t], v[t], pos, g, g, *own)
            between()
            lens.add_(1)
            between()
            outs.append(nv.nvfp4_kv_prefix_attention(q[t], *pre, plens, groups, *own, lens, g, g, 0.1))
            between()
            pos.add_(1)
            between()
        return torch.stack(outs)

    want = run(torch.cuda.synchronize)
    for _ in range(5):
        assert torch.equal(run(lambda: None), want)


def test_offsets_rewritten_in_place_between_calls(nv):
    """Offsets, lengths and group bounds that a kernel rewrites right ahead of each call: the bits of calls with waits between."""
    n, seqs, pairs = 20000, 40, 20
    r = synth.rng(9)
    logp = P.dev((-3 * r.random(n)).astype(np.float32))
    old, adv = logp + 0.1, P.dev(r.standard_normal(seqs).astype(np.float32))
    offs = [P.dev(np.sort(r.integers(0, n + 1, seqs + 1)).astype(np.int32)) for _ in range(7)]
    pre = tuple(P.dev(a) for a in G.cache(3, 500, 2, 91)[:2] + G.cache(3, 500, 2, 92)[:2])
    own = tuple(P.dev(a) for a in G.cache(30, 90, 2, 93)[:2] + G.cache(30, 90, 2, 94)[:2])
    q = P.dev_bf16(synth.bf16_bits(r.standard_normal((30, 6, D)).astype(np.float32)))
    g = torch.tensor([0.002], device="cuda")
    groups = [ints(np.sort(r.integers(0, 31, 4))) for _ in range(7)]
    plens, lens = [ints(r.integers(0, 501, 3)) for _ in range(7)], [ints(r.integers(0, 91, 30)) for _ in range(7)]

    def run(between):
        off, gr, pl, ln, outs = offs[0].clone(), groups[0].clone(), plens[0].clone(), lens[0].clone(), []
        for i in range(200):
            for into, of in ((off, offs), (gr, groups), (pl, plens), (ln, lens)):
                into.copy_(of[i % 7])
            between()
            outs.append(nv.policy_loss(logp, old, adv, off)[1])
            between()
            off.copy_(offs[(i + 3) % 7])
            between()
            outs.append(nv.preference_loss(logp, off)[0])
            between()
            outs.append(nv.nvfp4_kv_prefix_attention(q, *pre, pl, gr, *own, ln, g, g, 0.1).float().sum((1, 2)))
            between()
        return torch.cat(outs)

    want = run(torch.cuda.synchronize)
    for _ in range(5):
        assert torch.equal(run(lambda: None), want)
