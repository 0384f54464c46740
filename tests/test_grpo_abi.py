"""Host-side validation of the ragged cache calls, the shared-prefix attention and the losses: bad arguments come back as
their status before a GPU is touched, and the binding refuses tensors that the call does not take (CPU only)."""
import numpy as np
import pytest
import torch

from tests import _grpo as G

A = [0x100000000 * i for i in range(1, 16)]
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def nv():
    from nvfp4_quantized_rl_gb300 import _build
    _build.build()
    import nvfp4_quantized_rl_gb300 as m
    return m


def caller(fn, ok):
    return lambda **o: fn(*{**ok, **o}.values(), None)


@pytest.mark.parametrize("write", [True, False])
def test_ragged_validation(nv, write):
    if write:
        ok = dict(k=A[0], v=A[1], dtype=0, T=100, ldk=512, ldv=512, H=4, D=128, off=A[2], pos=A[3], B=3, gk=A[4], gv=A[5],
                  kc=A[6], ks=A[7], vc=A[8], vs=A[9], L=50)
        call = caller(nv.lib().nvfp4_kv_append_ragged, ok)
    else:
        ok = dict(kc=A[6], ks=A[7], gk=A[4], vc=A[8], vs=A[9], gv=A[5], L=50, H=4, D=128, off=A[2], pos=A[3], B=3, T=100,
                  k=A[0], v=A[1], dtype=0, ldk=512, ldv=512)
        call = caller(nv.lib().nvfp4_kv_read, ok)
    assert call(dtype=2) == 1 and call(T=-1) == 1 and call(B=-1) == 1 and call(H=0) == 1 and call(D=0) == 1 and call(L=0) == 1
    assert call(ldk=511) == 1 and call(ldv=0) == 1
    for name in ("k", "v", "off", "gk", "gv", "kc", "ks", "vc", "vs"):
        assert call(**{name: None}) == 1, name
    assert call(D=24, ldk=96, ldv=96) == 3 and call(ldk=516) == 3 and call(dtype=1, ldv=514) == 3
    assert call(H=1 << 20) == 3 and call(T=1 << 31) == 3 and call(B=(1 << 20) + 1) == 3 and call(D=1 << 62) == 3
    assert call(ldk=1 << 47) == 3 and call(L=1 << 47) == 3
    for name in ("k", "v", "kc", "ks", "vc", "vs"):
        assert call(**{name: ok[name] + 8}) == 2, name
    for name in ("off", "pos", "gk", "gv"):
        assert call(**{name: ok[name] + 2}) == 2, name
    assert call(T=0, k=None) == 0 and call(B=0, off=None) == 0
    last_k, last_cache = A[0] + 2 * (99 * 512 + 512) - 16, A[6] + 3 * 50 * 4 * 64 - 16
    assert call(kc=last_k) == 7 and call(ks=A[0]) == 7 and call(v=last_cache) == 7
    if write:
        assert call(vs=A[6] + 16) == 7 and call(off=A[6] + 4) == 7 and call(gk=A[7]) == 7 and call(pos=A[9]) == 7
    else:
        assert call(off=A[0] + 4) == 7 and call(pos=A[1]) == 7 and call(gv=A[1] + 4) == 7
        assert call(v=A[0]) == 7 and call(v=A[0] + 16) == 7 and call(v=A[0] + 1024, ldk=520, ldv=520) == 7
        assert call(v=A[0] + 1024, ldk=1024) == 7  # other strides


def test_prefix_attention_validation(nv):
    ok = dict(q=A[0], ldq=3584, pkc=A[1], pks=A[2], pvc=A[3], pvs=A[4], pl=A[5], gr=A[6], P=2, Lp=100, kc=A[7], ks=A[8], vc=A[9],
              vs=A[10], lens=A[11], Lmax=30, gk=A[12], gv=A[12] + 4, B=8, Hq=28, Hkv=4, D=128, scale=0.1, out=A[13], ws=A[14],
              wsb=1 << 32)
    call = caller(nv.lib().nvfp4_kv_prefix_attention, ok)
    for bad in (dict(B=-1), dict(Hq=0), dict(Hkv=0), dict(D=0), dict(Lp=0), dict(Lmax=-1), dict(P=0), dict(P=1025),
                dict(scale=NAN), dict(scale=INF), dict(ldq=3583)):
        assert call(**bad) == 1, bad
    for bad in (dict(D=64), dict(Hq=27, ldq=4000), dict(Hq=68, ldq=9000), dict(B=16384), dict(ldq=3588), dict(Lp=1 << 30),
                dict(Lmax=1 << 28), dict(Lp=1 << 62)):
        assert call(**bad) == 3, bad
    for name in ("q", "pkc", "pks", "pvc", "pvs", "pl", "gr", "kc", "ks", "vc", "vs", "lens", "gk", "gv", "out"):
        assert call(**{name: None}) == 1, name
    for name in ("q", "pkc", "pks", "pvc", "pvs", "kc", "ks", "vc", "vs", "out", "ws"):
        assert call(**{name: ok[name] + 8}) == 2, name
    for name in ("pl", "gr", "lens", "gk", "gv"):
        assert call(**{name: ok[name] + 2}) == 2, name
    need = nv.workspace_bytes(nv.OP_KV_PREFIX_ATTENTION, 8, 4, 30, 7, 2)
    assert need > 0 and call(ws=None) == 4 and call(wsb=need - 1) == 4
    assert call(out=A[0]) == 7 and call(out=A[1] + 16) == 7 and call(gr=A[13]) == 7 and call(ws=A[7] + 16) == 7
    assert call(ws=A[13] + 64) == 7 and call(lens=A[14] + 64) == 7
    assert call(B=0, q=None) == 0
    for bad in ((-1, 4, 30, 7, 2), (8, 0, 30, 7, 2), (8, 4, 30, 0, 2), (8, 4, 30, 17, 2), (8, 4, 30, 7, 0), (8, 4, 30, 7, 1025)):
        assert nv.workspace_bytes(nv.OP_KV_PREFIX_ATTENTION, *bad) == 0
    assert nv.workspace_bytes(nv.OP_KV_PREFIX_ATTENTION, 0, 4, 30, 7, 2) >= 0


def test_policy_validation(nv):
    ok = dict(lp=A[0], old=A[1], ref=A[2], adv=A[3], per=0, w=A[4], mask=A[5], off=A[6], n=100, B=3, lo=0.2, hi=0.2, dual=0.0,
              kl=0.1, mode=0, norm=1.0, loss=A[7], stats=A[8], coef=A[9], ws=A[10], wsb=1 << 20)
    call = caller(nv.lib().policy_loss, ok)
    ok2 = {k: v for k, v in ok.items() if k not in ("mode", "norm", "loss", "stats", "coef", "ws", "wsb")}
    back = caller(nv.lib().policy_loss_backward, {**ok2, "coef": A[9], "dl": A[7], "out": A[8]})
    for f in (call, back):
        for bad in (dict(n=-1), dict(B=-1), dict(lo=-0.1), dict(lo=1.0), dict(lo=NAN), dict(hi=-0.1), dict(hi=INF), dict(hi=NAN),
                    dict(dual=0.5), dict(dual=-1.0), dict(dual=INF), dict(dual=NAN), dict(kl=-1.0), dict(kl=NAN), dict(kl=INF),
                    dict(lp=None), dict(old=None), dict(adv=None), dict(off=None), dict(coef=None) if f is back else dict(loss=None)):
            assert f(**bad) == 1, bad
        assert f(n=1 << 31) == 3 and f(B=(1 << 31) - 1) == 3
        for name in ("lp", "old", "ref", "adv", "w", "off", "coef"):
            assert f(**{name: A[11] + 2}) == 2, name
    for bad in (dict(mode=3), dict(mode=-1), dict(mode=2, norm=0.0), dict(mode=2, norm=-1.0), dict(mode=2, norm=INF),
                dict(mode=2, norm=NAN)):
        assert call(**bad) == 1, bad
    need = nv.workspace_bytes(nv.OP_POLICY_LOSS, 100, 3, 0)
    assert call(ws=None) == 4 and call(wsb=need - 1) == 4 and call(ws=A[10] + 8) == 2
    assert call(loss=A[0] + 396) == 7 and call(stats=A[7]) == 7 and call(coef=A[8] + 28) == 7 and call(coef=A[5] + 96) == 7
    assert call(ws=A[3] + 0) == 7 and call(coef=A[10] + need - 16) == 7
    assert back(out=A[0]) == 7 and back(out=A[9] - 396) == 7 and back(dl=A[8] + 396) == 7 and back(mask=A[8] + 399) == 7
    assert back(adv=A[8] - 8) == 7 and back(adv=A[8] - 396, per=1) == 7
    assert back(n=0, lp=None, old=None) == 0


def test_preference_validation(nv):
    ok = dict(lp=A[0], ref=A[1], mask=A[2], off=A[3], n=100, pairs=3, beta=0.1, margin=0.0, eps=0.0, mean=0, loss=A[4],
              rewards=A[5], coef=A[6], ws=A[7], wsb=1 << 20)
    call = caller(nv.lib().preference_loss, ok)
    for bad in (dict(n=-1), dict(pairs=-1), dict(beta=0.0), dict(beta=-1.0), dict(beta=NAN), dict(beta=INF), dict(margin=INF),
                dict(margin=NAN), dict(eps=-0.1), dict(eps=1.0), dict(eps=NAN), dict(lp=None), dict(off=None), dict(loss=None)):
        assert call(**bad) == 1, bad
    assert call(n=1 << 31) == 3 and call(pairs=1 << 30) == 3
    for name in ("lp", "ref", "off", "loss", "rewards", "coef"):
        assert call(**{name: ok[name] + 2}) == 2, name
    need = nv.workspace_bytes(nv.OP_PREFERENCE_LOSS, 100, 3, 0)
    assert call(ws=None) == 4 and call(wsb=need - 1) == 4 and call(ws=A[7] + 4) == 2
    assert call(loss=A[0]) == 7 and call(rewards=A[4] + 8) == 7 and call(coef=A[3] + 24) == 7 and call(ws=A[6] - need + 16) == 7
    assert call(pairs=0, off=None) == 0
    back = caller(nv.lib().preference_loss_backward, dict(mask=A[0], off=A[1], n=100, pairs=3, coef=A[2], dl=A[3], out=A[4]))
    assert back(n=-1) == 1 and back(pairs=-1) == 1 and back(off=None) == 1 and back(coef=None) == 1 and back(out=None) == 1
    assert back(n=1 << 31) == 3 and back(pairs=1 << 30) == 3 and back(off=A[1] + 1) == 2 and back(out=A[4] + 2) == 2
    assert back(out=A[0] + 96) == 7 and back(out=A[2]) == 7 and back(dl=A[4] + 396) == 7 and back(n=0, out=None) == 0


def test_workspace_sizes_of_the_losses(nv):
    assert nv.workspace_bytes(nv.OP_POLICY_LOSS, 1 << 31, 1, 0) == 0 and nv.workspace_bytes(nv.OP_POLICY_LOSS, -1, 1, 0) == 0
    assert nv.workspace_bytes(nv.OP_POLICY_LOSS, 0, 0, 0) > 0 and nv.workspace_bytes(nv.OP_PREFERENCE_LOSS, 0, 1, 0) > 0
    assert nv.workspace_bytes(nv.OP_PREFERENCE_LOSS, 1, 1 << 30, 0) == 0


class OnGpu:
    """A CPU tensor that says it is on device 0, for the checks that need no GPU."""

    def __init__(self, t):
        self.t = t

    def get_device(self):
        return 0

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_binding_refuses_cpu_and_wrong_tensors(nv):
    k = torch.zeros(5, 2, 32)
    i = torch.zeros(3, dtype=torch.int32)
    c = [torch.zeros(2, 4, 2, w, dtype=torch.uint8) for w in (16, 2, 16, 2)]
    g = torch.zeros(1)
    with pytest.raises(ValueError):
        nv.nvfp4_kv_append_ragged(k, k, i, None, g, g, *c)
    with pytest.raises(ValueError):
        nv.nvfp4_kv_read(c[0], c[1], g, c[2], c[3], g, i, None, 5)
    with pytest.raises(ValueError):
        nv.nvfp4_kv_prefix_attention(k.bfloat16(), *c, i, i, None, None, None, None, None, g, g, 1.0)
    with pytest.raises(ValueError):
        nv.policy_loss(g, g, g, i)
    with pytest.raises(ValueError):
        nv.preference_loss(g, i)
    with pytest.raises(ValueError):
        nv.preference_loss_backward(i, torch.zeros(2), None, 4)
    for bad in (k.half(), k.int()):
        with pytest.raises(TypeError):
            nv._packed_rows(OnGpu(bad), "k")
    for bad in (k[0], k.transpose(0, 1), k[:, :, ::2], k.expand(2, 5, 2, 32), k[:1].expand(4, 2, 32)):
        with pytest.raises(ValueError):
            nv._packed_rows(OnGpu(bad), "k")
    assert nv._packed_rows(OnGpu(torch.zeros(5, 9, 32)[:, 2:4]), "k") == (nv.F32, 5, 2, 32, 288, 0)
    assert nv._packed_rows(OnGpu(torch.zeros(5, 9, 32).bfloat16()[2:3, 2:4]), "k") == (nv.BF16, 1, 2, 32, 64, 0)
    on = [OnGpu(t) for t in c]
    assert nv._cache_arrays(on, 32, 0)[1:] == (2, 4, 2)
    for n in range(4):
        for bad in (c[n].int(), c[n][:, ::2], torch.zeros(2, 4, 2, 3, dtype=torch.uint8)):
            with pytest.raises(ValueError):
                nv._cache_arrays([OnGpu(bad) if j == n else t for j, t in enumerate(on)], 32, 0)
    with pytest.raises(ValueError):
        nv._cache_arrays(on, 32, 1)
    for bad in (torch.zeros(2), torch.zeros(1).double()):
        with pytest.raises(ValueError):
            nv._scale_arrays(OnGpu(bad), OnGpu(g), 0)
    lp = OnGpu(torch.zeros(10))
    with pytest.raises(TypeError):
        nv._loss_arrays(lp, OnGpu(i), 1, (), OnGpu(torch.zeros(10)))
    for off, per, mask in ((i.long(), 1, None), (i.view(1, 3), 1, None), (i[:0], 1, None), (i[:2], 2, None),
                           (i, 1, torch.zeros(9, dtype=torch.bool))):
        with pytest.raises(ValueError):
            nv._loss_arrays(lp, OnGpu(off), per, (), None if mask is None else OnGpu(mask))
    with pytest.raises(ValueError):
        nv._loss_arrays(lp, OnGpu(i), 1, (("logp_old", OnGpu(torch.zeros(9))),), None)


# ---- the definitions that the GPU tests compare with ----------------------------------------------------------


def test_definition_of_the_policy_loss():
    """Closed forms, and torch's autograd of the formula written with min and clamp."""
    r = np.random.default_rng(0)
    off = np.array([0, 4, 4, 11], np.int32)
    old = -r.random(12).astype(np.float32)
    lp = (old + 0.4 * r.standard_normal(12)).astype(np.float32)
    ref = (old + 0.4 * r.standard_normal(12)).astype(np.float32)
    adv, w = np.array([1.0, 9.0, -2.0], np.float32), r.random(12).astype(np.float32)
    mask = np.array([1, 1, 0, 1, 1, 1, 1, 0, 1, 1, 1, 1], bool)
    assert G.policy(old, old, adv, off)["loss"][0] == pytest.approx(-(4 * 1 - 7 * 2) / 11)  # r = 1
    seq = np.repeat([0, 2], [4, 7])
    for mode, norm in ((0, 1.0), (1, 1.0), (2, 7.0)):
        got = G.policy(lp, old, adv, off, ref=ref, weights=w, mask=mask, low=0.2, high=0.3, dual=1.5, kl=0.25, mode=mode, norm=norm)
        x = torch.tensor(lp.astype(np.float64), requires_grad=True)
        m = torch.tensor(mask[:11].astype(np.float64))
        d = x[:11] - torch.tensor(old[:11].astype(np.float64))
        A = torch.tensor(adv.astype(np.float64))[seq]
        gain = torch.minimum(d.exp() * A, d.exp().clamp(1 - G.f32(0.2), 1 + G.f32(0.3)) * A)
        gain = torch.where(A < 0, torch.maximum(gain, 1.5 * A), gain)
        y = torch.tensor(ref[:11].astype(np.float64)) - x[:11]
        each = -torch.tensor(w[:11].astype(np.float64)) * gain + 0.25 * (y.exp() - y - 1)
        count = np.array([3.0, 6.0])[(seq > 0).astype(int)]
        c = m / m.sum() if mode == 0 else m / torch.tensor(count) / 2 if mode == 1 else m / 7
        loss = (c * each).sum()
        loss.backward()
        assert got["loss"][0] == pytest.approx(loss.item(), rel=1e-12)
        assert np.allclose(got["dlogp"], x.grad.numpy(), rtol=1e-12, atol=1e-15)
        assert got["stats"][6] == 9 and got["stats"][7] == 2


def test_definition_of_the_preference_loss():
    r = np.random.default_rng(1)
    off = np.array([0, 3, 3, 7, 9], np.int32)
    lp, ref = -r.random(9).astype(np.float32), -r.random(9).astype(np.float32)
    mask = np.array([1, 0, 1, 1, 1, 1, 0, 1, 1], bool)
    got = G.preference(lp, off, ref=ref, mask=mask, beta=0.5, margin=0.25, smoothing=0.125, mean=True)
    x = torch.tensor(lp.astype(np.float64), requires_grad=True)
    d = (x - torch.tensor(ref.astype(np.float64))) * torch.tensor(mask.astype(np.float64))
    s = torch.stack([d[:3].sum() / 2, d[3:3].sum(), d[3:7].sum() / 3, d[7:].sum() / 2])
    h = 0.5 * (s[::2] - s[1::2]) - 0.25
    ls = torch.nn.functional.logsigmoid
    loss = -0.875 * ls(h) - 0.125 * ls(-h)
    loss.sum().backward()
    assert np.allclose(got["loss"], loss.detach().numpy(), rtol=1e-12) and np.allclose(got["rewards"], 0.5 * s.detach().numpy())
    assert np.allclose(got["dlogp"], x.grad.numpy(), rtol=1e-12, atol=1e-15)


def test_definition_of_the_attention():
    """Against torch on one joined cache, and the cases without tokens."""
    r = np.random.default_rng(2)
    pre, own = [r.standard_normal((2, 6, 2, 128)) for _ in range(2)], [r.standard_normal((4, 5, 2, 128)) for _ in range(2)]
    q = r.standard_normal((4, 6, 128))
    out, tol = G.attention(q, pre, own, [6, 0], [0, 2, 3], [5, 0, 0, 2], 0.1)
    assert np.all(out[2] == 0) and np.all(tol > -1)
    for b, (kp, ko) in enumerate([(6, 5), (6, 0), (0, 0), (0, 2)]):
        if kp + ko == 0:
            continue
        k, v = (torch.tensor(np.concatenate([pre[i][0, :kp], own[i][b, :ko]])).repeat_interleave(3, 1) for i in range(2))
        p = torch.softmax(0.1 * torch.einsum("hd,thd->ht", torch.tensor(q[b]), k), -1)
        assert np.allclose(out[b], torch.einsum("ht,thd->hd", p, v).numpy())


def test_definition_of_the_rows():
    x = np.random.default_rng(3).standard_normal((7, 2, 32)).astype(np.float32)
    codes, scales = G.encode(x, np.float32(0.001))
    v = G.values(codes, scales, np.float32(0.001))
    # nothing above 6 x 448 x g = 2.688 can be held; below, a code is off by half its widest step (1) of a scale that
    # is within 2^-4 of the block's largest / 6
    assert np.max(np.abs(v - np.clip(x, -2.688, 2.688))) <= np.abs(x).max() / 6 * 1.0625
    assert G.packed_to_cache([1, 3, 3, 5], [0, 9, 4], 6, 5) == [None, (0, 0), (0, 1), (2, 4), (2, None), None]
