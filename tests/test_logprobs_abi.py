"""Host-side validation of the logits operators: bad arguments come back as their status before a GPU is touched,
and the binding refuses tensors that the call does not take (CPU only; addresses are never dereferenced)."""
import pytest
import torch

A0, A1, A2, A3, A4, A5, A6 = (0x1000000 * i for i in range(1, 8))


@pytest.fixture(scope="module")
def nv():
    from nvfp4_quantized_rl_gb300 import _build
    _build.build()
    import nvfp4_quantized_rl_gb300 as m
    return m


def _sizes(call):
    """Refusals that the four calls share; call(**overrides) -> status."""
    assert call(dtype=2) == 1 and call(M=-1) == 1 and call(V=0) == 1 and call(ld=99) == 1 and call(x=None) == 1
    for s in (0.0, -1.0, float("nan"), float("inf"), 2.0 ** -21, 2.0 ** 21):
        assert call(scale=s) == 1, s
    assert call(V=(1 << 22) + 1, ld=1 << 23) == 3 and call(M=1 << 31) == 3
    assert call(M=1 << 20, ld=1 << 29) == 3 and call(M=4, ld=1 << 62) == 3  # more than 2^48 elements
    assert call(x=A0 + 1) == 2 and call(dtype=1, x=A0 + 2) == 2
    assert call(M=0, x=None) == 0


def test_token_logprobs_validation(nv):
    ok = dict(x=A0, dtype=0, M=4, V=100, ld=104, tok=A1, scale=1.0, k=3, lp=A2, h=A3, lse=A4, ids=A5, top=A6)

    def call(**o):
        a = {**ok, **o}
        return nv.lib().token_logprobs(a["x"], a["dtype"], a["M"], a["V"], a["ld"], a["tok"], a["scale"], a["k"],
                                       a["lp"], a["h"], a["lse"], a["ids"], a["top"], None)
    _sizes(call)
    assert call(k=-1) == 1 and call(k=101) == 1 and call(k=257, V=1000, ld=1000) == 3
    assert call(tok=None) == 1                                   # logp without tokens
    assert call(ids=None) == 1 and call(top=None) == 1
    assert call(k=0, lp=None, h=None, lse=None) == 1             # nothing to compute
    assert call(tok=A1 + 2) == 2 and call(top=A6 + 1) == 2
    assert call(lp=A0 + 40) == 7 and call(h=A1) == 7             # over an input
    assert call(lse=A3 + 4) == 7 and call(top=A5 + 8) == 7       # over another output
    assert call(lp=A0 + 2 * (3 * 104 + 100) - 4) == 7            # over the last logits


def test_token_logprobs_backward_validation(nv):
    ok = dict(x=A0, dtype=0, M=4, V=100, ld=104, tok=A1, scale=1.0, lse=A2, h=A3, dlp=A4, dh=A5, dx=A6, ldd=100)

    def call(**o):
        a = {**ok, **o}
        return nv.lib().token_logprobs_backward(a["x"], a["dtype"], a["M"], a["V"], a["ld"], a["tok"], a["scale"],
                                                a["lse"], a["h"], a["dlp"], a["dh"], a["dx"], a["ldd"], None)
    _sizes(call)
    assert call(lse=None) == 1 and call(dlp=None, dh=None) == 1 and call(tok=None) == 1 and call(h=None) == 1
    assert call(dx=None) == 1 and call(ldd=99) == 1 and call(ldd=1 << 47) == 3
    assert call(dx=A6 + 1) == 2 and call(dlp=A4 + 2) == 2
    assert call(dx=A0) == 7                                      # the logits with another row stride
    assert call(dx=A0 + 2, ldd=104) == 7 and call(dx=A2 - 100) == 7


@pytest.mark.parametrize("mode", [0, 1])
def test_topk_distill_validation(nv, mode):
    ok = dict(x=A0, dtype=0, M=4, V=100, ld=104, scale=1.0, ids=A1, t=A2, k=3, mode=mode, loss=A3, lse=A4, rest=A5)

    def call(**o):
        a = {**ok, **o}
        return nv.lib().topk_distill(a["x"], a["dtype"], a["M"], a["V"], a["ld"], a["scale"], a["ids"], a["t"], a["k"],
                                     a["mode"], a["loss"], a["lse"], a["rest"], None)
    _sizes(call)
    assert call(k=0) == 1 and call(k=257) == 3 and call(mode=2) == 1 and call(mode=-1) == 1
    assert call(ids=None) == 1 and call(t=None) == 1 and call(loss=None) == 1
    assert call(t=A2 + 2) == 2 and call(lse=A4 + 1) == 2
    assert call(loss=A1 + 40) == 7 and call(lse=A3 + 8) == 7 and call(loss=A0 + 10 * 4) == 7

    ok2 = dict(x=A0, dtype=1, M=4, V=100, ld=104, scale=1.0, ids=A1, t=A2, k=3, mode=mode, lse=A3, rest=A4, dl=A5,
               dx=A6, ldd=100)

    def back(**o):
        a = {**ok2, **o}
        return nv.lib().topk_distill_backward(a["x"], a["dtype"], a["M"], a["V"], a["ld"], a["scale"], a["ids"],
                                              a["t"], a["k"], a["mode"], a["lse"], a["rest"], a["dl"], a["dx"],
                                              a["ldd"], None)
    _sizes(lambda **o: back(**{"dtype": 0, **o}))
    assert back(k=0) == 1 and back(k=257) == 3 and back(mode=2) == 1
    assert back(lse=None) == 1 and back(dl=None) == 1 and back(dx=None) == 1 and back(ids=None) == 1
    if mode == nv.DISTILL_TAIL:
        assert back(rest=None) == 1
    assert back(dx=A6 + 2) == 2 and back(dl=A5 + 2) == 2
    assert back(dx=A0) == 7 and back(dx=A1) == 7


def test_binding_refuses_cpu_and_wrong_tensors(nv):
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        nv.token_logprobs(x)
    with pytest.raises(ValueError):
        nv.topk_distill(x, torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1))
    # the checks that need no GPU, by the helpers that every call uses (a tensor that says it is on device 0)
    class OnGpu:
        def __init__(self, t):
            self.t = t

        def get_device(self):
            return 0

        def __getattr__(self, name):
            return getattr(self.t, name)
    for bad in (x.half(), x.to(torch.int16)):
        with pytest.raises(TypeError):
            nv._logit_rows(OnGpu(bad))
    for bad in (x, OnGpu(x[0]), OnGpu(x.t()), OnGpu(x[:, ::2]), OnGpu(x[:1].expand(3, 8))):
        with pytest.raises(ValueError):
            nv._logit_rows(bad)
    assert nv._logit_rows(OnGpu(torch.zeros(3, 9)[:, 1:6])) == (nv.F32, 3, 5, 9, 0)
    assert nv._logit_rows(OnGpu(torch.zeros(1, 9).bfloat16()[:, :6])) == (nv.BF16, 1, 6, 9, 0)
    ok = OnGpu(torch.zeros(2, dtype=torch.int32))
    assert nv._row_array(ok, "tokens", torch.int32, (2,), 0) == ok.t.data_ptr()
    assert nv._row_array(None, "tokens", torch.int32, (2,), 0) is None
    for bad in (torch.zeros(2, dtype=torch.int64), torch.zeros(3, dtype=torch.int32),
                torch.zeros(4, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError):
            nv._row_array(OnGpu(bad), "tokens", torch.int32, (2,), 0)
    with pytest.raises(ValueError):
        nv._row_array(ok, "tokens", torch.int32, (2,), 1)  # another device than the logits'
