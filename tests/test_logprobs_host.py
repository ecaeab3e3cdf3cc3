"""Arguments that spec_token_logprobs and its gradient refuse, on the host (no kernel is launched)."""

import pytest

EINVAL, EWORKSPACE, EUNSUPPORTED = -1, -2, -4
FAKE = 0x7F0000000000  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def L():
    import rejection_sampling_verify_10_amd as R
    return R.lib()


def forward(L, **kw):
    a = dict(z=FAKE, dtype=1, stride=1000, R=4, V=1000, tok=FAKE, M=1, T=1.0, top=5, lp=FAKE, h=FAKE, st=FAKE, ids=FAKE,
             tlp=FAKE, ws=FAKE, wsb=0, stream=None)
    a.update(kw)
    return L.spec_token_logprobs(*a.values())


def backward(L, **kw):
    a = dict(z=FAKE, dtype=1, stride=1000, R=4, V=1000, tok=FAKE, M=1, st=FAKE, g=FAKE, gh=None, T=1.0, out=FAKE + 4096,
             ostride=1000, stream=None)
    a.update(kw)
    return L.spec_token_logprobs_grad(*a.values())


BOTH = [dict(z=None), dict(dtype=2), dict(R=0), dict(V=0), dict(M=-1), dict(tok=None), dict(tok=FAKE + 2), dict(z=FAKE + 1),
        dict(stride=999), dict(T=0.0), dict(T=-1.0), dict(T=float("nan")), dict(T=float("inf")), dict(T=1e-39)]


@pytest.mark.parametrize("bad", BOTH + [dict(top=-1), dict(lp=None), dict(ids=None), dict(tlp=None), dict(lp=FAKE + 2),
                                        dict(h=FAKE + 1), dict(st=FAKE + 2), dict(ids=FAKE + 1), dict(tlp=FAKE + 3)])
def test_forward_refuses(L, bad):
    assert forward(L, **bad) == EINVAL


@pytest.mark.parametrize("bad", BOTH + [dict(M=0), dict(st=None), dict(g=None), dict(out=None), dict(ostride=999),
                                        dict(gh=FAKE + 2), dict(out=FAKE + 4097), dict(out=FAKE, ostride=1001)])
def test_backward_refuses(L, bad):
    assert backward(L, **bad) == EINVAL


@pytest.mark.parametrize("bad", [dict(V=(1 << 20) + 1, stride=1 << 21), dict(M=65), dict(stride=1 << 41),
                                 dict(R=1 << 24, V=1 << 20, stride=1 << 20)])
def test_past_the_limits(L, bad):
    ostride = {"ostride": bad["stride"]} if "stride" in bad else {}
    assert forward(L, **bad) == EUNSUPPORTED and backward(L, **bad, **ostride) == EUNSUPPORTED


def test_top_past_its_limit(L):
    assert forward(L, top=65) == EUNSUPPORTED


def test_workspace(L):
    need = L.spec_token_logprobs_workspace_bytes(1, 128256, 5, 1)
    assert need > 0
    long = dict(R=1, V=128256, stride=128256)
    assert forward(L, wsb=need - 1, **long) == EWORKSPACE
    assert forward(L, ws=None, wsb=need, **long) == EWORKSPACE
    assert forward(L, ws=FAKE + 16, wsb=need, **long) == EWORKSPACE
    assert L.spec_token_logprobs_workspace_bytes(4, 1000, 5, 2) == 0
    assert L.spec_token_logprobs_workspace_bytes(0, 1000, 5, 1) == 0
    assert L.spec_token_logprobs_workspace_bytes(4, 1000, 65, 1) == 0
    assert L.spec_token_logprobs_workspace_bytes(4000, 32000, 5, 1) == 0      # a workgroup a row: nothing to join


def test_binding_refuses():
    import torch
    import rejection_sampling_verify_10_amd as R
    with pytest.raises(ValueError, match="GPU"):
        R.token_logprobs(torch.zeros(2, 5), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError, match="bfloat16"):
        R.token_logprobs(torch.zeros(2, 5, dtype=torch.float16), torch.zeros(2, dtype=torch.int32))


@pytest.mark.parametrize("shape,stride,ok", [((2, 3, 5), (15, 5, 1), True), ((2, 3, 5), (24, 8, 1), True),
                                             ((2, 3, 5), (20, 5, 1), False), ((2, 1, 5), (7, 1, 1), True),
                                             ((3, 5), (4, 1), False), ((5, 3), (1, 5), False), ((0, 5), (5, 1), False),
                                             ((1, 1), (1, 9), True)])
def test_rows_at_one_distance(shape, stride, ok):
    import torch
    from rejection_sampling_verify_10_amd.logprobs import _logit_rows

    class Stand:
        dtype, is_cuda = torch.bfloat16, True

        def __init__(self):
            self.shape = torch.Size(shape)

        def dim(self):
            return len(shape)

        def stride(self, d=None):
            return stride if d is None else stride[d]

    if ok:
        n = 1
        for s in shape[:-1]:
            n *= s
        assert _logit_rows(Stand(), "logits")[0] == n
    else:
        with pytest.raises(ValueError):
            _logit_rows(Stand(), "logits")
