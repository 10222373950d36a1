"""The host side of nucleus_sample_given and nucleus_spec_verify_given: bad
arguments are refused before anything is launched (the addresses below are
never dereferenced), and the binding's checks of tensors."""
import ctypes

import pytest
import torch

EINVAL, EWORKSPACE = -1, -2
A = [1 << (20 + i) for i in range(12)]


@pytest.fixture(scope="module")
def L():
    import nucleus_sampling_amd as ns

    return ns.lib()


def _opt(**kw):
    import nucleus_sampling_amd as ns

    o = ns._Options()
    for k, v in kw.items():
        setattr(o, k, v)
    return ctypes.byref(o)


def _sample(L, x=A[0], B=2, V=8, T=A[1], P=A[2], K=None, MP=None, U=A[3], ud=0, N=1, tok=A[4], cnt=A[5], lp=None,
            pr=None, opt=None):
    return L.nucleus_sample_given(x, B, V, T, P, K, MP, U, ud, N, tok, cnt, lp, pr, opt)


def _verify(L, P=A[0], Q=A[1], D=A[2], B=2, V=8, U=A[3], ud=0, tok=A[4], acc=A[5], opt=None):
    return L.nucleus_spec_verify_given(P, Q, D, B, V, U, ud, tok, acc, opt)


OTHERS = (dict(flags=1), dict(seeds=A[9]), dict(out_min_kept_logit=A[9]), dict(out_logprobs=A[9]),
          dict(allowed_mask=A[9]), dict(history=A[9], history_len=4), dict(repetition_penalty=A[9]),
          dict(frequency_penalty=A[9]), dict(presence_penalty=A[9]), dict(split_give_up_row=1))


def test_sample_given_argument_errors(L):
    for kw in (dict(x=None), dict(T=None), dict(P=None), dict(U=None), dict(tok=None), dict(cnt=None), dict(B=-1),
               dict(B=1 << 31), dict(V=0), dict(V=1 << 31), dict(N=0), dict(N=-1), dict(N=1 << 31), dict(ud=1),
               dict(ud=2), dict(x=A[0] + 2), dict(T=A[1] + 1), dict(P=A[2] + 2), dict(K=A[6] + 2), dict(MP=A[6] + 1),
               dict(U=A[3] + 2), dict(U=A[3] + 4, ud=3), dict(tok=A[4] + 2), dict(cnt=A[5] + 1), dict(lp=A[6] + 2),
               dict(pr=A[6] + 2)):
        assert _sample(L, **kw) == EINVAL, kw
    for kw in (dict(dtype=3), dict(dtype=-1), dict(row_stride=7), dict(row_stride=-8), *OTHERS):
        assert _sample(L, opt=_opt(**kw)) == EINVAL, kw
    assert _sample(L, B=0) == 0
    assert _sample(L, B=0, x=None, T=None, P=None, U=None, tok=None, cnt=None) == 0


def test_spec_verify_given_argument_errors(L):
    ws = dict(workspace=1 << 40, workspace_bytes=1 << 20)
    for kw in (dict(P=None), dict(Q=None), dict(D=None), dict(U=None), dict(tok=None), dict(B=-1), dict(V=0),
               dict(V=1 << 31), dict(ud=1), dict(ud=-1), dict(P=A[0] + 2), dict(Q=A[1] + 1), dict(D=A[2] + 2),
               dict(U=A[3] + 2), dict(U=A[3] + 4, ud=3), dict(tok=A[4] + 2), dict(acc=A[5] + 2)):
        assert _verify(L, opt=_opt(**ws), **kw) == EINVAL, kw
    for kw in (dict(dtype=1), dict(dtype=2), dict(row_stride=9), *OTHERS):
        assert _verify(L, opt=_opt(**ws, **kw)) == EINVAL, kw
    assert _verify(L, B=1 << 20, V=1 << 30, opt=_opt(**ws)) == EINVAL  # more chunks than a grid holds
    assert _verify(L, V=40000) == EWORKSPACE
    assert _verify(L, V=40000, opt=_opt(workspace=1 << 40, workspace_bytes=255)) == EWORKSPACE
    assert _verify(L, V=40000, opt=_opt(workspace=(1 << 40) + 128, workspace_bytes=4096)) == EWORKSPACE
    assert _verify(L, B=0) == 0


def test_spec_given_workspace(L):
    assert L.nucleus_spec_given_workspace_bytes(256, 128256) == 256 * 16 * 8
    assert L.nucleus_spec_given_workspace_bytes(1, 32769) == 256
    assert L.nucleus_spec_given_workspace_bytes(500, 32768) == 0  # short rows need none
    assert L.nucleus_spec_given_workspace_bytes(0, 8) == 0
    assert L.nucleus_spec_given_workspace_bytes(-1, 8) == 0 and L.nucleus_spec_given_workspace_bytes(2, 0) == 0


def test_sample_given_workspace(L):
    """Long rows of smaller batches are split, if a workspace is given; one
    that is too small or off its boundary is refused."""
    size = L.nucleus_given_workspace_bytes
    assert size(0, 128256, 0) == 0 and size(4, 0, 0) == 0 and size(4, 128256, 3) == 0
    assert size(15, 1024, 0) == 0 and size(1, 128256, 0) > 0
    assert size(4, 128256, 0) > size(1, 128256, 0)
    need = size(2, 128256, 0)
    assert _sample(L, V=128256, opt=_opt(workspace=1 << 40, workspace_bytes=need - 1)) == EWORKSPACE
    assert _sample(L, V=128256, opt=_opt(workspace=(1 << 40) + 128, workspace_bytes=need)) == EWORKSPACE


def test_the_other_entry_points_refuse_16_bit_floats(L):
    """NUCLEUS_F16 is the new calls' alone."""
    o = _opt(dtype=2)
    assert L.nucleus_sample(A[0], 2, 8, A[1], A[2], None, None, ctypes.c_uint64(0), ctypes.c_uint64(0), A[3], A[4],
                            None, o) == EINVAL
    assert L.nucleus_sample_rejection(A[0], 2, 8, A[1], A[2], None, ctypes.c_uint64(0), ctypes.c_uint64(0), A[3], A[4],
                                      o) == EINVAL


def test_binding_refuses_what_it_cannot_take():
    import nucleus_sampling_amd as ns

    x = torch.zeros(2, 8)
    u = torch.zeros(2, 1)
    with pytest.raises(ns.NucleusError):
        ns.sample_given(x, 1.0, 0.9, u)  # no CPU path
    with pytest.raises(TypeError):
        ns.sample_given(x.double(), 1.0, 0.9, u)
    with pytest.raises(ns.NucleusError, match="inference"):
        ns.sample_given(x.requires_grad_(), 1.0, 0.9, u)
    with pytest.raises(ValueError):
        ns.spec_verify_given(torch.zeros(2, 8), torch.zeros(2, 8), [0, 0], torch.zeros(2, 2))


def test_sample_hidden_has_no_cpu_path():
    import nucleus_sampling_amd as ns

    with pytest.raises(ns.NucleusError):
        ns.sample_hidden(torch.zeros(2, 8), torch.zeros(16, 8), 1.0, 0.9, uniforms=torch.zeros(2, 1))
    with pytest.raises(ns.NucleusError):
        ns.sample_hidden(torch.zeros(2, 8), torch.zeros(16, 8), 1.0, 0.9)
