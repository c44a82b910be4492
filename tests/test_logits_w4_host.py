"""Host-only checks of the entry points that take logits and 4-bit weights: bad arguments
are refused before a device is touched, empty problems are answered, and a machine without
a supported GPU reports a status."""
import ctypes

import pytest
import torch

import invariant_token_logprob_gb300 as rlk

A16 = ctypes.c_void_p(1 << 20)
A4 = ctypes.c_void_p((1 << 20) + 4)
A2 = ctypes.c_void_p((1 << 20) + 2)
A1 = ctypes.c_void_p((1 << 20) + 1)


@pytest.fixture(scope="module")
def L():
    from invariant_token_logprob_gb300 import _build
    _build.build()
    return rlk.lib()


def fwd(L, x=A16, dtype=0, stride=100, tg=A16, bits=None, bstride=0, T=4, V=100, it=1.0, k=2, out=A16, ids=A16):
    return L.rlk_token_logprobs(x, dtype, stride, tg, bits, bstride, T, V, ctypes.c_float(it), k, out, out, out,
                                ids, ids, None)


def bwd(L, x=A16, dtype=0, stride=100, tg=A16, T=4, V=100, it=1.0, lse=A16, ent=A16, g=A16, ids=A16, k=2, out=A4,
        ostride=100):
    return L.rlk_token_logprobs_backward(x, dtype, stride, tg, None, 0, T, V, ctypes.c_float(it), lse, ent, g, g, g,
                                         ids, ids, k, out, ostride, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=3), 1), (dict(dtype=-1), 1), (dict(T=-1), 1), (dict(V=0), 1), (dict(V=1 << 31, stride=1 << 31), 1),
    (dict(T=1 << 31), 1), (dict(it=0.0), 1), (dict(it=float("nan")), 1), (dict(it=float("inf")), 1), (dict(k=-1), 1),
    (dict(k=33), 1), (dict(stride=99), 1), (dict(stride=1 << 61), 1), (dict(x=None), 1), (dict(tg=None), 1),
    (dict(out=None), 1), (dict(ids=None), 1), (dict(x=A1), 2), (dict(x=A2, dtype=2), 2), (dict(out=A2), 2),
    (dict(bits=A16, bstride=3), 1), (dict(bits=A2, bstride=4), 2),
])
def test_forward_refusals(L, kw, expect):
    assert fwd(L, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=7), 1), (dict(V=-2), 1), (dict(stride=5), 1), (dict(ostride=99), 1), (dict(lse=None), 1),
    (dict(ent=None), 1), (dict(out=None), 1), (dict(ids=None), 1), (dict(k=40), 1), (dict(out=A1), 2),
    (dict(lse=A2), 2), (dict(out=A16, ostride=104), 1),
])
def test_backward_refusals(L, kw, expect):
    assert bwd(L, **kw) == expect


def linear(L, x=A16, dtype=0, c=A16, s=A16, T=2, N=10, K=64, group=32, y=A16, odt=2):
    return L.rlk_linear_w4(x, dtype, c, s, None, T, N, K, group, y, odt, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=2), 1), (dict(odt=1), 1), (dict(odt=5), 1), (dict(T=-1), 1), (dict(N=-1), 1), (dict(K=0), 1),
    (dict(K=48), 2), (dict(group=16), 1), (dict(group=0), 1), (dict(N=1 << 31), 1), (dict(N=1 << 30, K=1 << 20), 1),
    (dict(T=1 << 30, N=1 << 20), 1),
    (dict(x=None), 1), (dict(c=None), 1), (dict(s=None), 1), (dict(y=None), 1), (dict(x=A4), 2), (dict(c=A4), 2),
    (dict(s=A4), 2), (dict(y=A2), 2),
])
def test_linear_refusals(L, kw, expect):
    assert linear(L, **kw) == expect


def test_quantize_refusals(L):
    q, d = L.rlk_quantize_w4, L.rlk_dequantize_w4
    assert q(A16, 2, 4, 64, 32, A16, A16, None, None) == 1
    assert q(A16, 0, 4, 72, 32, A16, A16, None, None) == 2
    assert q(None, 0, 4, 64, 32, A16, A16, None, None) == 1
    assert q(A4, 0, 4, 64, 32, A16, A16, None, None) == 2
    assert q(None, 0, 0, 64, 32, None, None, None, None) == 0
    assert d(A16, A16, None, 0, 4, 64, 32, A16, 1, None) == 1
    assert d(A16, A16, None, 0, 4, 64, 32, None, 0, None) == 1
    assert d(None, None, None, 0, 0, 64, 32, None, 0, None) == 0


def test_empty_problems_and_no_gpu(L):
    assert fwd(L, T=0, x=None, tg=None, out=None, ids=None) == 0
    assert bwd(L, T=0, x=None, tg=None, out=None, ids=None, lse=None) == 0
    assert linear(L, T=0, x=None, y=None) == 0
    assert linear(L, N=0, c=None, s=None, x=None, y=None) == 0
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; covered by the gpu tests")
    assert fwd(L) == bwd(L) == linear(L) == 3
    assert L.rlk_quantize_w4(A16, 0, 4, 64, 32, A16, A16, None, None) == 3


def test_pack_and_unpack():
    q = torch.randint(0, 16, (5, 96), generator=torch.Generator().manual_seed(0)).to(torch.uint8)
    w = rlk.pack_w4(q)
    assert w.shape == (5, 12) and torch.equal(rlk.unpack_w4(w), q)
    word = int(w[2, 1]) & 0xFFFFFFFF
    for i in range(4):  # the pair (2i, 2i + 1) in the halves of a register
        pair = (word >> (4 * i)) & 0x000F000F
        assert (pair & 15, pair >> 16) == (int(q[2, 8 + 2 * i]), int(q[2, 8 + 2 * i + 1]))


def test_binding_refuses_cpu_tensors():
    x, tg = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        rlk.token_logprobs(x, tg)
    with pytest.raises(ValueError, match="CUDA"):
        rlk.linear_w4(torch.zeros(1, 32, dtype=torch.bfloat16), torch.zeros(2, 4, dtype=torch.int32),
                      torch.zeros(2, 1, dtype=torch.bfloat16), group=32)
    with pytest.raises(ValueError, match="CUDA"):
        rlk.quantize_w4(torch.zeros(2, 32, dtype=torch.bfloat16), 32)


@pytest.mark.parametrize("zeros", [A1, A2, ctypes.c_void_p((1 << 20) + 3)])
def test_linear_refuses_zero_points_off_a_word(L, zeros):
    """The product copies zero points in words of four bytes."""
    assert L.rlk_linear_w4(A16, 0, A16, A16, zeros, 2, 10, 64, 32, A16, 2, None) == 2
    assert L.rlk_linear_w4(A16, 0, A16, A16, zeros, 0, 10, 64, 32, A16, 2, None) == 0  # nothing to do
    if not torch.cuda.is_available():  # byte by byte elsewhere: any address goes on to the device's check
        assert L.rlk_linear_w4(A16, 0, A16, A16, A4, 2, 10, 64, 32, A16, 2, None) == 3
        assert L.rlk_quantize_w4(A16, 0, 4, 64, 32, A16, A16, zeros, None) == 3
        assert L.rlk_dequantize_w4(A16, A16, zeros, 0, 4, 64, 32, A16, 0, None) == 3


def test_wait_selftest_refusals(L):
    f = L.rlk_selftest_wait_timeout_w4
    assert f(A16, A16, A16, A16, 0, None) == 1 and f(A16, A16, A16, A16, 3, None) == 1
    assert f(None, A16, A16, A16, 1, None) == 1 and f(A16, A16, A16, None, 2, None) == 1
    assert f(A4, A16, A16, A16, 1, None) == 2 and f(A16, A16, A16, A2, 1, None) == 2
    if not torch.cuda.is_available():
        assert f(A16, A16, A16, A16, 1, None) == 3
