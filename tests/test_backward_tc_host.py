"""The tensor-core backwards without a GPU: the reference gradients against
automatic differentiation, and every refusal of the ABI and of the binding."""
import ctypes
import math

import numpy as np
import pytest
import torch

import attention_bwd_ref as ref
from diffusion_transformers_b200 import binattn

A = 0x10000
P = ctypes.c_void_p


def ptr(a):
    return P(a) if a else None


def test_reference_gradients_are_autograds():
    rng = np.random.default_rng(0)
    B, H, N, d, c = 2, 2, 7, 8, 0.3
    x = [torch.tensor(rng.standard_normal((B, H, N, d)), requires_grad=True) for _ in range(3)]
    bias = torch.tensor(rng.standard_normal((H, N, N)), requires_grad=True)
    dO = rng.standard_normal((B, H, N, d))
    with torch.no_grad():
        bias[1, :, 5:] = -torch.inf
    o = torch.softmax(c * x[0] @ x[1].transpose(-1, -2) + bias, -1) @ x[2]
    (o * torch.tensor(dO)).sum().backward()
    got = ref.gradients(*[t.detach().numpy() for t in x], dO, bias.detach().numpy(), c)
    for name, t in (("dq", x[0]), ("dk", x[1]), ("dv", x[2]), ("dbias", bias)):
        assert np.allclose(got[name][0], t.grad.numpy(), atol=1e-12), name
    empty = bias.detach().numpy().copy()
    empty[0, 3] = -np.inf
    got = ref.gradients(*[t.detach().numpy() for t in x], dO, empty, c)
    assert not got["dq"][0][:, 0, 3].any() and not got["dbias"][0][0, 3].any() and np.isfinite(got["dv"][0]).all()


def test_sign_words():
    d = 72
    on = np.random.default_rng(1).random((2, 3, 5, d)) < 0.5
    w = np.zeros((2, 3, 5, 3), np.uint32)
    for ch in range(d):
        w[..., ch // 32] |= on[..., ch].astype(np.uint32) << np.uint32(ch % 32)
    assert np.array_equal(ref.signs(torch.from_numpy(w.view(np.int32)), d), np.where(on, 1.0, -1.0))


def _ref(q=A, k=A, bias=None, v=A, dO=A, scale=0.1, B=1, H=2, N=16, d=64, dq=A, dk=A, dv=A, db=A, ws=A, wsb=1 << 24):
    return binattn.lib().binattn_ref_bf16_backward(ptr(q), ptr(k), ptr(bias), ptr(v), ptr(dO), ctypes.c_float(scale), B, H,
                                                   N, d, ptr(dq), ptr(dk), ptr(dv), ptr(db), ptr(ws),
                                                   ctypes.c_size_t(wsb), None)


def _bin(q=A, k=A, bias=None, v=A, dO=A, scale=0.1, B=1, H=2, N=16, d=64, dq=A, dk=A, dv=A, db=A, ws=A, wsb=1 << 24):
    return binattn.lib().binattn_backward_bf16(ptr(q), ptr(k), P(A), P(A), ptr(bias), ptr(v), ptr(dO),
                                               ctypes.c_float(scale), B, H, N, d, ptr(dv), ptr(dq), ptr(dk), ptr(db),
                                               ptr(ws), ctypes.c_size_t(wsb), None)


@pytest.mark.parametrize("f,size", [(_ref, "binattn_ref_bf16_backward_workspace_bytes"),
                                    (_bin, "binattn_backward_bf16_workspace_bytes")], ids=["ref", "binary"])
def test_refusals(f, size):
    L = binattn.lib()
    for name in ("q", "k", "v", "dO", "dq", "dk", "dv", "ws"):
        assert f(**{name: 0}) == 1, name
        assert f(**{name: A + 8}) == 4, name
    assert f(bias=A + 2) == 4 and f(db=A + 4) == 4
    assert f(scale=math.nan) == 8 and f(scale=math.inf) == 8
    assert f(N=0) == 2 and f(d=129) == 2 and f(B=300, H=300) == 2 and f(N=65536) == 2
    assert f(d=33) == 5 and f(d=4) == 5
    need = getattr(L, size)(1, 2, 16, 64, 0, 1)
    assert need > 0 and f(wsb=need - 1) == 8 and b"workspace" in L.binattn_last_error_message()


@pytest.mark.parametrize("size,bin", [("binattn_ref_bf16_backward_workspace_bytes", False),
                                      ("binattn_backward_bf16_workspace_bytes", True)])
def test_workspace_bytes(size, bin):
    f = getattr(binattn.lib(), size)
    r = lambda x: -(-x // 256) * 256  # noqa: E731
    for B, H, N, d in [(1, 1, 1, 8), (2, 16, 4096, 72), (64, 12, 197, 64), (5, 3, 136, 128)]:
        npad = -(-N // 64) * 64
        rows = r(B * H * npad * 4)
        # two row vectors, the four operands in tiles, the padded alphas
        base = 2 * rows + 4 * r(B * H * npad * (-(-d // 16) * 16) * 2) + (2 * rows if bin else 0)
        assert f(B, H, N, d, 0, 0) == base
        pad = r(H * N * (-(-N // 8) * 8) * 2) if N % 8 else 0
        pad += rows  # with a bias the row's sum is kept beside its max
        assert f(B, H, N, d, 1, 0) == base + pad
        sums = f(B, H, N, d, 1, 1) - base - pad
        nb = min(4, 256 // (-(-d // 16) * 16))
        if B <= nb:
            assert sums == 0
        else:  # a whole number of fp32 [H, N, N], no more than there are chunks
            assert any(sums == r(k * H * N * N * 4) for k in range(1, -(-B // nb) + 1))
    assert f(0, 1, 1, 8, 0, 0) == 0 and f(1, 1, 1, 12, 0, 0) == 0 and f(1, 1, 1, 136, 0, 0) == 0


def test_binding_refusals():
    B, H, N, d = 2, 3, 37, 72
    bf = dict(dtype=torch.bfloat16)
    q, v = torch.zeros(B, H, N, d, **bf), torch.zeros(B, H, N, d, **bf)
    bias = torch.zeros(H, N, N, **bf)
    qb, aq = torch.zeros(B, H, N, 3, dtype=torch.int32), torch.zeros(B, H, N)

    def raises(exc, match, fn, *a, **kw):
        with pytest.raises(exc, match=match):
            fn(*a, **kw)

    cpu = "libbinattn takes CUDA tensors"
    raises(ValueError, cpu, binattn.ref_bf16_backward, q, q, bias, v, v, 0.1)
    raises(ValueError, cpu, binattn.backward_bf16, qb, qb, aq, aq, None, v, v, 0.1)
    raises(ValueError, "k has shape", binattn.ref_bf16_backward, q, q[:1], bias, v, v, 0.1)
    raises(TypeError, "dO has dtype", binattn.ref_bf16_backward, q, q, bias, v, v.float(), 0.1)
    raises(ValueError, "bias has shape", binattn.ref_bf16_backward, q, q, bias[:1], v, v, 0.1)
    raises(ValueError, "dO has shape", binattn.backward_bf16, qb, qb, aq, aq, bias, v, v[:1], 0.1)
    raises(ValueError, "q_bits has shape", binattn.backward_bf16, qb[..., :2], qb, aq, aq, bias, v, v, 0.1)
    raises(TypeError, "bias has dtype", binattn.backward_bf16, qb, qb, aq, aq, bias.float(), v, v, 0.1)
