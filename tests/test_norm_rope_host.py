"""The norm and rotation of queries and keys without a GPU: the tables, the
reference formulas against differences, and every refusal of the ABI and of the
binding."""
import ctypes
import math

import numpy as np
import pytest
import torch

import norm_rope_ref as ref
from diffusion_transformers_b200 import binattn

A = 0x10000  # aligned fake device addresses: never dereferenced by refused calls
P = ctypes.c_void_p


def ptr(a):
    return P(a) if a else None


def test_rope_tables():
    c, s = binattn.rope_tables(torch.arange(5), 8)
    assert c.shape == s.shape == (5, 4) and c.dtype == torch.float32
    ang = np.arange(5)[:, None] * 10000.0 ** (-np.arange(4) / 4)
    assert np.array_equal(c.numpy(), np.cos(ang).astype(np.float32))
    assert np.array_equal(s.numpy(), np.sin(ang).astype(np.float32))
    # a patch grid: the first half of the pairs turns by the row, the second by the column
    yx = torch.stack(torch.meshgrid(torch.arange(3), torch.arange(4), indexing="ij"), -1).view(12, 2)
    c2, _ = binattn.rope_tables(yx, 8, theta=100.0)
    f = 100.0 ** (-np.arange(2) / 2)
    want = np.cos(np.concatenate([yx[:, :1].numpy() * f, yx[:, 1:].numpy() * f], 1)).astype(np.float32)
    assert np.array_equal(c2.numpy(), want)
    assert binattn.rope_tables(yx[None].expand(2, 12, 2), 8)[0].shape == (2, 12, 4)
    # far positions keep their angle (64 bits): position 2^40, lowest frequency
    c3, _ = binattn.rope_tables(torch.tensor([2 ** 40]), 2)
    assert c3.item() == np.float32(math.cos(2.0 ** 40))
    assert binattn.rope_tables(torch.arange(3), 0)[0].shape == (3, 0)
    with pytest.raises(ValueError, match="rot"):
        binattn.rope_tables(yx, 6)


@pytest.mark.parametrize("inter", [False, True])
def test_reference_gradient_is_the_difference_quotient(inter):
    rng = np.random.default_rng(0)
    B, H, N, d, rot, eps = 2, 2, 3, 10, 6, 1e-3
    x, dz = rng.standard_normal((2, B, H, N, d))
    w = torch.tensor(rng.standard_normal(d))
    cos, sin = binattn.rope_tables(torch.arange(N) + 3, rot)
    dx, _, dw, _ = ref.backward(x, dz, w, cos, sin, eps, inter)

    def loss(x, w):
        return float((ref.forward(x, torch.tensor(w), cos, sin, eps, inter)[0] * dz).sum())

    h = 1e-6
    for _ in range(20):
        at = tuple(rng.integers(0, n) for n in x.shape)
        e = np.zeros_like(x)
        e[at] = h
        assert abs((loss(x + e, w.numpy()) - loss(x - e, w.numpy())) / (2 * h) - dx[at]) < 1e-7
    for ch in range(d):
        e = np.zeros(d)
        e[ch] = h
        assert abs((loss(x, w.numpy() + e) - loss(x, w.numpy() - e)) / (2 * h) - dw[ch]) < 1e-7


def _fwd(q=A, k=A, dt=1, st=None, wq=A, wk=A, c=A, s=A, rot=8, eps=1e-6, B=1, H=2, N=4, d=16, o1=A, o2=A, pack=False):
    L = binattn.lib()
    strides = (ctypes.c_int64 * 6)(*st) if st else None
    head = [ptr(q), ptr(k), dt, strides, ptr(wq), ptr(wk), ptr(c), ptr(s), rot, 0, 0, ctypes.c_float(eps), B, H, N, d]
    if pack:
        return L.binattn_norm_rope_pack(*head, ptr(o1), P(A), P(A), ptr(o2), None)
    return L.binattn_norm_rope(*head, ptr(o1), ptr(o2), None)


@pytest.mark.parametrize("pack", [False, True])
def test_forward_refusals(pack):
    f = lambda **kw: _fwd(pack=pack, **kw)  # noqa: E731
    assert f(q=0) == 1 and f(k=0) == 1 and f(o1=0) == 1 and f(o2=0) == 1
    assert f(c=0) == 1 and f(s=0) == 1
    assert f(dt=2) == 3
    assert f(q=A + 1) == 4 and f(k=A + 1) == 4 and f(q=A + 2, dt=0) == 4
    assert f(wq=A + 4) == 4 and f(wk=A + 4) == 4 and f(c=A + 4) == 4 and f(o1=A + 8) == 4
    assert f(N=0) == 2 and f(d=129) == 2 and f(d=0) == 2 and f(B=300, H=300) == 2 and f(N=65536) == 2
    assert f(rot=7) == 2 and f(rot=18) == 2 and f(rot=-2) == 2
    assert f(eps=0.0) == 8 and f(eps=-1.0) == 8 and f(eps=math.nan) == 8 and f(eps=math.inf) == 8
    assert f(B=2, st=[-1, 64, 16, 128, 64, 16]) == 8
    assert b"negative" in binattn.lib().binattn_last_error_message()


def _bwd(q=A, g1=A, gdt=1, dq=A, dk=A, gst=None, dwq=A, ws=A, wsb=1 << 20, B=2, H=2, N=4, d=16, dt=1):
    st = (ctypes.c_int64 * 6)(*gst) if gst else None
    return binattn.lib().binattn_norm_rope_backward(
        ptr(q), P(A), dt, None, ptr(g1), P(A), gdt, P(A), P(A), P(A), P(A), 8, 0, 0, ctypes.c_float(1e-6), B, H, N, d,
        ptr(dq), ptr(dk), st, ptr(dwq), P(A), ptr(ws), ctypes.c_size_t(wsb), None)


def test_backward_refusals():
    assert _bwd(q=0) == 1 and _bwd(g1=0) == 1 and _bwd(dq=0) == 1 and _bwd(dk=0) == 1
    assert _bwd(gdt=9) == 3 and _bwd(dt=9) == 3
    assert _bwd(g1=A + 8) == 4 and _bwd(dq=A + 1) == 4 and _bwd(dwq=A + 4) == 4 and _bwd(ws=A + 8) == 4
    assert _bwd(N=0) == 2
    assert _bwd(ws=0) == 1
    need = binattn.lib().binattn_norm_rope_backward_workspace_bytes(2, 2, 4, 16)
    assert need >= 2 * 2 * 16 * 4 and _bwd(wsb=need - 1) == 8
    # rows of dq or dk that share elements: a token stride below d, a stride of 0,
    # heads inside a token's row
    ok = [128, 64, 16]
    for bad in ([128, 64, 15], [0, 64, 16], [128, 8, 32], [128, 0, 16]):
        assert _bwd(gst=bad + ok) == 8 and _bwd(gst=ok + bad) == 8
        assert b"overlap" in binattn.lib().binattn_last_error_message()
    assert binattn.lib().binattn_norm_rope_backward_workspace_bytes(0, 2, 4, 16) == 0
    assert binattn.lib().binattn_norm_rope_backward_workspace_bytes(1, 2, 4, 129) == 0


def test_binding_refusals():
    B, H, N, d = 2, 3, 5, 16
    bf = torch.bfloat16
    q, k = torch.zeros(B, H, N, d, dtype=bf), torch.zeros(B, H, N, d, dtype=bf)
    w = torch.ones(d)
    c, s = binattn.rope_tables(torch.arange(N), d)

    def raises(exc, match, fn, *a, **kw):
        with pytest.raises(exc, match=match):
            fn(*a, **kw)

    cpu = "libbinattn takes CUDA tensors"
    for fn in (binattn.norm_rope, binattn.norm_rope_pack):
        raises(ValueError, cpu, fn, q, k, w, w, c, s)
        raises(ValueError, cpu, fn, q, k, None, None, None, None)
        raises(ValueError, cpu, fn, q, k, w, w, c.expand(B, N, d // 2), s.expand(B, N, d // 2))
        raises(TypeError, "float32 or bfloat16", fn, q.half(), k, w, w, c, s)
        raises(TypeError, "k has dtype", fn, q, k.float(), w, w, c, s)
        raises(ValueError, "k has shape", fn, q, k[:, :2], w, w, c, s)
        raises(ValueError, "w_q has shape", fn, q, k, w[:3], w, c, s)
        raises(TypeError, "w_k has dtype", fn, q, k, w, w.to(bf), c, s)
        raises(ValueError, "cos has shape", fn, q, k, w, w, c[:3], s)
        raises(ValueError, "sin has shape", fn, q, k, w, w, c, s[:, :3])
        raises(ValueError, "go together", fn, q, k, w, w, c, None)
        raises(ValueError, "last stride", fn, q.transpose(2, 3).contiguous().transpose(2, 3), k, w, w, c, s)
        raises(ValueError, r"\[B, H, N, d\]", fn, q[0], k, w, w, c, s)
    raises(ValueError, "q_out has shape", binattn.norm_rope, q, k, w, w, c, s, q_out=q[:1])
    raises(ValueError, cpu, binattn.norm_rope_backward, q, k, q, k, w, w, c, s)
    raises(TypeError, "upstream", binattn.norm_rope_backward, q, k, q.half(), k.half(), w, w, c, s)
    raises(TypeError, "dk_out has dtype", binattn.norm_rope_backward, q, k, q.float(), k, w, w, c, s)
    raises(ValueError, "dq has shape", binattn.norm_rope_backward, q, k, q, k, w, w, c, s, dq=q[:1])
