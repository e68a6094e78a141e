"""The norm and rotation of queries and keys, its sign-bit form and its gradient
on the GPU, against the formulas in 64 bits (norm_rope_ref)."""
import numpy as np
import pytest
import torch

import norm_rope_ref as ref
from diffusion_transformers_b200 import binattn
from norm_rope_ref import close, f64

pytestmark = pytest.mark.gpu

EPS = 1e-6


def make(B, H, N, d, rot, dtype, layout, per_batch=False, weights=True, seed=0, zeros=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if layout == "qkv":      # views of a projection's output [B, N, 3, H, d]
        buf = randn(B, N, 3, H, d).to(dtype)
        q, k = buf[:, :, 0].permute(0, 2, 1, 3), buf[:, :, 1].permute(0, 2, 1, 3)
    elif layout == "odd":    # rows at an odd distance, off any 16-byte boundary
        buf = randn(2, B, H, N, d + 1).to(dtype)
        q, k = buf[0, ..., 1:], buf[1, ..., :d]
    elif layout == "broadcast":  # one batch entry and head for all
        q, k = randn(1, 1, N, d).to(dtype).expand(B, H, N, d), randn(1, H, N, d).to(dtype).expand(B, H, N, d)
    else:
        q, k = randn(B, H, N, d).to(dtype), randn(B, H, N, d).to(dtype)
    if zeros:
        for t in (q, k):
            t[torch.rand(t.shape, generator=g, device="cuda") < zeros] = -0.0
    w = [1 + 0.3 * randn(d) if weights else None for _ in range(2)]
    cos = sin = None
    if rot:
        pos = torch.arange(N, device="cuda")
        if per_batch:
            pos = torch.stack([pos + 1000 * b for b in range(B)])[..., None]
        cos, sin = binattn.rope_tables(pos, rot)
    return q, k, w[0], w[1], cos, sin


# (B, H, N, d, rot, layout): one token, one channel, every lane count of the
# vector kernel that has a tail (d = 24 .. 120), partial rotations, the scalar
# kernel's shapes, views and broadcasts, and a DiT-XL/2 head shape
CASES = [(1, 16, 1, 64, 64, "qkv"), (1, 1, 1, 1, 0, "plain"), (1, 1, 1, 2, 2, "plain"), (2, 3, 5, 8, 8, "plain"),
         (2, 3, 7, 24, 16, "qkv"), (1, 2, 33, 40, 8, "plain"), (2, 2, 9, 120, 120, "qkv"), (3, 2, 11, 128, 64, "plain"),
         (2, 2, 13, 64, 0, "qkv"), (2, 2, 13, 72, 36, "qkv"), (1, 3, 17, 33, 32, "qkv"), (1, 3, 17, 127, 126, "plain"),
         (2, 2, 19, 64, 64, "odd"), (2, 3, 21, 72, 72, "broadcast"), (64, 3, 31, 16, 16, "qkv"), (2, 4, 1029, 72, 72, "qkv")]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True], ids=["half", "inter"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_pack(case, inter, dtype):
    B, H, N, d, rot, layout = case
    q, k, wq, wk, cos, sin = make(B, H, N, d, rot, dtype, layout, per_batch=B > 1, seed=N)
    out = binattn.norm_rope(q, k, wq, wk, cos, sin, EPS, interleaved=inter)
    packed = binattn.norm_rope_pack(q, k, wq, wk, cos, sin, EPS, interleaved=inter)
    for t, (x, w) in enumerate(((q, wq), (k, wk))):
        z, size = ref.forward(f64(x), w, cos, sin, EPS, inter)
        assert out[t].dtype == dtype and out[t].is_contiguous()
        close(out[t], z, size, d, dtype, f"z[{t}]")
        on = ref.signs(f64(x), w, cos, sin, inter)
        assert np.array_equal(packed[2 * t].cpu().numpy().view(np.uint32), ref.words(on)), f"bits[{t}]"
        close(packed[2 * t + 1], np.abs(z).mean(-1), size.mean(-1), d, torch.float32, f"alpha[{t}]")


@pytest.mark.parametrize("case", [(2, 3, 9, 64, 64, "plain"), (1, 2, 9, 30, 30, "plain")], ids=str)
@pytest.mark.parametrize("inter", [False, True], ids=["half", "inter"])
def test_pack_at_zero(case, inter):
    # products that cancel exactly (both members alike, the sine equal to the
    # cosine) and rows of zeros, of either sign, give set bits; values one step
    # apart give the sign of that step
    B, H, N, d, rot, layout = case
    q, k, _, _, cos, sin = make(B, H, N, d, rot, torch.bfloat16, layout, zeros=0.2)
    cos = torch.full_like(cos, 0.70710677)
    sin = cos.clone()
    a, b = ref.pairs(d, rot, inter)
    q[..., b] = q[..., a]
    q[0, 0, 0] = 0.0
    q[0, 0, 1] = -0.0
    k[..., b] = (k[..., a].view(torch.int16) + 1).view(torch.bfloat16)  # one step further from zero
    k[..., 1, :] = -k[..., 1, :]
    w = torch.full((d,), 0.37, device="cuda")
    packed = binattn.norm_rope_pack(q, k, w, w, cos, sin, EPS, interleaved=inter)
    for t, x in enumerate((q, k)):
        on = ref.signs(f64(x), w, cos, sin, inter)
        assert np.array_equal(packed[2 * t].cpu().numpy().view(np.uint32), ref.words(on))
    assert (packed[0][0, 0, :2].cpu() == torch.tensor(ref.words(np.ones((1, d), bool)).view(np.int32))).all()
    assert (packed[1][0, 0, :2] == 0).all()


@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32], ids=["gbf16", "gf32"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True], ids=["half", "inter"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case, inter, dtype, grad):
    B, H, N, d, rot, layout = case
    q, k, wq, wk, cos, sin = make(B, H, N, d, rot, dtype, layout, per_batch=B > 1, seed=N + 1)
    g = torch.Generator(device="cuda").manual_seed(7)
    dz = [torch.randn(B, H, N, d, generator=g, device="cuda").to(grad) for _ in range(2)]
    got = binattn.norm_rope_backward(q, k, *dz, wq, wk, cos, sin, EPS, interleaved=inter)
    rows = B * H * N
    for t, (x, w) in enumerate(((q, wq), (k, wk))):
        dx, sx, dw, sw = ref.backward(f64(x), f64(dz[t]), w, cos, sin, EPS, inter)
        close(got[t], dx, sx, d, dtype, f"dx[{t}]")
        # dw: each row's product, then chains of at most rows additions in all
        close(got[2 + t], dw, sw, d, torch.float32, f"dw[{t}]", steps=rows)


def test_backward_into_the_projections_gradient():
    # dq and dk as views of one [B, N, 3, H, d] buffer; what lies between them
    # (the gradient of V) stays as it was, and the sums are the same bits twice
    B, H, N, d = 2, 3, 37, 72
    q, k, wq, wk, cos, sin = make(B, H, N, d, d, torch.bfloat16, "qkv")
    dz = [torch.randn(B, H, N, d, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    want = binattn.norm_rope_backward(q, k, *dz, wq, wk, cos, sin, EPS)
    buf = torch.full((B, N, 3, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    views = [buf[:, :, t].permute(0, 2, 1, 3) for t in range(2)]
    got = binattn.norm_rope_backward(q, k, *dz, wq, wk, cos, sin, EPS, dq=views[0], dk=views[1])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert (buf[:, :, 2] == 7.0).all()


def test_no_weights_and_no_rotation():
    B, H, N, d = 2, 2, 5, 72
    q, k, *_ = make(B, H, N, d, 0, torch.bfloat16, "plain", weights=False)
    dz = [torch.randn(B, H, N, d, device="cuda") for _ in range(2)]
    z = binattn.norm_rope(q, k, None, None, None, None)
    dq, dk, dwq, dwk = binattn.norm_rope_backward(q, k, *dz, None, None, None, None)
    assert dwq is None and dwk is None
    for got, x in ((z[0], q), (z[1], k)):
        ref_z, size = ref.forward(f64(x), None, None, None, EPS, False)
        close(got, ref_z, size, d, torch.bfloat16, "z")
    close(dq, *ref.backward(f64(q), f64(dz[0]), None, None, None, EPS, False)[:2], d, torch.bfloat16, "dq")
    # one weight only: the other gradient is skipped
    w = torch.ones(d, device="cuda")
    _, _, dwq, dwk = binattn.norm_rope_backward(q, k, *dz, None, w, None, None)
    assert dwq is None
    close(dwk, *ref.backward(f64(k), f64(dz[1]), w, None, None, EPS, False)[2:], d, torch.float32, "dw_k", steps=20)


def test_another_stream_and_a_replayed_graph():
    B, H, N, d = 2, 3, 129, 64
    q, k, wq, wk, cos, sin = make(B, H, N, d, d, torch.bfloat16, "plain")
    dz = [torch.randn(B, H, N, d, device="cuda", dtype=torch.bfloat16) for _ in range(2)]

    def step(stream=None):
        return (*binattn.norm_rope(q, k, wq, wk, cos, sin, stream=stream),
                *binattn.norm_rope_pack(q, k, wq, wk, cos, sin, stream=stream),
                *binattn.norm_rope_backward(q, k, *dz, wq, wk, cos, sin, stream=stream))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    q.copy_(torch.randn_like(q))
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(held, step()))


@pytest.mark.parametrize("backward", [binattn.backward, binattn.backward_bf16])
def test_through_the_binary_attention(backward):
    # projection -> norm, rotation and sign bits -> binary attention -> its
    # backward -> the projection's gradient (straight-through), against the
    # same chain in 64 bits from the kernels' own bits and alphas
    B, H, N, d = 2, 2, 65, 64
    q, k, wq, wk, cos, sin = make(B, H, N, d, d, torch.bfloat16, "qkv")
    v, dO = (torch.randn(B, H, N, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    scale = d ** -0.5
    qb, aq, kb, ak = binattn.norm_rope_pack(q, k, wq, wk, cos, sin)
    o = binattn.forward(qb, kb, aq, ak, None, v, scale)
    dV, ds, dt, _ = backward(qb, kb, aq, ak, None, v, dO, scale, with_dbias=False)
    # fp32 gradients are good to 2e-4; bf16 ones are off by two half steps (dlogit, the result)
    tol = 2e-4 if dV.dtype == torch.float32 else 2 * 2.0 ** -8
    dq, dk, dwq, dwk = binattn.norm_rope_backward(q, k, ds, dt, wq, wk, cos, sin)
    s, t = (torch.tensor(np.where(ref.signs(f64(x), w, cos, sin, False), 1.0, -1.0)
                         * np.abs(ref.forward(f64(x), w, cos, sin, EPS, False)[0]).mean(-1, keepdims=True))
            for x, w in ((q, wq), (k, wk)))
    s.requires_grad_(), t.requires_grad_()
    vv = v.cpu().double().requires_grad_()
    out = torch.softmax(scale * s @ t.transpose(-1, -2), -1) @ vv
    (out * dO.cpu().double()).sum().backward()
    # P is rounded to bf16 in the forward, O is stored in bf16: two half steps
    assert (o.cpu().double() - out).norm() <= 2 * 2.0 ** -8 * out.norm()
    assert (dV.cpu().double() - vv.grad).norm() <= tol * vv.grad.norm()
    for x, w, g, dx, dw in ((q, wq, s.grad, dq, dwq), (k, wk, t.grad, dk, dwk)):
        rx, _, rw, _ = ref.backward(f64(x), g.numpy(), w, cos, sin, EPS, False)
        # the attention's gradients, then half a step of bf16
        assert np.linalg.norm(f64(dx) - rx) <= (2.0 ** -8 + 2 * tol) * np.linalg.norm(rx)
        assert np.linalg.norm(f64(dw) - rw) <= 2 * tol * np.linalg.norm(rw)


def test_past_32_bits():
    # more than 2^31 elements: the last rows against the formulas
    B, H, N, d = 8, 40, 65535, 104
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.empty(B, H, N, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    assert q.numel() > 2 ** 31
    cos, sin = binattn.rope_tables(torch.arange(N, device="cuda"), d)
    w = torch.ones(d, device="cuda")
    z, _ = binattn.norm_rope(q, q, w, w, cos, sin)
    bits, alpha, _, _ = binattn.norm_rope_pack(q, q, w, w, cos, sin)
    x = q[-1:, -1:, -5:]
    want, size = ref.forward(f64(x), w, cos[-5:], sin[-5:], EPS, False)
    close(z[-1:, -1:, -5:], want, size, d, torch.bfloat16, "z")
    assert np.array_equal(bits[-1:, -1:, -5:].cpu().numpy().view(np.uint32), ref.words(ref.signs(f64(x), w, cos[-5:], sin[-5:], False)))
    close(alpha[-1:, -1:, -5:], np.abs(want).mean(-1), size.mean(-1), d, torch.float32, "alpha")
    dq, _, dw, _ = binattn.norm_rope_backward(q, q, z, z, w, w, cos, sin)
    dx, sx, _, _ = ref.backward(f64(x), f64(z[-1:, -1:, -5:]), w, cos[-5:], sin[-5:], EPS, False)
    close(dq[-1:, -1:, -5:], dx, sx, d, torch.bfloat16, "dx")
    assert torch.isfinite(dw).all()


def test_through_the_bf16_attention():
    # projection -> norm and rotation -> bf16 attention -> its backward -> the
    # projection's gradient, against the same chain in 64 bits
    B, H, N, d = 2, 2, 65, 64
    q, k, wq, wk, cos, sin = make(B, H, N, d, d, torch.bfloat16, "qkv", seed=5)
    v, dO = (torch.randn(B, H, N, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    scale = d ** -0.5
    zq, zk = binattn.norm_rope(q, k, wq, wk, cos, sin)
    o = binattn.ref_bf16_forward(zq, zk, None, v, scale)
    dzq, dzk, dv, _ = binattn.ref_bf16_backward(zq, zk, None, v, dO, scale, with_dbias=False)
    dq, dk, _, _ = binattn.norm_rope_backward(q, k, dzq, dzk, wq, wk, cos, sin)
    s, t, vv = (x.cpu().double().requires_grad_() for x in (zq, zk, v))
    out = torch.softmax(scale * s @ t.transpose(-1, -2), -1) @ vv
    (out * dO.cpu().double()).sum().backward()
    assert (o.cpu().double() - out).norm() <= 2 * 2.0 ** -8 * out.norm()
    assert (dv.cpu().double() - vv.grad).norm() <= 2 * 2.0 ** -8 * vv.grad.norm()
    for x, w, gz, dx in ((q, wq, s.grad, dq), (k, wk, t.grad, dk)):
        want, _, _, _ = ref.backward(f64(x), gz.numpy(), w, cos, sin, EPS, False)
        # dlogit rounded, the attention's gradient rounded, this one rounded: half a step each
        assert np.linalg.norm(f64(dx) - want) <= 3 * 2.0 ** -8 * np.linalg.norm(want)
