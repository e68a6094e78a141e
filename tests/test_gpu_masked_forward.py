"""The forwards under masks that leave rows or their first keys empty, against
the formula in 64 bits: every forward that takes a dense bias, and the gradients
that go with them."""
import numpy as np
import pytest
import torch

import attention_bwd_ref as bwd_ref
import masked_forward_ref as ref
from attention_bwd_ref import f64, signs
from diffusion_transformers_b200 import binattn

pytestmark = pytest.mark.gpu


def make(B, H, N, d, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k, v, dO = (torch.randn(B, H, N, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(4))
    return q, k, v, dO, ref.masked_bias(H, N, seed).cuda()


def binary(q, k, d):
    packed = [binattn.pack(t) for t in (q, k)]
    return packed, [signs(b, d) * f64(a)[..., None] for b, a in packed]


def check(out, want, what):
    val, bound = want
    g = f64(out)
    broken = int((~np.isfinite(g)).any(-1).sum())
    assert broken == 0, f"{what}: {broken} rows are not finite"
    bad = np.abs(g - val) > bound
    n = int(bad.sum())
    assert n == 0, f"{what}: {n} beyond the bound, first at {np.argwhere(bad)[0]}"
    assert not out[:, 3].any() and not out[:, 0, 0].any(), what  # nothing but -inf


# the TMA-fed pipeline (d <= 80), with N % 8 == 0 and padded, several tiles and
# items; wide heads; one odd N each
SHAPES = [(2, 4, 150, 72), (1, 4, 200, 64), (3, 5, 520, 72), (1, 4, 141, 128), (2, 4, 264, 96), (1, 4, 144, 16)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_binary(shape):
    B, H, N, d = shape
    q, k, v, _, bias = make(*shape, seed=N)
    ((qb, aq), (kb, ak)), (s, t) = binary(q, k, d)
    c = d ** -0.5
    want = ref.forward(s, t, f64(v), f64(bias), c)
    outs = {"forward": binattn.forward(qb, kb, aq, ak, bias, v, c), "forward_ws": binattn.forward_ws(qb, kb, aq, ak, bias, v, c),
            "fused": binattn.forward_fused_ws(q, kb, ak, bias, v, c),
            "static": binattn.forward_static_ws(qb, kb, aq, ak, bias, v, c)}
    for engine in ("simt", "popc_tc", "tc"):
        outs[engine] = binattn.forward(qb, kb, aq, ak, bias, v, c, engine=engine)
    if d <= 80:
        outs["bias_ld"] = binattn.forward_bias_ld_ws(qb, kb, aq, ak, binattn.pad_bias(bias), v, c)
        per_sample = bias[None].expand(B, H, N, N).contiguous()
        outs["sample_bias"] = binattn.forward_sample_bias_ws(qb, kb, aq, ak, per_sample, v, c)
    torch.cuda.synchronize()
    binattn.device_status()
    for name, out in outs.items():
        check(out, want, f"{name} {shape}")


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_bf16(shape):
    B, H, N, d = shape
    q, k, v, _, bias = make(*shape, seed=N + 1)
    c = d ** -0.5
    want = ref.forward(f64(q), f64(k), f64(v), f64(bias), c)
    check(binattn.ref_bf16_forward(q, k, bias, v, c), want, f"ref {shape}")
    check(binattn.ref_bf16_forward_ws(q, k, bias, v, c), want, f"ref_ws {shape}")
    binattn.device_status()


@pytest.mark.parametrize("kind", ["ref", "binary"])
def test_split_tail(kind):
    # more row pairs than SMs and 32 key tiles or more: the last pairs' key halves
    # are joined by a kernel of their own; rows with nothing in one half or in both
    B, H, N, d = 5, 4, 2048, 64
    q, k, v, _, bias = make(B, H, N, d, seed=3)
    c = d ** -0.5
    packed, st = binary(q, k, d)
    if kind == "ref":
        out, st = binattn.ref_bf16_forward_ws(q, k, bias, v, c), (f64(q), f64(k))
    else:
        (qb, aq), (kb, ak) = packed
        assert binattn.workspace_bytes(B, H, N, d, True) > 0
        out = binattn.forward_ws(qb, kb, aq, ak, bias, v, c)
    check(out, ref.forward(*st, f64(v), f64(bias), c), f"split {kind}")
    # the split pairs are the last head's: move the masks there
    bias = bias.flip(0).contiguous()
    if kind == "ref":
        out = binattn.ref_bf16_forward_ws(q, k, bias, v, c)
    else:
        out = binattn.forward_ws(qb, kb, aq, ak, bias, v, c)
    check(out.flip(1), [t[:, ::-1] for t in ref.forward(*st, f64(v), f64(bias), c)], f"split {kind} flipped")


@pytest.mark.parametrize("kind", ["ref", "binary"])
def test_a_masked_training_step(kind):
    # forward and backward of the same masked rows: sum O dO is what dV says it
    # is, and the gradients are those of the 64-bit forward
    B, H, N, d = 2, 4, 150, 72
    q, k, v, dO, bias = make(B, H, N, d, seed=5)
    c = d ** -0.5
    packed, st = binary(q, k, d)
    if kind == "ref":
        out = binattn.ref_bf16_forward(q, k, bias, v, c)
        _, _, dv, _ = binattn.ref_bf16_backward(q, k, bias, v, dO, c)
        st = f64(q), f64(k)
    else:
        (qb, aq), (kb, ak) = packed
        out = binattn.forward(qb, kb, aq, ak, bias, v, c)
        dv, _, _, _ = binattn.backward_bf16(qb, kb, aq, ak, bias, v, dO, c)
    val, bound = ref.forward(*st, f64(v), f64(bias), c)
    check(out, (val, bound), kind)
    # O is linear in V: sum O dO = sum V dV, per head
    G, V = f64(dO), f64(v)
    slack = (bound * np.abs(G)).sum((2, 3)) + (bwd_ref.gradients(*st, V, G, f64(bias), c)["dv"][1] * np.abs(V)).sum((2, 3))
    assert (np.abs((f64(out) * G).sum((2, 3)) - (f64(dv) * V).sum((2, 3))) <= slack).all()
