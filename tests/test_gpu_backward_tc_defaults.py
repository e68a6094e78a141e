"""What the tensor-core backwards compute when with_dbias is left out: the bias'
gradient where there is a bias, and no [H, N, N] kernel and memory where there is
none."""
import pytest
import torch

from diffusion_transformers_b200 import binattn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["ref", "binary"])
def test_dbias_comes_with_a_bias(kind):
    B, H, N, d = 1, 4, 2048, 64
    g = torch.Generator(device="cuda").manual_seed(0)
    q, k, v, dO = (torch.randn(B, H, N, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(4))
    bias = torch.zeros(H, N, N, dtype=torch.bfloat16, device="cuda")
    (qb, aq), (kb, ak) = binattn.pack(q), binattn.pack(k)

    def call(bias, **kw):
        if kind == "ref":
            return binattn.ref_bf16_backward(q, k, bias, v, dO, 0.125, **kw)
        return binattn.backward_bf16(qb, kb, aq, ak, bias, v, dO, 0.125, **kw)

    call(None)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    held = torch.cuda.memory_allocated()
    out = call(None)
    assert out[3] is None
    assert torch.cuda.max_memory_allocated() - held < 2 * H * N * N
    for kw in ({}, {"with_dbias": True}):
        assert call(bias, **kw)[3].shape == (H, N, N)
    assert call(bias, with_dbias=False)[3] is None
    # a zero bias' gradient without a bias, when it is asked for
    assert call(None, with_dbias=True)[3].shape == (H, N, N)
