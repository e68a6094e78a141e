"""norm_rope_pack at the most rows a call takes: 65535 heads of 65535 tokens, just
below 2^32, from an input that all heads share."""
import pytest
import torch

from diffusion_transformers_b200 import binattn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,rot", [(8, 8), (6, 4)], ids=["vector", "scalar"])
def test_most_rows(d, rot):
    B, H, N = 255, 257, 65535
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB")
    g = torch.Generator(device="cuda").manual_seed(0)
    q, k = (torch.randn(1, 1, N, d, generator=g, device="cuda") for _ in range(2))
    cos, sin = binattn.rope_tables(torch.arange(N, device="cuda"), rot)
    want = binattn.norm_rope_pack(q, k, None, None, cos, sin)
    got = binattn.norm_rope_pack(q.expand(B, H, N, d), k.expand(B, H, N, d), None, None, cos, sin)
    torch.cuda.synchronize()
    for a, w in zip(got, want):
        assert a.shape[:3] == (B, H, N)
        for b in range(B):  # entry by entry: comparisons of all of it at once take as much memory again
            assert torch.equal(a[b], w[0].expand_as(a[b])), b
    del got
    torch.cuda.empty_cache()
