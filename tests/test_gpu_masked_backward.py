"""The tensor-core backwards under every mask that the forwards are tested under, at
narrow and wide heads, against the formulas in 64 bits."""
import pytest
import torch

import masked_forward_ref as masks
from diffusion_transformers_b200 import binattn
from test_gpu_backward_tc import KINDS, call, check_all, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", [(2, 4, 150, 72), (1, 4, 200, 64), (5, 4, 141, 128), (2, 4, 264, 96), (9, 4, 144, 16)], ids=str)
def test_masked_gradients(kind, shape):
    B, H, N, d = shape
    c = make(B, H, N, d, True, seed=N)
    c["bias"] = masks.masked_bias(H, N, N).cuda()
    got = call(kind, c, d ** -0.5)
    torch.cuda.synchronize()
    binattn.device_status()
    check_all(kind, c, d ** -0.5, got, f"masked {shape}")
    dq, dk, dv, db = got
    masked = c["bias"] == float("-inf")
    assert not db[masked].any()                       # a masked pair's logit moves nothing
    assert not dq[:, 3].any() and not dk[:, 3].any() and not dv[:, 3].any()
    # keys that no query sees get nothing (head 2's rows 10 .. 19 see the first 130
    # only where they see nothing better: they have ordinary keys behind)
    assert not dk[:, 2, :130].any() and not dv[:, 2, :130].any()
    assert torch.equal(got[0], call(kind, c, d ** -0.5, with_dbias=False)[0])
