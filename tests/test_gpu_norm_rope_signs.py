"""Sign bits of norm_rope_pack where 64-bit products cannot tell them: a product
of three fp32 numbers has up to 72 bits. With any integer m,
(m + 2)(m + 3)(m + 7) - (m + 1)(m + 5)(m + 6) = 12, some 2^-66 of either
product at 24 bits each, so rounded to 64-bit numbers the two are alike. The
expected bits come from integer arithmetic."""
import numpy as np
import pytest
import torch

import norm_rope_ref as ref
from diffusion_transformers_b200 import binattn

LO, HI = (1, 5, 6), (2, 3, 7)  # added to m: factors of the smaller and the larger product


def factors(half, seed):
    """m per pair, 24-bit numbers."""
    return np.random.default_rng(seed).integers(2 ** 23, 2 ** 24 - 8, half)


def arguments(d, rot, inter, seed):
    """x [1, 2, 2, d] (heads: plus and minus), w [d], tables [2, rot / 2], bits [1, 2, 2, d], all from
    integers: at token 0 z_a is -+12 steps, at token 1 z_b is +-12."""
    a, b = ref.pairs(d, rot, inter)
    m = factors(rot // 2, seed)
    x, w = np.full(d, 2 ** 23), np.full(d, 2 ** 23)
    x[a], w[a] = m + LO[0], m + LO[1]
    x[b], w[b] = m + HI[0], m + HI[1]
    cos, sin = np.stack([m + LO[2], m + HI[2]]), np.stack([m + HI[2], -(m + LO[2])])
    on = np.ones((1, 2, 2, d), bool)
    for h, s in enumerate((1, -1)):
        for n in range(2):
            for p in range(rot // 2):
                u, v = s * int(x[a[p]]) * int(w[a[p]]), s * int(x[b[p]]) * int(w[b[p]])
                on[0, h, n, a[p]] = u * int(cos[n, p]) - v * int(sin[n, p]) >= 0
                on[0, h, n, b[p]] = u * int(sin[n, p]) + v * int(cos[n, p]) >= 0
            on[0, h, n, rot:] = s > 0
    f = [torch.tensor(t * 2.0 ** -e, dtype=torch.float32) for t, e in ((x, 23), (w, 23), (cos, 24), (sin, 24))]
    return torch.stack([f[0], -f[0]])[None, :, None].repeat(1, 1, 2, 1), *f[1:], on


CASES = [(64, 64, False), (72, 72, True), (64, 16, False), (40, 36, True), (31, 30, False), (2, 2, True)]


@pytest.mark.parametrize("d,rot,inter", CASES)
def test_the_numbers_are_exact_and_64_bits_do_not_tell(d, rot, inter):
    x, w, cos, sin, on = arguments(d, rot, inter, d)
    a, b = ref.pairs(d, rot, inter)
    for t in (x, w, cos, sin):
        assert t.dtype == torch.float32
    assert not on[0, 0, 0, a].any() and on[0, 1, 0, a].all()    # -12, +12
    assert on[0, 0, 1, b].all() and not on[0, 1, 1, b].any()    # +12, -12
    rounded = ref.signs(x.double().numpy(), w, cos, sin, inter)
    assert (rounded != on).any()


@pytest.mark.gpu
@pytest.mark.parametrize("d,rot,inter", CASES)
def test_signs_of_the_exact_difference(d, rot, inter):
    x, w, cos, sin, on = (t.cuda() if isinstance(t, torch.Tensor) else t for t in arguments(d, rot, inter, d))
    bits = binattn.norm_rope_pack(x, x, w, w, cos, sin, interleaved=inter)
    for got in (bits[0], bits[2]):
        assert np.array_equal(got.cpu().numpy().view(np.uint32), ref.words(on))
