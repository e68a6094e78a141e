"""The tensor-core backwards against differences of the loss in a direction that a
wrong gradient cannot hide in, and at long rows key by key."""
import numpy as np
import pytest
import torch

import attention_bwd_ref as ref
from attention_bwd_ref import H8, f64
from diffusion_transformers_b200 import binattn
from test_gpu_backward_tc import KINDS, call, make, want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
def test_differences_along_the_gradients_signs(kind):
    # along x = sign(gradient) the loss changes by sum |gradient|, which no sum of
    # rounding errors comes near: zeros, flipped signs or lost terms all show
    B, H, N, d, scale = 2, 2, 40, 64, 0.125
    c = make(B, H, N, d, True, seed=8)
    got = call(kind, c, scale)
    q, k, v, dO, bias = (f64(c[n]) for n in ("q", "k", "v", "dO", "bias"))
    if kind == "binary":
        q, k = (ref.signs(b, d) * f64(a)[..., None] for b, a in (binattn.pack(c[n]) for n in "qk"))

    def loss(q, k, v, bias):
        L = scale * q @ np.swapaxes(k, -1, -2) + bias
        P = np.exp(L - L.max(-1, keepdims=True))
        return float(((P / P.sum(-1, keepdims=True)) @ v * dO).sum())

    args = [q, k, v, bias]
    w = want(kind, c, scale)

    def quotient(i, x, step):
        hi, lo = list(args), list(args)
        hi[i], lo[i] = args[i] + step * x, args[i] - step * x
        return (loss(*hi) - loss(*lo)) / (2 * step)

    rng = np.random.default_rng(1)
    for i, (g, name) in enumerate(zip(got, ("dq", "dk", "dv", "dbias"))):
        g, (_, bound) = f64(g), w[name]
        x = np.sign(g)
        slope = quotient(i, x, 1e-6)
        assert slope > 4 * bound.sum(), f"{name}: the bound would hide the gradient"
        assert abs(slope - np.abs(g).sum()) <= bound.sum() + 1e-4 * slope
        # and single elements against their own bounds, the largest among them
        at = [np.unravel_index(np.abs(g).argmax(), g.shape)]
        at += [tuple(rng.integers(0, n) for n in g.shape) for _ in range(30)]
        for e in at:
            x = np.zeros(g.shape)
            x[e] = 1.0
            # rounding noise of the loss (about 1e3 terms of size 1) over the step
            assert abs(quotient(i, x, 1e-4) - g[e]) <= bound[e] + 1e-7, (name, e)


def long_statistics(q, k, G, V, scale, step=4096):
    """LSE and D of every row, in 64 bits, block by block of rows."""
    lse, D = [], []
    for r in range(0, q.shape[0], step):
        L = scale * q[r:r + step] @ k.T
        dP = G[r:r + step] @ V.T
        lse.append(torch.logsumexp(L, -1))
        D.append((torch.exp(L - lse[-1][:, None]) * dP).sum(-1))
    return torch.cat(lse), torch.cat(D)


@pytest.mark.parametrize("kind", KINDS)
def test_longest_rows_key_by_key(kind):
    # N = 65535: dV and dK of sampled keys (ends and edges of tiles, and between)
    # against 64 bits over all query rows, and dV's sums with random rounding
    N, d, scale = 65535, 64, 0.125
    c = make(1, 1, N, d, False, seed=14)
    _, dk, dv, _ = call(kind, c, scale, with_dbias=False)
    torch.cuda.synchronize()
    binattn.device_status()
    q, k = (c[n][0, 0].double() for n in "qk")
    if kind == "binary":
        q, k = (torch.tensor(ref.signs(b, d)[0, 0], device="cuda") * a[0, 0].double()[:, None]
                for b, a in (binattn.pack(c[n]) for n in "qk"))
    G, V = c["dO"][0, 0].double(), c["v"][0, 0].double()
    lse, D = long_statistics(q, k, G, V, scale)
    keys = torch.tensor([0, 1, 63, 64, 127, 128, 129, 4095, 4096, 33333, 40000, N - 128, N - 65, N - 64, N - 63, N - 1],
                        device="cuda")
    P = torch.exp(scale * q @ k[keys].T - lse[:, None])         # [N, keys]
    dL = P * (G @ V[keys].T - D[:, None])
    for got, val, name in ((dv[0, 0, keys], P.T @ G, "dv"), (dk[0, 0, keys], scale * dL.T @ q, "dk")):
        for i in range(len(keys)):  # 64 channels each: 5e-3 is beyond 3 x the two roundings' mean square
            off = float((got[i].double() - val[i]).norm() / val[i].norm())
            assert off <= 1e-2, f"{kind} {name} of key {int(keys[i])}: off by {off:.2e}"
        assert float((got.double() - val).norm() / val.norm()) <= 5e-3, f"{kind} {name}"
    check_mass(dv, c["dO"])


def check_mass(dv, dO):
    """sum_j dV_j = sum_i dO_i per channel, with roundings that add up at random:
    of P (H P |dO| per pair; P's squares add up to less than sum P = 1 per row)
    and of dV, each uniform within half a step (H / sqrt(3) in the mean square), and
    six deviations."""
    off = (dv.double().sum(2) - dO.double().sum(2)).abs()
    spread = H8 / 3 ** 0.5 * ((dO.double() ** 2).sum(2) + (dv.double() ** 2).sum(2)).sqrt()
    assert (off <= 6 * spread).all(), float((off / spread).max())


@pytest.mark.parametrize("kind", KINDS)
def test_long_rows_mass(kind):
    c = make(2, 16, 4096, 72, True, seed=12)
    _, _, dv, _ = call(kind, c, 72 ** -0.5, with_dbias=False)
    check_mass(dv, c["dO"])
