"""The tensor-core backwards where a call takes more than one chunk of the batch
without a split of the chunks (sums of dbias in fp32 over the chunks, rounded with
the last), and more than one item per CTA at wide heads."""
import pytest
import torch

import attention_bwd_ref as ref
from attention_bwd_ref import H8, U
from diffusion_transformers_b200 import binattn
from test_gpu_backward_tc import KINDS, call, make

pytestmark = pytest.mark.gpu


def blocks64(kind, c, scale, heads):
    """dq, dk, dv, dbias of some heads in 64 bits on the GPU, head by head ({name: [B, heads, N, d] or
    [heads, N, N]}), and dbias' bound (attention_bwd_ref's: E of every entry, the sum over the batch, the rounding)."""
    B, H, N, d = c["q"].shape
    D = torch.float64
    out = {n: torch.empty(B, len(heads), N, d, dtype=D, device="cuda") for n in ("dq", "dk", "dv")}
    out["dbias"], err, mag = (torch.zeros(len(heads), N, N, dtype=D, device="cuda") for _ in range(3))
    if kind == "binary":
        packed = [binattn.pack(c[n]) for n in "qk"]
    for i, h in enumerate(heads):
        for b in range(B):
            q, k = (c[n][b, h].to(D) for n in "qk")
            if kind == "binary":
                q, k = (torch.tensor(ref.signs(w[b, h], d), device="cuda") * a[b, h].to(D)[:, None] for w, a in packed)
            G, V = c["dO"][b, h].to(D), c["v"][b, h].to(D)
            L, size = scale * q @ k.T, abs(scale) * q.abs() @ k.abs().T
            if c["bias"] is not None:
                L += c["bias"][h].to(D)
                size += c["bias"][h].to(D).abs()
            P = torch.softmax(L, -1)
            out["dv"][b, i] = P.T @ G
            dP, edP = G @ V.T, (d + 8) * U * G.abs() @ V.abs().T
            DD = (P * dP).sum(-1, keepdim=True)
            dL = P * (dP - DD)
            delta = (d + 8) * U * float(size.max()) + 2.0 ** -21
            eD = ((N + 8) * U + 4 * delta) * (P * dP.abs()).sum(-1, keepdim=True) + (P * edP).sum(-1, keepdim=True)
            err[i] += P * (4 * delta * (dP.abs() + DD.abs()) + 2 * edP + eD)
            mag[i] += dL.abs()
            out["dq"][b, i], out["dk"][b, i] = scale * dL @ k, scale * dL.T @ q
            out["dbias"][i] += dL
    out["bound"] = (err + (B + 2) * U * mag) * (1 + H8) + H8 * out["dbias"].abs() + 1e-37
    return out


def close(got, val, what):
    # P or dL rounded, the result rounded: half a step of bf16 each, at random
    # (H / sqrt(3) in the mean square at the most), as attention_bwd_ref's check
    off = float((got.double() - val).norm() / val.norm())
    assert off <= 5e-3, f"{what}: off by {off:.2e}"


# chunks of 3 batch entries (d = 72) and of 2 (d = 128): all in one split where
# there are many query tiles and heads, so that one array holds the sums so far
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,H,N,d,splits", [(8, 16, 1024, 72, 1), (4, 8, 1100, 72, 2), (5, 12, 1027, 128, 1)], ids=str)
def test_chunks_added_up(kind, B, H, N, d, splits):
    c = make(B, H, N, d, True, seed=20)
    size = binattn.ref_bf16_backward_workspace_bytes if kind == "ref" else binattn.backward_bf16_workspace_bytes
    sums = size(B, H, N, d, True, True) - size(B, H, N, d, True, False)
    assert sums == -(-4 * splits * H * N * N // 256) * 256
    scale = d ** -0.5
    got = call(kind, c, scale)
    torch.cuda.synchronize()
    binattn.device_status()
    heads = [0, H - 1]
    w = blocks64(kind, c, scale, heads)
    for name, g in zip(("dq", "dk", "dv"), got):
        close(g[:, heads], w[name], f"{kind} {name}")
    close(got[3][heads], w["dbias"], f"{kind} dbias")
    # element by element: an addend lost or added twice shows on its own
    beyond = int(((got[3][heads].double() - w["dbias"]).abs() > w["bound"]).sum())
    assert beyond == 0, f"{kind} dbias: {beyond} beyond the bound"
    assert all(torch.equal(a, b) for a, b in zip(got, call(kind, c, scale)))


@pytest.mark.parametrize("bias", [True, False], ids=["bias", "nobias"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,H,N,d", [(4, 40, 130, 128), (3, 21, 700, 96), (2, 90, 257, 88)], ids=str)
def test_wide_heads_several_items_per_cta(kind, bias, B, H, N, d):
    # more items than SMs: the kept operands (here in shared memory), dL over the
    # scores and the accumulators are used again
    assert B * H * -(-N // 128) > 148 + 148 // 2
    c = make(B, H, N, d, bias, seed=21)
    got = call(kind, c, d ** -0.5, with_dbias=bias)
    torch.cuda.synchronize()
    binattn.device_status()
    heads = sorted({0, 1, H // 2, H - 2, H - 1})
    w = blocks64(kind, c, d ** -0.5, heads)
    for name, g in zip(("dq", "dk", "dv"), got):
        for b in range(B):  # entry by entry: one item gone wrong is not averaged away
            for i, h in enumerate(heads):
                for n0 in range(0, N, 128):
                    close(g[b, h, n0:n0 + 128], w[name][b, i, n0:n0 + 128], f"{kind} {name} entry {b} head {h} rows {n0}")
    if bias:
        close(got[3][heads], w["dbias"], f"{kind} dbias")
