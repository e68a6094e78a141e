"""What the operators around and behind the attention cost: the per-head norm
and rotation of queries and keys (also ending in sign bits), its gradient, and
the backward of the bf16 and of the binary attention.

``run`` computes them in elementary torch operations (``own`` false) or through
the package's calls (``own`` true), on the same inputs. The sizes are those of
the package's workloads (DeiT-B, ViT-L/16 at 384 px, DiT-XL/2 at 512 and 1024 px,
and a 256-token head pair), and odd ones between them.
"""
import math

import numpy as np
import torch

own = False
EPS = 1e-6


def listed():
    return [
        # one token of 16 heads, straight from a fused projection: latency alone
        dict(name="norm_rope one token", op="norm_rope", B=1, H=16, N=1, d=64, R=64, inter=False, dtype="bf16", fused=True,
             per_batch=False),
        # DiT-XL/2 at 1024 px: queries and keys as views of the projection's output
        dict(name="norm_rope dit_xl_1024", op="norm_rope", B=2, H=16, N=4096, d=72, R=72, inter=False, dtype="bf16", fused=True,
             per_batch=False),
        # ViT-L/16 at 384 px in fp32, positions per image, the last 16 channels not rotated
        dict(name="norm_rope_pack vit_l384 fp32", op="norm_rope_pack", B=4, H=16, N=577, d=64, R=48, inter=True, dtype="f32",
             fused=False, per_batch=True),
        # DiT-XL/2 at 512 px: serving, the binary attention's input in one pass
        dict(name="norm_rope_pack dit_xl_512", op="norm_rope_pack", B=8, H=16, N=1024, d=72, R=72, inter=True, dtype="bf16",
             fused=True, per_batch=False),
        # DeiT-B with 197 tokens: training
        dict(name="norm_rope_backward deit_b", op="norm_rope_backward", B=64, H=12, N=197, d=64, R=64, inter=False, dtype="bf16",
             fused=True, per_batch=False),
        # DiT-XL/2 at 1024 px: training
        dict(name="norm_rope_backward dit_xl_1024", op="norm_rope_backward", B=2, H=16, N=4096, d=72, R=72, inter=True,
             dtype="bf16", fused=True, per_batch=False),
        # a 256-token head pair: the smallest training step
        dict(name="ref_bf16_backward tiny", op="ref_bf16_backward", B=1, H=2, N=256, d=64, bias=True, pad=0),
        # DeiT-B: 197 tokens (no multiple of anything), learned bias and its gradient
        dict(name="ref_bf16_backward deit_b", op="ref_bf16_backward", B=64, H=12, N=197, d=64, bias=True, pad=0),
        # DiT-XL/2 at 1024 px without a bias
        dict(name="ref_bf16_backward dit_xl_1024", op="ref_bf16_backward", B=2, H=16, N=4096, d=72, bias=False, pad=0),
        # an odd length and the widest heads; 5 padded keys masked by the bias
        dict(name="backward_bf16 odd", op="backward_bf16", B=2, H=3, N=333, d=128, bias=True, pad=5),
        # DiT-XL/2 at 512 px without a bias
        dict(name="backward_bf16 dit_xl_512", op="backward_bf16", B=8, H=16, N=1024, d=72, bias=False, pad=0),
        # DiT-XL/2 at 1024 px with the learned dense bias and its gradient
        dict(name="backward_bf16 dit_xl_1024", op="backward_bf16", B=2, H=16, N=4096, d=72, bias=True, pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_pack", "norm_rope_backward", "ref_bf16_backward", "backward_bf16"])
    H = rng.randint(1, 16)
    N = _log(rng, 1, 4096)
    if op.endswith("bf16") or op.startswith("ref"):
        d = 8 * rng.randint(1, 16)
        B = max(1, min(64, 2 * 16 * 4096 * 4096 * 72 // (H * N * N * max(d, 72))))
        B = rng.randint(1, B)
        return dict(op=op, B=B, H=H, N=N, d=d, bias=rng.random() < 0.5, pad=min(rng.choice([0, 0, 1, 9]), N - 1))
    d = rng.choice([rng.randint(2, 128), 8 * rng.randint(1, 16)])
    R = rng.choice([d - d % 2, 2 * rng.randint(1, d // 2)])
    B = rng.randint(1, max(1, min(64, 2 * 16 * 4096 * 72 // (2 * H * N * d))))
    return dict(op=op, B=B, H=H, N=N, d=d, R=R, inter=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f32"]),
                fused=rng.random() < 0.5, per_batch=rng.random() < 0.3)


def _bits(x):
    """Sign words [..., ceil(d / 32)] int32 of x: bit c % 32 of word c // 32 is x_c >= 0."""
    d = x.shape[-1]
    W = (d + 31) // 32
    p = torch.nn.functional.pad((x >= 0).to(torch.int64), (0, 32 * W - d)).view(*x.shape[:-1], W, 32)
    w = (p << torch.arange(32, device=x.device)).sum(-1)
    return torch.where(w >= 2**31, w - 2**32, w).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    B, H, N, d = case["B"], case["H"], case["N"], case["d"]
    s = dict(case)
    if case["op"].startswith("norm_rope"):
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        if case["fused"]:  # the projection's output [B, N, 3, H, d], q and k as views of it
            qkv = randn(B, N, 3, H, d, dtype=dt)
            s["q"], s["k"] = qkv[:, :, 0].permute(0, 2, 1, 3), qkv[:, :, 1].permute(0, 2, 1, 3)
        else:
            s["q"], s["k"] = randn(B, H, N, d, dtype=dt), randn(B, H, N, d, dtype=dt)
        s["w_q"], s["w_k"] = 1 + 0.1 * randn(d), 1 + 0.1 * randn(d)
        # angles of positions 0 .. N - 1 (per image: from an offset of its own), in 64 bits
        pos = torch.arange(N, device="cuda", dtype=torch.float64)
        if case["per_batch"]:
            pos = pos + torch.randint(0, 4096, (B, 1), generator=g, device="cuda").double()
        half = case["R"] // 2
        freq = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / max(half, 1))
        ang = pos[..., None] * freq
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        if case["op"] == "norm_rope_backward":
            s["dq"], s["dk"] = randn(B, H, N, d, dtype=dt), randn(B, H, N, d, dtype=dt)
        return s
    bf = torch.bfloat16
    q, k = randn(B, H, N, d, dtype=bf), randn(B, H, N, d, dtype=bf)
    s["v"], s["dO"], s["scale"] = randn(B, H, N, d, dtype=bf), randn(B, H, N, d, dtype=bf), 1 / math.sqrt(d)
    s["bias"] = None
    if case["bias"] or case["pad"]:
        s["bias"] = (0.5 * randn(H, N, N)).to(bf)
        if case["pad"]:
            s["bias"][:, :, N - case["pad"]:] = -math.inf
    if case["op"] == "ref_bf16_backward":
        s["q"], s["k"] = q, k
    else:
        s["q_bits"], s["k_bits"] = _bits(q), _bits(k)
        s["alpha_q"], s["alpha_k"] = q.float().abs().mean(-1), k.float().abs().mean(-1)
    return s


def _pairs(d, R, inter, dev):
    """Channel indices of the first and second member of every rotated pair."""
    p = torch.arange(R // 2, device=dev)
    return (2 * p, 2 * p + 1) if inter else (p, p + R // 2)


def _turn(y, cos, sin, inter, back=False):
    """y [B, H, N, d] with its pairs turned by the angles (back: by minus the angles)."""
    a, b = _pairs(y.shape[-1], 2 * cos.shape[-1], inter, y.device)
    c, s = (t if t.dim() == 2 else t[:, None] for t in (cos.to(y.dtype), sin.to(y.dtype)))
    if back:
        s = -s
    z = y.clone()
    ya, yb = y[..., a], y[..., b]
    z[..., a] = ya * c - yb * s
    z[..., b] = ya * s + yb * c
    return z


def _plain_norm_rope(x, w, cos, sin, inter):
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return _turn(x * r * w, cos, sin, inter)


def _plain_pack(x, w, cos, sin, inter):
    # the sign in 64 bits (values next to zero), the scale in 32
    bits = _bits(_turn(x.double() * w.double(), cos, sin, inter))
    return bits, _plain_norm_rope(x, w, cos, sin, inter).abs().mean(-1)


def _plain_norm_rope_backward(x, dz, w, cos, sin, inter):
    xf, dy = x.float(), _turn(dz.float(), cos, sin, inter, back=True)
    r = torch.rsqrt(xf.square().mean(-1, keepdim=True) + EPS)
    xh = xf * r
    g = dy * w
    dx = r * (g - xh * (g * xh).mean(-1, keepdim=True))
    return dx.to(x.dtype), (dy.double() * xh.double()).sum((0, 1, 2)).float()


def _signs(bits, d):
    """+1 / -1 of packed sign words, fp32 [..., d]."""
    c = torch.arange(d, device=bits.device)
    return ((bits[..., c // 32] >> (c % 32)) & 1).float() * 2 - 1


def _plain_attention_backward(q, k, v, dO, bias, scale):
    """Gradients of softmax(scale q k^T + bias) v with respect to q, k, v and the bias, fp32."""
    L = scale * (q @ k.transpose(-1, -2))
    if bias is not None:
        L = L + bias.float()
    m = L.amax(-1, keepdim=True)
    P = torch.exp(L - torch.where(m == -math.inf, torch.zeros_like(m), m))
    del L
    P = P / P.sum(-1, keepdim=True).clamp_min(1e-30)
    v, dO = v.float(), dO.float()
    dV = P.transpose(-1, -2) @ dO
    dP = dO @ v.transpose(-1, -2)
    dL = P * (dP - (P * dP).sum(-1, keepdim=True))
    del P, dP
    return scale * (dL @ k), scale * (dL.transpose(-1, -2) @ q), dV, dL.sum(0)


def run(s):
    op = s["op"]
    if own:
        from diffusion_transformers_b200 import binattn
        if op == "norm_rope":
            z = binattn.norm_rope(s["q"], s["k"], s["w_q"], s["w_k"], s["cos"], s["sin"], EPS, interleaved=s["inter"])
            return dict(q=z[0], k=z[1])
        if op == "norm_rope_pack":
            z = binattn.norm_rope_pack(s["q"], s["k"], s["w_q"], s["w_k"], s["cos"], s["sin"], EPS, interleaved=s["inter"])
            return dict(q_bits=z[0], alpha_q=z[1], k_bits=z[2], alpha_k=z[3])
        if op == "norm_rope_backward":
            z = binattn.norm_rope_backward(s["q"], s["k"], s["dq"], s["dk"], s["w_q"], s["w_k"], s["cos"], s["sin"], EPS,
                                           interleaved=s["inter"])
            return dict(dq=z[0], dk=z[1], dw_q=z[2], dw_k=z[3])
        with_dbias = s["bias"] is not None
        if op == "ref_bf16_backward":
            z = binattn.ref_bf16_backward(s["q"], s["k"], s["bias"], s["v"], s["dO"], s["scale"], with_dbias=with_dbias)
            return dict(zip(("dq", "dk", "dv", "dbias"), z[:4 if with_dbias else 3]))
        z = binattn.backward_bf16(s["q_bits"], s["k_bits"], s["alpha_q"], s["alpha_k"], s["bias"], s["v"], s["dO"], s["scale"],
                                  with_dbias=with_dbias)
        return dict(zip(("dv", "ds", "dt", "dbias"), z[:4 if with_dbias else 3]))
    if op == "norm_rope":
        return {n: _plain_norm_rope(s[n], s["w_" + n], s["cos"], s["sin"], s["inter"]).to(s[n].dtype) for n in "qk"}
    if op == "norm_rope_pack":
        q, k = (_plain_pack(s[n], s["w_" + n], s["cos"], s["sin"], s["inter"]) for n in "qk")
        return dict(q_bits=q[0], alpha_q=q[1], k_bits=k[0], alpha_k=k[1])
    if op == "norm_rope_backward":
        q, k = (_plain_norm_rope_backward(s[n], s["d" + n], s["w_" + n], s["cos"], s["sin"], s["inter"]) for n in "qk")
        return dict(dq=q[0], dk=k[0], dw_q=q[1], dw_k=k[1])
    bf = torch.bfloat16
    if op == "ref_bf16_backward":
        dq, dk, dv, db = _plain_attention_backward(s["q"].float(), s["k"].float(), s["v"], s["dO"], s["bias"], s["scale"])
        out = dict(dq=dq.to(bf), dk=dk.to(bf), dv=dv.to(bf), dbias=db.to(bf))
    else:
        q = _signs(s["q_bits"], s["d"]) * s["alpha_q"][..., None]
        k = _signs(s["k_bits"], s["d"]) * s["alpha_k"][..., None]
        ds, dt, dv, db = _plain_attention_backward(q, k, s["v"], s["dO"], s["bias"], s["scale"])
        out = dict(dv=dv.to(bf), ds=ds.to(bf), dt=dt.to(bf), dbias=db.to(bf))
    if s["bias"] is None:
        del out["dbias"]
    return out


def work(case):
    B, H, N, d = case["B"], case["H"], case["N"], case["d"]
    rows = B * H * N
    if case["op"].startswith("norm_rope"):
        es = 2 if case["dtype"] == "bf16" else 4
        tables = 4 * case["R"] * N * (B if case["per_batch"] else 1)
        per = {"norm_rope": 2 * d * es, "norm_rope_pack": d * es + 4 * ((d + 31) // 32) + 4, "norm_rope_backward": 3 * d * es}
        return {"bytes": 2 * rows * per[case["op"]] + tables + 8 * d, "flops": 2 * rows * d * 10}
    pairs = H * N * N * 4 if case["bias"] or case["pad"] else 0  # the bias in, its gradient out
    qk = 4 * rows * d if case["op"] == "ref_bf16_backward" else 2 * rows * (4 * ((d + 31) // 32) + 4)
    return {"bytes": qk + 4 * rows * d + 6 * rows * d + pairs, "flops": 10 * B * H * N * N * d}


def exact(case, seed):
    """The same outputs from the definitions, in 64 bits, one (batch entry, head) at a time where they are large."""
    s = prepare(case, seed)
    B, H, N, d = case["B"], case["H"], case["N"], case["d"]
    D = torch.float64
    if case["op"].startswith("norm_rope"):
        half = case["R"] // 2
        # the rotation of every token as complex factors on the pairs
        turn = torch.complex(s["cos"].to(D), s["sin"].to(D)).reshape(-1, 1, N, half)
        first = slice(0, 2 * half, 2) if case["inter"] else slice(0, half)
        second = slice(1, 2 * half, 2) if case["inter"] else slice(half, 2 * half)

        def rotate(y, factor):
            z = torch.complex(y[..., first], y[..., second]) * factor
            out = y.clone()
            out[..., first], out[..., second] = z.real, z.imag
            return out

        res = {}
        for n in "qk":
            x, w = s[n].to(D), s["w_" + n].to(D)
            rms = (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt()
            if case["op"] == "norm_rope":
                res[n] = rotate(x / rms * w, turn)
            elif case["op"] == "norm_rope_pack":
                z = rotate(x / rms * w, turn)
                # the signs without the division by the (positive) norm: equal products cancel to an exact zero
                u = x * w
                left, right, over = u[..., first] * turn.real, u[..., second] * turn.imag, u >= 0
                over[..., first] = left >= right
                left, right = u[..., second] * turn.real, -(u[..., first] * turn.imag)
                over[..., second] = left >= right
                words = np.zeros((B, H, N, (d + 31) // 32), dtype=np.uint32)
                on = over.cpu().numpy()
                for c in range(d):
                    words[..., c // 32] |= on[..., c].astype(np.uint32) << np.uint32(c % 32)
                res[n + "_bits"] = torch.from_numpy(words.view(np.int32))
                res["alpha_" + n] = z.abs().sum(-1) / d
            else:
                xn = x / rms
                dy = rotate(s["d" + n].to(D), turn.conj())
                dxn = dy * w
                res["d" + n] = (dxn - xn * ((dxn * xn).sum(-1, keepdim=True) / d)) / rms
                res["dw_" + n] = torch.einsum("bhnd,bhnd->d", dy, xn)
        return res
    names = ("dq", "dk", "dv") if case["op"] == "ref_bf16_backward" else ("ds", "dt", "dv")
    res = {n: torch.empty(B, H, N, d, dtype=D, device="cuda") for n in names}
    db = None if s["bias"] is None else torch.zeros(H, N, N, dtype=D, device="cuda")
    chan = torch.arange(d, device="cuda")
    for b in range(B):
        for h in range(H):
            if case["op"] == "ref_bf16_backward":
                q, k = s["q"][b, h].to(D), s["k"][b, h].to(D)
            else:
                q, k = (torch.where((s[n + "_bits"][b, h][:, chan // 32] >> (chan % 32)) & 1 == 1, 1.0, -1.0).to(D)
                        * s["alpha_" + n][b, h].to(D)[:, None] for n in "qk")
            logits = torch.mm(q, k.t()) * s["scale"]
            if db is not None:
                logits += s["bias"][h].to(D)
            P = torch.softmax(logits, 1).nan_to_num(0.0)  # a row that the mask leaves empty has no weights
            up = s["dO"][b, h].to(D)
            res["dv"][b, h] = torch.mm(P.t(), up)
            dP = torch.mm(up, s["v"][b, h].to(D).t())
            dlog = P * dP
            dlog -= P * dlog.sum(1, keepdim=True)
            res[names[0]][b, h] = torch.mm(dlog, k) * s["scale"]
            res[names[1]][b, h] = torch.mm(dlog.t(), q) * s["scale"]
            if db is not None:
                db[h] += dlog
    if db is not None:
        res["dbias"] = db
    return res
