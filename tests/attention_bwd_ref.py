"""Attention's gradients in 64 bits, straight from the formulas, with the bounds
that the tensor-core backward's roundings allow.

U = 2^-24 and H = 2^-8 are half a step of fp32 and bf16, relative. With L the
logits, P the weights, dP = dO V^T, D = sum_j P dP and dL = P (dP - D):
 - a logit is a sum of d products and a few roundings more, so it is off by at
   most (d + 8) U (c sum |q||k| + |bias|), and 2^-21 for the exp; delta is the
   largest of these. A weight (its log-sum-exp is off by as much again) is off by
   4 delta P;
 - dP is off by (d + 8) U sum |dO||v|, D by that and by (N + 8) U and 4 delta on
   its weighted sum; so dL is off by E = P (4 delta (|dP| + |D|) + 2 dP's error +
   D's), before it is rounded to bf16 (H |dL|);
 - the products accumulate in fp32 (N U on the sum of magnitudes) and the
   result is rounded to bf16 (H of its value, and of the errors so far).
"""
import numpy as np
import torch

U, H8 = 2.0 ** -24, 2.0 ** -8


def f64(t):
    return t.detach().cpu().double().numpy()


def signs(bits, d):
    """+1 / -1 of packed sign words."""
    w = bits.detach().cpu().numpy().view(np.uint32)
    c = np.arange(d)
    return np.where((w[..., c // 32] >> np.uint32(0)) >> (c % 32).astype(np.uint32) & 1, 1.0, -1.0)


def gradients(q, k, v, dO, bias, c):
    """Gradients and error bounds: {"dq": (value, bound), ...}; numpy float64 in."""
    B, H, N, d = q.shape
    out = {n: (np.zeros((B, H, N, d)), np.zeros((B, H, N, d))) for n in ("dq", "dk", "dv")}
    db, eb, ab = np.zeros((H, N, N)), np.zeros((H, N, N)), np.zeros((H, N, N))
    for b in range(B):
        for h in range(H):
            Q, K, V, G = q[b, h], k[b, h], v[b, h], dO[b, h]
            L = c * Q @ K.T
            size = abs(c) * np.abs(Q) @ np.abs(K).T
            if bias is not None:
                L = L + bias[h]
                size = size + np.where(np.isfinite(bias[h]) & (np.abs(bias[h]) < 1e30), np.abs(bias[h]), 0)
            top = L.max(1, keepdims=True)
            e = np.exp(L - np.where(np.isfinite(top), top, 0))
            tot = e.sum(1, keepdims=True)
            P = e / np.where(tot > 0, tot, 1)
            delta = (d + 8) * U * size.max() + 2.0 ** -21
            dP = G @ V.T
            sdP = np.abs(G) @ np.abs(V).T
            edP = (d + 8) * U * sdP
            D = (P * dP).sum(1, keepdims=True)
            eD = ((N + 8) * U + 4 * delta) * (P * np.abs(dP)).sum(1, keepdims=True) + (P * edP).sum(1, keepdims=True)
            dL = P * (dP - D)
            E = P * (4 * delta * (np.abs(dP) + np.abs(D)) + 2 * edP + eD)
            # dL rounded to bf16, with its own error
            R = E + H8 * (np.abs(dL) + E)
            for name, val, err, mag in (
                    ("dq", c * dL @ K, abs(c) * R @ np.abs(K), abs(c) * np.abs(dL) @ np.abs(K)),
                    ("dk", c * dL.T @ Q, abs(c) * R.T @ np.abs(Q), abs(c) * np.abs(dL).T @ np.abs(Q)),
                    ("dv", P.T @ G, ((4 * delta + H8 * (1 + 4 * delta)) * P).T @ np.abs(G), P.T @ np.abs(G))):
                err = err + (N + 8) * U * (mag + err)
                out[name][0][b, h] = val
                out[name][1][b, h] = err * (1 + H8) + H8 * np.abs(val) + 1e-37
            db[h] += dL
            eb[h] += E
            ab[h] += np.abs(dL)
    err = eb + (B + 2) * U * ab
    out["dbias"] = (db, err * (1 + H8) + H8 * np.abs(db) + 1e-37)
    return out


def check(got: torch.Tensor, ref, what):
    g = f64(got)
    val, bound = ref
    assert got.dtype == torch.bfloat16 and g.shape == val.shape, what
    assert np.isfinite(g).all(), f"{what}: not finite"
    bad = np.abs(g - val) > bound
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} beyond the bound, first at {np.argwhere(bad)[0]}; "
                           f"worst ratio {(np.abs(g - val) / bound).max():.2f}")
    # and as a whole: rounding the weights or dL, and the result, to nearest is
    # off by H / sqrt(3) in the mean square at the most, each
    norm = np.linalg.norm(val)
    assert np.linalg.norm(g - val) <= 5e-3 * norm + np.linalg.norm(bound) * 1e-3, f"{what}: {np.linalg.norm(g - val) / norm:.2e}"
