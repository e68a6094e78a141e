"""Attention's forward under a mask in 64 bits, with the bound its roundings
allow, and a bias that masks rows in every way.

A row with nothing but -inf has no weights: its result is zero, as its
gradients are (binattn_backward_bf16). With H = 2^-8 half a step of bf16: P
rounded to bf16 is off by H P, which moves sum P V by H sum P |V| and the sum l
that it is divided by by H, so the quotient by H |O|; the logits are off by
delta as in attention_bwd_ref (and 4 U of the largest for the change of units),
which moves a weight by 4 delta; the result is rounded once, H |O|.
"""
import numpy as np
import torch

from attention_bwd_ref import H8, U

LOW = torch.finfo(torch.bfloat16).min
INF = float("inf")


def masked_bias(H, N, seed=0):
    """[H, N, N] bf16, H >= 4, N >= 140: head 0 unmasked but for its rows 0 .. 9;
    head 1 a causal mask from the right (key j >= i: the first tiles of late rows are
    all masked); head 2 a left-padded sequence (keys 0 .. 129 at -inf) with a few
    rows at the lowest value instead; head 3 wholly masked."""
    g = torch.Generator().manual_seed(seed)
    b = (0.5 * torch.randn(H, N, N, generator=g)).to(torch.bfloat16)
    b[0, 0] = -INF
    b[0, 1] = LOW                     # uniform weights
    b[0, 2] = -INF
    b[0, 2, N - 1] = 0.25             # one key, the last
    b[0, 3, :N // 2] = -INF           # nothing in the first half of the keys
    b[0, 4, N // 2:] = -INF           # nor in the second
    b[0, 5, :N - 3] = LOW             # the lowest value, then ordinary ones
    b[0, 6, 3:] = LOW                 # and the other way round
    b[0, 7] = -INF
    b[0, 7, 70:] = LOW                # -inf, then the lowest value: uniform from there on
    b[0, 8] = -1e30
    b[0, 8, 5] = LOW
    b[0, 9, :] = LOW
    b[0, 9, 100] = -INF
    b[1] += torch.full((N, N), -INF).tril(-1).to(torch.bfloat16)
    b[2, :, :130] = -INF
    b[2, 10:20, :130] = LOW
    b[3] = -INF
    return b


def forward(q, k, v, bias, c):
    """(O, bound); numpy float64 in, q and k with their alphas."""
    B, H, N, d = q.shape
    out, bound = np.zeros((B, H, N, d)), np.zeros((B, H, N, d))
    for b in range(B):
        for h in range(H):
            s = c * q[b, h] @ k[b, h].T
            L = s + bias[h]
            size = abs(c) * np.abs(q[b, h]) @ np.abs(k[b, h]).T
            size = size + np.where(np.isfinite(bias[h]) & (np.abs(bias[h]) < 1e28), np.abs(bias[h]), 0)
            top = L.max(1, keepdims=True)
            # values as low as these leave nothing of the scores in 32 bits
            L = np.where(np.abs(bias[h]) >= 1e28, bias[h], L)
            top = L.max(1, keepdims=True)
            e = np.exp(L - np.where(np.isfinite(top), top, 0))
            tot = e.sum(1, keepdims=True)
            P = e / np.where(tot > 0, tot, 1)
            O, spread = P @ v[b, h], P @ np.abs(v[b, h])
            delta = (d + 12) * U * size.max() + 2.0 ** -21
            err = (H8 + 4 * delta + (N + 8) * U) * (spread + np.abs(O))
            out[b, h], bound[b, h] = O, err * (1 + H8) + H8 * np.abs(O) + 1e-37
    return out, bound
