"""The tensor-core backwards on the GPU against the formulas in 64 bits
(attention_bwd_ref), at the sizes and masks where they can go wrong."""
import numpy as np
import pytest
import torch

import attention_bwd_ref as ref
from attention_bwd_ref import check, f64
from diffusion_transformers_b200 import binattn

pytestmark = pytest.mark.gpu

KINDS = ["ref", "binary"]


def make(B, H, N, d, bias=True, seed=0, peak=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, f=1.0):
        return (f * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)

    return dict(q=randn(B, H, N, d, f=peak), k=randn(B, H, N, d, f=peak), v=randn(B, H, N, d), dO=randn(B, H, N, d),
                bias=randn(H, N, N, f=0.5) if bias else None)


def call(kind, c, scale, with_dbias=True, **kw):
    """(dq or ds, dk or dt, dv, dbias) of the kernels."""
    if kind == "ref":
        return binattn.ref_bf16_backward(c["q"], c["k"], c["bias"], c["v"], c["dO"], scale, with_dbias=with_dbias, **kw)
    qb, aq = binattn.pack(c["q"])
    kb, ak = binattn.pack(c["k"])
    dV, ds, dt, db = binattn.backward_bf16(qb, kb, aq, ak, c["bias"], c["v"], c["dO"], scale, with_dbias=with_dbias, **kw)
    return ds, dt, dV, db


def want(kind, c, scale):
    q, k = f64(c["q"]), f64(c["k"])
    if kind == "binary":
        for_bits = [binattn.pack(c[n]) for n in "qk"]
        q, k = (ref.signs(b, c["q"].shape[3]) * f64(a)[..., None] for b, a in for_bits)
    return ref.gradients(q, k, f64(c["v"]), f64(c["dO"]), None if c["bias"] is None else f64(c["bias"]), scale)


def check_all(kind, c, scale, got, what=""):
    w = want(kind, c, scale)
    for name, g in zip(("dq", "dk", "dv", "dbias"), got):
        if g is not None:
            check(g, w[name], f"{kind} {what} {name}")


# (B, H, N, d): one key; fewer keys than a tile; whole and ragged tiles, odd tile
# counts; every operand width class (one panel, two, kept operands in shared
# memory); batches beyond one dbias chunk, and beyond the splits
CASES = [(1, 1, 1, 64), (3, 2, 1, 72), (2, 2, 3, 8), (1, 2, 64, 64), (2, 3, 65, 72), (1, 2, 127, 128), (2, 1, 128, 80),
         (1, 1, 129, 88), (2, 2, 197, 64), (1, 2, 200, 96), (1, 1, 320, 16), (9, 2, 70, 72), (5, 3, 136, 128),
         (64, 1, 33, 40), (2, 2, 577, 72)]


@pytest.mark.parametrize("bias", [True, False], ids=["bias", "nobias"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", CASES, ids=str)
def test_against_the_formulas(shape, kind, bias):
    B, H, N, d = shape
    c = make(B, H, N, d, bias, seed=N + d)
    got = call(kind, c, d ** -0.5)
    torch.cuda.synchronize()
    binattn.device_status()
    check_all(kind, c, d ** -0.5, got, shape)


@pytest.mark.parametrize("kind", KINDS)
def test_one_key_has_no_gradient_but_dv(kind):
    # softmax over one key is 1 whatever the logit: exact zeros
    for bias in (True, False):
        c = make(4, 2, 1, 72, bias, seed=3)
        dq, dk, dv, db = call(kind, c, 0.3)
        assert not dq.any() and not dk.any() and not db.any()
        assert torch.equal(dv, c["dO"])


@pytest.mark.parametrize("kind", KINDS)
def test_masks(kind):
    # a padded batch's last keys at -inf, a causal mask, a row left with one key,
    # a row with none, and a row all at the type's lowest value (uniform weights)
    B, H, N, d = 2, 3, 150, 72
    c = make(B, H, N, d, True, seed=1)
    b = c["bias"]
    b[0, :, N - 9:] = -torch.inf
    b[1] += torch.full((N, N), -torch.inf, device="cuda", dtype=torch.bfloat16).triu(1)
    b[2, 5] = -torch.inf
    b[2, 6] = -torch.inf
    b[2, 6, 77] = 0.25
    b[2, 7] = torch.finfo(torch.bfloat16).min
    b[2, 8, :100] = torch.finfo(torch.bfloat16).min
    got = call(kind, c, d ** -0.5)
    check_all(kind, c, d ** -0.5, got, "masked")
    dq, _, _, db = got
    assert not dq[:, 2, 5].any() and not db[2, 5].any()      # the empty row
    assert not db[0, :, N - 9:].any() and not db[1].triu(1).any()
    assert not dq[:, 2, 6].any()                             # one key: a constant


@pytest.mark.parametrize("kind", KINDS)
def test_whole_head_masked(kind):
    # nothing but -inf: every gradient of the head is zero, the others as ever
    c = make(2, 2, 65, 64, True, seed=4)
    c["bias"][1] = -torch.inf
    got = call(kind, c, 0.125)
    for g in got[:3]:
        assert not g[:, 1].any() and torch.isfinite(g).all()
    assert not got[3][1].any()
    check_all(kind, c, 0.125, got, "head masked")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("scale", [0.0, -0.2, 2.0])
def test_scales(kind, scale):
    # zero, negative, and so large that rows have one weight near 1
    c = make(2, 2, 130, 64, False, seed=5)
    check_all(kind, c, scale, call(kind, c, scale), f"scale {scale}")


@pytest.mark.parametrize("kind", KINDS)
def test_same_bits_twice_and_without_dbias(kind):
    c = make(5, 2, 197, 72, True, seed=6)
    first, second = call(kind, c, 0.1), call(kind, c, 0.1)
    for a, b in zip(first, second):
        assert torch.equal(a, b)
    third = call(kind, c, 0.1, with_dbias=False)
    assert third[3] is None and all(torch.equal(a, b) for a, b in zip(first[:3], third[:3]))


@pytest.mark.parametrize("kind", KINDS)
def test_dirty_workspace_and_guards(kind):
    # a workspace full of NaN patterns gives the same result, and nothing is
    # written behind its end
    c = make(7, 2, 133, 72, True, seed=7)
    size = getattr(binattn, ("ref_bf16_backward" if kind == "ref" else "backward_bf16") + "_workspace_bytes")
    need = size(7, 2, 133, 72, True, True)
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    got = call(kind, c, 0.1, workspace=ws[:need])
    assert all(torch.equal(a, b) for a, b in zip(got, call(kind, c, 0.1)))
    assert (ws[need:] == 0xFF).all()


@pytest.mark.parametrize("kind", KINDS)
def test_gradient_is_the_difference_quotient(kind):
    # the loss sum(O * dO) in 64 bits, along a random direction of each input
    B, H, N, d, c_ = 2, 2, 40, 64, 0.125
    c = make(B, H, N, d, True, seed=8)
    got = call(kind, c, c_)
    q, k, v, dO, bias = (f64(c[n]) for n in ("q", "k", "v", "dO", "bias"))
    if kind == "binary":
        q, k = (ref.signs(b, d) * f64(a)[..., None] for b, a in (binattn.pack(c[n]) for n in "qk"))

    def loss(q, k, v, bias):
        L = c_ * q @ np.swapaxes(k, -1, -2) + bias
        P = np.exp(L - L.max(-1, keepdims=True))
        return float(((P / P.sum(-1, keepdims=True)) @ v * dO).sum())

    rng = np.random.default_rng(0)
    args = [q, k, v, bias]
    w = want(kind, c, c_)
    for i, (g, name) in enumerate(zip(got, ("dq", "dk", "dv", "dbias"))):
        x = rng.choice([-1.0, 1.0], size=args[i].shape)
        hi, lo = list(args), list(args)
        hi[i], lo[i] = args[i] + 1e-5 * x, args[i] - 1e-5 * x
        # the bound of every element, added up, covers any direction of +-1
        assert abs((loss(*hi) - loss(*lo)) / 2e-5 - (f64(g) * x).sum()) <= w[name][1].sum() + 1e-4


@pytest.mark.parametrize("kind", KINDS)
def test_other_stream_and_replayed_graphs(kind):
    # two captured steps with a workspace each, replayed on two streams at once
    # with new inputs, beside eager calls
    c1, c2 = make(2, 2, 197, 72, True, seed=9), make(3, 2, 130, 64, False, seed=10)
    want1, want2 = call(kind, c1, 0.1), call(kind, c2, 0.1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        bits = [binattn.pack(c1[n]) for n in "qk"]
    if kind == "ref":
        got = binattn.ref_bf16_backward(c1["q"], c1["k"], c1["bias"], c1["v"], c1["dO"], 0.1, stream=s)
    else:
        dV, ds, dt, db = binattn.backward_bf16(bits[0][0], bits[1][0], bits[0][1], bits[1][1], c1["bias"], c1["v"],
                                               c1["dO"], 0.1, stream=s)
        got = ds, dt, dV, db
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want1))
    graphs, held = [], []
    for c in (c1, c2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            held.append(call(kind, c, 0.1))
        graphs.append(gr)
    for c in (c1, c2):
        c["dO"].copy_(torch.randn_like(c["dO"]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for st, gr in zip(streams, graphs):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    binattn.device_status()
    for h, c in zip(held, (c1, c2)):
        assert all(torch.equal(a, b) for a, b in zip(h, call(kind, c, 0.1)) if a is not None)


def test_agrees_with_the_cuda_core_backward():
    # the same gradients as binattn_backward's, up to bf16
    c = make(2, 3, 257, 72, True, seed=11)
    qb, aq = binattn.pack(c["q"])
    kb, ak = binattn.pack(c["k"])
    slow = binattn.backward(qb, kb, aq, ak, c["bias"], c["v"], c["dO"], 0.118)
    fast = binattn.backward_bf16(qb, kb, aq, ak, c["bias"], c["v"], c["dO"], 0.118)
    for a, b in zip(fast, slow):
        assert (a.float() - b).norm() <= 5e-3 * b.norm()


@pytest.mark.parametrize("kind", KINDS)
def test_long_rows(kind):
    # DiT-XL/2 at 1024 px with the bias: on every (b, h), sum_j dV_j = sum_i dO_i
    # and rows of dbias add up to 0; one head against the formulas in 64 bits
    B, H, N, d = 2, 16, 4096, 72
    c = make(B, H, N, d, True, seed=12)
    dq, dk, dv, db = call(kind, c, d ** -0.5)
    torch.cuda.synchronize()
    binattn.device_status()
    mass = c["dO"].double().sum(2)
    # dv is off by H per element of sum P |dO|, which adds up to H sum |dO| at the most, twice
    assert ((dv.double().sum(2) - mass).abs() <= 2 * 2.0 ** -8 * c["dO"].double().abs().sum(2)).all()
    rows = db.double().sum(-1).abs()
    assert (rows <= (2.0 ** -8 + 1e-3) * db.double().abs().sum(-1) + 1e-6).all()
    h, D = 7, torch.float64
    scale = d ** -0.5
    qk = [c[n][:, h].to(D) for n in "qk"]
    if kind == "binary":
        qk = [torch.tensor(ref.signs(*[t[:, h:h + 1] for t in binattn.pack(c[n])][:1], d)[:, 0], device="cuda")
              * binattn.pack(c[n])[1][:, h].to(D)[..., None] for n in "qk"]
    L = scale * qk[0] @ qk[1].transpose(-1, -2) + c["bias"][h].to(D)
    P = torch.softmax(L, -1)
    G, V = c["dO"][:, h].to(D), c["v"][:, h].to(D)
    dP = G @ V.transpose(-1, -2)
    dL = P * (dP - (P * dP).sum(-1, keepdim=True))
    for got, val in ((dq[:, h], scale * dL @ qk[1]), (dk[:, h], scale * dL.transpose(-1, -2) @ qk[0]),
                     (dv[:, h], P.transpose(-1, -2) @ G), (db[h], dL.sum(0))):
        assert (got.to(D) - val).norm() <= 5e-3 * val.norm()


def test_many_heads():
    # the most heads a call takes, each its own item of the kernels
    B, H, N, d, scale = 4369, 15, 3, 8, 0.3
    c = make(B, H, N, d, True, seed=13)
    dq, dk, dv, db = call("ref", c, scale)
    q, k, v, G = (c[n].double() for n in ("q", "k", "v", "dO"))
    P = torch.softmax(scale * q @ k.transpose(-1, -2) + c["bias"].double(), -1)
    dP = G @ v.transpose(-1, -2)
    dL = P * (dP - (P * dP).sum(-1, keepdim=True))
    for got, val in ((dq, scale * dL @ k), (dk, scale * dL.transpose(-1, -2) @ q), (dv, P.transpose(-1, -2) @ G),
                     (db, dL.sum(0))):
        assert (got.double() - val).norm() <= 5e-3 * val.norm()


@pytest.mark.parametrize("kind", KINDS)
def test_longest_rows(kind):
    # N = 65535, one head: what holds at any length, and sampled rows in 64 bits
    N, d, scale = 65535, 64, 0.125
    c = make(1, 1, N, d, False, seed=14)
    dq, dk, dv, _ = call(kind, c, scale, with_dbias=False)
    torch.cuda.synchronize()
    binattn.device_status()
    assert ((dv.double().sum(2) - c["dO"].double().sum(2)).abs() <= 2 * 2.0 ** -8 * c["dO"].double().abs().sum(2)).all()
    qk = [c[n][0, 0].double() for n in "qk"]
    if kind == "binary":
        qk = [torch.tensor(ref.signs(b, d)[0, 0], device="cuda") * a[0, 0].double()[:, None]
              for b, a in (binattn.pack(c[n]) for n in "qk")]
    rows = torch.tensor([0, 63, 64, 127, 128, 40000, N - 64, N - 1], device="cuda")
    P = torch.softmax(scale * qk[0][rows] @ qk[1].T, -1)
    dP = c["dO"][0, 0, rows].double() @ c["v"][0, 0].double().T
    want_dq = scale * (P * (dP - (P * dP).sum(-1, keepdim=True))) @ qk[1]
    assert (dq[0, 0, rows].double() - want_dq).norm() <= 5e-3 * want_dq.norm()
    assert torch.isfinite(dk.float()).all()
