"""The query / key norm with rotation on the GPU against its fp64 definition, and the layer that it belongs to.

Tolerances.  u = 2^-8 is half a bf16 step, relative; e = 2^-24 half an fp32 one.  An output is a sum of two
products of a few fp32 roundings each (norm, weight, cosine: 16 covers them), rounded once to bf16.  A weight's
gradient sums one term for each row, n e of the terms' magnitude; the sums run over at most rows terms.
"""
import numpy as np
import pytest
import torch

import linear_attn_oracle as lo

pytestmark = pytest.mark.gpu

from selective_state_space_43_b200 import ops  # noqa: E402

U, E = 2.0 ** -8, 2.0 ** -24
DTYPES = [torch.bfloat16, torch.float32]
CASES = [((1,), 1, 1, 8, 8), ((3,), 5, 2, 16, 0), ((2, 9), 4, 4, 64, 64), ((70,), 33, 1, 80, 40), ((5,), 64, 8, 128, 128),
         ((1, 130), 3, 3, 96, 48), ((17,), 7, 9, 256, 128), ((900,), 2, 1, 128, 64), ((2,), 40, 300, 32, 16),
         ((4,), 2, 2, 200, 200)]


def np64(t):
    return t.detach().cpu().double().numpy()


def make(lead, Hq, Hk, D, rot, dtype, seed, far=1 << 20):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, dt=dtype):
        return torch.randn(shape, generator=g).to(dt).cuda()

    return dict(q=normal(*lead, Hq, D), k=normal(*lead, Hk, D), q_weight=1 + 0.2 * normal(D, dt=torch.float32),
                k_weight=normal(D, dt=torch.float32), positions=torch.randint(0, far, lead, generator=g).cuda(),
                inv_freq=(10000.0 ** (-torch.arange(rot // 2) / max(1, rot // 2))).float().cuda(),
                dq_out=normal(*lead, Hq, D), dk_out=normal(*lead, Hk, D))


IN = ("q", "k", "q_weight", "k_weight", "positions", "inv_freq")


def bound(want, mag, dtype, n=16):
    return n * E * mag + (U * np.abs(want) if dtype == torch.bfloat16 else 0) + 1e-30


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("lead,Hq,Hk,D,rot", CASES)
def test_forward_and_backward(lead, Hq, Hk, D, rot, inter, dtype):
    x = make(lead, Hq, Hk, D, rot, dtype, D + Hq)
    args = [x[n] for n in IN]
    out = ops.qk_norm_rope(*args, eps=1e-5, interleaved=inter)
    got = ops.qk_norm_rope_backward(x["dq_out"], x["dk_out"], *args, eps=1e-5, interleaved=inter)
    torch.cuda.synchronize()
    for i, n in enumerate("qk"):
        w = x[n + "_weight"]
        y = lo.norm_rope(x[n], w, x["positions"], x["inv_freq"], 1e-5, inter)
        xx = np64(x[n])
        # both channels of a pair are below the row's largest normed one; the angle is off by pi e and its
        # function by 2 e
        mag = np.max(np.abs(xx / np.sqrt((xx * xx).mean(-1, keepdims=True) + 1e-5) * np64(w)), -1, keepdims=True)
        assert (np.abs(np64(out[i]) - y) <= bound(y, 2 * mag, dtype)).all()
        dx, dw, mx, mw = lo.norm_rope_grads(x[n], w, x["positions"], x["inv_freq"], 1e-5, inter, x["d%s_out" % n])
        # the turned gradients' errors are relative to the larger channel of the pair, so to the row's largest;
        # the mean over a row sums D terms
        big = np.max(mx, -1, keepdims=True)
        assert (np.abs(np64(got[n]) - dx) <= bound(dx, 2 * big, dtype, 16 + D)).all()
        rows = xx.size // D
        dy = np.max(np.abs(np64(x["d%s_out" % n])))
        assert (np.abs(np64(got[n + "_weight"]) - dw) <= (min(rows, 400) + 16) * E * (mw + dy * 4)
                + 8 * E * rows ** 0.5 * dy * 4).all()


@pytest.mark.parametrize("inter", [False, True])
def test_far_positions_and_gradient_against_differences(inter):
    """Positions up to 2^31 and below zero keep their angle; the gradient agrees with the forward's differences."""
    x = make((6,), 2, 1, 64, 64, torch.float32, 3)
    x["positions"] = torch.tensor([0, 1, -5, 2 ** 31, 2 ** 24 + 1, 123456789]).cuda()
    args = [x[n] for n in IN]
    q, k = ops.qk_norm_rope(*args, interleaved=inter)
    y = lo.norm_rope(x["q"], x["q_weight"], x["positions"], x["inv_freq"], 1e-6, inter)
    # fp64 angles of 2^31 are off by 2^-53 2^31 = 2^-22
    assert np.abs(np64(q) - y).max() <= (2.0 ** -22 + 16 * E) * 2 * np.abs(y).max()
    got = ops.qk_norm_rope_backward(x["dq_out"], x["dk_out"], *args, interleaved=inter)
    dirn, h = torch.randn_like(x["q"]), 2.0 ** -7
    f = []
    for s in (1, -1):
        f.append((ops.qk_norm_rope(x["q"] + s * h * dirn, *args[1:], interleaved=inter)[0].double()
                  * x["dq_out"].double()).sum().item())
    want = (got["q"].double() * dirn.double()).sum().item()
    # fp32 roundings of 768 outputs of size about 1, over 2 h, and a third derivative's term of order h^2
    assert abs((f[0] - f[1]) / (2 * h) - want) <= 16 * E * 768 / (2 * h) + 768 * h * h


@pytest.mark.parametrize("dtype", DTYPES)
def test_views_in_place_and_no_rows(dtype):
    Hq, Hk, D = 6, 2, 64
    wide = torch.randn(3, 50, (Hq + 2 * Hk) * D + 8, device="cuda").to(dtype)
    x = make((3, 50), Hq, Hk, D, 32, dtype, 1)
    q = wide[..., 8:8 + Hq * D].unflatten(-1, (Hq, D))
    k = wide[..., 8 + Hq * D:8 + (Hq + Hk) * D].unflatten(-1, (Hk, D))
    rest = [x[n] for n in IN[2:]]
    a = ops.qk_norm_rope(q, k, *rest)
    b = ops.qk_norm_rope(q.contiguous(), k.contiguous(), *rest)
    ga = ops.qk_norm_rope_backward(x["dq_out"], x["dk_out"], q, k, *rest)
    gb = ops.qk_norm_rope_backward(x["dq_out"], x["dk_out"], q.contiguous(), k.contiguous(), *rest)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and all(torch.equal(ga[n], gb[n]) for n in ga)
    qc, kc = q.contiguous(), k.contiguous()
    c = ops.qk_norm_rope(qc, kc, *rest, q_out=qc, k_out=kc)
    assert c[0] is qc and torch.equal(qc, a[0]) and torch.equal(kc, a[1])
    with pytest.raises(ops.SsdError):
        ops.qk_norm_rope(qc, kc, *rest, q_out=kc.new_empty(0).set_(qc.untyped_storage(), 0, qc.shape, qc.stride()),
                         k_out=qc.new_empty(0).set_(qc.untyped_storage(), 0, kc.shape, kc.stride()))
    none = make((0,), Hq, Hk, D, 32, dtype, 1)
    o = ops.qk_norm_rope(*[none[n] for n in IN])
    g = ops.qk_norm_rope_backward(none["dq_out"], none["dk_out"], *[none[n] for n in IN])
    assert o[0].shape == (0, Hq, D) and (g["q_weight"] == 0).all() and (g["k_weight"] == 0).all()


def test_rows_of_zeros_and_huge_rows():
    x = make((4,), 2, 2, 64, 32, torch.float32, 2)
    x["q"][1] = 0.0
    x["q"][2, 1] = 1e17
    x["k"][3] = 1e-20
    q, k = ops.qk_norm_rope(*[x[n] for n in IN])
    g = ops.qk_norm_rope_backward(x["dq_out"], x["dk_out"], *[x[n] for n in IN])
    assert (q[1] == 0).all()
    for i, n in enumerate("qk"):
        y = lo.norm_rope(x[n], x[n + "_weight"], x["positions"], x["inv_freq"], 1e-6, False)
        assert np.abs(np64((q, k)[i]) - y).max() <= 32 * E * np.abs(y).max()
        assert torch.isfinite(g[n]).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_the_layer(dtype):
    """Norm and rotation, prefill, gated norm of the output, then a token through the step: against fp64 all the way
    from the operator before, and the gradients back through both."""
    B, L, H, Hk, D, dv = 2, 200, 8, 4, 64, 64
    x = make((B, L), H, Hk, D, 32, dtype, 12, far=4000)
    v = torch.randn(B, L, Hk, dv, device="cuda").to(dtype)
    ld = -torch.exp(-torch.arange(H, device="cuda") * 0.8)
    w = torch.rand(H * dv, device="cuda") + 0.5
    args = [x[n] for n in IN]
    q, k = ops.qk_norm_rope(*args)
    o, S = ops.linear_attn_prefill(q, k, v, ld)
    y = ops.gated_rmsnorm(o.flatten(2), w, norm_groups=H)
    wo, wS, mo, _ = lo.prefill(q, k, v, ld, D ** -0.5)
    n = (D + 300) * E
    tol = n * mo + (U * np.abs(wo) + 1.02 * U * mo if dtype == torch.bfloat16 else 0)
    assert (np.abs(np64(o) - wo) <= tol).all()
    on = np64(o)
    want = (on / np.sqrt((on * on).mean(-1, keepdims=True) + 1e-5)).reshape(B, L, -1) * np64(w)
    assert (np.abs(np64(y) - want) <= 16 * E * np.abs(want) + (U * np.abs(want) if dtype == torch.bfloat16 else 0)
            + 1e-30).all()
    do = torch.randn_like(o)
    g = ops.linear_attn_backward(q, k, v, ld, do)
    gw, gm = lo.backward(q, k, v, ld, D ** -0.5, do)
    for name in "qkv":
        t = (D + 300) * E * gm[name] + (U * np.abs(gw[name]) + 1.02 * U * gm[name] if dtype == torch.bfloat16 else 0)
        assert (np.abs(np64(g[name]) - gw[name]) <= t).all()
    back = ops.qk_norm_rope_backward(g["q"], g["k"], *args)
    for name in "qk":
        dx, _, mx, _ = lo.norm_rope_grads(x[name], x[name + "_weight"], x["positions"], x["inv_freq"], 1e-6, False,
                                          g[name])
        big = np.max(mx, -1, keepdims=True)
        assert (np.abs(np64(back[name]) - dx) <= bound(dx, 2 * big, dtype, 16 + D)).all()
    t = make((B,), H, Hk, D, 32, dtype, 13, far=4000)
    qt, kt = ops.qk_norm_rope(*[t[n] if n in ("q", "k", "positions") else x[n] for n in IN])
    vt, S1 = torch.randn(B, Hk, dv, device="cuda").to(dtype), S.clone()
    ot = ops.linear_attn_decode_step(qt, kt, vt, ld, S1)
    w1, _, m1, _ = lo.prefill(qt[:, None], kt[:, None], vt[:, None], ld, D ** -0.5, S)
    assert (np.abs(np64(ot) - w1[:, 0]) <= n * m1[:, 0] + (U * np.abs(w1[:, 0]) if dtype == torch.bfloat16 else 0)).all()
    ops.device_status()


@pytest.mark.parametrize("dtype", DTYPES)
def test_without_an_epsilon(dtype):
    """eps = 0 with rows that do not fill a block: the places without a row add nothing to the weights' gradients."""
    x = make((5,), 3, 2, 64, 32, dtype, 12)
    args = [x[n] for n in IN]
    got = ops.qk_norm_rope_backward(x["dq_out"], x["dk_out"], *args, eps=0.0)
    for n in "qk":
        dx, dw, mx, mw = lo.norm_rope_grads(x[n], x[n + "_weight"], x["positions"], x["inv_freq"], 0.0, False,
                                            x["d%s_out" % n])
        big = np.max(mx, -1, keepdims=True)
        assert (np.abs(np64(got[n]) - dx) <= bound(dx, 2 * big, dtype, 16 + 64)).all()
        dy = np.max(np.abs(np64(x["d%s_out" % n])))
        # 15 terms, each off by 16 roundings of the pair's larger channel (|x r| <= sqrt(64) = 8)
        assert (np.abs(np64(got[n + "_weight"]) - dw) <= 32 * E * (mw + 15 * 8 * 2 * dy)).all()
