"""Linear attention and the query / key norm with rotation, on the CPU: the fp64 definitions against finite
differences, and every refusal of the C entry points (no call here reaches a kernel launch)."""
import ctypes

import numpy as np
import pytest
import torch

import linear_attn_oracle as lo
from selective_state_space_43_b200 import build as build_mod
from selective_state_space_43_b200 import ops

NULL, SHAPE, DTYPE, ALIGN, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5, 7
BASE = 1 << 40  # fake device addresses, far apart


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return ops.lib()


def rand(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape))


@pytest.mark.parametrize("cu", [None, [0, 3, 3, 4, 7]])
def test_gradients_of_the_definition_match_differences(cu):
    rng = np.random.default_rng(5)
    lead = (2, 4) if cu is None else (7,)
    n = 2 if cu is None else 4
    x = dict(q=rand(rng, *lead, 4, 3), k=rand(rng, *lead, 2, 3), v=rand(rng, *lead, 2, 5), init=rand(rng, n, 4, 3, 5))
    ld, do, dS = -torch.tensor([0.0, 0.1, 1.0, 3.0]).double(), rand(rng, *lead, 4, 5), rand(rng, n, 4, 3, 5)

    def loss(**kw):
        y = {**x, **kw}
        o, S, _, _ = lo.prefill(y["q"], y["k"], y["v"], ld, 0.7, y["init"], cu)
        return float((o * do.numpy()).sum() + (S * dS.numpy()).sum())

    got, _ = lo.backward(x["q"], x["k"], x["v"], ld, 0.7, do, x["init"], dS, cu)
    for name, key in (("q", "q"), ("k", "k"), ("v", "v"), ("init", "init_state")):
        dirn = rand(rng, *x[name].shape)
        h = 1e-5
        diff = (loss(**{name: x[name] + h * dirn}) - loss(**{name: x[name] - h * dirn})) / (2 * h)
        want = float((got[key] * dirn.numpy()).sum())
        # central differences of a quadratic form: exact but for cancellation, 2^-53 * |loss| / h
        assert abs(diff - want) <= 1e-7 * max(1.0, abs(want)), (name, diff, want)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_gradients_match_differences(interleaved):
    rng = np.random.default_rng(6)
    x, w, dy = rand(rng, 3, 2, 16), rand(rng, 16), rand(rng, 3, 2, 16)
    pos, freq = torch.tensor([0, 7, 131071]), torch.tensor([1.0, 0.3, 0.01, 1e-4])
    dx, dw, _, _ = lo.norm_rope_grads(x, w, pos, freq, 1e-6, interleaved, dy)
    for t, g in ((x, dx), (w, dw)):
        dirn, h = rand(rng, *t.shape), 1e-5
        f = [float((lo.norm_rope(*((t + s * h * dirn, w) if t is x else (x, t + s * h * dirn)), pos, freq, 1e-6,
                                 interleaved) * dy.numpy()).sum()) for s in (1, -1)]
        # the third derivative's term is of order h^2
        assert abs((f[0] - f[1]) / (2 * h) - float((g * dirn.numpy()).sum())) <= 1e-6


def la_dims(**kw):
    base = dict(batch=2, seqlen=64, nheads=8, kv_heads=4, key_dim=64, value_dim=128)
    base.update(kw)
    return ops.SsdLinearAttnDims(*[base[n] for n, _ in ops.SsdLinearAttnDims._fields_])


BAD_DIMS = [dict(batch=-1), dict(seqlen=-1), dict(nheads=0), dict(kv_heads=0), dict(kv_heads=3), dict(key_dim=0),
            dict(key_dim=12), dict(key_dim=136), dict(value_dim=4), dict(value_dim=256), dict(nheads=65536, kv_heads=1),
            dict(batch=1 << 31), dict(batch=1 << 28, nheads=16), dict(seqlen=1 << 31), dict(batch=1 << 16, seqlen=1 << 16)]


def vp(i, off=0):
    return ctypes.c_void_p(BASE * (i + 1) + off)


def prefill_call(L, d, dtype=ops.SSD_BF16, scale=1.0, strides=None, ptrs=None, ws=(None, 0)):
    p = dict(log_decay=vp(0), cu=None, q=vp(1), k=vp(2), v=vp(3), init=vp(4), o=vp(5), final=vp(6))
    p.update(ptrs or {})
    return L.ssd_linear_attn_prefill(ctypes.byref(d) if d else None, dtype, p["log_decay"], scale,
                                     ctypes.byref(strides) if strides else None, p["cu"], p["q"], p["k"], p["v"],
                                     p["init"], p["o"], p["final"], ws[0], ws[1], None)


def test_prefill_refuses(L):
    assert prefill_call(L, None) == NULL
    for bad in BAD_DIMS:
        assert prefill_call(L, la_dims(**bad)) == SHAPE, bad
    assert prefill_call(L, la_dims(), dtype=ops.SSD_BF16_YF32) == DTYPE
    assert prefill_call(L, la_dims(), dtype=7) == DTYPE
    for scale in (float("nan"), float("inf")):
        assert prefill_call(L, la_dims(), scale=scale) == SHAPE
    for name in ("log_decay", "q", "k", "v", "o", "final"):
        assert prefill_call(L, la_dims(), ptrs={name: None}) == NULL, name
    for i, name in ((1, "q"), (2, "k"), (3, "v"), (4, "init"), (5, "o"), (6, "final")):
        assert prefill_call(L, la_dims(), ptrs={name: vp(i, 8)}) == ALIGN, name
    assert prefill_call(L, la_dims(), ptrs=dict(log_decay=vp(0, 2))) == ALIGN
    assert prefill_call(L, la_dims(), ptrs=dict(cu=vp(7, 4))) == ALIGN
    w = (8 * 64, 4 * 64, 4 * 128)
    for j in range(3):
        st = list(w)
        st[j] -= 8
        assert prefill_call(L, la_dims(), strides=ops.SsdLinearAttnStrides(*st)) == SHAPE
        st[j] += 12
        assert prefill_call(L, la_dims(), strides=ops.SsdLinearAttnStrides(*st)) == ALIGN
        st[j] = 1 << 40
        assert prefill_call(L, la_dims(), strides=ops.SsdLinearAttnStrides(*st)) == SHAPE
    # outputs over inputs or one another
    for name in ("q", "k", "v", "init", "final", "log_decay"):
        i = dict(q=1, k=2, v=3, init=4, final=6, log_decay=0)[name]
        assert prefill_call(L, la_dims(), ptrs=dict(o=vp(i))) == UNSUPPORTED, name
    for i in (0, 1, 2, 3):
        assert prefill_call(L, la_dims(), ptrs=dict(final=vp(i))) == UNSUPPORTED
    assert prefill_call(L, la_dims(), ptrs=dict(final=vp(4, 32))) == UNSUPPORTED  # part of init_state
    assert prefill_call(L, la_dims(batch=0), ptrs=dict(q=None, k=None, v=None, o=None, final=None, init=None)) == 0


def test_prefill_wants_its_workspace(L):
    for dtype in (ops.SSD_F32, ops.SSD_BF16):
        for packed in (0, 1):
            for kw in (dict(), dict(batch=1, nheads=4, seqlen=100000)):
                d = la_dims(**kw)
                need = L.ssd_linear_attn_prefill_workspace_bytes(ctypes.byref(d), dtype, packed)
                ptrs = dict(cu=vp(7)) if packed else {}
                if need:
                    assert prefill_call(L, d, dtype, ptrs=ptrs) == WORKSPACE
                    assert prefill_call(L, d, dtype, ptrs=ptrs, ws=(vp(8), need - 1)) == WORKSPACE
                    assert prefill_call(L, d, dtype, ptrs=ptrs, ws=(vp(8, 8), need)) == ALIGN
                    assert prefill_call(L, d, dtype, ptrs=ptrs, ws=(vp(5), need)) == UNSUPPORTED
    assert L.ssd_linear_attn_prefill_workspace_bytes(ctypes.byref(la_dims(key_dim=7)), ops.SSD_BF16, 0) == 0


def backward_call(L, d, dtype=ops.SSD_BF16, scale=1.0, ptrs=None, ws=None):
    names = ["log_decay", "q", "k", "v", "init", "do", "d_final", "dq", "dk", "dv", "d_init"]
    p = {n: vp(i) for i, n in enumerate(names)}
    p["cu"] = None
    p.update(ptrs or {})
    if ws is None:
        ws = (vp(20), 1 << 40)
    return L.ssd_linear_attn_backward(ctypes.byref(d) if d else None, dtype, p["log_decay"], scale, p["cu"], p["q"],
                                      p["k"], p["v"], p["init"], p["do"], p["d_final"], p["dq"], p["dk"], p["dv"],
                                      p["d_init"], ws[0], ws[1], None)


def test_backward_refuses(L):
    assert backward_call(L, None) == NULL
    for bad in BAD_DIMS:
        assert backward_call(L, la_dims(**bad)) == SHAPE, bad
    assert backward_call(L, la_dims(), dtype=ops.SSD_BF16_YF32) == DTYPE
    assert backward_call(L, la_dims(), scale=float("nan")) == SHAPE
    names = ["log_decay", "q", "k", "v", "init", "do", "d_final", "dq", "dk", "dv", "d_init"]
    for name in ("log_decay", "q", "k", "v", "do", "dq", "dk", "dv"):
        assert backward_call(L, la_dims(), ptrs={name: None}) == NULL, name
    for i, name in enumerate(names):
        off = 2 if name == "log_decay" else 8
        assert backward_call(L, la_dims(), ptrs={name: vp(i, off)}) == ALIGN, name
    for out in ("dq", "dk", "dv", "d_init"):
        for i, name in enumerate(names):
            if name != out:
                assert backward_call(L, la_dims(), ptrs={out: vp(i)}) == UNSUPPORTED, (out, name)
        assert backward_call(L, la_dims(), ptrs={out: vp(20)}) == UNSUPPORTED
    need = L.ssd_linear_attn_backward_workspace_bytes(ctypes.byref(la_dims()), ops.SSD_BF16, 0)
    assert need > 0  # shared key and value heads
    assert backward_call(L, la_dims(), ws=(None, 0)) == WORKSPACE
    assert backward_call(L, la_dims(), ws=(vp(20), need - 1)) == WORKSPACE
    assert backward_call(L, la_dims(batch=0), ptrs={n: None for n in names if n != "log_decay"}) == 0


def decode_call(L, d, dtype=ops.SSD_BF16, scale=1.0, ptrs=None):
    p = dict(log_decay=vp(0), q=vp(1), k=vp(2), v=vp(3), state=vp(4), o=vp(5))
    p.update(ptrs or {})
    return L.ssd_linear_attn_decode_step(ctypes.byref(d) if d else None, dtype, p["log_decay"], scale, p["q"], p["k"],
                                         p["v"], p["state"], p["o"], None)


def test_decode_refuses(L):
    assert decode_call(L, None) == NULL
    for bad in BAD_DIMS:
        if "seqlen" not in bad:
            assert decode_call(L, la_dims(**bad)) == SHAPE, bad
    assert decode_call(L, la_dims(), dtype=ops.SSD_BF16_YF32) == DTYPE
    assert decode_call(L, la_dims(), scale=float("inf")) == SHAPE
    for i, name in enumerate(("log_decay", "q", "k", "v", "state", "o")):
        assert decode_call(L, la_dims(), ptrs={name: None}) == NULL, name
        assert decode_call(L, la_dims(), ptrs={name: vp(i, 2)}) == ALIGN, name
    for i in range(5):
        assert decode_call(L, la_dims(), ptrs=dict(o=vp(i))) == UNSUPPORTED
    for i in range(4):
        assert decode_call(L, la_dims(), ptrs=dict(state=vp(i))) == UNSUPPORTED
    assert decode_call(L, la_dims(batch=0), ptrs=dict(q=None, k=None, v=None, state=None, o=None)) == 0


QK = ["q", "k", "q_weight", "k_weight", "positions", "inv_freq", "q_out", "k_out"]
BAD_QK = [dict(tokens=-1), dict(q_heads=0), dict(k_heads=0), dict(head_dim=0), dict(head_dim=12), dict(head_dim=264),
          dict(rot_dim=-8), dict(rot_dim=12), dict(rot_dim=136), dict(tokens=1 << 31), dict(q_heads=1 << 20),
          dict(k_heads=1 << 20)]


def qk_dims(**kw):
    base = dict(tokens=5, q_heads=8, k_heads=2, head_dim=128, rot_dim=64, interleaved=0)
    base.update(kw)
    return ops.SsdQkDims(*[base[n] for n, _ in ops.SsdQkDims._fields_])


def qk_call(L, d, dtype=ops.SSD_BF16, eps=1e-6, strides=None, ptrs=None):
    p = {n: vp(i) for i, n in enumerate(QK)}
    p.update(ptrs or {})
    return L.ssd_qk_norm_rope(ctypes.byref(d) if d else None, dtype, eps, ctypes.byref(strides) if strides else None,
                              *[p[n] for n in QK], None)


def qk_backward_call(L, d, dtype=ops.SSD_BF16, eps=1e-6, strides=None, ptrs=None, ws=None):
    names = ["dq_out", "dk_out", "q", "k", "q_weight", "k_weight", "positions", "inv_freq", "dq", "dk", "dq_weight",
             "dk_weight"]
    p = {n: vp(i) for i, n in enumerate(names)}
    p.update(ptrs or {})
    ws = ws or (vp(20), 1 << 40)
    return L.ssd_qk_norm_rope_backward(ctypes.byref(d) if d else None, dtype, eps,
                                       ctypes.byref(strides) if strides else None, *[p[n] for n in names], ws[0],
                                       ws[1], None)


@pytest.mark.parametrize("call", [qk_call, qk_backward_call])
def test_norm_rope_refuses(L, call):
    assert call(L, None) == NULL
    for bad in BAD_QK:
        assert call(L, qk_dims(**bad)) == SHAPE, bad
    assert call(L, qk_dims(), dtype=ops.SSD_BF16_YF32) == DTYPE
    for eps in (-1.0, float("nan"), float("inf")):
        assert call(L, qk_dims(), eps=eps) == SHAPE
    assert call(L, qk_dims(), strides=ops.SsdQkStrides(8 * 128 - 8, 256)) == SHAPE
    assert call(L, qk_dims(), strides=ops.SsdQkStrides(8 * 128 + 4, 256)) == ALIGN
    assert call(L, qk_dims(), strides=ops.SsdQkStrides(8 * 128, 1 << 40)) == SHAPE
    for name in ("q", "k", "q_weight", "k_weight", "positions", "inv_freq"):
        assert call(L, qk_dims(), ptrs={name: None}) == NULL, name
        assert call(L, qk_dims(), ptrs={name: vp(9, 2)}) == ALIGN, name


def test_norm_rope_refuses_overlaps(L):
    for i, name in enumerate(QK):
        if name not in ("q_out", "q"):
            assert qk_call(L, qk_dims(), ptrs=dict(q_out=vp(i))) == UNSUPPORTED, name
        if name not in ("k_out", "k"):
            assert qk_call(L, qk_dims(), ptrs=dict(k_out=vp(i))) == UNSUPPORTED, name
    # in place only where the input is contiguous
    st = ops.SsdQkStrides(2000, 256)
    assert qk_call(L, qk_dims(), strides=st, ptrs=dict(q_out=vp(0))) == UNSUPPORTED
    assert qk_call(L, qk_dims(), ptrs=dict(q_out=vp(0, 256))) == UNSUPPORTED
    assert qk_call(L, qk_dims(tokens=0), ptrs={n: None for n in ("q", "k", "positions", "q_out", "k_out")}) == 0


def test_norm_rope_backward_refuses_overlaps_and_a_small_workspace(L):
    names = ["dq_out", "dk_out", "q", "k", "q_weight", "k_weight", "positions", "inv_freq", "dq", "dk", "dq_weight",
             "dk_weight"]
    for out in names[8:]:
        for i, name in enumerate(names):
            if name != out:
                assert qk_backward_call(L, qk_dims(), ptrs={out: vp(i)}) == UNSUPPORTED, (out, name)
    need = L.ssd_qk_norm_rope_backward_workspace_bytes(ctypes.byref(qk_dims()))
    assert need > 0
    assert qk_backward_call(L, qk_dims(), ws=(vp(20), need - 1)) == WORKSPACE


def test_a_workspace_over_an_input_is_refused(L):
    """The kernels write it while others still read the inputs."""
    d = la_dims(batch=1, nheads=4, seqlen=100000)
    need = L.ssd_linear_attn_prefill_workspace_bytes(ctypes.byref(d), ops.SSD_BF16, 0)
    assert need > 0
    for i in range(5):  # log_decay, q, k, v, init_state
        assert prefill_call(L, d, ws=(vp(i), need)) == UNSUPPORTED, i
    for i in range(11):
        assert backward_call(L, la_dims(), ws=(vp(i), 1 << 40)) == UNSUPPORTED, i
    for i in range(12):
        assert qk_backward_call(L, qk_dims(), ws=(vp(i), 1 << 30)) == UNSUPPORTED, i


def test_binding_checks_tensors():
    t = torch.zeros(1, 4, 2, 64)
    with pytest.raises(ValueError):
        ops.linear_attn_prefill(t, t, t, torch.zeros(2))  # not on a CUDA device
    with pytest.raises(ValueError):
        ops.linear_attn_backward(t, t, t, torch.zeros(2), t)
    with pytest.raises(ValueError):
        ops.linear_attn_decode_step(t[:, 0], t[:, 0], t[:, 0], torch.zeros(2), torch.zeros(1, 2, 64, 64))
    with pytest.raises(ValueError):
        ops.qk_norm_rope(t, t, torch.ones(64), torch.ones(64), torch.zeros(1, 4, dtype=torch.int64), torch.ones(32))
