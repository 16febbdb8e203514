"""Linear attention on the GPU against the fp64 token-by-token definition.

Tolerances.  u = 2^-8 is half a bf16 step, relative; e = 2^-24 half an fp32 one.  A bf16 output is rounded once
(u |o|), and the chunked form rounds each score, or each state element, to bf16 before its product with a value
or a query: every term of the sum is off by at most u of itself, so |error| <= u |o| + u mag (1 + small) with mag
the sum of the terms' absolute values.  fp32 sums of n terms are off by at most n e mag.  States from bf16 rows
carry their weights in enough bf16 parts that only fp32 rounding is left.
"""
import numpy as np
import pytest
import torch

import linear_attn_oracle as lo

pytestmark = pytest.mark.gpu

from selective_state_space_43_b200 import ops  # noqa: E402

U, E = 2.0 ** -8, 2.0 ** -24
DTYPES = [torch.bfloat16, torch.float32]


def np64(t):
    return t.detach().cpu().double().numpy()


def make(seed, lead, H, Hk, dk, dv, dtype, nseq=None, init=False, grads=False):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, dt=dtype):
        return torch.randn(shape, generator=g).to(dt).cuda()

    x = dict(q=normal(*lead, H, dk), k=normal(*lead, Hk, dk), v=normal(*lead, Hk, dv))
    x["log_decay"] = -torch.exp(torch.rand(H, generator=g) * -np.log(1024.0)).cuda()
    n = lead[0] if nseq is None else nseq
    x["init"] = normal(n, H, dk, dv, dt=torch.float32) if init else None
    if grads:
        x["do"] = normal(*lead, H, dv)
        x["d_final"] = normal(n, H, dk, dv, dt=torch.float32) if init else None
    return x


def n_terms(length, dk):
    """Roundings on the way of a sum of fp32 products: a dot product over dk, one over a chunk, one for each
    chunk that the state passes, and the few of the decays (exponents of l n are off by |l n| e, weighted by
    e^{l n}: below 1)."""
    return dk + 128 + length // 16 + 16


def check_out(got, want, mag, dtype, length, dk, what):
    got = np64(got)
    live = ~np.isnan(want)
    assert np.isfinite(got[live]).all(), what
    err, n = np.abs(got - want)[live], n_terms(length, dk)
    tol = n * E * mag[live] + 1e-30
    if dtype == torch.bfloat16:
        tol = tol + U * np.abs(want[live]) + 1.02 * U * mag[live]
    bad = err > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max(err / tol):.2f} of its bound"
    if dtype == torch.bfloat16 and err.size > 1000:
        # three independent roundings (score, state, output) of relative rms u / sqrt(3): on terms of random
        # signs their sum is below u sqrt(3) / sqrt(3) = u of the result's norm
        assert np.linalg.norm(err) <= 1.3 * U * np.linalg.norm(want[live]), what


def check_state(got, want, mag, length, dk, what):
    got = np64(got)
    err, tol = np.abs(got - want), n_terms(length, dk) * E * mag + 1e-30
    assert not (err > tol).any(), f"{what}: worst {np.nanmax(err / tol):.2f} of its bound"


SHAPES = [(1, 1, 1, 8, 8), (2, 1, 2, 64, 64), (2, 2, 1, 128, 64), (1, 31, 3, 64, 128), (3, 32, 2, 32, 96),
          (1, 127, 2, 128, 128), (2, 128, 1, 80, 40), (1, 129, 4, 64, 64), (2, 300, 3, 128, 128), (1, 517, 1, 96, 72),
          (1, 1100, 1, 128, 64), (2, 1025, 2, 64, 8)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,L,Hk,dk,dv", SHAPES)
def test_prefill(B, L, Hk, dk, dv, dtype):
    init, group = (B + L) % 2 == 1, 1 + L % 3
    x = make(L * 7 + dk, (B, L), Hk * group, Hk, dk, dv, dtype, init=init)
    o, S = ops.linear_attn_prefill(x["q"], x["k"], x["v"], x["log_decay"], x["init"])
    ops.device_status()
    wo, wS, mo, mS = lo.prefill(x["q"], x["k"], x["v"], x["log_decay"], dk ** -0.5, x["init"])
    check_out(o, wo, mo, dtype, L, dk, "o")
    check_state(S, wS, mS, L, dk, "final_state")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,L,Hk,dk,dv", SHAPES)
def test_backward(B, L, Hk, dk, dv, dtype):
    init, group = (B + L) % 2 == 0, 1 + L % 3
    x = make(L * 11 + dv, (B, L), Hk * group, Hk, dk, dv, dtype, init=init, grads=True)
    got = ops.linear_attn_backward(x["q"], x["k"], x["v"], x["log_decay"], x["do"], x["init"], x["d_final"], scale=0.3)
    ops.device_status()
    want, mag = lo.backward(x["q"], x["k"], x["v"], x["log_decay"], 0.3, x["do"], x["init"], x["d_final"])
    for name in "qkv":
        check_out(got[name], want[name], mag[name], dtype, L, max(dk, dv), "d" + name)
    check_state(got["init_state"], want["init_state"], mag["init_state"], L, max(dk, dv), "d_init_state")


CUTS = [[0, 5], [0, 0, 1, 1, 130, 386, 386], [3, 3, 131, 260, 300], [0, 128, 256, 384], [0, 1, 2, 3, 1029]]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cu", CUTS)
@pytest.mark.parametrize("dk,dv,init", [(64, 128, True), (128, 64, False), (40, 96, True)])
def test_packed(cu, dk, dv, init, dtype):
    """Empty, single-token and chunk-straddling sequences; rows in front of the first and behind the last one hold
    NaN and are neither read nor written."""
    T, n, H, Hk = cu[-1] + 37, len(cu) - 1, 4, 2
    x = make(sum(cu) + dk, (T,), H, Hk, dk, dv, dtype, nseq=n, init=init, grads=True)
    for name in ("q", "k", "v", "do"):
        x[name][cu[-1]:] = float("nan")
        x[name][:cu[0]] = float("inf")
    o = torch.full((T, H, dv), 7.0, dtype=dtype, device="cuda")
    o, S = ops.linear_attn_prefill_varlen(x["q"], x["k"], x["v"], x["log_decay"], cu, x["init"], scale=0.2, o=o)
    ops.device_status()
    assert (o[cu[-1]:] == 7).all() and (o[:cu[0]] == 7).all()
    clean = {k: None if v is None else torch.nan_to_num(v, 0, 0, 0) for k, v in x.items()}
    wo, wS, mo, mS = lo.prefill(clean["q"], clean["k"], clean["v"], x["log_decay"], 0.2, x["init"], cu)
    longest = max(b - a for a, b in zip(cu, cu[1:]))
    check_out(o, wo, mo, dtype, longest, dk, "o")
    check_state(S, wS, mS, longest, dk, "final_state")
    got = ops.linear_attn_backward(x["q"], x["k"], x["v"], x["log_decay"], x["do"], x["init"], x["d_final"], scale=0.2,
                                   cu_seqlens=torch.tensor(cu).cuda())
    ops.device_status()
    want, mag = lo.backward(clean["q"], clean["k"], clean["v"], x["log_decay"], 0.2, clean["do"], x["init"],
                            x["d_final"], cu)
    for name in "qkv":
        check_out(got[name], want[name], mag[name], dtype, longest, max(dk, dv), "d" + name)
    check_state(got["init_state"], want["init_state"], mag["init_state"], longest, max(dk, dv), "d_init_state")


@pytest.mark.parametrize("dtype", DTYPES)
def test_one_sequence_does_not_reach_another(dtype):
    """A sequence of infinities and NaN next to others, batched and packed: theirs stay as without it."""
    x = make(3, (3, 150), 2, 2, 64, 64, dtype, grads=True)
    dirty = {k: None if v is None else v.clone() for k, v in x.items()}
    for name in ("q", "k", "v", "do"):
        dirty[name][1] = float("nan")
        dirty[name][1, 3] = float("inf")
    cu = torch.tensor([0, 150, 300, 450]).cuda()
    for y, z in ((x, dirty),):
        runs = []
        for d in (y, z):
            o, S = ops.linear_attn_prefill(d["q"], d["k"], d["v"], d["log_decay"])
            g = ops.linear_attn_backward(d["q"], d["k"], d["v"], d["log_decay"], d["do"])
            flat = {n: d[n].flatten(0, 1) for n in ("q", "k", "v", "do")}
            op, Sp = ops.linear_attn_prefill_varlen(flat["q"], flat["k"], flat["v"], d["log_decay"], cu)
            runs.append([o, S, g["q"], g["k"], g["v"], g["init_state"], op.unflatten(0, (3, 150)), Sp])
        for a, b in zip(*runs):
            assert torch.equal(a[[0, 2]], b[[0, 2]])


@pytest.mark.parametrize("dtype", DTYPES)
def test_padding_behind_a_prompt_does_not_reach_it(dtype):
    """Right-padded batches: what stands behind a prompt's rows, a NaN outside its last chunk among it, changes
    nothing in front."""
    x = make(4, (2, 400), 2, 2, 64, 64, dtype)
    o, _ = ops.linear_attn_prefill(x["q"], x["k"], x["v"], x["log_decay"])
    y = {k: None if v is None else v.clone() for k, v in x.items()}
    for name in ("q", "k", "v"):
        y[name][:, 200:256] = 5.0
        y[name][:, 256:] = float("nan")
    o2, _ = ops.linear_attn_prefill(y["q"], y["k"], y["v"], y["log_decay"])
    assert torch.equal(o[:, :200], o2[:, :200])


@pytest.mark.parametrize("dtype", DTYPES)
def test_decays_at_their_ends(dtype):
    """log_decay 0 (a plain sum), one so fast that it underflows within a chunk, and -inf (each token alone)."""
    x = make(8, (1, 260), 4, 4, 64, 64, dtype, init=True, grads=True)
    x["log_decay"] = torch.tensor([0.0, -30.0, -1e30, float("-inf")]).cuda()
    o, S = ops.linear_attn_prefill(x["q"], x["k"], x["v"], x["log_decay"], x["init"])
    g = ops.linear_attn_backward(x["q"], x["k"], x["v"], x["log_decay"], x["do"], x["init"], x["d_final"])
    wo, wS, mo, mS = lo.prefill(x["q"], x["k"], x["v"], x["log_decay"], 0.125, x["init"])
    check_out(o, wo, mo, dtype, 260, 64, "o")
    check_state(S, wS, mS, 260, 64, "final_state")
    want, mag = lo.backward(x["q"], x["k"], x["v"], x["log_decay"], 0.125, x["do"], x["init"], x["d_final"])
    for name in "qkv":
        check_out(g[name], want[name], mag[name], dtype, 260, 64, "d" + name)
    check_state(g["init_state"], want["init_state"], mag["init_state"], 260, 64, "d_init_state")
    st = x["init"].clone()
    od = ops.linear_attn_decode_step(x["q"][:, 0], x["k"][:, 0], x["v"][:, 0], x["log_decay"], st)
    check_out(od, wo[:, 0], mo[:, 0], dtype, 1, 64, "decode")


@pytest.mark.parametrize("dtype", DTYPES)
def test_strided_rows_give_the_same_bits(dtype):
    H, Hk, dk, dv = 4, 2, 64, 128
    wide = torch.randn(2, 200, H * dk + Hk * (dk + dv) + 16, device="cuda").to(dtype)
    q, k, v = wide[..., 8:-8].split([H * dk, Hk * dk, Hk * dv], -1)
    q, k, v = q.unflatten(-1, (H, dk)), k.unflatten(-1, (Hk, dk)), v.unflatten(-1, (Hk, dv))
    ld = -torch.rand(H, device="cuda")
    a = ops.linear_attn_prefill(q, k, v, ld)
    b = ops.linear_attn_prefill(q.contiguous(), k.contiguous(), v.contiguous(), ld)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    cu = torch.tensor([0, 60, 200]).cuda()
    a = ops.linear_attn_prefill_varlen(q[1], k[1], v[1], ld, cu)
    b = ops.linear_attn_prefill_varlen(q[1].contiguous(), k[1].contiguous(), v[1].contiguous(), ld, cu)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_split_prompt_carries_its_state_in_place(dtype):
    """Two calls, the state handed on in the same tensor, against one; then tokens one at a time."""
    x = make(9, (2, 333), 4, 2, 128, 64, dtype, init=True)
    state = x["init"].clone()
    parts = []
    for a, b in ((0, 130), (130, 330)):
        o, s = ops.linear_attn_prefill(*(x[n][:, a:b].contiguous() for n in "qkv"), x["log_decay"], state,
                                       final_state=state)
        assert s is state
        parts.append(o)
    for t in range(330, 333):
        parts.append(ops.linear_attn_decode_step(*(x[n][:, t].contiguous() for n in "qkv"), x["log_decay"],
                                                 state)[:, None])
    wo, wS, mo, mS = lo.prefill(x["q"], x["k"], x["v"], x["log_decay"], 128 ** -0.5, x["init"])
    check_out(torch.cat(parts, 1), wo, mo, dtype, 333, 128, "o")
    check_state(state, wS, mS, 333, 128, "state")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,Hk,group,dk,dv", [(1, 1, 1, 8, 8), (1, 2, 3, 128, 128), (5, 3, 1, 128, 64), (33, 2, 2, 40, 96),
                                              (2, 1, 4, 64, 72), (300, 2, 1, 64, 128)])
def test_decode(B, Hk, group, dk, dv, dtype):
    H = Hk * group
    x = make(B + dv, (B,), H, Hk, dk, dv, dtype, init=True)
    state = x["init"].clone()
    S = np64(state)
    for step in range(3):
        y = make(1000 + step, (B,), H, Hk, dk, dv, dtype)
        o = ops.linear_attn_decode_step(y["q"], y["k"], y["v"], x["log_decay"], state, scale=0.5)
        wo, wS, mo, mS = lo.prefill(y["q"][:, None], y["k"][:, None], y["v"][:, None], x["log_decay"], 0.5,
                                    torch.from_numpy(S))
        err = np.abs(np64(o) - wo[:, 0])
        tol = n_terms(1, dk) * E * mo[:, 0] + (U * np.abs(wo[:, 0]) if dtype == torch.bfloat16 else 0)
        assert (err <= tol).all()
        check_state(state, wS, mS, 1, dk, "state")
        S = np64(state)
    ops.device_status()


def test_no_rows():
    z = torch.zeros(2, 0, 2, 64, device="cuda", dtype=torch.bfloat16)
    ld, init = torch.zeros(2, device="cuda"), torch.randn(2, 2, 64, 64, device="cuda")
    o, S = ops.linear_attn_prefill(z, z, z, ld, init)
    assert o.shape == (2, 0, 2, 64) and torch.equal(S, init)
    g = ops.linear_attn_backward(z, z, z, ld, z, init, init)
    assert torch.equal(g["init_state"], init)
    assert torch.equal(ops.linear_attn_prefill(z, z, z, ld)[1], torch.zeros_like(init))
    e = torch.zeros(0, 5, 2, 64, device="cuda", dtype=torch.bfloat16)
    o, S = ops.linear_attn_prefill(e, e, e, ld)
    assert o.numel() == 0 and S.numel() == 0
    assert ops.linear_attn_decode_step(e[:, 0], e[:, 0], e[:, 0], ld, S).numel() == 0


@pytest.mark.parametrize("dtype", DTYPES)
def test_bad_offsets_are_reported(dtype):
    x = make(1, (200,), 2, 2, 64, 64, dtype, nseq=3, init=True)
    good = ops.linear_attn_prefill_varlen(x["q"], x["k"], x["v"], x["log_decay"], [0, 100, 100, 200], x["init"])
    for cu in ([0, 100, 90, 200], [0, 100, 100, 201], [-1, 100, 100, 200], [0, 1 << 60, 100, 200]):
        o, S = ops.linear_attn_prefill_varlen(x["q"], x["k"], x["v"], x["log_decay"], cu, x["init"])
        with pytest.raises(ops.SsdError):
            ops.device_status()
        ops.device_status()  # reading clears it
        if cu[1] == 100 and cu[0] == 0:
            # short enough not to be cut into segments, so the valid sequences are computed; rows 90 .. 99 belong to two
            # of them in the first list
            assert torch.equal(o[:90], good[0][:90]) and torch.equal(S[0], good[1][0])


@pytest.mark.parametrize("dtype", DTYPES)
def test_graphs_streams_and_reuse(dtype):
    """A captured prefill, step and backward, replayed on new data on another stream, while eager calls of the same
    inputs run; two graphs at once."""
    dk, dv, H = 128, 64, 4
    x = make(2, (1, 700), H, 2, dk, dv, dtype, init=True, grads=True)
    tok = make(3, (1,), H, 2, dk, dv, dtype)
    state = x["init"].clone()

    def step():
        o, S = ops.linear_attn_prefill(x["q"], x["k"], x["v"], x["log_decay"], x["init"])
        state.copy_(S)
        t = ops.linear_attn_decode_step(tok["q"], tok["k"], tok["v"], x["log_decay"], state)
        g = ops.linear_attn_backward(x["q"], x["k"], x["v"], x["log_decay"], x["do"], x["init"], x["d_final"])
        return [o, S, t, g["q"], g["k"], g["v"], g["init_state"]]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    fresh = make(77, (1, 700), H, 2, dk, dv, dtype, init=True, grads=True)
    for name in ("q", "k", "v", "do", "init", "d_final"):
        x[name].copy_(fresh[name])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for g, _ in graphs:
            g.replay()
    eager = step()
    with torch.cuda.stream(side):
        graphs[0][0].replay()
    torch.cuda.synchronize()
    ops.device_status()
    for _, out in graphs:
        for a, b in zip(out[:2] + out[3:], eager[:2] + eager[3:]):
            assert torch.equal(a, b)


def test_two_calls_at_once_and_the_same_bits_each_time():
    x = make(5, (1, 3000), 8, 4, 64, 64, torch.bfloat16, init=True, grads=True)
    want = ops.linear_attn_backward(x["q"], x["k"], x["v"], x["log_decay"], x["do"], x["init"], x["d_final"])
    wo = ops.linear_attn_prefill(x["q"], x["k"], x["v"], x["log_decay"], x["init"])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append((ops.linear_attn_backward(x["q"], x["k"], x["v"], x["log_decay"], x["do"], x["init"],
                                                 x["d_final"]),
                        ops.linear_attn_prefill(x["q"], x["k"], x["v"], x["log_decay"], x["init"])))
    torch.cuda.synchronize()
    for g, o in got:
        assert all(torch.equal(g[n], want[n]) for n in want) and torch.equal(o[0], wo[0]) and torch.equal(o[1], wo[1])


def test_a_small_workspace_is_replaced_and_wrong_tensors_are_refused():
    x = make(6, (1, 3000), 4, 2, 64, 64, torch.bfloat16)
    args = (x["q"], x["k"], x["v"], x["log_decay"])
    a = ops.linear_attn_prefill(*args)
    b = ops.linear_attn_prefill(*args, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    c = ops.linear_attn_prefill(*args, workspace=torch.empty(1 << 26, dtype=torch.uint8, device="cuda"))
    assert torch.equal(a[0], b[0]) and torch.equal(a[0], c[0])
    with pytest.raises(TypeError):
        ops.linear_attn_prefill(x["q"].half(), x["k"].half(), x["v"].half(), x["log_decay"])
    with pytest.raises(TypeError):
        ops.linear_attn_prefill(x["q"], x["k"].float(), x["v"], x["log_decay"])
    with pytest.raises(ValueError):
        ops.linear_attn_prefill(x["q"], x["k"], x["v"], x["log_decay"][:3])
    with pytest.raises(ValueError):
        ops.linear_attn_prefill(x["q"].transpose(1, 2), x["k"], x["v"], x["log_decay"])
    with pytest.raises(ops.SsdError):
        ops.linear_attn_prefill(x["q"], x["k"], x["v"], x["log_decay"], o=x["q"])


def workspace_bytes(L, H, Hk, dk, dv, dtype, packed=False, B=1, backward=False):
    import ctypes
    f = ops.lib().ssd_linear_attn_backward_workspace_bytes if backward else ops.lib().ssd_linear_attn_prefill_workspace_bytes
    return f(ctypes.byref(ops.SsdLinearAttnDims(B, L, H, Hk, dk, dv)), 1 if dtype == torch.bfloat16 else 0, packed)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("L,Hk,group,dk,dv,init", [(2500, 2, 1, 64, 128, True), (4096, 1, 2, 128, 64, False),
                                                   (3333, 1, 1, 96, 40, True)])
def test_long_sequences_in_segments(L, Hk, group, dk, dv, init, dtype):
    """Few heads on a long sequence: the sequence axis is cut (the workspace holds the segments' states)."""
    H = Hk * group
    assert workspace_bytes(L, H, Hk, dk, dv, dtype) > 0
    x = make(L, (1, L), H, Hk, dk, dv, dtype, init=init, grads=True)
    x["log_decay"][0] = -1e-4  # one head remembers across every segment
    o, S = ops.linear_attn_prefill(x["q"], x["k"], x["v"], x["log_decay"], x["init"])
    got = ops.linear_attn_backward(x["q"], x["k"], x["v"], x["log_decay"], x["do"], x["init"], x["d_final"])
    ops.device_status()
    wo, wS, mo, mS = lo.prefill(x["q"], x["k"], x["v"], x["log_decay"], dk ** -0.5, x["init"])
    check_out(o, wo, mo, dtype, L, dk, "o")
    check_state(S, wS, mS, L, dk, "final_state")
    want, mag = lo.backward(x["q"], x["k"], x["v"], x["log_decay"], dk ** -0.5, x["do"], x["init"], x["d_final"])
    for name in "qkv":
        check_out(got[name], want[name], mag[name], dtype, L, max(dk, dv), "d" + name)
    check_state(got["init_state"], want["init_state"], mag["init_state"], L, max(dk, dv), "d_init_state")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cu", [[0, 0, 1500, 1501, 4000], [5, 261, 2821, 2821, 3077, 4001], [0, 4000]])
def test_packed_segments(cu, dtype):
    T, n, H, Hk, dk, dv = cu[-1] + 70, len(cu) - 1, 2, 1, 64, 64
    assert workspace_bytes(T, H, Hk, dk, dv, dtype, True, n) > 0
    x = make(sum(cu), (T,), H, Hk, dk, dv, dtype, nseq=n, init=True, grads=True)
    x["log_decay"][0] = -3e-4
    for name in ("q", "k", "v", "do"):
        x[name][cu[-1]:] = float("nan")
        x[name][:cu[0]] = float("nan")
    o = torch.full((T, H, dv), 7.0, dtype=dtype, device="cuda")
    o, S = ops.linear_attn_prefill_varlen(x["q"], x["k"], x["v"], x["log_decay"], cu, x["init"], o=o)
    got = ops.linear_attn_backward(x["q"], x["k"], x["v"], x["log_decay"], x["do"], x["init"], x["d_final"],
                                   cu_seqlens=cu)
    ops.device_status()
    assert (o[cu[-1]:] == 7).all() and (o[:cu[0]] == 7).all()
    clean = {k: None if v is None else torch.nan_to_num(v, 0, 0, 0) for k, v in x.items()}
    wo, wS, mo, mS = lo.prefill(clean["q"], clean["k"], clean["v"], x["log_decay"], 0.125, x["init"], cu)
    check_out(o, wo, mo, dtype, 4000, dk, "o")
    check_state(S, wS, mS, 4000, dk, "final_state")
    want, mag = lo.backward(clean["q"], clean["k"], clean["v"], x["log_decay"], 0.125, clean["do"], x["init"],
                            x["d_final"], cu)
    for name in "qkv":
        check_out(got[name], want[name], mag[name], dtype, 4000, dk, "d" + name)
    check_state(got["init_state"], want["init_state"], mag["init_state"], 4000, dk, "d_init_state")


@pytest.mark.parametrize("dtype", DTYPES)
def test_bad_offsets_in_segments(dtype):
    x = make(1, (4000,), 2, 2, 64, 64, dtype, nseq=3, init=True, grads=True)
    for cu in ([0, 3000, 2000, 4000], [0, 2000, 3000, 4001], [-1, 100, 100, 4000], [0, 1 << 60, 100, 4000],
               [4000, 0, 4000, 0]):
        ops.linear_attn_prefill_varlen(x["q"], x["k"], x["v"], x["log_decay"], cu, x["init"])
        with pytest.raises(ops.SsdError):
            ops.device_status()
        ops.linear_attn_backward(x["q"], x["k"], x["v"], x["log_decay"], x["do"], x["init"], x["d_final"], cu_seqlens=cu)
        with pytest.raises(ops.SsdError):
            ops.device_status()
        ops.device_status()


@pytest.mark.parametrize("L,H,dk,dv", [(1, 1, 64, 64), (1, 3, 128, 8), (2, 1, 32, 128), (5, 2, 64, 64), (128, 1, 96, 96)])
def test_a_lone_chunk_rounds_its_outputs_only(L, H, dk, dv):
    """Few outputs may share one score, whose rounding would then be all of theirs: a sequence of one chunk keeps its
    scores in two bf16 parts (2^-16 of themselves off), so that only the outputs' own rounding shows."""
    x = make(L + dk, (3, L), H, H, dk, dv, torch.bfloat16)
    o, _ = ops.linear_attn_prefill(x["q"], x["k"], x["v"], x["log_decay"])
    wo, _, mo, _ = lo.prefill(x["q"], x["k"], x["v"], x["log_decay"], dk ** -0.5)
    assert (np.abs(np64(o) - wo) <= U * np.abs(wo) * 1.001 + (2.0 ** -15 + n_terms(L, dk) * E) * mo).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("Hk", [1, 2])
@pytest.mark.parametrize("rows,cu", [(300, [7, 100, 263]), (4000, [5, 261, 2821, 3077]), (40, [9, 9]), (10, [10, 10])])
def test_gradients_outside_every_sequence_are_left_as_they_were(rows, cu, Hk, dtype):
    """The caller's dq, dk, dv through the C entry point, with heads of their own and shared ones (whose gradients are
    summed by a kernel of its own)."""
    import ctypes
    H, dk, dv, n = 2, 64, 40, len(cu) - 1
    x = make(rows, (rows,), H, Hk, dk, dv, dtype, nseq=n, grads=True)
    offsets = torch.tensor(cu).cuda()
    # the same call: a gradient of the initial state that nobody asks for leaves V' in fewer parts
    want = ops.linear_attn_backward(x["q"], x["k"], x["v"], x["log_decay"], x["do"], cu_seqlens=offsets,
                                    want_init_grads=False)
    got = {name: torch.full_like(x[name], 7.0) for name in "qkv"}
    ws = torch.full((workspace_bytes(rows, H, Hk, dk, dv, dtype, True, n, True) + 16,), 3, dtype=torch.uint8, device="cuda")
    ops._enqueue("ssd_linear_attn_backward", x["q"].device, ctypes.byref(ops.SsdLinearAttnDims(n, rows, H, Hk, dk, dv)),
                 1 if dtype == torch.bfloat16 else 0, x["log_decay"].data_ptr(), dk ** -0.5, offsets.data_ptr(),
                 x["q"].data_ptr(), x["k"].data_ptr(), x["v"].data_ptr(), None, x["do"].data_ptr(), None,
                 got["q"].data_ptr(), got["k"].data_ptr(), got["v"].data_ptr(), None, ws.data_ptr(), ws.numel())
    ops.device_status()
    for name in "qkv":
        assert torch.equal(got[name][cu[0]:cu[-1]], want[name][cu[0]:cu[-1]]), name
        assert (got[name][:cu[0]] == 7).all() and (got[name][cu[-1]:] == 7).all(), name


@pytest.mark.parametrize("B,L,H,dk,dv", [(1, 8191, 16, 128, 128), (1, 6000, 20, 64, 64), (3, 2500, 8, 128, 64)])
def test_segments_give_the_same_bits_over_many_runs(B, L, H, dk, dv):
    """The warps of the states' pass run up to two chunks apart: none may be taken for another's."""
    assert workspace_bytes(L, H, H, dk, dv, torch.bfloat16, B=B) > 0
    x = make(L, (B, L), H, H, dk, dv, torch.bfloat16, grads=True)
    args = (x["q"], x["k"], x["v"], x["log_decay"])
    o, S = ops.linear_attn_prefill(*args)
    g = ops.linear_attn_backward(*args, x["do"])
    ops.device_status()
    for _ in range(100):
        o2, S2 = ops.linear_attn_prefill(*args)
        g2 = ops.linear_attn_backward(*args, x["do"])
        assert torch.equal(o, o2) and torch.equal(S, S2) and all(torch.equal(g[n], g2[n]) for n in g)
    ops.device_status()


@pytest.mark.parametrize("L,H,dk,dv", [(1, 1, 64, 128), (1, 2, 32, 64), (4, 1, 128, 64), (90, 2, 96, 40), (128, 1, 128, 128)])
@pytest.mark.parametrize("packed", [False, True])
def test_a_lone_chunk_with_a_state_rounds_its_outputs_only(L, H, dk, dv, packed):
    """The same for the state that such a sequence starts from, its outputs and its gradients; more items than SMs and
    longer sequences between them."""
    n = 90
    x = make(L + dv, (n, L), H, H, dk, dv, torch.bfloat16, init=True, grads=True)
    cu = list(range(0, n * L + 1, L)) if packed else None
    if packed:
        for name in ("q", "k", "v", "do"):
            x[name] = x[name].flatten(0, 1)
    args = (x["q"], x["k"], x["v"], x["log_decay"])
    o, S = (ops.linear_attn_prefill_varlen(*args, cu, x["init"]) if packed else ops.linear_attn_prefill(*args, x["init"]))
    g = ops.linear_attn_backward(*args, x["do"], x["init"], x["d_final"], cu_seqlens=cu)
    ops.device_status()
    wo, wS, mo, mS = lo.prefill(*args, dk ** -0.5, x["init"], cu)
    want, mag = lo.backward(*args, dk ** -0.5, x["do"], x["init"], x["d_final"], cu)
    check_state(S, wS, mS, L, dk, "final_state")
    for got, w, m in [(o, wo, mo)] + [(g[name], want[name], mag[name]) for name in "qkv"]:
        # two parts each of scores and of the state are off by 2^-16 of themselves
        assert (np.abs(np64(got) - w) <= U * np.abs(w) * 1.001 + (2.0 ** -15 + n_terms(L, max(dk, dv)) * E) * m).all()


def test_lone_chunks_between_longer_sequences():
    """Sequences of one chunk, of more and of none in one CTA's hands, one behind the other."""
    lens = [1, 300, 0, 5, 128, 129, 2, 700, 64] * 12
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    x = make(21, (cu[-1],), 4, 2, 64, 64, torch.bfloat16, nseq=len(lens), init=True, grads=True)
    args = (x["q"], x["k"], x["v"], x["log_decay"])
    o, S = ops.linear_attn_prefill_varlen(*args, cu, x["init"])
    g = ops.linear_attn_backward(*args, x["do"], x["init"], x["d_final"], cu_seqlens=cu)
    ops.device_status()
    wo, wS, mo, mS = lo.prefill(*args, 0.125, x["init"], cu)
    check_out(o, wo, mo, torch.bfloat16, 700, 64, "o")
    check_state(S, wS, mS, 700, 64, "final_state")
    want, mag = lo.backward(*args, 0.125, x["do"], x["init"], x["d_final"], cu)
    for name in "qkv":
        check_out(g[name], want[name], mag[name], torch.bfloat16, 700, 64, "d" + name)
    check_state(g["init_state"], want["init_state"], mag["init_state"], 700, 64, "d_init_state")
