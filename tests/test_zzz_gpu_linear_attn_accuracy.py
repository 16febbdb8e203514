"""Linear attention on the GPU: how near its results are, where the token-by-token comparison alone would let more through.

u = 2^-8 is half a bf16 step, relative; e = 2^-24 half an fp32 one.  Rounding a normal variable to bf16 is off by a value
even in +-u 2^k where 2^k <= |x| < 2^(k+1): u / sqrt(3) sqrt(sum_k 4^k P_k) = 0.425 u of its norm.  A bf16 output is rounded
once (0.425 u), and where its terms (a score, or an element of the state) are rounded once before, terms of random
signs, by sqrt(2) 0.425 u = 0.60 u of the result's norm.
"""
import numpy as np
import pytest
import torch

import linear_attn_oracle as lo

pytestmark = pytest.mark.gpu

from selective_state_space_43_b200 import ops  # noqa: E402
from test_zzz_gpu_linear_attn import DTYPES, E, U, make, n_terms, np64, workspace_bytes  # noqa: E402


def starts(lens, first=0):
    cu = [first]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def check_state(got, want, mag, length, dk, what):
    """Sums of fp32 roundings, every value finite."""
    err, tol = np.abs(np64(got) - want), n_terms(length, dk) * E * mag + 1e-30
    assert (err <= tol).all(), f"{what}: {(~(err <= tol)).sum()} of {err.size} off"


def check_lone_chunk(got, want, mag, length, dk, what):
    """Scores and the state that the outputs start from in two bf16 parts each, 2^-16 of themselves off: the outputs' own
    rounding is all that shows."""
    err = np.abs(np64(got) - want)
    tol = U * np.abs(want) * 1.001 + (2.0 ** -15 + n_terms(length, dk) * E) * mag
    assert (err <= tol).all(), f"{what}: {(~(err <= tol)).sum()} of {err.size} off, worst {np.max(err / (tol + 1e-30)):.2f}"


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (96, 128), (40, 40)])
def test_lone_chunks_of_a_cut_batch_round_their_outputs_only(dk, dv):
    """Short sequences of a packed batch that is cut into segments: as exact as in a batch that is not."""
    lens = [1, 4000, 2, 0, 4, 128, 1, 90, 3]
    cu, H = starts(lens), 1
    assert workspace_bytes(cu[-1], H, H, dk, dv, torch.bfloat16, True, len(lens)) > 0
    assert workspace_bytes(cu[-1], H, H, dk, dv, torch.bfloat16, True, len(lens), True) > 0
    x = make(dk + dv, (cu[-1],), H, H, dk, dv, torch.bfloat16, nseq=len(lens), init=True, grads=True)
    args = (x["q"], x["k"], x["v"], x["log_decay"])
    o, S = ops.linear_attn_prefill_varlen(*args, cu, x["init"])
    g = ops.linear_attn_backward(*args, x["do"], x["init"], x["d_final"], cu_seqlens=cu)
    ops.device_status()
    wo, wS, mo, mS = lo.prefill(*args, dk ** -0.5, x["init"], cu)
    want, mag = lo.backward(*args, dk ** -0.5, x["do"], x["init"], x["d_final"], cu)
    check_state(S, wS, mS, 4000, dk, "final_state")
    check_state(g["init_state"], want["init_state"], mag["init_state"], 4000, max(dk, dv), "d_init_state")
    for i, n in enumerate(lens):
        if n > 128:
            continue
        at = slice(cu[i], cu[i + 1])
        check_lone_chunk(o[at], wo[at], mo[at], n, dk, f"o of sequence {i}")
        for name in "qkv":
            check_lone_chunk(g[name][at], want[name][at], mag[name][at], n, max(dk, dv), f"d{name} of sequence {i}")


@pytest.mark.parametrize("L", [2049, 2100])
def test_a_segment_of_one_chunk_rounds_its_outputs_only(L):
    """A long sequence whose last segment (of 256, 512, 1024 or 2048 rows) is one chunk, from row 2048 on: it starts from a
    joined state."""
    H, dk, dv = 8, 64, 64
    assert workspace_bytes(L, H, H, dk, dv, torch.bfloat16) > 0
    x = make(L, (1, L), H, H, dk, dv, torch.bfloat16, init=True)
    x["log_decay"][:] = -1e-3
    args = (x["q"], x["k"], x["v"], x["log_decay"])
    o, S = ops.linear_attn_prefill(*args, x["init"])
    wo, wS, mo, mS = lo.prefill(*args, dk ** -0.5, x["init"])
    check_state(S, wS, mS, L, dk, "final_state")
    err = np64(o)[:, 2048:] - wo[:, 2048:]
    # one rounding is 0.425 u, two are 0.60 u; 512 values or more leave the former within a tenth (three deviations)
    assert np.linalg.norm(err) <= 0.5 * U * np.linalg.norm(wo[:, 2048:])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cu", [[0, 0, 1, 1, 130, 386, 386], [3, 3, 131, 260, 300], [5, 261, 2821, 2821, 3077, 4001]])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 40)])
def test_states_among_rows_of_nan_are_finite(cu, dk, dv, dtype):
    """States and gradients of states in packed batches whose buffers hold NaN outside every sequence; a workspace and
    outputs that held NaN before."""
    T, n, H, Hk = cu[-1] + 37, len(cu) - 1, 2, 1
    x = make(sum(cu) + dk, (T,), H, Hk, dk, dv, dtype, nseq=n, init=True, grads=True)
    clean = {k: v.clone() for k, v in x.items()}
    for name in ("q", "k", "v", "do"):
        x[name][cu[-1]:] = float("nan")
        x[name][:cu[0]] = float("inf")
    nan = float("nan")
    need = max(workspace_bytes(T, H, Hk, dk, dv, dtype, True, n, b) for b in (False, True))
    ws = torch.full((need // 4 + 4,), nan, device="cuda")
    o = torch.full((T, H, dv), nan, device="cuda").to(dtype)
    S = torch.full((n, H, dk, dv), nan, device="cuda")
    ops.linear_attn_prefill_varlen(x["q"], x["k"], x["v"], x["log_decay"], cu, x["init"], workspace=ws, o=o, final_state=S)
    ws.fill_(nan)
    g = ops.linear_attn_backward(x["q"], x["k"], x["v"], x["log_decay"], x["do"], x["init"], x["d_final"], cu_seqlens=cu,
                                 workspace=ws)
    ops.device_status()
    longest = max(b - a for a, b in zip(cu, cu[1:]))
    args = [clean[k] for k in ("q", "k", "v", "log_decay")] + [dk ** -0.5]
    _, wS, _, mS = lo.prefill(*args, x["init"], cu)
    want, mag = lo.backward(*args, clean["do"], x["init"], x["d_final"], cu)
    check_state(S, wS, mS, longest, dk, "final_state")
    check_state(g["init_state"], want["init_state"], mag["init_state"], longest, max(dk, dv), "d_init_state")
    assert torch.isfinite(o[cu[0]:cu[-1]]).all() and all(torch.isfinite(g[name][cu[0]:cu[-1]]).all() for name in "qkv")


@pytest.mark.parametrize("dtype", DTYPES)
def test_states_of_the_step_are_finite(dtype):
    x = make(31, (33,), 4, 2, 40, 96, dtype, init=True)
    state = x["init"].clone()
    ops.linear_attn_decode_step(x["q"], x["k"], x["v"], x["log_decay"], state)
    _, wS, _, mS = lo.prefill(x["q"][:, None], x["k"][:, None], x["v"][:, None], x["log_decay"], 40 ** -0.5, x["init"])
    check_state(state, wS, mS, 1, 40, "state")


@pytest.mark.parametrize("L,Hk,group,dk,dv", [(300, 3, 1, 128, 128), (1025, 2, 2, 64, 64), (2500, 2, 1, 64, 128)])
def test_bf16_results_are_off_by_two_roundings(L, Hk, group, dk, dv):
    x = make(L + 1, (1, L), Hk * group, Hk, dk, dv, torch.bfloat16, init=True, grads=True)
    args = (x["q"], x["k"], x["v"], x["log_decay"])
    o, _ = ops.linear_attn_prefill(*args, x["init"])
    g = ops.linear_attn_backward(*args, x["do"], x["init"], x["d_final"])
    wo, _, _, _ = lo.prefill(*args, dk ** -0.5, x["init"])
    want, _ = lo.backward(*args, dk ** -0.5, x["do"], x["init"], x["d_final"])
    for name, a, w in [("o", o, wo)] + [(n, g[n], want[n]) for n in "qkv"]:
        rel = np.linalg.norm(np64(a) - w) / np.linalg.norm(w)
        # 0.60 u, and a quarter over for terms that are not normal
        assert rel <= 0.75 * U, (name, rel)


@pytest.mark.parametrize("dtype", DTYPES)
def test_captured_steps_give_what_eager_ones_give(dtype):
    """Prefill, two tokens and gradients in a graph, each run with states of its own; every output is compared."""
    H, dk, dv = 4, 128, 64
    x = make(2, (1, 700), H, 2, dk, dv, dtype, init=True, grads=True)
    toks = [make(3 + i, (1,), H, 2, dk, dv, dtype) for i in range(2)]
    names = ("q", "k", "v", "do", "init", "d_final")

    def step(state):
        o, S = ops.linear_attn_prefill(x["q"], x["k"], x["v"], x["log_decay"], x["init"])
        state.copy_(S)
        outs = [ops.linear_attn_decode_step(t["q"], t["k"], t["v"], x["log_decay"], state) for t in toks]
        g = ops.linear_attn_backward(x["q"], x["k"], x["v"], x["log_decay"], x["do"], x["init"], x["d_final"])
        return [o, S, state] + outs + [g["q"], g["k"], g["v"], g["init_state"]]

    states = [torch.empty_like(x["init"]) for _ in range(3)]
    step(states[2])
    torch.cuda.synchronize()
    graphs = []
    for s in states[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(s)
        graphs.append((g, out))
    fresh = make(77, (1, 700), H, 2, dk, dv, dtype, init=True, grads=True)
    for name in names:
        x[name].copy_(fresh[name])
    for t, seed in zip(toks, (78, 79)):
        for name, v in make(seed, (1,), H, 2, dk, dv, dtype).items():
            if name in ("q", "k", "v"):
                t[name].copy_(v)
    for s in states:
        s.fill_(float("nan"))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for g, _ in graphs:
            g.replay()
    eager = step(states[2])
    torch.cuda.synchronize()
    ops.device_status()
    for _, out in graphs:
        for i, (a, b) in enumerate(zip(out, eager)):
            assert torch.isfinite(b).all() and torch.equal(a, b), i
    S = np64(eager[1])
    for i, t in enumerate(toks):
        w, S, m, mS = lo.prefill(t["q"][:, None], t["k"][:, None], t["v"][:, None], x["log_decay"], dk ** -0.5,
                                 torch.from_numpy(S))
        tol = n_terms(2, dk) * E * m[:, 0] + (U * np.abs(w[:, 0]) if dtype == torch.bfloat16 else 0)
        assert (np.abs(np64(eager[3 + i]) - w[:, 0]) <= tol).all()
    check_state(eager[2], S, mS + np.abs(S), 2, dk, "state")
