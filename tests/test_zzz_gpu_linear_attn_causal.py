"""Linear attention on the GPU: a non-finite value reaches only what the recurrence makes of it.

o_t = scale q_t S_t depends on q_t and on k, v of rows up to t; in the gradient dq_t on d(o)_t and on k, v up to t,
dk_t and dv_t on q, d(o) from t on and on v_t or k_t.  So a NaN or an infinity in one row leaves every output that does
not depend on it as it was, bit for bit, and makes all that do NaN or infinite.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

from selective_state_space_43_b200 import ops  # noqa: E402
from test_zzz_gpu_linear_attn import DTYPES, make, workspace_bytes  # noqa: E402

NAN, INF = float("nan"), float("inf")


def clean_and_dirty(x, name, where, value, call):
    y = {k: None if v is None else v.clone() for k, v in x.items()}
    y[name][where] = value
    out = call(x), call(y)
    ops.device_status()
    return out


def check(got, clean, touched, what):
    """`touched`: True where the output depends on the planted value."""
    same = got == clean
    assert same[~touched].all(), f"{what}: {(~same[~touched]).sum().item()} values that do not depend on it changed"
    assert not torch.isfinite(got[touched]).any(), f"{what}: a value that depends on it is finite"


def prefill(x, cu=None):
    a = (x["q"], x["k"], x["v"], x["log_decay"])
    out = ops.linear_attn_prefill(*a, x["init"]) if cu is None else ops.linear_attn_prefill_varlen(*a, cu, x["init"])
    return dict(zip(("o", "S"), out))


def backward(x, cu=None):
    return ops.linear_attn_backward(x["q"], x["k"], x["v"], x["log_decay"], x["do"], x["init"], x["d_final"],
                                    cu_seqlens=cu)


def touched(t, *wheres):
    m = torch.zeros_like(t, dtype=torch.bool)
    for w in wheres:
        m[w] = True
    return m


ALL = slice(None)
# sequence length, planted row: inside, at the start and at the end of a chunk of 128 or of 32 rows, in short last chunks
ROWS = [(100, 0), (100, 37), (100, 99), (128, 127), (200, 65), (200, 150), (200, 199), (300, 255), (300, 256)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 72), (40, 128)])
@pytest.mark.parametrize("L,row", ROWS)
def test_prefill_rows(L, row, dk, dv, dtype):
    H, Hk = 4, 2
    x = make(L + row, (2, L), H, Hk, dk, dv, dtype, init=True)
    ch = (7 * row + 3) % dv
    for value in (NAN, INF, -INF):
        for name, where, hit in (
                ("q", (1, row, 2), dict(o=(1, row, 2), S=None)),
                ("k", (1, row, 1, 5), dict(o=(1, slice(row, None), slice(2, 4)), S=(1, slice(2, 4), 5))),
                ("v", (1, row, 0, ch), dict(o=(1, slice(row, None), slice(0, 2), ch), S=(1, slice(0, 2), ALL, ch))),
                ("init", (1, 3, 2, ch), dict(o=(1, ALL, 3, ch), S=(1, 3, 2, ch)))):
            a, b = clean_and_dirty(x, name, where, value, prefill)
            for n in a:
                check(b[n], a[n], touched(a[n], *([] if hit[n] is None else [hit[n]])), f"{n} of {name}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 72), (40, 128)])
@pytest.mark.parametrize("L,row", ROWS)
def test_gradient_rows(L, row, dk, dv, dtype):
    H = 3
    x = make(L + row, (2, L), H, H, dk, dv, dtype, init=True, grads=True)
    cv, ck = (5 * row + 1) % dv, (3 * row + 2) % dk
    up, back = slice(row, None), slice(0, row + 1)
    for value in (NAN, -INF):
        for name, where, hit in (
                # the channel of k is a key row of the state: dq of that channel, dv of the row
                ("k", (1, row, 1, ck), dict(q=[(1, up, 1, ck)], k=[], v=[(1, row, 1)], init_state=[])),
                ("v", (1, row, 1, cv), dict(q=[(1, up, 1)], k=[(1, row, 1)], v=[], init_state=[])),
                ("q", (1, row, 1, ck), dict(q=[], k=[(1, back, 1, ck)], v=[(1, back, 1)], init_state=[(1, 1, ck)])),
                ("do", (1, row, 1, cv), dict(q=[(1, row, 1)], k=[(1, back, 1)], v=[(1, back, 1, cv)],
                                             init_state=[(1, 1, ALL, cv)]))):
            a, b = clean_and_dirty(x, name, where, value, backward)
            for n in a:
                check(b[n], a[n], touched(a[n], *hit[n]), f"gradient of {n}, planted in {name}")


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_of_a_cut_packed_batch(dtype):
    """The same in segments: one long sequence among short ones, the planted rows in each."""
    lens = [3, 3000, 1, 0, 90]
    cu = [5]
    for n in lens:
        cu.append(cu[-1] + n)
    H, T, dk, dv = 2, cu[-1] + 20, 64, 64
    assert workspace_bytes(T, H, H, dk, dv, dtype, True, len(lens)) > 0
    assert workspace_bytes(T, H, H, dk, dv, dtype, True, len(lens), True) > 0
    offsets = torch.tensor(cu).cuda()
    x = make(11, (T,), H, H, dk, dv, dtype, nseq=len(lens), init=True, grads=True)
    x["log_decay"][0] = -1e-3
    inside = slice(cu[0], cu[-1])
    for seq, row in ((0, 1), (1, 700), (1, 1300), (1, 2999), (2, 0), (4, 40)):
        r, a0, a1 = cu[seq] + row, cu[seq], cu[seq + 1]
        for name, hit_f, hit_b in (
                ("v", dict(o=[(slice(r, a1), 1, 9)], S=[(seq, 1, ALL, 9)]),
                 dict(q=[(slice(r, a1), 1)], k=[(r, 1)], v=[], init_state=[])),
                ("k", dict(o=[(slice(r, a1), 1)], S=[(seq, 1, 9)]),
                 dict(q=[(slice(r, a1), 1, 9)], k=[], v=[(r, 1)], init_state=[])),
                ("do", None, dict(q=[(r, 1)], k=[(slice(a0, r + 1), 1)], v=[(slice(a0, r + 1), 1, 9)],
                                  init_state=[(seq, 1, ALL, 9)]))):
            for call, hit in ((prefill, hit_f), (backward, hit_b)):
                if hit is None:
                    continue
                a, b = clean_and_dirty(x, name, (r, 1, 9), NAN, lambda y: call(y, offsets))
                for n in a:
                    t = touched(a[n], *hit[n])
                    if n in ("S", "init_state"):
                        check(b[n], a[n], t, f"{n}, planted in {name} of sequence {seq}")
                    else:
                        check(b[n][inside], a[n][inside], t[inside], f"{n}, planted in {name} of sequence {seq}")
    ops.device_status()


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_behind_a_padded_prompt(dtype):
    """Right-padded batches: whatever stands behind a prompt's last row, in the same chunk too, changes nothing."""
    x = make(4, (2, 400), 2, 2, 64, 64, dtype)
    o, _ = ops.linear_attn_prefill(x["q"], x["k"], x["v"], x["log_decay"])
    for end in (1, 30, 127, 129, 200, 399):
        for value in (NAN, INF, 3e38):
            y = {k: None if v is None else v.clone() for k, v in x.items()}
            for name in ("q", "k", "v"):
                y[name][:, end:] = value
            o2, _ = ops.linear_attn_prefill(y["q"], y["k"], y["v"], y["log_decay"])
            assert torch.equal(o[:, :end], o2[:, :end]), (end, value)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("share", [0.02, 0.5, 1.0])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 96)])
def test_many_sequences_some_of_them_padded(dk, dv, share, dtype):
    """More sequences than SMs, in place: from a row on, some hold NaN in q, k, v (a batch padded with whatever was there)."""
    g = torch.Generator().manual_seed(5)
    H, Hk, n = 4, 2, 260
    lens = [(0, 1, 5, 100, 128, 129, 300)[int(i)] for i in torch.randint(0, 7, (n,), generator=g)]
    cu = [0]
    for m in lens:
        cu.append(cu[-1] + m)
    offsets = torch.tensor(cu).cuda()
    x = make(17, (cu[-1],), H, Hk, dk, dv, dtype, nseq=n, init=True, grads=True)
    y = {k: v.clone() for k, v in x.items()}
    padded = torch.zeros(n, dtype=torch.bool, device="cuda")
    front = torch.ones(cu[-1], dtype=torch.bool, device="cuda")
    for i, m in enumerate(lens):
        if m and float(torch.rand((), generator=g)) < share:
            row = int(torch.randint(0, m, (), generator=g))
            padded[i] = True
            front[cu[i] + row:cu[i + 1]] = False
            for name in ("q", "k", "v"):
                y[name][cu[i] + row:cu[i + 1]] = NAN
    S = [z["init"].clone() for z in (x, y)]
    o = [ops.linear_attn_prefill_varlen(z["q"], z["k"], z["v"], z["log_decay"], offsets, s, final_state=s)[0]
         for z, s in zip((x, y), S)]
    a, b = backward(x, offsets), backward(y, offsets)
    ops.device_status()
    assert torch.equal(o[0][front], o[1][front]) and not torch.isfinite(o[1][~front]).any()
    assert torch.equal(S[0][~padded], S[1][~padded]) and not torch.isfinite(S[1][padded]).any()
    assert torch.equal(a["q"][front], b["q"][front])
    whole = torch.ones(cu[-1], dtype=torch.bool, device="cuda")  # rows of the sequences that hold no NaN
    for i, m in enumerate(lens):
        whole[cu[i]:cu[i + 1]] = not bool(padded[i])
    for name in "kv":
        assert torch.equal(a[name][whole], b[name][whole]), name
    assert torch.equal(a["init_state"][~padded], b["init_state"][~padded])


@pytest.mark.parametrize("dtype", DTYPES)
def test_scores_that_overflow_do_not_reach_earlier_rows(dtype):
    """Keys so large that their scores are infinite although they are not, with values of zero."""
    x = make(6, (2, 200), 2, 2, 64, 64, dtype)
    o, _ = ops.linear_attn_prefill(x["q"], x["k"], x["v"], x["log_decay"])
    y = {k: None if v is None else v.clone() for k, v in x.items()}
    y["k"][:, 70:] = 3e38
    y["v"][:, 70:] = 0
    o2, _ = ops.linear_attn_prefill(y["q"], y["k"], y["v"], y["log_decay"])
    ops.device_status()
    assert torch.equal(o[:, :70], o2[:, :70])
