"""Timed cases of the linear-attention layer's operators: the per-head norm and rotation of queries and keys
(forward and backward), decayed linear attention over prompts (forward and backward) and its single-token step.

With ``own`` false ``run`` computes the plain form in elementary torch operations, in 32 bits, rounded once at
the end; with ``own`` true it makes the calls of ``selective_state_space_43_b200.ops``.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
PLAIN_CHUNK = 128


# ---- cases ------------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step's queries and keys of 256 sequences: latency
        dict(name="norm_rope decode", op="norm_rope", tokens=256, heads=64, kv_heads=8, dim=128, rot=128,
             interleaved=False, dtype="bf16"),
        # a whole prompt batch of a 64-head layer, 4 x 8192 tokens, partial rotation
        dict(name="norm_rope prompt", op="norm_rope", tokens=32768, heads=64, kv_heads=64, dim=64, rot=32,
             interleaved=True, dtype="bf16"),
        # training, one 4096-token sequence of a 128-head layer
        dict(name="norm_rope backward", op="norm_rope_bwd", tokens=4096, heads=128, kv_heads=128, dim=128, rot=64,
             interleaved=False, dtype="bf16"),
        # a small fp32 model with an odd head width and few heads
        dict(name="norm_rope backward fp32", op="norm_rope_bwd", tokens=1237, heads=10, kv_heads=2, dim=80, rot=40,
             interleaved=True, dtype="fp32"),
        # the prompt batch of a 64-head layer, chunked prefill (starts from a state)
        dict(name="prefill batch", op="prefill", batch=4, length=8192, heads=64, kv_heads=64, dk=128, dv=64,
             init=True, packed=False, dtype="bf16"),
        # one long prompt on few heads: the sequence axis is all the parallelism there is
        dict(name="prefill one prompt", op="prefill", batch=1, length=8191, heads=16, kv_heads=16, dk=128, dv=128,
             init=False, packed=False, dtype="bf16"),
        # continuous batching: packed ragged prompts, keys and values shared by groups of heads
        dict(name="prefill packed", op="prefill", batch=24, length=16384, heads=40, kv_heads=8, dk=64, dv=64,
             init=True, packed=True, dtype="bf16"),
        # the small fp32 layer
        dict(name="prefill fp32", op="prefill", batch=1, length=256, heads=4, kv_heads=4, dk=32, dv=64,
             init=False, packed=False, dtype="fp32"),
        # one token for each of 256 running sequences of a 128-head layer
        dict(name="decode batch", op="decode", batch=256, heads=128, kv_heads=128, dk=128, dv=64, dtype="bf16"),
        # one token of a single conversation: latency
        dict(name="decode single", op="decode", batch=1, heads=64, kv_heads=64, dk=128, dv=128, dtype="bf16"),
        # training, one 4096-token sequence of a 128-head layer
        dict(name="backward", op="backward", batch=1, length=4096, heads=128, kv_heads=128, dk=128, dv=64,
             init=False, packed=False, dtype="bf16"),
        # training on short packed sequences, shared keys and values, gradients of the initial states too
        dict(name="backward packed", op="backward", batch=7, length=3001, heads=16, kv_heads=4, dk=64, dv=128,
             init=True, packed=True, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))) - 0.5))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "prefill", "prefill", "decode", "backward"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    kv = rng.choice([1, 2, 4, 5, 8, 16])
    heads = kv * rng.choice([1, 1, 2, 4])
    if op.startswith("norm_rope"):
        dim = rng.choice([32, 64, 80, 96, 128, 256])
        rot = rng.choice([dim, dim // 2, 16])
        most = (1 << 27) // ((heads + kv) * dim)
        return dict(op=op, tokens=_spread(rng, 1, min(40000, most)), heads=heads, kv_heads=kv, dim=dim, rot=rot,
                    interleaved=rng.random() < 0.5, dtype=dtype)
    dk, dv = (rng.choice([64, 64, 128, 128, 32, 96]) for _ in range(2))
    if op == "decode":
        most = (1 << 28) // (heads * dk * dv)
        return dict(op=op, batch=_spread(rng, 1, min(512, most)), heads=heads, kv_heads=kv, dk=dk, dv=dv, dtype=dtype)
    most = (1 << 30 if dtype == "bf16" else 1 << 28) // (heads * dk * dv)  # fp32 has no tensor cores to run on
    tokens = _spread(rng, 1, max(16, min(32768, 8 * most)))
    packed = rng.random() < 0.5
    batch = _spread(rng, 1, 16)
    return dict(op=op, batch=batch, length=tokens if packed else max(1, tokens // batch), heads=heads, kv_heads=kv,
                dk=dk, dv=dv, init=rng.random() < 0.5, packed=packed, dtype=dtype)


def _lengths(case):
    """Lengths of a packed batch's sequences: ragged, one of them empty, one of a single token."""
    rng = random.Random(1000003 * case["length"] + case["batch"])
    n, total = case["batch"], case["length"]
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    if n >= 4:
        big = max(range(n), key=lambda i: lens[i])
        for i, want in ((0 if big != 0 else 1, 0), (2 if big != 2 else 3, 1)):
            lens[big] += lens[i] - want
            lens[i] = want
    return lens


# ---- inputs -----------------------------------------------------------------------------------------------

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    dt = _dtype(case)

    def normal(*shape, dtype=dt):
        return torch.randn(shape, generator=g, device=DEV, dtype=dtype)

    s = dict(case=case)
    op, H, Hk = case["op"], case["heads"], case["kv_heads"]
    if op.startswith("norm_rope"):
        T, D = case["tokens"], case["dim"]
        # queries, keys and values as one projection writes them; the operator reads its part in place
        qkv = normal(T, (H + 2 * Hk) * D)
        s["q"] = qkv[:, :H * D].unflatten(1, (H, D))
        s["k"] = qkv[:, H * D:(H + Hk) * D].unflatten(1, (Hk, D))
        s["q_weight"] = 1 + 0.1 * normal(D, dtype=torch.float32)
        s["k_weight"] = 1 + 0.1 * normal(D, dtype=torch.float32)
        start = torch.randint(0, 1 << 17, (1,), generator=g, device=DEV)
        s["positions"] = (start + torch.arange(T, device=DEV)).to(torch.int64)
        half = case["rot"] // 2
        s["inv_freq"] = (10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)).float()
        if op == "norm_rope_bwd":
            s["dq_out"], s["dk_out"] = normal(T, H, D), normal(T, Hk, D)
        return s

    B, dk, dv = case["batch"], case["dk"], case["dv"]
    # decays spread evenly in the logarithm of their reach, 1 to 1024 tokens
    s["log_decay"] = -torch.exp(torch.rand(H, generator=g, device=DEV) * -math.log(1024.0))
    lead = (B,) if op == "decode" else (case["length"],) if case["packed"] else (B, case["length"])
    s["q"], s["k"], s["v"] = normal(*lead, H, dk), normal(*lead, Hk, dk), normal(*lead, Hk, dv)
    if op == "decode":
        s["state"] = normal(B, H, dk, dv, dtype=torch.float32)
        return s
    s["init_state"] = normal(B, H, dk, dv, dtype=torch.float32) if case["init"] else None
    s["cu_seqlens"] = None
    if case["packed"]:
        ends = torch.tensor([0] + _lengths(case), dtype=torch.int64).cumsum(0)
        s["cu_seqlens"] = ends.to(DEV)
    if op == "backward":
        s["do"] = normal(*lead, H, dv)
        s["d_final_state"] = normal(B, H, dk, dv, dtype=torch.float32) if case["init"] else None
    return s


# ---- one pass -----------------------------------------------------------------------------------------------

def run(state):
    return (_own if own else _plain)(state)


def _own(s):
    from selective_state_space_43_b200 import ops
    c = s["case"]
    op = c["op"]
    if op == "norm_rope":
        return ops.qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], s["inv_freq"], eps=EPS,
                                interleaved=c["interleaved"])
    if op == "norm_rope_bwd":
        return ops.qk_norm_rope_backward(s["dq_out"], s["dk_out"], s["q"], s["k"], s["q_weight"], s["k_weight"],
                                         s["positions"], s["inv_freq"], eps=EPS, interleaved=c["interleaved"])
    if op == "decode":
        return ops.linear_attn_decode_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"]), s["state"]
    if op == "prefill":
        if c["packed"]:
            return ops.linear_attn_prefill_varlen(s["q"], s["k"], s["v"], s["log_decay"], s["cu_seqlens"],
                                                  init_state=s["init_state"])
        return ops.linear_attn_prefill(s["q"], s["k"], s["v"], s["log_decay"], init_state=s["init_state"])
    return ops.linear_attn_backward(s["q"], s["k"], s["v"], s["log_decay"], s["do"], init_state=s["init_state"],
                                    d_final_state=s["d_final_state"], cu_seqlens=s["cu_seqlens"],
                                    want_init_grads=c["init"])


def _plain(s):
    c = s["case"]
    op, dt = c["op"], _dtype(c)
    if op == "norm_rope":
        cos, sin = _angles(s)
        return tuple(_norm_rope(s[x].float(), s[x + "_weight"], cos, sin, c["interleaved"]).to(dt) for x in "qk")
    if op == "norm_rope_bwd":
        cos, sin = _angles(s)
        (dq, dwq), (dk, dwk) = (_norm_rope_bwd(s["d%s_out" % x].float(), s[x].float(), s[x + "_weight"], cos, sin,
                                               c["interleaved"]) for x in "qk")
        return dict(q=dq.to(dt), k=dk.to(dt), q_weight=dwq, k_weight=dwk)
    scale, group = c["dk"] ** -0.5, c["heads"] // c["kv_heads"]
    if op == "decode":
        q, k, v = (s[x].float() for x in "qkv")
        k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
        st = s["state"]
        st.mul_(torch.exp(s["log_decay"])[None, :, None, None]).add_(k[..., :, None] * v[..., None, :])
        return (scale * (q[..., :, None] * st).sum(-2)).to(dt), st
    q, k, v = (_batch(s, s[x]) for x in "qkv")  # [B, H, L, D]
    k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
    ld, S0 = s["log_decay"].double(), s["init_state"]
    lens = _lens(s, q.shape[2])
    if op == "prefill":
        o = _decayed(q, k, v, ld, 1, scale, None if S0 is None else scale * S0)
        return _unbatch(s, o).to(dt), _state_after(k, v, ld, lens, 0, S0)
    do, dS = _batch(s, s["do"]), s["d_final_state"]
    dq = _decayed(do, v, k, ld, 1, scale, None if S0 is None else scale * S0.transpose(-1, -2))
    # the keys' and values' gradients run against the time: rows reversed within each sequence
    rq, rk, rv, rdo = (_reverse(x, lens) for x in (q, k, v, do))
    dk = _reverse(_decayed(rv, rdo, rq, ld, 0, scale, None if dS is None else dS.transpose(-1, -2)), lens)
    dv = _reverse(_decayed(rk, rq, rdo, ld, 0, scale, dS), lens)
    dk, dv = (x.unflatten(1, (-1, group)).sum(2) for x in (dk, dv))
    grads = dict(q=_unbatch(s, dq).to(dt), k=_unbatch(s, dk).to(dt), v=_unbatch(s, dv).to(dt))
    if c["init"]:
        grads["init_state"] = _state_after(scale * rq, rdo, ld, lens, 1, dS)
    return grads


# ---- plain forms ------------------------------------------------------------------------------------------

def _angles(s):
    # in 64 bits: a far position times a frequency has no digits left in 32
    a = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    return a.cos().float(), a.sin().float()


def _pairs(x, rot, interleaved):
    r = x[..., :rot]
    return (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])


def _join(a, b, rest, interleaved):
    r = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((r, rest), -1)


def _norm_rope(x, w, cos, sin, interleaved):
    n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    rot = 2 * cos.shape[-1]
    a, b = _pairs(n, rot, interleaved)
    return _join(a * cos - b * sin, b * cos + a * sin, n[..., rot:], interleaved)


def _norm_rope_bwd(dy, x, w, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    a, b = _pairs(dy, rot, interleaved)
    dn = _join(a * cos + b * sin, b * cos - a * sin, dy[..., rot:], interleaved)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xh, dh = x * r, dn * w
    return r * (dh - xh * (dh * xh).mean(-1, keepdim=True)), (dn * xh).sum((0, 1))


def _lens(s, length):
    cu = s["cu_seqlens"]
    return torch.full((s["case"]["batch"],), length, device=DEV) if cu is None else cu[1:] - cu[:-1]


def _batch(s, x):
    """[B, L, H, D] or packed [T, H, D] rows as fp32 [B, H, L, D], zeros behind each sequence's end."""
    if s["cu_seqlens"] is not None:
        n = max(1, max(_lengths(s["case"])))
        at = torch.arange(n, device=DEV)
        cu = s["cu_seqlens"]
        rows = cu[:-1, None] + at
        x = x[rows.clamp(max=x.shape[0] - 1)] * (rows < cu[1:, None])[..., None, None]
    return x.float().transpose(1, 2)


def _unbatch(s, x):
    x = x.transpose(1, 2)
    if s["cu_seqlens"] is None:
        return x
    lens = _lens(s, 0)
    return x[torch.arange(x.shape[1], device=DEV) < lens[:, None]]


def _reverse(x, lens):
    """The rows of [B, H, L, D] in reverse order within each sequence's length (rows behind it stay zero)."""
    at = torch.arange(x.shape[2], device=DEV)
    src = lens[:, None] - 1 - at
    return x.gather(2, src.clamp(min=0)[:, None, :, None].expand_as(x)) * (src >= 0)[:, None, :, None]


def _decayed(q, k, v, ld, shift, scale, S0):
    """o_i = scale sum_{j<=i} e^{ld (i-j)} (q_i . k_j) v_j + e^{ld (i+shift)} q_i S0, over chunks."""
    B, H, L, _ = q.shape
    C = PLAIN_CHUNK
    nc = -(-L // C)
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, nc * C - L)).unflatten(2, (nc, C)) for x in (q, k, v))
    at = torch.arange(C, device=DEV, dtype=torch.float64)
    far = at[:, None] - at
    mask = torch.where(far >= 0, torch.exp(ld[:, None, None] * far.clamp(min=0)), 0.0).float()
    o = (q @ k.transpose(-1, -2) * (scale * mask)[None, :, None]) @ v
    end = torch.exp(ld[:, None] * (C - 1 - at)).float()  # a row's weight in the state behind its chunk
    chunk = (k * end[None, :, None, :, None]).transpose(-1, -2) @ v
    c = torch.arange(nc, device=DEV, dtype=torch.float64)
    apart = c[:, None] - 1 - c  # chunks between the end of one and the start of another
    carry = torch.where(apart >= 0, torch.exp(ld[:, None, None] * C * apart.clamp(min=0)), 0.0).float()
    before = (carry[None] @ chunk.flatten(3)).unflatten(3, chunk.shape[3:])
    inside = torch.exp(ld[:, None] * (at + 1)).float()
    o = o + scale * inside[None, :, None, :, None] * (q @ before)
    if S0 is not None:
        t = torch.arange(nc * C, device=DEV, dtype=torch.float64).unflatten(0, (nc, C))
        o = o + torch.exp(ld[:, None, None] * (t + shift)).float()[None, ..., None] * (q @ S0[:, :, None])
    return o.flatten(2, 3)[:, :, :L]


def _state_after(k, v, ld, lens, shift, S0):
    """sum_t e^{ld (len-1-t+shift)} k_t v_t^T + e^{ld len} S0."""
    t = lens[:, None] - 1 - torch.arange(k.shape[2], device=DEV)
    w = torch.where(t[:, None] >= 0, torch.exp(ld[:, None] * (t[:, None].clamp(min=0) + shift)), 0.0).float()
    S = (k * w[..., None]).transpose(-1, -2) @ v
    if S0 is not None:
        S = S + torch.exp(ld * lens[:, None]).float()[..., None, None] * S0
    return S


# ---- from the definition, in 64 bits ----------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("norm_rope"):
        return _exact_norm_rope(s, op == "norm_rope_bwd")
    scale, group = case["dk"] ** -0.5, case["heads"] // case["kv_heads"]
    q, k, v = (s[x].double() for x in "qkv")
    decay = s["log_decay"].double()
    if op == "decode":
        S = s["state"].double() * decay.exp()[:, None, None]
        S += torch.einsum("bhk,bhv->bhkv", k.repeat_interleave(group, 1), v.repeat_interleave(group, 1))
        return torch.einsum("bhk,bhkv->bhv", q, S) * scale, S
    grads = op == "backward"
    S0 = s["init_state"]
    S0 = torch.zeros(case["batch"], case["heads"], case["dk"], case["dv"], device=DEV) if S0 is None else S0
    leaves = [x.double().requires_grad_(grads) for x in (q, k, v, S0)]
    q, k, v, S0 = leaves
    if case["packed"]:
        cu = s["cu_seqlens"].tolist()
        got = [_recurrence(q[a:b], k[a:b], v[a:b], decay, S0[i], scale, group)
               for i, (a, b) in enumerate(zip(cu, cu[1:]))]
        o, S = torch.cat([x[0] for x in got]), torch.stack([x[1] for x in got])
    else:
        got = [_recurrence(q[i], k[i], v[i], decay, S0[i], scale, group) for i in range(case["batch"])]
        o, S = torch.stack([x[0] for x in got]), torch.stack([x[1] for x in got])
    if not grads:
        return o, S
    loss = (o * s["do"].double()).sum()
    if s["d_final_state"] is not None:
        loss = loss + (S * s["d_final_state"].double()).sum()
    dq, dk, dv, dS0 = torch.autograd.grad(loss, leaves)
    out = dict(q=dq, k=dk, v=dv)
    if case["init"]:
        out["init_state"] = dS0
    return out


def _recurrence(q, k, v, decay, S, scale, group):
    """One sequence [L, H, D] from the state S [H, Dk, Dv]: a few tokens at a time, the state carried on."""
    k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
    outs = []
    step = 96
    for a in range(0, q.shape[0], step):
        qc, kc, vc = q[a:a + step], k[a:a + step], v[a:a + step]
        n = qc.shape[0]
        i = torch.arange(n, device=DEV, dtype=torch.float64)
        D = torch.exp(decay[:, None, None] * (i[:, None] - i).clamp(min=0)).tril()
        A = torch.einsum("ihk,jhk->hij", qc, kc) * D
        o = torch.einsum("hij,jhv->ihv", A, vc)
        o = o + torch.einsum("ihk,hkv,hi->ihv", qc, S, torch.exp(decay[:, None] * (i + 1)))
        outs.append(o * scale)
        S = torch.exp(decay * n)[:, None, None] * S
        S = S + torch.einsum("jhk,jhv,hj->hkv", kc, vc, torch.exp(decay[:, None] * (n - 1 - i)))
    return (torch.cat(outs) if outs else q.new_zeros(0, q.shape[1], v.shape[-1])), S


def _exact_norm_rope(s, grads):
    c = s["case"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       s["positions"].double()[:, None] * s["inv_freq"].double())[:, None]
    rot = c["rot"]

    def forward(x, w):
        n = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w
        head, rest = n[..., :rot], n[..., rot:]
        z = head.unflatten(-1, (-1, 2)) if c["interleaved"] else head.unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
        return torch.cat((z.flatten(-2) if c["interleaved"] else z.transpose(-1, -2).flatten(-2), rest), -1)

    out = []
    for n in "qk":
        x, w = (t.double().detach().requires_grad_(grads) for t in (s[n], s[n + "_weight"]))
        y = forward(x, w)
        out.append(torch.autograd.grad(y, (x, w), s["d%s_out" % n].double()) if grads else y)
    if not grads:
        return tuple(out)
    return dict(q=out[0][0], k=out[1][0], q_weight=out[0][1], k_weight=out[1][1])


# ---- what a pass cannot do without --------------------------------------------------------------------------

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    H, Hk = case["heads"], case["kv_heads"]
    if case["op"].startswith("norm_rope"):
        T, D = case["tokens"], case["dim"]
        x = T * (H + Hk) * D
        if case["op"] == "norm_rope":
            return dict(bytes=2 * x * e + 8 * T + 8 * D, flops=8 * x)
        return dict(bytes=3 * x * e + 8 * T + 16 * D, flops=16 * x)
    B, dk, dv = case["batch"], case["dk"], case["dv"]
    st = B * H * dk * dv * 4
    if case["op"] == "decode":
        return dict(bytes=2 * st + B * (H * (dk + dv) + Hk * (dk + dv)) * e, flops=5 * B * H * dk * dv)
    T = case["length"] if case["packed"] else B * case["length"]
    rows = T * (H * (dk + dv) + Hk * (dk + dv)) * e
    if case["op"] == "prefill":  # the recurrence: an outer product into the state and a read of it for each token
        return dict(bytes=rows + st * (2 if case["init"] else 1), flops=4 * T * H * dk * dv)
    # q, k, v, do read, dq, dk, dv written; two states and three reads of them for each token
    grads = T * (H * dk + Hk * (dk + dv)) * e
    return dict(bytes=rows + grads + (3 * st if case["init"] else 0), flops=10 * T * H * dk * dv)
