"""Measured cases of the gated delta rule (recurrent, chunkwise, backward)
and of the fused residual norm (forward, backward).

`run` computes a case either in its plain form (elementary torch operations,
32-bit floats inside, rounded once at the end) or, with `own` set, through
the library's entry points.  `exact` computes the same outputs from the
definitions in 64 bits, token by token.

Per (sequence, value head), with row vectors q_t, k_t (dk), v_t (dv), a log
decay g_t <= 0, a write strength b_t and a float32 state S [dk, dv]:
    S <- exp(g_t) S;  x_t = b_t (v_t - k_t S);  S <- S + k_t^T x_t;  o_t = scale q_t S
q and k have key_heads heads, each shared by heads / key_heads value heads.
Tokens at or behind a sequence's length are not part of it: their rows of
the output stay as they were and their gradients are zero.

Residual norm on rows of `hidden` channels, rms(x) = x / sqrt(mean(x^2) + eps):
    h = x + residual_scale * swish(gate) * (rms(y) * post);  n = rms(h) * pre
"""
import math

import torch

own = False

CHUNK = 64
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def _delta(op, name, batch, heads, key_heads, tokens, dk, dv, dtype, ragged=False, state_in=False,
           state_out=False):
    return {"name": name, "op": op, "batch": batch, "heads": heads, "key_heads": key_heads,
            "tokens": tokens, "dk": dk, "dv": dv, "dtype": dtype, "ragged": ragged,
            "state_in": state_in, "state_out": state_out}


def _norm(op, name, rows, hidden, dtype, gate=True, post=True):
    return {"name": name, "op": op, "rows": rows, "hidden": hidden, "dtype": dtype, "gate": gate,
            "post": post}


def listed():
    return [
        # one user's next token: 16 heads, the smallest call, latency counts
        _delta("recurrent", "step_one", 1, 16, 16, 1, 128, 128, "bf16"),
        # a full decode batch at the library's 16 heads of 256: the state is the traffic
        _delta("recurrent", "step_batch128", 128, 16, 16, 1, 256, 256, "bf16"),
        # a long prompt that hands its state to decoding
        _delta("chunkwise", "prefill_long", 1, 16, 8, 8192, 128, 128, "bf16", state_out=True),
        # forward of a training step: no state leaves, values wider than keys
        _delta("chunkwise", "train_forward", 4, 16, 16, 2048, 128, 256, "bf16"),
        # a padded batch of prompts of uneven length continued from their states
        _delta("chunkwise", "prefill_ragged", 5, 12, 4, 777, 64, 128, "bf16", ragged=True,
               state_in=True, state_out=True),
        # float32, as a check of a model's numerics is run
        _delta("chunkwise", "prefill_f32", 2, 4, 4, 1000, 128, 64, "f32", state_out=True),
        # backward of a training step
        _delta("backward", "train_backward", 2, 16, 16, 4096, 128, 128, "bf16"),
        # backward of a padded batch with shared keys in float32
        _delta("backward", "backward_ragged_f32", 3, 6, 2, 333, 64, 128, "f32", ragged=True),
        # between two blocks of a training step or a prefill of 16384 tokens
        _norm("norm", "norm_train", 16384, 4096, "bf16"),
        # between two blocks of a decode step, without a gate
        _norm("norm", "norm_step", 8, 2048, "bf16", gate=False),
        # backward of the first
        _norm("norm_backward", "norm_backward_train", 8192, 4096, "bf16"),
        # an odd float32 shape, no norm behind the block
        _norm("norm_backward", "norm_backward_f32", 1111, 1032, "f32", post=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["recurrent", "chunkwise", "chunkwise", "backward", "backward", "norm",
                     "norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("norm", "norm_backward"):
        hidden = 8 * _log(rng, 8, 1024)
        case = _norm(op, "", _log(rng, 1, max(1, (1 << 25) // hidden)), hidden, dtype,
                     rng.random() < 0.7, rng.random() < 0.7)
    else:
        key_heads = _log(rng, 1, 16)
        heads = key_heads * rng.choice([1, 1, 2, 3])
        ragged, fresh, last = rng.random() < 0.3, rng.random() < 0.5, rng.random() < 0.5
        if op == "recurrent":
            dk, dv = rng.choice([64, 128, 256]), rng.choice([64, 128, 256])
            tokens = _log(rng, 1, 16)
            batch = _log(rng, 1, max(1, min(128, (1 << 26) // (heads * dk * dv * tokens))))
            case = _delta(op, "", batch, heads, key_heads, tokens, dk, dv, dtype, ragged)
        else:
            dk, dv = rng.choice([64, 128]), rng.choice([64, 128, 256])
            room = (1 << 17) if dtype == "bf16" else (1 << 13)
            tokens = _log(rng, 1, min(8192, room // heads))
            batch = _log(rng, 1, max(1, min(16, room * 128 // (heads * tokens * max(dv, 128)))))
            case = _delta(op, "", batch, heads, key_heads, tokens, dk, dv, dtype, ragged,
                          op == "chunkwise" and not fresh, op == "chunkwise" and last)
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs
def _generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def prepare(case, seed):
    gen = _generator(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if case["op"] in ("norm", "norm_backward"):
        rows, hidden = case["rows"], case["hidden"]
        s = {"op": case["op"], "x": (2.0 * normal(rows, hidden)).to(dt),
             "y": (0.5 * normal(rows, hidden)).to(dt),
             "gate": normal(rows, hidden).to(dt) if case["gate"] else None,
             "post": 1.0 + 0.2 * normal(hidden) if case["post"] else None,
             "pre": 1.0 + 0.2 * normal(hidden), "scale": 0.5}
        if case["op"] == "norm_backward":
            s["dh"], s["dn"] = normal(rows, hidden).to(dt), normal(rows, hidden).to(dt)
        return s

    B, H, Hk, n = case["batch"], case["heads"], case["key_heads"], case["tokens"]
    dk, dv = case["dk"], case["dv"]

    def unit(x):                       # activated and brought to length one, as a layer does
        x = torch.nn.functional.silu(x)
        return (x / (x.norm(dim=-1, keepdim=True) + 1e-6)).to(dt)

    # decay rates spread over heads from long memories to short ones
    rate = torch.exp(torch.rand(H, generator=gen, device="cuda") * math.log(200.0) - 6.2)
    s = {"op": case["op"], "q": unit(normal(B, n, Hk, dk)), "k": unit(normal(B, n, Hk, dk)),
         "v": normal(B, n, H, dv).to(dt), "g": (-rate * torch.exp(0.7 * normal(B, n, H))).to(dt),
         "beta": torch.sigmoid(normal(B, n, H)).to(dt), "scale": dk ** -0.5, "lengths": None,
         "state": None}
    if case["ragged"]:
        lengths = torch.randint(0, n + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        lengths[-1] = n
        s["lengths"] = lengths
    if case["op"] == "recurrent" or case["state_in"]:
        s["state"] = 0.3 * normal(B, H, dk, dv)
    if case["op"] == "backward":
        s["d_out"] = normal(B, n, H, dv).to(dt)
    else:
        s["out"] = torch.zeros(B, n, H, dv, device="cuda", dtype=dt)
    s["state_out"] = torch.empty(B, H, dk, dv, device="cuda") if case["state_out"] else None
    if own:
        import linear_recurrent_sequence_02_b200 as rn
        if case["op"] == "chunkwise":
            need = rn.retnet_delta_workspace_size(B, H, Hk, n, dk, dv, dt)
            s["workspace"] = rn.retnet_workspace(need, "cuda")
        elif case["op"] == "backward":
            need = rn.retnet_delta_backward_workspace_size(B, H, Hk, n, dk, dv, dt)
            s["workspace"] = rn.retnet_workspace(need, "cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import linear_recurrent_sequence_02_b200 as rn
    op = s["op"]
    if op == "norm":
        h, n = rn.retnet_residual_norm(s["x"], s["y"], gate=s["gate"], post_norm=s["post"] is not None,
                                       post_weight=s["post"], pre_weight=s["pre"],
                                       residual_scale=s["scale"], eps=EPS)
        return {"h": h, "n": n}
    if op == "norm_backward":
        g = rn.retnet_residual_norm_backward(s["x"], s["y"], s["dn"], s["dh"], gate=s["gate"],
                                             post_norm=s["post"] is not None,
                                             post_weight=s["post"], pre_weight=s["pre"],
                                             residual_scale=s["scale"], eps=EPS)
        return {"dx": g.dx, "dy": g.dy, "dgate": g.dgate, "dpost": g.dpost_weight,
                "dpre": g.dpre_weight}
    qkvgb = (s["q"], s["k"], s["v"], s["g"], s["beta"])
    if op == "recurrent":
        rn.retnet_delta_recurrent(*qkvgb, s["state"], scale=s["scale"], lengths=s["lengths"],
                                  out=s["out"])
        return {"out": s["out"], "state": s["state"]}
    if op == "chunkwise":
        rn.retnet_delta_chunkwise(*qkvgb, scale=s["scale"], lengths=s["lengths"],
                                  state_in=s["state"], state_out=s["state_out"], out=s["out"],
                                  workspace=s["workspace"])
        return {"out": s["out"], "state": s["state_out"]}
    dq, dk, dv, dg, dbeta = rn.retnet_delta_backward(*qkvgb, s["d_out"], scale=s["scale"],
                                                     lengths=s["lengths"],
                                                     workspace=s["workspace"])
    return {"dq": dq, "dk": dk, "dv": dv, "dg": dg, "dbeta": dbeta}


# ------------------------------------------------------------------ plain form
def _run_plain(s):
    op = s["op"]
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_backward":
        return _plain_norm_backward(s)
    if op == "recurrent":
        return _plain_recurrent(s)
    return _plain_chunkwise(s) if op == "chunkwise" else _plain_backward(s)


def _rms(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _plain_norm(s):
    x, y = s["x"].float(), s["y"].float()
    z = y if s["post"] is None else y * _rms(y) * s["post"]
    if s["gate"] is not None:
        gate = s["gate"].float()
        z = z * gate * torch.sigmoid(gate)
    h = x + s["scale"] * z
    n = h * _rms(h) * s["pre"]
    dt = s["x"].dtype
    return {"h": h.to(dt), "n": n.to(dt)}


def _plain_norm_backward(s):
    x, y, dt = s["x"].float(), s["y"].float(), s["x"].dtype
    post, pre = s["post"], s["pre"]
    ry = _rms(y)
    yhat = y * ry
    z = y if post is None else yhat * post
    swish = 1.0
    if s["gate"] is not None:
        gate = s["gate"].float()
        sig = torch.sigmoid(gate)
        swish = gate * sig
    h = x + s["scale"] * z * swish
    rh = _rms(h)
    hhat = h * rh
    dn = s["dn"].float()
    dpre = (dn * hhat).sum(0)
    t = dn * pre
    dx = s["dh"].float() + rh * (t - hhat * (t * hhat).mean(-1, keepdim=True))
    da = s["scale"] * dx
    dgate = None
    if s["gate"] is not None:
        dgate = (da * z * (sig + swish * (1.0 - sig))).to(dt)
    dz = da * swish
    dpost = None
    dy = dz
    if post is not None:
        dpost = (dz * yhat).sum(0)
        t = dz * post
        dy = ry * (t - yhat * (t * yhat).mean(-1, keepdim=True))
    return {"dx": dx.to(dt), "dy": dy.to(dt), "dgate": dgate, "dpost": dpost, "dpre": dpre}


def _live(s):
    """[B, n, 1] truth values of the tokens inside their sequences, or None."""
    if s["lengths"] is None:
        return None
    at = torch.arange(s["v"].shape[1], device="cuda")
    return (at[None, :] < s["lengths"][:, None])[..., None]


def _plain_recurrent(s):
    H, rep = s["v"].shape[2], s["v"].shape[2] // s["q"].shape[2]
    q = (s["q"].float() * s["scale"]).repeat_interleave(rep, 2)
    k = s["k"].float().repeat_interleave(rep, 2)
    v, beta = s["v"].float(), s["beta"].float()[..., None]
    decay = torch.exp(s["g"].float())[..., None, None]
    live = _live(s)
    S, out = s["state"], s["out"]
    for t in range(v.shape[1]):
        new = S * decay[:, t]
        x = beta[:, t] * (v[:, t] - (k[:, t].unsqueeze(-2) @ new).squeeze(-2))
        new = new + k[:, t].unsqueeze(-1) * x.unsqueeze(-2)
        o = (q[:, t].unsqueeze(-2) @ new).squeeze(-2).to(out.dtype)
        if live is None:
            S.copy_(new)
            out[:, t] = o
        else:
            S.copy_(torch.where(live[:, t, :, None, None], new, S))
            out[:, t] = torch.where(live[:, t, :, None], o, out[:, t])
    return {"out": out, "state": S}


def _chunks(s, names):
    """The tensors by chunks, [chunks, B, H, CHUNK, ...] float32, tokens outside a sequence zero."""
    live = _live(s)
    n, H = s["v"].shape[1:3]
    made = []
    for name in names:
        x = s[name].float()
        if live is not None:
            x = torch.where(live if x.dim() == 3 else live[..., None], x, torch.zeros((), device="cuda"))
        if x.shape[2] != H:
            x = x.repeat_interleave(H // x.shape[2], 2)
        pad = -n % CHUNK
        if pad:
            x = torch.cat([x, x.new_zeros(x.shape[0], pad, *x.shape[2:])], 1)
        x = x.reshape(x.shape[0], -1, CHUNK, *x.shape[2:])
        made.append(x.transpose(2, 3).transpose(0, 1).contiguous())
    return made


def _unchunk(x, s):
    """[chunks, B, H, CHUNK, ...] back to [B, tokens, H, ...]."""
    x = x.transpose(0, 1).transpose(2, 3)
    return x.reshape(x.shape[0], -1, *x.shape[3:])[:, :s["v"].shape[1]]


def _within(s):
    """What each chunk's equations need that does not depend on the state."""
    q, k, v, g, beta = _chunks(s, ("q", "k", "v", "g", "beta"))
    total = torch.cumsum(g.double(), -1)
    low = torch.ones(CHUNK, CHUNK, device="cuda").tril()
    between = torch.exp((total[..., :, None] - total[..., None, :]).clamp(max=0).float()) * low
    e, rest = torch.exp(total.float()), torch.exp((total[..., -1:] - total).float())
    kk = (k @ k.transpose(-1, -2)) * between * (1.0 - torch.eye(CHUNK, device="cuda"))
    M = kk * beta[..., None]
    P = (q @ k.transpose(-1, -2)) * between * s["scale"]
    T = torch.eye(CHUNK, device="cuda").expand_as(M).contiguous()
    for i in range(1, CHUNK):          # (1 + M) T = 1, row by row
        T[..., i:i + 1, :i] = -(M[..., i:i + 1, :i] @ T[..., :i, :i])
    return q, k, v, beta, between, e, rest, kk, M, P, T


def _plain_chunkwise(s):
    q, k, v, beta, _, e, rest, _, _, P, T = _within(s)
    T = T * beta[..., None, :]
    U, W = T @ v, (T * e[..., None, :]) @ k
    qe, ke = q * (s["scale"] * e)[..., None], (k * rest[..., None]).transpose(-1, -2)
    S = torch.zeros(*v.shape[1:3], k.shape[-1], v.shape[-1], device="cuda") \
        if s["state"] is None else s["state"]
    o = torch.empty_like(v)
    for c in range(v.shape[0]):
        X = U[c] - W[c] @ S
        o[c] = qe[c] @ S + P[c] @ X
        S = S * e[c, ..., -1, None, None] + ke[c] @ X
    o, live, out = _unchunk(o, s).to(s["out"].dtype), _live(s), s["out"]
    out.copy_(o if live is None else torch.where(live[..., None], o, out))
    if s["state_out"] is not None:
        s["state_out"].copy_(S)
    return {"out": out, "state": s["state_out"]}


def _plain_backward(s):
    q, k, v, beta, between, e, rest, kk, M, P, T = _within(s)
    (do,) = _chunks(s, ("d_out",))
    n, scale = v.shape[0], s["scale"]
    Tb = T * beta[..., None, :]
    U, W = Tb @ v, (Tb * e[..., None, :]) @ k
    qe, ke = q * (scale * e)[..., None], k * rest[..., None]
    X, S = torch.empty_like(v), v.new_zeros(n + 1, *v.shape[1:3], k.shape[-1], v.shape[-1])
    for c in range(n):
        X[c] = U[c] - W[c] @ S[c]
        S[c + 1] = S[c] * e[c, ..., -1, None, None] + ke[c].transpose(-1, -2) @ X[c]
    D, dX = torch.zeros_like(S), P.transpose(-1, -2) @ do
    inner = qe.transpose(-1, -2) @ do
    for c in range(n - 1, -1, -1):     # D[c]: gradient of the state behind chunk c - 1
        dX[c] += ke[c] @ D[c + 1]
        D[c] = D[c + 1] * e[c, ..., -1, None, None] + inner[c] - W[c].transpose(-1, -2) @ dX[c]
    S, D = S[:-1], D[1:]
    dR = T.transpose(-1, -2) @ dX
    low = torch.ones(CHUNK, CHUNK, device="cuda").tril()
    Xt = X.transpose(-1, -2)
    dP = (do @ Xt) * between * scale
    dM = -(dR @ Xt) * between * (low - torch.eye(CHUNK, device="cuda"))
    St, Dt = S.transpose(-1, -2), D.transpose(-1, -2)
    dq_state = (do @ St) * (scale * e)[..., None]
    dk_state = -(dR @ St) * (beta * e)[..., None]
    dk_next = (X @ Dt) * rest[..., None]
    dMb = dM * beta[..., None]
    dq = dq_state + dP @ k
    dk = dk_state + dk_next + dP.transpose(-1, -2) @ q + (dMb + dMb.transpose(-1, -2)) @ k
    seen = v - (k @ S) * e[..., None] - kk @ X             # v_t - k_t S_t: x_t without b_t
    dbeta = (dR * seen).sum(-1)
    # g_t acts on all that crosses from before token t to it or behind it
    pair = dP * (q @ k.transpose(-1, -2)) + dMb * (k @ k.transpose(-1, -2))
    row = pair.sum(-1) - pair.sum(-2) + (q * dq_state).sum(-1) + (k * dk_state).sum(-1)
    ahead = (k * dk_next).sum(-1)
    dg = torch.cumsum(row.flip(-1), -1).flip(-1) + torch.cumsum(ahead, -1) - ahead \
        + e[..., -1:] * (S * D).sum((-1, -2))[..., None]
    Hk, dt = s["q"].shape[2], s["q"].dtype

    def shared(x):                     # key heads gather the gradients of their value heads
        x = _unchunk(x, s)
        return x.reshape(*x.shape[:2], Hk, -1, x.shape[-1]).sum(3).to(dt)

    live = _live(s)
    grads = {"dq": shared(dq), "dk": shared(dk), "dv": _unchunk(dR * beta[..., None], s).to(dt),
             "dg": _unchunk(dg, s).to(dt), "dbeta": _unchunk(dbeta, s).to(dt)}
    if live is not None:
        for name, x in grads.items():
            x.masked_fill_(~(live if x.dim() == 3 else live[..., None]), 0)
    return grads


# ------------------------------------------------------------------ counts
def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        elements = case["rows"] * case["hidden"]
        return {"bytes": elements * size * (4 + case["gate"]), "flops": 12 * elements}
    if case["op"] == "norm_backward":
        elements = case["rows"] * case["hidden"]
        return {"bytes": elements * size * (6 + 2 * case["gate"]), "flops": 30 * elements}
    B, H, Hk, n = case["batch"], case["heads"], case["key_heads"], case["tokens"]
    dk, dv = case["dk"], case["dv"]
    if case["ragged"]:                 # lengths are uniform in 0..n, the last one is n
        n = n * (B + 1) / (2 * B)
    row_bytes = B * n * (2 * Hk * dk + 2 * H * dv + 2 * H) * size
    state = 4 * B * H * dk * dv
    product = 2.0 * B * H * n * dk * dv          # one vector-matrix product a token and head
    if case["op"] == "recurrent":
        return {"bytes": row_bytes + 2 * state, "flops": 3 * product}
    if case["op"] == "chunkwise":
        return {"bytes": row_bytes + state * (case["state_in"] + case["state_out"]),
                "flops": 3 * product}
    return {"bytes": row_bytes + B * n * (2 * Hk * dk + H * dv + 2 * H) * size,
            "flops": 8 * product}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm_backward"):
        return _exact_norm(s, case)
    f = torch.float64
    B, n, H, dv = s["v"].shape
    dk, rep = s["q"].shape[-1], H // s["q"].shape[2]
    share = torch.arange(H, device="cuda") // rep
    live = torch.ones(B, n, dtype=torch.bool, device="cuda")
    if s["lengths"] is not None:
        live = torch.arange(n, device="cuda")[None] < s["lengths"][:, None]
    # a token outside its sequence neither decays nor writes
    alpha = torch.where(live[..., None], s["g"].to(f).exp(), torch.ones((), dtype=f, device="cuda"))
    beta = torch.where(live[..., None], s["beta"].to(f), torch.zeros((), dtype=f, device="cuda"))
    q, k, v = s["q"].to(f)[:, :, share] * s["scale"], s["k"].to(f)[:, :, share], s["v"].to(f)
    S = torch.zeros(B, H, dk, dv, dtype=f, device="cuda") if s["state"] is None else s["state"].to(f)

    def step(S, t):
        S = alpha[:, t, :, None, None] * S
        miss = v[:, t] - torch.einsum("bhk,bhkv->bhv", k[:, t], S)
        x = beta[:, t, :, None] * miss
        return S + k[:, t, :, :, None] * x[:, :, None, :], miss, x

    if case["op"] != "backward":
        out = torch.zeros(B, n, H, dv, dtype=f, device="cuda")
        for t in range(n):
            S, _, _ = step(S, t)
            out[:, t] = torch.einsum("bhk,bhkv->bhv", q[:, t], S)
        out = torch.where(live[..., None, None], out, torch.zeros((), dtype=f, device="cuda"))
        whole = case["op"] == "recurrent" or case["state_out"]
        return {"out": out, "state": S if whole else None}

    do = torch.where(live[..., None, None], s["d_out"].to(f), torch.zeros((), dtype=f, device="cuda"))
    span = 64                          # states are kept every `span` tokens and made again between
    kept = []
    for t in range(n):
        if t % span == 0:
            kept.append(S)
        S, _, _ = step(S, t)
    dq, dk_ = torch.zeros_like(q), torch.zeros_like(k)
    dv_, dg, db = torch.zeros_like(v), torch.zeros_like(alpha), torch.zeros_like(alpha)
    D = torch.zeros_like(S)
    for c in range(len(kept) - 1, -1, -1):
        states, misses, S = [], [], kept[c]
        for t in range(c * span, min(n, (c + 1) * span)):
            states.append(S)
            S, miss, x = step(S, t)
            misses.append((miss, x, S))
        for i in range(len(states) - 1, -1, -1):
            t, old = c * span + i, states[i]
            miss, x, new = misses[i]
            dq[:, t] = torch.einsum("bhkv,bhv->bhk", new, do[:, t])
            D = D + q[:, t, :, :, None] * do[:, t, :, None, :]
            dx = torch.einsum("bhk,bhkv->bhv", k[:, t], D)
            dmiss = beta[:, t, :, None] * dx
            faded = alpha[:, t, :, None, None] * old
            db[:, t] = (dx * miss).sum(-1)
            dv_[:, t] = dmiss
            dk_[:, t] = torch.einsum("bhkv,bhv->bhk", D, x) - torch.einsum("bhkv,bhv->bhk", faded, dmiss)
            D = D - k[:, t, :, :, None] * dmiss[:, :, None, :]
            dg[:, t] = (D * faded).sum((-1, -2))
            D = alpha[:, t, :, None, None] * D
    Hk = s["q"].shape[2]
    dq = (dq * s["scale"]).reshape(B, n, Hk, rep, dk).sum(3)
    dk_ = dk_.reshape(B, n, Hk, rep, dk).sum(3)
    zero = torch.zeros((), dtype=f, device="cuda")
    return {"dq": torch.where(live[..., None, None], dq, zero),
            "dk": torch.where(live[..., None, None], dk_, zero),
            "dv": torch.where(live[..., None, None], dv_, zero),
            "dg": torch.where(live[..., None], dg, zero),
            "dbeta": torch.where(live[..., None], db, zero)}


def _exact_norm(s, case):
    """The forward from the definition; the gradients are autograd's of it."""
    f = torch.float64

    def leaf(x):
        return None if x is None else x.to(f).requires_grad_(case["op"] == "norm_backward")

    x, y, gate, post, pre = (leaf(s[name]) for name in ("x", "y", "gate", "post", "pre"))
    z = y
    if post is not None:
        z = post * y / torch.sqrt(y.pow(2).mean(-1, keepdim=True) + EPS)
    if gate is not None:
        z = z * (gate / (1.0 + torch.exp(-gate)))
    h = x + s["scale"] * z
    n = pre * h / torch.sqrt(h.pow(2).mean(-1, keepdim=True) + EPS)
    if case["op"] == "norm":
        return {"h": h, "n": n}
    torch.autograd.backward([h, n], [s["dh"].to(f), s["dn"].to(f)])

    def grad(t):
        return None if t is None else t.grad

    return {"dx": x.grad, "dy": y.grad, "dgate": grad(gate), "dpost": grad(post), "dpre": pre.grad}
