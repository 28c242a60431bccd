"""Linear attention with a decay for each head (linattn_*) and the layer norm with the
residual stream's sum in front of it (layernorm_*), as they are measured: for prompts,
for training and for single tokens.

    attention  S_t = exp(g_t) S_{t-1} + k_t v_t^T,  y_t = scale S_t^T q_t, per head; g comes
               with every token or is a constant of the head; consecutive heads may share
               q and k
    norm       h = x + residual in the stream's type, y = (h - mean) rstd weight + bias, per row

With `own` false, run() computes them from elementary torch operations in 32 bits, with
`own` true it calls the library.  exact() computes them in 64 bits, the attention and its
gradients token by token.
"""
import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5
CHUNK = 64


# ---------------------------------------------------------------- cases

def _attn(name, mode, B, T, H, Dk, Dv, shared=1, per_token=True, dtype="bf16", ragged=False, state=False):
    """shared: how many consecutive heads have q and k in common."""
    return {"name": name, "op": "attn", "mode": mode, "B": B, "T": T, "H": H, "Dk": Dk, "Dv": Dv, "shared": shared,
            "per_token": per_token, "dtype": dtype, "ragged": ragged, "state": state}


def _norm(name, mode, B, T, C, dtype="bf16", stream="bf16", residual=True, ragged=False):
    return {"name": name, "op": "norm", "mode": mode, "B": B, "T": T, "C": C, "dtype": dtype, "stream": stream,
            "residual": residual, "ragged": ragged}


def listed():
    return [
        # One user's prompt of 2048 tokens, 32 heads of 128.
        _attn("attn_prompt", "prompt", 1, 2048, 32, 128, 128),
        # A prefill batch with constant decays, the sizes of the repository's prefill workload.
        _attn("attn_prompt_batch", "prompt", 4, 4096, 40, 64, 64, per_token=False),
        # A padded batch of prompts of odd lengths (one empty) going on from earlier states; odd head sizes, shared keys.
        _attn("attn_prompt_ragged_f32", "prompt", 5, 1237, 12, 48, 80, shared=3, dtype="f32", ragged=True, state=True),
        # One layer of a training step at the repository's forward workload's sizes.
        _attn("attn_train", "train", 8, 1024, 32, 64, 64),
        # Training on two long sequences whose heads share queries and keys in fours.
        _attn("attn_train_long", "train", 2, 16384, 32, 128, 128, shared=4),
        # The next token of one user: latency.
        _attn("attn_step_one", "step", 1, 1, 32, 64, 64),
        # The next token of a full serving batch, the sizes of the repository's decode workload.
        _attn("attn_step_batch", "step", 256, 1, 64, 64, 64),
        # The norm in front of one user's next token: latency.
        _norm("norm_step_one", "prompt", 1, 1, 2048),
        # The norm over a prefill batch of 8 x 4096 tokens.
        _norm("norm_prompt_batch", "prompt", 8, 4096, 4096),
        # One layer of a training step: outputs and every gradient.
        _norm("norm_train", "train", 8, 1024, 2048),
        # A stream kept in 32 bits between bf16 layers.
        _norm("norm_train_stream_f32", "train", 4, 2048, 4096, stream="f32"),
        # Odd, ragged sequences in 32 bits, the first norm of a model (nothing is added).
        _norm("norm_train_ragged_f32", "train", 3, 1531, 960, dtype="f32", stream="f32", residual=False, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "norm"])
    mode = rng.choice(["prompt", "train", "step"] if op == "attn" else ["prompt", "train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        C = _log(rng, 64, 16384)
        if rng.random() < 0.6:
            C = max(64, C // 64 * 64)
        stream = rng.choice([dtype, "f32"])
        rows = _log(rng, 1, max(1, (8 * 4096 * 4096 if mode == "prompt" else 4 * 2048 * 4096) // C // (2 if stream == "f32" else 1)))
        B = _log(rng, 1, min(rows, 64))
        c = _norm("", mode, B, max(1, rows // B), C, dtype, stream, rng.random() < 0.7, B > 1 and rng.random() < 0.4)
    else:
        Dk, Dv = (rng.choice([64, 64, 128, 128, rng.randint(8, 128)]) for _ in range(2))
        H = rng.choice([1, 4, 12, 16, 24, 32, 32, 40, 64])
        shared = rng.choice([s for s in (1, 1, 2, 4) if H % s == 0])
        most = 16384 * 32 * 128 // (H * max(Dk, Dv)) // (2 if dtype == "f32" else 1)
        T = 1 if mode == "step" else _log(rng, 1, min(16384, most))
        B = _log(rng, 1, 256) if mode == "step" else _log(rng, 1, max(1, min(64, most // T)))
        c = _attn("", mode, B, T, H, Dk, Dv, shared, rng.random() < 0.7, dtype, mode != "step" and B > 1 and rng.random() < 0.4,
                  rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def _lengths(case, gen):
    """Tokens of each sequence: uniform, the longest fills the batch, one is empty."""
    if not case["ragged"]:
        return None
    n = torch.randint(1, case["T"] + 1, (case["B"],), generator=gen, device=DEVICE, dtype=torch.int32)
    n[0] = case["T"]
    if case["B"] > 2:
        n[case["B"] // 2] = 0
    return n


def _slots(B, gen):
    """A pool of more states than rows, the rows' places in it in no order.  In a batch of four
    or more the last eighth are rows without a request; no request has the pool's last state."""
    S = B + max(2, B // 4)
    at = torch.randperm(S - 1, generator=gen, device=DEVICE)[:B].to(torch.int32)
    if B >= 4:
        at[B - B // 8:] = -1
    return S, at


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    f32 = torch.float32
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device=DEVICE) * std + mean).to(dtype)

    B, T, mode = case["B"], case["T"], case["mode"]
    s = {"case": dict(case), "mode": mode, "lengths": None if mode == "step" else _lengths(case, gen)}
    if case["op"] == "norm":
        C, stream = case["C"], DTYPES[case["stream"]]
        plain = not case["residual"]
        s["x"] = normal(B, T, C, std=0.7, mean=0.1, dtype=stream if plain else dt)
        s["residual"] = None if plain else normal(B, T, C, std=1.5, dtype=stream)
        s["weight"], s["bias"] = normal(C, std=0.2, mean=1.0, dtype=f32), normal(C, std=0.2, dtype=f32)
        if mode == "train":
            s["dy"] = normal(B, T, C)
            s["dh"] = normal(B, T, C, dtype=stream)
        return s
    H, Dk, Dv, few = case["H"], case["Dk"], case["Dv"], case["H"] // case["shared"]
    row = (B,) if mode == "step" else (B, T)
    s["q"], s["k"], s["v"] = normal(*row, few, Dk), normal(*row, few, Dk), normal(*row, H, Dv)
    s["scale"] = Dk ** -0.5
    if case["per_token"]:
        # Step sizes softplus(normal - 3) times rates between 1 and 16, the heads from slow to fast.
        rate = torch.exp(torch.linspace(0.0, math.log(16.0), H, device=DEVICE))
        s["g"] = -rate * torch.log1p(torch.exp(normal(*row, H, mean=-3.0, dtype=f32)))
    else:
        # Memories of 32 to 512 tokens over the heads.
        s["g"] = torch.log1p(-torch.exp2(-torch.linspace(5.0, 9.0, H, device=DEVICE)))
    if mode == "step":
        S, s["slots"] = _slots(B, gen)
        s["state"] = normal(S, H, Dk, Dv, dtype=f32)
    else:
        s["state"] = normal(B, H, Dk, Dv, dtype=f32) if case["state"] else None
        if mode == "train":
            s["dy"] = normal(B, T, H, Dv)
            s["dstate"] = normal(B, H, Dk, Dv, dtype=f32) if case["state"] else None
    return s


# ---------------------------------------------------------------- plain forms

def _valid(lengths, T):
    """[B, T] truth values: the token belongs to its sequence."""
    return torch.arange(T, device=lengths.device)[None] < lengths[:, None]


def _chunks(x, H, n, there):
    """[B, T, h, D] -> [B, H, n, CHUNK, D] in 32 bits: padding is 0, a shared head comes once for each of its heads."""
    B, T, h, D = x.shape
    x = x.float()
    if there is not None:
        x = torch.where(there[..., None, None], x, 0.0)
    x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, n * CHUNK - T))
    return x.reshape(B, n, CHUNK, h, D).permute(0, 3, 1, 2, 4).repeat_interleave(H // h, 1)


def _tokens(x, T):
    """[B, H, n, CHUNK, D] -> [B, T, H, D]"""
    B, H, n, L, D = x.shape
    return x.permute(0, 2, 3, 1, 4).reshape(B, n * L, H, D)[:, :T]


def _shared_sum(x, like):
    """Gradients of each head -> of the heads that are there, in their type."""
    B, T, H, D = x.shape
    return x.reshape(B, T, like.shape[2], -1, D).sum(3).to(like.dtype)


def _chain(first, decay, parts, back=False):
    """States between chunks: each chunk's decay times the state before it, plus its part.  Returns the
    state that goes into each chunk and the last one."""
    into, state = torch.empty_like(parts), first
    n = parts.shape[2]
    for c in (reversed(range(n)) if back else range(n)):
        into[:, :, c] = state
        state = decay[:, :, c, None, None] * state + parts[:, :, c]
    return into, state


def _plain_attn(s):
    case, dtype, scale, lengths = s["case"], s["q"].dtype, s["scale"], s["lengths"]
    B, T, H, Dk, Dv = (case[n] for n in ("B", "T", "H", "Dk", "Dv"))
    n = -(-T // CHUNK)
    there = None if lengths is None else _valid(lengths, T)
    q, k, v = (_chunks(s[x], H, n, there) for x in "qkv")
    g = s["g"].expand(B, T, H)[..., None]
    X = _chunks(g, H, n, there)[..., 0].double().cumsum(-1)   # over a chunk: 64 bits, 32 lose the differences of far sums
    order = torch.arange(CHUNK, device=X.device)
    w = torch.where(order[:, None] >= order, X[..., :, None] - X[..., None, :], -math.inf).float().exp()
    into, out_of, all_of = X.float().exp()[..., None], (X[..., -1:] - X).float().exp()[..., None], X[..., -1].float().exp()
    S0 = torch.zeros(B, H, Dk, Dv, device=q.device) if s["state"] is None else s["state"]
    S, last = _chain(S0, all_of, (k * out_of).transpose(-1, -2) @ v)
    y = (w * (q @ k.transpose(-1, -2))) @ v + into * (q @ S)
    out = {"y": (_tokens(y, T) * scale).to(dtype), "state": last}
    if s["mode"] != "train":
        return out
    dy = _chunks(s["dy"], H, n, there) * scale
    E0 = torch.zeros_like(S0) if s["dstate"] is None else s["dstate"]
    E, dfirst = _chain(E0, all_of, (q * into).transpose(-1, -2) @ dy, back=True)
    wd = w * (dy @ v.transpose(-1, -2))
    wq = w * (q @ k.transpose(-1, -2))
    dq = wd @ k + into * (dy @ S.transpose(-1, -2))
    dk = wd.transpose(-1, -2) @ q + out_of * (v @ E.transpose(-1, -2))
    dv = wq.transpose(-1, -2) @ dy + out_of * (k @ E)
    # What each running sum of g changes; the sum over the tokens behind a chunk is that of its last state.
    dX = (q * dq).sum(-1) - (k * dk).sum(-1)
    behind = (E * (all_of[..., None, None] * S + (k * out_of).transpose(-1, -2) @ v)).sum((-1, -2))
    dg = _tokens((dX.flip(-1).cumsum(-1).flip(-1) + behind[..., None])[..., None], T)[..., 0]
    if there is not None:
        dg = torch.where(there[..., None], dg, 0.0)
    out["dq"], out["dk"], out["dv"] = (_shared_sum(_tokens(d, T), s[x]) for d, x in ((dq, "q"), (dk, "k"), (dv, "v")))
    out["dg"] = dg if case["per_token"] else dg.sum((0, 1))
    if s["state"] is not None:
        out["dstate"] = dfirst
    return out


def _plain_attn_step(s):
    H = s["case"]["H"]
    q, k, v = (s[x].float().repeat_interleave(H // s[x].shape[1], 1) for x in "qkv")
    at = s["slots"].long()   # -1, a row without a request, reads the pool's last state and writes it back
    there = (at >= 0)[:, None, None]
    old = s["state"][at]
    new = torch.exp(s["g"].expand(len(at), H))[..., None, None] * old + k[..., None] * v[..., None, :]
    y = (q[..., None] * new).sum(-2) * s["scale"]
    s["state"][at] = torch.where(there[..., None], new, old)
    return {"y": torch.where(there, y, 0.0).to(s["q"].dtype), "state": s["state"]}


def _plain_norm(s):
    x, dtype = s["x"], DTYPES[s["case"]["dtype"]]
    there = None if s["lengths"] is None else _valid(s["lengths"], x.shape[1])[..., None]

    def pad(t):
        return t if there is None else torch.where(there, t, torch.zeros((), dtype=t.dtype, device=t.device))

    h = pad(x if s["residual"] is None else (x.float() + s["residual"].float()).to(s["residual"].dtype))
    off = h.float()
    off = off - off.mean(-1, keepdim=True)
    rstd = torch.rsqrt((off * off).mean(-1, keepdim=True) + EPS)
    xh = off * rstd
    out = {"y": pad((xh * s["weight"] + s["bias"]).to(dtype))}
    if s["residual"] is not None:
        out["h"] = h
    if s["mode"] != "train":
        return out
    dy = pad(s["dy"]).float()
    dxh = dy * s["weight"]
    dh = rstd * (dxh - dxh.mean(-1, keepdim=True) - xh * (dxh * xh).mean(-1, keepdim=True)) + s["dh"].float()
    out["dresidual"] = pad(dh.to(h.dtype))
    if s["residual"] is not None:
        out["dx"] = pad(dh.to(x.dtype))
    out["dweight"], out["dbias"] = (dy * xh).sum((0, 1)), dy.sum((0, 1))
    return out


# ---------------------------------------------------------------- the library's calls

def _own_attn(s):
    from linear_rnn_sequence_wkv7_amd import linattn
    args, kw = (s["q"], s["k"], s["v"], s["g"]), dict(scale=s["scale"])
    if s["mode"] == "step":
        y = linattn.linattn_step(*args, s["state"], state_index=s["slots"], **kw)
        return {"y": y, "state": s["state"]}
    kw.update(state=s["state"], lengths=s["lengths"])
    y, state = linattn.linattn_forward(*args, **kw)
    out = {"y": y, "state": state}
    if s["mode"] == "train":
        grads = linattn.linattn_backward(*args, s["dy"], dstate=s["dstate"], return_dstate=s["state"] is not None, **kw)
        out.update({"d" + n: grads[n] for n in "qkvg"})
        if s["state"] is not None:
            out["dstate"] = grads["state"]
    return out


def _own_norm(s):
    from linear_rnn_sequence_wkv7_amd import layernorm
    kw = dict(weight=s["weight"], bias=s["bias"], lengths=s["lengths"])
    train = s["mode"] == "train"
    y, h, mean, rstd = layernorm.layernorm_forward(s["x"], residual=s["residual"], eps=EPS, y_dtype=s["case"]["dtype"],
                                                   return_stats=train, **kw)
    out = {"y": y}
    if s["residual"] is not None:
        out["h"] = h
    if train:
        grads = layernorm.layernorm_backward(h, s["dy"], mean, rstd, dh=s["dh"], x_dtype=s["case"]["dtype"] if s["residual"] is not None else None, **kw)
        out.update(dresidual=grads["h"], dweight=grads["weight"], dbias=grads["bias"])
        if s["residual"] is not None:
            out["dx"] = grads["x"]
    return out


def run(state):
    if state["case"]["op"] == "norm":
        return _own_norm(state) if own else _plain_norm(state)
    if own:
        return _own_attn(state)
    return _plain_attn_step(state) if state["mode"] == "step" else _plain_attn(state)


# ---------------------------------------------------------------- work

def work(case):
    """Inputs read once, outputs written once; a state is read and written once per sequence, in a
    step only the rows' own.  Operations of the attention per token and head: 4 Dk Dv (the state's
    update and its readout), in training 12 (three gradients, the state's gradient)."""
    B, T, mode = case["B"], case["T"], case["mode"]
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        st = 2 if case["stream"] == "bf16" else 4
        n, C = B * T * case["C"], case["C"]
        res = 1 if case["residual"] else 0
        forward = n * ((e + 2 * st if res else st) + e) + 8 * C
        if mode == "prompt":
            return {"bytes": forward, "flops": n * (8 + res)}
        # the backward's own inputs dy and dh; its gradients, of the branch too where its type is another
        return {"bytes": forward + n * (e + 2 * st + (e if res and e != st else 0)) + 8 * C, "flops": n * 24}
    H, Dk, Dv, few = case["H"], case["Dk"], case["Dv"], case["H"] // case["shared"]
    states = B - B // 8 if mode == "step" and B >= 4 else B
    qk, v, st = 2 * B * T * few * Dk, B * T * H * Dv, 4 * states * H * Dk * Dv
    g = 4 * (B * T * H if case["per_token"] else H)
    read = st if case["state"] or mode == "step" else 0
    per = B * T * H * Dk * Dv
    if mode == "train":
        return {"bytes": e * (2 * qk + 4 * v) + 2 * g + st + (3 * st if case["state"] else 0), "flops": 12 * per}
    return {"bytes": e * (qk + 2 * v) + g + read + st, "flops": 4 * per}


# ---------------------------------------------------------------- 64 bits

def _attn64(s):
    """The recurrences as they are written, one token after another: the state forwards (y, dq), its
    gradient backwards (dk, dv, dg), with the states of a run of tokens computed again from its first."""
    case, RUN = s["case"], 128
    B, T, H, Dk, Dv = (case[n] for n in ("B", "T", "H", "Dk", "Dv"))
    f64 = torch.float64
    heads = {x: torch.arange(H, device=DEVICE) // (H // s[x].shape[2]) for x in "qkv"}
    n = torch.full((B,), T, device=DEVICE) if s["lengths"] is None else s["lengths"]

    def token(x, t):
        """Token t of every head; 0 in padding."""
        y = s[x][:, t].double()
        y = y[:, heads[x]] if x in heads else y
        return torch.where((t < n).reshape(B, 1, 1), y, 0.0)

    def rate(t):
        g = (s["g"][:, t] if case["per_token"] else s["g"]).double().expand(B, H)
        return torch.where((t < n)[:, None], g, 0.0).exp()[..., None, None]

    def after(S, t):
        return rate(t) * S + token("k", t)[..., None] * token("v", t)[..., None, :]

    train = s["mode"] == "train"
    S = torch.zeros(B, H, Dk, Dv, dtype=f64, device=DEVICE) if s["state"] is None else s["state"].double()
    kept, y, dq = [], torch.zeros(B, T, H, Dv, dtype=f64, device=DEVICE), torch.zeros(B, T, H, Dk, dtype=f64, device=DEVICE)
    for t in range(T):
        if train and t % RUN == 0:
            kept.append(S)
        S = after(S, t)
        y[:, t] = (token("q", t)[..., None, :] @ S)[..., 0, :] * s["scale"]
        if train:
            dq[:, t] = (S @ token("dy", t)[..., None])[..., 0] * s["scale"]
    out = {"y": y, "state": S}
    if not train:
        return out
    E = torch.zeros_like(S) if s["dstate"] is None else s["dstate"].double()
    dk, dv, dg = torch.zeros_like(dq), torch.zeros_like(y), torch.zeros(B, T, H, dtype=f64, device=DEVICE)
    for c in reversed(range(len(kept))):
        states = [kept[c]]
        for t in range(c * RUN, min(T, (c + 1) * RUN) - 1):
            states.append(after(states[-1], t))
        for t in reversed(range(c * RUN, c * RUN + len(states))):
            E = E + token("q", t)[..., None] * (token("dy", t) * s["scale"])[..., None, :]
            dk[:, t] = (E @ token("v", t)[..., None])[..., 0]
            dv[:, t] = (token("k", t)[..., None, :] @ E)[..., 0, :]
            a = rate(t)
            dg[:, t] = a[..., 0, 0] * (E * states[t - c * RUN]).sum((-1, -2))
            E = a * E
    keep = (torch.arange(T, device=DEVICE)[None] < n[:, None])[..., None]
    dg = torch.where(keep, dg, 0.0)

    def share(d, x):
        d = torch.where(keep[..., None], d, 0.0)
        return torch.stack([d[:, :, heads[x] == i].sum(2) for i in range(s[x].shape[2])], 2)

    out.update(dq=share(dq, "q"), dk=share(dk, "k"), dv=share(dv, "v"), dg=dg if case["per_token"] else dg.sum((0, 1)))
    if s["state"] is not None:
        out["dstate"] = E
    return out


def _step64(s):
    H, out = s["case"]["H"], torch.zeros(s["v"].shape[0], s["case"]["H"], s["case"]["Dv"], dtype=torch.float64, device=DEVICE)
    pool = s["state"].double()
    rows = torch.nonzero(s["slots"] >= 0)[:, 0]
    at = s["slots"][rows].long()
    per_head = torch.arange(H, device=DEVICE) // s["case"]["shared"]
    g = s["g"].double().expand(len(out), H)[rows]
    S = pool[at] * g.exp().reshape(len(rows), H, 1, 1)
    S = S + s["k"][rows].double()[:, per_head].unsqueeze(3) * s["v"][rows].double().unsqueeze(2)
    out[rows] = (s["q"][rows].double()[:, per_head].unsqueeze(2) @ S).squeeze(2) * s["scale"]
    pool[at] = S
    return {"y": out, "state": pool}


def _norm64(s):
    """Row by row of the tokens that are there, gradients by automatic differentiation."""
    x, residual, train = s["x"], s["residual"], s["mode"] == "train"
    B, T, C = x.shape
    rows = torch.ones(B, T, dtype=torch.bool, device=DEVICE)
    if s["lengths"] is not None:
        rows = torch.arange(T, device=DEVICE).expand(B, T) < s["lengths"].reshape(B, 1)
    stream = x.dtype if residual is None else residual.dtype
    h = x[rows].double() if residual is None else x[rows].double() + residual[rows].double()
    h = h.to(stream).double().requires_grad_(train)   # the stream is held in its type
    weight, bias = (p.double().requires_grad_(train) for p in (s["weight"], s["bias"]))

    def whole(v):
        full = torch.zeros(B, T, C, dtype=torch.float64, device=DEVICE)
        full[rows] = v.detach()
        return full

    with torch.set_grad_enabled(train):
        y = (h - h.mean(1, keepdim=True)) / torch.sqrt(h.var(1, unbiased=False, keepdim=True) + EPS) * weight + bias
    out = {"y": whole(y)}
    if residual is not None:
        out["h"] = whole(h)
    if train:
        ((y * s["dy"][rows].double()).sum() + (h * s["dh"][rows].double()).sum()).backward()
        out["dresidual"] = whole(h.grad)
        if residual is not None:
            out["dx"] = out["dresidual"]
        out["dweight"], out["dbias"] = weight.grad, bias.grad
    return out


def exact(case, seed):
    if case["op"] == "attn" and case["mode"] == "train" and case["B"] * case["T"] * case["H"] * case["Dk"] * case["Dv"] > 2 ** 35:
        return None
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _norm64(s)
    with torch.no_grad():
        return _step64(s) if case["mode"] == "step" else _attn64(s)
