"""The gated delta rule, layer norm and counter-based dropout: what is measured.

Each case is one call as a program makes it: a prompt or a training batch
through the chunked gated delta rule, its gradients, one decoded token, the
norm between two blocks (dropout and residual sum in front of it) in both
directions, and dropout alone.  `own` selects between the plain torch form of
an operator and the library's entry point; both take the same inputs and
return the same outputs.

Gated delta rule (per batch element and head; S [headdim, dstate] fp32):

    S_t = exp(g_t) (S_{t-1} - beta_t (S_{t-1} k_t) k_t^T) + beta_t v_t k_t^T
    y_t = scale S_t q_t

Dropout: element i of a tensor is kept when word i % 4 of Philox4x32-10
(counter i / 4 in words 0 and 1, offset in words 2 and 3, key = seed) is at
least floor(p 2^32), and is then multiplied by 1 / (1 - p).
"""
import math

import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16
DTYPES = {"f32": F32, "bf16": BF16}
DEV = "cuda"
CHUNK = 64
MASK32 = 0xFFFFFFFF
NORM_EPS = 1e-5


# ------------------------------------------------------------------ cases
def _delta(op, batch, seqlen, heads, groups, headdim, dstate, dtype, out, ragged=False, h0=False):
    return {"op": op, "batch": batch, "seqlen": seqlen, "heads": heads, "groups": groups, "headdim": headdim,
            "dstate": dstate, "dtype": dtype, "out": out, "ragged": ragged, "h0": h0}


def _norm(op, rows, dim, dtype, res, out, p):
    return {"op": op, "rows": rows, "dim": dim, "dtype": dtype, "res": res, "out": out, "p": p}


def _drop(n, dtype, p):
    return {"op": "dropout", "n": n, "dtype": dtype, "p": p}


def listed():
    return [
        # one sequence decoding: the latency of a token
        {"name": "step_one", **_delta("delta_step", 1, 1, 32, 1, 64, 128, "bf16", "bf16")},
        # a full serving batch decoding: the state's bandwidth
        {"name": "step_batch", **_delta("delta_step", 128, 1, 16, 16, 128, 128, "bf16", "bf16")},
        # one long prompt: few heads, a long axis
        {"name": "fwd_prompt", **_delta("delta_fwd", 1, 16384, 16, 16, 128, 128, "bf16", "bf16")},
        # a training batch in the Mamba-2 workload's head layout, y in fp32
        {"name": "fwd_train", **_delta("delta_fwd", 8, 4096, 32, 1, 64, 128, "bf16", "f32")},
        # a padded batch of short prompts of odd sizes in fp32, resumed from a state
        {"name": "fwd_ragged_f32", **_delta("delta_fwd", 5, 777, 6, 2, 80, 96, "f32", "f32", True, True)},
        # gradients of a training batch
        {"name": "bwd_train", **_delta("delta_bwd", 4, 2048, 16, 16, 128, 128, "bf16", "bf16")},
        # gradients of a padded batch in fp32 with shared heads
        {"name": "bwd_ragged_f32", **_delta("delta_bwd", 3, 333, 4, 2, 48, 40, "f32", "f32", True, True)},
        # the norm of one decoded token of a 768-wide model
        {"name": "norm_token", **_norm("norm_fwd", 1, 768, "bf16", "bf16", "bf16", 0.0)},
        # dropout, fp32 residual and norm of a 2560-wide model's training batch, 4 x 8192 tokens
        {"name": "norm_train", **_norm("norm_fwd", 32768, 2560, "bf16", "f32", "bf16", 0.1)},
        # and its gradients
        {"name": "norm_train_bwd", **_norm("norm_bwd", 32768, 2560, "bf16", "f32", "bf16", 0.1)},
        # a short odd tensor
        {"name": "dropout_small", **_drop(12347, "f32", 0.5)},
        # an activation of 4 x 8192 tokens x 5120 channels
        {"name": "dropout_large", **_drop(4 * 8192 * 5120, "bf16", 0.1)},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["delta_step", "delta_fwd", "delta_fwd", "delta_bwd", "delta_bwd", "norm_fwd", "norm_bwd", "dropout"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    out = rng.choice([dtype, "f32"])
    if op.startswith("delta"):
        groups = rng.choice([1, 2, 4, 8])
        heads = groups * rng.choice([1, 2, 4])
        headdim = rng.choice([16, 33, 48, 64, 80, 128, 128])
        dstate = rng.choice([16, 27, 40, 64, 96, 128, 128])
        if op == "delta_step":
            return _delta(op, _log_int(rng, 1, 128), 1, heads, groups, headdim, dstate, dtype, out)
        batch = rng.randint(1, 4)
        # at most the work of the largest listed call in this direction
        each = (24 if op == "delta_bwd" else 7) * batch * heads * headdim * dstate
        top = min(4096 if op == "delta_bwd" else 16384, int(50e9 / each))
        return _delta(op, batch, _log_int(rng, 1, top), heads, groups, headdim, dstate, dtype, out,
                      rng.random() < 0.4, rng.random() < 0.5)
    if op == "dropout":
        return _drop(_log_int(rng, 1, 1 << 27), dtype, rng.choice([0.0, 0.1, 0.25, 0.5, rng.random()]))
    dim = _log_int(rng, 3, 8192)
    return _norm(op, _log_int(rng, 1, (1 << 26) // dim), dim, dtype, rng.choice([dtype, "f32"]), out,
                 rng.choice([0.0, 0.1, rng.random() * 0.9]))


# ----------------------------------------------------------------- inputs
def _lengths(case):
    """Tokens of each batch element.  Ragged: a whole row, one token, none, then spread over the range."""
    B, L = case["batch"], case["seqlen"]
    if not case["ragged"]:
        return [L] * B
    return ([L, 1, 0] + [L * (2 * b + 1) // (2 * B) for b in range(3, B)])[:B]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 1_000_003 + 17)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    op, dt = case["op"], DTYPES[case["dtype"]]
    st = {"case": case, "op": op}
    if op.startswith("delta"):
        B, L, H, G, P, N = (case[k] for k in ("batch", "seqlen", "heads", "groups", "headdim", "dstate"))

        def unit(x):
            return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + 1e-6)

        # gates as a mixer makes them: decay -A softplus(dt + bias) with the
        # step between 1e-3 and 1e-1 where dt = 0, write strength sigmoid
        A = 1.0 + 15.0 * torch.rand(H, generator=gen, device=DEV)
        step = 1e-3 + (1e-1 - 1e-3) * torch.rand(H, generator=gen, device=DEV)
        bias = torch.log(torch.expm1(step))
        pre = normal(B, L, H) + bias
        st.update(q=unit(normal(B, L, G, N)).to(dt), k=unit(normal(B, L, G, N)).to(dt), v=normal(B, L, H, P).to(dt),
                  g=-A * torch.log1p(torch.exp(pre)), beta=torch.sigmoid(normal(B, L, H)), scale=N ** -0.5,
                  out=DTYPES[case["out"]], lengths=None, h0=None, dout=None, dlast=None)
        if op == "delta_step":
            for k in ("q", "k", "v", "g", "beta"):
                st[k] = st[k][:, 0].contiguous()
            st["state"] = normal(B, H, P, N) * 0.3
            return st
        if case["ragged"]:
            st["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device=DEV)
        if case["h0"]:
            st["h0"] = normal(B, H, P, N) * 0.3
        if op == "delta_bwd":
            st["dout"] = normal(B, L, H, P).to(st["out"])
            if case["h0"]:
                st["dlast"] = normal(B, H, P, N) * 0.3
        return st
    st.update(p=case["p"], seed=seed * 7919 + 5, offset=seed + 3)
    if op == "dropout":
        st["x"] = normal(case["n"]).to(dt)
        return st
    R, D = case["rows"], case["dim"]
    res, out = DTYPES[case["res"]], DTYPES[case["out"]]
    st.update(weight=1.0 + 0.1 * normal(D), bias=0.1 * normal(D), res=res, out=out)
    if op == "norm_fwd":
        st.update(x=normal(R, D).to(dt), residual=(2.0 * normal(R, D) + 0.5).to(res))
        return st
    s = (2.0 * normal(R, D) + 0.5).to(res)
    mean = s.float().mean(-1)
    rstd = torch.rsqrt((s.float() - mean[:, None]).square().mean(-1) + NORM_EPS)
    st.update(s=s, mean=mean, rstd=rstd, dy=normal(R, D).to(out), dresidual=(0.5 * normal(R, D)).to(res), dtype=dt)
    return st


# ------------------------------------------------------------ plain forms
def _valid(st, L):
    """[B, L] truth of the tokens inside each sequence (None: all are)."""
    if st["lengths"] is None:
        return None
    return torch.arange(L, device=DEV)[None, :] < st["lengths"][:, None]


def _chunked(q, k, v, g, beta, scale, h0):
    """The delta rule over 64-token chunks in fp32: the tokens of a chunk meet
    through the inverse of a unit lower triangular matrix, the state passes
    from chunk to chunk.  q .. beta [B, H, L, .], L a multiple of 64."""
    B, H, L, N = q.shape
    P = v.shape[-1]
    n = L // CHUNK
    q, k, v = (x.reshape(B, H, n, CHUNK, -1) for x in (q * scale, k, v))
    g, beta = (x.reshape(B, H, n, CHUNK) for x in (g, beta))
    cum = g.cumsum(-1)
    tri = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    gam = (cum[..., :, None] - cum[..., None, :]).masked_fill(~tri, -torch.inf).exp()
    kt = k.transpose(-1, -2).contiguous()
    M = (beta[..., None] * gam * (k @ kt)).tril(-1)
    # the inverse of I + M, in blocks of 1, 2, 4, .. 64: joining two blocks
    # takes the part of M below them between their inverses
    T = torch.eye(CHUNK, device=q.device).expand_as(M).contiguous()
    at = torch.arange(CHUNK, device=q.device)
    for s in (1, 2, 4, 8, 16, 32):
        join = (at[:, None] // s == at[None, :] // s + 1) & (at[None, :] // s % 2 == 0)
        T = T - T @ (M * join) @ T
    e = cum.exp()
    U0 = T @ (beta[..., None] * v)
    W = T @ ((beta * e)[..., None] * k)
    A = gam * (q @ kt)
    tail = (cum[..., -1:] - cum).exp()
    kd = (tail[..., None] * k).transpose(-1, -2).contiguous()
    qe = e[..., None] * q
    S = h0.transpose(-1, -2).contiguous() if h0 is not None else q.new_zeros(B, H, N, P)
    ys = []
    for c in range(n):
        U = U0[:, :, c] - W[:, :, c] @ S
        ys.append(qe[:, :, c] @ S + A[:, :, c] @ U)
        S = e[:, :, c, -1, None, None] * S + kd[:, :, c] @ U
    return torch.stack(ys, 2).reshape(B, H, L, P), S.transpose(-1, -2)


def _delta_plain(st, q, k, v, g, beta, h0):
    """fp32 y [B, L, H, P] and last state from inputs in fp32."""
    B, L, G, N = q.shape
    H = v.shape[2]
    ok = _valid(st, L)
    if ok is not None:
        # a token past the end: no write, no decay
        beta = beta * ok[..., None]
        g = g * ok[..., None]
    pad = -L % CHUNK

    def lay(x, heads):
        x = x if heads == H else x.repeat_interleave(H // heads, 2)
        x = torch.cat([x, x.new_zeros(B, pad, *x.shape[2:])], 1) if pad else x
        return x.transpose(1, 2).contiguous()

    y, last = _chunked(lay(q, G), lay(k, G), lay(v, H), lay(g, H), lay(beta, H), st["scale"], h0)
    y = y[:, :, :L].transpose(1, 2)
    return (y if ok is None else y * ok[..., None, None]), last


def _plain_delta_fwd(st):
    y, last = _delta_plain(st, st["q"].float(), st["k"].float(), st["v"].float(), st["g"], st["beta"], st["h0"])
    return {"y": y.to(st["out"]).contiguous(), "last_state": last.contiguous()}


def _plain_delta_bwd(st):
    names = ["q", "k", "v", "g", "beta"] + (["h0"] if st["h0"] is not None else [])
    with torch.enable_grad():
        x = {n: st[n].float().detach().requires_grad_(True) for n in names}
        y, last = _delta_plain(st, x["q"], x["k"], x["v"], x["g"], x["beta"], x.get("h0"))
        loss = (y * st["dout"].float()).sum()
        if st["dlast"] is not None:
            loss = loss + (last * st["dlast"]).sum()
        grads = torch.autograd.grad(loss, [x[n] for n in names])
    return {"d" + n: d.to(st[n].dtype) for n, d in zip(names, grads)}


def _plain_delta_step(st):
    S, H = st["state"], st["v"].shape[1]
    r = H // st["q"].shape[1]
    q, k = (st[n].float().repeat_interleave(r, 1) for n in ("q", "k"))
    S = S * st["g"].exp()[..., None, None]
    u = st["beta"][..., None] * (st["v"].float() - (S * k[:, :, None, :]).sum(-1))
    S = S + u[..., None] * k[:, :, None, :]
    y = (S * (st["scale"] * q)[:, :, None, :]).sum(-1)
    st["state"].copy_(S)
    return {"y": y.to(st["out"]), "state": st["state"]}


def _mul32(a, m):
    """High and low words of a product of 32-bit words held in 64 bits (the
    low 64 bits of a wrapped product are exact)."""
    w = a * m
    return (w >> 32) & MASK32, w & MASK32


def _keep(n, p, seed, offset):
    """Truth of the n elements that dropout keeps."""
    i = torch.arange((n + 3) // 4, dtype=torch.int64, device=DEV)
    c0, c1 = i & MASK32, i >> 32
    c2, c3 = torch.full_like(i, offset & MASK32), torch.full_like(i, offset >> 32)
    k0, k1 = seed & MASK32, (seed >> 32) & MASK32
    for _ in range(10):
        h0, l0 = _mul32(c0, 0xD2511F53)
        h1, l1 = _mul32(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & MASK32, (k1 + 0xBB67AE85) & MASK32
    words = torch.stack([c0, c1, c2, c3], -1).reshape(-1)[:n]
    return words >= int(p * 4294967296.0)


def _dropped(x, p, seed, offset):
    """x in fp32 with dropout."""
    if p == 0.0:
        return x.float()
    keep = _keep(x.numel(), p, seed, offset).reshape(x.shape)
    return torch.where(keep, x.float() * (1.0 / (1.0 - p)), 0.0)


def _plain_dropout(st):
    return {"y": _dropped(st["x"], st["p"], st["seed"], st["offset"]).to(st["x"].dtype)}


def _plain_norm_fwd(st):
    s = _dropped(st["x"], st["p"], st["seed"], st["offset"]) + st["residual"].float()
    mean = s.mean(-1)
    d = s - mean[:, None]
    rstd = torch.rsqrt(d.square().mean(-1) + NORM_EPS)
    y = d * rstd[:, None] * st["weight"] + st["bias"]
    return {"y": y.to(st["out"]), "residual": s.to(st["res"]), "mean": mean, "rstd": rstd}


def _plain_norm_bwd(st):
    xhat = (st["s"].float() - st["mean"][:, None]) * st["rstd"][:, None]
    dy = st["dy"].float()
    w = dy * st["weight"]
    ds = (w - w.mean(-1, keepdim=True) - xhat * (w * xhat).mean(-1, keepdim=True)) * st["rstd"][:, None]
    ds = ds + st["dresidual"].float()
    return {"dx": _dropped(ds, st["p"], st["seed"], st["offset"]).to(st["dtype"]), "dresidual": ds.to(st["res"]),
            "dweight": (dy * xhat).sum(0), "dbias": dy.sum(0)}


_PLAIN = {"delta_step": _plain_delta_step, "delta_fwd": _plain_delta_fwd, "delta_bwd": _plain_delta_bwd,
          "norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "dropout": _plain_dropout}


# ------------------------------------------------- the library's own calls
def _own(st):
    import selective_state_space_25_amd as ss

    op = st["op"]
    if op == "delta_step":
        y = ss.delta_step(st["state"], st["q"], st["k"], st["v"], st["g"], st["beta"], out_dtype=st["out"])
        return {"y": y, "state": st["state"]}
    if op == "delta_fwd":
        y, last = ss.delta_fwd(st["q"], st["k"], st["v"], st["g"], st["beta"], lengths=st["lengths"], h0=st["h0"],
                               out_dtype=st["out"])
        return {"y": y, "last_state": last}
    if op == "delta_bwd":
        return ss.delta_bwd(st["q"], st["k"], st["v"], st["g"], st["beta"], st["dout"], lengths=st["lengths"],
                            h0=st["h0"], dlast_state=st["dlast"])
    if op == "dropout":
        return {"y": ss.dropout(st["x"], st["p"], st["seed"], st["offset"])}
    if op == "norm_fwd":
        y, s, mean, rstd = ss.layer_norm_fwd(st["x"], st["weight"], st["bias"], residual=st["residual"], eps=NORM_EPS,
                                             p=st["p"], seed=st["seed"], offset=st["offset"], out_dtype=st["out"])
        return {"y": y, "residual": s, "mean": mean, "rstd": rstd}
    return ss.layer_norm_bwd(st["dy"], st["s"], st["weight"], st["mean"], st["rstd"], dresidual=st["dresidual"],
                             p=st["p"], seed=st["seed"], offset=st["offset"], x_dtype=st["dtype"])


def run(state):
    if own:
        return _own(state)
    with torch.no_grad():
        return _PLAIN[state["op"]](state)


# ------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2}
    es = size[case["dtype"]]
    if op == "dropout":
        return {"bytes": 2 * es * case["n"], "flops": case["n"]}
    if op.startswith("norm"):
        n, so, sr = case["rows"] * case["dim"], size[case["out"]], size[case["res"]]
        if op == "norm_fwd":
            return {"bytes": n * (es + 2 * sr + so) + 8 * (case["rows"] + case["dim"]), "flops": 9 * n}
        return {"bytes": n * (so + 3 * sr + es) + 8 * case["rows"] + 12 * case["dim"], "flops": 16 * n}
    B, H, G, P, N = (case[k] for k in ("batch", "heads", "groups", "headdim", "dstate"))
    so = size[case["out"]]
    tokens = sum(_lengths(case)) if op != "delta_step" else B
    state = 4 * B * H * P * N
    ins = tokens * (2 * G * N * es + H * P * es + 8 * H)
    if op == "delta_step":
        return {"bytes": 2 * state + ins + tokens * H * P * so, "flops": 7 * tokens * H * P * N}
    h0 = state if case["h0"] else 0
    padded = B * case["seqlen"]
    if op == "delta_fwd":
        return {"bytes": ins + padded * H * P * so + state + h0, "flops": 7 * tokens * H * P * N}
    outs = padded * (2 * G * N * es + H * P * es + 8 * H)
    return {"bytes": ins + outs + tokens * H * P * so + 3 * h0, "flops": 24 * tokens * H * P * N}


# --------------------------------------------------- the definition, fp64
def _exact_inputs(st):
    H = st["v"].shape[-2]
    r = H // st["q"].shape[-2]
    head = torch.arange(H, device=DEV) // r
    d = {n: st[n].double() for n in ("v", "g", "beta")}
    d["q"], d["k"] = (st[n].double().index_select(st[n].dim() - 2, head) for n in ("q", "k"))
    if st.get("lengths") is not None:
        live = (torch.arange(d["v"].shape[1], device=DEV) < st["lengths"][:, None]).double()
    else:
        live = torch.ones(d["v"].shape[:-2], dtype=torch.float64, device=DEV)
    return d, live


def _token(S, d, live, t):
    """One token's decayed state, error and new state; a token past the end leaves the state."""
    m = live[:, t, None]
    Sa = S * torch.exp(d["g"][:, t] * m)[..., None, None]
    k = d["k"][:, t]
    err = d["v"][:, t] - torch.matmul(Sa, k[..., None])[..., 0]
    u = (d["beta"][:, t] * m)[..., None] * err
    return Sa, err, u, Sa + u[..., None] * k[:, :, None, :]


def _exact_delta(st, op):
    d, live = _exact_inputs(st)
    B, L, H, P = d["v"].shape
    N = d["q"].shape[-1]
    S = st["h0"].double() if st["h0"] is not None else torch.zeros(B, H, P, N, dtype=torch.float64, device=DEV)
    every = 64
    kept = []
    ys = torch.empty(B, L, H, P, dtype=torch.float64, device=DEV)
    for t in range(L):
        if t % every == 0:
            kept.append(S)
        S = _token(S, d, live, t)[3]
        ys[:, t] = st["scale"] * torch.matmul(S, d["q"][:, t, :, :, None])[..., 0] * live[:, t, None, None]
    if op == "delta_fwd":
        return {"y": ys, "last_state": S}
    out = {n: torch.zeros_like(d[n]) for n in ("q", "k", "v", "g", "beta")}
    D = st["dlast"].double() if st["dlast"] is not None else torch.zeros_like(S)
    for c in range(len(kept) - 1, -1, -1):
        S, hist = kept.pop(), []
        for t in range(c * every, min(L, (c + 1) * every)):
            Sa, err, u, S = _token(S, d, live, t)
            hist.append((t, Sa, err, u, S))
        for t, Sa, err, u, St in reversed(hist):
            m = live[:, t, None]
            q, k, beta = d["q"][:, t], d["k"][:, t], d["beta"][:, t]
            dy = st["dout"][:, t].double() * (st["scale"] * m[..., None])
            D = D + dy[..., None] * q[:, :, None, :]
            out["q"][:, t] = torch.matmul(dy[:, :, None, :], St)[:, :, 0]
            du = torch.matmul(D, k[..., None])[..., 0] * m[..., None]
            de = beta[..., None] * du
            out["v"][:, t] = de
            out["beta"][:, t] = (du * err).sum(-1)
            out["k"][:, t] = (torch.matmul(u[:, :, None, :], D) - torch.matmul(de[:, :, None, :], Sa))[:, :, 0] * m[..., None]
            X = D - de[..., None] * k[:, :, None, :]
            out["g"][:, t] = (X * Sa).sum((-1, -2)) * m
            D = X * torch.exp(d["g"][:, t] * m)[..., None, None]
    G = st["q"].shape[2]
    for n in ("q", "k"):
        out[n] = out[n].reshape(B, L, G, H // G, N).sum(3)
    got = {"d" + n: x for n, x in out.items()}
    if st["h0"] is not None:
        got["dh0"] = D
    return got


def _exact_step(st):
    d, _ = _exact_inputs(st)
    S = st["state"].double() * torch.exp(d["g"])[..., None, None]
    err = d["v"] - torch.matmul(S, d["k"][..., None])[..., 0]
    S = S + (d["beta"][..., None] * err)[..., None] * d["k"][:, :, None, :]
    return {"y": st["scale"] * torch.matmul(S, d["q"][..., None])[..., 0], "state": S}


def _words(i, seed, offset):
    """The four words of Philox4x32-10 at counters i, with 16-bit limb products."""
    def mul(a, m):
        low = a * (m & 0xFFFF)
        up = a * (m >> 16) + (low >> 16)
        return up >> 16, ((up & 0xFFFF) << 16) | (low & 0xFFFF)

    x = [i % 2 ** 32, i // 2 ** 32, torch.zeros_like(i) + offset % 2 ** 32, torch.zeros_like(i) + offset // 2 ** 32]
    for r in range(10):
        ka = (seed + r * 0x9E3779B9) % 2 ** 32
        kb = (seed // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32
        (ha, la), (hb, lb) = mul(x[0], 0xD2511F53), mul(x[2], 0xCD9E8D57)
        x = [hb ^ x[1] ^ ka, lb, ha ^ x[3] ^ kb, la]
    return x


def _exact_dropped(x, p, seed, offset):
    n = x.numel()
    y = x.double().reshape(-1).clone()
    if p == 0.0:
        return y.reshape(x.shape)
    limit = int(p * 2 ** 32)
    for j, w in enumerate(_words(torch.arange((n + 3) // 4, device=DEV), seed, offset)):
        part = y[j::4]
        part *= (w[: part.numel()] >= limit) / (1.0 - p)
    return y.reshape(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op == "delta_step":
        return _exact_step(st)
    if op.startswith("delta"):
        return _exact_delta(st, op)
    if op == "dropout":
        return {"y": _exact_dropped(st["x"], st["p"], st["seed"], st["offset"])}
    w = st["weight"].double()
    D = case["dim"]
    if op == "norm_fwd":
        s = _exact_dropped(st["x"], st["p"], st["seed"], st["offset"]) + st["residual"].double()
        mean = s.sum(-1) / D
        s2 = s - mean[:, None]
        rstd = 1.0 / torch.sqrt((s2 * s2).sum(-1) / D + NORM_EPS)
        return {"y": s2 * rstd[:, None] * w + st["bias"].double(), "residual": s, "mean": mean, "rstd": rstd}
    dy, rstd = st["dy"].double(), st["rstd"].double()[:, None]
    z = (st["s"].double() - st["mean"].double()[:, None]) * rstd
    wdy = dy * w
    ds = rstd * (wdy - (wdy.sum(-1) / D)[:, None] - z * ((wdy * z).sum(-1) / D)[:, None]) + st["dresidual"].double()
    return {"dx": _exact_dropped(ds, st["p"], st["seed"], st["offset"]), "dresidual": ds,
            "dweight": (dy * z).sum(0), "dbias": dy.sum(0)}
