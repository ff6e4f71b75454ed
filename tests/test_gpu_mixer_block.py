"""A Mamba-2 block made of the new operators, as a model runs it: residual norm,
projection, mixer, gated norm, projection; prompt and tokens, and training."""
import pytest
import torch

import selective_state_space_25_amd as ss

pytestmark = pytest.mark.gpu

F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64
DEV = "cuda:0"
H, P, G, N, K, WIDE = 4, 64, 1, 64, 4, 96
INNER, C = H * P, H * P + 2 * G * N


def weights(seed=1):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s, by=1.0: (by * torch.randn(s, generator=gen)).to(DEV)
    return {"norm": 1 + r(WIDE, by=0.1), "w_in": r(INNER + C + H, WIDE, by=WIDE ** -0.5), "conv_w": r(C, K, by=0.5),
            "conv_b": r(C, by=0.1), "A": -torch.exp(r(H, by=0.5)), "D": 1 + r(H, by=0.1), "dt_bias": r(H, by=0.5) - 2,
            "gate_norm": 1 + r(INNER, by=0.1), "w_out": r(WIDE, INNER, by=INNER ** -0.5)}


def split(rows):
    return rows[..., :INNER], rows[..., INNER:INNER + C], rows[..., INNER + C:]


class Block:
    def __init__(self, w, dtype):
        self.w = {k: v.to(dtype) if k in ("w_in", "w_out") else v for k, v in w.items()}
        self.dtype = dtype

    def prompt(self, x, residual, lengths=None):
        w = self.w
        y, s, _, _ = ss.rms_norm_fwd(x, w["norm"], residual)
        z, xbc, dt = split(y @ w["w_in"].t())
        y, state, conv = ss.mamba2_conv_fwd(xbc, dt, w["conv_w"], w["conv_b"], w["A"], w["D"], w["dt_bias"], ngroups=G,
                                            dstate=N, lengths=lengths, out_dtype=self.dtype)
        y = y.reshape(*y.shape[:2], INNER)
        y, _, _, _ = ss.rms_norm_fwd(y, w["gate_norm"], gate=z)
        return y @ w["w_out"].t(), s, state, conv

    def token(self, x, residual, state, conv):
        w = self.w
        y, s, _, _ = ss.rms_norm_fwd(x, w["norm"], residual)
        z, xbc, dt = split(y @ w["w_in"].t())
        y = ss.mamba2_conv_step(state, conv, xbc, dt, w["conv_w"], w["conv_b"], w["A"], w["D"], w["dt_bias"],
                                out_dtype=self.dtype)
        y, _, _, _ = ss.rms_norm_fwd(y.reshape(-1, INNER), w["gate_norm"], gate=z)
        return y @ w["w_out"].t(), s


def reference(w, x, residual):
    """The block in fp64, token by token, differentiable."""
    s = x + residual
    y = s * torch.rsqrt(s.square().mean(-1, keepdim=True) + 1e-5) * w["norm"]
    z, xbc, dt = split(y @ w["w_in"].t())
    B, L, _ = xbc.shape
    pad = torch.cat([xbc.new_zeros(B, K - 1, C), xbc], 1)
    v = torch.nn.functional.silu(sum(pad[:, k:k + L] * w["conv_w"][:, k] for k in range(K)) + w["conv_b"])
    step = torch.nn.functional.softplus(dt + w["dt_bias"])
    S, ys = x.new_zeros(B, H, P, N), []
    for t in range(L):
        xt, b, c = v[:, t, :INNER].reshape(B, H, P), v[:, t, INNER:INNER + N], v[:, t, INNER + N:]
        a = torch.exp(step[:, t] * w["A"])[..., None, None]
        S = a * S + (step[:, t, :, None] * xt)[..., None] * b[:, None, None]
        ys.append((S * c[:, None, None]).sum(-1) + w["D"][:, None] * xt)
    y = torch.stack(ys, 1).reshape(B, L, INNER) * torch.nn.functional.silu(z)
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-5) * w["gate_norm"]
    return y @ w["w_out"].t(), s


@pytest.mark.parametrize("L", [20, 150])
def test_prompt_then_tokens(gpu, L):
    """What a prompt and then tokens give is what the reference gives for the
    whole sequence.  fp32: the projections' sums (256 and 96 terms) and the
    mixer's, under 2^-24 times a few thousand terms of the outputs' size."""
    w = weights()
    gen = torch.Generator().manual_seed(2)
    x, res = (torch.randn(2, L + 3, WIDE, generator=gen).to(DEV) for _ in range(2))
    block = Block(w, F32)
    out, s, state, conv = block.prompt(x[:, :L].contiguous(), res[:, :L].contiguous())
    outs = [out]
    for t in range(L, L + 3):
        y, _ = block.token(x[:, t].contiguous(), res[:, t].contiguous(), state, conv)
        outs.append(y[:, None])
    ref, rs = reference({k: v.double() for k, v in w.items()}, x.double(), res.double())
    torch.cuda.synchronize()
    got = torch.cat(outs, 1).double()
    assert torch.equal(s, (x + res)[:, :L])
    assert (got - ref).abs().max() <= 4096 * 2.0 ** -24 * ref.abs().max()


def test_padded_batch_is_its_sequences(gpu):
    """Each row of a padded batch comes out as it does alone, up to the fp32
    sums' order (segments depend on the batch)."""
    w = weights()
    gen = torch.Generator().manual_seed(3)
    block = Block(w, F32)
    n = [150, 1, 0, 70]
    x, res = (torch.randn(4, 150, WIDE, generator=gen).to(DEV) for _ in range(2))
    out, _, state, conv = block.prompt(x, res, torch.tensor(n, dtype=torch.int32, device=DEV))
    for i, m in enumerate(n):
        if m == 0:
            assert not state[i].any() and not conv[i].any()
            continue
        one, _, st, cv = block.prompt(x[i:i + 1, :m].contiguous(), res[i:i + 1, :m].contiguous())
        top = one.abs().max()
        assert (out[i:i + 1, :m] - one).abs().max() <= 4096 * 2.0 ** -24 * top
        assert (state[i:i + 1] - st).abs().max() <= 4096 * 2.0 ** -24 * st.abs().max()
        assert (conv[i:i + 1] - cv).abs().max() <= 4096 * 2.0 ** -24 * cv.abs().max()


def test_training(gpu):
    """Gradients of the whole block through the library's backward calls
    against fp64 autograd of the reference.  fp32 throughout; what bounds the
    difference are the Mamba-2 gradients' own (1e-3 of a gradient's root mean
    square, their tests' bound) times the sums behind them."""
    w = weights()
    gen = torch.Generator().manual_seed(4)
    B, L = 2, 80
    x, res, dy = (torch.randn(B, L, WIDE, generator=gen).to(DEV) for _ in range(3))
    # forward, keeping what the gradients need
    h, s, rstd, _ = ss.rms_norm_fwd(x, w["norm"], res)
    rows = h @ w["w_in"].t()
    z, xbc, dt = split(rows)
    (v, b, c), _ = ss.short_conv_fwd(xbc, w["conv_w"], w["conv_b"], split=[INNER, G * N, G * N])
    args = (v.reshape(B, L, H, P), dt.contiguous(), w["A"], b.reshape(B, L, G, N), c.reshape(B, L, G, N), w["D"], None, w["dt_bias"])
    y, _ = ss.mamba2_fwd(*args)
    y = y.reshape(B, L, INNER)
    gated, _, grstd, _ = ss.rms_norm_fwd(y, w["gate_norm"], gate=z)
    out = gated @ w["w_out"].t()
    # backward
    g = {"w_out": dy.reshape(-1, WIDE).t() @ gated.reshape(-1, INNER)}
    gg = ss.rms_norm_bwd(dy @ w["w_out"], y, w["gate_norm"], grstd, gate=z)
    g["gate_norm"] = gg["dweight"]
    m = ss.mamba2_bwd(*args, dout=gg["dx"].reshape(B, L, H, P))
    g["A"], g["D"], g["dt_bias"] = m["dA"], m["dD"], m["ddt_bias"]
    cg = ss.short_conv_bwd(xbc, w["conv_w"], w["conv_b"], [m["dx"].reshape(B, L, INNER), m["dB"].reshape(B, L, G * N),
                                                            m["dC"].reshape(B, L, G * N)])
    g["conv_w"], g["conv_b"] = cg["dweight"], cg["dbias"]
    drows = torch.cat([gg["dgate"], cg["dx"], m["ddt"]], -1)
    g["w_in"] = drows.reshape(-1, INNER + C + H).t() @ h.reshape(-1, WIDE)
    ng = ss.rms_norm_bwd(drows @ w["w_in"], s, w["norm"], rstd)
    g["norm"], g["x"], g["res"] = ng["dweight"], ng["dx"], ng["dresidual"]
    torch.cuda.synchronize()
    leaf = {k: t.double().requires_grad_(True) for k, t in {**w, "x": x, "res": res}.items()}
    ref, _ = reference(leaf, leaf["x"], leaf["res"])
    (ref * dy.double()).sum().backward()
    assert (out.double() - ref).abs().max() <= 2e-3 * ref.abs().max()
    for k in g:
        r = leaf[k].grad
        assert (g[k].double() - r).abs().max() <= 5e-3 * r.abs().max(), k
