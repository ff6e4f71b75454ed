"""A small recall model built from the gated delta rule, layer norm and dropout.

    python examples/delta_block.py [--steps 200] [--dtype bf16]

A token carries a key and, unless it asks, a value; a token that asks has to
be answered with the value last written to its key.  Each block is

    s = dropout(x) + s;   x = W_o delta(layer_norm(s))

so the norm, the residual sum and the dropout are one call in either direction
(layer_norm_fwd, layer_norm_bwd).  The script trains the model (delta_fwd,
delta_bwd), then reads a sequence as a prompt (delta_fwd with last_state) and
goes on token by token (bind_delta_step on the same state), and compares these
answers with those of the whole sequence at once.  The projections and the
loss are torch's.
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_25_amd as ss  # noqa: E402

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


class DropoutAddNorm(torch.autograd.Function):
    """(layer_norm(s), s) of s = dropout(x) + residual, the residual stream in fp32."""

    @staticmethod
    def forward(ctx, x, residual, weight, bias, p, seed, offset):
        y, s, mean, rstd = ss.layer_norm_fwd(x.contiguous(), weight, bias, residual, p=p, seed=seed, offset=offset)
        ctx.save_for_backward(s, weight, mean, rstd)
        ctx.drop, ctx.dtype = (p, seed, offset), x.dtype
        return y, s

    @staticmethod
    def backward(ctx, dy, ds):
        s, weight, mean, rstd = ctx.saved_tensors
        p, seed, offset = ctx.drop
        g = ss.layer_norm_bwd(dy.contiguous(), s, weight, mean, rstd, ds.contiguous(), p=p, seed=seed, offset=offset,
                              x_dtype=ctx.dtype)
        return g["dx"], g["dresidual"], g["dweight"], g["dbias"], None, None, None


class Delta(torch.autograd.Function):
    """The gated delta rule from an empty state."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta):
        args = tuple(t.contiguous() for t in (q, k, v, g, beta))
        ctx.save_for_backward(*args)
        return ss.delta_fwd(*args, return_last_state=False, out_dtype=q.dtype)[0]

    @staticmethod
    def backward(ctx, dout):
        g = ss.delta_bwd(*ctx.saved_tensors, dout.contiguous())
        return g["dq"], g["dk"], g["dv"], g["dg"], g["dbeta"]


class Block(torch.nn.Module):
    def __init__(self, dim, heads, headdim, dstate):
        super().__init__()
        self.sizes = heads, headdim, dstate
        self.norm_w = torch.nn.Parameter(torch.ones(dim))
        self.norm_b = torch.nn.Parameter(torch.zeros(dim))
        self.qkv = torch.nn.Linear(dim, heads * (2 * dstate + headdim), bias=False)
        self.gates = torch.nn.Linear(dim, 2 * heads)
        with torch.no_grad():   # slow decays to begin with
            self.gates.bias[:heads] = -5.0
        self.out = torch.nn.Linear(heads * headdim, dim, bias=False)

    def inputs(self, x):
        """q, k, v in x's dtype and the fp32 gates of normed tokens x [batch, L, dim]."""
        heads, headdim, dstate = self.sizes
        q, k, v = F.linear(x, self.qkv.weight.to(x.dtype)).split([heads * dstate, heads * dstate, heads * headdim], -1)
        shape = x.shape[:-1] + (heads, -1)
        q, k = (F.normalize(t.reshape(shape).float(), dim=-1).to(x.dtype) for t in (q, k))
        decay, write = F.linear(x.float(), self.gates.weight, self.gates.bias).split(heads, -1)
        return q, k, v.reshape(shape), -F.softplus(decay), torch.sigmoid(write)

    def project(self, y):
        return F.linear(y.flatten(-2), self.out.weight.to(y.dtype))


class Recall(torch.nn.Module):
    def __init__(self, keys=32, values=32, dim=128, heads=4, headdim=32, dstate=32, layers=2, p=0.1, dtype="bf16"):
        super().__init__()
        self.dtype, self.p = DTYPES[dtype], p
        self.key = torch.nn.Embedding(keys, dim)
        self.value = torch.nn.Embedding(values + 1, dim)   # the last one: a token that asks
        self.blocks = torch.nn.ModuleList(Block(dim, heads, headdim, dstate) for _ in range(layers))
        self.norm_w = torch.nn.Parameter(torch.ones(dim))
        self.norm_b = torch.nn.Parameter(torch.zeros(dim))
        self.head = torch.nn.Linear(dim, values)

    def embed(self, tokens):
        """The stream's first term, and the fp32 residual it is added to."""
        x = (self.key(tokens[..., 0]) + self.value(tokens[..., 1])).to(self.dtype)
        return x, torch.zeros(x.shape, device=x.device)

    def forward(self, tokens, seed=None):
        """Logits [batch, L, values] of tokens [batch, L, 2]; seed: of this step's dropout (None: no dropout)."""
        p = 0.0 if seed is None else self.p
        x, s = self.embed(tokens)
        for i, block in enumerate(self.blocks):
            h, s = DropoutAddNorm.apply(x, s, block.norm_w, block.norm_b, p, seed or 0, i)
            x = block.project(Delta.apply(*block.inputs(h)))
        h, s = DropoutAddNorm.apply(x, s, self.norm_w, self.norm_b, p, seed or 0, len(self.blocks))
        return self.head(h.float())

    @torch.no_grad()
    def prefill(self, tokens):
        """Logits of a prompt's last token, and the blocks' states after it."""
        x, s = self.embed(tokens)
        states = []
        for block in self.blocks:
            h, s = ss.layer_norm_fwd(x, block.norm_w, block.norm_b, s)[:2]
            y, last = ss.delta_fwd(*(t.contiguous() for t in block.inputs(h)), out_dtype=self.dtype)
            states.append(last)
            x = block.project(y)
        h = ss.layer_norm_fwd(x, self.norm_w, self.norm_b, s)[0]
        return self.head(h[:, -1].float()), states

    @torch.no_grad()
    def decoder(self, states):
        """A function from one token [batch, 2] to its logits, which updates
        the states in place.  Call it on the stream that is current here: the
        bound calls stay on it."""
        batch = states[0].shape[0]
        bound = []
        for block, state in zip(self.blocks, states):
            heads, headdim, dstate = block.sizes
            new = lambda *shape, dtype=self.dtype: torch.empty(shape, dtype=dtype, device=state.device)
            args = (new(batch, heads, dstate), new(batch, heads, dstate), new(batch, heads, headdim),
                    new(batch, heads, dtype=torch.float32), new(batch, heads, dtype=torch.float32))
            call, y = ss.bind_delta_step(state, *args, out_dtype=self.dtype)
            bound.append((block, args, call, y))

        @torch.no_grad()
        def step(token):
            x, s = self.embed(token)
            for block, args, call, y in bound:
                h, s = ss.layer_norm_fwd(x, block.norm_w, block.norm_b, s)[:2]
                for dst, src in zip(args, block.inputs(h)):
                    dst.copy_(src)
                call()
                x = block.project(y)
            return self.head(ss.layer_norm_fwd(x, self.norm_w, self.norm_b, s)[0].float())

        return step


def batch_of(batch, L, keys, values, gen):
    """Tokens [batch, L, 2] and answers [batch, L] (-100: nothing asked, or the key not written yet)."""
    key = torch.randint(keys, (batch, L), generator=gen)
    value = torch.randint(values, (batch, L), generator=gen)
    asks = torch.rand(batch, L, generator=gen) < 0.5
    answer = torch.full((batch, L), -100)
    held = torch.full((batch, keys), -100)
    rows = torch.arange(batch)
    for t in range(L):
        now = held[rows, key[:, t]]
        answer[:, t] = torch.where(asks[:, t], now, answer[:, t])
        held[rows, key[:, t]] = torch.where(asks[:, t], now, value[:, t])
    return torch.stack([key, torch.where(asks, values, value)], -1), answer


def train(model, steps, batch=16, L=160, keys=32, values=32, lr=3e-3, seed=0, log=None):
    """Losses of `steps` updates."""
    dev = model.norm_w.device
    gen = torch.Generator().manual_seed(seed)
    opt = torch.optim.AdamW(model.parameters(), lr=lr)
    losses = []
    for i in range(steps):
        tokens, answer = (t.to(dev) for t in batch_of(batch, L, keys, values, gen))
        loss = F.cross_entropy(model(tokens, seed=i).flatten(0, 1), answer.flatten(), ignore_index=-100)
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
        if log and (i % 20 == 0 or i + 1 == steps):
            log(f"step {i:4d}  loss {losses[-1]:.4f}")
    return losses


def decode_gap(model, prompt, tokens):
    """Largest difference between the logits of `tokens` [batch, L, 2] at once
    and as a prompt of `prompt` tokens followed by one token at a time."""
    with torch.no_grad():
        whole = model(tokens)
    logits, states = model.prefill(tokens[:, :prompt].contiguous())
    step = model.decoder(states)
    gap = (logits - whole[:, prompt - 1]).abs().max()
    for t in range(prompt, tokens.shape[1]):
        gap = torch.maximum(gap, (step(tokens[:, t]) - whole[:, t]).abs().max())
    return float(gap)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--dtype", choices=sorted(DTYPES), default="bf16")
    args = ap.parse_args()
    torch.manual_seed(0)
    model = Recall(dtype=args.dtype).to("cuda")
    train(model, args.steps, log=lambda line: print(line, flush=True))
    tokens, answer = (t.to("cuda") for t in batch_of(8, 200, 32, 32, torch.Generator().manual_seed(1)))
    with torch.no_grad():
        asked = answer >= 0
        right = (model(tokens).argmax(-1) == answer)[asked].float().mean()
    print(f"answers right: {100 * float(right):.1f} % of {int(asked.sum())}")
    print(f"prompt and single tokens against the whole sequence: logits differ by at most {decode_gap(model, 150, tokens):.2e}")


if __name__ == "__main__":
    main()
