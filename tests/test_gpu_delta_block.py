"""The example that runs the gated delta rule, layer norm and dropout together."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("delta_block", os.path.join(ROOT, "examples", "delta_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_recall_answers_on_cpu():
    """The task's own answers, by replaying each sequence with a dict."""
    ex = _example()
    tokens, answer = ex.batch_of(3, 50, 5, 7, torch.Generator().manual_seed(3))
    for b in range(3):
        held = {}
        for t in range(50):
            key, value = tokens[b, t].tolist()
            if value == 7:
                assert answer[b, t] == held.get(key, -100)
            else:
                assert answer[b, t] == -100
                held[key] = value


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_trains(dtype):
    """A uniform guess costs ln 32 = 3.47; the mean of the last ten losses has to be well under it."""
    ex = _example()
    torch.manual_seed(0)
    losses = ex.train(ex.Recall(dtype=dtype).to("cuda"), 120)
    assert losses[0] > 3.0
    assert sum(losses[-10:]) / 10 < 2.0


@pytest.mark.gpu
@pytest.mark.parametrize("prompt", [1, 16, 17, 64, 150])
def test_decode_continues_prompt(prompt):
    """fp32: sums of at most 128 + 64 terms of size one, reordered, in each of
    some ten layers: 10 * 192 * 2^-24 = 1.1e-4, times ten for the norms."""
    ex = _example()
    torch.manual_seed(1)
    model = ex.Recall(dtype="f32").to("cuda")
    tokens, _ = ex.batch_of(3, 160, 32, 32, torch.Generator().manual_seed(2))
    assert ex.decode_gap(model, prompt, tokens.to("cuda")) < 1.2e-3


@pytest.mark.gpu
def test_gradients_against_plain_torch():
    """The model's parameter gradients against autograd through a plain fp64
    recurrence (no dropout).  fp32 chains of a few hundred terms, three norms
    deep: 1e-4 of each gradient's largest entry."""
    ex = _example()
    torch.manual_seed(2)
    model = ex.Recall(dim=48, heads=2, headdim=20, dstate=12, dtype="f32").to("cuda")
    tokens, answer = (t.to("cuda") for t in ex.batch_of(2, 70, 32, 32, torch.Generator().manual_seed(4)))

    def loss_of(logits):
        return torch.nn.functional.cross_entropy(logits.flatten(0, 1), answer.flatten(), ignore_index=-100)

    loss_of(model(tokens)).backward()
    got = {n: p.grad.cpu().double() for n, p in model.named_parameters()}

    ref = ex.Recall(dim=48, heads=2, headdim=20, dstate=12, dtype="f32")
    ref.load_state_dict({n: t.cpu() for n, t in model.state_dict().items()})
    ref.double()
    tokens, answer = tokens.cpu(), answer.cpu()

    def delta(q, k, v, g, beta):
        S = torch.zeros(q.shape[0], q.shape[2], v.shape[-1], q.shape[-1], dtype=torch.float64)
        ys = []
        for t in range(q.shape[1]):
            S = S * torch.exp(g[:, t])[..., None, None]
            u = beta[:, t, :, None] * (v[:, t] - (S @ k[:, t, :, :, None])[..., 0])
            S = S + u[..., None] * k[:, t, :, None]
            ys.append((S @ q[:, t, :, :, None])[..., 0] * q.shape[-1] ** -0.5)
        return torch.stack(ys, 1)

    x, s = ref.key(tokens[..., 0]) + ref.value(tokens[..., 1]), 0
    for block in ref.blocks:
        s = s + x
        h = torch.nn.functional.layer_norm(s, s.shape[-1:], block.norm_w, block.norm_b)
        heads, headdim, dstate = block.sizes
        q, k, v = block.qkv(h).split([heads * dstate, heads * dstate, heads * headdim], -1)
        q, k, v = (t.unflatten(-1, (heads, -1)) for t in (q, k, v))
        q, k = (t / t.norm(dim=-1, keepdim=True) for t in (q, k))
        decay, write = block.gates(h).split(heads, -1)
        y = delta(q, k, v, -torch.nn.functional.softplus(decay), torch.sigmoid(write))
        x = block.out(y.flatten(-2))
    h = torch.nn.functional.layer_norm(s + x, s.shape[-1:], ref.norm_w, ref.norm_b)
    loss_of(ref.head(h)).backward()
    for n, p in ref.named_parameters():
        assert (got[n] - p.grad).abs().max() <= 1e-4 * p.grad.abs().max(), n
