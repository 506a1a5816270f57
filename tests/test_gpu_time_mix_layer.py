"""The time-mixing layer (gemm_rwkv_amd/time_mix.py), which runs the operators
and the quantized products together, against the same layer written in 64-bit
torch on the CPU: served in one batch and in parts through slots, and its
gradients.

Tolerances.  Between the two lie roundings to u = 2^-11 (fp16) or 2^-8 (bf16)
of some sixteen intermediates in a row (mixtures, projections, decay, kappa,
y, gate, output): sqrt(16) u if they are independent.  The raw decay is an
exponent and the state remembers some tens of tokens, which multiplies its
share by up to eight: relative L2 errors stay under 32 u.  The backward pass
rounds as often again and reads the rounded forward values: 64 u."""

import numpy as np
import pytest
import torch

from gemm_rwkv_amd import time_mix as tm
from gpu_helpers import say
from oracle import quant

pytestmark = pytest.mark.gpu

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def plain(p, x, delta, lens, shift, state, width):
    """The layer in float64, token by token."""
    heads = width // 64
    full = x + delta
    h = torch.nn.functional.layer_norm(full, (width,), p["gamma"], p["beta"], tm.NORM_EPS)
    outs, lasts, states, t = [], [], [], 0
    for i, n in enumerate(lens):
        prev, S = shift[i], state[i]
        for _ in range(n):
            m = [h[t] + (prev - h[t]) * p["mu"][j] for j in range(6)]
            r, k, v = p["W_r"] @ m[0], p["W_k"] @ m[2], p["W_v"] @ m[3]
            w = p["w0"] + torch.tanh(m[1] @ p["A_w"]) @ p["B_w"]
            rate = torch.sigmoid(p["a0"] + m[4] @ p["A_a"] @ p["B_a"])
            g = torch.sigmoid(m[5] @ p["A_g"]) @ p["B_g"]
            kappa = torch.nn.functional.normalize((k * p["k_k"]).view(heads, 64), dim=-1)
            k = (k * (1 + (rate - 1) * p["k_a"])).view(heads, 64)
            r, v = r.view(heads, 64), v.view(heads, 64)
            decay = torch.exp(-np.exp(-0.5) * torch.sigmoid(w)).view(heads, 1, 64)
            u = (S * -kappa[:, None, :]).sum(-1, keepdim=True)
            S = S * decay + u * (kappa * rate.view(heads, 64))[:, None, :] + v[:, :, None] * k[:, None, :]
            y = (S * r[:, None, :]).sum(-1)
            y = torch.nn.functional.layer_norm(y, (64,), eps=tm.HEAD_EPS).view(-1) * p["head_gamma"] + p["head_beta"]
            y = y + ((r * k * p["u"].view(heads, 64)).sum(-1, keepdim=True) * v).view(-1)
            outs.append(p["W_o"] @ (y * g))
            prev = h[t]
            t += 1
        lasts.append(prev)
        states.append(S)
    return full, torch.stack(outs), torch.stack(lasts), torch.stack(states)


def near(got, want, bound, what):
    g, w = got.detach().double().cpu(), want.detach()
    assert g.shape == w.shape and torch.isfinite(g).all(), what
    err = float((g - w).norm() / w.norm())
    assert err <= bound, (what, err, bound)


def inputs(width, lens, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    n, t = len(lens), sum(lens)
    x, d, sh = (torch.randn(m, width, generator=gen).to(dtype) for m in (t, t, n))
    st = torch.randn(n, width // 64, 64, 64, generator=gen) * 0.3
    return x, d, sh, st


@pytest.mark.parametrize("width", [128, 640])
@pytest.mark.parametrize("lens", [[1, 1, 1], [3, 0, 21, 1, 40]], ids=str)
def test_served_against_float64(width, lens):
    say("serve", width, lens)
    layer = tm.TimeMix(width, rank=16, seed=3).quantize()
    p = {q: z.detach().double().cpu() for q, z in layer.params.items()}
    for q in "rkvo":
        codes = quant.quantize(p["W_" + q].float().numpy(), quant.W4_SYM, 64)
        p["W_" + q] = torch.from_numpy(np.asarray(quant.dequant(quant.W4_SYM, codes, 64), dtype=np.float64))
    x, d, sh, st = inputs(width, lens, torch.float16, 5)
    slots = torch.randperm(len(lens) + 2, generator=torch.Generator().manual_seed(1))[:len(lens)]
    shift, state = layer.states(len(lens) + 2)
    shift[slots.cuda()], state[slots.cuda()] = sh.cuda(), st.cuda()
    full, out = layer.serve(x.cuda(), d.cuda(), tm.offsets(lens), shift, state, slots.int().cuda())
    torch.cuda.synchronize()
    want = plain(p, x.double(), d.double(), lens, sh.double(), st.double(), width)
    u = U[torch.float16]
    near(full, want[0], u, "x'")
    near(out, want[1], 32 * u, "out")
    near(shift[slots.cuda()], want[2], 32 * u, "shift")
    near(state[slots.cuda()], want[3], 32 * u, "state")


def test_prompts_and_decode_in_parts():
    """Prompts, then token by token with slots in another order: as in one go."""
    width, lens, more = 256, [5, 40, 1], 6
    say("serve in parts")
    layer = tm.TimeMix(width, rank=16, seed=4).quantize()
    total = [m + more for m in lens]
    x, d, _, _ = inputs(width, total, torch.float16, 6)
    begin = np.concatenate([[0], np.cumsum(total)])
    shift, state = layer.states(3)
    slots = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    _, want = layer.serve(x.cuda(), d.cuda(), tm.offsets(total), shift, state, slots)
    shift2, state2 = layer.states(3)
    rows = np.concatenate([np.arange(b, b + m) for b, m in zip(begin, lens)])
    got = torch.empty_like(want)
    got[rows] = layer.serve(x[rows].cuda(), d[rows].cuda(), tm.offsets(lens), shift2, state2, slots)[1]
    order = [1, 2, 0]
    for i in range(more):
        rows = np.array([begin[s] + lens[s] + i for s in order])
        got[rows] = layer.serve(x[rows].cuda(), d[rows].cuda(), tm.offsets([1] * 3), shift2, state2, slots[order].contiguous())[1]
    torch.cuda.synchronize()
    u = U[torch.float16]
    for a, b, what in ((got, want, "out"), (shift2, shift, "shift"), (state2, state, "state")):
        near(a, b.double().cpu(), 32 * u, what)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
def test_gradients_against_float64(dtype):
    width, lens = 128, [19, 1, 0, 44]
    say("gradients", dtype)
    layer = tm.TimeMix(width, rank=16, dtype=dtype, seed=7)
    x, d, sh, st = inputs(width, lens, dtype, 8)
    gen = torch.Generator().manual_seed(9)
    weights = [torch.randn(*s, generator=gen) * f for s, f in
               (((64, width), 0.3), ((64, width), 1.0), ((4, width), 0.5), ((4, 2, 64, 64), 0.1))]
    for z in layer.params.values():
        z.requires_grad_(True)
    dev = [z.cuda().requires_grad_(True) for z in (x, d, sh, st)]
    outs = layer.train(dev[0], dev[1], tm.offsets(lens), dev[2], dev[3])
    sum((o.float() * w.cuda()).sum() for o, w in zip(outs, weights)).backward()
    p = {q: z.detach().double().cpu().requires_grad_(True) for q, z in layer.params.items()}
    ref = [z.double().requires_grad_(True) for z in (x, d, sh, st)]
    want = plain(p, ref[0], ref[1], lens, ref[2], ref[3], width)
    sum((o * w.double()).sum() for o, w in zip(want, weights)).backward()
    u = U[dtype]
    for o, w, what in zip(outs, want, ("x'", "out", "shift", "state")):
        near(o, w, 32 * u, what)
    for q in p:
        near(layer.params[q].grad, p[q].grad, 64 * u, "d" + q)
    for o, w, what in zip(dev, ref, ("dx", "ddelta", "dshift", "dstate")):
        near(o.grad, w.grad, 64 * u, what)


def test_command(capsys):
    say("the command")
    capsys.readouterr()
    assert tm.main(["--width", "256", "--prompts", "5,37", "--tokens", "3", "--train", "100"]) == 0
    lines = capsys.readouterr().out.splitlines()
    assert len(lines) == 5 and lines[0].startswith("prompts 5,37") and "decode, 2 sequences" in lines[1]
    loss = [float(z.rsplit(" ", 1)[1]) for z in lines[2:]]
    assert loss[2] < loss[0]
