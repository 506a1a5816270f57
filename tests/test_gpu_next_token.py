"""A model's end (gemm_rwkv_amd/next_token.py), the norm that leaves 8-bit rows,
the block product and the draw together, against the 64-bit oracle; and behind a
time-mixing layer that continues its own tokens, eagerly and replayed from a
graph.

Each stage is held to the oracle of what the one before it left: the logits to
the product of the codes (k * 2^-24 of sum |x w|, fp32 sums of exact products),
the tokens to the draw from the logits (equal), the codes to the norm, to within
what an h in fp32 would need (the kernel's is fp64): 2^-17 of S = |n gamma| + |gamma|
mean|x| / rms + |beta|; a code's value half a step more, 2^-4 of h or 2^-10 of the scale.
"""

import numpy as np
import pytest
import torch

from gemm_rwkv_amd import next_token as nx, rq, time_mix as tm
from gpu_helpers import say
from oracle import codecs, next_token as nt, quant, ref

pytestmark = pytest.mark.gpu

KINDS = {None: nt.NONE, "rms": nt.RMS, "layer": nt.LAYER}


def rows(seed, m, c, dtype):
    g = np.random.default_rng(seed)
    x = g.standard_normal((m, c))
    x[:, c // 3] *= 20.0
    return torch.from_numpy(x).to("cuda", dtype)


def filters(seed, m):
    """One row of each kind: no filter, greedy, top_k, top_p, min_p and all."""
    g = np.random.default_rng(seed)
    kind = np.arange(m) % 6

    def f32(a):
        return torch.from_numpy(np.asarray(a, dtype=np.float32)).cuda()
    return dict(temperature=f32(np.where(kind == 1, 0.0, 0.8)),
                top_k=torch.from_numpy(np.where((kind == 2) | (kind == 5), 20, 0).astype(np.int32)).cuda(),
                top_p=f32(np.where((kind == 3) | (kind == 5), 0.9, 1.0)), min_p=f32(np.where(kind >= 4, 0.02, 0.0)),
                u=f32(g.random(m)))


def check_tokens(token, logprob, logits, how):
    how = {q: v.cpu().numpy() for q, v in how.items()}
    z = logits.double().cpu().numpy()
    for i in range(len(z)):
        want, lp = nt.sample(z[i], **{q: float(v[i]) if q != "top_k" else int(v[i]) for q, v in how.items()})
        assert int(token[i]) == want, i
        assert abs(float(logprob[i]) - lp) <= 1e-6 + 2.0 ** -23 * abs(lp), i


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("m,width,vocab,norm", [(1, 128, 100, "layer"), (7, 640, 1003, "rms"), (33, 2048, 5001, "layer"),
                                                 (6, 1152, 8, None), (300, 256, 777, "rms")])
def test_head_against_float64(m, width, vocab, norm, dtype):
    say("head", m, width, vocab, norm, dtype)
    head = nx.Head(width, vocab, norm=norm, seed=m).quantize()
    x, delta, how = rows(m, m, width, dtype), rows(m + 1, m, width, dtype), filters(m, m)
    # the codes
    p = {q: v.double().cpu().numpy() for q, v in head.params.items()}
    full, codes, scales = nx.norm_quantize(x, delta, head.params["gamma"], head.params["beta"], norm)
    sum64 = x.double().cpu().numpy() + delta.double().cpu().numpy()
    assert torch.equal(full, (x.float() + delta.float()).to(dtype))
    h = nt.normed(sum64, KINDS[norm], p["gamma"], p["beta"], tm.NORM_EPS)
    n = nt.normed(sum64, KINDS[norm], None, None, tm.NORM_EPS)
    mean = np.abs(sum64).mean(-1, keepdims=True) / np.sqrt((sum64 ** 2).mean(-1, keepdims=True)) if norm else 0.0
    S = np.abs(n * p["gamma"]) + np.abs(p["gamma"]) * mean + np.abs(p["beta"])
    xq, sx = codes.cpu().numpy(), scales.cpu().numpy()
    step = np.exp2(sx[:, :width // 128].astype(float) - 127).repeat(128, 1)
    assert not sx[:, width // 128:].any()
    err = np.abs(codecs.e4m3_decode(xq) * step - h)
    assert (err <= np.maximum(2.0 ** -4 * np.abs(h), 2.0 ** -10 * step) + 2.0 ** -17 * S * (1 + 2.0 ** -4)).all()
    # the weight, the logits, the tokens
    wq, sw = nt.quantize_weight(head.params["W"].cpu().numpy())
    q = head.quantized
    assert np.array_equal(q.codes.cpu().numpy()[:wq.size].reshape(wq.shape), wq)
    assert np.array_equal(q.scales.cpu().numpy()[:sw.size].reshape(sw.shape), sw)
    again, logits = head.logits(x, delta)
    assert torch.equal(again, full) and logits.shape == (m, vocab) and logits.dtype == torch.float32
    a, b = nt.values(xq, sx, 1), nt.values(wq, sw, 128)
    err = np.abs(logits.double().cpu().numpy() - a @ b.T)
    assert (err <= width * 2.0 ** -24 * (np.abs(a) @ np.abs(b).T) + 1e-30).all()
    token, logprob = head.next(x, delta, **how)
    check_tokens(token, logprob, logits, how)


def test_one_scale_a_row_for_the_other_products():
    """The same norm in front of the products with a scale per row and channel."""
    m, c, n = 40, 512, 256
    g = np.random.default_rng(2)
    x, gamma = rows(3, m, c, torch.float16), torch.from_numpy(1 + 0.1 * g.standard_normal(c)).float().cuda()
    w = (g.standard_normal((n, c)) * c ** -0.5).astype(np.float32)
    for fmt, kind, product in ((rq.RQ_FP8_E4M3_CH, "fp8", rq.rq_gemm_fp8), (rq.RQ_I8_CH, "int8", rq.rq_gemm_int8)):
        full, codes, scales = nx.norm_quantize(x, gamma=gamma, norm="rms", fmt=fmt)
        assert full is x and scales.shape == (m,)
        y = torch.empty(m, n, dtype=torch.float16, device="cuda")
        product(codes, scales, m, rq.quantize(torch.from_numpy(w).cuda(), fmt), y, n)
        want, bound = ref.w8a8_ref(codes.cpu().numpy().view(np.int8 if kind == "int8" else np.uint8), scales.cpu().numpy(), kind, fmt,
                                   quant.quantize_rows(w, kind))
        ok, info = ref.compare(y.cpu().numpy(), want, bound)
        assert ok, (kind, info)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32], ids=["f16", "bf16", "f32"])
def test_sample_takes_any_strides(dtype):
    """Rows that are packed oddly, transposed, expanded, behind an offset or cut
    from a longer matrix draw what their copies draw."""
    g = np.random.default_rng(9)
    z = torch.from_numpy(g.standard_normal((12, 1003)) * 2).to("cuda", dtype)
    views = [z, z.t().contiguous().t(), z[3:4].expand(12, 1003), z.flatten()[5:5 + 11 * 1000].view(11, 1000), z[:, 100:900], z[::2],
             z[4:5, 3:]]
    for v in views:
        how = filters(4, len(v))
        token, logprob = nx.sample(v, **how)
        check_tokens(token, logprob, v, how)


def test_empty_batches():
    head = nx.Head(128, 40).quantize()
    x = torch.zeros(0, 128, dtype=torch.float16, device="cuda")
    full, logits = head.logits(x, x)
    assert full.shape == (0, 128) and logits.shape == (0, 40)
    token, logprob = head.next(x, u=0.5)
    assert token.shape == (0,) and token.dtype == torch.int32 and logprob.shape == (0,)


def test_numbers_and_generator():
    """A number stands for every row; without u a generator's seed fixes the draw."""
    z = rows(1, 20, 500, torch.float16)
    want = nx.sample(z, temperature=torch.full((20,), 0.7).cuda(), top_k=torch.full((20,), 9, dtype=torch.int32).cuda(),
                     u=torch.full((20,), 0.4).cuda())
    got = nx.sample(z, temperature=0.7, top_k=9, u=0.4)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    a, b = (nx.sample(z, generator=torch.Generator("cuda").manual_seed(5))[0] for _ in range(2))
    assert torch.equal(a, b)
    u = torch.rand(20, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    assert torch.equal(a, nx.sample(z, u=u)[0])


def decoder(n, width=256, vocab=2003):
    layer, head = tm.TimeMix(width, rank=16, seed=1).quantize(), nx.Head(width, vocab, seed=2).quantize()
    embed = rows(7, vocab, width, torch.float16)
    slots, one = torch.arange(n, dtype=torch.int32, device="cuda"), tm.offsets([1] * n)
    return layer, head, embed, slots, one


def test_decodes_behind_a_layer_eagerly_and_replayed():
    """Three sequences continue their own tokens for eight steps; the same steps
    replayed from one captured graph, with eager work between, leave the same
    tokens; a second stream's sequences in between keep out of them."""
    n, steps = 3, 8
    layer, head, embed, slots, one = decoder(n)
    us = torch.rand(steps, n, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    how = dict(temperature=torch.full((n,), 0.9).cuda(), top_k=torch.tensor([0, 40, 0], dtype=torch.int32).cuda(),
               top_p=torch.tensor([1.0, 0.95, 0.8]).cuda(), min_p=torch.tensor([0.0, 0.0, 0.01]).cuda())
    first = torch.tensor([5, 0, 2002], dtype=torch.int32, device="cuda")

    def step(token, state, u, ws):
        x, delta = layer.serve(embed[token.long()], None, one, *state, slots, ws=ws)
        _, logits = head.logits(x, delta)
        return nx.sample(logits, u=u, **how) + (logits,)

    ws = torch.zeros(rq.rq_workspace_bytes(), dtype=torch.uint8, device="cuda")
    state, token, want = layer.states(n), first, []
    for i in range(steps):
        token, logprob, logits = step(token, state, us[i], ws)
        check_tokens(token, logprob, logits, dict(how, u=us[i]))
        want.append(token.tolist())

    state, token, u = layer.states(n), first.clone(), us[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(token, layer.states(n), u, ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, logprob, logits = step(token, state, u, ws)
        token.copy_(out)
    other, ws2, got = layer.states(n), torch.zeros_like(ws), []
    torch.cuda.synchronize()
    for i in range(steps):
        u.copy_(us[i])
        graph.replay()
        with torch.cuda.stream(side):
            step(first, other, us[0], ws2)
        got.append(token.tolist())
        torch.cuda.synchronize()
    assert got == want


def test_batched_rows_draw_what_single_ones_do():
    """A row's token and its probability do not depend on the rows beside it."""
    head = nx.Head(384, 1500, seed=4).quantize()
    x, how = rows(8, 18, 384, torch.float16), filters(5, 18)
    _, logits = head.logits(x)
    token, logprob = nx.sample(logits, **how)
    for i in range(18):
        t, lp = nx.sample(logits[i:i + 1], **{q: v[i:i + 1] for q, v in how.items()})
        assert t.item() == token[i].item() and lp.item() == logprob[i].item()


def test_command_runs(capsys):
    assert nx.main(["--width", "256", "--vocab", "1003", "--prompts", "3,17", "--tokens", "4", "--top-k", "30", "--top-p", "0.9"]) == 0
    said = capsys.readouterr().out.splitlines()
    assert len(said) == 3 and all(0 <= int(t) < 1003 for row in said[1:] for t in row.split())


def test_far_rows():
    """Rows whose logits, or codes, start past 2^31 elements and 2^32 bytes."""
    say("far rows: logits")
    base, reps = 440, 75
    z = torch.empty(base * reps, 65544, dtype=torch.float16, device="cuda")
    part = rows(2, base, 65544, torch.float16)
    for i in range(reps):
        z[i * base:(i + 1) * base] = part
    u = torch.rand(base, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    want = nx.sample(part[:, :65536], temperature=0.8, top_k=30, u=u)
    got = nx.sample(z[:, :65536], temperature=0.8, top_k=30, u=u.repeat(reps))
    assert torch.equal(got[0].view(reps, base), want[0].expand(reps, base))
    assert torch.equal(got[1].view(reps, base), want[1].expand(reps, base))
    del z, part, got
    say("far rows: codes")
    base, reps = 1000, 263
    x = rows(3, base, 8192, torch.float16)
    _, codes, scales = nx.norm_quantize(x)
    _, far, fscales = nx.norm_quantize(x.repeat(reps, 1))
    for i in (0, 131, 262):
        assert torch.equal(far[i * base:(i + 1) * base], codes) and torch.equal(fscales[i * base:(i + 1) * base], scales)


def test_calls_at_once_on_two_streams():
    """Each stream's tokens are those of its rows alone."""
    head = nx.Head(512, 4001, seed=6).quantize()
    xs = [rows(s, 40, 512, torch.float16) for s in (1, 2)]
    hows = [filters(s, 40) for s in (1, 2)]
    want = [head.next(x, **how) for x, how in zip(xs, hows)]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(head.next(xs[i], **hows[i]))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(a, b) for pair in g for a, b in zip(pair, w))
