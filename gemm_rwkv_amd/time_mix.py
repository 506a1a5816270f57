"""One RWKV-7 time-mixing layer on librq, for serving and for training.

    python -m gemm_rwkv_amd.time_mix                       # width 2048: prompts, decode, a training step
    python -m gemm_rwkv_amd.time_mix --width 768 --prompts 5,37,300 --tokens 32

``shift_norm``, ``time_mix`` and ``head_gate`` are the library's operators as
differentiable torch functions over rows [tokens][width] of fp16 or bf16;
parameters and states are fp32, offsets int32.  Other types, shapes that do not
fit and tensors elsewhere than on the current GPU are refused (TypeError,
ValueError).  They are differentiable once: a gradient of their gradient is an
error.  ``TimeMix`` is the layer: ``train``
runs it on its dense weights under autograd, ``serve`` on group-wise int4
R/K/V/O weights, continuing the sequences whose states lie in slots (prompts
of any lengths and single tokens, in one batch or in turn).

The layer, with x' = x + delta and six mixtures m_i of its shifted norm:
    r, k, v = W_r m_0, W_k m_2, W_v m_3
    w       = w0 + tanh(m_1 A_w) B_w                  (raw decay)
    rate    = sigmoid(a0 + m_4 A_a B_a)
    g       = sigmoid(m_5 A_g) B_g
    kappa   = k k_k, of unit length in each head;   k' = k (1 + (rate - 1) k_a)
    y       = the state recurrence of r, w, k', v, -kappa, kappa rate
    out     = W_o head_gate(y, r, k', v, g)
It is a model's first layer: RWKV-7's later ones also mix the first layer's v
into theirs, which is not done here.
"""

import argparse
import sys

import torch
import torch.nn.functional as F
from torch.autograd.function import once_differentiable

from . import rq

HEAD = 64
MIXTURES = "rwkvag"
NORM_EPS, HEAD_EPS = 1e-5, 64e-5
_CODE = {torch.float16: rq.RQ_F16, torch.bfloat16: rq.RQ_BF16}


def _rows(**rows):
    """Refuses rows that are not of one 16-bit type and one shape [tokens][width]."""
    (name, x), *others = rows.items()
    if x.dtype not in _CODE:
        raise TypeError("%s is %s, not float16 or bfloat16" % (name, x.dtype))
    if x.dim() != 2:
        raise ValueError("%s has shape %s, not [tokens][width]" % (name, list(x.shape)))
    for other, t in others:
        if t is not None:
            _same(other, t, x.dtype, x.shape)


def _same(name, t, dtype, shape):
    if t.dtype != dtype:
        raise TypeError("%s is %s, not %s" % (name, t.dtype, dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, not %s" % (name, list(t.shape), list(shape)))


def _heads(x):
    if x.shape[1] % HEAD:
        raise ValueError("a width of %d is not in heads of %d" % (x.shape[1], HEAD))
    return x.shape[1] // HEAD


def _sequences(cu):
    """How many sequences the offsets cu are of."""
    if cu.dtype != torch.int32:
        raise TypeError("cu is %s, not torch.int32" % cu.dtype)
    if cu.dim() != 1 or cu.numel() == 0:
        raise ValueError("cu has shape %s, not [sequences + 1]" % list(cu.shape))
    return cu.numel() - 1


def _on_gpu(*ts):
    """The library's calls go to the current device."""
    for t in ts:
        if t is not None and not (t.is_cuda and t.device.index == torch.cuda.current_device()):
            raise ValueError("a tensor on %s; all have to be on the current GPU" % t.device)


def _dense(*ts):
    return [t if t is None else t.contiguous() for t in ts]


def _workspace(x):
    """Memory for one call: of torch's allocator on the current stream, so that
    calls on other streams and threads, whose kernels may run at the same time,
    have other memory.  (These entries leave its split counters alone.)"""
    return torch.empty(rq.rq_workspace_bytes(), dtype=torch.uint8, device=x.device)


class _ShiftNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, delta, mu, gamma, beta, shift, cu):
        _rows(x=x, delta=delta)
        (t, c), n = x.shape, _sequences(cu)
        if mu.dim() != 2:
            raise ValueError("mu has shape %s, not [mixtures][width]" % list(mu.shape))
        _same("mu", mu, torch.float32, (mu.shape[0], c))
        _same("gamma", gamma, torch.float32, (c,))
        _same("beta", beta, torch.float32, (c,))
        if shift is not None:
            _same("shift", shift, x.dtype, (n, c))
        _on_gpu(x, delta, mu, gamma, beta, shift, cu)
        x, delta, mu, gamma, beta, shift, cu = _dense(x, delta, mu, gamma, beta, shift, cu)
        full = x if delta is None else torch.empty_like(x)
        out = torch.empty(mu.shape[0], t, c, dtype=x.dtype, device=x.device)
        last = torch.empty(n, c, dtype=x.dtype, device=x.device)
        rq.rq_shift_norm(_CODE[x.dtype], x, delta, 1.0, t, c, c, cu, n, gamma, beta, NORM_EPS, mu, mu.shape[0], shift, last, None, n,
                         None if delta is None else full, out, c)
        ctx.save_for_backward(full, mu, gamma, beta, shift, cu)
        ctx.with_delta = delta is not None
        ctx.set_materialize_grads(False)
        return (full if ctx.with_delta else x.view_as(x)), out, last

    @staticmethod
    @once_differentiable
    def backward(ctx, dfull, dout, dlast):
        x, mu, gamma, beta, shift, cu = ctx.saved_tensors
        (t, c), n = x.shape, cu.numel() - 1
        dfull, dout, dlast = _dense(dfull, dout, dlast)
        if dout is None:
            dout = torch.zeros(mu.shape[0], t, c, dtype=x.dtype, device=x.device)
        dx = torch.empty_like(x)
        dshift = None if shift is None else torch.empty_like(shift)
        dgamma, dbeta, dmu = torch.empty_like(gamma), torch.empty_like(beta), torch.empty_like(mu)
        rq.rq_shift_norm_backward(_CODE[x.dtype], x, 1.0, t, c, c, cu, n, gamma, beta, NORM_EPS, mu, mu.shape[0], shift, dout, c,
                                  dfull, dlast, dx, None, dshift, dgamma, dbeta, dmu, ws=_workspace(x))
        return dx, dx if ctx.with_delta else None, dmu, dgamma, dbeta, dshift, None


class _TimeMix(torch.autograd.Function):
    @staticmethod
    def forward(ctx, r, w, k, v, a, b, state, cu):
        _rows(r=r, w=w, k=k, v=v, a=a, b=b)
        (t, c), n = r.shape, _sequences(cu)
        if state is None:
            _heads(r)
        else:
            _same("state", state, torch.float32, (n, _heads(r), HEAD, HEAD))
        _on_gpu(r, w, k, v, a, b, state, cu)
        rows = _dense(r, w, k, v, a, b)
        state, cu = _dense(state, cu)
        y = torch.empty_like(rows[0])
        last = torch.empty(n, c // HEAD, HEAD, HEAD, dtype=torch.float32, device=r.device)
        rq.rq_time_mix(_CODE[r.dtype], *rows, t, c // HEAD, c, cu, n, state, last, None, n, y, c, ws=_workspace(y))
        ctx.save_for_backward(*rows, state, cu)
        ctx.set_materialize_grads(False)
        return y, last

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dlast):
        *rows, state, cu = ctx.saved_tensors
        (t, c), n = rows[0].shape, cu.numel() - 1
        dy, dlast = _dense(dy, dlast)
        if dy is None:
            dy = torch.zeros_like(rows[0])
        grads = [torch.empty_like(x) for x in rows]
        dstate = None if state is None else torch.empty_like(state)
        rq.rq_time_mix_backward(_CODE[dy.dtype], *rows, t, c // HEAD, c, cu, n, state, dy, dlast, *grads, dstate)
        return (*grads, dstate, None)


class _HeadGate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, r, k, v, g, gamma, beta, u):
        _rows(y=y, r=r, k=k, v=v, g=g)
        _heads(y)
        for name, param in (("gamma", gamma), ("beta", beta), ("u", u)):
            _same(name, param, torch.float32, y.shape[1:])
        _on_gpu(y, r, k, v, g, gamma, beta, u)
        rows = _dense(y, r, k, v, g)
        params = _dense(gamma, beta, u)
        t, c = y.shape
        out = torch.empty_like(rows[0])
        rq.rq_head_gate(_CODE[y.dtype], *rows, t, c // HEAD, c, params[0], params[1], HEAD_EPS, params[2], out, c)
        ctx.save_for_backward(*rows, *params)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        *rows, gamma, beta, u = ctx.saved_tensors
        t, c = dout.shape
        grads = [torch.empty_like(x) for x in rows]
        dparams = [torch.empty_like(x) for x in (gamma, beta, u)]
        rq.rq_head_gate_backward(_CODE[dout.dtype], *rows, t, c // HEAD, c, gamma, beta, HEAD_EPS, u, dout.contiguous(), *grads, *dparams,
                                 ws=_workspace(dout))
        return (*grads, *dparams)


def shift_norm(x, delta, mu, gamma, beta, cu, shift=None):
    """(x + delta, mixtures [nmix][tokens][width], last norm of each sequence
    [nseq][width]); delta and shift (the norm before each sequence) may be None."""
    return _ShiftNorm.apply(x, delta, mu, gamma, beta, shift, cu)


def time_mix(r, w, k, v, a, b, cu, state=None):
    """(y, states after [nseq][heads][64][64]) of the state recurrence."""
    return _TimeMix.apply(r, w, k, v, a, b, state, cu)


def head_gate(y, r, k, v, g, gamma, beta, u):
    """The norm of each head, the bonus and the gate."""
    return _HeadGate.apply(y, r, k, v, g, gamma, beta, u)


class TimeMix:
    """A time-mixing layer with random weights.  params: name -> tensor, the
    matrices of `dtype`, the vectors in fp32."""

    def __init__(self, width, rank=64, dtype=torch.float16, seed=0, device="cuda"):
        if width % 128:
            raise ValueError("width must be a multiple of 128 (int4 weights, heads of 64)")
        self.width, self.dtype, self.device = width, dtype, device
        gen = torch.Generator().manual_seed(seed)

        def draw(*shape, scale=1.0):
            return torch.randn(*shape, generator=gen) * scale

        p = {"W_" + q: draw(width, width, scale=width ** -0.5) for q in "rkvo"}
        for q in "wag":
            p["A_" + q] = draw(width, rank, scale=width ** -0.5)
            p["B_" + q] = draw(rank, width, scale=rank ** -0.5)
        p = {q: x.to(dtype) for q, x in p.items()}
        p.update(mu=torch.rand(len(MIXTURES), width, generator=gen), gamma=1 + draw(width, scale=0.1), beta=draw(width, scale=0.1),
                 w0=draw(width) - 2, a0=draw(width), k_k=1 + draw(width, scale=0.1), k_a=1 + draw(width, scale=0.1),
                 head_gamma=1 + draw(width, scale=0.1), head_beta=draw(width, scale=0.1), u=draw(width, scale=0.1))
        self.params = {q: x.to(device) for q, x in p.items()}
        self.quantized = None

    def quantize(self, group=64):
        """The four projections as int4 codes for serve()."""
        self.quantized = {q: rq.quantize(self.params["W_" + q].float(), rq.RQ_W4_SYM, group) for q in "rkvo"}
        return self

    def states(self, slots):
        """(shift, state) arrays of `slots` zeroed entries."""
        return (torch.zeros(slots, self.width, dtype=self.dtype, device=self.device),
                torch.zeros(slots, self.width // HEAD, HEAD, HEAD, device=self.device))

    def _inner(self, mixes, k):
        """Raw decay, gate, k', -kappa and kappa rate from the mixtures and k."""
        p = self.params
        w = p["w0"] + (torch.tanh(mixes[1] @ p["A_w"]) @ p["B_w"]).float()
        rate = torch.sigmoid(p["a0"] + (mixes[4] @ p["A_a"] @ p["B_a"]).float())
        g = torch.sigmoid(mixes[5] @ p["A_g"]) @ p["B_g"]
        kf = k.float()
        kappa = F.normalize((kf * p["k_k"]).view(-1, self.width // HEAD, HEAD), dim=-1).view(-1, self.width)
        bonus = kf * (1 + (rate - 1) * p["k_a"])
        return (x.to(self.dtype) for x in (w, g, bonus, -kappa, kappa * rate))

    def train(self, x, delta, cu, shift=None, state=None):
        """(x + delta, the layer's output, last norms, states after), all
        differentiable."""
        p = self.params
        full, mixes, last = shift_norm(x, delta, p["mu"], p["gamma"], p["beta"], cu, shift)
        r, k, v = (F.linear(mixes[i], p["W_" + q]) for i, q in ((0, "r"), (2, "k"), (3, "v")))
        w, g, k, a, b = self._inner(mixes, k)
        y, after = time_mix(r, w, k, v, a, b, cu, state)
        return full, F.linear(head_gate(y, r, k, v, g, p["head_gamma"], p["head_beta"], p["u"]), p["W_o"]), last, after

    def _product(self, x, q, ws):
        m, c = x.shape
        y = torch.empty_like(x)
        return (rq.rq_gemm_small_m if m <= 32 else rq.rq_gemm_w4)(x, m, c, self.quantized[q], y, c, ws=ws)

    @torch.no_grad()
    def serve(self, x, delta, cu, shift, state, slots, ws=None):
        """(x + delta, the layer's output) of sequences that continue the
        entries slots[i] of shift and state, which are updated in place.  ws:
        a workspace of rq.rq_workspace_bytes() bytes, zeroed once; calls that
        may run at the same time, on several streams, need one each (None: the
        binding's, which all calls without one share)."""
        if self.quantized is None:
            raise RuntimeError("call quantize() first")
        if self.dtype != torch.float16:
            raise TypeError("the quantized products take float16")
        _rows(x=x, delta=delta)
        p, n, heads, nslots = self.params, _sequences(cu), self.width // HEAD, shift.shape[0]
        _same("x", x, self.dtype, (x.shape[0], self.width))
        _same("shift", shift, self.dtype, (nslots, self.width))
        _same("state", state, torch.float32, (nslots, heads, HEAD, HEAD))
        if not (shift.is_contiguous() and state.is_contiguous()):
            raise ValueError("shift and state are updated in place and have to be contiguous")
        if slots is not None:
            _same("slots", slots, torch.int32, (n,))
        _on_gpu(x, delta, cu, shift, state, slots)
        m, c = x.shape
        x, delta, cu, slots = _dense(x, delta, cu, slots)
        full = x if delta is None else torch.empty_like(x)
        if m == 0:      # empty sequences: what the slots hold stays
            return full, torch.empty_like(x)
        mixes = torch.empty(len(MIXTURES), m, c, dtype=x.dtype, device=x.device)
        rq.rq_shift_norm(rq.RQ_F16, x, delta, 1.0, m, c, c, cu, n, p["gamma"], p["beta"], NORM_EPS, p["mu"], len(MIXTURES),
                         shift, shift, slots, nslots, None if delta is None else full, mixes, c)
        if m <= 32:
            r, k, v = (torch.empty_like(x) for _ in range(3))
            rq.rq_fused_rkv(mixes[0], mixes[2], mixes[3], m, c, *(self.quantized[q] for q in "rkv"), r, k, v, c, ws=ws)
        else:
            r, k, v = (self._product(mixes[i], q, ws) for i, q in ((0, "r"), (2, "k"), (3, "v")))
        w, g, k, a, b = self._inner(mixes, k)
        y = torch.empty_like(x)
        rq.rq_time_mix(rq.RQ_F16, r, w, k, v, a, b, m, heads, c, cu, n, state, state, slots, nslots, y, c, ws=ws)
        gated = torch.empty_like(x)
        rq.rq_head_gate(rq.RQ_F16, y, r, k, v, g, m, heads, c, p["head_gamma"], p["head_beta"], HEAD_EPS, p["u"], gated, c)
        return full, self._product(gated, "o", ws)


def offsets(lens, device="cuda"):
    """int32 device offsets of sequences of the given lengths."""
    return torch.tensor([0] + list(lens), device=device).cumsum(0).to(torch.int32)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--prompts", default="37,512,5,200", help="lengths of the prompts, served as one batch")
    ap.add_argument("--tokens", type=int, default=16, help="tokens decoded after them, one a call")
    ap.add_argument("--train", type=int, default=1024, help="tokens of the training step's sequence")
    args = ap.parse_args(argv)
    lens = [int(n) for n in args.prompts.split(",")]
    if min(lens) < 1:
        ap.error("a prompt has at least one token")
    n = len(lens)
    layer = TimeMix(args.width).quantize()
    shift, state = layer.states(n)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")

    def timed(f):
        start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        out = f()
        stop.record()
        torch.cuda.synchronize()
        return out, 1e3 * start.elapsed_time(stop)

    def rows(m):
        return torch.randn(m, args.width, device="cuda").half()

    x, cu = rows(sum(lens)), offsets(lens)
    layer.serve(x, None, cu, *layer.states(n), slots)                     # loads the kernels
    (_, out), us = timed(lambda: layer.serve(x, None, cu, shift, state, slots))
    print("prompts %s: %.0f us, output rms %.4f" % (args.prompts, us, out.float().pow(2).mean().sqrt()))
    x, delta = out[cu[1:].long() - 1], None
    one = offsets([1] * n)
    for i in range(args.tokens):
        (x, delta), us = timed(lambda: layer.serve(x, delta, one, shift, state, slots))
    if args.tokens:
        print("decode, %d sequences: %.0f us the last of %d tokens, output rms %.4f"
              % (n, us, args.tokens, delta.float().pow(2).mean().sqrt()))
    for q in layer.params.values():
        q.requires_grad_(True)
    x, want, cu = rows(args.train), rows(args.train), offsets([args.train])
    for step in range(3):
        def go():
            # the sum, not the mean, whose 16-bit gradients would vanish
            loss = (layer.train(x, None, cu)[1].float() - want.float()).pow(2).sum()
            loss.backward()
            return loss.item() / x.numel()
        loss, us = timed(go)
        print("training step %d on %d tokens: %.0f us, loss %.4f" % (step, args.train, us, loss))
        with torch.no_grad():
            for q in layer.params.values():
                # a step of 5% of the parameter's length down its gradient
                q -= (0.05 * q.float().norm() * F.normalize(q.grad.float().flatten(), dim=0).view_as(q)).to(q.dtype)
                q.grad = None
    return 0


if __name__ == "__main__":
    sys.exit(main())
