"""From a model's last residual to its next token on librq, in 8 bits.

    python -m gemm_rwkv_amd.next_token                     # width 2048, vocabulary 65536: prompts, then decode
    python -m gemm_rwkv_amd.next_token --width 768 --vocab 50277 --prompts 5,37 --tokens 32 --top-k 50 --top-p 0.9

``norm_quantize``, ``block_product`` and ``sample`` are the library's operators as
torch functions; ``Head`` runs them one after the other: the final norm, straight
to e4m3 codes with a power of two per 128 columns, the product with the
vocabulary's rows, whose logits are fp32, and the draw.  The command puts a head
behind a time-mixing layer and lets it continue its own tokens.

Like the rest of the quantized path they serve and do not train: inputs that
require gradients are refused where autograd records.  Types, shapes that do not
fit and tensors elsewhere than on the current GPU are refused as in ``time_mix``
(TypeError, ValueError); the library refuses sizes past its own (``rq.RqError``).
"""

import argparse
import sys

import torch

from . import rq
from .time_mix import _CODE, _dense, _on_gpu, _rows, _same, NORM_EPS, TimeMix, offsets

NORMS = {None: rq.RQ_NORM_NONE, "rms": rq.RQ_NORM_RMS, "layer": rq.RQ_NORM_LAYER}
_CODE_Y = {**_CODE, torch.float32: rq.RQ_F32}
_ONE_PER_ROW = (rq.RQ_FP8_E4M3_CH, rq.RQ_I8_CH)


def _served(*ts):
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in ts):
        raise RuntimeError("8-bit codes have no gradient: call this under torch.no_grad()")


def norm_quantize(x, delta=None, gamma=None, beta=None, norm="layer", eps=NORM_EPS, fmt=rq.RQ_FP8_E4M3_B128):
    """(x + delta, codes uint8 [rows][width], scales) of the norm ("layer",
    "rms" or None) of x + delta.  Scales are uint8 [rows][block_scale_row(width)]
    in rq.RQ_FP8_E4M3_B128, fp32 [rows] in rq.RQ_FP8_E4M3_CH and rq.RQ_I8_CH.
    (rq.rq_norm_quantize also takes a factor of delta, and writes the sum in place.)"""
    _rows(x=x, delta=delta)
    (m, c) = x.shape
    if norm not in NORMS:
        raise ValueError("norm is %r, not one of %s" % (norm, list(NORMS)))
    if fmt != rq.RQ_FP8_E4M3_B128 and fmt not in _ONE_PER_ROW:
        raise ValueError("format %r is none that rows are quantized to" % (fmt,))
    for name, t in (("gamma", gamma), ("beta", beta)):
        if t is not None:
            _same(name, t, torch.float32, (c,))
    _served(x, delta, gamma, beta)
    _on_gpu(x, delta, gamma, beta)
    x, delta, gamma, beta = _dense(x, delta, gamma, beta)
    full = x if delta is None else torch.empty_like(x)
    codes = torch.empty(m, c, dtype=torch.uint8, device=x.device)
    if fmt == rq.RQ_FP8_E4M3_B128:
        scales = torch.empty(m, rq.block_scale_row(c), dtype=torch.uint8, device=x.device)
    else:
        scales = torch.empty(m, dtype=torch.float32, device=x.device)
    if m:
        rq.rq_norm_quantize(_CODE[x.dtype], NORMS[norm], x, delta, 1.0, m, c, c, gamma, beta, eps, fmt, None if delta is None else full,
                            codes, scales)
    return full, codes, scales


def block_product(codes, scales, w, dtype=torch.float16):
    """[rows][w.n] in `dtype` (float16, bfloat16 or float32), the product of
    norm_quantize's codes and scales with the RQ_FP8_E4M3_B128 weight w.  Its
    rows lie a multiple of 8 elements apart.  Sums are fp32 where dtype is float32
    or there are at most 16 rows; else see rq_gemm_fp8_block in rq.h."""
    if dtype not in _CODE_Y:
        raise TypeError("dtype is %s, not float16, bfloat16 or float32" % dtype)
    if w.format != rq.RQ_FP8_E4M3_B128:
        raise ValueError("w is of format %d, not rq.RQ_FP8_E4M3_B128" % w.format)
    if codes.dim() != 2:
        raise ValueError("codes has shape %s, not [rows][width]" % list(codes.shape))
    m = codes.shape[0]
    _same("codes", codes, torch.uint8, (m, w.k))
    _same("scales", scales, torch.uint8, (m, rq.block_scale_row(w.k)))
    _on_gpu(codes, scales, w.codes, w.scales)
    codes, scales = _dense(codes, scales)
    y = torch.empty(m, -(-w.n // 8) * 8, dtype=dtype, device=codes.device)
    if m and w.n:
        rq.rq_gemm_fp8_block(codes, scales, m, w, _CODE_Y[dtype], y, y.shape[1])
    return y[:, :w.n]


def _per_row(name, v, rows, dtype, device):
    """One value a row: a number, or a tensor of `dtype`; None stays."""
    if v is None:
        return None
    if not torch.is_tensor(v):
        return torch.full((rows,), v, dtype=dtype, device=device)
    _same(name, v, dtype, (rows,))
    return v


def sample(logits, temperature=None, top_k=None, top_p=None, min_p=None, u=None, generator=None):
    """(tokens int32 [rows], the logarithms of their probabilities fp32 [rows])
    of logits [rows][vocab] in fp16, bf16 or fp32.  The filters (rq.h,
    rq_sample) and u, the uniform numbers in [0, 1) that decide, are numbers or
    tensors with one value a row (top_k int32, the others fp32); without u it is
    drawn from `generator`.  A row with nothing to draw gets token -1.

    A number is written to a tensor by a launch of its own, some 4 us of each
    call, and so is u: one row of 65536 by three filters takes 15.5 us a call with
    tensors, 26 with numbers, 31 with u drawn as well.  Loops keep tensors."""
    if logits.dtype not in _CODE_Y:
        raise TypeError("logits is %s, not float16, bfloat16 or float32" % logits.dtype)
    if logits.dim() != 2 or logits.shape[1] == 0:
        raise ValueError("logits has shape %s, not [rows][vocab]" % list(logits.shape))
    _served(logits)
    rows, vocab = logits.shape
    dev = logits.device
    temperature, top_p, min_p, u = (_per_row(name, v, rows, torch.float32, dev) for name, v in
                                    (("temperature", temperature), ("top_p", top_p), ("min_p", min_p), ("u", u)))
    top_k = _per_row("top_k", top_k, rows, torch.int32, dev)
    _on_gpu(logits, temperature, top_k, top_p, min_p, u)
    if u is None:
        u = torch.rand(rows, device=dev, generator=generator)
    temperature, top_k, top_p, min_p, u = _dense(temperature, top_k, top_p, min_p, u)
    ld = logits.stride(0) if rows > 1 else -(-vocab // 8) * 8
    if logits.stride(1) != 1 or ld < vocab or ld % 8 or logits.data_ptr() % 16:
        ld = -(-vocab // 8) * 8
        padded = torch.empty(rows, ld, dtype=logits.dtype, device=dev)
        padded[:, :vocab] = logits
        logits = padded
    token = torch.empty(rows, dtype=torch.int32, device=dev)
    logprob = torch.empty(rows, dtype=torch.float32, device=dev)
    if rows:
        rq.rq_sample(_CODE_Y[logits.dtype], logits, rows, vocab, ld, temperature, top_k, top_p, min_p, u, token, logprob)
    return token, logprob


class Head:
    """A model's end with random weights: gamma and beta [width] (fp32) of its
    final norm, W [vocab][width] of its logits.  All of them may be replaced
    before quantize()."""

    def __init__(self, width, vocab, norm="layer", seed=0, device="cuda"):
        if width % 128:
            raise ValueError("width must be a multiple of 128 (a scale per 128 columns)")
        if norm not in NORMS:
            raise ValueError("norm is %r, not one of %s" % (norm, list(NORMS)))
        self.width, self.vocab, self.norm = width, vocab, norm
        gen = torch.Generator().manual_seed(seed)
        p = {"gamma": 1 + 0.1 * torch.randn(width, generator=gen), "beta": 0.1 * torch.randn(width, generator=gen),
             "W": torch.randn(vocab, width, generator=gen) * 2 * width ** -0.5}
        self.params = {q: x.to(device) for q, x in p.items()}
        self.quantized = None

    def quantize(self):
        """W as e4m3 codes with a power of two per 128 x 128."""
        self.quantized = rq.quantize(self.params["W"].float(), rq.RQ_FP8_E4M3_B128)
        return self

    @torch.no_grad()
    def logits(self, x, delta=None, dtype=torch.float32):
        """(x + delta, logits [rows][vocab]) of residual rows x and the last
        layer's output delta."""
        if self.quantized is None:
            raise RuntimeError("call quantize() first")
        p = self.params
        full, codes, scales = norm_quantize(x, delta, p["gamma"], p["beta"], self.norm)
        return full, block_product(codes, scales, self.quantized, dtype)

    @torch.no_grad()
    def next(self, x, delta=None, **how):
        """(tokens, log-probabilities) drawn for residual rows; how: sample()'s
        arguments."""
        return sample(self.logits(x, delta)[1], **how)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--vocab", type=int, default=65536)
    ap.add_argument("--prompts", default="37,512,5,200", help="lengths of the prompts, served as one batch")
    ap.add_argument("--tokens", type=int, default=16, help="tokens drawn for each of them")
    ap.add_argument("--temperature", type=float, default=1.0)
    ap.add_argument("--top-k", type=int, default=0, help="0: all")
    ap.add_argument("--top-p", type=float, default=1.0)
    ap.add_argument("--min-p", type=float, default=0.0)
    ap.add_argument("--seed", type=int, default=0)
    args = ap.parse_args(argv)
    lens = [int(n) for n in args.prompts.split(",")]
    if min(lens) < 1:
        ap.error("a prompt has at least one token")
    n = len(lens)
    layer, head = TimeMix(args.width).quantize(), Head(args.width, args.vocab).quantize()
    gen = torch.Generator("cuda").manual_seed(args.seed)
    embed = torch.randn(args.vocab, args.width, device="cuda", generator=gen).half()
    how = {q: torch.full((n,), v, device="cuda") for q, v in
           (("temperature", args.temperature), ("top_p", args.top_p), ("min_p", args.min_p))}
    how.update(top_k=torch.full((n,), args.top_k, dtype=torch.int32, device="cuda"), generator=gen)
    shift, state = layer.states(n)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    cu, one = offsets(lens), offsets([1] * n)
    tokens = torch.randint(args.vocab, (sum(lens),), device="cuda", generator=gen)
    x, delta = layer.serve(embed[tokens], None, cu, shift, state, slots)
    ends = cu[1:].long() - 1
    x, delta = x[ends], delta[ends]
    said = []
    for i in range(args.tokens):
        start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        token, logprob = head.next(x, delta, **how)
        stop.record()
        said.append(token)
        x, delta = layer.serve(embed[token.long()], None, one, shift, state, slots)
        torch.cuda.synchronize()
    if said:
        print("prompts %s, a head of %d x %d: %.0f us the last draw of %d, mean log-probability %.3f"
              % (args.prompts, args.vocab, args.width, 1e3 * start.elapsed_time(stop), len(said), logprob.mean()))
        for row in torch.stack(said, 1).tolist():
            print(" ".join(map(str, row)))
    return 0


if __name__ == "__main__":
    sys.exit(main())
