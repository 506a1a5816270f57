"""From a model's last residual to its next token in 8 bits, as this library's users call it: cases, inputs, plain forms
and 64-bit values.

Three operators, each with the form that prompts take and the one for single tokens:

* ``norm``: x' = x + alpha delta, RMS or layer norm (or none), and the row as e4m3 or int8 codes with one scale per row or
  one power of two per 128 columns;
* ``product``: y = x W^T of e4m3 codes, x with a scale per row and 128 k, W with one per 128 x 128;
* ``sample``: one token per row of logits by temperature, top-k, top-p and min-p from a given uniform number.

``run`` with ``own`` false computes them with elementary torch operations in fp32 (sampling, whose tokens change where a
sum passes a border, in fp64); with ``own`` true it makes the library's calls.  ``exact`` works in fp64, the sampling row by
row.
"""

import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
CODES = {"f16": 6, "bf16": 9, "f32": 10}            # the library's type codes
FORMATS = {"row8": 4, "rowi8": 5, "block8": 11}     # e4m3 per row, int8 per row, e4m3 per block of 128
NORMS = {"none": 0, "rms": 1, "layer": 2}
EPS = 1e-5
BLOCK = 128


# ------------------------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------------------------

def _norm(name, norm, rows, width, dtype, fmt, delta):
    c = {"op": "norm", "norm": norm, "rows": rows, "width": width, "dtype": dtype, "format": fmt, "delta": delta}
    return dict(c, name=name) if name else c


def _product(name, m, n, k, dtype):
    c = {"op": "product", "m": m, "n": n, "k": k, "dtype": dtype}
    return dict(c, name=name) if name else c


def _sample(name, rows, vocab, dtype, filters):
    c = {"op": "sample", "rows": rows, "vocab": vocab, "dtype": dtype, "filters": filters}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user's next token before the head, 1.5B model: nothing but latency
        _norm("norm decode 1", "layer", 1, 2048, "f16", "block8", True),
        # the same for a full decode batch of a 7.2B model, for the product with row scales
        _norm("norm decode 32", "rms", 32, 4096, "f16", "row8", True),
        # ragged prompts of the 2.9B model, 1021 tokens in all
        _norm("norm prompts 1021", "rms", 1021, 2560, "bf16", "block8", True),
        # a long prefill chunk of the 7.2B model
        _norm("norm prefill 8192", "layer", 8192, 4096, "f16", "block8", True),
        # a square projection of the 1.5B model for one token
        _product("product decode 1", 1, 2048, 2048, "f16"),
        # the head of the 7.2B model for a full decode batch, logits in fp32
        _product("product head 32", 32, 65536, 4096, "f32"),
        # channel mixing's key over ragged prompts, 2.9B model
        _product("product prompts 999", 999, 10240, 2560, "bf16"),
        # the same of the 7.2B model over a chunk of 1024 tokens
        _product("product prefill 1024", 1024, 16384, 4096, "f16"),
        # one user's token: the usual filters together
        _sample("sample decode 1", 1, 65536, "f16", "chat"),
        # a decode batch in which every request has filters of its own
        _sample("sample batch 32", 32, 65536, "f16", "mixed"),
        # many requests that only set a nucleus
        _sample("sample nucleus 128", 128, 65536, "f32", "nucleus"),
        # rollouts: plain draws by temperature for many rows, an odd vocabulary
        _sample("sample rollouts 509", 509, 50277, "bf16", "plain"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "product", "product", "sample"))
    if op == "norm":
        width = BLOCK * rng.randint(6, 64)
        rows = _log(rng, 1, 8192 * 4096 // width)
        return _norm("", rng.choice(("rms", "layer", "none")), rows, width, rng.choice(("f16", "bf16")),
                     rng.choice(("row8", "rowi8", "block8", "block8")), rng.random() < 0.7)
    if op == "product":
        k, n = BLOCK * rng.randint(6, 64), _log(rng, 200, 40000)
        return _product("", _log(rng, 1, min(1500, 1024 * 16384 * 4096 // (n * k))), n, k, rng.choice(("f16", "bf16", "f32")))
    vocab = _log(rng, 300, 131072)
    return _sample("", _log(rng, 1, min(600, 509 * 50277 // vocab)), vocab, rng.choice(("f16", "bf16", "f32")),
                   rng.choice(("plain", "chat", "nucleus", "mixed")))


# ------------------------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------------------------

def _exponent(most):
    """The smallest e in -127..127 with most <= 448 * 2^e (448 = 0.875 * 2^9)."""
    part, e = torch.frexp(most.float())
    return torch.where(most > 0, e - 8 - (part <= 0.875).int(), -127).clamp(-127, 127)


def _scale_row(k):
    """Bytes of one row of block scales: one per 128 k, in words of four."""
    return 4 * -(-k // (4 * BLOCK))


def _power(e):
    return torch.ldexp(torch.ones((), device=e.device, dtype=torch.float64), e.double())


def _block_codes(x, rows_per):
    """e4m3 codes of x [n][k] with one power of two per rows_per x 128, and those scales' bytes [blocks][scale row]."""
    n, k = x.shape
    nb = -(-n // rows_per)
    most = torch.zeros(nb * rows_per, k // BLOCK, device=x.device)
    most[:n] = x.abs().view(n, -1, BLOCK).amax(-1)
    e = _exponent(most.view(nb, rows_per, -1).amax(1))
    inv = _power(-e).float().repeat_interleave(rows_per, 0)[:n]
    codes = (x.view(n, -1, BLOCK) * inv[..., None]).view(n, k).to(torch.float8_e4m3fn)
    bytes_ = torch.zeros(nb, _scale_row(k), dtype=torch.uint8, device=x.device)
    bytes_[:, :k // BLOCK] = (e + 127).to(torch.uint8)
    return codes.view(torch.uint8), bytes_


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt, dev = TYPES[case["dtype"]], "cuda"
    s = {"case": case, "dt": dt}

    def normal(*shape, scale=1.0, mean=0.0, to=torch.float32):
        return torch.randn(*shape, generator=g, device=dev).mul_(scale).add_(mean).to(to)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    if case["op"] == "norm":
        r, c = case["rows"], case["width"]
        s["x"] = normal(r, c, scale=1.5, to=dt)
        s["x"][:, c // 3] *= 50.0     # residual streams have channels that stand far out
        s["delta"] = normal(r, c, to=dt) if case["delta"] else None
        plain = case["norm"] == "none"
        s["gamma"] = None if plain else normal(c, scale=0.2, mean=1.0)
        s["beta"] = normal(c, scale=0.1) if case["norm"] == "layer" else None
        s["x_out"] = torch.empty_like(s["x"]) if case["delta"] else None
        s["codes"] = torch.empty(r, c, dtype=torch.uint8, device=dev)
        s["scales"] = torch.empty(r, _scale_row(c), dtype=torch.uint8, device=dev) if case["format"] == "block8" \
            else torch.empty(r, device=dev)
    elif case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        # a normed row, some of its channels large; weights as a layer's
        x = normal(m, k) * (1.0 + 20.0 * (uniform(k) < 0.01))
        s["xq"], s["sx"] = _block_codes(x, 1)
        s["wq"], s["sw"] = _block_codes(normal(n, k, scale=k ** -0.5) * torch.exp(normal(n, 1, scale=0.3)), BLOCK)
        s["y"] = torch.empty(m, n, dtype=dt, device=dev)
    else:
        r, v, ld = case["rows"], case["vocab"], -(-case["vocab"] // 8) * 8
        # most tokens far down, a few dozens a row that compete; some rows sure of themselves, some not
        z = normal(r, ld, scale=2.0, mean=-6.0)
        z.scatter_add_(1, torch.randint(0, v, (r, 48), generator=g, device=dev), 14.0 * uniform(r, 48) * (0.4 + uniform(r, 1)))
        s["logits"] = z.to(dt)
        f = case["filters"]
        mixed = f == "mixed"
        s["T"] = 0.5 + uniform(r)
        s["top_k"] = s["top_p"] = s["min_p"] = None
        if f == "chat":
            s["top_k"] = torch.full((r,), 50, dtype=torch.int32, device=dev)
            s["top_p"] = torch.full((r,), 0.9, device=dev)
            s["min_p"] = torch.full((r,), 0.02, device=dev)
        elif f == "nucleus":
            s["top_p"] = 0.3 + 0.65 * uniform(r)
        elif mixed:
            s["T"] = torch.where(uniform(r) < 0.15, 0.0, s["T"])          # some take the best
            s["top_k"] = torch.where(uniform(r) < 0.5, torch.exp(uniform(r) * 6.0).int(), 0).int()
            s["top_p"] = torch.where(uniform(r) < 0.5, 0.3 + 0.65 * uniform(r), 1.0)
            s["min_p"] = torch.where(uniform(r) < 0.3, 0.1 * uniform(r), 0.0)
        s["u"] = uniform(r)
        s["token"], s["logprob"] = torch.empty(r, dtype=torch.int32, device=dev), torch.empty(r, device=dev)
    return s


# ------------------------------------------------------------------------------------------------------------------
# the library's calls
# ------------------------------------------------------------------------------------------------------------------

def _own(s):
    from gemm_rwkv_amd import rq
    c = s["case"]
    code = CODES[c["dtype"]]
    if c["op"] == "norm":
        r, w = c["rows"], c["width"]
        rq.rq_norm_quantize(code, NORMS[c["norm"]], s["x"], s["delta"], 0.5, r, w, w, s["gamma"], s["beta"], EPS,
                            FORMATS[c["format"]], s["x_out"], s["codes"], s["scales"])
        return _norm_outputs(s, s["codes"], s["scales"], s["x_out"])
    if c["op"] == "product":
        w = rq.QWeight(FORMATS["block8"], 0, c["n"], c["k"], s["wq"], s["sw"])
        rq.rq_gemm_fp8_block(s["xq"], s["sx"], c["m"], w, code, s["y"], c["n"])
        return s["y"]
    rq.rq_sample(code, s["logits"], c["rows"], c["vocab"], s["logits"].shape[1], s["T"], s["top_k"], s["top_p"],
                 s["min_p"], s["u"], s["token"], s["logprob"])
    return {"token": s["token"], "logprob": s["logprob"]}


def _norm_outputs(s, codes, scales, x_out):
    """Codes and scales as the values that they stand for."""
    fmt = s["case"]["format"]
    codes = codes.view(torch.int8).to(torch.float16) if fmt == "rowi8" else codes.view(torch.float8_e4m3fn)
    out = {"codes": codes, "scales": scales.view(torch.float8_e8m0fnu) if fmt == "block8" else scales}
    return out if x_out is None else dict(out, x=x_out)


# ------------------------------------------------------------------------------------------------------------------
# the plain forms
# ------------------------------------------------------------------------------------------------------------------

def _normed(s, x):
    """The norm of rows x, in x's own precision."""
    norm = s["case"]["norm"]
    if norm == "rms":
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    elif norm == "layer":
        x = x - x.mean(-1, keepdim=True)
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    if s["gamma"] is not None:
        x = x * s["gamma"]
    return x if s["beta"] is None else x + s["beta"]


def _quantized(s, h):
    """(codes, scales) of normed rows."""
    r, c = h.shape
    fmt = s["case"]["format"]
    if fmt == "block8":
        e = _exponent(h.view(r, -1, BLOCK).abs().amax(-1))
        codes = (h.view(r, -1, BLOCK) * _power(-e).to(h.dtype)[..., None]).view(r, c).float().to(torch.float8_e4m3fn)
        scales = torch.zeros(r, _scale_row(c), dtype=torch.uint8, device=h.device)
        scales[:, :c // BLOCK] = (e + 127).to(torch.uint8)
        return codes.view(torch.uint8), scales
    scale = (h.abs().amax(-1) / (127.0 if fmt == "rowi8" else 448.0)).float()
    q = h / scale.to(h.dtype)[:, None]
    return (q.round().to(torch.int8) if fmt == "rowi8" else q.float().to(torch.float8_e4m3fn)).view(torch.uint8), scale


def _norm_plain(s):
    x = s["x"].float()
    if s["delta"] is not None:
        x = x + 0.5 * s["delta"].float()
    codes, scales = _quantized(s, _normed(s, x))
    return _norm_outputs(s, codes, scales, None if s["delta"] is None else x.to(s["dt"]))


def _values(codes, scale_bytes, rows_per, to):
    """What e4m3 codes [n][k] with block scales stand for."""
    n, k = codes.shape
    scale = _power(scale_bytes[:, :k // BLOCK].int() - 127).to(to).repeat_interleave(rows_per, 0)[:n]
    return (codes.view(torch.float8_e4m3fn).to(to).view(n, -1, BLOCK) * scale[..., None]).view(n, k)


def _product_plain(s):
    x, w = _values(s["xq"], s["sx"], 1, torch.float32), _values(s["wq"], s["sw"], BLOCK, torch.float32)
    return (x @ w.T).to(s["dt"])


def _sample_plain(s):
    c = s["case"]
    z = s["logits"][:, :c["vocab"]].double()
    z = torch.where(z.isnan(), -math.inf, z)
    top = z.amax(-1, keepdim=True)
    T = s["T"].double()[:, None]
    x = (z - top) / T
    x = torch.where(T > 0, x, torch.where(z == top, 0.0, -math.inf))
    x, order = x.sort(dim=-1, descending=True, stable=True)
    w = x.exp()
    rank = torch.arange(c["vocab"], device=z.device)
    keep = rank == 0                         # the best one stays whatever the filters say
    if s["top_k"] is not None:
        w = w * ((s["top_k"][:, None] <= 0) | (rank < s["top_k"][:, None]))
    if s["top_p"] is not None:
        before, p = w.cumsum(-1) - w, s["top_p"].double()[:, None]
        w = w * (keep | ~(p < 1) | (before < p * w.sum(-1, keepdim=True)))
    if s["min_p"] is not None:
        w = w * (keep | (w >= s["min_p"].double()[:, None]))
    T0 = ~(T > 0)
    w = torch.where(T0, keep.double(), w)
    mass = torch.zeros_like(w).scatter_(1, order, w).cumsum(-1)     # in the tokens' own order
    token = (mass <= s["u"].double()[:, None] * mass[:, -1:]).sum(-1, keepdim=True)
    at = torch.zeros_like(x).scatter_(1, order, x).gather(1, token)
    return {"token": token[:, 0].int(), "logprob": (at - mass[:, -1:].log())[:, 0].float()}


def run(state):
    if own:
        return _own(state)
    return {"norm": _norm_plain, "product": _product_plain, "sample": _sample_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------------------------

def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["width"]
        scales = case["rows"] * (_scale_row(case["width"]) if case["format"] == "block8" else 4)
        vectors = {"none": 0, "rms": 4, "layer": 8}[case["norm"]] * case["width"]
        return {"bytes": n * (3 + (4 if case["delta"] else 0)) + scales + vectors, "flops": 12 * n}
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        out = 4 if case["dtype"] == "f32" else 2
        return {"bytes": m * k + n * k + (m + -(-n // BLOCK)) * _scale_row(k) + m * n * out, "flops": 2 * m * n * k}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * (4 if case["dtype"] == "f32" else 2) + 28 * case["rows"], "flops": 4 * n}


# ------------------------------------------------------------------------------------------------------------------
# 64-bit values, from the definitions
# ------------------------------------------------------------------------------------------------------------------

def _e4m3_grid():
    """The values of e4m3 that are not negative, rising."""
    return torch.tensor([m / 512 for m in range(8)] + [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1],
                        dtype=torch.float64, device="cuda")


def _nearest_e4m3(v):
    """v to the nearest value of e4m3, ties to the even code."""
    grid = _e4m3_grid()
    a = v.abs()
    hi = torch.searchsorted(grid, a).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.copysign(grid[pick], v)


def _exact_norm(case, s):
    full, x_out = s["x"].double(), None
    if s["delta"] is not None:
        full = x_out = full + 0.5 * s["delta"].double()
    h = _normed(s, full)
    fmt, (r, c) = case["format"], full.shape
    if fmt == "block8":
        most = h.view(r, -1, BLOCK).abs().amax(-1)
        e = torch.ceil(torch.log2(most / 448.0))
        e = torch.where(most <= 448.0 * torch.exp2(e - 1), e - 1, torch.where(most > 448.0 * torch.exp2(e), e + 1, e))
        e = torch.where(most > 0, e, -127).clamp(-127, 127)
        scales = torch.full((r, _scale_row(c)), 2.0 ** -127, dtype=torch.float64, device="cuda")
        scales[:, :c // BLOCK] = torch.exp2(e)
        step = torch.exp2(e).repeat_interleave(BLOCK, 1)
    else:
        scales = h.abs().amax(-1) / (127.0 if fmt == "rowi8" else 448.0)
        step = scales.float().double()[:, None]
    codes = torch.cat([(p / q).round() if fmt == "rowi8" else _nearest_e4m3(p / q)
                       for p, q in zip(h.split(1024), step.split(1024))])
    out = {"codes": codes, "scales": scales}
    return out if x_out is None else dict(out, x=x_out)


def _exact_sample(case, s):
    tokens, logprobs = [], []
    for i in range(case["rows"]):
        z = s["logits"][i, :case["vocab"]].double()
        T = float(s["T"][i])
        if T <= 0:
            tokens.append(int((z == z.max()).nonzero()[0]))
            logprobs.append(0.0)
            continue
        w = torch.softmax(z / T, 0)
        value, order = w.sort(descending=True, stable=True)
        n = len(value)
        if s["top_k"] is not None and int(s["top_k"][i]) > 0:
            n = min(n, int(s["top_k"][i]))
        if s["top_p"] is not None and float(s["top_p"][i]) < 1:
            mass = value[:n].cumsum(0)
            n = 1 + int((mass[:-1] < float(s["top_p"][i]) * mass[-1]).sum())
        if s["min_p"] is not None:
            n = max(1, int((value[:n] >= float(s["min_p"][i]) * value[0]).sum()))
        kept = order[:n].sort().values
        mass = w[kept].cumsum(0)
        j = int(torch.searchsorted(mass, float(s["u"][i]) * mass[-1], right=True))
        tokens.append(int(kept[j]))
        logprobs.append(math.log(float(w[kept[j]] / mass[-1])))
    return {"token": torch.tensor(tokens, dtype=torch.int32), "logprob": torch.tensor(logprobs, dtype=torch.float64)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    if case["op"] == "product":
        k = case["k"]
        x = s["xq"].view(torch.float8_e4m3fn).double() * torch.exp2(s["sx"][:, :k // BLOCK].double() - 127).repeat_interleave(BLOCK, 1)
        sw = torch.exp2(s["sw"][:, :k // BLOCK].double() - 127).repeat_interleave(BLOCK, 1)
        w = s["wq"].view(torch.float8_e4m3fn).split(BLOCK)
        return torch.cat([x @ (part.double() * scale).T for part, scale in zip(w, sw)], 1)
    return _exact_sample(case, s)
