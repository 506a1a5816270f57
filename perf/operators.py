"""The time-mix operators of an RWKV-7 layer as this library's users call them: their cases, inputs, plain forms and
64-bit values.

Three operators stand between the quantized projections of a layer, each with its gradient:

* ``shift_norm``: x' = x + alpha delta, layer norm, then n mixtures of each normed row with the row of the token before
  it (the six inputs of time mixing, or the one of channel mixing);
* ``time_mix``: the per-head state recurrence S_t = S_{t-1} diag(w_t) + (S_{t-1} a_t) b_t^T + v_t k_t^T, y_t = S_t r_t,
  w_t = exp(-exp(-1/2) sigmoid(raw_t)), heads of 64, states in fp32;
* ``head_gate``: the norm over each head's 64 outputs, the r.k bonus on v, and the gate.

``run`` with ``own`` false computes them with elementary torch operations in fp32, the recurrence in chunks of 16 tokens
(products between chunks, one loop along the sequence); with ``own`` true it makes the library's calls.  ``exact``
walks token by token in fp64 and takes gradients by automatic differentiation.
"""

import math

import torch

own = False

HEAD = 64
LN_EPS = 1e-5
HEAD_EPS = 64e-5
DECAY = math.exp(-0.5)   # log w = -DECAY * sigmoid(raw)
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
STEP_FLOPS = 36864       # one head and token: S a, the decay, two outer products, S r
BACK_FLOPS = 118784      # the same again, and the reverse step with its nine products
ELEMENTWISE = {"shift_norm": 12, "head_gate": 14}


# ------------------------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------------------------

def _case(name, op, back, dtype, width, nseq, tokens, **more):
    c = {"op": op, "backward": back, "dtype": dtype, "width": width, "nseq": nseq, "tokens": tokens}
    c.update(more)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one user's next token on the 1.5B layer: nothing but latency
        _case("state decode 1", "time_mix", False, "f16", 2048, 1, 1),
        # a full decode batch on the 7.2B layer, states in a pool that holds half as many again
        _case("state decode 32", "time_mix", False, "f16", 4096, 32, 32),
        # prompts of mixed lengths that arrive together, 2.9B layer
        _case("state prompts ragged", "time_mix", False, "f16", 2560, 7, 1021),
        # one long document, 1.5B layer
        _case("state document 16384", "time_mix", False, "f16", 2048, 1, 16384),
        # a training step's recurrence on the 1.5B layer: four sequences of 1024
        _case("state training back", "time_mix", True, "bf16", 2048, 4, 4096),
        # packed samples of odd lengths on the 0.1B layer
        _case("state packed back", "time_mix", True, "f16", 768, 9, 1531),
        # the norm and the six mixtures before a decode step of 32 requests
        _case("mix decode 32", "shift_norm", False, "f16", 4096, 32, 32, nmix=6),
        # the same before a ragged prefill, 2.9B layer
        _case("mix prompts ragged", "shift_norm", False, "bf16", 2560, 7, 4099, nmix=6),
        # its gradient in the training step
        _case("mix training back", "shift_norm", True, "bf16", 2048, 4, 4096, nmix=6),
        # the norm and the gate after a decode step of 32 requests
        _case("gate decode 32", "head_gate", False, "f16", 4096, 1, 32),
        # after a long prefill chunk
        _case("gate prefill 8192", "head_gate", False, "f16", 2560, 1, 8192),
        # its gradient in the training step
        _case("gate training back", "head_gate", True, "bf16", 2048, 1, 4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("time_mix", "time_mix", "shift_norm", "head_gate"))
    back = rng.random() < 0.4
    dtype = rng.choice(("f16", "bf16"))
    heads = rng.randint(12, 64)
    if op == "time_mix":
        if not back and rng.random() < 0.35:     # decode: one token each
            nseq = _log(rng, 1, 33)
            return _case("", op, False, dtype, HEAD * heads, nseq, nseq)
        tokens = _log(rng, 2, (4096 * 32 if back else 16384 * 32) // heads)
        return _case("", op, back, dtype, HEAD * heads, rng.randint(1, min(tokens, 12)), tokens)
    tokens = _log(rng, 1, 4096 * 32 // heads)
    if op == "head_gate":
        return _case("", op, back, dtype, HEAD * heads, 1, tokens)
    return _case("", op, back, dtype, HEAD * heads, rng.randint(1, min(tokens, 12)), tokens, nmix=rng.choice((1, 6)))


def lengths(case):
    """The sequences' lengths: all equal where they divide, else spread from short to long and out of order."""
    n, total = case["nseq"], case["tokens"]
    if total % n == 0:
        return [total // n] * n
    share = [1 + (5 * i + 2) % n for i in range(n)]
    got = [max(1, total * s // sum(share)) for s in share]
    got[share.index(max(share))] += total - sum(got)
    return got


# ------------------------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt, dev = TYPES[case["dtype"]], "cuda"
    T, C, n = case["tokens"], case["width"], case["nseq"]
    H = C // HEAD
    lens = lengths(case)

    def normal(*shape, scale=1.0, mean=0.0, to=dt):
        return torch.randn(*shape, generator=g, device=dev).mul_(scale).add_(mean).to(to)

    ends = [0]
    for m in lens:
        ends.append(ends[-1] + m)
    even = len(set(lens)) == 1
    s = {"case": case, "lens": lens, "T": T, "C": C, "H": H, "n": n, "dt": dt, "code": {"f16": 6, "bf16": 9}[case["dtype"]],
         "cu": None if even else torch.tensor(ends, dtype=torch.int32, device=dev)}

    def empty(*shape, to=dt):
        return torch.empty(*shape, dtype=to, device=dev)

    f32 = torch.float32
    if case["op"] == "time_mix":
        # receptance, key and value as the projections leave them; the raw decays of a trained layer run from
        # channels that forget at once to channels that keep hundreds of tokens; the removal direction is a unit
        # vector with a part that neighbouring tokens share
        s["r"], s["k"], s["v"] = normal(T, C), normal(T, C, scale=0.5), normal(T, C)
        s["w"] = (torch.randn(C, generator=g, device=dev).mul_(2.0).sub_(1.5) + normal(T, C, scale=0.5, to=f32)).to(dt)
        kk = normal(T, H, HEAD, to=f32) + 0.7 * normal(1, H, HEAD, to=f32)
        kk = kk / kk.norm(dim=-1, keepdim=True)
        rate = torch.sigmoid(normal(T, H, HEAD, to=f32))
        s["a"], s["b"] = (-kk).reshape(T, C).to(dt), (kk * rate).reshape(T, C).to(dt)
        if not case["backward"]:
            nslots = n + (n + 1) // 2
            s["slots"] = torch.randperm(nslots, generator=g, device=dev)[:n].to(torch.int32)
            s["nslots"] = nslots
            s["state"] = normal(nslots, H, HEAD, HEAD, to=f32)
            s["y"] = empty(T, C)
        else:
            s["state"] = normal(n, H, HEAD, HEAD, to=f32)
            s["dy"], s["dstate"] = normal(T, C), normal(n, H, HEAD, HEAD, scale=0.1, to=f32)
            s["grads"] = [empty(T, C) for _ in range(6)]
            s["dstate_in"] = empty(n, H, HEAD, HEAD, to=f32)
    elif case["op"] == "shift_norm":
        m = case["nmix"]
        s["m"], s["alpha"] = m, 0.5
        s["gamma"], s["beta"] = normal(C, scale=0.2, mean=1.0, to=f32), normal(C, scale=0.1, to=f32)
        s["mu"] = torch.rand(m, C, generator=g, device=dev)
        s["x"] = normal(T, C, scale=1.5)
        s["x"][:, C // 3] *= 50.0   # residual streams have channels that stand far out
        s["shift"] = normal(n, C)
        if not case["backward"]:
            s["delta"] = normal(T, C)
            s["x_out"], s["out"], s["shift_out"] = empty(T, C), empty(m, T, C), empty(n, C)
        else:
            s["dout"], s["dx_out"], s["dshift"] = normal(m, T, C), normal(T, C), normal(n, C)
            s["dx"], s["ddelta"], s["dshift_in"] = empty(T, C), empty(T, C), empty(n, C)
            s["dgamma"], s["dbeta"], s["dmu"] = empty(C, to=f32), empty(C, to=f32), empty(m, C, to=f32)
    else:
        s["gamma"], s["beta"] = normal(C, scale=0.2, mean=1.0, to=f32), normal(C, scale=0.1, to=f32)
        s["u"] = normal(C, scale=0.3, to=f32)
        s["y"], s["r"], s["k"], s["v"], s["g"] = (normal(T, C, scale=q) for q in (2.0, 1.0, 0.5, 1.0, 1.0))
        if not case["backward"]:
            s["out"] = empty(T, C)
        else:
            s["dout"] = normal(T, C)
            s["grads"] = [empty(T, C) for _ in range(5)]
            s["dgamma"], s["dbeta"], s["du"] = (empty(C, to=f32) for _ in range(3))
    return s


# ------------------------------------------------------------------------------------------------------------------
# the library's calls
# ------------------------------------------------------------------------------------------------------------------

def _own(s):
    from gemm_rwkv_amd import rq
    op, back = s["case"]["op"], s["case"]["backward"]
    T, C, H, n, code, cu = s["T"], s["C"], s["H"], s["n"], s["code"], s["cu"]
    if op == "time_mix" and not back:
        rq.rq_time_mix(code, s["r"], s["w"], s["k"], s["v"], s["a"], s["b"], T, H, C, cu, n, s["state"], s["state"],
                       s["slots"], s["nslots"], s["y"], C)
        return {"y": s["y"], "state": s["state"]}
    if op == "time_mix":
        rq.rq_time_mix_backward(code, s["r"], s["w"], s["k"], s["v"], s["a"], s["b"], T, H, C, cu, n, s["state"],
                                s["dy"], s["dstate"], *s["grads"], s["dstate_in"])
        return dict(zip(("dr", "dw", "dk", "dv", "da", "db"), s["grads"]), dstate=s["dstate_in"])
    if op == "shift_norm" and not back:
        rq.rq_shift_norm(code, s["x"], s["delta"], s["alpha"], T, C, C, cu, n, s["gamma"], s["beta"], LN_EPS, s["mu"],
                         s["m"], s["shift"], s["shift_out"], None, n, s["x_out"], s["out"], C)
        return {"x": s["x_out"], "out": s["out"], "shift": s["shift_out"]}
    if op == "shift_norm":
        rq.rq_shift_norm_backward(code, s["x"], s["alpha"], T, C, C, cu, n, s["gamma"], s["beta"], LN_EPS, s["mu"],
                                  s["m"], s["shift"], s["dout"], C, s["dx_out"], s["dshift"], s["dx"], s["ddelta"],
                                  s["dshift_in"], s["dgamma"], s["dbeta"], s["dmu"])
        return {k: s[k] for k in ("dx", "ddelta", "dshift_in", "dgamma", "dbeta", "dmu")}
    if not back:
        rq.rq_head_gate(code, s["y"], s["r"], s["k"], s["v"], s["g"], T, H, C, s["gamma"], s["beta"], HEAD_EPS, s["u"],
                        s["out"], C)
        return {"out": s["out"]}
    rq.rq_head_gate_backward(code, s["y"], s["r"], s["k"], s["v"], s["g"], T, H, C, s["gamma"], s["beta"], HEAD_EPS,
                             s["u"], s["dout"], *s["grads"], s["dgamma"], s["dbeta"], s["du"])
    return dict(zip(("dy", "dr", "dk", "dv", "dg"), s["grads"]), dgamma=s["dgamma"], dbeta=s["dbeta"], du=s["du"])


# ------------------------------------------------------------------------------------------------------------------
# the plain forms
# ------------------------------------------------------------------------------------------------------------------

def _grid(s, chunk):
    """Token index of each (sequence, chunk, place), and which places hold a token."""
    lens = torch.tensor(s["lens"], device="cuda")
    most = max(s["lens"])
    pos = torch.arange(-(-most // chunk) * chunk, device="cuda")
    start = torch.cumsum(lens, 0) - lens
    held = pos < lens[:, None]
    return torch.where(held, start[:, None] + pos, 0), held


def _chunks(s, x, at, held, chunk):
    """[sequence][head][chunk][place][64] in fp32, zeros where there is no token."""
    x = x.float().view(s["T"], s["H"], HEAD)[at] * held[..., None, None]
    n, most = at.shape
    return x.view(n, most // chunk, chunk, s["H"], HEAD).permute(0, 3, 1, 2, 4)


def _tokens(s, x, held):
    """The inverse of _chunks, in the inputs' type."""
    n, most = held.shape
    return x.permute(0, 2, 3, 1, 4).reshape(n, most, s["C"])[held].to(s["dt"])


def _chunked(s, state):
    """What a chunk contributes, in terms of the state before it: with u_t = S_{t-1} a_t and decays W accumulated
    within the chunk, U = T (A S^T + Ak V), Y = R S^T + Qb U + Qk V, S' = (S + U^T B + V^T K) diag(W)."""
    chunk = min(16, max(s["lens"]))
    at, held = _grid(s, chunk)
    r, k, v, a, b = (_chunks(s, s[q], at, held, chunk) for q in ("r", "k", "v", "a", "b"))
    raw = s["w"].float().view(s["T"], s["H"], HEAD)[at]
    sig = torch.sigmoid(raw) * held[..., None, None]
    n, most = at.shape
    sig = sig.view(n, most // chunk, chunk, s["H"], HEAD).permute(0, 3, 1, 2, 4)
    logw = -DECAY * sig
    run_ = torch.cumsum(logw, -2)
    grow, fall, before = torch.exp(-run_), torch.exp(run_), torch.exp(run_ - logw)
    d = {"held": held, "sig": sig, "grow": grow, "fall": fall, "before": before,
         "R": r * fall, "A": a * before, "K": k * grow, "B": b * grow, "V": v, "end": fall[..., -1, :, None]}
    kt, bt = d["K"].mT, d["B"].mT
    d["Ab"], d["Ak"] = (d["A"] @ bt).tril(-1), (d["A"] @ kt).tril(-1)
    d["Qb"], d["Qk"] = (d["R"] @ bt).tril(), (d["R"] @ kt).tril()
    T = torch.eye(chunk, device="cuda").expand_as(d["Ab"]).clone()
    for i in range(1, chunk):     # rows of (1 - Ab)^-1, each from those above it
        T[..., i, :i] = (d["Ab"][..., i, :i, None] * T[..., :i, :i]).sum(-2)
    d["T"] = T
    TA, TV = T @ d["A"], T @ (d["Ak"] @ v)
    S, before_, U = state.mT, [], []
    for c in range(most // chunk):
        before_.append(S)
        U.append(TA[:, :, c] @ S + TV[:, :, c])
        S = (S + bt[:, :, c] @ U[-1] + kt[:, :, c] @ v[:, :, c]) * d["end"][:, :, c]
    d["S"], d["U"], d["last"] = torch.stack(before_, 2), torch.stack(U, 2), S
    return d


def _time_mix(s):
    slots = s["slots"].long()
    d = _chunked(s, s["state"][slots])
    y = d["R"] @ d["S"] + d["Qb"] @ d["U"] + d["Qk"] @ d["V"]
    s["state"][slots] = d["last"].mT
    return {"y": _tokens(s, y, d["held"]), "state": s["state"]}


def _time_mix_back(s):
    d = _chunked(s, s["state"])
    A, B, K, R, S, T, U, V = (d[q] for q in "ABKRSTUV")
    dY = _chunks(s, s["dy"], *_grid(s, R.shape[3]), R.shape[3])
    own_ = d["Qb"].mT @ dY
    D, after, Z = s["dstate"].mT, [], []
    for c in reversed(range(R.shape[2])):
        D = D * d["end"][:, :, c]
        after.append(D)
        Z.append(T[:, :, c].mT @ (own_[:, :, c] + B[:, :, c] @ D))
        D = D + R[:, :, c].mT @ dY[:, :, c] + A[:, :, c].mT @ Z[-1]
    dstate = D.mT.contiguous()
    D, Z = torch.stack(after[::-1], 2), torch.stack(Z[::-1], 2)
    dQb, dQk = (dY @ U.mT).tril(), (dY @ V.mT).tril()
    dAb, dAk = (Z @ U.mT).tril(-1), (Z @ V.mT).tril(-1)
    dV = d["Qk"].mT @ dY + K @ D + d["Ak"].mT @ Z
    dR = dY @ S.mT + dQb @ B + dQk @ K
    dA = Z @ S.mT + dAb @ B + dAk @ K
    dB = U @ D.mT + dQb.mT @ R + dAb.mT @ A
    dK = V @ D.mT + dQk.mT @ R + dAk.mT @ A
    last = ((S + B.mT @ U + K.mT @ V) * D).sum(-1)
    per = R * dR - B * dB - K * dK
    per[..., :-1, :] += (A * dA)[..., 1:, :]
    per[..., -1, :] += last
    dlog = per.flip(-2).cumsum(-2).flip(-2)
    dw = dlog * -DECAY * d["sig"] * (1 - d["sig"])
    got = {"dr": dR * d["fall"], "dw": dw, "dk": dK * d["grow"], "dv": dV, "da": dA * d["before"], "db": dB * d["grow"]}
    return dict({q: _tokens(s, x, d["held"]) for q, x in got.items()}, dstate=dstate)


def _first(s):
    """Which tokens open a sequence, and the row that each sequence opens and ends at."""
    ends = torch.cumsum(torch.tensor(s["lens"], device="cuda"), 0)
    starts = ends - torch.tensor(s["lens"], device="cuda")
    return starts, ends - 1


def _shift_norm(s):
    x = s["x"].float() + s["alpha"] * s["delta"].float()
    mid = x - x.mean(-1, keepdim=True)
    h = mid * torch.rsqrt(mid.square().mean(-1, keepdim=True) + LN_EPS) * s["gamma"] + s["beta"]
    starts, ends = _first(s)
    prev = torch.cat([h[:1], h[:-1]])
    prev[starts] = s["shift"].float()
    out = h + (prev - h) * s["mu"][:, None, :]
    return {"x": x.to(s["dt"]), "out": out.to(s["dt"]), "shift": h[ends].to(s["dt"])}


def _shift_norm_back(s):
    x, dout = s["x"].float(), s["dout"].float()
    mid = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt(mid.square().mean(-1, keepdim=True) + LN_EPS)
    norm = mid * rstd
    h = norm * s["gamma"] + s["beta"]
    starts, ends = _first(s)
    prev = torch.cat([h[:1], h[:-1]])
    prev[starts] = s["shift"].float()
    dmu = (dout * (prev - h)).sum(1)
    dprev = (dout * s["mu"][:, None, :]).sum(0)
    dh = dout.sum(0) - dprev
    dshift_in = dprev[starts]
    dprev[starts] = 0
    dh[:-1] += dprev[1:]
    dh[ends] += s["dshift"].float()
    dn = dh * s["gamma"]
    dx = (dn - dn.mean(-1, keepdim=True) - norm * (dn * norm).mean(-1, keepdim=True)) * rstd + s["dx_out"].float()
    return {"dx": dx.to(s["dt"]), "ddelta": (s["alpha"] * dx).to(s["dt"]), "dshift_in": dshift_in.to(s["dt"]),
            "dgamma": (dh * norm).sum(0), "dbeta": dh.sum(0), "dmu": dmu}


def _heads(s, *names):
    return [s[q].float().view(-1, s["H"], HEAD) for q in names]


def _head_gate(s):
    y, r, k, v, g = _heads(s, "y", "r", "k", "v", "g")
    gamma, beta, u = (s[q].view(s["H"], HEAD) for q in ("gamma", "beta", "u"))
    mid = y - y.mean(-1, keepdim=True)
    norm = mid * torch.rsqrt(mid.square().mean(-1, keepdim=True) + HEAD_EPS)
    out = (norm * gamma + beta + (r * k * u).sum(-1, keepdim=True) * v) * g
    return {"out": out.view(s["T"], s["C"]).to(s["dt"])}


def _head_gate_back(s):
    y, r, k, v, g, dout = _heads(s, "y", "r", "k", "v", "g", "dout")
    gamma, beta, u = (s[q].view(s["H"], HEAD) for q in ("gamma", "beta", "u"))
    mid = y - y.mean(-1, keepdim=True)
    rstd = torch.rsqrt(mid.square().mean(-1, keepdim=True) + HEAD_EPS)
    norm = mid * rstd
    bonus = (r * k * u).sum(-1, keepdim=True)
    dg = dout * (norm * gamma + beta + bonus * v)
    dz = dout * g
    db = (dz * v).sum(-1, keepdim=True)
    dn = dz * gamma
    dy = (dn - dn.mean(-1, keepdim=True) - norm * (dn * norm).mean(-1, keepdim=True)) * rstd
    got = {"dy": dy, "dr": db * k * u, "dk": db * r * u, "dv": dz * bonus, "dg": dg}
    got = {q: x.reshape(s["T"], s["C"]).to(s["dt"]) for q, x in got.items()}
    return dict(got, dgamma=(dz * norm).sum(0).view(-1), dbeta=dz.sum(0).view(-1), du=(db * r * k).sum(0).view(-1))


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    return {("time_mix", False): _time_mix, ("time_mix", True): _time_mix_back, ("shift_norm", False): _shift_norm,
            ("shift_norm", True): _shift_norm_back, ("head_gate", False): _head_gate,
            ("head_gate", True): _head_gate_back}[c["op"], c["backward"]](state)


# ------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------------------------

def work(case):
    T, C, n = case["tokens"], case["width"], case["nseq"]
    rows, state = 2 * T * C, 4 * n * C * HEAD
    if case["op"] == "time_mix" and not case["backward"]:
        return {"bytes": 7 * rows + 2 * state, "flops": T * (C // HEAD) * STEP_FLOPS}
    if case["op"] == "time_mix":
        return {"bytes": 13 * rows + 3 * state, "flops": T * (C // HEAD) * BACK_FLOPS}
    if case["op"] == "shift_norm":
        m = case["nmix"]
        planes, small = (3 + m, 2) if not case["backward"] else (4 + m, 3)
        params = 4 * C * (2 + m) * (2 if case["backward"] else 1)
        return {"bytes": planes * rows + small * 2 * n * C + params, "flops": T * C * (ELEMENTWISE["shift_norm"] + 3 * m)}
    planes = 11 if case["backward"] else 6
    return {"bytes": planes * rows + 12 * C * (2 if case["backward"] else 1),
            "flops": T * C * ELEMENTWISE["head_gate"] * (3 if case["backward"] else 1)}


# ------------------------------------------------------------------------------------------------------------------
# 64-bit values, from the definitions
# ------------------------------------------------------------------------------------------------------------------

def _leaf(x, shape=None):
    x = x.detach().double()
    return (x if shape is None else x.view(shape)).clone().requires_grad_()


def _walk(lens, r, w, k, v, a, b, states):
    """The recurrence as it is defined, one token after the other; the sequences side by side while they last."""
    decay = torch.exp(-DECAY * torch.sigmoid(w))
    starts = [sum(lens[:i]) for i in range(len(lens))]
    ys, order = [], []
    S = states
    for t in range(max(lens, default=0)):
        live = [i for i, m in enumerate(lens) if m > t]
        at = torch.tensor([starts[i] + t for i in live], device=r.device)
        whole = len(live) == len(lens)
        pick = None if whole else torch.tensor(live, device=r.device)
        P = S if whole else S[pick]
        u = (P * a[at][:, :, None, :]).sum(-1)
        N = P * decay[at][:, :, None, :] + u[..., None] * b[at][:, :, None, :] + v[at][..., None] * k[at][:, :, None, :]
        ys.append((N * r[at][:, :, None, :]).sum(-1))
        order.append(at)
        S = N if whole else S.index_copy(0, pick, N)
    y = torch.empty_like(r).index_copy(0, torch.cat(order), torch.cat(ys))
    return y, S


def exact(case, seed):
    s = prepare(case, seed)
    T, C, H = s["T"], s["C"], s["H"]
    back = case["backward"]
    with torch.set_grad_enabled(back):
        if case["op"] == "time_mix":
            ins = [_leaf(s[q], (T, H, HEAD)) for q in ("r", "w", "k", "v", "a", "b")]
            if not back:
                slots = s["slots"].long()
                pool = s["state"].double()
                y, S = _walk(s["lens"], *ins, pool[slots])
                pool[slots] = S
                return {"y": y.reshape(T, C), "state": pool}
            states = _leaf(s["state"])
            y, S = _walk(s["lens"], *ins, states)
            total = (y * s["dy"].double().view(T, H, HEAD)).sum() + (S * s["dstate"].double()).sum()
            got = torch.autograd.grad(total, ins + [states])
            return dict({q: x.reshape(T, C) for q, x in zip(("dr", "dw", "dk", "dv", "da", "db"), got)}, dstate=got[-1])
        if case["op"] == "shift_norm":
            x, gamma, beta, mu, shift = (_leaf(s[q]) for q in ("x", "gamma", "beta", "mu", "shift"))
            full = x if back else x + s["alpha"] * s["delta"].double()
            mean = full.mean(-1, keepdim=True)
            var = ((full - mean) ** 2).mean(-1, keepdim=True)
            h = (full - mean) / torch.sqrt(var + LN_EPS) * gamma + beta
            parts, lasts, at = [], [], 0
            for i, m in enumerate(s["lens"]):
                parts += [shift[i:i + 1], h[at:at + m - 1]]
                lasts.append(h[at + m - 1])
                at += m
            prev, last = torch.cat(parts), torch.stack(lasts)
            out = torch.stack([h + (prev - h) * mu[i] for i in range(s["m"])])
            if not back:
                return {"x": full, "out": out, "shift": last}
            total = (out * s["dout"].double()).sum() + (full * s["dx_out"].double()).sum() + (last * s["dshift"].double()).sum()
            dx, dgamma, dbeta, dmu, dshift = torch.autograd.grad(total, [x, gamma, beta, mu, shift])
            return {"dx": dx, "ddelta": s["alpha"] * dx, "dshift_in": dshift, "dgamma": dgamma, "dbeta": dbeta, "dmu": dmu}
        y, r, k, v, g = (_leaf(s[q], (T, H, HEAD)) for q in ("y", "r", "k", "v", "g"))
        gamma, beta, u = (_leaf(s[q]) for q in ("gamma", "beta", "u"))
        mean = y.mean(-1, keepdim=True)
        var = ((y - mean) ** 2).mean(-1, keepdim=True)
        z = (y - mean) / torch.sqrt(var + HEAD_EPS) * gamma.view(H, HEAD) + beta.view(H, HEAD)
        z = z + (r * k * u.view(H, HEAD)).sum(-1, keepdim=True) * v
        out = z * g
        if not back:
            return {"out": out.reshape(T, C)}
        got = torch.autograd.grad((out * s["dout"].double().view(T, H, HEAD)).sum(), [y, r, k, v, g, gamma, beta, u])
        names = ("dy", "dr", "dk", "dv", "dg")
        return dict({q: x.reshape(T, C) for q, x in zip(names, got)}, dgamma=got[5], dbeta=got[6], du=got[7])
