"""The operators around a recurrent layer, measured: the short causal
convolution in front of it, the selective state space scan, and the norms
after and before a block with its gate and residual scale.

Every case is one pass of one operator in one direction: "fwd" (prompts),
"bwd" (training) or "step" (one new token for each sequence).  ``run`` takes
the operators in their plain form, or through the framework's calls where
``own`` is true; ``exact`` holds the definitions in 64 bits.

Layouts are token-major: x, u, delta, z [B, T, D]; B, C [B, T, G, S]; a packed
batch has B = 1 and offsets ``cu`` of its sequences.  Sequences are ragged and
may be empty.  What a layer takes out of one projection (z beside u, C beside
B, the convolution's input) is a slice of that projection's output here too.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # the convolution over the 32 heads of 128 channels of one projection
        # of a two-sequence prompt
        dict(name="conv prompt", op="conv", dir="fwd", type=BF16, batch=2, tokens=8192, dim=4096, width=4, act=True, bias=False, state=False, sliced=True),
        # training on a packed batch of ragged documents, one of them empty
        dict(name="conv packed training", op="conv", dir="bwd", type=BF16, lengths="1 3 0 517 2048 1023 4097 511", dim=4096, width=4, act=True, bias=True, state=True, sliced=True),
        # one token for each of 256 sequences being served, the q, k and v
        # channels of a layer in one call
        dict(name="conv tokens", op="conv", dir="step", type=BF16, batch=256, dim=12288, width=4, act=True, bias=False),
        # a two-sequence prompt through the scan, 16 states a channel
        dict(name="scan prompt", op="scan", dir="fwd", type=BF16, batch=2, tokens=8192, dim=4096, states=16, groups=1, gate=True, skip=True, state=False),
        # a short prompt in full precision: a small model's first call, latency counts
        dict(name="scan short prompt", op="scan", dir="fwd", type=F32, batch=1, tokens=128, dim=256, states=16, groups=1, gate=True, skip=True, state=False),
        # a packed batch of ragged prompts that go on from their states, an
        # odd number of channels in two groups
        dict(name="scan packed prompts", op="scan", dir="fwd", type=BF16, lengths="2048 1 777 0 4095 63 1209", dim=1002, states=16, groups=2, gate=True, skip=True, state=True),
        # a training step's backward pass
        dict(name="scan training", op="scan", dir="bwd", type=BF16, batch=2, tokens=4096, dim=4096, states=16, groups=1, gate=True, skip=True, state=False),
        # one token for each of 256 sequences being served
        dict(name="scan tokens", op="scan", dir="step", type=BF16, batch=256, dim=4096, states=16, groups=1, gate=True, skip=True),
        # the gated norm of a layer's output per head, before its projection
        dict(name="norm heads", op="norm", dir="fwd", type=BF16, residual="", rows=16384, heads=32, width=128, gate="sigmoid", first=False, post=True, pre=False, scale=False),
        # a block's end and the next one's start: norm, gate, scale, residual
        # stream in full precision, next norm
        dict(name="norm block", op="norm", dir="fwd", type=BF16, residual=F32, rows=16384, heads=1, width=4096, gate="silu", first=False, post=True, pre=True, scale=True),
        # the same boundary in training
        dict(name="norm block training", op="norm", dir="bwd", type=BF16, residual=BF16, rows=8192, heads=1, width=4096, gate="sigmoid", first=False, post=True, pre=True, scale=True),
        # the boundary for 256 single tokens, an odd width in full precision
        dict(name="norm tokens", op="norm", dir="fwd", type=F32, residual=F32, rows=256, heads=1, width=1001, gate="", first=False, post=True, pre=True, scale=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _ragged(rng, total, n):
    """n lengths with the given sum, spread unevenly, some of them empty."""
    w = [0.0 if rng.random() < 0.15 else rng.random() ** 3 for _ in range(n)]
    s = sum(w)
    if s == 0:
        return [total] + [0] * (n - 1)
    lens = [int(total * x / s) for x in w]
    lens[lens.index(max(lens))] += total - sum(lens)
    return lens


def draw(rng):
    op = rng.choice(["conv", "scan", "scan", "norm"])
    kind = rng.choice([BF16, BF16, F32])
    if op == "norm":
        case = dict(op=op, dir=rng.choice(["fwd", "bwd"]), type=kind)
        if rng.random() < 0.4:
            heads, width = rng.choice([4, 8, 32]), rng.choice([32, 64, 128, 96])
            pre, residual, scale = False, "", False
            rows = _log_int(rng, 1, 16384 * 4096 // (heads * width) // 2)
        else:
            heads, width = 1, _log_int(rng, 64, 8192)
            residual = rng.choice([kind, F32])
            pre, scale = rng.random() < 0.8, rng.random() < 0.7
            rows = _log_int(rng, 1, 16384 * 4096 // width // 2)
        case.update(residual=residual, rows=min(rows, 65536), heads=heads, width=width, gate=rng.choice(["sigmoid", "silu", ""]), first=rng.random() < 0.3,
                    post=rng.random() < 0.8 or not pre, pre=pre, scale=scale)
        return case
    case = dict(op=op, dir=rng.choice(["fwd", "fwd", "bwd", "step"]), type=kind)
    dim = rng.choice([64, 256, 1000, 2048, 4096, _log_int(rng, 16, 4096)])
    if case["dir"] == "step":
        case.update(batch=_log_int(rng, 1, 256), dim=dim)
    else:
        states = 16
        most = 2 ** 30 // (dim * states) if case["dir"] == "fwd" else 2 ** 29 // (dim * states)
        tokens = _log_int(rng, 1, min(most, 16384))
        if rng.random() < 0.5:
            case.update(lengths=" ".join(map(str, _ragged(rng, tokens, rng.randint(1, 12)))), dim=dim)
        else:
            batch = rng.choice([1, 1, 2, 3])
            case.update(batch=batch, tokens=max(1, tokens // batch), dim=dim)
        case.update(state=rng.random() < 0.5)
    if op == "conv":
        case.update(width=rng.choice([2, 3, 4, 4]), act=rng.random() < 0.8, bias=rng.random() < 0.5)
        if case["dir"] != "step":
            case.update(sliced=rng.random() < 0.5)
    else:
        groups = 2 if dim % 2 == 0 and rng.random() < 0.3 else 1
        case.update(states=rng.choice([16, 16, 8, 12]), groups=groups, gate=rng.random() < 0.8, skip=rng.random() < 0.8)
    return case


# ----------------------------------------------------------------- the inputs

_DTYPE = {BF16: torch.bfloat16, F32: torch.float32}


def _lengths(case):
    if "lengths" in case:
        return [int(x) for x in case["lengths"].split()]
    return [case["tokens"]] * case["batch"]


def _offsets(case):
    cu = [0]
    for n in _lengths(case):
        cu.append(cu[-1] + n)
    return cu


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _DTYPE[case["type"]]

    def randn(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * std

    def rand(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    s = {"case": case}
    if case["op"] == "norm":
        lead = (case["rows"], case["heads"], case["width"])
        width = case["width"]
        # a block's output and its gate's logits; the stream grows over the layers
        s["x"] = randn(*lead, std=1.5).to(dt)
        s["gate"] = randn(*lead).to(dt) if case["gate"] else None
        s["residual"] = randn(*lead, std=4.0).to(_DTYPE[case["residual"]]) if case["residual"] else None
        s["post_weight"] = 1 + randn(width, std=0.2) if case["post"] else None
        s["pre_weight"] = 1 + randn(width, std=0.2) if case["pre"] else None
        s["scale"] = 0.5 + randn(width, std=0.1) if case["scale"] else None
        if case["dir"] == "bwd":
            s["d_out"] = randn(*lead).to(_DTYPE[case["residual"]] if case["residual"] else dt)
            s["d_normed"] = randn(*lead).to(dt) if case["pre"] else None
        return s
    D = case["dim"]
    step = case["dir"] == "step"
    packed = "lengths" in case
    lead = (case["batch"], 1) if step else (1, sum(_lengths(case))) if packed else (case["batch"], case["tokens"])
    n = case["batch"] if step else len(_lengths(case))
    s["cu"] = torch.tensor(_offsets(case), dtype=torch.int32, device="cuda") if packed else None
    if case["op"] == "conv":
        W = case["width"]
        x = randn(*lead, 3 * D if case.get("sliced") else D).to(dt)
        # the middle one of the three that a projection gives
        s["x"] = x[..., D:2 * D] if case.get("sliced") else x
        s["weight"] = randn(D, W, std=1 / math.sqrt(W))
        s["bias"] = randn(D, std=0.1) if case["bias"] else None
        s["state"] = randn(n, W - 1, D).to(dt) if step or case["state"] else None
        if case["dir"] == "bwd":
            s["d_out"] = randn(*lead, D).to(dt)
            s["d_final"] = randn(n, W - 1, D).to(dt) if case["state"] else None
        return s
    S, G = case["states"], case["groups"]
    s["u"] = randn(*lead, D).to(dt)
    s["z"] = randn(*lead, 2 * D).to(dt)[..., D:] if case["gate"] else None
    s["delta"] = randn(*lead, D, std=0.5).to(dt)
    # step sizes between 0.001 and 0.1 through the softplus, rates near 1 .. S
    dt0 = torch.exp(rand(D) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
    s["delta_bias"] = dt0 + torch.log(-torch.expm1(-dt0))
    s["A"] = -torch.exp(torch.log(torch.arange(1, S + 1, device="cuda", dtype=torch.float32)) + randn(D, S, std=0.1))
    bc = randn(*lead, G, 2 * S).to(dt)
    s["Bm"], s["Cm"] = bc[..., :S], bc[..., S:]
    s["D"] = 1 + randn(D, std=0.1) if case["skip"] else None
    s["state"] = randn(n, D, S, std=0.5) if step or case["state"] else None
    if case["dir"] == "bwd":
        s["d_out"] = randn(*lead, D).to(dt)
        s["d_final"] = randn(n, D, S) if case["state"] else None
    return s


# ------------------------------------------------------------------- one pass

def run(state):
    s, c = state, state["case"]
    if own:
        return _own(s, c)
    return {"conv": _plain_conv, "scan": _plain_scan, "norm": _plain_norm}[c["op"]](s, c)


def _own(s, c):
    from gated_delta_rule_156_b200 import kda
    if c["op"] == "conv":
        act = "silu" if c["act"] else "none"
        if c["dir"] == "fwd":
            return kda.short_conv_fwd(s["x"], s["weight"], s["bias"], s["state"], s["cu"], activation=act)
        if c["dir"] == "bwd":
            return _kept(kda.short_conv_bwd(s["x"], s["weight"], s["bias"], s["state"], s["cu"], s["d_out"], s["d_final"], activation=act))
        return kda.short_conv_step(s["x"], s["weight"], s["bias"], s["state"], activation=act), s["state"]
    if c["op"] == "scan":
        args = (s["u"], s["delta"], s["A"], s["Bm"], s["Cm"])
        more = dict(D=s["D"], z=s["z"], delta_bias=s["delta_bias"], softplus=True)
        if c["dir"] == "fwd":
            return kda.ssm_scan_fwd(*args, initial_state=s["state"], cu_seqlens=s["cu"], **more)
        if c["dir"] == "bwd":
            return _kept(kda.ssm_scan_bwd(*args, d_out=s["d_out"], d_final_state=s["d_final"], initial_state=s["state"], cu_seqlens=s["cu"], **more))
        return kda.ssm_step(*args, state=s["state"], **more), s["state"]
    args = dict(post_weight=s["post_weight"], gate=s["gate"], residual=s["residual"], scale=s["scale"], pre_weight=s["pre_weight"],
                gate_act=c["gate"] or "none", gate_first=c["first"], eps=1e-6)
    if c["dir"] == "fwd":
        return _kept(kda.block_norm_fwd(s["x"], **args))
    return _kept(kda.block_norm_bwd(s["x"], d_out=s["d_out"], d_normed=s["d_normed"], **args))


def _kept(outs):
    return tuple(x for x in outs if x is not None)


# ------------------------------------------------------------ the plain forms

def _token_index(s, tokens, batch):
    """(first token of every token's sequence, its sequence, the offsets) over the flat tokens."""
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(batch + 1, device="cuda") * (tokens // batch)
    seq = torch.searchsorted(cu, torch.arange(tokens, device="cuda"), right=True) - 1
    return cu[seq], seq, cu


def _silu_grad(x):
    sg = torch.sigmoid(x)
    return sg * (1 + x * (1 - sg))


def _plain_conv(s, c):
    dt, W, D = s["x"].dtype, c["width"], c["dim"]
    w = s["weight"]
    if c["dir"] == "step":
        past = torch.cat([s["state"].float(), s["x"].float()], dim=1)
        pre = (past * w.t()).sum(1, keepdim=True)
        pre = pre if s["bias"] is None else pre + s["bias"]
        s["state"].copy_(past[:, 1:])
        return (pre * torch.sigmoid(pre) if c["act"] else pre).to(dt), s["state"]
    lead = s["x"].shape[:2]
    N = lead[0] * lead[1]
    x = s["x"].reshape(N, D).float()
    start, seq, cu = _token_index(s, N, lead[0])
    n = cu.numel() - 1
    past = torch.zeros(n, W - 1, D, device="cuda") if s["state"] is None else s["state"].float()
    t = torch.arange(N, device="cuda")
    # row r of `rows` is input r, row N + n' (W - 1) + j row j of sequence n's past
    rows = torch.cat([x, past.reshape(n * (W - 1), D)])
    at = [torch.where(t - back >= start, t - back, N + seq * (W - 1) + (W - 1) + (t - back - start)) for back in range(W - 1, -1, -1)]
    pre = sum(rows[at[j]] * w[:, j] for j in range(W))
    pre = pre if s["bias"] is None else pre + s["bias"]
    # the last W - 1 inputs of every sequence, its past where it is shorter
    back = torch.arange(W - 1, 0, -1, device="cuda")
    last = cu[1:, None] - back
    keep = torch.where(last >= cu[:-1, None], last, N + torch.arange(n, device="cuda")[:, None] * (W - 1) + (W - 1) + last - cu[:-1, None])
    if c["dir"] == "fwd":
        out = pre * torch.sigmoid(pre) if c["act"] else pre
        return out.to(dt).reshape(*lead, D), rows[keep].to(dt)
    dpre = s["d_out"].reshape(N, D).float()
    dpre = dpre * _silu_grad(pre) if c["act"] else dpre
    dw = torch.stack([(dpre * rows[at[j]]).sum(0) for j in range(W)], 1)
    drows = sum(torch.zeros_like(rows).index_copy(0, at[j], dpre * w[:, j]) for j in range(W))
    if s["d_final"] is not None:
        drows = drows.index_add(0, keep.reshape(-1), s["d_final"].float().reshape(-1, D))
    outs = (drows[:N].to(dt).reshape(*lead, D), dw, dpre.sum(0) if s["bias"] is not None else None, drows[N:].reshape(n, W - 1, D).to(dt))
    return _kept(outs)


def _chain(a, b, longest):
    """h_t = a_t h_{t-1} + b_t along dim 0 by doubling: after the step of k, (a_t, b_t) stands for the last 2k tokens."""
    k = 1
    while k < longest:
        b = torch.cat([b[:k], torch.addcmul(b[k:], a[k:], b[:-k])])
        if 2 * k < longest:
            a = torch.cat([a[:k], a[k:] * a[:-k]])
        k *= 2
    return b


def _plain_scan(s, c):
    dt, D, S, G = s["u"].dtype, c["dim"], c["states"], c["groups"]
    lead = s["u"].shape[:2]
    N = lead[0] * lead[1]
    u = s["u"].reshape(N, D).float()
    raw = s["delta"].reshape(N, D).float() + s["delta_bias"]
    step = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    A = s["A"]
    per = D // G
    Bm = s["Bm"].reshape(N, G, S).float().repeat_interleave(per, 1)
    Cm = s["Cm"].reshape(N, G, S).float().repeat_interleave(per, 1)
    skip = s["D"] if s["D"] is not None else torch.zeros(D, device="cuda")
    a = torch.exp(step[..., None] * A)
    b = (step * u)[..., None] * Bm
    if c["dir"] == "step":
        h = a * s["state"] + b
        s["state"].copy_(h)
        y = (h * Cm).sum(-1) + skip * u
        if s["z"] is not None:
            z = s["z"].reshape(N, D).float()
            y = y * z * torch.sigmoid(z)
        return y.to(dt).reshape(*lead, D), s["state"]
    start, seq, cu = _token_index(s, N, lead[0])
    n = cu.numel() - 1
    first = start == torch.arange(N, device="cuda")
    full = (cu[1:] > cu[:-1])
    past = torch.zeros(n, D, S, device="cuda") if s["state"] is None else s["state"]
    heads, tails = cu[:-1][full], cu[1:][full] - 1
    b = b.index_add(0, heads, a[heads] * past[full])
    linked = a * (~first).float()[:, None, None]
    longest = max(_lengths(c))
    h = _chain(linked, b, longest)
    y = (h * Cm).sum(-1) + skip * u
    z = s["z"].reshape(N, D).float() if s["z"] is not None else None
    if c["dir"] == "fwd":
        final = past.clone()
        final[full] = h[tails]
        y = y if z is None else y * z * torch.sigmoid(z)
        return y.to(dt).reshape(*lead, D), final
    dout = s["d_out"].reshape(N, D).float()
    dy = dout if z is None else dout * z * torch.sigmoid(z)
    dz = None if z is None else (dout * y * _silu_grad(z)).to(dt).reshape(*lead, D)
    dC = (dy[..., None] * h).reshape(N, G, per, S).sum(2)
    g = dy[..., None] * Cm
    if s["d_final"] is not None:
        g = g.index_add(0, tails, s["d_final"][full])
    # dh_t = g_t + a_{t+1} dh_{t+1}: the same chain over the reversed tokens
    after = torch.cat([linked[1:], torch.zeros_like(linked[:1])])
    dh = _chain(after.flip(0), g.flip(0), longest).flip(0)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before = before * (~first).float()[:, None, None]
    before[heads] = past[full]
    da = dh * before * a
    dpast = s["d_final"].clone() if s["d_final"] is not None else torch.zeros_like(past)
    dpast[full] = a[heads] * dh[heads]
    fed = (dh * Bm).sum(-1)
    du = fed * step + dy * skip
    draw_ = ((da * A).sum(-1) + fed * u) * torch.sigmoid(raw)
    outs = (du.to(dt).reshape(*lead, D), draw_.to(dt).reshape(*lead, D), (da * step[..., None]).sum(0),
            (dh * (step * u)[..., None]).reshape(N, G, per, S).sum(2).to(dt).reshape(*lead, G, S), dC.to(dt).reshape(*lead, G, S),
            (dy * u).sum(0) if s["D"] is not None else None, dz, draw_.sum(0), dpast)
    return _kept(outs)


def _plain_norm(s, c):
    dt, eps = s["x"].dtype, 1e-6
    x = s["x"].float()
    gate = s["gate"].float() if s["gate"] is not None else None
    act, dact = None, None
    if gate is not None:
        sg = torch.sigmoid(gate)
        act, dact = (sg, sg * (1 - sg)) if c["gate"] == "sigmoid" else (gate * sg, sg * (1 + gate * (1 - sg)))
    before, behind = act is not None and c["first"], act is not None and not c["first"]
    h = x * act if before else x
    inv = torch.rsqrt((h * h).mean(-1, keepdim=True) + eps) if s["post_weight"] is not None else None
    q = h * inv * s["post_weight"] if inv is not None else h
    p = q * act if behind else q
    out = p if s["scale"] is None else p * s["scale"]
    rt = dt
    if s["residual"] is not None:
        out, rt = out + s["residual"].float(), s["residual"].dtype
    inv2 = torch.rsqrt((out * out).mean(-1, keepdim=True) + eps) if s["pre_weight"] is not None else None
    if c["dir"] == "fwd":
        return _kept((out.to(rt), (out * inv2 * s["pre_weight"]).to(dt) if inv2 is not None else None))
    rows = tuple(range(x.dim() - 1))
    dr = s["d_out"].float()
    dpre = dscale = dpost = dgate = None
    if inv2 is not None:
        dn, unit = s["d_normed"].float(), out * inv2
        dpre = (dn * unit).sum(rows)
        v = dn * s["pre_weight"]
        dr = dr + inv2 * (v - unit * (v * unit).mean(-1, keepdim=True))
    dp = dr
    if s["scale"] is not None:
        dscale = (dr * p).sum(rows)
        dp = dr * s["scale"]
    if behind:
        dgate = dp * q * dact
        dp = dp * act
    if inv is not None:
        unit = h * inv
        dpost = (dp * unit).sum(rows)
        v = dp * s["post_weight"]
        dp = inv * (v - unit * (v * unit).mean(-1, keepdim=True))
    dx = dp
    if before:
        dgate, dx = dp * x * dact, dp * act
    return _kept((dx.to(dt), dgate.to(dt) if dgate is not None else None, dr.to(rt) if s["residual"] is not None else None, dpost, dscale, dpre))


# ------------------------------------------------------- what it cannot do without

def work(case):
    e = 2 if case["type"] == BF16 else 4
    if case["op"] == "norm":
        n = case["rows"] * case["heads"] * case["width"]
        r = {"": 0, BF16: 2, F32: 4}[case["residual"]]
        o = r or e
        gate = e if case["gate"] else 0
        pre = e if case["pre"] else 0
        if case["dir"] == "fwd":
            return {"bytes": n * (e + gate + r + o + pre), "flops": n * 14}
        return {"bytes": n * (2 * e + 2 * gate + 2 * r + o + pre), "flops": n * 40}
    D = case["dim"]
    N = case["batch"] if case["dir"] == "step" else sum(_lengths(case))
    n = case["batch"] if case["dir"] == "step" else len(_lengths(case))
    if case["op"] == "conv":
        W = case["width"]
        states = n * (W - 1) * D * e
        small = D * W * 4 + (D * 4 if case["bias"] else 0)
        if case["dir"] == "fwd":
            return {"bytes": N * D * 2 * e + small + states * (2 if case["state"] else 1), "flops": N * D * (2 * W + 4)}
        if case["dir"] == "bwd":
            return {"bytes": N * D * 3 * e + 2 * small + states * (3 if case["state"] else 1), "flops": N * D * (6 * W + 10)}
        return {"bytes": N * D * 2 * e + small + 2 * states, "flops": N * D * (2 * W + 4)}
    S, G = case["states"], case["groups"]
    gate = e if case["gate"] else 0
    states = n * D * S * 4
    small = D * (S + 2) * 4
    tokens = N * (D * (3 * e + gate) + 2 * G * S * e)
    if case["dir"] == "fwd":
        return {"bytes": tokens + small + states * (2 if case["state"] else 1), "flops": N * D * (7 * S + 12)}
    if case["dir"] == "bwd":
        return {"bytes": N * (D * (5 * e + 2 * gate) + 4 * G * S * e) + 2 * small + states * (3 if case["state"] else 1), "flops": N * D * (21 * S + 40)}
    return {"bytes": tokens + small + 2 * states, "flops": N * D * (7 * S + 12)}


# --------------------------------------------------------- the definitions, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    return {"conv": _exact_conv, "scan": _exact_scan, "norm": _exact_norm}[case["op"]](d, case)


def _exact_conv(d, c):
    D, W = c["dim"], c["width"]

    def one(x, past, w, bias):
        line = torch.cat([past, x])
        pre = torch.nn.functional.conv1d(line.t()[None], w[:, None], bias, groups=D)[0].t() if x.shape[0] else x
        return (torch.nn.functional.silu(pre) if c["act"] else pre), line[line.shape[0] - (W - 1):]

    if c["dir"] == "step":
        outs, finals = zip(*[one(d["x"][i], d["state"][i], d["weight"], d["bias"]) for i in range(c["batch"])])
        return torch.stack(outs), torch.stack(finals)
    cu, n = _offsets(c), len(_lengths(c))
    lead = d["x"].shape[:2]
    x = d["x"].reshape(-1, D)
    past = d["state"] if d["state"] is not None else torch.zeros(n, W - 1, D, device="cuda", dtype=torch.float64)
    w, bias = d["weight"], d["bias"]
    if c["dir"] == "bwd":
        x, past, w = (v.detach().requires_grad_() for v in (x, past, w))
        bias = bias.detach().requires_grad_() if bias is not None else None
    outs, finals = zip(*[one(x[cu[i]:cu[i + 1]], past[i], w, bias) for i in range(n)])
    out, final = torch.cat(outs), torch.stack(finals)
    if c["dir"] == "fwd":
        return out.reshape(*lead, D), final
    loss = (out * d["d_out"].reshape(-1, D)).sum()
    if d["d_final"] is not None:
        loss = loss + (final * d["d_final"]).sum()
    loss.backward()
    return _kept((x.grad.reshape(*lead, D), w.grad, bias.grad if bias is not None else None, past.grad if past.grad is not None else torch.zeros_like(past)))


def _exact_scan(d, c):
    D, S, G = c["dim"], c["states"], c["groups"]
    lead = d["u"].shape[:2]
    per = D // G
    u, Bm, Cm = d["u"].reshape(-1, D), d["Bm"].reshape(-1, G, 1, S), d["Cm"].reshape(-1, G, 1, S)
    raw = d["delta"].reshape(-1, D) + d["delta_bias"]
    step = torch.nn.functional.softplus(raw, threshold=60.0)
    z = d["z"].reshape(-1, D) if d["z"] is not None else None
    A, skip = d["A"], d["D"]
    lens = [1] * c["batch"] if c["dir"] == "step" else _lengths(c)
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    n, longest = len(lens), max(lens)
    dev = {"device": "cuda", "dtype": torch.float64}
    past = (d["state"] if d["state"] is not None else torch.zeros(n, D, S, **dev))[order]
    first = torch.tensor([cu[i] for i in order], device="cuda")
    active = [sum(x > p for x in lens) for p in range(longest)]  # sequences, longest first, that have token p
    y = torch.zeros(u.shape[0], D, **dev)
    h, hist = past.clone(), []
    for p in range(longest):
        m = active[p]
        at = first[:m] + p
        dt, x = step[at], u[at]
        h[:m] = torch.exp(dt[..., None] * A) * h[:m] + ((dt * x).view(m, G, per, 1) * Bm[at]).view(m, D, S)
        y[at] = (h[:m].view(m, G, per, S) * Cm[at]).sum(-1).view(m, D)
        if c["dir"] == "bwd":
            hist.append(h[:m].clone())
    if skip is not None:
        y = y + skip * u
    back = torch.argsort(torch.tensor(order, device="cuda"))
    if c["dir"] != "bwd":
        out = y if z is None else y * torch.nn.functional.silu(z)
        return out.reshape(*lead, D), h[back]
    dout = d["d_out"].reshape(-1, D)
    sg = torch.sigmoid(z) if z is not None else None
    dy = dout if z is None else dout * z * sg
    dz = None if z is None else (dout * y * (sg + z * sg * (1 - sg))).reshape(*lead, D)
    dh = d["d_final"][order].clone() if d["d_final"] is not None else torch.zeros(n, D, S, **dev)
    du, ddt = dy * (skip if skip is not None else 0.0), torch.zeros_like(u)
    dA, dB, dC = torch.zeros_like(A), torch.zeros(u.shape[0], G, S, **dev), torch.zeros(u.shape[0], G, S, **dev)
    for p in range(longest - 1, -1, -1):
        m = active[p]
        at = first[:m] + p
        dt, x, g = step[at], u[at], dy[at]
        dC[at] = (g.view(m, G, per, 1) * hist[p].view(m, G, per, S)).sum(2)
        now = dh[:m] + (g.view(m, G, per, 1) * Cm[at]).view(m, D, S)
        dB[at] = ((dt * x)[..., None] * now).view(m, G, per, S).sum(2)
        into = (now.view(m, G, per, S) * Bm[at]).sum(-1).view(m, D)
        du[at] += into * dt
        decay = torch.exp(dt[..., None] * A)
        old = hist[p - 1][:m] if p else past[:m]
        rate = now * decay * old
        dA += (rate * dt[..., None]).sum(0)
        ddt[at] = (rate * A).sum(-1) + into * x
        dh[:m] = now * decay
        hist[p] = None if p else hist[p]
    ddelta = ddt * torch.sigmoid(raw)
    return _kept((du.reshape(*lead, D), ddelta.reshape(*lead, D), dA, dB.reshape(*lead, G, S), dC.reshape(*lead, G, S),
                  (dy * u).sum(0) if skip is not None else None, dz, ddelta.sum(0), dh[back]))


def _exact_norm(d, c):
    names = ("x", "gate", "residual", "post_weight", "scale", "pre_weight")
    v = {k: d[k].detach().requires_grad_(c["dir"] == "bwd") if d[k] is not None else None for k in names}
    act = {"": None, "sigmoid": torch.sigmoid, "silu": torch.nn.functional.silu}[c["gate"]]

    def rms(x, w):
        return x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w

    p = v["x"]
    if act and c["first"]:
        p = p * act(v["gate"])
    if v["post_weight"] is not None:
        p = rms(p, v["post_weight"])
    if act and not c["first"]:
        p = p * act(v["gate"])
    if v["scale"] is not None:
        p = p * v["scale"]
    if v["residual"] is not None:
        p = p + v["residual"]
    normed = rms(p, v["pre_weight"]) if v["pre_weight"] is not None else None
    if c["dir"] == "fwd":
        return _kept((p, normed))
    loss = (p * d["d_out"]).sum()
    if normed is not None:
        loss = loss + (normed * d["d_normed"]).sum()
    loss.backward()
    return _kept(tuple(v[k].grad if v[k] is not None else None for k in names))
