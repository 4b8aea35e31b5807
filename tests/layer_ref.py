"""The layer operators' definitions in 64 bits on the CPU, token by token and
differentiable: the reference of the short convolution, the selective scan and
the block norm.  Inputs are double tensors; ``offsets`` are the sequences'
token offsets (host ints)."""
import torch

# Half a rounding step, relative to the value.
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def h64(t):
    return None if t is None else t.detach().cpu().double()


def offsets_of(B, T, lengths=None):
    if lengths is None:
        return [i * T for i in range(B + 1)]
    o = [0]
    for n in lengths:
        o.append(o[-1] + n)
    return o


def act(x, name):
    if name == "none":
        return x
    s = 1 / (1 + torch.exp(-x))
    return s if name == "sigmoid" else x * s


def short_conv(x, weight, bias, past, offsets, activation):
    """x [tokens, D], past [n, W-1, D] or None -> (out, final_state)."""
    W, D = weight.shape[1], x.shape[1]
    outs, finals = [], []
    for s in range(len(offsets) - 1):
        before = past[s] if past is not None else x.new_zeros(W - 1, D)
        line = torch.cat([before, x[offsets[s]:offsets[s + 1]]])
        n = line.shape[0] - (W - 1)
        pre = sum(line[j:j + n] * weight[:, j] for j in range(W))
        if bias is not None:
            pre = pre + bias
        outs.append(act(pre, activation))
        finals.append(line[n:])
    return torch.cat(outs), torch.stack(finals)


def ssm_scan(u, delta, A, Bm, Cm, D, z, delta_bias, past, offsets, softplus):
    """u, delta, z [tokens, D]; Bm, Cm [tokens, G, S]; past [n, D, S] or None
    -> (out, final_state)."""
    dim, per = u.shape[1], u.shape[1] // Bm.shape[1]
    raw = delta if delta_bias is None else delta + delta_bias
    step = torch.log1p(torch.exp(-raw.abs())) + raw.clamp(min=0) \
        if softplus else raw
    outs, finals = [], []
    for s in range(len(offsets) - 1):
        h = past[s] if past is not None else u.new_zeros(dim, A.shape[1])
        for t in range(offsets[s], offsets[s + 1]):
            b = Bm[t].repeat_interleave(per, 0)
            c = Cm[t].repeat_interleave(per, 0)
            h = torch.exp(step[t][:, None] * A) * h + \
                (step[t] * u[t])[:, None] * b
            y = (h * c).sum(1)
            if D is not None:
                y = y + D * u[t]
            if z is not None:
                y = y * act(z[t], "silu")
            outs.append(y)
        finals.append(h)
    out = torch.stack(outs) if outs else u[:0]
    return out, torch.stack(finals)


def block_norm(x, post_weight, gate, residual, scale, pre_weight, gate_act,
               gate_first, eps, hold=False):
    """``hold``: no gradient through the norms' roots (see check's level)."""
    def rms(v, w):
        root = torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
        return v / (root.detach() if hold else root) * w

    p = x
    if gate is not None and gate_first:
        p = p * act(gate, gate_act)
    if post_weight is not None:
        p = rms(p, post_weight)
    if gate is not None and not gate_first:
        p = p * act(gate, gate_act)
    if scale is not None:
        p = p * scale
    out = p if residual is None else residual + p
    return out, None if pre_weight is None else rms(out, pre_weight)


def grads(fn, inputs, d_outs):
    """Gradients of sum(d_out * out) at every tensor of ``inputs`` (None where
    the input is None)."""
    leaves = [None if t is None else t.clone().requires_grad_()
              for t in inputs]
    outs = fn(*leaves)
    loss = sum((o * d).sum() for o, d in zip(outs, d_outs)
               if o is not None and d is not None)
    got = torch.autograd.grad(loss, [t for t in leaves if t is not None],
                              allow_unused=True)
    got = iter(got)
    return [None if t is None else
            (lambda g: torch.zeros_like(t) if g is None else g)(next(got))
            for t in leaves]


def check(name, got, ref, tol, dtype=None, terms=None):
    """Relative L2 over the whole tensor, and each element against the larger
    of itself and the tensor's root mean square, plus half a rounding step of
    the output's type.  ``terms``: the size of the terms whose difference ref
    is; rounding is relative to them where they are larger."""
    got = got.detach().cpu()
    dtype = dtype or got.dtype
    got, ref = got.double(), ref.detach()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{name}: not finite"
    if not ref.numel():
        return
    tol = tol + HALF[dtype]
    err, norm = (got - ref).norm(), ref.norm()
    if terms is not None:
        norm = torch.maximum(norm, terms.norm())
    if norm == 0:
        assert err == 0, f"{name}: {float(err):.3e} where all is zero"
        return
    assert err <= tol * norm + 1e-30, \
        f"{name}: rel-L2 {float(err / norm):.3e} > {tol:.2e}"
    rms = norm / ref.numel() ** 0.5
    worst = ((got - ref).abs() / torch.maximum(ref.abs(), rms)).max()
    # one element: the fp32 sums are off relative to their terms, a few times
    # the tensor's level at most
    assert worst <= HALF[dtype] + 16 * tol, \
        f"{name}: worst element {float(worst):.3e} (tol {tol:.2e})"
