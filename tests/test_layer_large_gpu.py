"""The layer operators at sizes whose kernels take their long runs: rings and
slots that wrap, blocks that meet many rows, four sequences a thread.  Against
the 64-bit reference, on the GPU."""
import pytest
import torch

import layer_ref as R
from gated_delta_rule_156_b200 import kda as K

pytestmark = pytest.mark.gpu
DEV = "cuda"
IO = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 2.0 ** -24


def d64(t):
    return None if t is None else t.detach().double()


def check(name, got, ref, tol, terms=None):
    """As R.check, where the tensors are: relative L2, and each element against
    the larger of itself and the root mean square."""
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{name}: not finite"
    half = R.HALF[got.dtype]
    tol = tol + half
    got, ref = got.detach().double(), ref.detach()
    norm = ref.norm() if terms is None else torch.maximum(ref.norm(),
                                                          terms.norm())
    err = (got - ref).norm()
    assert err <= tol * norm + 1e-30, \
        f"{name}: rel-L2 {float(err / norm):.3e} > {tol:.2e}"
    rms = norm / ref.numel() ** 0.5
    worst = ((got - ref).abs() / torch.maximum(ref.abs(), rms + 1e-30)).max()
    assert worst <= half + 16 * tol, \
        f"{name}: worst element {float(worst):.3e} (tol {tol:.2e})"


def maker(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return lambda *s: torch.randn(s, generator=g, device=DEV)


# ---- convolution ---------------------------------------------------------

# W + 1 products and the activation, as in the small tests; the weights'
# gradients also sum over tokens: a thread's 64, then 8 runs, then the blocks,
# with errors of partial sums of independent terms (root of the count each)
TOL_CONV, TOL_W = 24 * EPS, 40 * EPS


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,lens,D,W,act", [
    (2, 5000, None, 4096, 4, "silu"),       # runs of 32 and 64 tokens
    (1, 0, [0, 1, 5000, 63, 3, 2500, 257, 0, 2300], 4096, 4, "silu"),
    (1, 9600, None, 4096, 3, "none"),
    (1, 0, [777, 4500, 2, 0, 901], 3331, 2, "silu"),   # single channels
    (1, 0, [31, 1200, 33, 64, 32, 1300], 4096, 4, "silu")])
def test_conv_long_runs(io, B, T, lens, D, W, act):
    randn, dt = maker(B + T + D + W), IO[io]
    offs = R.offsets_of(B, T, lens)
    n, N = len(offs) - 1, offs[-1]
    lead = (B, T) if lens is None else (1, N)
    cu = None if lens is None else torch.tensor(offs, dtype=torch.int32,
                                                device=DEV)
    x = randn(*lead, D).to(dt)
    w, bias = randn(D, W) * 0.5, randn(D) * 0.1
    past, d_final = randn(n, W - 1, D).to(dt), randn(n, W - 1, D).to(dt)
    d_out = randn(*lead, D).to(dt)
    out, fin = K.short_conv_fwd(x, w, bias, past, cu, activation=act)
    got = K.short_conv_bwd(x, w, bias, past, cu, d_out, d_final,
                           activation=act)
    ins = [d64(x).reshape(N, D), d64(w), d64(bias), d64(past)]

    def fn(*a):
        return R.short_conv(*a, offs, act)
    out_r, fin_r = fn(*ins)
    check("out", out.reshape(N, D), out_r, TOL_CONV)
    assert torch.equal(fin.double(), fin_r)
    del out_r
    ref = R.grads(fn, ins, (d64(d_out).reshape(N, D), d64(d_final)))
    for name, x_, r, tol in zip(("dx", "d_weight", "d_bias", "d_past"),
                                (got[0].reshape(N, D), *got[1:]), ref,
                                (TOL_CONV, TOL_W, TOL_W, TOL_CONV)):
        check(name, x_, r, tol)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N,T,D,W", [(255, 1, 12288, 4), (254, 3, 12288, 2),
                                     (253, 2, 12288, 3), (69, 2, 8999, 4)])
def test_conv_tokens_of_many_sequences(io, N, T, D, W):
    randn, dt = maker(N + T + D), IO[io]
    x = randn(N, T, 2 * D).to(dt)[..., D:]  # D = 8999: at an odd offset
    w, bias, state = randn(D, W) * 0.5, randn(D) * 0.1, \
        randn(N, W - 1, D).to(dt)
    ref = R.short_conv(d64(x).reshape(N * T, D), d64(w), d64(bias),
                       d64(state), R.offsets_of(N, T), "silu")
    out = K.short_conv_step(x, w, bias, state)
    check("out", out.reshape(N * T, D), ref[0], TOL_CONV)
    assert torch.equal(state.double(), ref[1])


# ---- scan ------------------------------------------------------------------

def scan_inputs(lead, D, S, G, io, seed, odd=False):
    """odd: B and C start at odd elements of a wider row."""
    randn, dt = maker(seed), IO[io]
    o = 1 if odd else 0
    bc = randn(*lead, G, 2 * S + 3 * o).to(dt)
    return dict(u=randn(*lead, D).to(dt), delta=(randn(*lead, D) - 1).to(dt),
                A=-torch.exp(randn(D, S) * 0.5), Bm=bc[..., o:S + o],
                Cm=bc[..., S + 2 * o:2 * S + 2 * o], D=randn(D),
                z=randn(*lead, 2 * D).to(dt)[..., D:],
                delta_bias=randn(D) * 0.2)


def scan_flat(d, n):
    return [d64(d[k]) if k in ("A", "D", "delta_bias") else
            d64(d[k]).reshape(n, *d[k].shape[2:])
            for k in ("u", "delta", "A", "Bm", "Cm", "D", "z", "delta_bias")]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N,T,D,S,G,odd", [
    (257, 1, 4096, 16, 1, False), (258, 2, 4096, 16, 2, False),
    (259, 1, 4096, 16, 1, True), (257, 2, 4096, 8, 1, False),
    (255, 1, 4096, 12, 1, False), (257, 1, 4000, 5, 4, True),
    (31, 2, 4096, 64, 1, False), (49, 1, 1024, 128, 1, True)])
def test_scan_tokens_of_many_sequences(io, N, T, D, S, G, odd):
    d = scan_inputs((N, T), D, S, G, io, N + T + D + S, odd)
    state = maker(3)(N, D, S)
    ref = R.ssm_scan(*scan_flat(d, N * T), d64(state), R.offsets_of(N, T),
                     True)
    out = K.ssm_step(d["u"], d["delta"], d["A"], d["Bm"], d["Cm"], state,
                     D=d["D"], z=d["z"], delta_bias=d["delta_bias"])
    # units of 2^-24 a token: the exponential 4, its argument (the step's 11,
    # two roundings) times a decay 5, the input's step 11 and two products 2,
    # the sum 1; then the sum over states, and z's activation
    tol = (23 * T + S ** 0.5 + 8) * EPS
    check("out", out.reshape(N * T, D), ref[0], tol)
    check("state", state, ref[1], tol)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D,S,G", [(4, 200, 2048, 16, 2),
                                       (3, 77, 4096, 8, 1)])
def test_scan_of_many_channels(io, B, T, D, S, G):
    # enough CTAs not to be split, many tiles of each
    d = scan_inputs((B, T), D, S, G, io, B + T + D)
    randn, offs = maker(5), R.offsets_of(B, T)
    past, d_final = randn(B, D, S), randn(B, D, S)
    d_out = randn(B, T, D).to(IO[io])
    kw = dict(D=d["D"], z=d["z"], delta_bias=d["delta_bias"],
              initial_state=past)
    args = (d["u"], d["delta"], d["A"], d["Bm"], d["Cm"])
    ins = scan_flat(d, B * T) + [d64(past)]

    def fn(*a):
        return R.ssm_scan(*a, offs, True)
    out_r, fin_r = fn(*ins)
    # as a token's above; a term lives for at most 64 tokens here (steps of a
    # tenth at least at rates of 0.2 and more), and errors of different tokens
    # are independent
    tol = (23 * 64 ** 0.5 + 16) * EPS
    out, fin = K.ssm_scan_fwd(*args, **kw)
    check("out", out.reshape(B * T, D), out_r, tol)
    check("final_state", fin, fin_r, tol)
    ref = R.grads(fn, ins, (d64(d_out).reshape(B * T, D), d64(d_final)))
    got = K.ssm_scan_bwd(*args, d_out=d_out, d_final_state=d_final, **kw)
    names = ("u", "delta", "A", "Bm", "Cm", "D", "z", "delta_bias", "past")
    for name, x, r in zip(names, got, ref):
        # a gradient meets the states and its own chain
        check("d " + name, x.reshape(r.shape), r, 2 * tol)


# ---- block norm ----------------------------------------------------------

TOL_NORM = 48 * EPS  # as in the small tests
IN = ("x", "post_weight", "gate", "residual", "scale", "pre_weight")
OUT = ("x", "gate", "residual", "post_weight", "scale", "pre_weight")


def norm_case(lead, io, res, parts, act, first, d_outs="on", sliced=False):
    """parts: p post_weight, g gate, r residual, s scale, n pre_weight;
    d_outs: o d_out, n d_normed (None where missing)."""
    randn, dt, rt = maker(sum(lead)), IO[io], IO[res]
    w, has_r = lead[-1], "r" in parts
    x = randn(*lead).to(dt)
    gate = randn(lead[0], 3, *lead[1:]).to(dt)[:, 2] if sliced else \
        randn(*lead).to(dt)
    d = dict(x=x, gate=gate if "g" in parts else None,
             residual=randn(*lead).to(rt) if has_r else None,
             post_weight=1 + 0.2 * randn(w) if "p" in parts else None,
             scale=0.5 + 0.2 * randn(w) if "s" in parts else None,
             pre_weight=1 + 0.2 * randn(w) if "n" in parts else None)
    d_out = randn(*lead).to(rt if has_r else dt) if "o" in d_outs else None
    d_normed = randn(*lead).to(dt) if "n" in parts and "n" in d_outs else None
    kw = {k: d[k] for k in IN[1:]}
    kw.update(gate_act=act, gate_first=first)
    ins = [d64(d[k]) for k in IN]

    def fn(*a, hold=False):
        return R.block_norm(*a, act, first, 1e-6, hold=hold)
    out_r, normed_r = fn(*ins)
    out, normed = K.block_norm_fwd(x, **kw)
    check("out", out, out_r, TOL_NORM)
    if normed is not None:
        check("normed", normed, normed_r, TOL_NORM)
    del out_r, normed_r
    dy = d64(d_out), d64(d_normed)
    ref = dict(zip(IN, R.grads(fn, ins, dy)))
    # the size of the terms whose difference a norm's gradient is
    terms = dict(zip(IN, R.grads(lambda *a: fn(*a, hold=True), ins, dy)))
    got = dict(zip(OUT, K.block_norm_bwd(x, d_out=d_out, d_normed=d_normed,
                                         **kw)))
    rows = x.numel() // w
    for k in OUT:
        if d[k] is None:
            assert got[k] is None
            continue
        # sums over rows: rounding grows with the root of their number
        tol = 2 * TOL_NORM + (0 if k in ("x", "gate", "residual") else
                              rows ** 0.5 * EPS)
        check("d " + k, got[k], ref[k], tol, terms[k])


@pytest.mark.parametrize("parts,act,first,d_outs", [
    ("pgrsn", "sigmoid", False, "on"), ("pgrsn", "silu", False, "on"),
    ("pgrsn", "sigmoid", True, "on"), ("pgrsn", "silu", True, "on"),
    ("prsn", "none", False, "on"), ("pgrsn", "none", False, "on"),
    ("pgn", "silu", False, "on"), ("gr", "silu", False, "o"),
    ("rsn", "none", False, "on"), ("p", "none", False, "o"),
    ("pgrsn", "silu", False, "n"), ("pgrsn", "sigmoid", True, "o")])
@pytest.mark.parametrize("io,res,rows,width", [
    ("bf16", "f32", 1001, 4096), ("bf16", "bf16", 10001, 512),
    ("f32", "f32", 1203, 2048), ("f32", "f32", 10001, 256)])
def test_norm_wide_rows_two_at_a_time(io, res, rows, width, parts, act, first,
                                      d_outs):
    norm_case((rows, width), io, res, parts, act, first, d_outs)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("act,first", [("silu", False), ("sigmoid", True)])
@pytest.mark.parametrize("tokens,heads,width", [(1501, 3, 512),
                                                (6001, 32, 128),
                                                (4003, 5, 33)])
def test_norm_many_heads(io, act, first, tokens, heads, width):
    norm_case((tokens, heads, width), io, io, "pg", act, first, sliced=True)


@pytest.mark.parametrize("io,res", [("bf16", "f32"), ("bf16", "bf16"),
                                    ("f32", "f32")])
@pytest.mark.parametrize("rows,width", [
    (100001, 64), (30001, 136), (9001, 1000), (5001, 1001), (3001, 3690),
    (1001, 6144), (701, 8191), (701, 9000), (601, 16384), (601, 16383)])
def test_norm_many_rows(io, res, rows, width):
    norm_case((rows, width), io, res, "pgrsn", "silu", False)
