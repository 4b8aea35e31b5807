"""kda_short_conv_fwd / _bwd / _step against the 64-bit reference."""
import pytest
import torch

import layer_ref as R
from gated_delta_rule_156_b200 import kda as K

pytestmark = pytest.mark.gpu
DEV = "cuda"
IO = {"bf16": torch.bfloat16, "f32": torch.float32}
# fp32 sums of W + 1 terms, the activation through exp and a quotient
# (a few units of 2^-24 of the largest term each)
TOL = 24 * 2.0 ** -24
# the weights' gradients also sum over tokens: rounding errors of partial sums
# grow with the square root of the count, at most 2^-24 sqrt(tokens) here
TOL_W = 40 * 2.0 ** -24


def make(lead, D, W, io, seed, sliced=False, bias=True, past=None):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*s):
        return torch.randn(s, generator=g, device=DEV)
    dt = IO[io]
    x = randn(*lead, 3 * D).to(dt)[..., D:2 * D] if sliced else \
        randn(*lead, D).to(dt)
    return dict(x=x, weight=randn(D, W) * 0.5,
                bias=randn(D) * 0.1 if bias else None,
                past=randn(past, W - 1, D).to(dt) if past else None,
                d_out=randn(*lead, D).to(dt),
                d_final=randn(past or lead[0], W - 1, D).to(dt))


def reference(d, offsets, act, grad=True):
    D = d["x"].shape[-1]
    flat = R.h64(d["x"]).reshape(-1, D)
    ins = [flat, R.h64(d["weight"]), R.h64(d["bias"]), R.h64(d["past"])]

    def fn(x, w, b, p):
        return R.short_conv(x, w, b, p, offsets, act)
    outs = fn(*ins)
    if not grad:
        return outs
    if ins[3] is None:
        ins[3] = torch.zeros(len(offsets) - 1, d["weight"].shape[1] - 1, D,
                             dtype=torch.float64)
    return outs, R.grads(fn, ins, (R.h64(d["d_out"]).reshape(-1, D),
                                   R.h64(d["d_final"])))


def compare(d, offsets, cu, act):
    (out_r, fin_r), (dx_r, dw_r, db_r, dp_r) = reference(d, offsets, act)
    out, fin = K.short_conv_fwd(d["x"], d["weight"], d["bias"], d["past"], cu,
                                activation=act)
    dx, dw, db, dp = K.short_conv_bwd(d["x"], d["weight"], d["bias"],
                                      d["past"], cu, d["d_out"], d["d_final"],
                                      activation=act)
    torch.cuda.synchronize()
    D = d["x"].shape[-1]
    R.check("out", out.reshape(-1, D), out_r, TOL)
    assert torch.equal(fin.cpu().double(), fin_r)  # copies of inputs
    R.check("dx", dx.reshape(-1, D), dx_r, TOL)
    R.check("dw", dw, dw_r, TOL_W)
    if db is not None:
        R.check("db", db, db_r, TOL_W)
    R.check("d_initial_state", dp, dp_r, TOL)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D,W,act,sliced,bias,state", [
    (1, 1, 8, 4, "silu", False, True, False),      # one token
    (2, 3, 16, 4, "silu", False, False, True),     # shorter than the taps
    (2, 130, 64, 4, "silu", True, True, True),
    (1, 77, 37, 3, "none", False, True, True),     # odd channels: single loads
    (3, 65, 40, 2, "silu", True, True, False),
    (2, 300, 1000, 4, "silu", False, True, False),
    (1, 1025, 24, 3, "silu", False, False, True)])
def test_dense(io, B, T, D, W, act, sliced, bias, state):
    d = make((B, T), D, W, io, B + T + D, sliced, bias, B if state else None)
    compare(d, R.offsets_of(B, T), None, act)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("D,state", [(64, True), (33, True), (64, False)])
def test_packed(io, W, D, state):
    lens = [0, 1, 2, 3, 0, 40, 16, 5, 257, 0]
    offs = R.offsets_of(0, 0, lens)
    cu = torch.tensor(offs, dtype=torch.int32, device=DEV)
    d = make((1, offs[-1]), D, W, io, W * D, True, True,
             len(lens) if state else None)
    if not state:
        d["d_final"] = torch.zeros(len(lens), W - 1, D, dtype=IO[io],
                                   device=DEV).normal_()
    compare(d, offs, cu, "silu")


def test_tokens_of_no_sequence_are_left_alone():
    # offsets 3 .. 20 of 32 tokens: the others are not read and not written
    offs = [3, 10, 10, 20]
    cu = torch.tensor(offs, dtype=torch.int32, device=DEV)
    d = make((1, 32), 24, 4, "bf16", 5)
    nan = torch.full_like(d["x"], float("nan"))
    x = nan.clone()
    x[:, 3:20] = d["x"][:, 3:20]
    out = torch.full_like(x, 7.0)
    _, fin = K.short_conv_fwd(x, d["weight"], d["bias"], None, cu, out=out)
    out2, fin2 = K.short_conv_fwd(d["x"][:, 3:20].contiguous(), d["weight"],
                                  d["bias"], None,
                                  torch.tensor([0, 7, 7, 17], dtype=torch.int32,
                                               device=DEV))
    assert torch.equal(out[:, 3:20], out2) and torch.equal(fin, fin2)
    assert (out[:, :3] == 7).all() and (out[:, 20:] == 7).all()
    dy = nan.clone()
    dy[:, 3:20] = d["d_out"][:, 3:20]
    a = K.short_conv_bwd(x, d["weight"], d["bias"], None, cu, dy)
    b = K.short_conv_bwd(d["x"][:, 3:20].contiguous(), d["weight"], d["bias"],
                         None, torch.tensor([0, 7, 7, 17], dtype=torch.int32,
                                            device=DEV),
                         d["d_out"][:, 3:20].contiguous())
    assert torch.equal(a[0][:, 3:20], b[0])
    # the runs of tokens are cut elsewhere, so the sums' order differs
    R.check("dw", a[1], b[1].cpu().double(), TOL_W)
    R.check("db", a[2], b[2].cpu().double(), TOL_W)


def test_no_tokens():
    d = make((2, 0), 16, 4, "bf16", 1, past=2)
    out, fin = K.short_conv_fwd(d["x"], d["weight"], d["bias"], d["past"])
    assert out.shape == (2, 0, 16) and torch.equal(fin, d["past"])
    dx, dw, db, dp = K.short_conv_bwd(d["x"], d["weight"], d["bias"],
                                      d["past"], None, d["d_out"],
                                      d["d_final"])
    assert (dw == 0).all() and (db == 0).all()
    assert torch.equal(dp, d["d_final"])
    d = make((0, 5), 16, 4, "bf16", 1)
    out, fin = K.short_conv_fwd(d["x"], d["weight"])
    assert out.shape == (0, 5, 16) and fin.shape == (0, 3, 16)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N,T,D,W", [(1, 1, 8, 4), (5, 1, 37, 3), (33, 3, 64, 2),
                                     (256, 1, 1000, 4), (3, 9, 24, 4)])
def test_step(io, N, T, D, W):
    d = make((N, T), D, W, io, N + T + D, True, True, N)
    state = d["past"].clone()
    out = K.short_conv_step(d["x"], d["weight"], d["bias"], state)
    out_r, fin_r = reference(d, R.offsets_of(N, T), "silu", grad=False)
    R.check("out", out.reshape(-1, D), out_r, TOL)
    assert torch.equal(state.cpu().double(), fin_r)
    # the same as the prompt kernel's tokens
    out2, fin2 = K.short_conv_fwd(d["x"], d["weight"], d["bias"], d["past"])
    assert torch.equal(out, out2) and torch.equal(state, fin2)


def test_misaligned_slices_match_aligned():
    d = make((2, 50), 64, 4, "bf16", 3, past=2)
    wide = torch.zeros(2, 50, 64 + 7, dtype=torch.bfloat16, device=DEV)
    wide[..., 3:67] = d["x"]
    a = K.short_conv_fwd(d["x"], d["weight"], d["bias"], d["past"])
    b = K.short_conv_fwd(wide[..., 3:67], d["weight"], d["bias"], d["past"])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a = K.short_conv_bwd(d["x"], d["weight"], d["bias"], d["past"], None,
                         d["d_out"])
    b = K.short_conv_bwd(wide[..., 3:67], d["weight"], d["bias"], d["past"],
                         None, d["d_out"])
    assert torch.equal(a[0], b[0])


def test_non_finite_inputs_stay_where_they_are():
    d = make((2, 40), 16, 4, "f32", 9)
    d["x"][1, 20, 5] = float("nan")
    d["x"][0, 10, 3] = float("inf")
    out, _ = K.short_conv_fwd(d["x"], d["weight"], d["bias"])
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[1, 20:24, 5] = True
    want[0, 10:14, 3] = True
    assert not (bad & ~want).any()      # silu of -inf is 0 or NaN, of inf inf
    assert bad[1, 20:24, 5].all()


def test_offsets_past_32_bits():
    # a slice whose last token lies past 2^31 elements
    stride, T, D = 1 << 17, 20000, 64
    wide = torch.empty(1, T, stride, dtype=torch.bfloat16, device=DEV)
    x = wide[..., 1000:1000 + D]
    x.copy_(torch.randn(1, T, D, device=DEV))
    w = torch.randn(D, 4, device=DEV)
    a = K.short_conv_fwd(x, w)
    b = K.short_conv_fwd(x.contiguous(), w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_repeats_are_bit_identical():
    d = make((2, 700), 96, 4, "bf16", 4, past=2)
    a = K.short_conv_bwd(d["x"], d["weight"], d["bias"], d["past"], None,
                         d["d_out"], d["d_final"])
    for _ in range(3):
        b = K.short_conv_bwd(d["x"], d["weight"], d["bias"], d["past"], None,
                             d["d_out"], d["d_final"])
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_refusals():
    d = make((2, 10), 16, 4, "bf16", 1)
    bad = [
        lambda: K.short_conv_fwd(d["x"].transpose(1, 2), d["weight"]),
        lambda: K.short_conv_fwd(d["x"], d["weight"].bfloat16()),
        lambda: K.short_conv_fwd(d["x"], d["weight"][:8]),
        lambda: K.short_conv_fwd(d["x"], d["weight"], d["bias"][:8]),
        lambda: K.short_conv_fwd(d["x"].half(), d["weight"]),
        lambda: K.short_conv_fwd(d["x"][:, :5], d["weight"]),  # two strides
        lambda: K.short_conv_fwd(d["x"], d["weight"], None,
                                 torch.zeros(2, 4, 16, device=DEV)),
        lambda: K.short_conv_bwd(d["x"], d["weight"], None, None, None,
                                 d["d_out"].float()),
        lambda: K.short_conv_fwd(d["x"], d["weight"], cu_seqlens=torch.tensor(
            [0, 10], dtype=torch.int32, device=DEV)),          # B = 2
        lambda: K.short_conv_fwd(d["x"], d["weight"].cpu()),
    ]
    for f in bad:
        with pytest.raises((ValueError, K.KdaError)):
            f()
    with pytest.raises(K.KdaError, match="UNSUPPORTED"):
        K.short_conv_fwd(d["x"], torch.zeros(16, 5, device=DEV))
    with pytest.raises(KeyError):
        K.short_conv_fwd(d["x"], d["weight"], activation="gelu")
