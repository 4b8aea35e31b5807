"""kda_block_norm_fwd / _bwd against the 64-bit reference."""
import ctypes
import threading

import pytest
import torch

import layer_ref as R
from gated_delta_rule_156_b200 import kda as K

pytestmark = pytest.mark.gpu
DEV = "cuda"
IO = {"bf16": torch.bfloat16, "f32": torch.float32}
# fp32: the mean's sum (pairwise over lanes, at most 32 terms in a row), the
# reciprocal root, the gate's exp and quotient, and five products
TOL = 48 * 2.0 ** -24
NAMES = ("x", "post_weight", "gate", "residual", "scale", "pre_weight")
OUT = ("x", "gate", "residual", "post_weight", "scale", "pre_weight")


def make(lead, io, res, seed, parts="pgrsn", sliced=False):
    """parts: p post_weight, g gate, r residual, s scale, n pre_weight."""
    g = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*s):
        return torch.randn(s, generator=g, device=DEV)
    dt, rt = IO[io], IO[res]
    w = lead[-1]
    if sliced:
        x = randn(*lead[:-1], 2 * w).to(dt)[..., :w] if len(lead) == 2 else \
            randn(lead[0], 2, *lead[1:]).to(dt)[:, 1]
        gate = randn(lead[0], 3, *lead[1:]).to(dt)[:, 2]
    else:
        x, gate = randn(*lead).to(dt), randn(*lead).to(dt)
    d = dict(x=x * 1, gate=gate if "g" in parts else None,
             residual=randn(*lead).to(rt) if "r" in parts else None,
             post_weight=1 + 0.2 * randn(w) if "p" in parts else None,
             scale=0.5 + 0.2 * randn(w) if "s" in parts else None,
             pre_weight=1 + 0.2 * randn(w) if "n" in parts else None)
    d["x"] = x
    d["d_out"] = randn(*lead).to(rt if "r" in parts else dt)
    d["d_normed"] = randn(*lead).to(dt) if "n" in parts else None
    return d


def compare(d, act="sigmoid", first=False, eps=1e-6):
    ins = [R.h64(d[n]) for n in NAMES]

    def fn(*a):
        return R.block_norm(*a, act, first, eps)
    out_r, normed_r = fn(*ins)
    kw = {n: d[n] for n in NAMES[1:]}
    kw.update(gate_act=act, gate_first=first, eps=eps)
    out, normed = K.block_norm_fwd(d["x"], **kw)
    R.check("out", out, out_r, TOL)
    if normed_r is not None:
        R.check("normed", normed, normed_r, TOL)
    d_outs = R.h64(d["d_out"]), R.h64(d["d_normed"])
    ref = dict(zip(NAMES, R.grads(fn, ins, d_outs)))
    # a norm's gradient r (v - hat mean(v hat)) is the difference of two
    # terms, each rounded relative to itself: with width 1 they cancel to
    # eps / (x^2 + eps) of their size, so the error is held against r v, the
    # gradient with the root held fixed
    terms = dict(zip(NAMES, R.grads(lambda *a: R.block_norm(
        *a, act, first, eps, hold=True), ins, d_outs)))
    got = dict(zip(OUT, K.block_norm_bwd(d["x"], d_out=d["d_out"],
                                         d_normed=d["d_normed"], **kw)))
    torch.cuda.synchronize()
    rows = d["x"].numel() // d["x"].shape[-1]
    for n in OUT:
        if d[n] is None:
            assert got[n] is None
        else:
            # sums over rows: rounding grows with the root of their number
            t = 2 * TOL if n in ("x", "gate", "residual") else \
                2 * TOL + rows ** 0.5 * 2.0 ** -24
            R.check("d " + n, got[n], ref[n], t, terms=terms[n])


@pytest.mark.parametrize("io,res", [("bf16", "bf16"), ("bf16", "f32"),
                                    ("f32", "f32")])
@pytest.mark.parametrize("rows,width", [
    (1, 1), (3, 7), (70, 64), (5, 100), (9, 256), (33, 1001), (4, 4096),
    (300, 512), (2, 8192), (3, 5000), (2, 16384), (2, 16383)])
def test_block(io, res, rows, width):
    compare(make((rows, width), io, res, rows + width))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,heads,width", [(1, 1, 128), (7, 4, 128),
                                                (65, 3, 64), (40, 5, 96),
                                                (13, 2, 33), (600, 8, 32)])
@pytest.mark.parametrize("act,first", [("sigmoid", False), ("silu", True),
                                       ("silu", False), ("none", False)])
def test_gated_heads(io, tokens, heads, width, act, first):
    d = make((tokens, heads, width), io, io, tokens + width, "pg", sliced=True)
    compare(d, act, first)


@pytest.mark.parametrize("parts", ["", "p", "g", "r", "s", "n", "rn", "pg",
                                   "gr", "rs", "prn", "gs", "pgrs", "sn"])
@pytest.mark.parametrize("first", [False, True])
def test_parts(parts, first):
    compare(make((37, 136), "bf16", "bf16", 3, parts), "silu", first)


def test_bf16_parts_with_fp32_out():
    # no residual, but an fp32 out asked for
    d = make((20, 64), "bf16", "f32", 5, "pg")
    out = torch.empty(20, 64, device=DEV)
    K.block_norm_fwd(d["x"], d["post_weight"], d["gate"], out=out)
    ref, _ = R.block_norm(*(R.h64(d[n]) for n in NAMES), "sigmoid", False, 1e-6)
    R.check("out", out, ref, TOL)


def test_zero_rows_and_eps():
    d = make((6, 72), "f32", "f32", 8)
    d["x"][2] = 0
    d["x"][3] = 0
    d["residual"][3] = 0       # a row whose both norms are of zeros
    compare(d, eps=1e-5)
    # eps 0 and no zero row: absent rows of the block must not disturb sums
    d = make((3, 40), "f32", "f32", 9)
    compare(d, eps=0.0)


def test_large_values():
    # squares up to 1e30 stay finite in fp32
    d = make((5, 256), "f32", "f32", 4)
    d["x"] *= 1e15
    compare(d)


def test_no_rows():
    d = make((0, 64), "bf16", "f32", 1)
    kw = {n: d[n] for n in NAMES[1:]}
    out, normed = K.block_norm_fwd(d["x"], **kw)
    assert out.shape == (0, 64) and normed.shape == (0, 64)
    got = dict(zip(OUT, K.block_norm_bwd(d["x"], d_out=d["d_out"],
                                         d_normed=d["d_normed"], **kw)))
    for n in ("post_weight", "scale", "pre_weight"):
        assert (got[n] == 0).all()


def test_missing_gradients_are_zero():
    d = make((20, 128), "bf16", "bf16", 2)
    kw = {n: d[n] for n in NAMES[1:]}
    z, zn = torch.zeros_like(d["d_out"]), torch.zeros_like(d["d_normed"])
    for a, b in (((d["d_out"], None), (d["d_out"], zn)),
                 ((None, d["d_normed"]), (z, d["d_normed"])),
                 ((None, None), (z, zn))):
        x = K.block_norm_bwd(d["x"], d_out=a[0], d_normed=a[1], **kw)
        y = K.block_norm_bwd(d["x"], d_out=b[0], d_normed=b[1], **kw)
        assert all(torch.equal(p, q) for p, q in zip(x, y))


@pytest.mark.parametrize("io,res", [("bf16", "f32"), ("bf16", "bf16")])
def test_residual_in_place(io, res):
    d = make((50, 1000), io, res, 6)
    kw = {n: d[n] for n in NAMES[1:]}
    out, normed = K.block_norm_fwd(d["x"], **kw)
    r = d["residual"].clone()
    kw["residual"] = r
    out2, normed2 = K.block_norm_fwd(d["x"], out=r, **kw)
    assert out2 is r and torch.equal(out, r) and torch.equal(normed, normed2)


def test_misaligned_rows_match_aligned():
    d = make((20, 64), "bf16", "bf16", 7)
    wide = torch.zeros(20, 73, dtype=torch.bfloat16, device=DEV)
    x = wide[:, 3:67]
    x.copy_(d["x"])
    kw = {n: d[n] for n in NAMES[1:]}
    a, b = K.block_norm_fwd(d["x"], **kw), K.block_norm_fwd(x, **kw)
    # the sums' order differs
    for p, q in zip(a, b):
        R.check("out", q, p.cpu().double(), 2 * TOL + 2.0 ** -8)


def test_non_finite_inputs_stay_in_their_row():
    d = make((9, 200), "f32", "f32", 9)
    d["x"][4, 7] = float("nan")
    d["residual"][6, 3] = float("inf")
    kw = {n: d[n] for n in NAMES[1:]}
    out, normed = K.block_norm_fwd(d["x"], **kw)
    ok = [i for i in range(9) if i not in (4, 6)]
    assert torch.isfinite(out[ok]).all() and torch.isfinite(normed[ok]).all()
    assert torch.isnan(out[4]).all() and torch.isinf(out[6, 3])


def test_rows_past_32_bits():
    # rows whose elements lie past 2^31
    n, w = 70000, 64
    wide = torch.empty(n, 1 << 15, dtype=torch.bfloat16, device=DEV)
    x = wide[:, 512:512 + w]
    x.copy_(torch.randn(n, w, device=DEV))
    p = 1 + 0.1 * torch.randn(w, device=DEV)
    a, _ = K.block_norm_fwd(x, p)
    b, _ = K.block_norm_fwd(x.contiguous(), p)
    assert torch.equal(a, b)


def test_repeats_are_bit_identical():
    d = make((3000, 256), "bf16", "bf16", 4)
    kw = {n: d[n] for n in NAMES[1:]}
    a = K.block_norm_bwd(d["x"], d_out=d["d_out"], d_normed=d["d_normed"], **kw)
    for _ in range(3):
        b = K.block_norm_bwd(d["x"], d_out=d["d_out"], d_normed=d["d_normed"],
                             **kw)
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_refusals():
    d = make((4, 64), "bf16", "bf16", 1)
    kw = {n: d[n] for n in NAMES[1:]}
    bad = [
        lambda: K.block_norm_fwd(d["x"].t(), **kw),
        lambda: K.block_norm_fwd(d["x"], **{**kw, "scale": d["scale"][:3]}),
        lambda: K.block_norm_fwd(d["x"], **{**kw, "gate": d["gate"].float()}),
        lambda: K.block_norm_fwd(d["x"], **{**kw, "residual": d["residual"].half()}),
        lambda: K.block_norm_fwd(d["x"].float(), residual=d["residual"]),
        lambda: K.block_norm_fwd(d["x"], normed=torch.empty_like(d["x"])),
        lambda: K.block_norm_fwd(d["x"], eps=-1.0),
        lambda: K.block_norm_fwd(d["x"], out=d["x"]),
        lambda: K.block_norm_bwd(d["x"], d_normed=d["d_normed"]),
        lambda: K.block_norm_fwd(torch.zeros(2, 16385, device=DEV)),
        lambda: K.block_norm_fwd(torch.zeros(2, 0, device=DEV)),
    ]
    for f in bad:
        with pytest.raises((ValueError, K.KdaError)):
            f()


@pytest.mark.parametrize("widths,act", [((4096, 2048), "sigmoid"),
                                        ((8192, 6000), "none")])
def test_threads_with_different_widths(widths, act):
    # host threads in the same kernel with different amounts of shared memory:
    # what one call allows the kernel must not be taken back by another before
    # its launch.  The C calls alone, on prepared arguments, so that the
    # threads are inside them (and without the interpreter's lock) most of the
    # time
    lib, calls, outs, want = K.library(), [], [], []
    for w in widths:
        d = make((64, w), "bf16", "bf16", w)
        ins = [d[n] for n in NAMES] + [d["d_out"], d["d_normed"]]
        kw = dict({n: d[n] for n in NAMES[1:]}, gate_act=act)
        want.append(K.block_norm_bwd(d["x"], d_out=d["d_out"],
                                     d_normed=d["d_normed"], **kw))
        shape, _ = K._norm_shape(*ins[:6], torch.bfloat16, act, False, 1e-6)
        for _ in range(2):  # two threads of each width
            got = [torch.empty_like(t) for t in want[-1]]
            outs.append((got, want[-1]))
            calls.append((ctypes.byref(shape),
                          *[t.data_ptr() for t in ins + got],
                          torch.cuda.Stream(), ins))
    torch.cuda.synchronize()
    failed, start = [], threading.Barrier(len(calls))

    def work(*args, stream, keep):
        start.wait()
        for _ in range(5000):
            st = lib.kda_block_norm_bwd(*args, stream.cuda_stream)
            if st != K.KDA_OK:
                failed.append(st)
                return
        stream.synchronize()

    threads = [threading.Thread(target=work, args=c[:-2],
                                kwargs=dict(stream=c[-2], keep=c[-1]))
               for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, [K.STATUS_NAMES[s] for s in failed]
    torch.cuda.synchronize()
    for got, ref in outs:
        assert all(torch.equal(p, q) for p, q in zip(got, ref))
