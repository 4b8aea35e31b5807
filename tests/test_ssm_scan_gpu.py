"""kda_ssm_scan_fwd / _bwd and kda_ssm_step against the 64-bit reference."""
import pytest
import torch

import layer_ref as R
from gated_delta_rule_156_b200 import kda as K

pytestmark = pytest.mark.gpu
DEV = "cuda"
IO = {"bf16": torch.bfloat16, "f32": torch.float32}


def tol(T):
    """A step of the recurrence multiplies by an exponential good to 2^-22,
    of an argument rounded twice (|step A| <= 4 here: 2^-21), and rounds
    twice: at most 2^-20 of a term's size a step, and a term lives for at most
    T steps.  Terms decay, so half of that for the typical one; 32 steps' worth
    for the sums over states and channels."""
    return (0.5 * T + 32) * 2.0 ** -20


def make(lead, D, S, G, io, seed, z=True, skip=True, bias=True, past=None,
         sliced=True):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*s):
        return torch.randn(s, generator=g, device=DEV)
    dt = IO[io]
    bc = randn(*lead, G, 2 * S).to(dt)
    d = dict(u=randn(*lead, D).to(dt), delta=(randn(*lead, D) - 1).to(dt),
             A=-torch.exp(randn(D, S) * 0.5), Bm=bc[..., :S], Cm=bc[..., S:],
             D=randn(D) if skip else None,
             z=randn(*lead, 2 * D).to(dt)[..., D:] if z else None,
             delta_bias=randn(D) * 0.2 if bias else None,
             past=randn(past, D, S) if past else None,
             d_out=randn(*lead, D).to(dt))
    d["d_final"] = randn(past or lead[0], D, S)
    if not sliced:
        d["Bm"], d["Cm"] = d["Bm"].contiguous(), d["Cm"].contiguous()
        d["z"] = d["z"].contiguous() if z else None
    return d


NAMES = ("u", "delta", "A", "Bm", "Cm", "D", "z", "delta_bias", "past")


def flat64(d):
    n = d["u"].shape[0] * d["u"].shape[1]

    def f(name):
        t = R.h64(d[name])
        return t if t is None or name in ("A", "D", "delta_bias", "past") \
            else t.reshape(n, *t.shape[2:])
    return [f(n) for n in NAMES]


def compare(d, offsets, cu=None, softplus=True):
    T = max(b - a for a, b in zip(offsets, offsets[1:]))
    ins = flat64(d)
    n, D, S = len(offsets) - 1, d["u"].shape[-1], d["A"].shape[1]

    def fn(*x):
        return R.ssm_scan(*x, offsets, softplus)
    out_r, fin_r = fn(*ins)
    kw = dict(D=d["D"], z=d["z"], delta_bias=d["delta_bias"],
              initial_state=d["past"], cu_seqlens=cu, softplus=softplus)
    args = (d["u"], d["delta"], d["A"], d["Bm"], d["Cm"])
    out, fin = K.ssm_scan_fwd(*args, **kw)
    R.check("out", out.reshape(-1, D), out_r, tol(T))
    R.check("final_state", fin, fin_r, tol(T))
    if ins[8] is None:
        ins[8] = torch.zeros(n, D, S, dtype=torch.float64)
    ref = R.grads(fn, ins, (R.h64(d["d_out"]).reshape(-1, D),
                            R.h64(d["d_final"])))
    got = K.ssm_scan_bwd(*args, d_out=d["d_out"], d_final_state=d["d_final"],
                         **kw)
    torch.cuda.synchronize()
    for name, x, r in zip(NAMES, got, ref):
        if x is None:
            assert d[name] is None
            continue
        # a gradient meets the forward's states and its own chain
        R.check("d " + name, x.reshape(r.shape), r, 2 * tol(T))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D,S,G,over", [
    (1, 1, 4, 16, 1, {}),                              # one token
    (2, 7, 32, 16, 1, dict(past=2)),
    (1, 8, 33, 16, 1, dict(z=False)),                  # one chunk, odd channels
    (2, 65, 40, 16, 2, dict(past=2, skip=False)),      # groups of 20 channels
    (1, 100, 70, 1, 1, dict(past=1, bias=False)),      # one state
    (1, 40, 30, 5, 3, dict(past=1)),                   # odd states, 3 groups
    (2, 33, 64, 8, 1, dict(z=False, skip=False, bias=False, sliced=False)),
    (1, 37, 24, 12, 1, dict(past=1, sliced=False)),
    (1, 50, 20, 32, 2, dict(past=1)),
    (1, 29, 12, 64, 1, {}),
    (1, 20, 9, 128, 1, dict(past=1)),
    (1, 17, 6, 100, 3, {})])
def test_dense(io, B, T, D, S, G, over):
    d = make((B, T), D, S, G, io, B + T + D + S, **over)
    compare(d, R.offsets_of(B, T))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D,S,G,state", [(48, 16, 2, True), (33, 16, 1, False),
                                         (10, 40, 1, True)])
def test_packed(io, D, S, G, state):
    lens = [0, 1, 8, 9, 0, 40, 7, 33, 0]
    offs = R.offsets_of(0, 0, lens)
    cu = torch.tensor(offs, dtype=torch.int32, device=DEV)
    d = make((1, offs[-1]), D, S, G, io, D + S, past=len(lens))
    if not state:
        d["past"] = None
    compare(d, offs, cu)


def test_without_softplus():
    d = make((1, 30), 24, 16, 1, "f32", 3, past=1)
    d["delta"] = d["delta"].abs() * 0.3
    d["delta_bias"] = d["delta_bias"].abs()
    compare(d, [0, 30], softplus=False)


def test_tiny_and_huge_steps():
    # softplus far below and above zero: steps of 1e-9 and of 60
    d = make((1, 24), 16, 16, 1, "f32", 8, past=1)
    d["delta"][:, ::3] = -20.0
    d["delta"][:, 1::3, ::2] = 60.0
    compare(d, [0, 24])


def test_empty_sequences_pass_their_states_through():
    d = make((1, 5), 16, 16, 1, "bf16", 2, past=3)
    cu = torch.tensor([0, 0, 5, 5], dtype=torch.int32, device=DEV)
    kw = dict(D=d["D"], z=d["z"], delta_bias=d["delta_bias"],
              initial_state=d["past"], cu_seqlens=cu)
    args = (d["u"], d["delta"], d["A"], d["Bm"], d["Cm"])
    _, fin = K.ssm_scan_fwd(*args, **kw)
    assert torch.equal(fin[0], d["past"][0]) and torch.equal(fin[2], d["past"][2])
    got = K.ssm_scan_bwd(*args, d_out=d["d_out"], d_final_state=d["d_final"], **kw)
    assert torch.equal(got[8][0], d["d_final"][0])
    assert torch.equal(got[8][2], d["d_final"][2])


def test_no_tokens():
    d = make((2, 0), 16, 16, 1, "bf16", 2, past=2)
    args = (d["u"], d["delta"], d["A"], d["Bm"], d["Cm"])
    kw = dict(D=d["D"], z=d["z"], delta_bias=d["delta_bias"],
              initial_state=d["past"])
    out, fin = K.ssm_scan_fwd(*args, **kw)
    assert out.shape == (2, 0, 16) and torch.equal(fin, d["past"])
    got = K.ssm_scan_bwd(*args, d_out=d["d_out"], d_final_state=d["d_final"], **kw)
    assert (got[2] == 0).all() and (got[5] == 0).all() and (got[7] == 0).all()
    assert torch.equal(got[8], d["d_final"])


def test_tokens_of_no_sequence_are_left_alone():
    offs = [3, 12, 12, 20]
    cu = torch.tensor(offs, dtype=torch.int32, device=DEV)
    cu0 = torch.tensor([0, 9, 9, 17], dtype=torch.int32, device=DEV)
    d = make((1, 32), 24, 16, 1, "bf16", 5, past=3, sliced=False)
    inner = {k: d[k][:, 3:20].contiguous() for k in
             ("u", "delta", "Bm", "Cm", "z", "d_out")}
    for k in inner:  # what belongs to no sequence is not read
        d[k][:, :3] = float("nan")
        d[k][:, 20:] = float("nan")
    kw = dict(D=d["D"], delta_bias=d["delta_bias"], initial_state=d["past"])

    def fwd(x, cu, **over):
        return K.ssm_scan_fwd(x["u"], x["delta"], d["A"], x["Bm"], x["Cm"],
                              z=x["z"], cu_seqlens=cu, **kw, **over)

    def bwd(x, cu):
        return K.ssm_scan_bwd(x["u"], x["delta"], d["A"], x["Bm"], x["Cm"],
                              z=x["z"], cu_seqlens=cu, d_out=x["d_out"],
                              d_final_state=d["d_final"], **kw)
    out = torch.full_like(d["u"], 7.0)
    _, fin = fwd(d, cu, out=out)
    out2, fin2 = fwd(inner, cu0)
    assert torch.equal(out[:, 3:20], out2) and torch.equal(fin, fin2)
    assert (out[:, :3] == 7).all() and (out[:, 20:] == 7).all()
    a, b = bwd(d, cu), bwd(inner, cu0)
    for i in (0, 1, 3, 4, 6):
        assert torch.equal(a[i][:, 3:20], b[i]), NAMES[i]
    for i in (2, 5, 7, 8):
        assert torch.equal(a[i], b[i]), NAMES[i]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N,T,D,S,G", [(1, 1, 4, 16, 1), (5, 1, 33, 16, 1),
                                       (3, 4, 30, 5, 3), (64, 1, 256, 16, 2),
                                       (2, 2, 20, 64, 1), (2, 1, 7, 128, 1)])
def test_step(io, N, T, D, S, G):
    d = make((N, T), D, S, G, io, N + T + D + S, past=N)
    state = d["past"].clone()
    kw = dict(D=d["D"], z=d["z"], delta_bias=d["delta_bias"])
    args = (d["u"], d["delta"], d["A"], d["Bm"], d["Cm"])
    out = K.ssm_step(*args, state=state, **kw)
    out_r, fin_r = R.ssm_scan(*flat64(d), R.offsets_of(N, T), True)
    R.check("out", out.reshape(-1, D), out_r, tol(T))
    R.check("state", state, fin_r, tol(T))


def test_prompt_then_tokens():
    # a prompt of 40 and 9 single tokens give what a prompt of 49 gives
    d = make((2, 49), 64, 16, 1, "f32", 11)
    kw = dict(D=d["D"], delta_bias=d["delta_bias"])

    def cut(a, b):
        return [d[k][:, a:b].contiguous() for k in
                ("u", "delta", "Bm", "Cm", "z")]
    u, dl, Bm, Cm, z = cut(0, 49)
    whole, fin = K.ssm_scan_fwd(u, dl, d["A"], Bm, Cm, z=z, **kw)
    u, dl, Bm, Cm, z = cut(0, 40)
    first, state = K.ssm_scan_fwd(u, dl, d["A"], Bm, Cm, z=z, **kw)
    outs = [first]
    for t in range(40, 49):
        u, dl, Bm, Cm, z = cut(t, t + 1)
        outs.append(K.ssm_step(u, dl, d["A"], Bm, Cm, state=state, z=z, **kw))
    got = torch.cat(outs, 1)
    R.check("out", got, whole.cpu().double(), 2 * tol(49))
    R.check("state", state, fin.cpu().double(), 2 * tol(49))


def test_final_state_in_place():
    d = make((2, 20), 32, 16, 1, "bf16", 12, past=2)
    kw = dict(D=d["D"], z=d["z"], delta_bias=d["delta_bias"])
    args = (d["u"], d["delta"], d["A"], d["Bm"], d["Cm"])
    out, fin = K.ssm_scan_fwd(*args, initial_state=d["past"], **kw)
    st = d["past"].clone()
    out2, fin2 = K.ssm_scan_fwd(*args, initial_state=st, final_state=st, **kw)
    assert fin2 is st and torch.equal(fin, st) and torch.equal(out, out2)


def test_misaligned_slices_match_aligned():
    d = make((2, 50), 64, 16, 1, "bf16", 3, sliced=False)

    def off(t, k):  # the same values at an odd element offset
        w = torch.zeros(*t.shape[:2], t[0, 0].numel() + 9, dtype=t.dtype,
                        device=DEV)
        w = w[..., k:k + t[0, 0].numel()]
        w.copy_(t.reshape(*t.shape[:2], -1))
        return w if t.dim() == 3 else w.unsqueeze(2)
    a = (d["u"], d["delta"], d["A"], d["Bm"], d["Cm"])
    b = (off(d["u"], 1), off(d["delta"], 3), d["A"], off(d["Bm"], 5),
         off(d["Cm"], 7))
    kw = dict(D=d["D"], delta_bias=d["delta_bias"])
    for x, y in zip(K.ssm_scan_fwd(*a, z=d["z"], **kw),
                    K.ssm_scan_fwd(*b, z=off(d["z"], 1), **kw)):
        assert torch.equal(x, y)
    for name, x, y in zip(
            NAMES, K.ssm_scan_bwd(*a, z=d["z"], d_out=d["d_out"], **kw),
            K.ssm_scan_bwd(*b, z=off(d["z"], 1), d_out=d["d_out"], **kw)):
        if name in ("D", "delta_bias"):
            # single loads give a thread other tokens of a channel, so these
            # sums over 100 tokens are added in another order: each of 100
            # partial sums rounds by 2^-24 of at most the sum of the terms
            R.check("d " + name, y, x.cpu().double(), 100 * 2.0 ** -24)
        else:
            assert torch.equal(x, y), name


def test_non_finite_inputs_stay_in_their_channel():
    d = make((2, 40), 32, 16, 1, "f32", 9)
    d["u"][1, 20, 5] = float("nan")
    args = (d["u"], d["delta"], d["A"], d["Bm"], d["Cm"])
    out, fin = K.ssm_scan_fwd(*args, D=d["D"], z=d["z"],
                              delta_bias=d["delta_bias"])
    want = torch.zeros(2, 40, 32, dtype=torch.bool, device=DEV)
    want[1, 20:, 5] = True
    assert torch.equal(torch.isnan(out), want)
    assert torch.isnan(fin[1, 5]).all() and torch.isfinite(fin[0]).all()


def test_long_memory():
    # decays near 1 over a long sequence: the rounding of the decay factors
    # adds up over their memory
    T, D, S = 3000, 8, 16
    d = make((1, T), D, S, 1, "f32", 21, past=1)
    d["delta"] = torch.full_like(d["delta"], -7.0) + d["delta"] * 0.1
    compare(d, [0, T])


def test_offsets_past_32_bits():
    stride, T, D = 1 << 17, 20000, 16
    wide = torch.empty(1, T, stride, dtype=torch.bfloat16, device=DEV)
    u = wide[..., 1000:1000 + D]
    u.copy_(torch.randn(1, T, D, device=DEV))
    d = make((1, T), D, 16, 1, "bf16", 6, z=False)
    kw = dict(D=d["D"], delta_bias=d["delta_bias"])
    args = (d["delta"], d["A"], d["Bm"], d["Cm"])
    a = K.ssm_scan_fwd(u, *args, **kw)
    b = K.ssm_scan_fwd(u.contiguous(), *args, **kw)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_many_sequences():
    # more sequences than a grid axis other than x holds
    n = 70000
    g = torch.Generator(device=DEV).manual_seed(3)
    u = torch.randn(1, n, 4, generator=g, device=DEV)
    B = torch.randn(1, n, 1, 2, generator=g, device=DEV)
    A = -torch.ones(4, 2, device=DEV)
    cu = torch.arange(n + 1, dtype=torch.int32, device=DEV)
    out, fin = K.ssm_scan_fwd(u, u, A, B, B, cu_seqlens=cu)
    dt = torch.nn.functional.softplus(u.double())
    h = (dt * u.double())[0, :, :, None] * B[0].double()
    R.check("state", fin, h.cpu(), tol(1))
    R.check("out", out[0], (h * B[0].double()).sum(-1).cpu(), tol(1))


def test_repeats_are_bit_identical():
    d = make((2, 200), 96, 16, 1, "bf16", 4, past=2)
    kw = dict(D=d["D"], z=d["z"], delta_bias=d["delta_bias"],
              initial_state=d["past"], d_out=d["d_out"],
              d_final_state=d["d_final"])
    args = (d["u"], d["delta"], d["A"], d["Bm"], d["Cm"])
    a = K.ssm_scan_bwd(*args, **kw)
    for _ in range(3):
        b = K.ssm_scan_bwd(*args, **kw)
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_refusals():
    d = make((2, 10), 16, 16, 2, "bf16", 1)
    args = [d["u"], d["delta"], d["A"], d["Bm"], d["Cm"]]

    def swapped(i, t):
        x = list(args)
        x[i] = t
        return x
    bad = [
        swapped(1, d["delta"].float()), swapped(1, d["delta"][:, :5]),
        swapped(2, d["A"][:8]), swapped(2, d["A"].bfloat16()),
        swapped(3, d["Bm"][..., :8]), swapped(4, d["Cm"].transpose(2, 3)),
        swapped(0, d["u"].cpu()), swapped(0, d["u"][:, :, :15]),
        swapped(4, d["Cm"].expand(2, 10, 2, 16)[:1].expand(2, 10, 2, 16)),
    ]
    for x in bad:
        with pytest.raises((ValueError, K.KdaError)):
            K.ssm_scan_fwd(*x)
    with pytest.raises(ValueError):
        K.ssm_scan_bwd(*args)  # no d_out
    with pytest.raises(ValueError):
        K.ssm_scan_fwd(*args, initial_state=torch.zeros(2, 16, 16, device=DEV,
                                                        dtype=torch.bfloat16))
    with pytest.raises(K.KdaError):  # three groups of 16 channels
        x = torch.zeros(2, 10, 3, 16, dtype=torch.bfloat16, device=DEV)
        K.ssm_scan_fwd(d["u"], d["delta"], d["A"], x, x)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lens,D,S,G", [
    ([700], 24, 16, 1),                   # one sequence in segments of 128
    ([385], 9, 5, 3),                     # a last segment of one token
    ([0, 1000, 3, 0, 128, 256, 1], 20, 16, 2),  # packed: ends on and off cuts
    ([640], 6, 64, 1)])
def test_split_into_segments(io, lens, D, S, G):
    # few channels: the scan runs in segments side by side
    offs = R.offsets_of(0, 0, lens)
    cu = torch.tensor(offs, dtype=torch.int32, device=DEV) \
        if len(lens) > 1 else None
    d = make((1, offs[-1]), D, S, G, io, sum(lens) + D, past=len(lens))
    compare(d, offs, cu)


def test_split_in_place_and_repeated():
    d = make((1, 2000), 64, 16, 1, "bf16", 31, past=1)
    args = (d["u"], d["delta"], d["A"], d["Bm"], d["Cm"])
    out, fin = K.ssm_scan_fwd(*args, initial_state=d["past"])
    for _ in range(3):
        st = d["past"].clone()
        out2, _ = K.ssm_scan_fwd(*args, initial_state=st, final_state=st)
        assert torch.equal(out, out2) and torch.equal(fin, st)


def test_split_backward_repeats_and_matches_one_segment():
    # a sequence in segments, and the same sequence in a batch wide enough
    # not to be split (its copies): other roundings at the joins only
    T, D, S = 1500, 64, 16
    d = make((1, T), D, S, 1, "f32", 33, past=1)
    kw = dict(D=d["D"], z=d["z"], delta_bias=d["delta_bias"],
              initial_state=d["past"], d_out=d["d_out"],
              d_final_state=d["d_final"])
    args = (d["u"], d["delta"], d["A"], d["Bm"], d["Cm"])
    a = K.ssm_scan_bwd(*args, **kw)
    for _ in range(2):
        b = K.ssm_scan_bwd(*args, **kw)
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    n = 200

    def many(t):
        return t.expand(n, *t.shape[1:]).contiguous()
    kw.update(z=many(d["z"]), initial_state=many(d["past"]),
              d_out=many(d["d_out"]), d_final_state=many(d["d_final"]))
    c = K.ssm_scan_bwd(many(d["u"]), many(d["delta"]), d["A"], many(d["Bm"]),
                       many(d["Cm"]), **kw)
    for name, x, y in zip(NAMES, a, c):
        if name in ("A", "D", "delta_bias"):
            y = y / n  # a sum of n equal terms, rounded n times at most
            R.check("d " + name, x, y.cpu().double(), 4 * tol(T) + n * 2.0 ** -24)
        else:
            R.check("d " + name, x, y[:1].cpu().double(), 4 * tol(T))


@pytest.mark.parametrize("copies", [1, 200])
def test_infinite_states_stay_infinite(copies):
    # one sequence in segments, and enough copies of it not to be split: a
    # decay greater than 0 leaves an infinite state infinite, also where the
    # decay of a whole segment is too small for fp32
    T, D, S = 1500, 64, 16
    d = make((1, T), D, S, 1, "f32", 41, past=1)
    d["past"][0, 7, 3] = float("inf")
    d["past"][0, 9, 0] = float("-inf")
    d["past"][0, 9, 1] = float("nan")
    d["A"][7, 3] = -3.0  # a segment's decay is around exp(-140)

    def many(t):
        return t.expand(copies, *t.shape[1:]).contiguous()
    kw = dict(D=d["D"], delta_bias=d["delta_bias"],
              initial_state=many(d["past"]))
    args = (many(d["u"]), many(d["delta"]), d["A"], many(d["Bm"]),
            many(d["Cm"]))
    out, fin = K.ssm_scan_fwd(*args, **kw)
    want = many(d["past"])
    bad = ~torch.isfinite(want)
    assert torch.equal(torch.isfinite(fin), ~bad)
    assert torch.equal(fin[bad].nan_to_num(7.0), want[bad].nan_to_num(7.0))
    assert torch.isinf(out[:, :, 7]).all() and torch.isnan(out[:, :, 9]).all()
    ok = [c for c in range(D) if c not in (7, 9)]
    assert torch.isfinite(out[:, :, ok]).all()
    # backward: dC = dy h sees the infinite state (and, with it, NaN), the
    # gradients that no state enters do not
    got = K.ssm_scan_bwd(*args, d_out=many(d["d_out"]), **kw)
    assert torch.isinf(got[4][..., 3]).all()
    for i in (0, 3, 8):
        assert torch.isfinite(got[i]).all(), NAMES[i]
    assert torch.isfinite(got[4][..., 4:]).all()


@pytest.mark.parametrize("copies", [1, 200])
def test_growth_of_nothing_is_nothing(copies):
    # a positive A: eight tokens' growth is beyond fp32, but a state of 0
    # stays 0 until an input comes
    T, D = 1000, 64
    u = torch.zeros(copies, T, D, device=DEV)
    delta = torch.zeros_like(u)
    A = torch.full((D, 16), 50.0, device=DEV)
    bc = torch.ones(copies, T, 1, 16, device=DEV)
    out, fin = K.ssm_scan_fwd(u, delta, A, bc, bc)
    assert (out == 0).all() and (fin == 0).all()
    got = K.ssm_scan_bwd(u, delta, A, bc, bc, d_out=torch.zeros_like(u))
    for x in got:
        assert x is None or (x == 0).all()


def test_steps_keep_their_relative_accuracy():
    # with u = B = 1 and no past a single token's state is its step, and with
    # one channel d_B is the step as well.  Units of 2^-24: the exponential 4,
    # its argument's remainder 1, 2 + e 1, the reciprocal 2, their product 1,
    # the series 1, the last product 1
    bound = 11 * 2.0 ** -24
    delta = torch.linspace(-80, 20, 4001, device=DEV).reshape(-1, 1, 1)
    want = torch.nn.functional.softplus(delta.double(), threshold=60)
    one = torch.ones_like(delta)
    A, bc = -torch.ones(1, 1, device=DEV), one.unsqueeze(-1)
    _, fin = K.ssm_scan_fwd(one, delta, A, bc, bc)
    state = torch.zeros_like(fin)
    K.ssm_step(one, delta, A, bc, bc, state)
    got = K.ssm_scan_bwd(one, delta, A, bc, bc, d_out=one)
    for name, x in (("prompt", fin), ("token", state), ("backward", got[3])):
        worst = (x.reshape(want.shape).double() / want - 1).abs().max()
        assert worst <= bound, f"{name}: {float(worst):.3e} > {bound:.3e}"



@pytest.mark.parametrize("copies", [1, 200])
def test_a_decay_is_as_good_as_its_chunks(copies):
    # States of 1 that only decay, over T equal steps: a factor's error comes
    # T times, so what counts is how many factors there are.  The error of one
    # exponential is read off a single token: of one step (the factor of a
    # token) and of eight (that of a chunk, the steps' sum being exact here).
    # A scan that multiplies tokens' factors misses by T times the first; held
    # to chunks it may miss by T / 8 times the second, plus the rounding of
    # the running products (2 a token, independent, 4 standard deviations of
    # 2^-24 at most) and of 16 segments' exponentials (2^-21 each).  The
    # chunk's own product, which its exponential replaces, is 8 equal factors
    # multiplied up from 1: 7 products, each off by up to 2^-25, and by the
    # same in every chunk, so T / 8 times 7 2^-25 more.
    T, D, S, dt = 2048, 64, 16, 2.0 ** -10
    g = torch.Generator(device=DEV).manual_seed(17)
    A = -(0.1 + 0.9 * torch.rand(D, S, generator=g, device=DEV))

    def inputs(n, t, step):
        u = torch.zeros(n, t, D, device=DEV)
        bc = torch.ones(n, t, 1, S, device=DEV)
        return u, torch.full_like(u, step), A, bc, bc

    def one_factor(step):  # its relative error
        state = torch.ones(1, D, S, device=DEV)
        K.ssm_step(*inputs(1, 1, step), state, softplus=False)
        return state.double() / torch.exp(step * A.double()) - 1

    start = torch.ones(copies, D, S, device=DEV)
    args = inputs(copies, T, dt)
    _, fin = K.ssm_scan_fwd(*args, initial_state=start, softplus=False)
    got = K.ssm_scan_bwd(*args, initial_state=start, softplus=False,
                         d_out=torch.zeros_like(args[0]), d_final_state=start)
    want = torch.exp(T * dt * A.double())
    own = T / 8 * one_factor(8 * dt).abs()
    bound = own + T / 8 * 7 * 2.0 ** -25 + \
        4 * (2 * T) ** 0.5 * 2.0 ** -24 + 16 * 2.0 ** -21
    # the bound means something: many a state's factors would break it
    assert (T * one_factor(dt).abs() > bound).float().mean() > 0.05
    for name, x in (("final state", fin), ("d_initial_state", got[8]),
                    # T dt h dh, one term a token and copy, of two decays
                    ("dA", got[2][None] / (copies * T * dt))):
        err = (x.double() / want - 1).abs()
        over = (err / (2 * bound if name == "dA" else bound)).max()
        assert over <= 1, f"{name}: {float(over):.2f} of the bound"
