"""The layer operators together, as a layer runs them: convolution, recurrence
(the delta rule of kda.h or the selective scan), gated norm, block boundary;
in prompts, in training, token by token, inside CUDA graphs, on other streams,
and without reading their workspace before writing it."""
import numpy as np
import pytest
import torch

import layer_ref as R
import parity as PY
from gated_delta_rule_156_b200 import kda as K
from oracle import kda_oracle

pytestmark = pytest.mark.gpu
DEV = "cuda"


def randn(*shape, seed, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


class DeltaLayer:
    """conv + SiLU over a fused q/k/v projection, the delta rule with its
    prologue, the gated norm per head, the block boundary."""

    def __init__(self, H=2, d=64, W=4):
        self.H, self.d, self.n = H, d, H * d
        self.w = randn(3 * self.n, W, seed=1) * 0.5
        self.o_norm = 1 + 0.1 * randn(d, seed=2)
        self.post = 1 + 0.1 * randn(self.n, seed=3)
        self.pre = 1 + 0.1 * randn(self.n, seed=4)
        self.scale = 0.5 + 0.1 * randn(self.n, seed=5)
        self.pro = dict(normalize_qk=True, q_scale=d ** -0.5)

    def heads(self, y):
        B, T, _ = y.shape
        return [t.contiguous().view(B, T, self.H, self.d)
                for t in y.split(self.n, dim=-1)]

    def rest(self, o, gate, res):
        B, T = o.shape[:2]
        o, _ = K.block_norm_fwd(o, self.o_norm, gate.view(o.shape))
        return K.block_norm_fwd(o.view(B, T, self.n), self.post, residual=res,
                                scale=self.scale, pre_weight=self.pre)

    def prompt(self, x, gate, la, beta, res):
        y, conv = K.short_conv_fwd(x, self.w)
        q, k, v = self.heads(y)
        o, s = K.chunk_fwd(q, k, v, la, beta, prologue=self.pro)
        return (*self.rest(o, gate, res), conv, s)

    def token(self, x, gate, la, beta, res, conv, s):
        y = K.short_conv_step(x, self.w, None, conv)
        q, k, v = self.heads(y)
        o = K.recurrent_step(q, k, v, la, beta, s, prologue=self.pro)
        return self.rest(o, gate, res)


def delta_inputs(B, T, H=2, d=64):
    n = H * d
    bf = torch.bfloat16
    return (randn(B, T, 3 * n, seed=11, dtype=bf),
            randn(B, T, n, seed=12, dtype=bf),
            -torch.nn.functional.softplus(randn(B, T, H, d, seed=13)) / 16,
            torch.sigmoid(randn(B, T, H, seed=14)),
            randn(B, T, n, seed=15))


def test_delta_layer_prompt_against_the_oracle():
    L, B, T = DeltaLayer(), 2, 130
    x, gate, la, beta, res = delta_inputs(B, T)
    out, normed, _, s = L.prompt(x, gate, la, beta, res)
    torch.cuda.synchronize()
    y, _ = R.short_conv(R.h64(x).reshape(B * T, -1), R.h64(L.w), None, None,
                        [0, T, 2 * T], "silu")
    q, k, v = [t.reshape(B, T, L.H, L.d) for t in y.split(L.n, dim=-1)]
    q = q / q.norm(dim=-1, keepdim=True) * L.d ** -0.5
    k = k / k.norm(dim=-1, keepdim=True)
    o, sr = kda_oracle.recurrent(q.numpy(), k.numpy(), v.numpy(),
                                 R.h64(la).numpy(), R.h64(beta).numpy(), None)
    o, _ = R.block_norm(torch.from_numpy(np.asarray(o)), R.h64(L.o_norm),
                        R.h64(gate).view(B, T, L.H, L.d), None, None, None,
                        "sigmoid", False, 1e-6)
    ref, ref_n = R.block_norm(o.reshape(B, T, L.n), R.h64(L.post), None,
                              R.h64(res), R.h64(L.scale), R.h64(L.pre), "none",
                              False, 1e-6)
    # the delta rule's own bf16 tolerance carries through the norms
    PY.check("out", out.cpu(), ref, PY.TOL_BF16)
    PY.check("normed", normed.float().cpu(), ref_n, PY.TOL_BF16)
    PY.check("state", s.cpu(), sr, PY.TOL_BF16)


def test_delta_layer_tokens_follow_the_prompt():
    L, B, T, P = DeltaLayer(), 2, 40, 33
    ins = delta_inputs(B, T)
    out, normed, _, s = L.prompt(*ins)
    o1, n1, conv, st = L.prompt(*[t[:, :P].contiguous() for t in ins])
    for t in range(P, T):
        o, n = L.token(*[a[:, t:t + 1].contiguous() for a in ins], conv, st)
        PY.check("out", o.cpu(), out[:, t:t + 1].cpu(), 2 * PY.TOL_BF16)
        PY.check("normed", n.float().cpu(), normed[:, t:t + 1].float().cpu(),
                 2 * PY.TOL_BF16)
    PY.check("state", st.cpu(), s.cpu(), 2 * PY.TOL_BF16)


def scan_layer(B, T, D=64, S=16, dtype=torch.float32):
    """A scan layer's tensors: x beside z in one projection, B beside C."""
    xz = randn(B, T, 2 * D, seed=21, dtype=dtype)
    bc = randn(B, T, 1, 2 * S, seed=22, dtype=dtype)
    return dict(x=xz[..., :D], z=xz[..., D:], Bm=bc[..., :S], Cm=bc[..., S:],
                delta=randn(B, T, D, seed=23, dtype=dtype) - 1,
                w=randn(D, 4, seed=24) * 0.5, bias=randn(D, seed=25) * 0.1,
                A=-torch.exp(randn(D, S, seed=26) * 0.5), D=randn(D, seed=27),
                res=randn(B, T, D, seed=28, dtype=dtype),
                post=1 + 0.1 * randn(D, seed=29), pre=1 + 0.1 * randn(D, seed=30),
                d_out=randn(B, T, D, seed=31, dtype=dtype),
                d_normed=randn(B, T, D, seed=32, dtype=dtype))


def scan_forward(p):
    u, _ = K.short_conv_fwd(p["x"], p["w"], p["bias"])
    o, _ = K.ssm_scan_fwd(u, p["delta"], p["A"], p["Bm"], p["Cm"], D=p["D"],
                          z=p["z"])
    out, normed = K.block_norm_fwd(o, p["post"], residual=p["res"],
                                   pre_weight=p["pre"])
    return u, o, out, normed


def scan_backward(p, u, o):
    do, _, dres, dpost, _, dpre = K.block_norm_bwd(
        o, p["post"], residual=p["res"], pre_weight=p["pre"],
        d_out=p["d_out"], d_normed=p["d_normed"])
    du, dd, dA, dB, dC, dD, dz, _, _ = K.ssm_scan_bwd(
        u, p["delta"], p["A"], p["Bm"], p["Cm"], D=p["D"], z=p["z"], d_out=do)
    dx, dw, db, _ = K.short_conv_bwd(p["x"], p["w"], p["bias"], None, None, du)
    return dict(x=dx, z=dz, Bm=dB, Cm=dC, delta=dd, w=dw, bias=db, A=dA, D=dD,
                res=dres, post=dpost, pre=dpre)


def test_scan_layer_gradients():
    B, T, D = 2, 50, 64
    p = scan_layer(B, T)
    u, o, out, normed = scan_forward(p)
    got = scan_backward(p, u, o)
    names = list(got)
    flat = {"x", "z", "Bm", "Cm", "delta", "res"}

    def fn(*ins):
        q = dict(zip(names, ins))
        offs = R.offsets_of(B, T)
        u, _ = R.short_conv(q["x"], q["w"], q["bias"], None, offs, "silu")
        o, _ = R.ssm_scan(u, q["delta"], q["A"], q["Bm"], q["Cm"], q["D"],
                          q["z"], None, None, offs, True)
        return R.block_norm(o, q["post"], None, q["res"], None, q["pre"],
                            "none", False, 1e-6)
    ins = [R.h64(p[n]).reshape(B * T, *p[n].shape[2:]) if n in flat
           else R.h64(p[n]) for n in names]
    ref_out, ref_normed = fn(*ins)
    # three fp32 stages, the scan's the widest: 0.5 T + 32 roundings of 2^-20,
    # and as much again for each of the two stages behind it
    tol = 4 * (0.5 * T + 32) * 2.0 ** -20
    R.check("out", out.reshape(B * T, D), ref_out, tol)
    R.check("normed", normed.reshape(B * T, D), ref_normed, tol)
    ref = R.grads(fn, ins, (R.h64(p["d_out"]).reshape(B * T, D),
                            R.h64(p["d_normed"]).reshape(B * T, D)))
    for n, r in zip(names, ref):
        R.check("d " + n, got[n].reshape(r.shape), r, 2 * tol)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layer_in_a_graph_with_new_inputs(dtype):
    p = scan_layer(2, 70, dtype=dtype)

    def step():
        u, o, out, normed = scan_forward(p)
        return [out, normed, *scan_backward(p, u, o).values()]
    step()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    # two graphs: each holds its own workspace
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step()
        graphs.append((g, outs))
    for seed in (100, 200):
        for n in ("res", "delta", "d_out", "d_normed"):
            p[n].copy_(randn(*p[n].shape, seed=seed))
        want = step()
        for g, outs in graphs:
            g.replay()
        torch.cuda.synchronize()
        for g, outs in graphs:
            assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_steps_in_a_graph():
    B, D, S = 8, 96, 16
    p = scan_layer(B, 1, D, S, torch.bfloat16)
    conv0 = randn(B, 3, D, seed=50, dtype=torch.bfloat16)
    h0 = randn(B, D, S, seed=51)

    def token(conv, h):
        u = K.short_conv_step(p["x"], p["w"], p["bias"], conv)
        o = K.ssm_step(u, p["delta"], p["A"], p["Bm"], p["Cm"], state=h,
                       D=p["D"], z=p["z"])
        return K.block_norm_fwd(o, p["post"], residual=p["res"],
                                pre_weight=p["pre"])
    conv, h = conv0.clone(), h0.clone()
    want = [token(conv, h) for _ in range(3)]
    c2, h2 = conv0.clone(), h0.clone()
    token(c2.clone(), h2.clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = token(c2, h2)
    c2.copy_(conv0)
    h2.copy_(h0)
    for i in range(3):
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(want[i], outs))
    assert torch.equal(conv, c2) and torch.equal(h, h2)


def test_two_streams_at_once():
    # the calls of two streams overlap; each has its own workspace and result
    ps = [scan_layer(1, 300, D=256, dtype=torch.bfloat16) for _ in range(2)]
    ps[1]["delta"] = ps[1]["delta"] * 0.5
    want = []
    for p in ps:
        u, o, *_ = scan_forward(p)
        want.append(scan_backward(p, u, o))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    for _ in range(3):
        got = []
        for s, p in zip(streams, ps):
            with torch.cuda.stream(s):
                u, o, *_ = scan_forward(p)
                got.append(scan_backward(p, u, o))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(a[n], b[n]) for n in a)


def test_stream_argument():
    p = scan_layer(2, 90, dtype=torch.bfloat16)
    want = K.ssm_scan_fwd(p["x"], p["delta"], p["A"], p["Bm"], p["Cm"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = K.ssm_scan_fwd(p["x"], p["delta"], p["A"], p["Bm"], p["Cm"],
                         stream=s)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_workspace_is_written_before_it_is_read(monkeypatch):
    lens = [0, 9, 64, 1, 130, 0]
    offs = R.offsets_of(0, 0, lens)
    cu = torch.tensor(offs, dtype=torch.int32, device=DEV)
    p = scan_layer(1, offs[-1], dtype=torch.bfloat16)

    def calls():
        a = K.ssm_scan_bwd(p["x"], p["delta"], p["A"], p["Bm"], p["Cm"],
                           D=p["D"], z=p["z"], d_out=p["d_out"], cu_seqlens=cu)
        b = K.short_conv_bwd(p["x"], p["w"], p["bias"], None, cu, p["d_out"])
        c = K.block_norm_bwd(p["x"], p["post"], residual=p["res"],
                             pre_weight=p["pre"], d_out=p["d_out"],
                             d_normed=p["d_normed"])
        torch.cuda.synchronize()
        return [t.clone() for t in (*a, *b, *c) if t is not None]
    monkeypatch.delenv("KDA_WORKSPACE_FILL", raising=False)
    want = calls()
    monkeypatch.setenv("KDA_WORKSPACE_FILL", "127")
    got = calls()
    for i, (a, b) in enumerate(zip(want, got)):
        assert torch.equal(a, b), i


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_tensors_of_another_device():
    p = {k: v.to("cuda:1") for k, v in scan_layer(1, 20).items()}
    q = scan_layer(1, 20)
    assert torch.cuda.current_device() == 0
    a = K.short_conv_fwd(p["x"], p["w"])
    b = K.short_conv_fwd(q["x"], q["w"])
    assert torch.equal(a[0].cpu(), b[0].cpu())
    with pytest.raises(ValueError):
        K.short_conv_fwd(p["x"], q["w"])


@pytest.mark.parametrize("packed", [False, True])
def test_split_workspace_is_written_before_it_is_read(packed, monkeypatch):
    # few channels: the scan and its backward run in segments
    lens = [1500, 0, 3, 1200, 257]
    T = sum(lens)
    cu = torch.tensor(R.offsets_of(0, 0, lens), dtype=torch.int32,
                      device=DEV) if packed else None
    p = scan_layer(1, T, dtype=torch.bfloat16)

    def calls():
        kw = dict(D=p["D"], z=p["z"], cu_seqlens=cu)
        args = (p["x"], p["delta"], p["A"], p["Bm"], p["Cm"])
        a = K.ssm_scan_fwd(*args, **kw)
        b = K.ssm_scan_bwd(*args, d_out=p["d_out"], **kw)
        torch.cuda.synchronize()
        return [t.clone() for t in (*a, *b) if t is not None]
    kern, _ = K.ssm_scan_bwd_plan(1, T, 64, 16, 1, torch.bfloat16, packed,
                                  len(lens))
    assert kern == 6  # split
    monkeypatch.delenv("KDA_WORKSPACE_FILL", raising=False)
    want = calls()
    monkeypatch.setenv("KDA_WORKSPACE_FILL", "127")
    got = calls()
    for i, (a, b) in enumerate(zip(want, got)):
        assert torch.isfinite(b.float()).all(), i
        assert torch.equal(a, b), i


def test_graphs_replayed_on_two_streams():
    # two captured backward passes replayed at once: each has its workspace
    ps = [scan_layer(1, 1000, D=96, dtype=torch.bfloat16) for _ in range(2)]
    ps[1]["delta"] = ps[1]["delta"] * 0.5

    def run(p):
        u, o, *_ = scan_forward(p)
        return list(scan_backward(p, u, o).values())
    want = [[t.clone() for t in run(p)] for p in ps]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for p in ps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(p))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in ps]
    for _ in range(5):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(a, b) for a, b in zip(w, o))
