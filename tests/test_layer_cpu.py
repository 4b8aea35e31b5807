"""The layer operators on the host: the 64-bit reference against hand-made
values and differences, the refusals of the binding, the backward's plan, and
(in a child process that sees no GPU) the C ABI's refusals."""
import os
import subprocess
import sys

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import layer_ref as R
from gated_delta_rule_156_b200 import build as kbuild
from gated_delta_rule_156_b200 import kda as K

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return K.library()


def randn(*shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g, dtype=torch.float64)


def test_conv_reference_by_hand():
    x = torch.tensor([[1.0], [2.0], [5.0]], dtype=torch.float64)
    w = torch.tensor([[10.0, 1.0]], dtype=torch.float64)
    past = torch.tensor([[[3.0]], [[7.0]]], dtype=torch.float64)
    out, fin = R.short_conv(x, w, None, past, [0, 2, 3], "none")
    assert out[:, 0].tolist() == [31.0, 12.0, 75.0]
    assert fin[:, 0, 0].tolist() == [2.0, 5.0]
    # an empty sequence keeps its past; a short one the end of it
    w3 = torch.tensor([[1.0, 1.0, 1.0]], dtype=torch.float64)
    past = torch.tensor([[[3.0], [4.0]], [[7.0], [8.0]]], dtype=torch.float64)
    _, fin = R.short_conv(x[:1], w3, None, past, [0, 0, 1], "none")
    assert fin[..., 0].tolist() == [[3.0, 4.0], [8.0, 1.0]]


def test_scan_reference_by_hand():
    one = torch.ones(2, 1, dtype=torch.float64)
    A = torch.full((1, 1), -0.5, dtype=torch.float64)
    B = C = torch.ones(2, 1, 1, dtype=torch.float64)
    past = torch.full((1, 1, 1), 4.0, dtype=torch.float64)
    out, fin = R.ssm_scan(one, 2 * one, A, B, C, None, None, None, past,
                          [0, 2], False)
    e = torch.exp(torch.tensor(-1.0, dtype=torch.float64))
    h1 = 4 * e + 2
    h2 = h1 * e + 2
    assert torch.allclose(out[:, 0], torch.stack([h1, h2]))
    assert torch.allclose(fin[0, 0, 0], h2)


def test_norm_reference_by_hand():
    x = torch.tensor([[3.0, 4.0]], dtype=torch.float64)
    r = torch.tensor([[1.0, 1.0]], dtype=torch.float64)
    one = torch.ones(2, dtype=torch.float64)
    out, normed = R.block_norm(x, one, None, r, 2 * one, one, "none", False, 0)
    s = 12.5 ** 0.5
    want = torch.tensor([[1 + 6 / s, 1 + 8 / s]], dtype=torch.float64)
    assert torch.allclose(out, want)
    assert torch.allclose((normed ** 2).mean(), torch.ones((), dtype=torch.float64))


@pytest.mark.parametrize("which", ["conv", "scan", "norm"])
def test_reference_gradients_by_differences(which):
    if which == "conv":
        ins = [randn(5, 3, seed=1), randn(3, 4, seed=2), randn(3, seed=3),
               randn(3, 3, 3, seed=4)]

        def fn(x, w, b, p):
            return R.short_conv(x, w, b, p, [0, 4, 4, 5], "silu")
    elif which == "scan":
        ins = [randn(4, 2, seed=1), randn(4, 2, seed=2), -randn(2, 3, seed=3).exp(),
               randn(4, 1, 3, seed=4), randn(4, 1, 3, seed=5), randn(2, seed=6),
               randn(4, 2, seed=7), randn(2, seed=8), randn(2, 2, 3, seed=9)]

        def fn(u, d, A, B, C, D, z, b, p):
            return R.ssm_scan(u, d, A, B, C, D, z, b, p, [0, 3, 4], True)
    else:
        ins = [randn(3, 4, seed=1), randn(4, seed=2), randn(3, 4, seed=3),
               randn(3, 4, seed=4), randn(4, seed=5), randn(4, seed=6)]

        def fn(x, w, g, r, s, p):
            return R.block_norm(x, w, g, r, s, p, "silu", False, 1e-6)
    assert torch.autograd.gradcheck(fn, [t.requires_grad_() for t in ins])


def test_c_abi_refusals_in_a_process_without_gpus(lib):
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run(
        [sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
         os.path.join(ROOT, "tests", "fake_address_layer.py")],
        cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and "skipped" not in r.stdout, r.stdout[-2000:]


def test_host_tensors_are_refused(lib):
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError, match="CUDA"):
        K.short_conv_fwd(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        K.ssm_scan_fwd(x, x, torch.zeros(8, 16), torch.zeros(1, 4, 1, 16),
                       torch.zeros(1, 4, 1, 16))
    with pytest.raises(ValueError, match="CUDA"):
        K.block_norm_fwd(x, torch.zeros(8))


def test_token_strides():
    # token strides follow from shape and stride alone
    for x, inner, want in ((torch.zeros(2, 5, 24)[..., 8:16], 1, 24),
                           (torch.zeros(2, 5, 24)[:, 1:3, :8], 1, None),
                           (torch.zeros(2, 5, 24)[:, :1, :8], 1, 120),
                           (torch.zeros(1, 5, 24)[:, 1:3, :8], 1, 24),
                           (torch.zeros(10, 3, 4, 8)[:, 1], 2, 96),
                           (torch.zeros(10, 4, 16)[..., :8], 2, None),
                           (torch.zeros(10, 1, 16)[..., :8], 2, 16),
                           (torch.zeros(4, 8).t(), 1, None),
                           (torch.zeros(1, 8).expand(4, 8), 1, None)):
        assert K._token_stride(x, inner) == want, (x.shape, x.stride())


def test_scan_bwd_plan(lib):
    # the saving pass, the backward pass, the sums of dB and dC and of the rest
    kern, ws = K.ssm_scan_bwd_plan(2, 4096, 4096, 16, 1, torch.bfloat16)
    assert kern == 4
    # few channels: both passes over the recurrence in segments
    assert K.ssm_scan_bwd_plan(1, 4096, 64, 16, 1, torch.bfloat16)[0] == 6
    # at least the states at every 8th token
    assert ws >= 2 * 4096 // 8 * 4096 * 16 * 4
    _, wsp = K.ssm_scan_bwd_plan(1, 1000, 64, 16, 2, torch.float32, True, 7)
    assert wsp > 0
    with pytest.raises(K.KdaError):
        K.ssm_scan_bwd_plan(1, 10, 64, 129, 1, torch.float32)
    with pytest.raises(K.KdaError):
        K.ssm_scan_bwd_plan(1, 10, 64, 16, 3, torch.float32)


def test_saved_state_ids_never_meet():
    # piece c of 8 tokens of a sequence at `start` has id start // 8 + s + c
    g = torch.Generator().manual_seed(0)
    for _ in range(200):
        n = int(torch.randint(1, 9, (1,), generator=g))
        lens = torch.randint(0, 40, (n,), generator=g).tolist()
        seen, start = set(), int(torch.randint(0, 9, (1,), generator=g))
        for s, length in enumerate(lens):
            for c in range((length + 7) // 8):
                i = start // 8 + s + c
                assert i not in seen
                seen.add(i)
            start += length
        assert not seen or max(seen) < start // 8 + n + 1


def test_sizes_beyond_the_abi_fields_are_refused():
    # 2^32 + 5 tokens must not reach the 32-bit field as 5; the tensors are
    # fakes without memory
    big, bf = 2 ** 32 + 5, torch.bfloat16
    with FakeTensorMode():
        def fake(*shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device="cuda")
        x, w = fake(1, big, 1, dtype=bf), fake(1, 4)
        bc = fake(1, big, 1, 1, dtype=bf)
        calls = [
            lambda: K._conv_shape(x, w, None, None, "silu"),
            lambda: K._conv_shape(fake(1, 5, 1), w, None,
                                  fake(big, dtype=torch.int32), "silu"),
            lambda: K._ssm_shape(x, x, fake(1, 1), bc, bc, None, None, None,
                                 None, True),
            lambda: K._norm_shape(fake(3, big, dtype=bf), None, None, None,
                                  None, None, bf, "none", False, 1e-6),
            lambda: K.ssm_scan_bwd_plan(1, big, 64, 16, 1, bf),
        ]
        for call in calls:
            with pytest.raises(ValueError, match="2\\^31"):
                call()
        # the number of the norm's rows has 64 bits
        shape, _ = K._norm_shape(fake(big, 3, dtype=bf), None, None, None,
                                 None, None, bf, "none", False, 1e-6)
        assert shape.tokens == big and shape.width == 3


def test_norm_strides():
    # rows at one stride, or tokens at one stride with dense heads; a
    # contiguous tensor goes with either, the two forms not with each other
    with FakeTensorMode():
        def fake(*shape):
            return torch.empty(shape, device="cuda")

        def strides(x, gate):
            s, _ = K._norm_shape(x, None, gate, None, None, None,
                                 torch.float32, "silu", False, 1e-6)
            return s.tokens, s.heads, s.x_stride, s.gate_stride
        dense, rows = fake(5, 4, 32), fake(5, 4, 48)[..., :32]
        heads = fake(5, 3, 4, 32)[:, 1]
        assert strides(dense, rows) == (20, 1, 0, 48)
        assert strides(rows, rows) == (20, 1, 48, 48)
        assert strides(dense, heads) == (5, 4, 0, 384)
        assert strides(heads, dense) == (5, 4, 384, 0)
        for x, gate in ((rows, heads), (heads, rows)):
            with pytest.raises(ValueError, match="dense"):
                strides(x, gate)
