"""Host-side refusals of the layer operators' C ABI, exercised with fake
device addresses that are never dereferenced.  Like fake_address_abi.py, this
file only runs in a process that sees no GPU (test_layer_cpu.py starts it that
way); anywhere else it skips itself."""
import ctypes
import os

import pytest

if os.environ.get("CUDA_VISIBLE_DEVICES", None) != "":
    pytest.skip("runs only in a process with no visible GPU",
                allow_module_level=True)

from gated_delta_rule_156_b200 import build as kbuild  # noqa: E402
from gated_delta_rule_156_b200 import kda as K  # noqa: E402

OK, INV, UNS, MIS, CUDA = 0, 1, 2, 3, 4
BASE, GAP = 0x7000_0000_0000, 0x1000_0000


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return K.library()


def addr(i):
    return None if i is None else i if i > 1000 else BASE + i * GAP


def call(lib, name, shape, names, over):
    """name(shape, tensors..., stream 0) with the tensors at fake addresses
    1, 2, ...; `over` replaces some (None: a null pointer)."""
    assert set(over) <= set(names)
    ptrs = [addr(over.get(n, i + 1)) for i, n in enumerate(names)]
    return getattr(lib, name)(None if shape is None else ctypes.byref(shape),
                              *ptrs, None)


CONV_FWD = "x weight bias past cu out final".split()
CONV_BWD = "x weight bias past cu d_out d_final dx dw db dpast".split()
CONV_STEP = "x weight bias state out".split()
SSM_FWD = "u delta A B C skip z bias h0 cu out final".split()
SSM_BWD = ("u delta A B C skip z bias h0 cu d_out d_final du ddelta dA dB dC "
           "dskip dz dbias dh0").split()
SSM_STEP = "u delta A B C skip z bias state out".split()
NORM_FWD = "x post gate residual scale pre out normed".split()
NORM_BWD = ("x post gate residual scale pre d_out d_normed dx dgate dres dpost "
            "dscale dpre").split()


def conv(**kw):
    d = dict(B=1, T=64, D=64, W=4, n_seqs=2, io_dtype=0, activation=1,
             x_stride=0)
    d.update(kw)
    return K.KdaConvShape(**d)


def ssm(**kw):
    d = dict(B=1, T=64, D=64, S=16, G=2, n_seqs=2, io_dtype=0, softplus=1)
    d.update(kw)
    return K.KdaSsmShape(**d)


def norm(**kw):
    d = dict(tokens=8, heads=2, width=64, io_dtype=0, residual_dtype=1,
             gate_act=1, gate_first=0, eps=1e-6)
    d.update(kw)
    return K.KdaNormShape(**d)


@pytest.mark.parametrize("name,names,step", [
    ("kda_short_conv_fwd", CONV_FWD, False),
    ("kda_short_conv_bwd", CONV_BWD, False),
    ("kda_short_conv_step", CONV_STEP, True)])
def test_conv(lib, name, names, step):
    def c(shape, **over):
        return call(lib, name, shape, names, over)
    assert c(None) == INV
    for bad in (dict(T=-1), dict(B=-1), dict(D=0), dict(io_dtype=5),
                dict(activation=2), dict(activation=-1), dict(x_stride=63),
                dict(x_stride=-64), dict(x_stride=1 << 40),
                dict(x_stride=2 ** 62)):
        assert c(conv(**bad)) == INV, bad
    for bad in (dict(W=1), dict(W=5), dict(D=(1 << 20) + 1),
                dict(T=2 ** 31 - 1)):
        assert c(conv(**bad)) == UNS, bad
    assert c(conv(), x=None) == INV
    assert c(conv(), weight=None) == INV
    assert c(conv(), x=BASE + GAP + 1) == MIS
    assert c(conv(), weight=BASE + 2 * GAP + 2) == MIS
    out = "dx" if "dx" in names else "out"
    assert c(conv(), **{out: None}) == INV
    assert c(conv(), **{out: 1}) == INV        # over x
    assert c(conv(), **{out: BASE + GAP + 64 * 64 * 2 - 2}) == INV
    if step:
        assert c(conv(), state=None) == INV
        assert c(conv(), state=BASE + GAP) == INV
    else:
        assert c(conv(B=2)) == INV             # packed with B != 1
        assert c(conv(n_seqs=0)) == INV
        last = "final" if "final" in names else "dpast"
        assert c(conv(), **{last: names.index("past") + 1}) == INV
    if "dw" in names:
        assert c(conv(), dw=None) == INV
        assert c(conv(), d_out=None) == INV
        assert c(conv(), dw=names.index("dx") + 1) == INV
    # a fine call gets as far as the device
    assert c(conv()) == CUDA


@pytest.mark.parametrize("name,names,step", [
    ("kda_ssm_scan_fwd", SSM_FWD, False), ("kda_ssm_scan_bwd", SSM_BWD, False),
    ("kda_ssm_step", SSM_STEP, True)])
def test_ssm(lib, name, names, step):
    def c(shape, **over):
        return call(lib, name, shape, names, over)
    assert c(None) == INV
    for bad in (dict(T=-1), dict(D=0), dict(S=0), dict(G=0), dict(G=3),
                dict(io_dtype=2), dict(u_stride=63), dict(delta_stride=1),
                dict(z_stride=-1), dict(b_group_stride=15),
                dict(b_stride=31), dict(c_stride=31),
                dict(c_group_stride=20, c_stride=32),
                dict(u_stride=1 << 40), dict(b_stride=2 ** 62),
                dict(c_group_stride=2 ** 62)):
        assert c(ssm(**bad)) == INV, bad
    for bad in (dict(S=129), dict(D=1 << 21), dict(T=2 ** 31 - 1)):
        assert c(ssm(**bad)) == UNS, bad
    for n in ("u", "delta", "A", "B", "C"):
        assert c(ssm(), **{n: None}) == INV, n
    assert c(ssm(), u=BASE + GAP + 1) == MIS
    assert c(ssm(), A=BASE + 3 * GAP + 2) == MIS
    out = "du" if "du" in names else "out"
    assert c(ssm(), **{out: None}) == INV
    assert c(ssm(), **{out: 1}) == INV
    if step:
        assert c(ssm(), state=None) == INV
    else:
        assert c(ssm(B=2)) == INV
        assert c(ssm(n_seqs=0)) == INV
    if "final" in names:
        # the final state may be the initial state, but not part of it
        at = BASE + (names.index("h0") + 1) * GAP
        assert c(ssm(), final=at + 16) == INV
        assert c(ssm(), final=at) == CUDA
    if "dz" in names:
        for n, i in (("skip", "dskip"), ("z", "dz"), ("bias", "dbias")):
            assert c(ssm(), **{n: None}) == INV, n      # gradient without input
        assert c(ssm(), dz=None) == INV                 # z without its gradient
        assert c(ssm(), dA=None) == INV
        assert c(ssm(), dB=names.index("dC") + 1) == INV
    assert c(ssm()) == CUDA


@pytest.mark.parametrize("name,names", [("kda_block_norm_fwd", NORM_FWD),
                                        ("kda_block_norm_bwd", NORM_BWD)])
def test_norm(lib, name, names):
    def c(shape, **over):
        return call(lib, name, shape, names, over)
    assert c(None) == INV
    for bad in (dict(tokens=-1), dict(heads=0), dict(width=0),
                dict(io_dtype=9), dict(residual_dtype=2), dict(gate_act=3),
                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(x_stride=127), dict(gate_stride=-128),
                dict(x_stride=1 << 40)):
        assert c(norm(**bad)) == INV, bad
    for bad in (dict(width=16385), dict(io_dtype=1, residual_dtype=0),
                dict(tokens=1 << 40), dict(heads=65536)):
        assert c(norm(**bad)) == UNS, bad
    assert c(norm(), x=None) == INV
    assert c(norm(), x=BASE + GAP + 1) == MIS
    if name.endswith("fwd"):
        assert c(norm(), out=None) == INV
        assert c(norm(), normed=None) == INV
        assert c(norm(), pre=None) == INV           # normed without a weight
        assert c(norm(), out=1) == INV              # over x
        at = BASE + (names.index("residual") + 1) * GAP
        assert c(norm(), out=at) == CUDA            # in place
        assert c(norm(), out=at + 4) == INV
    else:
        for n in ("post", "gate", "residual", "scale", "pre"):
            assert c(norm(), **{n: None}) == INV, n
        assert c(norm(), dgate=None) == INV
        assert c(norm(), dx=names.index("d_out") + 1) == INV
    assert c(norm()) == CUDA
