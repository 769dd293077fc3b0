"""Which arrays the outputs of the operators around the mixer may lie over, without a GPU: every
call here is refused on the host (the allowed ones by a later check, of another argument)."""
import ctypes

import pytest

from test_abi import hm   # noqa: F401  (the fixture that builds and imports the package)
from test_around_abi import FAKE, _fill, _scan_bwd, _seam

FWD = ("gate", "r", "r_out", "xn")
BWD = ("gate", "r_out", "dr_out", "dxn", "dy", "dgate", "dr")


def _detail(hm, entry, a):      # noqa: F811
    assert getattr(hm.lib, entry)(ctypes.byref(a), None) == hm.HM_ERR_INVALID_ARG
    return hm.lib.hm_last_error_detail().decode()


def _over(a, out, inp, stride=None):
    setattr(a, out, getattr(a, inp))
    if stride:
        setattr(a, out + "_stride", stride)
    return a


@pytest.mark.parametrize("out", ["r_out", "xn"])
@pytest.mark.parametrize("inp", ["y", "gate", "r"])
def test_seam_forward(hm, out, inp):        # noqa: F811
    def make():
        return _seam(hm, "NormGateArgs", FWD, pre_w=FAKE + 2)
    assert "misaligned parameter" in _detail(hm, "hm_norm_gate_fwd", _over(make(), out, inp))
    assert "%s is %s with another stride" % (out, inp) in _detail(hm, "hm_norm_gate_fwd", _over(make(), out, inp, 520))
    one = _fill(_over(make(), out, inp, 520), (), rows=1)       # a single row has no stride
    assert "misaligned parameter" in _detail(hm, "hm_norm_gate_fwd", one)


ALLOWED = {("dy", n) for n in ("y", "gate", "r_out", "dr_out", "dxn")}
ALLOWED |= {("dgate", n) for n in ("gate", "r_out", "dr_out", "dxn")} | {("dr", n) for n in ("r_out", "dr_out", "dxn")}


@pytest.mark.parametrize("out", ["dy", "dgate", "dr"])
@pytest.mark.parametrize("inp", ["y", "gate", "r_out", "dr_out", "dxn", "dy", "dgate", "dr"])
def test_seam_backward(hm, out, inp):       # noqa: F811
    if out == inp:
        return

    def make():
        return _seam(hm, "NormGateBwdArgs", BWD, workspace=None)
    same = _detail(hm, "hm_norm_gate_bwd", _over(make(), out, inp))
    other = _detail(hm, "hm_norm_gate_bwd", _over(make(), out, inp, 520))
    if (out, inp) in ALLOWED:
        assert "workspace" in same and "%s is %s with another stride" % (out, inp) in other
    else:
        assert "must not be" in same and "must not be" in other


def test_seam_backward_without_an_array(hm):    # noqa: F811
    """An input that is not read (r_out without dxn, dgate without a gate) stands in no one's way."""
    a = _seam(hm, "NormGateBwdArgs", BWD, workspace=None, dxn=None)
    assert "workspace" in _detail(hm, "hm_norm_gate_bwd", _over(a, "dr", "r_out"))
    a = _seam(hm, "NormGateBwdArgs", BWD, workspace=None, gate=None)
    assert "workspace" in _detail(hm, "hm_norm_gate_bwd", _over(a, "dgate", "dy"))


def test_parameter_gradients_are_arrays_of_their_own(hm):       # noqa: F811
    names = ("dscale", "dpost_w", "dpost_b", "dpre_w", "dpre_b")
    own = {n: (40 + i) * FAKE for i, n in enumerate(names)}
    assert "workspace" in _detail(hm, "hm_norm_gate_bwd", _seam(hm, "NormGateBwdArgs", BWD, workspace=None, **own))
    for i, n in enumerate(names):
        for m in names[:i]:
            a = _seam(hm, "NormGateBwdArgs", BWD, workspace=None, **dict(own, **{n: own[m]}))
            assert "parameter gradients are the same" in _detail(hm, "hm_norm_gate_bwd", a)
    a = _scan_bwd(hm, d_dt_bias=FAKE, workspace=None)
    assert "dA_log and d_dt_bias" in _detail(hm, "hm_gated_scan_bwd", a)


@pytest.mark.parametrize("out,inp", [("q_out", "k"), ("k_out", "q"), ("k_out", "q_out")])
def test_rotary(hm, out, inp):      # noqa: F811
    B, L, H, d = 2, 100, 8, 128
    a = _fill(hm.RotaryArgs(), (), B=B, L=L, Hq=H, Hk=H, d=d, rot=64, io_dtype=hm.HM_BF16, base=1e4, factor=1.0,
              mscale=1.0, q=FAKE, k=2 * FAKE, q_out=3 * FAKE, k_out=4 * FAKE)
    for n in ("q", "k", "q_out", "k_out"):
        for ax, st in (("b", L * H * d), ("t", H * d), ("h", d)):
            setattr(a, "%s_stride_%s" % (n, ax), st)
    assert "the other's array" in _detail(hm, "hm_rotary", _over(a, out, inp))
