"""The operators around the mixer without a GPU: struct layouts against
include/hm.h, sizes, and the refusal of bad calls before anything is launched."""
import ctypes

import pytest

from test_abi import _c_layout, hm   # noqa: F401  (the fixture that builds and imports the package)

FAKE = 1 << 20      # an aligned address; validation never dereferences it


@pytest.mark.parametrize("cname,pyname", [("hm_gated_scan_args", "GatedScanArgs"),
                                          ("hm_gated_scan_bwd_args", "GatedScanBwdArgs"),
                                          ("hm_gated_step_args", "GatedStepArgs"),
                                          ("hm_norm_gate_args", "NormGateArgs"),
                                          ("hm_norm_gate_bwd_args", "NormGateBwdArgs"),
                                          ("hm_rotary_args", "RotaryArgs")])
def test_struct_layouts_match_the_header(hm, cname, pyname):    # noqa: F811
    cls = getattr(hm, pyname)
    fields = [f[0] for f in cls._fields_]
    size, offs = _c_layout(cname, fields)
    assert ctypes.sizeof(cls) == size
    assert [getattr(cls, f).offset for f in fields] == offs


def _fill(a, pointers, **kw):
    for n in pointers:
        setattr(a, n, FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _scan(hm, **kw):    # noqa: F811
    B, L, D = 3, 300, 512
    a = _fill(hm.GatedScanArgs(), ("x", "dt", "A_log"), B=B, L=L, D=D, io_dtype=hm.HM_BF16, y=2 * FAKE)
    for n in ("x", "dt", "y"):
        setattr(a, n + "_stride_b", L * D)
        setattr(a, n + "_stride_t", D)
    return _fill(a, (), **kw)


def _scan_bwd(hm, **kw):    # noqa: F811
    B, L, D = 3, 300, 512
    a = _fill(hm.GatedScanBwdArgs(), ("x", "dt", "dy", "A_log", "dA_log", "states", "workspace"), B=B, L=L, D=D,
              io_dtype=hm.HM_BF16, dx=2 * FAKE, ddt=3 * FAKE, states_bytes=1 << 30, workspace_bytes=1 << 30)
    for n in ("x", "dt", "dy", "dx", "ddt"):
        setattr(a, n + "_stride_b", L * D)
        setattr(a, n + "_stride_t", D)
    return _fill(a, (), **kw)


def test_gated_scan_refusals(hm):   # noqa: F811
    bad, uns = hm.HM_ERR_INVALID_ARG, hm.HM_ERR_UNSUPPORTED

    def call(**kw):
        return hm.lib.hm_gated_scan_fwd(ctypes.byref(_scan(hm, **kw)), None)
    assert call(B=-1) == bad and call(L=-1) == bad and call(D=0) == bad
    assert call(D=1 << 25) == uns
    assert call(io_dtype=7) == bad and call(input_scale=3) == bad and call(input_scale=-1) == bad
    for n in ("x", "dt", "A_log"):
        assert call(**{n: None}) == bad, n
    assert call(y=None) == bad                              # and neither h_out nor states
    assert b"NULL" in hm.lib.hm_last_error_detail()
    assert call(x=FAKE + 1) == bad and call(A_log=FAKE + 2) == bad and call(lengths=FAKE + 2) == bad
    assert call(x_stride_t=511) == bad and call(dt_stride_b=100) == bad and call(y_stride_t=0) == bad
    assert call(y=FAKE) == bad                              # y is x
    assert call(states=FAKE, states_bytes=16) == bad and b"states" in hm.lib.hm_last_error_detail()
    assert call(states=FAKE + 8, states_bytes=1 << 30) == bad
    assert hm.lib.hm_gated_scan_fwd(None, None) == bad
    assert call(B=0) == hm.HM_OK                            # nothing to do, nothing launched
    assert hm.hm_gated_scan_states_size(_scan(hm, D=0)) == 0
    one, two = (hm.hm_gated_scan_states_size(_scan(hm, L=L)) for L in (4096, 8192))
    assert 0 < one < two <= 2 * one and two <= 3 * 8192 * 512 // 8


def test_gated_scan_bwd_refusals(hm):   # noqa: F811
    bad = hm.HM_ERR_INVALID_ARG

    def call(**kw):
        return hm.lib.hm_gated_scan_bwd(ctypes.byref(_scan_bwd(hm, **kw)), None)
    for n in ("x", "dt", "dy", "dx", "ddt", "A_log", "dA_log", "states", "workspace"):
        assert call(**{n: None}) == bad, n
    assert call(dx=FAKE) == bad and call(ddt=2 * FAKE) == bad       # over x; over dx
    assert call(workspace_bytes=8) == bad and b"workspace" in hm.lib.hm_last_error_detail()
    assert call(workspace=FAKE + 16) == bad and call(states_bytes=64) == bad
    assert call(dy_stride_t=10) == bad and call(io_dtype=2) == bad and call(dh0=FAKE + 1) == bad
    assert hm.lib.hm_gated_scan_bwd(None, None) == bad
    assert hm.hm_gated_scan_bwd_workspace_size(_scan_bwd(hm)) > 0
    assert hm.hm_gated_scan_bwd_workspace_size(_scan_bwd(hm, B=-1)) == 0


def test_gated_step_refusals(hm):   # noqa: F811
    bad = hm.HM_ERR_INVALID_ARG

    def call(**kw):
        a = _fill(hm.GatedStepArgs(), ("x", "dt", "A_log", "h", "h_out"), B=4, D=512, io_dtype=hm.HM_F32,
                  y=2 * FAKE, x_stride=512, dt_stride=512, y_stride=512)
        return hm.lib.hm_gated_scan_step(ctypes.byref(_fill(a, (), **kw)), None)
    for n in ("x", "dt", "y", "A_log", "h", "h_out"):
        assert call(**{n: None}) == bad, n
    assert call(x_stride=500) == bad and call(y=FAKE) == bad and call(D=0) == bad and call(h=FAKE + 2) == bad
    assert call(B=0) == hm.HM_OK


def _seam(hm, cls, names, **kw):     # noqa: F811
    a = _fill(getattr(hm, cls)(), ("y",), rows=64, D=512, io_dtype=hm.HM_BF16, eps=1e-5, alpha=1.0, post=1)
    for i, n in enumerate(names):
        setattr(a, n, (i + 2) * FAKE)
        setattr(a, n + "_stride", 512)
    a.y_stride = 512
    return _fill(a, (), **kw)


def test_norm_gate_refusals(hm):    # noqa: F811
    bad, uns = hm.HM_ERR_INVALID_ARG, hm.HM_ERR_UNSUPPORTED

    def call(**kw):
        return hm.lib.hm_norm_gate_fwd(ctypes.byref(_seam(hm, "NormGateArgs", ("gate", "r", "r_out", "xn"), **kw)), None)
    assert call(y=None) == bad and call(r_out=None, xn=None) == bad and call(xn=4 * FAKE) == bad    # xn is r_out
    assert call(eps=0.0) == bad and call(eps=float("nan")) == bad and call(alpha=float("inf")) == bad
    assert call(norm=2) == bad and call(io_dtype=3) == bad and call(rows=-1) == bad and call(D=0) == bad
    assert call(D=16385) == uns and call(gate_stride=100) == bad and call(r=FAKE + 1) == bad
    assert call(pre_w=FAKE + 2) == bad
    assert hm.lib.hm_norm_gate_fwd(None, None) == bad
    assert call(rows=0) == hm.HM_OK

    rows = ("gate", "r_out", "dr_out", "dxn", "dy", "dgate", "dr")

    def back(**kw):
        a = _seam(hm, "NormGateBwdArgs", rows, workspace=FAKE, workspace_bytes=1 << 30)
        return hm.lib.hm_norm_gate_bwd(ctypes.byref(_fill(a, (), **kw)), None)
    for n in ("y", "r_out", "dy", "dgate", "workspace"):
        assert back(**{n: None}) == bad, n
    assert back(dr_out=None, dxn=None) == bad
    assert back(workspace_bytes=64) == bad and b"workspace" in hm.lib.hm_last_error_detail()
    assert back(workspace=FAKE + 64) == bad and back(dscale=FAKE + 1) == bad and back(dxn_stride=10) == bad
    assert back(D=20000) == uns
    assert hm.lib.hm_norm_gate_bwd(None, None) == bad
    assert hm.hm_norm_gate_bwd_workspace_size(_seam(hm, "NormGateBwdArgs", rows)) > 0
    assert hm.hm_norm_gate_bwd_workspace_size(_seam(hm, "NormGateBwdArgs", rows, eps=-1.0)) == 0


def test_rotary_refusals(hm):   # noqa: F811
    bad, uns = hm.HM_ERR_INVALID_ARG, hm.HM_ERR_UNSUPPORTED

    def call(**kw):
        B, L, H, d = 2, 100, 8, 128
        a = _fill(hm.RotaryArgs(), ("q", "k"), B=B, L=L, Hq=H, Hk=H, d=d, rot=64, io_dtype=hm.HM_BF16, base=1e4,
                  factor=1.0, orig_len=2048.0, beta_slow=1.0, beta_fast=32.0, mscale=1.0, q_out=2 * FAKE,
                  k_out=3 * FAKE)
        for n in ("q", "k", "q_out", "k_out"):
            for ax, st in (("b", L * H * d), ("t", H * d), ("h", d)):
                setattr(a, "%s_stride_%s" % (n, ax), st)
        return hm.lib.hm_rotary(ctypes.byref(_fill(a, (), **kw)), None)
    for n in ("q", "k", "q_out", "k_out"):
        assert call(**{n: None}) == bad, n
    assert call(rot=0) == bad and call(rot=63) == bad and call(rot=130) == bad and call(rot=-2) == bad
    assert call(d=2048, rot=64) in (bad, uns) and call(layout=2) == bad and call(scaling=4) == bad
    assert call(base=0.0) == bad and call(base=float("nan")) == bad and call(mscale=float("inf")) == bad
    assert call(scaling=hm.HM_ROTARY_LINEAR, factor=0.0) == bad
    assert call(scaling=hm.HM_ROTARY_NTK, rot=2) == bad
    assert call(scaling=hm.HM_ROTARY_BY_PARTS, beta_fast=1.0) == bad
    assert call(scaling=hm.HM_ROTARY_BY_PARTS, orig_len=0.0) == bad
    assert call(q_stride_h=100) == bad and call(k_out_stride_t=-5) in (bad, uns) and call(positions=FAKE + 4) == bad
    assert call(q_out=FAKE, q_out_stride_t=2048) == bad         # in place with other strides
    assert hm.lib.hm_rotary(None, None) == bad
    assert call(B=0) == hm.HM_OK and call(L=0) == hm.HM_OK


def test_helpers_refuse_what_the_library_cannot_see(hm):    # noqa: F811
    import torch
    x, p = torch.zeros(2, 5, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="shape"):
        hm.gated_scan_args(x, x[:, :4], x, p)
    with pytest.raises(ValueError, match="bfloat16"):
        hm.gated_scan_args(x, x.bfloat16(), x, p)
    with pytest.raises(ValueError, match="contiguous"):
        hm.gated_scan_args(x, x.transpose(1, 2).contiguous().transpose(1, 2), x, p)
    with pytest.raises(ValueError, match="A_log"):
        hm.gated_scan_args(x, x, x, p.double())
    with pytest.raises(ValueError, match="lengths"):
        hm.gated_scan_args(x, x, x, p, lengths=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="device memory"):
        hm.gated_scan_args(x, x, x, p)
    with pytest.raises(ValueError, match="equally spaced"):
        hm._row_stride(torch.zeros(4, 6, 8)[:, ::2][:, :2])
    assert hm._row_stride(torch.zeros(4, 6, 8)[:, :1]) == 48 and hm._row_stride(torch.zeros(4, 6, 8)) == 8
    q = torch.zeros(2, 5, 4, 8)
    with pytest.raises(ValueError, match="positions"):
        hm.rotary_args(q, None, q, None, positions=torch.zeros(2, 5, dtype=torch.int32))
    with pytest.raises(ValueError, match="shape"):
        hm.rotary_args(q, q[:, :4], q, q)


def test_helpers_refuse_tensors_of_another_device(hm, monkeypatch):     # noqa: F811
    import torch

    class On:
        is_cuda = True

        def __init__(self, dev):
            self.dev = dev

        def get_device(self):
            return self.dev
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    hm._one_device("x", On(0), None, On(0))
    with pytest.raises(ValueError, match="cuda:1"):
        hm._one_device("x", On(0), On(1))
