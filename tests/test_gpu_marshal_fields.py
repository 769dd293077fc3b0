"""Every field of the argument structs against the tensor it stands for: a tensor, and where rows
may be strided a stride, of its own for every argument, through both fillers."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["native", "python"])
def hm(request, monkeypatch):
    import torch
    assert torch.cuda.is_available()
    import selective_ssm_sequence_b200 as mod
    if request.param == "python":
        monkeypatch.setattr(mod, "_native", mod._NoFiller())
    else:
        assert mod._filler().__name__.endswith("_marshal")
    return mod


class _Rows:
    """[.., D] tensors, each with row strides that no other one has."""

    def __init__(self):
        self.n = 0

    def __call__(self, *shape, dtype=None):
        import torch
        self.n += 1
        return torch.zeros(*shape[:-1], shape[-1] + 8 * self.n, dtype=dtype or torch.bfloat16,
                           device="cuda")[..., :shape[-1]]


def _fields(a, tensors, strides=(), **plain):
    """The pointers of the struct, the named strides, and the rest as given."""
    for name, t in tensors.items():
        assert getattr(a, name) == t.data_ptr(), name
    for name, axes in strides:
        for suffix, axis in axes:
            assert getattr(a, "%s_stride%s" % (name, suffix)) == tensors[name].stride(axis), name
    for name, v in plain.items():
        assert getattr(a, name) == v, name
    given = set(tensors) | set(plain) | {n + "_stride" + s for n, axes in strides for s, _ in axes}
    assert given == {f[0] for f in a._fields_}
    assert len({t.data_ptr() for t in tensors.values()}) == len(tensors)


def test_recurrence(hm):
    import torch
    B, L, D = 3, 5, 24
    f = lambda *s: torch.zeros(*s, device="cuda")                           # noqa: E731
    u8 = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")         # noqa: E731
    rows = _Rows()
    t = {n: rows(B, L, D) for n in ("x", "dt", "y")}
    t |= dict(A_log=f(D), dt_bias=f(D), h0=f(B, D), h_out=f(B, D), states=u8(512),
              lengths=torch.zeros(B, dtype=torch.int32, device="cuda"))
    axes = (("_b", 0), ("_t", 1))
    _fields(hm.gated_scan_args(**t, input_scale=2), t, [(n, axes) for n in ("x", "dt", "y")], B=B, L=L, D=D,
            io_dtype=hm.HM_BF16, input_scale=2, states_bytes=512)
    names = ("x", "dt", "dy", "dx", "ddt")
    t = {n: rows(B, L, D) for n in names}
    t |= dict(A_log=f(D), dA_log=f(D), states=u8(768), dt_bias=f(D), d_dt_bias=f(D), dh_out=f(B, D), dh0=f(B, D),
              lengths=torch.zeros(B, dtype=torch.int32, device="cuda"), workspace=u8(1024))
    _fields(hm.gated_scan_bwd_args(**t, input_scale=1), t, [(n, axes) for n in names], B=B, L=L, D=D,
            io_dtype=hm.HM_BF16, input_scale=1, states_bytes=768, workspace_bytes=1024)
    t = {n: rows(B, D) for n in ("x", "dt", "y")}
    t |= dict(h=f(B, D), h_out=f(B, D), A_log=f(D), dt_bias=f(D))
    _fields(hm.gated_step_args(**t, input_scale=1), t, [(n, (("", 0),)) for n in ("x", "dt", "y")], B=B, D=D,
            io_dtype=hm.HM_BF16, input_scale=1)


def test_seam(hm):
    import torch
    n, D = 6, 16
    f = lambda: torch.zeros(D, device="cuda")                               # noqa: E731
    rows = _Rows()
    names = ("y", "r", "r_out", "xn", "gate")
    t = {k: rows(n, D, dtype=torch.float32) for k in names}
    t |= {k: f() for k in ("scale", "post_w", "post_b", "pre_w", "pre_b")}
    plain = dict(rows=n, D=D, io_dtype=hm.HM_F32, norm=1, post=0, eps=0.25, alpha=0.5)
    _fields(hm.norm_gate_args(**t, norm=1, post=False, eps=0.25, alpha=0.5), t, [(k, (("", 0),)) for k in names], **plain)
    names = ("y", "r_out", "dr_out", "dxn", "dy", "dr", "gate", "dgate")
    t = {k: rows(n, D, dtype=torch.float32) for k in names}
    t |= {k: f() for k in ("scale", "post_w", "post_b", "pre_w", "dscale", "dpost_w", "dpost_b", "dpre_w", "dpre_b")}
    t["workspace"] = torch.zeros(512, dtype=torch.uint8, device="cuda")
    _fields(hm.norm_gate_bwd_args(**t, norm=1, post=False, eps=0.25, alpha=0.5), t, [(k, (("", 0),)) for k in names],
            workspace_bytes=512, **plain)


def test_rotary(hm):
    import torch
    B, L, d = 2, 5, 16
    rows = _Rows()
    t = dict(q=rows(B, L, 4, d), k=rows(B, L, 2, d), q_out=rows(B, L, 4, d), k_out=rows(B, L, 2, d))
    t["positions"] = torch.zeros(B, 2 * L, dtype=torch.int64, device="cuda")[:, ::2]
    plain = dict(layout=1, scaling=3, transpose=1, rot=8, base=5e5, factor=8.0, orig_len=100.0, beta_slow=0.5,
                 beta_fast=20.0, mscale=1.25, pos0=7)
    a = hm.rotary_args(**t, **plain)
    assert (a.pos_stride_b, a.pos_stride_t) == (2 * L, 2)
    _fields(a, t, [(n, (("_b", 0), ("_t", 1), ("_h", 2))) for n in ("q", "k", "q_out", "k_out")], B=B, L=L, Hq=4, Hk=2,
            d=d, io_dtype=hm.HM_BF16, pos_stride_b=2 * L, pos_stride_t=2, **plain)
