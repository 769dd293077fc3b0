"""The native argument filler gives the same struct as the Python helpers, and leaves to them
(None) whatever it does not know; a call with tensors that it refuses raises as ever."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hm():
    import torch
    assert torch.cuda.is_available()
    import selective_ssm_sequence_b200 as mod
    return mod


class _Nothing:
    def __getattr__(self, name):
        return lambda *a: None


def _calls(hm):
    import torch
    e = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device="cuda")        # noqa: E731
    B, L, D = 3, 7, 24
    f = lambda *s: e(*s, t=torch.float32)                                           # noqa: E731
    i32, i64, u8 = torch.int32, torch.int64, torch.uint8
    xz = e(B, L, 2 * D)
    x, dt, y = xz[..., :D], xz[..., D:], e(B, L, D)
    p, h, n = f(D), f(B, D), e(B, t=i32)
    yield lambda: hm.gated_scan_args(x, dt, y, p)
    yield lambda: hm.gated_scan_args(x, dt, None, p, dt_bias=p, h0=h, h_out=h, lengths=n, input_scale=2,
                                     states=e(4096, t=u8))
    yield lambda: hm.gated_scan_bwd_args(x, dt, y, y, xz[..., :D], p, p, e(4096, t=u8))
    yield lambda: hm.gated_scan_bwd_args(x, dt, y, y, y, p, p, e(1024, t=torch.float32), dt_bias=p, d_dt_bias=p,
                                         dh_out=h, dh0=h, lengths=n, input_scale=1, workspace=e(512, t=u8))
    yield lambda: hm.gated_step_args(x[:, 0], dt[:, 1], y[:, 2], h, h, p, dt_bias=p, input_scale=1)
    yield lambda: hm.norm_gate_args(y, y, y, None, gate=y, norm=1, post=False, eps=1e-6, alpha=0.25, scale=p, pre_w=p)
    yield lambda: hm.norm_gate_args(x[0], None, None, dt[1], post_w=p, post_b=p, pre_b=p)
    yield lambda: hm.norm_gate_bwd_args(y, y, y, y, y, y, gate=y, dgate=y, norm=1, scale=p, post_w=p, post_b=p, pre_w=p,
                                        dscale=p, dpost_w=p, dpost_b=p, dpre_w=p, dpre_b=p, workspace=e(512, t=u8))
    yield lambda: hm.norm_gate_bwd_args(x[0], None, dt[0], None, dt[1], None, post=False)
    q, k = e(B, L, 4, 16), e(B, L, 6, 16)[:, :, ::3]
    yield lambda: hm.rotary_args(q, k, q, k, rot=8, base=5e5, layout=1, scaling=3, factor=8.0, orig_len=4096,
                                 mscale=1.25, transpose=True, positions=e(1, L, t=i64))
    yield lambda: hm.rotary_args(q, None, q.clone(), None, pos0=1 << 40, positions=e(B, 1, t=i64), scaling=1, factor=2)


def test_same_structs(hm, monkeypatch):
    for call in list(_calls(hm)):
        native = call()
        with monkeypatch.context() as m:
            m.setattr(hm, "_filler", lambda: _Nothing())
            plain = call()
        for (name, _), at in zip(native._fields_, range(99)):
            a, b = getattr(native, name), getattr(plain, name)
            # buffers made within the call, and a clone, are new ones each time
            assert a == b or name in ("states", "workspace", "lengths", "positions", "q_out"), name


def test_gives_up_and_refuses(hm):
    import torch
    m = hm._filler()
    x, p = torch.zeros(2, 5, 8, device="cuda"), torch.zeros(8, device="cuda")
    none = [None] * 4
    assert m.gated_scan(x, x, None, p, None, *none, 0) is not None
    for bad in (x.cpu(), x.half(), x[:, :4], x.transpose(1, 2).contiguous().transpose(1, 2), 7, "x", None, x[0]):
        assert m.gated_scan(x, bad, None, p, None, *none, 0) is None
    assert m.gated_scan(x, x, None, p.double(), None, *none, 0) is None
    assert m.gated_scan(x, x, None, p, None, *none, 1 << 70) is None
    assert m.gated_scan(x, x, None, p[None], None, *none, 0) is None
    with pytest.raises(TypeError):
        m.gated_scan(x)
    with pytest.raises(ValueError, match="shape"):
        hm.gated_scan_args(x, x[:, :4], x, p)
    with pytest.raises(ValueError, match="float16"):
        hm.gated_step_args(x[0], x[0].half(), x[0], x[0], x[0], p)
    q = torch.zeros(2, 5, 4, 8, device="cuda")
    with pytest.raises(ValueError, match="come together"):
        hm.rotary_args(q, q, q, None)
    with pytest.raises(ValueError, match="positions"):
        hm.rotary_args(q, None, q, None, positions=torch.zeros(2, 4, dtype=torch.int64, device="cuda"))
    buf = hm.alloc_workspace(1000)
    assert buf.numel() >= 1000 and buf.data_ptr() % 256 == 0 and hm.alloc_workspace(0).numel() >= 1
