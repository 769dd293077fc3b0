"""What the helpers of the operators around the mixer accept, without a GPU: the device check is
put aside, so that a helper fills its struct (or refuses) from CPU tensors."""
import pytest

from test_abi import hm   # noqa: F401  (the fixture that builds and imports the package)


@pytest.fixture
def on_cpu(hm, monkeypatch):    # noqa: F811
    monkeypatch.setattr(hm, "_one_device", lambda *a: None)
    return hm


def _broadcast():
    """[.., 8] tensors with a broadcast leading axis, over few stored rows."""
    import torch
    return (torch.zeros(4, 1, 8).expand(4, 6, 8), torch.zeros(6, 8).expand(4, 6, 8), torch.zeros(1, 8).expand(4, 6, 8),
            torch.zeros(4, 3, 1, 8).expand(4, 3, 6, 8), torch.zeros(4, 1, 6, 8).expand(4, 3, 6, 8))


@pytest.mark.parametrize("i", range(5))
def test_row_stride_refuses_broadcast_axes(hm, i):      # noqa: F811
    with pytest.raises(ValueError, match="repeats its rows"):
        hm._row_stride(_broadcast()[i])


def test_row_stride_of_what_is_equally_spaced(hm):      # noqa: F811
    import torch
    z = torch.zeros(4, 6, 24)
    for t, want in ((z, 24), (z[..., :8], 24), (z[:, ::2, :8], 48), (z[:1, :, 8:], 24), (z[:, :1], 144),
                    (z[:1, :1, :8], 8), (z[:, 2], 144), (torch.zeros(1, 1, 8).expand(1, 1, 8), 8),
                    (torch.zeros(4, 0, 8), 8), (torch.zeros(0, 3, 8)[..., :4], 4)):
        assert hm._row_stride(t) == want, (tuple(t.shape), t.stride())
    with pytest.raises(ValueError, match="equally spaced"):
        hm._row_stride(z[:, :4])


def test_seam_helpers_refuse_broadcast_rows(on_cpu):
    """Among them the gradient that comes back through a sum over the tokens."""
    import torch
    y = torch.zeros(4, 6, 8, requires_grad=True)
    grad = []
    z = y * 1.0
    z.register_hook(grad.append)
    z.sum(1).backward(torch.zeros(4, 8))
    assert grad[0].shape == y.shape and grad[0].stride() == (8, 0, 1)
    with pytest.raises(ValueError, match="not contiguous"):     # and that of a sum over everything
        on_cpu.norm_gate_bwd_args(y, y, torch.zeros(1, 1, 1).expand(4, 6, 8), y, y, y)
    y, e = y.detach(), [torch.zeros(4, 6, 8) for _ in range(3)]
    for b in (grad[0], *_broadcast()[:3]):
        for call in (lambda: on_cpu.norm_gate_args(b, y, e[0], e[1]), lambda: on_cpu.norm_gate_args(y, b, e[0], e[1]),
                     lambda: on_cpu.norm_gate_args(y, y, e[0], e[1], gate=b),
                     lambda: on_cpu.norm_gate_args(y, y, b, e[1]), lambda: on_cpu.norm_gate_args(y, y, e[0], b),
                     lambda: on_cpu.norm_gate_bwd_args(b, y, y, y, e[0], e[1]),
                     lambda: on_cpu.norm_gate_bwd_args(y, b, y, y, e[0], e[1]),
                     lambda: on_cpu.norm_gate_bwd_args(y, y, b, y, e[0], e[1]),
                     lambda: on_cpu.norm_gate_bwd_args(y, y, y, b, e[0], e[1]),
                     lambda: on_cpu.norm_gate_bwd_args(y, y, y, y, e[0], b),
                     lambda: on_cpu.norm_gate_bwd_args(y, y, y, y, e[0], e[1], gate=b, dgate=e[2]),
                     lambda: on_cpu.norm_gate_bwd_args(y, y, y, y, e[0], e[1], gate=y, dgate=b)):
            with pytest.raises(ValueError, match="repeats its rows"):
                call()
        a = on_cpu.norm_gate_args(y, b.contiguous(), e[0], e[1])
        assert (a.rows, a.D, a.r_stride) == (24, 8, 8)


def test_buffers_are_dense(on_cpu):
    """A buffer of repeated or spaced bytes has fewer of its own than its count says."""
    import torch
    B, L, D = 2, 5, 8
    x, p, u8 = torch.zeros(B, L, D), torch.zeros(D), torch.uint8
    dense = torch.zeros(1 << 12, dtype=u8)
    for bad in (torch.zeros(1, dtype=u8).expand(1 << 12), torch.zeros(1 << 13, dtype=u8)[::2]):
        for call in (lambda: on_cpu.gated_scan_args(x, x, x, p, states=bad),
                     lambda: on_cpu.gated_scan_bwd_args(x, x, x, x, x, p, p, bad),
                     lambda: on_cpu.gated_scan_bwd_args(x, x, x, x, x, p, p, dense, workspace=bad),
                     lambda: on_cpu.norm_gate_bwd_args(x, x, x, x, x, x, workspace=bad)):
            with pytest.raises(ValueError, match="must be contiguous"):
                call()
    a = on_cpu.gated_scan_bwd_args(x, x, x, x, x, p, p, dense, workspace=dense[256:])
    assert (a.states_bytes, a.workspace_bytes) == (1 << 12, (1 << 12) - 256)


def test_helpers_without_the_native_filler(on_cpu, monkeypatch):
    """Where _marshal cannot be imported the helpers fill their structs in Python, with one warning."""
    import sys
    import torch
    monkeypatch.setitem(sys.modules, on_cpu.__name__ + "._marshal", None)
    monkeypatch.delattr(on_cpu, "_marshal", raising=False)
    monkeypatch.setattr(on_cpu, "_native", None)
    x, p = torch.zeros(2, 5, 8), torch.zeros(8)
    with pytest.warns(RuntimeWarning, match="_marshal.so cannot be used"):
        a = on_cpu.gated_scan_args(x, x, x, p)
    assert (a.B, a.L, a.D, a.x) == (2, 5, 8, x.data_ptr())
    # a buffer as before there was a filler: a dense allocation, its start moved to 256 bytes
    empty = torch.empty
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch, "empty", lambda *s, device=None, **kw: empty(*s, **kw))
    buf = on_cpu.alloc_workspace(1000)
    assert buf.numel() >= 1000 and buf.data_ptr() % 256 == 0
