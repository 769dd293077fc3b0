"""What the helpers of the operators around the mixer accept, on the GPU, where the native
filler looks at the tensors first."""
import numpy as np
import pytest

import workloads as wl
from gpu_common import dev_tensor, to_np
from oracle import around

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hm():
    import torch
    assert torch.cuda.is_available()
    import selective_ssm_sequence_b200 as mod
    return mod


def _rand(name, shape):
    return wl.round_f32(np.asarray(wl.normal(61, name, shape)))


def test_seam_takes_no_broadcast_rows(hm):
    """Forward and backward refuse rows repeated along an axis; a dense copy of them gives the
    definition's result.  Elements are sums of a few products whose fp32 errors are 2^-18 of the
    sum of their absolute values, which is below 8 for rows of 8 values of order one whose rms
    is above 1/2 (asserted): 2^-15."""
    import torch
    B, L, D = 4, 6, 8
    y, g = dev_tensor(_rand("y", (B, L, D)), "f32"), dev_tensor(_rand("g", (B, 1, D)), "f32").expand(B, L, D)
    o, x, dy, dr, dg = (torch.empty(B, L, D, device="cuda") for _ in range(5))
    f = lambda *a, **k: hm.hm_norm_gate_fwd(hm.norm_gate_args(*a, **k))     # noqa: E731
    for call in (lambda: f(y, g, o, x), lambda: f(g, y, o, x), lambda: f(y, y, o, x, gate=g), lambda: f(y, y, g, x),
                 lambda: hm.norm_gate_bwd_args(y, y, g, y, dy, dr), lambda: hm.norm_gate_bwd_args(y, y, y, g, dy, dr),
                 lambda: hm.norm_gate_bwd_args(y, g, y, y, dy, dr),
                 lambda: hm.norm_gate_bwd_args(y, y, y, y, dy, dr, gate=g, dgate=dg)):
        with pytest.raises(ValueError, match="repeats its rows"):
            call()
    f(y, y, o, x, gate=g.contiguous())
    rows = lambda t: to_np(t).reshape(-1, D)                                # noqa: E731
    assert all(np.sqrt((rows(t) ** 2).mean(-1)).min() > 0.5 for t in (y, o))
    want = around.norm_gate(rows(y), rows(y), rows(g))
    for got, w in zip((o, x), want):
        assert np.allclose(rows(got), w, rtol=0, atol=2.0 ** -15)
    b = hm.norm_gate_bwd_args(y, o, g.contiguous(), x, dy, dr)
    ws = hm.alloc_workspace(hm.hm_norm_gate_bwd_workspace_size(b))
    b.workspace, b.workspace_bytes = ws.data_ptr(), ws.numel()
    hm.hm_norm_gate_bwd(b)
    want = around.norm_gate_bwd(rows(y), rows(o), rows(g), rows(x), None)
    assert np.allclose(rows(dr), want["dr"], rtol=0, atol=2.0 ** -15)
    assert np.allclose(rows(dy), want["dy"], rtol=0, atol=2.0 ** -15)


def test_buffers_are_dense(hm):
    import torch
    x, p, u8 = torch.zeros(2, 5, 8, device="cuda"), torch.zeros(8, device="cuda"), torch.uint8
    dense = torch.zeros(1 << 12, dtype=u8, device="cuda")
    for bad in (torch.zeros(1, dtype=u8, device="cuda").expand(1 << 12), dense[::2]):
        for call in (lambda: hm.gated_scan_args(x, x, x, p, states=bad),
                     lambda: hm.gated_scan_bwd_args(x, x, x, x, x, p, p, bad),
                     lambda: hm.gated_scan_bwd_args(x, x, x, x, x, p, p, dense, workspace=bad),
                     lambda: hm.norm_gate_bwd_args(x, x, x, x, x, x, workspace=bad)):
            with pytest.raises(ValueError, match="must be contiguous"):
                call()
    assert hm.gated_scan_args(x, x, x, p, states=dense).states_bytes == 1 << 12


@pytest.mark.parametrize("io,n,D", [("bf16", 37, 64), ("bf16", 5, 2048), ("bf16", 9, 6000), ("bf16", 11, 302),
                                    ("f32", 7, 1001), ("f32", 300, 512)])
def test_seam_forward_in_place(hm, io, n, D):
    """r_out and xn over any of y, gate and r, in each form of the forward: the same bits."""
    import torch
    src = [dev_tensor(_rand(k, (n, D)), io) for k in ("y", "gate", "r")]
    o, x = torch.empty_like(src[0]), torch.empty_like(src[0])

    def run(y, gate, r, o, x):
        hm.hm_norm_gate_fwd(hm.norm_gate_args(y, r, o, x, gate=gate, norm=hm.HM_NORM_LAYER, alpha=0.7))
    run(*src, o, x)
    for i in range(3):
        for j in range(3):
            if i != j:
                t = [s.clone() for s in src]
                run(*t, t[i], t[j])
                assert torch.equal(t[i], o) and torch.equal(t[j], x), (i, j)
