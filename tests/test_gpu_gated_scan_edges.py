"""The gated recurrence where its gates leave the ordinary range."""
import numpy as np
import pytest

import workloads as wl
from gpu_common import dev_tensor, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hm():
    import torch
    assert torch.cuda.is_available()
    import selective_ssm_sequence_b200 as mod
    return mod


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("scale", ["HM_INPUT_PLAIN", "HM_INPUT_UNIT"])
@pytest.mark.parametrize("L,D,n", [(1, 64, None), (5, 64, None), (70, 65, None), (300, 64, (300, 0, 37)),
                                   (300, 33, (299, 1, 16))])
@pytest.mark.parametrize("bias", [1e30, 2.9e38, float("inf")])
def test_a_bias_that_forgets_all(hm, io, scale, L, D, n, bias):
    """Steps that large leave a = 0 and beta = 1, so h_t = x_t and g_t = dy_t with dh_out at the
    last token, and nothing else has a gradient; the ends of sequences inside a run of tokens
    must not see the bias.  beta = sqrt(1 - 0) and products with it are exact or off by units of
    2^-24; a result is rounded once to the io type."""
    import torch
    B, rnd = 3, wl.round_bf16 if io == "bf16" else wl.round_f32
    x, dt, dy = (rnd(np.asarray(wl.normal(71, k, (B, L, D)))) for k in ("x", "dt", "dy"))
    dh = wl.round_f32(np.asarray(wl.normal(71, "dh", (B, D))))
    h0 = wl.round_f32(np.asarray(wl.normal(71, "h0", (B, D))))
    f32 = lambda *s: torch.full(s, 7.0, device="cuda")      # noqa: E731
    tx, tdt, tdy = (dev_tensor(v, io) for v in (x, dt, dy))
    y, dx, ddt = (torch.full_like(tx, 7.0) for _ in range(3))
    A, b, h, dA, db, dh0 = f32(D) * 0, f32(D) * 0 + bias, f32(B, D), f32(D), f32(D), f32(B, D)
    lengths = None if n is None else torch.tensor(n, dtype=torch.int32, device="cuda")
    kw = dict(dt_bias=b, lengths=lengths, input_scale=getattr(hm, scale))
    a = hm.gated_scan_args(tx, tdt, y, A, h0=dev_tensor(h0, "f32"), h_out=h, **kw)
    st = hm.alloc_workspace(hm.hm_gated_scan_states_size(a))
    a.states, a.states_bytes = st.data_ptr(), st.numel()
    hm.hm_gated_scan_fwd(a)
    g = hm.gated_scan_bwd_args(tx, tdt, tdy, dx, ddt, A, dA, st, d_dt_bias=db, dh_out=dev_tensor(dh, "f32"), dh0=dh0,
                               **kw)
    ws = hm.alloc_workspace(hm.hm_gated_scan_bwd_workspace_size(g))
    g.workspace, g.workspace_bytes = ws.data_ptr(), ws.numel()
    hm.hm_gated_scan_bwd(g)
    half = 2.0 ** -8 if io == "bf16" else 2.0 ** -22
    near = lambda got, want, r: np.all(np.abs(to_np(got) - want) <= r * np.abs(want))   # noqa: E731
    for s in range(B):
        m = L if n is None else n[s]
        assert near(y[s, :m], x[s, :m], half) and (y[s, m:] == 7.0).all()
        assert near(h[s], x[s, m - 1] if m else h0[s], 2.0 ** -22)
        want = dy[s, :m].copy()
        if m:
            want[-1] += dh[s]
        assert near(dx[s, :m], want, half) and (dx[s, m:] == 7.0).all()
        assert not ddt[s, :m].any() and (ddt[s, m:] == 7.0).all()
        assert near(dh0[s], dh[s] if m == 0 else 0 * dh[s], 0.0)
    assert not dA.any() and not db.any()
    assert hm.hm_get_device_error() == hm.HM_OK


@pytest.mark.parametrize("bias", [1e30, 2.9e38, float("inf")])
def test_one_token(hm, bias):
    import torch
    x = dev_tensor(wl.round_f32(np.asarray(wl.normal(72, "x", (3, 40)))), "f32")
    h, y, A = torch.ones_like(x), torch.zeros_like(x), torch.zeros(40, device="cuda")
    hm.hm_gated_scan_step(hm.gated_step_args(x, x, y, h, h, A, dt_bias=torch.full_like(A, bias)))
    assert torch.equal(y, x) and torch.equal(h, x)


FIRST_CALL = r"""
import torch
import selective_ssm_sequence_b200 as hm
B, L, D = 1, 4096, 128       # few channels: clusters of 16
g = torch.Generator(device="cuda").manual_seed(3)
x, dt, dy = (torch.randn(B, L, D, generator=g, device="cuda").bfloat16() for _ in range(3))
A, dA, y, dx, ddt = torch.zeros(D, device="cuda"), torch.zeros(D, device="cuda"), *(torch.zeros_like(x) for _ in range(3))
a = hm.gated_scan_args(x, dt, y, A)
st = hm.alloc_workspace(hm.hm_gated_scan_states_size(a))
a = hm.gated_scan_args(x, dt, y, A, states=st)
b = hm.gated_scan_bwd_args(x, dt, dy, dx, ddt, A, dA, st)
ws = hm.alloc_workspace(hm.hm_gated_scan_bwd_workspace_size(b))
b = hm.gated_scan_bwd_args(x, dt, dy, dx, ddt, A, dA, st, workspace=ws)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    hm.hm_gated_scan_fwd(a)
    hm.hm_gated_scan_bwd(b)
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (y, dx, ddt, dA)]
hm.hm_gated_scan_fwd(a)
hm.hm_gated_scan_bwd(b)
assert all(torch.equal(s, t) for s, t in zip(got, (y, dx, ddt, dA))) and dA.abs().sum() > 0
assert hm.hm_get_device_error() == hm.HM_OK
"""


def test_a_process_whose_first_call_is_captured():
    """What the library asks the device about clusters of 16 it may ask while a stream is captured."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
