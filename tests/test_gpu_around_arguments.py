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


@pytest.mark.parametrize("io,n,D", [("bf16", 37, 64), ("bf16", 301, 2048), ("bf16", 150, 6000), ("bf16", 9, 302),
                                    ("f32", 7, 8192), ("f32", 11, 1001), ("bf16", 5, 16384)])
def test_seam_backward_in_place(hm, io, n, D):
    """Each output over each input that the header lets it lie over, in each form of the backward:
    the same bits; and two or three of them at once."""
    import torch
    names = ("y", "gate", "r_out", "dr_out", "dxn")
    src = {k: dev_tensor(_rand(k, (n, D)), io) for k in names}

    def run(t, dy, dgate, dr):
        d = {k: torch.empty(D, device="cuda") for k in ("dscale", "dpost_w", "dpre_b")}
        kw = dict(gate=t["gate"], dgate=dgate, norm=hm.HM_NORM_LAYER, alpha=0.7, **d)
        b = hm.norm_gate_bwd_args(t["y"], t["r_out"], t["dr_out"], t["dxn"], dy, dr, **kw)
        ws = hm.alloc_workspace(hm.hm_norm_gate_bwd_workspace_size(b))
        hm.hm_norm_gate_bwd(hm.norm_gate_bwd_args(t["y"], t["r_out"], t["dr_out"], t["dxn"], dy, dr, workspace=ws, **kw))
        return [dy, dgate, dr, *d.values()]
    want = run(src, *(torch.empty_like(src["y"]) for _ in range(3)))
    may = {0: names, 1: names[1:], 2: names[2:]}
    plans = [{o: k} for o in range(3) for k in may[o]]
    plans += [{0: "y", 1: "gate", 2: "r_out"}, {0: "dxn", 1: "dr_out", 2: "r_out"}, {0: "gate", 1: "r_out", 2: "dxn"}]
    for plan in plans:
        t = {k: v.clone() for k, v in src.items()}
        out = [t[plan[o]] if o in plan else torch.empty_like(src["y"]) for o in range(3)]
        assert all(torch.equal(a, b) for a, b in zip(run(t, *out), want)), plan


@pytest.fixture(params=["native", "python"])
def filler(hm, monkeypatch, request):
    """With the native filler, and with the helpers on their own."""
    if request.param == "python":
        monkeypatch.setattr(hm, "_native", hm._NoFiller())
    else:
        assert hm._filler().__name__.endswith("_marshal")
    return hm


def _buf(hm, n):
    b = hm.alloc_workspace(n)
    assert b.data_ptr() % 256 == 0 and b.numel() >= n
    return b


def test_recurrence_through_both_fillers(filler):
    """Every argument a tensor of its own, so that none can stand for another.  fp32 against the
    definition: a rounding, 2^-24, and 2^-19 of the magnitudes that the definition returns (gates
    good to a few 2^-22, carried through the recurrence); all |z| here are below 32."""
    import torch
    B, L, D = 3, 40, 24
    f = lambda n, *s: dev_tensor(_rand(n, s), "f32")                        # noqa: E731
    x, dt, dy, A, bias, dh = f("x", B, L, D), f("dt", B, L, D), f("dy", B, L, D), f("A", D), f("b", D), f("dh", B, D)
    h0 = f("h0", B, D)
    e = lambda *s: torch.full(s, 7.0, device="cuda")                        # noqa: E731
    y, h, dx, ddt, dA, db, dh0 = e(B, L, D), e(B, D), e(B, L, D), e(B, L, D), e(D), e(D), e(B, D)
    lengths = torch.tensor([40, 0, 17], dtype=torch.int32, device="cuda")
    a = filler.gated_scan_args(x, dt, y, A, dt_bias=bias, h0=h0, h_out=h, lengths=lengths, input_scale=1)
    st = _buf(filler, filler.hm_gated_scan_states_size(a))
    filler.hm_gated_scan_fwd(filler.gated_scan_args(x, dt, y, A, dt_bias=bias, h0=h0, h_out=h, lengths=lengths,
                                                    input_scale=1, states=st))
    kw = dict(dt_bias=bias, d_dt_bias=db, dh_out=dh, dh0=dh0, lengths=lengths, input_scale=1)
    b = filler.gated_scan_bwd_args(x, dt, dy, dx, ddt, A, dA, st, **kw)
    ws = _buf(filler, filler.hm_gated_scan_bwd_workspace_size(b))
    filler.hm_gated_scan_bwd(filler.gated_scan_bwd_args(x, dt, dy, dx, ddt, A, dA, st, workspace=ws, **kw))
    assert filler.hm_get_device_error() == filler.HM_OK

    def near(got, want, mag):
        assert np.all(np.abs(got - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -19 * mag + 1e-37)
    o = [to_np(t) for t in (x, dt, dy, A, bias)]
    o = dict(x=o[0], dt=o[1], A_log=o[3], dt_bias=o[4], h0=to_np(h0), lengths=lengths.cpu().numpy(), scale=around.STEP)
    wy, wh, mag = around.gated_scan(**o)
    g = around.gated_scan_bwd(dy=to_np(dy), dh_out=to_np(dh), **o)
    for s, n in enumerate((40, 0, 17)):
        near(to_np(y[s, :n]), wy[s, :n], mag[s, :n])
        near(to_np(h[s]), wh[s], mag[s, n - 1] if n else 0.0)
        for got, k in ((dx, "dx"), (ddt, "ddt")):
            near(to_np(got[s, :n]), g[k][0][s, :n], g[k][1][s, :n])
    for got, k in ((dA, "dA_log"), (db, "d_dt_bias"), (dh0, "dh0")):
        near(to_np(got), *g[k])
    yt, ht = e(B, D), e(B, D)
    filler.hm_gated_scan_step(filler.gated_step_args(x[:, 0], dt[:, 1], yt, h0, ht, A, dt_bias=bias, input_scale=2))
    wy, wh, mag = around.gated_scan(o["x"][:, :1], o["dt"][:, 1:2], o["A_log"], o["dt_bias"], h0=o["h0"],
                                    scale=around.UNIT)
    near(to_np(yt), wy[:, 0], mag[:, 0])
    near(to_np(ht), wh, mag[:, 0])


def test_seam_through_both_fillers(filler):
    """As above; a result is a sum of a few products whose errors are 2^-18 of their absolute sum.
    The terms are products of up to eight values of order one (at most 4, most below 1) over a
    row's deviation above 1/2, and the parameters' gradients sum 10 rows of them: below 2^8."""
    import torch
    n, D = 10, 48
    f = lambda k, *s: dev_tensor(_rand(k, s), "f32")                        # noqa: E731
    y, gate, r, dr_out, dxn = (f(k, n, D) for k in ("y", "gate", "r", "dr", "dxn"))
    scale, post_w, post_b, pre_w, pre_b = (f(k, D) for k in ("sc", "w1", "b1", "w2", "b2"))
    e = lambda *s: torch.full(s, 7.0, device="cuda")                        # noqa: E731
    r_out, xn, dy, dgate, dr = (e(n, D) for _ in range(5))
    d = {k: e(D) for k in ("dscale", "dpost_w", "dpost_b", "dpre_w", "dpre_b")}
    kw = dict(norm=1, eps=1e-4, alpha=0.5, scale=scale, post_w=post_w, post_b=post_b, pre_w=pre_w)
    filler.hm_norm_gate_fwd(filler.norm_gate_args(y, r, r_out, xn, gate=gate, pre_b=pre_b, **kw))
    b = filler.norm_gate_bwd_args(y, r_out, dr_out, dxn, dy, dr, gate=gate, dgate=dgate, **d, **kw)
    ws = _buf(filler, filler.hm_norm_gate_bwd_workspace_size(b))
    filler.hm_norm_gate_bwd(filler.norm_gate_bwd_args(y, r_out, dr_out, dxn, dy, dr, gate=gate, dgate=dgate,
                                                      workspace=ws, **d, **kw))
    o = dict(layer=True, eps=1e-4, alpha=0.5, scale=to_np(scale), post_w=to_np(post_w), post_b=to_np(post_b),
             pre_w=to_np(pre_w))
    want = around.norm_gate(to_np(y), to_np(r), to_np(gate), pre_b=to_np(pre_b), **o)
    back = around.norm_gate_bwd(to_np(y), to_np(r_out), to_np(dr_out), to_np(dxn), to_np(gate), **o)
    got = dict(d, dy=dy, dr=dr, dgate=dgate)
    for g, w in [(r_out, want[0]), (xn, want[1])] + [(got[k], back[k]) for k in got]:
        assert np.abs(to_np(g) - w).max() < 2.0 ** -10


def test_rotary_through_both_fillers(filler):
    """As above; the stated error of an angle and a rounding: 2^-21 of (|u| + |v|) < 2^3 mscale."""
    import torch
    B, L = 2, 9
    q, k = dev_tensor(_rand("q", (B, L, 4, 16)), "f32"), dev_tensor(_rand("k", (B, L, 2, 16)), "f32")
    oq, ok = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    pos = torch.tensor(np.random.default_rng(5).integers(0, 1000, (B, L)), device="cuda")
    kw = dict(rot=12, base=5e5, factor=8.0, orig_len=100.0, beta_slow=0.5, beta_fast=20.0, mscale=1.25)
    filler.hm_rotary(filler.rotary_args(q, k, oq, ok, layout=1, scaling=3, positions=pos, transpose=True, **kw))
    for got, x in ((oq, q), (ok, k)):
        want = around.rotary(to_np(x), pos.cpu().numpy(), interleaved=True, scaling="by_parts", transpose=True, **kw)
        assert np.abs(to_np(got) - want).max() < 2.0 ** -17
