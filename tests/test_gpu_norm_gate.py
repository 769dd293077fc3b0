"""The seam between two blocks (post-norm, gate, scaled residual, pre-norm) on
the GPU against its fp64 definition, forward and backward.

Tolerances: one rounding to the io type (eps / 2 of the value) on top of fp32
arithmetic.  An element is a sum of a few products of factors with relative
errors below 2^-20 (sums over a row run through trees of at most a few dozen
levels, rsqrt and exp to a few units of 2^-24), so 2^-18 of the sum of their
absolute values covers it; sums over rows likewise."""
import numpy as np
import pytest

import workloads as wl
from gpu_common import dev_tensor, to_np
from oracle import around

pytestmark = pytest.mark.gpu

DELTA = 2.0 ** -18
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
ROWS = ("y", "gate", "r", "r_out", "dr_out", "dxn")


@pytest.fixture(scope="module")
def hm():
    import torch
    assert torch.cuda.is_available()
    import selective_ssm_sequence_b200 as mod
    return mod


def _inputs(seed, n, D, io, layer=True, mean=0.5):
    rnd = wl.round_bf16 if io == "bf16" else wl.round_f32
    c = {k: rnd(np.asarray(wl.normal(seed, k, (n, D))) + (mean if k in ("y", "r", "r_out") else 0.0)) for k in ROWS}
    for k in ("scale", "post_w", "post_b", "pre_w", "pre_b"):
        c[k] = wl.round_f32(np.asarray(wl.normal(seed, k, (D,))) * 0.3 + (1.0 if k.endswith("w") else 0.2))
    if not layer:
        c["post_b"] = c["pre_b"] = None
    return c


def _dev(a, io, pad=0):
    import torch
    if a is None:
        return None
    t = dev_tensor(a, io)
    if not pad or t.dim() == 1:
        return t
    big = torch.full((a.shape[0], a.shape[1] + 2 * pad), float("nan"), dtype=t.dtype, device="cuda")
    big[:, pad:pad + a.shape[1]] = t
    return big[:, pad:pad + a.shape[1]]


def _near(got, want, mag, half, what):
    err, tol = np.abs(got - want), half * np.abs(want) + DELTA * mag * (1 + half) + 1e-37
    assert not (err > tol).any(), "%s: %d of %d off, worst %.3g of its tolerance" % (
        what, (err > tol).sum(), err.size, (err / tol).max())


def _abs_norm(u, mag, w, b, layer, eps):
    """Sum of absolute terms of norm(u) w + b, for an input with magnitude `mag`."""
    mean = np.abs(u).mean(-1, keepdims=True) if layer else 0.0
    c = u - u.mean(-1, keepdims=True) if layer else u
    rstd = 1 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    # the statistics' own error: the row's mean square of `mag` against that of the row
    grow = 1 + np.sqrt((mag * mag).mean(-1, keepdims=True)) * rstd
    return (mag + mean) * rstd * grow * np.abs(1.0 if w is None else w) + np.abs(0.0 if b is None else b)


def _fwd_mag(c, layer, post, gated, eps, alpha):
    m = np.abs(c["y"])
    if post:
        m = _abs_norm(c["y"], m, c["post_w"], c["post_b"], layer, eps)
    if gated:
        m = m * np.abs(c["gate"])
    m = np.abs(c["r"]) + abs(alpha) * np.abs(c["scale"]) * m
    r_out, _ = around.norm_gate(c["y"], c["r"], c["gate"] if gated else None, layer, post, eps, alpha, c["scale"],
                                c["post_w"], c["post_b"])
    return m, _abs_norm(r_out, m, c["pre_w"], c["pre_b"], layer, eps)


def _kw(c, layer, post, eps, alpha):
    return dict(layer=layer, post=post, eps=eps, alpha=alpha, scale=c["scale"], post_w=c["post_w"],
                post_b=c["post_b"], pre_w=c["pre_w"])


def _gpu_kw(hm, c, layer, post, eps, alpha):
    return dict(norm=hm.HM_NORM_LAYER if layer else hm.HM_NORM_RMS, post=post, eps=eps, alpha=alpha,
                **{k: _dev(c[k], "f32") for k in ("scale", "post_w", "post_b", "pre_w")})


def _forward(hm, c, io, layer, post, gated, eps=1e-5, alpha=0.7, pad=0):
    n, D = c["y"].shape
    r_out, xn = _dev(np.full((n, D), 7.0), io, pad), _dev(np.full((n, D), 7.0), io, pad)
    hm.hm_norm_gate_fwd(hm.norm_gate_args(
        _dev(c["y"], io, pad), _dev(c["r"], io, pad), r_out, xn, gate=_dev(c["gate"], io, pad) if gated else None,
        pre_b=_dev(c["pre_b"], "f32"), **_gpu_kw(hm, c, layer, post, eps, alpha)))
    want = around.norm_gate(c["y"], c["r"], c["gate"] if gated else None, pre_b=c["pre_b"],
                            **_kw(c, layer, post, eps, alpha))
    for got, w, m, k in zip((r_out, xn), want, _fwd_mag(c, layer, post, gated, eps, alpha), ("r_out", "xn")):
        _near(to_np(got), w, m, HALF[io], k)


def _backward(hm, c, io, layer, post, gated, eps=1e-5, alpha=0.7, pad=0, has=("dr_out", "dxn")):
    import torch
    n, D = c["y"].shape
    dy, dr, dgate = (_dev(np.full((n, D), 7.0), io, pad) for _ in range(3))
    d = {k: torch.full((D,), float("nan"), device="cuda") for k in ("dscale", "dpost_w", "dpost_b", "dpre_w", "dpre_b")}
    gate = _dev(c["gate"], io, pad) if gated else None
    b = hm.norm_gate_bwd_args(_dev(c["y"], io, pad), _dev(c["r_out"], io, pad) if "dxn" in has else None,
                              *(_dev(c[k], io, pad) if k in has else None for k in ("dr_out", "dxn")), dy, dr,
                              gate=gate, dgate=dgate if gated else None, **d,
                              **_gpu_kw(hm, c, layer, post, eps, alpha))
    ws = hm.alloc_workspace(hm.hm_norm_gate_bwd_workspace_size(b))
    ws.fill_(255)
    b.workspace, b.workspace_bytes = ws.data_ptr(), ws.numel()
    hm.hm_norm_gate_bwd(b)
    args = (c["y"], c["r_out"], c["dr_out"] if "dr_out" in has else None, c["dxn"] if "dxn" in has else None,
            c["gate"] if gated else None)
    want = around.norm_gate_bwd(*args, **_kw(c, layer, post, eps, alpha))
    # magnitudes: the chain with absolute values
    A = np.abs
    dr_m = A(c["dr_out"]) if "dr_out" in has else np.zeros((n, D))
    mag = {"dpre_w": np.zeros(D), "dpre_b": np.zeros(D)}

    def back(dm, w, u, um, rstd):
        dm = dm * A(w)
        return (dm + um * (dm * um).mean(-1, keepdims=True) + dm.mean(-1, keepdims=True)) * rstd

    def unit(u):
        _, v, rstd = around._norm(u, None, None, layer, eps)
        return v, _abs_norm(u, A(u), None, None, layer, eps), rstd
    if "dxn" in has:
        v, vm, rstd = unit(c["r_out"])
        mag["dpre_w"], mag["dpre_b"] = (A(c["dxn"]) * vm).sum(0), A(c["dxn"]).sum(0)
        dr_m = dr_m + back(A(c["dxn"]), c["pre_w"], v, vm, rstd)
    um, rstd = A(c["y"]), 1.0
    vm = um
    if post:
        u, um, rstd = unit(c["y"])
        vm = um * A(c["post_w"]) + (0.0 if c["post_b"] is None else A(c["post_b"]))
    dm = alpha * A(c["scale"]) * dr_m
    g = A(c["gate"]) if gated else 1.0
    mm, dn = vm * g, dm * g
    mag["dgate"] = dm * vm * (1 + g)
    mag["dscale"] = alpha * (dr_m * mm).sum(0)
    mag["dpost_w"], mag["dpost_b"] = (dn * um).sum(0), dn.sum(0)
    mag["dy"] = back(dn, c["post_w"], None, um, rstd) if post else dn
    mag["dr"] = dr_m
    for k, t in (("dy", dy), ("dr", dr)) + ((("dgate", dgate),) if gated else ()):
        _near(to_np(t), want[k], mag[k], HALF[io], k)
    for k, t in d.items():
        if post or not k.startswith("dpost"):
            _near(to_np(t), want[k], mag[k], 2.0 ** -24, k)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("n,D", [(1, 1), (3, 8), (2, 37), (5, 256), (4, 1000), (3, 1001), (300, 64), (7, 2048),
                                 (2, 4100), (2, 8192), (2, 16384)])
def test_parity(hm, io, layer, n, D):
    c = _inputs(31, n, D, io, layer)
    _forward(hm, c, io, layer, True, True)
    _backward(hm, c, io, layer, True, True)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("layer,post,gated", [(a, b, g) for a in (False, True) for b in (False, True)
                                              for g in (False, True)])
def test_variants(hm, io, layer, post, gated):
    c = _inputs(32, 9, 520, io, layer)
    _forward(hm, c, io, layer, post, gated)
    _backward(hm, c, io, layer, post, gated)
    _backward(hm, c, io, layer, post, gated, has=("dxn",))
    _backward(hm, c, io, layer, post, gated, has=("dr_out",))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D,pad", [(256, 8), (256, 1), (75, 5)])
def test_strided_rows(hm, io, D, pad):
    c = _inputs(33, 11, D, io)
    _forward(hm, c, io, True, True, True, pad=pad)
    _backward(hm, c, io, True, True, True, pad=pad)


def test_many_rows(hm):
    """More rows than blocks of the backward: every thread's running sums take several rows."""
    c = _inputs(34, 3001, 128, "bf16")
    _forward(hm, c, "bf16", False, True, True)
    _backward(hm, c, "bf16", False, True, True)
    _backward(hm, _inputs(35, 1000, 24, "f32"), "f32", True, True, True)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n,D", [(33, 8), (17, 64), (13, 72), (9, 128), (2500, 16)])
def test_narrow_rows(hm, io, n, D):
    """Rows that share a warp, in numbers that leave its last teams without one."""
    c = _inputs(37, n, D, io, True)
    _forward(hm, c, io, True, True, True)
    _backward(hm, c, io, True, True, True)
    _backward(hm, c, io, False, True, False)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("n,D", [(1, 264), (700, 264), (601, 1000), (1203, 2048), (299, 2056), (450, 4096), (200, 4104),
                                 (151, 8192)])
def test_backward_rows_at_a_time(hm, io, layer, n, D):
    """Odd numbers of rows, threads without columns, several steps of a block."""
    _backward(hm, _inputs(38, n, D, io, layer), io, layer, True, True)


def test_far_from_zero_mean(hm):
    """A mean many times the spread: the variance comes from centred values."""
    c = _inputs(36, 6, 512, "f32", mean=300.0)
    _forward(hm, c, "f32", True, True, False)


def test_edges(hm):
    """Rows of zeros, a row with an infinity and one with NaN among ordinary ones, large gates;
    parameters, residual and outputs left out."""
    import torch
    c = _inputs(37, 6, 264, "f32")
    c["y"][1], c["r"][1] = 0.0, 0.0
    c["gate"][2], c["gate"][3] = 200.0, -200.0
    _forward(hm, c, "f32", False, True, True)
    y, r = c["y"].copy(), c["r"].copy()
    y[0, 5], y[4, 7] = np.inf, np.nan
    args = [_dev(v, "f32") for v in (y, r)] + [torch.empty(6, 264, device="cuda") for _ in range(2)]
    hm.hm_norm_gate_fwd(hm.norm_gate_args(*args, gate=_dev(c["gate"], "f32")))
    want, _ = around.norm_gate(c["y"], c["r"], c["gate"])
    rows = [1, 2, 3, 5]
    assert np.allclose(to_np(args[2])[rows], want[rows], rtol=1e-5, atol=1e-5)
    assert np.isnan(to_np(args[2])[4]).all() and np.isnan(to_np(args[3])[4]).all()
    # no residual, no parameters, one output at a time
    for out in (0, 1):
        o = torch.full((6, 264), 7.0, device="cuda")
        hm.hm_norm_gate_fwd(hm.norm_gate_args(_dev(c["y"], "f32"), None, o if out == 0 else None,
                                              o if out == 1 else None, norm=hm.HM_NORM_LAYER))
        want = around.norm_gate(c["y"], None, layer=True)[out]
        assert np.allclose(to_np(o), want, rtol=1e-5, atol=1e-5)
    e = torch.zeros(0, 8, device="cuda")
    hm.hm_norm_gate_fwd(hm.norm_gate_args(e, e, e, torch.zeros_like(e)))
    d = torch.full((8,), 3.0, device="cuda")
    b = hm.norm_gate_bwd_args(e, e, e, e, torch.zeros_like(e), None, dpre_w=d)
    hm.hm_norm_gate_bwd(b)
    assert not d.any()


def test_in_place(hm):
    """r_out over r, xn over y; dr over dr_out, dy over y, dgate over gate: the same bits."""
    import torch
    c = _inputs(38, 40, 1024, "bf16")
    y, r, gate, r_out, dr_out, dxn = (_dev(c[k], "bf16") for k in ROWS)
    kw = _gpu_kw(hm, c, True, True, 1e-5, 0.7)
    o, x = torch.empty_like(y), torch.empty_like(y)
    hm.hm_norm_gate_fwd(hm.norm_gate_args(y, r, o, x, gate=gate, **kw))
    y2, r2 = y.clone(), r.clone()
    hm.hm_norm_gate_fwd(hm.norm_gate_args(y2, r2, r2, y2, gate=gate, **kw))
    assert torch.equal(r2, o) and torch.equal(y2, x)
    outs = [torch.empty_like(y) for _ in range(3)]

    def back(y, gate, dr_out, dy, dr, dgate):
        b = hm.norm_gate_bwd_args(y, r_out, dr_out, dxn, dy, dr, gate=gate, dgate=dgate, **kw)
        ws = hm.alloc_workspace(hm.hm_norm_gate_bwd_workspace_size(b))
        b.workspace, b.workspace_bytes = ws.data_ptr(), ws.numel()
        hm.hm_norm_gate_bwd(b)
        torch.cuda.synchronize()
    back(y, gate, dr_out, *outs)
    yc, gc, dc = y.clone(), gate.clone(), dr_out.clone()
    back(yc, gc, dc, yc, dc, gc)
    assert all(torch.equal(a, b) for a, b in zip(outs, (yc, dc, gc)))


def test_gradient_against_differences(hm):
    import torch
    c = _inputs(39, 4, 48, "f32")
    kw = _kw(c, True, True, 1e-5, 0.7)
    c["r_out"] = wl.round_f32(around.norm_gate(c["y"], c["r"], c["gate"], pre_b=c["pre_b"], **kw)[0])
    dy, dr, dgate = (torch.empty(4, 48, device="cuda") for _ in range(3))
    dw = torch.empty(48, device="cuda")
    b = hm.norm_gate_bwd_args(*(_dev(c[k], "f32") for k in ("y", "r_out", "dr_out", "dxn")), dy, dr,
                              gate=_dev(c["gate"], "f32"), dgate=dgate, dpost_w=dw,
                              **_gpu_kw(hm, c, True, True, 1e-5, 0.7))
    ws = hm.alloc_workspace(hm.hm_norm_gate_bwd_workspace_size(b))
    b.workspace, b.workspace_bytes = ws.data_ptr(), ws.numel()
    hm.hm_norm_gate_bwd(b)
    r = np.random.default_rng(1)
    for name, got in (("y", dy), ("r", dr), ("gate", dgate), ("post_w", dw)):
        d = r.normal(size=c[name].shape)

        def loss(e):
            v = dict(c, **{name: c[name] + e * d})
            o, x = around.norm_gate(v["y"], v["r"], v["gate"], pre_b=v["pre_b"], **_kw(v, True, True, 1e-5, 0.7))
            return (c["dr_out"] * o).sum() + (c["dxn"] * x).sum()
        q = (loss(1e-5) - loss(-1e-5)) / 2e-5
        # fp32 gradients: 2^-18 of magnitudes some ten times their own
        assert abs((to_np(got) * d).sum() - q) < 1e-4 * np.abs(to_np(got) * d).sum(), name


def test_captured(hm):
    """A captured forward and backward replayed on new data give the eager call's bits."""
    import torch
    c = _inputs(40, 600, 512, "bf16")
    kw = _gpu_kw(hm, c, False, True, 1e-5, 0.7)
    src = {k: _dev(c[k], "bf16") for k in ROWS}
    buf = {k: torch.zeros_like(v) for k, v in src.items()}

    def calls(s):
        out = [torch.zeros_like(s["y"]) for _ in range(5)]
        d = torch.zeros(512, device="cuda")
        f = hm.norm_gate_args(s["y"], s["r"], out[0], out[1], gate=s["gate"], **kw)
        b = hm.norm_gate_bwd_args(s["y"], s["r_out"], s["dr_out"], s["dxn"], out[2], out[3], gate=s["gate"],
                                  dgate=out[4], dscale=d, **kw)
        ws = hm.alloc_workspace(hm.hm_norm_gate_bwd_workspace_size(b))
        b.workspace, b.workspace_bytes = ws.data_ptr(), ws.numel()
        return out + [d], f, b, ws
    want, f, b, _keep = calls(src)
    hm.hm_norm_gate_fwd(f)
    hm.hm_norm_gate_bwd(b)
    got, f, b, _keep2 = calls(buf)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hm.hm_norm_gate_fwd(f)
        hm.hm_norm_gate_bwd(b)
    for k, v in src.items():
        buf[k].copy_(v)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("io,n,D", [("bf16", 37, 64), ("f32", 9, 128), ("bf16", 301, 2048), ("bf16", 150, 6000),
                                    ("f32", 7, 8192)])
def test_backward_in_place(hm, io, n, D):
    """dy over y, dgate over gate, dr over dxn: the same bits, in each form of the backward."""
    import torch
    c = _inputs(39, n, D, io)
    y, r, gate, r_out, dr_out, dxn = (_dev(c[k], io) for k in ROWS)
    kw = _gpu_kw(hm, c, True, True, 1e-5, 0.7)

    def back(y, gate, dxn, dy, dr, dgate):
        b = hm.norm_gate_bwd_args(y, r_out, dr_out, dxn, dy, dr, gate=gate, dgate=dgate, **kw)
        ws = hm.alloc_workspace(hm.hm_norm_gate_bwd_workspace_size(b))
        b.workspace, b.workspace_bytes = ws.data_ptr(), ws.numel()
        hm.hm_norm_gate_bwd(b)
        torch.cuda.synchronize()
    outs = [torch.empty_like(y) for _ in range(3)]
    back(y, gate, dxn, *outs)
    yc, gc, dc = y.clone(), gate.clone(), dxn.clone()
    back(yc, gc, dc, yc, dc, gc)
    assert all(torch.equal(a, b) for a, b in zip(outs, (yc, dc, gc)))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("n,D,pad", [(5, 2, 0), (77, 34, 0), (30, 130, 0), (2600, 170, 0), (41, 254, 0), (9, 302, 0),
                                     (700, 1002, 0), (3, 2050, 2), (6, 4094, 0), (4, 8190, 0), (50, 256, 2)])
def test_rows_of_pairs(hm, io, layer, n, D, pad):
    """Even widths and offsets that are no multiples of 16 bytes."""
    c = _inputs(40, n, D, io, layer)
    _forward(hm, c, io, layer, True, True, pad=pad)
    _backward(hm, c, io, layer, True, True, pad=pad)
    _backward(hm, c, io, layer, False, False, pad=pad)
