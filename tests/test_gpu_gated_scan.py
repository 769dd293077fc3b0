"""The channel-wise gated recurrence on the GPU against its fp64 definition.

Tolerances: an io-typed result is rounded once (half a step, eps / 2 of the
value) on top of fp32 arithmetic.  Every exponent and input factor is formed with
a relative error of a few 2^-22 (z = dt + bias is rounded; the polynomial of
log(1 + e), exp2 and sqrt are good to 2^-21.5 and better): 2^-19 covers them
together.  A relative error delta of an exponent la is one of |la| delta of the
decay e^la, so a decay counts 1 + |la| times; the magnitudes that the definition
returns carry this through the recurrence and its adjoint.  Sums
a rounded z shifts Delta by |z| 2^-24 of itself at most (d log softplus / dz = sigmoid(z) /
softplus(z) <= 1), so beyond |z| = 32 that share, |z|_max 2^-24, is added to 2^-19.  A step
below the normal fp32 range, Delta < 2^-126, may be taken as zero; with HM_INPUT_UNIT its
sqrt(2 Delta e^A_log) reaches 2^-62.5 e^(A_log / 2), which is the absolute floor.  A
decay below 2^-126 may be taken as zero, which shifts what it multiplies (the state or
an adjoint, and in the gradients the rate and log a) by 2^-126 of that.  Sums
over tokens add less than 2^-19 of their absolute sum (fp32 partial sums of at
most a few thousand terms, relative 2^-24 each in a chain of at most 2^5 per level)."""
import numpy as np
import pytest

import workloads as wl
from gpu_common import dev_tensor, to_np
from oracle import around

pytestmark = pytest.mark.gpu

DELTA = 2.0 ** -19
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module")
def hm():
    import torch
    assert torch.cuda.is_available()
    import selective_ssm_sequence_b200 as mod
    return mod


def _near(got, want, mag, half, what, delta=DELTA, floor=0.0):
    err = np.abs(got - want)
    tol = half * np.abs(want) + delta * mag * (1 + half) + 1e-37 + floor
    bad = err > tol
    assert not bad.any(), "%s: %d off, worst %.3g of its tolerance at %s" % (
        what, bad.sum(), (err / tol).max(), np.unravel_index((err / tol).argmax(), err.shape))


def _inputs(seed, B, L, D, io, start=True, wide=False):
    """Seeded inputs as stored; `wide`: step sizes and rates from far to either side."""
    rnd = (wl.round_bf16 if io == "bf16" else wl.round_f32)
    n = lambda name, shape: np.asarray(wl.normal(seed, name, shape), np.float64)     # noqa: E731
    x, dt, dy = (rnd(n(k, (B, L, D))) for k in ("x", "dt", "dy"))
    if wide:
        dt = rnd(dt * 12.0)
    A_log = wl.round_f32(n("A", (D,)) * (3.0 if wide else 1.0))
    return dict(x=x, dt=dt, dy=dy, A_log=A_log, dt_bias=wl.round_f32(n("bias", (D,)) - 3.0),
                h0=wl.round_f32(n("h0", (B, D))) if start else None, dh_out=wl.round_f32(n("dh", (B, D))))


def _rows(a, io, pad):
    """Device copy of [B, L, D]; with `pad`, a slice of wider rows that start `pad` elements in."""
    import torch
    t = dev_tensor(a, io)
    if not pad:
        return t
    big = torch.full((*a.shape[:2], a.shape[2] + 2 * pad), float("nan"), dtype=t.dtype, device="cuda")
    big[..., pad:pad + a.shape[2]] = t
    return big[..., pad:pad + a.shape[2]]


def _run(hm, c, io, scale, lengths=None, pad=0, backward=True, alias_state=False):
    """Forward and backward through the C ABI; outputs prefilled with 7 to see what is written."""
    import torch
    B, L, D = c["x"].shape
    x, dt = _rows(c["x"], io, pad), _rows(c["dt"], io, pad)
    y = _rows(np.full((B, L, D), 7.0), io, pad)
    f32 = lambda v: None if v is None else dev_tensor(v, "f32")     # noqa: E731
    A, bias, h0 = f32(c["A_log"]), f32(c["dt_bias"]), f32(c["h0"])
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    h_out = h0 if alias_state else torch.full((B, D), float("nan"), device="cuda")
    a = hm.gated_scan_args(x, dt, y, A, dt_bias=bias, h0=h0, h_out=h_out, lengths=ln, input_scale=scale)
    nan = torch.full((hm.hm_gated_scan_states_size(a) // 4 + 1,), float("nan"), device="cuda")
    a.states, a.states_bytes = nan.data_ptr(), nan.numel() * 4
    hm.hm_gated_scan_fwd(a)
    out = {"y": y, "h_out": h_out}
    if backward:
        dy = _rows(c["dy"], io, pad)
        dx, ddt = _rows(np.full((B, L, D), 7.0), io, pad), _rows(np.full((B, L, D), 7.0), io, pad)
        g = {k: torch.full(s, float("nan"), device="cuda") for k, s in (("dA_log", (D,)), ("d_dt_bias", (D,)),
                                                                        ("dh0", (B, D)))}
        b = hm.gated_scan_bwd_args(x, dt, dy, dx, ddt, A, g["dA_log"], nan, dt_bias=bias,
                                   d_dt_bias=g["d_dt_bias"], dh_out=f32(c["dh_out"]), dh0=g["dh0"], lengths=ln,
                                   input_scale=scale)
        ws = hm.alloc_workspace(hm.hm_gated_scan_bwd_workspace_size(b))
        ws.fill_(255)
        b.workspace, b.workspace_bytes = ws.data_ptr(), ws.numel()
        hm.hm_gated_scan_bwd(b)
        out |= {"dx": dx, "ddt": ddt} | g
    torch.cuda.synchronize()
    assert hm.hm_get_device_error() == hm.HM_OK
    if pad:     # nothing beside the rows
        for k in ("y", "dx", "ddt"):
            if k in out:
                whole = out[k]._base if out[k]._base is not None else out[k]
                side = torch.cat([whole[..., :pad], whole[..., -pad:]], -1)
                assert bool(torch.isnan(side).all()), k
    return {k: to_np(v) for k, v in out.items()}


def _check(hm, c, io, scale, lengths=None, pad=0, backward=True):
    half = HALF[io]
    got = _run(hm, c, io, scale, lengths, pad, backward)
    kw = dict(dt_bias=c["dt_bias"], h0=c["h0"], lengths=lengths, scale=scale)
    y, h, mag = around.gated_scan(c["x"], c["dt"], c["A_log"], **kw)
    B, L, _ = c["x"].shape
    z = np.abs(c["dt"] + c["dt_bias"]).max() if L else 0.0
    delta = DELTA + (z * 2.0 ** -24 if z > 32 else 0.0)
    tiny = 2.0 ** -62.5 * np.exp(c["A_log"].max() / 2) if scale == around.UNIT and z > 87 else 0.0    # e^-87.3 = 2^-126
    on = np.ones((B, L), bool) if lengths is None else np.arange(L)[None] < np.clip(lengths, 0, L)[:, None]
    for k in ("y", "dx", "ddt"):
        if k in got:
            assert np.all(got[k][~on] == 7.0), "rows of %s behind a sequence's end were written" % k
            got[k] = np.where(on[..., None], got[k], 0.0)
    # the largest state, rate and log a of the case, for the decays flushed to zero
    flush = 2.0 ** -126 * (1 + mag.max()) * (1 + np.exp(c["A_log"].max())) * (1 + z * np.exp(c["A_log"].max())) if L else 0.0
    _near(got["y"], y, mag, half, "y", delta, tiny * np.abs(c["x"]).sum(1).max() + flush)
    last = mag.max(1) if L else np.zeros_like(h)      # a bound of the last magnitude, padded batches too
    _near(got["h_out"], h, last + np.abs(h), 2.0 ** -24, "h_out", delta, tiny * np.abs(c["x"]).sum(1).max() + flush if L else 0.0)
    if backward:
        want = around.gated_scan_bwd(c["x"], c["dt"], c["dy"], c["A_log"], dh_out=c["dh_out"], **kw)
        # every adjoint is at most the sum of what enters it
        grad = (np.abs(c["dy"]).sum(1).max() + np.abs(c["dh_out"]).max()) * (1 + np.abs(c["x"]).max()) if L else 0.0
        for k, (v, m) in want.items():
            _near(got[k], v, m, half if k in ("dx", "ddt") else 2.0 ** -24, k, delta,
                  (tiny + flush) * grad * (B * L if k in ("dA_log", "d_dt_bias") else 1))
    return got


SCALES = [around.PLAIN, around.STEP, around.UNIT]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("B,L,D", [(1, 1, 1), (2, 3, 5), (1, 63, 64), (3, 64, 96), (2, 65, 130), (1, 257, 40),
                                   (2, 1000, 8), (1, 2049, 24)])
def test_parity(hm, io, scale, B, L, D):
    _check(hm, _inputs(11, B, L, D, io, start=L % 2 == 0), io, scale)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("scale", SCALES)
def test_wide_gates(hm, io, scale):
    """Gates far to either side: decays of 0 and of 1, steps of 0, memories of thousands of tokens."""
    c = _inputs(12, 2, 700, 32, io, wide=True)
    c["dt"][:, 5], c["dt"][:, 6], c["dt"][:, 7] = -200.0, 200.0, 0.0
    c["dt"][0, 100:300, 0] = -120.0         # nothing decays, and with the scaled inputs nothing enters
    _check(hm, c, io, scale)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[0, 5, 300, 299], [300, 0, 0, 1], [64, 65, 128, 127], [-3, 400, 256, 257]])
def test_padded_batches(hm, io, lengths):
    c = _inputs(13, 4, 300, 72, io)
    for b, n in enumerate(lengths):         # what stands behind an end must not matter, NaN and infinities too
        c["x"][b, max(0, n):], c["dt"][b, max(0, n):], c["dy"][b, max(0, n):] = np.nan, np.inf, np.nan
    got = _run(hm, c, io, around.UNIT, lengths)
    for b, n in enumerate(lengths):
        n = max(0, n)
        for k in ("x", "dt", "dy"):
            c[k][b, n:] = 0.0
    got2 = _check(hm, c, io, around.UNIT, lengths)
    on = np.arange(300)[None] < np.clip(lengths, 0, 300)[:, None]
    for k in got:
        assert np.array_equal(got[k][on] if got[k].ndim == 3 else got[k],
                              got2[k][on] if got2[k].ndim == 3 else got2[k]), k


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D,pad", [(64, 8), (64, 1), (37, 3), (128, 64)])
def test_strided_rows(hm, io, D, pad):
    _check(hm, _inputs(14, 2, 150, D, io), io, around.STEP, pad=pad)


def test_long_and_wide(hm):
    """Many chunks, and more channels than one block of threads: the shapes that split over blocks."""
    _check(hm, _inputs(15, 1, 5000, 200, "bf16"), "bf16", around.UNIT)
    _check(hm, _inputs(16, 3, 130, 2056, "bf16"), "bf16", around.STEP, lengths=[130, 17, 128])
    _check(hm, _inputs(17, 40, 33, 260, "f32"), "f32", around.PLAIN)


@pytest.mark.parametrize("io,scale,D,pad", [("bf16", 2, 64, 0), ("f32", 1, 72, 0), ("bf16", 1, 33, 0),
                                            ("bf16", 0, 34, 2)])
def test_few_channels_of_a_long_sequence(hm, io, scale, D, pad):
    """Clusters of 16, and the backward in two passes; sequences that end early, one of them at once."""
    _check(hm, _inputs(24, 3, 8300, D, io), io, scale, lengths=[8300, 0, 8193], pad=pad)


def test_no_tokens(hm):
    """L = 0 hands the state on and gives zero parameter gradients; B = 0 does nothing."""
    import torch
    c = _inputs(18, 2, 0, 16, "f32")
    got = _run(hm, c, "f32", around.STEP)
    assert np.array_equal(got["h_out"], c["h0"]) and np.array_equal(got["dh0"], c["dh_out"])
    assert not got["dA_log"].any() and not got["d_dt_bias"].any()
    x = torch.zeros(0, 4, 16, device="cuda")
    A = torch.zeros(16, device="cuda")
    hm.hm_gated_scan_fwd(hm.gated_scan_args(x, x, x, A))
    dA = torch.full((16,), 3.0, device="cuda")
    b = hm.gated_scan_bwd_args(x, x, x, torch.zeros_like(x), torch.zeros_like(x), A, dA, None)
    hm.hm_gated_scan_bwd(b)
    assert not dA.any()


def test_state_in_place_and_carried(hm):
    """h_out over h0, and a sequence cut in two equals the whole; state alone without y."""
    import torch
    c = _inputs(19, 2, 200, 64, "f32")
    whole = _run(hm, c, "f32", around.UNIT, backward=False)
    again = _run(hm, c, "f32", around.UNIT, backward=False, alias_state=True)
    assert np.array_equal(whole["h_out"], again["h_out"]) and np.array_equal(whole["y"], again["y"])
    x, dt, A, bias, h = (dev_tensor(c[k], "f32") for k in ("x", "dt", "A_log", "dt_bias", "h0"))
    y = torch.empty_like(x)
    for s in (slice(0, 70), slice(70, 200)):
        hm.hm_gated_scan_fwd(hm.gated_scan_args(x[:, s], dt[:, s], y[:, s], A, dt_bias=bias, h0=h, h_out=h,
                                                input_scale=around.UNIT))
    h2 = torch.zeros_like(h)
    hm.hm_gated_scan_fwd(hm.gated_scan_args(x, dt, None, A, dt_bias=bias, h0=dev_tensor(c["h0"], "f32"), h_out=h2,
                                            input_scale=around.UNIT))
    want, hw, mag = around.gated_scan(c["x"], c["dt"], c["A_log"], c["dt_bias"], c["h0"], scale=around.UNIT)
    _near(to_np(y), want, mag, 2.0 ** -24, "y of the two pieces")
    assert np.array_equal(to_np(h2), whole["h_out"])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("B,D,pad", [(1, 1, 0), (3, 64, 0), (5, 1001, 0), (2, 96, 4), (64, 2048, 0), (7, 33, 1)])
def test_step(hm, io, scale, B, D, pad):
    import torch
    c = _inputs(20, 1, B, D, io)
    h0 = wl.round_f32(np.asarray(wl.normal(21, "h", (B, D))))
    x, dt = _rows(c["x"], io, pad)[0], _rows(c["dt"], io, pad)[0]
    y, A, bias, h = torch.full_like(x, 7.0), dev_tensor(c["A_log"], "f32"), dev_tensor(c["dt_bias"], "f32"), \
        dev_tensor(h0, "f32")
    h2 = torch.zeros_like(h)
    hm.hm_gated_scan_step(hm.gated_step_args(x, dt, y, h, h2, A, dt_bias=bias, input_scale=scale))
    hm.hm_gated_scan_step(hm.gated_step_args(x, dt, torch.empty_like(y), h, h, A, dt_bias=bias, input_scale=scale))
    assert torch.equal(h, h2)
    want, hw, mag = around.gated_scan(c["x"][0][:, None], c["dt"][0][:, None], c["A_log"], c["dt_bias"], h0, None,
                                      scale)
    _near(to_np(y), want[:, 0], mag[:, 0], HALF[io], "y")
    _near(to_np(h2), hw, mag[:, 0], 2.0 ** -24, "h_out")


def test_steps_continue_a_sequence(hm):
    import torch
    c = _inputs(22, 2, 40, 48, "bf16")
    x, dt, A, bias, h = (dev_tensor(c[k], "bf16" if c[k].ndim == 3 else "f32")
                         for k in ("x", "dt", "A_log", "dt_bias", "h0"))
    y = torch.empty_like(x)
    hm.hm_gated_scan_fwd(hm.gated_scan_args(x[:, :30], dt[:, :30], y[:, :30], A, dt_bias=bias, h0=h, h_out=h))
    for t in range(30, 40):
        hm.hm_gated_scan_step(hm.gated_step_args(x[:, t], dt[:, t], y[:, t], h, h, A, dt_bias=bias))
    want, hw, mag = around.gated_scan(c["x"], c["dt"], c["A_log"], c["dt_bias"], c["h0"])
    _near(to_np(y), want, mag, HALF["bf16"], "y")
    _near(to_np(h), hw, mag[:, -1], 2.0 ** -24, "h")


def test_gradient_against_differences(hm):
    """The GPU's gradient along a direction against the fp64 definition's difference quotient."""
    c = _inputs(23, 2, 90, 16, "f32")
    got = _run(hm, c, "f32", around.UNIT)
    kw = dict(dt_bias=c["dt_bias"], h0=c["h0"], scale=around.UNIT)
    r = np.random.default_rng(0)
    for name, g in (("x", "dx"), ("dt", "ddt"), ("A_log", "dA_log")):
        d = r.normal(size=c[name].shape)

        def loss(e):
            v = dict(c, **{name: c[name] + e * d})
            y, h, _ = around.gated_scan(v["x"], v["dt"], v["A_log"], **kw)
            return (c["dy"] * y).sum() + (c["dh_out"] * h).sum()
        q = (loss(1e-5) - loss(-1e-5)) / 2e-5
        # fp32 gradients (2^-19 of magnitudes a few times their own) and the quotient's 1e-10 of its curvature
        assert abs((got[g] * d).sum() - q) < 1e-4 * np.abs(got[g] * d).sum()


def test_same_bits_on_streams_and_in_a_graph(hm):
    """Two calls give the same bits; so does a captured call replayed on new data, on a side stream."""
    import torch
    c = _inputs(24, 2, 700, 128, "bf16")
    one, two = _run(hm, c, "bf16", around.STEP), _run(hm, c, "bf16", around.STEP)
    for k in one:
        assert np.array_equal(one[k], two[k]), k
    x, dt, dy = (dev_tensor(c[k], "bf16") for k in ("x", "dt", "dy"))
    A, bias, h0, dh = (dev_tensor(c[k], "f32") for k in ("A_log", "dt_bias", "h0", "dh_out"))
    bufs = [torch.zeros_like(x) for _ in range(3)]
    y, dx, ddt = bufs
    h_out, dh0 = torch.zeros_like(h0), torch.zeros_like(h0)
    dA, db = torch.zeros_like(A), torch.zeros_like(A)
    sx, sdt, sdy = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    a = hm.gated_scan_args(sx, sdt, y, A, dt_bias=bias, h0=h0, h_out=h_out, input_scale=around.STEP)
    st = hm.alloc_workspace(hm.hm_gated_scan_states_size(a))
    a.states, a.states_bytes = st.data_ptr(), st.numel()
    b = hm.gated_scan_bwd_args(sx, sdt, sdy, dx, ddt, A, dA, st, dt_bias=bias, d_dt_bias=db, dh_out=dh, dh0=dh0,
                               input_scale=around.STEP)
    ws = hm.alloc_workspace(hm.hm_gated_scan_bwd_workspace_size(b))
    b.workspace, b.workspace_bytes = ws.data_ptr(), ws.numel()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        hm.hm_gated_scan_fwd(a)
        hm.hm_gated_scan_bwd(b)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            hm.hm_gated_scan_fwd(a)
            hm.hm_gated_scan_bwd(b)
    for s, v in ((sx, x), (sdt, dt), (sdy, dy)):
        s.copy_(v)
    graph.replay()
    torch.cuda.synchronize()
    for k, t in (("y", y), ("h_out", h_out), ("dx", dx), ("ddt", ddt), ("dA_log", dA), ("d_dt_bias", db),
                 ("dh0", dh0)):
        assert np.array_equal(to_np(t), one[k]), k


@pytest.mark.parametrize("B,L,D", [(1, 5000, 64), (40, 90, 128), (1, 9000, 130), (2, 0, 24)])
def test_states_in_place(hm, B, L, D):
    """h_out over h0 and dh0 over dh_out with one block a sequence, clusters and two passes."""
    import torch
    c = _inputs(25, B, L, D, "bf16")
    x, dt, dy = (dev_tensor(c[k], "bf16") for k in ("x", "dt", "dy"))
    A, bias, h0, dh = (dev_tensor(c[k], "f32") for k in ("A_log", "dt_bias", "h0", "dh_out"))
    got = []
    for place in (False, True):
        h, g = h0.clone(), dh.clone()
        ho, go = (h, g) if place else (torch.zeros_like(h), torch.zeros_like(g))
        y, dx, ddt, dA = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(A)
        a = hm.gated_scan_args(x, dt, y, A, dt_bias=bias, h0=h, h_out=ho, input_scale=around.STEP)
        st = hm.alloc_workspace(hm.hm_gated_scan_states_size(a))
        a.states, a.states_bytes = st.data_ptr(), st.numel()
        hm.hm_gated_scan_fwd(a)
        b = hm.gated_scan_bwd_args(x, dt, dy, dx, ddt, A, dA, st, dt_bias=bias, dh_out=g, dh0=go,
                                   input_scale=around.STEP)
        ws = hm.alloc_workspace(hm.hm_gated_scan_bwd_workspace_size(b))
        b.workspace, b.workspace_bytes = ws.data_ptr(), ws.numel()
        hm.hm_gated_scan_bwd(b)
        got.append((y, ho, dx, ddt, dA, go))
    for u, v in zip(*got):
        assert torch.equal(u, v)


def test_two_passes_captured(hm):
    """A long sequence of few channels, its backward captured and replayed on new data."""
    import torch
    c = _inputs(26, 1, 8500, 40, "bf16")
    one = _run(hm, c, "bf16", around.UNIT)
    x, dt, dy = (dev_tensor(c[k], "bf16") for k in ("x", "dt", "dy"))
    A, bias, h0, dh = (dev_tensor(c[k], "f32") for k in ("A_log", "dt_bias", "h0", "dh_out"))
    s = [torch.zeros_like(x) for _ in range(3)]
    y, dx, ddt, dh0, dA = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(dh), \
        torch.zeros_like(A)
    a = hm.gated_scan_args(s[0], s[1], y, A, dt_bias=bias, h0=h0, input_scale=around.UNIT)
    st = hm.alloc_workspace(hm.hm_gated_scan_states_size(a))
    a.states, a.states_bytes = st.data_ptr(), st.numel()
    b = hm.gated_scan_bwd_args(s[0], s[1], s[2], dx, ddt, A, dA, st, dt_bias=bias, dh_out=dh, dh0=dh0,
                               input_scale=around.UNIT)
    ws = hm.alloc_workspace(hm.hm_gated_scan_bwd_workspace_size(b))
    b.workspace, b.workspace_bytes = ws.data_ptr(), ws.numel()
    hm.hm_gated_scan_fwd(a)
    hm.hm_gated_scan_bwd(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hm.hm_gated_scan_fwd(a)
        hm.hm_gated_scan_bwd(b)
    for t, v in zip(s, (x, dt, dy)):
        t.copy_(v)
    graph.replay()
    torch.cuda.synchronize()
    for k, t in (("y", y), ("dx", dx), ("ddt", ddt), ("dA_log", dA), ("dh0", dh0)):
        assert np.array_equal(to_np(t), one[k]), k
