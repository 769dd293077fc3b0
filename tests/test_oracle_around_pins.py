"""Pins of the fp64 definitions in oracle/around.py, on the CPU: closed forms,
invariances and, for the gradients, central differences of the forward."""
import numpy as np
import pytest

from oracle import around

rng = np.random.default_rng


def _scan_case(seed, B=2, L=7, D=3):
    r = rng(seed)
    return dict(x=r.normal(size=(B, L, D)), dt=r.normal(size=(B, L, D)), A_log=r.uniform(-1, 1, D),
                dt_bias=r.normal(size=D), h0=r.normal(size=(B, D)))


def test_gates_closed_forms():
    # exp(-softplus(z)) = sigmoid(-z): at A_log = 0 the decay is that sigmoid
    z = np.linspace(-30, 30, 41)
    _, _, _, a, _ = around.gates(z, np.zeros(1))
    assert np.allclose(a, 1 / (1 + np.exp(z)), rtol=1e-12)
    _, _, _, a, beta = around.gates(z, np.zeros(1), scale=around.UNIT)
    assert np.allclose(a * a + beta * beta, 1.0, rtol=1e-14)


@pytest.mark.parametrize("scale", [around.PLAIN, around.STEP, around.UNIT])
def test_scan_equals_its_sum_form_and_splits(scale):
    c = _scan_case(1)
    y, h, mag = around.gated_scan(scale=scale, **c)
    _, _, la, _, beta = around.gates(c["dt"], c["A_log"], c["dt_bias"], scale)
    cum = np.cumsum(la, 1)
    for t in range(7):
        want = np.exp(cum[:, t]) * c["h0"] + sum(np.exp(cum[:, t] - cum[:, j]) * beta[:, j] * c["x"][:, j]
                                                 for j in range(t + 1))
        assert np.allclose(y[:, t], want, rtol=1e-12)
    assert np.all(mag >= np.abs(y)) and np.array_equal(h, y[:, -1])
    cut = dict(c, x=c["x"][:, :3], dt=c["dt"][:, :3])
    _, hm, _ = around.gated_scan(scale=scale, **cut)
    y2, h2, _ = around.gated_scan(scale=scale, **dict(c, x=c["x"][:, 3:], dt=c["dt"][:, 3:], h0=hm))
    assert np.allclose(y2, y[:, 3:], rtol=1e-13) and np.allclose(h2, h, rtol=1e-13)


def test_unit_input_keeps_the_variance():
    r = rng(2)
    x = r.normal(size=(1, 400, 2000))
    y, _, _ = around.gated_scan(x, np.zeros_like(x), np.full(2000, -2.0), h0=r.normal(size=(1, 2000)),
                                scale=around.UNIT)
    # variance of a mean of 2000 squared normals: 2 / 2000, six standard deviations
    assert np.all(np.abs((y ** 2).mean(-1) - 1) < 6 * np.sqrt(2 / 2000))


def test_lengths_cut_the_sequence():
    c = _scan_case(3, B=3)
    y, h, _ = around.gated_scan(lengths=[0, 4, 99], **c)
    assert np.array_equal(h[0], c["h0"][0]) and not y[0].any() and not y[1, 4:].any()
    one = {k: (v[1:2, :4] if v.ndim == 3 else v) for k, v in c.items() if k != "h0"}
    y1, h1, _ = around.gated_scan(h0=c["h0"][1:2], **one)
    assert np.allclose(y[1, :4], y1[0]) and np.allclose(h[1], h1[0])


def _diff(f, v, d, eps=1e-5):
    """Central difference of f along direction d."""
    return (f(v + eps * d) - f(v - eps * d)) / (2 * eps)


@pytest.mark.parametrize("scale", [around.PLAIN, around.STEP, around.UNIT])
@pytest.mark.parametrize("lengths", [None, [3, 7]])
def test_scan_gradients_against_differences(scale, lengths):
    c = _scan_case(4)
    r = rng(5)
    dy, dh = r.normal(size=c["x"].shape), r.normal(size=c["h0"].shape)

    def loss(**kw):
        y, h, _ = around.gated_scan(scale=scale, lengths=lengths, **dict(c, **kw))
        return (dy * y).sum() + (dh * h).sum()

    g = around.gated_scan_bwd(dy=dy, dh_out=dh, scale=scale, lengths=lengths, **c)
    for name, grad in (("x", "dx"), ("dt", "ddt"), ("A_log", "dA_log"), ("dt_bias", "d_dt_bias"), ("h0", "dh0")):
        for _ in range(3):
            d = r.normal(size=c[name].shape)
            # error of a central difference: eps^2 times a third derivative of order one
            assert np.isclose((g[grad][0] * d).sum(), _diff(lambda v: loss(**{name: v}), c[name], d), rtol=1e-6,
                              atol=1e-7)
        assert np.all(g[grad][1] >= np.abs(g[grad][0]) * (1 - 1e-12))


def _seam_case(seed, n=3, D=10):
    r = rng(seed)
    return (dict(y=r.normal(size=(n, D)), r=r.normal(size=(n, D)), gate=r.normal(size=(n, D)),
                 scale=r.normal(size=D), post_w=r.normal(size=D), post_b=r.normal(size=D), pre_w=r.normal(size=D),
                 pre_b=r.normal(size=D)), r)


def test_norms_closed_forms():
    c, _ = _seam_case(6)
    r_out, xn = around.norm_gate(c["y"], None, layer=True, eps=1e-12)
    assert np.allclose(r_out.mean(-1), 0, atol=1e-12) and np.allclose(r_out.var(-1), 1)
    assert np.allclose(xn, r_out)           # the norm of a normalised row is itself
    r_out, _ = around.norm_gate(c["y"], None, eps=1e-12)
    assert np.allclose((r_out ** 2).mean(-1), 1)
    # scaling the branch's output leaves its norm; a gate of zero leaves the residual
    a = around.norm_gate(eps=1e-15, **c)
    b = around.norm_gate(eps=1e-15, **dict(c, y=7 * c["y"]))
    assert np.allclose(a, b)
    assert np.array_equal(around.norm_gate(**dict(c, gate=np.zeros_like(c["gate"])))[0], c["r"])


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_seam_gradients_against_differences(layer, post, gated):
    c, r = _seam_case(7)
    c = dict(c, gate=c["gate"] if gated else None)
    kw = dict(layer=layer, post=post, eps=1e-5, alpha=0.6)
    d0, d1 = r.normal(size=c["y"].shape), r.normal(size=c["y"].shape)

    def loss(**over):
        a, b = around.norm_gate(**kw, **dict(c, **over))
        return (d0 * a).sum() + (d1 * b).sum()

    r_out, _ = around.norm_gate(**kw, **c)
    g = around.norm_gate_bwd(c["y"], r_out, d0, d1, gate=c["gate"], scale=c["scale"], post_w=c["post_w"],
                             post_b=c["post_b"], pre_w=c["pre_w"], **kw)
    names = ["y", "r", "scale", "pre_w", "pre_b"] + ["gate"] * gated + ["post_w", "post_b"] * post
    for name in names:
        d = r.normal(size=c[name].shape)
        assert np.isclose((g["d" + name] * d).sum(), _diff(lambda v: loss(**{name: v}), c[name], d), rtol=1e-6,
                          atol=1e-7), name


def test_rotary_closed_forms():
    r = rng(8)
    x = r.normal(size=(2, 5, 3, 8))
    pos = np.arange(5)[None]
    y = around.rotary(x, pos)
    assert np.allclose(y[:, 0], x[:, 0])
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    # the turn undone by its transpose; composition of positions; the product of two turned
    # vectors goes by the difference of their positions
    assert np.allclose(around.rotary(y, pos, transpose=True), x)
    assert np.allclose(around.rotary(y, 3 + 0 * pos), around.rotary(x, pos + 3))
    k = r.normal(size=x.shape)
    p = (around.rotary(x, pos + 9) * around.rotary(k, pos + 2)).sum(-1)
    assert np.allclose(p, (around.rotary(x, pos + 7) * around.rotary(k, pos)).sum(-1))
    # interleaved is the half layout with its elements in another order
    order = np.arange(8).reshape(2, 4).T.ravel()
    assert np.allclose(around.rotary(x[..., order], pos, interleaved=True), y[..., order])
    # part of the head: the rest unchanged, the first part a smaller head's
    z = around.rotary(x, pos, rot=4)
    assert np.array_equal(z[..., 4:], x[..., 4:])
    assert np.allclose(z[..., :4], around.rotary(x[..., :4], pos))
    # a quarter turn of a single pair
    q = around.rotary(np.array([1.0, 0.0]).reshape(1, 1, 1, 2), np.array([[1]]), mscale=2.0)
    assert np.allclose(q.ravel(), [2 * np.cos(1), 2 * np.sin(1)])


def test_rotary_scalings():
    th = around.rotary_theta(64)
    assert np.allclose(around.rotary_theta(64, scaling="linear", factor=4.0), th / 4)
    ntk = around.rotary_theta(64, scaling="ntk", factor=4.0)
    assert np.isclose(ntk[0], th[0]) and np.isclose(ntk[-1], th[-1] / 4)    # fastest kept, slowest divided
    bp = around.rotary_theta(64, scaling="by_parts", factor=4.0, orig_len=4096)
    turns = 4096 * th / (2 * np.pi)
    assert np.allclose(bp[turns >= 32], th[turns >= 32]) and np.allclose(bp[turns <= 1], th[turns <= 1] / 4)
    mid = (turns < 32) & (turns > 1)
    assert mid.any() and np.all((bp[mid] < th[mid]) & (bp[mid] > th[mid] / 4))
