"""Rotary positions on the GPU against the fp64 definition.

Tolerance: one rounding to the io type (eps / 2 of the value); the sine and
cosine are within 2^-22 (a turn's fraction rounded to 2^-26, times 2 pi, and
their own last bits) and the products and sum round to 2^-24 each, so
mscale (|u| + |v|) 2^-21 covers the rest."""
import numpy as np
import pytest

import workloads as wl
from gpu_common import dev_tensor, to_np
from oracle import around

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module")
def hm():
    import torch
    assert torch.cuda.is_available()
    import selective_ssm_sequence_b200 as mod
    return mod


def _rand(seed, name, shape, io):
    return (wl.round_bf16 if io == "bf16" else wl.round_f32)(np.asarray(wl.normal(seed, name, shape)))


def _check(got, x, pos, io, what, far=1.0, **kw):
    """`far` positions add |pos| theta 2^-48 to the angle: below 2^-22 up to 2^26."""
    want = around.rotary(x, pos, **kw)
    rot = kw.get("rot") or x.shape[-1]
    mag = np.zeros_like(x)
    inter = kw.get("interleaved")
    u, v = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    mag[..., u] = mag[..., v] = (np.abs(x[..., u]) + np.abs(x[..., v])) * abs(kw.get("mscale", 1.0))
    err, tol = np.abs(got - want), HALF[io] * np.abs(want) + mag * far * 2.0 ** -21
    assert not (err > tol).any(), "%s: %d off, worst %.3g of its tolerance" % (
        what, (err > tol).sum(), (err[tol > 0] / tol[tol > 0]).max())
    if rot < x.shape[-1]:
        assert np.array_equal(got[..., rot:], x[..., rot:]), what


def _names(hm, interleaved=False, scaling="none", rot=0, **kw):
    s = {"none": hm.HM_ROTARY_PLAIN, "linear": hm.HM_ROTARY_LINEAR, "ntk": hm.HM_ROTARY_NTK,
         "by_parts": hm.HM_ROTARY_BY_PARTS}[scaling]
    return dict(kw, rot=rot, scaling=s, layout=hm.HM_ROTARY_INTERLEAVED if interleaved else hm.HM_ROTARY_HALF)


def _run(hm, io, B, L, Hq, Hk, d, positions=None, pos0=0, **kw):
    import torch
    q, k = _rand(41, "q", (B, L, Hq, d), io), _rand(41, "k", (B, L, Hk, d), io)
    tq, tk = dev_tensor(q, io), dev_tensor(k, io)
    oq, ok = torch.full_like(tq, 7.0), torch.full_like(tk, 7.0)
    tp = None if positions is None else torch.tensor(positions, dtype=torch.int64, device="cuda")
    hm.hm_rotary(hm.rotary_args(tq, tk, oq, ok, positions=tp, pos0=pos0, **_names(hm, **kw)))
    pos = np.asarray(positions) if positions is not None else pos0 + np.arange(L)[None]
    for got, x, n in ((oq, q, "q"), (ok, k, "k")):
        _check(to_np(got), x, pos, io, n, **kw)
    # in place
    hm.hm_rotary(hm.rotary_args(tq, tk, tq, tk, positions=tp, pos0=pos0, **_names(hm, **kw)))
    assert torch.equal(tq, oq) and torch.equal(tk, ok)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(2, 2), (6, 4), (64, 64), (64, 16), (80, 32), (96, 24), (256, 64), (256, 256),
                                   (50, 50), (1024, 1024), (128, 126)])
def test_parity(hm, io, interleaved, d, rot):
    _run(hm, io, 2, 5, 3, 1, d, rot=rot, interleaved=interleaved)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "by_parts"])
@pytest.mark.parametrize("transpose", [False, True])
def test_scalings_and_transpose(hm, io, scaling, transpose):
    kw = dict(scaling=scaling, factor=8.0, orig_len=512.0, mscale=1.2) if scaling != "none" else {}
    _run(hm, io, 1, 300, 2, 2, 128, transpose=transpose, **kw)
    _run(hm, io, 1, 33, 5, 1, 96, rot=48, interleaved=True, transpose=transpose, pos0=100000, **kw)


@pytest.mark.parametrize("Hq,Hk,B,L", [(1, 1, 1, 1), (8, 2, 3, 1), (9, 0, 2, 7), (0, 3, 2, 2), (32, 4, 1, 70), (5, 5, 1, 3)])
def test_heads(hm, Hq, Hk, B, L):
    _run(hm, "bf16", B, L, Hq, Hk, 64, rot=32)


def test_positions(hm):
    """Own positions of every token, negative and far ones; shared along either axis."""
    r = np.random.default_rng(3)
    _run(hm, "f32", 3, 9, 2, 1, 64, positions=r.integers(-(1 << 20), 1 << 20, (3, 9)))
    _run(hm, "f32", 3, 9, 2, 1, 64, positions=r.integers(0, 1 << 26, (3, 1)))
    _run(hm, "f32", 3, 9, 2, 1, 64, positions=np.arange(9)[None] * 7)
    _run(hm, "f32", 1, 4, 1, 1, 32, pos0=(1 << 26) - 2)


def test_far_positions_keep_their_angle(hm):
    """Positions behind 2^32 turn the fastest pair (theta = 1) by pos mod 2 pi: against the
    residue computed in integers with 2 pi to 200 bits.  The angle's error, pos 2^-48 / 2 pi of
    a turn, grows with the position."""
    import torch
    two_pi = 0x6487ED5110B4611A62633145C06E0E68948127044533E63A0105DF531D89CD91   # floor(2 pi 2^252)
    x = np.array([1.0, 0.0]).reshape(1, 1, 1, 2)
    for pos in ((1 << 32) + 1, (1 << 36) + 12345, -(1 << 34) - 5):
        ang = ((pos << 252) % two_pi) / 2.0 ** 252
        t = dev_tensor(x, "f32")
        hm.hm_rotary(hm.rotary_args(t, None, t, None, positions=torch.tensor([[pos]], device="cuda")))
        tol = abs(pos) * 2.0 ** -48 + 2.0 ** -21
        assert np.allclose(to_np(t).ravel(), [np.cos(ang), np.sin(ang)], rtol=0, atol=tol), pos


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("off", [0, 1, 8])
def test_strides(hm, io, interleaved, off):
    """q and k as slices of one projection [B, L, (Hq + 2 Hk) d + off]; outputs head-major."""
    import torch
    B, L, Hq, Hk, d = 2, 11, 4, 2, 32
    z = dev_tensor(_rand(42, "z", (B, L, (Hq + 2 * Hk) * d + off), io), io)
    q = z[..., off:off + Hq * d].unflatten(-1, (Hq, d))
    k = z[..., off + Hq * d:off + (Hq + Hk) * d].unflatten(-1, (Hk, d))
    oq = torch.full((B, Hq, L, d), 7.0, dtype=z.dtype, device="cuda").transpose(1, 2)
    ok = torch.full((B, Hk, L, d), 7.0, dtype=z.dtype, device="cuda").transpose(1, 2)
    before = z.clone()
    hm.hm_rotary(hm.rotary_args(q, k, oq, ok, **_names(hm, rot=16, interleaved=interleaved)))
    assert torch.equal(z, before)
    for got, x in ((oq, q), (ok, k)):
        _check(to_np(got), to_np(x), np.arange(L)[None], io, "strided", rot=16, interleaved=interleaved)
    # in place: the rest of the projection stays
    hm.hm_rotary(hm.rotary_args(q, k, q, k, **_names(hm, rot=16, interleaved=interleaved)))
    assert torch.equal(q, oq) and torch.equal(k, ok)
    assert torch.equal(z[..., :off], before[..., :off])
    assert torch.equal(z[..., off + (Hq + Hk) * d:], before[..., off + (Hq + Hk) * d:])


def test_empty_and_captured(hm):
    import torch
    e = torch.zeros(0, 3, 2, 8, device="cuda")
    hm.hm_rotary(hm.rotary_args(e, e, e, e))
    q, k = (dev_tensor(_rand(43, n, (2, 50, 4, 64), "bf16"), "bf16") for n in "qk")
    want = [torch.empty_like(q), torch.empty_like(k)]
    hm.hm_rotary(hm.rotary_args(q, k, *want, pos0=9))
    sq, sk, oq, ok = (torch.zeros_like(q) for _ in range(4))
    a = hm.rotary_args(sq, sk, oq, ok, pos0=9)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hm.hm_rotary(a)
    sq.copy_(q)
    sk.copy_(k)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(oq, want[0]) and torch.equal(ok, want[1])


def test_gradient_is_the_transpose(hm):
    """<R q, g> = <q, R^T g>, and differences of the definition along a direction."""
    import torch
    kw = dict(scaling="by_parts", factor=8.0, orig_len=512.0, mscale=1.2, rot=32)
    q, g = _rand(44, "q", (1, 40, 2, 64), "f32"), _rand(44, "g", (1, 40, 2, 64), "f32")
    tg = dev_tensor(g, "f32")
    hm.hm_rotary(hm.rotary_args(tg, None, tg, None, transpose=True, **_names(hm, **kw)))
    pos = np.arange(40)[None]
    q_dot = (around.rotary(q + 0.5 * g, pos, **kw) - around.rotary(q - 0.5 * g, pos, **kw))
    # linear in q, so the quotient along g is exact; 2^-21 mscale (|u| + |v|) per element against
    # g sums to at most 2^-21 mscale 2 sum g^2, doubled for the fp32 rounding of the results
    assert abs((q_dot * g).sum() - (to_np(tg) * g).sum()) < 2.0 ** -20 * 1.2 * 2 * (g * g).sum()
