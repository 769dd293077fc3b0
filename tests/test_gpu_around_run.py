"""The operators around the mixer run together, as a hybrid stack uses them: rotary positions on
the queries and keys, the mixer's scan, the seam to the next block, the channel-wise recurrence,
the next seam; prefill then single tokens; and a training step through recurrence and seam.

Each stage is checked against its fp64 definition on the inputs it was really given (the stored
results of the stage before), at that stage's own tolerance."""
import numpy as np
import pytest

import oracle
import workloads as wl
from gpu_common import TOL_BF16, dev_tensor, rel_err, to_np
from oracle import around

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hm():
    import torch
    assert torch.cuda.is_available()
    import selective_ssm_sequence_b200 as mod
    return mod


def _bf(seed, name, shape, std=1.0):
    return wl.round_bf16(np.asarray(wl.normal(seed, name, shape)) * std)


def _f32(seed, name, shape, std=1.0, mean=0.0):
    return wl.round_f32(np.asarray(wl.normal(seed, name, shape)) * std + mean)


def test_hybrid_stack_prefill_and_decode(hm):
    import torch
    B, L, H, d, p = 2, 192, 2, 256, 128
    E, T = H * d, 3                                     # T tokens decoded after the prefill
    dev = lambda a, io="bf16": dev_tensor(a, io)        # noqa: E731
    q, k, v, gate, res = (_bf(51, n, (B, L, E)) for n in ("q", "k", "v", "gate", "res"))
    W_q, W_k = _bf(51, "Wq", (p, d), d ** -0.5), _bf(51, "Wk", (p, d), d ** -0.5)
    dth, A_h = _f32(51, "dth", (B, L, H)), _f32(51, "Ah", (H,), 0.5)
    dtc, A_c = _bf(51, "dtc", (B, L + T, E)), _f32(51, "Ac", (E,), 0.5)
    bias, w1, w2, sc = (_f32(51, n, (E,), 0.1, m) for n, m in (("bias", -3), ("w1", 1), ("w2", 1), ("sc", 0.7)))

    tq, tk = dev(q).view(B, L, H, d), dev(k).view(B, L, H, d)
    rq, rk = torch.empty_like(tq), torch.empty_like(tk)
    rot = dict(rot=64, base=10000.0)
    hm.hm_rotary(hm.rotary_args(tq, tk, rq, rk, **rot))
    for got, x in ((rq, tq), (rk, tk)):
        want = around.rotary(to_np(x), np.arange(L)[None], **rot)
        assert np.all(np.abs(to_np(got) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19)

    tv = dev(v).view(B, L, H, d)
    o = torch.empty_like(tv)
    a = hm.scan_args(rq, rk, tv, o, W_q=dev(W_q), W_k=dev(W_k), dt=dev(dth, "f32"), A_log=dev(A_h, "f32"))
    ws = hm.alloc_workspace(hm.hm_scan_workspace_size(a))
    a.workspace, a.workspace_bytes = ws.data_ptr(), ws.numel()
    hm.hm_scan_chunked_fwd(a)
    want = oracle.scan_fwd(to_np(rq), to_np(rk), v.reshape(B, L, H, d), W_q, W_k, dt=dth, A_log=A_h)
    assert rel_err(to_np(o), want) <= TOL_BF16

    # post-norm, gate, residual, next pre-norm
    r1, x1 = torch.empty(B, L, E, dtype=torch.bfloat16, device="cuda"), torch.empty(B, L, E, dtype=torch.bfloat16, device="cuda")
    f = lambda z: dev(z, "f32")                         # noqa: E731
    seam = dict(post_w=f(w1), pre_w=f(w2), scale=f(sc), alpha=0.5)
    hm.hm_norm_gate_fwd(hm.norm_gate_args(o.view(B, L, E), dev(res), r1, x1, gate=dev(gate), **seam))
    ref = lambda y, r, g: around.norm_gate(to_np(y).reshape(-1, E), to_np(r).reshape(-1, E), g.reshape(-1, E),      # noqa: E731
                                           post_w=w1, pre_w=w2, scale=sc, alpha=0.5)
    for got, w in zip((r1, x1), ref(o, dev(res), gate)):
        assert rel_err(to_np(got).reshape(-1, E), w) <= 2.0 ** -8 + 2.0 ** -14

    # the channel-wise recurrence over the prefill, then token by token on its state
    y1, h = torch.empty_like(x1), torch.empty(B, E, device="cuda")
    tdt, tA, tb = dev(dtc), f(A_c), f(bias)
    hm.hm_gated_scan_fwd(hm.gated_scan_args(x1, tdt[:, :L], y1, tA, dt_bias=tb, h_out=h, input_scale=hm.HM_INPUT_UNIT))
    wy, wh, _ = around.gated_scan(to_np(x1), dtc[:, :L], A_c, bias, scale=around.UNIT)
    assert rel_err(to_np(y1), wy) <= 2.0 ** -8 + 2.0 ** -14 and rel_err(to_np(h), wh) <= 2.0 ** -14
    xt = dev(_bf(52, "xt", (B, T, E)))
    yt, rt, nt = (torch.empty(B, E, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    for t in range(T):
        hm.hm_gated_scan_step(hm.gated_step_args(xt[:, t], tdt[:, L + t], yt, h, h, tA, dt_bias=tb,
                                                 input_scale=hm.HM_INPUT_UNIT))
        wy, wh, _ = around.gated_scan(to_np(xt[:, t:t + 1]), dtc[:, L + t:L + t + 1], A_c, bias, h0=wh,
                                      scale=around.UNIT)
        assert rel_err(to_np(yt), wy[:, 0]) <= 2.0 ** -8 + 2.0 ** -14
        hm.hm_norm_gate_fwd(hm.norm_gate_args(yt, xt[:, t], rt, nt, **seam))
        want = around.norm_gate(to_np(yt), to_np(xt[:, t]), post_w=w1, pre_w=w2, scale=sc, alpha=0.5)
        for got, w in zip((rt, nt), want):
            assert rel_err(to_np(got), w) <= 2.0 ** -8 + 2.0 ** -14
    assert hm.hm_get_device_error() == hm.HM_OK


def test_training_step_through_recurrence_and_seam(hm):
    """x -> recurrence -> seam, and its gradients chained by hand, in fp32: along a direction
    against the difference quotient of the fp64 composition.  fp32 gradients of magnitudes some
    ten times their own (2^-18 each) and a quotient good to 1e-9: 1e-4 of the absolute sum."""
    import torch
    B, L, D = 2, 150, 96
    c = {n: _f32(53, n, (B, L, D)) for n in ("x", "dt", "gate", "res", "dr", "dxn")}
    pr = {n: _f32(53, n, (D,), 0.2, m) for n, m in (("A_log", 0), ("bias", -2), ("w1", 1), ("b1", 0), ("w2", 1), ("sc", 1))}
    t = {n: dev_tensor(a, "f32") for n, a in {**c, **pr}.items()}
    n = lambda *s: torch.empty(*s, device="cuda")       # noqa: E731
    y, h = n(B, L, D), n(B, D)
    a = hm.gated_scan_args(t["x"], t["dt"], y, t["A_log"], dt_bias=t["bias"], h_out=h, input_scale=hm.HM_INPUT_UNIT)
    st = hm.alloc_workspace(hm.hm_gated_scan_states_size(a))
    a.states, a.states_bytes = st.data_ptr(), st.numel()
    hm.hm_gated_scan_fwd(a)
    kw = dict(norm=hm.HM_NORM_LAYER, alpha=0.8, scale=t["sc"], post_w=t["w1"], post_b=t["b1"], pre_w=t["w2"])
    r, xn = n(B, L, D), n(B, L, D)
    hm.hm_norm_gate_fwd(hm.norm_gate_args(y, t["res"], r, xn, gate=t["gate"], **kw))
    dy, dr, dg, dw1, dsc = n(B, L, D), n(B, L, D), n(B, L, D), n(D), n(D)
    b = hm.norm_gate_bwd_args(y, r, t["dr"], t["dxn"], dy, dr, gate=t["gate"], dgate=dg, dpost_w=dw1, dscale=dsc, **kw)
    ws = hm.alloc_workspace(hm.hm_norm_gate_bwd_workspace_size(b))
    b.workspace, b.workspace_bytes = ws.data_ptr(), ws.numel()
    hm.hm_norm_gate_bwd(b)
    dx, ddt, dA, db = n(B, L, D), n(B, L, D), n(D), n(D)
    g = hm.gated_scan_bwd_args(t["x"], t["dt"], dy, dx, ddt, t["A_log"], dA, st, dt_bias=t["bias"], d_dt_bias=db,
                               input_scale=hm.HM_INPUT_UNIT)
    ws2 = hm.alloc_workspace(hm.hm_gated_scan_bwd_workspace_size(g))
    g.workspace, g.workspace_bytes = ws2.data_ptr(), ws2.numel()
    hm.hm_gated_scan_bwd(g)

    def loss(**over):
        v = {**c, **pr, **over}
        yy, _, _ = around.gated_scan(v["x"], v["dt"], v["A_log"], v["bias"], scale=around.UNIT)
        ro, xo = around.norm_gate(yy, v["res"], v["gate"], layer=True, alpha=0.8, scale=v["sc"], post_w=v["w1"],
                                  post_b=v["b1"], pre_w=v["w2"])
        return (v["dr"] * ro).sum() + (v["dxn"] * xo).sum()

    rng = np.random.default_rng(7)
    for name, got in (("x", dx), ("dt", ddt), ("A_log", dA), ("bias", db), ("gate", dg), ("res", dr), ("w1", dw1),
                      ("sc", dsc)):
        base = {**c, **pr}[name].astype(np.float64)
        d = rng.normal(size=base.shape)
        quot = (loss(**{name: base + 1e-5 * d}) - loss(**{name: base - 1e-5 * d})) / 2e-5
        have = to_np(got) * d
        assert abs(have.sum() - quot) < 1e-4 * np.abs(have).sum(), name
