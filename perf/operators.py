"""The operators around the mixer that are timed, each in two forms.

Three families, as a decoder stack built on this package uses them:

* the channel-wise gated recurrence, ``h_t = a_t h_{t-1} + beta_t x_t`` with
  ``a_t = exp(-softplus(dt_t + bias) exp(A_log))`` per channel: a whole
  sequence forward, a training step (forward and backward), one token;
* the seam between two blocks: post-norm, gate, scaled residual, next block's
  pre-norm, forward and backward;
* rotary positions on queries and keys, forward and transposed (its backward).

With ``own`` false ``run`` computes them with elementary torch operations in
32 bits; with ``own`` true it calls the package.
"""
import math

import torch

own = False

SCALES = {"plain": 0, "step": 1, "unit": 2}
BF16, F32 = "bf16", "f32"


# --------------------------------------------------------------------- cases

def listed():
    return [
        # one recurrent layer of the mixer's batch: 8 sequences of 4096, width 2048
        {"name": "recur_fwd_b8_l4096", "kind": "recur_fwd", "B": 8, "L": 4096, "D": 2048, "dtype": BF16,
         "scale": "step", "strided": False, "ragged": False, "start": False},
        # prefill of one long document: little parallelism besides the channels and time itself
        {"name": "recur_fwd_l32768", "kind": "recur_fwd", "B": 1, "L": 32768, "D": 2048, "dtype": BF16,
         "scale": "unit", "strided": False, "ragged": False, "start": True},
        # a padded batch in fp32 with an odd width (rows off every vector boundary), x and dt
        # halves of one projection, one sequence of it empty
        {"name": "recur_fwd_ragged_f32", "kind": "recur_fwd", "B": 5, "L": 1531, "D": 1001, "dtype": F32,
         "scale": "plain", "strided": True, "ragged": True, "start": True},
        # training on the prefill's batch
        {"name": "recur_train_b4_l2048", "kind": "recur_train", "B": 4, "L": 2048, "D": 2048, "dtype": BF16,
         "scale": "step", "strided": False, "ragged": False, "start": False},
        # training on one long document
        {"name": "recur_train_l32768", "kind": "recur_train", "B": 1, "L": 32768, "D": 2048, "dtype": BF16,
         "scale": "unit", "strided": False, "ragged": False, "start": True},
        # serving: one token of 256 sequences
        {"name": "recur_step_256", "kind": "recur_step", "B": 256, "D": 2048, "dtype": BF16, "scale": "step"},
        # the seam between two blocks over the mixer's batch
        {"name": "norm_fwd_32768", "kind": "norm_fwd", "rows": 32768, "D": 2048, "dtype": BF16, "norm": "rms",
         "gate": True, "post": True},
        # the same seam while serving 256 sequences
        {"name": "norm_fwd_256", "kind": "norm_fwd", "rows": 256, "D": 2048, "dtype": BF16, "norm": "rms",
         "gate": True, "post": True},
        # its backward over the prefill's batch, layer norms with scale and shift
        {"name": "norm_bwd_8192", "kind": "norm_bwd", "rows": 8192, "D": 2048, "dtype": BF16, "norm": "layer",
         "gate": True, "post": True},
        # Pythia's rotary: the first quarter of each head, half layout, over the prefill's batch
        {"name": "rotary_quarter_b4_l2048", "kind": "rotary", "B": 4, "L": 2048, "Hq": 8, "Hk": 8, "d": 256, "rot": 64,
         "dtype": BF16, "layout": "half", "scaling": "none", "transpose": False, "positions": False},
        # gradients of a long document: whole head, interleaved pairs, frequencies scaled by parts
        {"name": "rotary_long_bwd_l32768", "kind": "rotary", "B": 1, "L": 32768, "Hq": 8, "Hk": 8, "d": 256, "rot": 256,
         "dtype": BF16, "layout": "interleaved", "scaling": "by_parts", "transpose": True, "positions": False},
        # serving: one token of 256 sequences, each at its own far position, with shared key heads
        {"name": "rotary_step_256", "kind": "rotary", "B": 256, "L": 1, "Hq": 8, "Hk": 2, "d": 256, "rot": 256,
         "dtype": BF16, "layout": "half", "scaling": "linear", "transpose": False, "positions": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["recur_fwd", "recur_train", "recur_step", "norm_fwd", "norm_bwd", "rotary"])
    dtype = rng.choice([BF16, BF16, F32])
    size = 2 if dtype == BF16 else 4
    if kind in ("recur_fwd", "recur_train"):
        D = _log_int(rng, 48, 4096)
        if rng.random() < 0.6:
            D = max(64, D // 64 * 64)
        most = (1 << 27) // size // D       # elements of x at most those of the longest listed case
        L = _log_int(rng, 1, min(32768, most))
        B = _log_int(rng, 1, max(1, min(32, most // L)))
        return {"kind": kind, "B": B, "L": L, "D": D, "dtype": dtype, "scale": rng.choice(sorted(SCALES)),
                "strided": rng.random() < 0.4, "ragged": rng.random() < 0.4, "start": rng.random() < 0.5}
    if kind == "recur_step":
        D = _log_int(rng, 64, 8192)
        return {"kind": kind, "B": _log_int(rng, 1, 1024), "D": D if rng.random() < 0.4 else max(64, D // 64 * 64),
                "dtype": dtype, "scale": rng.choice(sorted(SCALES))}
    if kind in ("norm_fwd", "norm_bwd"):
        D = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            D = max(64, D // 64 * 64)
        return {"kind": kind, "rows": _log_int(rng, 1, max(1, (1 << 26) // size // D)), "D": D, "dtype": dtype,
                "norm": rng.choice(["rms", "layer"]), "gate": rng.random() < 0.7, "post": rng.random() < 0.7}
    d = rng.choice([32, 64, 80, 96, 128, 192, 256])
    rot = d if rng.random() < 0.5 else max(4, d // rng.choice([2, 4]) // 2 * 2)
    Hq = rng.choice([1, 2, 4, 8, 12, 16, 32])
    Hk = rng.choice([h for h in (1, 2, 4, 8, 12, 16, 32) if Hq % h == 0])
    most = (1 << 28) // size // ((Hq + Hk) * d)
    L = _log_int(rng, 1, min(32768, most))
    return {"kind": kind, "B": _log_int(rng, 1, max(1, min(256, most // L))), "L": L, "Hq": Hq, "Hk": Hk, "d": d,
            "rot": rot, "dtype": dtype, "layout": rng.choice(["half", "interleaved"]),
            "scaling": rng.choice(["none", "linear", "ntk", "by_parts"]), "transpose": rng.random() < 0.4,
            "positions": rng.random() < 0.5}


# -------------------------------------------------------------------- inputs

class _Rand:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=self.g, device="cuda") * std).to(dtype)

    def uniform(self, lo, hi, *shape):
        return torch.rand(*shape, generator=self.g, device="cuda") * (hi - lo) + lo

    def ints(self, lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=self.g, device="cuda")


def _type(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float32


def prepare(case, seed):
    r, t, kind = _Rand(seed), _type(case), case["kind"]
    s = {"case": case}
    if kind.startswith("recur"):
        B, D = case["B"], case["D"]
        # step sizes from 1e-3 to 0.1 at dt = 0, as state-space layers are initialised
        step = torch.exp(r.uniform(math.log(1e-3), math.log(0.1), D))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["A_log"] = r.uniform(0.0, math.log(16.0), D)
        if kind == "recur_step":
            s["x"], s["dt"] = r.normal(B, D, dtype=t), r.normal(B, D, dtype=t)
            s["h"] = r.normal(B, D)
            s["y"], s["h_out"] = torch.zeros_like(s["x"]), torch.zeros_like(s["h"])
            return s
        L = case["L"]
        if case["strided"]:     # one projection's output, x and dt side by side
            xz = r.normal(B, L, 2 * D, dtype=t)
            s["x"], s["dt"] = xz[..., :D], xz[..., D:]
        else:
            s["x"], s["dt"] = r.normal(B, L, D, dtype=t), r.normal(B, L, D, dtype=t)
        s["h0"] = r.normal(B, D) if case["start"] else None
        s["lengths"] = None
        if case["ragged"]:
            n = r.ints(0, L, B)
            n[B // 2] = L
            if B > 2:
                n[0] = 0
            s["lengths"] = n.to(torch.int32)
        s["y"] = torch.zeros(B, L, D, dtype=t, device="cuda")
        s["h_out"] = torch.zeros(B, D, device="cuda")
        if kind == "recur_train":
            s["dy"], s["dh_out"] = r.normal(B, L, D, dtype=t), r.normal(B, D)
            s["dx"], s["ddt"] = torch.zeros_like(s["y"]), torch.zeros_like(s["y"])
            s["dA_log"], s["d_dt_bias"] = torch.zeros(D, device="cuda"), torch.zeros(D, device="cuda")
            s["dh0"] = torch.zeros(B, D, device="cuda")
        return s
    if kind.startswith("norm"):
        n, D = case["rows"], case["D"]
        s["y"] = r.normal(n, D, std=0.5, dtype=t)
        s["gate"] = r.normal(n, D, dtype=t) if case["gate"] else None
        layer = case["norm"] == "layer"
        for p in ("post", "pre"):
            on = p == "pre" or case["post"]
            s[p + "_w"] = 1.0 + r.normal(D, std=0.1) if on else None
            s[p + "_b"] = r.normal(D, std=0.1) if on and layer else None
        s["scale"] = 0.5 + r.normal(D, std=0.1)
        s["alpha"], s["eps"] = 0.7071, 1e-5
        new = lambda: torch.zeros_like(s["y"])                                  # noqa: E731
        if kind == "norm_fwd":
            s["r"] = r.normal(n, D, dtype=t)
            s["r_out"], s["xn"] = new(), new()
        else:       # r_out as the forward left it; gradients of both its outputs
            s["r_out"] = r.normal(n, D, std=1.2, dtype=t)
            s["dr_out"], s["dxn"] = r.normal(n, D, dtype=t), r.normal(n, D, dtype=t)
            s["dy"], s["dr"], s["dgate"] = new(), new(), new() if case["gate"] else None
            for p in ("post_w", "post_b", "pre_w", "pre_b", "scale"):
                s["d" + p] = None if s[p] is None else torch.zeros_like(s[p])
        return s
    B, L, d = case["B"], case["L"], case["d"]
    s["q"], s["k"] = r.normal(B, L, case["Hq"], d, dtype=t), r.normal(B, L, case["Hk"], d, dtype=t)
    s["q_out"], s["k_out"] = torch.zeros_like(s["q"]), torch.zeros_like(s["k"])
    s["pos"] = None
    if case["positions"]:       # sequences at places of their own in a context of up to 2^20 tokens
        s["pos"] = r.ints(0, (1 << 20) - L, B, 1) + torch.arange(L, device="cuda")
    return s


def _rope_scaling(case):
    """base, factor, orig_len, beta_slow, beta_fast, mscale of the case's scaling."""
    factor = {"none": 1.0, "linear": 4.0, "ntk": 4.0, "by_parts": 8.0}[case["scaling"]]
    return 10000.0, factor, 4096, 1.0, 32.0, 1.0 + 0.1 * math.log(factor) if case["scaling"] == "by_parts" else 1.0


# --------------------------------------------------------------- plain forms

def _scan(a, u):
    """h_t = a_t h_{t-1} + u_t along dim 1 from h = 0, by doubling: after the pass with
    shift s each entry holds the composition of the last 2 s steps (log2 L passes over the
    data; every factor is a product of decays, so nothing overflows)."""
    L, s = a.shape[1], 1
    while s < L:
        u = torch.cat([u[:, :s], u[:, s:] + a[:, s:] * u[:, :-s]], 1)
        a = torch.cat([a[:, :s], a[:, s:] * a[:, :-s]], 1)
        s *= 2
    return u


def _gates(x, dt, s, scale):
    z = dt.float() + s["dt_bias"]
    step = z.clamp(min=0) + torch.log1p(torch.exp(-z.abs()))
    la = -step * torch.exp(s["A_log"])
    a = torch.exp(la)
    beta = None if scale == "plain" else step if scale == "step" else torch.sqrt(-torch.expm1(2 * la))
    return z, step, la, a, beta


def _recur(s, case):
    x, h0, scale = s["x"].float(), s["h0"], case["scale"]
    z, step, la, a, beta = _gates(x, s["dt"], s, scale)
    L = case["L"]
    live = None
    if s["lengths"] is not None:        # steps behind a sequence's end neither decay nor add
        live = (torch.arange(L, device=x.device)[None] < s["lengths"][:, None])[..., None]
        a = torch.where(live, a, 1.0)
        x = torch.where(live, x, 0.0)
    u = x if beta is None else x * beta
    if h0 is not None:
        u = torch.cat([u[:, :1] + a[:, :1] * h0[:, None], u[:, 1:]], 1)
    h = _scan(a, u)
    y = (h if live is None else torch.where(live, h, 0.0)).to(s["x"].dtype)
    out = {"y": y, "h_out": h[:, -1].clone()}
    if case["kind"] == "recur_fwd":
        return out
    dy = s["dy"].float()
    if live is not None:
        dy = torch.where(live, dy, 0.0)
    dy = torch.cat([dy[:, :-1], dy[:, -1:] + s["dh_out"][:, None]], 1)
    # g_t = dy_t + a_{t+1} g_{t+1}
    nxt = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    g = _scan(nxt.flip(1), dy.flip(1)).flip(1)
    first = torch.zeros_like(h[:, :1]) if h0 is None else h0[:, None]
    dla = g * a * torch.cat([first, h[:, :-1]], 1)
    dstep = 0.0
    dx = g if beta is None else g * beta
    if scale == "step":
        dstep = g * x
    elif scale == "unit":
        dla = dla - torch.where(beta > 0, g * x * a * a / beta, 0.0)
    dstep = dstep - dla * torch.exp(s["A_log"])
    ddt = dstep * torch.sigmoid(z)
    dA = dla * la
    if live is not None:
        dx, ddt, dA = (torch.where(live, v, 0.0) for v in (dx, ddt, dA))
    out |= {"dx": dx.to(s["x"].dtype), "ddt": ddt.to(s["x"].dtype), "dA_log": dA.sum((0, 1)),
            "d_dt_bias": ddt.sum((0, 1)), "dh0": a[:, 0] * g[:, 0]}
    return out


def _recur_step(s, case):
    x = s["x"].float()
    _, _, _, a, beta = _gates(x, s["dt"], s, case["scale"])
    h = a * s["h"] + (x if beta is None else x * beta)
    return {"y": h.to(s["x"].dtype), "h_out": h}


def _unit_rows(v, layer, eps):
    if layer:
        v = v - v.mean(-1, keepdim=True)
    rstd = torch.rsqrt((v * v).mean(-1, keepdim=True) + eps)
    return v * rstd, rstd


def _affine(v, w, b):
    return v * w if b is None else v * w + b


def _norm_fwd(s, case):
    layer, eps = case["norm"] == "layer", s["eps"]
    n = s["y"].float()
    if s["post_w"] is not None:
        n = _affine(_unit_rows(n, layer, eps)[0], s["post_w"], s["post_b"])
    if s["gate"] is not None:
        g = s["gate"].float()
        n = n * g * torch.sigmoid(g)
    r = s["r"].float() + s["alpha"] * s["scale"] * n
    xn = _affine(_unit_rows(r, layer, eps)[0], s["pre_w"], s["pre_b"])
    return {"r_out": r.to(s["y"].dtype), "xn": xn.to(s["y"].dtype)}


def _unit_rows_grad(dw, unit, rstd, layer):
    c = dw - unit * (dw * unit).mean(-1, keepdim=True)
    if layer:
        c = c - dw.mean(-1, keepdim=True)
    return c * rstd


def _norm_bwd(s, case):
    layer, eps, t = case["norm"] == "layer", s["eps"], s["y"].dtype
    dxn = s["dxn"].float()
    unit, rstd = _unit_rows(s["r_out"].float(), layer, eps)
    out = {"dpre_w": (dxn * unit).sum(0)}
    if layer:
        out["dpre_b"] = dxn.sum(0)
    dr = s["dr_out"].float() + _unit_rows_grad(dxn * s["pre_w"], unit, rstd, layer)
    out["dr"] = dr.to(t)
    n = s["y"].float()
    if s["post_w"] is not None:
        unit, rstd = _unit_rows(n, layer, eps)
        n = _affine(unit, s["post_w"], s["post_b"])
    dm, m = dr * (s["alpha"] * s["scale"]), n
    if s["gate"] is not None:
        g = s["gate"].float()
        sg = torch.sigmoid(g)
        m = n * g * sg
        out["dgate"] = (dm * n * sg * (1 + g * (1 - sg))).to(t)
        dn = dm * g * sg
    else:
        dn = dm
    out["dscale"] = (dr * m).sum(0) * s["alpha"]
    if s["post_w"] is not None:
        out["dpost_w"] = (dn * unit).sum(0)
        if layer:
            out["dpost_b"] = dn.sum(0)
        dn = _unit_rows_grad(dn * s["post_w"], unit, rstd, layer)
    out["dy"] = dn.to(t)
    return out


def _angles(case, pos):
    """[.., rot / 2] angles in 64 bits: far positions times small frequencies."""
    base, factor, orig, slow, fast, _ = _rope_scaling(case)
    rot = case["rot"]
    i = torch.arange(rot // 2, device=pos.device, dtype=torch.float64)
    if case["scaling"] == "ntk":
        base = base * factor ** (rot / (rot - 2))
    theta = base ** (-2 * i / rot)
    if case["scaling"] == "linear":
        theta = theta / factor
    if case["scaling"] == "by_parts":
        keep = ((orig * theta / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        theta = theta * ((1 - keep) / factor + keep)
    return pos.double()[..., None] * theta


def _rotary(s, case):
    rot, m = case["rot"], _rope_scaling(case)[5]
    pos = s["pos"] if s["pos"] is not None else torch.arange(case["L"], device="cuda")[None]
    ang = _angles(case, pos)[:, :, None]
    cs, sn = (torch.cos(ang) * m).float(), (torch.sin(ang) * m).float()
    if case["transpose"]:
        sn = -sn
    out = {}
    for name in ("q", "k"):
        v = s[name].float()
        w = v[..., :rot]
        if case["layout"] == "half":
            x, y = w[..., :rot // 2], w[..., rot // 2:]
            w = torch.cat([x * cs - y * sn, x * sn + y * cs], -1)
        else:
            x, y = w[..., 0::2], w[..., 1::2]
            w = torch.stack([x * cs - y * sn, x * sn + y * cs], -1).flatten(-2)
        out[name] = torch.cat([w, v[..., rot:]], -1).to(s[name].dtype)
    return out


# ------------------------------------------------------- the package's calls

def _own_recur(s, case):
    import selective_ssm_sequence_b200 as hm
    scale = SCALES[case["scale"]]
    train = case["kind"] == "recur_train"
    a = hm.gated_scan_args(s["x"], s["dt"], s["y"], s["A_log"], dt_bias=s["dt_bias"], h0=s["h0"], h_out=s["h_out"],
                           lengths=s["lengths"], input_scale=scale)
    out = {"y": s["y"], "h_out": s["h_out"]}
    if not train:
        hm.hm_gated_scan_fwd(a)
        return out
    states = hm.alloc_workspace(hm.hm_gated_scan_states_size(a))
    a.states, a.states_bytes = states.data_ptr(), states.numel()
    hm.hm_gated_scan_fwd(a)
    b = hm.gated_scan_bwd_args(s["x"], s["dt"], s["dy"], s["dx"], s["ddt"], s["A_log"], s["dA_log"], states,
                               dt_bias=s["dt_bias"], d_dt_bias=s["d_dt_bias"], dh_out=s["dh_out"], dh0=s["dh0"],
                               lengths=s["lengths"], input_scale=scale)
    ws = hm.alloc_workspace(hm.hm_gated_scan_bwd_workspace_size(b))
    b.workspace, b.workspace_bytes = ws.data_ptr(), ws.numel()
    hm.hm_gated_scan_bwd(b)
    return out | {k: s[k] for k in ("dx", "ddt", "dA_log", "d_dt_bias", "dh0")}


def _own_step(s, case):
    import selective_ssm_sequence_b200 as hm
    hm.hm_gated_scan_step(hm.gated_step_args(s["x"], s["dt"], s["y"], s["h"], s["h_out"], s["A_log"],
                                             dt_bias=s["dt_bias"], input_scale=SCALES[case["scale"]]))
    return {"y": s["y"], "h_out": s["h_out"]}


def _own_norm(s, case):
    import selective_ssm_sequence_b200 as hm
    norm = hm.HM_NORM_LAYER if case["norm"] == "layer" else hm.HM_NORM_RMS
    common = dict(norm=norm, post=case["post"], eps=s["eps"], alpha=s["alpha"], gate=s["gate"], scale=s["scale"],
                  post_w=s["post_w"], post_b=s["post_b"], pre_w=s["pre_w"])
    if case["kind"] == "norm_fwd":
        hm.hm_norm_gate_fwd(hm.norm_gate_args(s["y"], s["r"], s["r_out"], s["xn"], pre_b=s["pre_b"], **common))
        return {"r_out": s["r_out"], "xn": s["xn"]}
    a = hm.norm_gate_bwd_args(s["y"], s["r_out"], s["dr_out"], s["dxn"], s["dy"], s["dr"], dgate=s["dgate"],
                              dscale=s["dscale"], dpost_w=s["dpost_w"], dpost_b=s["dpost_b"], dpre_w=s["dpre_w"],
                              dpre_b=s["dpre_b"], **common)
    ws = hm.alloc_workspace(hm.hm_norm_gate_bwd_workspace_size(a))
    a.workspace, a.workspace_bytes = ws.data_ptr(), ws.numel()
    hm.hm_norm_gate_bwd(a)
    return {k: s[k] for k in ("dpre_w", "dpre_b", "dr", "dgate", "dscale", "dpost_w", "dpost_b", "dy")
            if s[k] is not None}


def _own_rotary(s, case):
    import selective_ssm_sequence_b200 as hm
    base, factor, orig, slow, fast, m = _rope_scaling(case)
    hm.hm_rotary(hm.rotary_args(
        s["q"], s["k"], s["q_out"], s["k_out"], rot=case["rot"], base=base, positions=s["pos"],
        layout=hm.HM_ROTARY_HALF if case["layout"] == "half" else hm.HM_ROTARY_INTERLEAVED,
        scaling={"none": hm.HM_ROTARY_PLAIN, "linear": hm.HM_ROTARY_LINEAR, "ntk": hm.HM_ROTARY_NTK,
                 "by_parts": hm.HM_ROTARY_BY_PARTS}[case["scaling"]],
        factor=factor, orig_len=orig, beta_slow=slow, beta_fast=fast, mscale=m, transpose=case["transpose"]))
    return {"q": s["q_out"], "k": s["k_out"]}


def run(s):
    case = s["case"]
    kind = case["kind"]
    if kind in ("recur_fwd", "recur_train"):
        return _own_recur(s, case) if own else _recur(s, case)
    if kind == "recur_step":
        return _own_step(s, case) if own else _recur_step(s, case)
    if kind == "rotary":
        return _own_rotary(s, case) if own else _rotary(s, case)
    if own:
        return _own_norm(s, case)
    return _norm_fwd(s, case) if kind == "norm_fwd" else _norm_bwd(s, case)


# ---------------------------------------------------------------------- work

def work(case):
    e, kind = 2 if case["dtype"] == BF16 else 4, case["kind"]
    if kind in ("recur_fwd", "recur_train"):
        n, D, B = case["B"] * case["L"] * case["D"], case["D"], case["B"]
        if kind == "recur_fwd":         # x, dt in, y out; h0, h_out, the two parameters
            return {"bytes": 3 * n * e + 4 * (2 * B * D + 2 * D), "flops": 12 * n}
        return {"bytes": 6 * n * e + 4 * (4 * B * D + 4 * D), "flops": 36 * n}
    if kind == "recur_step":
        n = case["B"] * case["D"]
        return {"bytes": n * (3 * e + 8) + 8 * case["D"], "flops": 12 * n}
    if kind.startswith("norm"):
        n, D, g = case["rows"] * case["D"], case["D"], int(case["gate"])
        if kind == "norm_fwd":          # y, gate, r in; r_out, xn out
            return {"bytes": (4 + g) * n * e + 4 * 5 * D, "flops": 20 * n}
        return {"bytes": (6 + 2 * g) * n * e + 4 * 10 * D, "flops": 45 * n}
    n = case["B"] * case["L"] * (case["Hq"] + case["Hk"]) * case["d"]
    return {"bytes": 2 * n * e + (8 * case["B"] * case["L"] if case["positions"] else 0),
            "flops": 3 * n * case["rot"] // case["d"]}


# --------------------------------------------------------------------- exact

def _softplus64(z):
    return torch.logaddexp(z, torch.zeros_like(z))


def _exact_recur(s, case):
    """Token by token, in 64 bits."""
    B, L, D, scale = case["B"], case["L"], case["D"], case["scale"]
    x, z = s["x"].double(), s["dt"].double() + s["dt_bias"].double()
    rate = s["A_log"].double().exp()
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), L, device="cuda")
    delta = _softplus64(z)
    a = torch.exp(-delta * rate)
    if scale == "plain":
        beta = torch.ones_like(a)
    elif scale == "step":
        beta = delta
    else:
        beta = torch.sqrt((-torch.expm1(-2 * delta * rate)).clamp(min=0))
    h = torch.zeros(B, D, dtype=torch.float64, device="cuda") if s["h0"] is None else s["h0"].double()
    before = torch.empty_like(a)        # h_{t-1} of every token
    y = torch.zeros_like(a)
    on = torch.arange(L, device="cuda")[None] < n[:, None]
    for t in range(L):
        before[:, t] = h
        new = torch.addcmul(beta[:, t] * x[:, t], a[:, t], h)
        h = new if s["lengths"] is None else torch.where(on[:, t, None], new, h)
        y[:, t] = h
    y *= on[..., None]
    out = {"y": y, "h_out": h}
    if case["kind"] == "recur_fwd":
        return out
    del y
    carry = s["dh_out"].double()        # gradient of h_t from what follows token t
    dy, g = s["dy"].double(), torch.zeros_like(a)
    for t in range(L - 1, -1, -1):
        gt = dy[:, t] + carry
        back = a[:, t] * gt
        if s["lengths"] is None:
            g[:, t], carry = gt, back
        else:
            g[:, t] = torch.where(on[:, t, None], gt, 0.0)
            carry = torch.where(on[:, t, None], back, carry)
    del dy
    dlog = g * a * before
    del before
    if scale == "unit":
        dlog -= torch.nan_to_num(g * x * a.square() / beta, nan=0.0, posinf=0.0, neginf=0.0)
    ddelta = -dlog * rate
    if scale == "step":
        ddelta += g * x
    ddt = ddelta / (1 + torch.exp(-z))
    return out | {"dx": g * beta, "ddt": ddt, "dA_log": (dlog * -delta * rate).sum((0, 1)),
                  "d_dt_bias": ddt.sum((0, 1)), "dh0": carry}


def _exact_step(s, case):
    z = s["dt"].double() + s["dt_bias"].double()
    delta, rate = _softplus64(z), s["A_log"].double().exp()
    beta = {"plain": torch.ones_like(delta), "step": delta,
            "unit": torch.sqrt(-torch.expm1(-2 * delta * rate))}[case["scale"]]
    h = torch.exp(-delta * rate) * s["h"].double() + beta * s["x"].double()
    return {"y": h, "h_out": h}


def _exact_norm(s, case):
    """The forward from its definition; the gradients by differentiating it in 64 bits."""
    D = case["D"]
    v = {k: s[k].double().clone() for k in ("y", "gate", "post_w", "post_b", "pre_w", "pre_b", "scale")
         if s[k] is not None}

    def norm(u, w, b):
        centre = u.sum(-1, keepdim=True) / D if case["norm"] == "layer" else 0.0
        var = ((u - centre) ** 2).sum(-1, keepdim=True) / D
        n = (u - centre) / torch.sqrt(var + s["eps"]) * w
        return n if b is None else n + b

    def branch():
        n = norm(v["y"], v["post_w"], v.get("post_b")) if "post_w" in v else v["y"]
        if "gate" in v:
            n = n * (v["gate"] / (1 + torch.exp(-v["gate"])))
        return s["alpha"] * v["scale"] * n

    if case["kind"] == "norm_fwd":
        r = s["r"].double() + branch()
        return {"r_out": r, "xn": norm(r, v["pre_w"], v.get("pre_b"))}
    for t in v.values():
        t.requires_grad_(True)
    r = s["r_out"].double().requires_grad_(True)
    loss = (norm(r, v["pre_w"], v.get("pre_b")) * s["dxn"].double()).sum()
    names = [k for k in ("pre_w", "pre_b") if k in v]
    got = torch.autograd.grad(loss, [r] + [v[k] for k in names])
    dr = s["dr_out"].double() + got[0]
    out = {"dr": dr} | {"d" + k: g for k, g in zip(names, got[1:])}
    names = [k for k in ("y", "gate", "scale", "post_w", "post_b") if k in v]
    got = torch.autograd.grad((branch() * dr).sum(), [v[k] for k in names])
    return out | {"d" + k: g for k, g in zip(names, got)}


def _exact_rotary(s, case):
    """Each pair as a complex number times m e^(i angle) (its conjugate for the transpose)."""
    base, factor, orig, slow, fast, m = _rope_scaling(case)
    rot = case["rot"]
    theta = []
    for i in range(rot // 2):
        b = base * factor ** (rot / (rot - 2)) if case["scaling"] == "ntk" else base
        th = math.exp(-2 * i / rot * math.log(b))
        if case["scaling"] == "linear":
            th /= factor
        elif case["scaling"] == "by_parts":
            g = min(1.0, max(0.0, (orig * th / (2 * math.pi) - slow) / (fast - slow)))
            th = (1 - g) * th / factor + g * th
        theta.append(th)
    pos = s["pos"] if s["pos"] is not None else torch.arange(case["L"], device="cuda").expand(1, -1)
    ang = pos.double().unsqueeze(-1) * torch.tensor(theta, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.full_like(ang, m), -ang if case["transpose"] else ang).unsqueeze(2)
    out = {}
    for name in ("q", "k"):
        v = s[name].double().clone()
        if case["layout"] == "half":
            w = torch.complex(v[..., :rot // 2].contiguous(), v[..., rot // 2:rot].contiguous()) * turn
            v[..., :rot // 2], v[..., rot // 2:rot] = w.real, w.imag
        else:
            w = torch.complex(v[..., 0:rot:2].contiguous(), v[..., 1:rot:2].contiguous()) * turn
            v[..., 0:rot:2], v[..., 1:rot:2] = w.real, w.imag
        out[name] = v
    return out


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("recur_fwd", "recur_train"):
        return _exact_recur(s, case)
    if kind == "recur_step":
        return _exact_step(s, case)
    if kind == "rotary":
        return _exact_rotary(s, case)
    return _exact_norm(s, case)
