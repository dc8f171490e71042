"""The operators that train the block's dense branch, as cases to be measured.

Three families, each in its plain form (elementary torch operations in 32 bits) and, where
`own` is true, as the calls that a user makes of mixture_experts_ffn_05_b200.train:

  norm   RMS norm or layer norm, forward and backward: y and the row statistics, then dx and
         the gradients of the gain and the bias.  With `keep` the forward pass stores x in
         8 bits and the backward pass reads that copy in place of x.
  act8   an activation written as an 8-bit checkpoint and read back.
  mlp    the gated feed-forward block y = (act(x Wg^T) * (x Wu^T)) Wd^T.  `part` is forward,
         backward (from pre-activations kept in 16 bits) or step: forward and backward with
         x and the pre-activations kept in 8 bits.

An 8-bit checkpoint holds groups of 32 consecutive values of a row: s = the smallest power of
two (at least 2^-126) with max|v| <= Q s, Q = 127 (int8) or 448 (E4M3); codes are v / s,
rounded to nearest even.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
GROUP = 32


def listed():
    return [
        # a single token's norm: launch latency alone
        {"name": "norm_rms_T1", "op": "norm", "kind": "rms", "T": 1, "H": 2816, "dtype": "bf16",
         "bias": False, "keep": "none"},
        # rows that no 16-byte load fits, an odd number of them
        {"name": "norm_layer_odd_f16", "op": "norm", "kind": "layer", "T": 4095, "H": 1001,
         "dtype": "f16", "bias": True, "keep": "none"},
        # the layer's pre norm over a long batch, its input kept in 8 bits
        {"name": "norm_rms_int8_T16384", "op": "norm", "kind": "rms", "T": 16384, "H": 2816,
         "dtype": "bf16", "bias": False, "keep": "int8"},
        # the widest rows of the interface, in fp32
        {"name": "norm_layer_f32_T8192", "op": "norm", "kind": "layer", "T": 8192, "H": 6144,
         "dtype": "f32", "bias": True, "keep": "none"},
        # a short ragged batch of dense activations
        {"name": "act8_e4m3_T333", "op": "act8", "T": 333, "C": 2112, "dtype": "f16",
         "keep": "e4m3"},
        # the dense pre-activations of a long batch
        {"name": "act8_int8_T16384", "op": "act8", "T": 16384, "C": 4224, "dtype": "bf16",
         "keep": "int8"},
        # a decode batch through the dense MLP, nothing kept: bound by the weights' bytes
        {"name": "mlp_forward_T8", "op": "mlp", "part": "forward", "act": "gelu_tanh", "T": 8,
         "H": 2816, "D": 2112, "dtype": "bf16", "keep": "none"},
        # sizes that are no multiple of any tile, the other activation, fp16
        {"name": "mlp_forward_ragged_f16", "op": "mlp", "part": "forward", "act": "silu",
         "T": 1001, "H": 1000, "D": 1352, "dtype": "f16", "keep": "16"},
        # a training batch of the layer's dense MLP, pre-activations kept in 16 bits
        {"name": "mlp_forward_T8192", "op": "mlp", "part": "forward", "act": "gelu_tanh",
         "T": 8192, "H": 2816, "D": 2112, "dtype": "bf16", "keep": "16"},
        # the smallest micro-batch: the gradients' bytes bind
        {"name": "mlp_backward_T64", "op": "mlp", "part": "backward", "act": "gelu_tanh", "T": 64,
         "H": 2816, "D": 2112, "dtype": "bf16", "keep": "16"},
        # an ordinary micro-batch
        {"name": "mlp_backward_T4096", "op": "mlp", "part": "backward", "act": "gelu_tanh",
         "T": 4096, "H": 2816, "D": 2112, "dtype": "bf16", "keep": "16"},
        # a whole training step of a long batch from 8-bit checkpoints
        {"name": "mlp_step_int8_T16384", "op": "mlp", "part": "step", "act": "gelu_tanh",
         "T": 16384, "H": 2816, "D": 2112, "dtype": "bf16", "keep": "int8"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "act8", "mlp", "mlp"))
    if op == "norm":
        c = {"op": op, "kind": rng.choice(("rms", "layer")), "T": _log(rng, 1, 16384),
             "H": _log(rng, 128, 6144), "dtype": rng.choice(("bf16", "bf16", "f16", "f32")),
             "keep": rng.choice(("none", "int8", "e4m3"))}
        c["bias"] = c["kind"] == "layer" and rng.random() < 0.7
        if rng.random() < 0.6:
            c["H"] = -(-c["H"] // 8) * 8
        return c
    if op == "act8":
        c = {"op": op, "T": _log(rng, 1, 16384), "C": _log(rng, 64, 6144),
             "dtype": rng.choice(("bf16", "f16", "f32")), "keep": rng.choice(("int8", "e4m3"))}
        if rng.random() < 0.6:
            c["C"] = -(-c["C"] // 8) * 8
        return c
    part = rng.choice(("forward", "backward", "step"))
    return {"op": op, "part": part, "act": rng.choice(("gelu_tanh", "silu")),
            "T": _log(rng, 1, 8192), "H": 8 * _log(rng, 16, 384), "D": 8 * _log(rng, 16, 300),
            "dtype": rng.choice(("bf16", "bf16", "f16")),
            "keep": rng.choice(("int8", "e4m3")) if part == "step" else
            rng.choice(("none", "16")) if part == "forward" else "16"}


# ------------------------------------------------------------------------------- inputs

def _inputs(case, seed):
    """The tensors a program has before the call; weights as a layer's draw has them
    (N(0, 0.02), gains U(0.5, 1.5)), activations N(0, 1) with a few strong channels."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    def channels(n):
        return 1.0 + 4.0 * (torch.rand(n, generator=g, device="cuda") < 0.01)

    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        x = normal(T, H) * channels(H) + 0.25 * normal(T, 1)
        s = {"x": x.to(dt), "dy": normal(T, H).to(dt),
             "gain": (torch.rand(H, generator=g, device="cuda") + 0.5).to(dt), "bias": None}
        if case["bias"]:
            s["bias"] = normal(H, std=0.1).to(dt)
        return s
    if case["op"] == "act8":
        return {"x": (normal(case["T"], case["C"]) * channels(case["C"])).to(dt)}
    T, H, D = case["T"], case["H"], case["D"]
    s = {"x": normal(T, H).to(dt), "w_gate_up": normal(2 * D, H, std=0.02).to(dt),
         "w_down": normal(H, D, std=0.02).to(dt)}
    if case["part"] != "forward":
        s["dy"] = normal(T, H).to(dt)
    if case["part"] == "backward":
        s["gu"] = (s["x"].float() @ s["w_gate_up"].float().t()).to(dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:  # the configuration, workspace and output buffers that a program keeps
        _prepare_own(s)
    return s


# ------------------------------------------------------------------------- the plain form

def _scale_exponents(v, fmt):
    """Exponent of each group's scale: max|v| = m 2^e with m in [0.5, 1), Q = f 2^n, so the
    smallest power of two with max|v| <= Q s is 2^(e - n), or the next one when m > f."""
    f, n = (127 / 128, 7) if fmt == "int8" else (448 / 512, 9)
    m, e = torch.frexp(v.abs().amax(dim=-1, keepdim=True))
    k = e - n + (m > f).to(e.dtype)
    return k.clamp_min(-126)


def _eight_bits(v, fmt):
    """The values that an 8-bit checkpoint of v [rows][cols] stands for, in v's precision."""
    rows, cols = v.shape
    pad = -cols % GROUP
    w = torch.nn.functional.pad(v, (0, pad)).reshape(rows, -1, GROUP)
    k = _scale_exponents(w, fmt)
    q = torch.ldexp(w, -k)
    q = torch.round(q) if fmt == "int8" else q.to(torch.float8_e4m3fn).to(v.dtype)
    return torch.ldexp(q, k).reshape(rows, -1)[:, :cols]


def _halves8(gu, fmt):
    """Gate and up halves kept in 8 bits, each with groups of its own."""
    g, u = gu.chunk(2, dim=1)
    return torch.cat((_eight_bits(g, fmt), _eight_bits(u, fmt)), dim=1)


def _norm(s, f):
    """Forward and backward of the norm in the precision of torch type f."""
    c = s["case"]
    x, dy, gain = s["x"].to(f), s["dy"].to(f), s["gain"].to(f)
    layer = c["kind"] == "layer"
    mean = x.mean(dim=1, keepdim=True) if layer else torch.zeros_like(x[:, :1])
    rstd = torch.rsqrt(((x - mean) ** 2).mean(dim=1, keepdim=True) + EPS)
    y = (x - mean) * rstd * gain
    if s["bias"] is not None:
        y = y + s["bias"].to(f)
    kept = x if c["keep"] == "none" else _eight_bits(x, c["keep"])
    xhat = (kept - mean) * rstd
    a = dy * gain
    dx = a - xhat * (a * xhat).mean(dim=1, keepdim=True)
    if layer:
        dx = dx - a.mean(dim=1, keepdim=True)
    out = {"y": y, "rstd": rstd[:, 0], "dx": dx * rstd, "d_gain": (dy * xhat).sum(dim=0)}
    if layer:
        out["mean"] = mean[:, 0]
    if s["bias"] is not None:
        out["d_bias"] = dy.sum(dim=0)
    return out


def _act(g, name):
    """The activation of the gate and its derivative."""
    if name == "silu":
        sg = 1 / (1 + torch.exp(-g))
        return g * sg, sg * (1 + g * (1 - sg))
    k0, k1 = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(k0 * (g + k1 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k0 * (1 + 3 * k1 * g * g)


def _mlp(s, f):
    """The part of the gated MLP that the case asks for, in the precision of torch type f."""
    c = s["case"]
    x, wgu, wd = s["x"].to(f), s["w_gate_up"].to(f), s["w_down"].to(f)
    out = {}
    if c["part"] != "backward":
        gu = x @ wgu.t()
        g, u = gu.chunk(2, dim=1)
        out["y"] = (_act(g, c["act"])[0] * u) @ wd.t()
        if c["part"] == "forward":
            if c["keep"] == "16":
                out["gu"] = gu
            return out
        gu, x = _halves8(gu, c["keep"]), _eight_bits(x, c["keep"])
    else:
        gu = s["gu"].to(f)
    dy = s["dy"].to(f)
    g, u = gu.chunk(2, dim=1)
    a, da = _act(g, c["act"])
    dh = dy @ wd
    dgu = torch.cat((dh * u * da, dh * a), dim=1)
    out["dx"] = dgu @ wgu
    out["dw_gate_up"] = dgu.t() @ x
    out["dw_down"] = dy.t() @ (a * u)
    return out


FP32_OUTPUTS = ("rstd", "mean", "d_gain", "d_bias")


def _rounded(out, case):
    dt = DTYPES[case["dtype"]]
    return {n: v if n in FP32_OUTPUTS else v.to(dt) for n, v in out.items()}


def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    if c["op"] == "act8":
        return _eight_bits(s["x"].float(), c["keep"]).to(DTYPES[c["dtype"]])
    return _rounded((_norm if c["op"] == "norm" else _mlp)(s, torch.float32), c)


# ---------------------------------------------------------------- the framework's kernels

def _prepare_own(s):
    from mixture_experts_ffn_05_b200 import train
    c = s["case"]
    x, dt = s["x"], DTYPES[c["dtype"]]
    f32 = {"dtype": torch.float32, "device": "cuda"}
    if c["op"] == "act8":
        s["kept"] = train.act8(c["T"], c["C"], c["keep"])
        s["back"] = torch.empty_like(x)
        return
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        s["cfg"] = train.NormConfig(cols=H, kind=c["kind"], eps=EPS, dtype=dt, param_dtype=dt)
        s["ws"] = train.norm_workspace(s["cfg"], T)
        s["y"], s["dx"] = torch.empty_like(x), torch.empty_like(x)
        s["rstd"] = torch.empty(T, **f32)
        s["mean"] = torch.empty(T, **f32) if c["kind"] == "layer" else None
        s["d_gain"] = torch.empty(H, **f32)
        s["d_bias"] = torch.empty(H, **f32) if c["bias"] else None
        s["kept"] = None if c["keep"] == "none" else train.act8(T, H, c["keep"])
        return
    T, H, D = c["T"], c["H"], c["D"]
    s["cfg"] = train.MlpConfig(hidden=H, inter=D, act=c["act"], dtype=dt)
    s["ws"] = train.mlp_workspace(s["cfg"], T)
    if c["part"] != "backward":
        s["y"] = torch.empty_like(x)
        s["kept_gu"] = None
        if c["keep"] == "16":
            s["kept_gu"] = torch.empty(T, 2 * D, dtype=dt, device="cuda")
        elif c["keep"] != "none":
            s["kept_gu"] = train.act8(T, D, c["keep"], parts=2)
            s["kept_x"] = train.act8(T, H, c["keep"])
    if c["part"] != "forward":
        s["dx"] = torch.empty_like(x)
        s["dw_gate_up"] = torch.empty_like(s["w_gate_up"])
        s["dw_down"] = torch.empty_like(s["w_down"])


def _run_own(s):
    from mixture_experts_ffn_05_b200 import train
    c = s["case"]
    x = s["x"]
    if c["op"] == "act8":
        train.moe_act_encode(x, s["kept"])
        train.moe_act_decode(s["kept"], s["back"])
        return s["back"]
    if c["op"] == "norm":
        train.moe_norm_forward(s["cfg"], x, s["gain"], s["bias"], s["y"], s["mean"], s["rstd"],
                               kept=s["kept"])
        train.moe_norm_backward(s["cfg"], x if s["kept"] is None else s["kept"], s["gain"],
                                s["mean"], s["rstd"], s["dy"], s["dx"], s["d_gain"],
                                s["d_bias"], s["ws"])
        names = ("y", "rstd", "mean", "dx", "d_gain", "d_bias")
        return {n: s[n] for n in names if s[n] is not None}
    out = {}
    if c["part"] != "backward":
        train.moe_mlp_forward(s["cfg"], x, s["w_gate_up"], s["w_down"], s["y"], s["ws"],
                              kept_gu=s["kept_gu"])
        out["y"] = s["y"]
        if c["part"] == "forward":
            if c["keep"] == "16":
                out["gu"] = s["kept_gu"]
            return out
        train.moe_act_encode(x, s["kept_x"])
        x, gu = s["kept_x"], s["kept_gu"]
    else:
        gu = s["gu"]
    train.moe_mlp_backward(s["cfg"], x, gu, s["w_gate_up"], s["w_down"], s["dy"], s["dx"],
                           s["dw_gate_up"], s["dw_down"], s["ws"])
    out.update({n: s[n] for n in ("dx", "dw_gate_up", "dw_down")})
    return out


# ------------------------------------------------------------------------------ the floor

def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    per8 = 1 + 1 / GROUP  # bytes of a value in 8 bits with its share of the scale
    if case["op"] == "act8":
        n = case["T"] * case["C"]
        return {"bytes": n * 2 * (es + per8), "flops": 4 * n}
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        n = T * H
        stats = 4 * T * (2 if case["kind"] == "layer" else 1)
        params = H * (2 * es + 4 + (es + 4 if case["bias"] else 0))
        # forward: x in, y out; backward: x (or its copy) and dy in, dx out
        x_again = es if case["keep"] == "none" else 2 * per8  # the copy is written, then read
        return {"bytes": n * (4 * es + x_again) + 2 * stats + params, "flops": 18 * n}
    T, H, D = case["T"], case["H"], case["D"]
    weights = 3 * H * D * es
    kept = 2 * per8 if case["keep"] in ("int8", "e4m3") else es
    bytes_, flops = 0, 0
    if case["part"] != "backward":
        bytes_ += weights + 2 * T * H * es  # x in, y out
        flops += 6 * T * H * D
        if case["keep"] != "none":  # the pre-activations out
            bytes_ += T * 2 * D * (es if case["part"] == "forward" else kept / 2)
        if case["part"] == "step":  # x read again for its copy, which is written
            bytes_ += T * H * kept / 2
    if case["part"] != "forward":
        half = kept / 2 if case["part"] == "step" else es
        # x, pre-activations, dy and the weights in; dx and the weights' gradients out
        bytes_ += T * H * (half + 2 * es) + T * 2 * D * half + 2 * weights
        flops += 12 * T * H * D
    return {"bytes": bytes_, "flops": flops}


# ------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """The outputs from the operators' definitions in 64 bits, written with row-wise sums of
    their own: a normalised row's gradient as the projection that it is, the MLP's
    activations through the logistic function."""
    s = _inputs(case, seed)
    d = {n: v.double() for n, v in s.items() if v is not None}
    fmt = case["keep"]

    def kept(v):
        cols = v.shape[1]
        out = torch.empty_like(v)
        whole = cols // GROUP * GROUP
        for lo, hi, wide in ((0, whole, GROUP), (whole, cols, cols - whole)):
            if hi == lo:
                continue
            w = v[:, lo:hi].reshape(v.shape[0], -1, wide)
            top = w.abs().amax(dim=2, keepdim=True)
            q = 127.0 if fmt == "int8" else 448.0
            scale = torch.exp2(torch.ceil(torch.log2(top / q)).clamp_min(-126))
            # the logarithm may miss a border by its own rounding: put it right
            scale = torch.where(scale * q < top, scale * 2, scale)
            scale = torch.where((scale * q / 2 >= top) & (scale > 2.0 ** -126), scale / 2, scale)
            r = w / scale
            if fmt == "int8":
                r = r.round()
            else:  # three bits after the leading one, down to steps of 2^-9
                step = torch.exp2(torch.floor(torch.log2(r.abs().clamp_min(2.0 ** -6))) - 3)
                r = (r / step).round() * step
            out[:, lo:hi] = (r * scale).reshape(v.shape[0], -1)
        return out

    if case["op"] == "act8":
        return kept(d["x"])
    if case["op"] == "norm":
        x, dy, g = d["x"], d["dy"], d["gain"]
        n = x.shape[1]
        layer = case["kind"] == "layer"
        mu = x.sum(1) / n if layer else x.new_zeros(x.shape[0])
        r = (((x - mu[:, None]).pow(2).sum(1) / n) + EPS).pow(-0.5)
        z = (x - mu[:, None]) * r[:, None]
        out = {"y": z * g + (d["bias"] if "bias" in d else 0.0), "rstd": r}
        if fmt != "none":
            z = (kept(x) - mu[:, None]) * r[:, None]
        p = dy * g
        out["dx"] = r[:, None] * (p - z * ((p * z).sum(1) / n)[:, None] -
                                  ((p.sum(1) / n)[:, None] if layer else 0.0))
        out["d_gain"] = (dy * z).sum(0)
        if layer:
            out["mean"] = mu
        if "bias" in d:
            out["d_bias"] = dy.sum(0)
        return out

    x, w1, w2, D = d["x"], d["w_gate_up"], d["w_down"], case["D"]

    def gate(v):
        """act(v) = v L(c(v)) with the logistic L: c(v) = v (silu) or 2 k (v + a v^3)."""
        if case["act"] == "silu":
            c, dc = v, torch.ones_like(v)
        else:
            k = 2 * math.sqrt(2 / math.pi)
            c, dc = k * (v + 0.044715 * v.pow(3)), k * (1 + 3 * 0.044715 * v.pow(2))
        sig = torch.sigmoid(c)
        return v * sig, sig + v * sig * (1 - sig) * dc

    out = {}
    if case["part"] == "backward":
        a, b = d["gu"][:, :D], d["gu"][:, D:]
    else:
        a, b = x @ w1[:D].t(), x @ w1[D:].t()
        out["y"] = (gate(a)[0] * b) @ w2.t()
        if case["part"] == "forward":
            if fmt == "16":
                out["gu"] = torch.cat((a, b), 1)
            return out
        a, b, x = kept(a), kept(b), kept(x)
    v, dv = gate(a)
    dh = d["dy"] @ w2
    da, db = dh * b * dv, dh * v
    out["dx"] = da @ w1[:D] + db @ w1[D:]
    out["dw_gate_up"] = torch.cat((da.t() @ x, db.t() @ x), 0)
    out["dw_down"] = d["dy"].t() @ (v * b)
    return out
