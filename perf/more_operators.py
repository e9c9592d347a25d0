"""Cases of the operators that join blocks: the norms after a block and before the next one with
the block's gate and the residual's scale, and the projections into and out of a block (a matrix
product with bias, activation and residual), in bf16, fp32 and from e4m3; for prompts, for single
tokens and for training.

`run` computes an operator in plain torch operations in fp32 or, with `own` set, through the
package's entry points.  `exact` computes the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ---- cases ---------------------------------------------------------------------------------
def listed():
    return [
        # A decode batch between two blocks: the block's output is normed, scaled by a learned gate
        # per channel, added, and normed for the next block.  Latency counts.
        {"name": "join_step_64x4096", "op": "join", "B": 64, "T": 1, "D": 4096, "dtype": "bf16", "res": "bf16",
         "gate": "channel", "sigmoid": False, "post": True, "pre": True, "scale": 1.0},
        # A prompt of 16k tokens with an output gate per token and channel, taken through a sigmoid.
        {"name": "join_prompt_16384x4096_token_gate", "op": "join", "B": 1, "T": 16384, "D": 4096, "dtype": "bf16",
         "res": "bf16", "gate": "token", "sigmoid": True, "post": True, "pre": True, "scale": 1.0},
        # A training step: fp32 residual stream, one gate row per sequence (a conditioned block);
        # width H * d = 16 * 128.
        {"name": "join_train_4x2048x2048_sequence_gate", "op": "join_train", "B": 4, "T": 2048, "D": 2048,
         "dtype": "bf16", "res": "f32", "gate": "sequence", "sigmoid": False, "post": True, "pre": True, "scale": 1.0},
        # Training in fp32 at odd sizes, a scaled residual and a learned gate.
        {"name": "join_train_3x1111x777_f32", "op": "join_train", "B": 3, "T": 1111, "D": 777, "dtype": "f32",
         "res": "f32", "gate": "channel", "sigmoid": False, "post": True, "pre": True, "scale": 0.5},
        # One token for each of 16 sequences into a wide projection: the weight's bytes count.
        {"name": "linear_step_16x4096_to_8192_silu", "op": "linear", "M": 16, "K": 4096, "N": 8192, "dtype": "bf16",
         "res": None, "bias": True, "act": "silu", "slice": False},
        # A prompt batch's output projection onto the residual stream.
        {"name": "linear_prompt_8192x4096_to_4096_residual", "op": "linear", "M": 8192, "K": 4096, "N": 4096,
         "dtype": "bf16", "res": "bf16", "bias": False, "act": None, "slice": False},
        # fp32 at odd sizes: the input is a slice of wider rows.
        {"name": "linear_ragged_777x1028_to_1001_f32", "op": "linear", "M": 777, "K": 1028, "N": 1001, "dtype": "f32",
         "res": None, "bias": True, "act": "gelu", "slice": True},
        # A training step of a widening projection (the bench workload's tokens and H * d = 2048 channels).
        {"name": "linear_train_8192x2048_to_8192_gelu", "op": "linear_train", "M": 8192, "K": 2048, "N": 8192,
         "dtype": "bf16", "res": None, "bias": True, "act": "gelu", "slice": False},
        # A training step of an output projection onto an fp32 residual stream, ragged token count and width.
        {"name": "linear_train_2500x4096_to_1000_f32_residual", "op": "linear_train", "M": 2500, "K": 4096, "N": 1000,
         "dtype": "bf16", "res": "f32", "bias": True, "act": None, "slice": False},
        # One token for each of 64 sequences in 8 bits, as the norm with e4m3 output leaves them.
        {"name": "linear_e4m3_step_64x4096_to_4096", "op": "linear_e4m3", "M": 64, "K": 4096, "N": 4096,
         "dtype": "bf16", "res": None, "bias": True, "act": None, "slice": False},
        # A prompt of 16k tokens in 8 bits onto the residual stream.
        {"name": "linear_e4m3_prompt_16384x4096_to_4096", "op": "linear_e4m3", "M": 16384, "K": 4096, "N": 4096,
         "dtype": "bf16", "res": "bf16", "bias": False, "act": None, "slice": False},
    ]


MOST = 8e11  # a drawn product's operations: a little under those of the largest listed case


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["join", "join_train", "linear", "linear", "linear_train", "linear_e4m3"])
    odd = rng.random() < 0.3  # a width of any value rather than a multiple of 64
    width = lambda lo, hi: _log(rng, lo, hi) if odd else max(1, _log(rng, lo, hi) // 64) * 64  # noqa: E731
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("join"):
        D = width(256, 8192)
        most = (1 << 26) // D // (2 if op == "join_train" else 1)
        T = min(_log(rng, 1, 16384), most)
        B = max(1, min(_log(rng, 1, 64), most // T))
        return {"op": op, "B": B, "T": T, "D": D, "dtype": dtype,
                "res": "f32" if dtype == "f32" else rng.choice(["bf16", "f32"]),
                "gate": rng.choice(["none", "channel", "sequence", "token"]), "sigmoid": rng.random() < 0.4,
                "post": rng.random() < 0.8, "pre": rng.random() < 0.85, "scale": rng.choice([1.0, 1.0, 0.5, 2.0])}
    K, N = width(64, 8192), width(64, 8192)
    M = _log(rng, 1, 16384)
    flops = 2.0 * K * N * (3 if op == "linear_train" else 1) * (4 if dtype == "f32" else 1)
    M = max(1, min(M, int(MOST / flops)))
    if op == "linear_e4m3":
        dtype = "bf16"
    return {"op": op, "M": M, "K": K, "N": N, "dtype": dtype,
            "res": rng.choice([None, "f32"] if dtype == "f32" else [None, "bf16", "f32"]),
            "bias": rng.random() < 0.6, "act": rng.choice([None, None, "silu", "gelu"]),
            "slice": op != "linear_e4m3" and rng.random() < 0.2}


# ---- inputs --------------------------------------------------------------------------------
class _Draws:
    def __init__(self, seed):
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(seed)

    def normal(self, *shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, device=DEV, generator=self.g) * std).to(dtype)


def _in_8_bits(v):
    """Rows in e4m3 and a scale for each."""
    scale = v.abs().amax(1) / 448.0
    return (v / scale[:, None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    r, c = _Draws(seed), case
    dt = DTYPES[c["dtype"]]
    s = {"case": c}
    if c["op"].startswith("join"):
        B, T, D, res = c["B"], c["T"], c["D"], DTYPES[c["res"]]
        s["x"] = r.normal(B, T, D, dtype=dt)
        s["r"] = r.normal(B, T, D, std=3.0, dtype=res)
        s["w"] = 1.0 + r.normal(D, std=0.1) if c["pre"] else None
        s["wp"] = 1.0 + r.normal(D, std=0.1) if c["post"] else None
        shape = {"none": None, "channel": (D,), "sequence": (B, 1, D), "token": (B, T, D)}[c["gate"]]
        # a learned gate per channel is an fp32 parameter; the others leave a projection
        s["gate"] = None if shape is None else r.normal(*shape, dtype=torch.float32 if c["gate"] == "channel" else dt)
        if c["op"] == "join_train":
            s["dy"] = r.normal(B, T, D, dtype=dt) if c["pre"] else None
            s["dsum"] = r.normal(B, T, D, dtype=res)
        return s
    M, K, N = c["M"], c["K"], c["N"]
    wide = r.normal(M, K + 64 if c["slice"] else K)
    weight = r.normal(N, K, std=K ** -0.5)
    if c["op"] == "linear_e4m3":
        s["x"], s["sx"] = _in_8_bits(wide)
        s["w"], s["sw"] = _in_8_bits(weight)
    else:
        s["x"] = wide.to(dt)[:, :K]
        s["w"] = weight.to(dt)
    s["b"] = r.normal(N, std=0.1, dtype=dt) if c["bias"] else None
    s["r"] = r.normal(M, N, dtype=DTYPES[c["res"]]) if c["res"] else None
    if c["op"] == "linear_train":
        s["dy"] = r.normal(M, N, dtype=DTYPES[c["res"] or c["dtype"]])
    return s


# ---- one pass ------------------------------------------------------------------------------
def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _rstd(f):
    return torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)


def _plain_gate(s):
    """The gate's values in fp32, or None."""
    if s["gate"] is None:
        return None
    g = s["gate"].float()
    return torch.sigmoid(g) if s["case"]["sigmoid"] else g


def _plain_block(s):
    """The block's output once normed, and before; fp32."""
    x = s["x"].float()
    return (x if s["wp"] is None else x * _rstd(x) * s["wp"]), x


def _plain_sum(s, n, g):
    sm = s["r"].float() * s["case"]["scale"] + (n if g is None else g * n)
    return sm.to(s["r"].dtype)  # as stored, which is what is normed


def _plain_join(s):
    n, _ = _plain_block(s)
    sm = _plain_sum(s, n, _plain_gate(s))
    if s["w"] is None:
        return [sm]
    f = sm.float()
    return [sm, (f * _rstd(f) * s["w"]).to(s["x"].dtype)]


def _plain_join_train(s):
    c = s["case"]
    n, x = _plain_block(s)
    g = _plain_gate(s)
    sm = _plain_sum(s, n, g)
    out = {"s": sm}
    ds = s["dsum"].float()
    if s["w"] is not None:
        f, dy = sm.float(), s["dy"].float()
        rstd = _rstd(f)
        out["y"] = (f * rstd * s["w"]).to(s["x"].dtype)
        wd = s["w"] * dy
        ds = ds + rstd * (wd - f * (rstd * rstd * (wd * f).mean(-1, keepdim=True)))
        out["dweight"] = (dy * f * rstd).sum((0, 1))
    out["dresidual"] = (c["scale"] * ds).to(s["r"].dtype)
    dn = ds
    if g is not None:
        dg = ds * n
        dg = {"channel": lambda: dg.sum((0, 1)), "sequence": lambda: dg.sum(1, keepdim=True),
              "token": lambda: dg}[c["gate"]]()
        if c["sigmoid"]:
            dg = dg * (g * (1 - g))
        out["dgate"] = dg.to(s["gate"].dtype)
        dn = ds * g
    if s["wp"] is not None:
        rstd = _rstd(x)
        out["dpost_weight"] = (dn * x * rstd).sum((0, 1))
        wd = s["wp"] * dn
        dn = rstd * (wd - x * (rstd * rstd * (wd * x).mean(-1, keepdim=True)))
    out["dx"] = dn.to(s["x"].dtype)
    return out


def _plain_act(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * 0.5 * (1 + torch.erf(z * 0.5 ** 0.5))
    return z


def _plain_act_grad(z, act):
    if act == "silu":
        g = torch.sigmoid(z)
        return g * (1 + z * (1 - g))
    return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5


def _plain_finish(s, z, dtype):
    y = _plain_act(z, s["case"]["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    return y.to(s["r"].dtype if s["r"] is not None else dtype)


def _plain_product(s):
    z = s["x"].float() @ s["w"].float().t()
    return z if s["b"] is None else z + s["b"].float()


def _plain_linear(s):
    return [_plain_finish(s, _plain_product(s), s["x"].dtype)]


def _plain_linear_train(s):
    z = _plain_product(s)
    out = [_plain_finish(s, z, s["x"].dtype)]
    dz = s["dy"].float()
    if s["case"]["act"] is not None:
        dz = dz * _plain_act_grad(z, s["case"]["act"])
    out += [(dz @ s["w"].float()).to(s["x"].dtype), (dz.t() @ s["x"].float()).to(s["w"].dtype)]
    if s["b"] is not None:
        out.append(dz.sum(0).to(s["b"].dtype))
    return out


def _plain_linear_e4m3(s):
    z = (s["x"].float() @ s["w"].float().t()) * s["sx"][:, None] * s["sw"]
    if s["b"] is not None:
        z = z + s["b"].float()
    return [_plain_finish(s, z, torch.bfloat16)]


_plain = {"join": _plain_join, "join_train": _plain_join_train, "linear": _plain_linear,
          "linear_train": _plain_linear_train, "linear_e4m3": _plain_linear_e4m3}


# ---- the same through the package ----------------------------------------------------------
def _own_join(s):
    import gated_delta_rule_chunkwise_gb300 as ldn
    c = s["case"]
    y, sm = ldn.gated_add_rmsnorm(s["x"], s["r"], s["w"], s["wp"], s["gate"], residual_scale=c["scale"],
                                  gate_sigmoid=c["sigmoid"], eps=EPS)
    return [sm] if y is None else [sm, y]


def _own_join_train(s):
    import gated_delta_rule_chunkwise_gb300 as ldn
    c = s["case"]
    y, sm = ldn.gated_add_rmsnorm(s["x"], s["r"], s["w"], s["wp"], s["gate"], residual_scale=c["scale"],
                                  gate_sigmoid=c["sigmoid"], eps=EPS)
    g = ldn.gated_add_rmsnorm_backward(s["dy"], s["x"], sm, s["w"], s["wp"], s["gate"], s["dsum"],
                                       residual_scale=c["scale"], gate_sigmoid=c["sigmoid"], eps=EPS)
    out = {"s": sm, "dx": g["dx"], "dresidual": g["dresidual"]}
    if s["w"] is not None:
        out["y"], out["dweight"] = y, g["dweight"]
    if s["wp"] is not None:
        out["dpost_weight"] = g["dpost_weight"]
    if s["gate"] is not None:
        out["dgate"] = g["dgate"]
    return out


def _own_linear(s):
    import gated_delta_rule_chunkwise_gb300 as ldn
    return [ldn.linear(s["x"], s["w"], s["b"], s["r"], activation=s["case"]["act"])]


def _own_linear_train(s):
    import gated_delta_rule_chunkwise_gb300 as ldn
    act = s["case"]["act"]
    if act is None:
        y, z = ldn.linear(s["x"], s["w"], s["b"], s["r"]), None
    else:
        y, z = ldn.linear(s["x"], s["w"], s["b"], s["r"], activation=act, save_z=True)
    g = ldn.linear_backward(s["dy"], s["x"], s["w"], z, activation=act, bias=s["b"] is not None)
    out = [y, g["dx"], g["dweight"]]
    if s["b"] is not None:
        out.append(g["dbias"])
    return out


def _own_linear_e4m3(s):
    import gated_delta_rule_chunkwise_gb300 as ldn
    return [ldn.linear_e4m3(s["x"], s["sx"], s["w"], s["sw"], s["b"], s["r"], activation=s["case"]["act"])]


_own = {"join": _own_join, "join_train": _own_join_train, "linear": _own_linear, "linear_train": _own_linear_train,
        "linear_e4m3": _own_linear_e4m3}


# ---- the least work ------------------------------------------------------------------------
def work(case):
    c, e = case, 2 if case["dtype"] == "bf16" else 4
    if c["op"].startswith("join"):
        n, r = c["B"] * c["T"] * c["D"], 2 if c["res"] == "bf16" else 4
        gate = {"none": 0, "channel": 4 * c["D"], "sequence": e * c["B"] * c["D"], "token": e * n}[c["gate"]]
        par = 4 * c["D"] * (c["post"] + c["pre"])
        fwd = n * (e + 2 * r + (e if c["pre"] else 0)) + gate + par
        if c["op"] == "join":
            return {"bytes": fwd, "flops": 14 * n}
        # dy and dsum in, dx and dresidual out, the parameters' gradients
        return {"bytes": fwd + n * ((e if c["pre"] else 0) + r + e + r) + gate + par, "flops": 40 * n}
    M, K, N = c["M"], c["K"], c["N"]
    r = {None: 0, "bf16": 2, "f32": 4}[c["res"]]
    y = r or e
    if c["op"] == "linear_e4m3":
        return {"bytes": M * K + N * K + 4 * (M + N) + M * N * (y + r) + (2 * N if c["bias"] else 0),
                "flops": 2 * M * N * K}
    fwd = e * (M * K + N * K + (N if c["bias"] else 0)) + M * N * (y + r)
    if c["op"] == "linear":
        return {"bytes": fwd, "flops": 2 * M * N * K}
    return {"bytes": fwd + e * (M * K + N * K + (N if c["bias"] else 0)) + M * N * y, "flops": 6 * M * N * K}


# ---- the definitions in 64 bits ------------------------------------------------------------
def exact(case, seed):
    s = {k: v.float().double() if torch.is_tensor(v) else v for k, v in prepare(case, seed).items()}
    return _exact_join(s) if case["op"].startswith("join") else _exact_linear(s)


def _exact_normed(v, w):
    """Rows over their root mean square, times w; the first, and one over that root."""
    inv = 1.0 / torch.sqrt(torch.mean(v ** 2, dim=1) + EPS)
    xh = torch.einsum("rd,r->rd", v, inv)
    return xh * w, xh, inv


def _exact_norm_grad(gxh, xh, inv):
    """What reaches the row from what reaches the normed one."""
    dot = torch.einsum("rd,rd->r", gxh, xh) / xh.shape[1]
    return (gxh - xh * dot[:, None]) * inv[:, None]


def _exact_join(s):
    c = s["case"]
    B, T, D = c["B"], c["T"], c["D"]
    flat = lambda v: None if v is None else v.reshape(-1, D)  # noqa: E731
    x, r, w, wp = flat(s["x"]), flat(s["r"]), s["w"], s["wp"]
    n, xh, inv = (x, None, None) if wp is None else _exact_normed(x, wp)
    if s["gate"] is None:
        gate = torch.ones(1, D, dtype=torch.float64, device=DEV)
    else:
        gate = flat(s["gate"])
        if c["sigmoid"]:
            gate = 1.0 / (1.0 + torch.exp(-gate))
    each = gate.repeat_interleave(B * T // gate.shape[0], 0)
    sm = (c["scale"] * r + each * n).to(DTYPES[c["res"]]).double()  # what is stored is what is normed
    shape = lambda v: v.reshape(B, T, D)  # noqa: E731
    if w is not None:
        y, sh, sinv = _exact_normed(sm, w)
    if c["op"] == "join":
        return [shape(sm)] if w is None else [shape(sm), shape(y)]
    out = {"s": shape(sm)}
    ds = flat(s["dsum"])
    if w is not None:
        dy = flat(s["dy"])
        out["y"], out["dweight"] = shape(y), torch.einsum("rd,rd->d", dy, sh)
        ds = ds + _exact_norm_grad(dy * w, sh, sinv)
    out["dresidual"] = shape(c["scale"] * ds)
    if s["gate"] is not None:
        dg = (ds * n).reshape(gate.shape[0], -1, D).sum(1)
        if c["sigmoid"]:
            dg = dg * gate * (1.0 - gate)
        out["dgate"] = dg.reshape(s["gate"].shape)
    dn = ds * each
    if wp is not None:
        out["dpost_weight"] = torch.einsum("rd,rd->d", dn, xh)
        dn = _exact_norm_grad(dn * wp, xh, inv)
    out["dx"] = shape(dn)
    return out


def _exact_linear(s):
    c = s["case"]
    x, w = s["x"], s["w"]
    if c["op"] == "linear_e4m3":
        x, w = x * s["sx"][:, None], w * s["sw"][:, None]
    z = torch.einsum("mk,nk->mn", x, w)
    if s["b"] is not None:
        z = z + s["b"]
    if c["act"] == "silu":
        sig = 1.0 / (1.0 + torch.exp(-z))
        y, slope = z * sig, sig + z * sig * (1.0 - sig)
    elif c["act"] == "gelu":
        normal = torch.special.erfc(-z / math.sqrt(2.0)) / 2.0  # the normal distribution's integral up to z
        y, slope = z * normal, normal + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
    else:
        y, slope = z, torch.ones_like(z)
    if s["r"] is not None:
        y = y + s["r"]
    if c["op"] != "linear_train":
        return [y]
    dz = s["dy"] * slope
    out = [y, torch.einsum("mn,nk->mk", dz, w), torch.einsum("mn,mk->nk", dz, x)]
    if s["b"] is not None:
        out.append(torch.einsum("mn->n", dz))
    return out
