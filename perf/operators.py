"""Cases of the operators around a recurrent token mixer: the RMS norm with the residual's
addition and an 8-bit output, the short causal convolution with a carried state, and the
selective state space scan; for prompts, for single tokens and for training.

`run` computes an operator in plain torch operations (fp32, or fp64 where a rounding border
decides) or, with `own` set, through the package's entry points.  `exact` computes the same
outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100  # a group whose largest magnitude is below counts as this large


# ---- cases ---------------------------------------------------------------------------------
def listed():
    return [
        # A decode batch's block input: residual add, norm, and e4m3 for the next projection in
        # the 1 x 128 scaling blocks of a block-scaled product.  Latency counts.
        {"name": "norm_step_64x4096_e4m3_g128", "op": "norm", "rows": 64, "dim": 4096, "dtype": "bf16", "res": "bf16",
         "eight": True, "group": 128},
        # The same for a prompt of 16k tokens, one scale per token.
        {"name": "norm_prompt_16384x4096_e4m3", "op": "norm", "rows": 16384, "dim": 4096, "dtype": "bf16",
         "res": "bf16", "eight": True, "group": 0},
        # A training step's norm: fp32 residual stream, forward and backward; width H * d = 16 * 128.
        {"name": "norm_train_8192x2048", "op": "norm_train", "rows": 8192, "dim": 2048, "dtype": "bf16", "res": "f32"},
        # A prompt batch: x is one half of the input projection's output, the state goes to decoding.
        {"name": "conv_prompt_b4_t2048_c4096_w4", "op": "conv", "B": 4, "T": 2048, "C": 4096, "W": 4, "dtype": "bf16",
         "bias": True, "act": True, "state": False, "ragged": False},
        # Right-padded prompts that continue cached sequences; odd sizes, fp32, width not a multiple of 8.
        {"name": "conv_ragged_b7_t777_c1028_w3_f32", "op": "conv", "B": 7, "T": 777, "C": 1028, "W": 3, "dtype": "f32",
         "bias": False, "act": True, "state": True, "ragged": True},
        # One token for each of 64 sequences.
        {"name": "conv_step_b64_c4096_w4", "op": "conv_step", "B": 64, "C": 4096, "W": 4, "dtype": "bf16",
         "bias": True, "act": True},
        # A training step of the convolution (the bench workload's tokens and H * d = 2048 channels).
        {"name": "conv_train_b4_t2048_c2048_w4", "op": "conv_train", "B": 4, "T": 2048, "C": 2048, "W": 4,
         "dtype": "bf16", "bias": True, "act": True, "state": False, "ragged": False},
        # A prompt batch of the scan: four prompts of 2048 tokens.
        {"name": "scan_prompt_b4_t2048_d4096_n16", "op": "scan", "B": 4, "T": 2048, "D": 4096, "N": 16, "G": 1,
         "dtype": "bf16", "z": True, "h0": False, "ragged": False},
        # One long document alone: few channels for the whole card.
        {"name": "scan_long_b1_t32768_d2048_n16", "op": "scan", "B": 1, "T": 32768, "D": 2048, "N": 16, "G": 1,
         "dtype": "bf16", "z": True, "h0": False, "ragged": False},
        # Right-padded fp32 prompts continuing from states, two groups, a larger state, no output gate.
        {"name": "scan_ragged_b6_t509_d1000_n64_g2_f32", "op": "scan", "B": 6, "T": 509, "D": 1000, "N": 64, "G": 2,
         "dtype": "f32", "z": False, "h0": True, "ragged": True},
        # One token for each of 64 sequences.
        {"name": "scan_step_b64_d4096_n16", "op": "scan_step", "B": 64, "D": 4096, "N": 16, "G": 1, "dtype": "bf16",
         "z": True},
        # A training step of the scan: forward and backward.
        {"name": "scan_train_b2_t2048_d4096_n16", "op": "scan_train", "B": 2, "T": 2048, "D": 4096, "N": 16, "G": 1,
         "dtype": "bf16", "z": True, "h0": False, "ragged": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_train", "conv", "conv_step", "conv_train", "scan", "scan_step", "scan_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    odd = rng.random() < 0.3  # a width of any value rather than a multiple of 64
    width = lambda lo, hi: _log(rng, lo, hi) if odd else max(1, _log(rng, lo, hi) // 64) * 64  # noqa: E731
    if op in ("norm", "norm_train"):
        dim = width(256, 8192)
        rows = min(_log(rng, 1, 16384), (1 << 26) // dim // (2 if op == "norm_train" else 1))
        c = {"op": op, "rows": rows, "dim": dim, "dtype": dtype,
             "res": "f32" if dtype == "f32" else rng.choice(["bf16", "f32"])}
        if op == "norm":
            c |= {"eight": rng.random() < 0.7, "group": rng.choice([0, 128])}
        return c
    if op == "conv_step":
        return {"op": op, "B": _log(rng, 1, 256), "C": width(256, 8192), "W": rng.randint(2, 8), "dtype": dtype,
                "bias": rng.random() < 0.5, "act": rng.random() < 0.8}
    if op in ("conv", "conv_train"):
        C = width(256, 8192)
        T = _log(rng, 2, 32768)
        B = max(1, min(_log(rng, 1, 16), (1 << 25) // (T * C)))
        T = min(T, (1 << 25) // (B * C))
        return {"op": op, "B": B, "T": T, "C": C, "W": rng.randint(2, 8), "dtype": dtype, "bias": rng.random() < 0.5,
                "act": rng.random() < 0.8, "state": rng.random() < 0.5, "ragged": rng.random() < 0.4}
    N, G = rng.choice([8, 16, 16, 32, 64]), rng.choice([1, 1, 2, 4])
    D = max(G, width(256, 8192) // G * G)
    if op == "scan_step":
        return {"op": op, "B": _log(rng, 1, 256), "D": D, "N": N, "G": G, "dtype": dtype, "z": rng.random() < 0.7}
    most = (1 << 28) if op == "scan" else (1 << 27)
    T = _log(rng, 2, 32768)
    T = min(T, most // (D * N))
    B = max(1, min(_log(rng, 1, 16), most // (T * D * N)))
    return {"op": op, "B": B, "T": T, "D": D, "N": N, "G": G, "dtype": dtype, "z": rng.random() < 0.7,
            "h0": rng.random() < 0.5, "ragged": rng.random() < 0.4}


# ---- inputs --------------------------------------------------------------------------------
class _Draws:
    def __init__(self, seed):
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(seed)

    def normal(self, *shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, device=DEV, generator=self.g) * std).to(dtype)

    def uniform(self, *shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, device=DEV, generator=self.g) * (hi - lo) + lo

    def lens(self, B, T):
        n = torch.randint(0, T + 1, (B,), device=DEV, generator=self.g, dtype=torch.int32)
        n[0] = T
        return n


def prepare(case, seed):
    r, c, op = _Draws(seed), case, case["op"]
    dt = DTYPES[c["dtype"]]
    s = {"case": c}
    if op in ("norm", "norm_train"):
        rows, dim, res = c["rows"], c["dim"], DTYPES[c["res"]]
        s["x"] = r.normal(rows, dim, dtype=dt)
        s["r"] = r.normal(rows, dim, std=3.0, dtype=res)
        s["w"] = 1.0 + r.normal(dim, std=0.1)
        if op == "norm_train":
            s["dy"] = r.normal(rows, dim, dtype=dt)
            s["dsum"] = r.normal(rows, dim, dtype=res)
        return s
    if op.startswith("conv"):
        B, C, W = c["B"], c["C"], c["W"]
        s["w"] = r.normal(C, W, std=W ** -0.5)
        s["b"] = r.normal(C, std=0.1) if c["bias"] else None
        if op == "conv_step":
            s["x"] = r.normal(B, 2 * C, dtype=dt)[:, :C]
            s["state"] = r.normal(B, W - 1, C, dtype=dt)
            return s
        T = c["T"]
        s["x"] = r.normal(B, T, 2 * C, dtype=dt)[:, :, :C]
        s["state"] = r.normal(B, W - 1, C, dtype=dt) if c["state"] else None
        s["lens"] = r.lens(B, T) if c["ragged"] else None
        if op == "conv_train":
            s["dy"] = r.normal(B, T, C, dtype=dt)
            s["dstate_out"] = r.normal(B, W - 1, C, dtype=dt) if c["state"] else None
        return s
    B, D, N, G = c["B"], c["D"], c["N"], c["G"]
    lead = (B,) if op == "scan_step" else (B, c["T"])
    u = r.normal(*lead, D)
    s["u"] = (u * torch.sigmoid(u)).to(dt)  # what leaves the convolution
    s["delta"] = r.normal(*lead, D, std=0.5, dtype=dt)
    s["A"] = -torch.arange(1, N + 1, device=DEV, dtype=torch.float32) * torch.exp(r.normal(D, N, std=0.1))
    rank = max(1, D // 16)
    proj = r.normal(*lead, rank + 2 * G * N, dtype=dt)  # the projection to (rank | B | C)
    s["B"] = proj[..., rank:rank + G * N].unflatten(-1, (G, N))
    s["C"] = proj[..., rank + G * N:].unflatten(-1, (G, N))
    s["D"] = 1.0 + r.normal(D, std=0.1)
    step = torch.exp(r.uniform(D, lo=math.log(1e-3), hi=math.log(1e-1)))
    s["bias"] = step + torch.log(-torch.expm1(-step))  # softplus of it is `step`
    s["z"] = r.normal(*lead, 2 * D, dtype=dt)[..., D:] if c["z"] else None
    if op == "scan_step":
        s["h"] = r.normal(B, D, N, std=0.5)
        return s
    s["h0"] = r.normal(B, D, N, std=0.5) if c["h0"] else None
    s["lens"] = r.lens(B, c["T"]) if c["ragged"] else None
    if op == "scan_train":
        s["dy"] = r.normal(*lead, D, dtype=dt)
        s["dh"] = r.normal(B, D, N, std=0.5) if c["h0"] else None
    return s


# ---- one pass ------------------------------------------------------------------------------
def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _live(s, T):
    """[B, T, 1]: whether a row lies inside its sequence; None where all do."""
    n = s["lens"]
    return None if n is None else (torch.arange(T, device=n.device) < n[:, None])[:, :, None]


def _plain_add(s):
    """The residual sum as it is stored."""
    return (s["x"].float() + s["r"].float()).to(s["r"].dtype)


def _plain_norm(s):
    c = s["case"]
    sm = _plain_add(s)
    f = sm.double() if c["eight"] else sm.float()  # what falls next to a border of 8 bits is decided in 64
    y = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + 1e-6) * s["w"]
    if not c["eight"]:
        return [y.to(s["x"].dtype), sm]
    rows, dim = y.shape
    g = c["group"] or dim
    pad = torch.nn.functional.pad(y, (0, -dim % g)).unflatten(1, (-1, g))
    top = pad.abs().amax(-1).clamp_min(AMAX_FLOOR)
    q = (pad * (E4M3_MAX / top)[:, :, None]).flatten(1)[:, :dim].float().to(torch.float8_e4m3fn)
    scale = (top / E4M3_MAX).float()
    return [q, scale if c["group"] else scale[:, 0], sm]


def _plain_norm_train(s):
    sm = _plain_add(s)
    f, dy, w = sm.float(), s["dy"].float(), s["w"]
    rstd = torch.rsqrt((f * f).mean(-1, keepdim=True) + 1e-6)
    y = f * rstd * w
    wd = w * dy
    m = (wd * f).mean(-1, keepdim=True)
    ds = s["dsum"].float() + rstd * (wd - f * (rstd * rstd * m))
    dw = (dy * f * rstd).sum(0)
    return [y.to(s["x"].dtype), sm, ds.to(s["x"].dtype), ds.to(s["r"].dtype), dw]


def _silu_grad(p):
    g = torch.sigmoid(p)
    return g * (1 + p * (1 - g))


def _conv_rows(s):
    """The rows -(W-1) .. T-1 in fp32, padding rows zero."""
    c, x = s["case"], s["x"].float()
    B, T, C = x.shape
    live = _live(s, T)
    if live is not None:
        x = torch.where(live, x, torch.zeros_like(x))
    st = s["state"].float() if s["state"] is not None else x.new_zeros(B, c["W"] - 1, C)
    return torch.cat([st, x], 1), live


def _conv_pre(rows, s, T):
    W = s["case"]["W"]
    p = sum(rows[:, j:j + T] * s["w"][:, j] for j in range(W))
    return p if s["b"] is None else p + s["b"]


def _plain_conv(s):
    c = s["case"]
    T, W = c["T"], c["W"]
    rows, live = _conv_rows(s)
    p = _conv_pre(rows, s, T)
    y = p * torch.sigmoid(p) if c["act"] else p
    if live is None:
        last = rows[:, T:]
    else:
        y = torch.where(live, y, torch.zeros_like(y))
        at = s["lens"].long()[:, None] + torch.arange(W - 1, device=p.device)
        last = rows.gather(1, at[:, :, None].expand(-1, -1, c["C"]))
    return [y.to(s["x"].dtype), last.to(s["x"].dtype)]


def _plain_conv_step(s):
    c = s["case"]
    rows = torch.cat([s["state"], s["x"][:, None]], 1)
    p = (rows.float() * s["w"].t()).sum(1)
    if s["b"] is not None:
        p = p + s["b"]
    y = p * torch.sigmoid(p) if c["act"] else p
    return [y.to(s["x"].dtype), rows[:, 1:].contiguous()]


def _plain_conv_train(s):
    c, x = s["case"], s["x"]
    T, W = c["T"], c["W"]
    y, last = _plain_conv(s)
    rows, live = _conv_rows(s)
    dp = s["dy"].float()
    if c["act"]:
        dp = dp * _silu_grad(_conv_pre(rows, s, T))
    if live is not None:
        dp = torch.where(live, dp, torch.zeros_like(dp))
    drows = torch.zeros_like(rows)
    dw = []
    for j in range(W):
        drows[:, j:j + T] += dp * s["w"][:, j]
        dw.append((dp * rows[:, j:j + T]).sum((0, 1)))
    if s["dstate_out"] is not None:
        n = s["lens"].long() if live is not None else torch.full((x.shape[0],), T, device=x.device)
        at = n[:, None] + torch.arange(W - 1, device=x.device)
        drows.scatter_add_(1, at[:, :, None].expand(-1, -1, c["C"]), s["dstate_out"].float())
    out = [y, last, drows[:, W - 1:].to(x.dtype), torch.stack(dw, 1)]
    if s["b"] is not None:
        out.append(dp.sum((0, 1)))
    if s["state"] is not None:
        out.append(drows[:, :W - 1].to(x.dtype))
    return out


def _scan(a, x):
    """h_t = a_t h_{t-1} + x_t along dimension 1, by doubling the reach."""
    k, T = 1, x.shape[1]
    while k < T:
        x = torch.cat([x[:, :k], x[:, k:] + a[:, k:] * x[:, :-k]], 1)
        if 2 * k < T:
            a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return x


def _channels(m, D):
    """[B, T, G, N] to [B, T, D, N]: every channel its group's row."""
    G = m.shape[-2]
    return m.float().unsqueeze(-2).expand(*m.shape[:-1], D // G, m.shape[-1]).flatten(-3, -2) if G > 1 else m.float()


def _scan_forward(s):
    c, u = s["case"], s["u"].float()
    D, T = c["D"], c["T"]
    Bm, Cm, z = _channels(s["B"], D), _channels(s["C"], D), s["z"]
    raw = s["delta"].float() + s["bias"]
    dt = torch.nn.functional.softplus(raw)
    live = _live(s, T)
    if live is not None:  # a row past the end leaves the state as it is
        dt = torch.where(live, dt, torch.zeros_like(dt))
    a = torch.exp(dt[..., None] * s["A"])
    x = (dt * u)[..., None] * Bm
    if s["h0"] is not None:
        x[:, 0] += a[:, 0] * s["h0"]
    h = _scan(a, x)
    del x
    pre = (h * Cm).sum(-1) + s["D"] * u
    y = pre if z is None else pre * (z.float() * torch.sigmoid(z.float()))
    if live is not None:
        y = torch.where(live, y, torch.zeros_like(y))
    return y.to(s["u"].dtype), h, a, dt, raw, pre, live


def _plain_scan(s):
    y, h = _scan_forward(s)[:2]
    return [y, h[:, -1].contiguous()]


def _plain_scan_step(s):
    c, u = s["case"], s["u"].float()
    dt = torch.nn.functional.softplus(s["delta"].float() + s["bias"])
    D = c["D"]
    Bm, Cm = _channels(s["B"], D), _channels(s["C"], D)
    h = torch.exp(dt[..., None] * s["A"]) * s["h"] + (dt * u)[..., None] * Bm
    y = (h * Cm).sum(-1) + s["D"] * u
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z * torch.sigmoid(z))
    return [y.to(s["u"].dtype), h]


def _plain_scan_train(s):
    c = s["case"]
    D, G, N = c["D"], c["G"], c["N"]
    y, h, a, dt, raw, pre, live = _scan_forward(s)
    u, dy = s["u"].float(), s["dy"].float()
    if live is not None:
        dy = torch.where(live, dy, torch.zeros_like(dy))
    out = {"y": y, "h": h[:, -1].contiguous()}
    yb = dy
    if s["z"] is not None:
        z = s["z"].float()
        yb = dy * (z * torch.sigmoid(z))
        out["dz"] = (dy * pre * _silu_grad(z)).to(s["z"].dtype)
    first = s["h0"][:, None] if s["h0"] is not None else torch.zeros_like(h[:, :1])
    before = torch.cat([first, h[:, :-1]], 1)
    grouped = lambda m: m.unflatten(2, (G, D // G)).sum(3)  # noqa: E731
    out["dC"] = grouped(yb[..., None] * h).to(s["C"].dtype)
    del h
    # g_t = C_t yb_t + a_{t+1} g_{t+1}: the same recurrence from the other end
    g = yb[..., None] * _channels(s["C"], D)
    if s["dh"] is not None:
        g[:, -1] += s["dh"]
    after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    g = _scan(after.flip(1), g.flip(1)).flip(1)
    del after
    du_ = dt * u
    out["dB"] = grouped(g * du_[..., None]).to(s["B"].dtype)
    q = (g * _channels(s["B"], D)).sum(-1)
    w = g * a
    if s["h0"] is not None:
        out["dh0"] = w[:, 0].contiguous()
    w = w * before
    del g, a, before
    ddt = (w * s["A"]).sum(-1) + u * q
    dA = (w * dt[..., None]).sum((0, 1))
    ddelta = ddt * torch.sigmoid(raw)
    if live is not None:
        ddelta = torch.where(live, ddelta, torch.zeros_like(ddelta))
    out["du"] = (dt * q + s["D"] * yb).to(s["u"].dtype)
    out["ddelta"] = ddelta.to(s["delta"].dtype)
    out["dA"], out["dD"], out["ddelta_bias"] = dA, (yb * u).sum((0, 1)), ddelta.sum((0, 1))
    return out


_plain = {"norm": _plain_norm, "norm_train": _plain_norm_train, "conv": _plain_conv, "conv_step": _plain_conv_step,
          "conv_train": _plain_conv_train, "scan": _plain_scan, "scan_step": _plain_scan_step,
          "scan_train": _plain_scan_train}


# ---- the same through the package ----------------------------------------------------------
def _own_norm(s):
    import gated_delta_rule_chunkwise_gb300 as ldn
    c = s["case"]
    if not c["eight"]:
        y, sm = ldn.add_rmsnorm(s["x"], s["r"], s["w"], eps=1e-6)
        return [y, sm]
    q, scale, sm = ldn.add_rmsnorm_e4m3(s["x"], s["r"], s["w"], eps=1e-6, group=c["group"])
    return [q, scale, sm]


def _own_norm_train(s):
    import gated_delta_rule_chunkwise_gb300 as ldn
    y, sm = ldn.add_rmsnorm(s["x"], s["r"], s["w"], eps=1e-6)
    g = ldn.add_rmsnorm_backward(s["dy"], sm, s["w"], s["dsum"], eps=1e-6)
    return [y, sm, g["dx"], g["dresidual"], g["dweight"]]


def _own_conv(s):
    import gated_delta_rule_chunkwise_gb300 as ldn
    y, last = ldn.short_conv(s["x"], s["w"], s["b"], s["state"], lens=s["lens"], activation=s["case"]["act"])
    return [y, last]


def _own_conv_step(s):
    import gated_delta_rule_chunkwise_gb300 as ldn
    state = torch.empty_like(s["state"])  # not in place: every pass starts from the same state
    y = ldn.short_conv_step(s["x"], s["w"], s["b"], s["state"], state_out=state, activation=s["case"]["act"])
    return [y, state]


def _own_conv_train(s):
    import gated_delta_rule_chunkwise_gb300 as ldn
    act = s["case"]["act"]
    y, last = ldn.short_conv(s["x"], s["w"], s["b"], s["state"], lens=s["lens"], activation=act)
    g = ldn.short_conv_backward(s["x"], s["w"], s["b"], s["dy"], s["state"], s["dstate_out"], lens=s["lens"],
                                activation=act)
    out = [y, last, g["dx"], g["dweight"]]
    if s["b"] is not None:
        out.append(g["dbias"])
    if s["state"] is not None:
        out.append(g["dstate"])
    return out


def _own_scan(s):
    import gated_delta_rule_chunkwise_gb300 as ldn
    y, h = ldn.selective_scan(s["u"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"], s["bias"], s["h0"],
                              lens=s["lens"])
    return [y, h]


def _own_scan_step(s):
    import gated_delta_rule_chunkwise_gb300 as ldn
    h = torch.empty_like(s["h"])  # not in place, as above
    y = ldn.selective_scan_step(s["u"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"], s["bias"], s["h"],
                                h_out=h)
    return [y, h]


def _own_scan_train(s):
    import gated_delta_rule_chunkwise_gb300 as ldn
    y, h, states = ldn.selective_scan(s["u"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"], s["bias"], s["h0"],
                                      lens=s["lens"], save_states=True)
    g = ldn.selective_scan_backward(s["u"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"], s["bias"], states,
                                    s["dy"], s["dh"], lens=s["lens"])
    out = {"y": y, "h": h}
    for k in ("du", "ddelta", "dA", "dB", "dC", "dD", "ddelta_bias"):
        out[k] = g[k]
    if s["z"] is not None:
        out["dz"] = g["dz"]
    if s["h0"] is not None:
        out["dh0"] = g["dh0"]
    return out


_own = {"norm": _own_norm, "norm_train": _own_norm_train, "conv": _own_conv, "conv_step": _own_conv_step,
        "conv_train": _own_conv_train, "scan": _own_scan, "scan_step": _own_scan_step, "scan_train": _own_scan_train}


# ---- the least work ------------------------------------------------------------------------
def work(case):
    c, op = case, case["op"]
    e = 2 if c["dtype"] == "bf16" else 4
    if op in ("norm", "norm_train"):
        n, r = c["rows"] * c["dim"], 2 if c["res"] == "bf16" else 4
        if op == "norm":
            out = 1 if c["eight"] else e
            scales = 4 * c["rows"] * (-(-c["dim"] // c["group"]) if c["group"] else 1) if c["eight"] else 0
            return {"bytes": n * (e + 2 * r + out) + scales + 4 * c["dim"], "flops": 6 * n}
        return {"bytes": n * (e + r + r + e + e + r + e + (r if r != e else 0)) + 8 * c["dim"], "flops": 16 * n}
    if op.startswith("conv"):
        n, W = c["B"] * c.get("T", 1) * c["C"], c["W"]
        par = 4 * c["C"] * (W + (1 if c["bias"] else 0))
        st = c["B"] * (W - 1) * c["C"] * e
        if op == "conv_step":
            return {"bytes": 2 * n * e + 2 * st + par, "flops": n * (2 * W + 4)}
        if op == "conv":
            return {"bytes": 2 * n * e + (2 if c["state"] else 1) * st + par, "flops": n * (2 * W + 4)}
        return {"bytes": 4 * n * e + (4 if c["state"] else 1) * st + 2 * par, "flops": n * (6 * W + 14)}
    rows = c["B"] * c.get("T", 1)
    n, bc, state = rows * c["D"], rows * 2 * c["G"] * c["N"], c["B"] * c["D"] * c["N"] * 4
    par = 4 * c["D"] * (c["N"] + 2)
    if op == "scan_step":
        return {"bytes": e * (n * (4 if c["z"] else 3) + bc) + 2 * state + par, "flops": n * (7 * c["N"] + 12)}
    if op == "scan":
        return {"bytes": e * (n * (4 if c["z"] else 3) + bc) + state * (2 if c["h0"] else 1) + par,
                "flops": n * (7 * c["N"] + 12)}
    return {"bytes": e * (n * (8 if c["z"] else 6) + 2 * bc) + state * (4 if c["h0"] else 1) + 2 * par,
            "flops": n * (28 * c["N"] + 40)}


# ---- the definitions in 64 bits ------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    for k, v in list(s.items()):
        if torch.is_tensor(v) and v.is_floating_point() and k not in ("x", "r"):
            s[k] = v.double()
    return _exact[case["op"].split("_")[0]](s)


def _exact_norm(s):
    c = s["case"]
    # the sum is stored in the residual's type, and what is stored is what is normalised
    sm = (s["x"].double() + s["r"].double()).to(s["r"].dtype).double()
    inv = 1.0 / torch.sqrt(torch.mean(sm ** 2, dim=1) + 1e-6)
    xh = torch.einsum("rd,r->rd", sm, inv)
    y = xh * s["w"]
    if c["op"] == "norm_train":
        gy = s["dy"] * s["w"]
        dot = torch.einsum("rd,rd->r", gy, xh) / c["dim"]
        ds = s["dsum"] + (gy - xh * dot[:, None]) * inv[:, None]
        return [y, sm, ds, ds, torch.einsum("rd,rd->d", s["dy"], xh)]
    if not c["eight"]:
        return [y, sm]
    q, scale = torch.empty_like(y), []
    g = c["group"] or c["dim"]
    for at in range(0, c["dim"], g):
        part = y[:, at:at + g]
        sc = torch.maximum(part.abs().max(1).values, torch.full_like(inv, AMAX_FLOOR)) / E4M3_MAX
        v = part / sc[:, None]
        _, e = torch.frexp(v)  # |v| in [2^(e-1), 2^e): steps of 2^(e-4), of 2^-9 below 2^-6
        step = torch.exp2(torch.clamp(e.double() - 4, min=-9.0))
        q[:, at:at + g] = torch.clamp(torch.round(v / step) * step, -E4M3_MAX, E4M3_MAX)
        scale.append(sc)
    return [q, torch.stack(scale, 1) if c["group"] else scale[0], sm]


def _exact_conv(s):
    c = s["case"]
    B, C, W = c["B"], c["C"], c["W"]
    step = c["op"] == "conv_step"
    T = 1 if step else c["T"]
    x = s["x"].double().reshape(B, T, C)
    n = [T] * B if step or s["lens"] is None else [int(v) for v in s["lens"].tolist()]
    train = c["op"] == "conv_train"
    y, last = torch.zeros_like(x), torch.zeros(B, W - 1, C, dtype=torch.float64, device=DEV)
    dx, dw = torch.zeros_like(x), torch.zeros(C, W, dtype=torch.float64, device=DEV)
    db, dst = torch.zeros(C, dtype=torch.float64, device=DEV), torch.zeros_like(last)
    for b in range(B):  # one sequence at a time, no padding anywhere
        head = s["state"][b] if s["state"] is not None else torch.zeros(W - 1, C, dtype=torch.float64, device=DEV)
        seq = torch.cat([head, x[b, :n[b]]])
        last[b] = seq[n[b]:]
        if n[b] == 0:
            if train and s["dstate_out"] is not None:
                dst[b] = s["dstate_out"][b]
            continue
        win = seq.unfold(0, W, 1)  # [n, C, W]
        p = torch.einsum("tcw,cw->tc", win, s["w"])
        if s["b"] is not None:
            p = p + s["b"]
        sig = 1.0 / (1.0 + torch.exp(-p))
        y[b, :n[b]] = p * sig if c["act"] else p
        if not train:
            continue
        dp = s["dy"][b, :n[b]]
        if c["act"]:
            dp = dp * (sig + p * sig * (1.0 - sig))
        dw += torch.einsum("tc,tcw->cw", dp, win)
        db += dp.sum(0)
        dseq = torch.zeros_like(seq)
        for i in range(W):
            dseq[i:i + n[b]] += dp * s["w"][:, i]
        if s["dstate_out"] is not None:
            dseq[n[b]:] += s["dstate_out"][b]
        dst[b], dx[b, :n[b]] = dseq[:W - 1], dseq[W - 1:]
    if step:
        return [y[:, 0], last]
    out = [y, last]
    if train:
        out += [dx, dw]
        if s["b"] is not None:
            out.append(db)
        if s["state"] is not None:
            out.append(dst)
    return out


def _exact_scan(s):
    """Token by token."""
    c = s["case"]
    B, D, N, G = c["B"], c["D"], c["N"], c["G"]
    step = c["op"] == "scan_step"
    T = 1 if step else c["T"]
    if T * (3 if c["op"] == "scan_train" else 1) * max(B * D * N / 1e6, 0.25) > 150000:
        return None
    f = lambda m: m.unsqueeze(1) if step else m  # noqa: E731
    u, raw, Bm, Cm = f(s["u"]), f(s["delta"]) + s["bias"], f(s["B"]), f(s["C"])
    z = None if s["z"] is None else f(s["z"])
    dt = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    per = D // G
    wide = lambda m, t: m[:, t].repeat_interleave(per, dim=1)  # noqa: E731  [B, D, N]
    n = torch.full((B,), T, device=DEV) if step or s["lens"] is None else s["lens"]
    h = s["h"] if step else s["h0"] if s["h0"] is not None else torch.zeros(B, D, N, dtype=torch.float64, device=DEV)
    train = c["op"] == "scan_train"
    hs, pre = [h], torch.zeros(B, T, D, dtype=torch.float64, device=DEV)
    for t in range(T):
        new = torch.exp(dt[:, t, :, None] * s["A"]) * h + (dt[:, t] * u[:, t])[:, :, None] * wide(Bm, t)
        h = torch.where((t < n)[:, None, None], new, h)
        pre[:, t] = torch.einsum("bdn,bdn->bd", h, wide(Cm, t)) + s["D"] * u[:, t]
        if train:
            hs.append(h)
    on = (torch.arange(T, device=DEV)[None] < n[:, None])[:, :, None].double()
    sz = 1.0 if z is None else z / (1.0 + torch.exp(-z))
    y = pre * sz * on
    if step:
        return [y[:, 0], h]
    if not train:
        return [y, h]
    dy = s["dy"] * on
    yb = dy * sz
    g = s["dh"].clone() if s["dh"] is not None else torch.zeros_like(h)
    out = {"y": y, "h": h}
    du, ddelta = torch.zeros_like(pre), torch.zeros_like(pre)
    dB, dC = torch.zeros(B, T, G, N, dtype=torch.float64, device=DEV), torch.zeros(B, T, G, N, dtype=torch.float64,
                                                                                    device=DEV)
    dA = torch.zeros(D, N, dtype=torch.float64, device=DEV)
    for t in reversed(range(T)):
        m = on[:, t, :, None]
        gt = (g + yb[:, t, :, None] * wide(Cm, t)) * m
        dC[:, t] = (yb[:, t, :, None] * hs[t + 1]).reshape(B, G, per, N).sum(2)
        dB[:, t] = (gt * (dt[:, t] * u[:, t])[:, :, None]).reshape(B, G, per, N).sum(2)
        decayed = gt * torch.exp(dt[:, t, :, None] * s["A"])
        hit = decayed * hs[t]
        along = torch.einsum("bdn,bdn->bd", gt, wide(Bm, t))
        dA += torch.einsum("bdn,bd->dn", hit, dt[:, t])
        ddelta[:, t] = ((hit * s["A"]).sum(-1) + along * u[:, t]) / (1.0 + torch.exp(-raw[:, t]))
        du[:, t] = along * dt[:, t] + s["D"] * yb[:, t]
        g = decayed + g * (1 - m)
    out |= {"du": du, "ddelta": ddelta, "dA": dA, "dB": dB, "dC": dC, "dD": torch.einsum("btd,btd->d", yb, u),
            "ddelta_bias": ddelta.sum((0, 1))}
    if z is not None:
        sig = 1.0 / (1.0 + torch.exp(-z))
        out["dz"] = dy * pre * (sig + z * sig * (1.0 - sig))
    if s["h0"] is not None:
        out["dh0"] = g
    return out


_exact = {"norm": _exact_norm, "conv": _exact_conv, "scan": _exact_scan}
