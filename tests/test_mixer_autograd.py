"""The torch.autograd binding of the operators around a token mixer: gradients through
``loss.backward()`` equal the library's gradients of the same inputs, and a chain of the
three agrees with torch's own differentiation of the formulas in 64 bits."""
import numpy as np
import pytest

import gated_delta_rule_chunkwise_gb300 as ldn
from tests.test_mixer_parity import conv_inputs, dev, norm_inputs, rounded, scan_inputs, scan_tensors

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_chunkwise_gb300 import build
    build.build()
    ldn.load()


def leaf(t):
    return None if t is None else t.detach().clone().requires_grad_()


def test_add_rmsnorm_gradients():
    import torch
    from gated_delta_rule_chunkwise_gb300 import autograd as ag
    x, r, w = norm_inputs(6, 72, "bf16", "f32")
    a, b, c = leaf(dev(x, "bf16")), leaf(dev(r)), leaf(dev(w))
    dy, ds = torch.randn_like(a), torch.randn_like(b)
    y, s = ag.add_rmsnorm(a, b, c)
    torch.autograd.backward([y, s], [dy, ds])
    g = ldn.add_rmsnorm_backward(dy, s.detach(), c.detach(), ds)
    assert torch.equal(a.grad, g["dx"]) and torch.equal(b.grad, g["dresidual"]) and torch.equal(c.grad, g["dweight"])
    # the sum alone, and no residual at all
    a, b = leaf(a), leaf(b)
    ag.add_rmsnorm(a, b, c)[1].backward(ds)
    assert torch.equal(b.grad, ds) and torch.equal(a.grad, ds.bfloat16())
    a, c = leaf(a), leaf(c)
    y, s = ag.add_rmsnorm(a, None, c)
    assert s is a
    y.backward(dy)
    g = ldn.add_rmsnorm_backward(dy, a.detach(), c.detach())
    assert torch.equal(a.grad, g["dx"]) and torch.equal(c.grad, g["dweight"])


def test_short_conv_gradients():
    import torch
    from gated_delta_rule_chunkwise_gb300 import autograd as ag
    p = conv_inputs(2, 21, 40, 4, "bf16", True, True)
    x, w, b, st = (leaf(dev(p[k], d)) for k, d in (("x", "bf16"), ("w", "f32"), ("b", "f32"), ("state", "bf16")))
    lens = torch.tensor([21, 9], dtype=torch.int32, device="cuda")
    y, last = ag.short_conv(x, w, b, st, lens=lens)
    dy, dl = torch.randn_like(y), torch.randn_like(last)
    torch.autograd.backward([y, last], [dy, dl])
    g = ldn.short_conv_backward(x.detach(), w.detach(), b.detach(), dy, st.detach(), dl, lens=lens)
    for t, k in ((x, "dx"), (w, "dweight"), (b, "dbias"), (st, "dstate")):
        assert torch.equal(t.grad, g[k]), k


@pytest.mark.parametrize("whole", [True, False])
def test_selective_scan_gradients(whole):
    import torch
    from gated_delta_rule_chunkwise_gb300 import autograd as ag
    opts = {} if whole else dict(z=False, skip=False, bias=False, h0=False)
    p = scan_inputs(2, 50, 24, 16, 2, "bf16", **opts)
    t = [leaf(m) for m in (*scan_tensors(p, [50, 50], "bf16"), dev(p["h0"]))]
    y, h = ag.selective_scan(*t)
    dy, dh = torch.randn_like(y), torch.randn_like(h)
    torch.autograd.backward([y, h] if whole else [y], [dy, dh] if whole else [dy])
    d = [None if m is None else m.detach() for m in t]
    states = ldn.selective_scan(*d, save_states=True)[2]
    g = ldn.selective_scan_backward(*d[:8], states, dy, dh if whole else None)
    for m, k in zip(t, ("du", "ddelta", "dA", "dB", "dC", "dD", "dz", "ddelta_bias", "dh0")):
        if m is not None:
            assert torch.equal(m.grad, g[k]), k


def test_gradients_of_gradients_are_refused():
    import torch
    from gated_delta_rule_chunkwise_gb300 import autograd as ag
    x = torch.randn(2, 9, 16, device="cuda", requires_grad=True)
    w, taps = torch.ones(16, device="cuda"), torch.ones(16, 4, device="cuda")
    A, Bm = -torch.ones(16, 8, device="cuda"), torch.randn(2, 9, 1, 8, device="cuda")
    for f in (lambda: ag.add_rmsnorm(x, x.detach(), w)[0], lambda: ag.short_conv(x, taps)[0],
              lambda: ag.selective_scan(x, x, A, Bm, Bm)[0]):
        g, = torch.autograd.grad((f() ** 2).sum(), x, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            g.sum().backward()


def test_a_block_trains():
    """Gradients of every parameter of norm -> convolution -> scan in fp32 against torch's
    differentiation of the same formulas in 64 bits."""
    import torch
    from gated_delta_rule_chunkwise_gb300 import autograd as ag
    r = np.random.default_rng(5)
    B, T, D, N, W, R = 2, 45, 24, 8, 4, 5
    f = lambda *s, k=1.0: rounded(r.normal(size=s) * k, "f32")  # noqa: E731
    raw = dict(x=f(B, T, D), r=f(B, T, D), nw=1 + f(D, k=0.1), cw=f(D, W, k=0.5), cb=f(D, k=0.1),
               wx=f(R + 2 * N, D, k=D ** -0.5), wdt=f(D, R, k=R ** -0.5), A=-np.exp(f(D, N, k=0.5)), Ds=f(D),
               bias=f(D, k=0.5) - 2, wz=f(D, D, k=D ** -0.5))
    raw = {k: rounded(v, "f32") for k, v in raw.items()}
    dy = f(B, T, D)

    def split(db):
        return db[..., :R], db[..., R:R + N].unflatten(-1, (1, N)), db[..., R + N:].unflatten(-1, (1, N))

    def plain(p):
        s = p["x"] + p["r"]
        n = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + 1e-6) * p["nw"]
        pad = torch.cat([n.new_zeros(B, W - 1, D), n], 1)
        c = torch.nn.functional.silu(sum(pad[:, j:j + T] * p["cw"][:, j] for j in range(W)) + p["cb"])
        d, Bm, Cm = split(c @ p["wx"].t())
        dt = torch.nn.functional.softplus(d @ p["wdt"].t() + p["bias"])
        h, ys = n.new_zeros(B, D, N), []
        for t in range(T):
            h = torch.exp(dt[:, t, :, None] * p["A"]) * h + (dt[:, t] * c[:, t])[..., None] * Bm[:, t]
            ys.append((h * Cm[:, t]).sum(-1) + p["Ds"] * c[:, t])
        return torch.stack(ys, 1) * torch.nn.functional.silu(n @ p["wz"].t()) + s

    def ours(p):
        n, s = ag.add_rmsnorm(p["x"], p["r"], p["nw"])
        c, _ = ag.short_conv(n, p["cw"], p["cb"])
        d, Bm, Cm = split(c @ p["wx"].t())
        y, _ = ag.selective_scan(c, d @ p["wdt"].t(), p["A"], Bm, Cm, p["Ds"], n @ p["wz"].t(), p["bias"])
        return y + s

    torch.backends.cuda.matmul.allow_tf32 = False
    g = {}
    for name, fn, dt in (("want", plain, torch.float64), ("got", ours, torch.float32)):
        p = {k: torch.from_numpy(v).to("cuda", dt).requires_grad_() for k, v in raw.items()}
        fn(p).backward(torch.from_numpy(dy).to("cuda", dt))
        g[name] = {k: v.grad.double() for k, v in p.items()}
    # five stages each way in fp32, sums of at most B T = 90 terms, magnitudes of a few times a
    # gradient's largest value (cancellation in the sums over tokens): 10 x 100 x 16 roundings
    for k in raw:
        off = (g["got"][k] - g["want"][k]).abs().max() / g["want"][k].abs().max()
        assert off <= 16000 * 2.0 ** -24, (k, float(off))
