"""Calls of the operators around a token mixer that their documentation allows and that are easy
to miss: outputs at any element's address, sequences and channel counts near the largest int,
several threads, streams and saved tensors, sizes at which a block walks many rows or tokens."""
import numpy as np
import pytest

import gated_delta_rule_chunkwise_gb300 as ldn
from tests import _mixer_ref as ref
from tests.test_mixer_parity import _t, dev, host, rounded, scan_inputs, scan_tensors, within  # noqa: F401

pytestmark = pytest.mark.gpu
U = ref.U


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_chunkwise_gb300 import build
    build.build()
    ldn.load()


def ptr(t):
    return None if t is None else t.data_ptr()


# ---- outputs of the scan's gradient at any element's address ----
def backward_into(t, states, dy, dh, g, dtype, softplus=True):
    """ldn_ssm_backward into the given tensors."""
    import torch
    u, dl, A, Bm, Cm, Ds, z, bias = t
    B, T, D = u.shape
    G, N = Bm.shape[2:]
    need = ldn.ldn_ssm_backward_workspace_size(B, T, D, N, G)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    ld = lambda m, w: w if m is None else m.stride(1)  # noqa: E731
    st = ldn.ldn_ssm_backward(ptr(u), ld(u, D), ptr(dl), ld(dl, D), ptr(A), ptr(Bm), ld(Bm, G * N), ptr(Cm),
                              ld(Cm, G * N), ptr(Ds), ptr(z), ld(z, D), ptr(bias), ptr(states), None, ptr(dy), ptr(dh),
                              ptr(g["du"]), ptr(g["ddelta"]), ptr(g["dA"]), ptr(g["dB"]), ptr(g["dC"]), ptr(g["dD"]),
                              ptr(g["dz"]), ptr(g["ddelta_bias"]), ptr(g["dh0"]), B, T, D, N, G, int(softplus),
                              ldn.LDN_F32 if dtype == "f32" else ldn.LDN_BF16, ptr(ws), need,
                              torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    return st


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shifted", ["du", "ddelta", "dz", "dB", "dC", "dA", "dD", "ddelta_bias"])
def test_scan_gradients_at_any_address(dtype, shifted):
    """Aligned inputs, one output a slice that starts at an odd element: the same values bit for
    bit, and nothing written around the slice."""
    import torch
    p = scan_inputs(2, 70, 32, 16, 2, dtype)
    t = scan_tensors(p, [70, 70], dtype)
    h0 = dev(p["h0"])
    states = ldn.selective_scan(*t, h0, save_states=True)[2]
    r = np.random.default_rng(8)
    dy, dh = dev(r.normal(size=(2, 70, 32)), dtype), dev(r.normal(size=(2, 32, 16)))
    want = ldn.selective_scan_backward(*t, states, dy, dh)
    got, edges = {}, {}
    for k, w in want.items():
        off = 1 if k == shifted else 0
        flat = torch.full((w.numel() + 16,), 7.0, dtype=w.dtype, device="cuda")
        got[k], edges[k] = flat[off:off + w.numel()].view(w.shape), (flat[:off], flat[off + w.numel():])
    assert backward_into(t, states, dy, dh, got, dtype) == ldn.LDN_OK
    for k, w in want.items():
        assert torch.equal(got[k], w), k
        assert all((e == 7.0).all() for e in edges[k]), k


# ---- sizes near the largest int ----
def room(gb):
    """Skips where the GPU has not that many GB free."""
    import torch
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gb * 1e9:
        pytest.skip(f"needs {gb} GB of free GPU memory")


@pytest.mark.parametrize("dtype,T", [("f32", 1 << 29), ("bf16", 1 << 30)])
def test_rows_behind_the_end_of_a_very_long_sequence(dtype, T):
    """One channel, unsplit, five rows of 2^29 or 2^30: the vectors of the rows behind them, four
    or two a row, are more than an int counts, and all are zeroed."""
    import torch
    room(30)
    try:
        x = torch.empty(1, T, 1, dtype=_t(dtype), device="cuda")
        x[:, :5] = 0.5
        m = torch.empty(1, T, 1, 8, dtype=_t(dtype), device="cuda")
        m[:, :5] = 0.25
        y = torch.full((1, T, 1), 7.0, dtype=_t(dtype), device="cuda")
        A = -torch.ones(1, 8, device="cuda")
        none = torch.empty(0, dtype=torch.uint8, device="cuda")
        lens = torch.tensor([5], dtype=torch.int32, device="cuda")
        _, h = ldn.selective_scan(x, x, A, m, m, lens=lens, out=y, workspace=none)
        cut = lambda v: v[:, :5].contiguous()  # noqa: E731
        y5, h5 = ldn.selective_scan(cut(x), cut(x), A, cut(m), cut(m), workspace=none)
        assert torch.equal(y[:, :5], y5) and torch.equal(h, h5)
        assert torch.count_nonzero(y[:, 5:]).item() == 0
    finally:
        x = m = y = None
        torch.cuda.empty_cache()


@pytest.mark.parametrize("more", [8, 9])
def test_conv_step_of_very_many_channels(more):
    """8 x (2^28 + 8 or 9) taps are more than an int counts: the first and the last channels against
    the formula."""
    import torch
    room(30)
    C, W = (1 << 28) + more, 8
    try:
        f = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda").normal_()  # noqa: E731
        x, state, w = f(1, C), f(1, W - 1, C), torch.empty(C, W, device="cuda").normal_()
        y = ldn.short_conv_step(x, w, None, state, activation=False, state_out=torch.empty_like(state))
        for part in (slice(0, 64), slice(C - 64, C)):
            seq = np.concatenate([host(state[0, :, part]), host(x[:, part])])
            terms = seq.T * host(w[part])
            want = terms.sum(1)
            within(y[0, part], want, np.abs(want) * ref.HALF["bf16"] + np.abs(terms).sum(1) * W * U, "y")
    finally:
        x = state = w = y = None
        torch.cuda.empty_cache()


def test_scan_step_of_very_many_groups():
    """2^28 + 4 groups of one channel and eight states: a group's place in a row of B or C is past
    an int in the last ones."""
    import torch
    room(60)
    D, N = (1 << 28) + 4, 8
    try:
        u = torch.empty(1, D, dtype=torch.bfloat16, device="cuda").uniform_(0.5, 1)
        m = torch.empty(1, D, N, dtype=torch.bfloat16, device="cuda").uniform_(0.5, 1)
        h = torch.zeros(1, D, N, device="cuda")
        A = torch.zeros(D, N, device="cuda")     # nothing decays: h = dt u B, y = sum C h, all terms positive
        y = ldn.selective_scan_step(u, u, A, m, m, None, None, None, h, delta_softplus=False)
        for part in (slice(0, 64), slice(D - 64, D)):
            uu, mm = host(u[0, part]), host(m[0, part])
            hh = (uu * uu)[:, None] * mm
            within(h[0, part], hh, hh * 4 * U, "h")
            want = (hh * mm).sum(1)
            within(y[0, part], want, want * (ref.HALF["bf16"] + (N + 8) * U), "y")
    finally:
        u = m = h = A = y = None
        torch.cuda.empty_cache()


# ---- a workspace that is too small ----
def test_scan_with_a_small_workspace_beside_its_outputs():
    """A workspace smaller than the segments need is not used, so what lies behind it may be an
    output: results as without one, the workspace untouched."""
    import torch
    p = scan_inputs(1, 600, 20, 16, 1, "f32")
    t = scan_tensors(p, [600], "f32")
    h0 = dev(p["h0"])
    need = ldn.ldn_ssm_scan_workspace_size(1, 600, 20, 16, 1)
    assert need > 256
    n, nh = 600 * 20, 20 * 16
    arena = torch.full((64 + n + nh,), 7.0, device="cuda")
    small, y, h = arena[:64].view(torch.uint8), arena[64:64 + n].view(1, 600, 20), arena[64 + n:].view(1, 20, 16)
    assert small.numel() < need
    ldn.selective_scan(*t, h0, out=y, h_final=h, workspace=small)
    want = ldn.selective_scan(*t, h0, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert torch.equal(y, want[0]) and torch.equal(h, want[1]) and (arena[:64] == 7.0).all()
    # one that is large enough is used, and may not be shared with an output
    with pytest.raises(ldn.LdnError):
        ldn.selective_scan(*t, h0, out=y, h_final=h, workspace=arena.view(torch.uint8))


# ---- rows past a sequence's end ----
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [8, 16, 32, 64])
def test_scan_gradients_past_the_end_are_zero_whatever_the_state(dtype, N):
    """A NaN in one token's input makes a channel's state NaN from there on; the gradients of the
    rows past the sequence's end stay zero, and those before the token are what they are."""
    import torch
    n = [37, 64]
    p = scan_inputs(2, 70, 24, N, 2, dtype)
    t, gl = scan_tensors(p, n, dtype), dev(np.array(n))
    t[0][0, 30, 5] = float("nan")
    dy = dev(np.random.default_rng(1).normal(size=(2, 70, 24)), dtype)
    states = ldn.selective_scan(*t, dev(p["h0"]), lens=gl, save_states=True)[2]
    g = ldn.selective_scan_backward(*t, states, dy, None, lens=gl)
    for k in ("du", "ddelta", "dz", "dB", "dC"):
        for i in range(2):
            assert (g[k][i, n[i]:] == 0).all(), k
    assert torch.isnan(g["dC"][0, 30:37, 0]).all() and torch.isfinite(g["dC"][0, :30]).all()
    assert torch.isfinite(g["dC"][:, :, 1]).all() and all(torch.isfinite(g[k][1]).all() for k in ("du", "dB", "dC"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C,W", [(8, 4), (7, 3), (12, 8)])
def test_conv_gradients_of_a_padded_batch_are_those_without_padding(dtype, C, W):
    """Infinite inputs at a sequence's end and an infinite weight: the gradients of a padded batch
    are the same as of the sequence alone, and zero past its end."""
    import torch
    r = np.random.default_rng(W)
    n, T = 21, 40
    x, dy = dev(r.normal(size=(1, T, C)), dtype), dev(r.normal(size=(1, T, C)), dtype)
    w = dev(r.normal(size=(C, W)))
    x[0, n - 1, 2] = float("inf")
    w[5, 1] = float("inf")
    for act in (False, True):
        g = ldn.short_conv_backward(x, w, None, dy, lens=torch.tensor([n], dtype=torch.int32, device="cuda"),
                                    activation=act)
        cut = lambda m: m[:, :n].contiguous()  # noqa: E731
        want = ldn.short_conv_backward(cut(x), w, None, cut(dy), activation=act)
        assert (g["dx"][0, n:] == 0).all()
        same = lambda a, b: bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())  # noqa: E731
        assert same(g["dx"][:, :n], want["dx"])
        # the tokens of one sequence may be cut into other runs: sums to rounding, infinities and NaN alike
        a, b = host(g["dweight"]), host(want["dweight"])
        assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(np.isinf(a), np.isinf(b))
        # |silu'| <= 1.1, |x| < 5, n roundings on either side
        mag = np.broadcast_to((np.abs(host(dy[0, :n])) * 1.1).sum(0)[:, None] * 5, a.shape)
        ok = np.isfinite(b)
        assert (np.abs(a[ok] - b[ok]) <= mag[ok] * 2 * n * U).all()
        if not act:
            assert np.isinf(b[2]).any()


# ---- several host threads ----
def test_wide_norm_gradients_from_several_threads():
    """The C entry points are re-entrant: threads that call the gradient of rows of different
    widths at once (ctypes gives up the interpreter's lock) all get what a call alone gives."""
    import threading

    import torch
    rows = 3
    calls = []
    for D in (32768, 8200, 20000, 9001):
        g = torch.Generator(device="cuda").manual_seed(D)
        f = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        dy, s, w, s_ = f(rows, D), f(rows, D), f(D), torch.cuda.Stream()
        need = ldn.ldn_add_rmsnorm_backward_workspace_size(rows, D)
        dx, dw, ws = torch.empty_like(dy), torch.empty_like(w), torch.empty(need, dtype=torch.uint8, device="cuda")
        want = ldn.add_rmsnorm_backward(dy, s, w)
        calls.append((want, dx, dw, (ptr(dy), ptr(s), ptr(w), None, ptr(dx), None, ptr(dw), rows, D, ldn.LDN_F32,
                                     ldn.LDN_F32, 1e-6, ptr(ws), need, s_.cuda_stream), (dy, s, w, s_, ws)))
    torch.cuda.synchronize()
    start, failed = threading.Barrier(len(calls)), []

    def work(args):
        start.wait()
        for _ in range(1500):
            st = ldn.ldn_add_rmsnorm_backward(*args)
            if st != ldn.LDN_OK:
                failed.append((args[8], st))
                return

    threads = [threading.Thread(target=work, args=(c[3],)) for c in calls]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not failed
    for want, dx, dw, _, _ in calls:
        assert torch.equal(dx, want["dx"]) and torch.equal(dw, want["dweight"])


# ---- gradients and saved tensors ----
def test_calls_that_record_no_gradient_warn():
    """Where an argument requires a gradient and a graph is recorded, the call without one says
    so at the caller's line; autograd's forms, no_grad and plain tensors are quiet."""
    import warnings

    import torch
    from gated_delta_rule_chunkwise_gb300 import autograd as ag
    x = torch.randn(2, 9, 16, device="cuda")
    w, taps = torch.ones(16, device="cuda"), torch.ones(16, 4, device="cuda", requires_grad=True)
    A, m = -torch.ones(16, 8, device="cuda"), torch.randn(2, 9, 1, 8, device="cuda")
    wp, Ap = w.clone().requires_grad_(), A.clone().requires_grad_()
    calls = {"add_rmsnorm": lambda f: f.add_rmsnorm(x, x, wp), "short_conv": lambda f: f.short_conv(x, taps),
             "selective_scan": lambda f: f.selective_scan(x, x, Ap, m, m)}
    for name, f in calls.items():
        with pytest.warns(UserWarning, match=f"autograd.{name}") as got:
            y = f(ldn)[0]
        assert len(got) == 1 and got[0].filename == __file__ and not y.requires_grad
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            assert f(ag)[0].requires_grad
            with torch.no_grad():
                assert torch.equal(f(ldn)[0], y)
    with pytest.warns(UserWarning, match="add_rmsnorm_e4m3"):
        ldn.add_rmsnorm_e4m3(x, x, wp)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        ldn.add_rmsnorm(x, x, w)
        with pytest.raises(UserWarning):        # as an exception it ends the call
            ldn.add_rmsnorm(x, x, wp)


def test_writing_into_a_saved_tensor_is_noticed():
    """A tensor that a graph has saved and a later call writes (its sum in place, a state, an
    output): the backward pass refuses, as after torch's own in-place operations."""
    import torch
    from gated_delta_rule_chunkwise_gb300 import autograd as ag
    x, w = torch.randn(4, 64, device="cuda"), torch.ones(64, device="cuda", requires_grad=True)
    taps = torch.randn(64, 4, device="cuda", requires_grad=True)
    A, m = -torch.ones(64, 8, device="cuda"), torch.randn(1, 4, 1, 8, device="cuda")
    other = torch.randn(4, 64, device="cuda")
    state, h = torch.randn(1, 3, 64, device="cuda"), torch.randn(1, 64, 8, device="cuda")

    def norm(write):
        y, s = ag.add_rmsnorm(x, other, w)
        if write:
            ldn.add_rmsnorm(x, s.detach(), w.detach(), residual_out=s.detach())
        return y

    def conv(write, how):
        st = state.clone()
        y, _ = ag.short_conv(other[None], taps, None, st)
        if write:
            how(st)
        return y

    def plain(write, how):      # torch's own graph
        hh = h.clone()
        y = (hh * torch.ones_like(h).requires_grad_()).sum()
        if write:
            how(hh)
        return y

    c = taps.detach()
    ways = [lambda write: norm(write),
            lambda write: conv(write, lambda st: ldn.short_conv(x[None], c, None, st, state_out=st)),
            lambda write: conv(write, lambda st: ldn.short_conv_step(x[:1], c, None, st)),
            lambda write: conv(write, lambda st: ldn.short_conv_step(x[:1], c, None, st.clone(), state_out=st)),
            lambda write: plain(write, lambda hh: ldn.selective_scan_step(x[:1], x[:1], A, m[:, 0], m[:, 0], None, None,
                                                                          None, hh)),
            lambda write: plain(write, lambda hh: ldn.selective_scan(x[None], x[None], A, m, m, h_final=hh))]
    for f in ways:
        f(False).sum().backward()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            f(True).sum().backward()
    with torch.inference_mode():        # such tensors have no versions
        st = torch.randn(1, 3, 64, device="cuda")
    before = st.clone()
    ldn.short_conv_step(x[:1], c, None, st)
    assert not torch.equal(st, before)


def test_negated_views_are_refused():
    """The imaginary part of a conjugate is a view whose memory holds the other sign."""
    import torch
    z = torch.randn(2, 9, 16, dtype=torch.complex64, device="cuda")
    neg = z.conj().imag
    assert neg.is_neg()
    w, taps, plain = torch.ones(16, device="cuda"), torch.ones(16, 4, device="cuda"), torch.randn(2, 9, 16, device="cuda")
    A, m = -torch.ones(16, 8, device="cuda"), torch.randn(2, 9, 1, 8, device="cuda")
    same = torch._neg_view(plain)
    for bad in (neg, same):
        for f in (lambda: ldn.add_rmsnorm(plain, bad, w), lambda: ldn.add_rmsnorm(bad, None, w),
                  lambda: ldn.short_conv(bad, taps), lambda: ldn.selective_scan(plain, bad, A, m, m),
                  lambda: ldn.short_conv(plain, taps, out=bad)):
            with pytest.raises(ValueError):
                f()
    with pytest.raises(ValueError, match="negated"):
        ldn.short_conv(same, taps)


# ---- memory on another stream ----
def test_arguments_freed_after_a_call_on_another_stream():
    """Arguments that are dropped right after a call with stream=, while that stream is still
    busy: tensors made next do not get their memory before the call has run."""
    import torch
    n = 1 << 22
    side = torch.cuda.Stream()
    x = torch.randn(n // 64, 64, device="cuda")
    w, taps = torch.randn(64, device="cuda"), torch.randn(64, 4, device="cuda")
    want_y, want_s = ldn.add_rmsnorm(x, x, w)
    want_c = ldn.short_conv(x[None], taps)[0]
    torch.cuda.synchronize()
    for call in (lambda a: ldn.add_rmsnorm(a, a, w, stream=side), lambda a: ldn.short_conv(a[None], taps, stream=side)):
        a = x.clone()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)      # about 0.1 s
        got = call(a)
        del a
        over = [torch.full((n // 64, 64), float("nan"), device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        del over
        if got[0].dim() == 2:
            assert torch.equal(got[0], want_y) and torch.equal(got[1], want_s)
        else:
            assert torch.equal(got[0], want_c)


# ---- e4m3 next to a border ----
def settled_e4m3(s, w, group):
    """What 448 |s w| / max |s w| is in e4m3: the quotient in 64 bits, stored in fp32, rounded to
    nearest even; and the quotient."""
    rows, D = s.shape
    p, g = s * w, group or D
    n = -(-D // g)
    pad = np.zeros((rows, n * g))
    pad[:, :D] = np.abs(p)
    top = np.repeat(pad.reshape(rows, n, g).max(-1), g, axis=1)[:, :D]
    v = (p * (448.0 / top)).astype(np.float32).astype(np.float64)
    return ref.e4m3(v), v


@pytest.mark.parametrize("D", [2048, 1001, 4096, 5001, 9008, 9001, 20000, 20001])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_e4m3_borders_are_decided_as_in_64_bits(D, group, dtype, res):
    """No value falls to the other side of the middle of two e4m3 numbers than in 64 bits, and what
    is in the middle goes to the even one: weights drawn, and equal ones, whose quotients of two
    short numbers are often in the middle."""
    import torch
    r = np.random.default_rng(D + group)
    rows = max(300, 3_000_000 // D)
    x, rr = r.normal(size=(rows, D)), 3 * r.normal(size=(rows, D))
    # rows on a grid of a sixteenth have many values in the middle in fp32 too
    x[::2], rr[::2] = np.round(x[::2] * 16) / 16, np.round(rr[::2] * 16) / 16
    gx, gr = dev(x, dtype), dev(rr, res)
    for w in (rounded(1 + 0.1 * r.normal(size=D), "f32"), np.ones(D), np.full(D, -0.75)):
        q, scale, s = ldn.add_rmsnorm_e4m3(gx, gr, dev(w), group=group)
        want, v = settled_e4m3(host(s), w, group)
        normal = np.abs(v) >= 2.0 ** -6             # below, borders stay with fp32
        got = host(q)
        assert np.array_equal(got[normal], want[normal]), (got != want)[normal].sum()
        assert (np.abs(got - v)[~normal] <= 2.0 ** -10 + 2.0 ** -26).all()
        again = ldn.add_rmsnorm_e4m3(gx, gr, dev(w), group=group)
        assert torch.equal(q.view(torch.uint8), again[0].view(torch.uint8)) and torch.equal(scale, again[1])


@pytest.mark.parametrize("group", [0, 128])
def test_e4m3_of_rows_that_are_not_ordinary(group):
    """Groups below the least magnitude, zeros, infinite and NaN rows among ordinary ones."""
    import torch
    r = np.random.default_rng(5)
    x = dev(r.normal(size=(6, 256)))
    w = torch.ones(256, device="cuda")
    tiny = w * 1e-33
    q, scale, _ = ldn.add_rmsnorm_e4m3(x, None, tiny, group=group)
    assert torch.equal(scale, torch.full_like(scale, 2.0 ** -100 / 448))
    y = ref.norm(host(x), host(tiny), 1e-6) * 448 * 2.0 ** 100
    within(q, y, np.maximum(np.abs(y) * 2.0 ** -4, 2.0 ** -10) + np.abs(y) * 40 * U, "tiny")
    x[1], x[2, 7], x[3, 200], x[4] = 0, float("nan"), float("inf"), 3e-20
    q, scale, _ = ldn.add_rmsnorm_e4m3(x, None, w, group=group)
    f = q.float()
    assert (f[1] == 0).all() and torch.isnan(f[2]).all() and torch.isnan(f[3, 200]) and torch.isfinite(f[3, :200]).all()
    # |y| = 3e-17 in every channel of row 4
    assert (f[4] == 448).all() and torch.isfinite(scale[[0, 1, 4, 5]]).all()
    # without a residual the type of one does not matter
    b = dev(host(x), "bf16")
    want = ldn.add_rmsnorm_e4m3(b, None, w, group=group)
    out, sc = torch.empty_like(want[0]), torch.empty_like(want[1])
    st = ldn.ldn_add_rmsnorm_e4m3(ptr(b), None, ptr(w), ptr(out), ptr(sc), None, 6, 256, group, ldn.LDN_BF16, ldn.LDN_F32,
                                  1e-6, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == ldn.LDN_OK and torch.equal(out.view(torch.uint8), want[0].view(torch.uint8))
    assert torch.equal(sc, want[1])
