"""Norms of queries and keys with the rotation, and their gradients, against their formulas in 64 bits.

The tolerances are the bounds of tests/norm_ref.py: FP32 arithmetic, one rounding of what is stored."""
import numpy as np
import pytest
import torch

import sparse_attention_indexer_dsa_gb300 as dsa
from tests import norm_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def host(t):
    return t.detach().double().cpu().numpy()


def close(got, want, tol, what):
    got = host(got) if torch.is_tensor(got) else got
    assert np.isfinite(got).all(), what
    over = np.abs(got - want) - tol
    assert (over <= 0).all(), (what, np.unravel_index(over.argmax(), over.shape), float(over.max()))


def inputs(rng, T, H, Hk, D, src, norm, wt="f32", strided=True, std=1.0, far=1 << 20):
    x = rng.standard_normal((T, H + Hk, D)) * std
    x[rng.random(x.shape) < 0.02] *= 9.0
    x = torch.from_numpy(x).cuda().to(DT[src])
    q, k = (x[:, :H], x[:, H:]) if strided else (x[:, :H].contiguous(), x[:, H:].contiguous())
    def row(m, s):
        return (m + s * torch.from_numpy(rng.standard_normal(D))).cuda().to(DT[wt])
    w = [row(1.0, 0.2), row(1.0, 0.2)] + ([row(0.0, 0.2), row(0.0, 0.2)] if norm == "layer" else [None, None])
    pos = torch.from_numpy(rng.integers(0, far, T).astype(np.int32)).cuda()
    return q, k, pos, w


def check_forward(q, k, pos, w, got, norm, rope_dim, inter, out, **kw):
    for x, y, wi, bi, what in ((q, got[0], w[0], w[2], "q"), (k, got[1], w[1], w[3], "k")):
        if x is None:
            assert y is None
            continue
        a = (host(x), None if wi is None else host(wi), None if bi is None else host(bi), host(pos))
        want = R.forward(*a, norm, EPS, rope_dim, inter, **kw)
        close(y, want, R.forward_tol(*a, norm, EPS, rope_dim, inter, out, want), what)


@pytest.mark.parametrize("norm,inter", [("rms", False), ("layer", False), ("rms", True), ("layer", True)])
@pytest.mark.parametrize("D,rope_dim", [(64, 64), (64, 8), (128, 128), (128, 64), (128, 24), (128, 0)])
@pytest.mark.parametrize("src,out", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_forward(norm, inter, D, rope_dim, src, out):
    rng = np.random.default_rng([ord(norm[0]), inter, D, rope_dim, len(src), len(out)])
    q, k, pos, w = inputs(rng, 13, 6, 3, D, src, norm)
    got = dsa.norm_rope(q, k, pos, *w, norm=norm, eps=EPS, rope_dim=rope_dim, rope_interleaved=inter, out_dtype=DT[out])
    check_forward(q, k, pos, w, got, norm, rope_dim, inter, out)


@pytest.mark.parametrize("T,H,Hk", [(1, 1, 1), (1, 64, 8), (33, 1, 1), (200, 20, 5), (5, 128, 128), (3, 1, 0), (40, 3, 0),
                                    (1000, 2, 1), (7, 1024, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_forward_shapes(T, H, Hk, D):
    rng = np.random.default_rng([T, H, Hk, D])
    q, k, pos, w = inputs(rng, T, H, max(Hk, 1), D, "bf16", "rms", wt="bf16", strided=Hk > 0)
    if Hk == 0:
        k, w = None, [w[0], None, None, None]
    got = dsa.norm_rope(q, k, pos, *w, eps=EPS)
    check_forward(q, k, pos, w, got, "rms", D, False, "bf16")


def test_no_weights_in_place_and_given_outputs():
    rng = np.random.default_rng(5)
    q, k, pos, _ = inputs(rng, 50, 7, 2, 128, "bf16", "rms")
    none = [None] * 4
    got = dsa.norm_rope(q, k, pos, eps=EPS)
    check_forward(q, k, pos, none, got, "rms", 128, False, "bf16")
    wide = torch.full((50, 12, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    out = (wide[:, 1:8], wide[:, 9:11])
    assert dsa.norm_rope(q, k, pos, eps=EPS, out=out)[0] is out[0]
    assert torch.equal(out[0], got[0]) and torch.equal(out[1], got[1])
    assert (wide[:, [0, 8, 11]] == 7.0).all()
    dsa.norm_rope(q, k, pos, eps=EPS, out=(q, k))          # over the inputs
    assert torch.equal(q, got[0]) and torch.equal(k, got[1])


def test_frequencies_and_far_positions():
    rng = np.random.default_rng(6)
    q, k, _, w = inputs(rng, 9, 2, 1, 64, "f32", "rms")
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1 << 20, 65535, -12345, 7], dtype=torch.int32, device="cuda")
    freq = [float(f) for f in rng.uniform(-1.0, 1.0, 16)]
    got = dsa.norm_rope(q, k, pos, *w, eps=EPS, rope_dim=32, inv_freq=freq)
    # (the reference's own angles in 64 bits lose bits far out: those positions are held to exact ones below)
    near = [i for i in range(9) if abs(int(pos[i])) <= 1 << 20]
    p = pos[near]
    check_forward(q[near], k[near], p, w, (got[0][near], got[1][near]), "rms", 32, False, "f32", inv_freq=freq)
    a = R.forward(host(q), host(w[0]), None, host(pos), "rms", EPS, 32, False, inv_freq=freq)
    assert np.abs(host(got[0]) - a).max() < 1e-4


def test_rows_do_not_touch_one_another():
    rng = np.random.default_rng(7)
    q, k, pos, w = inputs(rng, 11, 5, 2, 128, "f32", "layer", strided=False)
    want = dsa.norm_rope(q, k, pos, *w, norm="layer", eps=EPS)
    q2, k2 = q.clone(), k.clone()
    q2[3, 1, 5] = float("nan")
    k2[8, 0, 127] = float("inf")
    got = dsa.norm_rope(q2, k2, pos, *w, norm="layer", eps=EPS)
    bad = torch.zeros(11, 5, dtype=torch.bool, device="cuda")
    bad[3, 1] = True
    assert got[0][bad].isnan().all() and torch.equal(got[0][~bad], want[0][~bad])
    bad = torch.zeros(11, 2, dtype=torch.bool, device="cuda")
    bad[8, 0] = True
    assert not got[1][bad].isfinite().any() and torch.equal(got[1][~bad], want[1][~bad])
    zero = torch.zeros_like(q)
    y, _ = dsa.norm_rope(zero, None, pos, w[0], q_bias=w[2], norm="layer", eps=EPS, rope_dim=0)
    assert torch.equal(y, w[2].expand_as(y))


def test_empty_and_ranges_of_values():
    q = torch.empty(0, 4, 64, device="cuda")
    pos = torch.empty(0, dtype=torch.int32, device="cuda")
    a, b = dsa.norm_rope(q, q[:, :1], pos)
    assert a.shape == (0, 4, 64) and b.shape == (0, 1, 64)
    g = dsa.norm_rope_backward(q, q[:, :1], q, q[:, :1], pos, norm="layer")
    assert g.q.shape == q.shape and all((t == 0).all() for t in g[2:])
    rng = np.random.default_rng(8)
    for std in (1e-12, 1e12):          # FP32 squares of 1e12 sum to 1e26; below eps the norm is linear
        q, k, pos, w = inputs(rng, 20, 3, 1, 128, "f32", "rms", std=std)
        check_forward(q, k, pos, w, dsa.norm_rope(q, k, pos, *w, eps=EPS), "rms", 128, False, "f32")


def grads(q, k, pos, w, dq, dk, norm, rope_dim, inter, ws=None):
    return dsa.norm_rope_backward(dq, dk, q, k, pos, w[0], w[1], norm=norm, eps=EPS, rope_dim=rope_dim,
                                  rope_interleaved=inter, ws=ws)


def check_backward(q, k, pos, w, dq, dk, g, norm, rope_dim, inter, src):
    for x, d, wi, gx, gw, gb, what in ((q, dq, w[0], g.q, g.q_weight, g.q_bias, "q"), (k, dk, w[1], g.k, g.k_weight, g.k_bias, "k")):
        if x is None:
            assert gx is None and gw is None and gb is None
            continue
        a = (host(d), host(x), None if wi is None else host(wi), host(pos), norm, EPS, rope_dim, inter)
        dx, dw, db = R.backward(*a)
        tx, tw, tb = R.backward_tol(*a, src, dx)
        close(gx, dx, tx, what)
        close(gw, dw, tw, what + "_weight")
        if norm == "layer":
            close(gb, db, tb, what + "_bias")
        else:
            assert gb is None


@pytest.mark.parametrize("norm,inter", [("rms", False), ("layer", False), ("rms", True), ("layer", True)])
@pytest.mark.parametrize("D,rope_dim", [(64, 64), (64, 16), (128, 128), (128, 40), (128, 0)])
@pytest.mark.parametrize("src,grad", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_backward(norm, inter, D, rope_dim, src, grad):
    rng = np.random.default_rng([ord(norm[0]), inter, D, rope_dim, len(src), len(grad)])
    q, k, pos, w = inputs(rng, 29, 5, 2, D, src, norm)
    d = torch.from_numpy(rng.standard_normal((29, 7, D))).cuda().to(DT[grad])
    dq, dk = d[:, :5], d[:, 5:]
    g = grads(q, k, pos, w, dq, dk, norm, rope_dim, inter)
    check_backward(q, k, pos, w, dq, dk, g, norm, rope_dim, inter, src)


@pytest.mark.parametrize("T,H,Hk", [(1, 1, 1), (1, 64, 8), (700, 3, 1), (40, 128, 128), (9, 3, 0), (3000, 16, 2)])
@pytest.mark.parametrize("D", [64, 128])
def test_backward_shapes_and_bits(T, H, Hk, D):
    rng = np.random.default_rng([T, H, Hk, D, 1])
    q, k, pos, w = inputs(rng, T, H, max(Hk, 1), D, "bf16", "rms", wt="bf16")
    d = torch.from_numpy(rng.standard_normal((T, H + 1 + Hk, D))).cuda().to(torch.bfloat16)
    dq, dk = d[:, :H], d[:, H:H + Hk]
    if Hk == 0:
        k, dk, w = None, None, [w[0], None, None, None]
    ws = dsa.norm_rope_workspace(D)
    g = grads(q, k, pos, w, dq, dk, "rms", D, False, ws)
    assert dsa.read_status(ws) == 0
    check_backward(q, k, pos, w, dq, dk, g, "rms", D, False, "bf16")
    again = grads(q, k, pos, w, dq, dk, "rms", D, False, ws)
    for a, b in zip(g, again):
        assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("norm,inter", [("rms", False), ("layer", True)])
def test_gradients_against_differences(norm, inter):
    """d loss of the forward kernel itself, with loss = sum dy y in 64 bits: central differences of step h are off by
    the forward's FP32 rounding over h and by h^2 third derivatives."""
    rng = np.random.default_rng(12)
    q, k, pos, w = inputs(rng, 3, 2, 1, 64, "f32", norm, strided=False, far=5000)
    w = [t if t is None else t.float() for t in w]
    dq, dk = (torch.from_numpy(rng.standard_normal(t.shape)).cuda().float() for t in (q, k))
    g = grads(q, k, pos, w, dq, dk, norm, 32, inter)

    def loss(q, k, w):
        a, b = dsa.norm_rope(q, k, pos, *w, norm=norm, eps=EPS, rope_dim=32, rope_interleaved=inter)
        return float((a.double() * dq.double()).sum() + (b.double() * dk.double()).sum())

    h = 2.0 ** -6
    # an output is off by at most some 40 half steps of the pair it is part of (norm_ref.lost, the turn): both losses by
    # that of sum |dy| 2 |y|; third derivatives of a row of 64 normed values are below 50
    y = dsa.norm_rope(q, k, pos, *w, norm=norm, eps=EPS, rope_dim=32, rope_interleaved=inter)
    size = sum(float((a.double().abs() * b.double().abs()).sum()) for a, b in zip(y, (dq, dk)))
    noise = 2 * 40 * 2.0 ** -24 * size / h
    for i, (x, gx) in enumerate(((q, g.q), (k, g.k), (w[0], g.q_weight), (w[1], g.k_weight))):
        for at in rng.integers(0, x.numel(), 6):
            v = []
            for s in (h, -h):
                y = x.clone()
                y.view(-1)[at] += s
                args = [q, k, list(w)]
                if i < 2:
                    args[i] = y
                else:
                    args[2][i - 2] = y
                v.append(loss(*args))
            diff = (v[0] - v[1]) / (2 * h)
            assert abs(diff - float(gx.view(-1)[at])) < noise + 50 * h * h, (i, int(at))


def test_streams_and_graphs():
    rng = np.random.default_rng(13)
    q, k, pos, w = inputs(rng, 300, 8, 2, 128, "bf16", "rms")
    d = torch.randn(300, 10, 128, device="cuda").bfloat16()
    want, gw = dsa.norm_rope(q, k, pos, *w), grads(q, k, pos, w, d[:, :8], d[:, 8:], "rms", 128, False)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = [torch.zeros_like(t) for t in want]
        ws = dsa.norm_rope_workspace(128)
        dsa.norm_rope(q, k, pos, *w, out=tuple(out))
    s.synchronize()
    assert torch.equal(out[0], want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = dsa.norm_rope(q, k, pos, *w)
        g = grads(q, k, pos, w, d[:, :8], d[:, 8:], "rms", 128, False, ws)
    for t in (*y, *(t for t in g if t is not None)):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y[0], want[0]) and torch.equal(y[1], want[1])
    assert all(torch.equal(a, b) for a, b in zip(g, gw) if a is not None)


def test_angles_of_the_farthest_positions():
    """Turns from the frequencies' own bits in rational arithmetic: an angle is as good at 2^31 positions as at one."""
    from fractions import Fraction
    pi = Fraction(314159265358979323846264338327950288419716939937510582097494459, 10 ** 62)
    rng = np.random.default_rng(8)
    at = [0, 1, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 1900000001, -1700000003]
    q, k, _, w = inputs(rng, len(at), 3, 1, 128, "f32", "rms")
    pos = torch.tensor(at, dtype=torch.int32, device="cuda")
    freq = [float(f) for f in np.concatenate([rng.uniform(-1.0, 1.0, 60), [1.0, 1e-9, -1e-9, 1234.567]])]
    got = dsa.norm_rope(q, k, pos, *w, eps=EPS, inv_freq=freq)
    ang = np.array([[float((Fraction(f) * p / (2 * pi)) % 1) for f in freq] for p in at]) * (2 * np.pi)
    for x, y, wi in ((q, got[0], w[0]), (k, got[1], w[1])):
        a = (host(x), host(wi), None, host(pos))
        want = R.rotate(R.forward(*a, "rms", EPS, 0, False), ang, 128, False)
        close(y, want, R.forward_tol(*a, "rms", EPS, 128, False, "f32", want), "far")


def test_two_calls_at_once():
    rng = np.random.default_rng(14)
    q, k, pos, w = inputs(rng, 3000, 8, 2, 128, "bf16", "layer")
    d = torch.randn(3000, 10, 128, device="cuda").bfloat16()
    want, gw = dsa.norm_rope(q, k, pos, *w, norm="layer"), grads(q, k, pos, w, d[:, :8], d[:, 8:], "layer", 128, False)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [dsa.norm_rope_workspace(128) for _ in streams]
    got = [[] for _ in streams]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((dsa.norm_rope(q, k, pos, *w, norm="layer"),
                               grads(q, k, pos, w, d[:, :8], d[:, 8:], "layer", 128, False, spaces[i])))
    torch.cuda.synchronize()
    for y, g in got[0] + got[1]:
        assert torch.equal(y[0], want[0]) and torch.equal(y[1], want[1])
        assert all(torch.equal(a, b) for a, b in zip(g, gw))


def test_more_than_32_bits_of_elements():
    T, H, D = 540000, 64, 128            # 4.4e9 elements
    rng = np.random.default_rng(15)
    tail, _, pos, w = inputs(rng, 50, H, 1, D, "bf16", "rms", strided=False)
    d = torch.randn(50, H, D, device="cuda").bfloat16()
    q, g = torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
    q[-50:], g[-50:] = tail, d
    at = torch.zeros(T, dtype=torch.int32, device="cuda")
    at[-50:] = pos
    got, _ = dsa.norm_rope(q, None, at, w[0])
    want, _ = dsa.norm_rope(tail, None, pos, w[0])
    assert torch.equal(got[-50:], want) and not got[:-50].any()
    del got
    a, b = dsa.norm_rope_backward(g, None, q, None, at, w[0]), dsa.norm_rope_backward(d, None, tail, None, pos, w[0])
    assert torch.equal(a.q[-50:], b.q) and not a.q[:-50].any()


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_whatever_the_forward_call_takes_has_a_gradient(norm):
    rng = np.random.default_rng(16)
    q, k, pos, _ = inputs(rng, 21, 3, 2, 64, "f32", norm, strided=False)
    qw, kw, qb, kb = (torch.from_numpy(rng.standard_normal(64)).cuda().float() for _ in range(4))
    if norm == "rms":
        for b in (dict(q_bias=qb), dict(k_bias=kb)):
            with pytest.raises(dsa.DsaError, match="bias"):
                dsa.norm_rope(q, k, pos, qw, kw, norm=norm, **b)
        return
    w = [qw, kw, qb, kb]
    check_forward(q, k, pos, w, dsa.norm_rope(q, k, pos, *w, norm=norm, eps=EPS), norm, 64, False, "f32")
    d = torch.from_numpy(rng.standard_normal((21, 5, 64))).cuda().float()
    g = grads(q, k, pos, w, d[:, :3], d[:, 3:], norm, 64, False)
    assert all(t is not None for t in g)
    check_backward(q, k, pos, w, d[:, :3], d[:, 3:], g, norm, 64, False, "f32")


def test_angles_of_the_highest_frequencies():
    """As test_angles_of_the_farthest_positions, for frequencies up to their bound."""
    from fractions import Fraction
    pi = Fraction(314159265358979323846264338327950288419716939937510582097494459, 10 ** 62)
    rng = np.random.default_rng(17)
    at = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1234567890]
    q, k, _, w = inputs(rng, len(at), 3, 1, 64, "f32", "rms")
    pos = torch.tensor(at, dtype=torch.int32, device="cuda")
    freq = [float(f) for f in np.concatenate([2.0 ** rng.uniform(20, 48, 28), [2.0 ** 48, -2.0 ** 48, 2.0 ** 47 + 1, 3.0]])]
    got = dsa.norm_rope(q, k, pos, *w, eps=EPS, inv_freq=freq)
    ang = np.array([[float((Fraction(f) * p / (2 * pi)) % 1) for f in freq] for p in at]) * (2 * np.pi)
    for x, y, wi in ((q, got[0], w[0]), (k, got[1], w[1])):
        a = (host(x), host(wi), None, host(pos))
        want = R.rotate(R.forward(*a, "rms", EPS, 0, False), ang, 64, False)
        close(y, want, R.forward_tol(*a, "rms", EPS, 64, False, "f32", want), "high")


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("rope_dim", [0, 64])
def test_what_a_non_finite_element_does_to_its_row(norm, value, rope_dim):
    rng = np.random.default_rng(18)
    q, _, pos, w = inputs(rng, 7, 4, 1, 128, "f32", norm, strided=False)
    kw = dict(q_bias=w[2], norm=norm, eps=EPS, rope_dim=rope_dim)
    want, _ = dsa.norm_rope(q, None, pos, w[0], **kw)
    q2 = q.clone()
    q2[4, 2, 10] = value
    got, _ = dsa.norm_rope(q2, None, pos, w[0], **kw)
    rows = torch.ones(7, 4, dtype=torch.bool, device="cuda")
    rows[4, 2] = False
    assert torch.equal(got[rows], want[rows])
    lost = torch.ones(128, dtype=torch.bool, device="cuda")
    if norm == "rms" and not np.isnan(value):      # x / inf but for the element, or its pair
        lost[:] = False
        lost[[10, 42] if rope_dim else [10]] = True
        assert (got[4, 2][~lost] == 0).all()
    assert got[4, 2][lost].isnan().all()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rope_dim,at,pair", [(0, 10, 10), (64, 100, 100), (64, 10, None)])
def test_what_a_non_finite_gradient_does_to_the_sums(norm, inter, value, rope_dim, at, pair):
    """A weight's gradient is the sum over its own column, and its partner's where the two are rotated."""
    if pair is None:
        pair = at ^ 1 if inter else at + 32
    rng = np.random.default_rng(20)
    q, k, pos, w = inputs(rng, 40, 3, 2, 128, "f32", norm, strided=False)
    d = torch.from_numpy(rng.standard_normal((40, 5, 128))).cuda().float()
    dq, dk = d[:, :3].contiguous(), d[:, 3:].contiguous()
    want = grads(q, k, pos, w, dq, dk, norm, rope_dim, inter)
    dq[7, 1, at] = value
    got = grads(q, k, pos, w, dq, dk, norm, rope_dim, inter)
    rest = torch.ones(128, dtype=torch.bool, device="cuda")
    rest[[at, pair]] = False
    for a, b in ((got.q_weight, want.q_weight), (got.q_bias, want.q_bias)):
        if a is not None:
            assert torch.equal(a[rest], b[rest]) and not a[at].isfinite()
    for a, b in ((got.k, want.k), (got.k_weight, want.k_weight), (got.k_bias, want.k_bias)):
        assert a is b is None or torch.equal(a, b)
    rows = torch.ones(40, 3, dtype=torch.bool, device="cuda")
    rows[7, 1] = False
    assert torch.equal(got.q[rows], want.q[rows])


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("log2", [-60, 60])
def test_the_largest_and_smallest_rows(norm, D, log2):
    """Largest elements of 2^60, of 2^-60 without eps, every element as large or one alone."""
    rng = np.random.default_rng([19, D])
    x = np.ldexp(np.where(rng.random((6, 2, D)) < 0.5, -1.0, 1.0), log2)
    x[3:, :, 1:] *= 2.0 ** -9
    if norm == "layer":
        x -= x.mean(-1, keepdims=True)
        x *= 2.0 ** log2 / np.abs(x).max(-1, keepdims=True)
        x = x.astype(np.float32).astype(np.float64)
    q = torch.from_numpy(x).cuda().float()
    got, _ = dsa.norm_rope(q, None, None, norm=norm, eps=0.0, rope_dim=0)
    a = (x, None, None, np.zeros(6), norm, 0.0, 0, False)
    want = R.forward(*a)
    close(got, want, R.forward_tol(*a, "f32", want), "far")
