"""The dense products (lq_dense_linear, lq_gated_linear and their backward
passes) against the formulas in float64.

Tolerances, derived before the first run.  eps is torch.finfo(type).eps, so a
rounding to the type is off by at most eps / 2 of the value.
  * A product sum over n terms: products of 16-bit values are exact in float32;
    the tensor core adds 16 terms per instruction and is allowed 2^-21 of the
    running sum of magnitudes per instruction (four units in the last place;
    its additions do not round to nearest), plus two float32 additions (bias,
    residual): acc(n) = (n / 16 + 4) 2^-21 of A = sum |a| |b| (+ |bias|).
  * Activations have slopes up to 1.13 and are computed in float32 with the
    hardware exponential and reciprocal: 1.13 acc + 2^-19 of the value, and
    2^-20 absolute per unit of |z| near zero crossings of the gate.
  * dz is rounded to the type before the products: (eps / 2 + 2^-18) of |dz|,
    and act' may be off by 2^-19 absolute (values up to 1.13), so dz by 2^-19
    of its other factors; the products add acc(n) of A' = sum |dz'| |w|, where
    |dz'| includes those factors.
  * every output: eps / 2 of its value, and half a subnormal step for f16.
"""
import math

import pytest
import torch

from bit_ptq_looped_b200 import lq

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
SUB = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 0.0}


def half_step(dt):
    return torch.finfo(dt).eps / 2


def acc(n):
    return (n / 16 + 4) * 2.0 ** -21


def normal(seed, *shape, scale=1.0, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def act64(act, z):
    F = torch.nn.functional
    return {lq.LQ_ACT_NONE: lambda v: v * 1.0, lq.LQ_ACT_RELU: F.relu, lq.LQ_ACT_SILU: F.silu,
            lq.LQ_ACT_GELU: F.gelu,
            lq.LQ_ACT_GELU_TANH: lambda v: F.gelu(v, approximate="tanh")}[act](z)


def slope64(act, z):
    z = z.detach().clone().requires_grad_()
    return torch.autograd.grad(act64(act, z).sum(), z)[0]


def close(got, want, tol, what):
    dt = got.dtype
    tol = tol + half_step(dt) * (want.abs() + tol) + SUB[dt]
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst error / tolerance "
                           f"{float((err / (tol + 1e-300)).max())}, first at "
                           f"{bad.nonzero()[0].tolist()}")


def check_dense(M, N, K, dt, act, bias, residual, seed=0):
    x = normal(seed, M, K, dtype=dt)
    w = normal(seed + 1, N, K, scale=K ** -0.5, dtype=dt)
    b = normal(seed + 2, N, dtype=dt) if bias else None
    r = normal(seed + 3, M, N, dtype=dt) if residual else None
    y, z = lq.lq_dense_linear(x, w, b, act=act, residual=r, want_z=True)
    y2, none = lq.lq_dense_linear(x, w, b, act=act, residual=r)
    assert none is None and torch.equal(y, y2), "saving z changes y"
    z64 = x.double() @ w.double().T
    A = x.double().abs() @ w.double().abs().T
    if bias:
        z64, A = z64 + b.double(), A + b.double().abs()
    close(z, z64, acc(K) * A, "z")
    y64 = act64(act, z64)
    tol = 1.13 * acc(K) * A
    if act != lq.LQ_ACT_NONE:
        tol = tol + 2.0 ** -19 * y64.abs() + 2.0 ** -20 * z64.abs()
    if residual:
        y64 = y64 + r.double()
        tol = tol + 2.0 ** -23 * y64.abs()
    close(y, y64, tol, "y")


def check_dense_bwd(M, N, K, dt, act, g_dtype=None, seed=0):
    dy = normal(seed, M, N, dtype=dt)
    x = normal(seed + 1, M, K, dtype=dt)
    w = normal(seed + 2, N, K, scale=K ** -0.5, dtype=dt)
    z = normal(seed + 3, M, N, scale=2.0, dtype=dt) if act != lq.LQ_ACT_NONE else None
    dx, dw, db = lq.lq_dense_linear_bwd(dy, x, w, z, act=act, want_db=True, g_dtype=g_dtype)
    D = dy.double()
    if z is None:
        dz, mag, rel, ab = D, D.abs(), 0.0, 0.0
    else:
        dz = D * slope64(act, z.double())
        mag, rel, ab = dz.abs(), half_step(dt) + 2.0 ** -18, 2.0 ** -19
    off = rel * mag + ab * D.abs() + (SUB[dt] if z is not None else 0.0)  # error of dz
    W, X = w.double().abs(), x.double().abs()
    close(dx, dz @ w.double(), off @ W + acc(N) * ((mag + off) @ W), "dx")
    close(dw, dz.T @ x.double(), off.T @ X + acc(M) * ((mag + off).T @ X), "dw")
    # db sums the float32 dz: no rounding to the type, float32 additions
    f32 = (2.0 ** -18 * mag + ab * D.abs()).sum(0) if z is not None else 0.0
    close(db, dz.sum(0), f32 + (M / 8 + 64) * 2.0 ** -24 * mag.sum(0), "db")
    return dx, dw, db


def check_gated(M, N, K, dt, act, bias, seed=0):
    x = normal(seed, M, K, dtype=dt)
    wg = normal(seed + 1, N, K, scale=K ** -0.5, dtype=dt)
    wu = normal(seed + 2, N, K, scale=K ** -0.5, dtype=dt)
    bg = normal(seed + 3, N, dtype=dt) if bias else None
    bu = normal(seed + 4, N, dtype=dt) if bias else None
    h, g, u = lq.lq_gated_linear(x, wg, wu, bg, bu, act=act, want_gu=True)
    h2, _, _ = lq.lq_gated_linear(x, wg, wu, bg, bu, act=act)
    assert torch.equal(h, h2), "saving g and u changes h"
    X = x.double()
    g64, u64 = X @ wg.double().T, X @ wu.double().T
    Ag, Au = X.abs() @ wg.double().abs().T, X.abs() @ wu.double().abs().T
    if bias:
        g64, u64 = g64 + bg.double(), u64 + bu.double()
        Ag, Au = Ag + bg.double().abs(), Au + bu.double().abs()
    close(g, g64, acc(K) * Ag, "g")
    close(u, u64, acc(K) * Au, "u")
    a64 = act64(act, g64)
    ta = 1.13 * acc(K) * Ag + 2.0 ** -19 * a64.abs() + 2.0 ** -20 * g64.abs()
    tu = acc(K) * Au
    close(h, a64 * u64, ta * (u64.abs() + tu) + a64.abs() * tu + 2.0 ** -23 * (a64 * u64).abs(),
          "h")


def check_gated_bwd(M, N, K, dt, act, g_dtype=None, seed=0):
    dh, g, u = (normal(seed + i, M, N, dtype=dt) for i in range(3))
    x = normal(seed + 3, M, K, dtype=dt)
    wg = normal(seed + 4, N, K, scale=K ** -0.5, dtype=dt)
    wu = normal(seed + 5, N, K, scale=K ** -0.5, dtype=dt)
    dx, dwg, dwu, dbg, dbu = lq.lq_gated_linear_bwd(dh, g, u, x, wg, wu, act=act, want_db=True,
                                                    g_dtype=g_dtype)
    H, G, U, X = dh.double(), g.double(), u.double(), x.double()
    a, s = act64(act, G), slope64(act, G)
    dg, du = H * U * s, H * a
    rel = half_step(dt) + 2.0 ** -18
    og = rel * dg.abs() + 2.0 ** -19 * (H * U).abs() + SUB[dt]
    ou = rel * du.abs() + 2.0 ** -20 * (H * G).abs() + SUB[dt]
    Wg, Wu = wg.double(), wu.double()
    mg, mu = dg.abs() + og, du.abs() + ou
    close(dx, dg @ Wg + du @ Wu, og @ Wg.abs() + ou @ Wu.abs() +
          acc(2 * N) * (mg @ Wg.abs() + mu @ Wu.abs()), "dx")
    close(dwg, dg.T @ X, og.T @ X.abs() + acc(M) * (mg.T @ X.abs()), "dwg")
    close(dwu, du.T @ X, ou.T @ X.abs() + acc(M) * (mu.T @ X.abs()), "dwu")
    f = (M / 8 + 64) * 2.0 ** -24
    close(dbg, dg.sum(0), (2.0 ** -18 * dg.abs() + 2.0 ** -19 * (H * U).abs()).sum(0) +
          f * dg.abs().sum(0), "dbg")
    close(dbu, du.sum(0), (2.0 ** -18 * du.abs() + 2.0 ** -20 * (H * G).abs()).sum(0) +
          f * du.abs().sum(0), "dbu")


SHAPES = [(1, 8, 8), (1, 1, 8), (2, 3, 24), (3, 1000, 520), (4, 257, 264), (7, 65, 72), (8, 256, 256), (9, 255, 264),
          (16, 1000, 1032), (17, 64, 64), (33, 1, 8), (127, 128, 128), (128, 130, 40),
          (129, 257, 200), (300, 1000, 520), (1000, 264, 2048), (513, 2049, 256),
          (2300, 640, 72), (1, 2048, 5632), (13, 5632, 2048)]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_dense_shapes(M, N, K, dt):
    check_dense(M, N, K, TYPES[dt], lq.LQ_ACT_SILU, True, True)
    check_dense(M, N, K, TYPES[dt], lq.LQ_ACT_NONE, False, False, seed=10)


@pytest.mark.parametrize("act", lq.LQ_ACTS.values(), ids=lq.LQ_ACTS.keys())
@pytest.mark.parametrize("M", [5, 200])
def test_dense_activations(M, act):
    for bias, residual in ((False, True), (True, False)):
        check_dense(M, 136, 128, torch.bfloat16, act, bias, residual)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_dense_backward_shapes(M, N, K, dt):
    check_dense_bwd(M, N, K, TYPES[dt], lq.LQ_ACT_GELU)
    check_dense_bwd(M, N, K, TYPES[dt], lq.LQ_ACT_NONE, seed=10)


@pytest.mark.parametrize("act", lq.LQ_ACTS.values(), ids=lq.LQ_ACTS.keys())
def test_dense_backward_activations(act):
    check_dense_bwd(150, 136, 72, torch.float16, act)
    check_dense_bwd(150, 136, 72, torch.bfloat16, act, g_dtype=torch.float32)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gated_shapes(M, N, K, dt):
    check_gated(M, N, K, TYPES[dt], lq.LQ_ACT_SILU, True)
    check_gated(M, N, K, TYPES[dt], lq.LQ_ACT_GELU_TANH, False, seed=10)


@pytest.mark.parametrize("act", lq.LQ_ACTS.values(), ids=lq.LQ_ACTS.keys())
@pytest.mark.parametrize("M", [3, 140])
def test_gated_activations(M, act):
    check_gated(M, 72, 136, torch.bfloat16, act, True)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gated_backward_shapes(M, N, K, dt):
    check_gated_bwd(M, N, K, TYPES[dt], lq.LQ_ACT_SILU)


@pytest.mark.parametrize("act", lq.LQ_ACTS.values(), ids=lq.LQ_ACTS.keys())
def test_gated_backward_activations(act):
    check_gated_bwd(150, 136, 72, torch.bfloat16, act)
    check_gated_bwd(65, 40, 72, torch.float16, act, g_dtype=torch.float32)


def test_many_tiles_and_long_contractions():
    """More tiles than SMs (both accumulators and the ring wrap many times) and a
    contraction of many thousands."""
    check_dense(4200, 5632, 256, torch.bfloat16, lq.LQ_ACT_NONE, True, True)
    check_gated(4200, 2816, 256, torch.bfloat16, lq.LQ_ACT_SILU, False)
    check_dense_bwd(20000, 264, 136, torch.float16, lq.LQ_ACT_RELU)
    check_gated_bwd(9000, 1000, 512, torch.bfloat16, lq.LQ_ACT_SILU)
    # few tiles: the contraction in slices that another pass adds up
    check_gated_bwd(8192, 100, 136, torch.bfloat16, lq.LQ_ACT_SILU)
    check_gated_bwd(8192, 100, 136, torch.float16, lq.LQ_ACT_GELU, g_dtype=torch.float32)
    check_dense_bwd(33, 5632, 264, torch.bfloat16, lq.LQ_ACT_NONE)
    check_dense_bwd(70, 5001, 264, torch.bfloat16, lq.LQ_ACT_SILU)


# few tiles over a contraction long enough that a cluster of CTAs shares a tile
SHARED = [(17, 1, 1544), (33, 65, 2048), (40, 72, 1600), (64, 2048, 2048), (100, 1003, 2064),
          (128, 257, 5632), (129, 2048, 5632), (257, 130, 2056), (300, 264, 8000)]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("M,N,K", SHARED)
def test_shared_tiles(M, N, K, dt):
    check_dense(M, N, K, TYPES[dt], lq.LQ_ACT_GELU, True, True)
    check_dense(M, N, K, TYPES[dt], lq.LQ_ACT_NONE, False, False, seed=10)
    check_gated(M, N, K, TYPES[dt], lq.LQ_ACT_SILU, True, seed=20)
    check_gated(M, N, K, TYPES[dt], lq.LQ_ACT_RELU, False, seed=30)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("M,N,K", [(17, 1040, 264), (100, 5001, 72), (129, 2048, 1000),
                                   (260, 4100, 512)])
def test_shared_tiles_backward(M, N, K, dt):
    """dx over N; of the gated form over both factors, whose border lies inside a
    member's part (N = 1040)."""
    check_dense_bwd(M, N, K, TYPES[dt], lq.LQ_ACT_SILU)
    check_dense_bwd(M, N, K, TYPES[dt], lq.LQ_ACT_NONE, seed=10)
    check_gated_bwd(M, N, K, TYPES[dt], lq.LQ_ACT_GELU)


@pytest.mark.parametrize("N", [200, 201, 130, 195])
def test_shared_tiles_in_place_repeatable_and_within_rows(N):
    dt, K = torch.bfloat16, 2048
    for M in (20, 130):
        x, w = normal(1, M, K, dtype=dt), normal(2, N, K, scale=K ** -0.5, dtype=dt)
        r = normal(3, M, N, dtype=dt)
        want, _ = lq.lq_dense_linear(x, w, residual=r)
        assert torch.equal(want, lq.lq_dense_linear(x, w, residual=r)[0])
        buf = torch.full((M * N + 4096,), 7.0, dtype=dt, device="cuda")
        y = buf[:M * N].view(M, N)
        y.copy_(r)
        lq.lq_dense_linear(x, w, residual=y, y=y)
        assert torch.equal(y, want) and bool((buf[M * N:] == 7).all())
        # a row's values do not depend on the rows beside it
        bad = x.clone()
        bad[3] = float("nan")
        got = lq.lq_dense_linear(bad, w, residual=r)[0]
        keep = torch.arange(M, device="cuda") != 3
        assert torch.equal(got[keep], want[keep]) and bool(got[3].isnan().all())


def test_shared_tiles_on_two_streams_and_replayed():
    """Chains of calls that read each other's outputs, on two streams at once and as
    a replayed graph, against the same chain alone."""
    dt, n = torch.bfloat16, 2048
    ws = [normal(i, n, n, scale=n ** -0.5, dtype=dt) for i in range(3)]

    def chain(x, outs):
        for i, y in enumerate(outs):
            lq.lq_dense_linear(x, ws[i % 3], act=lq.LQ_ACT_SILU, residual=x, y=y)
            x = y

    xs = [normal(10 + i, 60 + i, n, dtype=dt) for i in range(2)]
    outs = [[torch.empty_like(x) for _ in range(12)] for x in xs]
    want = []
    for x, o in zip(xs, outs):
        chain(x, o)
        torch.cuda.synchronize()
        want.append([y.clone() for y in o])
        for y in o:
            y.zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for st, x, o in zip(streams, xs, outs):
            with torch.cuda.stream(st):
                chain(x, o)
    torch.cuda.synchronize()
    for o, e in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, e))
    for y in outs[0]:
        y.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(xs[0], outs[0])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs[0], want[0]))
    lq.lq_check_device()


@pytest.mark.parametrize("N", [200, 201, 130, 195])
def test_residual_in_place_and_repeatable(N):
    dt = torch.bfloat16
    for M in (6, 333):
        x, w = normal(1, M, 128, dtype=dt), normal(2, N, 128, dtype=dt)
        r = normal(3, M, N, dtype=dt)
        want, _ = lq.lq_dense_linear(x, w, residual=r)
        again, _ = lq.lq_dense_linear(x, w, residual=r)
        assert torch.equal(want, again)
        got, _ = lq.lq_dense_linear(x, w, residual=r, y=r)
        assert got is r and torch.equal(got, want)


def test_rows_behind_the_output_stay():
    """Neither the rows behind the last one nor the values after an odd row end
    are written."""
    for M, N, K in ((5, 9, 16), (100, 9, 16), (129, 65, 64), (300, 200, 64), (131, 130, 64),
                    (333, 703, 64)):
        buf = torch.full((M * N + 4096,), 7.0, dtype=torch.float16, device="cuda")
        y = buf[:M * N].view(M, N)
        lq.lq_dense_linear(normal(1, M, K, dtype=torch.float16),
                           normal(2, N, K, dtype=torch.float16), y=y)
        assert bool((buf[M * N:] == 7).all())
        dyb = normal(3, M, N, dtype=torch.float16)
        buf = torch.full((N * K + 4096,), 7.0, dtype=torch.float32, device="cuda")
        lq.lq_dense_linear_bwd(dyb, normal(1, M, K, dtype=torch.float16), None, want_dx=False,
                               dw=buf[:N * K].view(N, K))
        assert bool((buf[N * K:] == 7).all())


@pytest.mark.parametrize("M", [0, 1, 700, 8192])
def test_float32_weight_gradients_accumulate(M):
    """The gradient of a weight shared by the loops, added up loop by loop."""
    dt, N, K = torch.bfloat16, 72, 136
    dw = torch.full((N, K), 0.5, device="cuda")
    db = torch.full((N,), -0.25, device="cuda")
    want_w, want_b = dw.double(), db.double()
    tol_w, tol_b = torch.zeros_like(want_w), torch.zeros_like(want_b)
    for t in range(3):
        dy, x = normal(2 * t, M, N, dtype=dt), normal(2 * t + 1, M, K, dtype=dt)
        w = normal(9, N, K, dtype=dt)
        lq.lq_dense_linear_bwd(dy, x, w, dw=dw, db=db, accumulate=True)
        want_w = want_w + dy.double().T @ x.double()
        want_b = want_b + dy.double().sum(0)
        tol_w = tol_w + acc(M) * (dy.double().abs().T @ x.double().abs()) + 2.0 ** -23 * 100
        tol_b = tol_b + (M / 8 + 64) * 2.0 ** -24 * dy.double().abs().sum(0) + 2.0 ** -23 * 100
    assert bool(((dw - want_w).abs() <= tol_w).all()) and bool(((db - want_b).abs() <= tol_b).all())
    if M == 0:
        assert bool((dw == 0.5).all()) and bool((db == -0.25).all())


def test_no_rows():
    dt, N, K = torch.float16, 40, 24
    e = lambda n: torch.empty((0, n), dtype=dt, device="cuda")
    w = normal(1, N, K, dtype=dt)
    assert lq.lq_dense_linear(e(K), w)[0].shape == (0, N)
    assert lq.lq_gated_linear(e(K), w, w.clone(), want_gu=True)[0].shape == (0, N)
    dx, dw, db = lq.lq_dense_linear_bwd(e(N), e(K), w, e(N), act=lq.LQ_ACT_SILU, want_db=True)
    assert dx.shape == (0, K) and not dw.any() and not db.any()
    out = lq.lq_gated_linear_bwd(e(N), e(N), e(N), e(K), w, w.clone(), want_db=True)
    assert out[0].shape == (0, K) and not any(t.any() for t in out[1:])


def test_backward_parts_alone_give_the_same_bits():
    dt, M, N, K = torch.bfloat16, 210, 100, 64
    dh, g, u = (normal(i, M, N, dtype=dt) for i in range(3))
    x = normal(3, M, K, dtype=dt)
    wg, wu = normal(4, N, K, dtype=dt), normal(5, N, K, dtype=dt)
    full = lq.lq_gated_linear_bwd(dh, g, u, x, wg, wu, want_db=True)
    dx = lq.lq_gated_linear_bwd(dh, g, u, None, wg, wu, want_dw=False)[0]
    assert torch.equal(dx, full[0])
    for name, want in (("dwg", full[1]), ("dwu", full[2])):
        o = torch.empty((N, K), dtype=dt, device="cuda")
        lq.lq_gated_linear_bwd(dh, g, u, x, None, None, want_dx=False, want_dw=False, **{name: o})
        assert torch.equal(o, want), name
    db = lq.lq_gated_linear_bwd(dh, g, u, x, wg, wu, want_dx=False, want_dw=False, want_db=True)
    assert torch.equal(db[3], full[3]) and torch.equal(db[4], full[4])


def test_gradients_against_differences():
    """Central differences of the library's own forward pass along random
    directions, in f16 with an exactly representable step: the forward values
    are rounded to f16 (2^-11), so the sum over n outputs weighted by v is
    known to 2^-11 sqrt(n)-ish; the bound takes every rounding at its worst
    share of 4 sigma."""
    dt, M, N, K = torch.float16, 24, 48, 32
    x = normal(1, M, K, dtype=dt)
    wg, wu = normal(2, N, K, scale=K ** -0.5, dtype=dt), normal(3, N, K, scale=K ** -0.5, dtype=dt)
    v = normal(4, M, N, dtype=dt)
    h, g, u = lq.lq_gated_linear(x, wg, wu, want_gu=True)
    dx, dwg, dwu, _, _ = lq.lq_gated_linear_bwd(v, g, u, x, wg, wu)
    step = 2.0 ** -5
    for t, grad in ((x, dx), (wg, dwg), (wu, dwu)):
        for trial in range(3):
            d = torch.sign(normal(10 + trial, *t.shape, dtype=torch.float32))
            sides = []
            for sgn in (1, -1):
                moved = (t.float() + sgn * step * d).to(dt)
                a = [moved if s is t else s for s in (x, wg, wu)]
                hh = lq.lq_gated_linear(*a)[0].double()
                sides.append((float((hh * v.double()).sum()), float(hh.square().sum()),
                              moved.double()))
            num = sides[0][0] - sides[1][0]
            ana = float((grad.double() * (sides[0][2] - sides[1][2])).sum())
            # f16 rounding of h on both sides, of the gradient, and the cubic term
            noise = 4 * 2.0 ** -11 * math.sqrt(2 * (v.double().square() * 1.0).mean() *
                                               max(sides[0][1], sides[1][1]))
            gn = 4 * 2.0 ** -10 * float(grad.double().norm()) * 2 * step
            cubic = 0.02 * abs(ana) + 4 * step ** 3 * float(grad.double().norm())
            assert abs(num - ana) <= noise + gn + cubic, (num, ana, noise, gn, cubic)


@pytest.mark.parametrize("M", [4, 200])
def test_infinite_and_nan_rows_stay_in_their_rows(M):
    """Rows do not mix in the forward pass and in dx: what a padding row holds
    reaches no other row."""
    dt = torch.bfloat16
    x, w = normal(1, M, 64, dtype=dt), normal(2, 72, 64, dtype=dt)
    want = lq.lq_dense_linear(x, w, act=lq.LQ_ACT_SILU)[0]
    xb = x.clone()
    xb[1], xb[3, 0] = float("nan"), float("inf")
    got = lq.lq_dense_linear(xb, w, act=lq.LQ_ACT_SILU)[0]
    keep = [i for i in range(M) if i not in (1, 3)]
    assert torch.equal(got[keep], want[keep])
    assert bool(got[1].isnan().all())


def test_large_activation_arguments():
    """Saturated activations and their slopes stay finite and right."""
    dt = torch.bfloat16
    zs = [0.0, -0.0, 1e-30, -1e-30, 20.0, -20.0, 88.5, -88.5, 1e4, -1e4, 1e20, -1e20, 1e30]
    z = torch.tensor(zs + [0.0] * 3, device="cuda").to(dt).view(1, -1)
    one = torch.ones_like(z)
    x, w = torch.zeros((1, 8), dtype=dt, device="cuda"), torch.zeros((16, 8), dtype=dt,
                                                                     device="cuda")
    for act in lq.LQ_ACTS.values():
        db = lq.lq_dense_linear_bwd(one, x, w, z, act=act, want_dx=False, want_dw=False,
                                    want_db=True)[2]
        want = slope64(act, z.double().clamp(-1e6, 1e6))[0]
        assert bool((db.double() - want).abs().max() <= 2.0 ** -8 * 1.13 + 2.0 ** -19), act
        y = lq.lq_dense_linear(x, w, z[0], act=act)[0][0]
        want = act64(act, z.double())[0]
        assert bool(((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -18).all()), act


def test_other_stream_and_graph():
    """Calls on a stream of their own, and two captured graphs that share a
    workspace, replayed in turn with new inputs."""
    dt, M, N, K = torch.bfloat16, 150, 136, 128
    w = normal(2, N, K, dtype=dt)
    z = normal(3, M, N, dtype=dt)
    dy = normal(4, M, N, dtype=dt)
    xs = [normal(5 + i, M, K, dtype=dt) for i in range(2)]
    want = [lq.lq_dense_linear_bwd(dy, x, w, z, act=lq.LQ_ACT_SILU, want_db=True) for x in xs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lq.lq_dense_linear_bwd(dy, xs[0], w, z, act=lq.LQ_ACT_SILU, want_db=True, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    n = lq.lib().lq_dense_linear_bwd_workspace_bytes(M, N, K, lq.LQ_ACT_SILU)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    graphs, outs, ins = [], [], []
    for x in xs:
        xi = torch.zeros_like(x)
        o = [torch.empty_like(t) for t in want[0]]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lq.lq_dense_linear_bwd(dy, xi, w, z, act=lq.LQ_ACT_SILU, dx=o[0], dw=o[1], db=o[2],
                                   ws=ws)
        graphs.append(g), outs.append(o), ins.append(xi)
    for _ in range(2):
        for i in (0, 1):
            ins[i].copy_(xs[i])
            graphs[i].replay()
        ws.fill_(255)
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i]))
    lq.lq_check_device()


def test_two_streams_at_once():
    """Calls on two streams with their own workspaces, forward and backward, tiles
    of CTA pairs among them."""
    dt = torch.bfloat16
    sets = [(normal(s, 700, 520, dtype=dt), normal(s + 1, 1200, 520, dtype=dt),
             normal(s + 2, 1200, 520, dtype=dt), normal(s + 3, 700, 1200, dtype=dt))
            for s in (0, 10)]

    def step(x, wg, wu, dh, stream=None):
        h, g, u = lq.lq_gated_linear(x, wg, wu, want_gu=True, stream=stream)
        return (h,) + lq.lq_gated_linear_bwd(dh, g, u, x, wg, wu, want_db=True, stream=stream)

    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i in (0, 1):
            got[i].append(step(*sets[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


def test_captured_behind_copies_and_joins():
    """In a captured graph behind a memset, a copy and a join of another stream: the
    calls wait for all of them."""
    dt, M, N, K = torch.float16, 260, 392, 1032
    x, w = normal(1, M, K, dtype=dt), normal(2, N, K, dtype=dt)
    b, r = normal(3, N, dtype=dt), normal(4, M, N, dtype=dt)
    want, _ = lq.lq_dense_linear(x, w, b, act=lq.LQ_ACT_SILU, residual=r)
    xi, wi, ri = torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(r)
    y = torch.empty_like(want)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        xi.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(20):  # work that takes longer than what runs beside it
                wi.copy_(w)
                ri.copy_(r)
        xi.copy_(x)
        torch.cuda.current_stream().wait_stream(side)
        lq.lq_dense_linear(xi, wi, b, act=lq.LQ_ACT_SILU, residual=ri, y=y)
        lq.lq_dense_linear(xi, wi, b, act=lq.LQ_ACT_SILU, residual=y, y=y)
        xi.fill_(float("nan"))
    want2, _ = lq.lq_dense_linear(x, w, b, act=lq.LQ_ACT_SILU, residual=want)
    for _ in range(5):
        y.zero_(), wi.zero_(), ri.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want2)


def test_same_weight_twice_and_shared_inputs():
    """The same tensor as both projections, and as several operands of a call."""
    dt, M, N, K = torch.bfloat16, 150, 72, 72
    for M in (3, 150):
        x, w = normal(1, M, K, dtype=dt), normal(2, N, K, scale=0.1, dtype=dt)
        h, g, u = lq.lq_gated_linear(x, w, w, want_gu=True)
        h2, _, _ = lq.lq_gated_linear(x, w, w.clone())
        assert torch.equal(h, h2) and torch.equal(g, u)
        a = lq.lq_gated_linear_bwd(x, x, x, x, w, w)
        b = lq.lq_gated_linear_bwd(x.clone(), x.clone(), x.clone(), x, w, w.clone())
        assert all(torch.equal(p, q) for p, q in zip(a[:3], b[:3]))
        y, _ = lq.lq_dense_linear(x, w, residual=x)
        y2, _ = lq.lq_dense_linear(x, w, residual=x.clone())
        assert torch.equal(y, y2)


def test_feed_forward_block_step():
    """One training step of a block's feed-forward half through the entry points:
    gate and up, the down projection with its residual, the output head, the
    distillation loss, and all gradients back to the input, against autograd in
    float64 (relative norms: each 16-bit rounding along the chain contributes
    at most half a step of its tensor; there are at most eight on the longest
    path, and the loss's own gradient adds two)."""
    dt, M, d, f, V, k = torch.float16, 96, 64, 168, 517, 20
    x = normal(1, M, d, dtype=dt)
    wg, wu = normal(2, f, d, scale=d ** -0.5, dtype=dt), normal(3, f, d, scale=d ** -0.5, dtype=dt)
    wd = normal(4, d, f, scale=f ** -0.5, dtype=dt)
    head = normal(5, V, d, scale=d ** -0.5, dtype=dt)
    tv, ti = torch.topk(normal(6, M, V, scale=2.0, dtype=torch.float32), k, dim=1)
    weight = torch.full((M,), 16.0, device="cuda")
    h, g, u = lq.lq_gated_linear(x, wg, wu, want_gu=True)
    y, _ = lq.lq_dense_linear(h, wd, residual=x)
    logits, _ = lq.lq_dense_linear(y, head)
    loss, dl = lq.lq_distill_loss(logits, tv, ti, weight=weight, want_grad=True)
    dy, dhead, _ = lq.lq_dense_linear_bwd(dl, y, head)
    dh, dwd, _ = lq.lq_dense_linear_bwd(dy, h, wd)
    dx, dwg, dwu, _, _ = lq.lq_gated_linear_bwd(dh, g, u, x, wg, wu)
    dx = dx + dy
    P = [t.double().requires_grad_() for t in (x, wg, wu, wd, head)]
    X, WG, WU, WD, HD = P
    Y = (torch.nn.functional.silu(X @ WG.T) * (X @ WU.T)) @ WD.T + X
    log_q = torch.log_softmax(Y @ HD.T, 1).gather(1, ti)
    log_p = torch.log_softmax(tv.double(), 1)
    L = 16.0 * (log_p.exp() * (log_p - log_q)).sum(1)
    want = torch.autograd.grad(L.sum(), P)
    L = L.detach()
    tol = 10 * half_step(dt)
    assert float((loss - L).norm() / L.norm()) <= tol
    for got, ref, name in zip((dx, dwg, dwu, dwd, dhead), want, ("dx", "dwg", "dwu", "dwd",
                                                                 "dhead")):
        assert float((got.double() - ref).norm() / ref.norm()) <= tol, name


def test_refusals():
    dt = torch.bfloat16
    x, w = normal(1, 4, 16, dtype=dt), normal(2, 8, 16, dtype=dt)
    for bad in (lambda: lq.lq_dense_linear(x.cpu(), w), lambda: lq.lq_dense_linear(x, w.half()),
                lambda: lq.lq_dense_linear(x.t(), w), lambda: lq.lq_dense_linear(x, w[:, :8]),
                lambda: lq.lq_dense_linear(x, w, y=torch.empty((8, 4), dtype=dt, device="cuda")),
                lambda: lq.lq_dense_linear_bwd(x, None, None),
                lambda: lq.lq_dense_linear_bwd(normal(3, 4, 8, dtype=dt), x, w, want_db=True,
                                               accumulate=True)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(lq.LQError) as e:
        lq.lq_dense_linear(x.float(), w.float())
    assert e.value.status == lq.LQ_ERR_UNSUPPORTED
    with pytest.raises(lq.LQError) as e:
        lq.lq_dense_linear(normal(1, 4, 12, dtype=dt), normal(2, 8, 12, dtype=dt))
    assert e.value.status == lq.LQ_ERR_SHAPE
    with pytest.raises(lq.LQError) as e:
        lq.lq_dense_linear(x, w, act=9)
    assert e.value.status == lq.LQ_ERR_UNSUPPORTED
    buf = normal(1, 64, 16, dtype=dt)
    with pytest.raises(lq.LQError) as e:  # y over x
        lq.lq_dense_linear(buf[:16], normal(2, 16, 16, dtype=dt), y=buf[8:24])
    assert e.value.status == lq.LQ_ERR_ARG
    with pytest.raises(lq.LQError) as e:  # a view that starts between 16-byte boundaries
        lq.lq_dense_linear(buf.view(-1)[4:4 + 64].view(4, 16), w)
    assert e.value.status == lq.LQ_ERR_ALIGN
    with pytest.raises(lq.LQError) as e:
        lq.lq_dense_linear_bwd(normal(3, 40, 8, dtype=dt), normal(1, 40, 16, dtype=dt), w,
                               normal(3, 40, 8, dtype=dt), act=lq.LQ_ACT_SILU,
                               ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == lq.LQ_ERR_WORKSPACE
