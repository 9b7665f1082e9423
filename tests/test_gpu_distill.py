"""lq_distill_loss against its definition in float64.

Tolerances, derived before the first run.  With c = log2(e) / temp rounded to
float32 the exponents carry 2^-24 of (|z - lse|) / temp, the hardware
exponential 2^-22, the float32 sums of a thread (at most a few hundred terms)
their own roundings, so S is known to about 2^-20 and each log q to
e_q = 2^-20 + 2^-23 |log q|.  The loss is a sum of p-weighted differences:
|error| <= w (sum p (e_q + 2^-22 |log p|) + R (2^-20 (1 + |log R| + |log Q|) + d_R ...)),
d_R = 2^-23 from the float32 log-partition.  A gradient entry is
w / temp (C q - p): relative 2^-19 (|log q| + 1) of q and p each, then the
rounding to the logits' type, eps / 2.
"""
import math

import pytest
import torch

from bit_ptq_looped_b200 import lq

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# the smallest step near zero (the exponential flushes float32 subnormals)
SUB = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -24}


def rand(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda") * scale


def oracle(z, tv, ti, t_lse, w, temp):
    """Row by row from the definition, float64: (loss, grad, tolerance of the
    loss, tolerance of the gradient before its rounding)."""
    M, V = z.shape
    loss, tl = torch.zeros(M, dtype=torch.float64), torch.zeros(M, dtype=torch.float64)
    grad = torch.zeros((M, V), dtype=torch.float64)
    tg = torch.zeros((M, V), dtype=torch.float64)
    Z, TV, TI = z.double().cpu() / temp, tv.double().cpu() / temp, ti.cpu()
    for m in range(M):
        wm = 1.0 if w is None else float(w[m])
        seen, pos, val = set(), [], []
        for i in range(TI.shape[1]):
            v = int(TI[m, i])
            if 0 <= v < V and v not in seen:
                seen.add(v), pos.append(v), val.append(float(TV[m, i]))
        if wm == 0 or (t_lse is None and not pos):
            continue
        val = torch.tensor(val, dtype=torch.float64)
        log_q = torch.log_softmax(Z[m], 0)
        q = log_q.exp()
        idx = torch.tensor(pos, dtype=torch.int64)
        hidden = torch.zeros(V, dtype=torch.bool)
        hidden[idx] = True
        R = 0.0
        if t_lse is None:
            log_p = torch.log_softmax(val, 0)
            # every teacher logit -inf: no mass at all (0 / 0 in the softmax)
            log_p = torch.where(log_p.isnan(), torch.full_like(log_p, -math.inf), log_p)
            p = log_p.exp()
        else:
            log_p = val - float(t_lse[m])
            p = log_p.exp()
            R = max(0.0, 1.0 - float(p.sum()))
        C = float(p.sum()) + R if t_lse is not None else (1.0 if float(p.sum()) > 0 else 0.0)
        on = p > 0
        lq_top = log_q[idx][on]
        L = float((p[on] * (log_p[on] - lq_top)).sum())
        e_q = 2.0 ** -20 + 2.0 ** -23 * lq_top.abs()
        T = float((p[on] * (e_q + 2.0 ** -22 * log_p[on].abs() + 2.0 ** -23)).sum())
        Q = float(q[~hidden].sum())
        k = 0.0
        if R > 0 and Q > 0:
            L += R * (math.log(R) - math.log(Q))
            dR = 2.0 ** -22
            T += R * 2.0 ** -19 * (1 + abs(math.log(R)) + abs(math.log(Q))) + \
                dR * (2 + abs(math.log(R)) + abs(math.log(Q)))
            k = R / Q
        d = torch.where(hidden, torch.zeros(1, dtype=torch.float64), q * (C - k))
        d[idx] = C * q[idx] - p
        e = 2.0 ** -19 * (1 + log_q.abs())
        e = torch.where(log_q.isinf(), torch.zeros_like(e), e)
        t = q * e * (C + k) + (q * 2.0 ** -21 * (1 + 1 / max(Q, 1e-30)) if k else 0.0)
        t[idx] = (q * e)[idx] * max(C, 1.0) + p * 2.0 ** -19 * (1 + log_p.clamp(min=-1e4).abs())
        loss[m], tl[m] = wm * L, abs(wm) * T
        grad[m], tg[m] = wm / temp * d, abs(wm) / temp * t
    return loss, grad, tl, tg


def check(z, tv, ti, t_lse=None, w=None, temp=1.0, in_place=False):
    L, G, tl, tg = oracle(z, tv, ti, t_lse, w, temp)
    only, none = lq.lq_distill_loss(z, tv, ti, t_lse=t_lse, weight=w, temp=temp)
    assert none is None
    zi = z.clone()
    loss, grad = lq.lq_distill_loss(zi, tv, ti, t_lse=t_lse, weight=w, temp=temp, want_grad=True,
                                    grad=zi if in_place else None)
    if not in_place:
        assert torch.equal(zi.nan_to_num(), z.nan_to_num()), "the logits changed"
    assert torch.equal(only, loss), "the gradient changes the loss"
    lo = loss.double().cpu()
    ok = (lo - L).abs() <= tl + 2.0 ** -23 * L.abs()
    assert bool(ok.all()), f"loss {lo[~ok][:4]} want {L[~ok][:4]} tolerance {tl[~ok][:4]}"
    g = grad.double().cpu()
    fi = torch.finfo(z.dtype)
    tol = tg + fi.eps / 2 * (G.abs() + tg) + SUB[z.dtype]
    bad = ~((g - G).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(),
                           float(((g - G).abs() / tol).max()))
    return loss, grad


def case(seed, M, V, k, dt, spread=0.7, scale=3.0, index=torch.int64):
    teacher = rand(seed, M, V, scale=scale)
    z = (teacher + rand(seed + 1, M, V, scale=spread)).to(dt)
    tv, ti = torch.topk(teacher, k, dim=1)
    return teacher, z, tv.contiguous(), ti.to(index).contiguous()


SHAPES = [(1, 1, 1), (3, 2, 1), (2, 7, 7), (5, 31, 3), (4, 33, 33), (3, 100, 17), (7, 1003, 64),
          (2, 4096, 1000), (130, 515, 9), (2, 49152, 1000), (3, 50001, 128), (1, 100003, 1000)]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("M,V,k", SHAPES)
def test_listed_distribution(M, V, k, dt):
    _, z, tv, ti = case(M + V, M, V, k, TYPES[dt])
    check(z, tv, ti)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("M,V,k", SHAPES)
def test_rest_class(M, V, k, dt):
    teacher, z, tv, ti = case(M + V, M, V, k, TYPES[dt], index=torch.int32)
    check(z, tv, ti, t_lse=torch.logsumexp(teacher, 1))


@pytest.mark.parametrize("temp", [0.5, 2.0, 3.7])
def test_temperature_weights_and_teacher_types(temp):
    for t_dt in TYPES.values():
        teacher, z, tv, ti = case(5, 9, 301, 12, torch.bfloat16)
        tv = tv.to(t_dt)
        w = torch.tensor([0.0, 1.0, 0.25, 3.0, 0.0, -1.0, 1e-3, 1.0, 0.5], device="cuda")
        check(z, tv, ti, w=w, temp=temp)
        check(z, tv, ti, t_lse=torch.logsumexp(teacher.double() / temp, 1).float(), w=w, temp=temp)


def test_wide_rows_over_every_cluster_size():
    """One row and many, so that a row is one slice, two, four or eight."""
    for M, V, dt in ((1, 1000, "bf16"), (40, 20011, "bf16"), (90, 20011, "f32"),
                     (160, 20011, "f16"), (300, 20011, "bf16"), (2, 380001, "f32"),
                     (1, 524288, "bf16")):
        teacher, z, tv, ti = case(V, M, V, 50, TYPES[dt])
        rows = slice(0, min(M, 6))
        L, G, tl, tg = oracle(z[rows], tv[rows], ti[rows], None, None, 1.0)
        loss, grad = lq.lq_distill_loss(z, tv, ti, want_grad=True)
        assert bool(((loss[rows].double().cpu() - L).abs() <= tl + 2.0 ** -23 * L.abs()).all())
        fi = torch.finfo(z.dtype)
        tol = tg + fi.eps / 2 * (G.abs() + tg) + SUB[z.dtype]
        assert bool(((grad[rows].double().cpu() - G).abs() <= tol).all())
        # the last row of the batch against the same row alone (other slices)
        again, _ = lq.lq_distill_loss(z[M - 1:].clone(), tv[M - 1:].clone(), ti[M - 1:].clone())
        assert float((again - loss[M - 1:]).abs().max()) <= 1e-5 * float(loss.abs().max())


def test_in_place_and_neighbouring_rows():
    for V in (257, 1000, 33001):
        for dt in TYPES.values():
            _, z, tv, ti = case(V, 5, V, 8, dt)
            _, want = lq.lq_distill_loss(z, tv, ti, want_grad=True)
            _, got = check(z, tv, ti, in_place=True)
            assert torch.equal(got, want)


def test_nothing_behind_the_last_row_is_written():
    M, V, k = 3, 1001, 5
    for dt in TYPES.values():
        _, z, tv, ti = case(1, M, V, k, dt)
        buf = torch.full((M * V + 64,), 7.0, dtype=dt, device="cuda")
        lo = torch.full((M + 8,), 7.0, device="cuda")
        lq.lq_distill_loss(z, tv, ti, loss=lo[:M], grad=buf[:M * V].view(M, V))
        assert bool((buf[M * V:] == 7).all()) and bool((lo[M:] == 7).all())


def test_padding_entries_repeated_indices_and_empty_rows():
    M, V, k = 6, 500, 8
    teacher, z, tv, ti = case(3, M, V, k, torch.float32)
    ti[0, 5:] = -1                     # a shorter list
    ti[1] = V                          # no entry at all
    ti[2, 3] = ti[2, 0]                # listed again: counts at its first place
    ti[2, 7] = ti[2, 0]
    ti[3] = ti[3, 0].item()            # one entry, eight times
    tv[4, 2] = -math.inf               # a teacher logit that is masked
    tv[5] = -math.inf                  # all of them
    big = torch.tensor([2 ** 40, -2 ** 40, 2 ** 32 + 1], device="cuda")
    ti[0, 5:8] = big
    loss, grad = check(z, tv, ti)
    assert loss[1] == 0 and not grad[1].any() and loss[5] == 0 and not grad[5].any()
    check(z, tv, ti, t_lse=torch.logsumexp(teacher, 1))


def test_rows_of_weight_zero_count_nothing():
    M, V, k = 4, 700, 9
    for dt in TYPES.values():
        teacher, z, tv, ti = case(4, M, V, k, dt)
        w = torch.tensor([1.0, 0.0, 0.0, 2.0], device="cuda")
        want_l, want_g = lq.lq_distill_loss(z, tv, ti, weight=w, want_grad=True)
        z[1], z[2, 5] = float("nan"), float("inf")
        tv[1] = float("nan")
        for lse in (None, torch.logsumexp(teacher, 1)):
            loss, grad = lq.lq_distill_loss(z, tv, ti, t_lse=lse, weight=w, want_grad=True)
            assert not loss[1:3].any() and not grad[1:3].any()
            if lse is None:
                assert torch.equal(loss, want_l) and torch.equal(grad, want_g)


def test_masked_vocabulary():
    """Student logits of -inf (and the type's lowest value): no mass, zero
    gradient, whether listed by a teacher of no mass or not listed."""
    for dt in TYPES.values():
        teacher, z, tv, ti = case(6, 4, 900, 11, dt)
        hide = torch.ones(900, dtype=torch.bool, device="cuda")
        hide[ti.flatten()] = False
        z[:, hide.nonzero().flatten()[::3]] = -math.inf
        z[:, hide.nonzero().flatten()[1::3]] = torch.finfo(dt).min
        z[3] = torch.where(hide, torch.full_like(z[3], -math.inf), z[3])  # only listed ones left
        loss, grad = check(z, tv, ti)
        assert not grad[z == -math.inf].any()
        check(z, tv, ti, t_lse=torch.logsumexp(teacher, 1))


def test_close_and_concentrated_distributions():
    """Student equal to the teacher (loss and gradient at rounding level), nearly
    all mass in the list, and far-away maxima (no overflow)."""
    for dt in TYPES.values():
        teacher, z, tv, ti = case(7, 5, 2000, 100, dt, spread=0.0, scale=8.0)
        check(z, tv, ti)
        check(z, tv, ti, t_lse=torch.logsumexp(teacher, 1))
        check((z.float() + 200).to(dt), tv + 300, ti, t_lse=torch.logsumexp(teacher + 300, 1))
        check((z.float() - 200).to(dt), tv - 300, ti)


def test_offsets_past_32_bits():
    """A batch of more than 2^31 logits: its last rows."""
    V, k = 49152, 16
    M = 2 ** 31 // V + 3
    z = torch.zeros((M, V), dtype=torch.bfloat16, device="cuda")
    _, tail, tv1, ti1 = case(8, 2, V, k, torch.bfloat16)
    z[-2:] = tail
    tv, ti = torch.zeros((M, k), device="cuda"), torch.zeros((M, k), dtype=torch.int32,
                                                             device="cuda")
    ti += torch.arange(k, device="cuda", dtype=torch.int32)
    tv[-2:], ti[-2:] = tv1, ti1.int()
    L, G, tl, tg = oracle(tail, tv1, ti1, None, None, 1.0)
    loss, _ = lq.lq_distill_loss(z, tv, ti, grad=z)
    assert bool(((loss[-2:].double().cpu() - L).abs() <= tl + 2.0 ** -23 * L.abs()).all())
    tol = tg + torch.finfo(torch.bfloat16).eps / 2 * (G.abs() + tg) + 2.0 ** -126
    assert bool(((z[-2:].double().cpu() - G).abs() <= tol).all())
    # every other row: q uniform, p uniform over its k entries
    want = math.log(V / k)
    assert float((loss[:-2].double() - want).abs().max()) <= 1e-5 * want


def test_gradient_against_differences():
    """Central differences of the float32 loss: the loss is known to about
    2^-20 of its logarithms (here below 8), so a difference over 2 step has
    noise 2^-17 / (2 step) per row, and a cubic term below step^2."""
    teacher, z, tv, ti = case(9, 3, 120, 7, torch.float32)
    step = 2.0 ** -4
    for lse in (None, torch.logsumexp(teacher, 1)):
        _, grad = lq.lq_distill_loss(z, tv, ti, t_lse=lse, want_grad=True)
        for trial in range(4):
            d = torch.sign(rand(20 + trial, 3, 120))
            up = lq.lq_distill_loss(z + step * d, tv, ti, t_lse=lse)[0]
            dn = lq.lq_distill_loss(z - step * d, tv, ti, t_lse=lse)[0]
            num = (up - dn).double() / (2 * step)
            ana = (grad.double() * d.double()).sum(1)
            assert bool(((num - ana).abs() <= 2.0 ** -17 / (2 * step) + step ** 2).all())


def test_streams_graphs_and_two_calls_at_once():
    teacher, z, tv, ti = case(10, 40, 5003, 32, torch.bfloat16)
    _, z2, tv2, ti2 = case(11, 40, 5003, 32, torch.bfloat16)
    want = lq.lq_distill_loss(z, tv, ti, want_grad=True)
    want2 = lq.lq_distill_loss(z2, tv2, ti2, want_grad=True)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = [(lq.lq_distill_loss(z, tv, ti, want_grad=True, stream=a),
            lq.lq_distill_loss(z2, tv2, ti2, want_grad=True, stream=b)) for _ in range(4)]
    a.synchronize(), b.synchronize()
    for g1, g2 in got:
        assert all(torch.equal(p, q) for p, q in zip(g1 + g2, want + want2))
    zi = torch.zeros_like(z)
    lo, gr = torch.empty_like(want[0]), torch.empty_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lq.lq_distill_loss(zi, tv, ti, loss=lo, grad=gr)
    for src, ref in ((z, want), (z, want)):
        zi.copy_(src)
        lo.fill_(float("nan")), gr.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(lo, ref[0]) and torch.equal(gr, ref[1])


def test_no_rows_and_refusals():
    e = torch.empty((0, 10), dtype=torch.bfloat16, device="cuda")
    t, i = torch.empty((0, 2), device="cuda"), torch.empty((0, 2), dtype=torch.int64, device="cuda")
    loss, grad = lq.lq_distill_loss(e, t, i, want_grad=True)
    assert loss.shape == (0,) and grad.shape == (0, 10)
    _, z, tv, ti = case(12, 2, 40, 3, torch.float32)
    for bad in (lambda: lq.lq_distill_loss(z.cpu(), tv, ti),
                lambda: lq.lq_distill_loss(z, tv, ti.float()),
                lambda: lq.lq_distill_loss(z, tv, ti[:, :2]),
                lambda: lq.lq_distill_loss(z, tv, ti, weight=torch.ones(3, device="cuda")),
                lambda: lq.lq_distill_loss(z.t(), tv, ti),
                lambda: lq.lq_distill_loss(z.double(), tv, ti)):
        with pytest.raises(ValueError):
            bad()
    for kw, status in ((dict(temp=0.0), lq.LQ_ERR_ARG), (dict(temp=float("nan")), lq.LQ_ERR_ARG),
                       (dict(temp=float("inf")), lq.LQ_ERR_ARG)):
        with pytest.raises(lq.LQError) as err:
            lq.lq_distill_loss(z, tv, ti, **kw)
        assert err.value.status == status
    with pytest.raises(lq.LQError) as err:  # more entries than vocabulary
        lq.lq_distill_loss(z[:, :2].contiguous(), tv, ti)
    assert err.value.status == lq.LQ_ERR_SHAPE
    buf = torch.zeros(3 * 40, device="cuda")
    with pytest.raises(lq.LQError) as err:  # a gradient that overlaps the logits elsewhere
        lq.lq_distill_loss(buf[:80].view(2, 40), tv, ti, grad=buf[40:].view(2, 40))
    assert err.value.status == lq.LQ_ERR_ARG
