"""lq_distill_loss where its numbers are far apart: listed logits far above the
others, nothing outside the list.  The oracle differentiates the float64 loss itself.

Tolerances, derived before the first run.  With d = (reference maximum - z) /
temp >= 0 an exponential carries 3 * 2^-24 d from its exponent (difference,
factor, product), 2^-22 from the hardware, and a float32 sum of a thread some
hundred roundings of 2^-24 at random: e(d) = 2^-18 + 2^-22 d relative for an
exponential over its sum.  d averaged over a softmax of V entries is at most
log V < 12, so a logarithm of a sum is off by 2^-18.  log q and log Q add the
rounding of log2(e) / temp, 2^-24 of their size: 2^-18 + 2^-23 |log q|.  The
teacher's p carries 2^-22 + 2^-23 |log p|, and R = 1 - sum p the same of the sum:
d_R = 2^-20 for p over a few hundred entries (sum p |log p| <= log k < 6).
"""
import math

import pytest
import torch

from bit_ptq_looped_b200 import lq

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# the smallest step near zero (the exponential flushes float32 subnormals)
SUB = {torch.float32: 2.0 ** -124, torch.bfloat16: 2.0 ** -124, torch.float16: 2.0 ** -24}
D_R = 2.0 ** -20


def rand(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda") * scale


def log_sum(y):
    """log sum exp(y) as (m, l), m + l: apart, or l is lost beside an m of 1e38, and
    with it the gradient."""
    m = y.detach().max()
    return m, torch.log(torch.exp(y - m).sum())


def row_oracle(z, tv, ti, t_lse, w, temp):
    """One row: (loss, grad, tolerance of each but for the last rounding)."""
    V = z.numel()
    Z = z.double().cpu().requires_grad_()
    y = Z / temp
    pos, val = [], []
    for v, t in zip(ti.tolist(), tv.double().tolist()):
        if 0 <= v < V and v not in pos:
            pos.append(v), val.append(t / temp)
    zero = torch.zeros(V, dtype=torch.float64)
    if w == 0 or (t_lse is None and not pos):
        return 0.0, zero, 0.0, zero
    idx = torch.tensor(pos, dtype=torch.int64)
    hidden = torch.zeros(V, dtype=torch.bool)
    hidden[idx] = True
    t = torch.tensor(val, dtype=torch.float64)
    R = 0.0
    if t_lse is None:
        log_p = t - t.max() - log_sum(t)[1]
    else:
        log_p = t - t_lse
        R = max(0.0, 1.0 - float(log_p.exp().sum()))
    p = log_p.exp()
    m, l = log_sum(y)
    on = p > 0
    log_q = y[idx][on] - m - l
    loss = (p[on] * (log_p[on] - log_q)).sum()
    rest = y[~hidden]
    log_Q = torch.tensor(0.0)
    if R > 0 and bool((rest > -math.inf).any()):
        m_rest, l_rest = log_sum(rest)
        log_Q = m_rest - m + l_rest - l
        loss = loss + R * (math.log(R) - log_Q)
    else:
        R = 0.0
    g, = torch.autograd.grad(loss, Z)
    with torch.no_grad():
        tl = float((p[on] * (2.0 ** -18 + 2.0 ** -23 * log_q.abs() + 2.0 ** -22 +
                             2.0 ** -23 * log_p[on].abs())).sum())
        # an error of p moves its own term as well
        tl += float((p[on] * (2.0 ** -22 + 2.0 ** -23 * log_p[on].abs()) *
                     (log_p[on] - log_q).abs()).sum())
        C = float(p.sum()) + R
        q = (y - m - l).exp()
        tg = C * q * (2.0 ** -18 + 2.0 ** -22 * (y.max() - y).clamp(max=1e4))
        tg[idx] += p * (2.0 ** -21 + 2.0 ** -22 * log_p.clamp(min=-1e4).abs())
        if R:
            size = abs(math.log(R)) + abs(float(log_Q))
            tl += R * (2.0 ** -18 + 2.0 ** -23 * size) + D_R * (2 + size)
            s = torch.where(hidden, zero, (y - m_rest - l_rest).exp())
            tg += s * (R * (2.0 ** -18 + 2.0 ** -22 * (rest.max() - y).clamp(0, 1e4)) + D_R)
    return w * float(loss.detach()), g * w, abs(w) * tl, abs(w) / temp * tg


def check(z, tv, ti, t_lse=None, w=None, temp=1.0, rows=None):
    """The whole call against the oracle on some of its rows."""
    loss, grad = lq.lq_distill_loss(z, tv, ti, t_lse=t_lse, weight=w, temp=temp, want_grad=True)
    only, _ = lq.lq_distill_loss(z, tv, ti, t_lse=t_lse, weight=w, temp=temp)
    assert torch.equal(only.nan_to_num(), loss.nan_to_num()), "the gradient changes the loss"
    eps = torch.finfo(z.dtype).eps / 2
    for m in range(z.shape[0]) if rows is None else rows:
        L, G, tl, tg = row_oracle(z[m], tv[m], ti[m], None if t_lse is None else float(t_lse[m]),
                                  1.0 if w is None else float(w[m]), temp)
        got = float(loss[m])
        assert abs(got - L) <= tl + 2.0 ** -24 * abs(L), (m, got, L, tl)
        g = grad[m].double().cpu()
        err = (g - G).abs() / (tg + eps * (G.abs() + tg) + SUB[z.dtype])
        assert bool((err <= 1).all()), (m, int((~(err <= 1)).sum()), float(err.max()),
                                        int(err.nan_to_num(math.inf).argmax()))
    return loss, grad


def apart(seed, M, V, k, dt, gap, R):
    """k listed logits about `gap` above the others; the teacher leaves mass R."""
    ti = torch.stack([torch.randperm(V, generator=torch.Generator().manual_seed(seed + m))[:k]
                      for m in range(M)]).cuda()
    z = rand(seed, M, V)
    z.scatter_add_(1, ti, torch.full((M, k), float(gap), device="cuda"))
    tv = rand(seed + 1, M, k)
    return z.to(dt), tv, ti, torch.logsumexp(tv.double(), 1) - math.log(1 - R)


# a row in one CTA, and one shared by a cluster of eight
@pytest.mark.parametrize("M,V,k", [(3, 1000, 64), (2, 49152, 64)])
@pytest.mark.parametrize("gap", [-110, 60, 80, 84, 86, 90, 110, 200, 800, 10000])
@pytest.mark.parametrize("temp", [0.5, 1.0])
def test_rest_class_far_below_the_list(M, V, k, gap, temp):
    for name, R in (("f32", 0.1), ("bf16", 0.95), ("f16", 0.5)):
        z, tv, ti, lse = apart(gap + V, M, V, k, TYPES[name], gap, R)
        lse = torch.logsumexp(tv.double() / temp, 1) - math.log(1 - R)
        loss, grad = check(z, tv, ti, t_lse=lse.float(), temp=temp)
        if gap > 200:  # the unlisted entries' gradients sum to -R / temp
            sums = grad.double().scatter(1, ti, 0.0).sum(1) * temp
            assert float((sums + R).abs().max()) <= 2.0 ** -8 * R + 1e-3


def test_one_listed_logit_far_above_the_others():
    z = torch.zeros(4, 49152, device="cuda")
    z[:, 17] = 110.0
    tv, ti = torch.zeros(4, 1, device="cuda"), torch.full((4, 1), 17, device="cuda")
    check(z, tv, ti, t_lse=torch.full((4,), -math.log(0.9), device="cuda"))


@pytest.mark.parametrize("mask", [-100.0, -700.0, -1e4])
def test_a_finite_mask_over_everything_unlisted(mask):
    for name in ("f32", "bf16"):
        z, tv, ti, lse = apart(5, 2, 20011, 100, TYPES[name], 0.0, 0.3)
        rest = torch.full_like(z, mask).scatter(1, ti, z.gather(1, ti))
        check(rest, tv, ti, t_lse=lse.float())


def test_a_row_does_not_depend_on_the_batch():
    """One CTA a row (a batch of 400) and eight (the row alone): the same loss and
    gradient within twice the tolerance."""
    for gap in (0, 86, 110, 800):
        z, tv, ti, lse = apart(gap, 400, 20011, 50, torch.float32, gap, 0.4)
        loss, grad = check(z, tv, ti, t_lse=lse.float(), rows=(0, 399))
        one, g1 = check(z[399:].clone(), tv[399:].clone(), ti[399:].clone(),
                        t_lse=lse[399:].float())
        assert float((one - loss[399:]).abs()) <= 2.0 ** -17 * (1 + float(loss[399].abs()))
        assert float((g1[0] - grad[399]).abs().max()) <= 2.0 ** -17


def test_no_mass_outside_the_list():
    """Every unlisted logit -inf, or nothing unlisted at all, while the teacher leaves
    mass R: the returned loss has no R term, and its gradient P q - p sums to zero."""
    for M, V, k in ((3, 900, 11), (2, 33001, 50), (4, 17, 17)):
        for name, R in (("f32", 0.3), ("bf16", 0.9), ("f16", 0.01)):
            z, tv, ti, lse = apart(V, M, V, k, TYPES[name], 0.0, R)
            only = torch.full_like(z, -math.inf).scatter(1, ti, z.gather(1, ti))
            loss, grad = check(only, tv, ti, t_lse=lse.float())
            assert not grad.gather(1, ti).isnan().any()
            assert not grad.scatter(1, ti, 0.0).any()
            eps = torch.finfo(z.dtype).eps / 2
            size = grad.double().abs().sum(1)
            assert bool((grad.double().sum(1).abs() <= 2.0 ** -17 + eps * size + k * SUB[z.dtype])
                        .all())


def test_gradient_against_differences_without_mass_outside():
    """Central differences over the listed logits of such a row; noise and cubic term
    as for ordinary rows: the loss is known to 2^-20 of its logarithms (below 8)."""
    z, tv, ti, lse = apart(3, 3, 120, 9, torch.float32, 0.0, 0.4)
    z = torch.full_like(z, -math.inf).scatter(1, ti, z.gather(1, ti))
    lse = lse.float()
    _, grad = lq.lq_distill_loss(z, tv, ti, t_lse=lse, want_grad=True)
    step = 2.0 ** -4
    for trial in range(4):
        d = torch.sign(rand(40 + trial, 3, 120))
        up = lq.lq_distill_loss(z + step * d, tv, ti, t_lse=lse)[0]
        dn = lq.lq_distill_loss(z - step * d, tv, ti, t_lse=lse)[0]
        num = (up - dn).double() / (2 * step)
        ana = (grad.double() * d.double()).sum(1)
        assert bool(((num - ana).abs() <= 2.0 ** -17 / (2 * step) + step ** 2).all())


@pytest.mark.parametrize("name", TYPES)
def test_masked_entries_next_to_ordinary_ones(name):
    """-inf and the type's lowest value between ordinary logits, listed or not."""
    dt = TYPES[name]
    teacher = rand(6, 4, 900, scale=3.0)
    z = (teacher + rand(7, 4, 900, scale=0.7)).to(dt)
    tv, ti = torch.topk(teacher, 11, dim=1)
    hide = torch.ones(900, dtype=torch.bool, device="cuda")
    hide[ti.flatten()] = False
    at = hide.nonzero().flatten()
    z[:, at[::3]] = -math.inf
    z[:, at[1::3]] = torch.finfo(dt).min
    for lse in (None, torch.logsumexp(teacher, 1)):
        loss, grad = check(z, tv, ti, t_lse=lse)
        assert not grad[z == -math.inf].any()


def lowest(dt):
    return torch.finfo(dt).min


@pytest.mark.parametrize("M,V,k", [(3, 1000, 64), (2, 49152, 64), (300, 8001, 20)])
@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("temp", [0.5, 1.0, 3.0])
def test_blocks_masked_with_the_lowest_value(M, V, k, name, temp):
    """A padded vocabulary, or whole regions, masked with the type's lowest value: the
    threads that see nothing else count nothing."""
    dt = TYPES[name]
    for lo, hi in ((V - V // 5, V), (0, V // 3), (V // 4, V // 2)):
        z, tv, ti, lse = apart(V + lo, M, V, k, dt, 3.0, 0.2)
        mask = torch.zeros(M, V, dtype=torch.bool, device="cuda")
        mask[:, lo:hi] = True
        mask.scatter_(1, ti, False)
        z = torch.where(mask, torch.full_like(z, lowest(dt)), z)
        lse = (torch.logsumexp(tv.double() / temp, 1) - math.log(0.8)).float()
        for t_lse in (None, lse):
            loss, grad = check(z, tv, ti, t_lse=t_lse, temp=temp, rows=(0, M - 1))
            assert not grad[mask].any() and not loss.isnan().any()


@pytest.mark.parametrize("M,V", [(3, 1000), (2, 49152)])
def test_rows_of_nothing_but_the_lowest_value(M, V):
    """Equal logits are a uniform distribution wherever they lie, the teacher's too;
    masked with the lowest value outside the list, the rest class costs R times the
    distance."""
    for name, dt in TYPES.items():
        z, tv, ti, lse = apart(V, M, V, 30, dt, 0.0, 0.3)
        flat = torch.full_like(z, lowest(dt))
        for t_lse in (None, lse.float()):
            check(flat, tv, ti, t_lse=t_lse)
        check(z, torch.full_like(tv, lowest(torch.float32)), ti)
        check(z, torch.full_like(tv, lowest(dt)).to(dt), ti)
        check(torch.full_like(z, lowest(dt)).scatter(1, ti, z.gather(1, ti)), tv, ti,
              t_lse=lse.float())
        # a listed logit that is masked while the teacher gives it mass
        check(z.scatter(1, ti[:, :1], lowest(dt)), tv, ti)
        check(z.scatter(1, ti[:, :1], lowest(dt)), tv, ti, t_lse=lse.float())
        top = z.clone()
        top[:, V // 2:] = -lowest(dt) / 2  # and the far side: most of the mass up there
        top[:, :V // 2] = lowest(dt)
        check(top, tv, ti, t_lse=lse.float())


def test_small_temperatures():
    """logits over the temperature past float32's range."""
    z, tv, ti, lse = apart(1, 3, 1000, 20, torch.float32, 0.0, 0.3)
    for temp in (1e-3, 1e-10, 1e-30):
        scaled = z * temp
        scaled[:, 500:] = -1e37
        scaled = scaled.scatter(1, ti, (z * temp).gather(1, ti))
        for t_lse in (None, lse.float()):
            loss, grad = check(scaled, tv * temp, ti, t_lse=t_lse, temp=temp)
            assert not loss.isinf().any()


@pytest.mark.parametrize("M,V,k", [(3, 100, 7), (2, 1000, 64), (2, 49152, 64), (300, 20011, 20)])
@pytest.mark.parametrize("name", TYPES)
def test_not_a_number_reaches_the_loss(M, V, k, name):
    """A NaN among the logits makes its row's loss and gradient NaN, wherever it is and
    also where a whole block of them fills a thread; NaN among the teacher's values
    likewise.  Other rows are as without it."""
    dt = TYPES[name]
    z, tv, ti, lse = apart(V, M, V, k, dt, 1.0, 0.3)
    nan = float("nan")
    for t_lse in (None, lse.float()):
        want = lq.lq_distill_loss(z[:1].clone(), tv[:1].clone(), ti[:1].clone(), want_grad=True,
                                  t_lse=None if t_lse is None else t_lse[:1].clone())
        for lo, hi in ((50, 51), (V - 1, V), (16, 48), (0, V)):
            bad = z.clone()
            bad[1, lo:hi] = nan
            loss, grad = lq.lq_distill_loss(bad, tv, ti, t_lse=t_lse, want_grad=True)
            assert loss[1].isnan() and grad[1].isnan().all(), (lo, hi)
            assert not loss[0].isnan() and not grad[0].isnan().any()
            if M == 3 and V == 100:  # the row alone is cut as in the batch
                assert torch.equal(loss[:1], want[0]) and torch.equal(grad[:1], want[1])
        for n in (1, k):
            badt = tv.clone()
            badt[1, :n] = nan
            loss, grad = lq.lq_distill_loss(z, badt, ti, t_lse=t_lse, want_grad=True)
            assert loss[1].isnan() and not loss[0].isnan()
            assert grad[1].gather(0, ti[1, :n]).isnan().all()


def test_a_replayed_graph_reads_its_inputs_anew():
    """Logits, teacher values and indices, log-partition and weights copied in anew
    between replays: nothing of the capture or of the replay before stays."""
    M, V, k = 40, 5003, 32
    batches = []
    for seed in (1, 2, 3):
        z, tv, ti, lse = apart(seed, M, V, k, torch.bfloat16, 2.0, 0.3)
        batches.append((z, tv, ti, lse.float(), rand(seed + 9, M).abs()))
    for tail in (False, True):
        want = [lq.lq_distill_loss(z, tv, ti, t_lse=lse if tail else None, weight=w,
                                   want_grad=True) for z, tv, ti, lse, w in batches]
        held = [torch.zeros_like(t) for t in batches[0]]
        loss, grad = torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lq.lq_distill_loss(held[0], held[1], held[2], t_lse=held[3] if tail else None,
                               weight=held[4], loss=loss, grad=grad)
        for i in (0, 1, 2, 0):
            for t, src in zip(held, batches[i]):
                t.copy_(src)
            loss.fill_(float("nan")), grad.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(loss, want[i][0]) and torch.equal(grad, want[i][1])
        assert not torch.equal(want[0][0], want[1][0])
