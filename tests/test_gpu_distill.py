"""The distillation loss and its gradient against the float64 oracle.

Tolerances count roundings, u = 2^-24.  With R the range of the row's finite
z = logit / T, a cell's exponential has a relative error of at most e = (4 R
+ 8) u (the difference from the reference, the factor log2(e) / T and the
product are rounded, each by u of up to R, and the exponential itself by a
few u), a sum of them e + 132 u (at most 128 terms in fp32 per thread, then
fp64), which is what the log-sum-exps are off by: delta = (4 R + 140) u.
  loss      w T^2 (delta + 2 u |terms|), and its own rounding u |loss|
  gradient  w T (q + p_r-share) (e + delta + |lse| u where the stats were
            stored in fp32), the known cells w T (q delta + u (q + p)), and
            the output type's half step of the value; fp16 below 2^-14 has
            the absolute step 2^-25
"""

import numpy as np
import pytest
import torch

import oracle as orc
import post_weight_quantization_15_amd as gq

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    gq.load_library()
    return torch.device("cuda:0")


def inputs(n, vocab, k, dtype, T, tail, seed=0, scale=2.5, noise=1.0):
    rng = np.random.default_rng([seed, n, vocab, k])
    z = torch.from_numpy((scale * rng.normal(size=(n, vocab))).astype(np.float32))
    teacher = z.numpy().astype(np.float64) + noise * rng.normal(size=(n, vocab))
    idx = np.argsort(-teacher, axis=1, kind="stable")[:, :k].astype(np.int32)
    t = np.take_along_axis(teacher, idx, 1).astype(np.float32)
    t_lse = None
    if tail:
        s = teacher / T
        top = s.max(1)
        t_lse = (top + np.log(np.exp(s - top[:, None]).sum(1))).astype(np.float32)
    w = rng.uniform(0.5, 2.0, n).astype(np.float32)
    return z.to(dtype), idx, t, t_lse, w


def to(dev, v):
    return None if v is None else torch.from_numpy(np.ascontiguousarray(v)).to(dev)


def bounds(z, idx, t, T, t_lse, w, stored=False, grad=None):
    """(bound of loss, bound of the gradient before its type's rounding)"""
    z64 = z.double().numpy() / T
    n, vocab = z64.shape
    lb, gb = np.zeros(n), np.zeros((n, vocab))
    for i in range(n):
        if w[i] == 0:
            continue
        fin = z64[i][np.isfinite(z64[i])]
        R = float(fin.max() - fin.min())
        e, delta = (4 * R + 8) * U, (4 * R + 140) * U
        known, p_of, rest, p, ids = orc.distill_targets(idx[i], t[i], vocab, T,
                                                        None if t_lse is None else t_lse[i])
        lse = fin.max() + np.log(np.exp(fin - fin.max()).sum())
        q = np.exp(z64[i] - lse)
        mass = np.abs(np.log(p[p > 0])).dot(p[p > 0]) + np.abs(p * np.where(p > 0, z64[i][ids] - lse, 0)).sum()
        lb[i] = w[i] * T * T * (delta + 2 * U * (mass + 1))
        d = e + delta + (2 * U * (abs(lse) + np.abs(fin).max()) if stored else 0.0)
        out = np.ones(vocab, bool)
        out[known] = False
        share = np.zeros(vocab)
        if t_lse is not None and np.isfinite(z64[i][out]).any() and rest > 0:
            zo = z64[i][out]
            share[out] = rest * np.exp(zo - zo.max()) / np.exp(zo - zo.max()).sum()
        up = 1.0 if grad is None else grad[i]
        gb[i] = w[i] * T * up * ((q + share) * (d + 4 * U))
        gb[i][known] += w[i] * T * up * 2 * U * p_of
    return lb, gb


def half_step(dtype, g):
    if dtype is torch.float32:
        return U * np.abs(g) + 1e-38
    if dtype is torch.float16:
        return np.maximum(2.0 ** -11 * np.abs(g), 2.0 ** -25)
    return 2.0 ** -8 * np.abs(g) + 1e-38


def near(got, want, bound, what):
    got = got.cpu().double().numpy()
    assert np.array_equal(np.isfinite(got), np.isfinite(want)), f"{what}: finite elsewhere"
    f = np.isfinite(want)
    err = np.abs(got[f] - want[f])
    b = (bound * (1 + 2.0 ** -7))[f] + 1e-38
    assert (err <= b).all(), f"{what}: {float((err / b).max()):.3g} of the bound"


def check(dev, z, idx, t, t_lse, w, T, pad=0, shift=0):
    n, vocab = z.shape
    dt = z.dtype
    wide = torch.zeros(n, vocab + pad + shift, dtype=dt)
    wide[:, shift:shift + vocab] = z
    zg = wide.to(dev)[:, shift:shift + vocab]
    kw = dict(temperature=T, t_lse=to(dev, t_lse), weight=to(dev, w))
    got = gq.gptq_distill_loss(zg, to(dev, idx), to(dev, t), want_grad=True, **kw)
    alone = gq.gptq_distill_loss(zg, to(dev, idx), to(dev, t), **kw)
    up = np.random.default_rng(n).uniform(0.5, 2.0, n).astype(np.float32)
    back = gq.gptq_distill_backward(zg, got["stats"], to(dev, idx), to(dev, t), to(dev, up), **kw)
    torch.cuda.synchronize()
    wn = np.ones(n) if w is None else w
    loss, grad = orc.distill(z.double().numpy(), idx, t, T, t_lse, wn)
    lb, gb = bounds(z, idx, t, T, t_lse, wn)
    near(got["loss"], loss, lb + U * np.abs(loss), "loss")
    near(got["dlogits"], grad, gb + half_step(dt, grad), "gradient")
    assert torch.equal(alone["loss"], got["loss"]) and torch.equal(alone["stats"], got["stats"])
    gb2 = bounds(z, idx, t, T, t_lse, wn, stored=True, grad=up)[1]
    g2 = grad * up[:, None].astype(np.float64)
    near(back, g2, gb2 + half_step(dt, g2), "backward")
    return got


CASES = [
    # n, vocab, k, T
    (1, 1, 1, 1.0), (3, 7, 7, 1.0), (2, 64, 5, 0.7), (5, 1000, 1, 2.0), (4, 1003, 100, 1.5),
    (3, 8191, 64, 1.0), (2, 9000, 300, 1.0), (3, 33000, 20, 2.0), (2, 50021, 1024, 1.0),
    (2, 131072, 64, 1.0), (1, 140001, 33, 1.3), (1, 262144, 10, 1.0), (40, 500, 16, 1.0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "n%d_V%d_k%d_T%g" % c)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32],
                         ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_matches_oracle(dev, case, dtype, tail):
    n, vocab, k, T = case
    z, idx, t, t_lse, w = inputs(n, vocab, k, dtype, T, tail)
    if vocab > 10:
        idx[0, k // 2 + 1:] = -1                  # a row that knows less
        idx[-1, 0] = vocab                        # out of range: padding too
    check(dev, z, idx, t, t_lse, w if n > 2 else None, T)


@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (5, 3)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_distill_strided_logits(dev, pad, shift, dtype):
    for vocab in (777, 20000):
        z, idx, t, t_lse, w = inputs(5, vocab, 9, dtype, 1.0, True, seed=2)
        check(dev, z, idx, t, t_lse, w, 1.0, pad, shift)


@pytest.mark.parametrize("tail", [False, True])
def test_rows_that_do_not_count(dev, tail):
    """Weight 0 reads nothing of the row; a row that knows no id has no loss."""
    z, idx, t, t_lse, w = inputs(6, 2000, 8, torch.float32, 1.0, tail, seed=3)
    w[1] = 0.0
    z[1] = float("nan")
    idx[3] = -1
    if tail:
        t_lse[1] = np.nan
    zg = z.to(dev)
    kw = dict(t_lse=to(dev, t_lse), weight=to(dev, w))
    got = gq.gptq_distill_loss(zg, to(dev, idx), to(dev, t), want_grad=True, **kw)
    back = gq.gptq_distill_backward(zg, got["stats"], to(dev, idx), to(dev, t),
                                    torch.ones(6, device=dev), **kw)
    for g in (got["dlogits"], back):
        assert not g[1].any() and bool(torch.isfinite(g).all())
    assert float(got["loss"][1]) == 0.0 and float(got["loss"][3]) == 0.0
    # known to be nothing, the rest class is everything: q (1 - 1 / 1)
    assert float(got["dlogits"][3].abs().max()) <= (1e-6 if tail else 0.0)
    keep = [0, 2, 4, 5]
    z2 = z[keep]
    check(dev, z2, idx[keep], t[keep], None if t_lse is None else t_lse[keep], w[keep], 1.0)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masked_tokens(dev, tail, dtype):
    """Cells of -inf and of the type's lowest value have probability 0 and
    gradient 0; one that the teacher likes makes the loss inf."""
    z, idx, t, t_lse, w = inputs(5, 3001, 8, dtype, 1.0, tail, seed=4)
    low = torch.finfo(dtype).min
    for r in range(5):
        gone = np.setdiff1d(np.arange(0, 3001, 3), idx[r])
        z[r, gone] = -float("inf") if r != 2 else low
    t[3, 2] = -np.inf                    # known to be impossible
    ref = z.clone()
    ref[2][ref[2] == low] = -float("inf")     # exp(low - max) is 0 in fp64 as well
    check_z = check(dev, ref, idx, t, t_lse, w, 1.0)
    got = gq.gptq_distill_loss(z.to(dev), to(dev, idx), to(dev, t), t_lse=to(dev, t_lse),
                               weight=to(dev, w), want_grad=True)
    assert torch.equal(got["loss"], check_z["loss"]) and torch.equal(got["dlogits"], check_z["dlogits"])
    z[4, idx[4, 0]] = -float("inf")
    got = gq.gptq_distill_loss(z.to(dev), to(dev, idx), to(dev, t), t_lse=to(dev, t_lse),
                               weight=to(dev, w), want_grad=True)
    assert float(got["loss"][4]) == float("inf") and bool(torch.isfinite(got["dlogits"][4].float()).all())


def test_confident_student_and_full_knowledge(dev):
    """Nearly all student mass on the known ids (the rest's share is a sum of
    its own, not a difference), and a teacher known whole (no rest)."""
    z, idx, t, t_lse, w = inputs(4, 5000, 6, torch.float32, 1.0, True, seed=5)
    for r in range(4):
        z[r, idx[r]] += 18.0 + 10.0 * r
    check(dev, z, idx, t, t_lse, w, 1.0)
    z, idx, t, t_lse, w = inputs(3, 300, 300, torch.float32, 1.0, True, seed=6)
    got = gq.gptq_distill_loss(z.to(dev), to(dev, idx), to(dev, t), t_lse=to(dev, t_lse),
                               want_grad=True)
    loss, grad = orc.distill(z.double().numpy(), idx, t, 1.0)
    # t_lse in fp32 is off by u |t_lse|, and the probabilities by as much
    assert np.abs(got["loss"].cpu().double().numpy() - loss).max() < 200 * U
    assert np.abs(got["dlogits"].cpu().double().numpy() - grad).max() < 200 * U


def test_an_id_named_twice_counts_twice(dev):
    z, idx, t, t_lse, w = inputs(3, 900, 6, torch.float32, 1.0, False, seed=7)
    idx[1, 3] = idx[1, 0]
    idx[2, 5] = idx[2, 4]
    check(dev, z, idx, t, None, w, 1.0)
    z, idx, t, t_lse, w = inputs(3, 900, 6, torch.float32, 1.0, True, seed=8)
    idx[0, 2] = idx[0, 5]
    t[0, 2] -= 3.0
    check(dev, z, idx, t, t_lse, w, 1.0)


def test_not_finite_rows_stay_alone(dev):
    z, idx, t, t_lse, w = inputs(5, 4000, 6, torch.bfloat16, 1.0, True, seed=9)
    first = gq.gptq_distill_loss(z.to(dev), to(dev, idx), to(dev, t), t_lse=to(dev, t_lse), want_grad=True)
    z[1, 77] = float("nan")
    z[3] = -float("inf")
    got = gq.gptq_distill_loss(z.to(dev), to(dev, idx), to(dev, t), t_lse=to(dev, t_lse), want_grad=True)
    assert torch.isnan(got["loss"][1]) and torch.isnan(got["loss"][3])
    for r in (0, 2, 4):
        assert torch.equal(got["loss"][r], first["loss"][r])
        assert torch.equal(got["dlogits"][r], first["dlogits"][r])


@pytest.mark.parametrize("vocab", [700, 30000, 140001])
def test_in_place_captured_and_other_memory(dev, vocab):
    """The gradient over the logits, a captured call replayed on other logits,
    and rows behind the last one left as they were."""
    z, idx, t, t_lse, w = inputs(4, vocab, 12, torch.bfloat16, 1.0, True, seed=10)
    ix, tt, tl = to(dev, idx), to(dev, t), to(dev, t_lse)
    want = gq.gptq_distill_loss(z.to(dev), ix, tt, t_lse=tl, want_grad=True)
    big = torch.full((6, vocab), 3.0, dtype=torch.bfloat16, device=dev)
    big[:4] = z.to(dev)
    got = gq.gptq_distill_loss(big[:4], ix, tt, t_lse=tl, dlogits=big[:4])
    assert torch.equal(got["loss"], want["loss"]) and torch.equal(big[:4], want["dlogits"])
    assert bool((big[4:] == 3.0).all())
    zg = z.to(dev)
    out = torch.empty_like(zg)
    up = torch.ones(4, device=dev)
    g = torch.cuda.CUDAGraph()
    gq.gptq_distill_loss(zg, ix, tt, t_lse=tl)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        cap = gq.gptq_distill_loss(zg, ix, tt, t_lse=tl, dlogits=out)
        back = gq.gptq_distill_backward(zg, cap["stats"], ix, tt, up, t_lse=tl)
    for k in range(3):
        zg.copy_((z * (1.0 + 0.1 * k)).to(dev))
        g.replay()
        torch.cuda.synchronize()
        e = gq.gptq_distill_loss(zg, ix, tt, t_lse=tl, want_grad=True)
        b = gq.gptq_distill_backward(zg, e["stats"], ix, tt, up, t_lse=tl)
        torch.cuda.synchronize()
        assert torch.equal(e["loss"], cap["loss"]) and torch.equal(e["dlogits"], out)
        assert torch.equal(b, back)


def test_gradient_is_the_loss_s_difference(dev):
    """fp32 logits moved by h = 1/8 along random directions: the difference of
    the losses is grad . step within the third derivative's share, h^2 |step|^3
    / 6 <= 4e-4 for steps of at most 1/8 (the third derivative of a log-sum-exp
    along a direction s is at most 2 max |s|^3), and the losses' rounding."""
    z, idx, t, t_lse, w = inputs(4, 600, 12, torch.float32, 1.0, True, seed=11)
    rng = np.random.default_rng(12)
    step = torch.from_numpy(rng.uniform(-1, 1, size=z.shape).astype(np.float32) / 8)
    up, down = z + step, z - step
    ix, tt, tl = to(dev, idx), to(dev, t), to(dev, t_lse)
    grad = gq.gptq_distill_loss(z.to(dev), ix, tt, t_lse=tl, want_grad=True)["dlogits"].cpu().double()
    a = gq.gptq_distill_loss(up.to(dev), ix, tt, t_lse=tl)["loss"].cpu().double()
    b = gq.gptq_distill_loss(down.to(dev), ix, tt, t_lse=tl)["loss"].cpu().double()
    real = ((up.double() - down.double()) / 2 * grad).sum(1)
    # two log-sum-exps (all cells, the rest): (1 + 1) 2 s^3 / 6 each side
    assert float(((a - b) / 2 - real).abs().max()) <= 4 * (1 / 8) ** 3 / 6 + 1e-4


@pytest.mark.parametrize("case", [(300, 9000, torch.bfloat16), (300, 4100, torch.float32),
                                  (257, 30001, torch.float16), (2, 40000, torch.bfloat16),
                                  (3, 20003, torch.float32)],
                         ids=lambda c: "n%d_V%d_%s" % (c[0], c[1], str(c[2])[6:]))
def test_many_and_middling_rows(dev, case):
    """Rows that share a CU, and those of the length between."""
    n, vocab, dtype = case
    z, idx, t, t_lse, w = inputs(n, vocab, 5, dtype, 1.0, True, seed=13)
    w[n // 2] = 0.0
    check(dev, z, idx, t, t_lse, w, 1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("vocab", [900, 9000, 140001])
def test_log_probabilities_as_logits(dev, dtype, vocab):
    """No cell above 0, some at 0 or -0: the maximum is taken all the same."""
    z, idx, t, t_lse, w = inputs(4, vocab, 7, dtype, 1.0, True, seed=14)
    z = (z.double() - torch.logsumexp(z.double(), 1, keepdim=True)).to(dtype)
    z[1, 11] = -0.0
    z[2, 5] = 0.0
    z[2, 6] = -0.0
    z[3, 1::2] = -float("inf")
    idx[3] = idx[3] // 2 * 2
    idx[3] = np.where(np.isin(np.arange(7), np.unique(idx[3], return_index=True)[1]), idx[3], -1)
    check(dev, z, idx, t, t_lse, w, 1.0)


@pytest.mark.parametrize("shift", [1, 3])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradient_at_another_alignment(dev, shift, dtype):
    z, idx, t, t_lse, w = inputs(3, 5003, 7, dtype, 1.0, True, seed=15)
    ix, tt, tl = to(dev, idx), to(dev, t), to(dev, t_lse)
    want = gq.gptq_distill_loss(z.to(dev), ix, tt, t_lse=tl, want_grad=True)
    wide = torch.full((4, 5003 + 9), 3.0, dtype=dtype, device=dev)
    out = wide[:3, shift:shift + 5003]
    got = gq.gptq_distill_loss(z.to(dev), ix, tt, t_lse=tl, dlogits=out)
    assert torch.equal(out, want["dlogits"]) and torch.equal(got["loss"], want["loss"])
    out.zero_()
    assert float(wide.double().sum()) == 3.0 * (5003 + 9 + 3 * 9)


@pytest.mark.parametrize("vocab", [900, 9000, 140001])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("far", [2.0 ** 20, 2.0 ** 22, -2.0 ** 22])
def test_logits_far_from_zero(dev, vocab, tail, far):
    """Only differences of logits count: whole numbers moved by a large one
    (exact in fp32) keep the loss and both gradients, within the bounds of the
    logits that were not moved (the stats of such rows are not relied on)."""
    z, idx, t, t_lse, w = inputs(3, vocab, 9, torch.float32, 2.0, tail, seed=16, scale=6.0)
    z = torch.round(z)
    kw = dict(temperature=2.0, t_lse=to(dev, t_lse), weight=to(dev, w))
    zg = (z + far).to(dev)
    got = gq.gptq_distill_loss(zg, to(dev, idx), to(dev, t), want_grad=True, **kw)
    back = gq.gptq_distill_backward(zg, got["stats"], to(dev, idx), to(dev, t),
                                    torch.ones(3, device=dev), **kw)
    loss, grad = orc.distill(z.double().numpy(), idx, t, 2.0, t_lse, w)
    lb, gb = bounds(z, idx, t, 2.0, t_lse, w)
    near(got["loss"], loss, lb + U * np.abs(loss), "loss")
    near(got["dlogits"], grad, gb + half_step(torch.float32, grad), "gradient")
    near(back, grad, gb + half_step(torch.float32, grad), "backward")


@pytest.mark.parametrize("T", [0.5, 1.0, 2.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("vocab", [1000, 16000, 140000])
def test_a_row_of_nothing_but_the_lowest_value(dev, dtype, T, vocab):
    """Equal logits, however low: q = 1 / vocab.  A second row of the lowest
    value but for one cell at half of it: all mass there."""
    z = torch.full((2, vocab), torch.finfo(dtype).min, dtype=dtype, device=dev)
    z[1, 7] = torch.finfo(dtype).min / 2
    ti = torch.tensor([[3, 5], [7, -1]], dtype=torch.int32, device=dev)
    tt = torch.zeros(2, 2, device=dev)
    got = gq.gptq_distill_loss(z, ti, tt, temperature=T, want_grad=True)
    back = gq.gptq_distill_backward(z, got["stats"], ti, tt, torch.ones(2, device=dev), temperature=T)
    loss = got["loss"].cpu().double()
    # log 1/2 - log 1/vocab, each log-sum-exp within 140 u and its own rounding
    want = T * T * np.log(vocab / 2)
    assert abs(float(loss[0]) - want) <= T * T * 160 * U + U * want
    assert abs(float(loss[1])) <= T * T * 160 * U
    for g in (got["dlogits"], back):
        g = g.cpu().double()
        q = T / vocab
        half = float(half_step(dtype, np.array(q))) + 160 * U * q
        assert float((g[0, 8:] - q).abs().max()) <= half
        hot = T * (0.5 - 1 / vocab)
        assert float((g[0, 3] + hot).abs()) <= float(half_step(dtype, np.array(hot))) + 160 * U
        assert float(g[1].abs().max()) <= T * 160 * U


def without_rest(case, vocab, k, dtype, seed=17):
    """Rows whose class of all others is left out: every other cell -inf, no
    other cell, or known probabilities beyond 1."""
    z, idx, t, _, w = inputs(4, k if case == "whole" else vocab, k, dtype, 1.5, False, seed=seed)
    if case == "masked":
        for r in range(4):
            z[r, np.setdiff1d(np.arange(vocab), idx[r])] = -float("inf")
    known = np.log(np.exp(t.astype(np.float64) / 1.5).sum(1))
    off = np.array([0.3, 0.7, 1.5, 3.0]) * (-0.5 if case == "over" else 1)
    return z, idx, t, (known + off).astype(np.float32), w


@pytest.mark.parametrize("case,vocab,k", [("masked", 700, 9), ("masked", 9001, 200), ("masked", 140001, 5),
                                          ("whole", 0, 1), ("whole", 0, 40), ("whole", 0, 1000),
                                          ("over", 700, 9), ("over", 20003, 64), ("over", 140001, 5)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32],
                         ids=["bf16", "f16", "f32"])
def test_without_the_rest_class(dev, case, vocab, k, dtype):
    """Held against the oracle; the target's sum P stands before q and the
    log-sum-exp, and so before their errors."""
    T = 1.5
    z, idx, t, t_lse, w = without_rest(case, vocab, k, dtype)
    kw = dict(temperature=T, t_lse=to(dev, t_lse), weight=to(dev, w))
    got = gq.gptq_distill_loss(z.to(dev), to(dev, idx), to(dev, t), want_grad=True, **kw)
    up = np.array([0.5, 1.0, 1.5, 2.0], np.float32)
    back = gq.gptq_distill_backward(z.to(dev), got["stats"], to(dev, idx), to(dev, t), to(dev, up), **kw)
    torch.cuda.synchronize()
    loss, grad = orc.distill(z.double().numpy(), idx, t, T, t_lse, w)
    lb, gb = bounds(z, idx, t, T, t_lse, w)
    P = np.maximum(1.0, np.exp(t.astype(np.float64) / T - t_lse[:, None]).sum(1))
    near(got["loss"], loss, lb * P + U * np.abs(loss), "loss")
    near(got["dlogits"], grad, gb * P[:, None] + half_step(dtype, grad), "gradient")
    gb2 = bounds(z, idx, t, T, t_lse, w, stored=True, grad=up)[1]
    g2 = grad * up[:, None].astype(np.float64)
    near(back, g2, gb2 * P[:, None] + half_step(dtype, g2), "backward")


@pytest.mark.parametrize("case", ["masked", "whole", "over"])
def test_gradient_without_the_rest_class_is_the_loss_s_difference(dev, case):
    """As for rows with that class: steps of at most 1/8 on z, 1/12 on z / T, the
    third derivative of P log-sum-exps at most 2 P (step / T)^3, times T^2 w."""
    T = 1.5
    z, idx, t, t_lse, w = without_rest(case, 600, 12, torch.float32)
    rng = np.random.default_rng(18)
    step = torch.from_numpy(rng.uniform(-1, 1, size=z.shape).astype(np.float32) / 8)
    up, down = z + step, z - step
    kw = dict(temperature=T, t_lse=to(dev, t_lse), weight=to(dev, w))
    ix, tt = to(dev, idx), to(dev, t)
    grad = gq.gptq_distill_loss(z.to(dev), ix, tt, want_grad=True, **kw)["dlogits"].cpu().double()
    a = gq.gptq_distill_loss(up.to(dev), ix, tt, **kw)["loss"].cpu().double()
    b = gq.gptq_distill_loss(down.to(dev), ix, tt, **kw)["loss"].cpu().double()
    move = torch.where(torch.isfinite(z), (up.double() - down.double()) / 2, 0.0)
    P = torch.from_numpy(np.exp(t.astype(np.float64) / T - t_lse[:, None]).sum(1))
    bound = torch.from_numpy(w).double() * T * T * (2 * P * (1 / 12) ** 3 / 6 + (1 + P) * 1e-5)
    assert bool((((a - b) / 2 - (move * grad).sum(1)).abs() <= bound).all())


@pytest.mark.parametrize("vocab", [900, 9000, 140001])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32],
                         ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [0.5, 1.0])
@pytest.mark.parametrize("low", ["lowest", "far", "half"])
def test_all_others_far_below_the_known_ids(dev, vocab, dtype, T, low):
    """The cells outside S at the type's lowest value (a mask that is no -inf),
    some of them twice as low as the others, or moved down by 2^14: q_r is 0,
    and the cells get -w T p_r times their softmax among themselves, in both
    passes.  A cell's exponential is off by (4 R + 8) u, R their own range, the
    sum by 140 u in all."""
    n, k = 3, 6
    rng = np.random.default_rng([19, vocab])
    idx = np.stack([rng.permutation(vocab)[:k] for _ in range(n)]).astype(np.int32)
    t = rng.normal(size=(n, k)).astype(np.float32)
    out = np.ones((n, vocab), bool)
    out[np.arange(n)[:, None], idx] = False
    z = torch.zeros(n, vocab, dtype=dtype)
    own = np.zeros((n, vocab))                       # the cells' logits but for a common part
    if low == "far":
        own = rng.integers(0, 2, size=(n, vocab)) * 16.0
        z[:] = torch.from_numpy(own - 2.0 ** 14).to(dtype)
        own = (z.double().numpy() + 2.0 ** 14) / T   # bf16 and fp16 keep what they can
    else:
        bottom = torch.finfo(dtype).min
        z[:] = bottom
        if low == "half":
            z[:, 1::2] = bottom / 2
            own[:, 0::2] = -np.inf
    zs = torch.from_numpy(rng.normal(size=(n, k)).astype(np.float32)).to(dtype)
    z[torch.arange(n)[:, None], torch.from_numpy(idx).long()] = zs
    s = t.astype(np.float64) / T
    t_lse = (np.log(np.exp(s).sum(1)) + np.log(1 / np.array([0.7, 0.5, 0.9]))).astype(np.float32)
    w = np.array([1.0, 0.5, 0.25], np.float32)
    kw = dict(temperature=T, t_lse=to(dev, t_lse), weight=to(dev, w))
    got = gq.gptq_distill_loss(z.to(dev), to(dev, idx), to(dev, t), want_grad=True, **kw)
    back = gq.gptq_distill_backward(z.to(dev), got["stats"], to(dev, idx), to(dev, t),
                                    torch.ones(n, device=dev), **kw)
    torch.cuda.synchronize()
    p = np.exp(s - t_lse[:, None])
    q = np.exp(zs.double().numpy() / T)
    want, bound = np.zeros((n, vocab)), np.zeros((n, vocab))
    for r in range(n):
        e = np.where(out[r], np.exp(own[r] - own[r][out[r]].max()), 0.0)
        R = np.ptp(own[r][out[r] & np.isfinite(own[r])])
        want[r] = -w[r] * T * (1 - p[r].sum()) * e / e.sum()
        want[r, idx[r]] = w[r] * T * (q[r] / q[r].sum() - p[r])
        bound[r] = (4 * R + 160) * U * np.abs(want[r])
        bound[r, idx[r]] = 160 * U * w[r] * T
    assert bool(torch.isfinite(got["loss"]).all())
    near(got["dlogits"], want, bound + half_step(dtype, want), "gradient")
    near(back, want, bound + half_step(dtype, want), "backward")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32],
                         ids=["bf16", "f16", "f32"])
def test_long_rows_sums_do_not_drift(dev, dtype):
    """The longest rows: the first half of the cells at 0, the others with an
    exponential of 1/2 + 7e-6, of which a running fp32 sum in the hundreds loses
    all but the half, every time (84 u of a thread's 256 cells).  Summed in
    fp64 beyond a few cells the row is off by an exponential's (4 R + 8) u, R =
    log 2, and the few cells' 16 u."""
    V = 262144
    T = float(np.float32(-1.0 / np.log(0.5 + 7e-6)))
    z = torch.zeros(2, V, dtype=dtype, device=dev)
    z[:, V // 2:] = -1.0
    ti = torch.tensor([[0, V - 1], [5, -1]], dtype=torch.int32, device=dev)
    tt = torch.zeros(2, 2, device=dev)
    got = gq.gptq_distill_loss(z, ti, tt, temperature=T, want_grad=True)
    lse = np.log(V / 2 * (1.0 + np.exp(-1.0 / T)))
    loss = T * T * np.array([np.log(0.5) + 0.5 / T + lse, lse])
    off = (4 * np.log(2) + 24) * U
    err = np.abs(got["loss"].cpu().double().numpy() - loss)
    assert (err <= T * T * off + U * loss).all(), err / U
    grad = np.where(np.arange(V) < V // 2, 1.0, np.exp(-1.0 / T)) * T * np.exp(-lse)
    g = got["dlogits"].cpu().double().numpy()
    rest = np.ones(V, bool)
    rest[[0, 5, V - 1]] = False
    # the cells' own exponential and the sum's
    bound = 2 * off * grad + half_step(dtype, grad)
    assert (np.abs(g - grad)[:, rest] <= bound[rest]).all()
