"""Top-k gating and its gradient against 64-bit references."""

import math

import pytest
import torch

import combine_topk_ids_expert_amd as mx
from tests import experts_util as eu

pytestmark = pytest.mark.gpu

DEV = eu.DEV
INF = math.inf


def _reference(x, k, scoring, bias, renormalize, scale):
    """ids, float64 weights of logits x (CPU)."""
    x = x.double()
    x = torch.where(torch.isnan(x), -INF, x)
    key = x
    if bias is not None:
        key = torch.where(x > -INF, 1 / (1 + torch.exp(-x)) + bias.double(), -INF)
        key = torch.where(torch.isnan(key), -INF, key)
        x = torch.where(key > -INF, x, -INF)
    top, ids = torch.sort(key, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    on = top > -INF
    chosen = torch.gather(x, 1, ids)
    if scoring == "softmax":
        m = x.amax(1, keepdim=True)
        def e(v):
            return torch.where(v == m, torch.where(m > -INF, 1.0, 0.0), torch.exp(v - m)).nan_to_num(0.0)
        p = torch.where(on, e(chosen), 0.0)
        total = (p if renormalize else e(x)).sum(1, keepdim=True)
    else:
        p = torch.where(on, 1 / (1 + torch.exp(-chosen)), 0.0)
        total = p.sum(1, keepdim=True) if renormalize else torch.ones(len(x), 1, dtype=torch.float64)
    w = torch.where(total > 0, p / total, 0.0) * scale
    return torch.where(on, ids, -1).int(), w


def _tolerance(x, E, w):
    """exp(l - m): the difference is rounded (|l - m| 2^-24 in the exponent),
    the exponential to two steps; sums of up to E terms, quotient and scale."""
    span = x.double().nan_to_num(0.0, 0.0, 0.0).abs().amax(1, keepdim=True) * 2
    return w.abs() * (span + E + 8) * eu.U32 + 1e-37


def _run(x, k, **kw):
    ids = torch.full((len(x), k), 99, dtype=torch.int32, device=DEV)
    w = torch.full((len(x), k), math.nan, device=DEV)
    mx.topk_gating(x.to(DEV), ids, w, **kw)
    return ids, w


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 8, 8), (65, 64, 1), (33, 65, 6), (17, 128, 8),
                                   (9, 256, 8), (5, 288, 8), (7, 300, 10), (4, 511, 64),
                                   (6, 1024, 33), (1000, 160, 6)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("scoring,bias,renormalize,scale",
                         [("softmax", False, True, 1.0), ("softmax", False, False, 2.5),
                          ("sigmoid", True, True, 2.5), ("sigmoid", False, False, 1.0)])
def test_topk_gating(T, E, k, dtype, scoring, bias, renormalize, scale):
    print("case:", T, E, k, dtype, scoring, bias, renormalize, scale, flush=True)
    x = eu.normal((T, E), dtype, T + E, 2.0)
    b = eu.normal((E,), torch.float32, 5, 0.1) if bias else None
    ids, w = _run(x, k, scoring=scoring, bias=None if b is None else b.to(DEV),
                  renormalize=renormalize, scale=scale)
    want_ids, want = _reference(x, k, scoring, b, renormalize, scale)
    assert torch.equal(ids.cpu(), want_ids)
    assert ((w.cpu().double() - want).abs() <= _tolerance(x, E, want)).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("E", [12, 130])
def test_ties_masks_and_infinities(scoring, renormalize, E):
    """Equal logits (signed zeros among them) by lower index; -inf, the type's
    lowest value, NaN and +inf; rows with fewer than k experts left and none."""
    k = 6
    low = torch.finfo(torch.float32).min
    x = torch.zeros(10, E)
    x[1, ::2] = -0.0
    x[2] = -INF
    x[3] = math.nan
    x[4, 3:] = -INF
    x[5] = low
    x[6, [2, 7]] = INF
    x[7, [1, 4]] = math.nan
    x[8] = eu.normal((E,), torch.float32, 1).round()
    x[9] = -INF
    x[9, E - 1] = low
    ids, w = _run(x, k, scoring=scoring, renormalize=renormalize)
    want_ids, want = _reference(x, k, scoring, None, renormalize, 1.0)
    assert torch.equal(ids.cpu(), want_ids)
    got = w.cpu().double()
    assert torch.isfinite(got).all()
    assert ((got - want).abs() <= _tolerance(x.clamp(-8, 8), E, want)).all()
    assert (ids[2] == -1).all() and (w[2] == 0).all()
    assert ids[4].tolist() == [0, 1, 2, -1, -1, -1]


def test_bias_selects_only_and_may_switch_off():
    x = eu.normal((50, 96), torch.float32, 3)
    b = eu.normal((96,), torch.float32, 4)
    b[7], b[11], b[13] = -INF, math.nan, 3.0
    ids, w = _run(x, 8, scoring="sigmoid", bias=b.to(DEV))
    want_ids, want = _reference(x, 8, "sigmoid", b, True, 1.0)
    assert torch.equal(ids.cpu(), want_ids)
    assert not ((ids == 7) | (ids == 11)).any() and (ids == 13).any(1).all()
    assert ((w.cpu().double() - want).abs() <= _tolerance(x, 96, want)).all()


def test_keys_closer_than_float32():
    """Sigmoids near 1 differ by less than float32 resolves: the bias decides
    only among what float64 holds equal."""
    x = torch.full((1, 64), 18.0)
    x[0, 40] = 18.5
    x[0, 9] = 18.25
    ids, _ = _run(x, 3, scoring="sigmoid", bias=torch.full((64,), 0.5, device=DEV))
    assert ids.tolist() == [[40, 9, 0]]


def _gradient(x, ids, g, scoring, renormalize, scale):
    """The formula's gradient by float64 autograd over each token's picks."""
    x = x.double()
    out = torch.zeros_like(x)
    for t in range(len(x)):
        v = x[t].clone()
        able = (v > -INF)                                        # not NaN, not -inf
        pick = [j for j in range(ids.shape[1])
                if 0 <= int(ids[t, j]) < x.shape[1] and bool(able[int(ids[t, j])])]
        if not pick:
            continue
        idx = torch.tensor([int(ids[t, j]) for j in pick])
        keep = able.nonzero()[:, 0]
        leaf = v[keep].clone().requires_grad_()
        full = torch.zeros_like(v).index_put((keep,), leaf)
        chosen = full[idx]
        if scoring == "softmax":
            w = torch.softmax(chosen, 0) if renormalize else \
                torch.exp(chosen - torch.logsumexp(leaf, 0))
        else:
            s = torch.sigmoid(chosen)
            w = s / s.sum() if renormalize else s
        (scale * (w * g[t, pick].double()).sum()).backward()
        out[t, keep] = leaf.grad
    return out


def _gradient_tolerance(x, g, E, scale, dtype, want):
    """Each weight is off by a relative (span + E + 8) 2^-24 (see _tolerance);
    the gradient is a sum of at most 2 k products of weights (at most 1) and
    g, of which 1 / sum s (at least 1 / max s) takes part for sigmoids."""
    span = x.double().nan_to_num(0.0, 0.0, 0.0).abs().amax(1, keepdim=True) * 2
    size = g.double().abs().sum(1, keepdim=True) * scale
    return size * (span + E + 2 * g.shape[1] + 16) * eu.U32 * 2 + eu.rounding(want, dtype)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 8, 8), (33, 65, 6), (17, 128, 8), (5, 288, 8),
                                   (4, 511, 64), (3, 1024, 10)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("scoring,renormalize,scale",
                         [("softmax", True, 1.0), ("softmax", False, 2.5),
                          ("sigmoid", True, 2.5), ("sigmoid", False, 1.0)])
def test_topk_gating_backward(T, E, k, dtype, scoring, renormalize, scale):
    print("case: backward", T, E, k, dtype, scoring, renormalize, scale, flush=True)
    x = eu.normal((T, E), dtype, T * E, 2.0)
    ids, _ = _run(x, k, scoring=scoring, renormalize=renormalize, scale=scale)
    g = eu.normal((T, k), torch.float32, 6)
    out = torch.full((T, E), math.nan, dtype=dtype, device=DEV)
    mx.topk_gating_backward(x.to(DEV), ids, g.to(DEV), out, scoring=scoring,
                            renormalize=renormalize, scale=scale)
    want = _gradient(x, ids.cpu(), g, scoring, renormalize, scale)
    tol = _gradient_tolerance(x, g, E, scale, dtype, want)
    assert ((out.cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_backward_of_masked_rows_and_untrusted_ids(scoring, renormalize):
    E, k = 70, 4
    x = eu.normal((6, E), torch.float32, 7)
    x[0] = -INF
    x[1, 2:] = -INF
    x[2, 5] = math.nan
    ids = torch.tensor([[0, 1, 2, 3], [0, 1, -1, -1], [4, 5, 6, 7], [3, 3, 9, 3],
                        [-5, E, 2**30, 11], [-1, -1, -1, -1]], dtype=torch.int32)
    g = eu.normal((6, k), torch.float32, 8)
    out = torch.full((6, E), math.nan, device=DEV)
    mx.topk_gating_backward(x.to(DEV), ids.to(DEV), g.to(DEV), out, scoring=scoring,
                            renormalize=renormalize)
    want = _gradient(x, ids, g, scoring, renormalize, 1.0)
    tol = _gradient_tolerance(x, g, E, 1.0, torch.float32, want)
    assert ((out.cpu().double() - want).abs() <= tol).all()
    assert (out[0] == 0).all() and (out[5] == 0).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_backward_against_differences(scoring, renormalize):
    """Central differences of the forward call: (w(x + h) - w(x - h)) / 2h is
    off by h^2 / 6 of a third derivative (below 1 here) and by the weights'
    float32 roundings over h."""
    T, E, k, h = 4, 20, 5, 2.0 ** -6
    x = eu.normal((T, E), torch.float32, 9)
    ids, _ = _run(x, k, scoring=scoring, renormalize=renormalize)
    g = eu.normal((T, k), torch.float32, 10)
    out = torch.empty(T, E, device=DEV)
    mx.topk_gating_backward(x.to(DEV), ids, g.to(DEV), out, scoring=scoring,
                            renormalize=renormalize)
    size = g.abs().sum(1)
    for e in range(E):
        side = []
        for s in (h, -h):
            y = x.clone()
            y[:, e] += s
            i, w = _run(y, E, scoring=scoring, renormalize=False)
            p = torch.zeros(T, E, device=DEV).scatter_(1, i.long(), w).cpu().double()
            p = torch.gather(p, 1, ids.cpu().long())
            if renormalize:
                p = p / p.sum(1, keepdim=True)
            side.append((p * g.double()).sum(1))
        diff = (side[0] - side[1]) / (2 * h)
        assert ((out[:, e].cpu().double() - diff).abs() <= size * (h * h / 6 + 64 * eu.U32 / h)).all()


def test_bindings_refuse():
    x = torch.zeros(4, 8, device=DEV)
    ids = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    w = torch.zeros(4, 2, device=DEV)
    for bad, kind in (
        (lambda: mx.topk_gating(x.double(), ids, w), TypeError),
        (lambda: mx.topk_gating(x, ids.long(), w), TypeError),
        (lambda: mx.topk_gating(x, ids, w.half()), ValueError),
        (lambda: mx.topk_gating(x, ids[:3].contiguous(), w), ValueError),
        (lambda: mx.topk_gating(x, ids, w, scoring="relu"), ValueError),
        (lambda: mx.topk_gating(x, ids, w, bias=torch.zeros(8, device=DEV)), ValueError),
        (lambda: mx.topk_gating(x, ids, w, scoring="sigmoid", bias=torch.zeros(7, device=DEV)),
         ValueError),
        (lambda: mx.topk_gating(x, torch.zeros(4, 9, dtype=torch.int32, device=DEV),
                                torch.zeros(4, 9, device=DEV)), mx.MxError),
        (lambda: mx.topk_gating(x[:, ::2], ids, w), ValueError),
        (lambda: mx.topk_gating_backward(x, ids, w, x.half()), ValueError),
    ):
        with pytest.raises(kind):
            bad()
    none = torch.empty(0, 8, device=DEV)
    mx.topk_gating(none, ids[:0], w[:0])
