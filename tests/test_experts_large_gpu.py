"""Arrays past 2^31 elements: rows, weights, results and logits whose offsets do
not fit 32 bits.  Only the far end is computed and compared; the near end keeps
what it held."""

import pytest
import torch

import combine_topk_ids_expert_amd as mx
from tests import experts_util as eu

pytestmark = pytest.mark.gpu

DEV = eu.DEV
BF16, F32 = torch.bfloat16, torch.float32
LIVE = 40


def _far(rows, width, dtype, seed):
    """A tensor of rows x width whose last LIVE rows are N(0, 1)."""
    t = torch.empty(rows, width, dtype=dtype, device=DEV)
    t[:4] = 7.0
    end = eu.normal((LIVE, width), dtype, seed)
    t[rows - LIVE:] = end.to(DEV)
    return t, end


def _offsets(rows):
    return torch.tensor([rows - LIVE, rows - LIVE, rows], dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("n,k", [(48, 2304), (2304, 64)])
def test_far_rows(n, k):
    rows = (1 << 20) + 64
    print("case: far rows", rows, n, k, flush=True)
    x, end = _far(rows, k, BF16, 1)
    w = eu.normal((2, n, k), BF16, 2)
    out = torch.empty(rows, n, dtype=F32, device=DEV)
    out[:4] = 7.0
    mx.grouped_gemm(x, w.to(DEV), _offsets(rows), out)
    a, b = end.double(), w[1].double()
    eu.check(out[rows - LIVE:], a @ b.T, k * eu.U32 * (a.abs() @ b.abs().T), F32)
    assert (out[:4] == 7.0).all()
    wt = w.transpose(1, 2).contiguous().to(DEV)
    out[rows - LIVE:] = 0
    mx.grouped_gemm(x, wt, _offsets(rows), out, transpose_weight=True)
    eu.check(out[rows - LIVE:], a @ b.T, k * eu.U32 * (a.abs() @ b.abs().T), F32)


def test_far_rows_of_gradients():
    rows, n, k = (1 << 20) + 64, 2304, 48
    print("case: far rows of gradients", flush=True)
    d, dend = _far(rows, n, BF16, 3)
    x, xend = _far(rows, k, BF16, 4)
    g = torch.full((2, n, k), 5.0, device=DEV)
    mx.grouped_gemm_wgrad(d, x, _offsets(rows), g)
    a, b = dend.double(), xend.double()
    eu.check(g[1], a.T @ b, LIVE * eu.U32 * (a.abs().T @ b.abs()), F32)
    assert (g[0] == 0).all()
    gu, guend = _far(rows, 2 * n, BF16, 5)
    out = torch.empty_like(gu)
    out[:4] = 7.0
    mx.silu_mul_backward(d, gu, _offsets(rows), out)
    gate, up, s = guend[:, :n].double(), guend[:, n:].double(), torch.sigmoid(guend[:, :n].double())
    want = torch.cat((a * up * s * (1 + gate * (1 - s)), a * gate * s), 1)
    eu.check(out[rows - LIVE:], want, want.abs() * 2 ** -18 + 2 ** -20 * (a.abs().repeat(1, 2)), BF16)
    assert (out[:4] == 7.0).all()


def test_far_experts():
    E, n, k = 70, 8192, 4096
    print("case: far experts", flush=True)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[E] = 3
    x = eu.normal((3, k), BF16, 6)
    w = torch.empty(E, n, k, dtype=BF16, device=DEV)
    end = eu.normal((n, k), BF16, 7)
    w[E - 1] = end.to(DEV)
    out = torch.empty(3, n, dtype=F32, device=DEV)
    mx.grouped_gemm(x.to(DEV), w, off, out)
    a, b = x.double(), end.double()
    eu.check(out, a @ b.T, k * eu.U32 * (a.abs() @ b.abs().T), F32)
    del w
    g = torch.full((E, n, k), 5.0, device=DEV)
    d = eu.normal((3, n), BF16, 8)
    mx.grouped_gemm_wgrad(d.to(DEV), x.to(DEV), off, g)
    c = d.double()
    eu.check(g[E - 1], c.T @ a, 3 * eu.U32 * (c.abs().T @ a.abs()), F32)
    assert (g[:E - 1] == 0).all()


def test_far_experts_in_4_bits():
    E, n, k, group = 140, 8192, 4096, 128
    print("case: far experts in 4 bits", flush=True)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[E] = 3
    x = eu.normal((3, k), BF16, 9)
    w = torch.empty(E, n, k // 2, dtype=torch.uint8, device=DEV)
    sc = torch.ones(E, n, k // group, dtype=BF16, device=DEV)
    g = torch.Generator().manual_seed(10)
    end = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    w[E - 1] = end.to(DEV)
    out = torch.empty(3, n, dtype=BF16, device=DEV)
    mx.grouped_gemm_w4(x.to(DEV), w, sc, off, out)
    q = torch.stack((end & 15, end >> 4), -1).view(n, k).double() - 8
    a = x.double()
    err = 12 * eu.U32 * a.abs().sum(1, keepdim=True) * 144 + 33 * eu.U32 * (a.abs() @ q.abs().T)
    eu.check(out, a @ q.T, err, BF16)


def test_far_tokens():
    """More tokens than one launch takes, and logits past 2^31."""
    T, E = (1 << 25) + 100, 64
    print("case: far tokens", flush=True)
    x = torch.zeros(T, E, dtype=torch.float16, device=DEV)
    places = [0, (1 << 25) - 1, 1 << 25, T - 1]
    for i, t in enumerate(places):
        x[t, 10 + i] = 3.0
        x[t, 40] = 2.0
    ids = torch.full((T, 2), 99, dtype=torch.int32, device=DEV)
    w = torch.full((T, 2), float("nan"), device=DEV)
    mx.topk_gating(x, ids, w)
    for i, t in enumerate(places):
        assert ids[t].tolist() == [10 + i, 40]
    rest = torch.ones(T, dtype=torch.bool, device=DEV)
    rest[places] = False
    assert (ids[rest] == torch.tensor([0, 1], dtype=torch.int32, device=DEV)).all()
    assert (w[rest] == 0.5).all()
    grad = torch.zeros(T, 2, device=DEV)
    grad[places, 0] = 1.0
    out = torch.full_like(x, float("nan"))
    mx.topk_gating_backward(x, ids, grad, out)
    p = float(torch.sigmoid(torch.tensor(1.0, dtype=torch.float64)))
    for i, t in enumerate(places):
        assert abs(float(out[t, 10 + i]) - p * (1 - p)) < 2 ** -11
        assert abs(float(out[t, 40]) + p * (1 - p)) < 2 ** -11
    assert (out[rest] == 0).all()
