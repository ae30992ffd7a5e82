"""The experts' products, their gradients and the gated activation's gradient
against 64-bit references, with tolerances that count roundings
(experts_util).  Rows outside the segments hold NaN on entry, and the outputs
there keep a sentinel."""

import pytest
import torch

import combine_topk_ids_expert_amd as mx
from tests import experts_util as eu

pytestmark = pytest.mark.gpu

DEV = eu.DEV
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SENTINEL = -77.0

# row counts of the experts: empty ones, one row, both sides of the tile sizes
COUNTS = {
    "one": [1],
    "tiny": [0, 1, 2, 0, 3],
    "sixteens": [15, 16, 17, 0, 33],
    "tiles": [63, 64, 65, 128, 129, 0, 193],
    "big": [256, 257, 0, 700],
}


def _poison(shape, dtype):
    return torch.full(shape, SENTINEL, dtype=dtype, device=DEV)


def _untouched(out, seg):
    rest = out.detach().cpu()[~eu.live(seg)]
    assert (rest == SENTINEL).all(), "a row outside the segments was written"


def _print(*a):
    print("case:", *a, flush=True)


@pytest.mark.parametrize("counts", sorted(COUNTS))
@pytest.mark.parametrize("n,k", [(64, 64), (256, 512), (40, 72), (33, 200), (130, 328), (7, 45)])
@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (F16, F32)])
def test_grouped_gemm(counts, n, k, dtype, out_dtype):
    _print("grouped_gemm", counts, n, k, dtype, out_dtype)
    seg = eu.segments(COUNTS[counts], align=16, extra=5)
    x = eu.rows_with_nan(seg, k, dtype, 1)
    w = eu.normal((len(seg["spans"]), n, k), dtype, 2)
    out = _poison((seg["rows"], n), out_dtype)
    got = mx.grouped_gemm(x.to(DEV), w.to(DEV), seg["offsets"], out, seg["sizes"])
    assert got is out
    y, s = eu.products(seg, x, w)
    m = eu.live(seg)
    eu.check(out[m.to(DEV)], y[m], (k * eu.U32 * s)[m], out_dtype)
    _untouched(out, seg)


@pytest.mark.parametrize("counts", ["tiny", "tiles", "big"])
@pytest.mark.parametrize("n,k", [(64, 64), (128, 264), (24, 40), (17, 72), (150, 61)])
@pytest.mark.parametrize("dtype,out_dtype,keep", [(BF16, BF16, True), (F16, F16, False),
                                                  (BF16, F32, True)])
def test_grouped_gemm_gated(counts, n, k, dtype, out_dtype, keep):
    _print("gated", counts, n, k, dtype, out_dtype, keep)
    seg = eu.segments(COUNTS[counts], align=1, extra=3)
    x = eu.rows_with_nan(seg, k, dtype, 3)
    w = eu.normal((len(seg["spans"]), 2 * n, k), dtype, 4, k ** -0.5)
    out = _poison((seg["rows"], n), out_dtype)
    gu = _poison((seg["rows"], 2 * n), out_dtype) if keep else None
    mx.grouped_gemm(x.to(DEV), w.to(DEV), seg["offsets"], out, silu_mul=True, gate_up=gu)
    if seg["rows"] > int(seg["offsets"][-1]):
        _untouched(out, seg)
    y, s = eu.products(seg, x, w)
    m = eu.live(seg)
    h, err = eu.gated(y, k * eu.U32 * s)
    eu.check(out[m.to(DEV)], h[m], err[m], out_dtype, "output")
    if keep:
        eu.check(gu[m.to(DEV)], y[m], (k * eu.U32 * s)[m], out_dtype, "gate_up")
        _untouched(gu, seg)


@pytest.mark.parametrize("counts", ["one", "tiny", "tiles", "big"])
@pytest.mark.parametrize("n,k", [(64, 64), (328, 520), (40, 72), (33, 61), (9, 200)])
@pytest.mark.parametrize("dtype,out_dtype", [(BF16, F32), (F16, F16)])
def test_grouped_gemm_transposed(counts, n, k, dtype, out_dtype):
    """The rows' gradient: output [rows, n] from input [rows, k], weight [E, k, n]."""
    _print("transposed", counts, n, k, dtype, out_dtype)
    seg = eu.segments(COUNTS[counts], align=8, extra=1)
    x = eu.rows_with_nan(seg, k, dtype, 5)
    w = eu.normal((len(seg["spans"]), k, n), dtype, 6)
    out = _poison((seg["rows"], n), out_dtype)
    mx.grouped_gemm(x.to(DEV), w.to(DEV), seg["offsets"], out, seg["sizes"], transpose_weight=True)
    y, s = eu.products(seg, x, w.transpose(1, 2))
    m = eu.live(seg)
    eu.check(out[m.to(DEV)], y[m], (k * eu.U32 * s)[m], out_dtype)
    _untouched(out, seg)


@pytest.mark.parametrize("counts", sorted(COUNTS))
@pytest.mark.parametrize("n,k", [(64, 64), (264, 328), (40, 24), (33, 72), (9, 61)])
@pytest.mark.parametrize("dtype,out_dtype,accumulate", [(BF16, F32, False), (F16, F16, False),
                                                        (BF16, F32, True), (BF16, BF16, True)])
def test_grouped_gemm_wgrad(counts, n, k, dtype, out_dtype, accumulate):
    _print("wgrad", counts, n, k, dtype, out_dtype, accumulate)
    seg = eu.segments(COUNTS[counts], align=16, extra=2)
    d = eu.rows_with_nan(seg, n, dtype, 7)
    x = eu.rows_with_nan(seg, k, dtype, 8)
    E = len(seg["spans"])
    old = eu.normal((E, n, k), out_dtype, 9)
    out = old.to(DEV) if accumulate else torch.full((E, n, k), float("nan"), dtype=out_dtype,
                                                    device=DEV)
    mx.grouped_gemm_wgrad(d.to(DEV), x.to(DEV), seg["offsets"], out, seg["sizes"],
                          accumulate=accumulate)
    for e, (b, c) in enumerate(seg["spans"]):
        a, m = d[b:b + c].double(), x[b:b + c].double()
        want, s = a.T @ m, a.abs().T @ m.abs()
        if accumulate:
            want, s = want + old[e].double(), s + old[e].double().abs()
        eu.check(out[e], want, (c + 1) * eu.U32 * s, out_dtype, f"expert {e}")


def _fp8(t):
    return t.to(torch.float8_e4m3fn)


@pytest.mark.parametrize("counts", ["one", "tiny", "sixteens", "tiles", "big"])
@pytest.mark.parametrize("n,k,gated", [(128, 128, False), (80, 256, True), (33, 384, False),
                                       (272, 128, True), (208, 512, False)])
@pytest.mark.parametrize("out_dtype", [BF16, F16])
def test_grouped_gemm_fp8(counts, n, k, gated, out_dtype):
    _print("fp8", counts, n, k, gated, out_dtype)
    seg = eu.segments(COUNTS[counts], align=16, extra=4)
    E, wide = len(seg["spans"]), 2 * n if gated else n
    m = eu.live(seg)
    x = _fp8(eu.normal((seg["rows"], k), F32, 10, 60.0).clamp(-448, 448))
    xs = eu.normal((seg["rows"], k // 128), F32, 11).abs() * 0.02 + 0.005
    x.view(torch.uint8)[~m] = 0x7f
    xs[~m] = float("nan")
    w = _fp8(eu.normal((E, wide, k), F32, 12, 60.0).clamp(-448, 448))
    ws = (eu.normal((E, -(-wide // 128), k // 128), F32, 13).abs() + 0.1) * 0.02 * k ** -0.5
    out = _poison((seg["rows"], n), out_dtype)
    mx.grouped_gemm_fp8(x.to(DEV), xs.to(DEV), w.to(DEV), ws.to(DEV), seg["offsets"], out,
                        seg["sizes"], silu_mul=gated)
    xd = torch.where(m[:, None], x.float(), torch.zeros(())).double()
    xd = xd * torch.where(m[:, None], xs, torch.zeros(())).double().repeat_interleave(128, 1)
    wd = w.float().double() * ws.double().repeat_interleave(128, 1)[:, :wide].repeat_interleave(128, 2)
    y, s = eu.products(seg, xd, wd)
    # the matrix instruction keeps a block's products to 2^-13 of their absolute
    # sum (the bound stated in mxmoe.h); the scales and sums over blocks are float32
    err = (2.0 ** -13 + (k // 128 + 3) * eu.U32) * s
    if gated:
        y, err = eu.gated(y, err)
    eu.check(out[m.to(DEV)], y[m], err[m], out_dtype)
    _untouched(out, seg)


@pytest.mark.parametrize("counts", sorted(COUNTS))
@pytest.mark.parametrize("n,k,group,gated", [(64, 128, 128, False), (40, 256, 32, True),
                                             (33, 192, 64, False), (100, 640, 64, True),
                                             (17, 32, 32, False), (130, 1152, 128, True)])
@pytest.mark.parametrize("dtype,zeros", [(BF16, False), (F16, True)])
def test_grouped_gemm_w4(counts, n, k, group, gated, dtype, zeros):
    _print("w4", counts, n, k, group, gated, dtype, zeros)
    seg = eu.segments(COUNTS[counts], align=4, extra=4)
    E, wide = len(seg["spans"]), 2 * n if gated else n
    g = torch.Generator().manual_seed(14)
    q = torch.randint(0, 256, (E, wide, k // 2), generator=g, dtype=torch.uint8)
    sc = ((0.5 + torch.rand((E, wide, k // group), generator=g)) * k ** -0.5 / 5).to(dtype)
    z = torch.randint(0, 16, (E, wide, k // group), generator=g, dtype=torch.uint8) if zeros else None
    x = eu.rows_with_nan(seg, k, dtype, 15)
    out = _poison((seg["rows"], n), dtype)
    mx.grouped_gemm_w4(x.to(DEV), q.to(DEV), sc.to(DEV), seg["offsets"], out, seg["sizes"],
                       zeros=None if z is None else z.to(DEV), silu_mul=gated)
    w = torch.stack((q & 15, q >> 4), -1).view(E, wide, k).double()
    zero = 8.0 if z is None else z.double().repeat_interleave(group, 2)
    s64 = sc.double().repeat_interleave(group, 2)
    y, s = eu.products(seg, x, (w - zero) * s64)
    # |x| (B + 16) s is what the sums hold: group / 32 matrix instructions and
    # two subtractions' roundings on it, then k / group multiply-adds on y
    bias = 128 if dtype == BF16 else 1024
    held = eu.products(seg, x.abs(), s64 * (bias + 16))[0]
    err = (group // 32 + 2) * 2 * eu.U32 * held + (k // group + 1) * eu.U32 * s
    if gated:
        y, err = eu.gated(y, err)
    m = eu.live(seg)
    eu.check(out[m.to(DEV)], y[m], err[m], dtype)
    _untouched(out, seg)


@pytest.mark.parametrize("counts", ["one", "tiny", "tiles"])
@pytest.mark.parametrize("n", [8, 64, 520, 2056, 33, 7])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("in_place", [False, True])
def test_silu_mul_backward(counts, n, dtype, in_place):
    _print("silu_mul_backward", counts, n, dtype, in_place)
    seg = eu.segments(COUNTS[counts], align=8, extra=3)
    m = eu.live(seg)
    gu = eu.normal((seg["rows"], 2 * n), dtype, 16, 3.0)
    gu[m, :1] = -60.0                                # the sigmoid's far ends
    gu[m, n - 1:n] = 60.0
    d = eu.rows_with_nan(seg, n, dtype, 17)
    src = gu.to(DEV)
    out = src if in_place else _poison((seg["rows"], 2 * n), dtype)
    if in_place:
        src[~m.to(DEV)] = SENTINEL
    mx.silu_mul_backward(d.to(DEV), src, seg["offsets"], out, seg["sizes"])
    g, u, dd = gu[m][:, :n].double(), gu[m][:, n:].double(), d[m].double()
    s = torch.sigmoid(g)
    want = torch.cat((dd * u * s * (1 + g * (1 - s)), dd * g * s), 1)
    # the sigmoid is off by (4 + |g|) roundings (g log2 e, 2^x, the sum, the
    # quotient), 1 - s by as many of s; five more roundings in the products
    es = (4 + g.abs()) * eu.U32
    t = 1 + g * (1 - s)
    et = g.abs() * (s * es + 2 * eu.U32) + t.abs() * eu.U32
    err = torch.cat(((dd * u * s).abs() * ((es + 4 * eu.U32) * t.abs() + et),
                     (dd * g * s).abs() * (es + 3 * eu.U32)), 1)
    eu.check(out[m.to(DEV)], want, err, dtype)
    _untouched(out, seg)


def test_whole_segments_without_sizes_and_untrusted_offsets():
    """Without sizes the whole segment counts; offsets and counts outside the
    arrays are clipped."""
    n = k = 64
    x = eu.normal((40, k), BF16, 20)
    w = eu.normal((4, n, k), BF16, 21)
    off = torch.tensor([0, 10, 10, 25, 2**30], dtype=torch.int32, device=DEV)
    sizes = torch.tensor([[2**31 - 1] * 3, [5] * 3, [-4] * 3, [2**30] * 3], dtype=torch.int32,
                         device=DEV)
    y = torch.stack([x.double() @ w[e].double().T for e in range(4)])
    s = torch.stack([x.double().abs() @ w[e].double().abs().T for e in range(4)])
    for z, spans in ((None, [(0, 0, 10), (2, 10, 25), (3, 25, 40)]),
                     (sizes, [(0, 0, 10), (3, 25, 40)])):
        out = _poison((40, n), F32)
        mx.grouped_gemm(x.to(DEV), w.to(DEV), off, out, z)
        wg = torch.full((4, n, k), float("nan"), device=DEV)
        mx.grouped_gemm_wgrad(x.to(DEV), x.to(DEV), off, wg, z)
        done = torch.zeros(40, dtype=torch.bool)
        for e, b, t in spans:
            eu.check(out[b:t], y[e][b:t], k * eu.U32 * s[e][b:t], F32)
            done[b:t] = True
            xe = x[b:t].double()
            eu.check(wg[e], xe.T @ xe, 16 * eu.U32 * (xe.abs().T @ xe.abs()), F32)
        assert (out.cpu()[~done] == SENTINEL).all()
        rest = [e for e in range(4) if e not in [v[0] for v in spans]]
        assert (wg[rest] == 0).all()
    out = _poison((40, n), F32)
    mx.grouped_gemm(x.to(DEV), w.to(DEV), torch.full((5,), -7, dtype=torch.int32, device=DEV), out)
    assert (out == SENTINEL).all()


def test_one_row_does_not_reach_another():
    """An infinity or a NaN in one row, or in another expert's weights, stays
    there (the tiles share registers and LDS)."""
    n, k = 96, 160
    seg = eu.segments([3, 20, 70])
    x = eu.normal((seg["rows"], k), BF16, 22)
    w = eu.normal((3, n, k), BF16, 23)
    q = torch.randint(0, 256, (3, n, k // 2), generator=torch.Generator().manual_seed(24),
                      dtype=torch.uint8)
    sc = torch.ones(3, n, k // 32, dtype=BF16)
    bad = [1, 9, 40]
    calls = {
        "gemm": lambda a: mx.grouped_gemm(a, w.to(DEV), seg["offsets"],
                                          torch.empty(seg["rows"], n, device=DEV)),
        "transposed": lambda a: mx.grouped_gemm(
            a, w.transpose(1, 2).contiguous().to(DEV), seg["offsets"],
            torch.empty(seg["rows"], n, device=DEV), transpose_weight=True),
        "w4": lambda a: mx.grouped_gemm_w4(a, q.to(DEV), sc.to(DEV), seg["offsets"],
                                           torch.empty(seg["rows"], n, dtype=BF16, device=DEV)),
    }
    for name, call in calls.items():
        _print("rows apart", name)
        clean = call(x.to(DEV)).cpu()
        y = x.clone()
        y[bad[0], 5] = float("inf")
        y[bad[1], 150] = float("nan")
        y[bad[2], 0] = float("-inf")
        got = call(y.to(DEV)).cpu()
        rest = [r for r in range(seg["rows"]) if r not in bad]
        assert torch.equal(got[rest], clean[rest])
        assert not torch.isfinite(got[bad].float()).any()


def test_results_do_not_depend_on_the_batch():
    """A row's result is the same bits alone and among others (bf16 and 4 bits)."""
    n, k = 200, 384
    counts = [5, 0, 130, 64]
    seg = eu.segments(counts)
    x = eu.normal((seg["rows"], k), F16, 25).to(DEV)
    w = eu.normal((4, n, k), F16, 26).to(DEV)
    whole = mx.grouped_gemm(x, w, seg["offsets"], torch.empty(seg["rows"], n, device=DEV))
    again = mx.grouped_gemm(x, w, seg["offsets"], torch.empty(seg["rows"], n, device=DEV))
    assert torch.equal(whole, again)
    for e, (b, c) in enumerate(seg["spans"]):
        off = torch.zeros(5, dtype=torch.int32)
        off[e + 1:] = c
        part = mx.grouped_gemm(x[b:b + c].contiguous(), w, off.to(DEV),
                               torch.empty(c, n, device=DEV))
        assert torch.equal(part, whole[b:b + c])


def test_many_experts():
    """1024 experts, most of them empty."""
    E, n, k = 1024, 48, 64
    counts = [0] * E
    for e, c in ((0, 2), (1, 70), (63, 1), (64, 3), (500, 20), (1022, 9), (1023, 33)):
        counts[e] = c
    seg = eu.segments(counts, align=4)
    x = eu.rows_with_nan(seg, k, BF16, 27)
    w = eu.normal((E, n, k), BF16, 28)
    m = eu.live(seg)
    y, s = eu.products(seg, x, w)
    out = _poison((seg["rows"], n), F32)
    mx.grouped_gemm(x.to(DEV), w.to(DEV), seg["offsets"], out, seg["sizes"])
    eu.check(out[m.to(DEV)], y[m], (k * eu.U32 * s)[m], F32)
    _untouched(out, seg)
    q = torch.randint(0, 256, (E, n, k // 2), generator=torch.Generator().manual_seed(29),
                      dtype=torch.uint8)
    sc = torch.full((E, n, k // 64), 0.125, dtype=BF16)
    out = _poison((seg["rows"], n), BF16)
    mx.grouped_gemm_w4(x.to(DEV), q.to(DEV), sc.to(DEV), seg["offsets"], out, seg["sizes"])
    wq = (torch.stack((q & 15, q >> 4), -1).view(E, n, k).double() - 8) * 0.125
    y, s = eu.products(seg, x, wq)
    held = eu.products(seg, x.abs(), torch.full((E, n, k), 18.0))[0]
    eu.check(out[m.to(DEV)], y[m], (8 * eu.U32 * held + 2 * eu.U32 * s)[m], BF16)
    _untouched(out, seg)


def test_no_rows():
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    w = torch.zeros(3, 64, 64, dtype=BF16, device=DEV)
    x = torch.empty(0, 64, dtype=BF16, device=DEV)
    assert mx.grouped_gemm(x, w, off, torch.empty(0, 64, device=DEV)).shape == (0, 64)
    g = torch.full((3, 64, 64), 5.0, device=DEV)
    mx.grouped_gemm_wgrad(x, x, off, g, accumulate=True)
    assert (g == 5).all()
    mx.grouped_gemm_wgrad(x, x, off, g)
    assert (g == 0).all()


def test_bindings_refuse():
    seg = eu.segments([4, 4])
    x = torch.zeros(8, 64, dtype=BF16, device=DEV)
    w = torch.zeros(2, 32, 64, dtype=BF16, device=DEV)
    out = torch.zeros(8, 32, dtype=BF16, device=DEV)
    off = seg["offsets"]
    for bad, kind in (
        (lambda: mx.grouped_gemm(x.float(), w, off, out), TypeError),
        (lambda: mx.grouped_gemm(x, w.half(), off, out), TypeError),
        (lambda: mx.grouped_gemm(x, w[:1], off, out), ValueError),
        (lambda: mx.grouped_gemm(x, w, off, out[:, :16].contiguous()), ValueError),
        (lambda: mx.grouped_gemm(x.t().contiguous().t(), w, off, out), ValueError),
        (lambda: mx.grouped_gemm(x, w, off.long(), out), TypeError),
        (lambda: mx.grouped_gemm(x, w, off, out, seg["sizes"][:1].contiguous()), ValueError),
        (lambda: mx.grouped_gemm(x, w, off, out, gate_up=out), ValueError),
        (lambda: mx.grouped_gemm(x, w, off, out, silu_mul=True, transpose_weight=True), ValueError),
        (lambda: mx.grouped_gemm(x.cpu(), w, off, out), ValueError),
        (lambda: mx.grouped_gemm_wgrad(out, x[:4].contiguous(), off, w), ValueError),
        (lambda: mx.silu_mul_backward(out, out, off, out), ValueError),
        (lambda: mx.grouped_gemm_w4(x, torch.zeros(2, 32, 32, dtype=torch.uint8, device=DEV),
                                    torch.zeros(2, 32, 4, dtype=BF16, device=DEV), off, out),
         ValueError),
        (lambda: mx.grouped_gemm_fp8(x.to(torch.float8_e4m3fn),
                                     torch.zeros(8, 1, device=DEV),
                                     w.to(torch.float8_e4m3fn), torch.zeros(2, 1, 1, device=DEV),
                                     off, out), ValueError),
    ):
        with pytest.raises(kind):
            bad()


def test_bound_calls_repeat():
    seg = eu.segments([20, 0, 90])
    x = eu.normal((110, 128), BF16, 30).to(DEV)
    w = eu.normal((3, 64, 128), BF16, 31).to(DEV)
    out = torch.empty(110, 64, dtype=BF16, device=DEV)
    want = mx.grouped_gemm(x, w, seg["offsets"], torch.empty_like(out))
    call = mx.bind(mx.grouped_gemm, x, w, seg["offsets"], out)
    assert call() is out and torch.equal(out, want)
    x.mul_(2)
    call()
    assert torch.equal(out, mx.grouped_gemm(x, w, seg["offsets"], torch.empty_like(out)))
