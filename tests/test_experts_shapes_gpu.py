"""The expert products in calls with many output tiles, where tiles of 256
columns run: for few rows to an expert with 128 rows each, for many with 256
(the small calls of test_experts_gpu run with 128 x 128).  Same references and
tolerances."""

import pytest
import torch

import combine_topk_ids_expert_amd as mx
from tests import experts_util as eu

pytestmark = pytest.mark.gpu

DEV = eu.DEV
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SENTINEL = -77.0

# 40 experts of 12 rows on average, and 8 of 250
FEW = [0, 1, 5, 70, 0, 129, 16, 17] + [2, 0, 3, 31, 33, 9, 0, 64] + [1] * 16 + [0] * 7 + [80]
MANY = [256, 257, 0, 700, 193, 64, 129, 401]
COUNTS = {"few": FEW, "many": MANY}
# 512 tiles of 128 rows x 256 columns and more: (500 / 128 + 40) x 16, (2000 / 128 + 8) x 24
WIDTH = {"few": 4096, "many": 6016}


def _run(call, seg, n, out_dtype):
    out = torch.full((seg["rows"], n), SENTINEL, dtype=out_dtype, device=DEV)
    call(out)
    got = out.cpu()
    m = eu.live(seg)
    assert (got[~m] == SENTINEL).all(), "a row outside the segments was written"
    return got[m]


@pytest.mark.parametrize("counts", ["few", "many"])
@pytest.mark.parametrize("more,k", [(0, 64), (0, 72), (8, 328), (40, 512), (3, 61)])
@pytest.mark.parametrize("dtype,out_dtype", [(BF16, F32), (F16, F16)])
def test_grouped_gemm(counts, more, k, dtype, out_dtype):
    n = WIDTH[counts] + more
    print("case: grouped_gemm", counts, n, k, dtype, out_dtype, flush=True)
    seg = eu.segments(COUNTS[counts], align=4, extra=5)
    x = eu.rows_with_nan(seg, k, dtype, 1)
    w = eu.normal((len(seg["spans"]), n, k), dtype, 2)
    got = _run(lambda out: mx.grouped_gemm(x.to(DEV), w.to(DEV), seg["offsets"], out, seg["sizes"]),
               seg, n, out_dtype)
    y, s = eu.products(seg, x, w)
    m = eu.live(seg)
    eu.check(got, y[m], (k * eu.U32 * s)[m], out_dtype)


@pytest.mark.parametrize("counts", ["few", "many"])
@pytest.mark.parametrize("more,k", [(0, 64), (8, 328), (24, 136), (1, 61)])
@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (F16, F32)])
def test_grouped_gemm_gated(counts, more, k, dtype, out_dtype):
    n = WIDTH[counts] // 2 + more
    print("case: gated", counts, n, k, dtype, out_dtype, flush=True)
    seg = eu.segments(COUNTS[counts], align=4, extra=5)
    x = eu.rows_with_nan(seg, k, dtype, 3)
    w = eu.normal((len(seg["spans"]), 2 * n, k), dtype, 4, k ** -0.5)
    gu = torch.full((seg["rows"], 2 * n), SENTINEL, dtype=out_dtype, device=DEV)
    got = _run(lambda out: mx.grouped_gemm(x.to(DEV), w.to(DEV), seg["offsets"], out, seg["sizes"],
                                           silu_mul=True, gate_up=gu), seg, n, out_dtype)
    y, s = eu.products(seg, x, w)
    m = eu.live(seg)
    h, err = eu.gated(y, k * eu.U32 * s)
    eu.check(got, h[m], err[m], out_dtype, "output")
    gu = gu.cpu()
    assert (gu[~m] == SENTINEL).all()
    eu.check(gu[m], y[m], (k * eu.U32 * s)[m], out_dtype, "gate_up")


@pytest.mark.parametrize("counts", ["few", "many"])
@pytest.mark.parametrize("more,k", [(0, 64), (8, 328), (72, 200), (7, 61)])
@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (F16, F32)])
def test_grouped_gemm_transposed(counts, more, k, dtype, out_dtype):
    n = WIDTH[counts] + more
    print("case: transposed", counts, n, k, dtype, out_dtype, flush=True)
    seg = eu.segments(COUNTS[counts], align=4, extra=5)
    x = eu.rows_with_nan(seg, k, dtype, 5)
    w = eu.normal((len(seg["spans"]), k, n), dtype, 6)
    got = _run(lambda out: mx.grouped_gemm(x.to(DEV), w.to(DEV), seg["offsets"], out, seg["sizes"],
                                           transpose_weight=True), seg, n, out_dtype)
    y, s = eu.products(seg, x, w.transpose(1, 2))
    m = eu.live(seg)
    eu.check(got, y[m], (k * eu.U32 * s)[m], out_dtype)


@pytest.mark.parametrize("counts", ["few", "many"])
@pytest.mark.parametrize("more,k,gated", [(0, 128, False), (33, 384, False), (16, 512, True),
                                          (48, 256, True)])
def test_grouped_gemm_fp8(counts, more, k, gated):
    n = WIDTH[counts] // (2 if gated else 1) + more
    wide = 2 * n if gated else n
    print("case: fp8", counts, n, k, gated, flush=True)
    seg = eu.segments(COUNTS[counts], align=4, extra=5)
    E, m = len(seg["spans"]), eu.live(seg)
    fp8 = torch.float8_e4m3fn
    x = eu.normal((seg["rows"], k), F32, 10, 60.0).clamp(-448, 448).to(fp8)
    xs = eu.normal((seg["rows"], k // 128), F32, 11).abs() * 0.02 + 0.005
    x.view(torch.uint8)[~m] = 0x7f
    xs[~m] = float("nan")
    w = eu.normal((E, wide, k), F32, 12, 60.0).clamp(-448, 448).to(fp8)
    ws = (eu.normal((E, -(-wide // 128), k // 128), F32, 13).abs() + 0.1) * 0.02 * k ** -0.5
    got = _run(lambda out: mx.grouped_gemm_fp8(x.to(DEV), xs.to(DEV), w.to(DEV), ws.to(DEV),
                                               seg["offsets"], out, seg["sizes"], silu_mul=gated),
               seg, n, BF16)
    xd = x[m].float().double() * xs[m].double().repeat_interleave(128, 1)
    rows = torch.zeros(seg["rows"], k, dtype=torch.float64)
    rows[m] = xd
    y = torch.zeros(seg["rows"], wide, dtype=torch.float64)
    s = torch.zeros_like(y)
    for e, (b, c) in enumerate(seg["spans"]):
        if c == 0:
            continue
        we = w[e].float().double() * ws[e].double().repeat_interleave(128, 0)[:wide] \
            .repeat_interleave(128, 1)
        y[b:b + c], s[b:b + c] = rows[b:b + c] @ we.T, rows[b:b + c].abs() @ we.abs().T
    err = (2.0 ** -13 + (k // 128 + 3) * eu.U32) * s    # the bound of test_experts_gpu
    if gated:
        y, err = eu.gated(y, err)
    eu.check(got, y[m], err[m], BF16)


def test_a_row_has_the_same_bits_in_every_tile_shape():
    """Calls of one expert's rows run with small tiles, the whole batch with
    tiles of 128 x 256 or 256 x 256."""
    for counts in ("few", "many"):
        n, k = WIDTH[counts], 264
        seg = eu.segments(COUNTS[counts])
        E = len(seg["spans"])
        x = eu.normal((seg["rows"], k), F16, 25).to(DEV)
        w = eu.normal((E, n, k), F16, 26).to(DEV)
        whole = mx.grouped_gemm(x, w, seg["offsets"], torch.empty(seg["rows"], n, device=DEV))
        for e, (b, c) in enumerate(seg["spans"]):
            if c == 0 or c == 1 and e > 16:
                continue
            off = torch.tensor([0, c], dtype=torch.int32, device=DEV)
            part = mx.grouped_gemm(x[b:b + c], w[e:e + 1], off, torch.empty(c, n, device=DEV))
            assert torch.equal(part, whole[b:b + c]), (counts, e)
