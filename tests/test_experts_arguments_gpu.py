"""Arguments of the expert products that are allowed and out of the ordinary:
offsets that do not ascend, arrays that begin off 16 bytes, views of larger
arrays."""

import pytest
import torch

import combine_topk_ids_expert_amd as mx
from tests import experts_util as eu

pytestmark = pytest.mark.gpu

DEV = eu.DEV
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SENTINEL = -77.0


@pytest.mark.parametrize("offsets", [[0, 50, 10, 60], [10, 0, 20, 30], [0, 2**30, 5, 2**30],
                                     [0, 20, 40, -3]])
def test_products_leave_out_segments_that_do_not_ascend(offsets):
    print("case: descending", offsets, flush=True)
    n = k = 64
    x = eu.normal((60, k), BF16, 1).to(DEV)
    w = eu.normal((3, n, k), BF16, 2).to(DEV)
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    q = torch.zeros(3, n, k // 2, dtype=torch.uint8, device=DEV)
    sc = torch.ones(3, n, k // 32, dtype=BF16, device=DEV)
    for call in (lambda o: mx.grouped_gemm(x, w, off, o),
                 lambda o: mx.grouped_gemm(x, w, off, o, transpose_weight=True),
                 lambda o: mx.grouped_gemm(x, torch.cat((w, w), 1), off, o, silu_mul=True),
                 lambda o: mx.grouped_gemm_w4(x, q, sc, off, o)):
        out = torch.full((60, n), SENTINEL, dtype=BF16, device=DEV)
        call(out)
        assert (out == SENTINEL).all()


def test_bounds_past_the_array_do_not_count_as_descending():
    """Both clip to the array's end: an empty segment behind a whole one."""
    n = k = 64
    x = eu.normal((40, k), BF16, 3)
    w = eu.normal((2, n, k), BF16, 4)
    off = torch.tensor([0, 2**30, 100], dtype=torch.int32, device=DEV)
    out = torch.full((40, n), SENTINEL, device=DEV)
    mx.grouped_gemm(x.to(DEV), w.to(DEV), off, out)
    a, m = x.double(), w[0].double()
    eu.check(out, a @ m.T, k * eu.U32 * (a.abs() @ m.abs().T), F32)


def _off(t, by):
    """t on the GPU, in an array that begins `by` elements earlier."""
    flat = torch.zeros(t.numel() + by, dtype=t.dtype, device=DEV)
    v = flat[by:].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.parametrize("dx,dw,do", [(1, 0, 0), (0, 3, 0), (0, 0, 1), (5, 1, 3), (8, 8, 8)])
def test_arrays_off_16_bytes(dx, dw, do):
    print("case: off", dx, dw, do, flush=True)
    n, k = 72, 136
    seg = eu.segments([5, 0, 70, 33], align=4, extra=2)
    m = eu.live(seg)
    x = eu.rows_with_nan(seg, k, F16, 5)
    xd = _off(x, dx)
    for name, shape, kw in (("plain", (4, n, k), {}), ("gated", (4, 2 * n, k), {"silu_mul": True}),
                            ("transposed", (4, k, n), {"transpose_weight": True})):
        w = eu.normal(shape, F16, 6, k ** -0.5)
        for dtype in (F16, F32):
            out = _off(torch.full((seg["rows"], n), SENTINEL, dtype=dtype), do)
            gu = _off(torch.full((seg["rows"], 2 * n), SENTINEL, dtype=dtype), do) \
                if name == "gated" else None
            mx.grouped_gemm(xd, _off(w, dw), seg["offsets"], out, seg["sizes"],
                            **({"gate_up": gu} if name == "gated" else {}), **kw)
            y, s = eu.products(seg, x, w.transpose(1, 2) if name == "transposed" else w)
            err = k * eu.U32 * s
            if name == "gated":
                eu.check(gu.cpu()[m], y[m], err[m], dtype, name)
                assert (gu.cpu()[~m] == SENTINEL).all()
                y, err = eu.gated(y, err)
            eu.check(out.cpu()[m], y[m], err[m], dtype, name)
            assert (out.cpu()[~m] == SENTINEL).all()
    d = eu.rows_with_nan(seg, n, F16, 7)
    for dtype in (F16, F32):
        g = _off(torch.zeros(4, n, k, dtype=dtype), do)
        mx.grouped_gemm_wgrad(_off(d, dw), xd, seg["offsets"], g, seg["sizes"])
        for e, (b, c) in enumerate(seg["spans"]):
            a, v = d[b:b + c].double(), x[b:b + c].double()
            eu.check(g[e], a.T @ v, (c + 1) * eu.U32 * (a.abs().T @ v.abs()), dtype, "wgrad")
    gu = eu.normal((seg["rows"], 2 * n), F16, 8)
    gg = _off(torch.full((seg["rows"], 2 * n), SENTINEL, dtype=F16), do)
    mx.silu_mul_backward(_off(d, dw), _off(gu, dx), seg["offsets"], gg, seg["sizes"])
    ref = torch.full((seg["rows"], 2 * n), SENTINEL, dtype=F16, device=DEV)
    mx.silu_mul_backward(d.to(DEV), gu.to(DEV), seg["offsets"], ref, seg["sizes"])
    assert torch.equal(gg, ref)


def test_fp8_and_4_bit_arrays_off_16_bytes_are_refused():
    off = torch.tensor([0, 8], dtype=torch.int32, device=DEV)
    f8 = torch.float8_e4m3fn
    x = torch.zeros(8 * 128 + 8, dtype=torch.uint8, device=DEV)[8:].view(f8).view(8, 128)
    w = torch.zeros(1, 128, 128, dtype=torch.uint8, device=DEV).view(f8)
    out = torch.zeros(8, 128, dtype=BF16, device=DEV)
    with pytest.raises(mx.MxError):
        mx.grouped_gemm_fp8(x, torch.ones(8, 1, device=DEV), w, torch.ones(1, 1, 1, device=DEV),
                            off, out)
    x = torch.zeros(8 * 128 + 4, dtype=BF16, device=DEV)[4:].view(8, 128)
    with pytest.raises(mx.MxError):
        mx.grouped_gemm_w4(x, torch.zeros(1, 128, 64, dtype=torch.uint8, device=DEV),
                           torch.ones(1, 128, 1, dtype=BF16, device=DEV), off, out)


def test_calls_at_once_on_two_streams():
    """Two calls share nothing: 20 of each on two streams give the bits of each
    alone."""
    seg = eu.segments([30, 0, 300, 77])
    x = eu.normal((seg["rows"], 256), BF16, 9).to(DEV)
    w = eu.normal((4, 512, 256), BF16, 10).to(DEV)
    q = torch.randint(0, 256, (4, 512, 128), generator=torch.Generator().manual_seed(11),
                      dtype=torch.uint8).to(DEV)
    sc = torch.full((4, 512, 2), 0.125, dtype=BF16, device=DEV)
    new = lambda: torch.empty(seg["rows"], 512, dtype=BF16, device=DEV)  # noqa: E731
    want = mx.grouped_gemm(x, w, seg["offsets"], new()), \
        mx.grouped_gemm_w4(x, q, sc, seg["offsets"], new())
    got = [[new() for _ in range(20)] for _ in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i in range(20):
        with torch.cuda.stream(streams[0]):
            mx.grouped_gemm(x, w, seg["offsets"], got[0][i])
        with torch.cuda.stream(streams[1]):
            mx.grouped_gemm_w4(x, q, sc, seg["offsets"], got[1][i])
    torch.cuda.synchronize()
    for j in range(2):
        assert all(torch.equal(g, want[j]) for g in got[j])


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_gated_rows_have_the_same_bits_stored_by_vectors_and_by_elements(dtype):
    n, k = 128, 64
    seg = eu.segments([50, 131])
    x = eu.normal((seg["rows"], k), dtype, 12).to(DEV)
    w = eu.normal((2, 2 * n, k), dtype, 13).to(DEV)
    out = [_off(torch.zeros(seg["rows"], n, dtype=dtype), by) for by in (0, 1)]
    for o in out:
        mx.grouped_gemm(x, w, seg["offsets"], o, silu_mul=True)
    assert torch.equal(*out)
