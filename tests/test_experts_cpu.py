"""The C ABI of the expert products and the router on the host: bad arguments
are refused with the documented status before any HIP call (fake device
addresses are never dereferenced on these paths)."""

import pytest

import combine_topk_ids_expert_amd as mx

OK, INVALID, DTYPE, MISALIGNED = range(4)
F32, F16, BF16, FP8, I32, I64 = range(6)
P = 0x10000
S = None
TRANSPOSED, SILU = 1, 2


@pytest.fixture(scope="module", params=["loaded", "checked"])
def lib(request):
    return mx.load_library() if request.param == "loaded" else mx.open_library(mx.CHECKED_LIBRARY)


def _call(fn, defaults, **kw):
    assert set(kw) <= set(defaults)
    return fn(*{**defaults, **kw}.values(), S)


GEMM = dict(x=P, w=P, dtype=BF16, rows=64, E=4, n=32, k=64, flags=0, off=P, sizes=P, out=P,
            out_dtype=BF16, gate_up=None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=F32), DTYPE), (dict(dtype=FP8), DTYPE), (dict(out_dtype=I32), DTYPE),
    (dict(rows=-1), INVALID), (dict(rows=2**31), INVALID), (dict(E=0), INVALID),
    (dict(E=1025), INVALID), (dict(n=0), INVALID), (dict(k=0), INVALID),
    (dict(n=2**20 + 1), INVALID), (dict(k=2**20 + 1), INVALID), (dict(flags=4), INVALID),
    (dict(flags=TRANSPOSED | SILU), INVALID), (dict(gate_up=P), INVALID),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(out=None), INVALID),
    (dict(off=None), INVALID), (dict(off=P + 2), MISALIGNED), (dict(sizes=P + 2), MISALIGNED),
    (dict(x=P + 1), MISALIGNED), (dict(w=P + 1), MISALIGNED), (dict(out=P + 1), MISALIGNED),
    (dict(out=P + 2, out_dtype=F32), MISALIGNED),
    (dict(flags=SILU, gate_up=P + 2, out_dtype=F32), MISALIGNED),
    (dict(rows=0), OK), (dict(rows=0, x=None, w=None, out=None), OK)])
def test_grouped_gemm(lib, kw, status):
    assert _call(lib.mx_grouped_gemm, GEMM, **kw) == status


GEMM8 = dict(x=P, xs=P, w=P, ws=P, rows=64, E=4, n=32, k=256, flags=0, off=P, sizes=None, out=P,
             out_dtype=BF16)


@pytest.mark.parametrize("kw,status", [
    (dict(out_dtype=F32), DTYPE), (dict(out_dtype=FP8), DTYPE), (dict(k=64), INVALID),
    (dict(flags=TRANSPOSED), INVALID), (dict(flags=SILU, n=24), INVALID), (dict(E=0), INVALID),
    (dict(x=None), INVALID), (dict(xs=None), INVALID), (dict(w=None), INVALID),
    (dict(ws=None), INVALID), (dict(out=None), INVALID), (dict(off=None), INVALID),
    (dict(x=P + 8), MISALIGNED), (dict(w=P + 8), MISALIGNED), (dict(xs=P + 2), MISALIGNED),
    (dict(ws=P + 2), MISALIGNED), (dict(out=P + 1), MISALIGNED), (dict(rows=0), OK)])
def test_grouped_gemm_fp8(lib, kw, status):
    assert _call(lib.mx_grouped_gemm_fp8, GEMM8, **kw) == status


GEMM4 = dict(x=P, dtype=F16, w=P, scales=P, zeros=None, group=64, rows=64, E=4, n=32, k=256,
             flags=0, off=P, sizes=None, out=P)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=F32), DTYPE), (dict(group=16), INVALID), (dict(group=256), INVALID),
    (dict(group=0), INVALID), (dict(group=-64), INVALID), (dict(k=96), INVALID),
    (dict(flags=TRANSPOSED), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID),
    (dict(scales=None), INVALID), (dict(out=None), INVALID), (dict(n=0), INVALID),
    (dict(x=P + 8), MISALIGNED), (dict(w=P + 4), MISALIGNED), (dict(scales=P + 1), MISALIGNED),
    (dict(out=P + 1), MISALIGNED), (dict(rows=0), OK)])
def test_grouped_gemm_w4(lib, kw, status):
    assert _call(lib.mx_grouped_gemm_w4, GEMM4, **kw) == status


WGRAD = dict(d=P, x=P, dtype=BF16, rows=64, E=4, n=32, k=64, off=P, sizes=P, out=P,
             out_dtype=F32, accumulate=0)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=F32), DTYPE), (dict(out_dtype=I64), DTYPE), (dict(rows=-1), INVALID),
    (dict(n=0), INVALID), (dict(k=0), INVALID), (dict(d=None), INVALID), (dict(x=None), INVALID),
    (dict(out=None), INVALID), (dict(out=None, rows=0), INVALID), (dict(off=None), INVALID),
    (dict(d=P + 1), MISALIGNED), (dict(out=P + 2), MISALIGNED), (dict(sizes=P + 1), MISALIGNED)])
def test_grouped_gemm_wgrad(lib, kw, status):
    assert _call(lib.mx_grouped_gemm_wgrad, WGRAD, **kw) == status


SILU_BACK = dict(d=P, gu=P, dtype=BF16, rows=64, E=4, n=32, off=P, sizes=P, out=P)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=F32), DTYPE), (dict(n=0), INVALID), (dict(E=0), INVALID), (dict(d=None), INVALID),
    (dict(gu=None), INVALID), (dict(out=None), INVALID), (dict(off=None), INVALID),
    (dict(d=P + 1), MISALIGNED), (dict(gu=P + 1), MISALIGNED), (dict(out=P + 1), MISALIGNED),
    (dict(rows=0), OK)])
def test_silu_mul_backward(lib, kw, status):
    assert _call(lib.mx_silu_mul_backward, SILU_BACK, **kw) == status


GATING = dict(x=P, dtype=F32, T=10, E=64, k=8, scoring=0, bias=None, renorm=1, scale=1.0, ids=P,
              w=P)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=I32), DTYPE), (dict(dtype=FP8), DTYPE), (dict(T=-1), INVALID), (dict(E=0), INVALID),
    (dict(E=1025), INVALID), (dict(k=0), INVALID), (dict(k=65, E=100), INVALID),
    (dict(E=4, k=5), INVALID), (dict(scoring=2), INVALID), (dict(bias=P), INVALID),
    (dict(bias=P + 2, scoring=1), MISALIGNED), (dict(x=None), INVALID), (dict(ids=None), INVALID),
    (dict(w=None), INVALID), (dict(T=2**31, k=1), INVALID), (dict(x=P + 2), MISALIGNED),
    (dict(ids=P + 2), MISALIGNED), (dict(w=P + 2), MISALIGNED), (dict(T=0), OK)])
def test_topk_gating(lib, kw, status):
    assert _call(lib.mx_topk_gating, GATING, **kw) == status


GATING_BACK = dict(x=P, dtype=BF16, T=10, E=64, k=8, scoring=1, renorm=0, scale=1.0, ids=P, w=P,
                   out=P)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=I64), DTYPE), (dict(E=0), INVALID), (dict(k=65, E=100), INVALID),
    (dict(scoring=-1), INVALID), (dict(out=None), INVALID), (dict(x=None), INVALID),
    (dict(out=P + 1), MISALIGNED), (dict(x=P + 1), MISALIGNED), (dict(T=0), OK)])
def test_topk_gating_backward(lib, kw, status):
    assert _call(lib.mx_topk_gating_backward, GATING_BACK, **kw) == status


MUTATED = {
    "topk_gating": {"topk_ids", "topk_weights"}, "topk_gating_backward": {"grad_logits"},
    "grouped_gemm": {"output", "gate_up"}, "grouped_gemm_fp8": {"output"},
    "grouped_gemm_w4": {"output"}, "grouped_gemm_wgrad": {"grad_weight"},
    "silu_mul_backward": {"grad_gate_up"},
}


@pytest.mark.parametrize("name", sorted(MUTATED))
def test_operator_schema_marks_the_outputs(name):
    import torch
    import combine_topk_ids_expert_amd.ops  # noqa: F401  (registers torch.ops.mxmoe)
    schema = getattr(torch.ops.mxmoe, name).default._schema
    written = {a.name for a in schema.arguments
               if a.alias_info is not None and a.alias_info.is_write}
    assert written == MUTATED[name] and len(schema.returns) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(flags=SILU, n=2**15, k=2**15), OK), (dict(flags=SILU, n=2**15 + 1, k=2**15), INVALID)])
def test_gated_products_stay_in_32_bit_offsets(lib, kw, status):
    assert _call(lib.mx_grouped_gemm, GEMM, rows=0, **kw) == status
