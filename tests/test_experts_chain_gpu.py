"""The expert layer as a whole, from router logits to tokens and back: gating,
routing, dispatch, the two products with the gated activation, combine, and the
gradients of rows, weights and logits, against a float64 layer with torch's
autograd.  Also on other streams, in a captured graph, as custom operators, and
through the FP8 and 4-bit products of serving."""

import numpy as np
import pytest
import torch

import combine_topk_ids_expert_amd as mx
import combine_topk_ids_expert_amd.ops  # noqa: F401  (registers torch.ops.mxmoe)
from tests import experts_util as eu

pytestmark = pytest.mark.gpu

DEV = eu.DEV
BF16 = torch.bfloat16
T, E, K, H, N = 50, 6, 2, 128, 96


def _inputs(seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H), generator=g).to(BF16)
    logits = torch.randn((T, E), generator=g) * 1.5
    logits[:, 4] = -float("inf")                       # an expert nobody gets
    w1 = (torch.randn((E, 2 * N, H), generator=g) * H ** -0.5).to(BF16)
    w2 = (torch.randn((E, H, N), generator=g) * N ** -0.5).to(BF16)
    dout = torch.randn((T, H), generator=g).to(BF16)
    return x, logits, w1, w2, dout


def _buffers(align=16):
    b = mx.empty_routing(T, K, E, DEV, row_align=align)
    rows = b["input_permutation"].numel()

    def nan(*shape, dtype=BF16):
        return torch.full(shape, float("nan"), dtype=dtype, device=DEV)
    b.update(ids=torch.empty(T, K, dtype=torch.int32, device=DEV), weights=nan(T, K, dtype=torch.float32),
             xd=nan(rows, H), gate_up=nan(rows, 2 * N), h=nan(rows, N), y=nan(rows, H),
             out=nan(T, H, dtype=torch.float32), align=align)
    return b


def _forward(b, x, logits, w1, w2):
    mx.topk_gating(logits, b["ids"], b["weights"])
    mx.prepare_moe_input(b["ids"], b["expert_offsets"], b["problem_sizes1"], b["problem_sizes2"],
                         b["input_permutation"], b["output_permutation"], E, N, H,
                         row_align=b["align"], workspace=b["workspace"])
    mx.dispatch_rows(x, b["output_permutation"], K, b["xd"])
    o, z = b["expert_offsets"], b["problem_sizes1"]
    mx.grouped_gemm(b["xd"], w1, o, b["h"], z, silu_mul=True, gate_up=b["gate_up"])
    mx.grouped_gemm(b["h"], w2, o, b["y"], b["problem_sizes2"])
    mx.apply_shuffle_mul_sum(b["y"], b["out"], b["output_permutation"], b["weights"])


def _backward(b, logits, w1, w2, dout):
    """Gradients of x, the weights and the logits.  The gradient of combine is
    dispatch (dy of a pick: its weight times dout) and a dot product a pick."""
    o, z = b["expert_offsets"], b["problem_sizes1"]
    perm = b["output_permutation"].long()
    dw = (b["y"][perm].view(T, K, H).float() * dout.float()[:, None]).sum(2)
    dy = torch.full_like(b["y"], float("nan"))
    dy[perm] = (dout.float()[:, None] * b["weights"][..., None]).to(BF16).view(T * K, H)
    g = {"w1": torch.empty_like(w1, dtype=torch.float32), "w2": torch.empty_like(w2, dtype=torch.float32),
         "x": torch.empty(T, H, device=DEV), "logits": torch.empty_like(logits)}
    dh, dgu, dxd = torch.full_like(b["h"], float("nan")), torch.full_like(b["gate_up"], float("nan")), \
        torch.full_like(b["xd"], float("nan"))
    mx.grouped_gemm(dy, w2, o, dh, z, transpose_weight=True)
    mx.grouped_gemm_wgrad(dy, b["h"], o, g["w2"], z)
    mx.silu_mul_backward(dh, b["gate_up"], o, dgu, z)
    mx.grouped_gemm(dgu, w1, o, dxd, z, transpose_weight=True)
    mx.grouped_gemm_wgrad(dgu, b["xd"], o, g["w1"], z)
    mx.apply_shuffle_mul_sum(dxd, g["x"], b["output_permutation"])
    mx.topk_gating_backward(logits, b["ids"], dw, g["logits"])
    return g


def _reference(x, logits, w1, w2, dout):
    x, logits, w1, w2 = (v.double().requires_grad_() for v in (x, logits, w1, w2))
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    w = torch.softmax(top[:, :K], 1)
    out = torch.zeros(T, H, dtype=torch.float64)
    rows = []
    for t in range(T):
        acc = 0
        for j in range(K):
            e = int(ids[t, j])
            gu = w1[e] @ x[t]
            h = torch.nn.functional.silu(gu[:N]) * gu[N:]
            acc = acc + w[t, j] * (w2[e] @ h)
        rows.append(acc)
    out = torch.stack(rows)
    (out * dout.double()).sum().backward()
    return ids[:, :K].int(), out.detach(), {"x": x.grad, "logits": logits.grad, "w1": w1.grad,
                                            "w2": w2.grad}


def _near(got, want, what, roundings):
    """bf16 intermediates: each of `roundings` stored values is off by half a step
    (2^-8); in the 2-norm independent roundings add up to at most their sum."""
    off = (got.detach().cpu().double() - want).norm() / want.norm()
    assert off <= roundings * 2.0 ** -8, f"{what}: {float(off):.3g}"


@pytest.mark.parametrize("align", [1, 16])
def test_layer_forward_and_backward(align):
    x, logits, w1, w2, dout = _inputs()
    b = _buffers(align)
    dx, dl, d1, d2, dd = (v.to(DEV) for v in (x, logits, w1, w2, dout))
    _forward(b, dx, dl, d1, d2)
    ids, out, grads = _reference(x, logits, w1, w2, dout)
    assert torch.equal(b["ids"].cpu(), ids)
    _near(b["out"], out, "out", 2)                     # h, y
    g = _backward(b, dl, d1, d2, dd)
    _near(g["w2"], grads["w2"], "w2", 2)               # h, dy
    _near(g["w1"], grads["w1"], "w1", 4)               # dy, dh, gate_up, dgu
    _near(g["x"], grads["x"], "x", 5)                  # the same and dxd
    _near(g["logits"], grads["logits"].nan_to_num(0.0), "logits", 2)
    assert (g["w1"][4] == 0).all() and (g["w2"][4] == 0).all() and (g["logits"][:, 4] == 0).all()


def test_layer_on_another_stream_and_in_a_graph():
    """The same bits on a side stream, in a replayed graph (three replays, with
    new inputs and eager work between them) and eagerly."""
    eager = _buffers()
    graph_b = _buffers()
    side = torch.cuda.Stream()
    ins = [v.to(DEV) for v in _inputs(1)]
    static = [v.clone() for v in ins]
    with torch.cuda.stream(side):
        _forward(graph_b, *static[:4])
    side.synchronize()
    _forward(eager, *ins[:4])
    torch.cuda.synchronize()
    assert torch.equal(graph_b["out"], eager["out"])
    if mx.bounds_checked():
        pytest.skip("the bounds-checked library refuses capture")
    graph = torch.cuda.CUDAGraph()
    grads = {}
    with torch.cuda.graph(graph):
        _forward(graph_b, *static[:4])
        # the library's backward calls, into buffers of their own
        grads["w1"] = torch.empty(E, 2 * N, H, device=DEV)
        mx.grouped_gemm_wgrad(graph_b["gate_up"], graph_b["xd"], graph_b["expert_offsets"],
                              grads["w1"], graph_b["problem_sizes1"])
    for seed in (2, 3, 4):
        ins = [v.to(DEV) for v in _inputs(seed)]
        for s, v in zip(static, ins):
            s.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        eager = _buffers()
        _forward(eager, *ins[:4])
        want = torch.empty_like(grads["w1"])
        mx.grouped_gemm_wgrad(eager["gate_up"], eager["xd"], eager["expert_offsets"], want,
                              eager["problem_sizes1"])
        torch.cuda.synchronize()
        assert torch.equal(graph_b["ids"], eager["ids"])
        assert torch.equal(graph_b["out"], eager["out"])
        assert torch.equal(grads["w1"], want)


def test_two_streams_at_once():
    """Calls on two streams share nothing: the same bits as one after the other."""
    ins = [[v.to(DEV) for v in _inputs(s)] for s in (5, 6)]
    alone = [_buffers() for _ in ins]
    for b, i in zip(alone, ins):
        _forward(b, *i[:4])
    both = [_buffers() for _ in ins]
    streams = [torch.cuda.Stream() for _ in ins]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, b, i in zip(streams, both, ins):
            with torch.cuda.stream(s):
                _forward(b, *i[:4])
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert torch.equal(a["out"], b["out"])


def test_operators_are_the_calls():
    x, logits, w1, w2, _ = (v.to(DEV) for v in _inputs(7))
    a, b = _buffers(), _buffers()
    _forward(a, x, logits, w1, w2)
    q = torch.ops.mxmoe
    q.topk_gating(logits, b["ids"], b["weights"], "softmax", None, True, 1.0)
    q.prepare_moe_input(b["ids"], b["expert_offsets"], b["problem_sizes1"], b["problem_sizes2"],
                        b["input_permutation"], b["output_permutation"], E, N, H, None, 16, 128,
                        b["workspace"])
    q.dispatch_rows(x, b["output_permutation"], K, b["xd"], None, None)
    q.grouped_gemm(b["xd"], w1, b["expert_offsets"], b["h"], b["problem_sizes1"], False, True,
                   b["gate_up"])
    q.grouped_gemm(b["h"], w2, b["expert_offsets"], b["y"], None, False, False, None)
    q.apply_shuffle_mul_sum(b["y"], b["out"], b["output_permutation"], b["weights"])
    assert torch.equal(a["out"], b["out"])
    ga, gb = torch.empty_like(a["gate_up"]), torch.empty_like(a["gate_up"])
    mx.silu_mul_backward(a["h"], a["gate_up"], a["expert_offsets"], ga)
    q.silu_mul_backward(a["h"], a["gate_up"], a["expert_offsets"], gb, None)
    rows = int(a["expert_offsets"][-1])
    assert torch.equal(ga[:rows].view(torch.int16), gb[:rows].view(torch.int16))
    la, lb = torch.empty_like(logits), torch.empty_like(logits)
    mx.topk_gating_backward(logits, a["ids"], a["weights"], la)
    q.topk_gating_backward(logits, a["ids"], a["weights"], lb, "softmax", True, 1.0)
    assert torch.equal(la, lb)


def test_serving_from_fp8_dispatch():
    """dispatch_rows_fp8's codes and scales straight into the FP8 products."""
    x, logits, w1, _, _ = _inputs(8)
    b = _buffers()
    d = x.to(DEV)
    mx.topk_gating(logits.to(DEV), b["ids"], b["weights"])
    mx.prepare_moe_input(b["ids"], b["expert_offsets"], b["problem_sizes1"], None,
                         b["input_permutation"], b["output_permutation"], E, N, H, row_align=16,
                         workspace=b["workspace"])
    rows = b["xd"].shape[0]
    codes = torch.full((rows, H), 0x7f, dtype=torch.uint8, device=DEV)
    scales = torch.full((rows, H // 128), float("nan"), device=DEV)
    mx.dispatch_rows_fp8(d, b["output_permutation"], K, codes, scales)
    wq = (w1.float() * 64).to(torch.float8_e4m3fn)
    ws = torch.full((E, 2, 1), 1 / 64)
    mx.grouped_gemm_fp8(codes, scales, wq.to(DEV), ws.to(DEV), b["expert_offsets"], b["h"],
                        b["problem_sizes1"], silu_mul=True)
    inp = b["input_permutation"].cpu()
    off = b["expert_offsets"].cpu().numpy()
    used = inp >= 0
    xq = codes.view(torch.float8_e4m3fn).cpu().float().double() * scales.cpu().double()
    expert = torch.from_numpy(np.searchsorted(off, np.arange(rows), side="right") - 1)
    got = b["h"].cpu()
    for r in used.nonzero()[:, 0].tolist():
        w = wq[expert[r]].float().double() / 64
        y, s = w @ xq[r], w.abs() @ xq[r].abs()
        h, err = eu.gated(y[None], (2.0 ** -13 * s)[None])
        eu.check(got[r:r + 1], h, err, BF16, f"row {r}")
