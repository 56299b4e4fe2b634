"""A layer of routed experts in 8-bit floating point, without a number
returning to the host:

    slots -> experts' rows       qg_moe_sort (offsets, places)
    tokens -> rows as codes      qg_moe_dispatch (e4m3, a scale for 128 elements)
    rows x [gate; up]            qgemm_e4m3_moe (128 x 128 block scales)
    silu(gate) * up -> codes     torch, then qg_moe_dispatch without places
    rows x down                  qgemm_e4m3_moe
    rows -> tokens               qg_moe_combine with the router's weights

The whole layer is captured into one CUDA graph and replayed on new tokens,
whatever their experts.

    python examples/expert_layer.py [--tokens 4096] [--experts 64] [--top 8]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_only_quantized_i4g_gb300 as qg  # noqa: E402

BLOCK = 128
E4M3 = torch.float8_e4m3fn


def blocks(n: int) -> int:
    return -(-n // BLOCK)


def expect(name: str, t: torch.Tensor, dtype: torch.dtype, *shape: int) -> None:
    """The library gets addresses alone: the type, the shape and whole rows one after another are checked here."""
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} {list(shape)}, not {t.dtype} {list(t.shape)} with strides "
                         f"{list(t.stride())}")


def pack(w: torch.Tensor):
    """f32 weights [.., O, I] as e4m3 codes and one f32 scale for each 128 x 128 block (largest value -> 448)."""
    *lead, o, i = w.shape
    nbo, nbi = blocks(o), blocks(i)
    p = torch.nn.functional.pad(w, (0, nbi * BLOCK - i, 0, nbo * BLOCK - o)).view(*lead, nbo, BLOCK, nbi, BLOCK)
    scale = p.abs().amax((-3, -1)).clamp_min(1e-30) / 448.0
    codes = (p / scale[..., :, None, :, None]).to(E4M3)
    codes = codes.view(torch.uint8).reshape(*lead, nbo * BLOCK, nbi * BLOCK)[..., :o, :i].contiguous()
    return codes.view(E4M3), scale.contiguous()


class ExpertLayer:
    """`up` f32 [E, 2 F, H] (gate rows, then up rows) and `down` f32 [E, H, F]; at most `tokens` tokens a call."""

    def __init__(self, up: torch.Tensor, down: torch.Tensor, tokens: int, top: int):
        dev = up.device
        self.E, two_f, self.H = up.shape
        self.F, self.top, self.tokens = two_f // 2, top, tokens
        self.up, self.up_scale = pack(up)
        self.down, self.down_scale = pack(down)
        n = self.rows = tokens * top
        self.offsets = torch.zeros(self.E + 1, dtype=torch.int32, device=dev)
        self.place = torch.zeros(n, dtype=torch.int32, device=dev)
        self.x = torch.zeros(n, self.H, dtype=E4M3, device=dev)
        self.x_scale = torch.zeros(n, blocks(self.H), device=dev)
        self.gu = torch.zeros(n, two_f, dtype=torch.bfloat16, device=dev)
        self.act = torch.zeros(n, self.F, dtype=torch.bfloat16, device=dev)
        self.a = torch.zeros(n, self.F, dtype=E4M3, device=dev)
        self.a_scale = torch.zeros(n, blocks(self.F), device=dev)
        self.y = torch.zeros(n, self.H, dtype=torch.bfloat16, device=dev)
        self.ws_bytes = max(qg.qg_moe_sort_workspace_bytes(tokens, top, self.E),
                            qg.qgemm_e4m3_workspace_bytes(n, self.H, two_f, self.E),
                            qg.qgemm_e4m3_workspace_bytes(n, self.F, self.H, self.E))
        self.ws = torch.empty(max(self.ws_bytes, 1), dtype=torch.uint8, device=dev)

    def __call__(self, out: torch.Tensor, tokens: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor) -> None:
        """tokens bf16 [T, H], ids int32 [T, top] (outside [0, E): no expert here), weights f32 [T, top] -> out bf16."""
        t, k, n = tokens.shape[0], self.top, self.rows
        if t > self.tokens:
            raise ValueError(f"{t} tokens, but the layer was made for {self.tokens}")
        if tokens.dtype != torch.bfloat16 or tokens.shape[1:] != (self.H,) or tokens.stride(1) != 1:
            raise ValueError(f"tokens must be bfloat16 rows of {self.H} elements side by side")
        expect("out", out, torch.bfloat16, t, self.H)
        expect("ids", ids, torch.int32, t, k)
        expect("weights", weights, torch.float32, t, k)
        ws = (self.ws, self.ws_bytes)
        qg.check(qg.qg_moe_sort(self.offsets, None, self.place, ids, t, k, self.E, *ws))
        qg.check(qg.qg_moe_dispatch(self.x, qg.QG_E4M3, self.x_scale, tokens, qg.QG_BF16, tokens.stride(0), self.place,
                                    t, k, self.H, n))
        qg.check(qg.qgemm_e4m3_moe(qg.QG_FMT_FP8B128, self.gu, qg.QG_BF16, self.x, self.x_scale, self.up, self.up_scale,
                                   self.offsets, self.E, n, self.H, 2 * self.F, *ws))
        torch.mul(torch.nn.functional.silu(self.gu[:, :self.F]), self.gu[:, self.F:], out=self.act)
        qg.check(qg.qg_moe_dispatch(self.a, qg.QG_E4M3, self.a_scale, self.act, qg.QG_BF16, self.F, None, n, 1, self.F, n))
        qg.check(qg.qgemm_e4m3_moe(qg.QG_FMT_FP8B128, self.y, qg.QG_BF16, self.a, self.a_scale, self.down, self.down_scale,
                                   self.offsets, self.E, n, self.F, self.H, *ws))
        qg.check(qg.qg_moe_combine(out, qg.QG_BF16, self.y, qg.QG_BF16, weights, self.place, t, k, self.H, n))


class Dispatch(torch.autograd.Function):
    """Token rows [T, H] to their experts' rows, copied, by places int32 [T, top]; their gradient comes back summed over
    a token's slots."""

    @staticmethod
    def forward(ctx, x, place, n_rows):
        expect("place", place, torch.int32, x.shape[0], place.shape[-1])
        x = x.contiguous()
        rows = torch.zeros(n_rows, x.shape[1], dtype=x.dtype, device=x.device)
        t = TYPES[x.dtype]
        qg.check(qg.qg_moe_dispatch(rows, t, None, x, t, x.shape[1], place, x.shape[0], place.shape[1], x.shape[1], n_rows))
        ctx.save_for_backward(place)
        return rows

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        place, = ctx.saved_tensors
        grad = grad.contiguous()
        dx = torch.empty(place.shape[0], grad.shape[1], dtype=grad.dtype, device=grad.device)
        t = TYPES[grad.dtype]
        qg.check(qg.qg_moe_combine(dx, t, grad, t, None, place, place.shape[0], place.shape[1], grad.shape[1], grad.shape[0]))
        return dx, None, None


class Combine(torch.autograd.Function):
    """Experts' rows [n, H] back to their tokens with the router's weights f32 [T, top] by places int32 [T, top];
    gradients of rows and weights."""

    @staticmethod
    def forward(ctx, y, weights, place):
        y, weights = y.contiguous(), weights.contiguous()
        expect("place", place, torch.int32, *place.shape[:1], place.shape[-1])
        expect("weights", weights, torch.float32, *place.shape)
        out = torch.empty(place.shape[0], y.shape[1], dtype=y.dtype, device=y.device)
        t = TYPES[y.dtype]
        qg.check(qg.qg_moe_combine(out, t, y, t, weights, place, place.shape[0], place.shape[1], y.shape[1], y.shape[0]))
        ctx.save_for_backward(y, weights, place)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        y, weights, place = ctx.saved_tensors
        grad = grad.contiguous()
        dy = torch.zeros_like(y) if ctx.needs_input_grad[0] else None
        dw = torch.empty_like(weights) if ctx.needs_input_grad[1] else None
        qg.check(qg.qg_moe_combine_grad(dy, dw, grad, TYPES[grad.dtype], y, TYPES[y.dtype], weights, place, place.shape[0],
                                        place.shape[1], y.shape[1], y.shape[0]))
        return dy, dw, None


TYPES = {torch.float32: qg.QG_F32, torch.bfloat16: qg.QG_BF16, torch.float16: qg.QG_F16}


def capture(layer: ExpertLayer, out, tokens, ids, weights) -> torch.cuda.CUDAGraph:
    """The layer as a graph on these tensors, after one run on a stream of its own (out holds its result); what the
    current stream has been given so far, such as the tokens and the layer's buffers, comes first."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(out, tokens, ids, weights)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(out, tokens, ids, weights)
    return graph


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--top", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=5120)
    ap.add_argument("--width", type=int, default=2048)
    a = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)
    up = torch.randn(a.experts, 2 * a.width, a.hidden, generator=g, device="cuda") * a.hidden ** -0.5
    down = torch.randn(a.experts, a.hidden, a.width, generator=g, device="cuda") * a.width ** -0.5
    layer = ExpertLayer(up, down, a.tokens, a.top)
    del up, down
    x = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").bfloat16()
    ids = torch.zeros(a.tokens, a.top, dtype=torch.int32, device="cuda")
    weights = torch.zeros(a.tokens, a.top, device="cuda")
    out = torch.empty_like(x)

    def route():
        top = torch.topk(torch.randn(a.tokens, a.experts, generator=g, device="cuda"), a.top, 1)
        ids.copy_(top.indices)
        weights.copy_(torch.softmax(top.values, 1))
    route()
    graph = capture(layer, out, x, ids, weights)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for i in range(22):
        if i == 2:
            begin.record()
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    rc, status = qg.qg_device_status()
    qg.check(rc or status)
    ms = begin.elapsed_time(end) / 20
    flops = 6.0 * a.tokens * a.top * a.hidden * a.width
    print(f"{a.tokens} tokens, {a.experts} experts of {a.width}, {a.top} a token: {ms * 1e3:.1f} us, "
          f"{flops / ms / 1e9:.0f} TFLOP/s over the whole layer")


if __name__ == "__main__":
    main()
