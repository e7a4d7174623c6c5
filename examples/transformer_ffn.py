"""The feed-forward halves of two transformer layers, decode step by decode step.

Layer 0 is dense: residual addition, norm and quantisation in one call, the
gated projection, the down projection (``DenseFfn``).  Layer 1 is a mixture of
experts: the same norm call writes a bf16 copy of its result, which the router
and the experts read.  The step is captured once into a CUDA graph and replayed.

    python examples/transformer_ffn.py [--hidden 1024] [--tokens 8] [--steps 20]

Weights and activations are random; the attention halves are left out.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import moe_expert_ffn_02_gb300 as moe  # noqa: E402


def fp8_blocks(*shape):
    """Random [..., out, in] weights in E4M3 with an fp32 scale per 128 x 128 block."""
    w = torch.randn(*shape, device="cuda") * 0.02
    *lead, n, k = shape
    blocks = w.view(*lead, n // 128, 128, k // 128, 128)
    s = blocks.abs().amax((-3, -1)) / 448.0
    q = (blocks / s[..., :, None, :, None]).reshape(shape).to(torch.float8_e4m3fn)
    return q, s


def expert_layer(hidden, inter, experts, top_k):
    w = {"router_w": torch.randn(experts, hidden, device="cuda") * 0.05, "router_b": None}
    for name, lead, n, k in (("gate", (experts,), inter, hidden), ("up", (experts,), inter, hidden), ("down", (experts,), hidden, inter)):
        q, w["s_" + name] = fp8_blocks(*lead, n, k)
        w["w_" + name] = q.view(torch.uint8)
        q, w["sh_s_" + name] = fp8_blocks(n, k)
        w["sh_" + name] = q.view(torch.uint8)
    return moe.Layer(hidden, inter, experts, top_k, w)


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--hidden", type=int, default=1024)
    p.add_argument("--tokens", type=int, default=8)
    p.add_argument("--steps", type=int, default=20)
    args = p.parse_args()
    h, t = args.hidden, args.tokens
    torch.manual_seed(0)

    norm0, norm1 = (moe.RmsNorm(1 + 0.1 * torch.randn(h, device="cuda")) for _ in range(2))
    dense = moe.DenseFfn(norm0, moe.Fp8GatedLinear(*fp8_blocks(2 * h, h), *fp8_blocks(2 * h, h)), moe.Fp8Linear(*fp8_blocks(h, 2 * h)))
    layer = expert_layer(h, h // 2, experts=16, top_k=4)
    mode = moe.MODE_DECODE if t <= 64 else moe.MODE_PREFILL
    forward = moe.moe_forward_decode if t <= 64 else moe.moe_forward_prefill
    ws, ws_bytes = layer.workspace(t, mode)

    x = torch.randn(t, h, device="cuda").bfloat16()           # what the attention half of layer 0 adds
    res = torch.zeros(t, h, device="cuda")                    # fp32 residual stream
    y0, n1, y1 = (torch.empty(t, h, dtype=torch.bfloat16, device="cuda") for _ in range(3))

    def step():
        dense(x, res, y0)                                     # res += x; y0 = FFN(norm(res))
        norm1(y0, res, res_out=res, y=n1)                     # res += y0; n1 = norm(res)
        forward(layer.handle, n1.data_ptr(), t, y1.data_ptr(), None, ws, ws_bytes, torch.cuda.current_stream().cuda_stream)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        res.zero_()
        graph.replay()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(args.steps):
        graph.replay()
    end.record()
    res.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for part in (dense.gate_up, dense.down):
        assert part.device_status() == (0, 0)
    v = x.float() + y0.float()
    print(f"{t} tokens, hidden {h}: {begin.elapsed_time(end) / args.steps * 1e3:.1f} us a step")
    print(f"rms: residual {v.square().mean().sqrt():.3f}, dense FFN {y0.float().square().mean().sqrt():.4f}, experts {y1.float().square().mean().sqrt():.4f}")
    assert torch.allclose(res, v, atol=1e-5) and torch.isfinite(y1).all()


if __name__ == "__main__":
    main()
