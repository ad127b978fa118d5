"""A tensor-parallel MLP block in low precision, its P ranks emulated on one GPU.

    python examples/tensor_parallel_block.py [--tokens 512] [--ranks 4]

One step between two all-reduce sites, every kernel from libecho.so:

  echo_norm          joins the last all-reduced output with the residual stream
                     and quantizes the next block's input to int8
  echo_matmul_int8   each rank's column-parallel product (all ranks share the
                     tokens' codes)
  echo_linear_int8   each rank's row-parallel product of its slice, the partial
                     sums
  echo_allreduce     4-bit, with the error fed back
  echo_norm          joins its result; and backwards,
  echo_norm_backward the join's gradients

The same block in fp32 with exact weights shows how far the low precision is off.
"""
import argparse
import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def quantize_rows(w):
    """Weights [..., depth] to int8 codes and one scale a row (done once)."""
    scale = w.abs().amax(-1) / 127
    return torch.round(w / scale[..., None]).to(torch.int8), scale


def run(tokens=512, width=1024, inner=4096, ranks=4, seed=0):
    """The errors of one step, relative to fp32, by name."""
    from bit_error_compensated_gb300 import echo
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")               # noqa: E731
    P, part = ranks, inner // ranks
    up, down = rand(P, part, width) / math.sqrt(width), rand(P, width, part) / math.sqrt(inner)
    up8, up_scale = quantize_rows(up)
    down8, down_scale = quantize_rows(down)
    w_post, w_pre = 1 + 0.1 * rand(width), 1 + 0.1 * rand(width)
    x, y = rand(tokens, width).bfloat16(), rand(tokens, width).bfloat16()

    # what a model keeps for the site
    join = echo.echo_norm_plan(width, torch.bfloat16, torch.float32, kind=echo.ECHO_NORM_RMS, post=True)
    params = echo.NormParams(join, w_post=w_post, w_pre=w_pre)
    site = echo.echo_plan(P, tokens * width, 128, 4)
    codes = torch.empty(tokens, width, dtype=torch.int8, device="cuda")
    scales = torch.empty(tokens, device="cuda")
    residual = torch.empty_like(x)
    stats = torch.empty(tokens, 4, device="cuda")
    hidden = torch.empty(P, tokens, part, dtype=torch.bfloat16, device="cuda")
    hidden8 = torch.empty(P, tokens, part, dtype=torch.int8, device="cuda")
    hidden_scales = torch.empty(P, tokens, device="cuda")
    partial = torch.empty(P, tokens, width, dtype=torch.bfloat16, device="cuda")
    summed = torch.empty_like(partial)
    out, h = torch.empty_like(x), torch.empty_like(x)

    # the step
    echo.echo_norm(join, params, x, y, residual, None, codes=codes, scales=scales)
    echo.echo_matmul_int8(codes, scales, up8, up_scale, hidden)
    hidden.relu_()
    echo.echo_linear_int8(hidden, down8, down_scale, partial, hidden8, hidden_scales)
    flat = [t.view(-1) for t in partial], [t.view(-1) for t in summed]
    echo.echo_allreduce(site, *flat, echo.COMP_DEFAULT)
    block = summed[0]                       # every rank's row holds the same bits
    echo.echo_norm(join, params, residual, block, out, h, stats=stats)

    # and the join's gradients, for a loss that weights out and h at random
    d_out, d_h = rand(tokens, width).bfloat16(), rand(tokens, width).bfloat16()
    dx, dy = torch.empty_like(x), torch.empty_like(x)
    grads = {"w_post": torch.empty_like(w_post), "w_pre": torch.empty_like(w_pre)}
    echo.echo_norm_backward(join, params, residual, block, stats, d_out, d_h, dx, dy, echo.NormParams(join, **grads))

    # the same in fp32, by torch and its automatic differentiation
    norm = lambda v, w: v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6) * w    # noqa: E731
    r32 = x.float() + norm(y.float(), w_post)
    mid = torch.relu(torch.einsum("td,pcd->ptc", norm(r32, w_pre), up))
    block32 = torch.einsum("ptc,pdc->td", mid, down)
    out32 = r32 + norm(block32, w_post)
    leaves = [t.detach().float().requires_grad_() for t in (residual, block, w_post, w_pre)]
    out_ref = leaves[0] + norm(leaves[1], leaves[2])
    want = torch.autograd.grad([out_ref, norm(out_ref, leaves[3])], leaves, [d_out.float(), d_h.float()])

    off = lambda a, b: float((a.float() - b).norm() / b.norm())                  # noqa: E731
    return {"residual": off(residual, r32), "block": off(block, block32), "out": off(out, out32),
            "h": off(h, norm(out32, w_pre)), "dx": off(dx, want[0]), "dy": off(dy, want[1]),
            "dw_post": off(grads["w_post"], want[2]), "dw_pre": off(grads["w_pre"], want[3]),
            "status": max(echo.echo_get_status(site), echo.echo_matmul_status())}


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--ranks", type=int, default=4)
    args = ap.parse_args()
    for name, value in run(tokens=args.tokens, ranks=args.ranks).items():
        print(f"{name:10s} {value:.3g}")


if __name__ == "__main__":
    main()
