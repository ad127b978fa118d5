"""The attention half of a tensor-parallel block as a server runs it, its P ranks
emulated on one GPU: a prompt, then tokens one at a time.

    python examples/tensor_parallel_decode.py [--sequences 8] [--prompt 200] [--steps 4] [--ranks 4]

Every kernel is from libecho.so; weights and cache are in groups of 4 bits:

  echo_quantize_weights  each rank's projections, once
  echo_norm              joins the last all-reduced output with the residual
                         stream and normalises the block's input
  echo_linear_int4       each rank's query, key and value projections (all ranks
                         share the tokens)
  echo_cache_append      the new tokens' keys and values, quantised into pages
  echo_attention         all ranks' heads over the sequences' pages
  echo_linear_int4       each rank's output projection of its heads' slice, the
                         partial sums
  echo_allreduce         4-bit, with the error fed back

The same step in 64 bits, from the weights and the cache as they are held, shows
how far the arithmetic is off, and from the original ones what 4 bits cost.
"""
import argparse
import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


class Projection:
    """Weights [ranks][channels][depth] in 4-bit groups, and the values that they hold."""

    def __init__(self, w, group=128):
        from bit_error_compensated_gb300 import echo
        self.group, self.exact = group, w.double()
        ranks, channels, depth = w.shape
        self.codes = torch.empty(ranks, channels, (depth + 1) // 2, dtype=torch.uint8, device=w.device)
        self.meta = torch.empty(ranks, channels, (depth + group - 1) // group, dtype=torch.int32, device=w.device)
        echo.echo_quantize_weights(w, self.codes, self.meta, group=group)

    def held(self):
        code = torch.stack([self.codes & 15, self.codes >> 4], -1).flatten(-2).double()
        both = self.meta.view(torch.float16).view(*self.meta.shape, 2).double()
        step, zero = (both[..., i].repeat_interleave(self.group, -1)[..., :code.shape[-1]] for i in (0, 1))
        return step * (code - zero)

    def __call__(self, x, out):
        from bit_error_compensated_gb300 import echo
        echo.echo_linear_int4(x, self.codes, self.meta, out, group=self.group)
        return out


def run(sequences=8, prompt=200, steps=4, ranks=4, width=1024, heads=16, kv_heads=8, dim=64, page=32, bits=4, seed=0):
    """The largest errors over the steps, relative, by name."""
    from bit_error_compensated_gb300 import echo
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")              # noqa: E731
    P, bf = ranks, torch.bfloat16
    part = lambda n: n * dim // P                                                # noqa: E731
    wq, wk, wv = (Projection(rand(P, part(n), width) / math.sqrt(width)) for n in (heads, kv_heads, kv_heads))
    wo = Projection(rand(P, width, part(heads)) / math.sqrt(heads * dim))

    # what a server keeps: the join's plan, the cache, the batch's arrays
    join = echo.echo_norm_plan(width, bf, post=False)
    most = (prompt + steps + page - 1) // page
    cache = echo.Cache(sequences * most, page, kv_heads, dim, bits)
    table = torch.randperm(sequences * most, generator=gen, device="cuda").int().view(sequences, most)
    lengths = torch.zeros(sequences, dtype=torch.int32, device="cuda")
    off = {}
    for step in range(1 + steps):
        new = prompt if step == 0 else 1
        T = sequences * new
        starts = torch.arange(0, T + 1, new, dtype=torch.int32, device="cuda")
        lengths += new
        batch = echo.CacheBatch(starts, lengths, table)
        x, y = rand(T, width).to(bf), rand(T, width).to(bf)
        residual, h = torch.empty_like(x), torch.empty_like(x)
        q, k, v = (torch.empty(T, n * dim, dtype=bf, device="cuda") for n in (heads, kv_heads, kv_heads))
        attended = torch.empty_like(q)
        partial = torch.empty(P, T, width, dtype=bf, device="cuda")
        summed = torch.empty_like(partial)
        site = echo.echo_plan(P, T * width, 128, 4)

        # the step
        echo.echo_norm(join, None, x, y, residual, h)
        for w, t in ((wq, q), (wk, k), (wv, v)):             # ranks' channels side by side in a token's row
            w(h, t.view(T, P, -1).transpose(0, 1))
        as_heads = lambda t: t.view(T, -1, dim)                                  # noqa: E731
        echo.echo_cache_append(cache, batch, as_heads(k), as_heads(v))
        echo.echo_attention(cache, batch, as_heads(q), as_heads(attended))
        wo(attended.view(T, P, -1).transpose(0, 1), partial)
        echo.echo_allreduce(site, [t.view(-1) for t in partial], [t.view(-1) for t in summed], echo.COMP_DEFAULT)

        # the same in 64 bits, attention over what the cache holds
        length = prompt + step
        whole = echo.CacheBatch(torch.arange(0, sequences * length + 1, length, dtype=torch.int32, device="cuda"), lengths, table)
        kept = [torch.empty(sequences * length, kv_heads, dim, device="cuda") for _ in range(2)]
        echo.echo_cache_read(cache, whole, *kept)
        keys, values = (t.view(sequences, length, kv_heads, dim).double().repeat_interleave(heads // kv_heads, 2) for t in kept)
        qs = q.view(sequences, new, heads, dim).double()
        score = torch.einsum("bthd,bshd->bhts", qs, keys) / math.sqrt(dim)
        place = torch.arange(length, device="cuda")
        score.masked_fill_(place > place[length - new:, None], -math.inf)
        want = torch.einsum("bhts,bshd->bthd", torch.softmax(score, -1), values).reshape(T, -1)
        block = torch.einsum("tpk,pdk->td", attended.view(T, P, -1).double(), wo.held())
        query = torch.einsum("td,pcd->tpc", h.double(), wq.held()).reshape(T, -1)
        plain = torch.einsum("td,pcd->tpc", h.double(), wq.exact).reshape(T, -1)
        now = {"query": (q, query), "attention": (attended, want), "block": (summed[0], block),
               "partial": (partial.double().sum(0), block), "weights": (query, plain)}
        for name, (got, ref) in now.items():
            off[name] = max(off.get(name, 0.0), float((got.double() - ref).norm() / ref.norm()))
    off["status"] = max(echo.echo_serving_status(), echo.echo_get_status(site))
    return off


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("sequences", 8), ("prompt", 200), ("steps", 4), ("ranks", 4)):
        ap.add_argument("--" + name, type=int, default=value)
    for name, value in run(**vars(ap.parse_args())).items():
        print(f"{name:10s} {value:.3g}")


if __name__ == "__main__":
    main()
