"""Plain 64-bit implementations of the operators of a serving step, and what
the kernels' roundings may add up to.  They run on whatever device their
tensors are on."""
import math

import torch


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def groups(v, bits):
    """Codes, steps and zero points of groups along the last dimension; a group
    with a non-finite value or a step beyond fp16 gets codes 0, a step of NaN and
    a zero point of 0."""
    v = v.double()
    top = 2 ** bits - 1
    lo, hi = v.amin(-1, keepdim=True).clamp(max=0), v.amax(-1, keepdim=True).clamp(min=0)
    wide = hi - lo
    # the least fp16 number s with s * top >= wide, from a candidate near it
    s = (wide / torch.full_like(wide, top)).half()
    bits16 = s.view(torch.int16).clone()
    for _ in range(2):
        bits16 += (bits16.view(torch.float16).double() * top < wide).to(torch.int16)
    for _ in range(2):
        below = (bits16 - 1).clamp(min=0)
        bits16 = torch.where((bits16 > 0) & (below.view(torch.float16).double() * top >= wide), below, bits16)
    s = bits16.view(torch.float16).double()
    s = torch.where(s == 0, torch.ones_like(s), s)
    bad = ~torch.isfinite(v).all(-1, keepdim=True) | ~torch.isfinite(s)
    z = torch.round(-lo / s).clamp(0, top)
    code = (torch.round(v / s) + z).clamp(0, top)
    nan = torch.full_like(s, math.nan)
    return (torch.where(bad, torch.zeros_like(code), code).to(torch.uint8), torch.where(bad, nan, s),
            torch.where(bad, torch.zeros_like(z), z))


def pack(code, bits):
    if bits == 8:
        return code.contiguous()
    if code.shape[-1] % 2:
        code = torch.nn.functional.pad(code, (0, 1))
    return code[..., 0::2] | (code[..., 1::2] << 4)


def unpack(packed, bits):
    return packed if bits == 8 else torch.stack([packed & 15, packed >> 4], -1).flatten(-2)


def words(s, z):
    """One int32 a group: the step's fp16 bits low, the zero point's high."""
    return torch.cat([s, z], -1).half().view(torch.int32).squeeze(-1)


def steps(meta):
    """(step, zero point) of words, in 64 bits, with a last dimension of 1."""
    both = meta.contiguous().view(torch.float16).view(*meta.shape, 2).double()
    return both[..., :1], both[..., 1:]


def sequences(starts, lengths, tokens):
    """(sequence, row, place) of each row that belongs to one, from host lists."""
    out = []
    for b in range(len(lengths)):
        n = starts[b + 1] - starts[b]
        out += [(b, starts[b] + i, lengths[b] - n + i) for i in range(n) if 0 <= starts[b] + i < tokens]
    return out


class Held:
    """What a cache holds for the first `keys` places of a sequence and a head."""

    def __init__(self, cache, table_row, keys, head):
        place = torch.arange(keys, device=cache.codes.device)
        page = table_row.long()[place // cache.page_size]
        self.there = (page >= 0) & (page < cache.pages)
        page, at = page.clamp(0, cache.pages - 1), place % cache.page_size
        self.k, self.v = (self._of(cache, page, at, i, head) for i in (0, 1))

    def _of(self, cache, page, at, i, head):
        code = unpack(cache.codes[page, i, head, at], cache.bits).double()
        s, z = steps(cache.meta[page, i, head, at])
        return {"code": code, "s": s, "z": z, "value": s * (code - z)}


def attention(cache, q, starts, lengths, table, scale, causal=True, window=0):
    """(out, lse, tolerance) in 64 bits.  The tolerance is what the kernels'
    arithmetic may be off before out is rounded, element by element:
      weights   p_j = w_j s_j is rounded to f16: by 2^-11 of itself, or by half a
                subnormal step, 2^-25 of a p_j that is no less than 1 when the
                largest is scaled to between 1 and 2^8: n 2^-25 max p |c - z|;
      scores    fp32 sums of D products: (D + 4) 2^-23 of their absolute values;
                the exponential's argument and its function 4 2^-23 of the score
                and 2^-20; an error e of the scores changes a weight by e, and
                so out by 2 e of the mean of |v|;
      sums      n + 64 fp32 additions of p_j (c_j - z_j): (n + 64) 2^-23 of the
                mean of |v|."""
    T, H, D = q.shape
    group = H // cache.heads
    out = torch.zeros(T, H, D, dtype=torch.float64, device=q.device)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    room = table.shape[1] * cache.page_size
    for b in range(len(lengths)):
        rows = [(r, p) for bb, r, p in sequences(starts, lengths, T) if bb == b]
        keys = min(lengths[b], room)
        if not rows or keys <= 0:
            continue
        row = torch.tensor([r for r, _ in rows], device=q.device)
        place = torch.tensor([p for _, p in rows], device=q.device)
        for h in range(cache.heads):
            held = Held(cache, table[b], keys, h)
            qs = q[row, h * group:(h + 1) * group].double().flatten(0, 1)
            at = place.repeat_interleave(group)[:, None]
            key = torch.arange(keys, device=q.device)
            seen = held.there[None] & (at >= 0)              # a token before the begin sees nothing
            if causal:
                seen &= key <= at
                if window:
                    seen &= key > at - window
            score = (qs @ held.k["value"].T) * scale
            score = torch.where(seen, score, torch.full_like(score, -math.inf))
            top = score.amax(1, keepdim=True)
            any_key = seen.any(1, keepdim=True)
            w = torch.where(seen, torch.exp(score - torch.where(any_key, top, torch.zeros_like(top))), torch.zeros_like(score))
            total = w.sum(1, keepdim=True)
            safe = torch.where(any_key, total, torch.ones_like(total))
            hide = lambda t: torch.where(seen.any(0)[:, None], t, torch.zeros_like(t))        # noqa: E731
            v, s, c, z = (hide(held.v[n]) for n in ("value", "s", "code", "z"))
            got = (w @ v) / safe
            # NaN steps reach only the rows that see them
            bad_v = ((seen.double() @ torch.isnan(held.v["s"]).double()) > 0) | torch.isnan(total)
            clean = torch.nan_to_num(v)
            got = torch.where(bad_v, torch.full_like(got, math.nan), (torch.nan_to_num(w) @ clean) / safe)
            p = torch.nan_to_num(w * torch.nan_to_num(s).T)
            n = seen.sum(1, keepdim=True)
            mean = (torch.nan_to_num(w) @ clean.abs()) / safe
            plain = torch.nan_to_num(qs.abs() @ held.k["value"].abs().T)
            plain = torch.where(seen, plain, torch.zeros_like(plain)).amax(1, keepdim=True) * abs(scale)
            big = torch.where(seen, torch.nan_to_num(score), torch.zeros_like(score)).abs().amax(1, keepdim=True)
            off = (D + 4) * 2.0 ** -23 * plain + 4 * 2.0 ** -23 * (big + 40) + 2.0 ** -20
            err = ((2.0 ** -11 + 2 * off + (n + 64) * 2.0 ** -23) * mean
                   + n * 2.0 ** -25 * p.amax(1, keepdim=True) * (c - z).abs().amax() / safe)
            none = ~any_key
            out[row, h * group:(h + 1) * group] = torch.where(none, torch.zeros_like(got), got).view(len(row), group, D)
            tol[row, h * group:(h + 1) * group] = torch.where(none, torch.zeros_like(err), torch.nan_to_num(err)).view(len(row), group, D)
            logs = torch.where(any_key, top + torch.log(safe), torch.full_like(top, -math.inf))
            lse[row, h * group:(h + 1) * group] = logs.view(len(row), group)
    return out, lse, tol


def linear4(x, code, s, z, group):
    """x [tokens][depth] with weights of codes [channels][depth] and steps and
    zero points [channels][groups]: (out, sum of |x| |w|), in 64 bits."""
    depth = x.shape[-1]
    wide = lambda t: t.repeat_interleave(group, -1)[..., :depth]                 # noqa: E731
    w = wide(s) * (code.double() - wide(z))
    return x.double() @ w.T, x.double().abs() @ w.abs().T
