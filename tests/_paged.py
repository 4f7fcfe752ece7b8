"""Inputs and 64-bit definitions of the paged-cache operators for their tests
(torch, fp64, written from the formulas in include/dit_paged.h)."""
import math

import torch

BF16_HALF = 2.0 ** -8  # half a step of bf16, relative


def ints(values, device="cuda"):
    return torch.tensor(values, dtype=torch.int32, device=device)


def cumulative(values):
    out = [0]
    for v in values:
        out.append(out[-1] + v)
    return out


class Batch:
    """A packed batch of chunks over a paged cache.  Every buffer starts as
    NaN; rows, slots and table entries that an operator may read are filled."""

    def __init__(self, chunks, pasts, hq, hk, d, page=16, pad=8, seed=0, hnd=False, slack=2, scale=1.0, kv_lens=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.chunks, self.pasts, self.hq, self.hk, self.d, self.page = chunks, pasts, hq, hk, d, page
        slots = [-(-n // pad) * pad for n in chunks]
        self.first = cumulative(slots)
        self.rows = self.first[-1] + slack
        self.cs, self.cp = ints(cumulative(chunks)), ints(self.first)
        # the tokens each sequence may look at; slots behind them stay NaN
        self.kv = [a + b for a, b in zip(chunks, pasts)] if kv_lens is None else kv_lens
        width = 3 * hq * d + 16  # q is a column slice of a wider buffer
        self.buf = torch.full((self.rows, width), math.nan, dtype=torch.bfloat16, device="cuda")
        self.q = self.buf[:, 8:8 + hq * d]
        self.k = torch.full((self.rows, hk * d), math.nan, dtype=torch.bfloat16, device="cuda")
        self.v = torch.full_like(self.k, math.nan)
        for b, n in enumerate(chunks):
            r = slice(self.first[b], self.first[b] + n)
            for t in (self.q, self.k, self.v):
                t[r] = torch.randn(n, t.size(1), device="cuda", generator=g).mul_(scale).bfloat16()
        need = [-(-max(a, c + e) // page) for a, c, e in zip(self.kv, chunks, pasts)]
        order = torch.randperm(sum(need) + 3, generator=torch.Generator().manual_seed(seed)).tolist()
        self.max_pages = max(need + [1]) + 1
        table, at = [], 0
        for n in need:
            table.append(order[at:at + n] + [-1] * (self.max_pages - n))
            at += n
        self.table_host = table
        self.table = ints(table).view(len(chunks), self.max_pages)
        shape = (len(order), hk, page, d) if hnd else (len(order), page, hk, d)
        self.k_cache = torch.full(shape, math.nan, dtype=torch.bfloat16, device="cuda")
        self.v_cache = torch.full(shape, math.nan, dtype=torch.bfloat16, device="cuda")
        if hnd:
            self.k_cache, self.v_cache = self.k_cache.transpose(1, 2), self.v_cache.transpose(1, 2)
        self.gen = g

    def place(self, b, first, last):
        pos = torch.arange(first, last, device="cuda")
        return self.table[b].long()[pos // self.page], pos % self.page

    def fill(self, scale=1.0):
        """Keys and values of every token below kv."""
        for b, n in enumerate(self.kv):
            where = self.place(b, 0, n)
            for c in (self.k_cache, self.v_cache):
                c[where] = torch.randn(n, self.hk, self.d, device="cuda", generator=self.gen).mul_(scale).bfloat16()
        return self

    def kv_lens(self):
        return ints(self.kv)

    def sizes(self):
        return dict(num_q_heads=self.hq, num_kv_heads=self.hk, head_dim=self.d)

    def valid(self):
        mask = torch.zeros(self.rows, dtype=torch.bool, device="cuda")
        for b, n in enumerate(self.chunks):
            mask[self.first[b]:self.first[b] + n] = True
        return mask


def reference_attention(x: Batch, causal, window, scale=None, dead_pages=()):
    """(out, lse, weight): fp64 [rows, hq, d], [rows, hq] and sum_j p_j |v_j|
    (the size that the rounding of the probabilities is relative to), and the
    largest sum |q_d k_d| scale per row (that of the scores).  Padding rows 0."""
    scale = 1.0 / math.sqrt(x.d) if scale is None else scale
    out = torch.zeros(x.rows, x.hq, x.d, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(out)
    lse = torch.zeros(x.rows, x.hq, dtype=torch.float64, device="cuda")
    mass = torch.zeros_like(lse)
    group = x.hq // x.hk
    for b, n in enumerate(x.chunks):
        total = x.kv[b]
        if n == 0:
            continue
        page, slot = x.place(b, 0, total)
        keys, values = x.k_cache[page, slot].double(), x.v_cache[page, slot].double()
        for dead in dead_pages:
            keys[page == dead] = 0
            values[page == dead] = 0
        j = torch.arange(total, device="cuda")[None]
        p = (total - n + torch.arange(n, device="cuda"))[:, None]
        sees = (j <= p) if causal else torch.ones(n, total, dtype=torch.bool, device="cuda")
        if window:
            sees = sees & (j > p - window)
        r = slice(x.first[b], x.first[b] + n)
        q = x.q[r].double().view(n, x.hq, x.d)
        for h in range(x.hq):
            kh, vh = keys[:, h // group], values[:, h // group]
            s = (q[:, h] @ kh.T * scale).masked_fill(~sees, -math.inf)
            top = s.amax(-1, keepdim=True) if total else torch.full((n, 1), -math.inf, dtype=torch.float64, device="cuda")
            e = torch.exp(s - torch.where(torch.isfinite(top), top, 0.0))
            total_e = e.sum(-1, keepdim=True)
            pr = torch.where(total_e > 0, e / total_e, 0.0)
            out[r, h], size[r, h] = pr @ vh, pr @ vh.abs()
            lse[r, h] = (top + torch.log(total_e))[:, 0]
            if total:
                mass[r, h] = ((q[:, h].abs() @ kh.abs().T) * scale).masked_fill(~sees, 0.0).amax(-1)
    return out, lse, size, mass


def check_attention(x: Batch, out, lse, causal, window, scale=None, dead_pages=()):
    """Every valid row within the roundings' bounds of the definition.

    o: each probability is rounded to bf16 (2^-8 of it), which moves o by at
    most 2^-8 sum p|v|; fp32 scores of D products are off by at most
    D 2^-24 sum|qk| scale < 2^-16 (4 + mass) for the sizes here, exponentials
    and sums add less than 2^-16; o is rounded once more (2^-8 of itself).
    lse: no rounding to bf16, only the fp32 ones."""
    ref, ref_lse, size, mass = reference_attention(x, causal, window, scale, dead_pages)
    ok = x.valid()
    o = out.double().view(x.rows, x.hq, x.d)[ok]
    assert bool(torch.isfinite(o).all()), "non-finite output"
    soft = 2.0 ** -16 * (4 + mass[ok][..., None])
    tol = BF16_HALF * ref[ok].abs() * (1 + BF16_HALF) + (BF16_HALF + soft) * (1 + BF16_HALF) * size[ok]
    worst = ((o - ref[ok]).abs() - tol).max() if o.numel() else torch.zeros(())
    assert float(worst) <= 0, f"output off by {float((o - ref[ok]).abs().max())}, past its bound by {float(worst)}"
    if lse is not None:
        a, r = lse.double()[ok], ref_lse[ok]
        none = torch.isinf(r)
        assert bool((a[none] == r[none]).all()), "lse of a row that sees nothing"
        bound = 2.0 ** -18 * (4 + mass[ok] + torch.where(none, 0.0, r).abs())
        err = torch.where(none, 0.0, (a - torch.where(none, 0.0, r)).abs())
        err[none] = 0
        assert bool((err <= bound).all()), f"lse off by {float(err.max())}"


def reference_rotation(x, chunks, first, heads, d, rotary, mode, freqs, gain, starts, weight=None, eps=1e-6,
                       grids=None, grid_freqs=None, sections=None):
    """fp64 [rows, heads, d] of the valid rows (others 0), and the size of the
    terms each element is made of."""
    y = torch.zeros(x.size(0), heads, d, dtype=torch.float64, device=x.device)
    size = torch.zeros_like(y)
    half = rotary // 2
    lo = torch.arange(half, device=x.device) if mode == "half" else 2 * torch.arange(half, device=x.device)
    hi = lo + (half if mode == "half" else 1)
    for b, n in enumerate(chunks):
        if n == 0:
            continue
        rows = x[first[b]:first[b] + n].double().view(n, heads, d)
        if weight is not None:
            rows = rows * torch.rsqrt(rows.pow(2).mean(-1, keepdim=True) + eps) * weight.double()
        o, sz = rows.clone(), rows.abs()
        if mode != "none":
            for i in range(n):
                p = max(starts[b], 0) + i
                ang = p * freqs.double()
                if grids is not None:
                    t, h, w = grids[b]
                    if p < t * h * w:
                        at = [p // (h * w)] * (sections[0] // 2) + [p // w % h] * (sections[1] // 2) + \
                            [p % w] * (sections[2] // 2)
                        ang = torch.tensor(at, dtype=torch.float64, device=x.device) * grid_freqs
                    else:
                        ang = (p - t * h * w) * freqs.double()
                c, s = torch.cos(ang) * gain, torch.sin(ang) * gain
                a, z = rows[i][:, lo], rows[i][:, hi]
                o[i][:, lo], o[i][:, hi] = a * c - z * s, a * s + z * c
                both = gain * (a.abs() + z.abs())
                sz[i][:, lo], sz[i][:, hi] = both, both
        y[first[b]:first[b] + n], size[first[b]:first[b] + n] = o, sz
    return y, size


def check_rotation(got, ref, size, what=""):
    """One rounding to bf16 (2^-8 of the value) behind fp32 arithmetic: the
    hardware sine and cosine are within 2^-21 and the reduced angle within
    2^-22, the norm's sum, root and products within 2^-20 of the value, so a
    term is off by less than 2^-18 of its size."""
    soft = 2.0 ** -18 * size
    tol = BF16_HALF * (ref.abs() + soft) + soft
    err = (got.double().view_as(ref) - ref).abs()
    assert bool(torch.isfinite(err).all()), f"{what}: non-finite"
    worst = float((err - tol).max()) if err.numel() else 0.0
    assert worst <= 0, f"{what}: off by {float(err.max())}, past its bound by {worst}"
