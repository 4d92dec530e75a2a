"""Plain 64-bit forms of the rotary positions, the head norm, appending to a
paged cache and attention over it, for the tests, and the tolerances of the
library's results, derived from its arithmetic (all on the CPU).

Notation as in attention_ref: u half a step of the element type, E = 2^-24 half
a step of fp32.

Rotation. The angle a = p f is formed in 64 bits by both sides, off by at most
2^-51 |a| together; the library's reduced angle is rounded to fp32 (at most pi / 4
in size: 0.8 E), its Taylor sums have at most six terms with rounded coefficients
and six roundings, each of a partial sum of at most 1.6: cosine and sine are off by
less than 20 E + 2^-51 |a|. A product pair adds 3 E relative to |a cos| + |b sin|.
Norm: a sum of d squares (d additions at most, positive: relative d E), times 1 / d
and plus eps (4 E), its inverse root (half of that, plus 4 E), two products (2 E):
relative (d / 2 + 10) E."""
import torch

from attention_ref import E, half_step


def cpu(t):
    return None if t is None else t.detach().cpu().double()


def tiny(dtype):
    """Half the smallest step of a result: below the normal range a rounding is absolute."""
    return {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -127}[dtype]


def pair_index(r, interleaved):
    i = torch.arange(r // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)


def turn(x, err, a, gain, interleaved, inverse=False):
    """x [B, L, H, d] turned by angles a [B, L, r / 2], with its error."""
    r = 2 * a.shape[-1]
    if r == 0:
        return x, err
    y, ey = x.clone(), err.clone()
    i, j = pair_index(r, interleaved)
    c, s = torch.cos(a)[:, :, None] * gain, torch.sin(a)[:, :, None] * gain * (-1 if inverse else 1)
    p, q = x[..., i], x[..., j]
    y[..., i], y[..., j] = p * c - q * s, p * s + q * c
    off = abs(gain) * (24 * E + 2.0 ** -51 * a.abs())[:, :, None]
    e = off * (p.abs() + q.abs()) + abs(gain) * (err[..., i] + err[..., j])
    ey[..., i], ey[..., j] = e, e
    return y, ey


class Rotation:
    """What rotate_heads makes of x [B, L, H, d], and its gradient."""

    def __init__(self, dtype, positions, frequencies, interleaved, gain, norm_eps, weight, lengths, B, L, d):
        self.dtype, self.inter, self.gain, self.eps = dtype, bool(interleaved), float(gain), norm_eps
        self.u = half_step(dtype)
        self.w = torch.ones(d, dtype=torch.float64) if weight is None else cpu(weight)
        p = torch.arange(L).expand(B, L) if positions is None else positions.cpu().long().expand(B, L)
        f = torch.zeros(0, dtype=torch.float64) if frequencies is None else frequencies.cpu()
        self.a = p.double()[..., None] * f
        n = torch.full((B,), L) if lengths is None else lengths.cpu().long().clamp(0, L)
        self.live = (torch.arange(L)[None, :] < n[:, None])[:, :, None, None]
        self.rel = (d / 2 + 10) * E

    def _norm(self, x):
        if self.eps is None:
            return x, torch.zeros_like(x), None
        r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + self.eps)
        return x * r * self.w, (x * r * self.w).abs() * self.rel, r

    def forward(self, x):
        x = torch.where(self.live, cpu(x), torch.zeros((), dtype=torch.float64))
        n, err, _ = self._norm(x)
        y, err = turn(n, err, self.a, self.gain, self.inter)
        y = torch.where(self.live, y, torch.zeros_like(y))
        err = torch.where(self.live, err, torch.zeros_like(err))
        return y, err + self.u * y.abs() * 1.01 + tiny(self.dtype)

    def grad(self, dy, x=None):
        """((dx, tolerance), (dw, tolerance) or None)"""
        zero = torch.zeros((), dtype=torch.float64)
        dy = torch.where(self.live, cpu(dy), zero)
        g, eg = turn(dy, torch.zeros_like(dy), self.a, self.gain, self.inter, inverse=True)
        g, eg = torch.where(self.live, g, zero), torch.where(self.live, eg, zero)
        if self.eps is None:
            return (g, eg + self.u * g.abs() * 1.01 + tiny(self.dtype)), None
        x = torch.where(self.live, cpu(x), zero)
        d = x.shape[-1]
        r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + self.eps)
        xh, v = x * r, g * self.w
        m = (v * xh).mean(-1, keepdim=True)
        em = (eg * self.w.abs() * xh.abs()).mean(-1, keepdim=True) + ((d + 8) * E + 4 * self.rel) * (v * xh).abs().mean(-1, keepdim=True)
        dx = r * (v - xh * m)
        ex = r * (eg * self.w.abs() + xh.abs() * em + (2 * self.rel + 8 * E) * (v.abs() + (xh * m).abs()))
        dx, ex = torch.where(self.live, dx, zero), torch.where(self.live, ex, zero)
        terms = (g * xh).flatten(0, 2)
        dw = terms.sum(0)
        ew = (eg * xh.abs()).flatten(0, 2).sum(0) + (self.rel + (terms.shape[0] + 8) * E) * terms.abs().sum(0)
        return (dx, ex + self.u * dx.abs() * 1.01 + tiny(self.dtype)), (dw, ew + 2.0 ** -127)


def append_ref(k, v, k_cache, v_cache, page_table, cache_lengths, new_lengths=None, positions=None, frequencies=None,
               interleaved=False, gain=1.0, norm_eps=None, k_weight=None, q=None, q_weight=None):
    """(k_cache, tolerance, v_cache, lengths, q_out, tolerance) after appending, token by token."""
    B, L, H, d = k.shape
    pages, size = k_cache.shape[:2]
    table, cap = page_table.cpu().tolist(), page_table.shape[1] * size
    before = [min(max(int(n), 0), cap) for n in cache_lengths.cpu()]
    new = [L] * B if new_lengths is None else [min(max(int(n), 0), L) for n in new_lengths.cpu()]
    pos = torch.tensor([[before[b] + i for i in range(L)] for b in range(B)]).reshape(B, L) if positions is None else positions
    live = torch.tensor(new, dtype=torch.int32)
    mk = lambda w: Rotation(k.dtype, pos, frequencies, interleaved, gain, norm_eps, w, live, B, L, d)  # noqa: E731
    kn, kt = mk(k_weight).forward(k)
    kc, vc = cpu(k_cache), cpu(v_cache)
    tol = torch.zeros_like(kc)
    exact_copy = frequencies is None and norm_eps is None
    for b in range(B):
        for i in range(new[b]):
            j = before[b] + i
            if j >= cap or not 0 <= table[b][j // size] < pages:
                continue
            at = table[b][j // size], j % size
            kc[at], vc[at] = kn[b, i], cpu(v[b, i])
            tol[at] = 0.0 if exact_copy else kt[b, i]
    total = torch.tensor([min(x + y, cap) for x, y in zip(before, new)], dtype=torch.int32)
    qn, qt = (None, None) if q is None else mk(q_weight).forward(q)
    return kc, tol, vc, total, qn, qt


def table_of(lens, size, pages, gen, extra=0):
    """A page table [B, C] over `pages` pages in a drawn order, no page twice; behind a
    sequence's pages it holds numbers that are no pages."""
    need = [(n + size - 1) // size for n in lens]
    assert sum(need) <= pages
    order = torch.randperm(pages, generator=gen).tolist()
    width = max(need + [0]) + extra
    t = torch.full((len(lens), width), -7, dtype=torch.int32)
    t[:, width - width // 2:] = 2 ** 31 - 1
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    return t


class PagedRef:
    """paged_attention in 64 bits, with tolerances as attention_ref.Ref derives them (two_parts: the
    weights are held in two parts of the element type, which leaves 2^-16 (bf16) or 2^-22 of them)."""

    def __init__(self, q, k_cache, v_cache, page_table, key_lengths, scale=None, query_lengths=None, first=0, recent=None):
        dtype = q.dtype
        u, f16 = half_step(dtype), dtype == torch.float16
        B, m, Hq, d = q.shape
        pages, size, H, dv = v_cache.shape
        G = Hq // H
        scale = d ** -0.5 if scale is None else scale
        cap = page_table.shape[1] * size
        first, recent = min(first, cap), None if recent is None else min(recent, cap + m)
        self.out = torch.zeros(B, m, Hq, dv, dtype=torch.float64)
        self.out_tol = torch.zeros(B, m, Hq, dv, dtype=torch.float64)
        self.lse = torch.full((B, Hq, m), -float("inf"), dtype=torch.float64)
        self.lse_tol = torch.zeros(B, Hq, m, dtype=torch.float64)
        few = m * G <= 32 and dtype != torch.float32
        weight_step = {torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -22, torch.float32: 0.0}[dtype] if few else u
        for b in range(B):
            n = min(max(int(key_lengths[b]), 0), cap)
            rows = m if query_lengths is None else min(max(int(query_lengths[b]), 0), m)
            ids = page_table[b].cpu().long()
            ok = (ids >= 0) & (ids < pages)
            ids = torch.where(ok, ids, torch.zeros_like(ids))
            if pages == 0 or n == 0:
                continue
            need = (n + size - 1) // size
            take = lambda c: c[ids[:need].to(c.device)].flatten(0, 1)[:n].cpu().double()  # noqa: E731
            K, V = take(k_cache), take(v_cache)  # [n, H, .]
            live = ok[:need].repeat_interleave(size)[:n]
            j = torch.arange(n)
            for i in range(rows):
                p = n - rows + i
                see = live & (j <= p)
                if recent is not None:
                    see = see & ((j > p - recent) | (j < first))
                at = torch.nonzero(see)[:, 0]
                if not len(at):
                    continue
                for h in range(Hq):
                    x = q[b, i, h].cpu().double()
                    k, v = K[at, h // G], V[at, h // G]
                    s = (k @ x) * scale
                    z = torch.logsumexp(s, 0)
                    w = torch.exp(s - z)
                    mag = (k.abs() @ x.abs()) * scale
                    dw = E * ((d + 4) * mag.max() + 16)
                    rel = dw + E * (len(at) + 64)
                    y = w @ v
                    self.lse[b, h, i] = z
                    self.lse_tol[b, h, i] = rel + 4 * E * z.abs() + 4 * E
                    self.out[b, i, h] = y
                    W = w @ v.abs()
                    small = 2.0 ** -25 * v.abs().sum(0) if f16 else 0.0
                    self.out_tol[b, i, h] = u * y.abs() * 1.01 + (weight_step * 1.01 + 2 * rel) * W + small + tiny(dtype) * 4
