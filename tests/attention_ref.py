"""Plain 64-bit forms of the attention operators for the tests, and the
tolerances of the library's results, derived from its arithmetic.

Notation: u is half a step of the element type (finfo.eps / 2), e = 2^-24 half a
step of fp32. The library computes scores, statistics and sums in fp32 from
the stored elements:
  * a score's d products and sums, the scale and the bias are off by at most
    e (d + 4) (scale sum |q||k| + |bias|), which moves a weight by that
    relative amount; the statistics are sums of n weights, off by e (n + 64)
    relative (n additions at most, exp2 and log2 within a few e);
  * weights (and dS) are rounded to the element type before their product:
    relative u, or for fp16 below its normal range 2^-25 absolute, against a sum
    of weights of at least 1;
  * a result is rounded once: relative u.
"""
import numpy as np
import torch

E = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def _live(B, Hkv, Lk, key_bias, key_lengths):
    """[B, Hkv, Lk] bias in 64 bits, -inf where masked."""
    add = torch.zeros(B, Hkv, Lk, dtype=torch.float64)
    if key_bias is not None:
        kb = key_bias.detach().cpu().double()
        add = add + (kb if kb.dim() == 3 else kb[:, None, :])
        add[add <= -1e30] = -float("inf")
    if key_lengths is not None:
        n = key_lengths.cpu().long().clamp(0, Lk)
        add[(torch.arange(Lk)[None, :] >= n[:, None])[:, None, :].expand(B, Hkv, Lk)] = -float("inf")
    return add


def _rows(B, Lq, query_lengths):
    n = torch.full((B,), Lq) if query_lengths is None else query_lengths.cpu().long().clamp(0, Lq)
    return torch.arange(Lq)[None, :] < n[:, None]


class Ref:
    """All results of one call in 64 bits on the CPU, with tolerances."""

    def __init__(self, q, k, v=None, scale=None, key_bias=None, query_lengths=None, key_lengths=None, lse=None):
        self.u = half_step(q.dtype)
        self.f16 = q.dtype == torch.float16
        B, Lq, Hq, d = q.shape
        Lk, Hkv = k.shape[1], k.shape[2]
        G = Hq // Hkv
        self.scale = d ** -0.5 if scale is None else scale
        self.rows = _rows(B, Lq, query_lengths)  # [B, Lq]
        add = _live(B, Hkv, Lk, key_bias, key_lengths).repeat_interleave(G, 1)  # [B, Hq, Lk]
        self.dead = add == -float("inf")
        c = lambda t: t.detach().cpu().double()  # noqa: E731
        self.Q = c(q).permute(0, 2, 1, 3).masked_fill(~self.rows[:, None, :, None], 0.0)  # [B, Hq, Lq, d]
        dead_kv = self.dead[:, ::G]  # [B, Hkv, Lk]
        clean = lambda t: c(t).permute(0, 2, 1, 3).masked_fill(dead_kv[..., None], 0.0).repeat_interleave(G, 1)  # noqa: E731
        self.K = clean(k)
        self.G = G
        self.S = self.Q @ self.K.transpose(2, 3) * self.scale + add[:, :, None, :]
        if Lk:
            finite = add.masked_fill(self.dead, 0.0).abs()
            # relative error of a weight from its score, per row
            mag = self.Q.abs() @ self.K.abs().transpose(2, 3) * self.scale + finite[:, :, None, :]
            self.dw = E * ((d + 4) * mag.amax(3) + 16)  # [B, Hq, Lq]
            m = self.S.amax(3)
        else:
            self.dw = torch.zeros(B, Hq, Lq, dtype=torch.float64)
            m = torch.full((B, Hq, Lq), -float("inf"), dtype=torch.float64)
        m = torch.where(m == -float("inf"), torch.zeros_like(m), m)
        P = torch.exp(self.S - m[..., None])
        total = P.sum(3)
        empty = (total == 0) | ~self.rows[:, None, :]
        self.lse = torch.where(empty, torch.full_like(total, -float("inf")), m + torch.log(total))
        if lse is not None:  # the weights as the caller's lse makes them
            self.lse = c(lse)
            empty = self.lse == -float("inf")
        L = torch.where(empty, torch.full_like(self.lse, float("inf")), self.lse)
        self.P = torch.exp(self.S - L[..., None])
        self.empty = empty
        self.sum_err = E * (Lk + 64)
        self.lse_tol = self.dw + self.sum_err + 4 * E * torch.where(empty, torch.zeros_like(total), self.lse.abs()) + 4 * E
        if v is not None:
            self.V = clean(v)
            out = self.P @ self.V
            W = self.P @ self.V.abs()
            self.out = out.permute(0, 2, 1, 3)
            tiny = 2.0 ** -25 * self.V.abs().sum(2, keepdim=True) if self.f16 else 0.0
            self.out_tol = (self.u * (out.abs() + 1.01 * W) + 2 * (self.dw + self.sum_err)[..., None] * W + tiny
                            + (2.0 ** -24 if self.f16 else 0.0)).permute(0, 2, 1, 3)

    def _kv(self, x):
        """[B, Hq, Lk, d] -> sum over the group -> [B, Lk, Hkv, d]"""
        B, Hq, Lk, d = x.shape
        return x.reshape(B, Hq // self.G, self.G, Lk, d).sum(2).permute(0, 2, 1, 3)

    def mass(self, mass_in=None, row_weight=None):
        """(value, tolerance) of the gathered weight [B, Hkv, Lk]."""
        B, Hq, Lq, Lk = self.P.shape
        w = torch.ones(B, Lq, dtype=torch.float64) if row_weight is None else row_weight.cpu().double()
        w = torch.where(self.rows, w, torch.zeros_like(w))
        x = self.P * w[:, None, :, None]
        rel = (self.dw + E * (Lq * self.G + 64) + 8 * E * (1 + torch.where(self.empty, torch.zeros_like(self.lse), self.lse.abs()))
               + self.sum_err)[..., None]
        err = (x.abs() * rel).reshape(B, Hq // self.G, self.G, Lq, Lk).sum((2, 3))
        x = x.reshape(B, Hq // self.G, self.G, Lq, Lk).sum((2, 3))
        base = 0.0 if mass_in is None else mass_in.cpu().double()
        return base + x, err + 2 * E * (abs(base) + x.abs()) + 1e-30

    def grads(self, dout, out):
        """((dq, tol), (dk, tol), (dv, tol)) with D from the given out."""
        c = lambda t: t.detach().cpu().double().permute(0, 2, 1, 3).masked_fill(~self.rows[:, None, :, None], 0.0)  # noqa: E731
        dO, O = c(dout), c(out)
        P, u, sc = self.P, self.u, self.scale
        n = P.shape[3] + P.shape[2] * self.G + 64
        D = (dO * O).sum(3, keepdim=True)
        dP = dO @ self.V.transpose(2, 3)
        dS = P * (dP - D)
        # dS: its factors' fp32 errors, then its rounding
        width = self.V.shape[3] + 8
        mag = dO.abs() @ self.V.abs().transpose(2, 3) + (dO.abs() * O.abs()).sum(3, keepdim=True)
        rel = (self.dw + 8 * E * (1 + torch.where(self.empty, torch.zeros_like(self.lse), self.lse.abs())))[..., None]
        tiny = 2.0 ** -25 if self.f16 else 0.0
        live = (P > 0) | (self.S > -float("inf"))
        eS = rel * dS.abs() + E * width * P * mag + u * 1.01 * dS.abs() + tiny * live
        eP = rel * P + u * 1.01 * P + tiny * live
        res = []
        floor = 2.0 ** -24 if self.f16 else 1e-38
        for val, err, absval in (
                (dS @ self.K * sc, eS @ self.K.abs() * sc, dS.abs() @ self.K.abs() * sc),
                (dS.transpose(2, 3) @ self.Q * sc, eS.transpose(2, 3) @ self.Q.abs() * sc, dS.abs().transpose(2, 3) @ self.Q.abs() * sc),
                (P.transpose(2, 3) @ dO, eP.transpose(2, 3) @ dO.abs(), P.transpose(2, 3) @ dO.abs())):
            tol = err + E * n * absval
            if not res:
                val, tol = val.permute(0, 2, 1, 3), tol.permute(0, 2, 1, 3)
            else:
                val, tol = self._kv(val), self._kv(tol)
            res.append((val, tol + u * val.abs() + floor))
        return res


def assert_close(got, want, tol, what):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    same = got == want  # infinities included
    err = torch.where(same, torch.zeros_like(got), (got - want).abs())
    bad = ~(err <= tol)
    if bad.any():
        i = tuple(int(x) for x in torch.nonzero(bad)[0])
        t = tol if not torch.is_tensor(tol) else tol.expand(err.shape)[i]
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; at {i}: {float(got[i])!r} for "
                             f"{float(want[i])!r}, tolerance {float(t):.3e}")


def evict_ref(k, v, mass, keep, key_lengths=None, first=0, recent=0):
    """(kept indices per [batch][head] as numpy arrays)."""
    B, n, H, _ = k.shape
    w = mass.cpu().numpy().astype(np.float64)
    out = []
    for b in range(B):
        ln = n if key_lengths is None else min(max(int(key_lengths[b]), 0), n)
        row = []
        for h in range(H):
            if ln <= keep:
                row.append(np.arange(ln))
                continue
            lo, hi = first, ln - recent
            mid = w[b, h, lo:hi]
            mid = np.where(np.isnan(mid), -np.inf, mid)
            nan = np.isnan(w[b, h, lo:hi])
            order = np.lexsort((np.arange(lo, hi), nan, -mid))  # heaviest, NaN behind -inf, lowest index
            sel = np.sort(lo + order[: keep - first - recent])
            row.append(np.concatenate([np.arange(lo), sel, np.arange(hi, ln)]).astype(np.int64))
        out.append(row)
    return out
