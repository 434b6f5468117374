"""Inputs and plain references for rotations and 4-bit paged caches.

Tolerances of the attention over a 4-bit cache, as attend4 has them (u = 2^-24, D = head_dim, G = D / 32 blocks, n
visible tokens; v_tc = s code + m of a block).  `wide` is a call of more than 16 entries a sequence and KV head.
  kmag     up to 16 entries: |s code| + |m|, as codes and minima meet q in products of their own; wide: |k|, K being
           f16 values.  mag = max_t scale * sum_c |q_c| kmag_tc over visible t.
  logits   products of exact codes (wide: f16 values), summed in binary32 by the tensor cores (each addition off by at
           most 2 u of the sum's largest part), scaled and summed over the blocks, the minima against block sums of q
           whose two f16 halves keep 2^-22; two roundings of the base-2 exponent: (2 D + 4 G + 24) u mag; ex2 2 ulp.
  lost     what q loses.  Up to 16 entries it is an E5M2 and an E4M3 code, off by at most 2^-21 of its row's largest
           magnitude; attend4 allows 2^-17 (test_gpu_q4_queries.py holds the kernel to 2^-21).  Wide: f16 times a power of
           two that brings the largest to [2^14, 2^15), off by at most 2^-39 of it; and K rounded to f16, 2^-11 mag, or
           where it is below f16's normal numbers 2^-25 scale sum_c |q_c|.
  weights  off by a factor 1 +- e, e = 2 ((2 D + 4 G + 24) u mag + lost) + 8 u (weight and reference); sums of n terms
           another n 2 u.
  out      2 (e + (n + 16) 2 u) wabs, wabs = sum_t w_t |v_t| / sum_t w_t; V and the weights rounded to f16, 2^-11 each:
           1.01 2^-10 wabs; V below f16's normal numbers 2^-25; weights below them are off by 2^-25, where the largest is
           about 2^7: n 2^-32 max |v| (twice that where a rounded-up reference leaves the largest at 2^6, which no
           case comes near).
  lse      e + (n + 16) 2 u + 4 u |lse|.
"""
from __future__ import annotations

import math

import torch

import indexed_sparse_attention_gb300 as qsa
from paged_cases import BF16_HALF, Paged, U, dev, make_paged


def order4(D: int) -> torch.Tensor:
    """Where channel c's nibble lies in a row: index into the row's D nibbles, low nibble first."""
    c = torch.arange(D)
    g, n, j = c // 32, c % 32 // 4, c % 4
    return 4 * (n * (D // 32) + g) + j


def encode4(x: torch.Tensor):
    """Codes (uint8 [..., D / 2]) and (scale, minimum) pairs (float16 [..., D / 32, 2]) of f32 rows, as the
    header defines them."""
    D = x.shape[-1]
    b = x.float().reshape(*x.shape[:-1], D // 32, 32)
    odd = ~(b.abs() <= 65280.0).all(-1, keepdim=True)
    b0 = torch.where(odd, torch.zeros_like(b), b)
    lo, hi = b0.amin(-1, keepdim=True), b0.amax(-1, keepdim=True)
    m, s = lo.half(), ((hi - lo) / 15.0).half()
    s = torch.where(odd, torch.full_like(s, math.nan), s)
    sf = s.float()
    c = torch.where(sf > 0, torch.round((b0 - m.float()) / sf).clamp(0, 15), torch.zeros_like(b0)).to(torch.uint8)
    nib = torch.zeros(*x.shape[:-1], D, dtype=torch.uint8)
    nib[..., order4(D)] = c.reshape(*x.shape[:-1], D)
    nib = nib.reshape(*x.shape[:-1], D // 2, 2)
    return nib[..., 0] | (nib[..., 1] << 4), torch.cat((s, m), -1)


def split4(codes: torch.Tensor, pairs: torch.Tensor):
    """(code, scale, minimum) of every value, 64-bit [..., D]."""
    D = codes.shape[-1] * 2
    nib = torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], D)
    code = nib[..., order4(D)].double()
    s, m = (pairs[..., i].double().repeat_interleave(32, -1) for i in range(2))
    return code, s, m


class Paged4(Paged):
    """A 4-bit paged cache on the CPU: k, v are codes, scale the records."""

    def seq_parts(self, i: int):
        """(code, scale, minimum) of K and of V of sequence i's tokens, each [Hkv, L, D]."""
        n = self.lens[i]
        ids = self.table[i, :-(-n // self.page)].long()
        rec = self.scale[ids].reshape(*self.scale[ids].shape[:3], 2, -1, 2)
        out = []
        for x, w in ((self.k, 0), (self.v, 1)):
            parts = split4(x[ids], rec[..., w, :, :])
            out.append([y.transpose(0, 1).reshape(y.shape[1], -1, y.shape[3])[:, :n] for y in parts])
        return out

    def seq_kv(self, i: int):
        return [c * s + m for c, s, m in self.seq_parts(i)]

    def device(self, out_dtype=torch.float32):
        def put(x):
            x = x.to(dev())
            return x if self.order == "head" else x.transpose(1, 2).contiguous().transpose(1, 2)
        cache = qsa.PagedCache(put(self.k), put(self.v), put(self.scale), kv_dtype=qsa.Q4)
        batch = qsa.PagedBatch(self.table.to(dev()), torch.tensor(self.lens, dtype=torch.int32, device=dev()),
                               self.row_start.to(dev()), n_rows=self.q.shape[0], max_rows=max(self.rows, default=0))
        return cache, batch, self.q.to(dev())


def make_paged4(lens, rows, *, poison=False, lean=1.0, **kw) -> Paged4:
    """make_paged in 4 bits; K's channels lie apart from zero by a constant each.  With poison, the codes of
    slots that belong to no token are set, and their scales and minima NaN and infinite."""
    x = make_paged(lens, rows, dtype="bf16", **kw)
    g = torch.Generator().manual_seed(kw.get("seed", 0) + 1)
    D = x.k.shape[-1]
    k = x.k.float() + torch.randn(x.k.shape[1], 1, D, generator=g) * lean
    (kc, kp), (vc, vp) = encode4(k), encode4(x.v.float())
    scale = torch.cat((kp.flatten(-2), vp.flatten(-2)), -1)
    y = Paged4(kc, vc, scale, x.table, x.lens, x.rows, x.row_start, x.q, x.page, x.order)
    if poison:
        used = torch.zeros(kc.shape[0], x.page, dtype=torch.bool)
        for i, n in enumerate(lens):
            for t in range(n):
                used[x.table[i, t // x.page], t % x.page] = True
        off = ~used[:, None].expand(-1, kc.shape[1], -1)
        y.k[off], y.v[off] = 0xFF, 0xFF
        y.scale[off] = torch.tensor([math.nan, math.inf] * (D // 16), dtype=torch.float16)
    return y


def attend4(x: Paged4, window=0, sinks=0, scale=None, most=None):
    """(out, lse, out tolerance without output rounding, lse tolerance) in 64 bits; most: the call's max_rows, where
    it is not x's."""
    R, Hq, D = x.q.shape
    Hkv = x.k.shape[1]
    G = Hq // Hkv
    scale = scale or D ** -0.5
    wide = (max(x.rows, default=0) if most is None else most) * G > 16
    out = torch.zeros(R, Hq, D, dtype=torch.float64)
    lse = torch.full((R, Hq), -math.inf, dtype=torch.float64)
    otol = torch.zeros(R, Hq, D, dtype=torch.float64)
    ltol = torch.zeros(R, Hq, dtype=torch.float64)
    for i, (n, r) in enumerate(zip(x.lens, x.rows)):
        if r == 0 or n == 0:
            continue
        r0 = int(x.row_start[i])
        K, V = x.seq_parts(i)
        pos = torch.arange(n - r, n)[:, None]
        t = torch.arange(n)[None]
        see = t <= pos
        if window:
            see &= (t > pos - window) | (t < sinks)
        live = see.any(0)
        cnt = see.sum(1)[:, None].double()
        for h in range(Hkv):
            kc, ks, km, vc, vs, vm = (torch.where(live[:, None], y[h], 0.0) for y in (*K, *V))
            kh, vh = kc * ks + km, vc * vs + vm
            kmag = kh.abs() if wide else (kc * ks).abs() + km.abs()
            qh = x.q[r0:r0 + r, h * G:(h + 1) * G].double()
            hide = ~see[:, None]
            z = (torch.einsum("rgd,td->rgt", qh, kh) * scale).masked_fill(hide, -math.inf)
            mag = (torch.einsum("rgd,td->rgt", qh.abs(), kmag) * scale).masked_fill(hide, 0.0).amax(-1)
            # Up to 16 entries q is two E4M3 codes, off by at most 2^-17 of the row's largest; more take it as f16.
            lost = (1.01 * 2.0 ** (-39 if wide else -17) * scale * qh.abs().amax(-1, keepdim=True) * kmag.sum(-1)).masked_fill(hide, 0.0).amax(-1)
            if wide:
                lost = lost + 2.0 ** -11 * 1.01 * mag + 2.0 ** -25 * scale * qh.abs().sum(-1)
            e = 2 * ((2 * D + 4 * (D // 32) + 24) * U * mag + lost) + 8 * U
            L = torch.logsumexp(z, -1)
            w = torch.exp(z - L[..., None]).nan_to_num(0.0)
            sl = slice(h * G, (h + 1) * G)
            out[r0:r0 + r, sl] = torch.einsum("rgt,td->rgd", w, vh)
            lse[r0:r0 + r, sl] = L
            wabs = torch.einsum("rgt,td->rgd", w, vh.abs())
            rounded = 1.01 * 2.0 ** -10 * wabs + 2.0 ** -25 + cnt[..., None] * 2.0 ** -32 * vh.abs().max()
            otol[r0:r0 + r, sl] = (2 * (e + (cnt + 16) * 2 * U))[..., None] * wabs + rounded
            ltol[r0:r0 + r, sl] = e + (cnt + 16) * 2 * U + 4 * U * L.abs().nan_to_num(0.0, posinf=0.0)
    return out, lse, otol, ltol


def turned(x: torch.Tensor, pos, rot: int, pairs: bool, w, magnitude=1.0) -> torch.Tensor:
    """x [rows, heads, D] rotated in 64 bits."""
    y = x.double().clone()
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if pairs else (i, i + rot // 2)
    th = torch.as_tensor(pos, dtype=torch.float64)[:, None, None] * torch.tensor(w, dtype=torch.float64)
    c, s = magnitude * th.cos(), magnitude * th.sin()
    xa, xb = x[..., a].double(), x[..., b].double()
    y[..., a], y[..., b] = xa * c - xb * s, xa * s + xb * c
    return y


def assert_turned(got: torch.Tensor, x: torch.Tensor, pos, rot, pairs, w, magnitude=1.0, farthest=None):
    """got against the rotation in 64 bits.  cos and sin: the reduced angle (binary32 in [-1/8, 1/8] of a turn:
    2^-25 of it, times 2 pi / 8), sincospi (2 ulp) and the magnitude's product: 6 u; two products and a sum: 3 u of
    the pair's magnitudes.  The frequency, and its quotient by 2 pi, are binary64: 2^-52 of the angle of the farthest
    position (given where pos is reduced), doubled.  Then one rounding to the type."""
    want = turned(x, pos, rot, pairs, w, magnitude)
    y = x.double().abs()
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if pairs else (i, i + rot // 2)
    size = torch.zeros_like(y)
    size[..., a] = size[..., b] = (y[..., a] + y[..., b]) * abs(magnitude)
    far = (torch.as_tensor(pos, dtype=torch.float64).abs().max() if farthest is None else farthest) * max(abs(f) for f in w) * 2.0 ** -51
    tol = (10 * U + float(far)) * size
    tol = tol + want.abs() * (1.01 * torch.finfo(got.dtype).eps / 2) * (size > 0)
    err = (got.double().cpu() - want).abs()
    assert (err <= tol).all(), f"worst {float((err / tol.clamp(min=1e-300)).max()):.2f} of its tolerance"


__all__ = ["BF16_HALF", "Paged4", "assert_turned", "attend4", "encode4", "make_paged4", "order4", "split4", "turned"]
