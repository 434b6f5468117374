"""Inputs and plain references for the paged-cache tests: attention over a paged
cache in 64 bits, rows written into pages, and the keeping of pages.

Tolerances of the attention, from its arithmetic (u = 2^-24, D = head_dim, n
visible tokens; all sums in binary32):
  logits   a dot product of D terms and its scaling: |dz| <= (D + 4) u zmag,
           zmag = max_t scale * sum_d |q_d k_td|; two roundings of the base-2
           exponent: 2 u (|z| + |m|) <= 4 u zmag; ex2 is within 2 ulp: 4 u.
           fp8 caches: Q goes into the product as the sum of two E4M3 codes, of the
           value times a power of two that brings the row's maximum qmax to
           [2^7, 2^8), and of what the first leaves.  bf16's 8 significant bits are
           two codes' 4, and E4M3's smallest step is 2^-9, so values from 2^-2 on
           are exact; below, half a step is lost: dq <= min(2^-10, |q|) after the
           scaling, 2^-17 qmax where |q| < 2^-9 qmax.  |dz| grows by
           zlost = max_t scale * sum_d dq_d |k_td|.
  weights  so each weight is off by a factor 1 +- e with e = (2 D + 24) u zmag +
           8 u + 2 zlost (weight and maximum), and the sums of n terms add n u.
  out      |d out| <= 2 (e + (n + 16) u) wabs, wabs = sum_t w_t |v_t| / sum_t w_t;
           for bf16 and fp8 caches each weight is rounded to bf16 before the
           product with V: another 2^-8 wabs; a bf16 output: 2^-8 |out|.
  lse      |d lse| <= e + (n + 16) u + 4 u |lse|.
"""
from __future__ import annotations

import dataclasses
import math

import torch

import indexed_sparse_attention_gb300 as qsa

U = 2.0 ** -24
BF16_HALF = 2.0 ** -8


def dev():
    return torch.device("cuda", 0)


def encode_fp8(x: torch.Tensor):
    """E4M3 codes (uint8) and f16 scale of each row of f32 values."""
    scale = (x.abs().amax(-1, keepdim=True) / 448.0).half()
    s = scale.float()
    y = torch.where(s > 0, x / s, torch.zeros_like(x)).clamp(-448.0, 448.0)
    return y.to(torch.float8_e4m3fn).view(torch.uint8), scale


@dataclasses.dataclass
class Paged:
    """A paged cache with its batch, on the CPU; values(k or v) as 64-bit rows."""
    k: torch.Tensor            # [n_pages, Hkv, P, D] stored type (uint8 for fp8)
    v: torch.Tensor
    scale: torch.Tensor | None
    table: torch.Tensor
    lens: list
    rows: list
    row_start: torch.Tensor
    q: torch.Tensor
    page: int
    order: str

    def seq_kv(self, i: int):
        """K and V of sequence i's tokens, [Hkv, L, D] in 64 bits."""
        n = self.lens[i]
        ids = self.table[i, :-(-n // self.page)].long()
        out = []
        for x, w in ((self.k, 0), (self.v, 1)):
            y = (x[ids].view(torch.float8_e4m3fn).float() if self.scale is not None else x[ids]).double()
            if self.scale is not None:
                y = y * self.scale[ids][..., w:w + 1].double()
            out.append(y.transpose(0, 1).reshape(y.shape[1], -1, y.shape[3])[:, :n])
        return out

    def device(self, out_dtype=torch.float32):
        """(cache, batch, q) on the GPU, pages in the case's memory order."""
        def put(x):
            x = x.to(dev())
            return x if self.order == "head" else x.transpose(1, 2).contiguous().transpose(1, 2)
        cache = qsa.PagedCache(put(self.k), put(self.v), None if self.scale is None else put(self.scale))
        batch = qsa.PagedBatch(self.table.to(dev()), torch.tensor(self.lens, dtype=torch.int32, device=dev()),
                               self.row_start.to(dev()), n_rows=self.q.shape[0], max_rows=max(self.rows, default=0))
        return cache, batch, self.q.to(dev())


def make_paged(lens, rows, *, dtype="bf16", D=128, Hkv=2, G=12, page=16, order="head", seed=0, poison=False,
               pad_rows=0, spare=3) -> Paged:
    """Sequences of `lens` tokens whose last `rows` tokens are query rows.  With
    poison, everything that belongs to no token (free pages, slots behind the
    last token) is NaN."""
    g = torch.Generator().manual_seed(seed)
    counts = [-(-n // page) for n in lens]
    n_pages = sum(counts) + spare
    perm = torch.randperm(n_pages, generator=g)
    table = torch.full((len(lens), max(max(counts), 1) + 1), -1, dtype=torch.int32)
    k = torch.randn(n_pages, Hkv, page, D, generator=g)
    v = torch.randn(n_pages, Hkv, page, D, generator=g)
    used = torch.zeros(n_pages, page, dtype=torch.bool)
    at = 0
    for i, (c, n) in enumerate(zip(counts, lens)):
        ids = perm[at:at + c]
        table[i, :c] = ids.int()
        at += c
        for j, p in enumerate(ids.tolist()):
            used[p, :min(page, n - j * page)] = True
    scale = None
    if dtype == "fp8":
        (k, ks), (v, vs) = encode_fp8(k), encode_fp8(v)
        scale = torch.cat((ks, vs), -1)
        if poison:
            k[~used[:, None].expand(-1, Hkv, -1)] = 0x7F   # the E4M3 NaN
            v[~used[:, None].expand(-1, Hkv, -1)] = 0x7F
            scale[~used[:, None].expand(-1, Hkv, -1)] = float("nan")
    else:
        t = torch.bfloat16 if dtype == "bf16" else torch.float32
        k, v = k.to(t), v.to(t)
        if poison:
            k[~used[:, None].expand(-1, Hkv, -1)] = float("nan")
            v[~used[:, None].expand(-1, Hkv, -1)] = float("inf")
    starts = [0]
    for r in rows:
        starts.append(starts[-1] + r)
    heat = torch.linspace(0.5, 3.0, Hkv * G)[None, :, None]
    q = torch.randn(starts[-1] + pad_rows, Hkv * G, D, generator=g) * heat
    q = q.to(torch.float32 if dtype == "f32" else torch.bfloat16)
    return Paged(k, v, scale, table, list(lens), list(rows), torch.tensor(starts, dtype=torch.int32), q, page, order)


def attend64(x: Paged, window=0, sinks=0, scale=None):
    """(out, lse, out tolerance without output rounding, lse tolerance) in 64 bits."""
    R, Hq, D = x.q.shape
    Hkv = x.k.shape[1]
    G = Hq // Hkv
    scale = scale or D ** -0.5
    out = torch.zeros(R, Hq, D, dtype=torch.float64)
    lse = torch.full((R, Hq), -math.inf, dtype=torch.float64)
    otol = torch.zeros(R, Hq, D, dtype=torch.float64)
    ltol = torch.zeros(R, Hq, dtype=torch.float64)
    rounded = 0.0 if x.q.dtype == torch.float32 else BF16_HALF
    for i, (n, r) in enumerate(zip(x.lens, x.rows)):
        if r == 0 or n == 0:
            continue
        r0 = int(x.row_start[i])
        K, V = x.seq_kv(i)
        pos = torch.arange(n - r, n)[:, None]
        t = torch.arange(n)[None]
        see = t <= pos
        if window:
            see &= (t > pos - window) | (t < sinks)
        live = see.any(0)                       # what no row sees may hold anything
        for h in range(Hkv):
            kh, vh = K[h].clone(), V[h].clone()
            kh[~live], vh[~live] = 0.0, 0.0
            qh = x.q[r0:r0 + r, h * G:(h + 1) * G].double()
            z = torch.einsum("rgd,td->rgt", qh, kh) * scale
            mag = torch.einsum("rgd,td->rgt", qh.abs(), kh.abs()) * scale
            mag = mag.masked_fill(~see[:, None], 0.0).amax(-1)
            z = z.masked_fill(~see[:, None], -math.inf)
            L = torch.logsumexp(z, -1)
            w = torch.exp(z - L[..., None]).nan_to_num(0.0)
            cnt = see.sum(1)[:, None].double()
            e = (2 * D + 24) * U * mag + 8 * U
            if x.scale is not None:
                qmax = qh.abs().amax(-1, keepdim=True)
                dq = torch.where(qh.abs() < 2.0 ** -9 * qmax, torch.minimum(qh.abs(), 2.0 ** -17 * qmax), 0.0)
                lost = torch.einsum("rgd,td->rgt", dq, kh.abs()) * scale
                e = e + 2 * lost.masked_fill(~see[:, None], 0.0).amax(-1)
            sl = slice(h * G, (h + 1) * G)
            out[r0:r0 + r, sl] = torch.einsum("rgt,td->rgd", w, vh)
            wabs = torch.einsum("rgt,td->rgd", w, vh.abs())
            lse[r0:r0 + r, sl] = L
            otol[r0:r0 + r, sl] = (2 * (e + (cnt + 16) * U) + rounded)[..., None] * wabs + 1e-30
            ltol[r0:r0 + r, sl] = e + (cnt + 16) * U + 4 * U * L.abs().nan_to_num(0.0, posinf=0.0)
    return out, lse, otol, ltol


def assert_attended(got_out, got_lse, ref, rows_used=None):
    out, lse, otol, ltol = ref
    n = out.shape[0] if rows_used is None else rows_used
    o, l = got_out[:n].double().cpu(), got_lse[:n].double().cpu()
    out, lse, otol, ltol = out[:n], lse[:n], otol[:n], ltol[:n]
    if got_out.dtype == torch.bfloat16:
        otol = otol + BF16_HALF * out.abs() * 1.01
    none = torch.isinf(lse)
    assert torch.equal(torch.isinf(l) & (l < 0), none), "rows with / without visible tokens differ"
    assert not torch.isnan(o).any() and not torch.isnan(l).any()
    assert (o[none] == 0).all()
    err = (o - out).abs()
    assert (err <= otol).all(), f"out: worst {float((err / otol.clamp(min=1e-30)).max()):.2f} of its tolerance ({float(err.max()):.3e})"
    lerr = (l - lse).abs()[~none]
    assert (lerr <= ltol[~none]).all(), f"lse: worst error {float(lerr.max()):.3e}"


class Pool:
    """The page bookkeeping in plain Python, in the order the header gives it."""

    def __init__(self, places, pages_each, n_pages, page, k=None, v=None):
        self.table = [[-1] * pages_each for _ in range(places)]
        self.lens = [0] * places
        self.refs = [0] * n_pages
        self.page = page
        self.data = [d for d in (k, v) if d is not None]   # [layers, n_pages, Hkv, page, D], changed in place
        self.unserved = 0

    def _pages(self, n):
        return -(-n // self.page)

    def _served(self, needs):
        """Free pages in ascending order for each need, or None."""
        free = [p for p, r in enumerate(self.refs) if r == 0]
        at, given = 0, []
        for n in needs:
            given.append(free[at:at + n] if n == 0 or at + n <= len(free) else None)
            at += n
        return given

    def _valid(self, places):
        return [0 <= s < len(self.lens) and s not in places[:i] for i, s in enumerate(places)]

    def extend(self, seqs, n_new):
        ok = self._valid(seqs)
        needs = []
        for i, (s, a) in enumerate(zip(seqs, n_new)):
            ok[i] = ok[i] and a >= 0 and self.lens[s] + a <= len(self.table[s]) * self.page
            needs.append(self._pages(self.lens[s] + a) - self._pages(self.lens[s]) if ok[i] else 0)
        for s, a, good, new in zip(seqs, n_new, ok, self._served(needs)):
            if not good or new is None:
                self.unserved += 1
                continue
            have = self._pages(self.lens[s])
            for j, p in enumerate(new):
                self.table[s][have + j] = p
                self.refs[p] = 1
            self.lens[s] += a

    def fork(self, src, dst, keep=None):
        ok = self._valid(dst)
        needs, lens = [], []
        for i, (s, d) in enumerate(zip(src, dst)):
            ok[i] = ok[i] and 0 <= s < len(self.lens) and self.lens[d] == 0 and (keep is None or keep[i] >= 0)
            n = (self.lens[s] if keep is None else min(self.lens[s], keep[i])) if ok[i] else 0
            lens.append(n)
            needs.append(1 if n % self.page else 0)
        todo = list(zip(src, dst, ok, lens, self._served(needs)))
        for s, d, good, n, new in todo:
            if not good or new is None:
                self.unserved += 1
                continue
            full = n // self.page
            for j in range(full):
                self.table[d][j] = self.table[s][j]
                self.refs[self.table[s][j]] += 1
            if new:
                self.table[d][full] = new[0]
                self.refs[new[0]] = 1
                for x in self.data:
                    x[:, new[0], :, :n % self.page] = x[:, self.table[s][full], :, :n % self.page]
            self.lens[d] = n

    def free(self, seqs, keep=None):
        ok = self._valid(seqs)
        todo = []
        for i, s in enumerate(seqs):
            k = 0 if keep is None else keep[i]
            if ok[i] and k >= 0:
                k = min(k, self.lens[s])
                if k % self.page and k < self.lens[s] and self.refs[self.table[s][k // self.page]] > 1:
                    ok[i] = False
            todo.append((s, k, ok[i] and k >= 0))
        for s, k, good in todo:
            if not good:
                self.unserved += 1
                continue
            for j in range(self._pages(k), self._pages(self.lens[s])):
                self.refs[self.table[s][j]] -= 1
                self.table[s][j] = -1
            self.lens[s] = k

    def compact(self):
        used = [p for p, r in enumerate(self.refs) if r > 0]
        n = len(used)
        src, dst = [p for p in used if p >= n], [p for p in range(n) if self.refs[p] == 0]
        to = dict(zip(src, dst))
        for a, b in to.items():
            for x in self.data:
                x[:, b] = x[:, a]
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        return n
