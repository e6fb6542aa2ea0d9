"""Helpers of the tests of the paged cache of 8-bit codes: random problems, and
the operators in float64, written from the formulas in include/cf_paged8.h.

Tolerances of attention are computed beside the reference from the values
themselves, with u half a step of the storage type and e = 2^-23 one fp32
operation (tensor-core sums may truncate):
  a score of d products, its scale and the bound's are off by
    ds <= (d + 4) e scale ks sum|q k|;
  in base 2 it is taken together with log2 vs, whose error and the sums' are
    db <= 3 e (max|s| / ln 2 + max|log2 vs| + 4);
  so a weight w_j = p_j vs_j is off by the factor 1 + 2 ds + 2 db, enters the
  product with half a step of fp16, 2^-11, and below 2^-14 of the row's largest
  by 2^-32 of it at most; the sum over n keys adds n e.
  |err o_c| <= u |o_c| + (2^-11 + 2 (2 ds + 2 db + (n + 8) e)) sum_j w_j |v_jc|
               + 2^-31 max_j w_j sum_j |v_jc|
  |err lse| <= 2 ds + db + (n + 8) e + 4 e |lse|
A code stands for x_i / amax * Q with an error of up to half a step of the code
(int8: 1/2; e4m3: 2^-4 of the value, at least 2^-10), and what moves x_i itself."""
from __future__ import annotations

import math

import torch

from paged_util import DT, E, half_step, ref_rope

CODE = {"int8": (torch.int8, 127.0), "e4m3": (torch.float8_e4m3fn, 448.0)}


def quantise(x, code):
    """Codes (the code's type) and scales of heads x [.., d] in float64."""
    dt, top = CODE[code]
    amax = x.abs().amax(-1, keepdim=True)
    y = torch.where(amax < 2.0 ** -100, torch.zeros_like(x), x / amax.clamp(min=2.0 ** -100) * top)
    codes = (y.round() if code == "int8" else y.float()).to(dt)
    return codes, torch.where(amax < 2.0 ** -100, torch.zeros_like(amax), amax / top)[..., 0].float()


class Problem8:
    """A ragged batch over a paged cache of codes, on the GPU."""

    def __init__(self, q_len, kv_len, nq=4, nkv=2, d=128, page=16, dtype="bf16", code="e4m3", layout=0,
                 interleaved=False, extra_tokens=0, seed=0, spare=2, q_scale=2.0, max_pages=None):
        g = torch.Generator().manual_seed(seed)
        self.q_len, self.kv_len, self.nq, self.nkv, self.d = list(q_len), list(kv_len), nq, nkv, d
        self.page, self.dtype, self.code, self.layout = page, dtype, code, layout
        self.batch, self.tokens = len(q_len), sum(q_len) + extra_tokens
        self.max_q = max(max(q_len), 1)
        self.starts = [sum(q_len[:b]) for b in range(self.batch + 1)]
        used = [-(-max(n, 0) // page) for n in kv_len]
        self.max_pages = max_pages or max(max(used), 1)
        self.num_pages = sum(used) + spare
        order = torch.randperm(self.num_pages, generator=g).tolist()
        table = torch.full((self.batch, self.max_pages), -7, dtype=torch.int32)
        for b in range(self.batch):
            for i in range(used[b]):
                table[b, i] = order.pop()
        self.table = table.cuda()
        self.interleaved = interleaved
        inner = (page, nkv) if layout == 0 else (nkv, page)
        x = torch.randn(2, self.num_pages, *inner, d, generator=g).double()
        x *= 0.2 + 1.6 * torch.rand(2, self.num_pages, *inner, 1, generator=g)
        codes, scales = quantise(x, code)
        if layout == 0:
            scales = scales.transpose(2, 3)
        self.scales = torch.stack([scales[0], scales[1]], -1).contiguous().cuda()
        codes = codes.cuda()
        if interleaved:
            self.pool = codes.view(torch.uint8).transpose(0, 1).contiguous().view(codes.dtype)
            self.k_pages, self.v_pages = self.pool[:, 0], self.pool[:, 1]
        else:
            self.k_pages, self.v_pages = codes[0].clone(), codes[1].clone()
        dt = DT[dtype]
        self.q = (q_scale * torch.randn(self.tokens, nq, d, generator=g)).to(dt).cuda()
        self.k = torch.randn(self.tokens, nkv, d, generator=g).to(dt).cuda()
        self.v = torch.randn(self.tokens, nkv, d, generator=g).to(dt).cuda()
        self.q_start = torch.tensor(self.starts, dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(self.kv_len, dtype=torch.int32, device="cuda")

    def config(self, **kw):
        c = dict(n_q_heads=self.nq, n_kv_heads=self.nkv, head_dim=self.d, page_size=self.page,
                 num_pages=self.num_pages, max_pages=self.max_pages, max_batch=self.batch,
                 max_tokens=max(self.tokens, 1), dtype=self.dtype, layout=self.layout, code=self.code,
                 page_stride=2 * self.page * self.nkv * self.d if self.interleaved else 0)
        c.update(kw)
        return c

    def held(self, b, lo, hi):
        """Codes [hi - lo, nkv, d] of K and V, and their scales [.., nkv], of positions lo .. hi - 1 in float64."""
        j = torch.arange(lo, hi, device="cuda")
        ids, slot = self.table[b][j // self.page].long(), j % self.page
        out = []
        for pool in (self.k_pages, self.v_pages):
            x = pool.float().double()
            out.append(x[ids, slot] if self.layout == 0 else x[ids, :, slot])
        s = self.scales[ids, :, slot].double()
        return out[0], out[1], s[..., 0], s[..., 1]


def ref_attention8(pr, window=0, sinks=0, scale=None, kv_len=None):
    """out, lse in float64 and their tolerances, on the GPU; rows of tokens that belong to no sequence stay NaN."""
    T, nq, d, G = pr.tokens, pr.nq, pr.d, pr.nq // pr.nkv
    scale = scale or 1 / math.sqrt(d)
    u = half_step(pr.dtype)
    nan = float("nan")
    out, tol = (torch.full((T, nq, d), nan, dtype=torch.float64, device="cuda") for _ in range(2))
    lse, ltol = (torch.full((T, nq), nan, dtype=torch.float64, device="cuda") for _ in range(2))
    for b in range(pr.batch):
        L, n, t0 = (kv_len or pr.kv_len)[b], pr.q_len[b], pr.starts[b]
        if n == 0:
            continue
        K, V, ks, vs = pr.held(b, 0, max(L, 0))
        j = torch.arange(max(L, 0), device="cuda")
        for lo in range(0, n, 256):
            rows = slice(t0 + lo, t0 + min(n, lo + 256))
            p = torch.arange(L - n + lo, L - n + min(n, lo + 256), device="cuda")[:, None]
            see = j <= p
            if window:
                see &= (p - j < window) | (j < sinks)
            any_ = see.any(-1)
            for h in range(nq):
                g = h // G
                q = pr.q[rows, h].double()
                s = scale * (q @ K[:, g].T) * ks[:, g]
                a = scale * (q.abs() @ K[:, g].abs().T) * ks[:, g].abs()
                s, a = s.masked_fill(~see, -math.inf), a.masked_fill(~see, 0)
                if L <= 0:
                    out[rows, h], tol[rows, h], lse[rows, h], ltol[rows, h] = 0, 0, -math.inf, 0
                    continue
                ds = a.amax(-1, keepdim=True) * (d + 4) * E
                m = s.amax(-1, keepdim=True)
                w = torch.exp(s - torch.where(any_[:, None], m, 0))
                tot = w.sum(-1, keepdim=True)
                w = torch.where(see, w / tot * vs[:, g], 0)
                lv = torch.where(vs[:, g] > 0, vs[:, g], 1).log2().abs().nan_to_num(0).max()
                db = 3 * E * (a.amax(-1, keepdim=True) / math.log(2) + lv + 4)
                N = see.sum(-1, keepdim=True)
                o = w @ V[:, g]
                out[rows, h] = torch.where(any_[:, None], o, 0)
                va = torch.where(see, 1.0, 0.0).double() @ V[:, g].abs()
                tol[rows, h] = u * o.abs() + (2.0 ** -11 + 2 * (2 * ds + 2 * db + (N + 8) * E)) * \
                    (w.abs() @ V[:, g].abs()) + 2.0 ** -31 * w.amax(-1, keepdim=True) * va + 1e-30
                if pr.dtype == "f16":  # outputs below 2^-14 lose bits
                    tol[rows, h] += 2.0 ** -25
                x = (m + torch.log(tot))[:, 0]
                lse[rows, h] = torch.where(any_, x, -math.inf)
                ltol[rows, h] = (2 * ds + db + (N + 8) * E)[:, 0] + 4 * E * x.abs()
    return out, tol, lse, ltol


def check_codes(codes, scale, x, moved, code, what):
    """codes [.., d] and scale [..] of heads x [.., d] that are known to within `moved` (of each element)."""
    top = CODE[code][1]
    c, s = codes.float().double(), scale.double()
    amax = x.abs().amax(-1)
    most = moved.amax(-1)
    assert ((s * top - amax).abs() <= most + 4 * 2.0 ** -24 * amax).all(), f"{what}: scales"
    y = x / amax[..., None].clamp(min=2.0 ** -100) * top
    dy = (moved / amax[..., None].clamp(min=2.0 ** -100) + most[..., None] / amax[..., None].clamp(min=2.0 ** -100) *
          y.abs() / top + 4 * 2.0 ** -24 * y.abs() / top) * top
    step = torch.full_like(y, 0.5) if code == "int8" else (y.abs() + dy).clamp(min=2.0 ** -6) * 2.0 ** -4
    bad = ~((c - y).abs() <= step + dy)
    assert not bad.any(), f"{what}: {int(bad.sum())} codes off, first at {bad.nonzero()[0].tolist()}: " \
        f"{c[bad][0]} for {y[bad][0]}"


__all__ = ["CODE", "DT", "E", "Problem8", "check_codes", "half_step", "quantise", "ref_attention8", "ref_rope"]
