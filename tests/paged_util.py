"""Helpers of the paged-cache tests: random problems, and the operators in
float64 on the CPU, written from the formulas in include/cf_paged.h.

Tolerances are computed beside the reference from the values themselves:
  u      half a step of the storage type (2^-8 bf16, 2^-11 fp16, 2^-24 fp32),
         the rounding of an output, and of a probability where those are
         rounded to 16 bits;
  e      2^-23, one fp32 operation (tensor-core sums may truncate).
A score s = scale q.k of d products is off by at most (d + 2) e sum|q k| scale
=: ds, its exponential by the factor 1 + 2 ds + 4 e; a sum over n keys adds n
e.  So |err o_c| <= u |o_c| + (u_p + 2 (2 ds + (n + 8) e)) sum_j p_j |v_jc|,
the normalisation doubling the second term, and
|err lse| <= 2 ds + (n + 8) e + 4 e |lse|.
A rotated pair (a, b): cos and sin are off by 2^-22, the two products and
their sum by 2 e: |err| <= u |x| + 2^-20 (|a| + |b|)."""
from __future__ import annotations

import math

import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E = 2.0 ** -23


def half_step(dtype):
    return torch.finfo(DT[dtype]).eps / 2


class Problem:
    """A ragged batch over a paged cache, on the CPU in storage types."""

    def __init__(self, q_len, kv_len, nq=4, nkv=2, d=128, page=16, dtype="bf16", layout=0,
                 interleaved=False, extra_tokens=0, prefix=0, seed=0, spare=2, max_pages=None,
                 q_scale=2.0):
        g = torch.Generator().manual_seed(seed)
        dt = DT[dtype]
        self.q_len, self.kv_len, self.nq, self.nkv, self.d = list(q_len), list(kv_len), nq, nkv, d
        self.page, self.dtype, self.layout, self.prefix = page, dtype, layout, prefix
        self.batch = len(q_len)
        self.tokens = sum(q_len) + extra_tokens
        self.max_q = max(max(q_len), 1)
        self.starts = [sum(q_len[:b]) for b in range(self.batch + 1)]
        used = [-(-max(n, 0) // page) for n in kv_len]
        n_pre = -(-prefix // page)
        self.max_pages = max_pages or max(max(used), 1)
        self.num_pages = sum(used) + n_pre + spare
        order = torch.randperm(self.num_pages, generator=g).tolist()
        self.table = torch.full((self.batch, self.max_pages), -7, dtype=torch.int32)
        for b in range(self.batch):
            for i in range(used[b]):
                self.table[b, i] = order.pop()
        self.prefix_table = torch.tensor([order.pop() for _ in range(n_pre)] or [0],
                                         dtype=torch.int32)
        shape = (page, nkv, d) if layout == 0 else (nkv, page, d)
        n = 2 if interleaved else 1
        self.pools = [torch.randn(self.num_pages, n, *shape, generator=g).to(dt)
                      for _ in range(1 if interleaved else 2)]
        self.interleaved = interleaved
        self.q = (q_scale * torch.randn(self.tokens, nq, d, generator=g)).to(dt)
        self.k = torch.randn(self.tokens, nkv, d, generator=g).to(dt)
        self.v = torch.randn(self.tokens, nkv, d, generator=g).to(dt)

    def split(self, pools):
        """k_pages and v_pages as views of the pools."""
        if self.interleaved:
            return pools[0][:, 0], pools[0][:, 1]
        return pools[0][:, 0], pools[1][:, 0]

    def config(self, **kw):
        c = dict(n_q_heads=self.nq, n_kv_heads=self.nkv, head_dim=self.d, page_size=self.page,
                 num_pages=self.num_pages, max_pages=self.max_pages, max_batch=self.batch,
                 max_tokens=max(self.tokens, 1), dtype=self.dtype, layout=self.layout,
                 page_stride=2 * self.page * self.nkv * self.d if self.interleaved else 0)
        c.update(kw)
        return c

    def slot(self, pool, table_row, j):
        """View [nkv, d] of position j in a pool [pages, ...]."""
        page = pool[int(table_row[j // self.page])]
        return page[j % self.page] if self.layout == 0 else page[:, j % self.page]

    def gather(self, pool, table_row, js):
        if not js:
            return torch.zeros(0, self.nkv, self.d, dtype=torch.float64)
        return torch.stack([self.slot(pool, table_row, j) for j in js]).double()


def visible(p, length, window, sinks):
    hi = min(p, length - 1)
    return [j for j in range(hi + 1) if window == 0 or p - j < window or j < sinks]


def ref_attention(pr: Problem, window=0, sinks=0, scale=None, kv_len=None, k=None, v=None):
    """out, lse [T, nq, ..] in float64 and their tolerances; rows of tokens
    that belong to no sequence stay NaN."""
    kp, vp = pr.split(pr.pools) if k is None else (k, v)
    T, nq, d, G = pr.tokens, pr.nq, pr.d, pr.nq // pr.nkv
    scale = scale or 1 / math.sqrt(d)
    u = half_step(pr.dtype)
    u_p = 0.0 if pr.dtype == "f32" else u
    nan = float("nan")
    out, tol = (torch.full((T, nq, d), nan, dtype=torch.float64) for _ in range(2))
    lse, ltol = (torch.full((T, nq), nan, dtype=torch.float64) for _ in range(2))
    pre = list(range(pr.prefix))
    Kp = pr.gather(kp, pr.prefix_table, pre)
    Vp = pr.gather(vp, pr.prefix_table, pre)
    for b in range(pr.batch):
        L = (kv_len or pr.kv_len)[b]
        n = pr.q_len[b]
        p0 = L - n
        need = sorted(set(j for i in range(n) for j in visible(p0 + i, L, window, sinks)))
        K = torch.cat([Kp, pr.gather(kp, pr.table[b], need)])
        V = torch.cat([Vp, pr.gather(vp, pr.table[b], need)])
        at = torch.tensor(need, dtype=torch.long)
        for i in range(n):
            t, p = pr.starts[b] + i, p0 + i
            see = at <= p
            if window:
                see &= (p - at < window) | (at < sinks)
            see = torch.cat([torch.full((pr.prefix,), p >= 0), see & (p >= 0)])
            if not see.any():
                out[t], tol[t], lse[t], ltol[t] = 0, 0, -math.inf, 0
                continue
            for h in range(nq):
                Kh, Vh, q = K[see, h // G], V[see, h // G], pr.q[t, h].double()
                s = scale * (Kh @ q)
                ds = float((scale * (Kh.abs() @ q.abs())).max()) * (d + 2) * E
                m = s.max()
                w = torch.exp(s - m)
                tot = w.sum()
                w = w / tot
                out[t, h] = w @ Vh
                N = len(s)
                tol[t, h] = u * out[t, h].abs() + \
                    (u_p + 2 * (2 * ds + (N + 8) * E)) * (w @ Vh.abs()) + 1e-30
                if pr.dtype == "f16":  # probabilities and outputs below 2^-14 lose bits
                    tol[t, h] += 2.0 ** -24 * (1 + Vh.abs().sum(0))
                lse[t, h] = m + torch.log(tot)
                ltol[t, h] = 2 * ds + (N + 8) * E + 4 * E * lse[t, h].abs()
    return out, tol, lse, ltol


def ref_rope(x, P, theta, r, axis_of):
    """x [T, heads, d] float64 rotated by P [axes][T]; (result, |a| + |b|)."""
    y, s = x.clone(), torch.zeros_like(x)
    for i in range(r // 2):
        ang = torch.tensor([float(p) for p in P[axis_of[i]]], dtype=torch.float64) * theta ** (
            -2.0 * i / r)
        c, sn = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
        a, b = x[..., i], x[..., i + r // 2]
        y[..., i], y[..., i + r // 2] = a * c - b * sn, b * c + a * sn
        s[..., i] = s[..., i + r // 2] = a.abs() + b.abs()
    return y, s


def axes_of(r, sections, interleaved):
    n = r // 2
    if not sections:
        return [0] * n
    if interleaved:
        return [i % 3 if i // 3 < sections[i % 3] else 0 for i in range(n)]
    return [0] * sections[0] + [1] * sections[1] + [2] * sections[2]
