"""The paged cache's operators on the GPU against float64 (paged_util)."""
import math

import pytest
import torch

from attention_block_gb300 import binding
from paged_util import DT, Problem, axes_of, half_step, ref_attention, ref_rope

pytestmark = pytest.mark.gpu
OK, RANGE = binding.CF_OK, binding.CF_ERR_DEVICE_POS_RANGE


def dev(x):
    return x.cuda()


def close(got, want, tol, what):
    got = got.double().cpu()
    same = (got == want) | (got.isnan() & want.isnan())  # infinities and untouched rows
    err = torch.where(same, torch.zeros_like(want), (got - want).abs())
    bad = ~(err <= tol.nan_to_num(0))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at " \
        f"{bad.nonzero()[0].tolist()}: {got[bad][0]} for {want[bad][0]} (tol {tol[bad][0]})"


class Run:
    """One problem on the GPU behind one handle."""

    def __init__(self, pr, poison=True, **cfg):
        self.pr = pr
        if poison:  # slots that no row sees hold NaN
            self.poison()
        self.pools = [dev(p) for p in pr.pools]
        self.k_pages, self.v_pages = pr.split(self.pools)
        self.kv = binding.PagedKv(**pr.config(**cfg))
        self.q = dev(pr.q)
        self.q_start = torch.tensor(pr.starts, dtype=torch.int32, device="cuda")
        self.kv_len = torch.tensor(pr.kv_len, dtype=torch.int32, device="cuda")
        self.table, self.ptable = dev(pr.table), dev(pr.prefix_table)
        self.out = torch.full((pr.tokens, pr.nq, pr.d), float("nan"), dtype=DT[pr.dtype],
                              device="cuda")
        self.lse = torch.full((pr.tokens, pr.nq), float("nan"), device="cuda")

    def poison(self):
        pr = self.pr
        kp, vp = pr.split(pr.pools)
        keep = [(pr.table[b], j) for b in range(pr.batch) for j in range(max(pr.kv_len[b], 0))]
        keep += [(pr.prefix_table, j) for j in range(pr.prefix)]
        saved = [(r, j, pr.slot(kp, r, j).clone(), pr.slot(vp, r, j).clone()) for r, j in keep]
        kp[...] = float("nan")
        vp[...] = float("nan")
        for r, j, a, b in saved:
            pr.slot(kp, r, j)[...] = a
            pr.slot(vp, r, j)[...] = b

    def attend(self, window=0, sinks=0, q_start="own", max_q=None, stream=None, lse=True):
        pr = self.pr
        qs = self.q_start if q_start == "own" else q_start
        a = (pr.batch, pr.tokens, max_q or pr.max_q, self.q, qs, self.kv_len, self.table)
        l = self.lse if lse else None
        if pr.prefix:
            self.kv.prefix_attention(*a, self.ptable, pr.prefix, self.k_pages, self.v_pages,
                                     self.out, lse=l, stream=stream)
        else:
            self.kv.attention(*a, self.k_pages, self.v_pages, self.out, lse=l, window=window,
                              n_sinks=sinks, stream=stream)

    def check(self, window=0, sinks=0, status=OK, **kw):
        out, tol, lse, ltol = ref_attention(self.pr, window, sinks, **kw)
        assert self.kv.status() == status
        close(self.out, out, tol, "out")
        close(self.lse, lse, ltol, "lse")


def attend_and_check(pr, window=0, sinks=0, **kw):
    r = Run(pr, **kw)
    r.attend(window, sinks)
    r.check(window, sinks)
    return r


TYPES = ["bf16", "f16", "f32"]


# ------------------------------------------------------------- attention --
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads", [(4, 4), (8, 2), (7, 1), (16, 1), (6, 2)], ids=str)
@pytest.mark.parametrize("d", [64, 128])
def test_single_tokens(dtype, heads, d):
    pr = Problem([1] * 5, [1, 2, 63, 130, 517], *heads, d=d, dtype=dtype, seed=1)
    r = attend_and_check(pr)
    first = r.out.clone()
    r.out.fill_(float("nan"))
    r.attend(q_start=None)  # the form without starts
    assert torch.equal(first, r.out)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("page", [1, 2, 8, 16, 64, 256])
@pytest.mark.parametrize("layout,inter", [(0, False), (1, False), (0, True), (1, True)])
def test_pages(dtype, page, layout, inter):
    pr = Problem([1, 3, 1], [200, 97, 64], page=page, layout=layout, interleaved=inter,
                 dtype=dtype, seed=2)
    attend_and_check(pr)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_len,kv_len", [
    ([2, 1, 3], [2, 500, 3]),            # few rows, two of them whole prompts
    ([1, 40, 0, 7, 129], [300, 40, 55, 200, 129]),   # mixed prompts, steps and an idle sequence
    ([257], [600]),
    ([64, 64], [64, 127]),
], ids=str)
def test_ragged_tokens(dtype, d, q_len, kv_len):
    attend_and_check(Problem(q_len, kv_len, 4, 2, d=d, dtype=dtype, seed=3))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (17, 0), (64, 4), (100, 130), (128, 1),
                                          (1000, 5), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("q_len,kv_len", [([1, 1, 1, 1], [1, 65, 300, 513]),
                                          ([5, 150, 2], [400, 150, 129])], ids=str)
def test_window_and_sinks(dtype, window, sinks, q_len, kv_len):
    attend_and_check(Problem(q_len, kv_len, 8, 2, dtype=dtype, seed=4), window, sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,n,window,sinks", [((8, 8), 3000, 500, 4), ((8, 2), 2500, 0, 0),
                                                  ((4, 4), 2049, 128, 130)], ids=str)
def test_long_prompts_against_plain_torch(dtype, d, heads, n, window, sinks):
    """Many items per block, twenty times over: every run gives the same bits,
    and they are within the roundings of the 64-bit result."""
    nq, nkv = heads
    g = torch.Generator(device="cuda").manual_seed(n)
    page, pages = 64, -(-n // 64)
    kp, vp = (torch.randn(pages, page, nkv, d, generator=g, device="cuda").to(DT[dtype])
              for _ in range(2))
    q = (2 * torch.randn(n, nq, d, generator=g, device="cuda")).to(DT[dtype])
    kv = binding.PagedKv(n_q_heads=nq, n_kv_heads=nkv, head_dim=d, page_size=page,
                         num_pages=pages, max_pages=pages, max_batch=1, max_tokens=n, dtype=dtype)
    st = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1)
    outs = []
    for _ in range(20):
        outs.append(torch.full_like(q, float("nan")))
        kv.attention(1, n, n, q, st, st[1:], table, kp, vp, outs[-1], window=window, n_sinks=sinks)
    assert kv.status() == OK
    K, V = (x.reshape(-1, nkv, d)[:n].double().repeat_interleave(nq // nkv, 1) for x in (kp, vp))
    i = torch.arange(n, device="cuda")
    hide = i[None] > i[:, None]
    if window:
        hide |= (i[:, None] - i[None] >= window) & (i[None] >= sinks)
    u = half_step(dtype)
    for h in range(nq):
        w = (q[:, h].double() @ K[:, h].T / math.sqrt(d)).masked_fill_(hide, -math.inf).softmax(-1)
        want, mag = w @ V[:, h], w @ V[:, h].abs()
        # both roundings, and the fp32 scores: |q k| / sqrt(d) <= 64 d 2^-23 stays below u / 2
        tol = u * want.abs() + (u + 2.0 ** -12) * mag + 2.0 ** -24
        err = (outs[0][:, h].double() - want).abs()
        assert (err <= tol).all(), (h, (err - tol).max())
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_that_see_nothing(dtype):
    """No keys at all, more tokens than keys, an idle sequence, and tokens
    behind the last sequence (left as they were)."""
    pr = Problem([1, 5, 0, 2, 40], [0, 3, 9, 2, 20], 4, 2, dtype=dtype, extra_tokens=3, seed=5)
    r = attend_and_check(pr)
    assert (r.out[0] == 0).all() and torch.isinf(r.lse[0]).all()
    assert r.out[-3:].isnan().all() and r.lse[-3:].isnan().all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("q_len", [[1, 1], [3, 2], [70, 20]], ids=str)
def test_unseen_slots_and_table_entries_do_not_matter(dtype, q_len):
    """Pages that lie wholly behind the window may be gone: their table entry
    is no page, and what sinks and window leave out holds NaN."""
    pr = Problem(q_len, [400, 333], 8, 2, dtype=dtype, seed=6)
    window, sinks = 90, 4
    kp, vp = pr.split(pr.pools)
    for b in range(2):
        lo = max(0, pr.kv_len[b] - q_len[b] - window + 1)
        for j in range(sinks, lo):
            pr.slot(kp, pr.table[b], j)[...] = float("nan")
            pr.slot(vp, pr.table[b], j)[...] = float("inf")
    r = Run(pr)
    want = ref_attention(pr, window, sinks)
    for b in range(2):
        lo = max(0, pr.kv_len[b] - q_len[b] - window + 1)
        gone = [i for i in range(1, pr.max_pages) if (i + 1) * pr.page <= lo]
        r.table[b, gone] = 2 ** 31 - 1
    r.attend(window, sinks)
    assert r.kv.status() == OK
    close(r.out, want[0], want[1], "out")
    close(r.lse, want[2], want[3], "lse")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,q_len,kv_len,window,sinks", [
    ((4, 4), [3], [40], 0, 0), ((8, 2), [2, 4], [70, 4], 20, 1),        # few rows
    ((2, 2), [300], [300], 0, 0), ((4, 2), [150, 60], [400, 60], 0, 0),  # many
    ((2, 1), [200], [500], 70, 9)], ids=str)
def test_infinities_that_some_rows_see_reach_no_others(dtype, d, heads, q_len, kv_len, window, sinks):
    """Keys and values of infinity or NaN at positions that later (or, behind
    the window, earlier) tokens see: the other rows stay exact, and the rows
    that see them get them."""
    pr = Problem(q_len, kv_len, *heads, d=d, dtype=dtype, seed=12)
    kp, vp = pr.split(pr.pools)
    hit = {}
    for b in range(pr.batch):
        p0 = kv_len[b] - q_len[b]
        hit[b] = sorted({kv_len[b] - 1, p0 + q_len[b] // 2, p0 + 1, max(p0 - 5, 0)})
        for n, j in enumerate(hit[b]):
            v = pr.slot(vp, pr.table[b], j)
            v[:, n::7] = [math.inf, -math.inf, math.nan, math.inf][n]
    clean = [p.clone() for p in pr.pools]
    want = ref_attention(pr, window, sinks)
    r = Run(pr)
    r.attend(window, sinks)
    assert r.kv.status() == OK
    got = r.out.double().cpu()
    finite = want[0].isfinite()
    assert torch.equal(got.isfinite(), finite)
    assert torch.equal(got.isnan(), want[0].isnan())
    close(torch.where(finite, got, 0.0), torch.where(finite, want[0], 0.0),
          torch.where(finite, want[1], 0.0), "finite values")
    assert (got[want[0].isinf()] == want[0][want[0].isinf()]).all()
    close(r.lse, want[2], want[3], "lse")
    # a key of NaN at the last position: only the last token's row knows of it
    pr.pools = clean
    kp, vp = pr.split(pr.pools)
    for b in range(pr.batch):
        for j in hit[b]:
            pr.slot(vp, pr.table[b], j)[...] = 1.0
        pr.slot(kp, pr.table[b], kv_len[b] - 1)[...] = math.nan
    want = ref_attention(pr, window, sinks)
    r = Run(pr)
    r.attend(window, sinks)
    last = [pr.starts[b + 1] - 1 for b in range(pr.batch)]
    keep = [t for t in range(pr.tokens) if t not in last]
    close(r.out[keep], want[0][keep], want[1][keep], "rows before the last")
    assert r.out[last].isnan().all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("q_len,kv_len", [([3, 2], [40, 9]), ([150, 20, 300], [170, 20, 300])], ids=str)
def test_infinities_behind_a_prefix(dtype, q_len, kv_len):
    """The same beside a shared prefix: own values that some rows see, twice on
    one handle, with a call without any between."""
    pr = Problem(q_len, kv_len, 8, 2, dtype=dtype, prefix=200, seed=36)
    plain = ref_attention(pr)
    r0 = Run(pr)
    kp, vp = pr.split(pr.pools)
    for b in range(pr.batch):
        p0 = kv_len[b] - q_len[b]
        pr.slot(vp, pr.table[b], p0 + 1)[:, ::5] = math.inf
        pr.slot(vp, pr.table[b], kv_len[b] - 1)[:, 1::5] = math.nan
    want = ref_attention(pr)
    r = Run(pr)
    finite = want[0].isfinite()
    for call in range(2):
        r.out.fill_(0.0)
        r.attend()
        assert r.kv.status() == OK
        got = r.out.double().cpu()
        assert torch.equal(got.isfinite(), finite) and torch.equal(got.isnan(), want[0].isnan())
        close(torch.where(finite, got, 0.0), torch.where(finite, want[0], 0.0),
              torch.where(finite, want[1], 0.0), "finite values")
        if call == 0:
            r.k_pages, r0.k_pages = r0.k_pages, r.k_pages
            r.v_pages, r0.v_pages = r0.v_pages, r.v_pages
            r.attend()
            close(r.out, plain[0], plain[1], "the call between")
            r.k_pages, r.v_pages = r0.k_pages, r0.v_pages


@pytest.mark.parametrize("dtype", TYPES)
def test_infinite_keys_and_extreme_scores(dtype):
    """Scores of +-6e4 and values near the type's limits: no overflow on the
    way, and -inf scores (a key of -inf) weigh nothing."""
    pr = Problem([1, 1], [40, 70], 2, 2, d=64, dtype=dtype, seed=7, q_scale=1.0)
    kp, vp = pr.split(pr.pools)
    pr.q[0, :, 0] = 600.0
    pr.q[0, :, 1:] = 0
    pr.slot(kp, pr.table[0], 3)[:, 0] = 600.0
    pr.slot(kp, pr.table[0], 9)[:, 0] = -600.0
    pr.slot(kp, pr.table[0], 11)[:, 0] = -math.inf
    vp.mul_(1000.0)
    attend_and_check(pr)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("prefix", [1, 16, 100, 321])
@pytest.mark.parametrize("q_len,kv_len,heads", [
    ([1] * 3, [1, 20, 130], (4, 2)), ([2, 0, 4], [2, 5, 40], (8, 2)), ([1] * 40, [3] * 40, (8, 2)),
    ([60, 3], [60, 70], (6, 2))], ids=str)
def test_shared_prefix(dtype, prefix, q_len, kv_len, heads):
    attend_and_check(Problem(q_len, kv_len, *heads, dtype=dtype, prefix=prefix, seed=8))


@pytest.mark.parametrize("dtype", TYPES)
def test_prefix_with_empty_rows_and_untouched_tail(dtype):
    pr = Problem([1, 3, 1], [0, 2, 17], 4, 2, dtype=dtype, prefix=50, extra_tokens=2, seed=9)
    r = attend_and_check(pr)
    assert (r.out[0] == 0).all() and r.out[-2:].isnan().all()


def test_prefix_of_length_zero_is_plain_attention():
    pr = Problem([1, 4], [33, 90], 4, 2, seed=10)
    r = Run(pr)
    r.kv.prefix_attention(2, pr.tokens, 4, r.q, r.q_start, r.kv_len, r.table, None, 0, r.k_pages,
                          r.v_pages, r.out, lse=r.lse)
    r.check()


@pytest.mark.parametrize("dtype", TYPES)
def test_scale_and_strided_queries(dtype):
    pr = Problem([1, 6], [40, 100], 4, 2, dtype=dtype, seed=11)
    r = Run(pr, scale=0.25)
    wide = torch.randn(pr.tokens, pr.nq * pr.d + 64, device="cuda").to(DT[dtype])
    wide[:, :pr.nq * pr.d] = r.q.view(pr.tokens, -1)
    r.q = wide[:, :pr.nq * pr.d].view(pr.tokens, pr.nq, pr.d)
    assert r.q.stride(0) == pr.nq * pr.d + 64
    r.attend()
    r.check(scale=0.25)


# ---------------------------------------------------------------- append --
def run_append(pr, theta=1e4, rope_dim=0, sections=None, inter=False, rope_pos=None, in_place=False,
               q_start="own", poison=True):
    r = Run(pr, poison=poison, rope_theta=theta, rope_dim=rope_dim, rope_sections=sections,
            rope_interleaved=inter)
    qkv = torch.cat([x.reshape(pr.tokens, -1) for x in (pr.q, pr.k, pr.v)], 1).cuda()
    a, b = pr.nq * pr.d, (pr.nq + pr.nkv) * pr.d
    q = qkv[:, :a].view(pr.tokens, pr.nq, pr.d)
    k, v = (qkv[:, x:y].view(pr.tokens, pr.nkv, pr.d) for x, y in ((a, b), (b, qkv.shape[1])))
    q_out = q if in_place else r.out
    rp = dev(torch.tensor(rope_pos, dtype=torch.int32)) if rope_pos is not None else None
    r.kv.append(pr.batch, pr.tokens, q, k, v, r.q_start if q_start == "own" else q_start, r.kv_len,
                r.table, r.k_pages, r.v_pages, q_out, rope_pos=rp)
    return r, q_out


def check_append(pr, r, q_out, theta=1e4, rope_dim=0, sections=None, inter=False, rope_pos=None,
                 status=OK, tail=None):
    assert r.kv.status() == status
    u, rd = half_step(pr.dtype), rope_dim or pr.d
    kw, vw = (x.clone() for x in pr.split(pr.pools))
    p_of = [None] * pr.tokens
    where = [None] * pr.tokens
    for b in range(pr.batch):
        for i in range(pr.q_len[b]):
            p = pr.kv_len[b] - pr.q_len[b] + i
            if p >= 0:
                p_of[pr.starts[b] + i], where[pr.starts[b] + i] = p, (pr.table[b], p)
    P = rope_pos or [[p or 0 for p in p_of]] * 3
    which = axes_of(rd, sections, inter)
    qw, qs = ref_rope(pr.q.double(), P, theta, rd, which)
    kr, ks = ref_rope(pr.k.double(), P, theta, rd, which)
    got_k, got_v = (x.cpu() for x in (r.k_pages, r.v_pages))
    for t in range(pr.tokens):
        if where[t] is None:
            continue
        close(q_out[t], qw[t], u * qw[t].abs() + 2.0 ** -20 * qs[t] + 1e-7, f"q {t}")
        gk, gv = (pr.slot(x, *where[t]) for x in (got_k, got_v))
        close(gk, kr[t], u * kr[t].abs() + 2.0 ** -20 * ks[t] + 1e-7, f"k {t}")
        assert torch.equal(gv, pr.v[t]), f"v {t}"
        pr.slot(kw, *where[t])[...] = gk  # every other slot stays as it was
        pr.slot(vw, *where[t])[...] = gv
    for got, want in ((got_k, kw), (got_v, vw)):
        assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0)), "a slot of no new token"


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout,inter", [(0, False), (1, True)])
def test_append(dtype, d, layout, inter):
    pr = Problem([1, 5, 0, 33], [100, 5, 4, 50], 4, 2, d=d, dtype=dtype, layout=layout,
                 interleaved=inter, extra_tokens=2, seed=20)
    r, q = run_append(pr)
    check_append(pr, r, q)
    assert q[-2:].isnan().all()  # tokens behind the last sequence


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("q_len", [1, 700])
def test_append_many_and_single(dtype, q_len):
    n = [1] * 9 if q_len == 1 else [q_len, 1, 3000]
    pr = Problem(n, [x + 7 for x in n], 3, 1, d=64, page=64, dtype=dtype, seed=21)
    r, q = run_append(pr, q_start=None if q_len == 1 else "own", poison=False)
    check_append(pr, r, q)


@pytest.mark.parametrize("dtype", TYPES)
def test_append_in_place_on_the_merged_projection(dtype):
    pr = Problem([2, 3], [9, 30], 4, 2, dtype=dtype, seed=22)
    r, q = run_append(pr, in_place=True)
    check_append(pr, r, q)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rope_dim", [16, 32, 112])
def test_append_partial_rotation(dtype, rope_dim):
    pr = Problem([2, 3], [9, 30], 4, 2, dtype=dtype, seed=23)
    r, q = run_append(pr, rope_dim=rope_dim, theta=5e5)
    check_append(pr, r, q, rope_dim=rope_dim, theta=5e5)
    assert torch.equal(q[..., rope_dim:].cpu(), pr.q[..., rope_dim:])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,sections,inter", [(128, (16, 24, 24), False), (128, (64, 0, 0), False),
                                              (128, (24, 20, 20), True), (64, (12, 10, 10), True),
                                              (64, (0, 16, 16), False)])
def test_append_three_axes(dtype, d, sections, inter):
    pr = Problem([7, 1], [9, 30], 4, 2, d=d, dtype=dtype, seed=24)
    rp = [[0, 1, 5, 100000, 2 ** 31 - 1, -3, 77, 9], [3, 1, 4, 1, 5, 9, 2, 6],
          [8, 7, 6, 5, 4, 3, 2, -2 ** 31]]
    r, q = run_append(pr, sections=sections, inter=inter, rope_pos=rp)
    # angles in float64: a position of 2^31 times a rate leaves 2^-22
    check_append(pr, r, q, sections=sections, inter=inter, rope_pos=rp)


@pytest.mark.parametrize("dtype", TYPES)
def test_append_far_positions_one_axis(dtype):
    pr = Problem([4], [4], 2, 2, dtype=dtype, seed=25)
    rp = [[131071, 1048577, 16777217, 2 ** 30 + 1]]
    r, q = run_append(pr, theta=1e6, rope_pos=rp)
    check_append(pr, r, q, theta=1e6, rope_pos=rp)


def test_append_without_queries():
    pr = Problem([2, 1], [5, 9], 4, 2, seed=26)
    r = Run(pr)
    k, v = dev(pr.k), dev(pr.v)
    r.kv.append(2, 3, None, k, v, r.q_start, r.kv_len, r.table, r.k_pages, r.v_pages, None)
    q_fake, _ = ref_rope(pr.q.double(), [[3, 4, 8]], 1e4, 128, [0] * 64)
    check_append(pr, r, q_fake)


def test_append_skips_tokens_before_the_start_and_reports_them():
    pr = Problem([3, 2], [2, 6], 4, 2, seed=27)
    r, q = run_append(pr)
    check_append(pr, r, q, status=RANGE)
    assert q[0].isnan().all()
    assert r.kv.status() == OK  # reading cleared it


# ------------------------------------------------- what the device reports --
def test_bad_lengths_and_pages_are_reported_and_stay_in_bounds():
    pr = Problem([1, 2, 1, 1], [20, 30, 40, 33], 4, 2, seed=30)
    r = Run(pr)
    good = ref_attention(pr)
    r.kv_len[0] = -1
    r.kv_len[1] = pr.max_pages * pr.page + 1
    r.table[2, 1] = pr.num_pages  # positions 16..31 of sequence 2 have no page
    r.attend()
    assert r.kv.status() == RANGE and r.kv.status() == OK
    assert (r.out[:3] == 0).all() and torch.isinf(r.lse[:3]).all()
    close(r.out[4], good[0][4], good[1][4], "the good sequence")
    K, V = (pr.gather(x, pr.table[2], list(range(40))) for x in pr.split(pr.pools))
    K[16:32] = V[16:32] = 0
    w = torch.softmax(torch.einsum("hd,shd->hs", pr.q[3].double(), K.repeat_interleave(2, 1)) /
                      math.sqrt(128), -1)
    o = torch.einsum("hs,shd->hd", w, V.repeat_interleave(2, 1))
    a = torch.einsum("hs,shd->hd", w, V.abs().repeat_interleave(2, 1))
    close(r.out[3], o, 2.0 ** -8 * (o.abs() + a) + 1e-3 * a, "the sequence with a lost page")


def test_more_tokens_than_max_q_and_bad_starts_are_reported():
    pr = Problem([2, 3, 1], [20, 30, 40], 4, 2, seed=31)
    r = Run(pr)
    good = ref_attention(pr)
    r.attend(max_q=2)
    assert r.kv.status() == RANGE
    assert (r.out[2:5] == 0).all()
    close(r.out[:2], good[0][:2], good[1][:2], "a good sequence")
    r.out.fill_(float("nan"))
    r.q_start.copy_(torch.tensor([0, 2, 1, 99], dtype=torch.int32))
    r.attend()
    assert r.kv.status() == RANGE
    close(r.out[:2], good[0][:2], good[1][:2], "a good sequence")
    assert r.out[2:].isnan().all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("prefix", [0, 40])
def test_bad_starts_and_lengths_of_prompts_are_reported(dtype, prefix):
    pr = Problem([70, 3, 40], [90, 30, 40], 4, 2, dtype=dtype, prefix=prefix, seed=33)
    r = Run(pr)
    good = ref_attention(pr)
    r.attend(max_q=69)
    assert r.kv.status() == RANGE
    assert (r.out[:70] == 0).all() and torch.isinf(r.lse[:70]).all()
    close(r.out[70:], good[0][70:], good[1][70:], "good sequences")
    r.out.fill_(float("nan"))
    r.q_start.copy_(torch.tensor([0, 70, 60, 999], dtype=torch.int32))
    r.attend()
    assert r.kv.status() == RANGE
    close(r.out[:70], good[0][:70], good[1][:70], "the good sequence")
    assert r.out[70:].isnan().all()
    r.q_start.copy_(torch.tensor(pr.starts, dtype=torch.int32))
    r.attend()
    r.check()


def test_strides_that_overflow_are_refused():
    pr = Problem([1, 2], [20, 30], 4, 2, seed=34)
    r = Run(pr)
    for stride in (2 ** 62, (1 << 40) + 8):
        with pytest.raises(binding.CfError) as e:
            r.kv.attention(2, 3, 2, r.q, r.q_start, r.kv_len, r.table, r.k_pages, r.v_pages, r.out,
                           q_stride=stride)
        assert e.value.code == binding.CF_ERR_INVALID_ARG


# -------------------------------------------------------------- refusals --
def test_refusals():
    pr = Problem([1, 2], [20, 30], 4, 2, seed=32)
    r = Run(pr)
    kv, INV, ALIAS = r.kv, binding.CF_ERR_INVALID_ARG, binding.CF_ERR_ALIAS
    L, s = binding.lib(), torch.cuda.current_stream().cuda_stream
    qp, kp, vp, op = (x.data_ptr() for x in (r.q, r.k_pages, r.v_pages, r.out))
    base = dict(h=kv.handle, batch=2, n=3, max_q=2, q=qp, qs=512, st=r.q_start.data_ptr(),
                kl=r.kv_len.data_ptr(), tab=r.table.data_ptr(), k=kp, v=vp, w=0, sk=0, out=op,
                lse=None, stream=s)

    def att(**kw):
        return L.cf_paged_attention(*dict(base, **kw).values())

    for kw in (dict(batch=3), dict(batch=-1), dict(n=4), dict(n=-1), dict(max_q=0), dict(max_q=4),
               dict(q=None), dict(q=qp + 2), dict(qs=511), dict(qs=516), dict(st=r.q_start.data_ptr() + 1),
               dict(kl=None), dict(tab=None), dict(k=None), dict(v=vp + 8), dict(w=-1), dict(sk=-1),
               dict(out=None), dict(out=op + 2), dict(lse=r.lse.data_ptr() + 2), dict(st=None)):
        assert att(**kw) == INV, kw
    for kw in (dict(out=qp), dict(out=kp), dict(out=vp), dict(lse=kp), dict(lse=op),
               dict(lse=r.table.data_ptr())):
        assert att(**kw) == ALIAS, kw
    assert att(batch=0) == OK and att(n=0) == OK
    pre = lambda n, t: L.cf_paged_prefix_attention(  # noqa: E731
        kv.handle, 2, 3, 2, qp, 512, base["st"], base["kl"], base["tab"], t, n, kp, vp, op, None, s)
    assert pre(-1, base["tab"]) == INV and pre(5, None) == INV
    k, v = dev(pr.k), dev(pr.v)
    ap = dict(h=kv.handle, b=2, n=3, q=qp, k=k.data_ptr(), v=v.data_ptr(), qs=512, ks=256,
              st=base["st"], kl=base["kl"], rp=None, tab=base["tab"], kp=kp, vp=vp, qo=op, qos=512,
              stream=s)

    def app(**kw):
        return L.cf_paged_append(*dict(ap, **kw).values())

    for kw in (dict(b=3), dict(n=4), dict(st=None), dict(q=None), dict(qo=None), dict(k=None),
               dict(v=None), dict(qs=500), dict(qs=516), dict(ks=255), dict(qos=8), dict(kp=None),
               dict(vp=vp + 4), dict(kl=None), dict(tab=None), dict(rp=base["st"] + 2)):
        assert app(**kw) == INV, kw
    for kw in (dict(qo=qp, qos=520), dict(qo=ap["k"]), dict(qo=kp), dict(k=kp), dict(v=vp),
               dict(vp=kp), dict(tab=kp)):
        assert app(**kw) == ALIAS, kw
    assert app(n=0) == OK
    assert kv.status() == OK
    for bad in (dict(q=r.q.float()), dict(q=r.q.cpu()), dict(q=r.q[:2]), dict(q=r.q.transpose(1, 2))):
        with pytest.raises(binding.CfError):
            kv.attention(2, 3, 2, bad["q"], r.q_start, r.kv_len, r.table, r.k_pages, r.v_pages, r.out)
    with pytest.raises(binding.CfError):
        kv.attention(2, 3, 2, r.q, r.q_start.long(), r.kv_len, r.table, r.k_pages, r.v_pages, r.out)
    with pytest.raises(binding.CfError):
        kv.attention(2, 3, 2, r.q, r.q_start, r.kv_len, r.table, r.k_pages[1:], r.v_pages, r.out)
    torch.cuda.synchronize()
    assert r.out.isnan().all()


# ------------------------------------------- streams, graphs, whole runs --
def test_capture_replay_with_growing_lengths_and_two_handles_on_two_streams():
    """Append and attention captured once, replayed while lengths grow; a
    second handle works on another stream at the same time."""
    prs = [Problem([1] * 6, [50, 1, 16, 17, 200, 130], 8, 2, seed=s, max_pages=16, spare=40)
           for s in (40, 41)]
    runs, graphs, streams, news = [], [], [], []
    for pr in prs:
        spare = sorted(set(range(pr.num_pages)) - set(pr.table.flatten().tolist()))
        for b in range(pr.batch):
            for i in range(pr.max_pages):
                if pr.table[b, i] < 0 and i * pr.page < pr.kv_len[b] + 8:
                    pr.table[b, i] = spare.pop()
        r = Run(pr, poison=False)
        st = torch.cuda.Stream()
        k, v, q = dev(pr.k), dev(pr.v), dev(pr.q)
        g = torch.cuda.CUDAGraph()
        st.wait_stream(torch.cuda.current_stream())
        torch.cuda.synchronize()
        r.q = torch.empty_like(q)
        with torch.cuda.graph(g, stream=st):
            r.kv.append(6, 6, q, k, v, None, r.kv_len, r.table, r.k_pages, r.v_pages, r.q)
            r.attend(q_start=None)
        runs.append(r), graphs.append(g), streams.append(st), news.append((q, k, v))
    for step in range(4):
        for pr, r, g, st, (q, k, v) in zip(prs, runs, graphs, streams, news):
            gen = torch.Generator().manual_seed(step)
            pr.kv_len = [n + 1 for n in pr.kv_len]
            pr.q, pr.k, pr.v = (torch.randn(*x.shape, generator=gen).to(x.dtype) for x in (pr.q, pr.k, pr.v))
            with torch.cuda.stream(st):
                r.kv_len.copy_(torch.tensor(pr.kv_len, dtype=torch.int32))
                for a, b in zip((q, k, v), (pr.q, pr.k, pr.v)):
                    a.copy_(b)
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for pr, r in zip(prs, runs):
            q0 = pr.q
            pr.q = r.q.cpu()  # the rotated queries; append has its own tests
            pr.pools = [p.cpu() for p in r.pools]
            r.check()
            pr.q = q0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_prompt_then_steps_equal_one_prompt(dtype):
    """A prompt appended and attended in pieces (whole, then token by token,
    then with a shared prefix) gives the rows of the one-piece run."""
    n, nq, nkv, d, page = 90, 8, 2, 128, 16
    g = torch.Generator().manual_seed(50)
    q, k, v = (torch.randn(n, h, d, generator=g).to(DT[dtype]).cuda() for h in (nq, nkv, nkv))
    kv = binding.PagedKv(n_q_heads=nq, n_kv_heads=nkv, head_dim=d, page_size=page, num_pages=12,
                         max_pages=6, max_batch=2, max_tokens=n, dtype=dtype)
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(2, 6)
    kp, vp = (torch.zeros(12, page, nkv, d, dtype=DT[dtype], device="cuda") for _ in range(2))

    def i32(*x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def step(seq, lo, hi):
        """Tokens lo..hi-1 of the text into sequence seq."""
        qr, out = torch.empty_like(q[lo:hi]), torch.empty_like(q[lo:hi])
        a = (i32(0, hi - lo), i32(hi), table[seq:seq + 1])
        kv.append(1, hi - lo, q[lo:hi], k[lo:hi], v[lo:hi], *a, kp, vp, qr)
        kv.attention(1, hi - lo, hi - lo, qr, *a, kp, vp, out)
        return qr, out

    qr, whole = step(0, 0, n)
    parts = [step(1, 0, 41)[1]] + [step(1, t, t + 1)[1] for t in range(41, n)]
    assert torch.equal(kp[:6].float(), kp[6:].float())  # both caches hold the same
    # two computations of one value: each within u (1 + sum p |v| / |o|); compared in norm
    diff = (torch.cat(parts).double() - whole.double()).norm() / whole.double().norm()
    assert diff <= 4 * half_step(dtype), diff
    # the first 64 positions as a shared prefix of one sequence holding the rest
    out = torch.empty_like(q[64:])
    kv.prefix_attention(1, n - 64, n - 64, qr[64:].contiguous(), i32(0, n - 64), i32(n - 64),
                        table[0, 4:].contiguous().view(1, -1).repeat(1, 3), table[0, :4].contiguous(),
                        64, kp, vp, out)
    assert kv.status() == OK
    diff = (out.double() - whole[64:].double()).norm() / whole[64:].double().norm()
    assert diff <= 4 * half_step(dtype), diff


def test_the_dense_block_and_the_paged_run_agree():
    """cf_decode_attn_block's cache slots and attention against append and
    attention over pages that view the same dense cache."""
    from attention_block_gb300 import synth
    w = synth.custom(name="paged_vs_block", hidden=1024, n_q_heads=8, n_kv_heads=2, head_dim=128,
                     batch=3, s_max=320, dtype="bf16", positions="list:299,0,150")
    t = synth.make_layer(w, seed=3, device="cuda")
    blk = binding.DecodeAttnBlock(hidden=w.hidden, n_q_heads=8, n_kv_heads=2, head_dim=128,
                                  max_batch=3, s_max=320, rope_theta=w.rope_theta,
                                  rms_eps=w.rms_eps, dtype="bf16")
    kc, vc, out = t["k_cache"].clone(), t["v_cache"].clone(), torch.empty_like(t["hidden"])
    dbg = torch.zeros(3 * (2 * 8 * 128 + 2 * 2 * 128 + 1024), device="cuda")
    blk.set_debug(dbg)
    blk(3, t["hidden"], t["ln_weight"], t["w_qkv"], t["w_o"], kc, vc, t["positions"], out)
    assert blk.status() == OK
    blk.close()
    o_blk = dbg[3 * (8 + 2 * 2) * 128:][:3 * 8 * 128].view(3, 8, 128)
    x = t["hidden"].double()
    xn = x / (x.pow(2).mean(-1, keepdim=True) + w.rms_eps).sqrt() * t["ln_weight"].double()
    qkv = (xn @ t["w_qkv"].double()).to(torch.bfloat16)
    kv = binding.PagedKv(n_q_heads=8, n_kv_heads=2, head_dim=128, page_size=64, num_pages=15,
                         max_pages=5, max_batch=3, max_tokens=3, dtype="bf16",
                         rope_theta=w.rope_theta)
    table = torch.arange(15, dtype=torch.int32, device="cuda").view(3, 5)
    kp, vp = (t[c].clone().view(15, 64, 2, 128) for c in ("k_cache", "v_cache"))
    lens = t["positions"] + 1
    q_rot = torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda")
    o = torch.empty_like(q_rot)
    q, k, v = qkv[:, :1024].view(3, 8, 128), qkv[:, 1024:1280].view(3, 2, 128), qkv[:, 1280:].view(3, 2, 128)
    kv.append(3, 3, q, k, v, None, lens, table, kp, vp, q_rot)
    kv.attention(3, 3, 1, q_rot, None, lens, table, kp, vp, o)
    assert kv.status() == OK
    for a, b, what in ((kp.view_as(kc), kc, "k"), (vp.view_as(vc), vc, "v")):
        # the block rotates the fp32 projection, this run its 16-bit rounding
        d = (a.double() - b.double()).abs().max()
        assert d <= 4 * 2.0 ** -8 * b.double().abs().max(), (what, d)
    rel = (o.double() - o_blk.double()).norm() / o_blk.double().norm()
    assert rel <= 4 * 2.0 ** -8, rel


def test_offsets_past_32_bits():
    """A pool of more than 2^32 elements; the sequence's pages lie at its end."""
    nkv, d, page = 8, 128, 64
    num = 2 ** 32 // (nkv * d * page) + 64
    if torch.cuda.mem_get_info()[0] < 5 * num * page * nkv * d:
        pytest.skip("needs 20 GB of device memory")
    g = torch.Generator(device="cuda").manual_seed(60)
    kp, vp = (torch.zeros(num, page, nkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kv = binding.PagedKv(n_q_heads=8, n_kv_heads=nkv, head_dim=d, page_size=page, num_pages=num,
                         max_pages=4, max_batch=2, max_tokens=300)
    kv.close()
    kv = binding.PagedKv(n_q_heads=8, n_kv_heads=nkv, head_dim=d, page_size=page, num_pages=num,
                         max_pages=4, max_batch=2, max_tokens=300, dtype="bf16")
    table = torch.tensor([[num - 1, num - 5, num - 9, num - 2], [0, 1, 2, num - 3]],
                         dtype=torch.int32, device="cuda")
    for n in ((200, 100), (1, 1)):
        lens = torch.tensor([250, 256], dtype=torch.int32, device="cuda")
        T = sum(n)
        st = torch.tensor([0, n[0], T], dtype=torch.int32, device="cuda")
        q, k, v = (torch.randn(T, 8, d, generator=g, device="cuda").bfloat16() for _ in range(3))
        qr, o = torch.empty_like(q), torch.empty_like(q)
        kv.append(2, T, q, k, v, st, lens, table, kp, vp, qr)
        kv.attention(2, T, max(n), qr, st, lens, table, kp, vp, o)
        assert kv.status() == OK
        for b in range(2):
            K, V = (x[table[b].long()].reshape(-1, nkv, d)[:int(lens[b])].double() for x in (kp, vp))
            assert torch.equal(V[int(lens[b]) - n[b]:], v[int(st[b]):int(st[b + 1])].double())
            s = torch.einsum("nhd,shd->hns", qr[int(st[b]):int(st[b + 1])].double(), K) / math.sqrt(d)
            p = torch.arange(int(lens[b]) - n[b], int(lens[b]), device="cuda")[:, None]
            s.masked_fill_(torch.arange(int(lens[b]), device="cuda")[None] > p, -math.inf)
            want = torch.einsum("hns,shd->nhd", s.softmax(-1), V)
            err = (o[int(st[b]):int(st[b + 1])].double() - want).norm() / want.norm()
            assert err <= 2 * 2.0 ** -8, err


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("case", [
    dict(q_len=[1] * 700, kv=lambda b: b % 41, heads=(4, 1), d=64),          # runs of sequences per thread
    dict(q_len=[2] * 600, kv=lambda b: 2 + b % 37, heads=(16, 1), d=64),     # more row tiles than threads
    dict(q_len=[1] * 40 + [0] * 300 + [3], kv=lambda b: 5 + b, heads=(2, 2), d=128),
    dict(q_len=[1, 0, 1100, 1], kv=lambda b: [900, 3, 1200, 31][b], heads=(2, 1), d=64, window=33, sinks=2),
], ids=["700x1", "600x2", "idle", "long"])
def test_many_sequences(dtype, case):
    n = len(case["q_len"])
    pr = Problem(case["q_len"], [max(case["kv"](b), 0) for b in range(n)], *case["heads"],
                 d=case["d"], dtype=dtype, seed=70)
    attend_and_check(pr, case.get("window", 0), case.get("sinks", 0))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("q_len,heads,prefix", [
    ([1] * 300, (8, 4), 40),      # short prefix, more items than blocks
    ([4] * 150, (8, 2), 700),     # drafts: states of whole items and of cut ones
    ([200] * 3, (4, 2), 300),     # prompts behind a prefix
    ([1], (4, 4), 5000),          # few rows, one long prefix
], ids=str)
def test_prefix_of_large_batches(dtype, q_len, heads, prefix):
    pr = Problem(q_len, [n + 3 * (b % 9) for b, n in enumerate(q_len)], *heads, d=64,
                 dtype=dtype, prefix=prefix, seed=71)
    attend_and_check(pr)


def test_calls_of_every_kind_on_one_handle_repeat_their_bits():
    """Few rows, many rows, windows and prefixes in turn, twice: nothing of a
    call stays behind in the workspace, and no order of arrival shows."""
    pr = Problem([1] * 9 + [70, 130], [40 * (b + 1) for b in range(11)], 8, 2, seed=72, prefix=90)
    r = Run(pr)
    one = torch.arange(10, dtype=torch.int32, device="cuda")

    def all_calls():
        got = []
        for call in range(4):
            out, lse = torch.empty_like(r.out), torch.empty_like(r.lse)
            a = (r.k_pages, r.v_pages, out)
            if call == 0:    # the first nine sequences, single tokens
                r.kv.attention(9, 9, 1, r.q, one, r.kv_len, r.table, *a, lse=lse)
                out, lse = out[:9], lse[:9]
            elif call == 1:
                r.kv.attention(11, pr.tokens, 130, r.q, r.q_start, r.kv_len, r.table, *a, lse=lse,
                               window=50, n_sinks=3)
            elif call == 2:
                r.kv.prefix_attention(11, pr.tokens, 130, r.q, r.q_start, r.kv_len, r.table,
                                      r.ptable, 90, *a, lse=lse)
            else:
                r.kv.prefix_attention(9, 9, 1, r.q, None, r.kv_len, r.table, r.ptable, 90, *a,
                                      lse=lse)
                out, lse = out[:9], lse[:9]
            got += [out.clone(), lse.clone()]
        return got

    first = all_calls()
    for _ in range(3):
        for x, y in zip(first, all_calls()):
            assert torch.equal(x, y)
    want = ref_attention(pr)
    close(first[4], want[0], want[1], "prefix")
    assert r.kv.status() == OK


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("head_dim", [64, 128])
def test_prefix_with_many_short_prompts(dtype, head_dim):
    # more than 16 rows a head, several items to a block, rows that see nothing, sequences without
    # tokens; then twice more on the handle: every call finds the lists empty again
    pr = Problem([8, 5, 0, 9] * 60, [8, 130, 0, 4] * 60, 8, 2, d=head_dim, dtype=dtype, prefix=300,
                 seed=31)
    r = attend_and_check(pr)
    first = r.out.clone()
    for _ in range(2):
        r.out.fill_(float("nan"))
        r.attend()
        assert torch.equal(r.out, first)
    assert r.kv.status() == OK


@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("q_len,kv_len,heads,prefix,window", [
    ([1], [5000], (4, 1), 0, 0),              # 4 rows, the positions over many blocks
    ([1, 1], [3001, 5], (16, 1), 0, 700),     # 16 rows, one block has nothing to see
    ([3, 0, 2], [900, 4, 2], (6, 2), 333, 0),  # a prefix, an idle sequence
    ([130], [700], (3, 1), 0, 90),            # several row tiles, rows of two tokens in one
], ids=str)
def test_fp32_over_many_blocks(head_dim, q_len, kv_len, heads, prefix, window):
    pr = Problem(q_len, kv_len, *heads, d=head_dim, dtype="f32", prefix=prefix, seed=32)
    r = attend_and_check(pr, window, 2 if window else 0)
    first = r.out.clone()
    for _ in range(2):  # the tickets are back at zero, the order of arrival does not show
        r.out.fill_(float("nan"))
        r.attend(window, 2 if window else 0)
        assert torch.equal(r.out, first)


@pytest.mark.parametrize("q_len,heads", [
    ([1] * 193, (4, 2)), ([0, 1, 2, 0] * 150, (4, 2)), ([1] * 700, (5, 1)),
    ([0] * 400 + [40] + [0] * 300, (6, 1)), ([1] * 3 + [0] * 37000 + [2] * 40, (3, 1))], ids=lambda x: str(len(x)))
def test_fp32_finds_its_sequences(q_len, heads):
    pr = Problem(q_len, [n + b % 5 for b, n in enumerate(q_len)], *heads, d=64, page=8,
                 dtype="f32", seed=35)
    attend_and_check(pr)


@pytest.mark.parametrize("prefix", [0, 60])
def test_captured_prompts_replay_with_other_lengths(prefix):
    pr = Problem([100, 3, 40], [150, 3, 90], 8, 2, seed=73, prefix=prefix, max_pages=16, spare=60)
    spare = sorted(set(range(pr.num_pages)) - set(pr.table.flatten().tolist()) -
                   set(pr.prefix_table.tolist()))
    for b in range(3):
        for i in range(16):
            if pr.table[b, i] < 0:
                pr.table[b, i] = spare.pop() if spare else 0
    r = Run(pr, poison=False)
    r.attend()  # kernels are loaded before the capture
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        r.attend()
        r.attend()
    for lens, starts in (([150, 3, 90], [0, 100, 103, 143]), ([100, 77, 41], [0, 100, 103, 143]),
                         ([230, 1, 70], [0, 70, 71, 120])):
        r.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        r.q_start.copy_(torch.tensor(starts, dtype=torch.int32))
        r.out.fill_(float("nan")), r.lse.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        pr.kv_len, pr.starts = lens, starts
        pr.q_len = [starts[b + 1] - starts[b] for b in range(3)]
        r.check()


def test_another_device_or_stream():
    """The call goes to torch's current stream, or to the one given."""
    pr = Problem([1, 1], [300, 17], 4, 2, seed=74)
    r = Run(pr)
    want = ref_attention(pr)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for how in ("current", "given", "raw"):
        r.out.fill_(float("nan"))
        s.wait_stream(torch.cuda.current_stream())
        if how == "current":
            with torch.cuda.stream(s):
                r.attend()
        else:
            r.attend(stream=s if how == "given" else s.cuda_stream)
        s.synchronize()
        close(r.out, want[0], want[1], how)


def test_workspace_follows_the_largest_call():
    """Handles of the smallest size, and outputs next to their neighbours."""
    pr = Problem([1], [33], 8, 2, seed=75)
    r = Run(pr)
    big = torch.full((3, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    r.out = big[1:2]
    r.attend()
    want = ref_attention(pr)
    close(big[1:2], want[0], want[1], "out")
    assert (big[0] == 7).all() and (big[2] == 7).all()
