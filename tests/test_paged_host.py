"""Host-side checks of the paged cache's C ABI: symbols, and refusals that
come before CUDA is touched."""
import ctypes
import os
import random
import re

import pytest

from attention_block_gb300 import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = dict(n_q_heads=32, n_kv_heads=8, head_dim=128, page_size=16, num_pages=64, max_pages=16,
            max_batch=4, max_tokens=64, dtype="bf16")


def test_every_declared_function_is_exported_and_bound():
    text = open(os.path.join(ROOT, "include", "cf_paged.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(cf_paged_[a-z_]+)\s*\(", text))
    assert {"cf_paged_create", "cf_paged_append", "cf_paged_attention",
            "cf_paged_prefix_attention", "cf_paged_get_status", "cf_paged_destroy"} == names
    lib = binding.lib()
    for n in names:
        assert hasattr(lib, n) and n in binding.SIGNATURES


@pytest.mark.parametrize("kw,code", [
    (dict(n_q_heads=0), binding.CF_ERR_INVALID_ARG),
    (dict(n_kv_heads=5), binding.CF_ERR_INVALID_ARG),
    (dict(n_q_heads=70000, n_kv_heads=70000), binding.CF_ERR_INVALID_ARG),
    (dict(head_dim=0), binding.CF_ERR_INVALID_ARG),
    (dict(head_dim=96), binding.CF_ERR_UNSUPPORTED),
    (dict(head_dim=256), binding.CF_ERR_UNSUPPORTED),
    (dict(page_size=0), binding.CF_ERR_INVALID_ARG),
    (dict(page_size=24), binding.CF_ERR_UNSUPPORTED),
    (dict(page_size=2048), binding.CF_ERR_UNSUPPORTED),
    (dict(num_pages=0), binding.CF_ERR_INVALID_ARG),
    (dict(max_pages=0), binding.CF_ERR_INVALID_ARG),
    (dict(max_pages=1 << 30), binding.CF_ERR_INVALID_ARG),
    (dict(max_batch=0), binding.CF_ERR_INVALID_ARG),
    (dict(max_batch=65536), binding.CF_ERR_INVALID_ARG),
    (dict(max_tokens=0), binding.CF_ERR_INVALID_ARG),
    (dict(dtype=3), binding.CF_ERR_INVALID_ARG),
    (dict(layout=2), binding.CF_ERR_INVALID_ARG),
    (dict(page_stride=16 * 8 * 128 - 8), binding.CF_ERR_INVALID_ARG),
    (dict(page_stride=16 * 8 * 128 + 4), binding.CF_ERR_INVALID_ARG),
    (dict(rope_theta=0.0), binding.CF_ERR_INVALID_ARG),
    (dict(rope_theta=float("inf")), binding.CF_ERR_INVALID_ARG),
    (dict(rope_dim=8), binding.CF_ERR_INVALID_ARG),
    (dict(rope_dim=144), binding.CF_ERR_INVALID_ARG),
    (dict(rope_dim=-16), binding.CF_ERR_INVALID_ARG),
    (dict(rope_sections=(16, 24, 23)), binding.CF_ERR_INVALID_ARG),
    (dict(rope_sections=(-16, 56, 24)), binding.CF_ERR_INVALID_ARG),
    (dict(rope_sections=(4, 30, 30), rope_interleaved=True), binding.CF_ERR_INVALID_ARG),
    (dict(scale=-1.0), binding.CF_ERR_INVALID_ARG),
    (dict(scale=float("nan")), binding.CF_ERR_INVALID_ARG),
])
def test_create_rejects_bad_config_before_cuda(kw, code):
    rc, h = binding.cf_paged_create_rc(binding.make_paged_config(**dict(BASE, **kw)))
    assert rc == code and not h


@pytest.mark.parametrize("kw", [
    dict(num_pages=2 ** 31 - 1, page_size=1024, n_q_heads=65535, n_kv_heads=65535),
    dict(num_pages=1 << 25, page_stride=1 << 40)], ids=str)
def test_pools_whose_bytes_pass_63_bits_are_refused(kw):
    rc, h = binding.cf_paged_create_rc(binding.make_paged_config(**dict(BASE, **kw)))
    assert rc == binding.CF_ERR_INVALID_ARG and not h


def test_null_arguments():
    assert binding.cf_paged_create_rc(None)[0] == binding.CF_ERR_INVALID_ARG
    lib = binding.lib()
    assert lib.cf_paged_append(None, 1, 1, None, None, None, 0, 0, *([None] * 7), 0, None) == \
        binding.CF_ERR_INVALID_ARG
    assert lib.cf_paged_attention(None, 1, 1, 1, None, 0, *([None] * 5), 0, 0,
                                  *([None] * 3)) == binding.CF_ERR_INVALID_ARG
    assert lib.cf_paged_prefix_attention(None, 1, 1, 1, None, 0, *([None] * 4), 0,
                                         *([None] * 5)) == binding.CF_ERR_INVALID_ARG
    assert lib.cf_paged_get_status(None) == binding.CF_ERR_INVALID_ARG
    lib.cf_paged_destroy(None)


# --------------------------------------- how the many-row kernel cuts its work --
def line_of(q_start, kv_len, n_tokens, max_q, group, nkv, window, sinks, grid):
    """Runs (block, sequence, row tile, KV head, tiles, first, count, first and
    last slot), units of the call and of a block."""
    i32 = ctypes.c_int32
    st = (i32 * len(q_start))(*q_start) if q_start else None
    runs, line = (i32 * (9 << 16))(), (ctypes.c_int64 * 2)()
    n = binding.lib().cf_test_paged_line(len(kv_len), n_tokens, max_q, group, nkv, window, sinks, grid,
                                         st, (i32 * len(kv_len))(*kv_len), 1 << 16, runs, line)
    assert 0 <= n <= 1 << 16, n
    return [tuple(runs[9 * i:9 * i + 9]) for i in range(n)], line[0], line[1]


def items_of(q_start, kv_len, n_tokens, max_q, group, nkv, window, sinks):
    """Every item (sequence, row tile, KV head) in order, with its number of key tiles: those with a
    position that one of its rows sees, at least one."""
    items = []
    for b, length in enumerate(kv_len):
        t0, t1 = (q_start[b], q_start[b + 1]) if q_start else (b, b + 1)
        if not 0 <= t0 <= t1 <= n_tokens:
            continue
        n = t1 - t0
        if n > max_q or not 0 <= length <= 1 << 30:
            length = 0
        for j in range(-(-n * group // 256)):
            tiles = set()
            for r in range(256 * j, min(256 * j + 256, n * group), 1 if group < 4 else group // 2):
                for p in {length - n + r // group, length - n + min(256 * j + 255, n * group - 1) // group}:
                    lo = max(0, p - window + 1) if window else 0
                    tiles |= set(range(lo // 128, p // 128 + 1)) if p >= 0 else set()
                    tiles |= set(range(-(-min(sinks, lo) // 128))) if p >= 0 else set()
            items += [(b, j, h, max(1, len(tiles))) for h in range(nkv)]
    return items


def check_line(q_start, kv_len, n_tokens, max_q, group=4, nkv=2, window=0, sinks=0, grid=152):
    runs, total, upc = line_of(q_start, kv_len, n_tokens, max_q, group, nkv, window, sinks, grid)
    items = items_of(q_start, kv_len, n_tokens, max_q, group, nkv, window, sinks)
    assert total == sum(t + 5 for *_, t in items) and upc == -(-total // grid)
    at = 0
    for b, j, h, tiles in items:  # the runs are the items' tiles, in order, once each
        done, slots = 0, set()
        while done < tiles:
            block, *item, n, first, count, s0, s1 = runs[at]
            assert (tuple(item), n, first) == ((b, j, h), tiles, done) and count > 0
            assert 0 <= s0 <= s1 < 2 * grid and s0 <= 2 * block + 1 and 2 * block <= s1 + 1
            assert at == 0 or block >= runs[at - 1][0]
            done, at = done + count, at + 1
    assert at == len(runs)


FAR = [0, 64, 2000, 128, 192, 256, 320, 384, 448]


@pytest.mark.parametrize("q_start,kv_len,n_tokens,max_q", [
    (FAR, [1000, 5, 5, 1 << 20, 100, 64, 80, 90], 512, 64),   # a start too large before a long one
    (FAR, [5000, 5, 5, 700, 100, 64, 80, 90], 512, 64),
    ([300, 400, 200, 300, 100, 200, 0, 100], [400, 1, 300, 1, 250, 1, 700], 400, 100),
    ([0, 500, 0, 500, 0, 500], [500, 1, 900, 1, 600], 500, 500),
    ([-2 ** 31, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1], [50, 40, 30], 70, 70),
    ([5, 4, 3, 2, 1, 0], [5, 4, 3, 2, 1], 5, 5),
], ids=["far-long", "far-lost", "falling", "claimed-twice", "limits", "none"])
def test_malformed_starts_leave_one_line_of_work(q_start, kv_len, n_tokens, max_q):
    check_line(q_start, kv_len, n_tokens, max_q)
    check_line(q_start, kv_len, n_tokens, max_q, group=1, nkv=3, window=130, sinks=7, grid=5)


@pytest.mark.parametrize("seed", range(40))
def test_any_starts_and_lengths_leave_one_line_of_work(seed):
    r = random.Random(seed)
    batch = r.choice((1, 3, 17, 700))
    n_tokens = r.randint(1, 3 * batch + 400)
    cuts = sorted(r.randint(0, n_tokens) for _ in range(batch + 1))
    for _ in range(r.choice((0, 0, 1, 3, batch))):  # entries that are moved, out of order or of bounds
        cuts[r.randrange(batch + 1)] = r.choice((-1, n_tokens + 1, r.randint(0, n_tokens), 2 ** 31 - 1))
    lens = [r.choice((0, 1, -1, r.randint(0, 3000), r.randint(0, 300))) for _ in range(batch)]
    window = r.choice((0, 0, 1, 100, 1000))
    check_line(cuts, lens, n_tokens, r.choice((n_tokens, max(1, n_tokens // 2))),
               group=r.choice((1, 3, 4, 7, 40)), nkv=r.choice((1, 2, 5)), window=window,
               sinks=r.choice((0, 4, 200)) if window else 0, grid=r.choice((1, 5, 152)))
    if n_tokens >= batch:
        check_line(None, lens, batch, 1, group=40)
