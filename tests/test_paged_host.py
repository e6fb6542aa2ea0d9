"""Host-side checks of the paged cache's C ABI: symbols, and refusals that
come before CUDA is touched."""
import os
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
