"""Host-side checks of the C ABI of the paged cache of 8-bit codes: symbols,
and refusals that come before CUDA is touched."""
import os
import re

import pytest

from attention_block_gb300 import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = dict(n_q_heads=32, n_kv_heads=8, head_dim=128, page_size=16, num_pages=64, max_pages=16,
            max_batch=4, max_tokens=64, dtype="bf16")


def test_every_declared_function_is_exported_and_bound():
    text = open(os.path.join(ROOT, "include", "cf_paged8.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(cf_paged8_[a-z_]+)\s*\(", text))
    assert {"cf_paged8_create", "cf_paged8_append", "cf_paged8_attention", "cf_paged8_read",
            "cf_paged8_get_status", "cf_paged8_destroy"} == names
    for n in names:
        assert hasattr(binding.lib(), n) and n in binding.SIGNATURES


@pytest.mark.parametrize("kw,code", [
    (dict(n_q_heads=0), binding.CF_ERR_INVALID_ARG),
    (dict(n_kv_heads=5), binding.CF_ERR_INVALID_ARG),
    (dict(head_dim=96), binding.CF_ERR_UNSUPPORTED),
    (dict(page_size=24), binding.CF_ERR_UNSUPPORTED),
    (dict(dtype=3), binding.CF_ERR_INVALID_ARG),
    (dict(dtype="f32"), binding.CF_ERR_UNSUPPORTED),
    (dict(code=2), binding.CF_ERR_INVALID_ARG),
    (dict(code=-1), binding.CF_ERR_INVALID_ARG),
    (dict(layout=2), binding.CF_ERR_INVALID_ARG),
    (dict(page_stride=16 * 8 * 128 - 16), binding.CF_ERR_INVALID_ARG),
    (dict(page_stride=16 * 8 * 128 + 8), binding.CF_ERR_INVALID_ARG),
    (dict(rope_theta=0.0), binding.CF_ERR_INVALID_ARG),
    (dict(rope_sections=(16, 24, 23)), binding.CF_ERR_INVALID_ARG),
    (dict(scale=-1.0), binding.CF_ERR_INVALID_ARG),
    (dict(num_pages=1 << 25, page_stride=1 << 40), binding.CF_ERR_INVALID_ARG),
])
def test_create_rejects_bad_config_before_cuda(kw, code):
    rc, h = binding.cf_paged8_create_rc(binding.make_paged8_config(**dict(BASE, **kw)))
    assert rc == code and not h


def test_null_arguments():
    assert binding.cf_paged8_create_rc(None)[0] == binding.CF_ERR_INVALID_ARG
    lib = binding.lib()
    assert lib.cf_paged8_append(None, 1, 1, None, None, None, 0, 0, *([None] * 8), 0, None) == \
        binding.CF_ERR_INVALID_ARG
    assert lib.cf_paged8_attention(None, 1, 1, 1, None, 0, *([None] * 6), 0, 0,
                                   *([None] * 3)) == binding.CF_ERR_INVALID_ARG
    assert lib.cf_paged8_read(None, 1, 1, *([None] * 8), 0, None) == binding.CF_ERR_INVALID_ARG
    assert lib.cf_paged8_get_status(None) == binding.CF_ERR_INVALID_ARG
    lib.cf_paged8_destroy(None)
