"""Host-side checks of the C ABI of the 4-bit products: symbols, and refusals
that come before CUDA is touched."""
import os
import re

import pytest

from attention_block_gb300 import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = dict(in_features=256, out_features=128, group=128, max_rows=4, dtype="bf16")
INVALID, UNSUPPORTED = binding.CF_ERR_INVALID_ARG, binding.CF_ERR_UNSUPPORTED


def test_every_declared_function_is_exported_and_bound():
    text = open(os.path.join(ROOT, "include", "cf_w4.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(cf_w4_[a-z_]+)\s*\(", text))
    assert {"cf_w4_create", "cf_w4_packed_bytes", "cf_w4_pack", "cf_w4_matvec", "cf_w4_get_status",
            "cf_w4_destroy"} == names
    for n in names:
        assert hasattr(binding.lib(), n) and n in binding.SIGNATURES


@pytest.mark.parametrize("kw,code", [
    (dict(in_features=0), INVALID), (dict(in_features=200), INVALID), (dict(in_features=1 << 21), INVALID),
    (dict(out_features=0), INVALID), (dict(out_features=127), INVALID), (dict(out_features=1 << 25), INVALID),
    (dict(group=0), INVALID), (dict(group=16), UNSUPPORTED), (dict(group=256), UNSUPPORTED),
    (dict(zeros=2), INVALID), (dict(max_rows=0), INVALID), (dict(max_rows=65), UNSUPPORTED),
    (dict(dtype=3), INVALID), (dict(in_features=1 << 20, out_features=1 << 24), INVALID)])
def test_create_rejects_bad_config_before_cuda(kw, code):
    rc, h = binding.cf_w4_create_rc(binding.make_w4_config(**dict(BASE, **kw)))
    assert rc == code and not h


def test_null_arguments():
    assert binding.cf_w4_create_rc(None)[0] == INVALID
    lib = binding.lib()
    assert lib.cf_w4_packed_bytes(None) == 0
    assert lib.cf_w4_pack(*([None] * 6)) == INVALID
    assert lib.cf_w4_matvec(None, 1, None, 0, *([None] * 4)) == INVALID
    assert lib.cf_w4_get_status(None) == INVALID
    lib.cf_w4_destroy(None)
