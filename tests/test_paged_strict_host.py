"""What the binding of the paged caches hands on for strided rows, on CPU tensors."""
import pytest
import torch

from attention_block_gb300 import binding


@pytest.mark.parametrize("kind", [binding.PagedKv, binding.Paged8Kv])
def test_a_stride_that_is_given_ends_within_the_tensor(kind):
    kv = kind.__new__(kind)
    kv.handle, kv._dtype, kv._dev = None, torch.float16, -1
    x = torch.zeros(6, 512, dtype=torch.float16)[:, :256]
    assert kv._rows(x, 6, 256, None, "x") == (x.data_ptr(), 512)
    assert kv._rows(x, 6, 256, 512, "x") == (x.data_ptr(), 512)
    assert kv._rows(x.unflatten(1, (2, 128)), 3, 256, 1024, "x") == (x.data_ptr(), 1024)
    assert kv._rows(x[:1], 1, 256, 999, "x") == (x.data_ptr(), 999)  # of a single row it says nothing
    assert kv._rows(x.data_ptr(), 6, 256, 4096, "x") == (x.data_ptr(), 4096)
    for n, stride in ((6, 520), (4, 1024), (2, 4096), (6, 2 ** 62)):
        with pytest.raises(binding.CfError) as e:
            kv._rows(x, n, 256, stride, "x")
        assert e.value.code == binding.CF_ERR_INVALID_ARG
