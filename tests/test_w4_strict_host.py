"""What the binding of the 4-bit products hands on for strided rows, with a call that only records its arguments."""
import pytest
import torch

from attention_block_gb300 import binding


@pytest.fixture
def product():
    """A W4Matvec of CPU tensors, 256 x 130, whose call returns what cf_w4_matvec says to strides below K."""
    m = binding.W4Matvec.__new__(binding.W4Matvec)
    m.cfg, m.handle, m._dev = binding.make_w4_config(256, 130, 64, max_rows=8), None, -1
    m._dtype, m.packed_bytes, m._raw_stream = torch.float16, 16, lambda d: 0
    m.strides = []

    def call(handle, rows, x, x_stride, *rest):
        m.strides.append(x_stride)
        return binding.CF_OK if x_stride >= 256 else binding.CF_ERR_INVALID_ARG

    m._matvec = call
    packed, out = torch.zeros(16, dtype=torch.uint8), torch.zeros(8, 130, dtype=torch.float16)
    m.go = lambda rows, x, **kw: m(rows, x, packed, out, **kw)
    return m


def test_a_tensor_of_repeated_rows_is_not_read_as_dense(product):
    one = torch.zeros(1, 256, dtype=torch.float16)
    with pytest.raises(binding.CfError):  # four rows of 256 behind one another are not there
        product.go(4, one.expand(4, 256))
    assert product.strides in ([], [0])
    product.go(1, one.expand(4, 256))
    assert product.strides[-1] == 256


def test_strides_of_tensors_and_addresses(product):
    x = torch.zeros(8, 512, dtype=torch.float16)
    product.go(8, x[:, :256])
    product.go(1, x[:1, :256])
    product.go(3, x.data_ptr())
    product.go(3, x.data_ptr(), x_stride=512)
    product.go(8, x[:, :256], x_stride=512)
    product.go(4, x[:, :256], x_stride=1024)  # every second row
    assert product.strides == [512, 256, 256, 512, 512, 1024]
    for rows, stride in ((8, 1024), (5, 1024), (2, 4096)):
        with pytest.raises(binding.CfError):
            product.go(rows, x[:, :256], x_stride=stride)
    with pytest.raises(binding.CfError):
        product.go(2, x[:1, :256].expand(2, 256), x_stride=256)
    assert len(product.strides) == 6
