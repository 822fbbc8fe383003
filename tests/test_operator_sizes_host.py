"""Sizes from 2^31 on, which do not fit the C interface's int, are refused before
anything is launched (no GPU needed: the tensors have no memory)."""
import pytest
import torch

import sparse_linear_hybrid_b200 as sl


class Fake:
    """A tensor of a given shape, type and strides on CUDA device 0, without memory."""

    def __init__(self, shape, dtype=torch.bfloat16):
        self.meta = torch.empty(shape, dtype=dtype, device="meta")
        self.shape, self.dtype, self.device = self.meta.shape, dtype, torch.device("cuda", 0)

    def __getattr__(self, name):  # dim, numel, stride, is_contiguous
        return getattr(self.meta, name)

    def get_device(self):
        return 0

    def data_ptr(self):
        return 0x10000000


@pytest.fixture
def device(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(sl, "_stream", lambda s: None)


def call(name):
    def fail(*a):
        raise AssertionError(f"{name} was called with {a}")
    return fail


@pytest.mark.parametrize("shape", [(2 ** 32 + 64,), (2 ** 31,), (2 ** 32 + 3, 1), (1, 2 ** 33 + 32), (2 ** 16, 2 ** 16 + 1, 33)])
def test_checkpoints(device, shape):
    x = Fake(shape)
    kept = sl.Checkpoint(Fake(shape, torch.uint8), Fake(sl._ckpt_scales_shape(shape), torch.uint8), "int8", torch.bfloat16)
    for name in ("salad_ckpt_pack", "salad_ckpt_unpack"):
        with pytest.raises(sl.SaladError) as e:
            sl._ckpt_call(call(name), name, [x], [kept], "int8", None)
        assert e.value.status == sl.SALAD_ERR_UNSUPPORTED


@pytest.mark.parametrize("shape", [(1, 2 ** 32 + 1, 1, 2), (2 ** 32 + 1, 1, 1, 2), (1, 1, 1, 2 ** 32 + 2)])
def test_rotary_positions(device, shape):
    x, freq = Fake(shape), Fake((1,), torch.float64)
    for fn in (sl.rope_forward, sl.rope_backward):
        with pytest.raises(sl.SaladError) as e:
            fn(x, None, freq)
        assert e.value.status == sl.SALAD_ERR_UNSUPPORTED
