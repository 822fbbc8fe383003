"""Checkpoints whose memory is used again: a refused call leaves them as they were."""
import pytest
import torch

import sparse_linear_hybrid_b200 as sl

pytestmark = pytest.mark.gpu


def test_a_refused_call_leaves_a_checkpoint_as_it_was():
    x = torch.randn(6, 64, device="cuda")
    c, other = sl.ckpt_pack(x), sl.ckpt_pack(torch.randn(4, 33, device="cuda"))
    want, codes = sl.ckpt_unpack(c), c.codes.clone()
    apart = torch.randn(4, 3, 64, device="cuda").half()[:, :2].transpose(0, 1)  # rows at several distances
    bad = sl.Checkpoint(c.codes.view(2, 3, 64), c.scales.view(2, 3, 2), "int8", torch.float32)
    with pytest.raises(ValueError):
        sl.ckpt_pack(torch.empty(6, 128, device="cuda").half()[:, ::2], fmt="e4m3", out=c)
    with pytest.raises(ValueError):
        sl.ckpt_pack(apart[:, :3], fmt="e4m3", out=bad)
    with pytest.raises(sl.SaladError):  # rows on top of each other
        sl.ckpt_pack(torch.randn(64, device="cuda").half().expand(6, 64), fmt="e4m3", out=c)
    with pytest.raises(sl.SaladError):  # codes inside the values
        sl.ckpt_pack([torch.randn(4, 33, device="cuda"), c.codes.view(torch.bfloat16)[:, :32]], fmt="e4m3",
                     out=[other, sl.Checkpoint(c.codes[:, :32].contiguous(), c.codes.view(-1)[:6].view(6, 1), "int8", torch.float32)])
    assert (c.fmt, c.dtype, bad.fmt) == ("int8", torch.float32, "int8")
    assert torch.equal(c.codes, codes) and torch.equal(sl.ckpt_unpack(c), want)
    assert other.fmt == "e4m3"  # (its own launch came first and was taken)
    again = sl.ckpt_pack(x.half(), fmt="e4m3", out=c)
    assert again is c and (c.fmt, c.dtype) == ("e4m3", torch.float16)
    empty = sl.ckpt_pack(torch.empty(0, 64, device="cuda"))
    assert sl.ckpt_pack(torch.empty(0, 64, device="cuda").half(), fmt="e4m3", out=empty).fmt == "e4m3"


def test_an_output_is_given_once():
    """Of several layouts, or more tensors than a launch takes, each goes by itself: the library's own check of overlaps
    does not see two of them."""
    x = torch.randn(4, 33, device="cuda")
    apart = torch.randn(4, 40, device="cuda")[:, :32]
    c, a = sl.ckpt_pack(x), sl.ckpt_pack(x[:, :32].contiguous())
    for xs, outs in (([x[:, :32].contiguous(), apart], [a, a]), ([x] * 5, [c, *sl.ckpt_pack([x] * 3), c])):
        with pytest.raises(ValueError, match="twice"):
            sl.ckpt_pack(xs, out=outs)
    y = torch.empty_like(x)
    with pytest.raises(ValueError, match="twice"):
        sl.ckpt_unpack([c] * 5, out=[y, *(torch.empty_like(x) for _ in range(3)), y])
    assert [s.fmt for s in sl.ckpt_pack([x, x], out=[None, c])] == ["int8", "int8"]
