"""Rotary positions on the GPU against the rotation in 64 bits.

Tolerance per element: half a step of the output type (relative 2^-8 bf16,
2^-11 fp16, 2^-24 fp32) plus 1e-6 (|x1| + |x2|) scale for the arithmetic before
that rounding: the reduced angle is rounded to fp32 (<= 2^-24 of a half turn,
1.9e-7 rad), sine and cosine to 2 units (2.4e-7), two fp32 products and a sum
(1.8e-7); together 6.1e-7 of |x1| + |x2|.
"""
import math

import numpy as np
import pytest
import torch

import sparse_linear_hybrid_b200 as sl

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def turned(x, freq, sections, interleaved, scale, pos, sign=1.0):
    """fp64 [B, N, heads, d] and the bound's |x1| + |x2|; pos [B, N, axes]."""
    x = x.double().cpu().numpy()
    f = freq.cpu().numpy()
    rot = 2 * len(f)
    axis = np.repeat(np.arange(len(sections)), sections)
    angle = sign * pos[:, :, axis].astype(np.float64) * f
    c, s = (scale * g(angle)[:, :, None] for g in (np.cos, np.sin))
    i1, i2 = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved else (np.arange(rot // 2), np.arange(rot // 2, rot))
    y, size = x.copy(), np.zeros_like(x)
    a, b = x[..., i1], x[..., i2]
    y[..., i1], y[..., i2] = a * c - b * s, b * c + a * s
    size[..., i1] = size[..., i2] = scale * (np.abs(a) + np.abs(b))
    return y, size


def check(got, ref, size):
    err = np.abs(got.double().cpu().numpy() - ref)
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 0.0   # fp16 steps below 2^-14 have one size
    lim = HALF_STEP[got.dtype] * (np.abs(ref) + 1e-6 * size) + 1e-6 * size + tiny
    worst = float(np.max(err - lim))
    assert worst <= 0, worst


def grid_positions(T, H, W, origin=(0, 0, 0)):
    g = np.stack(np.meshgrid(np.arange(T), np.arange(H), np.arange(W), indexing="ij"), -1).reshape(-1, 3)
    return (g + np.asarray(origin))[None]


CASES = [
    # B, N, heads of q and k, d, rot, interleaved, type, output type
    (1, 1, 1, 1, 64, 64, False, torch.bfloat16, torch.bfloat16),
    (3, 1, 12, 4, 128, 64, True, torch.bfloat16, torch.bfloat16),
    (2, 333, 5, 3, 128, 128, False, torch.float32, torch.float32),
    (2, 77, 3, 3, 64, 48, True, torch.float32, torch.bfloat16),
    (1, 129, 40, 40, 128, 128, True, torch.float16, torch.float16),
    (2, 50, 3, 2, 80, 34, False, torch.bfloat16, torch.bfloat16),   # the narrow path
    (1, 9, 2, 1, 7, 6, True, torch.float16, torch.float32),
    (1, 3, 2, 2, 512, 512, False, torch.bfloat16, torch.float16),
    (1, 2, 1, 1, 2, 2, False, torch.float32, torch.float32),
]


@pytest.mark.parametrize("B,N,hq,hk,d,rot,inter,kind,to", CASES)
@pytest.mark.parametrize("inverse", [False, True])
def test_positions(B, N, hq, hk, d, rot, inter, kind, to, inverse):
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k = (torch.randn(B, N, h, d, generator=g, device="cuda").to(kind) for h in (hq, hk))
    freq, scale = sl.rope_inv_freq(rot, scaling="yarn", factor=4.0, original_length=4096)
    pos = torch.randint(-2 ** 31, 2 ** 31, (B, N), generator=g, device="cuda").to(torch.int32)
    pos[0, 0] = 2 ** 31 - 1
    fn = sl.rope_backward if inverse else sl.rope_forward
    got = fn(q, k, freq, interleaved=inter, scale=scale, positions=pos, out_dtype=to)
    at = pos.cpu().numpy()[..., None]
    for x, y in zip((q, k), got):
        assert y.dtype == to
        # far positions: p f is rounded to fp64 (2^-53 of an angle up to 2^31: 2.4e-7 rad, and as much again
        # for the half turns), on both sides of the comparison
        ref, size = turned(x, freq, [rot // 2], inter, scale, at, -1.0 if inverse else 1.0)
        check(y, ref, 2 * size)
    # q alone gives the same
    assert torch.equal(fn(q, None, freq, interleaved=inter, scale=scale, positions=pos, out_dtype=to)[0], got[0])


@pytest.mark.parametrize("grid,sections,inter,origin", [
    ((3, 9, 13), (22, 21, 21), True, (0, 0, 0)), ((1, 1, 1), (0, 32, 32), False, (5, -2, 7)),
    ((5, 2, 31), (10, 44, 10), False, (100, 3, 0))])
def test_grid_of_a_fused_projection(grid, sections, inter, origin):
    """q and k as views of one [B, N, 3, heads, d] tensor, turned into new tensors and in place."""
    N, d, h = math.prod(grid), 128, 3
    g = torch.Generator(device="cuda").manual_seed(6)
    qkv = torch.randn(2, N, 3, h, d, generator=g, device="cuda").bfloat16()
    before = qkv.clone()
    freq, scale = sl.rope_inv_freq(d, sections=sections)
    q, k = qkv[:, :, 0], qkv[:, :, 1]
    kw = dict(sections=sections, interleaved=inter, scale=scale, grid=grid, origin=origin)
    got = sl.rope_forward(q, k, freq, **kw)
    pos = np.repeat(grid_positions(*grid, origin), 2, 0)
    for x, y in zip((q, k), got):
        check(y, *turned(x, freq, sections, inter, scale, pos))
    # explicit positions, shared by the sequences, give the same
    p = torch.from_numpy(pos[0].astype(np.int32)).cuda()
    same = sl.rope_forward(q, k, freq, sections=sections, interleaved=inter, scale=scale, positions=p)
    assert torch.equal(same[0], got[0]) and torch.equal(same[1], got[1])
    sl.rope_forward(q, k, freq, q_out=q, k_out=k, **kw)
    assert torch.equal(qkv[:, :, 0], got[0]) and torch.equal(qkv[:, :, 1], got[1])
    assert torch.equal(qkv[:, :, 2], before[:, :, 2])


def test_default_positions_and_head_major_strides():
    d, N = 64, 37
    x = torch.randn(2, 4, N, d, device="cuda")               # [B, heads, N, d]
    freq, _ = sl.rope_inv_freq(d)
    y = torch.full_like(x, math.nan)
    sl.rope_forward(x.transpose(1, 2), None, freq, origin=(11, 0, 0), q_out=y.transpose(1, 2))
    pos = np.tile((np.arange(N) + 11)[None, :, None], (2, 1, 1))
    check(y.transpose(1, 2), *turned(x.transpose(1, 2), freq, [d // 2], False, 1.0, pos))


def test_gradient():
    """The backward is the forward's transpose (against differences: the map is linear) and turns it back."""
    d = 64
    freq, scale = sl.rope_inv_freq(32, scaling="yarn", factor=8.0, original_length=2048)
    x, dy = torch.randn(1, 21, 2, d, device="cuda"), torch.randn(1, 21, 2, d, device="cuda")
    kw = dict(interleaved=True, scale=scale)
    dx = sl.rope_backward(dy, None, freq, **kw)[0]
    step = torch.randn_like(x)
    there = (sl.rope_forward(x + step, None, freq, **kw)[0].double() - sl.rope_forward(x - step, None, freq, **kw)[0].double()) / 2
    # 2,688 products of size 1 with errors of 1e-6 each, adding up like a random walk: 5e-5; bound four times that
    assert abs(float((there * dy.double()).sum() - (dx.double() * step.double()).sum())) <= 2e-4
    back = sl.rope_backward(sl.rope_forward(x, None, freq, **kw)[0], None, freq, **kw)[0]
    back[..., :32] /= scale ** 2
    assert float((back - x).abs().max()) <= 1e-5


def test_infinities_stay_in_their_pair():
    d = 64
    freq, _ = sl.rope_inv_freq(32)
    x = torch.randn(1, 4, 1, d, device="cuda").bfloat16()
    x[0, 2, 0, 3], x[0, 2, 0, 40] = math.nan, math.inf
    y = sl.rope_forward(x, None, freq)[0]
    bad = ~torch.isfinite(y)
    assert bad.nonzero().tolist() == [[0, 2, 0, 3], [0, 2, 0, 19], [0, 2, 0, 40]]


def test_stream_and_graph():
    """A captured call replays on new values; a call on another stream than the current one."""
    d = 128
    freq, _ = sl.rope_inv_freq(d)
    x = torch.randn(1, 300, 4, d, device="cuda").bfloat16()
    y = torch.empty_like(x)
    sl.rope_forward(x, None, freq, q_out=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sl.rope_forward(x, None, freq, q_out=y)
    x.normal_()
    graph.replay()
    want = sl.rope_forward(x, None, freq)[0]
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y.zero_()
    side.wait_stream(torch.cuda.current_stream())
    sl.rope_forward(x, None, freq, q_out=y, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
