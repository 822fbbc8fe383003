"""Differential attention, rotary positions and 8-bit checkpoints at the 1.3B video
layer's size (32,760 tokens, 12 heads of 128), at sampled places against 64 bits.
The bounds are those of test_gpu_diff and test_gpu_rope."""
import numpy as np
import pytest
import torch

import sparse_linear_hybrid_b200 as sl
from test_gpu_ckpt import definition, rounded
from test_gpu_diff import decode_reference, rows_ok
from test_gpu_rope import check as check_rope
from test_gpu_rope import grid_positions, turned

pytestmark = pytest.mark.gpu

GRID, HEADS = (21, 30, 52), 12
N = 21 * 30 * 52


def normal(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


@pytest.mark.parametrize("d", [64, 128])
def test_differential_attention(d):
    q, k, v, dout = (normal(100 + i, 1, N, HEADS, d) for i in range(4))
    lam = torch.linspace(0.2, 0.8, HEADS, device="cuda")
    rp, ci = sl.build_block_mask(*GRID, 128, np.tile(np.int32([1, 10, 13]), (HEADS, 1)))
    ws = sl.new_diff_workspace(1, N, HEADS, d)
    out, out2, lse = sl.diff_attn_forward_lse(q, k, v, rp, ci, lam, workspace=ws)
    got = sl.diff_attn_backward(q, k, v, out, out2, dout, lse, rp, ci, lam, t_row_ptr=rp, t_col_idx=ci, workspace=ws)
    assert sl.check_status(ws) == sl.SALAD_OK
    nb = -(-N // 128)
    keep = torch.zeros(nb, nb, dtype=torch.bool, device="cuda")
    ptr, col = rp.cpu().numpy(), ci.cpu().numpy()
    for r in range(nb):
        keep[r, torch.from_numpy(col[ptr[r]:ptr[r + 1]]).cuda().long()] = True
    block = torch.arange(N, device="cuda") // 128
    rows = torch.cat([torch.arange(0, N, 499, device="cuda"), torch.tensor([127, 128, N - 1], device="cuda")])
    c, scale = d // 2, (d // 2) ** -0.5
    for h in (0, HEADS - 1):
        Q, K, V, G, lh = *(x[0, :, h].double() for x in (q, k, v, dout)), float(lam[h])

        def maps(at):
            seen = keep[block[at]][:, block]
            return [torch.softmax((Q[at, s] @ K[:, s].T * scale).masked_fill(~seen, -torch.inf), -1) for s in (slice(0, c), slice(c, d))]

        p1, p2 = maps(rows)
        ref, size = (p1 - lh * p2) @ V, (p1 + lh * p2) @ V.abs()
        assert bool(((out[0, rows, h].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2 * 2.0 ** -8 + 2e-4) * size).all())
        dp = G[rows] @ V.T
        ds = [p1 * (dp - (p1 * dp).sum(-1, keepdim=True)), -lh * p2 * (dp - (p2 * dp).sum(-1, keepdim=True))]
        rows_ok(got["dq"][0, rows, h], scale * torch.cat([ds[0] @ K[:, :c], ds[1] @ K[:, c:]], -1), "dq")
        dk, dv = torch.zeros(len(rows), d, dtype=torch.float64, device="cuda"), torch.zeros(len(rows), d, dtype=torch.float64, device="cuda")
        dlam = size = 0.0
        for first in range(0, N, 2048):
            at = torch.arange(first, min(first + 2048, N), device="cuda")
            p1, p2 = maps(at)
            dp = G[at] @ V.T
            d1, d2 = (p1 * dp).sum(-1, keepdim=True), (p2 * dp).sum(-1, keepdim=True)
            dlam, size = dlam - float(d2.sum()), size + float((p2 * dp.abs()).sum())
            p1, p2, dp = p1[:, rows], p2[:, rows], dp[:, rows]
            dk[:, :c] += scale * (p1 * (dp - d1)).T @ Q[at, :c]
            dk[:, c:] -= lh * scale * (p2 * (dp - d2)).T @ Q[at, c:]
            dv += (p1 - lh * p2).T @ G[at]
        rows_ok(got["dk"][0, rows, h], dk, "dk")
        rows_ok(got["dv"][0, rows, h], dv, "dv")
        assert abs(float(got["dlam"][h]) - dlam) <= 2.0 ** -24 * abs(dlam) + 1e-4 * size


def test_decode():
    q, k, v = normal(110, 2, 1, HEADS, 128), normal(111, 2, N, HEADS, 128), normal(112, 2, N, HEADS, 128)
    lam, lens = torch.linspace(0.2, 0.8, HEADS, device="cuda"), [N, N - 5001]
    out = sl.diff_attn_decode(q, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), lam)
    ref, size = decode_reference(q, k, v, lens, lam)
    assert bool(((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-5 * size).all())


def test_a_cache_of_more_than_2_to_the_32_bytes():
    """Keys behind 2^32 bytes (and 2^31 elements) of one sequence's cache."""
    cap, Hh, d = 1_500_000, 12, 128
    assert cap * Hh * d > 2 ** 31
    k, v = (torch.zeros(1, cap, Hh, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, tail = normal(120, 1, 1, Hh, d), 333
    k[:, :cap - tail, :, 0], k[:, :cap - tail, :, 64] = -200.0, -200.0
    k[:, cap - tail:], v[:, cap - tail:] = normal(121, 1, tail, Hh, d), normal(122, 1, tail, Hh, d)
    q[..., 0], q[..., 64] = 20.0, 20.0  # (the others score -500: nothing in fp32 or bf16 is left of them)
    lam = torch.linspace(0.2, 0.8, Hh, device="cuda")
    out = sl.diff_attn_decode(q, k, v, torch.tensor([cap], dtype=torch.int32, device="cuda"), lam)
    ref, size = decode_reference(q, k[:, cap - tail:], v[:, cap - tail:], [tail], lam)
    assert bool(((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-5 * size).all())


def test_rotary_positions():
    sections, d = (22, 21, 21), 128
    freq, scale = sl.rope_inv_freq(d, sections=sections)
    q, k = normal(130, 1, N, HEADS, d), normal(131, 1, N, HEADS, d)
    got = sl.rope_forward(q, k, freq, sections=sections, interleaved=True, scale=scale, grid=GRID)
    rows = torch.cat([torch.arange(0, N, 97, device="cuda"), torch.tensor([N - 1], device="cuda")])
    pos = grid_positions(*GRID)[:, rows.cpu().numpy()]
    for x, y in zip((q, k), got):
        check_rope(y[:, rows], *turned(x[:, rows], freq, sections, True, scale, pos))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_checkpoints(fmt):
    x = normal(140, N, HEADS * 128)
    c = sl.ckpt_pack(x, fmt=fmt)
    rows = torch.arange(0, N, 211, device="cuda")
    byte, val = definition(x[rows], fmt)
    assert np.array_equal(c.scales[rows].cpu().numpy(), byte)
    assert torch.equal(sl.ckpt_unpack(c)[rows].cpu(), rounded(val, torch.bfloat16))
