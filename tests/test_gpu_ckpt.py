"""8-bit activation checkpoints on the GPU: codes and scale bytes equal to the
definition's (every step is exact, so nothing is tolerated), the layer's backward
from them against the oracle's at the decoded values, and a training step that
rotates q and k, keeps 8-bit q, k, v and goes back through both."""
import numpy as np
import pytest
import torch

import oracle
import salad_inputs as si
import sparse_linear_hybrid_b200 as sl
from parity import to_dev
from test_gpu_backward import check_elements

pytestmark = pytest.mark.gpu

LARGEST = {"int8": 127.0, "e4m3": 448.0}
FINITE = {torch.float32: 3.4028234663852886e38, torch.bfloat16: 3.3895313892515355e38, torch.float16: 65504.0}


def definition(x, fmt):
    """Scale bytes and decoded values (fp64) of a [rows, cols] tensor, group by group."""
    x = x.double().cpu().numpy()
    rows, cols = x.shape
    G = (cols + 31) // 32
    byte, val = np.zeros((rows, G), np.uint8), np.zeros((rows, cols))
    for g in range(G):
        part = x[:, 32 * g:32 * g + 32]
        bad = ~np.isfinite(part).all(1)
        amax = np.where(bad, 0, np.abs(np.where(np.isfinite(part), part, 0)).max(1))
        m, e = np.frexp(amax / LARGEST[fmt])
        e = np.clip(np.where(m == 0.5, e - 1, e), -127, 127)
        e = np.where(amax == 0, -127, e)
        y = part / np.ldexp(1.0, e)[:, None]
        with np.errstate(all="ignore"):
            if fmt == "int8":
                code = np.rint(y)
            else:
                unit = np.ldexp(1.0, np.maximum(np.frexp(y)[1] - 1, -6) - 3)
                code = np.rint(y / unit) * unit
        val[:, 32 * g:32 * g + 32] = np.where(bad[:, None], np.nan, code * np.ldexp(1.0, e)[:, None])
        byte[:, g] = np.where(bad, 255, e + 127)
    return byte, val


def rounded(val, kind):
    """fp64 values in a type, capped at its largest."""
    v = torch.from_numpy(np.clip(val, -FINITE[kind], FINITE[kind]))
    return v.to(kind)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 31), (5, 33), (1, 32), (70, 64), (351, 128), (33, 1536), (1000, 100)])
def test_codes(rows, cols, kind, fmt):
    g = torch.Generator(device="cuda").manual_seed(rows * 7 + cols)
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-6, 7, (rows, 1), generator=g, device="cuda"))
    x = x.to(kind)
    x[rows // 2, : min(cols, 32)] = 0
    c = sl.ckpt_pack(x, fmt=fmt)
    byte, val = definition(x, fmt)
    assert np.array_equal(c.scales.cpu().numpy(), byte)
    back = sl.ckpt_unpack(c)
    assert back.dtype == kind and torch.equal(back.cpu(), rounded(val, kind))
    assert torch.equal(sl.ckpt_unpack(c, dtype=torch.float32).double().cpu(), torch.from_numpy(val))
    # what was kept is kept again without a change
    again = sl.ckpt_pack(sl.ckpt_unpack(c, dtype=torch.float32), fmt=fmt)
    assert torch.equal(sl.ckpt_unpack(again, dtype=torch.float32), sl.ckpt_unpack(c, dtype=torch.float32))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("cols", [64, 40])
def test_edges(kind, fmt, cols):
    """Infinities and NaN, the largest and smallest magnitudes, ties, powers of two around the largest code."""
    tiny = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}[kind]
    x = torch.zeros(12, cols, dtype=torch.float64)
    x[0, 3], x[1, 5], x[2, cols - 1] = np.inf, -np.inf, np.nan
    x[3, :5] = torch.tensor([FINITE[kind], -FINITE[kind], 1.0, 0.5, 0.25])
    x[4, :4] = torch.tensor([tiny, -tiny, 3 * tiny, 0])
    x[5, :32] = torch.arange(32) * 4 + 1.5
    x[6, :8] = torch.tensor([127.0, 126.5, 0.5, 1.5, 2.5, -0.5, -1.5, -127.0])
    x[7, :8] = torch.tensor([127.5, 126.5, 0.5, 1.5, 2.5, -0.5, -1.5, -127.0])
    x[8, :6] = torch.tensor([448.0, 432.0, 26.0, 27.0, 2.0 ** -10, 3 * 2.0 ** -11])
    x[9, :3] = torch.tensor([450.0, 1.0, 17.0])
    x[10] = -1.0
    x = x.to(kind).cuda()
    c = sl.ckpt_pack(x, fmt=fmt)
    byte, val = definition(x, fmt)
    assert np.array_equal(c.scales.cpu().numpy(), byte)
    back = sl.ckpt_unpack(c).cpu()
    want = rounded(val, kind)
    assert torch.equal(torch.isnan(back), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(back), torch.nan_to_num(want))


def test_views_of_a_fused_projection_and_of_an_output():
    qkv = torch.randn(2, 45, 3, 4, 64, device="cuda").bfloat16()
    parts = [qkv[:, :, i] for i in range(3)]
    kept = sl.ckpt_pack(parts, fmt="e4m3")
    for x, c in zip(parts, kept):
        assert c.codes.shape == x.shape and c.scales.shape == (2, 45, 4, 2)
        alone = sl.ckpt_pack(x.contiguous(), fmt="e4m3")
        assert torch.equal(alone.codes, c.codes) and torch.equal(alone.scales, c.scales)
    into = torch.full_like(qkv, 7.0)
    sl.ckpt_unpack(kept[:2], out=[into[:, :, 0], into[:, :, 2]])
    assert torch.equal(into[:, :, 0], sl.ckpt_unpack(kept[0])) and torch.equal(into[:, :, 2], sl.ckpt_unpack(kept[1]))
    assert bool((into[:, :, 1] == 7).all())
    # tensors of several layouts in one call, memory used again
    mixed = [torch.randn(5, 33, device="cuda"), torch.randn(64, device="cuda").half(), qkv]
    a = sl.ckpt_pack(mixed)
    for x, c in zip(mixed, a):
        one = sl.ckpt_pack(x)
        assert torch.equal(one.codes, c.codes) and torch.equal(one.scales, c.scales)
    assert sl.ckpt_pack(mixed[0] * 2, out=a[0]) is a[0]
    assert sl.ckpt_pack(torch.empty(0, 64, device="cuda")).codes.numel() == 0


def test_graph_replay():
    x = torch.randn(64, 256, device="cuda").bfloat16()
    c, y = sl.ckpt_pack(x), torch.empty_like(x)
    sl.ckpt_unpack(c, out=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sl.ckpt_unpack(sl.ckpt_pack(x, out=c), out=y)
    x.normal_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, sl.ckpt_unpack(sl.ckpt_pack(x)))


def check_rows(got, ref, name, floor):
    """The layer backward's own bound per row (relative 2e-2 plus 2e-3 of the RMS row, from
    the bf16 products) plus bf16's half step, 2^-8 of every value, plus `floor`: the part of
    a row that cancels.  ds_ij = p_ij (dout_i . v_j - D_i) with D_i = dout_i . out_i from the
    bf16 output, which is off by 2^-8 of each value at most, so |dD_i| <= 2^-8 |dout_i| |out_i|
    and a row of dq by scale sum_j p_ij |dD_i| |k_j| <= scale 2^-8 |dout_i| |out_i| max|k|
    (dk likewise with max|q| where one query holds all of the weight).  With a single token dq
    and dk are 0 and this is all that is left."""
    d = ref.shape[-1]
    rn, en = (np.linalg.norm(a.reshape(-1, d), axis=1) for a in (ref, got - ref))
    lim = (2e-2 + 2.0 ** -8) * rn + 2e-3 * np.sqrt(np.mean(rn ** 2)) + floor
    assert np.all(np.isfinite(got)) and np.all(en <= lim), (name, float(np.max(en / lim)))


@pytest.mark.parametrize("B,T,H,W,Hh,d,window,fmt", [
    (2, 3, 9, 13, 2, 128, (1, 3, 4), "int8"), (1, 2, 8, 16, 3, 64, (1, 2, 3), "e4m3"), (1, 1, 1, 1, 1, 64, (0, 0, 0), "int8")])
def test_backward(B, T, H, W, Hh, d, window, fmt):
    wl = si.Workload("ck", B=B, Hh=Hh, d=d, T=T, H=H, W=W, block=128, window=window, seed=91)
    inp = si.make_inputs(wl, v_mean=0.5)
    q, k, v, w = (to_dev(a) for a in (inp.q, inp.k, inp.v, inp.w_proj))
    gate = torch.from_numpy(inp.gate).cuda()
    rng = np.random.default_rng(92)
    dout_bits = si.f32_to_bf16_bits(rng.standard_normal(inp.q.shape, dtype=np.float32))
    rp, ci = sl.build_block_mask(T, H, W, 128, inp.windows)
    kept = sl.ckpt_pack([q, k, v], fmt=fmt)
    ws = sl.new_ckpt_backward_workspace(B, wl.N, Hh, d)
    got = sl.attn_backward_ckpt(*kept, to_dev(dout_bits), rp, ci, w, gate, workspace=ws)
    again = sl.attn_backward_ckpt(*kept, to_dev(dout_bits), rp, ci, w, gate, workspace=ws)
    assert sl.check_status(ws) == sl.SALAD_OK
    assert all(torch.equal(got[n], again[n]) for n in got)
    bits = [x.view(torch.int16).cpu().numpy().view(np.uint16) for x in sl.ckpt_unpack(kept)]
    orp, oci = oracle.block_mask(T, H, W, 128, inp.windows)
    ref = oracle.backward(*bits, 128, orp, oci, inp.w_proj, inp.gate, si.bf16_bits_to_f32(dout_bits).astype(np.float64))
    floor = 0.0
    if wl.N == 1:
        size = {x: float(torch.linalg.vector_norm(t.double(), dim=-1).max()) for x, t in zip("qkv", sl.ckpt_unpack(kept))}
        out = oracle.forward(*bits, 128, orp, oci, inp.w_proj, inp.gate)
        floor = d ** -0.5 * 2.0 ** -8 * np.linalg.norm(si.bf16_bits_to_f32(dout_bits)) * np.linalg.norm(out) * max(size["q"], size["k"])
    for name in ("dq", "dk", "dv"):
        assert got[name].dtype == torch.bfloat16
        check_rows(got[name].double().cpu().numpy(), ref[name], name, floor if name != "dv" else 0.0)
    for name in ("dw", "dgate"):
        check_elements(got[name].cpu().numpy().astype(np.float64), ref[name], name)


def test_training_step():
    """Fused projection -> rotation -> layer -> 8-bit q, k, v -> gradients -> rotation back, in a captured graph too."""
    B, T, H, W, Hh, d = 1, 3, 9, 13, 2, 128
    N, sections = T * H * W, (22, 21, 21)
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.randn(B, N, 3, Hh, d, generator=g, device="cuda").bfloat16()
    dout = torch.randn(B, N, Hh, d, generator=g, device="cuda").bfloat16()
    w = (torch.randn(d, d, generator=g, device="cuda") / d ** 0.5).bfloat16()
    gate = torch.rand(B, Hh, generator=g, device="cuda")
    freq, scale = sl.rope_inv_freq(d, sections=sections)
    kw = dict(sections=sections, interleaved=True, scale=scale, grid=(T, H, W))
    rp, ci = sl.build_block_mask(T, H, W, 128, np.tile(np.int32([1, 3, 4]), (Hh, 1)))
    ws, wsb = sl.new_workspace(B, N, Hh, d), sl.new_ckpt_backward_workspace(B, N, Hh, d)

    def step():
        q, k = sl.rope_forward(qkv[:, :, 0], qkv[:, :, 1], freq, **kw)
        v = qkv[:, :, 2].contiguous()
        out = sl.attn_forward(q, k, v, rp, ci, w, gate, 128, workspace=ws)
        kept = sl.ckpt_pack([q, k, v])
        grads = sl.attn_backward_ckpt(*kept, dout, rp, ci, w, gate, workspace=wsb)
        dq, dk = sl.rope_backward(grads["dq"], grads["dk"], freq, **kw)
        return out, dq, dk, grads["dv"], grads["dw"], kept

    first = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first[:5], captured[:5]))
    # the same from the parts: the bf16 gradients are attn_backward's rounded once
    q, k, v = sl.ckpt_unpack(first[5])
    out, lse = sl.attn_forward_lse(q, k, v, rp, ci, w, gate, 128)
    full = sl.attn_backward(q, k, v, out, dout, lse, rp, ci, w, gate)
    want = sl.rope_backward(full["dq"].bfloat16(), full["dk"].bfloat16(), freq, **kw)
    assert torch.equal(first[1], want[0]) and torch.equal(first[2], want[1])
    assert torch.equal(first[3], full["dv"].bfloat16()) and torch.equal(first[4], full["dw"])
