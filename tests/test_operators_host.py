"""Host-only checks of rotary positions, 8-bit checkpoints and differential
attention (no GPU needed): the frequencies of rope_inv_freq, and bad arguments
refused with the documented status before anything is launched (the pointers are
never dereferenced)."""
import ctypes
import math
import struct

import numpy as np
import pytest
import torch

import sparse_linear_hybrid_b200 as sl

FAKE = 0x100000


@pytest.fixture(scope="module")
def L():
    from sparse_linear_hybrid_b200 import build
    build.build()
    return sl.lib()


def rope(L, tensors=None, count=None, **kw):
    a = dict(x_type=1, y_type=1, B=1, N=8, d=64, rot=64, inter=0, freq=FAKE, pairs=(32,), axes=None, pos=None, pos_b=0,
             gh=1, gw=1, origin=None, scale=1.0, inverse=0)
    a.update(kw)
    row = a["d"] * 2
    if tensors is None:
        tensors = [dict(x=0x10000000, y=0x20000000, heads=2, xs=(8 * row, row, a["d"]), ys=(8 * row, row, a["d"]))]
    packed = b"".join(struct.pack("PPi4x6q", t["x"], t["y"], t["heads"], *t["xs"], *t["ys"]) for t in tensors)
    pairs = struct.pack("%di" % len(a["pairs"]), *a["pairs"])
    return L.salad_rope(packed, len(tensors) if count is None else count, a["x_type"], a["y_type"], a["B"], a["N"], a["d"],
                        a["rot"], a["inter"], a["freq"], pairs, len(a["pairs"]) if a["axes"] is None else a["axes"], a["pos"],
                        a["pos_b"], a["gh"], a["gw"], a["origin"], a["scale"], a["inverse"], None)


def view(x, y, heads=2, n=8, d=64, sn=None, sb=None):
    sn = heads * d if sn is None else sn
    sb = n * sn if sb is None else sb
    return dict(x=x, y=y, heads=heads, xs=(sb, sn, d), ys=(sb, sn, d))


def test_rope_refusals(L):
    bad = sl.SALAD_ERR_INVALID_ARG
    for kw in (dict(x_type=3), dict(y_type=-1), dict(B=0), dict(N=0), dict(rot=0), dict(rot=7, pairs=(3,)), dict(rot=66, pairs=(33,)),
               dict(freq=None), dict(freq=FAKE + 4), dict(pairs=(31,)), dict(pairs=(33, -1)), dict(axes=0),
               dict(pairs=(8, 8, 8, 8)), dict(pos=FAKE + 2), dict(pos=FAKE, pos_b=-1), dict(gh=0), dict(gw=0),
               dict(scale=math.inf), dict(scale=math.nan), dict(count=0), dict(count=3), dict(d=0)):
        assert rope(L, **kw) == bad, kw
    assert rope(L, d=514, rot=64) == sl.SALAD_ERR_UNSUPPORTED
    assert rope(L, B=1 << 16, N=1 << 15) == sl.SALAD_ERR_UNSUPPORTED
    for t in (view(0, 0x20000000), view(0x10000000, 0), view(0x10000001, 0x20000000), view(0x10000000, 0x20000000, heads=0),
              dict(x=0x10000000, y=0x20000000, heads=2, xs=(1024, -1, 64), ys=(1024, 128, 64)),
              dict(x=0x10000000, y=0x20000000, heads=2, xs=(1024, 128, 64), ys=(1024, 128, 32)),    # heads of y overlap
              dict(x=0x10000000, y=0x20000000, heads=2, xs=(1024, 128, 64), ys=(1024, 0, 64)),      # all tokens in one place
              view(0x10000000, 0x10000000 + 128),                                                   # y inside x, not x itself
              dict(x=0x10000000, y=0x10000000, heads=2, xs=(1024, 128, 64), ys=(1024, 256, 64))):   # the same start, other strides
        assert rope(L, [t]) == bad, t
    # q and k: outputs that overlap, and each other's inputs
    assert rope(L, [view(0x10000000, 0x20000000), view(0x30000000, 0x20000000)]) == bad
    assert rope(L, [view(0x10000000, 0x30000000), view(0x30000000, 0x20000000)]) == bad
    # side by side in one tensor, but reaching into each other
    assert rope(L, [view(0x10000000, 0x10000000, sn=384), view(0x10000000 + 128, 0x10000000 + 128, sn=384)]) == bad
    assert rope(L, [view(0x10000000, 0x20000000, sn=384), view(0x10000000 + 256, 0x20000000 + 640, sn=384)]) == bad


def test_rope_positions_stay_within_int32(L):
    for origin in ((2 ** 31 - 7, 0, 0), (0, 2 ** 31 - 1, 0), (0, 0, 2 ** 31 - 1)):
        assert rope(L, origin=struct.pack("3i", *origin)) == sl.SALAD_ERR_INVALID_ARG


def ckpt(L, fn="salad_ckpt_pack", tensors=None, rows=4, cols=64, type_=1, fmt=0, count=None):
    tensors = tensors or [(0x10000000, cols, 0x20000000, 0x30000000)]
    packed = b"".join(struct.pack("PqPP", *t) for t in tensors)
    return getattr(L, fn)(packed, len(tensors) if count is None else count, rows, cols, type_, fmt, None)


@pytest.mark.parametrize("fn", ["salad_ckpt_pack", "salad_ckpt_unpack"])
def test_checkpoint_refusals(L, fn):
    bad = sl.SALAD_ERR_INVALID_ARG
    for kw in (dict(rows=0), dict(cols=0), dict(type_=4), dict(fmt=2), dict(count=0), dict(count=5),
               dict(tensors=[(0, 64, 0x20000000, 0x30000000)]), dict(tensors=[(0x10000000, 64, 0, 0x30000000)]),
               dict(tensors=[(0x10000000, 64, 0x20000000, 0)]), dict(tensors=[(0x10000001, 64, 0x20000000, 0x30000000)]),
               dict(tensors=[(0x10000000, 63, 0x20000000, 0x30000000)]),                        # rows overlap
               dict(tensors=[(0x10000000, 64, 0x10000000 + 100, 0x30000000)]),                  # codes inside the values
               dict(tensors=[(0x10000000, 64, 0x20000000, 0x20000000 + 8)]),                    # scales inside the codes
               dict(tensors=[(0x10000000, 64, 0x20000000, 0x30000000), (0x11000000, 64, 0x20000000, 0x31000000)])):
        if fn == "salad_ckpt_unpack" and len(kw.get("tensors", [])) == 2:
            kw = dict(tensors=[(0x10000000, 64, 0x20000000, 0x30000000), (0x10000000, 64, 0x21000000, 0x31000000)])
        if fn == "salad_ckpt_unpack" and kw.get("tensors", [(0,) * 4])[0][3] == 0x20000000 + 8:
            continue  # both are only read
        assert ckpt(L, fn, **kw) == bad, kw
    assert ckpt(L, fn, rows=1 << 30, cols=64) == sl.SALAD_ERR_UNSUPPORTED


def test_checkpoint_backward_refusals(L):
    size = L.salad_ckpt_backward_workspace_bytes(1, 256, 2, 64)
    assert size > L.salad_layer_backward_workspace_bytes(1, 256, 2, 64) + 256 * 2 * 64 * (4 * 2 + 3 * 4) and size % 256 == 0
    assert L.salad_ckpt_backward_workspace_bytes(1, 256, 2, 96) == 0 and L.salad_ckpt_backward_workspace_bytes(0, 1, 1, 64) == 0

    def call(**kw):
        a = dict(qc=0x1000000, qs=0x2000000, kc=0x3000000, ks=0x4000000, vc=0x5000000, vs=0x6000000, fmt=0, dout=0x7000000, B=1,
                 N=256, H=2, d=64, block=128, rp=FAKE, w=FAKE, gate=FAKE, scale=0.0, eps=1e-6, dq=0x8000000, dk=0x9000000,
                 dv=0xA000000, dw=FAKE, ws=0x40000000, bytes=1 << 34)
        a.update(kw)
        return L.salad_attn_backward_ckpt(a["qc"], a["qs"], a["kc"], a["ks"], a["vc"], a["vs"], a["fmt"], a["dout"], a["B"],
                                          a["N"], a["H"], a["d"], a["block"], a["rp"], FAKE, FAKE, FAKE, 0, a["w"], a["gate"],
                                          a["scale"], a["eps"], a["dq"], a["dk"], a["dv"], a["dw"], FAKE, a["ws"], a["bytes"], None)
    bad = sl.SALAD_ERR_INVALID_ARG
    for kw in (dict(qc=None), dict(vs=None), dict(kc=0x3000008), dict(fmt=2), dict(dout=None), dict(rp=None), dict(w=FAKE + 8),
               dict(eps=-1.0), dict(scale=math.nan), dict(dq=None), dict(dq=0x8000008), dict(dk=0x8000000), dict(dv=0x5000000),
               dict(ws=0x40000010), dict(B=0)):
        assert call(**kw) == bad, kw
    for kw in (dict(d=96), dict(block=64), dict(B=40000), dict(H=40000, B=2)):
        assert call(**kw) == sl.SALAD_ERR_UNSUPPORTED, kw
    assert call(bytes=size - 1) == sl.SALAD_ERR_WORKSPACE


def test_differential_refusals(L):
    size = L.salad_diff_workspace_bytes(1, 300, 2, 64)
    assert size == 256 + 2 * 4 * 384 * 4 + 256 and L.salad_diff_workspace_bytes(1, 300, 2, 32) == 0
    bad = sl.SALAD_ERR_INVALID_ARG

    def forward(**kw):
        a = dict(q=0x1000000, k=0x2000000, v=0x3000000, B=1, N=300, H=2, d=64, block=128, rp=FAKE, ci=FAKE, lam=FAKE, lt=1, scale=0.0,
                 out=0x4000000, out2=None, lse=None, ws=0x40000000, bytes=1 << 30)
        a.update(kw)
        return L.salad_diff_forward(a["q"], a["k"], a["v"], a["B"], a["N"], a["H"], a["d"], a["block"], a["rp"], a["ci"], 0,
                                    a["lam"], a["lt"], a["scale"], a["out"], a["out2"], a["lse"], a["ws"], a["bytes"], None)
    for kw in (dict(q=None), dict(k=0x2000008), dict(out=0x1000000), dict(out2=0x5000000), dict(lse=FAKE), dict(lam=None),
               dict(lt=2), dict(lam=FAKE + 1), dict(scale=math.inf), dict(ws=None), dict(ws=0x40000010), dict(B=0), dict(N=0),
               dict(rp=None), dict(ci=None), dict(out2=0x4000000, lse=0x6000000), dict(out2=0x5000000, lse=0x4000000)):
        assert forward(**kw) == bad, kw
    for kw in (dict(d=32), dict(block=64), dict(H=70000), dict(N=(1 << 30) + 1), dict(B=1 << 20, H=1000)):
        assert forward(**kw) == sl.SALAD_ERR_UNSUPPORTED, kw
    assert forward(bytes=size - 1) == sl.SALAD_ERR_WORKSPACE

    def backward(**kw):
        a = dict(out2=0x5000000, dout=0x6000000, lse=0x7000000, trp=FAKE, dq=0x8000000, dk=0x9000000, dv=0xA000000, dlam=FAKE,
                 block=128, bytes=1 << 30, lt=0)
        a.update(kw)
        return L.salad_diff_backward(0x1000000, 0x2000000, 0x3000000, 0x4000000, a["out2"], a["dout"], a["lse"], 1, 300, 2, 64,
                                     a["block"], FAKE, FAKE, a["trp"], FAKE, 0, FAKE, a["lt"], 0.0, a["dq"], a["dk"], a["dv"],
                                     a["dlam"], 0x40000000, a["bytes"], None)
    for kw in (dict(out2=None), dict(dout=None), dict(lse=None), dict(trp=None), dict(dq=0x1000000), dict(dk=0x8000000),
               dict(dv=0x4000000), dict(dlam=None), dict(dlam=FAKE + 2), dict(dq=0x8000004), dict(lt=3)):
        assert backward(**kw) == bad, kw
    assert backward(block=64) == sl.SALAD_ERR_UNSUPPORTED and backward(bytes=300) == sl.SALAD_ERR_WORKSPACE

    def decode(**kw):
        a = dict(q=0x1000000, k=0x2000000, v=0x3000000, B=2, Nq=1, cap=100, H=2, d=64, lens=FAKE, lam=FAKE, lt=0, scale=0.0, out=0x4000000)
        a.update(kw)
        return L.salad_diff_decode(a["q"], a["k"], a["v"], a["B"], a["Nq"], a["cap"], a["H"], a["d"], a["lens"], a["lam"], a["lt"],
                                   a["scale"], a["out"], None)
    for kw in (dict(q=None), dict(v=0x3000004), dict(lens=None), dict(lens=FAKE + 1), dict(lam=FAKE + 2), dict(out=0x2000000),
               dict(Nq=0), dict(cap=0), dict(scale=math.nan), dict(lt=2)):
        assert decode(**kw) == bad, kw
    for kw in (dict(d=96), dict(Nq=140000), dict(B=1 << 20, H=1 << 10), dict(cap=(1 << 30) + 1)):
        assert decode(**kw) == sl.SALAD_ERR_UNSUPPORTED, kw


def test_frequencies():
    f, scale = sl.rope_inv_freq(64, base=1000.0, device="cpu")
    assert f.dtype == torch.float64 and scale == 1.0
    # base^(-j/32), each rounded a few times: 2^-50 covers power and exponent
    assert np.allclose(f.numpy(), [1000.0 ** (-j / 32) for j in range(32)], rtol=2.0 ** -48, atol=0)
    f, _ = sl.rope_inv_freq(128, sections=(22, 21, 21), device="cpu")
    assert f.numel() == 64 and f[0] == f[22] == f[43] == 1.0 and abs(f[23] - 10000.0 ** (-1 / 21)) < 1e-12
    g, _ = sl.rope_inv_freq(64, base=1000.0, scaling="linear", factor=4.0, device="cpu")
    assert np.allclose(g.numpy() * 4, [1000.0 ** (-j / 32) for j in range(32)], rtol=2.0 ** -48, atol=0)
    g, _ = sl.rope_inv_freq(64, base=1000.0, scaling="ntk", factor=4.0, device="cpu")
    assert g[0] == 1.0 and abs(g[31] / f.new_tensor(1000.0 ** (-31 / 32) / 4) - 1) < 1e-12      # the slowest is divided by 4
    y, scale = sl.rope_inv_freq(64, scaling="yarn", factor=8.0, original_length=2048, device="cpu")
    p = np.array([10000.0 ** (-j / 32) for j in range(32)])
    turns = 2048 * p / (2 * math.pi)
    assert scale == 0.1 * math.log(8.0) + 1.0
    assert np.allclose(y.numpy()[turns > 32], p[turns > 32], rtol=1e-14) and np.allclose(y.numpy()[turns < 1], p[turns < 1] / 8, rtol=1e-14)
    between = (turns < 32) & (turns > 1)
    assert np.all((y.numpy() < p)[between]) and np.all((y.numpy() > p / 8)[between])
    for kw in (dict(rot=5), dict(rot=0), dict(rot=8, sections=(3,)), dict(rot=8, sections=(5, -1)), dict(rot=8, scaling="no"),
               dict(rot=8, base=0.0), dict(rot=8, factor=0.5), dict(rot=8, scaling="yarn", factor=2.0),
               dict(rot=8, scaling="yarn", factor=2.0, original_length=64, beta_fast=1.0, beta_slow=2.0)):
        with pytest.raises(ValueError):
            sl.rope_inv_freq(device="cpu", **kw)


def test_the_bindings_take_cuda_tensors_only():
    x = torch.zeros(1, 128, 1, 64, dtype=torch.bfloat16)
    f = torch.zeros(32, dtype=torch.float64)
    idx = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: sl.rope_forward(x, x, f), lambda: sl.rope_backward(x, None, f), lambda: sl.ckpt_pack(x),
                 lambda: sl.ckpt_unpack(sl.Checkpoint(x.to(torch.uint8), x.to(torch.uint8), "int8", torch.bfloat16)),
                 lambda: sl.diff_attn_forward(x, x, x, idx, idx, torch.zeros(1)),
                 lambda: sl.diff_attn_forward_lse(x, x, x, idx, idx, torch.zeros(1)),
                 lambda: sl.diff_attn_backward(x, x, x, x, x, x, torch.zeros(2, 1, 1, 128), idx, idx, torch.zeros(1)),
                 lambda: sl.diff_attn_decode(x, x, x, idx, torch.zeros(1))):
        with pytest.raises(TypeError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="format"):
        sl.ckpt_pack(x, fmt="int4")
