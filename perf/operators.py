"""Operators around the attention layer, measured: rotary positions, 8-bit activation checkpoints, differential attention.

Each case is one call (or one forward and backward) as a training or sampling program makes it.
"own" selects the framework's calls; otherwise the same mathematics runs in elementary torch operations.
"""
import functools
import math

import numpy as np
import torch

own = False

BLOCK = 128          # tokens of a mask block
GROUP = 32           # values that share a scale in an 8-bit checkpoint
LOG2_MAX = {"int8": (127.0, 6), "e4m3": (448.0, 8)}  # largest code, exponent of its leading bit


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one streamed token of four sequences at far positions, half the head rotated, frequencies stretched for a long context
        dict(name="rope token", op="rope", B=4, N=1, heads=12, d=128, rot=64, sections="32", interleaved=False, kind="bfloat16",
             to="bfloat16", inverse=False, grid="", far=1000000, stretch=8.0),
        # q and k of the 1.3B video layer: 21 x 30 x 52 latent grid, three position axes, pairs side by side
        dict(name="rope video 1.3B", op="rope", B=1, N=32760, heads=12, d=128, rot=128, sections="22,21,21", interleaved=True,
             kind="bfloat16", to="bfloat16", inverse=False, grid="21,30,52", far=0, stretch=1.0),
        # fp32 gradients of the 14B video layer's q and k taken back through the rotation, stored as bf16
        dict(name="rope gradient 14B", op="rope", B=1, N=75600, heads=40, d=128, rot=128, sections="22,21,21", interleaved=True,
             kind="float32", to="bfloat16", inverse=True, grid="21,45,80", far=0, stretch=1.0),
        # 8-bit copy of a small activation and back
        dict(name="checkpoint small", op="ckpt", rows=351, cols=128, parts=1, fmt="int8", kind="bfloat16"),
        # q, k and v of the 1.3B layer, taken out of the fused projection's output, kept in 8 bits and read back
        dict(name="checkpoint qkv 1.3B", op="ckpt", rows=32760, cols=1536, parts=3, fmt="e4m3", kind="bfloat16"),
        # the layer's gradients from an 8-bit checkpoint on a six-frame clip
        dict(name="backward from 8 bits", op="ckpt_backward", B=1, T=6, H=30, W=52, heads=4, d=128, window="1,10,13", fmt="int8"),
        # two frames of a small grid: latency
        dict(name="differential small", op="diff", B=1, T=4, H=8, W=8, heads=2, d=64, window="1,4,4", random_rows=0, train=False),
        # the 1.3B layer's grid and window at 90 % block sparsity, no gradients kept
        dict(name="differential 1.3B", op="diff", B=1, T=21, H=30, W=52, heads=12, d=128, window="1,10,13", random_rows=0, train=False),
        # forward and backward of a ragged batch with its own mask for each head, some rows empty
        dict(name="differential step ragged", op="diff", B=2, T=3, H=9, W=39, heads=3, d=64, window="0,0,0", random_rows=3, train=True),
        # forward and backward of a six-frame clip
        dict(name="differential step", op="diff", B=1, T=6, H=30, W=52, heads=12, d=128, window="1,10,13", random_rows=0, train=True),
        # one token against short caches of different lengths, one of them empty
        dict(name="differential token short", op="diff_decode", B=3, Nq=1, cap=517, heads=12, d=64, empty=True),
        # one token against a cache as long as the video layer's sequence
        dict(name="differential token long", op="diff_decode", B=4, Nq=1, cap=32760, heads=12, d=128, empty=False),
    ]


def text(numbers):
    return ",".join(str(n) for n in numbers)


def ints(text):
    return [int(n) for n in text.split(",") if n]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "ckpt", "ckpt_backward", "diff", "diff", "diff_decode"])
    d = rng.choice([64, 128])
    if op == "rope":
        axes = rng.choice([1, 1, 3])
        rot = d if rng.random() < 0.6 else rng.choice([d // 2, d // 4 * 3, d // 2 + 4])
        a = rot // 2 // axes
        grid = [_log(rng, 1, 20), _log(rng, 1, 40), _log(rng, 1, 60)] if axes == 3 else []
        kind = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
        return dict(op=op, B=rng.randint(1, 3), N=math.prod(grid) if grid else _log(rng, 1, 30000), heads=rng.randint(1, 24), d=d, rot=rot,
                    sections=text([rot // 2 - (axes - 1) * a] + [a] * (axes - 1)), interleaved=rng.random() < 0.5, kind=kind,
                    to="bfloat16" if kind == "bfloat16" or rng.random() < 0.4 else kind, inverse=rng.random() < 0.5, grid=text(grid),
                    far=0 if grid else _log(rng, 1, 2000000), stretch=rng.choice([1.0, 1.0, 4.0, 32.0]))
    if op == "ckpt":
        return dict(op=op, rows=_log(rng, 1, 30000), cols=rng.choice([_log(rng, 1, 4000), 64 * _log(rng, 1, 40)]), parts=rng.randint(1, 3),
                    fmt=rng.choice(["int8", "e4m3"]), kind=rng.choice(["bfloat16", "bfloat16", "float16", "float32"]))
    if op == "ckpt_backward":
        return dict(op=op, B=rng.randint(1, 2), T=rng.randint(1, 4), H=_log(rng, 2, 24), W=_log(rng, 2, 40), heads=rng.randint(1, 4), d=d,
                    window=text([rng.randint(0, 2), rng.randint(1, 10), rng.randint(1, 12)]), fmt=rng.choice(["int8", "e4m3"]))
    if op == "diff":
        train = rng.random() < 0.5
        top = 30 if train else 40
        return dict(op=op, B=rng.randint(1, 2), T=rng.randint(1, 6 if train else 12), H=_log(rng, 1, top), W=_log(rng, 1, top),
                    heads=rng.randint(1, 8), d=d, window=text([rng.randint(0, 3), rng.randint(0, 12), rng.randint(0, 14)]),
                    random_rows=rng.choice([0, 0, 4]), train=train)
    return dict(op=op, B=rng.randint(1, 4), Nq=rng.choice([1, 1, 1, 2, 4]), cap=_log(rng, 1, 30000), heads=rng.randint(1, 16), d=d,
                empty=rng.random() < 0.3)


# ------------------------------------------------------------------ inputs

@functools.lru_cache(maxsize=32)
def window_blocks(T, H, W, window):
    """bool [nb, nb]: block pairs that hold a token pair within the window on every axis (raster order)."""
    wt, wh, ww = window
    n = T * H * W
    nb = -(-n // BLOCK)
    t, y, x = (a.reshape(-1) for a in np.meshgrid(np.arange(T), np.arange(H), np.arange(W), indexing="ij"))
    me, keep = np.arange(n) // BLOCK, np.zeros((nb, nb), dtype=bool)
    lo, hi = np.maximum(x - ww, 0), np.minimum(x + ww, W - 1)
    for dt in range(-min(wt, T - 1), min(wt, T - 1) + 1):
        for dy in range(-min(wh, H - 1), min(wh, H - 1) + 1):
            ok = (t + dt >= 0) & (t + dt < T) & (y + dy >= 0) & (y + dy < H)
            row = ((t + dt) * H + (y + dy)) * W
            a, b = ((row + lo)[ok]) // BLOCK, ((row + hi)[ok]) // BLOCK
            keep[me[ok], a] = True     # a run of at most 2 * 14 + 1 tokens meets at most two blocks
            keep[me[ok], b] = True
    return keep


def block_mask(case, seed):
    """bool [groups, nb, nb]: the same window for every head, or random rows per (batch, head) with some of them empty."""
    n = case["T"] * case["H"] * case["W"]
    nb = -(-n // BLOCK)
    if not case.get("random_rows"):
        return np.repeat(window_blocks(case["T"], case["H"], case["W"], tuple(ints(case["window"])))[None], case["heads"], 0)
    g = np.random.default_rng(seed + 17)
    keep = g.random((case["B"] * case["heads"], nb, nb)) < case["random_rows"] / nb
    keep[:, 2::5] = False
    return keep


def csr(keep, dev):
    rows = keep.reshape(-1, keep.shape[-1])
    ptr = np.concatenate([[0], np.cumsum(rows.sum(1))]).astype(np.int32)
    return torch.from_numpy(ptr).to(dev), torch.from_numpy(np.nonzero(rows)[1].astype(np.int32)).to(dev)


def frequencies(case):
    """fp64 frequencies of every pair: each axis has its own geometric series; `stretch` divides those of long wavelengths."""
    f = []
    for n in ints(case["sections"]):
        f += [10000.0 ** (-j / n) for j in range(n)]
    f = np.asarray(f)
    if case["stretch"] > 1:
        turns = 8192 * f / (2 * math.pi)
        part = np.clip((turns - 1) / 31, 0, 1)
        f = f / case["stretch"] * (1 - part) + f * part
    return f


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16, by=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * by).to(dtype)

    s = {"case": case}
    op = case["op"]
    if op == "rope":
        kind = getattr(torch, case["kind"])
        shape = (case["B"], case["N"], case["heads"], case["d"])
        s["q"], s["k"] = normal(*shape, dtype=kind), normal(*shape, dtype=kind)
        s["freq"] = torch.from_numpy(frequencies(case)).to(dev)
        s["scale"] = 0.1 * math.log(case["stretch"]) + 1.0
        s["positions"] = None
        if not case["grid"]:
            first = torch.randint(0, case["far"] + 1, (case["B"], 1), generator=g, device=dev)
            s["positions"] = (first + torch.arange(case["N"], device=dev)).to(torch.int32)
    elif op == "ckpt":
        wide = normal(case["rows"], case["parts"], case["cols"], dtype=getattr(torch, case["kind"]))
        heavy = torch.rand(case["cols"], generator=g, device=dev) < 0.01  # a few channels are much larger than the rest
        wide[..., heavy] *= 20
        wide[::7, 0, : min(GROUP, case["cols"])] = 0
        s["parts"] = [wide[:, i] for i in range(case["parts"])]
    elif op == "ckpt_backward":
        n = case["T"] * case["H"] * case["W"]
        shape = (case["B"], n, case["heads"], case["d"])
        s["q"], s["k"], s["v"], s["dout"] = normal(*shape), normal(*shape), normal(*shape), normal(*shape)
        s["w"] = normal(case["d"], case["d"], by=case["d"] ** -0.5)
        s["gate"] = torch.rand(case["B"], case["heads"], generator=g, device=dev)
        keep = block_mask(case, seed)
        s["row_ptr"], s["col_idx"] = csr(keep, dev)
        s["keep"] = torch.from_numpy(keep).to(dev)
        # the checkpoint that the forward pass left behind
        s["codes"] = [pack(s[x].reshape(-1, case["heads"] * case["d"]), case["fmt"]) for x in "qkv"]
    elif op == "diff":
        n = case["T"] * case["H"] * case["W"]
        shape = (case["B"], n, case["heads"], case["d"])
        s["q"], s["k"], s["v"] = normal(*shape), normal(*shape), normal(*shape)
        s["dout"] = normal(*shape) if case["train"] else None
        s["lam"] = (0.2 + 0.6 * torch.rand(case["heads"], generator=g, device=dev)).to(torch.bfloat16)
        keep = block_mask(case, seed)
        s["row_ptr"], s["col_idx"] = csr(keep, dev)
        s["t_row_ptr"], s["t_col_idx"] = csr(np.ascontiguousarray(keep.transpose(0, 2, 1)), dev)
        s["keep"] = torch.from_numpy(keep).to(dev)
    else:
        cache = (case["B"], case["cap"], case["heads"], case["d"])
        s["q"] = normal(case["B"], case["Nq"], case["heads"], case["d"])
        s["k"], s["v"] = normal(*cache), normal(*cache)
        s["lam"] = (0.2 + 0.6 * torch.rand(case["heads"], generator=g, device=dev)).to(torch.bfloat16)
        s["lens"] = lengths(case, seed).to(dev)
    return s


def lengths(case, seed):
    g = np.random.default_rng(seed + 29)
    n = g.integers(max(1, case["cap"] * 3 // 4), case["cap"] + 1, case["B"]).astype(np.int32)
    n[0] = 0 if case["empty"] else case["cap"]
    return torch.from_numpy(n)


# ------------------------------------------------------------------ plain forms

def coordinates(case, positions, dev):
    """[B or 1, N, axes] positions."""
    if positions is not None:
        return positions[..., None]
    T, H, W = ints(case["grid"])
    n = torch.arange(case["N"], device=dev)
    return torch.stack([n // (H * W), n // W % H, n % W], -1)[None]


def rotate(case, x, cos, sin):
    """x [B, N, heads, d] rotated, in fp32; cos and sin [B or 1, N, 1, rot / 2]."""
    y = x.float()
    a, b = pairs(case, y)
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], -1).flatten(-2) if case["interleaved"] else torch.cat([ra, rb], -1)
    return torch.cat([turned, y[..., case["rot"]:]], -1).to(getattr(torch, case["to"]))


def pairs(case, y):
    r = y[..., :case["rot"]]
    return (r[..., 0::2], r[..., 1::2]) if case["interleaved"] else r.chunk(2, -1)


def turns(s):
    """cos and sin of every token's angles, formed in 64 bits and rounded to 32 (angles of far positions need them)."""
    case = s["case"]
    axis = torch.repeat_interleave(torch.arange(len(ints(case["sections"])), device=s["freq"].device),
                                   torch.tensor(ints(case["sections"]), device=s["freq"].device))
    angle = coordinates(case, s["positions"], s["freq"].device)[..., axis].double() * s["freq"]
    if case["inverse"]:
        angle = -angle
    return ((s["scale"] * f(angle)).float()[:, :, None] for f in (torch.cos, torch.sin))


def power(e):
    """2^e in fp32 for whole e in [-127, 127], exact."""
    return ((e.clamp_min(-126) + 127) << 23).to(torch.int32).view(torch.float32) * torch.where(e < -126, 0.5, 1.0)


def pack(x, fmt):
    """Codes and the exponents' bytes (exponent + 127) of a [rows, cols] activation, groups of 32 along cols."""
    top, lead = LOG2_MAX[fmt]
    rows, cols = x.shape
    groups = -(-cols // GROUP)
    v = torch.nn.functional.pad(x.float(), (0, groups * GROUP - cols)).view(rows, groups, GROUP)
    amax = v.abs().amax(-1)
    e = torch.frexp(amax).exponent - 1 - lead
    e = e + (amax * power((-e).clamp(-127, 127)) > top)
    e = torch.where(amax == 0, torch.full_like(e, -127), e).clamp(-127, 127)
    scaled = (v * power(-e[..., None])).reshape(rows, -1)[:, :cols]
    codes = scaled.round().to(torch.int8) if fmt == "int8" else scaled.to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), (e + 127).to(torch.uint8)


def unpack(codes, scales, fmt, dtype):
    values = codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).float()
    e = scales.int().repeat_interleave(GROUP, -1)[:, :codes.shape[1]] - 127
    return (values * power(e)).to(dtype)


def kept_blocks(keep):
    """For one head: [nb, m] kept key blocks of each row (padded with block 0) and which of them are real."""
    m = max(1, int(keep.sum(-1).max()))
    order = torch.argsort((~keep).to(torch.int8), dim=-1, stable=True)[:, :m]
    return order, torch.gather(keep, 1, order)


def blocks_of(x):
    """[N, w] as [nb, 128, w] with zero rows behind the last token, in fp32."""
    nb = -(-x.shape[0] // BLOCK)
    return torch.nn.functional.pad(x.float(), (0, 0, 0, nb * BLOCK - x.shape[0])).view(nb, BLOCK, -1)


def real_keys(idx, real, n):
    """bool [nb, 1, m * 128]: the keys of the kept blocks that are tokens."""
    at = idx[..., None] * BLOCK + torch.arange(BLOCK, device=idx.device)
    return ((at < n) & real[..., None]).flatten(1)[:, None]


def softmax_of(scores, seen):
    """Probabilities over the seen keys; a row that sees none is zero."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    return p / p.sum(-1, keepdim=True).clamp_min(1e-30)


def scattered(blocks, idx, n):
    """Sums [nb, m * 128, w] contributions of the gathered key blocks into [N, w]."""
    nb, w = idx.shape[0], blocks.shape[-1]
    total = torch.zeros(nb, BLOCK, w, device=blocks.device)
    total.index_add_(0, idx.reshape(-1), blocks.view(-1, BLOCK, w))
    return total.view(-1, w)[:n]


def diff_head(q, k, v, dout, lam, keep):
    """One head of differential attention: out, or (out, dq, dk, dv, dlam) with dout, in fp32."""
    n, d = q.shape
    tau = (d // 2) ** -0.5
    idx, real = kept_blocks(keep)
    seen = real_keys(idx, real, n)
    qb = blocks_of(q)
    kg, vg = (blocks_of(x)[idx].flatten(1, 2) for x in (k, v))
    q1, q2 = qb.chunk(2, -1)
    k1, k2 = kg.chunk(2, -1)
    p1 = softmax_of(tau * q1 @ k1.mT, seen)
    p2 = softmax_of(tau * q2 @ k2.mT, seen)
    a = p1 - lam * p2
    out = (a @ vg).flatten(0, 1)[:n]
    if dout is None:
        return out
    db = blocks_of(dout)
    dp = db @ vg.mT
    d2 = (p2 * dp).sum(-1, keepdim=True)
    ds1 = tau * p1 * (dp - (p1 * dp).sum(-1, keepdim=True))
    ds2 = -lam * tau * p2 * (dp - d2)
    dq = torch.cat([ds1 @ k1, ds2 @ k2], -1).flatten(0, 1)[:n]
    dk = scattered(torch.cat([ds1.mT @ q1, ds2.mT @ q2], -1), idx, n)
    return out, dq, dk, scattered(a.mT @ db, idx, n), -d2.sum()


def layer_head(q, k, v, dout, w, gate, keep):
    """One head of the layer's backward, in fp32: dq, dk, dv, dw, dgate."""
    n, d = q.shape
    tau, eps = d ** -0.5, 1e-6
    idx, real = kept_blocks(keep)
    seen = real_keys(idx, real, n)
    qb, db = blocks_of(q), blocks_of(dout)
    kg, vg = (blocks_of(x)[idx].flatten(1, 2) for x in (k, v))
    p = softmax_of(tau * qb @ kg.mT, seen)
    dp = db @ vg.mT
    ds = tau * p * (dp - (p * dp).sum(-1, keepdim=True))
    dq = (ds @ kg).flatten(0, 1)[:n]
    dk = scattered(ds.mT @ qb, idx, n)
    dv = scattered(p.mT @ db, idx, n)
    q, k, v, dout, w = q.float(), k.float(), v.float(), dout.float(), w.float()
    a, r = q.relu(), k.relu()
    S, z = r.mT @ v, r.sum(0)
    den = (a @ z + eps)[:, None]
    o = a @ S / den
    y = o @ w
    do = gate * dout @ w.mT
    du = do / den
    dden = -(do * o).sum(-1, keepdim=True) / den
    dS, dz = a.mT @ du, (dden * a).sum(0)
    dq = dq + (q > 0) * (du @ S.mT + dden * z)
    dk = dk + (k > 0) * (v @ dS.mT + dz)
    return dq, dk, dv + r @ dS, o.mT @ (gate * dout), (dout * y).sum()


def by_head(keep, B, heads):
    """(b, h, mask row group) of every head of a batch; masks are per head or per (b, h)."""
    return [(b, h, b * heads + h if keep.shape[0] == B * heads and B > 1 else h) for b in range(B) for h in range(heads)]


def joined(parts, B, heads):
    """A list over (b, h) of [N, d] as bf16 [B, N, heads, d]."""
    x = torch.stack(list(parts))
    return x.view(B, heads, *x.shape[1:]).transpose(1, 2).to(torch.bfloat16).contiguous()


def plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "rope":
        cos, sin = turns(s)
        return rotate(case, s["q"], cos, sin), rotate(case, s["k"], cos, sin)
    if op == "ckpt":
        codes = [pack(x, case["fmt"]) for x in s["parts"]]
        return [(unpack(c, e, case["fmt"], x.dtype), e) for (c, e), x in zip(codes, s["parts"])]
    if op == "ckpt_backward":
        B, heads = case["B"], case["heads"]
        q, k, v = (unpack(c, e, case["fmt"], torch.bfloat16).view(s["q"].shape) for c, e in s["codes"])
        got = list(zip(*(layer_head(q[b, :, h], k[b, :, h], v[b, :, h], s["dout"][b, :, h], s["w"], s["gate"][b, h], s["keep"][g])
                         for b, h, g in by_head(s["keep"], B, heads))))
        return {"dq": joined(got[0], B, heads), "dk": joined(got[1], B, heads), "dv": joined(got[2], B, heads),
                "dw": torch.stack(got[3]).sum(0), "dgate": torch.stack(got[4]).view(B, heads)}
    if op == "diff":
        B, heads = case["B"], case["heads"]
        got = [diff_head(s["q"][b, :, h], s["k"][b, :, h], s["v"][b, :, h], s["dout"][b, :, h] if case["train"] else None,
                         s["lam"][h].float(), s["keep"][g]) for b, h, g in by_head(s["keep"], B, heads)]
        if not case["train"]:
            return {"out": joined(got, B, heads)}
        got = list(zip(*got))
        return {"out": joined(got[0], B, heads), "dq": joined(got[1], B, heads), "dk": joined(got[2], B, heads),
                "dv": joined(got[3], B, heads), "dlam": torch.stack(got[4]).view(B, heads).sum(0).to(s["lam"].dtype)}
    return diff_rows(s, torch.float32).to(torch.bfloat16)


def diff_rows(s, dtype):
    """A few query rows against the first lens[b] keys of each cache."""
    q, k, v = (s[x].to(dtype).transpose(1, 2) for x in "qkv")
    tau = (q.shape[-1] // 2) ** -0.5
    seen = (torch.arange(k.shape[2], device=k.device) < s["lens"][:, None])[:, None, None]
    (q1, q2), (k1, k2) = q.chunk(2, -1), k.chunk(2, -1)
    a = softmax_of(tau * q1 @ k1.mT, seen) - s["lam"].to(dtype)[:, None, None] * softmax_of(tau * q2 @ k2.mT, seen)
    return (a @ v).transpose(1, 2).contiguous()


# ------------------------------------------------------------------ the framework's calls

def kernels(s):
    import sparse_linear_hybrid_b200 as sl

    case, op = s["case"], s["case"]["op"]
    if op == "rope":
        call = sl.rope_backward if case["inverse"] else sl.rope_forward
        return call(s["q"], s["k"], s["freq"], sections=ints(case["sections"]), interleaved=case["interleaved"], scale=s["scale"],
                    positions=s["positions"], grid=ints(case["grid"]) or None, out_dtype=getattr(torch, case["to"]))
    if op == "ckpt":
        kept = sl.ckpt_pack(s["parts"], fmt=case["fmt"])
        return [(x, c.scales) for x, c in zip(sl.ckpt_unpack(kept), kept)]
    if op == "ckpt_backward":
        B, heads = case["B"], case["heads"]
        if "kept" not in s:
            s["kept"] = sl.ckpt_pack([s["q"], s["k"], s["v"]], fmt=case["fmt"])
            s["ws"] = sl.new_ckpt_backward_workspace(B, s["q"].shape[1], heads, case["d"])
        return sl.attn_backward_ckpt(*s["kept"], s["dout"], s["row_ptr"], s["col_idx"], s["w"], s["gate"], workspace=s["ws"])
    if op == "diff":
        per_bh = bool(case["random_rows"])
        if "ws" not in s:
            s["ws"] = sl.new_diff_workspace(case["B"], s["q"].shape[1], case["heads"], case["d"])
        args = (s["q"], s["k"], s["v"])
        mask = (s["row_ptr"], s["col_idx"])
        if not case["train"]:
            return {"out": sl.diff_attn_forward(*args, *mask, s["lam"], mask_per_bh=per_bh, workspace=s["ws"])}
        out, out2, lse = sl.diff_attn_forward_lse(*args, *mask, s["lam"], mask_per_bh=per_bh, workspace=s["ws"])
        grads = sl.diff_attn_backward(*args, out, out2, s["dout"], lse, *mask, s["lam"], t_row_ptr=s["t_row_ptr"],
                                      t_col_idx=s["t_col_idx"], mask_per_bh=per_bh, workspace=s["ws"])
        return {"out": out, **grads}
    return sl.diff_attn_decode(s["q"], s["k"], s["v"], s["lens"], s["lam"])


def run(s):
    return kernels(s) if own else plain(s)


# ------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    size = {"bfloat16": 2, "float16": 2, "float32": 4}
    if op == "rope":
        n = 2 * case["B"] * case["N"] * case["heads"] * case["d"]
        return {"bytes": n * (size[case["kind"]] + size[case["to"]]) + 4 * case["rot"], "flops": 3 * n * case["rot"] / case["d"]}
    if op == "ckpt":
        n = case["rows"] * case["cols"] * case["parts"]
        kept = n + case["rows"] * case["parts"] * -(-case["cols"] // GROUP)
        return {"bytes": 2 * (n * size[case["kind"]] + kept), "flops": 4 * n}
    if op == "diff_decode":
        live = int(lengths(case, 0).sum())
        row = case["heads"] * case["d"]
        return {"bytes": 2 * live * row * 2 + 2 * case["B"] * case["Nq"] * row * 2, "flops": 6 * live * row * case["Nq"]}
    n = case["T"] * case["H"] * case["W"]
    elements = case["B"] * n * case["heads"] * case["d"]
    keep = block_mask(case, 0)
    tokens = np.minimum(BLOCK, n - np.arange(keep.shape[-1]) * BLOCK)
    kept = float((keep * tokens[:, None] * tokens[None, :]).sum()) * (1 if case.get("random_rows") else case["B"])
    if op == "ckpt_backward":
        linear = 10 * elements * case["d"]
        return {"bytes": elements * (3 * (1 + 1 / GROUP) + 2 + 3 * 2), "flops": kept * 14 * case["d"] + linear}
    forward = {"bytes": elements * 8, "flops": kept * 6 * case["d"]}
    if not case["train"]:
        return forward
    return {"bytes": forward["bytes"] + elements * (2 + 6), "flops": forward["flops"] + kept * 10 * case["d"]}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        at = coordinates(case, s["positions"], s["freq"].device).double()
        made = []
        for x in (s["q"], s["k"]):
            y, first = x.double(), 0
            a, b = pairs(case, y)
            z = torch.zeros_like(y)
            z[..., case["rot"]:] = y[..., case["rot"]:]
            for axis, m in enumerate(ints(case["sections"])):
                part = slice(first, first + m)
                w = torch.polar(torch.full((), s["scale"], dtype=torch.float64, device=y.device),
                                (at[:, :, axis, None] * s["freq"][part] * (-1 if case["inverse"] else 1)))[:, :, None]
                turned = torch.complex(a[..., part], b[..., part]) * w
                i = torch.arange(first, first + m, device=y.device)
                z[..., 2 * i if case["interleaved"] else i] = turned.real
                z[..., 2 * i + 1 if case["interleaved"] else i + case["rot"] // 2] = turned.imag
                first += m
            made.append(z)
        return tuple(made)
    if op == "ckpt":
        return [(nearest(x.double(), case["fmt"]), None) for x in s["parts"]]
    if op == "diff_decode":
        made = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(s["lens"].tolist()):
            if n:
                h = case["d"] // 2
                q, k, v = s["q"][b].double(), s["k"][b, :n].double(), s["v"][b, :n].double()
                p = [torch.softmax(torch.einsum("ihc,jhc->hij", q[..., c], k[..., c]) / math.sqrt(h), -1) for c in (slice(0, h), slice(h, None))]
                made[b] = torch.einsum("hij,jhc->ihc", p[0] - s["lam"].double()[:, None, None] * p[1], v)
        return made
    B, heads, n = case["B"], case["heads"], s["q"].shape[1]
    grads = op == "ckpt_backward" or case["train"]
    source = {x: s[x].double() for x in "qkv"}
    if op == "ckpt_backward":
        source = {x: nearest(s[x].double().flatten(2).flatten(0, 1), case["fmt"]).view(s[x].shape) for x in "qkv"}
    got = {x: torch.zeros(B, n, heads, case["d"], dtype=torch.float64, device="cuda") for x in ("out", "dq", "dk", "dv")}
    w = s["w"].double().requires_grad_(True) if op == "ckpt_backward" else None
    dw, dgate = torch.zeros((), dtype=torch.float64, device="cuda"), torch.zeros(B, heads, dtype=torch.float64, device="cuda")
    step = n if grads else 2048
    block = torch.arange(n, device="cuda") // BLOCK
    for b, h, g in by_head(s["keep"], B, heads):
        q, k, v = (source[x][b, :, h].clone().requires_grad_(grads) for x in "qkv")
        scalar = (s["gate"][b, h] if op == "ckpt_backward" else s["lam"][h]).double().requires_grad_(grads)
        for at in range(0, n, step):
            mine = slice(at, min(at + step, n))
            seen = s["keep"][g][block[mine]][:, block]
            none = ~seen.any(-1, keepdim=True)

            def map_of(x, y, t):
                z = (x @ y.T * t).masked_fill(~(seen | none), -math.inf)
                return torch.softmax(z, -1).masked_fill(none, 0.0)

            if op == "ckpt_backward":
                out = map_of(q[mine], k, case["d"] ** -0.5) @ v
                a = q[mine].relu()
                out = out + scalar * ((a @ (k.relu().T @ v)) / (a @ k.relu().sum(0) + 1e-6)[:, None]) @ w
            else:
                c = case["d"] // 2
                out = (map_of(q[mine, :c], k[:, :c], c ** -0.5) - scalar * map_of(q[mine, c:], k[:, c:], c ** -0.5)) @ v
            got["out"][b, mine, h] = out.detach()
        if grads:
            leaves = [q, k, v, scalar] + ([w] if w is not None else [])
            d = torch.autograd.grad(out, leaves, s["dout"][b, :, h].double())
            for x, y in zip(("dq", "dk", "dv"), d):
                got[x][b, :, h] = y
            dgate[b, h] = d[3]
            dw = dw + d[4] if w is not None else dw
    if op == "ckpt_backward":
        return {"dq": got["dq"], "dk": got["dk"], "dv": got["dv"], "dw": dw, "dgate": dgate}
    if not case["train"]:
        return {"out": got["out"]}
    return {**got, "dlam": dgate.sum(0)}


def nearest(x, fmt):
    """What a group's 8-bit codes stand for, from the definition: the smallest power of two that holds the group, nearest codes, ties to even."""
    rows, cols = x.shape
    made = torch.empty_like(x)
    top = LOG2_MAX[fmt][0]
    for c in range(0, cols, GROUP):
        part = x[:, c:c + GROUP]
        m, e = torch.frexp(part.abs().amax(-1, keepdim=True) / top)  # the ratio is m 2^e with m in [1/2, 1)
        unit = torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e).clamp(-127, 127))
        y = part / unit
        grid = torch.ones_like(y) if fmt == "int8" else torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
        made[:, c:c + GROUP] = torch.round(y / grid) * grid * unit
    return made
