"""Differential attention on the GPU against its definition in 64 bits.

Forward, per element.  A weight enters the value product as bf16, off by 2^-8 of
itself at most, and the row sum adds the same rounded weights, so a map's output
is off by at most 2 2^-8 sum_j p_ij |v_j|; the output is rounded once, 2^-8 of
itself.  Scores, exponentials and sums in fp32 (and the cubic for one exponential
pair in four, 7.5e-5) add less than 2e-4 of the same sum.
  |got - ref| <= 2^-8 |ref| + (2 2^-8 + 2e-4) (sum_j p_1 |v| + |lam| sum_j p_2 |v|)

Gradients, per row, as for the layer's backward (whose products and roundings are
the same): ||got - ref|| <= 2e-2 ||row|| + 2e-3 RMS(rows) plus bf16's half step,
2^-8 ||row||.  Where a row cancels (one token, or maps so sharp that dp_ij is near
D_i wherever p_ij is not small) the errors of D are what is left.  D_m is formed
from the outputs, so |dD_2,i| <= sum_f |dout_f| e_2,f and |dD_1,i| <= sum_f |dout_f| e_f +
|lam| |dD_2,i| with e and e_2 the forward's bounds above; ds_m is off by p_m |dD_m|, a
row of dq by `floor` = scale sum_m c_m sum_j p_m,ij |dD_m,i| ||k_m,j|| (c = 1, |lam|) and
a row of dk by the same sum over i with ||q_m,i||.  Those cases add it.
dlam: its terms are fp32 products of fp32 sums, off by 1e-4 of their size (the
cubic), plus the half step of its type."""
import math

import numpy as np
import pytest
import torch

import sparse_linear_hybrid_b200 as sl

pytestmark = pytest.mark.gpu


def csr(keep):
    rows = keep.reshape(-1, keep.shape[-1])
    ptr = np.concatenate([[0], np.cumsum(rows.sum(1))]).astype(np.int32)
    return torch.from_numpy(ptr).cuda(), torch.from_numpy(np.nonzero(rows)[1].astype(np.int32)).cuda()


def make(B, N, Hh, d, keep, seed, spread=1.0, lam_type=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k, v, dout = (torch.randn(B, N, Hh, d, generator=g, device="cuda").bfloat16() for _ in range(4))
    q = (q * spread).bfloat16()
    lam = (torch.rand(Hh, generator=g, device="cuda") * 1.2 - 0.2).to(lam_type)
    return q, k, v, dout, lam, *csr(keep), *csr(np.ascontiguousarray(keep.transpose(0, 2, 1)))


def maps(q, k, keep, scale, b, h, per_bh, Hh):
    """The two maps of one head in 64 bits, zero rows where no key is kept."""
    n, d = q.shape[1], q.shape[3]
    block = torch.arange(n, device="cuda") // 128
    seen = torch.from_numpy(keep[b * Hh + h if per_bh else h]).cuda()[block][:, block]
    out = []
    for c in (slice(0, d // 2), slice(d // 2, d)):
        s = (q[b, :, h, c].double() @ k[b, :, h, c].double().T * scale).masked_fill(~seen, -math.inf)
        top = s.amax(-1, keepdim=True)
        e = torch.exp(s - torch.where(torch.isfinite(top), top, 0.0))
        out.append((e / e.sum(-1, keepdim=True).clamp_min(1e-300), torch.logsumexp(s, -1)))
    return out


def check_forward(q, k, v, keep, lam, got, out2, lse, per_bh, scale=None):
    B, N, Hh, d = q.shape
    scale = scale or (d // 2) ** -0.5
    for b in range(B):
        for h in range(Hh):
            (p1, s1), (p2, s2) = maps(q, k, keep, scale, b, h, per_bh, Hh)
            x, lh = v[b, :, h].double(), float(lam[h])
            ref, size = (p1 - lh * p2) @ x, (p1 + abs(lh) * p2) @ x.abs()
            lim = 2.0 ** -8 * ref.abs() + (2 * 2.0 ** -8 + 2e-4) * size
            err = (got[b, :, h].double() - ref).abs()
            assert bool((err <= lim).all()), float((err - lim).max())
            if out2 is not None:
                r2, z2 = p2 @ x, p2 @ x.abs()
                assert bool(((out2[b, :, h].double() - r2).abs() <= 2.0 ** -8 * r2.abs() + (2 * 2.0 ** -8 + 2e-4) * z2).all())
                for m, s in enumerate((s1, s2)):
                    mine = lse[m, b, h].double()
                    none = torch.isinf(s)
                    assert torch.equal(torch.isinf(mine), none)
                    # fp32 scores (up to 2^-20 of their size), the cubic's 7.5e-5, fp32 sums
                    assert bool(((mine - s)[~none].abs() <= 2e-4 + 2.0 ** -18 * s[~none].abs()).all())


def rows_ok(got, ref, name, floor=0.0):
    d = ref.shape[-1]
    rn, en = ref.reshape(-1, d).norm(dim=1), (got.double() - ref).reshape(-1, d).norm(dim=1)
    lim = (2e-2 + 2.0 ** -8) * rn + 2e-3 * rn.square().mean().sqrt() + floor
    assert bool(torch.isfinite(got).all()) and bool((en <= lim).all()), (name, float((en / lim).max()))


def reference_gradients(q, k, v, dout, keep, lam, per_bh):
    B, N, Hh, d = q.shape
    scale = (d // 2) ** -0.5
    dq, dk, dv = (torch.zeros(q.shape, dtype=torch.float64, device="cuda") for _ in range(3))
    fq, fk = (torch.zeros(q.shape[:3], dtype=torch.float64, device="cuda") for _ in range(2))
    dlam, size = torch.zeros(Hh, dtype=torch.float64, device="cuda"), torch.zeros(Hh, dtype=torch.float64, device="cuda")
    c = d // 2
    for b in range(B):
        for h in range(Hh):
            (p1, _), (p2, _) = maps(q, k, keep, scale, b, h, per_bh, Hh)
            x, g, lh = v[b, :, h].double(), dout[b, :, h].double(), lam[h].double()
            dp = g @ x.T
            ds1 = p1 * (dp - (p1 * dp).sum(-1, keepdim=True))
            ds2 = -lh * p2 * (dp - (p2 * dp).sum(-1, keepdim=True))
            qq, kk = q[b, :, h].double(), k[b, :, h].double()
            dq[b, :, h, :c], dq[b, :, h, c:] = scale * ds1 @ kk[:, :c], scale * ds2 @ kk[:, c:]
            dk[b, :, h, :c], dk[b, :, h, c:] = scale * ds1.T @ qq[:, :c], scale * ds2.T @ qq[:, c:]
            dv[b, :, h] = (p1 - lh * p2).T @ g
            dlam[h] -= (p2 * dp).sum()
            size[h] += (p2 * dp.abs()).sum()
            err = lambda ref, z: 2.0 ** -8 * ref.abs() + (2 * 2.0 ** -8 + 2e-4) * z  # noqa: E731
            d2 = (g.abs() * err(p2 @ x, p2 @ x.abs())).sum(-1)
            d1 = (g.abs() * err((p1 - lh * p2) @ x, (p1 + lh.abs() * p2) @ x.abs())).sum(-1) + lh.abs() * d2
            for p, dd, f, s in ((p1, d1, 1.0, slice(0, c)), (p2, d2, lh.abs(), slice(c, d))):
                fq[b, :, h] += scale * f * dd * (p @ kk[:, s].norm(dim=-1))
                fk[b, :, h] += scale * f * (p.T @ (dd * qq[:, s].norm(dim=-1)))
    return dq, dk, dv, dlam, size, fq.reshape(-1), fk.reshape(-1)


def random_keep(groups, nb, rate, seed, empty=True):
    keep = np.random.default_rng(seed).random((groups, nb, nb)) < rate
    if empty:
        keep[:, ::3] = False
        keep[:, :, ::4] = False
    return keep


CASES = [
    # B, N, heads, d, per_bh, rate, empty rows, spread, lam's type
    (1, 1, 1, 64, False, 1.1, False, 1.0, torch.bfloat16),
    (2, 1, 3, 128, True, 1.1, False, 1.0, torch.float32),
    (1, 127, 2, 128, False, 1.1, False, 1.0, torch.bfloat16),
    (1, 129, 2, 64, False, 1.1, False, 4.0, torch.float32),
    (2, 700, 3, 128, True, 0.5, True, 1.0, torch.bfloat16),
    (2, 1000, 2, 64, True, 0.4, True, 1.0, torch.bfloat16),
    (1, 1152, 2, 128, False, 0.6, True, 12.0, torch.float32),   # sharp maps: the running maximum moves
    (1, 2050, 1, 64, False, 1.1, False, 1.0, torch.bfloat16),
    (1, 300, 2, 64, True, -1.0, False, 1.0, torch.bfloat16),    # no block kept at all
]


@pytest.mark.parametrize("B,N,Hh,d,per_bh,rate,empty,spread,kind", CASES)
def test_forward_and_gradients(B, N, Hh, d, per_bh, rate, empty, spread, kind):
    nb = -(-N // 128)
    keep = random_keep(B * Hh if per_bh else Hh, nb, rate, N + d, empty)
    q, k, v, dout, lam, rp, ci, trp, tci = make(B, N, Hh, d, keep, N + Hh, spread, kind)
    ws = sl.new_diff_workspace(B, N, Hh, d)
    kw = dict(mask_per_bh=per_bh, workspace=ws)
    plain = sl.diff_attn_forward(q, k, v, rp, ci, lam, **kw)
    out, out2, lse = sl.diff_attn_forward_lse(q, k, v, rp, ci, lam, **kw)
    assert sl.check_status(ws) == sl.SALAD_OK
    assert torch.equal(plain, out)
    check_forward(q, k, v, keep, lam, out, out2, lse, per_bh)
    got = sl.diff_attn_backward(q, k, v, out, out2, dout, lse, rp, ci, lam, t_row_ptr=trp, t_col_idx=tci, **kw)
    assert sl.check_status(ws) == sl.SALAD_OK
    dq, dk, dv, dlam, size, fq, fk = reference_gradients(q, k, v, dout, keep, lam, per_bh)
    cancels = N == 1 or spread > 1
    rows_ok(got["dq"], dq, "dq", fq if cancels else 0.0)
    rows_ok(got["dk"], dk, "dk", fk if cancels else 0.0)
    rows_ok(got["dv"], dv, "dv")
    assert got["dlam"].dtype == kind
    half = 2.0 ** -8 if kind == torch.bfloat16 else 2.0 ** -24
    assert bool(((got["dlam"].double() - dlam).abs() <= half * dlam.abs() + 1e-4 * size).all()), (got["dlam"], dlam)
    again = sl.diff_attn_backward(q, k, v, out, out2, dout, lse, rp, ci, lam, t_row_ptr=trp, t_col_idx=tci, **kw)
    assert all(torch.equal(got[n], again[n]) for n in got)
    if per_bh:  # the transpose built on the GPU
        built = sl.diff_attn_backward(q, k, v, out, out2, dout, lse, rp, ci, lam, **kw)
        assert all(torch.equal(got[n], built[n]) for n in got)


def test_window_mask_and_scale():
    T, H, W, Hh, d = 3, 9, 39, 2, 128
    N = T * H * W
    win = np.int32([[1, 3, 4], [0, 2, 38]])
    rp, ci = sl.build_block_mask(T, H, W, 128, win)
    nb = -(-N // 128)
    keep = np.zeros((Hh * nb, nb), bool)
    ptr, col = rp.cpu().numpy(), ci.cpu().numpy()
    for r in range(Hh * nb):
        keep[r, col[ptr[r]:ptr[r + 1]]] = True
    keep = keep.reshape(Hh, nb, nb)
    q, k, v, dout, lam, *_ = make(1, N, Hh, d, keep, 8)
    out = sl.diff_attn_forward(q, k, v, rp, ci, lam, softmax_scale=0.31)
    check_forward(q, k, v, keep, lam, out, None, None, False, 0.31)
    # equal halves and lam 1: both maps form the same O and l, and out = fma(O, 1/l, -(O (1/l) rounded to fp32)) is
    # that product's rounding, 2^-24 of the map's output at most, which no value of v exceeds
    same = torch.cat([q[..., :64]] * 2, -1).contiguous(), torch.cat([k[..., :64]] * 2, -1).contiguous()
    gone = sl.diff_attn_forward(*same, v, rp, ci, torch.ones(Hh, device="cuda"))
    assert float(gone.abs().max()) <= 2.0 ** -24 * float(v.abs().max())
    # with lam 0 it is attention over the first halves alone
    zero = sl.diff_attn_forward(q, k, v, rp, ci, torch.zeros(Hh, device="cuda"))
    check_forward(q, k, v, keep, torch.zeros(Hh), zero, None, None, False)


def test_gradients_against_differences():
    """The forward in 64 bits moved along a direction, against the GPU's gradients."""
    B, N, Hh, d = 1, 260, 2, 64
    keep = random_keep(Hh, 3, 0.7, 4, empty=False)
    keep[:, np.arange(3), np.arange(3)] = True
    q, k, v, dout, lam, rp, ci, trp, tci = make(B, N, Hh, d, keep, 2, lam_type=torch.float32)
    out, out2, lse = sl.diff_attn_forward_lse(q, k, v, rp, ci, lam)
    got = sl.diff_attn_backward(q, k, v, out, out2, dout, lse, rp, ci, lam, t_row_ptr=trp, t_col_idx=tci)
    g = torch.Generator(device="cuda").manual_seed(9)

    def loss(x):
        total = 0.0
        for h in range(Hh):
            (p1, _), (p2, _) = maps(x["q"], x["k"], keep, (d // 2) ** -0.5, 0, h, False, Hh)
            total = total + float((((p1 - x["lam"][h] * p2) @ x["v"][0, :, h]) * dout[0, :, h].double()).sum())
        return total

    base = {"q": q.double(), "k": k.double(), "v": v.double(), "lam": lam.double()}
    for name in base:
        step = torch.randn(base[name].shape, generator=g, device="cuda", dtype=torch.float64)
        eps = 1e-5
        up, down = ({**base, name: base[name] + s * eps * step} for s in (1, -1))
        slope = (loss(up) - loss(down)) / (2 * eps)
        mine = got["d" + name].double()
        # a gradient's relative error (2e-2 per row by the bound above) against a random direction adds up
        # like a random walk: 2e-2 of the norm of the products
        lim = 2e-2 * float((mine * step).norm()) + 1e-4 * abs(slope)
        assert abs(slope - float((mine * step).sum())) <= lim, name


# Per head and map: step of 64 keys -> (level, which of its keys carry it); a level is 2 units of score (nats) in a row
# of amplitude 16.  One pair of keys in four has its exponential from the cubic: keys 6 and 7 of every 8.
LEAPS = [
    ({1: (31, "all")}, {}),
    ({}, {1: (30, "all"), 3: (70, "one"), 5: (178, "all"), 10: (200, "all")}),
    ({2: (45, "cubic")}, {4: (178, "cubic"), 6: (190, "cubic")}),
    ({10: (100, "cubic")}, {10: (250, "one")}),
]


@pytest.mark.parametrize("d", [64, 128])
def test_scores_far_above_the_first_keys(d):
    """Later keys whose scores pass the first keys' by up to 500 (2^721): in all keys of a step, in one, or only where the
    cubic forms the exponential; several times, in one map or both, in the short last tile.

    Scores of size S come from up to four matrix products, each off by 2^-23 of the largest term at most, and are stored
    in fp32: off by 8 2^-23 S, a weight by twice that of itself (its own score and the sum's)."""
    N, Hh = 680, len(LEAPS)
    nb, c, S = -(-N // 128), d // 2, 500.0
    keep = np.ones((Hh, nb, nb), bool)
    q, k, v, dout, lam, rp, ci, trp, tci = make(1, N, Hh, d, keep, 31, lam_type=torch.float32)
    scale = 0.125  # amplitude 16: a level is 2
    amp = torch.tensor([16.0, 8.0, 0.0, -16.0, 16.0], device="cuda")[torch.arange(N, device="cuda") % 5]
    for h, both in enumerate(LEAPS):
        for m, steps in enumerate(both):
            q[0, :, h, m * c] = amp.bfloat16()
            k[0, :, h, m * c] = 0
            for u, (level, which) in steps.items():
                j = torch.arange(64 * u, min(64 * u + 64, N), device="cuda")
                j = {"all": j, "one": j[5:6], "cubic": j[(j % 8) >= 6]}[which]
                k[0, j, h, m * c] = level
    kw = dict(softmax_scale=scale)
    out, out2, lse = sl.diff_attn_forward_lse(q, k, v, rp, ci, lam, **kw)
    more = 2 * 8 * 2.0 ** -23 * S
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    for h in range(Hh):
        (p1, s1), (p2, s2) = maps(q, k, keep, scale, 0, h, False, Hh)
        x, lh = v[0, :, h].double(), float(lam[h])
        for got, ref, size in ((out, (p1 - lh * p2) @ x, (p1 + abs(lh) * p2) @ x.abs()), (out2, p2 @ x, p2 @ x.abs())):
            lim = 2.0 ** -8 * ref.abs() + (2 * 2.0 ** -8 + 2e-4 + more) * size
            assert bool(((got[0, :, h].double() - ref).abs() <= lim).all()), h
        for m, s in enumerate((s1, s2)):
            assert bool(((lse[m, 0, h].double() - s).abs() <= 2e-4 + 2.0 ** -18 * s.abs()).all()), (h, m)
    assert torch.equal(out, sl.diff_attn_forward(q, k, v, rp, ci, lam, **kw))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [0, 6, 71, 130, 199])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_kept_key_without_a_value_shows(d, at, bad):
    """NaN or infinity in one kept key (where the cubic forms its exponential and where not, in the first step, a later
    one, the short last one) makes every row of that map NaN, as by the formula; the other head stays."""
    keep = np.ones((2, 2, 2), bool)
    q, k, v, _, lam, rp, ci, *_ = make(1, 200, 2, d, keep, 19)
    clean = sl.diff_attn_forward(q, k, v, rp, ci, lam)
    q[0, :, 0, 3] = 1.0  # (an infinite score is positive: its weight is inf / inf)
    k[0, at, 0, 3] = bad
    out, out2, lse = sl.diff_attn_forward_lse(q, k, v, rp, ci, lam)
    assert bool(torch.isnan(out[0, :, 0]).all())
    assert torch.equal(out[0, :, 1], clean[0, :, 1]) and bool(torch.isfinite(out2).all())
    if math.isnan(bad):
        assert bool(torch.isnan(lse[0, 0, 0]).all()) and bool(torch.isfinite(lse[1]).all())


def test_what_is_not_kept_is_not_read():
    """Infinities and NaN in blocks that no row keeps do not reach the output or the gradients."""
    N, d = 512, 128
    keep = np.zeros((1, 4, 4), bool)
    keep[0, 0, 0] = keep[0, 1, [0, 3]] = keep[0, 3, 3] = True
    keep[0, 1, 1] = True
    q, k, v, dout, lam, rp, ci, trp, tci = make(1, N, 1, d, keep, 12)
    clean = sl.diff_attn_forward_lse(q, k, v, rp, ci, lam)
    kn, vn = k.clone(), v.clone()
    kn[:, 256:384], vn[:, 256:384] = math.nan, math.inf
    dirty = sl.diff_attn_forward_lse(q, kn, vn, rp, ci, lam)
    assert all(torch.equal(a, b) for a, b in zip(clean, dirty))
    assert bool((clean[0][:, 256:384] == 0).all()) and bool(torch.isinf(clean[2][:, :, :, 256:384]).all())
    kw = dict(t_row_ptr=trp, t_col_idx=tci)
    a = sl.diff_attn_backward(q, k, v, clean[0], clean[1], dout, clean[2], rp, ci, lam, **kw)
    b = sl.diff_attn_backward(q, kn, vn, dirty[0], dirty[1], dout, dirty[2], rp, ci, lam, **kw)
    assert all(torch.equal(a[n], b[n]) for n in a)
    assert bool((a["dk"][:, 256:384] == 0).all()) and bool((a["dq"][:, 256:384] == 0).all())


def decode_reference(q, k, v, lens, lam):
    B, Nq, Hh, d = q.shape
    ref, size = (torch.zeros(q.shape, dtype=torch.float64, device="cuda") for _ in range(2))
    for b in range(B):
        n = min(max(int(lens[b]), 0), k.shape[1])
        if n:
            c = d // 2
            x = v[b, :n].double()
            p = [torch.softmax(torch.einsum("ihc,jhc->hij", q[b][..., s].double(), k[b, :n][..., s].double()) * c ** -0.5, -1)
                 for s in (slice(0, c), slice(c, d))]
            lh = lam.double()[:, None, None]
            ref[b] = torch.einsum("hij,jhc->ihc", p[0] - lh * p[1], x)
            size[b] = torch.einsum("hij,jhc->ihc", p[0] + lh.abs() * p[1], x.abs())
    return ref, size


@pytest.mark.parametrize("B,Nq,cap,Hh,d,lens", [
    (1, 1, 1, 1, 64, [1]), (1, 1, 5, 2, 128, [3]), (4, 1, 517, 3, 64, [0, 517, 1, 300]), (3, 2, 100, 5, 128, [-4, 200, 99]),
    (2, 3, 2000, 12, 128, [2000, 65]), (1, 7, 333, 1, 64, [333]), (1, 1, 20000, 1, 128, [19999]), (64, 1, 70, 8, 64, list(range(64)))])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_decode(B, Nq, cap, Hh, d, lens, kind):
    g = torch.Generator(device="cuda").manual_seed(cap)
    q = (torch.randn(B, Nq, Hh, d, generator=g, device="cuda") * 2).bfloat16()
    k, v = (torch.randn(B, cap, Hh, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    lam = (torch.rand(Hh, generator=g, device="cuda") - 0.2).to(kind)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for b, x in enumerate(lens):  # what lies behind a sequence is not read
        if max(x, 0) < cap:
            k[b, max(x, 0):], v[b, max(x, 0):] = math.nan, math.inf
    out = sl.diff_attn_decode(q, k, v, n, lam)
    ref, size = decode_reference(q, k, v, lens, lam)
    # fp32 throughout: sums of up to 20,000 terms and scores of size 30 leave 1e-5 of the weighted values; one rounding
    assert bool(((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-5 * size).all())
    assert torch.equal(out, sl.diff_attn_decode(q, k, v, n, lam))


def test_decode_follows_the_full_attention():
    """A sequence's tokens one by one against its own cache give the rows of the block form (one block: all see all)."""
    N, Hh, d = 100, 2, 128
    q, k, v, _, lam, rp, ci, *_ = make(1, N, Hh, d, np.ones((Hh, 1, 1), bool), 77)
    full = sl.diff_attn_forward(q, k, v, rp, ci, lam)
    lens = torch.tensor([N], dtype=torch.int32, device="cuda")
    for i in (0, 57, 99):
        one = sl.diff_attn_decode(q[:, i:i + 1].contiguous(), k, v, lens, lam)
        ref, size = decode_reference(q[:, i:i + 1], k, v, [N], lam)
        assert bool(((full[:, i:i + 1].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2 * 2.0 ** -8 + 2e-4) * size).all())
        assert bool(((one.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-5 * size).all())


def test_training_step_in_a_graph():
    """Rotation, differential attention, 8-bit q, k, v, gradients and rotation back: eager, captured and replayed on new
    inputs, beside another captured call with a workspace of its own."""
    B, T, H, W, Hh, d = 2, 2, 9, 13, 2, 64
    N = T * H * W
    g = torch.Generator(device="cuda").manual_seed(21)
    q0, k0, v, dout = (torch.randn(B, N, Hh, d, generator=g, device="cuda").bfloat16() for _ in range(4))
    lam = torch.tensor([0.3, 0.7], device="cuda")
    rp, ci = sl.build_block_mask(T, H, W, 128, np.tile(np.int32([1, 2, 3]), (Hh, 1)))
    sections = (12, 10, 10)
    freq, scale = sl.rope_inv_freq(d, sections=sections)
    kw = dict(sections=sections, interleaved=True, scale=scale, grid=(T, H, W))
    ws, other = sl.new_diff_workspace(B, N, Hh, d), sl.new_diff_workspace(B, N, Hh, d)

    def step():
        q, k = sl.rope_forward(q0, k0, freq, **kw)
        out, out2, lse = sl.diff_attn_forward_lse(q, k, v, rp, ci, lam, workspace=ws)
        kept = sl.ckpt_pack([q, k, v], fmt="int8")
        q8, k8, v8 = sl.ckpt_unpack(kept)
        grads = sl.diff_attn_backward(q8, k8, v8, out, out2, dout, lse, rp, ci, lam, workspace=ws)
        dq, dk = sl.rope_backward(grads["dq"], grads["dk"], freq, **kw)
        return out, dq, dk, grads["dv"], grads["dlam"]

    step()
    torch.cuda.synchronize()
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    with torch.cuda.graph(second):
        beside = sl.diff_attn_forward(q0, k0, v, rp, ci, lam, workspace=other)
    for t in (q0, k0, v, dout):
        t.normal_()
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second.replay()
    graph.replay()
    torch.cuda.synchronize()
    want = step()
    assert all(torch.equal(a, b) for a, b in zip(captured, want))
    assert torch.equal(beside, sl.diff_attn_forward(q0, k0, v, rp, ci, lam))
    assert sl.check_status(ws) == sl.SALAD_OK and sl.check_status(other) == sl.SALAD_OK


def test_what_a_call_allocates_is_of_its_stream():
    """A call on a stream that is still busy: its workspace, dropped when the call returns, may not be given to a tensor
    of the current stream, and its results are those of the current stream's call."""
    B, N, Hh, d = 1, 700, 2, 64
    nb = -(-N // 128)
    q, k, v, dout, lam, rp, ci, trp, tci = make(B, N, Hh, d, np.ones((Hh, nb, nb), bool), 6)
    w, gate = torch.zeros(d, d, device="cuda").bfloat16(), torch.ones(B, Hh, device="cuda")
    kept = sl.ckpt_pack([q, k, v])
    out, out2, lse = sl.diff_attn_forward_lse(q, k, v, rp, ci, lam)
    calls = (
        (sl.new_diff_workspace(B, N, Hh, d).numel(), lambda **kw: sl.diff_attn_backward(q, k, v, out, out2, dout, lse, rp, ci, lam, **kw)),
        (sl.new_ckpt_backward_workspace(B, N, Hh, d).numel(), lambda **kw: sl.attn_backward_ckpt(*kept, dout, rp, ci, w, gate, **kw)))
    side = torch.cuda.Stream()
    for size, call in calls:
        want = call()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)  # a tenth of a second or so
        got = call(stream=side)
        mine = torch.full((size,), 7, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        assert bool((mine == 7).all())
        assert all(torch.equal(want[n], got[n]) for n in want)


def test_a_wait_that_runs_out_is_reported():
    """With a limit of 0 every wait that is not already satisfied fails at once: an error status, no hang."""
    keep = np.ones((2, 3, 3), bool)
    q, k, v, dout, lam, rp, ci, *_ = make(1, 384, 2, 128, keep, 5)
    ws = sl.new_diff_workspace(1, 384, 2, 128)
    good = sl.diff_attn_forward_lse(q, k, v, rp, ci, lam, workspace=ws)
    sl.set_wait_limit_ns(0)
    try:
        sl.diff_attn_forward(q, k, v, rp, ci, lam, workspace=ws)
        assert sl.check_status(ws) == sl.SALAD_ERR_DEVICE_TIMEOUT
        sl.diff_attn_backward(q, k, v, good[0], good[1], dout, good[2], rp, ci, lam, workspace=ws)
        assert sl.check_status(ws) == sl.SALAD_ERR_DEVICE_TIMEOUT
    finally:
        sl.set_wait_limit_ns(2000000000)
    again = sl.diff_attn_forward_lse(q, k, v, rp, ci, lam, workspace=ws)
    assert sl.check_status(ws) == sl.SALAD_OK and all(torch.equal(a, b) for a, b in zip(good, again))
