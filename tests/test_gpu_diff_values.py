"""Differential attention at the borders of its values: scores of -inf, queries
without a value, large values, one weight that holds a row, and gradients at
q, k, v decoded from 8 bits.  The bounds are those of test_gpu_diff's docstring
where nothing else is said."""
import math

import numpy as np
import pytest
import torch

import sparse_linear_hybrid_b200 as sl
from test_gpu_diff import check_forward, decode_reference, make, maps, reference_gradients, rows_ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("late", [150, 158, 199])
def test_one_weight_that_holds_a_row_is_exact(late, d):
    """A late key that outweighs all the others gives its own value: the weight and the sum that it is divided by are
    rounded alike, whatever the weight is.

    Key 0 has the level 0, key `late` a level of L = 12.4 to 15.5 (in log2, by row) and all the others -86, so the rest of
    the row weighs 2^-12.4 of it at most.  With |v| in [1, 2), values 4 apart at most, it moves the output by 2^-10.4, and
    a bf16 value of 1 or more is left by 2^-9 at least."""
    N = 200
    keep = np.ones((1, 2, 2), bool)
    q, k, v, _, _, rp, ci, *_ = make(1, N, 1, d, keep, 43)
    level = 12.5 + 3 * torch.arange(N, device="cuda") / N
    q.zero_()
    k.zero_()
    for m in (0, d // 2):
        q[0, :, 0, m] = (level * math.log(2.0)).bfloat16()
        q[0, :, 0, m + 1] = 60.0
        k[0, :, 0, m + 1] = -1.0
        k[0, 0, 0, m + 1] = k[0, late, 0, m + 1] = 0
        k[0, late, 0, m] = 1
    v = ((1 + torch.rand(v.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(44)) * 0.99)
         * torch.where(torch.rand(v.shape, device="cuda") < 0.5, -1.0, 1.0)).bfloat16().clamp(-1.9921875, 1.9921875)
    want = v[:, late:late + 1].expand(1, N, 1, d)
    out, out2, lse = sl.diff_attn_forward_lse(q, k, v, rp, ci, torch.zeros(1, device="cuda"), softmax_scale=1.0)
    assert torch.equal(out, want) and torch.equal(out2, want)
    assert torch.equal(out, sl.diff_attn_forward(q, k, v, rp, ci, torch.zeros(1, device="cuda"), softmax_scale=1.0))


# keys of score -inf in map 1 (in map 2 for the second head)
DECODE = {"one key": ([0], 1), "alone in its slot": ([4], 5), "the first ones": (list(range(40)), 300),
          "all but one": ([j for j in range(517) if j != 300], 517), "every other": (list(range(0, 2000, 2)), 2000),
          "the last run": (list(range(1990, 2000)), 2000)}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [1, 2, 3])
@pytest.mark.parametrize("name", DECODE)
def test_decode_weighs_a_score_of_minus_infinity_with_nothing(name, Nq, d):
    at, n = DECODE[name]
    g = torch.Generator(device="cuda").manual_seed(n + d)
    q, k, v = (torch.randn(1, m, 2, d, generator=g, device="cuda").bfloat16() for m in (Nq, n + 3, n + 3))
    q[0, :, 0, 3], q[0, :, 1, d // 2 + 3] = 1.0, 1.0
    k[0, at, 0, 3], k[0, at, 1, d // 2 + 3] = -math.inf, -math.inf
    lam = torch.tensor([0.5, 0.8], device="cuda")
    out = sl.diff_attn_decode(q, k, v, torch.tensor([n], dtype=torch.int32, device="cuda"), lam)
    ref, size = decode_reference(q, k, v, [n], lam)  # (a map whose keys all score -inf: 0 / 0, NaN, as by the formula)
    assert torch.equal(torch.isnan(out), torch.isnan(ref)) and bool(torch.isnan(ref).any()) == (n == 1)
    assert n == 1 or bool(((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-5 * size).all())


@pytest.mark.parametrize("lam", [math.inf, math.nan])
def test_a_sequence_without_keys_is_zero_for_every_lambda(lam):
    q, k, v = (torch.randn(2, n, 1, 64, device="cuda").bfloat16() for n in (1, 9, 9))
    out = sl.diff_attn_decode(q, k, v, torch.tensor([0, 5], dtype=torch.int32, device="cuda"), torch.full((1,), lam, device="cuda"))
    assert bool((out[0] == 0).all()) and not bool(torch.isfinite(out[1]).any())


# keys of score -inf among 200: whole steps of 64, all but the cubic's positions, all but the last key
FORWARD = {"first step": range(64), "two steps and more": range(131), "all but the last": range(199), "first key": [0],
           "every other": range(0, 200, 2), "cubic": [j for j in range(200) if j % 8 >= 6],
           "all but the cubic's": [j for j in range(200) if j % 8 < 6], "the short last step": range(192, 200)}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name", FORWARD)
def test_forward_weighs_a_score_of_minus_infinity_with_nothing(name, d):
    keep = np.ones((2, 2, 2), bool)
    q, k, v, _, lam, rp, ci, *_ = make(1, 200, 2, d, keep, 23, lam_type=torch.float32)
    q[0, :, 0, 3], q[0, :, 1, d // 2 + 3] = 1.0, 1.0
    at = list(FORWARD[name])
    k[0, at, 0, 3], k[0, at, 1, d // 2 + 3] = -math.inf, -math.inf
    out, out2, lse = sl.diff_attn_forward_lse(q, k, v, rp, ci, lam)
    assert bool(torch.isfinite(out).all())
    check_forward(q, k, v, keep, lam, out, out2, lse, False)
    assert torch.equal(out, sl.diff_attn_forward(q, k, v, rp, ci, lam))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 64, 200])
def test_a_row_of_scores_of_minus_infinity_has_no_value(n, d):
    """Kept keys that all score -inf: 0 / 0 by the formula, and a log-sum-exp of -inf.  (No kept key at all: 0.)"""
    nb = -(-n // 128)
    q, k, v, _, lam, rp, ci, *_ = make(1, n, 2, d, np.ones((2, nb, nb), bool), 24)
    clean = sl.diff_attn_forward_lse(q, k, v, rp, ci, lam)
    q[0, :, 0, 3] = 1.0
    k[0, :, 0, 3] = -math.inf
    out, out2, lse = sl.diff_attn_forward_lse(q, k, v, rp, ci, lam)
    assert bool(torch.isnan(out[0, :, 0]).all()) and bool((lse[0, 0, 0] == -math.inf).all())
    assert all(torch.equal(a, b) for a, b in ((out[:, :, 1], clean[0][:, :, 1]), (out2, clean[1]), (lse[1], clean[2][1])))


@pytest.mark.parametrize("d", [64, 128])
def test_large_values_beside_scores_far_above_the_first_keys(d):
    """Values up to 2^88 in rows whose later scores pass the first keys' by 2^10 to 2^110: sums stay in fp32's range, as
    the output does.  Scores of up to 90 are off by 8 2^-23 90 each, a weight by twice that."""
    N, top = 680, 2.0 ** 88
    keep = np.ones((2, 6, 6), bool)
    q, k, v, _, _, rp, ci, *_ = make(1, N, 2, d, keep, 41)
    lam = torch.tensor([0.5, -0.25], device="cuda")
    v = (v.float().clamp(-1, 1) * top).bfloat16()
    scale, amp = 0.125, torch.tensor([16.0, 8.0, 4.0, 2.0, 0.0], device="cuda")[torch.arange(N, device="cuda") % 5]
    for h in range(2):
        for m in range(2):
            at = m * (d // 2)
            q[0, :, h, at] = amp.bfloat16()
            k[0, :, h, at] = 0
            k[0, 64:, h, at] = 4 + 3.0 * (h + m)      # 2^11 to 2^29 above the first step at the amplitude 16
            k[0, 400:, h, at] = 30                    # 2^87
            k[0, 601 + h, h, at] = 38                 # 2^110, in one key
    out, out2, lse = sl.diff_attn_forward_lse(q, k, v, rp, ci, lam, softmax_scale=scale)
    more = 2 * 8 * 2.0 ** -23 * 90
    for h in range(2):
        (p1, _), (p2, _) = maps(q, k, keep, scale, 0, h, False, 2)
        x, lh = v[0, :, h].double(), float(lam[h])
        for got, ref, size in ((out, (p1 - lh * p2) @ x, (p1 + abs(lh) * p2) @ x.abs()), (out2, p2 @ x, p2 @ x.abs())):
            lim = 2.0 ** -8 * ref.abs() + (2 * 2.0 ** -8 + 2e-4 + more) * size
            assert bool(((got[0, :, h].double() - ref).abs() <= lim).all()), h


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [0, 5, 6, 7, 70, 150, 199])
@pytest.mark.parametrize("bad,map_", [(math.nan, 0), (math.nan, 1), (math.inf, 0)])
def test_a_query_without_a_value_shows_in_every_gradient(d, at, bad, map_):
    """NaN or infinity in one query: its dq, and dk and dv of every key that it keeps, are NaN by the formula, wherever the
    cubic forms its exponentials; keys that it does not keep, and the other head, stay."""
    keep = np.ones((2, 2, 2), bool)
    keep[0] = [[True, True], [False, True]]  # the second block of queries does not keep the first block of keys
    q, k, v, dout, lam, rp, ci, trp, tci = make(1, 200, 2, d, keep, 29)
    kw = dict(t_row_ptr=trp, t_col_idx=tci)

    def gradients():
        out, out2, lse = sl.diff_attn_forward_lse(q, k, v, rp, ci, lam)
        return sl.diff_attn_backward(q, k, v, out, out2, dout, lse, rp, ci, lam, **kw)
    clean = gradients()
    q[0, at, 0, map_ * (d // 2) + 3] = bad
    got = gradients()
    kept = slice(0, 200) if at < 128 else slice(128, 200)
    half = slice(map_ * (d // 2), (map_ + 1) * (d // 2))
    assert bool(torch.isnan(got["dq"][0, at, 0, half]).all())
    assert bool(torch.isnan(got["dv"][0, kept, 0]).all()) and bool(torch.isnan(got["dk"][0, kept, 0, half]).all())
    assert bool(torch.isnan(got["dlam"][0])) == (map_ == 1)
    if at >= 128:
        assert all(torch.equal(got[n][0, :128, 0], clean[n][0, :128, 0]) for n in ("dq", "dk", "dv"))
    assert all(torch.equal(got[n][0, :, 1], clean[n][0, :, 1]) for n in ("dq", "dk", "dv"))
    assert torch.equal(got["dlam"][1], clean["dlam"][1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [200, 330])
def test_gradients_beside_a_score_of_minus_infinity(N, d):
    """A key that scores -inf for every query weighs nothing: dlam and the other keys' dk and dv are those of the formula,
    also where the last tile of queries is short (dq is 0 times the infinite key, NaN)."""
    nb = -(-N // 128)
    keep = np.ones((2, nb, nb), bool)
    q, k, v, dout, lam, rp, ci, *_ = make(1, N, 2, d, keep, 37, lam_type=torch.float32)
    q[0, :, 0, 3], q[0, :, 1, d // 2 + 3] = 1.0, 1.0
    k[0, [3, 6, 71, N - 1], 0, 3], k[0, [7, 130], 1, d // 2 + 3] = -math.inf, -math.inf
    out, out2, lse = sl.diff_attn_forward_lse(q, k, v, rp, ci, lam)
    got = sl.diff_attn_backward(q, k, v, out, out2, dout, lse, rp, ci, lam)
    _, dk, dv, dlam, size, *_ = reference_gradients(q, k, v, dout, keep, lam, False)
    for name, ref in (("dk", dk), ("dv", dv)):
        for h in range(2):
            other = torch.isfinite(k[0, :, h]).all(-1)
            rows_ok(got[name][0, other, h], ref[0, other, h], name)
    assert bool(((got["dlam"].double() - dlam).abs() <= 2.0 ** -24 * dlam.abs() + 1e-4 * size).all())


def test_a_mask_that_is_not_symmetric():
    """Rows per head, not symmetric, and no transposed mask given: the gradients are those with it."""
    N, Hh, d = 300, 2, 64
    keep = np.zeros((Hh, 3, 3), bool)
    keep[0] = np.tril(np.ones((3, 3), bool))
    keep[1, :, 1] = keep[1, 2, 0] = True
    q, k, v, dout, lam, rp, ci, trp, tci = make(1, N, Hh, d, keep, 53)
    out, out2, lse = sl.diff_attn_forward_lse(q, k, v, rp, ci, lam)
    args = (q, k, v, out, out2, dout, lse, rp, ci, lam)
    want = sl.diff_attn_backward(*args, t_row_ptr=trp, t_col_idx=tci)
    got = sl.diff_attn_backward(*args)
    assert all(torch.equal(got[n], want[n]) for n in want)
    w, gate = (torch.randn(d, d, device="cuda") / 8).bfloat16(), torch.rand(1, Hh, device="cuda")
    args = (*sl.ckpt_pack([q, k, v]), dout, rp, ci, w, gate)
    want = sl.attn_backward_ckpt(*args, t_row_ptr=trp, t_col_idx=tci)
    got = sl.attn_backward_ckpt(*args)
    assert all(torch.equal(got[n], want[n]) for n in want)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_gradients_at_decoded_values(fmt):
    """A training step that keeps q, k and v in 8 bits: the backward gets the out, out2 and lse of a forward on the decoded
    values, and gives the gradients at them."""
    B, N, Hh, d = 2, 333, 2, 128
    keep = np.random.default_rng(47).random((Hh, 3, 3)) < 0.7
    keep[:, np.arange(3), np.arange(3)] = True
    q, k, v, dout, lam, rp, ci, trp, tci = make(B, N, Hh, d, keep, 48, lam_type=torch.float32)
    q, k, v = sl.ckpt_unpack(sl.ckpt_pack([q, k, v], fmt=fmt))
    out, out2, lse = sl.diff_attn_forward_lse(q, k, v, rp, ci, lam)
    got = sl.diff_attn_backward(q, k, v, out, out2, dout, lse, rp, ci, lam, t_row_ptr=trp, t_col_idx=tci)
    dq, dk, dv, dlam, size, *_ = reference_gradients(q, k, v, dout, keep, lam, False)
    for name, ref in (("dq", dq), ("dk", dk), ("dv", dv)):
        rows_ok(got[name], ref, name)
    assert bool(((got["dlam"].double() - dlam).abs() <= 2.0 ** -24 * dlam.abs() + 1e-4 * size).all())


def test_training_step_with_8_bit_inputs():
    """Rotation, forward, q, k and v kept in 8 bits; then decoded, forward again, gradients, rotation back: the gradients at
    the decoded values, eager, and captured and replayed on new inputs."""
    B, T, H, W, Hh, d = 1, 2, 9, 13, 2, 64
    N, sections = T * H * W, (12, 10, 10)
    keep = np.ones((Hh, 2, 2), bool)
    q0, k0, v, dout, lam, *_ = make(B, N, Hh, d, keep, 59, lam_type=torch.float32)
    rp, ci = sl.build_block_mask(T, H, W, 128, np.tile(np.int32([1, 8, 12]), (Hh, 1)))  # (every block: `keep`)
    assert ci.numel() == keep.sum()
    freq, scale = sl.rope_inv_freq(d, sections=sections)
    kw = dict(sections=sections, interleaved=True, scale=scale, grid=(T, H, W))
    ws = sl.new_diff_workspace(B, N, Hh, d)

    def step():
        q, k = sl.rope_forward(q0, k0, freq, **kw)
        out = sl.diff_attn_forward(q, k, v, rp, ci, lam, workspace=ws)
        kept = sl.ckpt_pack([q, k, v])
        decoded = sl.ckpt_unpack(kept)
        again = sl.diff_attn_forward_lse(*decoded, rp, ci, lam, workspace=ws)
        grads = sl.diff_attn_backward(*decoded, *again[:2], dout, again[2], rp, ci, lam, t_row_ptr=rp, t_col_idx=ci, workspace=ws)
        return [out, *decoded, *grads.values(), *sl.rope_backward(grads["dq"], grads["dk"], freq, **kw)]

    def check(out, q, k, v8, dq, dk, dv, dlam, dq0, dk0):
        check_forward(*sl.rope_forward(q0, k0, freq, **kw), v, keep, lam, out, None, None, False)
        ref = reference_gradients(q, k, v8, dout, keep, lam, False)
        for name, got, want in (("dq", dq, ref[0]), ("dk", dk, ref[1]), ("dv", dv, ref[2])):
            rows_ok(got, want, name)
        assert bool(((dlam.double() - ref[3]).abs() <= 2.0 ** -24 * ref[3].abs() + 1e-4 * ref[4]).all())
        assert all(torch.equal(a, b) for a, b in zip((dq0, dk0), sl.rope_backward(dq, dk, freq, **kw)))

    check(*step())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for t in (q0, k0, v, dout):
        t.normal_()
    graph.replay()
    torch.cuda.synchronize()
    check(*captured)
    assert sl.check_status(ws) == sl.SALAD_OK
