"""The layer's calls with a stream of the caller's: what they allocate is of that
stream, so that memory of a call that still runs is not given out again, and a mask
that is transposed on the way is transposed on that stream."""
import pytest
import torch

import sparse_linear_hybrid_b200 as sl

pytestmark = pytest.mark.gpu


def test_the_layers_calls_keep_their_memory_on_their_stream():
    B, N, Hh, d = 1, 700, 2, 64
    nb = -(-N // 128)
    g = torch.Generator(device="cuda").manual_seed(61)
    q, k, v, dout = (torch.randn(B, N, Hh, d, generator=g, device="cuda").bfloat16() for _ in range(4))
    w, gate = (torch.randn(d, d, generator=g, device="cuda") / 8).bfloat16(), torch.rand(B, Hh, generator=g, device="cuda")
    rp, ci = sl.build_topk_mask(q, k, 128, 3)
    kw = dict(mask_per_bh=True)
    out, lse = sl.attn_forward_lse(q, k, v, rp, ci, w, gate, 128, **kw)
    w_x, beta, t_emb = torch.randn(Hh, d, device="cuda"), torch.randn(Hh, device="cuda"), torch.randn(B, 32, device="cuda")
    w_t = torch.randn(Hh, 32, device="cuda")
    calls = {
        "attn_forward": lambda **s: [sl.attn_forward(q, k, v, rp, ci, w, gate, 128, **kw, **s)],
        "attn_forward_lse": lambda **s: sl.attn_forward_lse(q, k, v, rp, ci, w, gate, 128, **kw, **s),
        "attn_forward_static": lambda **s: [sl.attn_forward_static(q, k, v, rp, ci, w, gate, 128, **s)],
        "attn_backward": lambda **s: sl.attn_backward(q, k, v, out, dout, lse, rp, ci, w, gate, **kw, **s).values(),
        "attn_backward_sparse": lambda **s: sl.attn_backward_sparse(q, k, v, out, dout, lse, rp, ci, **kw, **s),
        "gate_forward": lambda **s: [sl.gate_forward(q, t_emb, w_t, w_x, beta, 0.3, **s)],
        "build_topk_mask": lambda **s: sl.build_topk_mask(q, k, 128, 3, **s),
        "transpose_block_mask": lambda **s: sl.transpose_block_mask(rp, ci, B * Hh, nb, **s),
        "linear_state": lambda **s: sl.linear_state(k, v, **s),
    }
    side = torch.cuda.Stream()
    for name, call in calls.items():
        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)  # some twentieth of a second
        got = list(call(stream=side))
        # memory of every size that the call has just dropped, written on the current stream
        mine = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in (512, 4096, 65536, 1 << 20, 1 << 22, 1 << 24) for _ in range(4)]
        torch.cuda.synchronize()
        assert all(bool((m == 7).all()) for m in mine), name
        assert all(torch.equal(a, b) for a, b in zip(want, got)), name
