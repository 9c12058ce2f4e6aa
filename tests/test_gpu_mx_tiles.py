"""Microscaled products and experts at shapes that reach every way of dealing
tiles: both token tiles of the pair kernel with several tiles a pair, a short last
group of row tiles, runs that begin and end inside a tile of the experts."""
import numpy as np
import pytest
import torch

from oracle import mx
from test_gpu_mx import (check, f64, lora_terms, moe_case, moe_reference, no_device_errors, normal, product_bound,  # noqa: F401
                         qb)
from test_gpu_mx_adapter import gradient_and_bound

pytestmark = pytest.mark.gpu


def form(qb, *args, **kw):  # noqa: F811
    return qb.qlora_selftest_mx_form(*args, num_sms=torch.cuda.get_device_properties(0).multi_processor_count, **kw)


def expect(want):
    """The tile sizes below are what 148 SMs take."""
    if torch.cuda.get_device_properties(0).multi_processor_count == 148:
        assert want


# token tile, tiles a pair (of 74): 256, 3.9; 128, 8.2
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("rows,cols,m,tile", [(4730, 330, 3830, 256), (4700, 72, 4090, 128)])
def test_pairs_with_several_tiles(qb, rows, cols, m, tile, fmt):  # noqa: F811
    expect(form(qb, rows, cols, fmt, m) == ("pair", tile))
    w, x = normal((rows, cols), 0.02, 1), normal((m, cols), 1.0, 2)
    q = qb.qlora_mx_quantize(w.cuda(), fmt)
    wv, xv = f64(qb.qlora_mx_dequantize(q)), mx.round_trip(f64(x), fmt, True)
    want = xv @ wv.T
    Y = qb.qlora_mx_linear_fwd(q, x.cuda())[0]
    check(Y, want, product_bound(want, xv, wv), "Y")
    assert torch.equal(qb.qlora_mx_linear_fwd(q, x.cuda())[0], Y)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("rows,cols,m,r,tile", [(4728, 320, 3830, 72, 256), (4704, 64, 4090, 136, 128)])
def test_pairs_with_several_tiles_and_an_adapter(qb, rows, cols, m, r, tile, fmt):  # noqa: F811
    expect(form(qb, rows, cols, fmt, m, r) == ("pair", tile))
    w, x = normal((rows, cols), 0.02, 1), normal((m, cols), 1.0, 2)
    a, b, s = normal((r, cols), 0.02, 3), normal((rows, r), 0.02, 4), 16.0 / r
    q = qb.qlora_mx_quantize(w.cuda(), fmt)
    Y, XA = qb.qlora_mx_linear_fwd(q, x.cuda(), a.cuda(), b.cuda(), s)
    wv, xv = f64(qb.qlora_mx_dequantize(q)), mx.round_trip(f64(x), fmt, True)
    term, slack = lora_terms(f64(x), f64(a), f64(b), s)
    want = xv @ wv.T + term
    check(Y, want, product_bound(want, xv, wv) + slack, "Y")


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("rows,cols,m,r,tile", [(320, 4736, 3830, 72, 256), (72, 4736, 4090, 136, 128)])
def test_backward_of_pairs_with_several_tiles(qb, rows, cols, m, r, tile, fmt):  # noqa: F811
    expect(form(qb, rows, cols, fmt, m, r, backward=True) == ("pair", tile))
    w, dy, x = normal((rows, cols), 0.02, 1), normal((m, rows), 1e-3, 2), normal((m, cols), 1.0, 5)
    a, b, s = normal((r, cols), 0.02, 3), normal((rows, r), 0.02, 4), 16.0 / r
    qt = qb.qlora_mx_quantize(w.cuda(), fmt, transpose=True)
    dX, dA, dB = qb.qlora_mx_linear_bwd(qt, dy.cuda(), x.cuda(), a.cuda(), b.cuda(), s)
    X, dY, A, B = f64(x), f64(dy), f64(a), f64(b)
    wt, gv = f64(qb.qlora_mx_dequantize(qt)), mx.round_trip(dY, fmt, True)
    term, slack = lora_terms(dY, B.T, A.T, s)
    want = gv @ wt.T + term
    check(dX, want, product_bound(want, gv, wt) + slack, "dX")
    check(dA, *gradient_and_bound(dY @ B, X, rows, s, np.abs(dY) @ np.abs(B)), "dA")
    want, bound = gradient_and_bound(X @ A.T, dY, cols, s, np.abs(X) @ np.abs(A).T)
    check(dB, want.T, bound.T, "dB")


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_a_short_last_group_of_row_tiles(qb, fmt):  # noqa: F811
    """48 MB of codes are 48 row tiles of 256 x 8192: 51 and a part are swept in two groups."""
    rows, cols, m = 13070, 8192, 300
    w, x = torch.randn(rows, cols, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).mul_(0.02), normal((m, cols), 1.0, 2)
    q = qb.qlora_mx_quantize(w.to(torch.bfloat16), fmt)
    Y = qb.qlora_mx_linear_fwd(q, x.cuda())[0]
    pick = np.sort(np.random.default_rng(0).choice(rows, 150, replace=False))
    pick = np.unique(np.concatenate([pick, [0, 12287, 12288, 12289, 13055, 13056, rows - 1]]))
    at = torch.from_numpy(pick).cuda()
    wv, xv = f64(qb.qlora_mx_dequantize(q)[at]), mx.round_trip(f64(x), fmt, True)
    want = xv @ wv.T
    check(Y[:, at], want, product_bound(want, xv, wv), "Y")


# ---------------------------------------------------------------- the adapter at 17 to 64 tokens, and rank 256
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("given_xa", [True, False])
@pytest.mark.parametrize("rows,cols,m,r", [(392, 640, 17, 64), (256, 320, 32, 136), (1000, 1088, 33, 8), (520, 4096, 64, 256),
                                           (136, 1024, 200, 256)])
def test_backward_with_an_adapter_over_a_weight(qb, rows, cols, m, r, given_xa, fmt):  # noqa: F811
    w, dy, x = normal((rows, cols), 0.02, 1), normal((m, rows), 1e-3, 2), normal((m, cols), 1.0, 5)
    a, b, s = normal((r, cols), 0.02, 3), normal((rows, r), 0.02, 4), 16.0 / r
    qt = qb.qlora_mx_quantize(w.cuda(), fmt, transpose=True)
    X, dY, A, B = f64(x), f64(dy), f64(a), f64(b)
    xa = torch.from_numpy(X @ A.T).float().cuda() if given_xa else None
    dX, dA, dB = qb.qlora_mx_linear_bwd(qt, dy.cuda(), x.cuda(), a.cuda(), b.cuda(), s, XA=xa)
    term, slack = lora_terms(dY, B.T, A.T, s)
    wt, gv = mx.round_trip(f64(w).T, fmt), mx.round_trip(dY, fmt, True)
    want = gv @ wt.T + term
    check(dX, want, product_bound(want, gv, wt) + slack, "dX")
    check(dA, *gradient_and_bound(dY @ B, X, rows, s, np.abs(dY) @ np.abs(B)), "dA")
    want, bound = gradient_and_bound(X @ A.T, dY, cols, s, np.abs(X) @ np.abs(A).T)
    check(dB, want.T, bound.T, "dB")


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("m,r", [(3, 64), (16, 8)])
def test_gradients_of_few_tokens_see_no_stale_work_buffer(qb, m, r, fmt):  # noqa: F811
    """All three results are bit for bit those of a fresh work buffer (every sum has a fixed order)."""
    rows, cols = 520, 1344
    x, dy = normal((m, cols), 1.0, 2).cuda(), normal((m, rows), 1e-3, 3).cuda()
    qt = qb.qlora_mx_quantize(normal((rows, cols), 0.02, 1).cuda(), fmt, transpose=True)
    a, b = normal((r, cols), 0.02, 4).cuda(), normal((rows, r), 0.02, 5).cuda()
    want = qb.qlora_mx_linear_bwd(qt, dy, x, a, b, 0.25)
    for fill in (0xFF, 0x7F):
        ws = torch.full((qb.qlora_mx_linear_workspace_size(rows, cols, fmt, m, r)[1],), fill, dtype=torch.uint8, device="cuda")
        assert all(torch.equal(u, v) for u, v in zip(qb.qlora_mx_linear_bwd(qt, dy, x, a, b, 0.25, workspace=ws), want))


# ---------------------------------------------------------------- experts
# Tiles and steps a tile on 148 SMs: up 192 x 4 (all 16 experts in use); up 256 x 3, runs over three tiles;
# down 150 x 4 (hidden 19200, four experts of one step each).
@pytest.mark.parametrize("experts,hidden,inner,m,top_k", [(16, 1024, 1536, 16, 4), (32, 768, 1024, 16, 4), (4, 19200, 128, 6, 2)])
def test_experts_in_runs_across_tiles(qb, experts, hidden, inner, m, top_k):  # noqa: F811
    q13, q2, router, x = moe_case(qb, experts, hidden, inner, m, experts + m, std=0.02)
    ids, p, y, off = moe_reference(qb, q13, q2, router, x, top_k)
    assert len(np.unique(ids)) * (inner // 128) > 148 or hidden // 128 > 148
    Y, got_ids, got_p = qb.qlora_mx_moe_fwd(q13, q2, router, x, top_k)
    assert np.array_equal(got_ids.cpu().numpy(), ids)
    assert np.all(np.abs(f64(got_p) - p) <= p * 2.0 ** -17)
    check(Y, y, off, "Y")
    need = qb.qlora_mx_moe_workspace_size(experts, hidden, inner, m, top_k)
    for fill in (0xFF, 0x7F, 0x00):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(qb.qlora_mx_moe_fwd(q13, q2, router, x, top_k, workspace=ws)[0], Y)
