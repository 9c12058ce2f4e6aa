"""Corners of the microscaled operators on the GPU that the shape sweeps do not reach."""
import numpy as np
import pytest
import torch

from oracle import mx
from test_gpu_mx import check, f64, moe_case, no_device_errors, normal, product_bound, qb, upload  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- the two global scales of NVFP4
@pytest.mark.parametrize("per_row", [False, True])
@pytest.mark.parametrize("m", [1, 12, 40, 150])
def test_results_near_the_ends_of_the_range(qb, m, per_row):  # noqa: F811
    """Tokens of 2^118 and 2^-100 give the result of tokens of 1, scaled: a result
    that bf16 holds is not lost on the way to it."""
    w, x = normal((300, 640), 0.02, 1).cuda(), normal((m, 640), 1.0, 2).cuda()
    q = qb.qlora_mx_quantize(w, "nvfp4", per_row=per_row)
    y = qb.qlora_mx_linear_fwd(q, x)[0]
    for e in (118, -100):
        got = qb.qlora_mx_linear_fwd(q, x * 2.0 ** e)[0]
        assert torch.equal(got, y * 2.0 ** e)


@pytest.mark.parametrize("m", [1, 12, 40, 150])
@pytest.mark.parametrize("we,xe,wf,xf,top", [
    (30, 90, 0, 0, None),              # scales of 2^40 and 2^100; the blocks of 2^30 and of 2^90 get the scale 0
    (33, 93, 0, 0, 126),               # those of 2^33 and 2^93 are kept
    (33, 93, -130, -112, -116),        # scales of 2^-90 and 2^-12
    (33, 93, -130, -150, None)])       # scales of 2^-90 and 2^-50: 2^-154
def test_global_scales_whose_product_no_float_holds(qb, we, xe, wf, xf, top, m):  # noqa: F811
    """One value of W below its tensor's scale meets one of X below its token's:
    a single product, so the result is the exact one, rounded to bf16."""
    def scaled(t, e):
        return (t.double() * 2.0 ** e).to(torch.bfloat16)

    w, x = torch.zeros(64, 64, dtype=torch.bfloat16), torch.zeros(m, 64, dtype=torch.bfloat16)
    w[0, 0], w[1, 16] = 2.0 ** 51, 2.0 ** we
    x[:, 32], x[:, 16] = 2.0 ** 111, 2.0 ** xe
    if xf == -150:
        x[:, 0] = 2.0 ** 111                               # and a product of 2^-118
    w, x = scaled(w, wf), scaled(x, xf)
    want = mx.round_trip(f64(x), "nvfp4", True) @ mx.round_trip(f64(w), "nvfp4").T
    assert top is None or (want[:, 1] == 2.0 ** top).all()
    got = qb.qlora_mx_linear_fwd(qb.qlora_mx_quantize(w.cuda(), "nvfp4"), x.cuda())[0]
    assert torch.equal(got.cpu(), torch.from_numpy(want).to(torch.bfloat16))


@pytest.mark.parametrize("m", [1, 12, 40, 150])
@pytest.mark.parametrize("g,e", [(1.2345, 0), (3.0e-41, 100), (1.0e-33, 80), (1.0e30, -100)])
def test_a_foreign_global_scale(qb, m, g, e):  # noqa: F811
    """Any positive float is taken as a weight's global scale, one below the normal range too."""
    w, x = f64(normal((200, 320), 1.0, 1)), normal((m, 320), 1.0, 2)
    q = upload(qb, w, "nvfp4")
    q.global_scale.fill_(g)
    x = x * 2.0 ** e
    wv = mx.values(*mx.quantize(w, "nvfp4")[:2], q.global_scale.double().cpu().numpy(), "nvfp4")
    xv = mx.round_trip(f64(x), "nvfp4", True)
    check(qb.qlora_mx_linear_fwd(q, x.cuda())[0], xv @ wv.T, product_bound(xv @ wv.T, xv, wv) * (1 + 2.0 ** -20), "Y")


# ---------------------------------------------------------------- dequantisation
def bf16_once(v):
    """float64 values of few bits -> the nearest bf16 value, ties to even, subnormals included."""
    step = 2.0 ** (np.maximum(np.frexp(v)[1] - 1, -126) - 7.0)
    return np.rint(v / step) * step


def foreign_scales():
    """(global scales, E4M3 bytes): scales g that put some level * S * g next to a
    tie of bf16, nearer than fp32 resolves, then random ones down to where the
    values are subnormal."""
    lv, g, sb = mx.e4m3_levels(), [], []
    for s in range(0x38, 0x40):                            # S of 1 .. 1.875
        for level in (1.0, 1.5):
            tie = (np.arange(128, 256) + 0.5) / 128
            c = (tie / (level * lv[s])).astype(np.float32)
            p = np.float64(c) * level * lv[s]
            c = c[bf16_once(p) != bf16_once(p.astype(np.float32).astype(np.float64))]
            g += list(c)
            sb += [s] * len(c)
    assert len(g) > 100
    rng = np.random.default_rng(0)
    g += list((rng.uniform(1, 2, 600) * 2.0 ** rng.integers(-140, 100, 600)).astype(np.float32))
    sb += list(rng.integers(1, 127, 600))
    return np.array(g, np.float32), np.array(sb, np.uint8)


@pytest.mark.parametrize("cols", [16, 11])
def test_dequantize_rounds_once_under_any_global_scale(qb, cols):  # noqa: F811
    g, sb = foreign_scales()
    codes = np.broadcast_to(np.arange(16, dtype=np.uint8)[::-1][:cols], (len(g), cols)).copy()
    q = qb.MXTensor(torch.from_numpy(mx.pack(codes)).reshape(-1).cuda(), torch.from_numpy(mx.tile_scales(sb[:, None])).cuda(),
                    torch.from_numpy(g).cuda(), len(g), cols, "nvfp4")
    want = mx.values(codes, sb[:, None], g.astype(np.float64), "nvfp4")
    assert np.array_equal(f64(qb.qlora_mx_dequantize(q)), bf16_once(want))


# ---------------------------------------------------------------- calls that overlap
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("m,size", [(1, 4096), (3, 2048), (5, 1001)])
def test_one_launch_products_in_a_chain(qb, m, size, fmt):  # noqa: F811
    """Each product starts while the one that writes its tokens still runs (and the
    first of a round while its weight is still being quantised); the result is that
    of the same calls with a wait after each.  (4096 x 4096 NVFP4 takes two launches.)"""
    if torch.cuda.get_device_properties(0).multi_processor_count == 148:
        assert qb.qlora_selftest_mx_form(size, size, fmt, m) == (("stream", 16) if (size, fmt) == (4096, "nvfp4") else ("few", 8))
    ws = [normal((size, size), size ** -0.5, i).cuda() for i in range(4)]
    x = normal((m, size), 1.0, 9).cuda()
    out = [qb.empty_mx(size, size, x.device, fmt) for _ in ws]

    def chain(wait):
        y, all_y = x, []
        for w, q in zip(ws, out):
            qb.qlora_mx_quantize(w, out=q)
            for _ in range(3):
                y = qb.qlora_mx_linear_fwd(q, y)[0]
                if wait:
                    torch.cuda.synchronize()
                all_y.append(y)
        return all_y

    want = chain(True)
    assert all(torch.isfinite(y).all() for y in want)
    for _ in range(5):
        for q in out:
            q.codes.fill_(0x77)
        assert all(torch.equal(a, b) for a, b in zip(chain(False), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(False)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---------------------------------------------------------------- routing
def test_a_nan_logit_is_the_largest(qb):  # noqa: F811
    """Experts whose logit is NaN for some tokens: chosen first there, the lowest
    index first, as a descending stable sort has it, and seen in p and Y."""
    q13, q2, router, x = moe_case(qb, 12, 256, 128, 6, 3)
    x[:, 7] = 0
    x[2, 7], x[4, 7] = float("inf"), float("inf")
    router[:, 7] = 1
    router[5, 7] = router[9, 7] = 0                        # inf * 0; every other logit of these tokens is inf
    ids_want = torch.sort(x.float() @ router.float().t(), dim=1, descending=True, stable=True)[1][:, :4]
    Y, ids, p = qb.qlora_mx_moe_fwd(q13, q2, router, x, 4)
    assert torch.equal(ids.long(), ids_want) and ids[2].tolist() == [5, 9, 0, 1]
    for t in range(6):
        bad = t in (2, 4)
        assert bool(p[t].isnan().all()) is bad and bool(Y[t].isnan().all()) is bad
        assert bad or (p[t].sum() - 1).abs() < 1e-5


# ---------------------------------------------------------------- the adapter under far global scales
@pytest.mark.parametrize("m", [3, 40, 150])
@pytest.mark.parametrize("g", [2.0e-39, 2.0 ** -140])
def test_an_adapter_of_zeros_under_a_tiny_global_scale(qb, m, g):  # noqa: F811
    """1 / g is no float, but the rank-r term of zeros divided by g is zero, forward and backward."""
    w, x, dy = normal((128, 192), 1.0, 1), normal((m, 192), 1.0, 2).cuda(), normal((m, 128), 1.0, 3).cuda()
    zero, b = torch.zeros(8, 192, dtype=torch.bfloat16, device="cuda"), normal((128, 8), 0.02, 4).cuda()
    q, qt = upload(qb, f64(w), "nvfp4"), upload(qb, f64(w).T, "nvfp4")
    q.global_scale.fill_(g)
    qt.global_scale.fill_(g)
    plain, back = qb.qlora_mx_linear_fwd(q, x)[0], qb.qlora_mx_linear_bwd(qt, dy)[0]
    assert torch.isfinite(plain).all() and torch.isfinite(back).all()
    assert torch.equal(qb.qlora_mx_linear_fwd(q, x, zero, b, 0.5)[0], plain)
    a = normal((8, 192), 0.02, 5).cuda()
    assert torch.equal(qb.qlora_mx_linear_bwd(qt, dy, x, a, torch.zeros_like(b), 0.5)[0], back)


@pytest.mark.parametrize("m", [1, 12, 40, 150])
def test_a_rank_term_that_overflows_is_infinite(qb, m):  # noqa: F811
    """X A^T (dY B) of one token and one rank is past fp32's range: the token's Y
    (dX) takes the sign of B (A), as the formula has it, and the others do not see it."""
    rows, cols, r = 136, 192, 8
    w, x, dy = normal((rows, cols), 0.02, 1).cuda(), normal((m, cols), 1.0, 2).cuda(), normal((m, rows), 1.0, 3).cuda()
    a, b = normal((r, cols), 0.02, 4).cuda(), normal((rows, r), 0.02, 5).cuda()
    q, qt = qb.qlora_mx_quantize(w), qb.qlora_mx_quantize(w, transpose=True)
    x[:, 5], dy[:, 7] = 0, 0
    a[0, 5], b[7, 0] = 2.0 ** 100, 2.0 ** 100
    clean, back = qb.qlora_mx_linear_fwd(q, x, a, b, 0.5)[0], qb.qlora_mx_linear_bwd(qt, dy, x, a, b, 0.5)[0]
    x[0, 5], dy[0, 7] = 2.0 ** 60, 2.0 ** 60
    Y, dX = qb.qlora_mx_linear_fwd(q, x, a, b, 0.5)[0], qb.qlora_mx_linear_bwd(qt, dy, x, a, b, 0.5)[0]
    assert torch.equal(Y[0].float(), torch.copysign(torch.full((rows,), float("inf"), device="cuda"), b[:, 0].float()))
    assert torch.equal(dX[0].float(), torch.copysign(torch.full((cols,), float("inf"), device="cuda"), a[0].float()))
    assert torch.equal(Y[1:], clean[1:]) and torch.equal(dX[1:], back[1:])
