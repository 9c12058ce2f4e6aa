"""The microscaled 4-bit operators on the GPU against the 64-bit oracle."""
import functools

import numpy as np
import pytest
import torch

from oracle import mx

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_nf4_quantized_encode_b200 as m
    return m


@pytest.fixture(autouse=True)
def no_device_errors(qb):
    yield
    torch.cuda.synchronize()
    assert qb.qlora_read_device_errors() == 0


def normal(shape, std=1.0, seed=0):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.standard_normal(shape) * std).to(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


def parts(q):
    """A library tensor's codes [rows, pitch], scales and global scale as numpy."""
    g = None if q.global_scale is None else q.global_scale.cpu().numpy().astype(np.float64)
    nc = q.rows * (-(-q.cols // 32) * 16)
    return q.codes[:nc].cpu().numpy().reshape(q.rows, -1), q.scales.cpu().numpy(), g


def upload(qb, x, fmt, per_row=False):
    """Quantise with the oracle and put the result on the GPU."""
    codes, sb, g = mx.quantize(x, fmt, per_row)
    return qb.MXTensor(torch.from_numpy(mx.pack(codes)).reshape(-1).cuda(), torch.from_numpy(mx.tile_scales(sb)).cuda(),
                       None if g is None else torch.from_numpy(g).float().cuda(), *x.shape, fmt)


def same_as_oracle(q, x, fmt, per_row):
    codes, sb, g = mx.quantize(x, fmt, per_row)
    got_c, got_s, got_g = parts(q)
    if g is not None:
        assert np.array_equal(got_g, np.broadcast_to(g, got_g.shape))
    assert np.array_equal(got_s, mx.tile_scales(sb))
    assert np.array_equal(got_c, mx.pack(codes))


FORMS = [("mxfp4", False), ("nvfp4", False), ("nvfp4", True)]
SHAPES = [(1, 1), (1, 8192), (3, 31), (5, 32), (7, 33), (128, 64), (129, 1000), (100, 1999), (257, 8200), (2, 22016),
          (300, 16), (33, 8193), (700, 4160), (601, 9001), (20, 16000), (9, 1001), (17, 2047), (64, 36), (40, 4098)]


@pytest.mark.parametrize("fmt,per_row", FORMS)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_bit_for_bit(qb, rows, cols, fmt, per_row):
    w = normal((rows, cols), 0.02, rows + cols)
    same_as_oracle(qb.qlora_mx_quantize(w.cuda(), fmt, per_row=per_row), f64(w), fmt, per_row)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 300), (300, 1), (64, 128), (129, 65), (200, 1000), (1001, 72), (31, 999)])
def test_quantize_transposed_bit_for_bit(qb, rows, cols, fmt):
    w = normal((rows, cols), 0.02, rows + cols)
    q = qb.qlora_mx_quantize(w.cuda(), fmt, transpose=True)
    assert (q.rows, q.cols) == (cols, rows)
    same_as_oracle(q, f64(w).T, fmt, False)


@pytest.mark.parametrize("fmt,per_row", FORMS)
def test_quantize_every_bf16_value_and_ties(qb, fmt, per_row):
    """All finite bf16 bit patterns, in an order that mixes magnitudes: every
    scale, subnormals, zeros of both signs, both overflow ends and, with the
    multiples of small powers of two among them, every tie."""
    bits = np.arange(1 << 16, dtype=np.uint32)
    bits = bits[(bits & 0x7F80) != 0x7F80]
    sorted_rows = bits[np.argsort(bits & 0x7FFF, kind="stable")]
    mixed = np.random.default_rng(1).permutation(bits)
    all_bits = np.concatenate([sorted_rows, mixed]).astype(np.uint16).reshape(-1, 120)
    ties = np.outer(2.0 ** np.arange(-20, 20), np.arange(-56, 64) / 8.0)      # quarter and eighth steps
    w = torch.cat([torch.from_numpy(all_bits.view(np.int16)).view(torch.bfloat16), torch.from_numpy(ties).to(torch.bfloat16)])
    q = qb.qlora_mx_quantize(w.cuda(), fmt, per_row=per_row)
    same_as_oracle(q, f64(w), fmt, per_row)


@pytest.mark.parametrize("fmt,per_row", FORMS)
def test_a_value_that_is_not_finite_spoils_its_block_alone(qb, fmt, per_row):
    w = normal((9, 200), 1.0, 3)
    w[0, 0], w[3, 77], w[8, 199] = float("inf"), float("nan"), float("-inf")
    x = f64(w)
    q = qb.qlora_mx_quantize(w.cuda(), fmt, per_row=per_row)
    same_as_oracle(q, x, fmt, per_row)
    back = f64(qb.qlora_mx_dequantize(q))
    want = mx.round_trip(x, fmt, per_row)
    assert np.array_equal(back, want, equal_nan=True)
    assert np.isnan(back).sum() == 2 * mx.BLOCK[fmt] + 200 % mx.BLOCK[fmt]
    t = qb.qlora_mx_quantize(w.cuda(), fmt, transpose=True)
    same_as_oracle(t, x.T, fmt, False)


@pytest.mark.parametrize("fmt,per_row", FORMS)
@pytest.mark.parametrize("rows,cols", [(1, 1), (129, 1000), (64, 128), (33, 8193)])
def test_dequantize_bit_for_bit(qb, rows, cols, fmt, per_row):
    x = f64(normal((rows, cols), 3.0, rows))
    q = upload(qb, x, fmt, per_row)
    assert np.array_equal(f64(qb.qlora_mx_dequantize(q)), mx.round_trip(x, fmt, per_row))


def test_dequantize_rounds_a_foreign_global_scale_once(qb):
    """A global scale that is no power of two: the product of three numbers of
    2, 4 and 24 bits, rounded to float (by 2^-24 of the value at most) and then
    to bf16, whose seven stored bits put values of [1, 2) 2^-7 apart: half a
    step is 2^-8 of the value."""
    x = f64(normal((64, 256), 1.0, 5))
    q = upload(qb, x, "nvfp4")
    q.global_scale.mul_(1.2345)
    want = mx.values(*mx.quantize(x, "nvfp4")[:2], q.global_scale.double().cpu().numpy(), "nvfp4")
    got = f64(qb.qlora_mx_dequantize(q))
    assert np.all(np.abs(got - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -23))


def test_zero_sized_and_given_destinations(qb):
    assert qb.qlora_mx_quantize(torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")).rows == 0
    w = normal((40, 96), 1.0, 2).cuda()
    out = qb.empty_mx(40, 96, w.device, "nvfp4")
    out.codes.fill_(0xAA)
    out.scales.fill_(0x7F)
    assert qb.qlora_mx_quantize(w, out=out) is out
    same_as_oracle(out, f64(w), "nvfp4", False)
    with pytest.raises(ValueError, match="describes"):
        qb.qlora_mx_quantize(w, out=qb.empty_mx(96, 40, w.device))
    back = torch.empty(40, 96, dtype=torch.bfloat16, device="cuda")
    assert qb.qlora_mx_dequantize(out, back) is back


# ---------------------------------------------------------------- the linear layer
def product_bound(y, x, w):
    """What the product may be off by: Y is rounded to bf16 once (half a step,
    2^-8 of the value); before that the tensor core adds 64 products at a time
    to an fp32 sum, each addition off by at most 2^-22 of the magnitudes that
    went in (a truncated 24-bit sum and its inner alignment)."""
    return np.abs(y) * 2.0 ** -8 + (x.shape[1] / 64 + 2) * 2.0 ** -22 * (np.abs(x) @ np.abs(w).T) + 1e-37


def check(got, want, bound, name):
    got = f64(got)
    assert got.shape == want.shape
    over = np.abs(got - want) - bound
    assert np.all(over <= 0), f"{name}: {np.sum(~(over <= 0))} of {over.size} off, worst {over.max():.3g} over the bound"


def lora_terms(x, a, b, s):
    """s (x a^T) b^T and what taking bf16(s x a^T) may put it off by, with the fp32 sum of x a^T."""
    xa = s * (x @ a.T)
    slack = np.abs(xa) * 2.0 ** -8 + abs(s) * (x.shape[1] / 16 + 2) * 2.0 ** -22 * (np.abs(x) @ np.abs(a).T)
    return xa @ b.T, slack @ np.abs(b).T + (b.shape[1] / 16 + 2) * 2.0 ** -22 * (np.abs(xa) @ np.abs(b).T)


LAYERS = [(1, 1, 1), (8, 64, 1), (128, 256, 1), (64, 64, 16), (300, 520, 17), (392, 640, 33), (256, 4096, 65),
          (130, 130, 129), (2048, 8192, 3), (1001, 1999, 77), (512, 1024, 300), (136, 90, 257), (4096, 96, 5),
          (129, 7000, 64), (300, 72, 129), (1030, 2100, 520), (520, 4096, 1030), (20000, 300, 2),
          (300, 20000, 9), (5000, 3000, 40), (45000, 96, 3), (70000, 40, 1), (1000, 9000, 7),
          (9472, 512, 12)]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("rows,cols,m", LAYERS)
def test_linear_fwd(qb, rows, cols, m, fmt):
    w, x = f64(normal((rows, cols), 0.02, 1)), normal((m, cols), 1.0, 2)
    q = upload(qb, w, fmt)
    Y, XA = qb.qlora_mx_linear_fwd(q, x.cuda())
    assert XA is None
    wv, xv = mx.round_trip(w, fmt), mx.round_trip(f64(x), fmt, True)
    check(Y, xv @ wv.T, product_bound(xv @ wv.T, xv, wv), "Y")


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("rows,cols,m,r", [(8, 64, 1, 8), (256, 256, 16, 8), (392, 640, 33, 64), (3000, 8192, 5, 64), (3000, 8192, 16, 64), (5000, 2048, 16, 256), (1000, 4096, 129, 136), (4096, 256, 64, 136),
                                           (2048, 704, 300, 256)])
def test_linear_fwd_with_an_adapter(qb, rows, cols, m, r, fmt):
    w, x = f64(normal((rows, cols), 0.02, 1)), normal((m, cols), 1.0, 2)
    a, b, s = normal((r, cols), 0.02, 3), normal((rows, r), 0.02, 4), 16.0 / r
    q = upload(qb, w, fmt)
    Y, XA = qb.qlora_mx_linear_fwd(q, x.cuda(), a.cuda(), b.cuda(), s)
    wv, xv = mx.round_trip(w, fmt), mx.round_trip(f64(x), fmt, True)
    term, slack = lora_terms(f64(x), f64(a), f64(b), s)
    want = xv @ wv.T + term
    check(Y, want, product_bound(want, xv, wv) + slack, "Y")
    check(XA, f64(x) @ f64(a).T, (cols / 16 + 2) * 2.0 ** -22 * (np.abs(f64(x)) @ np.abs(f64(a)).T), "XA")


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("rows,cols,m", [(1, 1, 1), (1999, 1001, 77), (640, 392, 16), (4096, 256, 300)])
def test_linear_bwd_without_an_adapter(qb, rows, cols, m, fmt):
    w, dy = normal((rows, cols), 0.02, 1), normal((m, rows), 1e-3, 2)
    qt = qb.qlora_mx_quantize(w.cuda(), fmt, transpose=True)
    dX, dA, dB = qb.qlora_mx_linear_bwd(qt, dy.cuda())
    assert dA is None and dB is None
    wt, gv = mx.round_trip(f64(w).T, fmt), mx.round_trip(f64(dy), fmt, True)
    check(dX, gv @ wt.T, product_bound(gv @ wt.T, gv, wt), "dX")


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("given_xa,need_dx", [(True, True), (False, True), (False, False)])
@pytest.mark.parametrize("rows,cols,m,r", [(256, 320, 7, 8), (392, 640, 200, 64), (136, 1024, 129, 136)])
def test_linear_bwd_with_an_adapter(qb, rows, cols, m, r, given_xa, need_dx, fmt):
    w, dy, x = normal((rows, cols), 0.02, 1), normal((m, rows), 1e-3, 2), normal((m, cols), 1.0, 5)
    a, b, s = normal((r, cols), 0.02, 3), normal((rows, r), 0.02, 4), 16.0 / r
    qt = qb.qlora_mx_quantize(w.cuda(), fmt, transpose=True)
    xa = (x.float() @ a.float().T).cuda() if given_xa else None
    dX, dA, dB = qb.qlora_mx_linear_bwd(qt, dy.cuda(), x.cuda(), a.cuda(), b.cuda(), s, XA=xa, need_dx=need_dx)
    X, dY, A, B = f64(x), f64(dy), f64(a), f64(b)
    term, slack = lora_terms(dY, B.T, A.T, s)
    if need_dx:
        wt, gv = mx.round_trip(f64(w).T, fmt), mx.round_trip(dY, fmt, True)
        want = gv @ wt.T + term
        check(dX, want, product_bound(want, gv, wt) + slack, "dX")
    else:
        assert dX is None
    # the rank-r operands of the gradients are taken as bf16 (2^-8 of each), the sums before and after in fp32
    sums = (max(rows, cols, m) / 16 + 4) * 2.0 ** -22
    G, XA = dY @ B, X @ A.T
    g_off = np.abs(G) * 2.0 ** -8 + sums * (np.abs(dY) @ np.abs(B))
    xa_off = np.abs(XA) * 2.0 ** -8 + sums * (np.abs(X) @ np.abs(A).T)
    check(dA, s * G.T @ X, s * (g_off.T @ np.abs(X)) + sums * s * (np.abs(G).T @ np.abs(X)), "dA")
    check(dB, s * dY.T @ XA, s * (np.abs(dY).T @ xa_off) + sums * s * (np.abs(dY).T @ np.abs(XA)), "dB")


def test_gradient_against_differences(qb):
    """<dX, v> against (f(x + h v) - f(x - h v)) / 2h of f(x) = <dy, Y(x)> with
    x and x +- h v on the quantiser's grid, where q is the identity.  W too lies
    on the grid in both directions (every block of rows and of columns holds a 6
    and multiples of 1/2), and dy as well, so both sides are sums of products of
    multiples of 1/2: exact but for one rounding of Y and dX to bf16 each."""
    rows, cols, m = 64, 96, 32
    rng = np.random.default_rng(0)
    lv = np.array([-4.0, -3, -2, -1.5, -1, -0.5, 0, 0.5, 1, 1.5, 2, 3, 4])
    w = rng.choice(lv, (rows, cols))
    np.fill_diagonal(w[:, :64], 6.0)
    w[0::32, :] = 6.0
    w[:, 0::32] = 6.0
    x = rng.choice([-2.0, -1, 0, 1, 2], (m, cols))
    x[:, 0::32] = 6.0
    v = rng.choice([-1.0, 0, 1], (m, cols))
    v[:, 0::32] = 0.0
    dy = rng.choice([-2.0, -1, 0, 1, 2, 4], (m, rows))
    dy[:, 0::32] = 6.0
    t = lambda z: torch.from_numpy(z).to(torch.bfloat16).cuda()  # noqa: E731
    q, qt = qb.qlora_mx_quantize(t(w)), qb.qlora_mx_quantize(t(w), transpose=True)
    assert np.array_equal(f64(qb.qlora_mx_dequantize(q)), w) and np.array_equal(f64(qb.qlora_mx_dequantize(qt)), w.T)
    dX = f64(qb.qlora_mx_linear_bwd(qt, t(dy))[0])
    up = f64(qb.qlora_mx_linear_fwd(q, t(x + v))[0])
    down = f64(qb.qlora_mx_linear_fwd(q, t(x - v))[0])
    left, right = (dX * v).sum(), (dy * (up - down)).sum() / 2
    slack = 2.0 ** -8 * ((np.abs(dX) * np.abs(v)).sum() + (np.abs(dy) * (np.abs(up) + np.abs(down))).sum() / 2)
    assert abs(left - right) <= slack
    exact = ((dy @ w) * v).sum()
    assert abs(left - exact) <= 2.0 ** -8 * (np.abs(dy @ w) * np.abs(v)).sum()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("m", [1, 40, 200])
def test_linear_is_bit_reproducible_and_token_independent(qb, m, fmt):
    """The same call twice gives the same bits, and a token's result does not
    depend on which tokens share its tile."""
    w, x = normal((520, 3000), 0.02, 1).cuda(), normal((m, 3000), 1.0, 2).cuda()
    q = qb.qlora_mx_quantize(w, fmt)
    first = qb.qlora_mx_linear_fwd(q, x)[0]
    for _ in range(5):
        assert torch.equal(qb.qlora_mx_linear_fwd(q, x)[0], first)
    if m > 1:
        other = x.clone()
        other[1:] *= 100.0
        assert torch.equal(qb.qlora_mx_linear_fwd(q, other)[0][0], first[0])


def test_linear_nan_stays_in_its_row(qb):
    w, x = normal((200, 512), 0.02, 1).cuda(), normal((20, 512), 1.0, 2).cuda()
    for fmt in ("mxfp4", "nvfp4"):
        q = qb.qlora_mx_quantize(w, fmt)
        clean = qb.qlora_mx_linear_fwd(q, x)[0]
        bad = x.clone()
        bad[3, 100], bad[19, 0] = float("nan"), float("inf")
        got = qb.qlora_mx_linear_fwd(q, bad)[0]
        assert got[3].isnan().all() and got[19].isnan().all()
        keep = [i for i in range(20) if i not in (3, 19)]
        assert torch.equal(got[keep], clean[keep])


def test_linear_refusals(qb):
    q = qb.qlora_mx_quantize(normal((64, 128)).cuda(), "nvfp4")
    x = normal((4, 128)).cuda()
    a, b = normal((8, 128)).cuda(), normal((64, 8)).cuda()
    for bad in (x.float(), x[:, :64], normal((128, 4)).cuda().t(), x.cpu()):
        with pytest.raises(ValueError, match="X"):
            qb.qlora_mx_linear_fwd(q, bad)
    with pytest.raises(ValueError, match="together"):
        qb.qlora_mx_linear_fwd(q, x, a)
    with pytest.raises(ValueError, match="B"):
        qb.qlora_mx_linear_fwd(q, x, a, b.t().contiguous())
    with pytest.raises(qb.QloraError, match="work buffer"):
        qb.qlora_mx_linear_fwd(q, x, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(qb.QloraError, match="shape"):
        qb.qlora_mx_linear_fwd(q, x[:0])
    with pytest.raises(qb.QloraError, match="shape"):          # an adapter needs cols % 64 == 0
        odd = qb.qlora_mx_quantize(normal((64, 72)).cuda())
        qb.qlora_mx_linear_fwd(odd, normal((4, 72)).cuda(), normal((8, 72)).cuda(), b)
    per_row = qb.qlora_mx_quantize(normal((64, 128)).cuda(), "nvfp4", per_row=True)
    with pytest.raises(qb.QloraError, match="unsupported"):
        qb.qlora_mx_linear_fwd(per_row, x, a, b)
    with pytest.raises(ValueError, match="need X"):
        qb.qlora_mx_linear_bwd(q, normal((4, 128)).cuda(), A=normal((8, 64)).cuda(), B=normal((128, 8)).cuda())


@pytest.mark.parametrize("m", [1, 5, 16, 40, 150])
def test_linear_with_a_scale_per_weight_row(qb, m):
    w, x = f64(normal((200, 300), 0.02, 1)) * np.logspace(-3, 3, 200)[:, None], normal((m, 300), 1.0, 2)
    w = f64(torch.from_numpy(w).to(torch.bfloat16))
    q = upload(qb, w, "nvfp4", True)
    wv, xv = mx.round_trip(w, "nvfp4", True), mx.round_trip(f64(x), "nvfp4", True)
    check(qb.qlora_mx_linear_fwd(q, x.cuda())[0], xv @ wv.T, product_bound(xv @ wv.T, xv, wv), "Y")


def test_rows_behind_the_last_token_are_left_as_they_were(qb):
    w, x = normal((200, 320), 0.02, 1).cuda(), normal((77, 320), 1.0, 2).cuda()
    q = qb.qlora_mx_quantize(w)
    whole = torch.full((90, 200), 7.0, dtype=torch.bfloat16, device="cuda")
    qb.qlora_mx_linear_fwd(q, x, Y=whole[:77])
    assert (whole[77:] == 7).all() and torch.equal(whole[:77], qb.qlora_mx_linear_fwd(q, x)[0])


@pytest.mark.parametrize("m", [3, 300])
def test_linear_on_another_stream_and_in_a_graph(qb, m):
    """A side stream while another call runs, and a captured call replayed on new inputs."""
    w = normal((512, 2048), 0.02, 1).cuda()
    q = qb.qlora_mx_quantize(w, "nvfp4")
    xs = [normal((m, 2048), 1.0, i).cuda() for i in range(4)]
    want = [qb.qlora_mx_linear_fwd(q, x)[0] for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [qb.qlora_mx_linear_fwd(q, x)[0] for x in xs]
    again = [qb.qlora_mx_linear_fwd(q, x)[0] for x in xs]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and all(torch.equal(a, b) for a, b in zip(want, again))
    static = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = qb.qlora_mx_linear_fwd(q, static)[0]
    for x, y in zip(xs, want):
        static.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y)


# ---------------------------------------------------------------- mixture of experts
def moe_case(qb, experts, hidden, inner, m, seed=0, std=0.05):
    w13, w2 = normal((experts * 2 * inner, hidden), std, seed), normal((experts * hidden, inner), std, seed + 1)
    router, x = normal((experts, hidden), std, seed + 2), normal((m, hidden), 1.0, seed + 3)
    q13, q2 = qb.qlora_mx_quantize(w13.cuda()), qb.qlora_mx_quantize(w2.cuda())
    return q13, q2, router.cuda(), x.cuda()


def moe_reference(qb, q13, q2, router, x, top_k):
    """(ids, p, y, what y may be off by).  h reaches its quantiser off by the
    product's own error; where that can move a code (or a block's scale) to its
    neighbour, the difference of the two values counts."""
    E, H, F = router.shape[0], q13.cols, q2.cols
    w13 = f64(qb.qlora_mx_dequantize(q13)).reshape(E, 2, F, H)
    w2 = f64(qb.qlora_mx_dequantize(q2)).reshape(E, H, F)
    X = f64(x)
    xv = mx.round_trip(X, "mxfp4")
    logits = X @ f64(router).T
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :top_k]
    top = np.take_along_axis(logits, ids, 1)
    p = np.exp(top - top[:, :1])
    p /= p.sum(1, keepdims=True)
    y, off = np.zeros((len(X), H)), np.zeros((len(X), H))
    with np.errstate(over="ignore"):
        for t in range(len(X)):
            for j, e in enumerate(ids[t]):
                g, u = w13[e, 0] @ xv[t], w13[e, 1] @ xv[t]
                dg, du = ((H / 64 + 2) * 2.0 ** -22 * (np.abs(w) @ np.abs(xv[t])) for w in w13[e])
                silu = g / (1 + np.exp(-g))
                h = silu * u
                d = 1.1 * np.abs(u) * dg + np.abs(silu) * du + dg * du + 2.0 ** -20 * np.abs(h)     # |silu'| < 1.1
                hv = mx.round_trip(h[None], "mxfp4")[0]
                b, db = h.reshape(-1, 32), d.reshape(-1, 32)
                slack = np.zeros_like(b)
                for sign in (-1, 1):
                    amax = np.maximum((np.abs(b) + sign * db).max(1), 0)
                    exp = np.where(amax > 0, np.frexp(amax)[1] - 3, -127).clip(-127)
                    step = 2.0 ** exp.astype(float)[:, None]
                    for v in (b - db, b, b + db):
                        val = mx.LEVELS[mx.nearest_code(np.abs(v) / step)] * np.sign(v) * step
                        slack = np.maximum(slack, np.abs(val - hv.reshape(-1, 32)))
                o = w2[e] @ hv
                y[t] += p[t, j] * o
                off[t] += p[t, j] * (np.abs(w2[e]) @ slack.ravel() + (F / 64 + 4) * 2.0 ** -22 * (np.abs(w2[e]) @ np.abs(hv))
                                     + 2.0 ** -18 * np.abs(o))      # p: the logits' error, exp and a division
    return ids, p, y, off + np.abs(y) * 2.0 ** -8 + 1e-37


@pytest.mark.parametrize("experts,hidden,inner,m,top_k", [
    (1, 128, 128, 1, 1), (4, 256, 128, 1, 2), (8, 384, 256, 16, 8), (16, 512, 384, 5, 3), (64, 1024, 128, 16, 6),
    (33, 640, 128, 9, 16), (250, 256, 128, 16, 10), (5, 128, 1152, 3, 1), (2, 2048, 640, 16, 2)])
def test_moe(qb, experts, hidden, inner, m, top_k):
    q13, q2, router, x = moe_case(qb, experts, hidden, inner, m, experts + m)
    ids, p, y, off = moe_reference(qb, q13, q2, router, x, top_k)
    Y, got_ids, got_p = qb.qlora_mx_moe_fwd(q13, q2, router, x, top_k)
    assert np.array_equal(got_ids.cpu().numpy(), ids)
    assert np.all(np.abs(f64(got_p) - p) <= p * 2.0 ** -17)
    check(Y, y, off, "Y")
    for _ in range(3):
        assert torch.equal(qb.qlora_mx_moe_fwd(q13, q2, router, x, top_k)[0], Y)


def test_moe_ties_take_the_lowest_index(qb):
    q13, q2, router, x = moe_case(qb, 40, 256, 128, 6)
    router[:] = router[:1]
    assert torch.equal(qb.qlora_mx_moe_fwd(q13, q2, router, x, 5)[1].cpu(), torch.arange(5, dtype=torch.int32).expand(6, 5))
    router[20:] *= -1
    router[0] = 0                                             # logit 0 between the two groups
    ids = qb.qlora_mx_moe_fwd(q13, q2, router, x, 16)[1].cpu().numpy()
    logits = f64(x) @ f64(router).T
    assert np.array_equal(ids, np.argsort(-logits, axis=1, kind="stable")[:, :16])


def test_moe_every_token_on_one_expert_and_far_apart_logits(qb):
    q13, q2, router, x = moe_case(qb, 8, 256, 128, 16, 5)
    x[:, 0] = 8.0
    router[:, 0] = torch.arange(8, device="cuda").to(torch.bfloat16) * 40          # expert 7 always wins, by hundreds
    ids, p, y, off = moe_reference(qb, q13, q2, router, x, 3)
    Y, got_ids, got_p = qb.qlora_mx_moe_fwd(q13, q2, router, x, 3)
    assert np.array_equal(got_ids.cpu().numpy(), ids) and (got_p[:, 0] == 1).all() and (got_p[:, 1:] == 0).all()
    check(Y, y, off, "Y")


def test_moe_nan_token_stays_alone(qb):
    q13, q2, router, x = moe_case(qb, 8, 256, 128, 4, 7)
    clean = qb.qlora_mx_moe_fwd(q13, q2, router, x, 2)[0]
    bad = x.clone()
    bad[2, 5] = float("nan")
    Y, ids, _ = qb.qlora_mx_moe_fwd(q13, q2, router, bad, 2)
    assert Y[2].isnan().all() and ((ids >= 0) & (ids < 8)).all()
    assert torch.equal(Y[[0, 1, 3]], clean[[0, 1, 3]])


def test_moe_in_a_graph_with_a_workspace_of_its_own(qb):
    q13, q2, router, x = moe_case(qb, 16, 512, 256, 4, 9)
    xs = [normal((4, 512), 1.0, 50 + i).cuda() for i in range(3)]
    want = [qb.qlora_mx_moe_fwd(q13, q2, router, v, 4) for v in xs]
    ws = torch.full((qb.qlora_mx_moe_workspace_size(16, 512, 256, 4, 4),), 0xFF, dtype=torch.uint8, device="cuda")
    static = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = qb.qlora_mx_moe_fwd(q13, q2, router, static, 4, workspace=ws)
    for v, w in zip(xs, want):
        static.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, w))


def test_moe_refusals(qb):
    q13, q2, router, x = moe_case(qb, 4, 256, 128, 3)
    with pytest.raises(ValueError, match="rows"):
        qb.qlora_mx_moe_fwd(q13, q2, router[:3], x, 2)
    with pytest.raises(ValueError, match="X"):
        qb.qlora_mx_moe_fwd(q13, q2, router, x.float(), 2)
    with pytest.raises(qb.QloraError, match="shape"):
        qb.qlora_mx_moe_fwd(q13, q2, router, x, 5)
    with pytest.raises(qb.QloraError, match="shape"):
        qb.qlora_mx_moe_fwd(q13, q2, router, normal((17, 256)).cuda(), 2)
    nv = qb.qlora_mx_quantize(normal((4 * 256, 256)).cuda(), "nvfp4")
    with pytest.raises(qb.QloraError, match="unsupported"):
        qb.qlora_mx_moe_fwd(nv, q2, router, x, 2)


def test_layers_in_a_row(qb):
    """A block as it would be used: a projection with its adapter, the routed
    layer, a projection back; each step is checked in its own test, here the
    chain must equal the same chain on dequantised inputs of each step."""
    m, H, F, E = 8, 512, 256, 8
    q13, q2, router, x = moe_case(qb, E, H, F, m, 21)
    w1, w2 = normal((H, H), 0.05, 1).cuda(), normal((H, H), 0.05, 2).cuda()
    a, b = normal((16, H), 0.05, 3).cuda(), normal((H, 16), 0.05, 4).cuda()
    qa, qc = qb.qlora_mx_quantize(w1, "nvfp4"), qb.qlora_mx_quantize(w2, "mxfp4")
    y1, _ = qb.qlora_mx_linear_fwd(qa, x, a, b, 0.5)
    y2, _, _ = qb.qlora_mx_moe_fwd(q13, q2, router, y1, 2)
    y3, _ = qb.qlora_mx_linear_fwd(qc, y2)
    xv, wv = mx.round_trip(f64(x), "nvfp4", True), f64(qb.qlora_mx_dequantize(qa))
    term, slack = lora_terms(f64(x), f64(a), f64(b), 0.5)
    check(y1, xv @ wv.T + term, product_bound(xv @ wv.T + term, xv, wv) + slack, "first")
    _, _, want, off = moe_reference(qb, q13, q2, router, y1, 2)
    check(y2, want, off, "experts")
    xv, wv = mx.round_trip(f64(y2), "mxfp4"), f64(qb.qlora_mx_dequantize(qc))
    check(y3, xv @ wv.T, product_bound(xv @ wv.T, xv, wv), "last")
    dy = normal((m, H), 1e-3, 9).cuda()
    qct = qb.qlora_mx_quantize(w2, "mxfp4", transpose=True)
    d2 = qb.qlora_mx_linear_bwd(qct, dy)[0]
    gv, wt = mx.round_trip(f64(dy), "mxfp4"), f64(qb.qlora_mx_dequantize(qct))
    check(d2, gv @ wt.T, product_bound(gv @ wt.T, gv, wt), "back")


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("m,r", [(1, 0), (3, 64), (16, 8), (40, 64), (64, 0), (200, 64)])
def test_work_buffers_may_hold_anything(qb, m, r, fmt):
    """A work buffer full of NaN patterns gives what a fresh one gives, forward and backward."""
    rows, cols = 520, 1344
    w, x, dy = normal((rows, cols), 0.02, 1).cuda(), normal((m, cols), 1.0, 2).cuda(), normal((m, rows), 1e-3, 3).cuda()
    q, qt = qb.qlora_mx_quantize(w, fmt), qb.qlora_mx_quantize(w, fmt, transpose=True)
    a, b = (normal((r, cols), 0.02, 4).cuda(), normal((rows, r), 0.02, 5).cuda()) if r else (None, None)
    f, g = qb.qlora_mx_linear_workspace_size(rows, cols, fmt, m, r)
    for fill in (0xFF, 0x7F):
        ws = torch.full((max(f, g),), fill, dtype=torch.uint8, device="cuda")
        got = qb.qlora_mx_linear_fwd(q, x, a, b, 0.25, workspace=ws)
        want = qb.qlora_mx_linear_fwd(q, x, a, b, 0.25)
        assert all(torch.equal(u, v) for u, v in zip(got, want) if u is not None)
        ws.fill_(fill)
        back = qb.qlora_mx_linear_bwd(qt, dy, x, a, b, 0.25, workspace=ws)
        want = qb.qlora_mx_linear_bwd(qt, dy, x, a, b, 0.25)
        if m > 16 or not r:                       # with fewer tokens dA and dB are as of qlora_linear_bwd: no split
            assert all(torch.equal(u, v) for u, v in zip(back, want) if u is not None)
        else:
            assert torch.equal(back[0], want[0])


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("m", [1, 20, 150])
def test_zeros_and_far_magnitudes(qb, m, fmt):
    """Zero tokens give exact zeros; tokens of 2^40 and 2^-40 (and zeros between
    them) give the result of tokens of 1, scaled."""
    w, x = normal((300, 640), 0.02, 1).cuda(), normal((m, 640), 1.0, 2).cuda()
    q = qb.qlora_mx_quantize(w, fmt)
    assert (qb.qlora_mx_linear_fwd(q, torch.zeros_like(x))[0] == 0).all()
    y = qb.qlora_mx_linear_fwd(q, x)[0]
    for e in (40, -40):
        assert torch.equal(qb.qlora_mx_linear_fwd(q, x * 2.0 ** e)[0], y * 2.0 ** e)
    x[0] = 0
    y2 = qb.qlora_mx_linear_fwd(q, x)[0]
    assert (y2[0] == 0).all() and torch.equal(y2[1:], y[1:])
    z = qb.qlora_mx_quantize(torch.zeros_like(w), fmt)
    assert (qb.qlora_mx_linear_fwd(z, x)[0] == 0).all() and (qb.qlora_mx_dequantize(z) == 0).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("m", [1, 12, 40, 150])
def test_adapter_with_far_magnitudes(qb, m, fmt):
    """Tokens and gradients of 2^-100 and 2^100 give the result of ones of 1, scaled:
    the rank-r term rides on global scales whose product no float holds."""
    rows, cols, r = 256, 640, 64
    w, x, dy = normal((rows, cols), 0.02, 1).cuda(), normal((m, cols), 1.0, 2).cuda(), normal((m, rows), 1.0, 3).cuda()
    a, b = normal((r, cols), 0.02, 4).cuda(), normal((rows, r), 0.02, 5).cuda()
    q, qt = qb.qlora_mx_quantize(w, fmt), qb.qlora_mx_quantize(w, fmt, transpose=True)
    y, d = qb.qlora_mx_linear_fwd(q, x, a, b, 0.25)[0], qb.qlora_mx_linear_bwd(qt, dy, x, a, b, 0.25)[0]
    for e in (-100, 100):
        assert torch.equal(qb.qlora_mx_linear_fwd(q, x * 2.0 ** e, a, b, 0.25)[0], y * 2.0 ** e)
        assert torch.equal(qb.qlora_mx_linear_bwd(qt, dy * 2.0 ** e, x, a, b, 0.25)[0], d * 2.0 ** e)


def test_offsets_past_32_bits(qb):
    """2.4e9 weights (4.8 GB): the last rows are quantised, dequantised and
    multiplied as they are alone."""
    rows, cols, tail = 40000, 60000, 192          # 40000 = 312 * 128 + 64: the tail begins on a scale tile
    w = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    w.normal_(std=0.02, generator=torch.Generator(device="cuda").manual_seed(1))
    q, small = qb.qlora_mx_quantize(w), qb.qlora_mx_quantize(w[rows - tail:].contiguous())
    pitch = -(-cols // 32) * 16
    assert torch.equal(q.codes[-tail * pitch:], small.codes) and torch.equal(q.scales[-small.scales.numel():], small.scales)
    for m in (1, 16, 50, 200):
        x = normal((m, cols), 1.0, m).cuda()
        assert torch.equal(qb.qlora_mx_linear_fwd(q, x)[0][:, rows - tail:], qb.qlora_mx_linear_fwd(small, x)[0])
    assert torch.equal(qb.qlora_mx_dequantize(q)[rows - tail:], qb.qlora_mx_dequantize(small))
    del q
    t = qb.qlora_mx_quantize(w, transpose=True)   # rows of w are its contraction
    last = qb.qlora_mx_quantize(w[:, cols - 96:].contiguous(), transpose=True)
    tp = -(-rows // 32) * 16
    assert torch.equal(t.codes[-96 * tp:], last.codes)


def test_two_calls_at_once(qb):
    """Calls of different kinds on two streams, each with its own work buffers, give what they give alone."""
    w, x, big = normal((3000, 2048), 0.02, 1).cuda(), normal((5, 2048), 1.0, 2).cuda(), normal((700, 2048), 1.0, 3).cuda()
    q = qb.qlora_mx_quantize(w, "nvfp4")
    q13, q2, router, xe = moe_case(qb, 16, 512, 256, 9, 4)
    jobs = [lambda: qb.qlora_mx_linear_fwd(q, x)[0], lambda: qb.qlora_mx_linear_fwd(q, big)[0],
            lambda: qb.qlora_mx_moe_fwd(q13, q2, router, xe, 4)[0], lambda: qb.qlora_mx_quantize(big, "nvfp4").codes,
            lambda: qb.qlora_mx_linear_fwd(q, big[:40].contiguous())[0]]
    want = [j() for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] += [j() for j in (jobs if i == 0 else jobs[::-1])]
    torch.cuda.synchronize()
    for k in range(25):
        assert torch.equal(got[0][k], want[k % 5]) and torch.equal(got[1][k], want[4 - k % 5])


@pytest.mark.parametrize("m,r", [(1, 0), (1, 64), (30, 0), (300, 64)])
def test_inputs_that_arrive_just_before(qb, m, r):
    """The tokens are written by a copy, or by another stream that is waited for,
    right before the call; eagerly and in a captured graph."""
    w = normal((11008, 1024), 0.02, 1).cuda()
    q = qb.qlora_mx_quantize(w, "nvfp4")
    a, b = (normal((r, 1024), 0.02, 4).cuda(), normal((11008, r), 0.02, 5).cuda()) if r else (None, None)
    xs = [normal((m, 1024), 1.0, i).cuda() for i in range(3)]
    want = [qb.qlora_mx_linear_fwd(q, x, a, b, 0.25)[0] for x in xs]
    x, src, side = xs[0].clone(), xs[0].clone(), torch.cuda.Stream()

    def copied():
        x.copy_(src)
        return qb.qlora_mx_linear_fwd(q, x, a, b, 0.25)[0]

    def from_another_stream():
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            w.float().sum()
            x.copy_(src)
        torch.cuda.current_stream().wait_stream(side)
        return qb.qlora_mx_linear_fwd(q, x, a, b, 0.25)[0]

    for call in (copied, from_another_stream):
        for v, y in zip(xs, want):
            src.copy_(v)
            assert torch.equal(call(), y)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call()
        for v, y in zip(xs, want):
            src.copy_(v)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, y)


def test_weight_quantised_just_before(qb):
    """Quantise, use, overwrite and use again without a wait between."""
    ws = [normal((4096, 1024), 0.02, i).cuda() for i in range(4)]
    x = normal((2, 1024), 1.0, 9).cuda()
    for fmt in ("mxfp4", "nvfp4"):
        want = []
        for w in ws:
            want.append(qb.qlora_mx_linear_fwd(qb.qlora_mx_quantize(w, fmt), x)[0])
            torch.cuda.synchronize()
        out, got = qb.empty_mx(4096, 1024, x.device, fmt), []
        for _ in range(5):
            for w in ws:
                got.append(qb.qlora_mx_linear_fwd(qb.qlora_mx_quantize(w, out=out), x)[0])
        torch.cuda.synchronize()
        assert all(torch.equal(g, want[i % 4]) for i, g in enumerate(got))
