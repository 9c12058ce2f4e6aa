"""The rank-r branch of the microscaled layer on the GPU: what its sums and
operands may be off by, where the weight itself contributes nothing."""
import numpy as np
import pytest
import torch

from test_gpu_mx import check, f64, no_device_errors, normal, qb  # noqa: F401

pytestmark = pytest.mark.gpu

# A float carried as two bf16 parts: the first is off by 2^-8 of it at most, the second by 2^-9 of that.
PARTS = 2.0 ** -17


def sums(n):
    """An fp32 sum of n products taken 16 at a time, each addition off by at most 2^-22 of the magnitudes."""
    return (n / 16 + 2) * 2.0 ** -22


def term_and_bound(x, a, b, s):
    """s (x a^T) b^T rounded to bf16 once, its middle factor carried as two bf16 parts (after one multiplication
    by s and two divisions in fp32), all sums fp32."""
    xa, mag = s * (x @ a.T), abs(s) * (np.abs(x) @ np.abs(a).T)
    off = np.abs(xa) * (PARTS + 2.0 ** -22) + sums(x.shape[1]) * mag
    want = xa @ b.T
    return want, np.abs(want) * 2.0 ** -8 + off @ np.abs(b).T + sums(2 * b.shape[1]) * (np.abs(xa) @ np.abs(b).T)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("rows,cols,m,r", [(520, 256, 1, 64), (2048, 256, 12, 136), (520, 320, 40, 64), (520, 256, 64, 256),
                                           (392, 320, 150, 136), (256, 256, 300, 8)])
def test_adapter_term_is_not_taken_from_rounded_operands(qb, rows, cols, m, r, fmt):  # noqa: F811
    """Over a weight of zeros the layer is the rank-r term alone, and where its 64
    or more products nearly cancel an operand of eight bits would show."""
    a, b, s = normal((r, cols), 0.02, 3), normal((rows, r), 0.02, 4), 16.0 / r
    x, dy = normal((m, cols), 1.0, 2), normal((m, rows), 1.0, 5)
    q = qb.qlora_mx_quantize(torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda"), fmt)
    qt = qb.qlora_mx_quantize(torch.zeros(cols, rows, dtype=torch.bfloat16, device="cuda"), fmt)
    Y, _ = qb.qlora_mx_linear_fwd(q, x.cuda(), a.cuda(), b.cuda(), s)
    check(Y, *term_and_bound(f64(x), f64(a), f64(b), s), "Y")
    dX, _, _ = qb.qlora_mx_linear_bwd(qt, dy.cuda(), x.cuda(), a.cuda(), b.cuda(), s)
    check(dX, *term_and_bound(f64(dy), f64(b).T, f64(a).T, s), "dX")


def gradient_and_bound(g, x, k, s, exact):
    """s g^T x with g a sum of k products (magnitudes `exact` of them summed): g, times s, carried as two bf16
    parts, the tokens summed in fp32."""
    m = len(x)
    want = s * g.T @ x
    off = np.abs(g) * (PARTS + 2.0 ** -22) + sums(k) * exact
    return want, abs(s) * (off.T @ np.abs(x) + sums(2 * m) * (np.abs(g).T @ np.abs(x))) + 2.0 ** -23 * np.abs(want)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("given_xa", [True, False])
@pytest.mark.parametrize("rows,cols,m,r", [(72, 128, 5, 8), (72, 128, 17, 136), (136, 64, 40, 64), (72, 128, 64, 256), (64, 192, 300, 64),
                                           (1000, 64, 150, 72)])
def test_adapter_gradients_are_not_taken_from_rounded_operands(qb, rows, cols, m, r, given_xa, fmt):  # noqa: F811
    a, b, s = normal((r, cols), 0.02, 3), normal((rows, r), 0.02, 4), 16.0 / r
    x, dy = normal((m, cols), 1.0, 2), normal((m, rows), 1.0, 5)
    qt = qb.qlora_mx_quantize(normal((rows, cols), 0.02, 1).cuda(), fmt, transpose=True)
    X, dY, A, B = f64(x), f64(dy), f64(a), f64(b)
    xa = torch.from_numpy(X @ A.T).float().cuda() if given_xa else None
    dA, dB = qb.qlora_mx_linear_bwd(qt, dy.cuda(), x.cuda(), a.cuda(), b.cuda(), s, XA=xa)[1:]
    check(dA, *gradient_and_bound(dY @ B, X, rows, s, np.abs(dY) @ np.abs(B)), "dA")
    want, bound = gradient_and_bound(X @ A.T, dY, cols, s, np.abs(X) @ np.abs(A).T)
    check(dB, want.T, bound.T, "dB")


# A sum of n positive numbers whose parts of 512 are taken on the tensor core, 32 additions off by 2^-22 of the part
# at most, and added up in fp32, off by 2^-24 each.
def long_sum(n):
    return 32 * 2.0 ** -22 + n / 512 * 2.0 ** -24


def positive(shape, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(shape, generator=gen, device="cuda").add_(0.5).to(torch.bfloat16)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_long_contractions_of_the_backward_do_not_drift(qb, fmt):  # noqa: F811
    """Sums of 65536 positive products, in problems with enough tiles that no
    contraction is split.  One token per column (row) of X (dY) brings a single G
    (X A^T) to dA (dB) as it is; a one-hot dY makes G exact and leaves the sum
    over the tokens."""
    n, m, r, s = 65536, 148 * 128, 8, 1.0
    eye = torch.zeros(m, 64, dtype=torch.bfloat16, device="cuda")
    eye[:64] = torch.eye(64)
    long = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    long[:64] = positive((64, n), 1)
    low, wide = positive((n, r), 2), positive((r, 64), 3)
    zeros = lambda *z: qb.qlora_mx_quantize(torch.zeros(*z, dtype=torch.bfloat16, device="cuda"), fmt)  # noqa: E731
    want = f64(long[:64]) @ f64(low)
    # G = dY B
    dA = qb.qlora_mx_linear_bwd(zeros(64, n), long, eye, wide, low, s, XA=torch.zeros(m, r, device="cuda"), need_dx=False)[1]
    check(dA, want.T, (long_sum(n) + PARTS) * want.T, "dA of G")
    # X A^T, recomputed
    dB = qb.qlora_mx_linear_bwd(zeros(n, 64), eye, long, low.t().contiguous(), wide.t().contiguous(), s, need_dx=False)[2]
    check(dB, want, (long_sum(n) + PARTS) * want, "dB of X A^T")
    # the sum over the tokens
    del long
    x = positive((n, m), 4)
    hot = torch.zeros(n, 64, dtype=torch.bfloat16, device="cuda")
    hot[:, 0] = 1
    b = positive((64, r), 5)
    dA = qb.qlora_mx_linear_bwd(zeros(m, 64), hot, x, positive((r, m), 6), b, s, XA=torch.zeros(n, r, device="cuda"), need_dx=False)[1]
    want = f64(b)[0][:, None] * f64(sum(p.double().sum(0) for p in x.split(4096)))
    check(dA, want, (long_sum(n) + 2.0 ** -22) * want, "dA over the tokens")
