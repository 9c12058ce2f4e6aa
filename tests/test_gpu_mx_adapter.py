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
