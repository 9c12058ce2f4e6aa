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
          (300, 16), (33, 8193)]


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
