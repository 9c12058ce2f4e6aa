"""The host side of the microscaled operators (no GPU): sizes, refusals and which
form a call takes."""
import ctypes

import pytest

qb = pytest.importorskip("bit_nf4_quantized_encode_b200")
lib = qb._lib


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_backward_of_few_tokens_reserves_no_dx_in_fp32(fmt):
    """Between a layer of 64 and one of 65536 columns the work buffer grows by
    counters and at most 32 partial tiles of 32 KB, not by [m, cols] floats."""
    wide, narrow = (qb.qlora_mx_linear_workspace_size(4096, c, fmt, 16, 8)[1] for c in (65536, 64))
    assert wide - narrow < 16 * (65536 - 64) * 4 // 2


def test_quantize_refuses_a_work_buffer_elsewhere(monkeypatch):
    """A caller's work buffer on another device, or with gaps, does not reach the library."""
    import torch

    monkeypatch.setattr(qb, "_need_bf16_cuda", lambda name, t: None)
    monkeypatch.setattr(qb.MXTensor, "c_struct", lambda self: None)
    calls = []
    monkeypatch.setattr(qb, "_on", lambda device, where, fn, *args: calls.append(where))
    w, out = torch.zeros(1024, 1024, dtype=torch.bfloat16), qb.empty_mx(1024, 1024, "cpu", "nvfp4")
    for bad in (torch.empty(8192, dtype=torch.uint8, device="meta"), torch.empty(16384, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            qb.qlora_mx_quantize(w, out=out, workspace=bad)
    assert not calls
    qb.qlora_mx_quantize(w, out=out, workspace=torch.empty(8192, dtype=torch.uint8))
    assert calls == ["qlora_mx_quantize"]


def test_import_without_torchs_private_stream_getter():
    """The stream handle comes from torch's private getter where there is one, else from the public call."""
    import subprocess
    import sys
    code = ("import torch; del torch._C._cuda_getCurrentRawStream; import bit_nf4_quantized_encode_b200 as qb; "
            "torch.cuda.current_stream = lambda i: type('S', (), {'cuda_stream': 40 + i}); assert qb._raw_stream(2) == 42")
    subprocess.run([sys.executable, "-c", code], check=True)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_form_of_a_product(fmt):
    form = lambda *a, **k: qb.qlora_selftest_mx_form(*a[:2], fmt, *a[2:], **k)  # noqa: E731
    assert form(22016, 8192, 1) == ("few", 8) and form(8192, 22016, 16, 64) == ("stream", 16)
    assert form(22016, 8192, 1, backward=True) == ("stream", 16)
    assert form(512, 512, 17) == ("stream", 32) and form(512, 512, 64) == ("stream", 64)
    assert form(512, 512, 65) == ("pair", 128)
    assert form(8192, 8192, 8192) == ("pair", 256) and form(8192, 320, 8192, 64, backward=True)[0] == "pair"
    f = lib.qlora_selftest_mx_form
    out = ctypes.c_int32()
    assert f(64, 64, 7, 4, 0, 0, 148, out, out) == -4 and f(64, 64, 0, 0, 0, 0, 148, out, out) == -2
    assert f(64, 64, 0, 4, 0, 0, 1, out, out) == -2 and f(64, 64, 0, 4, 0, 0, 148, None, out) == -1


@pytest.mark.parametrize("rows,cols,m,r", [(2048, 4096, 1, 0), (8192, 4096, 4, 16), (2048, 2048, 8, 0), (4096, 2048, 8, 64)])
def test_nvfp4_leaves_one_launch_earlier(rows, cols, m, r):
    """Where the quantisation within the product costs NVFP4 more than a launch (16 to 23% measured)."""
    assert qb.qlora_selftest_mx_form(rows, cols, "nvfp4", m, r) == ("stream", 16)
    assert qb.qlora_selftest_mx_form(rows, cols, "mxfp4", 1) == ("few", 8)
