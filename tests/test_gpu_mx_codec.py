"""MX quantiser and dequantiser on the GPU against the float64 oracle, bit for
bit: codes, scale bytes and element values."""
import numpy as np
import pytest
import torch

from oracle import mx as omx
from qlora_parameter_efficient_amd import mx
from tests.gpu_helpers import DEV, announce

pytestmark = pytest.mark.gpu

SRC = {"bf16": torch.bfloat16, "f32": torch.float32}


def check(X, fmt, what=""):
    announce(f"mx codec {fmt} {X.dtype} {tuple(X.shape)} {what}")
    rows, cols = X.shape
    qz = mx.lq_mx_quantize(X, fmt)
    back = {d: mx.lq_mx_dequantize(qz, d) for d in SRC.values()}
    torch.cuda.synchronize()
    x = X.detach().cpu().to(torch.float64).numpy()
    codes, scales = omx.mx_quantize(x, fmt)
    assert np.array_equal(qz.scales.cpu().numpy(), scales)
    assert np.array_equal(qz.codes.cpu().numpy(), codes)
    want = torch.from_numpy(omx.mx_dequantize(codes, scales, fmt, cols))
    for d, got in back.items():
        assert got.shape == (rows, cols)
        # float64 -> float32 is exact (or overflows to infinity at 2^128), then one rounding
        assert torch.equal(torch.nan_to_num(got.cpu().float(), nan=7.5),
                           torch.nan_to_num(want.float().to(d).float(), nan=7.5))


@pytest.mark.parametrize("fmt", omx.FORMATS)
@pytest.mark.parametrize("src", list(SRC))
@pytest.mark.parametrize("shape", [(1, 1), (1, 32), (3, 33), (5, 31), (2, 64), (7, 100), (1, 4096),
                                   (129, 255), (33, 1000), (64, 4096), (3, 11008)])
def test_shapes(fmt, src, shape):
    g = torch.Generator().manual_seed(sum(shape))
    X = torch.randn(shape, generator=g) * torch.exp2(torch.randint(-12, 12, shape, generator=g))
    check(X.to(SRC[src]).to(DEV), fmt)


@pytest.mark.parametrize("fmt", omx.FORMATS)
@pytest.mark.parametrize("src", list(SRC))
def test_special_values(fmt, src):
    top = omx.GRID[fmt][-1]
    mids = (omx.GRID[fmt][1:] + omx.GRID[fmt][:-1]) / 2
    rows = [
        np.zeros(32), -np.zeros(32), np.full(32, 1e-40), np.full(32, 3.3e38), np.full(32, -1.0),
        np.r_[top, -mids[:31] if len(mids) > 31 else np.pad(-mids, (0, 31 - len(mids)))],
        np.r_[np.inf, np.ones(31)], np.r_[np.ones(31), np.nan], np.r_[-np.inf, np.inf, np.zeros(30)],
        np.r_[2.0**-126, 2.0**-133 * np.arange(31)], np.r_[1e30, 1e-30 * np.ones(31)],
        np.r_[top * 2.0**-127, np.linspace(0, top, 31) * 2.0**-127],
        np.r_[top * (1 + 2.0**-6), np.linspace(-top, top, 31)],
        np.r_[3.38953139e38, -3.38953139e38, np.zeros(30)],
    ]
    check(torch.tensor(np.array(rows), dtype=torch.float32).to(SRC[src]).to(DEV), fmt)


@pytest.mark.parametrize("src", list(SRC))
def test_every_grid_boundary_at_every_scale(src):
    """Grid values, midpoints and their neighbours, scaled over float32's exponents."""
    for fmt in omx.FORMATS:
        grid = omx.GRID[fmt]
        v = np.concatenate([grid, (grid[1:] + grid[:-1]) / 2])
        v = np.pad(v, (0, -len(v) % 31)).reshape(-1, 31)
        v = np.concatenate([np.full((len(v), 1), grid[-1]), v], 1)
        out = [v * 2.0**e * s for e in range(-149, 119, 3) for s in (1, -1)]
        check(torch.tensor(np.concatenate(out), dtype=torch.float32).to(SRC[src]).to(DEV), fmt)


@pytest.mark.parametrize("fmt", omx.FORMATS)
def test_every_code_at_every_scale_byte(fmt):
    """Dequantisation of all 256 code bytes under all 256 scale bytes."""
    announce(f"mx dequantise all codes {fmt}")
    per = 32 if fmt == "fp8" else 16  # code bytes per block
    c = np.arange(256, dtype=np.uint8).reshape(1, 256)
    codes = np.repeat(c, 256, 0)
    nb = 256 // per
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], nb, 1)
    cols = nb * 32
    q = mx.MxTensor(torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), 256, cols, fmt)
    want = torch.from_numpy(omx.mx_dequantize(codes, scales, fmt, cols))
    for d in SRC.values():
        got = mx.lq_mx_dequantize(q, d).cpu().float()
        assert torch.equal(torch.nan_to_num(got, nan=7.5, posinf=8.5, neginf=9.5),
                           torch.nan_to_num(want.float().to(d).float(), nan=7.5, posinf=8.5, neginf=9.5))


def test_most_elements():
    """2^35 elements, the codec's limit (128 GiB of float32): every slice of the
    rows equals the same call on the slice alone."""
    free, _ = torch.cuda.mem_get_info()
    free += torch.cuda.memory_reserved() - torch.cuda.memory_allocated()
    if free < 160 << 30:
        pytest.skip("needs 160 GiB of free device memory")
    torch.cuda.empty_cache()
    rows, cols, n = 1 << 20, 1 << 15, 1 << 16
    announce("mx codec 2^35 elements")
    q = mx.MxTensor(torch.empty((rows, cols // 2), dtype=torch.uint8, device=DEV).random_(),
                    torch.empty((rows, cols // 32), dtype=torch.uint8, device=DEV).random_(100, 150),
                    rows, cols, "fp4")
    cut = lambda t, a: mx.MxTensor(t.codes[a:a + n], t.scales[a:a + n], n, cols, "fp4")  # noqa: E731
    for dt in (torch.float32, torch.bfloat16):
        out = mx.lq_mx_dequantize(q, dt)
        for a in range(0, rows, n):
            assert torch.equal(out[a:a + n], mx.lq_mx_dequantize(cut(q, a), dt)), a
        if dt is torch.float32:
            del out
            torch.cuda.empty_cache()
    z = mx.lq_mx_quantize(out, "fp4")
    for a in range(0, rows, n):
        part, whole = mx.lq_mx_quantize(out[a:a + n], "fp4"), cut(z, a)
        assert torch.equal(part.codes, whole.codes) and torch.equal(part.scales, whole.scales), a
    del out, z, q
    torch.cuda.empty_cache()


@pytest.mark.parametrize("fmt", omx.FORMATS)
@pytest.mark.parametrize("src", list(SRC))
def test_misaligned_source_and_bytes_past_the_end(fmt, src):
    """A source that starts at one element past an allocation, and outputs
    followed by bytes that must stay."""
    import ctypes
    from qlora_parameter_efficient_amd import lq
    rows, cols = 9, 45
    flat = torch.randn(1 + rows * cols, generator=torch.Generator().manual_seed(1)).to(SRC[src]).to(DEV)
    X = flat[1:].view(rows, cols)
    announce(f"mx codec misaligned {fmt} {src}")
    nc = mx.lib().lq_mx_codes_bytes(mx.FORMATS[fmt], rows, cols)
    ns = mx.lib().lq_mx_scales_bytes(rows, cols)
    codes = torch.full((nc + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    scales = torch.full((ns + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    assert mx.lib().lq_mx_quantize(X.data_ptr(), lq._dt(X), rows, cols, mx.FORMATS[fmt],
                                   codes.data_ptr(), scales.data_ptr(), lq._stream()) == 0
    wc, wsc = omx.mx_quantize(X.cpu().double().numpy(), fmt)
    assert np.array_equal(codes[:nc].cpu().numpy(), wc.ravel())
    assert np.array_equal(scales[:ns].cpu().numpy(), wsc.ravel())
    assert (codes[nc:] == 0xA5).all() and (scales[ns:] == 0xA5).all()
    s = mx.LqMxStruct(mx.FORMATS[fmt], 0, rows, cols, codes.data_ptr(), scales.data_ptr())
    out = torch.full((1 + rows * cols + 32,), 3.0, dtype=SRC[src], device=DEV)
    assert mx.lib().lq_mx_dequantize(ctypes.byref(s), out[1:].data_ptr(), lq._dt(out),
                                     lq._stream()) == 0
    want = torch.from_numpy(omx.mx_dequantize(wc, wsc, fmt, cols)).to(SRC[src])
    assert torch.equal(out[1:1 + rows * cols].cpu().view(rows, cols), want)
    assert out[0] == 3.0 and (out[1 + rows * cols:] == 3.0).all()
