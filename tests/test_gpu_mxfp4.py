"""MXFP4 on the GPU: quantisation (bit-exact), dequantisation, and the W4A16
and W4A4 products against their 64-bit forms (bounds of dense_ref)."""
import numpy as np
import pytest
import torch

import nvfp4_weight_only_router_b200 as lib
from tests import dense_ref as R

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _randn(seed, shape, dtype, dev, scale=1.0):
    gen = torch.Generator(device=dev).manual_seed(seed)
    return (torch.randn(shape, generator=gen, device=dev) * scale).to(dtype)


def _check_quantize(x):
    codes, scales = lib.mxfp4_quantize(x)
    torch.cuda.synchronize()
    q0, s0 = R.mx_encode(x.cpu().double().numpy())
    assert np.array_equal(scales.cpu().numpy(), s0)
    assert np.array_equal(codes.cpu().numpy(), q0)
    return codes, scales


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 31), (3, 32), (2, 33), (5, 100), (7, 257), (33, 512), (9, 2816), (2, 2101)])
def test_quantize(dev, dtype, rows, K):
    codes, scales = _check_quantize(_randn(rows * K, (rows, K), dtype, dev))
    for t in (F32, BF):
        v = lib.mxfp4_dequantize(codes, scales, K, t)
        ref = R.mx_decode(codes.cpu().numpy(), scales.cpu().numpy(), K)
        assert v.dtype == t and np.array_equal(v.cpu().double().numpy(), ref)


@pytest.mark.parametrize("dtype", [BF, F16, F32])
def test_quantize_ties_and_extremes(dev, dtype):
    t = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6.5, 7.5, -5, -2.5, 0, -0.0, 4, 6, 1] * 2)
    big, tiny = float(torch.finfo(dtype).max), float(torch.finfo(dtype).smallest_normal)
    rows = [t, t * 2.0 ** -9, np.zeros(32), np.full(32, -0.0), np.full(32, big), np.linspace(-big, big, 32) / 2,
            np.full(32, tiny), np.linspace(0, tiny, 32), np.r_[np.zeros(31), 1.0]]
    x = torch.tensor(np.stack(rows)).to(dtype).to(dev)
    # subnormal inputs down to the type's smallest
    sub = torch.zeros((1, 32), dtype=dtype, device=dev)
    sub.view(torch.int32 if dtype == F32 else torch.int16)[0, :3] = torch.tensor([1, 3, 5], device=dev).to(
        torch.int32 if dtype == F32 else torch.int16)
    _check_quantize(torch.cat((x, sub)))


def test_quantize_non_finite_blocks(dev):
    x = _randn(3, (4, 96), F32, dev)
    x[0, 5], x[1, 40], x[2, 95] = float("nan"), float("inf"), float("-inf")
    codes, scales = _check_quantize(x)
    v = lib.mxfp4_dequantize(codes, scales)
    bad = torch.isnan(v).view(4, 3, 32)
    assert bad.all(-1).sum() == bad.any(-1).sum() == 3 and bad[0, 0].all() and bad[1, 1].all() and bad[2, 2].all()


def test_quantize_strided_and_unaligned(dev):
    base = _randn(4, (6, 200), BF, dev)
    for x in (base[:, :96], base[:, 1:97], base[1:, 8:104], base[::2, 3:70], base[2:3, 5:50]):
        _check_quantize(x)
    assert lib.mxfp4_quantize(base[:0])[0].shape == (0, 112)


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("rows,K", [(2500, 2112), (2500, 2104), (2500, 2100), (2311, 2101), (160001, 37), (700001, 5)])
def test_quantize_many_blocks(dev, dtype, rows, K):
    """Whole and ragged rows on and off the 32- and 16-byte grids, with the steps
    that a large tensor takes; and back, across the ends of rows."""
    x = _randn(rows + K, (rows, K), dtype, dev)
    codes, scales = lib.mxfp4_quantize(x)
    v = lib.mxfp4_dequantize(codes, scales, K)
    assert torch.equal(v.double(), R.mx_round(x))
    assert torch.equal(lib.mxfp4_dequantize(codes, scales, K, BF), v.to(BF))
    # the part past K of each row's last block holds zeros
    if K % 32:
        last = codes.view(rows, -1, 16)[:, -1].to(torch.int32)
        nibbles = torch.stack((last & 15, last >> 4), -1).view(rows, 32)
        assert (nibbles[:, K % 32:] == 0).all()


def test_quantize_past_32_bit_offsets(dev):
    """More than 2^31 elements: the last rows as their own call gives them."""
    rows, K = (1 << 31) // 2048 + 64, 2048
    x = torch.empty((rows, K), dtype=BF, device=dev)
    x[-64:] = _randn(5, (64, K), BF, dev)
    codes, scales = lib.mxfp4_quantize(x)
    c0, s0 = lib.mxfp4_quantize(x[-64:].clone())
    assert torch.equal(codes[-64:], c0) and torch.equal(scales[-64:], s0)
    v = lib.mxfp4_dequantize(codes, scales, dtype=BF)
    assert torch.equal(v[-64:], lib.mxfp4_dequantize(c0, s0, dtype=BF))


# ----------------------------------------------------------------- products
def _weight(seed, N, K, dev, scale=1.0):
    w = lib.Mxfp4Weight.quantize(_randn(seed, (N, K), BF, dev, scale))
    return w, torch.from_numpy(R.mx_decode(w.codes.cpu().numpy(), w.scales.cpu().numpy(), K)).to(dev)


def _check(x, weight, w64, act, a4, stream=None):
    y = (lib.mxfp4_linear_a4 if a4 else lib.mxfp4_linear)(x, weight, act)
    x64 = R.mx_round(x) if a4 else x.double()
    ref, bound = R.linear64(x64, w64, act, x.dtype)
    assert lib.device_status() == 0
    R.assert_within(y, ref, bound, f"{'a4' if a4 else 'a16'} {list(x.shape)} {act}")
    return y


SHAPES = [(64, 32), (8, 64), (72, 96), (256, 256), (200, 288), (520, 1056), (2816, 704)]


@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("T", [1, 7, 8, 9, 16, 17, 32, 33, 127, 128, 129, 257])
def test_linear(dev, T, N, K):
    weight, w64 = _weight(N + K, N, K, dev)
    x = _randn(T, (T, K), BF, dev)
    _check(x, weight, w64, None, False)
    _check(x, weight, w64, None, True)
    _check(x.to(F16), weight, w64, None, True)


@pytest.mark.parametrize("act", ["gelu_tanh", "silu"])
@pytest.mark.parametrize("N,K", [(16, 32), (48, 64), (272, 160), (1408, 2816), (528, 1024)])
@pytest.mark.parametrize("T", [1, 5, 12, 30, 33, 130, 300])
def test_linear_gated(dev, T, N, K, act):
    weight, w64 = _weight(N + K, N, K, dev, K ** -0.5)
    x = _randn(T, (T, K), BF, dev)
    _check(x, weight, w64, act, False)
    _check(x, weight, w64, act, True)
    _check(x.to(F16), weight, w64, act, True)


@pytest.mark.parametrize("T,N,K,act", [(4096, 4224, 2816, "gelu_tanh"), (1111, 2816, 2112, None), (64, 4224, 2816, "silu"),
                                       (2000, 1000, 544, None), (700, 8192, 512, None), (2300, 2816, 704, None),
                                       (2100, 528, 160, "silu")])
def test_linear_large(dev, T, N, K, act):
    """The layer's sizes and others that take each tile width."""
    weight, w64 = _weight(1, N, K, dev, K ** -0.5)
    x = _randn(2, (T, K), BF, dev)
    _check(x, weight, w64, act, False)
    _check(x, weight, w64, act, True)


@pytest.mark.parametrize("T,N,K,act", [(200, 9472, 160, None), (200, 9472, 160, "silu"), (1000, 3456, 288, None),
                                       (100, 12000, 96, None), (70, 12032, 224, "gelu_tanh")])
def test_linear_tile_widths(dev, T, N, K, act):
    """Sizes at which each tile width is taken that the others do not reach, and
    several tiles of one row block on a cluster."""
    weight, w64 = _weight(N, N, K, dev, K ** -0.5)
    x = _randn(T, (T, K), BF, dev)
    _check(x, weight, w64, act, False)
    _check(x, weight, w64, act, True)
    _check(x.to(F16), weight, w64, act, True)


@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("N,K", [(48, 4128), (208, 6400)])
@pytest.mark.parametrize("T", [1, 2, 5, 12, 30, 60])
def test_linear_long_rows(dev, T, N, K, act):
    """Rows of weights longer than a CTA keeps in flight at once."""
    weight, w64 = _weight(N + K, N, K, dev, K ** -0.5)
    x = _randn(T, (T, K), BF, dev)
    _check(x, weight, w64, act, False)
    _check(x, weight, w64, act, True)
    _check(x.to(F16), weight, w64, act, True)


@pytest.mark.parametrize("T", [1, 7, 20, 100, 300, 2200])
def test_linear_every_scale(dev, T):
    """Every scale byte that the quantiser writes (0 to 252), the smallest with
    large activations, the largest with small ones."""
    N, K = 256, 64
    gen = torch.Generator(dev).manual_seed(T)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=dev, generator=gen)
    byte = torch.arange(N, device=dev, dtype=torch.int32).clamp(max=252)
    scales = byte.to(torch.uint8)[:, None].expand(N, K // 32).contiguous()
    weight = lib.Mxfp4Weight(codes, scales, K)
    w64 = torch.from_numpy(R.mx_decode(codes.cpu().numpy(), scales.cpu().numpy(), K)).to(dev)
    for rows, s in ((slice(0, 128), 2.0 ** 60), (slice(128, 256), 2.0 ** -60)):
        x = _randn(T, (T, K), BF, dev, s)
        for a4, f in ((False, lib.mxfp4_linear), (True, lib.mxfp4_linear_a4)):
            y = f(x, weight)[:, rows]
            ref, bound = R.linear64(R.mx_round(x) if a4 else x.double(), w64[rows], None, BF)
            R.assert_within(y, ref, bound, f"a4 {a4} {s}")


@pytest.mark.parametrize("T,N,act", [(40, 9472, None), (40, 9472, "silu"), (600, 4736, None)])
def test_linear_scales_wide(dev, T, N, act):
    """Scales on both sides of the second factor next to one another, in the
    tiles that wide weights take; NaN scales reach their columns alone."""
    K = 160
    gen = torch.Generator(dev).manual_seed(T + N)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=dev, generator=gen)
    scales = torch.randint(120, 136, (N, K // 32), dtype=torch.uint8, device=dev, generator=gen)
    w64 = torch.from_numpy(R.mx_decode(codes.cpu().numpy(), scales.cpu().numpy(), K)).to(dev)
    x = _randn(T, (T, K), BF, dev, 2.0 ** -8)
    for a4 in (False, True):
        _check(x, lib.Mxfp4Weight(codes, scales, K), w64, act, a4)
    rows = [0, 77, N // 2 - 1]   # with an activation: of the gate
    scales[rows, 3] = 255
    for f in (lib.mxfp4_linear, lib.mxfp4_linear_a4):
        y = f(x, lib.Mxfp4Weight(codes, scales, K), act)
        assert torch.isnan(y[:, rows]).all() and torch.isnan(y).sum() == T * len(rows)


@pytest.mark.parametrize("T", [3, 70, 2050])
def test_linear_scale_range(dev, T):
    """Block scales over most of the byte's range, above and below the point
    where the bf16 decoding takes its second factor; NaN scales reach exactly
    their output columns."""
    N, K = 64, 128
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=dev, generator=torch.Generator(dev).manual_seed(6))
    scales = torch.zeros((N, K // 32), dtype=torch.uint8, device=dev)
    scales[:] = (torch.arange(N, device=dev, dtype=torch.int32) * 3 + 30).to(torch.uint8)[:, None]
    weight = lib.Mxfp4Weight(codes, scales, K)
    w64 = torch.from_numpy(R.mx_decode(codes.cpu().numpy(), scales.cpu().numpy(), K)).to(dev)
    x = _randn(7, (T, K), BF, dev)
    for a4 in (False, True):
        y = _check(x, weight, w64, None, a4)
        assert torch.isfinite(y).all()
    scales[5, 2] = 255
    for f in (lib.mxfp4_linear, lib.mxfp4_linear_a4):
        y = f(x, lib.Mxfp4Weight(codes, scales, K))
        assert torch.isnan(y[:, 5]).all() and torch.isnan(y).sum() == T


@pytest.mark.parametrize("T", [6, 100, 140, 2200])
def test_linear_non_finite_rows(dev, T):
    """A NaN or infinity in one token reaches that token's outputs alone."""
    weight, _ = _weight(8, 64, 96, dev)
    x = _randn(9, (T, 96), BF, dev)
    for f in (lib.mxfp4_linear, lib.mxfp4_linear_a4):
        clean = f(x, weight)
        z = x.clone()
        z[1, 40], z[T - 1, 3] = float("nan"), float("inf")
        y = f(z, weight)
        keep = [t for t in range(T) if t not in (1, T - 1)]
        assert torch.equal(y[keep], clean[keep])
        assert torch.isnan(y[1]).all() and not torch.isfinite(y[T - 1]).any()


@pytest.mark.parametrize("T", [5, 60, 150, 2100])
def test_linear_strides_streams_and_repeats(dev, T):
    weight, w64 = _weight(10, 96, 128, dev)
    wide = _randn(11, (T + 2, 400), BF, dev)
    x = wide[1:T + 1, 16:144]
    for a4, f in ((False, lib.mxfp4_linear), (True, lib.mxfp4_linear_a4)):
        odd = wide[1:T + 1, 24:152]                                    # rows on the 16-byte grid alone
        assert torch.equal(_check(odd, weight, w64, None, a4), f(odd.contiguous(), weight))
        y = _check(x, weight, w64, None, a4)
        assert torch.equal(y, f(x.contiguous(), weight)) and torch.equal(y, f(x, weight))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        z = f(x, weight, stream=s)
        s.synchronize()
        assert torch.equal(z, y)
        # captured and replayed, next to an eager call of the same shapes
        static = x.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = f(static, weight)
        static.copy_(wide[:T, 32:160])
        g.replay()
        eager = f(wide[:T, 32:160], weight)
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
    assert lib.mxfp4_linear(x[:0], weight).shape == (0, 96)
    with pytest.raises(lib.NVFP4Error):
        lib.mxfp4_linear(wide[:T, 1:129], weight)                      # misaligned rows
    with pytest.raises(lib.NVFP4Error):
        lib.mxfp4_linear(x.to(F16), weight)
    with pytest.raises(ValueError):
        lib.mxfp4_linear(x, weight, activation="relu")
    with pytest.raises(ValueError):
        lib.mxfp4_linear(x[:, :96], weight)


def test_linear_past_32_bit_offsets(dev):
    """Outputs of more than 2^31 elements: the last rows of many."""
    T, N, K, n = (1 << 20) - 3, 4096, 32, 61
    weight, w64 = _weight(14, N, K, dev)
    x = torch.zeros((T, K), dtype=BF, device=dev)
    x[-n:] = _randn(15, (n, K), BF, dev)
    for a4, f in ((False, lib.mxfp4_linear), (True, lib.mxfp4_linear_a4)):
        y = f(x, weight)
        ref, bound = R.linear64(R.mx_round(x[-n:]) if a4 else x[-n:].double(), w64, None, BF)
        assert lib.device_status() == 0 and (y[:n] == 0).all() and (y[-2 * n:-n] == 0).all()
        R.assert_within(y[-n:], ref, bound, f"a4 {a4}")


def test_weight_copies(dev):
    """Copies of a weight hold their own arrays."""
    import copy
    import pickle
    weight, _ = _weight(12, 64, 96, dev)
    x = _randn(13, (40, 96), BF, dev)
    y = lib.mxfp4_linear(x, weight)
    for other in (copy.deepcopy(weight), pickle.loads(pickle.dumps(weight))):
        assert other.codes.data_ptr() != weight.codes.data_ptr()
        before = other.codes.clone()
        weight.codes.zero_()
        assert torch.equal(other.codes, before) and torch.equal(lib.mxfp4_linear(x, other), y)
        weight.codes.copy_(before)
