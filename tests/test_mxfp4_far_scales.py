"""MXFP4 scale bytes 253 and 254: values of 2^128 and above, beyond bf16 and fp32.

A product with them is exact all the same where it is in fp32's range: a zero
activation makes zero, a small one a finite sum.
"""
import numpy as np
import pytest

import weight_only_bit_gptq_amd as gq
from oracle import mx_ref

torch = pytest.importorskip("torch")
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gq.library()
    return torch.device("cuda:0")


def operands(M, N, K, seed):
    """Every third column has a far block (bytes 250 .. 254), under small activations, some of them zero."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    scales = rng.integers(118, 132, (N, K // 32)).astype(np.uint8)
    scales[::3, 1] = rng.integers(250, 255, len(scales[::3]))
    x = rng.standard_normal((M, K))
    x[:, 32:64] *= 2.0 ** -20
    x[:, 40] = 0.0
    x[0, 32:64] = 0.0                                             # a row without a far product
    return x, codes, scales


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 3, 20, 40, 130])
@pytest.mark.parametrize("kind", ["fp16", "bf16", "mxfp4"])
def test_products(dev, M, kind):
    N, K = 70, 544
    x, codes, scales = operands(M, N, K, seed=M)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    if kind == "mxfp4":
        xc, xs = mx_ref.quantize(x)
        x = mx_ref.values(xc, xs)
        y = gq.mxfp4_gemm(t(xc), t(codes), t(scales), x_scales=t(xs), out_dtype=torch.float32)
    else:
        xt = torch.from_numpy(x.astype(np.float32)).to(DTYPES[kind])
        x = xt.double().numpy()
        y = gq.mxfp4_gemm(xt.to(dev), t(codes), t(scales), out_dtype=torch.float32)
    ref, mag = mx_ref.gemm(x, mx_ref.values(codes, scales))
    assert mag.max() < 2.0 ** 126 and (M == 1 or mag.max() > 2.0 ** 100)
    y = y.double().cpu().numpy()
    assert np.isfinite(y).all()
    bound = mx_ref.sum_error(K) * mag
    assert (np.abs(y - ref) <= bound + 2.0 ** -24 * (np.abs(ref) + bound)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T", [1, 20])
def test_expert_layer_with_zero_hidden_values(dev, T, dtype):
    """Far blocks of the down weights meet hidden values that are exactly zero: they add nothing."""
    H, I, E, k = 128, 64, 4, 2
    rng = np.random.default_rng(T)
    xt = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(DTYPES[dtype])
    wt = torch.from_numpy((rng.standard_normal((E, H)) / np.sqrt(H)).astype(np.float32)).to(DTYPES[dtype])
    uc, us = mx_ref.quantize(rng.standard_normal((E, 2 * I, H)) * 0.1)
    dc, ds = mx_ref.quantize(rng.standard_normal((E, H, I)) * 0.1)
    uc[:, :32] = 0                                                # gates 0 .. 31 are zero, and so are h's
    ds[:, ::2, 0] = 254
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    y = gq.moe_layer(xt.to(dev), wt.to(dev), k, gq.MxExperts(t(uc), t(us)), gq.MxExperts(t(dc), t(ds)))
    ref, bound = mx_ref.moe_layer(xt.double().numpy(), wt.double().numpy(), k, mx_ref.values(uc, us),
                                  np.where(np.repeat(ds == 254, 32, -1), 0.0, mx_ref.values(dc, ds)), True,
                                  torch.finfo(y.dtype).eps)
    if dtype == "fp16":
        bound = bound + 2.0 ** -25
    y = y.double().cpu().numpy()
    assert np.isfinite(y).all() and (np.abs(y - ref) <= bound).all()


@pytest.mark.gpu
def test_values(dev):
    """All codes under bytes 250 .. 254: rounded once, to infinity where the type ends."""
    codes = np.tile(np.arange(256, dtype=np.uint8).reshape(16, 16), (5, 1))
    scales = np.repeat(np.arange(250, 255, dtype=np.uint8), 16)[:, None]
    want = torch.from_numpy(mx_ref.values(codes, scales)).double()
    t = lambda a: torch.from_numpy(a).to(dev)
    for out in (torch.float32, torch.bfloat16, torch.float16):
        got = gq.mxfp4_dequant(t(codes), t(scales), out).cpu()
        # 4 and 6 times 2^126, 2 to 6 times 2^127: 2^128 and above
        ref = torch.where(want.abs() >= 2.0 ** 128, torch.sign(want) * float("inf"), want)
        assert torch.equal(got.double(), ref.to(torch.float32).to(out).double()), out


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 20, 40, 130])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_infinite_activations_and_nan_blocks_beside_far_blocks(dev, M, dtype):
    N, K = 70, 320
    x, codes, scales = operands(M, N, K, seed=7)
    scales[1, 1] = 255                                            # column 1 is NaN, columns 0, 3, .. are far
    scales[4, 2], scales[7, 2] = 0, 1                             # and two blocks too small to be scaled down
    x[M - 1, 70] = np.inf
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    xt = torch.from_numpy(x.astype(np.float32)).to(DTYPES[dtype])
    y = gq.mxfp4_gemm(xt.to(dev), t(codes), t(scales), out_dtype=torch.float32).double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        ref, mag = mx_ref.gemm(xt.double().numpy(), mx_ref.values(codes, scales))
        bound = mx_ref.sum_error(K) * mag
        bound = bound + 2.0 ** -24 * (np.abs(ref) + bound)
    assert np.array_equal(np.isnan(y), np.isnan(ref)) and np.array_equal(np.isinf(y), np.isinf(ref))
    assert np.array_equal(np.sign(y[np.isinf(y)]), np.sign(ref[np.isinf(ref)]))
    fine = np.isfinite(ref)
    assert (np.abs(y[fine] - ref[fine]) <= bound[fine]).all()
