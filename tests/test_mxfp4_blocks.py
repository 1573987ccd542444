"""fp16 products with MXFP4 weights whose blocks fp16 cannot scale, but need not (gptq_mxfp4_gemm).

Blocks of zeros and columns past N leave a product on its ordinary path: the
result is, bit for bit, that of the same weights with ordinary scale bytes there.
(Another path adds in another order, which fp32 outputs of these sums show.)
"""
import numpy as np
import pytest

import weight_only_bit_gptq_amd as gq
from oracle import mx_ref

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gq.library()
    return torch.device("cuda:0")


def operands(M, N, K, seed):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).half()
    codes = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    scales = rng.integers(118, 132, (N, K // 32)).astype(np.uint8)
    return rng, x, codes, scales


def product(dev, x, codes, scales):
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    return gq.mxfp4_gemm(x.to(dev), t(codes), t(scales), out_dtype=torch.float32).cpu()


def assert_bound(y, x, codes, scales, K):
    ref, mag = mx_ref.gemm(x.double().numpy(), mx_ref.values(codes, scales))
    bound = mx_ref.sum_error(K) * mag
    assert (np.abs(y.double().numpy() - ref) <= bound + 2.0 ** -24 * (np.abs(ref) + bound)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 48, 4096), (16, 96, 1056), (20, 64, 2048), (40, 80, 4096), (130, 300, 1024)])
def test_blocks_of_zeros_take_any_scale(dev, M, N, K):
    rng, x, codes, scales = operands(M, N, K, seed=M + N)
    zero = rng.random((N, K // 32)) < 0.05
    zero[3] = True                                                # a pruned or padded row
    wide = codes.reshape(N, K // 32, 16)
    wide[zero] = rng.choice([0x00, 0x08, 0x80, 0x88], (int(zero.sum()), 16))     # +0 and -0
    plain = np.where(zero, 127, scales).astype(np.uint8)
    y = product(dev, x, codes, plain)
    assert_bound(y, x, codes, plain, K)
    for byte in (0, 90, 103, 141, 250, 254):
        z = product(dev, x, codes, np.where(zero, byte, scales).astype(np.uint8))
        assert torch.equal(z, y), byte
    # the quantiser's own: a block of zeros gets byte 0
    v = mx_ref.values(codes, plain)
    assert torch.equal(product(dev, x, *mx_ref.quantize(v)), product(dev, x, codes_of(v), normal_bytes(v)))


def codes_of(v):
    return mx_ref.quantize(v)[0]


def normal_bytes(v):
    s = mx_ref.quantize(v)[1]
    return np.where(s == 0, 127, s).astype(np.uint8)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 20, 130])
def test_zero_codes_under_a_nan_scale_are_nan(dev, M):
    _, x, codes, scales = operands(M, 40, 256, seed=M)
    codes[5, 16:32] = 0
    scales[5, 1] = 255
    y = product(dev, x, codes, scales)
    assert torch.isnan(y[:, 5]).all() and torch.isfinite(y[:, torch.arange(40) != 5]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 20, 130])
def test_nonzero_blocks_beside_zero_ones_keep_their_scale(dev, M):
    """One value in an otherwise zero block, at a scale that fp16 cannot hold."""
    N, K = 40, 544
    rng, x, codes, scales = operands(M, N, K, seed=M + 1)
    wide = codes.reshape(N, K // 32, 16)
    for n in range(N):
        b = int(rng.integers(K // 32))
        wide[n, b] = 0
        wide[n, b, rng.integers(16)] = rng.choice([0x01, 0x70, 0x0F])
        scales[n, b] = rng.choice([0, 60, 103, 141, 160])
    y = product(dev, x, codes, scales)
    assert_bound(y, x, codes, scales, K)


@pytest.mark.gpu
@pytest.mark.parametrize("M,K", [(1, 4096), (16, 2080), (20, 4096)])
@pytest.mark.parametrize("N,more", [(17, 32), (47, 64), (64 + 16, 128)])
def test_columns_past_the_end_leave_the_path_alone(dev, M, K, N, more):
    """N off the column tiles: bit for bit the first columns of the product with whole tiles."""
    _, x, codes, scales = operands(M, more, K, seed=N)
    y = product(dev, x, codes[:N], scales[:N])
    assert torch.equal(y, product(dev, x, codes, scales)[:, :N])
    assert_bound(y, x, codes[:N], scales[:N], K)
