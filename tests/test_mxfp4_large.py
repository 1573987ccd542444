"""MXFP4 quantise and dequantise beyond 2^32 threads' worth of values (81 GiB of GPU memory)."""
import pytest

import weight_only_bit_gptq_amd as gq

torch = pytest.importorskip("torch")

M, K = (1 << 15) + 1, 1 << 20                                     # 64 GiB of bf16 and a row


@pytest.mark.gpu
def test_more_values_than_one_grid_holds():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GiB of free GPU memory")
    g = torch.Generator(device="cuda").manual_seed(0)
    codes = torch.randint(0, 256, (M, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(118, 132, (M, K // 32), dtype=torch.uint8, device="cuda", generator=g)
    v = gq.mxfp4_dequant(codes, scales, torch.bfloat16)
    # both ends, the rows about every 2^30 pieces of 16 bytes (8192 rows), and one in the middle
    rows = sorted({0, 1, 4321, M - 2, M - 1} | {r + d for r in range(8192, M, 8192) for d in (-1, 0)})
    for r in rows:
        assert torch.equal(v[r:r + 1], gq.mxfp4_dequant(codes[r:r + 1], scales[r:r + 1], torch.bfloat16)), r
    del codes, scales
    c, s = gq.mxfp4_quantize(v)
    for r in rows:
        cr, sr = gq.mxfp4_quantize(v[r:r + 1])
        assert torch.equal(c[r:r + 1], cr) and torch.equal(s[r:r + 1], sr), r
    del v, c, s
    torch.cuda.empty_cache()
