"""Every kernel that an MXFP4 quantisation or product may be given, at ragged sizes that are given it.

The plan is asked (host only) which kernel a shape takes, so that no change of
the plan leaves one untested; the results are compared with the fp64 oracle in
full.
"""
import ctypes
import os

import numpy as np
import pytest

import weight_only_bit_gptq_amd as gq
from oracle import mx_ref

torch = pytest.importorskip("torch")

needs_lib = pytest.mark.skipif(not os.path.exists(gq.library_path()),
                               reason="libgptq.so not built (run __graft_entry__.build())")
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
TYPE = {"fp16": 0, "bf16": 1, "fp32": 2, "mxfp4": 3}

# (kind, M, N, K, scale bytes at an odd address) -> kernel, and whether K is split
PRODUCTS = [
    ("bf16", 5, 33, 32, False, "mx_stream_kernel<true, 1, 1>", False),
    ("bf16", 15, 100, 4160, False, "mx_stream_kernel<true, 1, 1>", True),
    ("bf16", 31, 130, 4128, False, "mx_stream_kernel<true, 2, 1>", True),
    ("fp16", 3, 33, 8224, False, "mx_stream_kernel<false, 1, 1>", True),
    ("fp16", 31, 130, 544, True, "mx_stream_kernel<false, 2, 1>", False),
    ("bf16", 60, 41, 192, False, "mx_tile_kernel<true, 64>", False),
    ("bf16", 108, 35, 672, False, "mx_tile_kernel<true, 64>", True),
    ("fp16", 97, 301, 1056, False, "mx_tile_kernel<false, 64>", True),
    ("bf16", 515, 8201, 352, False, "mx_tile_kernel<true, 128>", False),
    ("bf16", 1598, 35, 2848, False, "mx_tile_kernel<true, 128>", True),
    ("fp16", 515, 8202, 352, True, "mx_tile_kernel<false, 128>", False),
    ("fp16", 1598, 35, 2848, False, "mx_tile_kernel<false, 128>", True),
    ("mxfp4", 7, 70, 4128, False, "mx4_stream_kernel<1, 1>", True),
    ("mxfp4", 29, 70, 288, True, "mx4_stream_kernel<2, 1>", False),
    ("mxfp4", 37, 69, 3680, False, "mx4_stream_kernel<4, 1>", True),
    ("mxfp4", 175, 259, 96, False, "mx4_tile_kernel<2, 2, false>", False),
    ("mxfp4", 75, 77, 1568, False, "mx4_tile_kernel<2, 2, false>", True),
    ("mxfp4", 112, 57, 384, False, "mx4_tile_kernel<2, 4, true>", False),
    ("mxfp4", 107, 71, 3200, False, "mx4_tile_kernel<2, 4, true>", True),
    ("mxfp4", 801, 4623, 640, False, "mx4_tile_kernel<2, 2, true>", False),
    ("mxfp4", 1181, 6551, 640, False, "mx4_tile_kernel<4, 2, true>", False),
    ("mxfp4", 1181, 6551, 640, True, "mx4_tile_kernel<4, 2, false>", False),
    ("mxfp4", 1169, 6691, 352, False, "mx4_tile_kernel<4, 2, false>", False),
]
QUANTISATIONS = [("fp16", 3, 96, 1), ("bf16", 513, 8224, 1), ("fp32", 33, 1056, 1),
                 ("fp16", 2051, 8224, 4), ("bf16", 2051, 8224, 4), ("fp32", 1031, 8160, 4)]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gq.library()
    return torch.device("cuda:0")


def plan(kind, M, N, K, scales, out_type=2, x_scales=0x20000, out=0x50000):
    buf = ctypes.create_string_buffer(256)
    rc = gq.library().gptq_mxfp4_gemm_describe(0x10000, TYPE[kind], x_scales if kind == "mxfp4" else None, 0x30000, scales,
                                               M, N, K, out, out_type, buf, 256)
    assert rc == 0
    return buf.value.decode()


@needs_lib
@pytest.mark.parametrize("kind,M,N,K,odd,kernel,split", PRODUCTS)
def test_the_plan_gives_the_shape_its_kernel(kind, M, N, K, odd, kernel, split):
    text = plan(kind, M, N, K, 0x40001 if odd else 0x40000)
    assert text.startswith(f"gptq::{kernel} grid=") and (int(text.rsplit("=", 1)[1]) > 1) == split, text


@needs_lib
def test_every_kernel_has_a_shape():
    named = {p[5] for p in PRODUCTS}
    assert named == {f"mx_stream_kernel<{b}, {m}, 1>" for b in ("true", "false") for m in (1, 2)} | \
        {f"mx4_stream_kernel<{m}, 1>" for m in (1, 2, 4)} | \
        {f"mx_tile_kernel<{b}, {m}>" for b in ("true", "false") for m in (64, 128)} | \
        {"mx4_tile_kernel<4, 2, true>", "mx4_tile_kernel<4, 2, false>", "mx4_tile_kernel<2, 2, true>",
         "mx4_tile_kernel<2, 2, false>", "mx4_tile_kernel<2, 4, true>"}
    # and whatever the plan gives is among them
    for kind in ("fp16", "bf16", "mxfp4"):
        for M in (1, 16, 17, 32, 33, 64, 65, 128, 129, 300, 513, 1000, 2048, 5000):
            for N in (1, 31, 500, 4096, 12289, 28672):
                for K in (32, 160, 512, 4096, 11008, 16384):
                    for s in (0x40000, 0x40002):
                        assert plan(kind, M, N, K, s).split(" grid")[0][len("gptq::"):] in named


@needs_lib
def test_describe_refusals_and_short_buffers():
    lib = gq.library()
    buf = ctypes.create_string_buffer(b"x" * 15, 16)
    assert lib.gptq_mxfp4_gemm_describe(0x10000, 1, None, 0x30000, 0x40000, 3, 17, 64, 0x50000, 1, buf, 8) == 0
    assert buf.value == b"gptq::m"
    assert lib.gptq_mxfp4_gemm_describe(0x10000, 1, None, 0x30000, 0x40000, 0, 17, 64, 0x50000, 1, buf, 16) == 0
    assert buf.value == b"none (M = 0)"
    assert lib.gptq_mxfp4_gemm_describe(0x10000, 1, None, 0x30000, 0x40000, 3, 17, 65, 0x50000, 1, buf, 16) == -3
    assert buf.value == b""
    assert lib.gptq_mxfp4_gemm_describe(0x10000, 1, None, 0x30000, 0x40000, 3, 17, 64, 0x50000, 1, None, 16) == -1
    assert lib.gptq_mxfp4_quantize_describe(1, 3, 64, buf, 0) == -1
    assert lib.gptq_mxfp4_quantize_describe(3, 3, 64, buf, 16) == -9
    assert lib.gptq_mxfp4_quantize_describe(1, 3, 40, buf, 16) == -3
    assert lib.gptq_mxfp4_quantize_describe(1, -1, 64, buf, 16) == -3
    assert lib.gptq_mxfp4_quantize_describe(1, 0, 64, buf, 16) == 0 and buf.value == b"none (M = 0)"


def pieces_per_thread(dtype, M, K):
    buf = ctypes.create_string_buffer(256)
    assert gq.library().gptq_mxfp4_quantize_describe(TYPE[dtype], M, K, buf, 256) == 0
    name = buf.value.decode().split(" ")
    assert name[0] == f"gptq::mx_quantize_kernel<{TYPE[dtype]},", buf.value
    return int(name[1][:-1])


@needs_lib
@pytest.mark.parametrize("dtype,M,K,per", QUANTISATIONS)
def test_the_plan_gives_the_quantisation_its_kernel(dtype, M, K, per):
    assert pieces_per_thread(dtype, M, K) == per
    if per == 4:                                                  # the last workgroup is ragged
        assert M * K // (4 if dtype == "fp32" else 8) % 1024 != 0


# ------------------------------------------------------------------ GPU
def at_address(a, dev, odd):
    buf = torch.empty(a.size + 4, dtype=torch.uint8, device=dev)
    v = buf[1:1 + a.size] if odd else buf[:a.size]
    v.copy_(torch.from_numpy(np.ascontiguousarray(a)).flatten())
    return v.view(a.shape)


def assert_close(y, ref, mag, K, what):
    eps = torch.finfo(y.dtype).eps / 2
    y = y.double().cpu().numpy()
    bound = mx_ref.sum_error(K) * mag
    bound = bound + eps * (np.abs(ref) + bound) + (2.0 ** -25 if eps == 2.0 ** -11 else 0.0)
    excess = np.abs(y - ref) - bound
    assert np.isfinite(y).all() and excess.max() <= 0, f"{what}: over by {excess.max():.3e}"


@pytest.mark.gpu
@pytest.mark.parametrize("kind,M,N,K,odd,kernel,split", PRODUCTS)
def test_product(dev, kind, M, N, K, odd, kernel, split):
    rng = np.random.default_rng(M + N + K)
    codes = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    scales = rng.integers(118, 132, (N, K // 32)).astype(np.uint8)
    x = rng.standard_normal((M, K)) * np.exp(0.5 * rng.standard_normal((M, 1)))
    w, ws = at_address(codes, dev, False), at_address(scales, dev, odd)
    outs = [torch.float32, torch.bfloat16 if kind == "bf16" else torch.float16]
    if kind == "mxfp4":
        c, s = gq.mxfp4_quantize(torch.from_numpy(x.astype(np.float32)).to(dev))
        x = mx_ref.values(c.cpu().numpy(), s.cpu().numpy())
        s = at_address(s.cpu().numpy(), dev, odd)
        ys = [gq.mxfp4_gemm(c, w, ws, x_scales=s, out_dtype=t) for t in outs]
        xs_ptr, x_ptr = s.data_ptr(), c
    else:
        xt = torch.from_numpy(x.astype(np.float32)).to(DTYPES[kind])
        x = xt.double().numpy()
        xt = xt.to(dev)
        ys = [gq.mxfp4_gemm(xt, w, ws, out_dtype=t) for t in outs]
        xs_ptr, x_ptr = None, xt
    for y, t in zip(ys, (2, 1 if kind == "bf16" else 0)):
        text = plan(kind, M, N, K, ws.data_ptr(), t, xs_ptr, y.data_ptr())
        assert text.startswith(f"gptq::{kernel} grid="), text
    ref, mag = mx_ref.gemm(x, mx_ref.values(codes, scales))
    for y in ys:
        assert_close(y, ref, mag, K, f"{kernel} {x_ptr.dtype} {y.dtype}")


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(97, 301, 1056), (515, 8202, 352), (1598, 35, 2848)])
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
def test_tiles_with_scales_outside_the_types_range(dev, kind, M, N, K):
    """A tile's products taken again, on 64 and 128 rows, with K whole and split; most tiles stay as they are."""
    rng = np.random.default_rng(N)
    codes = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    scales = rng.integers(118, 132, (N, K // 32)).astype(np.uint8)
    x = rng.standard_normal((M, K))
    x[:, 32:64] *= 2.0 ** -20
    for n in range(0, N, 97):
        scales[n, 3] = rng.choice([60, 90, 103, 141, 150])
        scales[n, 1] = rng.choice([0, 1, 252, 253, 254])
        codes[n, 64:80] = 0x88                                    # block 4: zeros under a small byte
        scales[n, 4] = 0
    xt = torch.from_numpy(x.astype(np.float32)).to(DTYPES[kind])
    t = lambda a: torch.from_numpy(a).to(dev)
    y = gq.mxfp4_gemm(xt.to(dev), t(codes), t(scales), out_dtype=torch.float32)
    ref, mag = mx_ref.gemm(xt.double().numpy(), mx_ref.values(codes, scales))
    assert_close(y, ref, mag, K, f"{kind} {M} {N} {K}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,M,K,per", QUANTISATIONS)
def test_quantisation(dev, dtype, M, K, per):
    assert pieces_per_thread(dtype, M, K) == per
    t = {**DTYPES, "fp32": torch.float32}[dtype]
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn((M, K), generator=g, device=dev) * torch.exp(torch.randn((M, 1), generator=g, device=dev))
    x[:, :32] = 0.0
    x = x.to(t)
    codes, scales = gq.mxfp4_quantize(x)
    # all of it against quantisations of few rows, which one piece a thread makes
    for r in range(0, M, 256):
        part = x[r:r + 256].contiguous()
        assert pieces_per_thread(dtype, part.shape[0], K) == 1
        c, s = gq.mxfp4_quantize(part)
        assert torch.equal(codes[r:r + 256], c) and torch.equal(scales[r:r + 256], s), r
    # and rows of both ends and between against the oracle
    rows = sorted({0, 1, M // 3, M // 2, M - 2, M - 1} & set(range(M)))
    c, s = mx_ref.quantize(x[rows].double().cpu().numpy())
    assert np.array_equal(codes[rows].cpu().numpy(), c) and np.array_equal(scales[rows].cpu().numpy(), s)
