"""The MXFP4 product and the expert layer on a stream that has no workspace and cannot get one."""
import ctypes

import numpy as np
import pytest

import weight_only_bit_gptq_amd as gq
from oracle import mx_ref

torch = pytest.importorskip("torch")


@pytest.fixture()
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gq.release()                                                  # no stream has a workspace
    yield torch.device("cuda:0")
    gq.release()


def layer_inputs(dev, T=3, H=64, I=32, E=4):
    rng = np.random.default_rng(3)
    xt = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).bfloat16()
    wt = torch.from_numpy((rng.standard_normal((E, H)) / 8).astype(np.float32)).bfloat16()
    u, d = mx_ref.quantize(rng.standard_normal((E, 2 * I, H)) * 0.1), mx_ref.quantize(rng.standard_normal((E, H, I)) * 0.1)
    ref, bound = mx_ref.moe_layer(xt.double().numpy(), wt.double().numpy(), 2, mx_ref.values(*u), mx_ref.values(*d), True,
                                  2.0 ** -7)
    t = lambda a: torch.from_numpy(a).to(dev)
    return (xt.to(dev), wt.to(dev), 2, gq.MxExperts(t(u[0]), t(u[1])), gq.MxExperts(t(d[0]), t(d[1]))), ref, bound


# (kind, M, N, K): split over K by the streaming kernels and by both tiles
SPLIT = [("bf16", 15, 100, 4160), ("fp16", 108, 35, 672), ("mxfp4", 7, 70, 4128), ("mxfp4", 107, 71, 3200)]


def product_inputs(dev, kind, M, N, K):
    rng = np.random.default_rng(M)
    codes = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    scales = rng.integers(118, 132, (N, K // 32)).astype(np.uint8)
    x = rng.standard_normal((M, K)).astype(np.float32)
    t = lambda a: torch.from_numpy(a).to(dev)
    if kind == "mxfp4":
        c, s = mx_ref.quantize(x)
        x, args, kw = mx_ref.values(c, s), t(c), dict(x_scales=t(s))
    else:
        xt = torch.from_numpy(x).to(torch.float16 if kind == "fp16" else torch.bfloat16)
        x, args, kw = xt.double().numpy(), xt.to(dev), {}
    ref, mag = mx_ref.gemm(x, mx_ref.values(codes, scales))
    bound = mx_ref.sum_error(K) * mag
    return (args, t(codes), t(scales)), kw, ref, bound + 2.0 ** -24 * (np.abs(ref) + bound)


def k_splits(x, codes, scales, M, N, K, kind, xs):
    buf = ctypes.create_string_buffer(256)
    kinds = {"fp16": 0, "bf16": 1, "mxfp4": 3}
    assert gq.library().gptq_mxfp4_gemm_describe(x.data_ptr(), kinds[kind], xs.data_ptr() if xs is not None else None,
                                                 codes.data_ptr(), scales.data_ptr(), M, N, K, x.data_ptr(), 2, buf, 256) == 0
    return int(buf.value.decode().rsplit("=", 1)[1])


def close(y, ref, bound):
    return (np.abs(y.double().cpu().numpy() - ref) <= bound).all()


@pytest.mark.gpu
def test_layer_without_a_workspace_reports_it_and_writes_nothing(dev, monkeypatch):
    args, ref, bound = layer_inputs(dev)
    out = torch.full_like(args[0], 7.0)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    monkeypatch.setenv("GPTQ_TEST_FAIL_WORKSPACE", "1")
    with torch.cuda.stream(st), pytest.raises(gq.GptqError) as err:
        gq.moe_layer(*args, out=out)
    st.synchronize()
    assert err.value.code == -6 and (out == 7.0).all()
    monkeypatch.delenv("GPTQ_TEST_FAIL_WORKSPACE")
    with torch.cuda.stream(st):
        gq.moe_layer(*args, out=out)
    st.synchronize()
    assert close(out, ref, bound)


@pytest.mark.gpu
@pytest.mark.parametrize("kind,M,N,K", SPLIT)
def test_product_without_a_workspace_runs_unsplit(dev, monkeypatch, kind, M, N, K):
    args, kw, ref, bound = product_inputs(dev, kind, M, N, K)
    assert k_splits(*args, M, N, K, kind, kw.get("x_scales")) > 1
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    monkeypatch.setenv("GPTQ_TEST_FAIL_WORKSPACE", "1")
    with torch.cuda.stream(st):
        y = gq.mxfp4_gemm(*args, out_dtype=torch.float32, **kw)
    st.synchronize()
    assert close(y, ref, bound)
    monkeypatch.delenv("GPTQ_TEST_FAIL_WORKSPACE")
    with torch.cuda.stream(st):
        z = gq.mxfp4_gemm(*args, out_dtype=torch.float32, **kw)
    st.synchronize()
    assert close(z, ref, bound)


@pytest.mark.gpu
def test_capture_before_the_first_call(dev):
    """The layer is refused and leaves the capture as it is; products are captured unsplit and replay right."""
    layer, _, _ = layer_inputs(dev)
    x, wr, k, up, down = layer
    cases = [product_inputs(dev, *c) for c in SPLIT]
    untouched = torch.full_like(x, 7.0)
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        ys = [gq.mxfp4_gemm(*args, out_dtype=torch.float32, **kw) for args, kw, _, _ in cases]
        rc = gq.library().gptq_moe_layer(x.data_ptr(), 1, wr.data_ptr(), *x.shape, 32, 4, k, 1, ctypes.byref(up._stack),
                                         ctypes.byref(down._stack), untouched.data_ptr(),
                                         torch.cuda.current_stream().cuda_stream)
    assert rc == -6
    for _ in range(3):
        for y in ys:
            y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(close(y, ref, bound) for y, (_, _, ref, bound) in zip(ys, cases))
        assert (untouched == 7.0).all()
        # eager calls (their stream has a workspace of its own by then) between the replays
        assert all(close(gq.mxfp4_gemm(*args, out_dtype=torch.float32, **kw), ref, bound) for args, kw, ref, bound in cases)
