"""Hidden values of the mixture-of-experts layer far from 1 (gptq_moe_layer, GPTQ experts).

Sizes of x and scales of the down weights are chosen so that silu(gate) * up,
times the router's weight, lies far below or above fp16's range while the output
does not.  The bound is oracle.mx_ref.moe_layer's, element by element; it has no
absolute term but half of fp16's smallest step at the output.
"""
import numpy as np
import pytest

import oracle
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


def exact_in(a, dtype):
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DTYPES[dtype])
    return t, t.double().numpy()


def stack(rng, E, K, N, bits, gs, tiled, dtype, scale):
    """Random packed words under scales around `scale`: (GPU arguments, fp64 values [E, N, K])."""
    G = K // gs
    words = lambda *s: rng.integers(0, 2 ** 32, s, dtype=np.uint64).astype(np.uint32).view(np.int32)
    qw, qz = words(E, K * bits // 32, N), words(E, G, N * bits // 32)
    st, s = exact_in(rng.uniform(0.5, 1.5, (E, G, N)) * scale / 2 ** (bits - 1), dtype)
    w = np.stack([oracle.dequant_ref(qw[e], qz[e], s[e], None, bits, gs, True, K, N, act=dtype).astype(np.float64).T
                  for e in range(E)])
    if tiled:
        qw = np.stack([oracle.repack_tiled(qw[e], bits) for e in range(E)])
    return (qw, qz, st, bits, gs, True), w


def experts(args, dev):
    t = lambda a: (a if isinstance(a, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(a))).to(dev)
    return gq.GptqExperts(t(args[0]), t(args[1]), t(args[2]), *args[3:])


def layer(dev, T, H, I, E, k, bits, tiled, dtype, x_scale, down_scale, renorm, seed, gs=32):
    """(output in fp64, its oracle, bound, the oracle's weighted hidden values' largest magnitude, inputs)."""
    rng = np.random.default_rng(seed)
    xt, x = exact_in(rng.standard_normal((T, H)) * x_scale, dtype)
    wt, wr = exact_in(rng.standard_normal((E, H)) / np.sqrt(H), dtype)
    a1, w1 = stack(rng, E, H, 2 * I, bits, gs, tiled, dtype, 0.1)
    a2, w2 = stack(rng, E, I, H, bits, gs, tiled, dtype, down_scale)
    s1, s2 = experts(a1, dev), experts(a2, dev)
    y = gq.moe_layer(xt.to(dev), wt.to(dev), k, s1, s2, renormalize=renorm)
    ref, bound = mx_ref.moe_layer(x, wr, k, w1, w2, renorm, torch.finfo(y.dtype).eps)
    if dtype == "fp16":
        bound = bound + 2.0 ** -25
    ids, c = mx_ref.route(x, wr, k, renorm)
    top = 0.0
    for t in range(T):
        for j in range(k):
            gu = w1[ids[t, j]] @ x[t]
            top = max(top, float(np.abs(c[t, j] * gu[:I] / (1 + np.exp(-np.clip(gu[:I], -700, 700))) * gu[I:]).max()))
    return y.double().cpu().numpy(), ref, bound, top, (xt.to(dev), wt.to(dev), k, s1, s2)


def assert_within(y, ref, bound):
    assert np.isfinite(y).all()
    excess = np.abs(y - ref) - bound
    i = np.unravel_index(np.argmax(excess), excess.shape)
    assert excess[i] <= 0, f"{y[i]} for {ref[i]} at {i}, bound {bound[i]:.3e}"


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [2, 3, 4, 8])
@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,E,k", [(1, 64, 4), (5, 48, 8), (20, 4, 2)])
def test_small_weighted_hidden_values(dev, bits, tiled, dtype, T, E, k):
    """Many experts without renormalisation and small x: weighted hidden values of 1e-5 and below."""
    y, ref, bound, top, _ = layer(dev, T, 256, 128, E, k, bits, tiled, dtype, 2.0 ** -7, 512.0, False, seed=bits + T)
    assert top < 5e-4 and np.abs(ref).max() > 2.0 ** -10
    assert_within(y, ref, bound)


@pytest.mark.gpu
@pytest.mark.parametrize("gs", [32, 128])
def test_tiny_hidden_values_under_large_down_weights(dev, gs):
    """h of about 1e-9: below fp16's smallest step, made visible by the down weights."""
    y, ref, bound, top, _ = layer(dev, 3, 256, 256, 6, 2, 4, False, "fp16", 2.0 ** -14, 2.0 ** 13, True, seed=3, gs=gs)
    assert top < 2.0 ** -24 and np.abs(ref).max() > 2.0 ** -14
    assert_within(y, ref, bound)


@pytest.mark.gpu
@pytest.mark.parametrize("bits,tiled", [(2, True), (4, False), (4, True), (8, False)])
@pytest.mark.parametrize("T", [1, 20])
def test_hidden_values_above_the_fp16_range(dev, bits, tiled, T):
    y, ref, bound, top, _ = layer(dev, T, 256, 128, 4, 2, bits, tiled, "fp16", 512.0, 2.0 ** -10, True, seed=T)
    assert top > 2.0 * 65504 and np.abs(ref).max() < 65504
    assert_within(y, ref, bound)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [9, 40])
def test_zero_nan_and_infinite_fp16_tokens_stay_in_their_row(dev, T):
    """A row of zeros (its hidden values have no largest magnitude), a NaN and an infinity beside ordinary rows."""
    y, ref, bound, _, (x, wr, k, s1, s2) = layer(dev, T, 128, 64, 4, 2, 4, True, "fp16", 1.0, 0.1, True, seed=6)
    assert_within(y, ref, bound)
    x = x.clone()
    x[1] = 0.0
    x[2, 7], x[5, 0] = float("nan"), float("inf")
    z = gq.moe_layer(x, wr, k, s1, s2)
    good = [t for t in range(T) if t not in (1, 2, 5)]
    assert (np.abs(z.double().cpu().numpy() - ref)[good] <= bound[good]).all()
    assert (z[1] == 0).all() and torch.isnan(z[2]).all() and not torch.isfinite(z[5]).any()
    assert torch.equal(z.isnan(), gq.moe_layer(x, wr, k, s1, s2).isnan())


@pytest.mark.gpu
@pytest.mark.parametrize("T,I,k", [(4, 96, 3), (21, 96, 3), (22, 96, 3), (64, 96, 1), (16, 1024, 4), (16, 1056, 4),
                                   (66, 96, 3), (70, 96, 3), (130, 96, 3)])
@pytest.mark.parametrize("bits,tiled", [(4, True), (8, False)])
def test_sizes_around_the_ways_h_is_split(dev, T, I, k, bits, tiled):
    """Rows (64) and values (65536) at the limit and beyond, several launches, a last launch of either kind."""
    y, ref, bound, _, (x, wr, k, s1, s2) = layer(dev, T, 128, I, 6, k, bits, tiled, "fp16", 0.25, 2.0, False, seed=T)
    assert_within(y, ref, bound)
    assert torch.equal(gq.moe_layer(x, wr, k, s1, s2, renormalize=False),
                       gq.moe_layer(x, wr, k, s1, s2, renormalize=False))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 20])
def test_mxfp4_gate_up_before_fp16_gptq_down(dev, T):
    H, I, E, k = 256, 96, 8, 2
    rng = np.random.default_rng(T)
    xt, x = exact_in(rng.standard_normal((T, H)) * 2.0 ** -5, "fp16")
    wt, wr = exact_in(rng.standard_normal((E, H)) / np.sqrt(H), "fp16")
    codes, scales = mx_ref.quantize(rng.standard_normal((E, 2 * I, H)) * 0.1)
    codes.reshape(E, 2 * I, H // 32, 16)[:, ::5, 1] = 0           # blocks of zeros, scale byte 0
    scales[:, ::5, 1] = 0
    a2, w2 = stack(rng, E, I, H, 3, 32, True, "fp16", 64.0)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    y = gq.moe_layer(xt.to(dev), wt.to(dev), k, gq.MxExperts(t(codes), t(scales)), experts(a2, dev))
    ref, bound = mx_ref.moe_layer(x, wr, k, mx_ref.values(codes, scales), w2, True, torch.finfo(y.dtype).eps)
    assert_within(y.double().cpu().numpy(), ref, bound + 2.0 ** -25)
