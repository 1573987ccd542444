// MXFP4 quantisation and its inverse: elementwise, bound by HBM.
//
// Quantise: block of 32 values -> byte = max(e - 2, 0), e the exponent field of
// the block's largest magnitude in fp32 (2^(byte - 127) is then the largest
// power of two that puts that magnitude into the format's top binade, 4 .. 8),
// then each value over the scale to the nearest e2m1 code (ties to even,
// saturating at 6).  A lane takes 16 consecutive bytes, so that every load and
// store of a wave is one contiguous run; four lanes (eight for fp32) share a
// block: the largest magnitude is a maximum of the absolute values' bit
// patterns (monotonic, and infinities and NaN come out on top), lane exchanges
// join them.  Measured, 28672 x 8192: bf16 92 us quantise (6.4 TB/s), 84 us back
// (7.1); fp32 170 us quantise, 144 us back (7.4).
#include <algorithm>
#include <cstdio>

#include "mx_device.hpp"
#include "mx_kernels.hpp"

namespace gptq {

// Pieces of 16 bytes a thread quantises: 4, their loads in flight together, where
// every CU still gets eight workgroups, else 1 (us with 4 and with 1: 28672 x 8192
// bf16 92 and 98, 2048 x 8192 fp16 8.8 and 9.7; 512 x 8192 bf16 4.0 and 3.7, 333 x
// 4096 fp16 3.2 and 2.8).  Dequantising, mostly stores, takes 1 at any size (84
// against 87 at 28672 x 8192 bf16).
constexpr int kMxPieces = 4;
constexpr int64_t kMxWideFrom = (int64_t)256 * 8 * 256 * kMxPieces;

// A lane's 16 bytes: eight values of a 16-bit type, four of fp32.
// Largest magnitude's bits of one lane's values.
template <int TYPE> __device__ __forceinline__ uint32_t top_bits(const u32x4_t& r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (TYPE == kTypeF32) {
      m = max(m, r[i] & 0x7FFFFFFFu);
    } else {
      const uint32_t a = r[i] & 0x7FFF7FFFu;
      m = max(m, max(a & 0xFFFFu, a >> 16));
    }
  }
  return m;
}

template <int TYPE> __device__ __forceinline__ uint32_t exponent_of(uint32_t bits) {
  if constexpr (TYPE == kTypeF32) return bits >> 23;
  else if constexpr (TYPE == kTypeBf16) return bits >> 7;
  else return __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)bits)) >> 23;
}

// The lane's codes: eight in a word, four (fp32) in its low half.
template <int TYPE> __device__ __forceinline__ uint32_t encode(const u32x4_t& r, float s) {
  uint32_t w = 0;
  if constexpr (TYPE == kTypeF32) {
    auto f = [](uint32_t u) __attribute__((always_inline)) { return __uint_as_float(u); };
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f(r[0]), f(r[1]), s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f(r[2]), f(r[3]), s, 1);
  } else if constexpr (TYPE == kTypeBf16) {
    auto p = [](uint32_t u) __attribute__((always_inline)) { return __builtin_bit_cast(bf16x2_t, u); };
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, p(r[0]), s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, p(r[1]), s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, p(r[2]), s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, p(r[3]), s, 3);
  } else {
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, as_half2(r[0]), s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, as_half2(r[1]), s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, as_half2(r[2]), s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, as_half2(r[3]), s, 3);
  }
  return w;
}

// `pieces` of 16 bytes of x, a multiple of the lanes that share a block: those
// are all inside or all past the end.
template <int TYPE, int U>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const void* __restrict__ x, int64_t pieces,
                                                          void* __restrict__ codes, uint8_t* __restrict__ scales) {
  constexpr bool F32 = TYPE == kTypeF32;
  const int64_t first = (int64_t)blockIdx.x * (256 * U) + threadIdx.x;
  u32x4_t r[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (first + 256 * u < pieces) r[u] = __builtin_nontemporal_load(static_cast<const u32x4_t*>(x) + first + 256 * u);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t p = first + 256 * u;
    if (p >= pieces) break;
    uint32_t m = top_bits<TYPE>(r[u]);
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));   // lanes 1 0 3 2
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));   // lanes 2 3 0 1
    if constexpr (F32) m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x141, 0xF, 0xF, true));   // lanes 7 .. 0
    const uint32_t e = exponent_of<TYPE>(m);
    const uint32_t byte = e == 255u ? 255u : e > 2u ? e - 2u : 0u;
    const uint32_t w = e == 255u ? 0u : encode<TYPE>(r[u], mx_scale(byte));
    if constexpr (F32) static_cast<uint16_t*>(codes)[p] = (uint16_t)w;
    else static_cast<uint32_t*>(codes)[p] = w;
    if ((threadIdx.x & (F32 ? 7 : 3)) == 0) scales[p >> (F32 ? 3 : 2)] = (uint8_t)byte;
  }
}

// One 16-byte store per piece, contiguous over a wave: a piece is eight values
// of a 16-bit type or four of fp32 (two stores of half lines per eight fp32
// values took 398 us for 28672 x 8192, 1.06 GB; whole lines 144).
template <int TYPE>
__global__ __launch_bounds__(256) void mx_dequant_kernel(const void* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales, int64_t pieces,
                                                         void* __restrict__ out) {
  constexpr bool F32 = TYPE == kTypeF32;
  const int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (p >= pieces) return;
  const uint32_t w = F32 ? (uint32_t)static_cast<const uint16_t*>(codes)[p] : static_cast<const uint32_t*>(codes)[p];
  const float s = mx_scale(scales[p >> (F32 ? 3 : 2)]);
  if constexpr (F32) {
    const f32x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0);
    const f32x2_t hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
    __builtin_nontemporal_store(floatx4_t{lo[0], lo[1], hi[0], hi[1]}, static_cast<floatx4_t*>(out) + p);
  } else {
    const half8_t v = mx_frag<TYPE == kTypeBf16>(w, s);
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4_t, v), static_cast<u32x4_t*>(out) + p);
  }
}

// Pieces of one launch: a grid holds fewer than 2^32 threads.  64 GiB of
// dequantised values are that many, and a larger grid wraps without an error.
constexpr int64_t kMxLaunchPieces = (int64_t)1 << 30;

template <int TYPE>
hipError_t quantize_typed(const void* x, int64_t pieces, uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  constexpr int CODES = TYPE == kTypeF32 ? 2 : 4, PER_BLOCK = TYPE == kTypeF32 ? 8 : 4;   // bytes, pieces of a block
  for (int64_t p = 0; p < pieces; p += kMxLaunchPieces) {
    const int64_t n = std::min(pieces - p, kMxLaunchPieces);
    const void* xs = static_cast<const char*>(x) + 16 * p;
    uint8_t *c = codes + CODES * p, *s = scales + p / PER_BLOCK;
    if (n >= kMxWideFrom) {
      const unsigned grid = (unsigned)((n + 256 * kMxPieces - 1) / (256 * kMxPieces));
      mx_quantize_kernel<TYPE, kMxPieces><<<grid, 256, 0, stream>>>(xs, n, c, s);
    } else {
      mx_quantize_kernel<TYPE, 1><<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(xs, n, c, s);
    }
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

template <int TYPE>
hipError_t dequant_typed(const uint8_t* codes, const uint8_t* scales, int64_t pieces, void* out, hipStream_t stream) {
  constexpr int CODES = TYPE == kTypeF32 ? 2 : 4, PER_BLOCK = TYPE == kTypeF32 ? 8 : 4;
  for (int64_t p = 0; p < pieces; p += kMxLaunchPieces) {
    const int64_t n = std::min(pieces - p, kMxLaunchPieces);
    mx_dequant_kernel<TYPE><<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(codes + CODES * p, scales + p / PER_BLOCK, n,
                                                                            static_cast<char*>(out) + 16 * p);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

void describe_mx_quantize(int type, int64_t M, int64_t K, char* buf, size_t n) {
  const int64_t pieces = M * K / (type == kTypeF32 ? 4 : 8), one = std::min(pieces, kMxLaunchPieces);
  const int per = one >= kMxWideFrom ? kMxPieces : 1;
  std::snprintf(buf, n, "gptq::mx_quantize_kernel<%d, %d> grid=%lld block=256 launches=%lld", type, per,
                       (long long)((one + 256 * per - 1) / (256 * per)),
                       (long long)((pieces + kMxLaunchPieces - 1) / kMxLaunchPieces));
}

hipError_t launch_mx_quantize(const void* x, int type, int64_t M, int64_t K, uint8_t* codes, uint8_t* scales,
                              hipStream_t stream) {
  const int64_t pieces = M * K / (type == kTypeF32 ? 4 : 8);
  if (type == kTypeF16) return quantize_typed<kTypeF16>(x, pieces, codes, scales, stream);
  if (type == kTypeBf16) return quantize_typed<kTypeBf16>(x, pieces, codes, scales, stream);
  return quantize_typed<kTypeF32>(x, pieces, codes, scales, stream);
}

hipError_t launch_mx_dequant(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K, void* out, int type,
                             hipStream_t stream) {
  const int64_t pieces = M * K / (type == kTypeF32 ? 4 : 8);
  if (type == kTypeF16) return dequant_typed<kTypeF16>(codes, scales, pieces, out, stream);
  if (type == kTypeBf16) return dequant_typed<kTypeBf16>(codes, scales, pieces, out, stream);
  return dequant_typed<kTypeF32>(codes, scales, pieces, out, stream);
}

}  // namespace gptq
