// Device-side building blocks of the MXFP4 kernels.
//
// MXFP4: blocks of 32 consecutive k share one power-of-two scale
// 2^(byte - 127) (byte 255: the block is NaN); each value is a 4-bit e2m1 code
// (sign, two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two
// codes to a byte, the even k in the low nibble.  A matrix [R, K] is codes
// uint8 [R, K/2] and scales uint8 [R, K/32], row-major, so one block is 16
// contiguous bytes: the operand one lane holds for a gfx950 scaled MFMA.
//
// gfx950 converts between e2m1 and fp32 / fp16 / bf16 in hardware, a pair at a
// time under a power-of-two scale given as the exponent field of a float.
// Measured over all 256 codes pairs x 256 scale bytes: decoding equals the
// format's value rounded to nearest even in the target type (bf16 and fp32
// hold every value of bytes up to 252, the quantiser's largest, exactly; under
// 253 and 254 the large codes pass 2^128 and become infinities; fp16 is exact for
// bytes 104 .. 140), byte 0 is 2^-127 and byte 255 gives NaN; encoding rounds to
// nearest even and saturates at 6.
#pragma once

#include "gptq_device.hpp"

namespace gptq {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

constexpr int kTypeF16 = 0, kTypeBf16 = 1, kTypeF32 = 2, kTypeMxfp4 = 3;

__device__ __forceinline__ float mx_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// Eight codes (one dword, k order) under scale s -> eight fp16 or bf16 values.
template <bool BF16> __device__ __forceinline__ half8_t mx_frag(uint32_t w, float s) {
  u32x4_t r;
  if constexpr (BF16) {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
  } else {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 0));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 1));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 2));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 3));
  }
  return __builtin_bit_cast(half8_t, r);
}

// Whether fp16 holds every value of a block with this scale byte exactly:
// the smallest, 0.5 * 2^(byte - 127), is a multiple of 2^-24 from byte 104 on,
// the largest, 6 * 2^(byte - 127), at most 49152 up to byte 140.
__device__ __forceinline__ bool mx_fits_f16(uint32_t byte) { return byte - 104u <= 36u; }
// Whether a block's 32 codes are all +-0: zeros are zeros under any scale, and
// the quantiser gives a block of zeros byte 0 (fp16 x, 1% such blocks, us where
// they count as outside fp16's range and where not: 512 rows, 22016 x 4096, 374
// and 103; one row, 28672 x 8192, 51 and 30).
__device__ __forceinline__ bool mx_zero(const u32x4_t& c) { return ((c[0] | c[1] | c[2] | c[3]) & 0x77777777u) == 0; }

// fp16 values as the exact sum of two bf16 values (11 = 8 + 3 significant
// bits): the operands used where a block's scale is outside fp16's range.
__device__ __forceinline__ void split_f16(const half8_t& a, half8_t* hi, half8_t* lo) {
  u32x4_t h, l;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const float f0 = (float)a[2 * v], f1 = (float)a[2 * v + 1];
    h[v] = bf16_pair(f0, f1);
    const float h0 = __uint_as_float(h[v] << 16), h1 = __uint_as_float(h[v] & 0xFFFF0000u);
    // an infinity is its own high part
    l[v] = bf16_pair(h0 == f0 ? 0.f : f0 - h0, h1 == f1 ? 0.f : f1 - h1);
  }
  *hi = __builtin_bit_cast(half8_t, h);
  *lo = __builtin_bit_cast(half8_t, l);
}

// Under bytes 253 and 254 the large codes are beyond bf16 and fp32.  Where a wave
// meets such a byte it takes a quarter of all its weights, which bf16 holds
// exactly, four times (a block left out of some products would add 0 to them, and
// NaN beside an infinite activation).  No weights of any use come here.
constexpr uint32_t kMxExact = 252;
__device__ __forceinline__ bool mx_far(uint32_t byte) { return byte > kMxExact && byte < 255u; }
// Eight codes in bf16, or a quarter of them.
__device__ __forceinline__ half8_t mx_frag_bf16(bool quarter, uint32_t w, uint32_t byte) {
  if (!quarter) return mx_frag<true>(w, mx_scale(byte));
  const float s = mx_scale(byte == 255u || byte < 4u ? byte : byte - 2u), m = byte < 4u ? 0.25f : 1.f;
  const f32x2_t v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0), v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
  const f32x2_t v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2), v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
  const u32x4_t r = {bf16_pair(v0[0] * m, v0[1] * m), bf16_pair(v1[0] * m, v1[1] * m), bf16_pair(v2[0] * m, v2[1] * m),
                     bf16_pair(v3[0] * m, v3[1] * m)};
  return __builtin_bit_cast(half8_t, r);
}

template <bool BF16> __device__ __forceinline__ floatx4_t mfma16(const half8_t& a, const half8_t& b, const floatx4_t& c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
  else return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// 16 rows x 16 columns x 128 k of two MXFP4 operands: lane l holds row (or
// column) l % 16 and block l / 16 of each, 16 bytes of codes and, in byte SA /
// SB of the scale dwords, the block's scale.
template <int SA, int SB>
__device__ __forceinline__ floatx4_t mfma16_mx(const u32x4_t& a, const u32x4_t& b, const floatx4_t& c, uint32_t sa,
                                               uint32_t sb) {
  const i32x8_t a8 = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8_t b8 = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, 4, 4, SA, (int)sa, SB, (int)sb);
}

// 32 rows x 32 columns x 64 k: lane l holds row (or column) l % 32, block l / 32.
template <int SA, int SB>
__device__ __forceinline__ floatx16_t mfma32_mx(const u32x4_t& a, const u32x4_t& b, const floatx16_t& c, uint32_t sa,
                                                uint32_t sb) {
  const i32x8_t a8 = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8_t b8 = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, SA, (int)sa, SB, (int)sb);
}

// One fp32 result rounded once to the output type.
__device__ __forceinline__ void store_typed(void* out, int64_t i, float v, int type) {
  if (type == kTypeF16) static_cast<_Float16*>(out)[i] = (_Float16)v;
  else if (type == kTypeBf16) static_cast<uint16_t*>(out)[i] = (uint16_t)(bf16_pair(v, v) & 0xFFFFu);
  else static_cast<float*>(out)[i] = v;
}

// A byte range as a buffer resource: loads at offsets past its end return zero
// without touching memory, so tails and unused rows need no branch.
constexpr uint32_t kPast = 0xFFFFFFF0u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ u32x4_t load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0);
}
__device__ __forceinline__ uint32_t load4(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0);
}
__device__ __forceinline__ uint32_t load1(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return (uint32_t)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(r, (int)off, 0, 0);
}

// Values that another workgroup wrote in this launch go through agent-scope
// relaxed atomics, coherent across the XCDs' L2s by themselves.
template <class T> __device__ __forceinline__ void put_agent(T* p, T v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <class T> __device__ __forceinline__ T get_agent(const T* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Sum of the `n` splits' values at p, p + stride, ... in split order.  All loads
// are issued before the first is used: one after the other each would cost a
// trip past the L2s (a layer of 23 tokens over 16 splits spent 18 us on them).
template <int MAX> __device__ __forceinline__ float sum_splits(const float* p, int64_t stride, int n) {
  float v[MAX];
#pragma unroll
  for (int k = 0; k < MAX; ++k) v[k] = k < n ? get_agent(p + k * stride) : 0.f;
  float s = v[0];
#pragma unroll
  for (int k = 1; k < MAX; ++k) s += v[k];
  return s;
}
// Whether this workgroup is the last of `total` to arrive at cnt, which it then
// leaves at zero for the next launch.  A workgroup's stores complete (vmcnt 0,
// then a barrier) before its arrival is counted.
__device__ __forceinline__ bool last_arrival(uint32_t* cnt, uint32_t total, int* flag) {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0x0F70);
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __syncthreads();
  if (threadIdx.x == 0) {
    const bool last = __hip_atomic_fetch_add(cnt, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == total - 1;
    if (last) put_agent(cnt, 0u);
    *flag = last;
  }
  __syncthreads();
  return *flag != 0;
}

}  // namespace gptq
