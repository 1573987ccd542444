// extern "C" entry points of the MXFP4 and mixture-of-experts operators:
// argument checks and launches on the caller's stream.  No exception leaves
// this file; every failure is a gptq_status code.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <new>

#include "gptq.h"
#include "mx_device.hpp"
#include "mx_kernels.hpp"

static_assert(gptq::kTypeF16 == GPTQ_TYPE_F16 && gptq::kTypeBf16 == GPTQ_TYPE_BF16 && gptq::kTypeF32 == GPTQ_TYPE_F32 &&
                  gptq::kTypeMxfp4 == GPTQ_TYPE_MXFP4,
              "type codes");

namespace {

constexpr int64_t kMaxElems = (int64_t)1 << 31;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// an MXFP4 matrix [rows, K] and its 16-bit or fp32 values
int check_mx(const void* values, const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K) {
  if (rows < 0 || K <= 0 || K % 32 != 0 || K > ((int64_t)1 << 20) || rows >= kMaxElems) return GPTQ_ERR_BAD_SHAPE;
  if (rows > 0 && (!values || !codes || !scales)) return GPTQ_ERR_NULL_PTR;
  if (!aligned(values, 16) || !aligned(codes, 16)) return GPTQ_ERR_MISALIGNED;
  return GPTQ_OK;
}

// one expert stack [rows -> cols]
int check_stack(const gptq_experts* s, int64_t rows, int64_t cols) {
  if (!s) return GPTQ_ERR_NULL_PTR;
  if (!s->weight || !s->scales) return GPTQ_ERR_NULL_PTR;
  if (rows * cols >= kMaxElems) return GPTQ_ERR_BAD_SHAPE;
  if (s->bits == 0) {
    if (!aligned(s->weight, 16)) return GPTQ_ERR_MISALIGNED;
    return GPTQ_OK;
  }
  if (s->bits != 2 && s->bits != 3 && s->bits != 4 && s->bits != 8) return GPTQ_ERR_BAD_BITS;
  if (!s->zeros) return GPTQ_ERR_NULL_PTR;
  if (s->group_size <= 0 || rows % s->group_size != 0 || s->group_size % 32 != 0) return GPTQ_ERR_BAD_GROUP;
  if ((s->is_v2 != 0 && s->is_v2 != 1) || (s->tiled != 0 && s->tiled != 1)) return GPTQ_ERR_BAD_ARG;
  if (!aligned(s->weight, 16) || !aligned(s->scales, 8) || !aligned(s->zeros, 4)) return GPTQ_ERR_MISALIGNED;
  return GPTQ_OK;
}

gptq::ExpertStack stack_of(const gptq_experts* s, int64_t rows, int64_t cols) {
  gptq::ExpertStack e{};
  e.weight = s->weight;
  e.scales = s->scales;
  e.bits = s->bits;
  if (s->bits == 0) {
    e.weight_stride = cols * rows / 2;
    e.scales_stride = cols * rows / 32;
    return e;
  }
  e.zeros = s->zeros;
  e.group_size = s->group_size;
  e.zero_offset = s->is_v2 ? 0 : 1;
  e.tiled = s->tiled;
  const int64_t G = rows / s->group_size;
  e.weight_stride = cols * rows / 8 * s->bits;
  e.zeros_stride = G * cols / 8 * s->bits;
  e.scales_stride = G * cols * 2;
  return e;
}

gptq::MxGemmArgs args_of(const void* x, int x_type, const uint8_t* x_scales, const uint8_t* codes,
                         const uint8_t* scales, int64_t M, int64_t N, int64_t K, void* out, int out_type) {
  gptq::MxGemmArgs a{};
  a.x = x;
  a.x_scales = x_scales;
  a.codes = codes;
  a.scales = scales;
  a.out = out;
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.x_type = x_type;
  a.out_type = out_type;
  return a;
}

int status_of(hipError_t err) { return err == hipSuccess ? GPTQ_OK : GPTQ_ERR_LAUNCH; }

}  // namespace

extern "C" {

int gptq_mxfp4_quantize_check(const void* x, int x_type, int64_t M, int64_t K, const uint8_t* codes,
                              const uint8_t* scales) {
  if (x_type < GPTQ_TYPE_F16 || x_type > GPTQ_TYPE_F32) return GPTQ_ERR_BAD_ARG;
  return check_mx(x, codes, scales, M, K);
}

int gptq_mxfp4_quantize(const void* x, int x_type, int64_t M, int64_t K, uint8_t* codes, uint8_t* scales,
                        void* stream) {
  const int rc = gptq_mxfp4_quantize_check(x, x_type, M, K, codes, scales);
  if (rc != GPTQ_OK || M == 0) return rc;
  return status_of(gptq::launch_mx_quantize(x, x_type, M, K, codes, scales, reinterpret_cast<hipStream_t>(stream)));
}

int gptq_mxfp4_dequant(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K, void* out, int out_type,
                       void* stream) {
  const int rc = gptq_mxfp4_quantize_check(out, out_type, M, K, codes, scales);
  if (rc != GPTQ_OK || M == 0) return rc;
  return status_of(gptq::launch_mx_dequant(codes, scales, M, K, out, out_type, reinterpret_cast<hipStream_t>(stream)));
}

int gptq_mxfp4_gemm_check(const void* x, int x_type, const uint8_t* x_scales, const uint8_t* codes,
                          const uint8_t* scales, int64_t M, int64_t N, int64_t K, const void* out, int out_type) {
  const bool fp4 = x_type == GPTQ_TYPE_MXFP4;
  if (!fp4 && x_type != GPTQ_TYPE_F16 && x_type != GPTQ_TYPE_BF16) return GPTQ_ERR_BAD_ARG;
  if (out_type < GPTQ_TYPE_F16 || out_type > GPTQ_TYPE_F32) return GPTQ_ERR_BAD_ARG;
  if (fp4 != (x_scales != nullptr) && M > 0) return fp4 ? GPTQ_ERR_NULL_PTR : GPTQ_ERR_BAD_ARG;
  if (M < 0 || N <= 0 || K <= 0 || K % 32 != 0 || M > ((int64_t)1 << 24) || N > ((int64_t)1 << 20) ||
      K > ((int64_t)1 << 20) || M * K >= kMaxElems || N * K >= kMaxElems || M * N >= kMaxElems)
    return GPTQ_ERR_BAD_SHAPE;
  if (!codes || !scales || (M > 0 && (!x || !out))) return GPTQ_ERR_NULL_PTR;
  if (!aligned(codes, 16) || !aligned(x, 16) || !aligned(out, 4)) return GPTQ_ERR_MISALIGNED;
  return GPTQ_OK;
}

int gptq_mxfp4_quantize_describe(int x_type, int64_t M, int64_t K, char* buf, int64_t buflen) {
  if (!buf || buflen <= 0) return GPTQ_ERR_NULL_PTR;
  buf[0] = '\0';
  if (x_type < GPTQ_TYPE_F16 || x_type > GPTQ_TYPE_F32) return GPTQ_ERR_BAD_ARG;
  const int rc = check_mx(nullptr, nullptr, nullptr, 0, K);
  if (rc != GPTQ_OK || M < 0 || M >= kMaxElems) return GPTQ_ERR_BAD_SHAPE;
  if (M == 0) std::snprintf(buf, (size_t)buflen, "none (M = 0)");
  else gptq::describe_mx_quantize(x_type, M, K, buf, (size_t)buflen);
  return GPTQ_OK;
}

int gptq_mxfp4_gemm_describe(const void* x, int x_type, const uint8_t* x_scales, const uint8_t* codes,
                             const uint8_t* scales, int64_t M, int64_t N, int64_t K, const void* out, int out_type,
                             char* buf, int64_t buflen) {
  if (!buf || buflen <= 0) return GPTQ_ERR_NULL_PTR;
  buf[0] = '\0';
  const int rc = gptq_mxfp4_gemm_check(x, x_type, x_scales, codes, scales, M, N, K, out, out_type);
  if (rc != GPTQ_OK) return rc;
  if (M == 0) {
    std::snprintf(buf, (size_t)buflen, "none (M = 0)");
  } else {
    gptq::MxGemmArgs a = args_of(x, x_type, x_scales, codes, scales, M, N, K, const_cast<void*>(out), out_type);
    size_t counters = 0;
    gptq::plan_mx_gemm(&a, true, &counters);
    const gptq::MxKernel k = gptq::mx_gemm_kernel(a);
    std::snprintf(buf, (size_t)buflen, "%s grid=%u block=%u k_splits=%d", k.name, k.grid, k.block, a.splits);
  }
  return GPTQ_OK;
}

int gptq_mxfp4_gemm(const void* x, int x_type, const uint8_t* x_scales, const uint8_t* codes, const uint8_t* scales,
                    int64_t M, int64_t N, int64_t K, void* out, int out_type, void* stream) {
  const int rc = gptq_mxfp4_gemm_check(x, x_type, x_scales, codes, scales, M, N, K, out, out_type);
  if (rc != GPTQ_OK || M == 0) return rc;
  gptq::MxGemmArgs a = args_of(x, x_type, x_scales, codes, scales, M, N, K, out, out_type);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  try {
    size_t counters = 0;
    const size_t bytes = gptq::plan_mx_gemm(&a, true, &counters);
    if (bytes > 0) {
      void* base = nullptr;
      if (gptq::stream_workspace(st, bytes, counters, &base, &a.cnt)) a.ws = static_cast<float*>(base);
      else gptq::plan_mx_gemm(&a, false, &counters);
    }
    return status_of(gptq::launch_mx_gemm(a, st));
  } catch (const std::bad_alloc&) {
    return GPTQ_ERR_NO_MEM;
  } catch (...) {
    return GPTQ_ERR_DEVICE;
  }
}

int gptq_moe_layer_check(const void* x, int x_type, const void* w_router, int64_t T, int64_t H, int64_t I, int64_t E,
                         int64_t k, int renormalize, const gptq_experts* gate_up, const gptq_experts* down,
                         const void* out) {
  if (x_type != GPTQ_TYPE_F16 && x_type != GPTQ_TYPE_BF16) return GPTQ_ERR_BAD_ARG;
  if (renormalize != 0 && renormalize != 1) return GPTQ_ERR_BAD_ARG;
  if (T < 0 || H <= 0 || I <= 0 || H % 32 != 0 || I % 32 != 0 || H > ((int64_t)1 << 20) || I > ((int64_t)1 << 19) ||
      T > ((int64_t)1 << 24) || T * H >= kMaxElems)
    return GPTQ_ERR_BAD_SHAPE;
  if (E < 1 || E > 1024 || k < 1 || k > 16 || k > E) return GPTQ_ERR_BAD_ARG;
  if (!w_router || (T > 0 && (!x || !out))) return GPTQ_ERR_NULL_PTR;
  int rc = check_stack(gate_up, H, 2 * I);
  if (rc == GPTQ_OK) rc = check_stack(down, I, H);
  if (rc != GPTQ_OK) return rc;
  if (!aligned(x, 16) || !aligned(w_router, 16) || !aligned(out, 16)) return GPTQ_ERR_MISALIGNED;
  return GPTQ_OK;
}

int gptq_moe_layer(const void* x, int x_type, const void* w_router, int64_t T, int64_t H, int64_t I, int64_t E,
                   int64_t k, int renormalize, const gptq_experts* gate_up, const gptq_experts* down, void* out,
                   void* stream_ptr) {
  try {
    const int rc = gptq_moe_layer_check(x, x_type, w_router, T, H, I, E, k, renormalize, gate_up, down, out);
    if (rc != GPTQ_OK || T == 0) return rc;
    hipStream_t stream = reinterpret_cast<hipStream_t>(stream_ptr);
    gptq::MoeArgs a{};
    a.w_router = w_router;
    a.bf16 = x_type == GPTQ_TYPE_BF16;
    a.H = (int)H;
    a.I = (int)I;
    a.E = (int)E;
    a.k = (int)k;
    a.renorm = renormalize;
    a.gate_up = stack_of(gate_up, H, 2 * I);
    a.down = stack_of(down, I, H);
    // more tokens than one launch takes: in turn
    const int64_t step = std::min<int64_t>(T, gptq::kMoeTokens);
    size_t bytes = 0, counters = 0;
    for (int64_t n : {step, T % step}) {             // full launches and the last one: their shapes differ
      if (n == 0) continue;
      size_t c = 0;
      a.T = (int)n;
      bytes = std::max(bytes, gptq::plan_moe(&a, nullptr, &c));
      counters = std::max(counters, c);
    }
    void* base = nullptr;
    uint32_t* cnt = nullptr;
    if (!gptq::stream_workspace(stream, bytes, counters, &base, &cnt)) return GPTQ_ERR_NO_MEM;
    a.cnt = cnt;
    for (int64_t t = 0; t < T; t += step) {
      a.T = (int)std::min(step, T - t);
      a.x = static_cast<const uint16_t*>(x) + t * H;
      a.out = static_cast<uint16_t*>(out) + t * H;
      size_t c = 0;
      gptq::plan_moe(&a, static_cast<char*>(base), &c);
      const hipError_t err = gptq::launch_moe(a, stream);
      if (err != hipSuccess) return GPTQ_ERR_LAUNCH;
    }
    return GPTQ_OK;
  } catch (const std::bad_alloc&) {
    return GPTQ_ERR_NO_MEM;
  } catch (...) {
    return GPTQ_ERR_DEVICE;
  }
}

}  // extern "C"
