// Products of few rows with MXFP4 weights, out[M, N] = x[M, K] . dequant(W[N, K])^T:
// the streaming product (stream_gemm.hpp), bound by the weights' bytes, with x
// in 16 bits, or in MXFP4 on the scaled MFMA, which multiplies 4-bit operands
// and their block scales directly.
#include <algorithm>
#include <cmath>

#include "mx_kernels.hpp"
#include "stream_gemm.hpp"

namespace gptq {

constexpr int kStreamSplits = 8;                   // workgroups along K per tile, at most

// A workgroup's results: the k waves' sums join in LDS, and with K split over
// workgroups the splits' sums through memory, added in split order by the last
// to arrive.  red: nwc nwk MT CT x 1 KB.
template <int MT, int CT>
__device__ __forceinline__ void finish_stream(const MxGemmArgs& a, const floatx4_t (&acc)[MT][CT], floatx4_t* red, int* flag,
                                              int n0, int nmt, int split, int tile) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cw = wave % a.nwc, kw = wave / a.nwc;
  if (a.nwk > 1) {
    __syncthreads();                               // the staged rows are no longer read
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (mt >= nmt) break;
#pragma unroll
      for (int j = 0; j < CT; ++j) red[(wave * MT * CT + mt * CT + j) * 64 + lane] = acc[mt][j];
    }
    __syncthreads();
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    if (mt >= nmt) break;
#pragma unroll
    for (int j = 0; j < CT; ++j) {
      const int t = mt * CT + j;
      if (t % a.nwk != kw) continue;
      floatx4_t s = acc[mt][j];
      if (a.nwk > 1) {
        s = red[(cw * MT * CT + t) * 64 + lane];
        for (int k = 1; k < a.nwk; ++k) s += red[((k * a.nwc + cw) * MT * CT + t) * 64 + lane];
      }
      const int m = 16 * mt + 4 * (lane >> 4), n = n0 + (cw * CT + j) * 16 + (lane & 15);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (m + i >= a.M || n >= a.N) continue;
        const int64_t o = (int64_t)(m + i) * a.N + n;
        if (a.splits > 1) put_agent(a.ws + (int64_t)split * a.M * a.N + o, s[i]);
        else store_typed(a.out, o, s[i], a.out_type);
      }
    }
  }
  if (a.splits == 1 || !last_arrival(a.cnt + tile, (uint32_t)a.splits, flag)) return;
  const int cols = 16 * CT * a.nwc;
  for (int i = threadIdx.x; i < a.M * cols; i += blockDim.x) {
    const int n = n0 + i % cols;
    if (n >= a.N) continue;
    const int64_t o = (int64_t)(i / cols) * a.N + n;
    store_typed(a.out, o, sum_splits<kStreamSplits>(a.ws + o, (int64_t)a.M * a.N, a.splits), a.out_type);
  }
}

// Workgroup -> (split, column tile); every workgroup has all rows, at most 16 MT.
struct StreamPlace {
  int split, tile, n0;
};
template <int CT> __device__ __forceinline__ StreamPlace place_of(const MxGemmArgs& a) {
  const int cols = 16 * CT * a.nwc, tiles = (a.N + cols - 1) / cols;
  const int b = (int)blockIdx.x, split = b / tiles, tile = b - split * tiles;
  return StreamPlace{split, tile, tile * cols};
}

// LDS of one phase: nwk k waves' units of x and every wave's units of weights.
template <bool BF16, int MT, int CT>
__global__ __launch_bounds__(512, MT == 1 ? 4 : 2) void mx_stream_kernel(MxGemmArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ uint32_t off[16 * MT];
  __shared__ int flag;
  typedef MxWeights<BF16, CT> W;
  const int lane = threadIdx.x & 63, nw = a.nwc * a.nwk;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cw = wave % a.nwc, kw = wave / a.nwc;
  const StreamPlace at = place_of<CT>(a);
  const int rows = a.M, nmt = (rows + 15) >> 4;
  W w;
  w.place(a.K, lane);
  w.bind(a.codes, a.scales, a.N, a.K);
#pragma unroll
  for (int j = 0; j < CT; ++j) w.row0[j] = (uint32_t)(at.n0 + (cw * CT + j) * 16);
  const int units = (a.K + W::KU - 1) / W::KU, ua = at.split * a.split_tiles, ub = min(units, ua + a.split_tiles);
  const int phases = (ub - ua + a.nwk - 1) / a.nwk;
  StagedRows x;
  x.rsrc = buffer_of(a.x, (uint32_t)a.M * (uint32_t)a.K * 2u);
  x.off = off;
  x.plane = 0;
  x.rows = rows;
  x.K = a.K;
  x.kp = a.nwk * W::KU;
  const uint32_t xbytes = (uint32_t)rows * x.kp * 2u, phase = xbytes + nw * W::BYTES;
  auto weights = [&](int p) __attribute__((always_inline)) { return lds + (p & 1) * phase + xbytes + wave * W::BYTES; };
  auto rows_at = [&](int p) __attribute__((always_inline)) { return lds + (p & 1) * phase; };
  typename W::Regs r0, r1;
  w.load(ua + kw, ua + kw < ub, weights(0), &r0);
  if (threadIdx.x < rows) off[threadIdx.x] = threadIdx.x * (uint32_t)a.K * 2u;
  __syncthreads();
  floatx4_t acc[MT][CT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int j = 0; j < CT; ++j) acc[mt][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};
  UnitOperand<W, MT> operand{nullptr, w, {}, (uint32_t)((lane & 15) < rows ? lane & 15 : 0), xbytes, kw * (W::KU / 8)};
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int m = 16 * mt + (lane & 15);
    operand.row[mt] = (uint32_t)(m < rows ? m : (int)operand.swz) * x.kp * 2u;
  }
  auto issue = [&](int p, typename W::Regs* r) __attribute__((always_inline)) {
    const int unit = ua + p * a.nwk + kw;
    w.load(unit, unit < ub, weights(p), r);
    x.template issue<1>((ua + p * a.nwk) * W::KU, ub * W::KU, rows_at(p), wave, nw, lane);
  };
  auto compute = [&](int p, const typename W::Regs& r) __attribute__((always_inline)) {
    const int unit = ua + p * a.nwk + kw;
    operand.lds = rows_at(p);
    if (unit < ub) w.template multiply<MT, 1>(weights(p), r, unit, operand, nmt, acc);
  };
  x.template issue<1>(ua * W::KU, ub * W::KU, rows_at(0), wave, nw, lane);
  for (int p = 0; p < phases; p += 2) {
    phase_ready();
    if (p + 1 < phases) issue(p + 1, &r1);
    compute(p, r0);
    if (p + 1 >= phases) break;
    phase_ready();
    if (p + 2 < phases) issue(p + 2, &r0);
    compute(p + 1, r1);
  }
  finish_stream<MT, CT>(a, acc, reinterpret_cast<floatx4_t*>(lds), &flag, at.n0, nmt, at.split, at.tile);
}

// MXFP4 activations: both operands' blocks as they are; lane l holds row l % 16
// of x and column l % 16 of W.  The column waves of one k wave share x.
template <int MT, int CT>
__global__ __launch_bounds__(512, 2) void mx4_stream_kernel(MxGemmArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ int flag;
  typedef MxTiles<MT> X;
  typedef MxTiles<CT> W;
  const int lane = threadIdx.x & 63, nw = a.nwc * a.nwk;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cw = wave % a.nwc, kw = wave / a.nwc;
  const StreamPlace at = place_of<CT>(a);
  const int nmt = (a.M + 15) >> 4;
  X x;
  x.place(a.K, lane);
  x.bind(static_cast<const uint8_t*>(a.x), a.x_scales, a.M, a.K);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) x.row0[mt] = 16u * (uint32_t)mt;
  W w;
  w.place(a.K, lane);
  w.bind(a.codes, a.scales, a.N, a.K);
#pragma unroll
  for (int j = 0; j < CT; ++j) w.row0[j] = (uint32_t)(at.n0 + (cw * CT + j) * 16);
  floatx4_t acc[MT][CT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int j = 0; j < CT; ++j) acc[mt][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};
  const int units = (a.K + 511) / 512, ua = at.split * a.split_tiles, ub = min(units, ua + a.split_tiles);
  const int phases = (ub - ua + a.nwk - 1) / a.nwk;
  const uint32_t phase = a.nwk * X::BYTES + nw * W::BYTES;
  typename X::Regs x0, x1;
  typename W::Regs w0, w1;
  auto xs_at = [&](int p) __attribute__((always_inline)) { return lds + (p & 1) * phase + kw * X::BYTES; };
  auto ws_at = [&](int p) __attribute__((always_inline)) {
    return lds + (p & 1) * phase + a.nwk * X::BYTES + wave * W::BYTES;
  };
  auto issue = [&](int p, typename X::Regs* xr, typename W::Regs* wr) __attribute__((always_inline)) {
    const int unit = ua + p * a.nwk + kw;
    w.load_scales(unit, unit < ub, wr);            // scales first, see MxWeights::load
    x.load_scales(unit, unit < ub, xr);
    w.load_codes(unit, unit < ub, ws_at(p), 0, 1);
    x.load_codes(unit, unit < ub, xs_at(p), cw, a.nwc);
  };
  auto compute = [&](int p, const typename X::Regs& xr, const typename W::Regs& wr) __attribute__((always_inline)) {
    const int unit = ua + p * a.nwk + kw;
    if (unit >= ub) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u32x4_t wv[CT];
      uint32_t ws[CT];
#pragma unroll
      for (int t = 0; t < CT; ++t) {
        wv[t] = w.block(ws_at(p), t, j);
        ws[t] = w.byte_of(wr, t, j, unit);
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        if (mt >= nmt) break;
        const u32x4_t xv = x.block(xs_at(p), mt, j);
        const uint32_t xs = x.byte_of(xr, mt, j, unit);
#pragma unroll
        for (int t = 0; t < CT; ++t) acc[mt][t] = mfma16_mx<0, 0>(xv, wv[t], acc[mt][t], xs, ws[t]);
      }
    }
  };
  issue(0, &x0, &w0);
  for (int p = 0; p < phases; p += 2) {
    phase_ready();
    if (p + 1 < phases) issue(p + 1, &x1, &w1);
    compute(p, x0, w0);
    if (p + 1 >= phases) break;
    phase_ready();
    if (p + 2 < phases) issue(p + 2, &x0, &w0);
    compute(p + 1, x1, w1);
  }
  finish_stream<MT, CT>(a, acc, reinterpret_cast<floatx4_t*>(lds), &flag, at.n0, nmt, at.split, at.tile);
}

// Dynamic LDS of a launch: two phases, or the k waves' sums.
template <int MT, int CT> size_t stream_lds(const MxGemmArgs& a) {
  const size_t nw = (size_t)a.nwc * a.nwk, sums = a.nwk > 1 ? nw * MT * CT * 1024 : 0;
  const size_t x = a.x_type == kTypeMxfp4 ? (size_t)a.nwk * MT * 4096 : (size_t)a.M * a.nwk * 1024;
  return std::max(sums, 2 * (x + nw * CT * 4096));
}

// (the kernels add less than 1 KB of static LDS)
constexpr size_t kStreamLds = 158 * 1024;
size_t lds_of(const MxGemmArgs& a) {
  return a.M <= 16 ? stream_lds<1, 1>(a) : a.M <= 32 ? stream_lds<2, 1>(a) : stream_lds<4, 1>(a);
}

// (16-bit x has at most 32 rows here: MT <= 2)
template <int MT, int CT> MxKernel stream_kernel_of(const MxGemmArgs& a, const char* const (&names)[3]) {
  const int cols = 16 * CT * a.nwc;
  MxKernel k{mx4_stream_kernel<MT, CT>, names[0], 0, 64u * (unsigned)(a.nwc * a.nwk), stream_lds<MT, CT>(a)};
  k.grid = (unsigned)((a.N + cols - 1) / cols) * (unsigned)a.splits;
  if constexpr (MT <= 2) {
    if (a.x_type == kTypeBf16) k.fn = mx_stream_kernel<true, MT, CT>, k.name = names[1];
    else if (a.x_type == kTypeF16) k.fn = mx_stream_kernel<false, MT, CT>, k.name = names[2];
  } else if (a.x_type != kTypeMxfp4) {
    k.fn = nullptr;                                // not planned
  }
  return k;
}

size_t plan_mx_gemm(MxGemmArgs* a, bool allow_split, size_t* counter_bytes) {
  *counter_bytes = 0;
  a->tile_m = 0;
  a->splits = 1;
  const bool mx = a->x_type == kTypeMxfp4;
  // 16-bit x of more than 32 rows: the staged rows leave no LDS for weights in
  // flight (64 rows of 12288 x 4096: 91 us that way, 21 as tiles)
  if (a->M <= (mx ? 64 : 32)) {
    // column and k waves per workgroup, measured on MI355X (us; c4k2: four
    // column waves by two k waves; s4: four workgroups along K per tile).
    // 16-bit x: one row, 12288 x 4096 c1k4 8.1, c2k2 8.2; 28672 x 8192 c1k4 31.1,
    // c4k2 28.7.  Sixteen rows, 12288 x 4096 c4k2 11.9, c1k4 34; 4096 x 11008 c4k2
    // s4 12.8, s2 16.9.  More column waves share each staged row of x.  MXFP4 x,
    // 12288 x 4096: one row c2k2 6.7, c1k4 8.1; 17 rows c2k2 8.6, c4k2 8.8; 64
    // rows c4k2 14.0, c4k1 16.0.
    const int units = (a->K + 511) / 512;
    if (mx) {
      a->nwc = a->M <= 32 ? 2 : 4;
      a->nwk = 2;
    } else {
      a->nwc = a->M <= 4 ? 1 : 4;
      a->nwk = a->M <= 4 ? 4 : 2;
    }
    while (a->nwk > 1 && (a->nwk / 2 >= units || lds_of(*a) > kStreamLds)) a->nwk /= 2;
    while (a->nwc > 1 && lds_of(*a) > kStreamLds) a->nwc /= 2;
    // fewer tiles than CUs: split K, two phases at least per workgroup
    const int cols = 16 * a->nwc, tiles = (a->N + cols - 1) / cols;
    int splits = 1;
    if (allow_split) splits = std::max(1, std::min({256 / tiles, units / (2 * a->nwk), kStreamSplits}));
    a->split_tiles = (units + splits - 1) / splits;
    a->splits = (units + a->split_tiles - 1) / a->split_tiles;
    if (a->splits == 1) return 0;
    *counter_bytes = (size_t)tiles * 4;
    return (size_t)a->splits * (size_t)a->M * (size_t)a->N * 4;
  }
  // Tiles: rows per tile and splits of K by a time model (us) of the measured
  // times: k tiles in a row, times the workgroups a CU takes in turn, plus a
  // split's fixed cost and its partial sums' traffic.  16-bit x: 0.9 per k tile of
  // 128 rows and 0.72 of 64 (512 x 22016 x 4096: 101 and 119 us; 64 x 12288 x 4096
  // takes 21.5 where the model says 17.6; 256-row tiles, one wave per SIMD, were
  // slower or equal everywhere); MXFP4: 1 per k tile of 128 x 128, two workgroups
  // to a CU, and 2.6 of 256 x 256 (2048 x 28672 x 8192: 376 and 306 us; 700 x 5000 x
  // 4096: 16 and 32).
  const int kt = mx ? 256 : 64, ktiles = (a->K + kt - 1) / kt;
  a->pair_stores = a->N % 2 == 0;
  a->quad_stores = (reinterpret_cast<uintptr_t>(a->out) & 15) == 0;
  double best = 0.0;
  for (int tm : {64, 128, 256}) {
    if (mx ? tm == 64 : tm == 256) continue;
    const int tn = mx ? tm : 256;
    const int64_t tiles = (int64_t)((a->M + tm - 1) / tm) * ((a->N + tn - 1) / tn);
    const double per_tile = mx ? (tm == 128 ? 1.0 : 2.6) : tm == 128 ? 0.9 : 0.72;
    for (int splits = 1; splits <= (allow_split ? 16 : 1); ++splits) {
      const int each = (ktiles + splits - 1) / splits, used = (ktiles + each - 1) / each;
      const double traffic = (double)used * a->M * a->N * 4;
      if (splits > 1 && (each < 2 || traffic > (double)(64 << 20))) break;
      const double turns = std::ceil((double)tiles * used / 256);
      const double time = each * per_tile * turns +
                          (used > 1 ? 4.3 + 2 * traffic / 8e6 : 0.0);
      if (best == 0.0 || time < best) {
        best = time;
        a->tile_m = tm;
        a->tile_n = tn;
        a->splits = used;
        a->split_tiles = each;
      }
    }
  }
  a->tiles_m = (a->M + a->tile_m - 1) / a->tile_m;
  a->tiles_n = (a->N + a->tile_n - 1) / a->tile_n;
  return a->splits > 1 ? (size_t)a->splits * (size_t)a->M * (size_t)a->N * 4 : 0;
}

MxKernel mx_gemm_kernel(const MxGemmArgs& a) {
  if (a.tile_m != 0) return mx_tile_kernel_of(a);
  if (a.M <= 16)
    return stream_kernel_of<1, 1>(a, {"gptq::mx4_stream_kernel<1, 1>", "gptq::mx_stream_kernel<true, 1, 1>",
                                      "gptq::mx_stream_kernel<false, 1, 1>"});
  if (a.M <= 32)
    return stream_kernel_of<2, 1>(a, {"gptq::mx4_stream_kernel<2, 1>", "gptq::mx_stream_kernel<true, 2, 1>",
                                      "gptq::mx_stream_kernel<false, 2, 1>"});
  return stream_kernel_of<4, 1>(a, {"gptq::mx4_stream_kernel<4, 1>", "", ""});
}

hipError_t launch_mx_kernel(const MxKernel& k, const MxGemmArgs& a, hipStream_t stream) {
  if (k.fn == nullptr) return hipErrorInvalidValue;
  if (k.lds > 64 * 1024) {
    const hipError_t err =
        hipFuncSetAttribute(reinterpret_cast<const void*>(k.fn), hipFuncAttributeMaxDynamicSharedMemorySize, (int)k.lds);
    if (err != hipSuccess) return err;
  }
  k.fn<<<k.grid, k.block, k.lds, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_mx_gemm(const MxGemmArgs& a, hipStream_t stream) {
  return a.tile_m != 0 ? launch_mx_tile(a, stream) : launch_mx_kernel(mx_gemm_kernel(a), a, stream);
}

}  // namespace gptq
