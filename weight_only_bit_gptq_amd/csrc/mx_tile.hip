// Products of many rows with MXFP4 weights: out = x . dequant(W)^T as an MFMA
// GEMM over tiles, x in fp16 / bf16 (32x32x16 MFMA on weights converted in
// registers) or in MXFP4 (32x32x64 scaled MFMA on the codes).  Rows go to LDS 128
// bytes at a time (64 k of 16 bits, 256 of MXFP4) by buffer loads with an LDS
// destination, 16-byte slots XOR-swizzled so that the 16 rows one LDS read
// serves at once fall into 16 different bank groups.  Which k a matrix
// instruction takes is free as long as both operands agree.  Offsets past a
// tensor read zero without touching memory, so tails in k, M and N need no
// branch.
#include <algorithm>
#include <type_traits>

#include "mx_kernels.hpp"
#include "stream_gemm.hpp"

namespace gptq {

// ---- x in 16 bits: BM x 256 tiles, 64 k per k tile.  Four waves split the
// columns, so no two convert or load the same weights, which go from global
// memory straight into registers in operand order: half h of a wave (lanes
// 32 h ..) holds block h of a tile for its two columns.  x goes through three LDS
// stages; loads run two k tiles ahead.
template <bool BF16, int BM>
__device__ __forceinline__ void mx_tile_body(const MxGemmArgs& a) {
  constexpr int MS = BM / 32, XI = BM / 32;        // 1 KB x loads per wave and tile
  constexpr int KT = 64, NT = 2;                   // k per tile, 32-column tiles per wave
  __shared__ __align__(16) uint8_t lds0[BM * 128];
  __shared__ __align__(16) uint8_t lds1[BM * 128];
  __shared__ __align__(16) uint8_t lds2[BM * 128];
  auto stage = [&](auto c) __attribute__((always_inline)) -> uint8_t* {
    constexpr int s = decltype(c)::value;
    return s == 0 ? lds0 : s == 1 ? lds1 : lds2;
  };
  const int tid = threadIdx.x, lane = tid & 63, c = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // workgroup -> split, tile: tiles in column-major order, consecutive ones on
  // one XCD (workgroups are dealt round-robin over the eight)
  const int nt = a.tiles_m * a.tiles_n;
  const int per = (nt + 7) >> 3;
  const int b = (int)blockIdx.x, sk = b / (8 * per), bt = b - sk * 8 * per;
  const int t = (bt & 7) * per + (bt >> 3);
  if (t >= nt) return;
  const int m0 = t % a.tiles_m * BM, n0 = t / a.tiles_m * 128 * NT + wave * 32 * NT;
  const int all = (a.K + KT - 1) / KT, kt0 = sk * a.split_tiles, ktiles = min(a.split_tiles, all - kt0);
  const uint32_t rowb = (uint32_t)a.K * 2u;          // bytes of a row of x
  // ends of this split's part of K, as bytes of a row of x and as blocks
  const int blocks = a.K / 32;
  const uint32_t x_end = min(rowb, (uint32_t)(kt0 + ktiles) * 128u);
  const int w_end = min(blocks, (kt0 + ktiles) * (KT / 32));

  // ---- x
  const __amdgpu_buffer_rsrc_t xr = buffer_of(a.x, (uint32_t)a.M * rowb);
  uint32_t xoff[XI], xk[XI];                       // row offset (or past the end) and byte within the row
#pragma unroll
  for (int i = 0; i < XI; ++i) {
    const int s = (XI * wave + i) * 64 + lane, m = s >> 3;
    xoff[i] = m0 + m < a.M ? (uint32_t)(m0 + m) * rowb : 0xF0000000u;
    xk[i] = 16u * (uint32_t)((s & 7) ^ ((m >> 1) & 7));
  }
  auto load_x = [&](int kt, auto st) __attribute__((always_inline)) {
    uint8_t* sl = stage(st);
    const uint32_t at = (uint32_t)(kt0 + kt) * 128u;
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      const bool ok = at + xk[i] < x_end;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, (__attribute__((address_space(3))) void*)(sl + (XI * wave + i) * 1024),
                                               16, (int)(ok ? xoff[i] + at + xk[i] : kPast), 0, 0, 0);
    }
  };
  // ---- weights: lane (c, h) holds columns NT c + j of the wave's 32 NT
  const __amdgpu_buffer_rsrc_t wr = buffer_of(a.codes, (uint32_t)a.N * (uint32_t)(a.K / 2));
  const __amdgpu_buffer_rsrc_t wsr = buffer_of(a.scales, (uint32_t)a.N * (uint32_t)blocks);
  uint32_t wrow[NT], srow[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int n = min(n0 + NT * c + j, a.N - 1);
    wrow[j] = (uint32_t)n * (uint32_t)(a.K / 2);
    srow[j] = (uint32_t)n * (uint32_t)blocks;
  }
  u32x4_t w[3][NT];
  uint32_t ws[3][NT];
  auto load_w = [&](int kt, auto st) __attribute__((always_inline)) {
    constexpr int s = decltype(st)::value;
    const int blk = 2 * (kt0 + kt) + h;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      w[s][j] = load16(wr, blk < w_end ? wrow[j] + 16u * (uint32_t)blk : kPast);
      ws[s][j] = load1(wsr, blk < w_end ? srow[j] + (uint32_t)blk : kPast);
    }
  };

  floatx16_t acc[MS][NT];
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MS; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  };
  clear();
  bool fits = true;                                // fp16 x: every scale met lies in fp16's range
  uint32_t top = 0;                                // bf16 x: the largest scale byte met

  // 16 bytes of row 32 i + c at the half's slot of step s
  auto read_x = [&](const uint8_t* sl, int i, int s) __attribute__((always_inline)) {
    const int m = 32 * i + c;
    return *reinterpret_cast<const u32x4_t*>(sl + m * 128 + (((4 * h + s) ^ ((m >> 1) & 7)) * 16));
  };

  auto mfma = [&](const u32x4_t& xv, const half8_t& wv, const floatx16_t& d, auto bf) __attribute__((always_inline)) {
    if constexpr (decltype(bf)::value)
      return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, xv), __builtin_bit_cast(bf16x8_t, wv), d,
                                                     0, 0, 0);
    else return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8_t, xv), wv, d, 0, 0, 0);
  };
  auto compute = [&](int kt, auto st) __attribute__((always_inline)) {
    constexpr int s3 = decltype(st)::value;
    const uint8_t* sl = stage(st);
    if constexpr (BF16) {
#pragma unroll
      for (int j = 0; j < NT; ++j) top = max(top, ws[s3][j]);
    } else {
      bool inside = true;
#pragma unroll
      for (int j = 0; j < NT; ++j) inside = inside && mx_fits_f16(ws[s3][j]);
      if (!__all(inside)) {                        // ordinary weights do not come here
#pragma unroll
        for (int j = 0; j < NT; ++j)
          fits = fits && (mx_fits_f16(ws[s3][j]) || mx_zero(w[s3][j]) || 2 * (kt0 + kt) + h >= w_end);
      }
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      half8_t wv[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) wv[j] = mx_frag<BF16>(w[s3][j][s], mx_scale(ws[s3][j]));
#pragma unroll
      for (int i = 0; i < MS; ++i) {
        const u32x4_t xv = read_x(sl, i, s);
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = mfma(xv, wv[j], acc[i][j], std::bool_constant<BF16>());
      }
    }
  };

  // One k tile.  Loads come in the order x, weights, tile after tile: all but the
  // newest tile's have arrived after this wait (per wave; the barrier makes it
  // all waves'), among them tile kt's x.
  constexpr int PER_TILE = XI + 2 * NT;
  auto step = [&](int kt, auto st, auto far) __attribute__((always_inline)) {
    // vmcnt(PER_TILE), lgkmcnt(0)
    __builtin_amdgcn_s_waitcnt((PER_TILE & 0xF) | ((PER_TILE >> 4) << 14) | 0x70);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    load_x(kt + 2, far);
    load_w(kt + 2, far);
    compute(kt, st);
  };
  typedef std::integral_constant<int, 0> S0;
  typedef std::integral_constant<int, 1> S1;
  typedef std::integral_constant<int, 2> S2;
  load_x(0, S0{});
  load_w(0, S0{});
  load_x(1, S1{});
  load_w(1, S1{});
  // tiles past the last (the loop runs in threes) multiply zeros
  for (int kt = 0; kt < ktiles; kt += 3) {
    step(kt, S0{}, S2{});
    step(kt + 1, S1{}, S0{});
    step(kt + 2, S2{}, S1{});
  }

  // a scale outside the type's range, for fp16 of a block that is not all zeros,
  // somewhere in the tile's columns (weights of ordinary size never meet one): the
  // tile again with the weights in bf16 and fp16 x as two bf16 parts
  if (__syncthreads_or((BF16 ? top <= kMxExact : fits) ? 0 : 1)) {
    clear();
    for (int kt = 0; kt < ktiles; ++kt) {
      __syncthreads();
      load_x(kt, S0{});
      load_w(kt, S0{});
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
      bool far = false;
#pragma unroll
      for (int j = 0; j < NT; ++j) far = far || mx_far(ws[0][j]);
      far = __any(far);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        half8_t wv[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) wv[j] = mx_frag_bf16(far, w[0][j][s], ws[0][j]);
#pragma unroll
        for (int i = 0; i < MS; ++i) {
          half8_t hi = __builtin_bit_cast(half8_t, read_x(lds0, i, s)), lo;
          if (!BF16) split_f16(hi, &hi, &lo);
#pragma unroll 1
          for (int times = far ? 4 : 1; times > 0; --times)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              acc[i][j] = mfma(__builtin_bit_cast(u32x4_t, hi), wv[j], acc[i][j], std::true_type());
              if (!BF16) acc[i][j] = mfma(__builtin_bit_cast(u32x4_t, lo), wv[j], acc[i][j], std::true_type());
            }
        }
      }
    }
  }

  // ---- results: NT adjacent columns per lane; one compact loop per kind of
  // store (a body with every kind in it is not unrolled, and the sums then
  // live in memory)
  const int n = n0 + NT * c;
  auto each = [&](auto store) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MS; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int m = m0 + 32 * i + 8 * (v >> 2) + 4 * h + (v & 3);
        if (m < a.M) store((int64_t)m * a.N + n, acc[i][0][v], acc[i][1][v]);
      }
  };
  const bool ok0 = n < a.N, ok1 = n + 1 < a.N;
  if (a.splits > 1 || a.out_type == kTypeF32) {
    float* out = a.splits > 1 ? a.ws + (int64_t)sk * a.M * a.N : static_cast<float*>(a.out);
    each([&](int64_t o, float v0, float v1) __attribute__((always_inline)) {
      if (ok0) out[o] = v0;
      if (ok1) out[o + 1] = v1;
    });
  } else if (a.pair_stores) {
    if (!ok0) return;
    uint32_t* out = static_cast<uint32_t*>(a.out);
    if (a.out_type == kTypeBf16)
      each([&](int64_t o, float v0, float v1) __attribute__((always_inline)) { out[o >> 1] = bf16_pair(v0, v1); });
    else
      each([&](int64_t o, float v0, float v1) __attribute__((always_inline)) {
        out[o >> 1] = as_u32(half2_t{(_Float16)v0, (_Float16)v1});
      });
  } else {
    uint16_t* out = static_cast<uint16_t*>(a.out);
    const bool bf = a.out_type == kTypeBf16;
    each([&](int64_t o, float v0, float v1) __attribute__((always_inline)) {
      const uint32_t p = bf ? bf16_pair(v0, v1) : as_u32(half2_t{(_Float16)v0, (_Float16)v1});
      if (ok0) out[o] = (uint16_t)p;
      if (ok1) out[o + 1] = (uint16_t)(p >> 16);
    });
  }
}

template <bool BF16, int BM> __global__ __launch_bounds__(256, 2) void mx_tile_kernel(MxGemmArgs a) {
  mx_tile_body<BF16, BM>(a);
}

// ---- x in MXFP4: 64 W x 64 W tiles, 256 k per k tile.  Four waves, two by two,
// each W x W matrix-instruction tiles.  Rows of x and of W both go through LDS
// (a wave's own rows straight into registers meet 64 cache lines per load, 16
// bytes of each, and then bound the kernel: 346 us at 2048 x 28672 x 8192, with
// W = 4, for 306 to 317 now), S stages, S - 1 k tiles ahead: two where two workgroups
// share a CU or the tile is large, four where there is at most a workgroup per
// CU (333 x 4096 x 11008: 22 us with four, 24 with two).  Half h of a wave
// takes blocks 4 h + s in step s, so a lane's four scale bytes are one dword;
// scale bytes go to a table [row][2 dwords] per stage.
// What a step multiplies was read during the step before: with one wave per
// SIMD (W = 4: 256 sums per lane) nothing else hides an LDS read.
template <int W, int S, bool ALIGNED>
__global__ __launch_bounds__(256, W == 4 || S == 4 ? 1 : 2) void mx4_tile_kernel(MxGemmArgs a) {
  static_assert(ALIGNED || S == 2, "scale bytes through registers: one tile ahead");
  constexpr int B = 64 * W, ROWS = 2 * B, LOADS = ROWS / 32, SR = ROWS / 256;   // rows of both, 1 KB loads per wave
  constexpr int SL = ROWS / 128;                   // 256-byte scale loads per wave (ALIGNED)
  constexpr int STAGE = ROWS * 128, TABLE = ROWS * 8;
  extern __shared__ __align__(16) uint8_t lds[];   // S stages, S tables
  const int tid = threadIdx.x, lane = tid & 63, c = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nt = a.tiles_m * a.tiles_n;
  const int per = (nt + 7) >> 3;
  const int b = (int)blockIdx.x, sk = b / (8 * per), bt = b - sk * 8 * per;
  const int t = (bt & 7) * per + (bt >> 3);
  if (t >= nt) return;
  const int m0 = t % a.tiles_m * B, n0 = t / a.tiles_m * B;
  const uint32_t rowb = (uint32_t)a.K / 2, blocks = (uint32_t)a.K / 32;
  const int all = (a.K + 255) / 256, kt0 = sk * a.split_tiles, ktiles = min(a.split_tiles, all - kt0);

  const __amdgpu_buffer_rsrc_t xr = buffer_of(a.x, (uint32_t)a.M * rowb), wr = buffer_of(a.codes, (uint32_t)a.N * rowb);
  const __amdgpu_buffer_rsrc_t xsr = buffer_of(a.x_scales, (uint32_t)a.M * blocks),
                               wsr = buffer_of(a.scales, (uint32_t)a.N * blocks);
  // load i of wave w fills rows 8 (LOADS w + i) + lane / 8 of the stage, the
  // first B of them x's; the lane's 16 bytes go to slot lane % 8.  Waves 0 and 1
  // load x, waves 2 and 3 W.  Rows past M or N lie past the end.
  const bool is_x = wave < 2;
  const int lr = 8 * (LOADS * (wave & 1)) + (lane >> 3);               // row of load 0 within its operand
  const uint32_t row0 = (uint32_t)((is_x ? m0 : n0) + lr) * rowb;
  const uint32_t piece[2] = {16u * (uint32_t)((lane & 7) ^ ((lr >> 1) & 7)), 16u * (uint32_t)((lane & 7) ^ (((lr + 8) >> 1) & 7))};
  // scale bytes of tile kt: whole dwords straight into the table, or bytes
  // through registers that store_scales puts there
  uint32_t sv[SR][2];
  const int sr0 = (wave * SL * 64 + lane) >> 1, sd = lane & 1;         // row and dword of scale load 0
  auto issue_scales = [&](int kt, uint8_t* table) __attribute__((always_inline)) {
    const uint32_t sat = (uint32_t)(kt0 + kt) * 8u;
    if constexpr (ALIGNED) {
#pragma unroll
      for (int i = 0; i < SL; ++i) {
        const uint32_t r = (uint32_t)((is_x ? m0 : n0 - B) + sr0 + 32 * i);
        const bool ok = sat + 4u * sd < blocks;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            is_x ? xsr : wsr, (__attribute__((address_space(3))) void*)(table + (wave * SL + i) * 256), 4,
            (int)(ok ? r * blocks + sat + 4u * sd : kPast), 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < SR; ++i) {
        const int r = tid + 256 * i;               // row of the table
        const bool x = r < B;                      // whole waves are on one side
        const uint32_t base = (uint32_t)(x ? m0 + r : n0 + r - B) * blocks + sat;
        auto get = [&](__amdgpu_buffer_rsrc_t rs) __attribute__((always_inline)) {
#pragma unroll
          for (int d = 0; d < 2; ++d) {
            sv[i][d] = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              sv[i][d] |= load1(rs, sat + 4 * d + k < blocks ? base + 4 * d + k : kPast) << (8 * k);
          }
        };
        if (__builtin_amdgcn_readfirstlane(x)) get(xsr);
        else get(wsr);
      }
    }
  };
  const __amdgpu_buffer_rsrc_t rows = is_x ? xr : wr;
  auto issue_rows = [&](int kt, uint8_t* stage, int i) __attribute__((always_inline)) {
    const uint32_t k = (uint32_t)(kt0 + kt) * 128u + piece[i & 1];
    dma16(rows, stage + (LOADS * wave + i) * 1024, k < rowb ? row0 + (uint32_t)(8 * i) * rowb + k : kPast);
  };
  auto store_scales = [&](uint8_t* table) __attribute__((always_inline)) {
    if constexpr (!ALIGNED) {
#pragma unroll
      for (int i = 0; i < SR; ++i)
        *reinterpret_cast<u32x2_t*>(table + (tid + 256 * i) * 8) = u32x2_t{sv[i][0], sv[i][1]};
    }
  };

  floatx16_t acc[W][W];
#pragma unroll
  for (int i = 0; i < W; ++i)
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  const int wm = 32 * W * (wave & 1), wn = 32 * W * (wave >> 1);
  const int swz = (c >> 1) & 7;                    // rows 32 i + c: the same for every i
  // the stage's k tile, and between its matrix instructions the loads of tile
  // `next`, one after each row of them: all at once they would hold the wave
  // until the address unit has taken them (2048 x 28672 x 8192: 335 -> 318 us; without any
  // loads in the loop it takes 250)
  auto compute = [&](const uint8_t* stage, const uint8_t* table, int next, uint8_t* far) __attribute__((always_inline)) {
    const uint8_t* xrow = stage + (wm + c) * 128;
    const uint8_t* wrow = stage + (B + wn + c) * 128;
    uint32_t xsc[W], wsc[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      xsc[i] = *reinterpret_cast<const uint32_t*>(table + (wm + 32 * i + c) * 8 + 4 * h);
      wsc[i] = *reinterpret_cast<const uint32_t*>(table + (B + wn + 32 * i + c) * 8 + 4 * h);
    }
    u32x4_t xv[2][W], wv[2][W];
    auto read = [&](int s) __attribute__((always_inline)) {
      const int slot = ((4 * h + s) ^ swz) * 16;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        xv[s & 1][i] = *reinterpret_cast<const u32x4_t*>(xrow + 32 * 128 * i + slot);
        wv[s & 1][i] = *reinterpret_cast<const u32x4_t*>(wrow + 32 * 128 * i + slot);
      }
    };
    read(0);
    auto step = [&](auto sc) __attribute__((always_inline)) {
      constexpr int s = decltype(sc)::value;
      if constexpr (s < 3) read(s + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < W; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) acc[i][j] = mfma32_mx<s, s>(xv[s & 1][i], wv[s & 1][j], acc[i][j], xsc[i], wsc[j]);
        __builtin_amdgcn_sched_barrier(0);
        issue_rows(next, far, W * s + i);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    step(std::integral_constant<int, 0>());
    step(std::integral_constant<int, 1>());
    step(std::integral_constant<int, 2>());
    step(std::integral_constant<int, 3>());
  };
  static_assert(LOADS == 4 * W, "one load after each row of matrix instructions");
  auto stage_of = [&](int kt) __attribute__((always_inline)) { return lds + (kt & (S - 1)) * STAGE; };
  auto table_of = [&](int kt) __attribute__((always_inline)) { return lds + S * STAGE + (kt & (S - 1)) * TABLE; };
#pragma unroll
  for (int kt = 0; kt < S - 1; ++kt) {
    issue_scales(kt, table_of(kt));
#pragma unroll
    for (int i = 0; i < LOADS; ++i) issue_rows(kt, stage_of(kt), i);
  }
  store_scales(table_of(0));
  // tiles after the last: past K zeros; past a split read and not used
  constexpr int NEWER = (S - 2) * (LOADS + SL);    // loads of the tiles after this one
  for (int kt = 0; kt < ktiles; ++kt) {
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt((NEWER & 0xF) | ((NEWER >> 4) << 14) | 0x70);   // vmcnt(NEWER), lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    issue_scales(kt + S - 1, table_of(kt + S - 1));
    compute(stage_of(kt), table_of(kt), kt + S - 1, stage_of(kt + S - 1));
    store_scales(table_of(kt + 1));
  }

  // ---- results
  auto each = [&](auto store) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int m = m0 + wm + 32 * i + 8 * (v >> 2) + 4 * h + (v & 3);
        if (m < a.M) {
#pragma unroll
          for (int j = 0; j < W; ++j) {
            const int n = n0 + wn + 32 * j + c;
            if (n < a.N) store((int64_t)m * a.N + n, acc[i][j][v]);
          }
        }
      }
  };
  if (a.splits > 1 || a.out_type == kTypeF32) {
    float* out = a.splits > 1 ? a.ws + (int64_t)sk * a.M * a.N : static_cast<float*>(a.out);
    each([&](int64_t o, float v) __attribute__((always_inline)) { out[o] = v; });
  } else if (a.out_type == kTypeBf16) {
    uint16_t* out = static_cast<uint16_t*>(a.out);
    each([&](int64_t o, float v) __attribute__((always_inline)) { out[o] = (uint16_t)bf16_pair(v, v); });
  } else {
    _Float16* out = static_cast<_Float16*>(a.out);
    each([&](int64_t o, float v) __attribute__((always_inline)) { out[o] = (_Float16)v; });
  }
}

// The splits' fp32 sums added in split order, rounded once.
__global__ __launch_bounds__(256) void mx_split_sum_kernel(MxGemmArgs a) {
  const int64_t total = (int64_t)a.M * a.N;
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= total) return;
  if ((total & 3) == 0 && a.quad_stores) {
    floatx4_t s = *reinterpret_cast<const floatx4_t*>(a.ws + i);
    for (int k = 1; k < a.splits; ++k) s += *reinterpret_cast<const floatx4_t*>(a.ws + k * total + i);
    if (a.out_type == kTypeF32) {
      *reinterpret_cast<floatx4_t*>(static_cast<float*>(a.out) + i) = s;
    } else {
      const u32x2_t o = a.out_type == kTypeBf16
                            ? u32x2_t{bf16_pair(s[0], s[1]), bf16_pair(s[2], s[3])}
                            : u32x2_t{as_u32(half2_t{(_Float16)s[0], (_Float16)s[1]}),
                                      as_u32(half2_t{(_Float16)s[2], (_Float16)s[3]})};
      *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(a.out) + i) = o;
    }
  } else {
    for (int64_t e = i; e < i + 4 && e < total; ++e) {
      float s = a.ws[e];
      for (int k = 1; k < a.splits; ++k) s += a.ws[k * total + e];
      store_typed(a.out, e, s, a.out_type);
    }
  }
}

#define MX_KERNEL(...) MxKernel{__VA_ARGS__, "gptq::" #__VA_ARGS__, grid, 256, 0}
MxKernel mx_tile_kernel_of(const MxGemmArgs& a) {
  const int nt = a.tiles_m * a.tiles_n;
  const unsigned grid = (unsigned)(8 * ((nt + 7) / 8) * a.splits);
  if (a.x_type != kTypeMxfp4) {
    if (a.x_type == kTypeBf16) return a.tile_m == 128 ? MX_KERNEL(mx_tile_kernel<true, 128>) : MX_KERNEL(mx_tile_kernel<true, 64>);
    return a.tile_m == 128 ? MX_KERNEL(mx_tile_kernel<false, 128>) : MX_KERNEL(mx_tile_kernel<false, 64>);
  }
  const bool aligned = (a.K / 32) % 4 == 0 && (reinterpret_cast<uintptr_t>(a.scales) & 3) == 0 &&
                       (reinterpret_cast<uintptr_t>(a.x_scales) & 3) == 0;
  auto staged = [](MxKernel k, int rows, int stages) {
    k.lds = (size_t)stages * rows * (128 + 8);
    return k;
  };
  if (a.tile_m == 256)
    return staged(aligned ? MX_KERNEL(mx4_tile_kernel<4, 2, true>) : MX_KERNEL(mx4_tile_kernel<4, 2, false>), 512, 2);
  if (!aligned) return staged(MX_KERNEL(mx4_tile_kernel<2, 2, false>), 256, 2);
  if (nt * a.splits <= 256) return staged(MX_KERNEL(mx4_tile_kernel<2, 4, true>), 256, 4);
  return staged(MX_KERNEL(mx4_tile_kernel<2, 2, true>), 256, 2);
}
#undef MX_KERNEL

hipError_t launch_mx_tile(const MxGemmArgs& a, hipStream_t stream) {
  hipError_t err = launch_mx_kernel(mx_tile_kernel_of(a), a, stream);
  if (err == hipSuccess && a.splits > 1) {
    const int64_t quads = ((int64_t)a.M * a.N + 3) / 4;
    mx_split_sum_kernel<<<(unsigned)((quads + 255) / 256), 256, 0, stream>>>(a);
    err = hipGetLastError();
  }
  return err;
}

}  // namespace gptq
