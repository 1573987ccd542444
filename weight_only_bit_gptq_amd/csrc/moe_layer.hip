// A whole mixture-of-experts layer for a few tokens, in three kernels (four where
// fp16 hidden values are split first, see row_scale):
//   router    a workgroup per token: its logits in fp64, the k best experts
//             and their weights
//   gate_up   per expert and column tile: gate and up columns of the same
//             outputs in one workgroup, so silu(gate) * up needs no exchange
//   down      per column tile, over all reached experts one after the other: an
//             expert's sums are added, times the router's weights, to a table
//             [token][column] in LDS, fp32; with several workgroups along the
//             experts their tables go through memory and the last to arrive adds
//             them.  Rounded once
// A (token, rank) pair p = t * k + j owns a row of h.  Which tokens an expert
// has, each workgroup finds for itself in the T * k choices (at most 1024), so
// the kernels exchange nothing but those arrays.  The products are the
// streaming product of stream_gemm.hpp: bound by the reached experts' weight
// bytes, each read once.
#include <algorithm>
#include <type_traits>

#include "mx_kernels.hpp"
#include "stream_gemm.hpp"

namespace gptq {

constexpr int kMoeMaxSplits = 16;
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 16;
constexpr int kMaxPairs = kMoeTokens * kMaxTopK;

// ---------------------------------------------------------------- router
template <bool BF16> __device__ __forceinline__ double f64_of(uint32_t bits16) {
  if constexpr (BF16) return (double)bf16_to_f32(bits16);
  else return (double)(float)__builtin_bit_cast(_Float16, (uint16_t)bits16);
}
// order of logits: any NaN on top, ties to the lower index
__device__ __forceinline__ bool before(double a, int ia, double b, int ib) {
  const bool na = a != a, nb = b != b;
  if (na || nb) return na && (!nb || ia < ib);
  return a > b || (a == b && ia < ib);
}

// Sixteen waves; a wave takes EG experts at a time over the whole of H, U
// pieces of eight values per lane in flight.  The choice compares near values,
// hence fp64: products of 16-bit values are exact and the sums' rounding
// (2^-53) is far below any difference that the inputs can mean.
template <bool BF16, int EG, int U>
__global__ __launch_bounds__(1024) void moe_router_kernel(MoeArgs a) {
  __shared__ double lg[kMaxExperts];
  __shared__ int rank[kMaxExperts];
  __shared__ double top[kMaxTopK];
  const int tid = threadIdx.x, lane = tid & 63, t = blockIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t rowb = (uint32_t)a.H * 2u;
  const __amdgpu_buffer_rsrc_t xr = buffer_of(static_cast<const char*>(a.x) + (int64_t)t * rowb, rowb);
  for (int e = tid; e < a.E; e += 1024) rank[e] = 0;
  for (int e0 = wave * EG; e0 < a.E; e0 += 16 * EG) {
    const int ne = min(EG, a.E - e0);
    const __amdgpu_buffer_rsrc_t wr =
        buffer_of(static_cast<const char*>(a.w_router) + (int64_t)e0 * rowb, (uint32_t)ne * rowb);
    double s[EG] = {};
    for (uint32_t at = 16u * lane; at < rowb; at += 1024u * U) {
      u32x4_t x[U], w[EG][U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t off = at + 1024u * u;
        x[u] = load16(xr, off);                    // past the row: zero
#pragma unroll
        for (int g = 0; g < EG; ++g) w[g][u] = load16(wr, off < rowb ? g * rowb + off : kPast);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const double x0 = f64_of<BF16>(x[u][i] & 0xFFFFu), x1 = f64_of<BF16>(x[u][i] >> 16);
#pragma unroll
          for (int g = 0; g < EG; ++g) {
            s[g] = fma(f64_of<BF16>(w[g][u][i] & 0xFFFFu), x0, s[g]);
            s[g] = fma(f64_of<BF16>(w[g][u][i] >> 16), x1, s[g]);
          }
        }
    }
    // the lanes' sums: while there are several experts, each half of the lanes
    // keeps half of them
    int g = 0, d = 32;
#pragma unroll
    for (int n = EG; n > 1; n >>= 1, d >>= 1) {
      const bool up = (lane & d) != 0;
#pragma unroll
      for (int i = 0; i < n / 2; ++i) {
        const double give = up ? s[i] : s[i + n / 2], keep = up ? s[i + n / 2] : s[i];
        s[i] = keep + __shfl_xor(give, d);
      }
      g = 2 * g + (up ? 1 : 0);
    }
#pragma unroll
    for (int e = EG == 1 ? 32 : EG == 2 ? 16 : 8; e > 0; e >>= 1) s[0] += __shfl_xor(s[0], e);
    // expert of the lane: its upper lane bits choose halves, so g is in order
    if ((lane & (EG == 1 ? 63 : EG == 2 ? 31 : 15)) == 0 && g < ne) lg[e0 + g] = s[0];
  }
  __syncthreads();
  // rank of an expert: how many come before it, counted by 1024 / E threads
  const int parts = 1024 / a.E;
  if (tid < parts * a.E) {
    const int e = tid % a.E;
    const double v = lg[e];
    int n = 0;
    for (int o = tid / a.E; o < a.E; o += parts) n += before(lg[o], o, v, e) ? 1 : 0;
    atomicAdd(&rank[e], n);
  }
  __syncthreads();
  for (int e = tid; e < a.E; e += 1024) {
    const int r = rank[e];
    if (r < a.k) {
      a.chosen[t * a.k + r] = e;
      top[r] = lg[e];
    }
  }
  __syncthreads();
  if (wave == 0) {
    const double best = top[0];
    const float mine = lane < a.k ? expf((float)(top[lane] - best)) : 0.f;
    float sum = mine;
    if (!a.renorm) {
      sum = 0.f;
      for (int e = lane; e < a.E; e += 64) sum += expf((float)(lg[e] - best));
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
    if (lane < a.k) a.weight[t * a.k + lane] = mine / sum;
  }
}

// ---------------------------------------------------------------- the products
// Column of lane position c (0..15) in tile j of a segment that starts at n0:
// adjacent columns per lane in the checkpoint layout, 16-column tiles else.
template <int FMT, bool TILED, int CS> __device__ __forceinline__ int column_of(int n0, int j, int c) {
  if constexpr (FMT != 0 && !TILED) return n0 + CS * c + j;
  else return n0 + 16 * j + c;
}

// 16-column tiles per segment and 128-row parts per unit.  The checkpoint
// layout keeps a row of N words apart, so its loads take two adjacent columns; a
// unit is about 4 KB of a wave's columns.
constexpr int segment_tiles(int fmt, bool tiled) { return fmt != 0 && !tiled ? 2 : 1; }
constexpr int unit_parts(int fmt, int ct) {
  const int parts = fmt == 0 ? 4 : 4096 / (256 * fmt * ct);
  return parts < 1 ? 1 : parts > 4 ? 4 : parts;
}

template <int FMT, bool TILED, bool BF16, int CS, int CT, bool ONE> struct WeightsOf {
  typedef GptqWeights<FMT, TILED, BF16, CS, CT, unit_parts(FMT, CT), ONE> type;
};
template <bool TILED, bool BF16, int CS, int CT, bool ONE> struct WeightsOf<0, TILED, BF16, CS, CT, ONE> {
  typedef MxWeights<BF16, CT> type;
};
// e wave-uniform; after place_columns
template <int FMT, class W> __device__ __forceinline__ void bind_expert(W* w, const ExpertStack& s, int e, int N, int K) {
  const char* weight = static_cast<const char*>(s.weight) + e * s.weight_stride;
  const char* scales = static_cast<const char*>(s.scales) + e * s.scales_stride;
  if constexpr (FMT == 0) {
    w->bind(reinterpret_cast<const uint8_t*>(weight), reinterpret_cast<const uint8_t*>(scales), N, K);
  } else {
    const char* zeros = reinterpret_cast<const char*>(s.zeros) + e * s.zeros_stride;
    w->bind(reinterpret_cast<const int32_t*>(weight), reinterpret_cast<const int32_t*>(zeros), scales, N, K, s.group_size);
  }
}
// segment g of the wave's columns starts at n0 + g * distance
template <int FMT, bool TILED, int CS, int CT, class W>
__device__ __forceinline__ void place_columns(W* w, const ExpertStack& s, int N, int K, int n0, int distance, int lane) {
  if constexpr (FMT == 0) {
    w->place(K, lane);
#pragma unroll
    for (int j = 0; j < CT; ++j) w->row0[j] = (uint32_t)(n0 + j / CS * distance + 16 * (j % CS));
  } else {
    int col[CT];
#pragma unroll
    for (int j = 0; j < CT; ++j) col[j] = j / CS * distance + column_of<FMT, TILED, CS>(n0, j % CS, lane & 15);
    w->place(N, K, s.group_size, s.zero_offset, col, lane >> 4);
  }
}

// A hidden value enters the down product as two parts, the 16-bit value and the
// 16-bit rest: one part alone would add a rounding as large as the output's own.
// Where the down weights are exact in bf16 (bf16 GPTQ, and MXFP4 whatever x's
// type) the parts are bf16, split here: 16 bits of the value, at fp32's range.
__device__ __forceinline__ void split_store(uint16_t* hi, uint16_t* lo, float v) {
  const uint32_t p = bf16_pair(v, 0.f) & 0xFFFFu;
  const float top = bf16_to_f32(p);
  *hi = (uint16_t)p;
  *lo = (uint16_t)(bf16_pair(__builtin_isinf(top) ? 0.f : v - top, 0.f) & 0xFFFFu);
}
// fp16 GPTQ down weights need fp16 parts, whose range (2^-24 .. 65504) hidden
// values leave on both sides.  So h stays fp32 in memory, beside the largest
// magnitude of each pair's row in every column tile, and is split under the power
// of two that puts a row's largest into 2^14 .. 2^15 (at most 2^60): 22 bits of
// every value, or 2^-39 of the row's largest.  The flush undoes the scale.  (A
// value per tile and not one raised by atomics: one token over 64 experts of 2048
// x 1024, gate_up 9.5 us and 13.5, 64 atomics meeting at an address.)
// Few values (up to kWidePairs rows and kWideValues values) are split by the down
// product in LDS, every column tile anew; more by a kernel of its own first (us for
// the layer, without it and with it: one token, 64 experts of 2048 x 1024, k 8,
// 28.3 and 31.1; 5 tokens, 13 experts of 3840 x 256, k 4, 31.4 and 33.8; 32 tokens,
// 16 experts of 2048 x 1024, k 2, 54.6 and 56.2; 8 tokens, 8 experts of 4096 x 14336,
// k 2, 200 and 189; 64 tokens, 16 experts of 2048 x 2048, k 16, 443 and 279).
constexpr int kWidePairs = 64, kWideValues = 1 << 16;
constexpr int kTopExponent = 14, kMostScale = 60;
__device__ __forceinline__ int row_scale(uint32_t top) {
  return min(kTopExponent + 127 - (int)(top >> 23), kMostScale);
}
// two values under a scale as two parts; the second is at most 8, beside an
// infinity it is NaN, which becomes -64
__device__ __forceinline__ void split_wide(float a, float b, float scale, uint32_t* hi, uint32_t* lo) {
  const half2_t h = {(_Float16)__builtin_fmaf(a, scale, 0.f), (_Float16)__builtin_fmaf(b, scale, 0.f)};
  const half2_t l = {(_Float16)__builtin_fmaf(a, scale, -(float)h[0]), (_Float16)__builtin_fmaf(b, scale, -(float)h[1])};
  *hi = as_u32(h);
  *lo = as_u32(__builtin_elementwise_max(l, half2_t{(_Float16)-64.f, (_Float16)-64.f}));
}
__device__ __forceinline__ float scale_of(int exponent) { return __uint_as_float((uint32_t)(127 + exponent) << 23); }

// Every pair's row split once, eight values a thread; the router's weight takes
// the inverse of the scale.
__global__ __launch_bounds__(256) void moe_split_kernel(MoeArgs a) {
  __shared__ uint32_t top[4];
  const int pairs = a.T * a.k, parts = (a.I + 2047) / 2048;
  const int p = (int)blockIdx.x / parts, i = ((int)blockIdx.x % parts * 256 + (int)threadIdx.x) * 8;
  const float* h = static_cast<const float*>(a.h) + (int64_t)p * a.I + i;
  floatx4_t f[2] = {};
  if (i < a.I) {
    f[0] = *reinterpret_cast<const floatx4_t*>(h);
    f[1] = *reinterpret_cast<const floatx4_t*>(h + 4);
  }
  uint32_t m = 0;
  for (int t = threadIdx.x; t < a.up_tiles; t += 256) m = max(m, a.top[t * pairs + p]);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
  if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = m;
  __syncthreads();
  const int s = row_scale(max(max(top[0], top[1]), max(top[2], top[3])));
  if (i == 0) a.weight[p] = ldexpf(a.weight[p], -s);
  if (i >= a.I) return;
  u32x4_t hi, lo;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    uint32_t x, y;
    split_wide(f[v >> 1][2 * (v & 1)], f[v >> 1][2 * (v & 1) + 1], scale_of(s), &x, &y);
    hi[v] = x;
    lo[v] = y;
  }
  uint16_t* out = a.split_h + (int64_t)p * a.I + i;
  *reinterpret_cast<u32x4_t*>(out) = hi;
  *reinterpret_cast<u32x4_t*>(out + (int64_t)pairs * a.I) = lo;
}

// largest of the 16 lanes of a row of lanes, in each of them
__device__ __forceinline__ uint32_t max16(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));    // lanes 1 0 3 2
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));    // lanes 2 3 0 1
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x141, 0xF, 0xF, true));   // lanes 7 .. 0
  return max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x140, 0xF, 0xF, true));  // lanes 15 .. 0
}

// Rows of fp32 in LDS, row r `kp` k in chunks of 256 (1 KB): loaded as they are,
// then split in place, a chunk by one wave: the parts 0, then the parts 1, 512
// bytes each, 16-byte pieces (eight k) of row r at slot p ^ (r % 16).  (Splitting
// in the operand reads takes every column wave 20 instructions per 32 k: one
// token over 64 experts of 2048 x 1024, 4-bit, down 13.7 us, here 10.7.)
struct WideRows {
  __amdgpu_buffer_rsrc_t rsrc;
  int rows, K, kp;                   // kp a power of two, 256 at least

  // k [k0, k0 + kp) of every row into lds; lane r of `off` holds row r's byte
  // offset; k >= min(K, end) reads zero
  __device__ __forceinline__ void issue(int k0, int end, uint8_t* lds, uint32_t off, int wave, int nw, int lane) const {
    const int stop = min(K, end), lg = __builtin_ctz(kp) - 8;
    for (int i = wave; i < rows << lg; i += nw) {
      const uint32_t base = (uint32_t)__builtin_amdgcn_readlane((int)off, i >> lg);
      const int k = k0 + 256 * (i & ((1 << lg) - 1)) + 4 * lane;
      dma16(rsrc, lds + 1024 * i, k < stop ? base + 4u * (uint32_t)k : kPast);
    }
  }
  // lane r of `e` holds the exponent of row r's scale; four chunks' reads at once
  __device__ __forceinline__ void split(uint8_t* lds, int e, int wave, int nw, int lane) const {
    constexpr int U = 4;
    const int lg = __builtin_ctz(kp) - 8, chunks = rows << lg;
    const int to = 16 * (lane >> 1) + 8 * (lane & 1);
    for (int i0 = wave; i0 < chunks; i0 += U * nw) {
      floatx4_t f[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u * nw < chunks) f[u] = *reinterpret_cast<const floatx4_t*>(lds + 1024 * (i0 + u * nw) + 16 * lane);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * nw, r = i >> lg;
        if (i >= chunks) break;
        const float scale = scale_of(__builtin_amdgcn_readlane(e, r));
        u32x2_t hi, lo;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          uint32_t x, y;
          split_wide(f[u][2 * v], f[u][2 * v + 1], scale, &x, &y);
          hi[v] = x;
          lo[v] = y;
        }
        uint8_t* at = lds + 1024 * i + (to ^ (16 * (r & 15)));
        *reinterpret_cast<u32x2_t*>(at) = hi;
        *reinterpret_cast<u32x2_t*>(at + 512) = lo;
      }
    }
  }
};

// Operand reads of one unit from split rows (one row tile; an absent row reads
// row 0).  `row`: the unit's first piece, a multiple of 16 within the row.
template <class W> struct WideOperand {
  const uint8_t* lds;
  const W& w;
  uint32_t row, swz;
  __device__ __forceinline__ half8_t operator()(int, int pl, int s) const {
    const uint32_t p = w.piece(s);
    return *reinterpret_cast<const half8_t*>(lds + row + 1024u * (p >> 5) + 256u * (p >> 4 & 1u) + 512u * (uint32_t)pl +
                                             16u * ((p & 15u) ^ swz));
  }
};

// Rows of one expert beyond a row block's are taken by further workgroups.  Workgroup
// (slot, row block, tile): with no fewer pairs than experts a slot is an
// expert; else it is a pair and stands for the pair's expert, unless an earlier
// pair has the same one.
template <int FMT, bool TILED, bool BF16, bool HBF16, int MT, int CS, bool ONE>
__global__ __launch_bounds__(512, 2) void moe_gate_up_kernel(MoeArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ int pair_of[16 * MT];
  __shared__ uint32_t off[16 * MT];
  __shared__ uint32_t top[16 * MT];                // bits of the rows' largest |h| (fp32 h)
  constexpr int CT = 2 * CS;
  typedef typename WeightsOf<FMT, TILED, BF16, CS, CT, ONE>::type W;
  const MoeShape& g = a.up_shape;
  const int B = g.block_rows;                      // at most 16 MT
  const int cols = 16 * CS * g.nwc, tiles = (a.I + cols - 1) / cols, pairs = a.T * a.k;
  const int lane = threadIdx.x & 63, nw = g.nwc * g.nwk;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cw = wave % g.nwc, kw = wave / g.nwc;
  const int tile = (int)blockIdx.x % tiles, sb = (int)blockIdx.x / tiles;
  const int slot = sb / a.row_blocks, rb = sb % a.row_blocks;
  const int n0 = tile * cols + 16 * CS * cw;
  const bool by_pair = pairs < a.E;
  const int e = by_pair ? __builtin_amdgcn_readfirstlane(a.chosen[slot]) : slot;
  W w;
  place_columns<FMT, TILED, CS, CT>(&w, a.gate_up, 2 * a.I, a.H, n0, a.I, lane);
  bind_expert<FMT, W>(&w, a.gate_up, e, 2 * a.I, a.H);
  const int units = (a.H + W::KU - 1) / W::KU, phases = (units + g.nwk - 1) / g.nwk;
  const bool mine = n0 < a.I;                      // a wave past the last column loads nothing
  const uint32_t wbytes = nw * W::BYTES;
  const uint32_t phase = wbytes + (uint32_t)B * g.nwk * W::KU * 2u;
  auto weights = [&](int p) __attribute__((always_inline)) { return lds + (p & 1) * phase + wave * W::BYTES; };
  auto rows_at = [&](int p) __attribute__((always_inline)) { return lds + (p & 1) * phase + wbytes; };
  typename W::Regs r0, r1;
  // experts by slot: the weights do not wait for the rows
  const bool early = !by_pair || a.T == 1;
  if (early) w.load(kw, mine && kw < units, weights(0), &r0);
  // the expert's pairs, in order (at most one per token)
  int count = 0;
  if (by_pair && a.T == 1) {
    count = 1;
    if (threadIdx.x == 0) {
      pair_of[0] = slot;
      off[0] = 0;
    }
  } else {
    constexpr int U = 4;
    for (int i0 = 0; i0 < pairs; i0 += 64 * U) {
      int c[U];
#pragma unroll
      for (int u = 0; u < U; ++u) c[u] = i0 + 64 * u + lane < pairs ? a.chosen[i0 + 64 * u + lane] : -1;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint64_t m = __ballot(c[u] == e);
        const int p = i0 + 64 * u + lane;
        if (by_pair && count == 0 && m != 0 && i0 + 64 * u + __builtin_ctzll(m) != slot) return;
        const int at = count + __builtin_popcountll(m & ((1ull << lane) - 1)) - rb * B;
        if (wave == 0 && c[u] == e && at >= 0 && at < B) {
          pair_of[at] = p;
          off[at] = (uint32_t)(p / a.k) * (uint32_t)a.H * 2u;
        }
        count += __builtin_popcountll(m);
      }
    }
  }
  const int rows = min(B, count - rb * B);
  if (rows <= 0) return;
  if (!early) w.load(kw, mine && kw < units, weights(0), &r0);
  if (!HBF16 && threadIdx.x < 16 * MT) top[threadIdx.x] = 0;
  __syncthreads();
  const int nmt = (rows + 15) >> 4;
  StagedRows x;
  x.rsrc = buffer_of(a.x, (uint32_t)a.T * (uint32_t)a.H * 2u);
  x.off = off;
  x.plane = 0;
  x.rows = rows;
  x.K = a.H;
  x.kp = g.nwk * W::KU;
  x.template issue<1>(0, a.H, rows_at(0), wave, nw, lane);
  floatx4_t acc[MT][CT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int j = 0; j < CT; ++j) acc[mt][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};
  UnitOperand<W, MT> operand{nullptr, w, {}, (uint32_t)((lane & 15) < rows ? lane & 15 : 0), 0, kw * (W::KU / 8)};
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int m = 16 * mt + (lane & 15);
    operand.row[mt] = (uint32_t)(m < rows ? m : (int)operand.swz) * x.kp * 2u;
  }
  auto issue = [&](int p, typename W::Regs* r) __attribute__((always_inline)) {
    const int unit = p * g.nwk + kw;
    w.load(unit, mine && unit < units, weights(p), r);
    x.template issue<1>(p * x.kp, a.H, rows_at(p), wave, nw, lane);
  };
  auto compute = [&](int p, const typename W::Regs& r) __attribute__((always_inline)) {
    const int unit = p * g.nwk + kw;
    operand.lds = rows_at(p);
    if (mine && unit < units) w.template multiply<MT, 1>(weights(p), r, unit, operand, nmt, acc);
  };
  for (int p = 0; p < phases; p += 2) {
    phase_ready();
    if (p + 1 < phases) issue(p + 1, &r1);
    compute(p, r0);
    if (p + 1 >= phases) break;
    phase_ready();
    if (p + 2 < phases) issue(p + 2, &r0);
    compute(p + 1, r1);
  }
  // the k waves' sums, then silu(gate) * up
  floatx4_t* red = reinterpret_cast<floatx4_t*>(lds);
  if (g.nwk > 1) {
    __syncthreads();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (mt >= nmt) break;
#pragma unroll
      for (int j = 0; j < CT; ++j) red[((kw * g.nwc + cw) * MT * CT + mt * CT + j) * 64 + lane] = acc[mt][j];
    }
    __syncthreads();
  }
  uint16_t* hi = static_cast<uint16_t*>(a.h);
  uint16_t* lo = hi + (int64_t)pairs * a.I;
  if (mine) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (mt >= nmt) break;
#pragma unroll
      for (int j = 0; j < CS; ++j) {
        if ((mt * CS + j) % g.nwk != kw) continue;
        floatx4_t gate = acc[mt][j], up = acc[mt][CS + j];
        if (g.nwk > 1) {
          gate = up = floatx4_t{0.f, 0.f, 0.f, 0.f};
          for (int k = 0; k < g.nwk; ++k) {
            gate += red[((k * g.nwc + cw) * MT * CT + mt * CT + j) * 64 + lane];
            up += red[((k * g.nwc + cw) * MT * CT + mt * CT + CS + j) * 64 + lane];
          }
        }
        const int m = 16 * mt + 4 * (lane >> 4), n = column_of<FMT, TILED, CS>(n0, j, lane & 15);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (m + i < rows) {
            const int64_t o = (int64_t)pair_of[m + i] * a.I + n;
            const float v = gate[i] / (1.f + expf(-gate[i])) * up[i];
            if constexpr (HBF16) {
              split_store(hi + o, lo + o, v);
            } else {
              static_cast<float*>(a.h)[o] = v;
              const uint32_t most = max16(__float_as_uint(v) & 0x7FFFFFFFu);
              if ((lane & 15) == 0) atomicMax(&top[m + i], most);
            }
          }
        }
      }
    }
  }
  if constexpr (!HBF16) {
    __syncthreads();
    if ((int)threadIdx.x < rows) a.top[tile * pairs + pair_of[threadIdx.x]] = top[threadIdx.x];
  }
}

// Workgroup (split, tile): phases (expert, row block, part of I) in expert
// order, a consecutive share of all units per workgroup.  A wave's sums of one
// expert's rows are added, times the router's weights, to its LDS table
// [token][column] before the next.
// WIDE: h is fp32 and split here.
template <int FMT, bool TILED, bool BF16, int CS, bool ONE, bool WIDE>
__global__ __launch_bounds__(512, 2) void moe_down_kernel(MoeArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ int count[kMaxExperts];               // pairs of an expert, then its first sorted pair
  __shared__ int16_t reached[kMaxExperts];         // the experts reached, ascending
  __shared__ int16_t first[kMaxExperts + 1];       // first sorted pair of each of them
  __shared__ int16_t sorted[kMaxPairs], place[kMaxPairs];
  __shared__ int flag;
  static_assert(kMaxPairs <= kMaxExperts, "factor in count's place");
  static_assert(kWidePairs <= 64, "WIDE: the pairs are few");
  float* factor = reinterpret_cast<float*>(count); // once sorted: what a pair's sums are multiplied by,
  int16_t* scale = place;                          // and the exponent of its row's scale (WIDE)
  constexpr int MT = 1;
  typedef typename WeightsOf<FMT, TILED, BF16, CS, CS, ONE>::type W;
  const MoeShape& g = a.down_shape;
  const int B = g.block_rows;                      // at most 16
  const int cols = 16 * CS * g.nwc, tiles = (a.H + cols - 1) / cols, pairs = a.T * a.k;
  const int split = (int)blockIdx.x / tiles, tile = (int)blockIdx.x % tiles;
  const int tid = threadIdx.x, lane = tid & 63, nw = g.nwc * g.nwk;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int cw = wave % g.nwc, kw = wave / g.nwc;
  const int n0 = tile * cols + 16 * CS * cw;
  const bool mine = n0 < a.H;
  // used once the pairs are sorted, loaded beside what the sort waits for
  const int tops = WIDE ? pairs * a.up_tiles : 0;
  const uint32_t first_top = tid < tops ? a.top[tid] : 0u;
  const float first_weight = tid < pairs ? a.weight[tid] : 0.f;

  // pairs sorted by expert (within one in any order: rows do not mix)
  if (pairs <= 64) {
    // few: every lane counts what comes before its pair
    if (wave == 0) {
      count[lane] = 0;
      const int e = lane < pairs ? a.chosen[lane] : kMaxExperts;
      int before_pair = 0, before_expert = 0;
      bool again = false;
      for (int o = 0; o < pairs; ++o) {
        const int eo = __builtin_amdgcn_readlane(e, o);
        before_pair += eo < e || (eo == e && o < lane) ? 1 : 0;
        again |= eo == e && o < lane;
      }
      const uint64_t leaders = __ballot(lane < pairs && !again);
      for (int o = 0; o < pairs; ++o)
        if ((leaders >> o & 1) != 0 && __builtin_amdgcn_readlane(e, o) < e) ++before_expert;
      if (lane < pairs) {
        sorted[before_pair] = (int16_t)lane;
        if (!again) {
          reached[before_expert] = (int16_t)e;
          first[before_expert] = (int16_t)before_pair;
        }
      }
      if (lane == 0) {
        flag = __builtin_popcountll(leaders);
        first[flag] = (int16_t)pairs;
      }
    }
    __syncthreads();
  } else {
    for (int e = tid; e < a.E; e += blockDim.x) count[e] = 0;
    __syncthreads();
    for (int p = tid; p < pairs; p += blockDim.x) place[p] = (int16_t)atomicAdd(&count[a.chosen[p]], 1);
    __syncthreads();
    if (wave == 0) {
      int n = 0, sum = 0;
      for (int e0 = 0; e0 < a.E; e0 += 64) {
        const int c = e0 + lane < a.E ? count[e0 + lane] : 0;
        const uint64_t m = __ballot(c > 0);
        int s = c;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
          const int o = __shfl_up(s, d);
          if (lane >= d) s += o;
        }
        if (c > 0) {
          const int at = n + __builtin_popcountll(m & ((1ull << lane) - 1));
          reached[at] = (int16_t)(e0 + lane);
          first[at] = (int16_t)(sum + s - c);
        }
        if (e0 + lane < a.E) count[e0 + lane] = sum + s - c;
        n += __builtin_popcountll(m);
        sum += __shfl(s, 63);
      }
      if (lane == 0) {
        flag = n;
        first[n] = (int16_t)pairs;
      }
    }
    __syncthreads();
    for (int p = tid; p < pairs; p += blockDim.x) sorted[count[a.chosen[p]] + place[p]] = (int16_t)p;
    __syncthreads();                               // count and place are free
  }
  if (WIDE) {
    auto raise = [&](int i, uint32_t top) __attribute__((always_inline)) { atomicMax(&count[i % pairs], (int)top); };
    if (tid < tops) raise(tid, first_top);
    for (int i = tid + blockDim.x; i < tops; i += blockDim.x) raise(i, a.top[i]);
    __syncthreads();
  }
  for (int p = tid; p < pairs; p += blockDim.x) {
    const float c = p == tid ? first_weight : a.weight[p];
    const int s = WIDE ? row_scale((uint32_t)count[p]) : 0;
    factor[p] = WIDE ? ldexpf(c, -s) : c;
    scale[p] = (int16_t)s;
  }
  const int experts = __builtin_amdgcn_readfirstlane(flag);

  W w;
  place_columns<FMT, TILED, CS, CS>(&w, a.down, a.H, a.I, n0, 0, lane);
  const int units = (a.I + W::KU - 1) / W::KU, kp = g.nwk * W::KU;
  const uint32_t wbytes = nw * W::BYTES, phase = wbytes + (uint32_t)B * kp * 4u;
  const uint32_t tokens = (uint32_t)a.T * cols * 4u;
  float* table = reinterpret_cast<float*>(lds + 2 * phase + kw * tokens);
  for (int i = tid; i < g.nwk * a.T * cols; i += blockDim.x) reinterpret_cast<float*>(lds + 2 * phase)[i] = 0.f;
  uint32_t* off = reinterpret_cast<uint32_t*>(lds + 2 * phase + g.nwk * tokens);    // [2][B]
  int exponents[2] = {0, 0};                       // lane r: of row r's scale, per buffer (WIDE)
  auto weights = [&](int b) __attribute__((always_inline)) { return lds + b * phase + wave * W::BYTES; };
  auto rows_at = [&](int b) __attribute__((always_inline)) { return lds + b * phase + wbytes; };
  const uint32_t plane = (uint32_t)pairs * (uint32_t)a.I * 2u;
  typename std::conditional<WIDE, WideRows, StagedRows>::type x;
  x.rsrc = buffer_of(BF16 || WIDE ? a.h : a.split_h, 2u * plane);
  if constexpr (!WIDE) x.plane = plane;
  x.K = a.I;
  x.kp = kp;
  floatx4_t acc[MT][CS];
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int j = 0; j < CS; ++j) acc[mt][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};
  };
  clear();
  __syncthreads();

  // this workgroup's units [f0, f1) of all experts' units in a row
  const int total = experts * units;
  const int f0 = (int)((int64_t)total * split / a.splits), f1 = (int)((int64_t)total * (split + 1) / a.splits);
  struct Phase {
    int slot, rb, unit;              // first unit of the phase within the expert
    int end;                         // the workgroup's last unit of the expert
    int base, rows;                  // sorted pairs of the row block
  };
  auto at_slot = [&](Phase* p) __attribute__((always_inline)) {
    p->unit = max(f0 - p->slot * units, 0);
    p->end = min(f1 - p->slot * units, units);
  };
  auto at_block = [&](Phase* p) __attribute__((always_inline)) {
    p->base = __builtin_amdgcn_readfirstlane(first[p->slot]) + p->rb * B;
    p->rows = min(B, __builtin_amdgcn_readfirstlane(first[p->slot + 1]) - p->base);
  };
  // the next phase; false after the last
  auto advance = [&](Phase* p) __attribute__((always_inline)) {
    p->unit += g.nwk;
    if (p->unit < p->end) return true;
    ++p->rb;
    if (p->base + B >= __builtin_amdgcn_readfirstlane(first[p->slot + 1])) {
      p->rb = 0;
      ++p->slot;
      if (p->slot * units >= f1) return false;
    }
    at_slot(p);
    at_block(p);
    return true;
  };
  auto issue = [&](const Phase& p, int b, typename W::Regs* r) __attribute__((always_inline)) {
    bind_expert<FMT, W>(&w, a.down, __builtin_amdgcn_readfirstlane(reached[p.slot]), a.H, a.I);
    w.load(p.unit + kw, mine && p.unit + kw < p.end, weights(b), r);
    if constexpr (WIDE) {
      const int q = lane < p.rows ? sorted[p.base + lane] : 0;
      exponents[b] = scale[q];
      x.rows = p.rows;
      x.issue(p.unit * W::KU, p.end * W::KU, rows_at(b), (uint32_t)q * (uint32_t)a.I * 4u, wave, nw, lane);
    } else {
      // every wave writes the same offsets (its own lanes read them back)
      if (lane < p.rows) off[b * B + lane] = (uint32_t)sorted[p.base + lane] * (uint32_t)a.I * 2u;
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      x.off = off + b * B;
      x.rows = p.rows;
      x.template issue<2>(p.unit * W::KU, p.end * W::KU, rows_at(b), wave, nw, lane);
    }
  };
  auto compute = [&](const Phase& p, int b, const typename W::Regs& r) __attribute__((always_inline)) {
    if (!mine || p.unit + kw >= p.end) return;
    const uint32_t swz = (uint32_t)((lane & 15) < p.rows ? lane & 15 : 0);
    if constexpr (WIDE) {
      const uint32_t first = (uint32_t)kw * (W::KU / 8);
      const WideOperand<W> operand{rows_at(b), w, swz * kp * 4u + 1024u * (first >> 5) + 256u * (first >> 4 & 1u), swz};
      w.template multiply<MT, 2>(weights(b), r, p.unit + kw, operand, 1, acc);
    } else {
      UnitOperand<W, MT> operand{rows_at(b), w, {swz * kp * 2u}, swz, (uint32_t)(p.rows * kp * 2), kw * (W::KU / 8)};
      w.template multiply<MT, 2>(weights(b), r, p.unit + kw, operand, 1, acc);
    }
  };
  // the rows of phase p are complete: add them to their tokens
  auto flush = [&](const Phase& p) __attribute__((always_inline)) {
    if (mine) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = 4 * (lane >> 4) + i;
        if (m < p.rows) {
          const int q = sorted[p.base + m];
          const float f = factor[q];
          float* t = table + (q / a.k) * cols + 16 * CS * cw;
#pragma unroll
          for (int j = 0; j < CS; ++j) t[column_of<FMT, TILED, CS>(0, j, lane & 15)] += acc[0][j][i] * f;
        }
      }
    }
    clear();
  };
  if (f0 < f1) {
    Phase cur{f0 / units, 0, 0, 0, 0, 0};
    at_slot(&cur);
    at_block(&cur);
    typename W::Regs r0, r1;
    issue(cur, 0, &r0);
    auto step = [&](int b, const typename W::Regs& now, typename W::Regs* then) __attribute__((always_inline)) {
      Phase next = cur;
      const bool more = advance(&next);
      phase_ready();
      if (more) issue(next, b ^ 1, then);
      if constexpr (WIDE) {                        // the next phase's loads are under way
        x.rows = cur.rows;
        x.split(rows_at(b), exponents[b], wave, nw, lane);
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        __builtin_amdgcn_s_waitcnt(0xC07F);        // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
      }
      compute(cur, b, now);
      if (!more || next.slot != cur.slot || next.rb != cur.rb) flush(cur);
      cur = next;
      return more;
    };
    while (true) {
      if (!step(0, r0, &r1)) break;
      if (!step(1, r1, &r0)) break;
    }
  }
  __syncthreads();
  const float* all = reinterpret_cast<const float*>(lds + 2 * phase);
  for (int i = tid; i < a.T * cols; i += blockDim.x) {
    const int n = tile * cols + i % cols;
    if (n >= a.H) continue;
    float s = all[i];
    for (int k = 1; k < g.nwk; ++k) s += all[k * a.T * cols + i];
    const int64_t o = (int64_t)(i / cols) * a.H + n;
    if (a.splits > 1) put_agent(a.part + (int64_t)split * a.T * a.H + o, s);
    else store_typed(a.out, o, s, a.bf16 ? kTypeBf16 : kTypeF16);
  }
  if (a.splits == 1 || !last_arrival(a.cnt + tile, (uint32_t)a.splits, &flag)) return;
  for (int i = tid; i < a.T * cols; i += blockDim.x) {
    const int n = tile * cols + i % cols;
    if (n >= a.H) continue;
    const int64_t o = (int64_t)(i / cols) * a.H + n;
    store_typed(a.out, o, sum_splits<kMoeMaxSplits>(a.part + o, (int64_t)a.T * a.H, a.splits),
                a.bf16 ? kTypeBf16 : kTypeF16);
  }
}

// ---------------------------------------------------------------- host
namespace {

constexpr int kMoeCUs = 256;
constexpr size_t kMoeLds = 144 * 1024;             // beside up to 13 KB of static LDS

int unit_of(const ExpertStack& s, int segments) {
  const int cs = segment_tiles(s.bits, s.tiled != 0);
  return 128 * unit_parts(s.bits, cs * segments);
}
// LDS of two phases (and the down product's token tables and row offsets)
size_t phase_lds(const ExpertStack& s, int segments, int planes, int rows, const MoeShape& g) {
  const size_t w = s.bits == 0 ? (size_t)4096 * segments * g.nwc * g.nwk : 0;
  return 2 * (w + (size_t)rows * g.nwk * unit_of(s, segments) * 2 * planes);
}
size_t up_lds(const MoeArgs& a) {
  const MoeShape& g = a.up_shape;
  const size_t ct = 2 * (size_t)segment_tiles(a.gate_up.bits, a.gate_up.tiled != 0);
  const size_t sums = g.nwk > 1 ? (size_t)g.nwc * g.nwk * (g.block_rows > 16 ? 2 : 1) * ct * 1024 : 0;
  return std::max(sums, phase_lds(a.gate_up, 2, 1, g.block_rows, g));
}
size_t down_lds(const MoeArgs& a) {
  const MoeShape& g = a.down_shape;
  const size_t cols = 16 * (size_t)segment_tiles(a.down.bits, a.down.tiled != 0) * g.nwc;
  return phase_lds(a.down, 1, 2, g.block_rows, g) + (size_t)g.nwk * a.T * cols * 4 + 2 * (size_t)g.block_rows * 4;
}

}  // namespace

size_t plan_moe(MoeArgs* a, char* base, size_t* counter_bytes) {
  const size_t T = (size_t)a->T, P = T * (size_t)a->k;
  MoeShape& u = a->up_shape;
  MoeShape& d = a->down_shape;
  // Rows per row block: about twice what an expert has on average, so that most
  // experts are one row block, whose weights are read once (more rows repeat the
  // reads, mostly out of a cache), while the rows' share of LDS stays small: it
  // decides how many workgroups a CU holds and so the weight bytes in flight
  // (16 tokens over 8 experts of 4096 x 14336, MXFP4: blocks of 16 rows 203 us, of
  // 8 183).
  const int slots = (int)std::min<size_t>((size_t)a->E, P);
  int block = 8;
  while (block < 32 && (size_t)block * a->E < 2 * P) block *= 2;
  u.block_rows = std::min(a->T, block);
  d.block_rows = std::min(u.block_rows, 16);
  a->row_blocks = (a->T + u.block_rows - 1) / u.block_rows;
  // Column waves share the staged rows, k waves (at least as many as make up
  // x's chunks of 512 k) need fewer column tiles.  Eight waves (four where a
  // wave's registers leave two per SIMD); fewer columns and more k while the
  // workgroups are fewer than the CUs.  Measured (us for the layer): 4 tokens
  // over 32 experts of 2048 x 1024, MXFP4, gate_up c4k2 27, c1k4 35; one token, 64
  // experts, 4-bit tiled c2k4 29.5, c4k2 30.7; 33 tokens, 8-bit checkpoint layout
  // c1k4 166, c2k4 202; 16 tokens, MXFP4, down c4k2 183, c8k1 182, c4k1 203.
  const int ku = unit_of(a->gate_up, 2), kd = unit_of(a->down, 1);
  const int uc = 16 * segment_tiles(a->gate_up.bits, a->gate_up.tiled != 0);
  const int dc = 16 * segment_tiles(a->down.bits, a->down.tiled != 0);
  u.nwk = std::max(1, 512 / ku);
  u.nwc = std::max(1, (uc == 32 ? 4 : 8) / u.nwk);
  while (u.nwc > 1 && slots * ((a->I + uc * u.nwc - 1) / (uc * u.nwc)) < kMoeCUs) {
    u.nwc /= 2;
    if (u.nwk * ku * 2 <= a->H) u.nwk *= 2;
  }
  while (up_lds(*a) > kMoeLds && u.nwk * ku > 512) u.nwk /= 2;
  while (up_lds(*a) > kMoeLds && u.nwc > 1) u.nwc /= 2;
  // (no k wave without a unit of an expert: 5 tokens over 45 experts of 2944 x
  // 512, 2 bits, c4k1 50, c2k4 68)
  d.nwk = a->down.bits ? 4 : 2;
  while (d.nwk * kd > 512 && d.nwk / 2 * kd >= a->I) d.nwk /= 2;
  d.nwc = 8 / d.nwk;
  while (d.nwc > 1 && (a->H + dc * d.nwc - 1) / (dc * d.nwc) * kMoeMaxSplits < kMoeCUs) d.nwc /= 2;
  while (down_lds(*a) > kMoeLds && d.nwk * kd > 512) d.nwk /= 2;
  while (down_lds(*a) > kMoeLds && d.nwc > 1) d.nwc /= 2;
  // splits: one round of the workgroups that fit (at most two per CU)
  const int tiles = (a->H + dc * d.nwc - 1) / (dc * d.nwc);
  const int units = slots * ((a->I + kd - 1) / kd);
  const int fit = down_lds(*a) + 13 * 1024 <= 80 * 1024 ? 2 : 1;
  a->splits = std::max(1, std::min({fit * kMoeCUs / tiles, units / d.nwk, kMoeMaxSplits}));
  *counter_bytes = (size_t)tiles * 4;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* p = base + off;
    off += (bytes + 255) & ~(size_t)255;
    return p;
  };
  a->chosen = reinterpret_cast<int32_t*>(take(P * 4));
  a->weight = reinterpret_cast<float*>(take(P * 4));
  a->up_tiles = (a->I + uc * u.nwc - 1) / (uc * u.nwc);
  a->top = reinterpret_cast<uint32_t*>(take(P * (size_t)a->up_tiles * 4));
  a->h = take(P * (size_t)a->I * 4);
  const bool fp16_parts = !a->bf16 && a->down.bits != 0;
  a->split_first = fp16_parts && (P > (size_t)kWidePairs || P * (size_t)a->I > (size_t)kWideValues);
  a->split_h = reinterpret_cast<uint16_t*>(take(a->split_first ? P * (size_t)a->I * 4 : 0));
  a->part = reinterpret_cast<float*>(take(a->splits > 1 ? (size_t)a->splits * T * (size_t)a->H * 4 : 0));
  return off;
}

template <class Kernel>
hipError_t launch_shaped(Kernel kernel, unsigned grid, const MoeShape& g, int unit, size_t lds, const MoeArgs& a,
                         hipStream_t stream) {
  if (g.nwk * unit % 512 != 0) return hipErrorInvalidValue;   // x is staged in chunks of 512 k
  if (lds > 64 * 1024) {
    const hipError_t err = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (err != hipSuccess) return err;
  }
  kernel<<<grid, 64 * g.nwc * g.nwk, lds, stream>>>(a);
  return hipGetLastError();
}

template <int FMT, bool TILED, bool BF16, bool HBF16, int MT>
hipError_t gate_up_typed(const MoeArgs& a, hipStream_t stream) {
  constexpr int CS = segment_tiles(FMT, TILED);
  const MoeShape& g = a.up_shape;
  const int cols = 16 * CS * g.nwc;
  const unsigned grid = (unsigned)(std::min(a.E, a.T * a.k) * a.row_blocks * ((a.I + cols - 1) / cols));
  const size_t lds = up_lds(a);
  const int unit = unit_of(a.gate_up, 2);
  if (FMT == 0 || a.gate_up.group_size % 128 == 0)
    return launch_shaped(moe_gate_up_kernel<FMT, TILED, BF16, HBF16, MT, CS, true>, grid, g, unit, lds, a, stream);
  if constexpr (FMT != 0)
    return launch_shaped(moe_gate_up_kernel<FMT, TILED, BF16, HBF16, MT, CS, false>, grid, g, unit, lds, a, stream);
  return hipErrorInvalidValue;
}

template <int FMT, bool TILED, bool BF16, bool WIDE> hipError_t down_typed(const MoeArgs& a, hipStream_t stream) {
  constexpr int CS = segment_tiles(FMT, TILED);
  const MoeShape& g = a.down_shape;
  const int cols = 16 * CS * g.nwc;
  const unsigned grid = (unsigned)(a.splits * ((a.H + cols - 1) / cols));
  const size_t lds = down_lds(a);
  const int unit = unit_of(a.down, 1);
  if (FMT == 0 || a.down.group_size % 128 == 0)
    return launch_shaped(moe_down_kernel<FMT, TILED, BF16, CS, true, WIDE>, grid, g, unit, lds, a, stream);
  if constexpr (FMT != 0)
    return launch_shaped(moe_down_kernel<FMT, TILED, BF16, CS, false, WIDE>, grid, g, unit, lds, a, stream);
  return hipErrorInvalidValue;
}

template <int FMT, bool TILED, bool BF16, bool HBF16> hipError_t gate_up_rows(const MoeArgs& a, hipStream_t stream) {
  return a.up_shape.block_rows <= 16
                 ? gate_up_typed<FMT, TILED, BF16, HBF16, 1>(a, stream)
                 : gate_up_typed<FMT, TILED, BF16, HBF16, 2>(a, stream);
}
template <int FMT, bool TILED> hipError_t gate_up_format(const MoeArgs& a, hipStream_t stream) {
  if (a.bf16) return gate_up_rows<FMT, TILED, true, true>(a, stream);
  return a.down.bits == 0 ? gate_up_rows<FMT, TILED, false, true>(a, stream)
                          : gate_up_rows<FMT, TILED, false, false>(a, stream);
}
template <int FMT, bool TILED> hipError_t down_format(const MoeArgs& a, hipStream_t stream) {
  if constexpr (FMT != 0) {
    if (!a.bf16) {
      return a.split_first ? down_typed<FMT, TILED, false, false>(a, stream)
                           : down_typed<FMT, TILED, false, true>(a, stream);
    }
  }
  return down_typed<FMT, TILED, true, false>(a, stream);   // MXFP4: bf16 parts whatever x's type
}

template <bool BF16> hipError_t router_typed(const MoeArgs& a, hipStream_t stream) {
  // experts per wave: all sixteen waves busy first, then fewer passes over x
  if (a.E <= 16) moe_router_kernel<BF16, 1, 8><<<a.T, 1024, 0, stream>>>(a);
  else if (a.E <= 32) moe_router_kernel<BF16, 2, 4><<<a.T, 1024, 0, stream>>>(a);
  else moe_router_kernel<BF16, 4, 2><<<a.T, 1024, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_moe(const MoeArgs& a, hipStream_t stream) {
  hipError_t err = a.bf16 ? router_typed<true>(a, stream) : router_typed<false>(a, stream);
  if (err != hipSuccess) return err;
  const int g = a.gate_up.bits, gt = a.gate_up.tiled;
  if (g == 0) err = gate_up_format<0, false>(a, stream);
  else if (g == 2) err = gt ? gate_up_format<2, true>(a, stream) : gate_up_format<2, false>(a, stream);
  else if (g == 3) err = gt ? gate_up_format<3, true>(a, stream) : gate_up_format<3, false>(a, stream);
  else if (g == 4) err = gt ? gate_up_format<4, true>(a, stream) : gate_up_format<4, false>(a, stream);
  else err = gt ? gate_up_format<8, true>(a, stream) : gate_up_format<8, false>(a, stream);
  if (err != hipSuccess) return err;
  if (a.split_first) {
    moe_split_kernel<<<(unsigned)(a.T * a.k * ((a.I + 2047) / 2048)), 256, 0, stream>>>(a);
    err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  const int d = a.down.bits, dt = a.down.tiled;
  if (d == 0) err = down_format<0, false>(a, stream);
  else if (d == 2) err = dt ? down_format<2, true>(a, stream) : down_format<2, false>(a, stream);
  else if (d == 3) err = dt ? down_format<3, true>(a, stream) : down_format<3, false>(a, stream);
  else if (d == 4) err = dt ? down_format<4, true>(a, stream) : down_format<4, false>(a, stream);
  else err = dt ? down_format<8, true>(a, stream) : down_format<8, false>(a, stream);
  return err;
}

}  // namespace gptq
