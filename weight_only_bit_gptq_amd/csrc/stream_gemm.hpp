// The streaming product of a few rows with quantised weights, shared by the
// MXFP4 GEMM (few rows) and the mixture-of-experts layer.
//
// It is bound by the weights' bytes, each read once, so everything else keeps
// out of their way.  A workgroup's waves are nwc column waves (16 CT columns
// each) times nwk k waves; K advances in phases of nwk units (512 k for MXFP4,
// 128 UPP for the GPTQ formats), one k wave's unit each.  While a phase is
// multiplied the next one's loads are in flight: rows of x and MXFP4 weights
// into LDS (buffer loads with an LDS destination), GPTQ words, whose loads are
// whole 64-byte rows already, into registers.  x goes through LDS although each
// wave reads it once: an operand load from global memory costs the address
// unit as much as a weight load, and there are four to eight of them per
// weight load (measured at 12288 x 4096 MXFP4, everything straight into
// registers: 13 us for one row, 110 us for 64; a read of the weights alone is
// 5.2 us).
//
// Every load is a buffer load: offsets past a tensor read zero without touching
// memory, so k tails, absent units and the phase after the last need no branch
// (a zero activation times any finite weight adds nothing).
//
// Lane l of a wave holds column l % 16 of each 16-column tile and k quarter
// q = l / 16; which k a quarter covers is the weight format's choice, the
// activations follow it.
#pragma once

#include "mx_device.hpp"

namespace gptq {

__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, (int)off, 0, 0, 0);
}

// ---- MXFP4 matrix: codes [N, K/2], scales [N, K/32], T tiles of 16 of its N
// rows.  A unit is 512 k: 16 blocks, 256 contiguous bytes of a row.  The codes
// of a unit go to LDS by four loads per tile, each of four whole 256-byte
// pieces (measured at 28672 x 8192, one row: 64-byte pieces straight into
// operand registers 30 us, 32-byte ones 62 us), block b of row r at slot
// b ^ r, so that reading one block of 16 rows meets 16 different bank groups.
// Quarter q multiplies blocks 4 j + q, j = 0 .. 3.  Scales: where rows of
// scales are whole dwords, one load takes a row's 16 bytes for all quarters and
// each shifts its own out; else every quarter loads its four bytes.
template <int T> struct MxTiles {
  static constexpr int KU = 512, BYTES = 4096 * T;   // LDS of a unit
  struct Regs { uint32_t s[T][4]; };
  __amdgpu_buffer_rsrc_t codes, scales;
  uint32_t row0[T];                  // first row of each tile
  uint32_t rowb, blocks, q, n, shift, rows;
  bool words;

  // the matrix [N, K] at c, s (a wave-uniform pointer pair)
  __device__ __forceinline__ void bind(const uint8_t* c, const uint8_t* s, int N, int K) {
    rows = (uint32_t)N;
    codes = buffer_of(c, (uint32_t)N * (uint32_t)(K / 2));
    scales = buffer_of(s, (uint32_t)N * (uint32_t)(K / 32));
    words = ((K / 32) & 3) == 0 && (reinterpret_cast<uintptr_t>(s) & 3) == 0;
    shift = words ? 8 * q : 0;
  }
  __device__ __forceinline__ void place(int K, int lane) {
    rowb = (uint32_t)K / 2;
    blocks = (uint32_t)K / 32;
    q = lane >> 4;
    n = lane & 15;
  }
  // 1 KB loads i of the unit's 4 T, i = from, from + step, ...: rows past N lie
  // past the end of the buffer
  __device__ __forceinline__ void load_codes(int unit, bool live, uint8_t* lds, int from, int step) const {
#pragma unroll
    for (int i = 0; i < 4 * T; ++i) {
      if (i % step != from) continue;
      const uint32_t r = 4 * (i & 3) + q, b = 16u * (uint32_t)unit + (n ^ r);
      dma16(codes, lds + 1024 * i, live && b < blocks ? (row0[i >> 2] + r) * rowb + 16u * b : kPast);
    }
  }
  __device__ __forceinline__ void load_scales(int unit, bool live, Regs* r) const {
#pragma unroll
    for (int j = 0; j < T; ++j) {
      const uint32_t at = (row0[j] + n) * blocks + 16u * (uint32_t)unit;
      if (words) {
        const u32x4_t v = load16(scales, live ? at : kPast);
#pragma unroll
        for (int i = 0; i < 4; ++i) r->s[j][i] = v[i];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t b = 4 * i + q;
          r->s[j][i] = load1(scales, live && 16u * (uint32_t)unit + b < blocks ? at + b : kPast);
        }
      }
    }
  }
  // scale byte of block 4 j + q of the lane's row: 127 past the row's end,
  // where a word may hold the next row's bytes
  __device__ __forceinline__ uint32_t byte_of(const Regs& r, int t, int j, int unit) const {
    return 16u * (uint32_t)unit + 4 * j + q < blocks ? (r.s[t][j] >> shift) & 0xFFu : 127u;
  }
  // and in rows past N, where it reads as 0: outside fp16's range (16 rows of fp16
  // x, 4095 x 11008, 17.7 us, and 11.9)
  __device__ __forceinline__ uint32_t byte_inside(const Regs& r, int t, int j, int unit) const {
    return row0[t] + n < rows ? byte_of(r, t, j, unit) : 127u;
  }
  // the 16 bytes of block 4 j + q of the lane's row
  __device__ __forceinline__ u32x4_t block(const uint8_t* lds, int t, int j) const {
    return *reinterpret_cast<const u32x4_t*>(lds + 4096 * t + 256 * n + 16 * ((4 * j + q) ^ n));
  }
};

// MXFP4 weights times 16-bit rows.
template <bool BF16, int CT> struct MxWeights : MxTiles<CT> {
  typedef MxTiles<CT> Tiles;
  typedef typename Tiles::Regs Regs;
  static constexpr int KU = 512;
  // index of the 16-byte piece (eight k) of step s = 4 j + v within a unit
  __device__ __forceinline__ uint32_t piece(int s) const { return 16 * (s >> 2) + 4 * this->q + (s & 3); }
  __device__ __forceinline__ void load(int unit, bool live, uint8_t* lds, Regs* r) const {
    // scales first: their two variants share registers, and the wait that the
    // compiler puts between them must find nothing in flight
    this->load_scales(unit, live, r);
    this->load_codes(unit, live, lds, 0, 1);
  }
  // acc += a . unit by the path of scales outside the type's range: the weights in
  // bf16, fp16 activations as two bf16 parts
  template <int MT, int PL, class A>
  __device__ __forceinline__ void multiply_bf16(const uint8_t* lds, const uint32_t (&b)[CT][4], const A& a, int nmt,
                                                floatx4_t (&acc)[MT][CT]) const {
    bool far = false;
#pragma unroll
    for (int t = 0; t < CT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) far = far || mx_far(b[t][j]);
    far = __any(far);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u32x4_t c[CT];
#pragma unroll
      for (int t = 0; t < CT; ++t) c[t] = this->block(lds, t, j);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        half8_t w[CT];
#pragma unroll
        for (int t = 0; t < CT; ++t) w[t] = mx_frag_bf16(far, c[t][v], b[t][j]);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          if (mt >= nmt) break;
#pragma unroll
          for (int pl = 0; pl < PL; ++pl) {
            half8_t hi = a(mt, pl, 4 * j + v), lo;
            if (!BF16) split_f16(hi, &hi, &lo);
#pragma unroll 1
            for (int times = far ? 4 : 1; times > 0; --times)
#pragma unroll
              for (int t = 0; t < CT; ++t) {
                acc[mt][t] = mfma16<true>(hi, w[t], acc[mt][t]);
                if (!BF16) acc[mt][t] = mfma16<true>(lo, w[t], acc[mt][t]);
              }
          }
        }
      }
    }
  }
  // acc += a . unit, a(mt, pl, step) the rows' eight values
  template <int MT, int PL, class A>
  __device__ __forceinline__ void multiply(const uint8_t* lds, const Regs& r, int unit, const A& a, int nmt,
                                           floatx4_t (&acc)[MT][CT]) const {
    uint32_t b[CT][4];
    bool fits = true;
    uint32_t top = 0;
#pragma unroll
    for (int t = 0; t < CT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        b[t][j] = BF16 ? this->byte_of(r, t, j, unit) : this->byte_inside(r, t, j, unit);
        if (BF16) top = max(top, b[t][j]);
        else fits = fits && mx_fits_f16(b[t][j]);
      }
    if (!BF16 && !__all(fits)) {                   // ordinary weights do not come here
      fits = true;
#pragma unroll
      for (int t = 0; t < CT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) fits = fits && (mx_fits_f16(b[t][j]) || mx_zero(this->block(lds, t, j)));
    }
    if (!BF16 && !__all(fits)) return multiply_bf16<MT, PL>(lds, b, a, nmt, acc);
    floatx4_t before[MT][CT];                      // bf16: the sums, should a byte be above 252
    if constexpr (BF16) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int t = 0; t < CT; ++t) before[mt][t] = acc[mt][t];
    }
    // four steps' operands are read at once, the next four while these multiply:
    // an LDS read per step leaves its latency in every step
    constexpr int D = MT * PL <= 2 ? 2 : 1;
    u32x4_t c[D][CT];
    half8_t x[D][4][MT][PL];
    auto read = [&](int j, int d) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < CT; ++t) c[d][t] = this->block(lds, t, j);
#pragma unroll
      for (int v = 0; v < 4; ++v)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          if (mt >= nmt) break;
#pragma unroll
          for (int pl = 0; pl < PL; ++pl) x[d][v][mt][pl] = a(mt, pl, 4 * j + v);
        }
    };
    if constexpr (D == 2) read(0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int d = j % D;
      if constexpr (D == 1) read(j, 0);
      else if (j < 3) read(j + 1, (j + 1) % D);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        half8_t w[CT];
#pragma unroll
        for (int t = 0; t < CT; ++t)
          w[t] = mx_frag<BF16>(c[d][t][v], mx_scale(b[t][j]));
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          if (mt >= nmt) break;
#pragma unroll
          for (int pl = 0; pl < PL; ++pl)
#pragma unroll
            for (int t = 0; t < CT; ++t) acc[mt][t] = mfma16<BF16>(x[d][v][mt][pl], w[t], acc[mt][t]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (BF16) {
      if (__any(top > kMxExact)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int t = 0; t < CT; ++t) acc[mt][t] = before[mt][t];
        __atomic_signal_fence(__ATOMIC_SEQ_CST);   // nothing stays in registers for it
        multiply_bf16<MT, PL>(lds, b, a, nmt, acc);
      }
    }
  }
};

// ---- GPTQ weights of one expert, no act order.  A unit is UPP times four
// 32-row chunks; quarter q holds the 8-row block q of each chunk.  Columns come in segments
// of CS tiles: in the checkpoint layout a lane's CS columns are adjacent (one
// load of CS words), in the tiled layout the tiles are.  ONE: one group per
// four chunks (group_size % 128 == 0); else each may have its own (group_size %
// 32 == 0), and quarter q loads chunk q's scales and zeros for all four (a load
// per chunk and quarter would be more loads than the weights' own: an 8-bit
// layer with groups of 64 spent 185 us with them).
template <int BITS, bool TILED, bool BF16, int CS, int CT, int UPP, bool ONE> struct GptqWeights {
  static constexpr int KU = 128 * UPP, BYTES = 0, L = Block<BITS>::LOADS, SEG = CT / CS;
  static constexpr bool PAIRS = TILED && BITS == 4;
  // scale and zero loads per segment: a lane's adjacent columns share one
  static constexpr int ZC = TILED ? 1 : CS, ZS = CS / ZC;
  static_assert(ZC <= 2, "a scale load holds two columns");
  struct Regs {
    uint32_t w[UPP][4][L][CT];
    uint32_t z[UPP][SEG * ZS][BITS == 3 ? 2 : 1];
    uint32_t s[UPP][SEG * ZS];
  };
  __amdgpu_buffer_rsrc_t qw, qz, sc;
  uint32_t woff[SEG][TILED ? CS : 1];
  int col[CT];
  int chunks, cpg, q, N, zrow;
  int zero_offset;
  uint32_t magic;

  __device__ __forceinline__ void bind(const int32_t* qweight, const int32_t* qzeros, const void* scales, int n, int K,
                                       int group_size) {
    const uint32_t G = (uint32_t)(K / group_size);
    qw = buffer_of(qweight, (uint32_t)(K / 32 * BITS) * (uint32_t)n * 4u);
    qz = buffer_of(qzeros, G * (uint32_t)(n / 32 * BITS) * 4u);
    sc = buffer_of(scales, G * (uint32_t)n * 2u);
  }
  __device__ __forceinline__ void place(int n, int K, int group_size, int zoff, const int (&c)[CT], int quarter) {
    chunks = K / 32;
    cpg = group_size / 32;
    q = quarter;
    N = n;
    zrow = n / 32 * BITS;
    zero_offset = zoff;
    asm volatile("v_mov_b32 %0, 0x64006400" : "=v"(magic));
#pragma unroll
    for (int j = 0; j < CT; ++j) col[j] = c[j];
    const int r0 = block_row0<BITS>(0, q);
#pragma unroll
    for (int g = 0; g < SEG; ++g) {
      if constexpr (TILED) {
#pragma unroll
        for (int j = 0; j < CS; ++j)
          woff[g][j] = ((uint32_t)(col[g * CS + j] >> 4) * (uint32_t)chunks * BITS + (uint32_t)r0) * 64u +
                       (uint32_t)(col[g * CS + j] & 15) * 4u;
      } else {
        woff[g][0] = ((uint32_t)r0 * (uint32_t)N + (uint32_t)col[g * CS]) * 4u;
      }
    }
  }
  __device__ __forceinline__ uint32_t piece(int s) const { return (uint32_t)(4 * s + q); }
  __device__ __forceinline__ void load(int unit, bool live, uint8_t*, Regs* r) const {
    const int last = live ? chunks : 0;              // chunks that may be read
    const uint32_t rowb = TILED ? 64u : (uint32_t)N * 4u;
    const uint32_t second = L == 2 ? (uint32_t)(block_row1<BITS>(0, q) - block_row0<BITS>(0, q)) * rowb : 0u;
#pragma unroll
    for (int u = 0; u < UPP; ++u) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int c = 4 * (UPP * unit + u) + s;
        const bool ok = c < last;
        const uint32_t base = (uint32_t)c * BITS * rowb;
#pragma unroll
        for (int l = 0; l < L; ++l) {
          const uint32_t add = base + (l ? second : 0u);
#pragma unroll
          for (int g = 0; g < SEG; ++g) {
            if constexpr (TILED) {
#pragma unroll
              for (int j = 0; j < CS; ++j) r->w[u][s][l][g * CS + j] = load4(qw, ok ? woff[g][j] + add : kPast);
            } else {
              const uint32_t off = ok ? woff[g][0] + add : kPast;
              if constexpr (CS == 2) {
                const u32x2_t v = __builtin_amdgcn_raw_buffer_load_b64(qw, (int)off, 0, 0);
                r->w[u][s][l][g * 2] = v[0];
                r->w[u][s][l][g * 2 + 1] = v[1];
              } else {
                r->w[u][s][l][g] = load4(qw, off);
              }
            }
          }
        }
      }
      {
        const int c = 4 * (UPP * unit + u) + (ONE ? 0 : q);
        const bool ok = c < last;
        const uint32_t g = (uint32_t)(min(c, chunks - 1) / cpg);
#pragma unroll
        for (int t = 0; t < SEG * ZS; ++t) {
          const int n = col[t * ZC];
          const uint32_t bit = (uint32_t)n * BITS, zo = (g * (uint32_t)zrow + (bit >> 5)) * 4u;
          const uint32_t so = (g * (uint32_t)N + (uint32_t)n) * 2u;
          r->z[u][t][0] = load4(qz, ok ? zo : kPast);
          if constexpr (BITS == 3) r->z[u][t][1] = load4(qz, ok && (bit & 31) + 3 * ZC > 32 ? zo + 4u : kPast);
          // one column: the word that holds it (a 16-bit load is widened where it is
          // issued, and that waits for every load before it)
          r->s[u][t] = load4(sc, ok ? so & ~3u : kPast);
        }
      }
    }
  }
  // a value that quarter s loaded, in every quarter
  __device__ __forceinline__ uint32_t of_chunk(uint32_t v, int s) const {
    if constexpr (ONE) return v;
    else return (uint32_t)__builtin_amdgcn_ds_bpermute((16 * s + (int)(threadIdx.x & 15)) * 4, (int)v);
  }
  template <int MT, int PL, class A>
  __device__ __forceinline__ void multiply(const uint8_t*, const Regs& r, int, const A& a, int nmt,
                                           floatx4_t (&acc)[MT][CT]) const {
    half2_t neg[CT][4], sp[CT];
    float bs[CT], bc[CT];
    half8_t x[4][MT][PL];
#pragma unroll
    for (int us = 0; us < 4 * UPP; ++us) {
      const int u = us >> 2, s = us & 3;
      if (s == 0) {                                // four steps' operands at once
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            if (mt >= nmt) break;
#pragma unroll
            for (int pl = 0; pl < PL; ++pl) x[i][mt][pl] = a(mt, pl, us + i);
          }
      }
      half8_t w[CT];
#pragma unroll
      for (int j = 0; j < CT; ++j) {
        if (s == 0 || !ONE) {
          const int t = j / ZC;
          const uint32_t sh = ((uint32_t)col[t * ZC] * BITS) & 31u, z0 = of_chunk(r.z[u][t][0], s);
          uint32_t zz;
          if constexpr (BITS == 3) zz = __builtin_amdgcn_alignbit(of_chunk(r.z[u][t][1], s), z0, sh);
          else zz = z0 >> sh;
          const int z = (int)((zz >> (BITS * (j % ZC))) & ((1u << BITS) - 1u)) + zero_offset;
          const int half = ZC == 2 ? j % ZC : col[t] & 1;
          const uint32_t sv = (of_chunk(r.s[u][t], s) >> (16 * half)) & 0xFFFFu;
          if constexpr (BF16) {
            bs[j] = bf16_to_f32(sv);
            bc[j] = -(float)z * bs[j];
          } else {
            sp[j] = as_half2(sv * 0x10001u);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              if constexpr (PAIRS) neg[j][v] = half2_t{neg_offset<4>(v, z), neg_offset<4>(v, z)};
              else neg[j][v] = neg_offset_natural<BITS>(v, z, z);
            }
          }
        }
        // the weights rounded once to the scales' type, as the format says
        u32x4_t b;
        const uint32_t w0 = r.w[u][s][0][j], w1 = r.w[u][s][L - 1][j];
        if constexpr (BF16) {
          float f[8];
          if constexpr (PAIRS) block4_regs_f32(w0, f);
          else block_fields_f32<BITS>(w0, w1, q, f);
#pragma unroll
          for (int v = 0; v < 4; ++v)
            b[v] = bf16_pair(__builtin_fmaf(f[2 * v], bs[j], bc[j]), __builtin_fmaf(f[2 * v + 1], bs[j], bc[j]));
        } else {
          uint32_t p[4];
          if constexpr (PAIRS) unpack_block<4>(w0, 0u, 0u, p, magic);
          else unpack_block_natural<BITS>(w0, w1, q, p, magic);
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            half2_t d;
            if constexpr (PAIRS) d = pair_minus_zero<4>(p[v], v, neg[j][v]);
            else d = pair_minus_zero_natural<BITS>(p[v], v, neg[j][v]);
            b[v] = as_u32(d * sp[j]);
          }
        }
        w[j] = __builtin_bit_cast(half8_t, b);
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        if (mt >= nmt) break;
#pragma unroll
        for (int pl = 0; pl < PL; ++pl) {
#pragma unroll
          for (int j = 0; j < CT; ++j) acc[mt][j] = mfma16<BF16>(x[s][mt][pl], w[j], acc[mt][j]);
        }
      }
    }
  }
};

// ---- rows of x in LDS: row r (of PL planes x rows) is `kp` k in 16-byte
// pieces, piece p at slot p ^ (r % 16), so that the 16 rows one operand read
// serves fall into 16 different bank groups.
struct StagedRows {
  __amdgpu_buffer_rsrc_t rsrc;
  const uint32_t* off;               // LDS: byte offset of each row
  uint32_t plane;                    // byte distance of the planes
  int rows, K, kp;                   // kp a multiple of 512

  // k [k0, k0 + kp) of every row into lds; k >= min(K, end) reads zero
  template <int PL> __device__ __forceinline__ void issue(int k0, int end, uint8_t* lds, int wave, int nw, int lane) const {
    const int chunks = kp >> 9, stop = min(K, end);
    int r = 0, c = wave;
    while (c >= chunks) {
      c -= chunks;
      ++r;
    }
    while (r < rows) {
      const uint32_t base = (uint32_t)__builtin_amdgcn_readfirstlane((int)off[r]);
      const int k = k0 + 8 * ((64 * c + lane) ^ (r & 15));
#pragma unroll
      for (int pl = 0; pl < PL; ++pl)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rsrc, (__attribute__((address_space(3))) void*)(lds + ((pl * rows + r) * kp + 512 * c) * 2), 16,
            (int)(k < stop ? base + pl * plane + 2u * (uint32_t)k : kPast), 0, 0, 0);
      c += nw;
      while (c >= chunks) {
        c -= chunks;
        ++r;
      }
    }
  }
};

// Operand reads of one unit from a staged phase: lane row l % 16 of row tile
// mt (an absent row reads row 0: its results are never used).
template <class W, int MT> struct UnitOperand {
  const uint8_t* lds;
  const W& w;
  uint32_t row[MT], swz, plane;      // byte offsets; plane: rows * kp * 2
  int first;                         // first piece of the unit within the phase
  __device__ __forceinline__ half8_t operator()(int mt, int pl, int s) const {
    const uint32_t p = (uint32_t)first + ((uint32_t)w.piece(s) ^ swz);
    return *reinterpret_cast<const half8_t*>(lds + row[mt] + pl * plane + 16u * p);
  }
};

// Every load this wave has issued is complete, and every wave's: LDS holds the
// phase, and the buffer of the phase before is free.
__device__ __forceinline__ void phase_ready() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0x0070);              // vmcnt(0) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

}  // namespace gptq
