// Kernel argument blocks and launch entry points of the MXFP4 and
// mixture-of-experts operators (internal to libgptq.so).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gptq {

hipError_t launch_mx_quantize(const void* x, int type, int64_t M, int64_t K, uint8_t* codes, uint8_t* scales,
                              hipStream_t stream);
hipError_t launch_mx_dequant(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K, void* out, int type,
                             hipStream_t stream);

// Kernel and launch shape of a quantisation, as text.
void describe_mx_quantize(int type, int64_t M, int64_t K, char* buf, size_t n);

struct MxGemmArgs {
  const void* x;             // [M, K] fp16 / bf16, or MXFP4 codes [M, K/2]
  const uint8_t* x_scales;   // [M, K/32] (MXFP4 activations)
  const uint8_t* codes;      // [N, K/2]
  const uint8_t* scales;     // [N, K/32]
  void* out;                 // [M, N]
  int M, N, K;
  int x_type, out_type;
  // K in `splits` parts of split_tiles k tiles (units of the streaming kernel);
  // with splits > 1 fp32 sums go to ws [splits, M, N] first
  int splits, split_tiles;
  float* ws;
  // tiles (many rows): tile_m rows by tile_n columns; tile_m == 0: the
  // streaming kernel, nwc column waves by nwk k waves per workgroup, arrivals
  // of a tile's splits counted in cnt
  int tile_m, tile_n, tiles_m, tiles_n;
  int pair_stores;           // two adjacent 16-bit outputs may be stored as one word
  int quad_stores;           // out is 16-byte aligned
  int nwc, nwk;
  uint32_t* cnt;
};
// Fills in the launch shape; returns the workspace bytes it wants (0: none).
size_t plan_mx_gemm(MxGemmArgs* a, bool allow_split, size_t* counter_bytes);
hipError_t launch_mx_gemm(const MxGemmArgs& a, hipStream_t stream);
hipError_t launch_mx_tile(const MxGemmArgs& a, hipStream_t stream);
// A planned product's kernel: what is launched, its name, grid and LDS.
struct MxKernel {
  void (*fn)(MxGemmArgs);
  const char* name;
  unsigned grid, block;
  size_t lds;                // dynamic
};
MxKernel mx_gemm_kernel(const MxGemmArgs& a);
MxKernel mx_tile_kernel_of(const MxGemmArgs& a);
hipError_t launch_mx_kernel(const MxKernel& k, const MxGemmArgs& a, hipStream_t stream);

// One stack of expert weights, [rows -> cols] per expert.
struct ExpertStack {
  const void* weight;        // MXFP4 codes [E, cols, rows/2] or qweight
  const int32_t* zeros;      // GPTQ
  const void* scales;        // MXFP4 uint8 [E, cols, rows/32] or 16-bit [E, G, cols]
  int bits;                  // 0: MXFP4
  int group_size, zero_offset, tiled;
  int64_t weight_stride, zeros_stride, scales_stride;   // bytes per expert
};

// Launch shape of one of the layer's products: nwc column waves by nwk k waves
// per workgroup, rows of one expert per row block.
struct MoeShape {
  int nwc, nwk, block_rows;
};

struct MoeArgs {
  const void* x;             // [T, H]
  const void* w_router;      // [E, H]
  void* out;                 // [T, H]
  int bf16;
  int T, H, I, E, k, renorm;
  ExpertStack gate_up, down;
  int32_t* chosen;           // [T * k] expert of pair t * k + j
  float* weight;             // [T * k] its weight
  void* h;                   // hidden values: [2, T * k, I] in two bf16 parts, or, before
                             // fp16 GPTQ down weights, [T * k, I] in fp32
  uint32_t* top;             // fp32 h: [up_tiles, T * k] bits of the largest |h| of a
  int up_tiles;              // row in each of gate_up's column tiles
  int split_first;           // fp32 h goes to split_h [2, T * k, I], two fp16 parts, in
  uint16_t* split_h;         // a kernel of its own; else the down product splits it
  MoeShape up_shape, down_shape;
  int row_blocks;            // gate_up: row blocks an expert may have
  // down product: workgroups per column tile; with several, their fp32 sums
  // [splits, T, H] go to part, the last to arrive (counted in cnt[tile], zero
  // between launches) adds them
  int splits;
  float* part;
  uint32_t* cnt;
};
constexpr int kMoeTokens = 64;   // tokens of one launch
// Launch shape and the workspace arrays from `base`; returns the bytes they
// take, and the counters' in *counter_bytes.
size_t plan_moe(MoeArgs* a, char* base, size_t* counter_bytes);
hipError_t launch_moe(const MoeArgs& a, hipStream_t stream);

// The library's workspace of (device, stream): `counters` uint32 zeros that
// every kernel leaves at zero, then `bytes`.  False when it cannot be had
// (no memory, or the stream is being captured and it would have to grow).
bool stream_workspace(hipStream_t stream, size_t bytes, size_t counter_bytes, void** base, uint32_t** counters);

}  // namespace gptq
