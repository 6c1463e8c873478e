// Weights in 4 bits: the packed layout and the launchers.
//
// An [M][K] matrix is cut into blocks of 128 rows by 128 columns, row block by
// row block, the column blocks of one side by side; a block is
//   codes   8192 bytes: for each 16 rows (mi), each 64 columns (h) and each lane
//           4 g + t of a warp four words, in the order in which a warp's products
//           of 16 by 16 take them: word w holds row 16 mi + g + 8 (w / 2), and of
//           its two column steps s = 4 h + 2 (w % 2) and s + 1 the columns
//           16 s + 2 t + {0, 1, 8, 9}.  Pair p (of the four pairs of neighbours)
//           has its even column in bits 4 p and its odd one in bits 16 + 4 p: one
//           shift and one mask leave two codes at the low ends of two 16-bit lanes;
//   scales  [128 / group][128 rows] of the scale type;
//   zeros   [128 / group][128 rows] bytes, if the matrix has them.
// Rows past M and columns past K have scale 0 and code and zero point 8.
#pragma once
#include <stdint.h>

#include "common.cuh"

namespace dfl {

constexpr int kW4Tile = 128;          // rows and columns of a block
constexpr int kW4Codes = 8192;        // bytes of its codes
constexpr int kW4Zero = 8;            // the zero point of a matrix without zeros

struct W4View {
  int M, K, group, scale_f32, zeros;
  int kt;              // column blocks
  int block_bytes;
  const uint8_t* packed;
  __host__ __device__ __forceinline__ const uint8_t* block(int mt, int k) const {
    return packed + ((long long)mt * kt + k) * block_bytes;
  }
  __host__ __device__ __forceinline__ int groups() const { return kW4Tile / group; }
};

// The scale and the zero point of row r (of 128) in group gi of a block.
__device__ __forceinline__ float w4_scale(const W4View& w, const uint8_t* block, int gi, int r) {
  const int i = gi * kW4Tile + r;
  return w.scale_f32 ? reinterpret_cast<const float*>(block + kW4Codes)[i]
                     : to_f<bf16>(reinterpret_cast<const bf16*>(block + kW4Codes)[i]);
}
__device__ __forceinline__ int w4_zero(const W4View& w, const uint8_t* block, int gi, int r) {
  if (!w.zeros) return kW4Zero;
  return block[kW4Codes + w.groups() * kW4Tile * (w.scale_f32 ? 4 : 2) + gi * kW4Tile + r];
}
// Byte of the codes at which the words of (mi, h, lane) begin.
__host__ __device__ __forceinline__ int w4_word_at(int mi, int h, int lane) { return ((mi * 2 + h) * 32 + lane) * 16; }
// Row and first column of pair p of word w: see above.
__host__ __device__ __forceinline__ int w4_row(int mi, int lane, int w) { return mi * 16 + (lane >> 2) + 8 * (w >> 1); }
__host__ __device__ __forceinline__ int w4_col(int h, int lane, int w, int p) {
  return 16 * (4 * h + 2 * (w & 1) + (p >> 1)) + 2 * (lane & 3) + 8 * (p & 1);
}

// What a product does with its sums: out = y + add, or the activation over pairs of rows.
struct W4Epi {
  const float* add;  // null: none
  int swiglu;
  void* out;         // float32; with the activation of x's type
};

cudaError_t w4_pack(const W4View& w, const uint8_t* codes, const void* scales, const uint8_t* zeros, cudaStream_t s);
cudaError_t w4_quantize(const W4View& w, int dtype, const void* src, long long ld, cudaStream_t s);
cudaError_t w4_unpack(const W4View& w, int dtype, void* dst, cudaStream_t s);
// float32 x on the CUDA cores.
cudaError_t w4_linear_core(const W4View& w, const void* x, long long ldx, int rows, const W4Epi& epi,
                           cudaStream_t s);

// Scratch of the tensor-core products: two pieces a run, of 128 by (rows, rounded up to a power of two, 8 at least)
// floats; w4_max_runs() * 4 tickets, zero between calls; the status word.
struct W4Scratch {
  float* part;
  int* tickets;
  int* status;
};
// How a product is split, and its scratch.
struct W4Run {
  int blocks, per, runs;  // blocks of the matrix, blocks a run, runs
  float* part;            // [runs][2][float4 of sums a thread][128 threads][4]
  int* tickets;           // [runs][4 warps] of the row block that begins in the run and ends in a later one
  int* status;
  unsigned long long wait_ns;
};
// Up to this many rows go to the kernel fed from registers, whose CTAs share an SM; more take one for themselves.
constexpr int kW4MmaRows = 16;
W4Run w4_run(const W4View& w, const W4Scratch& sc, int rows);
int w4_max_runs();
// Floats of partial sums that calls of up to max_rows rows need.
size_t w4_part_floats(int max_rows);
// bf16 x on the tensor cores, up to 16 rows: fed from registers; more: from TMEM and shared memory.
cudaError_t w4_linear_mma(const W4View& w, const void* x, long long ldx, int rows, const W4Epi& epi,
                          const W4Scratch& sc, cudaStream_t s);
// (A 2-D map over bf16 rows [rows][cols], ld elements apart: boxes of 64 columns, 128 bytes swizzled, by box_rows.)
bool make_rows_map(const void* x, int rows, int cols, long long ld, int box_rows, CUtensorMap* out);
cudaError_t w4_linear_tc(const W4View& w, const void* x, long long ldx, int rows, const W4Epi& epi, const W4Scratch& sc,
                         cudaStream_t s);

}  // namespace dfl
