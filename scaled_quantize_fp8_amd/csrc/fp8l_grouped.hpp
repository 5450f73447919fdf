// Linear layers over ragged groups of rows (one weight matrix per group, the
// experts of a mixture): the tiles of all groups in one launch.
//
//   rows:      C[t, j] = sum_k A(t, k) B_e(j, k) / (sa sb[e]) (+ bias[e][j])
//              for the rows t of group e (the forward, and dX with B_e read
//              crosswise); C, A [T, ..] in group order.
//   contract:  C_e[i, j] = sum_{t in e} A(t, i) B(t, j) / (sa sb)  (dW): both
//              operands crosswise, the contraction is the group's rows.
//
// The tile bodies are the dense GEMMs' (fp8l_gemm.hpp, fp8l_gemm4.hpp,
// fp8l_gemm5.hpp): a block moves the operand pointers to its group and tile
// and runs one.  A tile never spans two groups; rows past the group's end
// read as zeros through the buffer range (the body's A resource ends with
// the group) and are not stored.
//
// Rows: how many tiles there are is known on the device only; the grid has a
// block for every tile that there could be (each group may add one row of
// tiles to the T rows' own), and a block without a tile ends at once.  Tiles
// are numbered group by group, inside a group down tile rows first, and XCD
// x gets the x-th eighth of them, so an expert's weights are read into one
// or two L2s.  (A loop over tiles in as many blocks as fit the chip does not
// pay: the compiler keeps the tile's lane constants alive across the loop
// and spills over a hundred registers.)
//
// Contract: every group has the same tiles, whatever its rows (none: its dW
// is zeros), so the grid is exact; each group's tiles are dealt over all
// XCDs, because their lengths differ from group to group.
#pragma once

#include "fp8l_gemm5.hpp"
#include "fp8l_gemm6.hpp"
#include "fp8l_group.hpp"

namespace fp8l {

struct GroupStrides {
  int64_t b;       // bytes from one group's B to the next (rows)
  int64_t c;       // elements from one group's C to the next (contract)
  int32_t sb;      // floats from one group's scale_b to the next (0: shared)
  int32_t bias;    // elements from one group's bias to the next
};

// What a launch does besides its tiles, in block 0: the ring folds left by
// the quantizes before it, and for operands that came quantized their scale
// snapshots (n floats) and zero amax.
struct GroupedSide {
  RingFold fold[2];
  const float* scale_src[2];
  float* scale_dst[2];
  float* amax_dst[2];
  int32_t n[2];
};

FP8L_DEV void grouped_side(const GroupedSide& s) {
  if (blockIdx.x != 0) return;
  for (int o = 0; o < 2; ++o) {
    if (s.scale_dst[o])
      for (int i = threadIdx.x; i < s.n[o]; i += blockDim.x) s.scale_dst[o][i] = s.scale_src[o][i];
    if (s.amax_dst[o] && threadIdx.x == 0) *s.amax_dst[o] = 0.0f;
  }
  if (threadIdx.x < 64) {
    if (s.fold[0].ring) ring_fold_wave(s.fold[0]);
    if (s.fold[1].ring) ring_fold_wave(s.fold[1]);
  }
}

// Tile bodies.  kBlocks: blocks per CU (LDS).
template <int LA, int LB, int FA, int FB>
struct TileAny {  // any size, stride and alignment
  static constexpr int kBM = fp8l::kBM, kBN = fp8l::kBN, kThreads = kGThreads, kBlocks = 2;
  static constexpr int kLds = kGemmLds;
  FP8L_DEV static void run(const GemmArgs& g, int tm, int tn, uint8_t* s) {
    gemm_tile<LA, LB, FA, FB>(g, tm, tn, s);
  }
};
template <int LA, int LB, int FA, int FB>
struct Tile256 {
  static constexpr int kBM = 256, kBN = 256, kThreads = 512, kBlocks = 1;
  static constexpr int kLds = gemm4_lds_bytes<FA == kI8>();
  FP8L_DEV static void run(const GemmArgs& g, int tm, int tn, uint8_t* s) {
    gemm4_tile<LA, LB, FA, FB>(g, tm, tn, s);
  }
};
template <int LA, int LB, int FA, int FB>
struct Tile128x256 {
  static constexpr int kBM = 128, kBN = 256, kThreads = 256, kBlocks = 2;
  static constexpr int kLds = gemm6_lds_bytes<FA == kI8>();
  FP8L_DEV static void run(const GemmArgs& g, int tm, int tn, uint8_t* s) {
    gemm6_tile<LA, LB, FA, FB>(g, tm, tn, s);
  }
};
template <int LA, int LB, int FA, int FB>
struct Tile128 {
  static constexpr int kBM = 128, kBN = 128, kThreads = 512, kBlocks = 1;
  static constexpr int kLds = gemm5_lds_bytes<FA == kI8>();
  FP8L_DEV static void run(const GemmArgs& g, int tm, int tn, uint8_t* s) {
    gemm5_tile<LA, LB, FA, FB>(g, tm, tn, s);
  }
};

// Move a problem's operands to tile row tm (of bm rows) of a group; A ends
// with the group.  I8: scale_a holds one scale per row.
template <bool I8>
FP8L_DEV void move_to_rows(GemmArgs& g, const GroupStrides& st, const GroupSpan& sp, int tm,
                           int bm) {
  const int64_t row = sp.start + (int64_t)tm * bm;
  g.a += row * g.lda;
  g.c += row * g.ldc;
  g.Mc = min<int64_t>(sp.end - row, bm);
  g.b += sp.e * st.b;
  g.scale_b += (int64_t)sp.e * st.sb;
  if (I8) g.scale_a += row;
  if (g.bias) g.bias = reinterpret_cast<const uint16_t*>(g.bias) + (int64_t)sp.e * st.bias;
}

template <class Tile, bool I8>
__global__ __launch_bounds__(Tile::kThreads, Tile::kBlocks) void grouped_rows_kernel(
    GemmArgs g, Groups gr, GroupStrides st, GroupedSide side) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem_rows[];
  int tm, tn;
  const GroupSpan sp = rows_work(gr, Tile::kBM, g.tiles_n, tm, tn);
  if (sp.e >= 0) {
    move_to_rows<I8>(g, st, sp, tm, Tile::kBM);
    Tile::run(g, 0, tn, smem_rows);
  }
  grouped_side(side);
}

// pad: blocks per group, the group's tiles rounded up to a multiple of 8.
template <class Tile>
__global__ __launch_bounds__(Tile::kThreads, Tile::kBlocks) void grouped_contract_kernel(
    GemmArgs g, Groups gr, GroupStrides st, int pad) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem_contract[];
  const int e = blockIdx.x / pad, l = blockIdx.x % pad;
  if (l >= g.tiles_m * g.tiles_n) return;
  int tm, tn;
  tile_coords_xcd(l, g.tiles_m, g.tiles_n, tm, tn);
  const int start = __builtin_amdgcn_readfirstlane(group_edge(gr, e));
  const int end = max(__builtin_amdgcn_readfirstlane(group_edge(gr, e + 1)), start);
  GemmArgs t = g;
  t.a += (int64_t)start * g.lda;
  t.b += (int64_t)start * g.ldb;
  t.Kc = end - start;
  t.c += e * st.c;
  Tile::run(t, tm, tn, smem_contract);
}

// ---------------------------------------------------------------- db

// Column sums of ragged groups: each group's rows are cut into chunks of
// kColRowsPerChunk and the chunks numbered group by group; block
// (chunk, strip) = (blockIdx.x / strips, blockIdx.x % strips) writes one row
// of ws.  A chunk never spans two groups, so ws needs no clearing: the
// finalize reads exactly the chunks of its group.  Thread (tx, ty) owns 8
// columns and rows ty, ty + 8, .. of the chunk; all sums in fp32, in an
// order that the sizes alone fix.
FP8L_DEV void chunk_sum_store(const float cs[8], float* ws, int64_t chunk, int64_t strip,
                              int64_t cols) {
  __shared__ float shsum[8][kColStrip + 1];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < 8; ++i) shsum[ty][tx * 8 + i] = cs[i];
  __syncthreads();
  const int64_t gc = strip * kColStrip + threadIdx.x;
  float t = 0.0f;
#pragma unroll
  for (int y = 0; y < 8; ++y) t += shsum[y][threadIdx.x];
  if (gc < cols) ws[chunk * cols + gc] = t;
}

// G [T, cols] quantized and summed in one pass (the grouped form of
// quantize_colsum_kernel: same codes, amax and ring finalize).  Rows of no
// group are neither read nor written.
template <int IN, int FMT, int SMODE>
__global__ __launch_bounds__(kQThreads) void quantize_groupsum_kernel(QArgs a, Groups gr,
                                                                      int strips) {
  const float s = launch_scale<FMT, SMODE>(a);
  const int chunk = blockIdx.x / strips, strip = blockIdx.x % strips;
  const GroupSpan sp = find_group(gr, kColRowsPerChunk, chunk);
  uint32_t mx = 0;
  if (sp.e >= 0) {
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t c0 = (int64_t)strip * kColStrip + tx * 8;
    const int64_t r0 = sp.start + (int64_t)sp.unit * kColRowsPerChunk;
    const int64_t r1 = min<int64_t>(r0 + kColRowsPerChunk, sp.end);
    float cs[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = 0.0f;
    if (c0 < a.cols) {
      const int cnt = (int)min<int64_t>(8, a.cols - c0);
      if (a.vec_ok && cnt == 8) {
        float v[4][8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int64_t r = r0 + ty + 8 * k;
          if (r < r1) {
            load8<IN>(a.x, r * a.cols + c0, v[k]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[k][i] = 0.0f;
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int64_t r = r0 + ty + 8 * k;
          uint32_t lm = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            lm = max(lm, absbits(v[k][i]));
            cs[i] += v[k][i];
          }
          if (r < r1) *reinterpret_cast<uint2*>(a.q + r * a.cols + c0) = quant8<FMT>(v[k], s, lm);
          mx = max(mx, lm);
        }
      } else {
        for (int64_t r = r0 + ty; r < r1; r += 8) {
          float v[8];
          mx = max(mx, quant_scalar8<IN, FMT>(a.x, a.q, r * a.cols + c0, cnt, s, v));
#pragma unroll
          for (int i = 0; i < 8; ++i) cs[i] += v[i];
        }
      }
    }
    chunk_sum_store(cs, a.colsum, chunk, strip, a.cols);
  }
  finish_launch<FMT, SMODE>(a, mx, s, blockIdx.x, gridDim.x);
}

// The same sums of pre-quantized codes (decoded; the finalize applies 1/sg).
template <int FMT>
__global__ __launch_bounds__(kQThreads) void groupsum_fp8_kernel(const uint8_t* g8, int64_t cols,
                                                                 Groups gr, int strips, int vec,
                                                                 float* ws) {
  const int chunk = blockIdx.x / strips, strip = blockIdx.x % strips;
  const GroupSpan sp = find_group(gr, kColRowsPerChunk, chunk);
  if (sp.e < 0) return;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int64_t c0 = (int64_t)strip * kColStrip + tx * 8;
  const int64_t r0 = sp.start + (int64_t)sp.unit * kColRowsPerChunk;
  const int64_t r1 = min<int64_t>(r0 + kColRowsPerChunk, sp.end);
  float cs[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) cs[i] = 0.0f;
  const int cnt = (int)max<int64_t>(0, min<int64_t>(8, cols - c0));
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t r = r0 + ty + 8 * k;
    if (r >= r1 || cnt <= 0) continue;
    const uint8_t* p = g8 + r * cols + c0;
    if (vec && cnt == 8) {
      const uint2 w = *reinterpret_cast<const uint2*>(p);
#pragma unroll
      for (int i = 0; i < 8; ++i) cs[i] += fp8_to_f32<FMT>(((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 0xffu);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < cnt) cs[i] += fp8_to_f32<FMT>(p[i]);
    }
  }
  chunk_sum_store(cs, ws, chunk, strip, cols);
}

}  // namespace fp8l
