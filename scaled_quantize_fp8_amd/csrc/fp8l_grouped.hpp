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

// Tile of block b of a contract problem; pad: blocks per group, the group's
// tiles rounded up to a multiple of 8.
template <class Tile>
FP8L_DEV void contract_block(GemmArgs& g, const Groups& gr, const GroupStrides& st, int pad, int b,
                             uint8_t* smem) {
  const int e = b / pad, l = b % pad;
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
  Tile::run(t, tm, tn, smem);
}

template <class Tile>
__global__ __launch_bounds__(Tile::kThreads, Tile::kBlocks) void grouped_contract_kernel(
    GemmArgs g, Groups gr, GroupStrides st, int pad) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem_contract[];
  contract_block<Tile>(g, gr, st, pad, blockIdx.x, smem_contract);
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

// Scale mode of a small dynamic quantize: every block takes the amax of the
// whole tensor itself (it is in L2 after the first), which saves the two
// launches of an amax pass (130 x 256: one launch of 6.9 us in the place of
// three of 4 to 5 us).
constexpr int kScaleLocal = 4;
constexpr int64_t kLocalMost = 65536;  // elements

template <int IN>
FP8L_DEV uint32_t block_absmax(const QArgs& a, uint32_t* sh) {
  const int64_t n = limited(a.n, a.limit);
  uint32_t mx = 0;
  const int64_t nv = a.vec_ok ? n / 8 : 0;
  for (int64_t c = threadIdx.x; c < nv; c += kQThreads) {
    float v[8];
    load8<IN>(a.x, 8 * c, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = max(mx, absbits(v[i]));
  }
  for (int64_t c = 8 * nv + threadIdx.x; c < n; c += kQThreads)
    mx = max(mx, absbits(load1<IN>(a.x, c)));
  return block_max_u32(mx, sh);
}

// G [T, cols] quantized and summed in one pass (the grouped form of
// quantize_colsum_kernel: same codes, amax and ring finalize).  The first
// chunks are the rows before the first group, quantized like the rest but in
// no sum; rows behind the last group are neither read nor written.  most:
// chunks that the workspace holds (offsets that break the contract can give
// more).
template <int IN, int FMT, int SMODE>
__global__ __launch_bounds__(kQThreads) void quantize_groupsum_kernel(QArgs a, Groups gr,
                                                                      int strips, int most) {
  float s;
  if constexpr (SMODE == kScaleLocal) {
    __shared__ uint32_t sh_amax[kQThreads / 64];
    const float m = __uint_as_float(block_absmax<IN>(a, sh_amax));
    s = scale_from_amax(m, FmtTraits<FMT>::kMax, 1.0f);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      *a.scale_used = s;
      *a.amax_out = m;
    }
  } else {
    s = launch_scale<FMT, SMODE>(a);
  }
  const int chunk = blockIdx.x / strips, strip = blockIdx.x % strips;
  const int lead_rows = group_edge(gr, 0), lead = units_of(lead_rows, kColRowsPerChunk);
  const GroupSpan sp = chunk < lead ? GroupSpan{0, 0, lead_rows, chunk, 0}
                                    : find_group(gr, kColRowsPerChunk, chunk - lead);
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
    if (chunk >= lead && chunk - lead < most)
      chunk_sum_store(cs, a.colsum, chunk - lead, strip, a.cols);
  }
  if constexpr (SMODE != kScaleLocal)
    finish_launch<FMT, SMODE>(a, mx, s, blockIdx.x, gridDim.x);
}

// db of one group and a strip of columns by one block (256 threads or more,
// every thread calls it).  sh: kDbLds bytes of LDS.
constexpr int kDbLds = 8 * 256 * 4;
struct DbArgs {
  uint16_t* db;        // [E][N], null: none
  const float* ws;     // chunk sums of a quantized-here G, or null: sum g8
  int32_t most;        // chunks in ws
  const uint8_t* g8;   // codes of a G that came quantized
  int32_t g8_e5m2, vec;
  const float* scale;  // of g8 (the sums are of decoded codes), else null
  int64_t N;
};

FP8L_DEV int db_strip(const DbArgs& a) { return a.ws ? 64 : 256; }  // columns (as db_blocks on the host)

FP8L_DEV void db_store(const DbArgs& a, int e, int64_t n, float t) {
  if (a.scale) t *= 1.0f / *a.scale;
  a.db[(int64_t)e * a.N + n] = (uint16_t)f32_to_bf16(t);
}

// From the chunk sums: wave w adds chunks w, w + 4, .., the four sums meet in
// wave order.  A group without rows gets 0; chunks past ws (offsets that
// break the contract) are not read.
FP8L_DEV void db_from_chunks(const DbArgs& a, const Groups& gr, int e, int strip, float* sh) {
  const GroupSpan sp = group_span(gr, kColRowsPerChunk, e);
  // (before < 0: such offsets can give more chunks than 32 bits count)
  const int chunks =
      sp.before < 0 ? 0 : min(units_of(sp.end - sp.start, kColRowsPerChunk), a.most - sp.before);
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t n = (int64_t)strip * 64 + lane;
  float s = 0.0f;
  if (n < a.N && w < 4)
    for (int c = w; c < chunks; c += 4) s += a.ws[(int64_t)(sp.before + c) * a.N + n];
  if (w < 4) sh[w * 64 + lane] = s;
  __syncthreads();
  if (w == 0 && n < a.N)
    db_store(a, e, n, sh[lane] + sh[64 + lane] + sh[128 + lane] + sh[192 + lane]);
}

// From the codes, in one go: 16 lanes a row (16 columns each), 4 rows a wave
// instruction, eight of them in flight; a wave's four row partials meet in an
// xor tree, the waves' in wave order.  All orders are fixed by the sizes.
template <int FMT>
FP8L_DEV void db_from_codes(const DbArgs& a, const Groups& gr, int e, int strip, float* sh) {
  const int start = __builtin_amdgcn_readfirstlane(group_edge(gr, e));
  const int end = max(__builtin_amdgcn_readfirstlane(group_edge(gr, e + 1)), start);
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, nw = blockDim.x >> 6;
  const int64_t c0 = (int64_t)strip * 256 + 16 * (lane & 15);
  const int cnt = (int)min<int64_t>(16, a.N - c0);
  float s[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) s[i] = 0.0f;
  if (cnt > 0) {
    int r = start + 4 * w + (lane >> 4);
    const uint8_t* p = a.g8 + (int64_t)r * a.N + c0;
    const int64_t step = (int64_t)4 * nw * a.N;
    if (a.vec && cnt == 16) {
      for (; r < end; r += 8 * 4 * nw, p += 8 * step) {
        uint4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)  // rows past the end: the first one again, not added
          v[k] = *reinterpret_cast<const uint4*>(p + (r + 4 * nw * k < end ? k * step : 0));
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (r + 4 * nw * k >= end) continue;
          const uint32_t q[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
          for (int i = 0; i < 16; ++i)
            s[i] += fp8_to_f32<FMT>((q[i >> 2] >> (8 * (i & 3))) & 0xffu);
        }
      }
    } else {
      for (; r < end; r += 4 * nw, p += step)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i < cnt) s[i] += fp8_to_f32<FMT>(p[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    s[i] += __shfl_xor(s[i], 16);
    s[i] += __shfl_xor(s[i], 32);
    if (lane < 16) sh[w * 256 + 16 * lane + i] = s[i];
  }
  __syncthreads();
  const int64_t n = (int64_t)strip * 256 + threadIdx.x;
  if (threadIdx.x < 256 && n < a.N) {
    float t = sh[threadIdx.x];
    for (int k = 1; k < nw; ++k) t += sh[k * 256 + threadIdx.x];
    db_store(a, e, n, t);
  }
}

FP8L_DEV void db_block(const DbArgs& a, const Groups& gr, int b, float* sh) {
  const int width = db_strip(a), strips = (int)((a.N + width - 1) / width);
  const int e = b / strips, strip = b % strips;
  if (a.ws) db_from_chunks(a, gr, e, strip, sh);
  else if (a.g8_e5m2) db_from_codes<kE5M2>(a, gr, e, strip, sh);
  else db_from_codes<kE4M3>(a, gr, e, strip, sh);
}

// The whole backward behind the quantize in one launch: dX in blocks
// [0, nx), dW in [nx, nx + nw), db in the rest (nx and nw multiples of 8, so
// each problem keeps its XCD order).  All three wait only for the quantize;
// in one grid the tail of one is filled by the next, and two launches (about
// 4 us each on the GPU) go: 4093 rows, 32 experts of 1024 -> 4096 155 -> 132 us;
// 16384 rows, 8 experts of 1536 -> 6912 355 -> 321, where db from the codes
// as a pass and a launch of its own took 37 + 10 us.  dX's tiles, with the
// longer contraction as a rule, come first.
template <class TX, class TW>
__global__ __launch_bounds__(TX::kThreads, TX::kBlocks) void grouped_bwd_kernel(
    GemmArgs gx, GemmArgs gw, Groups gr, GroupStrides sx, GroupStrides sw, GroupedSide side, int nx,
    int nw, int pad, DbArgs db) {
  static_assert(TX::kThreads == TW::kThreads, "one block size");
  extern __shared__ __attribute__((aligned(16))) uint8_t smem_bwd[];
  const int b = blockIdx.x;
  if (b < nx) {
    int tm, tn;
    const GroupSpan sp = rows_work(gr, TX::kBM, gx.tiles_n, tm, tn);
    if (sp.e >= 0) {
      move_to_rows<false>(gx, sx, sp, tm, TX::kBM);
      TX::run(gx, 0, tn, smem_bwd);
    }
    grouped_side(side);
  } else if (b < nx + nw) {
    contract_block<TW>(gw, gr, sw, pad, b - nx, smem_bwd);
  } else {
    db_block(db, gr, b - nx - nw, reinterpret_cast<float*>(smem_bwd));
  }
}

}  // namespace fp8l
