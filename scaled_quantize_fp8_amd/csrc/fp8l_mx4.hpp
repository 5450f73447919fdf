// Linear layers in microscaled 4-bit floating point: blocks of 32 values
// along K share a power of two (E8M0, a biased exponent in a byte), elements
// are E2M1 (sign, two exponent bits, one of significand: 0, 0.5, 1, 1.5, 2,
// 3, 4, 6) [MX: OCP Microscaling Formats specification v1.0].
//
//   quantize  amax of a block = 1.f 2^a:  scale 2^(a - 2) (2 is E2M1's largest
//             exponent), not below 2^-127; elements x / scale, rounded to
//             nearest, ties to even, saturating at 6.  x / scale is exact in
//             32 bits, so the codes are those of the definition.  A block that
//             holds a NaN or an infinity gets the scale NaN (0xFF) and zeros.
//   product   Y[m, n] = sum over blocks of 2^(ex + ew) sum_32 qx qw (+ b[n]),
//             by the scaled MFMA, summed in 32 bits, rounded once.
//
// Layout of a matrix [rows, K], with B = ceil(K / 32) blocks a row:
//   codes   [rows][16 B] bytes, element 2 j of a row in byte j's low half;
//           elements past K are zeros, so every row is whole blocks and any K
//           takes the same path.
//   scales  [ceil(B / 4)][rows][4] bytes: one 32-bit word holds the four
//           blocks of a step of 128 values, and the words of neighbouring rows
//           lie side by side, so that a wave fetches its rows' scales of a
//           step as one contiguous piece (row-major scales would touch a line
//           per row for 4 bytes of it).  Bytes past B are zeros.
#pragma once

#include "fp8l_gemm3.hpp"
#include "fp8l_grouped.hpp"
#include "fp8l_mx4_span.hpp"
#include "fp8l_values.hpp"

namespace fp8l {

constexpr int kMxThreads = 256;

struct MxQuantArgs {
  const void* x;       // [mats][rows][K]
  uint8_t* codes;
  uint32_t* scales;    // words
  int64_t rows, K;
  int32_t steps, blocks;  // ceil(K / 128), ceil(K / 32)
  int32_t rows_log;       // rows of a block's tile: 1 << rows_log (0..4)
  const int32_t* valid;   // device row count, or null: all rows
};

// Biased exponent of a block's scale from the bits of its amax, 255: NaN.
FP8L_DEV uint32_t mx_scale(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - 2;
  return amax_bits > 0x7f7fffffu ? 255u : (uint32_t)max(e, 0);
}
// 1 / scale, exact (2^(127 - e) with e <= 252 is a normal number).
FP8L_DEV float mx_inverse(uint32_t e) { return __uint_as_float((254u - e) << 23); }

// Eight values already divided by their scale to eight codes.
FP8L_DEV uint32_t mx_codes8(const float v[8], float inv) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0] * inv, v[1] * inv, 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2] * inv, v[3] * inv, 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4] * inv, v[5] * inv, 1.0f, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6] * inv, v[7] * inv, 1.0f, 3);
  return w;
}

// 16 lanes hold a step of 128 values, lane sl of them values 8 sl and on: four
// lanes a block, whose amax they share by two DPP steps; then the four blocks'
// exponents meet in a word.  inside: the lane's block is one of the row's.
struct MxEight {
  uint32_t codes, word;
};
FP8L_DEV MxEight mx_eight(const float v[8], bool inside, int sl) {
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) mx = max(mx, absbits(v[i]));
  mx = max(mx, (uint32_t)__builtin_amdgcn_mov_dpp((int)mx, 0xB1, 0xF, 0xF, false));
  mx = max(mx, (uint32_t)__builtin_amdgcn_mov_dpp((int)mx, 0x4E, 0xF, 0xF, false));
  const uint32_t e = inside ? mx_scale(mx) : 0u;
  MxEight r;
  r.word = e << (8 * (sl >> 2));
  r.word |= (uint32_t)__builtin_amdgcn_mov_dpp((int)r.word, 0x141, 0xF, 0xF, false);
  r.word |= (uint32_t)__builtin_amdgcn_mov_dpp((int)r.word, 0x140, 0xF, 0xF, false);
  r.codes = e == 255u ? 0u : mx_codes8(v, mx_inverse(e));
  return r;
}

// A block of 256 threads walks its tile of rows along K, kU steps at a time
// with their loads in flight together (11008 x 4096 bf16, 114 MB in and out:
// 22 us with X in the last-level cache, where one step at a time takes 34; 26
// from memory).
// VEC: K a multiple of 8.
template <int IN, bool VEC>
__global__ __launch_bounds__(kMxThreads) void mx4_quantize_kernel(MxQuantArgs a) {
  constexpr int kU = IN == kInF32 ? 2 : 4;
  const int sl = threadIdx.x & 15, grp = threadIdx.x >> 4;
  const int per = 1 << a.rows_log;           // rows of the tile
  const int across = 16 >> a.rows_log;       // steps side by side
  const int64_t rows = a.valid ? min<int64_t>(max(*a.valid, 0), a.rows) : a.rows;
  const int64_t mat = blockIdx.z;
  const int64_t row_bytes = (int64_t)a.blocks * 16;
  for (int64_t r0 = (int64_t)blockIdx.x * per; r0 < rows; r0 += (int64_t)gridDim.x * per) {
    const int64_t r = r0 + (grp & (per - 1));
    const int64_t at = (mat * a.rows + r) * a.K;
    for (int64_t s0 = (int64_t)blockIdx.y * across * kU + (grp >> a.rows_log); s0 < a.steps;
         s0 += (int64_t)gridDim.y * across * kU) {
      Raw<IN, 8> raw[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int64_t k = (s0 + u * across) * 128 + 8 * sl;
        raw[u].zero();
        if (r < rows && k + 8 <= a.K) raw[u].load(a.x, at + k);
      }
      if constexpr (!VEC) {
        // the row's last piece, where it is not whole
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int64_t k = (s0 + u * across) * 128 + 8 * sl;
          if (r < rows && k < a.K && k + 8 > a.K) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (k + i < a.K) raw[u].put(i, load1<IN>(a.x, at + k + i));
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int64_t s = s0 + u * across;
        const bool inside = 4 * s + (sl >> 2) < a.blocks;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = raw[u].get(i);
        const MxEight e = mx_eight(v, inside, sl);
        if (r < rows && s < a.steps) {
          if (inside)
            *reinterpret_cast<uint32_t*>(a.codes + (mat * a.rows + r) * row_bytes + s * 64 + 4 * sl) =
                e.codes;
          if (sl == 0) a.scales[(mat * a.steps + s) * a.rows + r] = e.word;
        }
      }
    }
  }
}

struct MxDequantArgs {
  const uint8_t* codes;
  const uint32_t* scales;
  void* out;            // [mats][rows][K]
  int64_t rows, K;
  int32_t steps, blocks, vec, rows_log;
};

// The values of the codes, rounded once to the output's type, kU steps in
// flight.
template <int IN>
__global__ __launch_bounds__(kMxThreads) void mx4_dequantize_kernel(MxDequantArgs a) {
  constexpr int kU = 4;
  const int sl = threadIdx.x & 15, grp = threadIdx.x >> 4;
  const int per = 1 << a.rows_log, across = 16 >> a.rows_log;
  const int64_t mat = blockIdx.z;
  const int64_t row_bytes = (int64_t)a.blocks * 16;
  for (int64_t r = (int64_t)blockIdx.x * per + (grp & (per - 1)); r < a.rows;
       r += (int64_t)gridDim.x * per) {
    const uint8_t* const codes = a.codes + (mat * a.rows + r) * row_bytes;
    for (int64_t s0 = (int64_t)blockIdx.y * across * kU + (grp >> a.rows_log); s0 < a.steps;
         s0 += (int64_t)gridDim.y * across * kU) {
      uint32_t w[kU], word[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const MxPiece p = mx_piece(s0 + u * across, sl, a.K);
        w[u] = *reinterpret_cast<const uint32_t*>(codes + p.byte);
        word[u] = a.scales[(mat * a.steps + p.step) * a.rows + r];
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int64_t k = (s0 + u * across) * 128 + 8 * sl;
        const uint32_t e = (word[u] >> (8 * (sl >> 2))) & 255u;
        float v[8];
        const f32x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 0);
        const f32x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 1);
        const f32x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 2);
        const f32x2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 3);
        v[0] = p0.x; v[1] = p0.y; v[2] = p1.x; v[3] = p1.y;
        v[4] = p2.x; v[5] = p2.y; v[6] = p3.x; v[7] = p3.y;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[i] = e == 255u ? __uint_as_float(0x7fc00000u) : __builtin_ldexpf(v[i], (int)e - 127);
        if (k >= a.K) continue;
        const int64_t at = (mat * a.rows + r) * a.K + k;
        if (a.vec) {
          store8<IN>(a.out, at, v);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (k + i < a.K) store1<IN>(a.out, at + i, v[i]);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- products

// A tile's problem: operands moved to its rows of X and columns of Y.
struct MxArgs {
  const uint8_t* a;      // codes of X, [M][ld]
  const uint32_t* sa;    // its scale words, step s at sa + s * sa_step
  const uint8_t* b;      // codes of W, [N][ld]
  const uint32_t* sb;
  int64_t ld, sa_step, sb_step;
  int64_t M, N;          // rows and columns from here on
  int32_t steps;         // ceil(K / 128)
  uint16_t* c;           // [M][ldc], bf16 or fp16
  int64_t ldc;
  const uint16_t* bias;  // in c's type, or null
  int32_t out_f16, c_vec;
  int32_t tiles_m, tiles_n;
};

struct MxStrides {  // from one group's W to the next
  int64_t b, sb, bias;
};

FP8L_DEV void mx_move(MxArgs& g, int64_t row, int64_t rows, int64_t col) {
  g.a += row * g.ld;
  g.sa += row;
  g.M = rows;
  g.b += col * g.ld;
  g.sb += col;
  g.N -= col;
  g.c += row * g.ldc + col;
  if (g.bias) g.bias += col;
}

// A descriptor of values that all lanes hold alike, in scalar registers from the
// start: what a division left in vector registers the compiler would otherwise
// bring over again in a loop around every load.
FP8L_DEV __amdgpu_buffer_rsrc_t mx_rsrc(const void* p, int64_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  return make_rsrc(reinterpret_cast<const void*>((uint64_t)hi << 32 | lo),
                   __builtin_amdgcn_readfirstlane((uint32_t)bytes));
}

FP8L_DEV float mx_half(const MxArgs& g, uint32_t h) {
  return g.out_f16 ? f16_to_f32(h) : bf16_to_f32(h);
}
FP8L_DEV uint2 mx_pack4(const MxArgs& g, const float v[4]) {
  if (g.out_f16)
    return make_uint2(f32_to_f16(v[0]) | (f32_to_f16(v[1]) << 16),
                      f32_to_f16(v[2]) | (f32_to_f16(v[3]) << 16));
  return make_uint2(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]));
}

// A wave's way of reading MFMA operands: 16 rows of W and 16 NX of X, a piece
// (two steps: 128 bytes, a whole line, of every row) at a time.  The 16x16x128
// MFMA takes a block of 32 values and its scale per lane (lane 16 q + r: row r,
// block q of the step), so lanes side by side want different rows: loaded that
// way, a load of 64 x 16 bytes keeps the address unit busy for 64 clocks.  Here
// eight lanes load a row's line (16 clocks), and the wave turns it round in its
// own part of LDS, without a barrier: 33 rows of 11008 -> 4096 9.4 us against
// 11.8, 16 rows 7.4 against 9.6, 512 rows in 16 experts of 1536 -> 6912 21.9
// against 45.2.
template <int NX>
struct MxPieces {
  static constexpr int kOperands = 1 + NX;   // 0: W, 1 + m: X's rows from 16 m on
  static constexpr int kPiece = 2048 + 128;  // bytes of codes [16][128], scale words [2][16]
  // LDS holds W and two of X at a time: all five of 64 rows would leave room for
  // one block per CU (64 rows of 4096 -> 11008 15.3 us, so 12.0).
  static constexpr int kPlaces = kOperands < 3 ? kOperands : 3, kWave = kPlaces * kPiece;
  struct Regs {
    v4i c[kOperands][2];
    uint32_t e[1 + (NX + 1) / 2];
  };
  __amdgpu_buffer_rsrc_t rb, rsb, ra, rsa;
  uint32_t ld, sb_step, sa_step, steps, j0;
  uint8_t* mine;

  // j0: the wave's first column from g's on, of cols in reach.
  FP8L_DEV MxPieces(const MxArgs& g, uint32_t j0, int64_t cols, uint8_t* mine)
      : rb(mx_rsrc(g.b, cols * g.ld)),
        // words of rows past the end are those of other rows, or zeros past the
        // last step: they meet zero codes or columns that are not stored
        rsb(mx_rsrc(g.sb, mx_scale_span(g.steps, (int32_t)g.sb_step, (int32_t)cols))),
        ra(mx_rsrc(g.a, NX ? g.M * g.ld : 0)),
        rsa(mx_rsrc(g.sa, NX ? mx_scale_span(g.steps, (int32_t)g.sa_step, (int32_t)g.M) : 0)),
        ld((uint32_t)g.ld), sb_step((uint32_t)g.sb_step), sa_step((uint32_t)g.sa_step),
        steps((uint32_t)g.steps), j0(j0), mine(mine) {}

  // Piece p, zeros past the last block (a wave's first one is loaded whether it
  // has one or not).
  FP8L_DEV void load(Regs& t, uint32_t p) const {
    const uint32_t lane = threadIdx.x & 63, row = lane >> 3, k = 128 * p + 16 * (lane & 7);
#pragma unroll
    for (int o = 0; o < kOperands; ++o)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t at = (o ? 16 * (o - 1) : j0) + 8 * j + row;
        t.c[o][j] = __builtin_bit_cast(
            v4i, __builtin_amdgcn_raw_buffer_load_b128(o ? ra : rb, k < ld ? at * ld + k : kMxNowhere,
                                                       0, 0));
      }
    const uint32_t s = 2 * p + (lane >> 4 & 1), r = lane & 15, half = lane >> 5;
#pragma unroll
    for (int i = 0; i < 1 + (NX + 1) / 2; ++i) {
      const uint32_t m = 2 * (i - 1) + half;  // of X
      const bool in = s < steps && (i ? m < NX : half == 0);
      const uint32_t at = i ? s * sa_step + 16 * m + r : s * sb_step + j0 + r;
      t.e[i] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(i ? rsa : rsb, in ? 4 * at : kMxNowhere,
                                                              0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  }

  // 16-byte chunk of a row's line: rows that are read together spread over the banks.
  FP8L_DEV static uint32_t chunk(uint32_t row, uint32_t c) {
    return 128 * row + 16 * (c ^ (row & 7));
  }

  // W to place 0; rows 16 m to 16 m + 32 of X to places 1 and 2 (m even).
  FP8L_DEV void put_w(const Regs& t) const {
    const uint32_t lane = threadIdx.x & 63;
    put_codes(t, 0, 0);
    if (lane < 32) *reinterpret_cast<uint32_t*>(mine + 2048 + 4 * lane) = t.e[0];
    asm volatile("" ::: "memory");  // other lanes' bytes are read next
  }
  FP8L_DEV void put_x(const Regs& t, int m) const {
    const uint32_t lane = threadIdx.x & 63, half = lane >> 5;
    asm volatile("" ::: "memory");  // what lay there has been read
    put_codes(t, 1 + m, 1);
    if (m + 1 < NX) put_codes(t, 2 + m, 2);
    if (m + 1 < NX || half == 0)
      *reinterpret_cast<uint32_t*>(mine + (1 + half) * kPiece + 2048 + 4 * (lane & 31)) =
          t.e[1 + m / 2];
    asm volatile("" ::: "memory");
  }
  FP8L_DEV void put_codes(const Regs& t, int o, int place) const {
    const uint32_t lane = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      *reinterpret_cast<v4i*>(mine + place * kPiece + chunk(8 * j + (lane >> 3), lane & 7)) =
          t.c[o][j];
  }

  // The operand at a place, of the piece's step u.
  FP8L_DEV v8i codes(int place, int u) const {
    const uint32_t r = threadIdx.x & 15, q = (threadIdx.x & 63) >> 4;
    const v4i a = *reinterpret_cast<const v4i*>(mine + place * kPiece + chunk(r, 4 * u + q));
    return v8i{a.x, a.y, a.z, a.w, 0, 0, 0, 0};
  }
  FP8L_DEV uint32_t scale(int place, int u) const {  // (bytes past the last block are zeros)
    const uint32_t r = threadIdx.x & 15, q = (threadIdx.x & 63) >> 4;
    return mine[place * kPiece + 2048 + 4 * (16 * u + r) + q];
  }
};

// Few rows (decoding): a wave multiplies 16 columns by all rows; KW waves of a
// block share a tile column and split K, their partial sums meet in LDS in wave
// order.
template <int MT>
struct MxSkinny {
  using P = MxPieces<MT>;
  static constexpr int kBM = 16 * MT, kWaveN = 16, kThreads = 512, kLds = 8 * P::kWave;
  static_assert(kLds >= 8 * MT * 1024 && kLds <= 65536, "partial sums fit, and need no larger limit");

  FP8L_DEV static v4f mma(v8i b, v8i a, v4f c, uint32_t sb, uint32_t sa) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, 4, 4, 0, (int)sb, 0, (int)sa);
  }
  FP8L_DEV static void store(const MxArgs& g, int row, int64_t j, v4f acc) {
    if (row >= g.M || j >= g.N) return;
    float v[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      v[t] = acc[t];
      if (g.bias && j + t < g.N) v[t] += mx_half(g, g.bias[j + t]);
    }
    const uint2 w = mx_pack4(g, v);
    uint16_t* const dst = g.c + row * g.ldc + j;
    if (g.c_vec) {
      *reinterpret_cast<uint2*>(dst) = w;
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (j + t < g.N) dst[t] = (uint16_t)((t < 2 ? w.x : w.y) >> (16 * (t & 1)));
    }
  }

  // The sums of all K: of the KW waves of a column in wave order.
  FP8L_DEV static void finish(const MxArgs& g, const v4f (&acc)[MT], int KW, uint8_t* smem) {
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j0 = wave / KW * kWaveN, JW = 8 / KW;
    if (KW == 1) {
#pragma unroll
      for (int m = 0; m < MT; ++m) store(g, 16 * m + r, j0 + 4 * q, acc[m]);
      return;
    }
    // partial sums: [wave][fragment][lane] x 16 bytes
    v4f* const part = reinterpret_cast<v4f*>(smem);
#pragma unroll
    for (int m = 0; m < MT; ++m) part[(wave * MT + m) * 64 + lane] = acc[m];
    __syncthreads();
    for (int f = wave; f < JW * MT; f += 8) {
      const int fj = f / MT, fm = f % MT;
      const v4f* src = part + (fj * KW * MT + fm) * 64 + lane;
      v4f s = src[0];
      for (int w = 1; w < KW; ++w) {
        const v4f o = src[w * MT * 64];
#pragma unroll
        for (int t = 0; t < 4; ++t) s[t] += o[t];
      }
      store(g, 16 * fm + r, fj * kWaveN + 4 * q, s);
    }
  }

  // g: moved to the tile's rows (at most kBM) and the block's first column.
  FP8L_DEV static void run(const MxArgs& g, int KW, uint8_t* smem) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int jw = wave / KW, kw = wave % KW, JW = 8 / KW;
    const P w(g, jw * kWaveN, min<int64_t>(g.N, JW * kWaveN), smem + wave * P::kWave);
    v4f acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const uint32_t pieces = ((uint32_t)g.steps + 1) / 2;
    // one piece on its way while the last is multiplied (two or three cost the
    // registers of other waves: 16 rows of 11008 -> 4096 6.9 us, 7.9, 7.9)
    typename P::Regs t;
    w.load(t, kw);
    for (uint32_t p = kw; p < pieces; p += KW) {
      w.put_w(t);
      v8i b[2];
      uint32_t eb[2];
#pragma unroll
      for (int m = 0; m < MT; m += 2) {
        w.put_x(t, m);
        if (m + 2 >= MT) w.load(t, p + KW);  // past the last: zeros
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (m == 0) b[u] = w.codes(0, u), eb[u] = w.scale(0, u);
#pragma unroll
          for (int i = 0; i < 2 && m + i < MT; ++i)
            acc[m + i] = mma(b[u], w.codes(1 + i, u), acc[m + i], eb[u], w.scale(1 + i, u));
        }
      }
      asm volatile("" ::: "memory");  // before the next piece is put there
    }
    if (KW > 1) __syncthreads();  // the partial sums take the pieces' place
    finish(g, acc, KW, smem);
  }
};

// The skinny kernel for a high-precision X of so few rows that every block
// quantizes them itself, into LDS, while its first pieces of W are on the way:
// one launch instead of two.  The block of the first tile column writes codes
// and scales out.  (Quantizing in the registers of the wave that multiplies
// needs no LDS, but does 16 rows' work for one row: 16.8 us against 13.0 of two
// launches for one token, 4096 -> 11008.)
struct MxFusedX {
  const void* x;     // [M][K]
  int64_t K;
  uint8_t* codes;    // [M][ld]
  uint32_t* scales;  // words [steps][sa_step]
};

template <int IN>
struct MxFused {
  using S = MxSkinny<1>;
  using P = MxPieces<0>;
  static constexpr int kSize = IN == kInF32 ? 4 : 2, kOwn = 8 * P::kWave;
  static_assert(kOwn >= 8 * 1024, "partial sums");
  // LDS: pieces, then partial sums; scale words [steps][rows]; codes [rows][ld]
  static int lds(int rows, int64_t ld, int64_t steps) {
    return kOwn + (int)(((steps * rows * 4 + 15) & ~15LL) + rows * ld);
  }

  // g, fx: moved to the tile's rows (at most 16) and the block's first column.
  FP8L_DEV static void run(const MxArgs& g, const MxFusedX& fx, bool write, int KW, uint8_t* smem) {
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int jw = wave / KW, kw = wave % KW, JW = 8 / KW;
    const int j0 = jw * S::kWaveN, rows = (int)g.M;
    const P w(g, j0, min<int64_t>(g.N, JW * S::kWaveN), smem + wave * P::kWave);
    typename P::Regs t;
    w.load(t, kw);
    uint32_t* const xe = reinterpret_cast<uint32_t*>(smem + kOwn);
    uint8_t* const xc = smem + kOwn + ((g.steps * rows * 4 + 15) & ~15);
    const uint32_t ld = (uint32_t)g.ld, K = (uint32_t)fx.K;
    // 16 lanes a step of 128 values, as in the quantize kernel
    const int sl = threadIdx.x & 15;
    for (int i = threadIdx.x >> 4; i < rows * g.steps; i += 32) {
      const int row = i / g.steps, s = i - row * g.steps;
      const uint32_t k = 128 * s + 8 * sl;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.0f;
      if (k < K) load8<IN>(fx.x, (int64_t)row * K + k, v);
      const MxEight e = mx_eight(v, k < 2 * ld, sl);
      if (k < 2 * ld) {
        *reinterpret_cast<uint32_t*>(xc + row * ld + 64 * s + 4 * sl) = e.codes;
        if (write) *reinterpret_cast<uint32_t*>(fx.codes + (int64_t)row * ld + 64 * s + 4 * sl) = e.codes;
      }
      if (sl == 0) {
        xe[s * rows + row] = e.word;
        if (write) fx.scales[(int64_t)s * g.sa_step + row] = e.word;
      }
    }
    lds_barrier();
    // rows past the last one take its values: their sums are not stored
    const int rr = min(r, rows - 1);
    v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
    const uint32_t pieces = ((uint32_t)g.steps + 1) / 2;
    for (uint32_t p = kw; p < pieces; p += KW) {
      w.put_w(t);
      w.load(t, p + KW);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int s = 2 * p + u;
        if (s >= g.steps) continue;
        const uint32_t k = 64 * s + 16 * q;
        const v4i a = *reinterpret_cast<const v4i*>(xc + rr * ld + (k < ld ? k : 0));
        const v8i fa = {a.x, a.y, a.z, a.w, 0, 0, 0, 0};
        acc = S::mma(w.codes(0, u), fa, acc, w.scale(0, u), xe[s * rows + rr] >> (8 * q));
      }
      asm volatile("" ::: "memory");
    }
    if (KW > 1) __syncthreads();
    const v4f sums[1] = {acc};
    S::finish(g, sums, KW, smem);
  }
};

// Move to the group's tile: rows from tm bm on, columns from tn bn on.
FP8L_DEV void mx_group(MxArgs& g, const MxStrides& st, const GroupSpan& sp, int tm, int bm) {
  g.b += sp.e * st.b;
  g.sb += sp.e * st.sb;
  if (g.bias) g.bias += sp.e * st.bias;
  const int64_t row = sp.start + (int64_t)tm * bm;
  mx_move(g, row, min<int64_t>(sp.end - row, bm), 0);
}

template <int MT>
__global__ __launch_bounds__(512) void mx4_skinny_kernel(MxArgs g, int kw) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem_mx[];
  using S = MxSkinny<MT>;
  const int tm = blockIdx.x / g.tiles_n, tn = blockIdx.x % g.tiles_n;
  const int64_t row = (int64_t)tm * S::kBM;
  mx_move(g, row, min<int64_t>(g.M - row, S::kBM), (int64_t)tn * (8 / kw) * S::kWaveN);
  S::run(g, kw, smem_mx);
}

template <int MT>
__global__ __launch_bounds__(512) void mx4_skinny_groups_kernel(MxArgs g, Groups gr, MxStrides st,
                                                                int kw) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem_mx[];
  using S = MxSkinny<MT>;
  int tm, tn;
  const GroupSpan sp = rows_work(gr, S::kBM, g.tiles_n, tm, tn);
  if (sp.e < 0) return;
  mx_group(g, st, sp, tm, S::kBM);
  mx_move(g, 0, g.M, (int64_t)tn * (8 / kw) * S::kWaveN);
  S::run(g, kw, smem_mx);
}

template <int IN>
__global__ __launch_bounds__(512, 4) void mx4_fused_kernel(MxArgs g, MxFusedX fx, int kw) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem_mx[];
  mx_move(g, 0, g.M, (int64_t)blockIdx.x * (8 / kw) * 16);
  MxFused<IN>::run(g, fx, blockIdx.x == 0, kw, smem_mx);
}

template <int IN>
__global__ __launch_bounds__(512, 4) void mx4_fused_groups_kernel(MxArgs g, MxFusedX fx, Groups gr,
                                                               MxStrides st, int kw) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem_mx[];
  int tm, tn;
  const GroupSpan sp = rows_work(gr, 16, g.tiles_n, tm, tn);
  if (sp.e < 0) return;
  mx_group(g, st, sp, tm, 16);
  const int64_t row = sp.start + 16 * (int64_t)tm;
  fx.x = reinterpret_cast<const uint8_t*>(fx.x) + row * fx.K * MxFused<IN>::kSize;
  fx.codes += row * g.ld;
  fx.scales += row;
  mx_move(g, 0, g.M, (int64_t)tn * (8 / kw) * 16);
  MxFused<IN>::run(g, fx, tn == 0, kw, smem_mx);
}

}  // namespace fp8l
