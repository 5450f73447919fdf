// GEMM for few rows (decoding): C[i, j] = sum_k A(i, k) B(j, k), at most
// 16 MT rows of A per tile, FP8 or 8-bit integers, both operands
// k-contiguous; scales, bias and rounding as in the other GEMM kernels.
//
// With a handful of rows the matrix pipes idle and the time is that of
// reading B once from HBM.  So there is no LDS staging and no barrier in the
// K loop: every wave reads its own 16 rows of B straight into MFMA
// operand registers, many 16-byte loads in flight, and A (small, in L2) the
// same way.  The MFMA does not care which K position sits in which lane as
// long as A and B agree, so a lane takes bytes [16 q, 16 q + 16) and
// [64 + 16 q, 64 + 16 q + 16) of a 128-byte piece of K (q = lane / 16): each
// load instruction covers 64 contiguous bytes of 16 rows and two of them
// whole 128-byte lines.
//
// A block has 8 waves.  KW of them share a tile column and split K (pieces
// of 128 bytes dealt round-robin, so that together they read whole rows),
// 8 / KW tile columns stand beside each other.  KW is chosen so that the
// waves fill the chip: 1 when there are columns enough, up to 8 for a narrow
// B.  The KW partial sums meet in LDS and are added in wave order (int32:
// exactly), so results do not depend on timing.
//
// Measured: 24 rows over 19 of 64 experts of 1536 -> 6912 (202 MB of weights
// and outputs) 43 us, 4.7 TB/s, against 71 us on 128x128 tiles; 16 rows over 13
// of 16 experts of 4096 -> 11008 in integers 103 us, 5.7 TB/s, against 122;
// one row of 4096 -> 11008 (45 MB) 12.6 us, where start-up and the two
// memory round trips of a wave weigh as much as the bandwidth.  Four pieces
// in flight per wave beat eight (128 registers keep two blocks on a CU: 43
// against 53 us).
#pragma once

#include "fp8l_gemm3.hpp"
#include "fp8l_grouped.hpp"
#include "fp8l_i8.hpp"

namespace fp8l {

// K pieces of 128 bytes loaded at once: as many as the 128 registers of two
// blocks per CU hold (64 integer rows of any alignment still spill 13, in
// groups 6).
template <int MT, bool I8, bool ANY>
constexpr int skinny_unroll() { return MT == 1 ? 4 : ((MT == 4 || ANY) && (I8 || (ANY && MT == 4)) ? 1 : 2); }

// ANY: rows of any alignment and sizes of any kind, through load16_any.
template <int FA, int FB, int MT, bool ANY = false>
struct Skinny {
  static constexpr int kBM = 16 * MT, kWaveN = 16, kThreads = 512, kLds = 8 * MT * 1024;
  static constexpr bool I8 = FA == kI8;
  static constexpr int kU = skinny_unroll<MT, I8, ANY>();

  // Scales and bias of this lane's four outputs of a 16x16 fragment (row
  // `row`, columns j .. j + 3) as loaded: nothing is computed from them
  // before the store, so nothing waits for them while the operands load.
  struct Epi {
    float sa, sb[4];
    uint16_t b[4];
  };
  FP8L_DEV static Epi epi(const GemmArgs& g, int row, int64_t j) {
    Epi e = epi_cols(g, j);
    e.sa = g.scale_a[I8 && row < g.Mc ? row : 0];
    return e;
  }
  FP8L_DEV static Epi epi_cols(const GemmArgs& g, int64_t j) {
    Epi e;
    e.sa = 1.0f;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      // Nc a multiple of 8: all four columns or none
      const int64_t jt = j + (ANY ? t : 0) < g.Nc ? j + t : t * !ANY;
      e.sb[t] = g.scale_b[I8 ? jt : 0];
      e.b[t] = g.bias_kind != kBiasNone ? reinterpret_cast<const uint16_t*>(g.bias)[jt] : 0;
    }
    return e;
  }
  FP8L_DEV static void store(const GemmArgs& g, int row, int64_t j, v4f acc, const Epi& e) {
    if (row >= g.Mc || j >= g.Nc) return;
    const float isa = 1.0f / e.sa;
    float v[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const float c = isa * (1.0f / e.sb[t]);
      const float b = I8 && g.out_f16 ? f16_to_f32(e.b[t]) : bf16_to_f32(e.b[t]);
      v[t] = I8 ? i8_value(acc[t], c, b) : __builtin_fmaf(acc[t], c, b);
    }
    uint2 w;
    if (I8 && g.out_f16)
      w = make_uint2(f32_to_f16(v[0]) | (f32_to_f16(v[1]) << 16),
                     f32_to_f16(v[2]) | (f32_to_f16(v[3]) << 16));
    else
      w = make_uint2(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]));
    uint16_t* const dst = g.c + row * g.ldc + j;
    if (!ANY || (g.c_vec && j + 4 <= g.Nc)) {  // Nc a multiple of 8: all four columns or none
      *reinterpret_cast<uint2*>(dst) = w;
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (j + t < g.Nc) dst[t] = (uint16_t)((t < 2 ? w.x : w.y) >> (16 * (t & 1)));
    }
  }

  // ANY: bytes [k, k + 16) of row i of p, zeros past K and the rows: the
  // first byte (the operand's where none is valid) and their number.
  FP8L_DEV static const uint8_t* where(const uint8_t* p, int64_t ld, int64_t i, int64_t rows,
                                       int64_t k, int64_t K, int& n) {
    const bool ok = i < rows && k < K;
    n = ok ? (int)min<int64_t>(16, K - k) : 0;
    return ok ? p + i * ld + k : p;
  }
  // One operand's F fragments of the pieces at k[0 .. 2 kU): all loads in
  // flight together, unless some lane's words reach past the operand's end.
  template <int F>
  FP8L_DEV static void load_any(const uint8_t* p, int64_t ld, int64_t i0, int64_t rows, int64_t K,
                                const int64_t (&k)[2 * kU], v8i (&out)[kU][F]) {
    const uint8_t* const end = p + (rows - 1) * ld + K;
    bool ok = true;
    int n;
#pragma unroll
    for (int h = 0; h < 2 * kU; ++h)
#pragma unroll
      for (int f = 0; f < F; ++f)
        ok = ok && any_window(where(p, ld, i0 + 16 * f, rows, k[h], K, n), end);
    uint4 v[2 * kU][F];
    if (__all(ok)) {
      uint32_t e[2 * kU][F];
#pragma unroll
      for (int h = 0; h < 2 * kU; ++h)
#pragma unroll
        for (int f = 0; f < F; ++f)
          load_words(where(p, ld, i0 + 16 * f, rows, k[h], K, n), v[h][f], e[h][f]);
#pragma unroll
      for (int h = 0; h < 2 * kU; ++h)
#pragma unroll
        for (int f = 0; f < F; ++f) {
          const uint8_t* const a = where(p, ld, i0 + 16 * f, rows, k[h], K, n);
          v[h][f] = join16(v[h][f], e[h][f], a, n);
        }
    } else {
#pragma unroll
      for (int h = 0; h < 2 * kU; ++h)
#pragma unroll
        for (int f = 0; f < F; ++f) {
          const uint8_t* const a = where(p, ld, i0 + 16 * f, rows, k[h], K, n);
          v[h][f] = n ? load16_any(a, n) : make_uint4(0, 0, 0, 0);
        }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const uint4 a = v[2 * u][f], b = v[2 * u + 1][f];
        out[u][f] = v8i{(int)a.x, (int)a.y, (int)a.z, (int)a.w,
                        (int)b.x, (int)b.y, (int)b.z, (int)b.w};
      }
  }

  FP8L_DEV static v8i load2(__amdgpu_buffer_rsrc_t rs, uint32_t lo, uint32_t hi) {
    const v4i a = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rs, lo, 0, 0));
    const v4i b = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rs, hi, 0, 0));
    return v8i{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  }

  // Tile column tn (of 16 * 8 / KW columns) of the rows g.a .. (g.Mc of them).
  FP8L_DEV static void run(const GemmArgs& g, int tn, int KW, uint8_t* smem) {
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int jw = wave / KW, kw = wave % KW, JW = 8 / KW;
    const int64_t jb = (int64_t)tn * JW * kWaveN;  // the block's first column
    const int64_t j0 = jb + jw * kWaveN;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(g.a, (uint32_t)(g.Mc * g.lda));
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(g.b, (uint32_t)(g.Nc * g.ldb));
    // row offsets; rows past the end lie past the buffer and read as zeros
    uint32_t oa[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) oa[m] = (uint32_t)((16 * m + r) * g.lda);
    const uint32_t ob = (uint32_t)((j0 + r) * g.ldb);
    v4f acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    // the epilogue's operands, in flight with the first pieces (with KW > 1
    // another wave may finish the fragment; it then finds them in cache)
    Epi e0 = epi(g, r, j0 + 4 * q);
    const uint32_t K = (uint32_t)g.Kc;
    const uint32_t pieces = (K + 127) / 128;
    for (uint32_t p = kw; p < pieces; p += KW * kU) {
      v8i fa[kU][MT], fb[kU][1];
      if constexpr (ANY) {
        int64_t k[2 * kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          k[2 * u] = (int64_t)(p + u * KW) * 128 + 16 * q;
          k[2 * u + 1] = k[2 * u] + 64;
        }
        load_any<1>(g.b, g.ldb, j0 + r, g.Nc, g.Kc, k, fb);
        load_any<MT>(g.a, g.lda, r, g.Mc, g.Kc, k, fa);
      } else {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const uint32_t k0 = (p + u * KW) * 128 + 16 * q, k1 = k0 + 64;
          // bytes past K (the next row's) and pieces past the last: zeros
          fb[u][0] = load2(rb, k0 < K ? ob + k0 : 0x80000000u, k1 < K ? ob + k1 : 0x80000000u);
#pragma unroll
          for (int m = 0; m < MT; ++m)
            fa[u][m] = load2(ra, k0 < K ? oa[m] + k0 : 0x80000000u, k1 < K ? oa[m] + k1 : 0x80000000u);
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m] = mma_16x16<FA, FB>(fb[u][0], fa[u][m], acc[m]);
    }
    if (KW == 1) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (m > 0) e0 = epi(g, 16 * m + r, j0 + 4 * q);
        store(g, 16 * m + r, j0 + 4 * q, acc[m], e0);
      }
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
        for (int t = 0; t < 4; ++t) s[t] = add_sums<I8>(s[t], o[t]);
      }
      const int row = 16 * fm + r;
      const int64_t j = jb + fj * kWaveN + 4 * q;
      store(g, row, j, s, epi(g, row, j));
    }
  }
};

// The skinny kernel for integer layers whose high-precision X has so few rows
// that every block quantizes them itself (fp8l_i8.hpp gives the rule and the
// arithmetic): one launch instead of two.  The block's first pieces of B are
// in flight meanwhile.  The codes stay in LDS, from where the K loop reads
// them; the block of the first tile column writes codes and scales out.
struct FusedX {
  const void* x;  // row 0 of the tile
  int8_t* q;
  float* scale;
};

template <int IN>
struct SkinnyFused {
  static constexpr int kBM = 16, kWaveN = 16, kThreads = 512, kU = 4;
  static constexpr bool I8 = true;
  using S = Skinny<kI8, kI8, 1>;
  static constexpr int kPart = S::kLds;         // partial sums
  static constexpr int kHead = kPart + 16 * 8 * 4 + 16 * 4;  // + amax per row and wave, + scales
  // LDS for rows of K codes
  static int lds(int rows, int64_t K) { return (int)(((kHead + 15) & ~15) + rows * K); }

  FP8L_DEV static void run(const GemmArgs& g, const FusedX& fx, bool write, int tn, int KW,
                           uint8_t* smem) {
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int jw = wave / KW, kw = wave % KW, JW = 8 / KW;
    const int64_t jb = (int64_t)tn * JW * kWaveN, j0 = jb + jw * kWaveN;
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(g.b, (uint32_t)(g.Nc * g.ldb));
    const uint32_t ob = (uint32_t)((j0 + r) * g.ldb);
    const uint32_t K = (uint32_t)g.Kc, pieces = (K + 127) / 128;
    const int rows = (int)g.Mc;
    uint32_t* const red = reinterpret_cast<uint32_t*>(smem + kPart);  // [row][wave of the row]
    float* const sc = reinterpret_cast<float*>(smem + kPart + 16 * 8 * 4);
    uint8_t* const xs = smem + ((kHead + 15) & ~15);
    auto load_b = [&](uint32_t p, v8i (&fb)[kU]) {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const uint32_t k0 = (p + u * KW) * 128 + 16 * q, k1 = k0 + 64;
        fb[u] = S::load2(rb, k0 < K ? ob + k0 : 0x80000000u, k1 < K ? ob + k1 : 0x80000000u);
      }
    };
    v8i fb[kU];
    load_b(kw, fb);
    typename S::Epi e0 = S::epi_cols(g, j0 + 4 * q);

    // amax: wpr waves share a row (8, 4, 2 or 1 for 1, 2, up to 4, more rows)
    const int wpr = rows == 1 ? 8 : (rows == 2 ? 4 : (rows <= 4 ? 2 : 1));
    const int sub = wave % wpr;
    for (int i = wave / wpr; i < rows; i += 8 / wpr) {
      uint32_t mx = 0;
      for (uint32_t c = 8 * (64 * sub + lane); c < K; c += 512 * wpr) {
        float v[8];
        load8<IN>(fx.x, (int64_t)i * K + c, v);
#pragma unroll
        for (int t = 0; t < 8; ++t) mx = max(mx, absbits(v[t]));
      }
      mx = wave_max_u32(mx);
      if (lane == 0) red[i * 8 + sub] = mx;
    }
    __syncthreads();
    for (int i = wave / wpr; i < rows; i += 8 / wpr) {
      uint32_t mx = 0;
      for (int w = 0; w < wpr; ++w) mx = max(mx, red[i * 8 + w]);
      const float s = row_scale(mx);
      const bool ok = mx <= 0x7f7fffffu;
      if (sub == 0 && lane == 0) {
        sc[i] = s;
        if (write) fx.scale[i] = s;
      }
      for (uint32_t c = 8 * (64 * sub + lane); c < K; c += 512 * wpr) {
        float v[8];
        load8<IN>(fx.x, (int64_t)i * K + c, v);
        const uint2 w = make_uint2(i8x4(v, s, ok), i8x4(v + 4, s, ok));
        *reinterpret_cast<uint2*>(xs + i * K + c) = w;
        if (write) *reinterpret_cast<uint2*>(fx.q + (int64_t)i * K + c) = w;
      }
    }
    __syncthreads();

    v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (uint32_t p = kw; p < pieces; p += KW * kU) {
      if (p != (uint32_t)kw) load_b(p, fb);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const uint32_t k0 = (p + u * KW) * 128 + 16 * q, k1 = k0 + 64;
        v4i a = {0, 0, 0, 0}, b = a;
        if (r < rows && k0 < K) a = *reinterpret_cast<const v4i*>(xs + r * K + k0);
        if (r < rows && k1 < K) b = *reinterpret_cast<const v4i*>(xs + r * K + k1);
        acc = mma_16x16<kI8, kI8>(fb[u], v8i{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}, acc);
      }
    }
    if (KW == 1) {
      e0.sa = sc[r < rows ? r : 0];
      S::store(g, r, j0 + 4 * q, acc, e0);
      return;
    }
    v4f* const part = reinterpret_cast<v4f*>(smem);
    part[wave * 64 + lane] = acc;
    __syncthreads();
    if (wave < JW) {
      const v4f* src = part + wave * KW * 64 + lane;
      v4f s = src[0];
      for (int w = 1; w < KW; ++w) {
        const v4f o = src[w * 64];
#pragma unroll
        for (int t = 0; t < 4; ++t) s[t] = add_sums<true>(s[t], o[t]);
      }
      const int64_t j = jb + wave * kWaveN + 4 * q;
      typename S::Epi e = S::epi_cols(g, j);
      e.sa = sc[r < rows ? r : 0];
      S::store(g, r, j, s, e);
    }
  }
};

template <int IN>
__global__ __launch_bounds__(512, 4) void skinny_fused_kernel(GemmArgs g, FusedX fx, int KW) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem_skinny[];
  SkinnyFused<IN>::run(g, fx, blockIdx.x == 0, blockIdx.x, KW, smem_skinny);
}

template <int IN>
__global__ __launch_bounds__(512, 4) void skinny_fused_groups_kernel(GemmArgs g, Groups gr,
                                                                     GroupStrides st, FusedX fx,
                                                                     int KW) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem_skinny[];
  int tm, tn;
  const GroupSpan sp = rows_work(gr, 16, g.tiles_n, tm, tn);
  if (sp.e < 0) return;
  const int64_t row = sp.start + 16 * (int64_t)tm;
  move_to_rows<true>(g, st, sp, tm, 16);
  constexpr int eb = IN == kInF32 ? 4 : 2;
  fx.x = reinterpret_cast<const uint8_t*>(fx.x) + row * g.Kc * eb;
  fx.q += row * g.Kc;
  fx.scale += row;
  SkinnyFused<IN>::run(g, fx, tn == 0, tn, KW, smem_skinny);
}

// Dense: block = (tile column, tile row); consecutive blocks take the tile
// rows of one column first, so a B with several tile rows is reread from L2.
template <class S>
__global__ __launch_bounds__(512, 4) void skinny_kernel(GemmArgs g, int KW) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem_skinny[];
  const int tm = blockIdx.x % g.tiles_m, tn = blockIdx.x / g.tiles_m;
  const int64_t row = (int64_t)tm * S::kBM;
  g.a += row * g.lda;
  g.c += row * g.ldc;
  g.Mc = min<int64_t>(g.Mc - row, S::kBM);
  if (S::I8) g.scale_a += row;
  S::run(g, tn, KW, smem_skinny);
}

// Groups: as grouped_rows_kernel, in units of 16 MT rows.
template <class S>
__global__ __launch_bounds__(512, 4) void skinny_groups_kernel(GemmArgs g, Groups gr, GroupStrides st,
                                                            GroupedSide side, int KW) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem_skinny[];
  int tm, tn;
  const GroupSpan sp = rows_work(gr, S::kBM, g.tiles_n, tm, tn);
  if (sp.e >= 0) {
    move_to_rows<S::I8>(g, st, sp, tm, S::kBM);
    S::run(g, tn, KW, smem_skinny);
  }
  grouped_side(side);
}

}  // namespace fp8l
