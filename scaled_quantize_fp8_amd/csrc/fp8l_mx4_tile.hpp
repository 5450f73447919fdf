// Tiles of the 4-bit product for many rows: 256x256 (eight waves) and
// 128x256 (four waves, two blocks per CU), each wave 128 rows by 64 columns.
//
// The schedule is the 8-bit tiles' (fp8l_gemm4.hpp, fp8l_gemm6.hpp): operands
// go by DMA into a ring of LDS stages of 64 bytes of K per row (128 values
// here), fragments of the next step are read while the current one's MFMAs
// run, A fragments single-buffered, B fragments double-buffered, here in two
// asm blocks a step instead of five (8192 x 8192 x 8192: 287 us against 289 to
// 294).  A 32x32x64
// MFMA takes 16 bytes of codes per lane, so a lane's 32 bytes of a step feed
// two: its low half (block 2 h of the step, h = lane / 32) and its high half
// (block 2 h + 1), each with that block's scale.  Which blocks meet in which
// instruction does not matter as long as both operands agree.  Per step a wave
// issues 16 MFMAs of 8 passes: the LDS traffic per matrix cycle is that of the
// 8-bit tiles.
//
// What bounds it: 8192 x 8192 x 8192 runs at 3.8 P/s (the vendor library's
// product 3.05), matrix cores busy 52% of the cycles at 1.7 GHz, the clock that
// the power limit leaves for these operands; with zeros for operands the same
// kernel takes 240 us at 2.4.  Tried, no faster with real operands: 16x16x128
// MFMAs (alone 8.5 P/s where these reach 6.5), four waves of 128x128 with a
// third less LDS traffic (305 us), the stages' loads dealt to other waves at
// other times (313).
//
// Scales travel with the codes: a step's 4-byte words of the tile's rows and
// columns (one DMA load of 64 words per wave, more for 128x256) lie behind the
// codes of the stage, and a lane reads the two bytes of its blocks as one
// 16-bit word, the first for the low half, the second for the high half.
#pragma once

#include "fp8l_mx4.hpp"

namespace fp8l {

// MFMAs of one asm block: accumulator, B and A fragments and their scales.
struct MxSlot {
  v16f* c;
  const v8i* b;
  const v8i* x;
  const uint32_t* sb;
  const uint32_t* sx;
};

#define FP8L_XL(i)                                                                        \
  "v_mfma_scale_f32_32x32x64_f8f6f4 %[c" #i "], %[b" #i "], %[x" #i "], %[c" #i "], %[t" #i \
  "], %[u" #i "] op_sel_hi:[0,0,0] cbsz:4 blgp:4\n\t"
#define FP8L_XH(i)                                                                        \
  "v_mfma_scale_f32_32x32x64_f8f6f4 %[c" #i "], %[d" #i "], %[y" #i "], %[c" #i "], %[t" #i \
  "], %[u" #i "] op_sel:[1,1,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4\n\t"
#define FP8L_XM4                                                                          \
  FP8L_XL(0) FP8L_XL(1) FP8L_XL(2) FP8L_XL(3) FP8L_XH(0) FP8L_XH(1) FP8L_XH(2) FP8L_XH(3)
#define FP8L_XI(i)                                                              \
  [b##i] "v"(lo4(*m[i].b)), [d##i] "v"(hi4(*m[i].b)), [x##i] "v"(lo4(*m[i].x)), \
      [y##i] "v"(hi4(*m[i].x)), [t##i] "v"(*m[i].sb), [u##i] "v"(*m[i].sx)
#define FP8L_XI4 FP8L_XI(0), FP8L_XI(1), FP8L_XI(2), FP8L_XI(3)

FP8L_DEV void mx_mfma_only(const MxSlot (&m)[4]) {
  // s_nop 1: operands may have just been written by VALU
  asm volatile("s_nop 1\n\t" FP8L_XM4 "" : FP8L_CO4 : FP8L_XI4);
}

// A fragments f and f + 1 of the next step at offset OFF (their scales at SOFF)
// and, WITH_B, its B fragments, read while the four fragment products m run.
FP8L_DEV v8i join8(v4i a, v4i b) { return v8i{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}; }
template <int OFF, int SOFF>
FP8L_DEV void mx_read_a(const uint32_t (&a)[2], uint32_t sa, v8i* n, uint32_t* e,
                        const MxSlot (&m)[4]) {
  v4i r0, r1, r2, r3;
  uint32_t e0, e1;
  asm volatile(FP8L_RKC(r0, a0, o0) FP8L_RKC(r1, a1, o0) FP8L_RKC(r2, a0, o1) FP8L_RKC(r3, a1, o1)
               "ds_read_u16 %[e0], %[sa] offset:%[s0]\n\t"
               "ds_read_u16 %[e1], %[sa] offset:%[s1]\n\t" FP8L_XM4 "s_waitcnt lgkmcnt(0)"
               : [r0] "=&v"(r0), [r1] "=&v"(r1), [r2] "=&v"(r2), [r3] "=&v"(r3), [e0] "=&v"(e0),
                 [e1] "=&v"(e1), FP8L_CO4
               : [a0] "v"(a[0]), [a1] "v"(a[1]), [sa] "v"(sa), [o0] "n"(OFF), [o1] "n"(OFF + 2048),
                 [s0] "n"(SOFF), [s1] "n"(SOFF + 128), FP8L_XI4
               : "memory");
  n[0] = join8(r0, r1), n[1] = join8(r2, r3), e[0] = e0, e[1] = e1;
}
FP8L_DEV void mx_read_ab(const uint32_t (&a)[2], uint32_t sa, const uint32_t (&b)[2], uint32_t sb,
                         v8i* na, uint32_t* ea, v8i* nb, uint32_t* eb, const MxSlot (&m)[4]) {
  v4i r0, r1, r2, r3, r4, r5, r6, r7;
  uint32_t e0, e1, e2, e3;
  asm volatile(
      "ds_read_b128 %[r0], %[a0]\n\tds_read_b128 %[r1], %[a1]\n\t"
      "ds_read_b128 %[r4], %[p0]\n\tds_read_b128 %[r5], %[p1]\n\t"
      "ds_read_b128 %[r2], %[a0] offset:2048\n\tds_read_b128 %[r3], %[a1] offset:2048\n\t"
      "ds_read_b128 %[r6], %[p0] offset:2048\n\tds_read_b128 %[r7], %[p1] offset:2048\n\t"
      "ds_read_u16 %[e0], %[sa]\n\tds_read_u16 %[e1], %[sa] offset:128\n\t"
      "ds_read_u16 %[e2], %[sb]\n\tds_read_u16 %[e3], %[sb] offset:128\n\t" FP8L_XM4
      "s_waitcnt lgkmcnt(0)"
      : [r0] "=&v"(r0), [r1] "=&v"(r1), [r2] "=&v"(r2), [r3] "=&v"(r3), [r4] "=&v"(r4),
        [r5] "=&v"(r5), [r6] "=&v"(r6), [r7] "=&v"(r7), [e0] "=&v"(e0), [e1] "=&v"(e1),
        [e2] "=&v"(e2), [e3] "=&v"(e3), FP8L_CO4
      : [a0] "v"(a[0]), [a1] "v"(a[1]), [p0] "v"(b[0]), [p1] "v"(b[1]), [sa] "v"(sa), [sb] "v"(sb),
        FP8L_XI4
      : "memory");
  na[0] = join8(r0, r1), na[1] = join8(r2, r3), ea[0] = e0, ea[1] = e1;
  nb[0] = join8(r4, r5), nb[1] = join8(r6, r7), eb[0] = e2, eb[1] = e3;
}

template <int WGM>
struct MxTile {
  static constexpr int WGN = 4, NW = WGM * WGN;
  static constexpr int kBM = 128 * WGM, kBN = 256, kThreads = 64 * NW;
  static constexpr int kBlocks = WGM == 2 ? 1 : 2;   // per CU (LDS)
  static constexpr int kStages = WGM == 2 ? 4 : 3;
  using OA = Op3<kKContig, kBM, NW>;
  using OB = Op3<kKContig, kBN, NW>;
  // scale words of a step: the tile's rows, then its columns, fetched 64 per
  // DMA load, every wave the same number of loads (surplus ones fetch zeros)
  static constexpr int kScaleLoads = ((kBM + kBN) / 64 + NW - 1) / NW;
  static constexpr int kScaleBytes = kScaleLoads * NW * 256;
  static constexpr int kCodes = OA::kBytes + OB::kBytes;
  static constexpr int kStep = kCodes + kScaleBytes;
  static constexpr int kDma = OA::kPerWave + OB::kPerWave + kScaleLoads;
  static constexpr int RS = kBN * 2 + 16;  // staged output row
  static constexpr int kBiasOff = kStages * kStep > kBM * RS ? kStages * kStep : kBM * RS;
  static constexpr int kLds = kBiasOff + kBN * 2;
  static_assert(kBlocks * kLds <= 160 * 1024, "LDS");

  // g: moved to the tile's rows (at most kBM) and columns.
  FP8L_DEV static void run(const MxArgs& g, uint8_t* smem) {
    constexpr int FM = 4, FN = 2;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(wave);
    const int rows = (int)min<int64_t>(g.M, kBM), cols = (int)min<int64_t>(g.N, kBN);
    const uint32_t a_bytes = (uint32_t)(rows * g.ld), b_bytes = (uint32_t)(cols * g.ld);
    OA oa;
    OB ob;
    oa.init(g.ld, 0, rows, g.ld);
    ob.init(g.ld, 0, cols, g.ld);
    const int ra0 = wave / WGN * 128, rb0 = wave % WGN * 64;
    FragBase<OA, FM> fra;
    FragBase<OB, FN> frb;
    fra.init(smem, ra0);
    frb.init(smem + OA::kBytes, rb0);
    const uint32_t sbase = lds_off(smem) + kCodes + 4 * (lane & 31) + 2 * (lane >> 5);
    const uint32_t sra = sbase + 4 * ra0, srb = sbase + 4 * (kBM + rb0);
    v16f acc[FM][FN];
#pragma unroll
    for (int a = 0; a < FM; ++a)
#pragma unroll
      for (int b = 0; b < FN; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[a][b][e] = 0.0f;

    // nk K steps (padded to even); steps 0 .. nk are loaded, those past K
    // being all zeros
    const int nk = (g.steps + 1) & ~1;
    auto step_buf = [&](int kt) { return smem + (kt % kStages) * kStep; };
    auto scale_load = [&](int kt, auto i_tag) {
      const int c = wv * kScaleLoads + decltype(i_tag)::value;  // 64 words
      const bool row = c < kBM / 64;
      const int first = 64 * (row ? c : c - kBM / 64);
      const int n = row ? rows : cols;
      const uint32_t* p = row ? g.sa + kt * g.sa_step : g.sb + kt * g.sb_step;
      const uint32_t bytes =
          kt < g.steps && c < (kBM + kBN) / 64 ? (uint32_t)(4 * n) : 0u;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          mx_rsrc(p, bytes),
          (__attribute__((address_space(3))) void*)(step_buf(kt) + kCodes + 256 * c), 4,
          4u * (first + lane), 0, 0, 0);
    };
    auto issue_step = [&](int kt) {
      const __amdgpu_buffer_rsrc_t ra_k = oa.step_rsrc(g.a, a_bytes, kt);
      const __amdgpu_buffer_rsrc_t rb_k = ob.step_rsrc(g.b, b_bytes, kt);
      static_for<OA::kPerWave>([&](auto i) {
        oa.template issue_step<decltype(i)::value>(ra_k, step_buf(kt), kt, wv);
      });
      static_for<OB::kPerWave>([&](auto i) {
        ob.template issue_step<decltype(i)::value>(rb_k, step_buf(kt) + OA::kBytes, kt, wv);
      });
      static_for<kScaleLoads>([&](auto i) { scale_load(kt, i); });
    };

    v8i fa[FM], fb[2][FN];
    uint32_t ea[FM], eb[2][FN];
    auto slot = [&](int a, int b, int buf) {
      return MxSlot{&acc[a][b], &fb[buf][b], &fa[a], &eb[buf][b], &ea[a]};
    };
    // the columns' bias, in words, behind the ring: older than every stage, so
    // the waits below cover it (kept out of the epilogue, where every tile would
    // wait for it: 8200 rows through 16 experts of 1536 -> 6912 113 us, so 103)
    const bool staged = g.bias && ((uintptr_t)g.bias & 3) == 0 && (cols & 1) == 0;
    if (staged && wv < 2)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          mx_rsrc(g.bias, 2 * cols),
          (__attribute__((address_space(3))) void*)(smem + kBiasOff + 256 * wv), 4,
          256u * wv + 4u * lane, 0, 0, 0);
    for (int s = 0; s < kStages && s <= nk; ++s) issue_step(s);
    if (nk > 0) {
      // nk >= 2: the steps after the first may still be in flight
      const int later = min(kStages - 1, nk);
      if (later >= 3) wait_vm<3 * kDma>();
      else wait_vm<2 * kDma>();
      barrier_only();
#pragma unroll
      for (int f = 0; f < FM; f += 2) OA::read2(step_buf(0), ra0 + 32 * f, fa[f], fa[f + 1]);
      OB::read2(step_buf(0) + OA::kBytes, rb0, fb[0][0], fb[0][1]);
      asm volatile(
          "ds_read_u16 %0, %6\n\t"
          "ds_read_u16 %1, %6 offset:128\n\t"
          "ds_read_u16 %2, %6 offset:256\n\t"
          "ds_read_u16 %3, %6 offset:384\n\t"
          "ds_read_u16 %4, %7\n\t"
          "ds_read_u16 %5, %7 offset:128\n\t"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(ea[0]), "=&v"(ea[1]), "=&v"(ea[2]), "=&v"(ea[3]), "=&v"(eb[0][0]), "=&v"(eb[0][1])
          : "v"(sra), "v"(srb)
          : "memory");
      const MxSlot m[4] = {slot(0, 0, 0), slot(0, 1, 0), slot(1, 0, 0), slot(1, 1, 0)};
      mx_mfma_only(m);
    }

    // Step kt: on entry the products of A fragments 0 and 1 of step kt are issued;
    // fa, ea hold step kt's A fragments, fb[CUR], eb[CUR] its B fragments.
    const __amdgpu_buffer_rsrc_t ra_all = mx_rsrc(g.a, a_bytes);
    const __amdgpu_buffer_rsrc_t rb_all = mx_rsrc(g.b, b_bytes);
    auto kstep_body = [&](int kt, auto cur_tag, auto fast_tag) {
      constexpr int CUR = decltype(cur_tag)::value, NXT = CUR ^ 1;
      constexpr bool FAST = decltype(fast_tag)::value;
      if constexpr (FAST) {
        wait_vm<(kStages - 2) * kDma>();
      } else {
        // step kt+1 landed: later steps may be in flight
        const int later = min(kStages - 2, nk - kt - 1);
        if (later >= 2) wait_vm<2 * kDma>();
        else if (later == 1) wait_vm<kDma>();
        else wait_vm<0>();
      }
      barrier_only();  // step kt+1 visible to all; step kt's buffer is free
      const bool refill = FAST || kt + kStages <= nk;
      const int kf = kt + kStages;
      uint8_t* const sf = step_buf(kf);
      auto load = [&](auto j_tag) {
        constexpr int j = decltype(j_tag)::value;
        if constexpr (j >= OA::kPerWave + OB::kPerWave) {
          if (refill) scale_load(kf, std::integral_constant<int, j - OA::kPerWave - OB::kPerWave>{});
        } else if constexpr (FAST) {
          if constexpr (j < OA::kPerWave)
            oa.template issue_full<j>(ra_all, sf, (uint32_t)kf * oa.kstep, wv);
          else
            ob.template issue_full<j - OA::kPerWave>(rb_all, sf + OA::kBytes,
                                                     (uint32_t)kf * ob.kstep, wv);
        } else if (refill) {
          const __amdgpu_buffer_rsrc_t ra_k = oa.step_rsrc(g.a, a_bytes, kf);
          const __amdgpu_buffer_rsrc_t rb_k = ob.step_rsrc(g.b, b_bytes, kf);
          if constexpr (j < OA::kPerWave)
            oa.template issue_step<j>(ra_k, sf, kf, wv);
          else
            ob.template issue_step<j - OA::kPerWave>(rb_k, sf + OA::kBytes, kf, wv);
        }
      };
      const uint32_t d = (uint32_t)(((kt + 1) % kStages) * kStep);
      const uint32_t a0[2] = {fra.a[0] + d, fra.a[1] + d}, b0[2] = {frb.a[0] + d, frb.a[1] + d};
      constexpr int kHalf = (kDma + 1) / 2;
      {  // A 0 and 1, B <- step kt+1; products of A 2 and 3
        const MxSlot m[4] = {slot(2, 0, CUR), slot(2, 1, CUR), slot(3, 0, CUR), slot(3, 1, CUR)};
        mx_read_ab(a0, sra + d, b0, srb + d, &fa[0], &ea[0], fb[NXT], eb[NXT], m);
      }
      static_for<kHalf>(load);
      {  // A 2 and 3 <- step kt+1; products of A 0 and 1 of step kt+1
        const MxSlot m[4] = {slot(0, 0, NXT), slot(0, 1, NXT), slot(1, 0, NXT), slot(1, 1, NXT)};
        mx_read_a<4096, 256>(a0, sra + d, &fa[2], &ea[2], m);
      }
      static_for<kDma - kHalf>([&](auto j) {
        load(std::integral_constant<int, kHalf + decltype(j)::value>{});
      });
    };
    // steps whose refill (step kt + kStages) ends at or before K; an even count
    const int nf = (int)(g.ld / kBK3);
    const int kfast = max(0, min(nk, nf - kStages)) & ~1;
    int kt = 0;
    for (; kt < kfast; kt += 2) {
      kstep_body(kt, std::integral_constant<int, 0>{}, std::true_type{});
      kstep_body(kt + 1, std::integral_constant<int, 1>{}, std::true_type{});
    }
    for (; kt < nk; kt += 2) {
      kstep_body(kt, std::integral_constant<int, 0>{}, std::false_type{});
      kstep_body(kt + 1, std::integral_constant<int, 1>{}, std::false_type{});
    }
    wait_vm<0>();  // the DMA of step nk (zeros) must not land in the staging area (nk 0: the bias)

    // Epilogue: bias, one rounding, staged through LDS (rows padded by 16
    // bytes) and stored as whole rows.
    mfma_drain();
    barrier_only();
#pragma unroll
    for (int b = 0; b < FN; ++b) {
#pragma unroll
      for (int grp = 0; grp < 4; ++grp) {
        const int jl = rb0 + 32 * b + 8 * grp + 4 * (lane >> 5);
        float bias[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          bias[t] = 0.0f;
          if (staged)
            bias[t] = mx_half(g, reinterpret_cast<const uint16_t*>(smem + kBiasOff)[jl + t]);
          else if (g.bias && jl + t < cols)
            bias[t] = mx_half(g, g.bias[jl + t]);
        }
#pragma unroll
        for (int a = 0; a < FM; ++a) {
          const int il = ra0 + 32 * a + (lane & 31);
          float v[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) v[t] = acc[a][b][4 * grp + t] + bias[t];
          *reinterpret_cast<uint2*>(smem + il * RS + jl * 2) = mx_pack4(g, v);
        }
      }
    }
    lds_barrier();
    if (g.c_vec) {
      constexpr int kChunks = kBN / 8;
#pragma unroll 4
      for (int q = tid; q < kBM * kChunks; q += kThreads) {
        const int r = q / kChunks, ch = q % kChunks;
        if (r < rows && 8 * ch < cols)
          __builtin_nontemporal_store(*reinterpret_cast<const v4u*>(smem + r * RS + ch * 16),
                                      reinterpret_cast<v4u*>(g.c + r * g.ldc + 8 * ch));
      }
    } else {
      for (int q = tid; q < kBM * kBN; q += kThreads) {
        const int r = q / kBN, c = q % kBN;
        if (r < rows && c < cols)
          g.c[r * g.ldc + c] = *reinterpret_cast<const uint16_t*>(smem + r * RS + c * 2);
      }
    }
  }
};

template <int WGM>
__global__ __launch_bounds__(MxTile<WGM>::kThreads, MxTile<WGM>::kBlocks) void mx4_tile_kernel(
    MxArgs g) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem_mx[];
  int tm, tn;
  tile_coords_xcd(blockIdx.x, g.tiles_m, g.tiles_n, tm, tn);
  const int64_t row = (int64_t)tm * MxTile<WGM>::kBM;
  mx_move(g, row, g.M - row, (int64_t)tn * MxTile<WGM>::kBN);
  MxTile<WGM>::run(g, smem_mx);
}

template <int WGM>
__global__ __launch_bounds__(MxTile<WGM>::kThreads, MxTile<WGM>::kBlocks) void
mx4_tile_groups_kernel(MxArgs g, Groups gr, MxStrides st) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem_mx[];
  int tm, tn;
  const GroupSpan sp = rows_work(gr, MxTile<WGM>::kBM, g.tiles_n, tm, tn);
  if (sp.e < 0) return;
  mx_group(g, st, sp, tm, MxTile<WGM>::kBM);
  mx_move(g, 0, g.M, (int64_t)tn * MxTile<WGM>::kBN);
  MxTile<WGM>::run(g, smem_mx);
}

}  // namespace fp8l
