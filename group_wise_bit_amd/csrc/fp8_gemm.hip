// Product of two block-scaled e4m3 matrices:
//   y[m, n] = sum over kb of sx[kb][m] * sw[n / 128][kb] * P_kb[m, n],
//   P_kb[m, n] = sum over the block's k of x[m, k] * w[n, k],
// with x in 1 x 128 blocks and w in 128 x 128 blocks. One v_mfma_f32_16x16x128_f8f6f4
// forms a 16 x 16 tile of P_kb: its 128 k are exactly one scale block, so the scales
// (float32) enter with one float32 product and fused multiply-add per output and block; in
// tiles of 16-bit outputs, E8M0 scales enter in the instruction itself. The two agree while
// the product of the scales is a normal float32; beyond, the second keeps what the first
// rounds to 0 or infinity.
//
// Precision. The FP8 matrix cores add the products of 8 adjacent k (8 bytes of a lane)
// after dropping bits below 2^-13 of the largest of them (measured: a product 2^-14 times
// its neighbour's vanishes, in another group of 8 it counts down to 2^-23); the sums of
// the groups and the accumulator are float32. What goes depends on how unequal the 8
// products are: of the result's 2-norm 2e-5 on normal data, 3e-5 to 7e-5 with 1 % of the
// channels 20 times larger, 6e-5 to 8e-5 with them 200 times larger; at worst 7 * 2^-13 of
// each group's largest product. Next to the rounding of a bf16 output (1.7e-3) that does not
// show; the error of a float16 one (2.1e-4) grows by 0.5, 1 to 3 and 4 to 7 %. It buys twice
// the rate, so 16-bit outputs take it; who wants float32 sums asks for a float32 output and
// rounds that. For these, EXACT: the codes are widened to bf16 (exactly, the scaled
// FP8 conversion at scale 1) and multiplied by v_mfma_f32_16x16x32_bf16, whose products
// are exact and whose sums are float32.
//
// The weights are the A operand (a lane of the result holds 4 adjacent n of one m). The
// lane's 32 bytes of an operand may hold any 32 of the 128 k as long as x and w agree;
// lane l takes k = 32 (l / 16) .. + 31 of row l % 16 on both sides.
#include <type_traits>

#include "fp8.hpp"

namespace gwb {

typedef int fg_i32x8_t __attribute__((ext_vector_type(8)));
typedef float fg_f32x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void fg_lds_void_t;

// One operand of a 16 x 16 x 128 step: the lane's 32 codes, or the same widened to bf16.
struct Codes {
  U4 a, b;
};
typedef __bf16 fg_bf16x8_t __attribute__((ext_vector_type(8)));
struct Wide {
  fg_bf16x8_t v[4];
};
__device__ __forceinline__ fg_i32x8_t fg_regs(const Codes& c) {
  return fg_i32x8_t{(int)c.a.x, (int)c.a.y, (int)c.a.z, (int)c.a.w, (int)c.b.x, (int)c.b.y, (int)c.b.z, (int)c.b.w};
}
__device__ __forceinline__ fg_bf16x8_t widen8(uint32_t a, uint32_t b) {
  const U4 v{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false)),
             __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true)),
             __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false)),
             __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true))};
  return __builtin_bit_cast(fg_bf16x8_t, v);
}
__device__ __forceinline__ Wide widen(const Codes& c) {
  return Wide{widen8(c.a.x, c.a.y), widen8(c.a.z, c.a.w), widen8(c.b.x, c.b.y), widen8(c.b.z, c.b.w)};
}
// The 16 x 16 products of one block of 128 k.
__device__ __forceinline__ fg_f32x4_t mfma128(const Codes& w, const Codes& x) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fg_regs(w), fg_regs(x), fg_f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0,
                                                          0, 0, 0, 0);   // e4m3 x e4m3, unscaled
}
__device__ __forceinline__ fg_f32x4_t mfma128(const Wide& w, const Wide& x) {
  fg_f32x4_t c{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[i], x.v[i], c, 0, 0, 0);
  return c;
}
// The same added to c, with E8M0 scale bytes: sw of the weight's block, sx of the lane's x row.
__device__ __forceinline__ fg_f32x4_t mfma128_scaled(const Codes& w, const Codes& x, fg_f32x4_t c, int sw, int sx) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fg_regs(w), fg_regs(x), c, 0, 0, 0, sw, 0, sx);
}

// Wait until at most LEFT of this wavefront's memory loads (the LDS fills included) are
// outstanding, then for the whole block.
template <int LEFT>
__device__ __forceinline__ void fg_stage_barrier() {
  static_assert(LEFT < 64, "vmcnt has 6 bits");
  // (not __syncthreads, which waits for every pending fill)
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070 | (LEFT & 15) | (LEFT >> 4) << 14);   // vmcnt(LEFT), lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// E8M0 byte -> 2^(byte - 127), 255 -> NaN.
__device__ __forceinline__ float e8m0_to_f32(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7FC00000u : b << 23);
}
template <bool E8>
__device__ __forceinline__ float load_scale(const void* s, int64_t i) {
  if constexpr (E8) return e8m0_to_f32(static_cast<const uint8_t*>(s)[i]);
  else return static_cast<const float*>(s)[i];
}

// Workgroups go round-robin over the 8 XCDs, each with its own L2: every XCD gets a
// contiguous range of tiles, run in bands of up to 8 row tiles across the column tiles.
__device__ __forceinline__ void fg_tile(int id, int gx, int gy, int& bx, int& by) {
  const int T = gx * gy, xcd = id & 7, rem = T & 7;
  const int t = xcd * (T >> 3) + min(xcd, rem) + (id >> 3);
  const int band = t / (8 * gy), first = band * 8, rows = min(8, gx - first);
  const int r = t - first * gy;
  bx = first + r % rows;
  by = r / rows;
}

// 4 adjacent outputs of row m from column n. vec: rows and the pointer allow one store of
// 4 elements (then N % 4 == 0 too).
template <typename TY>
__device__ __forceinline__ void store4(TY* __restrict__ y, int64_t ldy, int64_t m, int n, int N, fg_f32x4_t v, bool vec) {
  TY* p = y + m * ldy + n;
  if (vec) {
    if (n >= N) return;
    if constexpr (sizeof(TY) == 4) *reinterpret_cast<float4*>(p) = float4{v[0], v[1], v[2], v[3]};
    else if constexpr (__is_same(TY, uint16_t)) *reinterpret_cast<uint2*>(p) = uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    else {
      typedef _Float16 h4_t __attribute__((ext_vector_type(4)));
      *reinterpret_cast<uint2*>(p) = __builtin_bit_cast(uint2, h4_t{(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]});
    }
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n + r < N) p[r] = fp8_narrow<TY>(v[r]);
  }
}

// 16 bytes per lane from base + off + uniform straight to LDS, lane l to p + 16 l. Buffer
// loads: the compiler takes the global form for a flat access, next to which it waits for
// every pending load instead of counting them. (off + uniform is below 2^32: at most 255
// rows of 2^23 bytes and a row.)
using FillSource = __amdgpu_buffer_rsrc_t;
__device__ __forceinline__ FillSource fill_source(const uint8_t* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, 0xFFFFFFFFu, 0x00020000);
}
constexpr int kNonTemporal = 2;   // the load instruction's nt bit
template <bool ONCE = false>
__device__ __forceinline__ void fill16(FillSource base, uint8_t* p, uint32_t off, uint32_t uniform) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(base, (fg_lds_void_t*)p, 16, off, uniform, 0, ONCE ? kNonTemporal : 0);
}

// ---------------------------------------------------------------- tiles
// Block: WM x WN wavefronts, each 16*MT rows of x by 64*NG columns (per 64 columns 4 tiles
// of 16 whose A rows are interleaved so that a lane ends with 16 adjacent columns). K in
// stages of 128 through a ring of D LDS tiles, filled from memory without registers
// (buffer loads to LDS: 8 rows of 128 bytes per instruction). A tile row's 16-byte
// chunk c lies in slot c ^ f, f a function of the row's operand lane i that differs
// between the lanes a read serves together. Rows past M or N load the last row's data and
// are not stored. With K % 128 != 0 the last stage's missing chunks re-read the last valid
// one (no byte outside a row is read) and the x operands are cleared there; what meets the
// zeros is a code of the same output's own row. ONCE: the weight is loaded non-temporally,
// for a single row of tiles (64 x 34816 x 5120: 38 us and 41).
// Stages in flight pay where memory or latency bounds a tile (64 x 34816 x 5120, 64 x 192 tiles:
// 51 us with two, 38 with four; 128 x 34816 x 5120, 128 x 192 tiles: 60 with two, 47 with three).
// E8M0 scales of 16-bit outputs go to the matrix cores themselves (the scaled
// instruction), everything else takes the product of the two scales as one float32 fma
// per output and stage.
//
// Order within a stage (fixed by scheduling barriers; the compiler's own order reads each
// operand right before its use): per column tile u, the next tile's operand is read, then
// u's products run with the scaled additions of tile u - 1 between them. The stage's one
// barrier stands before the last column tile: by then every operand of the stage is in
// registers and the next stage's fills have landed, so the next stage's operands are read
// during that tile's products. 256 x 256 tiles, 4096 x 34816 x 5120: 637 us with E8M0 scales
// (2.29 PFLOP/s), the matrix cores busy 58 % of the cycles, LDS about as long.
__device__ __forceinline__ int fg_swz(int i) { return (i & 7) ^ ((i >> 3) & 1); }
__device__ __forceinline__ int fg_wlane(int row) { return (row & 3) | (((row >> 4) & 3) << 2); }

template <int MT, int NG, int WM, int WN, int D, bool ONCE, bool E8, typename TY>
__global__ __launch_bounds__(64 * WM * WN) void fp8_gemm_kernel(GemmArgs g, int gx, int gy) {
  constexpr bool EXACT = sizeof(TY) == 4, HW = E8 && !EXACT;
  constexpr int NT = 4 * NG, NW = WM * WN, BM = 16 * MT * WM, BN = 64 * NG * WN;
  constexpr int IX = BM / 8 / NW, IW = BN / 8 / NW;   // fill instructions per wavefront
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "whole fills");
  // x tile, w tile, x scales: one object (with two, the compiler waits for every pending
  // fill before each read of LDS)
  constexpr int LX = 0, LW = BM * 128, LS = LW + BN * 128;
  __shared__ __align__(16) uint8_t lds[D][LS + BM * 4];
  const auto slot = [](int kb) { return (unsigned)kb % D; };
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int i = lane & 15, q = lane >> 4;
  int bx, by;
  fg_tile(blockIdx.x, gx, gy, bx, by);
  const int64_t m0 = (int64_t)bx * BM, n0 = (int64_t)by * BN;
  const FillSource xb = fill_source(g.x + m0 * g.ldx), wb = fill_source(g.w + n0 * g.ldw);
  const int mlast = (int)min((int64_t)BM, g.M - m0) - 1, nlast = (int)min((int64_t)BN, g.N - n0) - 1;
  const int KB = (g.K + 127) / 128, nv = (g.K - (KB - 1) * 128) / 16;   // chunks in the last stage
  // this block's stages: all, or one of the K splits
  const int k0 = (int)((int64_t)KB * blockIdx.y / gridDim.y), k1 = (int)((int64_t)KB * (blockIdx.y + 1) / gridDim.y);

  uint32_t xo[IX], wo[IW];
  int xc[IX], wc[IW];
#pragma unroll
  for (int j = 0; j < IX; ++j) {
    const int row = 8 * (j * NW + wv) + (lane >> 3);
    xc[j] = (lane & 7) ^ fg_swz(row & 15);
    xo[j] = (uint32_t)min(row, mlast) * (uint32_t)g.ldx + 16 * xc[j];
  }
#pragma unroll
  for (int j = 0; j < IW; ++j) {
    const int row = 8 * (j * NW + wv) + (lane >> 3);
    wc[j] = (lane & 7) ^ fg_swz(fg_wlane(row));
    wo[j] = (uint32_t)min(row, nlast) * (uint32_t)g.ldw + 16 * wc[j];
  }
  // the j-th of a stage's IX + IW fills
  const auto fill = [&](int kb, int j) {
    uint8_t* l = &lds[slot(kb)][0];
    const int last = kb == KB - 1 ? nv - 1 : 7;
    if (j < IX) {
      const int v = j < IX ? j : 0;
      fill16(xb, l + LX + (j * NW + wv) * 1024, xo[v] - 16 * max(xc[v] - last, 0), kb * 128);
    } else {
      const int v = j - IX < IW ? j - IX : 0;
      fill16<ONCE>(wb, l + LW + (v * NW + wv) * 1024, wo[v] - 16 * max(wc[v] - last, 0), kb * 128);
    }
  };

  const int wm = wv % WM, wn = wv / WM;
  const int64_t mw = m0 + 16 * MT * wm, nw = n0 + 64 * NG * wn;
  // Scales, as float32 or (HW) as the bytes the scaled instruction takes. The x scales of a
  // stage go through LDS: float32 ones of deep rings with the fills, others by a thread per
  // row that loads them two stages ahead and stores them one stage ahead (with D > 2 by
  // every wavefront, to keep branches out of the count of pending loads). The wavefront's
  // columns lie in one row block of the weight (NG = 3: each 64 of them in one); a lane
  // holds that block's scale of stage (kb / 64) * 64 + lane.
  static_assert(NG <= 3, "weight scales: one per wavefront, or one per 64 columns");
  constexpr int SB = NG == 3 ? 3 : 1;
  using Scale = typename std::conditional<HW, int, float>::type;
  const auto scale_at = [&](const void* p, int64_t at) -> Scale {
    if constexpr (HW) return static_cast<const uint8_t*>(p)[at];
    else return load_scale<E8>(p, at);
  };
  static_assert((BM & (BM - 1)) == 0 && BM >= 64 && BM <= 64 * NW, "whole wavefronts of rows");
  constexpr bool DMA = !E8 && D > 2, ALL = D > 2;
  const bool loads_sx = 64 * wv < BM;
  const int row_sx = threadIdx.x & (BM - 1);
  const int64_t msx = min(m0 + row_sx, g.M - 1), nlb = (g.N - 1) / 128;
  Scale sx = 0, sw[SB];
  const auto load_sx = [&](int kb) {
    if (!DMA && (ALL || loads_sx)) sx = scale_at(g.sx, (int64_t)min(kb, k1 - 1) * g.ldsx + msx);
  };
  const auto store_sx = [&](int kb) {
    if (!DMA && (ALL || loads_sx)) reinterpret_cast<Scale*>(&lds[slot(kb)][LS])[row_sx] = sx;
  };
  const auto fill_sx = [&](int kb) {
    if (DMA && loads_sx) {
      const float* src = static_cast<const float*>(g.sx) + (int64_t)kb * g.ldsx + msx;
      __builtin_amdgcn_global_load_lds(src, (fg_lds_void_t*)(&lds[slot(kb)][LS] + wv * 256), 4, 0, 0);
    }
  };
  const auto load_sw = [&](int kb) {
#pragma unroll
    for (int b = 0; b < SB; ++b)
      sw[b] = scale_at(g.sw, min((nw + 64 * b) / 128, nlb) * g.ldsw + min((kb & ~63) + lane, k1 - 1));
#pragma unroll
    for (int b = 0; b < SB; ++b) asm volatile("" : "+v"(sw[b]));   // wait here, once in 64 stages, not at every use
  };
  const auto sw_of = [&](int kb, int b) {
    return __builtin_bit_cast(Scale, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sw[b]), kb & 63));
  };
  const auto block_of = [](int u) { return SB == 1 ? 0 : u >> 2; };
  // operands in LDS
  const int s0 = 16 * ((2 * q) ^ fg_swz(i)), s1 = 16 * ((2 * q + 1) ^ fg_swz(i));
  const int lx = LX + (16 * MT * wm + i) * 128, lw = LW + (64 * NG * wn + 16 * (i >> 2) + (i & 3)) * 128;
  const auto read_x = [&](int kb, int t) {
    const uint8_t* p = &lds[slot(kb)][0] + lx + t * 2048;
    return Codes{ld16(p + s0), ld16(p + s1)};
  };
  const auto read_w = [&](int kb, int u) {
    const uint8_t* p = &lds[slot(kb)][0] + lw + ((u >> 2) * 64 + (u & 3) * 4) * 128;
    return Codes{ld16(p + s0), ld16(p + s1)};
  };
  const auto read_sx = [&](int kb, int t) {
    return reinterpret_cast<const Scale*>(&lds[slot(kb)][LS])[16 * (MT * wm + t) + i];
  };

  fg_f32x4_t acc[NT][MT], p[2][HW ? 1 : MT];
  // this stage's factors of each x tile (HW: its scales), and the last stage's last
  constexpr int CB = HW ? 1 : SB;
  Scale c[CB][MT], cp[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    c[CB - 1][t] = 0;
    if constexpr (!HW) p[1][t] = fg_f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < NT; ++u) acc[u][t] = fg_f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }

  // D = 2: fills go out in two halves, the first after the barrier that frees their buffer
  // (before the last column tile of the stage two before), the second with the next
  // stage's first tile: at 4096 x 34816 x 5120 with E8M0 scales all at once takes 5 % more, in
  // quarters 6 %. D > 2: the fills of stage kb + D - 1 start in stage kb, all of them before
  // its barrier, which leaves the fills of the D - 2 stages after the next in flight.
  constexpr int FILLS = IX + IW, PER = D == 2 ? (FILLS + 1) / 2 : (FILLS + NT - 2) / (NT - 1), AHEAD = (D - 2) * FILLS;
  load_sx(k0);
  load_sw(k0);
#pragma unroll
  for (int j = 0; j < FILLS; ++j) fill(k0, j);
  fill_sx(k0);
  store_sx(k0);
  load_sx(k0 + 1);
  if constexpr (D > 2) {
#pragma unroll
    for (int d = 1; d < D - 1; ++d) {
      if (k0 + d < k1) {
#pragma unroll
        for (int j = 0; j < FILLS; ++j) fill(k0 + d, j);
        fill_sx(k0 + d);
      }
    }
    if (k0 + D - 1 <= k1) fg_stage_barrier<AHEAD>();
    else fg_stage_barrier<0>();
  } else {
    fg_stage_barrier<0>();
    if (k0 + 1 < k1) {
#pragma unroll
      for (int j = 0; j < PER; ++j) fill(k0 + 1, j);
      fill_sx(k0 + 1);
    }
  }
  Codes xr[MT], wr[2];
#pragma unroll
  for (int t = 0; t < MT; ++t) xr[t] = read_x(k0, t);
  wr[0] = read_w(k0, 0);

  // LEFT: 0 for the last stage, 2 while fills go on, else 1
  const auto stage = [&](int kb, auto left) {
    constexpr int LEFT = decltype(left)::value;
    if ((kb & 63) == 0 && kb > k0) load_sw(kb);
    Scale w[SB];
#pragma unroll
    for (int b = 0; b < SB; ++b) w[b] = sw_of(kb, b);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      cp[t] = c[CB - 1][t];
      const Scale s = read_sx(kb, t);
#pragma unroll
      for (int b = 0; b < CB; ++b) c[b][t] = HW ? s : s * w[b];
    }
    if constexpr (LEFT > 0) store_sx(kb + 1);
    if constexpr (LEFT > 0) load_sx(kb + 2);
    if constexpr (LEFT == 0) {
      const int left = kb == KB - 1 ? nv : 8;       // x chunks past K count as zeros
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        if (2 * q >= left) xr[t].a = U4{0, 0, 0, 0};
        if (2 * q + 1 >= left) xr[t].b = U4{0, 0, 0, 0};
      }
    }
    Wide xw[EXACT ? MT : 1];
    if constexpr (EXACT) {
#pragma unroll
      for (int t = 0; t < MT; ++t) xw[t] = widen(xr[t]);
    }
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      if (u < NT - 1) {
        wr[(u + 1) & 1] = read_w(kb, u + 1);
      } else if (LEFT > 0) {
        fg_stage_barrier<LEFT == 2 ? AHEAD : 0>();
        wr[0] = read_w(kb + 1, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
      Wide ww;
      if constexpr (EXACT) ww = widen(wr[u & 1]);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        if constexpr (HW) {
          acc[u][t] = mfma128_scaled(wr[u & 1], xr[t], acc[u][t], w[block_of(u)], c[0][t]);
        } else {
          if constexpr (EXACT) p[u & 1][t] = mfma128(ww, xw[t]);
          else p[u & 1][t] = mfma128(wr[u & 1], xr[t]);
          const int v = u > 0 ? u - 1 : NT - 1;
          const float s = u > 0 ? c[block_of(v)][t] : cp[t];
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[v][t][r] = __builtin_fmaf(p[(u + 1) & 1][t][r], s, acc[v][t][r]);
        }
        if (LEFT > 0 && u == NT - 1) xr[t] = read_x(kb + 1, t);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (u == (D == 2 ? NT - 1 : 0) && LEFT == 2) fill_sx(D == 2 ? kb + 2 : kb + D - 1);
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        if constexpr (D == 2) {
          const int f = u == NT - 1 ? j : (u + 1) * PER + j;
          if (f < FILLS && LEFT > (u == NT - 1 ? 1 : 0)) fill(u == NT - 1 ? kb + 2 : kb + 1, f);
        } else {
          if (u < NT - 1 && u * PER + j < FILLS && LEFT == 2) fill(kb + D - 1, u * PER + j);
        }
      }
    }
  };
  constexpr int DRAIN = D == 2 ? 2 : D - 1;
  int kb = k0;
  for (; kb + DRAIN < k1; ++kb) stage(kb, std::integral_constant<int, 2>{});
  for (; kb + 1 < k1; ++kb) stage(kb, std::integral_constant<int, 1>{});
  stage(kb, std::integral_constant<int, 0>{});
  if constexpr (!HW) {
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[NT - 1][t][r] = __builtin_fmaf(p[1][t][r], c[CB - 1][t], acc[NT - 1][t][r]);
  }
  // Nothing of the products may move into the branch below: its lanes past M are off, and a
  // matrix instruction reads its operands from every lane.
#pragma unroll
  for (int u = 0; u < NT; ++u)
#pragma unroll
    for (int t = 0; t < MT; ++t) asm volatile("" : "+v"(acc[u][t]));
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int64_t m = mw + 16 * t + i;
    if (m >= g.M) continue;
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      const int n = (int)(nw + 64 * (u >> 2) + 16 * q + 4 * (u & 3));
      if (gridDim.y > 1) store4(g.part + (int64_t)blockIdx.y * g.M * g.N, g.N, m, n, (int)g.N, acc[u][t], g.N % 4 == 0);
      else store4((TY*)g.y, g.ldy, m, n, (int)g.N, acc[u][t], g.vec);
    }
  }
}

// y = the splits' sums added in order. V outputs per thread: 4 adjacent ones where the
// partial rows and y allow it.
template <int V, typename TY>
__global__ __launch_bounds__(256) void fp8_gemm_sum_kernel(const float* __restrict__ part, int S, int64_t M, int64_t N,
                                                           TY* __restrict__ y, int64_t ldy) {
  const int64_t per = N / V, v = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (v >= M * per) return;
  const int64_t m = v / per, n = (v - m * per) * V;
  fg_f32x4_t sum{0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = 0; s < S; ++s) {
    const float* p = part + ((int64_t)s * M + m) * N + n;
    if constexpr (V == 4) sum += *reinterpret_cast<const fg_f32x4_t*>(p);
    else sum[0] += *p;
  }
  if constexpr (V == 4) store4(y, ldy, m, (int)n, (int)N, sum, true);
  else y[m * ldy + n] = fp8_narrow<TY>(sum[0]);
}

// ---------------------------------------------------------------- few rows
// The weight's bytes bound a product with few rows of x. A block owns 16*NT columns and
// its NW wavefronts split K into bands; a wavefront streams its band through a ring of D
// stages in its own part of LDS (global_load_lds_dwordx4: whole 128-byte lines, D - 1
// stages in flight without registers, and no barrier, since it alone writes and reads
// them). XI fills of 8 rows bring x, 2*NT the weight. The products of the two scales of up
// to kPiece stages are formed beforehand. The bands' float32 sums are added through LDS in
// wavefront order. 1 x 5120 x 17408 18 us (4.9 TB/s), 12 x 34816 x 5120 32 us (5.5 TB/s),
// 1 x 4096 x 14336 11 us (5.2 TB/s).
constexpr int kPiece = 16;
template <int MT, int XI, int NT, int NW, int D, bool E8, typename TY>
__global__ __launch_bounds__(64 * NW) void fp8_gemm_rows_kernel(GemmArgs g) {
  constexpr bool EXACT = sizeof(TY) == 4;
  constexpr int BN = 16 * NT, BM = 16 * MT, PITCH = BN + 4, OPS = 2 * NT + XI;
  constexpr int STAGE = OPS * 1024, TABLE = kPiece * BM * 4, WAVE = D * STAGE + TABLE;
  static_assert(XI == 2 * MT || (MT == 1 && XI == 1), "8 or 16*MT rows of x");
  static_assert(BM * PITCH * 4 <= WAVE && D * OPS < 64, "sums fit the ring, fills fit the counter");
  __shared__ __align__(16) uint8_t lds[NW * WAVE];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int i = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * BN, nb = n0 / 128;   // BN divides 128: one row block
  const int KB = (g.K + 127) / 128, nv = (g.K - (KB - 1) * 128) / 16;
  const int k0 = (int)((int64_t)KB * wv / NW), k1 = (int)((int64_t)KB * (wv + 1) / NW);
  uint8_t* ring = lds + wv * WAVE;
  float* table = reinterpret_cast<float*>(ring + D * STAGE);

  // Row 8f + lane / 8 of fill f: x rows, then the weight's rows, each tile's row of operand
  // lane r at 16 u + r (column 4 NT (r / 4) + 4 u + r % 4, so a lane's results are adjacent).
  const uint8_t* src[OPS];
  const int chunk = (lane & 7) ^ fg_swz(lane >> 3), chunk8 = (lane & 7) ^ fg_swz(8 + (lane >> 3));
#pragma unroll
  for (int f = 0; f < OPS; ++f) {
    const int row = 8 * (f < XI ? f : f - XI) + (lane >> 3), u = row >> 4, r = row & 15;
    src[f] = f < XI ? g.x + min((int64_t)row, g.M - 1) * g.ldx
                    : g.w + min(n0 + 4 * NT * (r >> 2) + 4 * u + (r & 3), g.N - 1) * g.ldw;
  }
  const auto fill = [&](int kb, int slot) {
    const int last = kb == KB - 1 ? nv - 1 : 7;   // missing chunks re-read the last valid one
    const int64_t c0 = (int64_t)kb * 128 + 16 * min(chunk, last), c1 = (int64_t)kb * 128 + 16 * min(chunk8, last);
#pragma unroll
    for (int f = 0; f < OPS; ++f) {
      const uint8_t* p = src[f] + (((f < XI ? f : f - XI) & 1) ? c1 : c0);
      // the weight is read once: non-temporal
      if (f < XI) __builtin_amdgcn_global_load_lds(p, (fg_lds_void_t*)(ring + slot * STAGE + f * 1024), 16, 0, 0);
      else __builtin_amdgcn_global_load_lds(p, (fg_lds_void_t*)(ring + slot * STAGE + f * 1024), 16, 0, kNonTemporal);
    }
  };

  fg_f32x4_t acc[NT][MT];
#pragma unroll
  for (int u = 0; u < NT; ++u)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[u][t] = fg_f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int s0 = 16 * ((2 * q) ^ fg_swz(i)), s1 = 16 * ((2 * q + 1) ^ fg_swz(i));
  const int ix = XI == 1 ? (i & 7) : i;           // 8 rows loaded: columns 8.. of the tile repeat them, unstored
  const int sx0 = XI == 1 ? 16 * ((2 * q) ^ fg_swz(ix)) : s0, sx1 = XI == 1 ? 16 * ((2 * q + 1) ^ fg_swz(ix)) : s1;

  const auto compute = [&](int kb, int slot, int at) {
    const uint8_t* l = ring + slot * STAGE;
    Codes w[NT], x[MT];
    float c[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      x[t] = Codes{ld16(l + (16 * t + ix) * 128 + sx0), ld16(l + (16 * t + ix) * 128 + sx1)};
      c[t] = table[at * BM + 16 * t + i];
    }
#pragma unroll
    for (int u = 0; u < NT; ++u)
      w[u] = Codes{ld16(l + (8 * XI + 16 * u + i) * 128 + s0), ld16(l + (8 * XI + 16 * u + i) * 128 + s1)};
    const int left = kb == KB - 1 ? nv : 8;         // x chunks past K count as zeros
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      if (2 * q >= left) x[t].a = U4{0, 0, 0, 0};
      if (2 * q + 1 >= left) x[t].b = U4{0, 0, 0, 0};
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        fg_f32x4_t p;
        if constexpr (EXACT) p = mfma128(widen(w[u]), widen(x[t]));
        else p = mfma128(w[u], x[t]);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[u][t][r] = __builtin_fmaf(p[r], c[t], acc[u][t][r]);
      }
    }
  };

  for (int p0 = k0; p0 < k1; p0 += kPiece) {
    const int pe = min(p0 + kPiece, k1), n = pe - p0;
    float c[kPiece * BM / 64];
#pragma unroll
    for (int v = 0; v < kPiece * BM / 64; ++v) {
      const int kb = p0 + min((64 * v + lane) / BM, n - 1);
      const int64_t m = min((int64_t)((64 * v + lane) % BM), g.M - 1);
      if (64 * v < n * BM) c[v] = load_scale<E8>(g.sx, (int64_t)kb * g.ldsx + m) * load_scale<E8>(g.sw, nb * g.ldsw + kb);
    }
    for (int d = 0; d < D - 1 && d < n; ++d) fill(p0 + d, d);
#pragma unroll
    for (int v = 0; v < kPiece * BM / 64; ++v)
      if (64 * v < n * BM) table[64 * v + lane] = c[v];
    int slot = 0, next = D - 1;
    for (int kb = p0; kb < pe; ++kb) {
      if (kb + D - 1 < pe) {
        fill(kb + D - 1, next);
        __builtin_amdgcn_s_waitcnt(0x0F70 | ((D - 1) * OPS & 15) | ((D - 1) * OPS >> 4) << 14);
      } else {
        __builtin_amdgcn_s_waitcnt(0x0F70);       // the last D - 1 stages
      }
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      compute(kb, slot, kb - p0);
      // this stage's reads are done before the next fill takes its slot: the products used them
      __builtin_amdgcn_sched_barrier(0);
      slot = slot + 1 == D ? 0 : slot + 1;
      next = next + 1 == D ? 0 : next + 1;
    }
  }

  float* part = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int u = 0; u < NT; ++u)
      *reinterpret_cast<fg_f32x4_t*>(part + (16 * t + i) * PITCH + 4 * NT * q + 4 * u) = acc[u][t];
  __syncthreads();
  for (int v = threadIdx.x; v < BM * BN; v += 64 * NW) {
    const int m = v / BN, n = v % BN;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) sum += reinterpret_cast<const float*>(lds + w * WAVE)[m * PITCH + n];
    if (m < g.M && n0 + n < g.N) ((TY*)g.y)[m * g.ldy + n0 + n] = fp8_narrow<TY>(sum);
  }
}

template <int MT, int XI, int NT, int NW, int D, bool E8, typename TY>
static void rows_gemm_launch(const GemmArgs& g, hipStream_t st) {
  hipLaunchKernelGGL((fp8_gemm_rows_kernel<MT, XI, NT, NW, D, E8, TY>), dim3((unsigned)((g.N + 16 * NT - 1) / (16 * NT))),
                     dim3(64 * NW), 0, st, g);
}

// ---------------------------------------------------------------- launch
template <int MT, int NG, int WM, int WN, int D, bool ONCE, bool E8, typename TY>
static void tile_launch(const GemmArgs& g, int splits, hipStream_t st) {
  constexpr int BM = 16 * MT * WM, BN = 64 * NG * WN;
  const int gx = (int)((g.M + BM - 1) / BM), gy = (int)((g.N + BN - 1) / BN);
  hipLaunchKernelGGL((fp8_gemm_kernel<MT, NG, WM, WN, D, ONCE, E8, TY>), dim3((unsigned)(gx * gy), (unsigned)splits),
                     dim3(64 * WM * WN), 0, st, g, gx, gy);
  if (splits > 1) {
    const bool vec = g.vec && g.N % 4 == 0;
    const dim3 grid((unsigned)((g.M * (g.N / (vec ? 4 : 1)) + 255) / 256));
    if (vec) hipLaunchKernelGGL((fp8_gemm_sum_kernel<4, TY>), grid, dim3(256), 0, st, g.part, splits, g.M, g.N, (TY*)g.y, g.ldy);
    else hipLaunchKernelGGL((fp8_gemm_sum_kernel<1, TY>), grid, dim3(256), 0, st, g.part, splits, g.M, g.N, (TY*)g.y, g.ldy);
  }
}

template <bool E8, typename TY>
static void gemm_launch(const GemmArgs& g, const GemmPlan& p, hipStream_t st) {
  constexpr bool EXACT = sizeof(TY) == 4;   // widened operands take twice the registers: no 256 x 256 tiles
  switch (p.kernel) {
    case kRows8: return rows_gemm_launch<1, 1, 2, 4, 2, E8, TY>(g, st);
    case kRows8Deep: return rows_gemm_launch<1, 1, 2, 8, 2, E8, TY>(g, st);
    case kRows8Narrow: return rows_gemm_launch<1, 1, 1, 8, 2, E8, TY>(g, st);
    case kRows16: return rows_gemm_launch<1, 2, 2, 4, 2, E8, TY>(g, st);
    case kRows16Deep: return rows_gemm_launch<1, 2, 2, 8, 2, E8, TY>(g, st);
    case kRows16Narrow: return rows_gemm_launch<1, 2, 1, 8, 2, E8, TY>(g, st);
    case kRows32: return rows_gemm_launch<2, 4, 2, 4, 2, E8, TY>(g, st);
    case kRows32Deep: return rows_gemm_launch<2, 4, 2, 8, 2, E8, TY>(g, st);
    case kRows32Narrow: return rows_gemm_launch<2, 4, 1, 8, 2, E8, TY>(g, st);
    case kTile64: return tile_launch<1, 1, 4, 1, 4, false, E8, TY>(g, p.splits, st);
    case kTile64x128:
      if constexpr (!EXACT) tile_launch<1, 2, 4, 1, 4, true, E8, TY>(g, 1, st);
      return;
    case kTile64x192:
      if constexpr (!EXACT) tile_launch<1, 3, 4, 1, 4, true, E8, TY>(g, 1, st);
      return;
    case kTile128:
      // EXACT: 4 wavefronts of 64 x 64 widen fewer codes, which bounds it, than 8 of 32 x 64
      // (512 x 34816 x 5120: 217 us and 289)
      if constexpr (EXACT) return tile_launch<4, 1, 2, 2, 2, false, E8, TY>(g, p.splits, st);
      else return tile_launch<2, 1, 4, 2, 2, false, E8, TY>(g, p.splits, st);
    case kTile128Deep: return tile_launch<2, 1, 4, 2, 4, false, E8, TY>(g, p.splits, st);
    case kTile128x192:
      if constexpr (!EXACT) tile_launch<1, 3, 8, 1, 3, false, E8, TY>(g, 1, st);
      return;
    case kTile256x192:
      if constexpr (!EXACT) tile_launch<2, 3, 8, 1, 2, false, E8, TY>(g, 1, st);
      return;
    case kTile256:
      if constexpr (!EXACT) {
        const int64_t n = p.wide;   // the rest to 128 x 128 tiles
        GemmArgs a = g;
        a.N = n;
        tile_launch<4, 2, 4, 2, 2, false, E8, TY>(a, 1, st);
        if (n < g.N) {
          a.N = g.N - n;
          a.w += n * g.ldw;
          a.sw = (const char*)g.sw + n / 128 * g.ldsw * (E8 ? 1 : 4);
          a.y = (TY*)g.y + n;
          tile_launch<2, 1, 4, 2, 4, false, E8, TY>(a, 1, st);
        }
      }
  }
}

void launch_fp8_gemm(const GemmArgs& g, bool e8m0, int32_t y_dtype, hipStream_t st) {
  const GemmPlan p = fp8_gemm_plan(g.M, g.N, g.K, y_dtype == 0);
  if (y_dtype == 0) e8m0 ? gemm_launch<true, float>(g, p, st) : gemm_launch<false, float>(g, p, st);
  else if (y_dtype == 1) e8m0 ? gemm_launch<true, uint16_t>(g, p, st) : gemm_launch<false, uint16_t>(g, p, st);
  else e8m0 ? gemm_launch<true, _Float16>(g, p, st) : gemm_launch<false, _Float16>(g, p, st);
}

}  // namespace gwb
