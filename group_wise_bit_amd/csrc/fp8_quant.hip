// Quantization to e4m3 with block scales: rows (1 x 128 blocks), rows of
// SiLU(gate) * up, weights (128 x 128 blocks), and the root-mean-square norm with the
// residual's addition in front of it. Scales and codes as fp8.hpp states them.
#include "fp8.hpp"

namespace gwb {

// ---------------------------------------------------------------- rows
// Tile: 16 rows x 512 columns (4 blocks of 128), one workgroup. A wavefront takes R rows,
// 1 KB (16-bit types) of one row per load instruction, all loads before any use; 16 lanes
// hold a block, so its maximum is four DPP steps. Row scales lie [column block][row], so
// the tile's 4 x 16 scales go through LDS and leave as runs of 16 rows. SILU: the value is
// SiLU(gate) * up, up `K` columns after gate.
// Reads and writes every element once: HBM bound for many rows (SILU 2048 x 17408, 179 MB,
// 33 us, 5.4 TB/s; rows 8192 x 4096, 101 MB, 18.5 us, 5.4 TB/s), latency for few. R = 4
// keeps more loads in flight per wavefront, R = 1 has a quarter of the dependent work in
// one. R = 1 up to kRowSpread tiles (R = 4 -> R = 1: SILU 5 x 17408, 34 tiles, 5.0 -> 3.4 us;
// 256 x 17408, 544 tiles, 8.5 -> 7.5; rows 1024 x 4096, 512 tiles, 4.2 -> 3.9; but
// 2048 x 4096, 1024 tiles, 5.6 -> 6.1).
constexpr int kRowTile = 16, kRowSpread = 768;
template <typename T, bool ALIGNED, bool SILU, int R>
__global__ __launch_bounds__(64 * kRowTile / R) void fp8_rows_kernel(
    const T* __restrict__ x, int64_t ldx, int M, int K, uint8_t* __restrict__ codes, int64_t ldc,
    void* __restrict__ scales, int64_t lds, bool e8m0, int tiles_k) {
  __shared__ float ss[4][kRowTile];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int tk = blockIdx.x % tiles_k;
  const int64_t m0 = (int64_t)(blockIdx.x / tiles_k) * kRowTile;
  const int k = tk * 512 + lane * 8, n = min(max(K - k, 0), 8);
  float v[R][8], u[SILU ? R : 1][8];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t m = m0 + R * wv + i;
    const T* p = x + m * ldx + k;
    const int nr = m < M ? n : 0;
    fp8_load8<ALIGNED>(p, nr, v[i]);
    if constexpr (SILU) fp8_load8<ALIGNED>(p + K, nr, u[i]);
  }
  if (!ALIGNED && n < 8) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t m = m0 + R * wv + i;
      const T* p = x + m * ldx + k;
      const int nr = m < M ? n : 0;
      fp8_load_rest<ALIGNED>(p, nr, v[i]);
      if constexpr (SILU) fp8_load_rest<ALIGNED>(p + K, nr, u[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t m = m0 + R * wv + i;
    if constexpr (SILU) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = silu(v[i][j]) * u[i][j];
    }
    const BlockScale b = block_scale(lanes_max<16>(absmax8(v[i])), e8m0);
    fp8_store_codes8<ALIGNED>(codes + m * ldc + k, m < M ? n : 0, v[i], b.r);
    if ((lane & 15) == 0) ss[lane >> 4][R * wv + i] = b.s;
  }
  __syncthreads();
  const int t = threadIdx.x, kb = tk * 4 + (t >> 4);
  const int64_t m = m0 + (t & 15);
  if (t < 64 && kb * 128 < K && m < M) store_scale(scales, (int64_t)kb * lds + m, ss[t >> 4][t & 15], e8m0);
}

template <typename T, bool ALIGNED, bool SILU>
static void rows_launch(const void* x, int64_t ldx, int64_t M, int64_t K, const Fp8Out& o, hipStream_t st) {
  const int tiles_k = (int)((K + 511) / 512);
  const int64_t tiles = (M + kRowTile - 1) / kRowTile * tiles_k;
  const dim3 grid((unsigned)tiles);
  if (tiles <= kRowSpread)
    hipLaunchKernelGGL((fp8_rows_kernel<T, ALIGNED, SILU, 1>), grid, dim3(64 * kRowTile), 0, st, (const T*)x, ldx,
                       (int)M, (int)K, o.codes, o.ld, o.scales, o.ld_scales, o.e8m0, tiles_k);
  else
    hipLaunchKernelGGL((fp8_rows_kernel<T, ALIGNED, SILU, 4>), grid, dim3(16 * kRowTile), 0, st, (const T*)x, ldx,
                       (int)M, (int)K, o.codes, o.ld, o.scales, o.ld_scales, o.e8m0, tiles_k);
}

template <typename T>
static void rows_launch(bool silu, const void* x, int64_t ldx, int64_t M, int64_t K, const Fp8Out& o, bool aligned,
                        hipStream_t st) {
  if (silu) aligned ? rows_launch<T, true, true>(x, ldx, M, K, o, st) : rows_launch<T, false, true>(x, ldx, M, K, o, st);
  else aligned ? rows_launch<T, true, false>(x, ldx, M, K, o, st) : rows_launch<T, false, false>(x, ldx, M, K, o, st);
}

void launch_fp8_rows(int32_t dtype, bool silu, const void* x, int64_t ldx, int64_t M, int64_t K, const Fp8Out& o,
                     bool aligned, hipStream_t st) {
  if (dtype == 0) rows_launch<float>(silu, x, ldx, M, K, o, aligned, st);
  else if (dtype == 1) rows_launch<uint16_t>(silu, x, ldx, M, K, o, aligned, st);
  else rows_launch<_Float16>(silu, x, ldx, M, K, o, aligned, st);
}

// ---------------------------------------------------------------- weights
// One 128 x 128 block per 256-thread workgroup: 16 lanes span the 128 columns, 16 rows
// per pass, 8 passes held in registers (8 independent loads per lane), so the weight is
// read once. HBM bound: 34816 x 5120 from bfloat16 (535 MB) 95 us, 5.6 TB/s.
template <typename T, bool ALIGNED>
__global__ __launch_bounds__(256) void fp8_blocks_kernel(const T* __restrict__ w, int64_t ldw, int N, int K,
                                                         uint8_t* __restrict__ codes, int64_t ldc,
                                                         void* __restrict__ scales, int64_t lds, bool e8m0,
                                                         int blocks_k) {
  __shared__ float sm[4];
  const int kb = blockIdx.x % blocks_k, nb = blockIdx.x / blocks_k;
  const int k = kb * 128 + (threadIdx.x & 15) * 8, n = min(max(K - k, 0), 8);
  const int64_t r0 = (int64_t)nb * 128 + (threadIdx.x >> 4);
  float v[8][8], amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    fp8_load8<ALIGNED>(w + r * ldw + k, r < N ? n : 0, v[i]);
  }
  if (!ALIGNED && n < 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = r0 + 16 * i;
      fp8_load_rest<ALIGNED>(w + r * ldw + k, r < N ? n : 0, v[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, absmax8(v[i]));
  amax = wave_max_f32(amax);
  if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = amax;
  __syncthreads();
  const BlockScale b = block_scale(fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3])), e8m0);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    fp8_store_codes8<ALIGNED>(codes + r * ldc + k, r < N ? n : 0, v[i], b.r);
  }
  if (threadIdx.x == 0) store_scale(scales, (int64_t)nb * lds + kb, b.s, e8m0);
}

template <typename T>
static void blocks_launch(const void* w, int64_t ldw, int64_t N, int64_t K, const Fp8Out& o, bool aligned,
                          hipStream_t st) {
  const int bk = (int)((K + 127) / 128);
  const dim3 grid((unsigned)((N + 127) / 128 * bk));
  if (aligned)
    hipLaunchKernelGGL((fp8_blocks_kernel<T, true>), grid, dim3(256), 0, st, (const T*)w, ldw, (int)N, (int)K, o.codes,
                       o.ld, o.scales, o.ld_scales, o.e8m0, bk);
  else
    hipLaunchKernelGGL((fp8_blocks_kernel<T, false>), grid, dim3(256), 0, st, (const T*)w, ldw, (int)N, (int)K,
                       o.codes, o.ld, o.scales, o.ld_scales, o.e8m0, bk);
}

void launch_fp8_blocks(int32_t dtype, const void* w, int64_t ldw, int64_t N, int64_t K, const Fp8Out& o, bool aligned,
                       hipStream_t st) {
  if (dtype == 0) blocks_launch<float>(w, ldw, N, K, o, aligned, st);
  else if (dtype == 1) blocks_launch<uint16_t>(w, ldw, N, K, o, aligned, st);
  else blocks_launch<_Float16>(w, ldw, N, K, o, aligned, st);
}

// ---------------------------------------------------------------- norm
// WPR wavefronts take a row and hold it in registers between the two passes the norm needs
// (the sum of squares, then the scaled values), so the row is read once; a workgroup holds
// as many rows as its wavefronts allow. h = x + residual is one float32 addition rounded
// to the row's type, and the norm is that of the rounded h, which is what a later reader
// of the residual stream sees. A lane takes U units of 8 columns; 16 lanes hold a block of
// 128. residual_out may be x or residual: each lane reads its elements before it writes
// them. HBM bound for many rows, latency for few. Measured at 8192 x 5120 (295 MB): a row
// per workgroup with U = 1 68 us; U = 3 on 4 wavefronts 61; the residual stored
// non-temporally, where it is too large to wait for its reader in the cache, 55 (5.4 TB/s).
// float32 rows leave as two half-lines per lane: ordinary stores, which L2 joins, are
// faster there (2048 x 5120 30 us against 34). Runs of 32 workgroups go to one XCD, so that
// its L2 joins the neighbouring rows' 4-byte scales into lines (8192 x 2048: 24.4 -> 23.3 us).
// 7 and 8 units per lane (beyond 49152 columns) do not fit the 128 registers that 1024 threads
// leave a lane where rows are unaligned (up to 81 spilled) or, with 8, float32 (49): 256 x 65535
// takes 60 us, 256 x 65536 29.
constexpr int64_t kNormStream = 32 << 20;   // bytes of residual beyond which it is streamed
template <typename T, bool ALIGNED, int U>
__global__ __launch_bounds__(1024) void rmsnorm_fp8_kernel(NormArgs a, int wpr, bool stream) {
  __shared__ float sw[16];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int sub = wv % wpr, rows = (int)(blockDim.x >> 6) / wpr;
  const unsigned id = blockIdx.x, bid = gridDim.x % 256 ? id : (id & ~255u) + ((id & 7) << 5) + ((id & 255) >> 3);
  const int64_t row = (int64_t)bid * rows + wv / wpr, m = min(row, a.M - 1);   // past M: the last row, unstored
  const bool live = row < a.M;
  const int k0 = (sub * 64 + lane) * 8, step = wpr * 512;
  const T* x = (const T*)a.x + m * a.ldx;
  float h[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int k = k0 + u * step;
    fp8_load8<ALIGNED>(x + k, min(max(a.K - k, 0), 8), h[u]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) fp8_load_rest<ALIGNED>(x + k0 + u * step, a.K - k0 - u * step, h[u]);
  if (a.residual) {
    const T* r = (const T*)a.residual + m * a.ldr;
    float rv[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * step;
      fp8_load8<ALIGNED>(r + k, min(max(a.K - k, 0), 8), rv[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) fp8_load_rest<ALIGNED>(r + k0 + u * step, a.K - k0 - u * step, rv[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * step;
#pragma unroll
      for (int j = 0; j < 8; ++j) h[u][j] = fp8_widen(fp8_narrow<T>(h[u][j] + rv[u][j]));
      if (a.residual_out && live)
        fp8_store8<ALIGNED>((T*)a.residual_out + m * a.ldro + k, min(max(a.K - k, 0), 8), h[u], stream);
    }
  }
  float sum = 0.0f;
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(h[u][j], h[u][j], sum);
  sum = wave_sum_f32(sum);
  if (wpr > 1) {
    if (lane == 0) sw[wv] = sum;
    __syncthreads();
    sum = 0.0f;
    for (int w = 0; w < wpr; ++w) sum += sw[wv - sub + w];
  }
  const float rstd = 1.0f / sqrtf(sum / (float)a.K + a.eps);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int k = k0 + u * step, n = min(max(a.K - k, 0), 8);
    float g[8];
    if (!a.gain) {
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = 1.0f;
    } else if (a.gain_f32) {
      fp8_load8<ALIGNED, false>((const float*)a.gain + k, n, g);
      fp8_load_rest<ALIGNED>((const float*)a.gain + k, n, g);
    } else {
      fp8_load8<ALIGNED, false>((const T*)a.gain + k, n, g);
      fp8_load_rest<ALIGNED>((const T*)a.gain + k, n, g);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = h[u][j] * rstd * g[j];
    if (a.y && live) fp8_store8<ALIGNED>((T*)a.y + m * a.ldy + k, n, g);
    if (a.out.codes) {
      const BlockScale b = block_scale(lanes_max<16>(n > 0 ? absmax8(g) : 0.0f), a.out.e8m0);
      fp8_store_codes8<ALIGNED>(a.out.codes + m * a.out.ld + k, live ? n : 0, g, b.r);
      if ((lane & 15) == 0 && n > 0 && live)
        store_scale(a.out.scales, (int64_t)(k / 128) * a.out.ld_scales + m, b.s, a.out.e8m0);
    }
  }
}

template <typename T, bool ALIGNED>
static void norm_launch(const NormArgs& a, hipStream_t st) {
  const int units = (a.K + 7) / 8;
  int wpr = 1;
  // At most a row per CU: 1 unit per lane, since a row's latency counts (1 x 5120 3.6 us, with
  // 3 units 4.9; 256 x 5120 5.2 and 6.4; but 1024 x 5120 12.7 and 10.6). Beyond that 3 units,
  // 5 on 8 wavefronts (4096 x 17408: 88 us, with 3 on 16 wavefronts 94).
  while (wpr < 16 && units > (a.M <= 256 ? 1 : wpr == 8 ? 5 : 3) * 64 * wpr) wpr *= 2;
  const int u = (units + 64 * wpr - 1) / (64 * wpr), waves = wpr > 4 ? wpr : 4, rows = waves / wpr;
  int64_t blocks = (a.M + rows - 1) / rows;
  if (blocks >= 512) blocks = (blocks + 255) / 256 * 256;
  const dim3 grid((unsigned)blocks), block(64 * waves);
  const bool stream = sizeof(T) == 2 && a.M * a.K * 2 >= kNormStream;
  switch (u) {
#define GWB_NORM(U) case U: hipLaunchKernelGGL((rmsnorm_fp8_kernel<T, ALIGNED, U>), grid, block, 0, st, a, wpr, stream); break;
    GWB_NORM(1) GWB_NORM(2) GWB_NORM(3) GWB_NORM(4) GWB_NORM(5) GWB_NORM(6) GWB_NORM(7) GWB_NORM(8)
#undef GWB_NORM
  }
}

void launch_rmsnorm_fp8(int32_t dtype, const NormArgs& a, bool aligned, hipStream_t st) {
  if (dtype == 0) aligned ? norm_launch<float, true>(a, st) : norm_launch<float, false>(a, st);
  else if (dtype == 1) aligned ? norm_launch<uint16_t, true>(a, st) : norm_launch<uint16_t, false>(a, st);
  else aligned ? norm_launch<_Float16, true>(a, st) : norm_launch<_Float16, false>(a, st);
}

}  // namespace gwb
