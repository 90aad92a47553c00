// Layer norm forward, and the backward of the layer norm and the RMS norm
// (HBM-bound).
//
// Forward, per row r of C values (r = bf16(res_in + x) or x):
//   mean = sum(r) / C,  var = sum((r - mean)^2) / C,  rstd = 1 / sqrt(var + eps)
//   y = bf16((r - mean) * rstd * gain + shift)
// Backward, with xhat = (r - mean) * rstd (RMS norm: r * rstd) and w = dy * gain:
//   dx = bf16(dres + rstd * (w - mean_C(w) - xhat * mean_C(w * xhat)))
//   (RMS norm: without mean_C(w))
//   dgain[c] = sum_rows dy * xhat,  dshift[c] = sum_rows dy
//
// A team of threads holds one row in registers, so the two-pass variance (sum
// of squares about the mean; no cancellation when |mean| >> sqrt(var)) and the
// two row sums of the backward cost no second read.  All sums are fp32; every
// output is rounded once.
#include "common.cuh"
#include "launch.h"
#include "pipeline.cuh"

namespace qffn {
namespace {

// Sums of `a` and `b` over the T threads of a team, in every thread.  Teams of
// a warp reduce by shuffles; a larger team is the whole block, and `red` (2 x
// 32 floats, one of two buffers used in turn) carries the warps' sums.
template <int T>
QFFN_DEVI void team_sum2(float& a, float& b, float* red) {
  a = warp_sum(a);
  b = warp_sum(b);
  if (T > 32) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) {
      red[warp] = a;
      red[32 + warp] = b;
    }
    __syncthreads();
    a = warp_sum(lane < T / 32 ? red[lane] : 0.0f);
    b = warp_sum(lane < T / 32 ? red[32 + lane] : 0.0f);
  }
}

QFFN_DEVI void unpack8(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = bf16_lo(w[j]);
    f[2 * j + 1] = bf16_hi(w[j]);
  }
}
QFFN_DEVI uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
QFFN_DEVI float absmax8(uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) m = fmaxf(m, fmaxf(fabsf(bf16_lo(w[j])), fabsf(bf16_hi(w[j]))));
  return m;
}

// ------------------------------------------------------------------ layer norm forward
// One row per team of T threads; thread t owns the 16-byte chunks t, t+T, ...
template <int T, int V, int BLOCK>
__global__ void __launch_bounds__(BLOCK) layernorm_kernel(uint16_t* res_out, uint16_t* y, float* mean_out,
                                                          float* rstd_out, float* stats,
                                                          const uint16_t* res_in, const uint16_t* x,
                                                          const uint16_t* gain, const uint16_t* shift,
                                                          float eps, int64_t N, int C) {
  __shared__ float red[2][64];
  const int t = threadIdx.x % T;
  const int64_t row = int64_t(blockIdx.x) * (BLOCK / T) + threadIdx.x / T;
  const bool live = row < N;                 // a team of T > 32 is the block: always live
  const int nchunk = C >> 3;
  const size_t base = live ? size_t(row) * size_t(C) : 0;
  uint4 rv[V];
  float sum = 0.0f, unused = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + i * T;
    if (live && c < nchunk) {
      uint4 r = ld16_once(x + base + size_t(c) * 8);
      if (res_in != nullptr) {
        const uint4 a = ld16_once(res_in + base + size_t(c) * 8);
        // bf16 + bf16 in fp32, one rounding: the residual stream is kept in bf16
        r.x = pack_bf16x2(bf16_lo(a.x) + bf16_lo(r.x), bf16_hi(a.x) + bf16_hi(r.x));
        r.y = pack_bf16x2(bf16_lo(a.y) + bf16_lo(r.y), bf16_hi(a.y) + bf16_hi(r.y));
        r.z = pack_bf16x2(bf16_lo(a.z) + bf16_lo(r.z), bf16_hi(a.z) + bf16_hi(r.z));
        r.w = pack_bf16x2(bf16_lo(a.w) + bf16_lo(r.w), bf16_hi(a.w) + bf16_hi(r.w));
        stg16(res_out + base + size_t(c) * 8, r);
      }
      rv[i] = r;
      float f[8];
      unpack8(r, f);
      sum += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
    }
  }
  team_sum2<T>(sum, unused, red[0]);
  const float mean = sum / float(C);
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (live && t + i * T < nchunk) {
      float f[8];
      unpack8(rv[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(f[j] - mean, f[j] - mean, ss);
    }
  }
  team_sum2<T>(ss, unused, red[1]);
  const float rstd = 1.0f / sqrtf(ss / float(C) + eps);
  if (live && t == 0) {
    mean_out[row] = mean;
    rstd_out[row] = rstd;
  }
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + i * T;
    if (live && c < nchunk) {
      float f[8], g[8], s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      unpack8(rv[i], f);
      unpack8(ld16_ro(gain + size_t(c) * 8), g);
      if (shift != nullptr) unpack8(ld16_ro(shift + size_t(c) * 8), s);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = fmaf((f[j] - mean) * rstd, g[j], s[j]);
      const uint4 o = pack8(f);
      stg16(y + base + size_t(c) * 8, o);
      amax = fmaxf(amax, absmax8(o));
    }
  }
  if (stats != nullptr) {
    amax = warp_max(amax);
    if ((threadIdx.x & 31) == 0) atomic_max_nonneg(stats, amax);
  }
}

// ------------------------------------------------------------------ norm backward
// Persistent: block b takes the rows (or, with teams of a warp, the groups of
// rows) b, b + gridDim.x, ...; a thread owns the same columns of every row, so
// the column sums stay in its registers until the end, when the block writes
// its partial row of dgain (and dshift).  column_sum_kernel adds the blocks'
// partial rows in a fixed order: no atomics, the same bits each run.

// dx of one 16-byte chunk, from the row's c1 = mean(w xhat) and c2 = mean(w).
template <bool CENTRED>
QFFN_DEVI uint4 norm_dx8(uint4 dv, uint4 rv, uint4 gv, uint4 ev, float mu, float rs, float c1, float c2) {
  float d[8], x[8], g[8], e[8];
  unpack8(dv, d);
  unpack8(rv, x);
  unpack8(gv, g);
  unpack8(ev, e);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float xh = CENTRED ? (x[j] - mu) * rs : x[j] * rs;
    float v = fmaf(-xh, c1, d[j] * g[j]);
    if (CENTRED) v -= c2;
    e[j] = fmaf(v, rs, e[j]);
  }
  return pack8(e);
}
// The chunk's terms of the row sums (s1 += w xhat, s2 += w) and column sums.
template <bool CENTRED>
QFFN_DEVI void norm_sums8(uint4 dv, uint4 rv, uint4 gv, float mu, float rs, float& s1, float& s2, float (&dg)[8],
                          float (&ds)[8]) {
  float d[8], x[8], g[8];
  unpack8(dv, d);
  unpack8(rv, x);
  unpack8(gv, g);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float xh = CENTRED ? (x[j] - mu) * rs : x[j] * rs;
    const float w = d[j] * g[j];
    s1 = fmaf(w, xh, s1);
    if (CENTRED) s2 += w;
    dg[j] = fmaf(d[j], xh, dg[j]);
    if (CENTRED) ds[j] += d[j];
  }
}

struct NormBwd {
  uint16_t* dx;
  float* partial;            // [gridDim.x][CENTRED ? 2 : 1][C]
  float* stats;
  const uint16_t* dy;
  const uint16_t* dres;
  const uint16_t* r;
  const float* mean;
  const float* rstd;
  const uint16_t* gain;
  int64_t N;
  int C;
  int stages;                // ring form
};

// Rows of at most 512 values: a warp per row, eight rows per block in flight.
template <bool CENTRED, int V>
__global__ void __launch_bounds__(256) norm_backward_warp_kernel(const NormBwd a) {
  constexpr int TEAMS = 8;
  __shared__ float comb[TEAMS * 32 * V * 8];
  const int t = threadIdx.x & 31, team = threadIdx.x >> 5;
  const int nchunk = a.C >> 3;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 gv[V];
  float dg[V][8], ds[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + i * 32;
    gv[i] = c < nchunk ? ld16_ro(a.gain + size_t(c) * 8) : zero;
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[i][j] = ds[i][j] = 0.0f;
  }
  const float inv_c = 1.0f / float(a.C);
  float amax = 0.0f;
  for (int64_t row = int64_t(blockIdx.x) * TEAMS + team; row < a.N; row += int64_t(gridDim.x) * TEAMS) {
    const size_t base = size_t(row) * size_t(a.C);
    uint4 dv[V], rv[V], ev[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * 32;
      dv[i] = rv[i] = ev[i] = zero;
      if (c < nchunk) {
        dv[i] = ld16_once(a.dy + base + size_t(c) * 8);
        rv[i] = ld16_once(a.r + base + size_t(c) * 8);
        if (a.dres != nullptr) ev[i] = ld16_once(a.dres + base + size_t(c) * 8);
      }
    }
    const float mu = CENTRED ? a.mean[row] : 0.0f, rs = a.rstd[row];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (t + i * 32 < nchunk) norm_sums8<CENTRED>(dv[i], rv[i], gv[i], mu, rs, s1, s2, dg[i], ds[i]);
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * 32;
      if (c < nchunk) {
        const uint4 o = norm_dx8<CENTRED>(dv[i], rv[i], gv[i], ev[i], mu, rs, s1 * inv_c, s2 * inv_c);
        stg16(a.dx + base + size_t(c) * 8, o);
        amax = fmaxf(amax, absmax8(o));
      }
    }
  }
  if (a.stats != nullptr) {
    amax = warp_max(amax);
    if (t == 0) atomic_max_nonneg(a.stats, amax);
  }
  float* prow = a.partial + size_t(blockIdx.x) * size_t(CENTRED ? 2 : 1) * size_t(a.C);
#pragma unroll
  for (int k = 0; k < (CENTRED ? 2 : 1); ++k) {
    // the block's warps added in order through shared memory
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) comb[((team * 32 + t) * V + i) * 8 + j] = k == 0 ? dg[i][j] : ds[i][j];
    __syncthreads();
    for (int idx = threadIdx.x; idx < a.C; idx += 256) {
      const int chunk = idx >> 3, j = idx & 7;
      float s = 0.0f;
      for (int m = 0; m < TEAMS; ++m) s += comb[((m * 32 + chunk % 32) * V + chunk / 32) * 8 + j];
      prow[size_t(k) * a.C + idx] = s;
    }
  }
}

__device__ unsigned int g_status;
constexpr unsigned long long kWaitLimitNs = 2000000000ull;
constexpr unsigned long long kDrainLimitNs = 200000000ull;
constexpr int kMaxStages = 8;

// Longer rows: the block is the team.  A row's three inputs come by bulk copy
// into one stage of a shared-memory ring, `stages` rows deep, so the loads of
// the next rows are in flight while a row is reduced and written; threads need
// registers for the column sums only.  A stage is refilled by thread 0 one row
// later, after that row's barrier (inside team_sum2), which every thread
// reaches only when it has read the stage.  Measured at 16384 x 4096 (layer
// norm, with dres): loads into registers 148 us, two to three rows in flight
// per SM; see the launch for the ring's figures.
template <bool CENTRED, int T, int V>
__global__ void __launch_bounds__(T) norm_backward_kernel(const NormBwd a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[2][64];
  __shared__ __align__(8) uint64_t bars[kMaxStages];
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  const int t = threadIdx.x;
  const int nchunk = a.C >> 3;
  const uint32_t row_bytes = uint32_t(a.C) * 2u;
  const int inputs = a.dres != nullptr ? 3 : 2;
  const uint32_t stage_bytes = row_bytes * uint32_t(inputs);
  if (t == 0) {
    for (int s = 0; s < a.stages; ++s) mbar_init(smem_u32(&bars[s]), 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  __syncthreads();
  auto load_row = [&](int64_t row, int s) {       // thread 0
    const uint32_t bar = smem_u32(&bars[s]), dst = smem_u32(ring) + uint32_t(s) * stage_bytes;
    const size_t base = size_t(row) * size_t(a.C);
    mbar_expect_tx(bar, stage_bytes);
    bulk_load(dst, a.dy + base, row_bytes, bar);
    bulk_load(dst + row_bytes, a.r + base, row_bytes, bar);
    if (inputs == 3) bulk_load(dst + 2 * row_bytes, a.dres + base, row_bytes, bar);
  };
  int64_t next_load = blockIdx.x;                 // thread 0: next row to request
  int fill = 0;                                   //   and its stage
  if (t == 0)
    for (; fill < a.stages && next_load < a.N; ++fill, next_load += gridDim.x) load_row(next_load, fill);
  uint4 gv[V];
  float dg[V][8], ds[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + i * T;
    gv[i] = c < nchunk ? ld16_ro(a.gain + size_t(c) * 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[i][j] = ds[i][j] = 0.0f;
  }
  const float inv_c = 1.0f / float(a.C);
  float amax = 0.0f;
  int buf = 0, s = 0, refill = -1;
  uint32_t parity = 0;
  bool ok = true;
  float mu_next = 0.0f, rs_next = 0.0f;
  if (int64_t(blockIdx.x) < a.N) {
    mu_next = CENTRED ? a.mean[blockIdx.x] : 0.0f;
    rs_next = a.rstd[blockIdx.x];
  }
  for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x) {
    const float mu = mu_next, rs = rs_next;
    if (row + gridDim.x < a.N) {
      mu_next = CENTRED ? a.mean[row + gridDim.x] : 0.0f;
      rs_next = a.rstd[row + gridDim.x];
    }
    // a wait that runs out raises the abort flag, which all threads see after the barrier below
    mbar_wait_bounded(smem_u32(&bars[s]), parity, abort_flag, &g_status, true, kWaitLimitNs);
    const uint8_t* st = ring + size_t(s) * stage_bytes;
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * T;
      if (c < nchunk)
        norm_sums8<CENTRED>(*reinterpret_cast<const uint4*>(st + c * 16),
                            *reinterpret_cast<const uint4*>(st + row_bytes + c * 16), gv[i], mu, rs, s1, s2, dg[i],
                            ds[i]);
    }
    team_sum2<T>(s1, s2, red[buf]);
    buf ^= 1;                                     // the next row's sums use the other buffer
    if (*abort_flag) { ok = false; break; }
    if (t == 0 && refill >= 0 && next_load < a.N) {   // the previous row's stage has been read by all
      load_row(next_load, refill);
      next_load += gridDim.x;
    }
    refill = s;
    const size_t base = size_t(row) * size_t(a.C);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * T;
      if (c < nchunk) {
        const uint4 ev = inputs == 3 ? *reinterpret_cast<const uint4*>(st + 2 * row_bytes + c * 16)
                                     : make_uint4(0, 0, 0, 0);
        const uint4 o = norm_dx8<CENTRED>(*reinterpret_cast<const uint4*>(st + c * 16),
                                          *reinterpret_cast<const uint4*>(st + row_bytes + c * 16), gv[i], ev, mu, rs,
                                          s1 * inv_c, s2 * inv_c);
        stg16(a.dx + base + size_t(c) * 8, o);
        amax = fmaxf(amax, absmax8(o));
      }
    }
    if (++s == a.stages) {
      s = 0;
      parity ^= 1u;
    }
  }
  if (!ok) {
    // no copy into shared memory is in flight when the block ends: every barrier's current phase
    if (t == 0)
      for (int k = 0; k < a.stages; ++k) {
        const uint32_t p = k < s ? parity ^ 1u : parity;
        mbar_wait_bounded(smem_u32(&bars[k]), p, abort_flag, &g_status, false, kDrainLimitNs);
      }
    return;
  }
  if (a.stats != nullptr) {
    amax = warp_max(amax);
    if ((t & 31) == 0) atomic_max_nonneg(a.stats, amax);
  }
  float* prow = a.partial + size_t(blockIdx.x) * size_t(CENTRED ? 2 : 1) * size_t(a.C);
#pragma unroll
  for (int k = 0; k < (CENTRED ? 2 : 1); ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * T;
      if (c < nchunk) {
        float4* dst = reinterpret_cast<float4*>(prow + size_t(k) * a.C + size_t(c) * 8);
        const float(&v)[8] = k == 0 ? dg[i] : ds[i];
        dst[0] = make_float4(v[0], v[1], v[2], v[3]);
        dst[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
}

// out[c] (+)= sum over p of partial[p][c], p in order within each of 8 strided
// groups, the groups added in order.  32 columns per block.
__global__ void __launch_bounds__(256) column_sum_kernel(float* out0, float* out1, const float* partial, int parts,
                                                         int64_t cols0, int64_t cols, int accumulate) {
  pdl_wait();
  __shared__ float s[8][33];
  const int64_t c = int64_t(blockIdx.x) * 32 + (threadIdx.x & 31);
  const int g = threadIdx.x >> 5;
  float v = 0.0f;
  if (c < cols)
    for (int p = g; p < parts; p += 8) v += partial[size_t(p) * size_t(cols) + size_t(c)];
  s[g][threadIdx.x & 31] = v;
  __syncthreads();
  if (g == 0 && c < cols) {
    for (int k = 1; k < 8; ++k) v += s[k][threadIdx.x];
    // columns [0, cols0) go to out0, the rest to out1; either may be absent
    float* dst = c < cols0 ? out0 : out1;
    const int64_t i = c < cols0 ? c : c - cols0;
    if (dst != nullptr) dst[i] = accumulate ? dst[i] + v : v;
  }
}

template <int T, int V, int BLOCK>
cudaError_t run_layernorm(uint16_t* res_out, uint16_t* y, float* mean, float* rstd, float* stats,
                          const uint16_t* res_in, const uint16_t* x, const uint16_t* gain,
                          const uint16_t* shift, float eps, int64_t N, int C, cudaStream_t s) {
  const int64_t rows = BLOCK / T;
  layernorm_kernel<T, V, BLOCK><<<unsigned((N + rows - 1) / rows), BLOCK, 0, s>>>(
      res_out, y, mean, rstd, stats, res_in, x, gain, shift, eps, N, C);
  return cudaGetLastError();
}

// Blocks per SM of the ring form, and the shared memory each may take.
int ring_blocks_per_sm(int C) { return C <= 1024 ? 4 : C <= 4096 ? 2 : 1; }

template <bool CENTRED, int T, int V>
cudaError_t run_ring(NormBwd a, int blocks, cudaStream_t s) {
  const int stage = a.C * 2 * (a.dres != nullptr ? 3 : 2);
  const int budget = 208 * 1024 / ring_blocks_per_sm(a.C);
  a.stages = budget / stage;
  if (a.stages > kMaxStages) a.stages = kMaxStages;
  const int bytes = a.stages * stage;
  static bool set[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !set[dev]) {
    e = cudaFuncSetAttribute(norm_backward_kernel<CENTRED, T, V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             208 * 1024);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  norm_backward_kernel<CENTRED, T, V><<<blocks, T, bytes, s>>>(a);
  return cudaGetLastError();
}

template <bool CENTRED>
cudaError_t norm_backward(const NormBwd& a, int blocks, cudaStream_t s) {
  if (a.C <= 512) {
    if (a.C <= 256) norm_backward_warp_kernel<CENTRED, 1><<<blocks, 256, 0, s>>>(a);
    else norm_backward_warp_kernel<CENTRED, 2><<<blocks, 256, 0, s>>>(a);
    return cudaGetLastError();
  }
  if (a.C <= 1024) return run_ring<CENTRED, 128, 1>(a, blocks, s);
  if (a.C <= 2048) return run_ring<CENTRED, 256, 1>(a, blocks, s);
  if (a.C <= 4096) return run_ring<CENTRED, 256, 2>(a, blocks, s);
  if (a.C <= 8192) return run_ring<CENTRED, 512, 2>(a, blocks, s);
  return run_ring<CENTRED, 512, 4>(a, blocks, s);
}

}  // namespace

int norm_backward_blocks(int64_t N, int C) {
  // fixed for the 152 SMs of the device, so that the workspace size needs no device query
  const int64_t cap = int64_t(kNumSMsHint) * (C <= 512 ? 4 : ring_blocks_per_sm(C));
  const int64_t need = C <= 512 ? (N + 7) / 8 : N;
  return int(need < cap ? (need > 0 ? need : 1) : cap);
}

cudaError_t norm_take_status(unsigned int* status) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_status, sizeof(v));
  if (e != cudaSuccess) return e;
  if (v != 0) e = cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
  *status = v;
  return e;
}

cudaError_t launch_layernorm(uint16_t* res_out, uint16_t* y, float* mean, float* rstd, float* stats,
                             const uint16_t* res_in, const uint16_t* x, const uint16_t* gain,
                             const uint16_t* shift, float eps, int64_t N, int C, cudaStream_t s) {
  if (stats != nullptr) {
    const cudaError_t e = cudaMemsetAsync(stats, 0, sizeof(float), s);
    if (e != cudaSuccess) return e;
  }
  if (N == 0) return cudaSuccess;
#define QFFN_LN(T, V, B) run_layernorm<T, V, B>(res_out, y, mean, rstd, stats, res_in, x, gain, shift, eps, N, C, s)
  if (C <= 256) return QFFN_LN(32, 1, 128);
  if (C <= 512) return QFFN_LN(32, 2, 128);
  if (C <= 1024) return QFFN_LN(32, 4, 128);
  if (C <= 2048) return QFFN_LN(128, 2, 128);
  if (C <= 4096) return QFFN_LN(128, 4, 128);
  if (C <= 8192) return QFFN_LN(256, 4, 256);
  return QFFN_LN(512, 4, 512);
#undef QFFN_LN
}

cudaError_t launch_column_sum(float* out0, float* out1, const float* partial, int parts, int64_t cols0, int64_t cols,
                              bool accumulate, cudaStream_t s) {
  if (cols == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((cols + 31) / 32));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, column_sum_kernel, out0, out1, partial, parts, cols0, cols, accumulate ? 1 : 0);
}

cudaError_t launch_norm_backward(uint16_t* dx, float* dgain, float* dshift, float* stats, const uint16_t* dy,
                                 const uint16_t* dres, const uint16_t* r, const float* mean, const float* rstd,
                                 const uint16_t* gain, int64_t N, int C, bool centred, bool accumulate,
                                 float* partial, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (stats != nullptr && (e = cudaMemsetAsync(stats, 0, sizeof(float), s)) != cudaSuccess) return e;
  if (N == 0) {
    // sums over no rows: zero, or unchanged when accumulating
    if (accumulate) return cudaSuccess;
    if ((e = cudaMemsetAsync(dgain, 0, size_t(C) * sizeof(float), s)) != cudaSuccess) return e;
    return dshift != nullptr ? cudaMemsetAsync(dshift, 0, size_t(C) * sizeof(float), s) : cudaSuccess;
  }
  const int blocks = norm_backward_blocks(N, C);
  const NormBwd a{dx, partial, stats, dy, dres, r, mean, rstd, gain, N, C, 0};
  e = centred ? norm_backward<true>(a, blocks, s) : norm_backward<false>(a, blocks, s);
  if (e != cudaSuccess) return e;
  return launch_column_sum(dgain, dshift, partial, blocks, C, centred ? 2 * int64_t(C) : C, accumulate, s);
}

}  // namespace qffn
