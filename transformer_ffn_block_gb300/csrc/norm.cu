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
// rows) b, b + gridDim.x, ...; thread t of a team owns the same columns of
// every row, so the column sums stay in its registers until the end, when the
// block writes its partial row of dgain (and dshift).  column_sum_kernel adds
// the blocks' partial rows in a fixed order: no atomics, the same bits each run.
template <bool CENTRED, int T, int V, int BLOCK>
__global__ void __launch_bounds__(BLOCK) norm_backward_kernel(uint16_t* dx, float* partial, float* stats,
                                                              const uint16_t* dy, const uint16_t* dres,
                                                              const uint16_t* r, const float* mean,
                                                              const float* rstd, const uint16_t* gain,
                                                              int64_t N, int C) {
  constexpr int TEAMS = BLOCK / T;
  __shared__ float red[2][64];
  __shared__ float comb[TEAMS > 1 ? TEAMS * T * V * 8 : 1];
  const int t = threadIdx.x % T, team = threadIdx.x / T;
  const int nchunk = C >> 3;
  uint4 gv[V];
  float dg[V][8], ds[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + i * T;
    gv[i] = c < nchunk ? ld16_ro(gain + size_t(c) * 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[i][j] = ds[i][j] = 0.0f;
  }
  const float inv_c = 1.0f / float(C);
  float amax = 0.0f;
  int buf = 0;
  for (int64_t row = int64_t(blockIdx.x) * TEAMS + team; row < N; row += int64_t(gridDim.x) * TEAMS) {
    const size_t base = size_t(row) * size_t(C);
    uint4 dv[V], rv[V], ev[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * T;
      dv[i] = rv[i] = ev[i] = make_uint4(0, 0, 0, 0);
      if (c < nchunk) {
        dv[i] = ld16_once(dy + base + size_t(c) * 8);
        rv[i] = ld16_once(r + base + size_t(c) * 8);
        if (dres != nullptr) ev[i] = ld16_once(dres + base + size_t(c) * 8);
      }
    }
    const float mu = CENTRED ? mean[row] : 0.0f, rs = rstd[row];
    float s1 = 0.0f, s2 = 0.0f;              // sum w * xhat, sum w
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (t + i * T < nchunk) {
        float d[8], x[8], g[8];
        unpack8(dv[i], d);
        unpack8(rv[i], x);
        unpack8(gv[i], g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float xh = CENTRED ? (x[j] - mu) * rs : x[j] * rs;
          const float w = d[j] * g[j];
          s1 = fmaf(w, xh, s1);
          if (CENTRED) s2 += w;
          dg[i][j] = fmaf(d[j], xh, dg[i][j]);
          if (CENTRED) ds[i][j] += d[j];
        }
      }
    }
    team_sum2<T>(s1, s2, red[buf]);
    buf ^= 1;                                // the next row's sums use the other buffer
    const float c1 = s1 * inv_c, c2 = s2 * inv_c;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * T;
      if (c < nchunk) {
        float d[8], x[8], g[8], e[8];
        unpack8(dv[i], d);
        unpack8(rv[i], x);
        unpack8(gv[i], g);
        unpack8(ev[i], e);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float xh = CENTRED ? (x[j] - mu) * rs : x[j] * rs;
          float v = fmaf(-xh, c1, d[j] * g[j]);
          if (CENTRED) v -= c2;
          e[j] = fmaf(v, rs, e[j]);
        }
        const uint4 o = pack8(e);
        stg16(dx + base + size_t(c) * 8, o);
        amax = fmaxf(amax, absmax8(o));
      }
    }
  }
  if (stats != nullptr) {
    amax = warp_max(amax);
    if ((threadIdx.x & 31) == 0) atomic_max_nonneg(stats, amax);
  }
  // partial rows: [gridDim.x][CENTRED ? 2 : 1][C]
  float* prow = partial + size_t(blockIdx.x) * size_t(CENTRED ? 2 : 1) * size_t(C);
#pragma unroll
  for (int k = 0; k < (CENTRED ? 2 : 1); ++k) {
    if (TEAMS > 1) {
      // the teams of the block added in order through shared memory
      __syncthreads();
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) comb[((team * T + t) * V + i) * 8 + j] = k == 0 ? dg[i][j] : ds[i][j];
      __syncthreads();
      for (int idx = threadIdx.x; idx < C; idx += BLOCK) {
        const int chunk = idx >> 3, j = idx & 7;
        const int tt = chunk % T, i = chunk / T;
        float s = 0.0f;
        for (int m = 0; m < TEAMS; ++m) s += comb[((m * T + tt) * V + i) * 8 + j];
        prow[size_t(k) * C + idx] = s;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = t + i * T;
        if (c < nchunk) {
          float4* dst = reinterpret_cast<float4*>(prow + size_t(k) * C + size_t(c) * 8);
          const float(&v)[8] = k == 0 ? dg[i] : ds[i];
          dst[0] = make_float4(v[0], v[1], v[2], v[3]);
          dst[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
      }
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

template <bool CENTRED, int T, int V, int BLOCK>
cudaError_t run_norm_backward(uint16_t* dx, float* partial, int blocks, float* stats, const uint16_t* dy,
                              const uint16_t* dres, const uint16_t* r, const float* mean, const float* rstd,
                              const uint16_t* gain, int64_t N, int C, cudaStream_t s) {
  norm_backward_kernel<CENTRED, T, V, BLOCK><<<blocks, BLOCK, 0, s>>>(dx, partial, stats, dy, dres, r, mean, rstd,
                                                                      gain, N, C);
  return cudaGetLastError();
}

template <bool CENTRED>
cudaError_t norm_backward(uint16_t* dx, float* partial, int blocks, float* stats, const uint16_t* dy,
                          const uint16_t* dres, const uint16_t* r, const float* mean, const float* rstd,
                          const uint16_t* gain, int64_t N, int C, cudaStream_t s) {
#define QFFN_NB(T, V, B) run_norm_backward<CENTRED, T, V, B>(dx, partial, blocks, stats, dy, dres, r, mean, rstd, gain, N, C, s)
  if (C <= 256) return QFFN_NB(32, 1, 256);
  if (C <= 512) return QFFN_NB(32, 2, 256);
  if (C <= 1024) return QFFN_NB(128, 1, 128);
  if (C <= 2048) return QFFN_NB(256, 1, 256);
  if (C <= 4096) return QFFN_NB(256, 2, 256);
  if (C <= 8192) return QFFN_NB(512, 2, 512);
  return QFFN_NB(1024, 2, 1024);
#undef QFFN_NB
}

// Threads per block and rows per block and pass of norm_backward's forms.
int bwd_block_threads(int C) { return C <= 512 ? 256 : C <= 1024 ? 128 : C <= 4096 ? 256 : C <= 8192 ? 512 : 1024; }
int bwd_rows(int C) { return C <= 512 ? 8 : 1; }

}  // namespace

int norm_backward_blocks(int64_t N, int C) {
  // three blocks of 256 threads' worth of work per SM (fixed for the 152 SMs of the
  // device so that the workspace size needs no device query)
  const int64_t per_sm = C <= 4096 ? 3 * 256 / bwd_block_threads(C) : 1;
  const int64_t cap = int64_t(kNumSMsHint) * (per_sm > 0 ? per_sm : 1);
  const int64_t need = (N + bwd_rows(C) - 1) / bwd_rows(C);
  return int(need < cap ? (need > 0 ? need : 1) : cap);
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
  e = centred ? norm_backward<true>(dx, partial, blocks, stats, dy, dres, r, mean, rstd, gain, N, C, s)
              : norm_backward<false>(dx, partial, blocks, stats, dy, dres, r, mean, rstd, gain, N, C, s);
  if (e != cudaSuccess) return e;
  return launch_column_sum(dgain, dshift, partial, blocks, C, centred ? 2 * int64_t(C) : C, accumulate, s);
}

}  // namespace qffn
