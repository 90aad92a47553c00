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
#include "act.cuh"
#include "common.cuh"
#include "launch.h"
#include "pipeline.cuh"
#include "umma.cuh"

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

// Eight bf16 as four float pairs, and back.
struct F8 {
  uint64_t p[4];
};
QFFN_DEVI F8 unpack8(uint4 v) { return F8{{bf16x2_to_f2(v.x), bf16x2_to_f2(v.y), bf16x2_to_f2(v.z), bf16x2_to_f2(v.w)}}; }
QFFN_DEVI uint32_t pack2(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return pack_bf16x2(lo, hi);
}
QFFN_DEVI uint4 pack8(const F8& f) { return make_uint4(pack2(f.p[0]), pack2(f.p[1]), pack2(f.p[2]), pack2(f.p[3])); }
QFFN_DEVI float f2_sum(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return lo + hi;
}
// Running max of |v| over the bf16 pairs of a chunk.
QFFN_DEVI uint32_t absmax8(uint32_t m, uint4 v) {
  return bf16x2_absmax(bf16x2_absmax(bf16x2_absmax(bf16x2_absmax(m, v.x), v.y), v.z), v.w);
}
QFFN_DEVI void record_absmax(float* stats, uint32_t m) {
  const float v = warp_max(fmaxf(bf16_lo(m), bf16_hi(m)));
  if ((threadIdx.x & 31) == 0) atomic_max_nonneg(stats, v);
}

__device__ unsigned int g_status;
constexpr unsigned long long kWaitLimitNs = 2000000000ull;
constexpr unsigned long long kDrainLimitNs = 200000000ull;
constexpr int kMaxStages = 8;

// ------------------------------------------------------------------ layer norm forward
struct LnFwd {
  uint16_t* res_out;
  uint16_t* y;
  float* mean;
  float* rstd;
  float* stats;
  const uint16_t* res_in;
  const uint16_t* x;
  const uint16_t* gain;
  const uint16_t* shift;
  float eps;
  int64_t N;
  int C;
};

// bf16 + bf16 in fp32, one rounding: the residual stream is kept in bf16.
QFFN_DEVI uint4 add8(uint4 a, uint4 b) {
  F8 x = unpack8(a);
  const F8 z = unpack8(b);
#pragma unroll
  for (int j = 0; j < 4; ++j) x.p[j] = f2_add(x.p[j], z.p[j]);
  return pack8(x);
}
QFFN_DEVI uint64_t sum8(const F8& f) { return f2_add(f2_add(f.p[0], f.p[1]), f2_add(f.p[2], f.p[3])); }
// ss += (f - mean)^2 of a chunk
QFFN_DEVI uint64_t squares8(const F8& f, uint64_t neg_mean, uint64_t ss) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t d = f2_add(f.p[j], neg_mean);
    ss = f2_fma(d, d, ss);
  }
  return ss;
}
// (f - mean) * rstd * gain + shift
QFFN_DEVI uint4 normed8(const F8& f, uint64_t neg_mean, uint64_t rstd, const F8& g, const F8& s) {
  F8 o;
#pragma unroll
  for (int j = 0; j < 4; ++j) o.p[j] = f2_fma(f2_mul(f2_add(f.p[j], neg_mean), rstd), g.p[j], s.p[j]);
  return pack8(o);
}

// One row per team of T threads; thread t owns the 16-byte chunks t, t+T, ...
// Small teams with up to four chunks a thread for many rows: a dozen rows or
// more of independent blocks per SM hide each other's loads and barriers (16384
// x 4096 with a residual 81 us, 6.6 TB/s; persistent blocks fed by bulk copies
// 85 to 98).  Larger teams for few rows, where a call is a launch and one round
// of loads (one row of 4096: 3.1 us against 4.1).
template <int T, int V, int BLOCK>
__global__ void __launch_bounds__(BLOCK) layernorm_kernel(const LnFwd a) {
  __shared__ float red[2][64];
  const int t = threadIdx.x % T;
  const int64_t row = int64_t(blockIdx.x) * (BLOCK / T) + threadIdx.x / T;
  const bool live = row < a.N;               // a team of T > 32 is the block: always live
  const int nchunk = a.C >> 3;
  const size_t base = live ? size_t(row) * size_t(a.C) : 0;
  pdl_wait();
  const uint16_t *gain = behind_wait(a.gain), *shift = behind_wait(a.shift);
  pdl_trigger();
  uint4 rv[V];
  uint64_t acc = 0ull;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + i * T;
    if (live && c < nchunk) {
      rv[i] = ld16_once(a.x + base + size_t(c) * 8);
      if (a.res_in != nullptr) {
        rv[i] = add8(ld16_once(a.res_in + base + size_t(c) * 8), rv[i]);
        stg16(a.res_out + base + size_t(c) * 8, rv[i]);
      }
      acc = f2_add(acc, sum8(unpack8(rv[i])));
    }
  }
  float sum = f2_sum(acc), unused = 0.0f;
  team_sum2<T>(sum, unused, red[0]);
  const float mean = sum / float(a.C);
  const uint64_t neg_mean = f2_dup(-mean);
  acc = 0ull;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (live && t + i * T < nchunk) acc = squares8(unpack8(rv[i]), neg_mean, acc);
  float ss = f2_sum(acc);
  team_sum2<T>(ss, unused, red[1]);
  const float rstd = 1.0f / sqrtf(ss / float(a.C) + a.eps);
  if (live && t == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
  uint32_t amax = 0u;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + i * T;
    if (live && c < nchunk) {
      F8 s{{0ull, 0ull, 0ull, 0ull}};
      if (shift != nullptr) s = unpack8(ld16_settled(shift + size_t(c) * 8));
      const uint4 o = normed8(unpack8(rv[i]), neg_mean, f2_dup(rstd), unpack8(ld16_settled(gain + size_t(c) * 8)), s);
      stg16(a.y + base + size_t(c) * 8, o);
      if (a.stats != nullptr) amax = absmax8(amax, o);
    }
  }
  if (a.stats != nullptr) record_absmax(a.stats, amax);
}

// ------------------------------------------------------------------ norm backward
// Persistent: block b takes the rows (or, with teams of a warp, the groups of
// rows) b, b + gridDim.x, ...; a thread owns the same columns of every row, so
// the column sums stay in its registers until the end, when the block writes
// its partial row of dgain (and dshift).  column_sum_kernel adds the blocks'
// partial rows in a fixed order: no atomics, the same bits each run.

// xhat of a pair.  The mean is subtracted first: the difference is exact or nearly
// so where the row lies far from zero, while rs x - rs mean would keep the rounding
// of rs mean, the same in every element of the row, in the sums.
template <bool CENTRED>
QFFN_DEVI uint64_t norm_hat(uint64_t x, uint64_t rs, uint64_t neg_mu) {
  return f2_mul(CENTRED ? f2_add(x, neg_mu) : x, rs);
}

// dx of one 16-byte chunk: e + rs w + k1 xhat + k2 with k1 = -rs c1, k2 = -rs c2.
template <bool CENTRED>
QFFN_DEVI uint4 norm_dx8(uint4 dv, uint4 rv, uint4 gv, uint4 ev, uint64_t rs, uint64_t neg_mu, uint64_t k1,
                         uint64_t k2) {
  const F8 d = unpack8(dv), x = unpack8(rv), g = unpack8(gv);
  F8 e = unpack8(ev);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t xh = norm_hat<CENTRED>(x.p[j], rs, neg_mu);
    // the sum of the three gradient terms first, dres last
    uint64_t v = CENTRED ? f2_fma(xh, k1, k2) : f2_mul(xh, k1);
    v = f2_fma(f2_mul(d.p[j], g.p[j]), rs, v);
    e.p[j] = f2_add(e.p[j], v);
  }
  return pack8(e);
}
// The chunk's terms of the row sums (s1 += w xhat, s2 += w) and column sums.
template <bool CENTRED>
QFFN_DEVI void norm_sums8(uint4 dv, uint4 rv, uint4 gv, uint64_t rs, uint64_t neg_mu, uint64_t& s1, uint64_t& s2,
                          uint64_t (&dg)[4], uint64_t (&ds)[4]) {
  const F8 d = unpack8(dv), x = unpack8(rv), g = unpack8(gv);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t xh = norm_hat<CENTRED>(x.p[j], rs, neg_mu);
    const uint64_t w = f2_mul(d.p[j], g.p[j]);
    s1 = f2_fma(w, xh, s1);
    if (CENTRED) s2 = f2_add(s2, w);
    dg[j] = f2_fma(d.p[j], xh, dg[j]);
    if (CENTRED) ds[j] = f2_add(ds[j], d.p[j]);
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
  __shared__ __align__(8) float comb[TEAMS * 32 * V * 8];
  const int t = threadIdx.x & 31, team = threadIdx.x >> 5;
  const int nchunk = a.C >> 3;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  pdl_wait();
  pdl_trigger();
  uint4 gv[V];
  uint64_t dg[V][4], ds[V][4];               // pairs of columns
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + i * 32;
    gv[i] = c < nchunk ? ld16_once(a.gain + size_t(c) * 8) : zero;
#pragma unroll
    for (int j = 0; j < 4; ++j) dg[i][j] = ds[i][j] = 0ull;
  }
  const float inv_c = 1.0f / float(a.C);
  uint32_t amax = 0u;
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
    const uint64_t rs2 = f2_dup(rs), nm2 = f2_dup(-mu);
    uint64_t p1 = 0ull, p2 = 0ull;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (t + i * 32 < nchunk) norm_sums8<CENTRED>(dv[i], rv[i], gv[i], rs2, nm2, p1, p2, dg[i], ds[i]);
    const uint64_t k1 = f2_dup(-rs * (warp_sum(f2_sum(p1)) * inv_c));
    const uint64_t k2 = f2_dup(-rs * (warp_sum(f2_sum(p2)) * inv_c));
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * 32;
      if (c < nchunk) {
        const uint4 o = norm_dx8<CENTRED>(dv[i], rv[i], gv[i], ev[i], rs2, nm2, k1, k2);
        stg16(a.dx + base + size_t(c) * 8, o);
        if (a.stats != nullptr) amax = absmax8(amax, o);
      }
    }
  }
  if (a.stats != nullptr) record_absmax(a.stats, amax);
  float* prow = a.partial + size_t(blockIdx.x) * size_t(CENTRED ? 2 : 1) * size_t(a.C);
#pragma unroll
  for (int k = 0; k < (CENTRED ? 2 : 1); ++k) {
    // the block's warps added in order through shared memory
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint64_t*>(&comb[((team * 32 + t) * V + i) * 8 + 2 * j]) = k == 0 ? dg[i][j] : ds[i][j];
    __syncthreads();
    for (int idx = threadIdx.x; idx < a.C; idx += 256) {
      const int chunk = idx >> 3, j = idx & 7;
      float s = 0.0f;
      for (int m = 0; m < TEAMS; ++m) s += comb[((m * 32 + chunk % 32) * V + chunk / 32) * 8 + j];
      prow[size_t(k) * a.C + idx] = s;
    }
  }
}

// Longer rows: the block is the team.  A row's three inputs come by bulk copy
// into one stage of a shared-memory ring, `stages` rows deep, so the loads of
// the next rows are in flight while a row is reduced and written; threads need
// registers for the column sums only.  A stage is refilled by thread 0 one row
// later, after that row's barrier (inside team_sum2), which every thread
// reaches only when it has read the stage.  Measured at 16384 x 4096 with dres
// (floor 79 us): loads into registers, two to three rows in flight per SM, 148
// us (layer norm) and 96 (RMS norm); this ring 96 and 82; with the arithmetic
// in pairs 82.5 and 80.5 (6.5 TB/s).
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
  pdl_wait();
  pdl_trigger();
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
  uint64_t dg[V][4], ds[V][4];               // pairs of columns
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + i * T;
    gv[i] = c < nchunk ? ld16_once(a.gain + size_t(c) * 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) dg[i][j] = ds[i][j] = 0ull;
  }
  const float inv_c = 1.0f / float(a.C);
  uint32_t amax = 0u;
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
    const uint64_t rs2 = f2_dup(rs), nm2 = f2_dup(-mu);
    uint64_t p1 = 0ull, p2 = 0ull;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * T;
      if (c < nchunk)
        norm_sums8<CENTRED>(*reinterpret_cast<const uint4*>(st + c * 16),
                            *reinterpret_cast<const uint4*>(st + row_bytes + c * 16), gv[i], rs2, nm2, p1, p2, dg[i],
                            ds[i]);
    }
    float s1 = f2_sum(p1), s2 = f2_sum(p2);
    team_sum2<T>(s1, s2, red[buf]);
    buf ^= 1;                                     // the next row's sums use the other buffer
    if (*abort_flag) { ok = false; break; }
    if (t == 0 && refill >= 0 && next_load < a.N) {   // the previous row's stage has been read by all
      load_row(next_load, refill);
      next_load += gridDim.x;
    }
    refill = s;
    const uint64_t k1 = f2_dup(-rs * (s1 * inv_c)), k2 = f2_dup(-rs * (s2 * inv_c));
    const size_t base = size_t(row) * size_t(a.C);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * T;
      if (c < nchunk) {
        const uint4 ev = inputs == 3 ? *reinterpret_cast<const uint4*>(st + 2 * row_bytes + c * 16)
                                     : make_uint4(0, 0, 0, 0);
        const uint4 o = norm_dx8<CENTRED>(*reinterpret_cast<const uint4*>(st + c * 16),
                                          *reinterpret_cast<const uint4*>(st + row_bytes + c * 16), gv[i], ev, rs2, nm2,
                                          k1, k2);
        stg16(a.dx + base + size_t(c) * 8, o);
        if (a.stats != nullptr) amax = absmax8(amax, o);
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
  if (a.stats != nullptr) record_absmax(a.stats, amax);
  float* prow = a.partial + size_t(blockIdx.x) * size_t(CENTRED ? 2 : 1) * size_t(a.C);
#pragma unroll
  for (int k = 0; k < (CENTRED ? 2 : 1); ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * T;
      if (c < nchunk) {
        ulonglong2* dst = reinterpret_cast<ulonglong2*>(prow + size_t(k) * a.C + size_t(c) * 8);
        const uint64_t(&v)[4] = k == 0 ? dg[i] : ds[i];
        dst[0] = make_ulonglong2(v[0], v[1]);
        dst[1] = make_ulonglong2(v[2], v[3]);
      }
    }
}

// Few rows: one launch.  Block b < N does row b; the blocks behind do 64 columns
// each of dgain and dshift, which need the given statistics only and read dy and
// r again (from L2).  Eight threads cover a row's 64 columns, T / 8 rows at a
// time, four loads in flight each; the partial sums are added in a fixed order.
template <bool CENTRED, int T>
__global__ void __launch_bounds__(T) norm_backward_short_kernel(const NormBwd a, float* dgain, float* dshift,
                                                                int accumulate) {
  __shared__ float red[64];
  __shared__ float comb[2][T / 32][64];
  const int t = threadIdx.x;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  pdl_wait();
  pdl_trigger();
  if (int64_t(blockIdx.x) < a.N) {
    constexpr int V = 2;
    const int64_t row = blockIdx.x;
    const size_t base = size_t(row) * size_t(a.C);
    const int nchunk = a.C >> 3;
    const float mu = CENTRED ? a.mean[row] : 0.0f, rs = a.rstd[row];
    uint4 dv[V], rv[V], ev[V], gv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * T;
      dv[i] = rv[i] = ev[i] = gv[i] = zero;
      if (c < nchunk) {
        dv[i] = ld16_once(a.dy + base + size_t(c) * 8);
        rv[i] = ld16_once(a.r + base + size_t(c) * 8);
        gv[i] = ld16_once(a.gain + size_t(c) * 8);
        if (a.dres != nullptr) ev[i] = ld16_once(a.dres + base + size_t(c) * 8);
      }
    }
    const uint64_t rs2 = f2_dup(rs), nm2 = f2_dup(-mu);
    uint64_t p1 = 0ull, p2 = 0ull, dg[4] = {0ull, 0ull, 0ull, 0ull}, ds[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
    for (int i = 0; i < V; ++i) norm_sums8<CENTRED>(dv[i], rv[i], gv[i], rs2, nm2, p1, p2, dg, ds);
    float s1 = f2_sum(p1), s2 = f2_sum(p2);
    team_sum2<T>(s1, s2, red);
    const float inv_c = 1.0f / float(a.C);
    const uint64_t k1 = f2_dup(-rs * (s1 * inv_c)), k2 = f2_dup(-rs * (s2 * inv_c));
    uint32_t amax = 0u;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * T;
      if (c < nchunk) {
        const uint4 o = norm_dx8<CENTRED>(dv[i], rv[i], gv[i], ev[i], rs2, nm2, k1, k2);
        stg16(a.dx + base + size_t(c) * 8, o);
        if (a.stats != nullptr) amax = absmax8(amax, o);
      }
    }
    if (a.stats != nullptr) record_absmax(a.stats, amax);
    return;
  }
  constexpr int kRows = T / 8, kFlight = 4;
  const int64_t col = (int64_t(blockIdx.x) - a.N) * 64 + (t & 7) * 8;
  uint64_t dg[4] = {0ull, 0ull, 0ull, 0ull}, ds[4] = {0ull, 0ull, 0ull, 0ull}, unused1 = 0ull, unused2 = 0ull;
  if (col < a.C) {
    for (int64_t row0 = t >> 3; row0 < a.N; row0 += kRows * kFlight) {
      uint4 dv[kFlight], rv[kFlight];
      float mu[kFlight], rs[kFlight];
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        const int64_t row = row0 + k * kRows;
        const bool live = row < a.N;
        const size_t i = size_t(live ? row : 0) * size_t(a.C) + size_t(col);
        dv[k] = live ? ld16_once(a.dy + i) : zero;
        rv[k] = live ? ld16_once(a.r + i) : zero;
        mu[k] = CENTRED && live ? a.mean[row] : 0.0f;
        rs[k] = live ? a.rstd[row] : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < kFlight; ++k)
        if (row0 + k * kRows < a.N)
          norm_sums8<CENTRED>(dv[k], rv[k], zero, f2_dup(rs[k]), f2_dup(-mu[k]), unused1, unused2, dg, ds);
    }
  }
  // the four rows of a warp, then the warps in order
  const int warp = t >> 5, lane = t & 31;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float v[4];
    f2_unpack(dg[j], v[0], v[1]);
    f2_unpack(ds[j], v[2], v[3]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] += __shfl_xor_sync(0xffffffffu, v[k], 8);
      v[k] += __shfl_xor_sync(0xffffffffu, v[k], 16);
    }
    if (lane < 8) {
      comb[0][warp][lane * 8 + 2 * j] = v[0];
      comb[0][warp][lane * 8 + 2 * j + 1] = v[1];
      comb[1][warp][lane * 8 + 2 * j] = v[2];
      comb[1][warp][lane * 8 + 2 * j + 1] = v[3];
    }
  }
  __syncthreads();
  const int which = t >> 6, c = t & 63;      // threads 0 .. 63 dgain, 64 .. 127 dshift
  const int64_t out = (int64_t(blockIdx.x) - a.N) * 64 + c;
  float* const dst = which == 0 ? dgain : which == 1 ? dshift : nullptr;
  if (dst != nullptr && out < a.C) {
    float v = comb[which][0][c];
    for (int w = 1; w < T / 32; ++w) v += comb[which][w][c];
    dst[out] = accumulate ? dst[out] + v : v;
  }
}

// out[c] (+)= sum over p of partial[p][c]: 32 groups of parts, p in order within
// each and eight loads in flight, the groups added in order.  32 columns per
// block.
__global__ void __launch_bounds__(1024) column_sum_kernel(float* out0, float* out1, const float* partial, int parts,
                                                          int64_t cols0, int64_t cols, int accumulate) {
  pdl_wait();
  pdl_trigger();
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int64_t c = int64_t(blockIdx.x) * 32 + lane;
  float v = 0.0f;
  if (c < cols) {
    const float* col = partial + c;
    int p = g;
    for (; p + 7 * 32 < parts; p += 8 * 32) {
      float t[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) t[k] = col[size_t(p + k * 32) * size_t(cols)];
#pragma unroll
      for (int k = 0; k < 8; ++k) v += t[k];
    }
    for (; p < parts; p += 32) v += col[size_t(p) * size_t(cols)];
  }
  s[g][lane] = v;
  __syncthreads();
  if (g == 0 && c < cols) {
    for (int k = 1; k < 32; ++k) v += s[k][lane];
    // columns [0, cols0) go to out0, the rest to out1; either may be absent
    float* dst = c < cols0 ? out0 : out1;
    const int64_t i = c < cols0 ? c : c - cols0;
    if (dst != nullptr) dst[i] = accumulate ? dst[i] + v : v;
  }
}

template <int T, int V, int BLOCK>
cudaError_t run_layernorm(const LnFwd& a, cudaStream_t s) {
  const int64_t rows = BLOCK / T;
  return launch_pdl(layernorm_kernel<T, V, BLOCK>, dim3(unsigned((a.N + rows - 1) / rows)), BLOCK, 0, s, a);
}

// Blocks per SM of the ring form: what their registers allow.  A row costs a
// block a barrier and the latencies around it whatever its length, so short
// rows need many blocks.
int ring_blocks_backward(int C) { return C <= 1024 ? 6 : C <= 2048 ? 4 : C <= 4096 ? 2 : 1; }

constexpr int kRingBytes = 208 * 1024;            // shared memory of an SM that the rings take

// Stages of a ring block with rows of `stage` bytes, and the kernel's permission to take that much.
cudaError_t ring_stages(const void* kernel, int stage, int blocks_per_sm, int* stages, bool (&set)[64]) {
  *stages = kRingBytes / blocks_per_sm / stage;
  if (*stages > kMaxStages) *stages = kMaxStages;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !set[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  return cudaSuccess;
}

template <bool CENTRED, int T, int V>
cudaError_t run_ring(NormBwd a, int blocks, cudaStream_t s) {
  static bool set[64] = {false};
  const int stage = a.C * 2 * (a.dres != nullptr ? 3 : 2);
  const cudaError_t e = ring_stages(reinterpret_cast<const void*>(norm_backward_kernel<CENTRED, T, V>), stage,
                                    ring_blocks_backward(a.C), &a.stages, set);
  if (e != cudaSuccess) return e;
  return launch_pdl(norm_backward_kernel<CENTRED, T, V>, dim3(unsigned(blocks)), T, size_t(a.stages) * size_t(stage), s, a);
}

template <bool CENTRED>
cudaError_t norm_backward(const NormBwd& a, int blocks, cudaStream_t s) {
  if (a.C <= 512) {
    if (a.C <= 256) return launch_pdl(norm_backward_warp_kernel<CENTRED, 1>, dim3(unsigned(blocks)), 256, 0, s, a);
    return launch_pdl(norm_backward_warp_kernel<CENTRED, 2>, dim3(unsigned(blocks)), 256, 0, s, a);
  }
  if (a.C <= 1024) return run_ring<CENTRED, 128, 1>(a, blocks, s);
  if (a.C <= 2048) return run_ring<CENTRED, 256, 1>(a, blocks, s);
  if (a.C <= 4096) return run_ring<CENTRED, 256, 2>(a, blocks, s);
  if (a.C <= 8192) return run_ring<CENTRED, 512, 2>(a, blocks, s);
  return run_ring<CENTRED, 512, 4>(a, blocks, s);
}

// Up to this many rows one launch that reads dy and r twice beats two (layer norm,
// us, one launch against two: 77 x 2048 2.1 / 5.2, about 512 x 4096 8.0 / 10.5,
// 512 x 1024 7.0 / 6.7, 512 x 256 4.9 / 3.9).
int64_t short_rows(int C) { return C <= 512 ? 256 : 512; }

template <bool CENTRED>
cudaError_t norm_backward_short(const NormBwd& a, float* dgain, float* dshift, bool accumulate, cudaStream_t s) {
  const dim3 grid(unsigned(a.N + (a.C + 63) / 64));
  const int acc = accumulate ? 1 : 0;
  if (a.C <= 2048) return launch_pdl(norm_backward_short_kernel<CENTRED, 128>, grid, 128, 0, s, a, dgain, dshift, acc);
  if (a.C <= 4096) return launch_pdl(norm_backward_short_kernel<CENTRED, 256>, grid, 256, 0, s, a, dgain, dshift, acc);
  if (a.C <= 8192) return launch_pdl(norm_backward_short_kernel<CENTRED, 512>, grid, 512, 0, s, a, dgain, dshift, acc);
  return launch_pdl(norm_backward_short_kernel<CENTRED, 1024>, grid, 1024, 0, s, a, dgain, dshift, acc);
}

}  // namespace

int norm_backward_blocks(int64_t N, int C) {
  // fixed for the 152 SMs of the device, so that the workspace size needs no device query
  const int64_t cap = int64_t(kNumSMsHint) * (C <= 512 ? 4 : ring_blocks_backward(C));
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
  const LnFwd a{res_out, y, mean, rstd, stats, res_in, x, gain, shift, eps, N, C};
  if (C <= 256) return run_layernorm<32, 1, 128>(a, s);
  if (C <= 512) return run_layernorm<32, 2, 128>(a, s);
  if (N >= 8 * int64_t(num_sms())) {
    if (C <= 1024) return run_layernorm<32, 4, 128>(a, s);
    if (C <= 2048) return run_layernorm<128, 2, 128>(a, s);
    if (C <= 4096) return run_layernorm<128, 4, 128>(a, s);
    if (C <= 8192) return run_layernorm<256, 4, 256>(a, s);
    return run_layernorm<512, 4, 512>(a, s);
  }
  if (C <= 1024) return run_layernorm<128, 1, 128>(a, s);
  if (C <= 2048) return run_layernorm<256, 1, 256>(a, s);
  if (C <= 4096) return run_layernorm<256, 2, 256>(a, s);
  if (C <= 8192) return run_layernorm<512, 2, 512>(a, s);
  return run_layernorm<1024, 2, 1024>(a, s);
}

cudaError_t launch_column_sum(float* out0, float* out1, const float* partial, int parts, int64_t cols0, int64_t cols,
                              bool accumulate, cudaStream_t s) {
  if (cols == 0) return cudaSuccess;
  return launch_pdl(column_sum_kernel, dim3(unsigned((cols + 31) / 32)), 1024, 0, s, out0, out1, partial, parts, cols0,
                    cols, accumulate ? 1 : 0);
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
  if (N <= short_rows(C) && dx != dy) {         // (its column sums read dy while rows of dx are written)
    const NormBwd b{dx, nullptr, stats, dy, dres, r, mean, rstd, gain, N, C, 0};
    return centred ? norm_backward_short<true>(b, dgain, dshift, accumulate, s)
                   : norm_backward_short<false>(b, dgain, nullptr, accumulate, s);
  }
  const int blocks = norm_backward_blocks(N, C);
  const NormBwd a{dx, partial, stats, dy, dres, r, mean, rstd, gain, N, C, 0};
  e = centred ? norm_backward<true>(a, blocks, s) : norm_backward<false>(a, blocks, s);
  if (e != cudaSuccess) return e;
  return launch_column_sum(dgain, dshift, partial, blocks, C, centred ? 2 * int64_t(C) : C, accumulate, s);
}

}  // namespace qffn
