// Row-scaled W8A16 GEMVs of the single-token FP8 decode FFN (metrale
// "dense_ffn_decode.rs", DenseFfnLayer::forward, FP8 arm: w8a16_gemv_dual
// for gate and up, silu_mul, w8a16_gemv for down).
//
//   out[r] = bf16(row_scale[r] * sum_k W[r,k] * x[k]),  W E4M3, x bf16.
//
// A team of TPR threads owns a row at a time: thread t holds the 16-byte
// chunks t, t+TPR, ... of the row and issues all of its loads (16-byte,
// non-allocating, one contiguous 16*TPR-byte span per load instruction)
// before using any, so every thread keeps the whole row in flight.  x sits
// in shared memory as bf16, the two 16-byte halves of each 32-byte chunk in
// separate planes so that a warp's 16-byte reads are consecutive words (no
// bank conflicts).  Products and sums are packed fp32x2 fmas: the E4M3 pairs
// go through the e4m3x2 -> f16x2 convert to float pairs, x pairs are widened
// from bf16 by shifts; even elements accumulate in the low half and odd ones
// in the high half.  (Staging x widened to fp32 instead was measured slower:
// twice the shared-memory reads for the same work.)  The per-row arithmetic
// (chunk order, pair order, halves added, warp butterfly, warps of a team in
// order) is the same
// code for the single and the dual form, so they agree bit for bit; the dual
// form reads x once for the gate and the up row of the same index.
//
// The fused-SiLU-input arm's down GEMV (w8a16_gemv_silu_input) reads g and u
// and forms h = bf16(silu(g) * u) while staging its input vector in shared
// memory, once per CTA, with the arithmetic of silu_mul; its output is the
// same as silu_mul followed by the plain GEMV.
//
// In the decode the dual GEMV applies silu_mul where g and u are produced and
// leaves h = bf16(silu(g) * u) in the gate buffer (the split-SiLU arm's
// buffer use); the down GEMV on h is a programmatic dependent launch whose
// CTAs start as the dual GEMV's CTAs retire and wait for h only right before
// reading it, its first weight loads issued before that wait.  The dual GEMV
// is itself a programmatic dependent launch; it issues its first weight loads
// before waiting for the preceding kernel only when the caller states that
// the weights are not being written by work that may still be running.
#include "common.cuh"
#include "launch.h"

namespace qffn {
namespace {

constexpr int kThreads = 256;
constexpr int kUSingle = 8;                // 16-byte loads in flight per thread
constexpr int kUDual = 4;                  //   (per matrix)
constexpr int kXU = 4;                     // input-vector loads in flight per thread

QFFN_DEVI uint64_t e4m3x2_to_f2(uint32_t two_codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(two_codes)));
  const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h));
  return f2_pack(f.x, f.y);
}

// acc += the 16 products of one weight chunk with its 16 x values (x as 16
// bf16 in two uint4), element pairs in order.
QFFN_DEVI void dot16(uint4 w, uint4 xa, uint4 xb, uint64_t& acc) {
  const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
  const uint32_t xw[8] = {xa.x, xa.y, xa.z, xa.w, xb.x, xb.y, xb.z, xb.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    acc = f2_fma(e4m3x2_to_f2(ww[j] & 0xFFFFu), bf16x2_to_f2(xw[2 * j]), acc);
    acc = f2_fma(e4m3x2_to_f2(ww[j] >> 16), bf16x2_to_f2(xw[2 * j + 1]), acc);
  }
}

struct Gemv {
  uint16_t* out[2];
  int even;                  // rows split evenly over the whole grid: one step per CTA
  const uint16_t* x;         // input bf16 [cols] (SILU_IN: the gate vector g)
  const uint16_t* x_up;      // SILU_IN: the up vector u; input = bf16(silu(g) * u)
  const uint8_t* w[2];
  const float* s[2];
  int rows, cols;
};

// SILU (dual only): the gate output slot receives h = bf16(silu(g) * u)
// instead of g -- the decode's silu_mul applied where g and u are produced,
// as the split-SiLU arm leaves h in the gate buffer.
// Four CTAs (1024 threads) per SM: 64 registers a thread.
template <bool DUAL, bool SILU, int TPR, bool SILU_IN = false>
__global__ void __launch_bounds__(kThreads, 4) gemv_kernel(const Gemv G, const bool early) {
  constexpr int kU = DUAL ? kUDual : kUSingle;
  extern __shared__ uint4 xs[];
  __shared__ float red[2][kThreads / 32];
  constexpr int RPB = kThreads / TPR;   // rows per block step
  constexpr int WPR = TPR / 32;         // warps per row
  const int rows = G.rows, cols = G.cols;
  const int nvec = cols >> 3;
  const int nchunk = cols >> 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = threadIdx.x / TPR, t = threadIdx.x % TPR;

  // The weights do not depend on the preceding kernel: with `early`, each team
  // issues the first batch of its first row before waiting for x.
  uint4 a[kU], b[kU];
  bool have = false;
  if (early) {
    const int row = G.even ? int(int64_t(blockIdx.x) * rows / gridDim.x) + sub : blockIdx.x * RPB + sub;
    const int rend = G.even ? int(int64_t(blockIdx.x + 1) * rows / gridDim.x) : rows;
    if (row < rend) {
      const uint8_t* r0 = G.w[0] + size_t(row) * size_t(cols);
      const uint8_t* r1 = DUAL ? G.w[1] + size_t(row) * size_t(cols) : nullptr;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int cc = t + TPR * u;
        if (cc < nchunk) {
          a[u] = ld16_stream(r0 + size_t(cc) * 16);
          if (DUAL) b[u] = ld16_stream(r1 + size_t(cc) * 16);
        }
      }
      have = true;
    }
  }
  pdl_wait();                        // x may come from the preceding kernel
  pdl_trigger();
  // Stage x: a thread issues up to kXU of its 16-byte loads before its first
  // shared-memory store, so staging costs one L2 round trip per kXU vectors
  // rather than one per vector (7 per thread for a 14336-long input).
  constexpr int kX = SILU_IN ? 2 : kXU;   // SiLU staging holds two vectors per load
  for (int i0 = threadIdx.x; i0 < nvec; i0 += kThreads * kX) {
    uint4 v[kX], vu[kX];
#pragma unroll
    for (int j = 0; j < kX; ++j) {
      const int i = i0 + j * kThreads;
      if (i < nvec) {
        v[j] = ld16_once(G.x + size_t(i) * 8);
        if constexpr (SILU_IN) vu[j] = ld16_once(G.x_up + size_t(i) * 8);
      }
    }
#pragma unroll
    for (int j = 0; j < kX; ++j) {
      const int i = i0 + j * kThreads;
      if (i < nvec) {
        // part-major layout: part p of chunk c at xs[p * nchunk + c], so the
        // lanes of a warp (consecutive chunks) read consecutive 16-byte words
        const int c = i >> 1, h = i & 1;
        if constexpr (SILU_IN) xs[h * nchunk + c] = swiglu8(v[j], vu[j]);
        else xs[h * nchunk + c] = v[j];
      }
    }
  }
  __syncthreads();

  const int base0 = G.even ? int(int64_t(blockIdx.x) * rows / gridDim.x) : blockIdx.x * RPB;
  const int rlim = G.even ? int(int64_t(blockIdx.x + 1) * rows / gridDim.x) : rows;
  const int bstep = G.even ? rows : gridDim.x * RPB;
  for (int base = base0; base < rlim; base += bstep) {
    const int row = base + sub;
    uint64_t acc0 = 0ull, acc1 = 0ull;
    if (row < rlim) {
      const uint8_t* r0 = G.w[0] + size_t(row) * size_t(cols);
      const uint8_t* r1 = DUAL ? G.w[1] + size_t(row) * size_t(cols) : nullptr;
      for (int c = t; c < nchunk; c += TPR * kU) {
        if (!have) {
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            const int cc = c + TPR * u;
            if (cc < nchunk) {
              a[u] = ld16_stream(r0 + size_t(cc) * 16);
              if (DUAL) b[u] = ld16_stream(r1 + size_t(cc) * 16);
            }
          }
        }
        have = false;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int cc = c + TPR * u;
          if (cc < nchunk) {
            const uint4 xa = xs[cc], xb = xs[nchunk + cc];
            dot16(a[u], xa, xb, acc0);
            if (DUAL) dot16(b[u], xa, xb, acc1);
          }
        }
      }
    }
    float s0, s1 = 0.0f;
    {
      float lo, hi;
      f2_unpack(acc0, lo, hi);
      s0 = warp_sum(lo + hi);
      if (DUAL) {
        f2_unpack(acc1, lo, hi);
        s1 = warp_sum(lo + hi);
      }
    }
    if (WPR > 1) {
      if (lane == 0) {
        red[0][warp] = s0;
        red[1][warp] = s1;
      }
      __syncthreads();
      if (t == 0) {
        float a0 = 0.0f, a1 = 0.0f;
        for (int w = 0; w < WPR; ++w) {
          a0 += red[0][warp + w];
          a1 += red[1][warp + w];
        }
        s0 = a0;
        s1 = a1;
      }
      __syncthreads();
    }
    if (t == 0 && row < rlim) {
      const uint16_t gb = f32_to_bf16(G.s[0][row] * s0);
      if (DUAL) {
        const uint16_t ub = f32_to_bf16(G.s[1][row] * s1);
        G.out[0][row] = SILU ? f32_to_bf16(silu_mul_f32(bf16_to_f32(gb), bf16_to_f32(ub))) : gb;
        G.out[1][row] = ub;
      } else {
        G.out[0][row] = gb;
      }
    }
  }
}

template <bool DUAL, bool SILU, int TPR, bool SILU_IN = false>
cudaError_t launch_t(const Gemv& G, bool pdl, bool early, cudaStream_t s) {
  const size_t smem = size_t(G.cols) * 2;
  auto fn = gemv_kernel<DUAL, SILU, TPR, SILU_IN>;
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
  }
  int per_sm = 0;
  cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, fn, kThreads, smem);
  if (e != cudaSuccess) return e;
  if (per_sm < 1) per_sm = 1;
  constexpr int RPB = kThreads / TPR;
  const int needed = (G.rows + RPB - 1) / RPB;
  const int cap = num_sms() * per_sm;
  cudaLaunchConfig_t cfg = {};
  // Fewer rows than one step of the full grid (the decode's down GEMV: 4096
  // rows of 8 per CTA step, 512 CTAs on 608 slots): the rows are split evenly
  // over the whole grid, 6 or 7 per CTA, instead of 8 per CTA on part of it,
  // so every SM gets about the same share (measured: 32.5 -> 32.2 us per
  // decode call, 33.7 -> 32.8 us without the stable-weights flag).
  Gemv G2 = G;
  G2.even = (!DUAL && needed < cap) ? 1 : 0;
  cfg.gridDim = dim3(G2.even ? cap : (needed < cap ? needed : cap));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, fn, G2, early);
}

template <bool DUAL, bool SILU>
cudaError_t launch_d(const Gemv& G, bool pdl, bool early, cudaStream_t s) {
  // one warp per row at every row length: the memory system is kept busy by
  // the number of rows in flight, and no cross-warp sums are needed
  return launch_t<DUAL, SILU, 32>(G, pdl, early, s);
}

}  // namespace

cudaError_t launch_gemv(uint16_t* out0, uint16_t* out1, const uint16_t* x, const uint8_t* w0,
                        const float* s0, const uint8_t* w1, const float* s1, int64_t rows,
                        int64_t cols, bool pdl, cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  Gemv G{};
  G.out[0] = out0;
  G.out[1] = out1;
  G.x = x;
  G.w[0] = w0;
  G.s[0] = s0;
  G.w[1] = w1;
  G.s[1] = s1;
  G.rows = int(rows);
  G.cols = int(cols);
  // standalone, or behind this library's own dual GEMV: the weights may be read early
  return w1 != nullptr ? launch_d<true, false>(G, pdl, true, s) : launch_d<false, false>(G, pdl, true, s);
}

cudaError_t launch_gemv_silu_input(uint16_t* out, const uint16_t* g, const uint16_t* u,
                                   const uint8_t* w, const float* row_scale, int64_t rows,
                                   int64_t cols, cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  Gemv G{};
  G.out[0] = out;
  G.x = g;
  G.x_up = u;
  G.w[0] = w;
  G.s[0] = row_scale;
  G.rows = int(rows);
  G.cols = int(cols);
  return launch_t<false, false, 32, true>(G, false, true, s);
}

cudaError_t launch_decode(uint16_t* out, const uint16_t* x, const uint8_t* w_gate,
                          const float* s_gate, const uint8_t* w_up, const float* s_up,
                          const uint8_t* w_down, const float* s_down, int64_t C, int64_t H,
                          uint16_t* g, uint16_t* u, bool early, cudaStream_t s) {
  Gemv G{};
  G.out[0] = g;                      // receives h = bf16(silu(g) * u)
  G.out[1] = u;
  G.x = x;
  G.w[0] = w_gate;
  G.s[0] = s_gate;
  G.w[1] = w_up;
  G.s[1] = s_up;
  G.rows = int(H);
  G.cols = int(C);
  // the dual GEMV reads its weights before the preceding kernel has finished
  // only when the caller allows it (`early`); the down GEMV's launch can start
  // only once every dual CTA has passed its own wait, so whatever preceded the
  // call has finished by then and its early weight loads are always safe
  cudaError_t e = launch_d<true, true>(G, true, early, s);
  if (e != cudaSuccess) return e;
  return launch_gemv(out, nullptr, g, w_down, s_down, nullptr, nullptr, C, H, true, s);
}

cudaError_t decode_take_status(unsigned int* status) {
  *status = 0;      // the decode kernels have no bounded waits
  return cudaSuccess;
}

}  // namespace qffn
