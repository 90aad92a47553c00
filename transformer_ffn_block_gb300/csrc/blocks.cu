// E4M3 with a power-of-two scale for each block of 128 values (sm_103a):
//
//   quantize_blocks         rows of bf16 -> codes and scales
//   swiglu_quantize_blocks  h = silu(g) * u -> codes and scales (and bf16 h)
//   rmsnorm_quantize_blocks r = res + x; y = r * rstd * gain -> codes and scales (and bf16 y)
//   quantize_weight_blocks  weights, a scale for each 128 x 128
//
// A block's scale is 2^(c - 127), stored as the E8M0 code c that the tensor cores
// take: the smallest power of two that holds the block's abs-max within E4M3's
// 448 = 1.75 * 2^8.  With amax = m * 2^e (1 <= m < 2) that is 2^(e - 8), or 2^(e - 7)
// where m > 1.75: read off the bits of amax, no logarithm and no division.  The
// codes are v * 2^(127 - c), an exact product, rounded once.  The values that are
// quantised are the fp32 ones (h, y before any rounding to bf16).
//
// All are bound by HBM.  A lane holds 8 values (16-byte loads, 8-byte stores of
// codes), so 16 lanes hold a block and four shuffles give its abs-max.
#include "act.cuh"
#include "common.cuh"
#include "launch.h"

namespace qffn {
namespace {

constexpr int kThreads = 256;

// Abs-max over the 16 lanes of a block, on the bits of |v|: ordered like the
// values, with infinity and NaN above all finite ones.
QFFN_DEVI uint32_t max16(uint32_t m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
// E8M0 code of a block's abs-max (its bits): 127 for zeros, 255 (NaN) where a value is not finite.
QFFN_DEVI uint32_t scale_code(uint32_t amax) {
  if (amax >= 0x7F800000u) return 255u;
  if (amax == 0u) return 127u;
  const int c = int(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return uint32_t(max(c, 0));
}
// 2^(127 - c); NaN for 255 (whose codes are all NaN)
QFFN_DEVI float code_inverse(uint32_t c) { return __uint_as_float(c == 255u ? 0x7FC00000u : (254u - c) << 23); }

// Eight values as four pairs.
using Eight = uint64_t[4];

// max(m, |a|, |b|), NaN if one is
QFFN_DEVI float max_abs(float m, float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}
// Abs-max of the eight, as bits.
QFFN_DEVI uint32_t amax8(const Eight& v) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a, b;
    f2_unpack(v[j], a, b);
    m = max_abs(m, a, b);
  }
  return __float_as_uint(m);
}
QFFN_DEVI uint2 codes8(const Eight& v, float inv) {
  uint32_t p[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a, b;
    f2_unpack(f2_mul(v[j], f2_dup(inv)), a, b);
    p[j] = f32x2_to_e4m3x2(a, b);
  }
  return make_uint2(p[0] | (p[1] << 16), p[2] | (p[3] << 16));
}
QFFN_DEVI void unpack8(uint4 w, Eight& v) {
  v[0] = bf16x2_to_f2(w.x);
  v[1] = bf16x2_to_f2(w.y);
  v[2] = bf16x2_to_f2(w.z);
  v[3] = bf16x2_to_f2(w.w);
}
QFFN_DEVI uint32_t pack2(uint64_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return pack_bf16x2(a, b);
}
QFFN_DEVI uint4 pack8(const Eight& v) { return make_uint4(pack2(v[0]), pack2(v[1]), pack2(v[2]), pack2(v[3])); }
QFFN_DEVI void stg8(void* p, uint2 v) { *reinterpret_cast<uint2*>(p) = v; }

// ------------------------------------------------------------------ rows, and SwiGLU
// Chunks of 8 values, a row padded to whole blocks of 16 chunks, so that the 16
// lanes of a block are in one half warp; a thread takes kFlight of them, all loads in
// flight at once.  The row of a chunk is a product with `magic` = floor(2^64 / chunks per
// row) + 1: exact for fewer than 2^44 chunks, as the divisor is at most 2^17.
// Measured: rows of 8192 x 8192 31.5 us (6.4 TB/s), SwiGLU 8192 x 14336 87.8 us (6.7 TB/s; with
// scalar arithmetic 123), 37 x 2048 2.3 us, most of it a launch.
constexpr int kFlight = 4;
template <bool SWIGLU>
__global__ void __launch_bounds__(kThreads, SWIGLU ? 4 : 6) rows_kernel(uint16_t* h, uint8_t* q, uint8_t* scale,
                                                                        const uint16_t* in, int64_t rows, int64_t cols,
                                                                        uint64_t magic) {
  const int64_t blocks = (cols + 127) >> 7;
  const int per_row = int(blocks) * 16, chunks = int(cols >> 3);
  const uint64_t at = uint64_t(blockIdx.x) * (kThreads * kFlight) + threadIdx.x;
  pdl_wait();
  pdl_trigger();
  uint4 a[kFlight], b[kFlight];
#pragma unroll
  for (int k = 0; k < kFlight; ++k) {
    const int64_t row = int64_t(__umul64hi(at + k * kThreads, magic));
    const int c = int(at + k * kThreads - uint64_t(row) * uint64_t(per_row));
    a[k] = b[k] = make_uint4(0, 0, 0, 0);
    if (row < rows && c < chunks) {
      const uint16_t* p = in + (SWIGLU ? 2 * row : row) * cols + c * 8;
      a[k] = ld16_stream(p);
      if (SWIGLU) b[k] = ld16_stream(p + cols);
    }
  }
#pragma unroll
  for (int k = 0; k < kFlight; ++k) {
    Eight v;
    unpack8(a[k], v);
    if (SWIGLU) {
      Eight u;
      unpack8(b[k], u);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = f2_mul(act_f2<ACT_SILU>(v[j]), u[j]);
    }
    const uint32_t code = scale_code(max16(amax8(v)));
    const int64_t row = int64_t(__umul64hi(at + k * kThreads, magic));
    const int c = int(at + k * kThreads - uint64_t(row) * uint64_t(per_row));
    if (row < rows && c < chunks) {
      const int64_t o = row * cols + c * 8;
      stg8(q + o, codes8(v, code_inverse(code)));
      if (SWIGLU && h != nullptr) stg16(h + o, pack8(v));
      if ((c & 15) == 0) scale[row * blocks + (c >> 4)] = uint8_t(code);
    }
  }
}

// ------------------------------------------------------------------ RMS norm
// TPR threads per row, which keep the row's V chunks of 8 values in registers
// between the sum of squares and the quantisation; rows of up to 1024 values take a
// warp each and no barrier.  Short rows go R at a time, so that a thread has about
// four loads in flight.
// FEW: the gain is requested with the row, for calls of few rows, which wait once; else
// after the sums, from L1, which leaves registers for more rows at a time (4096 x 16384 91 us
// with the gain in registers, 78 from L1).  Measured with a residual: 8192 x 4096 38.7 us (6.1
// TB/s), 16384 x 1024 21 us (5.6), 1 x 4096 2.1 us; without one, with half the loads in flight,
// 8192 x 4096 20.4 us (4.9).
template <int V, bool FEW>
constexpr int rows_at_once() { return FEW || V > 2 ? 1 : V == 2 ? 2 : 4; }

template <int TPR, int V, bool FEW>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR, (FEW || V <= 2 ? 1024 : 1280) / (TPR < 128 ? 128 : TPR)) rmsnorm_blocks_kernel(
    uint16_t* res_out, uint16_t* y, uint8_t* q, uint8_t* scale, float* rstd, const uint16_t* res_in,
    const uint16_t* x, const uint16_t* gain, float eps, int64_t N, int C, float inv_c) {
  constexpr int TEAMS = TPR < 128 ? 128 / TPR : 1, R = rows_at_once<V, FEW>();
  __shared__ float red[R][TPR / 32];
  const int tid = threadIdx.x % TPR;
  const int64_t row0 = (int64_t(blockIdx.x) * TEAMS + threadIdx.x / TPR) * R;
  const int chunks = C >> 3, blocks = (C + 127) >> 7;
  pdl_wait();
  const uint16_t* const gains = behind_wait(gain);
  pdl_trigger();
  uint4 r[R][V], g[V];
#pragma unroll
  for (int k = 0; k < R; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * TPR;
      r[k][i] = make_uint4(0, 0, 0, 0);
      if (row0 + k < N && c < chunks) r[k][i] = ld16_stream(x + size_t(row0 + k) * size_t(C) + size_t(c) * 8);
      if (k == 0) {
        g[i] = make_uint4(0, 0, 0, 0);
        if (FEW && c < chunks) g[i] = ld16_settled(gains + size_t(c) * 8);
      }
    }
  if (res_in != nullptr) {
    uint4 a[R][V];
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = tid + i * TPR;
        a[k][i] = make_uint4(0, 0, 0, 0);
        if (row0 + k < N && c < chunks) a[k][i] = ld16_stream(res_in + size_t(row0 + k) * size_t(C) + size_t(c) * 8);
      }
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = tid + i * TPR;
        Eight s, t;
        unpack8(a[k][i], s);
        unpack8(r[k][i], t);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = f2_add(s[j], t[j]);
        r[k][i] = pack8(s);
        if (row0 + k < N && c < chunks) stg16(res_out + size_t(row0 + k) * size_t(C) + size_t(c) * 8, r[k][i]);
      }
  }
  float ss[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    uint64_t squares[2] = {0ull, 0ull};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      Eight v;
      unpack8(r[k][i], v);
#pragma unroll
      for (int j = 0; j < 4; ++j) squares[j & 1] = f2_fma(v[j], v[j], squares[j & 1]);
    }
    float odd;
    f2_unpack(f2_add(squares[0], squares[1]), ss[k], odd);
    ss[k] = warp_sum(ss[k] + odd);
  }
  if (TPR > 32) {
#pragma unroll
    for (int k = 0; k < R; ++k)
      if ((threadIdx.x & 31) == 0) red[k][threadIdx.x >> 5] = ss[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < R; ++k) {
      ss[k] = red[k][0];
#pragma unroll
      for (int w = 1; w < TPR / 32; ++w) ss[k] += red[k][w];
    }
  }
  float rs[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    rs[k] = rsqrtf(fmaf(ss[k], inv_c, eps));
    if (row0 + k < N && tid == 0) rstd[row0 + k] = rs[k];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = tid + i * TPR;
    if (!FEW && c < chunks) g[i] = ld16_once(gains + size_t(c) * 8);
    Eight w;
    unpack8(g[i], w);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const bool in = row0 + k < N && c < chunks;
      Eight v;
      unpack8(r[k][i], v);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = f2_mul(f2_mul(v[j], f2_dup(rs[k])), w[j]);
      // (lanes without a chunk have zeros, also where rs is not finite)
      const uint32_t code = scale_code(max16(in ? amax8(v) : 0u));
      if (in) {
        const size_t o = size_t(row0 + k) * size_t(C) + size_t(c) * 8;
        stg8(q + o, codes8(v, code_inverse(code)));
        if (y != nullptr) stg16(y + o, pack8(v));
        if ((tid & 15) == 0) scale[size_t(row0 + k) * size_t(blocks) + size_t(c >> 4)] = uint8_t(code);
      }
    }
  }
}

// ------------------------------------------------------------------ weights
// One CTA per 128 x 128 of matrix blockIdx.z: a thread holds 8 values of each of 8 rows.
// Measured: 8192 x 8192 38.5 us (5.2 TB/s), once per set of weights.
__global__ void __launch_bounds__(kThreads) weight_blocks_kernel(uint8_t* q, uint8_t* scale, const uint16_t* w,
                                                                 int64_t rows, int64_t cols, int64_t row_blocks) {
  __shared__ uint32_t red[kThreads / 32];
  const int64_t col_blocks = gridDim.x;
  const int64_t m = blockIdx.z;
  const uint16_t* src = w + m * rows * cols;
  pdl_wait();
  pdl_trigger();
  for (int64_t b = blockIdx.y; b < row_blocks; b += gridDim.y) {
    const int64_t row0 = b * 128 + (threadIdx.x >> 4), col = int64_t(blockIdx.x) * 128 + (threadIdx.x & 15) * 8;
    uint4 v[8];
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t row = row0 + 16 * i;
      v[i] = make_uint4(0, 0, 0, 0);
      if (row < rows && col < cols) v[i] = ld16_stream(src + row * cols + col);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      Eight f;
      unpack8(v[i], f);
      top = max(top, amax8(f));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) top = max(top, red[k]);
    const uint32_t code = scale_code(top);
    const float inv = code_inverse(code);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t row = row0 + 16 * i;
      Eight f;
      unpack8(v[i], f);
      if (row < rows && col < cols) stg8(q + (m * rows + row) * cols + col, codes8(f, inv));
    }
    if (threadIdx.x == 0) scale[(m * row_blocks + b) * col_blocks + blockIdx.x] = uint8_t(code);
  }
}

template <int TPR, int V, bool FEW, typename... Args>
cudaError_t run_rmsnorm(int64_t N, int C, cudaStream_t s, Args... args) {
  constexpr int TEAMS = TPR < 128 ? 128 / TPR : 1, BLOCK = TPR < 128 ? 128 : TPR, ROWS = TEAMS * rows_at_once<V, FEW>();
  return launch_pdl(rmsnorm_blocks_kernel<TPR, V, FEW>, dim3(unsigned((N + ROWS - 1) / ROWS)), BLOCK, 0, s, args..., N, C,
                    1.0f / float(C));
}
// A warp per row up to 1024 values, then 128 threads up to 4096, then as many, in steps of 64, as
// hold the row in four chunks each, so that few are idle (of 9216 values 320, not 512: 49.9 us, so 39.3).
template <bool FEW, typename... Args>
cudaError_t choose_rmsnorm(int64_t N, int C, cudaStream_t s, Args... args) {
  const int chunks = C / 8;
  if (chunks <= 32) return run_rmsnorm<32, 1, FEW>(N, C, s, args...);
  if (chunks <= 64) return run_rmsnorm<32, 2, FEW>(N, C, s, args...);
  if (chunks <= 96) return run_rmsnorm<32, 3, FEW>(N, C, s, args...);
  if (chunks <= 128) return run_rmsnorm<32, 4, FEW>(N, C, s, args...);
  if (chunks <= 256) return run_rmsnorm<128, 2, FEW>(N, C, s, args...);
  if (chunks <= 384) return run_rmsnorm<128, 3, FEW>(N, C, s, args...);
  switch ((chunks + 255) / 256) {
    case 2: return run_rmsnorm<128, 4, FEW>(N, C, s, args...);
    case 3: return run_rmsnorm<192, 4, FEW>(N, C, s, args...);
    case 4: return run_rmsnorm<256, 4, FEW>(N, C, s, args...);
    case 5: return run_rmsnorm<320, 4, FEW>(N, C, s, args...);
    case 6: return run_rmsnorm<384, 4, FEW>(N, C, s, args...);
    case 7: return run_rmsnorm<448, 4, FEW>(N, C, s, args...);
    default: return run_rmsnorm<512, 4, FEW>(N, C, s, args...);
  }
}

template <bool SWIGLU>
cudaError_t run_rows(uint16_t* h, uint8_t* q, uint8_t* scale, const uint16_t* in, int64_t rows, int64_t cols,
                     cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  const int64_t per_row = (cols + 127) / 128 * 16;
  const int64_t grid = (rows * per_row + kThreads * kFlight - 1) / (kThreads * kFlight);
  if (grid > (int64_t(1) << 31) - 1) return cudaErrorInvalidValue;
  // (per_row >= 16 divides 2^64 at most evenly: then this is the quotient + 1 too)
  const uint64_t magic = ~uint64_t(0) / uint64_t(per_row) + 1 + ((per_row & (per_row - 1)) == 0 ? 1 : 0);
  return launch_pdl(rows_kernel<SWIGLU>, dim3(unsigned(grid)), kThreads, 0, s, h, q, scale, in, rows, cols, magic);
}

}  // namespace

cudaError_t launch_quantize_blocks(uint8_t* q, uint8_t* scale, const uint16_t* in, int64_t rows, int64_t cols,
                                   cudaStream_t s) {
  return run_rows<false>(nullptr, q, scale, in, rows, cols, s);
}

cudaError_t launch_swiglu_quantize_blocks(uint16_t* h, uint8_t* q, uint8_t* scale, const uint16_t* gate_up, int64_t N,
                                          int64_t H, cudaStream_t s) {
  return run_rows<true>(h, q, scale, gate_up, N, H, s);
}

cudaError_t launch_quantize_weight_blocks(uint8_t* q, uint8_t* scale, const uint16_t* w, int64_t count, int64_t rows,
                                          int64_t cols, cudaStream_t s) {
  if (count == 0 || rows == 0) return cudaSuccess;
  const int64_t row_blocks = (rows + 127) / 128;
  const dim3 grid(unsigned((cols + 127) / 128), unsigned(row_blocks < 65535 ? row_blocks : 65535), unsigned(count));
  return launch_pdl(weight_blocks_kernel, grid, kThreads, 0, s, q, scale, w, rows, cols, row_blocks);
}

cudaError_t launch_rmsnorm_quantize_blocks(uint16_t* res_out, uint16_t* y, uint8_t* q, uint8_t* scale, float* rstd,
                                           const uint16_t* res_in, const uint16_t* x, const uint16_t* gain, float eps,
                                           int64_t N, int C, cudaStream_t s) {
  if (N == 0) return cudaSuccess;
  if (N * C <= int64_t(num_sms()) * 32768)
    return choose_rmsnorm<true>(N, C, s, res_out, y, q, scale, rstd, res_in, x, gain, eps);
  return choose_rmsnorm<false>(N, C, s, res_out, y, q, scale, rstd, res_in, x, gain, eps);
}

}  // namespace qffn
