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

QFFN_DEVI uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
QFFN_DEVI uint32_t amax8(const float (&v)[8]) {
  uint32_t m = abs_bits(v[0]);
#pragma unroll
  for (int j = 1; j < 8; ++j) m = max(m, abs_bits(v[j]));
  return m;
}
QFFN_DEVI uint2 codes8(const float (&v)[8], float inv) {
  uint32_t p[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) p[j] = f32x2_to_e4m3x2(v[2 * j] * inv, v[2 * j + 1] * inv);
  return make_uint2(p[0] | (p[1] << 16), p[2] | (p[3] << 16));
}
QFFN_DEVI void unpack8(uint4 w, float (&v)[8]) {
  const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = bf16_lo(a[j]);
    v[2 * j + 1] = bf16_hi(a[j]);
  }
}
QFFN_DEVI uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
QFFN_DEVI void stg8(void* p, uint2 v) { *reinterpret_cast<uint2*>(p) = v; }

// ------------------------------------------------------------------ rows, and SwiGLU
// Chunks of 8 values, a row padded to whole blocks of 16 chunks, so that the 16
// lanes of a block are in one half warp; each thread strides over all of them,
// kFlight at a time.  Row and column advance by addition: one division per thread.
constexpr int kFlight = 4;
template <bool SWIGLU>
__global__ void __launch_bounds__(kThreads) rows_kernel(uint16_t* h, uint8_t* q, uint8_t* scale, const uint16_t* in,
                                                        int64_t rows, int64_t cols) {
  const int64_t blocks = (cols + 127) >> 7, per_row = blocks * 16, chunks = cols >> 3;
  const int64_t stride = int64_t(gridDim.x) * kThreads;
  const int64_t at = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  int64_t row = at / per_row, c = at - row * per_row;
  const int64_t drow = stride / per_row, dc = stride - drow * per_row;
  pdl_wait();
  pdl_trigger();
  // (the two halves of a warp may be at different rows, but leave together: a row
  // beyond the last is computed as zeros and not stored)
  while (__any_sync(0xffffffffu, row < rows)) {
    uint4 a[kFlight], b[kFlight];
    int64_t rr[kFlight], cc[kFlight];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      rr[k] = row;
      cc[k] = c;
      a[k] = b[k] = make_uint4(0, 0, 0, 0);
      if (row < rows && c < chunks) {
        const uint16_t* p = in + (SWIGLU ? 2 * row : row) * cols + c * 8;
        a[k] = ld16_stream(p);
        if (SWIGLU) b[k] = ld16_stream(p + cols);
      }
      row += drow;
      c += dc;
      if (c >= per_row) {
        c -= per_row;
        ++row;
      }
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      float v[8];
      unpack8(a[k], v);
      if (SWIGLU) {
        float u[8];
        unpack8(b[k], u);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = silu_mul_f32(v[j], u[j]);
      }
      const uint32_t code = scale_code(max16(amax8(v)));
      if (rr[k] >= rows) continue;
      if (cc[k] < chunks) {
        const int64_t o = rr[k] * cols + cc[k] * 8;
        stg8(q + o, codes8(v, code_inverse(code)));
        if (SWIGLU && h != nullptr) stg16(h + o, pack8(v));
      }
      if ((threadIdx.x & 15) == 0) scale[rr[k] * blocks + (cc[k] >> 4)] = uint8_t(code);
    }
  }
}

// ------------------------------------------------------------------ RMS norm
// TPR threads per row, which keep the row's V chunks of 8 values in registers
// between the sum of squares and the quantisation; rows of up to 1024 values take a
// warp each and no barrier.
template <int TPR, int V>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) rmsnorm_blocks_kernel(
    uint16_t* res_out, uint16_t* y, uint8_t* q, uint8_t* scale, float* rstd, const uint16_t* res_in,
    const uint16_t* x, const uint16_t* gain, float eps, int64_t N, int C) {
  constexpr int ROWS = TPR < 128 ? 128 / TPR : 1;
  __shared__ float red[TPR / 32];
  const int tid = threadIdx.x % TPR;
  const int64_t row = int64_t(blockIdx.x) * ROWS + threadIdx.x / TPR;
  const int chunks = C >> 3, blocks = (C + 127) >> 7;
  const bool live = row < N;
  const size_t base = size_t(row) * size_t(C);
  pdl_wait();
  const uint16_t* const gains = behind_wait(gain);
  pdl_trigger();
  uint4 r[V], g[V];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = tid + i * TPR;
    r[i] = g[i] = make_uint4(0, 0, 0, 0);
    if (live && c < chunks) {
      r[i] = ld16_stream(x + base + size_t(c) * 8);
      g[i] = ld16_settled(gains + size_t(c) * 8);
    }
  }
  if (res_in != nullptr) {
    uint4 a[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * TPR;
      a[i] = make_uint4(0, 0, 0, 0);
      if (live && c < chunks) a[i] = ld16_stream(res_in + base + size_t(c) * 8);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * TPR;
      float s[8], t[8];
      unpack8(a[i], s);
      unpack8(r[i], t);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += t[j];
      r[i] = pack8(s);
      if (live && c < chunks) stg16(res_out + base + size_t(c) * 8, r[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float v[8];
    unpack8(r[i], v);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
  }
  ss = warp_sum(ss);
  if (TPR > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = ss;
    __syncthreads();
    ss = red[0];
#pragma unroll
    for (int w = 1; w < TPR / 32; ++w) ss += red[w];
  }
  const float rs = 1.0f / sqrtf(ss / float(C) + eps);
  if (live && tid == 0) rstd[row] = rs;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = tid + i * TPR;
    float v[8], w[8];
    unpack8(r[i], v);
    unpack8(g[i], w);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] * rs * w[j];
    const bool in = live && c < chunks;
    // (lanes without a chunk have zeros, also where rs is not finite)
    const uint32_t code = scale_code(max16(in ? amax8(v) : 0u));
    if (in) {
      const size_t o = base + size_t(c) * 8;
      stg8(q + o, codes8(v, code_inverse(code)));
      if (y != nullptr) stg16(y + o, pack8(v));
      if ((tid & 15) == 0) scale[size_t(row) * size_t(blocks) + size_t(c >> 4)] = uint8_t(code);
    }
  }
}

// ------------------------------------------------------------------ weights
// One CTA per 128 x 128 of matrix blockIdx.z: a thread holds 8 values of each of 8 rows.
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
      float f[8];
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
      float f[8];
      unpack8(v[i], f);
      if (row < rows && col < cols) stg8(q + (m * rows + row) * cols + col, codes8(f, inv));
    }
    if (threadIdx.x == 0) scale[(m * row_blocks + b) * col_blocks + blockIdx.x] = uint8_t(code);
  }
}

template <int TPR>
cudaError_t run_rmsnorm(uint16_t* res_out, uint16_t* y, uint8_t* q, uint8_t* scale, float* rstd,
                        const uint16_t* res_in, const uint16_t* x, const uint16_t* gain, float eps, int64_t N, int C,
                        cudaStream_t s) {
  constexpr int ROWS = TPR < 128 ? 128 / TPR : 1, BLOCK = TPR < 128 ? 128 : TPR;
  const dim3 grid(unsigned((N + ROWS - 1) / ROWS));
  switch ((C / 8 + TPR - 1) / TPR) {
    case 1: return launch_pdl(rmsnorm_blocks_kernel<TPR, 1>, grid, BLOCK, 0, s, res_out, y, q, scale, rstd, res_in, x, gain, eps, N, C);
    case 2: return launch_pdl(rmsnorm_blocks_kernel<TPR, 2>, grid, BLOCK, 0, s, res_out, y, q, scale, rstd, res_in, x, gain, eps, N, C);
    case 3: return launch_pdl(rmsnorm_blocks_kernel<TPR, 3>, grid, BLOCK, 0, s, res_out, y, q, scale, rstd, res_in, x, gain, eps, N, C);
    default: return launch_pdl(rmsnorm_blocks_kernel<TPR, 4>, grid, BLOCK, 0, s, res_out, y, q, scale, rstd, res_in, x, gain, eps, N, C);
  }
}

template <bool SWIGLU>
cudaError_t run_rows(uint16_t* h, uint8_t* q, uint8_t* scale, const uint16_t* in, int64_t rows, int64_t cols,
                     cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  const int64_t slots = rows * ((cols + 127) / 128) * 16;
  int64_t grid = (slots + kThreads - 1) / kThreads;
  const int64_t cap = int64_t(num_sms()) * 8;
  if (grid > cap) grid = cap;
  return launch_pdl(rows_kernel<SWIGLU>, dim3(unsigned(grid)), kThreads, 0, s, h, q, scale, in, rows, cols);
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
  if (C <= 1024) return run_rmsnorm<32>(res_out, y, q, scale, rstd, res_in, x, gain, eps, N, C, s);
  if (C <= 4096) return run_rmsnorm<128>(res_out, y, q, scale, rstd, res_in, x, gain, eps, N, C, s);
  if (C <= 8192) return run_rmsnorm<256>(res_out, y, q, scale, rstd, res_in, x, gain, eps, N, C, s);
  return run_rmsnorm<512>(res_out, y, q, scale, rstd, res_in, x, gain, eps, N, C, s);
}

}  // namespace qffn
