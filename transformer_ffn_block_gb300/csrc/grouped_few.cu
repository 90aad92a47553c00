// Products of few rows per group, and block-scaled products of few rows: bound by
// the weights' way from HBM, so the weights are streamed once through mma.sync.
//
//   out[m, r] = bf16(sum_k W_g[r,k] x[m,k] (+ bias[r]) (+ res[m,r])),  m in group g
//
// A CTA owns 16 weight rows of one group; its warps take the rows' 256-byte groups
// (E4M3: 128-byte groups) in turn and their sums are added in order through shared
// memory (the operand layout and the reasons for it are those of skinny.cu).  The CTA goes over the
// group's rows 8 NT at a time; beyond the first pass its weights come from L2.
// blockIdx.y counts the groups that have rows, found from the offsets by a
// warp-wide search, so that empty groups cost nothing.
//
// Block scales (E4M3): a group of 128 bytes is one block.  Its products are summed by
// the tensor cores from zero, and the fp32 sum joins the total multiplied by
// 2^(cx + cw - 254), exactly.
//
// Measured, weights from HBM: 1 row of two of eight bf16 28672 x 4096 70 us (6.7 TB/s), of
// 4096 x 2048 7.8 us (4.3 TB/s); E4M3, 1 row of 4096 x 14336 13.0 us (4.5 TB/s), of 4096 x 4096
// 5.6 us, where start and end of a call, 3 us, are most of what is above the bytes.
#include "common.cuh"
#include "launch.h"

namespace qffn {
namespace {

// 64-byte chunks of a row per group
constexpr int chunks_of(bool fp8) { return fp8 ? 2 : 4; }
// Warps per SM that the registers are to leave room for
constexpr int warps_of(int nt) { return nt == 1 ? 32 : 16; }

struct FewGroupArgs {
  uint16_t* out;
  const uint8_t* w;
  const uint8_t* x;
  const uint8_t* x_scale;    // [M, blocks] E8M0 (E4M3 operands)
  const uint8_t* w_scale;    // [G, ceil(N / 128), blocks]
  const uint16_t* bias;
  const uint16_t* res;
  const int* offsets;        // NULL: one group of all rows
  int G, M, N;
  int64_t blocks;            // of 128 in a row of K
  int64_t row_bytes;
};

template <bool FP8>
QFFN_DEVI void mma_16x8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if (FP8)
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// v * 2^(a - 127) * 2^(b - 127) for two E8M0 codes (255: NaN), as a product with two
// factors of half the exponent each, which neither overflow nor lose bits where the
// result does not.
QFFN_DEVI float scaled(float v, uint32_t a, uint32_t b) {
  const uint32_t e = a + b, h = e >> 1;
  const float f = __uint_as_float(a == 255u || b == 255u ? 0x7FC00000u : h << 23);
  return v * f * __uint_as_float((e - h) << 23);
}

template <bool FP8, int NT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, warps_of(NT) / WARPS) few_groups_kernel(const FewGroupArgs a) {
  constexpr int TOK = 8 * NT, kU = chunks_of(FP8);
  __shared__ float red[WARPS][16][TOK + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int r0 = blockIdx.x * 16;
  pdl_wait();
  pdl_trigger();
  // the group of this CTA: the blockIdx.y-th of those with rows
  int group = 0, begin = 0, end = a.M;
  if (a.offsets != nullptr) {
    // (an offset counts as one within 0 .. M and not below any before it)
    int skip = int(blockIdx.y), top = 0;
    group = -1;
    for (int base = 0; base < a.G; base += 32) {
      const int i = base + lane;
      int lo = 0, hi = 0;
      if (i < a.G) {
        lo = min(max(a.offsets[i], top), a.M);
        hi = min(max(a.offsets[i + 1], top), a.M);
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int below = __shfl_up_sync(0xffffffffu, lo, o);
        if (lane >= o) lo = max(lo, below);
      }
      hi = max(hi, lo);
      top = __reduce_max_sync(0xffffffffu, hi);
      const uint32_t some = __ballot_sync(0xffffffffu, hi > lo);
      const int n = __popc(some);
      if (skip < n) {
        const int l = int(__fns(some, 0, skip + 1));
        group = base + l;
        begin = __shfl_sync(0xffffffffu, lo, l);
        end = __shfl_sync(0xffffffffu, hi, l);
        break;
      }
      skip -= n;
    }
    if (group < 0) return;
  }
  // this lane's two weight rows; a row beyond the last is read as the last and dropped
  const int64_t first = int64_t(group) * a.N;
  const uint8_t* wa = a.w + (first + min(r0 + g, a.N - 1)) * a.row_bytes + t * 16;
  const uint8_t* wb = a.w + (first + min(r0 + g + 8, a.N - 1)) * a.row_bytes + t * 16;
  const uint8_t* ws = FP8 ? a.w_scale + (int64_t(group) * ((a.N + 127) >> 7) + (r0 >> 7)) * a.blocks : nullptr;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int m0 = begin; m0 < end; m0 += TOK) {
    const uint8_t* xp[NT];
    const uint8_t* xs[NT][2];
    bool xl[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      xl[n] = m0 + n * 8 + g < end;
      xp[n] = a.x + int64_t(xl[n] ? m0 + n * 8 + g : begin) * a.row_bytes + t * 16;
      // the accumulator's columns are rows 2 t and 2 t + 1 of the eight
      if (FP8) {
#pragma unroll
        for (int j = 0; j < 2; ++j) xs[n][j] = a.x_scale + int64_t(min(m0 + n * 8 + 2 * t + j, end - 1)) * a.blocks;
      }
    }
    float c[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.0f;
    for (int64_t k0 = int64_t(warp) * (kU * 64); k0 < a.row_bytes; k0 += int64_t(WARPS) * (kU * 64)) {
      uint4 va[kU], vb[kU], vx[NT][kU];
      uint32_t sw = 0u, sx[NT][2];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int64_t k = k0 + u * 64;
        const bool in = k + t * 16 < a.row_bytes;      // the row's length is a multiple of 16 bytes
        va[u] = in ? ld16_stream(wa + k) : zero;
        vb[u] = in ? ld16_stream(wb + k) : zero;
      }
      if (FP8) {
        sw = ws[k0 >> 7];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) sx[n][j] = xs[n][j][k0 >> 7];
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int64_t k = k0 + u * 64;
        const bool in = k + t * 16 < a.row_bytes;
#pragma unroll
        for (int n = 0; n < NT; ++n) vx[n][u] = in && xl[n] ? ld16_once(xp[n] + k) : zero;
      }
      if (!FP8) {
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_16x8<FP8>(c[n], va[u].x, vb[u].x, va[u].y, vb[u].y, vx[n][u].x, vx[n][u].y);
            mma_16x8<FP8>(c[n], va[u].z, vb[u].z, va[u].w, vb[u].w, vx[n][u].z, vx[n][u].w);
          }
      } else {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float p[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            mma_16x8<FP8>(p, va[u].x, vb[u].x, va[u].y, vb[u].y, vx[n][u].x, vx[n][u].y);
            mma_16x8<FP8>(p, va[u].z, vb[u].z, va[u].w, vb[u].w, vx[n][u].z, vx[n][u].w);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) c[n][j] += scaled(p[j], sw, sx[n][j & 1]);
        }
      }
    }
    __syncthreads();                       // the sums of the rows before these have been read
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      red[warp][g][n * 8 + 2 * t] = c[n][0];
      red[warp][g][n * 8 + 2 * t + 1] = c[n][1];
      red[warp][g + 8][n * 8 + 2 * t] = c[n][2];
      red[warp][g + 8][n * 8 + 2 * t + 1] = c[n][3];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * TOK; i += WARPS * 32) {
      const int r = i % 16, mt = i / 16, m = m0 + mt;
      if (m >= end || r0 + r >= a.N) continue;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) v += red[w][r][mt];
      const size_t o = size_t(m) * size_t(a.N) + size_t(r0 + r);
      if (a.bias != nullptr) v += bf16_to_f32(a.bias[r0 + r]);
      if (a.res != nullptr) v += bf16_to_f32(a.res[o]);
      a.out[o] = f32_to_bf16(v);
    }
  }
}

template <bool FP8, int NT, int WARPS>
cudaError_t launch(const FewGroupArgs& a, unsigned tiles, unsigned slots, cudaStream_t s) {
  return launch_pdl(few_groups_kernel<FP8, NT, WARPS>, dim3(tiles, slots), WARPS * 32, 0, s, a);
}

template <bool FP8>
cudaError_t run(const FewGroupArgs& a, cudaStream_t s) {
  const unsigned tiles = unsigned((a.N + 15) / 16), slots = unsigned(a.G < a.M ? a.G : a.M);
  // warps per CTA as in skinny.cu
  const int64_t steps = a.row_bytes / (chunks_of(FP8) * 64), ctas = int64_t(tiles) * slots, sms = num_sms();
  const int rows = a.offsets == nullptr ? a.M : (a.M + a.G - 1) / a.G;
  if (rows <= 8) {
    if (ctas <= sms && steps >= 32) return launch<FP8, 1, 32>(a, tiles, slots, s);
    if (ctas <= 2 * sms && steps >= 16) return launch<FP8, 1, 16>(a, tiles, slots, s);
    return launch<FP8, 1, 8>(a, tiles, slots, s);
  }
  if (rows <= 16) {
    if (ctas <= sms && steps >= 16) return launch<FP8, 2, 16>(a, tiles, slots, s);
    return launch<FP8, 2, 8>(a, tiles, slots, s);
  }
  return launch<FP8, 4, 8>(a, tiles, slots, s);
}

}  // namespace

cudaError_t launch_few_groups(uint16_t* out, const void* x, const uint8_t* x_scale, const void* w,
                              const uint8_t* w_scale, const uint16_t* bias, const uint16_t* res, const int* offsets,
                              int64_t G, int64_t M, int64_t N, int64_t K, cudaStream_t s) {
  const bool fp8 = x_scale != nullptr;
  FewGroupArgs a{out, static_cast<const uint8_t*>(w), static_cast<const uint8_t*>(x), x_scale, w_scale, bias, res,
                 offsets, int(G), int(M), int(N), (K + 127) / 128, fp8 ? K : 2 * K};
  return fp8 ? run<true>(a, s) : run<false>(a, s);
}

}  // namespace qffn
