// Linear and gated layers for few rows of activations (decode) or few weights:
// bound by the weights' way from HBM.
//
//   out[m, r] = bf16(res + act(s * sum_k W[r,k] x[m,k] + bias[r]))   (and z)
//   h[m, r]   = bf16(act(g) * u),  g / u from rows r and H + r of W1
//
// A CTA owns 16 weight rows (gated: 8 gate rows and the 8 up rows of the same
// outputs); its 8, 16 or 32 warps take the row's 256-byte groups in turn.  The
// products run on the tensor cores with the weights as the 16-row operand and
// up to 8 NT activation rows as the other (mma.sync m16n8k16 bf16 / m16n8k32
// E4M3): the weights are used once, so what counts is that every lane loads 16
// contiguous bytes of a row, streams them past L1, and has eight such loads in
// flight.  A lane's 16 bytes do not fall on the k places that the instruction
// names, but a dot product does not care which k is called which as long as
// both operands agree, and x is loaded the same way.  The accumulator holds
// row g in c0, c1 and row g + 8 in c2, c3 of one lane, and the warps' sums are
// added in order through shared memory: no atomics, no second launch, the same
// bits each run.
#include "act.cuh"
#include "common.cuh"
#include "launch.h"

namespace qffn {
namespace {

constexpr int kU = 4;                      // 64-byte chunks per group: 256 bytes of a row

struct SkinnyArgs {
  uint16_t* out;
  uint16_t* z;
  const uint8_t* w;
  const uint8_t* x;
  const float* x_scale;
  const float* w_scale;
  const uint16_t* bias;
  const uint16_t* res;
  int act, M, N;             // N: output columns (gated: H); block (i, j) takes rows 8 NT j .. of x
  int64_t row_bytes;         // of one row of w and of x
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

QFFN_DEVI void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

QFFN_DEVI float act_any(int act, float z) {
  switch (act) {
    case ACT_RELU: return act_f32<ACT_RELU>(z);
    case ACT_GELU: return act_f32<ACT_GELU>(z);
    case ACT_GELU_TANH: return act_f32<ACT_GELU_TANH>(z);
    case ACT_SILU: return act_f32<ACT_SILU>(z);
    default: return z;
  }
}

template <bool FP8, bool GATED, int NT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, (NT == 1 ? 32 : 16) / WARPS) skinny_kernel(const SkinnyArgs a) {
  constexpr int TOK = 8 * NT;
  __shared__ float red[WARPS][16][TOK + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int r0 = blockIdx.x * (GATED ? 8 : 16), m0 = blockIdx.y * TOK;
  // this lane's two weight rows; a row beyond the last is read as the last and dropped
  const int64_t ra = GATED ? r0 + g : min(r0 + g, a.N - 1);
  const int64_t rb = GATED ? int64_t(a.N) + r0 + g : min(r0 + g + 8, a.N - 1);
  const uint8_t* wa = a.w + ra * a.row_bytes + t * 16;
  const uint8_t* wb = a.w + rb * a.row_bytes + t * 16;
  const uint8_t* xp[NT];
  bool xl[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    xl[n] = m0 + n * 8 + g < a.M;
    xp[n] = a.x + int64_t(xl[n] ? m0 + n * 8 + g : 0) * a.row_bytes + t * 16;
  }
  float c[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.0f;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  // With few CTAs, all resident at once, the first group's weights set out for L2
  // while the preceding kernel ends: a hint, so it may run before that kernel's
  // results are there.  Measured, us without and with, one row: 4096 x 14336 in part
  // in L2 17.45 / 15.9, from HBM 20.1 / 20.3, 4096 x 4096 7.0 / 6.9.  More CTAs than
  // that only disturb each other's order in HBM: 28672 x 4096 35.6 / 37.6, gated 4096
  // x 14336 35.4 / 36.6; and so does E4M3.
  if (!FP8 && NT == 1 && WARPS >= 16) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t k = int64_t(warp) * (kU * 64) + u * 64;
      if (k + t * 16 < a.row_bytes) {
        prefetch_l2(wa + k);
        prefetch_l2(wb + k);
      }
    }
  }
  pdl_wait();
  pdl_trigger();
  for (int64_t k0 = int64_t(warp) * (kU * 64); k0 < a.row_bytes; k0 += int64_t(WARPS) * (kU * 64)) {
    uint4 va[kU], vb[kU], vx[NT][kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t k = k0 + u * 64;
      const bool in = k + t * 16 < a.row_bytes;      // the row's length is a multiple of 16 bytes
      va[u] = in ? ld16_stream(wa + k) : zero;
      vb[u] = in ? ld16_stream(wb + k) : zero;
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t k = k0 + u * 64;
      const bool in = k + t * 16 < a.row_bytes;
#pragma unroll
      for (int n = 0; n < NT; ++n) vx[n][u] = in && xl[n] ? ld16_once(xp[n] + k) : zero;
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma_16x8<FP8>(c[n], va[u].x, vb[u].x, va[u].y, vb[u].y, vx[n][u].x, vx[n][u].y);
        mma_16x8<FP8>(c[n], va[u].z, vb[u].z, va[u].w, vb[u].w, vx[n][u].z, vx[n][u].w);
      }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    red[warp][g][n * 8 + 2 * t] = c[n][0];
    red[warp][g][n * 8 + 2 * t + 1] = c[n][1];
    red[warp][g + 8][n * 8 + 2 * t] = c[n][2];
    red[warp][g + 8][n * 8 + 2 * t + 1] = c[n][3];
  }
  __syncthreads();
  const float scale = FP8 ? a.x_scale[0] * a.w_scale[0] : 1.0f;
  constexpr int ROWS = GATED ? 8 : 16;
  for (int i = threadIdx.x; i < ROWS * TOK; i += WARPS * 32) {
    const int r = i % ROWS, mt = i / ROWS, m = m0 + mt;
    if (m >= a.M || r0 + r >= a.N) continue;
    float v = 0.0f, u = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      v += red[w][r][mt];
      if (GATED) u += red[w][r + 8][mt];
    }
    const size_t o = size_t(m) * size_t(a.N) + size_t(r0 + r);
    if (GATED) {
      a.out[o] = f32_to_bf16(act_any(a.act, v) * u);
    } else {
      v *= scale;
      if (a.bias != nullptr) v += bf16_to_f32(a.bias[r0 + r]);
      if (a.z != nullptr) a.z[o] = f32_to_bf16(v);
      v = act_any(a.act, v);
      if (a.res != nullptr) v += bf16_to_f32(a.res[o]);
      a.out[o] = f32_to_bf16(v);
    }
  }
}

template <bool FP8, bool GATED, int NT, int WARPS>
cudaError_t launch(const SkinnyArgs& a, unsigned tiles, cudaStream_t s) {
  return launch_pdl(skinny_kernel<FP8, GATED, NT, WARPS>, dim3(tiles, unsigned((a.M + 8 * NT - 1) / (8 * NT))), WARPS * 32, 0, s, a);
}

template <bool FP8, bool GATED>
cudaError_t run(const SkinnyArgs& a, cudaStream_t s) {
  const unsigned tiles = unsigned(GATED ? (a.N + 7) / 8 : (a.N + 15) / 16);
  // Warps per CTA: as many as keep every tile resident at once (an SM holds 32
  // warps of the 8-row form's registers, 16 of the wider form's), so that few
  // tiles still keep the memory system busy; no more than the row has groups.
  const int64_t groups = a.row_bytes / (kU * 64);
  const int sms = num_sms();
  if (a.M <= 8) {
    if (tiles <= unsigned(sms) && groups >= 32) return launch<FP8, GATED, 1, 32>(a, tiles, s);
    if (tiles <= unsigned(2 * sms) && groups >= 16) return launch<FP8, GATED, 1, 16>(a, tiles, s);
    return launch<FP8, GATED, 1, 8>(a, tiles, s);
  }
  if (a.M <= 16) {
    if (tiles <= unsigned(sms) && groups >= 16) return launch<FP8, GATED, 2, 16>(a, tiles, s);
    return launch<FP8, GATED, 2, 8>(a, tiles, s);
  }
  return launch<FP8, GATED, 4, 8>(a, tiles, s);
}

}  // namespace

// Up to 16 rows the weights' stream bounds the call and this form is the
// fastest at every size (measured: 16 rows, 4096 x 14336: 21.6 us against 24.4 by
// few_rows.cu; 28672 x 4096: 41.8 against 41.3).  Beyond, each block of 32 rows
// reads the weights again, through L2: about 4 ns per CTA and 7.3 ns per CTA
// and 1024 elements of K over the whole grid, against 4.5 us and more that a
// tcgen05 kernel takes to set up, fill and drain.  It is taken while that
// sum is below 4.4 us (E4M3, whose products cost the same and whose loads cost the
// other form half: 2.9 us).  Measured in us, this form against the other: 256 rows
// of 768 x 256 4.2 / 7.0, of 1024 x 1024 7.3 / 8.5, 64 rows of 4096 x 1024 7.7 /
// 7.8, 32 rows of 28672 x 4096 58 / 41, E4M3 64 rows of 4096 x 256 6.5 / 4.9.
bool skinny_rows(int64_t M, int64_t wrows, int64_t K, bool fp8) {
  if (M <= 16) return true;
  const int64_t ctas = (wrows + 15) / 16 * ((M + 31) / 32);
  return ctas * (K + 550) <= (fp8 ? 400000 : 600000);
}

cudaError_t launch_skinny(uint16_t* out, uint16_t* z, const void* x, const float* x_scale, const void* w,
                          const float* w_scale, const uint16_t* bias, const uint16_t* res, int act, int64_t M,
                          int64_t N, int64_t K, bool fp8, cudaStream_t s) {
  SkinnyArgs a{out, z, static_cast<const uint8_t*>(w), static_cast<const uint8_t*>(x), x_scale, w_scale, bias, res,
               act, int(M), int(N), fp8 ? K : 2 * K};
  return fp8 ? run<true, false>(a, s) : run<false, false>(a, s);
}

cudaError_t launch_skinny_gated(uint16_t* h, const uint16_t* x, const uint16_t* w1, int act, int64_t M, int64_t C,
                                int64_t H, cudaStream_t s) {
  SkinnyArgs a{h, nullptr, reinterpret_cast<const uint8_t*>(w1), reinterpret_cast<const uint8_t*>(x), nullptr, nullptr,
               nullptr, nullptr, act, int(M), int(H), 2 * C};
  return run<false, true>(a, s);
}

}  // namespace qffn
