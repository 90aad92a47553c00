// Internal launchers of the qffn kernels.  Each enqueues work on `s` and
// returns the CUDA error of the launch; argument checking is done by the
// C-ABI layer (api.cu) before any of these is called.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace qffn {

// Number of SMs of the current device (cached per device).
int num_sms();

// Launches `kernel` as a programmatic dependent launch: its blocks may be
// scheduled while the kernel before it on `s` drains.  Only for kernels that
// call pdl_wait() in every thread before they touch global memory.
//
// A kernel whose inputs were complete before the kernel launched just before it
// could start (that one having waited for them itself, in every thread, before
// its pdl_trigger()) may put its pdl_wait() at its end instead ("late wait"):
// it then runs beside the preceding kernel, on the SMs that one leaves free, and
// still counts as complete only after it, which is what the kernel behind
// relies on.  Neither may write what the other reads or writes.
template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*kernel)(Params...), dim3 grid, int block, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(block));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// ---- elementwise / reduction kernels (elementwise.cu)
cudaError_t launch_rmsnorm(uint16_t* res_out, uint16_t* y, float* rstd, float* stats,
                           const uint16_t* res_in, const uint16_t* x, const uint16_t* gain,
                           float eps, int64_t N, int C, cudaStream_t s);
cudaError_t launch_absmax(float* stats, const uint16_t* in, int64_t n, cudaStream_t s);
// Chained launches (pdl): the kernel is a programmatic dependent launch; it
// waits for the preceding kernel on `s` before touching global memory.
// zero_stat (optional): set to 0 by the kernel once that wait is over, so a
// later kernel of the same chain can record an abs-max there without a
// memset (which would break the chain).
cudaError_t launch_quantize(uint8_t* q, float* stats, const uint16_t* in, int64_t n,
                            cudaStream_t s, bool pdl = false, float* zero_stat = nullptr);
cudaError_t launch_quantize_rows(uint8_t* q, float* row_scale, const uint16_t* w, int64_t rows,
                                 int cols, cudaStream_t s);
// SwiGLU over gate_up [N, 2H]: writes h (if non-NULL) and max|h| into stats[0]
// (zeroed first).
cudaError_t launch_swiglu_absmax(uint16_t* h, float* stats, const uint16_t* gate_up, int64_t N,
                                 int64_t H, cudaStream_t s);
// Recomputes h from gate_up and quantises it with stats[0]; writes stats[1].
cudaError_t launch_swiglu_requant(uint8_t* hq, float* stats, const uint16_t* gate_up, int64_t N,
                                  int64_t H, cudaStream_t s);
cudaError_t launch_silu_mul(uint16_t* g, const uint16_t* u, int64_t n, bool pdl, cudaStream_t s);

// ---- tcgen05 FP8 GEMMs (gemm_fp8.cu)
// out[M,N] = bf16(a_scale*w_scale * A[M,K] . W[N,K]^T + bias[N] (+ out[M,N])):
// bias (bf16, optional) and, with `accumulate`, the previous contents of out
// are added to the scaled fp32 accumulator before the rounding.  With a_mn
// (w_mn) the operand is given MN-major, i.e. A as [K, M] (W as [K, N]) with
// the M (N) index contiguous; M (N) must then be a multiple of 16.
cudaError_t launch_gemm_bf16(uint16_t* out, const uint8_t* A, const float* a_scale,
                             const uint8_t* W, const float* w_scale, int64_t M, int64_t N,
                             int64_t K, cudaStream_t s, const uint16_t* bias = nullptr,
                             bool accumulate = false, bool a_mn = false, bool w_mn = false,
                             bool pdl = false);
// h[M,H] = bf16(silu(g)*u) with g, u the bf16-rounded gate / up products of
// W1 = [2H, K]; records max|h| into stats_h[0] (zeroed first by a memset,
// or, with `chained`, already zeroed by an earlier kernel of the chain: the
// GEMM is then a programmatic dependent launch).
cudaError_t launch_gemm_swiglu(uint16_t* h, float* stats_h, const uint8_t* A, const float* a_scale,
                               const uint8_t* W1, const float* w_scale, int64_t M, int64_t H,
                               int64_t K, cudaStream_t s, bool chained = false);
// hq[M,H] = e4m3(h * 448 / stats_h[0]) for the h of launch_gemm_swiglu, with
// the abs-max given (not recorded); writes stats_h[1] = scale.
cudaError_t launch_gemm_swiglu_quant(uint8_t* hq, float* stats_h, const uint8_t* A,
                                     const float* a_scale, const uint8_t* W1, const float* w_scale,
                                     int64_t M, int64_t H, int64_t K, cudaStream_t s,
                                     bool pdl = false);
// d_gu[M,2H] = SwiGLU gradient for dh [M,H] and the gate|up product of A and
// W1 = [2H, K] (the recompute of gate_up fused with swiglu_backward); records
// max|d_gu| into stats[0] (zeroed first).
cudaError_t launch_gemm_swiglu_bwd(uint16_t* d_gu, float* stats, const uint16_t* dh,
                                   const uint8_t* A, const float* a_scale, const uint8_t* W1,
                                   const float* w_scale, int64_t M, int64_t H, int64_t K,
                                   cudaStream_t s);
// Reads and clears the GEMM kernels' device status word of the current device.
cudaError_t gemm_take_status(unsigned int* status);
// SM clock cycles and nanoseconds that the first CTA of the most recent GEMM
// launch on the current device spent from its start to its end.
cudaError_t gemm_clock_sample(unsigned long long out[2]);
// Failure-path self-test of the GEMMs' bounded barrier wait (one CTA, two
// waits; out[4] as qffn_selftest_bounded_wait documents).
cudaError_t launch_wait_selftest(unsigned long long* out, int arrive, unsigned long long limit_ns,
                                 cudaStream_t s);

// ---- FP8 backward (backward.cu)
// out[Cc, R] = in[R, Cc]^T for E4M3 codes; R and Cc multiples of 16.
cudaError_t launch_transpose_u8(uint8_t* out, const uint8_t* in, int64_t R, int64_t Cc,
                                cudaStream_t s);
// dgu[N, 2H] = (dh * u * silu'(g) | dh * silu(g)) from gu = [N, 2H] (gate
// first) and dh [N, H]; records max|dgu| into stats[0] (zeroed first).
cudaError_t launch_swiglu_backward(uint16_t* dgu, float* stats, const uint16_t* dh,
                                   const uint16_t* gu, int64_t N, int64_t H, cudaStream_t s);

// ---- decode GEMVs (decode.cu)
// out0[r] = bf16(s0[r] * W0[r,:] . x); with W1 != NULL also out1 from W1, s1.
// With `pdl` the launch is a programmatic dependent launch that issues its
// first weight loads before waiting for the preceding kernel.
cudaError_t launch_gemv(uint16_t* out0, uint16_t* out1, const uint16_t* x, const uint8_t* w0,
                        const float* s0, const uint8_t* w1, const float* s1, int64_t rows,
                        int64_t cols, bool pdl, cudaStream_t s);
// out[r] = bf16(s[r] * W[r,:] . h) with h = bf16(silu(g) * u) formed while the
// input vector is staged (the fused-SiLU-input arm's down GEMV).
cudaError_t launch_gemv_silu_input(uint16_t* out, const uint16_t* g, const uint16_t* u,
                                   const uint8_t* w, const float* row_scale, int64_t rows,
                                   int64_t cols, cudaStream_t s);
// The whole decode FFN: the dual GEMV (g, u), then the down GEMV on
// h = bf16(silu(g) * u) formed in its prologue, launched as a programmatic
// dependent launch so its first weight loads overlap the dual GEMV's tail.
// `early`: the dual GEMV may read w_gate and w_up before the preceding kernel
// on the stream has finished.  Same bits as launch_gemv + launch_silu_mul +
// launch_gemv.
cudaError_t launch_decode(uint16_t* out, const uint16_t* x, const uint8_t* w_gate,
                          const float* s_gate, const uint8_t* w_up, const float* s_up,
                          const uint8_t* w_down, const float* s_down, int64_t C, int64_t H,
                          uint16_t* g, uint16_t* u, bool early, cudaStream_t s);
// ---- layer norm and the norms' backward (norm.cu)
cudaError_t launch_layernorm(uint16_t* res_out, uint16_t* y, float* mean, float* rstd, float* stats,
                             const uint16_t* res_in, const uint16_t* x, const uint16_t* gain,
                             const uint16_t* shift, float eps, int64_t N, int C, cudaStream_t s);
// Blocks of the backward, each of which writes one partial row of dgain (and
// of dshift, for the layer norm) into `partial`.
int norm_backward_blocks(int64_t N, int C);
cudaError_t launch_norm_backward(uint16_t* dx, float* dgain, float* dshift, float* stats, const uint16_t* dy,
                                 const uint16_t* dres, const uint16_t* r, const float* mean, const float* rstd,
                                 const uint16_t* gain, int64_t N, int C, bool centred, bool accumulate,
                                 float* partial, cudaStream_t s);
// Reads and clears the norm kernels' device status word of the current device.
cudaError_t norm_take_status(unsigned int* status);
// out0 [cols0], out1 [cols - cols0] (+)= the sum of the rows of partial [parts, cols],
// in a fixed order; either output may be NULL.  A programmatic dependent launch.
cudaError_t launch_column_sum(float* out0, float* out1, const float* partial, int parts, int64_t cols0,
                              int64_t cols, bool accumulate, cudaStream_t s);

// ---- linear and gated layers (linear.cu).  The *_workspace functions give the
// bytes `ws` must hold (0: none); shapes are checked by the caller.
size_t linear_workspace(int64_t M, int64_t N, int64_t K, bool fp8);
size_t gated_workspace(int64_t M, int64_t C, int64_t H);
size_t linear_backward_workspace(int64_t M, int64_t N, int64_t K);
size_t gated_backward_workspace(int64_t M, int64_t C, int64_t H);
cudaError_t launch_linear(uint16_t* out, uint16_t* z, const uint16_t* x, const uint16_t* w, const uint16_t* bias,
                          const uint16_t* res, int act, int64_t M, int64_t N, int64_t K, float* ws, cudaStream_t s);
cudaError_t launch_linear_fp8(uint16_t* out, uint16_t* z, const uint8_t* x, const float* x_scale, const uint8_t* w,
                              const float* w_scale, const uint16_t* bias, const uint16_t* res, int act, int64_t M,
                              int64_t N, int64_t K, float* ws, cudaStream_t s);
cudaError_t launch_linear_backward(uint16_t* dx, uint16_t* dw, float* dbias, const uint16_t* dout, const uint16_t* z,
                                   const uint16_t* x, const uint16_t* w, int act, int64_t M, int64_t N, int64_t K,
                                   bool accumulate, uint8_t* ws, cudaStream_t s);
cudaError_t launch_gated(uint16_t* h, const uint16_t* x, const uint16_t* w1, int act, int64_t M, int64_t C, int64_t H,
                         float* ws, cudaStream_t s);
cudaError_t launch_gated_backward(uint16_t* dx, uint16_t* dw1, const uint16_t* dh, const uint16_t* x,
                                  const uint16_t* w1, int act, int64_t M, int64_t C, int64_t H, bool accumulate,
                                  uint8_t* ws, cudaStream_t s);
// The forms for few rows or small weights (skinny.cu), which launch_linear* and
// launch_gated take where skinny_rows(); wrows: rows of the weight matrix.
bool skinny_rows(int64_t M, int64_t wrows, int64_t K, bool fp8);
cudaError_t launch_skinny(uint16_t* out, uint16_t* z, const void* x, const float* x_scale, const void* w,
                          const float* w_scale, const uint16_t* bias, const uint16_t* res, int act, int64_t M,
                          int64_t N, int64_t K, bool fp8, cudaStream_t s);
cudaError_t launch_skinny_gated(uint16_t* h, const uint16_t* x, const uint16_t* w1, int act, int64_t M, int64_t C,
                                int64_t H, cudaStream_t s);
// The forms for few rows on the tensor cores (few_rows.cu) and the estimate of
// their time in SM cycles, -1 where they do not apply.  No workspace.  w_mn: w given
// as [K, N] (bf16).  Gated: h from w1 = [2H, C], or, with dh, d_gu [M, 2H].
int64_t few_rows_cycles(int64_t M, int64_t N, int64_t K, bool gated, bool fp8, int64_t max_rows = 512);
cudaError_t launch_few_rows(uint16_t* out, uint16_t* z, const void* x, const float* x_scale, const void* w,
                            const float* w_scale, const uint16_t* bias, const uint16_t* res, int act, int64_t M,
                            int64_t N, int64_t K, bool fp8, bool w_mn, cudaStream_t s, bool late_wait = false);
cudaError_t launch_few_rows_gated(uint16_t* out, const uint16_t* x, const uint16_t* w1, const uint16_t* dh, int act,
                                  int64_t M, int64_t C, int64_t H, cudaStream_t s);
// E4M3 with block scales (E8M0):
cudaError_t launch_few_rows_blocks(uint16_t* out, const uint8_t* x, const uint8_t* x_scale, const uint8_t* w,
                                   const uint8_t* w_scale, const uint16_t* bias, const uint16_t* res, int64_t M,
                                   int64_t N, int64_t K, cudaStream_t s);
// Groups of rows with a matrix each (offsets on the device; x_scale NULL: bf16), and its estimate.
int64_t few_rows_grouped_cycles(int64_t G, int64_t M, int64_t N, int64_t K, bool fp8);
cudaError_t launch_few_rows_grouped(uint16_t* out, const void* x, const uint8_t* x_scale, const void* w,
                                    const uint8_t* w_scale, const int* offsets, int64_t G, int64_t M, int64_t N,
                                    int64_t K, cudaStream_t s);
// The input gradient of launch_grouped: dx [M, K] = dout [M, N] w_g.
cudaError_t launch_few_rows_grouped_dx(uint16_t* dx, const uint16_t* dout, const uint16_t* w, const int* offsets, int64_t G,
                                       int64_t M, int64_t N, int64_t K, cudaStream_t s);
cudaError_t few_rows_take_status(unsigned int* status);
// Reads and clears the linear kernels' device status word of the current device.
cudaError_t linear_take_status(unsigned int* status);

// ---- E4M3 with a scale per block of 128 (blocks.cu); scales are E8M0 codes
cudaError_t launch_quantize_blocks(uint8_t* q, uint8_t* scale, const uint16_t* in, int64_t rows, int64_t cols,
                                   cudaStream_t s);
cudaError_t launch_quantize_weight_blocks(uint8_t* q, uint8_t* scale, const uint16_t* w, int64_t count, int64_t rows,
                                          int64_t cols, cudaStream_t s);
cudaError_t launch_swiglu_quantize_blocks(uint16_t* h, uint8_t* q, uint8_t* scale, const uint16_t* gate_up, int64_t N,
                                          int64_t H, cudaStream_t s);
cudaError_t launch_rmsnorm_quantize_blocks(uint16_t* res_out, uint16_t* y, uint8_t* q, uint8_t* scale, float* rstd,
                                           const uint16_t* res_in, const uint16_t* x, const uint16_t* gain, float eps,
                                           int64_t N, int C, cudaStream_t s);

// ---- products of groups of rows with a matrix each, and block-scaled products.
// x, w: bf16, or E4M3 with x_scale and w_scale; offsets NULL: one group of all M rows.
// Few rows (grouped_few.cu):
cudaError_t launch_few_groups(uint16_t* out, const void* x, const uint8_t* x_scale, const void* w,
                              const uint8_t* w_scale, const uint16_t* bias, const uint16_t* res, const int* offsets,
                              int64_t G, int64_t M, int64_t N, int64_t K, cudaStream_t s);

// Any number of rows (grouped.cu), which takes the form above where that is the faster:
cudaError_t launch_linear_blocks(uint16_t* out, const uint8_t* x, const uint8_t* x_scale, const uint8_t* w,
                                 const uint8_t* w_scale, const uint16_t* bias, const uint16_t* res, int64_t M, int64_t N,
                                 int64_t K, cudaStream_t s);
cudaError_t launch_grouped(uint16_t* out, const void* x, const uint8_t* x_scale, const void* w, const uint8_t* w_scale,
                           const int* offsets, int64_t G, int64_t M, int64_t N, int64_t K, cudaStream_t s);
cudaError_t launch_grouped_backward(uint16_t* dx, uint16_t* dw, const uint16_t* dout, const uint16_t* x,
                                    const uint16_t* w, const int* offsets, int64_t G, int64_t M, int64_t N, int64_t K,
                                    bool accumulate, cudaStream_t s);
// Reads and clears the grouped kernels' device status word of the current device.
cudaError_t grouped_take_status(unsigned int* status);

// Reads and clears the decode kernels' device status word of the current device.
cudaError_t decode_take_status(unsigned int* status);

}  // namespace qffn
