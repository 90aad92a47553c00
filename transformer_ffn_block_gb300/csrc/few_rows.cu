// Linear and gated layers for up to a few hundred rows of activations on the
// tensor cores (tcgen05, sm_103a): the weights are the 128-row operand.
//
//   D[n, m] = sum_k W[n, k] x[m, k]   n: 128 weight rows per CTA,
//                                     m: bn <= 128 activation rows
//
// With so few rows the bytes of the weights bound the call.  A tile of 256
// activation rows would be mostly padding, and there are too few tiles for the
// SMs; here the MMA's N is the number of activation rows (a multiple of 32), and
// K is split over the CTAs of a cluster (1, 2, 4 or 8).  Each CTA sums its part
// of K in TMEM, sends each other CTA of the cluster that one's share of the
// activation rows (bulk copies between their shared memories), adds its own
// share in a fixed order and applies the epilogue to it.  One launch, no partial
// sums in global memory, no workspace, the same bits each run.  (Measured at 64
// x 4096 x 4096: partial sums in a workspace with a second kernel to join them
// 13.8 us, 3 us of it from the first kernel's end to the second's; SM pairs in
// clusters of 8, of which 16 do not fit on the GPU at once, 20.6 us; the shares
// fetched by loads from the other CTAs' shared memory, 16 bytes a lane, 12.1 us,
// 2 us of it for 32 KB per CTA.)
//
// Per CTA: one warp's lane loads (TMA, 128-byte swizzle) 128 weight rows and
// the tile's activation rows, 128 bytes of K per stage; one thread issues the
// MMAs; then all eight warps read TMEM.  Gated forms: the 128 rows are 64 gate
// rows and the 64 up rows of the same outputs.  Every mbarrier wait is bounded,
// as in linear.cu.
//
// GROUPED: rows in groups with a matrix each (see grouped.cu), a cluster per (tile of
// 128 weight rows, tile of rows of one group).  The host launches as many tiles of rows as
// there can be; a cluster finds its group from the offsets, and one beyond the last ends.
// With W_MN it is their input gradient.
//
// OP_BLOCKS: E4M3 with a power-of-two scale per block of 128, which the tensor cores
// multiply (grouped.cu says how): two warps write the scales of 512 of K at a time to
// shared memory, the issuing thread copies them to TMEM in front of their MMAs.
#include <cuda.h>

#include "act.cuh"
#include "common.cuh"
#include "launch.h"
#include "pipeline.cuh"
#include "tensor_map.h"
#include "umma.cuh"

namespace qffn {
namespace {

constexpr int kThreads = 256;
constexpr int ROW_BYTES = 128;             // one swizzle atom row
constexpr int BOX_BYTES = 128 * ROW_BYTES;
constexpr int STEPS = 4;                   // MMAs per stage (32 bytes of K each)
constexpr int kMaxStages = 12;
constexpr int kMaxSplits = 8;
constexpr unsigned long long kWaitLimitNs = 2000000000ull;
constexpr unsigned long long kDrainLimitNs = 200000000ull;

constexpr int OP_BF16 = 0, OP_E4M3 = 1, OP_BLOCKS = 2;
constexpr int kScaleStages = 4, kScaleBytes = 2 * 512;   // 128 weight rows, 128 rows of x: 4 bytes each
constexpr int EPI_LINEAR = 0, EPI_GATED = 1, EPI_GATED_BWD = 2;
constexpr int stage_k(int op) { return op == OP_BF16 ? 64 : 128; }   // elements of K per stage

__device__ unsigned int g_status;

struct FewArgs {
  uint16_t* out;
  uint16_t* z;
  const uint16_t* bias;
  const uint16_t* in;       // EPI_LINEAR: residual (optional); GATED_BWD: dh
  const float* a_scale;     // E4M3 operands; else NULL
  const float* w_scale;
  const uint8_t* x_blocks;  // OP_BLOCKS: E8M0 scales [M, blocks] and [ceil(N / 128), blocks]
  const uint8_t* w_blocks;
  int blocks;
  const int* offsets;       // GROUPED
  int G;
  int act;
  int M, N;                 // activation rows; output columns (gated: H)
  int num_kb, splits;       // K blocks of a stage each; parts of K (CTAs per cluster)
  int bn, tiles_m;          // activation rows per tile; tiles of activation rows
  int stages, stage_bytes;
  int recv_bytes;           // shared memory for the other CTAs' sums, behind the stages
  int tmem_cols;
  int late_wait;            // does not read the preceding kernel's results (see launch.h)
};

// D(tmem) (+)= A(smem) . B(smem)^T
template <int OP>
QFFN_DEVI void mma_one(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  if (OP == OP_BF16)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// The same with block scales at TMEM columns sfa and sfb.
QFFN_DEVI void mma_one_blocks(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                              uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}
// The scales of 128 rows, 512 bytes of shared memory, to four TMEM columns (see grouped.cu).
QFFN_DEVI void copy_scales(uint32_t taddr, uint32_t saddr) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc_scales(saddr)) : "memory");
}
// Arrive once on `bar` when all previously issued MMAs of this thread have completed.
QFFN_DEVI void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// Descriptor of MMA step i of the weights.  K-major: 32 bytes along the 128-byte
// rows per step.  MN-major (bf16): the 128 rows lie in two boxes of 64 rows x 64
// of K; a step is 16 K rows of 128 bytes in both, whose distance is the leading
// byte offset (see linear.cu).
template <bool MN>
QFFN_DEVI uint64_t w_desc(uint32_t base, int i) {
  if (!MN) return sdesc_sw128(base + uint32_t(i) * 32u);
  const uint64_t d = sdesc_sw128(base + uint32_t(i) * 16u * ROW_BYTES);
  return (d & ~(uint64_t(0x3FFF) << 16)) | (uint64_t(BOX_BYTES / 2 >> 4) << 16);
}

QFFN_DEVI bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, bool honour_abort = true,
                         unsigned long long limit = kWaitLimitNs) {
  return mbar_wait_bounded(bar, parity, abort_flag, &g_status, honour_abort, limit);
}

// Bulk copy from this CTA's shared memory into another's (shared::cluster
// addresses), completing on a barrier of that CTA.
QFFN_DEVI void send_bulk(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "r"(src), "r"(bytes), "r"(bar)
      : "memory");
}
QFFN_DEVI void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
QFFN_DEVI void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

QFFN_DEVI uint32_t pack2(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return pack_bf16x2(lo, hi);
}
QFFN_DEVI uint4 pack8(const uint64_t (&v)[4]) { return make_uint4(pack2(v[0]), pack2(v[1]), pack2(v[2]), pack2(v[3])); }
QFFN_DEVI void unpack8(uint4 v, uint64_t (&f)[4]) {
  f[0] = bf16x2_to_f2(v.x);
  f[1] = bf16x2_to_f2(v.y);
  f[2] = bf16x2_to_f2(v.z);
  f[3] = bf16x2_to_f2(v.w);
}

// The activation is a run-time choice here: it is applied to few elements.
template <int ACT>
QFFN_DEVI void act8_t(uint64_t (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = act_f2<ACT>(v[j]);
}
QFFN_DEVI void act8(int act, uint64_t (&v)[4]) {
  switch (act) {
    case ACT_RELU: act8_t<ACT_RELU>(v); break;
    case ACT_GELU: act8_t<ACT_GELU>(v); break;
    case ACT_GELU_TANH: act8_t<ACT_GELU_TANH>(v); break;
    case ACT_SILU: act8_t<ACT_SILU>(v); break;
    default: break;
  }
}
template <int ACT>
QFFN_DEVI void act_grad8_t(const uint64_t (&v)[4], uint64_t (&f)[4], uint64_t (&df)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) act_grad_f2<ACT>(v[j], f[j], df[j]);
}
QFFN_DEVI void act_grad8(int act, const uint64_t (&v)[4], uint64_t (&f)[4], uint64_t (&df)[4]) {
  switch (act) {
    case ACT_RELU: act_grad8_t<ACT_RELU>(v, f, df); break;
    case ACT_GELU: act_grad8_t<ACT_GELU>(v, f, df); break;
    case ACT_GELU_TANH: act_grad8_t<ACT_GELU_TANH>(v, f, df); break;
    case ACT_SILU: act_grad8_t<ACT_SILU>(v, f, df); break;
    default: act_grad8_t<ACT_NONE>(v, f, df); break;
  }
}

// Eight sums of row m of this CTA's share, from weight row n on, the parts in
// order: slot j < SPLITS - 1 of `recv` holds part j (j < part) or j + 1.
template <int SPLITS>
QFFN_DEVI void sum8(const float* own, const float* recv, int share, int part, int m, int n, uint64_t (&v)[4]) {
  ulonglong2 a[SPLITS], b[SPLITS];
#pragma unroll
  for (int j = 0; j < SPLITS; ++j) {
    const float* src = j == part ? own : recv + (j < part ? j : j - 1) * share * 128;
    const ulonglong2* p = reinterpret_cast<const ulonglong2*>(src + m * 128 + n);
    a[j] = p[0];
    b[j] = p[1];
  }
  v[0] = a[0].x;
  v[1] = a[0].y;
  v[2] = b[0].x;
  v[3] = b[0].y;
#pragma unroll
  for (int j = 1; j < SPLITS; ++j) {
    v[0] = f2_add(v[0], a[j].x);
    v[1] = f2_add(v[1], a[j].y);
    v[2] = f2_add(v[2], b[j].x);
    v[3] = f2_add(v[3], b[j].y);
  }
}

// The parts added and the epilogue for this CTA's share, the activation rows
// part * share .. of the tile (share = bn / SPLITS), for the tile's weight rows.
// `row0`: the tile's first row; rows from `row_end` on are not the tile's.
template <int OP, int EPI, int SPLITS>
QFFN_DEVI void finish(const FewArgs& args, const float* sums, const float* recv, int part, int n0, int row0, int row_end) {
  constexpr bool GATED = EPI != EPI_LINEAR;
  constexpr int TPM = GATED ? 8 : 16;        // threads per activation row, eight outputs each
  const int share = args.bn / SPLITS;
  const float* own = sums + part * share * 128;
  const int nl = int(threadIdx.x) % TPM * 8, n = n0 + nl;
  if (n >= args.N) return;
  const float scale = OP == OP_E4M3 ? args.a_scale[0] * args.w_scale[0] : 1.0f;
  uint64_t bias[4] = {0ull, 0ull, 0ull, 0ull};
  if (EPI == EPI_LINEAR && args.bias != nullptr) unpack8(ld16_once(args.bias + n), bias);
  const int m0 = row0 + part * share;
  const int rows = min(share, row_end - m0);
#pragma unroll 2
  for (int ml = int(threadIdx.x) / TPM; ml < rows; ml += kThreads / TPM) {
    const size_t m = size_t(m0) + size_t(ml);
    const size_t o = m * size_t(args.N) + size_t(n);
    uint4 in4 = make_uint4(0, 0, 0, 0);
    if (args.in != nullptr) in4 = ld16_once(args.in + o);
    uint64_t v[4], t[4];
    sum8<SPLITS>(own, recv, share, part, ml, nl, v);
    unpack8(in4, t);
    if (EPI == EPI_LINEAR) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (OP == OP_E4M3) v[j] = f2_mul(v[j], f2_dup(scale));
        v[j] = f2_add(v[j], bias[j]);
      }
      if (args.z != nullptr) stg16(args.z + o, pack8(v));
      act8(args.act, v);
      if (args.in != nullptr) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = f2_add(v[j], t[j]);
      }
      stg16(args.out + o, pack8(v));
    } else {
      uint64_t up[4];
      sum8<SPLITS>(own, recv, share, part, ml, 64 + nl, up);
      if (EPI == EPI_GATED) {
        act8(args.act, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = f2_mul(v[j], up[j]);
        stg16(args.out + o, pack8(v));
      } else {
        uint64_t f[4], df[4];
        act_grad8(args.act, v, f, df);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] = f2_mul(f2_mul(t[j], up[j]), df[j]);
          f[j] = f2_mul(t[j], f[j]);
        }
        uint16_t* dst = args.out + m * 2 * size_t(args.N) + size_t(n);
        stg16(dst, pack8(v));
        stg16(dst + args.N, pack8(f));
      }
    }
  }
}

// Grid: one cluster of `splits` CTAs per (tile of 128 weight rows, tile of bn
// activation rows).
template <int OP, bool W_MN, int EPI, bool GROUPED = false>
__global__ void __launch_bounds__(kThreads)
    few_rows_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                    const FewArgs args) {
  constexpr bool GATED = EPI != EPI_LINEAR;
  extern __shared__ uint8_t smem_raw[];
  constexpr bool BLOCKS = OP == OP_BLOCKS;
  __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 3 + (BLOCKS ? 2 * kScaleStages : 0)];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t bar0 = smem_u32(bars);
  // full[s]: the loads of stage s landed; empty[s]: the MMAs reading it are done;
  // done: this CTA's sums are complete; drain: all MMAs issued have completed;
  // recv: the other CTAs' sums for this one's share have arrived
  auto full_bar = [&](int s) { return bar0 + 8u * uint32_t(s); };
  auto empty_bar = [&](int s) { return bar0 + 8u * uint32_t(kMaxStages + s); };
  const uint32_t done_bar = bar0 + 8u * uint32_t(2 * kMaxStages);
  const uint32_t drain_bar = bar0 + 8u * uint32_t(2 * kMaxStages + 1);
  const uint32_t recv_bar = bar0 + 8u * uint32_t(2 * kMaxStages + 2);
  // sfull[s]: the scales of stage s are written; sempty[s]: copied
  auto sfull_bar = [&](int s) { return bar0 + 8u * uint32_t(2 * kMaxStages + 3 + s); };
  auto sempty_bar = [&](int s) { return bar0 + 8u * uint32_t(2 * kMaxStages + 3 + kScaleStages + s); };
  const uint32_t scales = smem_u32(smem) + uint32_t(args.stages * args.stage_bytes + args.recv_bytes);

  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int part = int(cluster_ctarank());
  // (clusters next to each other read the same weights)
  const int tile = int(cluster_id_x()) / args.tiles_m, mt = int(cluster_id_x()) % args.tiles_m;

  if (threadIdx.x == 0) {
    for (int s = 0; s < args.stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(done_bar, 1);
    mbar_init(drain_bar, 1);
    mbar_init(recv_bar, 1);
    if (BLOCKS)
      for (int s = 0; s < kScaleStages; ++s) {
        mbar_init(sfull_bar(s), 1);
        mbar_init(sempty_bar(s), 1);
      }
    *abort_flag = 0;
    mbar_init_fence();
    if (args.splits > 1) mbar_expect_tx(recv_bar, uint32_t(args.recv_bytes));
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                 "r"(args.tmem_cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_arrive();        // this CTA can receive (waited for before any CTA sends)
  const uint32_t tmem_base = tmem_slot;
  if (!args.late_wait) pdl_wait();
  pdl_trigger();
  int row0 = mt * args.bn, row_end = args.M, group = 0;
  if constexpr (GROUPED) {
    // the group and the rows of the mt-th tile (an offset counts as one within 0 .. M and not
    // below any before it)
    int skip = mt, top = 0;
    group = -1;
    for (int base = 0; base < args.G; base += 32) {
      const int i = base + lane;
      int lo = 0, hi = 0;
      if (i < args.G) {
        lo = min(max(args.offsets[i], top), args.M);
        hi = min(max(args.offsets[i + 1], top), args.M);
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int below = __shfl_up_sync(0xffffffffu, lo, o);
        if (lane >= o) lo = max(lo, below);
      }
      hi = max(hi, lo);
      const int own = (hi - lo + args.bn - 1) / args.bn;
      int tiles = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int below = __shfl_up_sync(0xffffffffu, tiles, o);
        if (lane >= o) tiles += below;
      }
      const uint32_t reach = __ballot_sync(0xffffffffu, tiles > skip);
      if (reach != 0u) {
        const int l = __ffs(int(reach)) - 1;
        group = base + l;
        row0 = __shfl_sync(0xffffffffu, lo, l) + (skip - __shfl_sync(0xffffffffu, tiles - own, l)) * args.bn;
        row_end = __shfl_sync(0xffffffffu, hi, l);
        break;
      }
      skip -= __shfl_sync(0xffffffffu, tiles, 31);
      top = __reduce_max_sync(0xffffffffu, hi);
    }
    if (group < 0) {                         // (the same in the whole cluster)
      cluster_wait();
      if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(args.tmem_cols)
                     : "memory");
      return;
    }
  }

  const int per = (args.num_kb + args.splits - 1) / args.splits;
  const int kb0 = part * per, kb1 = min(args.num_kb, kb0 + per);   // every part has at least one
  // first output of this CTA (gated: 64 outputs, 128 otherwise)
  const int n0 = tile * (GATED ? 64 : 128);
  if (warp == 0) {
    if (elect_one()) {
      // ------------------------------------------------------------ producer
      uint32_t issued = 0, issued_parity = 0;
      int s = 0;
      uint32_t ph = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(empty_bar(s), ph ^ 1u, abort_flag)) break;
        mbar_expect_tx(full_bar(s), uint32_t(args.stage_bytes));
        const uint32_t fb = full_bar(s);
        const uint32_t dw = smem_u32(smem) + uint32_t(s * args.stage_bytes), dx = dw + BOX_BYTES;
        const int k0 = kb * stage_k(OP);
        if (GATED) {
          tma_load_2d(dw, &tmW, fb, k0, n0);
          tma_load_2d(dw + BOX_BYTES / 2, &tmW, fb, k0, args.N + n0);
        } else if (GROUPED && W_MN) {
          tma_load_3d(dw, &tmW, fb, n0, k0, group);
          tma_load_3d(dw + BOX_BYTES / 2, &tmW, fb, n0 + 64, k0, group);
        } else if (GROUPED) {
          tma_load_3d(dw, &tmW, fb, k0, n0, group);
        } else if (W_MN) {
          tma_load_2d(dw, &tmW, fb, n0, k0);
          tma_load_2d(dw + BOX_BYTES / 2, &tmW, fb, n0 + 64, k0);
        } else {
          tma_load_2d(dw, &tmW, fb, k0, n0);
        }
        tma_load_2d(dx, &tmX, fb, k0, row0);
        issued |= 1u << s;
        issued_parity = (issued_parity & ~(1u << s)) | (ph << s);
        if (++s == args.stages) {
          s = 0;
          ph ^= 1u;
        }
      }
      // every phase armed completes before shared memory is reused or released
      for (int k = 0; k < args.stages; ++k)
        if (issued & (1u << k)) mbar_wait(full_bar(k), (issued_parity >> k) & 1u, abort_flag, false, kDrainLimitNs);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one()) {
      // ------------------------------------------------------------ MMA issuer
      // D fp32, operand formats, W MN-major, N = bn, M = 128 (see linear.cu)
      // (OP_BLOCKS: E8M0 scales, bit 23; see grouped.cu)
      const uint32_t idesc = (BLOCKS ? 1u << 23 : 1u << 4) | (OP == OP_BF16 ? (1u << 7) | (1u << 10) : 0u) |
                             (W_MN ? 1u << 15 : 0u) | (uint32_t(args.bn >> 3) << 17) | (uint32_t(128 >> 4) << 24);
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      uint32_t sf = 0;                       // TMEM columns of the current scales
      bool ready = false;                    // the next stage was there before this one's MMAs were issued
      for (int kb = kb0; kb < kb1; ++kb) {
        if (BLOCKS && ((kb - kb0) & 3) == 0) {
          const int chunk = (kb - kb0) >> 2, ss = chunk % kScaleStages;
          if (!mbar_wait(sfull_bar(ss), uint32_t(chunk / kScaleStages) & 1u, abort_flag)) { ok = false; break; }
          tc_fence_after();
          sf = tmem_base + uint32_t(args.bn + 8 * (chunk & 1));
          copy_scales(sf, scales + uint32_t(ss * kScaleBytes));
          copy_scales(sf + 4, scales + uint32_t(ss * kScaleBytes + 512));
          mma_commit(sempty_bar(ss));
        }
        if (!ready && !mbar_wait(full_bar(s), ph, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const uint32_t a0 = smem_u32(smem) + uint32_t(s * args.stage_bytes), b0 = a0 + BOX_BYTES, empty = empty_bar(s);
        if (++s == args.stages) {
          s = 0;
          ph ^= 1u;
        }
        ready = kb + 1 < kb1 && mbar_test_wait(full_bar(s), ph);
        if (BLOCKS) {
          const uint32_t which = uint32_t((kb - kb0) & 3);
#pragma unroll
          for (int i = 0; i < STEPS; ++i)
            mma_one_blocks(tmem_base, w_desc<W_MN>(a0, i), sdesc_sw128(b0 + uint32_t(i) * 32u),
                           idesc | (which << 4) | (which << 29), sf, sf + 4, uint32_t((kb - kb0) | i));
        } else
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
          mma_one<OP>(tmem_base, w_desc<W_MN>(a0, i), sdesc_sw128(b0 + uint32_t(i) * 32u), idesc,
                      uint32_t((kb - kb0) | i));
        mma_commit(empty);
      }
      if (ok) mma_commit(done_bar);
      mma_commit(drain_bar);
      mbar_wait(drain_bar, 0, abort_flag, false, kDrainLimitNs);
    }
    __syncwarp();
  } else if (BLOCKS && (warp == 3 || warp == 4)) {
    // -------------------------------------------------------------- scales
    // Each warp every second chunk of four blocks.  Lane l: the words of rows l, l + 32, l +
    // 64, l + 96 of x; the 128 weight rows have one word.
    const int chunks = (kb1 - kb0 + 3) / 4;
    const uint8_t* const wb = args.w_blocks + size_t(group * ((args.N + 127) / 128) + tile) * size_t(args.blocks);
    const bool whole = ((reinterpret_cast<uintptr_t>(args.x_blocks) | reinterpret_cast<uintptr_t>(args.w_blocks) | uintptr_t(args.blocks | kb0)) & 3u) == 0;
    const uint8_t* const xs_end = args.x_blocks + size_t(args.M) * size_t(args.blocks);
    const uint8_t* const ws_end = args.w_blocks + size_t(args.G > 0 ? args.G : 1) * size_t((args.N + 127) / 128) * size_t(args.blocks);
    bool going = true;
    for (int c = warp - 3; going && c < chunks; c += 2) {
      const int first = kb0 + 4 * c, n = min(4, kb1 - first);
      const uint8_t* xp[4];
      bool within = scales_within(wb + first, args.w_blocks, ws_end);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        xp[i] = args.x_blocks + size_t(min(row0 + 32 * i + lane, args.M - 1)) * size_t(args.blocks) + size_t(first);
        within = within && (32 * i >= args.bn || scales_within(xp[i], args.x_blocks, xs_end));
      }
      uint32_t word_w, word_x[4];
      if (whole) {
        word_w = scales_word(wb + first)[0];
#pragma unroll
        for (int i = 0; i < 4; ++i) word_x[i] = 32 * i < args.bn ? scales_word(xp[i])[0] : 0u;
      } else if (__all_sync(0xffffffffu, within)) {
        word_w = scales_joined(wb + first);
#pragma unroll
        for (int i = 0; i < 4; ++i) word_x[i] = 32 * i < args.bn ? scales_joined(xp[i]) : 0u;
      } else {
        word_w = scales_bytes(wb + first, n);
#pragma unroll
        for (int i = 0; i < 4; ++i) word_x[i] = 32 * i < args.bn ? scales_bytes(xp[i], n) : 0u;
      }
      const int ss = c % kScaleStages;
      going = __all_sync(0xffffffffu, mbar_wait(sempty_bar(ss), (uint32_t(c / kScaleStages) & 1u) ^ 1u, abort_flag));
      if (!going) break;
      const uint32_t dst = scales + uint32_t(ss * kScaleBytes + lane * 16);
      sts16(dst, make_uint4(word_w, word_w, word_w, word_w));
      sts16(dst + 512, make_uint4(word_x[0], word_x[1], word_x[2], word_x[3]));
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(sfull_bar(ss));
    }
    __syncwarp();
  }
  const bool ok = __all_sync(0xffffffffu, mbar_wait(done_bar, 0, abort_flag));
  tc_fence_after();
  // ---------------------------------------------------------------- this part's sums into shared memory
  // [bn activation rows][128 weight rows] fp32, over the stages (all read)
  float* const sums = reinterpret_cast<float*>(smem);
  if (ok) {
    const int q = warp & 3;
    for (int c = (warp >> 2) * 32; c < args.bn; c += 64) {
      uint32_t v[32];
      tmem_ld32(tmem_base + (uint32_t(q * 32) << 16) + uint32_t(c), v);
#pragma unroll
      for (int j = 0; j < 32; ++j) sums[(c + j) * 128 + q * 32 + lane] = __uint_as_float(v[j]);
    }
  }
  tc_fence_before();
  fence_proxy_async_smem();
  __syncthreads();
  cluster_wait();
  const float* recv = reinterpret_cast<const float*>(smem + args.stages * args.stage_bytes);
  bool have = ok;
  if (args.splits > 1) {
    if (ok && warp == 0) {
      // lane j sends part j its share; the slots of the receiver skip its own part
      const uint32_t bytes = uint32_t(args.bn / args.splits) * 512u;
      if (lane < args.splits && lane != part) {
        const uint32_t slot = uint32_t(part < lane ? part : part - 1);
        send_bulk(map_to_rank(smem_u32(recv) + slot * bytes, uint32_t(lane)), smem_u32(sums) + uint32_t(lane) * bytes,
                  bytes, map_to_rank(recv_bar, uint32_t(lane)));
      }
      __syncwarp();
    }
    have = mbar_wait(recv_bar, 0, abort_flag) && ok;
    __syncwarp();
  }
  cluster_arrive();        // this CTA has received all; its own sends are done when all have arrived
  // ---------------------------------------------------------------- the parts added, epilogue
  if (have) {
    switch (args.splits) {
      case 1: finish<OP, EPI, 1>(args, sums, recv, part, n0, row0, row_end); break;
      case 2: finish<OP, EPI, 2>(args, sums, recv, part, n0, row0, row_end); break;
      case 4: finish<OP, EPI, 4>(args, sums, recv, part, n0, row0, row_end); break;
      default: finish<OP, EPI, 8>(args, sums, recv, part, n0, row0, row_end); break;
    }
  }
  __syncwarp();
  cluster_wait();
  if (args.late_wait) pdl_wait();    // this kernel is not complete before the preceding one
  if (warp == 2) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(args.tmem_cols)
                 : "memory");
  }
}

// ------------------------------------------------------------------ host side
// Shared memory per CTA: two CTAs per SM where a few stages of the narrow
// tiles fit twice, so that one's set-up and exchange overlap the other's loads.
constexpr int kSmemOne = 200 * 1024, kSmemTwo = 100 * 1024;

template <int OP, bool W_MN, int EPI, bool GROUPED = false>
cudaError_t launch(const CUtensorMap& w, const CUtensorMap& x, FewArgs a, int clusters, cudaStream_t s) {
  const auto fn = few_rows_kernel<OP, W_MN, EPI, GROUPED>;
  const int bytes = a.stages * a.stage_bytes + a.recv_bytes + (OP == OP_BLOCKS ? kScaleStages * kScaleBytes : 0) + 1024;
  static bool set[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !set[dev]) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemOne + 1024);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(clusters) * unsigned(a.splits));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = size_t(bytes);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(a.splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, fn, w, x, a);
}

// Clusters of `size` CTAs that fit on the current device at once with one CTA per
// SM (cached per device; the same for every form, whose shared memory is that
// of one CTA per SM).
cudaError_t max_clusters(int size, int* n) {
  static int cached[64][4] = {};
  const int i = size == 2 ? 1 : size == 4 ? 2 : 3;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && cached[dev][i] > 0) {
    *n = cached[dev][i];
    return cudaSuccess;
  }
  const auto fn = few_rows_kernel<OP_BF16, false, EPI_LINEAR>;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemOne + 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(num_sms() / size * size));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemOne + 1024;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(size);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaOccupancyMaxActiveClusters(n, fn, &cfg);
  if (e == cudaSuccess && dev >= 0 && dev < 64) cached[dev][i] = *n;
  return e;
}

}  // namespace

namespace {
// Clusters and parts of K of a product with N outputs (gated: N = H).  Parts: as
// many as leave every cluster on the GPU at once, each with at least four
// stages (clusters of 8 do not fill it: 16 of them, which would take 128 of 152
// SMs, run in two rounds).
cudaError_t split_k(int clusters, int num_kb, int* splits) {
  *splits = 1;
  for (int s = 2; s <= kMaxSplits && num_kb >= 4 * s; s *= 2) {
    int fit = 0;
    const cudaError_t e = max_clusters(s, &fit);
    if (e != cudaSuccess) return e;
    if (clusters > fit) break;
    *splits = s;
  }
  // every part has at least one stage
  while (*splits > 1 && (*splits - 1) * ((num_kb + *splits - 1) / *splits) >= num_kb) *splits /= 2;
  return cudaSuccess;
}
cudaError_t few_rows_split(int64_t M, int64_t N, int64_t K, bool gated, bool fp8, int* clusters, int* splits,
                           int* num_kb) {
  *num_kb = int((K + stage_k(fp8 ? OP_E4M3 : OP_BF16) - 1) / stage_k(fp8 ? OP_E4M3 : OP_BF16));
  *clusters = int((gated ? (N + 63) / 64 : (N + 127) / 128) * ((M + 127) / 128));
  return split_k(*clusters, *num_kb, splits);
}

// Rows per tile: the rows spread evenly over tiles of at most 128, in steps of 32.
int few_rows_bn(int64_t M) {
  const int64_t tiles = (M + 127) / 128;
  return int(((M + tiles - 1) / tiles + 31) / 32 * 32);
}
}  // namespace

// Up to `max_rows` rows (beyond: -1): an estimate in SM cycles, 5700 for the call, per
// round of clusters 500 for each stage and 39 for each row of a tile, 3900 for an
// exchange.  Fitted to 64 to 512 rows of the forms without block scales; with them, for
// which it is asked up to 4096 rows, calls take 6150, 520, 37 and 1300 (11% rms on 70 sizes of 9
// to 4000 rows), near enough that the choice by it (launch_linear_blocks) is 0.3%
// behind the better form on average.  Measured in us, here against
// linear.cu's forms: 64 rows of 2048 x 2048 6.9 / 8.2, of 4096 x 4096 10.6 / 12.9, of 4096 x
// 14336 23.3 / 28.4, of 4096 x 1024 6.7 / 6.2, of 14336 x 4096 23.1 / 22.3, 128 rows of
// 4096 x 4096 13.4 / 13.8, of 2048 x 2048 9.1 / 8.2, 256 rows of 14336 x 4096 33 / 27.5.
int64_t few_rows_cycles(int64_t M, int64_t N, int64_t K, bool gated, bool fp8, int64_t max_rows) {
  if (M > max_rows) return -1;
  int clusters, splits, num_kb;
  if (few_rows_split(M, N, K, gated, fp8, &clusters, &splits, &num_kb) != cudaSuccess) return -1;
  const int64_t rounds = (int64_t(clusters) * splits + kNumSMsHint - 1) / kNumSMsHint;
  return 5700 + rounds * (((num_kb + splits - 1) / splits) * 500 + 39 * few_rows_bn(M)) + (splits > 1 ? 3900 : 0);
}

// Stages, shared memory and TMEM of a CTA.
void size_cta(FewArgs& a, int clusters, int op) {
  a.stage_bytes = BOX_BYTES + a.bn * ROW_BYTES;
  const bool two = clusters * a.splits > kNumSMsHint;
  a.recv_bytes = (a.splits - 1) * (a.bn / a.splits) * 512;
  // (the sums, bn x 512 bytes, take at most 64 KB of the stages' 96 to 200 KB)
  const int extra = a.recv_bytes + (op == OP_BLOCKS ? kScaleStages * kScaleBytes : 0);
  a.stages = ((two ? kSmemTwo : kSmemOne) - extra) / a.stage_bytes;
  if (a.stages > kMaxStages) a.stages = kMaxStages;
  a.tmem_cols = 32;
  while (a.tmem_cols < a.bn + (op == OP_BLOCKS ? 16 : 0)) a.tmem_cols *= 2;   // (two slots of scales)
}

// One product: x [M, K] (K-major), W [wrows, K] or, w_mn, [K, wrows].
template <int OP, bool W_MN, int EPI>
cudaError_t few_rows_product(uint16_t* out, uint16_t* z, const void* x, const float* x_scale, const void* w,
                             const float* w_scale, const uint16_t* bias, const uint16_t* in, int act, int64_t M,
                             int64_t N, int64_t K, cudaStream_t s, bool late_wait = false,
                             const uint8_t* x_blocks = nullptr, const uint8_t* w_blocks = nullptr) {
  constexpr bool GATED = EPI != EPI_LINEAR;
  FewArgs a{};
  a.late_wait = late_wait ? 1 : 0;
  a.out = out;
  a.z = z;
  a.bias = bias;
  a.in = in;
  a.a_scale = x_scale;
  a.w_scale = w_scale;
  a.x_blocks = x_blocks;
  a.w_blocks = w_blocks;
  a.blocks = int((K + 127) / 128);
  a.act = act;
  a.M = int(M);
  a.N = int(N);
  a.tiles_m = int((M + 127) / 128);
  a.bn = few_rows_bn(M);
  int clusters = 0;
  const cudaError_t e = few_rows_split(M, N, K, GATED, OP != OP_BF16, &clusters, &a.splits, &a.num_kb);
  if (e != cudaSuccess) return e;
  size_cta(a, clusters, OP);
  CUtensorMap mw, mx;
  const bool bf16 = OP == OP_BF16;
  const bool ok = (W_MN ? make_operand_map(&mw, w, bf16, K, N, 64)
                        : make_operand_map(&mw, w, bf16, GATED ? 2 * N : N, K, GATED ? 64 : 128)) &&
                  make_operand_map(&mx, x, bf16, M, K, a.bn);
  if (!ok) return cudaErrorInvalidValue;
  return launch<OP, W_MN, EPI>(mw, mx, a, clusters, s);
}
cudaError_t launch_few_rows(uint16_t* out, uint16_t* z, const void* x, const float* x_scale, const void* w,
                            const float* w_scale, const uint16_t* bias, const uint16_t* res, int act, int64_t M,
                            int64_t N, int64_t K, bool fp8, bool w_mn, cudaStream_t s, bool late_wait) {
  if (fp8) return few_rows_product<OP_E4M3, false, EPI_LINEAR>(out, z, x, x_scale, w, w_scale, bias, res, act, M, N, K, s);
  if (w_mn)
    return few_rows_product<OP_BF16, true, EPI_LINEAR>(out, z, x, nullptr, w, nullptr, bias, res, act, M, N, K, s, late_wait);
  return few_rows_product<OP_BF16, false, EPI_LINEAR>(out, z, x, nullptr, w, nullptr, bias, res, act, M, N, K, s);
}

cudaError_t launch_few_rows_blocks(uint16_t* out, const uint8_t* x, const uint8_t* x_scale, const uint8_t* w,
                                   const uint8_t* w_scale, const uint16_t* bias, const uint16_t* res, int64_t M,
                                   int64_t N, int64_t K, cudaStream_t s) {
  return few_rows_product<OP_BLOCKS, false, EPI_LINEAR>(out, nullptr, x, nullptr, w, nullptr, bias, res, ACT_NONE, M, N,
                                                        K, s, false, x_scale, w_scale);
}

// Groups of rows: rows per tile, a quarter above the average group's, in steps of 32; tiles
// of rows, as many as there can be.
namespace {
int grouped_bn(int64_t G, int64_t M) {
  const int64_t rows = M / (G < M ? G : M) * 5 / 4;
  return rows >= 128 ? 128 : int((rows + 31) / 32 * 32);
}
int64_t grouped_clusters(int64_t G, int64_t M, int64_t N) {
  return (N + 127) / 128 * (M / grouped_bn(G, M) + (G < M ? G : M));
}
// Those that have rows where the groups are of average size.
int64_t expected_clusters(int64_t G, int64_t M, int64_t N) {
  const int64_t groups = G < M ? G : M, bn = grouped_bn(G, M);
  return (N + 127) / 128 * groups * ((M / groups + bn - 1) / bn);
}
// K is split for all of them, or for the expected ones where each part has 20 stages: the
// others take their turns too, some 2 us (184 rows in 15 groups of 152 x 11648 in parts of two 15.2
// us, of four 10.4; 400 in eight of 512 x 2048 7.2 and 10.0).
cudaError_t grouped_split(int64_t G, int64_t M, int64_t N, int num_kb, int* splits) {
  int all = 1;
  cudaError_t e = split_k(int(grouped_clusters(G, M, N)), num_kb, &all);
  if (e == cudaSuccess) e = split_k(int(expected_clusters(G, M, N)), num_kb, splits);
  if (*splits > all && num_kb < 20 * *splits) *splits = all;
  return e;
}
// out [M, N] from x [M, K] and w [G, N, K] or, W_MN, [G, K, N].
template <int OP, bool W_MN = false>
cudaError_t grouped_product(uint16_t* out, const void* x, const uint8_t* x_scale, const void* w, const uint8_t* w_scale,
                            const int* offsets, int64_t G, int64_t M, int64_t N, int64_t K, cudaStream_t s) {
  FewArgs a{};
  a.out = out;
  a.x_blocks = x_scale;
  a.w_blocks = w_scale;
  a.blocks = int((K + 127) / 128);
  a.offsets = offsets;
  a.G = int(G);
  a.M = int(M);
  a.N = int(N);
  a.act = ACT_NONE;
  a.bn = grouped_bn(G, M);
  a.tiles_m = int(M / a.bn + (G < M ? G : M));
  a.num_kb = int((K + stage_k(OP) - 1) / stage_k(OP));
  const int clusters = int(grouped_clusters(G, M, N));
  const cudaError_t e = grouped_split(G, M, N, a.num_kb, &a.splits);
  if (e != cudaSuccess) return e;
  size_cta(a, int(expected_clusters(G, M, N)), OP);
  CUtensorMap mw, mx;
  const bool bf16 = OP == OP_BF16;
  const int64_t pitch = K * (bf16 ? 2 : 1);
  const bool ok = (W_MN ? make_operand_map_3d(&mw, w, bf16, G, K, N, N * 2, K * N * 2, 64)
                        : make_operand_map_3d(&mw, w, bf16, G, N, K, pitch, N * pitch, 128)) &&
                  make_operand_map(&mx, x, bf16, M, K, a.bn);
  if (!ok) return cudaErrorInvalidValue;
  return launch<OP, W_MN, EPI_LINEAR, true>(mw, mx, a, clusters, s);
}
}  // namespace

// An estimate as few_rows_cycles for groups of rows of average size, fitted to 60 of 2 to 3000
// rows in 1 to 64 groups, in E4M3 and bf16: 7800 for the call, per round of clusters 500 for
// each stage and 34 for each row of a tile, 1500 for an exchange.
int64_t few_rows_grouped_cycles(int64_t G, int64_t M, int64_t N, int64_t K, bool fp8) {
  if (grouped_clusters(G, M, N) > 4 * kNumSMsHint) return -1;
  const int64_t clusters = expected_clusters(G, M, N);
  const int num_kb = int((K + stage_k(fp8 ? OP_E4M3 : OP_BF16) - 1) / stage_k(fp8 ? OP_E4M3 : OP_BF16));
  int splits = 1;
  if (grouped_split(G, M, N, num_kb, &splits) != cudaSuccess) return -1;
  const int64_t rounds = (clusters * splits + kNumSMsHint - 1) / kNumSMsHint;
  return 7800 + rounds * (((num_kb + splits - 1) / splits) * 500 + 34 * grouped_bn(G, M)) + (splits > 1 ? 1500 : 0);
}

cudaError_t launch_few_rows_grouped(uint16_t* out, const void* x, const uint8_t* x_scale, const void* w,
                                    const uint8_t* w_scale, const int* offsets, int64_t G, int64_t M, int64_t N,
                                    int64_t K, cudaStream_t s) {
  return x_scale != nullptr ? grouped_product<OP_BLOCKS>(out, x, x_scale, w, w_scale, offsets, G, M, N, K, s)
                            : grouped_product<OP_BF16>(out, x, nullptr, w, nullptr, offsets, G, M, N, K, s);
}

cudaError_t launch_few_rows_grouped_dx(uint16_t* dx, const uint16_t* dout, const uint16_t* w, const int* offsets, int64_t G,
                                       int64_t M, int64_t N, int64_t K, cudaStream_t s) {
  return grouped_product<OP_BF16, true>(dx, dout, nullptr, w, nullptr, offsets, G, M, K, N, s);
}

cudaError_t launch_few_rows_gated(uint16_t* out, const uint16_t* x, const uint16_t* w1, const uint16_t* dh, int act,
                                  int64_t M, int64_t C, int64_t H, cudaStream_t s) {
  if (dh != nullptr)
    return few_rows_product<OP_BF16, false, EPI_GATED_BWD>(out, nullptr, x, nullptr, w1, nullptr, nullptr, dh, act, M, H, C, s);
  return few_rows_product<OP_BF16, false, EPI_GATED>(out, nullptr, x, nullptr, w1, nullptr, nullptr, nullptr, act, M, H, C, s);
}

cudaError_t few_rows_take_status(unsigned int* status) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_status, sizeof(v));
  if (e != cudaSuccess) return e;
  if (v != 0) e = cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
  *status = v;
  return e;
}

}  // namespace qffn
