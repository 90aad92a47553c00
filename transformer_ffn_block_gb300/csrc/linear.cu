// Linear layers on the 5th-generation tensor cores (tcgen05, sm_103a) with
// bf16 or E4M3 operands and a fused epilogue:
//
//   EPI_LINEAR     out[M,N] = bf16(res + act(z)),  z = s * A[M,K] . W[N,K]^T + bias,
//                  z also stored (bf16) on request; s = 1 for bf16 operands
//   EPI_GATED      h[M,H]   = bf16(act(g) * u),  g / u the products with rows
//                  [0,H) / [H,2H) of W1, kept in fp32
//   EPI_GATED_BWD  d_gu[M,2H] = (dh * u * act'(g) | dh * act(g)) for the
//                  recomputed g, u and dh [M,H] read in the epilogue
//   EPI_PARTIAL    fp32 sums over one part of K, joined by join_kernel, which
//                  then applies one of the epilogues above
//
// The matmul and the epilogues of a transformer block's feed-forward half
// (llmq "llama_model.cpp", LLamaModel::_forward_block and _backward_block) in
// unquantised form; the gradients use EPI_LINEAR with MN-major operands
// (dx = dz . W, dW = dz^T . x read dz, W and x where they lie).
//
// Pipeline: SM pairs (2-CTA clusters), persistent over 256 x 256 tiles, one
// tcgen05.mma.cta_group::2 (M = 256, N = 256) chain per tile; CTA r of a pair
// stages rows [128 r, 128 r + 128) of A and of the tile's 256 weight rows, 128
// bytes of K per stage and row, six stages (eight of narrow units).  One warp loads
// (TMA, 128-byte swizzle), one thread of the leader issues the MMAs, eight warps
// per CTA run the epilogue out of one of two TMEM accumulators while the next
// tile accumulates in the other.  Per SM and byte of K this loads 16 + 16 KB per
// 128 x 256 outputs; a bf16 MMA takes twice the cycles of an E4M3 one over the
// same bytes of shared memory, so the operand feed has room to spare.  Units of
// fewer columns were bound by the issue of their MMAs, 70 cycles each with the
// issuing thread chosen by its lane's number, 24 by elect.sync; that and stages of
// one swizzle row instead of two took 512 x 4096 x 4096 from 19.4 to 16.0 us and
// the gated 8192 x 4096 x 14336 from 1066 to 1054.
//
// Every mbarrier wait is bounded; see gemm_fp8.cu for how a wait that runs out
// ends the kernel (abort flag, status word, drained copies and MMAs).
#include <cuda.h>

#include "act.cuh"
#include "common.cuh"
#include "launch.h"
#include "pipeline.cuh"
#include "tensor_map.h"
#include "umma.cuh"

namespace qffn {
namespace {

constexpr int BM = 128;                    // rows of A per CTA (256 per pair)
constexpr int BN = 256;                    // accumulator columns
constexpr int ROW_BYTES = 128;             // one swizzle atom row
constexpr int OP_BYTES = 128 * ROW_BYTES;  // an operand's share of a stage: 128 rows of one swizzle row
constexpr int MN_BOX_BYTES = 64 * ROW_BYTES;   // MN-major: 64 values by 64 of K, two boxes to the share
constexpr int MAX_STAGES = 8;
constexpr int RING_BYTES = 6 * 2 * OP_BYTES;   // the stages: six of whole units, eight of narrow ones
constexpr int STEPS = 4;                   // MMAs per stage (32 bytes of K each)
constexpr int EPI_WARPS = 8;
constexpr int NUM_THREADS = 64 + 32 * EPI_WARPS;
constexpr int TMEM_COLS = 2 * BN;
constexpr int NUM_BARS = 2 * MAX_STAGES + 5;
constexpr int STAGING_BOX = 32 * 128;      // a warp's transposing box: 32 rows x 32 fp32
constexpr int STAGING_BYTES = EPI_WARPS * STAGING_BOX;
constexpr int SMEM_BYTES = RING_BYTES + STAGING_BYTES + 1024 + NUM_BARS * 8 + 16;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory of one CTA");
constexpr int GROUP_M = 8;
constexpr uint16_t kBothCtas = 0x3;
constexpr uint16_t kLeaderOnly = 0x1;
constexpr unsigned long long kWaitLimitNs = 2000000000ull;
constexpr unsigned long long kDrainLimitNs = 200000000ull;

constexpr int OP_BF16 = 0, OP_E4M3 = 1;
constexpr int stage_k(int op) { return op == OP_BF16 ? 64 : 128; }   // elements of K per stage

constexpr int EPI_LINEAR = 0, EPI_GATED = 1, EPI_GATED_BWD = 2, EPI_PARTIAL = 3;

// Instruction descriptor: D fp32 (bits 4-5 = 1); A and B formats at bits 7-9
// and 10-12 (kind::f16: 1 = bf16; kind::f8f6f4: 0 = E4M3); bits 15 / 16: A / B
// MN-major; N >> 3 at bits 17-22, M >> 4 at bits 24-28 (M = 256 over the pair).
QFFN_DEVI constexpr uint32_t idesc_for(int op, bool a_mn, bool b_mn, int n) {
  return (1u << 4) | (op == OP_BF16 ? (1u << 7) | (1u << 10) : 0u) | (a_mn ? 1u << 15 : 0u) |
         (b_mn ? 1u << 16 : 0u) | (uint32_t(n >> 3) << 17) | (uint32_t((2 * BM) >> 4) << 24);
}

QFFN_DEVI uint32_t pack2(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return pack_bf16x2(lo, hi);
}
QFFN_DEVI uint4 pack8(const uint64_t (&v)[4]) { return make_uint4(pack2(v[0]), pack2(v[1]), pack2(v[2]), pack2(v[3])); }

__device__ unsigned int g_status;

struct LinArgs {
  const float* a_scale;     // E4M3 operands: one float each; NULL: no scaling
  const float* w_scale;
  uint16_t* out;            // [M, N] (GATED_BWD: [M, 2N])
  uint16_t* z;              // EPI_LINEAR, optional
  const uint16_t* bias;     // EPI_LINEAR, optional
  const uint16_t* in;       // [M, N]: EPI_LINEAR residual or previous output (optional), GATED_BWD dh
  int M, N;                 // output rows and columns (gated: columns = H)
  int narrow;               // every unit is BN >> narrow accumulator columns wide
  int bn, stages;           // SWAP: accumulator columns of a unit, stages of the ring
  int up_row;               // gated: first up row of W1 (= H)
  int tiles_m, tiles_n, num_units, num_kb;
  int band_n;               // N-blocks per raster band
  int split_from;           // units from here on are 128-column halves of the last tiles
  int early, early_units;   // the first `early` pairs share the first early_units units, all pairs the rest
  int splits, kb_per_split, m_pad;   // EPI_PARTIAL
  float* partial;           // EPI_PARTIAL: [splits][m_pad][N]
  int late_wait;            // does not read the preceding kernel's results (see launch.h)
};

// D(tmem, both CTAs) (+)= A(smem, both CTAs) . B(smem, both CTAs)^T
template <int OP>
QFFN_DEVI void mma_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  if (OP == OP_BF16)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Shared-memory descriptor of MMA step i of a stage's operand.
// K-major: 32 bytes along its 128-byte rows per step.  MN-major (16-bit types):
// the operand's 128 M (N) values lie in two boxes of 64 values x 64 K rows; a step
// is 16 K rows of 128 bytes (8-row groups 1024 bytes apart) in both boxes, whose
// distance is the leading byte offset.
template <bool MN>
QFFN_DEVI uint64_t step_desc(uint32_t base, int i) {
  if (!MN) return sdesc_sw128(base + uint32_t(i) * 32u);
  const uint64_t d = sdesc_sw128(base + uint32_t(i) * 16u * ROW_BYTES);
  return (d & ~(uint64_t(0x3FFF) << 16)) | (uint64_t(MN_BOX_BYTES >> 4) << 16);
}

QFFN_DEVI bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, bool honour_abort = true,
                         unsigned long long limit = kWaitLimitNs) {
  return mbar_wait_bounded(bar, parity, abort_flag, &g_status, honour_abort, limit);
}

struct Unit {
  int mb, nb;      // pair M-block (256 rows), N-block
  int half;        // -1: whole tile; 0 / 1: first / second half of a split one (narrow = 0 only)
  int sp;          // EPI_PARTIAL: part of K
};

template <int EPI>
QFFN_DEVI Unit unit_coords(int u, const LinArgs& a) {
  Unit r;
  r.half = -1;
  r.sp = 0;
  int tile = u;
  if (EPI == EPI_PARTIAL) {
    tile = u / a.splits;
    r.sp = u - tile * a.splits;
  } else if (u >= a.split_from) {
    tile = a.split_from + ((u - a.split_from) >> 1);
    r.half = (u - a.split_from) & 1;
  }
  // bands of band_n N-blocks; within a band, groups of GROUP_M M-blocks sweep
  // the band's N-blocks, M fastest, odd groups backwards.  (Every warp of the
  // epilogue computes this for every unit, in the open: a division is some 40
  // instructions, so those that have a known answer are left out.)
  const int band_tiles = a.tiles_m * a.band_n;
  const int band = tile < band_tiles ? 0 : tile / band_tiles;
  const int n0 = band * a.band_n;
  const int wb = min(a.band_n, a.tiles_n - n0);
  const int t = tile - band * band_tiles;
  const int per_group = GROUP_M * wb;
  const int group = t < per_group ? 0 : t / per_group;
  const int first_m = group * GROUP_M;
  const int gsize = min(a.tiles_m - first_m, GROUP_M);
  const int k = t - group * per_group;
  const int col = gsize == GROUP_M ? k / GROUP_M : gsize == 1 ? k : k / gsize;
  r.mb = first_m + k - col * gsize;
  r.nb = n0 + ((group & 1) ? wb - 1 - col : col);
  return r;
}

// The units of a pair, in order: first_unit, then next_unit of it.
QFFN_DEVI int first_unit(int pair, const LinArgs& a) { return pair < a.early ? pair : a.early_units + pair; }
QFFN_DEVI int next_unit(int un, int pair, int num_pairs, const LinArgs& a) {
  if (un >= a.early_units) return un + num_pairs;
  return un + a.early < a.early_units ? un + a.early : a.early_units + pair;
}

// tmB: B with boxes of 128 >> narrow rows; tmBh: of 64 rows, for the half tiles.
// SWAP: A is W and B is x with boxes of bn / 2 rows, so a unit is 256 output
// columns (the TMEM lanes) by bn output rows.
template <int OP, int EPI, int ACT, bool A_MN, bool B_MN, bool SWAP>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    linear_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ CUtensorMap tmBh, const LinArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sStaging = smem + RING_BYTES;
  // a stage: this CTA's A rows, then its B rows
  const int bn = SWAP ? args.bn : BN >> args.narrow;           // accumulator columns of a whole unit
  const uint32_t ring = smem_u32(smem), stage_bytes = uint32_t(OP_BYTES + bn / 2 * ROW_BYTES);
  const int stages = SWAP ? args.stages : args.narrow == 0 ? 6 : MAX_STAGES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sStaging + STAGING_BYTES);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NUM_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t bar0 = smem_u32(bars);
  // full[s] (leader): both CTAs' loads of stage s landed; empty[s]: the MMAs
  // reading stage s are done; tfull[a]: accumulator a is complete; tempty[a]
  // (leader): both CTAs' epilogue warps have read it; drain: all MMAs done
  auto full_bar = [&](int s) { return bar0 + 8u * uint32_t(s); };
  auto empty_bar = [&](int s) { return bar0 + 8u * uint32_t(MAX_STAGES + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * uint32_t(2 * MAX_STAGES + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * uint32_t(2 * MAX_STAGES + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * uint32_t(2 * MAX_STAGES + 4);

  constexpr bool GATED = EPI == EPI_GATED || EPI == EPI_GATED_BWD;
  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = int(cluster_id_x()), num_pairs = int(num_clusters_x());

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 2 * EPI_WARPS);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  cluster_sync_all();      // both CTAs' barriers exist before either signals the other's
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  if (!args.late_wait) pdl_wait();   // nothing in global memory is touched before the preceding kernel is done
  const uint16_t* const bias_row = behind_wait(args.bias);
  pdl_trigger();

  // K blocks of a unit
  auto kb_begin = [&](const Unit& u) { return EPI == EPI_PARTIAL ? u.sp * args.kb_per_split : 0; };
  auto kb_end = [&](const Unit& u) {
    return EPI == EPI_PARTIAL ? min(args.num_kb, (u.sp + 1) * args.kb_per_split) : args.num_kb;
  };

  if (warp == 0) {
    if (elect_one()) {
      // ------------------------------------------------------------ producer
      uint32_t issued = 0, issued_parity = 0, ph = 0;
      int s = 0;
      bool ok = true;
      for (int un = first_unit(pair, args); ok && un < args.num_units; un = next_unit(un, pair, num_pairs, args)) {
        const Unit u = unit_coords<EPI>(un, args);
        const int rowA = (SWAP ? u.nb : u.mb) * (2 * BM) + int(rank) * BM;
        // this CTA's weight rows: half of the tile's 256 (of a half tile's
        // 128); gated: CTA 0 the gate rows, CTA 1 the matching up rows
        const int rowB = SWAP    ? u.mb * bn + int(rank) * (bn / 2)
                         : GATED ? (rank == 0 ? 0 : args.up_row) + u.nb * (bn / 2) + (u.half < 0 ? 0 : u.half * 64)
                         : u.half < 0 ? u.nb * bn + int(rank) * (bn / 2)
                                      : u.nb * BN + u.half * 128 + int(rank) * 64;
        const uint32_t stage_tx = 2u * (u.half < 0 ? stage_bytes : uint32_t(OP_BYTES + OP_BYTES / 2));
        const int kb1 = kb_end(u);
        for (int kb = kb_begin(u); kb < kb1; ++kb) {
          if (!mbar_wait(empty_bar(s), ph ^ 1u, abort_flag)) { ok = false; break; }
          if (rank == 0) mbar_expect_tx(full_bar(s), stage_tx);
          const uint32_t fb = map_to_rank(full_bar(s), 0);
          const int k0 = kb * stage_k(OP);
          const uint32_t da = ring + uint32_t(s) * stage_bytes, db = da + uint32_t(OP_BYTES);
          if (A_MN) {
            tma_load_2d_pair(da, &tmA, fb, rowA, k0);
            tma_load_2d_pair(da + MN_BOX_BYTES, &tmA, fb, rowA + 64, k0);
          } else {
            tma_load_2d_pair(da, &tmA, fb, k0, rowA);
          }
          if (B_MN) {
            tma_load_2d_pair(db, &tmB, fb, rowB, k0);
            // (the 64 rows of a half tile or a narrow unit are one box)
            if (u.half < 0 && args.narrow == 0) tma_load_2d_pair(db + MN_BOX_BYTES, &tmB, fb, rowB + 64, k0);
          } else {
            tma_load_2d_pair(db, u.half < 0 ? &tmB : &tmBh, fb, k0, rowB);
          }
          issued |= 1u << s;
          issued_parity = (issued_parity & ~(1u << s)) | (ph << s);
          if (++s == stages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      // before shared memory is released every phase the leader armed completes, and
      // the MMAs' last arrivals reach this CTA
      for (int k = 0; k < stages; ++k)
        if (issued & (1u << k)) {
          if (rank == 0) mbar_wait(full_bar(k), (issued_parity >> k) & 1u, abort_flag, false, kDrainLimitNs);
          mbar_wait(empty_bar(k), (issued_parity >> k) & 1u, abort_flag, false, kDrainLimitNs);
        }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      // ------------------------------------------------------------ MMA issuer (leader)
      int s = 0, local = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int un = first_unit(pair, args); ok && un < args.num_units;
           un = next_unit(un, pair, num_pairs, args), ++local) {
        const int acc = local & 1;
        const uint32_t aph = uint32_t(local >> 1) & 1u;
        if (!mbar_wait_cluster_bounded(tempty_bar(acc), aph ^ 1u, abort_flag, &g_status, kWaitLimitNs)) break;
        tc_fence_after();
        const Unit u = unit_coords<EPI>(un, args);
        const uint32_t d_tmem = tmem_base + uint32_t(acc * BN);
        const uint32_t idesc = idesc_for(OP, A_MN, B_MN, u.half < 0 ? bn : BN / 2);
        const int kb0 = kb_begin(u), kb1 = kb_end(u);
        bool ready = false;                  // the next stage was there before this one's MMAs were issued
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!ready && !mbar_wait(full_bar(s), ph, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a0 = ring + uint32_t(s) * stage_bytes, b0 = a0 + uint32_t(OP_BYTES), empty = empty_bar(s);
          if (++s == stages) {
            s = 0;
            ph ^= 1u;
          }
          ready = kb + 1 < kb1 && mbar_test_wait(full_bar(s), ph);
#pragma unroll
          for (int i = 0; i < STEPS; ++i)
            mma_pair<OP>(d_tmem, step_desc<A_MN>(a0, i), step_desc<B_MN>(b0, i), idesc,
                         uint32_t((kb - kb0) | i));
          mma_commit_mc(empty, kBothCtas);
        }
        if (!ok) break;
        mma_commit_mc(tfull_bar(acc), kBothCtas);
      }
      mma_commit_mc(drain_bar, kLeaderOnly);
      mbar_wait(drain_bar, 0, abort_flag, false, kDrainLimitNs);
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- epilogue
    // EPI_WARPS / 4 warps per TMEM lane quarter q (rows 32 q .. 32 q + 31 of
    // the CTA's 128), which share the unit's groups of 32 output columns.
    // A TMEM load gives a lane one row's 32 columns; a warp's box of shared
    // memory turns that into the layout of the global accesses, lane l with 8
    // columns (8 (l & 3) ..) of the rows (l >> 2) + 8 i, so that every load and
    // store of 16 bytes per lane covers eight rows of 64 contiguous bytes
    // (partial sums: 128).  Both directions use the box without bank conflicts.
    constexpr int WG = EPI_WARPS / 4;
    const int q = warp & 3, wg = (warp - 2) >> 2;
    const float scale = args.a_scale != nullptr ? args.a_scale[0] * args.w_scale[0] : 1.0f;
    const int sub = lane >> 2, ch = lane & 3;
    const uint32_t box = smem_u32(sStaging + (q * WG + wg) * STAGING_BOX);
    // 32 fp32 columns (rows of 128 bytes, 16-byte chunk c of row r at c ^ (r & 7)):
    // this lane's row is written at row32 ^ 16 c, its turned share read at
    // turn32 and turn32 ^ 16, plus 1024 i
    const uint32_t row32 = box + uint32_t(lane) * 128u + (uint32_t(lane & 7) << 4);
    const uint32_t turn32 = box + uint32_t(sub) * 128u + (uint32_t((2 * ch) ^ sub) << 4);
    // (a lane's column: at col32 ^ 16 (r & 7), plus 128 r)
    const uint32_t col32 = box + uint32_t(lane) * 4u;
    // 32 bf16 columns (rows of 64 bytes, chunk c of row r at c ^ (r / 2 & 3)): row
    // at row16 ^ 16 c, turned share at turn16 plus 512 i; a second such box behind
    const uint32_t row16 = box + uint32_t(lane) * 64u + (uint32_t((lane >> 1) & 3) << 4);
    const uint32_t turn16 = box + uint32_t(sub) * 64u + (uint32_t(ch ^ ((sub >> 1) & 3)) << 4);
    constexpr uint32_t kBox2 = 32 * 64;
    constexpr bool kRead = EPI == EPI_LINEAR || EPI == EPI_GATED_BWD;   // may read a bf16 tensor
    int local = 0;
    constexpr bool kPlain = EPI == EPI_LINEAR && ACT == ACT_NONE && !SWAP;
    const bool plain = kPlain && args.bias == nullptr && args.z == nullptr;
    if (plain) {
      // out = bf16(s * sum (+ in)) alone, the gradients': with few K blocks per unit
      // the epilogue bounds the kernel, so it takes 64 columns at a time (whole
      // 128-byte lines), turns them as bf16, and requests what it adds a unit ahead
      // (weight gradient of one row, 8192 x 4096, us: 32 columns through fp32 22.1, so
      // 14.7; added to the previous one 41.2 and 32.3).  The box holds 32 rows of 128
      // bytes, chunk c of row r at c ^ (r & 7); a lane writes its accumulator row and
      // takes chunk ch8 of the rows sub8 + 4 i.
      const int sub8 = lane >> 3, ch8 = lane & 7;
      const uint32_t turn8 = box + uint32_t(sub8) * 128u + (uint32_t(ch8 ^ sub8) << 4);
      const size_t step4 = size_t(4) * size_t(args.N);
      struct Part {
        int g0, g1, col;                     // groups of this warp, column of this lane's share of group 0
        uint32_t rows;                       // bit i: row sub8 + 4 i exists
        size_t at;                           // element offset of that share's first row
      };
      auto part_of = [&](const Unit& u) {
        Part p;
        const int row0 = u.mb * (2 * BM) + int(rank) * BM + q * 32;
        p.g0 = wg;
        p.g1 = (u.half < 0 ? bn : BN / 2) / 64;
        p.col = u.nb * bn + (u.half < 0 ? 0 : u.half * 128) + ch8 * 8;
        p.rows = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) p.rows |= (row0 + sub8 + 4 * i < args.M ? 1u : 0u) << i;
        p.at = size_t(row0 + sub8) * size_t(args.N) + size_t(p.col);
        return p;
      };
      uint4 in8[2][8];
      auto request = [&](const Part& p, int k, uint4 (&d)[8]) {
        const int g = p.g0 + k * WG;
        const uint32_t live = g < p.g1 && p.col + g * 64 < args.N ? p.rows : 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          d[i] = make_uint4(0, 0, 0, 0);
          if ((live >> i) & 1u) d[i] = ld16_stream(args.in + (p.at + size_t(g * 64) + size_t(i) * step4));
        }
      };
      int un = first_unit(pair, args);
      Part p = part_of(unit_coords<EPI>(un, args));
      if (args.in != nullptr) {
        request(p, 0, in8[0]);
        request(p, 1, in8[1]);
      }
      for (; un < args.num_units; ++local) {
        const int acc = local & 1;
        const uint32_t aph = uint32_t(local >> 1) & 1u;
        const uint32_t tbase = tmem_base + (uint32_t(q * 32) << 16) + uint32_t(acc * BN);
        const int next = next_unit(un, pair, num_pairs, args);
        const bool awaited = next < args.num_units && next_unit(next, pair, num_pairs, args) < args.num_units;
        const Part p_next = part_of(unit_coords<EPI>(next < args.num_units ? next : un, args));
        if (!mbar_wait(tfull_bar(acc), aph, abort_flag)) break;
        tc_fence_after();
        auto loaded = [&](int g) {
          if (g + WG >= p.g1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && awaited) mbar_arrive_remote_relaxed(map_to_rank(tempty_bar(acc), 0));
          }
        };
        if (p.g0 >= p.g1) loaded(p.g0);      // (a unit with fewer groups than warps)
#pragma unroll
        for (int k = 0; k < 2; ++k) {        // a warp has two groups at most
          const int g = p.g0 + k * WG;
          __syncwarp();                      // the previous group has been read out of the box
          if (args.in != nullptr) {
#pragma unroll
            for (int i = 0; i < 8; ++i) sts16((turn8 ^ uint32_t((i & 1) << 6)) + 512u * i, in8[k][i]);
            __syncwarp();
            if (next < args.num_units) request(p_next, k, in8[k]);
          }
          if (g >= p.g1) continue;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t v[32];
            tmem_ld32(tbase + uint32_t(g * 64 + h * 32), v);
            if (h == 1) loaded(g);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t addr = row32 ^ uint32_t(16 * (4 * h + c));
              uint64_t z[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                z[j] = f2_pack(__uint_as_float(v[8 * c + 2 * j]), __uint_as_float(v[8 * c + 2 * j + 1]));
                if (OP == OP_E4M3) z[j] = f2_mul(z[j], f2_dup(scale));
              }
              if (args.in != nullptr) {
                const uint4 d = lds16(addr);
                const uint32_t dw[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) z[j] = f2_add(z[j], bf16x2_to_f2(dw[j]));
              }
              sts16(addr, pack8(z));
            }
          }
          __syncwarp();
          const uint32_t live = p.col + g * 64 < args.N ? p.rows : 0u;
          uint16_t* const dst = args.out + (p.at + size_t(g * 64));
          uint4 o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = lds16((turn8 ^ uint32_t((i & 1) << 6)) + 512u * i);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if ((live >> i) & 1u) stg16(dst + size_t(i) * step4, o[i]);
        }
        un = next;
        p = p_next;
      }
    }
    for (int un = plain ? args.num_units : first_unit(pair, args); un < args.num_units; un = next_unit(un, pair, num_pairs, args), ++local) {
      const int acc = local & 1;
      const uint32_t aph = uint32_t(local >> 1) & 1u;
      const Unit u = unit_coords<EPI>(un, args);
      // output row and column of the unit's group 0 for this warp; SWAP: the
      // groups are of 32 rows and the warp's quarter of the lanes is 32 columns
      const int row0 = SWAP ? u.mb * bn : u.mb * (2 * BM) + int(rank) * BM + q * 32;
      const int row_end = SWAP ? min(args.M, row0 + bn) : args.M;
      const int first_col = SWAP    ? u.nb * (2 * BM) + int(rank) * BM + q * 32
                            : GATED ? u.nb * (bn / 2) + (u.half < 0 ? 0 : u.half * 64)
                                    : u.nb * bn + (u.half < 0 ? 0 : u.half * 128);
      const uint32_t tbase = tmem_base + (uint32_t(q * 32) << 16) + uint32_t(acc * BN);
      const int acc_cols = u.half < 0 ? bn : BN / 2;
      const int groups = GATED ? acc_cols / 64 : (acc_cols + 31) / 32;
      // this warp's groups, next to each other: whole 128-byte lines from one
      // warp (interleaved groups: 8192 x 8192 x 64 with a residual 80 us, so 73)
      const int share = (groups + WG - 1) / WG, g0 = wg * share, g1 = min(groups, g0 + share);
      // this lane's part of the global accesses of group g: rows sub + 8 i behind
      // the group's first (bit i of live_rows: there is one), element offset of the first
      uint32_t rows = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) rows |= (row0 + sub + 8 * i < args.M ? 1u : 0u) << i;
      const size_t at = size_t(row0 + sub) * size_t(args.N) + size_t(first_col + ch * 8);
      const size_t step = size_t(8) * size_t(args.N);
      auto col = [&](int g) { return first_col + (SWAP ? 0 : g * 32) + ch * 8; };
      auto live_rows = [&](int g) {
        if (col(g) >= args.N) return 0u;
        if (!SWAP) return rows;
        uint32_t v = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) v |= (row0 + g * 32 + sub + 8 * i < row_end ? 1u : 0u) << i;
        return v;
      };
      auto offset = [&](int g) { return SWAP ? at + size_t(4 * g) * step : at + size_t(g * 32); };
      // what a group reads from global memory, requested a group ahead (the
      // first group's before the accumulator is awaited)
      uint4 next_bias = make_uint4(0, 0, 0, 0), next_in[4];
      auto request = [&](int g) {
        const uint32_t live = g < g1 ? live_rows(g) : 0u;
        if (EPI == EPI_LINEAR && args.bias != nullptr)
          next_bias = live != 0u ? ld16_settled(bias_row + col(g)) : make_uint4(0, 0, 0, 0);
        if (kRead && args.in != nullptr) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            next_in[i] = make_uint4(0, 0, 0, 0);
            if ((live >> i) & 1u) next_in[i] = ld16_stream(args.in + (offset(g) + size_t(i) * step));
          }
        }
      };
      if (kRead) request(g0);
      if (!mbar_wait(tfull_bar(acc), aph, abort_flag)) break;
      tc_fence_after();
      // after this warp's last load of the accumulator: hand it back (if another
      // unit takes it: no arrival is on its way when the leader ends)
      const int next = next_unit(un, pair, num_pairs, args);
      const bool awaited = next < args.num_units && next_unit(next, pair, num_pairs, args) < args.num_units;
      auto loaded = [&](int g) {
        if (g + 1 >= g1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0 && awaited) mbar_arrive_remote_relaxed(map_to_rank(tempty_bar(acc), 0));
        }
      };
      if (g0 >= g1) loaded(g0);              // (a unit with fewer groups than warps)
      for (int g = g0; g < g1; ++g) {
        const uint32_t live = live_rows(g);
        if (!GATED) {
          uint4 in4[4];
          uint64_t bias[4];
          const uint32_t bw[4] = {next_bias.x, next_bias.y, next_bias.z, next_bias.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) bias[j] = bf16x2_to_f2(bw[j]);
          if (EPI == EPI_LINEAR && args.in != nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i) in4[i] = next_in[i];
          }
          {
            uint32_t v[32];
            tmem_ld32(tbase + uint32_t(g * 32), v);
            loaded(g);
            __syncwarp();                    // the previous group has been read out of the box
            if (SWAP) {                      // the lane is a column of the box
#pragma unroll
              for (int c = 0; c < 32; ++c) sts4((col32 ^ uint32_t(16 * (c & 7))) + uint32_t(128 * c), v[c]);
            } else {
#pragma unroll
              for (int c = 0; c < 8; ++c)
                sts16(row32 ^ uint32_t(16 * c), make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]));
            }
            __syncwarp();
          }
          if (kRead) request(g + 1);
          const size_t o = EPI == EPI_PARTIAL
                               ? (size_t(u.sp) * size_t(args.m_pad)) * size_t(args.N) + offset(g)
                               : offset(g);
          uint4 los[4], his[4];              // all reads issued before the first is used
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            los[i] = lds16(turn32 + 1024u * i);
            his[i] = lds16((turn32 ^ 16u) + 1024u * i);
          }
          if (EPI == EPI_PARTIAL) {
            float* const dst = args.partial + o;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if ((live >> i) & 1u) {
                stg16(dst + size_t(i) * step, los[i]);
                stg16(dst + size_t(i) * step + 4, his[i]);
              }
          } else {
            // each step over all four rows: sixteen independent pairs, so that the
            // two warps of a scheduler cover the latencies of the activation
            uint64_t z[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              z[i][0] = f2_pack(__uint_as_float(los[i].x), __uint_as_float(los[i].y));
              z[i][1] = f2_pack(__uint_as_float(los[i].z), __uint_as_float(los[i].w));
              z[i][2] = f2_pack(__uint_as_float(his[i].x), __uint_as_float(his[i].y));
              z[i][3] = f2_pack(__uint_as_float(his[i].z), __uint_as_float(his[i].w));
              if (OP == OP_E4M3) {
#pragma unroll
                for (int j = 0; j < 4; ++j) z[i][j] = f2_mul(z[i][j], f2_dup(scale));
              }
            }
            if (args.bias != nullptr) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) z[i][j] = f2_add(z[i][j], bias[j]);
            }
            if (args.z != nullptr) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if ((live >> i) & 1u) stg16(args.z + (o + size_t(i) * step), pack8(z[i]));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) z[i][j] = act_f2<ACT>(z[i][j]);
            if (args.in != nullptr) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t iw[4] = {in4[i].x, in4[i].y, in4[i].z, in4[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) z[i][j] = f2_add(z[i][j], bf16x2_to_f2(iw[j]));
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if ((live >> i) & 1u) stg16(args.out + (o + size_t(i) * step), pack8(z[i]));
          }
        } else {
          __syncwarp();                      // the previous group has been read out of the boxes
          if (EPI == EPI_GATED_BWD) {
            // dh into the box, read back row by row below
#pragma unroll
            for (int i = 0; i < 4; ++i) sts16(turn16 + 512u * i, next_in[i]);
            __syncwarp();
            request(g + 1);
          }
          const int up_off = acc_cols / 2;   // accumulator column of u
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            const uint32_t c = uint32_t(g * 32 + h * 16);
            uint32_t gv[16], uv[16];
            tmem_ld16x2_issue(tbase + c, tbase + uint32_t(up_off) + c, gv, uv);
            tmem_wait_ld16(gv, uv);
            if (h == 1) loaded(g);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t off = row16 ^ uint32_t(16 * (h * 2 + k));
              uint32_t p[4], p2[4];
              uint4 d4 = make_uint4(0, 0, 0, 0);
              if (EPI == EPI_GATED_BWD) d4 = lds16(off);
              const uint32_t dw[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint64_t gp = f2_pack(__uint_as_float(gv[8 * k + 2 * j]), __uint_as_float(gv[8 * k + 2 * j + 1]));
                const uint64_t up = f2_pack(__uint_as_float(uv[8 * k + 2 * j]), __uint_as_float(uv[8 * k + 2 * j + 1]));
                if (EPI == EPI_GATED) {
                  p[j] = pack2(f2_mul(act_f2<ACT>(gp), up));
                } else {
                  uint64_t f, df;
                  act_grad_f2<ACT>(gp, f, df);
                  const uint64_t d = bf16x2_to_f2(dw[j]);
                  p[j] = pack2(f2_mul(f2_mul(d, up), df));
                  p2[j] = pack2(f2_mul(d, f));
                }
              }
              sts16(off, make_uint4(p[0], p[1], p[2], p[3]));
              if (EPI == EPI_GATED_BWD) sts16(off + kBox2, make_uint4(p2[0], p2[1], p2[2], p2[3]));
            }
          }
          __syncwarp();
          // d_gu has rows of 2 N
          uint16_t* const dst = EPI == EPI_GATED_BWD
                                    ? args.out + (at + size_t(row0 + sub) * size_t(args.N) + size_t(g * 32))
                                    : args.out + (at + size_t(g * 32));
          const size_t dstep = EPI == EPI_GATED_BWD ? 2 * step : step;
          uint4 first[4], second[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            first[i] = lds16(turn16 + 512u * i);
            if (EPI == EPI_GATED_BWD) second[i] = lds16(turn16 + 512u * i + kBox2);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (((live >> i) & 1u) == 0u) continue;
            stg16(dst + size_t(i) * dstep, first[i]);
            if (EPI == EPI_GATED_BWD) stg16(dst + size_t(i) * dstep + args.N, second[i]);
          }
        }
      }
    }
  }

  // Both CTAs finish together: the leader's MMAs write the peer's TMEM and
  // both CTAs signal barriers of the other.
  // (Nothing remote is left to order: every arrival and copy that the other CTA
  // makes here has been waited for.  So the barrier need not wait for this
  // kernel's global stores, 0.3 us.)
  tc_fence_before();
  __syncthreads();
  cluster_sync_relaxed();
  if (args.late_wait) pdl_wait();    // this kernel is not complete before the preceding one
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS)
                 : "memory");
  }
}

// ------------------------------------------------------------------ joining the parts of K
// Eight output columns per thread: the parts' fp32 sums added in order, then
// the epilogue.  partial is [splits][m_pad][ld]; gated forms read columns c
// and H + c.
template <int EPI, int ACT>
__global__ void __launch_bounds__(256) join_kernel(uint16_t* out, uint16_t* out2, const float* partial,
                                                   const uint16_t* bias, const uint16_t* in, const float* a_scale,
                                                   const float* w_scale, int splits, int64_t m_pad, int64_t ld,
                                                   int64_t M, int64_t N) {
  pdl_wait();
  pdl_trigger();
  const int64_t per_row = N >> 3;
  const int64_t total = M * per_row;
  const float scale = a_scale != nullptr ? a_scale[0] * w_scale[0] : 1.0f;
  auto sum8 = [&](int64_t row, int64_t col, float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 0.0f;
    for (int s = 0; s < splits; ++s) {
      const float4* p = reinterpret_cast<const float4*>(partial + (size_t(s) * size_t(m_pad) + size_t(row)) * size_t(ld) + size_t(col));
      const float4 a = p[0], b = p[1];
      f[0] += a.x; f[1] += a.y; f[2] += a.z; f[3] += a.w;
      f[4] += b.x; f[5] += b.y; f[6] += b.z; f[7] += b.w;
    }
  };
  auto pack = [](const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  };
  auto unpack = [](uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = bf16_lo(w[j]);
      f[2 * j + 1] = bf16_hi(w[j]);
    }
  };
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < total; i += int64_t(gridDim.x) * 256) {
    const int64_t row = i / per_row, col = (i - row * per_row) * 8;
    float z[8], t[8];
    sum8(row, col, z);
    if (EPI == EPI_LINEAR) {
#pragma unroll
      for (int j = 0; j < 8; ++j) z[j] *= scale;
      if (bias != nullptr) {
        unpack(ld16_once(bias + col), t);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] += t[j];
      }
      if (out2 != nullptr) stg16(out2 + row * N + col, pack(z));
#pragma unroll
      for (int j = 0; j < 8; ++j) z[j] = act_f32<ACT>(z[j]);
      if (in != nullptr) {
        unpack(ld16_once(in + row * N + col), t);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] += t[j];
      }
      stg16(out + row * N + col, pack(z));
    } else {
      float up[8];
      sum8(row, N + col, up);
      if (EPI == EPI_GATED) {
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = act_f32<ACT>(z[j]) * up[j];
        stg16(out + row * N + col, pack(z));
      } else {
        unpack(ld16_once(in + row * N + col), t);
        float du[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float f, df;
          act_grad_f32<ACT>(z[j], f, df);
          z[j] = t[j] * up[j] * df;
          du[j] = t[j] * f;
        }
        stg16(out + row * 2 * N + col, pack(z));
        stg16(out + row * 2 * N + N + col, pack(du));
      }
    }
  }
}

// ------------------------------------------------------------------ dz = dout * act'(z) and its column sums
// A block covers 256 columns (one warp's 32 lanes x 8 columns) and every
// (8 * gridDim.y)-th group of rows; thread (warp w, lane l) owns columns
// 8 l .. 8 l + 7 of rows w, w + 8, ...  The column sums are taken from the fp32
// dz before its rounding; the block's eight warps are added in order and
// column_sum_kernel adds the blocks' (few rows take one block per 256 columns,
// which writes dbias itself).  ACT_NONE (dz = dout) only sums.
constexpr int kRowsInFlight = 4;           // loads issued per thread before the first is used
template <int ACT>
__global__ void __launch_bounds__(256) act_backward_kernel(uint16_t* dz, float* partial, float* dbias,
                                                           const uint16_t* dout, const uint16_t* z, int64_t M,
                                                           int64_t N, int accumulate) {
  __shared__ __align__(8) float comb[8][256 + 8];
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  const int64_t col = int64_t(blockIdx.x) * 256 + l * 8;
  const bool live = col < N;
  pdl_wait();
  pdl_trigger();
  uint64_t s[4] = {0ull, 0ull, 0ull, 0ull};
  if (live) {
    const int64_t step = int64_t(gridDim.y) * 8;
    for (int64_t row0 = int64_t(blockIdx.y) * 8 + w; row0 < M; row0 += kRowsInFlight * step) {
      uint4 d4[kRowsInFlight], z4[kRowsInFlight];
#pragma unroll
      for (int k = 0; k < kRowsInFlight; ++k) {
        const int64_t row = row0 + k * step;
        d4[k] = z4[k] = make_uint4(0, 0, 0, 0);
        if (row < M) {
          const size_t i = size_t(row) * size_t(N) + size_t(col);
          d4[k] = ld16_once(dout + i);
          if (ACT != ACT_NONE) z4[k] = ld16_once(z + i);
        }
      }
#pragma unroll
      for (int k = 0; k < kRowsInFlight; ++k) {
        const int64_t row = row0 + k * step;
        if (row >= M) break;
        uint64_t d[4] = {bf16x2_to_f2(d4[k].x), bf16x2_to_f2(d4[k].y), bf16x2_to_f2(d4[k].z), bf16x2_to_f2(d4[k].w)};
        if (ACT != ACT_NONE) {
          const uint32_t zw[4] = {z4[k].x, z4[k].y, z4[k].z, z4[k].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint64_t f, df;
            act_grad_f2<ACT>(bf16x2_to_f2(zw[j]), f, df);
            d[j] = f2_mul(d[j], df);
          }
          stg16(dz + size_t(row) * size_t(N) + size_t(col), pack8(d));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = f2_add(s[j], d[j]);
      }
    }
  }
  if (dbias == nullptr) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) *reinterpret_cast<uint64_t*>(&comb[w][l * 8 + 2 * j]) = s[j];
  __syncthreads();
  const int64_t c = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (c < N) {
    float v = comb[0][threadIdx.x];
    for (int k = 1; k < 8; ++k) v += comb[k][threadIdx.x];
    if (gridDim.y > 1) partial[size_t(blockIdx.y) * size_t(N) + size_t(c)] = v;
    else dbias[c] = accumulate ? dbias[c] + v : v;
  }
}

// ------------------------------------------------------------------ host side
// An MMA operand: [rows, k] K-major or, `mn`, [k, rows] as it lies in memory.
template <int OP>
bool operand_map(CUtensorMap* map, const void* ptr, int64_t rows, int64_t k, bool mn, int box_rows = 128) {
  return mn ? make_operand_map(map, ptr, OP == OP_BF16, k, rows, 64)
            : make_operand_map(map, ptr, OP == OP_BF16, rows, k, box_rows);
}

// 2-CTA clusters of a form that fit on the device at once (cached per device).
template <int OP, int EPI, int ACT, bool A_MN, bool B_MN, bool SWAP = false>
cudaError_t max_pairs(int* pairs) {
  static int cached[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && cached[dev] > 0) {
    *pairs = cached[dev];
    return cudaSuccess;
  }
  const auto fn = linear_kernel<OP, EPI, ACT, A_MN, B_MN, SWAP>;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (num_sms() / 2));
  cfg.blockDim = dim3(NUM_THREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  e = cudaOccupancyMaxActiveClusters(&n, fn, &cfg);
  if (e != cudaSuccess) return e;
  if (n < 1) return cudaErrorInvalidConfiguration;
  if (dev >= 0 && dev < 64) cached[dev] = n;
  *pairs = n;
  return cudaSuccess;
}

struct Maps {
  CUtensorMap a, b, bh;
};

template <int OP, int EPI, int ACT, bool A_MN, bool B_MN, bool SWAP = false>
cudaError_t launch(const Maps& m, const LinArgs& a, int pairs, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * unsigned(a.num_units < pairs ? a.num_units : pairs));
  cfg.blockDim = dim3(NUM_THREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, linear_kernel<OP, EPI, ACT, A_MN, B_MN, SWAP>, m.a, m.b, m.bh, a);
}

// How a product [M, K] x [N, K]^T is cut: into units of 256 rows by 256 >> narrow
// columns, and the parts of K where even narrow units would leave SM pairs idle.
struct Plan {
  int tiles_m, tiles_n, tiles, num_kb, narrow, splits, kb_per_split;
  int64_t m_pad;
  int64_t cycles;            // estimate
};
constexpr int kPlanPairs = kNumSMsHint / 2;   // fixed, so a workspace size needs no device query
constexpr int kFixedCycles = 7800;            // of a call: launch, first loads, end
constexpr int64_t kNextKernelCycles = 6000;   // from a kernel's start to the next one's
constexpr int stage_cycles(int narrow) { return narrow == 0 ? 512 : narrow == 1 ? 308 : 288; }

// What a product leaves idle at its end: this many SM pairs for so many cycles.
struct Idle {
  int pairs;
  int64_t cycles;
};
// max_narrow: 2, or 1 where B is MN-major (its boxes are 64 columns wide).
Plan make_plan(int64_t M, int64_t N, int64_t K, int op, int max_narrow) {
  Plan p;
  p.tiles_m = int((M + 2 * BM - 1) / (2 * BM));
  p.num_kb = int((K + stage_k(op) - 1) / stage_k(op));
  p.m_pad = (M + 31) / 32 * 32;
  p.narrow = 0;
  p.splits = 1;
  const int64_t whole = int64_t(p.tiles_m) * ((N + BN - 1) / BN);
  const int64_t rest = whole % kPlanPairs;       // (a last round of up to half the pairs' number: half tiles)
  const int64_t last = rest == 0 ? 0 : whole > kPlanPairs && 2 * rest <= kPlanPairs ? 1 : 2;
  const int64_t half_rounds = 2 * (whole / kPlanPairs) + last;
  p.cycles = half_rounds * p.num_kb * 256 + kFixedCycles + 2560;
  if (2 * whole <= kPlanPairs) {
    // Less than half a round of whole tiles: the cheapest of narrower units and
    // parts of K, in SM cycles, fitted to measurements of 64 to 1000 rows: a stage
    // takes its MMAs' cycles or what the loads and the issue of the MMAs take,
    // the last unit's epilogue 2560 >> narrow, joining parts 5700 and for each 450
    // and one for 700 outputs.  (us, parts of K alone / this choice: 512 x 4096 x
    // 4096 21 / 15.6, 200 x 1024 x 4096 13.2 / 9.9, 256 x 1024 x 1024 9.5 / 5.7.)
    int64_t best = -1;
    for (int n = 0; n <= max_narrow; ++n) {
      const int64_t units = int64_t(p.tiles_m) * ((N + (BN >> n) - 1) / (BN >> n));
      const int stage = stage_cycles(n);
      for (int s = 1; s <= 16 && (s == 1 || (s * 8 <= p.num_kb && units * s <= kPlanPairs)); ++s) {
        const int64_t rounds = (units * s + kPlanPairs - 1) / kPlanPairs;
        const int64_t join = s == 1 ? 0 : 5700 + (450 + M * N / 700) * s;
        const int64_t cost = rounds * ((p.num_kb + s - 1) / s) * stage + kFixedCycles + (2560 >> n) + join;
        if (best < 0 || cost < best) {
          best = cost;
          p.narrow = n;
          p.splits = s;
        }
      }
    }
    p.cycles = best;
  }
  p.tiles_n = int((N + (BN >> p.narrow) - 1) / (BN >> p.narrow));
  p.tiles = p.tiles_m * p.tiles_n;
  p.kb_per_split = (p.num_kb + p.splits - 1) / p.splits;
  if (p.num_kb > 0) p.splits = (p.num_kb + p.kb_per_split - 1) / p.kb_per_split;
  return p;
}
// The same product with the operands exchanged: units of 256 output columns by
// bn rows, a multiple of 32, so that the rows divide evenly into tiles.  A stage
// takes 117 + 1.55 bn cycles, 288 at least (fitted, as above).  Taken where that
// estimate is the lower (us, without and with: 333 x 8192 x 2048 with GELU 18.3 /
// 16.3, 260 x 8192 x 4096 25.8 / 18.9, 700 x 4096 x 4096 23.4 / 19.9, 333 x 4096 x
// 14336 41.6 / 39.7).
struct SwapPlan {
  int tiles_m, tiles_n, bn;
  int64_t unit, cycles;
};
SwapPlan make_swap_plan(int64_t M, int64_t N, int64_t K, int op) {
  SwapPlan best{0, 0, 0, 0, -1};
  const int64_t num_kb = (K + stage_k(op) - 1) / stage_k(op);
  const int64_t first = (M + BN - 1) / BN;
  for (int64_t t = first; t < first + 4; ++t) {
    SwapPlan p;
    p.bn = int(((M + t - 1) / t + 31) / 32 * 32);
    p.tiles_m = int((M + p.bn - 1) / p.bn);
    p.tiles_n = int((N + 2 * BM - 1) / (2 * BM));
    const int64_t stage = 117 + 31 * p.bn / 20;
    p.unit = num_kb * (stage > 288 ? stage : 288);
    p.cycles = (int64_t(p.tiles_m) * p.tiles_n + kPlanPairs - 1) / kPlanPairs * p.unit + kFixedCycles + 12 * p.bn;
    if (best.cycles < 0 || p.cycles < best.cycles) best = p;
  }
  return best;
}
// Whether few_rows.cu takes a product (N: output columns, gated H): where its
// estimate is the lower.  No form beats the weights' way from HBM, about 2900
// bytes a cycle; where that bounds both, the exchanged form is the faster (64 rows
// of 28672 x 4096 40.2 us, few_rows.cu 41.6, this one unexchanged 44.3).
bool takes_few_rows(int64_t M, int64_t N, int64_t K, bool gated, bool fp8, bool b_mn) {
  const int op = fp8 ? OP_E4M3 : OP_BF16;
  const int64_t wrows = gated ? 2 * N : N;
  const int64_t few = few_rows_cycles(M, N, K, gated, fp8);
  if (few < 0) return false;
  const int64_t hbm = kFixedCycles + wrows * K * (fp8 ? 1 : 2) / 2900;
  const int64_t here = make_plan(M, wrows, K, op, b_mn ? 1 : 2).cycles;
  if (gated) return few < (here > hbm ? here : hbm + 1);
  const int64_t swapped = make_swap_plan(M, N, K, op).cycles;
  return few < here && few < swapped && swapped > hbm;
}
// (A workspace size must not depend on the device: it covers the plan whether or
// not few_rows.cu is taken.)
size_t plan_bytes(const Plan& p, int64_t N) {
  return p.splits > 1 ? size_t(p.splits) * size_t(p.m_pad) * size_t(N) * sizeof(float) : 0;
}

// N-blocks per raster band: about 32 MB of weights, so that a band stays in L2
// while the row groups cycle through it (measured for the FP8 gate|up GEMM,
// gemm_fp8.cu); one band where the activations are the larger operand.
int band_blocks(int tiles_n, int64_t M, int64_t N, int64_t k_bytes) {
  if (N <= M) return tiles_n;
  int64_t b = (int64_t(32) << 20) / (int64_t(BN) * (k_bytes > 0 ? k_bytes : 1));
  if (b < 1) b = 1;
  return b > tiles_n ? tiles_n : int(b);
}

template <int EPI, int ACT>
cudaError_t launch_join(uint16_t* out, uint16_t* out2, const float* partial, const uint16_t* bias, const uint16_t* in,
                        const float* a_scale, const float* w_scale, const Plan& p, int64_t ld, int64_t M, int64_t N,
                        cudaStream_t s) {
  const int64_t total = M * (N / 8);
  int64_t blocks = (total + 255) / 256;
  const int64_t cap = int64_t(num_sms()) * 8;
  if (blocks > cap) blocks = cap;
  return launch_pdl(join_kernel<EPI, ACT>, dim3(unsigned(blocks)), 256, 0, s, out, out2, partial, bias, in, a_scale,
                    w_scale, p.splits, p.m_pad, ld, M, N);
}

// One product in the exchanged form (B K-major or, `B_MN`, [K, N] as it lies).
template <int OP, int ACT, bool B_MN>
cudaError_t product_swapped(const SwapPlan& p, uint16_t* out, uint16_t* z, const void* A, const float* a_scale,
                            const void* B, const float* w_scale, const uint16_t* bias, const uint16_t* in, int64_t M,
                            int64_t N, int64_t K, cudaStream_t s, bool late_wait, Idle* after) {
  Maps m;
  if (!operand_map<OP>(&m.a, B, N, K, B_MN) || !operand_map<OP>(&m.b, A, M, K, false, p.bn / 2))
    return cudaErrorInvalidValue;
  m.bh = m.b;
  LinArgs a{};
  a.M = int(M);
  a.N = int(N);
  a.bn = p.bn;
  a.stages = RING_BYTES / (OP_BYTES + p.bn / 2 * ROW_BYTES);
  if (a.stages > MAX_STAGES) a.stages = MAX_STAGES;
  a.tiles_m = p.tiles_m;
  a.tiles_n = p.tiles_n;
  a.band_n = band_blocks(p.tiles_n, M, N, K * (OP == OP_BF16 ? 2 : 1));
  a.num_kb = int((K + stage_k(OP) - 1) / stage_k(OP));
  a.num_units = a.split_from = p.tiles_m * p.tiles_n;
  a.splits = 1;
  a.late_wait = late_wait ? 1 : 0;
  a.a_scale = a_scale;
  a.w_scale = w_scale;
  a.bias = bias;
  a.out = out;
  a.z = z;
  a.in = in;
  int pairs = 0;
  const cudaError_t e = max_pairs<OP, EPI_LINEAR, ACT, B_MN, false, true>(&pairs);
  if (e != cudaSuccess) return e;
  if (after != nullptr) {
    const int r = a.num_units % pairs;
    *after = a.num_units < pairs ? Idle{pairs - a.num_units, p.unit - kNextKernelCycles}
             : r == 0            ? Idle{0, 0}
                                 : Idle{pairs - r, p.unit};
  }
  return launch<OP, EPI_LINEAR, ACT, B_MN, false, true>(m, a, pairs, s);
}

// One product with its epilogue.  EPI_LINEAR: N output columns; gated forms:
// N = H and B = W1 [2H, K].  `partial` holds plan_bytes().  `before`: what the
// kernel launched last leaves idle, if this one may start beside it (late_wait);
// `after` receives what this one does.
template <int OP, int EPI, int ACT, bool A_MN, bool B_MN>
cudaError_t product(uint16_t* out, uint16_t* z, const void* A, const float* a_scale, const void* B,
                    const float* w_scale, const uint16_t* bias, const uint16_t* in, int64_t M, int64_t N, int64_t K,
                    float* partial, cudaStream_t s, bool late_wait = false, Idle before = {0, 0},
                    Idle* after = nullptr) {
  constexpr bool GATED = EPI == EPI_GATED || EPI == EPI_GATED_BWD;
  const int64_t brows = GATED ? 2 * N : N;
  const Plan p = make_plan(M, brows, K, OP, B_MN ? 1 : 2);
  if constexpr (EPI == EPI_LINEAR && !A_MN) {
    const SwapPlan sp = make_swap_plan(M, N, K, OP);
    if (sp.cycles < p.cycles)
      return product_swapped<OP, ACT, B_MN>(sp, out, z, A, a_scale, B, w_scale, bias, in, M, N, K, s, late_wait, after);
  }
  Maps m;
  if (!operand_map<OP>(&m.a, A, M, K, A_MN) || !operand_map<OP>(&m.b, B, brows, K, B_MN, 128 >> p.narrow))
    return cudaErrorInvalidValue;
  m.bh = m.b;
  LinArgs a{};
  a.M = int(M);
  a.tiles_m = p.tiles_m;
  a.num_kb = p.num_kb;
  a.up_row = int(N);
  a.narrow = p.narrow;
  a.late_wait = late_wait ? 1 : 0;
  a.splits = 1;
  int pairs = 0;
  cudaError_t e;
  if (p.splits > 1) {
    a.partial = partial;
    a.N = int(brows);
    a.tiles_n = p.tiles_n;
    a.band_n = p.tiles_n;
    a.splits = p.splits;
    a.kb_per_split = p.kb_per_split;
    a.m_pad = int(p.m_pad);
    a.num_units = a.split_from = p.tiles * p.splits;
    if ((e = max_pairs<OP, EPI_PARTIAL, ACT_NONE, A_MN, B_MN>(&pairs)) != cudaSuccess) return e;
    if ((e = launch<OP, EPI_PARTIAL, ACT_NONE, A_MN, B_MN>(m, a, pairs, s)) != cudaSuccess) return e;
    return launch_join<EPI, ACT>(out, z, partial, bias, in, a_scale, w_scale, p, brows, M, N, s);
  }
  a.N = int(N);
  a.a_scale = a_scale;
  a.w_scale = w_scale;
  a.bias = bias;
  a.out = out;
  a.z = z;
  a.in = in;
  a.tiles_n = GATED ? int((N + (128 >> p.narrow) - 1) / (128 >> p.narrow)) : p.tiles_n;
  a.band_n = band_blocks(a.tiles_n, M, brows, K * (OP == OP_BF16 ? 2 : 1));
  a.num_units = a.split_from = a.tiles_m * a.tiles_n;
  if ((e = max_pairs<OP, EPI, ACT, A_MN, B_MN>(&pairs)) != cudaSuccess) return e;
  // a last partial wave of R <= pairs / 2 tiles runs as 2 R half tiles in half the time
  // (a unit's epilogue, beside the next one's products, takes some 4000 cycles)
  int64_t unit = int64_t(p.num_kb) * stage_cycles(p.narrow);
  if (unit < 4000 >> p.narrow) unit = 4000 >> p.narrow;
  auto last_wave = [&](int units) { return units > pairs ? units % pairs : 0; };
  auto halves = [&](int r) { return p.narrow == 0 && r > 0 && 2 * r <= pairs; };
  if (before.pairs > 0 && before.pairs < pairs && a.num_units > pairs) {
    // The first before.pairs pairs start early (clusters start in the order of
    // their numbers) and take `extra` units more than the others: as many as end
    // while the rest of the SMs is still busy, and with the fewest rounds of
    // units.  (Input and weight gradient, us, without and with: M = 4096, N = 8192,
    // K = 2048 165 / 152, 700, 5000, 2056 46 / 40.5, 1111, 4104, 2056 50 / 43.7.)
    const int64_t fit = before.cycles / unit;
    int64_t best = -1;
    for (int extra = 0; extra <= fit && a.num_units - extra * before.pairs > pairs; ++extra) {
      const int rest = a.num_units - extra * before.pairs;
      const int r = last_wave(rest);
      const int64_t half_rounds = 2 * (rest / pairs) + (r == 0 ? 0 : halves(r) ? 1 : 2);
      if (best < 0 || half_rounds < best) {
        best = half_rounds;
        a.early = before.pairs;
        a.early_units = extra * before.pairs;
      }
    }
    if (a.early_units == 0) a.early = 0;
  }
  const int r = last_wave(a.num_units - a.early_units);
  if (after != nullptr)
    // (a kernel of one round leaves them from its start, but the next is launched later)
    *after = a.num_units < pairs ? Idle{pairs - a.num_units, unit - kNextKernelCycles}
             : r == 0            ? Idle{0, 0}
             : halves(r)         ? Idle{pairs - 2 * r, unit / 2}
                                 : Idle{pairs - r, unit};
  if (halves(r)) {
    if (!B_MN && !operand_map<OP>(&m.bh, B, brows, K, false, 64)) return cudaErrorInvalidValue;
    a.split_from = a.num_units - r;
    a.num_units += r;
  }
  return launch<OP, EPI, ACT, A_MN, B_MN>(m, a, pairs, s);
}

int act_backward_blocks(int64_t M, int64_t N) {
  if (M <= 64) return 1;
  const int64_t cols = (N + 255) / 256;
  int64_t rows = (int64_t(kNumSMsHint) * 8 + cols - 1) / cols;   // about eight blocks per SM
  const int64_t need = (M + 7) / 8;
  if (rows > need) rows = need;
  return int(rows < 1 ? 1 : (rows > 65535 ? 65535 : rows));
}

size_t round256(size_t v) { return (v + 255) / 256 * 256; }

// linear backward workspace: dz [M,N] bf16 | column partials | parts of K of dx | of dw
void linear_bwd_offsets(int64_t M, int64_t N, int64_t K, size_t off[5]) {
  off[0] = 0;
  off[1] = round256(size_t(M) * size_t(N) * 2);
  off[2] = off[1] + round256(size_t(act_backward_blocks(M, N)) * size_t(N) * sizeof(float));
  off[3] = off[2] + round256(plan_bytes(make_plan(M, K, N, OP_BF16, 1), K));
  off[4] = off[3] + round256(plan_bytes(make_plan(N, K, M, OP_BF16, 1), K));
}

// gated backward workspace: d_gu [M,2H] bf16 | parts of K of the recomputation or of dx | of dw1
void gated_bwd_offsets(int64_t M, int64_t C, int64_t H, size_t off[4]) {
  off[0] = 0;
  off[1] = round256(size_t(M) * size_t(2 * H) * 2);
  const size_t a = plan_bytes(make_plan(M, 2 * H, C, OP_BF16, 2), 2 * H);
  const size_t b = plan_bytes(make_plan(M, C, 2 * H, OP_BF16, 1), C);
  off[2] = off[1] + round256(a > b ? a : b);
  off[3] = off[2] + round256(plan_bytes(make_plan(2 * H, C, M, OP_BF16, 1), C));
}

}  // namespace

size_t linear_workspace(int64_t M, int64_t N, int64_t K, bool fp8) {
  return skinny_rows(M, N, K, fp8) ? 0 : plan_bytes(make_plan(M, N, K, fp8 ? OP_E4M3 : OP_BF16, 2), N);
}
size_t gated_workspace(int64_t M, int64_t C, int64_t H) {
  return skinny_rows(M, 2 * H, C, false) ? 0 : plan_bytes(make_plan(M, 2 * H, C, OP_BF16, 2), 2 * H);
}
size_t linear_backward_workspace(int64_t M, int64_t N, int64_t K) {
  size_t off[5];
  linear_bwd_offsets(M, N, K, off);
  return off[4];
}
size_t gated_backward_workspace(int64_t M, int64_t C, int64_t H) {
  size_t off[4];
  gated_bwd_offsets(M, C, H, off);
  return off[3];
}

#define QFFN_ACT_SWITCH(act, EXPR)                                 \
  switch (act) {                                                   \
    case ACT_RELU: { constexpr int ACT = ACT_RELU; return EXPR; }  \
    case ACT_GELU: { constexpr int ACT = ACT_GELU; return EXPR; }  \
    case ACT_GELU_TANH: { constexpr int ACT = ACT_GELU_TANH; return EXPR; } \
    case ACT_SILU: { constexpr int ACT = ACT_SILU; return EXPR; }  \
    default: { constexpr int ACT = ACT_NONE; return EXPR; }        \
  }

cudaError_t launch_linear(uint16_t* out, uint16_t* z, const uint16_t* x, const uint16_t* w, const uint16_t* bias,
                          const uint16_t* res, int act, int64_t M, int64_t N, int64_t K, float* ws, cudaStream_t s) {
  if (M == 0) return cudaSuccess;
  if (skinny_rows(M, N, K, false)) return launch_skinny(out, z, x, nullptr, w, nullptr, bias, res, act, M, N, K, false, s);
  if (takes_few_rows(M, N, K, false, false, false))
    return launch_few_rows(out, z, x, nullptr, w, nullptr, bias, res, act, M, N, K, false, false, s);
  QFFN_ACT_SWITCH(act, (product<OP_BF16, EPI_LINEAR, ACT, false, false>(out, z, x, nullptr, w, nullptr, bias, res, M, N,
                                                                        K, ws, s)));
}

cudaError_t launch_linear_fp8(uint16_t* out, uint16_t* z, const uint8_t* x, const float* x_scale, const uint8_t* w,
                              const float* w_scale, const uint16_t* bias, const uint16_t* res, int act, int64_t M,
                              int64_t N, int64_t K, float* ws, cudaStream_t s) {
  if (M == 0) return cudaSuccess;
  if (skinny_rows(M, N, K, true)) return launch_skinny(out, z, x, x_scale, w, w_scale, bias, res, act, M, N, K, true, s);
  if (takes_few_rows(M, N, K, false, true, false))
    return launch_few_rows(out, z, x, x_scale, w, w_scale, bias, res, act, M, N, K, true, false, s);
  QFFN_ACT_SWITCH(act, (product<OP_E4M3, EPI_LINEAR, ACT, false, false>(out, z, x, x_scale, w, w_scale, bias, res, M, N,
                                                                        K, ws, s)));
}

cudaError_t launch_gated(uint16_t* h, const uint16_t* x, const uint16_t* w1, int act, int64_t M, int64_t C, int64_t H,
                         float* ws, cudaStream_t s) {
  if (M == 0) return cudaSuccess;
  if (skinny_rows(M, 2 * H, C, false)) return launch_skinny_gated(h, x, w1, act, M, C, H, s);
  if (takes_few_rows(M, H, C, true, false, false)) return launch_few_rows_gated(h, x, w1, nullptr, act, M, C, H, s);
  QFFN_ACT_SWITCH(act, (product<OP_BF16, EPI_GATED, ACT, false, false>(h, nullptr, x, nullptr, w1, nullptr, nullptr,
                                                                       nullptr, M, H, C, ws, s)));
}

namespace {
template <int ACT>
cudaError_t run_act_backward(uint16_t* dz, float* partial, float* dbias, const uint16_t* dout, const uint16_t* z,
                             int64_t M, int64_t N, bool accumulate, cudaStream_t s) {
  const dim3 grid(unsigned((N + 255) / 256), unsigned(act_backward_blocks(M, N)));
  return launch_pdl(act_backward_kernel<ACT>, grid, 256, 0, s, dz, partial, dbias, dout, z, M, N, accumulate ? 1 : 0);
}
cudaError_t act_backward(uint16_t* dz, float* partial, float* dbias, const uint16_t* dout, const uint16_t* z, int act,
                         int64_t M, int64_t N, bool accumulate, cudaStream_t s) {
  QFFN_ACT_SWITCH(act, (run_act_backward<ACT>(dz, partial, dbias, dout, z, M, N, accumulate, s)));
}
cudaError_t gated_bwd_product(uint16_t* dgu, const uint16_t* dh, const uint16_t* x, const uint16_t* w1, int act,
                              int64_t M, int64_t C, int64_t H, float* part, cudaStream_t s) {
  if (takes_few_rows(M, H, C, true, false, false)) return launch_few_rows_gated(dgu, x, w1, dh, act, M, C, H, s);
  QFFN_ACT_SWITCH(act, (product<OP_BF16, EPI_GATED_BWD, ACT, false, false>(dgu, nullptr, x, nullptr, w1, nullptr,
                                                                           nullptr, dh, M, H, C, part, s)));
}
// dx [M,K] = dz [M,N] . W [N,K];  dw [N,K] (+)= dz^T . x [M,K]: W, dz and x read
// where they lie.  `ready`: dz was complete before the kernel launched last may
// have started, so dx need not wait for that one either; dw never reads what
// the kernel before it writes and starts on the SMs that dx leaves free
// (512 x 1024 x 1024, both: 18 us, one after the other 19.9).
cudaError_t grad_products(uint16_t* dx, uint16_t* dw, const uint16_t* dz, const uint16_t* x, const uint16_t* w,
                          int64_t M, int64_t N, int64_t K, bool accumulate, float* part_dx, float* part_dw, bool ready,
                          cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  Idle idle{0, 0};
  if (dx != nullptr) {
    e = takes_few_rows(M, K, N, false, false, true)
            ? launch_few_rows(dx, nullptr, dz, nullptr, w, nullptr, nullptr, nullptr, ACT_NONE, M, K, N, false, true, s,
                              ready)
            : product<OP_BF16, EPI_LINEAR, ACT_NONE, false, true>(dx, nullptr, dz, nullptr, w, nullptr, nullptr,
                                                                  nullptr, M, K, N, part_dx, s, ready, Idle{0, 0}, &idle);
    if (e != cudaSuccess) return e;
    ready = true;
  }
  return product<OP_BF16, EPI_LINEAR, ACT_NONE, true, true>(dw, nullptr, dz, nullptr, x, nullptr, nullptr,
                                                            accumulate ? dw : nullptr, N, K, M, part_dw, s, ready,
                                                            idle);
}
}  // namespace

cudaError_t launch_linear_backward(uint16_t* dx, uint16_t* dw, float* dbias, const uint16_t* dout, const uint16_t* z,
                                   const uint16_t* x, const uint16_t* w, int act, int64_t M, int64_t N, int64_t K,
                                   bool accumulate, uint8_t* ws, cudaStream_t s) {
  cudaError_t e;
  if (M == 0) {
    // sums over no rows: zero, or unchanged when accumulating
    if (accumulate) return cudaSuccess;
    if ((e = cudaMemsetAsync(dw, 0, size_t(N) * size_t(K) * 2, s)) != cudaSuccess) return e;
    return dbias != nullptr ? cudaMemsetAsync(dbias, 0, size_t(N) * sizeof(float), s) : cudaSuccess;
  }
  size_t off[5];
  linear_bwd_offsets(M, N, K, off);
  uint16_t* dzb = reinterpret_cast<uint16_t*>(ws + off[0]);
  float* cols = reinterpret_cast<float*>(ws + off[1]);
  float* part_dx = reinterpret_cast<float*>(ws + off[2]);
  float* part_dw = reinterpret_cast<float*>(ws + off[3]);
  const uint16_t* dz = act == ACT_NONE ? dout : dzb;
  bool ready = false;        // the kernel launched last neither writes dz nor precedes its completion
  if (act != ACT_NONE || dbias != nullptr) {
    if ((e = act_backward(dzb, cols, dbias, dout, z, act, M, N, accumulate, s)) != cudaSuccess) return e;
    if (dbias != nullptr && act_backward_blocks(M, N) > 1) {
      if ((e = launch_column_sum(dbias, nullptr, cols, act_backward_blocks(M, N), N, N, accumulate, s)) != cudaSuccess)
        return e;
      ready = true;
    }
  }
  return grad_products(dx, dw, dz, x, w, M, N, K, accumulate, part_dx, part_dw, ready, s);
}

cudaError_t launch_gated_backward(uint16_t* dx, uint16_t* dw1, const uint16_t* dh, const uint16_t* x,
                                  const uint16_t* w1, int act, int64_t M, int64_t C, int64_t H, bool accumulate,
                                  uint8_t* ws, cudaStream_t s) {
  if (M == 0) return accumulate ? cudaSuccess : cudaMemsetAsync(dw1, 0, size_t(2 * H) * size_t(C) * 2, s);
  size_t off[4];
  gated_bwd_offsets(M, C, H, off);
  uint16_t* dgu = reinterpret_cast<uint16_t*>(ws + off[0]);
  float* part = reinterpret_cast<float*>(ws + off[1]);
  const cudaError_t e = gated_bwd_product(dgu, dh, x, w1, act, M, C, H, part, s);
  if (e != cudaSuccess) return e;
  return grad_products(dx, dw1, dgu, x, w1, M, 2 * H, C, accumulate, part, reinterpret_cast<float*>(ws + off[2]), false,
                       s);
}

cudaError_t linear_take_status(unsigned int* status) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_status, sizeof(v));
  if (e != cudaSuccess) return e;
  if (v != 0) e = cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
  *status = v;
  return e;
}

}  // namespace qffn
