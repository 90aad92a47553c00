// Products grouped by expert and block-scaled products on the 5th-generation tensor
// cores (tcgen05, sm_103a), groups of rows with a matrix each:
//
//   KIND_FORWARD   out[m,n]  = bf16(sum_k x[m,k] w_g[n,k] (+ bias[n]) (+ in[m,n])),  m in group g;
//                  bf16, or E4M3 with a power-of-two scale per block of 128
//   KIND_BACKWARD  dx[m,k]   = bf16(sum_n dout[m,n] w_g[n,k])  and
//                  dw_g[n,k] = bf16(sum_{m in g} dout[m,n] x[m,k] (+ dw_g[n,k])), in one
//                  launch; w, dout and x are read where they lie
//
// The pipeline is that of linear.cu: SM pairs, persistent over units of work, one
// warp loads by TMA into a ring of stages (128 bytes of K each), one thread issues
// tcgen05.mma.cta_group::2, eight warps per CTA run the epilogue out of one of two
// accumulators while the other fills.  What is new:
//
// - The sizes of the groups are on the device.  Every CTA reads the offsets once
//   into a table of units in shared memory; the roles look their units up there.  The
//   widest unit is chosen there too, so that the units fill the pairs' rounds.
// - The units of the weight gradients follow those of dx in one launch, the longest
//   groups' first: one tail at the end, of the smallest units, instead of two (16384 rows
//   unevenly in eight groups of 4096 x 2048 371 -> 360 us, 800 in 16 of 2048 x 1032, added,
//   94 -> 86).
// - The weights are the 256-row operand and the rows of x the other (as in linear.cu's
//   exchanged form), so that the width of a unit, 32 to 256 rows of x, follows the
//   group: its rows are spread evenly over its tiles, and a group of a few rows costs
//   its weights' bytes and no more.  The rows of x come in boxes of 128, 64, 32 and 16
//   rows.
// - The weight gradient's contraction runs over a group's rows, which end anywhere. The
//   last stage of a unit may hold rows of the next group: only the MMAs (of 16 rows) that
//   the group reaches are issued, and a warp overwrites the rows behind it in the last of
//   them with zeros in shared memory, in both operands, so that neither finite values nor
//   NaN of a neighbour meet a group.
// - E4M3: tcgen05.mma.kind::mxf8f6f4.block_scale takes E8M0 scales for every 32
//   values of K from TMEM; a scale per 128 is the same byte in four MMAs.  Four warps
//   read the scales of 512 of K at a time (one byte per row of x and block, one per
//   128 weight rows and block), lay them out in shared memory, and the issuing thread
//   copies them to TMEM (tcgen05.cp) in front of the MMAs that use them.  The tensor
//   cores then scale for nothing; sums never leave TMEM.
//
// Every mbarrier wait is bounded; see gemm_fp8.cu for how a wait that runs out
// ends the kernel (abort flag, status word, drained copies and MMAs).
#include <cuda.h>

#include "common.cuh"
#include "launch.h"
#include "pipeline.cuh"
#include "tensor_map.h"
#include "umma.cuh"

namespace qffn {
namespace {

constexpr int OP_BF16 = 0, OP_BLOCKS = 1;
constexpr int KIND_FORWARD = 0, KIND_BACKWARD = 1;

constexpr int BM = 128;                    // weight rows per CTA (256 per pair)
constexpr int ROW_BYTES = 128;             // one swizzle atom row
constexpr int OP_BYTES = 128 * ROW_BYTES;  // an operand's share of a stage: 128 rows of one swizzle row
constexpr int MN_BOX_BYTES = 64 * ROW_BYTES;   // MN-major: 64 values by 64 of K, two boxes to the share
constexpr int STEPS = 4;                   // MMAs per stage (32 bytes of K each)
// (Sixteen warps in the backward's epilogue, us against eight: 1 row in each of 64 groups of
// 2048 x 1024 55 / 60, 1000 in each of eight of 4096 x 2048 179 / 166.)
constexpr int EPI_WARPS = 8;
constexpr int SCALE_WARPS = 4;
constexpr int MAX_STAGES = 10;
constexpr int SF_STAGES = SCALE_WARPS;     // stages of scales, 512 of K each, one for each warp that fills them
constexpr int SF_BYTES = 3 * 512;          // 128 weight rows, 256 rows of x: 4 bytes each
constexpr int NUM_BARS = 4 * MAX_STAGES + 6 + 2 * SF_STAGES;
constexpr int UNIT_SLOTS = 16;             // more than the units whose stages are in flight
constexpr int INFO_INTS = 2 * UNIT_SLOTS + 12;
constexpr int SMEM_LIMIT = 227 * 1024 - 1024;  // (behind the alignment to 1024 bytes)
constexpr int TMEM_COLS = 512;
constexpr int GROUP_M = 8;
constexpr uint16_t kBothCtas = 0x3;
constexpr uint16_t kLeaderOnly = 0x1;
constexpr unsigned long long kWaitLimitNs = 2000000000ull;
constexpr unsigned long long kDrainLimitNs = 200000000ull;

constexpr int stage_k(int op) { return op == OP_BF16 ? 64 : 128; }   // elements of K per stage
constexpr int MAX_BN = 256;                // columns of an accumulator
// a warp's transposing box: 32 rows x 32 bf16, backward 32 x 64
constexpr int staging_box(int kind) { return 32 * (kind == KIND_BACKWARD ? 128 : 64); }
constexpr int num_threads(int op, int kind) {
  return 32 * (2 + EPI_WARPS + (op == OP_BLOCKS ? SCALE_WARPS : kind == KIND_BACKWARD ? 1 : 0));
}
constexpr int fixed_bytes(int op, int kind) {
  return EPI_WARPS * staging_box(kind) + (op == OP_BLOCKS ? SF_STAGES * SF_BYTES : 0) + NUM_BARS * 8 + 16 + INFO_INTS * 4;
}
// First column of the scales: two slots of 16.  Below them are two accumulators, 224 columns
// apart, or 192 where units are wider than 224: those share 64 columns, and a unit starts
// when the epilogue has read these, which it does first.  (Units of 224 rows at most
// against 256: 8192 rows in eight groups of 28672 x 4096 692 us / 677, 8192 rows of
// 4096 x 2048 45.3 / 44.1, of 4096 x 512 20.0 / 20.7.)
constexpr int SF_TMEM = 448;

// Instruction descriptors.  kind::f16: D fp32 (bits 4-5 = 1), A and B bf16 (bits 7-9,
// 10-12 = 1); kind::mxf8f6f4: bits 4-5 / 29-30 which byte of the scales' words B / A
// takes, A and B E4M3 (0), scales E8M0 (bit 23).  Both: bits 15 / 16 A / B MN-major,
// N >> 3 at bits 17-22, M >> 4 at bits 24-28 (M = 256 over the pair).
QFFN_DEVI uint32_t idesc_for(int op, bool a_mn, bool b_mn, int n) {
  return (op == OP_BF16 ? (1u << 4) | (1u << 7) | (1u << 10) : 1u << 23) | (a_mn ? 1u << 15 : 0u) |
         (b_mn ? 1u << 16 : 0u) | (uint32_t(n >> 3) << 17) | (uint32_t((2 * BM) >> 4) << 24);
}

__device__ unsigned int g_status;

struct GroupArgs {
  uint16_t* out;            // [M, N]; backward: dx (NULL: none)
  uint16_t* dw;             // backward: [G, rows, N]
  const uint16_t* bias;     // forward, optional
  const uint16_t* in;       // what is added: [M, N], backward the previous dw; optional
  const uint8_t* x_scale;   // E4M3: [M, blocks] and [G, n_blocks, blocks]
  const uint8_t* w_scale;
  int blocks, n_blocks;
  const int* offsets;       // NULL: one group of all rows
  int G, M, N;
  int rows;                 // backward: rows of a matrix
  int tiles_n;              // units of 256 across a row of N
  int tiles_r;              // backward: units of 256 across a matrix's rows
  int bn_cap;               // most rows of a unit, a multiple of 32
  int late_wait;            // does not read the preceding kernel's results (see launch.h)
  int band_n;               // units across N that are swept together
  int num_kb;               // stages of K of out
  int stages, stage_bytes;  // stage_bytes: with room for bn_cap / 2 rows of x
};

// D(tmem, both CTAs) (+)= A(smem, both CTAs) . B(smem, both CTAs)^T
QFFN_DEVI void mma_pair_f16(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// The same with E4M3 operands and the scales at TMEM columns sfa and sfb.
QFFN_DEVI void mma_pair_blocks(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                               uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}
// 32 rows of 16 bytes of each CTA's shared memory to four columns of its TMEM, for
// all four lane quarters: the scales of 128 rows, row r in lane r % 32 and word r / 32.
QFFN_DEVI void copy_scales(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}
// Shared-memory descriptor of MMA step i of a stage's operand (see linear.cu).
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

// Hands this CTA's shared memory over to the thread of the leader that waits on the leader's `bar`
// (the writes are ordered before it by fence_proxy_async_smem() and __syncwarp()).
QFFN_DEVI void hand_over(uint32_t bar, uint32_t rank) {
  if (rank == 0) mbar_arrive(bar);
  else mbar_arrive_remote(map_to_rank(bar, 0));
}

QFFN_DEVI void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Sixteen lanes by 32 columns of TMEM at each of two addresses, without waiting
// (tmem_wait_ld16 makes them usable): registers 4 c .. 4 c + 3 of a thread hold columns
// 8 c + 2 (lane % 4) and the next, of lane lane / 4 and of lane lane / 4 + 8.
QFFN_DEVI void tmem_ld_blocks_issue(uint32_t ta, uint32_t tb, uint32_t (&a)[16], uint32_t (&b)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n"
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]), "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15]), "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3]), "=r"(b[4]), "=r"(b[5]), "=r"(b[6]), "=r"(b[7]), "=r"(b[8]), "=r"(b[9]), "=r"(b[10]), "=r"(b[11]), "=r"(b[12]), "=r"(b[13]), "=r"(b[14]), "=r"(b[15])
      : "r"(ta), "r"(tb)
      : "memory");
}
// Four 8 x 8 blocks of 16-bit values between shared memory and the threads' fragments,
// transposed; lane l gives the address of row l % 8 of block l / 8.
QFFN_DEVI void stmatrix_trans(uint32_t addr, const uint32_t (&p)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(p[0]), "r"(p[1]),
               "r"(p[2]), "r"(p[3])
               : "memory");
}
QFFN_DEVI void ldmatrix_trans(uint32_t addr, uint32_t (&p)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3])
               : "r"(addr)
               : "memory");
}

QFFN_DEVI uint32_t pack2(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return pack_bf16x2(lo, hi);
}
QFFN_DEVI uint4 pack8(const uint64_t (&v)[4]) { return make_uint4(pack2(v[0]), pack2(v[1]), pack2(v[2]), pack2(v[3])); }

// The table of units in shared memory: off[0 .. G] the offsets (within 0 .. M, none below
// the one before it), first[0 .. G] the number of the first unit of out of each group,
// shape[0 .. G - 1] how its rows are cut; backward: order[0 .. G - 1] the groups, those with
// rows first.
struct Table {
  const int* off;
  const int* first;
  const int* shape;
  const int* order;
  int G;
  int cap;            // most rows of a unit
};
struct Unit {
  int group;
  int begin, rows;    // the group's rows
  int row0, bn;       // of out: first row of the unit, its width
  int nb, kb;         // 256-wide unit of the row of N (of dw: of the matrix's rows, and of the row)
};

QFFN_DEVI int group_rows(const int* off, int g) { return off[g + 1] - off[g]; }

// n / d for n >= 0, d > 0: by the reciprocal where floats hold both, which an integer
// division takes five times as long for.
QFFN_DEVI int quick_div(int n, int d) {
  if (n >= 1 << 22) return n / d;
  int q = int(__fdividef(float(n), float(d)));
  const int r = n - q * d;
  q += r >= d ? 1 : r < 0 ? -1 : 0;
  return q;
}

// A group's rows in 32s, spread evenly over tiles of `cap` 32s at most: the tiles (4 bits up)
// and the 32s of the narrowest.
QFFN_DEVI int shape_of(int rows, int cap) {
  const int parts = (rows + 31) >> 5, tiles = quick_div(parts + cap - 1, cap);
  return tiles << 4 | (tiles > 0 ? quick_div(parts, tiles) : 0);
}

// The group of the last unit that a thread looked up: its first unit and the next group's, its
// rows in 32s spread over tm tiles, `wider` of `least` + 1 and the others of `least`.
struct Cursor {
  int group = -1, first = 0, next = 0, begin, rows, tm, least, wider;
};
// Unit u of out.  (Every role looks up every unit: with divisions in the open 900 cycles, in
// which the issuing thread left the tensor cores without work.)
QFFN_DEVI Unit rows_unit(int u, Cursor& c, const Table& t, const GroupArgs& a) {
  if (u >= c.next) {
    int lo = c.group + 1, hi = t.G - 1;      // the last group whose first unit is u or before
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (t.first[mid] <= u) lo = mid;
      else hi = mid - 1;
    }
    c.group = lo;
    c.first = t.first[lo];
    c.next = t.first[lo + 1];
    c.begin = t.off[lo];
    c.rows = group_rows(t.off, lo);
    const int shape = t.shape[lo];
    c.tm = shape >> 4;
    c.least = shape & 15;
    c.wider = ((c.rows + 31) >> 5) - c.least * c.tm;
  }
  Unit r;
  r.group = c.group;
  r.begin = c.begin;
  r.rows = c.rows;
  // bands of band_n; within a band, groups of GROUP_M tiles of rows sweep its columns, odd
  // groups backwards (see linear.cu)
  int k = u - c.first, mt = 0;
  r.nb = k;
  if (c.tm > 1) {
    int n0 = 0, wb = a.tiles_n, sweep = 0;
    if (a.band_n < a.tiles_n) {
      const int band = quick_div(k, c.tm * a.band_n);
      n0 = band * a.band_n;
      wb = min(a.band_n, a.tiles_n - n0);
      k -= n0 * c.tm;
    }
    if (c.tm > GROUP_M) {
      sweep = quick_div(k, GROUP_M * wb);
      k -= sweep * GROUP_M * wb;
    }
    const int size = min(c.tm - sweep * GROUP_M, GROUP_M);
    const int col = size == GROUP_M ? k / GROUP_M : quick_div(k, size);
    mt = sweep * GROUP_M + k - col * size;
    r.nb = n0 + ((sweep & 1) ? wb - 1 - col : col);
  }
  r.bn = 32 * (c.least + (mt < c.wider ? 1 : 0));
  r.row0 = r.begin + 32 * (mt * c.least + min(mt, c.wider));
  r.kb = 0;
  return r;
}
// Unit u of the weight gradients of the groups with rows.
QFFN_DEVI Unit weight_unit(int u, const Table& t, const GroupArgs& a) {
  const int per_group = a.tiles_r * a.tiles_n;
  Unit r;
  const int at = quick_div(u, per_group);
  r.group = t.order[at];
  r.begin = t.off[r.group];
  r.rows = group_rows(t.off, r.group);
  const int k = u - at * per_group;
  r.nb = quick_div(k, a.tiles_n);
  r.kb = k - r.nb * a.tiles_n;
  r.row0 = 0;
  r.bn = a.N - r.kb * 256 <= 128 ? 128 : 256;
  return r;
}

// Whether a stage of dw whose group has `left` more rows holds rows behind it in an MMA's 16.
QFFN_DEVI bool rows_to_clear(int left) { return left < 64 && (left & 15) != 0; }

template <bool B>
struct Flag {
  static constexpr bool value = B;
};

struct Maps {
  CUtensorMap w;        // the weights [G, rows, cols]
  CUtensorMap x[4];     // rows of x (backward: of dout) in boxes of 128, 64, 32, 16
  CUtensorMap dout_mn, x_mn;   // backward: boxes of 64 rows by 64 values
  CUtensorMap dw;              // [G, rows, cols] in boxes of 32 rows by 64 values
};

template <int OP, int KIND>
__global__ void __launch_bounds__(num_threads(OP, KIND), 1)
    grouped_kernel(const __grid_constant__ Maps maps, const GroupArgs args) {
  constexpr bool BACKWARD = KIND == KIND_BACKWARD;
  const uint32_t stage = uint32_t(args.stage_bytes);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t ring = smem_u32(smem);
  uint8_t* sStaging = smem + args.stages * args.stage_bytes;
  uint8_t* sScales = sStaging + EPI_WARPS * staging_box(KIND);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sScales + (OP == OP_BLOCKS ? SF_STAGES * SF_BYTES : 0));
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NUM_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* units_bn = reinterpret_cast<int*>(tmem_slot + 4);   // of the units in flight: width (of dw: negative), rows
  int* units_rows = units_bn + UNIT_SLOTS;
  int* one = units_rows + UNIT_SLOTS;                  // the table of one group of all rows: off, first, order, shape
  int* chosen = one + 6;                               // the cap, groups with rows, and see `spare`
  int* table_off = one + 12;
  int* table_first = table_off + args.G + 1;
  int* table_shape = table_first + args.G + 1;
  int* table_order = table_shape + args.G;             // backward
  int* found = table_order + (BACKWARD ? args.G : 0);  // a number per epilogue warp
  const uint32_t bar0 = smem_u32(bars);
  // full[s] (leader): both CTAs' loads of stage s landed; empty[s]: the MMAs
  // reading stage s are done; tfull[a]: accumulator a is complete; tempty[a]
  // (leader): both CTAs' epilogue warps have read it; drain: all MMAs done;
  // sfull[s] (leader): both CTAs' scales of stage s are written; sempty[s]: copied;
  // backward, a stage of dw with rows behind its group: tail[s]: this CTA's loads landed,
  // cleared[s] (leader): both CTAs have cleared those rows; table: this CTA's table is there
  auto full_bar = [&](int s) { return bar0 + 8u * uint32_t(s); };
  auto empty_bar = [&](int s) { return bar0 + 8u * uint32_t(MAX_STAGES + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * uint32_t(2 * MAX_STAGES + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * uint32_t(2 * MAX_STAGES + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * uint32_t(2 * MAX_STAGES + 4);
  auto sfull_bar = [&](int s) { return bar0 + 8u * uint32_t(2 * MAX_STAGES + 5 + s); };
  auto tail_bar = [&](int s) { return bar0 + 8u * uint32_t(2 * MAX_STAGES + 5 + 2 * SF_STAGES + s); };
  auto cleared_bar = [&](int s) { return bar0 + 8u * uint32_t(3 * MAX_STAGES + 5 + 2 * SF_STAGES + s); };
  const uint32_t table_bar = bar0 + 8u * uint32_t(4 * MAX_STAGES + 5 + 2 * SF_STAGES);
  auto sempty_bar = [&](int s) { return bar0 + 8u * uint32_t(2 * MAX_STAGES + 5 + SF_STAGES + s); };

  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = int(cluster_id_x()), num_pairs = int(num_clusters_x());

  if (threadIdx.x == 0) {
    for (int s = 0; s < args.stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 2 * EPI_WARPS);
    }
    mbar_init(drain_bar, 1);
    mbar_init(table_bar, 1);
    if (OP == OP_BLOCKS)
      for (int s = 0; s < SF_STAGES; ++s) {
        mbar_init(sfull_bar(s), 2);
        mbar_init(sempty_bar(s), 1);
      }
    if (BACKWARD)
      for (int s = 0; s < args.stages; ++s) {
        mbar_init(tail_bar(s), 1);
        mbar_init(cleared_bar(s), 2);
      }
    *abort_flag = 0;
    one[0] = one[2] = one[4] = 0;
    one[1] = args.M;
    one[5] = shape_of(args.M, args.bn_cap >> 5);
    one[3] = (one[5] >> 4) * args.tiles_n;
    mbar_init_fence();
  }
  if (warp == 0 && lane >= 8 && lane < (BACKWARD ? 16 : 13)) tma_prefetch_desc(&maps.w + (lane - 8));
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
  // The table.  Without offsets it is that of one group, and every role looks up its first unit
  // ahead of the wait for the preceding kernel.  With them the epilogue's warps make it behind
  // that wait; the other roles have meanwhile looked up a unit of one group (pass 0): the first
  // instructions of a kernel come from L2, and a first lookup takes 2000 cycles where the next
  // takes 350 (4531 x 2048 x 1536 without offsets 17.2 us, so 15.6).  Nothing in global memory
  // is touched before the preceding kernel is done.
  const bool grouped = args.offsets != nullptr;
  Table table{one, one + 2, one + 5, one + 4, 1, args.bn_cap};
  int rows_units = BACKWARD && args.out == nullptr ? 0 : one[3];   // units of out, then those of dw
  int num_units = rows_units;
  // backward: groups with rows; this pair's units of out; the `spare` pairs behind the last unit of
  // out, which have one less of those, take `early` units of dw meanwhile, and the rest of dw goes
  // round from them on (by turns regardless: 3 rows in five groups of 3080 x 1672 29.8 us, so 26.1; 4459
  // in seven of 4864 x 320 44.0, so 37.0)
  int busy = 0, of_out = 0, spare = num_pairs, turn = pair, early = 0, early_all = 0;
  Cursor cursor;
  if (grouped && warp >= 2 && warp < 2 + EPI_WARPS) {
    constexpr int THREADS = 32 * EPI_WARPS;
    const int t = int(threadIdx.x) - 64, w = warp - 2;
    auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory"); };
    if (!args.late_wait) pdl_wait();
    pdl_trigger();
    for (int i = t; i <= args.G; i += THREADS)
      table_first[i] = min(max(args.offsets[i], 0), args.M);   // (as they are)
    sync();
    // An offset below one before it counts as that one, so that no two groups claim a row.
    // Where the widest units make few rounds, the width whose units take the least time is
    // chosen, their rounds by a stage's cycles, 117 + 1.55 bn and 288 at least (see linear.cu);
    // one width per warp.  (Not for more: narrower units keep less in flight.)
    const int parts = (args.bn_cap >> 5) - w;
    if (w == 0 || (!BACKWARD && parts > 0)) {
      int top = 0, n = 0;
      for (int base = 0; base < args.G; base += 32) {
        const int i = base + lane;
        int lo = 0, hi = 0;
        if (i < args.G) {
          lo = max(table_first[i], top);
          hi = max(table_first[i + 1], top);
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int below = __shfl_up_sync(0xffffffffu, lo, o);
          if (lane >= o) lo = max(lo, below);
        }
        hi = max(hi, lo);
        if (w == 0 && i < args.G) {
          table_off[i] = lo;
          if (i == args.G - 1) table_off[args.G] = hi;
        }
        if (!BACKWARD && i < args.G) n += quick_div(((hi - lo + 31) >> 5) + parts - 1, parts);
        top = __shfl_sync(0xffffffffu, hi, 31);
      }
      if (!BACKWARD) {
        n = int(__reduce_add_sync(0xffffffffu, unsigned(n)));
        // (a narrower width has eight times the rounds at most)
        const int rounds = min(quick_div(n * args.tiles_n + num_pairs - 1, num_pairs), 1000);
        const int cost = rounds * max(288, 117 + 31 * (32 * parts) / 20);
        if (lane == 0) found[w] = w > 0 || rounds <= 3 ? cost : -1;
      }
    } else if (!BACKWARD && lane == 0) {
      found[w] = 0x7FFFFFFF;
    }
    sync();
    int best = 0;
    if (!BACKWARD)
      for (int i = 1; i < EPI_WARPS; ++i)
        if (found[i] < found[best]) best = i;
    if (w == best) {
      const int cap = (args.bn_cap >> 5) - best;
      int total = 0;
      for (int base = 0; base < args.G; base += 32) {
        const int i = base + lane;
        const int shape = i < args.G ? shape_of(group_rows(table_off, i), cap) : 0;
        int n = (shape >> 4) * args.tiles_n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int below = __shfl_up_sync(0xffffffffu, n, o);
          if (lane >= o) n += below;
        }
        if (i < args.G) {
          table_shape[i] = shape;
          table_first[i + 1] = total + n;
        }
        total += __shfl_sync(0xffffffffu, n, 31);
      }
      if (lane == 0) {
        table_first[0] = 0;
        chosen[0] = 32 * cap;
      }
    }
    if (BACKWARD) {
      // the groups in the order of their weight gradients: the longest first, up to 256 of them
      // (each counts those before it); more as they come, those without rows last
      if (args.G <= THREADS) {
        const int n = t < args.G ? group_rows(table_off, t) : 0;
        if (t < args.G) {
          int at = 0;
#pragma unroll 4
          for (int j = 0; j < args.G; ++j) {
            const int m = group_rows(table_off, j);
            at += m > n || (m == n && j < t) ? 1 : 0;
          }
          table_order[at] = t;
        }
        const uint32_t some = __ballot_sync(0xffffffffu, n > 0);
        if (lane == 0) found[w] = __popc(some);
      } else if (w == 1) {
        int before_all = 0;
        for (int base = 0; base < args.G; base += 32) {
          const int i = base + lane;
          const bool rows = i < args.G && group_rows(table_off, i) > 0;
          const uint32_t some = __ballot_sync(0xffffffffu, rows);
          const int before = before_all + __popc(some & ((1u << lane) - 1u));
          if (i < args.G) table_order[rows ? before : args.G - 1 - (i - before)] = i;
          before_all += __popc(some);
        }
        if (lane < EPI_WARPS) found[lane] = lane == 0 ? before_all : 0;
      }
      sync();
      if (t == 0) {
        int n = 0;
        for (int i = 0; i < EPI_WARPS; ++i) n += found[i];
        chosen[1] = n;
        // a stage of out takes 500 cycles, one of dw 514, and its stores 4000, added to dw twice that
        const int units = args.out == nullptr ? 0 : table_first[args.G];
        const int rounds = quick_div(units, num_pairs), over = units - rounds * num_pairs;
        const int stages = n > 0 ? (group_rows(table_off, table_order[0]) + 63) / 64 : 0;
        chosen[2] = rounds;
        chosen[3] = num_pairs - over;
        chosen[4] = over > 0 ? quick_div(args.num_kb * 500, max(args.in != nullptr ? 8000 : 4000, stages * 514 + 2300)) : 0;
      }
    }
    sync();
    if (t == 0) mbar_arrive(table_bar);
  }
  // Takes the table, in pass 0 that of one group (false: the wait for it ran out).
  auto start = [&](int pass) -> bool {
    if (!grouped) return true;
    // (pass 0 reads the table of one group, there since the cluster's barrier, and waits for
    // nothing: the real table's barrier completes one phase in a launch, which may be over)
    if (pass == 1 && !mbar_wait(table_bar, 0, abort_flag)) {
      num_units = 0;
      return false;
    }
    const bool real = pass == 1;
    table = Table{real ? table_off : one,       real ? table_first : one + 2, real ? table_shape : one + 5,
                  real ? table_order : one + 4, real ? args.G : 1,            real ? chosen[0] : args.bn_cap};
    cursor = Cursor{};
    rows_units = BACKWARD && args.out == nullptr ? 0 : table.first[table.G];
    num_units = rows_units;
    if (BACKWARD && real) {
      busy = chosen[1];
      num_units += busy * args.tiles_r * args.tiles_n;
      spare = chosen[3];
      const int over = num_pairs - spare;
      of_out = chosen[2] + (pair < over ? 1 : 0);
      turn = pair < over ? spare + pair : pair - over;
      early = turn < spare ? chosen[4] : 0;
      early_all = chosen[4] * spare;
    }
    return true;
  };
  // Ends pass 0, behind which global memory may be read, and gives the next (2: under way).
  auto next_pass = [&](int pass) {
    if (pass == 0) {
      if (!args.late_wait) pdl_wait();
      pdl_trigger();
    }
    return grouped && pass == 0 ? 1 : 2;
  };
  // This pair's unit in round r.
  auto number = [&](int r) {
    if (!BACKWARD || r < of_out) return r * num_pairs + pair;
    const int k = r - of_out;
    return rows_units + turn + (k < early ? k * spare : early_all + (k - early) * num_pairs);
  };
  auto unit_at = [&](int u) {
    return BACKWARD && u >= rows_units ? weight_unit(u - rows_units, table, args) : rows_unit(u, cursor, table, args);
  };
  // stages of K of a unit
  auto stages_of = [&](int rows, bool weight) { return weight ? (rows + 63) / 64 : args.num_kb; };
  // the accumulators' distance, and whether they share columns
  auto sharing = [&] { return OP == OP_BLOCKS && table.cap > 224; };
  auto acc_columns = [&] { return OP == OP_BF16 ? MAX_BN : table.cap > 224 ? 192 : 224; };

  if (warp == 0) {
    if (elect_one()) {
      // ------------------------------------------------------------ producer
      uint32_t issued = 0, issued_parity = 0, ph = 0;
      uint32_t tails = 0, tail_parity = 0;   // stages whose tail barrier was armed, and its phase now
      int s = 0;
      bool ok = true;
      int pass = 0;
      for (int r = 0; ok; ++r) {
        if (pass < 2 && !start(pass)) break;
        const int un = number(r);
        if ((pass > 0 || !grouped) && un >= num_units) break;
        const Unit u = unit_at(pass > 0 || !grouped ? un : 0);
        if (pass < 2 && (pass = next_pass(pass)) == 1) {
          --r;
          continue;
        }
        const bool weight = BACKWARD && un >= rows_units;
        if (rank == 0) {                     // for the issuer (published by the arrival on the first stage's barrier)
          units_bn[r % UNIT_SLOTS] = weight ? -u.bn : u.bn;
          if (BACKWARD) units_rows[r % UNIT_SLOTS] = u.rows;
        }
        const int row_w = u.nb * (2 * BM) + int(rank) * BM;      // of the 256-row operand
        const int half = u.bn / 2;
        const int row_x = (weight ? u.kb * 256 : u.row0) + int(rank) * half;
        const uint32_t stage_tx = 2u * uint32_t(OP_BYTES + half * ROW_BYTES);
        const int num = stages_of(u.rows, weight);
        for (int kb = 0; kb < num; ++kb) {
          if (!mbar_wait(empty_bar(s), ph ^ 1u, abort_flag)) { ok = false; break; }
          const int k0 = kb * stage_k(OP);
          // a stage with rows to be cleared completes on this CTA's own barrier, for the warp
          // that does
          const bool tail = weight && rows_to_clear(u.rows - k0);
          if (rank == 0) {
            if (tail) mbar_arrive(full_bar(s));
            else mbar_expect_tx(full_bar(s), stage_tx);
          }
          if (tail) {
            mbar_expect_tx(tail_bar(s), stage_tx / 2u);
            tails |= 1u << s;
            tail_parity ^= 1u << s;
          }
          const uint32_t fb = tail ? map_to_rank(tail_bar(s), rank) : map_to_rank(full_bar(s), 0);
          const uint32_t da = ring + uint32_t(s) * stage;
          uint32_t db = da + uint32_t(OP_BYTES);
          if (weight) {
            const int row = u.begin + k0;
            tma_load_2d_pair(da, &maps.dout_mn, fb, row_w, row);
            tma_load_2d_pair(da + MN_BOX_BYTES, &maps.dout_mn, fb, row_w + 64, row);
            tma_load_2d_pair(db, &maps.x_mn, fb, row_x, row);
            if (half > 64) tma_load_2d_pair(db + MN_BOX_BYTES, &maps.x_mn, fb, row_x + 64, row);
          } else {
            if (BACKWARD) {
              tma_load_3d_pair(da, &maps.w, fb, row_w, k0, u.group);
              tma_load_3d_pair(da + MN_BOX_BYTES, &maps.w, fb, row_w + 64, k0, u.group);
            } else {
              tma_load_3d_pair(da, &maps.w, fb, k0, row_w, u.group);
            }
            int row = row_x;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              if (half & (128 >> b)) {
                tma_load_2d_pair(db, &maps.x[b], fb, k0, row);
                db += uint32_t((128 >> b) * ROW_BYTES);
                row += 128 >> b;
              }
            }
          }
          issued |= 1u << s;
          issued_parity = (issued_parity & ~(1u << s)) | (ph << s);
          if (++s == args.stages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      // before shared memory is released every phase the leader armed completes, and
      // the MMAs' last arrivals reach this CTA
      for (int k = 0; k < args.stages; ++k)
        if (issued & (1u << k)) {
          if (BACKWARD && (tails & (1u << k)))
            mbar_wait(tail_bar(k), ((tail_parity >> k) & 1u) ^ 1u, abort_flag, false, kDrainLimitNs);
          if (rank == 0) mbar_wait(full_bar(k), (issued_parity >> k) & 1u, abort_flag, false, kDrainLimitNs);
          mbar_wait(empty_bar(k), (issued_parity >> k) & 1u, abort_flag, false, kDrainLimitNs);
        }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      // ------------------------------------------------------------ MMA issuer (leader)
      int s = 0, local = 0, chunk = 0;
      uint32_t ph = 0, cleared_parity = 0;
      start(0);
      next_pass(0);                        // (a bounded wait begins behind the preceding kernel)
      bool ok = start(1);
      const bool shared = sharing();
      const int acc_cols = acc_columns();
      for (int un = number(0); ok && un < num_units; un = number(++local)) {
        const int acc = local & 1;
        if (!mbar_wait(full_bar(s), ph, abort_flag)) break;
        const int width = units_bn[local % UNIT_SLOTS], rows = BACKWARD ? units_rows[local % UNIT_SLOTS] : 0;
        const bool weight = BACKWARD && width < 0;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + uint32_t(acc * acc_cols);
        const uint32_t idesc = idesc_for(OP, BACKWARD, weight, weight ? -width : width);
        const int num = stages_of(rows, weight);
        uint32_t sf = 0;                     // TMEM columns of the current scales
        bool ready = true;                   // the next stage was there before this one's MMAs were issued
        for (int kb = 0; kb < num; ++kb) {
          if (OP == OP_BLOCKS && (kb & 3) == 0) {
            const int ss = chunk % SF_STAGES;
            if (!mbar_wait_cluster_bounded(sfull_bar(ss), uint32_t(chunk / SF_STAGES) & 1u, abort_flag, &g_status, kWaitLimitNs)) {
              ok = false;
              break;
            }
            tc_fence_after();
            sf = tmem_base + uint32_t(SF_TMEM + 16 * (chunk & 1));
            const uint32_t src = smem_u32(sScales) + uint32_t(ss * SF_BYTES);
            copy_scales(sf, sdesc_scales(src));
            copy_scales(sf + 4, sdesc_scales(src + 512));
            copy_scales(sf + 8, sdesc_scales(src + 1024));
            mma_commit_mc(sempty_bar(ss), kBothCtas);
            ++chunk;
          }
          if (!ready && !mbar_wait(full_bar(s), ph, abort_flag)) { ok = false; break; }
          if (weight && rows_to_clear(rows - kb * 64)) {
            if (!mbar_wait_cluster_bounded(cleared_bar(s), (cleared_parity >> s) & 1u, abort_flag, &g_status, kWaitLimitNs)) {
              ok = false;
              break;
            }
            cleared_parity ^= 1u << s;
          }
          if (kb == 0) {
            // the accumulator has been read, or, where it shares columns with that of the unit
            // before, that unit's share of them (a warp that says so has read the one before)
            const int of = shared ? local - 1 : local - 2;
            if (of >= 0 && !mbar_wait_cluster_bounded(tempty_bar(of & 1), uint32_t(of >> 1) & 1u, abort_flag, &g_status, kWaitLimitNs)) {
              ok = false;
              break;
            }
          }
          tc_fence_after();
          const uint32_t a0 = ring + uint32_t(s) * stage, b0 = a0 + uint32_t(OP_BYTES), empty = empty_bar(s);
          if (++s == args.stages) {
            s = 0;
            ph ^= 1u;
          }
          ready = kb + 1 < num && mbar_test_wait(full_bar(s), ph);
          if (OP == OP_BLOCKS) {
            const uint32_t which = uint32_t(kb & 3);
            const uint32_t id = idesc | (which << 4) | (which << 29);
#pragma unroll
            for (int i = 0; i < STEPS; ++i)
              mma_pair_blocks(d_tmem, step_desc<false>(a0, i), step_desc<false>(b0, i), id, sf, sf + 4, uint32_t(kb | i));
          } else if (weight) {
#pragma unroll
            for (int i = 0; i < STEPS; ++i)
              if (kb * 64 + 16 * i < rows) mma_pair_f16(d_tmem, step_desc<true>(a0, i), step_desc<true>(b0, i), idesc, uint32_t(kb | i));
          } else {
#pragma unroll
            for (int i = 0; i < STEPS; ++i)
              mma_pair_f16(d_tmem, step_desc<BACKWARD>(a0, i), step_desc<false>(b0, i), idesc, uint32_t(kb | i));
          }
          mma_commit_mc(empty, kBothCtas);
        }
        if (!ok) break;
        mma_commit_mc(tfull_bar(acc), kBothCtas);
      }
      mma_commit_mc(drain_bar, kLeaderOnly);
      mbar_wait(drain_bar, 0, abort_flag, false, kDrainLimitNs);
    }
    __syncwarp();
  } else if (OP == OP_BLOCKS && warp >= 2 + EPI_WARPS) {
    // -------------------------------------------------------------- scales
    // Four blocks (512 of K, a chunk) at a time, the warps in turn: reading a few bytes of many
    // rows and publishing them takes a warp 1 to 2 us (with two warps instead of four 128 x
    // 4096 x 14336 took 30.0 us instead of 27.3).  Warp and stage of a chunk are its number modulo
    // four, so a stage is one warp's, as waits by parity need.  Lane l holds the words (four
    // blocks' bytes) of rows l, l + 32, ... of x; this CTA's 128 weight rows have one word.
    // Blocks behind the last are never multiplied with.
    const int mine = warp - (2 + EPI_WARPS);
    const bool whole = ((reinterpret_cast<uintptr_t>(args.x_scale) | reinterpret_cast<uintptr_t>(args.w_scale) | uintptr_t(args.blocks)) & 3u) == 0;
    const int chunks = (args.num_kb + 3) / 4;          // of a unit
    const uint8_t* const xs_end = args.x_scale + size_t(args.M) * size_t(args.blocks);
    const uint8_t* const ws_end = args.w_scale + size_t(args.G) * size_t(args.n_blocks) * size_t(args.blocks);
    const uint32_t dst = smem_u32(sScales) + uint32_t(mine * SF_BYTES + lane * 16);
    int r = 0, c = mine;
    uint32_t fills = 0;
    bool ok = true, fresh = true;
    int pass = 0;
    Unit u{};
    while (ok) {
      for (; c >= chunks; c -= chunks) {
        ++r;
        fresh = true;
      }
      if (pass < 2) {
        ok = __all_sync(0xffffffffu, start(pass));
        if (!ok) break;
        fresh = true;
      }
      const int un = number(r);
      if ((pass > 0 || !grouped) && un >= num_units) break;
      if (fresh) u = unit_at(pass > 0 || !grouped ? un : 0);
      fresh = false;
      const int left = args.blocks - 4 * c;
      const int block_w = min(u.nb * 2 + int(rank), args.n_blocks - 1);
      const uint8_t* const wp =
          args.w_scale + (size_t(u.group) * size_t(args.n_blocks) + size_t(block_w)) * size_t(args.blocks) + size_t(4 * c);
      // (rows behind the last count as that one; the addresses do not descend)
      const uint8_t* const last = args.x_scale + size_t(args.M - 1) * size_t(args.blocks) + size_t(4 * c);
      const uint8_t* xp[8];
      xp[0] = args.x_scale + size_t(min(u.row0 + lane, args.M - 1)) * size_t(args.blocks) + size_t(4 * c);
#pragma unroll
      for (int i = 1; i < 8; ++i) {
        const uint8_t* const p = xp[i - 1] + 32 * args.blocks;
        xp[i] = 32 * i >= u.bn ? xp[i - 1] : p < last ? p : last;
      }
      const bool within = scales_within(wp, args.w_scale, ws_end) && scales_within(xp[0], args.x_scale, xs_end) &&
                          scales_within(xp[7], args.x_scale, xs_end);
      if (pass < 2) {                        // (the addresses ahead of the wait for the preceding kernel)
        pass = next_pass(pass);
        if (pass == 1) continue;
      }
      uint32_t w, x[8];
      if (whole) {
        w = scales_word(wp)[0];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 32 * i < u.bn ? scales_word(xp[i])[0] : 0u;
      } else if (__all_sync(0xffffffffu, within)) {
        w = scales_joined(wp);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 32 * i < u.bn ? scales_joined(xp[i]) : 0u;
      } else {
        w = scales_bytes(wp, left);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 32 * i < u.bn ? scales_bytes(xp[i], left) : 0u;
      }
      ok = __all_sync(0xffffffffu, mbar_wait(sempty_bar(mine), (fills & 1u) ^ 1u, abort_flag));
      if (!ok) break;
      sts16(dst, make_uint4(w, w, w, w));
      sts16(dst + 512, make_uint4(x[0], x[1], x[2], x[3]));
      sts16(dst + 1024, make_uint4(x[4], x[5], x[6], x[7]));
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) hand_over(sfull_bar(mine), rank);
      ++fills;
      c += SCALE_WARPS;
    }
    // the issuer's last arrival on this stage reaches this CTA
    if (ok && fills > 0) mbar_wait(sempty_bar(mine), (fills & 1u) ^ 1u, abort_flag, false, kDrainLimitNs);
    __syncwarp();
  } else if (BACKWARD && warp >= 2 + EPI_WARPS) {
    // -------------------------------------------------------------- rows behind a group
    // The last stage of a unit of dw: rows behind the group's end, up to the next multiple of
    // 16, are overwritten with zeros in the four boxes of this CTA's operands (row r of a box
    // is its bytes 128 r ..).
    uint32_t parity = 0;
    int s = 0;
    next_pass(0);
    __all_sync(0xffffffffu, start(1));
    for (int r = 0, un = number(0); un < num_units; un = number(++r)) {
      const bool weight = un >= rows_units;
      const Unit u = weight ? unit_at(un) : Unit{};
      const int num = stages_of(u.rows, weight), live = u.rows - (num - 1) * 64;
      s = (s + num - 1) % args.stages;
      if (weight && rows_to_clear(live)) {
        if (!__all_sync(0xffffffffu, mbar_wait(tail_bar(s), (parity >> s) & 1u, abort_flag))) break;
        parity ^= 1u << s;
        const uint32_t at = ring + uint32_t(s) * stage + uint32_t(live * ROW_BYTES);
        for (int i = lane * 16; i < (-live & 15) * ROW_BYTES; i += 512) {
#pragma unroll
          for (int b = 0; b < 4; ++b) sts16(at + uint32_t(b * MN_BOX_BYTES + i), make_uint4(0, 0, 0, 0));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) hand_over(cleared_bar(s), rank);
      }
      s = s + 1 == args.stages ? 0 : s + 1;
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- epilogue
    // Two warps per TMEM lane quarter q (32 rows of the 256-row operand), which share
    // the unit's columns.  A box of shared memory turns the accumulator's layout into
    // that of the global accesses, 16 bytes per lane (see linear.cu).
    constexpr int WG = EPI_WARPS / 4;
    const int q = warp & 3, wg = (warp - 2) >> 2;
    const uint32_t box = smem_u32(sStaging + (q * WG + wg) * staging_box(KIND));
    start(1);
    if (!grouped) pdl_wait();
    const uint16_t* const bias_row = behind_wait(args.bias);
    const bool shared = sharing();
    const int acc_cols = acc_columns();
    int local = 0, un = number(0);
    {
      // out: the lanes are columns of the output, the accumulator's columns its rows, 32 at a
      // time.  TMEM loads of 16 lanes by 8 columns give each thread two neighbouring rows of
      // the output for one column, the fragment of an 8 x 8 block: rounded to bf16, blocks
      // are stored transposed (stmatrix) to a box of 32 rows x 64 bytes (chunk c of row r at
      // c ^ (r / 2 & 3)), from which rows of the output leave 16 bytes a lane.  What is added
      // takes the same way back (ldmatrix).  (The accumulator turned through the box in
      // fp32, a word at a time: 8192 x 4096 x 1024 33.8 us, so 29.1.)
      const int sub = lane >> 2, ch = lane & 3;
      const uint32_t turn16 = box + uint32_t(sub) * 64u + (uint32_t(ch ^ ((sub >> 1) & 3)) << 4);
      // this lane's row of the four blocks of eight rows: block of columns lane / 8, row lane % 8
      const uint32_t block8 = box + uint32_t(lane & 7) * 64u + (uint32_t((lane >> 3) ^ ((lane >> 1) & 3)) << 4);
      const size_t step = size_t(8) * size_t(args.N);
      for (; un < rows_units; un = number(++local)) {
        const int acc = local & 1;
        const uint32_t aph = uint32_t(local >> 1) & 1u;
        const Unit u = unit_at(un);
        const int row_end = min(u.begin + u.rows, u.row0 + u.bn);
        const int col0 = u.nb * (2 * BM) + int(rank) * BM + q * 32, col = col0 + ch * 8;
        const uint32_t tbase = tmem_base + (uint32_t(q * 32) << 16) + uint32_t(acc * acc_cols);
        // this warp's groups are g0, g0 + by, ..; the columns that the accumulators share first
        const int groups = u.bn / 32, by = shared && acc == 0 ? -WG : WG, g0 = by > 0 ? wg : groups - 1 - wg;
        // (a quarter of the lanes past the last column has none)
        const int count = col0 < args.N ? (groups - wg + WG - 1) / WG : 0;
        const size_t at = size_t(u.row0 + sub) * size_t(args.N) + size_t(col);
        const int rows_here = col < args.N ? row_end - u.row0 - sub : 0;   // group g: rows 8 i < rows_here - 32 g
        float bias[4] = {0.0f, 0.0f, 0.0f, 0.0f};      // of columns sub, 8 + sub, ..
        if (!BACKWARD && args.bias != nullptr) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (col0 + 8 * j < args.N) bias[j] = bf16_to_f32(bias_row[col0 + 8 * j + sub]);
        }
        uint4 next_in[4];                    // what is added, requested a group ahead
        auto request = [&](int g) {
          const int left = g >= 0 && g < groups ? rows_here - 32 * g : 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            next_in[i] = make_uint4(0, 0, 0, 0);
            if (8 * i < left) next_in[i] = ld16_stream(args.in + (at + size_t(4 * g + i) * step));
          }
        };
        if (!BACKWARD && args.in != nullptr) {
          // the first group's are requested here, the others' set out for L2
          if ((ch & 1) == 0)
            for (int k = 1, g = g0 + by; k < count; ++k, g += by) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (8 * i < rows_here - 32 * g) prefetch_l2(args.in + (at + size_t(4 * g + i) * step));
            }
          if (count > 0) request(g0);
        }
        if (!mbar_wait(tfull_bar(acc), aph, abort_flag)) { un = num_units; break; }
        tc_fence_after();
        const bool awaited = number(local + (shared ? 1 : 2)) < num_units;   // another unit waits for this accumulator
        auto loaded = [&](int k) {
          if (k == (shared ? 0 : count - 1)) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && awaited) mbar_arrive_remote_relaxed(map_to_rank(tempty_bar(acc), 0));
          }
        };
        auto issue = [&](int g, uint32_t (&lo)[16], uint32_t (&hi)[16]) {   // lanes 0 .. 15 and 16 .. 31 of the quarter
          tmem_ld_blocks_issue(tbase + uint32_t(g * 32), tbase + (16u << 16) + uint32_t(g * 32), lo, hi);
        };
        uint16_t* const dst = args.out + at;
        auto leave = [&](int g) {            // the box's rows to the output
          __syncwarp();
          uint4 o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = lds16(turn16 + 512u * i);
          uint16_t* row = dst + size_t(4 * g) * step;
          const int left = rows_here - 32 * g;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (8 * i < left) stg16(row, o[i]);
            row += step;
          }
        };
        // (two loops, so that the common one is free of branches)
        auto process = [&](auto extras, int g, const uint32_t (&lo)[16], const uint32_t (&hi)[16]) {
          __syncwarp();                      // the previous group has been read out of the box
          if (decltype(extras)::value && args.in != nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i) sts16(turn16 + 512u * i, next_in[i]);
            __syncwarp();
            request(g + by);
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {      // rows 8 c .. of the group, four blocks of columns
            uint32_t p[4];
            if (decltype(extras)::value) {
              uint64_t z[4] = {f2_pack(__uint_as_float(lo[4 * c]), __uint_as_float(lo[4 * c + 1])),
                               f2_pack(__uint_as_float(lo[4 * c + 2]), __uint_as_float(lo[4 * c + 3])),
                               f2_pack(__uint_as_float(hi[4 * c]), __uint_as_float(hi[4 * c + 1])),
                               f2_pack(__uint_as_float(hi[4 * c + 2]), __uint_as_float(hi[4 * c + 3]))};
              uint32_t d[4] = {0u, 0u, 0u, 0u};
              if (args.in != nullptr) ldmatrix_trans(block8 + 512u * c, d);
#pragma unroll
              for (int j = 0; j < 4; ++j) p[j] = pack2(f2_add(f2_add(z[j], f2_pack(bias[j], bias[j])), bf16x2_to_f2(d[j])));
            } else {
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                p[j] = pack_bf16x2(__uint_as_float(lo[4 * c + 2 * j]), __uint_as_float(lo[4 * c + 2 * j + 1]));
                p[2 + j] = pack_bf16x2(__uint_as_float(hi[4 * c + 2 * j]), __uint_as_float(hi[4 * c + 2 * j + 1]));
              }
            }
            stmatrix_trans(block8 + 512u * c, p);
          }
          leave(g);
        };
        auto unit = [&](auto extras) {
          for (int k = 0, g = g0; k < count; ++k, g += by) {
            uint32_t lo[16], hi[16];
            issue(g, lo, hi);
            tmem_wait_ld16(lo, hi);
            loaded(k);
            process(extras, g, lo, hi);
          }
        };
        if (count <= 0) loaded(shared ? 0 : count - 1);   // (a unit with fewer groups than warps)
        else if (!BACKWARD && (args.in != nullptr || args.bias != nullptr)) unit(Flag<!BACKWARD>{});
        else unit(Flag<false>{});
      }
    }
    if constexpr (BACKWARD) {
      // dw (+)= the sums: the lane is a row of the matrix; 64 columns at a time through a box
      // of 32 rows x 128 bytes (chunk c of row r at c ^ (r & 7)), whole 128-byte lines
      const int sub8 = lane >> 3, ch8 = lane & 7;
      const uint32_t row32 = box + uint32_t(lane) * 128u + (uint32_t(lane & 7) << 4);
      const uint32_t turn8 = box + uint32_t(sub8) * 128u + (uint32_t(ch8 ^ sub8) << 4);
      const size_t step4 = size_t(4) * size_t(args.N);
      struct Part {
        int col;                             // column of this lane's share of the first 64
        int row0, box_col, group;            // of the warp's first box
        uint32_t rows;                       // bit i: row sub8 + 4 i exists
        size_t at;
      };
      auto part_of = [&](const Unit& u) {
        Part p;
        const int row0 = u.nb * (2 * BM) + int(rank) * BM + q * 32;
        p.col = u.kb * 256 + ch8 * 8;
        p.row0 = row0;
        p.box_col = u.kb * 256;
        p.group = u.group;
        p.rows = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) p.rows |= (row0 + sub8 + 4 * i < args.rows ? 1u : 0u) << i;
        p.at = (size_t(u.group) * size_t(args.rows) + size_t(row0 + sub8)) * size_t(args.N) + size_t(p.col);
        return p;
      };
      constexpr int GROUPS = 4 / WG;         // groups of 64 columns of a warp
      uint4 in8[GROUPS][8];
      auto request = [&](const Part& p, int k, uint4 (&d)[8]) {
        const int g = wg + k * WG;
        const uint32_t live = p.col + g * 64 < args.N ? p.rows : 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          d[i] = make_uint4(0, 0, 0, 0);
          if ((live >> i) & 1u) d[i] = ld16_stream(args.in + (p.at + size_t(g * 64) + size_t(i) * step4));
        }
      };
      Part p{};
      if (un < num_units) {
        p = part_of(unit_at(un));
        if (args.in != nullptr) {
#pragma unroll
          for (int k = 0; k < GROUPS; ++k) request(p, k, in8[k]);
        }
      }
      for (; un < num_units; un = number(++local)) {
        const int acc = local & 1;
        const uint32_t aph = uint32_t(local >> 1) & 1u;
        const uint32_t tbase = tmem_base + (uint32_t(q * 32) << 16) + uint32_t(acc * acc_cols);
        const int next = number(local + 1);
        const bool awaited = number(local + 2) < num_units;
        const Part p_next = part_of(unit_at(next < num_units ? next : un));
        if (!mbar_wait(tfull_bar(acc), aph, abort_flag)) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < GROUPS; ++k) {
          const int g = wg + k * WG;
          if (lane == 0) bulk_wait_read_0();   // the previous group has been read out of the box
          __syncwarp();
          if (args.in != nullptr) {
#pragma unroll
            for (int i = 0; i < 8; ++i) sts16((turn8 ^ uint32_t((i & 1) << 6)) + 512u * i, in8[k][i]);
            __syncwarp();
            if (next < num_units) request(p_next, k, in8[k]);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t v[32];
            tmem_ld32(tbase + uint32_t(g * 64 + h * 32), v);
            if (h == 1 && k == GROUPS - 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0 && awaited) mbar_arrive_remote_relaxed(map_to_rank(tempty_bar(acc), 0));
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t addr = row32 ^ uint32_t(16 * (4 * h + c));
              uint64_t z[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                z[j] = f2_pack(__uint_as_float(v[8 * c + 2 * j]), __uint_as_float(v[8 * c + 2 * j + 1]));
              if (args.in != nullptr) {
                const uint4 d = lds16(addr);
                const uint32_t dw[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) z[j] = f2_add(z[j], bf16x2_to_f2(dw[j]));
              }
              sts16(addr, pack8(z));
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && p.box_col + g * 64 < args.N && p.row0 < args.rows) {
            tma_store_3d(&maps.dw, box, p.box_col + g * 64, p.row0, p.group);
            bulk_commit();
          }
        }
        p = p_next;
      }
      if (lane == 0) bulk_wait_all();
      // the gradient of a matrix without rows is zero, or what it was when adding
      if (args.in == nullptr && *abort_flag == 0) {
        const int per_group = args.tiles_r * args.tiles_n;
        for (int e = busy * per_group + pair; e < args.G * per_group; e += num_pairs) {
          const Part z = part_of(weight_unit(e, table, args));
#pragma unroll
          for (int k = 0; k < GROUPS; ++k) {
            const int g = wg + k * WG;
            const uint32_t live = z.col + g * 64 < args.N ? z.rows : 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if ((live >> i) & 1u) stg16(args.dw + (z.at + size_t(g * 64) + size_t(i) * step4), make_uint4(0, 0, 0, 0));
          }
        }
      }
    }
  }

  if (args.late_wait) pdl_wait();    // this kernel is not complete before the preceding one
  // Both CTAs finish together: the leader's MMAs write the peer's TMEM and
  // both CTAs signal barriers of the other.  (Every arrival and copy that the other
  // CTA makes here has been waited for, so the barrier orders no memory.)
  tc_fence_before();
  __syncthreads();
  cluster_sync_relaxed();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS)
                 : "memory");
  }
}

// ------------------------------------------------------------------ host side
// 2-CTA clusters of a form that fit on the device at once (cached per device).
template <int OP, int KIND>
cudaError_t max_pairs(int* pairs) {
  static int cached[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && cached[dev] > 0) {
    *pairs = cached[dev];
    return cudaSuccess;
  }
  const auto fn = grouped_kernel<OP, KIND>;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_LIMIT + 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (num_sms() / 2));
  cfg.blockDim = dim3(num_threads(OP, KIND));
  cfg.dynamicSmemBytes = SMEM_LIMIT + 1024;
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

// `units`: no fewer than the kernel will find
template <int OP, int KIND>
cudaError_t launch(const Maps& m, GroupArgs a, int64_t units, int pairs, cudaStream_t s) {
  const int table = (KIND == KIND_BACKWARD ? 16 : 12) * (a.G + 1) + 4 * EPI_WARPS;
  // (narrow units: more stages, whose loads' latency is what bounds them; 512 x 4096 x 2048
  // with six stages 11.3 us, with eight 10.7)
  a.stage_bytes = OP_BYTES + a.bn_cap / 2 * ROW_BYTES;
  a.stages = (SMEM_LIMIT - fixed_bytes(OP, KIND) - table) / a.stage_bytes;
  if (a.stages > MAX_STAGES) a.stages = MAX_STAGES;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * unsigned(units < pairs ? units : pairs));
  cfg.blockDim = dim3(num_threads(OP, KIND));
  cfg.dynamicSmemBytes = size_t(a.stages * a.stage_bytes + fixed_bytes(OP, KIND) + table + 1024);
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
  return cudaLaunchKernelEx(&cfg, grouped_kernel<OP, KIND>, m, a);
}

int ceil_div(int64_t a, int64_t b) { return int((a + b - 1) / b); }

// One group's rows are cut so that its units fill the SM pairs in the fewest and
// narrowest rounds, a stage taking 117 + 1.55 bn cycles and 288 at least (see linear.cu).
int cut_rows(int64_t M, int tiles_n, int pairs) {
  const int64_t parts = (M + 31) / 32;
  int best = MAX_BN;
  int64_t least = -1;
  for (int64_t tm = (parts + 7) / 8; tm < (parts + 7) / 8 + 8 && tm <= parts; ++tm) {
    const int bn = 32 * int((parts + tm - 1) / tm);
    const int64_t rounds = (tm * tiles_n + pairs - 1) / pairs;
    const int64_t stage = 117 + 31 * bn / 20;
    const int64_t cost = rounds * (stage > 288 ? stage : 288);
    if (least < 0 || cost < least) {
      best = bn;
      least = cost;
    }
  }
  return best;
}
// Most rows of a unit.  Several groups, whose sizes the host does not know: the widest, or 128
// where they have few rows, for the sake of more stages.
int choose_cap(int64_t G, int64_t M, int tiles_n, int pairs) {
  return G == 1 ? cut_rows(M, tiles_n, pairs) : M / G < 96 ? 128 : MAX_BN;
}

// out [M, N] from x [M, K] and w [G, N, K].
template <int OP>
cudaError_t forward(uint16_t* out, const void* x, const uint8_t* x_scale, const void* w, const uint8_t* w_scale,
                    const uint16_t* bias, const uint16_t* in, const int* offsets, int64_t G, int64_t M, int64_t N,
                    int64_t K, cudaStream_t s) {
  constexpr bool BF16 = OP == OP_BF16;
  const int64_t bytes = BF16 ? 2 : 1;
  Maps m{};
  bool ok = make_operand_map_3d(&m.w, w, BF16, G, N, K, K * bytes, K * N * bytes, 128);
  for (int b = 0; ok && b < 4; ++b) ok = make_operand_map(&m.x[b], x, BF16, M, K, 128 >> b);
  if (!ok) return cudaErrorInvalidValue;
  GroupArgs a{};
  a.out = out;
  a.bias = bias;
  a.in = in;
  a.x_scale = x_scale;
  a.w_scale = w_scale;
  a.blocks = ceil_div(K, 128);
  a.n_blocks = ceil_div(N, 128);
  a.offsets = offsets;
  a.G = int(G);
  a.M = int(M);
  a.N = int(N);
  a.tiles_n = ceil_div(N, 2 * BM);
  int pairs = 0;
  const cudaError_t e = max_pairs<OP, KIND_FORWARD>(&pairs);
  if (e != cudaSuccess) return e;
  a.num_kb = ceil_div(K, stage_k(OP));
  a.bn_cap = choose_cap(G, M, a.tiles_n, pairs);
  // bands of about 32 MB of weights where they are the larger operand (see linear.cu)
  const int64_t band = (int64_t(32) << 20) / (2 * BM * K * bytes);
  a.band_n = N <= M / G || band >= a.tiles_n ? a.tiles_n : band < 1 ? 1 : int(band);
  // (a cap chosen on the device is 32 at least)
  const int64_t units = (M / (offsets != nullptr ? 32 : a.bn_cap) + (G < M ? G : M)) * a.tiles_n;
  return launch<OP, KIND_FORWARD>(m, a, units, pairs, s);
}

// dx [M, K] (NULL: none) and dw [G, N, K] (+)= from dout [M, N], x [M, K] and w [G, N, K].
cudaError_t backward(uint16_t* dx, uint16_t* dw, const uint16_t* dout, const uint16_t* x, const uint16_t* w,
                     const int* offsets, int64_t G, int64_t M, int64_t N, int64_t K, bool accumulate, bool late_wait,
                     cudaStream_t s) {
  Maps m{};
  bool ok = make_operand_map_3d(&m.w, w, true, G, N, K, K * 2, K * N * 2, 64) &&
            make_operand_map(&m.dout_mn, dout, true, M, N, 64) && make_operand_map(&m.x_mn, x, true, M, K, 64);
  ok = ok && make_operand_map_3d(&m.dw, dw, true, G, N, K, K * 2, K * N * 2, 32);
  for (int b = 0; ok && b < 4; ++b) ok = make_operand_map(&m.x[b], dout, true, M, N, 128 >> b);
  if (!ok) return cudaErrorInvalidValue;
  GroupArgs a{};
  a.out = dx;
  a.dw = dw;
  a.in = accumulate ? dw : nullptr;
  a.late_wait = late_wait ? 1 : 0;
  a.offsets = offsets;
  a.G = int(G);
  a.M = int(M);
  a.N = int(K);
  a.rows = int(N);
  a.tiles_n = ceil_div(K, 256);
  a.tiles_r = ceil_div(N, 256);
  a.bn_cap = MAX_BN;
  a.num_kb = ceil_div(N, 64);
  const int64_t band = (int64_t(32) << 20) / (2 * BM * N * 2);
  a.band_n = K <= M / G || band >= a.tiles_n ? a.tiles_n : band < 1 ? 1 : int(band);
  int pairs = 0;
  const cudaError_t e = max_pairs<OP_BF16, KIND_BACKWARD>(&pairs);
  if (e != cudaSuccess) return e;
  const int64_t units = int64_t(a.tiles_r) * a.tiles_n * G + (dx != nullptr ? (M / a.bn_cap + (G < M ? G : M)) * a.tiles_n : 0);
  return launch<OP_BF16, KIND_BACKWARD>(m, a, units, pairs, s);
}

}  // namespace

// An estimate of a call's SM cycles behind its start and end, beside those of few_rows.cu: 9 for
// each row of a unit, and the stages at 117 + 1.55 bn and 440 at least.  (Fitted to whole calls of
// one round of units or a few, whose stages wait for their loads; cut_rows compares widths by the
// 288 that a stage takes in a long unit.)
int64_t unit_cycles(int64_t units, int64_t bn, int64_t num_kb) {
  const int64_t pairs = kNumSMsHint / 2, stage = 117 + 31 * bn / 20;
  return 9 * bn + (units + pairs - 1) / pairs * num_kb * (stage > 440 ? stage : 440);
}

// Which form a block-scaled layer takes.  grouped_few.cu up to 8 rows, and up to 16 and 32
// while the weights are small: us, it against few_rows.cu and this file: 1 row of 4096 x 14336
// 13.3 / 13.3 / 25, 9 of 3136 x 624 2.9 / 4.5 / 4.6, 15 of 632 x 2272 3.5 / 5.0 / 6.5, 16 of 4096 x
// 4096 7.0 / 7.2 / 10.5, 10 of 1144 x 10960 8.6 / 6.9 / 20, 26 of 184 x 256 2.7 / 3.9 / 3.8, 22 of 6888
// x 512 5.7 / 4.2 / 4.0.  few_rows.cu up to 4096 rows where nine tenths of its estimate are below
// this file's, 6000 cycles for the call (the pair chosen on 70 sizes of 9 to 4000 rows is 0.3%
// behind the better form on average): few_rows.cu against this, 64 rows of 4096 x 14336 14.4 / 25,
// of 4096 x 4096 8.2 / 10.6, 256 of 4096 x 4096 10.7 / 10.5, 512 of 4096 x 4096 13.7 / 11.5, of 2048 x
// 14336 21 / 25, 1700 of 152 x 11088 15 / 27, 2427 of 632 x 10016 25 / 21.
cudaError_t launch_linear_blocks(uint16_t* out, const uint8_t* x, const uint8_t* x_scale, const uint8_t* w,
                                 const uint8_t* w_scale, const uint16_t* bias, const uint16_t* res, int64_t M, int64_t N,
                                 int64_t K, cudaStream_t s) {
  if (M == 0) return cudaSuccess;
  if (M <= 8 || (M <= 16 && N * K <= (int64_t(1) << 23)) || (M <= 32 && N * K <= (int64_t(1) << 18)))
    return launch_few_groups(out, x, x_scale, w, w_scale, bias, res, nullptr, 1, M, N, K, s);
  const int64_t few = few_rows_cycles(M, N, K, false, true, 4096);
  if (few >= 0) {
    const int tiles_n = ceil_div(N, 2 * BM), bn = cut_rows(M, tiles_n, kNumSMsHint / 2);
    const int64_t here = 6000 + unit_cycles(int64_t(ceil_div(M, bn)) * tiles_n, bn, ceil_div(K, 128));
    if (9 * few < 10 * here) return launch_few_rows_blocks(out, x, x_scale, w, w_scale, bias, res, M, N, K, s);
  }
  return forward<OP_BLOCKS>(out, x, x_scale, w, w_scale, bias, res, nullptr, 1, M, N, K, s);
}

// The same for groups of the average size, with 9000 cycles for the call.
int64_t grouped_cycles(int op, int64_t G, int64_t M, int64_t N, int64_t K) {
  const int64_t groups = G < M ? G : M, rows = (M + groups - 1) / groups;
  const int cap = (M / G < 96 ? 128 : MAX_BN) / 32;
  const int64_t parts = (rows + 31) / 32, tiles = (parts + cap - 1) / cap, bn = 32 * ((parts + tiles - 1) / tiles);
  return 9000 + unit_cycles(groups * tiles * ceil_div(N, 2 * BM), bn, ceil_div(K, stage_k(op)));
}

// grouped_few.cu: up to 32 rows and 8 per group on average, while it has a few thousand CTAs
// (each costs 1.6 ns in E4M3).  Measured, us, it against this file: bf16 2 rows, 2 groups with
// rows of 4096 x 2048 7.5 / 10.6, of 14336 x 4096 36 / 39, 16 rows of one of four of 2048 x 2048 8.0
// / 9.7, 32 of one 13.6 / 9.7; E4M3 a row in each of two of 4096 x 2048 5.6 / 8.0, three in each
// of 64 of 4096 x 2048 114 / 84.
// few_rows.cu where its estimate is the lower (on 60 sizes, 2.3% in E4M3 and 1.1% in bf16 behind
// the better form on average).  It against this file: E4M3 184 rows in 15 groups of 152 x 11648
// 10.8 / 22.5, 196 in seven of 1264 x 8016 17.8 / 20.6, 40 in ten of 2728 x 2048 12.8 / 14.8, 1235 in
// one of 2376 x 2672 21.8 / 13.9, 2268 in six of 2656 x 288 15.2 / 10.0; bf16 the first 15.1 /
// 34.7, 554 in two of 144 x 3840 9.7 / 15.6, 600 in two of 4096 x 4096 32 / 22.
cudaError_t launch_grouped(uint16_t* out, const void* x, const uint8_t* x_scale, const void* w, const uint8_t* w_scale,
                           const int* offsets, int64_t G, int64_t M, int64_t N, int64_t K, cudaStream_t s) {
  if (M == 0) return cudaSuccess;
  const bool fp8 = x_scale != nullptr;
  if (M <= 32 && M <= 8 * G && (G < M ? G : M) * ((N + 15) / 16) <= (fp8 ? 2048 : 4096))
    return launch_few_groups(out, x, x_scale, w, w_scale, nullptr, nullptr, offsets, G, M, N, K, s);
  const int64_t few = few_rows_grouped_cycles(G, M, N, K, fp8);
  const int64_t here = grouped_cycles(fp8 ? OP_BLOCKS : OP_BF16, G, M, N, K);
  if (few >= 0 && few < here)
    return launch_few_rows_grouped(out, x, x_scale, w, w_scale, offsets, G, M, N, K, s);
  if (fp8) return forward<OP_BLOCKS>(out, x, x_scale, w, w_scale, nullptr, nullptr, offsets, G, M, N, K, s);
  return forward<OP_BF16>(out, x, nullptr, w, nullptr, nullptr, nullptr, offsets, G, M, N, K, s);
}

// Both gradients in one launch, unless a unit of dx, whose stages of N follow one another at 480
// cycles, takes longer than dx by few_rows.cu (N split over a cluster) and dw behind it, beside
// it where SMs are free: 7000 cycles for the call, 3400 for each round of units.  Measured,
// us, one launch against two: 3 rows of 8728 x 680 37.2 / 17.0, 2 in each of eight of 4096 x 1024
// 34.7 / 33.8, 156 in two of 1952 x 1288 15.5 / 17.9, 3 of 680 x 8728 10.2 / 16.7.
cudaError_t launch_grouped_backward(uint16_t* dx, uint16_t* dw, const uint16_t* dout, const uint16_t* x,
                                    const uint16_t* w, const int* offsets, int64_t G, int64_t M, int64_t N, int64_t K,
                                    bool accumulate, cudaStream_t s) {
  if (M == 0) return accumulate ? cudaSuccess : cudaMemsetAsync(dw, 0, size_t(G) * size_t(N) * size_t(K) * 2, s);
  const int64_t few = dx != nullptr ? few_rows_grouped_cycles(G, M, K, N, false) : -1;
  const int64_t units = G * ceil_div(N, 256) * ceil_div(K, 256), pairs = kNumSMsHint / 2;
  if (few >= 0 && few + 7000 + (units + pairs - 1) / pairs * 3400 < int64_t(ceil_div(N, 64)) * 480) {
    const cudaError_t e = launch_few_rows_grouped_dx(dx, dout, w, offsets, G, M, N, K, s);
    return e != cudaSuccess ? e : backward(nullptr, dw, dout, x, w, offsets, G, M, N, K, accumulate, true, s);
  }
  return backward(dx, dw, dout, x, w, offsets, G, M, N, K, accumulate, false, s);
}

cudaError_t grouped_take_status(unsigned int* status) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_status, sizeof(v));
  if (e != cudaSuccess) return e;
  if (v != 0) e = cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
  *status = v;
  return e;
}

}  // namespace qffn
