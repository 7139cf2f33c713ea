// afd_mx4_gemm.cu -- the grouped MXFP4 product on the tensor cores:
// tcgen05.mma kind::mxf4 (e2m1 x e2m1, one e8m0 scale per 32 columns of each
// operand, fp32 accumulate in TMEM).
//
//   y[r, m] = sum_k x[r, k] w[g(r), m, k]     x = code * 2^(scale - 127)
//
// A unit is 128 weight rows per SM x one token tile of one group.  The weight
// rows are the MMA's M side, the tokens its N side, so a group of few tokens
// takes a narrow instruction and not a mostly empty 128-row one.  Per 256
// columns a CTA takes 17 KB of weight (codes and scales together), the
// tokens' codes by TMA (128-byte swizzle) and their scales as the image that
// tcgen05.cp spreads over the lanes.  A group's rows start anywhere, so that
// image cannot be laid out before the groups are known: narrow, five warps
// gather it from the plain rows per stage; wide, a small kernel writes it
// beforehand (k_mx4_scale_image), or the SwiGLU product that codes the rows.
//
// Two forms.  Narrow (64 tokens, one SM): groups of few tokens, bound by the
// weights' bytes; the weight's stage is one bulk copy.  Wide (192 tokens, a
// pair of SMs, cta_group::2): two weight tiles share the token tile, each SM
// holds half of its codes and all of its scales, the leader issues for both.
// One SM per tile moves 43 KB into shared memory and 40 KB out of it per
// stage of 400 tensor cycles, over the 128 bytes a cycle shared memory has;
// the pair 31 and 28 KB.
//
// Measured (weights of 64 experts):
//   narrow, 1974 rows, 2816 x 2048 with SwiGLU: 36 us, 5.6 TB/s of what it has
//     to read (83 % of the copy rate); the weights' stream bounds it
//   wide, with its scale images, 79872 rows, 2816 x 2048 with SwiGLU: 201 us,
//     4.6 PFLOP/s; 2048 x 1408: 116 us, 4.0 PFLOP/s and 4.2 TB/s (twice the
//     bf16 rate).  The eight MMAs of a 512-column stage run for some 620 cycles,
//     77 each: 11.4 PFLOP/s on 76 pairs at 1.85 GHz, at which the two would take
//     81 and 40 us (the second's bytes 72).  A stage takes 1166 cycles over long
//     rows (K 8192 and more; 15 TB/s from L2), 1000 without loads.  Timing copies
//     of the second, when it took 119: 103 us without its epilogue, 93 without its
//     loads, 84 without either, 112 without the weights' loads alone.  It is not
//     the power: the board draws 1.37 of its 1.4 kW and reports its cap, but a
//     pass after 20 ms of rest takes as long as one of a 3 s run (118 and 122 us).
//   Not kept: asking L2 for a unit's first reads two units ahead (117 -> 128
//   us: the prefetches queue before the copies); stores that L2 evicts first
//   (no change) or plain 16-byte stores (3 us slower); a third slot of scales
//   in TMEM (2 us at best); the epilogue's next piece read from TMEM while one
//   is coded (SwiGLU 8 us slower: more instructions beside the issuer's).
//
// Warps: 0 weight copies, 1 MMA, from 2 scales, 3 or 7 token copies, 8-15
// epilogue.  All waits are bounded.
#include "afd_mx4.cuh"

#include <cudaTypedefs.h>

#include <cstdio>
#include <map>
#include <mutex>
#include <utility>

namespace {

__device__ uint32_t g_mx4_errors;  // calls without a context: waits that gave up

constexpr int BOX = 256;              // columns of one token box (128 bytes of codes)
constexpr int EPI_WARPS = 8;
constexpr int EPI_WARP0 = 8;          // a multiple of 4: a warp reads the TMEM lanes of its number mod 4
constexpr int NUM_THREADS = (EPI_WARP0 + EPI_WARPS) * 32;
// epilogue staging, two buffers per four warps, each 32 tokens x 128 output
// rows (SwiGLU: 64) of bf16 as boxes of 64 (128 bytes a token, 128-byte swizzle)
constexpr int EPI_BOX_BYTES = 32 * 128;
constexpr int EPI_BUF_BYTES = 2 * EPI_BOX_BYTES;
// lines of 8-byte words that the pair's copies take contiguous memory as: a
// weight block is 8 of 1088 bytes, a 128-column scale image 1 of 1024
constexpr int kBlkLines = 8, kImgLines = 1;
constexpr int MAX_GROUPS = 256;
// Bound of every wait, from its own start: a product may take longer than this
// as a whole, none of its waits does.
constexpr uint64_t kTimeoutNs = 2000000000ull;

// A stage's word for the MMA issuer, written by the copies' producer: bits
// 0-8 the instruction's N, 9-12 the 64-column steps, then first / last stage
// of its unit, and no more stages.  The issuer follows these words alone: it
// is the one thread of control on the tensor pipe's critical path, and
// finding its own units there cost 280 cycles a stage.
constexpr uint32_t INFO_FIRST = 1u << 13, INFO_LAST = 1u << 14, INFO_STOP = 1u << 15;

template <int BN, int CTAS>
struct Ring {
  // Columns per stage: 256 in seven stages, or 512 in three.  The wide form's
  // stages are short (four MMAs of 96 cycles per 256 columns) beside what a
  // stage costs in barriers and issue: with five of 256 columns that was 580
  // of its cycles.
  static constexpr int BK = CTAS == 2 ? 512 : 256;
  static constexpr int STAGES = CTAS == 2 ? 3 : 7;
  // A wide stage is filled, multiplied and freed in two parts of 256 columns,
  // each with barriers of its own, so that a part's copies start while the
  // other is multiplied; the issuer still goes round once per 512.
  static constexpr int PARTS = CTAS == 2 ? 2 : 1;
  static constexpr int BLKS = BK / kMx4BlkCols;          // weight blocks per stage
  static constexpr int PBLKS = BLKS / PARTS;             // and per part
  static constexpr int A_BYTES = BLKS * kMx4BlkBytes;
  // Narrow: warps that fill the token scales, a stage each in turn.  No more
  // than stages: a warp that has filled stage i waits next for the release of
  // i + SF_WARPS - STAGES, and a parity wait tells a phase from the one
  // before it only; with more warps than stages it could pass one round early.
  static constexpr int SF_WARPS = CTAS == 2 ? 0 : 5;
  static constexpr int TOKEN_WARP = CTAS == 2 ? 3 : 7;   // copies the tokens' codes
  static_assert(SF_WARPS <= STAGES && 2 + SF_WARPS <= (CTAS == 2 ? EPI_WARP0 : TOKEN_WARP), "scale warps");
  static constexpr int NB = (BN + 127) / 128;            // 128-row scale images per 128 columns
  static constexpr int B_ROWS = BN / CTAS;               // token rows whose codes a CTA holds
  static constexpr int X_BYTES = B_ROWS * (BOX / 2);     // one token box
  static constexpr int B_BYTES = BK / BOX * X_BYTES;
  static constexpr int S_BYTES = BLKS * NB * 512;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + S_BYTES;
  // TMEM columns: two accumulators, then slots of a stage's weight scales (4
  // per block) and token scales (4 NB); narrow: a slot per stage, wide: two
  // in turn, which is all that 512 columns leave room for
  static constexpr int SF_SLOTS = CTAS == 2 ? 2 : STAGES;
  static constexpr int SF_COLS = BLKS * (4 + 4 * NB);
  static constexpr int SF_BASE = 2 * BN;
  static constexpr int TMEM_COLS = SF_BASE + SF_SLOTS * SF_COLS <= 256 ? 256 : 512;
  static_assert(SF_BASE + SF_SLOTS * SF_COLS <= TMEM_COLS, "TMEM columns");
  static_assert(STAGE_BYTES % 1024 == 0 && A_BYTES % 1024 == 0, "swizzle alignment");
  struct Tail {
    uint64_t full[PARTS][STAGES];
    uint64_t empty[PARTS][STAGES];
    uint64_t sfull[PARTS][STAGES];  // wide: the part's scales are in TMEM
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
    int skip;                   // an earlier kernel of the step has failed
    uint32_t info[PARTS][STAGES];  // what the stage holds (INFO_*), for each part's readers
    int m_units;                // weight tiles (pairs of them), and (2^32 - 1) / m_units
    uint32_t m_magic;
    int tile0[MAX_GROUPS + 1];  // first unit of each group
    int row0[MAX_GROUPS];
    int rows[MAX_GROUPS];
    int nt0[MAX_GROUPS];        // wide: first token tile of each group (scale images)
    int wsum[NUM_THREADS / 32], nsum[NUM_THREADS / 32];
  };
  static constexpr size_t kEpiOffset = ((size_t)STAGES * STAGE_BYTES + sizeof(Tail) + 1023) / 1024 * 1024;
  static constexpr size_t kSmemBytes = 1024 + kEpiOffset + (size_t)(EPI_WARPS / 4) * 2 * EPI_BUF_BYTES;
  static_assert(kSmemBytes <= 232448, "over the per-CTA shared memory limit");
};

// matrix descriptors: K-major operand tiles with the 128-byte swizzle (rows
// of 128 bytes, groups of 8 rows 1024 bytes apart) and the 64-byte one (rows
// of 64 bytes, 512 apart); a scale image without swizzle (8 x 16-byte core
// matrices 128 bytes apart).  The upper word is the layout's, the lower the
// address in 16-byte units: one thread issues every MMA, so the loop only
// adds to the lower words (with whole descriptors built at each use it was
// the issuing thread that bounded the kernel: 1500 cycles a stage whatever
// the tile's width).
constexpr uint32_t kDescTokens = (1024u >> 4) | 1u << 14 | 2u << 29;
constexpr uint32_t kDescWeight = (512u >> 4) | 1u << 14 | 4u << 29;
constexpr uint32_t kDescScales = (128u >> 4) | 1u << 14;
__device__ __forceinline__ uint64_t desc(uint32_t hi, uint32_t addr16) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(addr16 | 1u << 16), "r"(hi));
  return d;
}

// kind::mxf4: A and B e2m1 (format 1), e8m0 scales (bit 23), K = 64, M = 128
// per SM; sf: the first of the two scale bytes used of each lane's four (0 or 2)
template <int CTAS>
__device__ __forceinline__ uint32_t idesc_mx4(int n, int sf) {
  return (uint32_t)sf << 4 | 1u << 7 | 1u << 10 | (uint32_t)(n >> 3) << 17 | 1u << 23 |
         (uint32_t)(CTAS * 128 >> 4) << 24 | (uint32_t)sf << 29;
}
// The issuing warp runs its loop as a whole and each of the next three is
// predicated on its elected lane: under a branch on the lane the operands
// would leave the uniform registers these instructions take them from.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(e));
  return e;
}
template <int CTAS>
__device__ __forceinline__ void mma_mx4(uint32_t elected, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if (CTAS == 2)
    asm volatile(
        "{ .reg .pred p, q; setp.ne.b32 p, %4, 0; setp.ne.b32 q, %7, 0;\n"
        "@q tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p; }"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb), "r"(elected)
        : "memory");
  else
    asm volatile(
        "{ .reg .pred p, q; setp.ne.b32 p, %4, 0; setp.ne.b32 q, %7, 0;\n"
        "@q tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p; }"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb), "r"(elected)
        : "memory");
}
// arrive on the barrier (of both CTAs of a pair) when the MMAs issued so far are done
template <int CTAS>
__device__ __forceinline__ void commit(uint32_t elected, uint32_t bar) {
  if (CTAS == 2)
    asm volatile(
        "{ .reg .pred q; setp.ne.b32 q, %1, 0;\n"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %2; }"
        ::"r"(bar), "r"(elected), "h"((uint16_t)3)
        : "memory");
  else
    asm volatile(
        "{ .reg .pred q; setp.ne.b32 q, %1, 0;\n"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(bar),
        "r"(elected)
        : "memory");
}
// 32 lanes x 16 bytes of shared memory into four TMEM columns, the same for
// each quarter of the lanes; in a pair, each CTA's shared memory at this
// address into its own TMEM
template <int CTAS>
__device__ __forceinline__ void cp_scales(uint32_t elected, uint32_t tmem, uint64_t desc) {
  if (CTAS == 2)
    asm volatile(
        "{ .reg .pred q; setp.ne.b32 q, %2, 0;\n"
        "@q tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1; }" ::"r"(tmem),
        "l"(desc), "r"(elected)
        : "memory");
  else
    asm volatile(
        "{ .reg .pred q; setp.ne.b32 q, %2, 0;\n"
        "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1; }" ::"r"(tmem),
        "l"(desc), "r"(elected)
        : "memory");
}

// arrive on this CTA's barrier
template <int CTAS>
__device__ __forceinline__ void commit_local(uint32_t elected, uint32_t bar) {
  if (CTAS == 2)
    asm volatile(
        "{ .reg .pred q; setp.ne.b32 q, %1, 0;\n"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(bar), "r"(elected)
        : "memory");
  else
    commit<1>(elected, bar);
}
// the scales of 128 columns: the weight's image, then the tokens'
template <int CTAS, int NB, int BLKS>
__device__ __forceinline__ void issue_scales(uint32_t el, int c, uint32_t sa, uint32_t ss, uint32_t sf) {
  cp_scales<CTAS>(el, sf + 4 * c, desc(kDescScales, sa + ((c * kMx4BlkBytes + kMx4BlkCodes) >> 4)));
#pragma unroll
  for (int b = 0; b < NB; b++)
    cp_scales<CTAS>(el, sf + 4 * BLKS + 4 * (c * NB + b), desc(kDescScales, ss + (c * NB + b) * 32));
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* tm, uint32_t src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(tm), "r"(src),
               "r"(c0), "r"(c1)
               : "memory");
}

// the pair (rank 0 leads)
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ int ld_cluster(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrive on the leader's barrier; one CTA: on its own.  Relaxed: it says that
// TMEM has been read (tcgen05.wait::ld has returned, the tcgen05 fence stands
// before it) and publishes no memory.
template <int CTAS>
__device__ __forceinline__ void arrive_leader(uint32_t bar) {
  if (CTAS == 2)
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(map_to_rank(bar, 0)) : "memory");
  else
    mbar_arrive(bar);
}
// a box into this CTA's shared memory, its bytes counted on the leader's barrier
__device__ __forceinline__ void tma_pair_load_2d(uint32_t dst, const CUtensorMap* tm, int c0, int c1,
                                                 uint32_t bar_cluster) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      ::"r"(dst), "l"(tm), "r"(c0), "r"(c1), "r"(bar_cluster)
      : "memory");
}

// (acquire at CTA scope: across the pair the barriers order copies, MMAs and
// TMEM reads only, never the peer's plain stores)
// (A function of its own: with the loop in every role's code the expert FFN of a
// prefill fan-in took 346 us, with the call 337.)
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
  uint32_t spins = 0;
  uint64_t start = 0;
  while (!mbar_try_wait(bar, parity)) {
    if ((++spins & 255u) == 0) {
      if (*abort_flag) return false;
      const uint64_t now = globaltimer_ns();
      if (start == 0) start = now;
      if (now - start > kTimeoutNs) {
        *abort_flag = 1;
        if (status) set_error(status, AFD_ERR_TIMEOUT); else atomicAdd(&g_mx4_errors, 1u);
        return false;
      }
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
  return mbar_try_wait(bar, parity) || wait_long(bar, parity, abort_flag, status);
}

__device__ __forceinline__ uint32_t mbar_test_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok;
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag, status));
}

// silu(g) * u = g / (1 + e^-g) * u.  The row is coded next, and a code moves by
// a whole step where the bf16 value falls on the other side of a midpoint, so
// every fp32 step is a full one: the exponential to an ulp, the quotient
// corrected by its exact remainder.  Of 23 M values 156 round to another bf16
// than their 64-bit values, as with the plain fp32 formula; with ex2.approx and
// rcp.approx alone 196, and the expert FFN of a prefill fan-in lay 2.9e-4 of
// its norm from the plain form's (now none).  15 instructions a value where
// those took 6, 6 % of that FFN's time; the division operator's own branch
// would be 50 %.  e^88 < 2^127: 1 + e stays finite for the remainder; over
// 2^126, g under -87.3, its reciprocal is zero, and so is the result.  An
// infinite g has inf - inf for a remainder; the minimum makes that a number.
__device__ __forceinline__ float swiglu_f(float g, float u) {
  const float y = 1.0f + expf(fminf(-g, 88.0f));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
  const float q = g * r;
  return fmaf(fminf(fmaf(-q, y, g), 3e38f), r, q) * u;
}

// TMEM lanes [l, l + 16) x 32 columns in the fragment layout: register 4 i
// + 2 h + j holds row lane / 4 + 8 h, column 8 i + 2 (lane % 4) + j
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// four 8 x 8 matrices of 16-bit values, transposed: lane 8 m + j gives the
// address of column j (16 bytes) of matrix m
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// the four warps of one staging buffer
__device__ __forceinline__ void group_sync(int half) {
  asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
}

// the same, and whether all of them pass ok: they leave together, so none
// waits at a later barrier for one that gave up
__device__ __forceinline__ bool group_all(int half, bool ok) {
  uint32_t r;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.b32 p, %2, 0; bar.red.and.pred q, %1, 128, p; selp.u32 %0, 1, 0, q; }"
      : "=r"(r)
      : "r"(1 + half), "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}

struct Unit {
  int group, mt, rows, n_mma, tile;
  int64_t row;  // first row of the token tile
};

// A role's walk over its units.  Consecutive units of a CTA (pair) lie one
// grid apart, so the group is found by stepping from the last one (a few shared
// loads), and by a search only over a run of empty groups.
template <int BN, int CTAS>
struct Walk {
  const Mx4GemmArgs& a;
  const typename Ring<BN, CTAS>::Tail* T;
  int ngroups, total;
  int unit, g;
  Unit t;
  __device__ __forceinline__ Walk(const Mx4GemmArgs& args, const typename Ring<BN, CTAS>::Tail* tail, int n,
                                  int tot)
      : a(args), T(tail), ngroups(n), total(tot), unit((int)blockIdx.x / CTAS), g(0) {
    decode();
  }
  __device__ __forceinline__ bool more() const { return unit < total; }
  __device__ __forceinline__ void next() {
    unit += (int)gridDim.x / CTAS;
    decode();
  }
  __device__ __forceinline__ void decode() {
    if (unit >= total) return;
#pragma unroll 1
    for (int i = 0; i < 4 && T->tile0[g + 1] <= unit; i++) g++;
    if (T->tile0[g + 1] <= unit) {
      int lo = g, hi = ngroups - 1;
      while (lo < hi) {  // last group whose first unit is <= unit (empty groups share it with the next)
        const int mid = (lo + hi + 1) >> 1;
        if (T->tile0[mid] <= unit) lo = mid; else hi = mid - 1;
      }
      g = lo;
    }
    t.group = g;
    const int u = unit - T->tile0[g], rows = T->rows[g];
    int nt;
    if (BN == 64) {  // the weights stream from HBM: a weight tile's token tiles side by side, for L2
      const int n_tiles = (rows + BN - 1) / BN;
      t.mt = n_tiles == 1 ? u : u / n_tiles;
      nt = u - t.mt * n_tiles;
    } else {         // the units running at once share token tiles
      const int m_units = T->m_units;
      nt = (int)__umulhi((uint32_t)u, T->m_magic);  // u / m_units, or one less
      if ((nt + 1) * m_units <= u) nt++;
      t.mt = u - nt * m_units;
      t.tile = T->nt0[g] + nt;
    }
    if (CTAS == 2) t.mt = 2 * t.mt + (int)cluster_rank();  // past an odd edge: computed, not stored
    t.row = (int64_t)T->row0[g] + (int64_t)nt * BN;
    t.rows = min(BN, rows - nt * BN);
    t.n_mma = CTAS == 2 ? (t.rows + 31) & ~31 : (t.rows + 15) & ~15;  // 16 of each CTA's rows
  }
};

// A lane's scale bytes of one stage: rows lane + 32 i, eight bytes each
// (columns kb * 256 ..), zero past the row's end or the last row.
template <int BN>
__device__ __forceinline__ void load_scales(const uint8_t* xs, int64_t x_rows, int pitch, int64_t row0, int kb,
                                            int lane, uint32_t (&v)[BN / 32][2]) {
  const int b0 = kb * 8;
#pragma unroll
  for (int i = 0; i < BN / 32; i++) {
    v[i][0] = v[i][1] = 0u;
    const int64_t row = row0 + lane + 32 * i;
    if (row >= x_rows) continue;
    const uint8_t* p = xs + row * pitch + b0;
    if ((pitch & 7) == 0) {
      const uint2 w = *reinterpret_cast<const uint2*>(p);
      v[i][0] = w.x;
      v[i][1] = w.y;
    } else if ((pitch & 3) == 0) {  // rows start on 4 bytes
      v[i][0] = *reinterpret_cast<const uint32_t*>(p);
      if (b0 + 4 < pitch) v[i][1] = *reinterpret_cast<const uint32_t*>(p + 4);
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++)
        if (b0 + j < pitch) v[i][j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
    }
  }
}

template <int BN, int CTAS>
__global__ void __launch_bounds__(NUM_THREADS, 1) k_mx4_gemm(const __grid_constant__ Mx4GemmArgs a) {
  using R = Ring<BN, CTAS>;
  constexpr int STAGES = R::STAGES;
  constexpr int NB = R::NB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  typename R::Tail* tail = reinterpret_cast<typename R::Tail*>(smem + (size_t)STAGES * R::STAGE_BYTES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool leader = CTAS == 1 || cluster_rank() == 0;
  int32_t* const status = a.status;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; s++) {
      for (int h = 0; h < R::PARTS; h++) {
        mbar_init(smem_u32(&tail->full[h][s]), CTAS == 2 ? 1 : 2);  // the producer (the leader's), the scale warp
        mbar_init(smem_u32(&tail->sfull[h][s]), 1);
        mbar_init(smem_u32(&tail->empty[h][s]), 1);
      }
    }
    for (int b = 0; b < 2; b++) {
      mbar_init(smem_u32(&tail->tfull[b]), 1);
      mbar_init(smem_u32(&tail->tempty[b]), CTAS * EPI_WARPS);
    }
    mbar_init(smem_u32(&tail->drain), 1);
    tail->abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    if (CTAS == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(&tail->tmem_base)),
                   "r"(R::TMEM_COLS));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(&tail->tmem_base)),
                   "r"(R::TMEM_COLS));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
  }
  // a.early: the rows alone come from the kernel before; the groups and the
  // weight are older, so this CTA's first weight copies go out while that
  // kernel's last CTAs run; the roles wait for its end before the first of their
  // own waits that depends on the rows, whose bound then counts this kernel only
  if (!a.early) {
    grid_dep_wait();
    grid_dep_launch();
  }
  if (threadIdx.x == 0) tail->skip = a.status ? read_status(a.status) : 0;
  // the groups: rows clamped to those there are, units counted
  const int ngroups = a.n_groups;
  int mine = 0, tiles = 0;
  if (threadIdx.x < ngroups) {
    const int g = threadIdx.x;
    const int lo = (int)min(max((int64_t)a.offsets[g], (int64_t)0), a.x_rows);
    const int hi = (int)min(max((int64_t)a.offsets[g + 1], (int64_t)lo), a.x_rows);
    tail->row0[g] = lo;
    tail->rows[g] = hi - lo;
    tiles = (hi - lo + BN - 1) / BN;
    mine = tiles * ((mx4_tiles(a.M, a.swiglu) + CTAS - 1) / CTAS);
  }
  int incl = mine, tincl = tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o), w = __shfl_up_sync(0xffffffffu, tincl, o);
    if (lane >= o) {
      incl += v;
      tincl += w;
    }
  }
  if (lane == 31) {
    tail->wsum[warp] = incl;
    tail->nsum[warp] = tincl;
  }
  __syncthreads();
  int before = 0, total = 0, tbefore = 0;
  for (int w = 0; w < NUM_THREADS / 32; w++) {
    if (w < warp) {
      before += tail->wsum[w];
      tbefore += tail->nsum[w];
    }
    total += tail->wsum[w];
  }
  if (threadIdx.x < ngroups) {
    tail->tile0[threadIdx.x + 1] = before + incl;
    tail->nt0[threadIdx.x] = tbefore + tincl - tiles;
  }
  if (threadIdx.x == 0) {
    tail->tile0[0] = 0;
    const int m = (mx4_tiles(a.M, a.swiglu) + CTAS - 1) / CTAS;
    tail->m_units = m;
    tail->m_magic = 0xffffffffu / (uint32_t)m;  // under 2^32 / m by at most 1: u m_magic / 2^32 > u / m - 1
  }
  tc_fence_before();
  __syncthreads();
  if (CTAS == 2) cluster_sync();  // both CTAs' barriers and TMEM columns are in place
  tc_fence_after();
  // A step that has failed has no rows, and perhaps no layer: no units.  The
  // pair decides together (each CTA's smem stays until the last cluster barrier).
  if (tail->skip || (CTAS == 2 && a.status && ld_cluster(map_to_rank(smem_u32(&tail->skip), cluster_rank() ^ 1u)))) total = 0;
  const uint32_t tmem = tail->tmem_base;
  volatile int* abort_flag = &tail->abort_flag;
  // the weight: the launch's own, or that of the layer the device chose for this step
  const DevMx4Weight* lw = a.layers && total > 0 ? &a.layers[a.item->layer].mx4[a.wsel] : nullptr;
  const CUtensorMap* tmW = lw ? lw->tm : a.tmW;
  const uint8_t* wbase = lw ? lw->packed : a.w;
  const uint32_t smem_base = smem_u32(smem);

  if (warp == 0 || warp == R::TOKEN_WARP) {
    if (lane == 0) {
      // ------------------------------ copies: warp 0 the weight's, another the
      // tokens' (one thread issuing them all was on the wide ring's path, and
      // the weight's need not wait where the rows must)
      const bool weights = warp == 0, tokens = !weights;
      if (tokens && a.early) grid_dep_wait();
      int s = 0, filled = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (Walk<BN, CTAS> w(a, tail, ngroups, total); w.more() && ok; w.next()) {
        const Unit& t = w.t;
        const int nk = mx4_kblocks(a.K);
        const int m_tiles = mx4_tiles(a.M, a.swiglu);
        const int64_t blk0 =  // the weight's blocks of this tile (past an odd edge: the last tile's again)
            ((int64_t)t.group * m_tiles + min(t.mt, m_tiles - 1)) * nk;
        for (int kb = 0; kb * R::BLKS < nk && ok; kb++) {
          // the ring is full of weights: what empties it follows the kernel before
          if (weights && a.early && filled++ == STAGES) grid_dep_wait();
#pragma unroll
          for (int h = 0; h < R::PARTS; h++) {
            ok = ok && wait_bar(smem_u32(&tail->empty[h][s]), ph ^ 1, abort_flag, status);
            if (!ok) break;
            const uint32_t full = smem_u32(&tail->full[h][s]);
            const int b0 = R::BLKS * kb + R::PBLKS * h;            // the part's first block
            const int blks = max(0, min(R::PBLKS, nk - b0));       // (a part may have none)
            const uint32_t sa = smem_base + s * R::STAGE_BYTES + h * R::PBLKS * kMx4BlkBytes;
            const uint32_t sx = smem_base + s * R::STAGE_BYTES + R::A_BYTES + h * R::X_BYTES;
            if (weights && leader) {
              const int left = (a.K - kb * R::BK + 63) / 64;
              tail->info[h][s] = (uint32_t)t.n_mma | (uint32_t)min(left, R::BK / 64) << 9 |
                                 (kb == 0 ? INFO_FIRST : 0u) | (left <= R::BK / 64 ? INFO_LAST : 0u);
              mbar_expect_tx(full, blks ? CTAS * (blks * kMx4BlkBytes + R::X_BYTES + (CTAS == 2 ? R::S_BYTES / 2 : 0)) : 0);
            }
            if (CTAS == 2) {
              const uint32_t full_leader = map_to_rank(full, 0);
              const int line = (int)(blk0 + b0) * kBlkLines;
              if (weights && blks)
                tma_pair_load_2d(sa, tmW + (blks == R::PBLKS ? 0 : 1), 0, line, full_leader);
              if (tokens && blks) {  // (past a lone block: zeros, and the next tile's images; neither is used)
                tma_pair_load_2d(sx, &a.tmX, b0 * (kMx4BlkCols / 2), (int)t.row + (leader ? 0 : t.n_mma / 2), full_leader);
                tma_pair_load_2d(smem_base + s * R::STAGE_BYTES + R::A_BYTES + R::B_BYTES + h * (R::S_BYTES / 2), &a.tmS,
                                 0, (t.tile * nk + b0) * kImgLines, full_leader);
              }
            } else {
              if (weights)
                bulk_load(sa, wbase + (blk0 + b0) * kMx4BlkBytes, blks * kMx4BlkBytes, full);
              else
                tma_load_2d(sx, &a.tmX, kb * (BOX / 2), (int)t.row, full);
            }
          }
          if (++s == STAGES) { s = 0; ph ^= 1; }
        }
      }
      if (weights && a.early) grid_dep_wait();
      if (weights && leader && ok)
        for (int h = 0; h < R::PARTS; h++) {
          if (!wait_bar(smem_u32(&tail->empty[h][s]), ph ^ 1, abort_flag, status)) break;
          tail->info[h][s] = INFO_STOP;
          mbar_arrive(smem_u32(&tail->full[h][s]));
          if (CTAS == 1) mbar_arrive(smem_u32(&tail->full[h][s]));  // for the scale warp, which has no such stage
        }
      // a wait gave up: the copies in flight land before the CTA leaves
      if (!ok)
        for (int i = 0; i < 10000; i++) __nanosleep(1000);
    }
  } else if (warp == 1) {
    // ------------------------------ MMA issuer
    if (a.early) grid_dep_wait();
    if (leader) {
      const uint32_t el = elect_one();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      // Each stage's barrier is tested, and its word read, while the stage
      // before it is being issued: the two round trips to shared memory would
      // otherwise stand between the stages (about 330 of 860 cycles a stage).
      // Wide, the tests come behind a stage's MMAs, which run for longer than
      // the tests take (before them: 2 us more of 119).
      int s = 0;
      uint32_t ph = 0;
      int acc = 0, slot = 0;
      uint32_t acc_ph = 0;
      bool ready = false;
      uint32_t word = 0;
      for (;;) {
        if (!ready) {
          if (!warp_wait(smem_u32(&tail->full[0][s]), ph, abort_flag, status)) break;
          if (CTAS == 2 && !warp_wait(smem_u32(&tail->sfull[0][s]), ph, abort_flag, status)) break;
          word = *(volatile uint32_t*)&tail->info[0][s];
        }
        const uint32_t info = __shfl_sync(0xffffffffu, word, 0);
        if (info & (INFO_STOP | INFO_FIRST)) {
          if (info & INFO_STOP) break;
          if (!warp_wait(smem_u32(&tail->tempty[acc]), acc_ph ^ 1, abort_flag, status)) break;
        }
        tc_fence_after();
        const int s1 = s + 1 == STAGES ? 0 : s + 1;
        const uint32_t ph1 = s + 1 == STAGES ? ph ^ 1 : ph;
        // the next stage's barriers, tested narrow before this one is issued, wide after
        auto look = [&]() {
          return mbar_test_wait(smem_u32(&tail->full[0][s1]), ph1) &
                 (CTAS == 2 ? mbar_test_wait(smem_u32(&tail->sfull[0][s1]), ph1) : 1u);
        };
        uint32_t test = 0;
        if (CTAS == 1) test = look();
        auto next_word = [&]() { word = *(volatile uint32_t*)&tail->info[0][s1]; };  // used when ready only
        const uint32_t id0 = idesc_mx4<CTAS>((int)(info & 511u), 0), id2 = id0 | idesc_mx4<CTAS>(0, 2);
        const uint32_t d = tm + (uint32_t)(acc * BN);
        const uint32_t sa = (smem_base + s * R::STAGE_BYTES) >> 4;
        const uint32_t sb = sa + (R::A_BYTES >> 4), ss = sb + (R::B_BYTES >> 4);
        const uint32_t sf = tm + (uint32_t)(R::SF_BASE + slot * R::SF_COLS);
        const int steps = (int)(info >> 9) & 15;
        const uint32_t more = (info & INFO_FIRST) ? 0u : 1u;
        auto scales = [&](int c) {  // of 128 columns (wide: the scale warp's part)
          if (CTAS == 1) issue_scales<CTAS, NB, R::BLKS>(el, c, sa, ss, sf);
        };
        auto mma = [&](int kk) {    // of 64 columns
          const int c = kk >> 1, o = kk & 1;
          mma_mx4<CTAS>(el, d, desc(kDescWeight, sa + ((c * kMx4BlkBytes + o * 32) >> 4)),
                        desc(kDescTokens, sb + (kk >> 2) * (R::X_BYTES >> 4) + (kk & 3) * 2), o ? id2 : id0, sf + 4 * c,
                        sf + 4 * R::BLKS + 4 * c * NB, kk > 0 ? 1u : more);
        };
        // wide: the first part is done with when these MMAs are; on to the second
        auto half_way = [&]() {
          if (CTAS == 1) return true;
          commit<CTAS>(el, smem_u32(&tail->empty[0][s]));
          const uint32_t test_half = mbar_test_wait(smem_u32(&tail->full[R::PARTS - 1][s]), ph) &
                                     mbar_test_wait(smem_u32(&tail->sfull[R::PARTS - 1][s]), ph);
          if (!__all_sync(0xffffffffu, test_half != 0) &&
              (!warp_wait(smem_u32(&tail->full[R::PARTS - 1][s]), ph, abort_flag, status) ||
               !warp_wait(smem_u32(&tail->sfull[R::PARTS - 1][s]), ph, abort_flag, status)))
            return false;
          tc_fence_after();
          return true;
        };
        constexpr int FULL = R::BK / 64;
        if (steps == FULL) {  // few branches between the instructions of a whole stage
#pragma unroll
          for (int c = 0; c < R::BLKS; c++) scales(c);
          if (CTAS == 1) ready = __all_sync(0xffffffffu, test != 0);
#pragma unroll
          for (int kk = 0; kk < FULL / 2; kk++) mma(kk);
          if (CTAS == 1) next_word();
          if (!half_way()) break;
#pragma unroll
          for (int kk = FULL / 2; kk < FULL; kk++) mma(kk);
        } else {              // the unit's last columns
#pragma unroll
          for (int c = 0; c < R::BLKS; c++)
            if (2 * c < steps) scales(c);
          if (CTAS == 1) {
            ready = __all_sync(0xffffffffu, test != 0);
            next_word();
          }
#pragma unroll
          for (int kk = 0; kk < FULL / 2; kk++)
            if (kk < steps) mma(kk);
          if (!half_way()) break;
#pragma unroll
          for (int kk = FULL / 2; kk < FULL - 1; kk++)
            if (kk < steps) mma(kk);
        }
        if (++slot == R::SF_SLOTS) slot = 0;
        commit<CTAS>(el, smem_u32(&tail->empty[R::PARTS - 1][s]));
        if (CTAS == 2) {
          ready = __all_sync(0xffffffffu, look() != 0);
          next_word();
        }
        s = s1;
        ph = ph1;
        if (info & INFO_LAST) {
          commit<CTAS>(el, smem_u32(&tail->tfull[acc]));
          if (++acc == 2) { acc = 0; acc_ph ^= 1; }
        }
      }
      // every issued MMA completes before TMEM is released
      commit_local<CTAS>(el, smem_u32(&tail->drain));
      const uint64_t dl = globaltimer_ns() + 100000000ull;
      while (!mbar_try_wait(smem_u32(&tail->drain), 0) && globaltimer_ns() < dl) {}
      __syncwarp();
    }
  } else if (CTAS == 2 && (warp == 2 || warp == 4)) {
    // ------------------------------ wide: scales into TMEM
    // Warps of their own issue them, half of a stage's each: six copies and four MMAs a stage from
    // one warp took longer to issue than the MMAs take to run.
    if (a.early) grid_dep_wait();
    if (leader) {
      const uint32_t el = elect_one();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const int h = warp == 2 ? 0 : R::PARTS - 1;
      int s = 0, n = 0;
      uint32_t ph = 0;
      for (;; n++) {
        if (!warp_wait(smem_u32(&tail->full[h][s]), ph, abort_flag, status)) break;
        const uint32_t info = __shfl_sync(0xffffffffu, *(volatile uint32_t*)&tail->info[h][s], 0);
        if (info & INFO_STOP) {
          if (lane == 0) mbar_arrive(smem_u32(&tail->sfull[h][s]));
          break;
        }
        tc_fence_after();
        const uint32_t sa = (smem_base + s * R::STAGE_BYTES) >> 4;
        const uint32_t ss = sa + ((R::A_BYTES + R::B_BYTES) >> 4);
        const uint32_t sf = tm + (uint32_t)(R::SF_BASE + (n % R::SF_SLOTS) * R::SF_COLS);
        if (n >= R::SF_SLOTS) {  // this part of the slot's last stage has been multiplied
          const int m = n - R::SF_SLOTS;
          if (!warp_wait(smem_u32(&tail->empty[h][m % STAGES]), (uint32_t)(m / STAGES) & 1u, abort_flag, status))
            break;
          tc_fence_after();
        }
        const int steps = (int)(info >> 9) & 15;
#pragma unroll
        for (int i = 0; i < R::PBLKS; i++) {
          const int c = h * R::PBLKS + i;
          if (2 * c < steps) issue_scales<CTAS, NB, R::BLKS>(el, c, sa, ss, sf);
        }
        commit_local<CTAS>(el, smem_u32(&tail->sfull[h][s]));
        if (++s == STAGES) { s = 0; ph ^= 1; }
      }
    }
    __syncwarp();
  } else if (CTAS == 1 && warp < 2 + R::SF_WARPS) {
    // ------------------------------ narrow: token scales, the warps take stages in turn
    if (a.early) grid_dep_wait();
    Walk<BN, CTAS> w(a, tail, ngroups, total);
    int kb = 0;
    auto advance = [&](int n) {  // n stages on
      kb += n;
      while (w.more()) {
        const int nkb = (a.K + R::BK - 1) / R::BK;
        if (kb < nkb) break;
        kb -= nkb;
        w.next();
      }
    };
    auto load = [&](uint32_t (&v)[BN / 32][2]) {
      if (w.more())
        load_scales<BN>(a.xs, a.x_rows, a.K / 32, w.t.row, kb, lane, v);
    };
    advance(warp - 2);
    uint32_t v[BN / 32][2];
    load(v);
    int it = warp - 2;
    while (w.more()) {
      const int s = it % STAGES;
      const uint32_t ph = (uint32_t)(it / STAGES) & 1u;
      bool ok = wait_bar(smem_u32(&tail->empty[0][s]), ph ^ 1, abort_flag, status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      uint8_t* ss = smem + (size_t)s * R::STAGE_BYTES + R::A_BYTES + R::B_BYTES;
#pragma unroll
      for (int c = 0; c < 2; c++)
#pragma unroll
        for (int b = 0; b < NB; b++) {
          uint32_t q[4];
#pragma unroll
          for (int j = 0; j < 4; j++) q[j] = 4 * b + j < BN / 32 ? v[4 * b + j < BN / 32 ? 4 * b + j : 0][c] : 0u;
          *reinterpret_cast<uint4*>(ss + (c * NB + b) * 512 + lane * 16) = make_uint4(q[0], q[1], q[2], q[3]);
        }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive_leader<CTAS>(smem_u32(&tail->full[0][s]));
      advance(R::SF_WARPS);
      load(v);
      it += R::SF_WARPS;
    }
  } else if (warp >= EPI_WARP0) {
    // ------------------------------ epilogue
    // Two groups of four warps take 32 token columns at a time in turn; a
    // warp reads its 32 TMEM lanes in the fragment layout, so that stmatrix
    // writes tokens as rows (a 32 x 32 piece in 4 instructions, where 2-byte
    // stores from the lane-per-row layout took 32) and, with SwiGLU, a
    // thread holds the gate and the up value of one output.  Whole pieces
    // leave shared memory by TMA, the last rows of a group by plain stores
    // (a box would run into the next group's rows).  Two buffers in turn, so
    // one barrier a piece: it says that this buffer is full and the other
    // one has been read.  Plain stores throughout made the epilogue, at 1750
    // cycles a piece, what bounded the wide form.
    if (a.early) grid_dep_wait();
    const int q = warp & 3;
    const int half = (warp - EPI_WARP0) >> 2;
    const int gt = threadIdx.x & 127;  // thread of the group
    uint8_t* ebase = smem + R::kEpiOffset + (size_t)half * 2 * EPI_BUF_BYTES;
    const int64_t shift = a.out_shift ? (int64_t)*a.out_shift : 0;
    int buf = 0;
    int acc = 0;
    uint32_t acc_ph = 0;
    for (Walk<BN, CTAS> w(a, tail, ngroups, total); w.more(); w.next()) {
      const Unit& t = w.t;
      bool ok = wait_bar(smem_u32(&tail->tfull[acc]), acc_ph, abort_flag, status);
      if (!group_all(half, ok)) break;
      tc_fence_after();
      const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN);
      const int64_t ldo = a.ldo, row0 = t.row - shift;  // first output row
      const int fmt = a.fmt;
      bool released = false;
      const int nstore = !a.dbg || dbg_in_range(a.dbg, status, AFD_DBG_GEMM_OUT, row0 + t.rows - 1, a.out_rows) ? t.rows : 0;
      // the group's piece is in the buffer: whole ones go out by TMA
      auto stored = [&](bool whole, int boxes, int col, int64_t row) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        if (gt == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the other buffer has been read
        group_sync(half);
        if (whole && gt == 0) {
          const uint32_t src = smem_u32(ebase + (buf ^ 1) * EPI_BUF_BYTES);
          const int cols = a.swiglu ? a.M / 2 : a.M;
          for (int b = 0; b < boxes; b++)
            if (col + 64 * b < cols) tma_store_2d(&a.tmO, src + b * EPI_BOX_BYTES, col + 64 * b, (int)row);
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
      };
      auto release = [&]() {  // this warp has read the accumulator
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_leader<CTAS>(smem_u32(&tail->tempty[acc]));
        released = true;
      };
      for (int c0 = half * 32; c0 < nstore; c0 += 64) {
        const bool last = c0 + 64 >= t.rows;
        const int nrows = min(32, t.rows - c0);
        if (!a.swiglu && fmt != OUT_ACT) {  // lane = output row: 32 neighbours per token already
          uint32_t v[32];
          tmem_ld_32x32b_x32(taddr + (uint32_t)c0, v);
          tmem_ld_wait();
          if (last) release();
          const int col = t.mt * 128 + q * 32 + lane;
          if (col < a.M) {
            const int64_t at = (row0 + c0) * ldo + col;
            if (fmt == OUT_F32) {
              float* dst = reinterpret_cast<float*>(a.out) + at;
#pragma unroll
              for (int c = 0; c < 32; c++)
                if (c < nrows) dst[(int64_t)c * ldo] = __uint_as_float(v[c]);
            } else {
              uint16_t* dh = reinterpret_cast<uint16_t*>(a.out) + at;
              uint8_t* dl = a.out_lo + at;
#pragma unroll
              for (int c = 0; c < 32; c++)
                if (c < nrows) {
                  const uint32_t b24 = y24_encode(__uint_as_float(v[c]));
                  dh[(int64_t)c * ldo] = (uint16_t)(b24 >> 8);
                  dl[(int64_t)c * ldo] = (uint8_t)(b24 & 0xffu);
                }
            }
          }
          continue;
        }
        uint8_t* ebuf = ebase + buf * EPI_BUF_BYTES;
        buf ^= 1;
        uint32_t x[16], y[16];  // output rows 0..15 and 16..31 (SwiGLU: gate, up)
        tmem_ld_16x256b_x4(taddr + (uint32_t)c0, x);
        tmem_ld_16x256b_x4(taddr + (16u << 16) + (uint32_t)c0, y);
        tmem_ld_wait();
        if (last) release();
        if (a.swiglu) {
          uint32_t h[8];
#pragma unroll
          for (int i = 0; i < 8; i++) {
            const float g0 = __uint_as_float(x[2 * i]), g1 = __uint_as_float(x[2 * i + 1]);
            h[i] = pack_bf16(swiglu_f(g0, __uint_as_float(y[2 * i])), swiglu_f(g1, __uint_as_float(y[2 * i + 1])));
          }
          const uint32_t at = smem_u32(ebuf) + (8 * (lane >> 4) + (lane & 7)) * 128 +
                              (((q * 2 + ((lane >> 3) & 1)) ^ (lane & 7)) << 4);
          stmatrix_x4_trans(at, h[0], h[1], h[2], h[3]);
          stmatrix_x4_trans(at + 16 * 128, h[4], h[5], h[6], h[7]);
          stored(nrows == 32 && fmt == OUT_ACT, 1, t.mt * 64, row0 + c0);
          const int I = a.M / 2;
          if (fmt == OUT_MX4) {
            // a thread codes 16 of a token's 64 features, two threads a block
            const int r = gt >> 2, f = t.mt * 64 + (gt & 3) * 16;
            const uint8_t* src = ebuf + r * 128;
            const uint4 lo = *reinterpret_cast<const uint4*>(src + (((gt & 3) * 2 ^ (r & 7)) << 4));
            const uint4 hi = *reinterpret_cast<const uint4*>(src + ((((gt & 3) * 2 + 1) ^ (r & 7)) << 4));
            const uint32_t hw[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; i++) m = __vmaxu2(m, hw[i] & 0x7fff7fffu);
            m = max(m << 16, m & 0x7fff0000u);
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            const uint32_t sc = mx4_scale_byte(m, 0);
            const float inv = mx4_inv_scale(sc);
            uint32_t code[2];
#pragma unroll
            for (int i = 0; i < 2; i++) {
              float v[8];
#pragma unroll
              for (int j = 0; j < 4; j++) {
                v[2 * j] = __uint_as_float(hw[4 * i + j] << 16) * inv;
                v[2 * j + 1] = __uint_as_float(hw[4 * i + j] & 0xffff0000u) * inv;
              }
              code[i] = sc == 255u ? 0u : mx4_encode8(v);
            }
            if (r < nrows && f < I) {
              const uint64_t at = (uint64_t)(row0 + c0 + r) * (uint32_t)ldo + (uint32_t)f;
              *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(a.out) + (at >> 1)) =
                  make_uint2(code[0], code[1]);
              if (CTAS == 1 && (gt & 1) == 0) a.out_lo[at >> 5] = (uint8_t)sc;
            }
            if (CTAS == 2 && (gt & 1) == 0 && r < nrows && t.tile < a.tiles) {
              // into the next product's scale images; zeros past inter's
              // end, so that no stray scale meets the zero columns there
              const int blk = f >> 5, nk2 = mx4_kblocks(I), rt = c0 + r;
              uint8_t* img = a.out_lo + (uint64_t)(uint32_t)(t.tile * nk2) * (NB * 512) +
                             (uint32_t)((rt >> 7) * 512 + (rt & 31) * 16 + ((rt >> 5) & 3) * 4);
              auto put = [&](int b, uint32_t v) {
                if (b < nk2 * 4) img[(uint32_t)((b >> 2) * (NB * 512) + (b & 3))] = (uint8_t)v;
              };
              put(blk, f < I ? sc : 0u);
              if (t.mt == mx4_tiles(a.M, 1) - 1) put(blk + 2, 0u);
            }
          } else if (nrows < 32) {
            const int r0 = gt >> 3, f = t.mt * 64 + (gt & 7) * 8;
#pragma unroll
            for (int p = 0; p < 2; p++) {
              const int r = r0 + 16 * p;
              if (r < nrows && f + 8 <= I)
                *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + (row0 + c0 + r) * ldo + f) =
                    *reinterpret_cast<const uint4*>(ebuf + r * 128 + (((gt & 7) ^ (r & 7)) << 4));
            }
          }
        } else {
          const uint32_t at =
              smem_u32(ebuf) + (q >> 1) * EPI_BOX_BYTES + (lane & 7) * 128 + ((((q & 1) * 4 + (lane >> 3)) ^ (lane & 7)) << 4);
#pragma unroll
          for (int i = 0; i < 4; i++)
            stmatrix_x4_trans(at + 8 * i * 128,
                              pack_bf16(__uint_as_float(x[4 * i]), __uint_as_float(x[4 * i + 1])),
                              pack_bf16(__uint_as_float(x[4 * i + 2]), __uint_as_float(x[4 * i + 3])),
                              pack_bf16(__uint_as_float(y[4 * i]), __uint_as_float(y[4 * i + 1])),
                              pack_bf16(__uint_as_float(y[4 * i + 2]), __uint_as_float(y[4 * i + 3])));
          stored(nrows == 32, 2, t.mt * 128, row0 + c0);
          if (nrows < 32) {
            const int r0 = gt >> 4, col = t.mt * 128 + (gt & 15) * 8;
#pragma unroll
            for (int p = 0; p < 4; p++) {
              const int r = r0 + 8 * p;
              if (r < nrows && col + 8 <= a.M)
                *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + (row0 + c0 + r) * ldo + col) =
                    *reinterpret_cast<const uint4*>(ebuf + ((gt >> 3) & 1) * EPI_BOX_BYTES + r * 128 +
                                                    (((gt & 7) ^ (r & 7)) << 4));
            }
          }
        }
      }
      if (!released) release();  // no columns of this unit were this group's
      if (++acc == 2) { acc = 0; acc_ph ^= 1; }
    }
    if (gt == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // written before the CTA leaves
  }

  tc_fence_before();
  __syncthreads();
  if (CTAS == 2) cluster_sync();  // no remote arrive, copy or MMA of the pair is outstanding past this point
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    if (CTAS == 2)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(R::TMEM_COLS));
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(R::TMEM_COLS));
  }
  // a CTA without units as well: this kernel's end says that the one before has ended
  if (a.early) grid_dep_wait();
}

constexpr int kWide = 192, kNarrow = 64;

// ---------------------------------------------------------------------------
// Token scales of the wide form: the plain rows' bytes into the images
// tcgen05.cp takes, [token tile][128-column block][1024 bytes] (row r's four
// bytes at (r / 128) * 512 + (r % 32) * 16 + (r % 128 / 32) * 4), so that a
// stage's are one copy.  Gathering them inside the product kept six warps
// and a proxy fence a stage busy: 20 us of a 150 us product, where this takes
// 4.5 us (79872 rows x 1408 columns).  A token tile's columns are split over
// CTAs as long as those all run at once: with one CTA per tile a product of
// 192 rows x 8192 columns took 23.4 us, with the split 16.9.
// ---------------------------------------------------------------------------
constexpr int kImgThreads = 256, kImgDeep = 4;
struct ImageArgs {
  const uint8_t* xs;
  int64_t x_rows;
  const int32_t* offsets;
  int n_groups, pitch, nk;
  uint8_t* image;
  const int32_t* status;  // of the step, or NULL
};
__global__ void __launch_bounds__(kImgThreads) k_mx4_scale_image(const __grid_constant__ ImageArgs a) {
  __shared__ int wsum[kImgThreads / 32];
  __shared__ int64_t tile_row;
  __shared__ int tile_rows, skip;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tile = (int)blockIdx.x;
  if (threadIdx.x == 0) tile_rows = 0;
  grid_dep_wait();
  grid_dep_launch();
  if (threadIdx.x == 0) skip = a.status ? read_status(a.status) : 0;
  int64_t lo = 0, hi = 0;
  if ((int)threadIdx.x < a.n_groups) {
    lo = min(max((int64_t)a.offsets[threadIdx.x], (int64_t)0), a.x_rows);
    hi = min(max((int64_t)a.offsets[threadIdx.x + 1], lo), a.x_rows);
  }
  const int tiles = (int)((hi - lo + kWide - 1) / kWide);
  int incl = tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  if (skip) return;
  for (int w = 0; w < warp; w++) incl += wsum[w];
  if (tile < incl && tile >= incl - tiles) {
    const int nt = tile - (incl - tiles);
    tile_row = lo + (int64_t)nt * kWide;
    tile_rows = (int)min((int64_t)kWide, hi - lo - (int64_t)nt * kWide);
  }
  __syncthreads();
  const int rows = tile_rows;
  if (rows == 0) return;  // past the last tile
  const uint8_t* src = a.xs + tile_row * a.pitch;
  uint8_t* dst = a.image + (int64_t)tile * a.nk * 1024;
  // a thread: the four rows l + 32 j of one half image, 16 bytes; kImgDeep of them at once
  const int n = a.nk * 64, step = (int)gridDim.y * kImgThreads;
  for (int i0 = (int)blockIdx.y * kImgThreads + threadIdx.x; i0 < n; i0 += kImgDeep * step) {
    uint32_t q[kImgDeep][4];
#pragma unroll
    for (int u = 0; u < kImgDeep; u++) {
      const int i = i0 + u * step, l = i & 31, b = (i >> 5) & 1, c = i >> 6;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const int r = b * 128 + j * 32 + l;
        q[u][j] = 0u;
        if (i >= n || r >= rows) continue;
        const uint8_t* p = src + (int64_t)r * a.pitch + 4 * c;
        if ((a.pitch & 3) == 0) {
          q[u][j] = *reinterpret_cast<const uint32_t*>(p);
        } else {
          for (int k = 0; k < 4; k++)
            if (4 * c + k < a.pitch) q[u][j] |= (uint32_t)p[k] << (8 * k);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kImgDeep; u++) {
      const int i = i0 + u * step, l = i & 31, b = (i >> 5) & 1, c = i >> 6;
      if (i < n) *reinterpret_cast<uint4*>(dst + c * 1024 + b * 512 + l * 16) = make_uint4(q[u][0], q[u][1], q[u][2], q[u][3]);
    }
  }
}

template <int BN, int CTAS>
cudaError_t launch_variant(const LaunchCtx& lc, const Mx4GemmArgs& a, int64_t units) {
  constexpr size_t smem = Ring<BN, CTAS>::kSmemBytes;
  static std::atomic<int> attr_done[kMaxCachedDevices];
  const cudaError_t e = smem_attr_once(k_mx4_gemm<BN, CTAS>, (int)smem, attr_done);
  if (e != cudaSuccess) return e;
  if (CTAS == 2) {
    const unsigned pairs = (unsigned)std::max<int64_t>(1, std::min<int64_t>((units + 1) / 2, lc.num_sms / 2));
    return launch_k_cluster(lc, k_mx4_gemm<BN, CTAS>, 2 * pairs, NUM_THREADS, smem, 2, a);
  }
  const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(units, lc.num_sms));
  return launch_k(lc, k_mx4_gemm<BN, CTAS>, grid, NUM_THREADS, smem, a);
}

}  // namespace

// Token tile of a product over `rows` rows in `groups` groups: 64 rows when
// the groups average 48 or fewer (the weights' bytes bound it: a deeper ring
// of narrower stages), else 192 (two accumulators and the scales fill the
// 512 TMEM columns).  Narrow / wide in us, 64 groups of drawn sizes, 2816 x
// 2048 with SwiGLU: average 31 36 / 41, 48 37 / 42, 56 39 / 43, 64 46 / 43, 80
// 57 / 44; of skewed sizes (the largest five times the smallest): 48 40 /
// 42, 56 44 / 42.  At 1248 rows a group 490 / 201.  The sizes themselves are on
// the device: groups without rows count in the average, so a few large groups
// among many empty ones take the narrow form, and a step of the work-item loop
// takes the form of its context's capacity.
int mx4_token_tile(int64_t rows, int groups) { return rows <= 48 * (int64_t)groups ? kNarrow : kWide; }

cudaError_t launch_mx4_gemm(const LaunchCtx& lc, const Mx4GemmArgs& a, int bn, int64_t units) {
  return bn == kNarrow ? launch_variant<kNarrow, 1>(lc, a, units) : launch_variant<kWide, 2>(lc, a, units);
}

static int encode_box(CUtensorMap* m, CUtensorMapDataType type, int es, const void* base, int64_t row_bytes,
                      int64_t pitch, int64_t rows, int box_bytes, int box_rows, CUtensorMapSwizzle swizzle) {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  std::call_once(once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  if (!encode) return AFD_ERR_CUDA;
  const cuuint64_t dims[2] = {(cuuint64_t)(row_bytes / es), (cuuint64_t)std::max<int64_t>(rows, 1)};
  const cuuint64_t str[1] = {(cuuint64_t)pitch};
  const cuuint32_t box[2] = {(cuuint32_t)(box_bytes / es), (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = encode(m, type, 2, const_cast<void*>(base), dims, str, box, estr,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    fprintf(stderr, "afd: cuTensorMapEncodeTiled failed (%d) for MXFP4 operands\n", (int)r);
    return AFD_ERR_CUDA;
  }
  return AFD_OK;
}

// token rows: boxes of one stage's columns x the rows one CTA holds
int encode_mx4_rows(CUtensorMap* m, const void* codes, int64_t rows, int K, int bn) {
  return encode_box(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, codes, K / 2, K / 2, rows, BOX / 2, bn == kNarrow ? Ring<kNarrow, 1>::B_ROWS : Ring<kWide, 2>::B_ROWS,
                      CU_TENSOR_MAP_SWIZZLE_128B);
}
// Scale images of `rows` rows in `groups` groups over K columns (wide form;
// 0 bytes for the narrow one)
int64_t mx4_image_tiles(int64_t rows, int groups) {
  return (rows + kWide - 1) / kWide + std::min<int64_t>(groups, rows);
}
int64_t mx4_image_bytes(int64_t rows, int groups, int K) {
  return mx4_token_tile(rows, groups) == kWide ? mx4_image_tiles(rows, groups) * mx4_kblocks(K) * 1024 : 0;
}
int64_t mx4_most_image_bytes(int64_t rows, int groups, int K) {
  return mx4_image_tiles(rows, groups) * mx4_kblocks(K) * 1024;
}
int encode_mx4_images(CUtensorMap* m, const void* image, int64_t bytes) {
  return encode_box(m, CU_TENSOR_MAP_DATA_TYPE_UINT64, 8, image, 1024, 1024, bytes / 1024, 1024,
                    Ring<kWide, 2>::PBLKS, CU_TENSOR_MAP_SWIZZLE_NONE);
}
cudaError_t launch_mx4_images(const LaunchCtx& lc, const uint8_t* scales, int64_t x_rows, const int32_t* offsets,
                              int64_t rows, int groups, int K, uint8_t* image, const int32_t* status) {
  const ImageArgs a{scales, x_rows, offsets, groups, K / 32, mx4_kblocks(K), image, status};
  // a tile's columns over several CTAs while those all run at once
  const int64_t tiles = mx4_image_tiles(rows, groups), most = ((int64_t)a.nk * 64 + kImgThreads - 1) / kImgThreads;
  const int64_t split = std::min(most, std::max<int64_t>(1, 8 * (int64_t)lc.num_sms / std::max<int64_t>(1, tiles)));
  return launch_k(lc, k_mx4_scale_image, dim3((unsigned)tiles, (unsigned)split), kImgThreads, 0, a);
}
// bf16 output rows: boxes of 64 columns x 32 rows
int encode_mx4_out(CUtensorMap* m, void* out, int64_t rows, int cols, int64_t ldo) {
  return encode_box(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, out, 2 * (int64_t)cols, 2 * ldo, rows, 128, 32,
                    CU_TENSOR_MAP_SWIZZLE_128B);
}
// packed weight: boxes of a part's blocks, and of one (the pair's copies
// count on the leader's barrier, which only tensor copies can)
int encode_mx4_weight(CUtensorMap* tm, const void* packed, int64_t bytes) {
  constexpr int line = kMx4BlkBytes / kBlkLines;
  int rc = AFD_OK;
  for (int i = 0; i < 2 && !rc; i++)
    rc = encode_box(tm + i, CU_TENSOR_MAP_DATA_TYPE_UINT64, 8, packed, line, line, bytes / line, line,
                    (i ? 1 : Ring<kWide, 2>::PBLKS) * kBlkLines, CU_TENSOR_MAP_SWIZZLE_NONE);
  return rc;
}

// The errors are counted and never cleared, and a caller is told of those since
// its own last call: with one word that the first caller cleared, a product on
// another stream or thread could give up and its caller hear of nothing.
extern "C" int afd_mx4_poll_status(void* cuda_stream) {
  uint32_t n = 0;
  int dev = 0;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(cuda_stream);
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaMemcpyFromSymbolAsync(&n, g_mx4_errors, sizeof n, 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
      cudaStreamSynchronize(stream) != cudaSuccess) {
    cudaGetLastError();
    return AFD_ERR_CUDA;
  }
  bool more = n != 0;
  try {
    thread_local std::map<std::pair<int, void*>, uint32_t> told;
    uint32_t& last = told[{dev, cuda_stream}];
    more = n != last;
    last = n;
  } catch (...) {  // no memory to keep it: told again
  }
  return more ? AFD_ERR_TIMEOUT : AFD_OK;
}

#ifdef AFD_DEBUG_BOUNDS
int mx4_plant_error() {
  uint32_t n = 0;
  if (cudaDeviceSynchronize() != cudaSuccess || cudaMemcpyFromSymbol(&n, g_mx4_errors, sizeof n) != cudaSuccess ||
      cudaMemcpyToSymbol(g_mx4_errors, &(++n), sizeof n) != cudaSuccess) {
    cudaGetLastError();
    return AFD_ERR_CUDA;
  }
  return AFD_OK;
}
#endif
