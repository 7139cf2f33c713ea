// afd_lora_tc.cu -- both products of the adapters for batches of many bf16
// rows and ranks of 33 to 64, on tcgen05:
//   u_t = w1[l] src_t,  out_t = base_t + scale[l] w2[l]^T u_t
// (afd_lora_tiles.cu: the others.)
//
// Bound by memory, so one CTA an SM keeps a deep ring of stages filled and its
// warps do not wait for each other: four gather rows by the plan's order
// (asynchronous copies, a stage each in turn), one issues the MMAs, eight turn
// u into the second product's operand and add to base.  An item is a tile of
// up to 128 rows of one adapter and a share of the output columns; a stage is
// 128 bytes of each row, of src and then of base, with the weight's 64 columns,
// and the ring runs on from product to product and from item to item.  Each
// share of a tile computes u anew, from L2 but for the first one's reads, which
// costs less than meeting.
//
// u goes into the second product as three bf16 parts, all of its bits.  The sums
// of the first product move from TMEM to registers every eight stages, since
// the tensor cores' fp32 sums cut where they should round.
//
// Measured: 13312 rows of 8 adapters, 2816 to 2048 columns, rank 64, 56 us, 3.4
// TB/s of what they have to move; afd_lora_tiles.cu's takes 75.  A CTA's first
// product takes 800 cycles a stage (31 bytes a cycle), half of them waiting for
// copies; the second 1700 (with two parts of u, the third is 3 us of the whole),
// waiting for the sums of earlier blocks to be stored: base in and out out at 2.2
// TB/s each over the 110 SMs that have a tile.  Before them stand 3 us of dependent
// reads, between them 2 us in which u goes through registers (96 rows a tile
// filled all 152 SMs and gained 2 us).  Not kept, at 53 us with two parts: sixteen
// summing warps with four accumulators (no change); gathering by TMA
// (tile::gather4: 1.5 us a stage); asking L2 for whole rows ahead (12 us slower);
// each copying warp a part of every stage (0.8 us of barriers and waits for each,
// whatever the ring's depth); a warp that waits for its last stage's copies and
// then says so (55 us; each lane's arrival by its copies' end 53; six copying
// warps, not four, half a microsecond less).
//
// All waits are bounded; one that gives up is counted (afd_lora_poll_status).
#include "afd_lora.cuh"

namespace {

__device__ uint32_t g_errors;  // waits that gave up

constexpr int TT = 128;
constexpr int kSumWarps = 8, kCopyWarps = 4;
constexpr int kThreads = (kSumWarps + kCopyWarps + 1) * 32;
constexpr int kCopyRows = 4, kCopies = TT / kCopyRows;  // rows of a warp's copy, copies of a stage
constexpr int kRowsBytes = TT * kLoraRowBytes;  // a stage's rows
constexpr int kFlush = 8;                       // stages between two moves of u's sums
constexpr uint64_t kTimeoutNs = 2000000000ull;

constexpr int RP = 64, KU = kLoraUParts;  // ranks of a part, padded; parts
constexpr int kStageBytes = kRowsBytes + RP * kLoraRowBytes;
constexpr int kUBytes = KU * kRowsBytes;        // u's parts, rows of 128 bytes
constexpr int S = (224 * 1024 - kUBytes) / kStageBytes;  // stages
constexpr int kBytes = S * kStageBytes + kUBytes;
static_assert(S >= kCopyWarps, "each copying warp has a stage");

// Operands have the 128-byte swizzle: K-major (8-row groups 1024 bytes apart),
// or MN-major of one 64-element atom (8-k groups 1024 bytes apart).
// bf16 x bf16 -> fp32, M 128; mn: B MN-major
__device__ __forceinline__ constexpr uint32_t idesc(int n, bool mn) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (mn ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (128u >> 4) << 24;
}

// false: the wait, or another one of the CTA, has given up
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  const uint64_t start = globaltimer_ns();
  uint32_t spins = 0;
  while (!mbar_try_wait(bar, parity)) {
    if ((++spins & 63u) == 0) {
      if (*abort_flag) return false;
      if (globaltimer_ns() - start > kTimeoutNs) {
        *abort_flag = 1;
        return false;
      }
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return mbar_try_wait(bar, parity) || wait_long(bar, parity, abort_flag);
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag));
}

// sixteen bytes in and out of shared memory
__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void sts16(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint32_t add_pair(uint32_t base, float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(base << 16) + a, __uint_as_float(base & 0xffff0000u) + b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// eight values' first PARTS bf16 parts
template <int PARTS>
__device__ __forceinline__ void split_eight(const float* v, uint4 (&to)[PARTS]) {
  uint32_t w[PARTS][4];
#pragma unroll
  for (int j = 0; j < 4; j++) {
    uint32_t p[PARTS];
    split_pair<PARTS>(make_float2(v[2 * j], v[2 * j + 1]), p);
#pragma unroll
    for (int x = 0; x < PARTS; x++) w[x][j] = p[x];
  }
#pragma unroll
  for (int x = 0; x < PARTS; x++) to[x] = make_uint4(w[x][0], w[x][1], w[x][2], w[x][3]);
}

// sixteen bytes of which `bytes` are read and the rest zero, or nothing at all
__device__ __forceinline__ void copy16_if(bool p, uint32_t dst, const void* src, int bytes) {
  asm volatile("{ .reg .pred p; setp.ne.b32 p, %3, 0;\n@p cp.async.cg.shared.global [%0], [%1], 16, %2; }" ::"r"(dst), "l"(src),
               "r"(bytes), "r"((int)p)
               : "memory");
}

// Shares of the output's columns, for the shortest longest CTA: an item costs
// its stages, those that are also written twice.  A lane tries each number.
__device__ __forceinline__ int shares_of(int tiles, int ctas, int n1, int blocks, int lane) {
  const int s = min(lane & 7, blocks - 1) + 1;
  const uint32_t cost = (uint32_t)((tiles * s + ctas - 1) / ctas) * (n1 + 2 * ((blocks + s - 1) / s));
  return (int)(__reduce_min_sync(0xffffffffu, cost << 4 | s) & 15u);
}

__global__ void __launch_bounds__(kThreads, 1) k_lora_tc(const __grid_constant__ LoraArgs a) {
  typedef uint16_t TO;
  constexpr int kMine = RP / 2;  // ranks of a thread that sums
  extern __shared__ __align__(1024) uint8_t smem[];
  // Of each stage: full; free again after the first product, after the second.
  // u's sums: complete, taken (two in turn); its parts are there; sums of a
  // block: complete, taken (two in turn).  A warp arrives once, not its 32
  // threads, which the barrier would count one after the other.
  __shared__ uint64_t full[S], empty1[S], empty2[S], ufull[2], uempty[2], uready, dfull[2], dempty[2];
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int4 head = *a.plan.head;
  const int n1 = (a.K + 63) / 64, blocks = (a.M + 63) / 64;
  const int shares = shares_of(head.x, gridDim.x, n1, blocks, lane), items = head.x * shares;
  const uint32_t ring = smem_u32(smem), us = ring + S * kStageBytes;
  if (tid < S) {
    mbar_init(smem_u32(&full[tid]), 32);
    mbar_init(smem_u32(&empty1[tid]), 1);
    mbar_init(smem_u32(&empty2[tid]), kSumWarps / 2);
    if (tid < 2) {
      mbar_init(smem_u32(&ufull[tid]), 1);
      mbar_init(smem_u32(&uempty[tid]), kSumWarps);
      mbar_init(smem_u32(&dfull[tid]), 1);
      mbar_init(smem_u32(&dempty[tid]), kSumWarps / 2);
    }
    if (tid == 0) {
      mbar_init(smem_u32(&uready), kSumWarps);
      abort_flag = 0;
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 256;" ::"r"(smem_u32(&tmem_base)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;  // columns: u's sums twice (64 each), a block's twice (64 each)
  const bool with_base = a.base != nullptr;
  volatile int* const gave_up = &abort_flag;
  bool good = true;
  // an item's blocks of 64 columns
  auto first_block = [&](int share) { return (int)((int64_t)blocks * share / shares); };

  if (warp >= kSumWarps && warp < kSumWarps + kCopyWarps) {  // ---- copies ----
    // A warp fills every kCopyWarps-th stage: what a stage costs one warp beside
    // its copies (two barriers, the wait) then passes while others copy.
    const int ch = lane & 7, r0 = lane >> 3;  // this lane's 16 bytes of rows r0 + 4 j
    int stage = 0, slot = 0;                  // of the ring, all warps'
    // by slot: its last use was for the second product; the uses for the
    // first, for the second so far, modulo 2
    uint32_t second = 0, odd1 = 0, odd2 = 0;
    for (int item = blockIdx.x; item < items && good; item += gridDim.x) {
      const int4 t = a.plan.tiles[item / shares];
      const int share = item % shares, m0 = first_block(share), n = n1 + first_block(share + 1) - m0;
      int32_t row[kCopies];
#pragma unroll
      for (int j = 0; j < kCopies; j++) row[j] = a.plan.order[t.y + min(r0 + kCopyRows * j, t.z - 1)];
      for (int i = 0; i < n; i++, stage++, slot = slot + 1 == S ? 0 : slot + 1) {
        const bool one = i < n1, two = second >> slot & 1;
        const uint32_t bit = 1u << slot;
        if (stage % kCopyWarps == warp - kSumWarps) {
          if (stage >= S) {
            good = warp_wait(smem_u32(two ? &empty2[slot] : &empty1[slot]), ((two ? odd2 : odd1) >> slot & 1) ^ 1, gave_up);
            if (!good) break;
          }
          const uint32_t st = ring + slot * kStageBytes;
          const int col = (one ? i : m0 + i - n1) * 64 + ch * 8, cols = one ? a.K : a.M;
          const bool in = col < cols;
          const int bytes = in ? 16 : 0;
          const char* nowhere = reinterpret_cast<const char*>(a.plan.head);
          // (rows r0 + 4 j lie 512 bytes apart, their chunk in one of two places)
          const uint32_t at0 = chunk_at(st, r0, ch), at1 = chunk_at(st, r0 + 4, ch) - 512;
          if (one || with_base) {
            const char* p = in ? reinterpret_cast<const char*>(one ? a.src : a.base) + col * 2 : nowhere;
            const uint32_t pitch = in ? (uint32_t)(one ? a.lds : a.ldb) * 2 : 0u;  // (under 2^32: lora_tc_takes)
#pragma unroll
            for (int j = 0; j < kCopies; j++)  // (rows past the tile's end: what is there, not stored)
              copy16_if(r0 + kCopyRows * j < t.z, (j & 1 ? at1 : at0) + j * 512, p + (uint64_t)(uint32_t)row[j] * pitch, bytes);
          }
          const char* w = in ? reinterpret_cast<const char*>(one ? a.w1 : a.w2) + (((int64_t)t.x * a.R + r0) * cols + col) * 2 : nowhere;
          const uint32_t wpitch = in ? cols * 2 * kCopyRows : 0;
#pragma unroll
          for (int j = 0; j < RP / kCopyRows; j++) {
            const bool with = r0 + kCopyRows * j < a.R;
            copy16_if(true, (j & 1 ? at1 : at0) + kRowsBytes + j * 512, with ? w + (uint64_t)j * wpitch : nowhere, with ? bytes : 0);
          }
          // each lane arrives when its copies have landed
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&full[slot])) : "memory");
        }
        second = one ? second & ~bit : second | bit;
        if (one) odd1 ^= bit; else odd2 ^= bit;
      }
    }
    asm volatile("cp.async.commit_group;\ncp.async.wait_group 0;" ::: "memory");
  } else if (warp == kSumWarps + kCopyWarps) {  // ---- products ----
    const uint32_t el = lora_elect(), d1 = idesc(RP, false), d2 = idesc(64, true);
    const int steps = (a.R + 15) / 16;
    int slot = 0;
    uint32_t turn = 0, group = 0, block = 0, done = 0;
    // The copies' writes, seen through the barrier, before the products' reads,
    // which go another way: once a stage here, not in every warp that copies.
    auto landed = [&]() {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      tc_fence_after();
    };
    auto next = [&]() {
      if (++slot == S) {
        slot = 0;
        turn++;
      }
    };
    for (int item = blockIdx.x; item < items && good; item += gridDim.x) {
      const int share = item % shares, n2 = first_block(share + 1) - first_block(share);
      for (int i = 0; i < n1; i++) {
        good = warp_wait(smem_u32(&full[slot]), turn & 1, gave_up);
        if (good && i % kFlush == 0 && group >= 2) good = warp_wait(smem_u32(&uempty[group & 1]), (group / 2 - 1) & 1, gave_up);
        if (!good) break;
        landed();
        const uint32_t st = (ring + slot * kStageBytes) >> 4;
#pragma unroll
        for (int ks = 0; ks < 4; ks++)
          lora_mma(el, tmem + (group & 1) * 64, lora_desc(st + ks * 2, 1), lora_desc(st + (kRowsBytes >> 4) + ks * 2, 1), d1,
                   i % kFlush != 0 || ks != 0);
        lora_commit(el, smem_u32(&empty1[slot]));
        if (i % kFlush == kFlush - 1 || i == n1 - 1) lora_commit(el, smem_u32(&ufull[group++ & 1]));
        next();
      }
      if (good) good = warp_wait(smem_u32(&uready), done++ & 1, gave_up);
      for (int j = 0; j < n2 && good; j++) {
        good = warp_wait(smem_u32(&full[slot]), turn & 1, gave_up);
        if (good && block >= 2) good = warp_wait(smem_u32(&dempty[block & 1]), (block / 2 - 1) & 1, gave_up);
        if (!good) break;
        landed();
        const uint32_t w = (ring + slot * kStageBytes + kRowsBytes) >> 4;
        for (int p = KU - 1; p >= 0; p--)
          for (int ks = 0; ks < steps; ks++)
            lora_mma(el, tmem + 128 + (block & 1) * 64, lora_desc((us + p * kRowsBytes >> 4) + ks * 2, 1),
                     lora_desc(w + ks * 128, 1), d2, p != KU - 1 || ks != 0);
        lora_commit(el, smem_u32(&dfull[block++ & 1]));
        next();
      }
    }
  } else if (warp < kSumWarps) {  // ---- sums: 32 rows, of half of the ranks, of every other block ----
    const int quarter = warp & 3, half = warp >> 2, row = quarter * 32 + lane;
    const uint32_t mine = tmem + ((uint32_t)quarter << 21);
    int slot = 0;
    uint32_t turn = 0, group = 0, block = 0;
    for (int item = blockIdx.x; item < items && good; item += gridDim.x) {
      const int4 t = a.plan.tiles[item / shares];
      const int share = item % shares, m0 = first_block(share), n2 = first_block(share + 1) - m0;
      const int64_t out_row = a.plan.order[t.y + min(row, t.z - 1)];
      const float scale = a.scale ? a.scale[t.x] : 1.0f;
      const int64_t part_row = t.y + (a.u_parts || a.other_parts ? a.plan.shift[t.x] : 0);
      float u[kMine];
#pragma unroll
      for (int r = 0; r < kMine; r++) u[r] = 0.0f;
      for (int i = 0; i < n1; i += kFlush, group++) {
        good = __all_sync(0xffffffffu, wait_bar(smem_u32(&ufull[group & 1]), group / 2 & 1, gave_up));
        if (!good) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < kMine; c += 16) {
          uint32_t v[16];
          tmem_ld_16(mine + (group & 1) * 64 + half * kMine + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int r = 0; r < 16; r++) u[c + r] += __uint_as_float(v[r]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&uempty[group & 1]));
      }
      if (!good) break;
      for (int i = 0; i < n1; i++)
        if (++slot == S) {
          slot = 0;
          turn++;
        }
      const int rank0 = half * kMine;
#pragma unroll
      for (int r = 0; r < kMine; r++)
        if (rank0 + r >= a.R) u[r] = 0.0f;
#pragma unroll
      for (int c = 0; c < kMine / 8; c++) {  // eight ranks: a chunk of each part
        uint4 p[KU];
        split_eight<KU>(u + 8 * c, p);
#pragma unroll
        for (int x = 0; x < KU; x++) sts16(chunk_at(us + x * kRowsBytes, row, rank0 / 8 + c), p[x]);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&uready));
      if (share == 0 && row < t.z) {
        if (a.u) {
          float* to = a.u + out_row * a.R + rank0;
          if (a.R % 4 == 0 && reinterpret_cast<uintptr_t>(a.u) % 16 == 0) {
#pragma unroll
            for (int r = 0; r < kMine; r += 4)
              if (rank0 + r < a.R) *reinterpret_cast<float4*>(to + r) = make_float4(u[r], u[r + 1], u[r + 2], u[r + 3]);
          } else {
#pragma unroll
            for (int r = 0; r < kMine; r++)
              if (rank0 + r < a.R) to[r] = u[r];
          }
        }
#pragma unroll
        for (int c = 0; c < kMine / 8; c++) {
          uint4 p[3];
          if (a.u_parts) {
            split_eight<3>(u + 8 * c, p);
#pragma unroll
            for (int x = 0; x < 3; x++)
              *reinterpret_cast<uint4*>(parts_at<RP>(a.u_parts, part_row + row, x * RP + rank0 + c * 8)) = p[x];
          }
          if (a.other_parts) {
            const float* o = a.other + out_row * a.R;
            float v[8];
#pragma unroll
            for (int r = 0; r < 8; r++) v[r] = rank0 + c * 8 + r < a.R ? o[rank0 + c * 8 + r] : 0.0f;
            split_eight<3>(v, p);
#pragma unroll
            for (int x = 0; x < 3; x++)
              *reinterpret_cast<uint4*>(parts_at<RP>(a.other_parts, part_row + row, x * RP + rank0 + c * 8)) = p[x];
          }
        }
      }
      if (share == 0 && (a.u_parts || a.other_parts) && row < t.w) {  // to a whole block: zeros
        const uint4 none = make_uint4(0u, 0u, 0u, 0u);
        for (int c = half; c < 3 * RP / 8; c += 2) {
          if (a.u_parts) *reinterpret_cast<uint4*>(parts_at<RP>(a.u_parts, part_row + t.z + row, c * 8)) = none;
          if (a.other_parts) *reinterpret_cast<uint4*>(parts_at<RP>(a.other_parts, part_row + t.z + row, c * 8)) = none;
        }
      }
      // this lane's 16 bytes of rows 4 h + lane / 8 of the warp's, as they are stored
      TO* at[8];
#pragma unroll
      for (int h = 0; h < 8; h++) {
        const int r = quarter * 32 + h * 4 + (lane >> 3);
        const int64_t to = a.plan.order[t.y + min(r, t.z - 1)];
        at[h] = r < t.z ? reinterpret_cast<TO*>(a.out) + to * a.ldo + m0 * 64 + (lane & 7) * 8 : nullptr;
      }
      for (int j = 0; j < n2; j++, block++) {
        if ((block & 1) == half) {
          const int m = (m0 + j) * 64;
          good = warp_wait(smem_u32(&dfull[half]), block / 2 & 1, gave_up) && warp_wait(smem_u32(&full[slot]), turn & 1, gave_up);
          if (!good) break;
          tc_fence_after();
          const uint32_t st = ring + slot * kStageBytes;
#pragma unroll
          for (int h = 0; h < 2; h++) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(mine + 128 + half * 64 + h * 32, v);
            tmem_ld_wait();
            if (h == 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_u32(&dempty[half]));
            }
#pragma unroll
            for (int c = 0; c < 4; c++) {
              const uint32_t to = chunk_at(st, row, h * 4 + c);
              uint4 b = with_base ? lds16(to) : make_uint4(0u, 0u, 0u, 0u);
              b.x = add_pair(b.x, scale * __uint_as_float(v[8 * c]), scale * __uint_as_float(v[8 * c + 1]));
              b.y = add_pair(b.y, scale * __uint_as_float(v[8 * c + 2]), scale * __uint_as_float(v[8 * c + 3]));
              b.z = add_pair(b.z, scale * __uint_as_float(v[8 * c + 4]), scale * __uint_as_float(v[8 * c + 5]));
              b.w = add_pair(b.w, scale * __uint_as_float(v[8 * c + 6]), scale * __uint_as_float(v[8 * c + 7]));
              sts16(to, b);
            }
          }
          __syncwarp();
#pragma unroll
          for (int h = 0; h < 8; h++) {
            const uint4 w = lds16(chunk_at(st, quarter * 32 + h * 4 + (lane >> 3), lane & 7));
            if (at[h] && m + (lane & 7) * 8 < a.M) *reinterpret_cast<uint4*>(at[h] + j * 64) = w;
          }
          // (the slot's next copy comes after these reads and writes)
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&empty2[slot]));
        }
        if (++slot == S) {
          slot = 0;
          turn++;
        }
      }
    }
  }
  __syncthreads();
  if (tid == 0 && abort_flag) atomicAdd(&g_errors, 1u);
  tc_fence_after();
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 256;" ::"r"(tmem));
  for (int64_t i = head.w + (int64_t)blockIdx.x * 32; i < a.T; i += (int64_t)gridDim.x * 32)
    copy_bare<TO>(a, a.plan.order + i, (int)min((int64_t)32, a.T - i), tid, kThreads);
}

}  // namespace

// Ranks of 33 to 64 only.  Microseconds, this kernel / afd_lora_tiles.cu's, two
// batches in turn (so that rows come from memory): 2048 to 2816 columns, 8
// adapters, rank 64: 1100 rows 25 / 23, 4000 31 / 35, 13312 57 / 76; 300 adapters:
// 4000 31 / 61, 400: 13312 61 / 96.  Narrow: 13312 rows of 64 columns 12 / 18, of
// 512 20 / 32; 4000 of 64 to 512 12 / 15; the other way, by 1 to 2 us, up to a few
// thousand rows of some hundred columns (1100 of 256, 4000 of 128).  Rank 32, 8
// adapters: 1100 25 / 20, 4000 29 / 44, 13312 51 / 55; rank 16: 25 / 14, 29 / 35, 49 /
// 47: ranks of 17 to 32 would need their parts for the weight gradients in a layout
// of their own here, and lose their small batches.  fp32 outputs, which are logits
// of few columns, gained nothing from it either.
bool lora_tc_takes(const LoraArgs& a) {
  return !a.src_f32 && !a.out_f32 && a.R > 32 && a.R <= 64 && a.how_src == 16 && a.how_w1 == 16 && a.how_w2 == 16 &&
         a.how_out == 16 && (!a.base || a.how_base == 16) && a.lds < (int64_t(1) << 31) &&
         (!a.base || a.ldb < (int64_t(1) << 31));
}

cudaError_t launch_lora_tc(const LaunchCtx& lc, const LoraArgs& a) {
  static std::atomic<int> done[kMaxCachedDevices];
  const cudaError_t e = smem_attr_once(k_lora_tc, kBytes, done);
  if (e != cudaSuccess) return e;
  return launch_k(lc, k_lora_tc, kLoraSms, kThreads, kBytes, a);
}

cudaError_t lora_tc_error_count(uint32_t* n, cudaStream_t stream) {
  return cudaMemcpyFromSymbolAsync(n, g_errors, sizeof *n, 0, cudaMemcpyDeviceToHost, stream);
}

#ifdef AFD_DEBUG_BOUNDS
int lora_tc_plant_error() {
  uint32_t n = 0;
  if (cudaDeviceSynchronize() != cudaSuccess || cudaMemcpyFromSymbol(&n, g_errors, sizeof n) != cudaSuccess ||
      cudaMemcpyToSymbol(g_errors, &(++n), sizeof n) != cudaSuccess) {
    cudaGetLastError();
    return AFD_ERR_CUDA;
  }
  return AFD_OK;
}
#endif
