// afd_lora_tiles.cu -- both products of the adapters for batches of many rows,
// of any type, alignment and rank (afd_lora_apply.cu: few rows, afd_lora_tc.cu:
// bf16 rows of whole 16 bytes, ranks of 33 to 64), 64 rows a tile:
//   u_t = w1[l] src_t,  out_t = base_t + scale[l] w2[l]^T u_t
//
// Bound by memory: src and base in, out out, at rank operations a byte.  So
// everything that comes from memory goes through one ring of shared memory
// stages filled by asynchronous copies, several stages ahead and from the
// first product's last ones straight into the second's first: a stage is 128
// bytes of each of the tile's 64 rows (of src, then of base) and the weight's
// matching columns.  The second product adds into base's stage where it lies,
// and each warp stores its 16 rows' 64 bytes whole.  Copies gather rows by
// the plan's order, so no row is moved beforehand.
//
// A cluster of C CTAs splits src's columns for the first product (the sums
// meet through distributed shared memory, in order) and out's for the second.
// The tensor cores' fp32 sums cut where they should round, so every four
// stages the sums move to registers that add with rounding.
//
// Measured (8 adapters, rank 16 and 8): 13312 rows, 2048 to 2816 columns bf16,
// 44 us, 4.7 TB/s of what they have to move (70 % of the copy rate); beside 64
// fp32 logits 17 us, 3.7 TB/s.  Between launch and first rows stand three
// dependent reads (plan, order, rows), some 3 us; with the SMs' three CTAs full
// of stages the rest runs near the copy rate.  fp32 rows take three MMAs for
// one and a split of every stage: 2000 rows of 60 logits to 1408 columns 12 us.
#include <cooperative_groups.h>

#include "afd_lora.cuh"

namespace {

namespace cg = cooperative_groups;
constexpr int TT = 64;
constexpr int kThreads = 256;
constexpr int kRowBytes = kLoraRowBytes;      // of a stage's row, of either operand
constexpr int kTileBytes = TT * kRowBytes;
constexpr int kFlush = 4;                     // stages between two moves of the sums
constexpr int kXStride = 80;                  // bytes, of a row's 32 values of one part

// stages, and CTAs an SM holds
template <int KC, int KS>
struct Form {
  static constexpr int kStages = KC == 1 ? 6 : KC == 2 ? 5 : KC == 4 ? 3 : 4;
  static constexpr int kStageBytes = kTileBytes + KC * 16 * kRowBytes;
  static constexpr int kUStride = KC * 16 + 4;
  // u's sums; its parts take their place where a warp cannot hold them
  static constexpr int KU = kLoraUParts;
  static constexpr bool kHold = KC * KU <= 8;
  // Of a row's part, its 16-byte chunks swapped as in chunk_at: padded instead,
  // ranks of 33 to 64 left two CTAs an SM (13312 rows of 2048 to 2816 fp32 outputs
  // 140 us, now 110; bf16 rows of 2049 to 2817 elements' pitch 207, now 127).
  static constexpr int kPBytes = KC * 32;
  static constexpr int kUBytes = kHold || TT * kUStride * 4 > KU * TT * kPBytes ? TT * kUStride * 4 : KU * TT * kPBytes;
  // an fp32 stage's rows as bf16 parts
  static constexpr int kXBytes = KS > 1 ? KS * TT * kXStride : 0;
  static constexpr int kBytes = kStages * kStageBytes + kUBytes + kXBytes;
  // An SM has 228 KB, of which a CTA takes 2 besides (fp32 rows: two CTAs; taken
  // for three in the clusters' size, 4000 rows of 2048 to 2816 fp32 columns took 49
  // us at rank 16 and 60 at 32, where they take 39 and 45).
  static constexpr int kCtas = KC <= 4 ? std::min(3, 228 * 1024 / (kBytes + 2048)) : 1;
};

__device__ __forceinline__ float2 lds_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds4(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void sts_f2(uint32_t addr, float x, float y) {
  asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}

// eight fp32 values, from two chunks, to their parts
template <int PARTS>
__device__ __forceinline__ void split_eight_at(uint32_t a, uint32_t b, uint4 (&to)[PARTS]) {
  uint32_t w[4][PARTS];
#pragma unroll
  for (int j = 0; j < 4; j++) split_pair<PARTS>(lds_f2((j < 2 ? a : b) + (j & 1) * 8), w[j]);
#pragma unroll
  for (int x = 0; x < PARTS; x++) to[x] = make_uint4(w[0][x], w[1][x], w[2][x], w[3][x]);
}

// A stage's rows and weights where some cannot be moved 16 bytes at a time:
// this thread's chunk of two rows and its share of the weight's.  Those that
// come through registers (bf16 rows of odd places) are all asked for before the
// first is stored.
template <int KC, typename T>
__device__ __noinline__ void slow_fill(uint32_t st, const T* row0, const T* row1, int c0, int cols, int how, const uint16_t* w,
                                       int ranks, int how_w, const void* any) {
  constexpr int E = 16 / (int)sizeof(T);  // elements of a row's chunk; chunks of a weight's row
  constexpr int kMine = (KC * 16 * E + kThreads - 1) / kThreads;
  const int tid = threadIdx.x, ch = tid & 7, r0 = tid >> 3;
  const uint32_t wst = st + kTileBytes;
  uint4 v[2], m[kMine];
  const bool bare = sizeof(T) == 2 && how == 0;  // (fp32 rows are of whole words)
  if (bare) {
    v[0] = load_words(reinterpret_cast<const uint16_t*>(row0), c0 + ch * E, row0 ? cols : 0);
    v[1] = load_words(reinterpret_cast<const uint16_t*>(row1), c0 + ch * E, row1 ? cols : 0);
  } else {
    copy_chunk<T>(chunk_at(st, r0, ch), row0, c0 + ch * E, cols, how, any);
    copy_chunk<T>(chunk_at(st, r0 + 32, ch), row1, c0 + ch * E, cols, how, any);
  }
#pragma unroll
  for (int x = 0; x < kMine; x++) {
    const int e = tid + x * kThreads, r = e / E, c = c0 + e % E * 8;
    const uint16_t* p = r < ranks ? w + (int64_t)r * cols : nullptr;
    if (how_w == 0) m[x] = load_words(p, c, p ? cols : 0);
    else if (r < KC * 16) copy_chunk<uint16_t>(chunk_at(wst, r, e % E), p, c, cols, how_w, any);
  }
  if (bare) {
    sts16(chunk_at(st, r0, ch), v[0]);
    sts16(chunk_at(st, r0 + 32, ch), v[1]);
  }
#pragma unroll
  for (int x = 0; x < kMine; x++) {
    const int e = tid + x * kThreads, r = e / E;
    if (how_w == 0 && r < KC * 16) sts16(chunk_at(wst, r, e % E), m[x]);
  }
}

// A warp's 16 rows of a block, 64 bytes each, from column `first`, where they
// cannot be stored 16 bytes at a time: neighbouring lanes neighbouring values
// (each lane its own 16 bytes' values one by one: four times the sectors, 78 us
// for 7956 rows of 1181 to 1031 columns that take 43).
template <typename TO>
__device__ __forceinline__ void slow_store(const LoraArgs& a, uint32_t st, const int32_t* rows, int first) {
  const int lane = threadIdx.x & 31, wt = threadIdx.x >> 5 & 3, half = threadIdx.x >> 7;
  if (sizeof(TO) == 4 || a.how_out) {  // two rows' 16 words at a time
    const int word = lane & 15, col = first + word * (4 / (int)sizeof(TO));
#pragma unroll
    for (int h = 0; h < 8; h++) {
      const int r = wt * 16 + 2 * h + (lane >> 4);
      const int64_t row = rows[r];
      if (row >= 0 && col < a.M)
        *reinterpret_cast<uint32_t*>(reinterpret_cast<TO*>(a.out) + row * a.ldo + col) =
            lds4(chunk_at(st, r, half * 4 + (word >> 2)) + (word & 3) * 4);
    }
  } else {  // a row's 32 values
#pragma unroll
    for (int h = 0; h < 16; h++) {
      const int r = wt * 16 + h;
      const int64_t row = rows[r];
      if (row >= 0 && first + lane < a.M)
        reinterpret_cast<uint16_t*>(a.out)[row * a.ldo + first + lane] =
            (uint16_t)(lds4(chunk_at(st, r, half * 4 + (lane >> 3)) + (lane >> 1 & 3) * 4) >> (lane & 1) * 16);
    }
  }
}

// WHOLE: all rows can be moved 16 bytes at a time, and no code for others is
// there (with two parts of u, 13312 rows of 2048 to 2816 columns 41.6 us, with
// that code 42.8; 7956 rows of 1184 to 1032 columns 18.7 and 21.4).
template <int KC, typename TS, typename TO, bool WHOLE>
__global__ void __launch_bounds__(kThreads, KC <= 4 ? 3 : 1) k_lora_tiles(const __grid_constant__ LoraArgs a) {
  constexpr int kS = LoraSrc<TS>::kParts, kU = kLoraUParts;
  typedef Form<KC, kS> F;
  constexpr int S = F::kStages;
  constexpr int KB = kRowBytes / (int)sizeof(TS), CB = kRowBytes / (int)sizeof(TO);  // columns of a stage
  constexpr int NT = CB / 16;                                                          // a warp's column tiles
  constexpr bool kHold = F::kHold;                                                     // u's operands stay in registers
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ int32_t rows[TT];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), q = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int wt = warp & 3, half = warp >> 2;  // 16 rows; first product: half of the ranks, second: of the columns
  const int4 head = *a.plan.head;
  const int64_t tile = blockIdx.x / C / 2;  // half of one of the plan's tiles
  int4 t = a.plan.tiles[tile];  // (read beside head; past its tiles there is room for more)
  if (tile >= head.x + head.y) return;
  const int skip = blockIdx.x / C % 2 * TT;
  if (t.z <= skip) return;
  t.y += skip;
  t.z -= skip;
  if (t.z > TT) t.w = 0;
  t.z = min(t.z, TT);
  if (tid < TT) rows[tid] = tid < t.z ? a.plan.order[t.y + tid] : -1;
  __syncthreads();
  if (t.x < 0) {
    copy_bare<TO>(a, rows, t.z, q * kThreads + tid, C * kThreads);
    return;
  }
  const uint32_t ring = smem_u32(smem);
  float* part = reinterpret_cast<float*>(smem + S * F::kStageBytes);  // [TT][kUStride]
  const uint32_t us = ring + S * F::kStageBytes, xs = us + F::kUBytes;
  const uint16_t* w1 = reinterpret_cast<const uint16_t*>(a.w1) + (int64_t)t.x * a.R * a.K;
  const uint16_t* w2 = reinterpret_cast<const uint16_t*>(a.w2) + (int64_t)t.x * a.R * a.M;
  const int all1 = (a.K + KB - 1) / KB, all2 = (a.M + CB - 1) / CB;
  const int k0 = all1 * q / C, n1 = all1 * (q + 1) / C - k0, m0 = all2 * q / C, n2 = all2 * (q + 1) / C - m0;
  const int n = n1 + n2;
  // This thread's chunk of rows tid / 8 and tid / 8 + 32 of a tile, and of the
  // weight's rows tid / kWc + i kWr: addresses that move on by a stage's columns.
  const int ch = tid & 7, r0 = tid >> 3;
  const bool fast1 = WHOLE || (a.how_src == 16 && a.how_w1 == 16), fast2 = WHOLE || (a.how_w2 == 16 && a.how_base == 16);
  const char *p0 = nullptr, *p1 = nullptr, *pw = nullptr;
  int left = 0, wleft = 0;  // columns from the chunk on; <= 0: none
  auto start = [&](const void* rows_at, int64_t ld, int size, int first, int cols, int chunk_cols, const uint16_t* w, int wide) {
    const char* b = reinterpret_cast<const char*>(rows_at);
    const int c0 = first * (kRowBytes / size) + ch * (16 / size);
    const int64_t row0 = rows[r0], row1 = rows[r0 + 32];
    p0 = b && row0 >= 0 ? b + (row0 * ld + c0) * size : nullptr;
    p1 = b && row1 >= 0 ? b + (row1 * ld + c0) * size : nullptr;
    left = cols - c0;
    const int wc = first * chunk_cols + tid % (chunk_cols / 8) * 8;
    pw = reinterpret_cast<const char*>(w + (int64_t)(tid / (chunk_cols / 8)) * wide + wc);
    wleft = cols - wc;
  };
  auto fill = [&](int i) {
    if (i < n) {
      const uint32_t st = ring + (i % S) * F::kStageBytes, wst = st + kTileBytes;
      if (i < n1 ? fast1 : fast2) {
        if (i == 0 && n1 > 0) start(a.src, a.lds, sizeof(TS), k0, a.K, KB, w1, a.K);
        if (i == n1) start(a.base, a.ldb, sizeof(TO), m0, a.M, CB, w2, a.M);
        copy16(chunk_at(st, r0, ch), p0 ? p0 : (const char*)a.plan.head, p0 && left > 0);
        copy16(chunk_at(st, r0 + 32, ch), p1 ? p1 : (const char*)a.plan.head, p1 && left > 0);
        if (p0) p0 += kRowBytes;
        if (p1) p1 += kRowBytes;
        const bool one = i < n1;
        const int cols = one ? KB : CB, wide = one ? a.K : a.M;
        left -= cols;
        const int per = cols / 8, wr = kThreads / per;  // chunks of a weight row; rows filled at a time
        const int r = tid / per, cc = tid % per;
#pragma unroll
        for (int x = 0; x < (KC * 16 * 8 + kThreads - 1) / kThreads; x++) {
          const int rr = r + x * wr;
          if (rr < KC * 16) {
            const bool in = rr < a.R && wleft > 0;
            copy16(chunk_at(wst, rr, cc), in ? pw + (int64_t)x * wr * wide * 2 : (const char*)a.plan.head, in);
          }
        }
        pw += cols * 2;
        wleft -= cols;
      } else {
        const int64_t row0 = rows[r0], row1 = rows[r0 + 32];
        if (i < n1) {
          const TS* p = reinterpret_cast<const TS*>(a.src);
          slow_fill<KC, TS>(st, row0 >= 0 ? p + row0 * a.lds : nullptr, row1 >= 0 ? p + row1 * a.lds : nullptr, (k0 + i) * KB, a.K,
                            a.how_src, w1, a.R, a.how_w1, a.plan.head);
        } else {
          const TO* p = reinterpret_cast<const TO*>(a.base);
          slow_fill<KC, TO>(st, p && row0 >= 0 ? p + row0 * a.ldb : nullptr, p && row1 >= 0 ? p + row1 * a.ldb : nullptr,
                            (m0 + i - n1) * CB, a.M, a.how_base, w2, a.R, a.how_w2, a.plan.head);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto ready = [&]() {  // the oldest stage is here, for all threads; the one before it is free
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
    __syncthreads();
  };
#pragma unroll
  for (int i = 0; i < S - 1; i++) fill(i);

  // ---- u: the warp's 16 rows x KC * 8 ranks ----
  float acc[KC][4], sum[KC][4];
#pragma unroll
  for (int i = 0; i < KC; i++)
#pragma unroll
    for (int x = 0; x < 4; x++) acc[i][x] = sum[i][x] = 0.0f;
  for (int i = 0; i < n1; i++) {
    ready();
    fill(i + S - 1);
    const uint32_t st = ring + (i % S) * F::kStageBytes, wst = st + kTileBytes;
    if (kS > 1) {  // the rows' parts, split once for all warps that multiply them
      const int r = tid >> 2, c8 = (tid & 3) * 8;
      uint4 v[kS];
      split_eight_at<kS>(chunk_at(st, r, c8 >> 2), chunk_at(st, r, (c8 >> 2) + 1), v);
#pragma unroll
      for (int y = 0; y < kS; y++)
        sts16(xs + (y * TT + r) * kXStride + c8 * 2, v[y]);
      __syncthreads();
    }
#pragma unroll
    for (int ks = 0; ks < KB / 16; ks++) {
      uint32_t x[kS][4];
      if (kS == 1) {
        ldsm4(chunk_at(st, wt * 16 + (lane & 15), ks * 2 + (lane >> 4)), x[0]);
      } else {
#pragma unroll
        for (int y = 0; y < kS; y++) ldsm4(xs + (y * TT + wt * 16 + (lane & 15)) * kXStride + (ks * 2 + (lane >> 4)) * 16, x[y]);
      }
      if (KC == 1) {
        uint32_t b0, b1;
        ldsm2(chunk_at(wst, half * 8 + (lane & 7), ks * 2 + ((lane >> 3) & 1)), b0, b1);
#pragma unroll
        for (int y = kS - 1; y >= 0; y--) mma_16x8x16(acc[0], x[y][0], x[y][1], x[y][2], x[y][3], b0, b1);
      } else {
#pragma unroll
        for (int j = 0; j < KC / 2; j++) {
          uint32_t b[4];
          ldsm4(chunk_at(wst, half * KC * 8 + j * 16 + (lane & 7) + ((lane >> 4) << 3), ks * 2 + ((lane >> 3) & 1)), b);
#pragma unroll
          for (int y = kS - 1; y >= 0; y--) {
            mma_16x8x16(acc[2 * j], x[y][0], x[y][1], x[y][2], x[y][3], b[0], b[1]);
            mma_16x8x16(acc[(2 * j + 1) % KC], x[y][0], x[y][1], x[y][2], x[y][3], b[2], b[3]);
          }
        }
      }
    }
    if (i % kFlush == kFlush - 1) {
#pragma unroll
      for (int j = 0; j < KC; j++)
#pragma unroll
        for (int x = 0; x < 4; x++) {
          sum[j][x] += acc[j][x];
          acc[j][x] = 0.0f;
        }
    }
  }
#pragma unroll
  for (int j = 0; j < KC; j++) {
    float* d = part + (wt * 16 + g) * F::kUStride + (half * KC + j) * 8 + 2 * c;
    *reinterpret_cast<float2*>(d) = make_float2(sum[j][0] + acc[j][0], sum[j][1] + acc[j][1]);
    *reinterpret_cast<float2*>(d + 8 * F::kUStride) = make_float2(sum[j][2] + acc[j][2], sum[j][3] + acc[j][3]);
  }
  if (C > 1) {
    // each thread the sums over the CTAs of its values, held until every CTA has read
    constexpr int kMine = TT * KC * 16 / kThreads;
    float v[kMine];
    cluster.sync();
#pragma unroll
    for (int i = 0; i < kMine; i++) {
      const int e = tid + i * kThreads, at = e / (KC * 16) * F::kUStride + e % (KC * 16);
      float w[8];  // (at most eight CTAs: all asked for, then added in order)
#pragma unroll
      for (int o = 0; o < 8; o++) w[o] = o < C ? cluster.map_shared_rank(part, o)[at] : 0.0f;
      v[i] = 0.0f;
#pragma unroll
      for (int o = 0; o < 8; o++) v[i] += w[o];
    }
    cluster.sync();
#pragma unroll
    for (int i = 0; i < kMine; i++) {
      const int e = tid + i * kThreads;
      part[e / (KC * 16) * F::kUStride + e % (KC * 16)] = v[i];
    }
  }
  __syncthreads();
  if (a.u && q == 0) {
    for (int e = tid; e < TT * KC * 16; e += kThreads) {
      const int i = e / (KC * 16), r = e % (KC * 16);
      if (i < t.z && r < a.R) a.u[(int64_t)rows[i] * a.R + r] = part[i * F::kUStride + r];
    }
  }
  if (a.u_parts || a.other_parts) {  // (rows to a whole block: zeros)
    const int64_t part_row = t.y + a.plan.shift[t.x];
    for (int e = tid + q * kThreads; e < (t.z + t.w) * KC * 8; e += C * kThreads) {
      const int i = e / (KC * 8), r = e % (KC * 8) * 2;
      const bool real = i < t.z;
      uint32_t p[3];
      if (a.u_parts) {
        split_pair<3>(real ? *reinterpret_cast<const float2*>(part + i * F::kUStride + r) : make_float2(0.0f, 0.0f), p);
#pragma unroll
        for (int x = 0; x < 3; x++) *reinterpret_cast<uint32_t*>(parts_at<KC * 16>(a.u_parts, part_row + i, x * KC * 16 + r)) = p[x];
      }
      if (a.other_parts) {
        const float* o = a.other + (int64_t)rows[real ? i : 0] * a.R + r;
        split_pair<3>(make_float2(real && r < a.R ? o[0] : 0.0f, real && r + 1 < a.R ? o[1] : 0.0f), p);
#pragma unroll
        for (int x = 0; x < 3; x++) *reinterpret_cast<uint32_t*>(parts_at<KC * 16>(a.other_parts, part_row + i, x * KC * 16 + r)) = p[x];
      }
    }
  }
  // ---- out: the warp's 16 rows x CB / 2 columns of each block ----
  const float scale = a.scale ? a.scale[t.x] : 1.0f;
  auto operand = [&](int ks, uint32_t (&p)[kU][4]) {
#pragma unroll
    for (int j = 0; j < 4; j++) {
      uint32_t w[kU];
      const float* v = part + (wt * 16 + g + (j & 1) * 8) * F::kUStride + ks * 16 + 2 * c + (j >> 1) * 8;
      split_pair<kU>(*reinterpret_cast<const float2*>(v), w);
#pragma unroll
      for (int y = 0; y < kU; y++) p[y][j] = w[y];
    }
  };
  uint32_t held[kHold ? KC : 1][kU][4];
  if (kHold) {
#pragma unroll
    for (int ks = 0; ks < KC; ks++) operand(ks, held[kHold ? ks : 0]);
  } else {  // as parts [kU][TT] of kPBytes, in the sums' place
    constexpr int kMine = TT * KC * 8 / kThreads;
    float2 v[kMine];
#pragma unroll
    for (int i = 0; i < kMine; i++) {
      const int e = tid + i * kThreads;
      v[i] = *reinterpret_cast<const float2*>(part + e / (KC * 8) * F::kUStride + e % (KC * 8) * 2);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMine; i++) {
      const int e = tid + i * kThreads;
      uint32_t p[kU];
      split_pair<kU>(v[i], p);
#pragma unroll
      for (int y = 0; y < kU; y++) {
        const int r = e / (KC * 8), col = e % (KC * 8) * 2;
        const uint32_t to = us + (y * TT + r) * F::kPBytes + (((col >> 3) ^ (r & 7)) << 4) + (col & 7) * 2;
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(p[y]) : "memory");
      }
    }
  }
  const int steps = (a.R + 15) / 16;
  // this lane's 16 bytes of rows g and g + 8 of the warp's
  TO* o[2];
#pragma unroll
  for (int h = 0; h < 2; h++) {
    const int64_t row = rows[wt * 16 + h * 8 + g];
    o[h] = row >= 0 ? reinterpret_cast<TO*>(a.out) + row * a.ldo + m0 * CB + (half * 4 + c) * (CB / 8) : nullptr;
  }
  for (int i = n1; i < n; i++) {
    ready();
    fill(i + S - 1);
    const uint32_t st = ring + (i % S) * F::kStageBytes, wst = st + kTileBytes;
    float d[NT][4];
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
      for (int x = 0; x < 4; x++) d[j][x] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < KC; ks++) {
      if (ks >= steps) break;
      if (!kHold) {
#pragma unroll
        for (int y = 0; y < kU; y++)
          ldsm4(us + (y * TT + wt * 16 + (lane & 15)) * F::kPBytes + (((ks * 2 + (lane >> 4)) ^ (lane & 7)) << 4), held[0][y]);
      }
      uint32_t(&u)[kU][4] = held[kHold ? ks : 0];
#pragma unroll
      for (int j = 0; j < NT / 2; j++) {
        uint32_t b[4];
        ldsm4t(chunk_at(wst, ks * 16 + (lane & 15), half * NT + 2 * j + (lane >> 4)), b);
#pragma unroll
        for (int y = kU - 1; y >= 0; y--) {
          mma_16x8x16(d[2 * j], u[y][0], u[y][1], u[y][2], u[y][3], b[0], b[1]);
          mma_16x8x16(d[2 * j + 1], u[y][0], u[y][1], u[y][2], u[y][3], b[2], b[3]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int r = wt * 16 + g + h * 8;
        if (sizeof(TO) == 2) {
          const uint32_t at = chunk_at(st, r, half * NT + j) + 4 * c;
          const uint32_t w = lds4(at);
          const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(w << 16) + scale * d[j][2 * h],
                                                         __uint_as_float(w & 0xffff0000u) + scale * d[j][2 * h + 1]);
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(*reinterpret_cast<const uint32_t*>(&v)) : "memory");
        } else {
          const int col = (half * NT + j) * 8 + 2 * c;
          const uint32_t at = chunk_at(st, r, col >> 2) + (col & 3) * 4;
          const float2 w = lds_f2(at);
          sts_f2(at, w.x + scale * d[j][2 * h], w.y + scale * d[j][2 * h + 1]);
        }
      }
    __syncwarp();
    const int first = (m0 + i - n1) * CB + half * (CB / 2);  // the half's first column
    if (WHOLE || a.how_out == 16) {
#pragma unroll
      for (int h = 0; h < 2; h++) {
        if (o[h] && first + c * (CB / 8) < a.M) {
          *reinterpret_cast<uint4*>(o[h]) = lds16(chunk_at(st, wt * 16 + h * 8 + g, half * 4 + c));
          o[h] += CB;
        }
      }
    } else {
      slow_store<TO>(a, st, rows, first);
    }
  }
}

template <int KC, typename TS, typename TO, bool WHOLE>
cudaError_t run(const LaunchCtx& lc, const LoraArgs& a) {
  typedef Form<KC, LoraSrc<TS>::kParts> F;
  static std::atomic<int> done[kMaxCachedDevices];
  cudaError_t e = smem_attr_once(k_lora_tiles<KC, TS, TO, WHOLE>, F::kBytes, done);
  if (e != cudaSuccess) return e;
  // As many CTAs a tile as fill the SMs; halves of tiles that hold rows, at most
  // (some of those of many adapters' last tiles do not: a third more is room).
  // Ranks over 32 have four times the sums to exchange: four CTAs at most (4399
  // rows of 1160 fp32 columns, rank 64: 68 us with four, 94 with eight).
  const int64_t tiles = 2 * a.plan.max_tiles, held = a.T / TT + std::min<int64_t>(a.T, a.L) + 1;
  unsigned C = KC >= 4 ? 4 : 8;
  while (C > 1 && held * C > kLoraSms * F::kCtas * 4 / 3) C /= 2;
  return launch_k_cluster(lc, k_lora_tiles<KC, TS, TO, WHOLE>, (unsigned)(tiles * C), kThreads, (size_t)F::kBytes, C, a);
}
template <typename TS, typename TO, bool WHOLE>
cudaError_t by_rank(const LaunchCtx& lc, const LoraArgs& a) {
  return a.R <= 16 ? run<1, TS, TO, WHOLE>(lc, a) : a.R <= 32 ? run<2, TS, TO, WHOLE>(lc, a)
       : a.R <= 64 ? run<4, TS, TO, WHOLE>(lc, a) : run<8, TS, TO, WHOLE>(lc, a);
}
template <typename TS, typename TO>
cudaError_t by_rows(const LaunchCtx& lc, const LoraArgs& a) {
  const bool whole = a.how_src == 16 && a.how_w1 == 16 && a.how_w2 == 16 && a.how_out == 16 && (!a.base || a.how_base == 16);
  return whole ? by_rank<TS, TO, true>(lc, a) : by_rank<TS, TO, false>(lc, a);
}

}  // namespace

cudaError_t launch_lora_tiles(const LaunchCtx& lc, const LoraArgs& a) {
  if (a.src_f32) return a.out_f32 ? by_rows<float, float>(lc, a) : by_rows<float, uint16_t>(lc, a);
  return a.out_f32 ? by_rows<uint16_t, float>(lc, a) : by_rows<uint16_t, uint16_t>(lc, a);
}
