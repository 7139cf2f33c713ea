// afd_lora_apply.cu -- both products of the adapters in one kernel, for batches
// of few rows (afd_lora_tiles.cu has the form for many):
//   u_t = w1[l] src_t,  out_t = base_t + scale[l] w2[l]^T u_t
// forward with (x, A, B), backward with (dy, B, A).
//
// A cluster takes a tile of up to 16 rows of one adapter, gathered by the plan's
// order.  First its warps share the columns of src in chunks of 32, each lane
// loading its operands of the tensor cores' products straight from
// global memory: the k order inside a chunk is free as long as both operands
// agree, so a lane takes 16 neighbouring bytes for its four k pairs.  The
// sums over the warps go through shared memory (65536 fp32 columns by one warp in
// one chain of MMAs left u 1440 half steps off), those over the CTAs through
// distributed shared memory, always in the same order.  Then the warps share
// the columns of out in blocks of 64.  u enters the second product as
// three bf16 parts, which keep its 24 bits.
//
// Measured (2048 to 2816 columns, rank 16): one row 4.4 us, 329 rows of 64
// adapters 8.3 us, where their bytes would take 2.2: a chain of reads that
// depend on each other (plan, order, rows and A, the CTAs' sums, B and base).
#include <cooperative_groups.h>

#include "afd_lora.cuh"

namespace {

namespace cg = cooperative_groups;
constexpr int kWarps = 8, TT = 16, kRedStride = TT + 8;
constexpr int kMove = 8;  // chunks between two moves of the sums

// eight neighbouring outputs: base + v, rounded once
template <typename TO>
__device__ __forceinline__ void add_eight(const void* base, TO* out, int c0, int n, bool vec, const float (&v)[8]) {
  if (c0 >= n) return;
  const TO* b = reinterpret_cast<const TO*>(base);
  if (vec) {
    if (sizeof(TO) == 2) {
      uint4 q = make_uint4(0u, 0u, 0u, 0u);
      if (b) q = *reinterpret_cast<const uint4*>(b + c0);
      uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const float lo = __uint_as_float(w[i] << 16) + v[2 * i], hi = __uint_as_float(w[i] & 0xffff0000u) + v[2 * i + 1];
        const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
        w[i] = *reinterpret_cast<const uint32_t*>(&r);
      }
      *reinterpret_cast<uint4*>(out + c0) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      float4 p = make_float4(0.0f, 0.0f, 0.0f, 0.0f), q = p;
      if (b) {
        p = *reinterpret_cast<const float4*>(b + c0);
        q = *reinterpret_cast<const float4*>(b + c0 + 4);
      }
      *reinterpret_cast<float4*>(out + c0) = make_float4(p.x + v[0], p.y + v[1], p.z + v[2], p.w + v[3]);
      *reinterpret_cast<float4*>(out + c0 + 4) = make_float4(q.x + v[4], q.y + v[5], q.z + v[6], q.w + v[7]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; i++) {
    if (c0 + i >= n) break;
    if (sizeof(TO) == 2) {
      const float f = (b ? __uint_as_float((uint32_t)b[c0 + i] << 16) : 0.0f) + v[i];
      out[c0 + i] = (TO)__bfloat16_as_ushort(__float2bfloat16_rn(f));
    } else {
      const float f = (b ? reinterpret_cast<const float*>(base)[c0 + i] : 0.0f) + v[i];
      reinterpret_cast<float*>(out)[c0 + i] = f;
    }
  }
}

// one value's parts, of row i among them
__device__ __forceinline__ void store_parts(uint16_t* to, int padded, int64_t i, int r, float v) {
  uint16_t p[3];
  split_bf16<3>(v, p);
#pragma unroll
  for (int x = 0; x < 3; x++)
    *(padded == 16   ? parts_at<16>(to, i, x * 16 + r)
      : padded == 32 ? parts_at<32>(to, i, x * 32 + r)
      : padded == 64 ? parts_at<64>(to, i, x * 64 + r)
                     : parts_at<128>(to, i, x * 128 + r)) = p[x];
}

template <int KC, typename TS, typename TO>
__global__ void __launch_bounds__(kWarps * 32) k_lora_apply(const __grid_constant__ LoraArgs a) {
  constexpr int kParts = LoraSrc<TS>::kParts, kU = kLoraUParts;
  constexpr int kRows = KC;                 // rank tiles of a pass
  constexpr int kCols = TT / 8;             // row tiles
  const bool vk = a.how_src == 16 && a.how_w1 == 16;
  const bool vm = a.how_w2 == 16 && a.how_out == 16 && (!a.base || a.how_base == 16);
  extern __shared__ __align__(16) uint8_t smem[];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), q = (int)cluster.block_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int4 head = *a.plan.head;
  const int64_t tile = blockIdx.x / C;
  const int4 t = a.plan.tiles[tile];  // (read beside head; past its tiles there is room for more)
  if (tile >= head.x + head.y) return;
  const int32_t* order = a.plan.order + t.y;
  if (t.x < 0) {
    copy_bare<TO>(a, order, t.z, q * kWarps * 32 + threadIdx.x, C * kWarps * 32);
    return;
  }
  const int rt = (a.R + 15) / 16, padded = lora_padded(a.R);  // rank tiles
  float* part = reinterpret_cast<float*>(smem);        // [rt * 16][TT]: this CTA's sums
  float* red = part + rt * 16 * TT;                    // [warps][kRows * 16][kRedStride]
  uint16_t* us = reinterpret_cast<uint16_t*>(red);     // [kU][TT][rt * 16 + 8], after the sums
  const int ustr = rt * 16 + 8;
  const uint16_t* w1 = reinterpret_cast<const uint16_t*>(a.w1) + (int64_t)t.x * a.R * a.K;
  const int chunks = (a.K + 31) / 32;
  const int64_t part_row = t.y + (a.u_parts || a.other_parts ? a.plan.shift[t.x] : 0);
  const TS* rows[kCols];
#pragma unroll
  for (int j = 0; j < kCols; j++) {
    const int i = j * 8 + g;
    rows[j] = i < t.z ? reinterpret_cast<const TS*>(a.src) + (int64_t)order[i] * a.lds : nullptr;
  }
  for (int r0 = 0; r0 < rt; r0 += kRows) {
    float acc[kRows][kCols][4];
#pragma unroll
    for (int i = 0; i < kRows; i++)
#pragma unroll
      for (int j = 0; j < kCols; j++)
#pragma unroll
        for (int x = 0; x < 4; x++) acc[i][j][x] = 0.0f;
    // The tensor cores' sums cut where they should round: every kMove chunks they
    // move to this warp's place in shared memory, each lane its own.
    float* mine = red + warp * kRows * 16 * kRedStride;
    bool moved = false;
    auto move = [&]() {
#pragma unroll
      for (int i = 0; i < kRows; i++)
#pragma unroll
        for (int j = 0; j < kCols; j++)
#pragma unroll
          for (int h = 0; h < 2; h++) {
            float2* d = reinterpret_cast<float2*>(mine + (i * 16 + h * 8 + g) * kRedStride + j * 8 + 2 * c);
            float2 v = make_float2(acc[i][j][2 * h], acc[i][j][2 * h + 1]);
            if (moved) v = make_float2(d->x + v.x, d->y + v.y);
            *d = v;
            acc[i][j][2 * h] = acc[i][j][2 * h + 1] = 0.0f;
          }
      moved = true;
    };
    int held = 0;
    for (int ch = q * kWarps + warp; ch < chunks; ch += C * kWarps) {
      const int k0 = ch * 32 + c * 8;
      uint4 w[kRows][2];
#pragma unroll
      for (int i = 0; i < kRows; i++)
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const int r = (r0 + i) * 16 + h * 8 + g;
          uint4 v[1];
          load_eight<uint16_t>(w1 + (int64_t)r * a.K, k0, r < a.R ? a.K : 0, vk, v);
          w[i][h] = v[0];
        }
#pragma unroll
      for (int j = 0; j < kCols; j++) {
        uint4 x[kParts];
        load_eight<TS>(rows[j], k0, rows[j] ? a.K : 0, vk, x);
#pragma unroll
        for (int p = kParts - 1; p >= 0; p--)
#pragma unroll
          for (int i = 0; i < kRows; i++) {
            mma_16x8x16(acc[i][j], w[i][0].x, w[i][1].x, w[i][0].y, w[i][1].y, x[p].x, x[p].y);
            mma_16x8x16(acc[i][j], w[i][0].z, w[i][1].z, w[i][0].w, w[i][1].w, x[p].z, x[p].w);
          }
      }
      if (++held == kMove) {
        move();
        held = 0;
      }
    }
    move();
    __syncthreads();
    for (int e = threadIdx.x; e < kRows * 16 * kCols * 8; e += kWarps * 32) {
      const int r = e / (kCols * 8), i = e % (kCols * 8);
      if (r0 + r / 16 < rt) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; w++) v += red[(w * kRows * 16 + r) * kRedStride + i];
        part[(r0 * 16 + r) * TT + i] = v;
      }
    }
    __syncthreads();
  }
  // the second product's share of this warp; its first columns' weight, which
  // does not depend on u, is asked for while the CTAs meet
  const uint16_t* w2 = reinterpret_cast<const uint16_t*>(a.w2) + (int64_t)t.x * a.R * a.M;
  const int items = (a.M + 63) / 64, all = C * kWarps;
  const int per = (items + all - 1) / all, first = (q * kWarps + warp) * per, groups = (rt + KC - 1) / KC;
  uint4 early[4][1];
  const bool ahead = KC == 1 && first < items;
  if (ahead) {
#pragma unroll
    for (int x = 0; x < 4; x++) {
      const int r = 2 * c + (x >> 1) * 8 + (x & 1);
      load_eight<uint16_t>(w2 + (int64_t)r * a.M, first * 64 + g * 8, r < a.R ? a.M : 0, vm, early[x]);
    }
    const int i = lane / 2;  // and the rows of base
    if (a.base && i < t.z)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const TO*>(a.base) + (int64_t)order[i] * a.ldb +
                                                    min(first * 64 + (lane & 1) * 32, a.M - 1)));
  }
  cluster.sync();
  for (int e = threadIdx.x; e < rt * 16 * TT; e += kWarps * 32) {
    const int r = e / TT, i = e % TT;
    float w[8], v = 0.0f;  // (at most eight CTAs: all asked for, then added in order)
#pragma unroll
    for (int o = 0; o < 8; o++) w[o] = i < t.z && o < C ? cluster.map_shared_rank(part, o)[e] : 0.0f;
#pragma unroll
    for (int o = 0; o < 8; o++) v += w[o];
    uint16_t p[kU];
    split_bf16<kU>(v, p);
#pragma unroll
    for (int x = 0; x < kU; x++) us[(x * TT + i) * ustr + r] = p[x];
    if (a.u && q == 0 && i < t.z && r < a.R) a.u[(int64_t)order[i] * a.R + r] = v;
    if (a.u_parts && q == 0 && i < t.z) store_parts(a.u_parts, padded, part_row + i, r, v);
  }
  if (q == C - 1) {  // (ranks past the last, and rows to a whole block: zeros)
    const int all = t.z + t.w, more = padded - rt * 16;
    for (int e = threadIdx.x; a.u_parts && e < all * padded; e += kWarps * 32) {
      const int r = e % padded, i = e / padded;
      if (i >= t.z || r >= padded - more) store_parts(a.u_parts, padded, part_row + i, r, 0.0f);
    }
    for (int e = threadIdx.x; a.other_parts && e < all * padded; e += kWarps * 32) {
      const int r = e % padded, i = e / padded;
      store_parts(a.other_parts, padded, part_row + i, r, r < a.R && i < t.z ? a.other[(int64_t)order[i] * a.R + r] : 0.0f);
    }
  }
  cluster.sync();  // (no CTA's sums are read after this)
  const float scale = a.scale ? a.scale[t.x] : 1.0f;
  uint32_t b[KC][8][2];
  for (int it = first; it < min(first + per, items); it++) {
    const int m0 = it * 64;
    float acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; i++)
#pragma unroll
      for (int x = 0; x < 4; x++) acc[i][x] = 0.0f;
    for (int gr = 0; gr < groups; gr++) {
#pragma unroll
      for (int kc = 0; kc < KC; kc++) {
        uint4 v[4][1];
        if (KC == 1 && it == first) {
#pragma unroll
          for (int x = 0; x < 4; x++) v[x][0] = early[x][0];
        } else {
#pragma unroll
          for (int x = 0; x < 4; x++) {
            const int r = (gr * KC + kc) * 16 + 2 * c + (x >> 1) * 8 + (x & 1);
            load_eight<uint16_t>(w2 + (int64_t)r * a.M, m0 + g * 8, r < a.R ? a.M : 0, vm, v[x]);
          }
        }
        pair_rows(v[0][0], v[1][0], v[2][0], v[3][0], b[kc]);
      }
#pragma unroll
      for (int kc = 0; kc < KC; kc++) {
        if (gr * KC + kc >= rt) break;
#pragma unroll
        for (int p = kU - 1; p >= 0; p--) {
          const uint16_t* u0 = us + (p * TT + g) * ustr + (gr * KC + kc) * 16 + 2 * c;
          const uint16_t* u1 = u0 + 8 * ustr;
          const uint32_t a0 = *reinterpret_cast<const uint32_t*>(u0), a1 = *reinterpret_cast<const uint32_t*>(u1);
          const uint32_t a2 = *reinterpret_cast<const uint32_t*>(u0 + 8), a3 = *reinterpret_cast<const uint32_t*>(u1 + 8);
#pragma unroll
          for (int i = 0; i < 8; i++) mma_16x8x16(acc[i], a0, a1, a2, a3, b[kc][i][0], b[kc][i][1]);
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const int i = g + h * 8;
      if (i >= t.z) continue;
      const int64_t row = order[i];
      const TO* br = a.base ? reinterpret_cast<const TO*>(a.base) + row * a.ldb : nullptr;
#pragma unroll
      for (int s = 0; s < 2; s++) {
        float v[8];
#pragma unroll
        for (int x = 0; x < 8; x++) v[x] = scale * acc[x][2 * h + s];
        add_eight<TO>(br, reinterpret_cast<TO*>(a.out) + row * a.ldo, m0 + c * 16 + s * 8, a.M, vm, v);
      }
    }
  }
}

template <int KC, typename TS, typename TO>
cudaError_t run(const LaunchCtx& lc, const LoraArgs& a) {
  const int rt = (a.R + 15) / 16;
  constexpr int kRed = kWarps * KC * 16 * kRedStride * 4;
  const int bytes = rt * 16 * TT * 4 + std::max(kRed, kLoraUParts * TT * (rt * 16 + 8) * 2);
  constexpr int kU = kLoraUParts * TT * (kLoraMaxRank + 8) * 2;
  static std::atomic<int> done[kMaxCachedDevices];
  cudaError_t e = smem_attr_once(k_lora_apply<KC, TS, TO>, kLoraMaxRank * TT * 4 + (kRed > kU ? kRed : kU), done);
  if (e != cudaSuccess) return e;
  const int64_t tiles = a.plan.max_tiles;
  unsigned C = 8;
  while (C > 1 && (tiles * C > 608 || (int64_t)C * kWarps > 2 * std::max((a.K + 31) / 32, (a.M + 63) / 64))) C /= 2;
  return launch_k_cluster(lc, k_lora_apply<KC, TS, TO>, (unsigned)(tiles * C), kWarps * 32, (size_t)bytes, C, a);
}
template <typename TS, typename TO>
cudaError_t by_rank(const LaunchCtx& lc, const LoraArgs& a) {
  return a.R <= 16 ? run<1, TS, TO>(lc, a) : a.R <= 32 ? run<2, TS, TO>(lc, a) : run<4, TS, TO>(lc, a);
}

}  // namespace

cudaError_t launch_lora_apply(const LaunchCtx& lc, const LoraArgs& a) {
  if (a.src_f32) return a.out_f32 ? by_rank<float, float>(lc, a) : by_rank<float, uint16_t>(lc, a);
  return a.out_f32 ? by_rank<uint16_t, float>(lc, a) : by_rank<uint16_t, uint16_t>(lc, a);
}
