// afd_lora_wgrad.cu -- the adapters' weight gradients from fp32 rows
// (afd_lora_wgrad_tc.cu: from bf16 ones), and the sum over an adapter's pieces:
//   da[l] = scale[l] sum_t v_t x_t^T,  db[l] = scale[l] sum_t u_t dy_t^T
// over the rows t of adapter l: [rank x columns] sums of outer products.
//
// A CTA takes one piece of an adapter's rows and a slab of columns of x or dy.
// Rows stream through a ring of shared memory stages of 16, gathered by
// asynchronous copies; they and u or v are split into three bf16 parts each,
// so that the products on the tensor cores keep 24 bits.  A warp holds 16
// ranks x 16 columns: splitting takes it longer than multiplying, and gates'
// logits have few columns (60 of them, 2000 rows: 25 us with 64 a warp, 9 with 16).  The tensor cores' fp32 sums cut where they
// should round, so every other stage they move to registers that add with
// rounding.  Adapters of several pieces leave partial sums, added in order by
// a second kernel, which also clears the gradients of adapters without rows.
#include "afd_lora.cuh"

namespace {

constexpr int kRows = 16;  // of a stage
constexpr int kCols = 16, kTiles = kCols / 8;  // of a warp

// rank groups of 16 x column groups of 16: one warp each
template <int RG>
struct Wg {
  static constexpr int kCg = RG == 1 ? 8 : RG <= 4 ? 4 : 2;
  static constexpr int kThreads = RG * kCg * 32;
  static constexpr int kSlab = kCg * kCols;
  static constexpr int kStageBytes = kRows * kSlab * 4;
  static constexpr int kStages = 6;
  static constexpr int kPStride = RG * 16 + 8;                 // bf16 of a row's parts
  static constexpr int kPartBytes = 3 * kRows * kPStride * 2;  // one stage's
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kBytes = kRing + 2 * kPartBytes;
  static constexpr int kCtas = kThreads == 256 ? 3 : 1;
};

template <int RG>
__device__ __forceinline__ void store_sums(const LoraWgradArgs& a, int which, const int4& pc, int rg, int m0, int lane,
                                           const float (&sum)[kTiles][4]) {
  const int N = a.N[which], g = lane >> 2, c = lane & 3;
  const float scale = a.scale ? a.scale[pc.x] : 1.0f;
  float* out = pc.w < 0 ? a.out[which] + (int64_t)pc.x * a.R * N : a.part[which] + (int64_t)pc.w * a.R * N;
#pragma unroll
  for (int h = 0; h < 2; h++) {
    const int r = rg * 16 + h * 8 + g;
    if (r >= a.R) continue;
    float* d = out + (int64_t)r * N;
#pragma unroll
    for (int j = 0; j < kTiles; j++) {
      const int col = m0 + j * 8 + 2 * c;
      const float v0 = scale * sum[j][2 * h], v1 = scale * sum[j][2 * h + 1];
      if (N % 2 == 0) {
        if (col < N) *reinterpret_cast<float2*>(d + col) = make_float2(v0, v1);
      } else {
        if (col < N) d[col] = v0;
        if (col + 1 < N) d[col + 1] = v1;
      }
    }
  }
}

template <int RG>
__device__ __forceinline__ void wgrad(const LoraWgradArgs& a, int which, int slab, const int4& pc, uint8_t* smem,
                                      const int32_t* rows) {
  typedef Wg<RG> W;
  constexpr int kQ = LoraSrc<float>::kParts, S = W::kStages;
  constexpr int kCB = kLoraRowBytes / 4;     // columns of a 128-byte row
  constexpr int kChunks = W::kSlab / 4;      // of a row
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int rg = warp % RG, cg = warp / RG;
  const int N = a.N[which], m0 = slab * W::kSlab + cg * kCols;
  const uint32_t ring = smem_u32(smem), parts = ring + W::kRing;
  const float* Q = reinterpret_cast<const float*>(a.q[which]);
  const float* P = a.p[which];
  const int how = a.how[which];
  const int n = (pc.z + kRows - 1) / kRows;

  auto fill = [&](int i) {
    if (i < n) {
      const uint32_t st = ring + (i % S) * W::kStageBytes;
#pragma unroll
      for (int e = tid; e < kRows * kChunks; e += W::kThreads) {
        const int r = e / kChunks, ch = e % kChunks, row = rows[min(i * kRows + r, kLoraMaxPiece - 1)];
        const bool in = i * kRows + r < pc.z;
        load_chunk<float>(chunk_at(st + (ch >> 3) * (kRows * kLoraRowBytes), r, ch & 7),
                       in ? Q + (int64_t)row * a.ldq[which] : nullptr,
                       slab * W::kSlab + ch * 4, N, how, a.plan.head);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // u or v of a stage: to registers, then as parts to shared memory
  constexpr int kMine = kRows * RG * 16 / W::kThreads;
  static_assert(kRows * RG * 16 % W::kThreads == 0, "values of a stage");
  float pv[kMine];
  auto take = [&](int i) {
#pragma unroll
    for (int j = 0; j < kMine; j++) {
      const int e = tid + j * W::kThreads, r = e % (RG * 16), t = i * kRows + e / (RG * 16);
      pv[j] = t < pc.z && r < a.R ? P[(int64_t)rows[t] * a.R + r] : 0.0f;
    }
  };
  auto put = [&](int i) {
#pragma unroll
    for (int j = 0; j < kMine; j++) {
      const int e = tid + j * W::kThreads, r = e % (RG * 16), t = e / (RG * 16);
      uint16_t p[3];
      split_bf16<3>(pv[j], p);
#pragma unroll
      for (int x = 0; x < 3; x++)
        asm volatile("st.shared.b16 [%0], %1;" ::"r"(parts + (i & 1) * W::kPartBytes + ((x * kRows + t) * W::kPStride + r) * 2),
                     "h"(p[x]) : "memory");
    }
  };
  float acc[kTiles][4], sum[kTiles][4];
#pragma unroll
  for (int j = 0; j < kTiles; j++)
#pragma unroll
    for (int x = 0; x < 4; x++) acc[j][x] = sum[j][x] = 0.0f;
#pragma unroll
  for (int i = 0; i < S - 1; i++) fill(i);
  take(0);
  put(0);
  for (int i = 0; i < n; i++) {
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
    __syncthreads();
    fill(i + S - 1);
    if (i + 1 < n) take(i + 1);
    const uint32_t st = ring + (i % S) * W::kStageBytes, ps = parts + (i & 1) * W::kPartBytes;
    if (m0 < N) {
#pragma unroll
      for (int ks = 0; ks < kRows / 16; ks++) {
        uint32_t p[3][4];
#pragma unroll
        for (int x = 0; x < 3; x++)
          ldsm4t(ps + ((x * kRows + ks * 16 + (lane & 7) + (lane >> 4) * 8) * W::kPStride + rg * 16 + ((lane >> 3) & 1) * 8) * 2, p[x]);
#pragma unroll
        for (int j = 0; j < kTiles; j++) {
          const int col = cg * kCols + j * 8 + g;
          const uint32_t t = st + col / kCB * (kRows * kLoraRowBytes);
          uint32_t b[kQ][2];
#pragma unroll
          for (int h = 0; h < 2; h++) {
            float2 v;
            const int r = ks * 16 + h * 8 + 2 * c, cc = col % kCB;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v.x) : "r"(chunk_at(t, r, cc >> 2) + (cc & 3) * 4) : "memory");
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v.y) : "r"(chunk_at(t, r + 1, cc >> 2) + (cc & 3) * 4) : "memory");
            uint32_t w[kQ];
            split_pair<kQ>(v, w);
#pragma unroll
            for (int y = 0; y < kQ; y++) b[y][h] = w[y];
          }
#pragma unroll
          for (int y = kQ - 1; y >= 0; y--)
#pragma unroll
            for (int x = 2 - y; x >= 0; x--)  // products under 2^-24 of the largest are left out
              mma_16x8x16(acc[j], p[x][0], p[x][1], p[x][2], p[x][3], b[y][0], b[y][1]);
        }
      }
      if (i & 1) {
#pragma unroll
        for (int j = 0; j < kTiles; j++)
#pragma unroll
          for (int x = 0; x < 4; x++) {
            sum[j][x] += acc[j][x];
            acc[j][x] = 0.0f;
          }
      }
    }
    if (i + 1 < n) put(i + 1);
  }
  if (m0 < N) {
#pragma unroll
    for (int j = 0; j < kTiles; j++)
#pragma unroll
      for (int x = 0; x < 4; x++) sum[j][x] += acc[j][x];
    store_sums<RG>(a, which, pc, rg, m0, lane, sum);
  }
}

template <int RG>
__global__ void __launch_bounds__(Wg<RG>::kThreads, Wg<RG>::kCtas) k_lora_wgrad(const __grid_constant__ LoraWgradArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ int32_t rows[kLoraMaxPiece];
  grid_dep_wait();
  const int4 head = *a.plan.head;
  if ((int)blockIdx.y >= head.z) return;
  const int4 pc = a.plan.pieces[blockIdx.y];
  for (int i = threadIdx.x; i < kLoraMaxPiece; i += Wg<RG>::kThreads) rows[i] = i < pc.z ? a.plan.order[pc.y + i] : 0;
  __syncthreads();
  const int nx = a.f32[0] ? (a.N[0] + Wg<RG>::kSlab - 1) / Wg<RG>::kSlab : 0;
  const int which = (int)blockIdx.x >= nx;
  wgrad<RG>(a, which, (int)blockIdx.x - (which ? nx : 0), pc, smem, rows);
}

// Adapters of several pieces: their partial sums in order.  Those without
// rows: zeros.  (One piece: already written.)  V values a thread at a time.
template <int V>
__global__ void __launch_bounds__(256) k_lora_wgrad_sum(const __grid_constant__ LoraWgradArgs a) {
  grid_dep_wait();
  const int l = blockIdx.y;
  const int pieces = a.plan.first[a.L + l];
  if (pieces == 1) return;
  const int64_t slot = a.plan.first[l];
  const int64_t n0 = (int64_t)a.R * a.N[0], all = n0 + (int64_t)a.R * a.N[1];
  for (int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V; e < all; e += (int64_t)gridDim.x * 256 * V) {
    const int w = e >= n0;
    const int64_t i = w ? e - n0 : e, size = w ? all - n0 : n0;
    const float* p = a.part[w] + slot * size + i;
    float* o = a.out[w] + l * size + i;
    if (V == 4) {
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
      for (int s = 0; s < pieces; s++) {
        const float4 x = *reinterpret_cast<const float4*>(p + s * size);
        v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
      }
      *reinterpret_cast<float4*>(o) = v;
    } else {
      float v = 0.0f;
#pragma unroll 4
      for (int s = 0; s < pieces; s++) v += p[s * size];
      *o = v;
    }
  }
}

template <int RG>
cudaError_t run(const LaunchCtx& lc, const LoraWgradArgs& a) {
  typedef Wg<RG> W;
  static std::atomic<int> done[kMaxCachedDevices];
  cudaError_t e = smem_attr_once(k_lora_wgrad<RG>, W::kBytes, done);
  if (e != cudaSuccess) return e;
  int slabs = 0;
  for (int w = 0; w < 2; w++)
    if (a.f32[w]) slabs += (a.N[w] + W::kSlab - 1) / W::kSlab;
  return launch_k(lc, k_lora_wgrad<RG>, dim3(slabs, (unsigned)a.plan.max_pieces), W::kThreads, W::kBytes, a);
}
cudaError_t by_rank(const LaunchCtx& lc, const LoraWgradArgs& a) {
  return a.R <= 16 ? run<1>(lc, a) : a.R <= 32 ? run<2>(lc, a) : a.R <= 64 ? run<4>(lc, a) : run<8>(lc, a);
}

}  // namespace

// Each kernel may start while the one before it ends, and waits for its end
// before all else (a block that left without waiting would let the next one
// start too early).
cudaError_t launch_lora_wgrad(LaunchCtx lc, const LoraWgradArgs& a) {
  lc.pdl = 1;
  cudaError_t e = cudaSuccess;
  if (!a.f32[0] || !a.f32[1]) e = launch_lora_wgrad_tc(lc, a);
  if (e == cudaSuccess && (a.f32[0] || a.f32[1])) e = by_rank(lc, a);
  if (e != cudaSuccess) return e;
  const int64_t all = (int64_t)a.R * (a.N[0] + a.N[1]);
  const bool four = (int64_t)a.R * a.N[0] % 4 == 0 && (int64_t)a.R * a.N[1] % 4 == 0;
  const dim3 sums((unsigned)std::min<int64_t>((all + (four ? 1023 : 255)) / (four ? 1024 : 256), 1024), a.L);
  return four ? launch_k(lc, k_lora_wgrad_sum<4>, sums, 256, 0, a) : launch_k(lc, k_lora_wgrad_sum<1>, sums, 256, 0, a);
}
