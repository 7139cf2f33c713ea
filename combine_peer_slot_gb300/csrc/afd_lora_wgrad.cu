// afd_lora_wgrad.cu -- the adapters' weight gradients, on tcgen05:
//   da[l] = scale[l] sum_t v_t x_t^T,  db[l] = scale[l] sum_t u_t dy_t^T
//
// The product's k runs over the rows, so both operands are used as they lie in
// memory, rows of neighbouring elements (MN-major), 64 of them to a 128-byte
// swizzled row: asynchronous copies gather x or dy by the plan's order
// straight into the layout the tensor cores read.  u or v comes as three bf16
// parts, which keep its 24 bits, written by the kernel of the products as the
// stages hold them: one bulk copy brings a stage's.  Rows of fp32, or not of
// whole 16 bytes, are first laid out in the plan's order as one or three bf16
// planes (k_lora_planes): 24 bits again, a stage for each plane (split by the
// threads that multiply, the gradients of 12000 fp32 rows of 3649 columns, rank
// 64, took 200 us more).  The parts of up to 32 ranks stand side by side in the
// 128 rows of one MMA and are added at the end, those of more take two or three
// MMAs.
//
// Sums in TMEM may cut where they should round, so they move to registers
// every four stages (128 rows) and start anew in the other accumulator, while
// the next MMAs run.
//
// Bound by memory: one CTA an SM runs through items (a piece of an adapter's
// rows, 256 columns of x or dy) with its warps apart: three copy, one issues the
// MMAs, sixteen sum and store, and the copies run on into the next item while
// the last is stored.  With all warps together, two CTAs of 128 columns an SM,
// a stage of 32 rows took 1150 to 1800 cycles of barrier, issue, wait and
// copying one after the other, and an item 9000 before and behind its stages
// (rank 64, 13312 rows: 62 us where this takes 48, and the sum of the pieces 8
// more).  What it has to read and write would take 21; a stage's copies take a
// warp 1200 to 2600 cycles, most while other warps store partial sums, and five
// stages are all that the staged output leaves room for.
//
// All waits are bounded; one that gives up is counted (afd_lora_poll_status).
#include "afd_lora.cuh"

namespace {

__device__ uint32_t g_lora_errors;  // waits that gave up

constexpr int kSumWarps = 16, kCopyWarps = 3;  // (and one more: five warps a scheduler leave 96 registers a thread)
constexpr int kThreads = (kSumWarps + kCopyWarps + 1) * 32;
constexpr int kRows = kLoraBlockRows, kSlab = 256;
constexpr int kAtom = kRows * kLoraRowBytes;     // 64 columns or ranks of a stage
constexpr int kFlush = 4;                        // stages between two moves of the sums
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr int kOutStride = 68;                   // floats, of the output's staging

// MP: ranks of a part, padded: the parts stand MP rows apart
template <int MP>
struct Tc {
  static constexpr int kMmas = MP <= 32 ? 1 : MP == 64 ? 2 : 3;  // a 16-row step
  static constexpr int kAtoms = lora_atoms(MP);                  // of the parts
  static constexpr int kStageBytes = (kSlab / 64 + kAtoms) * kAtom;
  // accumulator rows of a rank: this many, MP apart (MP 64: the first and
  // third part share theirs), which meet in shared memory
  static constexpr int kSums = MP <= 32 ? 3 : MP == 64 ? 2 : 1;
  static constexpr int kOutBytes = kSums > 1 ? 4 * 64 * kOutStride * 4 : 0;
  static constexpr int kStages = (224 * 1024 - kAtom - kOutBytes) / kStageBytes;
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kBytes = kRing + kAtom + kOutBytes;       // with an atom of zeros: MMA rows of no part
};

// bf16 x bf16 -> fp32, both operands MN-major, M 128, N 256
constexpr uint32_t kIdesc = 1u << 4 | 1u << 7 | 1u << 10 | 1u << 15 | 1u << 16 | (uint32_t)(kSlab >> 3) << 17 | (128u >> 4) << 24;

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
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity) || wait_long(bar, parity, abort_flag));
}

// of the 128 threads at a barrier: whether all say yes
__device__ __forceinline__ bool all_of(int id, bool yes) {
  uint32_t r;
  asm volatile("{ .reg .pred p, q; setp.ne.u32 p, %2, 0; bar.red.and.pred q, %1, 128, p; selp.u32 %0, 1, 0, q; }"
               : "=r"(r) : "r"(id), "r"((uint32_t)yes) : "memory");
  return r != 0;
}

// scaled values of a row from column c on
__device__ __forceinline__ void store_four(float* row, int c, int N, float scale, const float* v) {
  if (N % 4 == 0) {
    if (c < N) *reinterpret_cast<float4*>(row + c) = make_float4(scale * v[0], scale * v[1], scale * v[2], scale * v[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; j++)
      if (c + j < N) row[c + j] = scale * v[j];
  }
}
template <int COLS>
__device__ __forceinline__ void store_row(float* row, int c, int N, float scale, const float (&v)[COLS]) {
#pragma unroll
  for (int j = 0; j < COLS; j += 4) store_four(row, c + j, N, scale, v + j);
}

// a piece's stages: every 32 rows, once for each plane
__device__ __forceinline__ int stages_of(const int4& pc, int planes) { return (pc.z + kRows - 1) / kRows * planes; }

template <int MP>
__global__ void __launch_bounds__(kThreads, 1) k_lora_wgrad(const __grid_constant__ LoraWgradArgs a) {
  typedef Tc<MP> W;
  constexpr int S = W::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  // of each stage: full, free again; sums of a group of stages: complete, taken
  __shared__ uint64_t full[S], empty[S], dfull[2], dempty[2];
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, R = a.R;
  const int nx = (a.N[0] + kSlab - 1) / kSlab, slabs = nx + (a.N[1] + kSlab - 1) / kSlab;
  const uint32_t ring = smem_u32(smem), zero = ring + W::kRing;
  if (tid < kAtom / 16) *reinterpret_cast<uint4*>(smem + W::kRing + 16 * tid) = make_uint4(0u, 0u, 0u, 0u);
  if (tid < S) {
    mbar_init(smem_u32(&full[tid]), 33);  // a copying warp's lanes, and its bulk copy
    mbar_init(smem_u32(&empty[tid]), 1);
    if (tid < 2) {
      mbar_init(smem_u32(&dfull[tid]), 1);
      mbar_init(smem_u32(&dempty[tid]), kSumWarps);
    }
    if (tid == 0) abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)), "r"(2 * kSlab));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  tc_fence_after();
  grid_dep_wait();  // the products' kernel
  const uint32_t tmem = tmem_base;
  const int items = a.plan.head->z * slabs;
  volatile int* const gave_up = &abort_flag;
  bool good = true;
  int slot = 0, stage = 0;  // of the ring, over all items
  uint32_t turn = 0;
  auto next = [&]() {
    stage++;
    if (++slot == S) {
      slot = 0;
      turn++;
    }
  };

  if (warp >= kSumWarps && warp < kSumWarps + kCopyWarps) {  // ---- copies: every kCopyWarps-th stage ----
    for (int item = blockIdx.x; item < items && good; item += gridDim.x) {
      const int4 pc = a.plan.pieces[item / slabs];
      const int slab = item % slabs, which = slab >= nx, m0 = (slab - (which ? nx : 0)) * kSlab;
      const int N = a.N[which], col = m0 + lane * 8, planes = a.planes[which], n = stages_of(pc, planes);
      const uint16_t* P = a.parts[which] + (int64_t)(pc.y + a.plan.shift[pc.x]) / kRows * (W::kAtoms * kAtom / 2);
      const bool in = col < N;
      const int64_t pitch = in ? a.ldq[which] * 2 : 0;
      int plane = 0, block = 0;
      for (int i = 0; i < n; i++, next(), plane = plane + 1 < planes ? plane + 1 : (block++, 0)) {
        if (stage % kCopyWarps != warp - kSumWarps) continue;
        if (turn) {
          good = warp_wait(smem_u32(&empty[slot]), (turn - 1) & 1, gave_up);
          if (!good) break;
        }
        const uint32_t st = ring + slot * W::kStageBytes, bar = smem_u32(&full[slot]);
        const int t0 = block * kRows, have = min(kRows, pc.z - t0);  // rows of the piece; the others zero
        const int my_row = lane >= have ? 0 : a.ordered[which] ? pc.y + t0 + lane : a.plan.order[pc.y + t0 + lane];
        if (lane == 0) {
          mbar_expect_tx(bar, W::kAtoms * kAtom);
          bulk_load(st + kSlab / 64 * kAtom, P + (int64_t)block * (W::kAtoms * kAtom / 2), W::kAtoms * kAtom, bar);
        }
        const char* p = in ? reinterpret_cast<const char*>(a.q[which]) + (plane * a.plane[which] + col) * 2
                           : reinterpret_cast<const char*>(a.plan.head);
        const uint32_t to = st + (lane >> 3) * kAtom, ch = (lane & 7) << 4;
#pragma unroll
        for (int j = 0; j < kRows; j++) {
          const int row = __shfl_sync(0xffffffffu, my_row, j);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + j * kLoraRowBytes + (ch ^ (j & 7) << 4)),
                       "l"(p + row * pitch), "r"(in && j < have ? 16 : 0)
                       : "memory");
        }
        // each lane arrives when its copies have landed
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == kSumWarps + kCopyWarps) {  // ---- products ----
    const uint32_t el = lora_elect();
    uint32_t group = 0;
    for (int item = blockIdx.x; item < items && good; item += gridDim.x) {
      const int n = stages_of(a.plan.pieces[item / slabs], a.planes[item % slabs >= nx]);
      for (int i = 0; i < n; i++, next()) {
        good = warp_wait(smem_u32(&full[slot]), turn & 1, gave_up);
        if (good && i % kFlush == 0 && group >= 2) good = warp_wait(smem_u32(&dempty[group & 1]), (group / 2 - 1) & 1, gave_up);
        if (!good) break;
        // the copies' writes, seen through the barrier, before the products'
        // reads, which go another way
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_after();
        const uint32_t d = tmem + (group & 1) * kSlab;
        // atoms of 64 elements, 8-row groups 1024 bytes apart
        const uint32_t qa = (ring + slot * W::kStageBytes) >> 4, pa = qa + (kSlab / 64 * kAtom >> 4);
#pragma unroll
        for (int ks = 0; ks < kRows / 16; ks++)
#pragma unroll
          for (int x = W::kMmas - 1; x >= 0; x--) {
            const uint32_t at = pa + (x * 2 * kAtom >> 4), apart = 2 * x + 1 < W::kAtoms ? kAtom >> 4 : (zero >> 4) - at;
            lora_mma(el, d, lora_desc(at + (ks * 2048 >> 4), apart), lora_desc(qa + ks * 128, kAtom >> 4), kIdesc,
                     i % kFlush != 0 || ks != 0 || x != W::kMmas - 1);
          }
        lora_commit(el, smem_u32(&empty[slot]));
        if (i % kFlush == kFlush - 1 || i == n - 1) lora_commit(el, smem_u32(&dfull[group++ & 1]));
      }
    }
    if (!good) {  // (a wait has given up: time for bulk copies under way to land)
      const uint64_t start = globaltimer_ns();
      while (globaltimer_ns() - start < 1000000ull) {}
    }
  } else {  // ---- sums: accumulator row 32 (warp % 4) + lane, columns 64 (warp / 4) .. ----
    const int m = (warp & 3) * 32 + lane, cg = warp >> 2;
    const uint32_t mine = tmem + ((uint32_t)(warp & 3) << 21) + cg * 64;
    float* out_stage = reinterpret_cast<float*>(smem + W::kRing + kAtom) + cg * 64 * kOutStride;  // [64][kOutStride]
    uint32_t group = 0;
    auto meet = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + cg) : "memory"); };  // the four warps of these columns
    for (int item = blockIdx.x; item < items && good; item += gridDim.x) {
      const int4 pc = a.plan.pieces[item / slabs];
      const int slab = item % slabs, which = slab >= nx, m0 = (slab - (which ? nx : 0)) * kSlab + cg * 64;
      const int N = a.N[which], n = stages_of(pc, a.planes[which]);
      float sum[64];
#pragma unroll
      for (int j = 0; j < 64; j++) sum[j] = 0.0f;
      for (int i = 0; i < n; i += kFlush, group++) {
        good = warp_wait(smem_u32(&dfull[group & 1]), group / 2 & 1, gave_up);
        if (!good) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 64; c += 16) {
          uint32_t v[16];
          tmem_ld_16(mine + (group & 1) * kSlab + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; j++) sum[c + j] += __uint_as_float(v[j]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&dempty[group & 1]));
      }
      if (!all_of(1 + cg, good)) {  // (the four warps leave together: none waits for one that has left)
        good = false;
        break;
      }
      const float scale = a.scale ? a.scale[pc.x] : 1.0f;
      float* out = pc.w < 0 ? a.out[which] + (int64_t)pc.x * R * N : a.part[which] + (int64_t)pc.w * R * N;
      if (W::kSums == 1) {
        if (m < R) store_row<64>(out + (int64_t)m * N, m0, N, scale, sum);
        continue;
      }
      // the parts' sums meet, and go to memory a row's 64 columns at a time
      float* mine_out = out_stage + (m < MP ? m : m - MP) * kOutStride;
      if (m >= MP && m < W::kSums * MP) {
#pragma unroll
        for (int j = 0; j < 64; j += 4) *reinterpret_cast<float4*>(mine_out + j) = make_float4(sum[j], sum[j + 1], sum[j + 2], sum[j + 3]);
      }
      meet();
      if (m < MP) {
#pragma unroll
        for (int j = 0; j < 64; j += 4) {
#pragma unroll
          for (int x = 0; x < W::kSums - 1; x++) {
            const float4 v = *reinterpret_cast<const float4*>(mine_out + x * MP * kOutStride + j);
            sum[j] += v.x; sum[j + 1] += v.y; sum[j + 2] += v.z; sum[j + 3] += v.w;
          }
          *reinterpret_cast<float4*>(mine_out + j) = make_float4(sum[j], sum[j + 1], sum[j + 2], sum[j + 3]);
        }
      }
      meet();
      for (int r = (warp & 3) * 8 + (lane >> 2); r < R; r += 32) {
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; j++) v[j] = out_stage[r * kOutStride + (lane & 3) * 4 + j / 4 * 16 + j % 4];
#pragma unroll
        for (int j = 0; j < 4; j++) store_four(out + (int64_t)r * N, m0 + (lane & 3) * 4 + j * 16, N, scale, v + 4 * j);
      }
      meet();
    }
  }
  __syncthreads();
  if (tid == 0 && abort_flag) atomicAdd(&g_lora_errors, 1u);
  tc_fence_after();
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * kSlab));
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

// Rows in the plan's order as bf16 planes, a warp a row: three of an fp32 row
// (its parts), one of a bf16 row.
template <typename T>
__global__ void __launch_bounds__(256) k_lora_planes(const LoraPlan plan, const T* q, int64_t ldq, int N, int vec, uint16_t* to,
                                                     int64_t pitch, int64_t plane) {
  constexpr int kP = LoraSrc<T>::kParts;
  const int lane = threadIdx.x & 31;
  const int64_t rows = plan.head->w, step = (int64_t)gridDim.x * 8;
  for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < rows; i += step) {
    const T* from = q + (int64_t)plan.order[i] * ldq;
#pragma unroll 2
    for (int c = lane * 8; c < N; c += 256) {
      uint4 v[kP];
      if (sizeof(T) == 2 && !vec) v[0] = load_words(reinterpret_cast<const uint16_t*>(from), c, N);
      else load_eight<T>(from, c, N, vec, v);
#pragma unroll
      for (int x = 0; x < kP; x++) *reinterpret_cast<uint4*>(to + x * plane + i * pitch + c) = v[x];
    }
  }
}

template <int MP>
cudaError_t run(const LaunchCtx& lc, const LoraWgradArgs& a) {
  typedef Tc<MP> W;
  static std::atomic<int> done[kMaxCachedDevices];
  const cudaError_t e = smem_attr_once(k_lora_wgrad<MP>, W::kBytes, done);
  if (e != cudaSuccess) return e;
  return launch_k(lc, k_lora_wgrad<MP>, kLoraSms, kThreads, W::kBytes, a);
}

}  // namespace

cudaError_t launch_lora_planes(const LaunchCtx& lc, const LoraPlan& plan, int64_t tokens, const void* q, int64_t ldq, int N,
                               int f32, int vec, uint16_t* to) {
  const int64_t pitch = lora_plane_pitch(N), plane = tokens * pitch;
  const unsigned grid = (unsigned)std::min<int64_t>((tokens + 7) / 8, 8 * kLoraSms);
  if (f32) return launch_k(lc, k_lora_planes<float>, grid, 256, 0, plan, (const float*)q, ldq, N, vec, to, pitch, plane);
  return launch_k(lc, k_lora_planes<uint16_t>, grid, 256, 0, plan, (const uint16_t*)q, ldq, N, vec, to, pitch, plane);
}

// Each kernel may start while the one before it ends, and waits for its end
// before all else (a block that left without waiting would let the next one
// start too early).
cudaError_t launch_lora_wgrad(LaunchCtx lc, const LoraWgradArgs& a) {
  lc.pdl = 1;
  const cudaError_t e = a.R <= 16   ? run<16>(lc, a)
                        : a.R <= 32 ? run<32>(lc, a)
                        : a.R <= 64 ? run<64>(lc, a)
                                    : run<128>(lc, a);
  if (e != cudaSuccess) return e;
  const int64_t all = (int64_t)a.R * (a.N[0] + a.N[1]);
  const bool four = (int64_t)a.R * a.N[0] % 4 == 0 && (int64_t)a.R * a.N[1] % 4 == 0;
  const dim3 sums((unsigned)std::min<int64_t>((all + (four ? 1023 : 255)) / (four ? 1024 : 256), 1024), a.L);
  return four ? launch_k(lc, k_lora_wgrad_sum<4>, sums, 256, 0, a) : launch_k(lc, k_lora_wgrad_sum<1>, sums, 256, 0, a);
}

cudaError_t lora_error_count(uint32_t* n, cudaStream_t stream) {
  return cudaMemcpyFromSymbolAsync(n, g_lora_errors, sizeof *n, 0, cudaMemcpyDeviceToHost, stream);
}

#ifdef AFD_DEBUG_BOUNDS
int lora_plant_error() {
  uint32_t n = 0;
  if (cudaDeviceSynchronize() != cudaSuccess || cudaMemcpyFromSymbol(&n, g_lora_errors, sizeof n) != cudaSuccess ||
      cudaMemcpyToSymbol(g_lora_errors, &(++n), sizeof n) != cudaSuccess) {
    cudaGetLastError();
    return AFD_ERR_CUDA;
  }
  return AFD_OK;
}
#endif
