// afd_lora_wgrad_tc.cu -- the adapters' weight gradients from bf16 rows, on
// tcgen05 (fp32 rows: afd_lora_wgrad.cu):
//   da[l] = scale[l] sum_t v_t x_t^T,  db[l] = scale[l] sum_t u_t dy_t^T
//
// A CTA takes one piece of an adapter's rows and 128 columns of x or dy.  The
// product's k runs over the rows, so both operands are used as they lie in
// memory, rows of neighbouring elements (MN-major), 64 of them to a 128-byte
// swizzled row: asynchronous copies gather x or dy by the plan's order
// straight into the layout the tensor cores read.  u or v comes as three bf16
// parts, which keep its 24 bits, written by the kernel of the products as the
// stages hold them, so that one bulk copy brings a stage's: splitting fp32
// values here, once for each 128 columns, was more than half of the
// instructions (98 us where this takes @@), and by 16-byte copies of the threads
// they took more of the copies' rate than x and dy (61).  The parts of up
// to 32 ranks stand side by side in the 128 rows of one MMA and are added at
// the end, those of more take two or three MMAs.
//
// Sums in TMEM may cut where they should round, so they move to registers
// every four stages (128 rows) and start anew in the other accumulator, while
// the next MMAs run.  Bound by memory: 2 rank operations a byte (times three
// parts) are a fifth of what the tensor cores do in the time.
//
// Every wait is for MMAs or copies already issued, and bounded; one that gives up is
// counted (afd_mx4_poll_status).
#include "afd_lora.cuh"

namespace {

__device__ uint32_t g_lora_errors;  // waits that gave up

constexpr int kThreads = 256, kRows = 32, kSlab = 128;
constexpr int kAtom = kRows * kLoraRowBytes;     // 64 columns or ranks of a stage
constexpr int kFlush = 4;                        // stages between two moves of the sums
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr int kOutStride = 65;                   // floats, of the output's staging

// MP: ranks of a part, padded: the parts stand MP rows apart
template <int MP>
struct Tc {
  static constexpr int kMmas = MP <= 32 ? 1 : MP == 64 ? 2 : 3;  // a 16-row step
  static constexpr int kAtoms = lora_atoms(MP);                  // of the parts
  static constexpr int kStageBytes = (2 + kAtoms) * kAtom;
  static constexpr int kStages = MP == 16 ? 7 : MP == 32 ? 6 : MP == 64 ? 5 : 3;
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kBytes = kRing + kAtom;                   // and an atom of zeros: MMA rows of no part
  // accumulator rows of a rank: this many, this far apart (MP 64: the first
  // and third part share theirs)
  static constexpr int kSums = MP <= 32 ? 3 : MP == 64 ? 2 : 1;
  static_assert(128 * kOutStride * 4 <= kRing, "the output is staged in the ring");
};

// bf16 x bf16 -> fp32, both operands MN-major, M = N = 128
constexpr uint32_t kIdesc = 1u << 4 | 1u << 7 | 1u << 10 | 1u << 15 | 1u << 16 | (uint32_t)(kSlab >> 3) << 17 | (128u >> 4) << 24;

__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity) {
  const uint64_t start = globaltimer_ns();
  uint32_t spins = 0;
  while (!mbar_try_wait(bar, parity)) {
    if ((++spins & 255u) == 0 && globaltimer_ns() - start > kTimeoutNs) return false;
  }
  return true;
}
__device__ __forceinline__ bool wait_mma(uint32_t bar, uint32_t parity) {
  return mbar_try_wait(bar, parity) || wait_long(bar, parity);
}

template <int MP>
__global__ void __launch_bounds__(kThreads, 2) k_lora_wgrad_tc(const __grid_constant__ LoraWgradArgs a) {
  typedef Tc<MP> W;
  constexpr int S = W::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ int32_t rows[kLoraMaxPiece];
  __shared__ uint64_t bars[2], there[S];  // MMAs of a stage done; its parts there
  __shared__ uint32_t tmem_base;
  const int4 head = *a.plan.head;
  if ((int)blockIdx.y >= head.z) return;
  const int4 pc = a.plan.pieces[blockIdx.y];
  const int nx = a.f32[0] ? 0 : (a.N[0] + kSlab - 1) / kSlab;
  const int which = (int)blockIdx.x >= nx, m0 = ((int)blockIdx.x - (which ? nx : 0)) * kSlab;
  const int N = a.N[which], how = a.how[which], R = a.R;
  // blocks of the parts, as the stages hold them
  const uint16_t* P = a.parts[which] + (int64_t)(pc.y + a.plan.shift[pc.x]) / kLoraBlockRows * (W::kAtoms * kAtom / 2);
  const uint16_t* Q = reinterpret_cast<const uint16_t*>(a.q[which]);
  const int64_t ldq = a.ldq[which];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t ring = smem_u32(smem), zero = ring + W::kRing, bar = smem_u32(bars);
  for (int i = tid; i < pc.z; i += kThreads) rows[i] = a.plan.order[pc.y + i];
  *reinterpret_cast<uint4*>(smem + W::kRing + 16 * tid) = make_uint4(0u, 0u, 0u, 0u);
  if (tid == 0) {
    mbar_init(bar, 1);
    mbar_init(bar + 8, 1);
    for (int i = 0; i < S; i++) mbar_init(smem_u32(&there[i]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)), "r"(2 * kSlab));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  const int n = (pc.z + kRows - 1) / kRows;

  auto fill = [&](int i) {
    if (i < n) {
      const uint32_t st = ring + (i % S) * W::kStageBytes;
      const int ch = tid & 15;
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int r = (tid >> 4) + h * 16, t = i * kRows + r;
        load_chunk<uint16_t>(chunk_at(st + (ch >> 3) * kAtom, r, ch & 7), t < pc.z ? Q + (int64_t)rows[t] * ldq : nullptr,
                             m0 + ch * 8, N, how, a.plan.head);
      }
      if (tid == 0) {
        const uint32_t b = smem_u32(&there[i % S]);
        mbar_expect_tx(b, W::kAtoms * kAtom);
        bulk_load(st + 2 * kAtom, P + (int64_t)i * (W::kAtoms * kAtom / 2), W::kAtoms * kAtom, b);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // accumulator row 32 (warp % 4) + lane, columns 64 (warp / 4) ..
  float sum[64];
#pragma unroll
  for (int j = 0; j < 64; j++) sum[j] = 0.0f;
  const uint32_t mine = tmem + ((uint32_t)(warp & 3) << 21) + (warp >> 2) * 64;
  auto flush = [&](int group) {
    tc_fence_after();
    const uint32_t d = mine + (group & 1) * kSlab;
#pragma unroll
    for (int h = 0; h < 2; h++) {
      uint32_t v[32];
      tmem_ld_32x32b_x32(d + h * 32, v);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 32; j++) sum[h * 32 + j] += __uint_as_float(v[j]);
    }
    tc_fence_before();
  };
#pragma unroll
  for (int i = 0; i < S - 1; i++) fill(i);
  bool good = true;
  int i = 0;
  for (; i < n; i++) {
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    if (__syncthreads_or(!good)) break;
    if (warp == 0) {
      good = __all_sync(0xffffffffu, wait_mma(smem_u32(&there[i % S]), i / S & 1));
      tc_fence_after();
      const uint32_t el = lora_elect(), d = tmem + (i / kFlush & 1) * kSlab;
      // two atoms of 64 elements each, 8-row groups 1024 bytes apart
      const uint32_t qa = (ring + (i % S) * W::kStageBytes) >> 4, pa = qa + (2 * kAtom >> 4);
#pragma unroll
      for (int ks = 0; ks < kRows / 16; ks++)
#pragma unroll
        for (int x = W::kMmas - 1; x >= 0; x--)
          lora_mma(el, d, lora_desc(pa + (x * 2 * kAtom + ks * 2048 >> 4), 2 * x + 1 < W::kAtoms ? kAtom >> 4 : (zero >> 4) - (pa + (x * 2 * kAtom >> 4))),
                   lora_desc(qa + ks * 128, kAtom >> 4), kIdesc, i % kFlush != 0 || ks != 0 || x != W::kMmas - 1);
      lora_commit(el, bar + 8 * (i & 1));
    }
    if (i > 0) {  // the stage before: its ring slot is free, its sums complete
      good &= wait_mma(bar + 8 * ((i - 1) & 1), ((i - 1) >> 1) & 1);
      if (i % kFlush == 0) flush(i / kFlush - 1);
    }
    fill(i + S - 1);
  }
  if (i == n && n > 0) {
    good &= wait_mma(bar + 8 * ((n - 1) & 1), ((n - 1) >> 1) & 1);
    flush((n - 1) / kFlush);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  const bool bad = __syncthreads_or(!good);
  if (bad) {
    if (tid == 0) {
      atomicAdd(&g_lora_errors, 1u);
      for (int x = max(0, i - 1); x < min(n, i + S - 1); x++) wait_mma(smem_u32(&there[x % S]), x / S & 1);  // copies under way
    }
    __syncthreads();
  } else {
    const float scale = a.scale ? a.scale[pc.x] : 1.0f;
    float* out = pc.w < 0 ? a.out[which] + (int64_t)pc.x * R * N : a.part[which] + (int64_t)pc.w * R * N;
    float* stage = reinterpret_cast<float*>(smem);  // [128][kOutStride]
    for (int p = 0; p < 2; p++) {  // 64 columns at a time
      if (warp >> 2 == p) {
        float* s = stage + ((warp & 3) * 32 + lane) * kOutStride;
#pragma unroll
        for (int j = 0; j < 64; j++) s[j] = sum[j];
      }
      __syncthreads();
      for (int e = tid; e < R * 64; e += kThreads) {
        const int r = e >> 6, col = m0 + p * 64 + (e & 63);
        if (col < N) {
          float v = stage[r * kOutStride + (e & 63)];
#pragma unroll
          for (int x = 1; x < W::kSums; x++) v += stage[(x * MP + r) * kOutStride + (e & 63)];
          out[(int64_t)r * N + col] = scale * v;
        }
      }
      __syncthreads();
    }
  }
  tc_fence_after();
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * kSlab));
}

template <int MP>
cudaError_t run(const LaunchCtx& lc, const LoraWgradArgs& a) {
  typedef Tc<MP> W;
  static std::atomic<int> done[kMaxCachedDevices];
  cudaError_t e = smem_attr_once(k_lora_wgrad_tc<MP>, W::kBytes, done);
  if (e != cudaSuccess) return e;
  int slabs = 0;
  for (int w = 0; w < 2; w++)
    if (!a.f32[w]) slabs += (a.N[w] + kSlab - 1) / kSlab;
  return launch_k(lc, k_lora_wgrad_tc<MP>, dim3(slabs, (unsigned)a.plan.max_pieces), kThreads, W::kBytes, a);
}

}  // namespace

cudaError_t launch_lora_wgrad_tc(const LaunchCtx& lc, const LoraWgradArgs& a) {
  return a.R <= 16 ? run<16>(lc, a) : a.R <= 32 ? run<32>(lc, a) : a.R <= 64 ? run<64>(lc, a) : run<128>(lc, a);
}

cudaError_t lora_error_count(uint32_t* n, cudaStream_t stream) {
  return cudaMemcpyFromSymbolAsync(n, g_lora_errors, sizeof *n, 0, cudaMemcpyDeviceToHost, stream);
}
