// afd_lora.cu -- low-rank adapters of many requests beside a shared
// projection: the plan of a batch, the adapters' weight gradients and the C
// entry points.  The products themselves are in afd_lora_apply.cu.
#include "afd_lora.cuh"

namespace {

constexpr int kPlanWarps = 32;

// One CTA: a stable counting sort of the rows by adapter.  Each warp counts a
// run of the rows (lanes of one adapter find each other, so no two add to one
// counter at a time and no order depends on timing), the counts are summed over warps and adapters, and
// each warp places its run.
__global__ void __launch_bounds__(kPlanWarps * 32, 1) k_lora_plan(const int32_t* ids, int n, int L, LoraPlan p, int tile, int piece) {
  extern __shared__ int32_t cnt[];  // [warps][L + 1]
  __shared__ int32_t total[kLoraMaxAdapters + 1], rows0[kLoraMaxAdapters + 2], tile0[kLoraMaxAdapters + 2],
      piece0[kLoraMaxAdapters + 2], slot0[kLoraMaxAdapters + 2];
  __shared__ int32_t sums[4][kPlanWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, keys = L + 1;
  for (int i = threadIdx.x; i < kPlanWarps * keys; i += kPlanWarps * 32) cnt[i] = 0;
  __syncthreads();
  const int run = (n + kPlanWarps * 32 - 1) / (kPlanWarps * 32) * 32;
  const int lo = min((int64_t)n, (int64_t)warp * run), hi = min((int64_t)n, (int64_t)lo + run);
  int32_t* mine = cnt + warp * keys;
  constexpr int kAhead = 8;
  for (int pass = 0; pass < 2; pass++) {
    for (int base = lo; base < hi; base += kAhead * 32) {
      int key[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; i++) {
        const int t = base + i * 32 + lane;
        key[i] = t < hi ? ids[t] : -2;
      }
#pragma unroll
      for (int i = 0; i < kAhead; i++) {
        const int t = base + i * 32 + lane;
        const int k = t >= hi ? keys : (key[i] < 0 || key[i] >= L ? L : key[i]);
        const uint32_t same = __match_any_sync(0xffffffffu, k);
        const int before = __popc(same & ((1u << lane) - 1u));
        int at = 0;
        if (k < keys) at = mine[k];
        __syncwarp();
        if (k < keys && before == 0) mine[k] = at + __popc(same);
        if (pass && k < keys) p.order[at + before] = t;
        __syncwarp();
      }
    }
    if (pass) break;
    __syncthreads();
    // counts over the warps, exclusive
    for (int k = threadIdx.x; k < keys; k += kPlanWarps * 32) {
      int v = 0;
      for (int w = 0; w < kPlanWarps; w++) {
        const int x = cnt[w * keys + k];
        cnt[w * keys + k] = v;
        v += x;
      }
      total[k] = v;
    }
    __syncthreads();
    // rows, tiles, pieces and partial slots before each adapter: two
    // neighbouring adapters a thread (L + 1 <= 1025; the last one apart)
    int v[2][4], s[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int k = threadIdx.x * 2 + i, c = k < keys ? total[k] : 0;
      const int pieces = k < L ? (c + piece - 1) / piece : 0;
      const int add[4] = {c, (c + tile - 1) / tile, pieces, pieces > 1 ? pieces : 0};
#pragma unroll
      for (int x = 0; x < 4; x++) {
        v[i][x] = s[x];
        s[x] += add[x];
      }
    }
    int incl[4];
#pragma unroll
    for (int x = 0; x < 4; x++) {
      incl[x] = s[x];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl[x], o);
        if (lane >= o) incl[x] += y;
      }
      if (lane == 31) sums[x][warp] = incl[x];
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < 4; x++) {
      int before = incl[x] - s[x];
      for (int w = 0; w < warp; w++) before += sums[x][w];
      int32_t* to = x == 0 ? rows0 : x == 1 ? tile0 : x == 2 ? piece0 : slot0;
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const int k = threadIdx.x * 2 + i;
        if (k < keys) to[k] = before + v[i][x];
        if (k == keys - 1) to[keys] = before + s[x];  // (an adapter past the last adds nothing)
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kPlanWarps * keys; i += kPlanWarps * 32) cnt[i] += rows0[i % keys];
    if (threadIdx.x == 0) *p.head = make_int4(tile0[L], tile0[keys] - tile0[L], piece0[L], rows0[L]);
    for (int k = threadIdx.x; k < L; k += kPlanWarps * 32) {
      p.first[k] = slot0[k];
      p.first[L + k] = piece0[k + 1] - piece0[k];
    }
    // tile i: of the last adapter whose tiles start at or before it
    for (int i = threadIdx.x; i < tile0[keys]; i += kPlanWarps * 32) {
      int a = 0, b = keys;
      while (b - a > 1) {
        const int m = (a + b) / 2;
        if (tile0[m] <= i) a = m; else b = m;
      }
      const int at = (i - tile0[a]) * tile;
      p.tiles[i] = make_int4(a < L ? a : -1, rows0[a] + at, min(tile, total[a] - at), 0);
    }
    for (int i = threadIdx.x; i < piece0[L]; i += kPlanWarps * 32) {
      int a = 0, b = L;
      while (b - a > 1) {
        const int m = (a + b) / 2;
        if (piece0[m] <= i) a = m; else b = m;
      }
      const int j = i - piece0[a];
      p.pieces[i] = make_int4(a, rows0[a] + j * piece, min(piece, total[a] - j * piece),
                              piece0[a + 1] - piece0[a] > 1 ? slot0[a] + j : -1);
    }
    __syncthreads();
  }
}

// Weight gradients: out[r][n] = scale sum over the piece's rows of p[t][r]
// q[t][n].  A CTA takes a piece and up to 512 columns of x or dy, a warp 64 of
// them (or, of narrow matrices, a share of the rows); sixteen rows are one k
// step of the tensor cores, their columns loaded straight to operands
// (pair_rows), p in three bf16 parts from shared memory.
constexpr int kWgRows = 64;  // rows staged at a time
constexpr int kWgStride = kWgRows + 8;

template <int RT, typename TQ>
__device__ __forceinline__ void wgrad(const LoraWgradArgs& a, int which, int64_t block, const int4& pc, uint8_t* smem) {
  constexpr int kQ = LoraSrc<TQ>::kParts;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int N = a.N[which], blocks = (N + 63) / 64;
  int wc = 8;  // warps side by side over columns; the others share the rows
  while (wc > 1 && wc / 2 >= blocks) wc /= 2;
  const int share = 8 / wc, mine = warp / wc;
  const int m0 = (int)block * 512 + warp % wc * 64;
  const bool live = m0 < N;
  uint16_t* ps = reinterpret_cast<uint16_t*>(smem);  // [3][RT * 16][kWgStride]
  const int32_t* order = a.plan.order + pc.y;
  const float* P = a.p[which];
  const TQ* Q = reinterpret_cast<const TQ*>(a.q[which]);
  const bool vec = a.vec[which];
  const float scale = a.scale ? a.scale[pc.x] : 1.0f;
  float* out = pc.w < 0 ? a.out[which] + (int64_t)pc.x * a.R * N : a.part[which] + (int64_t)pc.w * a.R * N;
  for (int r0 = 0; r0 < a.R; r0 += RT * 16) {
    float acc[RT][8][4];
#pragma unroll
    for (int i = 0; i < RT; i++)
#pragma unroll
      for (int j = 0; j < 8; j++)
#pragma unroll
        for (int x = 0; x < 4; x++) acc[i][j][x] = 0.0f;
    for (int t0 = 0; t0 < pc.z; t0 += kWgRows) {
      __syncthreads();
      for (int e = threadIdx.x; e < RT * 16 * kWgRows; e += 256) {
        const int i = e / (RT * 16), r = e % (RT * 16);
        const float v = t0 + i < pc.z && r0 + r < a.R ? P[(int64_t)order[t0 + i] * a.R + r0 + r] : 0.0f;
        uint16_t p[3];
        split_bf16<3>(v, p);
#pragma unroll
        for (int x = 0; x < 3; x++) ps[(x * RT * 16 + r) * kWgStride + i] = p[x];
      }
      __syncthreads();
      if (live) {
#pragma unroll 2
        for (int s = mine; s < kWgRows / 16; s += share) {
          if (t0 + s * 16 >= pc.z) break;
          uint4 v[4][kQ];
#pragma unroll
          for (int x = 0; x < 4; x++) {
            const int i = t0 + s * 16 + 2 * c + (x >> 1) * 8 + (x & 1);
            const bool in = i < pc.z;
            load_eight<TQ>(in ? Q + (int64_t)order[i] * a.ldq[which] : Q, m0 + g * 8, in ? N : 0, vec, v[x]);
          }
#pragma unroll
          for (int y = kQ - 1; y >= 0; y--) {
            uint32_t b[8][2];
            pair_rows(v[0][y], v[1][y], v[2][y], v[3][y], b);
#pragma unroll
            for (int x = 2 - y; x >= 0; x--)  // products under 2^-24 of the largest are left out
#pragma unroll
              for (int i = 0; i < RT; i++) {
                const uint16_t* p0 = ps + (x * RT * 16 + i * 16 + g) * kWgStride + s * 16 + 2 * c;
                const uint16_t* p1 = p0 + 8 * kWgStride;
                const uint32_t a0 = *reinterpret_cast<const uint32_t*>(p0), a1 = *reinterpret_cast<const uint32_t*>(p1);
                const uint32_t a2 = *reinterpret_cast<const uint32_t*>(p0 + 8), a3 = *reinterpret_cast<const uint32_t*>(p1 + 8);
#pragma unroll
                for (int j = 0; j < 8; j++) mma_16x8x16(acc[i][j], a0, a1, a2, a3, b[j][0], b[j][1]);
              }
          }
        }
      }
    }
    if (share > 1) {  // the warps that shared the rows, in order
      float* red = reinterpret_cast<float*>(smem);  // [8 warps][32 values][32 lanes]
#pragma unroll
      for (int i = 0; i < RT; i++) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; j++)
#pragma unroll
          for (int x = 0; x < 4; x++) red[(warp * 32 + j * 4 + x) * 32 + lane] = acc[i][j][x];
        __syncthreads();
        if (mine == 0)
          for (int o = 1; o < share; o++)
#pragma unroll
            for (int j = 0; j < 8; j++)
#pragma unroll
              for (int x = 0; x < 4; x++) acc[i][j][x] += red[((warp + o * wc) * 32 + j * 4 + x) * 32 + lane];
      }
    }
    if (live && mine == 0) {
#pragma unroll
      for (int i = 0; i < RT; i++)
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const int r = r0 + i * 16 + h * 8 + g;
          if (r >= a.R) continue;
          float* d = out + (int64_t)r * N;
#pragma unroll
          for (int s = 0; s < 2; s++) {
            const int c0 = m0 + c * 16 + s * 8;
            float v[8];
#pragma unroll
            for (int x = 0; x < 8; x++) v[x] = scale * acc[i][x][2 * h + s];
            if (N % 8 == 0) {
              if (c0 < N) {
                *reinterpret_cast<float4*>(d + c0) = make_float4(v[0], v[1], v[2], v[3]);
                *reinterpret_cast<float4*>(d + c0 + 4) = make_float4(v[4], v[5], v[6], v[7]);
              }
            } else {
#pragma unroll
              for (int x = 0; x < 8; x++)
                if (c0 + x < N) d[c0 + x] = v[x];
            }
          }
        }
    }
  }
}

template <int RT, typename TX, typename TY>
__global__ void __launch_bounds__(256) k_lora_wgrad(const __grid_constant__ LoraWgradArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int4 head = *a.plan.head;
  if ((int)blockIdx.y >= head.z) return;
  const int4 pc = a.plan.pieces[blockIdx.y];
  const int nx = (a.N[0] + 511) / 512;
  if ((int)blockIdx.x < nx)
    wgrad<RT, TX>(a, 0, blockIdx.x, pc, smem);
  else
    wgrad<RT, TY>(a, 1, blockIdx.x - nx, pc, smem);
}

// Adapters of several pieces: their partial sums in order.  Those without
// rows: zeros.  (One piece: already written.)
__global__ void __launch_bounds__(256) k_lora_wgrad_sum(const __grid_constant__ LoraWgradArgs a) {
  const int l = blockIdx.y;
  const int pieces = a.plan.first[a.L + l];
  if (pieces == 1) return;
  const int64_t slot = a.plan.first[l];
  const int64_t n0 = (int64_t)a.R * a.N[0], all = n0 + (int64_t)a.R * a.N[1];
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < all; e += (int64_t)gridDim.x * 256) {
    const int w = e >= n0;
    const int64_t i = w ? e - n0 : e, size = w ? all - n0 : n0;
    float v = 0.0f;
#pragma unroll 4
    for (int s = 0; s < pieces; s++) v += a.part[w][(slot + s) * size + i];
    a.out[w][l * size + i] = v;
  }
}

template <int RT, typename TX, typename TY>
cudaError_t run_wgrad(const LaunchCtx& lc, const LoraWgradArgs& a) {
  constexpr int kStage = 3 * RT * 16 * kWgStride * 2, kRed = 8 * 32 * 32 * 4, kBytes = kStage > kRed ? kStage : kRed;
  const dim3 grid((a.N[0] + 511) / 512 + (a.N[1] + 511) / 512, (unsigned)a.plan.max_pieces);
  cudaError_t e = launch_k(lc, k_lora_wgrad<RT, TX, TY>, grid, 256, kBytes, a);
  if (e != cudaSuccess) return e;
  const int64_t all = (int64_t)a.R * (a.N[0] + a.N[1]);
  return launch_k(lc, k_lora_wgrad_sum, dim3((unsigned)std::min<int64_t>((all + 1023) / 1024, 128), a.L), 256, 0, a);
}
template <typename TX, typename TY>
cudaError_t wgrad_by_rank(const LaunchCtx& lc, const LoraWgradArgs& a) {
  return a.R <= 16 ? run_wgrad<1, TX, TY>(lc, a) : run_wgrad<2, TX, TY>(lc, a);
}

}  // namespace

cudaError_t launch_lora_wgrad(const LaunchCtx& lc, const LoraWgradArgs& a) {
  if (a.f32[0]) return a.f32[1] ? wgrad_by_rank<float, float>(lc, a) : wgrad_by_rank<float, uint16_t>(lc, a);
  return a.f32[1] ? wgrad_by_rank<uint16_t, float>(lc, a) : wgrad_by_rank<uint16_t, uint16_t>(lc, a);
}

namespace {
bool off_by(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }
int64_t size_of(int dtype) { return dtype == AFD_DTYPE_F32 ? 4 : 2; }
bool dtype_ok(int d) { return d == AFD_DTYPE_F32 || d == AFD_DTYPE_BF16; }
bool batch_ok(int64_t n, int L) { return n >= 0 && n <= kLoraMaxTokens && L >= 1 && L <= kLoraMaxAdapters; }
bool dims_ok(int K, int M, int R) {
  return K >= 1 && K <= kLoraMaxCols && M >= 1 && M <= kLoraMaxCols && R >= 1 && R <= kLoraMaxRank;
}
// rows of a matrix can be moved 16 bytes at a time
bool rows16(const void* p, int64_t ld, int dtype) { return !off_by(p, 16) && ld * size_of(dtype) % 16 == 0; }
}  // namespace

extern "C" int64_t afd_lora_plan_bytes(int64_t n_tokens, int n_adapters) {
  if (!batch_ok(n_tokens, n_adapters)) return -1;
  return lora_plan_at(nullptr, n_tokens, n_adapters).bytes;
}

extern "C" int afd_lora_plan(const int32_t* ids, int64_t n_tokens, int n_adapters, void* plan, int64_t plan_bytes,
                             void* cuda_stream) {
  if (!batch_ok(n_tokens, n_adapters) || !plan || off_by(plan, 256) || (n_tokens && !ids) || off_by(ids, 4))
    return AFD_ERR_ARG;
  const LoraPlan p = lora_plan_at(plan, n_tokens, n_adapters);
  if (plan_bytes < p.bytes) return AFD_ERR_CAPACITY;
  const int rc = check_device_ptrs({n_tokens ? ids : nullptr, plan});
  if (rc) return rc;
  const LaunchCtx lc{reinterpret_cast<cudaStream_t>(cuda_stream), 0, nullptr};
  static std::atomic<int> done[kMaxCachedDevices];
  cudaError_t e = smem_attr_once(k_lora_plan, kPlanWarps * (kLoraMaxAdapters + 1) * 4, done);
  if (e == cudaSuccess)
    e = launch_k(lc, k_lora_plan, 1, kPlanWarps * 32, (size_t)kPlanWarps * (n_adapters + 1) * 4, ids, (int)n_tokens,
                 n_adapters, p, lora_tile(n_tokens), lora_piece(n_tokens));
  if (e != cudaSuccess) {
    cudaGetLastError();
    return AFD_ERR_CUDA;
  }
  return AFD_OK;
}

extern "C" int afd_lora_apply(const void* plan, int64_t n_tokens, int n_adapters, const void* x, int64_t ldx,
                              int x_dtype, int K, const void* a, const void* b, int rank, int M, const float* scale,
                              const void* base, int64_t ldb, int y_dtype, void* out, int64_t ldo, float* u,
                              void* cuda_stream) {
  if (!batch_ok(n_tokens, n_adapters) || !dims_ok(K, M, rank) || !dtype_ok(x_dtype) || !dtype_ok(y_dtype) || ldx < K ||
      ldo < M || (base && ldb < M))
    return AFD_ERR_ARG;
  if (n_tokens == 0) return AFD_OK;
  if (!plan || off_by(plan, 256) || !x || !a || !b || !out || off_by(x, size_of(x_dtype)) || off_by(a, 2) ||
      off_by(b, 2) || off_by(scale, 4) || off_by(base, size_of(y_dtype)) || off_by(out, size_of(y_dtype)) ||
      off_by(u, 4) || (base == out && ldb != ldo))
    return AFD_ERR_ARG;
  const int rc = check_device_ptrs({plan, x, a, b, scale, base, out, u});
  if (rc) return rc;
  LoraArgs g{};
  g.plan = lora_plan_at(const_cast<void*>(plan), n_tokens, n_adapters);
  g.src = x; g.lds = ldx; g.w1 = a; g.w2 = b; g.scale = scale;
  g.base = base; g.ldb = ldb; g.out = out; g.ldo = ldo; g.u = u;
  g.T = n_tokens; g.K = K; g.M = M; g.R = rank;
  g.src_f32 = x_dtype == AFD_DTYPE_F32; g.out_f32 = y_dtype == AFD_DTYPE_F32;
  g.vk = K % 8 == 0 && rows16(x, ldx, x_dtype) && !off_by(a, 16);
  g.vm = M % 8 == 0 && rows16(out, ldo, y_dtype) && (!base || rows16(base, ldb, y_dtype)) && !off_by(b, 16);
  const LaunchCtx lc{reinterpret_cast<cudaStream_t>(cuda_stream), 0, nullptr};
  if (launch_lora_apply(lc, g) != cudaSuccess) {
    cudaGetLastError();
    return AFD_ERR_CUDA;
  }
  return AFD_OK;
}

namespace {
int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }
}  // namespace

extern "C" int64_t afd_lora_backward_workspace(int64_t n_tokens, int n_adapters, int K, int M, int rank) {
  if (!batch_ok(n_tokens, n_adapters) || !dims_ok(K, M, rank)) return -1;
  const LoraPlan p = lora_plan_at(nullptr, n_tokens, n_adapters);
  return up256(n_tokens * rank * 4) + up256(p.max_slots * rank * K * 4) + up256(p.max_slots * rank * M * 4);
}

extern "C" int afd_lora_backward(const void* plan, int64_t n_tokens, int n_adapters, const void* x, int64_t ldx,
                                 int x_dtype, int K, const void* dy, int64_t ldy, int y_dtype, int M, const float* u,
                                 const void* a, const void* b, int rank, const float* scale, const void* d_base,
                                 int64_t ldb, void* dx, int64_t ldd, float* da, float* db, void* workspace,
                                 int64_t workspace_bytes, void* cuda_stream) {
  if (!batch_ok(n_tokens, n_adapters) || !dims_ok(K, M, rank) || !dtype_ok(x_dtype) || !dtype_ok(y_dtype) || ldx < K ||
      ldy < M || ldd < K || (d_base && ldb < K))
    return AFD_ERR_ARG;
  const int64_t need = afd_lora_backward_workspace(n_tokens, n_adapters, K, M, rank);
  if (!da || !db || off_by(da, 16) || off_by(db, 16)) return AFD_ERR_ARG;
  if (n_tokens &&
      (!plan || off_by(plan, 256) || !x || !dy || !u || !a || !b || !dx || !workspace || off_by(workspace, 256) ||
       off_by(x, size_of(x_dtype)) || off_by(dy, size_of(y_dtype)) || off_by(u, 4) || off_by(a, 2) || off_by(b, 2) ||
       off_by(scale, 4) || off_by(d_base, size_of(x_dtype)) || off_by(dx, size_of(x_dtype)) ||
       (d_base == dx && ldb != ldd)))
    return AFD_ERR_ARG;
  if (workspace_bytes < need) return AFD_ERR_CAPACITY;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(cuda_stream);
  if (n_tokens == 0) {  // no rows: no gradient
    const int rc = check_device_ptrs({da, db});
    if (rc) return rc;
    if (cudaMemsetAsync(da, 0, (size_t)n_adapters * rank * K * 4, stream) != cudaSuccess ||
        cudaMemsetAsync(db, 0, (size_t)n_adapters * rank * M * 4, stream) != cudaSuccess) {
      cudaGetLastError();
      return AFD_ERR_CUDA;
    }
    return AFD_OK;
  }
  const int rc = check_device_ptrs({plan, x, dy, u, a, b, scale, d_base, dx, da, db, workspace});
  if (rc) return rc;
  float* v = reinterpret_cast<float*>(workspace);
  LoraArgs g{};
  g.plan = lora_plan_at(const_cast<void*>(plan), n_tokens, n_adapters);
  g.src = dy; g.lds = ldy; g.w1 = b; g.w2 = a; g.scale = scale;
  g.base = d_base; g.ldb = ldb; g.out = dx; g.ldo = ldd; g.u = v;
  g.T = n_tokens; g.K = M; g.M = K; g.R = rank;
  g.src_f32 = y_dtype == AFD_DTYPE_F32; g.out_f32 = x_dtype == AFD_DTYPE_F32;
  g.vk = M % 8 == 0 && rows16(dy, ldy, y_dtype) && !off_by(b, 16);
  g.vm = K % 8 == 0 && rows16(dx, ldd, x_dtype) && (!d_base || rows16(d_base, ldb, x_dtype)) && !off_by(a, 16);
  LoraWgradArgs w{};
  w.plan = g.plan;
  w.p[0] = v; w.p[1] = u; w.q[0] = x; w.q[1] = dy; w.ldq[0] = ldx; w.ldq[1] = ldy;
  w.out[0] = da; w.out[1] = db; w.N[0] = K; w.N[1] = M;
  w.part[0] = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + up256(n_tokens * rank * 4));
  w.part[1] = reinterpret_cast<float*>(reinterpret_cast<char*>(w.part[0]) + up256(g.plan.max_slots * rank * K * 4));
  w.f32[0] = g.out_f32; w.f32[1] = g.src_f32;
  w.vec[0] = K % 8 == 0 && rows16(x, ldx, x_dtype);
  w.vec[1] = M % 8 == 0 && rows16(dy, ldy, y_dtype);
  w.scale = scale; w.T = n_tokens; w.R = rank; w.L = n_adapters;
  const LaunchCtx lc{stream, 0, nullptr};
  cudaError_t e = launch_lora_apply(lc, g);
  if (e == cudaSuccess) e = launch_lora_wgrad(lc, w);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return AFD_ERR_CUDA;
  }
  return AFD_OK;
}
