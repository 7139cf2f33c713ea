// afd_lora.cu -- low-rank adapters of many requests beside a shared
// projection: the plan of a batch and the C entry points.  The products are in
// afd_lora_apply.cu (few rows), afd_lora_tiles.cu and afd_lora_tc.cu (many), the
// weight gradients in afd_lora_wgrad.cu.
#include "afd_lora.cuh"

#include <map>

namespace {

constexpr int kPlanWarps = 32;

// One CTA: a stable counting sort of the rows by adapter.  Each warp counts a
// run of the rows (lanes of one adapter find each other, so no two add to one
// counter at a time and no order depends on timing), the counts are summed over
// warps and adapters, and each warp places its run.  Made once for a batch:
// 329 rows 10 us, 13312 rows of 8 adapters 12 to 19, of 1024 up to 44.
__global__ void __launch_bounds__(kPlanWarps * 32, 1) k_lora_plan(const int32_t* ids, int n, int L, LoraPlan p, int tile, int piece) {
  extern __shared__ int32_t cnt[];  // [warps][L + 1]
  __shared__ int32_t total[kLoraMaxAdapters + 1], rows0[kLoraMaxAdapters + 2], tile0[kLoraMaxAdapters + 2],
      piece0[kLoraMaxAdapters + 2], slot0[kLoraMaxAdapters + 2], block0[kLoraMaxAdapters + 2];
  __shared__ int32_t sums[5][kPlanWarps];
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
    // rows, tiles, pieces, partial slots and blocks before each adapter: two
    // neighbouring adapters a thread (L + 1 <= 1025; the last one apart)
    int v[2][5], s[5] = {0, 0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int k = threadIdx.x * 2 + i, c = k < keys ? total[k] : 0;
      const int pieces = k < L ? (c + piece - 1) / piece : 0;
      const int add[5] = {c, (c + tile - 1) / tile, pieces, pieces > 1 ? pieces : 0, (c + kLoraBlockRows - 1) / kLoraBlockRows};
#pragma unroll
      for (int x = 0; x < 5; x++) {
        v[i][x] = s[x];
        s[x] += add[x];
      }
    }
    int incl[5];
#pragma unroll
    for (int x = 0; x < 5; x++) {
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
    for (int x = 0; x < 5; x++) {
      int before = incl[x] - s[x];
      for (int w = 0; w < warp; w++) before += sums[x][w];
      int32_t* to = x == 0 ? rows0 : x == 1 ? tile0 : x == 2 ? piece0 : x == 3 ? slot0 : block0;
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
      p.shift[k] = block0[k] * kLoraBlockRows - rows0[k];
    }
    // tile i: of the last adapter whose tiles start at or before it
    for (int i = threadIdx.x; i < tile0[keys]; i += kPlanWarps * 32) {
      int a = 0, b = keys;
      while (b - a > 1) {
        const int m = (a + b) / 2;
        if (tile0[m] <= i) a = m; else b = m;
      }
      const int at = (i - tile0[a]) * tile;
      p.tiles[i] = make_int4(a < L ? a : -1, rows0[a] + at, min(tile, total[a] - at),
                              a < L && at + tile >= total[a] ? (kLoraBlockRows - total[a] % kLoraBlockRows) % kLoraBlockRows : 0);
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

}  // namespace

namespace {
bool off_by(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }
int64_t size_of(int dtype) { return dtype == AFD_DTYPE_F32 ? 4 : 2; }
bool dtype_ok(int d) { return d == AFD_DTYPE_F32 || d == AFD_DTYPE_BF16; }
bool batch_ok(int64_t n, int L) { return n >= 0 && n <= kLoraMaxTokens && L >= 1 && L <= kLoraMaxAdapters; }
bool dims_ok(int K, int M, int R) {
  return K >= 1 && K <= kLoraMaxCols && M >= 1 && M <= kLoraMaxCols && R >= 1 && R <= kLoraMaxRank;
}
// how rows of n elements can be moved (LoraArgs)
int how_rows(const void* p, int64_t ld, int n, int dtype) {
  for (int b = 16; b >= 4; b /= 2)
    if (!off_by(p, b) && ld * size_of(dtype) % b == 0 && n * size_of(dtype) % b == 0) return b;
  return 0;
}
cudaError_t launch_products(const LaunchCtx& lc, LoraArgs& g) {
  const int ts = g.src_f32 ? AFD_DTYPE_F32 : AFD_DTYPE_BF16, to = g.out_f32 ? AFD_DTYPE_F32 : AFD_DTYPE_BF16;
  g.how_src = how_rows(g.src, g.lds, g.K, ts);
  g.how_w1 = how_rows(g.w1, g.K, g.K, AFD_DTYPE_BF16);
  g.how_w2 = how_rows(g.w2, g.M, g.M, AFD_DTYPE_BF16);
  g.how_base = how_rows(g.base, g.ldb, g.M, to);
  g.how_out = how_rows(g.out, g.ldo, g.M, to);
  if (lora_tile(g.T) == 16) return launch_lora_apply(lc, g);
  return lora_tc_takes(g) ? launch_lora_tc(lc, g) : launch_lora_tiles(lc, g);
}
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
  if (!apart({run_of(plan, p.bytes)}, {run_of(ids, n_tokens * 4)})) return AFD_ERR_ARG;
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
  const int64_t xs = size_of(x_dtype), ys = size_of(y_dtype), T = n_tokens, L = n_adapters;
  if (!apart({{out, ldo * ys, M * ys, T}, run_of(u, T * rank * 4)},
             {run_of(plan, afd_lora_plan_bytes(T, n_adapters)), {x, ldx * xs, K * xs, T}, run_of(a, L * rank * K * 2),
              run_of(b, L * rank * M * 2), run_of(scale, L * 4), {base == out ? nullptr : base, ldb * ys, M * ys, T}}))
    return AFD_ERR_ARG;
  const int rc = check_device_ptrs({plan, x, a, b, scale, base, out, u});
  if (rc) return rc;
  LoraArgs g{};
  g.plan = lora_plan_at(const_cast<void*>(plan), n_tokens, n_adapters);
  g.src = x; g.lds = ldx; g.w1 = a; g.w2 = b; g.scale = scale;
  g.base = base; g.ldb = ldb; g.out = out; g.ldo = ldo; g.u = u;
  g.T = n_tokens; g.K = K; g.M = M; g.R = rank; g.L = n_adapters;
  g.src_f32 = x_dtype == AFD_DTYPE_F32; g.out_f32 = y_dtype == AFD_DTYPE_F32;
  const LaunchCtx lc{reinterpret_cast<cudaStream_t>(cuda_stream), 0, nullptr};
  if (launch_products(lc, g) != cudaSuccess) {
    cudaGetLastError();
    return AFD_ERR_CUDA;
  }
  return AFD_OK;
}

namespace {
int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }
}  // namespace

// The workspace: parts of v and of u, the partial sums of da and db, and the
// planes of x and dy where the rows themselves cannot be copied to the tensor
// cores' operands (the pitches are not known when its size is asked for, so
// bf16 rows always count with one).
static int64_t lora_workspace(int64_t T, int L, int K, int M, int R, int x_f32, int y_f32) {
  const LoraPlan p = lora_plan_at(nullptr, T, L);
  return 2 * up256(lora_parts_bytes(T, L, lora_padded(R))) + up256(p.max_slots * R * K * 4) + up256(p.max_slots * R * M * 4) +
         up256(T * lora_plane_pitch(K) * 2 * (x_f32 ? 3 : 1)) + up256(T * lora_plane_pitch(M) * 2 * (y_f32 ? 3 : 1));
}

extern "C" int64_t afd_lora_backward_workspace(int64_t n_tokens, int n_adapters, int K, int M, int rank, int x_dtype, int y_dtype) {
  if (!batch_ok(n_tokens, n_adapters) || !dims_ok(K, M, rank) || !dtype_ok(x_dtype) || !dtype_ok(y_dtype)) return -1;
  return lora_workspace(n_tokens, n_adapters, K, M, rank, x_dtype == AFD_DTYPE_F32, y_dtype == AFD_DTYPE_F32);
}

extern "C" int afd_lora_backward(const void* plan, int64_t n_tokens, int n_adapters, const void* x, int64_t ldx,
                                 int x_dtype, int K, const void* dy, int64_t ldy, int y_dtype, int M, const float* u,
                                 const void* a, const void* b, int rank, const float* scale, const void* d_base,
                                 int64_t ldb, void* dx, int64_t ldd, float* da, float* db, void* workspace,
                                 int64_t workspace_bytes, void* cuda_stream) {
  if (!batch_ok(n_tokens, n_adapters) || !dims_ok(K, M, rank) || !dtype_ok(x_dtype) || !dtype_ok(y_dtype) || ldx < K ||
      ldy < M || ldd < K || (d_base && ldb < K))
    return AFD_ERR_ARG;
  const int64_t need = afd_lora_backward_workspace(n_tokens, n_adapters, K, M, rank, x_dtype, y_dtype);
  if (!da || !db || off_by(da, 16) || off_by(db, 16)) return AFD_ERR_ARG;
  if (n_tokens &&
      (!plan || off_by(plan, 256) || !x || !dy || !u || !a || !b || !dx || !workspace || off_by(workspace, 256) ||
       off_by(x, size_of(x_dtype)) || off_by(dy, size_of(y_dtype)) || off_by(u, 4) || off_by(a, 2) || off_by(b, 2) ||
       off_by(scale, 4) || off_by(d_base, size_of(x_dtype)) || off_by(dx, size_of(x_dtype)) ||
       (d_base == dx && ldb != ldd)))
    return AFD_ERR_ARG;
  if (workspace_bytes < need) return AFD_ERR_CAPACITY;
  const int64_t xs = size_of(x_dtype), ys = size_of(y_dtype), T = n_tokens, L = n_adapters;
  if (!apart({{dx, ldd * xs, K * xs, T}, run_of(da, L * rank * K * 4), run_of(db, L * rank * M * 4), run_of(workspace, T ? need : 0)},
             {run_of(plan, T ? afd_lora_plan_bytes(T, n_adapters) : 0), {x, ldx * xs, K * xs, T}, {dy, ldy * ys, M * ys, T},
              run_of(u, T * rank * 4), run_of(a, T ? L * rank * K * 2 : 0), run_of(b, T ? L * rank * M * 2 : 0),
              run_of(scale, T ? L * 4 : 0), {d_base == dx ? nullptr : d_base, ldb * xs, K * xs, T}}))
    return AFD_ERR_ARG;
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
  char* at = reinterpret_cast<char*>(workspace);
  auto take = [&](int64_t bytes) {
    char* r = at;
    at += up256(bytes);
    return r;
  };
  LoraArgs g{};
  g.plan = lora_plan_at(const_cast<void*>(plan), n_tokens, n_adapters);
  g.src = dy; g.lds = ldy; g.w1 = b; g.w2 = a; g.scale = scale;
  g.base = d_base; g.ldb = ldb; g.out = dx; g.ldo = ldd;
  g.T = n_tokens; g.K = M; g.M = K; g.R = rank; g.L = n_adapters;
  g.src_f32 = y_dtype == AFD_DTYPE_F32; g.out_f32 = x_dtype == AFD_DTYPE_F32;
  g.u_parts = reinterpret_cast<uint16_t*>(take(lora_parts_bytes(n_tokens, n_adapters, lora_padded(rank))));
  g.other_parts = reinterpret_cast<uint16_t*>(take(lora_parts_bytes(n_tokens, n_adapters, lora_padded(rank))));
  g.other = u;
  LoraWgradArgs w{};
  w.plan = g.plan;
  w.parts[0] = g.u_parts; w.parts[1] = g.other_parts;
  w.out[0] = da; w.out[1] = db; w.N[0] = K; w.N[1] = M;
  w.part[0] = reinterpret_cast<float*>(take(g.plan.max_slots * rank * K * 4));
  w.part[1] = reinterpret_cast<float*>(take(g.plan.max_slots * rank * M * 4));
  w.scale = scale; w.R = rank; w.L = n_adapters;
  const LaunchCtx lc{stream, 0, nullptr};
  const void* rows[2] = {x, dy};
  const int64_t ld[2] = {ldx, ldy};
  const int dtype[2] = {x_dtype, y_dtype};
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < 2 && e == cudaSuccess; i++) {
    const int f32 = dtype[i] == AFD_DTYPE_F32, how = how_rows(rows[i], ld[i], w.N[i], dtype[i]);
    w.planes[i] = f32 ? 3 : 1;
    w.q[i] = rows[i];
    w.ldq[i] = ld[i];
    if (f32 || how != 16) {
      uint16_t* to = reinterpret_cast<uint16_t*>(take(n_tokens * lora_plane_pitch(w.N[i]) * 2 * w.planes[i]));
      e = launch_lora_planes(lc, g.plan, n_tokens, rows[i], ld[i], w.N[i], f32, how == 16 && w.N[i] % 8 == 0, to);
      w.q[i] = to;
      w.ldq[i] = lora_plane_pitch(w.N[i]);
      w.plane[i] = n_tokens * w.ldq[i];
      w.ordered[i] = 1;
    }
  }
  if (e == cudaSuccess) e = launch_products(lc, g);
  if (e == cudaSuccess) e = launch_lora_wgrad(lc, w);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return AFD_ERR_CUDA;
  }
  return AFD_OK;
}

// The errors are counted and never cleared, and a caller is told of those since
// its own last call, so that no caller takes another's.
extern "C" int afd_lora_poll_status(void* cuda_stream) {
  uint32_t n[2] = {0, 0};
  int dev = 0;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(cuda_stream);
  if (cudaGetDevice(&dev) != cudaSuccess || lora_error_count(&n[0], stream) != cudaSuccess ||
      lora_tc_error_count(&n[1], stream) != cudaSuccess || cudaStreamSynchronize(stream) != cudaSuccess) {
    cudaGetLastError();
    return AFD_ERR_CUDA;
  }
  const uint32_t all = n[0] + n[1];
  bool more = all != 0;
  try {
    thread_local std::map<std::pair<int, void*>, uint32_t> told;
    uint32_t& last = told[{dev, cuda_stream}];
    more = all != last;
    last = all;
  } catch (...) {  // no memory to keep it: told again
  }
  return more ? AFD_ERR_TIMEOUT : AFD_OK;
}
