// afd_balance.cu -- the load of the experts and the gradient of the routing
// choice: per-expert counts and a balance loss for each sequence of the batch
// (afd_balance_loss), the gradient of that loss and of the chosen weights with
// respect to the logits (afd_route_backward).
//
//   p_te = softmax(l_t)_e, or s_te / sum_e s_te with s = 1 / (1 + exp(-l))
//   loss_s = E / (k n_s^2) sum_e counts_se sum_{t in s} p_te
//
// A warp takes a row: lane l holds the experts [l PER, (l + 1) PER).
#include <cooperative_groups.h>

#include "afd_internal.cuh"

namespace {

namespace cg = cooperative_groups;

constexpr int kFinal = 8;  // CTAs that finish one sequence: 32 experts each

struct GateArgs {
  const void* logits;
  int64_t ld;
  const int32_t* ids;
  const int32_t* off;  // [S + 1], or NULL: one sequence of all rows
  int n, E, k, S, sigmoid;
  int vec;             // a lane's run of logits can be loaded whole
  // forward
  float* loss;
  int32_t* counts;     // backward: read
  float* part;         // [S][chunks][E] sums of p, then as many counts
  int chunks;
  // backward
  const float* dw;     // [n, k] or NULL
  const float* dloss;  // [S] or NULL
  int renorm;
  float scale;
  void* d;
  int64_t ldd;
  int dvec;
  int per_block;       // rows of a block
};

template <typename LT>
__device__ __forceinline__ float load_one(const void* p, int64_t i);
template <>
__device__ __forceinline__ float load_one<float>(const void* p, int64_t i) {
  return reinterpret_cast<const float*>(p)[i];
}
template <>
__device__ __forceinline__ float load_one<uint16_t>(const void* p, int64_t i) {
  return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << 16);
}

template <int BYTES>
struct Run;
template <>
struct Run<4> { typedef uint32_t T; };
template <>
struct Run<8> { typedef uint2 T; };
template <>
struct Run<16> { typedef uint4 T; };

// PER neighbouring logits of a row; experts past the last one read as -inf
template <typename LT, int PER>
__device__ __forceinline__ void load_row(const void* p, int64_t i0, int have, int vec, float (&v)[PER]) {
  if (vec && have >= PER) {
    constexpr int kBytes = PER * (int)sizeof(LT) < 16 ? PER * (int)sizeof(LT) : 16;
    typedef typename Run<kBytes>::T V;
    union {
      V q[PER * sizeof(LT) / kBytes];
      LT e[PER];
    } u;
    const V* s = reinterpret_cast<const V*>(reinterpret_cast<const LT*>(p) + i0);
#pragma unroll
    for (int i = 0; i < (int)(PER * sizeof(LT) / kBytes); i++) u.q[i] = s[i];
#pragma unroll
    for (int i = 0; i < PER; i++) v[i] = load_one<LT>(u.e, i);
    return;
  }
#pragma unroll
  for (int i = 0; i < PER; i++) v[i] = i < have ? load_one<LT>(p, i0 + i) : -INFINITY;
}

template <typename LT>
__device__ __forceinline__ LT rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t rounded<uint16_t>(float v) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

template <typename LT, int PER>
__device__ __forceinline__ void store_row(void* p, int64_t i0, int have, int vec, const float (&v)[PER]) {
  LT* d = reinterpret_cast<LT*>(p) + i0;
  if (vec && have >= PER) {
    constexpr int kBytes = PER * (int)sizeof(LT) < 16 ? PER * (int)sizeof(LT) : 16;
    typedef typename Run<kBytes>::T V;
    union {
      V q[PER * sizeof(LT) / kBytes];
      LT e[PER];
    } u;
#pragma unroll
    for (int i = 0; i < PER; i++) u.e[i] = rounded<LT>(v[i]);
#pragma unroll
    for (int i = 0; i < (int)(PER * sizeof(LT) / kBytes); i++) reinterpret_cast<V*>(d)[i] = u.q[i];
    return;
  }
#pragma unroll
  for (int i = 0; i < PER; i++)
    if (i < have) d[i] = rounded<LT>(v[i]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// s = 1 / (1 + exp(-l)) and 1 - s, each to fp32's precision of itself
__device__ __forceinline__ void sigmoid_pair(float l, float& s, float& rest) {
  const float e = expf(-fabsf(l)), r = 1.0f / (1.0f + e), q = e * r;
  s = l >= 0.0f ? r : q;  // (NaN: q, which is NaN)
  rest = l >= 0.0f ? q : r;
}

// What one row's sums of exponentials are.
struct RowSum {
  float top, z;  // largest logit, sum of exp(l - top)
};

// p of a row from its logits.  sigmoid: rest = 1 - s as well.  A row of -inf
// has p = 0.  Scores whose sum nears fp32's smallest number come from logits
// under -60, where s = exp(l) (1 - 1e-26): their shares are the softmax's.
template <int PER>
__device__ __forceinline__ RowSum shares(const float (&l)[PER], int sigmoid, float (&p)[PER], float (&rest)[PER]) {
  RowSum r{0.0f, 0.0f};
  if (sigmoid) {
#pragma unroll
    for (int i = 0; i < PER; i++) {
      sigmoid_pair(l[i], p[i], rest[i]);
      r.z += p[i];
    }
    r.z = warp_sum(r.z);
    if (!(r.z < 1e-30f)) {
      const float inv = 1.0f / r.z;
#pragma unroll
      for (int i = 0; i < PER; i++) p[i] *= inv;
      return r;
    }
  }
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; i++) top = fmaxf(top, l[i]);
  r.top = warp_max(top);
  r.z = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; i++) {
    p[i] = l[i] == -INFINITY ? 0.0f : expf(l[i] - r.top);
    r.z += p[i];
  }
  r.z = warp_sum(r.z);
  const float inv = r.z == 0.0f ? 0.0f : 1.0f / r.z;
#pragma unroll
  for (int i = 0; i < PER; i++) p[i] *= inv;
  return r;
}

// rows [lo, hi) of sequence s, inside [0, n]
__device__ __forceinline__ void sequence(const GateArgs& a, int s, int& lo, int& hi) {
  lo = 0;
  hi = a.n;
  if (a.off) {
    lo = min(max(a.off[s], 0), a.n);
    hi = max(lo, min(max(a.off[s + 1], 0), a.n));
  }
}

// E / (k n^2) sum_e counts p, over the 32 WARPS' values of one block
__device__ __forceinline__ float loss_of(const GateArgs& a, int rows, double dot) {
  return rows ? (float)(dot * (double)a.E / ((double)a.k * (double)rows * (double)rows)) : 0.0f;
}

// Block (c, s): the rows lo + c, lo + c + chunks, .. of sequence s, a warp
// each.  One chunk: the sequence's loss at once; else its share of the sums.
// Sums of p: at most rows / (warps chunks) terms in a lane's fp32 chain, then
// the warps' in order.  Counts are whole numbers, so their order is free.
template <typename LT, int PER, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) k_balance(const __grid_constant__ GateArgs a) {
  __shared__ float sums[WARPS][32 * PER];
  __shared__ int32_t cnt[32 * PER];
  __shared__ double dots[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = lane * PER, have = a.E - e0;
  const int s = blockIdx.y, c = blockIdx.x;
  for (int e = threadIdx.x; e < 32 * PER; e += WARPS * 32) cnt[e] = 0;
  int lo, hi;
  sequence(a, s, lo, hi);
  __syncthreads();
  float acc[PER];
#pragma unroll
  for (int i = 0; i < PER; i++) acc[i] = 0.0f;
  for (int64_t row = (int64_t)lo + c * WARPS + warp; row < hi; row += (int64_t)a.chunks * WARPS) {
    float l[PER], p[PER], rest[PER];
    load_row<LT, PER>(a.logits, row * a.ld + e0, have, a.vec, l);
    const int id = lane < a.k ? a.ids[row * a.k + lane] : -1;
    shares<PER>(l, a.sigmoid, p, rest);
#pragma unroll
    for (int i = 0; i < PER; i++) acc[i] += p[i];
    if (id >= 0 && id < a.E) atomicAdd(&cnt[id], 1);
  }
#pragma unroll
  for (int i = 0; i < PER; i++) sums[warp][e0 + i] = acc[i];
  __syncthreads();
  double dot = 0.0;
  for (int e = threadIdx.x; e < a.E; e += WARPS * 32) {
    float v = 0.0f;
#pragma unroll 8
    for (int w = 0; w < WARPS; w++) v += sums[w][e];
    if (a.chunks > 1) {
      const int64_t at = ((int64_t)s * a.chunks + c) * a.E + e;
      a.part[at] = v;
      reinterpret_cast<int32_t*>(a.part)[(int64_t)a.S * a.chunks * a.E + at] = cnt[e];
    } else {
      a.counts[(int64_t)s * a.E + e] = cnt[e];
      dot += (double)v * (double)cnt[e];
    }
  }
  if (a.chunks > 1) return;
#pragma unroll
  for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
  if (lane == 0) dots[warp] = dot;
  __syncthreads();
  if (threadIdx.x == 0) {
    double v = 0.0;
    for (int w = 0; w < WARPS; w++) v += dots[w];
    a.loss[s] = loss_of(a, hi - lo, v);
  }
}

// The chunks' sums to counts and loss: a cluster per sequence, CTA q the
// experts [32 q, 32 q + 32), lane = expert, warps stride the chunks; sums in
// 64 bits, in a fixed order.
__global__ void __cluster_dims__(kFinal, 1, 1) __launch_bounds__(256) k_balance_finish(const __grid_constant__ GateArgs a) {
  __shared__ double sums[8][32];
  __shared__ int32_t cnts[8][32];
  __shared__ double dot_of[kFinal];
  cg::cluster_group cluster = cg::this_cluster();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, q = blockIdx.x, s = blockIdx.y;
  const int e = q * 32 + lane;
  cudaGridDependencySynchronize();
  double v = 0.0;
  int32_t n = 0;
  if (e < a.E) {
    const float* p = a.part + (int64_t)s * a.chunks * a.E + e;
    const int32_t* m = reinterpret_cast<const int32_t*>(a.part) + (int64_t)a.S * a.chunks * a.E + (int64_t)s * a.chunks * a.E + e;
#pragma unroll 4
    for (int c = warp; c < a.chunks; c += 8) {
      v += (double)p[(int64_t)c * a.E];
      n += m[(int64_t)c * a.E];
    }
  }
  sums[warp][lane] = v;
  cnts[warp][lane] = n;
  __syncthreads();
  if (warp == 0) {
    for (int w = 1; w < 8; w++) {
      v += sums[w][lane];
      n += cnts[w][lane];
    }
    if (e < a.E) a.counts[(int64_t)s * a.E + e] = n;
    double dot = v * (double)n;
#pragma unroll
    for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (lane == 0) *cluster.map_shared_rank(&dot_of[q], 0) = dot;
  }
  cluster.sync();
  if (q == 0 && threadIdx.x == 0) {
    double d = 0.0;
    for (int i = 0; i < kFinal; i++) d += dot_of[i];
    int lo, hi;
    sequence(a, s, lo, hi);
    a.loss[s] = loss_of(a, hi - lo, d);
  }
}

// d loss / d logits and d weights / d logits of a row in one pass.  With
// G_e = d_loss E counts_e / (k n^2) the balance part is p (G - sum p G), times
// 1 - s under sigmoid; the shares add up to 1, so a constant may be taken off
// G: the mean count is, in whole numbers, which leaves nothing to cancel.
//   w_j = c s_j:            d s_j = c d w_j
//   w_j = c s_j / sum s_i:  share_j (d w_j - sum share d w) c, through log s
// Chosen shares come from their own logits, so that a row whose chosen scores
// are all tiny keeps its precision.
template <typename LT, int PER>
__global__ void __launch_bounds__(256) k_route_backward(const __grid_constant__ GateArgs a) {
  __shared__ float added[8][32 * PER];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = lane * PER, have = a.E - e0;
  float* add = added[warp];
#pragma unroll
  for (int i = 0; i < PER; i++) add[e0 + i] = 0.0f;
  __syncwarp();
  const int64_t first = (int64_t)blockIdx.x * a.per_block;
  const int64_t last = min((int64_t)a.n, first + a.per_block);
  int seq = -1, lo = 0, hi = 0;  // the sequence of g
  int next = 0;                  // the first sequence that may hold the row
  float g[PER];
#pragma unroll
  for (int i = 0; i < PER; i++) g[i] = 0.0f;
  if (a.dloss && a.off) {  // the last sequence that starts at or before the first row
    int b = 0, e = a.S;
    while (e - b > 1) {
      const int m = (b + e) / 2;
      if (a.off[m] <= first) b = m; else e = m;
    }
    next = b;
  }
  for (int64_t row = first + warp; row < last; row += 8) {
    float l[PER], p[PER], rest[PER];
    load_row<LT, PER>(a.logits, row * a.ld + e0, have, a.vec, l);
    int id = -1;
    float dw = 0.0f, my_l = -INFINITY;
    if (a.dw && lane < a.k) {
      id = a.ids[row * a.k + lane];
      if (id < 0 || id >= a.E) id = -1;
      if (id >= 0) {
        dw = a.dw[row * a.k + lane] * a.scale;
        my_l = load_one<LT>(a.logits, row * a.ld + id);
      }
    }
    if (a.dloss && !(seq >= 0 && row >= lo && row < hi)) {
      int found = -1;
      for (; next < a.S; next++) {
        sequence(a, next, lo, hi);
        if (row < lo) break;
        if (row < hi) {
          found = next;
          break;
        }
      }
      seq = found;
      if (seq >= 0) {
        int32_t n[PER];
        int64_t total = 0;
#pragma unroll
        for (int i = 0; i < PER; i++) {
          n[i] = i < have ? a.counts[(int64_t)seq * a.E + e0 + i] : 0;
          total += n[i];
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        const float rows = (float)(hi - lo), f = a.dloss[seq] / ((float)a.k * rows) / rows;
#pragma unroll
        for (int i = 0; i < PER; i++) g[i] = (float)((int64_t)n[i] * a.E - total) * f;
      } else {
#pragma unroll
        for (int i = 0; i < PER; i++) g[i] = 0.0f;
      }
    }
    bool bad = false;
#pragma unroll
    for (int i = 0; i < PER; i++) bad |= l[i] != l[i] || (!a.sigmoid && l[i] == INFINITY);
    const RowSum r = shares<PER>(l, a.sigmoid, p, rest);
    float inner = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; i++) inner += p[i] * g[i];
    inner = warp_sum(inner);
    float part = 0.0f;
    if (a.dw) {
      float s = 0.0f, my_rest = 1.0f;
      if (a.sigmoid) sigmoid_pair(my_l, s, my_rest);
      if (a.renorm) {
        float total = a.sigmoid ? warp_sum(s) : 0.0f;
        if (!a.sigmoid || total < 1e-30f) {
          const float top = warp_max(my_l);
          // (under -745 the scores are 0 in fp64 too, and so are the weights)
          s = my_l == -INFINITY || (!a.sigmoid && top - r.top < -745.0f) ? 0.0f : expf(my_l - top);
          total = warp_sum(s);
        }
        const float share = total == 0.0f ? 0.0f : s / total;
        part = share * (dw - warp_sum(share * dw));
        if (a.sigmoid) part *= my_rest;
      } else if (a.sigmoid) {
        part = s * my_rest * dw;
      } else {
        s = my_l == -INFINITY ? 0.0f : expf(my_l - r.top) / r.z;
        part = s * dw;
        inner += warp_sum(part);
      }
      // to the experts' lanes; an id that stands twice in a row is added twice
      const uint32_t same = __match_any_sync(0xffffffffu, id >= 0 ? id : ~lane);
      if (__any_sync(0xffffffffu, (same & (same - 1)) != 0u)) {
        for (int j = 0; j < a.k; j++) {
          if (lane == j && id >= 0) add[id] += part;
          __syncwarp();
        }
      } else if (id >= 0) {
        add[id] = part;
      }
      __syncwarp();
    }
    const float nan = __int_as_float(0x7fc00000);
    bad = __any_sync(0xffffffffu, bad);
    float d[PER];
#pragma unroll
    for (int i = 0; i < PER; i++) {
      d[i] = p[i] * (g[i] - inner);
      if (a.sigmoid) d[i] *= rest[i];
      if (a.dw) d[i] += add[e0 + i];
      if (bad) d[i] = nan;
    }
    store_row<LT, PER>(a.d, row * a.ldd + e0, have, a.dvec, d);
    if (a.dw) {
      __syncwarp();
      if (id >= 0) add[id] = 0.0f;
      __syncwarp();
    }
  }
}

// A lane's run of PER elements of LT can be moved whole from this matrix.
template <typename LT, int PER>
int whole(const void* p, int64_t ld) {
  const uintptr_t run = std::min<uintptr_t>(16, PER * sizeof(LT));
  return reinterpret_cast<uintptr_t>(p) % run == 0 && ld * (int64_t)sizeof(LT) % (int64_t)run == 0;
}

constexpr int kOneBlockRows = 512;
int balance_chunks(int64_t n, int S) {
  if (n <= kOneBlockRows) return 1;
  const int64_t most = (n + 15) / 16;  // two rows a warp at least
  return (int)std::max<int64_t>(1, std::min<int64_t>(most, (304 + S - 1) / S));
}

template <typename LT, int PER>
cudaError_t run_balance(LaunchCtx lc, GateArgs a) {
  a.vec = whole<LT, PER>(a.logits, a.ld);
  if (a.chunks == 1) return launch_k(lc, k_balance<LT, PER, 16>, dim3(1, a.S), 16 * 32, 0, a);
  cudaError_t e = launch_k(lc, k_balance<LT, PER, 8>, dim3(a.chunks, a.S), 8 * 32, 0, a);
  if (e != cudaSuccess) return e;
  lc.pdl = 1;
  return launch_k(lc, k_balance_finish, dim3(kFinal, a.S), 256, 0, a);
}
template <typename LT, int PER>
cudaError_t run_backward(const LaunchCtx& lc, GateArgs a) {
  a.vec = whole<LT, PER>(a.logits, a.ld);
  a.dvec = whole<LT, PER>(a.d, a.ldd);
  a.per_block = 8;
  return launch_k(lc, k_route_backward<LT, PER>, (unsigned)((a.n + a.per_block - 1) / a.per_block), 256, 0, a);
}
template <typename LT>
cudaError_t run_gate(const LaunchCtx& lc, const GateArgs& a, bool forward) {
  if (a.E <= 64) return forward ? run_balance<LT, 2>(lc, a) : run_backward<LT, 2>(lc, a);
  if (a.E <= 128) return forward ? run_balance<LT, 4>(lc, a) : run_backward<LT, 4>(lc, a);
  return forward ? run_balance<LT, 8>(lc, a) : run_backward<LT, 8>(lc, a);
}

bool misaligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

bool gate_args_ok(int64_t ld, int n, int dtype, int E, int k, int score, int S, const void* off) {
  return n >= 0 && E >= 1 && E <= 256 && k >= 1 && k <= 16 && k <= E && ld >= E &&
         (dtype == AFD_DTYPE_F32 || dtype == AFD_DTYPE_BF16) &&
         (score == AFD_SCORE_SOFTMAX || score == AFD_SCORE_SIGMOID) && S >= 1 && S <= 65535 && (off || S == 1) &&
         !misaligned(off, 4);
}

}  // namespace

extern "C" int64_t afd_balance_workspace(int n_tokens, int num_experts, int n_seqs) {
  if (n_tokens < 0 || num_experts < 1 || num_experts > 256 || n_seqs < 1 || n_seqs > 65535) return -1;
  const int c = balance_chunks(n_tokens, n_seqs);
  return c == 1 ? 0 : (int64_t)n_seqs * c * num_experts * 8;
}

extern "C" int afd_balance_loss(const void* logits, int64_t ld, int n_tokens, int logits_dtype, const int32_t* ids,
                                int num_experts, int topk, int score, const int32_t* seq_offsets, int n_seqs,
                                float* loss, int32_t* counts, void* workspace, int64_t workspace_bytes,
                                void* cuda_stream) {
  if (!gate_args_ok(ld, n_tokens, logits_dtype, num_experts, topk, score, n_seqs, seq_offsets)) return AFD_ERR_ARG;
  const uintptr_t esz = logits_dtype == AFD_DTYPE_F32 ? 4 : 2;
  const int64_t need = afd_balance_workspace(n_tokens, num_experts, n_seqs);
  if ((n_tokens && (!logits || !ids)) || !loss || !counts || misaligned(logits, esz) || misaligned(ids, 4) ||
      misaligned(loss, 4) || misaligned(counts, 4) || (need && (!workspace || misaligned(workspace, 256))))
    return AFD_ERR_ARG;
  if (need > workspace_bytes) return AFD_ERR_CAPACITY;
  const int rc = check_device_ptrs({n_tokens ? logits : nullptr, n_tokens ? ids : nullptr, seq_offsets, loss, counts,
                                    need ? workspace : nullptr});
  if (rc) return rc;
  GateArgs a{};
  a.logits = logits; a.ld = ld; a.ids = ids; a.off = seq_offsets;
  a.n = n_tokens; a.E = num_experts; a.k = topk; a.S = n_seqs; a.sigmoid = score == AFD_SCORE_SIGMOID;
  a.loss = loss; a.counts = counts; a.part = reinterpret_cast<float*>(workspace);
  a.chunks = balance_chunks(n_tokens, n_seqs);
  const LaunchCtx lc{reinterpret_cast<cudaStream_t>(cuda_stream), 0, nullptr};
  if ((logits_dtype == AFD_DTYPE_F32 ? run_gate<float>(lc, a, true) : run_gate<uint16_t>(lc, a, true)) != cudaSuccess) {
    cudaGetLastError();
    return AFD_ERR_CUDA;
  }
  return AFD_OK;
}

extern "C" int afd_route_backward(const void* logits, int64_t ld, int n_tokens, int logits_dtype, const int32_t* ids,
                                  int num_experts, int topk, int score, int renorm, float routed_scaling,
                                  const float* d_weights, const int32_t* seq_offsets, int n_seqs,
                                  const int32_t* counts, const float* d_loss, void* d_logits, int64_t ldd,
                                  void* cuda_stream) {
  if (!gate_args_ok(ld, n_tokens, logits_dtype, num_experts, topk, score, n_seqs, seq_offsets) || ldd < num_experts ||
      (!counts != !d_loss))
    return AFD_ERR_ARG;
  if (n_tokens == 0) return AFD_OK;
  const uintptr_t esz = logits_dtype == AFD_DTYPE_F32 ? 4 : 2;
  if (!logits || !d_logits || (d_weights && !ids) || misaligned(logits, esz) || misaligned(d_logits, esz) ||
      misaligned(ids, 4) || misaligned(d_weights, 4) || misaligned(counts, 4) || misaligned(d_loss, 4))
    return AFD_ERR_ARG;
  const int rc = check_device_ptrs({logits, ids, d_weights, seq_offsets, counts, d_loss, d_logits});
  if (rc) return rc;
  GateArgs a{};
  a.logits = logits; a.ld = ld; a.ids = ids; a.off = seq_offsets;
  a.n = n_tokens; a.E = num_experts; a.k = topk; a.S = n_seqs; a.sigmoid = score == AFD_SCORE_SIGMOID;
  a.counts = const_cast<int32_t*>(counts); a.dw = d_weights; a.dloss = d_loss; a.renorm = renorm != 0;
  a.scale = routed_scaling; a.d = d_logits; a.ldd = ldd;
  const LaunchCtx lc{reinterpret_cast<cudaStream_t>(cuda_stream), 0, nullptr};
  if ((logits_dtype == AFD_DTYPE_F32 ? run_gate<float>(lc, a, false) : run_gate<uint16_t>(lc, a, false)) != cudaSuccess) {
    cudaGetLastError();
    return AFD_ERR_CUDA;
  }
  return AFD_OK;
}
