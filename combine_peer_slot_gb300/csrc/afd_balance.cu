// afd_balance.cu -- the load of the experts and the gradient of the routing
// choice: per-expert counts and a balance loss for each sequence of the batch
// (afd_balance_loss), the gradient of that loss and of the chosen weights with
// respect to the logits (afd_route_backward).
//
//   p_te = softmax(l_t)_e, or s_te / sum_e s_te with s = 1 / (1 + exp(-l))
//   loss_s = E / (k n_s^2) sum_e counts_se sum_{t in s} p_te
//
// A row is LANES lanes of eight neighbouring experts: 8, 16 or 32 lanes for up
// to 64, 128 or 256 experts, so a warp holds 4, 2 or 1 rows and a row's sums
// take 3 to 5 exchanges for four rows at a time (with a warp to a row of 64 the
// exchanges were most of the instructions).  Each pass loads the next row's
// logits before it computes with the present one's.
//
// Measured: 13312 rows of 64 experts, 4 sequences: counts and loss 5 and 4 us
// (sums; their finish, which begins as the sums end), gradient 5.4; of 256 experts
// 8, 6 and 10, with the chosen weights' gradient 14, where the bytes would take 2,
// 4 and 4.  Bound by instructions and the latency of a row's exchanges: some 500 a
// row of 256 (an exponential, a quotient and the products of each expert), at half
// the issue rate with 24 warps an SM.
#include <cooperative_groups.h>

#include "afd_internal.cuh"

namespace {

namespace cg = cooperative_groups;

constexpr int kPer = 8;     // experts of a lane
constexpr int kFinal = 8;   // most CTAs that finish one sequence: 32 experts each
constexpr int kWarps = 16;  // of a block of k_balance
constexpr int kMaxChunks = 320;

struct GateArgs {
  const void* logits;
  int64_t ld;
  const int32_t* ids;
  const int32_t* off;  // [S + 1], or NULL: one sequence of all rows
  int n, E, k, S, sigmoid;
  int vec;             // rows of logits can be loaded 16 bytes at a time
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

// a lane's eight logits of a row; experts past the last one read as -inf
template <typename LT>
__device__ __forceinline__ void load_row(const void* p, int64_t i0, int have, int vec, float (&v)[kPer]) {
  if (vec && have >= kPer) {
    constexpr int kQ = kPer * (int)sizeof(LT) / 16;
    union {
      uint4 q[kQ];
      LT e[kPer];
    } u;
    const uint4* s = reinterpret_cast<const uint4*>(reinterpret_cast<const LT*>(p) + i0);
#pragma unroll
    for (int i = 0; i < kQ; i++) u.q[i] = s[i];
#pragma unroll
    for (int i = 0; i < kPer; i++) v[i] = load_one<LT>(u.e, i);
    return;
  }
#pragma unroll
  for (int i = 0; i < kPer; i++) v[i] = i < have ? load_one<LT>(p, i0 + i) : -INFINITY;
}

template <typename LT>
__device__ __forceinline__ LT rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t rounded<uint16_t>(float v) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

template <typename LT>
__device__ __forceinline__ void store_row(void* p, int64_t i0, int have, int vec, const float (&v)[kPer]) {
  LT* d = reinterpret_cast<LT*>(p) + i0;
  if (vec && have >= kPer) {
    constexpr int kQ = kPer * (int)sizeof(LT) / 16;
    union {
      uint4 q[kQ];
      LT e[kPer];
    } u;
#pragma unroll
    for (int i = 0; i < kPer; i++) u.e[i] = rounded<LT>(v[i]);
#pragma unroll
    for (int i = 0; i < kQ; i++) reinterpret_cast<uint4*>(d)[i] = u.q[i];
    return;
  }
#pragma unroll
  for (int i = 0; i < kPer; i++)
    if (i < have) d[i] = rounded<LT>(v[i]);
}

// over the lanes of a row
template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int LANES>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// two sums, two largest values of a row in the time of one
template <int LANES>
__device__ __forceinline__ void row_sums(float& v, float& w) {
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) {
    const float x = __shfl_xor_sync(0xffffffffu, v, o), y = __shfl_xor_sync(0xffffffffu, w, o);
    v += x;
    w += y;
  }
}
template <int LANES>
__device__ __forceinline__ void row_maxima(float& v, float& w) {
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) {
    const float x = __shfl_xor_sync(0xffffffffu, v, o), y = __shfl_xor_sync(0xffffffffu, w, o);
    v = fmaxf(v, x);
    w = fmaxf(w, y);
  }
}

// s = 1 / (1 + exp(-l)) and 1 - s, each to fp32's precision of itself; the
// denominator is between 1 and 2, where the quotient's short form is within an
// ulp (the full one is a third of the row's instructions)
__device__ __forceinline__ void sigmoid_pair(float l, float& s, float& rest) {
  const float e = expf(-fabsf(l)), r = __fdividef(1.0f, 1.0f + e), q = e * r;
  s = l >= 0.0f ? r : q;  // (NaN: q, which is NaN)
  rest = l >= 0.0f ? q : r;
}

// The exponentials of a row's logits and of its chosen ones (KIDS a lane), each
// relative to their own largest, and their sums: 0 throughout where all are
// -inf.  top: the row's largest.  Scores that are 0 in fp64 too (and
// route_select's weights with them) are none: under softmax those of chosen far
// enough below top, under sigmoid those of logits whose exp(-l) leaves fp64.
constexpr float kSigmoidNone = -709.78271484375f;  // the largest such fp32 value
template <int LANES, int KIDS>
__device__ __forceinline__ void exponentials(const float (&l)[kPer], const float (&cl)[KIDS], int sigmoid,
                                             float (&x)[kPer], float& z, float (&cx)[KIDS], float& cz, float& top) {
  float ctop = -INFINITY;
  top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPer; i++) top = fmaxf(top, l[i]);
#pragma unroll
  for (int j = 0; j < KIDS; j++) ctop = fmaxf(ctop, cl[j]);
  row_maxima<LANES>(top, ctop);
  z = cz = 0.0f;
  const float least = sigmoid ? kSigmoidNone : -INFINITY;  // (NaN is above it, and stays)
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    x[i] = l[i] <= least ? 0.0f : expf(l[i] - top);
    z += x[i];
  }
  const bool none = !sigmoid && ctop - top < -745.0f;
#pragma unroll
  for (int j = 0; j < KIDS; j++) {
    cx[j] = cl[j] <= least || none ? 0.0f : expf(cl[j] - ctop);
    cz += cx[j];
  }
  row_sums<LANES>(z, cz);
}

// A row's shares p, and of its chosen logits cl the scores' shares of the
// chosen (cs; renorm) or the scores; under sigmoid the 1 - s of both as well.
// Scores whose sum nears fp32's smallest number come from logits under -60,
// where s = exp(l) (1 - 1e-26): their shares are the softmax's, of those that
// fp64 holds.
template <int LANES, int KIDS>
__device__ __forceinline__ void shares(const float (&l)[kPer], const float (&cl)[KIDS], int sigmoid, bool renorm,
                                       float (&p)[kPer], float (&rest)[kPer], float (&cs)[KIDS], float (&crest)[KIDS]) {
  float z = 0.0f, cz = 0.0f;
  bool small = false, csmall = false;
  if (sigmoid) {
#pragma unroll
    for (int i = 0; i < kPer; i++) {
      sigmoid_pair(l[i], p[i], rest[i]);
      z += p[i];
    }
#pragma unroll
    for (int j = 0; j < KIDS; j++) {
      sigmoid_pair(cl[j], cs[j], crest[j]);
      cz += cs[j];
    }
    row_sums<LANES>(z, cz);
    small = z < 1e-30f;
    csmall = renorm && cz < 1e-30f;
  }
  if (!sigmoid || __any_sync(0xffffffffu, small || csmall)) {
    float x[kPer], cx[KIDS], xz, cxz, top;
    exponentials<LANES, KIDS>(l, cl, sigmoid, x, xz, cx, cxz, top);
    if (!sigmoid || small) {  // (the warp's other rows keep their sigmoids)
      z = xz;
#pragma unroll
      for (int i = 0; i < kPer; i++) p[i] = x[i];
    }
    if (!sigmoid || csmall) {
      cz = cxz;
#pragma unroll
      for (int j = 0; j < KIDS; j++) {
        cs[j] = cx[j];
        if (!sigmoid && !renorm) cs[j] = cl[j] == -INFINITY ? 0.0f : expf(cl[j] - top) / xz;
      }
    }
  }
  const float inv = z == 0.0f ? 0.0f : 1.0f / z;
#pragma unroll
  for (int i = 0; i < kPer; i++) p[i] *= inv;
  if (renorm) {
    const float cinv = cz == 0.0f ? 0.0f : 1.0f / cz;
#pragma unroll
    for (int j = 0; j < KIDS; j++) cs[j] *= cinv;
  }
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

// E / (k n^2) sum_e counts p
__device__ __forceinline__ float loss_of(const GateArgs& a, int rows, double dot) {
  return rows ? (float)(dot * (double)a.E / ((double)a.k * (double)rows * (double)rows)) : 0.0f;
}

// A sequence's rows are shared by `chunks` blocks of kWarps warps.  One chunk:
// its loss at once; else a block's share of the sums.  Sums of p: a lane's rows
// kRun at a time in fp32, the runs in fp64 (one fp32 chain over all rows of a
// sequence that many others leave one block was 1e-4 off), then the warp's rows
// and the warps in order.  Counts are whole numbers, so their order is free.
// (The runs' sums stay in shared memory: as registers they halve the blocks an SM
// holds, or spill 100 bytes a thread.)
constexpr int kRun = 64;
template <typename LT, int LANES>
__global__ void __launch_bounds__(kWarps * 32) k_balance(const __grid_constant__ GateArgs a) {
  constexpr int kE = LANES * kPer, kAtOnce = 32 / LANES, kIds = LANES < 16 ? 2 : 1;
  __shared__ double runs[kPer][kWarps * 32];                     // each thread's own
  float(*sums)[kE] = reinterpret_cast<float(*)[kE]>(&runs[0][0]);  // [kWarps], in their place afterwards
  __shared__ int32_t cnt[kE];
  __shared__ double dots[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % LANES;
  const int e0 = sub * kPer, have = a.E - e0, s = blockIdx.y, c = blockIdx.x;
  for (int e = threadIdx.x; e < kE; e += kWarps * 32) cnt[e] = 0;
  if (a.chunks > 1) cudaTriggerProgrammaticLaunchCompletion();  // (the second kernel waits for this one's end)
  int lo, hi;
  sequence(a, s, lo, hi);
  __syncthreads();
  float acc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; i++) acc[i] = 0.0f;
  const int64_t step = (int64_t)a.chunks * kWarps * kAtOnce;
  int64_t row = (int64_t)lo + (c * kWarps + warp) * kAtOnce + lane / LANES;
  float next[kPer];
  int nid[kIds];
  auto load = [&](int64_t at) {
    const bool in = at < hi;
    load_row<LT>(a.logits, in ? at * a.ld + e0 : 0, in ? have : 0, a.vec, next);
#pragma unroll
    for (int j = 0; j < kIds; j++) nid[j] = in && sub + j * LANES < a.k ? a.ids[at * a.k + sub + j * LANES] : -1;
  };
  // (the same passes for all rows of the warp: the first one's)
  const int64_t passes = max((int64_t)0, ((int64_t)hi - (row - lane / LANES) + step - 1) / step);
  if (passes) load(row);
  for (int64_t i = 0; i < passes; i++) {
    float l[kPer], p[kPer], rest[kPer];
    int id[kIds];
#pragma unroll
    for (int x = 0; x < kPer; x++) l[x] = next[x];
#pragma unroll
    for (int j = 0; j < kIds; j++) id[j] = nid[j];
    row += step;
    if (i + 1 < passes) load(row);
    const float none[1] = {-INFINITY};
    float cs[1], crest[1];
    shares<LANES, 1>(l, none, a.sigmoid, false, p, rest, cs, crest);
#pragma unroll
    for (int x = 0; x < kPer; x++) acc[x] += p[x];
#pragma unroll
    for (int j = 0; j < kIds; j++)
      if (id[j] >= 0 && id[j] < a.E) atomicAdd(&cnt[id[j]], 1);
    if (i % kRun == kRun - 1) {
#pragma unroll
      for (int x = 0; x < kPer; x++) {
        runs[x][threadIdx.x] = (i == kRun - 1 ? 0.0 : runs[x][threadIdx.x]) + (double)acc[x];
        acc[x] = 0.0f;
      }
    }
  }
  if (passes >= kRun) {
#pragma unroll
    for (int x = 0; x < kPer; x++) acc[x] = (float)(runs[x][threadIdx.x] + (double)acc[x]);
  }
  __syncthreads();
#pragma unroll
  for (int x = 0; x < kPer; x++) {
#pragma unroll
    for (int o = LANES; o < 32; o <<= 1) acc[x] += __shfl_xor_sync(0xffffffffu, acc[x], o);
    if (lane < LANES) sums[warp][e0 + x] = acc[x];
  }
  __syncthreads();
  double dot = 0.0;
  for (int e = threadIdx.x; e < a.E; e += kWarps * 32) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; w++) v += sums[w][e];
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
    for (int w = 0; w < (a.E + 31) / 32; w++) v += dots[w];
    a.loss[s] = loss_of(a, hi - lo, v);
  }
}

// The chunks' sums to counts and loss: a cluster per sequence, CTA q the
// experts [32 q, 32 q + 32), lane = expert, warps stride the chunks, all in a
// fixed order: fp32 over the chunks (at most 10 terms a warp and 32 warps),
// 64 bits over the experts.
__global__ void __launch_bounds__(1024) k_balance_finish(const __grid_constant__ GateArgs a) {
  __shared__ float sums[32][32];
  __shared__ int32_t cnts[32][33];
  __shared__ double dot_of[kFinal];
  cg::cluster_group cluster = cg::this_cluster();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, q = blockIdx.x, s = blockIdx.y;
  const int e = q * 32 + lane;
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // this CTA has started
  cudaGridDependencySynchronize();
  float v = 0.0f;
  int32_t n = 0;
  if (e < a.E) {
    const float* p = a.part + (int64_t)s * a.chunks * a.E + e;
    const int32_t* m = reinterpret_cast<const int32_t*>(a.part) + (int64_t)(a.S + s) * a.chunks * a.E + e;
#pragma unroll
    for (int i = 0; i < kMaxChunks / 32; i++) {
      const int c = warp + i * 32;
      if (c < a.chunks) {
        v += p[(int64_t)c * a.E];
        n += m[(int64_t)c * a.E];
      }
    }
  }
  sums[warp][lane] = v;
  cnts[warp][lane] = n;
  __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // the CTA that is written to has, too
  if (warp == 0) {
    v = 0.0f;
    n = 0;
#pragma unroll
    for (int w = 0; w < 32; w++) {
      v += sums[w][lane];
      n += cnts[w][lane];
    }
    if (e < a.E) a.counts[(int64_t)s * a.E + e] = n;
    double dot = (double)v * (double)n;
#pragma unroll
    for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (lane == 0) *cluster.map_shared_rank(&dot_of[q], 0) = dot;
  }
  cluster.sync();
  if (q == 0 && threadIdx.x == 0) {
    double d = 0.0;
    for (int i = 0; i < (int)gridDim.x; i++) d += dot_of[i];
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
// DW: with the weights' gradient.
template <typename LT, int LANES, bool DW>
__global__ void __launch_bounds__(256, 3) k_route_backward(const __grid_constant__ GateArgs a) {
  constexpr int kE = LANES * kPer, kAtOnce = 32 / LANES, kIds = LANES < 16 ? 2 : 1;
  __shared__ __align__(16) float added[DW ? 8 : 1][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % LANES;
  const int e0 = sub * kPer, have = a.E - e0;
  float* add = added[DW ? warp : 0] + lane / LANES * kE;
  float4* mine = reinterpret_cast<float4*>(add + e0);  // (by fours: by ones, lanes would meet in eight banks)
  if (DW) {
    mine[0] = mine[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    __syncwarp();
  }
  const int64_t first = (int64_t)blockIdx.x * a.per_block;
  const int64_t last = min((int64_t)a.n, first + a.per_block);
  int seq = -1, lo = 0, hi = 0;  // the sequence of g
  int search = 0;                // the first sequence that may hold the row
  float g[kPer];
#pragma unroll
  for (int i = 0; i < kPer; i++) g[i] = 0.0f;
  float next[kPer], ndw[kIds], nl[kIds];
  int nid[kIds];
  auto load = [&](int64_t at) {
    const bool in = at < last;
    load_row<LT>(a.logits, in ? at * a.ld + e0 : 0, in ? have : 0, a.vec, next);
#pragma unroll
    for (int j = 0; j < kIds; j++) {
      int id = -1;
      if (DW && in && sub + j * LANES < a.k) {
        id = a.ids[at * a.k + sub + j * LANES];
        if (id < 0 || id >= a.E) id = -1;
      }
      nid[j] = id;
      ndw[j] = id >= 0 ? a.dw[at * a.k + sub + j * LANES] * a.scale : 0.0f;
      nl[j] = id >= 0 ? load_one<LT>(a.logits, at * a.ld + id) : -INFINITY;
    }
  };
  int64_t row = first + warp * kAtOnce + lane / LANES;
  load(row);
  if (a.dloss && a.off) {  // the last sequence that starts at or before the first row
    if (a.S <= 32) {
      search = __popc(__ballot_sync(0xffffffffu, lane > 0 && lane < a.S && a.off[lane] <= first));
    } else {
      int b = 0, e = a.S;
      while (e - b > 1) {
        const int m = (b + e) / 2;
        if (a.off[m] <= first) b = m; else e = m;
      }
      search = b;
    }
  }
  for (int64_t base = first + warp * kAtOnce; base < last; base += 8 * kAtOnce, row += 8 * kAtOnce) {
    float l[kPer], p[kPer], rest[kPer], dw[kIds], my_l[kIds];
    int id[kIds];
#pragma unroll
    for (int i = 0; i < kPer; i++) l[i] = next[i];
#pragma unroll
    for (int j = 0; j < kIds; j++) {
      id[j] = nid[j];
      dw[j] = ndw[j];
      my_l[j] = nl[j];
    }
    load(row + 8 * kAtOnce);
    const bool in = row < last;
    if (a.dloss && __any_sync(0xffffffffu, in && !(seq >= 0 && row >= lo && row < hi))) {
      int found = -1;
      for (; in && search < a.S; search++) {
        sequence(a, search, lo, hi);
        if (row < lo) break;
        if (row < hi) {
          found = search;
          break;
        }
      }
      seq = found;
      int32_t n[kPer];
      int64_t all = 0;
#pragma unroll
      for (int i = 0; i < kPer; i++) {
        n[i] = seq >= 0 && i < have ? a.counts[(int64_t)seq * a.E + e0 + i] : 0;
        all += n[i];
      }
#pragma unroll
      for (int o = LANES / 2; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
      const float rows = (float)(hi - lo), f = seq >= 0 ? a.dloss[seq] / ((float)a.k * rows) / rows : 0.0f;
#pragma unroll
      for (int i = 0; i < kPer; i++) g[i] = seq >= 0 ? (float)((int64_t)n[i] * a.E - all) * f : 0.0f;
    }
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kPer; i++) bad |= l[i] != l[i] || (!a.sigmoid && l[i] == INFINITY);
    const uint32_t bad_lanes = __ballot_sync(0xffffffffu, bad);
    float cs[kIds], crest[kIds];
    shares<LANES, kIds>(l, my_l, a.sigmoid, DW && a.renorm, p, rest, cs, crest);
    float inner = 0.0f, mean = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; i++) inner += p[i] * g[i];
    if (DW) {
#pragma unroll
      for (int j = 0; j < kIds; j++) mean += cs[j] * dw[j];
      row_sums<LANES>(inner, mean);
      float part[kIds];
#pragma unroll
      for (int j = 0; j < kIds; j++) {
        part[j] = cs[j] * (a.renorm ? dw[j] - mean : dw[j]);
        if (a.sigmoid) part[j] *= crest[j];
      }
      if (!a.sigmoid && !a.renorm) inner += mean;
      // to the experts' lanes; an id that stands twice in a row is added twice
#pragma unroll
      for (int j = 0; j < kIds; j++) {
        const uint32_t same = __match_any_sync(0xffffffffu, id[j] >= 0 ? lane / LANES * 256 + id[j] : ~lane);
        if (__any_sync(0xffffffffu, (same & (same - 1)) != 0u)) {
          for (int x = 0; x < LANES; x++) {
            if (sub == x && id[j] >= 0) add[id[j]] += part[j];
            __syncwarp();
          }
        } else if (id[j] >= 0) {
          add[id[j]] += part[j];
        }
        __syncwarp();
      }
    } else {
      inner = row_sum<LANES>(inner);
    }
    const float nan = __int_as_float(0x7fc00000);
    bad = (bad_lanes >> (lane / LANES * LANES) & (LANES == 32 ? 0xffffffffu : (1u << (LANES & 31)) - 1u)) != 0u;
    float d[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i++) {
      d[i] = p[i] * (g[i] - inner);
      if (a.sigmoid) d[i] *= rest[i];
    }
    if (DW) {
      const float4 u = mine[0], v = mine[1];
      d[0] += u.x; d[1] += u.y; d[2] += u.z; d[3] += u.w;
      d[4] += v.x; d[5] += v.y; d[6] += v.z; d[7] += v.w;
    }
    if (bad) {
#pragma unroll
      for (int i = 0; i < kPer; i++) d[i] = nan;
    }
    if (in) store_row<LT>(a.d, row * a.ldd + e0, have, a.dvec, d);
    if (DW) {
      __syncwarp();
      mine[0] = mine[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      __syncwarp();
    }
  }
}

// rows can be moved 16 bytes at a time, eight elements a lane
int whole(const void* p, int64_t ld, int size) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0;
}

// Blocks that share a sequence.  Up to 512 rows one block each finishes at
// once; more rows take the second kernel, with one pass over its warps' rows to
// each block and at most kMaxChunks shares (two blocks an SM) to add.
constexpr int kOneBlockRows = 512;
int balance_chunks(int64_t n, int E, int S) {
  if (n <= kOneBlockRows) return 1;
  const int at_once = kWarps * (E <= 64 ? 4 : E <= 128 ? 2 : 1);
  return (int)std::max<int64_t>(1, std::min<int64_t>((n + at_once - 1) / at_once, kMaxChunks / S));
}

template <typename LT, int LANES>
cudaError_t run_balance(LaunchCtx lc, GateArgs a) {
  a.vec = whole(a.logits, a.ld, sizeof(LT));
  const cudaError_t e = launch_k(lc, k_balance<LT, LANES>, dim3(a.chunks, a.S), kWarps * 32, 0, a);
  if (e != cudaSuccess || a.chunks == 1) return e;
  lc.pdl = 1;
  const unsigned ctas = a.E <= 32 ? 1 : a.E <= 64 ? 2 : a.E <= 128 ? 4 : 8;
  return launch_k_cluster(lc, k_balance_finish, dim3(ctas, a.S), 1024, 0, ctas, a);
}
template <typename LT, int LANES>
cudaError_t run_backward(const LaunchCtx& lc, GateArgs a) {
  a.vec = whole(a.logits, a.ld, sizeof(LT));
  a.dvec = whole(a.d, a.ldd, sizeof(LT));
  // passes of 8 warps' rows a block: one, and more from where the 456 blocks
  // that run at a time (three an SM) have one each
  const int64_t at_once = 8 * 32 / LANES;
  a.per_block = (int)(at_once * std::max<int64_t>(1, (a.n + 456 * at_once - 1) / (456 * at_once)));
  const unsigned grid = (unsigned)((a.n + a.per_block - 1) / a.per_block);
  return a.dw ? launch_k(lc, k_route_backward<LT, LANES, true>, grid, 256, 0, a)
              : launch_k(lc, k_route_backward<LT, LANES, false>, grid, 256, 0, a);
}
template <typename LT>
cudaError_t run_gate(const LaunchCtx& lc, const GateArgs& a, bool forward) {
  if (a.E <= 64) return forward ? run_balance<LT, 8>(lc, a) : run_backward<LT, 8>(lc, a);
  if (a.E <= 128) return forward ? run_balance<LT, 16>(lc, a) : run_backward<LT, 16>(lc, a);
  return forward ? run_balance<LT, 32>(lc, a) : run_backward<LT, 32>(lc, a);
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
  const int c = balance_chunks(n_tokens, num_experts, n_seqs);
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
  const int64_t T = n_tokens, E = num_experts;
  if (!apart({run_of(loss, n_seqs * 4), run_of(counts, n_seqs * E * 4), run_of(workspace, need)},
             {{logits, ld * (int64_t)esz, E * (int64_t)esz, T}, run_of(ids, T * topk * 4), run_of(seq_offsets, (n_seqs + 1) * 4)}))
    return AFD_ERR_ARG;
  const int rc = check_device_ptrs({n_tokens ? logits : nullptr, n_tokens ? ids : nullptr, seq_offsets, loss, counts,
                                    need ? workspace : nullptr});
  if (rc) return rc;
  GateArgs a{};
  a.logits = logits; a.ld = ld; a.ids = ids; a.off = seq_offsets;
  a.n = n_tokens; a.E = num_experts; a.k = topk; a.S = n_seqs; a.sigmoid = score == AFD_SCORE_SIGMOID;
  a.loss = loss; a.counts = counts; a.part = reinterpret_cast<float*>(workspace);
  a.chunks = balance_chunks(n_tokens, num_experts, n_seqs);
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
  const int64_t T = n_tokens, width = num_experts * (int64_t)esz;
  const bool in_place = d_logits == logits && (ldd == ld || T == 1);
  if (!apart({{d_logits, ldd * (int64_t)esz, width, T}},
             {{in_place ? nullptr : logits, ld * (int64_t)esz, width, T}, run_of(d_weights ? ids : nullptr, T * topk * 4),
              run_of(d_weights, T * topk * 4), run_of(seq_offsets, (n_seqs + 1) * 4),
              run_of(counts, (int64_t)n_seqs * num_experts * 4), run_of(d_loss, n_seqs * 4)}))
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
