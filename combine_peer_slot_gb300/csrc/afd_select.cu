// afd_select.cu -- the routing choice on given logits (afd_route_select):
// softmax or sigmoid scores, a balance bias that takes part in the choice
// only, expert groups, top-k, and the chosen scores as gate weights.
//
//   s_e = softmax(l)_e or 1 / (1 + exp(-l_e)),   c_e = s_e + b_e
//   a group's rank: the sum of its group_top best c; topk_groups groups stay
//   ids = the topk largest c among them, w = s[ids] (/ their sum) * scale
//
// The choice is that of the exact scores: equal c go to the lower index, and
// two values closer than fp32 arithmetic can tell apart are decided in fp64.
// Without a bias c rises with the logit, so the logits themselves are
// compared, which is exact as it stands.  With one, the fp32 choice is taken
// with one candidate more than needed and kept when every gap that decided
// something exceeds what the fp32 errors can add up to (the bounds stand at
// the checks); the other rows, under one in a hundred for logits of unit
// spread, run choose_exact.  Comparing in fp64 throughout would cost the
// fp64 pipe's rate, far below fp32's on this GPU, for every score.
#include "afd_internal.cuh"

namespace {

constexpr int kSelWarps = 8;
constexpr int kMaxPer = 8;  // experts per lane: 32 * 8 = 256

struct SelArgs {
  const void* logits;
  int64_t ld;
  const float* bias;
  int32_t* ids;
  float* w;
  int n, E, k, sigmoid, G, tg, gtop, renorm;
  float scale;
};

// order-preserving map of the fp32 values to unsigned (NaN excluded), with
// -inf at 0x007fffff; 0 is below every value.  v + 0 turns -0 into +0.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float(o ^ ((o & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

template <typename LT>
__device__ __forceinline__ float load_logit(const void* p, int64_t i);
template <>
__device__ __forceinline__ float load_logit<float>(const void* p, int64_t i) {
  return reinterpret_cast<const float*>(p)[i];
}
template <>
__device__ __forceinline__ float load_logit<uint16_t>(const void* p, int64_t i) {
  return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << 16);
}

// One row decided in fp64, by one warp; expert e = lane + 32 m.
template <typename LT>
__device__ __noinline__ void choose_exact(const SelArgs& a, int64_t row, int lane) {
  const int64_t l0 = row * a.ld;
  double top = -INFINITY;
  for (int e = lane; e < a.E; e += 32) top = fmax(top, (double)load_logit<LT>(a.logits, l0 + e));
  for (int o = 16; o; o >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
  double z = 0.0, s[kMaxPer], c[kMaxPer];
  for (int m = 0; m < kMaxPer; m++) {
    const int e = lane + 32 * m;
    s[m] = 0.0;
    c[m] = -INFINITY;
    if (e >= a.E) continue;
    const double l = (double)load_logit<LT>(a.logits, l0 + e);
    if (l == -INFINITY) continue;
    s[m] = a.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - top);
    z += s[m];
  }
  for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  for (int m = 0; m < kMaxPer; m++) {
    const int e = lane + 32 * m;
    if (e >= a.E || load_logit<LT>(a.logits, l0 + e) == -INFINITY) continue;
    if (!a.sigmoid) s[m] /= z;
    c[m] = a.bias ? s[m] + (double)a.bias[e] : (double)load_logit<LT>(a.logits, l0 + e);
  }
  if (a.G > 1) {
    const int per = a.E / a.G;
    double gs = -INFINITY;  // lane g: group g
    for (int g = 0; g < a.G; g++) {
      double m1 = -INFINITY, m2 = -INFINITY;
      for (int m = 0; m < kMaxPer; m++) {
        const int e = lane + 32 * m;
        if (e >= a.E || e / per != g) continue;
        const double v = c[m] > -INFINITY && !a.bias && a.gtop == 2 ? s[m] : c[m];
        m2 = fmax(m2, fmin(m1, v));
        m1 = fmax(m1, v);
      }
      for (int o = 16; o; o >>= 1) {
        const double o1 = __shfl_xor_sync(0xffffffffu, m1, o), o2 = __shfl_xor_sync(0xffffffffu, m2, o);
        m2 = fmax(fmin(m1, o1), fmax(m2, o2));
        m1 = fmax(m1, o1);
      }
      if (lane == g) gs = a.gtop == 2 && m2 > -INFINITY ? m1 + m2 : m1;
    }
    int ahead = 0;
    for (int g = 0; g < a.G; g++) {
      const double v = __shfl_sync(0xffffffffu, gs, g);
      ahead += v > gs || (v == gs && g < lane);
    }
    const uint32_t keep = __ballot_sync(0xffffffffu, lane < a.G && ahead < a.tg);
    for (int m = 0; m < kMaxPer; m++) {
      const int e = lane + 32 * m;
      if (e < a.E && !((keep >> (e / per)) & 1u)) c[m] = -INFINITY;
    }
  }
  int my_id = -1;
  double my_s = 0.0;
  for (int j = 0; j < a.k; j++) {
    double best = -INFINITY, bs = 0.0;
    int bi = 0x7fffffff;
    for (int m = 0; m < kMaxPer; m++)
      if (c[m] > best) {
        best = c[m];
        bs = s[m];
        bi = lane + 32 * m;
      }
    for (int o = 16; o; o >>= 1) {
      const double ov = __shfl_xor_sync(0xffffffffu, best, o), os = __shfl_xor_sync(0xffffffffu, bs, o);
      const int oi = __shfl_xor_sync(0xffffffffu, bi, o);
      if (ov > best || (ov == best && oi < bi)) {
        best = ov;
        bs = os;
        bi = oi;
      }
    }
    if (best == -INFINITY) break;
    if (lane == (bi & 31)) c[bi >> 5] = -INFINITY;
    if (lane == j) {
      my_id = bi;
      my_s = bs;
    }
  }
  if (a.renorm) {
    double sum = my_s;
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (sum > 0.0) my_s /= sum;
  }
  if (lane < a.k) {
    a.ids[row * a.k + lane] = my_id;
    a.w[row * a.k + lane] = (float)(my_s * (double)a.scale);
  }
}

// One warp per row; lane l holds experts [l * PER, (l + 1) * PER), so the
// lowest lane of a tie holds the lowest index.
template <typename LT, int PER>
__global__ void __launch_bounds__(kSelWarps * 32) k_route_select(const __grid_constant__ SelArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kSelWarps + (threadIdx.x >> 5);
  if (row >= a.n) return;
  const int e0 = lane * PER;
  float l[PER], s[PER];
  uint32_t key[PER];  // what is compared; 0: not to be chosen
  float top = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < PER; i++) {
    l[i] = e0 + i < a.E ? load_logit<LT>(a.logits, row * a.ld + e0 + i) : -INFINITY;
    bad |= l[i] != l[i] || (!a.sigmoid && l[i] == INFINITY);
    top = fmaxf(top, l[i]);
  }
  if (!a.sigmoid) {
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  float z = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; i++) {
    s[i] = l[i] == -INFINITY ? 0.0f : a.sigmoid ? 1.0f / (1.0f + expf(-l[i])) : expf(l[i] - top);
    z += s[i];
  }
  if (!a.sigmoid) {
#pragma unroll
    for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
#pragma unroll
    for (int i = 0; i < PER; i++) s[i] = z > 0.0f ? s[i] / z : 0.0f;
  }
  const bool scored = a.bias != nullptr;  // the choice is by score + bias, not by logit
  float c[PER];
#pragma unroll
  for (int i = 0; i < PER; i++) {
    c[i] = l[i];
    if (scored && e0 + i < a.E) {
      const float b = a.bias[e0 + i];
      bad |= b != b;
      if (l[i] > -INFINITY) c[i] = s[i] + b;
    }
    key[i] = c[i] > -INFINITY ? ordered(c[i]) : 0u;
  }
  if (__any_sync(0xffffffffu, bad)) {
    if (lane < a.k) {
      a.ids[row * a.k + lane] = -1;
      a.w[row * a.k + lane] = __int_as_float(0x7fc00000);
    }
    return;
  }
  // What two fp32 values of c may be off together, in units of the largest
  // score (1 for a sigmoid, 1 / z for a softmax) and of |c|.  u = 2^-24: a
  // sigmoid's error is at most 6 u (expf 2 ulp, the sum, the division), a
  // softmax score's 25 u of the largest score (the argument's rounding enters
  // as d u exp(-d) <= 0.37 u, expf 4 u, the sum of 256 terms in 8 + 5 steps
  // and the division under 20 u), adding b another u |c|.  Twice that stays
  // under unit times the larger of the two.
  const float smax = a.sigmoid ? 1.0f : (z > 0.0f ? 1.0f / z : 0.0f);
  const float unit = a.sigmoid ? 9.5367431640625e-07f : 3.814697265625e-06f;  // 2^-20, 2^-18
  bool close = false;
  if (a.G > 1) {
    const int per = a.E / a.G;
    float gs = -INFINITY;  // lane g: group g
    const bool by_score = scored || a.gtop == 2;
    for (int g = 0; g < a.G; g++) {
      float m1 = -INFINITY, m2 = -INFINITY;
      const int lo = g * per, hi = lo + per;
#pragma unroll
      for (int i = 0; i < PER; i++) {
        const bool in = e0 + i >= lo && e0 + i < hi && key[i] != 0u;
        const float v = in ? (scored || !by_score ? c[i] : s[i]) : -INFINITY;
        m2 = fmaxf(m2, fminf(m1, v));
        m1 = fmaxf(m1, v);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const float o1 = __shfl_xor_sync(0xffffffffu, m1, o), o2 = __shfl_xor_sync(0xffffffffu, m2, o);
        m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
        m1 = fmaxf(m1, o1);
      }
      if (lane == g) gs = a.gtop == 2 && m2 > -INFINITY ? m1 + m2 : m1;
    }
    int ahead = 0;
    for (int g = 0; g < a.G; g++) {
      const float v = __shfl_sync(0xffffffffu, gs, g);
      ahead += v > gs || (v == gs && g < lane);
    }
    const uint32_t keep = __ballot_sync(0xffffffffu, lane < a.G && ahead < a.tg);
    if (by_score && a.tg < a.G) {
      // the weakest group kept against the strongest left out; a sum of two
      // has twice the error and its own rounding, and |c| of each term counts
      uint32_t mag = 0u;
#pragma unroll
      for (int i = 0; i < PER; i++)
        if (scored && key[i] != 0u) mag = max(mag, __float_as_uint(fabsf(c[i])));
      const float cmax = __uint_as_float(__reduce_max_sync(0xffffffffu, mag));
      const float in = lane < a.G && ahead == a.tg - 1 ? gs : -INFINITY;
      const float out = lane < a.G && ahead == a.tg ? gs : -INFINITY;
      const float vin = unordered(__reduce_max_sync(0xffffffffu, ordered(in)));
      const float vout = unordered(__reduce_max_sync(0xffffffffu, ordered(out)));
      close = vout > -INFINITY && !(vin - vout > 2.0f * unit * (smax + cmax));
    }
#pragma unroll
    for (int i = 0; i < PER; i++)
      if (e0 + i < a.E && !((keep >> ((e0 + i) / per)) & 1u)) key[i] = 0u;
  }
  // the k best, and one more where fp32 may have erred
  int my_id = -1;
  float my_s = 0.0f, my_l = 0.0f;
  uint32_t my_key = 0u;
  const int rounds = scored ? a.k + 1 : a.k;
  for (int j = 0; j < rounds; j++) {
    uint32_t best = 0u;
#pragma unroll
    for (int i = 0; i < PER; i++) best = max(best, key[i]);
    const uint32_t v = __reduce_max_sync(0xffffffffu, best);
    if (v == 0u) break;
    const int owner = __ffs((int)__ballot_sync(0xffffffffu, best == v)) - 1;
    int id = 0;
    float sv = 0.0f, lv = 0.0f;
    bool done = false;
#pragma unroll
    for (int i = 0; i < PER; i++) {
      const bool hit = !done && key[i] == v;
      if (hit) {
        id = e0 + i;
        sv = s[i];
        lv = l[i];
        if (lane == owner) key[i] = 0u;
      }
      done |= hit;
    }
    id = __shfl_sync(0xffffffffu, id, owner);
    sv = __shfl_sync(0xffffffffu, sv, owner);
    lv = __shfl_sync(0xffffffffu, lv, owner);
    if (lane == j) {
      my_id = id;
      my_s = sv;
      my_l = lv;
      my_key = v;
    }
  }
  if (scored) {
    const uint32_t nk = __shfl_down_sync(0xffffffffu, my_key, 1);
    const float nl = __shfl_down_sync(0xffffffffu, my_l, 1);
    const int ni = __shfl_down_sync(0xffffffffu, my_id, 1);
    if (lane < a.k && my_key != 0u && nk != 0u) {
      const float v0 = unordered(my_key), v1 = unordered(nk);
      // equal logit and bias: equal values, rightly decided by index
      const bool same = my_l == nl && a.bias[my_id] == a.bias[ni];
      close |= !same && !(v0 - v1 > unit * fmaxf(smax, fmaxf(fabsf(v0), fabsf(v1))));
    }
  }
  float sum = lane < a.k ? my_s : 0.0f;
  if (a.renorm) {
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    // scores near fp32's smallest: their ratios need the wider exponent
    close |= sum < 1e-30f && lane < a.k && my_id >= 0;
  }
  if (__any_sync(0xffffffffu, close)) {
    choose_exact<LT>(a, row, lane);
    return;
  }
  if (lane < a.k) {
    a.ids[row * a.k + lane] = my_id;
    a.w[row * a.k + lane] = (a.renorm && sum > 0.0f ? my_s / sum : my_s) * a.scale;
  }
}

int64_t g_select_launches = 0;

template <typename LT>
cudaError_t launch_select(const LaunchCtx& lc, const SelArgs& a) {
  const unsigned grid = (unsigned)((a.n + kSelWarps - 1) / kSelWarps);
  if (a.E <= 64) return launch_k(lc, k_route_select<LT, 2>, grid, kSelWarps * 32, 0, a);
  if (a.E <= 128) return launch_k(lc, k_route_select<LT, 4>, grid, kSelWarps * 32, 0, a);
  return launch_k(lc, k_route_select<LT, 8>, grid, kSelWarps * 32, 0, a);
}

}  // namespace

extern "C" int afd_route_select(const void* logits, int64_t ld, int n_tokens, int logits_dtype,
                                const float* bias, int num_experts, int topk, int score,
                                int n_groups, int topk_groups, int group_top, int renorm,
                                float routed_scaling, int32_t* ids, float* weights,
                                void* cuda_stream) {
  if (n_tokens < 0 || num_experts < 1 || num_experts > 256 || topk < 1 || topk > 16 ||
      topk > num_experts || ld < num_experts ||
      (logits_dtype != AFD_DTYPE_F32 && logits_dtype != AFD_DTYPE_BF16) ||
      (score != AFD_SCORE_SOFTMAX && score != AFD_SCORE_SIGMOID) || n_groups < 1 || n_groups > 32 ||
      num_experts % n_groups || topk_groups < 1 || topk_groups > n_groups ||
      (group_top != 1 && group_top != 2) || topk > topk_groups * (num_experts / n_groups))
    return AFD_ERR_ARG;
  if (n_tokens == 0) return AFD_OK;
  const uintptr_t esz = logits_dtype == AFD_DTYPE_F32 ? 4 : 2;
  if (!logits || !ids || !weights || (reinterpret_cast<uintptr_t>(logits) % esz) ||
      (reinterpret_cast<uintptr_t>(ids) & 3) || (reinterpret_cast<uintptr_t>(weights) & 3) ||
      (reinterpret_cast<uintptr_t>(bias) & 3))
    return AFD_ERR_ARG;
  int rc = check_device_ptrs({logits, bias, ids, weights});
  if (rc) return rc;
  const SelArgs a{logits, ld, bias, ids, weights, n_tokens, num_experts, topk,
                  score == AFD_SCORE_SIGMOID, n_groups, topk_groups, group_top, renorm != 0, routed_scaling};
  const LaunchCtx lc{reinterpret_cast<cudaStream_t>(cuda_stream), 0, &g_select_launches};
  const cudaError_t e = logits_dtype == AFD_DTYPE_F32 ? launch_select<float>(lc, a) : launch_select<uint16_t>(lc, a);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return AFD_ERR_CUDA;
  }
  return AFD_OK;
}
