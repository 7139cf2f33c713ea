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
//
// Measured: 329 rows of 64 experts 2.4 us, the time of a launch; 13312 rows of
// 256 with sigmoid, bias and 8 groups, top 8: 22 us, where the logits' bytes
// would take 2; without groups 18, without bias either 11.  A row is some 1200
// instructions of a warp (scores, keys, sorting network, group ranks, nine
// warp-wide maxima), most of them on the half-rate integer pipe, which bounds
// it; the few rows that need choose_exact add 3 us of its latency at the end,
// or up to 10 where one has its groups to rank as well.
#include "afd_internal.cuh"

namespace {

constexpr int kSelWarps = 8;

struct SelArgs {
  const void* logits;
  int64_t ld;
  const float* bias;
  int32_t* ids;
  float* w;
  int n, E, k, sigmoid, G, tg, gtop, renorm;
  float scale;
  int vec, bvec;  // logits rows / bias: a lane's run of experts can be loaded whole
  int whole;      // an expert group is a power of two of lanes
  uint32_t gmagic;  // 65536 / (experts per group) + 1
};

// expert group of expert e < 256: e / per by multiplication, exact for all
// e, per <= 256 (e gmagic / 65536 is over e / per by at most e / 65536 < 1 / per)
__device__ __forceinline__ int group_of(const SelArgs& a, int e) { return (int)((uint32_t)e * a.gmagic >> 16); }

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

// PER consecutive values, 16 bytes at a time where the row allows it
template <typename LT, int PER>
__device__ __forceinline__ void load_run(const void* base, int64_t i0, int have, bool vec, float (&v)[PER]) {
  if (vec && have >= PER) {
    if (sizeof(LT) == 4) {
      if (PER % 4 == 0) {
#pragma unroll
        for (int i = 0; i < PER / 4; i++) {
          const float4 q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + i0)[i];
          v[4 * i] = q.x; v[4 * i + 1] = q.y; v[4 * i + 2] = q.z; v[4 * i + 3] = q.w;
        }
      } else {
        const float2 q = *reinterpret_cast<const float2*>(reinterpret_cast<const float*>(base) + i0);
        v[0] = q.x; v[1] = q.y;
      }
    } else {
      uint32_t w[PER / 2];
      const uint16_t* p = reinterpret_cast<const uint16_t*>(base) + i0;
      if (PER == 8) {
        const uint4 q = *reinterpret_cast<const uint4*>(p);
        w[0] = q.x; w[1 % (PER / 2)] = q.y; w[2 % (PER / 2)] = q.z; w[3 % (PER / 2)] = q.w;
      } else if (PER == 4) {
        const uint2 q = *reinterpret_cast<const uint2*>(p);
        w[0] = q.x; w[1 % (PER / 2)] = q.y;
      } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
      }
#pragma unroll
      for (int i = 0; i < PER / 2; i++) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < PER; i++) v[i] = i < have ? load_logit<LT>(base, i0 + i) : -INFINITY;
}

// (v, slot) above (w, slot'): the larger key, the lower slot of two equal.
// Packed as key << 32 | (31 - slot) one unsigned comparison says so.
__device__ __forceinline__ void order(uint64_t& a, uint64_t& b) {
  const uint64_t hi = a > b ? a : b, lo = a > b ? b : a;
  a = hi;
  b = lo;
}
template <int PER>
__device__ __forceinline__ void sort_down(uint64_t (&k)[PER]) {
  if (PER == 2) {
    order(k[0], k[1 % PER]);
  } else if (PER == 4) {
    order(k[0], k[1 % PER]); order(k[2 % PER], k[3 % PER]);
    order(k[0], k[2 % PER]); order(k[1 % PER], k[3 % PER]);
    order(k[1 % PER], k[2 % PER]);
  } else {  // Batcher's odd-even merge network for eight: 19 comparisons
    order(k[0], k[1 % PER]); order(k[2 % PER], k[3 % PER]); order(k[4 % PER], k[5 % PER]); order(k[6 % PER], k[7 % PER]);
    order(k[0], k[2 % PER]); order(k[1 % PER], k[3 % PER]); order(k[4 % PER], k[6 % PER]); order(k[5 % PER], k[7 % PER]);
    order(k[1 % PER], k[2 % PER]); order(k[5 % PER], k[6 % PER]);
    order(k[0], k[4 % PER]); order(k[1 % PER], k[5 % PER]); order(k[2 % PER], k[6 % PER]); order(k[3 % PER], k[7 % PER]);
    order(k[2 % PER], k[4 % PER]); order(k[3 % PER], k[5 % PER]);
    order(k[1 % PER], k[2 % PER]); order(k[3 % PER], k[4 % PER]); order(k[5 % PER], k[6 % PER]);
  }
}

__device__ __forceinline__ void merge_two(float& m1, float& m2, int o) {
  const float o1 = __shfl_xor_sync(0xffffffffu, m1, o), o2 = __shfl_xor_sync(0xffffffffu, m2, o);
  m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
  m1 = fmaxf(m1, o1);
}

// Scores that rank.  exp(x) = 2^(x log2 e); both instructions flush results
// under 2^-126 to zero, which the error bounds below, relative to the row's
// largest score, take in.
__device__ __forceinline__ float exp_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}
__device__ __forceinline__ float sigmoid_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.0f + exp_fast(-x)));
  return y;
}

// Contenders of one row: experts whose place fp32 cannot settle, with their
// exact values.
struct Contenders {
  uint8_t id[256];
  int64_t v[256];  // ordered64; first, for groups, the double's bits
};

// What two fp32 values of c may be off together, u = 2^-24: kScoreErr times
// the largest score (1 for a sigmoid, 1 / z for a softmax) and 2 u |c| for
// adding the bias.  exp_fast(x) is off by 2^-22 (4 u) and, from its argument's
// two roundings, by 2 u |x|; the reciprocal by 2 u.  Taken a little larger:
//   sigmoid: s (1 - s) times the exponential's (4 + 2.35 |l|) u, at most
//   1.6 u, the sum 1 + e and the division 5 u: 6.6 u, twice 13.2 u
//   softmax: the exponential's (4 + 3.35 d) u, d = top - l with its rounding,
//   on s = s_max exp(-d): 5.3 u; z over 256 terms 19 u, 1 / z and the product
//   3 u: 27 u, twice 54 u
// The sums of two that rank groups: twice as much, each |c| twice, and the
// two sums' roundings: kGroupErr of the largest score and 8 u max |c|.
constexpr float kU = 5.9604644775390625e-08f;
__device__ __forceinline__ float score_err(int sigmoid) { return sigmoid ? 14.0f * kU : 56.0f * kU; }
__device__ __forceinline__ float group_err(int sigmoid) { return sigmoid ? 28.0f * kU : 112.0f * kU; }

// fp64 to integers of the same order (NaN excluded): compared in a few cycles
// where the fp64 pipe takes tens
__device__ __forceinline__ int64_t ordered64(double v) {
  const int64_t b = __double_as_longlong(v + 0.0);
  return b ^ ((b >> 63) & 0x7fffffffffffffffll);
}

// Every lane's marked experts to the list, ascending; returns their number.
template <int PER>
__device__ __forceinline__ int gather_marked(Contenders& q, uint32_t marked, int e0, int lane) {
  int before = __popc(marked);
  const int mine = before;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  const int n = __shfl_sync(0xffffffffu, before, 31);
  int at = before - mine;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < PER; i++)
    if ((marked >> i) & 1u) q.id[at++] = (uint8_t)(e0 + i);
  __syncwarp();
  return n;
}

// One row decided by its exact scores, by one warp: fp32 picks the few
// contenders (all within the fp32 errors of the border), one lane each
// computes their fp64 values, and those are ranked.  fp64 for every expert
// took 22 to 45 us for the one row in hundreds that needs it, which then was
// the time of the launch.  open: this lane's experts that may be chosen;
// border: the k-th largest fp32 value among them; both only where the groups
// are settled (or there are none), else the groups are ranked here first.
template <typename LT, int PER>
__device__ __noinline__ void choose_exact(const SelArgs& a, int64_t row, int lane, Contenders& q, bool settled,
                                          uint32_t open, float border) {
  const int64_t l0 = row * a.ld;
  const int e0 = lane * PER;
  const bool scored = a.bias != nullptr, by_score = scored || (a.G > 1 && a.gtop == 2);
  float l[PER], s[PER], c[PER];
  float top = -INFINITY, cmax = 0.0f, zf = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; i++) {
    l[i] = e0 + i < a.E ? load_logit<LT>(a.logits, l0 + e0 + i) : -INFINITY;
    top = fmaxf(top, l[i]);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  double z = 1.0;
  if (!a.sigmoid) {
    z = 0.0;
#pragma unroll
    for (int i = 0; i < PER; i++)
      if (l[i] > -INFINITY) z += exp((double)l[i] - (double)top);
#pragma unroll
    for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    zf = (float)z;
  }
  auto score64 = [&](int e) {
    const double x = (double)load_logit<LT>(a.logits, l0 + e);
    return a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - (double)top) / z;
  };
  // exact value of expert e: what experts are chosen by, or (rank) what groups are ranked by
  auto value64 = [&](int e, bool rank) {
    if (scored) return score64(e) + (double)a.bias[e];
    return rank && by_score ? score64(e) : (double)load_logit<LT>(a.logits, l0 + e);
  };
  const float smax = a.sigmoid ? 1.0f : 1.0f / zf;
  uint32_t all = 0u;
#pragma unroll
  for (int i = 0; i < PER; i++) {
    s[i] = 0.0f;
    c[i] = l[i];
    if (l[i] > -INFINITY) {
      if (by_score) s[i] = a.sigmoid ? sigmoid_fast(l[i]) : exp_fast(l[i] - top) * smax;
      if (scored) c[i] = s[i] + a.bias[e0 + i];
      if (c[i] > -INFINITY) {
        all |= 1u << i;
        cmax = fmaxf(cmax, fabsf(c[i]));
      }
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) cmax = fmaxf(cmax, __shfl_xor_sync(0xffffffffu, cmax, o));
  const float tol = by_score ? score_err(a.sigmoid) * smax + (scored ? 2.0f * kU * cmax : 0.0f) : 0.0f;
  if (!settled) {
    open = all;
    if (a.G > 1) {
      uint32_t marked = 0u;
      int grp[PER];
      float rv[PER];  // what groups are ranked by
#pragma unroll
      for (int i = 0; i < PER; i++) {
        grp[i] = (open >> i) & 1u ? group_of(a, e0 + i) : -1;
        rv[i] = scored || !by_score ? c[i] : s[i];
      }
      for (int g = 0; g < a.G; g++) {
        float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
        for (int i = 0; i < PER; i++) {
          const float v = grp[i] == g ? rv[i] : -INFINITY;
          m2 = fmaxf(m2, fminf(m1, v));
          m1 = fmaxf(m1, v);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) merge_two(m1, m2, o);
        const float low = (a.gtop == 2 ? m2 : m1) - tol;
#pragma unroll
        for (int i = 0; i < PER; i++)
          if (grp[i] == g && !(rv[i] < low)) marked |= 1u << i;
      }
      const int n = gather_marked<PER>(q, marked, e0, lane);
      for (int i = lane; i < n; i += 32) q.v[i] = __double_as_longlong(value64(q.id[i], true));
      __syncwarp();
      double gs = -INFINITY;  // lane g: group g
      if (lane < a.G) {
        double m1 = -INFINITY, m2 = -INFINITY;
        for (int i = 0; i < n; i++)
          if (group_of(a, q.id[i]) == lane) {
            const double v = __longlong_as_double(q.v[i]);
            if (v > m1) {
              m2 = m1;
              m1 = v;
            } else if (v > m2) {
              m2 = v;
            }
          }
        gs = a.gtop == 2 && m2 > -INFINITY ? m1 + m2 : m1;
      }
      const int64_t og = ordered64(gs);
      int ahead = 0;
      for (int g = 0; g < a.G; g++) {
        const int64_t v = __shfl_sync(0xffffffffu, og, g);
        ahead += v > og || (v == og && g < lane);
      }
      const uint32_t keep = __ballot_sync(0xffffffffu, lane < a.G && ahead < a.tg);
#pragma unroll
      for (int i = 0; i < PER; i++)
        if (((open >> i) & 1u) && !((keep >> grp[i]) & 1u)) open &= ~(1u << i);
    }
    // the k-th largest fp32 value
    uint32_t left = open, kth = 0u;
    for (int j = 0; j < a.k; j++) {
      uint32_t best = 0u;
      int bi = 0;
#pragma unroll
      for (int i = 0; i < PER; i++) {
        const uint32_t o = (left >> i) & 1u ? ordered(c[i]) : 0u;
        if (o > best) {
          best = o;
          bi = i;
        }
      }
      kth = __reduce_max_sync(0xffffffffu, best);
      if (kth == 0u) break;
      const int owner = __ffs((int)__ballot_sync(0xffffffffu, best == kth)) - 1;
      if (lane == owner) left &= ~(1u << bi);
    }
    border = kth ? unordered(kth) : -INFINITY;
  }
  border -= tol;
  uint32_t marked = 0u;
#pragma unroll
  for (int i = 0; i < PER; i++)
    if (((open >> i) & 1u) && !(c[i] < border)) marked |= 1u << i;
  const int n = gather_marked<PER>(q, marked, e0, lane);
  for (int i = lane; i < n; i += 32) q.v[i] = ordered64(value64(q.id[i], false));
  __syncwarp();
  int my_id = -1;  // lane j: the j-th choice
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    int place = 32;
    if (i < n) {
      const int64_t v = q.v[i];
      place = 0;
      for (int j = 0; j < n; j++) place += q.v[j] > v || (q.v[j] == v && j < i);
    }
    for (int j = 0; j < a.k; j++) {
      const uint32_t who = __ballot_sync(0xffffffffu, place == j);
      if (who && lane == j) my_id = q.id[i0 + __ffs((int)who) - 1];
    }
  }
  // weights in fp32, but where their sum nears fp32's smallest number
  float my_l = 0.0f, my_s = 0.0f;
  if (my_id >= 0) {
    my_l = load_logit<LT>(a.logits, l0 + my_id);
    my_s = a.sigmoid ? 1.0f / (1.0f + expf(-my_l)) : expf(my_l - top) / zf;
  }
  float w = my_s;
  if (a.renorm) {
    float sum = my_s;
#pragma unroll
    for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (__shfl_sync(0xffffffffu, sum, 0) < 1e-30f) {
      const double m = my_id >= 0 ? score64(my_id) : 0.0;
      double all64 = m;
#pragma unroll
      for (int o = 16; o; o >>= 1) all64 += __shfl_xor_sync(0xffffffffu, all64, o);
      w = all64 > 0.0 ? (float)(m / all64) : 0.0f;
    } else {
      w = my_s / sum;
    }
  }
  if (lane < a.k) {
    a.ids[row * a.k + lane] = my_id;
    a.w[row * a.k + lane] = w * a.scale;
  }
}

// One warp per row; lane l holds experts [l * PER, (l + 1) * PER), so the
// lowest lane of a tie holds the lowest index.  A lane sorts its own values
// once; each choice is then one warp-wide integer maximum of the lanes'
// heads, and the owner moves to its next value.
template <typename LT, int PER>
__global__ void __launch_bounds__(kSelWarps * 32, 6) k_route_select(const __grid_constant__ SelArgs a) {
  __shared__ Contenders contenders[kSelWarps];
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kSelWarps + (threadIdx.x >> 5);
  if (row >= a.n) return;
  const int e0 = lane * PER, have = a.E - e0;
  float l[PER], s[PER], c[PER];
  load_run<LT, PER>(a.logits, row * a.ld + e0, have, a.vec, l);
  const bool scored = a.bias != nullptr;  // the choice is by score + bias, not by logit
  const bool by_score = scored || (a.G > 1 && a.gtop == 2);
  float b[PER];
  if (scored) load_run<float, PER>(a.bias, e0, have, a.bvec, b);
  float top = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < PER; i++) {
    bad |= l[i] != l[i] || (!a.sigmoid && l[i] == INFINITY);
    top = fmaxf(top, l[i]);
  }
  // Scores: 2^x and 1 / x as the hardware approximates them (2 and 1 ulp).
  // They rank; the chosen ones' weights are computed again in full.
  float z = 0.0f;
  if (!a.sigmoid) {
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
    for (int i = 0; i < PER; i++) {
      s[i] = l[i] == -INFINITY ? 0.0f : exp_fast(l[i] - top);
      z += s[i];
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if (by_score) {
      const float r = z > 0.0f ? 1.0f / z : 0.0f;
#pragma unroll
      for (int i = 0; i < PER; i++) s[i] *= r;
    }
  } else if (by_score) {
#pragma unroll
    for (int i = 0; i < PER; i++) s[i] = sigmoid_fast(l[i]);  // (-inf: 0)
  }
  uint64_t key[PER];  // high word: what is compared, 0 = not to be chosen
#pragma unroll
  for (int i = 0; i < PER; i++) {
    c[i] = l[i];
    if (scored) {
      bad |= i < have && b[i] != b[i];
      if (l[i] > -INFINITY) c[i] = s[i] + b[i];
    }
    key[i] = c[i] > -INFINITY ? (uint64_t)ordered(c[i]) << 32 | (uint32_t)(31 - i) : 0ull;
  }
  if (__any_sync(0xffffffffu, bad)) {
    if (lane < a.k) {
      a.ids[row * a.k + lane] = -1;
      a.w[row * a.k + lane] = __int_as_float(0x7fc00000);
    }
    return;
  }
  const float smax = a.sigmoid ? 1.0f : (z > 0.0f ? 1.0f / z : 0.0f);
  bool close = false;
  if (a.G > 1) {
    const int per = a.E / a.G;
    float gs;     // this lane's group's rank (whole), or lane g: group g's
    int ahead = 0;
    bool kept;    // whole: this lane's group stays
    uint32_t keep = 0u;
    float in, out;
    if (a.whole) {
      // a group is 1, 2, 4 .. lanes: each lane's own two best, merged over
      // the group's lanes (2 steps for 8 groups of 256, where going through
      // the groups one by one with the whole warp took 8 x 5)
      float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
      for (int i = 0; i < PER; i++) {
        const float v = key[i] != 0ull ? (scored || !by_score ? c[i] : s[i]) : -INFINITY;
        m2 = fmaxf(m2, fminf(m1, v));
        m1 = fmaxf(m1, v);
      }
      const int lanes = per / PER;
      for (int o = 1; o < lanes; o <<= 1) merge_two(m1, m2, o);
      gs = a.gtop == 2 && m2 > -INFINITY ? m1 + m2 : m1;
      const int mine = lane / lanes;
      for (int g = 0; g < a.G; g++) {
        const float v = __shfl_sync(0xffffffffu, gs, (g * lanes) & 31);
        ahead += v > gs || (v == gs && g < mine);
      }
      kept = ahead < a.tg;
      const bool real = mine < a.G;
      in = real && ahead == a.tg - 1 ? gs : -INFINITY;
      out = real && ahead == a.tg ? gs : -INFINITY;
    } else {
      gs = -INFINITY;
      for (int g = 0; g < a.G; g++) {
        float m1 = -INFINITY, m2 = -INFINITY;
        const int lo = g * per, hi = lo + per;
#pragma unroll
        for (int i = 0; i < PER; i++) {
          const bool here = e0 + i >= lo && e0 + i < hi && key[i] != 0ull;
          const float v = here ? (scored || !by_score ? c[i] : s[i]) : -INFINITY;
          m2 = fmaxf(m2, fminf(m1, v));
          m1 = fmaxf(m1, v);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) merge_two(m1, m2, o);
        if (lane == g) gs = a.gtop == 2 && m2 > -INFINITY ? m1 + m2 : m1;
      }
      for (int g = 0; g < a.G; g++) {
        const float v = __shfl_sync(0xffffffffu, gs, g);
        ahead += v > gs || (v == gs && g < lane);
      }
      keep = __ballot_sync(0xffffffffu, lane < a.G && ahead < a.tg);
      kept = false;
      in = lane < a.G && ahead == a.tg - 1 ? gs : -INFINITY;
      out = lane < a.G && ahead == a.tg ? gs : -INFINITY;
    }
    if (by_score && a.tg < a.G) {
      // the weakest group kept against the strongest left out; a sum of two
      // has twice the error and its own rounding, and |c| of each term counts
      uint32_t mag = 0u;
#pragma unroll
      for (int i = 0; i < PER; i++)
        if (scored && key[i] != 0ull) mag = max(mag, __float_as_uint(fabsf(c[i])));
      const float cmax = __uint_as_float(__reduce_max_sync(0xffffffffu, mag));
      const float vin = unordered(__reduce_max_sync(0xffffffffu, ordered(in)));
      const float vout = unordered(__reduce_max_sync(0xffffffffu, ordered(out)));
      close = vout > -INFINITY && !(vin - vout > group_err(a.sigmoid) * smax + 8.0f * kU * cmax);
    }
#pragma unroll
    for (int i = 0; i < PER; i++)
      if (a.whole ? !kept : (i < have && !((keep >> group_of(a, e0 + i)) & 1u))) key[i] = 0ull;
  }
  const bool settled = !__any_sync(0xffffffffu, close);
  uint32_t open = 0u;
  if (scored) {
#pragma unroll
    for (int i = 0; i < PER; i++)
      if (key[i] != 0ull) open |= 1u << i;
  }
  // the k best, and one more where fp32 may have erred: the lanes' sorted
  // values wait in shared memory, a lane's slots in the nibbles of one word
  sort_down<PER>(key);
  uint32_t* heads = reinterpret_cast<uint32_t*>(contenders[threadIdx.x >> 5].v);  // [PER + 1][32]
  uint32_t slots = 0u;
#pragma unroll
  for (int i = 0; i < PER; i++) {
    if (i) heads[i * 32 + lane] = (uint32_t)(key[i] >> 32);
    slots |= (31u - (uint32_t)key[i]) << (4 * i);
  }
  heads[PER * 32 + lane] = 0u;
  uint32_t head = (uint32_t)(key[0] >> 32);
  int at = lane;
  int my_id = -1;
  uint32_t my_key = 0u;
  const int rounds = scored ? a.k + 1 : a.k;
  for (int j = 0; j < rounds; j++) {
    const uint32_t v = __reduce_max_sync(0xffffffffu, head);
    if (v == 0u) break;
    const int owner = __ffs((int)__ballot_sync(0xffffffffu, head == v)) - 1;
    const int id = __shfl_sync(0xffffffffu, e0 + (int)(slots & 15u), owner);
    if (lane == owner) {
      at += 32;
      head = heads[at];
      slots >>= 4;
    }
    if (lane == j) {
      my_id = id;
      my_key = v;
    }
  }
  float my_l = 0.0f, my_s = 0.0f;
  if (my_id >= 0) {
    my_l = load_logit<LT>(a.logits, row * a.ld + my_id);
    my_s = a.sigmoid ? 1.0f / (1.0f + expf(-my_l)) : expf(my_l - top) / z;
  }
  if (scored) {
    auto clear = [&](float v0, float v1) {
      return v0 - v1 > score_err(a.sigmoid) * smax + 2.0f * kU * fmaxf(fabsf(v0), fabsf(v1));
    };
    const uint32_t nk = __shfl_down_sync(0xffffffffu, my_key, 1);
    const float nl = __shfl_down_sync(0xffffffffu, my_l, 1);
    const int ni = __shfl_down_sync(0xffffffffu, my_id, 1);
    bool twins = false;  // the last choice and the first one left out have equal logit and bias
    if (lane < a.k && my_key != 0u && nk != 0u && !clear(unordered(my_key), unordered(nk))) {
      // equal logit and bias: equal values, rightly decided by index
      const bool equal = my_l == nl && a.bias[my_id] == a.bias[ni];
      close |= !equal;
      twins = equal && lane == a.k - 1;
    }
    // The index decides between the two, but a third that fp32 cannot tell from
    // them may be larger than both: on down the order to a value clear of theirs.
    if (__any_sync(0xffffffffu, twins)) {
      const float kv = unordered(__shfl_sync(0xffffffffu, my_key, a.k - 1));
      const float kl = __shfl_sync(0xffffffffu, my_l, a.k - 1);
      const float kb = a.bias[__shfl_sync(0xffffffffu, my_id, a.k - 1)];
      for (;;) {
        const uint32_t v = __reduce_max_sync(0xffffffffu, head);
        if (v == 0u || clear(kv, unordered(v))) break;
        const int owner = __ffs((int)__ballot_sync(0xffffffffu, head == v)) - 1;
        const int id = __shfl_sync(0xffffffffu, e0 + (int)(slots & 15u), owner);
        if (load_logit<LT>(a.logits, row * a.ld + id) != kl || a.bias[id] != kb) {
          close = true;
          break;
        }
        if (lane == owner) {
          at += 32;
          head = heads[at];
          slots >>= 4;
        }
      }
    }
  }
  float sum = lane < a.k ? my_s : 0.0f;
  if (a.renorm) {
#pragma unroll
    for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);  // k <= 16: lanes 0 .. 15
    // scores near fp32's smallest: their ratios need the wider exponent
    close |= sum < 1e-30f && lane < a.k && my_id >= 0;
  }
  if (__any_sync(0xffffffffu, close)) {
    const uint32_t kth = __shfl_sync(0xffffffffu, my_key, a.k - 1);
    choose_exact<LT, PER>(a, row, lane, contenders[threadIdx.x >> 5], scored && settled, open,
                          kth ? unordered(kth) : -INFINITY);
    return;
  }
  if (lane < a.k) {
    a.ids[row * a.k + lane] = my_id;
    a.w[row * a.k + lane] = (a.renorm && sum > 0.0f ? my_s / sum : my_s) * a.scale;
  }
}

template <typename LT, int PER>
cudaError_t launch_per(const LaunchCtx& lc, SelArgs a) {
  const unsigned grid = (unsigned)((a.n + kSelWarps - 1) / kSelWarps);
  const uintptr_t run = std::min<uintptr_t>(16, PER * sizeof(LT)), brun = std::min<uintptr_t>(16, PER * 4);
  a.vec = reinterpret_cast<uintptr_t>(a.logits) % run == 0 && a.ld * (int64_t)sizeof(LT) % (int64_t)run == 0;
  a.bvec = reinterpret_cast<uintptr_t>(a.bias) % brun == 0;
  const int per = a.E / a.G, lanes = per / PER;
  a.gmagic = 65536u / (uint32_t)per + 1u;
  a.whole = per % PER == 0 && (lanes & (lanes - 1)) == 0;
  return launch_k(lc, k_route_select<LT, PER>, grid, kSelWarps * 32, 0, a);
}
template <typename LT>
cudaError_t launch_select(const LaunchCtx& lc, const SelArgs& a) {
  return a.E <= 64 ? launch_per<LT, 2>(lc, a) : a.E <= 128 ? launch_per<LT, 4>(lc, a) : launch_per<LT, 8>(lc, a);
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
                  score == AFD_SCORE_SIGMOID, n_groups, topk_groups, group_top, renorm != 0, routed_scaling, 0, 0, 0, 0};
  const LaunchCtx lc{reinterpret_cast<cudaStream_t>(cuda_stream), 0, nullptr};
  const cudaError_t e = logits_dtype == AFD_DTYPE_F32 ? launch_select<float>(lc, a) : launch_select<uint16_t>(lc, a);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return AFD_ERR_CUDA;
  }
  return AFD_OK;
}
