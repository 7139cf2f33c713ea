// afd_mx4_gemm.cu -- the grouped MXFP4 product on one SM per tile:
// tcgen05.mma kind::mxf4 (e2m1 x e2m1, one e8m0 scale per 32 columns of each
// operand, fp32 accumulate in TMEM).
//
//   y[r, m] = sum_k x[r, k] w[g(r), m, k]     x = code * 2^(scale - 127)
//
// A unit is 128 weight rows x one token tile of one group.  The weight rows
// are the MMA's M side, the tokens its N side, so a group of few tokens
// takes a narrow instruction and not a mostly empty 128-row one.  Per stage
// of 256 columns a CTA takes 17 KB of weight (codes and scales in one bulk
// copy), the tokens' codes by TMA (128-byte swizzle) and their scales, which
// two warps gather from the plain rows into the image tcgen05.cp spreads
// over the lanes: a group's rows start anywhere, so the tiled image could
// not be laid out before the groups are known.
//
// Warps: 0 copies, 1 MMA, 2-3 token scales, 4-11 epilogue.  All waits are
// bounded.
#include "afd_mx4.cuh"

#include <cudaTypedefs.h>

#include <cstdio>
#include <mutex>

namespace {

__device__ int32_t g_mx4_status;  // calls without a context

constexpr int BK = 256;               // columns per stage
constexpr int A_BYTES = 2 * kMx4BlkBytes;
constexpr int EPI_WARPS = 8;
constexpr int NUM_THREADS = 128 + EPI_WARPS * 32;
constexpr int EPI_PITCH_SWIGLU = 48;
constexpr int EPI_PITCH_BF16 = 80;
constexpr int EPI_BUF_BYTES = 32 * EPI_PITCH_BF16;
constexpr int MAX_GROUPS = 257;       // 256 experts and the shared rows
constexpr uint64_t kTimeoutNs = 2000000000ull;

template <int BN>
struct Ring {
  static constexpr int STAGES = BN > 64 ? 4 : 7;
  static constexpr int NB = (BN + 127) / 128;            // 128-row scale images per 128 columns
  static constexpr int B_BYTES = BN * (BK / 2);
  static constexpr int S_BYTES = 2 * NB * 512;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + S_BYTES;
  // TMEM columns: two accumulators, then per stage the weight scales (2 x 4)
  // and the token scales (2 x 4 NB)
  static constexpr int SF_COLS = 8 + 8 * NB;
  static constexpr int SF_BASE = 2 * BN;
  static constexpr int TMEM_COLS = SF_BASE + STAGES * SF_COLS <= 256 ? 256 : 512;
  static_assert(SF_BASE + STAGES * SF_COLS <= TMEM_COLS, "TMEM columns");
  static_assert(STAGE_BYTES % 1024 == 0 && A_BYTES % 1024 == 0, "swizzle alignment");
  struct Tail {
    uint64_t full[STAGES];
    uint64_t empty[STAGES];
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
    int tile0[MAX_GROUPS + 1];  // first unit of each group
    int row0[MAX_GROUPS];
    int rows[MAX_GROUPS];
    int wsum[NUM_THREADS / 32];
  };
  static constexpr size_t kEpiOffset = ((size_t)STAGES * STAGE_BYTES + sizeof(Tail) + 127) / 128 * 128;
  static constexpr size_t kSmemBytes = 1024 + kEpiOffset + (size_t)EPI_WARPS * EPI_BUF_BYTES;
  static_assert(kSmemBytes <= 232448, "over the per-CTA shared memory limit");
};

// matrix descriptors: K-major operand tiles with the 128-byte swizzle (rows
// of 128 bytes, groups of 8 rows 1024 bytes apart) and the 64-byte one (rows
// of 64 bytes, 512 apart); a scale image without swizzle (8 x 16-byte core
// matrices 128 bytes apart)
__device__ __forceinline__ uint64_t desc_of(uint32_t saddr, uint32_t sbo, uint32_t layout) {
  return (uint64_t)((saddr & 0x3FFFF) >> 4) | (uint64_t)1 << 16 | (uint64_t)(sbo >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)layout << 61;
}
__device__ __forceinline__ uint64_t desc_tokens(uint32_t saddr) { return desc_of(saddr, 1024, 2); }
__device__ __forceinline__ uint64_t desc_weight(uint32_t saddr) { return desc_of(saddr, 512, 4); }
__device__ __forceinline__ uint64_t desc_scales(uint32_t saddr) { return desc_of(saddr, 128, 0); }

// kind::mxf4: A and B e2m1 (format 1), e8m0 scales (bit 23), K = 64, M = 128;
// sf: the first of the two scale bytes used of each lane's four (0 or 2)
__device__ __forceinline__ uint32_t idesc_mx4(int n, int sf) {
  return (uint32_t)sf << 4 | 1u << 7 | 1u << 10 | (uint32_t)(n >> 3) << 17 | 1u << 23 | (uint32_t)(128 >> 4) << 24 |
         (uint32_t)sf << 29;
}
__device__ __forceinline__ void mma_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p; }"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}
// 32 lanes x 16 bytes of shared memory into four TMEM columns, the same for
// each quarter of the lanes
__device__ __forceinline__ void cp_scales(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint64_t deadline,
                                         int32_t* status) {
  uint32_t spins = 0;
  while (!mbar_try_wait(bar, parity)) {
    if ((++spins & 255u) == 0) {
      if (*abort_flag) return false;
      if (globaltimer_ns() > deadline) {
        *abort_flag = 1;
        set_error(status, AFD_ERR_TIMEOUT);
        return false;
      }
    }
  }
  return true;
}

__device__ __forceinline__ float silu_f(float g) { return __fdividef(g, 1.0f + __expf(-g)); }

struct Unit {
  int group, kind, mt, rows, n_mma;
  int64_t row;  // first row of the token tile
};

template <int BN>
__device__ __forceinline__ Unit decode_unit(const Mx4GemmArgs& a, const typename Ring<BN>::Tail* T, int ngroups,
                                            int unit) {
  int lo = 0, hi = ngroups - 1;
  while (lo < hi) {  // last group whose first unit is <= unit (empty groups share it with the next)
    const int mid = (lo + hi + 1) >> 1;
    if (T->tile0[mid] <= unit) lo = mid; else hi = mid - 1;
  }
  Unit t;
  t.group = lo;
  t.kind = lo == a.n_groups;
  const int u = unit - T->tile0[lo];
  const int n_tiles = (T->rows[lo] + BN - 1) / BN;
  const int m_tiles = mx4_tiles(a.M[t.kind], a.swiglu);
  int nt;
  if (BN == 64) {  // the weights stream from HBM: a weight tile's token tiles side by side, for L2
    nt = u % n_tiles;
    t.mt = u / n_tiles;
  } else {         // the units running at once share token tiles
    t.mt = u % m_tiles;
    nt = u / m_tiles;
  }
  t.row = (int64_t)T->row0[lo] + (int64_t)nt * BN;
  t.rows = min(BN, T->rows[lo] - nt * BN);
  t.n_mma = (t.rows + 15) & ~15;
  return t;
}

// A lane's scale bytes of one stage: rows lane + 32 i, eight bytes each
// (columns kb * 256 ..), zero past the row's end or the last row.
template <int BN>
__device__ __forceinline__ void load_scales(const uint8_t* xs, int64_t x_rows, int pitch, int64_t row0, int kb,
                                            int lane, uint32_t (&v)[BN / 32][2]) {
  const int b0 = kb * 8;
#pragma unroll
  for (int i = 0; i < BN / 32; i++) {
    v[i][0] = v[i][1] = 0u;
    const int64_t row = row0 + lane + 32 * i;
    if (row >= x_rows) continue;
    const uint8_t* p = xs + row * pitch + b0;
    if ((pitch & 3) == 0) {  // rows start on 4 bytes
      v[i][0] = *reinterpret_cast<const uint32_t*>(p);
      if (b0 + 4 < pitch) v[i][1] = *reinterpret_cast<const uint32_t*>(p + 4);
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++)
        if (b0 + j < pitch) v[i][j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
    }
  }
}

template <int BN>
__global__ void __launch_bounds__(NUM_THREADS, 1) k_mx4_gemm(const __grid_constant__ Mx4GemmArgs a) {
  using R = Ring<BN>;
  constexpr int STAGES = R::STAGES;
  constexpr int NB = R::NB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  typename R::Tail* tail = reinterpret_cast<typename R::Tail*>(smem + (size_t)STAGES * R::STAGE_BYTES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t* status = a.status ? a.status : &g_mx4_status;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; s++) {
      mbar_init(smem_u32(&tail->full[s]), 2);  // the copies' producer, the scale warp
      mbar_init(smem_u32(&tail->empty[s]), 1);
    }
    for (int b = 0; b < 2; b++) {
      mbar_init(smem_u32(&tail->tfull[b]), 1);
      mbar_init(smem_u32(&tail->tempty[b]), EPI_WARPS);
    }
    mbar_init(smem_u32(&tail->drain), 1);
    tail->abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tail->tmem_base)),
                 "r"(R::TMEM_COLS));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  grid_dep_wait();
  grid_dep_launch();
  // the groups: rows clamped to those there are, units counted
  const int ngroups = a.n_groups + a.has_shared;
  int mine = 0;
  if (threadIdx.x < ngroups) {
    const int g = threadIdx.x;
    const int kind = g == a.n_groups;
    int lo = 0, hi = (int)a.x_rows[1];
    if (!kind) {
      lo = (int)min(max((int64_t)a.offsets[g], (int64_t)0), a.x_rows[0]);
      hi = (int)min(max((int64_t)a.offsets[g + 1], (int64_t)lo), a.x_rows[0]);
    }
    tail->row0[g] = lo;
    tail->rows[g] = hi - lo;
    mine = (hi - lo + BN - 1) / BN * mx4_tiles(a.M[kind], a.swiglu);
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) tail->wsum[warp] = incl;
  __syncthreads();
  int before = 0, total = 0;
  for (int w = 0; w < NUM_THREADS / 32; w++) {
    if (w < warp) before += tail->wsum[w];
    total += tail->wsum[w];
  }
  if (threadIdx.x < ngroups) tail->tile0[threadIdx.x] = before + incl - mine;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tail->tmem_base;
  const uint64_t deadline = globaltimer_ns() + kTimeoutNs;
  volatile int* abort_flag = &tail->abort_flag;
  const uint32_t smem_base = smem_u32(smem);

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------ copies
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int unit = blockIdx.x; unit < total && ok; unit += gridDim.x) {
        const Unit t = decode_unit<BN>(a, tail, ngroups, unit);
        const int nk = mx4_kblocks(a.K[t.kind]);
        const int m_tiles = mx4_tiles(a.M[t.kind], a.swiglu);
        const uint8_t* w =
            a.w[t.kind] + ((int64_t)(t.kind ? 0 : t.group) * m_tiles + t.mt) * nk * (int64_t)kMx4BlkBytes;
        for (int kb = 0; kb * 2 < nk; kb++) {
          if (!wait_bar(smem_u32(&tail->empty[s]), ph ^ 1, abort_flag, deadline, status)) { ok = false; break; }
          const uint32_t full = smem_u32(&tail->full[s]);
          const uint32_t a_bytes = min(2, nk - 2 * kb) * kMx4BlkBytes;
          mbar_expect_tx(full, a_bytes + R::B_BYTES);
          const uint32_t sa = smem_base + s * R::STAGE_BYTES;
          bulk_load(sa, w + (int64_t)kb * 2 * kMx4BlkBytes, a_bytes, full);
          tma_load_2d(sa + A_BYTES, &a.tmX[t.kind], kb * (BK / 2), (int)t.row, full);
          if (++s == STAGES) { s = 0; ph ^= 1; }
        }
      }
      // a wait gave up: the copies in flight land before the CTA leaves
      if (!ok)
        for (int i = 0; i < 10000; i++) __nanosleep(1000);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ------------------------------ MMA issuer
      int s = 0;
      uint32_t ph = 0;
      int acc = 0;
      uint32_t acc_ph = 0;
      bool ok = true;
      for (int unit = blockIdx.x; unit < total && ok; unit += gridDim.x) {
        const Unit t = decode_unit<BN>(a, tail, ngroups, unit);
        const int K = a.K[t.kind];
        const uint32_t id0 = idesc_mx4(t.n_mma, 0), id2 = idesc_mx4(t.n_mma, 2);
        if (!wait_bar(smem_u32(&tail->tempty[acc]), acc_ph ^ 1, abort_flag, deadline, status)) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(acc * BN);
        for (int kb = 0; kb * BK < K; kb++) {
          if (!wait_bar(smem_u32(&tail->full[s]), ph, abort_flag, deadline, status)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = smem_base + s * R::STAGE_BYTES;
          const uint32_t sb = sa + A_BYTES, ss = sb + R::B_BYTES;
          const uint32_t sf = tmem + (uint32_t)(R::SF_BASE + s * R::SF_COLS);
          const int steps = min(4, (K - kb * BK + 63) / 64);
          for (int c = 0; c < (steps + 1) / 2; c++) {  // 128 columns: scales, then two MMAs
            cp_scales(sf + 4 * c, desc_scales(sa + c * kMx4BlkBytes + kMx4BlkCodes));
#pragma unroll
            for (int b = 0; b < NB; b++)
              cp_scales(sf + 8 + 4 * (c * NB + b), desc_scales(ss + (c * NB + b) * 512));
          }
          for (int kk = 0; kk < steps; kk++) {
            const int c = kk >> 1, o = kk & 1;
            mma_mx4(d, desc_weight(sa + c * kMx4BlkBytes + o * 32), desc_tokens(sb + kk * 32), o ? id2 : id0,
                    sf + 4 * c, sf + 8 + 4 * c * NB, (kb | kk) != 0);
          }
          tc_commit(smem_u32(&tail->empty[s]));
          if (++s == STAGES) { s = 0; ph ^= 1; }
        }
        if (!ok) break;
        tc_commit(smem_u32(&tail->tfull[acc]));
        if (++acc == 2) { acc = 0; acc_ph ^= 1; }
      }
      // every issued MMA completes before TMEM is released
      tc_commit(smem_u32(&tail->drain));
      const uint64_t dl = globaltimer_ns() + 100000000ull;
      while (!mbar_try_wait(smem_u32(&tail->drain), 0) && globaltimer_ns() < dl) {}
    }
  } else if (warp < 4) {
    // ------------------------------ token scales: the two warps take stages in turn
    int unit = blockIdx.x, kb = 0;
    Unit t;
    int nkb = 0;
    if (unit < total) {
      t = decode_unit<BN>(a, tail, ngroups, unit);
      nkb = (a.K[t.kind] + BK - 1) / BK;
    }
    auto advance = [&]() {
      if (++kb < nkb) return;
      kb = 0;
      unit += gridDim.x;
      if (unit >= total) return;
      t = decode_unit<BN>(a, tail, ngroups, unit);
      nkb = (a.K[t.kind] + BK - 1) / BK;
    };
    if (warp == 3 && unit < total) advance();
    uint32_t v[BN / 32][2];
    if (unit < total) load_scales<BN>(a.xs[t.kind], a.x_rows[t.kind], a.K[t.kind] / 32, t.row, kb, lane, v);
    int it = warp - 2;
    while (unit < total) {
      const int s = it % STAGES;
      const uint32_t ph = (uint32_t)(it / STAGES) & 1u;
      bool ok = wait_bar(smem_u32(&tail->empty[s]), ph ^ 1, abort_flag, deadline, status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      uint8_t* ss = smem + (size_t)s * R::STAGE_BYTES + A_BYTES + R::B_BYTES;
#pragma unroll
      for (int c = 0; c < 2; c++)
#pragma unroll
        for (int b = 0; b < NB; b++) {
          uint32_t q[4];
#pragma unroll
          for (int j = 0; j < 4; j++) q[j] = 4 * b + j < BN / 32 ? v[4 * b + j < BN / 32 ? 4 * b + j : 0][c] : 0u;
          *reinterpret_cast<uint4*>(ss + (c * NB + b) * 512 + lane * 16) = make_uint4(q[0], q[1], q[2], q[3]);
        }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&tail->full[s]));
      advance();
      if (unit < total) advance();
      if (unit < total) load_scales<BN>(a.xs[t.kind], a.x_rows[t.kind], a.K[t.kind] / 32, t.row, kb, lane, v);
      it += 2;
    }
  } else {
    // ------------------------------ epilogue (warps 4..11)
    const int q = warp & 3;
    const int half = (warp - 4) >> 2;
    uint8_t* ebuf = smem + R::kEpiOffset + (size_t)(warp - 4) * EPI_BUF_BYTES;
    const bool lo = lane < 16;
    int acc = 0;
    uint32_t acc_ph = 0;
    for (int unit = blockIdx.x; unit < total; unit += gridDim.x) {
      const Unit t = decode_unit<BN>(a, tail, ngroups, unit);
      bool ok = wait_bar(smem_u32(&tail->tfull[acc]), acc_ph, abort_flag, deadline, status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN);
      const int kind = t.kind;
      const int64_t ldo = a.ldo[kind];
      if (a.swiglu) {
        const int col0 = t.mt * 64 + q * 16, I = a.M[kind] / 2;
        for (int c0 = half * 32; c0 < t.rows; c0 += 64) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(taddr + (uint32_t)c0, v);
          tmem_ld_wait();
          uint16_t* sb = reinterpret_cast<uint16_t*>(ebuf);
#pragma unroll
          for (int j = 0; j < 16; j++) {
            const float x = __uint_as_float(v[j]), y = __uint_as_float(v[16 + j]);
            const float recv = __shfl_xor_sync(0xffffffffu, lo ? y : x, 16);
            const float g = lo ? x : recv;
            const float u = lo ? recv : y;
            const __nv_bfloat16 hv = __float2bfloat16_rn(silu_f(g) * u);
            const int tok = lo ? j : 16 + j;
            sb[(tok * EPI_PITCH_SWIGLU + (lo ? 0 : 32)) / 2 + (lane & 15)] = *reinterpret_cast<const uint16_t*>(&hv);
          }
          __syncwarp();
          const int r = c0 + lane;
          if (r < t.rows) {
            const uint4* src = reinterpret_cast<const uint4*>(ebuf + lane * EPI_PITCH_SWIGLU + (lo ? 0 : 32));
            uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out[kind]) + (t.row + r) * ldo + col0);
            if (col0 + 8 <= I) dst[0] = src[0];
            if (col0 + 16 <= I) dst[1] = src[1];
          }
          __syncwarp();
        }
      } else {
        const int col0 = t.mt * 128 + q * 32, M = a.M[kind];
        const int fmt = a.fmt[kind];
        for (int c0 = half * 32; c0 < t.rows; c0 += 64) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(taddr + (uint32_t)c0, v);
          tmem_ld_wait();
          if (fmt == OUT_F32) {
            if (col0 + lane < M) {
              float* dst = reinterpret_cast<float*>(a.out[kind]) + (t.row + c0) * ldo + col0 + lane;
#pragma unroll
              for (int c = 0; c < 32; c++)
                if (c0 + c < t.rows) dst[(int64_t)c * ldo] = __uint_as_float(v[c]);
            }
          } else if (fmt == OUT_Y24) {
            if (col0 + lane < M) {
              uint16_t* dh = reinterpret_cast<uint16_t*>(a.out[kind]) + (t.row + c0) * ldo + col0 + lane;
              uint8_t* dl = a.out_lo[kind] + (t.row + c0) * ldo + col0 + lane;
#pragma unroll
              for (int c = 0; c < 32; c++)
                if (c0 + c < t.rows) {
                  const uint32_t b24 = y24_encode(__uint_as_float(v[c]));
                  dh[(int64_t)c * ldo] = (uint16_t)(b24 >> 8);
                  dl[(int64_t)c * ldo] = (uint8_t)(b24 & 0xffu);
                }
            }
          } else {
#pragma unroll
            for (int c = 0; c < 32; c++) {
              const __nv_bfloat16 yv = __float2bfloat16_rn(__uint_as_float(v[c]));
              *reinterpret_cast<uint16_t*>(ebuf + c * EPI_PITCH_BF16 + lane * 2) =
                  *reinterpret_cast<const uint16_t*>(&yv);
            }
            __syncwarp();
            const int r = c0 + lane;
            if (r < t.rows) {
              const uint4* src = reinterpret_cast<const uint4*>(ebuf + lane * EPI_PITCH_BF16);
              uint4* dst =
                  reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out[kind]) + (t.row + r) * ldo + col0);
#pragma unroll
              for (int x = 0; x < 4; x++)
                if (col0 + 8 * x + 8 <= M) dst[x] = src[x];
            }
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&tail->tempty[acc]));
      if (++acc == 2) { acc = 0; acc_ph ^= 1; }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(R::TMEM_COLS));
  }
}

template <int BN>
cudaError_t launch_variant(const LaunchCtx& lc, const Mx4GemmArgs& a, int64_t units) {
  static std::atomic<int> attr_done[kMaxCachedDevices];
  const cudaError_t e = smem_attr_once(k_mx4_gemm<BN>, (int)Ring<BN>::kSmemBytes, attr_done);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(units, lc.num_sms));
  return launch_k(lc, k_mx4_gemm<BN>, grid, NUM_THREADS, Ring<BN>::kSmemBytes, a);
}

constexpr int kWide = 192, kNarrow = 64;

}  // namespace

// Token tile of a product over `rows` rows in `groups` groups: 64 rows when
// the groups average 48 or fewer (the weights' bytes bound it: a deeper ring
// of narrower stages), else 192 (two accumulators and the scales fill the
// 512 TMEM columns).
int mx4_token_tile(int64_t rows, int groups) { return rows <= 48 * (int64_t)groups ? kNarrow : kWide; }

cudaError_t launch_mx4_gemm(const LaunchCtx& lc, const Mx4GemmArgs& a, int bn, int64_t units) {
  return bn == kNarrow ? launch_variant<kNarrow>(lc, a, units) : launch_variant<kWide>(lc, a, units);
}

int encode_mx4_rows(CUtensorMap* m, const void* codes, int64_t rows, int K, int bn) {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  std::call_once(once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  if (!encode) return AFD_ERR_CUDA;
  const cuuint64_t dims[2] = {(cuuint64_t)(K / 2), (cuuint64_t)std::max<int64_t>(rows, 1)};
  const cuuint64_t str[1] = {(cuuint64_t)(K / 2)};
  const cuuint32_t box[2] = {BK / 2, (cuuint32_t)bn};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, str, box, estr,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    fprintf(stderr, "afd: cuTensorMapEncodeTiled failed (%d) for MXFP4 rows\n", (int)r);
    return AFD_ERR_CUDA;
  }
  return AFD_OK;
}

extern "C" int afd_mx4_poll_status(void* cuda_stream) {
  int32_t code = 0;
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(cuda_stream)) != cudaSuccess ||
      cudaMemcpyFromSymbol(&code, g_mx4_status, sizeof code) != cudaSuccess) {
    cudaGetLastError();
    return AFD_ERR_CUDA;
  }
  if (code) {
    const int32_t zero = 0;
    if (cudaMemcpyToSymbol(g_mx4_status, &zero, sizeof zero) != cudaSuccess) {
      cudaGetLastError();
      return AFD_ERR_CUDA;
    }
  }
  return code;
}
