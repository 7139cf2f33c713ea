// afd_mx4.cu -- MXFP4 coding on sm_103a (quantise, with the gather of routed
// rows; dequantise; packing of weights for the product) and the host side
// of the MXFP4 entry points.
#include <cuda_fp16.h>

#include <cstdio>
#include <cstring>

#include "afd_mx4.cuh"

namespace {

constexpr int kThreads = 256;

// Both coding kernels walk the matrix in chunks of eight (or four) values, a
// CTA kChunks * 256 consecutive ones, a thread every 256th of them: a warp's
// loads and stores are contiguous whatever the row length, and each thread
// has kChunks independent loads in flight.  The row of the CTA's first chunk
// takes one 64-bit division, the rest 32-bit ones by multiplication.
constexpr int kChunks = 4;
struct ChunkPos {
  int64_t row0;
  uint32_t c0, chunks, magic;
  __device__ __forceinline__ ChunkPos(int64_t first, int n, uint32_t m) : chunks((uint32_t)n), magic(m) {
    row0 = first / n;
    c0 = (uint32_t)(first - row0 * n);
  }
  // row and chunk of the CTA's i-th chunk
  __device__ __forceinline__ void at(int i, int64_t& row, int& c) const {
    const uint32_t v = c0 + (uint32_t)i;
    uint32_t q = __umulhi(v, magic);  // v / chunks, or one less (magic = (2^32 - 1) / chunks)
    if ((q + 1) * chunks <= v) q++;
    row = row0 + q;
    c = (int)(v - q * chunks);
  }
};

// ---------------------------------------------------------------------------
// quantise: four lanes hold one block of 32, eight values each (one 16-byte
// load of bf16, two of fp32).  The block's largest magnitude is an integer
// maximum of the sign-less bits (NaN and infinity sort above every number),
// the scale is a power of two and the division by it exact: every code is
// the nearest e2m1 value of the exact quotient.  Bound by memory: 13312 rows
// of 2048 bf16 values, 69 MB, take 11.9 us (5.8 TB/s), one row 1.8 us.
// ---------------------------------------------------------------------------
struct QuantArgs {
  const uint8_t* x;
  int64_t ld_bytes;
  int64_t x_rows;
  const int32_t* src;
  int topk;
  int64_t n_rows;
  int chunks;  // eight-value chunks per row
  uint32_t magic;
  int ceil_rule;
  uint32_t* codes;
  uint8_t* scales;
};

template <bool F32>
__device__ __forceinline__ void quantize_chunks(const QuantArgs& a, int64_t n_rows) {
  const int64_t total = n_rows * a.chunks;  // a multiple of 4: a block's lanes are all in or all out
  const int64_t first = (int64_t)blockIdx.x * (kThreads * kChunks);
  if (first >= total) return;
  const ChunkPos pos(first, a.chunks, a.magic);
  uint4 lo[kChunks], hi[kChunks];
#pragma unroll
  for (int u = 0; u < kChunks; u++) {
    const int i = u * kThreads + threadIdx.x;
    lo[u] = hi[u] = make_uint4(0, 0, 0, 0);
    if (first + i >= total) continue;
    int64_t r;
    int c;
    pos.at(i, r, c);
    if (a.src) {
      const int32_t s = a.src[r];
      r = s < 0 ? -1 : (int64_t)((uint32_t)s / (uint32_t)a.topk);
      if (r >= a.x_rows) r = -1;
    }
    if (r < 0) continue;
    const uint4* p = reinterpret_cast<const uint4*>(a.x + r * a.ld_bytes + (int64_t)c * (F32 ? 32 : 16));
    lo[u] = p[0];
    if (F32) hi[u] = p[1];
  }
#pragma unroll
  for (int u = 0; u < kChunks; u++) {
    const int64_t i = first + u * kThreads + threadIdx.x;
    const uint32_t w[8] = {lo[u].x, lo[u].y, lo[u].z, lo[u].w, hi[u].x, hi[u].y, hi[u].z, hi[u].w};
    float v[8];
    uint32_t m = 0;
    if (F32) {
#pragma unroll
      for (int j = 0; j < 8; j++) {
        v[j] = __uint_as_float(w[j]);
        m = max(m, w[j] & 0x7fffffffu);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; j++) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        m = __vmaxu2(m, w[j] & 0x7fff7fffu);
      }
      m = max(m << 16, m & 0x7fff0000u);
    }
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    if (i >= total) continue;
    const uint32_t s = mx4_scale_byte(m, a.ceil_rule);
    const float inv = mx4_inv_scale(s);
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] *= inv;
    a.codes[i] = s == 255u ? 0u : mx4_encode8(v);
    if ((threadIdx.x & 3) == 0) a.scales[i >> 2] = (uint8_t)s;
  }
}
template <bool F32>
__global__ void __launch_bounds__(kThreads) k_mx4_quantize(const __grid_constant__ QuantArgs a) {
  quantize_chunks<F32>(a, a.n_rows);
}

// ---------------------------------------------------------------------------
// the same for a step's gathered rows: position r of Xp is row r of the
// result.  The first thread also writes where the shared rows lie, for the
// products that follow (a step of the work-item loop knows it on the device
// only).  The launch's rows are the most there can be; the step's own are coded.
// ---------------------------------------------------------------------------
struct StepArgs {
  QuantArgs q;
  const FanIn* item;  // NULL: the counts are n and s
  int topk, has_shared, n, s;
  int32_t* offs;
  const int32_t* status;
};
__global__ void __launch_bounds__(kThreads) k_mx4_quantize_step(const __grid_constant__ StepArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  if (read_status(a.status)) return;
  int N = a.n, S = a.s;
  if (a.item) {
    N = a.item->grouped ? a.item->rtotal : a.item->total * a.topk;
    S = a.has_shared ? a.item->stotal : 0;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.offs[0] = N;
    a.offs[1] = N + S;
    a.offs[2] = 0;
    a.offs[3] = S;
  }
  quantize_chunks<false>(a.q, min(a.q.n_rows, (int64_t)N + S));
}

// ---------------------------------------------------------------------------
// dequantise: every value fits bf16 and fp32 exactly (three significant
// bits, exponents within both types').  Bound by memory.  A chunk is what
// 16 output bytes hold, eight bf16 or four fp32 values, so that a warp's
// stores are one run.  13312 x 2048 to bf16 take 10.2 us; 7996 x 1408 to
// fp32, 45 MB, 8.1 us (14 as two stores of eight values, which wrote half
// sectors).
// ---------------------------------------------------------------------------
struct DequantArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t n_rows;
  int chunks;
  uint32_t magic;
  uint8_t* out;
  int64_t ld_bytes;
};

template <bool F32>
__global__ void __launch_bounds__(kThreads) k_mx4_dequantize(const __grid_constant__ DequantArgs a) {
  const int64_t total = a.n_rows * a.chunks;
  const int64_t first = (int64_t)blockIdx.x * (kThreads * kChunks);
  const ChunkPos pos(first, a.chunks, a.magic);
  uint32_t code[kChunks];
  float scale[kChunks];
#pragma unroll
  for (int u = 0; u < kChunks; u++) {
    const int64_t i = first + u * kThreads + threadIdx.x;
    code[u] = i >= total ? 0u
              : F32      ? (uint32_t)reinterpret_cast<const uint16_t*>(a.codes)[i]
                         : reinterpret_cast<const uint32_t*>(a.codes)[i];
    scale[u] = i < total ? mx4_scale(a.scales[i >> (F32 ? 3 : 2)]) : 0.0f;
  }
#pragma unroll
  for (int u = 0; u < kChunks; u++) {
    const int i = u * kThreads + threadIdx.x;
    if (first + i >= total) continue;
    int64_t r;
    int c;
    pos.at(i, r, c);
    uint32_t h[4];  // pairs of fp16, which holds every e2m1 value
    asm("{ .reg .b8 b0, b1, b2, b3; mov.b32 {b0, b1, b2, b3}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, b0; cvt.rn.f16x2.e2m1x2 %1, b1;\n"
        "cvt.rn.f16x2.e2m1x2 %2, b2; cvt.rn.f16x2.e2m1x2 %3, b3; }"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(code[u]));
    float2 v[4];
#pragma unroll
    for (int j = 0; j < (F32 ? 2 : 4); j++) {
      v[j] = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
      v[j].x *= scale[u];
      v[j].y *= scale[u];
    }
    uint8_t* p = a.out + r * a.ld_bytes + (int64_t)c * 16;
    if (F32) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    } else {
      uint32_t b[4];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(v[j].x, v[j].y);
        b[j] = *reinterpret_cast<const uint32_t*>(&x);
      }
      *reinterpret_cast<uint4*>(p) = make_uint4(b[0], b[1], b[2], b[3]);
    }
  }
}

// ---------------------------------------------------------------------------
// weights [E][M][K] (codes and scales as plain rows) into the product's
// blocks; one CTA per block, once per layer
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kThreads)
k_mx4_pack(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t M, int K, int swiglu,
           int tiles, int nkb, uint8_t* __restrict__ packed) {
  const int64_t b = blockIdx.x;
  const int kb = (int)(b % nkb);
  const int t = (int)(b / nkb % tiles);
  const int64_t e = b / nkb / tiles;
  uint8_t* dst = packed + b * kMx4BlkBytes;
  // source row of tile row r, or -1 past the weight's edge
  auto source = [&](int r) -> int64_t {
    if (!swiglu) {
      const int64_t row = (int64_t)t * 128 + r;
      return row < M ? e * M + row : -1;
    }
    const int64_t f = (int64_t)t * 64 + (r >> 5) * 16 + (r & 15);
    if (f >= M / 2) return -1;
    return e * M + ((r & 16) ? M / 2 + f : f);
  };
  for (int i = threadIdx.x; i < 128 * 4; i += blockDim.x) {  // 16-byte chunks: 32 columns each
    const int r = i >> 2, c = i & 3;
    const int64_t row = source(r);
    const int col = kb * kMx4BlkCols + c * 32;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row >= 0 && col < K) v = *reinterpret_cast<const uint4*>(codes + row * (K / 2) + col / 2);
    *reinterpret_cast<uint4*>(dst + r * 64 + ((c ^ ((r >> 1) & 3)) << 4)) = v;
  }
  for (int i = threadIdx.x; i < 512; i += blockDim.x) {
    const int r = i >> 2, c = i & 3;
    const int64_t row = source(r);
    const int blk = kb * 4 + c;
    dst[kMx4BlkCodes + (r & 31) * 16 + (r >> 5) * 4 + c] =
        row >= 0 && blk < K / 32 ? scales[row * (K / 32) + blk] : (uint8_t)0;
  }
}

int64_t chunk_grid(int64_t chunks) { return (chunks + kThreads * kChunks - 1) / (kThreads * kChunks); }

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int make_lc(void* cuda_stream, LaunchCtx* lc) {
  *lc = LaunchCtx{reinterpret_cast<cudaStream_t>(cuda_stream), 0, nullptr};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&lc->num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return AFD_ERR_CUDA;
  }
  return AFD_OK;
}

int launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return AFD_OK;
  fprintf(stderr, "afd: %s: %s\n", what, cudaGetErrorString(e));
  cudaGetLastError();
  return AFD_ERR_CUDA;
}

constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int kMaxDim = 1 << 16;

bool dims_ok(int64_t M, int64_t K) { return M >= 1 && M <= kMaxDim && K >= kMx4Block && K <= kMaxDim; }

}  // namespace

cudaError_t launch_mx4_quantize(const LaunchCtx& lc, const void* x, int64_t ldx, int64_t x_rows, int f32,
                                const int32_t* src_rows, int topk, int64_t n_rows, int cols, int ceil_rule,
                                uint8_t* codes, uint8_t* scales) {
  const QuantArgs a{static_cast<const uint8_t*>(x), ldx * (f32 ? 4 : 2), x_rows, src_rows, topk, n_rows, cols / 8,
                    0xffffffffu / (uint32_t)(cols / 8), ceil_rule, reinterpret_cast<uint32_t*>(codes), scales};
  const int64_t grid = chunk_grid(n_rows * (cols / 8));
  if (grid >= (int64_t)1 << 31) return cudaErrorInvalidValue;
  return f32 ? launch_k(lc, k_mx4_quantize<true>, (unsigned)grid, kThreads, 0, a)
             : launch_k(lc, k_mx4_quantize<false>, (unsigned)grid, kThreads, 0, a);
}

cudaError_t launch_mx4_quantize_step(const LaunchCtx& lc, const void* xp, int cols, const FanIn* item,
                                     int topk, int n, int s, uint8_t* codes, uint8_t* scales, int32_t* offs,
                                     const int32_t* status) {
  const int64_t rows = (int64_t)n + s;
  const StepArgs a{{static_cast<const uint8_t*>(xp), (int64_t)cols * 2, rows, nullptr, 1, rows, cols / 8,
                    0xffffffffu / (uint32_t)(cols / 8), 0, reinterpret_cast<uint32_t*>(codes), scales},
                   item, topk, s > 0, n, s, offs, status};
  const int64_t grid = std::max<int64_t>(1, chunk_grid(rows * (cols / 8)));
  if (grid >= (int64_t)1 << 31) return cudaErrorInvalidValue;
  return launch_k(lc, k_mx4_quantize_step, (unsigned)grid, kThreads, 0, a);
}

cudaError_t launch_mx4_pack(const LaunchCtx& lc, const uint8_t* codes, const uint8_t* scales, int E, int64_t M,
                            int K, int swiglu, uint8_t* packed) {
  const int tiles = mx4_tiles(M, swiglu), nkb = mx4_kblocks(K);
  return launch_k(lc, k_mx4_pack, (unsigned)((int64_t)E * tiles * nkb), kThreads, 0, codes, scales, M, K, swiglu,
                  tiles, nkb, packed);
}

int mx4_product(LaunchCtx& lc, Mx4GemmArgs& a, const uint8_t* codes, const uint8_t* scales, uint8_t* image,
                int64_t x_rows, int64_t rows, const int32_t* offsets, int groups, int M, int K, int swiglu) {
  const int bn = mx4_token_tile(rows, groups);
  const int64_t img = mx4_image_bytes(rows, groups, K);
  const int64_t units = (int64_t)mx4_tiles(M, swiglu) * ((rows + bn - 1) / bn + std::min<int64_t>(groups, rows));
  if (units >= (int64_t)1 << 31 || img / 128 >= (int64_t)1 << 31) return AFD_ERR_UNSUPPORTED;
  int rc = encode_mx4_rows(&a.tmX, codes, x_rows, K, bn);
  if (!rc && img && !a.layers) rc = encode_mx4_weight(a.tmW, a.w, mx4_weight_bytes(groups, M, K, swiglu));
  if (!rc && a.fmt == OUT_ACT) rc = encode_mx4_out(&a.tmO, a.out, x_rows, swiglu ? M / 2 : M, a.ldo);
  if (!rc && img) rc = encode_mx4_images(&a.tmS, image, img);
  if (rc) return rc;
  if (img && scales) {
    rc = launched(launch_mx4_images(lc, scales, x_rows, offsets, rows, groups, K, image, a.status), "mx4 scale images");
    if (rc) return rc;
    // the product's set-up runs while the images are written: in a call without
    // a context (which has no status), in a step as its context's flags say
    if (!a.status) lc.pdl = 1;
  }
  a.xs = scales;
  a.x_rows = x_rows;
  a.M = M;
  a.K = K;
  a.offsets = offsets;
  a.n_groups = groups;
  a.swiglu = swiglu;
  a.tiles = (int)mx4_image_tiles(rows, groups);
  return launched(launch_mx4_gemm(lc, a, bn, units), "mx4 gemm");
}

// the products of the calls without a context
static int product(LaunchCtx& lc, const uint8_t* codes, const uint8_t* scales, uint8_t* image, int64_t n_rows,
                   const int32_t* offsets, int E, const void* w, int M, int K, int swiglu, int fmt, void* out,
                   int64_t ldo, uint8_t* out_scales = nullptr, int early = 0) {
  Mx4GemmArgs a;
  memset(&a, 0, sizeof a);
  a.w = static_cast<const uint8_t*>(w);
  a.out = out;
  a.out_lo = out_scales;
  a.early = early;
  a.ldo = ldo;
  a.fmt = fmt;
  return mx4_product(lc, a, codes, scales, image, n_rows, n_rows, offsets, E, M, K, swiglu);
}
static int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

extern "C" {

int afd_mx4_quantize(const void* x, int64_t ldx, int64_t x_rows, int cols, int dtype, const int32_t* src_rows,
                     int topk, int64_t n_rows, int scale_rule, uint8_t* codes, uint8_t* scales,
                     void* cuda_stream) {
  if ((dtype != AFD_DTYPE_F32 && dtype != AFD_DTYPE_BF16) || cols < kMx4Block || cols > kMaxDim || cols % kMx4Block ||
      x_rows < 0 || n_rows < 0 || n_rows > kMaxRows || x_rows > kMaxRows || ldx < cols || topk < 1 ||
      (scale_rule != AFD_MX4_SCALE_FLOOR && scale_rule != AFD_MX4_SCALE_CEIL) ||
      (!src_rows && n_rows > 0 && (n_rows != x_rows || topk != 1)))
    return AFD_ERR_ARG;
  const int es = dtype == AFD_DTYPE_F32 ? 4 : 2;
  if (n_rows == 0) return AFD_OK;
  if ((!x && x_rows > 0) || !codes || !scales || !aligned(x, 16) || (ldx * es) % 16 || !aligned(codes, 16) ||
      !aligned(src_rows, 4))
    return AFD_ERR_ARG;
  if (chunk_grid(n_rows * (cols / 8)) >= (int64_t)1 << 31) return AFD_ERR_UNSUPPORTED;
  int rc = check_device_ptrs({x, src_rows, codes, scales});
  LaunchCtx lc;
  if (!rc) rc = make_lc(cuda_stream, &lc);
  if (rc) return rc;
  return launched(launch_mx4_quantize(lc, x, ldx, x_rows, dtype == AFD_DTYPE_F32, src_rows, topk, n_rows, cols,
                                      scale_rule == AFD_MX4_SCALE_CEIL, codes, scales),
                  "mx4 quantize");
}

int afd_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t n_rows, int cols, int dtype, void* out,
                       int64_t ldo, void* cuda_stream) {
  if ((dtype != AFD_DTYPE_F32 && dtype != AFD_DTYPE_BF16) || cols < kMx4Block || cols > kMaxDim || cols % kMx4Block ||
      n_rows < 0 || n_rows > kMaxRows || ldo < cols)
    return AFD_ERR_ARG;
  const int es = dtype == AFD_DTYPE_F32 ? 4 : 2;
  if ((ldo * es) % 16) return AFD_ERR_ARG;
  if (n_rows == 0) return AFD_OK;
  if (!codes || !scales || !out || !aligned(codes, 16) || !aligned(out, 16)) return AFD_ERR_ARG;
  int rc = check_device_ptrs({codes, scales, out});
  LaunchCtx lc;
  if (!rc) rc = make_lc(cuda_stream, &lc);
  if (rc) return rc;
  const int chunks = cols / (16 / es);
  const int64_t grid = chunk_grid(n_rows * chunks);
  if (grid >= (int64_t)1 << 31) return AFD_ERR_UNSUPPORTED;
  const DequantArgs a{codes, scales, n_rows, chunks, 0xffffffffu / (uint32_t)chunks,
                      static_cast<uint8_t*>(out), ldo * es};
  return launched(es == 4 ? launch_k(lc, k_mx4_dequantize<true>, (unsigned)grid, kThreads, 0, a)
                          : launch_k(lc, k_mx4_dequantize<false>, (unsigned)grid, kThreads, 0, a),
                  "mx4 dequantize");
}

int64_t afd_mx4_weight_bytes(int num_experts, int M, int K, int swiglu) {
  if (num_experts < 1 || num_experts > 256 || !dims_ok(M, K) || K % kMx4Block || M % (swiglu ? 16 : 8)) return 0;
  return mx4_weight_bytes(num_experts, M, K, swiglu);
}

int afd_mx4_pack_weight(const uint8_t* codes, const uint8_t* scales, int num_experts, int M, int K, int swiglu,
                        void* packed, int64_t packed_bytes, void* cuda_stream) {
  const int64_t need = afd_mx4_weight_bytes(num_experts, M, K, swiglu);
  if (need == 0) return AFD_ERR_ARG;
  if (packed_bytes < need) return AFD_ERR_CAPACITY;
  if (!codes || !scales || !packed || !aligned(codes, 16) || !aligned(packed, 128)) return AFD_ERR_ARG;
  int rc = check_device_ptrs({codes, scales, packed});
  LaunchCtx lc;
  if (!rc) rc = make_lc(cuda_stream, &lc);
  if (rc) return rc;
  return launched(launch_mx4_pack(lc, codes, scales, num_experts, M, K, swiglu != 0, static_cast<uint8_t*>(packed)),
                  "mx4 pack weight");
}


int64_t afd_mx4_gemm_workspace(int64_t n_rows, int num_experts, int K) {
  if (n_rows < 0 || n_rows > kMaxRows || num_experts < 1 || num_experts > 256 || !dims_ok(1, K) || K % kMx4Block)
    return -1;
  return up256(mx4_image_bytes(n_rows, num_experts, K));
}

int afd_mx4_gemm(const uint8_t* codes, const uint8_t* scales, int64_t n_rows, const int32_t* offsets,
                 int num_experts, const void* weight, int M, int K, int swiglu, int out_dtype, void* out,
                 int64_t ldo, void* workspace, int64_t workspace_bytes, void* cuda_stream) {
  const int cols = swiglu ? M / 2 : M;
  if (afd_mx4_weight_bytes(num_experts, M, K, swiglu) == 0 || n_rows < 0 || n_rows > kMaxRows || ldo < cols ||
      (out_dtype != AFD_DTYPE_F32 && out_dtype != AFD_DTYPE_BF16))
    return AFD_ERR_ARG;
  if (swiglu && out_dtype != AFD_DTYPE_BF16) return AFD_ERR_UNSUPPORTED;
  if (n_rows == 0) return AFD_OK;
  const int64_t need = afd_mx4_gemm_workspace(n_rows, num_experts, K);
  if (workspace_bytes < need) return AFD_ERR_CAPACITY;
  if ((need && !workspace) || !aligned(workspace, 256)) return AFD_ERR_ARG;
  if (!codes || !scales || !offsets || !weight || !out || !aligned(codes, 16) || !aligned(weight, 128) ||
      !aligned(scales, 8) || !aligned(out, 16) || !aligned(offsets, 4) || ldo % 8)
    return AFD_ERR_ARG;
  int rc = check_device_ptrs({codes, scales, offsets, weight, out, need ? workspace : nullptr});
  LaunchCtx lc;
  if (!rc) rc = make_lc(cuda_stream, &lc);
  if (rc) return rc;
  return product(lc, codes, scales, static_cast<uint8_t*>(workspace), n_rows, offsets, num_experts, weight, M, K, swiglu != 0,
                 out_dtype == AFD_DTYPE_F32 ? OUT_F32 : OUT_ACT, out, ldo);
}

// workspace: h's codes and its scales (or their images), x's scale images
static int64_t ffn_scales_bytes(int64_t n_rows, int E, int inter) {
  return up256(std::max(n_rows * inter / 32, mx4_image_bytes(n_rows, E, inter)));
}
int64_t afd_mx4_ffn_workspace(int64_t n_rows, int num_experts, int hidden, int inter) {
  // (2 inter rows of w13 are within the limits as well)
  if (inter < kMx4Block || inter > kMaxDim / 2 || inter % kMx4Block) return -1;
  const int64_t img = afd_mx4_gemm_workspace(n_rows, num_experts, hidden);
  return img < 0 ? -1 : up256(n_rows * inter / 2) + ffn_scales_bytes(n_rows, num_experts, inter) + img;
}

int afd_mx4_ffn(const uint8_t* codes, const uint8_t* scales, int64_t n_rows, const int32_t* offsets,
                int num_experts, const void* w13, const void* wd, int hidden, int inter, int out_dtype, void* out,
                int64_t ldo, void* workspace, int64_t workspace_bytes, void* cuda_stream) {
  const int64_t need = afd_mx4_ffn_workspace(n_rows, num_experts, hidden, inter);
  if (need < 0 || ldo < hidden ||
      (out_dtype != AFD_DTYPE_F32 && out_dtype != AFD_DTYPE_BF16))
    return AFD_ERR_ARG;
  if (n_rows == 0) return AFD_OK;
  if (workspace_bytes < need) return AFD_ERR_CAPACITY;
  if (!codes || !scales || !offsets || !w13 || !wd || !out || !workspace || !aligned(codes, 16) ||
      !aligned(scales, 8) || !aligned(w13, 128) || !aligned(wd, 128) || !aligned(out, 16) || !aligned(offsets, 4) ||
      !aligned(workspace, 256) || ldo % 8)
    return AFD_ERR_ARG;
  int rc = check_device_ptrs({codes, scales, offsets, w13, wd, out, workspace});
  LaunchCtx lc;
  if (!rc) rc = make_lc(cuda_stream, &lc);
  if (rc) return rc;
  uint8_t* hc = static_cast<uint8_t*>(workspace);
  uint8_t* hs = hc + up256(n_rows * inter / 2);
  uint8_t* xi = hs + ffn_scales_bytes(n_rows, num_experts, inter);
  const bool wide = mx4_image_bytes(n_rows, num_experts, inter) > 0;
  rc = product(lc, codes, scales, xi, n_rows, offsets, num_experts, w13, 2 * inter, hidden, 1, OUT_MX4, hc, inter, hs);
  lc.pdl = 1;  // the second product's set-up runs while the first drains
  if (!rc)
    rc = product(lc, hc, wide ? nullptr : hs, hs, n_rows, offsets, num_experts, wd, hidden, inter, 0,
                 out_dtype == AFD_DTYPE_F32 ? OUT_F32 : OUT_ACT, out, ldo, nullptr, /*early=*/1);
  return rc;
}

}  // extern "C"
