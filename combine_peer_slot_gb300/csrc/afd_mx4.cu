// afd_mx4.cu -- MXFP4 coding on sm_103a (quantise, with the gather of routed
// rows; dequantise; packing of weights for the product) and the host side
// of the MXFP4 entry points.
#include <cstdio>
#include <cstring>

#include "afd_mx4.cuh"

namespace {

constexpr int kThreads = 256;
int64_t g_mx4_launches = 0;

// ---------------------------------------------------------------------------
// quantise: four lanes hold one block of 32, eight values each (one 16-byte
// load of bf16, two of fp32), so loads and the 4-byte code stores of a warp
// are contiguous.  The block's largest magnitude is an integer maximum of
// the sign-less bits (NaN and infinity sort above every number), the scale
// is a power of two and the division by it exact: every code is the nearest
// e2m1 value of the exact quotient.
// ---------------------------------------------------------------------------
struct QuantArgs {
  const uint8_t* x;
  int64_t ld_bytes;
  int64_t x_rows;
  const int32_t* src;
  int topk;
  int64_t n_rows;
  int chunks;  // eight-value chunks per row
  int ceil_rule;
  uint32_t* codes;
  uint8_t* scales;
};

template <bool F32>
__device__ __forceinline__ void load8(const uint8_t* p, float (&v)[8]) {
  if (F32) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

template <bool F32>
__global__ void __launch_bounds__(kThreads) k_mx4_quantize(const __grid_constant__ QuantArgs a) {
  const int64_t total = a.n_rows * a.chunks;  // a multiple of 4
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += stride) {
    const int64_t r = i / a.chunks;
    const int c = (int)(i - r * a.chunks);
    int64_t src = r;
    if (a.src) {
      const int32_t s = a.src[r];
      src = s < 0 ? -1 : s / a.topk;
    }
    float v[8] = {};
    if (src >= 0 && src < a.x_rows) load8<F32>(a.x + src * a.ld_bytes + (int64_t)c * (F32 ? 32 : 16), v);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
    const uint32_t quad = 0xfu << (threadIdx.x & 28);  // the block's four lanes are all here
    m = max(m, __shfl_xor_sync(quad, m, 1));
    m = max(m, __shfl_xor_sync(quad, m, 2));
    const uint32_t s = mx4_scale_byte(m, a.ceil_rule);
    const float inv = mx4_inv_scale(s);
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = s == 255u ? 0.0f : v[j] * inv;
    a.codes[i] = mx4_encode8(v);
    if ((threadIdx.x & 3) == 0) a.scales[i >> 2] = (uint8_t)s;
  }
}

// ---------------------------------------------------------------------------
// dequantise: eight values per thread.  Every value fits bf16 and fp32
// exactly (three significant bits, exponents within both types').
// ---------------------------------------------------------------------------
template <bool F32>
__global__ void __launch_bounds__(kThreads)
k_mx4_dequantize(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t total, int chunks,
                 uint8_t* out, int64_t ld_bytes) {
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += stride) {
    const int64_t r = i / chunks;
    const int c = (int)(i - r * chunks);
    const uint32_t w = codes[i];
    const float s = mx4_scale(scales[i >> 2]);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const uint32_t n = (w >> (4 * j)) & 15u, e = (n >> 1) & 3u;
      // e2m1: (1 + f / 2) 2^(e - 1), or f / 2 for e = 0
      const float mag = e ? __uint_as_float((126u + e) << 23 | (n & 1u) << 22) : 0.5f * (float)(n & 1u);
      v[j] = (n & 8u ? -mag : mag) * s;
    }
    uint8_t* p = out + r * ld_bytes + (int64_t)c * (F32 ? 32 : 16);
    if (F32) {
      reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint32_t h[4];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        h[j] = *reinterpret_cast<const uint32_t*>(&b);
      }
      *reinterpret_cast<uint4*>(p) = make_uint4(h[0], h[1], h[2], h[3]);
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

unsigned stride_grid(int64_t items, int num_sms) {
  const int64_t g = (items + kThreads - 1) / kThreads;
  return (unsigned)std::max<int64_t>(1, std::min<int64_t>(g, (int64_t)num_sms * 16));
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int make_lc(void* cuda_stream, LaunchCtx* lc) {
  *lc = LaunchCtx{reinterpret_cast<cudaStream_t>(cuda_stream), 0, &g_mx4_launches};
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
                    ceil_rule, reinterpret_cast<uint32_t*>(codes), scales};
  const unsigned grid = stride_grid(n_rows * (cols / 8), lc.num_sms);
  return f32 ? launch_k(lc, k_mx4_quantize<true>, grid, kThreads, 0, a)
             : launch_k(lc, k_mx4_quantize<false>, grid, kThreads, 0, a);
}

cudaError_t launch_mx4_pack(const LaunchCtx& lc, const uint8_t* codes, const uint8_t* scales, int E, int64_t M,
                            int K, int swiglu, uint8_t* packed) {
  const int tiles = mx4_tiles(M, swiglu), nkb = mx4_kblocks(K);
  return launch_k(lc, k_mx4_pack, (unsigned)((int64_t)E * tiles * nkb), kThreads, 0, codes, scales, M, K, swiglu,
                  tiles, nkb, packed);
}

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
  const int chunks = cols / 8;
  const int64_t total = n_rows * chunks;
  const uint32_t* c32 = reinterpret_cast<const uint32_t*>(codes);
  uint8_t* o = static_cast<uint8_t*>(out);
  return launched(es == 4 ? launch_k(lc, k_mx4_dequantize<true>, stride_grid(total, lc.num_sms), kThreads, 0, c32,
                                     scales, total, chunks, o, ldo * 4)
                          : launch_k(lc, k_mx4_dequantize<false>, stride_grid(total, lc.num_sms), kThreads, 0, c32,
                                     scales, total, chunks, o, ldo * 2),
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

// One product over the grouped rows.
static int product(const LaunchCtx& lc, const uint8_t* codes, const uint8_t* scales, int64_t n_rows,
                   const int32_t* offsets, int E, const void* w, int M, int K, int swiglu, int fmt, void* out,
                   int64_t ldo, uint8_t* out_scales = nullptr) {
  Mx4GemmArgs a;
  memset(&a, 0, sizeof a);
  const int bn = mx4_token_tile(n_rows, E);
  int rc = encode_mx4_rows(&a.tmX[0], codes, n_rows, K, bn);
  if (rc) return rc;
  a.xs[0] = scales;
  a.x_rows[0] = n_rows;
  a.w[0] = static_cast<const uint8_t*>(w);
  a.out[0] = out;
  a.out_lo[0] = out_scales;
  a.ldo[0] = ldo;
  a.fmt[0] = fmt;
  a.M[0] = M;
  a.K[0] = K;
  a.offsets = offsets;
  a.n_groups = E;
  a.swiglu = swiglu;
  const int64_t units = (int64_t)mx4_tiles(M, swiglu) * ((n_rows + bn - 1) / bn + std::min<int64_t>(E, n_rows));
  if (units >= (int64_t)1 << 31) return AFD_ERR_UNSUPPORTED;
  return launched(launch_mx4_gemm(lc, a, bn, units), "mx4 gemm");
}

int afd_mx4_gemm(const uint8_t* codes, const uint8_t* scales, int64_t n_rows, const int32_t* offsets,
                 int num_experts, const void* weight, int M, int K, int swiglu, int out_dtype, void* out,
                 int64_t ldo, void* cuda_stream) {
  const int cols = swiglu ? M / 2 : M;
  if (afd_mx4_weight_bytes(num_experts, M, K, swiglu) == 0 || n_rows < 0 || n_rows > kMaxRows || ldo < cols ||
      (out_dtype != AFD_DTYPE_F32 && out_dtype != AFD_DTYPE_BF16))
    return AFD_ERR_ARG;
  if (swiglu && out_dtype != AFD_DTYPE_BF16) return AFD_ERR_UNSUPPORTED;
  if (n_rows == 0) return AFD_OK;
  if (!codes || !scales || !offsets || !weight || !out || !aligned(codes, 16) || !aligned(weight, 128) ||
      !aligned(scales, 8) || !aligned(out, 16) || !aligned(offsets, 4) || ldo % 8)
    return AFD_ERR_ARG;
  int rc = check_device_ptrs({codes, scales, offsets, weight, out});
  LaunchCtx lc;
  if (!rc) rc = make_lc(cuda_stream, &lc);
  if (rc) return rc;
  return product(lc, codes, scales, n_rows, offsets, num_experts, weight, M, K, swiglu != 0,
                 out_dtype == AFD_DTYPE_F32 ? OUT_F32 : OUT_ACT, out, ldo);
}

// workspace: the codes and scales of h
int64_t afd_mx4_ffn_workspace(int64_t n_rows, int inter) {
  if (n_rows < 0 || n_rows > kMaxRows || inter < kMx4Block || inter > kMaxDim || inter % kMx4Block) return -1;
  const int64_t n = n_rows * inter;
  return (n / 2 + 255) / 256 * 256 + (n / 32 + 255) / 256 * 256;
}

int afd_mx4_ffn(const uint8_t* codes, const uint8_t* scales, int64_t n_rows, const int32_t* offsets,
                int num_experts, const void* w13, const void* wd, int hidden, int inter, int out_dtype, void* out,
                int64_t ldo, void* workspace, int64_t workspace_bytes, void* cuda_stream) {
  const int64_t need = afd_mx4_ffn_workspace(n_rows, inter);
  if (need < 0 || afd_mx4_weight_bytes(num_experts, 2 * inter, hidden, 1) == 0 ||
      afd_mx4_weight_bytes(num_experts, hidden, inter, 0) == 0 || ldo < hidden ||
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
  const int64_t n = n_rows * inter;
  uint8_t* hc = static_cast<uint8_t*>(workspace);
  uint8_t* hs = hc + (n / 2 + 255) / 256 * 256;
  rc = product(lc, codes, scales, n_rows, offsets, num_experts, w13, 2 * inter, hidden, 1, OUT_MX4, hc, inter, hs);
  lc.pdl = 1;  // the second launch's set-up runs while the first drains
  if (!rc)
    rc = product(lc, hc, hs, n_rows, offsets, num_experts, wd, hidden, inter, 0,
                 out_dtype == AFD_DTYPE_F32 ? OUT_F32 : OUT_ACT, out, ldo);
  return rc;
}

}  // extern "C"
