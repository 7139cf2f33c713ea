// afd_mx4.cuh -- what the MXFP4 translation units share: the format's
// arithmetic, the packed weight's layout and the launchers.
//
// MXFP4 (OCP Microscaling Formats 1.0): 32 consecutive values share one
// e8m0 scale 2^(s - 127) (byte s, 255 = NaN); each value is an e2m1 number,
// one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign (bit 3 of its nibble).  A
// row of K values is K / 2 bytes of codes (value 2 i in the low nibble of
// byte i) and K / 32 scale bytes.
#pragma once

#include "afd_internal.cuh"

constexpr int kMx4Block = 32;
// Packed weights: [expert][128-row tile][128-column block] of
//   8192 bytes of codes: row r's 64 bytes at r * 64, its 16-byte chunk c at
//        chunk c ^ ((r >> 1) & 3) (the 64-byte swizzle tcgen05.mma reads)
//    512 bytes of scales: row r's four at (r % 32) * 16 + (r / 32) * 4 (the
//        image tcgen05.cp.32x128b spreads over the TMEM lanes)
// contiguous, so one bulk copy moves any run of column blocks with its
// scales; rows and columns past the weight's edge are zero.  128 columns a
// block and not 256: inter sizes such as 1408 are whole blocks, where 256
// would read 9 % more than the weight holds.
constexpr int kMx4BlkCols = 128;
constexpr int kMx4BlkCodes = 128 * kMx4BlkCols / 2;
constexpr int kMx4BlkBytes = kMx4BlkCodes + 512;

// tiles and bytes of a packed weight [E][M][K]; with swiglu, tile t holds
// the gate and up rows of features [64 t, 64 t + 64): each 32 rows are 16
// gate rows, then the 16 matching up rows
__host__ __device__ inline int mx4_tiles(int64_t M, int swiglu) {
  return (int)(swiglu ? (M / 2 + 63) / 64 : (M + 127) / 128);
}
__host__ __device__ inline int mx4_kblocks(int K) { return (K + kMx4BlkCols - 1) / kMx4BlkCols; }
inline int64_t mx4_weight_bytes(int64_t E, int64_t M, int K, int swiglu) {
  return E * mx4_tiles(M, swiglu) * mx4_kblocks(K) * kMx4BlkBytes;
}

// Arguments of one grouped product: rows [offsets[g], offsets[g + 1]) times
// weight g.
#define OUT_MX4 3  // SwiGLU only: codes in out, scales in out_lo (ldo % 32 == 0)
struct Mx4GemmArgs {
  CUtensorMap tmX;           // codes of the rows (encode_mx4_rows)
  CUtensorMap tmW[2];        // the packed weight (encode_mx4_weight); the wide form's
  CUtensorMap tmS;           // the rows' scale images (encode_mx4_images); the wide form's
  CUtensorMap tmO;           // bf16 output (encode_mx4_out)
  const uint8_t* xs;         // the rows' scales [x_rows][K / 32]; the narrow form's
  int64_t x_rows;
  const uint8_t* w;          // the packed weight; the narrow form's
  void* out;
  uint8_t* out_lo;           // OUT_Y24: the low plane; OUT_MX4: the scales (wide: their images)
  int64_t ldo;               // output row pitch in elements
  const int32_t* out_shift;  // device, NULL = 0: row r goes to output row r - *out_shift
  int fmt;                   // OUT_*
  int M, K;
  const int32_t* offsets;    // [n_groups + 1], device
  int n_groups;
  int swiglu;
  int32_t* status;           // the step's: no work once it is set; NULL: waits that give up are counted (afd_mx4_poll_status)
  // layer chosen on the device: the weight is layers[item->layer].mx4[wsel], not tmW and w
  const DevLayer* layers;
  const FanIn* item;
  int wsel;
  // the kernel before writes the rows only; launched with lc.pdl
  int early;
  int tiles;                 // token tiles the images hold (more only for offsets that overlap)
  int64_t out_rows;          // rows the output holds, and the workspace's record, for the
  int64_t* dbg;              // debug build's check (NULL: not checked)
};
// bn: rows of a token tile (mx4_token_tile); units: an upper bound on the
// output tiles, which sizes the grid
#ifdef AFD_DEBUG_BOUNDS
int mx4_plant_error();  // counts one error as a product without a context does
#endif
int mx4_token_tile(int64_t rows, int groups);
cudaError_t launch_mx4_gemm(const LaunchCtx& lc, const Mx4GemmArgs& a, int bn, int64_t units);
int encode_mx4_rows(CUtensorMap* m, const void* codes, int64_t rows, int K, int bn);
int64_t mx4_image_tiles(int64_t rows, int groups);
int64_t mx4_image_bytes(int64_t rows, int groups, int K);
int64_t mx4_most_image_bytes(int64_t rows, int groups, int K);  // over all row counts up to rows
int encode_mx4_images(CUtensorMap* m, const void* image, int64_t bytes);
// x_rows: rows the scales hold; rows: the most the groups hold together
cudaError_t launch_mx4_images(const LaunchCtx& lc, const uint8_t* scales, int64_t x_rows, const int32_t* offsets,
                              int64_t rows, int groups, int K, uint8_t* image, const int32_t* status);
int encode_mx4_out(CUtensorMap* m, void* out, int64_t rows, int cols, int64_t ldo);
int encode_mx4_weight(CUtensorMap* tm /* [2]: a part's blocks, one block */, const void* packed, int64_t bytes);

cudaError_t launch_mx4_quantize(const LaunchCtx& lc, const void* x, int64_t ldx, int64_t x_rows, int f32,
                                const int32_t* src_rows, int topk, int64_t n_rows, int cols, int ceil_rule,
                                uint8_t* codes, uint8_t* scales);
// The step's gathered rows (n routed, then s shared; item: the device's own
// counts, n and s the most there can be) coded position by position, and
// offs = {n, n + s, 0, s} for the shared rows' products
cudaError_t launch_mx4_quantize_step(const LaunchCtx& lc, const void* xp, int cols, const FanIn* item, int topk, int n,
                                     int s, uint8_t* codes, uint8_t* scales, int32_t* offs,
                                     const int32_t* status);
// One product of the step or of a call.  image: the rows' scale images (wide
// form; written from scales unless that is NULL), rows: the most rows the
// groups hold together, x_rows: the rows that codes and scales hold.
// a: out, out_lo, ldo, out_shift, fmt, status, and layers / item / wsel or w.
int mx4_product(LaunchCtx& lc, Mx4GemmArgs& a, const uint8_t* codes, const uint8_t* scales, uint8_t* image,
                int64_t x_rows, int64_t rows, const int32_t* offsets, int groups, int M, int K, int swiglu);
cudaError_t launch_mx4_pack(const LaunchCtx& lc, const uint8_t* codes, const uint8_t* scales, int E, int64_t M,
                            int K, int swiglu, uint8_t* packed);

#ifdef __CUDACC__
// e8m0 byte -> fp32 2^(s - 127); 0 is fp32's subnormal 2^-127, 255 NaN
__device__ __forceinline__ float mx4_scale(uint32_t s) {
  return __uint_as_float(s == 0u ? 0x00400000u : s == 255u ? 0x7fc00000u : s << 23);
}
// The scale byte of a block whose largest magnitude has these fp32 bits.
// floor rule (the OCP format's): 2^(floor(log2 amax) - 2), under which a
// block's largest values up to 8 scales saturate to 6; ceil rule: the
// smallest power of two whose 6 reaches amax (mantissa over 1.5 takes the
// next one), up to 2^125: the 4 and 6 of a larger scale are no finite fp32.
// 255 for a block with a NaN or an infinity.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t amax_bits, int ceil_rule) {
  if (amax_bits >= 0x7f800000u) return 255u;
  const int e = (int)(amax_bits >> 23) - 2 + (ceil_rule && (amax_bits & 0x7fffffu) > 0x400000u);
  return (uint32_t)min(max(e, 0), 252);
}
// eight values, already divided by the scale, to eight nibbles: round to
// nearest, ties to an even code, saturating at 6
__device__ __forceinline__ uint32_t mx4_encode8(const float (&v)[8]) {
  uint32_t r;
  asm("{ .reg .b8 b0, b1, b2, b3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      "mov.b32 %0, {b0, b1, b2, b3}; }"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// 1 / scale as fp32: exact, scale bytes 0 .. 253 (255: 0, every code 0)
__device__ __forceinline__ float mx4_inv_scale(uint32_t s) {
  return s == 255u ? 0.0f : __uint_as_float((254u - s) << 23);
}
#endif
