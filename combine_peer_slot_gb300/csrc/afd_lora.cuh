// afd_lora.cuh -- low-rank adapters: the plan of a batch and what the kernels
// of its translation units share.
#pragma once

#include "afd_internal.cuh"

constexpr int kLoraMaxAdapters = 1024;
constexpr int kLoraMaxRank = 128;
constexpr int kLoraMaxCols = 65536;
constexpr int64_t kLoraMaxTokens = int64_t(1) << 24;

constexpr int kLoraSms = 152;  // CTAs of the kernels that hold one an SM
// Rows of one adapter that a tile of the products holds.  A decode step's rows
// bring many adapters of a few rows each; over a thousand rows the adapters'
// runs are longer.
inline int lora_tile(int64_t tokens) { return tokens <= 1024 ? 16 : 128; }
// Rows of one piece of the weight gradients' sums: enough pieces for all SMs,
// and few enough that their partial sums stay small (13312 rows of 8 adapters,
// rank 64: 512 and 1024 rows 112 us, 2048 121).
inline int lora_piece(int64_t tokens) { return tokens <= 4096 ? 128 : 512; }

// The plan, made on the device from the rows' adapter ids: the rows in adapter
// order (stable; rows without an adapter last), cut into tiles of one adapter.
//   head   {tiles, tiles of rows without an adapter, pieces, rows with one}
//   tiles  {adapter (-1: none), first row in order, rows, rows that an
//          adapter's last tile lacks to a whole block of 32}
//   pieces {adapter, first row in order, rows, slot of its partial sums or -1}
//   first  [adapters] first partial slot, then [adapters] pieces
//   shift  [adapters] from a row's place in order to its place among u_parts,
//          where each adapter begins with a block of 32 rows
struct LoraPlan {
  int4* head;
  int4* tiles;
  int4* pieces;
  int32_t* first;
  int32_t* shift;
  int32_t* order;   // [tokens]
  int64_t max_tiles, max_pieces, max_slots, bytes;
};
inline LoraPlan lora_plan_at(void* base, int64_t tokens, int64_t adapters) {
  LoraPlan p;
  const int64_t few = std::min(tokens, adapters);
  p.max_tiles = tokens / lora_tile(tokens) + few + 1;
  p.max_pieces = tokens / lora_piece(tokens) + few;
  // an adapter of several pieces has more than one piece's rows
  p.max_slots = 2 * (tokens / lora_piece(tokens));
  char* at = reinterpret_cast<char*>(base);
  auto take = [&](int64_t bytes) {
    char* r = at;
    at += (bytes + 15) / 16 * 16;
    return r;
  };
  p.head = reinterpret_cast<int4*>(take(16));
  p.tiles = reinterpret_cast<int4*>(take(16 * p.max_tiles));
  p.pieces = reinterpret_cast<int4*>(take(16 * std::max<int64_t>(1, p.max_pieces)));
  p.first = reinterpret_cast<int32_t*>(take(8 * adapters));
  p.shift = reinterpret_cast<int32_t*>(take(4 * adapters));
  p.order = reinterpret_cast<int32_t*>(take(4 * std::max<int64_t>(1, tokens)));
  p.bytes = at - reinterpret_cast<char*>(base);
  return p;
}

// out[t] = base[t] + scale[l] w2[l]^T u_t, u_t = w1[l] src[t], l = the row's adapter
struct LoraArgs {
  LoraPlan plan;
  const void* src;
  int64_t lds;
  const void* w1;      // bf16 [L][R][K]
  const void* w2;      // bf16 [L][R][M]
  const float* scale;  // [L] or NULL (1)
  const void* base;    // NULL: zeros; may be out
  int64_t ldb;
  void* out;
  int64_t ldo;
  float* u;            // [T][R] or NULL
  // for the weight gradients, or NULL: three bf16 parts of u as computed here
  // and of `other` [T][R], as their kernel copies them (parts_at)
  uint16_t* u_parts;
  const float* other;
  uint16_t* other_parts;
  int64_t T;
  int K, M, R, L;
  int src_f32, out_f32;
  // how rows can be moved: 16, 8 or 4 bytes at a time, 0 = by elements (bf16)
  int how_src, how_w1, how_w2, how_base, how_out;
};
// da[l] = scale[l] sum v_t x_t^T, db[l] = scale[l] sum u_t dy_t^T
struct LoraWgradArgs {
  LoraPlan plan;
  const uint16_t* parts[2];  // of v, of u (LoraArgs::u_parts)
  // rows x, dy: bf16, of whole 16 bytes; gathered by the plan's order or laid
  // out in it, one plane or three, `plane` elements apart
  const void* q[2];
  int64_t ldq[2], plane[2];
  int planes[2], ordered[2];
  float* out[2];             // [L][R][N]
  float* part[2];            // [slots][R][N]
  int N[2];
  const float* scale;
  int R, L;
};
inline int64_t lora_plane_pitch(int N) { return ((int64_t)N + 7) / 8 * 8; }
// Parts of u for the weight gradients: blocks of 32 rows (each adapter's first
// row begins one, the last is filled up with zeros), each the shared memory
// image of an MN-major operand with the 128-byte swizzle: atoms of 64 of a row's
// 3 MP values.  Values past those are never read into a sum.
constexpr int kLoraBlockRows = 32;
__host__ __device__ constexpr int lora_atoms(int MP) { return (3 * MP + 63) / 64; }
inline int64_t lora_parts_bytes(int64_t tokens, int64_t adapters, int MP) {
  return ((tokens + 31) / 32 + std::min(tokens, adapters)) * lora_atoms(MP) * 4096;
}
// ranks of one part
__host__ __device__ inline int lora_padded(int R) { return R <= 16 ? 16 : R <= 32 ? 32 : R <= 64 ? 64 : 128; }
cudaError_t launch_lora_apply(const LaunchCtx& lc, const LoraArgs& a);  // tiles of 16
cudaError_t launch_lora_tiles(const LaunchCtx& lc, const LoraArgs& a);  // tiles of 128, 64 at a time
bool lora_tc_takes(const LoraArgs& a);                                  // the next one's sizes and alignment
cudaError_t launch_lora_tc(const LaunchCtx& lc, const LoraArgs& a);     // tiles of 128
cudaError_t lora_tc_error_count(uint32_t* n, cudaStream_t stream);
cudaError_t launch_lora_planes(const LaunchCtx& lc, const LoraPlan& plan, int64_t tokens, const void* q, int64_t ldq, int N,
                               int f32, int vec, uint16_t* to);
cudaError_t launch_lora_wgrad(LaunchCtx lc, const LoraWgradArgs& a);
cudaError_t lora_error_count(uint32_t* n, cudaStream_t stream);  // waits that gave up, once the stream is there

#ifdef __CUDACC__
// D += A B on 16 x 8 x 16 bf16 values, fp32 sums: lane (g, c) = (lane / 4,
// lane % 4) holds of A rows g, g + 8 and of B column g the k pairs 2 c, 2 c + 8;
// of D rows g, g + 8, columns 2 c, 2 c + 1.
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// An fp32 value as a sum of bf16 values: the upper 8 bits of its fraction cut
// off, then the next 8, then the rest: three parts are the value.  Cutting, unlike rounding, cannot
// carry the largest finite values over to infinity; a value that is not finite
// is all in the first part (NaN stays NaN), with zeros behind it.
template <int PARTS>
__device__ __forceinline__ void split_bf16(float v, uint16_t (&p)[PARTS]) {
  const uint32_t b = __float_as_uint(v);
  const bool fine = (b & 0x7f800000u) != 0x7f800000u;
  p[0] = (uint16_t)(b >> 16);
  if (!fine && (b & 0x7fffffu)) p[0] |= 0x40u;
  float rest = fine ? v - __uint_as_float(b & 0xffff0000u) : 0.0f;
#pragma unroll
  for (int i = 1; i < PARTS; i++) {
    if (i == PARTS - 1) {
      p[i] = __bfloat16_as_ushort(__float2bfloat16_rn(rest));
    } else {
      const uint32_t r = __float_as_uint(rest);
      p[i] = (uint16_t)(r >> 16);
      rest -= __uint_as_float(r & 0xffff0000u);
    }
  }
}

// two neighbouring fp32 values to packed bf16 parts
template <int PARTS>
__device__ __forceinline__ void split_pair(float2 v, uint32_t (&p)[PARTS]) {
  uint16_t a[PARTS], b[PARTS];
  split_bf16<PARTS>(v.x, a);
  split_bf16<PARTS>(v.y, b);
#pragma unroll
  for (int i = 0; i < PARTS; i++) p[i] = (uint32_t)a[i] | (uint32_t)b[i] << 16;
}

// value m of a row's parts: part m / MP, rank m % MP
template <int MP>
__device__ __forceinline__ uint16_t* parts_at(uint16_t* to, int64_t row, int m) {
  const int r = (int)(row & 31);
  return to + (row >> 5) * (lora_atoms(MP) * 2048) + (m >> 6) * 2048 + r * 64 + (((m >> 3 & 7) ^ (r & 7)) << 3) + (m & 7);
}

template <typename T>
struct LoraSrc;
template <>
struct LoraSrc<uint16_t> { static constexpr int kParts = 1; };
template <>
struct LoraSrc<float> { static constexpr int kParts = 3; };

// Parts of u in the second product: all of fp32's bits, beside bf16 outputs too,
// since base or another rank may cancel what the upper ones make (two parts left
// bf16 outputs 1.1e-4 of their norm from those of an fp32 u, three 3 to 5e-5, and
// a third MMA takes 2 us of 45 over a prefill fan-in of rank 16, 2 of 112 in the
// gradients of rank 64).
constexpr int kLoraUParts = 3;

// Eight bf16 values of a row of any alignment from column c0, zeros from column
// n on: by the words that hold one of them at least (so nothing is read past
// the 4-byte word of the row's first or last value), shifted into place.
__device__ __forceinline__ uint4 load_words(const uint16_t* row, int c0, int n) {
  const int have = min(n - c0, 8);
  if (have <= 0) return make_uint4(0u, 0u, 0u, 0u);
  const uintptr_t at = reinterpret_cast<uintptr_t>(row + c0);
  const int odd = (int)(at >> 1 & 1);
  const uint32_t* from = reinterpret_cast<const uint32_t*>(at - 2 * odd);
  uint32_t w[5];
#pragma unroll
  for (int i = 0; i < 5; i++) w[i] = 2 * i < have + odd ? from[i] : 0u;
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    v[i] = __funnelshift_r(w[i], w[i + 1], 16 * odd);
    if (2 * i >= have) v[i] = 0u;
    else if (2 * i + 1 >= have) v[i] &= 0xffffu;
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// Eight neighbouring values of a row from column c0 as packed bf16 parts;
// columns from n on are zero.  vec: rows are 16-byte aligned and n % 8 == 0.
template <typename T>
__device__ __forceinline__ void load_eight(const T* row, int c0, int n, bool vec, uint4 (&v)[LoraSrc<T>::kParts]);
template <>
__device__ __forceinline__ void load_eight<uint16_t>(const uint16_t* row, int c0, int n, bool vec, uint4 (&v)[1]) {
  v[0] = make_uint4(0u, 0u, 0u, 0u);
  if (c0 >= n) return;
  if (vec) {
    v[0] = *reinterpret_cast<const uint4*>(row + c0);
    return;
  }
  uint32_t w[8];  // (load_words' longer code costs the rows that do not take it 5 % in afd_lora_apply.cu)
#pragma unroll
  for (int i = 0; i < 8; i++) w[i] = c0 + i < n ? (uint32_t)row[c0 + i] : 0u;
  v[0] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
}
template <>
__device__ __forceinline__ void load_eight<float>(const float* row, int c0, int n, bool vec, uint4 (&v)[3]) {
  float f[8];
  if (vec && c0 < n) {
    const float4 a = *reinterpret_cast<const float4*>(row + c0), b = *reinterpret_cast<const float4*>(row + c0 + 4);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) f[i] = c0 + i < n ? row[c0 + i] : 0.0f;
  }
  uint32_t w[3][8];
#pragma unroll
  for (int i = 0; i < 8; i++) {
    uint16_t p[3];
    split_bf16<3>(f[i], p);
#pragma unroll
    for (int j = 0; j < 3; j++) w[j][i] = p[j];
  }
#pragma unroll
  for (int j = 0; j < 3; j++)
    v[j] = make_uint4(w[j][0] | w[j][1] << 16, w[j][2] | w[j][3] << 16, w[j][4] | w[j][5] << 16, w[j][6] | w[j][7] << 16);
}

// Four rows' eight columns (rows 2 c, 2 c + 1, 2 c + 8, 2 c + 9 of sixteen) to
// B operands of eight products: in product i, column n of B is column 8 n + i
// of the 64, so lane (g, c) needs of its own loads (columns 8 g ..) only
__device__ __forceinline__ void pair_rows(const uint4& r0, const uint4& r1, const uint4& r2, const uint4& r3,
                                          uint32_t (&b)[8][2]) {
  const uint32_t x0[4] = {r0.x, r0.y, r0.z, r0.w}, x1[4] = {r1.x, r1.y, r1.z, r1.w};
  const uint32_t x2[4] = {r2.x, r2.y, r2.z, r2.w}, x3[4] = {r3.x, r3.y, r3.z, r3.w};
#pragma unroll
  for (int j = 0; j < 4; j++) {
    b[2 * j][0] = __byte_perm(x0[j], x1[j], 0x5410);
    b[2 * j][1] = __byte_perm(x2[j], x3[j], 0x5410);
    b[2 * j + 1][0] = __byte_perm(x0[j], x1[j], 0x7632);
    b[2 * j + 1][1] = __byte_perm(x2[j], x3[j], 0x7632);
  }
}

// ---- tiles in shared memory: rows of 128 bytes ----
constexpr int kLoraRowBytes = 128;
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void copy_few(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(in ? BYTES : 0), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm2(uint32_t addr, uint32_t& r0, uint32_t& r1) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// 16-byte chunk c of row r of a tile: chunks are swapped within a row so that
// eight rows' same chunk lie in different banks
__device__ __forceinline__ uint32_t chunk_at(uint32_t tile, int r, int c) {
  return tile + r * kLoraRowBytes + ((c ^ (r & 7)) << 4);
}

// The asynchronous copy of one chunk of a row from element c0 (n in the row;
// NULL: no row), zeros past its end; how: 16, 8 or 4 bytes at a time.
template <typename T>
__device__ __forceinline__ void copy_chunk(uint32_t dst, const T* row, int c0, int n, int how, const void* any) {
  const char* from = reinterpret_cast<const char*>(row + c0);
  const int left = row ? (n - c0) * (int)sizeof(T) : 0;  // bytes
  if (how == 16) {
    copy16(dst, left > 0 ? from : any, left > 0);
  } else if (how == 8) {
#pragma unroll
    for (int i = 0; i < 16; i += 8) copy_few<8>(dst + i, left > i ? from + i : any, left > i);
  } else {
#pragma unroll
    for (int i = 0; i < 16; i += 4) copy_few<4>(dst + i, left > i ? from + i : any, left > i);
  }
}

// Up to 128 rows without an adapter: out = base (nothing where they are the
// same), u = 0; by threads first, first + step, ..  Eight loads stand before
// their stores (one at a time, decode's few such rows took as long as all its
// products).
template <typename TO>
__device__ __forceinline__ void copy_bare(const LoraArgs& a, const int32_t* order, int rows, int first, int step) {
  constexpr int E = 16 / (int)sizeof(TO), kBatch = 8;
  const TO* base = reinterpret_cast<const TO*>(a.base);
  TO* out = reinterpret_cast<TO*>(a.out);
  if (a.base != a.out) {
    const bool vec = a.how_out == 16 && (!base || a.how_base == 16);
    const uint32_t per_row = vec ? a.M / E : a.M, all = rows * per_row;
    for (uint32_t i0 = first; i0 < all; i0 += kBatch * step) {
      uint4 v[kBatch];
      int64_t at[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; k++) {
        const uint32_t i = i0 + k * step;
        v[k] = make_uint4(0u, 0u, 0u, 0u);
        at[k] = -1;
        if (i < all) {
          const int64_t row = order[i / per_row];
          const uint32_t c = i % per_row * (vec ? E : 1);
          at[k] = row * a.ldo + c;
          if (base) {
            if (vec) v[k] = *reinterpret_cast<const uint4*>(base + row * a.ldb + c);
            else if (sizeof(TO) == 2) v[k].x = reinterpret_cast<const uint16_t*>(base)[row * a.ldb + c];
            else v[k].x = reinterpret_cast<const uint32_t*>(base)[row * a.ldb + c];
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; k++)
        if (at[k] >= 0) {
          if (vec) *reinterpret_cast<uint4*>(out + at[k]) = v[k];
          else if (sizeof(TO) == 2) reinterpret_cast<uint16_t*>(out)[at[k]] = (uint16_t)v[k].x;
          else reinterpret_cast<uint32_t*>(out)[at[k]] = v[k].x;
        }
    }
  }
  if (a.u)
    for (uint32_t i = first; i < (uint32_t)(rows * a.R); i += step) a.u[(int64_t)order[i / a.R] * a.R + i % a.R] = 0.0f;
}

// ---- tcgen05, one CTA: issued by the elected lane of a warp that runs its loop
// as a whole.  Under a branch on the lane the operands would leave the uniform
// registers that these instructions take them from: four MMAs and a commit
// then took 740 cycles. ----
__device__ __forceinline__ uint32_t lora_elect() {
  uint32_t e;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(e));
  return e;
}
// descriptors: the layout's upper word, address (16-byte units) and, of MN-major
// operands of two atoms, their distance in the lower
__device__ __forceinline__ uint64_t lora_desc(uint32_t addr16, uint32_t apart16) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(addr16 | apart16 << 16), "r"((1024u >> 4) | 1u << 14 | 2u << 29));
  return d;
}
__device__ __forceinline__ void lora_mma(uint32_t elected, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p, q; setp.ne.b32 p, %4, 0; setp.ne.b32 q, %5, 0;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void lora_commit(uint32_t elected, uint32_t bar) {
  asm volatile(
      "{ .reg .pred q; setp.ne.b32 q, %1, 0;\n"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(bar), "r"(elected)
      : "memory");
}
#endif
