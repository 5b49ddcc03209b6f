// Tiles of the paged cache in registers and their products on the matrix
// cores, shared by the softmax decode, the attention-weight and the chunk kernels.
//
// Scores are computed transposed, S^T = K Q^T (A = K: 16 tokens, B = Q: 16
// query rows), so that a lane holds the scores of ONE row (lane % 16) for the
// tokens of its lane group (lane / 16). These are the lanes and registers
// that the second product, O^T = V^T P^T, wants its B operand P^T in: the
// tokens of a bf16 tile are dealt to the A rows so that group c ends with
// tokens 8c .. 8c+7 (k indices of the 16x16x32 instruction), those of a
// float32 tile so that element i of group c is token 4c + i (k = c of the
// i-th 16x16x4 instruction). No value crosses lanes between the products, and
// row statistics, scores and outputs all sit at row = lane % 16.
#pragma once

#include <float.h>

#include <type_traits>

#include "launch.hpp"
#include "mfma.hpp"

namespace ekv {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// Tokens of one tile: two 16-token score tiles for bf16 caches (the 32 k
// indices of one V^T P^T instruction), one for float32 caches. A tile starts
// at a multiple of its length, so it lies in one page, or in two of 16 rows.
template <bool BF>
constexpr int kTile = BF ? 32 : 16;

// The physical pages of one tile: p0, and p1 for tokens 16..31 of a bf16 tile
// in 16-row pages (else equal to p0); -1 where the page table entry is not a
// physical page (such tokens are masked and page 0 is read in their place).
struct TilePages {
  int p0, p1;
};

// Geometry that the tile loads need: the pool, the rows of a page and the KV
// head, as byte strides.
struct KvView {
  const char* base;   // pool + KV head offset
  size_t page_bytes;  // num_kv_heads * page_size * head_dim * element size
  int page_size;      // a power of two
};

template <bool BF, int D>
__device__ __forceinline__ const char* row_ptr(const KvView& v, const TilePages& p, int t0,
                                               int tok) {
  constexpr int kRow = D * (BF ? 2 : 4);
  int pg = p.p0;
  if constexpr (BF) pg = (v.page_size == 16 && tok >= 16) ? p.p1 : p.p0;
  const int row = (t0 + tok) & (v.page_size - 1);
  return v.base + (size_t)max(pg, 0) * v.page_bytes + (size_t)row * kRow;
}

// Read once, so not kept in the caches.
template <typename T>
__device__ __forceinline__ T load_vec(const char* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const T*>(p));
}

// ---------------------------------------------------------------------------
// bf16 <-> float32 splits

// x = p0 + p1 + p2 exactly, each part a bf16 value (the top 8 significant
// bits left of what remains): parts as float32 with the low half clear.
__device__ __forceinline__ void split3(float x, uint32_t (&p)[3]) {
  p[0] = __float_as_uint(x) & 0xffff0000u;
  const float r1 = x - __uint_as_float(p[0]);
  p[1] = __float_as_uint(r1) & 0xffff0000u;
  p[2] = __float_as_uint(r1 - __uint_as_float(p[1]));
}

// (hi16(b) << 16) | hi16(a): two bf16 values of one register pair
__device__ __forceinline__ uint32_t pack_hi(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07060302u);
}
__device__ __forceinline__ uint32_t pack_lo(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x05040100u);
}

// bf16 bits of x rounded to nearest even, NaN kept
__device__ __forceinline__ uint32_t bf16_round(float x) {
  return x != x ? 0x7fc0u : bf16_rne_bits(x);
}

__device__ __forceinline__ bf16x8 as_bf(const u32x4& v) { return __builtin_bit_cast(bf16x8, v); }

// ---------------------------------------------------------------------------
// Tiles staged in LDS for several waves

// Byte addresses in LDS, as the 32-bit numbers that they are.
typedef uint32_t lds_at;
#define EKV_LDS __attribute__((address_space(3)))
__device__ __forceinline__ lds_at lds_addr(const void* p) {
  return (lds_at)(uintptr_t)(EKV_LDS const char*)p;
}
template <typename T>
__device__ __forceinline__ T lds_read(lds_at p) {
  return *(EKV_LDS const T*)p;
}

// A stage is two tiles of K and the same of V. Row r of 16-byte chunks lies at
// r * row bytes, chunk ch at slot ch ^ swizzle(r): the 16 tokens that a score
// operand reads at one chunk fall on different banks (without it all 16 hit
// the same ones), and so do the 4 rows x 2 chunks of a transposing read.
template <bool BF, int D>
struct Stage {
  static constexpr int kTokens = 2 * kTile<BF>;
  static constexpr int kRow = D * (BF ? 2 : 4);
  static constexpr int kChunks = kRow / 16;
  static constexpr int kBytes = kTokens * kRow;  // of K, and of V
  __device__ __forceinline__ static int swizzle(int r) {
    return (BF ? (r & 3) << 1 | ((r >> 4) & 1) | ((r >> 3) & 1) << 3 : r & 15) & (kChunks - 1);
  }
  __device__ __forceinline__ static int at(int r, int ch) {
    return r * kRow + ((ch ^ swizzle(r)) << 4);
  }
  // The place of chunk ch | by from that of chunk ch (no common bits; rows
  // are aligned to their length): one operation, no register per chunk.
  __device__ __forceinline__ static lds_at on(lds_at p, int by) { return p ^ (unsigned)(by << 4); }
};

// One K tile streamed into LDS by one wave for itself, whole rows at a time
// (a score operand loaded straight from memory touches 64 bytes of 16 rows at
// once: the weights of 128K tokens in 51.6 us, 45.5 by whole rows). Same layout
// as a stage.
template <bool BF, int D>
struct WaveTile {
  static constexpr int kBytes = Stage<BF, D>::kBytes / 2;
  static constexpr int kLoads = kBytes / 1024;
  static constexpr int kRow = Stage<BF, D>::kRow;
  int from[kLoads];  // this lane's source past the tile's first row, per load
  int row[kLoads];   // and its row (uniform over kRow / 16 lanes)
  __device__ __forceinline__ void init(int lane) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = i * 1024 + lane * 16;
      row[i] = at / kRow;
      from[i] = ((at % kRow / 16) ^ Stage<BF, D>::swizzle(row[i])) << 4;
    }
  }
  __device__ __forceinline__ void load(const KvView& v, const TilePages& p, int t0,
                                       char* dst) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      lds_load16(row_ptr<BF, D>(v, p, t0, row[i]) + from[i], dst + i * 1024);
  }
};

// ---------------------------------------------------------------------------
// Query rows as the B operand

// PARTS: bf16 parts of a query value (3 for float32 queries: the exact split
// above, so products with bf16 keys are exact; 1 for bf16 queries).
template <bool BF, int D, int PARTS>
struct QFrag;

template <int D, int PARTS>
struct QFrag<true, D, PARTS> {
  u32x4 f[PARTS][D / 32];
  // `row`: the row's first value (null: a row of zeros)
  __device__ __forceinline__ void load(const char* row, int c) {
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
      const int d = s * 32 + c * 8;
      if constexpr (PARTS == 1) {
        f[0][s] = row ? *reinterpret_cast<const u32x4*>(row + 2 * d) : u32x4{0, 0, 0, 0};
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const f32x4 x = row ? *reinterpret_cast<const f32x4*>(row + 4 * (d + 4 * h))
                              : f32x4{0, 0, 0, 0};
          uint32_t p[4][3];
#pragma unroll
          for (int e = 0; e < 4; ++e) split3(x[e], p[e]);
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            f[k][s][2 * h] = pack_hi(p[0][k], p[1][k]);
            f[k][s][2 * h + 1] = pack_hi(p[2][k], p[3][k]);
          }
        }
      }
    }
  }
};

template <int D, int PARTS>
struct QFrag<false, D, PARTS> {
  f32x4 f[D / 16];
  __device__ __forceinline__ void load(const char* row, int c) {
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
      f[s] = row ? *reinterpret_cast<const f32x4*>(row + 4 * (s * 16 + c * 4))
                 : f32x4{0, 0, 0, 0};
  }
};

// ---------------------------------------------------------------------------
// Key tiles and scores. z[i]: the score of this lane's row and token
// tile_token<BF>(lane group, i).

template <bool BF>
__device__ __forceinline__ constexpr int scores_per_lane() { return BF ? 8 : 4; }

template <bool BF>
__device__ __forceinline__ int tile_token(int c, int i) { return BF ? c * 8 + i : c * 4 + i; }

template <bool BF, int D>
struct KTile;

template <int D>
struct KTile<true, D> {
  u32x4 f[2][D / 32];
  __device__ __forceinline__ void load(const KvView& v, const TilePages& p, int t0, int lane) {
    const int m = lane & 15, c = lane >> 4;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const char* r = row_ptr<true, D>(v, p, t0, ((m >> 2) << 3) + u * 4 + (m & 3)) + c * 16;
#pragma unroll
      for (int s = 0; s < D / 32; ++s) f[u][s] = load_vec<u32x4>(r + s * 64);
    }
  }
  // tile `sub` of a stage
  __device__ __forceinline__ void read(lds_at st, int sub, int lane) {
    typedef Stage<true, D> St;
    const int m = lane & 15, c = lane >> 4;
    const lds_at r = st + St::at(((m >> 2) << 3) + (m & 3), c);
#pragma unroll
    for (int s = 0; s < D / 32; ++s)
#pragma unroll
      for (int u = 0; u < 2; ++u)  // 4 rows further: the same swizzle
        f[u][s] = lds_read<u32x4>(St::on(r, 4 * s) + sub * (St::kBytes / 2) + u * 4 * St::kRow);
  }
  template <int PARTS>
  __device__ __forceinline__ void scores(const QFrag<true, D, PARTS>& q, float (&z)[8]) const {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f32x4 a = {0, 0, 0, 0};
#pragma unroll
      for (int k = PARTS - 1; k >= 0; --k)
#pragma unroll
        for (int s = 0; s < D / 32; ++s)
          a = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf(f[u][s]), as_bf(q.f[k][s]), a, 0, 0,
                                                      0);
#pragma unroll
      for (int i = 0; i < 4; ++i) z[u * 4 + i] = a[i];
    }
  }
};

template <int D>
struct KTile<false, D> {
  f32x4 f[D / 16];
  __device__ __forceinline__ void load(const KvView& v, const TilePages& p, int t0, int lane) {
    const char* r = row_ptr<false, D>(v, p, t0, lane & 15) + (lane >> 4) * 16;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) f[s] = load_vec<f32x4>(r + s * 64);
  }
  __device__ __forceinline__ void read(lds_at st, int sub, int lane) {
    typedef Stage<false, D> St;
    const lds_at r = st + St::at(lane & 15, lane >> 4);
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
      f[s] = lds_read<f32x4>(St::on(r, 4 * s) + sub * (St::kBytes / 2));
  }
  template <int PARTS>
  __device__ __forceinline__ void scores(const QFrag<false, D, PARTS>& q, float (&z)[4]) const {
    // four sums of D/4 products each: shorter chains round less (one chain:
    // 1.8 times the error at D = 128) and do not wait for each other
    f32x4 a[4] = {{0, 0, 0, 0}, {0, 0, 0, 0}, {0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        a[e] = __builtin_amdgcn_mfma_f32_16x16x4f32(f[s][e], q.f[s][e], a[e], 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = (a[0][i] + a[1][i]) + (a[2][i] + a[3][i]);
  }
};

// ---------------------------------------------------------------------------
// Weights as the B operand of the second product

// PP bf16 parts: 3 (p exact, for float32 queries) or 2 (for bf16 ones, whose
// output is rounded to 8 bits: p to the nearest of 8 bits and what remains to
// the nearest of 8 more, at most 2^-17 of p off, to either side. Two cut-off
// parts are up to 2^-15 off, all to one side; one rounded part, 2^-8, moved
// the output's error against 64 bits from 1.66e-3 to 2.2e-3.)
template <bool BF, int PP>
struct PFrag;

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two values to the nearest bf16, ties to even.
__device__ __forceinline__ uint32_t nearest2(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

template <int PP>
struct PFrag<true, PP> {
  u32x4 b[PP];
  __device__ __forceinline__ void set(const float (&p)[8]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float x = p[2 * k], y = p[2 * k + 1];
      if constexpr (PP == 2) {
        const uint32_t h = nearest2(x, y);
        b[0][k] = h;
        b[1][k] = nearest2(x - __uint_as_float(h << 16), y - __uint_as_float(h & 0xffff0000u));
      } else {
        uint32_t u[3], w[3];
        split3(x, u);
        split3(y, w);
#pragma unroll
        for (int s = 0; s < PP; ++s) b[s][k] = pack_hi(u[s], w[s]);
      }
    }
  }
};

template <int PP>
struct PFrag<false, PP> {
  float b[4];
  __device__ __forceinline__ void set(const float (&p)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = p[i];
  }
};

// ---------------------------------------------------------------------------
// Output accumulator: rows x D, spread as acc[n][i]; `first(c, n, i)` below
// says which coordinates a lane holds.

template <bool BF, int D>
struct VTile;

// Each lane loads D/16 neighbouring coordinates of the 8 tokens of its group
// (a whole row per 16 lanes) and transposes them in registers: instruction n
// takes coordinate n of every lane, so its 16 A rows are d = (D/16) m + n.
template <int D>
struct VTile<true, D> {
  static constexpr int kAcc = D / 16;
  typedef typename std::conditional<D == 128, u32x4, u32x2>::type vec;
  vec f[8];
  __device__ __forceinline__ void load(const KvView& v, const TilePages& p, int t0, int lane) {
    const int m = lane & 15, c = lane >> 4;
    const char* r = row_ptr<true, D>(v, p, t0, c * 8) + m * (D / 8);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = load_vec<vec>(r + j * (D * 2));
  }
  __device__ __forceinline__ void clear(int j) { f[j] = vec(0); }
  // An infinity or NaN among the values held?
  __device__ __forceinline__ bool any_nonfinite() const {
    u16x2 big = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < D / 32; ++e)
        big = __builtin_elementwise_max(big, __builtin_bit_cast(u16x2, f[j][e] & 0x7fff7fffu));
    return big[0] >= 0x7f80 || big[1] >= 0x7f80;
  }
  // acc[n] += V^T P^T, instruction n
  template <int PP>
  __device__ __forceinline__ f32x4 mul(int n, const PFrag<true, PP>& p, f32x4 o) const {
    u32x4 a;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      a[k] = (n & 1) ? pack_hi(f[2 * k][n / 2], f[2 * k + 1][n / 2])
                     : pack_lo(f[2 * k][n / 2], f[2 * k + 1][n / 2]);
#pragma unroll
    for (int s = PP - 1; s >= 0; --s)
      o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf(a), as_bf(p.b[s]), o, 0, 0, 0);
    return o;
  }
  // coordinate of acc[n][i]
  __device__ __forceinline__ static int coord(int c, int n, int i) {
    return (c * 4 + i) * (D / 16) + n;
  }
};

template <int D>
struct VTile<false, D> {
  static constexpr int kAcc = D / 16;
  f32x4 f[4][D / 64];
  __device__ __forceinline__ void load(const KvView& v, const TilePages& p, int t0, int lane) {
    const int m = lane & 15, c = lane >> 4;
    const char* r = row_ptr<false, D>(v, p, t0, c * 4) + m * 16;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
        f[j][h] = load_vec<f32x4>(r + j * (D * 4) + h * 256);
  }
  __device__ __forceinline__ void clear(int j) {
#pragma unroll
    for (int h = 0; h < D / 64; ++h) f[j][h] = f32x4{0, 0, 0, 0};
  }
  __device__ __forceinline__ bool any_nonfinite() const {
    uint32_t big = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) big = max(big, __float_as_uint(f[j][h][e]) & 0x7fffffffu);
    return big >= 0x7f800000u;
  }
  template <int PP>
  __device__ __forceinline__ f32x4 mul(int n, const PFrag<false, PP>& p, f32x4 o) const {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o = __builtin_amdgcn_mfma_f32_16x16x4f32(f[j][n >> 2][n & 3], p.b[j], o, 0, 0, 0);
    return o;
  }
  __device__ __forceinline__ static int coord(int c, int n, int i) {
    return (n >> 2) * 64 + (c * 4 + i) * 4 + (n & 3);
  }
};

// ---------------------------------------------------------------------------
// Value tiles of a stage, used by several row tiles of a wave

template <bool BF, int D>
struct StageV;

// The transposing LDS read gives lane n of 16 the column n of 4 rows x 16
// columns: two make the 8 tokens of a group at coordinate 16 n + m, so acc[n][i]
// holds coordinate 16 n + 4 c + i, and nothing is shuffled in registers.
template <int D>
struct StageV<true, D> {
  static constexpr int kAcc = D / 16;
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  bf16x8 f[kAcc];
  __device__ __forceinline__ void read(lds_at st, int sub, int lane, int n) {
    typedef Stage<true, D> St;
    const int m = lane & 15, c = lane >> 4;
    const int r = c * 8 + (m >> 2);  // and the row 4 further: the same swizzle
    const lds_at at =
        St::on(st + St::at(r, (m >> 1) & 1) + (m & 1) * 8, 2 * n) + sub * (St::kBytes / 2);
    const s16x4 a0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((EKV_LDS s16x4*)at);
    const s16x4 a1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((EKV_LDS s16x4*)(at + 4 * St::kRow));
    f[n] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7));
  }
  template <int PP, int RT>
  __device__ __forceinline__ void add(const PFrag<true, PP> (&p)[RT], f32x4 (&acc)[RT][kAcc],
                                      int n) const {
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int s = PP - 1; s >= 0; --s)
        acc[t][n] =
            __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[n], as_bf(p[t].b[s]), acc[t][n], 0, 0, 0);
  }
  // acc[n] += V^T P^T of tile t0 read from memory, on the tokens `see` says
  // (a bit per token of this lane's group), where `mine`
  template <int PP>
  __device__ __forceinline__ static void add_slow(const KvView& v, const TilePages& pg, int t0,
                                                  int lane, const PFrag<true, PP>& p,
                                                  unsigned see, bool mine, f32x4 (&acc)[kAcc]) {
    const int m = lane & 15, c = lane >> 4;
    const char* r = row_ptr<true, D>(v, pg, t0, c * 8) + m * 2;
#pragma unroll 1
    for (int n = 0; n < kAcc; ++n) {
      u32x4 a = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t x = *reinterpret_cast<const uint16_t*>(r + j * (D * 2) + n * 32);
        a[j / 2] |= (see >> j & 1 ? x : 0u) << (j % 2 * 16);
      }
      f32x4 o = {0, 0, 0, 0};
#pragma unroll
      for (int s = PP - 1; s >= 0; --s)
        o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf(a), as_bf(p.b[s]), o, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < kAcc; ++k)
        if (k == n && mine) acc[k] += o;
    }
  }
  __device__ __forceinline__ static int coord(int c, int n) { return n * 16 + c * 4; }
};

template <int D>
struct StageV<false, D> {
  static constexpr int kAcc = D / 16;
  float f[kAcc][4];
  __device__ __forceinline__ void read(lds_at st, int sub, int lane, int n) {
    typedef Stage<false, D> St;
    const int m = lane & 15, c = lane >> 4;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      f[n][j] = lds_read<float>(St::on(st + St::at(c * 4 + j, m >> 2) + (m & 3) * 4, 4 * n) +
                                sub * (St::kBytes / 2));
  }
  template <int PP, int RT>
  __device__ __forceinline__ void add(const PFrag<false, PP> (&p)[RT], f32x4 (&acc)[RT][kAcc],
                                      int n) const {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int t = 0; t < RT; ++t)
        acc[t][n] = __builtin_amdgcn_mfma_f32_16x16x4f32(f[n][j], p[t].b[j], acc[t][n], 0, 0, 0);
  }
  template <int PP>
  __device__ __forceinline__ static void add_slow(const KvView& v, const TilePages& pg, int t0,
                                                  int lane, const PFrag<false, PP>& p,
                                                  unsigned see, bool mine, f32x4 (&acc)[kAcc]) {
    const int m = lane & 15, c = lane >> 4;
    const char* r = row_ptr<false, D>(v, pg, t0, c * 4) + m * 4;
#pragma unroll 1
    for (int n = 0; n < kAcc; ++n) {
      f32x4 o = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x = *reinterpret_cast<const float*>(r + j * (D * 4) + n * 64);
        o = __builtin_amdgcn_mfma_f32_16x16x4f32(see >> j & 1 ? x : 0.0f, p.b[j], o, 0, 0, 0);
      }
#pragma unroll
      for (int k = 0; k < kAcc; ++k)
        if (k == n && mine) acc[k] += o;
    }
  }
  __device__ __forceinline__ static int coord(int c, int n) { return n * 16 + c * 4; }
};

// An infinity or NaN among the values of tile `sub`?
template <bool BF, int D>
__device__ __forceinline__ bool stage_nonfinite(lds_at st, int sub, int lane) {
  constexpr int kTileBytes = Stage<BF, D>::kBytes / 2;
  uint32_t big = 0;
  u16x2 bh = {0, 0};
#pragma unroll
  for (int i = 0; i < kTileBytes / 1024; ++i) {
    const u32x4 x = lds_read<u32x4>(st + sub * kTileBytes + i * 1024 + lane * 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (BF)
        bh = __builtin_elementwise_max(bh, __builtin_bit_cast(u16x2, x[e] & 0x7fff7fffu));
      else
        big = max(big, x[e] & 0x7fffffffu);
    }
  }
  return BF ? bh[0] >= 0x7f80 || bh[1] >= 0x7f80 : big >= 0x7f800000u;
}

// ---------------------------------------------------------------------------
// Outputs

// Four finished coordinates of a row.
template <int PARTS>
__device__ __forceinline__ void store_out(void* out, size_t at, f32x4 o) {
  if constexpr (PARTS == 1) {
    uint32_t h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = bf16_round(o[e]);
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(out) + at) =
        u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
  } else {
    *reinterpret_cast<f32x4*>(static_cast<float*>(out) + at) = o;
  }
}

// ---------------------------------------------------------------------------
// The tokens a block of rows sees

// Row r sees tokens t < hi_r with t >= lo_r or t < sinks. A block's tiles are
// those of [0, sinks) and of [lo, hi) (lo the least lo_r, hi the largest
// hi_r), each once: ordinal v is tile v below ns, else tile v - ns + mt0.
struct TileSpan {
  int ns, mt0, n;
  __device__ __forceinline__ int tile(int v) const { return v < ns ? v : v - ns + mt0; }
};

// (bitwise: one compare and mask operation each, no branch)
__device__ __forceinline__ bool sees(int t, int lo, int hi, int sinks) {
  return (t < hi) & ((t >= lo) | (t < sinks));
}

template <int TT>
__device__ __forceinline__ TileSpan tile_span(int lo, int hi, int sinks) {
  TileSpan s;
  if (hi <= 0) {
    s.ns = s.mt0 = s.n = 0;
    return s;
  }
  s.mt0 = min(lo, hi) / TT;
  s.ns = min((min(sinks, hi) + TT - 1) / TT, s.mt0);
  s.n = s.ns + (hi + TT - 1) / TT - s.mt0;
  return s;
}

// max over the four lanes that share lane % 16
__device__ __forceinline__ float group_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16, kWave));
  return fmaxf(x, __shfl_xor(x, 32, kWave));
}
__device__ __forceinline__ float group_sum(float x) {
  x += __shfl_xor(x, 16, kWave);
  return x + __shfl_xor(x, 32, kWave);
}

}  // namespace ekv
