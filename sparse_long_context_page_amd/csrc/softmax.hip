// Softmax decode attention over the paged cache: a window with sinks, and a
// batch that shares a prefix.
//
//   z_t = q . k_t,  m = max z_t,  l = sum exp(z_t - m),
//   out = sum exp(z_t - m) v_t / l,  lse = m + ln l
//
// over the tokens a query sees. One pass over K and V: a wave holds 16 query
// rows a tile (the heads of one KV group, times query tokens or sequences),
// their reference m, sum l and output in registers, and walks tiles of tokens
// (softmax_impl.hpp). Any reference m gives the same quotient, so m follows
// the running maximum only when that has grown by more than kSlack: the sum
// stays below e^kSlack * tokens, far inside float32, and almost no tile pays
// for a rescale or a reduction across lanes.
//
// Two forms of a workgroup (chosen by kAttManyRows and the two bounds after it):
//  - few rows (attend_tokens): the waves share at most 16 rows and take turns
//    at the tiles, loaded from memory straight into the operands' registers;
//    bound by reading K and V (a window of 4096 for 64 sequences, 8 KV heads
//    of 128 bf16 dims: 1.08 GB in 169 us, 6.4 TB/s).
//  - many rows (attend_rows): each wave has row tiles of its own and all walk
//    the same tokens, staged once per workgroup in LDS by direct loads, one
//    stage ahead; bound by the matrix cores and the exponentials (2 x 512
//    queries of 32 heads over 2048 tokens: 34 GFLOP in 63 us, 0.55 PFLOP/s).
// The tokens of a row block are split over workgroups; the parts (m_s, l_s,
// o_s) are joined by a second kernel: out = sum e^(m_s - M) o_s / sum e^(m_s -
// M) l_s.
#include <atomic>

#include "softmax_impl.hpp"

namespace ekv {
namespace {

constexpr float kSlack = 6.0f;

// bf16 parts of a weight (PFrag) by those of a query, the same in both forms:
// how a row is rounded does not depend on the batch that it is in. The sum l
// is of the whole weights.
template <int PARTS>
constexpr int kWeightParts = PARTS == 1 ? 2 : 3;

constexpr long long kAloneBytes = 160 * 1024;

// Division of x < 2^31 by a positive constant: the quotient from the
// reciprocal is at most one short.
struct Divisor {
  uint32_t d, r;
};
Divisor divisor(int d) {
  const uint64_t r = (1ull << 32) / (uint32_t)(d < 1 ? 1 : d);
  return Divisor{(uint32_t)(d < 1 ? 1 : d), r > 0xffffffffull ? 0xffffffffu : (uint32_t)r};
}
__device__ __forceinline__ int quotient(int x, const Divisor& v) {
  const uint32_t q = __umulhi((uint32_t)x, v.r);
  return (int)(q + ((uint32_t)x - q * v.d >= v.d ? 1u : 0u));
}

struct AttendArgs {
  const void* q;
  const void* k_pool;
  const void* v_pool;
  const int32_t* prefix_table;  // prefix part: pages of the shared prefix
  const int32_t* block_table;
  const int32_t* seq_lens;
  void* out;
  float* lse;     // nullable
  float* part_o;  // [rows, slots, D]
  float* part_ml; // [rows, slots, 2]
  int batch, H, Hkv, g_bits, n, ps_bits, max_pages, num_phys;  // 2^g_bits heads a KV head
  int window, sinks;
  int prefix;                                  // tokens of the shared prefix (0: none)
  int pre_block, pre_splits;                   // rows per block and splits of the prefix part
  Divisor by_hkv, by_pre_splits, by_pre_blocks, by_blocks, by_splits;
  int row_block, row_blocks, splits;           // of the sequences' own part
  int slots;                                   // parts per row
  int own_items;                               // workgroups of that part: the first
};

// What one workgroup works on. Items go over the KV heads first: the blocks
// that read the same head's tokens are a multiple of num_kv_heads apart, so
// that with 8 heads they share an XCD and its L2.
struct Block {
  int b, g;       // sequence (prefix part: none) and KV head
  int r0, nrows;  // first row of the block among its rows, rows of it
  int split, splits, slot;
  bool pre;
};

__device__ __forceinline__ Block block_of(const AttendArgs& a, int item) {
  Block w;
  w.pre = item >= a.own_items;
  if (w.pre) item -= a.own_items;
  int x = quotient(item, a.by_hkv);
  w.g = item - x * a.Hkv;
  if (w.pre) {
    // the row blocks that read the same tokens follow each other
    w.split = quotient(x, a.by_pre_blocks);
    w.b = 0;
    w.r0 = (x - w.split * (int)a.by_pre_blocks.d) * a.pre_block;
    w.nrows = min(a.pre_block, (a.batch << a.g_bits) - w.r0);
    w.splits = a.pre_splits;
    w.slot = w.split;
  } else {
    const int y = quotient(x, a.by_splits);
    w.split = x - y * a.splits;
    w.b = quotient(y, a.by_blocks);
    w.r0 = (y - w.b * a.row_blocks) * a.row_block;
    w.nrows = min(a.row_block, (a.n << a.g_bits) - w.r0);
    w.splits = a.splits;
    w.slot = a.pre_splits + w.split;
  }
  return w;
}

// Index of row r of the block's part among all [batch, n, H] rows, and the
// tokens it sees.
__device__ __forceinline__ void row_of(const AttendArgs& a, const Block& w, int L, int r,
                                       int* row, int* lo, int* hi) {
  if (w.pre) {
    const int b = r >> a.g_bits;
    *row = b * a.H + (w.g << a.g_bits) + (r - (b << a.g_bits));
    *lo = 0;
    *hi = min(clamp_len(a.seq_lens[b], a.max_pages << a.ps_bits), a.prefix);
  } else {
    const int i = r >> a.g_bits;
    *row = (w.b * a.n + i) * a.H + (w.g << a.g_bits) + (r - (i << a.g_bits));
    const int pos = L - a.n + i;
    *hi = max(pos + 1, 0);
    *lo = max(max(pos - a.window + 1, a.prefix), 0);
  }
}

// Tokens [lo, hi) that some of the rows r0 .. r0 + nrows - 1 sees and [flo,
// fhi) that all of them see (besides the sinks).
struct Span {
  int lo, hi, flo, fhi;
};
__device__ __forceinline__ Span span_of(const AttendArgs& a, int L, int r0, int nrows) {
  const int p0 = L - a.n + (r0 >> a.g_bits), p1 = L - a.n + ((r0 + nrows - 1) >> a.g_bits);
  Span s;
  s.lo = max(max(p0 - a.window + 1, a.prefix), 0);
  s.hi = max(p1 + 1, 0);
  s.flo = max(max(p1 - a.window + 1, a.prefix), 0);
  s.fhi = max(p0 + 1, 0);
  return s;
}
// The same of prefix rows, from the lanes' own hi (rows that are none: 0).
__device__ __forceinline__ Span span_of_prefix(int hi, bool live) {
  int u = hi, f = live ? hi : INT32_MAX;
#pragma unroll
  for (int s = 1; s < 16; s <<= 1) {
    u = max(u, __shfl_xor(u, s, kWave));
    f = min(f, __shfl_xor(f, s, kWave));
  }
  return Span{0, __builtin_amdgcn_readfirstlane(u), 0, __builtin_amdgcn_readfirstlane(f)};
}

struct Views {
  KvView k, v;
  const int32_t* table;
};
template <bool BF, int D>
__device__ __forceinline__ Views views_of(const AttendArgs& a, const Block& w) {
  constexpr int kElem = BF ? 2 : 4;
  Views x;
  const size_t head_off = ((size_t)w.g << a.ps_bits) * (D * kElem);
  x.k.base = static_cast<const char*>(a.k_pool) + head_off;
  x.v.base = static_cast<const char*>(a.v_pool) + head_off;
  x.k.page_bytes = x.v.page_bytes = ((size_t)a.Hkv << a.ps_bits) * (D * kElem);
  x.k.page_size = x.v.page_size = 1 << a.ps_bits;
  x.table = w.pre ? a.prefix_table : a.block_table + (size_t)w.b * a.max_pages;
  return x;
}

// Table entry j, -1 past npages and where it is no physical page.
__device__ __forceinline__ int page_at(const AttendArgs& a, const int32_t* table, int npages,
                                       int j) {
  const int p = j < npages ? table[j] : -1;
  return p < a.num_phys ? p : -1;
}

// m before any token: below every score, and finite, also times log2(e)
// where weight() forms that product alone.
template <int PARTS>
constexpr float kLowest = PARTS == 1 ? -FLT_MAX / 2 : -FLT_MAX;

// exp(z - m). float32 queries: the difference first (no rounding near the
// maximum); bf16 ones: one multiply-add, |z| 2^-24 off.
template <int PARTS>
__device__ __forceinline__ float weight(float z, float m) {
  if constexpr (PARTS == 1) return __builtin_amdgcn_exp2f(fmaf(z, kLog2e, -m * kLog2e));
  return __builtin_amdgcn_exp2f((z - m) * kLog2e);
}

// The reference m follows the maximum of a tile's scores.
template <int N>
__device__ __forceinline__ void raise(float tmax, float& m, float& l, f32x4 (&acc)[N]) {
  const float mn = fmaxf(m, group_max(tmax));
  const float f = __builtin_amdgcn_exp2f((m - mn) * kLog2e);
  l *= f;
#pragma unroll
  for (int n = 0; n < N; ++n) acc[n] *= f;
  m = mn;
}

// A tile in which the rows see different tokens and some value is not finite,
// which must not meet the zero weight of a row that does not see it: one row
// at a time, on the values that it sees. (The weights are in l already.)
// kStage: acc lies as the many-rows form keeps it.
template <bool BF, int D, int PARTS, int PP, bool kStage, int N>
__device__ __forceinline__ void late_tile(const Views& x, TilePages pg, int t0, int lane,
                                          const QFrag<BF, D, PARTS>& q, int lo, int hi, int sinks,
                                          float m, f32x4 (&acc)[N]) {
  constexpr int NZ = scores_per_lane<BF>();
  const int c = lane >> 4, rl = lane & 15;
  const bool page_ok = (!BF || c < 2 ? pg.p0 : pg.p1) >= 0;
  KTile<BF, D> kt;
  float p[NZ];
  kt.load(x.k, pg, t0, lane);
  kt.template scores<PARTS>(q, p);
#pragma unroll
  for (int i = 0; i < NZ; ++i) {
    const int t = t0 + tile_token<BF>(c, i);
    p[i] = page_ok & sees(t, lo, hi, sinks) ? weight<PARTS>(p[i], m) : 0.0f;
  }
  PFrag<BF, PP> pf;
  pf.set(p);
#pragma unroll 1
  for (int r = 0; r < 16; ++r) {
    const int rlo = __shfl(lo, r, kWave), rhi = __shfl(hi, r, kWave);
    unsigned see = 0;
#pragma unroll
    for (int i = 0; i < NZ; ++i)
      see |= (unsigned)(page_ok & sees(t0 + tile_token<BF>(c, i), rlo, rhi, sinks)) << i;
    if constexpr (kStage) {
      StageV<BF, D>::template add_slow<PP>(x.v, pg, t0, lane, pf, see, rl == r, acc);
    } else {
      VTile<BF, D> vt;
      vt.load(x.v, pg, t0, lane);
#pragma unroll
      for (int i = 0; i < NZ; ++i)
        if (!(see >> i & 1)) vt.clear(i);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const f32x4 o = vt.template mul<PP>(n, pf, f32x4{0, 0, 0, 0});
        if (rl == r) acc[n] += o;
      }
    }
  }
}

__device__ __forceinline__ float inverse(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }
// (l is 0 or at least about 1: m is never above the largest score)
__device__ __forceinline__ float log_sum(float m, float l) {
  return l == 0.0f ? -INFINITY : m + kLn2 * __builtin_amdgcn_logf(l);
}

// ---------------------------------------------------------------------------
// Few rows

template <int D, int NW>
struct TokensLds {
  float o[NW][16][D + 4];
  float ml[NW][16][2];
};

template <bool BF, int D, int PARTS, int NW>
__device__ __forceinline__ void attend_tokens(const AttendArgs& a, const Block& w, char* smem) {
  constexpr int TT = kTile<BF>;
  constexpr int NZ = scores_per_lane<BF>();
  constexpr int PP = kWeightParts<PARTS>;
  constexpr int QB = PARTS == 1 ? 2 : 4;
  constexpr int kAcc = VTile<BF, D>::kAcc;
  TokensLds<D, NW>& sh = *reinterpret_cast<TokensLds<D, NW>*>(smem);

  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = lane >> 4, rl = lane & 15;

  const int L = w.pre ? a.prefix : clamp_len(a.seq_lens[w.b], a.max_pages << a.ps_bits);
  int lo = 0, hi = 0, row = 0;
  if (rl < w.nrows) row_of(a, w, L, w.r0 + rl, &row, &lo, &hi);
  const int sinks = a.sinks;
  const Span u = w.pre ? span_of_prefix(hi, rl < w.nrows) : span_of(a, L, w.r0, w.nrows);
  const TileSpan span = tile_span<TT>(u.lo, u.hi, sinks);
  const int per = quotient(span.n + w.splits - 1, w.pre ? a.by_pre_splits : a.by_splits);
  const int v0 = min(w.split * per, span.n), v1 = min(v0 + per, span.n);
  const int npages = (u.hi + (1 << a.ps_bits) - 1) >> a.ps_bits;
  const Views x = views_of<BF, D>(a, w);

  QFrag<BF, D, PARTS> q;
  q.load(rl < w.nrows ? static_cast<const char*>(a.q) + (size_t)row * (D * QB) : nullptr, c);

  f32x4 acc[kAcc];
#pragma unroll
  for (int n = 0; n < kAcc; ++n) acc[n] = f32x4{0, 0, 0, 0};
  float m = kLowest<PARTS>, l = 0.0f;

  for (int base = v0 + wave; base < v1; base += NW * kWave) {
    // pages of this wave's next 64 tiles, one tile per lane
    const int nt = min(kWave, (v1 - base + NW - 1) / NW);
    int pg0 = -1, pg1 = -1;
    if (lane < nt) {
      const int j = (span.tile(base + lane * NW) * TT) >> a.ps_bits;
      pg0 = pg1 = page_at(a, x.table, npages, j);
      if (BF && a.ps_bits == 4) pg1 = page_at(a, x.table, npages, j + 1);
    }
    KTile<BF, D> kt;
    VTile<BF, D> vt;
    auto pages = [&](int j) {
      return TilePages{__builtin_amdgcn_readlane(pg0, j), __builtin_amdgcn_readlane(pg1, j)};
    };
    auto start = [&](int j) { return span.tile(base + j * NW) * TT; };
    TilePages pc = pages(0);
    int t0 = start(0);
    kt.load(x.k, pc, t0, lane);
    vt.load(x.v, pc, t0, lane);
    uint64_t put_off = 0;
    for (int j = 0; j < nt; ++j) {
      float z[NZ];
      kt.template scores<PARTS>(q, z);
      TilePages pn = pc;
      int tn = t0;
      if (j + 1 < nt) {
        pn = pages(j + 1);
        tn = start(j + 1);
        kt.load(x.k, pn, tn, lane);
      }
      const bool full = pc.p0 >= 0 && pc.p1 >= 0 &&
                        (t0 + TT <= u.fhi && (t0 >= u.flo || t0 + TT <= sinks));
      const bool page_ok = (!BF || c < 2 ? pc.p0 : pc.p1) >= 0;
      if (!full) {
#pragma unroll
        for (int i = 0; i < NZ; ++i) {
          const int t = t0 + tile_token<BF>(c, i);
          z[i] = page_ok & sees(t, lo, hi, sinks) ? z[i] : -INFINITY;
        }
      }
      float tmax = z[0];
#pragma unroll
      for (int i = 1; i < NZ; ++i) tmax = fmaxf(tmax, z[i]);
      if (__any(tmax > m + kSlack)) raise(tmax, m, l, acc);
      float p[NZ];
#pragma unroll
      for (int i = 0; i < NZ; ++i) {
        p[i] = weight<PARTS>(z[i], m);
        l += p[i];
      }
      bool later = false;
      if (!full) {
        // tokens that no row sees take no part, whatever their rows hold
#pragma unroll
        for (int i = 0; i < NZ; ++i) {
          const int t = t0 + tile_token<BF>(c, i);
          if (!(page_ok & sees(t, u.lo, u.hi, sinks))) vt.clear(i);
        }
        later = __any(vt.any_nonfinite());
      }
      if (later) {
        put_off |= 1ull << j;
      } else {
        PFrag<BF, PP> pf;
        pf.set(p);
#pragma unroll
        for (int n = 0; n < kAcc; ++n) acc[n] = vt.template mul<PP>(n, pf, acc[n]);
      }
      if (j + 1 < nt) vt.load(x.v, pn, tn, lane);
      pc = pn;
      t0 = tn;
    }
    while (put_off) {
      const int j = __builtin_ctzll(put_off);
      put_off &= put_off - 1;
      late_tile<BF, D, PARTS, PP, false>(x, pages(j), start(j), lane, q, lo, hi, sinks, m, acc);
    }
  }

  // join the waves' parts
  l = group_sum(l);
  if (rl < w.nrows) {
    if (c == 0) {
      sh.ml[wave][rl][0] = m;
      sh.ml[wave][rl][1] = l;
    }
#pragma unroll
    for (int n = 0; n < kAcc; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) sh.o[wave][rl][VTile<BF, D>::coord(c, n, i)] = acc[n][i];
  }
  __syncthreads();
  constexpr int TPR = D / 4;  // threads per row, 4 coordinates each
  for (int r = tid / TPR; r < w.nrows; r += NW * kWave / TPR) {
    const int d = (tid % TPR) * 4;
    float M = -FLT_MAX;
#pragma unroll
    for (int v = 0; v < NW; ++v)
      if (!(sh.ml[v][r][1] == 0.0f)) M = fmaxf(M, sh.ml[v][r][0]);
    float ls = 0.0f;
    f32x4 o = {0, 0, 0, 0};
#pragma unroll
    for (int v = 0; v < NW; ++v) {
      const float lv = sh.ml[v][r][1];
      if (lv == 0.0f) continue;
      const float f = __builtin_amdgcn_exp2f((sh.ml[v][r][0] - M) * kLog2e);
      ls += f * lv;
      o += f * *reinterpret_cast<const f32x4*>(&sh.o[v][r][d]);
    }
    int grow, dlo, dhi;
    row_of(a, w, L, w.r0 + r, &grow, &dlo, &dhi);
    if (a.slots > 1) {
      const size_t part = (size_t)grow * a.slots + w.slot;
      *reinterpret_cast<f32x4*>(a.part_o + part * D + d) = o;
      if (d == 0) {
        a.part_ml[2 * part] = M;
        a.part_ml[2 * part + 1] = ls;
      }
    } else {
      store_out<PARTS>(a.out, (size_t)grow * D + d, o * inverse(ls));
      if (d == 0 && a.lse) a.lse[grow] = log_sum(M, ls);
    }
  }
}

// ---------------------------------------------------------------------------
// Many rows

// Row tiles a wave holds: two with bf16 queries (32 rows share each K and V
// operand); one with float32 ones, whose three parts fill the registers.
template <bool BF, int PARTS>
constexpr int kRowTiles = BF && PARTS == 1 ? 2 : 1;

// GR groups of four waves: each group takes its share of the workgroup's
// stages for all of its rows. A chunk of a prompt runs with two: a CU's eight
// waves finish a row block with one part (four waves and twice the splits: 14
// us more in the join of 32768 rows). A shared prefix runs with one, beside a
// workgroup that reads the sequences' own tokens.
constexpr int kRowWaves = 4;

template <bool BF, int D, int PARTS, int GR>
struct RowsLds {
  union {
    char st[GR][2][2][Stage<BF, D>::kBytes];  // [group][buffer][K, V]
    f32x4 o[GR > 1 ? GR - 1 : 1][kRowWaves][kRowTiles<BF, PARTS>][VTile<BF, D>::kAcc][kWave];
  };
  float ml[GR > 1 ? GR - 1 : 1][kRowWaves][kRowTiles<BF, PARTS>][16][2];
  __align__(16) int ok[GR][2][kRowWaves];  // 1: that quarter of the stage is in a physical page
};

template <bool BF, int D, int PARTS, int GR>
__device__ __forceinline__ void attend_rows(const AttendArgs& a, const Block& w, char* smem) {
  constexpr int TT = kTile<BF>;
  constexpr int NZ = scores_per_lane<BF>();
  constexpr int PP = kWeightParts<PARTS>;
  constexpr int QB = PARTS == 1 ? 2 : 4;
  constexpr int RT = kRowTiles<BF, PARTS>;
  constexpr int kAcc = VTile<BF, D>::kAcc;
  typedef Stage<BF, D> St;
  constexpr int ST = St::kTokens;
  constexpr int kChunk = 32;                          // stages between two looks at the table
  constexpr int kLoads = St::kBytes / kRowWaves / 1024;  // of K a wave and stage, and of V
  RowsLds<BF, D, PARTS, GR>& sh = *reinterpret_cast<RowsLds<BF, D, PARTS, GR>*>(smem);

  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wid = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wave = wid % kRowWaves, grp = wid / kRowWaves;
  const int c = lane >> 4, rl = lane & 15;

  const int L = w.pre ? a.prefix : clamp_len(a.seq_lens[w.b], a.max_pages << a.ps_bits);
  const int sinks = a.sinks;
  const int wr = wave * (16 * RT);                      // first row of this wave in the block
  const int wrows = max(min(16 * RT, w.nrows - wr), 0);  // its rows
  int lo[RT], hi[RT], row[RT];
  QFrag<BF, D, PARTS> q[RT];
  Span u = {INT32_MAX, 0, 0, INT32_MAX};
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    lo[t] = hi[t] = row[t] = 0;
    const int r = t * 16 + rl;
    if (r < wrows) row_of(a, w, L, w.r0 + wr + r, &row[t], &lo[t], &hi[t]);
    q[t].load(r < wrows ? static_cast<const char*>(a.q) + (size_t)row[t] * (D * QB) : nullptr, c);
    if (w.pre) {
      const Span s = span_of_prefix(hi[t], r < wrows);
      u = Span{0, max(u.hi, s.hi), 0, min(u.fhi, s.fhi)};
    }
  }
  if (!w.pre && wrows > 0) u = span_of(a, L, w.r0 + wr, wrows);
  // the workgroup's stages: those that any of its rows sees
  Span all = {0, a.prefix, 0, 0};
  if (!w.pre) all = span_of(a, L, w.r0, w.nrows);
  const TileSpan span = tile_span<ST>(all.lo, all.hi, sinks);
  const int per = quotient(span.n + w.splits - 1, w.pre ? a.by_pre_splits : a.by_splits);
  const int b0 = min(w.split * per, span.n), b1 = min(b0 + per, span.n);
  // stages of this group, and steps that every group makes
  const int steps = (b1 - b0 + GR - 1) / GR;
  const int v0 = min(b0 + grp * steps, b1), mine = min(steps, b1 - v0);
  const int npages = (all.hi + (1 << a.ps_bits) - 1) >> a.ps_bits;
  const Views x = views_of<BF, D>(a, w);

  // where this lane's 16 bytes of each direct load come from, past the row
  // that the wave's quarter of the stage starts with
  int from[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int at = i * 1024 + lane * 16;
    const int r = at / St::kRow, slot = at % St::kRow / 16;
    from[i] = r * St::kRow + ((slot ^ St::swizzle(wave * (ST / kRowWaves) + r)) << 4);
  }

  // page of this wave's quarter of each of the next stages, one stage per lane
  int base = v0, ns = 0, pg = -1;
  auto look = [&](int done) {
    base = v0 + done;
    ns = min(kChunk, max(mine - done, 0));
    pg = -1;
    if (lane < ns)
      pg = page_at(a, x.table, npages,
                   (span.tile(base + lane) * ST + wave * (ST / kRowWaves)) >> a.ps_bits);
  };
  auto stage = [&](int j) {
    const int p = __builtin_amdgcn_readlane(pg, j);
    const int t = span.tile(base + j) * ST + wave * (ST / kRowWaves);
    const size_t off =
        (size_t)max(p, 0) * x.k.page_bytes + (size_t)(t & ((1 << a.ps_bits) - 1)) * St::kRow;
    char* dst = sh.st[grp][j & 1][0] + wave * (St::kBytes / kRowWaves);
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      __builtin_amdgcn_global_load_lds(x.k.base + off + from[i], dst + i * 1024, 16, 0, 0);
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      __builtin_amdgcn_global_load_lds(x.v.base + off + from[i], dst + St::kBytes + i * 1024, 16, 0,
                                       0);
    if (lane == 0) sh.ok[grp][j & 1][wave] = p >= 0 ? 1 : 0;
  };
  // Before a stage is used: rows of this wave's quarter that no row of the
  // block sees hold whatever the page holds; as values they are cleared
  // (their weight is 0, but 0 times an infinity is not).
  auto settle = [&](int j) {
    wait_vmcnt<0>();
    const int p = __builtin_amdgcn_readlane(pg, j);
    constexpr int R = ST / kRowWaves;
    const int t = span.tile(base + j) * ST + wave * R;
    if (p >= 0 && t + R <= all.hi && (t >= all.lo || t + R <= sinks)) return;
    constexpr int kPer = kWave / R;  // lanes a row
    const int r = lane / kPer;
    if ((p >= 0) & sees(t + r, all.lo, all.hi, sinks)) return;
    char* dst = sh.st[grp][j & 1][1] + (wave * R + r) * St::kRow + lane % kPer * 16;
#pragma unroll
    for (int i = 0; i < St::kRow; i += kPer * 16)
      *reinterpret_cast<u32x4*>(dst + i) = u32x4{0, 0, 0, 0};
  };
  f32x4 acc[RT][kAcc];
  float m[RT], l[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
#pragma unroll
    for (int n = 0; n < kAcc; ++n) acc[t][n] = f32x4{0, 0, 0, 0};
    m[t] = kLowest<PARTS>;
    l[t] = 0.0f;
  }

  for (int done = 0; done < steps; done += kChunk) {
    const int nb = min(kChunk, steps - done);
    look(done);
    if (ns > 0) {
      stage(0);
      settle(0);
    }
    __syncthreads();
    uint64_t put_off = 0;  // two tiles a stage
    for (int j = 0; j < nb; ++j) {
      if (j + 1 < ns) stage(j + 1);
      const int ts = j < ns ? span.tile(base + j) * ST : 0;
      const lds_at kst = lds_addr(sh.st[grp][j & 1][0]), vst = kst + St::kBytes;
      // a stage that some of this wave's rows sees
      if (j < ns && ts < u.hi && (ts + ST > u.lo || ts < sinks)) {
        const int4 ok = *reinterpret_cast<const int4*>(sh.ok[grp][j & 1]);
        const bool full = __builtin_amdgcn_readfirstlane(ok.x & ok.y & ok.z & ok.w) &&
                          ts + ST <= u.fhi && (ts >= u.flo || ts + ST <= sinks);
        KTile<BF, D> kt;
        kt.read(kst, 0, lane);
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
          float p[RT][NZ];
#pragma unroll
          for (int t = 0; t < RT; ++t) kt.template scores<PARTS>(q[t], p[t]);
          __builtin_amdgcn_s_setprio(0);
          // the values, and the next tile's keys, are on their way while the
          // weights are formed
          if (sub == 0) kt.read(kst, 1, lane);
          StageV<BF, D> v;
#pragma unroll
          for (int n = 0; n < kAcc; ++n) v.read(vst, sub, lane, n);
          bool later = false;
          if (!full) {
            const int lowq = sub ? ok.z : ok.x, highq = sub ? ok.w : ok.y;
            const bool page_ok = (c < 2 ? lowq : highq) != 0;
#pragma unroll
            for (int i = 0; i < NZ; ++i) {
              const int tt = ts + sub * TT + tile_token<BF>(c, i);
#pragma unroll
              for (int t = 0; t < RT; ++t)
                p[t][i] = page_ok & sees(tt, lo[t], hi[t], sinks) ? p[t][i] : -INFINITY;
            }
            later = __any(stage_nonfinite<BF, D>(vst, sub, lane));
            if (later) put_off |= 1ull << (2 * j + sub);
          }
          float tmax[RT];
          bool rise = false;
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            tmax[t] = p[t][0];
#pragma unroll
            for (int i = 1; i < NZ; ++i) tmax[t] = fmaxf(tmax[t], p[t][i]);
            rise |= tmax[t] > m[t] + kSlack;
          }
          if (__any(rise)) {
#pragma unroll
            for (int t = 0; t < RT; ++t) raise(tmax[t], m[t], l[t], acc[t]);
          }
          PFrag<BF, PP> pf[RT];
#pragma unroll
          for (int t = 0; t < RT; ++t) {
#pragma unroll
            for (int i = 0; i < NZ; ++i) {
              p[t][i] = weight<PARTS>(p[t][i], m[t]);
              l[t] += p[t][i];
            }
            pf[t].set(p[t]);
          }
          // matrix instructions before the other wave's exponentials: the two
          // waves of a SIMD, in step after each barrier, then alternate
          // (2 x 512 queries, window of 8192: 224 -> 211 us)
          __builtin_amdgcn_s_setprio(1);
          if (!__builtin_expect(later, 0)) {
#pragma unroll
            for (int n = 0; n < kAcc; ++n) v.template add<PP, RT>(pf, acc, n);
          }
        }
      }
      if (j + 1 < ns) settle(j + 1);
      __syncthreads();
    }
    while (put_off) {
      const int j = __builtin_ctzll(put_off);
      put_off &= put_off - 1;
      const int t0 = span.tile(base + j / 2) * ST + (j & 1) * TT;
      TilePages pp;
      pp.p0 = pp.p1 = page_at(a, x.table, npages, t0 >> a.ps_bits);
      if (BF && a.ps_bits == 4) pp.p1 = page_at(a, x.table, npages, (t0 >> a.ps_bits) + 1);
#pragma unroll
      for (int t = 0; t < RT; ++t)
        late_tile<BF, D, PARTS, PP, true>(x, pp, t0, lane, q[t], lo[t], hi[t], sinks, m[t], acc[t]);
    }
  }

  // join the groups: the others leave their parts in LDS, lane by lane (every
  // stage has been read: the loop ends with a barrier)
#pragma unroll
  for (int t = 0; t < RT; ++t) l[t] = group_sum(l[t]);
  if (GR > 1 && grp > 0) {
#pragma unroll
    for (int t = 0; t < RT; ++t) {
#pragma unroll
      for (int n = 0; n < kAcc; ++n) sh.o[grp - 1][wave][t][n][lane] = acc[t][n];
      if (c == 0) {
        sh.ml[grp - 1][wave][t][rl][0] = m[t];
        sh.ml[grp - 1][wave][t][rl][1] = l[t];
      }
    }
  }
  if (GR > 1) __syncthreads();
  if (grp > 0) return;
#pragma unroll
  for (int t = 0; t < RT; ++t) {
#pragma unroll
    for (int e = 0; e < GR - 1; ++e) {
      const float me = sh.ml[e][wave][t][rl][0], le = sh.ml[e][wave][t][rl][1];
      const float mn = le == 0.0f ? m[t] : l[t] == 0.0f ? me : fmaxf(m[t], me);
      const float f = l[t] == 0.0f ? 0.0f : __builtin_amdgcn_exp2f((m[t] - mn) * kLog2e);
      const float fe = le == 0.0f ? 0.0f : __builtin_amdgcn_exp2f((me - mn) * kLog2e);
      l[t] = f * l[t] + fe * le;
#pragma unroll
      for (int n = 0; n < kAcc; ++n) acc[t][n] = f * acc[t][n] + fe * sh.o[e][wave][t][n][lane];
      m[t] = mn;
    }
  }
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const float ls = l[t];
    if (t * 16 + rl >= wrows) continue;
    if (a.slots > 1) {
      const size_t part = (size_t)row[t] * a.slots + w.slot;
      if (c == 0) {
        a.part_ml[2 * part] = m[t];
        a.part_ml[2 * part + 1] = ls;
      }
#pragma unroll
      for (int n = 0; n < kAcc; ++n)
        *reinterpret_cast<f32x4*>(a.part_o + part * D + StageV<BF, D>::coord(c, n)) = acc[t][n];
    } else {
      const float inv = inverse(ls);
#pragma unroll
      for (int n = 0; n < kAcc; ++n)
        store_out<PARTS>(a.out, (size_t)row[t] * D + StageV<BF, D>::coord(c, n), acc[t][n] * inv);
      if (c == 0 && a.lse) a.lse[row[t]] = log_sum(m[t], ls);
    }
  }
}

// What a launch runs: the few-rows form alone; the many-rows form alone (a
// window, two groups a workgroup); or the many-rows form over a shared prefix
// and the few-rows form over the rest. The last starts with the rest: its
// short workgroups, bound by memory, end one by one, and those of the prefix,
// which start in their places, are then out of step with each other (128
// sequences of 32K + 500 tokens: 139 us, the prefix first 149 to 168; dealt out
// among each other it was a sixth slower too: a CU is filled before the next,
// so pairs of one kind meet).
enum { kFewRows = 0, kManyRows = 1, kBesides = 2, kFewAlone = 3 };
constexpr int att_waves(int mode) {
  return mode == kManyRows || mode == kFewAlone ? 2 * kRowWaves : kRowWaves;
}

template <bool BF, int D, int PARTS, int MODE>
__global__ __launch_bounds__(att_waves(MODE) * kWave, 2) void attend_kernel(AttendArgs a) {
  extern __shared__ __align__(1024) char smem[];
  const Block w = block_of(a, blockIdx.x);
  if constexpr (MODE == kManyRows) {
    attend_rows<BF, D, PARTS, 2>(a, w, smem);
  } else if constexpr (MODE == kBesides) {
    if (w.pre)
      attend_rows<BF, D, PARTS, 1>(a, w, smem);
    else
      attend_tokens<BF, D, PARTS, kRowWaves>(a, w, smem);
  } else {
    attend_tokens<BF, D, PARTS, att_waves(MODE)>(a, w, smem);
  }
}

// Joins the parts of each row. D/4 threads hold 4 coordinates each of a row's
// parts s, s + SG, ...; the SG groups are joined through LDS. Bound by reading
// the parts (4096 rows of 17 parts, 128 dims: 36 MB in 8.2 us, 4.4 TB/s), and by
// latency where they are few (3.0 us).
constexpr int kJoinThreads = 256;

template <int D, int PARTS, int SG>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(const float* __restrict__ part_o,
                                                            const float* __restrict__ part_ml,
                                                            int slots, int rows,
                                                            void* __restrict__ out,
                                                            float* __restrict__ lse) {
  constexpr int TPR = D / 4;
  constexpr int kRows = kJoinThreads / (TPR * SG);
  constexpr int U = 4;  // parts of a thread in flight
  __shared__ f32x4 so[kRows][SG][TPR];
  __shared__ float sml[kRows][SG][2];
  const int tid = threadIdx.x, d4 = tid % TPR, sg = tid / TPR % SG, rr = tid / (TPR * SG);
  const int r = blockIdx.x * kRows + rr;
  float M = -FLT_MAX, l = 0.0f;
  f32x4 o = {0, 0, 0, 0};
  if (r < rows) {
    const f32x2* ml = reinterpret_cast<const f32x2*>(part_ml) + (size_t)r * slots;
    const f32x4* po = reinterpret_cast<const f32x4*>(part_o) + (size_t)r * slots * TPR + d4;
    for (int s0 = sg; s0 < slots; s0 += U * SG) {
      f32x2 x[U];
      f32x4 y[U];
#pragma unroll
      for (int e = 0; e < U; ++e) {
        const int s = min(s0 + e * SG, slots - 1);
        x[e] = ml[s];
        y[e] = po[(size_t)s * TPR];
      }
      float mn = M;
#pragma unroll
      for (int e = 0; e < U; ++e) {
        if (s0 + e * SG >= slots) x[e] = f32x2{-FLT_MAX, 0.0f};
        if (!(x[e][1] == 0.0f)) mn = fmaxf(mn, x[e][0]);
      }
      const float f = __builtin_amdgcn_exp2f((M - mn) * kLog2e);
      l *= f;
      o *= f;
      M = mn;
#pragma unroll
      for (int e = 0; e < U; ++e) {
        if (x[e][1] == 0.0f) continue;
        const float g = __builtin_amdgcn_exp2f((x[e][0] - M) * kLog2e);
        l += g * x[e][1];
        o += g * y[e];
      }
    }
  }
  if constexpr (SG > 1) {
    so[rr][sg][d4] = o;
    if (d4 == 0) {
      sml[rr][sg][0] = M;
      sml[rr][sg][1] = l;
    }
    __syncthreads();
    if (sg != 0) return;
    float mn = -FLT_MAX;
#pragma unroll
    for (int e = 0; e < SG; ++e)
      if (!(sml[rr][e][1] == 0.0f)) mn = fmaxf(mn, sml[rr][e][0]);
    l = 0.0f;
    o = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < SG; ++e) {
      const float le = sml[rr][e][1];
      if (le == 0.0f) continue;
      const float g = __builtin_amdgcn_exp2f((sml[rr][e][0] - mn) * kLog2e);
      l += g * le;
      o += g * so[rr][e][d4];
    }
    M = mn;
  }
  if (r >= rows) return;
  store_out<PARTS>(out, (size_t)r * D + d4 * 4, o * inverse(l));
  if (d4 == 0 && lse) lse[r] = log_sum(M, l);
}

// Raises a kernel's LDS limit on the current device, once (a repeat by two
// threads at the same time does no harm).
hipError_t raise_lds(const void* kernel, size_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (hipError_t e = hipGetDevice(&dev)) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load() & bit) return hipSuccess;
  if (hipError_t e =
          hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes))
    return e;
  done.fetch_or(bit);
  return hipSuccess;
}

template <bool BF, int D, int PARTS, int MODE>
hipError_t launch_mode(const AttendArgs& a, long long items, hipStream_t st) {
  constexpr size_t few = sizeof(TokensLds<D, MODE == kFewAlone ? att_waves(MODE) : kRowWaves>);
  constexpr size_t many = sizeof(RowsLds<BF, D, PARTS, MODE == kManyRows ? 2 : 1>);
  constexpr size_t lds = MODE == kFewRows || MODE == kFewAlone || few > many ? few : many;
  auto* f = attend_kernel<BF, D, PARTS, MODE>;
  if (lds > 64 * 1024) {
    static std::atomic<uint64_t> raised{0};  // devices whose kernel has the limit
    if (hipError_t e = raise_lds(reinterpret_cast<const void*>(f), lds, raised)) return e;
  }
  hipLaunchKernelGGL(f, dim3((unsigned)items), dim3(att_waves(MODE) * kWave), lds, st, a);
  return hipGetLastError();
}

template <bool BF, int D, int PARTS>
hipError_t launch(const AttendArgs& a, const AttendPlan& p, hipStream_t st) {
  if (p.own_rows) return launch_mode<BF, D, PARTS, kManyRows>(a, p.items, st);
  if (p.pre_rows) return launch_mode<BF, D, PARTS, kBesides>(a, p.items, st);
  if (p.alone) return launch_mode<BF, D, PARTS, kFewAlone>(a, p.items, st);
  return launch_mode<BF, D, PARTS, kFewRows>(a, p.items, st);
}

template <int D, int PARTS>
hipError_t join(const AttendPlan& p, const float* o, const float* ml, void* out, float* lse,
                hipStream_t st) {
  const int rows = (int)p.rows;
  constexpr int TPR = D / 4, kMost = kJoinThreads / TPR;
  const auto grid = [&](int sg) {
    return dim3((unsigned)((rows * (long long)sg * TPR + kJoinThreads - 1) / kJoinThreads));
  };
  // up to 8 parts: two groups of 4 in flight; more: the whole workgroup on a row
  if (p.slots <= 8)
    hipLaunchKernelGGL((join_kernel<D, PARTS, 2>), grid(2), dim3(kJoinThreads), 0, st, o, ml,
                       p.slots, rows, out, lse);
  else
    hipLaunchKernelGGL((join_kernel<D, PARTS, kMost>), grid(kMost), dim3(kJoinThreads), 0, st, o,
                       ml, p.slots, rows, out, lse);
  return hipGetLastError();
}

}  // namespace

// Parts of a row block's tokens: as many as make `want` workgroups in all (a
// full CU each), of at least `least` tiles. One part more where the CUs then
// share the blocks out more evenly by a fifth (300 blocks: 3 halves instead of
// 2 wholes on the fullest CU). Never just over `want` (56 blocks of the float32
// window in 10 parts, 560 workgroups: 18.6 us, in 9: 15.9).
static int splits_for(long long blocks, long long tiles, long long want, int least) {
  const auto share = [&](long long s) { return (double)((blocks * s + kNumCUs - 1) / kNumCUs) / s; };
  long long s = want / blocks;
  if (s < 1) s = 1;
  if (share(s + 1) < 0.8 * share(s)) ++s;
  const long long most = (tiles + least - 1) / least;
  if (s > most) s = most;
  if (s > kAttMaxSplits) s = kAttMaxSplits;
  return s < 1 ? 1 : (int)s;
}

AttendPlan plan_attend(const LaunchShape& s, bool q_bf16, int n, int window, int sinks,
                       int prefix_pages) {
  AttendPlan p;
  const int TT = s.bf16 ? kTile<true> : kTile<false>;
  const long long total = (long long)s.max_pages * s.page_size;
  const long long prefix = (long long)prefix_pages * s.page_size;
  const int many = kRowWaves * 16 * (s.bf16 && q_bf16 ? kRowTiles<true, 1> : kRowTiles<true, 3>);
  p.rows = (long long)s.batch * n * s.num_q_heads;
  const int own = n * s.group, pre = s.batch * s.group;
  // tiles that a block of `rows` of the sequences' own rows can see
  const auto seen_by = [&](int rows) {
    const long long span = (long long)window + rows / s.group + 1;
    const long long seen = total - prefix < span ? total - prefix : span;
    return (seen + TT - 1) / TT + 1 + (sinks + TT - 1) / TT;
  };
  // (a window's: at most 8 rows beside a prefix)
  p.own_rows = own >= kAttManyRows && (long long)s.batch * s.num_kv_heads * ((own + 15) / 16) *
                                              seen_by(16) > kAttFewTiles;
  p.pre_rows = prefix_pages > 0 && pre >= kAttManyRows &&
               s.num_kv_heads * ((pre + 15) / 16) * (prefix / TT) > kAttFewPrefixTiles;
  // eight waves a CU, four or eight a workgroup
  const int waves = att_waves(p.own_rows ? kManyRows : kFewRows);
  const long long want = (long long)8 / waves * kNumCUs;
  p.row_block = p.own_rows ? many : 16;
  p.row_blocks = (own + p.row_block - 1) / p.row_block;
  const long long tiles = seen_by(p.row_block);
  const long long blocks = (long long)s.batch * s.num_kv_heads * p.row_blocks;
  // a workgroup's tokens: at least one tile a wave, or two stages a group
  const int few = waves, many_tiles = waves;
  if (prefix_pages > 0) {
    p.pre_block = p.pre_rows ? many : 16;
    const long long pre_blocks =
        (long long)s.num_kv_heads * ((pre + p.pre_block - 1) / p.pre_block);
    p.pre_splits = splits_for(pre_blocks, (prefix + TT - 1) / TT, want,
                              p.pre_rows ? many_tiles : few);
    p.items = pre_blocks * p.pre_splits;
  }
  p.splits = total > prefix ? splits_for(blocks, tiles, want, p.own_rows ? many_tiles : few) : 0;
  // few tokens (K and V of a block in one or two loads of eight waves): one
  // part, of a workgroup of eight waves, and no join (window of 64 at 128 bf16
  // dims 8.1 -> 6.2 us, of 256 8.6 -> 8.0; of 512 8.9 against 10.0)
  p.alone = !prefix_pages && !p.own_rows && p.splits > 1 &&
            tiles * (2 * TT * s.head_dim * (s.bf16 ? 2 : 4)) <= kAloneBytes;
  if (p.alone) p.splits = 1;
  p.threads = kWave * att_waves(p.own_rows  ? kManyRows
                                : p.pre_rows ? kBesides
                                : p.alone    ? kFewAlone
                                             : kFewRows);
  p.own_items = blocks * p.splits;
  p.items += p.own_items;
  p.slots = p.pre_splits + p.splits;
  if (p.slots > 1) {
    const size_t parts = (size_t)p.rows * p.slots;
    p.ml_off = (parts * s.head_dim * 4 + 255) & ~(size_t)255;
    p.ws_bytes = p.ml_off + ((parts * 8 + 255) & ~(size_t)255);
  }
  return p;
}

hipError_t launch_attend(const LaunchShape& s, const AttendPlan& p, const void* q, bool q_bf16,
                         int n, const void* k_pool, const void* v_pool,
                         const int32_t* prefix_table, int prefix_pages,
                         const int32_t* block_table, const int32_t* seq_lens, int window,
                         int sinks, void* out, float* lse, void* ws, hipStream_t st) {
  AttendArgs a;
  a.q = q;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.prefix_table = prefix_table;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.out = out;
  a.lse = lse;
  a.part_o = static_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float*>(static_cast<char*>(ws) + p.ml_off);
  a.batch = s.batch;
  a.H = s.num_q_heads;
  a.Hkv = s.num_kv_heads;
  a.g_bits = __builtin_ctz(s.group);
  a.n = n;
  a.ps_bits = __builtin_ctz(s.page_size);
  a.max_pages = s.max_pages;
  a.num_phys = s.num_phys;
  a.window = window;
  a.sinks = sinks;
  a.prefix = prefix_pages * s.page_size;
  a.pre_block = p.pre_block;
  a.pre_splits = p.pre_splits;
  a.row_block = p.row_block;
  a.row_blocks = p.row_blocks;
  a.splits = p.splits;
  a.by_hkv = divisor(s.num_kv_heads);
  a.by_pre_splits = divisor(p.pre_splits);
  a.by_pre_blocks = divisor(
      p.pre_block ? (s.batch * s.group + p.pre_block - 1) / p.pre_block : 1);
  a.by_blocks = divisor(p.row_blocks);
  a.by_splits = divisor(p.splits);
  a.slots = p.slots;
  a.own_items = (int)p.own_items;
  if (!s.bf16) return s.head_dim == 64 ? launch<false, 64, 3>(a, p, st)
                                       : launch<false, 128, 3>(a, p, st);
  if (q_bf16) return s.head_dim == 64 ? launch<true, 64, 1>(a, p, st)
                                      : launch<true, 128, 1>(a, p, st);
  return s.head_dim == 64 ? launch<true, 64, 3>(a, p, st)
                          : launch<true, 128, 3>(a, p, st);
}

hipError_t launch_join(const LaunchShape& s, const AttendPlan& p, bool q_bf16, void* out,
                       float* lse, void* ws, hipStream_t st) {
  const float* o = static_cast<const float*>(ws);
  const float* ml = reinterpret_cast<const float*>(static_cast<const char*>(ws) + p.ml_off);
  if (s.head_dim == 64)
    return q_bf16 ? join<64, 1>(p, o, ml, out, lse, st) : join<64, 3>(p, o, ml, out, lse, st);
  return q_bf16 ? join<128, 1>(p, o, ml, out, lse, st) : join<128, 3>(p, o, ml, out, lse, st);
}

}  // namespace ekv
