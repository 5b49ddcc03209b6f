// alpha-entmax attention of a ragged batch of new tokens over the paged cache.
//
//   x_t = (alpha - 1) z_t, z_t = q . k_t;  sum_t [x_t - tau]_+^m = 1,
//   out = sum_t p_t v_t / sum_t p_t,  p_t = [x_t - tau]_+^m,  m = 1/(alpha-1)
//
// over the tokens up to the query's own position. Everything is computed from
// y_t = x_t - max x <= 0, whose threshold lies in [-1, 0).
//
// tau grows with every token added, so the threshold of the tokens seen so far
// (at first max x - 1) bounds the support from below: one pass over the scores
// on the matrix cores keeps, per row, the few tokens above it, and V is read for
// the support alone. Three kernels:
//   list_kernel    scores, and each row's list of tokens above the running bound
//   finish_kernel  a row's lists (one a part of its tokens) joined, tau solved,
//                  the support's V rows gathered
//   dense_kernel   rows whose support does not fit a list, by passes over all of
//                  their scores; the other workgroups leave at once
#include "softmax_impl.hpp"

namespace ekv {
namespace {

constexpr int kChunkWaves = 4;

struct __align__(16) Part {
  int32_t n;        // entries, or why there are none
  float mx, slack;  // the largest score; how far two scores may be off together
  float thr;        // a bound of the row's threshold from below, but for `slack`
};

struct ChunkArgs {
  const void* q;
  const void* k_pool;
  const void* v_pool;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* starts;
  void* out;
  float* tau;        // nullable
  int32_t* support;  // nullable
  int N, B, H, Hkv, g_bits, ps_bits, max_pages, num_phys;
  float am1, m;  // alpha - 1 and 1 / (alpha - 1)
  float rooted;  // 2 - alpha = 1 - 1/m
  float window;  // of a score below the row's maximum that may have a weight
  int whole;     // m if it is 1, 2, 3 or 4, else 0 (alpha = 4/3 of float32: 2.9999996)
  int tok_bits;  // 2^tok_bits tokens a list block
  int splits, few_splits;  // parts of a row's tokens; of blocks of at most 16 rows
  int cap;                 // entries of a list
  size_t few_parts;        // the first of the few-row blocks' parts
  unsigned few_items;      // their workgroups
  // workspace: per (row, part) the list, its length and how far its scores may
  // be off together, and per 16 rows a bit for each that needs the dense kernel
  uint64_t* lists;
  Part* parts;
  int32_t* dense;
};

// Entries of a list by alpha: support sizes grow as alpha falls (scores of
// spread 2.5, 32K tokens: 8 tokens on average and 20 at most at alpha 1.5, 67 and
// 140 at 1.25, 200 rows each), and with them the hits, so that a short list is
// pruned more often; a long one is more workspace. Measured, 4096 of 32K tokens at
// alpha 1.25, list and finish kernel: 256 entries 2.88 + 0.55 ms, 384 2.40 + 0.66,
// 512 2.32 + 0.67.
constexpr int cap_of(float alpha) { return alpha >= 1.5f ? 128 : 384; }
// Lengths that say why there is no list.
constexpr int kLong = -1;    // the support does not fit
constexpr int kNoNumber = -2;  // a score is NaN or +inf

// A block of rows: tokens i0 .. of sequence b (rows tok0 .. of q) and the heads
// of KV head g. rows = 0: none.
struct Rows {
  int b, g, tok0, i0, rows, n, L;
};

// Blocks of TB tokens are numbered so that sequence b's begin at starts[b] / TB
// + b: never fewer than it has, floor(starts[b+1] / TB) - floor(starts[b] / TB)
// + 1 >= ceil(n / TB), so that a workgroup finds its block by a search alone.
// 64 probes a step: two steps up to 4096 sequences.
__device__ __forceinline__ Rows find_rows(const ChunkArgs& a, int tok_bits, int id, int g,
                                          int lane) {
  const auto start = [&](int b) { return clamp_len(a.starts[b], a.N); };
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int step = (hi - lo + kWave - 1) / kWave, at = lo + lane * step;
    const bool below = lane == 0 || (at < hi && (start(at) >> tok_bits) + at <= id);
    lo += (63 - __builtin_clzll(__ballot(below))) * step;
    hi = min(hi, lo + step);
  }
  Rows r;
  const int s = start(lo), i0 = (id - (s >> tok_bits) - lo) << tok_bits;
  r.b = lo;
  r.g = g;
  r.n = start(lo + 1) - s;
  r.i0 = i0;
  r.tok0 = s + i0;
  r.rows = i0 >= 0 && i0 < r.n ? min(1 << tok_bits, r.n - i0) << a.g_bits : 0;
  r.L = clamp_len(a.seq_lens[lo], a.max_pages << a.ps_bits);
  return r;
}

// Row r of a block: tokens below `hi` are seen; its index among all rows.
__device__ __forceinline__ int seen(const ChunkArgs& a, const Rows& w, int r) {
  return max(w.L - w.n + w.i0 + (r >> a.g_bits) + 1, 0);
}
__device__ __forceinline__ size_t row_at(const ChunkArgs& a, const Rows& w, int r) {
  const int i = r >> a.g_bits;
  return (size_t)(w.tok0 + i) * a.H + (w.g << a.g_bits) + (r - (i << a.g_bits));
}

// The block of a sequence's last tokens (of several, the only one that may have
// few rows).
__device__ __forceinline__ Rows last_rows(const ChunkArgs& a, int b, int g) {
  Rows r;
  const int s = clamp_len(a.starts[b], a.N);
  r.b = b;
  r.g = g;
  r.n = clamp_len(a.starts[b + 1], a.N) - s;
  r.i0 = max(r.n - 1, 0) & ~((1 << a.tok_bits) - 1);
  r.tok0 = s + r.i0;
  r.rows = max(r.n - r.i0, 0) << a.g_bits;
  r.L = clamp_len(a.seq_lens[b], a.max_pages << a.ps_bits);
  return r;
}

// The first of the parts of row r of a list block, and how many. The parts of a
// block of few rows are more, for single tokens over long caches, and lie by
// sequence.
struct Parts {
  size_t first;
  int count;
};
__device__ __forceinline__ Parts parts_of(const ChunkArgs& a, const Rows& w, int r) {
  if (w.rows <= 16)
    return Parts{a.few_parts + (((size_t)w.b * a.Hkv + w.g) * 16 + r) * a.few_splits,
                 a.few_splits};
  return Parts{row_at(a, w, r) * a.splits, a.splits};
}

__device__ __forceinline__ int page_at(const ChunkArgs& a, const int32_t* table, int npages,
                                       int j) {
  const int p = j < npages ? table[j] : -1;
  return p < a.num_phys ? p : -1;
}

// u^m and u^(m-1) of u >= 0 (u = 0: 0, whatever m)
__device__ __forceinline__ void powers(const ChunkArgs& a, float u, float& pm, float& pm1) {
  if (a.whole == 2) {
    pm1 = u;
    pm = u * u;
  } else if (a.whole) {
    pm1 = a.whole == 1 ? (u > 0.0f ? 1.0f : 0.0f) : a.whole == 3 ? u * u : u * u * u;
    pm = pm1 * u;
  } else {
    pm1 = u > 0.0f ? __builtin_amdgcn_exp2f((a.m - 1.0f) * __builtin_amdgcn_logf(u)) : 0.0f;
    pm = pm1 * u;
  }
}

// A token's weight in the output, up to a factor that all tokens of its row share:
// u^m of u = y - t > 0 where m is whole, else (u / s)^m = (1 + y / s)^m, s = -t.
// Near alpha = 1, u is nearly 1, and u^m would be off by m times u's rounding; the
// logarithm of 1 + y / s is taken with what the sum's rounding lost put back.
__device__ __forceinline__ float weight_of(const ChunkArgs& a, float y, float t, float u) {
  if (a.whole) {
    float pm, pm1;
    powers(a, u, pm, pm1);
    return pm;
  }
  const float rs = __builtin_amdgcn_rcpf(-t), x = y * rs;
  const float w = 1.0f + x, e = w - 1.0f;
  const float near = e != 0.0f ? __builtin_amdgcn_logf(w) * (x * __builtin_amdgcn_rcpf(e))
                               : x * kLog2e;
  const float lg = x > -0.5f ? near : __builtin_amdgcn_logf(u * rs);
  return u > 0.0f ? __builtin_amdgcn_exp2f(a.m * lg) : 0.0f;
}

// s^(1 - 1/m), of m >= 1
__device__ __forceinline__ float root_of(const ChunkArgs& a, float s) {
  return a.whole == 1   ? 1.0f
         : a.whole == 2 ? __builtin_amdgcn_sqrtf(s)
                        : __builtin_amdgcn_exp2f(a.rooted * __builtin_amdgcn_logf(s));
}

// The threshold of one row, by steps from tau = -1 (max x = 0), where the sum
// s = sum u^m is at least 1. For m >= 1 Newton's steps are those of the convex
// norm (sum u^m)^(1/m) = 1, nearly straight where the support stays the same:
// from below, without passing the root. For m < 1 (alpha > 2) the sum is not
// convex: its own Newton steps, and every other step halves the bracket.
struct Threshold {
  float t = -1.0f, lo = -1.0f, hi = 0.0f;
  bool done = false;
  // s1 = sum u^(m-1) at t
  __device__ __forceinline__ void step(const ChunkArgs& a, float s, float s1, int i) {
    if (done) return;
    const bool over = s >= 1.0f;
    if (over) lo = t; else hi = t;
    const float eps = 6.0e-8f * fmaxf(-t, 1e-3f);
    float next;
    if (a.m >= 1.0f) {
      const float d = (s - root_of(a, s)) * __builtin_amdgcn_rcpf(s1);
      next = t + d;
      done = !(d > eps);  // from below; at or past the root only by rounding
      if (!(next < 0.0f)) next = 0.5f * (t + hi);
    } else {
      next = t + (s - 1.0f) / (a.m * s1);
      if ((i & 1) || !(next > lo && next < hi)) next = 0.5f * (lo + hi);
      done = hi - lo <= eps || next == t;
    }
    t = next;
  }
};
constexpr int kSteps = 64;  // of m < 1; others take under ten

template <int D>
struct DenseLds {
  float o[kChunkWaves][16][D + 4];
  float s[2][kChunkWaves][16][2];
};

// Those of a block's 16 rows at most that `which` has a bit for, by passes over
// all of their scores: the maximum, one pass a threshold step, and the weights'
// product with V. The workgroup's waves share the rows and take turns at the
// tiles. The other rows keep what their lists gave, in other roundings (with
// bf16 queries the weights of these are off by 2^-17). Right, but slow: K is read
// once a step for 16 rows, and a row's tokens are never split (weights on all
// tokens, alpha 1.5, 32/8 heads of 128 dims: a prompt of 2048 4.2 ms, 512 of 32K 15.1,
// one token over 32K 5.0).
template <bool BF, int D, int PARTS>
__device__ __forceinline__ void dense_rows(const ChunkArgs& a, const Rows& w, unsigned which,
                                           DenseLds<D>& sh) {
  constexpr int TT = kTile<BF>;
  constexpr int NZ = scores_per_lane<BF>();
  constexpr int PP = PARTS == 1 ? 2 : 3;
  constexpr int QB = PARTS == 1 ? 2 : 4;
  constexpr int kAcc = VTile<BF, D>::kAcc;
  constexpr int kElem = BF ? 2 : 4;
  constexpr int NW = kChunkWaves;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = lane >> 4, rl = lane & 15;
  const bool mine = which >> rl & 1;
  const int hi = mine ? seen(a, w, rl) : 0;
  const int top = seen(a, w, 31 - __builtin_clz(which));  // the last row sees the most
  const int tiles = (top + TT - 1) / TT, npages = (top + (1 << a.ps_bits) - 1) >> a.ps_bits;
  const size_t head_off = ((size_t)w.g << a.ps_bits) * (D * kElem);
  const size_t page_bytes = ((size_t)a.Hkv << a.ps_bits) * (D * kElem);
  const KvView kv{static_cast<const char*>(a.k_pool) + head_off, page_bytes, 1 << a.ps_bits};
  const KvView vv{static_cast<const char*>(a.v_pool) + head_off, page_bytes, 1 << a.ps_bits};
  const int32_t* table = a.block_table + (size_t)w.b * a.max_pages;

  QFrag<BF, D, PARTS> q;
  q.load(mine ? static_cast<const char*>(a.q) + row_at(a, w, rl) * (D * QB) : nullptr, c);

  // f(tile's first token, its pages, this lane's scores; -inf where hidden)
  auto each_tile = [&](auto f) {
    for (int v = wave; v < tiles; v += NW) {
      const int t0 = v * TT, j = t0 >> a.ps_bits;
      TilePages pg;
      pg.p0 = pg.p1 = page_at(a, table, npages, j);
      if (BF && a.ps_bits == 4) pg.p1 = page_at(a, table, npages, j + 1);
      KTile<BF, D> kt;
      kt.load(kv, pg, t0, lane);
      float z[NZ];
      kt.template scores<PARTS>(q, z);
      const bool page_ok = (!BF || c < 2 ? pg.p0 : pg.p1) >= 0;
#pragma unroll
      for (int i = 0; i < NZ; ++i)
        z[i] = (page_ok & (t0 + tile_token<BF>(c, i) < hi)) ? z[i] : -INFINITY;
      f(t0, pg, z);
    }
  };

  // the maximum; NaN stays
  float mx = -INFINITY;
  each_tile([&](int, const TilePages&, float (&z)[NZ]) {
#pragma unroll
    for (int i = 0; i < NZ; ++i) mx = !(z[i] <= mx) && mx == mx ? z[i] : mx;
  });
#pragma unroll
  for (int s = 16; s < 64; s <<= 1) {
    const float x = __shfl_xor(mx, s, kWave);
    mx = !(x <= mx) && mx == mx ? x : mx;
  }
  if (c == 0) sh.s[1][wave][rl][0] = mx;
  __syncthreads();
#pragma unroll
  for (int v = 0; v < NW; ++v) {
    const float x = sh.s[1][v][rl][0];
    mx = !(x <= mx) && mx == mx ? x : mx;
  }
  // rows that see nothing, or a score that is no number: no threshold to find
  const bool finite = mx > -INFINITY && mx < INFINITY;
  const float ref = finite ? mx : 0.0f;

  Threshold th;
  th.done = !finite;
  for (int i = 0; i < kSteps; ++i) {
    float s = 0.0f, s1 = 0.0f;
    each_tile([&](int, const TilePages&, float (&z)[NZ]) {
      float b = 0.0f, b1 = 0.0f;
#pragma unroll
      for (int e = 0; e < NZ; ++e) {
        float pm, pm1;
        powers(a, fmaxf((z[e] - ref) * a.am1 - th.t, 0.0f), pm, pm1);
        b += pm;
        b1 += pm1;
      }
      s += b;
      s1 += b1;
    });
    s = group_sum(s);
    s1 = group_sum(s1);
    const int buf = i & 1;
    if (c == 0) {
      sh.s[buf][wave][rl][0] = s;
      sh.s[buf][wave][rl][1] = s1;
    }
    __syncthreads();
    s = s1 = 0.0f;
#pragma unroll
    for (int v = 0; v < NW; ++v) {
      s += sh.s[buf][v][rl][0];
      s1 += sh.s[buf][v][rl][1];
    }
    th.step(a, s, s1, i);
    if (__all(th.done)) break;  // the same in every wave
  }

  f32x4 acc[kAcc];
#pragma unroll
  for (int n = 0; n < kAcc; ++n) acc[n] = f32x4{0, 0, 0, 0};
  float l = 0.0f;
  int live = 0;
  each_tile([&](int t0, const TilePages& pg, float (&z)[NZ]) {
    float p[NZ];
    unsigned see = 0;
    float b = 0.0f;
#pragma unroll
    for (int i = 0; i < NZ; ++i) {
      const float y = (z[i] - ref) * a.am1;
      const float u = finite ? fmaxf(y - th.t, 0.0f) : 0.0f;
      p[i] = weight_of(a, y, th.t, u);
      b += p[i];
      see |= (u > 0.0f ? 1u : 0u) << i;  // (a high power may be below float32)
    }
    l += b;
    live += __popc(see);
    if (!__any(see != 0)) return;
    VTile<BF, D> vt;
    vt.load(vv, pg, t0, lane);
    PFrag<BF, PP> pf;
    pf.set(p);
    if (!__any(vt.any_nonfinite())) {
#pragma unroll
      for (int n = 0; n < kAcc; ++n) acc[n] = vt.template mul<PP>(n, pf, acc[n]);
      return;
    }
    // a value that is no number must not meet the zero weight of a row: one
    // row at a time, on the tokens of its support
#pragma unroll 1
    for (int r = 0; r < 16; ++r) {
      const unsigned sr = __shfl(see, (lane & 48) | r, kWave);
      VTile<BF, D> vr;
      vr.load(vv, pg, t0, lane);
#pragma unroll
      for (int i = 0; i < NZ; ++i)
        if (!(sr >> i & 1)) vr.clear(i);
#pragma unroll
      for (int n = 0; n < kAcc; ++n) {
        const f32x4 o = vr.template mul<PP>(n, pf, f32x4{0, 0, 0, 0});
        if (rl == r) acc[n] += o;
      }
    }
  });

  // join the waves' parts
  l = group_sum(l);
  live += __shfl_xor(live, 16, kWave);
  live += __shfl_xor(live, 32, kWave);
  __syncthreads();  // the last step's sums have been read
  if (c == 0) {
    sh.s[0][wave][rl][0] = l;
    sh.s[0][wave][rl][1] = __int_as_float(live);
  }
#pragma unroll
  for (int n = 0; n < kAcc; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) sh.o[wave][rl][VTile<BF, D>::coord(c, n, i)] = acc[n][i];
  if (wave == 0 && c == 0) {
    // NaN for a row that sees nothing, or no number
    sh.s[1][0][rl][0] = finite ? fmaf(a.am1, mx, th.t) : NAN;
    sh.s[1][0][rl][1] = finite ? 1.0f : mx == -INFINITY ? 0.0f : NAN;
  }
  __syncthreads();
  constexpr int TPR = D / 4;
  for (int r = tid / TPR; r < 16; r += NW * kWave / TPR) {
    if (!(which >> r & 1)) continue;
    const int d = (tid % TPR) * 4;
    float ls = 0.0f;
    int lv = 0;
    f32x4 o = {0, 0, 0, 0};
#pragma unroll
    for (int v = 0; v < NW; ++v) {
      ls += sh.s[0][v][r][0];
      lv += __float_as_int(sh.s[0][v][r][1]);
      o += *reinterpret_cast<const f32x4*>(&sh.o[v][r][d]);
    }
    const float kind = sh.s[1][0][r][1];
    const size_t at = row_at(a, w, r);
    const float inv = kind == 1.0f ? 1.0f / ls : kind;
    f32x4 y = o * inv;
    if (kind != 1.0f) y = f32x4{kind, kind, kind, kind};
    store_out<PARTS>(a.out, at * D + d, y);
    if (d == 0) {
      if (a.tau) a.tau[at] = sh.s[1][0][r][0];
      if (a.support) a.support[at] = lv;
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
// Sums and maxima over the 16 lanes of a row of lanes, and over the four rows

__device__ __forceinline__ float sum16(float x) {
  x += partner<1>(x);
  x += partner<2>(x);
  x += partner<4>(x);
  return x + partner<8>(x);
}
__device__ __forceinline__ float max16(float x) {
  x = fmaxf(x, partner<1>(x));
  x = fmaxf(x, partner<2>(x));
  x = fmaxf(x, partner<4>(x));
  return fmaxf(x, partner<8>(x));
}
template <typename T, typename Op>
__device__ __forceinline__ T reduce16(T x, Op op) {
  x = op(x, partner<1>(x));
  x = op(x, partner<2>(x));
  x = op(x, partner<4>(x));
  return op(x, partner<8>(x));
}
// NaN if one is among them; no LDS traffic
__device__ __forceinline__ float max_across(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  x = __builtin_elementwise_maximum(__uint_as_float(r[0]), __uint_as_float(r[1]));
  const uint32_t v = __float_as_uint(x);
  const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return __builtin_elementwise_maximum(__uint_as_float(s[0]), __uint_as_float(s[1]));
}

// ---------------------------------------------------------------------------
// Lists. An entry is (score, token).

__device__ __forceinline__ uint64_t entry(float z, int t) {
  return (uint64_t)(uint32_t)t << 32 | __float_as_uint(z);
}
__device__ __forceinline__ float entry_z(uint64_t e) { return __uint_as_float((uint32_t)e); }
__device__ __forceinline__ int entry_t(uint64_t e) { return (int)(e >> 32); }

// The threshold over a row's entries, y relative to the maximum mx, by 16
// lanes; each(f) calls f(z) for the lane's own entries.
template <typename Each>
__device__ __forceinline__ float solve16(const ChunkArgs& a, float mx, bool any, Each each) {
  Threshold th;
  th.done = !any;
  for (int i = 0; i < kSteps; ++i) {
    float s = 0.0f, s1 = 0.0f;
    each([&](float z) {
      float pm, pm1;
      powers(a, fmaxf((z - mx) * a.am1 - th.t, 0.0f), pm, pm1);
      s += pm;
      s1 += pm1;
    });
    s = sum16(s);
    s1 = sum16(s1);
    th.step(a, s, s1, i);
    if (__all(th.done)) break;
  }
  return th.t;
}
// A score below every token of the support of threshold t, roundings included.
__device__ __forceinline__ float bound_of(const ChunkArgs& a, float mx, float t) {
  return mx + (t - 2.0e-6f) / a.am1 - 1.0e-6f * fabsf(mx);
}

// A score below every one that may have a weight beside the maximum mx. What is
// relative to mx is for the difference's own rounding: half a unit in the last
// place of mx, 2^-24 of it, may be more than the window itself. (mx = +inf: NaN,
// which bounds nothing.)
__device__ __forceinline__ float window_below(const ChunkArgs& a, float mx) {
  return mx - a.window - 1.0e-6f * fabsf(mx);
}

// One row's running state, the same in the four lanes that hold its scores.
struct Track {
  float mx = -INFINITY, thr = -INFINITY;
  int n = 0;
};

// Keeps the entries of one row's list above thr, in order: 16 lanes a row, four
// groups of 16 entries on their way.
__device__ __forceinline__ int filter16(uint64_t* list, int lane, int n, float thr) {
  constexpr int U = 4;
  const int sub = lane & 15;
  int kept = 0;
  for (int i = 0; i < n; i += U * 16) {
    uint64_t e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) e[u] = i + u * 16 + sub < n ? list[i + u * 16 + sub] : 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {  // (entries move forward only)
      const bool keep = i + u * 16 + sub < n && !(entry_z(e[u]) <= thr);
      const unsigned all = (unsigned)(__ballot(keep) >> (lane & 48)) & 0xffffu;
      if (keep) list[kept + __popc(all & ((1u << sub) - 1))] = e[u];
      kept += __popc(all);
    }
  }
  return kept;
}

// Prunes one row's list to the tokens above `bound`, or, where more than `few`
// are left, above the threshold of what it holds, which is the next bound; from
// `slack` below it. n: its length, before and after.
__device__ __forceinline__ float prune16(const ChunkArgs& a, uint64_t* list, int lane, float mx,
                                         float bound, float slack, int few, int& n) {
  const int sub = lane & 15;
  n = filter16(list, lane, n, bound - slack);
  if (!__any(n > few)) return bound;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
  const float t = solve16(a, mx, n > few, [&](auto f) {
    if (n <= few) return;
    for (int i = sub; i < n; i += 16) f(entry_z(list[i]));
  });
  if (n > few) bound = fmaxf(bound, bound_of(a, mx, t));
  n = filter16(list, lane, n, bound - slack);
  return bound;
}

// The lists of the 16 rows of a tile, 4 rows at a time. at(row): its list.
template <typename At>
__device__ __forceinline__ void prune(const ChunkArgs& a, Track& tr, int room, int lane, At at) {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");  // the entries are written
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {
    const int row = k * 4 + (lane >> 4);
    int kept = max(__shfl(tr.n, row, kWave), 0);
    const float thr = prune16(a, at(row), lane, __shfl(tr.mx, row, kWave),
                              __shfl(tr.thr, row, kWave), 0.0f, room / 2, kept);
    // back to the lanes that hold these rows' scores
    const int from = ((lane & 3) << 4), mine = (lane & 15) >> 2;
    const int kn = __shfl(kept, from, kWave);
    const float kt = __shfl(thr, from, kWave);
    if (mine == k && tr.n > 0) {
      tr.n = kn;
      tr.thr = fmaxf(tr.thr, kt);
      if (kn > room) {
        tr.n = kLong;
        tr.thr = INFINITY;
      }
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
}

// One tile's scores of a row tile against the rows' bounds; tokens above them
// to the lists, in the order of the tokens a lane holds, then of the lanes.
template <bool BF, typename At>
__device__ __forceinline__ void collect(const ChunkArgs& a, Track& tr,
                                        const float (&z)[scores_per_lane<BF>()], float tmax, int t0,
                                        int lane, At at) {
  const int c = lane >> 4;
  tr.mx = __builtin_elementwise_maximum(tr.mx, max_across(tmax));
  tr.thr = fmaxf(tr.thr, window_below(a, tr.mx));
  // this row's four lanes, and those of them below this one
  const uint64_t row = 0x0001000100010001ull << (lane & 15), below = row & lanemask_below(lane);
  uint64_t* list = at(lane & 15);
#pragma unroll
  for (int i = 0; i < scores_per_lane<BF>(); ++i) {
    const bool hit = z[i] > tr.thr;
    const uint64_t all = __ballot(hit);
    if (all == 0) continue;
    if (hit) list[tr.n + __popcll(all & below)] = entry(z[i], t0 + tile_token<BF>(c, i));
    tr.n += __popcll(all & row);
  }
}

template <int N>
__device__ __forceinline__ float max_of(const float (&z)[N]) {
  float m = z[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = __builtin_elementwise_maximum(m, z[i]);
  return m;
}

__device__ __forceinline__ float max_of4(const f32x4& x) {
  return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
}

// The length to hand on.
__device__ __forceinline__ int length_of(const Track& tr) {
  return tr.mx < INFINITY ? tr.n : kNoNumber;  // (NaN too)
}

struct Cache {
  KvView k;
  const int32_t* table;
  int npages;
};
template <bool BF, int D>
__device__ __forceinline__ Cache cache_of(const ChunkArgs& a, const Rows& w, int top) {
  constexpr int kElem = BF ? 2 : 4;
  Cache x;
  x.k = KvView{static_cast<const char*>(a.k_pool) + ((size_t)w.g << a.ps_bits) * (D * kElem),
               ((size_t)a.Hkv << a.ps_bits) * (D * kElem), 1 << a.ps_bits};
  x.table = a.block_table + (size_t)w.b * a.max_pages;
  x.npages = (top + (1 << a.ps_bits) - 1) >> a.ps_bits;
  return x;
}

// Stages whose tiles' own maxima go before the bounds. Whole calls with none, 2 and 8
// of them, us (the same one again differs by 0.3, of the mixed batch by 1.5): prompts
// of 64 23.7, 21.8, 21.8, of 256 44.2, 41.6, 42.0, of 2048 124.3, 121.2, 122.8; mixed
// batch of 32 757.7, 756.5, 757.4.
constexpr int kYoung = 2;

// Row tiles a wave holds: with a bf16 cache 64 rows share each K operand read from
// LDS (4096 of 32K tokens 1.15 ms, with 32 rows 1.55); float32 rows take the
// registers of more.
template <bool BF>
constexpr int kListTiles = BF ? 4 : 2;

// A float32 query over bf16 keys takes three bf16 parts to be exact. To look for
// the few tokens that matter its nearest bf16 does: a score of it is off by at
// most e = sum |q - q'| * max |k| (both known), so that no token within 2 e of a
// bound is dropped; the finish kernel takes those that are left once more, in
// float32. (Two chunks of 512 among 32K tokens, list and finish kernel: float32
// queries 380 + 69 us, bf16 queries 336 + 40; three parts take three times the
// matrix instructions.)
template <int D>
__device__ __forceinline__ void load_nearest(QFrag<true, D, 1>& q, const char* row, int c,
                                             float& off) {
  off = 0.0f;
#pragma unroll
  for (int s = 0; s < D / 32; ++s)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4 x = row ? *reinterpret_cast<const f32x4*>(row + 4 * (s * 32 + c * 8 + 4 * h))
                          : f32x4{0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t b = nearest2(x[2 * e], x[2 * e + 1]);
        q.f[0][s][2 * h + e] = b;
        // (2^-18: the sum of products of that part, in float32)
        off += fabsf(x[2 * e] - __uint_as_float(b << 16)) +
               fabsf(x[2 * e + 1] - __uint_as_float(b & 0xffff0000u)) +
               (fabsf(x[2 * e]) + fabsf(x[2 * e + 1])) * 0x1p-18f;
      }
    }
  off = group_sum(off);
}

// Half the dimensions of a staged K tile (the operands of KTile), and their part
// of the scores of NT row tiles: all of them take a step before any takes the
// next, so that no matrix instruction waits for the one before it. Halves, as one
// is read while the other is used, and only one is held from tile to tile: with
// whole tiles the registers overflowed.
template <bool BF, int D, int NT>
struct KHalf;

template <int D, int NT>
struct KHalf<true, D, NT> {
  static constexpr int kSteps = D / 64;
  typedef f32x4 Acc[NT][2];
  u32x4 f[2][kSteps];
  __device__ __forceinline__ void read(lds_at st, int tile, int lane, int h) {
    typedef Stage<true, D> St;
    const int m = lane & 15, c = lane >> 4;
    const lds_at r = st + St::at(((m >> 2) << 3) + (m & 3), c);
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int u = 0; u < 2; ++u)
        f[u][s] = lds_read<u32x4>(St::on(r, 4 * (s + h * kSteps)) + tile * (St::kBytes / 2) +
                                  u * 4 * St::kRow);
  }
  template <int PARTS>
  __device__ __forceinline__ void add(const QFrag<true, D, PARTS> (&q)[NT], int h, Acc& acc) const {
#pragma unroll
    for (int k = PARTS - 1; k >= 0; --k)
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            acc[t][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                as_bf(f[u][s]), as_bf(q[t].f[k][s + h * kSteps]), acc[t][u], 0, 0, 0);
  }
  __device__ __forceinline__ static void scores(const Acc& acc, float (&z)[NT][8]) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 8; ++i) z[t][i] = acc[t][i / 4][i % 4];
  }
};

template <int D, int NT>
struct KHalf<false, D, NT> {
  static constexpr int kSteps = D / 32;
  typedef f32x4 Acc[NT][4];  // four sums each, as KTile's
  f32x4 f[kSteps];
  __device__ __forceinline__ void read(lds_at st, int tile, int lane, int h) {
    typedef Stage<false, D> St;
    const lds_at r = st + St::at(lane & 15, lane >> 4);
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
      f[s] = lds_read<f32x4>(St::on(r, 4 * (s + h * kSteps)) + tile * (St::kBytes / 2));
  }
  template <int PARTS>
  __device__ __forceinline__ void add(const QFrag<false, D, PARTS> (&q)[NT], int h,
                                      Acc& acc) const {
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[t][e] = __builtin_amdgcn_mfma_f32_16x16x4f32(f[s][e], q[t].f[s + h * kSteps][e],
                                                           acc[t][e], 0, 0, 0);
  }
  __device__ __forceinline__ static void scores(const Acc& acc, float (&z)[NT][4]) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        z[t][i] = (acc[t][0][i] + acc[t][1][i]) + (acc[t][2][i] + acc[t][3][i]);
  }
};

constexpr int kFewCap = 96;  // of a wave's list in LDS

// A wave's hits wait in a queue until they fill a batch: a record is one lane's
// scores of a tile (NZ of one row), some above the row's bound. It takes a few
// instructions to queue one, and the work on rows and lists is done for 64 at
// once.
constexpr int kBatch = 64, kQueue = 4 * kBatch;  // (a tile brings 4 batches at most)

template <int NZ>
struct WaveRows {
  f32x4 z[NZ / 4][kQueue];
  int code[kQueue];       // row << 24 | the lane's first token
  f32x4 top[64];          // the largest scores of four classes of a row's tokens
  float thr[64];          // what a score has to pass, but for `off`
  int n[64];
  float off[64];          // of the row's scores, by the largest |key|
};

template <bool BF, int D>
union ListLds {
  struct {
    char st[2][Stage<BF, D>::kBytes];
    WaveRows<scores_per_lane<BF>()> rows[kChunkWaves];
    __align__(16) float kmax[2][kChunkWaves];
  } many;
  struct {
    uint64_t list[kChunkWaves][16][kFewCap];
    int n[kChunkWaves][16];
  } few;
};

// Takes the queue's hits to the rows' lists, 64 records at a time, a lane each,
// in the order of the queue. at(row): a row's list.
template <int NZ, typename At>
__device__ __forceinline__ void flush(const ChunkArgs& a, WaveRows<NZ>& w, int count, int lane,
                                      float kmax, At at) {
  const uint64_t below = lanemask_below(lane);
#pragma unroll 1
  for (int b = 0; b < count; b += kBatch) {
    const bool real = b + lane < count;
    const int code = real ? w.code[b + lane] : 0;
    const int row = code >> 24, tok = code & 0xffffff;
    float z[NZ];
#pragma unroll
    for (int i = 0; i < NZ / 4; ++i) {
      const f32x4 x = w.z[i][b + lane];
#pragma unroll
      for (int e = 0; e < 4; ++e) z[4 * i + e] = x[e];
    }
    // the new maxima first: they bound these very hits
    const float top = max_of(z);
    if (real && top < INFINITY)
      __hip_atomic_fetch_max(reinterpret_cast<float*>(&w.top[row]) + (tok / NZ & 3), top,
                             __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT);
    if (real && !(top < INFINITY)) w.n[row] = kNoNumber;
    // lanes of the same row
    uint64_t same = ~0ull;
#pragma unroll
    for (int i = 0; i < 6; ++i) {
      const bool bit = row >> i & 1;
      const uint64_t set = __ballot(bit);
      same &= bit ? set : ~set;
    }
    bool pending = real;
    for (;;) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      const int n = w.n[row];
      const float thr =
          fmaxf(w.thr[row], window_below(a, max_of4(w.top[row]))) - 2.0f * kmax * w.off[row];
      unsigned bits = 0;
#pragma unroll
      for (int i = 0; i < NZ; ++i) bits |= (z[i] > thr ? 1u : 0u) << i;
      pending = pending && bits != 0 && n >= 0;
      const int c = pending ? __popc(bits) : 0;
      // hits of the same row in the lanes before this one
      int to = n;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        to += __popcll(__ballot(c >> i & 1) & same & below) << i;
      const bool fits = pending && to + c <= a.cap;
      if (fits) {
        uint64_t* list = at(row) + to;
#pragma unroll
        for (int i = 0; i < NZ; ++i)
          if (bits >> i & 1) *list++ = entry(z[i], tok + i);
      }
      const uint64_t done = __ballot(fits) & same;
      if (fits && done >> lane == 1) w.n[row] = to + c;  // the last of the row
      pending = pending && !fits;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      const uint64_t long_ones = __ballot(pending);
      if (long_ones == 0) break;
      // prune that row's list and its neighbours', 4 rows at a time; thresholds are
      // solved where three quarters stay (where half do: 3.12 ms in place of 2.88, as
      // above with 256 entries)
      const int r = __builtin_amdgcn_readlane(row, __builtin_ctzll(long_ones));
      const int row4 = (r & ~3) + (lane >> 4);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");  // the entries are written
      int kept = max(w.n[row4], 0);
      const bool any = kept > 0;
      const float mx4 = max_of4(w.top[row4]);
      const float bound =
          prune16(a, at(row4), lane, mx4, fmaxf(w.thr[row4], window_below(a, mx4)),
                  2.0f * kmax * w.off[row4], a.cap / 4 * 3, kept);
      if ((lane & 15) == 0 && any) {
        const bool no_room = kept > a.cap - NZ;
        w.n[row4] = no_room ? kLong : kept;
        w.thr[row4] = fmaxf(w.thr[row4], bound);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  // A row's new bound, a row a lane: the threshold of the classes' four largest
  // scores alone, tokens like any others. It is nearly that of all tokens (the
  // largest ones lie apart; 32K tokens of spread 2.5 at alpha 1.5: 50 hits a row,
  // 43 by the exact threshold, 82 by the maximum alone). A few Newton steps from
  // below: stopped early, it bounds less.
  const f32x4 x = w.top[lane];
  const float mx = max_of4(x);
  float t = -1.0f;
  if (a.m >= 1.0f) {
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      float sum = 0.0f, sum1 = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float pm, pm1;
        powers(a, fmaxf((x[e] - mx) * a.am1 - t, 0.0f), pm, pm1);
        sum += pm;
        sum1 += pm1;
      }
      t += fmaxf((sum - root_of(a, sum)) * __builtin_amdgcn_rcpf(sum1), 0.0f);
    }
  }
  // (a row without a list takes no more hits; one without a score keeps its bound)
  w.thr[lane] = w.n[lane] < 0 ? INFINITY : fmaxf(w.thr[lane], bound_of(a, mx, t));
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// More than 16 rows: every wave has NT row tiles of its own, K staged in LDS for
// all of them. Bound by the matrix instructions, and beside them by hits (queue
// and flush): 4096 of 32K tokens, 32/8 heads of 128 dims, 1.16 ms or 890 TFLOP/s
// of the score product alone; without a hit 0.88 ms. A prompt of 2048, whose rows
// have nearly all of their hits before the bounds have settled: 86 us, its product
// 17.
template <bool BF, int D, int PARTS, int NT>
__device__ __forceinline__ void list_many(const ChunkArgs& a, const Rows& w, int split,
                                          ListLds<BF, D>& lds) {
  constexpr int TT = kTile<BF>;
  constexpr int NZ = scores_per_lane<BF>();
  constexpr int QB = PARTS == 1 ? 2 : 4;
  constexpr bool kNear = BF && PARTS > 1;  // scores of the queries' nearest bf16
  constexpr int QP = kNear ? 1 : PARTS;
  typedef Stage<BF, D> St;
  constexpr int ST = St::kTokens;
  constexpr int kQuarter = ST / kChunkWaves;
  constexpr int kLoads = St::kBytes / kChunkWaves / 1024;
  auto& sh = lds.many;

  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = lane >> 4, rl = lane & 15;
  const int wr = wave * NT * 16, wrows = max(min(NT * 16, w.rows - wr), 0);
  const int top = seen(a, w, w.rows - 1);
  const Cache x = cache_of<BF, D>(a, w, top);
  const int stages = (top + ST - 1) / ST, per = (stages + a.splits - 1) / a.splits;
  const int v0 = min(split * per, stages), v1 = min(v0 + per, stages);

  auto& mine = sh.rows[wave];
  mine.n[lane] = 0;
  mine.thr[lane] = -INFINITY;
  mine.top[lane] = f32x4{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  mine.off[lane] = 0.0f;
  int queued = 0;
  QFrag<BF, D, QP> q[NT];
  float thr[NT], kmax = 0.0f;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    thr[t] = -INFINITY;
    const bool live = t * 16 + rl < wrows;
    const char* row =
        live ? static_cast<const char*>(a.q) + row_at(a, w, wr + t * 16 + rl) * (D * QB) : nullptr;
    if constexpr (kNear) {
      float off;
      load_nearest<D>(q[t], row, c, off);
      if (c == 0) mine.off[t * 16 + rl] = off;
    } else {
      q[t].load(row, c);
    }
  }
  // tokens below `some` are seen by a row of this wave, below `every` by all
  const int some = wrows ? seen(a, w, wr + wrows - 1) : 0;
  const int every = wrows == NT * 16 ? seen(a, w, wr) : 0;

  int to[kLoads];  // where this lane's 16 bytes go
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int at = i * 1024 + lane * 16;
    const int r = at / St::kRow, ch = at % St::kRow / 16;
    to[i] = (wave * kQuarter + r) * St::kRow + ((ch ^ St::swizzle(wave * kQuarter + r)) << 4);
  }
  // the next 64 stages, one a lane: the page of this wave's quarter, and whether
  // all quarters lie in pages of the pool
  int base = v0, pg = -1;
  uint64_t valid = 0;
  auto look = [&](int v) {
    base = v;
    valid = ~0ull;
#pragma unroll
    for (int k = 0; k < kChunkWaves; ++k) {
      int p = -1;
      if (v + lane < v1)
        p = page_at(a, x.table, x.npages, ((v + lane) * ST + k * kQuarter) >> a.ps_bits);
      valid &= __ballot(p >= 0);
      if (k == wave) pg = p;
    }
  };
  // A stage goes through registers: asked for at the end of the stage two before
  // it, put into LDS at the end of the one before. (Direct loads into LDS have the
  // compiler wait for all of them at the next LDS read.)
  u32x4 raw[kLoads];
  auto ask = [&](int v) {
    const int p = __builtin_amdgcn_readlane(pg, v - base);
    const int t = v * ST + wave * kQuarter;
    const char* src = x.k.base + (size_t)max(p, 0) * x.k.page_bytes +
                      (size_t)(t & ((1 << a.ps_bits) - 1)) * St::kRow;
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      raw[i] = *reinterpret_cast<const u32x4*>(src + (i * 1024 + lane * 16));
  };
  auto put = [&](int v) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) *reinterpret_cast<u32x4*>(sh.st[v & 1] + to[i]) = raw[i];
    if constexpr (kNear) {
      // the largest |key| of this quarter's tokens that some row sees; one that is
      // no finite number gives scores that are none, and needs no room
      const int p = __builtin_amdgcn_readlane(pg, v - base);
      const int left = p >= 0 ? top - v * ST - wave * kQuarter : 0;  // tokens seen
      u16x2 big = {0, 0};
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          big = __builtin_elementwise_max(big,
                                          __builtin_bit_cast(u16x2, raw[i][e] & 0x7fff7fffu));
      int m = wave_max((int)max(big[0], big[1]));
      if (__builtin_expect(left < kQuarter || m >= 0x7f80, 0)) {
        m = 0;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int lo = raw[i][e] & 0x7fff, hi = raw[i][e] >> 16 & 0x7fff;
            const bool use = (i * 1024 + lane * 16) / St::kRow < left;
            m = max(m, use && lo < 0x7f80 ? lo : 0);
            m = max(m, use && hi < 0x7f80 ? hi : 0);
          }
        m = wave_max(m);
      }
      if (lane == 0) sh.kmax[v & 1][wave] = __uint_as_float((uint32_t)m << 16);
    }
  };
  // thr: the rows' bounds less what the scores may be off
  auto refresh = [&] {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      thr[t] = mine.thr[t * 16 + rl];
      if constexpr (kNear) thr[t] -= 2.0f * kmax * mine.off[t * 16 + rl];
    }
  };

  if (v0 < v1) {
    look(v0);
    ask(v0);
    put(v0);
    if (v0 + 1 < v1) ask(v0 + 1);
  }
  wait_vmcnt<0>();  // (the queries too: or the compiler waits for them in the loop)
  __syncthreads();
  // Tiles in turn, two a stage. The first half of a tile's keys is read from LDS
  // while the tile before it is looked through, the second half while the first
  // is used. One turn more empties the queue.
  int when = v0 + 1;  // the stage at which the queues are emptied next
  bool pages = true, pages_next = valid & 1;  // the stage lies in pages of the pool
  typedef KHalf<BF, D, NT> Half;
  Half k0;
  if (v0 < v1) k0.read(lds_addr(sh.st[0]), 2 * v0 & 3, lane, 0);
  for (int u = 2 * v0; u <= 2 * v1; ++u) {
    const int v = u >> 1, t0 = u * TT;
    const bool first = (u & 1) == 0;
    float z[NT][NZ];
    uint64_t lanes[NT], any = 0;  // lanes that have hits
    if (u < 2 * v1) {
      if (first) {
        pages = pages_next;
        if constexpr (kNear) {
          const f32x4 k = *reinterpret_cast<const f32x4*>(sh.kmax[v & 1]);
          const float m = max_of4(k);
          if (m > kmax) {
            kmax = m;
            refresh();
          }
        }
      }
      {
        Half k1;
        k1.read(lds_addr(sh.st[0]), u & 3, lane, 1);
        typename Half::Acc acc = {};
        __builtin_amdgcn_s_setprio(1);
        k0.template add<QP>(q, 0, acc);
        k1.template add<QP>(q, 1, acc);
        __builtin_amdgcn_s_setprio(0);
        Half::scores(acc, z);
      }
      if (!first) {
        // the other stage's keys, in place of those that every wave has read
        // before the last barrier
        if (v + 1 < v1) put(v + 1);
        pages_next = valid >> (v + 1 - base & 63) & 1;
        if (v + 2 < v1) {
          if (v + 2 - base == kWave) look(v + 2);
          ask(v + 2);
        }
        __syncthreads();
      }
      k0.read(lds_addr(sh.st[0]), (u + 1) & 3, lane, 0);  // (past the last: not used)
      if (t0 < some) {
        if (__builtin_expect(!pages || t0 + TT > every, 0)) {
          bool page_ok = true;
          if (!pages)
            page_ok = page_at(a, x.table, x.npages,
                              (t0 + tile_token<BF>(c, 0)) >> a.ps_bits) >= 0;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const int r = t * 16 + rl, hi = r < wrows && page_ok ? seen(a, w, wr + r) : 0;
#pragma unroll
            for (int i = 0; i < NZ; ++i)
              z[t][i] = t0 + tile_token<BF>(c, i) < hi ? z[t][i] : -INFINITY;
          }
        }
        float tmax[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) tmax[t] = max_of(z[t]);
        // until the bounds have settled, a tile's own maximum goes first
        if (__builtin_expect(v < v0 + kYoung, 0)) {
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float m = window_below(a, max_across(tmax[t]));  // (+inf has to be a hit: NaN here)
            if constexpr (kNear) m -= 2.0f * kmax * mine.off[t * 16 + rl];
            thr[t] = fmaxf(thr[t], m);
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          lanes[t] = __ballot(!(tmax[t] <= thr[t]));
          any |= lanes[t];
        }
      }
    }
    // The queues are emptied by all waves together, about when they hold a batch
    // (a row's hits become rarer as 1 / tokens): a wave that does so by itself
    // has the others wait at the next barrier. Before this tile's hits go in.
    // (4096 of 32K tokens, after 1/2, 1/4, 1/8, 1/16 of the tokens so far: 1293, 1218,
    // 1219, 1522 us.)
    int total = 0;
    if (any) {
#pragma unroll
      for (int t = 0; t < NT; ++t) total += __popcll(lanes[t]);
    }
    const bool due = first && v >= when;
    if (due) when = v + 1 + ((v - v0) >> 3);
    if (queued > 0 && (due || u == 2 * v1 || queued + total > kQueue)) {
      // (the arguments once more: they would fill the loop's scalar registers)
      auto kernarg = __builtin_amdgcn_kernarg_segment_ptr();
      asm volatile("" : "+s"(kernarg));
      const ChunkArgs b = *(const ChunkArgs*)kernarg;
      flush<NZ>(b, mine, queued, lane, kmax, [&](int row) {
        // (a row past the last has no hits: any address serves)
        return b.lists + (row_at(b, w, min(wr + row, w.rows - 1)) * b.splits + split) * b.cap;
      });
      queued = 0;
      refresh();
    }
    if (any == 0) continue;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (lanes[t] == 0) continue;
      const int at = __builtin_amdgcn_mbcnt_hi(
          (unsigned)(lanes[t] >> 32),
          __builtin_amdgcn_mbcnt_lo((unsigned)lanes[t], (unsigned)queued));
      if (__builtin_amdgcn_inverse_ballot_w64(lanes[t])) {
#pragma unroll
        for (int i = 0; i < NZ / 4; ++i)
          mine.z[i][at] = f32x4{z[t][4 * i], z[t][4 * i + 1], z[t][4 * i + 2], z[t][4 * i + 3]};
        mine.code[at] = ((t * 16 + rl) << 24) + t0 + tile_token<BF>(c, 0);
      }
      queued += __popcll(lanes[t]);
    }
  }
  if (lane < wrows)
    a.parts[row_at(a, w, wr + lane) * a.splits + split] =
        Part{mine.n[lane], max_of4(mine.top[lane]), 2.0f * kmax * mine.off[lane], mine.thr[lane]};
}

// At most 16 rows (single tokens): the waves share them and take turns at the
// tiles, loaded from memory straight into the operands' registers; each keeps
// lists of its own in LDS, joined at the end. Bound by memory: 30 sequences of 32K
// tokens (1.75 GB of keys) 320 us, 5.5 TB/s.
template <bool BF, int D, int PARTS>
__device__ __forceinline__ void list_few(const ChunkArgs& a, const Rows& w, int split,
                                         ListLds<BF, D>& lds) {
  constexpr int TT = kTile<BF>;
  constexpr int NZ = scores_per_lane<BF>();
  constexpr int QB = PARTS == 1 ? 2 : 4;
  constexpr int NW = kChunkWaves;
  auto& sh = lds.few;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = lane >> 4, rl = lane & 15;
  const int top = seen(a, w, w.rows - 1), every = w.rows == 16 ? seen(a, w, 0) : 0;
  const int hi = rl < w.rows ? seen(a, w, rl) : 0;
  const Cache x = cache_of<BF, D>(a, w, top);
  const int tiles = (top + TT - 1) / TT, per = (tiles + a.few_splits - 1) / a.few_splits;
  const int v0 = min(split * per, tiles), v1 = min(v0 + per, tiles);

  QFrag<BF, D, PARTS> q;
  q.load(rl < w.rows ? static_cast<const char*>(a.q) + row_at(a, w, rl) * (D * QB) : nullptr, c);
  Track tr;
  auto list = [&](int row) { return sh.list[wave][row]; };
  for (int base = v0 + wave; base < v1; base += NW * kWave) {
    // pages of this wave's next 64 tiles, one tile a lane
    const int nt = min(kWave, (v1 - base + NW - 1) / NW);
    int pg0 = -1, pg1 = -1;
    if (lane < nt) {
      const int j = ((base + lane * NW) * TT) >> a.ps_bits;
      pg0 = pg1 = page_at(a, x.table, x.npages, j);
      if (BF && a.ps_bits == 4) pg1 = page_at(a, x.table, x.npages, j + 1);
    }
    auto pages = [&](int j) {
      return TilePages{__builtin_amdgcn_readlane(pg0, j), __builtin_amdgcn_readlane(pg1, j)};
    };
    KTile<BF, D> kt;
    TilePages pc = pages(0);
    kt.load(x.k, pc, base * TT, lane);
    for (int j = 0; j < nt; ++j) {
      const int t0 = (base + j * NW) * TT;
      float z[NZ];
      kt.template scores<PARTS>(q, z);
      const TilePages now = pc;
      if (j + 1 < nt) {
        pc = pages(j + 1);
        kt.load(x.k, pc, t0 + NW * TT, lane);
      }
      if (now.p0 < 0 || now.p1 < 0 || t0 + TT > every) {
        const bool page_ok = (!BF || c < 2 ? now.p0 : now.p1) >= 0;
#pragma unroll
        for (int i = 0; i < NZ; ++i)
          z[i] = (page_ok & (t0 + tile_token<BF>(c, i) < hi)) ? z[i] : -INFINITY;
      }
      const float tmax = max_of(z);
      if (__any(!(tmax <= tr.thr))) {
        collect<BF>(a, tr, z, tmax, t0, lane, list);
        if (__any(tr.n > kFewCap - TT)) prune(a, tr, kFewCap - TT, lane, list);
      }
    }
  }
  if (c == 0) sh.n[wave][rl] = length_of(tr);
  __syncthreads();

  // join the waves' lists of a row, 16 lanes a row: what is within the window
  // of the joint maximum, or above the joint threshold if that is too much
  const int row = wave * 4 + c, sub = rl;
  int n[NW], worst = 0;
#pragma unroll
  for (int v = 0; v < NW; ++v) {
    n[v] = sh.n[v][row];
    worst = min(worst, n[v]);
  }
  auto each = [&](auto f) {
#pragma unroll
    for (int v = 0; v < NW; ++v)
      for (int i = sub; i < n[v]; i += 16) f(sh.list[v][row][i]);
  };
  float mx = -INFINITY;
  each([&](uint64_t e) { mx = fmaxf(mx, entry_z(e)); });
  mx = max16(mx);
  float thr = window_below(a, mx);
  int most = 0;
  each([&](uint64_t e) { most += entry_z(e) > thr ? 1 : 0; });
  const bool much = sum16((float)most) > (float)a.cap;
  if (__any(much)) {
    const float t = solve16(a, mx, much, [&](auto f) { each([&](uint64_t e) { f(entry_z(e)); }); });
    if (much) thr = fmaxf(thr, bound_of(a, mx, t));
  }
  const bool real = row < w.rows;
  const size_t part = parts_of(a, w, row).first + split;
  int kept = 0;
#pragma unroll
  for (int v = 0; v < NW; ++v)
    for (int i = 0; i < n[v]; i += 16) {
      const uint64_t e = i + sub < n[v] ? sh.list[v][row][i + sub] : 0;
      const bool keep = i + sub < n[v] && entry_z(e) > thr;
      const unsigned all = (unsigned)(__ballot(keep) >> (lane & 48)) & 0xffffu;
      const int at = kept + __popc(all & ((1u << sub) - 1));
      if (keep && real && at < a.cap) a.lists[part * a.cap + at] = e;
      kept += __popc(all);
    }
  if (sub == 0 && real)
    a.parts[part] = Part{worst < 0 ? worst : kept > a.cap ? kLong : kept, mx, 0.0f, thr};
}

template <bool BF>
constexpr int kListRows = kChunkWaves * 16 * kListTiles<BF>;

template <bool BF, int D, int PARTS>
__global__ __launch_bounds__(kChunkWaves * kWave, 2) void list_kernel(ChunkArgs a) {
  __shared__ __align__(1024) ListLds<BF, D> lds;
  // over the KV heads first: with 8 of them, the blocks that read the same
  // head's tokens share an XCD and its L2; then the parts. The blocks of few rows
  // come last: they are short and fill in behind the others (first, and last: odd
  // float32 chunks 283, 249 us, mixed batch of 32 761, 755).
  const unsigned many_items = gridDim.x - a.few_items;
  const bool few = blockIdx.x >= many_items;
  const int item = few ? blockIdx.x - many_items : blockIdx.x;
  const int splits = few ? a.few_splits : a.splits;
  const int x = item / a.Hkv, g = item - x * a.Hkv;
  const int id = x / splits, split = x - id * splits;
  const Rows w = few ? last_rows(a, id, g)
                     : find_rows(a, a.tok_bits, id, g, threadIdx.x & (kWave - 1));
  if (w.rows == 0 || few != w.rows <= 16) return;
  if (few)
    list_few<BF, D, PARTS>(a, w, split, lds);
  else if (w.rows <= 64)
    list_many<BF, D, PARTS, 1>(a, w, split, lds);
  else if (kListTiles<BF> == 2 || w.rows <= 128)
    list_many<BF, D, PARTS, 2>(a, w, split, lds);
  else
    list_many<BF, D, PARTS, kListTiles<BF>>(a, w, split, lds);
}

// ---------------------------------------------------------------------------
// tau and the output from the lists

// Times a bound is taken for lists too long for LDS, at most: each brings nearer
// the support of the row, or that it is too long.
constexpr int kJoins = 16;

// The lists of P parts as one: entry j of them lies at place(j).
template <int P>
struct Run {
  int before[P - 1], shift[P - 1], total = 0;
  __device__ __forceinline__ Run(const int* length, int first, int count, int cap) {
#pragma unroll
    for (int s = 0; s < P; ++s) {
      const int m = first + s < count ? length[first + s] : 0;
      total += m;
      if (s == P - 1) break;
      before[s] = total;
      shift[s] = cap - m;
    }
  }
  __device__ __forceinline__ int place(int j) const {
    int to = j;
#pragma unroll
    for (int s = 0; s < P - 1; ++s) to += j >= before[s] ? shift[s] : 0;
    return to;
  }
};

// 16 lanes a row, 16 rows a workgroup (as dense_kernel takes them). A row's
// entries go straight to the lanes' registers, LE a lane, where there are few
// enough of them, else through LDS, pruned. Each lane gathers D / 16 coordinates
// of the support's V rows. Bound by latency: lengths, entries, pages and V rows wait for
// each other, so a workgroup is small and many share a CU (the bound of five waves
// a SIMD: float32 queries, 4096 of 32K tokens, 187 us; without it 209). A prompt of
// 2048 39 us, of which 34 without the threshold's steps and 38 without the V rows.
// kDense: rows for the dense kernel are done here, by few workgroups, which need
// not share a CU: a launch less (kFewTiles).
template <bool BF, int D, int PARTS, int LE, bool kDense>
__global__ __launch_bounds__(kChunkWaves * kWave, kDense ? 1 : 5) void finish_kernel(ChunkArgs a, int tok_bits) {
  constexpr int kJoinCap = 16 * LE;
  constexpr int kElem = BF ? 2 : 4, kPer = D / 16;
  typedef uint32_t vec __attribute__((ext_vector_type(kPer * kElem / 4)));
  __shared__ uint64_t joint[16][kJoinCap];
  __shared__ int length[16][kChunkMaxSplits];
  __shared__ unsigned wave_dense[kChunkWaves];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), sub = tid & 15, row = tid >> 4;
  const int id = blockIdx.x / a.Hkv, g = blockIdx.x - id * a.Hkv;
  const Rows w = find_rows(a, tok_bits, id, g, lane);
  if (w.rows == 0) {
    if (!kDense && tid == 0) a.dense[blockIdx.x] = 0;
    return;
  }
  const bool real = row < w.rows;
  const size_t at = row_at(a, w, min(row, w.rows - 1));
  // the list block that the row is in, and its parts
  const int past = w.i0 & ((1 << a.tok_bits) - 1);  // tokens of that block before this tile
  Rows lw = w;
  lw.i0 -= past;
  lw.tok0 -= past;
  lw.rows = min(1 << a.tok_bits, w.n - lw.i0) << a.g_bits;
  const Parts pt = parts_of(a, lw, min(row, w.rows - 1) + (past << a.g_bits));
  const uint64_t* lists = a.lists + pt.first * a.cap;
  const Part* parts = a.parts + pt.first;
  uint64_t* list = joint[row];

  int worst = 0, total = 0;
  float mx = -INFINITY, low = -INFINITY, slack = 0.0f;
  for (int i = sub; i < pt.count; i += 16) {
    // (clamped, as tokens and pages are below: starts that do not ascend leave
    // parts that no block has written)
    const Part part = parts[i];
    const int m = min(max(part.n, 0), a.cap);
    length[row][i] = m;
    worst = min(worst, part.n);
    total += m;
    slack = fmaxf(slack, part.slack);
    if (part.n > 0) mx = fmaxf(mx, part.mx);
    if (part.n > 0) low = fmaxf(low, part.thr);
  }
  worst = reduce16(worst, [](int x, int y) { return min(x, y); });
  total = reduce16(total, [](int x, int y) { return x + y; });
  slack = max16(slack);
  mx = max16(mx);
  low = max16(low);
  if (worst < 0) total = 0;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");

  const int count = worst < 0 ? 0 : pt.count;

  // this lane's entries sub, sub + 16, ... of the row's n
  uint64_t e[LE];
  int n = total;
  if (!__any(total > kJoinCap || pt.count > 4)) {
    const Run<4> run(length[row], 0, count, a.cap);
#pragma unroll
    for (int i = 0; i < LE; ++i) {
      const int j = i * 16 + sub;
      e[i] = j < total ? lists[run.place(j)] : entry(-INFINITY, 0);
    }
  } else {
    // many: through LDS those that may have a weight, by the joint maximum and the
    // parts' bounds
    auto gather = [&](float thr) {
      int k = 0;
      auto take = [&](uint64_t x, bool mine) {
        const bool keep = mine && !(entry_z(x) <= thr);
        const unsigned all = (unsigned)(__ballot(keep) >> (lane & 48)) & 0xffffu;
        const int to = k + __popc(all & ((1u << sub) - 1));
        if (keep && to < kJoinCap) list[to] = x;
        k += __popc(all);
      };
      for (int s = 0; s < count; s += 8) {
        const Run<8> run(length[row], s, count, a.cap);
        for (int i = 0; i < run.total; i += LE * 16) {  // LE loads on their way
          uint64_t x[LE];
#pragma unroll
          for (int u = 0; u < LE; ++u) {
            const int j = i + u * 16 + sub;
            x[u] = j < run.total ? lists[s * a.cap + run.place(j)] : 0;
          }
#pragma unroll
          for (int u = 0; u < LE; ++u)
            if (i + u * 16 < run.total) take(x[u], i + u * 16 + sub < run.total);
        }
      }
      return k;
    };
    low = fmaxf(low, window_below(a, mx));
    n = gather(low - slack);
    // the first that fit bound the threshold of all
    for (int i = 0; i < kJoins && __any(n > kJoinCap); ++i) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      const bool much = n > kJoinCap;
      float big = -INFINITY;
#pragma unroll
      for (int k = 0; k < LE; ++k) big = fmaxf(big, much ? entry_z(list[k * 16 + sub]) : 0.0f);
      big = max16(big);
      const float t = solve16(a, big, much, [&](auto f) {
        for (int k = 0; k < LE; ++k)
          if (much) f(entry_z(list[k * 16 + sub]));
      });
      if (much) low = fmaxf(low, bound_of(a, big, t));
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      n = gather(low - slack);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int i = 0; i < LE; ++i)
      e[i] = i * 16 + sub < n ? list[min(i * 16 + sub, kJoinCap - 1)] : entry(-INFINITY, 0);
  }
  const bool dense = real && (worst == kLong || n > kJoinCap);
  // a bit for each of the workgroup's rows that is dense; the others go on
  const uint64_t lanes = __ballot(dense && sub == 0);
  if (lane == 0)
    wave_dense[tid / kWave] =
        (lanes & 1) | (lanes >> 15 & 2) | (lanes >> 30 & 4) | (lanes >> 45 & 8);
  __syncthreads();
  unsigned which = 0;
#pragma unroll
  for (int v = 0; v < kChunkWaves; ++v) which |= wave_dense[v] << (4 * v);
  if (!kDense && tid == 0) a.dense[blockIdx.x] = which;
  if (dense) n = total = 0;

  const char* kb = static_cast<const char*>(a.k_pool) + ((size_t)g << a.ps_bits) * (D * kElem) +
                   sub * (kPer * kElem);
  const char* vb = static_cast<const char*>(a.v_pool) + ((size_t)g << a.ps_bits) * (D * kElem) +
                   sub * (kPer * kElem);
  const size_t page_bytes = ((size_t)a.Hkv << a.ps_bits) * (D * kElem);
  // this lane's coordinates of K or V row `slot` (page * page_size + row)
  auto row_of = [&](const char* base, int slot) {
    return *reinterpret_cast<const vec*>(base + (size_t)(slot >> a.ps_bits) * page_bytes +
                                         (size_t)(slot & ((1 << a.ps_bits) - 1)) * (D * kElem));
  };
  auto coord = [](const vec& v, int d) {
    return BF ? (d & 1 ? bf16_hi(v[d / 2]) : bf16_lo(v[d / 2])) : __uint_as_float(v[BF ? 0 : d]);
  };
  const int32_t* table = a.block_table + (size_t)w.b * a.max_pages;
  const int last = (a.max_pages << a.ps_bits) - 1;
  auto slot_of = [&](int tok) {
    tok = min(max(tok, 0), last);
    const int page = min(max(table[tok >> a.ps_bits], 0), a.num_phys - 1);
    return (page << a.ps_bits) + (tok & ((1 << a.ps_bits) - 1));
  };
  auto solve = [&] {
    mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < LE; ++i) mx = fmaxf(mx, entry_z(e[i]));
    mx = max16(mx);
    return solve16(a, mx, n > 0, [&](auto f) {
#pragma unroll
      for (int i = 0; i < LE; ++i)
        if (i == 0 || __any(i * 16 < n)) f(entry_z(e[i]));
    });
  };
  // (asked for before the threshold is solved: the pages of a few tokens too many)
  int slot[LE];
#pragma unroll
  for (int i = 0; i < LE; ++i)
    slot[i] = i * 16 + sub < n ? slot_of(entry_t(e[i])) : 0;
  float t = solve();
  // scores of rounded queries: those that may be in the support again, in float32
  const bool again = BF && PARTS > 1 && __any(slack > 0.0f);
  if (again) {
    const float thr = bound_of(a, mx, t) - slack;
    int kept = 0;
#pragma unroll
    for (int i = 0; i < LE; ++i) {
      if (!__any(i * 16 < n)) break;
      const bool keep = i * 16 + sub < n && !(entry_z(e[i]) <= thr);
      const unsigned all = (unsigned)(__ballot(keep) >> (lane & 48)) & 0xffffu;
      if (keep)
        list[kept + __popc(all & ((1u << sub) - 1))] = entry(0.0f, slot[i]);
      kept += __popc(all);
    }
    n = kept;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    float q[kPer];
#pragma unroll
    for (int d = 0; d < kPer; ++d)
      q[d] = static_cast<const float*>(a.q)[at * D + sub * kPer + d];
    constexpr int U = 4;  // rows on their way
    for (int i = 0; i < n; i += U) {
      vec k[U];
      int at[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        at[j] = entry_t(list[min(i + j, n - 1)]);
        k[j] = row_of(kb, at[j]);
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        float z = 0.0f;
#pragma unroll
        for (int d = 0; d < kPer; ++d) z = fmaf(q[d], coord(k[j], d), z);
        z = sum16(z);
        if (sub == 0 && i + j < n) list[i + j] = entry(z, at[j]);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int i = 0; i < LE; ++i)
      e[i] = i * 16 + sub < n ? list[i * 16 + sub] : entry(-INFINITY, 0);
#pragma unroll
    for (int i = 0; i < LE; ++i) slot[i] = entry_t(e[i]);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    t = solve();
  }
  // the support: its weights and V rows, to LDS in order
  float l = 0.0f;
  int live = 0;
#pragma unroll
  for (int i = 0; i < LE; ++i) {
    if (!__any(i * 16 < n)) break;
    const float y = (entry_z(e[i]) - mx) * a.am1;
    const float u = n > 0 ? fmaxf(y - t, 0.0f) : 0.0f;
    const float p = weight_of(a, y, t, u);
    l += p;
    const bool keep = u > 0.0f;
    const unsigned all = (unsigned)(__ballot(keep) >> (lane & 48)) & 0xffffu;
    if (keep)
      list[live + __popc(all & ((1u << sub) - 1))] =
          entry(p, slot[i]);
    live += __popc(all);
  }
  l = sum16(l);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");

  float acc[kPer];
#pragma unroll
  for (int d = 0; d < kPer; ++d) acc[d] = 0.0f;
  constexpr int U = 8;  // rows on their way
  for (int i = 0; i < live; i += U) {
    float p[U];
    vec v[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const uint64_t x = list[min(i + k, live - 1)];
      p[k] = entry_z(x);
      v[k] = row_of(vb, entry_t(x));
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (i + k >= live) break;
#pragma unroll
      for (int d = 0; d < kPer; ++d) acc[d] = fmaf(p[k], coord(v[k], d), acc[d]);
    }
  }
  if (real && !dense) {
    const float inv = worst == kNoNumber ? NAN : total == 0 ? 0.0f : 1.0f / l;
#pragma unroll
    for (int d = 0; d < kPer; d += 4)
      store_out<PARTS>(a.out, at * D + sub * kPer + d,
                       f32x4{acc[d], acc[d + 1], acc[d + 2], acc[d + 3]} * inv);
    if (sub == 0) {
      if (a.tau) a.tau[at] = n > 0 ? fmaf(a.am1, mx, t) : NAN;
      if (a.support) a.support[at] = live;
    }
  }
  if constexpr (kDense) {
    __shared__ DenseLds<D> sh;
    if (which) dense_rows<BF, D, PARTS>(a, w, which, sh);
  }
}

template <bool BF, int D, int PARTS>
__global__ __launch_bounds__(kChunkWaves * kWave, 2) void dense_kernel(ChunkArgs a, int tok_bits) {
  __shared__ DenseLds<D> sh;
  const unsigned which = a.dense[blockIdx.x];
  if (which == 0) return;
  const int id = blockIdx.x / a.Hkv, g = blockIdx.x - id * a.Hkv;
  const Rows w = find_rows(a, tok_bits, id, g, threadIdx.x & (kWave - 1));
  dense_rows<BF, D, PARTS>(a, w, which, sh);
}

template <bool BF, int D, int PARTS, int LE>
void launch_finish(const ChunkArgs& a, const ChunkPlan& p, hipStream_t st) {
  const dim3 grid((unsigned)p.tiles), threads(kChunkWaves * kWave);
  if (p.kernels == 2)
    hipLaunchKernelGGL((finish_kernel<BF, D, PARTS, LE, true>), grid, threads, 0, st, a,
                       p.tile_bits);
  else
    hipLaunchKernelGGL((finish_kernel<BF, D, PARTS, LE, false>), grid, threads, 0, st, a,
                       p.tile_bits);
}

template <bool BF, int D, int PARTS>
hipError_t launch(const ChunkArgs& a, const ChunkPlan& p, int kernel, hipStream_t st) {
  const dim3 threads(kChunkWaves * kWave);
  if (kernel == 0)
    hipLaunchKernelGGL((list_kernel<BF, D, PARTS>), dim3((unsigned)p.items), threads, 0, st, a);
  else if (kernel == 1 && a.cap == 128)
    launch_finish<BF, D, PARTS, 8>(a, p, st);
  else if (kernel == 1)
    launch_finish<BF, D, PARTS, 16>(a, p, st);
  else
    hipLaunchKernelGGL((dense_kernel<BF, D, PARTS>), dim3((unsigned)p.tiles), threads, 0, st, a,
                       p.tile_bits);
  return hipGetLastError();
}

// Workgroups of the finish kernel up to which the dense rows are done there (beyond,
// the passes' registers keep too few of them on a CU). Prompts of 40, 264, 520, 648,
// 1032, 4104 workgroups, us: 13.3, 28.3, 39.6, 40.9, 48.6, 159 with the dense rows
// there, 15.2, 30.0, 41.5, 37.8, 44.8, 123 in a kernel of their own; with weights on
// all tokens 15.0, 51.9, 403, 428, 699, 4896 against 16.9, 53.3, 405, 416, 655, 4148;
// a float32 cache, 264, 520, 1032 workgroups: 57.5, 65.8, 106 against 59.2, 67.5, 89.
constexpr long long kFewTiles = 2 * kNumCUs;

}  // namespace

ChunkPlan plan_chunk(const LaunchShape& s, int num_tokens, float alpha) {
  ChunkPlan p;
  const int g_bits = __builtin_ctz(s.group);
  const int rows = s.bf16 ? kListRows<true> : kListRows<false>;
  p.tok_bits = __builtin_ctz(rows) - g_bits;
  p.tile_bits = 4 - g_bits;
  p.threads = kChunkWaves * kWave;
  p.tiles = ((long long)(num_tokens >> p.tile_bits) + s.batch) * s.num_kv_heads;
  p.kernels = p.tiles <= kFewTiles ? 2 : 3;
  const long long ids = (long long)(num_tokens >> p.tok_bits) + s.batch;
  const long long total = (long long)s.max_pages * s.page_size;
  // parts of a row's tokens: about two workgroups a CU where there are fewer
  // blocks; more parts bring more hits, as each begins without a bound (one, two,
  // four a CU, us: 4096 of 32K tokens 1260, 1261, 1378; mixed batch of 32 1050, 761,
  // 832; a prompt of 2048 153, 123, 130; odd float32 chunks 322, 283, 279)
  const auto parts_for = [&](long long want, long long blocks, long long least) {
    const long long n = want / (blocks > 0 ? blocks : 1), most = (total + least - 1) / least;
    const long long k = n < most ? n : most;
    return (int)(k < 1 ? 1 : k > kChunkMaxSplits ? kChunkMaxSplits : k);
  };
  const long long full = num_tokens >> p.tok_bits;
  p.splits = parts_for(2 * kNumCUs, (full > 0 ? full : 1) * s.num_kv_heads, 256);
  // single tokens: eight, and never a long cache by one workgroup (4, 8, 16 of
  // them: mixed batch of 32 1051, 1028, 1026 us)
  p.few_splits = parts_for(8 * kNumCUs, (long long)s.batch * s.num_kv_heads, 512);
  p.few_items = (long long)s.batch * s.num_kv_heads * p.few_splits;
  p.items = p.few_items + ids * s.num_kv_heads * p.splits;
  const auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  p.few_parts = (size_t)num_tokens * s.num_q_heads * p.splits;
  const size_t parts = p.few_parts + (size_t)p.few_items * 16;
  p.cap = cap_of(alpha);
  p.parts_off = parts * p.cap * 8;
  p.dense_off = p.parts_off + up(parts * sizeof(Part));
  p.ws_bytes = p.dense_off + up((size_t)p.tiles * 4);
  return p;
}

hipError_t launch_chunk(const LaunchShape& s, const ChunkPlan& p, int kernel, const void* q,
                        bool q_bf16, int num_tokens, const int32_t* token_starts,
                        const void* k_pool, const void* v_pool, const int32_t* block_table,
                        const int32_t* seq_lens, float alpha, void* out, float* tau,
                        int32_t* support, void* ws, hipStream_t st) {
  ChunkArgs a;
  a.q = q;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.starts = token_starts;
  a.out = out;
  a.tau = tau;
  a.support = support;
  a.N = num_tokens;
  a.B = s.batch;
  a.H = s.num_q_heads;
  a.Hkv = s.num_kv_heads;
  a.g_bits = __builtin_ctz(s.group);
  a.ps_bits = __builtin_ctz(s.page_size);
  a.max_pages = s.max_pages;
  a.num_phys = s.num_phys;
  a.am1 = (float)((double)alpha - 1.0);
  a.m = (float)(1.0 / ((double)alpha - 1.0));
  a.rooted = (float)(2.0 - (double)alpha);
  a.window = a.m * (1.0f + 4.0e-6f);
  a.whole = a.m == 1.0f || a.m == 2.0f || a.m == 3.0f || a.m == 4.0f ? (int)a.m : 0;
  a.tok_bits = p.tok_bits;
  a.splits = p.splits;
  a.few_splits = p.few_splits;
  a.few_parts = p.few_parts;
  a.few_items = (unsigned)p.few_items;
  a.cap = p.cap;
  a.lists = static_cast<uint64_t*>(ws);
  a.parts = reinterpret_cast<Part*>(static_cast<char*>(ws) + p.parts_off);
  a.dense = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + p.dense_off);
  if (!s.bf16) return s.head_dim == 64 ? launch<false, 64, 3>(a, p, kernel, st)
                                       : launch<false, 128, 3>(a, p, kernel, st);
  if (q_bf16) return s.head_dim == 64 ? launch<true, 64, 1>(a, p, kernel, st)
                                      : launch<true, 128, 1>(a, p, kernel, st);
  return s.head_dim == 64 ? launch<true, 64, 3>(a, p, kernel, st)
                          : launch<true, 128, 3>(a, p, kernel, st);
}

}  // namespace ekv
