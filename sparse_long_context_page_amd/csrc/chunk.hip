// alpha-entmax attention of a ragged batch of new tokens over the paged cache.
//
//   x_t = (alpha - 1) z_t, z_t = q . k_t;  sum_t [x_t - tau]_+^m = 1,
//   out = sum_t p_t v_t / sum_t p_t,  p_t = [x_t - tau]_+^m,  m = 1/(alpha-1)
//
// over the tokens up to the query's own position. Everything is computed from
// y_t = x_t - max x <= 0, whose threshold lies in [-1, 0).
#include "softmax_impl.hpp"

namespace ekv {
namespace {

constexpr int kChunkWaves = 4;

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
  int tok_bits;  // 2^tok_bits tokens a block of rows
  float am1, m;  // alpha - 1 and 1 / (alpha - 1)
  int whole;     // m if it is 1, 2, 3 or 4, else 0
};

// A block of rows: tokens i0 .. of sequence b (rows tok0 .. of q) and the heads
// of KV head g. rows = 0: none.
struct Rows {
  int b, g, tok0, i0, rows, n, L;
};

// Blocks of TB tokens are numbered so that sequence b's begin at starts[b] / TB
// + b: never fewer than it has, floor(starts[b+1] / TB) - floor(starts[b] / TB)
// + 1 >= ceil(n / TB), so that a workgroup finds its block by a search alone.
// 64 probes a step: two steps up to 4096 sequences.
__device__ __forceinline__ Rows find_rows(const ChunkArgs& a, int id, int g, int lane) {
  const auto start = [&](int b) { return clamp_len(a.starts[b], a.N); };
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int step = (hi - lo + kWave - 1) / kWave, at = lo + lane * step;
    const bool below = lane == 0 || (at < hi && (start(at) >> a.tok_bits) + at <= id);
    lo += (63 - __builtin_clzll(__ballot(below))) * step;
    hi = min(hi, lo + step);
  }
  Rows r;
  const int s = start(lo), i0 = (id - (s >> a.tok_bits) - lo) << a.tok_bits;
  r.b = lo;
  r.g = g;
  r.n = start(lo + 1) - s;
  r.i0 = i0;
  r.tok0 = s + i0;
  r.rows = i0 >= 0 && i0 < r.n ? min(1 << a.tok_bits, r.n - i0) << a.g_bits : 0;
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
      const float r = a.whole == 1 ? 1.0f
                      : a.whole == 2
                          ? __builtin_sqrtf(s)
                          : __builtin_amdgcn_exp2f((1.0f - 1.0f / a.m) * __builtin_amdgcn_logf(s));
      const float d = (s - r) / s1;
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

// Rows r0 .. r0 + 15 of a block by passes over all of their scores: the
// maximum, one pass a threshold step, and the weights' product with V. The
// workgroup's waves share the rows and take turns at the tiles.
template <bool BF, int D, int PARTS>
__device__ __forceinline__ void dense_rows(const ChunkArgs& a, const Rows& w, int r0,
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
  const int nrows = min(16, w.rows - r0);
  const bool mine = rl < nrows;
  const int hi = mine ? seen(a, w, r0 + rl) : 0;
  const int top = seen(a, w, r0 + nrows - 1);  // the last row sees the most
  const int tiles = (top + TT - 1) / TT, npages = (top + (1 << a.ps_bits) - 1) >> a.ps_bits;
  const size_t head_off = ((size_t)w.g << a.ps_bits) * (D * kElem);
  const size_t page_bytes = ((size_t)a.Hkv << a.ps_bits) * (D * kElem);
  const KvView kv{static_cast<const char*>(a.k_pool) + head_off, page_bytes, 1 << a.ps_bits};
  const KvView vv{static_cast<const char*>(a.v_pool) + head_off, page_bytes, 1 << a.ps_bits};
  const int32_t* table = a.block_table + (size_t)w.b * a.max_pages;

  QFrag<BF, D, PARTS> q;
  q.load(mine ? static_cast<const char*>(a.q) + row_at(a, w, r0 + rl) * (D * QB) : nullptr, c);

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
        z[i] = page_ok & (t0 + tile_token<BF>(c, i) < hi) ? z[i] : -INFINITY;
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
      float pm1;
      const float u = finite ? fmaxf((z[i] - ref) * a.am1 - th.t, 0.0f) : 0.0f;
      powers(a, u, p[i], pm1);
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
  for (int r = tid / TPR; r < nrows; r += NW * kWave / TPR) {
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
    const size_t at = row_at(a, w, r0 + r);
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

template <bool BF, int D, int PARTS>
__global__ __launch_bounds__(kChunkWaves * kWave, 2) void chunk_kernel(ChunkArgs a) {
  __shared__ DenseLds<D> sh;
  const int id = blockIdx.x / a.Hkv, g = blockIdx.x - id * a.Hkv;
  const Rows w = find_rows(a, id, g, threadIdx.x & (kWave - 1));
  for (int r0 = 0; r0 < w.rows; r0 += 16) dense_rows<BF, D, PARTS>(a, w, r0, sh);
}

template <bool BF, int D, int PARTS>
hipError_t launch(const ChunkArgs& a, long long items, hipStream_t st) {
  hipLaunchKernelGGL((chunk_kernel<BF, D, PARTS>), dim3((unsigned)items),
                     dim3(kChunkWaves * kWave), 0, st, a);
  return hipGetLastError();
}

}  // namespace

ChunkPlan plan_chunk(const LaunchShape& s, int num_tokens) {
  ChunkPlan p;
  p.tok_bits = 4 - __builtin_ctz(s.group);  // 16 rows
  p.threads = kChunkWaves * kWave;
  p.items = ((long long)(num_tokens >> p.tok_bits) + s.batch) * s.num_kv_heads;
  return p;
}

hipError_t launch_chunk(const LaunchShape& s, const ChunkPlan& p, const void* q, bool q_bf16,
                        int num_tokens, const int32_t* token_starts, const void* k_pool,
                        const void* v_pool, const int32_t* block_table, const int32_t* seq_lens,
                        float alpha, void* out, float* tau, int32_t* support, void* ws,
                        hipStream_t st) {
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
  a.tok_bits = p.tok_bits;
  a.am1 = (float)((double)alpha - 1.0);
  a.m = (float)(1.0 / ((double)alpha - 1.0));
  a.whole = a.m == 1.0f || a.m == 2.0f || a.m == 3.0f || a.m == 4.0f ? (int)a.m : 0;
  if (!s.bf16) return s.head_dim == 64 ? launch<false, 64, 3>(a, p.items, st)
                                       : launch<false, 128, 3>(a, p.items, st);
  if (q_bf16) return s.head_dim == 64 ? launch<true, 64, 1>(a, p.items, st)
                                      : launch<true, 128, 1>(a, p.items, st);
  return s.head_dim == 64 ? launch<true, 64, 3>(a, p.items, st)
                          : launch<true, 128, 3>(a, p.items, st);
}

}  // namespace ekv
