// Softmax decode attention over the paged cache: a window with sinks, and a
// batch that shares a prefix.
//
//   z_t = q . k_t,  m = max z_t,  l = sum exp(z_t - m),
//   out = sum exp(z_t - m) v_t / l,  lse = m + ln l
//
// over the tokens a query sees. One pass over K and V: a wave holds 16 query
// rows (the heads of one KV group, times query tokens or sequences), the
// reference m, the sum l and the output in registers, and walks its tiles
// (softmax_impl.hpp). Any reference m gives the same quotient, so m follows
// the running maximum only when that has grown by more than kSlack: the sum
// stays below e^kSlack * tokens, far inside float32, and almost no tile pays
// for a rescale or a reduction across lanes.
//
// Work is split over the tokens of a row block; the parts (m_s, l_s, o_s) are
// joined by a second kernel: out = sum e^(m_s - M) o_s / sum e^(m_s - M) l_s.
#include "softmax_impl.hpp"

namespace ekv {
namespace {

constexpr float kSlack = 6.0f;
constexpr int kAttWaves = 4;
constexpr int kAttThreads = kAttWaves * kWave;

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
  int batch, H, Hkv, G, n, ps, max_pages, num_phys;
  int window, sinks;
  int prefix;            // tokens of the shared prefix (0: none)
  int pre_tiles, pre_splits, pre_items;  // row tiles and splits of the prefix part
  int row_tiles, splits;                 // of the other part
  int slots;                             // parts per row
};

// What one workgroup works on.
struct Block {
  int b, g;       // sequence (prefix part: none) and KV head
  int r0, nrows;  // first row of the block among its rows, rows of it
  int split, splits, slot;
  bool pre;
};

__device__ __forceinline__ Block block_of(const AttendArgs& a, int item) {
  Block w;
  if (item < a.pre_items) {
    w.pre = true;
    w.b = 0;
    w.split = item % a.pre_splits;
    const int x = item / a.pre_splits;
    w.g = x % a.Hkv;
    w.r0 = x / a.Hkv * 16;
    w.nrows = min(16, a.batch * a.G - w.r0);
    w.splits = a.pre_splits;
    w.slot = w.split;
  } else {
    item -= a.pre_items;
    w.pre = false;
    w.split = item % a.splits;
    int x = item / a.splits;
    w.g = x % a.Hkv;
    x /= a.Hkv;
    w.r0 = x % a.row_tiles * 16;
    w.b = x / a.row_tiles;
    w.nrows = min(16, a.n * a.G - w.r0);
    w.splits = a.splits;
    w.slot = a.pre_items ? a.pre_splits + w.split : w.split;
  }
  return w;
}

// Index of row r of the block among all [batch, n, H] rows, and the tokens it
// sees.
__device__ __forceinline__ void row_of(const AttendArgs& a, const Block& w, int L, int r,
                                       size_t* row, int* lo, int* hi) {
  if (w.pre) {
    const int b = r / a.G;
    *row = (size_t)b * a.H + w.g * a.G + (r - b * a.G);
    *lo = 0;
    *hi = min(clamp_len(a.seq_lens[b], a.max_pages * a.ps), a.prefix);
  } else {
    const int i = r / a.G;
    *row = ((size_t)w.b * a.n + i) * a.H + w.g * a.G + (r - i * a.G);
    const int pos = L - a.n + i;
    *hi = max(pos + 1, 0);
    *lo = max(max(pos - a.window + 1, a.prefix), 0);
  }
}

template <bool BF, int D, int PARTS>
__global__ __launch_bounds__(kAttThreads, 2) void attend_kernel(AttendArgs a) {
  constexpr int TT = kTile<BF>;
  constexpr int NZ = scores_per_lane<BF>();
  constexpr int PP = PARTS == 3 ? 3 : 2;
  constexpr int PITCH = D + 4;
  constexpr int QB = PARTS == 1 ? 2 : 4;
  constexpr int kAcc = VTile<BF, D>::kAcc;
  __shared__ float so[kAttWaves][16][PITCH];
  __shared__ float sml[kAttWaves][16][2];

  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = lane >> 4, rl = lane & 15;
  const Block w = block_of(a, blockIdx.x);

  const int L = w.pre ? a.prefix : clamp_len(a.seq_lens[w.b], a.max_pages * a.ps);
  int lo = 0, hi = 0;
  size_t row = 0;
  if (rl < w.nrows) row_of(a, w, L, w.r0 + rl, &row, &lo, &hi);
  const int sinks = w.pre ? 0 : a.sinks;

  // tokens that some row sees, and that every row sees
  int ulo, uhi, flo, fhi;
  if (w.pre) {
    ulo = 0;
    uhi = hi;
    fhi = rl < w.nrows ? hi : INT32_MAX;
#pragma unroll
    for (int s = 1; s < 16; s <<= 1) {
      uhi = max(uhi, __shfl_xor(uhi, s, kWave));
      fhi = min(fhi, __shfl_xor(fhi, s, kWave));
    }
    uhi = __builtin_amdgcn_readfirstlane(uhi);
    fhi = __builtin_amdgcn_readfirstlane(fhi);
    flo = 0;
  } else {
    const int p0 = L - a.n + w.r0 / a.G, p1 = L - a.n + (w.r0 + w.nrows - 1) / a.G;
    ulo = max(max(p0 - a.window + 1, a.prefix), 0);
    uhi = max(p1 + 1, 0);
    flo = max(max(p1 - a.window + 1, a.prefix), 0);
    fhi = max(p0 + 1, 0);
  }
  const TileSpan span = tile_span<TT>(ulo, uhi, sinks);
  const int per = (span.n + w.splits - 1) / w.splits;
  const int v0 = min(w.split * per, span.n), v1 = min(v0 + per, span.n);

  const int32_t* table =
      w.pre ? a.prefix_table : a.block_table + (size_t)w.b * a.max_pages;
  const int npages = (uhi + a.ps - 1) / a.ps;
  KvView kv, vv;
  const size_t head_off = (size_t)w.g * a.ps * D * (BF ? 2 : 4);
  kv.base = static_cast<const char*>(a.k_pool) + head_off;
  vv.base = static_cast<const char*>(a.v_pool) + head_off;
  kv.page_bytes = vv.page_bytes = (size_t)a.Hkv * a.ps * D * (BF ? 2 : 4);
  kv.page_size = vv.page_size = a.ps;

  QFrag<BF, D, PARTS> q;
  q.load(rl < w.nrows ? static_cast<const char*>(a.q) + row * (D * QB) : nullptr, c);

  f32x4 acc[kAcc];
#pragma unroll
  for (int n = 0; n < kAcc; ++n) acc[n] = f32x4{0, 0, 0, 0};
  float m = -FLT_MAX, l = 0.0f;

  for (int base = v0 + wave; base < v1; base += kAttWaves * kWave) {
    // pages of this wave's next 64 tiles, one tile per lane
    const int nt = min(kWave, (v1 - base + kAttWaves - 1) / kAttWaves);
    int pg0 = -1, pg1 = -1;
    if (lane < nt) {
      const int t0 = span.tile(base + lane * kAttWaves) * TT;
      const int j = t0 / a.ps;
      pg0 = j < npages ? table[j] : -1;
      pg1 = pg0;
      if (BF && a.ps == 16) pg1 = j + 1 < npages ? table[j + 1] : -1;
      if (pg0 >= a.num_phys) pg0 = -1;
      if (pg1 >= a.num_phys) pg1 = -1;
    }
    KTile<BF, D> kt;
    VTile<BF, D> vt;
    auto pages = [&](int j) {
      return TilePages{__builtin_amdgcn_readlane(pg0, j), __builtin_amdgcn_readlane(pg1, j)};
    };
    auto start = [&](int j) { return span.tile(base + j * kAttWaves) * TT; };
    TilePages pc = pages(0);
    int t0 = start(0);
    kt.template load<true>(kv, pc, t0, lane);
    vt.template load<true>(vv, pc, t0, lane);
    uint64_t put_off = 0;
    for (int j = 0; j < nt; ++j) {
      float z[NZ];
      kt.template scores<PARTS>(q, z);
      TilePages pn = pc;
      int tn = t0;
      if (j + 1 < nt) {
        pn = pages(j + 1);
        tn = start(j + 1);
        kt.template load<true>(kv, pn, tn, lane);
      }
      const bool full = pc.p0 >= 0 && pc.p1 >= 0 &&
                        (t0 + TT <= fhi && (t0 >= flo || t0 + TT <= sinks));
      const bool page_ok = (!BF || c < 2 ? pc.p0 : pc.p1) >= 0;
      if (!full) {
#pragma unroll
        for (int i = 0; i < NZ; ++i) {
          const int t = t0 + tile_token<BF>(c, i);
          if (!(page_ok && t < hi && (t >= lo || t < sinks))) z[i] = -INFINITY;
        }
      }
      float tmax = z[0];
#pragma unroll
      for (int i = 1; i < NZ; ++i) tmax = fmaxf(tmax, z[i]);
      if (__any(tmax > m + kSlack)) {
        const float mn = fmaxf(m, group_max(tmax));
        const float f = exp2f((m - mn) * kLog2e);
        l *= f;
#pragma unroll
        for (int n = 0; n < kAcc; ++n) acc[n] *= f;
        m = mn;
      }
      float p[NZ];
#pragma unroll
      for (int i = 0; i < NZ; ++i) {
        p[i] = __builtin_amdgcn_exp2f((z[i] - m) * kLog2e);
        l += p[i];
      }
      bool later = false;
      if (!full) {
        // tokens no row sees take no part, whatever their rows hold; where
        // the rows differ in what they see, a value that is not finite must
        // not meet the zero weight of a row that does not see it: such a
        // tile's values wait
#pragma unroll
        for (int i = 0; i < NZ; ++i) {
          const int t = t0 + tile_token<BF>(c, i);
          if (!(page_ok && t < uhi && (t >= ulo || t < sinks))) vt.clear(i);
        }
        later = __any(vt.any_nonfinite());
      }
      if (later) put_off |= 1ull << j;
      else vt.template pv<PP>(p, acc);
      if (j + 1 < nt) vt.template load<true>(vv, pn, tn, lane);
      pc = pn;
      t0 = tn;
    }
    // the tiles put off: one row at a time, on the values that it sees (their
    // weights are in l already)
    while (put_off) {
      const int j = __builtin_ctzll(put_off);
      put_off &= put_off - 1;
      pc = pages(j);
      t0 = start(j);
      const bool page_ok = (!BF || c < 2 ? pc.p0 : pc.p1) >= 0;
      float p[NZ];
      kt.template load<true>(kv, pc, t0, lane);
      kt.template scores<PARTS>(q, p);
#pragma unroll
      for (int i = 0; i < NZ; ++i) {
        const int t = t0 + tile_token<BF>(c, i);
        const bool see = page_ok && t < hi && (t >= lo || t < sinks);
        p[i] = see ? __builtin_amdgcn_exp2f((p[i] - m) * kLog2e) : 0.0f;
      }
#pragma unroll 1
      for (int r = 0; r < 16; ++r) {
        const int rlo = __shfl(lo, r, kWave), rhi = __shfl(hi, r, kWave);
        vt.template load<true>(vv, pc, t0, lane);
#pragma unroll
        for (int i = 0; i < NZ; ++i) {
          const int t = t0 + tile_token<BF>(c, i);
          if (!(page_ok && t < rhi && (t >= rlo || t < sinks))) vt.clear(i);
        }
        vt.template pv<PP, true>(p, acc, rl == r);
      }
    }
  }

  // join the waves' parts
  l = group_sum(l);
  if (rl < w.nrows) {
    if (c == 0) {
      sml[wave][rl][0] = m;
      sml[wave][rl][1] = l;
    }
#pragma unroll
    for (int n = 0; n < kAcc; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) so[wave][rl][VTile<BF, D>::coord(c, n, i)] = acc[n][i];
  }
  __syncthreads();
  constexpr int TPR = D / 4;  // threads per row, 4 coordinates each
  for (int r = tid / TPR; r < w.nrows; r += kAttThreads / TPR) {
    const int d = (tid % TPR) * 4;
    float M = -FLT_MAX;
#pragma unroll
    for (int v = 0; v < kAttWaves; ++v)
      if (!(sml[v][r][1] == 0.0f)) M = fmaxf(M, sml[v][r][0]);
    float ls = 0.0f;
    f32x4 o = {0, 0, 0, 0};
#pragma unroll
    for (int v = 0; v < kAttWaves; ++v) {
      const float lv = sml[v][r][1];
      if (lv == 0.0f) continue;
      const float f = exp2f((sml[v][r][0] - M) * kLog2e);
      ls += f * lv;
      o += f * *reinterpret_cast<const f32x4*>(&so[v][r][d]);
    }
    size_t grow;
    int dlo, dhi;
    row_of(a, w, L, w.r0 + r, &grow, &dlo, &dhi);
    if (a.slots > 1) {
      const size_t part = grow * a.slots + w.slot;
      *reinterpret_cast<f32x4*>(a.part_o + part * D + d) = o;
      if (d == 0) {
        a.part_ml[2 * part] = M;
        a.part_ml[2 * part + 1] = ls;
      }
    } else {
      const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
      if constexpr (PARTS == 1) {
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = bf16_round(o[e] * inv);
        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + grow * D + d) =
            u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
      } else {
        *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + grow * D + d) = o * inv;
      }
      if (d == 0 && a.lse) a.lse[grow] = ls == 0.0f ? -INFINITY : M + kLn2 * log2f(ls);
    }
  }
}

// Joins the parts of each row: D/4 threads a row, 4 coordinates each.
template <int D, int PARTS>
__global__ __launch_bounds__(256) void join_kernel(const float* __restrict__ part_o,
                                                   const float* __restrict__ part_ml, int slots,
                                                   int rows, void* __restrict__ out,
                                                   float* __restrict__ lse) {
  constexpr int TPR = D / 4;
  const int r = blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
  if (r >= rows) return;
  const int d = (threadIdx.x % TPR) * 4;
  const float* ml = part_ml + (size_t)r * slots * 2;
  const float* po = part_o + (size_t)r * slots * D + d;
  float M = -FLT_MAX;
  for (int s = 0; s < slots; ++s)
    if (!(ml[2 * s + 1] == 0.0f)) M = fmaxf(M, ml[2 * s]);
  float l = 0.0f;
  f32x4 o = {0, 0, 0, 0};
  for (int s = 0; s < slots; ++s) {
    const float ls = ml[2 * s + 1];
    if (ls == 0.0f) continue;
    const float f = exp2f((ml[2 * s] - M) * kLog2e);
    l += f * ls;
    o += f * *reinterpret_cast<const f32x4*>(po + (size_t)s * D);
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  if constexpr (PARTS == 1) {
    uint32_t h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = bf16_round(o[e] * inv);
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(out) + (size_t)r * D + d) =
        u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
  } else {
    *reinterpret_cast<f32x4*>(static_cast<float*>(out) + (size_t)r * D + d) = o * inv;
  }
  if (d == 0 && lse) lse[r] = l == 0.0f ? -INFINITY : M + kLn2 * log2f(l);
}

template <bool BF, int D, int PARTS>
hipError_t launch(const AttendArgs& a, long long items, hipStream_t st) {
  hipLaunchKernelGGL((attend_kernel<BF, D, PARTS>), dim3((unsigned)items), dim3(kAttThreads), 0, st,
                     a);
  return hipGetLastError();
}

}  // namespace

// Parts of a row block's tokens: enough workgroups for kAttWgsPerCU a CU, of
// at least one tile per wave.
static int splits_for(long long blocks, long long tiles) {
  const long long want = (kAttWgsPerCU * kNumCUs + blocks - 1) / blocks;
  const long long most = (tiles + kAttWaves - 1) / kAttWaves;
  long long s = want < most ? want : most;
  if (s < 1) s = 1;
  if (s > kAttMaxSplits) s = kAttMaxSplits;
  return (int)s;
}

AttendPlan plan_attend(const LaunchShape& s, int n, int window, int sinks, int prefix_pages) {
  AttendPlan p;
  const int TT = s.bf16 ? kTile<true> : kTile<false>;
  const long long total = (long long)s.max_pages * s.page_size;
  const long long prefix = (long long)prefix_pages * s.page_size;
  p.rows = (long long)s.batch * n * s.num_q_heads;
  p.row_tiles = (n * s.group + 15) / 16;
  // tokens a row block of the sequences' own part can see
  const long long span = (long long)window + 16 / s.group + 1;
  const long long seen = total - prefix < span ? total - prefix : span;
  const long long tiles = (seen + TT - 1) / TT + 1 + (sinks + TT - 1) / TT;
  const long long blocks = (long long)s.batch * s.num_kv_heads * p.row_tiles;
  if (prefix_pages > 0) {
    p.pre_tiles = (s.batch * s.group + 15) / 16;
    const long long pre_blocks = (long long)s.num_kv_heads * p.pre_tiles;
    p.pre_splits = splits_for(pre_blocks, (prefix + TT - 1) / TT);
  }
  p.pre_items = (long long)s.num_kv_heads * p.pre_tiles * p.pre_splits;
  p.splits = total > prefix ? splits_for(blocks, tiles) : 0;
  p.items = p.pre_items + blocks * p.splits;
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
  a.G = s.group;
  a.n = n;
  a.ps = s.page_size;
  a.max_pages = s.max_pages;
  a.num_phys = s.num_phys;
  a.window = window;
  a.sinks = sinks;
  a.prefix = prefix_pages * s.page_size;
  a.pre_tiles = p.pre_tiles;
  a.pre_splits = p.pre_splits;
  a.pre_items = (int)p.pre_items;
  a.row_tiles = p.row_tiles;
  a.splits = p.splits;
  a.slots = p.slots;
  if (!s.bf16) return s.head_dim == 64 ? launch<false, 64, 3>(a, p.items, st)
                                       : launch<false, 128, 3>(a, p.items, st);
  if (q_bf16) return s.head_dim == 64 ? launch<true, 64, 1>(a, p.items, st)
                                      : launch<true, 128, 1>(a, p.items, st);
  return s.head_dim == 64 ? launch<true, 64, 3>(a, p.items, st)
                          : launch<true, 128, 3>(a, p.items, st);
}

hipError_t launch_join(const LaunchShape& s, const AttendPlan& p, bool q_bf16, void* out,
                       float* lse, void* ws, hipStream_t st) {
  const float* o = static_cast<const float*>(ws);
  const float* ml = reinterpret_cast<const float*>(static_cast<const char*>(ws) + p.ml_off);
  const int rows = (int)p.rows, per = 256 / (s.head_dim / 4);
  const dim3 grid((unsigned)((rows + per - 1) / per));
  if (s.head_dim == 64) {
    if (q_bf16) hipLaunchKernelGGL((join_kernel<64, 1>), grid, dim3(256), 0, st, o, ml, p.slots, rows, out, lse);
    else hipLaunchKernelGGL((join_kernel<64, 3>), grid, dim3(256), 0, st, o, ml, p.slots, rows, out, lse);
  } else {
    if (q_bf16) hipLaunchKernelGGL((join_kernel<128, 1>), grid, dim3(256), 0, st, o, ml, p.slots, rows, out, lse);
    else hipLaunchKernelGGL((join_kernel<128, 3>), grid, dim3(256), 0, st, o, ml, p.slots, rows, out, lse);
  }
  return hipGetLastError();
}

}  // namespace ekv
