// Accumulated attention weights of the cached tokens, and the eviction that
// keeps the heaviest of them.
//
//   weights:  w_out[b,g,t] = decay w_in[b,g,t] + sum over the heads h of KV
//             head g of p(h,t), p = exp(z - tau) or [(alpha-1) z - tau]_+^m
//   eviction: of each (sequence, KV head), the first `sinks` tokens, the last
//             `recent` ones and, of those between, the ones with the largest
//             weights (ties to the lower token), copied in order to new pages
#include "softmax_impl.hpp"

namespace ekv {
namespace {

// ---------------------------------------------------------------------------
// Weights. One pass over K: a wave takes tiles of one (sequence, KV head);
// scores as in the softmax decode (row = head = lane % 16), then the sum over
// rows by a butterfly across the 16 lanes that leaves each lane complete sums
// of its own tokens. Bound by reading K.

struct WeightArgs {
  const void* q;
  const void* k_pool;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const float* tau;
  const float* w_in;  // nullable
  float* w_out;
  int H, Hkv, G, ps, max_pages, num_phys;
  int window, sinks, splits;
  float decay, am1, m;
};

enum { kPowSoftmax = 0, kPow1 = 1, kPow2 = 2, kPow3 = 3, kPow4 = 4, kPowAny = 5 };

template <int POW>
__device__ __forceinline__ float weight_of(float z, float tau, float am1, float m) {
  if constexpr (POW == kPowSoftmax) return __builtin_amdgcn_exp2f((z - tau) * kLog2e);
  // not fmaxf: a NaN stays one
  float x = am1 * z - tau;
  x = x < 0.0f ? 0.0f : x;
  if constexpr (POW == kPow1) return x;
  if constexpr (POW == kPow2) return x * x;
  if constexpr (POW == kPow3) return x * x * x;
  if constexpr (POW == kPow4) return (x * x) * (x * x);
  return x == 0.0f ? 0.0f : exp2f(m * log2f(x));
}

template <bool BF, int D, int PARTS, int POW>
__global__ __launch_bounds__(256) void weights_kernel(WeightArgs a) {
  constexpr int TT = kTile<BF>;
  constexpr int NZ = scores_per_lane<BF>();
  constexpr int NW = 256 / kWave;
  constexpr int QB = PARTS == 1 ? 2 : 4;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = lane >> 4, rl = lane & 15;
  const int split = blockIdx.x % a.splits;
  const int x = blockIdx.x / a.splits;
  const int g = x % a.Hkv, b = x / a.Hkv;
  const int L = clamp_len(a.seq_lens[b], a.max_pages * a.ps);
  const int vis_lo = max(L - a.window, 0);
  const int tiles = (L + TT - 1) / TT;
  const int per = (tiles + a.splits - 1) / a.splits;
  const int v0 = min(split * per, tiles), v1 = min(v0 + per, tiles);
  const int npages = (L + a.ps - 1) / a.ps;
  const int32_t* table = a.block_table + (size_t)b * a.max_pages;
  KvView kv;
  kv.base = static_cast<const char*>(a.k_pool) + (size_t)g * a.ps * D * (BF ? 2 : 4);
  kv.page_bytes = (size_t)a.Hkv * a.ps * D * (BF ? 2 : 4);
  kv.page_size = a.ps;

  const bool live = rl < a.G;
  const size_t row = (size_t)b * a.H + g * a.G + rl;
  QFrag<BF, D, PARTS> q;
  q.load(live ? static_cast<const char*>(a.q) + row * (D * QB) : nullptr, c);
  const float tau = live ? a.tau[row] : 0.0f;

  const size_t wrow = ((size_t)b * a.Hkv + g) * ((size_t)a.max_pages * a.ps);
  typedef Butterfly<NZ, 16> Sum;
  const int own = Sum::first_index(rl);

  for (int base = v0 + wave; base < v1; base += NW * kWave) {
    const int nt = min(kWave, (v1 - base + NW - 1) / NW);
    int pg0 = -1, pg1 = -1;
    if (lane < nt) {
      const int j = (base + lane * NW) * TT / a.ps;
      pg0 = j < npages ? table[j] : -1;
      pg1 = pg0;
      if (BF && a.ps == 16) pg1 = j + 1 < npages ? table[j + 1] : -1;
      if (pg0 >= a.num_phys) pg0 = -1;
      if (pg1 >= a.num_phys) pg1 = -1;
    }
    auto pages = [&](int j) {
      return TilePages{__builtin_amdgcn_readlane(pg0, j), __builtin_amdgcn_readlane(pg1, j)};
    };
    KTile<BF, D> kt;
    TilePages pc = pages(0);
    kt.template load<true>(kv, pc, base * TT, lane);
    for (int j = 0; j < nt; ++j) {
      const int t0 = (base + j * NW) * TT;
      float z[NZ];
      kt.template scores<PARTS>(q, z);
      const TilePages pn = pages(min(j + 1, nt - 1));
      if (j + 1 < nt) kt.template load<true>(kv, pn, (base + (j + 1) * NW) * TT, lane);
      const bool page_ok = (!BF || c < 2 ? pc.p0 : pc.p1) >= 0;
#pragma unroll
      for (int i = 0; i < NZ; ++i) {
        const int t = t0 + tile_token<BF>(c, i);
        const bool see = live && page_ok && t < L && (t >= vis_lo || t < a.sinks);
        z[i] = see ? weight_of<POW>(z[i], tau, a.am1, a.m) : 0.0f;
      }
      Sum::reduce(z, rl);
      const int t = t0 + tile_token<BF>(c, own);
      if (Sum::owner(rl) && t < L)
        a.w_out[wrow + t] = (a.w_in ? a.decay * a.w_in[wrow + t] : 0.0f) + z[0];
      pc = pn;
    }
  }
}

// ---------------------------------------------------------------------------
// Selection: one workgroup per (sequence, KV head). A radix select over the
// order-preserving image of the weights, 8 bits a pass from the top, finds
// the smallest kept weight; each wave owns a contiguous stretch of tokens and
// the kept ones are written in order behind those of the waves before it.

constexpr int kEvThreads = 1024;
constexpr int kEvWaves = kEvThreads / kWave;

__device__ __forceinline__ uint32_t weight_order(float w) {
  return w != w ? 0xffffffffu : float_order(w + 0.0f);  // a NaN counts as the largest
}

__global__ __launch_bounds__(kEvThreads) void evict_select_kernel(
    const int32_t* __restrict__ lens, const float* __restrict__ weights, int Hkv, int max_tokens,
    int keep, int sinks, int recent, int32_t* __restrict__ kept, int32_t* __restrict__ new_lens) {
  __shared__ int hist[256];
  __shared__ int wcnt[kEvWaves][2];
  __shared__ int bc[2];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int row = blockIdx.x, b = row / Hkv;
  const int L = clamp_len(lens[b], max_tokens);
  const int n = min(L, keep);
  int32_t* out = kept + (size_t)row * keep;
  if (row % Hkv == 0 && tid == 0) new_lens[b] = n;
  for (int i = n + tid; i < keep; i += kEvThreads) out[i] = -1;
  if (L <= keep) {
    for (int i = tid; i < n; i += kEvThreads) out[i] = i;
    return;
  }
  // tokens [sinks, hi) compete for keep - sinks - recent places
  const int hi = L - recent;
  const float* w = weights + (size_t)row * max_tokens;
  uint32_t prefix = 0, pmask = 0;
  int k = keep - sinks - recent;  // places left among keys equal to the prefix
  for (int lo = 24; k > 0; lo -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int t = sinks + tid; t < hi; t += kEvThreads) {
      const uint32_t o = weight_order(w[t]);
      if ((o & pmask) == prefix) atomicAdd(&hist[(o >> lo) & 255], 1);
    }
    __syncthreads();
    if (wave == 0) {
      int c4[4], s = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) s += c4[i] = hist[4 * lane + i];
      const int incl = wave_incl_scan(s, lane);
      int above = lane_value(incl, kWave - 1) - incl;
      if (above < k && k <= above + s) {
#pragma unroll
        for (int i = 3; i >= 0; --i) {
          if (above < k && k <= above + c4[i]) {
            bc[0] = 4 * lane + i;
            bc[1] = above;
          }
          above += c4[i];
        }
      }
    }
    __syncthreads();
    prefix |= (uint32_t)bc[0] << lo;
    pmask |= 255u << lo;
    k -= bc[1];
    if (lo == 0) break;
  }
  // Kept: keys above the prefix, and the first k equal to it. (No places: the
  // mask is empty, every key equals the prefix, and k = 0 of them are kept.)
  const int per = ((hi - sinks + kEvWaves - 1) / kEvWaves + kWave - 1) & ~(kWave - 1);
  const int w0 = min(sinks + wave * per, hi), w1 = min(w0 + per, hi);
  int gt = 0, eq = 0;
  for (int t = w0 + lane; t < w1; t += kWave) {
    const uint32_t o = weight_order(w[t]) & pmask;
    gt += o > prefix;
    eq += o == prefix;
  }
  gt = wave_sum(gt);
  eq = wave_sum(eq);
  if (lane == 0) {
    wcnt[wave][0] = gt;
    wcnt[wave][1] = eq;
  }
  __syncthreads();
  int pos = sinks, eqs = 0;
  for (int v = 0; v < wave; ++v) {
    pos += wcnt[v][0];
    eqs += wcnt[v][1];
  }
  pos += min(eqs, k);
  for (int base = w0; base < w1; base += kWave) {
    const int t = base + lane;
    const uint32_t o = t < w1 ? weight_order(w[t]) & pmask : 0u;
    const bool is_eq = t < w1 && o == prefix;
    const uint64_t em = __ballot(is_eq);
    const int rank = eqs + __popcll(em & lanemask_below(lane));
    const bool take = t < w1 && (o > prefix || (is_eq && rank < k));
    const uint64_t tm = __ballot(take);
    if (take) out[pos + __popcll(tm & lanemask_below(lane))] = t;
    pos += __popcll(tm);
    eqs += __popcll(em);
  }
  for (int i = tid; i < sinks; i += kEvThreads) out[i] = i;
  for (int i = tid; i < recent; i += kEvThreads) out[keep - recent + i] = hi + i;
}

// ---------------------------------------------------------------------------
// Copy: kept rows of K and V to the new pages (row_bytes / 16 lanes a row),
// and the weights: the kept ones in slot order, 0 behind them. Workgroups
// below `chunks` of a (sequence, KV head) take kCopyRows slots each, those
// behind clear kClearTokens weights each.

constexpr int kCopyRows = 64;
constexpr int kClearTokens = 4096;

__global__ __launch_bounds__(256) void evict_copy_kernel(
    char* k_pool, char* v_pool, const int32_t* __restrict__ bt,
    const int32_t* __restrict__ lens, const float* __restrict__ weights,
    const int32_t* __restrict__ new_table, const int32_t* __restrict__ kept, int Hkv, int ps,
    int row_bytes, int max_pages, int num_phys, int keep, int chunks, int clears,
    float* __restrict__ new_weights) {
  const int row = blockIdx.x / (chunks + clears), chunk = blockIdx.x % (chunks + clears);
  const int b = row / Hkv, g = row % Hkv;
  const int max_tokens = max_pages * ps;
  const size_t wrow = (size_t)row * max_tokens;
  if (chunk >= chunks) {
    const int t0 = keep + (chunk - chunks) * kClearTokens;
    const int end = min(t0 + kClearTokens, max_tokens);
    for (int t = t0 + threadIdx.x; t < end; t += 256) new_weights[wrow + t] = 0.0f;
    return;
  }
  const int n = min(clamp_len(lens[b], max_tokens), keep);
  const int lanes = row_bytes / 16;
  const int off = (threadIdx.x % lanes) * 16;
  const size_t head = (size_t)g * ps * row_bytes, page = (size_t)Hkv * ps * row_bytes;
  const int32_t* list = kept + (size_t)row * keep;
  const int i0 = chunk * kCopyRows, end = min(n, i0 + kCopyRows);
  if (new_weights && threadIdx.x < kCopyRows) {
    const int i = i0 + threadIdx.x;
    if (i < min(keep, max_tokens)) new_weights[wrow + i] = i < n ? weights[wrow + list[i]] : 0.0f;
  }
  for (int i = i0 + threadIdx.x / lanes; i < end; i += 256 / lanes) {
    const int t = list[i];
    const int po = bt[(size_t)b * max_pages + t / ps];
    const int pn = new_table[(size_t)b * max_pages + i / ps];
    if (po < 0 || po >= num_phys || pn < 0 || pn >= num_phys) continue;
    const size_t src = po * page + head + (size_t)(t % ps) * row_bytes + off;
    const size_t dst = pn * page + head + (size_t)(i % ps) * row_bytes + off;
    const uint4 kx = *reinterpret_cast<const uint4*>(k_pool + src);
    const uint4 vx = *reinterpret_cast<const uint4*>(v_pool + src);
    *reinterpret_cast<uint4*>(k_pool + dst) = kx;
    *reinterpret_cast<uint4*>(v_pool + dst) = vx;
  }
}

template <bool BF, int D, int PARTS>
hipError_t launch_w(const WeightArgs& a, int pow, int items, hipStream_t st) {
  const dim3 grid((unsigned)items), block(256);
  switch (pow) {
    case kPowSoftmax: hipLaunchKernelGGL((weights_kernel<BF, D, PARTS, kPowSoftmax>), grid, block, 0, st, a); break;
    case kPow1: hipLaunchKernelGGL((weights_kernel<BF, D, PARTS, kPow1>), grid, block, 0, st, a); break;
    case kPow2: hipLaunchKernelGGL((weights_kernel<BF, D, PARTS, kPow2>), grid, block, 0, st, a); break;
    case kPow3: hipLaunchKernelGGL((weights_kernel<BF, D, PARTS, kPow3>), grid, block, 0, st, a); break;
    case kPow4: hipLaunchKernelGGL((weights_kernel<BF, D, PARTS, kPow4>), grid, block, 0, st, a); break;
    default: hipLaunchKernelGGL((weights_kernel<BF, D, PARTS, kPowAny>), grid, block, 0, st, a); break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_weights(const LaunchShape& s, const void* q, bool q_bf16, const void* k_pool,
                          const int32_t* bt, const int32_t* lens, float alpha, const float* tau,
                          int window, int sinks, float decay, const float* w_in, float* w_out,
                          hipStream_t st) {
  WeightArgs a;
  a.q = q;
  a.k_pool = k_pool;
  a.block_table = bt;
  a.seq_lens = lens;
  a.tau = tau;
  a.w_in = w_in;
  a.w_out = w_out;
  a.H = s.num_q_heads;
  a.Hkv = s.num_kv_heads;
  a.G = s.group;
  a.ps = s.page_size;
  a.max_pages = s.max_pages;
  a.num_phys = s.num_phys;
  a.window = window;
  a.sinks = sinks;
  a.decay = decay;
  const double am1 = (double)alpha - 1.0;
  a.am1 = (float)am1;
  a.m = alpha == 1.0f ? 0.0f : (float)(1.0 / am1);
  // integer exponents up to 4: as products (m within 1e-6 of the integer, as
  // for a float32 alpha of 4/3: x^1e-6 differs from 1 by less than 1e-5 at
  // x = 1e-4, whose power is 1e-12)
  int pow = kPowAny;
  if (alpha == 1.0f) pow = kPowSoftmax;
  else
    for (int m = 1; m <= 4; ++m)
      if (1.0 / am1 - m < 1e-6 && m - 1.0 / am1 < 1e-6) pow = m;
  const long long units = (long long)s.batch * s.num_kv_heads;
  const long long tiles = ((long long)s.max_pages * s.page_size + (s.bf16 ? 31 : 15)) / (s.bf16 ? 32 : 16);
  long long splits = (8 * kNumCUs + units - 1) / units;
  if (splits > (tiles + 3) / 4) splits = (tiles + 3) / 4;
  if (splits < 1) splits = 1;
  a.splits = (int)splits;
  const int items = (int)(units * splits);
  if (!s.bf16) return s.head_dim == 64 ? launch_w<false, 64, 3>(a, pow, items, st)
                                       : launch_w<false, 128, 3>(a, pow, items, st);
  if (q_bf16) return s.head_dim == 64 ? launch_w<true, 64, 1>(a, pow, items, st)
                                      : launch_w<true, 128, 1>(a, pow, items, st);
  return s.head_dim == 64 ? launch_w<true, 64, 3>(a, pow, items, st)
                          : launch_w<true, 128, 3>(a, pow, items, st);
}

hipError_t launch_evict_select(const LaunchShape& s, const int32_t* lens, const float* weights,
                               int keep, int sinks, int recent, int32_t* kept,
                               int32_t* new_lens, hipStream_t st) {
  hipLaunchKernelGGL(evict_select_kernel, dim3((unsigned)(s.batch * s.num_kv_heads)),
                     dim3(kEvThreads), 0, st, lens, weights, s.num_kv_heads,
                     s.max_pages * s.page_size, keep, sinks, recent, kept, new_lens);
  return hipGetLastError();
}

hipError_t launch_evict_copy(const LaunchShape& s, void* k_pool, void* v_pool, const int32_t* bt,
                             const int32_t* lens, const float* weights, int keep,
                             const int32_t* new_table, const int32_t* kept, float* new_weights,
                             hipStream_t st) {
  const int row_bytes = s.head_dim * (s.bf16 ? 2 : 4);
  const int max_tokens = s.max_pages * s.page_size;
  const int slots = keep < max_tokens ? keep : max_tokens;
  const int chunks = (slots + kCopyRows - 1) / kCopyRows;
  const int clears = new_weights ? (max_tokens - slots + kClearTokens - 1) / kClearTokens : 0;
  const long long rows = (long long)s.batch * s.num_kv_heads;
  hipLaunchKernelGGL(evict_copy_kernel, dim3((unsigned)(rows * (chunks + clears))), dim3(256), 0,
                     st, static_cast<char*>(k_pool), static_cast<char*>(v_pool), bt, lens, weights,
                     new_table, kept, s.num_kv_heads, s.page_size, row_bytes, s.max_pages,
                     s.num_phys, keep, chunks, clears, new_weights);
  return hipGetLastError();
}

}  // namespace ekv
