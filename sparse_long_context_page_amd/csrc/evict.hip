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
// Weights. One pass over K: scores as in the softmax decode (row = head =
// lane % 16), then the sum over rows by a butterfly across the 16 lanes that
// leaves each lane complete sums of its own tokens. Bound by reading K, which
// each wave streams through LDS of its own, one tile ahead. The tiles of all
// sequences, end to end, are shared out evenly over the workgroups of a KV
// head, whatever the lengths (an equal number of workgroups a sequence: 89
// against 7x us on lengths of 22K to 32K). No sum crosses a workgroup.

struct WeightArgs {
  const void* q;
  const void* k_pool;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const float* tau;
  const float* w_in;  // nullable
  float* w_out;
  int batch, H, Hkv, G, ps, max_pages, num_phys;
  int window, sinks, wgs;  // workgroups a KV head
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

constexpr int kWeightWaves = 4;

// Tiles [v0, v1) of sequence b.
template <bool BF, int D, int PARTS, int POW>
__device__ __forceinline__ void weights_of(const WeightArgs& a, int b, int g, int L, int v0,
                                           int v1, const WaveTile<BF, D>& tile,
                                           char (&buf)[2][WaveTile<BF, D>::kBytes], int wave,
                                           int lane) {
  constexpr int TT = kTile<BF>;
  constexpr int NZ = scores_per_lane<BF>();
  constexpr int NW = kWeightWaves;
  constexpr int QB = PARTS == 1 ? 2 : 4;
  const int c = lane >> 4, rl = lane & 15;
  const int vis_lo = max(L - a.window, 0);
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
    // the sum that this lane adds to, in tile j (0: none of its own)
    auto old_sum = [&](int j) {
      const int t = (base + j * NW) * TT + tile_token<BF>(c, own);
      return a.w_in && Sum::owner(rl) && t < L ? a.w_in[wrow + t] : 0.0f;
    };
    TilePages pc = pages(0);
    float old = old_sum(0);
    tile.load(kv, pc, base * TT, buf[0]);
    for (int j = 0; j < nt; ++j) {
      const int t0 = (base + j * NW) * TT;
      const TilePages pn = pages(min(j + 1, nt - 1));
      float next = 0.0f;
      if (j + 1 < nt) {
        next = old_sum(j + 1);
        tile.load(kv, pn, (base + (j + 1) * NW) * TT, buf[(j + 1) & 1]);
        wait_vmcnt<WaveTile<BF, D>::kLoads>();  // tile j has landed: the next one's are newer
      } else {
        wait_vmcnt<0>();
      }
      KTile<BF, D> kt;
      kt.read(buf[j & 1], 0, lane);
      float z[NZ];
      kt.template scores<PARTS>(q, z);
      const bool page_ok = (!BF || c < 2 ? pc.p0 : pc.p1) >= 0;
#pragma unroll
      for (int i = 0; i < NZ; ++i) {
        const int t = t0 + tile_token<BF>(c, i);
        const bool see = live && page_ok && t < L && (t >= vis_lo || t < a.sinks);
        z[i] = see ? weight_of<POW>(z[i], tau, a.am1, a.m) : 0.0f;
      }
      Sum::reduce(z, rl);
      const int t = t0 + tile_token<BF>(c, own);
      if (Sum::owner(rl) && t < L) a.w_out[wrow + t] = (a.w_in ? a.decay * old : 0.0f) + z[0];
      pc = pn;
      old = next;
    }
  }
}

template <bool BF, int D, int PARTS, int POW>
__global__ __launch_bounds__(kWeightWaves* kWave) void weights_kernel(WeightArgs a) {
  constexpr int TT = kTile<BF>;
  __shared__ __align__(16) char buf[kWeightWaves][2][WaveTile<BF, D>::kBytes];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  // KV heads first: what runs together reads neighbouring parts of a page
  const int g = blockIdx.x % a.Hkv, wg = blockIdx.x / a.Hkv;
  const int max_tokens = a.max_pages * a.ps;
  WaveTile<BF, D> tile;
  tile.init(lane);
  // every wave goes through the lengths, 64 sequences at a time: first for
  // the sum of all tiles, then for this workgroup's share [lo, hi) of them
  const auto tiles_of = [&](int b, int* L) {
    *L = b < a.batch ? clamp_len(a.seq_lens[b], max_tokens) : 0;
    return (*L + TT - 1) / TT;
  };
  long long total = 0;
  int L = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kWave) total += wave_sum(tiles_of(b0 + lane, &L));
  const long long lo = total * wg / a.wgs, hi = total * (wg + 1) / a.wgs;
  long long at = 0;
  for (int b0 = 0; b0 < a.batch && at < hi; b0 += kWave) {
    const int n = tiles_of(b0 + lane, &L);
    const int incl = wave_incl_scan(n, lane);
    const long long first = at + incl - n;
    uint64_t mine = __ballot(n > 0 && first < hi && first + n > lo);
    while (mine) {
      const int s = __builtin_ctzll(mine);
      mine &= mine - 1;
      const long long f = at + lane_value(incl - n, s);
      const int ns = lane_value(n, s);
      weights_of<BF, D, PARTS, POW>(a, b0 + s, g, lane_value(L, s), (int)max(lo - f, 0ll),
                                    (int)min(hi - f, (long long)ns), tile, buf[wave], wave, lane);
    }
    at += lane_value(incl, kWave - 1);
  }
}

// ---------------------------------------------------------------------------
// Selection: one workgroup per (sequence, KV head). A radix select over the
// order-preserving image of the weights finds the smallest kept one: digits of
// kDigit bits from the highest bit in which the keys differ (so that the first
// histogram is spread and its LDS atomics seldom meet), until the boundary
// digit is taken whole. Wave v holds the v-th stretch of the row, four
// neighbouring tokens a lane and step, in registers where it has at most
// kRegSteps steps (32768 tokens a row), else it reads it again for each pass;
// the kept tokens are written in order behind those of the waves before.

constexpr int kEvThreads = 1024;
constexpr int kEvWaves = kEvThreads / kWave;
constexpr int kDigit = 11;
constexpr int kBins = 1 << kDigit;
constexpr int kRegSteps = 8;   // steps of 4 * kWave tokens that a wave keeps in registers
constexpr int kStep = 4 * kWave;

__device__ __forceinline__ uint32_t weight_order(float w) {
  return w != w ? 0xffffffffu : float_order(w + 0.0f);  // a NaN counts as the largest
}

// Bins lie with a gap after every 32: a lane sums kPerLane neighbours, on
// other banks than the next lane's.
constexpr int kPerLane = kBins / kWave;
__host__ __device__ constexpr int bin_at(int b) { return b + b / kPerLane; }

struct EvictLds {
  int hist[bin_at(kBins)];
  uint32_t range[kEvWaves][2];
  int wcnt[kEvWaves][2];
  int bc[3];
};

// kRegs: the row fits the registers.
template <bool kRegs>
__device__ __forceinline__ void select_tokens(const float* __restrict__ w, int lo, int hi, int k,
                                              int pos, int32_t* __restrict__ out, EvictLds& sh) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  // stretches of whole steps, from the step that holds token lo
  const int first = lo & ~3;
  const int per = ((hi - first + kEvWaves * kStep - 1) / (kEvWaves * kStep)) * kStep;
  const int w0 = min(first + wave * per, hi), w1 = min(w0 + per, hi);
  const int steps = (w1 - w0 + kStep - 1) / kStep;
  // order keys of the lane's four tokens of step i; 0 (below every key) for
  // tokens that do not compete
  const auto load = [&](int i) -> uint4 {
    const int t = w0 + i * kStep + lane * 4;
    if (t >= w1) return make_uint4(0, 0, 0, 0);
    const float4 f = *reinterpret_cast<const float4*>(w + t);
    return make_uint4(t >= lo ? weight_order(f.x) : 0u,
                      t + 1 >= lo && t + 1 < w1 ? weight_order(f.y) : 0u,
                      t + 2 >= lo && t + 2 < w1 ? weight_order(f.z) : 0u,
                      t + 3 >= lo && t + 3 < w1 ? weight_order(f.w) : 0u);
  };
  uint4 reg[kRegs ? kRegSteps : 1];
  if constexpr (kRegs) {
#pragma unroll
    for (int i = 0; i < kRegSteps; ++i) reg[i] = load(i);
  }
  const auto each = [&](auto f) {
    if constexpr (kRegs) {
#pragma unroll
      for (int i = 0; i < kRegSteps; ++i) {
        f(reg[i].x);
        f(reg[i].y);
        f(reg[i].z);
        f(reg[i].w);
      }
    } else {
      constexpr int U = 4;  // loads in flight
      for (int i = 0; i < steps; i += U) {
        uint4 o[U];
#pragma unroll
        for (int e = 0; e < U; ++e) o[e] = load(i + e);
#pragma unroll
        for (int e = 0; e < U; ++e) {
          f(o[e].x);
          f(o[e].y);
          f(o[e].z);
          f(o[e].w);
        }
      }
    }
  };

  // the range of the keys
  uint32_t mn = 0xffffffffu, mx = 0;
  each([&](uint32_t o) {
    mn = min(mn, o - 1u);  // 0 wraps to the largest
    mx = max(mx, o);
  });
  mn = wave_min(mn);
  mx = wave_max(mx);
  if (lane == 0) {
    sh.range[wave][0] = mn;
    sh.range[wave][1] = mx;
  }
  for (int i = tid; i < bin_at(kBins); i += kEvThreads) sh.hist[i] = 0;
  __syncthreads();
#pragma unroll
  for (int v = 0; v < kEvWaves; ++v) {
    mn = min(mn, sh.range[v][0]);
    mx = max(mx, sh.range[v][1]);
  }
  ++mn;  // (there is a key: the row is longer than what is kept)
  // the boundary: keys above `prefix` (under the mask) and k equal ones stay
  uint32_t prefix = mx, pmask = 0xffffffffu;
  if (mn != mx) {
    int hb = 31 - __clz(mn ^ mx);
    pmask = ~((2u << hb) - 1u);
    prefix = mx & pmask;
    while (true) {
      const int sh0 = hb >= kDigit - 1 ? hb - (kDigit - 1) : 0;
      const uint32_t dmask = (2u << (hb - sh0)) - 1u;
      each([&](uint32_t o) {
        if (o != 0u && (o & pmask) == prefix) atomicAdd(&sh.hist[bin_at((o >> sh0) & dmask)], 1);
      });
      __syncthreads();
      if (wave == 0) {
        // the lane whose kPerLane bins, counted from the top, hold the
        // k-th key, then the bin among them
        int s = 0;
#pragma unroll 8
        for (int i = 0; i < kPerLane; ++i) s += sh.hist[bin_at(kBins - 1 - (lane * kPerLane + i))];
        const int below = wave_incl_scan(s, lane);
        const uint64_t hit = __ballot(below - s < k && k <= below);
        const int src = __builtin_ctzll(hit);
        const int base = lane_value(below - s, src);
        const int bin = kBins - 1 - (src * kPerLane + lane);
        const int cnt = lane < kPerLane ? sh.hist[bin_at(bin)] : 0;
        const int upto = base + wave_incl_scan(cnt, lane);
        if (upto - cnt < k && k <= upto) {
          sh.bc[0] = bin;
          sh.bc[1] = upto - cnt;
          sh.bc[2] = cnt;
        }
      }
      __syncthreads();
      prefix |= (uint32_t)sh.bc[0] << sh0;
      pmask |= dmask << sh0;
      k -= sh.bc[1];
      if (sh.bc[2] == k || sh0 == 0) break;
      hb = sh0 - 1;
      for (int i = tid; i < bin_at(kBins); i += kEvThreads) sh.hist[i] = 0;
      __syncthreads();
    }
  }

  // where each wave's kept tokens go
  int gt = 0, eq = 0;
  each([&](uint32_t o) {
    const uint32_t x = o & pmask;
    gt += x > prefix;
    eq += o != 0u && x == prefix;
  });
  gt = wave_sum(gt);
  eq = wave_sum(eq);
  if (lane == 0) {
    sh.wcnt[wave][0] = gt;
    sh.wcnt[wave][1] = eq;
  }
  __syncthreads();
  int eqs = 0;
  for (int v = 0; v < wave; ++v) {
    pos += sh.wcnt[v][0];
    eqs += sh.wcnt[v][1];
  }
  pos += min(eqs, k);
  const auto emit = [&](int i, const uint4& o) {
    const int t = w0 + i * kStep + lane * 4;
    const uint32_t k4[4] = {o.x, o.y, o.z, o.w};
    int e = 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) e += k4[r] != 0u && (k4[r] & pmask) == prefix;
    const int eincl = wave_incl_scan(e, lane);
    int rank = eqs + eincl - e;  // equal keys before this lane's
    bool take[4];
    int n = 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint32_t x = k4[r] & pmask;
      const bool is = k4[r] != 0u && x == prefix;
      take[r] = x > prefix || (is && rank < k);
      rank += is;
      n += take[r];
    }
    const int nincl = wave_incl_scan(n, lane);
    int at = pos + nincl - n;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (take[r]) out[at++] = t + r;
    pos += lane_value(nincl, kWave - 1);
    eqs += lane_value(eincl, kWave - 1);
  };
  if constexpr (kRegs) {
#pragma unroll
    for (int i = 0; i < kRegSteps; ++i)
      if (i < steps) emit(i, reg[i]);
  } else {
    uint4 o = load(0);
    for (int i = 0; i < steps; ++i) {
      const uint4 nx = load(i + 1);
      emit(i, o);
      o = nx;
    }
  }
}

__global__ __launch_bounds__(kEvThreads) void evict_select_kernel(
    const int32_t* __restrict__ lens, const float* __restrict__ weights, int Hkv, int max_tokens,
    int keep, int sinks, int recent, int32_t* __restrict__ kept, int32_t* __restrict__ new_lens) {
  __shared__ EvictLds sh;
  const int tid = threadIdx.x;
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
  const int hi = L - recent, places = keep - sinks - recent;
  for (int i = tid; i < sinks; i += kEvThreads) out[i] = i;
  for (int i = tid; i < recent; i += kEvThreads) out[keep - recent + i] = hi + i;
  if (places == 0) return;
  const float* w = weights + (size_t)row * max_tokens;
  if (hi - (sinks & ~3) <= kEvWaves * kRegSteps * kStep)
    select_tokens<true>(w, sinks, hi, places, sinks, out, sh);
  else
    select_tokens<false>(w, sinks, hi, places, sinks, out, sh);
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
  // as many workgroups as the CUs hold at once (their LDS: two at 128 dims),
  // each wave with a tile at least
  const int row = s.head_dim * (s.bf16 ? 2 : 4), tt = s.bf16 ? kTile<true> : kTile<false>;
  const long long lds = (long long)kWeightWaves * 2 * tt * row;
  const long long most = ((long long)s.max_pages * s.page_size + tt - 1) / tt * s.batch;
  long long wgs = ((long long)(kLdsPerCU / lds) * kNumCUs + s.num_kv_heads - 1) / s.num_kv_heads;
  if (wgs > (most + kWeightWaves - 1) / kWeightWaves) wgs = (most + kWeightWaves - 1) / kWeightWaves;
  a.batch = s.batch;
  a.wgs = (int)wgs;
  const int items = (int)(wgs * s.num_kv_heads);
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
