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
// each wave streams through LDS of its own, one tile ahead: 128K tokens, 8 KV
// heads of 128 bf16 dims in 44 us (6.2 TB/s), 8 sequences of 22K to 32K in 84
// us (5.7 TB/s). The tiles of all sequences, end to end, are shared out evenly
// over the workgroups of a KV head, whatever the lengths (an equal number of
// workgroups a sequence: 89 us for the 8). No sum crosses a workgroup. A window
// hides tokens from the sums, not from the reads (the 8 sequences, window of
// 4096: 86 us).

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

  const bool head = rl < a.G;
  const size_t row = (size_t)b * a.H + g * a.G + rl;
  QFrag<BF, D, PARTS> q;
  q.load(head ? static_cast<const char*>(a.q) + row * (D * QB) : nullptr, c);
  const float tau = head ? a.tau[row] : 0.0f;
  // a head whose decode saw nothing gave no token a weight (exp(z + inf) is not 0)
  const bool live = head && !(POW == kPowSoftmax ? tau == -INFINITY : tau != tau);

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
      kt.read(lds_addr(buf[j & 1]), 0, lane);
      float z[NZ];
      kt.template scores<PARTS>(q, z);
      const bool page_ok = (!BF || c < 2 ? pc.p0 : pc.p1) >= 0;
#pragma unroll
      for (int i = 0; i < NZ; ++i) {
        const int t = t0 + tile_token<BF>(c, i);
        const bool see = live & page_ok & sees(t, vis_lo, L, a.sinks);
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
  __shared__ __align__(1024) char buf[kWeightWaves][2][WaveTile<BF, D>::kBytes];
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
// Eviction, one kernel: `splits` workgroups per (sequence, KV head) each find
// the row's kept tokens, list those of their own share of the slots and copy
// these. (Finding them again costs reads that the L2 serves; handing a list
// from one kernel to the next cost a launch and left most CUs idle meanwhile:
// 15.7 -> 10.6 us for 1001 of 4001 tokens, 134 -> 128 us for 8192 of 22K to
// 32K tokens of 8 sequences, 8 KV heads of 128 bf16 dims: 4.3 TB/s, a large
// copy reaches 4.9.)
//
// The smallest kept weight comes from a radix select over the
// order-preserving image of the weights, less its least value: digits of
// kDigit bits from the range's highest bit (so that the first histogram is
// spread and its LDS atomics seldom meet), until the boundary digit is taken
// whole or holds so few keys that each can be ranked among them. Wave v holds the v-th
// stretch of the row, four neighbouring tokens a lane and step, in registers
// where it has at most kRegSteps steps (32768 tokens a row), else it reads it
// again for each pass (about six), in each of the row's workgroups: 32768 of
// 131072 tokens of 4 sequences in 320 us, 3.5 TB/s of the least bytes. The copy
// is bound by memory: kept rows of K and V read and written once.

constexpr int kEvWaves = kEvThreads / kWave;
constexpr int kDigit = 11;
constexpr int kBins = 1 << kDigit;
constexpr int kRegSteps = 8;   // steps of 4 * kWave tokens that a wave keeps in registers
constexpr int kStep = 4 * kWave;
constexpr int kFew = 256;      // boundary keys ranked one against the other

__device__ __forceinline__ uint32_t weight_order(float w) {
  return w != w ? 0xffffffffu : float_order(w + 0.0f);  // a NaN counts as the largest
}

// Set bits of m below this lane's.
__device__ __forceinline__ int lanes_below(uint64_t m) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
}

// Bins lie with a gap after every 32: a lane sums kPerLane neighbours, on
// other banks than the next lane's.
constexpr int kPerLane = kBins / kWave;
__host__ __device__ constexpr int bin_at(int b) { return b + b / kPerLane; }

struct EvictLds {
  int hist[bin_at(kBins)];
  __align__(16) uint32_t few[kFew];
  int nfew;
  uint32_t range[kEvWaves][2];
  int wcnt[kEvWaves][2];
  uint32_t bc[3];
};

// Calls keep_at(position among the kept, token) for the k heaviest of the
// tokens [lo, hi) (at least k + 1 of them), in token order per wave; positions
// count from pos. kRegs: the row fits the registers.
template <bool kRegs, typename Emit>
__device__ __forceinline__ void select_tokens(const float* __restrict__ w, int lo, int hi, int k,
                                              int pos, EvictLds& sh, Emit keep_at) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  // stretches of whole steps, from the step that holds token lo
  const int first = lo & ~3;
  const int per = ((hi - first + kEvWaves * kStep - 1) / (kEvWaves * kStep)) * kStep;
  const int w0 = min(first + wave * per, hi), w1 = min(w0 + per, hi);
  const int steps = (w1 - w0 + kStep - 1) / kStep;
  // keys of the lane's four tokens of step i: order keys less `low` (from 1
  // up), 0 for tokens that do not compete
  uint32_t low = 0;
  const auto load = [&](int i) -> uint4 {
    const int t = w0 + i * kStep + lane * 4;
    if (t >= w1) return make_uint4(0, 0, 0, 0);
    const float4 f = *reinterpret_cast<const float4*>(w + t);
    return make_uint4(t >= lo ? weight_order(f.x) - low : 0u,
                      t + 1 >= lo && t + 1 < w1 ? weight_order(f.y) - low : 0u,
                      t + 2 >= lo && t + 2 < w1 ? weight_order(f.z) - low : 0u,
                      t + 3 >= lo && t + 3 < w1 ? weight_order(f.w) - low : 0u);
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
        if (i * kStep >= per) break;  // the same in every wave
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
  if (tid == 0) sh.nfew = 0;
  __syncthreads();
#pragma unroll
  for (int v = 0; v < kEvWaves; ++v) {
    mn = min(mn, sh.range[v][0]);
    mx = max(mx, sh.range[v][1]);
  }
  // keys from 1 up: the digits then start at the range's own highest bit, not
  // at one that an exponent crosses (weights between 1e-3 and 10: 128 bins a
  // binade, not 8; 8.7 -> 3 us of LDS atomics for 32768 keys)
  low = mn;  // (one less than the least key: the row is longer than what is kept)
  mx -= low;
  mn = 1;
  if constexpr (kRegs) {
#pragma unroll
    for (int i = 0; i < kRegSteps; ++i) {
      reg[i].x -= reg[i].x ? low : 0u;
      reg[i].y -= reg[i].y ? low : 0u;
      reg[i].z -= reg[i].z ? low : 0u;
      reg[i].w -= reg[i].w ? low : 0u;
    }
  }
  // the boundary: keys above `prefix` (under the mask) and k equal ones stay
  uint32_t prefix = mx, pmask = 0xffffffffu;
  bool whole = false;  // every equal key stays
  if (mn != mx) {
    int hb = 31 - __clz(mn ^ mx);
    pmask = ~((2u << hb) - 1u);
    prefix = mx & pmask;
    while (true) {
      const int sh0 = hb >= kDigit - 1 ? hb - (kDigit - 1) : 0;
      const uint32_t dmask = (2u << (hb - sh0)) - 1u;
      each([&](uint32_t o) {
        if (o != 0u && (o & pmask) == prefix)
          atomicAdd(&sh.hist[bin_at((o >> sh0) & dmask)], 1);
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
      const int cnt = sh.bc[2];
      prefix |= sh.bc[0] << sh0;
      pmask |= dmask << sh0;
      k -= (int)sh.bc[1];
      whole = cnt == k;
      if (whole || sh0 == 0) break;
      if (cnt <= kFew) {
        // the boundary digit's keys, ranked by counting
        each([&](uint32_t o) {
          if (o != 0u && (o & pmask) == prefix) sh.few[atomicAdd(&sh.nfew, 1)] = o;
        });
        __syncthreads();
        if (tid < cnt) {
          const uint32_t o = sh.few[tid];
          int more = 0, same = 0;
#pragma unroll 4
          for (int i = 0; i < cnt; ++i) {
            more += sh.few[i] > o;
            same += sh.few[i] == o;
          }
          if (more < k && k <= more + same) {  // one value, maybe of several threads
            sh.bc[0] = o;
            sh.bc[1] = more;
            sh.bc[2] = same;
          }
        }
        __syncthreads();
        prefix = sh.bc[0];
        pmask = 0xffffffffu;
        k -= (int)sh.bc[1];
        whole = (int)sh.bc[2] == k;
        break;
      }
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
    bool take[4];
    if (whole) {  // no ranks among equals
#pragma unroll
      for (int r = 0; r < 4; ++r) take[r] = k4[r] != 0u && (k4[r] & pmask) >= prefix;
    } else {
      int e = 0;
#pragma unroll
      for (int r = 0; r < 4; ++r) e += k4[r] != 0u && (k4[r] & pmask) == prefix;
      const int eincl = wave_incl_scan(e, lane);
      int rank = eqs + eincl - e;  // equal keys before this lane's
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t x = k4[r] & pmask;
        const bool is = k4[r] != 0u && x == prefix;
        take[r] = x > prefix || (is && rank < k);
        rank += is;
      }
      eqs += lane_value(eincl, kWave - 1);
    }
    int at = pos, n = 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint64_t m = __ballot(take[r]);
      at += lanes_below(m);
      n += __popcll(m);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (take[r]) keep_at(at++, t + r);
    pos += n;
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

struct EvictArgs {
  char* k_pool;
  char* v_pool;
  const int32_t* bt;
  const int32_t* lens;
  const float* weights;
  const int32_t* new_table;
  int32_t* kept;
  int32_t* new_lens;
  float* new_weights;  // nullable
  int Hkv, ps_bits, max_pages, num_phys;
  int keep, sinks, recent, rows;
};

template <int ROW>  // bytes of a row
__global__ __launch_bounds__(kEvThreads) void evict_kernel(EvictArgs a, int splits) {
  __shared__ EvictLds sh;
  const int tid = threadIdx.x;
  const int row = blockIdx.x % a.rows, split = blockIdx.x / a.rows;
  const int b = row / a.Hkv, g = row - b * a.Hkv;
  const int max_tokens = a.max_pages << a.ps_bits;
  const int L = clamp_len(a.lens[b], max_tokens);
  const int n = min(L, a.keep);
  int32_t* kept = a.kept + (size_t)row * a.keep;
  if (g == 0 && split == 0 && tid == 0) a.new_lens[b] = n;
  // this workgroup's share of the slots, of the list behind them and of the
  // weights that end as 0
  const int per = (n + splits - 1) / splits;
  const int s0 = min(split * per, n), s1 = min(s0 + per, n);
  for (int i = n + split * kEvThreads + tid; i < a.keep; i += splits * kEvThreads) kept[i] = -1;
  const size_t wrow = (size_t)row * max_tokens;
  if (a.new_weights)
    for (int i = n + split * kEvThreads + tid; i < max_tokens; i += splits * kEvThreads)
      a.new_weights[wrow + i] = 0.0f;
  if (s0 == s1) return;

  if (L <= a.keep) {
    for (int i = s0 + tid; i < s1; i += kEvThreads) kept[i] = i;
  } else {
    // tokens [sinks, hi) compete for the places between
    const int hi = L - a.recent, end = a.keep - a.recent, places = end - a.sinks;
    for (int i = s0 + tid; i < min(s1, a.sinks); i += kEvThreads) kept[i] = i;
    for (int i = max(s0, end) + tid; i < s1; i += kEvThreads) kept[i] = hi + (i - end);
    if (places > 0 && s0 < end && s1 > a.sinks) {
      const float* w = a.weights + wrow;
      const auto keep_at = [&](int at, int t) {
        if (at >= s0 && at < s1) kept[at] = t;
      };
      if (hi - (a.sinks & ~3) <= kEvWaves * kRegSteps * kStep)
        select_tokens<true>(w, a.sinks, hi, places, a.sinks, sh, keep_at);
      else
        select_tokens<false>(w, a.sinks, hi, places, a.sinks, sh, keep_at);
    }
  }
  __syncthreads();  // the share's list is written

  if (a.new_weights)
    for (int i = s0 + tid; i < s1; i += kEvThreads)
      a.new_weights[wrow + i] = a.weights[wrow + kept[i]];
  constexpr int kLanes = ROW / 16;            // a row's lanes, 16 bytes each
  constexpr int kRows = kEvThreads / kLanes;  // rows at a time
  constexpr int U = 4;                        // of them a thread holds
  const int off = tid % kLanes * 16;
  const size_t page = ((size_t)a.Hkv << a.ps_bits) * ROW, head = ((size_t)g << a.ps_bits) * ROW;
  const int32_t* bt = a.bt + (size_t)b * a.max_pages;
  const int32_t* nt = a.new_table + (size_t)b * a.max_pages;
  const int rmask = (1 << a.ps_bits) - 1;
  for (int i0 = s0 + tid / kLanes; i0 < s1; i0 += U * kRows) {
    u32x4 kx[U], vx[U];
    int po[U], pn[U];
#pragma unroll
    for (int e = 0; e < U; ++e) {
      const int i = min(i0 + e * kRows, s1 - 1);
      const int t = kept[i];
      po[e] = bt[t >> a.ps_bits];
      pn[e] = i0 + e * kRows < s1 ? nt[i >> a.ps_bits] : -1;
      // (page 0 is read in the place of one that is not there)
      const bool there = po[e] >= 0 && po[e] < a.num_phys;
      const size_t src = (there ? (size_t)po[e] : 0) * page + head + (size_t)(t & rmask) * ROW + off;
      if (!there || pn[e] >= a.num_phys) pn[e] = -1;
      kx[e] = load_vec<u32x4>(a.k_pool + src);
      vx[e] = load_vec<u32x4>(a.v_pool + src);
    }
#pragma unroll
    for (int e = 0; e < U; ++e) {
      if (pn[e] < 0) continue;
      const size_t dst = (size_t)pn[e] * page + head + (size_t)((i0 + e * kRows) & rmask) * ROW + off;
      __builtin_nontemporal_store(kx[e], reinterpret_cast<u32x4*>(a.k_pool + dst));
      __builtin_nontemporal_store(vx[e], reinterpret_cast<u32x4*>(a.v_pool + dst));
    }
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

hipError_t launch_evict(const LaunchShape& s, void* k_pool, void* v_pool, const int32_t* bt,
                        const int32_t* lens, const float* weights, int keep, int sinks,
                        int recent, const int32_t* new_table, int32_t* kept, int32_t* new_lens,
                        float* new_weights, hipStream_t st) {
  EvictArgs a;
  a.k_pool = static_cast<char*>(k_pool);
  a.v_pool = static_cast<char*>(v_pool);
  a.bt = bt;
  a.lens = lens;
  a.weights = weights;
  a.new_table = new_table;
  a.kept = kept;
  a.new_lens = new_lens;
  a.new_weights = new_weights;
  a.Hkv = s.num_kv_heads;
  a.ps_bits = __builtin_ctz(s.page_size);
  a.max_pages = s.max_pages;
  a.num_phys = s.num_phys;
  a.keep = keep;
  a.sinks = sinks;
  a.recent = recent;
  a.rows = s.batch * s.num_kv_heads;
  // At most one workgroup a CU (its registers fill it) where the rows allow it:
  // 24 rows, 8000 of 16293 tokens, in 11 parts 70 us, in 10 53; of 64 slots at
  // least. From 129 rows a row is one workgroup, however many CUs stay free (4096
  // of 16384 tokens: 128 rows 4.6 TB/s read and written, 136 rows 4.0), and what
  // is over a multiple of the CUs runs by itself (256 rows 4.8, 264 rows 3.6).
  const int slots = keep < s.max_pages * s.page_size ? keep : s.max_pages * s.page_size;
  int splits = a.rows > kNumCUs ? 1 : kNumCUs / a.rows;
  if (splits > (slots + 63) / 64) splits = (slots + 63) / 64;
  const dim3 grid((unsigned)(a.rows * splits)), block(kEvThreads);
  switch (s.head_dim * (s.bf16 ? 2 : 4)) {
    case 128: hipLaunchKernelGGL(evict_kernel<128>, grid, block, 0, st, a, splits); break;
    case 256: hipLaunchKernelGGL(evict_kernel<256>, grid, block, 0, st, a, splits); break;
    default: hipLaunchKernelGGL(evict_kernel<512>, grid, block, 0, st, a, splits); break;
  }
  return hipGetLastError();
}

}  // namespace ekv
