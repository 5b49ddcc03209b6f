// New tokens into the paged cache: pages, positions and slots for a step's
// tokens (plan_kernel), and their heads normed, rotated and written
// (append_kernel).
#include "mfma.hpp"
#include "launch.hpp"

namespace ekv {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// Plan

struct PlanArgs {
  const int32_t* seq_lens;
  const int32_t* new_tokens;
  const int32_t* free_pages;
  const int32_t* free_count;
  int32_t* block_table;
  int32_t* new_lens;
  int32_t* token_starts;
  int32_t* positions;
  int32_t* slots;
  int32_t* free_left;
  int B, N, max_pages, num_phys, ps_bits, capacity;
};

// A sequence with tokens among a workgroup's rows.
struct PlanEntry {
  int start, end, len, first, b;  // first: its first new page's place from the stack's top; -1 refused
};

// One launch. A workgroup owns NT token rows and scans all sequences' lengths
// for itself, NT at a time (two prefix sums: rows, then pages), up to its last
// row; so no workgroup waits for another. The sequences that meet its rows
// (each has one row at least: NT of them at most) are listed in LDS, and a row
// finds its own by bisection. The row that opens a page writes it to the block
// table. Sums: rows saturate at N + 1 (64 lanes of at most 2^24 fit int32), and
// pages wanted by sequences that fit are at most N. Bound by latency (two
// dependent loads, the scan's barriers, the bisection).
template <int NT>
__global__ __launch_bounds__(NT) void plan_kernel(PlanArgs a) {
  constexpr int NW = NT / kWave;
  __shared__ PlanEntry entry[NT];
  __shared__ int wave_rows[NW], tmp[2 * NW], s_taken;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wid = tid / kWave;
  const int t0 = blockIdx.x * NT, t1 = min(t0 + NT, a.N);
  const int ps = 1 << a.ps_bits, most = a.max_pages << a.ps_bits;
  const int have = clamp_len(a.free_count[0], a.capacity);
  if (tid == 0) s_taken = 0;
  int rows = 0, pages = 0, listed = 0, before = 0;  // sums over the sequences so far
  for (int base = 0; base < a.B; base += NT) {
    const int b = base + tid;
    int L = 0, n = 0;
    if (b < a.B) {
      L = clamp_len(a.seq_lens[b], most);
      n = max(a.new_tokens[b], 0);
    }
    const int mine = min(n, a.N + 1);
    const int inc = wave_incl_scan(mine, lane);
    if (lane == kWave - 1) wave_rows[wid] = min(inc, a.N + 1);
    __syncthreads();
    int at = rows, sum = rows;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      at += w < wid ? wave_rows[w] : 0;
      sum += wave_rows[w];
    }
    const int start = min(at + inc - mine, a.N + 1), end = min(at + inc, a.N + 1);
    rows = min(sum, a.N + 1);
    const bool fits = n <= most - L && end <= a.N;
    const int held = (L + ps - 1) >> a.ps_bits;
    const int need = fits ? ((L + n + ps - 1) >> a.ps_bits) - held : 0;
    const bool rowed = n > 0 && start < t1;
    // both prefix sums at once, with their totals
    const int ip = wave_incl_scan(need, lane), ir = wave_incl_scan(rowed ? 1 : 0, lane);
    if (lane == kWave - 1) {
      tmp[2 * wid] = ip;
      tmp[2 * wid + 1] = ir;
    }
    before += __syncthreads_count(rowed && end <= t0);
    int bp = pages, br = listed;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      bp += w < wid ? tmp[2 * w] : 0;
      br += w < wid ? tmp[2 * w + 1] : 0;
      pages += tmp[2 * w];
      listed += tmp[2 * w + 1];
    }
    const int upto = bp + ip;
    const bool granted = fits && (need == 0 || upto <= have);
    if (rowed && end > t0)
      entry[br + ir - 1 - before] = PlanEntry{start, end, L, granted ? upto - need : -1, b};
    if (blockIdx.x == 0 && b < a.B) {
      a.new_lens[b] = granted ? L + n : L;
      a.token_starts[b] = min(start, a.N);
      if (granted && need > 0) atomicMax(&s_taken, upto);
    }
    if (blockIdx.x != 0 && rows >= t1) break;  // the rest have no rows here
    __syncthreads();
  }
  __syncthreads();
  if (blockIdx.x == 0 && tid == 0) {
    a.token_starts[a.B] = min(rows, a.N);
    a.free_left[0] = have - s_taken;
  }
  const int r = t0 + tid;
  if (r >= a.N) return;
  int pos = 0, slot = -1;
  if (r < rows) {
    // the last entry that starts at or before row r (there is one: the rows of
    // all sequences follow each other)
    int lo = 0, hi = listed - before;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (entry[mid].start <= r) lo = mid; else hi = mid;
    }
    const PlanEntry e = entry[lo];
    pos = e.len + (r - e.start);
    if (e.first >= 0) {
      const int held = (e.len + ps - 1) >> a.ps_bits, j = pos >> a.ps_bits;
      int32_t* cell = a.block_table + (size_t)e.b * a.max_pages + j;
      int page;
      if (j < held) {
        page = *cell;
      } else {
        page = a.free_pages[have - 1 - (e.first + j - held)];
        if ((pos & (ps - 1)) == 0) *cell = page;
      }
      if (page >= 0 && page < a.num_phys) slot = (page << a.ps_bits) + (pos & (ps - 1));
    }
  }
  a.positions[r] = pos;
  a.slots[r] = slot;
}

// ---------------------------------------------------------------------------
// Norm, rotation, append

struct AppendArgs {
  const char* x[3];  // queries, keys, values of the first token
  size_t stride[3];  // bytes from a token to the next
  const int32_t* positions;
  const int32_t* slots;
  const double* freqs;
  const int32_t* pair_axis;
  const float* weight[2];  // of queries and keys; null: no norm
  void* out[3];            // q_out, k_pool, v_pool
  int n, H, Hkv, ps_bits, num_slots, half, axes, interleaved;
  float eps, q_scale;
};

// 8 values of a row
template <bool BF>
__device__ __forceinline__ void load8(const char* row, int unit, u32x4 (&r)[BF ? 1 : 2]) {
  const u32x4* p = reinterpret_cast<const u32x4*>(row + unit * (BF ? 16 : 32));
#pragma unroll
  for (int i = 0; i < (BF ? 1 : 2); ++i) r[i] = __builtin_nontemporal_load(p + i);
}
template <bool BF>
__device__ __forceinline__ void widen(const u32x4 (&r)[BF ? 1 : 2], float* f) {
#pragma unroll
  for (int i = 0; i < (BF ? 1 : 2); ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (BF) {
        f[2 * e] = bf16_lo(r[0][e]);
        f[2 * e + 1] = bf16_hi(r[0][e]);
      } else {
        f[4 * i + e] = __uint_as_float(r[i][e]);
      }
    }
}
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
template <bool BF>
__device__ __forceinline__ void store8(char* row, int unit, const float* f) {
  u32x4* p = reinterpret_cast<u32x4*>(row + unit * (BF ? 16 : 32));
  if constexpr (BF) {
    u32x4 r;
#pragma unroll
    for (int e = 0; e < 4; ++e)  // to nearest even, NaN kept
      r[e] = __builtin_bit_cast(
          uint32_t, __builtin_convertvector(f32x2{f[2 * e], f[2 * e + 1]}, bf16x2));
    *p = r;
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      u32x4 r;
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] = __float_as_uint(f[4 * i + e]);
      p[i] = r;
    }
  }
}

// sin and cos of position * freq. The product and its reduction to [-pi, pi]
// run in float64 (float32 is 0.03 off at position 2^19 already); what float32
// loses of the reduced angle is put back by the first term of the series, so
// both are good to about their last bit.
__device__ __forceinline__ f32x2 turn(int position, double freq) {
  const double a = (double)position * freq;
  const double k = rint(a * 0.15915494309189535);
  const double r = fma(k, -2.4492935982947064e-16, fma(k, -6.283185307179586, a));
  const float f = (float)r, d = (float)(r - (double)f);
  float s, c;
  sincosf(f, &s, &c);
  return f32x2{fmaf(-d, s, c), fmaf(d, c, s)};
}

// A workgroup takes TW tokens: their angles once for all heads, into LDS, then
// every wave some of their heads, D/16 lanes a head and 16 values a lane, so
// that the two values of a half-split pair meet in one lane. All in float32,
// one rounding at the store. Bound by memory, a copy of the projection's
// output.
constexpr int kAppendThreads = 256;

template <bool XBF, bool QBF, bool KVBF, int D, int TW>
__global__ __launch_bounds__(kAppendThreads) void append_kernel(AppendArgs a) {
  constexpr int LPH = D / 16;  // lanes a head
  constexpr int HPB = kAppendThreads / LPH;
  constexpr int XB = XBF ? 2 : 4;
  __shared__ f32x2 rot[TW][D / 2];
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * TW;
  for (int i = tid; i < TW * a.half; i += kAppendThreads) {
    const int t = i / a.half, p = i - t * a.half;
    if (t0 + t >= a.n) break;
    int axis = 0;
    if (a.axes > 1) axis = min(max(a.pair_axis[p], 0), a.axes - 1);
    rot[t][p] = turn(a.positions[(size_t)axis * a.n + t0 + t], a.freqs[p]);
  }
  __syncthreads();
  const int j = tid % LPH;
  // this lane's two units of 8 values: of a half-split rotation the same place
  // in both halves, as far as it goes
  const int hu = a.interleaved ? 0 : a.half / 8;
  const int u0 = j < hu ? j : 2 * j, u1 = j < hu ? j + hu : 2 * j + 1;
  const int heads = a.H + 2 * a.Hkv;
  for (int i = tid / LPH; i < TW * heads; i += HPB) {
    const int t = i / heads, hh = i - t * heads;
    if (t0 + t >= a.n) break;
    const int kind = hh < a.H ? 0 : hh < a.H + a.Hkv ? 1 : 2;
    const int head = hh - (kind == 0 ? 0 : kind == 1 ? a.H : a.H + a.Hkv);
    const size_t token = t0 + t;
    int slot = 0;
    if (kind > 0) {
      slot = a.slots[token];
      if (slot < 0 || slot >= a.num_slots) continue;
    }
    const char* row = a.x[kind] + token * a.stride[kind] + (size_t)head * (D * XB);
    u32x4 raw[2][XBF ? 1 : 2];
    load8<XBF>(row, u0, raw[0]);
    load8<XBF>(row, u1, raw[1]);
    float y[2][8];
    widen<XBF>(raw[0], y[0]);
    widen<XBF>(raw[1], y[1]);
    if (kind < 2) {
      const float* w = a.weight[kind];
      if (w) {
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(y[0][e], y[0][e], fmaf(y[1][e], y[1][e], ss));
        ss += partner<1>(ss);
        ss += partner<2>(ss);
        if (LPH == 8) ss += partner<4>(ss);
        const float rs = rsqrtf(fmaf(ss, 1.0f / D, a.eps));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          y[0][e] *= rs * w[u0 * 8 + e];
          y[1][e] *= rs * w[u1 * 8 + e];
        }
      }
      if (j < hu) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const f32x2 cs = rot[t][j * 8 + e];
          const float p = y[0][e], q = y[1][e];
          y[0][e] = p * cs[0] - q * cs[1];
          y[1][e] = p * cs[1] + q * cs[0];
        }
      } else if (a.interleaved) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if ((2 * j + u) * 4 < a.half) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const f32x2 cs = rot[t][(2 * j + u) * 4 + e];
              const float p = y[u][2 * e], q = y[u][2 * e + 1];
              y[u][2 * e] = p * cs[0] - q * cs[1];
              y[u][2 * e + 1] = p * cs[1] + q * cs[0];
            }
          }
      }
    }
    if (kind == 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[0][e] *= a.q_scale;
        y[1][e] *= a.q_scale;
      }
      char* dst = static_cast<char*>(a.out[0]) + (token * a.H + head) * (D * (QBF ? 2 : 4));
      store8<QBF>(dst, u0, y[0]);
      store8<QBF>(dst, u1, y[1]);
    } else {
      const int page = slot >> a.ps_bits, prow = slot & ((1 << a.ps_bits) - 1);
      char* dst = static_cast<char*>(a.out[kind]) +
                  ((((size_t)page * a.Hkv + head) << a.ps_bits) + prow) * (D * (KVBF ? 2 : 4));
      store8<KVBF>(dst, u0, y[0]);
      store8<KVBF>(dst, u1, y[1]);
    }
  }
}

// Tokens of a workgroup: one, so that few tokens still fill the chip, up to
// kAppendFew; four beyond, which share the angles' work. One against four, us:
//   tokens             64          1024         3001         4096         8192
//   32/8 heads of 128  4.3 : 8.3   7.7 : 12.6   18.7 : 22.4  23.4 : 24.9  40.2 : 36.6
//   64/8 heads of 128  5.1 : 12.0  12.2 : 23.5  26.9 : 33.9  33.9 : 37.6  60.1 : 58.3
//   16/8, three axes   3.5 : 6.7   5.3 : 8.1    13.3 : 16.7  16.6 : 19.3  29.7 : 27.2
//   8/8 of 64, float32 3.4 : 4.8   5.9 : 6.7    13.5 : 13.5  18.7 : 17.5  34.3 : 33.2
//   1/1 of 64          3.4 : 3.3   4.0 : 3.4    5.0 : 3.6    5.8 : 3.7    8.6 : 4.4
// (fewer lanes than a workgroup's have a head of a lone token in the last two, 96
// and 12 of 256: they would pass over earlier.)
constexpr int kAppendFew = 4096;

template <bool XBF, bool QBF, bool KVBF, int D>
hipError_t launch_append_t(const AppendArgs& a, hipStream_t st) {
  if (a.n <= kAppendFew)
    hipLaunchKernelGGL((append_kernel<XBF, QBF, KVBF, D, 1>), dim3((unsigned)a.n),
                       dim3(kAppendThreads), 0, st, a);
  else
    hipLaunchKernelGGL((append_kernel<XBF, QBF, KVBF, D, 4>), dim3((unsigned)((a.n + 3) / 4)),
                       dim3(kAppendThreads), 0, st, a);
  return hipGetLastError();
}

template <bool XBF, bool QBF>
hipError_t launch_append_q(const AppendArgs& a, bool kv_bf16, int D, hipStream_t st) {
  if (kv_bf16)
    return D == 64 ? launch_append_t<XBF, QBF, true, 64>(a, st)
                   : launch_append_t<XBF, QBF, true, 128>(a, st);
  return D == 64 ? launch_append_t<XBF, QBF, false, 64>(a, st)
                 : launch_append_t<XBF, QBF, false, 128>(a, st);
}

}  // namespace

hipError_t launch_plan_tokens(const LaunchShape& s, int num_tokens, const int32_t* seq_lens,
                              const int32_t* new_tokens, const int32_t* free_pages,
                              int free_capacity, const int32_t* free_count, int32_t* block_table,
                              int32_t* new_lens, int32_t* token_starts, int32_t* positions,
                              int32_t* slots, int32_t* free_left, hipStream_t st) {
  const PlanArgs a{seq_lens,  new_tokens, free_pages, free_count, block_table,
                   new_lens,  token_starts, positions, slots, free_left,
                   s.batch,   num_tokens, s.max_pages, s.num_phys,
                   __builtin_ctz(s.page_size), free_capacity};
  constexpr int NT = 1024;
  hipLaunchKernelGGL((plan_kernel<NT>), dim3((unsigned)((num_tokens + NT - 1) / NT)), dim3(NT), 0,
                     st, a);
  return hipGetLastError();
}

hipError_t launch_append_kv(const LaunchShape& s, const AppendParams& p, hipStream_t st) {
  AppendArgs a;
  for (int i = 0; i < 3; ++i) {
    a.x[i] = static_cast<const char*>(p.x[i]);
    a.stride[i] = (size_t)p.stride[i] * (p.x_bf16 ? 2 : 4);
    a.out[i] = p.out[i];
  }
  a.positions = p.positions;
  a.slots = p.slots;
  a.freqs = p.freqs;
  a.pair_axis = p.pair_axis;
  a.weight[0] = p.q_weight;
  a.weight[1] = p.k_weight;
  a.n = p.num_tokens;
  a.H = s.num_q_heads;
  a.Hkv = s.num_kv_heads;
  a.ps_bits = __builtin_ctz(s.page_size);
  a.num_slots = s.num_phys * s.page_size;
  a.half = p.rot_dim / 2;
  a.axes = p.axes;
  a.interleaved = p.interleaved;
  a.eps = p.eps;
  a.q_scale = p.q_scale;
  if (p.x_bf16)
    return p.q_bf16 ? launch_append_q<true, true>(a, s.bf16, s.head_dim, st)
                    : launch_append_q<true, false>(a, s.bf16, s.head_dim, st);
  return p.q_bf16 ? launch_append_q<false, true>(a, s.bf16, s.head_dim, st)
                  : launch_append_q<false, false>(a, s.bf16, s.head_dim, st);
}

}  // namespace ekv
