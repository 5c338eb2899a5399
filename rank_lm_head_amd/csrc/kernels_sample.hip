// kernels_sample.hip — a token drawn from each row of logits, and drafted
// tokens checked against a target's logits.
//
// A row x over n columns, with temperature T, has the weights
//   w_v = exp((x_v - max x) / T).
// In the order of larger x first, ties to the lower column, what may be drawn
// is a prefix: of the top_k first columns, those before which less than top_p
// of these columns' mass lies, and of those the ones of weight min_p at least.
// The token is the lowest column at which the kept mass, summed in column
// order, passes u times the kept mass.
//
// Weights are held in 64 bits: as doubles where sums have no common reference
// yet, and otherwise as integers, w 2^S rounded, whose sums do not depend on
// their order. A polynomial of degree 9 gives 2^f to 4e-14, so that a random
// number, which falls between two sums, is held against sums good to 1e-13.
//
// sample_tiles_kernel reads the logits once: a wave takes 2048 columns and
// leaves their largest logit, those of the tile's eight groups of 256, and,
// where the row's settings need the whole mass, their sum of weights.
// sample_rows_kernel has a block per row. With a bound that at least k groups'
// maxima reach, it reads again only the groups that hold what passes the
// bound. Where that does not settle the row (flat rows under top_p, long
// top_k), it splits the whole row by value until the border is known.
// What bounds a large call is the one read of the logits; a small one, the
// two launches.
#include <algorithm>

#include "device.h"
#include "launch.h"
#include "topk.h"

namespace lrh {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kTile = 2048;                 // columns of a wave
constexpr int kGroup = 256;                 // columns under one kept maximum
constexpr int kGroups = kTile / kGroup;     // of a tile
constexpr int kPer = kTile / kWave;         // columns of a lane
constexpr int kRowThreads = 512;
constexpr int kRowWaves = kRowThreads / kWave;
constexpr int kBins = 2048;
constexpr int kBinsPer = kBins / kRowThreads;
constexpr int kList = 4096;                 // columns that a row's block holds in LDS
constexpr int kAskGroups = 2 * kRowThreads; // groups looked at a time
constexpr double kLog2e = 1.4426950408889634;
constexpr int kFirstK = 32, kSecondK = 512; // groups' maxima above the bound of top_p's first and second try

// 2^t of -1000 <= t <= 0 to 4e-14: 2^f = 1 + f g(f) for |f| <= 1/2, g by
// interpolation at the Chebyshev nodes.
__device__ __forceinline__ double exp2_f64(double t) {
  t = fmax(t, -1000.0);
  const double n = rint(t), f = t - n;
  double g = 1.0203121063391729e-07;
  g = fma(g, f, 1.3255224878668817e-06);
  g = fma(g, f, 1.525268684626772e-05);
  g = fma(g, f, 0.00015403455852453838);
  g = fma(g, f, 0.0013333558179043112);
  g = fma(g, f, 0.009618129159402558);
  g = fma(g, f, 0.055504108664760424);
  g = fma(g, f, 0.2402265069581299);
  g = fma(g, f, 0.6931471805599453);
  return ldexp(fma(g, f, 1.0), (int)n);
}

// 16 bytes from an address aligned to its elements only.
__device__ __forceinline__ u32x4 load16_any(const void* p) {
  u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

template <typename T> struct Elems;
template <> struct Elems<float> {
  static constexpr int n = 4;
  static __device__ __forceinline__ float get(u32x4 v, int e) { return __uint_as_float(v[e]); }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
};
template <> struct Elems<uint16_t> {
  static constexpr int n = 8;
  static __device__ __forceinline__ float get(u32x4 v, int e) {
    return __uint_as_float((e & 1) ? (v[e >> 1] & 0xffff0000u) : (v[e >> 1] << 16));
  }
  static __device__ __forceinline__ float one(const uint16_t* p) { return bf16_to_f32(*p); }
};

// NaN is no candidate, as -inf; +inf counts as the largest finite logit.
__device__ __forceinline__ float tame(float x) { return fminf(fmaxf(x, neg_inf()), __FLT_MAX__); }

struct Args {
  const void* x;
  int64_t ld;
  const int32_t* idx;       // rows x n ids (negative: no candidate), or NULL: the column
  const float* u;
  int64_t u_ld;             // numbers of a sequence
  const float* temperature; // of each sequence, or NULL: the value for all
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  float temperature_all, top_p_all, min_p_all;
  int top_k_all;
  int64_t rows;
  int n;
  int tiles;
  int per;                  // rows of a sequence
  int bits;                 // S
  float* gmax;              // [row][tile][kGroups]
  float* tmax;              // [row][tile]
  double* tsum;             // [row][tile]; a block may put integers of the kept mass there
  int32_t* token;
  float* prob;
  float* probs;
  // verification
  const int32_t* drafted;   // [sequence][per - 1]
  const int32_t* list;      // [sequence][per - 1][k], or NULL: the drafted token alone
  const float* q;           // and their probabilities
  int k;
  const int32_t* length;    // [sequence] drafted tokens, or NULL: per - 1
  int32_t* count;
  int32_t* state;           // [row] the token drawn there, or kAccepted
  uint32_t* arrived;        // [sequence]
};
constexpr int kAccepted = -2;

// A row's settings. top_k 0, top_p >= 1 and min_p <= 0 leave everything in.
struct How {
  double c;      // log2(e) / T
  double top_p;
  double least;  // log2(min_p), or -inf
  int top_k;
  __device__ __forceinline__ bool whole() const { return !top_k && top_p >= 1.0 && least == -__builtin_inf(); }
  // whether the mass of all columns is needed
  __device__ __forceinline__ bool mass() const { return !top_k && (top_p < 1.0 || whole()); }
};
__device__ __forceinline__ How how_of(const Args& a, int64_t seq) {
  How h;
  float t = a.temperature ? a.temperature[seq] : a.temperature_all;
  const int k = a.top_k ? a.top_k[seq] : a.top_k_all;
  const float p = a.top_p ? a.top_p[seq] : a.top_p_all;
  const float m = a.min_p ? a.min_p[seq] : a.min_p_all;
  h.top_k = k > 0 && k < a.n ? k : 0;
  if (!(t > 0.f)) {   // greedy
    t = 1.f;
    h.top_k = 1;
  }
  h.c = kLog2e / (double)t;
  h.top_p = p < 1.f ? (double)fmaxf(p, 0.f) : 1.0;   // NaN: 1
  h.least = m > 0.f ? log2((double)fminf(m, 1.f)) : -__builtin_inf();
  return h;
}

// log2 of a candidate's weight; m is finite.
__device__ __forceinline__ double log_weight(float x, float m, double c) { return ((double)x - (double)m) * c; }
__device__ __forceinline__ uint64_t to_int(double w, int bits) {   // w 2^bits, at most 2^51, to the nearest integer
  return (uint64_t)__double_as_longlong(fma(w, __longlong_as_double((long long)(1023 + bits) << 52), 4503599627370496.0)) &
         0xfffffffffffffull;
}
__device__ __forceinline__ uint64_t int_weight(float x, float m, double c, int bits) {
  return to_int(exp2_f64(log_weight(x, m, c)), bits);
}

// What the kept mass before a column has to stay below: p of the mass, 1 at least.
__device__ __forceinline__ uint64_t share_of(uint64_t mass, double p) {
  return max((uint64_t)ceil(p * (double)mass), (uint64_t)1);
}
// The place of u in the mass.
__device__ __forceinline__ uint64_t place_of(uint64_t mass, float u) {
  const double t = (double)fminf(fmaxf(u, 0.f), 1.f) * (double)mass;   // NaN: 0
  return min((uint64_t)t, mass - 1);
}

__device__ __forceinline__ uint64_t wave_sum_u64(uint64_t x) {
#pragma unroll
  for (int o = 32; o; o >>= 1) x += __shfl_xor((unsigned long long)x, o);
  return x;
}
__device__ __forceinline__ double wave_sum_f64(double x) {
#pragma unroll
  for (int o = 32; o; o >>= 1) x += __shfl_xor(x, o);
  return x;
}
__device__ __forceinline__ uint64_t wave_incl_scan_u64(uint64_t x) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint64_t y = __shfl_up((unsigned long long)x, o);
    x += lane >= o ? y : 0;
  }
  return x;
}
__device__ __forceinline__ float wave_max_f32(float x) {
  return __uint_as_float(order_key_inv(wave_max_u32(order_key(x))));
}
__device__ __forceinline__ uint64_t rl64(uint64_t x, int lane) {
  return (uint64_t)rl((uint32_t)(x >> 32), lane) << 32 | rl((uint32_t)x, lane);
}

// ---------------------------------------------------------------- the stream

// The tile's columns of a lane: 16-byte chunks, neighbouring lanes on
// neighbouring chunks.
template <typename T>
__device__ __forceinline__ int tile_col(int tile, int i) {
  constexpr int EP = Elems<T>::n;
  return tile * kTile + ((i / EP) * kWave + (int)(threadIdx.x & 63)) * EP + i % EP;
}
template <typename T>
__device__ __forceinline__ void load_tile(const Args& a, int64_t row, int tile, float (&v)[kPer]) {
  constexpr int EP = Elems<T>::n;
  const T* x = static_cast<const T*>(a.x) + row * a.ld;
#pragma unroll
  for (int i = 0; i < kPer; i += EP) {
    const int col = tile_col<T>(tile, i);
    if (col + EP <= a.n) {
      const u32x4 w = load16_any(x + col);
#pragma unroll
      for (int e = 0; e < EP; ++e) v[i + e] = tame(Elems<T>::get(w, e));
    } else {
#pragma unroll
      for (int e = 0; e < EP; ++e) v[i + e] = col + e < a.n ? tame(Elems<T>::one(x + col + e)) : neg_inf();
    }
  }
  if (a.idx) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int col = tile_col<T>(tile, i);
      if (col < a.n && a.idx[row * a.n + col] < 0) v[i] = neg_inf();
    }
  }
}

template <typename T, bool VERIFY>
__global__ void __launch_bounds__(kThreads) sample_tiles_kernel(Args a) {
  constexpr int EP = Elems<T>::n, CH = kPer / EP;   // chunks of a lane: one per group of 64 * EP columns
  const int64_t w = (int64_t)blockIdx.x * kWaves + wave_id();
  const int64_t row = w / a.tiles;
  if (row >= a.rows) return;
  const int tile = (int)(w % a.tiles), lane = threadIdx.x & 63;
  const int64_t seq = row / a.per;
  if constexpr (VERIFY) {
    const int j = (int)(row % a.per);
    if (j == 0 && tile == 0 && lane == 0) a.arrived[seq] = 0;
    if (a.length && j > max(a.length[seq], 0)) return;   // no such position
  }
  float v[kPer];
  load_tile<T>(a, row, tile, v);
  // chunk by chunk the maxima of rows of 16 lanes; lane i of a row keeps chunk i's
  float t = neg_inf();
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    float m = v[i * EP];
#pragma unroll
    for (int e = 1; e < EP; ++e) m = fmaxf(m, v[i * EP + e]);
    m = fmaxf(m, dpp<0xB1>(m));
    m = fmaxf(m, dpp<0x4E>(m));
    m = fmaxf(m, dpp<0x141>(m));
    m = fmaxf(m, dpp<0x140>(m));
    t = (lane & 15) == i ? m : t;
  }
  t = fmaxf(t, __shfl_xor(t, 16));
  float* g = a.gmax + (row * a.tiles + tile) * kGroups;
  if constexpr (EP == 4) {   // a chunk is a group
    t = fmaxf(t, __shfl_xor(t, 32));
    if (lane < kGroups) g[lane] = t;
  } else {                   // a chunk is two groups, of 32 lanes each
    if ((lane & 31) < CH) g[(lane & 31) * 2 + (lane >> 5)] = t;
  }
  const float m = wave_max_f32(t);
  if (lane == 0) a.tmax[row * a.tiles + tile] = m;
  const How h = how_of(a, seq);
  if (!h.mass()) return;
  double s = 0.0;
  if (m > neg_inf()) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const double e = exp2_f64(log_weight(fmaxf(v[i], -__FLT_MAX__), m, h.c));
      s += v[i] > neg_inf() ? e : 0.0;
    }
    s = wave_sum_f64(s);
  }
  if (lane == 0) a.tsum[row * a.tiles + tile] = s;
}

// ------------------------------------------------------------------- a row

// The order of a row's columns: cand_key of logit and column, larger first.
__device__ __forceinline__ uint64_t key_of(float x, int col) { return x > neg_inf() ? cand_key(x, col) : 0; }

// What a drafted list takes from the weights of its tokens: q of them.
struct Less {
  const int32_t* id;   // LDS
  const float* q;
  int k;               // 0: nothing
  double mass;         // the kept mass of the target row
  __device__ __forceinline__ double of(int col) const {
    double s = 0.0;
    for (int j = 0; j < k; ++j) s += id[j] == col ? (double)q[j] : 0.0;
    return s;
  }
  __device__ __forceinline__ uint64_t rest(uint64_t w, int col) const {
    if (!k || !w) return w;
    const double s = of(col);
    if (!(s > 0.0)) return w;
    const uint64_t gone = (uint64_t)rint(fmin(s * mass, 9e18));
    return w > gone ? w - gone : 0;
  }
};

// One wave, a column per lane: what is kept of the keys.
struct Kept {
  uint64_t w;       // the lane's weight, 0 where it is not kept
  uint64_t mass;    // of all kept
};
// n: lanes that hold keys. all: the row's mass if top_p goes by it (no
// top_k), else 0.
__device__ __forceinline__ Kept wave_keep(uint64_t key, float m, const How& h, int bits, int n, uint64_t all) {
  const double t = log_weight(key ? key_score(key) : m, m, h.c);
  uint64_t w = key ? to_int(exp2_f64(t), bits) : 0;
  bool in = key != 0;
  if (h.top_k || h.top_p < 1.0) {
    int rank = 0;
    uint64_t before = 0;
    for (int j = 0; j < n; ++j) {
      const uint64_t kj = rl64(key, j), wj = rl64(w, j);
      if (kj > key) {
        ++rank;
        before += wj;
      }
    }
    if (h.top_k) in = in && rank < h.top_k;
    if (h.top_p < 1.0) {
      const uint64_t mass = all ? all : wave_sum_u64(in ? w : 0);
      in = in && before < share_of(mass, h.top_p);
    }
  }
  in = in && t >= h.least;
  Kept k;
  k.w = in ? w : 0;
  k.mass = wave_sum_u64(k.w);
  return k;
}
// The lane whose column holds u's place in the mass (> 0), columns in the
// order of col.
__device__ __forceinline__ int wave_draw(uint64_t w, uint64_t mass, int col, float u, int n) {
  const uint64_t at = place_of(mass, u);
  uint64_t before = 0;
  for (int j = 0; j < n; ++j) {
    const uint64_t wj = rl64(w, j);
    const int cj = (int)rl((uint32_t)col, j);
    if (cj < col) before += wj;
  }
  const unsigned long long hit = __ballot(before <= at && at - before < w);
  return __ffsll(hit) - 1;
}

// Rows of at most 64 columns: a wave per row, a lane per column.
template <typename T>
__global__ void __launch_bounds__(kThreads) sample_lists_kernel(Args a) {
  const int64_t row = (int64_t)blockIdx.x * kWaves + wave_id();
  if (row >= a.rows) return;
  const int lane = threadIdx.x & 63;
  const How h = how_of(a, row);
  float x = lane < a.n ? tame(Elems<T>::one(static_cast<const T*>(a.x) + row * a.ld + lane)) : neg_inf();
  int id = lane;
  if (a.idx && lane < a.n) {
    id = a.idx[row * a.n + lane];
    if (id < 0) x = neg_inf();
  }
  const float m = wave_max_f32(x);
  const bool none = !(m > neg_inf());
  Kept k = wave_keep(key_of(x, lane), none ? 0.f : m, h, a.bits, a.n, 0);
  if (none) k.w = 0;
  if (a.probs && lane < a.n) a.probs[row * a.n + lane] = none ? 0.f : (float)((double)k.w / (double)k.mass);
  if (none) {
    if (lane == 0) {
      a.token[row] = -1;
      if (a.prob) a.prob[row] = 0.f;
    }
    return;
  }
  const int at = wave_draw(k.w, k.mass, lane, a.u[row * a.u_ld], a.n);
  if (lane == at) {
    a.token[row] = id;
    if (a.prob) a.prob[row] = (float)((double)k.w / (double)k.mass);
  }
}

struct Lds {
  uint64_t mass[kBins];
  uint32_t count[kBins];
  uint64_t list[kList];
  uint64_t few[kWave];
  uint64_t sum[kRowWaves + 2];
  uint64_t out[4];
  int ask[kAskGroups];
  int n_ask, n_list, n_few, pick;
  int32_t id[64];
  float q[64];
  int tile[64];             // of the list's tokens, and what they take from it
  uint64_t gone[64];
};

__device__ __forceinline__ uint64_t block_sum(uint64_t x, Lds& s) {
  x = wave_sum_u64(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s.sum[wave_id()] = x;
  __syncthreads();
  uint64_t all = 0;
#pragma unroll
  for (int w = 0; w < kRowWaves; ++w) all += s.sum[w];
  return all;
}
// Exclusive prefix over the threads; all: the total.
__device__ __forceinline__ uint64_t block_scan(uint64_t x, uint64_t& all, Lds& s) {
  const uint64_t incl = wave_incl_scan_u64(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) s.sum[wave_id()] = incl;
  __syncthreads();
  uint64_t before = incl - x;
  all = 0;
  const int wave = wave_id();
#pragma unroll
  for (int w = 0; w < kRowWaves; ++w) {
    if (w < wave) before += s.sum[w];
    all += s.sum[w];
  }
  return before;
}

// Of elements (key, weight) the last, in descending order of distinct keys
// from hi to lo, before which less than `target` (> 0) weight lies.
// each(lo, hi, f) calls f(key, weight) for the calling thread's elements with
// a weight above 0 in [lo, hi]; at least one there is. Halves the range of keys
// by 2^11 a step until at most `most` elements are left; these are put into
// `list` and n is their number (0: the element was found, its key is lo).
struct Range {
  uint64_t lo, hi, target;
  int n;
};
template <typename Each>
__device__ __forceinline__ Range block_narrow(const Each& each, Range r, int most, uint64_t* list, int* n_list, Lds& s) {
  const int tid = threadIdx.x;
  for (;;) {
    const uint64_t span = r.hi - r.lo;
    if (!span) {
      r.n = 0;
      return r;
    }
    const int shift = max(0, 64 - __clzll((long long)span) - 11);
    __syncthreads();
    for (int i = tid; i < kBins; i += kRowThreads) {
      s.mass[i] = 0;
      s.count[i] = 0;
    }
    if (tid == 0) s.pick = -1;
    __syncthreads();
    each(r.lo, r.hi, [&](uint64_t key, uint64_t w) {
      const int bin = (int)((r.hi - key) >> shift);
      atomicAdd(reinterpret_cast<unsigned long long*>(&s.mass[bin]), (unsigned long long)w);
      atomicAdd(&s.count[bin], 1u);
    });
    __syncthreads();
    uint64_t w[kBinsPer], mine = 0, all;
    uint32_t c[kBinsPer];
#pragma unroll
    for (int i = 0; i < kBinsPer; ++i) {
      w[i] = s.mass[tid * kBinsPer + i];
      c[i] = s.count[tid * kBinsPer + i];
      mine += w[i];
    }
    uint64_t before = block_scan(mine, all, s);
    int last = -1;
    uint64_t last_before = 0;
    uint32_t last_count = 0;
#pragma unroll
    for (int i = 0; i < kBinsPer; ++i) {
      if (c[i] && before < r.target) {
        last = tid * kBinsPer + i;
        last_before = before;
        last_count = c[i];
      }
      before += w[i];
    }
    if (last >= 0) atomicMax(&s.pick, last);
    __syncthreads();
    if (last >= 0 && s.pick == last) {
      s.out[0] = last_before;
      s.out[1] = last_count;
    }
    __syncthreads();
    if (s.pick < 0) {   // no element: not by any call here
      r.lo = r.hi;
      r.n = 0;
      return r;
    }
    const uint64_t top = r.hi - ((uint64_t)s.pick << shift);
    const uint64_t width = (1ull << shift) - 1;
    r.lo = top - r.lo > width ? top - width : r.lo;
    r.hi = top;
    r.target -= s.out[0];
    const int n = (int)s.out[1];
    if (n <= most) {
      if (tid == 0) *n_list = 0;
      __syncthreads();
      each(r.lo, r.hi, [&](uint64_t key, uint64_t) {
        const int at = atomicAdd(n_list, 1);
        if (at < most) list[at] = key;
      });
      __syncthreads();
      r.n = n;
      return r;
    }
  }
}
// The element itself, of keys in LDS.
template <typename Each, typename Weight>
__device__ __forceinline__ uint64_t block_find(const Each& each, const Weight& weight, Range r, Lds& s) {
  r = block_narrow(each, r, kWave, s.few, &s.n_few, s);
  if (!r.n) return r.lo;
  if (wave_id() == 0) {
    const int lane = threadIdx.x & 63;
    const uint64_t key = lane < r.n ? s.few[lane] : 0;
    const uint64_t w = key ? weight(key) : 0;
    uint64_t before = 0;
    int rank = 0;
    for (int j = 0; j < r.n; ++j) {
      const uint64_t kj = rl64(key, j), wj = rl64(w, j);
      if (kj > key) {
        before += wj;
        ++rank;
      }
    }
    const int kept = wave_count(key && before < r.target);
    if (key && rank == kept - 1) s.out[2] = key;
  }
  __syncthreads();
  return s.out[2];
}

// A bound that at least k of the groups' maxima reach, as an order key: lane
// by lane every 64th group (the largest of several where there are more than
// 64 * kHeld). 0 where there are not so many. Every wave finds the same.
constexpr int kHeld = 16;
__device__ __forceinline__ uint32_t group_bound(const float* gmax, int groups, int k) {
  const int lane = threadIdx.x & 63;
  uint32_t v[kHeld];
  uint32_t lo = ~0u, hi = 0;
#pragma unroll
  for (int e = 0; e < kHeld; ++e) v[e] = 0;
  for (int g0 = 0; g0 < groups; g0 += kWave * kHeld) {
#pragma unroll
    for (int e = 0; e < kHeld; ++e) {
      const int g = g0 + e * kWave + lane;
      const float x = g < groups ? gmax[g] : neg_inf();
      if (x > neg_inf()) v[e] = max(v[e], order_key(x));
    }
  }
  int have = 0;
#pragma unroll
  for (int e = 0; e < kHeld; ++e) {
    have += wave_count(v[e] != 0);
    hi = max(hi, v[e]);
    if (v[e]) lo = min(lo, v[e]);
  }
  if (have < k) return 0;
  lo = wave_min_u32(lo);
  hi = wave_max_u32(hi);
  while (lo < hi) {   // count(>= lo) >= k
    const uint32_t mid = lo + (hi - lo + 1) / 2;
    int c = 0;
#pragma unroll
    for (int e = 0; e < kHeld; ++e) c += wave_count(v[e] >= mid);
    if (c >= k) {
      lo = mid;
      if (c <= k + k / 4) break;
    } else {
      hi = mid - 1;
    }
  }
  return lo;
}

template <typename T>
struct RowCtx {
  const Args& a;
  Lds& s;
  int64_t row;
  How h;
  float m;
  uint64_t thr;     // kept: keys from here on, of weight h.least at least
  uint64_t mass;    // kept, in all

  __device__ __forceinline__ float at(int col) const {
    if (a.idx && a.idx[row * a.n + col] < 0) return neg_inf();
    return tame(Elems<T>::one(static_cast<const T*>(a.x) + row * a.ld + col));
  }
  __device__ __forceinline__ uint64_t key_at(int col) const { return key_of(at(col), col); }
  __device__ __forceinline__ uint64_t weight(uint64_t key) const { return int_weight(key_score(key), m, h.c, a.bits); }
  // the kept weight, 0 of what is not kept
  __device__ __forceinline__ uint64_t kept(uint64_t key) const {
    if (!key || key < thr) return 0;
    const double t = log_weight(key_score(key), m, h.c);
    return t >= h.least ? to_int(exp2_f64(t), a.bits) : 0;
  }

  // f(key) for all columns, a tile a wave
  template <typename F>
  __device__ __forceinline__ void each_col(const F& f) const {
    for (int tile = wave_id(); tile < a.tiles; tile += kRowWaves) {
      float v[kPer];
      load_tile<T>(a, row, tile, v);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (v[i] > neg_inf()) f(cand_key(v[i], tile_col<T>(tile, i)));
      }
    }
  }

  // LDS list of the columns that reach the bound, as keys; its length may be
  // above kList, then the list is not whole.
  __device__ __forceinline__ int gather(uint32_t bound) {
    const int groups = a.tiles * kGroups;
    const float* gmax = a.gmax + row * groups;
    const float least = bound ? __uint_as_float(order_key_inv(bound)) : -__FLT_MAX__;
    const int tid = threadIdx.x, lane = tid & 63;
    __syncthreads();
    if (tid == 0) s.n_list = 0;
    for (int g0 = 0; g0 < groups; g0 += kAskGroups) {
      __syncthreads();
      if (tid == 0) s.n_ask = 0;
      __syncthreads();
      for (int g = g0 + tid; g < min(groups, g0 + kAskGroups); g += kRowThreads)
        if (gmax[g] >= least) s.ask[atomicAdd(&s.n_ask, 1)] = g;
      __syncthreads();
      const int n = s.n_ask;
      for (int i = wave_id(); i < n; i += kRowWaves) {
        const int c0 = s.ask[i] * kGroup + lane;
        float v[kGroup / kWave];
#pragma unroll
        for (int j = 0; j < kGroup / kWave; ++j) v[j] = c0 + j * kWave < a.n ? at(c0 + j * kWave) : neg_inf();
#pragma unroll
        for (int j = 0; j < kGroup / kWave; ++j) {
          if (v[j] >= least) {
            const int p = atomicAdd(&s.n_list, 1);
            if (p < kList) s.list[p] = cand_key(v[j], c0 + j * kWave);
          }
        }
      }
    }
    __syncthreads();
    return s.n_list;
  }

  // thr and mass of the list, which holds all that may be kept. all: the
  // row's mass for top_p without top_k.
  __device__ __forceinline__ void keep_list(int n, uint32_t bound, uint64_t all) {
    const auto ones = [&](uint64_t lo, uint64_t hi, auto f) {
      for (int i = threadIdx.x; i < n; i += kRowThreads) {
        const uint64_t k = s.list[i];
        if (k >= lo && k <= hi) f(k, (uint64_t)1);
      }
    };
    const auto weights = [&](uint64_t lo, uint64_t hi, auto f) {
      for (int i = threadIdx.x; i < n; i += kRowThreads) {
        const uint64_t k = s.list[i];
        if (k >= lo && k <= hi) {
          const uint64_t w = weight(k);
          if (w) f(k, w);
        }
      }
    };
    const uint64_t hi = cand_key(m, 0);
    thr = max((uint64_t)bound << 32, (uint64_t)1);
    if (h.top_k && n > h.top_k)
      thr = block_find(ones, [](uint64_t) { return (uint64_t)1; }, Range{thr, hi, (uint64_t)h.top_k, 0}, s);
    if (h.top_p < 1.0) {
      if (!all) {
        uint64_t mine = 0;
        weights(thr, hi, [&](uint64_t, uint64_t w) { mine += w; });
        all = block_sum(mine, s);
      }
      const uint64_t p = block_find(weights, [&](uint64_t k) { return weight(k); },
                                    Range{thr, hi, share_of(all, h.top_p), 0}, s);
      thr = max(thr, p);
    }
    uint64_t mine = 0;
    for (int i = threadIdx.x; i < n; i += kRowThreads) mine += kept(s.list[i]);
    mass = block_sum(mine, s);
  }
  __device__ __forceinline__ int draw_list(int n, float u, Less less) {
    const auto weights = [&](uint64_t lo, uint64_t hi, auto f) {
      for (int i = threadIdx.x; i < n; i += kRowThreads) {
        const uint64_t k = (uint32_t)s.list[i];   // lower columns are larger
        if (k >= lo && k <= hi) {
          const uint64_t w = less.rest(kept(s.list[i]), key_id(s.list[i]));
          if (w) f(k, w);
        }
      }
    };
    uint64_t total = mass;
    if (less.k) {
      uint64_t mine = 0;
      weights(0, ~0ull, [&](uint64_t, uint64_t w) { mine += w; });
      total = block_sum(mine, s);
      if (!total) {
        less.k = 0;
        total = mass;
      }
    }
    const uint64_t k = block_find(weights, [&](uint64_t low) {
      const int col = (int)(0xFFFFFFFFu - (uint32_t)low);
      return less.rest(kept(key_at(col)), col);
    }, Range{0xFFFFFFFFu - (uint32_t)(a.n - 1), 0xFFFFFFFFu, place_of(total, u) + 1, 0}, s);
    return (int)(0xFFFFFFFFu - (uint32_t)k);
  }

  // The row as a whole: thr, mass, and the tiles' kept masses.
  __device__ __forceinline__ void keep_row(uint64_t all) {
    const uint64_t hi = cand_key(m, 0);
    const auto ones = [&](uint64_t lo, uint64_t up, auto f) {
      each_col([&](uint64_t k) {
        if (k >= lo && k <= up) f(k, (uint64_t)1);
      });
    };
    const auto weights = [&](uint64_t lo, uint64_t up, auto f) {
      each_col([&](uint64_t k) {
        if (k >= lo && k <= up) {
          const uint64_t w = weight(k);
          if (w) f(k, w);
        }
      });
    };
    int n = 0;
    const auto list_ones = [&](uint64_t lo, uint64_t up, auto f) {
      for (int i = threadIdx.x; i < n; i += kRowThreads)
        if (s.list[i] >= lo && s.list[i] <= up) f(s.list[i], (uint64_t)1);
    };
    const auto list_weights = [&](uint64_t lo, uint64_t up, auto f) {
      for (int i = threadIdx.x; i < n; i += kRowThreads)
        if (s.list[i] >= lo && s.list[i] <= up) f(s.list[i], weight(s.list[i]));
    };
    thr = 1;
    if (h.top_k) {
      const Range r = block_narrow(ones, Range{1, hi, (uint64_t)h.top_k, 0}, kList, s.list, &s.n_list, s);
      n = r.n;
      thr = n ? block_find(list_ones, [](uint64_t) { return (uint64_t)1; }, r, s) : r.lo;
    }
    if (h.top_p < 1.0) {
      if (!all) {
        uint64_t mine = 0;
        weights(thr, hi, [&](uint64_t, uint64_t w) { mine += w; });
        all = block_sum(mine, s);
      }
      const Range r = block_narrow(weights, Range{thr, hi, share_of(all, h.top_p), 0}, kList, s.list, &s.n_list, s);
      n = r.n;
      thr = max(thr, n ? block_find(list_weights, [&](uint64_t k) { return weight(k); }, r, s) : r.lo);
    }
    uint64_t* sums = reinterpret_cast<uint64_t*>(a.tsum) + row * a.tiles;
    uint64_t mine = 0;
    for (int tile = wave_id(); tile < a.tiles; tile += kRowWaves) {
      float v[kPer];
      load_tile<T>(a, row, tile, v);
      uint64_t w = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) w += kept(key_of(v[i], tile_col<T>(tile, i)));
      w = wave_sum_u64(w);
      if ((threadIdx.x & 63) == 0) {
        sums[tile] = w;
        mine += w;
      }
    }
    mass = block_sum(mine, s);
  }

  // A tile's kept mass: an integer (keep_row), or of the sum relative to the tile's maximum.
  __device__ __forceinline__ uint64_t tile_mass(int tile, bool ints) const {
    const int64_t i = row * a.tiles + tile;
    if (ints) return reinterpret_cast<const uint64_t*>(a.tsum)[i];
    const float t = a.tmax[i];
    if (!(t > neg_inf())) return 0;
    return (uint64_t)rint(a.tsum[i] * exp2_f64(log_weight(t, m, h.c)) * (double)(1ull << a.bits));
  }

  // The draw over the tiles' masses, then inside the tile. The masses may be
  // off by roundings; whatever they say, a column of weight 0 is never drawn.
  __device__ __forceinline__ int draw_tiles(bool ints, float u, Less less) {
    const int tid = threadIdx.x;
    const int each = (a.tiles + kRowThreads - 1) / kRowThreads;
    for (;;) {
      if (less.k) {   // what the list takes from its tokens' tiles
        __syncthreads();
        if (tid < less.k) {
          const int col = less.id[tid];
          bool first = col >= 0 && col < a.n;
          for (int j = 0; j < tid && first; ++j) first = less.id[j] != col;
          uint64_t w = 0;
          if (first) {
            w = kept(key_at(col));
            w -= less.rest(w, col);
          }
          s.tile[tid] = first ? col / kTile : -1;
          s.gone[tid] = w;
        }
        __syncthreads();
      }
      uint64_t mine = 0, total;
      const auto mass_of = [&](int tile) {
        uint64_t w = tile_mass(tile, ints), gone = 0;
        for (int j = 0; j < less.k; ++j) gone += s.tile[j] == tile ? s.gone[j] : 0;
        return w > gone ? w - gone : 0;
      };
      for (int i = 0; i < each; ++i) {
        const int tile = tid * each + i;
        if (tile < a.tiles) mine += mass_of(tile);
      }
      const uint64_t before = block_scan(mine, total, s);
      if (total) {
        const uint64_t at = place_of(total, u);
        if (before <= at && at - before < mine) {
          uint64_t b = before;
          for (int i = 0; i < each; ++i) {
            const int tile = tid * each + i;
            const uint64_t w = tile < a.tiles ? mass_of(tile) : 0;
            if (b <= at && at - b < w) {
              s.pick = tile;
              s.out[0] = at - b;
            }
            b += w;
          }
        }
        __syncthreads();
        uint64_t left = s.out[0];
        for (int tile = s.pick; tile < a.tiles; ++tile) {
          const int col = in_tile(tile, left, less, false);
          if (col >= 0) return col;
        }
      }
      // a place behind all of them: the last column with weight
      uint64_t none = 0;
      for (int tile = a.tiles - 1; tile >= 0; --tile) {
        const int col = in_tile(tile, none, less, true);
        if (col >= 0) return col;
      }
      if (!less.k) return -1;   // only of a row without candidates
      less.k = 0;               // the list covers the target: the target itself
    }
  }
  // The column of a tile that holds place `left`, which otherwise goes down
  // by the tile's mass; or the last column with weight; -1 if none.
  __device__ __forceinline__ int in_tile(int tile, uint64_t& left, const Less& less, bool last) {
    constexpr int kEach = kTile / kRowThreads;
    const int tid = threadIdx.x;
    uint64_t w[kEach], mine = 0, total;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int col = tile * kTile + tid * kEach + e;
      w[e] = 0;
      if (col < a.n) {
        w[e] = less.rest(kept(key_at(col)), col);
      }
      mine += w[e];
    }
    const uint64_t before = block_scan(mine, total, s);
    if (!total) return -1;
    if (last) left = total - 1;
    if (left >= total) {
      left -= total;
      return -1;
    }
    __syncthreads();
    if (before <= left && left - before < mine) {
      uint64_t b = before;
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        if (b <= left && left - b < w[e]) s.pick = tile * kTile + tid * kEach + e;
        b += w[e];
      }
    }
    __syncthreads();
    return s.pick;
  }
};

// The last of a sequence's blocks writes its tokens: the accepted ones, the
// one drawn behind them, and -1.
__device__ __forceinline__ void finish_sequence(const Args& a, int64_t seq, int drafted, Lds& s) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s.pick = __hip_atomic_fetch_add(&a.arrived[seq], 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)drafted;
  }
  __syncthreads();
  if (!s.pick || wave_id() != 0) return;
  __threadfence();
  const int lane = threadIdx.x & 63;
  const int32_t* state = a.state + seq * a.per;
  int taken = drafted;
  for (int j0 = 0; j0 <= drafted; j0 += kWave) {
    const int j = j0 + lane;
    const bool stop = j <= drafted &&
                      __hip_atomic_load(&state[j], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != kAccepted;
    const unsigned long long m = __ballot(stop);
    if (m) {
      taken = j0 + __ffsll(m) - 1;
      break;
    }
  }
  const int drawn = __hip_atomic_load(&state[taken], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (int j = lane; j < a.per; j += kWave)
    a.token[seq * a.per + j] = j < taken ? a.drafted[seq * (a.per - 1) + j] : j == taken ? drawn : -1;
  if (lane == 0) a.count[seq] = taken + (drawn >= 0);
}

template <typename T, bool VERIFY>
__global__ void __launch_bounds__(kRowThreads) sample_rows_kernel(Args a) {
  __shared__ Lds s;
  const int64_t row = blockIdx.x;
  const int64_t seq = row / a.per;
  const int j = (int)(row % a.per), tid = threadIdx.x, lane = tid & 63;
  int drafted = a.per - 1;
  if constexpr (VERIFY) {
    if (a.length) drafted = min(max(a.length[seq], 0), a.per - 1);
    if (j > drafted) return;
  }
  RowCtx<T> r{a, s, row, how_of(a, seq), neg_inf(), 1, 0};
  const How& h = r.h;

  // the row's maximum and mass
  float m = neg_inf();
  for (int t = tid; t < a.tiles; t += kRowThreads) m = fmaxf(m, a.tmax[row * a.tiles + t]);
  m = wave_max_f32(m);
  if (lane == 0) s.sum[wave_id()] = __float_as_uint(m);
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kRowWaves; ++w) m = fmaxf(m, __uint_as_float((uint32_t)s.sum[w]));
  __syncthreads();
  const bool none = !(m > neg_inf());
  r.m = m;

  // the list of a drafted position
  Less less{s.id, s.q, 0, 0.0};
  int x = -1;
  float ux = 0.f;
  double qx = 0.0;
  const bool check = VERIFY && j < drafted;
  if constexpr (VERIFY) {
    if (check) {
      const int64_t at = seq * (a.per - 1) + j;
      x = a.drafted[at];
      ux = a.u[seq * a.u_ld + j];
      less.k = a.list ? a.k : 1;
      if (tid < less.k) {
        s.id[tid] = a.list ? a.list[at * a.k + tid] : x;
        s.q[tid] = a.list ? fmaxf(a.q[at * a.k + tid], 0.f) : 1.f;
      }
      __syncthreads();
      qx = less.of(x);
    }
  }
  const float u = a.u[seq * a.u_ld + (VERIFY ? a.per - 1 : 0)];

  // what is kept: by one wave's lanes (way 0), by a list (1), by tiles (2: as
  // read, 3: as integers)
  int way = 2, n = 0;
  uint32_t bound = 0;
  uint64_t all = 0;
  if (!none) {
    if (h.mass()) {
      uint64_t mine = 0;
      for (int t = tid; t < a.tiles; t += kRowThreads) mine += r.tile_mass(t, false);
      all = block_sum(mine, s);
    }
    if (h.whole()) {
      r.mass = all;
    } else {
      way = 3;
      // least logit that min_p can leave in, a little below
      uint32_t floor_key = 0;
      if (h.least > -__builtin_inf()) {
        const double f = (double)m + h.least / h.c;   // c = 0: -inf or NaN
        if (f > -(double)__FLT_MAX__) floor_key = order_key((float)(f - (fabs(f) + fabs((double)m)) * 1e-6));
      }
      const int groups = a.tiles * kGroups;
      for (int k = h.top_k ? h.top_k : h.top_p < 1.0 ? kFirstK : groups + 1;; k = kSecondK) {
        bound = group_bound(a.gmax + row * groups, groups, k);
        // all that can be kept is in a list that reaches down to top_k columns or to min_p
        bool enough = h.top_k || !bound || bound <= floor_key;
        if (!(h.top_k && h.top_p < 1.0)) bound = max(bound, floor_key);
        n = r.gather(bound);
        if (n > kList) break;
        if (!enough) {   // or to top_p of the mass
          uint64_t mine = 0;
          for (int i = tid; i < n; i += kRowThreads) mine += r.weight(s.list[i]);
          enough = block_sum(mine, s) >= share_of(all, h.top_p);
        }
        if (enough) {
          way = n <= kWave ? 0 : 1;
          break;
        }
        if (k >= kSecondK) break;
      }
      if (way == 1) r.keep_list(n, bound, all);
      if (way == 3) r.keep_row(all);
    }
  }

  int drawn = -1;
  bool accepted = false;
  double kept_x = 0.0;
  if (none) {
    // nothing to draw
  } else if (way == 0) {
    if (wave_id() == 0) {
      const uint64_t key = lane < n ? s.list[lane] : 0;
      Kept k = wave_keep(key, m, h, a.bits, n, all);
      const int col = key ? key_id(key) : a.n + lane;
      if (check) {
        const unsigned long long hit = __ballot(key && col == x);
        const double wx = hit ? (double)rl64(k.w, __ffsll(hit) - 1) : 0.0;
        accepted = (double)ux * qx * (double)k.mass < wx;
        less.mass = (double)k.mass;
      }
      if (!accepted) {
        uint64_t w = k.w, mass = k.mass;
        if (check) {
          const uint64_t rest = less.rest(w, col), sum = wave_sum_u64(rest);
          if (sum) {
            w = rest;
            mass = sum;
          }
        }
        const int at = wave_draw(w, mass, col, u, n);
        drawn = __builtin_amdgcn_readlane(col, at);
        kept_x = (double)rl64(k.w, at);
      }
      r.mass = k.mass;
    }
  } else {
    if (check) {
      const bool real = x >= 0 && x < a.n;
      const double wx = real ? (double)r.kept(r.key_at(x)) : 0.0;
      accepted = (double)ux * qx * (double)r.mass < wx;
      less.mass = (double)r.mass;
    }
    if (!accepted) {
      drawn = way == 1 ? r.draw_list(n, u, less) : r.draw_tiles(way == 3, u, less);
      kept_x = drawn >= 0 ? (double)r.kept(r.key_at(drawn)) : 0.0;
    }
  }
  if (tid == 0) {   // wave 0 knows in every case
    if (!VERIFY) {
      a.token[row] = drawn < 0 ? -1 : a.idx ? a.idx[row * a.n + drawn] : drawn;
      if (a.prob) a.prob[row] = drawn < 0 ? 0.f : (float)(kept_x / (double)r.mass);
    } else {
      __hip_atomic_store(&a.state[row], accepted ? kAccepted : drawn, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  if constexpr (VERIFY) finish_sequence(a, seq, drafted, s);
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Space {
  size_t gmax, tmax, tsum, state, arrived, total;
};
Space space(int64_t rows, int64_t seqs, int64_t n) {
  const size_t tiles = (size_t)rows * ceil_div(n, kTile);
  Space s{};
  s.gmax = 0;
  s.tmax = align256(tiles * kGroups * 4);
  s.tsum = s.tmax + align256(tiles * 4);
  s.state = s.tsum + align256(tiles * 8);
  s.arrived = s.state + align256((size_t)rows * 4);
  s.total = s.arrived + align256((size_t)seqs * 4);
  return s;
}

Args make_args(const SampleArgs& in, int64_t seqs, int per, void* workspace) {
  Args a{};
  a.x = in.x;
  a.ld = in.ld;
  a.idx = in.idx;
  a.u = in.u;
  a.temperature = in.temperature;
  a.top_k = in.top_k;
  a.top_p = in.top_p;
  a.min_p = in.min_p;
  a.temperature_all = in.temperature_all;
  a.top_k_all = in.top_k_all;
  a.top_p_all = in.top_p_all;
  a.min_p_all = in.min_p_all;
  a.rows = seqs * per;
  a.n = (int)in.n;
  a.tiles = (int)ceil_div(in.n, kTile);
  a.per = per;
  a.u_ld = per;
  int log = 0;
  while ((int64_t(1) << log) < in.n) ++log;
  a.bits = std::min(51, 62 - log);
  a.token = in.token;
  a.prob = in.prob;
  a.probs = in.probs;
  if (workspace) {
    const Space s = space(a.rows, seqs, in.n);
    char* ws = static_cast<char*>(workspace);
    a.gmax = reinterpret_cast<float*>(ws + s.gmax);
    a.tmax = reinterpret_cast<float*>(ws + s.tmax);
    a.tsum = reinterpret_cast<double*>(ws + s.tsum);
    a.state = reinterpret_cast<int32_t*>(ws + s.state);
    a.arrived = reinterpret_cast<uint32_t*>(ws + s.arrived);
  }
  return a;
}

template <typename T, bool VERIFY>
hipError_t launch_rows(const Args& a, hipStream_t s) {
  const dim3 tiles((unsigned)ceil_div(a.rows * a.tiles, kWaves));
  hipLaunchKernelGGL((sample_tiles_kernel<T, VERIFY>), tiles, dim3(kThreads), 0, s, a);
  hipLaunchKernelGGL((sample_rows_kernel<T, VERIFY>), dim3((unsigned)a.rows), dim3(kRowThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace

bool sample_fits(int64_t rows, int64_t n) {
  return rows <= kMostThreads / kRowThreads && ceil_div(rows * ceil_div(n, kTile), kWaves) <= kMostThreads / kThreads;
}

size_t sample_workspace_bytes(int64_t B, int64_t n) { return n <= kWave ? 256 : space(B, B, n).total; }

hipError_t launch_sample(const SampleArgs& in, int64_t B, void* workspace, hipStream_t s) {
  const Args a = make_args(in, B, 1, in.n <= kWave ? nullptr : workspace);
  if (in.n <= kWave) {
    const dim3 grid((unsigned)ceil_div(B, kWaves)), block(kThreads);
    if (in.dtype == 0) hipLaunchKernelGGL(sample_lists_kernel<uint16_t>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(sample_lists_kernel<float>, grid, block, 0, s, a);
    return hipGetLastError();
  }
  return in.dtype == 0 ? launch_rows<uint16_t, false>(a, s) : launch_rows<float, false>(a, s);
}

size_t verify_workspace_bytes(int64_t B, int s, int64_t n) { return space(B * (s + 1), B, n).total; }

hipError_t launch_verify(const SampleArgs& in, const VerifyArgs& v, int64_t B, void* workspace, hipStream_t s) {
  Args a = make_args(in, B, v.s + 1, workspace);
  a.drafted = v.drafted;
  a.list = v.list;
  a.q = v.q;
  a.k = v.k;
  a.length = v.length;
  a.count = v.count;
  return in.dtype == 0 ? launch_rows<uint16_t, true>(a, s) : launch_rows<float, true>(a, s);
}

}  // namespace lrh
