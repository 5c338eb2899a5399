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
// their order. A single weight is good to 4e-14, the stream's sums to 2e-13 (a
// shorter exponential, since they are what a large call computes most of).
//
// sample_tiles_kernel reads the logits once: a wave takes 2048 columns and
// leaves their largest logit, of each of the tile's groups of 256 columns the
// largest logit, its place and that of the next best chunk of 16 bytes, and,
// where the row's settings need the whole mass, the sum of weights.
// sample_rows_kernel has a block per row. With a bound that at least k groups'
// maxima reach, it reads again only the chunks that hold what passes the
// bound. Where that does not settle the row (flat rows under top_p, long
// top_k), it splits the whole row by value until the border is known.
// What bounds a large call is the one read of the logits and, for rows that
// need their mass, the 64-bit exponentials (half rate); a small one, the
// chain of dependent steps in a row's block. 256 rows of 151936 columns, bf16,
// tiles / rows in us: top_k 20 17 / 12, top_k 200 17 / 21, top_p 0.9 at T = 0.8
// 39 / 15, no setting 32 / 7, top_p 0.9 of noise 40 / 110, of nearly equal
// logits 39 / 395, top_k 2000 17 / 305. With the high logits side by side, of
// which a group's maximum shows one, lists are longer: 17 / 18, 17 / 24, 39 / 20.
#include <algorithm>
#include <climits>

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
constexpr int kList = 2048;                 // columns that a row's block holds in LDS
constexpr int kValueBins = 2048;            // of a whole row's logits, even in value
constexpr double kLog2e = 1.4426950408889634;
constexpr int kFirstK = 40, kSecondK = 128, kThirdK = 512;   // groups' maxima above the bounds that top_p tries
constexpr int kMostMore = 128;              // columns missing at least, or a third of the mass: none of them is worth it

// 2^t of -1000 <= t <= 0 to 4e-14: 2^f = 1 + f g(f) for |f| <= 1/2, g by
// interpolation at the Chebyshev nodes. The nearest integer comes from the
// addition of 1.5 2^52, whose low bits hold it, and goes into the exponent as
// bits: conversions and ldexp of doubles run at a quarter of an addition's
// rate. The coefficients stand in scalar registers that the compiler knows
// nothing about; otherwise it copies each into a sum's register first.
struct Exp2 {
  double c0, c1, c2, c3, c4, c5, c6, c7, c8;
  __device__ __forceinline__ Exp2()
      : c0(1.0203121063391729e-07), c1(1.3255224878668817e-06), c2(1.525268684626772e-05), c3(0.00015403455852453838),
        c4(0.0013333558179043112), c5(0.009618129159402558), c6(0.055504108664760424), c7(0.2402265069581299),
        c8(0.6931471805599453) {
    asm("" : "+v"(c0), "+s"(c1), "+s"(c2), "+s"(c3), "+s"(c4), "+s"(c5), "+s"(c6), "+s"(c7), "+s"(c8));
  }
  __device__ __forceinline__ double in_range(double t) const {
    const double big = 6755399441055744.0;
    const double r = t + big, f = t - (r - big);
    double g = fma(c0, f, c1);
    g = fma(g, f, c2);
    g = fma(g, f, c3);
    g = fma(g, f, c4);
    g = fma(g, f, c5);
    g = fma(g, f, c6);
    g = fma(g, f, c7);
    g = fma(g, f, c8);
    const uint64_t w = (uint64_t)__double_as_longlong(fma(g, f, 1.0));
    const uint32_t n = (uint32_t)__double_as_longlong(r);
    return __longlong_as_double((long long)((uint64_t)((uint32_t)(w >> 32) + (n << 20)) << 32 | (uint32_t)w));
  }
  __device__ __forceinline__ double operator()(double t) const { return in_range(fmax(t, -1000.0)); }
};

// 2^(j / 32), and 2^f = 1 + f q(f) for |f| <= 1/64 to 2e-13 with three
// multiplications: what the stream sums. (x - m) c is rounded to 1/32 by the
// addition of 1.5 2^47, and the rest formed by one fma without rounding; the
// maximum's weight is 1, without an error, so that ties have equal masses
// whatever their tile. Per column this takes 11 64-bit instructions instead of
// 16, which bound rows that need their mass (256 x 151936 bf16, no setting: 32.0
// us, and 39.2 with the polynomial of degree 9).
__constant__ const double kPow32[32] = {
    1.0, 1.0218971486541166, 1.0442737824274138, 1.0671404006768237,
    1.0905077326652577, 1.1143867425958924, 1.1387886347566916, 1.1637248587775775,
    1.189207115002721, 1.215247359980469, 1.241857812073484, 1.2690509571917332,
    1.2968395546510096, 1.3252366431597413, 1.3542555469368927, 1.383909881963832,
    1.4142135623730951, 1.4451808069770467, 1.4768261459394993, 1.5091644275934228,
    1.5422108254079407, 1.5759808451078865, 1.6104903319492543, 1.645755478153965,
    1.681792830507429, 1.718619298122478, 1.7562521603732995, 1.7947090750031072,
    1.8340080864093424, 1.8741676341103, 1.9152065613971474, 1.9571441241754002,
};
struct TileExp {
  const double* pow;   // kPow32 in LDS
  double m, c;
  double a1, a2, a3, a4;
  __device__ __forceinline__ TileExp(const double* p, double m_, double c_)
      : pow(p), m(m_), c(c_), a1(0.693147180550011), a2(0.24022650695795306), a3(0.055504434191939005),
        a4(0.009618166713972776) {
    asm("" : "+s"(a1), "+s"(a2), "+s"(a3), "+v"(a4));
  }
  __device__ __forceinline__ double operator()(float x) const {
    const double big = 211106232532992.0, d = (double)x - m;
    const double r = fma(d, c, big), f = fma(d, c, -(r - big));
    const uint32_t n = (uint32_t)__double_as_longlong(r);   // 32 (x - m) c, rounded
    const uint64_t t = (uint64_t)__double_as_longlong(pow[n & 31]);
    const double p = __longlong_as_double((long long)((t & 0xffffffffull) | (uint64_t)((uint32_t)(t >> 32) + ((n & ~31u) << 15)) << 32));
    double q = fma(a4, f, a3);
    q = fma(q, f, a2);
    q = fma(q, f, a1);
    return fma(p * f, q, p);
  }
};

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
  bool sums;                // whether a row may need its mass
  float* gmax;              // [row][tile][kGroups]
  float* gsecond;           // its largest chunk of 16 bytes apart, and the lane of that chunk
  int32_t* gat;
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

// What the kept mass before a column has to stay below: p of the mass, 1 at least.
__device__ __forceinline__ uint64_t share_of(uint64_t mass, double p) {
  return max((uint64_t)ceil(p * (double)mass), (uint64_t)1);
}
__device__ __forceinline__ float hold(float u) { return fminf(fmaxf(u, 0.f), 1.f); }   // NaN: 0
// The place of u in the mass.
__device__ __forceinline__ uint64_t place_of(uint64_t mass, float u) {
  const double t = (double)hold(u) * (double)mass;
  return min((uint64_t)t, mass - 1);
}

__device__ __forceinline__ uint64_t rl64(uint64_t x, int lane) {
  return (uint64_t)rl((uint32_t)(x >> 32), lane) << 32 | rl((uint32_t)x, lane);
}
template <int Ctrl>
__device__ __forceinline__ uint64_t dpp_u64(uint64_t x) {
  return (uint64_t)dpp_u32<Ctrl>((uint32_t)(x >> 32)) << 32 | dpp_u32<Ctrl>((uint32_t)x);
}
// Sums over a wave, in every lane: rows of 16 lanes by DPP, then the four rows.
__device__ __forceinline__ uint64_t wave_sum_u64(uint64_t x) {
  x += dpp_u64<0xB1>(x);
  x += dpp_u64<0x4E>(x);
  x += dpp_u64<0x141>(x);
  x += dpp_u64<0x140>(x);
  return (rl64(x, 0) + rl64(x, 16)) + (rl64(x, 32) + rl64(x, 48));
}
__device__ __forceinline__ double as_f64(uint64_t x) { return __longlong_as_double((long long)x); }
__device__ __forceinline__ uint64_t as_u64(double x) { return (uint64_t)__double_as_longlong(x); }
__device__ __forceinline__ double wave_sum_f64(double x) {
  x += as_f64(dpp_u64<0xB1>(as_u64(x)));
  x += as_f64(dpp_u64<0x4E>(as_u64(x)));
  x += as_f64(dpp_u64<0x141>(as_u64(x)));
  x += as_f64(dpp_u64<0x140>(as_u64(x)));
  return (as_f64(rl64(as_u64(x), 0)) + as_f64(rl64(as_u64(x), 16))) +
         (as_f64(rl64(as_u64(x), 32)) + as_f64(rl64(as_u64(x), 48)));
}
template <int Ctrl>
__device__ __forceinline__ uint64_t dpp_shr_u64(uint64_t x) {
  return (uint64_t)dpp_shr_or_0<Ctrl>((uint32_t)(x >> 32)) << 32 | dpp_shr_or_0<Ctrl>((uint32_t)x);
}
__device__ __forceinline__ uint64_t wave_incl_scan_u64(uint64_t x) {
  x += dpp_shr_u64<0x111>(x);
  x += dpp_shr_u64<0x112>(x);
  x += dpp_shr_u64<0x114>(x);
  x += dpp_shr_u64<0x118>(x);
  const int row = (threadIdx.x & 63) >> 4;
  const uint64_t r0 = rl64(x, 15), r1 = r0 + rl64(x, 31), r2 = r1 + rl64(x, 47);
  return x + (row == 0 ? 0 : row == 1 ? r0 : row == 2 ? r1 : r2);
}
__device__ __forceinline__ float wave_max_f32(float x) {
  return __uint_as_float(order_key_inv(wave_max_u32(order_key(x))));
}

// Waits until the wave's stores and atomics have reached the memory that all
// compute units see: relaxed atomics of device scope go there without a stop in
// a cache, so that this wait between two of them, and a barrier between waves,
// orders them. (A release fence would write back the whole L2: heavy rows took
// 1100 us with it.)
__device__ __forceinline__ void wait_memory() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// ---------------------------------------------------------------- the stream

// The first column that a tile's wave reads: the last tile of a row is read
// from as far back as makes it whole, without its neighbour's columns.
__device__ __forceinline__ int tile_base(const Args& a, int tile) {
  return a.n < kTile ? 0 : min(tile * kTile, a.n - kTile);
}
// A lane's columns from there: 16-byte chunks, neighbouring lanes on
// neighbouring chunks.
template <typename T>
__device__ __forceinline__ int lane_col(int i) {
  constexpr int EP = Elems<T>::n;
  return ((i / EP) * kWave + (int)(threadIdx.x & 63)) * EP + i % EP;
}
template <typename T>
__device__ __forceinline__ void load_tile(const Args& a, int64_t row, int tile, float (&v)[kPer]) {
  constexpr int EP = Elems<T>::n;
  const int base = tile_base(a, tile);
  const T* x = static_cast<const T*>(a.x) + row * a.ld + base;
  if (a.n >= kTile) {
    u32x4 w[kPer / EP];
#pragma unroll
    for (int i = 0; i < kPer / EP; ++i) w[i] = load16_any(x + lane_col<T>(i * EP));
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = tame(Elems<T>::get(w[i / EP], i % EP));
    if (base < tile * kTile) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = base + lane_col<T>(i) < tile * kTile ? neg_inf() : v[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = lane_col<T>(i) < a.n ? tame(Elems<T>::one(x + lane_col<T>(i))) : neg_inf();
  }
  if (a.idx) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int col = base + lane_col<T>(i);
      if (col < a.n && a.idx[row * a.n + col] < 0) v[i] = neg_inf();
    }
  }
}

template <typename T, bool VERIFY>
__global__ void __launch_bounds__(kThreads) sample_tiles_kernel(Args a) {
  constexpr int EP = Elems<T>::n, CH = kPer / EP;   // chunks of a lane: one per group of 64 * EP columns
  __shared__ double pow[32];
  if (a.sums) {
    if (threadIdx.x < 32) pow[threadIdx.x] = kPow32[threadIdx.x];
    __syncthreads();
  }
  const uint32_t w = blockIdx.x * kWaves + wave_id();   // below 2^26: 32-bit divisions do
  const uint32_t row32 = w / (uint32_t)a.tiles;
  const int64_t row = row32;
  if (row >= a.rows) return;
  const int tile = (int)(w - row32 * a.tiles), lane = threadIdx.x & 63;
  const int64_t seq = VERIFY ? row32 / (uint32_t)a.per : row32;
  if constexpr (VERIFY) {
    const int j = (int)(row32 - (uint32_t)seq * a.per);
    if (j == 0 && tile == 0 && lane == 0) a.arrived[seq] = 0;
    if (a.length && j > max(a.length[seq], 0)) return;   // no such position
  }
  float v[kPer];
  load_tile<T>(a, row, tile, v);
  const How h = how_of(a, seq);
  const int64_t g0 = (row * a.tiles + tile) * kGroups;
  float m;
  if (h.whole()) {   // the maximum alone
    m = v[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) m = fmaxf(m, v[i]);
    m = wave_max_f32(m);
    if (lane < kGroups) a.gmax[g0 + lane] = lane ? neg_inf() : m;
  } else {
    // of the chunks of a group the two largest maxima, over rows of 16 lanes
    // by DPP; lane i of a row keeps those of its i-th chunks, then the rows join
    float chunk[CH], t1 = neg_inf(), t2 = neg_inf();
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      float m1 = v[i * EP];
#pragma unroll
      for (int e = 1; e < EP; ++e) m1 = fmaxf(m1, v[i * EP + e]);
      chunk[i] = m1;
      float o = dpp<0xB1>(m1), m2 = fminf(m1, o);
      m1 = fmaxf(m1, o);
      o = dpp<0x4E>(m1);
      m2 = fmaxf(fmaxf(m2, dpp<0x4E>(m2)), fminf(m1, o));
      m1 = fmaxf(m1, o);
      o = dpp<0x141>(m1);
      m2 = fmaxf(fmaxf(m2, dpp<0x141>(m2)), fminf(m1, o));
      m1 = fmaxf(m1, o);
      o = dpp<0x140>(m1);
      m2 = fmaxf(fmaxf(m2, dpp<0x140>(m2)), fminf(m1, o));
      m1 = fmaxf(m1, o);
      t1 = (lane & 15) == i ? m1 : t1;
      t2 = (lane & 15) == i ? m2 : t2;
    }
    const auto join = [&](int lanes) {
      const float o1 = __shfl_xor(t1, lanes), o2 = __shfl_xor(t2, lanes);
      t2 = fmaxf(fmaxf(t2, o2), fminf(t1, o1));
      t1 = fmaxf(t1, o1);
    };
    join(16);
    int at = 0;   // the lane whose chunk has the largest
    if constexpr (EP == 4) {   // a chunk is a group
      join(32);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int l = __ffsll((unsigned long long)__ballot(chunk[i] == readlane_f(t1, i))) - 1;
        at = lane == i ? l : at;
      }
      if (lane < kGroups) {
        a.gmax[g0 + lane] = t1;
        a.gsecond[g0 + lane] = t2;
        a.gat[g0 + lane] = at;
      }
    } else {                   // a chunk is two groups, of 32 lanes each
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const unsigned long long k = __ballot(chunk[i] == (lane < 32 ? readlane_f(t1, i) : readlane_f(t1, 32 + i)));
        at = lane == i ? __ffs((int)(uint32_t)k) - 1 : lane == 32 + i ? __ffs((int)(uint32_t)(k >> 32)) + 31 : at;
      }
      if ((lane & 31) < CH) {
        const int64_t g = g0 + (lane & 31) * 2 + (lane >> 5);
        a.gmax[g] = t1;
        a.gsecond[g] = t2;
        a.gat[g] = at;
      }
    }
    m = wave_max_f32(t1);
  }
  if (lane == 0) a.tmax[row * a.tiles + tile] = m;
  if (!a.sums || !h.mass()) return;
  double s = 0.0;
  if (m > neg_inf()) {
    const float low = fmaxf((float)((double)m - 990.0 / h.c - fabs((double)m) * 1e-6), -__FLT_MAX__);
    const double t = log_weight(low, m, h.c);
    if (t >= -1000.0 && t <= -900.0) {   // what is 2^-900 of the maximum and less, -inf among it, counts as nothing
      const TileExp ex(pow, m, h.c);
#pragma unroll
      for (int i = 0; i < kPer; ++i) s += ex(fmaxf(v[i], low));
    } else {   // temperatures at which the lowest fp32 weighs something, maxima beside which 990 / c is lost
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        s += v[i] > neg_inf() ? Exp2()(log_weight(fmaxf(v[i], -__FLT_MAX__), m, h.c)) : 0.0;
    }
    s = wave_sum_f64(s);
  }
  if (lane == 0) a.tsum[row * a.tiles + tile] = s;
}

// ------------------------------------------------------------------- a row

// The order of a row's columns: cand_key of logit and column, larger first.
__device__ __forceinline__ uint64_t key_of(float x, int col) { return x > neg_inf() ? cand_key(x, col) : 0; }

// What a drafted list takes from the weights of its tokens: q of them, as
// integers, each token once.
constexpr int kMapWords = 64;
struct Less {
  const int32_t* id;     // LDS; -1: none
  const uint64_t* q;
  const uint32_t* map;   // a bit for each id, modulo 2048
  int k;                 // 0: nothing
  __device__ __forceinline__ uint64_t rest(uint64_t w, int col) const {
    if (!k || !w || !(map[col >> 5 & (kMapWords - 1)] >> (col & 31) & 1)) return w;
    uint64_t gone = 0;
#pragma unroll 4
    for (int j = 0; j < k; ++j) gone = id[j] == col ? q[j] : gone;
    return w > gone ? w - gone : 0;
  }
};

// Items of a wave's lanes in LDS: every lane reads each in turn. (The same
// loops over readlane took six times as long: 64-bit compares with scalars.)
struct Item {
  uint64_t key, w;
};
__device__ __forceinline__ void wave_sync() {   // LDS writes before it are there for the wave's lanes behind it
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}
__device__ __forceinline__ void wave_put(Item* items, uint64_t key, uint64_t w) {
  wave_sync();
  items[threadIdx.x & 63] = Item{key, w};
  wave_sync();
}
// How many of the n items have larger keys, and their weight.
__device__ __forceinline__ uint64_t wave_before(const Item* items, int n, uint64_t key, int& rank) {
  uint64_t before = 0;
  rank = 0;
#pragma unroll 4
  for (int j = 0; j < n; ++j) {
    const Item it = items[j];
    const bool first = it.key > key;
    rank += first;
    before += first ? it.w : 0;
  }
  return before;
}

// One wave, a column per lane: what is kept of the keys.
struct Kept {
  uint64_t w;       // the lane's weight, 0 where it is not kept
  uint64_t mass;    // of all kept
};
// n: lanes that hold keys. all: the row's mass if top_p goes by it (no
// top_k), else 0.
__device__ __forceinline__ Kept wave_keep(uint64_t key, float m, const How& h, int bits, int n, uint64_t all,
                                          Item* items) {
  const double t = log_weight(key ? key_score(key) : m, m, h.c);
  const uint64_t w = key ? to_int(Exp2()(t), bits) : 0;
  bool in = key != 0;
  if (h.top_k || h.top_p < 1.0) {
    wave_put(items, key, w);
    int rank;
    const uint64_t before = wave_before(items, n, key, rank);
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
// order of col; columns are distinct.
__device__ __forceinline__ int wave_draw(uint64_t w, uint64_t mass, int col, float u, int n, Item* items) {
  const uint64_t at = place_of(mass, u);
  wave_put(items, ~(uint64_t)(uint32_t)col, w);
  int rank;
  const uint64_t before = wave_before(items, n, ~(uint64_t)(uint32_t)col, rank);
  const unsigned long long hit = __ballot(before <= at && at - before < w);
  return __ffsll(hit) - 1;
}

// Rows of at most 64 columns: a wave per row, a lane per column.
template <typename T>
__global__ void __launch_bounds__(kThreads) sample_lists_kernel(Args a) {
  __shared__ Item lds[kWaves][kWave];
  const int64_t row = (int64_t)blockIdx.x * kWaves + wave_id();
  if (row >= a.rows) return;
  Item* items = lds[wave_id()];
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
  Kept k = wave_keep(key_of(x, lane), none ? 0.f : m, h, a.bits, a.n, 0, items);
  if (none) k.w = 0;
  if (a.probs && lane < a.n) a.probs[row * a.n + lane] = none ? 0.f : (float)((double)k.w / (double)k.mass);
  if (none) {
    if (lane == 0) {
      a.token[row] = -1;
      if (a.prob) a.prob[row] = 0.f;
    }
    return;
  }
  const int at = wave_draw(k.w, k.mass, lane, a.u[row * a.u_ld], a.n, items);
  if (lane == at) {
    a.token[row] = id;
    if (a.prob) a.prob[row] = (float)((double)k.w / (double)k.mass);
  }
}

// A block runs most of what follows once, from cold instruction caches, so
// that loops stay rolled and each part stands in the code once: unrolled, the
// same steps took two to four times as long (256 rows under top_k 200: 105 us).
struct Lds {
  uint64_t key[kList], w[kList];   // the list, and its weights
  uint64_t mass[kRowThreads];      // bins, all 0 between their uses
  uint32_t count[kRowThreads];
  int four[kList];                 // places of four columns to look at
  int ask[2 * kRowThreads];        // groups to read
  uint32_t set[2 * kRowThreads];   // maxima of strided sets of columns
  uint32_t held[2 * kRowThreads];  // of a row of several windows of groups, the joint maxima
  Item items[kWave];
  uint64_t sum[kRowWaves];
  uint64_t win_before[kRowWaves];
  int win_bin[kRowWaves], win_count[kRowWaves];
  uint64_t out;
  double pow[32];
  int n_ask, n_four, n_list, n_few, pick;
  int32_t id[kWave];        // a drafted list
  uint64_t q[kWave];
  uint32_t map[kMapWords];
  int tile[kWave];          // its tokens' tiles, and what they take from them
  uint64_t gone[kWave];
};

// A barrier has to lie between a call of either and the next.
__device__ __forceinline__ uint64_t block_sum(uint64_t x, Lds& s) {
  x = wave_sum_u64(x);
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
  if ((threadIdx.x & 63) == 63) s.sum[wave_id()] = incl;
  __syncthreads();
  uint64_t before = incl - x;
  all = 0;
  const int wave = wave_id();
#pragma unroll
  for (int w = 0; w < kRowWaves; ++w) {
    const uint64_t y = s.sum[w];
    before += w < wave ? y : 0;
    all += y;
  }
  return before;
}

// Part of an order of distinct 64-bit keys, larger first: those in [lo, hi],
// and how much weight may lie before the last one sought, `target` > 0 of it.
struct Range {
  uint64_t lo, hi, target;
  int n;
};
// One step towards the last key before which less than `target` weight lies:
// the range is cut into 512 bins, whose weights and counts the threads add up
// (bins_add), and becomes the bin that holds it, with n keys.
__device__ __forceinline__ int shift_of(const Range& r) { return max(0, 64 - __clzll((long long)(r.hi - r.lo)) - 9); }
__device__ __forceinline__ void bins_add(uint64_t key, uint64_t w, const Range& r, int shift, Lds& s) {
  const int bin = (int)((r.hi - key) >> shift);
  atomicAdd(reinterpret_cast<unsigned long long*>(&s.mass[bin]), (unsigned long long)w);
  atomicAdd(&s.count[bin], 1u);
}
__device__ __forceinline__ Range bins_pick(Range r, int shift, Lds& s) {
  const int tid = threadIdx.x, wave = wave_id();
  __syncthreads();
  const uint64_t w = s.mass[tid];
  const uint32_t c = s.count[tid];
  s.mass[tid] = 0;
  s.count[tid] = 0;
  if (tid == 0) s.n_few = 0;
  uint64_t all;
  const uint64_t before = block_scan(w, all, s);
  const unsigned long long in = __ballot(c && before < r.target);   // the last of these
  if ((tid & 63) == (in ? 63 - __clzll((long long)in) : 0)) {
    s.win_bin[wave] = in ? tid : -1;
    s.win_count[wave] = (int)c;
    s.win_before[wave] = before;
  }
  __syncthreads();
  int win = -1;
#pragma unroll
  for (int v = 0; v < kRowWaves; ++v) win = s.win_bin[v] >= 0 ? v : win;
  if (win < 0) {   // no key with weight: not by any call here
    r.lo = r.hi;
    r.n = 1;
    return r;
  }
  const uint64_t top = r.hi - ((uint64_t)s.win_bin[win] << shift), width = (1ull << shift) - 1;
  r.lo = top - r.lo > width ? top - width : r.lo;
  r.hi = top;
  r.target -= s.win_before[win];
  r.n = s.win_count[win];
  return r;
}

// The last key & mask of the list's n before which less than the target lies,
// by weight or, with `ones`, by count; keys of weight 0 do not count. A barrier
// has to lie between the writing of the list and this.
__device__ __forceinline__ uint64_t list_find(Range r, int n, uint64_t mask, bool ones, Lds& s) {
  const int tid = threadIdx.x, lane = tid & 63;
  do {
    if (r.lo >= r.hi) return r.lo;
    const int shift = shift_of(r);
#pragma unroll 1
    for (int i = tid; i < n; i += kRowThreads) {
      const uint64_t k = s.key[i] & mask, w = ones ? 1 : s.w[i];
      if (w && k >= r.lo && k <= r.hi) bins_add(k, w, r, shift, s);
    }
    r = bins_pick(r, shift, s);
  } while (r.n > kWave);
#pragma unroll 1
  for (int i = tid; i < n; i += kRowThreads) {
    const uint64_t k = s.key[i] & mask, w = ones ? 1 : s.w[i];
    if (w && k >= r.lo && k <= r.hi) {
      const int at = atomicAdd(&s.n_few, 1);
      if (at < kWave) s.items[at] = Item{k, w};
    }
  }
  __syncthreads();
  const int few = min(s.n_few, kWave);
  const Item it = lane < few ? s.items[lane] : Item{0, 0};
  int rank;
  const uint64_t before = wave_before(s.items, few, it.key, rank);
  const int kept = wave_count(it.w && before < r.target);
  const unsigned long long hit = __ballot(it.w && rank == kept - 1);
  return hit ? rl64(it.key, __ffsll(hit) - 1) : r.lo;
}

// A maximum as an order key: 0 without a candidate, and one key for -0 and +0, which tie.
__device__ __forceinline__ uint32_t max_key(float m) { return m > neg_inf() ? order_key(m + 0.0f) : 0; }

// The groups' maxima of a row as max_key has them, in every wave: lane by lane
// every 64th. Of more groups than kHeldGroups, the largest of
// several.
constexpr int kHeld = 16, kHeldGroups = kHeld * kWave;
struct GroupMax {
  static constexpr int kOwn = kHeld / kRowWaves;
  uint32_t v[kHeld];
  float second[kOwn];   // of the groups that are this wave's to look at: every kRowWaves-th 64
  int at[kOwn];
  __device__ __forceinline__ void load(const Args& a, int64_t row, int g0, int groups) {
    const float* gmax = a.gmax + row * groups;
    float x[kHeld];
#pragma unroll
    for (int e = 0; e < kHeld; ++e) {
      const int g = g0 + e * kWave + (threadIdx.x & 63);
      x[e] = g < groups ? gmax[g] : neg_inf();
    }
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int64_t g = row * groups + min(g0 + (i * kRowWaves + wave_id()) * kWave + (int)(threadIdx.x & 63), groups - 1);
      second[i] = a.gsecond[g];
      at[i] = a.gat[g];
    }
#pragma unroll
    for (int e = 0; e < kHeld; ++e) v[e] = max_key(x[e]);
  }
  __device__ __forceinline__ uint32_t most() const {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < kHeld; ++e) m = max(m, v[e]);
    return wave_max_u32(m);
  }
  __device__ __forceinline__ int some() const {
    int n = 0;
#pragma unroll
    for (int e = 0; e < kHeld; ++e) n += wave_count(v[e] != 0);
    return n;
  }
  // A bound that at least k of them reach, and few more. 0 where there are not so many.
  __device__ __forceinline__ uint32_t bound(int k, uint32_t hi) const {
    uint32_t lo = ~0u;
#pragma unroll
    for (int e = 0; e < kHeld; ++e) lo = min(lo, v[e] ? v[e] : ~0u);
    if (some() < k) return 0;
    lo = wave_min_u32(lo);
#pragma unroll 1
    while (lo < hi) {   // count(>= lo) >= k
      const uint32_t mid = lo + (hi - lo + 1) / 2;
      int c = 0;
#pragma unroll
      for (int e = 0; e < kHeld; ++e) c += wave_count(v[e] >= mid);
      if (c >= k) {
        lo = mid;
        if (c <= k + max(k / 4, 4)) break;
      } else {
        hi = mid - 1;
      }
    }
    return lo;
  }
};

template <typename T>
struct RowCtx {
  const Args& a;
  Lds& s;
  int64_t row;
  How h;
  float m;
  Exp2 exp2;
  uint64_t thr;     // kept: keys from here on, of weight h.least at least
  uint64_t mass;    // kept, in all
  uint64_t own;     // the mass of the tile of the thread's number, as the stream left it

  // N columns; those that are not (col out of [from, end)) are no candidates.
  // All loads are on their way before the first is looked at.
  template <int N>
  __device__ __forceinline__ void load(const int (&col)[N], int from, int end, float (&x)[N]) const {
    const T* p = static_cast<const T*>(a.x) + row * a.ld;
    T raw[N];
#pragma unroll
    for (int q = 0; q < N; ++q) raw[q] = p[min(col[q], a.n - 1)];
    int id[N];
    if (a.idx) {
#pragma unroll
      for (int q = 0; q < N; ++q) id[q] = a.idx[row * a.n + min(col[q], a.n - 1)];
    }
#pragma unroll
    for (int q = 0; q < N; ++q) {
      x[q] = tame(Elems<T>::one(&raw[q]));
      if (col[q] < from || col[q] >= end || (a.idx && id[q] < 0)) x[q] = neg_inf();
    }
  }
  __device__ __forceinline__ float at(int col) const {
    const int c[1] = {col};
    float x[1];
    load(c, 0, a.n, x);
    return x[0];
  }
  __device__ __forceinline__ uint64_t key_at(int col) const { return key_of(at(col), col); }
  __device__ __forceinline__ uint64_t weight(uint64_t key) const {
    return to_int(exp2(log_weight(key_score(key), m, h.c)), a.bits);
  }
  // the kept weight, 0 of what is not kept
  __device__ __forceinline__ uint64_t kept(uint64_t key) const {
    if (!key || key < thr) return 0;
    const double t = log_weight(key_score(key), m, h.c);
    return t >= h.least ? to_int(exp2(t), a.bits) : 0;
  }
  // Four neighbouring columns from each col[4 q] on, all of them there; no ids.
  template <int N>
  __device__ __forceinline__ void load4(const int (&col)[4 * N], float (&x)[4 * N]) const {
    struct Raw {
      T v[4];
    } raw[N];
    const T* p = static_cast<const T*>(a.x) + row * a.ld;
#pragma unroll
    for (int q = 0; q < N; ++q) __builtin_memcpy(&raw[q], p + col[4 * q], sizeof(Raw));
#pragma unroll
    for (int q = 0; q < 4 * N; ++q) x[q] = tame(Elems<T>::one(&raw[q / 4].v[q % 4]));
  }
  // f(x, col) for the calling lane's columns in a tile of its wave's; x is -inf where there is no candidate
  template <typename F>
  __device__ __forceinline__ void each_of_tile(int tile, const F& f) const {
    const int end = min(a.n, (tile + 1) * kTile), lane = threadIdx.x & 63;
#pragma unroll 1
    for (int c0 = tile * kTile; c0 < end; c0 += 8 * kWave) {
      int col[8];
      float x[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) col[q] = c0 + q / 4 * 4 * kWave + lane * 4 + q % 4;
      if (c0 + 8 * kWave <= end && !a.idx) {
        load4<2>(col, x);
      } else {
        load(col, 0, end, x);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) f(x[q], col[q]);
    }
  }

  // The bound that at least k columns reach, where there are not as many
  // groups: the row's columns in kHeldGroups strided sets, their maxima in LDS.
  __device__ __forceinline__ uint32_t fine_bound(int k, uint32_t top, bool& made) {
    const int tid = threadIdx.x, lane = tid & 63;
    if (!made) {
      made = true;
      static_assert(kHeldGroups == 2 * kRowThreads, "two sets a thread");
      float m[2] = {neg_inf(), neg_inf()};
#pragma unroll 1
      for (int c0 = tid; c0 < a.n; c0 += 4 * kHeldGroups) {
        int col[8];
        float x[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) col[q] = c0 + q * kRowThreads;
        load(col, 0, a.n, x);
#pragma unroll
        for (int q = 0; q < 8; ++q) m[q & 1] = fmaxf(m[q & 1], x[q]);
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) s.set[tid + q * kRowThreads] = max_key(m[q]);
      __syncthreads();
    }
    GroupMax g;
#pragma unroll
    for (int e = 0; e < kHeld; ++e) g.v[e] = s.set[e * kWave + lane];
    return g.bound(k, top);
  }

  // LDS list of the columns that reach the bound, as keys; its length may be
  // above kList, then the list is not whole. A group whose second chunk stays
  // below the bound has its candidates in the chunk of its maximum; the others
  // are read, a wave on eight of them at a time. That gives the places of four
  // neighbouring columns with one that reaches the bound, or nearly only
  // these, which are then looked at one by one. Of a row of several windows of
  // groups, g holds the last one afterwards.
  __device__ __forceinline__ int gather(GroupMax& g, uint32_t bound) {
    constexpr int kAtOnce = 8, kOfLast = 1 << 30, EP = Elems<T>::n;
    static_assert(kGroup == 4 * kWave, "a lane has four columns of a group");
    const int groups = a.tiles * kGroups;
    const float least = bound ? __uint_as_float(order_key_inv(bound)) : -__FLT_MAX__;
    const uint32_t key = max(bound, 1u);
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
    __syncthreads();
    if (tid == 0) {
      s.n_list = 0;
      s.n_four = a.n < kTile ? (a.n + 3) / 4 : 0;
      s.n_ask = 0;
    }
    if (a.n < kTile) {   // all of them
      s.four[tid] = tid * 4;
    } else {
#pragma unroll 1
      for (int g0 = 0; g0 < groups; g0 += kHeldGroups) {
        if (groups > kHeldGroups) g.load(a, row, g0, groups);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < GroupMax::kOwn; ++i) {
          uint32_t v = 0;   // of the wave's i-th 64 groups
#pragma unroll
          for (int e = 0; e < kHeld; ++e) v = e == i * kRowWaves + wave ? g.v[e] : v;
          if (v >= key) {
            const int grp = g0 + (i * kRowWaves + wave) * kWave + lane, tile = grp / kGroups, in = grp % kGroups;
            if (g.second[i] >= least) {
              s.ask[atomicAdd(&s.n_ask, 1)] = grp;
            } else {
              const int p = atomicAdd(&s.n_four, EP / 4);
              const int c = (tile_base(a, tile) + in / (EP / 4) * (kWave * EP) + g.at[i] * EP) |
                            (tile == a.tiles - 1 ? kOfLast : 0);
#pragma unroll
              for (int q = 0; q < EP / 4; ++q)
                if (p + q < kList) s.four[p + q] = c + 4 * q;
            }
          }
        }
        __syncthreads();
        const int n = s.n_ask;
#pragma unroll 1
        for (int i = wave * kAtOnce; i < n; i += kRowWaves * kAtOnce) {
          int c[kAtOnce * 4], flag[kAtOnce];
          float v[kAtOnce * 4];
#pragma unroll
          for (int q = 0; q < kAtOnce; ++q) {
            const int grp = s.ask[min(i + q, n - 1)];
            c[q * 4] = tile_base(a, grp / kGroups) + grp % kGroups * kGroup + lane * 4;
            flag[q] = grp / kGroups == a.tiles - 1 ? kOfLast : 0;
          }
          load4<kAtOnce>(c, v);
          uint32_t found = 0;
#pragma unroll
          for (int q = 0; q < kAtOnce; ++q) {
            const float most = fmaxf(fmaxf(v[q * 4], v[q * 4 + 1]), fmaxf(v[q * 4 + 2], v[q * 4 + 3]));
            found |= most >= least && i + q < n ? 1u << q : 0u;
          }
          if (found) {
            int p = atomicAdd(&s.n_four, __popc(found));
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) {
              if (found >> q & 1) {
                if (p < kList) s.four[p] = c[q * 4] | flag[q];
                ++p;
              }
            }
          }
        }
        if (groups > kHeldGroups) {
          __syncthreads();
          if (tid == 0) s.n_ask = 0;
        }
      }
    }
    __syncthreads();
    const int n = s.n_four;
#pragma unroll 1
    for (int i = tid; i < min(n, kList); i += kRowThreads) {
      const int c = s.four[i] & ~kOfLast;
      int col[4];
      float v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) col[q] = c + q;
      // the last tile's groups begin among its neighbour's columns, which are in the neighbour's
      load(col, s.four[i] & kOfLast ? (a.tiles - 1) * kTile : 0, a.n, v);
      int some = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) some += v[q] >= least;
      if (some) {
        int p = atomicAdd(&s.n_list, some);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (v[q] >= least) {
            if (p < kList) s.key[p] = cand_key(v[q], col[q]);
            ++p;
          }
        }
      }
    }
    __syncthreads();
    return n > kList ? kList + 1 : s.n_list;
  }
  __device__ __forceinline__ uint64_t weigh_list(int n) const {   // the calling thread's share
    uint64_t mine = 0;
#pragma unroll 1
    for (int i = threadIdx.x; i < n; i += kRowThreads) {
      const uint64_t w = weight(s.key[i]);
      s.w[i] = w;
      mine += w;
    }
    return mine;
  }

  // A tile's mass from the stream's sums, relative to the tile's maximum.
  __device__ __forceinline__ uint64_t tile_mass(float t, double sum) const {
    if (!(t > neg_inf())) return 0;
    return (uint64_t)rint(sum * exp2(log_weight(t, m, h.c)) * (double)(1ull << a.bits));
  }
  __device__ __forceinline__ uint64_t tile_mass(int tile) const {
    if (tile == (int)threadIdx.x) return own;
    return tile_mass(a.tmax[row * a.tiles + tile], a.tsum[row * a.tiles + tile]);
  }
  // A tile's kept mass as an integer, where keep_row or split_row have put it.
  __device__ __forceinline__ uint64_t* tile_ints() const {
    return reinterpret_cast<uint64_t*>(a.tsum) + row * a.tiles;
  }
  __device__ __forceinline__ uint64_t tile_int(int tile) const {
    return __hip_atomic_load(tile_ints() + tile, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }

  // Whole rows under top_p alone. What is kept has a weight of (1 - p) / n of
  // the mass at least, as all lighter columns together have less than 1 - p of
  // it. Between that and the maximum, columns are counted in bins even in
  // value, along with where in its bin each stands; that gives a bin's mass to
  // about a millionth, and so the few bins in which the border must lie. A
  // second pass sums what is above these, tile by tile, and lists what is in
  // them, which also shows whether the border is there. False where it is not,
  // where that is too much for the list, or min_p leaves more out; else thr and
  // mass are known, and the tiles' ints.
  __device__ __forceinline__ bool keep_row(uint64_t all) {
    const int tid = threadIdx.x, lane = tid & 63;
    const uint64_t share = share_of(all, h.top_p);
    const double least = log2((1.0 - h.top_p) / a.n) * 1.001;   // the mass is 1 at least
    const float f = (float)((double)kValueBins / least * -h.c);   // bins per unit of logit
    if (!(f > 0.f && f < 1e30f) || h.least > -__builtin_inf()) return false;
    const auto bin_of = [&](float x) { return (m - x) * f; };
    uint64_t* bins = s.w;   // count << 40 | places in the bin, in 2^-16
    static_assert(kValueBins == kList, "the bins stand where the list's weights will");
    __syncthreads();
    for (int i = tid; i < kValueBins; i += kRowThreads) bins[i] = 0;
    if (tid < 32) s.pow[tid] = kPow32[tid];
    if (tid == 0) {
      s.n_list = 0;
      s.pick = kValueBins - 1;
      s.n_ask = kValueBins - 1;
    }
    __syncthreads();
#pragma unroll 1
    for (int tile = wave_id(); tile < a.tiles; tile += kRowWaves)
      each_of_tile(tile, [&](float x, int) {
        const float b = bin_of(x);   // inf of -inf
        if (b < (float)kValueBins) {
          const int i = (int)b;
          atomicAdd(reinterpret_cast<unsigned long long*>(&bins[i]),
                    1ull << 40 | (unsigned long long)((b - (float)i) * 65535.f));
        }
      });
    __syncthreads();
    // the bins through which the mass, off by 2^-13 of itself either way, reaches the share
    constexpr int kEach = kValueBins / kRowThreads;
    const double step = least / kValueBins;   // log2 of weight per bin
    uint64_t w[kEach], mine = 0, total;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const uint64_t b = bins[tid * kEach + i];
      const double count = (double)(uint32_t)(b >> 40), place = (double)(b & 0xffffffffffull) * (1.0 / 65535.0);
      // 2^(step x) = 1 + y x + (y x)^2 / 2 with y = step ln 2, the square's mean as of places spread evenly
      const double y = step * 0.6931471805599453;
      w[i] = (uint64_t)((count * (1.0 + y * y * (1.0 / 6.0)) + y * place) * exp2(step * (tid * kEach + i)) *
                        (double)(1ull << a.bits));
      mine += w[i];
    }
    const uint64_t before = block_scan(mine, total, s);
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
      uint64_t through = before;
      const uint64_t at = side ? share + (share >> 13) : share - (share >> 13);
      if (through < at && through + mine >= at) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          if (through < at && through + w[i] >= at) (side ? s.n_ask : s.pick) = tid * kEach + i;
          through += w[i];
        }
      }
    }
    __syncthreads();
    const float lo = (float)s.pick, hi = (float)(s.n_ask + 1);
    const TileExp ex(s.pow, m, h.c);
    mine = 0;
#pragma unroll 1
    for (int tile = wave_id(); tile < a.tiles; tile += kRowWaves) {
      uint64_t w = 0;
      each_of_tile(tile, [&](float x, int col) {
        const float b = bin_of(x);
        const uint64_t one = to_int(ex(b < lo ? x : m), a.bits);   // no branch: in a flat row some lane takes it
        w += b < lo ? one : 0;
        if (b >= lo && b < hi) {
          const int p = atomicAdd(&s.n_list, 1);
          if (p < kList) s.key[p] = cand_key(x, col);
        }
      });
      w = wave_sum_u64(w);
      if (lane == 0) {
        __hip_atomic_store(tile_ints() + tile, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        mine += w;
      }
    }
    wait_memory();
    __syncthreads();
    const int n = s.n_list;
    const uint64_t above = block_sum(mine, s);
    if (n > kList || n < 1 || above >= share) return false;
    __syncthreads();
    const uint64_t listed = block_sum(weigh_list(n), s);
    __syncthreads();
    if (above + listed < share && hi < (float)kValueBins) return false;
    if (!listed) return false;
    thr = list_find(Range{1, cand_key(m, 0), share - above, 0}, n, ~0ull, false, s);
    mine = 0;
    for (int i = tid; i < n; i += kRowThreads) {
      const uint64_t k = s.key[i];
      if (k < thr) continue;
      mine += s.w[i];
      __hip_atomic_fetch_add(tile_ints() + key_id(k) / kTile, s.w[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    wait_memory();
    __syncthreads();
    mass = above + block_sum(mine, s);
    return true;
  }

  // Any row: the order of its keys is cut into bins until what is left of it
  // fits the list, for top_k and for top_p, then the tiles' kept masses are summed.
  __device__ __forceinline__ void split_row(uint64_t all) {
    const int tid = threadIdx.x, lane = tid & 63;
    const uint64_t hi = cand_key(m, 0);
    thr = 1;
#pragma unroll 1
    for (int stage = 0; stage < 3; ++stage) {
      // 0: top_k, 1: its mass, 2: top_p
      if (stage == 0 ? !h.top_k : !(h.top_p < 1.0) || (stage == 1 && all)) continue;
      const bool ones = stage == 0;
      Range r{thr, hi, stage == 0 ? (uint64_t)h.top_k : stage == 2 ? share_of(all, h.top_p) : 1, kList + 1};
      uint64_t mine = 0;
      do {
        const int shift = shift_of(r);
        __syncthreads();
#pragma unroll 1
        for (int tile = wave_id(); tile < a.tiles; tile += kRowWaves)
          each_of_tile(tile, [&](float x, int col) {
            const uint64_t k = key_of(x, col);   // 0 of -inf, below every range
            if (k < r.lo || k > r.hi) return;
            const uint64_t w = ones ? 1 : weight(k);
            if (stage == 1) mine += w;
            else if (w) bins_add(k, w, r, shift, s);
          });
        if (stage == 1) break;
        r = bins_pick(r, shift, s);
      } while (r.n > kList && r.lo < r.hi);
      if (stage == 1) {
        __syncthreads();
        all = block_sum(mine, s);
        continue;
      }
      __syncthreads();
      if (tid == 0) s.n_list = 0;
      __syncthreads();
#pragma unroll 1
      for (int tile = wave_id(); tile < a.tiles; tile += kRowWaves)
        each_of_tile(tile, [&](float x, int col) {
          const uint64_t k = key_of(x, col);
          if (k < r.lo || k > r.hi || (!ones && !weight(k))) return;
          const int p = atomicAdd(&s.n_list, 1);
          if (p < kList) s.key[p] = k;
        });
      __syncthreads();
      const int n = min(s.n_list, kList);
      weigh_list(n);
      __syncthreads();
      thr = max(thr, list_find(r, n, ~0ull, ones, s));
    }
    uint64_t mine = 0;
    __syncthreads();
#pragma unroll 1
    for (int tile = wave_id(); tile < a.tiles; tile += kRowWaves) {
      uint64_t w = 0;
      each_of_tile(tile, [&](float x, int col) { w += kept(key_of(x, col)); });
      w = wave_sum_u64(w);
      if (lane == 0) {
        __hip_atomic_store(tile_ints() + tile, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        mine += w;
      }
    }
    wait_memory();
    __syncthreads();
    mass = block_sum(mine, s);
  }

  // The draw over the tiles' masses (ints: those of keep_row and split_row),
  // then inside the tile. The masses may be off by roundings; whatever they
  // say, a column of weight 0 is never drawn.
  __device__ __forceinline__ int draw_tiles(bool ints, float u, Less less) {
    const int tid = threadIdx.x;
    const int each = (a.tiles + kRowThreads - 1) / kRowThreads;
    for (;;) {
      __syncthreads();
      uint64_t mine = 0, total;
      const auto mass_of = [&](int tile) {
        const uint64_t w = ints ? tile_int(tile) : tile_mass(tile);
        uint64_t gone = 0;
#pragma unroll 4
        for (int j = 0; j < less.k; ++j) gone += s.tile[j] == tile ? s.gone[j] : 0;
        return w > gone ? w - gone : 0;
      };
      uint64_t one = 0;
      for (int i = 0; i < each; ++i) {
        const int tile = tid * each + i;
        one = tile < a.tiles ? mass_of(tile) : 0;
        mine += one;
      }
      const uint64_t before = block_scan(mine, total, s);
      uint64_t left = 0;
      int tile = a.tiles;
      if (total) {
        const uint64_t at = place_of(total, u);
        if (before <= at && at - before < mine) {
          uint64_t b = before;
          for (int i = 0; i < each; ++i) {
            const int t = tid * each + i;
            const uint64_t w = each == 1 ? one : t < a.tiles ? mass_of(t) : 0;
            if (b <= at && at - b < w) {
              s.pick = t;
              s.out = at - b;
            }
            b += w;
          }
        }
        __syncthreads();
        left = s.out;
        tile = s.pick;
      }
      // forwards to the column that holds the place; from behind the last tile,
      // backwards to the last column with weight
      bool last = false;
      while (tile >= 0) {
        if (tile == a.tiles) {
          last = true;
          if (--tile < 0) break;
        }
        const int col = in_tile(tile, left, less, last);
        if (col >= 0) return col;
        tile += last ? -1 : 1;
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
    int col[kEach];
    float x[kEach];
    uint64_t w[kEach], mine = 0, total;
#pragma unroll
    for (int e = 0; e < kEach; ++e) col[e] = tile * kTile + tid * kEach + e;
    load(col, 0, a.n, x);
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      w[e] = less.rest(kept(key_of(x[e], col[e])), col[e]);
      mine += w[e];
    }
    __syncthreads();
    const uint64_t before = block_scan(mine, total, s);
    if (!total) return -1;
    if (last) left = total - 1;
    if (left >= total) {
      left -= total;
      return -1;
    }
    if (before <= left && left - before < mine) {
      uint64_t b = before;
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        if (b <= left && left - b < w[e]) s.n_ask = col[e];
        b += w[e];
      }
    }
    __syncthreads();
    return s.n_ask;
  }
};

// The last of a sequence's blocks writes its tokens: the accepted ones, the
// one drawn behind them, and -1.
__device__ __forceinline__ void finish_sequence(const Args& a, int64_t seq, int drafted, Lds& s) {
  __syncthreads();
  if (threadIdx.x == 0) {
    wait_memory();
    s.pick = __hip_atomic_fetch_add(&a.arrived[seq], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)drafted;
  }
  __syncthreads();
  if (!s.pick || wave_id() != 0) return;
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

// More rows than CUs run two to a CU, in half the registers (BLOCKS 2: 1024
// rows of 32003 columns, bf16, top_k 20: 46 -> 32 us, top_p 0.9: 53 -> 36); a
// spill then costs a lone row 0.7 to 2 us, so up to 256 rows keep them all.
constexpr int kCus = 256;

template <typename T, bool VERIFY, int BLOCKS>
__global__ void __launch_bounds__(kRowThreads, BLOCKS * kRowWaves / 4) sample_rows_kernel(Args a) {
  __shared__ Lds s;
  const int64_t row = blockIdx.x;
  const int64_t seq = VERIFY ? blockIdx.x / (uint32_t)a.per : blockIdx.x;
  const int j = VERIFY ? (int)(blockIdx.x - (uint32_t)seq * a.per) : 0, tid = threadIdx.x, lane = tid & 63;
  int drafted = a.per - 1;
  if constexpr (VERIFY) {
    if (a.length) drafted = min(max(a.length[seq], 0), a.per - 1);
    if (j > drafted) return;
  }
  s.mass[tid] = 0;
  s.count[tid] = 0;
  // the row's maximum
  const int groups = a.tiles * kGroups;
  const float u = a.u[seq * a.u_ld + (VERIFY ? a.per - 1 : 0)];
  const bool check = VERIFY && j < drafted;
  int x = -1, id = -2, list_k = 1;
  float ux = 0.f, q = 0.f;
  if constexpr (VERIFY) {
    if (check) {   // in every wave, a lane per entry of the list
      const int64_t at = seq * (a.per - 1) + j;
      x = a.drafted[at];
      ux = hold(a.u[seq * a.u_ld + j]);
      list_k = a.list ? a.k : 1;
      if (lane < list_k) {
        id = a.list ? a.list[at * a.k + lane] : x;
        q = a.list ? fmaxf(a.q[at * a.k + lane], 0.f) : 1.f;   // NaN: 0
      }
    }
  }
  const int64_t own = row * a.tiles + min(tid, a.tiles - 1);
  const float own_max = a.tmax[own];
  const double own_sum = a.tsum[own];
  GroupMax g;
  g.load(a, row, 0, groups);
  RowCtx<T> r{a, s, row, how_of(a, seq), neg_inf(), Exp2(), 1, 0, 0};
  const How& h = r.h;
#pragma unroll 1
  for (int g0 = kHeldGroups; g0 < groups; g0 += kHeldGroups) {
    GroupMax more;
    more.load(a, row, g0, groups);
#pragma unroll
    for (int e = 0; e < kHeld; ++e) g.v[e] = max(g.v[e], more.v[e]);
  }
  if (groups > kHeldGroups && wave_id() == 0) {
#pragma unroll
    for (int e = 0; e < kHeld; ++e) s.held[e * kWave + lane] = g.v[e];
  }
  const uint32_t top = g.most();
  const bool none = !top;
  const float m = none ? neg_inf() : __uint_as_float(order_key_inv(top));
  r.m = m;

  // the logits of a drafted position's token and list
  double qx = 0.0;
  float logit_x = neg_inf(), logit = neg_inf();
  if constexpr (VERIFY) {
    if (check) {
      qx = wave_sum_f64(id == x ? (double)q : 0.0);
      if (x >= 0 && x < a.n) logit_x = r.at(x);
      if (id < 0 || id >= a.n) id = -1;
      if (wave_id() == 0 && id >= 0) logit = r.at(id);
    }
  }
  Less less{s.id, s.q, s.map, 0};
  // by wave 0, when the row's kept mass is known: what its list takes
  const auto take = [&](uint64_t mass) {
    double sum = 0.0;
    bool again = false;
    s.map[lane] = 0;
#pragma unroll 1
    for (int j = 0; j < list_k; ++j) {   // an id that occurs twice counts twice, at its first place
      const bool same = (int)rl((uint32_t)id, j) == id;
      sum += same ? (double)readlane_f(q, j) : 0.0;
      again = again || (same && j < lane);
    }
    const bool real = id >= 0 && !again && sum > 0.0;
    const uint64_t gone = real ? (uint64_t)rint(fmin(sum * (double)mass, 9e18)) : 0;
    if (real) atomicOr(&s.map[id >> 5 & (kMapWords - 1)], 1u << (id & 31));
    s.id[lane] = real ? id : -1;
    s.q[lane] = gone;
    s.tile[lane] = real ? id / kTile : -1;
    s.gone[lane] = real ? min(r.kept(key_of(logit, id)), gone) : 0;
  };

  // what is kept: by one wave's lanes (way 0), by a list (1), by tiles (2: as
  // the stream left them, 3: as integers)
  int way = 2, n = 0;
  uint32_t bound = 0;
  uint64_t all = 0;
  if (!none) {
    if (h.mass()) {
      if (tid < a.tiles) r.own = r.tile_mass(own_max, own_sum);
      uint64_t mine = r.own;
#pragma unroll 1
      for (int t = tid + kRowThreads; t < a.tiles; t += kRowThreads) mine += r.tile_mass(t);
      all = block_sum(mine, s);
    }
    if (h.whole()) {
      r.mass = all;
    } else {
      way = 3;
      // least logit that min_p can leave in, a little below; the largest logit reaches it
      uint32_t floor_key = 0;
      if (h.least > -__builtin_inf()) {
        const double f = (double)m + h.least / h.c;   // c = 0: -inf or NaN
        if (f > -(double)__FLT_MAX__) floor_key = min(max_key((float)(f - (fabs(f) + fabs((double)m)) * 1e-6)), top);
      }
      int k = h.top_k ? h.top_k : h.top_p < 1.0 ? kFirstK : INT_MAX;   // of min_p alone: no bound but its own
      const int held = min(groups, kHeldGroups);
      const bool full = g.some() >= held - held / 8 - kGroups;   // but for the last tile's
      bool made = false;
#pragma unroll 1
      for (;;) {
        bound = g.bound(k, top);
        // Few groups give no bound, or a list past a wave's lanes: finer maxima
        // (256 rows of 5000 columns, bf16, top_p 0.9: 31 -> 19 us; 64 of 1000, top_k 20: 19 -> 12;
        // 1024 of 32003, top_k 200: 256 -> 71). Of mostly empty groups a list
        // may hold all candidates, and is tried first.
        const bool finer = (!bound || (k <= kWave && held < 2 * k)) && k < INT_MAX && a.n > kWave;
        if (finer && full) bound = r.fine_bound(k, top, made);
        // all that can be kept is in a list that reaches down to top_k columns or to min_p
        bool enough = h.top_k || !bound || bound <= floor_key;
        if (!(h.top_k && h.top_p < 1.0)) bound = max(bound, floor_key);
        n = r.gather(g, bound);
        if (n > kList && finer && !full && !bound) {
          bound = r.fine_bound(k, top, made);
          n = r.gather(g, bound);
          enough = enough && h.top_k;
        }
        if (n > kList) break;
        bool flat = false, few = false;
        if (n > kWave || !enough) {
          const uint64_t listed = block_sum(r.weigh_list(n), s);
          if (!enough) {   // or to top_p of the mass
            const uint64_t share = share_of(all, h.top_p);
            enough = listed >= share;
            // of a flat row longer lists do not have it either: the others weigh less than the bound
            const double more = (double)(share - min(listed, share)) / ((double)r.weight((uint64_t)bound << 32) + 1.0);
            flat = more > kMostMore || listed < share / 3 * 2;
            few = more < kFirstK;
          }
        }
        if (enough) {
          way = n <= kWave ? 0 : 1;
          break;
        }
        if (k >= kThirdK || flat) break;
        k = k == kFirstK && few ? kSecondK : kThirdK;
        if (groups > kHeldGroups) {
#pragma unroll
          for (int e = 0; e < kHeld; ++e) g.v[e] = s.held[e * kWave + lane];
        }
      }
      if (way == 3 && !(h.mass() && r.keep_row(all))) r.split_row(all);
    }
  }

  int drawn = -1;
  bool accepted = false;
  double kept_x = 0.0;
  if (none) {
    // nothing to draw
  } else if (way == 0) {
    if (wave_id() == 0) {
      const uint64_t key = lane < n ? s.key[lane] : 0;
      Kept k = wave_keep(key, m, h, a.bits, n, all, s.items);
      const int col = key ? key_id(key) : a.n + lane;
      if (check) {
        const unsigned long long hit = __ballot(key && col == x);
        const double wx = hit ? (double)rl64(k.w, __ffsll(hit) - 1) : 0.0;
        accepted = (double)ux * qx * (double)k.mass < wx;
      }
      if (!accepted) {
        uint64_t w = k.w, mass = k.mass;
        if (check) {
          take(mass);
          less.k = list_k;
          wave_sync();
          const uint64_t rest = less.rest(w, col), sum = wave_sum_u64(rest);
          if (sum) {
            w = rest;
            mass = sum;
          }
        }
        const int at = wave_draw(w, mass, col, u, n, s.items);
        if (at >= 0) {   // the largest logit has weight
          drawn = __builtin_amdgcn_readlane(col, at);
          kept_x = (double)rl64(k.w, at);
        }
      }
      r.mass = k.mass;
    }
  } else {
    // the list: top_k's border, top_p's, and the column drawn, each by
    // list_find; the tiles' borders are known. What is kept is in the list, and
    // so not below its bound, also where top_k leaves the whole list in: a
    // drafted token need not be in it.
    if (way == 1) r.thr = max(r.thr, (uint64_t)bound << 32);
#pragma unroll 1
    for (int stage = way == 1 ? 0 : 2; stage < 3; ++stage) {
      Range f{max((uint64_t)bound << 32, (uint64_t)1), cand_key(m, 0), 0, 0};
      if (stage == 0) {
        if (!h.top_k || n <= h.top_k) continue;
        f.target = h.top_k;
      } else if (stage == 1) {
        if (!(h.top_p < 1.0)) continue;
        uint64_t mine = 0;
#pragma unroll 1
        for (int i = tid; i < n; i += kRowThreads)
          if (s.key[i] >= r.thr) mine += s.w[i];
        __syncthreads();
        const uint64_t listed = block_sum(mine, s);
        f.lo = max(f.lo, r.thr);
        f.target = share_of(all ? all : listed, h.top_p);
      } else {
        if (way == 1) {
          uint64_t mine = 0;
#pragma unroll 1
          for (int i = tid; i < n; i += kRowThreads) {
            const uint64_t w = r.kept(s.key[i]);
            s.w[i] = w;
            mine += w;
          }
          __syncthreads();
          r.mass = block_sum(mine, s);
        }
        if (check) {
          accepted = (double)ux * qx * (double)r.mass < (double)r.kept(key_of(logit_x, x));
          if (accepted) break;
          if (wave_id() == 0) take(r.mass);
          less.k = list_k;
          __syncthreads();
        }
        if (way != 1) {
          drawn = r.draw_tiles(way == 3, u, less);
          break;
        }
        uint64_t total = r.mass;
        if (check) {
          uint64_t mine = 0;
#pragma unroll 1
          for (int i = tid; i < n; i += kRowThreads) {
            const uint64_t w = less.rest(s.w[i], key_id(s.key[i]));
            s.w[i] = w;
            mine += w;
          }
          total = block_sum(mine, s);
          if (!total) {   // the list covers the target: the target itself
            total = r.mass;
#pragma unroll 1
            for (int i = tid; i < n; i += kRowThreads) s.w[i] = r.kept(s.key[i]);
          }
        }
        __syncthreads();
        f = Range{0xFFFFFFFFu - (uint32_t)(a.n - 1), 0xFFFFFFFFu, place_of(total, u) + 1, 0};
      }
      const uint64_t k = list_find(f, n, stage == 2 ? 0xFFFFFFFFull : ~0ull, stage == 0, s);
      if (stage < 2) r.thr = max(r.thr, k);
      else drawn = (int)(0xFFFFFFFFu - (uint32_t)k);
    }
    if (!accepted) kept_x = drawn >= 0 ? (double)r.kept(r.key_at(drawn)) : 0.0;
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
  size_t gmax, gsecond, gat, tmax, tsum, state, arrived, total;
};
Space space(int64_t rows, int64_t seqs, int64_t n) {
  const size_t tiles = (size_t)rows * ceil_div(n, kTile);
  Space s{};
  s.gmax = 0;
  s.gsecond = align256(tiles * kGroups * 4);
  s.gat = 2 * s.gsecond;
  s.tmax = 3 * s.gsecond;
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
  // as How::mass() goes by them, where they are known here
  const bool some_k = !in.top_k && in.top_k_all > 0 && in.top_k_all < in.n, greedy = !in.temperature && !(in.temperature_all > 0.f);
  const bool only_min_p = !in.top_p && !(in.top_p_all < 1.f) && !in.min_p && in.min_p_all > 0.f;
  a.sums = !(some_k || greedy || only_min_p);
  a.token = in.token;
  a.prob = in.prob;
  a.probs = in.probs;
  if (workspace) {
    const Space s = space(a.rows, seqs, in.n);
    char* ws = static_cast<char*>(workspace);
    a.gmax = reinterpret_cast<float*>(ws + s.gmax);
    a.gsecond = reinterpret_cast<float*>(ws + s.gsecond);
    a.gat = reinterpret_cast<int32_t*>(ws + s.gat);
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
  const auto rows = a.rows > kCus ? sample_rows_kernel<T, VERIFY, 2> : sample_rows_kernel<T, VERIFY, 1>;
  hipLaunchKernelGGL(rows, dim3((unsigned)a.rows), dim3(kRowThreads), 0, s, a);
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
