// kernels_beam.hip — beam search over a head's logits: the selection of the
// best continuations of all beams of a sequence, and the move of the beams'
// states behind it.
//
// Selection: of the m beams of a sequence, beam i with path score c_i and
// logits x_i over n columns, the nb best by
//   total(i, v) = c_i + x_iv - lse(x_i),   lse(x) = log sum_v exp(x_v),
// ties to the lower beam and then the lower column. A beam's own order does
// not depend on lse, so one pass over the logits makes both: a block takes a
// slice of one row into registers, sums its exponentials and keeps its nb
// best, and one block per sequence joins the slices and then the beams.
// What bounds it is the one read of the logits.
//
// lse and the totals are held in 64 bits, the sums inside a slice in
// 32 bits: two totals of different beams closer than
// about 1e-7 may come out in either order, all others in theirs.
#include <algorithm>

#include "device.h"
#include "launch.h"
#include "topk.h"

namespace lrh {

namespace {

constexpr int kThreads = 256;
constexpr int kBeamWaves = kThreads / kWave;
constexpr int kMostWaves = 16;   // of a block that joins: a wave per beam up to here
constexpr float kLog2eHi = 1.44269502162933349609f, kLog2eLo = 1.92596299112661746887e-8f;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ uint64_t wave_max_u64(uint64_t x) {
  const uint32_t hi = wave_max_u32((uint32_t)(x >> 32));
  const uint32_t lo = wave_max_u32((uint32_t)(x >> 32) == hi ? (uint32_t)x : 0u);
  return ((uint64_t)hi << 32) | lo;
}

template <int S>
__device__ __forceinline__ uint64_t lane_xor_u64(uint64_t x) {
  return ((uint64_t)(uint32_t)lane_xor<S>((int)(x >> 32)) << 32) | (uint32_t)lane_xor<S>((int)x);
}

__device__ __forceinline__ double wave_sum_f64(double x) {
#pragma unroll
  for (int o = 32; o; o >>= 1) x += __shfl_xor(x, o);
  return x;
}

// The order-preserving image of a total; 0 for what is no candidate (NaN, -inf).
__device__ __forceinline__ uint64_t total_key(double t) {
  if (!(t > -__builtin_inf())) return 0;
  const uint64_t u = (uint64_t)__double_as_longlong(t + 0.0);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double total_of(uint64_t k) {
  return __longlong_as_double((long long)((k >> 63) ? (k & 0x7fffffffffffffffull) : ~k));
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

struct SelectArgs {
  const void* x;
  int64_t ld;             // row stride of x
  const int32_t* idx;     // rows x n token ids (negative: no candidate), or NULL: the column
  const float* score;     // rows
  const uint8_t* ended;   // rows, or NULL
  int end_id;
  int64_t rows;           // B m
  int m;
  int64_t n;
  int nb;
  int slices;
  uint64_t* keys;         // [row][slice][nb] candidate keys, best first, 0 past the last
  float* top;             // [row][slice] the slice's largest logit
  float* sum;             // [row][slice] and the sum of exp(x - that)
  float* out_score;
  int32_t* out_beam;
  int32_t* out_token;
};

// One slice of one row: CH 16-byte chunks per thread, neighbouring threads on
// neighbouring chunks. The slice's nb best are at least as large as the
// nb-th largest of the maxima of 64 * KG groups of threads, a bound that few
// others pass (KG = 1 up to 16 best, 2 up to 32, else 4). Any bound that 16 KG
// group maxima at most reach will do: 64 threads then hold what passes it.
template <typename T, int CH, bool IDS, int KG>
__global__ void __launch_bounds__(kThreads) beam_slice_kernel(SelectArgs a) {
  constexpr int EP = Elems<T>::n, E = CH * EP;
  constexpr int kSlice = kThreads * E, kGroups = 64 * KG;
  __shared__ __attribute__((aligned(16))) uint64_t gmax[kGroups];
  __shared__ uint64_t cand[64 * E];
  __shared__ uint32_t red[kBeamWaves];
  __shared__ float reds[kBeamWaves];
  __shared__ int count;
  const int64_t row = blockIdx.x / a.slices;
  const int slice = blockIdx.x % a.slices;
  const int tid = threadIdx.x, wave = wave_id(), lane = tid & 63;
  if (a.ended && a.ended[row]) return;   // its one continuation needs no logits
  uint64_t* out = a.keys + (row * a.slices + slice) * a.nb;
  const T* x = static_cast<const T*>(a.x) + row * a.ld;
  const int64_t c0 = (int64_t)slice * kSlice;

  float v[E];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int64_t col = c0 + (int64_t)(c * kThreads + tid) * EP;
    if (col + EP <= a.n) {
      const u32x4 w = load16_any(x + col);
#pragma unroll
      for (int e = 0; e < EP; ++e) v[c * EP + e] = fmaxf(Elems<T>::get(w, e), neg_inf());   // NaN becomes -inf
    } else {
#pragma unroll
      for (int e = 0; e < EP; ++e) v[c * EP + e] = col + e < a.n ? fmaxf(Elems<T>::one(x + col + e), neg_inf()) : neg_inf();
    }
    if constexpr (IDS) {
#pragma unroll
      for (int e = 0; e < EP; ++e)
        if (col + e < a.n && a.idx[row * a.n + col + e] < 0) v[c * EP + e] = neg_inf();
    }
  }
  if (tid == 0) count = 0;
  float hi = neg_inf();
  int at = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    if (v[i] > hi) {
      hi = v[i];
      at = i;
    }
  }
  const auto col_of = [&](int i) { return (int)(c0 + (int64_t)((i / EP) * kThreads + tid) * EP + i % EP); };
  const uint64_t mine = hi > neg_inf() ? cand_key(hi, col_of(at)) : 0ull;
  uint64_t most = mine;
  if constexpr (KG <= 2) most = max(most, lane_xor_u64<1>(most));
  if constexpr (KG == 1) most = max(most, lane_xor_u64<2>(most));
  if (tid % (4 / KG) == 0) gmax[tid / (4 / KG)] = most;
  const uint32_t wm = wave_max_u32((uint32_t)(mine >> 32));
  if (lane == 0) red[wave] = wm;
  __syncthreads();
  uint32_t bm = 0;
#pragma unroll
  for (int w = 0; w < kBeamWaves; ++w) bm = max(bm, red[w]);
  if (!bm) {   // nothing in this slice
    if (tid < a.nb) out[tid] = 0;
    if (tid == 0) {
      a.top[row * a.slices + slice] = neg_inf();
      a.sum[row * a.slices + slice] = 0.f;
    }
    return;
  }
  uint64_t keys[KG];
#pragma unroll
  for (int i = 0; i < KG; ++i) keys[i] = gmax[i * 64 + lane];
  const uint64_t lim = max(wave_window_threshold<KG>(keys, a.nb, 16 * KG), (uint64_t)1);   // in every wave
  if (mine >= lim) {
    const float least = lim > 1 ? key_score(lim) : -__FLT_MAX__;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      if (v[i] >= least) {
        const uint64_t key = cand_key(v[i], col_of(i));
        if (key >= lim) cand[atomicAdd(&count, 1)] = key;
      }
    }
  }
  // log2(e) as the sum of two fp32: one alone is off by 1e-8 of every exponent, in one direction
  const float m = __uint_as_float(order_key_inv(bm));
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const float d = v[i] - m;
    s += exp2_hw(fmaf(d, kLog2eHi, d * kLog2eLo));   // 0 of -inf: m is finite
  }
  s = group_sum<kWave>(s);
  if (lane == 0) reds[wave] = s;
  __syncthreads();
  const int n = count;
  for (int i = tid; i < n; i += kThreads) {
    const uint64_t key = cand[i];
    int r = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) r += cand[j] > key;
    if (r < a.nb) out[r] = key;
  }
  if (tid >= n && tid < a.nb) out[tid] = 0;
  if (tid == 0) {
    a.top[row * a.slices + slice] = m;
    a.sum[row * a.slices + slice] = (reds[0] + reds[1]) + (reds[2] + reds[3]);
  }
}

// The beams' lists of a sequence in LDS, and the join over them: lane i
// holds the head of beam i's list; nb times the best head leaves.
struct Lists {
  uint64_t* total;   // [m][nb], 0 past the last
  int* col;          // [m][nb]
};

__device__ __forceinline__ void join_beams(const SelectArgs& a, int64_t b, const Lists& L) {
  const int lane = threadIdx.x & 63;
  int at = 0, beam = -1, col = 0;   // lane j: the j-th best
  uint64_t got = 0;
  uint64_t head = lane < a.m ? L.total[lane * a.nb] : 0;
  for (int j = 0; j < a.nb; ++j) {
    const uint64_t best = wave_max_u64(head);
    if (!best) break;
    const int win = __ffsll((unsigned long long)__ballot(head == best)) - 1;
    const int from = win * a.nb + __builtin_amdgcn_readlane(at, win);
    if (lane == j) {
      got = best;
      beam = win;
      col = from;
    }
    if (lane == win) {
      ++at;
      head = at < a.nb ? L.total[lane * a.nb + at] : 0;
    }
  }
  if (lane >= a.nb) return;
  const int64_t o = b * a.nb + lane;
  int token = -1;
  if (got) {
    const int64_t row = b * a.m + beam;
    const int c = L.col[col];
    token = a.ended && a.ended[row] ? a.end_id : a.idx ? a.idx[row * a.n + c] : c;
  }
  a.out_score[o] = got ? (float)total_of(got) : neg_inf();
  a.out_beam[o] = beam;
  a.out_token[o] = token;
}

// Joins the slices of each beam (a wave per beam) and then the beams. Of the
// slices' lists, a lane takes every 64th; a bound that at
// least nb of the lanes' best heads reach bounds the beam's nb best, and what
// passes it is ranked. (Lists that pass it more than kPassed times over, as ascending rows make them,
// take the best head nb times instead.)
constexpr int kPassed = 256;
__global__ void __launch_bounds__(kMostWaves* kWave) beam_join_kernel(SelectArgs a) {
  extern __shared__ uint64_t lds[];
  const Lists L{lds, reinterpret_cast<int*>(lds + a.m * a.nb)};
  const int64_t b = blockIdx.x;
  const int wave = wave_id(), lane = threadIdx.x & 63, waves = blockDim.x / kWave;
  for (int i = wave; i < a.m; i += waves) {
    const int64_t row = b * a.m + i;
    const double c = a.score[row];
    uint64_t* total = L.total + i * a.nb;
    int* col = L.col + i * a.nb;
    if (a.ended && a.ended[row]) {
      if (lane < a.nb) {
        total[lane] = lane == 0 ? total_key(c) : 0;
        col[lane] = 0;
      }
      continue;
    }
    const float* top = a.top + row * a.slices;
    const float* sum = a.sum + row * a.slices;
    const uint64_t* keys = a.keys + row * a.slices * a.nb;
    float hi = neg_inf();
    uint64_t best[1] = {0};
    for (int s = lane; s < a.slices; s += kWave) {
      hi = fmaxf(hi, top[s]);
      best[0] = max(best[0], keys[(int64_t)s * a.nb]);
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) hi = fmaxf(hi, __shfl_xor(hi, o));
    double l = 0.0;
    for (int s = lane; s < a.slices; s += kWave) {
      const float d = top[s] - hi;
      if (sum[s] != 0.f) l += (double)sum[s] * (double)exp2_hw(fmaf(d, kLog2eHi, d * kLog2eLo));
    }
    l = wave_sum_f64(l);
    const double logl = log(l);   // lse - hi: hi may be so large that their sum is hi

    const uint64_t lim = max(wave_window_threshold<1>(best, a.nb, min(a.nb + a.nb / 2, 64)), (uint64_t)1);
    uint64_t* mem = reinterpret_cast<uint64_t*>(L.col + a.m * a.nb + (a.m * a.nb & 1)) + wave * kPassed;
    int n = 0;   // keys that pass, in the same order in every lane's view
    if (a.slices <= kWave * 16) {
      for (int s0 = 0; s0 < a.slices; s0 += kWave) {
        const int s = s0 + lane;
        bool more = s < a.slices;
        for (int j = 0; j < a.nb && n <= kPassed; ++j) {
          const uint64_t k = more ? keys[(int64_t)s * a.nb + j] : 0;
          more = k >= lim;
          const unsigned long long mask = __ballot(more);
          if (!mask) break;
          const int at = n + lanes_below(mask);
          if (more && at < kPassed) mem[at] = k;
          n += __popcll(mask);
        }
      }
    } else {
      n = kPassed + 1;
    }
    const auto put = [&](int j, uint64_t k) {
      total[j] = k ? total_key((double)key_score(k) - (double)hi - logl + c) : 0;
      col[j] = k ? key_id(k) : 0;
    };
    if (n <= kPassed) {
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      for (int q = lane; q < n; q += kWave) {
        const uint64_t k = mem[q];
        int r = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j) r += mem[j] > k;
        if (r < a.nb) put(r, k);
      }
      for (int j = n + lane; j < a.nb; j += kWave) put(j, 0);
      continue;
    }
    uint64_t head = 0;
    const auto refill = [&](uint64_t below) {   // the best of the lane's lists below a key
      head = 0;
      for (int s = lane; s < a.slices; s += kWave)
        for (int j = 0; j < a.nb; ++j) {
          const uint64_t k = keys[(int64_t)s * a.nb + j];
          if (k < below) {
            head = max(head, k);
            break;
          }
        }
    };
    refill(~0ull);
    for (int j = 0; j < a.nb; ++j) {
      const uint64_t k = wave_max_u64(head);
      if (lane == 0) put(j, k);
      if (k && head == k) refill(k);
    }
  }
  __syncthreads();
  if (wave == 0) join_beams(a, b, L);
}

// Rows of at most 64 columns (candidate lists): a wave per beam, a lane per
// column, everything in one launch.
template <typename T>
__global__ void __launch_bounds__(kMostWaves* kWave) beam_lists_kernel(SelectArgs a) {
  extern __shared__ uint64_t lds[];
  const Lists L{lds, reinterpret_cast<int*>(lds + a.m * a.nb)};
  const int64_t b = blockIdx.x;
  const int wave = wave_id(), lane = threadIdx.x & 63, waves = blockDim.x / kWave;
  for (int i = wave; i < a.m; i += waves) {
    const int64_t row = b * a.m + i;
    const double c = a.score[row];
    uint64_t* total = L.total + i * a.nb;
    int* col = L.col + i * a.nb;
    if (a.ended && a.ended[row]) {
      if (lane < a.nb) {
        total[lane] = lane == 0 ? total_key(c) : 0;
        col[lane] = 0;
      }
      continue;
    }
    float x = lane < a.n ? Elems<T>::one(static_cast<const T*>(a.x) + row * a.ld + lane) : neg_inf();
    if (!(x > neg_inf()) || (a.idx && lane < a.n && a.idx[row * a.n + lane] < 0)) x = neg_inf();
    int id = lane;
    x += 0.f;   // -0 and +0 are the same score
    bitonic_sort_desc(x, id);
    const float hi = readlane_f(x, 0);
    const float d = x - hi;
    const double l = wave_sum_f64(x > neg_inf() ? (double)exp2_hw(fmaf(d, kLog2eHi, d * kLog2eLo)) : 0.0);
    const double logl = log(l);   // lse - hi: hi may be so large that their sum is hi
    if (lane < a.nb) {
      total[lane] = x > neg_inf() ? total_key((double)x - (double)hi - logl + c) : 0;
      col[lane] = id;
    }
  }
  __syncthreads();
  if (wave == 0) join_beams(a, b, L);
}

// ------------------------------------------------------------------ states

constexpr int kStatesPerLaunch = 32;
constexpr int kMoveBytes = 16384;   // a block's piece of a segment
constexpr int64_t kBlocksX = 1 << 20;             // a row of a launch's blocks
constexpr int64_t kMostBlocks = kBlocksX * 4096;

struct MoveState {
  const char* src;
  char* dst;
  int64_t segs;       // segments of a beam
  int64_t seg_bytes;
  int64_t pos_bytes;  // bytes of one position of a segment
  int64_t pieces;     // blocks per segment
  int64_t first;      // first block
};
struct MoveArgs {
  MoveState st[kStatesPerLaunch];
  int states;
  int64_t blocks;
  const int32_t* parent;   // B x nb
  const int32_t* length;   // B, or NULL
  int m, nb;
};

// A block copies one piece of one segment of one new beam: U is the widest
// unit that the addresses and sizes of all states allow.
template <typename U>
__global__ void __launch_bounds__(kThreads) beam_move_kernel(MoveArgs a) {
  const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (block >= a.blocks) return;
  int s = 0;
  while (s + 1 < a.states && block >= a.st[s + 1].first) ++s;
  const MoveState& st = a.st[s];
  int64_t i = block - st.first;
  const int64_t piece = i % st.pieces;
  i /= st.pieces;
  const int64_t seg = i % st.segs, slot = i / st.segs;
  const int64_t b = slot / a.nb;
  const int p = a.parent[slot];
  if (p < 0 || p >= a.m) return;
  int64_t live = st.seg_bytes;
  if (a.length) live = min(live, (int64_t)max(a.length[b], 0) * st.pos_bytes);
  const int64_t at = piece * kMoveBytes;
  const int64_t n = (min(live, at + kMoveBytes) - at) / (int64_t)sizeof(U);
  const U* __restrict__ src = reinterpret_cast<const U*>(st.src + ((b * a.m + p) * st.segs + seg) * st.seg_bytes + at);
  U* __restrict__ dst = reinterpret_cast<U*>(st.dst + (slot * st.segs + seg) * st.seg_bytes + at);
  int64_t j = threadIdx.x;
  for (; j + 3 * kThreads < n; j += 4 * kThreads) {   // four loads in flight
    U v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = src[j + q * kThreads];
#pragma unroll
    for (int q = 0; q < 4; ++q) __builtin_nontemporal_store(v[q], dst + j + q * kThreads);
  }
  for (; j < n; j += kThreads) dst[j] = src[j];
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// 16-byte chunks per thread of a slice: the most for which the rows still
// make four blocks per compute unit, so that few lists are left to join, and
// at most 32 elements (256 rows of 151936 bf16: 32.8 us with 64, 28.8 with 32,
// 43.7 with 16, whose bounds and ranks weigh more).
int slice_chunks(int64_t rows, int64_t n, int per_chunk) {
  for (int ch = 32 / per_chunk; ch > 1; ch /= 2)
    if (rows * ceil_div(n, (int64_t)kThreads * per_chunk * ch) >= 1024) return ch;
  return 1;
}
int slice_count(int dtype, int64_t rows, int64_t n) {
  const int per = dtype == 0 ? 8 : 4;
  return (int)ceil_div(n, (int64_t)kThreads * per * slice_chunks(rows, n, per));
}

template <typename T, int CH, bool IDS>
void go_slices(const SelectArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.rows * a.slices)), block(kThreads);
  if (a.nb <= 16) hipLaunchKernelGGL((beam_slice_kernel<T, CH, IDS, 1>), grid, block, 0, s, a);
  else if (a.nb <= 32) hipLaunchKernelGGL((beam_slice_kernel<T, CH, IDS, 2>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((beam_slice_kernel<T, CH, IDS, 4>), grid, block, 0, s, a);
}
template <typename T, int CH>
void go_slices(const SelectArgs& a, hipStream_t s) {
  if (a.idx) go_slices<T, CH, true>(a, s);
  else go_slices<T, CH, false>(a, s);
}
template <typename T>
void slices(const SelectArgs& a, hipStream_t s) {
  switch (slice_chunks(a.rows, a.n, Elems<T>::n)) {
    case 1: return go_slices<T, 1>(a, s);
    case 2: return go_slices<T, 2>(a, s);
    case 4: return go_slices<T, 4>(a, s);
    default:
      if constexpr (sizeof(T) == 4) go_slices<T, 8>(a, s);
  }
}

}  // namespace

bool beam_fits(int dtype, int64_t B, int m, int64_t n) {
  return n <= kWave || B * m * slice_count(dtype, B * m, n) <= kMostThreads / kThreads;
}

size_t beam_workspace_bytes(int dtype, int64_t B, int m, int64_t n, int nb) {
  if (n <= kWave) return 256;   // not used
  const int64_t rows = B * m;
  const size_t lists = (size_t)rows * slice_count(dtype, rows, n);
  return align256(lists * nb * 8) + 2 * align256(lists * 4);
}

hipError_t launch_beam_select(int dtype, const void* x, int64_t ld, const int32_t* idx, const float* score,
                              const uint8_t* ended, int end_id, int64_t B, int m, int64_t n, int nb, float* out_score,
                              int32_t* out_beam, int32_t* out_token, void* workspace, hipStream_t s) {
  SelectArgs a{};
  a.x = x;
  a.ld = ld;
  a.idx = idx;
  a.score = score;
  a.ended = ended;
  a.end_id = end_id;
  a.rows = B * m;
  a.m = m;
  a.n = n;
  a.nb = nb;
  a.out_score = out_score;
  a.out_beam = out_beam;
  a.out_token = out_token;
  const int waves = std::min(m, kMostWaves);
  const size_t lds = (size_t)m * nb * 12;   // at most 48 KiB; with the joining waves' own at most 80
  if (n <= kWave) {
    if (dtype == 0)
      hipLaunchKernelGGL(beam_lists_kernel<uint16_t>, dim3((unsigned)B), dim3(waves * kWave), lds, s, a);
    else
      hipLaunchKernelGGL(beam_lists_kernel<float>, dim3((unsigned)B), dim3(waves * kWave), lds, s, a);
    return hipGetLastError();
  }
  a.slices = slice_count(dtype, a.rows, n);
  const size_t lists = (size_t)a.rows * a.slices;
  char* ws = static_cast<char*>(workspace);
  a.keys = reinterpret_cast<uint64_t*>(ws);
  a.top = reinterpret_cast<float*>(ws + align256(lists * nb * 8));
  a.sum = reinterpret_cast<float*>(ws + align256(lists * nb * 8) + align256(lists * 4));
  if (dtype == 0) slices<uint16_t>(a, s);
  else slices<float>(a, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const size_t bytes = lds + 8 + (size_t)waves * kPassed * 8;
  if (bytes > 65536) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(beam_join_kernel),
                            hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(beam_join_kernel, dim3((unsigned)B), dim3(waves * kWave), bytes, s, a);
  return hipGetLastError();
}

hipError_t launch_beam_move(const BeamState* states, int n_states, const int32_t* parent, const int32_t* length,
                            int64_t B, int m, int nb, hipStream_t s) {
  for (int s0 = 0; s0 < n_states;) {
    MoveArgs a{};
    a.parent = parent;
    a.length = length;
    a.m = m;
    a.nb = nb;
    uintptr_t bits = 0;
    int64_t blocks = 0;
    while (s0 < n_states && a.states < kStatesPerLaunch) {
      const BeamState& in = states[s0];
      MoveState& st = a.st[a.states];
      st.src = static_cast<const char*>(in.src);
      st.dst = static_cast<char*>(in.dst);
      st.segs = length ? in.segs : 1;
      st.pos_bytes = in.pos_bytes;
      st.seg_bytes = in.positions * in.pos_bytes * (length ? 1 : in.segs);
      st.pieces = ceil_div(st.seg_bytes, kMoveBytes);
      const int64_t more = B * nb * st.segs * st.pieces;
      if (a.states && blocks + more > kMostBlocks) break;   // the rest in the next launch
      st.first = blocks;
      blocks += more;
      bits |= reinterpret_cast<uintptr_t>(in.src) | reinterpret_cast<uintptr_t>(in.dst) | (uintptr_t)st.seg_bytes;
      if (length) bits |= (uintptr_t)st.pos_bytes;
      if (more) ++a.states;
      ++s0;
    }
    if (!blocks) continue;
    if (blocks > kMostBlocks) return hipErrorInvalidValue;
    a.blocks = blocks;
    const int64_t x = std::min(blocks, kBlocksX);
    const dim3 grid((unsigned)x, (unsigned)ceil_div(blocks, x)), block(kThreads);
    if (bits % 16 == 0) hipLaunchKernelGGL(beam_move_kernel<u32x4>, grid, block, 0, s, a);
    else if (bits % 4 == 0) hipLaunchKernelGGL(beam_move_kernel<uint32_t>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(beam_move_kernel<uint8_t>, grid, block, 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace lrh
