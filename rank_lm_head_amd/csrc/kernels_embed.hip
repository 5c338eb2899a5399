// kernels_embed.hip — the rows of an embedding matrix at given tokens, and
// the matrix's gradient.
//
//   out[n, :] = scale W[t_n, :]            (zeros for t_n outside [0, V))
//   dW[v, :]  = scale sum_{n: t_n = v} dY[n, :]
//
// The lookup is one read and one write of each row. The gradient is made
// without atomics on values, so that it does not vary: the positions are
// sorted by token (a stable radix sort), a wave sums the rows of `chunk`
// neighbouring places of the sorted order in registers, and runs of one token
// that pass the end of a chunk are joined afterwards, chunk after chunk. Up to
// kFew positions go without a sort: each wave looks for the other positions
// of its token. Sums are fp32, scaled and rounded once.
//
// What bounds it is the write of dW, of which most rows are zeros. The sort,
// the sums and the join wait for memory rather than fill it, so each of their
// launches has blocks that clear rows beside them: rows of tokens that do not
// occur, or, while the sort is still running, any.
#include <algorithm>

#include "device.h"
#include "launch.h"
#include "topk.h"

namespace lrh {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / kWave;
constexpr int kDigitBits = 9;                 // of a pass of the sort, at most
constexpr int kDigits = 1 << kDigitBits;
constexpr int kSmallSort = 16384;             // places that one block sorts
constexpr int kSortTile = 4096;               // places of a block of the larger sort
constexpr int kFillPiece = 16384;             // bytes that a block clears at a time
constexpr int kFew = 512;                     // places that need no sort
constexpr int kMostBuckets = 4096;            // of neighbouring tokens, cleared by one block each
constexpr int kBucketRows = 4096;             // tokens of one, at most
constexpr int64_t kBucketBytes = 65536;       // of its rows, where there are so many
constexpr int64_t kSortBytes = 50 << 20, kSortBytesPer = 6144;   // cleared beside the sort: in all, and for each place
constexpr int64_t kJoinBytes = 12 << 20;      // and beside the join

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// 16 bytes at an address aligned to its elements only.
__device__ __forceinline__ u32x4 load16_any(const void* p) {
  u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
__device__ __forceinline__ void store16_any(void* p, u32x4 v) { __builtin_memcpy(p, &v, 16); }
typedef u32x4 u32x4_any __attribute__((aligned(2)));
// ... cleared. Past the caches where other blocks of the launch need those (4096
// places of 5120 bf16: the sums 46 us, 61 through them); through them in a
// launch that does little else (151936 x 563 bf16, 64 places: 24 us, 33 past them).
template <bool kPast = true>
__device__ __forceinline__ void clear16(void* p) {
  if (kPast) __builtin_nontemporal_store(u32x4{0u, 0u, 0u, 0u}, reinterpret_cast<u32x4_any*>(p));
  else *reinterpret_cast<u32x4_any*>(p) = u32x4{0u, 0u, 0u, 0u};
}

template <typename T> struct Elems;
template <> struct Elems<float> {
  static constexpr int n = 4;
  static __device__ __forceinline__ float get(u32x4 v, int e) { return __uint_as_float(v[e]); }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ u32x4 pack(const float (&f)[4]) {
    return u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
  }
};
template <> struct Elems<uint16_t> {
  static constexpr int n = 8;
  static __device__ __forceinline__ float get(u32x4 v, int e) {
    return __uint_as_float((e & 1) ? (v[e >> 1] & 0xffff0000u) : (v[e >> 1] << 16));
  }
  static __device__ __forceinline__ float one(const uint16_t* p) { return bf16_to_f32(*p); }
  static __device__ __forceinline__ u32x4 pack(const float (&f)[8]) {
    bf16x8 v;   // to the nearest, ties to even: an instruction for two
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = (__bf16)f[q];
    return __builtin_bit_cast(u32x4, v);
  }
};

// ------------------------------------------------------------------- lookup

struct EmbedArgs {
  const void* W;
  int64_t V, d;
  const int32_t* token;
  int64_t N;
  float scale;
  void* out;
  int pieces;   // of a row
};

// A wave copies one piece of one row: four 16-byte loads a lane in flight.
constexpr int kEmbedChunks = 4;
template <typename T>
__global__ void __launch_bounds__(kThreads) embed_kernel(EmbedArgs a) {
  constexpr int EP = Elems<T>::n;
  const uint32_t w = blockIdx.x * kWaves + wave_id(), n32 = w / (uint32_t)a.pieces;   // w < 2^26
  const int64_t n = n32;
  if (n >= a.N) return;
  const int64_t c0 = (int64_t)(w - n32 * a.pieces) * (kEmbedChunks * kWave * EP) + (threadIdx.x & 63) * EP;
  const int t = a.token[n];
  const bool have = t >= 0 && t < a.V;
  const T* src = static_cast<const T*>(a.W) + (have ? (int64_t)t * a.d : 0);
  T* dst = static_cast<T*>(a.out) + n * a.d;
  u32x4 v[kEmbedChunks];
#pragma unroll
  for (int i = 0; i < kEmbedChunks; ++i) {
    const int64_t c = c0 + i * (kWave * EP);
    v[i] = u32x4{0u, 0u, 0u, 0u};
    if (have && c + EP <= a.d) v[i] = load16_any(src + c);
  }
#pragma unroll
  for (int i = 0; i < kEmbedChunks; ++i) {
    const int64_t c = c0 + i * (kWave * EP);
    if (c + EP <= a.d) {
      if (a.scale != 1.f) {
        float f[EP];
#pragma unroll
        for (int e = 0; e < EP; ++e) f[e] = Elems<T>::get(v[i], e) * a.scale;
        v[i] = have ? Elems<T>::pack(f) : u32x4{0u, 0u, 0u, 0u};   // 0 of a missing token, whatever the scale
      }
      store16_any(dst + c, v[i]);
    } else {
      for (int64_t e = c; e < a.d; ++e)
        dst[e] = !have ? T(0) : a.scale != 1.f ? store_cast<T>(Elems<T>::one(src + e) * a.scale) : src[e];
    }
  }
}

// --------------------------------------------------------------------- sort

struct GradArgs {
  const void* dY;
  const int32_t* token;
  int64_t N, V, d;
  float scale;
  void* dW;
  bool add;             // to what dW holds; else its other rows are cleared
  int bits, passes;     // of a pass's digit, of the keys
  int at_bits;          // one block's sort: bits of a place
  int tiles;            // blocks of the larger sort
  uint32_t* count;      // [digit][tile]
  uint32_t *key[2], *at[2];   // sorted tokens (V: none) and their places; [0] holds the result
  int chunk;            // sorted places of a wave
  int64_t chunks;
  int pieces;           // waves along a row
  float* part;          // [chunk][2][d]: runs that began before the chunk, and that go on behind it
  int sum_blocks;       // blocks that sum or join; those behind them clear rows
  int bucket_bits;      // a bucket has 2^bucket_bits tokens
  int buckets;          // 0: dW is cleared as a whole before the sums
  int from, to;         // buckets that this launch clears
  uint32_t* start;      // [buckets + 1]: the first sorted place of each
};

__device__ __forceinline__ uint32_t key_of_token(const GradArgs& a, int t) {
  return t >= 0 && t < a.V ? (uint32_t)t : (uint32_t)a.V;
}
__device__ __forceinline__ uint32_t key_of(const GradArgs& a, int64_t i) { return key_of_token(a, a.token[i]); }

// The lanes whose digit (below kDigits) is this lane's; all of the wave's lanes
// call it. Four instructions a bit: the sort of one block is bound by them.
__device__ __forceinline__ unsigned long long same_digit(uint32_t digit, bool live) {
  const unsigned long long m = __ballot(live);
  uint32_t lo = (uint32_t)m, hi = (uint32_t)(m >> 32);
#pragma unroll
  for (int b = 0; b < kDigitBits; ++b) {
    const uint32_t t = (uint32_t)((int)(digit << (31 - b)) >> 31);   // all ones or none
    const unsigned long long v = __ballot(t != 0);
    lo &= ~((uint32_t)v ^ t);
    hi &= ~((uint32_t)(v >> 32) ^ t);
  }
  return (unsigned long long)hi << 32 | lo;
}

// Exclusive prefix sums of hist[digit][wave], digit by digit, in place.
// hist: [kSortWaves][1 << bits]; sums: kSortWaves words.
__device__ __forceinline__ void scan_hist(uint32_t* hist, int digits, uint32_t* sums) {
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  // a thread takes a digit's counts of 16 waves; with fewer threads than digits times that never
  uint32_t mine = 0, c[kSortWaves];
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) c[w] = tid < digits ? hist[w * digits + tid] : 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) mine += c[w];
  const uint32_t incl = wave_incl_scan_u32(mine);
  if (lane == 63) sums[wave] = incl;
  __syncthreads();
  uint32_t at = incl - mine;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) at += w < wave ? sums[w] : 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    if (tid < digits) hist[w * digits + tid] = at;
    at += c[w];
  }
  __syncthreads();
}

// Clears a share of dW: blocks [0, blocks) take pieces in turn.
__device__ __forceinline__ void clear(const GradArgs& a, size_t elem, int64_t block, int64_t blocks, int64_t from, int64_t to) {
  char* p = static_cast<char*>(a.dW);
  for (int64_t at = from + block * kFillPiece; at < to; at += blocks * kFillPiece) {
    const int64_t end = min(to, at + kFillPiece);
    for (int64_t o = at + (int64_t)threadIdx.x * 16; o < end; o += (int64_t)blockDim.x * 16) {
      if (o + 16 <= end) {
        clear16<>(p + o);
      } else {
        for (int64_t q = o; q < end; q += elem)
          if (elem == 2) *reinterpret_cast<uint16_t*>(p + q) = 0;
          else *reinterpret_cast<uint32_t*>(p + q) = 0;
      }
    }
  }
}

// Clears n bytes from p on, aligned to elements.
template <size_t kElem, bool kPast>
__device__ __forceinline__ void clear_bytes(char* p, int64_t n) {
  for (int64_t o = (int64_t)threadIdx.x * 16; o < n; o += (int64_t)blockDim.x * 16) {
    if (o + 16 <= n) {
      clear16<kPast>(p + o);
    } else {
      for (int64_t q = o; q < n; q += kElem)
        if (kElem == 2) *reinterpret_cast<uint16_t*>(p + q) = 0;
        else *reinterpret_cast<uint32_t*>(p + q) = 0;
    }
  }
}

// Clears the rows of a bucket whose tokens are not seen (a bit each, LDS), a
// run of rows at a time. The bits are looked through in registers, by words:
// one by one from LDS they took longer than the clearing (64 places, 151936
// tokens, d = 64 in bf16: 16 us of 23).
template <size_t kElem, bool kPast = true>
__device__ __forceinline__ void clear_unseen(const GradArgs& a, int bucket, const uint32_t* seen) {
  const int64_t r0 = (int64_t)bucket << a.bucket_bits, row = a.d * (int64_t)kElem;
  const int rows = (int)min((int64_t)1 << a.bucket_bits, a.V - r0);
  char* p = static_cast<char*>(a.dW) + r0 * row;
  static_assert(kBucketRows == 2 * kWave * 32, "a lane has two words");
  const int words = (rows + 31) / 32, lane = threadIdx.x & 63;
  const uint32_t low = lane < words ? seen[lane] : 0, high = lane + kWave < words ? seen[lane + kWave] : 0;
  const unsigned long long any_low = __ballot(low != 0), any_high = __ballot(high != 0);
  const auto word = [&](int i) {
    return i < kWave ? (uint32_t)__builtin_amdgcn_readlane((int)low, i)
                     : (uint32_t)__builtin_amdgcn_readlane((int)high, i - kWave);
  };
  int r = 0;
  while (r < rows) {
    const int i = r >> 5, bit = r & 31;
    uint32_t w = word(i) >> bit;
    if (w & 1) {   // past the seen ones; above the word's top come zeros
      r += w == ~0u ? 32 : __ffs((int)~w) - 1;
      continue;
    }
    // the first seen one from r on: in this word, or in the next word that has any
    int end = rows;
    if (w) {
      end = r + __ffs((int)w) - 1;
    } else {
      const unsigned long long l = i + 1 < kWave ? any_low >> (i + 1) << (i + 1) : 0;
      const int h0 = max(i + 1 - kWave, 0);
      const unsigned long long h = h0 < kWave ? any_high >> h0 << h0 : 0;
      const int next = l ? __ffsll(l) - 1 : h ? kWave + __ffsll(h) - 1 : -1;
      if (next >= 0) end = next * 32 + __ffs((int)word(next)) - 1;
    }
    clear_bytes<kElem, kPast>(p + r * row, (end - r) * row);
    r = end;
  }
}
__device__ __forceinline__ void see(const GradArgs& a, int bucket, uint32_t key, uint32_t* seen) {
  const int64_t r = (int64_t)key - ((int64_t)bucket << a.bucket_bits);
  if (r >= 0 && r >> a.bucket_bits == 0) atomicOr(&seen[r >> 5], 1u << (r & 31));
}
// The blocks' buckets in turn; the next one's keys are on their way while one
// is cleared. seen: kBucketRows / 32 words of LDS.
template <size_t kElem>
__device__ __forceinline__ void clear_buckets(const GradArgs& a, int block, int blocks, uint32_t* seen) {
  const int tid = threadIdx.x, words = ((1 << a.bucket_bits) + 31) / 32;
  const uint32_t* keys = a.key[0];
  int b = a.from + block;
  if (b >= a.to) return;
  int k0 = (int)a.start[b], k1 = (int)a.start[b + 1];
  uint32_t key = keys[min(k0 + tid, (int)a.N - 1)];
  while (b < a.to) {
    const int next = b + blocks, n = min(next, a.to - 1);
    const int n0 = (int)a.start[n], n1 = (int)a.start[n + 1];
    __syncthreads();
    for (int i = tid; i < words; i += blockDim.x) seen[i] = 0;
    __syncthreads();
    if (k0 + tid < k1) see(a, b, key, seen);
    for (int i = k0 + tid + blockDim.x; i < k1; i += 4 * blockDim.x) {   // a few frequent tokens' bucket
      uint32_t k[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) k[q] = keys[min(i + q * (int)blockDim.x, k1 - 1)];
#pragma unroll
      for (int q = 0; q < 4; ++q) see(a, b, k[q], seen);
    }
    key = keys[min(n0 + tid, (int)a.N - 1)];
    __syncthreads();
    clear_unseen<kElem>(a, b, seen);
    b = next;
    k0 = n0;
    k1 = n1;
  }
}

// Up to kSmallSort places: block 0 sorts them in LDS, a token and its place
// as one 32-bit word, while the other blocks clear dW. A wave owns a stretch
// of the places, so equal digits keep their order by wave, round and lane.
template <size_t kElem>
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(GradArgs a) {
  extern __shared__ uint32_t lds[];
  if (blockIdx.x > 0) {
    const int64_t row = a.d * (int64_t)kElem;
    const int64_t from = a.buckets ? min(a.V, (int64_t)a.from << a.bucket_bits) : 0;
    const int64_t to = a.buckets ? min(a.V, (int64_t)a.to << a.bucket_bits) : a.V;
    clear(a, kElem, blockIdx.x - 1, gridDim.x - 1, from * row, to * row);
    return;
  }
  constexpr int kMost = kSmallSort / kSortThreads;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  const int n = (int)a.N;
  uint32_t* sums = lds;                     // kSortWaves
  uint32_t* hist = lds + 64;                // [kSortWaves][kDigits]
  uint32_t* word = hist + kSortWaves * kDigits;   // n
  const int rounds = (n + kSortThreads - 1) / kSortThreads;
  const int first = wave * rounds * kWave;
  uint32_t v[kMost];
  int t[kMost];   // all loads on their way before the first is looked at
#pragma unroll
  for (int i = 0; i < kMost; ++i) t[i] = a.token[min(first + i * kWave + lane, n - 1)];
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int p = first + i * kWave + lane;
    v[i] = i < rounds && p < n ? key_of_token(a, t[i]) << a.at_bits | (uint32_t)p : 0u;
  }
  const int digits = 1 << a.bits;
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = a.at_bits + pass * a.bits;
    for (int i = tid; i < kSortWaves * digits; i += kSortThreads) hist[i] = 0;
    __syncthreads();
    uint32_t rank[kMost];
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      if (i < rounds) {
        const bool live = first + i * kWave + lane < n;
        const uint32_t digit = (v[i] >> shift) & (digits - 1);
        const unsigned long long same = same_digit(digit, live);
        uint32_t* h = hist + wave * digits + digit;
        const int below = lanes_below(same);
        uint32_t had = 0;
        if (live) had = *h;
        __builtin_amdgcn_wave_barrier();
        if (live && below == 0) *h = had + __popcll(same);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        rank[i] = had + below;
      }
    }
    __syncthreads();
    scan_hist(hist, digits, sums);
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      if (i < rounds && first + i * kWave + lane < n) {
        const uint32_t digit = (v[i] >> shift) & (digits - 1);
        word[hist[wave * digits + digit] + rank[i]] = v[i];
      }
    }
    __syncthreads();
    if (pass + 1 < a.passes) {
#pragma unroll
      for (int i = 0; i < kMost; ++i) {
        const int p = first + i * kWave + lane;
        if (i < rounds && p < n) v[i] = word[p];
      }
    }
  }
#pragma unroll 2
  for (int p = tid; p < n; p += kSortThreads) {
    const uint32_t x = word[p];
    a.key[0][p] = x >> a.at_bits;
    a.at[0][p] = x & (uint32_t)((1ull << a.at_bits) - 1);
    // where the buckets begin: those behind the place's predecessor's up to its own
    const int b = min((int)(x >> a.at_bits >> a.bucket_bits), a.buckets);
    const int before = p ? min((int)(word[p - 1] >> a.at_bits >> a.bucket_bits), a.buckets) : -1;
    for (int q = before + 1; a.buckets && q <= b; ++q) a.start[q] = p;
    if (p == n - 1)
      for (int q = b + 1; a.buckets && q <= a.buckets; ++q) a.start[q] = n;
  }
}

// The larger sort, a pass of it in three launches: each block counts the
// digits of its tile; one block makes places of the counts (and the others
// clear dW); each block moves its tile, in order.
constexpr int kTileRounds = kSortTile / kSortThreads;
__device__ __forceinline__ void tile_ranks(const GradArgs& a, int pass, const uint32_t (&key)[kTileRounds],
                                           uint32_t (&rank)[kTileRounds], uint32_t* hist, int64_t first) {
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int digits = 1 << a.bits, shift = pass * a.bits;
  for (int i = threadIdx.x; i < kSortWaves * digits; i += kSortThreads) hist[i] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kTileRounds; ++i) {
    const bool live = first + i * kWave + lane < a.N;
    const uint32_t digit = (key[i] >> shift) & (digits - 1);
    const unsigned long long same = same_digit(digit, live);
    uint32_t* h = hist + wave * digits + digit;
    const int below = lanes_below(same);
    uint32_t had = 0;
    if (live) had = *h;
    __builtin_amdgcn_wave_barrier();
    if (live && below == 0) *h = had + __popcll(same);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    rank[i] = had + below;
  }
  __syncthreads();
}
__device__ __forceinline__ void tile_keys(const GradArgs& a, int pass, int64_t first, uint32_t (&key)[kTileRounds]) {
  const int lane = threadIdx.x & 63;
  const uint32_t* from = pass == 0 ? reinterpret_cast<const uint32_t*>(a.token) : a.key[(a.passes - pass) & 1];
#pragma unroll
  for (int i = 0; i < kTileRounds; ++i) key[i] = from[min(first + i * kWave + lane, a.N - 1)];
#pragma unroll
  for (int i = 0; i < kTileRounds; ++i) key[i] = pass == 0 ? key_of_token(a, (int)key[i]) : key[i];
}

__global__ void __launch_bounds__(kSortThreads) embed_count_kernel(GradArgs a, int pass) {
  __shared__ uint32_t hist[kSortWaves * kDigits];
  const int64_t first = (int64_t)blockIdx.x * kSortTile + wave_id() * (kTileRounds * kWave);
  uint32_t key[kTileRounds], rank[kTileRounds];
  tile_keys(a, pass, first, key);
  tile_ranks(a, pass, key, rank, hist, first);
  const int digits = 1 << a.bits;
  for (int g = threadIdx.x; g < digits; g += kSortThreads) {
    uint32_t c = 0;
    for (int w = 0; w < kSortWaves; ++w) c += hist[w * digits + g];
    a.count[(int64_t)g * a.tiles + blockIdx.x] = c;
  }
}

template <size_t kElem>
__global__ void __launch_bounds__(kSortThreads) embed_places_kernel(GradArgs a, int pass) {
  if (blockIdx.x > 0) {   // a share of dW for each pass
    const int64_t bytes = a.V * a.d * (int64_t)kElem;
    const int64_t share = (bytes / a.passes) & ~(int64_t)15;
    clear(a, kElem, blockIdx.x - 1, gridDim.x - 1, share * pass, pass + 1 == a.passes ? bytes : share * (pass + 1));
    return;
  }
  __shared__ uint32_t sums[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  const int total = a.tiles << a.bits;
  uint32_t before = 0;
  for (int i0 = 0; i0 < total; i0 += kSortThreads * 4) {
    uint32_t c[4], mine = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = i0 + tid * 4 + q;
      c[q] = i < total ? a.count[i] : 0u;
      mine += c[q];
    }
    const uint32_t incl = wave_incl_scan_u32(mine);
    if (lane == 63) sums[wave] = incl;
    __syncthreads();
    uint32_t at = before + incl - mine, all = 0;
    for (int w = 0; w < kSortWaves; ++w) {
      if (w < wave) at += sums[w];
      all += sums[w];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = i0 + tid * 4 + q;
      if (i < total) a.count[i] = at;
      at += c[q];
    }
    before += all;
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kSortThreads) embed_move_kernel(GradArgs a, int pass) {
  __shared__ uint32_t hist[kSortWaves * kDigits];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int64_t first = (int64_t)blockIdx.x * kSortTile + wave * (kTileRounds * kWave);
  uint32_t key[kTileRounds], rank[kTileRounds];
  tile_keys(a, pass, first, key);
  tile_ranks(a, pass, key, rank, hist, first);
  const int digits = 1 << a.bits, shift = pass * a.bits;
  for (int g = threadIdx.x; g < digits; g += kSortThreads) {   // where each wave's digits begin
    uint32_t at = a.count[(int64_t)g * a.tiles + blockIdx.x];
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = hist[w * digits + g];
      hist[w * digits + g] = at;
      at += c;
    }
  }
  __syncthreads();
  const uint32_t* from = a.at[(a.passes - pass) & 1];
  uint32_t* to_key = a.key[(a.passes - pass - 1) & 1];
  uint32_t* to_at = a.at[(a.passes - pass - 1) & 1];
#pragma unroll
  for (int i = 0; i < kTileRounds; ++i) {
    const int64_t p = first + i * kWave + lane;
    if (p >= a.N) continue;
    const uint32_t o = hist[wave * digits + ((key[i] >> shift) & (digits - 1))] + rank[i];
    to_key[o] = key[i];
    to_at[o] = pass == 0 ? (uint32_t)p : from[p];
  }
}

// --------------------------------------------------------------------- sums

// A wave's columns of a row of dY or dW: 16 bytes a lane.
template <typename T>
struct Row {
  static constexpr int EP = Elems<T>::n;
  float f[EP];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int e = 0; e < EP; ++e) f[e] = 0.f;
  }
  __device__ __forceinline__ void add(u32x4 v) {
#pragma unroll
    for (int e = 0; e < EP; ++e) f[e] += Elems<T>::get(v, e);
  }
};

// EVEN: d is a multiple of a lane's 16 bytes.
template <typename T, bool EVEN>
__device__ __forceinline__ u32x4 load_piece(const T* row, int64_t c, int64_t d) {
  constexpr int EP = Elems<T>::n;
  if (EVEN) return load16_any(row + (c < d ? c : 0));
  if (c + EP <= d) return load16_any(row + c);
  float f[EP];
#pragma unroll
  for (int e = 0; e < EP; ++e) f[e] = c + e < d ? Elems<T>::one(row + c + e) : 0.f;
  return Elems<T>::pack(f);
}

// dW[key, c..] = scale r (+ what is there), rounded once.
template <typename T, bool EVEN>
__device__ __forceinline__ void put(const GradArgs& a, uint32_t key, int64_t c, Row<T>& r) {
  constexpr int EP = Elems<T>::n;
  if (c >= a.d) return;
  T* row = static_cast<T*>(a.dW) + (int64_t)key * a.d;
  float f[EP];
#pragma unroll
  for (int e = 0; e < EP; ++e) f[e] = r.f[e] * a.scale;
  if (a.add) {
    const u32x4 old = load_piece<T, EVEN>(row, c, a.d);
#pragma unroll
    for (int e = 0; e < EP; ++e) f[e] += Elems<T>::get(old, e);
  }
  if (EVEN || c + EP <= a.d) {
    store16_any(row + c, Elems<T>::pack(f));
  } else {
    for (int e = 0; c + e < a.d; ++e) row[c + e] = store_cast<T>(f[e]);
  }
}

template <typename T>
__device__ __forceinline__ float* part_of(const GradArgs& a, int64_t chunk, int side, int piece) {
  constexpr int EP = Elems<T>::n;
  return a.part + ((chunk * 2 + side) * a.pieces + piece) * (kWave * EP) + (threadIdx.x & 63) * EP;
}

// Sums of the sorted places [chunk * a.chunk, ...): runs inside the chunk go
// to dW, those that pass one of its ends to a.part. Lanes hold 64 places at
// a time; kAhead rows are on their way.
constexpr int kAhead = 16;
template <typename T, bool EVEN>
__global__ void __launch_bounds__(kThreads) embed_sum_kernel(GradArgs a) {
  constexpr int EP = Elems<T>::n;
  __shared__ uint32_t seen[kBucketRows / 32];
  if ((int)blockIdx.x >= a.sum_blocks) {
    clear_buckets<sizeof(T)>(a, blockIdx.x - a.sum_blocks, gridDim.x - a.sum_blocks, seen);
    return;
  }
  const uint32_t w = blockIdx.x * kWaves + wave_id();   // below 2^26
  const int64_t chunk = w / (uint32_t)a.pieces;
  if (chunk >= a.chunks) return;
  const int piece = (int)(w - (uint32_t)chunk * a.pieces), lane = threadIdx.x & 63;
  const int64_t c = (int64_t)piece * (kWave * EP) + lane * EP;
  const int64_t p0 = chunk * a.chunk, p1 = min(a.N, p0 + a.chunk);
  const uint32_t *keys = a.key[0], *at = a.at[0];
  const T* dY = static_cast<const T*>(a.dY);
  const uint32_t none = (uint32_t)a.V;
  const uint32_t before = p0 ? keys[p0 - 1] : none, behind = p1 < a.N ? keys[p1] : none;
  uint32_t run = keys[p0];
  bool began = p0 == 0 || before != run;   // the run begins in this chunk
  Row<T> sum, head;   // head: of the run that began before
  bool has_head = false;
  sum.zero();
  head.zero();
  for (int64_t q0 = p0; q0 < p1; q0 += kWave) {
    const int n = (int)min((int64_t)kWave, p1 - q0);
    const int key_l = lane < n ? (int)keys[q0 + lane] : (int)none;
    const int at_l = lane < n ? (int)at[q0 + lane] : 0;
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += kAhead) {
      u32x4 v[kAhead];   // rows of missing tokens and behind the last: any, and not added
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const uint32_t row = (uint32_t)__builtin_amdgcn_readlane(at_l, min(i0 + j, n - 1));
        v[j] = load_piece<T, EVEN>(dY + (int64_t)row * a.d, c, a.d);
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int i = i0 + j;
        if (i < n) {
          const uint32_t k = (uint32_t)__builtin_amdgcn_readlane(key_l, i);
          if (k != run) {
            if (run != none) {
              if (began) {
                put<T, EVEN>(a, run, c, sum);
              } else {
                head = sum;
                has_head = true;
              }
            }
            sum.zero();
            run = k;
            began = true;
          }
          if (k != none) sum.add(v[j]);
        }
      }
    }
  }
  if (has_head) {
    float* o = part_of<T>(a, chunk, 0, piece);
#pragma unroll
    for (int e = 0; e < EP; ++e) o[e] = head.f[e];
  }
  if (run == none) return;
  const bool more = behind == run;
  if (began && !more) {
    put<T, EVEN>(a, run, c, sum);
    return;
  }
  float* o = part_of<T>(a, chunk, began ? 1 : 0, piece);
#pragma unroll
  for (int e = 0; e < EP; ++e) o[e] = sum.f[e];
}

// Joins the runs that pass the end of the chunk that they begin in.
template <typename T, bool EVEN>
__global__ void __launch_bounds__(kThreads) embed_join_kernel(GradArgs a) {
  constexpr int EP = Elems<T>::n, kPartsAhead = 8;
  __shared__ uint32_t seen[kBucketRows / 32];
  if ((int)blockIdx.x >= a.sum_blocks) {
    clear_buckets<sizeof(T)>(a, blockIdx.x - a.sum_blocks, gridDim.x - a.sum_blocks, seen);
    return;
  }
  const uint32_t w = blockIdx.x * kWaves + wave_id();   // below 2^26
  const int64_t chunk = w / (uint32_t)a.pieces;
  if (chunk + 1 >= a.chunks) return;   // nothing behind it
  const int piece = (int)(w - (uint32_t)chunk * a.pieces), lane = threadIdx.x & 63;
  const int64_t c = (int64_t)piece * (kWave * EP) + lane * EP;
  const uint32_t* keys = a.key[0];
  const int64_t p0 = chunk * a.chunk, p1 = p0 + a.chunk;
  const uint32_t first = keys[p0], before = p0 ? keys[p0 - 1] : (uint32_t)a.V, run = keys[p1 - 1], behind = keys[p1];
  if (run == (uint32_t)a.V || behind != run) return;
  if (first == run && p0 > 0 && before == run) return;   // it began before
  Row<T> sum;
  const float* o = part_of<T>(a, chunk, 1, piece);
#pragma unroll
  for (int e = 0; e < EP; ++e) sum.f[e] = o[e];
  // the run's further chunks: those that begin with its token
  for (int64_t c0 = chunk + 1; c0 < a.chunks; c0 += kWave) {
    const bool in = c0 + lane < a.chunks && keys[(c0 + lane) * a.chunk] == run;
    const unsigned long long m = __ballot(in);
    const int n = m == ~0ull ? kWave : __ffsll((unsigned long long)~m) - 1;
    for (int i0 = 0; i0 < n; i0 += kPartsAhead) {
      float f[kPartsAhead][EP];
#pragma unroll
      for (int j = 0; j < kPartsAhead; ++j) {
        const float* o = part_of<T>(a, c0 + min(i0 + j, n - 1), 0, piece);
#pragma unroll
        for (int e = 0; e < EP; ++e) f[j][e] = o[e];
      }
#pragma unroll
      for (int j = 0; j < kPartsAhead; ++j) {
        if (i0 + j < n) {
#pragma unroll
          for (int e = 0; e < EP; ++e) sum.f[e] += f[j][e];
        }
      }
    }
    if (n < kWave) break;
  }
  put<T, EVEN>(a, run, c, sum);
}

// Up to kFew places, everything in one launch: a wave per place and piece of
// a row sums its token's rows if no earlier place has the token. (333 places of
// 256 fp32 columns, 4096 tokens: 17 us as sort, sums and join, of which the
// sort of one block was 7.)
template <typename T, bool EVEN>
__global__ void __launch_bounds__(kThreads) embed_few_kernel(GradArgs a) {
  constexpr int EP = Elems<T>::n, kEach = kFew / kWave;
  __shared__ uint32_t seen[kBucketRows / 32];
  const int n = (int)a.N;
  if ((int)blockIdx.x >= a.sum_blocks) {
    const int words = ((1 << a.bucket_bits) + 31) / 32, tid = threadIdx.x;
    uint32_t key[kFew / kThreads];
#pragma unroll
    for (int i = 0; i < kFew / kThreads; ++i) key[i] = key_of(a, min(tid + i * kThreads, n - 1));
    for (int b = blockIdx.x - a.sum_blocks; b < a.buckets; b += gridDim.x - a.sum_blocks) {
      __syncthreads();
      for (int i = tid; i < words; i += kThreads) seen[i] = 0;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kFew / kThreads; ++i) see(a, b, key[i], seen);   // a missing token may set a bit behind V's rows
      __syncthreads();
      clear_unseen<sizeof(T), false>(a, b, seen);
    }
    return;
  }
  const uint32_t w = blockIdx.x * kWaves + wave_id();   // below 2^26
  const int place = (int)(w / (uint32_t)a.pieces);
  if (place >= n) return;
  const int piece = (int)(w - (uint32_t)place * a.pieces), lane = threadIdx.x & 63;
  const int64_t c = (int64_t)piece * (kWave * EP) + lane * EP;
  const uint32_t mine = key_of(a, place);
  int t[kEach];
  uint32_t key[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) t[i] = a.token[min(i * kWave + lane, n - 1)];
#pragma unroll
  for (int i = 0; i < kEach; ++i) key[i] = i * kWave + lane < n ? key_of_token(a, t[i]) : (uint32_t)a.V;
  if (mine == (uint32_t)a.V) return;
  const T* dY = static_cast<const T*>(a.dY);
  Row<T> sum;
  sum.zero();
  bool first = true;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    unsigned long long m = __ballot(key[i] == mine);
    if (first && m) {
      if (i * kWave + __ffsll(m) - 1 != place) return;   // an earlier place has it
      first = false;
    }
    while (m) {
      u32x4 v[8];
      unsigned long long left = m;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = left ? i * kWave + __ffsll(left) - 1 : place;
        left &= left - 1;
        v[j] = load_piece<T, EVEN>(dY + (int64_t)at * a.d, c, a.d);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (m) sum.add(v[j]);
        m &= m - 1;
      }
    }
  }
  put<T, EVEN>(a, mine, c, sum);
}

struct GradPlan {
  int bits, passes, at_bits, tiles, chunk, pieces;
  int64_t chunks;
  bool few, small;
  int bucket_bits, buckets;
};
int bits_of(uint64_t x) { return x ? 64 - __builtin_clzll(x) : 0; }
GradPlan plan(int dtype, int64_t V, int64_t d, int64_t N) {
  GradPlan p;
  const int all = std::max(1, bits_of((uint64_t)V));   // of tokens and V itself
  p.passes = (all + kDigitBits - 1) / kDigitBits;
  p.bits = (all + p.passes - 1) / p.passes;
  p.at_bits = std::max(1, bits_of((uint64_t)(N - 1)));
  p.bucket_bits = 0;
  const int64_t row = d * (dtype == 0 ? 2 : 4), bucket = std::clamp<int64_t>(V * row / 1024, 4096, kBucketBytes);
  while ((V - 1) >> p.bucket_bits >= kMostBuckets || (row << p.bucket_bits < bucket && (1 << p.bucket_bits) < kBucketRows))
    ++p.bucket_bits;
  p.buckets = (int)((V - 1) >> p.bucket_bits) + 1;
  const bool fits = (1 << p.bucket_bits) <= kBucketRows;
  p.few = N <= kFew && fits;
  p.small = N <= kSmallSort && all + p.at_bits <= 32;
  if (!fits || !(p.few || p.small)) p.buckets = 0;
  p.tiles = (int)ceil_div(N, kSortTile);
  p.pieces = (int)ceil_div(d, kWave * (dtype == 0 ? 8 : 4));
  // Longer chunks leave fewer parts to join, as long as there are waves for all compute units.
  p.chunk = kAhead;
  while (p.chunk < 256 && ceil_div(N, 2 * p.chunk) * p.pieces >= 1024) p.chunk *= 2;
  p.chunks = ceil_div(N, p.chunk);
  return p;
}
struct GradSpace {
  size_t key[2], at[2], count, start, part, total;
};
GradSpace space(int dtype, int64_t V, int64_t d, int64_t N) {
  const GradPlan p = plan(dtype, V, d, N);
  GradSpace s{};
  size_t o = 0;
  const auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align256(bytes);
    return at;
  };
  if (p.few) {
    s.total = 256;   // not used
    return s;
  }
  s.key[0] = take((size_t)N * 4);
  s.at[0] = take((size_t)N * 4);
  s.start = take((size_t)(p.buckets + 1) * 4);
  if (!p.small) {
    s.key[1] = take((size_t)N * 4);
    s.at[1] = take((size_t)N * 4);
    s.count = take(((size_t)p.tiles << p.bits) * 4);
  }
  s.part = take((size_t)p.chunks * 2 * p.pieces * kWave * (dtype == 0 ? 8 : 4) * 4);
  s.total = o;
  return s;
}

template <typename T, bool EVEN>
hipError_t embed_grad(GradArgs a, const GradPlan& p, hipStream_t s) {
  // blocks that clear rows beside the others: four a compute unit at most
  const int64_t bytes = a.add ? 0 : a.V * a.d * (int64_t)sizeof(T);
  const auto blocks_for = [](int64_t n) { return (int)std::min<int64_t>(1024, ceil_div(n, kFillPiece)); };
  const int64_t waves = (p.few ? a.N : a.chunks) * a.pieces;
  a.sum_blocks = (int)ceil_div(waves, kWaves);
  if (p.few) {
    const int fill = std::min(p.buckets, blocks_for(bytes));
    hipLaunchKernelGGL((embed_few_kernel<T, EVEN>), dim3(a.sum_blocks + fill), dim3(kThreads), 0, s, a);
    return hipGetLastError();
  }
  // Buckets that each launch clears: beside the sort and the join what they
  // leave time for (at 6 MB a microsecond), the rest beside the sums. The sort
  // has the last ones, whose tokens are the rarest in most vocabularies: it
  // cannot know yet which rows the sums will write over. The first ones may
  // have most of the places to look at, for which the sums leave the most time.
  int by_sort = 0, by_join = 0;
  if (p.buckets && bytes) {
    const int64_t bucket = (bytes + p.buckets - 1) / p.buckets;
    by_sort = (int)std::min<int64_t>(p.buckets, (kSortBytes + a.N * kSortBytesPer) / bucket);
    by_join = a.chunks > 1 ? (int)std::min<int64_t>(p.buckets - by_sort, kJoinBytes / bucket) : 0;
  }
  if (p.small) {
    const size_t lds = (64 + kSortWaves * kDigits + (size_t)a.N) * 4;
    if (lds > 65536) {
      const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(embed_sort_kernel<sizeof(T)>),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
      if (e != hipSuccess) return e;
    }
    a.from = p.buckets - by_sort;
    a.to = p.buckets;
    const int fill = blocks_for(p.buckets ? bytes / p.buckets * by_sort : bytes);
    hipLaunchKernelGGL(embed_sort_kernel<sizeof(T)>, dim3(1 + fill), dim3(kSortThreads), lds, s, a);
  } else {
    for (int pass = 0; pass < a.passes; ++pass) {
      hipLaunchKernelGGL(embed_count_kernel, dim3(a.tiles), dim3(kSortThreads), 0, s, a, pass);
      hipLaunchKernelGGL(embed_places_kernel<sizeof(T)>, dim3(1 + blocks_for(bytes)), dim3(kSortThreads), 0, s, a, pass);
      hipLaunchKernelGGL(embed_move_kernel, dim3(a.tiles), dim3(kSortThreads), 0, s, a, pass);
    }
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const auto fill_for = [&](int buckets) { return bytes ? std::min(buckets, 1024) : 0; };
  a.from = 0;
  a.to = bytes ? p.buckets - by_sort - by_join : 0;
  hipLaunchKernelGGL((embed_sum_kernel<T, EVEN>), dim3(a.sum_blocks + fill_for(a.to - a.from)), dim3(kThreads), 0, s, a);
  a.from = a.to;
  a.to += by_join;
  if (a.chunks > 1)
    hipLaunchKernelGGL((embed_join_kernel<T, EVEN>), dim3(a.sum_blocks + fill_for(by_join)), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <size_t kElem>
__global__ void __launch_bounds__(kSortThreads) embed_clear_kernel(GradArgs a) {
  clear(a, kElem, blockIdx.x, gridDim.x, 0, a.V * a.d * (int64_t)kElem);
}

}  // namespace

bool embed_fits(int dtype, int64_t d, int64_t N) {
  const int64_t pieces = ceil_div(d, kEmbedChunks * kWave * (dtype == 0 ? 8 : 4));
  return ceil_div(N * pieces, kWaves) <= kMostThreads / kThreads;
}

bool embed_grad_fits(int dtype, int64_t V, int64_t d, int64_t N) {
  const GradPlan p = plan(dtype, V, d, N);
  return ceil_div((p.few ? N : p.chunks) * p.pieces, kWaves) + 1024 <= kMostThreads / kThreads;
}

hipError_t launch_embed(int dtype, const void* W, int64_t V, int64_t d, const int32_t* token, int64_t N, float scale,
                        void* out, hipStream_t s) {
  EmbedArgs a{W, V, d, token, N, scale, out, (int)ceil_div(d, kEmbedChunks * kWave * (dtype == 0 ? 8 : 4))};
  const dim3 grid((unsigned)ceil_div(N * a.pieces, kWaves)), block(kThreads);
  if (dtype == 0) hipLaunchKernelGGL(embed_kernel<uint16_t>, grid, block, 0, s, a);
  else hipLaunchKernelGGL(embed_kernel<float>, grid, block, 0, s, a);
  return hipGetLastError();
}

size_t embed_grad_workspace_bytes(int dtype, int64_t V, int64_t d, int64_t N) { return space(dtype, V, d, N).total; }

hipError_t launch_embed_grad(int dtype, const void* dY, const int32_t* token, int64_t N, int64_t V, int64_t d,
                             float scale, bool add, void* dW, void* workspace, hipStream_t s) {
  GradArgs a{};
  a.dY = dY;
  a.token = token;
  a.N = N;
  a.V = V;
  a.d = d;
  a.scale = scale;
  a.dW = dW;
  a.add = add;
  if (N == 0) {
    if (add) return hipSuccess;
    const size_t elem = dtype == 0 ? 2 : 4;
    const dim3 grid((unsigned)std::min<int64_t>(1024, ceil_div(V * d * (int64_t)elem, kFillPiece)));
    if (dtype == 0) hipLaunchKernelGGL(embed_clear_kernel<2>, grid, dim3(kSortThreads), 0, s, a);
    else hipLaunchKernelGGL(embed_clear_kernel<4>, grid, dim3(kSortThreads), 0, s, a);
    return hipGetLastError();
  }
  const GradPlan p = plan(dtype, V, d, N);
  const GradSpace sp = space(dtype, V, d, N);
  char* ws = static_cast<char*>(workspace);
  a.bits = p.bits;
  a.passes = p.passes;
  a.at_bits = p.at_bits;
  a.tiles = p.tiles;
  a.count = reinterpret_cast<uint32_t*>(ws + sp.count);
  for (int i = 0; i < 2; ++i) {
    a.key[i] = reinterpret_cast<uint32_t*>(ws + sp.key[i]);
    a.at[i] = reinterpret_cast<uint32_t*>(ws + sp.at[i]);
  }
  a.chunk = p.chunk;
  a.chunks = p.chunks;
  a.pieces = p.pieces;
  a.part = reinterpret_cast<float*>(ws + sp.part);
  a.start = reinterpret_cast<uint32_t*>(ws + sp.start);
  a.bucket_bits = p.bucket_bits;
  a.buckets = p.buckets;
  if (dtype == 0) return d % 8 ? embed_grad<uint16_t, false>(a, p, s) : embed_grad<uint16_t, true>(a, p, s);
  return d % 4 ? embed_grad<float, false>(a, p, s) : embed_grad<float, true>(a, p, s);
}

}  // namespace lrh
