// kernels_distill.hip — distillation of the low-rank head from a teacher's
// top logits: the loss and its gradients.
//
// For N rows z_n of the student (length r) and its head P (V x r), with a
// temperature T and the k teacher places (id, t) of each row:
//   q_n = softmax(P . z_n / T) over the whole vocabulary,
//   p_n = softmax(t / T) over the row's places that are not empty,
//   loss_n   = sum_j p_nj (log p_nj - s_nj / T) + lse_n,   s_nj = P[id_j] . z_n
//   dloss_n/dz_n = (sum_v q_nv P_v - sum_j p_nj P[id_j]) / T
//   dP       = sum_n w_n / T (q_n - p_n) z_n^T             (w: the rows' weights)
//
// The scores (N x V; 2.5 GB in fp32 at 4096 rows of a 151936-token
// vocabulary) are never stored: both passes keep one side in registers,
// stream the other through LDS and use each tile of scores where it is
// made. With X the side at rest and Y the streamed one, both compute
//   S = Y . X^T,   E = exp2(S log2(e)/T - c),   A += Y^T . E
//   rows pass    (X = Z, Y = P): c = a score near the row's largest; A is the
//                unnormalised sum_v q_v P_v, an attention over the
//                vocabulary whose keys and values are both P;
//   columns pass (X = P, Y = Z): c = lse_n - log(|w_n|/T), so E is already
//                |w_n| q_nv / T and A the dense part of dP.
// The matrix cores leave S with its X row in the lane and its Y rows in the
// lane's registers, which is (up to an order of the contracted index that
// the other operand follows) the layout in which E is the right operand of
// the second product: E never leaves the registers.
#include <limits.h>

#include <algorithm>
#include <type_traits>

#include "device.h"
#include "launch.h"
#include "topk.h"

namespace lrh {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4_t;
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int kRawBufferFlags = 0x00020000;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eLo = 1.92596299e-8f;   // log2(e) - kLog2e
constexpr float kLn2 = 0.6931471805599453f;
// The exponents of the rows pass are taken from the largest of a share's
// first scores, not from a running maximum: fp32 and bf16 have range to
// spare, so a score may pass the reference by 2^60 before a sum or a product
// could leave it, and neither the sums nor the accumulators (which would have
// to leave the matrix cores' registers for it) are ever rescaled.
constexpr float kMostSum = 0x1p60f;
constexpr int kWaves = 4;
constexpr int kMaxShares = 512;   // of a row of Z

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_hw(float x) { return __builtin_amdgcn_logf(x); }   // of normal numbers

// Two fp32 as packed bf16, each rounded to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  bf16x2 v;
  v[0] = (__bf16)lo;
  v[1] = (__bf16)hi;
  return __builtin_bit_cast(uint32_t, v);
}

struct StreamArgs {
  const void* X;        // nx x r, at rest in registers
  const void* Y;        // ny x ldy (r columns used), streamed
  int64_t nx, ny;
  int r, ldy;
  float scale;          // log2(e) / T
  int64_t whole;        // blocks of X that stream all of Y (the first ones)
  int splits;           // shares of Y of the others, one block each
  // rows pass: a share's maximum (log2 domain), sum and weighted sum of P
  float* pm;            // [share][nx]
  float* pl;
  float* po;            // [share][nx][RP]
  // columns pass
  // [tile] of the rows of Z: RB times c (+inf for rows without weight), RB
  // times the weight's sign as bit 15 of 16 bits, padding to 2 RB words
  const float* row_c;
  int row_block;        // RB
  const uint32_t* list_start;   // [groups + 1]: the teacher places of a group of columns in `list`
  const uint2* list;    // (row | local column << kRowBits, -w p / T), by row within a group
  int64_t groups;
  int chunk_bits;       // log2 of the places of a chunk of the list
  const uint32_t* chunk_in;     // [chunk] c0 | c1 << 16 of the group that it lies in, 0 if it is not in one
  float* chunk_part;    // [chunk] its results, in the order of the accumulators
  void* dP;             // V x r, from whole blocks
  float* part;          // [share][row of X past the whole blocks'][RP], from the others
};
constexpr int kRowBits = 20;   // N <= 2^20, groups of at most 2^12 columns
constexpr uint32_t kRowMask = (1u << kRowBits) - 1;

constexpr int kRowBlock = 64;   // RB of the fp32 kernel
__device__ __forceinline__ float* row_c_at(float* row_c, uint32_t n, uint32_t RB) {   // RB a power of two
  return row_c + n + (n & ~(RB - 1));
}
__device__ __forceinline__ uint16_t* row_sign_at(float* row_c, uint32_t n, uint32_t RB) {
  return reinterpret_cast<uint16_t*>(row_c + 2 * (n & ~(RB - 1)) + RB) + (n & (RB - 1));
}

// 16-byte chunk c of row y of an LDS tile sits at chunk c ^ swz_row(y). A wave
// reads the tile as the left operand of S (32 rows, one chunk each) and,
// transposed, of A (4 rows, 4 neighbouring chunks each); the two low row
// bits go to the high chunk bits so that both spread over all banks.
template <int RP>
__device__ __forceinline__ int swz_row(int y) {
  if constexpr (RP >= 128) return ((y & 3) << 2) | ((y >> 2) & 3);
  else if constexpr (RP == 64) return (((y >> 1) & 1) << 2) | ((y >> 2) & 3);
  else return (y >> 2) & 3;
}

// Where share `split` of `splits` (at most 2^10) begins in a list of teacher places.
__device__ __forceinline__ uint32_t share_of(uint32_t places, int split, int splits) {
  return (uint32_t)((uint64_t)places * (uint32_t)split / (uint32_t)splits);
}

// Rows of a tile: 32 for each of the waves that share one out, and at least
// 16 KiB.
template <int RP, int WX>
constexpr int bf16_tile_rows() {
  const int rows = 32 * (kWaves / WX);
  return rows < (RP <= 128 ? 64 : 32) ? (RP <= 128 ? 64 : 32) : rows;
}
// LDS of a block: two tiles and, for the columns pass, two sets of row values;
// results leave through it, 32 rows of at least 32 columns a wave.
template <int RP, int WX>
constexpr int bf16_lds_bytes() {
  const int tiles = 2 * bf16_tile_rows<RP, WX>() * (RP * 2 + 8), out = kWaves * 32 * 32 * 4;
  return tiles < out ? out : tiles;
}

// Stores a wave's 32 rows of results, RP columns of which `cols` exist, to
// rows ld elements apart, `rows` of which exist. In the accumulators a lane
// holds one row; it goes through the wave's part of the LDS (chunks of 16
// bytes swizzled by the row), CH columns at a time, so that whole lines leave.
template <int RP, int CH, typename T>
__device__ __forceinline__ void store_rows(const f32x16 (&acc)[RP / 32], uint16_t* scratch, T* dst, int64_t ld, int rows,
                                           int cols) {
  constexpr int kPer = 16 / (int)sizeof(T), kChunks = CH / kPer, kMask = kChunks < 16 ? kChunks - 1 : 15;
  const int lane = threadIdx.x & 63, h = lane >> 5, x = lane & 31;
  T* mem = reinterpret_cast<T*>(scratch);
#pragma unroll
  for (int c0 = 0; c0 < RP; c0 += CH) {
#pragma unroll
    for (int rt = 0; rt < CH / 32; ++rt)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x16& a = acc[c0 / 32 + rt];
        const f32x4 v = {a[g * 4], a[g * 4 + 1], a[g * 4 + 2], a[g * 4 + 3]};
        const int c = rt * 32 + g * 8 + h * 4;
        T* at = mem + x * CH + (((c / kPer) ^ (x & kMask)) * kPer + c % kPer);
        if constexpr (sizeof(T) == 2) *reinterpret_cast<uint2*>(at) = uint2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
        else *reinterpret_cast<f32x4*>(at) = v;
      }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int i = 0; i < 32 * kChunks / kWave; ++i) {
      const int p = i * kWave + lane, row = p / kChunks, c = p % kChunks;
      const u32x4 v = load16(mem + row * CH + (c ^ (row & kMask)) * kPer);
      if (row < rows && c0 + c * kPer < cols) *reinterpret_cast<u32x4*>(dst + row * ld + c0 + c * kPer) = v;
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

// Copies rows [row0, row0 + TY) of a matrix into an LDS tile, zeros past its end
// and past r columns.
template <int RP, int TY>
struct TileCopy {
  static constexpr int kChunks = RP / 8;
  static constexpr int kLoads = (TY * kChunks + kWaves * kWave - 1) / (kWaves * kWave);
  static constexpr bool kPart = TY * kChunks < kWaves * kWave;   // the first waves only
  uint32_t off[kLoads];
  const char* base;
  int64_t rows;
  uint32_t row_bytes;

  __device__ __forceinline__ void init(const void* Y, int64_t ny, int r, int ldy) {
    const int wave = wave_id(), lane = threadIdx.x & 63;
    base = static_cast<const char*>(Y);
    rows = ny;
    row_bytes = (uint32_t)ldy * 2u;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int p = (i * kWaves + wave) * kWave + lane;
      const int row = p / kChunks, c = (p % kChunks) ^ swz_row<RP>(row);
      off[i] = c * 8 < r ? (uint32_t)row * row_bytes + (uint32_t)c * 16u : 0x7ffffff0u;
    }
  }
  __device__ __forceinline__ void issue(uint16_t* tile, int64_t row0) const {
    const int wave = wave_id();
    const uint32_t bytes = (uint32_t)max(min(rows - row0, (int64_t)TY), (int64_t)0) * row_bytes;
    const uint64_t addr = reinterpret_cast<uint64_t>(base) + (uint64_t)row0 * row_bytes;
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)addr);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(addr >> 32));
    const __amdgpu_buffer_rsrc_t rsrc =
        __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(((uint64_t)hi << 32) | lo), (short)0,
                                          __builtin_amdgcn_readfirstlane((int)bytes), kRawBufferFlags);
    if (kPart && wave >= TY * kChunks / kWave) return;
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr_t)(tile + (i * kWaves + wave) * kWave * 8), 16,
                                               (int)off[i], 0, 0, 0);
  }
};

// The lane's places in a tile, in elements from its first row. The swizzle
// depends on the row within 16 only and touches the low 4 chunk bits, so a
// few registers hold all of them; subtiles, steps of 16 rows and chunks past
// 16 are constants added to a place.
template <int RP>
struct Places {
  static constexpr int kRow = RP >= 128 ? 8 : RP / 16;   // steps of 16 columns within 16 chunks
  static constexpr int kCol = RP >= 128 ? 4 : RP / 32;   // steps of 32 columns
  int row[kRow];       // left operand of S: row (lane & 31), 8 columns
  int col[2][kCol];    // left operand of A: rows 4 h + (lane & 15) / 4 and 8 more
  __device__ __forceinline__ void init() {
    const int lane = threadIdx.x & 63, h = lane >> 5, y = lane & 31;
#pragma unroll
    for (int i = 0; i < kRow; ++i) row[i] = y * RP + ((i * 2 + h) ^ swz_row<RP>(y)) * 8;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int v = b * 8 + h * 4 + ((lane & 15) >> 2);
#pragma unroll
      for (int i = 0; i < kCol; ++i) {
        const int c = i * 4 + ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
        col[b][i] = v * RP + (c ^ swz_row<RP>(v)) * 8 + (lane & 1) * 4;
      }
    }
  }
};

// S of one 32-row subtile: its rows as the left operand.
template <int RP, int XT>
__device__ __forceinline__ void scores(const uint16_t* subtile, const Places<RP>& at, const bf16x8 (&X)[XT][RP / 16],
                                       f32x16 (&S)[XT]) {
#pragma unroll
  for (int xt = 0; xt < XT; ++xt) S[xt] = f32x16{};
#pragma unroll
  for (int ks = 0; ks < RP / 16; ++ks) {
    const bf16x8 A = __builtin_bit_cast(bf16x8, load16(subtile + at.row[ks % at.kRow] + ks / at.kRow * 128));
#pragma unroll
    for (int xt = 0; xt < XT; ++xt) S[xt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(A, X[xt][ks], S[xt], 0, 0, 0);
  }
}

// 16 rows of a tile, transposed, as the left operand of A (32 columns from
// 32 rt): 16 lanes read 4 rows of 16 columns (lane i row i / 4, columns
// 4 (i % 4)..) and each receives a column. The 8 rows of a half wave come
// in the order in which the matrix cores leave S: 4 h + 0..3, 8 + 4 h + 0..3.
template <int RP>
__device__ __forceinline__ bf16x8 columns(const uint16_t* rows16, const Places<RP>& at, int rt) {
  typedef short s16x8 __attribute__((ext_vector_type(8)));
  const uint16_t* p = rows16 + rt / at.kCol * 128;
  const s16x4 va = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t)(p + at.col[0][rt % at.kCol]));
  const s16x4 vb = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t)(p + at.col[1][rt % at.kCol]));
  const s16x8 v = {va[0], va[1], va[2], va[3], vb[0], vb[1], vb[2], vb[3]};
  return __builtin_bit_cast(bf16x8, v);
}

// Rows 8 g + 4 h .. + 3 of the lane's column of a result.
__device__ __forceinline__ f32x4 quad(const f32x16& v, int g) {
  return f32x4{v[g * 4], v[g * 4 + 1], v[g * 4 + 2], v[g * 4 + 3]};
}

// Tiles of 32 rows of X that a wave owns. Two halve the LDS reads of each
// product, but from r = 128 on they take more than half of the registers, and
// the one wave that is left to a SIMD cannot hide its exponentials behind
// another's products: rows and columns pass at 4096 rows, r = 128, took 308
// and 334 us with one tile and two waves, 377 and 411 us with two and one.
constexpr int x_tiles(int RP) { return RP <= 64 ? 2 : 1; }

// A column group's teacher places, from e0 to e1 of the list. Whole chunks of
// the list (chunks c0 to c1) are summed by other blocks before the columns
// pass, so that a group that many rows name (a frequent token) does not hold
// one block up; the rest, before and behind them, are the group's own. (The
// gradient call of 4096 rows, r = 128, k = 32, without and with chunks: all
// places below 32 of the 151936 tokens 4937 and 621 us, below 1000 791 and
// 389, uniform 350 and 332.)
// A group adds as many results of blocks of its chunks, at most:
constexpr int most_parts(int RP) { return RP <= 256 ? 64 : 16; }
struct Listed {
  uint32_t e0, head, tail, e1;   // own places: from e0 on, `head` of them; from `tail` to e1
  int c0, c1;
  __device__ __forceinline__ Listed(uint32_t first, uint32_t end, int bits) : e0(first), e1(end) {
    c0 = (int)((first + (1u << bits) - 1) >> bits);
    c1 = (int)(end >> bits);
    if (c0 < c1) {
      head = ((uint32_t)c0 << bits) - first;
      tail = (uint32_t)c1 << bits;
    } else {
      c1 = c0;
      head = end - first;
      tail = end;
    }
  }
  __device__ __forceinline__ uint32_t count() const { return head + (e1 - tail); }
  __device__ __forceinline__ uint32_t at(uint32_t i) const { return i < head ? e0 + i : tail + (i - head); }
};

// f(accumulator, quad, where it is among the chunks' results) for all of a wave's.
template <int RP, int XT, typename F>
__device__ __forceinline__ void each_quad(int chunk, int wave, f32x16 (&acc)[XT][RP / 32], F&& f) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int xt = 0; xt < XT; ++xt)
#pragma unroll
    for (int rt = 0; rt < RP / 32; ++rt)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        f(acc[xt][rt], g, (((((int64_t)chunk * kWaves + wave) * XT + xt) * (RP / 32) + rt) * 4 + g) * (kWave * 4) + lane * 4);
}

// Adds the teacher's part of a block's columns, -w p / T z_n for places i0 to
// i1 (place i is a.list[where(i)]): the places' rows of Z are gathered into
// the tiles' LDS and go through the product of the dense part, with the places'
// weights as the right operand, each the sum of two bf16 (within 2^-17 of
// it; in one word).
template <int RP, int XT, int WX, typename At>
__device__ __forceinline__ void add_places(const StreamArgs& a, uint16_t* lds, const Places<RP>& at, uint32_t i0,
                                           uint32_t i1, At&& where, f32x16 (&acc)[XT][RP / 32]) {
  constexpr int TY = bf16_tile_rows<RP, WX>(), RT = RP / 32;
  constexpr int kLoads = TileCopy<RP, TY>::kLoads;
  const int lane = threadIdx.x & 63, h = lane >> 5, wave = wave_id(), wx = wave % WX;
  const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<void*>(a.Y), (short)0, (int)((uint32_t)a.ny * (uint32_t)(RP * 2)), kRawBufferFlags);
  const auto gather = [&](int buf, uint32_t base) {   // returns the lane's place (of TY)
    const uint32_t i = base + lane % TY;
    const uint2 en = i < i1 ? a.list[where(i)] : uint2{0u, 0u};
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int p = (j * kWaves + wave) * kWave + lane;
      const int row = p / (RP / 8), c = (p % (RP / 8)) ^ swz_row<RP>(row);
      const uint32_t n = (uint32_t)__shfl((int)en.x, row) & kRowMask;
      const uint32_t off = base + row < i1 ? n * (uint32_t)(RP * 2) + (uint32_t)c * 16u : 0xfffffff0u;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr_t)(lds + buf * TY * RP + (j * kWaves + wave) * kWave * 8),
                                               16, (int)off, 0, 0, 0);
    }
    return en;
  };
  uint2 en = gather(0, i0);
  for (int buf = 0; i0 < i1; i0 += TY, buf ^= 1) {
    __builtin_amdgcn_s_waitcnt(0xF70);
    __syncthreads();
    uint2 next = {0u, 0u};
    if (i0 + TY < i1) next = gather(buf ^ 1, i0 + TY);
    const uint16_t* tile = lds + buf * TY * RP;
#pragma unroll 1
    for (int s = 0; s < TY / 16; ++s) {
      if (i0 + s * 16 >= i1) break;
      bf16x8 hi[XT], lo[XT];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int y = s * 16 + (k >> 2) * 8 + h * 4 + (k & 3);
        const int col = (int)((uint32_t)__shfl((int)en.x, y) >> kRowBits) - wx * (32 * XT);
        const uint32_t w = (uint32_t)__shfl((int)en.y, y);
#pragma unroll
        for (int xt = 0; xt < XT; ++xt) {
          const uint32_t v = col == xt * 32 + (lane & 31) ? w : 0u;
          hi[xt][k] = __builtin_bit_cast(__bf16, (uint16_t)v);
          lo[xt][k] = __builtin_bit_cast(__bf16, (uint16_t)(v >> 16));
        }
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const bf16x8 A = columns<RP>(tile + s * 16 * RP, at, rt);
#pragma unroll
        for (int xt = 0; xt < XT; ++xt) {
          acc[xt][rt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(A, hi[xt], acc[xt][rt], 0, 0, 0);
          acc[xt][rt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(A, lo[xt], acc[xt][rt], 0, 0, 0);
        }
      }
    }
    en = next;
  }
}

// The teacher's part of a share of a group's whole chunks; of a group's chunks'
// blocks, the first most_parts have a share.
template <int RP, int XT>
__global__ void __launch_bounds__(kWaves* kWave, RP == 512 ? 1 : 2) chunk_kernel(StreamArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint16_t lds[];
  const uint32_t c = blockIdx.x;
  if (c << a.chunk_bits >= a.list_start[a.groups]) return;
  const uint32_t in = a.chunk_in[c];
  const uint32_t c0 = in & 0xffff, all = (in >> 16) - c0, j = c - c0, parts = min(all, (uint32_t)most_parts(RP));
  if (!in || j >= parts) return;
  Places<RP> at;
  at.init();
  f32x16 acc[XT][RP / 32] = {};
  add_places<RP, XT, kWaves>(a, lds, at, (c0 + share_of(all, j, parts)) << a.chunk_bits,
                             (c0 + share_of(all, j + 1, parts)) << a.chunk_bits, [](uint32_t i) { return i; }, acc);
  each_quad<RP, XT>((int)c, wave_id(), acc, [&](f32x16& v, int g, int64_t to) {
    *reinterpret_cast<f32x4*>(a.chunk_part + to) = quad(v, g);
  });
}

// bf16. RP: r rounded up to a tile size; a wave owns XT * 32 rows of X, WX of
// the block's four waves sit side by side on X and 4 / WX share out a
// tile's rows of Y.
template <int RP, int XT, int WX, bool ACC, bool COLS>
__global__ void __launch_bounds__(kWaves* kWave, RP == 512 ? 1 : 2) stream_bf16_kernel(StreamArgs a) {
  constexpr int TY = bf16_tile_rows<RP, WX>();
  constexpr int KS = RP / 16, RT = RP / 32, WY = kWaves / WX;
  extern __shared__ __attribute__((aligned(16))) uint16_t lds[];
  float* const rows = reinterpret_cast<float*>(lds + 2 * TY * RP);   // [buffer][offset, sign][TY]
  const int lane = threadIdx.x & 63, h = lane >> 5, wave = wave_id();
  const int wx = wave % WX, wy = wave / WX;
  const bool whole = blockIdx.x < a.whole;
  const int splits = whole ? 1 : a.splits;
  const int64_t xtile = whole ? blockIdx.x : a.whole + (blockIdx.x - a.whole) / splits;
  const int split = whole ? 0 : (int)((blockIdx.x - a.whole) % splits);
  const int64_t x0 = (xtile * WX + wx) * (32 * XT);

  f32x16 acc[XT][ACC ? RT : 1] = {};
  float m[XT], l[XT], odd[XT];   // the sum in two parts
#pragma unroll
  for (int xt = 0; xt < XT; ++xt) {
    m[xt] = neg_inf();
    l[xt] = 0.f;
  }

  const int64_t nt = (a.ny + TY - 1) / TY;
  const int64_t t_begin = nt * split / splits, t_end = nt * (split + 1) / splits;
  Places<RP> at;
  at.init();
  TileCopy<RP, TY> copy;
  copy.init(a.Y, a.ny, a.r, a.ldy);
  const auto stage = [&](int buf, int64_t t) {
    copy.issue(lds + buf * TY * RP, t * TY);
    if constexpr (COLS) {   // the rows' offsets and signs, kept tile by tile
      if (wave < TY / 32)
        __builtin_amdgcn_global_load_lds(
            (const __attribute__((address_space(1))) void*)(a.row_c + (t * 2 * TY + wave * kWave + lane)),
            (lds_ptr_t)(rows + buf * 2 * TY + wave * kWave), 4, 0, 0);
    }
  };
  if constexpr (COLS) {
    const Listed all(a.list_start[xtile], a.list_start[xtile + 1], a.chunk_bits);
    const uint32_t i0 = share_of(all.count(), split, splits), i1 = share_of(all.count(), split + 1, splits);
    if (i0 < i1) {
      add_places<RP, XT, WX>(a, lds, at, i0, i1, [&](uint32_t i) { return all.at(i); }, acc);
      __syncthreads();   // the tiles may be filled again
    }
  }
  // X, whole lines at a time, through the tiles' LDS.
  bf16x8 X[XT][KS];
  {
    constexpr int kRows = WX * 32 * XT, kUnits = (kRows + TY - 1) / TY;
    TileCopy<RP, TY> cx;
    cx.init(a.X, a.nx, a.r, a.r);
#pragma unroll
    for (int u = 0; u < kUnits; u += 2) {
      cx.issue(lds, xtile * kRows + u * TY);
      if (u + 1 < kUnits) cx.issue(lds + TY * RP, xtile * kRows + (u + 1) * TY);
      __builtin_amdgcn_s_waitcnt(0xF70);
      __syncthreads();
#pragma unroll
      for (int xt = 0; xt < XT; ++xt) {
        const int row = (wx * XT + xt) * 32 - u * TY;   // the wave's tile within the two
        if (kUnits <= 2 || (row >= 0 && row < 2 * TY)) {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
            X[xt][ks] = __builtin_bit_cast(
                bf16x8, load16(lds + row * RP + at.row[ks % at.kRow] + ks / at.kRow * 128));
        }
      }
      __syncthreads();
    }
  }

  // Calls f(subtile, row values, rows left) for this wave's subtiles of the
  // share. Rows left is a constant 32 but for the rows pass's last tile,
  // where the vocabulary may end (the columns pass pads its rows).
  const int64_t t_full = COLS ? t_end : min(t_end, a.ny / TY);
  const auto each_subtile = [&](auto&& f) {
    const auto one_tile = [&](int buf, int64_t t, auto last) {
      __builtin_amdgcn_s_waitcnt(0xF70);   // vmcnt(0): this wave's share of tile t has landed
      __syncthreads();                      // everyone's has, and every wave is done with the other buffer
      if (t + 1 < t_end) stage(buf ^ 1, t + 1);
#pragma unroll
      for (int i = 0; i < TY / 32 / WY; ++i) {
        const int sub = i * WY + wy;
        const uint16_t* subtile = lds + (buf * TY + sub * 32) * RP;
        const float* row_c = rows + buf * 2 * TY + sub * 32;
        if constexpr (last) f(subtile, row_c, rows + buf * 2 * TY + TY + sub * 16, (int)(a.ny - t * TY - sub * 32));
        else f(subtile, row_c, rows + buf * 2 * TY + TY + sub * 16, std::integral_constant<int, 32>());
      }
    };
    if (t_begin < t_end) stage(0, t_begin);
    for (int64_t t = t_begin; t < t_full; t += 2) {
      one_tile(0, t, std::false_type());
      if (t + 1 < t_full) one_tile(1, t + 1, std::false_type());
    }
    if constexpr (!COLS) {
      if (t_full < t_end) one_tile((int)(t_full - t_begin) & 1, t_full, std::true_type());
    }
    if constexpr (!COLS) __builtin_amdgcn_s_setprio(0);
    __syncthreads();   // the tiles may be filled again
  };
  const auto mask = [&](f32x16 (&S)[XT], int left) {   // the rows past the vocabulary's end
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if ((i >> 2) * 8 + h * 4 + (i & 3) >= left)
#pragma unroll
        for (int xt = 0; xt < XT; ++xt) S[xt][i] = neg_inf();
  };
  const auto largest = [&](const f32x16 (&S)[XT]) {
#pragma unroll
    for (int xt = 0; xt < XT; ++xt) {
      float v = S[xt][0];
#pragma unroll
      for (int i = 1; i < 16; ++i) v = fmaxf(v, S[xt][i]);
      m[xt] = fmaxf(m[xt], fmaxf(v, __shfl_xor(v, 32)) * a.scale);
    }
  };

  if constexpr (!COLS) {
    // The exponents' reference: the largest of the share's first 32 scores.
    if (t_begin < t_end) {
      stage(0, t_begin);
      __builtin_amdgcn_s_waitcnt(0xF70);
      __syncthreads();
      f32x16 S[XT];
      scores<RP, XT>(lds, at, X, S);
      mask(S, (int)min(a.ny - t_begin * TY, (int64_t)32));
      largest(S);
      __syncthreads();
    }
  }
  for (int attempt = 0;; ++attempt) {
#pragma unroll
    for (int xt = 0; xt < XT; ++xt) {
      l[xt] = odd[xt] = 0.f;
      if constexpr (!COLS) {
#pragma unroll
        for (int rt = 0; rt < (ACC ? RT : 1); ++rt) acc[xt][rt] = f32x16{};
      }
    }
    each_subtile([&](const uint16_t* tile, const float* row_c, const float* row_s, auto left) {
      f32x16 S[XT];
      // A wave's matrix instructions go before the other's vector instructions:
      // the two fall out of step sooner and wait less for the same unit (rows
      // pass, r = 128: 307 -> 295 us; the columns pass gains nothing, and
      // spills at r = 256).
      if constexpr (!COLS) __builtin_amdgcn_s_setprio(1);
      scores<RP, XT>(tile, at, X, S);
      if constexpr (!COLS) __builtin_amdgcn_s_setprio(0);
      uint32_t sign[8];
      if constexpr (COLS) {
        f32x4 c[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) c[g] = *reinterpret_cast<const f32x4*>(&row_c[g * 8 + h * 4]);
#pragma unroll
        for (int xt = 0; xt < XT; ++xt)
#pragma unroll
          for (int i = 0; i < 16; ++i) S[xt][i] = exp2_hw(fmaf(S[xt][i], a.scale, -c[i >> 2][i & 3]));
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          typedef float f32x2 __attribute__((ext_vector_type(2)));
          const f32x2 w = *reinterpret_cast<const f32x2*>(row_s + g * 4 + h * 2);
          sign[g * 2] = __float_as_uint(w[0]);
          sign[g * 2 + 1] = __float_as_uint(w[1]);
        }
      } else {
        if constexpr (!std::is_same_v<decltype(left), std::integral_constant<int, 32>>) mask(S, left);
#pragma unroll
        for (int xt = 0; xt < XT; ++xt)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            S[xt][i] = exp2_hw(fmaf(S[xt][i], a.scale, -m[xt]));
            (i & 1 ? odd : l)[xt] += S[xt][i];
          }
      }
      if constexpr (ACC) {
        // E as the right operand. It is rounded to bf16 here (off by at most
        // 2^-8 of itself, nearest even; q_lost makes it good where a
        // teacher's p is taken from it); products and sums stay in fp32.
#pragma unroll
        for (int s2 = 0; s2 < 2; ++s2) {
          bf16x8 E[XT];
          if (!COLS && s2 == 0) __builtin_amdgcn_s_setprio(1);
#pragma unroll
          for (int xt = 0; xt < XT; ++xt) {
            u32x4 v;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              v[i] = pack_bf16(S[xt][s2 * 8 + i * 2], S[xt][s2 * 8 + i * 2 + 1]);
              if constexpr (COLS) v[i] ^= sign[s2 * 4 + i];
            }
            E[xt] = __builtin_bit_cast(bf16x8, v);
          }
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            const bf16x8 A = columns<RP>(tile + s2 * 16 * RP, at, rt);
#pragma unroll
            for (int xt = 0; xt < XT; ++xt)
              acc[xt][rt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(A, E[xt], acc[xt][rt], 0, 0, 0);
          }
        }
      }
    });
    if constexpr (COLS) break;
    // A sum within its limit shows that no exponential passed it (they are
    // all positive). Past it, the share is done once more, from its largest
    // score.
    bool over = false;
#pragma unroll
    for (int xt = 0; xt < XT; ++xt) {
      l[xt] += odd[xt];
      over |= !(l[xt] <= kMostSum);
    }
    if (attempt || !__syncthreads_or(over)) break;
    each_subtile([&](const uint16_t* tile, const float*, const float*, auto left) {
      f32x16 S[XT];
      scores<RP, XT>(tile, at, X, S);
      mask(S, left);
      largest(S);
    });
    if constexpr (WY > 1) {   // the waves of a row keep one reference
      float* top = reinterpret_cast<float*>(lds);   // [wy][row of the block]
#pragma unroll
      for (int xt = 0; xt < XT; ++xt) {
        const int x = (wx * XT + xt) * 32 + (lane & 31);
        top[wy * (WX * 32 * XT) + x] = m[xt];   // (both halves of the wave hold it)
      }
      __syncthreads();
#pragma unroll
      for (int xt = 0; xt < XT; ++xt) {
        const int x = (wx * XT + xt) * 32 + (lane & 31);
#pragma unroll
        for (int y = 0; y < WY; ++y) m[xt] = fmaxf(m[xt], top[y * (WX * 32 * XT) + x]);
      }
      __syncthreads();
    }
  }

  uint16_t* const scratch = lds + wave * (bf16_lds_bytes<RP, WX>() / 2 / kWaves / 16 * 16);
  constexpr int kFit = bf16_lds_bytes<RP, WX>() / kWaves / 32;   // bytes of a row that fit the scratch
  constexpr int kOut2 = kFit >= RP * 2 ? RP : kFit >= RP ? RP / 2 : RP / 4;
  constexpr int kOut4 = kFit >= RP * 4 ? RP : kFit >= RP * 2 ? RP / 2 : RP / 4;
  if constexpr (COLS) {
    // The group's chunks (here and not before the dense part, where X needs the registers).
    const Listed all(a.list_start[xtile], a.list_start[xtile + 1], a.chunk_bits);
    const uint32_t parts = min(all.c1 - all.c0, most_parts(RP));
    for (uint32_t c = share_of(parts, split, splits); c < share_of(parts, split + 1, splits); ++c)
      each_quad<RP, XT>(all.c0 + (int)c, wave, acc, [&](f32x16& v, int g, int64_t at) {
        const f32x4 q = *reinterpret_cast<const f32x4*>(a.chunk_part + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[g * 4 + i] += q[i];
      });
#pragma unroll
    for (int xt = 0; xt < XT; ++xt) {
      const int64_t x = x0 + xt * 32;
      const int have = (int)min(a.nx - x, (int64_t)32);
      const int64_t first = a.whole * (WX * 32 * XT);
      if (splits > 1)
        store_rows<RP, kOut4>(acc[xt], scratch, a.part + ((int64_t)split * (a.nx - first) + x - first) * RP, RP, have, RP);
      else
        store_rows<RP, kOut2>(acc[xt], scratch, static_cast<uint16_t*>(a.dP) + x * a.r, a.r, have, a.r);
    }
  } else {
    if constexpr (WY > 1) {
      // The first wave of each row adds the others' sums to its own, in their
      // order, 16 registers at a time.
      float* sums = reinterpret_cast<float*>(lds);                    // [wy - 1][row]
      f32x4* parts = reinterpret_cast<f32x4*>(sums + (WY - 1) * WX * 32 * XT);   // [wy - 1][wx][quad][lane]
#pragma unroll
      for (int xt = 0; xt < XT; ++xt) {
        l[xt] += __shfl_xor(l[xt], 32);
        const int x = (wx * XT + xt) * 32 + (lane & 31);
        if (wy) sums[(wy - 1) * (WX * 32 * XT) + x] = l[xt];
      }
      __syncthreads();
#pragma unroll
      for (int xt = 0; xt < XT; ++xt) {
        const int x = (wx * XT + xt) * 32 + (lane & 31);
        if (!wy)
#pragma unroll
          for (int y = 0; y < WY - 1; ++y) l[xt] += sums[y * (WX * 32 * XT) + x];
#pragma unroll
        for (int rt = 0; rt < (ACC ? RT : 0); ++rt) {
          if (wy)
#pragma unroll
            for (int g = 0; g < 4; ++g) parts[(((wy - 1) * WX + wx) * 4 + g) * kWave + lane] = quad(acc[xt][rt], g);
          __syncthreads();
          if (!wy)
#pragma unroll
            for (int y = 0; y < WY - 1; ++y)
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                const f32x4 v = parts[((y * WX + wx) * 4 + g) * kWave + lane];
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[xt][rt][g * 4 + i] += v[i];
              }
          __syncthreads();
        }
      }
      if (wy) return;
    }
#pragma unroll
    for (int xt = 0; xt < XT; ++xt) {
      const int64_t x = x0 + xt * 32;
      const float lt = WY > 1 ? l[xt] : l[xt] + __shfl_xor(l[xt], 32);
      if (lane < 32 && x + lane < a.nx) {
        a.pm[(int64_t)split * a.nx + x + lane] = m[xt];
        a.pl[(int64_t)split * a.nx + x + lane] = lt;
      }
      if constexpr (ACC)
        store_rows<RP, kOut4>(acc[xt], scratch, a.po + ((int64_t)split * a.nx + x) * RP, RP,
                              (int)min(a.nx - x, (int64_t)32), RP);
    }
  }
}

// The columns pass for few rows (NS tiles of 32 at most), bf16: bound by the
// reading of P and the writing of dP, so it is laid out for many waves in
// flight rather than for reuse. All rows of Z sit in LDS and all weights of a
// wave's 32 columns in registers; dP then takes shape 32 columns of r at a
// time, which leaves room for a second block (r = 512: one block and 256
// accumulators in the general kernel; 64 rows, 151936 tokens: 173 -> 71 us).
// The teacher's weights are scattered into a table of the wave's columns by
// 16 rows, and join q's in fp32; a wave with any of them takes its weights as
// two bf16 (hi + lo, within 2^-17 of their sum), others as one.
template <int RP, int NS>
__global__ void __launch_bounds__(kWaves* kWave, 2) few_columns_kernel(StreamArgs a) {
  constexpr int TY = NS * 32, KS = RP / 16, RT = RP / 32;
  extern __shared__ __attribute__((aligned(16))) uint16_t lds[];
  const int lane = threadIdx.x & 63, h = lane >> 5, wave = wave_id();
  uint16_t* const scratch = lds + TY * RP + wave * (32 * 32);
  const int64_t x0 = ((int64_t)blockIdx.x * kWaves + wave) * 32;
  const uint32_t e0 = a.list_start[blockIdx.x], count = a.list_start[blockIdx.x + 1] - e0;

  TileCopy<RP, TY> copy;
  copy.init(a.Y, a.ny, RP, RP);
  copy.issue(lds, 0);
  bf16x8 X[KS];
  {
    const int64_t x = x0 + (lane & 31);
    const uint16_t* row = static_cast<const uint16_t*>(a.X) + min(x, a.nx - 1) * a.r;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int c = ks * 16 + h * 8;
      const bool ok = x < a.nx && c < a.r;
      const u32x4 v = load16(row + (ok ? c : 0));
      X[ks] = __builtin_bit_cast(bf16x8, ok ? v : u32x4{0u, 0u, 0u, 0u});
    }
  }
  // Place i of the block: its row and column and its weight, or kNone if it is
  // another wave's. An id that occurs more than once in a row has its
  // entries side by side; the first takes their sum, the others are kNone.
  constexpr uint32_t kNone = ~0u;
  const auto place = [&](uint32_t i) {
    uint2 en = {kNone, 0u};
    if (i >= count) return en;
    en = a.list[e0 + i];
    const uint32_t key = en.x;
    if ((int)(key >> (kRowBits + 5)) != wave || (i && a.list[e0 + i - 1].x == key)) return uint2{kNone, 0u};
    for (uint32_t j = i + 1; j < count && a.list[e0 + j].x == key; ++j)
      en.y = __float_as_uint(__uint_as_float(en.y) + __uint_as_float(a.list[e0 + j].y));
    return en;
  };
  const uint2 first = place(lane);
  const bool have = count > kWave || __ballot(first.x != kNone);
  Places<RP> at;
  at.init();
  __builtin_amdgcn_s_waitcnt(0xF70);
  __syncthreads();

  const auto ordered = [] {   // the wave's LDS writes come before its reads
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };
  bf16x8 E[NS][2], lo[NS][2] = {};
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    f32x16 S[1];
    const bf16x8(&X1)[1][KS] = reinterpret_cast<const bf16x8(&)[1][KS]>(X);
    scores<RP, 1>(lds + s * 32 * RP, at, X1, S);
    float e[16];
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t n = s * 32 + g * 8 + h * 4 + i;   // row_c is padded to 64 rows
        float* rc = const_cast<float*>(a.row_c);
        const float v = exp2_hw(fmaf(S[0][g * 4 + i], a.scale, -*row_c_at(rc, n, a.row_block)));
        e[g * 4 + i] = *row_sign_at(rc, n, a.row_block) ? -v : v;
      }
#pragma unroll
    for (int s2 = 0; s2 < 2; ++s2) {
      if (have) {
        float* table = reinterpret_cast<float*>(scratch);   // [column][row of 16]
#pragma unroll
        for (int i = 0; i < 2; ++i) *reinterpret_cast<f32x4*>(table + (i * kWave + lane) * 4) = f32x4{0.f, 0.f, 0.f, 0.f};
        ordered();
        for (uint32_t i = lane; i < (count + kWave - 1) / kWave * kWave; i += kWave) {
          const uint2 en = i < kWave ? first : place(i);
          const uint32_t row = en.x & kRowMask;
          if (en.x != kNone && row / 16 == (uint32_t)(s * 2 + s2))
            table[((en.x >> kRowBits) & 31) * 16 + row % 16] = __uint_as_float(en.y);
        }
        ordered();
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const f32x4 w = *reinterpret_cast<const f32x4*>(table + (lane & 31) * 16 + g * 8 + h * 4);
#pragma unroll
          for (int i = 0; i < 4; ++i) e[s2 * 8 + g * 4 + i] += w[i];
        }
        ordered();
      }
      u32x4 v, r;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float c0 = e[s2 * 8 + i * 2], c1 = e[s2 * 8 + i * 2 + 1];
        v[i] = pack_bf16(c0, c1);
        r[i] = pack_bf16(c0 - __uint_as_float(v[i] << 16), c1 - __uint_as_float(v[i] & 0xffff0000u));
      }
      E[s][s2] = __builtin_bit_cast(bf16x8, v);
      if (have) lo[s][s2] = __builtin_bit_cast(bf16x8, r);
    }
  }
  const int rows = (int)min(a.nx - x0, (int64_t)32);
  uint16_t* out = static_cast<uint16_t*>(a.dP) + x0 * a.r;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    if (rt * 32 >= a.r) break;
    f32x16 acc[1] = {};
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int s2 = 0; s2 < 2; ++s2) {
        const bf16x8 A = columns<RP>(lds + (s * 32 + s2 * 16) * RP, at, rt);
        acc[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(A, E[s][s2], acc[0], 0, 0, 0);
        if (have) acc[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(A, lo[s][s2], acc[0], 0, 0, 0);
      }
    store_rows<32, 32>(acc, scratch, out + rt * 32, a.r, rows, a.r - rt * 32);
  }
}

// fp32, on v_mfma_f32_16x16x4_f32: a wave owns 16 rows of X, the block 64.
// A tile holds 16 rows of Y, each padded by 4 words so that both reads of
// it (rows as the left operand of S, columns as that of A) spread over the
// banks.
template <int RP, bool ACC, bool COLS>
__global__ void __launch_bounds__(kWaves* kWave, 1) stream_f32_kernel(StreamArgs a) {
  constexpr int TY = 16, LD = RP + 4, KC = RP / 16, RT = RP / 16;
  constexpr int kBufs = RP <= 256 ? 2 : 1;   // as many as fit 64 KB
  __shared__ __attribute__((aligned(16))) float tiles[kBufs][TY * LD];
  const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15, wave = wave_id();
  const bool whole = blockIdx.x < a.whole;
  const int splits = whole ? 1 : a.splits;
  const int64_t xtile = whole ? blockIdx.x : a.whole + (blockIdx.x - a.whole) / splits;
  const int split = whole ? 0 : (int)((blockIdx.x - a.whole) % splits);
  const int64_t x0 = (xtile * kWaves + wave) * 16;
  const int64_t x = x0 + col;
  const float* Yp = static_cast<const float*>(a.Y);

  f32x4 X[KC];
#pragma unroll
  for (int c = 0; c < KC; ++c) {
    const int kk = c * 16 + g * 4;
    X[c] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (x < a.nx && kk < a.r) X[c] = *reinterpret_cast<const f32x4*>(static_cast<const float*>(a.X) + x * a.r + kk);
  }
  f32x4 acc[ACC ? RT : 1] = {};
  float m = neg_inf(), l = 0.f;

  const int64_t nt = (a.ny + TY - 1) / TY;
  const int64_t t_begin = nt * split / splits, t_end = nt * (split + 1) / splits;
  constexpr int kLoads = (TY * RP / 4 + kWaves * kWave - 1) / (kWaves * kWave);
  f32x4 next[kLoads];   // the next tile, on its way during a tile's products
  const auto load = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int p = i * kWaves * kWave + threadIdx.x;
      const int row = p / (RP / 4), c = (p % (RP / 4)) * 4;
      const int64_t y = t * TY + row;
      next[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (row < TY && y < a.ny && c < a.r) next[i] = *reinterpret_cast<const f32x4*>(Yp + y * a.ldy + c);
    }
  };
  if (t_begin < t_end) load(t_begin);
  for (int64_t t = t_begin; t < t_end; ++t) {
    float* const tile = tiles[t % kBufs];
    if constexpr (kBufs == 1) __syncthreads();
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int p = i * kWaves * kWave + threadIdx.x;
      const int row = p / (RP / 4), c = (p % (RP / 4)) * 4;
      if (row < TY) *reinterpret_cast<f32x4*>(tile + row * LD + c) = next[i];
    }
    __syncthreads();   // also: every wave is done with the tile before this one
    if (t + 1 < t_end) load(t + 1);
    const int64_t y0 = t * TY;
    f32x4 S = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < KC; ++c) {
      const f32x4 A = *reinterpret_cast<const f32x4*>(tile + col * LD + c * 16 + g * 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) S = __builtin_amdgcn_mfma_f32_16x16x4f32(A[j], X[c][j], S, 0, 0, 0);
    }
    if constexpr (COLS) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float* rc = const_cast<float*>(a.row_c);   // padded past ny
        const float e = exp2_hw(fmaf(S[i], a.scale, -*row_c_at(rc, (uint32_t)(y0 + g * 4 + i), kRowBlock)));
        S[i] = *row_sign_at(rc, (uint32_t)(y0 + g * 4 + i), kRowBlock) ? -e : e;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (y0 + g * 4 + i >= a.ny) S[i] = neg_inf();
      const float top = fmaxf(fmaxf(S[0], S[1]), fmaxf(S[2], S[3])) * a.scale;
      if (__ballot(top > m)) {
        float mn = fmaxf(top, __shfl_xor(top, 16));
        mn = fmaxf(m, fmaxf(mn, __shfl_xor(mn, 32)));
        const float s = mn == m ? 1.f : exp2_hw(m - mn);
        m = mn;
        l *= s;
        if constexpr (ACC) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) acc[rt] *= s;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) S[i] = exp2_hw(fmaf(S[i], a.scale, -m));
      l += (S[0] + S[1]) + (S[2] + S[3]);
    }
    if constexpr (ACC) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[rt] = __builtin_amdgcn_mfma_f32_16x16x4f32(tile[(g * 4 + i) * LD + rt * 16 + col], S[i], acc[rt], 0, 0, 0);
    }
  }

  if constexpr (COLS) {
    if (x0 < a.nx) {
      const uint32_t first = a.list_start[x0 / 16], places = a.list_start[x0 / 16 + 1] - first;
      const uint32_t e1 = first + share_of(places, split + 1, splits);
      uint32_t e0 = first + share_of(places, split, splits);
      // Sixteen places a step, four to a product; the next step's are on their way.
      uint2 en[4] = {};
      const auto take = [&] {
#pragma unroll
        for (int u = 0; u < 4; ++u) en[u] = a.list[min(e0 + u * 4 + g, e1 - 1)];
      };
      if (e0 < e1) take();
      while (e0 < e1) {
        float B[4];
        const float* z[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const bool mine = e0 + u * 4 + g < e1 && (int)(en[u].x >> kRowBits) == col;
          B[u] = mine ? __uint_as_float(en[u].y) : 0.f;
          z[u] = Yp + (int64_t)(en[u].x & kRowMask) * a.ldy + col;
        }
        e0 += 16;
        if (e0 < e1) take();
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          float A[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) A[u] = z[u][rt * 16];
#pragma unroll
          for (int u = 0; u < 4; ++u) acc[rt] = __builtin_amdgcn_mfma_f32_16x16x4f32(A[u], B[u], acc[rt], 0, 0, 0);
        }
      }
    }
    if (x >= a.nx) return;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int c = rt * 16 + g * 4;
      const int64_t first = a.whole * (kWaves * 16);
      if (splits > 1)
        *reinterpret_cast<f32x4*>(a.part + ((int64_t)split * (a.nx - first) + x - first) * RP + c) = acc[rt];
      else if (c < a.r) *reinterpret_cast<f32x4*>(static_cast<float*>(a.dP) + x * a.r + c) = acc[rt];
    }
  } else {
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (x >= a.nx) return;
    if (g == 0) {
      a.pm[(int64_t)split * a.nx + x] = m;
      a.pl[(int64_t)split * a.nx + x] = l;
    }
    if constexpr (ACC) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
        *reinterpret_cast<f32x4*>(a.po + ((int64_t)split * a.nx + x) * RP + rt * 16 + g * 4) = acc[rt];
    }
  }
}

// ----------------------------------------------------------- teacher places

template <typename T> __device__ __forceinline__ float widen(T x);
template <> __device__ __forceinline__ float widen<uint16_t>(uint16_t x) { return bf16_to_f32(x); }
template <> __device__ __forceinline__ float widen<float>(float x) { return x; }

__device__ __forceinline__ float dot8(const float* a, const float* b, float acc) {
#pragma unroll
  for (int i = 0; i < 8; ++i) acc = fmaf(a[i], b[i], acc);
  return acc;
}

// The scores of up to 32 TILES places against the row z, bit for bit as the
// streaming passes make them: the same instruction over the same 16 columns
// at a time. (An element of its result depends on its own row and column alone,
// wherever they sit and whichever operand they are.) Lanes l and l + 32 give the ids
// of places l, l + 32, .. (INT_MAX: none, score 0); place l + 32 t's score
// is got[t] of lane l. The whole wave takes part, but z is read once only, as the
// one row of the left operand.
template <int TILES, int kAhead>
__device__ __forceinline__ void place_scores(const uint16_t* __restrict__ P, const uint16_t* __restrict__ z, int r,
                                             const int (&id)[TILES], float (&got)[TILES]) {
  const int h = (threadIdx.x & 63) >> 5, x = threadIdx.x & 31;
  f32x16 S[TILES];
#pragma unroll
  for (int t = 0; t < TILES; ++t) S[t] = f32x16{};
  for (int c0 = 0; c0 < r; c0 += kAhead * 16) {
    u32x4 A[kAhead], B[TILES][kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int c = c0 + i * 16 + h * 8;
      A[i] = u32x4{0u, 0u, 0u, 0u};
      if (x == 0 && c < r) A[i] = load16(z + c);
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        B[t][i] = u32x4{0u, 0u, 0u, 0u};
        if (c < r && id[t] != INT_MAX) B[t][i] = load16(P + (int64_t)id[t] * r + c);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
#pragma unroll
      for (int t = 0; t < TILES; ++t)
        S[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, A[i]),
                                                       __builtin_bit_cast(bf16x8, B[t][i]), S[t], 0, 0, 0);
  }
#pragma unroll
  for (int t = 0; t < TILES; ++t) got[t] = S[t][0];
}

// What the rounding of a weight q to bf16 takes away from it (exact in fp32).
// The gradients are sums of q - p. Away from the teacher's places the rounding is
// 2^-8 of a term at most; at them it would be 2^-8 of q, however small q - p is
// (512 rows whose teacher is the student's own top 32, q = 0.55 and losses of
// 0.022: dP and dZ off by 7.1 and 4.7% in norm, 0.17% with it, which is the bf16
// results' own). So the places' weights are p - q_lost: N k scores made once
// more, and what the streams add up to is q - p in fp32.
__device__ __forceinline__ float q_lost(float q) { return q - __uint_as_float(pack_bf16(q, 0.f) << 16); }

// The teacher's distribution over a row's places, lane j holding place j's id
// (any, outside [0, V) past k) and logit: a place is empty (p = 0, id =
// INT_MAX) when its id lies outside [0, V) or its logit is NaN or -inf. logp
// is log p where p > 0. Returns whether the row has a place at all. The
// largest logit is taken away before the division by T, whose result alone may
// have no place in fp32 (T < 1, logits at the type's lowest value). The
// exponent is taken in two parts: log2(e) rounded to fp32 alone would be off
// by 1e-8 of it.
__device__ __forceinline__ bool teacher(int64_t V, float inv_t, int& id, float x, float& p, float& logp) {
  const bool real = id >= 0 && id < V && x > neg_inf();
  const uint32_t mk = wave_max_u32(real ? order_key(x) : 0u);
  if (!real) id = INT_MAX;
  p = 0.f;
  logp = 0.f;
  if (!mk) return false;
  const float d = (x - __uint_as_float(order_key_inv(mk))) * inv_t;
  const float e = real ? exp2_hw(fmaf(d, kLog2e, d * kLog2eLo)) : 0.f;
  const float s = group_sum<kWave>(e);
  p = e / s;
  if (p > 0.f) logp = d - log2_hw(s) * kLn2;
  return true;
}

// Joins the shares of the rows pass. A block takes one row and 4 L of its
// columns: L lanes hold 4 columns each, and 256 / L such groups share out the
// shares of the weighted sum and the teacher's places. The first block of a
// row also writes its lse and loss. What bounds it is the chain of dependent
// loads (shares' maxima, ids, the ids' rows), so a row gets as few blocks as
// its columns allow (49 us with four blocks a row at 2048 rows, r = 256, 40 with
// one), the first sums are on their way before their weights are made, and the
// registers leave room for five blocks a compute unit (4096 rows, r = 128, 16 shares:
// 35 us with four, 30 with five; the scores made again are 10 of them).
template <typename T, int L>
__global__ void __launch_bounds__(kWaves* kWave, sizeof(T) == 2 ? 5 : 3) distill_finish_kernel(
    const T* __restrict__ Z, const T* __restrict__ P, const int32_t* __restrict__ idx, const float* __restrict__ t,
    int64_t N, int64_t V, int r, int RP, int k, float inv_t, float scale, int ty_bits, int shares,
    const float* __restrict__ pm, const float* __restrict__ pl, const float* __restrict__ po, float* __restrict__ loss,
    float* __restrict__ lse, float* __restrict__ G) {
  __shared__ float sp[kWave], sdot[kWave], lost[kWave], red[kWaves * 2], share_w[kMaxShares];
  __shared__ __attribute__((aligned(16))) int sid[kWave];
  constexpr int kGroups = kWaves * kWave / L, kJoinCols = 4 * L;
  __shared__ f32x4 part[kGroups][L];
  const int chunks = G ? (r + kJoinCols - 1) / kJoinCols : 1;
  const int64_t n = blockIdx.x / chunks;
  const int chunk = blockIdx.x % chunks;
  const int tid = threadIdx.x, wave = wave_id(), lane = tid & 63;
  const int group = tid / L, sub = tid % L;
  const int c = chunk * kJoinCols + sub * 4;
  const bool sums = G && c < r;
  int id = lane < k ? idx[n * k + lane] : -1;
  const float tl = lane < k ? t[n * k + lane] : 0.f;
  float m = neg_inf();
  for (int s = tid; s < shares; s += kWaves * kWave) m = fmaxf(m, pm[(int64_t)s * N + n]);
  // the first shares' sums, on their way while their weights are made
  constexpr int kAhead = 16 / kGroups;
  f32x4 early[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int s = group + i * kGroups;
    early[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (sums && s < shares) early[i] = *reinterpret_cast<const f32x4*>(po + ((int64_t)s * N + n) * RP + c);
  }
  float p, logp;
  const bool any = teacher(V, inv_t, id, tl, p, logp);   // every wave: the same values
  if (wave == 0) {
    sid[lane] = id;
    sp[lane] = p;
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  if (lane == 0) red[wave] = m;
  __syncthreads();
  m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  float l = 0.f;
  for (int s = tid; s < shares; s += kWaves * kWave) {
    const float ps = pl[(int64_t)s * N + n];
    const float w = ps != 0.f ? exp2_hw(pm[(int64_t)s * N + n] - m) : 0.f;   // a share without rows has sum 0
    share_w[s] = w;
    l = fmaf(ps, w, l);
  }
  l = group_sum<kWave>(l);
  if (lane == 0) red[kWaves + wave] = l;
  if constexpr (sizeof(T) == 2) {   // the places' scores, and what their q have lost
    if (wave < k) {   // of place 4 j + w in lane j of wave w
      const int j = (lane & 15) * kWaves + wave;
      const int v[1] = {(lane & 31) < 16 ? sid[j] : INT_MAX};
      // the share that the id's tile belongs to, and its reference
      const double tiles = (double)((V + (1 << ty_bits) - 1) >> ty_bits);
      float ref = 0.f;
      if (v[0] != INT_MAX) {
        const int64_t share = (int64_t)((double)(((int64_t)(v[0] >> ty_bits) + 1) * shares - 1) / tiles);
        ref = pm[share * N + n];
      }
      float s[1];
      place_scores<1, 4>(P, Z + n * r, r, v, s);
      // An id that occurred before: q is in the sum once. Lanes 16 apart look through 16 places each.
      int again = 0;
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const u32x4 o = load16(sid + (lane & 48) + i);
#pragma unroll
        for (int u = 0; u < 4; ++u) again |= (int)o[u] == sid[j] && (lane & 48) + i + u < j;
      }
      again |= __shfl_xor(again, 16);
      again |= __shfl_xor(again, 32);
      if (lane < 16) {
        sdot[j] = s[0];
        lost[j] = again ? 0.f : q_lost(exp2_hw(fmaf(s[0], scale, -ref))) * exp2_hw(ref - m);
      }
    }
  } else if (chunk == 0) {   // the places' scores: 16 lanes per place
    for (int j = tid / 16; j < k; j += kWaves * 4) {
      const int v = sid[j];
      float d = 0.f;
      if (v != INT_MAX)
        for (int e = tid % 16 * 8; e < r; e += 128) d = dot8(P + (int64_t)v * r + e, Z + n * r + e, d);
      d = group_sum<16>(d);
      if (tid % 16 == 0) sdot[j] = d;
    }
  }
  constexpr int kPlaces = kWave / kGroups;   // of a group: k <= 64
  T places[kPlaces][4];
#pragma unroll
  for (int i = 0; i < kPlaces; ++i) {
    const int v = sid[group + i * kGroups];
    const T* q = P + (sums && v != INT_MAX ? (int64_t)v * r + c : 0);
    __builtin_memcpy(places[i], __builtin_assume_aligned(q, 4 * sizeof(T)), 4 * sizeof(T));
  }
  __syncthreads();
  l = (red[kWaves] + red[kWaves + 1]) + (red[kWaves + 2] + red[kWaves + 3]);
  if (chunk == 0 && wave == 0) {
    const float ls = (m + log2_hw(l)) * kLn2;
    const float s = lane < k && p > 0.f ? sdot[lane] * inv_t : 0.f;
    const float e = group_sum<kWave>(p > 0.f ? p * (logp - s + ls) : 0.f);
    if (lane == 0) {
      lse[n] = ls;
      loss[n] = any ? e : 0.f;
    }
  }
  if (!G) return;
  const float il = 1.f / l;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  if (sums) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int s = group + i * kGroups;
      const float w = s < shares ? share_w[s] : 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = w != 0.f ? fmaf(early[i][e], w, o[e]) : o[e];
    }
#pragma unroll 8
    for (int s = group + kAhead * kGroups; s < shares; s += kGroups) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(po + ((int64_t)s * N + n) * RP + c);
      const float w = share_w[s];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = w != 0.f ? fmaf(v[e], w, o[e]) : o[e];
    }
    o *= il;
#pragma unroll
    for (int i = 0; i < kPlaces; ++i) {
      const int j = group + i * kGroups;
      const bool real = sid[j] != INT_MAX;
      const float w = sizeof(T) == 2 ? fmaf(lost[j], il, -sp[j]) : -sp[j];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = real ? fmaf(w, widen<T>(places[i][e]), o[e]) : o[e];
    }
  }
  part[group][sub] = o;
  __syncthreads();
  if (group == 0 && c < r) {
#pragma unroll
    for (int g = 1; g < kGroups; ++g) o += part[g][sub];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = any ? o[i] * inv_t : 0.f;
    *reinterpret_cast<f32x4*>(G + n * r + c) = o;
  }
}

// Per row, before the columns pass: the exponent's offset and the sign of the
// weight, the row of Z (zeros without weight, so that what a masked row holds,
// NaN included, cannot reach dP), the places in ascending order of their ids
// with w p / T (less what the columns pass rounds away of w q / T, if P is given),
// and dZ = w G. One wave per row, all its loads but the places' rows up front.
template <typename T>
__global__ void __launch_bounds__(kWaves* kWave) distill_prep_kernel(
    const T* __restrict__ Z, const T* __restrict__ P, float scale, const int32_t* __restrict__ idx,
    const float* __restrict__ t, const float* __restrict__ lse, const float* __restrict__ G,
    const float* __restrict__ weight, int N, int64_t V, int r, int RP, int k, float inv_t, T* __restrict__ zc,
    float* __restrict__ row_c, int RB, int* __restrict__ srt_id, float* __restrict__ srt_w, T* __restrict__ dZ) {
  const int n = blockIdx.x * kWaves + wave_id();
  const int lane = threadIdx.x & 63;
  const int at = lane * 8;   // 8 columns a lane: r <= 512
  if (n >= N) {   // the last tile's rows past N
    if (zc && lane == 0) {
      *row_c_at(row_c, n, RB) = __builtin_inff();
      *row_sign_at(row_c, n, RB) = 0;
    }
    return;
  }
  const int64_t place = (int64_t)n * k + lane, elem = (int64_t)n * r + at;
  int id = lane < k ? idx[place] : -1;
  const float tl = lane < k ? t[place] : 0.f;
  const float w = weight ? weight[n] : 1.f;
  const float ls = lse[n];
  f32x4 g[2] = {};
  if (dZ && at < r) {
    g[0] = reinterpret_cast<const f32x4*>(G + elem)[0];
    g[1] = reinterpret_cast<const f32x4*>(G + elem)[1];
  }
  T z[8] = {};
  if (zc && at < r) __builtin_memcpy(z, __builtin_assume_aligned(Z + elem, 16), sizeof(z));

  float p, logp;
  const bool live = teacher(V, inv_t, id, tl, p, logp) && w != 0.f;
  const float c = w * inv_t;
  if (dZ && at < r) {
    T v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = store_cast<T>(live ? w * g[i >> 2][i & 3] : 0.f);
    __builtin_memcpy(__builtin_assume_aligned(dZ + elem, 16), v, sizeof(v));
  }
  if (!zc) return;
  if (at < RP) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = live ? z[i] : T(0);
    __builtin_memcpy(__builtin_assume_aligned(zc + (int64_t)n * RP + at, 16), z, sizeof(z));
  }
  // |c| may be subnormal: log2 of 2^64 |c| is not (and would not be finite for large ones)
  const bool small = fabsf(c) < 0x1p-64f;
  const float lc = log2_hw(small ? fabsf(c) * 0x1p64f : fabsf(c)) - (small ? 64.f : 0.f);
  const float offset = live ? ls * kLog2e - lc : __builtin_inff();
  if (lane == 0) {
    *row_c_at(row_c, n, RB) = offset;
    *row_sign_at(row_c, n, RB) = live && c < 0.f ? 0x8000 : 0;
  }
  const float wt = p * c;
  if (!live) id = INT_MAX;
  float lost = 0.f;
  if constexpr (sizeof(T) == 2) {
    if (P && live) {
      const int v[2] = {__shfl(id, lane & 31), __shfl(id, 32 + (lane & 31))};
      float got[2] = {};
      if (k > 32) place_scores<2, 4>(P, Z + (int64_t)n * r, r, v, got);
      else place_scores<1, 8>(P, Z + (int64_t)n * r, r, {v[0]}, reinterpret_cast<float(&)[1]>(got));
      const float behind = __shfl(got[1], lane & 31);
      const float s = lane < 32 ? got[0] : behind;
      lost = copysignf(1.f, c) * q_lost(exp2_hw(fmaf(s, scale, -offset)));
    }
  }
  int rank = 0;
  bool again = false;   // an id that occurred before: q is in the sum once
  for (int j = 0; j < k; ++j) {
    const int o = __builtin_amdgcn_readlane(id, j);
    rank += o < id || (o == id && j < lane);
    again |= o == id && j < lane;
  }
  if (lane < k) {
    srt_id[(int64_t)n * k + rank] = id;
    srt_w[(int64_t)n * k + rank] = again ? wt : wt - lost;
  }
}

// Byte g % 4 of table[g / 4][n]: how many of row n's places have an id below
// g * GC (g = 0 .. groups). A block takes 64 rows, their sorted ids in LDS; a
// wave walks up them, one lane per row, over a range of column groups.
constexpr int kTableWords = 4;   // words per wave
__global__ void __launch_bounds__(kWaves* kWave) distill_table_kernel(const int* __restrict__ srt_id, int N, int npad,
                                                                      int k, int GC, int64_t words, int row_blocks,
                                                                      uint32_t* __restrict__ table) {
  __shared__ int ids[kWave * (kWave + 1)];
  const int n0 = (int)(blockIdx.x % row_blocks) * kWave;
  const int rows = min(N - n0, kWave);
  const int lane = threadIdx.x & 63, wave = wave_id();
  int v[kWave / kWaves];
#pragma unroll
  for (int i = 0; i < kWave / kWaves; ++i) {
    const int row = i * kWaves + wave;
    v[i] = row < rows && lane < k ? srt_id[(int64_t)(n0 + row) * k + lane] : 0;
  }
#pragma unroll
  for (int i = 0; i < kWave / kWaves; ++i) ids[(i * kWaves + wave) * (kWave + 1) + lane] = v[i];
  __syncthreads();
  const int64_t w0 = ((int64_t)(blockIdx.x / row_blocks) * kWaves + wave) * kTableWords;
  const int* id = ids + lane * (kWave + 1);
  const int have = lane < rows ? k : 0;
  int j = 0, hi = have;
  while (j < hi) {   // first place at or above the range
    const int mid = (j + hi) >> 1;
    if (id[mid] < w0 * 4 * GC && id[mid] != INT_MAX) j = mid + 1;
    else hi = mid;
  }
  int next = j < have ? id[j] : INT_MAX;
  for (int64_t w = w0; w < min(w0 + kTableWords, words); ++w) {
    uint32_t v = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      while (next < (w * 4 + b) * GC && next != INT_MAX) {
        ++j;
        next = j < have ? id[j] : INT_MAX;
      }
      v |= (uint32_t)j << (8 * b);
    }
    table[w * npad + n0 + lane] = v;
  }
}

// A place's weight as the columns pass takes it: fp32, or (bf16, many rows)
// two bf16 that add up to it.
__device__ __forceinline__ uint32_t place_weight(float w, bool pairs) {
  if (!pairs) return __float_as_uint(w);
  const uint16_t hi = f32_to_bf16(w);
  return hi | (uint32_t)f32_to_bf16(w - bf16_to_f32(hi)) << 16;
}

// The places of each group of GC columns, ascending by row: a block per group,
// 8 rows a thread. The number of places below a group, summed over the rows,
// is where its list starts.
constexpr int kListWaves = 8, kListRows = kListWaves * kWave * 8;
__global__ void __launch_bounds__(kListWaves* kWave) distill_list_kernel(
    const uint32_t* __restrict__ table, const int* __restrict__ srt_id, const float* __restrict__ srt_w, int npad,
    int k, int GC, bool pairs, int bits, uint32_t chunks, uint32_t* __restrict__ start,
    uint2* __restrict__ list, uint32_t* __restrict__ chunk_in) {
  __shared__ uint32_t below[kListWaves], scan[kListWaves];
  const int64_t g = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int lo_bit = (int)(g & 3) * 8, hi_bit = (int)((g + 1) & 3) * 8;
  const uint32_t* lo = table + (g >> 2) * npad;
  const uint32_t* hi = table + ((g + 1) >> 2) * npad;
  uint32_t at = 0;
  for (int n = threadIdx.x * 4; n < npad; n += kListWaves * kWave * 4) {
    const u32x4 v = load16(lo + n);
#pragma unroll
    for (int q = 0; q < 4; ++q) at += (v[q] >> lo_bit) & 255;
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) at += (uint32_t)__shfl_xor((int)at, o);
  if (lane == 0) below[wave] = at;
  __syncthreads();
  at = 0;
#pragma unroll
  for (int w = 0; w < kListWaves; ++w) at += below[w];
  const uint32_t begin = at;
  if (threadIdx.x == 0) start[g] = at;
  for (int n0 = 0; n0 < npad; n0 += kListRows) {
    const int n = n0 + threadIdx.x * 8;
    uint32_t first[8], last[8];   // the rows' places in this group
    uint32_t mine = 0;
#pragma unroll
    for (int q = 0; q < 8; q += 4) {
      u32x4 a = {0u, 0u, 0u, 0u}, b = a;
      if (n < npad) {
        a = load16(lo + n + q);
        b = load16(hi + n + q);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        first[q + i] = (a[i] >> lo_bit) & 255;
        last[q + i] = (b[i] >> hi_bit) & 255;
        mine += last[q + i] - first[q + i];
      }
    }
    const uint32_t incl = wave_incl_scan_u32(mine);
    __syncthreads();
    if (lane == 63) scan[wave] = incl;
    __syncthreads();
    uint32_t o = at + incl - mine;
#pragma unroll
    for (int w = 0; w < kListWaves; ++w) {
      o += w < wave ? scan[w] : 0u;
      at += scan[w];
    }
    if (!mine) continue;
    // most rows have one place here or none: its loads for all 8 rows at once
    int id[8];
    float wt[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int64_t i = first[q] < last[q] ? (int64_t)(n + q) * k + first[q] : 0;
      id[q] = srt_id[i];
      wt[q] = srt_w[i];
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (first[q] < last[q])
        list[o++] = uint2{(uint32_t)(n + q) | (uint32_t)(id[q] - g * GC) << kRowBits, place_weight(-wt[q], pairs)};
      for (uint32_t j = first[q] + 1; j < last[q]; j += 2) {   // two at a time
        int jd[2];
        float jw[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int64_t i = (int64_t)(n + q) * k + min(j + u, last[q] - 1);
          jd[u] = srt_id[i];
          jw[u] = srt_w[i];
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (j + u < last[q])
            list[o++] = uint2{(uint32_t)(n + q) | (uint32_t)(jd[u] - g * GC) << kRowBits, place_weight(-jw[u], pairs)};
      }
    }
  }
  // the chunks that begin here: `at` is the list's end by now
  for (uint32_t c = ((begin + (1u << bits) - 1) >> bits) + threadIdx.x; c < chunks && c << bits < at;
       c += kListWaves * kWave)
    chunk_in[c] = (c + 1) << bits <= at ? (begin + (1u << bits) - 1) >> bits | (at >> bits) << 16 : 0u;
  if (g == (int64_t)gridDim.x - 1 && threadIdx.x == 0) start[g + 1] = at;
}

// dP of the rows that the columns pass split: the sum of the shares, in their
// order. rows, dP: from the first such row.
template <typename T>
__global__ void __launch_bounds__(256) distill_join_kernel(const float* __restrict__ part, int splits, int rows,
                                                           int r, int RP, T* __restrict__ dP) {
  const uint32_t i = (blockIdx.x * 256 + threadIdx.x) * 4;   // r is a multiple of 8
  const uint32_t v = i / (uint32_t)RP, c = i % (uint32_t)RP;
  if (v >= (uint32_t)rows || c >= (uint32_t)r) return;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int p = 0; p < splits; ++p) s += *reinterpret_cast<const f32x4*>(part + ((int64_t)p * rows + v) * RP + c);
  T o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = store_cast<T>(s[e]);
  __builtin_memcpy(__builtin_assume_aligned(dP + (int64_t)v * r + c, sizeof(o)), o, sizeof(o));
}

__global__ void __launch_bounds__(256) distill_zero_kernel(uint32_t* __restrict__ p, int64_t words) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < words; i += (int64_t)gridDim.x * 256) p[i] = 0;
}

// ---------------------------------------------------------------- host side

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
int round_rank(int r) { return r <= 32 ? 32 : r <= 64 ? 64 : r <= 128 ? 128 : r <= 256 ? 256 : 512; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int kTargetBlocks = 512;   // two blocks per compute unit

struct Plan {
  int RP;
  bool few;          // the columns pass for few rows
  int XT, WX;        // rows pass
  int TY;            // rows of P of a tile of the rows pass
  int row_splits;    // blocks along Y
  int GC;            // columns pass: columns of a group (bf16: a block, fp32: a wave)
  int64_t groups;
  int64_t col_whole; // blocks of the columns pass over all rows
  int col_splits;    // shares of the rows for the others
  int64_t split_rows;   // their rows of P
  int RB;            // rows of a tile of the columns pass
  int64_t npad;
  int chunk_bits;    // log2 of the places of a chunk of the list
  int64_t chunks;    // whole ones, at most
  // workspace offsets
  size_t pm, pl, po, fwd_total;
  size_t zc, row_c, srt_id, srt_w, table, start, list, part, chunk_in, chunk_part, bwd_total;
};

Plan plan(int dtype, int64_t V, int r, int64_t N, int k) {
  Plan p{};
  const size_t es = dtype == 0 ? 2 : 4;
  p.RP = round_rank(r);
  int64_t xblocks, ytiles, cblocks;
  if (dtype == 0) {
    p.XT = x_tiles(p.RP);
    p.WX = N <= 32 * p.XT && p.RP < 256 ? 1 : N <= 64 * p.XT ? 2 : 4;
    xblocks = ceil_div(N, p.WX * 32 * p.XT);
    p.TY = std::max(p.RP <= 128 ? 64 : 32, 32 * (kWaves / p.WX));
    p.few = N <= 64;
    p.GC = kWaves * 32 * (p.few ? 1 : p.XT);
  } else {
    p.XT = 1;
    p.WX = 4;
    xblocks = ceil_div(N, 64);
    p.TY = 16;
    p.GC = 16;
  }
  ytiles = ceil_div(V, p.TY);
  p.RB = dtype == 0 && p.RP > 128 ? 32 : 64;
  const int64_t slots = p.RP == 512 && dtype == 0 ? kTargetBlocks / 2 : kTargetBlocks;   // blocks at a time
  p.row_splits = (int)std::max<int64_t>(1, std::min<int64_t>({slots / xblocks, ytiles, kMaxShares}));
  p.groups = ceil_div(V, p.GC);
  cblocks = dtype == 0 ? p.groups : ceil_div(p.groups, kWaves);
  // The blocks of P's rows that do not fill the GPU once more share out the
  // rows of Z between them, down to about two tiles a share. (At 4096 rows,
  // r = 128, 1187 blocks of which 512 run at a time: 333 us with the last 163
  // in three shares and 7 for joining them, 345 without.)
  // In fp32 four blocks fit a compute unit up to r = 128 (2000 rows, 20000
  // tokens, r = 64: 313 blocks, 229 us whole and 126 + 5 in three shares).
  const int64_t ntiles = ceil_div(N, p.RB);
  const int64_t col_slots = dtype != 0 && p.RP <= 128 ? 2 * slots : slots;
  p.col_whole = cblocks / col_slots * col_slots;
  const int64_t rest = cblocks - p.col_whole;
  p.col_splits = rest ? (int)std::max<int64_t>(1, std::min<int64_t>(col_slots / rest, ntiles / 2)) : 1;
  if (p.few) p.col_splits = 1;
  if (p.col_splits == 1) p.col_whole = cblocks;
  p.split_rows = V - std::min(V, p.col_whole * (dtype == 0 ? p.GC : 64));
  p.npad = ceil_div(N, 64) * 64;
  // A chunk of 256 takes 10 us at r = 128 (1024: 40 us, longer than the columns
  // pass gains by it at 4096 rows); there are at most 512.
  p.chunk_bits = 8;
  while (N * k >> p.chunk_bits > 512) ++p.chunk_bits;
  p.chunks = dtype == 0 && !p.few ? N * k >> p.chunk_bits : 0;
  size_t o = 0;
  const auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align256(bytes);
    return at;
  };
  p.pm = take(size_t(p.row_splits) * N * 4);
  p.pl = take(size_t(p.row_splits) * N * 4);
  p.po = take(size_t(p.row_splits) * N * p.RP * 4);
  p.fwd_total = o;
  o = 0;
  p.zc = take(size_t(N) * p.RP * es);
  p.row_c = take(size_t(p.npad) * 8);
  p.srt_id = take(size_t(N) * k * 4);
  p.srt_w = take(size_t(N) * k * 4);
  p.table = take(size_t(p.groups / 4 + 1) * p.npad * 4);
  p.start = take(size_t(p.groups + 1) * 4);
  p.list = take(size_t(N) * k * 8);
  p.part = take(p.col_splits > 1 ? size_t(p.col_splits) * p.split_rows * p.RP * 4 : 0);
  p.chunk_in = take(size_t(p.chunks) * 4);
  p.chunk_part = take(size_t(p.chunks) * p.GC * p.RP * 4);
  p.bwd_total = o;
  return p;
}

template <int RP, int XT, int WX, bool ACC, bool COLS>
hipError_t go_bf16(const StreamArgs& a, hipStream_t s) {
  const int64_t blocks = a.whole + (ceil_div(a.nx, WX * 32 * XT) - a.whole) * a.splits;
  const auto kernel = stream_bf16_kernel<RP, XT, WX, ACC, COLS>;
  constexpr int bytes = bf16_lds_bytes<RP, WX>();
  if constexpr (bytes > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(kWaves * kWave), bytes, s, a);
  return hipGetLastError();
}

template <int RP>
hipError_t go_few(const StreamArgs& a, hipStream_t s) {
  const auto go = [&](auto kernel, int rows) -> hipError_t {
    const int bytes = (rows * RP + kWaves * 32 * 32) * 2;
    if (bytes > 65536) {
      const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kernel, dim3((unsigned)ceil_div(a.nx, kWaves * 32)), dim3(kWaves * kWave), bytes, s, a);
    return hipGetLastError();
  };
  return a.ny <= 32 ? go(few_columns_kernel<RP, 1>, 32) : go(few_columns_kernel<RP, 2>, 64);
}

template <int RP, int XT, bool ACC>
hipError_t go_rows(const StreamArgs& a, int WX, hipStream_t s) {
  if constexpr (RP < 256) {
    if (WX == 1) return go_bf16<RP, XT, 1, ACC, false>(a, s);
  }
  if (WX == 2) return go_bf16<RP, XT, 2, ACC, false>(a, s);
  return go_bf16<RP, XT, 4, ACC, false>(a, s);
}

template <bool ACC, bool COLS>
hipError_t stream(int dtype, const Plan& p, const StreamArgs& a, hipStream_t s) {
  if (dtype == 0) {
    if constexpr (COLS) {
      if (p.few) {
        switch (p.RP) {
          case 32: return go_few<32>(a, s);
          case 64: return go_few<64>(a, s);
          case 128: return go_few<128>(a, s);
          case 256: return go_few<256>(a, s);
          default: return go_few<512>(a, s);
        }
      }
      switch (p.RP) {
        case 32: return go_bf16<32, x_tiles(32), 4, true, true>(a, s);
        case 64: return go_bf16<64, x_tiles(64), 4, true, true>(a, s);
        case 128: return go_bf16<128, x_tiles(128), 4, true, true>(a, s);
        case 256: return go_bf16<256, x_tiles(256), 4, true, true>(a, s);
        default: return go_bf16<512, x_tiles(512), 4, true, true>(a, s);
      }
    } else {
      switch (p.RP) {
        case 32: return go_rows<32, x_tiles(32), ACC>(a, p.WX, s);
        case 64: return go_rows<64, x_tiles(64), ACC>(a, p.WX, s);
        case 128: return go_rows<128, x_tiles(128), ACC>(a, p.WX, s);
        case 256: return go_rows<256, x_tiles(256), ACC>(a, p.WX, s);
        default: return go_rows<512, x_tiles(512), ACC>(a, p.WX, s);
      }
    }
  }
  const dim3 grid((unsigned)(a.whole + (ceil_div(a.nx, 64) - a.whole) * a.splits)), block(kWaves * kWave);
  switch (p.RP) {
    case 32: hipLaunchKernelGGL((stream_f32_kernel<32, ACC, COLS>), grid, block, 0, s, a); break;
    case 64: hipLaunchKernelGGL((stream_f32_kernel<64, ACC, COLS>), grid, block, 0, s, a); break;
    case 128: hipLaunchKernelGGL((stream_f32_kernel<128, ACC, COLS>), grid, block, 0, s, a); break;
    case 256: hipLaunchKernelGGL((stream_f32_kernel<256, ACC, COLS>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((stream_f32_kernel<512, ACC, COLS>), grid, block, 0, s, a); break;
  }
  return hipGetLastError();
}

template <int RP>
hipError_t go_chunks(const Plan& p, const StreamArgs& a, hipStream_t s) {
  const auto kernel = chunk_kernel<RP, x_tiles(RP)>;
  constexpr int bytes = bf16_lds_bytes<RP, kWaves>();
  if constexpr (bytes > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kernel, dim3((unsigned)p.chunks), dim3(kWaves * kWave), bytes, s, a);
  return hipGetLastError();
}
hipError_t chunks(const Plan& p, const StreamArgs& a, hipStream_t s) {
  switch (p.RP) {
    case 32: return go_chunks<32>(p, a, s);
    case 64: return go_chunks<64>(p, a, s);
    case 128: return go_chunks<128>(p, a, s);
    case 256: return go_chunks<256>(p, a, s);
    default: return go_chunks<512>(p, a, s);
  }
}

template <typename T, int L>
void finish(const Plan& p, const DistillArgs& d, char* ws, hipStream_t s) {
  hipLaunchKernelGGL((distill_finish_kernel<T, L>), dim3((unsigned)(d.N * (d.G ? ceil_div(d.r, 4 * L) : 1))),
                     dim3(kWaves * kWave), 0, s, static_cast<const T*>(d.Z), static_cast<const T*>(d.P), d.idx, d.t,
                     d.N, d.V, d.r, p.RP, d.k, d.inv_t, d.scale, __builtin_ctz(p.TY), p.row_splits,
                     reinterpret_cast<float*>(ws + p.pm), reinterpret_cast<float*>(ws + p.pl),
                     reinterpret_cast<float*>(ws + p.po), d.loss, d.lse, d.G);
}
template <typename T>
void finish(const Plan& p, const DistillArgs& d, char* ws, hipStream_t s) {
  if (d.r <= 64 || !d.G) finish<T, 16>(p, d, ws, s);
  else if (d.r <= 128) finish<T, 32>(p, d, ws, s);
  else finish<T, 64>(p, d, ws, s);
}

template <typename T>
void prep(const Plan& p, const DistillArgs& d, char* ws, hipStream_t s) {
  hipLaunchKernelGGL(distill_prep_kernel<T>, dim3((unsigned)(p.npad / kWaves)), dim3(kWaves * kWave), 0, s,
                     static_cast<const T*>(d.Z),
                     d.dtype == 0 && !p.few ? static_cast<const T*>(d.P) : nullptr, d.scale, d.idx, d.t, d.lse,
                     d.G, d.weight, (int)d.N, d.V, d.r, p.RP, d.k, d.inv_t,
                     d.dP ? reinterpret_cast<T*>(ws + p.zc) : nullptr, reinterpret_cast<float*>(ws + p.row_c),
                     p.RB, reinterpret_cast<int*>(ws + p.srt_id),
                     reinterpret_cast<float*>(ws + p.srt_w), static_cast<T*>(d.dZ));
}

}  // namespace

bool distill_fits(int dtype, int64_t V, int r, int64_t N) {
  const Plan p = plan(dtype, V, r, N, 1);
  const int64_t lists = p.groups * kListWaves * kWave;
  const int64_t tables = p.npad / kWave * ceil_div(p.groups / 4 + 1, kTableWords * kWaves) * kWaves * kWave;
  return std::max(lists, tables) <= kMostThreads;
}

size_t distill_workspace_bytes(int dtype, int64_t V, int r, int64_t N, int k) {
  const Plan p = plan(dtype, V, r, N, k);
  return std::max(p.fwd_total, p.bwd_total);
}

hipError_t launch_distill(const DistillArgs& d, void* workspace, hipStream_t s) {
  const Plan p = plan(d.dtype, d.V, d.r, d.N, d.k);
  char* ws = static_cast<char*>(workspace);
  StreamArgs a{};
  a.X = d.Z;
  a.nx = d.N;
  a.Y = d.P;
  a.ny = d.V;
  a.r = d.r;
  a.ldy = d.r;
  a.scale = d.scale;
  a.splits = p.row_splits;
  a.pm = reinterpret_cast<float*>(ws + p.pm);
  a.pl = reinterpret_cast<float*>(ws + p.pl);
  a.po = reinterpret_cast<float*>(ws + p.po);
  const hipError_t e = d.G ? stream<true, false>(d.dtype, p, a, s) : stream<false, false>(d.dtype, p, a, s);
  if (e != hipSuccess) return e;
  if (d.dtype == 0) finish<uint16_t>(p, d, ws, s);
  else finish<float>(p, d, ws, s);
  return hipGetLastError();
}

hipError_t launch_distill_grad(const DistillArgs& d, void* workspace, hipStream_t s) {
  if (d.N == 0) {   // no rows: dP is zero (r is a multiple of 8, so bf16 rows are whole words)
    if (!d.dP) return hipSuccess;
    const int64_t words = d.V * d.r / (d.dtype == 0 ? 2 : 1);
    hipLaunchKernelGGL(distill_zero_kernel, dim3((unsigned)std::min<int64_t>(ceil_div(words, 256), 4096)), dim3(256),
                       0, s, static_cast<uint32_t*>(d.dP), words);
    return hipGetLastError();
  }
  const Plan p = plan(d.dtype, d.V, d.r, d.N, d.k);
  char* ws = static_cast<char*>(workspace);
  if (d.dtype == 0) prep<uint16_t>(p, d, ws, s);
  else prep<float>(p, d, ws, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !d.dP) return e;
  const int* srt_id = reinterpret_cast<int*>(ws + p.srt_id);
  const float* srt_w = reinterpret_cast<float*>(ws + p.srt_w);
  uint32_t* table = reinterpret_cast<uint32_t*>(ws + p.table);
  uint32_t* start = reinterpret_cast<uint32_t*>(ws + p.start);
  uint2* list = reinterpret_cast<uint2*>(ws + p.list);
  const int row_blocks = (int)(p.npad / kWave);
  const int64_t words = p.groups / 4 + 1;
  hipLaunchKernelGGL(distill_table_kernel, dim3((unsigned)(row_blocks * ceil_div(words, kTableWords * kWaves))),
                     dim3(kWaves * kWave), 0, s, srt_id, (int)d.N, (int)p.npad, d.k, p.GC, words, row_blocks, table);
  hipLaunchKernelGGL(distill_list_kernel, dim3((unsigned)p.groups), dim3(kListWaves * kWave), 0, s, table, srt_id,
                     srt_w, (int)p.npad, d.k, p.GC, d.dtype == 0 && !p.few, p.chunk_bits, (uint32_t)p.chunks, start, list,
                     reinterpret_cast<uint32_t*>(ws + p.chunk_in));
  StreamArgs a{};
  a.X = d.P;
  a.nx = d.V;
  a.Y = ws + p.zc;
  a.ny = d.N;
  a.r = d.r;
  a.ldy = p.RP;
  a.scale = d.scale;
  a.whole = p.col_whole;
  a.splits = p.col_splits;
  a.row_c = reinterpret_cast<float*>(ws + p.row_c);
  a.row_block = p.RB;
  a.list_start = start;
  a.list = list;
  a.dP = d.dP;
  a.part = reinterpret_cast<float*>(ws + p.part);
  a.groups = p.groups;
  a.chunk_bits = p.chunk_bits;
  a.chunk_in = reinterpret_cast<const uint32_t*>(ws + p.chunk_in);
  a.chunk_part = reinterpret_cast<float*>(ws + p.chunk_part);
  if (p.chunks) {
    e = chunks(p, a, s);
    if (e != hipSuccess) return e;
  }
  e = stream<true, true>(d.dtype, p, a, s);
  if (e != hipSuccess) return e;
  if (p.col_splits > 1) {   // at most 1024 blocks of rows (fp32, 64 rows each): the index fits 32 bits
    const dim3 grid((unsigned)ceil_div(p.split_rows * p.RP, 1024));
    const int64_t first = (d.V - p.split_rows) * d.r;
    if (d.dtype == 0)
      hipLaunchKernelGGL(distill_join_kernel<uint16_t>, grid, dim3(256), 0, s, a.part, p.col_splits,
                         (int)p.split_rows, d.r, p.RP, static_cast<uint16_t*>(d.dP) + first);
    else
      hipLaunchKernelGGL(distill_join_kernel<float>, grid, dim3(256), 0, s, a.part, p.col_splits,
                         (int)p.split_rows, d.r, p.RP, static_cast<float*>(d.dP) + first);
  }
  return hipGetLastError();
}

}  // namespace lrh
