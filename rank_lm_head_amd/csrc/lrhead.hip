// lrhead.hip — host side of the C ABI in include/lrhead.h.
//
// Every entry point validates its arguments on the host before it touches
// HIP, then enqueues the stage kernels on the caller's stream and returns.
// Nothing here allocates device memory or synchronises: the caller's
// workspace holds z and the per-slice candidate lists.
#include "lrhead.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <mutex>
#include <new>

#include "launch.h"

struct lrhead_s {
  uint32_t magic;
  int dtype;
  int64_t V, d, r, B_max;
  int k_max;
  const void* Q;
  const void* P;
  const void* W;
  char* ws;
  size_t ws_bytes;
  void* z;          // B_max x r, weight dtype
  float* part_s;    // candidate lists: rows x slices x k_max
  int* part_i;
  float* raw;       // raw scores of the streaming path: min(B_max, 8) x V
  uint64_t* b1_keys;  // one-row pass: slice lists (candidate keys)
  float* b1_lgs;      // one-row pass: their speculative exact logits
  uint32_t* sync;     // one-row pass: completion counters
  int n_cu;           // compute units of the device
  bool batch;       // bf16 with B_max > 4: the GEMM path's scratch exists
  lrh::BatchScratch bw;
  hipEvent_t ev_before;  // optional events attached to the score pass: its start
  hipEvent_t ev_after;   // and its end
};

static __device__ __align__(256) unsigned char scratch[size_t(LRHEAD_STATIC_SCRATCH_MB) << 20];

namespace {

constexpr uint32_t kMagic = 0x4c524844u;  // "LRHD"
constexpr int64_t kDownGemmRows = 256;     // rows from which z = Q . h may run on the GEMM kernel
constexpr int64_t kDownSplitMaxElems = 65536;   // ... when B * r is above this
// From this many (row, winner) pairs on, the merge rescores only the
// winners, after the ranking: its speculative rescoring of every candidate
// (a few more than k per row) reads more of W than it hides once many rows
// keep the chip busy. Cold calls at r = 128, speculative against not: k = 32:
// 45.5 against 38.6 us at 64 rows, 31.9 against 28.9 at 32, 27.3 against
// 28.0 at 24; k = 64: 29.2 against 26.1 at 16 rows, 24.1 against 25.5 at
// 12; k = 8: 32.6 against 33.7 at 64 rows. (A separate rescoring launch
// after a ranking-only merge measured 40.1 us at 64 rows, k = 32.)
constexpr int64_t kSpeculatePairsBelow = 1024;
constexpr int64_t kBMaxLimit = int64_t(1) << 20;
constexpr int64_t kSampleMaxN = int64_t(1) << 24;
constexpr int kVerifyMaxS = 255;

thread_local char g_err[512] = "";

int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return code;
}

int hip_fail(hipError_t e, const char* what) {
  return fail(LRHEAD_EHIP, "%s: %s", what, hipGetErrorString(e));
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
size_t elem_bytes(int dtype) { return dtype == LRHEAD_BF16 ? 2 : 4; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

struct Layout {
  size_t z, part_s, part_i, raw, b1_keys, b1_lgs, sync, batch, total;
};

// Most candidate lists any call with B <= B_max writes (B x slices), over
// both the streaming and the matrix-core selection.
int64_t max_list_rows(int64_t B_max, int64_t V) {
  int64_t best = 0;
  for (int64_t B = 1; B <= B_max; ++B) {
    int64_t rows = B * lrh::plan_vsplit(B, V);
    if (B <= lrh::kRowsMaxB) {
      const int64_t small = B * lrh::small_blocks(V);
      if (small > rows) rows = small;
    }
    if (rows > best) best = rows;
  }
  return best;
}

Layout layout(int dtype, int64_t V, int64_t r, int64_t B_max, int k_max) {
  Layout L;
  L.z = 0;
  const size_t zb = align256(size_t(B_max) * size_t(r) * elem_bytes(dtype));
  // the merge reads whole 16-byte chunks, up to 12 bytes past the last list
  const size_t lists = align256(size_t(max_list_rows(B_max, V)) * size_t(k_max) * 4 + 16);
  L.part_s = zb;
  L.part_i = zb + lists;
  // raw scores of the streaming path (bf16 heads, B <= kSmallB rows)
  const int64_t raw_rows = dtype == LRHEAD_BF16 ? (B_max < lrh::kSmallB ? B_max : lrh::kSmallB) : 0;
  L.raw = zb + 2 * lists;
  L.b1_keys = L.raw + align256(size_t(raw_rows) * size_t(V) * 4);
  L.b1_lgs = L.b1_keys + align256(size_t(lrh::kB1MaxLists) * lrh::kB1MaxList * 8);
  L.sync = L.b1_lgs + align256(size_t(lrh::kB1MaxLists) * lrh::kB1MaxList * 4);
  L.batch = L.sync + align256(size_t(lrh::kB1Counters) * 128);
  L.total = L.batch;
  if (lrh::batch_path(dtype, B_max)) L.total += align256(lrh::batch_scratch_bytes(V, B_max));
  return L;
}

int check_shapes(int dtype, int64_t V, int64_t d, int64_t r, int64_t B_max, int k_max) {
  if (dtype != LRHEAD_BF16 && dtype != LRHEAD_FP32) return fail(LRHEAD_EDTYPE, "unknown dtype %d", dtype);
  if (V < 1 || V > INT32_MAX) return fail(LRHEAD_ERANGE, "V = %lld outside [1, 2^31)", (long long)V);
  if (d < 8 || d > LRHEAD_D_MAX || d % 8) return fail(LRHEAD_ERANGE, "d = %lld: need a multiple of 8 in [8, %d]", (long long)d, LRHEAD_D_MAX);
  if (r < 8 || r > LRHEAD_R_MAX || r % 8) return fail(LRHEAD_ERANGE, "r = %lld: need a multiple of 8 in [8, %d]", (long long)r, LRHEAD_R_MAX);
  if (B_max < 1 || B_max > kBMaxLimit) return fail(LRHEAD_ERANGE, "B_max = %lld outside [1, 2^20]", (long long)B_max);
  if (k_max < 1 || k_max > LRHEAD_K_MAX || k_max > V)
    return fail(LRHEAD_ERANGE, "k_max = %d outside [1, min(%d, V)]", k_max, LRHEAD_K_MAX);
  return LRHEAD_OK;
}

int check_handle(const lrhead_s* h) {
  if (!h || h->magic != kMagic) return fail(LRHEAD_EINVAL, "invalid handle");
  return LRHEAD_OK;
}

int check_rows(const lrhead_s* h, const void* H, int64_t B) {
  if (B < 0 || B > h->B_max) return fail(LRHEAD_ERANGE, "B = %lld outside [0, B_max = %lld]", (long long)B, (long long)h->B_max);
  if (B > 0 && !H) return fail(LRHEAD_EINVAL, "H is NULL");
  if (!aligned16(H)) return fail(LRHEAD_EALIGN, "H is not 16-byte aligned");
  return LRHEAD_OK;
}

int check_k(const lrhead_s* h, int k) {
  if (k < 1 || k > h->k_max) return fail(LRHEAD_ERANGE, "k = %d outside [1, k_max = %d]", k, h->k_max);
  return LRHEAD_OK;
}

int check_out(const void* p, const char* name, bool required) {
  if (!p) return required ? fail(LRHEAD_EINVAL, "%s is NULL", name) : LRHEAD_OK;
  if (!aligned16(p)) return fail(LRHEAD_EALIGN, "%s is not 16-byte aligned", name);
  return LRHEAD_OK;
}

#define LRH_TRY(x)            \
  do {                        \
    const int rc_ = (x);      \
    if (rc_ != LRHEAD_OK) return rc_; \
  } while (0)

#define LRH_HIP(x, what)                 \
  do {                                   \
    const hipError_t e_ = (x);           \
    if (e_ != hipSuccess) return hip_fail(e_, what); \
  } while (0)

// The caller's profiling events, attached to the score pass's dispatch.
lrh::Timing timing(const lrhead_s* h) { return lrh::Timing{h->ev_before, h->ev_after}; }

// Down-projection, score pass with per-slice selection, and the merge of
// the slice lists; with `logits`, the merge also rescores the winners.
int enqueue_head(lrhead_s* h, const void* H, int64_t B, int k, int32_t* idx, float* score, float* logits,
                 hipStream_t s) {
  if (lrh::b1_path(h->dtype, B, h->r, h->V, h->n_cu)) {
    // one row: the down-projection (which also resets the pass's counters),
    // then a single pass that scores, selects, merges and rescores
    LRH_HIP(lrh::launch_down_wide(h->Q, H, (int)h->r, (int)h->d, B, h->z, h->sync, lrh::kB1Counters, h->b1_lgs,
                                  2 * lrh::b1_blocks(h->V, h->n_cu), s),
            "down-projection launch");
    lrh::B1Args a;
    a.P = h->P;
    a.Z = h->z;
    a.V = h->V;
    a.K = (int)h->r;
    a.k = k;
    a.L = lrh::b1_list_len(k);
    a.W = h->W;
    a.H = H;
    a.d = (int)h->d;
    a.keys = h->b1_keys;
    a.lgs = h->b1_lgs;
    a.raw = h->raw;
    a.sync = h->sync;
    a.n_cu = h->n_cu;
    a.idx = idx;
    a.score = score;
    a.logits = logits;
    LRH_HIP(lrh::launch_draft1(a, s, timing(h)), "score/selection launch");
    return LRHEAD_OK;
  }
  const bool rows = lrh::rows_path(h->dtype, B, h->r, h->V);
  const bool streaming = rows || lrh::small_path(h->dtype, B, h->r, h->V);
  if (!streaming && lrh::batch_path(h->dtype, B)) {
    // many rows. Up to 64 rows the down-projection takes one block per row
    // of Q and group of 8 rows (one launch); above that it is a GEMM worth
    // the pipelined kernel. The sparse score array is written only later in
    // the call, so the
    // split down-projection keeps its partial sums there when they fit.
    // Measured crossover: the split kernel is faster up to B * r = 65536
    // (B = 256 at r = 256: 144 against 149 us per call; B = 512 at r = 256:
    // 219 against 209 us).
    const size_t part_bytes = size_t(lrh::down_split_parts((int)h->d)) * size_t(B) * size_t(h->r) * 4;
    if (B <= lrh::kDownWideMaxB)
      LRH_HIP(lrh::launch_down_wide(h->Q, H, (int)h->r, (int)h->d, B, h->z, nullptr, 0, nullptr, 0, s),
              "down-projection launch");
    else if (B >= kDownGemmRows && B * h->r > kDownSplitMaxElems)
      LRH_HIP(lrh::launch_down_gemm(h->Q, H, (int)h->r, (int)h->d, B, h->z, h->bw.S, h->bw.S_bytes, s),
              "down-projection launch");
    else if (part_bytes <= h->bw.S_bytes)
      LRH_HIP(lrh::launch_down_split(h->Q, H, (int)h->r, (int)h->d, B, h->z, h->bw.S, s), "down-projection launch");
    else
      LRH_HIP(lrh::launch_down(h->dtype, h->Q, H, (int)h->r, (int)h->d, B, h->z, s), "down-projection launch");
    LRH_HIP(lrh::launch_batch_select(h->P, h->z, h->V, (int)h->r, B, k, h->bw, idx, score, s, timing(h)),
            "score/selection launch");
    if (logits)
      LRH_HIP(lrh::launch_rescore(h->dtype, h->W, H, idx, B, k, h->V, (int)h->d, logits, s), "rescore launch");
    return LRHEAD_OK;
  }
  int n_lists, list_len = k;
  const float* raw = nullptr;
  if (streaming) {
    LRH_HIP(lrh::launch_down_wide(h->Q, H, (int)h->r, (int)h->d, B, h->z, nullptr, 0, nullptr, 0, s),
            "down-projection launch");
    if (rows) {
      // no raw scores: the merge recomputes a slice it needs more of
      LRH_HIP(lrh::launch_select_rows(h->P, h->z, h->V, (int)h->r, B, k, h->part_s, h->part_i, s, timing(h)),
              "score/selection launch");
    } else {
      LRH_HIP(lrh::launch_select_small(h->P, h->z, h->V, (int)h->r, B, k, h->part_s, h->part_i, h->raw, s,
                                       timing(h)),
              "score/selection launch");
      raw = h->raw;
    }
    n_lists = lrh::small_blocks(h->V);
    list_len = lrh::small_list_len(k);
  } else {
    LRH_HIP(lrh::launch_down(h->dtype, h->Q, H, (int)h->r, (int)h->d, B, h->z, s), "down-projection launch");
    n_lists = lrh::plan_vsplit(B, h->V);
    LRH_HIP(lrh::launch_select(h->dtype, h->P, h->z, h->V, (int)h->r, B, k, n_lists, h->part_s, h->part_i, s,
                               timing(h)),
            "score/selection launch");
  }
  LRH_HIP(lrh::launch_merge(h->dtype, h->part_s, h->part_i, n_lists, list_len, rows, raw, rows ? h->P : nullptr,
                            rows ? h->z : nullptr, (int)h->r, h->V, B, k, h->W, H, (int)h->d, idx, score, logits,
                            B * k < kSpeculatePairsBelow, s),
          "merge launch");
  return LRHEAD_OK;
}

// The checks and settings a handle needs from the current device: it must be
// gfx950; the GEMM kernels of row batches get their LDS limit raised; the
// one-row pass sizes its grid by the compute units.
int device_setup(int dtype, int64_t B_max, int* n_cu) {
  int dev = 0;
  LRH_HIP(hipGetDevice(&dev), "hipGetDevice");
  hipDeviceProp_t prop;
  LRH_HIP(hipGetDeviceProperties(&prop, dev), "hipGetDeviceProperties");
  if (std::strncmp(prop.gcnArchName, "gfx950", 6) != 0)
    return fail(LRHEAD_EDEVICE, "device %d is %s, this library is built for gfx950", dev, prop.gcnArchName);
  if (lrh::batch_path(dtype, B_max)) LRH_HIP(lrh::batch_init(), "GEMM kernel set-up");
  LRH_HIP(hipDeviceGetAttribute(n_cu, hipDeviceAttributeMultiprocessorCount, dev), "hipDeviceGetAttribute");
  return LRHEAD_OK;
}

void fill_handle(lrhead_s* h, int dtype, int64_t V, int64_t d, int64_t r, const void* Q, const void* P,
                 const void* W, int64_t B_max, int k_max, void* workspace, size_t workspace_bytes, int n_cu) {
  const Layout L = layout(dtype, V, r, B_max, k_max);
  h->magic = kMagic;
  h->dtype = dtype;
  h->V = V;
  h->d = d;
  h->r = r;
  h->B_max = B_max;
  h->k_max = k_max;
  h->Q = Q;
  h->P = P;
  h->W = W;
  h->ws = static_cast<char*>(workspace);
  h->ws_bytes = workspace_bytes;
  h->z = h->ws + L.z;
  h->part_s = reinterpret_cast<float*>(h->ws + L.part_s);
  h->part_i = reinterpret_cast<int*>(h->ws + L.part_i);
  h->raw = reinterpret_cast<float*>(h->ws + L.raw);
  h->b1_keys = reinterpret_cast<uint64_t*>(h->ws + L.b1_keys);
  h->b1_lgs = reinterpret_cast<float*>(h->ws + L.b1_lgs);
  h->sync = reinterpret_cast<uint32_t*>(h->ws + L.sync);
  h->n_cu = n_cu;
  h->batch = lrh::batch_path(dtype, B_max);
  h->bw = h->batch ? lrh::batch_scratch(h->ws + L.batch, V, B_max) : lrh::BatchScratch{};
  h->ev_before = nullptr;
  h->ev_after = nullptr;
}

// ------------------------------------------------------- training, beams
int check_distill(int dtype, int64_t V, int64_t r, int64_t N, int k) {
  if (dtype != LRHEAD_BF16 && dtype != LRHEAD_FP32) return fail(LRHEAD_EDTYPE, "unknown dtype %d", dtype);
  if (V < 1 || V > INT32_MAX) return fail(LRHEAD_ERANGE, "V = %lld outside [1, 2^31)", (long long)V);
  if (r < 8 || r > LRHEAD_R_MAX || r % 8) return fail(LRHEAD_ERANGE, "r = %lld: need a multiple of 8 in [8, %d]", (long long)r, LRHEAD_R_MAX);
  if (N < 0 || N > kBMaxLimit) return fail(LRHEAD_ERANGE, "N = %lld outside [0, 2^20]", (long long)N);
  if (k < 1 || k > LRHEAD_K_MAX) return fail(LRHEAD_ERANGE, "k = %d outside [1, %d]", k, LRHEAD_K_MAX);
  if (!lrh::distill_fits(dtype, V, (int)r, N > 0 ? N : 1))
    return fail(LRHEAD_ERANGE, "V = %lld with N = %lld is too large for one call", (long long)V, (long long)N);
  return LRHEAD_OK;
}

int check_temperature(float t) {
  // also its reciprocal has to be a normal number
  if (!(t >= 1e-30f && t <= 1e30f)) return fail(LRHEAD_ERANGE, "temperature = %g outside [1e-30, 1e30]", (double)t);
  return LRHEAD_OK;
}

lrh::DistillArgs distill_args(int dtype, int64_t V, int64_t r, const void* P, const void* Z, int64_t N,
                              const int32_t* idx, const float* logits, int k, float temperature) {
  lrh::DistillArgs d{};
  d.dtype = dtype;
  d.V = V;
  d.N = N;
  d.r = (int)r;
  d.k = k;
  d.inv_t = (float)(1.0 / (double)temperature);
  d.scale = (float)(1.4426950408889634 / (double)temperature);
  d.P = P;
  d.Z = Z;
  d.idx = idx;
  d.t = logits;
  return d;
}

int check_beam(int dtype, int64_t B, int m, int64_t n, int nb) {
  if (dtype != LRHEAD_BF16 && dtype != LRHEAD_FP32) return fail(LRHEAD_EDTYPE, "unknown dtype %d", dtype);
  if (m < 1 || m > LRHEAD_K_MAX) return fail(LRHEAD_ERANGE, "m = %d outside [1, %d]", m, LRHEAD_K_MAX);
  if (nb < 1 || nb > LRHEAD_K_MAX) return fail(LRHEAD_ERANGE, "nb = %d outside [1, %d]", nb, LRHEAD_K_MAX);
  if (n < 1 || n > INT32_MAX) return fail(LRHEAD_ERANGE, "n = %lld outside [1, 2^31)", (long long)n);
  if (B < 0 || B > kBMaxLimit || !lrh::beam_fits(dtype, B > 0 ? B : 1, m, n))
    return fail(LRHEAD_ERANGE, "B = %lld outside [0, 2^20], or B m n too large for one call", (long long)B);
  return LRHEAD_OK;
}

int check_sampling(int dtype, int64_t B, int64_t per, int64_t n) {
  if (dtype != LRHEAD_BF16 && dtype != LRHEAD_FP32) return fail(LRHEAD_EDTYPE, "unknown dtype %d", dtype);
  if (n < 1 || n > kSampleMaxN) return fail(LRHEAD_ERANGE, "n = %lld outside [1, 2^24]", (long long)n);
  if (B < 0 || B > kBMaxLimit / per || !lrh::sample_fits(B * per, n))
    return fail(LRHEAD_ERANGE, "B = %lld is negative, or too many rows for one call", (long long)B);
  return LRHEAD_OK;
}

int check_embed(int dtype, int64_t V, int64_t d, int64_t N) {
  if (dtype != LRHEAD_BF16 && dtype != LRHEAD_FP32) return fail(LRHEAD_EDTYPE, "unknown dtype %d", dtype);
  if (V < 1 || V > INT32_MAX) return fail(LRHEAD_ERANGE, "V = %lld outside [1, 2^31)", (long long)V);
  if (d < 1 || d > LRHEAD_D_MAX) return fail(LRHEAD_ERANGE, "d = %lld outside [1, %d]", (long long)d, LRHEAD_D_MAX);
  if (N < 0 || N > kBMaxLimit) return fail(LRHEAD_ERANGE, "N = %lld outside [0, 2^20]", (long long)N);
  if (N > 0 && (!lrh::embed_fits(dtype, d, N) || !lrh::embed_grad_fits(dtype, V, d, N)))
    return fail(LRHEAD_ERANGE, "N = %lld rows of d = %lld are too many for one call", (long long)N, (long long)d);
  return LRHEAD_OK;
}

bool aligned_elem(const void* p, int dtype) { return reinterpret_cast<uintptr_t>(p) % elem_bytes(dtype) == 0; }

// Whether [a, a + an) and [b, b + bn) share a byte.
bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return an && bn && x < y + bn && y < x + an;
}

// Whether one of `outs` shares a byte with another of them or with one of `ins`.
struct Span {
  const void* p;
  size_t n;   // bytes; none where p is NULL
};
bool clash(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    const auto meets = [&](const Span& i) { return o->p && i.p && overlap(o->p, o->n, i.p, i.n); };
    if (std::any_of(o + 1, outs.end(), meets) || std::any_of(ins.begin(), ins.end(), meets)) return true;
  }
  return false;
}

int sample_args(lrh::SampleArgs* a, int dtype, const void* logits, int64_t ld, const float* u,
                const lrhead_sampling_t* how, int64_t n) {
  if (!logits || !u || !how) return fail(LRHEAD_EINVAL, "logits, u and how must be non-NULL");
  if (!aligned_elem(logits, dtype)) return fail(LRHEAD_EALIGN, "logits are not aligned to their elements");
  if (!aligned4(u) || !aligned4(how->temperature) || !aligned4(how->top_k) || !aligned4(how->top_p) ||
      !aligned4(how->min_p))
    return fail(LRHEAD_EALIGN, "u and the settings' arrays must be 4-byte aligned");
  a->dtype = dtype;
  a->x = logits;
  a->ld = ld;
  a->n = n;
  a->u = u;
  a->temperature = how->temperature;
  a->top_k = how->top_k;
  a->top_p = how->top_p;
  a->min_p = how->min_p;
  a->temperature_all = how->temperature_all;
  a->top_k_all = how->top_k_all;
  a->top_p_all = how->top_p_all;
  a->min_p_all = how->min_p_all;
  return LRHEAD_OK;
}

// ------------------------------------------------- allocation-free variant
// The workspace of lrhead_draft_static is `scratch` (file scope, below the
// namespace): one copy per GPU, resident until the process ends. In host
// code its name only stands for the symbol; its address on a device comes
// from hipGetSymbolAddress with that device current, looked up once per
// device and kept.
constexpr size_t kStaticScratchBytes = size_t(LRHEAD_STATIC_SCRATCH_MB) << 20;
constexpr int kMaxDevices = 64;
struct StaticDevice {
  bool ready;
  void* ptr;   // device address of `scratch` on this device
  int n_cu;
};
std::mutex g_static_mu;
StaticDevice g_static[kMaxDevices];

int static_device(int dtype, int64_t B, void** ptr, int* n_cu) {
  int dev = 0;
  LRH_HIP(hipGetDevice(&dev), "hipGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(LRHEAD_EDEVICE, "device %d beyond the %d supported", dev, kMaxDevices);
  std::lock_guard<std::mutex> lock(g_static_mu);
  StaticDevice& sd = g_static[dev];
  if (!sd.ready) {
    int cu = 0;
    LRH_TRY(device_setup(dtype, 1, &cu));
    void* p = nullptr;
    LRH_HIP(hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)), "hipGetSymbolAddress(scratch)");
    sd.ptr = p;
    sd.n_cu = cu;
    sd.ready = true;
  }
  if (lrh::batch_path(dtype, B)) LRH_HIP(lrh::batch_init(), "GEMM kernel set-up");
  *ptr = sd.ptr;
  *n_cu = sd.n_cu;
  return LRHEAD_OK;
}

}  // namespace

extern "C" {

size_t lrhead_workspace_bytes(int dtype, int64_t V, int64_t d, int64_t r, int64_t B_max, int k_max) {
  if (check_shapes(dtype, V, d, r, B_max, k_max) != LRHEAD_OK) return 0;
  return layout(dtype, V, r, B_max, k_max).total;
}

int lrhead_create(lrhead_t* out, int dtype, int64_t V, int64_t d, int64_t r, const void* Q, const void* P,
                  const void* W, int64_t B_max, int k_max, void* workspace, size_t workspace_bytes) {
  if (!out) return fail(LRHEAD_EINVAL, "out is NULL");
  *out = nullptr;
  LRH_TRY(check_shapes(dtype, V, d, r, B_max, k_max));
  if (!Q || !P || !W) return fail(LRHEAD_EINVAL, "Q, P and W must be non-NULL");
  if (!workspace) return fail(LRHEAD_EINVAL, "workspace is NULL");
  if (!aligned16(Q) || !aligned16(P) || !aligned16(W) || !aligned16(workspace))
    return fail(LRHEAD_EALIGN, "Q, P, W and workspace must be 16-byte aligned");
  const Layout L = layout(dtype, V, r, B_max, k_max);
  if (workspace_bytes < L.total)
    return fail(LRHEAD_EWORKSPACE, "workspace holds %zu bytes, needs %zu", workspace_bytes, L.total);
  int n_cu = 0;
  LRH_TRY(device_setup(dtype, B_max, &n_cu));
  lrhead_s* h = new (std::nothrow) lrhead_s;
  if (!h) return fail(LRHEAD_EINVAL, "out of host memory");
  fill_handle(h, dtype, V, d, r, Q, P, W, B_max, k_max, workspace, workspace_bytes, n_cu);
  *out = h;
  return LRHEAD_OK;
}

int lrhead_candidates(lrhead_t h, const void* H, int64_t B, int k, int32_t* idx, float* score, void* stream) {
  LRH_TRY(check_handle(h));
  LRH_TRY(check_rows(h, H, B));
  LRH_TRY(check_k(h, k));
  LRH_TRY(check_out(idx, "idx", B > 0));
  LRH_TRY(check_out(score, "score", false));
  if (B == 0) return LRHEAD_OK;
  return enqueue_head(h, H, B, k, idx, score, nullptr, static_cast<hipStream_t>(stream));
}

int fullhead_logits(lrhead_t h, const void* H, int64_t B, const int32_t* idx, int k, float* logits,
                    void* stream) {
  LRH_TRY(check_handle(h));
  LRH_TRY(check_rows(h, H, B));
  LRH_TRY(check_out(idx, "idx", false));
  if (idx) LRH_TRY(check_k(h, k));
  LRH_TRY(check_out(logits, "logits", B > 0));
  if (B == 0) return LRHEAD_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (!idx) {
    LRH_HIP(lrh::launch_dense(h->dtype, h->W, H, h->V, (int)h->d, B, logits, s), "dense logits launch");
    return LRHEAD_OK;
  }
  LRH_HIP(lrh::launch_rescore(h->dtype, h->W, H, idx, B, k, h->V, (int)h->d, logits, s), "rescore launch");
  return LRHEAD_OK;
}

int fullhead_topk(lrhead_t h, const void* H, int64_t B, int k, int32_t* idx, float* logits, void* stream) {
  LRH_TRY(check_handle(h));
  LRH_TRY(check_rows(h, H, B));
  LRH_TRY(check_k(h, k));
  LRH_TRY(check_out(idx, "idx", B > 0));
  LRH_TRY(check_out(logits, "logits", B > 0));
  if (B == 0) return LRHEAD_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (lrh::batch_path(h->dtype, B)) {
    LRH_HIP(lrh::launch_batch_select(h->W, H, h->V, (int)h->d, B, k, h->bw, idx, logits, s, timing(h)),
            "full-head selection launch");
    return LRHEAD_OK;
  }
  int n_lists;
  if (lrh::small_long_path(h->dtype, B, h->d, h->V)) {
    n_lists = lrh::small_blocks(h->V);
    LRH_HIP(lrh::launch_select_long(h->W, H, h->V, (int)h->d, B, k, h->part_s, h->part_i, s, timing(h)),
            "full-head selection launch");
  } else {
    n_lists = lrh::plan_vsplit(B, h->V);
    LRH_HIP(lrh::launch_select(h->dtype, h->W, H, h->V, (int)h->d, B, k, n_lists, h->part_s, h->part_i, s,
                               timing(h)),
            "full-head selection launch");
  }
  LRH_HIP(lrh::launch_merge(h->dtype, h->part_s, h->part_i, n_lists, k, false, nullptr, nullptr, nullptr, 0, h->V, B,
                            k, nullptr, nullptr, (int)h->d, idx, logits, nullptr, false, s),
          "merge launch");
  return LRHEAD_OK;
}

int lrhead_draft(lrhead_t h, const void* H, int64_t B, int k, int32_t* idx, float* score, float* logits,
                 void* stream) {
  LRH_TRY(check_handle(h));
  LRH_TRY(check_rows(h, H, B));
  LRH_TRY(check_k(h, k));
  LRH_TRY(check_out(idx, "idx", B > 0));
  LRH_TRY(check_out(score, "score", false));
  LRH_TRY(check_out(logits, "logits", B > 0));
  if (B == 0) return LRHEAD_OK;
  return enqueue_head(h, H, B, k, idx, score, logits, static_cast<hipStream_t>(stream));
}

int lrhead_draft_static(int dtype, int64_t V, int64_t d, int64_t r, const void* Q, const void* P, const void* W,
                        const void* H, int64_t B, int k, int32_t* idx, float* score, float* logits, void* stream) {
  if (B < 0) return fail(LRHEAD_ERANGE, "B = %lld is negative", (long long)B);
  LRH_TRY(check_shapes(dtype, V, d, r, B > 0 ? B : 1, k));
  if (!Q || !P || !W) return fail(LRHEAD_EINVAL, "Q, P and W must be non-NULL");
  if (!aligned16(Q) || !aligned16(P) || !aligned16(W)) return fail(LRHEAD_EALIGN, "Q, P and W must be 16-byte aligned");
  if (B > 0 && !H) return fail(LRHEAD_EINVAL, "H is NULL");
  if (!aligned16(H)) return fail(LRHEAD_EALIGN, "H is not 16-byte aligned");
  LRH_TRY(check_out(idx, "idx", B > 0));
  LRH_TRY(check_out(score, "score", false));
  LRH_TRY(check_out(logits, "logits", B > 0));
  if (B == 0) return LRHEAD_OK;
  const size_t need = layout(dtype, V, r, B, k).total;
  if (need > kStaticScratchBytes)
    return fail(LRHEAD_EWORKSPACE, "this call needs %zu bytes of scratch; the static scratch holds %zu", need,
                kStaticScratchBytes);
  void* ws = nullptr;
  int n_cu = 0;
  LRH_TRY(static_device(dtype, B, &ws, &n_cu));
  lrhead_s h;
  fill_handle(&h, dtype, V, d, r, Q, P, W, B, k, ws, kStaticScratchBytes, n_cu);
  return enqueue_head(&h, H, B, k, idx, score, logits, static_cast<hipStream_t>(stream));
}

int lrhead_branch(const float* logits, const int32_t* idx, const float* parent, int64_t B, int k, int nb,
                  float* probs, int32_t* br_idx, float* br_prob, float* br_path, void* stream) {
  if (B < 0) return fail(LRHEAD_ERANGE, "B = %lld is negative", (long long)B);
  if (k < 1 || k > LRHEAD_K_MAX) return fail(LRHEAD_ERANGE, "k = %d outside [1, %d]", k, LRHEAD_K_MAX);
  if (nb < 1 || nb > k) return fail(LRHEAD_ERANGE, "nb = %d outside [1, k = %d]", nb, k);
  if (B == 0) return LRHEAD_OK;
  if (!logits || !idx || !probs || !br_idx || !br_prob || !br_path)
    return fail(LRHEAD_EINVAL, "logits, idx, probs, br_idx, br_prob and br_path must be non-NULL");
  LRH_HIP(lrh::launch_branch(logits, idx, parent, B, k, nb, probs, br_idx, br_prob, br_path,
                             static_cast<hipStream_t>(stream)),
          "branch launch");
  return LRHEAD_OK;
}

size_t lrhead_factor_workspace_bytes(int64_t V, int64_t d, int r) {
  if (V < 1 || d < 1 || r < 1 || r > LRHEAD_R_MAX || r > d || r > V || V > INT32_MAX || d > LRHEAD_D_MAX) return 0;
  return lrh::factor_workspace_bytes(V, d, r);
}

int lrhead_factor(const void* W, int64_t V, int64_t d, int r, int q, const float* omega, void* P, void* Q,
                  void* workspace, size_t workspace_bytes, void* stream) {
  if (V < 1 || V > INT32_MAX) return fail(LRHEAD_ERANGE, "V = %lld outside [1, 2^31)", (long long)V);
  if (d < 1 || d > LRHEAD_D_MAX) return fail(LRHEAD_ERANGE, "d = %lld outside [1, %d]", (long long)d, LRHEAD_D_MAX);
  if (r < 1 || r > LRHEAD_R_MAX || r > d || r > V)
    return fail(LRHEAD_ERANGE, "r = %d outside [1, min(%d, d, V)]", r, LRHEAD_R_MAX);
  if (q < 0 || q > 8) return fail(LRHEAD_ERANGE, "q = %d outside [0, 8]", q);
  if (!W || !omega || !P || !Q || !workspace)
    return fail(LRHEAD_EINVAL, "W, omega, P, Q and workspace must be non-NULL");
  if (!aligned16(W) || !aligned16(omega) || !aligned16(P) || !aligned16(Q) || !aligned16(workspace))
    return fail(LRHEAD_EALIGN, "W, omega, P, Q and workspace must be 16-byte aligned");
  const size_t need = lrh::factor_workspace_bytes(V, d, r);
  if (workspace_bytes < need) return fail(LRHEAD_EWORKSPACE, "workspace holds %zu bytes, needs %zu", workspace_bytes, need);
  LRH_HIP(lrh::batch_init(), "GEMM kernel set-up");   // the W-sized products run on the GEMM kernel
  LRH_HIP(lrh::launch_factor(W, V, d, r, q, omega, P, Q, workspace, static_cast<hipStream_t>(stream)),
          "factor launch");
  return LRHEAD_OK;
}

size_t lrhead_distill_workspace_bytes(int dtype, int64_t V, int64_t r, int64_t N, int k) {
  if (check_distill(dtype, V, r, N, k) != LRHEAD_OK) return 0;
  return lrh::distill_workspace_bytes(dtype, V, (int)r, N > 0 ? N : 1, k);
}

int lrhead_distill(int dtype, int64_t V, int64_t r, const void* P, const void* Z, int64_t N, const int32_t* idx,
                   const float* logits, int k, float temperature, float* loss, float* lse, float* grad,
                   void* workspace, size_t workspace_bytes, void* stream) {
  LRH_TRY(check_distill(dtype, V, r, N, k));
  LRH_TRY(check_temperature(temperature));
  if (N == 0) return LRHEAD_OK;
  if (!P || !Z || !idx || !logits || !loss || !lse || !workspace)
    return fail(LRHEAD_EINVAL, "P, Z, idx, logits, loss, lse and workspace must be non-NULL");
  if (!aligned16(P) || !aligned16(Z) || !aligned16(grad) || !aligned16(workspace))
    return fail(LRHEAD_EALIGN, "P, Z, grad and workspace must be 16-byte aligned");
  if (!aligned4(idx) || !aligned4(logits) || !aligned4(loss) || !aligned4(lse))
    return fail(LRHEAD_EALIGN, "idx, logits, loss and lse must be 4-byte aligned");
  const size_t need = lrh::distill_workspace_bytes(dtype, V, (int)r, N, k);
  if (workspace_bytes < need) return fail(LRHEAD_EWORKSPACE, "workspace holds %zu bytes, needs %zu", workspace_bytes, need);
  lrh::DistillArgs d = distill_args(dtype, V, r, P, Z, N, idx, logits, k, temperature);
  d.loss = loss;
  d.lse = lse;
  d.G = grad;
  LRH_HIP(lrh::launch_distill(d, workspace, static_cast<hipStream_t>(stream)), "distillation launch");
  return LRHEAD_OK;
}

int lrhead_distill_grad(int dtype, int64_t V, int64_t r, const void* P, const void* Z, int64_t N, const int32_t* idx,
                        const float* logits, int k, float temperature, const float* lse, const float* grad,
                        const float* weight, void* dZ, void* dP, void* workspace, size_t workspace_bytes,
                        void* stream) {
  LRH_TRY(check_distill(dtype, V, r, N, k));
  LRH_TRY(check_temperature(temperature));
  if (N > 0 && (!P || !Z || !idx || !logits || !lse || !workspace))
    return fail(LRHEAD_EINVAL, "P, Z, idx, logits, lse and workspace must be non-NULL");
  if (N > 0 && dZ && !grad) return fail(LRHEAD_EINVAL, "dZ needs grad");
  if (!aligned16(P) || !aligned16(Z) || !aligned16(grad) || !aligned16(dZ) || !aligned16(dP) || !aligned16(workspace))
    return fail(LRHEAD_EALIGN, "P, Z, grad, dZ, dP and workspace must be 16-byte aligned");
  if (!aligned4(idx) || !aligned4(logits) || !aligned4(lse) || !aligned4(weight))
    return fail(LRHEAD_EALIGN, "idx, logits, lse and weight must be 4-byte aligned");
  lrh::DistillArgs d = distill_args(dtype, V, r, P, Z, N, idx, logits, k, temperature);
  if (N > 0) {
    const size_t need = lrh::distill_workspace_bytes(dtype, V, (int)r, N, k);
    if (workspace_bytes < need)
      return fail(LRHEAD_EWORKSPACE, "workspace holds %zu bytes, needs %zu", workspace_bytes, need);
  }
  d.lse = const_cast<float*>(lse);
  d.G = const_cast<float*>(grad);
  d.weight = weight;
  d.dZ = dZ;
  d.dP = dP;
  LRH_HIP(lrh::launch_distill_grad(d, workspace, static_cast<hipStream_t>(stream)), "distillation gradient launch");
  return LRHEAD_OK;
}

size_t lrhead_beam_workspace_bytes(int dtype, int64_t B, int m, int64_t n, int nb) {
  if (check_beam(dtype, B, m, n, nb) != LRHEAD_OK) return 0;
  return lrh::beam_workspace_bytes(dtype, B > 0 ? B : 1, m, n, nb);
}

int lrhead_beam_select(int dtype, const void* logits, int64_t ld, const int32_t* idx, const float* score,
                       const uint8_t* ended, int end_id, int64_t B, int m, int64_t n, int nb, float* out_score,
                       int32_t* out_beam, int32_t* out_token, void* workspace, size_t workspace_bytes, void* stream) {
  LRH_TRY(check_beam(dtype, B, m, n, nb));
  if (ld < n) return fail(LRHEAD_ERANGE, "ld = %lld below n = %lld", (long long)ld, (long long)n);
  if (B == 0) return LRHEAD_OK;
  if (!logits || !score || (!workspace && n > 64))
    return fail(LRHEAD_EINVAL, "logits, score and (for n > 64) workspace must be non-NULL");
  if (reinterpret_cast<uintptr_t>(logits) % elem_bytes(dtype))
    return fail(LRHEAD_EALIGN, "logits are not aligned to their elements");
  if (!aligned4(idx) || !aligned4(score) || !aligned16(workspace))
    return fail(LRHEAD_EALIGN, "idx and score must be 4-byte aligned, the workspace 16-byte");
  LRH_TRY(check_out(out_score, "out_score", true));
  LRH_TRY(check_out(out_beam, "out_beam", true));
  LRH_TRY(check_out(out_token, "out_token", true));
  const size_t need = lrh::beam_workspace_bytes(dtype, B, m, n, nb);
  if (workspace && workspace_bytes < need)
    return fail(LRHEAD_EWORKSPACE, "workspace holds %zu bytes, needs %zu", workspace_bytes, need);
  LRH_HIP(lrh::launch_beam_select(dtype, logits, ld, idx, score, ended, end_id, B, m, n, nb, out_score, out_beam,
                                  out_token, workspace, static_cast<hipStream_t>(stream)),
          "beam selection launch");
  return LRHEAD_OK;
}

int lrhead_reorder(const lrhead_state_t* states, int n_states, const int32_t* parent, const int32_t* length,
                   int64_t B, int m, int nb, void* stream) {
  if (n_states < 0 || n_states > LRHEAD_STATES_MAX)
    return fail(LRHEAD_ERANGE, "n_states = %d outside [0, %d]", n_states, LRHEAD_STATES_MAX);
  if (B < 0 || m < 1 || nb < 1) return fail(LRHEAD_ERANGE, "need B >= 0 and m, nb >= 1");
  if (B == 0 || n_states == 0) return LRHEAD_OK;
  if (!states || !parent) return fail(LRHEAD_EINVAL, "states and parent must be non-NULL");
  struct Range {   // half-open
    uintptr_t lo, hi;
    bool dst;
  };
  static thread_local Range ranges[2 * LRHEAD_STATES_MAX + 2];
  static thread_local lrh::BeamState moves[LRHEAD_STATES_MAX];
  int n = 0, n_moves = 0;
  for (int i = 0; i < n_states; ++i) {
    const lrhead_state_t& s = states[i];
    if (s.segs < 0 || s.positions < 0 || s.position_bytes < 0)
      return fail(LRHEAD_ERANGE, "state %d has a negative size", i);
    int64_t beam = 0, src = 0, dst = 0;
    if (__builtin_mul_overflow(s.segs, s.positions, &beam) || __builtin_mul_overflow(beam, s.position_bytes, &beam) ||
        __builtin_mul_overflow(beam, B, &beam) || __builtin_mul_overflow(beam, (int64_t)m, &src) ||
        __builtin_mul_overflow(beam, (int64_t)nb, &dst))
      return fail(LRHEAD_ERANGE, "state %d: its size passes 64 bits", i);
    if (beam == 0) continue;
    if (!s.src || !s.dst) return fail(LRHEAD_EINVAL, "state %d: src and dst must be non-NULL", i);
    const uintptr_t a = reinterpret_cast<uintptr_t>(s.src), b = reinterpret_cast<uintptr_t>(s.dst);
    ranges[n++] = {a, a + (uintptr_t)src, false};
    ranges[n++] = {b, b + (uintptr_t)dst, true};
    moves[n_moves++] = {s.src, s.dst, s.segs, s.positions, s.position_bytes};
  }
  int64_t slots = 0;
  if (__builtin_mul_overflow(B, (int64_t)nb * 4, &slots)) return fail(LRHEAD_ERANGE, "B nb passes 64 bits");
  ranges[n++] = {reinterpret_cast<uintptr_t>(parent), reinterpret_cast<uintptr_t>(parent) + (uintptr_t)slots, false};
  if (length)
    ranges[n++] = {reinterpret_cast<uintptr_t>(length), reinterpret_cast<uintptr_t>(length) + (uintptr_t)B * 4, false};
  std::sort(ranges, ranges + n, [](const Range& x, const Range& y) { return x.lo < y.lo; });
  uintptr_t any_end = 0, dst_end = 0;   // how far the ranges, and the destinations, before this one reach
  for (int i = 0; i < n; ++i) {
    if (ranges[i].lo < dst_end || (ranges[i].dst && ranges[i].lo < any_end))
      return fail(LRHEAD_EINVAL, "a destination overlaps another state, parent or length");
    any_end = std::max(any_end, ranges[i].hi);
    if (ranges[i].dst) dst_end = std::max(dst_end, ranges[i].hi);
  }
  LRH_HIP(lrh::launch_beam_move(moves, n_moves, parent, length, B, m, nb, static_cast<hipStream_t>(stream)),
          "state reordering launch");
  return LRHEAD_OK;
}

size_t lrhead_sample_workspace_bytes(int dtype, int64_t B, int64_t n) {
  if (check_sampling(dtype, B, 1, n) != LRHEAD_OK) return 0;
  return lrh::sample_workspace_bytes(B > 0 ? B : 1, n);
}

int lrhead_sample(int dtype, const void* logits, int64_t ld, const int32_t* idx, const float* u,
                  const lrhead_sampling_t* how, int64_t B, int64_t n, int32_t* token, float* prob, float* probs,
                  void* workspace, size_t workspace_bytes, void* stream) {
  LRH_TRY(check_sampling(dtype, B, 1, n));
  if (ld < n) return fail(LRHEAD_ERANGE, "ld = %lld below n = %lld", (long long)ld, (long long)n);
  if (probs && n > LRHEAD_K_MAX) return fail(LRHEAD_ERANGE, "probs with n = %lld above %d", (long long)n, LRHEAD_K_MAX);
  if (B == 0) return LRHEAD_OK;
  lrh::SampleArgs a{};
  LRH_TRY(sample_args(&a, dtype, logits, ld, u, how, n));
  if (!workspace && n > LRHEAD_K_MAX) return fail(LRHEAD_EINVAL, "workspace is NULL");
  if (!aligned4(idx) || !aligned16(workspace))
    return fail(LRHEAD_EALIGN, "idx must be 4-byte aligned, the workspace 16-byte");
  LRH_TRY(check_out(token, "token", true));
  LRH_TRY(check_out(prob, "prob", false));
  LRH_TRY(check_out(probs, "probs", false));
  const size_t need = lrh::sample_workspace_bytes(B, n);
  if (workspace && workspace_bytes < need)
    return fail(LRHEAD_EWORKSPACE, "workspace holds %zu bytes, needs %zu", workspace_bytes, need);
  const size_t rows = size_t(B) * 4, all = rows * size_t(n);
  if (clash({{token, rows}, {prob, rows}, {probs, all}, {workspace, need}},
            {{logits, (size_t(B - 1) * size_t(ld) + size_t(n)) * elem_bytes(dtype)}, {idx, all}, {u, rows},
             {how->temperature, rows}, {how->top_k, rows}, {how->top_p, rows}, {how->min_p, rows}}))
    return fail(LRHEAD_EINVAL, "an output or the workspace overlaps an input or another output");
  a.idx = idx;
  a.token = token;
  a.prob = prob;
  a.probs = probs;
  LRH_HIP(lrh::launch_sample(a, B, workspace, static_cast<hipStream_t>(stream)), "sampling launch");
  return LRHEAD_OK;
}

size_t lrhead_verify_workspace_bytes(int dtype, int64_t B, int s, int64_t n) {
  if (s < 0 || s > kVerifyMaxS || check_sampling(dtype, B, s + 1, n) != LRHEAD_OK) return 0;
  return lrh::verify_workspace_bytes(B > 0 ? B : 1, s, n);
}

int lrhead_verify(int dtype, const void* logits, int64_t ld, const int32_t* token, const int32_t* idx,
                  const float* probs, int k, const int32_t* length, const float* u, const lrhead_sampling_t* how,
                  int64_t B, int s, int64_t n, int32_t* out_token, int32_t* count, void* workspace,
                  size_t workspace_bytes, void* stream) {
  if (s < 0 || s > kVerifyMaxS) return fail(LRHEAD_ERANGE, "s = %d outside [0, %d]", s, kVerifyMaxS);
  LRH_TRY(check_sampling(dtype, B, s + 1, n));
  if (ld < n) return fail(LRHEAD_ERANGE, "ld = %lld below n = %lld", (long long)ld, (long long)n);
  if ((idx == nullptr) != (probs == nullptr)) return fail(LRHEAD_EINVAL, "idx and probs go together");
  if (idx && (k < 1 || k > LRHEAD_K_MAX)) return fail(LRHEAD_ERANGE, "k = %d outside [1, %d]", k, LRHEAD_K_MAX);
  if (B == 0) return LRHEAD_OK;
  lrh::SampleArgs a{};
  LRH_TRY(sample_args(&a, dtype, logits, ld, u, how, n));
  if ((!token && s > 0) || !workspace) return fail(LRHEAD_EINVAL, "token and workspace must be non-NULL");
  if (!aligned4(token) || !aligned4(idx) || !aligned4(probs) || !aligned4(length) || !aligned16(workspace))
    return fail(LRHEAD_EALIGN, "token, idx, probs and length must be 4-byte aligned, the workspace 16-byte");
  LRH_TRY(check_out(out_token, "out_token", true));
  LRH_TRY(check_out(count, "count", true));
  const size_t need = lrh::verify_workspace_bytes(B, s, n);
  if (workspace_bytes < need)
    return fail(LRHEAD_EWORKSPACE, "workspace holds %zu bytes, needs %zu", workspace_bytes, need);
  const size_t seqs = size_t(B) * 4, rows = seqs * size_t(s + 1), places = seqs * size_t(s);
  if (clash({{out_token, rows}, {count, seqs}, {workspace, need}},
            {{logits, ((size_t(B) * size_t(s + 1) - 1) * size_t(ld) + size_t(n)) * elem_bytes(dtype)},
             {token, places}, {idx, places * size_t(k)}, {probs, places * size_t(k)}, {length, seqs}, {u, rows},
             {how->temperature, seqs}, {how->top_k, seqs}, {how->top_p, seqs}, {how->min_p, seqs}}))
    return fail(LRHEAD_EINVAL, "an output or the workspace overlaps an input or another output");
  a.token = out_token;
  lrh::VerifyArgs v{};
  v.s = s;
  v.k = idx ? k : 1;
  v.drafted = token;
  v.list = idx;
  v.q = probs;
  v.length = length;
  v.count = count;
  LRH_HIP(lrh::launch_verify(a, v, B, workspace, static_cast<hipStream_t>(stream)), "verification launch");
  return LRHEAD_OK;
}

int lrhead_embed(int dtype, const void* W, int64_t V, int64_t d, const int32_t* token, int64_t N, float scale,
                 void* out, void* stream) {
  LRH_TRY(check_embed(dtype, V, d, N));
  if (!std::isfinite(scale)) return fail(LRHEAD_ERANGE, "scale is not finite");
  if (N == 0) return LRHEAD_OK;
  if (!W || !token || !out) return fail(LRHEAD_EINVAL, "W, token and out must be non-NULL");
  if (!aligned_elem(W, dtype) || !aligned_elem(out, dtype) || !aligned4(token))
    return fail(LRHEAD_EALIGN, "W, out and token must be aligned to their elements");
  const size_t row = size_t(d) * elem_bytes(dtype);
  if (clash({{out, size_t(N) * row}}, {{W, size_t(V) * row}, {token, size_t(N) * 4}}))
    return fail(LRHEAD_EINVAL, "out overlaps W or token");
  LRH_HIP(lrh::launch_embed(dtype, W, V, d, token, N, scale, out, static_cast<hipStream_t>(stream)),
          "embedding launch");
  return LRHEAD_OK;
}

size_t lrhead_embed_grad_workspace_bytes(int dtype, int64_t V, int64_t d, int64_t N) {
  if (check_embed(dtype, V, d, N) != LRHEAD_OK) return 0;
  return N > 0 ? lrh::embed_grad_workspace_bytes(dtype, V, d, N) : 256;
}

int lrhead_embed_grad(int dtype, const void* dY, const int32_t* token, int64_t N, int64_t V, int64_t d, float scale,
                      int add, void* dW, void* workspace, size_t workspace_bytes, void* stream) {
  LRH_TRY(check_embed(dtype, V, d, N));
  if (!std::isfinite(scale)) return fail(LRHEAD_ERANGE, "scale is not finite");
  if (!dW || (N > 0 && (!dY || !token || !workspace)))
    return fail(LRHEAD_EINVAL, "dY, token, dW and workspace must be non-NULL");
  if (!aligned_elem(dY, dtype) || !aligned_elem(dW, dtype) || !aligned4(token) || !aligned16(workspace))
    return fail(LRHEAD_EALIGN, "dY, dW and token must be aligned to their elements, the workspace to 16 bytes");
  const size_t row = size_t(d) * elem_bytes(dtype);
  if (N > 0) {
    const size_t need = lrh::embed_grad_workspace_bytes(dtype, V, d, N);
    if (workspace_bytes < need)
      return fail(LRHEAD_EWORKSPACE, "workspace holds %zu bytes, needs %zu", workspace_bytes, need);
    if (clash({{dW, size_t(V) * row}, {workspace, need}}, {{dY, size_t(N) * row}, {token, size_t(N) * 4}}))
      return fail(LRHEAD_EINVAL, "dW or the workspace overlaps dY or token, or each other");
  }
  LRH_HIP(lrh::launch_embed_grad(dtype, dY, token, N, V, d, scale, add != 0, dW, workspace,
                                 static_cast<hipStream_t>(stream)),
          "embedding gradient launch");
  return LRHEAD_OK;
}

int lrhead_set_stage_events(lrhead_t h, void* before, void* after) {
  LRH_TRY(check_handle(h));
  if ((before == nullptr) != (after == nullptr))
    return fail(LRHEAD_EINVAL, "give both events or neither");
  h->ev_before = static_cast<hipEvent_t>(before);
  h->ev_after = static_cast<hipEvent_t>(after);
  return LRHEAD_OK;
}

void lrhead_destroy(lrhead_t h) {
  if (h && h->magic == kMagic) {
    h->magic = 0;
    delete h;
  }
}

const char* lrhead_strerror(int code) {
  switch (code) {
    case LRHEAD_OK: return "success";
    case LRHEAD_EINVAL: return "invalid argument";
    case LRHEAD_ERANGE: return "size outside the supported range";
    case LRHEAD_EDTYPE: return "unknown dtype";
    case LRHEAD_EALIGN: return "pointer not 16-byte aligned";
    case LRHEAD_EWORKSPACE: return "workspace too small";
    case LRHEAD_EHIP: return "HIP error";
    case LRHEAD_EDEVICE: return "device is not gfx950";
    default: return "unknown error code";
  }
}

const char* lrhead_last_error(void) { return g_err; }

}  // extern "C"
