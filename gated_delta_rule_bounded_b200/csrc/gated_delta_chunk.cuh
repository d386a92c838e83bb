// gated_delta_chunk.cuh -- what the chunked kernels of the gated delta rule with one decay per value head share: the
// workspace blocks, tensor maps and bulk copies, the split of an fp32 value into two bf16 parts, bounded waits.
//
// Within a chunk of C = 64 tokens, with G_t the sum of the log decays up to token t, D[t][i] = e^{G_t - G_i} and S the
// state before the chunk:
//   M = strict(K K^T * D) diag(beta),  A = tril(Q K^T * D),  Z = -(I + M)^-1 M
//   R = V - e^G (K S);  delta = R + Z R;  U = beta delta
//   O = e^G (Q S) + A U;  S' = e^{G_C} S + (e^{G_C - G} K)^T U
// A scalar decay per token stays out of every operand: it scales rows of accumulators. So Q, K, V (and dO) enter the
// tensor cores as the bf16 values they are, exactly, and only what the kernels compute themselves has to be split:
// x = hi + lo, both bf16, leaves 2^-16 of x. Products of a split operand with an exact one take two MMAs, of two split
// ones three (hi hi, hi lo, lo hi), all accumulated in fp32; the state itself is carried in fp32 registers. Identity
// parts (delta = R + ..., not (I + Z) R) are added in fp32, outside the products.
#pragma once

#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <cstring>

#include "chunk_common.cuh"
#include "gated_delta.h"

namespace kda {
namespace {

// A workspace block per (chunk slot, value head): 64 x 64 bf16 tiles of 128-byte rows with the 128-byte swizzle, the
// images the MMAs read. [t][i] serves both as a K-major operand (N = t, K = i) and as an MN-major one (N = i, K = t).
constexpr int GB_ZH = 0;          // Z, high part
constexpr int GB_ZL = 8192;       // Z, low part
constexpr int GB_AH = 16384;      // A, high part
constexpr int GB_VEC = 24576;     // fp32 [64] each: e^G, e^{G_C - G}, beta, then e^{G_C} and a flag; 1 KB
constexpr int GB_BYTES = 25600;   // what the prefill reads
constexpr int GB_AL = 25600;      // A, low part (the gradients' blocks)
constexpr int GB_SUMS = 33792;    // the sums of log2 decays, high [64], low [64] (gradients only)
constexpr int GB_BYTES_BWD = 34304;
// Tokens 0-31 by tokens 32-63 of Z's two parts and of A's high part are zero, and no product of the prefill reads them: there,
// in that order, stand the quarters (0, 0), (1, 0) and (1, 1) of A's low part (the gradients read all of A, zeros too).
__host__ __device__ constexpr int gb_low_image(int h, int g) { return (h + g) * 8192; }
constexpr int VEC_E = 0, VEC_REST = 64, VEC_BETA = 128, VEC_ALL = 192, VEC_TINY = 193;  // floats within GB_VEC
// The least |beta| of a token in the gradients: 2^-66, 1e-20 of what the other tokens write, and dR = beta dY stays a normal
// number, and its two parts too, for dY down to 2^-51 (with 1e-30 dbeta lost digits from gradients of 1e-11 down).
constexpr float GD_TINY = 0x1p-66f;

__device__ __forceinline__ int64_t gd_slot_base(const GatedDeltaParams& p, int n, int64_t t0) {
  return p.cu ? t0 / C + n : (int64_t)n * ((p.T + C - 1) / C);
}

// The sequence, first token and number of tokens of a slot; 0 tokens where no sequence owns it.
__device__ __forceinline__ int gd_slot_tokens(const GatedDeltaParams& p, int64_t slot, int& n, int64_t& tc0, int64_t& brow) {
  int64_t t0, t1;
  if (p.cu) {
    int lo = 0, hi = p.N - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      gd_range(p, mid, t0, t1, brow);
      if (gd_slot_base(p, mid, t0) <= slot)
        lo = mid;
      else
        hi = mid - 1;
    }
    n = lo;
  } else {
    n = (int)((uint32_t)slot / (uint32_t)((p.T + C - 1) / C));  // slots and chunks are below 2^31
  }
  gd_range(p, n, t0, t1, brow);
  const int64_t j = slot - gd_slot_base(p, n, t0);
  tc0 = t0 + j * C;
  if (j < 0 || tc0 >= t1) return 0;
  return (int)min((int64_t)C, t1 - tc0);
}

// Few chains of many chunks leave most SMs idle. A sequence longer than L chunks is then split into segments of L: first
// every segment but the last runs from a state of zero, and once more as the map of states that it is (from the identity,
// its values zero); a small kernel joins them into the state at every segment's start; then all segments run at once. That
// is up to three times the work for as many times the SMs. The state at the start of segment s >= 1 is kept in the cell
// of span = 64 L tokens in which the segment starts; no two such segments start in one cell, since both their sequences
// would be longer than it. The maps likewise, in the cell after their segment.
constexpr int GD_SMS = 148;
}  // namespace
struct GatedDeltaSplit {
  const int* plan;  // L in device memory (packed sequences: their lengths are known there), or nullptr
  const int* order; // packed sequences by length, the longest first: its blocks should not start last; or nullptr
  int chunks;       // else L; 0: no splitting
  float* x;         // [cell][HV][K][V]
  float* m;         // [cell][HV] maps, transposed [K][K]; the cell of segment 1, which needs none, may hold a copy [K][V]
                    // of the sequence's given state, where the call overwrites that
  float* mb;        // the maps as they are, for the gradients, or nullptr
  int64_t x_size, m_size;  // floats of each
  __device__ __forceinline__ int length() const { return plan ? *plan : chunks; }
};
namespace {
struct GatedDeltaSegment {
  int n, s, count;            // sequence, segment and how many the sequence has
  int64_t t0, first, end, brow;
  int64_t cell0;              // segment s starts in cell cell0 + s (s >= 1)
};

__device__ __forceinline__ void gd_describe(const GatedDeltaParams& p, int n, int64_t span, GatedDeltaSegment& g) {
  int64_t t1;
  gd_range(p, n, g.t0, t1, g.brow);
  g.n = n;
  g.count = span && t1 - g.t0 > span ? (int)((t1 - g.t0 + span - 1) / span) : 1;
  g.cell0 = !span ? 0 : p.cu ? g.t0 / span : n * ((p.T + span - 1) / span);
  g.end = t1;
}
__device__ __forceinline__ void gd_place(GatedDeltaSegment& g, int s, int64_t span) {
  g.s = s;
  g.first = g.t0 + s * span;
  if (s + 1 < g.count) g.end = g.first + span;
}
// Segment number `at` of a call; false where no sequence owns the number.
__device__ __forceinline__ bool gd_segment(const GatedDeltaParams& p, int64_t at, int L, const int* order, GatedDeltaSegment& g) {
  const int64_t span = (int64_t)L * C;
  int64_t n = at, s = 0;
  if (span && p.cu) {
    int64_t t0, t1, brow;
    int lo = 0, hi = p.N - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      gd_range(p, mid, t0, t1, brow);
      if (t0 / span + mid <= at)
        lo = mid;
      else
        hi = mid - 1;
    }
    gd_range(p, lo, t0, t1, brow);
    n = lo;
    s = at - (t0 / span + lo);
  } else if (span) {
    const int64_t each = (p.T + span - 1) / span;
    n = at / each;
    s = at % each;
  }
  if (n >= p.N || s < 0) return false;
  if (!span && order) n = order[n];
  gd_describe(p, (int)n, span, g);
  if (s >= g.count) return false;
  gd_place(g, (int)s, span);
  return true;
}
// The segment s >= 1 that starts in a cell; false where none does.
__device__ __forceinline__ bool gd_cell(const GatedDeltaParams& p, int64_t cell, int L, GatedDeltaSegment& g) {
  const int64_t span = (int64_t)L * C;
  if (!span) return false;
  int64_t s;
  if (p.cu) {
    int64_t t0, t1, brow;
    int lo = 0, hi = p.N - 1;
    while (lo < hi) {  // the last sequence that starts no later than the cell
      const int mid = (lo + hi + 1) >> 1;
      gd_range(p, mid, t0, t1, brow);
      if (t0 <= cell * span)
        lo = mid;
      else
        hi = mid - 1;
    }
    gd_describe(p, lo, span, g);
    s = (cell * span - g.t0 + span - 1) / span;
  } else {
    const int64_t each = (p.T + span - 1) / span;
    if (cell >= p.N * each) return false;
    gd_describe(p, (int)(cell / each), span, g);
    s = cell % each;
  }
  if (s < 1 || s >= g.count) return false;
  gd_place(g, (int)s, span);
  return g.cell0 + s == cell;
}

__device__ __forceinline__ void gd_tma_load(uint32_t dst, const CUtensorMap* map, int x, int h, int t, int b, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(h), "r"(t), "r"(b), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void gd_tma_store(const CUtensorMap* map, uint32_t src, int x, int h, int t, int b) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(h), "r"(t), "r"(b), "r"(src)
               : "memory");
}
__device__ __forceinline__ void gd_bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void gd_bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void gd_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void gd_bar_init(uint32_t bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
template <int ID, int THREADS>
__device__ __forceinline__ void named_arrive() {
  asm volatile("bar.arrive %0, %1;" ::"n"(ID), "n"(THREADS) : "memory");
}
template <int ID, int THREADS>
__device__ __forceinline__ void named_sync() {
  asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(THREADS) : "memory");
}

// A bounded wait that gives up for the whole block: once one has expired, `*dead` is set, every later wait that is not
// already over returns at once and nothing new is issued, so the block runs to its end. A phase that is over costs one
// test; one that is not suspends the thread: polling would take issue slots and shared-memory cycles from the other warps.
__device__ __forceinline__ bool gd_test(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile("{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(done)
               : "r"(bar), "r"(parity)
               : "memory");
  return done != 0;
}
__device__ __forceinline__ void gd_wait(uint32_t bar, uint32_t parity, volatile int* dead, int* flag) {
  if (gd_test(bar, parity)) return;
  if (*dead) return;
  if (!mbar_try_wait_bounded(bar, parity)) {
    *dead = 1;
    atomicExch(flag, 1);
  }
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(f2_bits(a)), "l"(f2_bits(b)), "l"(f2_bits(c)));
  return bits_f2(d);
}
// x = hi + lo of two neighbouring values, each part a packed bf16 pair.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16(x, y);
  const float2 r = fma2(make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)), make_float2(-1.f, -1.f),
                        make_float2(x, y));
  lo = pack_bf16(r.x, r.y);
}
__device__ __forceinline__ float2 as_f2(uint32_t a, uint32_t b) { return make_float2(__uint_as_float(a), __uint_as_float(b)); }

__device__ __forceinline__ void tm_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tm_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_alloc(uint32_t slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols));
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tm_dealloc(uint32_t tmem, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
}

// One warp: the running sums of a chunk's log2 decays, in fp64 (lane l holds tokens 2l and 2l + 1), as two fp32 parts
// in gh and gl, and the block's vectors. Tokens past the sequence's end get no decay and no write strength. Strengths of a
// magnitude below `least` count as that.
__device__ __forceinline__ void gd_decays(const GatedDeltaParams& p, int hv, int64_t tc0, int64_t brow, int nv, int lane,
                                          float least, float* vec, float* gh, float* gl) {
  const float* g = p.g + brow * p.gs[0] + hv * p.gs[2] + tc0 * p.gs[1];
  const float* beta = p.beta + brow * p.bs[0] + hv * p.bs[2] + tc0 * p.bs[1];
  double x[2];
  bool tiny = false;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int t = 2 * lane + e;
    x[e] = t < nv ? (double)g[t * p.gs[1]] * 1.4426950408889634 : 0.0;
    // Far below what 2^x can hold, so that g = -inf keeps the sums' differences defined (and NaN stays NaN).
    x[e] = x[e] < -1e4 ? -1e4 : x[e];
    // In the gradients a write strength of zero becomes one too small to matter, so that dY = dR / beta is defined; VEC_TINY tells.
    const float b = t < nv ? beta[t * p.bs[1]] : 0.f;
    const bool small = t < nv && fabsf(b) < least;
    vec[VEC_BETA + t] = small ? least : b;
    tiny |= small;
  }
  double sum = x[0] + x[1];
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, sum, m);
    if (lane >= m) sum += y;
  }
  const double total = __shfl_sync(0xffffffffu, sum, 31);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int t = 2 * lane + e;
    const double G = e ? sum : sum - x[1];
    gh[t] = (float)G;
    gl[t] = (float)(G - (double)gh[t]);
    vec[VEC_E + t] = ex2((float)G);
    vec[VEC_REST + t] = ex2((float)(total - G));
  }
  tiny = __any_sync(0xffffffffu, tiny);
  if (lane == 0) {
    vec[VEC_ALL] = ex2((float)total);
    vec[VEC_TINY] = tiny ? 1.f : 0.f;
  }
}

// Zeroes rows [first, 64) of a tile of `atoms` 8 KB atoms of 128-byte rows (rows of 256 bytes when `atoms` is 0), by the
// `count` threads with index `idx`.
__device__ __forceinline__ void zero_rows(unsigned char* tile, int atoms, int first, int idx, int count) {
  const int pieces = (64 - first) * 16;  // 16-byte pieces of the 256 bytes a token has
  for (int e = idx; e < pieces; e += count) {
    const int row = first + (e >> 4), c = e & 15;
    unsigned char* at = atoms ? tile + (c >> 3) * 8192 + row * 128 + (c & 7) * 16 : tile + row * 256 + c * 16;
    *reinterpret_cast<uint4*>(at) = make_uint4(0u, 0u, 0u, 0u);
  }
}

template <typename F>
cudaError_t gd_smem_once(F* fn, int bytes, std::atomic<uint64_t>& configured) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;  // one configuration bit per device
  const uint64_t bit = 1ull << dev;
  if (!(configured.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  return cudaSuccess;
}

// A bf16 token tensor [B,T,heads,D] (element strides s = (b, t, h)) as a tensor map (D, heads, T, B), moved in boxes of
// `box` channels x 64 tokens of one head; channels past D read as zeros and are not written. The stride of an extent-1
// dimension never moves the pointer; it is given its contiguous value.
inline bool gd_token_map(CUtensorMap* m, const void* base, const int64_t s[3], int64_t B, int64_t T, int64_t heads, int64_t D,
                         int box, bool swizzle) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return static_cast<Encode>(nullptr);
    return reinterpret_cast<Encode>(f);
  }();
  if (!fn) return false;
  const int64_t sh = heads > 1 ? s[2] : D;
  const int64_t st = T > 1 ? s[1] : heads * sh;
  const int64_t sbt = B > 1 ? s[0] : T * st;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)T, (cuuint64_t)B};
  const cuuint64_t strides[3] = {(cuuint64_t)(sh * 2), (cuuint64_t)(st * 2), (cuuint64_t)(sbt * 2)};
  const cuuint32_t bx[4] = {(cuuint32_t)box, 1, (cuuint32_t)C, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, bx, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// Whether the chunked kernels take a shape, and the slots of a call.
inline bool gd_chunk_shape(int64_t K, int64_t V, kda_dtype dt) { return dt == KDA_BF16 && K <= 128 && V <= 256; }
inline int64_t gd_slots(int64_t B, int64_t T, int64_t n_seq) {
  return n_seq > 0 ? T / C + n_seq + 1 : B * ((T + C - 1) / C);
}

// How a call's sequences are split. Segments shorter than an SM's share of the chunks bring nothing: `least`, the
// shortest length considered, is three quarters of it, so that there are some 200 segments and as many cells at most.
struct GatedDeltaSplitShape {
  int chunks;     // L for every sequence; 0: whole, or (`packed`) left to the device, which knows the lengths
  int least;
  bool packed, grads;
  int64_t cells, segments;  // at most; 0: nothing is split
  int64_t ordered;          // sequences that are put in order
  size_t bytes;             // of the cells, the device's L and the order
};
GatedDeltaSplitShape gd_split_shape(int64_t B, int64_t T, int64_t HV, int64_t K, int64_t V, int64_t n_seq, bool grads);
// Lays a split's cells out at `ws`, which may be nullptr.
GatedDeltaSplit gd_split_carve(const GatedDeltaSplitShape& z, void* ws, int64_t HV, int64_t K, int64_t V);
// The states at the segments' starts from those of segments run from zero, or (`back`) the gradients at their ends; `given`:
// the sequences' own states (or final gradients), copied aside where `keep`.
cudaError_t launch_gated_delta_join(const GatedDeltaParams& p, const GatedDeltaSplit& split, const float* given, bool keep,
                                    bool back, cudaStream_t s);

// The forward's kernels, as the gradients use them too: with `dump` set, the block size is GB_BYTES_BWD and the
// chain also writes each chunk's start state and deltas there.
struct GatedDeltaDump {
  unsigned char* s;  // per (slot, value head): S^T [v][k] bf16, high 32 KB then low 32 KB (two 64-channel atoms each)
  unsigned char* delta;  // per (slot, value head): delta^T [v][t] bf16, high 16 KB then low 16 KB, one 64-token atom
};
cudaError_t launch_gated_delta_forward(const GatedDeltaParams& p, unsigned char* blocks, const GatedDeltaDump* dump,
                                       const GatedDeltaSplitShape& z, const GatedDeltaSplit& split, cudaStream_t s);

}  // namespace kda
