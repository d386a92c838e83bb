// layer_norm.cu -- layer norm over rows, forward and backward: of every head's output (rows of V values) or of a whole
// token (rows of H * V values).
//
//   forward    mean = sum x / D,  rstd = 1 / sqrt(sum (x - mean)^2 / D + eps),  y = (x - mean) rstd w + b
//   backward   with h = (x - mean) rstd and e = dy w:
//                dx = rstd (e - sum e / D - h sum (e h) / D),  dw = sum_rows dy h,  db = sum_rows dy
//
// Both are bound by memory: 2 (forward) or 3 (backward) element transfers for some ten operations, which only holds as
// long as the operations are few: all of them work on two values an instruction (f32x2). Every row is read once, in
// 16-byte pieces, and stays in registers between the sums and the result: a group of G lanes holds a row of one piece a
// lane (G = 8, 16 or 32, whichever leaves the fewest idle lanes; several rows a warp for the short rows of a head), or a
// whole block holds it. A lane loads the rows of the next round before it reduces this round's (forward: two rows at a
// time where rows are short). The variance is taken from the differences to the mean (a second pass over registers), not from a
// difference of two sums, which loses digits where the mean is large. Rows whose length or alignment does not allow
// 16-byte pieces take the same kernels with pieces of one element.
//
// The weight's gradient is a sum over rows. Each block walks rows with a fixed stride and keeps its share of dw and db
// in registers (the columns of a lane are the same in every row; in shared memory where a block has so many threads that
// they would not fit), the shares of a block's groups meet in shared memory, one partial row per block goes to the
// workspace, and a second kernel adds the partial rows. The order of the sums depends on the sizes alone: the same
// inputs give the same bits, with no atomics.
//
// Measured, bf16, L2 flushed before each call: 393,216 rows of 128 forward 39 us (5.2 TB/s of 6.6 a copy reaches),
// backward 70 us (4.4 TB/s), 4 of them for the sum of the partial rows; 8,191 rows of 2,047 in fp32, pieces of one element,
// backward 51 us, the kernels 48 + 5 against 43 + 5 for 8,192 rows of 2,048; a call of 64 rows of 12,288 4.3 us of kernel.
// In the backward pass of short rows nothing is saturated (L1 and shared memory 69 %, issue 59 %, DRAM 51 %): a warp waits
// in turn on its loads and on the eight shuffles a row. Tried, when it took 76 us: eight lanes a row with two pieces each,
// 88; rows staged by asynchronous copies four rounds ahead in shared memory, 74, but 165 instead of 131 for rows of 4,096.
#include <algorithm>
#include <atomic>

#include "chunk_common.cuh"
#include "gated_delta.h"

namespace kda {
namespace {

constexpr int BWD_BLOCKS = 4;                   // backward blocks of 256 threads an SM: 64 registers a thread
constexpr int LN_MAX_PARTS = 148 * BWD_BLOCKS;  // partial rows of dw and db (blocks of the backward kernel)

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Piece {
  T v[VEC];
};

template <int G>
__device__ __forceinline__ float group_sum(float x, float* red) {
  if constexpr (G > 0) {
#pragma unroll
    for (int m = G / 2; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
  } else {  // the whole block; `red` holds 32 floats
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    x = (threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
  }
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(f2_bits(a)), "l"(f2_bits(b)), "l"(f2_bits(c)));
  return bits_f2(d);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// A lane's share of a row: NV pieces of VEC elements, piece i from element (l + i g) VEC on. As values it is E / 2 pairs
// (one pair, the second value unused, for a single element); what lies past the row is zero.
template <typename T, int VEC, int NV>
struct Share {
  static constexpr int E = VEC * NV, PAIRS = (E + 1) / 2;
  Piece<T, VEC> p[NV];
  __device__ __forceinline__ void load(const T* row, int l, int g, int pieces) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (l + i * g < pieces) {
        p[i] = *reinterpret_cast<const Piece<T, VEC>*>(row + (int64_t)(l + i * g) * VEC);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) p[i].v[e] = from_f32<T>(0.f);
      }
    }
  }
  __device__ __forceinline__ float2 pair(int j) const {
    if constexpr (E == 1) return make_float2(to_f32(p[0].v[0]), 0.f);
    if constexpr (VEC == 1) return make_float2(to_f32(p[2 * j].v[0]), to_f32(p[(2 * j + 1) % NV].v[0]));
    if constexpr (sizeof(T) == 2 && VEC > 1) {
      const uint32_t u = *reinterpret_cast<const uint32_t*>(&p[2 * j / VEC].v[2 * j % VEC]);
      return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
    return make_float2(to_f32(p[2 * j / VEC].v[2 * j % VEC]), to_f32(p[2 * j / VEC].v[(2 * j + 1) % VEC]));
  }
  __device__ __forceinline__ void put(int j, float2 x) {
    if constexpr (E == 1) {
      p[0].v[0] = from_f32<T>(x.x);
    } else if constexpr (VEC == 1) {
      p[2 * j].v[0] = from_f32<T>(x.x);
      p[(2 * j + 1) % NV].v[0] = from_f32<T>(x.y);
    } else if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<uint32_t*>(&p[2 * j / VEC].v[2 * j % VEC]) = pack_bf16(x.x, x.y);
    } else {
      p[2 * j / VEC].v[2 * j % VEC] = from_f32<T>(x.x);
      p[2 * j / VEC].v[(2 * j + 1) % VEC] = from_f32<T>(x.y);
    }
  }
  __device__ __forceinline__ void store(T* row, int l, int g, int pieces) const {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (l + i * g < pieces) *reinterpret_cast<Piece<T, VEC>*>(row + (int64_t)(l + i * g) * VEC) = p[i];
  }
  // 1 where pair j's values belong to the row, 0 where not.
  static __device__ __forceinline__ float2 mask(int j, int l, int g, int pieces) {
    if constexpr (E == 1) return make_float2(l < pieces ? 1.f : 0.f, 0.f);
    if constexpr (VEC == 1) return make_float2(l + 2 * j * g < pieces ? 1.f : 0.f, l + (2 * j + 1) * g < pieces ? 1.f : 0.f);
    return both(l + (2 * j / VEC) * g < pieces ? 1.f : 0.f);
  }
};

template <int N>
__device__ __forceinline__ float sum_pairs(const float2 (&x)[N]) {
  float2 s = x[0];
#pragma unroll
  for (int j = 1; j < N; ++j) s = add2(s, x[j]);
  return s.x + s.y;
}

// The rows a block walks: R at a time for each group, `step` apart from one round to the next.
template <int R>
struct Walk {
  int64_t first, step, rounds;
  __device__ __forceinline__ Walk(int64_t rows, int group, int per_block) {
    first = (int64_t)blockIdx.x * per_block * R + group;
    step = (int64_t)gridDim.x * per_block * R;
    // Every lane of a warp makes the same number of rounds: the shuffles name the whole warp.
    rounds = (rows - (int64_t)blockIdx.x * per_block * R + step - 1) / step;
  }
};

// FULL: every lane's pieces lie in the row.
template <typename TX, typename TW, int VEC, int NV, int G, int R, int THREADS, bool FULL>
__global__ void __launch_bounds__(THREADS) layer_norm_kernel(LayerNormParams p) {
  __shared__ float red[2][32];
  using X = Share<TX, VEC, NV>;
  using W = Share<TW, VEC, NV>;
  constexpr int N = X::PAIRS;
  const int g = G > 0 ? G : blockDim.x;
  const int l = G > 0 ? threadIdx.x % (G > 0 ? G : 1) : threadIdx.x;
  const int per_block = G > 0 ? blockDim.x / (G > 0 ? G : 1) : 1;
  const int pieces = FULL ? 1 << 30 : p.D / VEC;
  const float inv_d = 1.f / (float)p.D;
  const TX* x = static_cast<const TX*>(p.x);
  TX* y = static_cast<TX*>(p.y);
  W w, b;
  if (p.weight) {
    w.load(static_cast<const TW*>(p.weight), l, g, pieces);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) w.put(j, both(1.f));
  }
  if (p.bias) {
    b.load(static_cast<const TW*>(p.bias), l, g, pieces);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) b.put(j, both(0.f));
  }
  const Walk<R> walk(p.rows, G > 0 ? threadIdx.x / (G > 0 ? G : 1) : 0, per_block);
  X next[R];
  auto fetch = [&](int64_t row0) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (row0 + (int64_t)r * per_block < p.rows) next[r].load(x + (row0 + (int64_t)r * per_block) * p.x_stride, l, g, pieces);
  };
  constexpr bool AHEAD = THREADS <= 512;  // beyond, the registers do not hold two rows
  if (AHEAD && walk.rounds > 0) fetch(walk.first);
  for (int64_t n = 0; n < walk.rounds; ++n) {
    const int64_t row0 = walk.first + n * walk.step;
    if (!AHEAD) fetch(row0);
    float2 v[R][N];
    float mean[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int j = 0; j < N; ++j) v[r][j] = next[r].pair(j);
    }
    if (AHEAD) fetch(row0 + walk.step);
#pragma unroll
    for (int r = 0; r < R; ++r) mean[r] = group_sum<G>(sum_pairs(v[r]), red[0]) * inv_d;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 sq = both(0.f);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        v[r][j] = add2(v[r][j], both(-mean[r]));
        if (!FULL || X::E == 1) v[r][j] = mul2(v[r][j], X::mask(j, l, g, pieces));
        sq = fma2(v[r][j], v[r][j], sq);
      }
      // rsqrt is good to two units in the last place.
      rstd[r] = rsqrtf(group_sum<G>(sq.x + sq.y, red[1]) * inv_d + p.eps);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = row0 + (int64_t)r * per_block;
      if (row >= p.rows) continue;
      X out;
#pragma unroll
      for (int j = 0; j < N; ++j) out.put(j, fma2(v[r][j], mul2(w.pair(j), both(rstd[r])), b.pair(j)));
      out.store(y + row * p.D, l, g, pieces);
      if (l == 0) {
        p.mean[row] = mean[r];
        p.rstd[row] = rstd[r];
      }
    }
  }
}

// SUMS: dw and db in shared memory instead of registers (a block a row only).
template <typename TX, typename TW, int VEC, int NV, int G, int THREADS, bool FULL, bool SUMS>
__global__ void __launch_bounds__(THREADS, G > 0 ? BWD_BLOCKS : 1) layer_norm_backward_kernel(LayerNormParams p) {
  __shared__ float red[2][2][32];
  extern __shared__ float part[];  // G > 0: [2][D] sums of the block's groups; SUMS: [2 N][threads] pairs
  using X = Share<TX, VEC, NV>;
  using W = Share<TW, VEC, NV>;
  constexpr int N = X::PAIRS;
  const int g = G > 0 ? G : blockDim.x;
  const int l = G > 0 ? threadIdx.x % (G > 0 ? G : 1) : threadIdx.x;
  const int per_block = G > 0 ? blockDim.x / (G > 0 ? G : 1) : 1;
  const int group = G > 0 ? threadIdx.x / (G > 0 ? G : 1) : 0;
  const int pieces = FULL ? 1 << 30 : p.D / VEC;
  const float inv_d = 1.f / (float)p.D;
  const TX* x = static_cast<const TX*>(p.x);
  const TX* dy = static_cast<const TX*>(p.dy);
  TX* dx = static_cast<TX*>(p.dx);
  W w;
  if (p.weight) {
    w.load(static_cast<const TW*>(p.weight), l, g, pieces);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) w.put(j, both(1.f));
  }
  float2 dw[SUMS ? 1 : N], db[SUMS ? 1 : N];
  float2* mine = reinterpret_cast<float2*>(part) + threadIdx.x;  // SUMS: pair j of dw at mine[2 j threads], of db one further
#pragma unroll
  for (int j = 0; j < N; ++j) {
    if constexpr (SUMS)
      mine[2 * j * blockDim.x] = mine[(2 * j + 1) * blockDim.x] = both(0.f);
    else
      dw[j] = db[j] = both(0.f);
  }
  const Walk<1> walk(p.rows, group, per_block);
  X nx, ng;
  float nm = 0.f, nr = 0.f;
  auto fetch = [&](int64_t row) {
    if (row < p.rows) {
      nx.load(x + row * p.x_stride, l, g, pieces);
      ng.load(dy + row * p.dy_stride, l, g, pieces);
      nm = p.mean[row];
      nr = p.rstd[row];
    } else {  // a row past the end adds nothing to the sums
#pragma unroll
      for (int j = 0; j < N; ++j) {
        nx.put(j, both(0.f));
        ng.put(j, both(0.f));
      }
      nm = nr = 0.f;
    }
  };
  constexpr bool AHEAD = THREADS <= 512;  // beyond, the registers do not hold two rows
  if (AHEAD) fetch(walk.first);
  for (int64_t n = 0; n < walk.rounds; ++n) {
    const int64_t row = walk.first + n * walk.step;
    if (!AHEAD) fetch(row);
    float2 h[N], e[N], a = both(0.f), b = a;
    const float rstd = nr;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      h[j] = mul2(add2(nx.pair(j), both(-nm)), both(rstd));
      e[j] = ng.pair(j);  // dy; zero past the row
    }
    if (AHEAD) fetch(row + walk.step);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if constexpr (SUMS) {
        float2 *pw = mine + 2 * j * blockDim.x, *pb = pw + blockDim.x;
        *pw = fma2(e[j], h[j], *pw);
        *pb = add2(*pb, e[j]);
      } else {
        dw[j] = fma2(e[j], h[j], dw[j]);
        db[j] = add2(db[j], e[j]);
      }
      e[j] = mul2(e[j], w.pair(j));
      a = add2(a, e[j]);
      b = fma2(e[j], h[j], b);
    }
    const float s1 = group_sum<G>(a.x + a.y, red[n & 1][0]) * inv_d;
    const float s2 = group_sum<G>(b.x + b.y, red[n & 1][1]) * inv_d;
    if (row < p.rows) {
      X out;
#pragma unroll
      for (int j = 0; j < N; ++j) out.put(j, mul2(both(rstd), add2(e[j], fma2(h[j], both(-s2), both(-s1)))));
      out.store(dx + row * p.D, l, g, pieces);
    }
  }
  if (!p.parts) return;
  float* out = p.parts + (int64_t)blockIdx.x * 2 * p.D;
  const int real = p.D / VEC;
  auto column = [&](int j, int e) { return X::E == 1 ? l : (VEC == 1 ? l + (2 * j + e) * g : (l + (2 * j / VEC) * g) * VEC + 2 * j % VEC + e); };
  auto inside = [&](int j, int e) { return X::E == 1 ? (e == 0 && l < real) : (VEC == 1 ? l + (2 * j + e) * g < real : l + (2 * j / VEC) * g < real); };
  if constexpr (G > 0) {
    // The groups add their shares one after another: a fixed order.
    for (int r = 0; r < per_block; ++r) {
      if (group == r) {
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (inside(j, e)) {
              float* a = part + column(j, e);
              const float u = e ? dw[j].y : dw[j].x, v = e ? db[j].y : db[j].x;
              a[0] = r ? a[0] + u : u;
              a[p.D] = r ? a[p.D] + v : v;
            }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < 2 * p.D; c += blockDim.x) out[c] = part[c];
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float2 u = SUMS ? mine[2 * j * blockDim.x] : dw[SUMS ? 0 : j], v = SUMS ? mine[(2 * j + 1) * blockDim.x] : db[SUMS ? 0 : j];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (inside(j, e)) {
          out[column(j, e)] = e ? u.y : u.x;
          out[p.D + column(j, e)] = e ? v.y : v.x;
        }
    }
  }
}

// dw and db: the sums of the partial rows. A block takes 32 of the 2 D columns; its 32 warps walk the parts.
template <typename TW>
__global__ void layer_norm_parts_kernel(const float* parts, int n, int D, TW* dw, TW* db) {
  __shared__ float red[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x;
  float sum = 0.f, more[3] = {0.f, 0.f, 0.f};
  if (col < 2 * D) {
    int r = threadIdx.y;
    for (; r + 96 < n; r += 128) {
      sum += parts[(int64_t)r * 2 * D + col];
#pragma unroll
      for (int i = 0; i < 3; ++i) more[i] += parts[(int64_t)(r + 32 * i + 32) * 2 * D + col];
    }
    for (; r < n; r += 32) sum += parts[(int64_t)r * 2 * D + col];
  }
  sum += (more[0] + more[1]) + more[2];
  red[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  sum = red[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
  const int c = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && c < 2 * D) {
    TW* out = c < D ? dw : db;
    if (out) out[c < D ? c : c - D] = from_f32<TW>(sum);
  }
}

template <typename TX, typename TW, int VEC, int NV, int G, int R, int THREADS, bool FULL>
cudaError_t launch_full(const LayerNormParams& p, int threads, cudaStream_t s) {
  const int64_t per_block = (G > 0 ? threads / (G > 0 ? G : 1) : 1) * R;
  const int64_t blocks = (p.rows + per_block - 1) / per_block;
  if (p.dx) {
    constexpr bool SUMS = G == 0 && VEC * NV > 8;
    auto kernel = layer_norm_backward_kernel<TX, TW, VEC, NV, G, THREADS, FULL, SUMS>;
    const int64_t rows_at_once = G > 0 ? threads / (G > 0 ? G : 1) : 1;
    const int grid = (int)std::min<int64_t>((p.rows + rows_at_once - 1) / rows_at_once, layer_norm_parts(p.rows, p.D));
    const size_t smem = G > 0 ? (p.parts ? 2 * (size_t)p.D * sizeof(float) : 0) : (SUMS ? 2 * (size_t)VEC * NV * threads * sizeof(float) : 0);
    if (SUMS) {  // beyond the 48 KB a kernel has without asking
      static std::atomic<uint64_t> configured{0};
      int dev = 0;
      cudaError_t e = cudaGetDevice(&dev);
      if (e == cudaSuccess && (dev < 0 || dev >= 64)) e = cudaErrorInvalidDevice;  // one configuration bit per device
      if (e == cudaSuccess && !(configured.load(std::memory_order_relaxed) >> dev & 1)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * VEC * NV * THREADS * (int)sizeof(float));
        if (e == cudaSuccess) configured.fetch_or(1ull << dev);
      }
      if (e != cudaSuccess) return e;
    }
    kernel<<<grid, threads, smem, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !p.parts) return e;
    layer_norm_parts_kernel<TW><<<(2 * p.D + 31) / 32, dim3(32, 32), 0, s>>>(
        p.parts, grid, p.D, static_cast<TW*>(p.dweight), static_cast<TW*>(p.dbias));
  } else {
    // Blocks walk rows too: the weights are read once a block. Up to 2,048 threads on each of 148 SMs, twice over.
    const int grid = (int)std::min<int64_t>(blocks, 148 * 2 * (2048 / threads));
    layer_norm_kernel<TX, TW, VEC, NV, G, R, THREADS, FULL><<<grid, threads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

template <typename TX, typename TW, int VEC, int NV, int G, int R, int THREADS>
cudaError_t launch_one(const LayerNormParams& p, int threads, cudaStream_t s) {
  return p.D == VEC * NV * (G > 0 ? G : threads) ? launch_full<TX, TW, VEC, NV, G, R, THREADS, true>(p, threads, s)
                                                 : launch_full<TX, TW, VEC, NV, G, R, THREADS, false>(p, threads, s);
}

// How a call's rows are spread: lanes a row (G, 0: a block), pieces a lane, rows at a time.
template <typename TX, typename TW, int VEC>
cudaError_t launch_vec(const LayerNormParams& p, cudaStream_t s) {
  const int pieces = p.D / VEC;
  if (pieces <= 8) return launch_one<TX, TW, VEC, 1, 8, 2, 256>(p, 256, s);
  if (pieces <= 16) return launch_one<TX, TW, VEC, 1, 16, 2, 256>(p, 256, s);
  if (pieces <= 32) return launch_one<TX, TW, VEC, 1, 32, 2, 256>(p, 256, s);
  // A block a row: eight elements a thread up to 512 threads, then as many as 1,024 threads need.
  auto threads = [&](int nv) { return ((pieces + nv - 1) / nv + 31) / 32 * 32; };
  if constexpr (VEC == 8) {
    if (pieces <= 512) return launch_one<TX, TW, VEC, 1, 0, 1, 512>(p, threads(1), s);
    return launch_one<TX, TW, VEC, 2, 0, 1, 1024>(p, threads(2), s);  // a row of 16,384 values has 2,048 pieces
  } else if constexpr (VEC == 4) {
    if (pieces <= 1024) return launch_one<TX, TW, VEC, 2, 0, 1, 512>(p, threads(2), s);
    return launch_one<TX, TW, VEC, 4, 0, 1, 1024>(p, threads(4), s);
  } else {
    if (pieces <= 4096) return launch_one<TX, TW, VEC, 8, 0, 1, 512>(p, threads(8), s);
    return launch_one<TX, TW, VEC, 16, 0, 1, 1024>(p, threads(16), s);
  }
}

bool aligned_rows(const void* ptr, int64_t stride, int64_t rows, size_t es) {
  return (reinterpret_cast<uintptr_t>(ptr) & 15) == 0 && (rows <= 1 || (stride * (int64_t)es) % 16 == 0);
}

template <typename TX, typename TW>
cudaError_t launch_types(const LayerNormParams& p, cudaStream_t s) {
  constexpr int VEC = 16 / (int)sizeof(TX);
  const bool wide = p.D % VEC == 0 && aligned_rows(p.x, p.x_stride, p.rows, sizeof(TX)) &&
                    (!p.y || aligned_rows(p.y, p.D, p.rows, sizeof(TX))) &&
                    (!p.dx || aligned_rows(p.dx, p.D, p.rows, sizeof(TX))) &&
                    (!p.dy || aligned_rows(p.dy, p.dy_stride, p.rows, sizeof(TX))) &&
                    (!p.weight || (reinterpret_cast<uintptr_t>(p.weight) % (VEC * sizeof(TW))) == 0) &&
                    (!p.bias || (reinterpret_cast<uintptr_t>(p.bias) % (VEC * sizeof(TW))) == 0);
  return wide ? launch_vec<TX, TW, VEC>(p, s) : launch_vec<TX, TW, 1>(p, s);
}

}  // namespace

int layer_norm_parts(int64_t rows, int D) {
  // A block's partial row costs 8 D bytes each way, beside 6 or 12 D of each of its rows: enough blocks to fill the GPU
  // (one of up to 1,024 threads an SM for wide rows, four of up to 512 otherwise), and no more.
  return (int)std::min<int64_t>(rows, D > 4096 ? 148 : LN_MAX_PARTS);
}

cudaError_t launch_layer_norm(const LayerNormParams& p, kda_dtype x, kda_dtype w, cudaStream_t s) {
  if (x == KDA_F32) return launch_types<float, float>(p, s);
  return w == KDA_F32 ? launch_types<__nv_bfloat16, float>(p, s) : launch_types<__nv_bfloat16, __nv_bfloat16>(p, s);
}

}  // namespace kda
