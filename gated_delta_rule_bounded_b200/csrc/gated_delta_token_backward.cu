// gated_delta_token_backward.cu -- gradients of the gated delta rule with one decay per value head for fp32 inputs: what
// sums over value columns, chunk by chunk. The two recurrences before it are in gated_delta_token.cu, the notation in
// gated_delta_chunk.cuh and gated_delta_chunk_backward.cu:
//
//   W = tril(dO delta^T * D) diag(beta),  X = -diag(beta) strict(C delta^T * D) diag(beta)     (C: the rows k^T dS)
//   dQ = e^G dO S^T + W K
//   dK = -e^G beta C S^T + e^{G_C - G} beta delta dS^T + W^T Q + X K + X^T K
//   dbeta = rowdot(C, delta),  dV = beta C
//   dg as there, from a = rowdot(Q, e^G dO S^T) - rowdot(K, e^G beta C S^T), b = rowdot(K, e^{G_C - G} beta delta dS^T) and
//   P = W * Q K^T + X * K K^T
//
// One block a chunk and query head; the value heads that share it one after another, dQ and dK summed in registers. All
// products are fp32 on the CUDA cores, two values an instruction, 16 x 16 threads with 4 tokens each: 7.3 M products a unit
// of K = V = 128, 29,000 cycles of an SM at its rate, beside some 38,000 of shared memory's port, which bounds the kernel
// with the eight warps an SM holds. S and dS stream through a tile of 32 columns; everything else of the chunk stays in
// shared memory. Measured: 62 us a unit; 4096 tokens x 8 heads 322 us, beside 784 and 1,039 us of the two recurrences
// (190 and 250 ns a token); one product an instruction 351.
#include "gated_delta_chunk.cuh"

namespace kda {
namespace {

constexpr int TB_THREADS = 256, LD = 132, LW = 68, TILE_V = 32;  // rows padded: float4s of 8 rows meet no bank twice
struct TokenGradsSmem {
  float k[C][LD], q[C][LD], o[C][LD], c[C][LD], delta[C][LD];
  float w[C][LW], x[C][LW];
  float tile[TILE_V][LD];  // S^T or dS^T
  float vec[256], gh[C], gl[C], beta[C];
  float a[C], b[C], col[C], row[C], part[16][C];
  float dot[8];
};

// acc[r][2 j + e] (columns 64 j + 4 tx + 2 e and the next) += s[r] B[...], the row of B at `row`.
__device__ __forceinline__ void add_row(float2 (&acc)[4][4], const float (&s)[4], const float* row, int tx, bool wide) {
  const float4 u = *reinterpret_cast<const float4*>(row + 4 * tx);
  const float4 z = wide ? *reinterpret_cast<const float4*>(row + 64 + 4 * tx) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float2 f = make_float2(s[r], s[r]);
    acc[r][0] = fma2(f, make_float2(u.x, u.y), acc[r][0]);
    acc[r][1] = fma2(f, make_float2(u.z, u.w), acc[r][1]);
    acc[r][2] = fma2(f, make_float2(z.x, z.y), acc[r][2]);
    acc[r][3] = fma2(f, make_float2(z.z, z.w), acc[r][3]);
  }
}
// acc[r] += sum over n of A[t0 + r][n] B[n]; A row-major, n a multiple of 4.
__device__ __forceinline__ void product(float2 (&acc)[4][4], const float* A, int lda, const float* B, int ldb, int n, int tx, bool wide) {
  for (int i = 0; i < n; i += 4) {
    float4 f[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) f[r] = *reinterpret_cast<const float4*>(A + r * lda + i);
    add_row(acc, {f[0].x, f[1].x, f[2].x, f[3].x}, B + i * ldb, tx, wide);
    add_row(acc, {f[0].y, f[1].y, f[2].y, f[3].y}, B + (i + 1) * ldb, tx, wide);
    add_row(acc, {f[0].z, f[1].z, f[2].z, f[3].z}, B + (i + 2) * ldb, tx, wide);
    add_row(acc, {f[0].w, f[1].w, f[2].w, f[3].w}, B + (i + 3) * ldb, tx, wide);
  }
}
// As product, with A transposed: A[n][t0 + r].
__device__ __forceinline__ void product_t(float2 (&acc)[4][4], const float* A, int lda, const float* B, int ldb, int n, int tx, bool wide) {
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float4 f = *reinterpret_cast<const float4*>(A + i * lda);
    add_row(acc, {f.x, f.y, f.z, f.w}, B + i * ldb, tx, wide);
  }
}
// acc[r][j] = A[t0 + r] . B[tx + 16 j] over n elements (even and odd ones summed apart), for two As.
__device__ __forceinline__ void pairs(float (&acc)[4][4], float (&acc2)[4][4], const float* A, const float* A2, const float* B, int n, int tx) {
  float2 x[4][4], y[4][4];
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int j = 0; j < 4; ++j) x[r][j] = y[r][j] = make_float2(0.f, 0.f);
  for (int i = 0; i < n; i += 4) {
    float4 f[4], g[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      f[r] = *reinterpret_cast<const float4*>(A + r * LD + i);
      g[r] = *reinterpret_cast<const float4*>(A2 + r * LD + i);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 u = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * LD + i);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        x[r][j] = fma2(make_float2(f[r].z, f[r].w), make_float2(u.z, u.w), fma2(make_float2(f[r].x, f[r].y), make_float2(u.x, u.y), x[r][j]));
        y[r][j] = fma2(make_float2(g[r].z, g[r].w), make_float2(u.z, u.w), fma2(make_float2(g[r].x, g[r].y), make_float2(u.x, u.y), y[r][j]));
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      acc[r][j] = x[r][j].x + x[r][j].y;
      acc2[r][j] = y[r][j].x + y[r][j].y;
    }
}
__device__ __forceinline__ float sum16(float x) {  // over the 16 lanes that share a row
#pragma unroll
  for (int m = 8; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

__global__ void __launch_bounds__(TB_THREADS, 1)
    gated_delta_token_grads_kernel(GatedDeltaParams p, GatedDeltaGrads d, GatedDeltaTokenDump fwd, GatedDeltaTokenDump rev) {
  extern __shared__ __align__(16) unsigned char raw[];
  TokenGradsSmem& sm = *reinterpret_cast<TokenGradsSmem*>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tx = tid & 15, ty = tid >> 4, r0 = 4 * ty;
  const int h = blockIdx.x % p.H;
  const int64_t slot = blockIdx.x / p.H;
  int n;
  int64_t tc0, brow;
  const int nv = gd_slot_tokens(p, slot, n, tc0, brow);
  if (nv == 0) return;
  const int K = p.K, V = p.V, rep = p.HV / p.H;
  const bool wide = K > 64;
  // Of a short chunk only the tokens that are there: warps of 8 tokens, contractions over tokens in steps of 4.
  const bool work = 8 * warp < nv;
  const int nt = (nv + 3) & ~3;
  // Rows past the sequence's end, and columns past K or V, are zeros.
  auto rows = [&](float (*to)[LD], const float* from, int64_t stride, int width) {
    for (int e = tid; e < C * 32; e += TB_THREADS) {
      const int t = e >> 5, c = (e & 31) * 4;
      *reinterpret_cast<float4*>(&to[t][c]) =
          t < nv && c < width ? *reinterpret_cast<const float4*>(from + t * stride + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  rows(sm.k, static_cast<const float*>(p.k) + brow * p.ks[0] + tc0 * p.ks[1] + h * p.ks[2], p.ks[1], K);
  rows(sm.q, static_cast<const float*>(p.q) + brow * p.qs[0] + tc0 * p.qs[1] + h * p.qs[2], p.qs[1], K);
  __syncthreads();
  float qk[4][4], kk[4][4];
  float2 dq[4][4] = {}, dk[4][4] = {};
  if (work) pairs(qk, kk, sm.q[r0], sm.k[r0], sm.k[0], K, tx);

  for (int hv = h * rep; hv < (h + 1) * rep; ++hv) {
    const int64_t first = (brow * p.T + tc0) * p.HV + hv;  // this chunk's rows of delta and C, and of dV
    __syncthreads();  // the value head before is done with the buffers
    rows(sm.o, static_cast<const float*>(d.d_o) + brow * p.os[0] + tc0 * p.os[1] + hv * p.os[2], p.os[1], V);
    rows(sm.c, rev.rows + first * V, (int64_t)p.HV * V, V);
    rows(sm.delta, fwd.rows + first * V, (int64_t)p.HV * V, V);
    if (warp == 0) gd_decays(p, hv, tc0, brow, nv, lane, 0.f, sm.vec, sm.gh, sm.gl);
    if (tid >= 64 && tid < 64 + C)
      sm.beta[tid - 64] = tid - 64 < nv ? p.beta[brow * p.bs[0] + hv * p.bs[2] + (tc0 + tid - 64) * p.bs[1]] : 0.f;
    __syncthreads();
    {  // dbeta and dV: four threads a token
      const int t = tid >> 2;
      const float b = sm.beta[t];
      float x = 0.f;
      for (int c = (tid & 3) * 4; c < V; c += 16) {
        const float4 u = *reinterpret_cast<const float4*>(&sm.c[t][c]), z = *reinterpret_cast<const float4*>(&sm.delta[t][c]);
        x = fmaf(u.x, z.x, fmaf(u.y, z.y, fmaf(u.z, z.z, fmaf(u.w, z.w, x))));
        if (t < nv)
          *reinterpret_cast<float4*>(static_cast<float*>(d.dv) + (first + (int64_t)t * p.HV) * V + c) =
              make_float4(b * u.x, b * u.y, b * u.z, b * u.w);
      }
      x += __shfl_xor_sync(0xffffffffu, x, 1);
      x += __shfl_xor_sync(0xffffffffu, x, 2);
      if ((tid & 3) == 0 && t < nv) d.dbeta[first + (int64_t)t * p.HV] = x;
    }
    if (!work) {
#pragma unroll
      for (int j = 0; j < 4; ++j) sm.part[ty][tx + 16 * j] = 0.f;
    } else {  // W, X, and P's sums over rows and columns
      float w[4][4], x[4][4], col[4] = {0.f, 0.f, 0.f, 0.f};
      pairs(w, x, sm.o[r0], sm.c[r0], sm.delta[0], V, tx);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = r0 + r;
        float row = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = tx + 16 * j;
          const float decay = i <= t ? ex2((sm.gh[t] - sm.gh[i]) + (sm.gl[t] - sm.gl[i])) * sm.beta[i] : 0.f;
          w[r][j] = i <= t ? w[r][j] * decay : 0.f;
          x[r][j] = i < t ? -x[r][j] * (decay * sm.beta[t]) : 0.f;
          sm.w[t][i] = w[r][j];
          sm.x[t][i] = x[r][j];
          const float both = i < t ? fmaf(w[r][j], qk[r][j], x[r][j] * kk[r][j]) : 0.f;
          row += both;
          col[j] += both;
        }
        row = sum16(row);
        if (tx == 0) sm.row[t] = row;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) sm.part[ty][tx + 16 * j] = col[j];
    }
    const size_t at = ((size_t)slot * p.HV + hv) * (size_t)K * V;
    const float *S = fwd.states + at, *dS = rev.states + at;
    float dot = 0.f;  // <S, dS>
    auto tile = [&](const float* from, const float* with, int v0) {
      __syncthreads();
      for (int e = tid; e < TILE_V * 32; e += TB_THREADS) {
        const int v = e >> 5, c = (e & 31) * 4;
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (v0 + v < V && c < K) {
          f = *reinterpret_cast<const float4*>(from + (size_t)(v0 + v) * K + c);
          if (with) {
            const float4 u = *reinterpret_cast<const float4*>(with + (size_t)(v0 + v) * K + c);
            dot = fmaf(f.x, u.x, fmaf(f.y, u.y, fmaf(f.z, u.z, fmaf(f.w, u.w, dot))));
          }
        }
        *reinterpret_cast<float4*>(&sm.tile[v][c]) = f;
      }
      __syncthreads();
    };
    {  // dO S^T and C S^T
      float2 y[4][4] = {}, z[4][4] = {};
      for (int v0 = 0; v0 < V; v0 += TILE_V) {
        tile(S, nullptr, v0);
        if (!work) continue;
        product(y, &sm.o[r0][v0], LD, sm.tile[0], LD, min(TILE_V, V - v0), tx, wide);
        product(z, &sm.c[r0][v0], LD, sm.tile[0], LD, min(TILE_V, V - v0), tx, wide);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = r0 + r;
        const float e = sm.vec[VEC_E + t], eb = -e * sm.beta[t];
        float a = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = 64 * (j >> 1) + 4 * tx + 2 * (j & 1);
          y[r][j] = mul2(y[r][j], make_float2(e, e));
          z[r][j] = mul2(z[r][j], make_float2(eb, eb));
          dq[r][j] = add2(dq[r][j], y[r][j]);
          dk[r][j] = add2(dk[r][j], z[r][j]);
          const float2 qt = *reinterpret_cast<const float2*>(&sm.q[t][c]), kt = *reinterpret_cast<const float2*>(&sm.k[t][c]);
          if (c < K) a = fmaf(qt.x, y[r][j].x, fmaf(qt.y, y[r][j].y, fmaf(kt.x, z[r][j].x, fmaf(kt.y, z[r][j].y, a))));
        }
        a = sum16(a);
        if (tx == 0) sm.a[t] = a;
      }
    }
    {  // delta dS^T
      float2 y[4][4] = {};
      for (int v0 = 0; v0 < V; v0 += TILE_V) {
        tile(dS, S, v0);
        if (work) product(y, &sm.delta[r0][v0], LD, sm.tile[0], LD, min(TILE_V, V - v0), tx, wide);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = r0 + r;
        const float e = sm.vec[VEC_REST + t] * sm.beta[t];
        float b = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = 64 * (j >> 1) + 4 * tx + 2 * (j & 1);
          y[r][j] = mul2(y[r][j], make_float2(e, e));
          dk[r][j] = add2(dk[r][j], y[r][j]);
          const float2 kt = *reinterpret_cast<const float2*>(&sm.k[t][c]);
          if (c < K) b = fmaf(kt.x, y[r][j].x, fmaf(kt.y, y[r][j].y, b));
        }
        b = sum16(b);
        if (tx == 0) sm.b[t] = b;
      }
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m);
    if (lane == 0) sm.dot[warp] = dot;
    __syncthreads();
    if (warp == 0) {  // dg: what a step from a token to the next adds, summed in fp64; lane l holds tokens 2l and 2l + 1
      double z[2], base = 0.0;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = 2 * lane + e;
        double col = 0.0;
#pragma unroll
        for (int i = 0; i < 16; ++i) col += (double)sm.part[i][t];
        z[e] = t < nv ? (double)sm.b[t] - (double)sm.a[t] + col - (double)sm.row[t] : 0.0;
        base += t < nv ? (double)sm.a[t] : 0.0;
      }
#pragma unroll
      for (int m = 16; m >= 1; m >>= 1) base += __shfl_xor_sync(0xffffffffu, base, m);
      double all = 0.0;
#pragma unroll
      for (int i = 0; i < 8; ++i) all += (double)sm.dot[i];
      base += (double)sm.vec[VEC_ALL] * all;
      double sum = z[0] + z[1];
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, sum, m);
        if (lane >= m) sum += y;
      }
      const double before = base + sum - (z[0] + z[1]);
      if (2 * lane < nv) d.dg[first + (int64_t)(2 * lane) * p.HV] = (float)before;
      if (2 * lane + 1 < nv) d.dg[first + (int64_t)(2 * lane + 1) * p.HV] = (float)(before + z[0]);
    }
    if (work) {
      product(dq, sm.w[r0], LW, sm.k[0], LD, nt, tx, wide);
      product(dk, sm.x[r0], LW, sm.k[0], LD, nt, tx, wide);
      product_t(dk, &sm.x[0][r0], LW, sm.k[0], LD, nt, tx, wide);
      product_t(dk, &sm.w[0][r0], LW, sm.q[0], LD, nt, tx, wide);
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (r0 + r >= nv) break;
    const int64_t row = ((brow * p.T + tc0 + r0 + r) * p.H + h) * K;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = 64 * j + 4 * tx;
      if (c >= K) break;
      *reinterpret_cast<float4*>(static_cast<float*>(d.dq) + row + c) = make_float4(dq[r][2 * j].x, dq[r][2 * j].y, dq[r][2 * j + 1].x, dq[r][2 * j + 1].y);
      *reinterpret_cast<float4*>(static_cast<float*>(d.dk) + row + c) = make_float4(dk[r][2 * j].x, dk[r][2 * j].y, dk[r][2 * j + 1].x, dk[r][2 * j + 1].y);
    }
  }
}

}  // namespace

// Workspace: S and dS per chunk and value head, delta and C per token and value head.
size_t gated_delta_token_backward_bytes(int64_t B, int64_t T, int64_t H, int64_t HV, int64_t K, int64_t V, int64_t n_seq) {
  return 8 * ((size_t)gd_slots(B, T, n_seq) * HV * K * V + (size_t)B * T * HV * V);
}

cudaError_t launch_gated_delta_token_backward(const GatedDeltaParams& p, const GatedDeltaGrads& d, void* ws, cudaStream_t s) {
  static std::atomic<uint64_t> cfg{0};
  cudaError_t e = gd_smem_once(gated_delta_token_grads_kernel, (int)sizeof(TokenGradsSmem), cfg);
  if (e != cudaSuccess) return e;
  const int64_t slots = gd_slots(p.B, p.T, p.cu ? p.N : 0);
  if (slots * p.H > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const size_t states = (size_t)slots * p.HV * p.K * p.V, rows = (size_t)p.B * p.T * p.HV * p.V;
  float* at = static_cast<float*>(ws);
  const GatedDeltaTokenDump fwd{at, at + 2 * states}, rev{at + states, at + 2 * states + rows};
  e = launch_gated_delta_token_keep(p, fwd, s);
  if (e == cudaSuccess) e = launch_gated_delta_token_reverse(p, d, rev, s);
  if (e != cudaSuccess) return e;
  gated_delta_token_grads_kernel<<<(unsigned)(slots * p.H), TB_THREADS, sizeof(TokenGradsSmem), s>>>(p, d, fwd, rev);
  return cudaGetLastError();
}

}  // namespace kda
