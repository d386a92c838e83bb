// gated_delta_chunk_backward.cu -- gradients of the gated delta rule with one decay per value head, in chunks. Notation in
// gated_delta_chunk.cuh; dX is dL/dX, dS the gradient of the state after the chunk, S the state before it.
//
//   dU = A^T dO + e^{G_C - G} (K dS)        dR = beta dU + Z^T (beta dU) = dV        dbeta = rowdot(dR, delta) / beta
//   dS_before = e^{G_C} dS + Q^T (e^G dO) - K^T (e^G dR)
//   dQ = e^G dO S^T + (dO U^T * D) K
//   dK = -e^G dR S^T + e^{G_C - G} U dS^T + (dO U^T * D)^T Q + X K + X^T K,   X = -strict(dR U^T * D)
//   dg_t = e^{G_C} <S, dS> + sum_{s >= t} a_s + sum_{s < t} b_s + sum_{s >= t > i} P[s][i]
//     a_s = e^{G_s} (q_s . S dO_s - k_s . S dR_s),  b_s = e^{G_C - G_s} k_s . dS U_s,
//     P = (dO U^T * D) * Q K^T + X * K K^T
// The last line counts, for each token, exactly the terms whose decay passes it. (The shorter dg_t = <dS_T, S_T> + sum over
// the later tokens of o . dO - v . dV holds as well, but its terms cancel: with the same split operands its error is ten
// times as large.)
//
// Four kernels: the forward's P and S (S keeps every chunk's start state and deltas), the same recurrence backwards
// (kernel R), and one block per (chunk, query head) for the rest (kernel G). The chunk's matrices never leave the chip;
// what passes through memory is S, dS (two bf16 parts, the images the products read), delta and dR (fp32): 192 KB a chunk
// and head.
#include "gated_delta_chunk.cuh"

namespace kda {

__device__ int g_gated_delta_bwd_timeout = 0;

namespace {

// ---------------------------------------------------------------------------------------------------------------------
// Kernel R: the recurrence of dS, from the last chunk to the first. As kernel S (accumulator lane v, columns t or k):
//   X   (A^T dO)^T = dO^T A               dO^T from shared memory, A in two parts, 8 MMAs; needs no state
//   P1  (K dS)^T = dS^T K^T               16 MMAs
//   --  dU = X + e^{G_C - G} P1, beta dU in two parts
//   P2  Z^T (beta dU)                     12 MMAs
//   --  dR = beta dU + P2, -e^G dR in two parts
//   P3  Q^T (e^G dO) (8 MMAs, under P1's read-out) + K^T (-e^G dR) (8 MMAs)
//   --  dS = e^{G_C} dS + P3 in fp32 registers
// Bound by that chain, as kernel S is. Measured, 4096 tokens x 96 heads: 220 us, 3.4 us a chunk (319 with dR written
// straight from the accumulator's layout, 16 bytes every 128; four tokens of a column next to each other coalesce).
// ---------------------------------------------------------------------------------------------------------------------
constexpr int R_THREADS = 576, R_COMPUTE = 512;
constexpr int RT_K = 0, RT_Q = 16384, RT_DO = 32768, RT_B = 49152;
constexpr int RT_BYTES = RT_B + GB_SUMS;      // 82,944
constexpr int R_IMG = 2 * RT_BYTES;            // dS's images, 64 KB, on their way out
constexpr int R_BARS = R_IMG + 65536;
constexpr int R_SMEM = R_BARS + 128;
constexpr uint32_t T_SH = 0, T_SL = 64, T_SD = 128, T_KS = 256, T_DA = 320, T_W = 384, T_GO = 448;  // X stands in T_DA

struct RMaps {
  CUtensorMap q, k, d_o;
};

// The images of dS^T, as GatedDeltaDump::s, and dR fp32 [t / 4][v][t & 3], per (slot, value head).
struct RDump {
  unsigned char* ds;
  float* dr;
};

// ADVANCE: the segment that starts in a cell, from a gradient of zero (the sequence's own for its last segment) to the
// gradient at its start, nothing else kept.
template <bool ADVANCE>
__global__ void __launch_bounds__(R_THREADS, 1)
    gated_delta_reverse_kernel(GatedDeltaParams p, GatedDeltaGrads d, const unsigned char* blocks, RDump dump,
                               GatedDeltaSplit split, const __grid_constant__ RMaps maps) {
  extern __shared__ __align__(1024) unsigned char sm[];
  const uint32_t sb = smem_u32(sm);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hv = blockIdx.x % p.HV;
  const int64_t at = blockIdx.x / p.HV;
  const int length = split.length();
  GatedDeltaSegment g;
  if (ADVANCE ? !gd_cell(p, at, length, g) : !gd_segment(p, at, length, split.order, g)) return;
  const int64_t t0 = g.first, t1 = g.end, brow = g.brow;
  const int n_chunks = (int)((t1 - t0 + C - 1) / C);
  const int64_t slot0 = gd_slot_base(p, g.n, g.t0) + (int64_t)g.s * length;
  const uint32_t bars = sb + R_BARS;
  const uint32_t b_full = bars, b_a = bars + 16, b_x = bars + 24, b_b = bars + 32, b_c = bars + 40;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + R_BARS + 64);
  volatile int* dead = reinterpret_cast<volatile int*>(sm + R_BARS + 72);
  int* flag = &g_gated_delta_bwd_timeout;
  if (tid == 0) {
    for (int i = 0; i < 6; ++i) gd_bar_init(bars + 8 * i, 1);
    *dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 16) tm_alloc(smem_u32(tslot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;

  // Step c works on chunk n_chunks - 1 - c.
  if (warp == 17) {  // loads
    if (elect_one()) {
      const int h = hv / (p.HV / p.H);
      int c = 0;
      for (; c < n_chunks; ++c) {
        if (c >= 2) gd_wait(b_c, c & 1, dead, flag);  // step c - 2's products have read the stage
        if (*dead) break;
        const int ch = n_chunks - 1 - c;
        const uint32_t st = sb + (c & 1) * RT_BYTES, bar = b_full + 8 * (c & 1);
        const int tc = (int)(t0 + (int64_t)ch * C);
        gd_expect(bar, RT_BYTES);
        gd_bulk_load(st + RT_B, blocks + ((size_t)(slot0 + ch) * p.HV + hv) * GB_BYTES_BWD, GB_SUMS, bar);
        for (int half = 0; half < 2; ++half) {
          gd_tma_load(st + RT_DO + half * 8192, &maps.d_o, 64 * half, hv, tc, (int)brow, bar);
          gd_tma_load(st + RT_K + half * 8192, &maps.k, 64 * half, h, tc, (int)brow, bar);
          gd_tma_load(st + RT_Q + half * 8192, &maps.q, 64 * half, h, tc, (int)brow, bar);
        }
      }
      if (*dead)
        for (int i = max(0, c - 2); i < c; ++i) mbar_wait(b_full + 8 * (i & 1), (i >> 1) & 1, flag);
    }
    __syncwarp();
  } else if (warp == 16) {  // products, and the bulk store of dS's images
    constexpr uint32_t id64 = idesc_bf16(64, 0, 0), id128 = idesc_bf16(128, 0, 1);
    auto form_x = [&](uint32_t st) {
      constexpr uint32_t id_x = idesc_bf16(64, 1, 1);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)
        tc_mma(tmem + T_DA, sdesc(st + RT_DO + (ks & 3) * 2048, 8192, 1024),
               sdesc(st + RT_B + (ks < 4 ? GB_AH : GB_AL) + (ks & 3) * 2048, 8192, 1024), id_x, ks > 0);
    };
    for (int c = 0; c < n_chunks; ++c) {
      const uint32_t st = sb + (c & 1) * RT_BYTES;
      gd_wait(b_full + 8 * (c & 1), (c >> 1) & 1, dead, flag);
      // X needs no state and runs while dS is split. P2's accumulator, in whose place it stands, has been read (barrier 4 of
      // the step before). Only the first step's chunk, a sequence's last, may have rows to zero first.
      if (c > 0 && __all_sync(0xffffffffu, *dead == 0) && elect_one()) form_x(st);
      __syncwarp();
      named_sync<1, R_COMPUTE + 32>();  // dS's parts, and the stage in order
      tc_fence_after();
      if (__all_sync(0xffffffffu, *dead == 0) && elect_one()) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          tc_mma_ts(tmem + T_KS, tmem + T_SH + 8 * ks, sdesc(st + RT_K + (ks >> 2) * 8192 + (ks & 3) * 32, 16, 1024), id64, ks > 0);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          tc_mma_ts(tmem + T_KS, tmem + T_SL + 8 * ks, sdesc(st + RT_K + (ks >> 2) * 8192 + (ks & 3) * 32, 16, 1024), id64, 1);
        if (c == 0) form_x(st);
        tc_commit(b_a);
      }
      __syncwarp();
      named_sync<2, R_COMPUTE + 32>();  // e^G dO's parts, and dS's images
      tc_fence_after();
      if (!ADVANCE && lane == 0) {
        gd_bulk_store(dump.ds + ((size_t)(slot0 + n_chunks - 1 - c) * p.HV + hv) * 65536, sb + R_IMG, 65536);
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
      __syncwarp();
      if (__all_sync(0xffffffffu, *dead == 0) && elect_one()) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          tc_mma_ts(tmem + T_SD, tmem + T_GO + 16 * ks, sdesc(st + RT_Q + ks * 2048, 8192, 1024), id128, ks > 0);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          tc_mma_ts(tmem + T_SD, tmem + T_GO + 16 * ks + 8, sdesc(st + RT_Q + ks * 2048, 8192, 1024), id128, 1);
      }
      __syncwarp();
      named_sync<3, R_COMPUTE + 32>();  // beta dU's parts
      tc_fence_after();
      if (__all_sync(0xffffffffu, *dead == 0) && elect_one()) {
        // Z^T is strictly upper: of 16-token step ks, tokens before its end only; the last step covers them all.
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int ks = 3 - i;
          const uint32_t id = idesc_bf16(16 * ks + 16, 0, 1), at = st + RT_B + ks * 2048;
          tc_mma_ts(tmem + T_DA, tmem + T_KS + 16 * ks, sdesc(at + GB_ZH, 8192, 1024), id, i > 0);
          tc_mma_ts(tmem + T_DA, tmem + T_KS + 16 * ks, sdesc(at + GB_ZL, 8192, 1024), id, 1);
          tc_mma_ts(tmem + T_DA, tmem + T_KS + 16 * ks + 8, sdesc(at + GB_ZH, 8192, 1024), id, 1);
        }
        tc_commit(b_b);
      }
      __syncwarp();
      named_sync<4, R_COMPUTE + 32>();  // -e^G dR's parts
      tc_fence_after();
      if (__all_sync(0xffffffffu, *dead == 0) && elect_one()) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          tc_mma_ts(tmem + T_SD, tmem + T_W + 16 * ks, sdesc(st + RT_K + ks * 2048, 8192, 1024), id128, 1);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          tc_mma_ts(tmem + T_SD, tmem + T_W + 16 * ks + 8, sdesc(st + RT_K + ks * 2048, 8192, 1024), id128, 1);
      }
      __syncwarp();
      // The copy of dS's images has left: after this commit the passes may write over them.
      if (!ADVANCE && lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      __syncwarp();
      if (__all_sync(0xffffffffu, *dead == 0) && elect_one()) tc_commit(b_c);
      __syncwarp();
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    if (*dead && n_chunks > 0 && lane == 0) {
      mbar_wait(b_c, 0, flag);
      mbar_wait(b_c, 1, flag);
    }
  } else {  // the passes
    const int quad = warp & 3, part = warp >> 2, v = 32 * quad + lane;
    const uint32_t tl = tmem + ((uint32_t)(32 * quad) << 16);
    const bool there = v < p.V;
    const size_t hbase = ((size_t)g.n * p.HV + hv) * (size_t)p.K * p.V;
    const float* from = d.d_sf ? d.d_sf + hbase : nullptr;
    if (g.s + 1 < g.count)
      from = ADVANCE ? nullptr : split.x + ((size_t)(g.cell0 + g.s + 1) * p.HV + hv) * split.x_size;
    else if (!ADVANCE && g.count > 1 && d.d_sf && d.d_sf == d.ds0)  // the first segment writes over the given gradient
      from = split.m + ((size_t)(g.cell0 + 1) * p.HV + hv) * split.m_size;
    float2 S[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int k = 32 * part + 2 * j;
      const bool in = from && there && k < p.K;
      S[j].x = in ? from[(size_t)k * p.V + v] : 0.f;
      S[j].y = in ? from[(size_t)(k + 1) * p.V + v] : 0.f;
    }
    float all = 1.f;
    for (int c = 0; c < n_chunks; ++c) {
      const int ch = n_chunks - 1 - c;
      unsigned char* st = sm + (c & 1) * RT_BYTES;
      const float* vec = reinterpret_cast<const float*>(st + RT_B + GB_VEC);
      const float4* ve = reinterpret_cast<const float4*>(vec + VEC_E + 16 * part);
      const float4* vr = reinterpret_cast<const float4*>(vec + VEC_REST + 16 * part);
      const float4* vb = reinterpret_cast<const float4*>(vec + VEC_BETA + 16 * part);
      const int64_t tc = t0 + (int64_t)ch * C;
      const int nv = (int)min((int64_t)C, t1 - tc);
      const size_t item = (size_t)(slot0 + ch) * p.HV + hv;
      gd_wait(b_full + 8 * (c & 1), (c >> 1) & 1, dead, flag);
      if (nv < C) {  // rows past the sequence's end hold other tokens, or anything: zeros instead
        zero_rows(st + RT_K, 2, nv, tid, R_COMPUTE);
        zero_rows(st + RT_Q, 2, nv, tid, R_COMPUTE);
        zero_rows(st + RT_DO, 2, nv, tid, R_COMPUTE);
        fence_async_smem();
        named_sync<5, R_COMPUTE>();
      }
      uint32_t sh[16], sl[16];
      {
        if (c > 0) {
          gd_wait(b_c, (c - 1) & 1, dead, flag);
          tc_fence_after();
          uint32_t r[32];
          tm_ld32(tl + T_SD + 32 * part, r);
#pragma unroll
          for (int j = 0; j < 16; ++j) S[j] = fma2(make_float2(all, all), S[j], as_f2(r[2 * j], r[2 * j + 1]));
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) split2(S[j].x, S[j].y, sh[j], sl[j]);
        tm_st16(tl + T_SH + 16 * part, sh);
        tm_st16(tl + T_SL + 16 * part, sl);
        tm_wait_st();
      }
      all = vec[VEC_ALL];
      tc_fence_before();
      named_arrive<1, R_COMPUTE + 32>();
      // Under P1: dS's images, and e^G dO in two parts.
      {
        unsigned char* img = sm + R_IMG + (part >> 1) * 16384 + v * 128;
#pragma unroll
        for (int j = 0; j < (ADVANCE ? 0 : 4); ++j) {
          const int at = ((4 * (part & 1) + j) ^ (v & 7)) << 4;
          *reinterpret_cast<uint4*>(img + at) = make_uint4(sh[4 * j], sh[4 * j + 1], sh[4 * j + 2], sh[4 * j + 3]);
          *reinterpret_cast<uint4*>(img + 32768 + at) = make_uint4(sl[4 * j], sl[4 * j + 1], sl[4 * j + 2], sl[4 * j + 3]);
        }
        fence_async_smem();
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int t = 16 * part + 2 * j;
          const float2 e = *reinterpret_cast<const float2*>(vec + VEC_E + t);
          const float x = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(st + RT_DO + sw_e(t, v, 8192)));
          const float y = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(st + RT_DO + sw_e(t + 1, v, 8192)));
          split2(e.x * x, e.y * y, hi[j], lo[j]);
        }
        tm_st8(tl + T_GO + 16 * part, hi);
        tm_st8(tl + T_GO + 16 * part + 8, lo);
        tm_wait_st();
        tc_fence_before();
        named_arrive<2, R_COMPUTE + 32>();
      }
      float2 dR[8];
      gd_wait(b_a, c & 1, dead, flag);
      tc_fence_after();
      {
        uint32_t r[16], x[16], hi[8], lo[8];
        tm_ld16(tl + T_KS + 16 * part, r);
        tm_ld16(tl + T_DA + 16 * part, x);
        tm_wait_ld();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 w = vr[j], b = vb[j];
          const float2 u0 = fma2(make_float2(w.x, w.y), as_f2(r[4 * j], r[4 * j + 1]), as_f2(x[4 * j], x[4 * j + 1]));
          const float2 u1 = fma2(make_float2(w.z, w.w), as_f2(r[4 * j + 2], r[4 * j + 3]), as_f2(x[4 * j + 2], x[4 * j + 3]));
          dR[2 * j] = mul2(make_float2(b.x, b.y), u0);
          dR[2 * j + 1] = mul2(make_float2(b.z, b.w), u1);
          split2(dR[2 * j].x, dR[2 * j].y, hi[2 * j], lo[2 * j]);
          split2(dR[2 * j + 1].x, dR[2 * j + 1].y, hi[2 * j + 1], lo[2 * j + 1]);
        }
        tm_st8(tl + T_KS + 16 * part, hi);
        tm_st8(tl + T_KS + 16 * part + 8, lo);
        tm_wait_st();
      }
      tc_fence_before();
      named_arrive<3, R_COMPUTE + 32>();
      gd_wait(b_b, c & 1, dead, flag);
      tc_fence_after();
      {
        uint32_t r[16], hi[8], lo[8];
        tm_ld16(tl + T_DA + 16 * part, r);
        tm_wait_ld();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 e = ve[j];
          dR[2 * j] = add2(dR[2 * j], as_f2(r[4 * j], r[4 * j + 1]));
          dR[2 * j + 1] = add2(dR[2 * j + 1], as_f2(r[4 * j + 2], r[4 * j + 3]));
          const float2 w0 = mul2(make_float2(-e.x, -e.y), dR[2 * j]), w1 = mul2(make_float2(-e.z, -e.w), dR[2 * j + 1]);
          split2(w0.x, w0.y, hi[2 * j], lo[2 * j]);
          split2(w1.x, w1.y, hi[2 * j + 1], lo[2 * j + 1]);
        }
        tm_st8(tl + T_W + 16 * part, hi);
        tm_st8(tl + T_W + 16 * part + 8, lo);
        tm_wait_st();
      }
      tc_fence_before();
      named_arrive<4, R_COMPUTE + 32>();
      // Under P3: dR for kernel G, four tokens of a column next to each other.
      float* rp = dump.dr + item * 8192 + (4 * part) * (4 * VT) + 4 * v;
#pragma unroll
      for (int j = 0; j < (ADVANCE ? 0 : 4); ++j)
        *reinterpret_cast<float4*>(rp + j * (4 * VT)) = make_float4(dR[2 * j].x, dR[2 * j].y, dR[2 * j + 1].x, dR[2 * j + 1].y);
    }
    if (n_chunks > 0) {
      gd_wait(b_c, (n_chunks - 1) & 1, dead, flag);
      tc_fence_after();
      uint32_t r[32];
      tm_ld32(tl + T_SD + 32 * part, r);
#pragma unroll
      for (int j = 0; j < 16; ++j) S[j] = fma2(make_float2(all, all), S[j], as_f2(r[2 * j], r[2 * j + 1]));
    }
    float* to = ADVANCE ? split.x + ((size_t)at * p.HV + hv) * split.x_size : d.ds0 && g.s == 0 ? d.ds0 + hbase : nullptr;
    if (to && there) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int k = 32 * part + 2 * j;
        if (k < p.K) {
          to[(size_t)k * p.V + v] = S[j].x;
          to[(size_t)(k + 1) * p.V + v] = S[j].y;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 16) tm_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------------------------------------------------
// Kernel G: dQ, dK, dbeta and dg of one chunk and query head; the value heads that share it one after another, dQ and dK
// summed in tensor memory (a fixed order, no atomics). Products with M = 128 lanes, in two groups:
//   lanes i (token):  dO delta^T and dR delta^T, with delta's two parts as the two halves of the lanes; K Q^T and K K^T
//   lanes k:          S dO, S dR, dS delta; K^T (dO U^T * D)^T, Q^T (dO U^T * D), K^T X^T, K^T X
// U = beta delta enters as delta, with beta on the accumulators. Every sum takes operands in two parts, those of dQ and dK
// too: they are to carry their own rounding to bf16 and no other of that size.
//
// A unit (chunk, value head) reads 240 KB: S and dS 64 KB each, delta and dR 32 KB each, K, Q and dO. That is what bounds
// the kernel in the end; one block fills an SM's shared memory, so blocks are persistent, a warp of its own loads, in the
// order in which the unit before releases its buffers (dS follows S through one buffer), another issues the products, and
// 16 warps do the passes. Measured, 4096 tokens x 96 heads (6,144 units, 1.8 GB): 441 us, 4.0 TB/s; some 18,700 cycles a
// unit, of which the passes issue 9,700 and shared memory's port takes 14,800; 96 value heads over 48: 467 us. With the D
// products' high parts alone 426 and 440 us, dQ and dK off by 1.4 times as much. One unit after another on 256 threads: 733 us.
// ---------------------------------------------------------------------------------------------------------------------
constexpr int G_THREADS = 576, G_COMPUTE = 512;
constexpr int G_S = 0;               // 64 KB: S's images, then dS's
constexpr int G_KQ = 65536;          // 32 KB: [64-channel half][K 64 rows ; Q 64 rows][128 B]
constexpr int G_DO = 98304;          // 16 KB
constexpr int G_D = 114688;          // 32 KB: delta^T [v][t] bf16, high then low
constexpr int G_DR = 147456;         // 32 KB: dR fp32 [t / 4][v][t & 3], then dR^T [v][t] bf16, high then low
constexpr int G_I = 180224;          // 16 KB: dV's tile [t][v]; an exchange buffer; (dO U^T * D)^T and X^T as [i][t] bf16,
                                     // high parts; dQ's tile [t][k]
constexpr int G_XB = 196608;         // 16 KB: the other exchange buffer, the low parts of those, then dK's tile
constexpr int G_VEC = 212992;        // 1.5 KB: the block's vectors and its sums of log2 decays
constexpr int G_F = G_VEC + 1536;    // partial sums, floats
constexpr int GF_X = 0, GF_COL = 256, GF_BETA = 768, GF_Z = 1024, GF_A = 1040;
constexpr int G_BARS = G_F + 1056 * 4;
constexpr int G_SMEM = G_BARS + 128;
// Tensor memory. ONE: what takes a split B operand has two accumulators next to each other, one for each part (N = 128: A is
// read once for both); DQ and DK stand in place of the first group, E3 in place of the inner products. With value heads that
// share a query head both parts go to one accumulator, which leaves DQ and DK columns of their own: they carry the sums from
// one value head to the next (in registers the sums spilled and a unit took 14.1 us instead of 10.5).
template <bool ONE>
struct GColumns {
  static constexpr uint32_t E1 = 0, E2 = 64, G1 = ONE ? 192 : 128, G2 = ONE ? 256 : 192, QK = ONE ? 384 : 256, KK = ONE ? 448 : 320;
  static constexpr uint32_t DQ = ONE ? 192 : 384, DK = ONE ? 256 : 448, E3 = ONE ? 384 : 256;
};

struct GMaps {
  CUtensorMap q, k, d_o, dq, dk, dv;
};

// Lane l gets the sum over the warp of element l & 15.
__device__ __forceinline__ float sum_columns(float (&v)[16], int lane) {
#pragma unroll
  for (int w = 8; w >= 1; w >>= 1) {
    const bool up = (lane & w) != 0;
#pragma unroll
    for (int j = 0; j < w; ++j) {
      const float send = up ? v[j] : v[j + w];
      const float recv = __shfl_xor_sync(0xffffffffu, send, w);
      v[j] = (up ? v[j + w] : v[j]) + recv;
    }
  }
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Walks a block's units: (chunk slot, query head) items blockIdx.x, + gridDim.x, ... that hold tokens, and for each the
// value heads that share the query head.
struct GUnits {
  int item, r, h, slot, nv, tc0, brow;  // few: they stay in registers through the whole unit
  __device__ __forceinline__ GUnits(const GatedDeltaParams& p, int items) : item(blockIdx.x), r(0), nv(0) { find(p, items); }
  __device__ __forceinline__ void find(const GatedDeltaParams& p, int items) {
    for (; item < items; item += gridDim.x) {
      int n;
      int64_t t, b;
      h = item % p.H;
      slot = item / p.H;
      nv = gd_slot_tokens(p, slot, n, t, b);
      tc0 = (int)t;
      brow = (int)b;
      if (nv > 0) break;
    }
  }
  __device__ __forceinline__ bool more(int items) const { return item < items; }
  __device__ __forceinline__ int hv(int rep) const { return h * rep + r; }
  __device__ __forceinline__ void next(const GatedDeltaParams& p, int items, int rep) {
    if (++r < rep) return;
    r = 0;
    item += gridDim.x;
    find(p, items);
  }
};

// ONE: no value heads share a query head, so nothing is carried from unit to unit.
template <bool ONE>
__global__ void __launch_bounds__(G_THREADS, 1)
    gated_delta_grads_kernel(GatedDeltaParams p, GatedDeltaGrads d, const unsigned char* blocks, GatedDeltaDump fwd, RDump rev,
                             int items, int rep, const __grid_constant__ GMaps maps) {
  using TG = GColumns<ONE>;
  extern __shared__ __align__(1024) unsigned char sm[];
  const uint32_t sb = smem_u32(sm);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float* F = reinterpret_cast<float*>(sm + G_F);
  const float* vec = reinterpret_cast<const float*>(sm + G_VEC);
  const float* gh = vec + 256;
  const float* gl = vec + 320;
  const uint32_t bars = sb + G_BARS;
  // Loads: dR, dO, S, delta, K and Q with the vectors, dS. Products: first group, second, third. Passes: S read, dS read,
  // the unit's accumulators and operands read.
  const uint32_t f_r = bars, f_o = bars + 8, f_s = bars + 16, f_d = bars + 24, f_kq = bars + 32, f_ds = bars + 40;
  const uint32_t m1 = bars + 48, m2 = bars + 56, m3 = bars + 64, z1 = bars + 72, z2 = bars + 80, s2 = bars + 88;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + G_BARS + 96);
  volatile int* dead = reinterpret_cast<volatile int*>(sm + G_BARS + 104);
  int* flag = &g_gated_delta_bwd_timeout;
  if (tid == 0) {
    for (int i = 0; i < 9; ++i) gd_bar_init(bars + 8 * i, 1);
    for (int i = 9; i < 12; ++i) gd_bar_init(bars + 8 * i, 16);
    *dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 16) tm_alloc(smem_u32(tslot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;

  if (warp == 17) {  // loads
    if (elect_one()) {
      auto load_ro = [&](const GUnits& u) {
        const size_t at = (size_t)u.slot * p.HV + u.hv(rep);
        gd_expect(f_r, 32768);
        gd_bulk_load(sb + G_DR, rev.dr + at * 8192, 32768, f_r);
        gd_expect(f_o, 16384);
        for (int i = 0; i < 2; ++i) gd_tma_load(sb + G_DO + i * 8192, &maps.d_o, 64 * i, u.hv(rep), u.tc0, u.brow, f_o);
      };
      auto load_sd = [&](const GUnits& u) {
        const size_t at = (size_t)u.slot * p.HV + u.hv(rep);
        gd_expect(f_s, 65536);
        gd_bulk_load(sb + G_S, fwd.s + at * 65536, 65536, f_s);
        gd_expect(f_d, 32768);
        gd_bulk_load(sb + G_D, fwd.delta + at * 32768, 32768, f_d);
      };
      auto load_kq = [&](const GUnits& u) {
        const size_t at = (size_t)u.slot * p.HV + u.hv(rep);
        gd_expect(f_kq, 32768 + 1536);
        for (int i = 0; i < 2; ++i) {
          gd_tma_load(sb + G_KQ + i * 16384, &maps.k, 64 * i, u.h, u.tc0, u.brow, f_kq);
          gd_tma_load(sb + G_KQ + i * 16384 + 8192, &maps.q, 64 * i, u.h, u.tc0, u.brow, f_kq);
        }
        const unsigned char* blk = blocks + at * GB_BYTES_BWD;
        gd_bulk_load(sb + G_VEC, blk + GB_VEC, 1024, f_kq);
        gd_bulk_load(sb + G_VEC + 1024, blk + GB_SUMS, 512, f_kq);
      };
      GUnits u(p, items);
      uint32_t par = 0;
      bool ds = false;
      if (u.more(items)) {
        load_ro(u);
        load_kq(u);
        load_sd(u);
      }
      while (u.more(items) && !*dead) {
        const size_t at = (size_t)u.slot * p.HV + u.hv(rep);
        gd_wait(m2, par, dead, flag);
        gd_wait(z1, par, dead, flag);
        if (*dead) break;
        gd_expect(f_ds, 65536);
        gd_bulk_load(sb + G_S, rev.ds + at * 65536, 65536, f_ds);
        ds = true;
        u.next(p, items, rep);
        if (!u.more(items)) break;
        load_ro(u);
        gd_wait(m3, par, dead, flag);
        gd_wait(z2, par, dead, flag);
        if (*dead) break;
        load_sd(u);
        gd_wait(s2, par, dead, flag);
        if (*dead) break;
        load_kq(u);
        par ^= 1;
      }
      if (*dead)  // give the loads that may still be in flight a bounded wait
        for (int i = 0; i < (ds ? 6 : 5); ++i) {
          mbar_wait(bars + 8 * i, 0, flag);
          mbar_wait(bars + 8 * i, 1, flag);
        }
    }
    __syncwarp();
  } else if (warp == 16) {  // products
    uint32_t par = 0;
    for (GUnits u(p, items); u.more(items); u.next(p, items, rep), par ^= 1) {
      gd_wait(f_o, par, dead, flag);
      gd_wait(f_kq, par, dead, flag);
      gd_wait(f_d, par, dead, flag);
      named_sync<1, G_COMPUTE + 32>();  // dR's images; rows past the end zeroed; the unit before has read its accumulators
      tc_fence_after();
      if (__all_sync(0xffffffffu, *dead == 0) && elect_one()) {
        constexpr uint32_t id_g1 = idesc_bf16(64, 1, 0), id_g2 = idesc_bf16(ONE ? 128 : 64, 1, 1), id_kk = idesc_bf16(64, 0, 0);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const uint64_t u_ = sdesc(sb + G_D + ks * 2048, 16384, 1024);
          tc_mma(tmem + TG::G1, u_, sdesc(sb + G_DO + (ks >> 2) * 8192 + (ks & 3) * 32, 16, 1024), id_g1, ks > 0);
          tc_mma(tmem + TG::G2, u_, sdesc(sb + G_DR + ks * 2048, 16384, 1024), id_g2, ks > 0);
          if (!ONE) tc_mma(tmem + TG::G2, u_, sdesc(sb + G_DR + 16384 + ks * 2048, 16384, 1024), id_g2, 1);
        }
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const uint32_t at = sb + G_KQ + (ks >> 2) * 16384 + (ks & 3) * 32;
          tc_mma(tmem + TG::QK, sdesc(at, 16, 1024), sdesc(at + 8192, 16, 1024), id_kk, ks > 0);
          // K as lanes 64-127: the 64 rows before it are some other operand's, and so are lanes 0-63.
          tc_mma(tmem + TG::KK, sdesc(at - 8192, 16, 1024), sdesc(at, 16, 1024), id_kk, ks > 0);
        }
        tc_commit(m1);
      }
      __syncwarp();
      gd_wait(f_s, par, dead, flag);
      if (__all_sync(0xffffffffu, *dead == 0) && elect_one()) {
        constexpr uint32_t id_e1 = idesc_bf16(64, 1, 0), id_e2 = idesc_bf16(64, 1, 1), id_g2 = idesc_bf16(ONE ? 128 : 64, 1, 1);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const uint64_t s_h = sdesc(sb + G_S + ks * 2048, 16384, 1024), s_l = sdesc(sb + G_S + 32768 + ks * 2048, 16384, 1024);
          const uint64_t o = sdesc(sb + G_DO + (ks >> 2) * 8192 + (ks & 3) * 32, 16, 1024);
          const uint64_t r = sdesc(sb + G_DR + ks * 2048, 16384, 1024);
          tc_mma(tmem + TG::E1, s_h, o, id_e1, ks > 0);
          tc_mma(tmem + TG::E1, s_l, o, id_e1, 1);
          tc_mma(tmem + TG::E2, s_h, r, id_g2, ks > 0);
          if (!ONE) tc_mma(tmem + TG::E2, s_h, sdesc(sb + G_DR + 16384 + ks * 2048, 16384, 1024), id_e2, 1);
          tc_mma(tmem + TG::E2, s_l, r, id_e2, 1);
        }
        tc_commit(m2);
      }
      __syncwarp();
      named_sync<2, G_COMPUTE + 32>();  // the images of dO U^T * D and X; the first group's accumulators are read
      tc_fence_after();
      if (__all_sync(0xffffffffu, *dead == 0) && elect_one()) {
        constexpr uint32_t id_tt = idesc_bf16(64, 1, 1), id_tn = idesc_bf16(64, 1, 0);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const uint64_t kt = sdesc(sb + G_KQ + ks * 2048, 16384, 1024), qt = sdesc(sb + G_KQ + 8192 + ks * 2048, 16384, 1024);
#pragma unroll
          for (int lo = 0; lo < 2; ++lo) {
            const uint32_t img = sb + (lo ? G_XB : G_I), more = lo || ks > 0 || (!ONE && u.r);
            tc_mma(tmem + TG::DQ, kt, sdesc(img + ks * 2048, 8192, 1024), id_tt, more);
            tc_mma(tmem + TG::DK, qt, sdesc(img + ks * 32, 16, 1024), id_tn, more);
            tc_mma(tmem + TG::DK, kt, sdesc(img + 8192 + ks * 2048, 8192, 1024), id_tt, 1);
            tc_mma(tmem + TG::DK, kt, sdesc(img + 8192 + ks * 32, 16, 1024), id_tn, 1);
          }
        }
      }
      __syncwarp();
      gd_wait(f_ds, par, dead, flag);
      if (__all_sync(0xffffffffu, *dead == 0) && elect_one()) {
        constexpr uint32_t id_e = idesc_bf16(64, 1, 1), id_ee = idesc_bf16(ONE ? 128 : 64, 1, 1);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const uint64_t u_ = sdesc(sb + G_D + ks * 2048, 16384, 1024);
          tc_mma(tmem + TG::E3, sdesc(sb + G_S + ks * 2048, 16384, 1024), u_, id_ee, ks > 0);
          if (!ONE) tc_mma(tmem + TG::E3, sdesc(sb + G_S + ks * 2048, 16384, 1024), sdesc(sb + G_D + 16384 + ks * 2048, 16384, 1024), id_e, 1);
          tc_mma(tmem + TG::E3, sdesc(sb + G_S + 32768 + ks * 2048, 16384, 1024), u_, id_e, 1);
        }
        tc_commit(m3);
      }
      __syncwarp();
    }
    if (*dead && lane == 0)
      for (int i = 6; i < 9; ++i) {
        mbar_wait(bars + 8 * i, 0, flag);
        mbar_wait(bars + 8 * i, 1, flag);
      }
    __syncwarp();
  } else {  // the passes
    const int quad = warp & 3, part = warp >> 2;
    const uint32_t tl = tmem + ((uint32_t)(32 * quad) << 16);
    const int t0 = 16 * part;  // this thread's 16 tokens, as columns
    uint32_t par = 0;
    for (GUnits u(p, items); u.more(items); u.next(p, items, rep), par ^= 1) {
      const int nv = u.nv;
      {  // dR to two bf16 parts, in place, and dbeta's sums; v = 32 quad + lane
        const int v = 32 * quad + lane;
        if (tid == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the unit before's dQ and dK tiles
        gd_wait(f_r, par, dead, flag);
        float x[16];
        const float4* dr = reinterpret_cast<const float4*>(sm + G_DR) + (4 * part) * VT + v;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 y = dr[j * VT];
          x[4 * j] = y.x;
          x[4 * j + 1] = y.y;
          x[4 * j + 2] = y.z;
          x[4 * j + 3] = y.w;
        }
        named_sync<3, G_COMPUTE>();
        if (nv == C) {  // dV is dR, rounded
          __nv_bfloat16* a = reinterpret_cast<__nv_bfloat16*>(sm + G_I) + t0 * VT + v;
#pragma unroll
          for (int j = 0; j < 16; ++j) a[j * VT] = __float2bfloat16_rn(x[j]);
        } else if (v < p.V) {
          const int64_t row = (int64_t)p.HV * p.V;
          __nv_bfloat16* a = static_cast<__nv_bfloat16*>(d.dv) + ((int64_t)u.brow * p.T + u.tc0 + t0) * row + (int64_t)u.hv(rep) * p.V + v;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (t0 + j < nv) a[j * row] = __float2bfloat16_rn(x[j]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split2(x[8 * j + 2 * e], x[8 * j + 2 * e + 1], hi[e], lo[e]);
          const uint32_t at = sw_chunk(v, 2 * part + j, 0);
          *reinterpret_cast<uint4*>(sm + G_DR + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(sm + G_DR + 16384 + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        if (nv < C) {  // rows past the sequence's end hold other tokens, or anything: zeros instead
          gd_wait(f_o, par, dead, flag);
          gd_wait(f_kq, par, dead, flag);
          for (int e = tid; e < (64 - nv) * 32; e += G_COMPUTE) {  // K's and Q's rows in both halves
            const int row = nv + (e >> 5), c = e & 31;
            *reinterpret_cast<uint4*>(sm + G_KQ + (c >> 4) * 16384 + ((c >> 3) & 1) * 8192 + row * 128 + (c & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          zero_rows(sm + G_DO, 2, nv, tid, G_COMPUTE);
        }
        fence_async_smem();
        tc_fence_before();
        named_arrive<1, G_COMPUTE + 32>();
        named_sync<3, G_COMPUTE>();
        if (tid == 0 && nv == C) {
          gd_tma_store(&maps.dv, sb + G_I, 0, u.hv(rep), u.tc0, u.brow);
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
        gd_wait(f_d, par, dead, flag);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t at = sw_chunk(v, 2 * part + j, 0);
          const uint4 a = *reinterpret_cast<const uint4*>(sm + G_D + at), b = *reinterpret_cast<const uint4*>(sm + G_D + 16384 + at);
          const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 y = add2(unpack_bf16(aw[e]), unpack_bf16(bw[e]));
            x[8 * j + 2 * e] *= y.x;
            x[8 * j + 2 * e + 1] *= y.y;
          }
        }
        const float sum = sum_columns(x, lane);
        if (lane < 16) F[GF_BETA + 64 * quad + t0 + lane] = sum;
      }
      uint4 zs[8];  // S's two parts, for <S, dS>: dS takes its place
      gd_wait(f_s, par, dead, flag);
#pragma unroll
      for (int i4 = 0; i4 < 8; ++i4)
        zs[i4] = *reinterpret_cast<const uint4*>(sm + G_S + (i4 >> 2) * 32768 + (tid + (i4 & 3) * G_COMPUTE) * 16);
      __syncwarp();
      if (lane == 0) mbar_arrive(z1);
      if (tid == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // dV's tile gives way to the exchange
      named_sync<3, G_COMPUTE>();
      gd_wait(f_kq, par, dead, flag);
      const bool tiny = vec[VEC_TINY] != 0.f;
      if (tiny && tid == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // dV's tile has arrived
      gd_wait(m1, par, dead, flag);
      tc_fence_after();
      float* xa = reinterpret_cast<float*>(sm + G_I);
      float* xb = reinterpret_cast<float*>(sm + G_XB);
      const int i = (32 * quad + lane) & 63;  // quads 0, 1: dO delta^T; quads 2, 3: dR delta^T
      if (quad < 2) {  // delta's high part: hand over dR delta^T
        uint32_t a[16], b[16];
        tm_ld16(tl + TG::G2 + t0, a);
        if (ONE) tm_ld16(tl + TG::G2 + 64 + t0, b);
        tm_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j) xb[(t0 + j) * 64 + i] = ONE ? __uint_as_float(a[j]) + __uint_as_float(b[j]) : __uint_as_float(a[j]);
      } else {  // its low part: hand over dO delta^T
        uint32_t a[16];
        tm_ld16(tl + TG::G1 + t0, a);
        tm_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j) xa[(t0 + j) * 64 + i] = __uint_as_float(a[j]);
      }
      named_sync<3, G_COMPUTE>();
      if (tiny && 32 * quad + lane < p.V)  // the gradient of a v that is written with strength zero
#pragma unroll 1
        for (int t = t0; t < min(t0 + 16, nv); ++t)
          if (fabsf(vec[VEC_BETA + t]) <= GD_TINY)
            static_cast<__nv_bfloat16*>(d.dv)[(((int64_t)u.brow * p.T + u.tc0 + t) * p.HV + u.hv(rep)) * p.V + 32 * quad + lane] =
                __float2bfloat16_rn(0.f);
      float X[16];     // this thread's share of x_t = dg_{t+1} - dg_t at its 16 tokens
      uint32_t pk[8], pl[8];  // its row of the images, two parts
      {
        const float* other = (quad < 2 ? xa : xb) + t0 * 64 + i;
        const float ghi = gh[i], glo = gl[i], b = quad < 2 ? vec[VEC_BETA + i] : -vec[VEC_BETA + i];
        const uint32_t t_own = tl + t0 + (quad < 2 ? TG::G1 : TG::G2), t_in = tl + t0 + (quad < 2 ? TG::QK : TG::KK);
        float col = 0.f;
#pragma unroll
        for (int p8 = 0; p8 < 16; p8 += 8) {
          uint32_t own[8], inner[8];  // inner: k_i . q_t, or k_i . k_t
          tm_ld8(t_own + p8, own);
          if (ONE && quad >= 2) {
            tm_ld8(t_own + 64 + p8, inner);
            tm_wait_ld();
#pragma unroll
            for (int j = 0; j < 8; ++j) own[j] = __float_as_uint(__uint_as_float(own[j]) + __uint_as_float(inner[j]));
          }
          tm_ld8(t_in + p8, inner);
          tm_wait_ld();
#pragma unroll
          for (int j = 0; j < 8; j += 4) {
            const float4 g4 = *reinterpret_cast<const float4*>(gh + t0 + p8 + j), l4 = *reinterpret_cast<const float4*>(gl + t0 + p8 + j);
            const float gt[4] = {g4.x, g4.y, g4.z, g4.w}, lt[4] = {l4.x, l4.y, l4.z, l4.w};
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int t = t0 + p8 + j + e;
              float x = __uint_as_float(own[j + e]) + other[(p8 + j + e) * 64];
              const float dec = b * ex2((gt[e] - ghi) + (lt[e] - glo));
              const bool keep = t < nv && (quad < 2 ? i <= t : i < t);
              y[e] = keep ? x * dec : 0.f;
              const float P = keep && i < t ? y[e] * __uint_as_float(inner[j + e]) : 0.f;
              X[p8 + j + e] = -P;
              col += P;
            }
            split2(y[0], y[1], pk[(p8 + j) >> 1], pl[(p8 + j) >> 1]);
            split2(y[2], y[3], pk[((p8 + j) >> 1) + 1], pl[((p8 + j) >> 1) + 1]);
          }
        }
        F[GF_COL + 64 * (4 * (quad >> 1) + part) + i] = col;
      }
      tc_fence_before();
      named_sync<3, G_COMPUTE>();  // the exchange buffers are read
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t at = (quad < 2 ? 0 : 8192) + sw_chunk(i, 2 * part + j, 0);
        *reinterpret_cast<uint4*>(sm + G_I + at) = make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
        *reinterpret_cast<uint4*>(sm + G_XB + at) = make_uint4(pl[4 * j], pl[4 * j + 1], pl[4 * j + 2], pl[4 * j + 3]);
      }
      fence_async_smem();
      named_arrive<2, G_COMPUTE + 32>();
      {  // <S, dS>
        gd_wait(f_ds, par, dead, flag);
        float z = 0.f;
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4) {
          const int at = (tid + i4 * G_COMPUTE) * 16;
          const uint4 x = *reinterpret_cast<const uint4*>(sm + G_S + at), y = *reinterpret_cast<const uint4*>(sm + G_S + 32768 + at);
          const uint4 a = zs[i4], b = zs[4 + i4];
          const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w}, xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 s = add2(unpack_bf16(aw[e]), unpack_bf16(bw[e])), g = add2(unpack_bf16(xw[e]), unpack_bf16(yw[e]));
            z = fmaf(s.x, g.x, z);
            z = fmaf(s.y, g.y, z);
          }
        }
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) z += __shfl_xor_sync(0xffffffffu, z, m);
        if (lane == 0) {
          F[GF_Z + warp] = z;
          mbar_arrive(z2);
        }
      }
      gd_wait(m3, par, dead, flag);
      tc_fence_after();
      {  // lane k; eight tokens at a time, so that nothing has to leave the registers
        const int k = 32 * quad + lane;
        const unsigned char* kq = sm + G_KQ + (k >> 6) * 16384 + 2 * (k & 7);
        const int kc = (k & 63) >> 3;
        const bool last = ONE || u.r == rep - 1;
        __nv_bfloat16* a = reinterpret_cast<__nv_bfloat16*>(sm + G_I) + t0 * VT + k;  // the tiles [t][k], over the images
        __nv_bfloat16* b = reinterpret_cast<__nv_bfloat16*>(sm + G_XB) + t0 * VT + k;
        const int64_t row = (int64_t)p.H * p.K, at = ((int64_t)u.brow * p.T + u.tc0 + t0) * row + (int64_t)u.h * p.K + k;
        float suma = 0.f;
#pragma unroll
        for (int part8 = 0; part8 < 16; part8 += 8) {
          const int tt = t0 + part8;
          float e[8], q8[8], k8[8];
#pragma unroll
          for (int j = 0; j < 8; j += 4) {
            const float4 w = *reinterpret_cast<const float4*>(vec + VEC_E + tt + j);
            e[j] = w.x;
            e[j + 1] = w.y;
            e[j + 2] = w.z;
            e[j + 3] = w.w;
          }
          uint32_t x[8], y[8];
          tm_ld8(tl + TG::E1 + tt, x);
          tm_ld8(tl + TG::DQ + tt, y);
          tm_wait_ld();
          // Token tt + j is row tt + j of the swizzled tile, and tt is a multiple of 8.
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float w = e[j] * __uint_as_float(x[j]);
            const float s = w * __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(kq + 8192 + (tt + j) * 128 + ((kc ^ j) << 4)));
            q8[j] = w + __uint_as_float(y[j]);
            suma += s;
            X[part8 + j] -= s;
          }
          uint32_t kk[8];
          tm_ld8(tl + TG::E2 + tt, x);
          if (ONE) tm_ld8(tl + TG::E2 + 64 + tt, y);
          tm_wait_ld();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            kk[j] = (uint32_t)*reinterpret_cast<const uint16_t*>(kq + (tt + j) * 128 + ((kc ^ j) << 4)) << 16;
            k8[j] = -e[j] * (ONE ? __uint_as_float(x[j]) + __uint_as_float(y[j]) : __uint_as_float(x[j]));
            const float s = k8[j] * __uint_as_float(kk[j]);
            suma += s;
            X[part8 + j] -= s;
          }
#pragma unroll
          for (int j = 0; j < 8; j += 4) {
            const float4 w = *reinterpret_cast<const float4*>(vec + VEC_REST + tt + j), v = *reinterpret_cast<const float4*>(vec + VEC_BETA + tt + j);
            e[j] = w.x * v.x;
            e[j + 1] = w.y * v.y;
            e[j + 2] = w.z * v.z;
            e[j + 3] = w.w * v.w;
          }
          tm_ld8(tl + TG::E3 + tt, x);
          if (ONE) tm_ld8(tl + TG::E3 + 64 + tt, y);
          tm_wait_ld();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float w = e[j] * (ONE ? __uint_as_float(x[j]) + __uint_as_float(y[j]) : __uint_as_float(x[j]));
            k8[j] += w;
            X[part8 + j] = fmaf(w, __uint_as_float(kk[j]), X[part8 + j]);
          }
          tm_ld8(tl + TG::DK + tt, x);
          tm_wait_ld();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            k8[j] += __uint_as_float(x[j]);
            if (last && nv == C) {
              a[(part8 + j) * VT] = __float2bfloat16_rn(q8[j]);
              b[(part8 + j) * VT] = __float2bfloat16_rn(k8[j]);
            } else if (last && k < p.K && tt + j < nv) {
              static_cast<__nv_bfloat16*>(d.dq)[at + (part8 + j) * row] = __float2bfloat16_rn(q8[j]);
              static_cast<__nv_bfloat16*>(d.dk)[at + (part8 + j) * row] = __float2bfloat16_rn(k8[j]);
            }
          }
          if (!last) {  // the next value head's products add to these
            tm_st8(tl + TG::DQ + tt, reinterpret_cast<const uint32_t(&)[8]>(q8));
            tm_st8(tl + TG::DK + tt, reinterpret_cast<const uint32_t(&)[8]>(k8));
          }
        }
        if (!last) tm_wait_st();
        fence_async_smem();
        const float sum = sum_columns(X, lane);
        if (lane < 16) F[GF_X + 64 * quad + t0 + lane] = sum;
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) suma += __shfl_xor_sync(0xffffffffu, suma, m);
        if (lane == 0) F[GF_A + warp] = suma;
      }
      tc_fence_before();
      named_sync<3, G_COMPUTE>();
      if (tid == 0 && nv == C && (ONE || u.r == rep - 1)) {
        gd_tma_store(&maps.dq, sb + G_I, 0, u.h, u.tc0, u.brow);
        gd_tma_store(&maps.dk, sb + G_XB, 0, u.h, u.tc0, u.brow);
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
      if (warp == 15) {  // dbeta and dg: lane l holds tokens 2l and 2l + 1
        float z = 0.f, total = 0.f;
        for (int w = 0; w < 16; ++w) {
          z += F[GF_Z + w];
          total += F[GF_A + w];
        }
        z *= vec[VEC_ALL];
        float x[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // x_t = b_t - a_t + sum_{s > t} P[s][t] - sum_{i < t} P[t][i]
          const int t = 2 * lane + e;
          float be = 0.f;
          x[e] = 0.f;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            be += F[GF_BETA + 64 * w + t];
            x[e] += F[GF_X + 64 * w + t] + F[GF_COL + 64 * w + t] + F[GF_COL + 64 * (w + 4) + t];
          }
          if (t < nv) d.dbeta[((int64_t)u.brow * p.T + u.tc0 + t) * p.HV + u.hv(rep)] = be / vec[VEC_BETA + t];
        }
        // dg_0 = z + sum of all a; dg_{t+1} = dg_t + x_t.
        float run = x[0] + x[1];
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
          const float o = __shfl_up_sync(0xffffffffu, run, m);
          if (lane >= m) run += o;
        }
        const float before = run - x[0] - x[1];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = 2 * lane + e;
          if (t < nv) d.dg[((int64_t)u.brow * p.T + u.tc0 + t) * p.HV + u.hv(rep)] = z + total + before + (e ? x[0] : 0.f);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(s2);
    }
    if (tid == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 16) tm_dealloc(tmem, 512);
}

struct Carved {
  unsigned char *blocks, *s, *ds, *delta;
  float* dr;
  size_t total;
};

// After the cells of a split.
Carved carve(void* ws, const GatedDeltaSplitShape& z, int64_t items) {
  Carved c;
  c.s = static_cast<unsigned char*>(ws) + z.bytes;
  c.ds = c.s + (size_t)items * 65536;
  c.delta = c.ds + (size_t)items * 65536;
  c.dr = reinterpret_cast<float*>(c.delta + (size_t)items * 32768);
  c.blocks = reinterpret_cast<unsigned char*>(c.dr + (size_t)items * 8192);
  c.total = z.bytes + (size_t)items * (2 * 65536 + 2 * 32768 + GB_BYTES_BWD);
  return c;
}

}  // namespace

size_t gated_delta_chunk_backward_bytes(int64_t B, int64_t T, int64_t H, int64_t HV, int64_t K, int64_t V, int64_t n_seq,
                                        kda_dtype dt, bool split) {
  if (!gd_chunk_shape(K, V, dt) || V > VT) return 0;
  const GatedDeltaSplitShape z = split ? gd_split_shape(B, T, HV, K, V, n_seq, true) : GatedDeltaSplitShape{};
  return carve(nullptr, z, gd_slots(B, T, n_seq) * HV).total;
}

cudaError_t launch_gated_delta_chunk_backward(const GatedDeltaParams& p, const GatedDeltaGrads& d, void* ws, size_t bytes,
                                              cudaStream_t s) {
  static std::atomic<uint64_t> cfg[4];
  const bool one = p.H == p.HV;
  auto grads = one ? gated_delta_grads_kernel<true> : gated_delta_grads_kernel<false>;
  cudaError_t e = gd_smem_once(gated_delta_reverse_kernel<false>, R_SMEM, cfg[0]);
  if (e == cudaSuccess) e = gd_smem_once(gated_delta_reverse_kernel<true>, R_SMEM, cfg[3]);
  if (e == cudaSuccess) e = gd_smem_once(grads, G_SMEM, cfg[one ? 1 : 2]);
  int dev = 0, sms = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t slots = gd_slots(p.B, p.T, p.cu ? p.N : 0);
  if (slots * p.HV > 0x7fffffff) return cudaErrorInvalidConfiguration;
  GatedDeltaSplitShape z = gd_split_shape(p.B, p.T, p.HV, p.K, p.V, p.cu ? p.N : 0, true);
  if (bytes < carve(nullptr, z, slots * p.HV).total) z = {};
  const GatedDeltaSplit split = gd_split_carve(z, ws, p.HV, p.K, p.V);
  const Carved c = carve(ws, z, slots * p.HV);
  RMaps r;
  GMaps g;
  const int64_t qk[3] = {p.T * p.H * p.K, (int64_t)p.H * p.K, p.K}, vv[3] = {p.T * p.HV * p.V, (int64_t)p.HV * p.V, p.V};
  if (!gd_token_map(&r.q, p.q, p.qs, p.B, p.T, p.H, p.K, 64, true) || !gd_token_map(&r.k, p.k, p.ks, p.B, p.T, p.H, p.K, 64, true) ||
      !gd_token_map(&r.d_o, d.d_o, p.os, p.B, p.T, p.HV, p.V, 64, true) ||
      !gd_token_map(&g.dq, d.dq, qk, p.B, p.T, p.H, p.K, 128, false) || !gd_token_map(&g.dk, d.dk, qk, p.B, p.T, p.H, p.K, 128, false) ||
      !gd_token_map(&g.dv, d.dv, vv, p.B, p.T, p.HV, p.V, 128, false))
    return cudaErrorNotSupported;
  g.q = r.q;
  g.k = r.k;
  g.d_o = r.d_o;
  const GatedDeltaDump fwd{c.s, c.delta};
  const RDump rev{c.ds, c.dr};
  e = launch_gated_delta_forward(p, c.blocks, &fwd, z, split, s);
  if (e != cudaSuccess) return e;
  if (z.cells) {  // the forward's states at the segments' starts have been read: the gradients take their cells
    gated_delta_reverse_kernel<true><<<(unsigned)(z.cells * p.HV), R_THREADS, R_SMEM, s>>>(p, d, c.blocks, rev, split, r);
    e = cudaGetLastError();
    if (e == cudaSuccess) e = launch_gated_delta_join(p, split, d.d_sf, d.d_sf && d.d_sf == d.ds0, true, s);
    if (e != cudaSuccess) return e;
  }
  const int64_t chains = (z.cells ? std::max<int64_t>(z.segments, p.N) : p.N) * p.HV;
  gated_delta_reverse_kernel<false><<<(unsigned)chains, R_THREADS, R_SMEM, s>>>(p, d, c.blocks, rev, split, r);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int items = (int)(slots * p.H);
  grads<<<(unsigned)std::min(items, std::max(sms, 1)), G_THREADS, G_SMEM, s>>>(p, d, c.blocks, fwd, rev, items, p.HV / p.H, g);
  return cudaGetLastError();
}

cudaError_t gated_delta_bwd_read_timeout(int* flag, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(flag, g_gated_delta_bwd_timeout, sizeof(int));
  if (e != cudaSuccess || !reset) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_gated_delta_bwd_timeout, &zero, sizeof(int));
}

}  // namespace kda
