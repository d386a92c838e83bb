// gated_delta_chunk.cu -- chunked prefill of the gated delta rule with one decay per value head: the state-independent
// operands of every chunk in parallel (kernel P), then the recurrence over chunks (kernel S). Notation in
// gated_delta_chunk.cuh.
#include "gated_delta_chunk.cuh"

namespace kda {

// Set to 1 by any block of these kernels whose bounded wait expired.
__device__ int g_gated_delta_timeout = 0;

namespace {

struct QkMaps {
  CUtensorMap q, k;
};

// ---------------------------------------------------------------------------------------------------------------------
// The length of a split's segments: which takes least time, counted in chunks of kernel S (2.6 us), when chains of at most
// `longest` chunks run in waves over the SMs; a wave costs a chunk more to start, the launches 3, a joined segment 0.7.
// Measured, 8 heads of 16,384 tokens: whole 667 us, estimated 668; in 19 segments 86 + 34 + 49 us, estimated 158.
// ---------------------------------------------------------------------------------------------------------------------
constexpr int SPLIT_LENGTHS = 31;
__host__ __device__ inline int split_length(int least, int i) {  // the least times 2^(i / 4), about
  const int64_t x = ((int64_t)least << (i >> 2)) * (i & 2 ? (i & 1 ? 27 : 23) : (i & 1 ? 19 : 16)) / 16;
  return x < (1 << 24) ? (int)x : 1 << 24;
}
__host__ __device__ inline float split_waves(float work, int longest) {
  return longest ? ceilf(work / ((float)GD_SMS * (float)longest)) * (float)(longest + 1) : 0.f;
}
struct SplitLoad {  // over all chains
  float work, ahead;  // chunks with outputs and without
  int longest, steps;
};
__host__ __device__ inline void split_add(SplitLoad& a, int chunks, int L, int heads, int tiles) {
  a.work += (float)chunks * (float)(heads * tiles);
  const int count = L > 0 && chunks > L ? (chunks + L - 1) / L : 1;
  const int longest = count > 1 ? L : chunks;
  a.longest = a.longest > longest ? a.longest : longest;
  if (count == 1) return;
  a.ahead += (float)heads * (float)L * ((float)(count - 1) * (float)tiles + (float)(count - 2));
  a.steps = a.steps > count - 1 ? a.steps : count - 1;
}
__host__ __device__ inline float split_time(const SplitLoad& a, int L) {
  const float t = split_waves(a.work, a.longest);
  return a.steps ? t + split_waves(a.ahead, L) + 3.f + 0.7f * (float)a.steps : t;
}

// What only the device knows of a packed call, before kernel P (as part of its first blocks it cost 8 us of 106, as a launch
// 4): block 0 plans the split, a length a warp (the last: none); the warps of the others each find one sequence's place in
// the order, how many are longer.
constexpr int PACKED_WARPS = SPLIT_LENGTHS + 1;
__global__ void __launch_bounds__(32 * PACKED_WARPS) gated_delta_packed_kernel(GatedDeltaParams p, int least, int* plan, int* order) {
  __shared__ float time[PACKED_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t t0, t1, brow;
  if (blockIdx.x > 0) {
    const int n = (blockIdx.x - 1) * PACKED_WARPS + warp;
    if (n >= p.N) return;
    gd_range(p, n, t0, t1, brow);
    const int64_t own = t1 - t0;
    int place = 0;
    for (int m = lane; m < p.N; m += 32) {
      gd_range(p, m, t0, t1, brow);
      place += t1 - t0 > own || (t1 - t0 == own && m < n);
    }
    place = __reduce_add_sync(0xffffffffu, place);
    if (lane == 0) order[place] = n;
    return;
  }
  if (!plan) return;
  const int L = warp < SPLIT_LENGTHS ? split_length(least, warp) : 0;
  SplitLoad a = {0.f, 0.f, 0, 0};
  for (int n = lane; n < p.N; n += 32) {
    gd_range(p, n, t0, t1, brow);
    split_add(a, (int)((t1 - t0 + C - 1) / C), L, p.HV, (p.V + VT - 1) / VT);
  }
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) {
    a.work += __shfl_xor_sync(0xffffffffu, a.work, m);
    a.ahead += __shfl_xor_sync(0xffffffffu, a.ahead, m);
    a.longest = max(a.longest, __shfl_xor_sync(0xffffffffu, a.longest, m));
    a.steps = max(a.steps, __shfl_xor_sync(0xffffffffu, a.steps, m));
  }
  if (lane == 0) time[warp] = split_time(a, L);
  __syncthreads();
  if (threadIdx.x == 0) {
    int best = SPLIT_LENGTHS;
    for (int i = SPLIT_LENGTHS - 1; i >= 0; --i)
      if (time[i] < time[best]) best = i;
    *plan = best < SPLIT_LENGTHS ? split_length(least, best) : 0;
  }
}

// ---------------------------------------------------------------------------------------------------------------------
// Kernel P: Z, A and the decay vectors of one chunk and value head, on four warps.
//
// One product on tcgen05, [K ; Q] K^T (M = 128, N = 64, 8 MMAs; both operands are inputs, so it is exact but for the
// fp32 accumulation); a warp then holds 32 rows of K K^T or of Q K^T. The decay ratios are formed from sums kept in two
// fp32 parts: pair by pair in the diagonal 32 x 32 blocks, as e^{G_t - G_31} e^{G_31 - G_i} below them; every factor is at
// most 1, whatever the decay. Then Z = -(I + M)^-1 M by halves: the diagonal 16 x 16 blocks by substitution in fp32, a block
// a warp, and Z21 = -(Y + Z22 Y), Y = M21 + M21 Z11, at 16 and at 32 rows on mma.sync. Those blocks are too small and the
// steps too many for tcgen05's round trips; M and Z stand in shared memory as the two bf16 parts that are Z's images in
// the end (Z written over M), so fragments come by ldmatrix, and Y turns from result to operand inside the registers
// (movmatrix). The steps depend on one another, so what bounds the kernel is their latency until enough blocks share an
// SM: five of 39 KB. Measured, 4096 tokens x 96 heads: 90 us for 358 MB (4.0 TB/s of 6.6; 256 threads and fp32 products
// for the solves 152, mma.sync on eight warps 104).
// ---------------------------------------------------------------------------------------------------------------------
constexpr int P_THREADS = 128;
constexpr int P_KQ = 0;                        // 32 KB: [64-channel half][K 64 rows ; Q 64 rows][128 B]
constexpr int P_Z = 0;                         // after the product, in its place: M's, then Z's two parts, and A's
constexpr int P_A = 16384;
constexpr int DG_LD = 20;                      // row stride of the diagonal blocks, floats
constexpr int P_DIAG = 32768;                  // M's diagonal blocks, fp32 [4][16][20]
constexpr int P_VEC = P_DIAG + 4 * 16 * DG_LD * 4;  // the block's vectors, 1 KB
constexpr int P_G = P_VEC + 1024;              // sums of log2 decays, high [64], low [64]; e^{G_31 - G_i} [32], times beta [32]
constexpr int P_BAR = P_G + 768;
constexpr int P_SMEM = P_BAR + 32;

__device__ __forceinline__ uint32_t mov_trans(uint32_t x) {  // an 8 x 8 block of bf16, transposed
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// A 16 x 16 block's two parts as the A operand, rows r0, columns c0.
struct FragA {
  uint32_t h[4], l[4];
};
__device__ __forceinline__ FragA load_a(uint32_t img, int r0, int c0, int lane) {
  FragA f;
  const uint32_t at = img + sw_chunk(r0 + (lane & 15), (c0 >> 3) + (lane >> 4), 0);
  ldsm_x4(at, f.h[0], f.h[1], f.h[2], f.h[3]);
  ldsm_x4(at + 8192, f.l[0], f.l[1], f.l[2], f.l[3]);
  return f;
}
__device__ __forceinline__ void mma_parts(float (&d)[4], const FragA& a, const uint32_t (&bh)[2], const uint32_t (&bl)[2]) {
  mma_bf16(d, a.h[0], a.h[1], a.h[2], a.h[3], bh[0], bh[1]);
  mma_bf16(d, a.h[0], a.h[1], a.h[2], a.h[3], bl[0], bl[1]);
  mma_bf16(d, a.l[0], a.l[1], a.l[2], a.l[3], bh[0], bh[1]);
}
// A 16 x 8 result as the B operand of the next product.
__device__ __forceinline__ void as_b(const float (&y)[4], uint32_t (&bh)[2], uint32_t (&bl)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h, l;
    split2(y[2 * i], y[2 * i + 1], h, l);
    bh[i] = mov_trans(h);
    bl[i] = mov_trans(l);
  }
}
// The negated 16 x 8 result at rows r0, columns c0 of the images.
__device__ __forceinline__ void store_neg(unsigned char* img, int r0, int c0, const float (&y)[4], int lane) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h, l;
    split2(-y[2 * i], -y[2 * i + 1], h, l);
    const uint32_t at = sw_e(r0 + (lane >> 2) + 8 * i, c0 + 2 * (lane & 3), 0);
    *reinterpret_cast<uint32_t*>(img + at) = h;
    *reinterpret_cast<uint32_t*>(img + 8192 + at) = l;
  }
}

// LO: for the gradients, A's low part in an image of its own and no write strength of zero.
template <bool LO>
__global__ void __launch_bounds__(P_THREADS, 5)
    gated_delta_intra_kernel(GatedDeltaParams p, unsigned char* blocks, int64_t stride, const __grid_constant__ QkMaps maps) {
  extern __shared__ __align__(1024) unsigned char sm[];
  const uint32_t sb = smem_u32(sm);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hv = blockIdx.x % p.HV;
  const int slot = blockIdx.x / p.HV;
  int n;
  int64_t tc0, brow;
  const int nv = gd_slot_tokens(p, slot, n, tc0, brow);
  if (nv == 0) return;
  float* diag = reinterpret_cast<float*>(sm + P_DIAG);
  float* vec = reinterpret_cast<float*>(sm + P_VEC);
  float* gh = reinterpret_cast<float*>(sm + P_G);
  float* gl = gh + 64;
  const uint32_t bar_in = sb + P_BAR, bar_mma = sb + P_BAR + 8;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + P_BAR + 16);
  volatile int* dead = reinterpret_cast<volatile int*>(sm + P_BAR + 24);
  int* flag = &g_gated_delta_timeout;
  if (tid == 0) {
    gd_bar_init(bar_in, 1);
    gd_bar_init(bar_mma, 1);
    *dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    gd_expect(bar_in, 32768);
    const int h = hv / (p.HV / p.H);
    for (int half = 0; half < 2; ++half) {
      gd_tma_load(sb + P_KQ + half * 16384, &maps.k, 64 * half, h, (int)tc0, (int)brow, bar_in);
      gd_tma_load(sb + P_KQ + half * 16384 + 8192, &maps.q, 64 * half, h, (int)tc0, (int)brow, bar_in);
    }
  }
  if (warp == 1) tm_alloc(smem_u32(tslot), 64);
  if (warp == 3) {
    gd_decays(p, hv, tc0, brow, nv, lane, LO ? GD_TINY : 0.f, vec, gh, gl);
    __syncwarp();
    const float c = ex2((gh[31] - gh[lane]) + (gl[31] - gl[lane]));
    gl[64 + lane] = c;
    gl[96 + lane] = c * vec[VEC_BETA + lane];
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  if (warp == 0) {  // one warp waits, suspended; polling would take issue slots from the SM's other blocks
    if (!mbar_wait(bar_in, 0, flag)) *dead = 1;
    if (__all_sync(0xffffffffu, *dead == 0) && elect_one()) {
      constexpr uint32_t id = idesc_bf16(64, 0, 0);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const uint64_t d = sdesc(sb + P_KQ + (ks >> 2) * 16384 + (ks & 3) * 32, 16, 1024);
        tc_mma(tmem, d, d, id, ks > 0);
      }
      tc_commit(bar_mma);
    }
    __syncwarp();
    if (*dead == 0 && !mbar_wait(bar_mma, 0, flag)) *dead = 1;
  }
  __syncthreads();
  tc_fence_after();
  // Warps 0, 1: rows t of K K^T, to M = strict(K K^T * D) diag(beta). Warps 2, 3: rows of Q K^T, to A. Zero above the diagonal.
  const bool is_q = warp >= 2;
  const int lower = warp & 1, t = 32 * lower + lane;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t r[32];
    if (half <= lower) {
      tm_ld32(tmem + ((uint32_t)(32 * warp) << 16) + 32 * half, r);
      const float ghi = gh[t], glo = gl[t];
      if (half == lower) {
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const int i0 = 32 * half + j;
          const float4 a = *reinterpret_cast<const float4*>(gh + i0), b = *reinterpret_cast<const float4*>(gl + i0);
          const float ah[4] = {a.x, a.y, a.z, a.w}, al[4] = {b.x, b.y, b.z, b.w};
          float4 w = make_float4(1.f, 1.f, 1.f, 1.f);
          if (!is_q) w = *reinterpret_cast<const float4*>(vec + VEC_BETA + i0);
          const float wb[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float d = wb[e] * ex2((ghi - ah[e]) + (glo - al[e]));
            r[j + e] = (is_q ? j + e <= lane : j + e < lane) ? __float_as_uint(__uint_as_float(r[j + e]) * d) : 0u;
          }
        }
      } else {
        const float f = ex2((ghi - gh[31]) + (glo - gl[31]));
        const float* gc = gl + (is_q ? 64 : 96);
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 c = *reinterpret_cast<const float4*>(gc + j);
          r[j] = __float_as_uint(__uint_as_float(r[j]) * (f * c.x));
          r[j + 1] = __float_as_uint(__uint_as_float(r[j + 1]) * (f * c.y));
          r[j + 2] = __float_as_uint(__uint_as_float(r[j + 2]) * (f * c.z));
          r[j + 3] = __float_as_uint(__uint_as_float(r[j + 3]) * (f * c.w));
        }
      }
      if (t >= nv) {  // a token past the end: whatever its row holds, not its products
#pragma unroll
        for (int j = 0; j < 32; ++j) r[j] = 0u;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) r[j] = 0u;
    }
    if (!is_q && half == lower) {
      float* d = diag + ((t >> 4) * 16 + (t & 15)) * DG_LD;
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        uint4 x;
        x.x = lane < 16 ? r[j] : r[16 + j];
        x.y = lane < 16 ? r[j + 1] : r[17 + j];
        x.z = lane < 16 ? r[j + 2] : r[18 + j];
        x.w = lane < 16 ? r[j + 3] : r[19 + j];
        *reinterpret_cast<uint4*>(d + j) = x;
      }
    }
    unsigned char* img = sm + (is_q ? P_A : P_Z);
    if (!LO && half > lower) continue;  // A's low part stands there
    // The low part's image, and its row and first 16-byte piece there. Without LO A's takes the upper right quarters.
    unsigned char* img_l = img + 8192;
    int tl = t, cl = 4 * half;
    if (!LO && is_q) {
      img_l = sm + gb_low_image(lower, half);
      tl = lane;
      cl = 4;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) split2(__uint_as_float(r[8 * j + 2 * e]), __uint_as_float(r[8 * j + 2 * e + 1]), hi[e], lo[e]);
      *reinterpret_cast<uint4*>(img + sw_chunk(t, 4 * half + j, 0)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(img_l + sw_chunk(tl, cl + j, 0)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  }
  __syncthreads();
  unsigned char* img = sm + P_Z;
  const uint32_t imgs = sb + P_Z;
  {  // Z of a diagonal block: z_i = -(M_ij + sum_{j<l<i} M_il z_l), column j = lane
    const float* m = diag + 16 * warp * DG_LD;
    const int j = lane & 15;
    float z[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s[2] = {m[i * DG_LD + j], 0.f};  // zero for i <= j
#pragma unroll
      for (int l = 0; l < i; l += 4) {
        const float4 x = *reinterpret_cast<const float4*>(m + i * DG_LD + l);
        const float xx[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (l + e < i) s[e & 1] = fmaf(xx[e], z[l + e], s[e & 1]);
      }
      z[i] = -(s[0] + s[1]);
    }
    if (lane < 16) {
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        uint32_t h, l;
        split2(z[i], z[i + 1], h, l);
        const uint32_t a0 = sw_e(16 * warp + i, 16 * warp + j, 0), a1 = sw_e(16 * warp + i + 1, 16 * warp + j, 0);
        *reinterpret_cast<uint16_t*>(img + a0) = (uint16_t)h;
        *reinterpret_cast<uint16_t*>(img + a1) = (uint16_t)(h >> 16);
        *reinterpret_cast<uint16_t*>(img + 8192 + a0) = (uint16_t)l;
        *reinterpret_cast<uint16_t*>(img + 8192 + a1) = (uint16_t)(l >> 16);
      }
    }
  }
  __syncthreads();
  if (warp < 2) {  // 16 rows: blocks (1, 0) and (3, 2)
    const int ra = 32 * warp + 16, rb = 32 * warp;
    const FragA m = load_a(imgs, ra, rb, lane);
    uint32_t bh[4], bl[4];
    const uint32_t at = imgs + sw_chunk(rb + (lane & 15), (rb >> 3) + (lane >> 4), 0);
    ldsm_x4_t(at, bh[0], bh[1], bh[2], bh[3]);
    ldsm_x4_t(at + 8192, bl[0], bl[1], bl[2], bl[3]);
    const FragA za = load_a(imgs, ra, ra, lane);
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      float y[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 x = add2(unpack_bf16(m.h[2 * nt + i]), unpack_bf16(m.l[2 * nt + i]));
        y[2 * i] = x.x;
        y[2 * i + 1] = x.y;
      }
      const uint32_t zh[2] = {bh[2 * nt], bh[2 * nt + 1]}, zl[2] = {bl[2 * nt], bl[2 * nt + 1]};
      mma_parts(y, m, zh, zl);
      uint32_t yh[2], yl[2];
      as_b(y, yh, yl);
      mma_parts(y, za, yh, yl);
      store_neg(img, ra, rb + 8 * nt, y, lane);
    }
  }
  __syncthreads();
  {  // 32 rows: the lower left quarter, 8 columns a warp
    const int c0 = 8 * warp;
    FragA m[2][2];
    float y[2][4];
    uint32_t bh[4], bl[4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) m[mt][ks] = load_a(imgs, 32 + 16 * mt, 16 * ks, lane);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t at = sw_e(32 + 16 * mt + (lane >> 2) + 8 * i, c0 + 2 * (lane & 3), 0);
        const float2 x = add2(unpack_bf16(*reinterpret_cast<const uint32_t*>(img + at)),
                              unpack_bf16(*reinterpret_cast<const uint32_t*>(img + 8192 + at)));
        y[mt][2 * i] = x.x;
        y[mt][2 * i + 1] = x.y;
      }
    }
    const uint32_t at = imgs + sw_chunk(lane, warp, 0);
    ldsm_x4_t(at, bh[0], bh[1], bh[2], bh[3]);
    ldsm_x4_t(at + 8192, bl[0], bl[1], bl[2], bl[3]);
    __syncthreads();  // M21 is in registers everywhere: Z21 may take its place
    uint32_t yh[2][2], yl[2][2];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const uint32_t zh[2] = {bh[2 * ks], bh[2 * ks + 1]}, zl[2] = {bl[2 * ks], bl[2 * ks + 1]};
        mma_parts(y[mt], m[mt][ks], zh, zl);
      }
      as_b(y[mt], yh[mt], yl[mt]);
    }
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
      for (int ks = 0; ks <= mt; ++ks) mma_parts(y[mt], load_a(imgs, 32 + 16 * mt, 32 + 16 * ks, lane), yh[ks], yl[ks]);
      store_neg(img, 32 + 16 * mt, c0, y[mt], lane);
    }
  }
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0) {
    unsigned char* out = blocks + ((size_t)slot * p.HV + hv) * (size_t)stride;
    gd_bulk_store(out, sb + P_Z, GB_VEC);
    gd_bulk_store(out + GB_VEC, sb + P_VEC, 1024);
    if (LO) {
      gd_bulk_store(out + GB_AL, sb + P_A + 8192, 8192);
      gd_bulk_store(out + GB_SUMS, sb + P_G, 512);
    }
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  }
  if (warp == 1) tm_dealloc(tmem, 64);
  if (*dead && tid == 0) {  // give what may still be in flight a bounded wait
    mbar_wait(bar_in, 0, flag);
    mbar_wait(bar_mma, 0, flag);
  }
}

// ---------------------------------------------------------------------------------------------------------------------
// Kernel S: the recurrence of one (sequence, value head, 128 value columns).
//
// Everything is transposed: accumulator lane v, columns t or k, so that a token's scalars scale columns. Per chunk:
//   P1  (K S)^T = S^T K^T       S^T in two parts from tensor memory: 16 MMAs of N = 64    (then Q S, 16 MMAs)
//   --  R = V - e^G (K S), in two parts to tensor memory
//   P2  Z R                     12 MMAs of N = 64, 48, 32 and 16 (Z is strictly lower)
//   --  delta = R + P2, U = beta delta; e^{G_C - G} U and U in two parts
//   P3  K^T (...)               8 MMAs of N = 128 into a fresh accumulator; then A U onto the output, 14 MMAs
//   --  S = e^{G_C} S + P3 in fp32 registers (32 a thread)
// The output's products take both parts too (A U: high high, high low and, in 6 MMAs of N = 32, low high): it is to carry its
// own rounding to bf16 and no other of that size. With high parts alone o was off by 1.4 times as much, and the kernel took
// 184 us instead of 187.
// The chain P1 -> R -> P2 -> U -> P3 -> S is what bounds it: 36 MMAs of its own (1,400 cycles at the pipe's rate), three times
// the 165 cycles from the last MMA to the threads that wait for it, and the threads' passes. So a warp of its own issues
// the MMAs (one elected thread: an N = 64 MMA leaves every 32 cycles), another feeds two stages by TMA a chunk ahead, and
// what the chain does not need runs in its gaps: V's loads under P1, the conversion of the previous chunk's output under
// P2, e^G on this chunk's under P3. MMAs run in the order they are issued, so what a later commit covers needs no barrier
// of its own. Measured, 4096 tokens x 96 heads: 187 us, 2.9 us a chunk (of some 5,600 cycles the passes issue 3,000);
// with the gradients' dumps 195.
// ---------------------------------------------------------------------------------------------------------------------
constexpr int S_THREADS = 576, S_COMPUTE = 512;  // 16 warps of passes, one of products, one of loads
// Shared memory: two stages (K, Q, V and the block; for the gradients, which form no output, K, V, Z and the vectors),
// then the output's staging tiles, 2 x 16 KB [t][v], or S's and delta's images on their way out, 64 KB and 32 KB.
enum { OUTPUT, DUMP, ADVANCE };  // what kernel S leaves: outputs, the gradients' operands, or end states only
template <int MODE>
struct SLayout {
  static constexpr int K = 0, V = 16384, Q = 32768, B = MODE == OUTPUT ? 49152 : 32768;
  static constexpr int VEC = B + (MODE == OUTPUT ? GB_VEC : 16384);
  static constexpr int STAGE = MODE == OUTPUT ? B + GB_BYTES : VEC + 1024;
  static constexpr int OUT = 2 * STAGE;
  static constexpr int DELTA = OUT + 65536;
  static constexpr int BARS = MODE == DUMP ? DELTA + 32768 : MODE == OUTPUT ? OUT + 32768 : OUT;
  static constexpr int SMEM = BARS + 128;
};
// Tensor memory, 512 columns: S^T's two parts; P3's accumulator, in whose place (dead between P3's read-out and the next
// P3) stand K S, then R's two parts, and P2's accumulator; the output of two chunks; e^{G_C - G} U and U, two parts.
constexpr uint32_t T_SH = 0, T_SL = 64, T_SD = 128, T_KS = 128, T_DA = 192, T_O = 256, T_W = 384, T_U = 448;

struct SMaps {
  CUtensorMap q, k, v, o;
};

// MODE: OUTPUT: the outputs and the final states. DUMP: for the gradients; keeps every chunk's start state and deltas and
// forms no output. ADVANCE: the segment before the one that starts in a cell, from a state of zero (the sequence's own for
// its first segment) to the cell's state; or, as one more tile of columns, from the identity with values of zero to the
// cell's map.
template <int MODE>
__global__ void __launch_bounds__(S_THREADS, 1)
    gated_delta_state_kernel(GatedDeltaParams p, const unsigned char* blocks, int64_t stride, GatedDeltaDump dump,
                             GatedDeltaSplit split, const __grid_constant__ SMaps maps) {
  extern __shared__ __align__(1024) unsigned char sm[];
  using L = SLayout<MODE>;
  constexpr int ST_BYTES = L::STAGE, S_OST = L::OUT, BARS = L::BARS;
  const uint32_t sb = smem_u32(sm);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_vt = (p.V + VT - 1) / VT, tiles = MODE == ADVANCE ? n_vt + 1 : n_vt;
  const int vt = blockIdx.x % tiles;
  const int hv = (blockIdx.x / tiles) % p.HV;
  const int64_t at = blockIdx.x / tiles / p.HV;
  // The plan and the joined states are earlier kernels' work; without them only the loads wait for kernel P's blocks.
  if (split.plan || split.order || (MODE != ADVANCE && split.x)) asm volatile("griddepcontrol.wait;" ::: "memory");
  const int length = split.length();
  const bool map = MODE == ADVANCE && vt == n_vt;
  GatedDeltaSegment g;
  if (MODE == ADVANCE) {
    if (!gd_cell(p, at, length, g) || (map && g.s == 1)) {
      asm volatile("griddepcontrol.wait;" ::: "memory");  // what follows this kernel follows kernel P
      return;
    }
    g.end = g.first;
    g.s -= 1;
    g.first -= (int64_t)length * C;
  } else if (!gd_segment(p, at, length, split.order, g)) {
    return;
  }
  const int64_t t0 = g.first, t1 = g.end, brow = g.brow;
  const int n_chunks = (int)((t1 - t0 + C - 1) / C);
  const int64_t slot0 = gd_slot_base(p, g.n, g.t0) + (int64_t)g.s * length;
  const uint32_t bars = sb + BARS;
  const uint32_t b_full = bars, b_a = bars + 16, b_b = bars + 24, b_c = bars + 32, b_d = bars + 40;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + BARS + 64);
  volatile int* dead = reinterpret_cast<volatile int*>(sm + BARS + 72);
  int* flag = &g_gated_delta_timeout;
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

  if (warp == 17) {  // loads
    if (elect_one()) {
      const int h = hv / (p.HV / p.H);
      asm volatile("griddepcontrol.wait;" ::: "memory");  // the blocks are kernel P's output
      int c = 0;
      for (; c < n_chunks; ++c) {
        if (c >= 2) gd_wait(b_d, c & 1, dead, flag);  // chunk c - 2's products have read the stage
        if (*dead) break;
        const uint32_t st = sb + (c & 1) * ST_BYTES, bar = b_full + 8 * (c & 1);
        const int tc = (int)(t0 + (int64_t)c * C);
        gd_expect(bar, map ? ST_BYTES - 16384 : ST_BYTES);
        for (int half = 0; half < 2; ++half) {
          gd_tma_load(st + L::K + half * 8192, &maps.k, 64 * half, h, tc, (int)brow, bar);
          if (MODE == OUTPUT) gd_tma_load(st + L::Q + half * 8192, &maps.q, 64 * half, h, tc, (int)brow, bar);
        }
        const unsigned char* blk = blocks + ((size_t)(slot0 + c) * p.HV + hv) * (size_t)stride;
        if (MODE != OUTPUT) {
          gd_bulk_load(st + L::B, blk + GB_ZH, 16384, bar);
          gd_bulk_load(st + L::VEC, blk + GB_VEC, 1024, bar);
        } else {
          gd_bulk_load(st + L::B, blk, GB_BYTES, bar);
        }
        if (!map) gd_tma_load(st + L::V, &maps.v, vt * VT, hv, tc, (int)brow, bar);
      }
      if (*dead)  // give the loads that may still be in flight a bounded wait
        for (int i = max(0, c - 2); i < c; ++i) mbar_wait(b_full + 8 * (i & 1), (i >> 1) & 1, flag);
    }
    __syncwarp();
  } else if (warp == 16) {  // products, and the bulk stores of what the passes have staged
    constexpr uint32_t id64 = idesc_bf16(64, 0, 0), id128 = idesc_bf16(128, 0, 1);
    for (int c = 0; c < n_chunks; ++c) {
      const uint32_t st = sb + (c & 1) * ST_BYTES;
      const uint32_t to = tmem + T_O + 64 * (c & 1);
      gd_wait(b_full + 8 * (c & 1), (c >> 1) & 1, dead, flag);
      named_sync<1, S_COMPUTE + 32>();  // S's parts
      tc_fence_after();
      if (__all_sync(0xffffffffu, *dead == 0) && elect_one()) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          tc_mma_ts(tmem + T_KS, tmem + T_SH + 8 * ks, sdesc(st + L::K + (ks >> 2) * 8192 + (ks & 3) * 32, 16, 1024), id64, ks > 0);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          tc_mma_ts(tmem + T_KS, tmem + T_SL + 8 * ks, sdesc(st + L::K + (ks >> 2) * 8192 + (ks & 3) * 32, 16, 1024), id64, 1);
        tc_commit(b_a);
        if (MODE == OUTPUT) {
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            tc_mma_ts(to, tmem + T_SH + 8 * ks, sdesc(st + L::Q + (ks >> 2) * 8192 + (ks & 3) * 32, 16, 1024), id64, ks > 0);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            tc_mma_ts(to, tmem + T_SL + 8 * ks, sdesc(st + L::Q + (ks >> 2) * 8192 + (ks & 3) * 32, 16, 1024), id64, 1);
        }
      }
      __syncwarp();
      named_sync<2, S_COMPUTE + 32>();  // R's parts (and S's images)
      tc_fence_after();
      if (__all_sync(0xffffffffu, *dead == 0) && elect_one()) {
        // Z is strictly lower: tokens t of 16-token step ks and later only.
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const uint32_t id = idesc_bf16(64 - 16 * ks, 0, 0), at = st + L::B + ks * (32 + 2048);
          tc_mma_ts(tmem + T_DA + 16 * ks, tmem + T_KS + 16 * ks, sdesc(at + GB_ZH, 16, 1024), id, ks > 0);
          tc_mma_ts(tmem + T_DA + 16 * ks, tmem + T_KS + 16 * ks, sdesc(at + GB_ZL, 16, 1024), id, 1);
          tc_mma_ts(tmem + T_DA + 16 * ks, tmem + T_KS + 16 * ks + 8, sdesc(at + GB_ZH, 16, 1024), id, 1);
        }
      }
      __syncwarp();
      // The copy of delta's images has left: after this commit the passes may write over them.
      if (MODE == DUMP && lane == 0) {
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        gd_bulk_store(dump.s + ((size_t)(slot0 + c) * p.HV + hv) * 65536, sb + S_OST, 65536);
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
      __syncwarp();
      if (__all_sync(0xffffffffu, *dead == 0) && elect_one()) tc_commit(b_b);
      __syncwarp();
      named_sync<3, S_COMPUTE + 32>(); // e^{G_C - G} U's parts; the previous chunk's output in its staging tile, or S's images
      tc_fence_after();
      if (__all_sync(0xffffffffu, *dead == 0) && elect_one()) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          tc_mma_ts(tmem + T_SD, tmem + T_W + 16 * ks, sdesc(st + L::K + ks * 2048, 8192, 1024), id128, ks > 0);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          tc_mma_ts(tmem + T_SD, tmem + T_W + 16 * ks + 8, sdesc(st + L::K + ks * 2048, 8192, 1024), id128, 1);
      }
      __syncwarp();
      // The copy of S's images has left: after this commit the passes may write over them.
      if (MODE == DUMP && lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      __syncwarp();
      if (__all_sync(0xffffffffu, *dead == 0) && elect_one()) {
        tc_commit(b_c);
        if (MODE != OUTPUT) tc_commit(b_d);
      }
      __syncwarp();
      if (MODE == DUMP) {
        named_sync<4, S_COMPUTE + 32>();  // delta's images
        if (lane == 0) {
          gd_bulk_store(dump.delta + ((size_t)(slot0 + c) * p.HV + hv) * 32768, sb + L::DELTA, 32768);
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
        __syncwarp();
      } else if (MODE == OUTPUT) {
        if (lane == 0) {
          if (c > 0) {  // every chunk but a segment's last is full
            gd_tma_store(&maps.o, sb + S_OST + ((c - 1) & 1) * 16384, vt * VT, hv, (int)(t0 + (int64_t)(c - 1) * C), (int)brow);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");  // the next chunk writes the other tile
          }
        }
        __syncwarp();
        named_sync<4, S_COMPUTE + 32>();  // U's parts; the output's state part is scaled
        tc_fence_after();
        if (__all_sync(0xffffffffu, *dead == 0) && elect_one()) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint32_t id = idesc_bf16(64 - 16 * ks, 0, 0), at = st + L::B + GB_AH + ks * (32 + 2048);
            tc_mma_ts(to + 16 * ks, tmem + T_U + 16 * ks, sdesc(at, 16, 1024), id, 1);
            tc_mma_ts(to + 16 * ks, tmem + T_U + 16 * ks + 8, sdesc(at, 16, 1024), id, 1);
          }
          // A's low part: of 32 x 32 quarter (h, g) tokens 32 h to the output, tokens 32 g of U.
#pragma unroll
          for (int i = 0; i < 6; ++i) {
            const int h = i > 1, g = i > 3, ks = 2 * g + (i & 1);
            tc_mma_ts(to + 32 * h, tmem + T_U + 16 * ks, sdesc(st + L::B + gb_low_image(h, g) + 64 + 32 * (i & 1), 16, 1024),
                      idesc_bf16(32, 0, 0), 1);
          }
          tc_commit(b_d);
        }
        __syncwarp();
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    if (*dead && n_chunks > 0 && lane == 0) {
      mbar_wait(b_d, 0, flag);
      mbar_wait(b_d, 1, flag);
    }
    __syncwarp();
  } else {  // the passes: lane v = 32 quad + lane of S^T; a quarter of the columns (32 channels, 16 tokens)
    const int quad = warp & 3, part = warp >> 2, v = 32 * quad + lane, vg = vt * VT + v;
    const uint32_t tl = tmem + ((uint32_t)(32 * quad) << 16);
    const bool there = map ? v < p.K : vg < p.V;
    const size_t hbase = ((size_t)g.n * p.HV + hv) * (size_t)p.K * p.V;
    const float* from = p.s0 ? p.s0 + hbase : nullptr;
    if (MODE == ADVANCE) {
      if (g.s > 0) from = nullptr;
    } else if (g.s > 0) {
      from = split.x + ((size_t)(g.cell0 + g.s) * p.HV + hv) * split.x_size;
    } else if (g.count > 1 && p.s0 == p.sf && p.s0) {  // the last segment writes over the given state
      from = split.m + ((size_t)(g.cell0 + 1) * p.HV + hv) * split.m_size;
    }
    float2 S[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int k = 32 * part + 2 * j;
      const bool in = from && there && k < p.K;  // K is even
      S[j].x = in ? from[(size_t)k * p.V + vg] : 0.f;
      S[j].y = in ? from[(size_t)(k + 1) * p.V + vg] : 0.f;
      if (map && there) S[j] = make_float2(k == v ? 1.f : 0.f, k + 1 == v ? 1.f : 0.f);
    }
    float all = 1.f;
    for (int c = 0; c < n_chunks; ++c) {
      unsigned char* st = sm + (c & 1) * ST_BYTES;
      const float* vec = reinterpret_cast<const float*>(st + L::VEC);
      const float4* ve = reinterpret_cast<const float4*>(vec + VEC_E + 16 * part);
      const float4* vr = reinterpret_cast<const float4*>(vec + VEC_REST + 16 * part);
      const float4* vb = reinterpret_cast<const float4*>(vec + VEC_BETA + 16 * part);
      const int nv = (int)min((int64_t)C, t1 - t0 - (int64_t)c * C);
      if (nv < C) {  // rows past the sequence's end hold other tokens, or anything: zeros instead
        gd_wait(b_full + 8 * (c & 1), (c >> 1) & 1, dead, flag);
        zero_rows(st + L::K, 2, nv, tid, S_COMPUTE);
        if (MODE == OUTPUT) zero_rows(st + L::Q, 2, nv, tid, S_COMPUTE);
        zero_rows(st + L::V, 0, nv, tid, S_COMPUTE);
        fence_async_smem();
        named_sync<5, S_COMPUTE>();
      }
      uint32_t sh[16], sl[16];
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
      tc_fence_before();
      named_arrive<1, S_COMPUTE + 32>();
      // Under P1: V's values of this thread (and S's images).
      gd_wait(b_full + 8 * (c & 1), (c >> 1) & 1, dead, flag);
      all = vec[VEC_ALL];
      float2 R[8];
      {
        const __nv_bfloat16* vp = reinterpret_cast<const __nv_bfloat16*>(st + L::V) + (16 * part) * VT + v;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          R[j] = map ? make_float2(0.f, 0.f) : make_float2(__bfloat162float(vp[2 * j * VT]), __bfloat162float(vp[(2 * j + 1) * VT]));
      }
      if (MODE == DUMP) {
        unsigned char* img = sm + S_OST + (part >> 1) * 16384 + v * 128;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int at = ((4 * (part & 1) + j) ^ (v & 7)) << 4;
          *reinterpret_cast<uint4*>(img + at) = make_uint4(sh[4 * j], sh[4 * j + 1], sh[4 * j + 2], sh[4 * j + 3]);
          *reinterpret_cast<uint4*>(img + 32768 + at) = make_uint4(sl[4 * j], sl[4 * j + 1], sl[4 * j + 2], sl[4 * j + 3]);
        }
        fence_async_smem();
      }
      gd_wait(b_a, c & 1, dead, flag);
      tc_fence_after();
      {
        uint32_t r[16], hi[8], lo[8];
        tm_ld16(tl + T_KS + 16 * part, r);
        tm_wait_ld();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 e = ve[j];
          R[2 * j] = fma2(make_float2(-e.x, -e.y), as_f2(r[4 * j], r[4 * j + 1]), R[2 * j]);
          R[2 * j + 1] = fma2(make_float2(-e.z, -e.w), as_f2(r[4 * j + 2], r[4 * j + 3]), R[2 * j + 1]);
          split2(R[2 * j].x, R[2 * j].y, hi[2 * j], lo[2 * j]);
          split2(R[2 * j + 1].x, R[2 * j + 1].y, hi[2 * j + 1], lo[2 * j + 1]);
        }
        tm_st8(tl + T_KS + 16 * part, hi);
        tm_st8(tl + T_KS + 16 * part + 8, lo);
        tm_wait_st();
      }
      tc_fence_before();
      named_arrive<2, S_COMPUTE + 32>();
      // Under P2: the previous chunk's output, which P1 followed through the pipe, to its staging tile.
      if (MODE == OUTPUT && c > 0) {
        uint32_t r[16];
        tm_ld16(tl + T_O + 64 * ((c - 1) & 1) + 16 * part, r);
        tm_wait_ld();
        __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(sm + S_OST + ((c - 1) & 1) * 16384) + (16 * part) * VT + v;
#pragma unroll
        for (int j = 0; j < 16; ++j) dst[j * VT] = __float2bfloat16_rn(__uint_as_float(r[j]));
        fence_async_smem();
      }
      gd_wait(b_b, c & 1, dead, flag);
      tc_fence_after();
      {
        uint32_t r[16], hi[8], lo[8];
        tm_ld16(tl + T_DA + 16 * part, r);
        tm_wait_ld();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 b = vb[j], w = vr[j];
          R[2 * j] = add2(R[2 * j], as_f2(r[4 * j], r[4 * j + 1]));  // delta
          R[2 * j + 1] = add2(R[2 * j + 1], as_f2(r[4 * j + 2], r[4 * j + 3]));
          const float2 u0 = mul2(make_float2(b.x, b.y), R[2 * j]), u1 = mul2(make_float2(b.z, b.w), R[2 * j + 1]);
          const float2 w0 = mul2(make_float2(w.x, w.y), u0), w1 = mul2(make_float2(w.z, w.w), u1);
          split2(w0.x, w0.y, hi[2 * j], lo[2 * j]);
          split2(w1.x, w1.y, hi[2 * j + 1], lo[2 * j + 1]);
          if (MODE == OUTPUT) {
            R[2 * j] = u0;
            R[2 * j + 1] = u1;
          }
        }
        tm_st8(tl + T_W + 16 * part, hi);
        tm_st8(tl + T_W + 16 * part + 8, lo);
        tm_wait_st();
      }
      tc_fence_before();
      named_arrive<3, S_COMPUTE + 32>();
      // Under P3: U's parts for the output and e^G on its state part (P2 followed it through the pipe), or the deltas.
      if (MODE == OUTPUT) {
        uint32_t r[16], hi[8], lo[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) split2(R[j].x, R[j].y, hi[j], lo[j]);
        tm_st8(tl + T_U + 16 * part, hi);
        tm_st8(tl + T_U + 16 * part + 8, lo);
        tm_ld16(tl + T_O + 64 * (c & 1) + 16 * part, r);
        tm_wait_ld();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 e = ve[j];
          const float2 x = mul2(make_float2(e.x, e.y), as_f2(r[4 * j], r[4 * j + 1]));
          const float2 y = mul2(make_float2(e.z, e.w), as_f2(r[4 * j + 2], r[4 * j + 3]));
          r[4 * j] = __float_as_uint(x.x);
          r[4 * j + 1] = __float_as_uint(x.y);
          r[4 * j + 2] = __float_as_uint(y.x);
          r[4 * j + 3] = __float_as_uint(y.y);
        }
        tm_st16(tl + T_O + 64 * (c & 1) + 16 * part, r);
        tm_wait_st();
        tc_fence_before();
        named_arrive<4, S_COMPUTE + 32>();
      } else if (MODE == DUMP) {
        unsigned char* img = sm + L::DELTA;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split2(R[4 * j + e].x, R[4 * j + e].y, hi[e], lo[e]);
          const uint32_t at = sw_chunk(v, 2 * part + j, 0);
          *reinterpret_cast<uint4*>(img + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(img + 16384 + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        fence_async_smem();
        named_arrive<4, S_COMPUTE + 32>();
      }
    }
    if (n_chunks > 0) {
      gd_wait(b_c, (n_chunks - 1) & 1, dead, flag);
      tc_fence_after();
      uint32_t r[32];
      tm_ld32(tl + T_SD + 32 * part, r);
#pragma unroll
      for (int j = 0; j < 16; ++j) S[j] = fma2(make_float2(all, all), S[j], as_f2(r[2 * j], r[2 * j + 1]));
      if (MODE == OUTPUT) {  // the last chunk's output, which may be partial, straight out
        gd_wait(b_d, (n_chunks - 1) & 1, dead, flag);
        tc_fence_after();
        uint32_t o[16];
        tm_ld16(tl + T_O + 64 * ((n_chunks - 1) & 1) + 16 * part, o);
        tm_wait_ld();
        const int64_t tc = t0 + (int64_t)(n_chunks - 1) * C + 16 * part;
        __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.o) + brow * p.os[0] + hv * p.os[2] + tc * p.os[1] + vg;
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (there && tc + j < t1) orow[j * p.os[1]] = __float2bfloat16_rn(__uint_as_float(o[j]));
      }
    }
    float* to = MODE == ADVANCE ? (map ? split.mb : split.x)
                : p.sf && g.s == g.count - 1 ? p.sf + hbase
                                             : nullptr;
    if (MODE == ADVANCE && to) to += ((size_t)at * p.HV + hv) * (map ? split.m_size : split.x_size);
    if (to && there) {
      const int row = map ? p.K : p.V, col = map ? v : vg;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int k = 32 * part + 2 * j;
        if (k < p.K) {
          to[(size_t)k * row + col] = S[j].x;
          to[(size_t)(k + 1) * row + col] = S[j].y;
        }
      }
    }
    if (map && there) {
      float4* across = reinterpret_cast<float4*>(split.m + ((size_t)at * p.HV + hv) * split.m_size + (size_t)v * p.K + 32 * part);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (32 * part + 4 * j < p.K) across[j] = make_float4(S[2 * j].x, S[2 * j].y, S[2 * j + 1].x, S[2 * j + 1].y);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 16) tm_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------------------------------------------------
// Joins the segments of a sequence, one after another: X[s + 1] += E_s X[s], X[s] the state at the start of segment s and
// E_s its map; the gradients (BACK): Y[s] += E_s^T Y[s + 1], Y[s] the gradient there. A block takes 8 columns of one value
// head; a warp 16 of the 128 terms of every sum, for all 128 rows, so that a map's element is needed by one thread only and
// goes straight to its registers, a step ahead (in rows of the terms: a warp reads whole lines; across them, 128 lines a
// warp for the same elements, a step took 3.7 us); the warps' shares meet in shared memory. All in fp32.
// ---------------------------------------------------------------------------------------------------------------------
constexpr int J_COLS = 8, J_THREADS = 256;
template <bool BACK>
__global__ void __launch_bounds__(J_THREADS) gated_delta_join_kernel(GatedDeltaParams p, GatedDeltaSplit split, const float* given, bool keep) {
  __shared__ __align__(16) float x[128][J_COLS];
  __shared__ __align__(16) float4 share[8][2][128];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int L = split.length();
  if (!L) return;
  const int tiles = p.V / J_COLS, v0 = (blockIdx.x % tiles) * J_COLS, hv = blockIdx.x / tiles % p.HV;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, K = p.K;
  const int k = threadIdx.x & 127, half = threadIdx.x >> 7;  // four columns of a row, where the shares meet
  const bool terms = 16 * warp < K;                          // K is a multiple of 16
  for (int n = blockIdx.x / tiles / p.HV; n < p.N; n += gridDim.x / tiles / p.HV) {
    GatedDeltaSegment g;
    gd_describe(p, n, (int64_t)L * C, g);
    if (g.count < 2) continue;
    auto state = [&](int s) {
      return reinterpret_cast<float4*>(split.x + ((size_t)(g.cell0 + s) * p.HV + hv) * split.x_size + (size_t)k * p.V + v0 + 4 * half);
    };
    if (keep && k < K)
      *reinterpret_cast<float4*>(split.m + ((size_t)(g.cell0 + 1) * p.HV + hv) * split.m_size + (size_t)k * p.V + v0 + 4 * half) =
          *reinterpret_cast<const float4*>(given + ((size_t)n * p.HV + hv) * split.x_size + (size_t)k * p.V + v0 + 4 * half);
    const int first = BACK ? g.count - 2 : 1, step = BACK ? -1 : 1, steps = g.count - 2;
    if (steps < 1) continue;
    float e[4][16];  // the map's elements of rows lane, lane + 32, ... and this warp's terms
    auto load = [&](int s) {
      const float* m = (BACK ? split.mb : split.m) + ((size_t)(g.cell0 + s + 1) * p.HV + hv) * split.m_size;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = lane + 32 * r;
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          if (terms && row < K) {
#pragma unroll
            for (int i = 0; i < 4; ++i) e[r][j + i] = m[(size_t)(16 * warp + j + i) * K + row];
          } else {
            e[r][j] = e[r][j + 1] = e[r][j + 2] = e[r][j + 3] = 0.f;
          }
        }
      }
    };
    load(first);
    *reinterpret_cast<float4*>(&x[k][4 * half]) = k < K ? *state(BACK ? first + 1 : first) : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < steps; ++i) {
      const int s = first + i * step;
      float4* own = state(BACK ? s : s + 1);
      float4 sum = k < K ? *own : make_float4(0.f, 0.f, 0.f, 0.f);
      __syncthreads();
      if (terms) {
        float2 y[4][4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int c = 0; c < 4; ++c) y[r][c] = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float4 u = *reinterpret_cast<const float4*>(x[16 * warp + j]), z = *reinterpret_cast<const float4*>(x[16 * warp + j] + 4);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float2 f = make_float2(e[r][j], e[r][j]);
            y[r][0] = fma2(f, make_float2(u.x, u.y), y[r][0]);
            y[r][1] = fma2(f, make_float2(u.z, u.w), y[r][1]);
            y[r][2] = fma2(f, make_float2(z.x, z.y), y[r][2]);
            y[r][3] = fma2(f, make_float2(z.z, z.w), y[r][3]);
          }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          share[warp][0][lane + 32 * r] = make_float4(y[r][0].x, y[r][0].y, y[r][1].x, y[r][1].y);
          share[warp][1][lane + 32 * r] = make_float4(y[r][2].x, y[r][2].y, y[r][3].x, y[r][3].y);
        }
      }
      if (i + 1 < steps) load(s + step);
      __syncthreads();
      for (int w = 0; 16 * w < K; ++w) {
        const float4 f = share[w][half][k];
        sum.x += f.x;
        sum.y += f.y;
        sum.z += f.z;
        sum.w += f.w;
      }
      *reinterpret_cast<float4*>(&x[k][4 * half]) = sum;
      if (k < K) *own = sum;
    }
    __syncthreads();
  }
}

}  // namespace

GatedDeltaSplitShape gd_split_shape(int64_t B, int64_t T, int64_t HV, int64_t K, int64_t V, int64_t n_seq, bool grads) {
  const int tiles = (int)((V + VT - 1) / VT);
  const int64_t share = gd_slots(B, T, n_seq) * HV * tiles * 3 / (4 * GD_SMS);
  GatedDeltaSplitShape z{};
  z.least = (int)std::min<int64_t>(std::max<int64_t>(share, 8), 1 << 20);
  const int64_t chunks = (T + C - 1) / C;
  // Packed: one sequence of all the tokens, which gains the most.
  const int64_t N = n_seq > 0 ? 1 : B;
  auto time = [&](int L) {
    SplitLoad a{0.f, 0.f, 0, 0};
    split_add(a, (int)std::min<int64_t>(chunks, 1 << 30), L, (int)HV, tiles);
    a.work *= (float)N;
    a.ahead *= (float)N;
    return split_time(a, L);
  };
  float best = time(0);
  for (int i = 0; i < SPLIT_LENGTHS; ++i)
    if (const float t = time(split_length(z.least, i)); t < best) {
      best = t;
      z.chunks = split_length(z.least, i);
    }
  // In the order that they are packed in, the chains of 16 sequences (13,337 tokens, one of 2,767) and 32 heads took 225 us on
  // 148 SMs, the longest first 160. Order and plan look at all sequences several times, so there is a limit.
  z.ordered = n_seq > 1 && n_seq <= 4096 ? n_seq : 0;
  z.bytes = (size_t)(z.ordered + 3) / 4 * 16;
  if (n_seq > 4096) z.chunks = 0;
  if (!z.chunks) return z;
  const int64_t span = (int64_t)(n_seq > 0 ? z.least : z.chunks) * C;
  z.packed = n_seq > 0;
  z.cells = z.packed ? T / span + 1 : B * ((T + span - 1) / span);
  z.segments = z.packed ? T / span + n_seq : z.cells;
  if (z.packed) z.chunks = 0;
  z.grads = grads;
  z.bytes += (size_t)z.cells * HV * K * (V + (grads ? 2 : 1) * std::max(K, V)) * 4 + 16;
  return z;
}

GatedDeltaSplit gd_split_carve(const GatedDeltaSplitShape& z, void* ws, int64_t HV, int64_t K, int64_t V) {
  GatedDeltaSplit split{nullptr, nullptr, z.chunks, nullptr, nullptr, nullptr, K * V, K * std::max(K, V)};
  float* end = static_cast<float*>(ws);
  auto take = [&](int64_t each) {
    float* at = end;
    end += (size_t)z.cells * HV * each;
    return at;
  };
  if (z.cells) {
    split.x = take(split.x_size);
    split.m = take(split.m_size);
    if (z.grads) split.mb = take(split.m_size);
    if (z.packed) split.plan = reinterpret_cast<int*>(end);
    end += 4;
  }
  if (z.ordered) split.order = reinterpret_cast<int*>(end);
  return split;
}

cudaError_t launch_gated_delta_join(const GatedDeltaParams& p, const GatedDeltaSplit& split, const float* given, bool keep,
                                    bool back, cudaStream_t s) {
  auto kernel = back ? gated_delta_join_kernel<true> : gated_delta_join_kernel<false>;
  const int64_t blocks = (int64_t)(p.V / J_COLS) * p.HV;
  const int64_t at_once = std::min<int64_t>(p.N, std::max<int64_t>(1, 4 * GD_SMS / blocks));
  if (blocks * at_once > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks * at_once));
  cfg.blockDim = dim3(J_THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p, split, given, keep);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

cudaError_t launch_gated_delta_forward(const GatedDeltaParams& p, unsigned char* blocks, const GatedDeltaDump* dump,
                                       const GatedDeltaSplitShape& z, const GatedDeltaSplit& split, cudaStream_t s) {
  static std::atomic<uint64_t> cfg[5];
  auto state = dump ? gated_delta_state_kernel<DUMP> : gated_delta_state_kernel<OUTPUT>;
  const int smem = dump ? SLayout<DUMP>::SMEM : SLayout<OUTPUT>::SMEM;
  cudaError_t e = gd_smem_once(dump ? gated_delta_intra_kernel<true> : gated_delta_intra_kernel<false>, P_SMEM, cfg[dump ? 1 : 0]);
  if (e == cudaSuccess) e = gd_smem_once(state, smem, cfg[dump ? 3 : 2]);
  if (e == cudaSuccess) e = gd_smem_once(gated_delta_state_kernel<ADVANCE>, SLayout<ADVANCE>::SMEM, cfg[4]);
  if (e != cudaSuccess) return e;
  QkMaps qk;
  SMaps sm;
  std::memset(&sm, 0, sizeof(sm));
  if (!gd_token_map(&qk.q, p.q, p.qs, p.B, p.T, p.H, p.K, 64, true) || !gd_token_map(&qk.k, p.k, p.ks, p.B, p.T, p.H, p.K, 64, true) ||
      !gd_token_map(&sm.v, p.v, p.vs, p.B, p.T, p.HV, p.V, 128, false) ||
      (!dump && !gd_token_map(&sm.o, p.o, p.os, p.B, p.T, p.HV, p.V, 128, false)))
    return cudaErrorNotSupported;  // nothing launched: the caller takes the other kernels
  sm.q = qk.q;
  sm.k = qk.k;
  const bool splits = z.cells > 0;
  const int64_t slots = gd_slots(p.B, p.T, p.cu ? p.N : 0), tiles = (p.V + VT - 1) / VT;
  const int64_t items = slots * p.HV, chains = (splits ? std::max<int64_t>(z.segments, p.N) : p.N) * p.HV * tiles;
  const int64_t ahead = z.cells * p.HV * (tiles + 1);
  if (items > 0x7fffffff || chains > 0x7fffffff || ahead > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const int64_t stride = dump ? GB_BYTES_BWD : GB_BYTES;
  if (split.plan || split.order) {
    gated_delta_packed_kernel<<<(unsigned)(1 + (z.ordered + PACKED_WARPS - 1) / PACKED_WARPS), 32 * PACKED_WARPS, 0, s>>>(p, z.least, const_cast<int*>(split.plan), const_cast<int*>(split.order));
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (dump)
    gated_delta_intra_kernel<true><<<(unsigned)items, P_THREADS, P_SMEM, s>>>(p, blocks, stride, qk);
  else
    gated_delta_intra_kernel<false><<<(unsigned)items, P_THREADS, P_SMEM, s>>>(p, blocks, stride, qk);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const GatedDeltaDump d = dump ? *dump : GatedDeltaDump{};
  cudaLaunchConfig_t cfgl = {};
  cfgl.blockDim = dim3(S_THREADS);
  cfgl.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfgl.attrs = attr;
  // Programmatic dependent launches: blocks set up while the last blocks of the kernel before finish. Every block of
  // every kernel waits for the kernel before it, so what an earlier one wrote is there too.
  cfgl.numAttrs = 1;
  if (splits) {
    cfgl.gridDim = dim3((unsigned)ahead);
    cfgl.dynamicSmemBytes = SLayout<ADVANCE>::SMEM;
    e = cudaLaunchKernelEx(&cfgl, gated_delta_state_kernel<ADVANCE>, p, static_cast<const unsigned char*>(blocks), stride, d, split, sm);
    if (e == cudaSuccess) e = launch_gated_delta_join(p, split, p.s0, p.s0 && p.s0 == p.sf, false, s);
    if (e != cudaSuccess) return e;
  }
  cfgl.gridDim = dim3((unsigned)chains);
  cfgl.dynamicSmemBytes = smem;
  e = cudaLaunchKernelEx(&cfgl, state, p, static_cast<const unsigned char*>(blocks), stride, d, split, sm);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

// Workspace: the cells of a split (which are fp32 and start it), then the blocks.
size_t gated_delta_chunk_bytes(int64_t B, int64_t T, int64_t H, int64_t HV, int64_t K, int64_t V, int64_t n_seq, kda_dtype dt,
                               bool split) {
  if (!gd_chunk_shape(K, V, dt)) return 0;
  // Short calls go token by token: one launch, and no chunk of 64 to fill. That takes a quarter of a us a token for every
  // warp that a scheduler has beyond its first, the chunked kernels 15 us at least and 7 for every further chain of an SM.
  // Measured, chunked and token by token: 32 heads, 1 token 15 and 3.9 us, 32 tokens 15 and 11.5, 48 tokens 15.2 and 15.3;
  // 96 heads, 16 tokens 15.4 and 14.2, 32 tokens 15.4 and 24; 8 x 96 heads, 8 tokens 66 and 53; 64 x 32 heads, 4 tokens 170
  // and 99, 16 tokens 174 and 213.
  // Packed, T counts all tokens, and one sequence may have them all: the warps are one sequence's. Every further sequence costs
  // its states' way in and out, 5 us for as many chains as SMs, and the chunked kernels a chunk too, 12 us: the difference is
  // worth 24 tokens at least. Measured, 32 heads, chunked and token by token: 16 sequences of 2 tokens 49 and 22 us, 40 of one
  // 119 and 47, 40 of 8 tokens 121 and 89 (132 where one has all but 39), 40 of 16 tokens 124 and 135; 96 heads, 64 of 4
  // tokens 529 and 296, 64 of 16 548 and 632.
  const double warps = (double)(n_seq > 0 ? 1 : B) * (double)HV * (double)V * 4 / 32 / (4 * GD_SMS);
  const double further = (double)n_seq * (double)HV * (double)((V + VT - 1) / VT) / GD_SMS;
  if (T <= 8 || (double)T * std::max(warps, 1.0) <= std::max(44.0, 24 * further)) return 0;
  return (split ? gd_split_shape(B, T, HV, K, V, n_seq, false).bytes : 0) + (size_t)gd_slots(B, T, n_seq) * HV * GB_BYTES;
}

cudaError_t launch_gated_delta_chunk(const GatedDeltaParams& p, void* ws, size_t bytes, cudaStream_t s) {
  const int64_t n_seq = p.cu ? p.N : 0;
  GatedDeltaSplitShape z = gd_split_shape(p.B, p.T, p.HV, p.K, p.V, n_seq, false);
  if (bytes < z.bytes + (size_t)gd_slots(p.B, p.T, n_seq) * p.HV * GB_BYTES) z = {};
  const GatedDeltaSplit split = gd_split_carve(z, ws, p.HV, p.K, p.V);
  return launch_gated_delta_forward(p, static_cast<unsigned char*>(ws) + z.bytes, nullptr, z, split, s);
}

cudaError_t gated_delta_bwd_read_timeout(int* flag, bool reset);  // gated_delta_chunk_backward.cu

cudaError_t gated_delta_read_timeout(int* flag, bool reset) {
  int fwd = 0, bwd = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&fwd, g_gated_delta_timeout, sizeof(int));
  const int zero = 0;
  if (e == cudaSuccess && reset) e = cudaMemcpyToSymbol(g_gated_delta_timeout, &zero, sizeof(int));
  if (e == cudaSuccess) e = gated_delta_bwd_read_timeout(&bwd, reset);
  *flag = fwd || bwd;
  return e;
}

}  // namespace kda
