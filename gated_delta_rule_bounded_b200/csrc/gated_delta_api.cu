// gated_delta_api.cu -- the C ABI of the gated delta rule with one decay per value head, and of layer norm: argument
// validation, kernel selection, status codes. Everything that can be refused is refused before a launch.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "gated_delta.h"
#include "kda_internal.h"

namespace {

int fail(int code, const char* fmt, ...) {
  char msg[384];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return kda::report_error(code, msg);
}

int ok() { return kda::report_error(KDA_OK, ""); }

int cuda_fail(cudaError_t e, const char* fn) {
  return fail(KDA_ERR_CUDA, "%s: %s (%s)", fn, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
  return x < y + nb && y < x + na;
}

struct Sizes {
  int64_t B, T, H, HV, K, V, n_seq;
};

constexpr int64_t MOST_ROWS = (int64_t)1 << 31;

// Sizes and types that every scan entry shares.
int check_sizes(const char* fn, kda_dtype dtype, const Sizes& z) {
  if (z.B < 0 || z.T < 0 || z.n_seq < 0) return fail(KDA_ERR_INVALID_ARG, "%s: negative size", fn);
  if (dtype != KDA_F32 && dtype != KDA_BF16) return fail(KDA_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
  if (z.H <= 0 || z.HV <= 0 || z.HV % z.H != 0)
    return fail(KDA_ERR_INVALID_ARG, "%s: HV must be a positive multiple of H (H=%lld, HV=%lld)", fn, (long long)z.H,
                (long long)z.HV);
  if (z.HV > 65535) return fail(KDA_ERR_UNSUPPORTED, "%s: HV must be at most 65535 (got %lld)", fn, (long long)z.HV);
  auto dim = [](int64_t d) { return d >= 16 && d <= 256 && d % 16 == 0; };
  if (!dim(z.K) || !dim(z.V))
    return fail(KDA_ERR_UNSUPPORTED, "%s: K and V must be multiples of 16 in [16,256] (K=%lld, V=%lld)", fn, (long long)z.K,
                (long long)z.V);
  if (z.B >= MOST_ROWS || z.T >= MOST_ROWS || z.n_seq >= MOST_ROWS ||
      (z.T > 0 && z.B * z.T > (MOST_ROWS - 1) / z.HV) || (z.n_seq > z.B ? z.n_seq : z.B) > (MOST_ROWS - 1) / (z.HV * 16))
    return fail(KDA_ERR_UNSUPPORTED, "%s: B*T*HV and 16*N*HV must be below 2^31", fn);
  return KDA_OK;
}

kda_layout dense_layout(const Sizes& z) {
  auto of = [&](int64_t heads, int64_t d) { return kda_strides{z.T * heads * d, heads * d, d}; };
  kda_layout L;
  L.q = L.k = of(z.H, z.K);
  L.v = L.o = of(z.HV, z.V);
  L.gate = L.beta = of(z.HV, 1);
  return L;
}

// Fills the parameters; rows of q, k, v and o have to start on 16-byte boundaries.
int check_tensors(const char* fn, kda_dtype dtype, const Sizes& z, const kda_layout* layout, const void* q, const void* k,
                  const void* v, const float* g, const float* beta, const void* o, kda::GatedDeltaParams& p) {
  if (!q || !k || !v || !g || !beta || !o) return fail(KDA_ERR_INVALID_ARG, "%s: null tensor pointer", fn);
  const kda_layout L = layout ? *layout : dense_layout(z);
  const int64_t es = dtype == KDA_F32 ? 4 : 2;
  const kda_strides* all[6] = {&L.q, &L.k, &L.v, &L.gate, &L.beta, &L.o};
  int64_t* out[6] = {p.qs, p.ks, p.vs, p.gs, p.bs, p.os};
  const void* base[6] = {q, k, v, g, beta, o};
  for (int i = 0; i < 6; ++i) {
    const kda_strides& s = *all[i];
    if (s.b < 0 || s.t < 0 || s.h < 0) return fail(KDA_ERR_INVALID_ARG, "%s: negative stride", fn);
    out[i][0] = s.b;
    out[i][1] = s.t;
    out[i][2] = s.h;
    if (i == 3 || i == 4) continue;
    const int64_t heads = i < 2 ? z.H : z.HV;
    if (!aligned16(base[i]) || (z.B > 1 && s.b * es % 16) || (z.T > 1 && s.t * es % 16) || (heads > 1 && s.h * es % 16))
      return fail(KDA_ERR_UNSUPPORTED, "%s: token rows must start on 16-byte boundaries", fn);
  }
  if ((reinterpret_cast<uintptr_t>(g) & 3) || (reinterpret_cast<uintptr_t>(beta) & 3))
    return fail(KDA_ERR_UNSUPPORTED, "%s: misaligned g or beta", fn);
  p.q = q;
  p.k = k;
  p.v = v;
  p.g = g;
  p.beta = beta;
  p.o = const_cast<void*>(o);
  p.T = z.T;
  p.B = (int)z.B;
  p.H = (int)z.H;
  p.HV = (int)z.HV;
  p.K = (int)z.K;
  p.V = (int)z.V;
  return KDA_OK;
}

// Rows of o on top of one another would be written by several blocks.
int check_output(const char* fn, const Sizes& z, const kda::GatedDeltaParams& p) {
  if ((z.B > 1 && p.os[0] == 0) || (z.T > 1 && p.os[1] == 0) || (z.HV > 1 && p.os[2] == 0))
    return fail(KDA_ERR_INVALID_ARG, "%s: o has a stride of zero over an extent above one", fn);
  return KDA_OK;
}

bool backward_dim(int64_t d) { return d == 16 || d == 32 || d == 64 || d == 128; }

// The workspace of a call; without `split`, the least that lets it run in chunks.
size_t prefill_bytes(const Sizes& z, kda_dtype dtype, bool split) {
  if (z.B * z.T == 0) return 0;
  return kda::gated_delta_chunk_bytes(z.B, z.T, z.H, z.HV, z.K, z.V, z.n_seq, dtype, split);
}

size_t backward_bytes(const Sizes& z, kda_dtype dtype, bool split) {
  if (z.B * z.T == 0) return 0;
  const size_t chunk = kda::gated_delta_chunk_backward_bytes(z.B, z.T, z.H, z.HV, z.K, z.V, z.n_seq, dtype, split);
  return chunk ? chunk : kda::gated_delta_token_backward_bytes(z.B, z.T, z.H, z.HV, z.K, z.V, z.n_seq);
}

}  // namespace

extern "C" {

int kda_gated_delta_prefill_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t HV, int64_t K, int64_t V,
                                            int64_t n_seq, kda_dtype dtype, size_t* bytes) {
  const char* fn = "kda_gated_delta_prefill_workspace_bytes";
  if (!bytes) return fail(KDA_ERR_INVALID_ARG, "%s: null output", fn);
  const Sizes z{B, T, H, HV, K, V, n_seq};
  if (int rc = check_sizes(fn, dtype, z)) return rc;
  *bytes = prefill_bytes(z, dtype, true);
  return ok();
}

int kda_gated_delta_prefill(const void* q, const void* k, const void* v, kda_dtype dtype, const float* g,
                            const float* beta, const float* initial_state, float* final_state,
                            const int32_t* cu_seqlens, int64_t n_seq, int64_t B, int64_t T, int64_t H, int64_t HV,
                            int64_t K, int64_t V, const kda_layout* layout, void* o, void* workspace,
                            size_t workspace_bytes, kda_stream_t stream) {
  const char* fn = "kda_gated_delta_prefill";
  const Sizes z{B, T, H, HV, K, V, cu_seqlens ? n_seq : 0};
  if (int rc = check_sizes(fn, dtype, z)) return rc;
  if (cu_seqlens && B != 1) return fail(KDA_ERR_INVALID_ARG, "%s: cu_seqlens requires B == 1 (got %lld)", fn, (long long)B);
  const int64_t N = cu_seqlens ? n_seq : B;
  const int64_t state = N * HV * K * V;
  if (initial_state && final_state && initial_state != final_state &&
      overlap(initial_state, (size_t)state * 4, final_state, (size_t)state * 4))
    return fail(KDA_ERR_INVALID_ARG, "%s: initial_state and final_state overlap partially", fn);
  if (!aligned16(initial_state) || !aligned16(final_state) || !aligned16(workspace))
    return fail(KDA_ERR_UNSUPPORTED, "%s: states and workspace must be 16-byte aligned", fn);
  if (workspace_bytes > 0 && !workspace) return fail(KDA_ERR_INVALID_ARG, "%s: workspace_bytes > 0 with a null workspace", fn);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (N == 0) return ok();
  if (B * T == 0) {  // an empty scan: the final state is the initial one, or zeros
    const cudaError_t e = kda::launch_state_copy(initial_state, final_state, state, s);
    return e == cudaSuccess ? ok() : cuda_fail(e, fn);
  }
  kda::GatedDeltaParams p{};
  if (int rc = check_tensors(fn, dtype, z, layout, q, k, v, g, beta, o, p)) return rc;
  if (int rc = check_output(fn, z, p)) return rc;
  p.s0 = initial_state;
  p.sf = final_state;
  p.cu = cu_seqlens;
  p.N = (int)N;
  const size_t need = prefill_bytes(z, dtype, false);
  // The chunked kernels read by TMA; a layout the driver makes no tensor map of (a stride of zero) goes token by token.
  cudaError_t e = cudaErrorNotSupported;
  if (need > 0 && workspace_bytes >= need) e = kda::launch_gated_delta_chunk(p, workspace, workspace_bytes, s);
  if (e == cudaErrorNotSupported) e = kda::launch_gated_delta_token(p, dtype, s);
  return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

int kda_gated_delta_decode_step(const void* q, const void* k, const void* v, kda_dtype dtype, const float* g,
                                const float* beta, float* state, int64_t B, int64_t H, int64_t HV, int64_t K, int64_t V,
                                const kda_layout* layout, void* o, kda_stream_t stream) {
  const char* fn = "kda_gated_delta_decode_step";
  const Sizes z{B, 1, H, HV, K, V, 0};
  if (int rc = check_sizes(fn, dtype, z)) return rc;
  if (B == 0) return ok();
  if (!state) return fail(KDA_ERR_INVALID_ARG, "%s: null state", fn);
  if (!aligned16(state)) return fail(KDA_ERR_UNSUPPORTED, "%s: the state must be 16-byte aligned", fn);
  kda::GatedDeltaParams p{};
  if (int rc = check_tensors(fn, dtype, z, layout, q, k, v, g, beta, o, p)) return rc;
  if (int rc = check_output(fn, z, p)) return rc;
  p.s0 = p.sf = state;
  p.N = (int)B;
  const cudaError_t e = kda::launch_gated_delta_decode(p, dtype, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

int kda_gated_delta_backward_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t HV, int64_t K, int64_t V,
                                             int64_t n_seq, kda_dtype dtype, size_t* bytes) {
  const char* fn = "kda_gated_delta_backward_workspace_bytes";
  if (!bytes) return fail(KDA_ERR_INVALID_ARG, "%s: null output", fn);
  const Sizes z{B, T, H, HV, K, V, n_seq};
  if (int rc = check_sizes(fn, dtype, z)) return rc;
  if (!backward_dim(K) || !backward_dim(V))
    return fail(KDA_ERR_UNSUPPORTED, "%s: K and V must be 16, 32, 64 or 128 (K=%lld, V=%lld)", fn, (long long)K, (long long)V);
  *bytes = backward_bytes(z, dtype, true);
  return ok();
}

int kda_gated_delta_backward(const void* q, const void* k, const void* v, kda_dtype dtype, const float* g,
                             const float* beta, const float* initial_state, const void* d_o, const float* d_final_state,
                             const int32_t* cu_seqlens, int64_t n_seq, int64_t B, int64_t T, int64_t H, int64_t HV,
                             int64_t K, int64_t V, const kda_layout* layout, void* dq, void* dk, void* dv, float* dg,
                             float* dbeta, float* d_initial_state, void* workspace, size_t workspace_bytes,
                             kda_stream_t stream) {
  const char* fn = "kda_gated_delta_backward";
  const Sizes z{B, T, H, HV, K, V, cu_seqlens ? n_seq : 0};
  if (int rc = check_sizes(fn, dtype, z)) return rc;
  if (cu_seqlens && B != 1) return fail(KDA_ERR_INVALID_ARG, "%s: cu_seqlens requires B == 1 (got %lld)", fn, (long long)B);
  if (!backward_dim(K) || !backward_dim(V))
    return fail(KDA_ERR_UNSUPPORTED, "%s: K and V must be 16, 32, 64 or 128 (K=%lld, V=%lld)", fn, (long long)K, (long long)V);
  const int64_t N = cu_seqlens ? n_seq : B;
  const int64_t state = N * HV * K * V;
  const void* buffers[] = {initial_state, d_final_state, d_initial_state, dq, dk, dv, dg, dbeta, workspace};
  for (const void* b : buffers)
    if (!aligned16(b)) return fail(KDA_ERR_UNSUPPORTED, "%s: states, gradients and workspace must be 16-byte aligned", fn);
  if (d_initial_state && d_final_state && d_initial_state != d_final_state &&
      overlap(d_initial_state, (size_t)state * 4, d_final_state, (size_t)state * 4))
    return fail(KDA_ERR_INVALID_ARG, "%s: d_initial_state and d_final_state overlap partially", fn);
  if (d_initial_state && initial_state && overlap(d_initial_state, (size_t)state * 4, initial_state, (size_t)state * 4))
    return fail(KDA_ERR_INVALID_ARG, "%s: d_initial_state overlaps initial_state", fn);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (N == 0) return ok();
  if (B * T == 0) {  // nothing to differentiate through: dL/dS_0 = dL/dS_T
    const cudaError_t e = kda::launch_state_copy(d_final_state, d_initial_state, state, s);
    return e == cudaSuccess ? ok() : cuda_fail(e, fn);
  }
  kda::GatedDeltaParams p{};
  if (int rc = check_tensors(fn, dtype, z, layout, q, k, v, g, beta, d_o, p)) return rc;
  if (!dq || !dk || !dv || !dg || !dbeta) return fail(KDA_ERR_INVALID_ARG, "%s: null gradient pointer", fn);
  const size_t need = backward_bytes(z, dtype, false);
  if (!workspace || workspace_bytes < need)
    return fail(KDA_ERR_INVALID_ARG, "%s: the workspace needs %zu bytes (got %zu)", fn, need, workspace_bytes);
  p.s0 = initial_state;
  p.cu = cu_seqlens;
  p.N = (int)N;
  p.o = nullptr;
  const kda::GatedDeltaGrads d{d_o, d_final_state, dq, dk, dv, dg, dbeta, d_initial_state};
  const bool chunked = kda::gated_delta_chunk_backward_bytes(B, T, H, HV, K, V, z.n_seq, dtype, false) > 0;
  const cudaError_t e = chunked ? kda::launch_gated_delta_chunk_backward(p, d, workspace, workspace_bytes, s)
                                : kda::launch_gated_delta_token_backward(p, d, workspace, s);
  if (e == cudaErrorNotSupported)  // nothing was launched
    return fail(KDA_ERR_UNSUPPORTED, "%s: the driver makes no tensor map of these strides (a stride of zero?)", fn);
  return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

// ---------------------------------------------------------------------------------------------------------------------

static int check_norm(const char* fn, kda_dtype dtype, kda_dtype weight_dtype, int64_t rows, int64_t D) {
  if (rows < 0 || D <= 0) return fail(KDA_ERR_INVALID_ARG, "%s: rows must not be negative and D must be positive", fn);
  if ((dtype != KDA_F32 && dtype != KDA_BF16) || (weight_dtype != KDA_F32 && weight_dtype != KDA_BF16))
    return fail(KDA_ERR_INVALID_ARG, "%s: unknown dtype", fn);
  if (dtype == KDA_F32 && weight_dtype != KDA_F32)
    return fail(KDA_ERR_UNSUPPORTED, "%s: fp32 rows take fp32 weights", fn);
  if (D > kda::LAYER_NORM_MAX_D)
    return fail(KDA_ERR_UNSUPPORTED, "%s: D must be at most %d (got %lld)", fn, kda::LAYER_NORM_MAX_D, (long long)D);
  return KDA_OK;
}

// Whether `rows` contiguous rows at y meet the rows of x, `stride` elements apart, anywhere but where y is x.
static bool rows_clash(const void* y, const void* x, int64_t stride, int64_t rows, int64_t D, kda_dtype dt) {
  const int64_t es = dt == KDA_F32 ? 4 : 2, width = D * es, step = stride * es;
  if (y == x && (stride == D || rows == 1)) return false;
  if (!overlap(y, (size_t)(rows * width), x, (size_t)((rows - 1) * step + width))) return false;
  const int64_t off = static_cast<const char*>(y) - static_cast<const char*>(x);
  return !(step > width && off > 0 && off % step >= width && off % step + rows * width <= step);  // between two rows
}

static bool aligned_to(const void* p, kda_dtype dt) { return reinterpret_cast<uintptr_t>(p) % (dt == KDA_F32 ? 4 : 2) == 0; }

int kda_layer_norm(const void* x, int64_t x_stride, kda_dtype dtype, const void* weight, const void* bias,
                   kda_dtype weight_dtype, float eps, int64_t rows, int64_t D, void* y, float* mean, float* rstd,
                   kda_stream_t stream) {
  const char* fn = "kda_layer_norm";
  if (int rc = check_norm(fn, dtype, weight_dtype, rows, D)) return rc;
  if (!std::isfinite(eps) || eps < 0.f) return fail(KDA_ERR_INVALID_ARG, "%s: eps must be finite and not negative", fn);
  if (rows == 0) return ok();
  if (!x || !y || !mean || !rstd) return fail(KDA_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (x_stride < 0) return fail(KDA_ERR_INVALID_ARG, "%s: negative stride", fn);
  if (!aligned_to(x, dtype) || !aligned_to(y, dtype) || !aligned_to(weight, weight_dtype) ||
      !aligned_to(bias, weight_dtype) || !aligned_to(mean, KDA_F32) || !aligned_to(rstd, KDA_F32))
    return fail(KDA_ERR_UNSUPPORTED, "%s: misaligned pointer", fn);
  if (rows_clash(y, x, x_stride, rows, D, dtype)) return fail(KDA_ERR_INVALID_ARG, "%s: y and x overlap partially", fn);
  kda::LayerNormParams p{};
  p.x = x;
  p.weight = weight;
  p.bias = bias;
  p.y = y;
  p.mean = mean;
  p.rstd = rstd;
  p.rows = rows;
  p.x_stride = x_stride;
  p.D = (int)D;
  p.eps = eps;
  const cudaError_t e = kda::launch_layer_norm(p, dtype, weight_dtype, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

int kda_layer_norm_backward_workspace_bytes(int64_t rows, int64_t D, size_t* bytes) {
  const char* fn = "kda_layer_norm_backward_workspace_bytes";
  if (!bytes) return fail(KDA_ERR_INVALID_ARG, "%s: null output", fn);
  if (int rc = check_norm(fn, KDA_F32, KDA_F32, rows, D)) return rc;
  *bytes = rows == 0 ? 0 : (size_t)kda::layer_norm_parts(rows, (int)D) * 2 * (size_t)D * sizeof(float);
  return ok();
}

int kda_layer_norm_backward(const void* d_y, int64_t d_y_stride, const void* x, int64_t x_stride, kda_dtype dtype,
                            const void* weight, kda_dtype weight_dtype, const float* mean, const float* rstd, int64_t rows,
                            int64_t D, void* dx, void* dweight, void* dbias, void* workspace, size_t workspace_bytes,
                            kda_stream_t stream) {
  const char* fn = "kda_layer_norm_backward";
  if (int rc = check_norm(fn, dtype, weight_dtype, rows, D)) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!aligned_to(d_y, dtype) || !aligned_to(x, dtype) || !aligned_to(dx, dtype) || !aligned_to(weight, weight_dtype) ||
      !aligned_to(dweight, weight_dtype) || !aligned_to(dbias, weight_dtype) || !aligned_to(mean, KDA_F32) ||
      !aligned_to(rstd, KDA_F32) || !aligned16(workspace))
    return fail(KDA_ERR_UNSUPPORTED, "%s: misaligned pointer", fn);
  if (rows == 0) {  // sums over no rows
    cudaError_t e = cudaSuccess;
    const size_t bytes = (size_t)D * (weight_dtype == KDA_F32 ? 4 : 2);
    if (dweight) e = cudaMemsetAsync(dweight, 0, bytes, s);
    if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, bytes, s);
    return e == cudaSuccess ? ok() : cuda_fail(e, fn);
  }
  if (!d_y || !x || !mean || !rstd || !dx) return fail(KDA_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (x_stride < 0 || d_y_stride < 0) return fail(KDA_ERR_INVALID_ARG, "%s: negative stride", fn);
  if (rows_clash(dx, x, x_stride, rows, D, dtype) || rows_clash(dx, d_y, d_y_stride, rows, D, dtype))
    return fail(KDA_ERR_INVALID_ARG, "%s: dx overlaps x or d_y partially", fn);
  kda::LayerNormParams p{};
  if (dweight || dbias) {
    const size_t need = (size_t)kda::layer_norm_parts(rows, (int)D) * 2 * (size_t)D * sizeof(float);
    if (!workspace || workspace_bytes < need)
      return fail(KDA_ERR_INVALID_ARG, "%s: the workspace needs %zu bytes (got %zu)", fn, need, workspace_bytes);
    p.parts = static_cast<float*>(workspace);
  }
  p.x = x;
  p.weight = weight;
  p.dy = d_y;
  p.dx = dx;
  p.dweight = dweight;
  p.dbias = dbias;
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  p.rows = rows;
  p.x_stride = x_stride;
  p.dy_stride = d_y_stride;
  p.D = (int)D;
  const cudaError_t e = kda::launch_layer_norm(p, dtype, weight_dtype, s);
  return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

}  // extern "C"
