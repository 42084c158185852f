// decay_api.cu -- the C ABI (include/kata.h) of linear attention with a
// per-head decay and of the 8-bit state cache: argument checks and launches.
#include "kata_internal.h"

#define KATA_API extern "C" __attribute__((visibility("default")))

namespace kata {
namespace {

bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
kata_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? KATA_OK : KATA_ERR_CUDA; }
bool width_ok(int w) { return w == 64 || w == 128; }

// Sizes that fit the grids and the 32-bit token and index arithmetic.
constexpr int kMaxTokens = 1 << 30, kMaxSequences = 1 << 20, kMaxHeads = 4096;
constexpr long long kMaxStride = 1ll << 36;  // elements; a tensor map's stride is below 2^40 bytes
// Every CTA of a walk looks for its sequence from the first on, 32 at a time, and with slots every CTA of a step for
// an earlier stream of its slot, so that a call's time grows with their square: 16384 sequences of 16 heads take
// 0.29 s, 32768 streams of 16 heads and dv = 64 26 ms (2.6 ms without slots).  A million of either would hold the
// GPU for many minutes.  At these bounds the search takes 2.4 and 1.5 s.
constexpr long long kMaxWalkSearch = 1ll << 35, kMaxStepSearch = 1ll << 41;

kata_status_t check_shape(int T, int H, int d, int dv, int N, kata_dtype_t dt, int walks) {
  if (T < 0 || H < 1 || N < 0) return KATA_ERR_INVALID_ARG;
  if (dt != KATA_BF16 && dt != KATA_F32) return KATA_ERR_INVALID_ARG;
  if (!width_ok(d) || !width_ok(dv)) return KATA_ERR_UNSUPPORTED;
  if (T > kMaxTokens || N > kMaxSequences || H > kMaxHeads) return KATA_ERR_UNSUPPORTED;
  // one CTA per segment, head and walk, and up to 16 for the scan of a split sequence, with at least 256 tokens to
  // a segment
  if (((long long)T / 256 * 16 + N) * H * 3 > 0x7fffffffll) return KATA_ERR_UNSUPPORTED;
  if ((long long)N * N * H * walks > kMaxWalkSearch) return KATA_ERR_UNSUPPORTED;
  return KATA_OK;
}

kata_status_t check_stride(long long stride, int H, int width, int unit) {
  if (stride < (long long)H * width) return KATA_ERR_INVALID_ARG;
  if (stride > kMaxStride) return KATA_ERR_UNSUPPORTED;
  return stride % unit ? KATA_ERR_MISALIGNED : KATA_OK;
}

kata_status_t check_workspace(size_t need, const void* ws, size_t bytes) {
  if (need == 0) return KATA_OK;
  if (!ws || bytes < need) return KATA_ERR_WORKSPACE;
  return aligned(ws, 256) ? KATA_OK : KATA_ERR_MISALIGNED;
}

bool overlap(const float* a, const float* b, size_t n) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + n * sizeof(float) && y < x + n * sizeof(float);
}

}  // namespace
}  // namespace kata

using namespace kata;

KATA_API size_t kata_fwd_linear_decay_workspace_size(int T, int H, int d, int dv, int N) {
  if (check_shape(T, H, d, dv, N, KATA_BF16, 1) != KATA_OK || T == 0 || N == 0) return 0;
  return decay_workspace_bytes(T, H, d, dv, N, 1);
}

KATA_API kata_status_t kata_fwd_linear_decay(const void* q, const void* k, const void* v, void* o, int T, int H, int d,
                                             int dv, long long q_stride, long long k_stride, long long v_stride,
                                             long long o_stride, const float* log_decay, float scale,
                                             const int* cu_seqlens, int N, const float* S0, float* S_out,
                                             const int* slots, int n_slots, const unsigned char* resume,
                                             int zero_outside, kata_dtype_t dtype, void* workspace,
                                             size_t workspace_bytes, void* stream) {
  kata_status_t s = check_shape(T, H, d, dv, N, dtype, 1);
  if (s != KATA_OK) return s;
  if (dtype != KATA_BF16) return KATA_ERR_UNSUPPORTED;
  if (!cu_seqlens && N != 1) return KATA_ERR_INVALID_ARG;
  if (n_slots < 0 || ((S0 || S_out) && !slots && n_slots < N)) return KATA_ERR_INVALID_ARG;
  if (N == 0 || (T == 0 && !S_out)) {
    // no sequence: every row of o is outside
    if (!zero_outside || T == 0) return KATA_OK;
    if (!o) return KATA_ERR_INVALID_ARG;
    if ((s = check_stride(o_stride, H, dv, 8)) != KATA_OK) return s;
    return from_cuda(cudaMemset2DAsync(o, (size_t)o_stride * 2, 0, (size_t)H * dv * 2, T,
                                       static_cast<cudaStream_t>(stream)));
  }
  if (!log_decay) return KATA_ERR_INVALID_ARG;
  for (const void* p : {(const void*)S0, (const void*)S_out})
    if (!aligned(p, 16)) return KATA_ERR_MISALIGNED;
  for (const void* p : {(const void*)log_decay, (const void*)cu_seqlens, (const void*)slots})
    if (!aligned(p, 4)) return KATA_ERR_MISALIGNED;
  // without slots the call's states are the first N of either pool
  if (S0 != S_out && overlap(S0, S_out, (size_t)(slots ? n_slots : N) * H * d * dv)) return KATA_ERR_INVALID_ARG;
  const DecayWalk w{q, k, v, o, q_stride, k_stride, v_stride, o_stride, d, dv, false, S0, false, S_out};
  const DecayShape sh{T, H, N, cu_seqlens, log_decay, scale, slots, n_slots, resume, zero_outside != 0};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) return from_cuda(launch_decay_empty(w, sh, wait_ctl(), st));
  if (!q || !k || !v || !o) return KATA_ERR_INVALID_ARG;
  for (const void* p : {q, k, v, (const void*)o})
    if (!aligned(p, 16)) return KATA_ERR_MISALIGNED;
  if ((s = check_stride(q_stride, H, d, 8)) != KATA_OK || (s = check_stride(k_stride, H, d, 8)) != KATA_OK ||
      (s = check_stride(v_stride, H, dv, 8)) != KATA_OK || (s = check_stride(o_stride, H, dv, 8)) != KATA_OK)
    return s;
  if ((s = check_workspace(decay_workspace_bytes(T, H, d, dv, N, 1), workspace, workspace_bytes)) != KATA_OK) return s;
  return from_cuda(launch_decay_walks(&w, 1, sh, workspace, wait_ctl(), st));
}

KATA_API size_t kata_bwd_linear_decay_workspace_size(int T, int H, int d, int dv, int N) {
  if (check_shape(T, H, d, dv, N, KATA_BF16, 3) != KATA_OK || T == 0 || N == 0) return 0;
  return decay_workspace_bytes(T, H, d, dv, N, 3);
}

KATA_API kata_status_t kata_bwd_linear_decay(const void* q, const void* k, const void* v, const void* dO, void* dq,
                                             void* dk, void* dv, int T, int H, int d, int dv_width,
                                             long long q_stride, long long k_stride, long long v_stride,
                                             const float* log_decay, float scale, const int* cu_seqlens, int N,
                                             const float* S0, const float* dS_out, float* dS0, kata_dtype_t dtype,
                                             void* workspace, size_t workspace_bytes, void* stream) {
  kata_status_t s = check_shape(T, H, d, dv_width, N, dtype, 3);
  if (s != KATA_OK) return s;
  if (dtype != KATA_BF16) return KATA_ERR_UNSUPPORTED;
  if (!cu_seqlens && N != 1) return KATA_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const long long ck = (long long)H * d, cv = (long long)H * dv_width;
  if (N == 0) {
    if (T == 0) return KATA_OK;
    if (!dq || !dk || !dv) return KATA_ERR_INVALID_ARG;
    cudaError_t e = cudaMemsetAsync(dq, 0, (size_t)T * ck * 2, st);
    if (e == cudaSuccess) e = cudaMemsetAsync(dk, 0, (size_t)T * ck * 2, st);
    if (e == cudaSuccess) e = cudaMemsetAsync(dv, 0, (size_t)T * cv * 2, st);
    return from_cuda(e);
  }
  if (T == 0 && !dS0) return KATA_OK;
  if (!log_decay) return KATA_ERR_INVALID_ARG;
  for (const void* p : {(const void*)S0, (const void*)dS_out, (const void*)dS0})
    if (!aligned(p, 16)) return KATA_ERR_MISALIGNED;
  for (const void* p : {(const void*)log_decay, (const void*)cu_seqlens})
    if (!aligned(p, 4)) return KATA_ERR_MISALIGNED;
  const size_t states = (size_t)N * H * d * dv_width;
  if (overlap(S0, dS0, states) || overlap(dS_out, dS0, states)) return KATA_ERR_INVALID_ARG;
  const DecayShape sh{T, H, N, cu_seqlens, log_decay, scale, nullptr, N, nullptr, true};
  const DecayWalk walks[3] = {
      {dO, v, k, dq, cv, v_stride, k_stride, ck, dv_width, d, false, S0, true, nullptr},
      {v, dO, q, dk, v_stride, cv, q_stride, ck, dv_width, d, true, dS_out, true, nullptr},
      {k, q, dO, dv, k_stride, q_stride, cv, cv, d, dv_width, true, dS_out, false, dS0},
  };
  if (T == 0) return from_cuda(launch_decay_empty(walks[2], sh, wait_ctl(), st));
  if (!q || !k || !v || !dO || !dq || !dk || !dv) return KATA_ERR_INVALID_ARG;
  for (const void* p : {q, k, v, dO, (const void*)dq, (const void*)dk, (const void*)dv})
    if (!aligned(p, 16)) return KATA_ERR_MISALIGNED;
  if ((s = check_stride(q_stride, H, d, 8)) != KATA_OK || (s = check_stride(k_stride, H, d, 8)) != KATA_OK ||
      (s = check_stride(v_stride, H, dv_width, 8)) != KATA_OK)
    return s;
  if ((s = check_workspace(decay_workspace_bytes(T, H, d, dv_width, N, 3), workspace, workspace_bytes)) != KATA_OK)
    return s;
  return from_cuda(launch_decay_walks(walks, 3, sh, workspace, wait_ctl(), st));
}

KATA_API kata_status_t kata_decode_step_linear_decay(const void* q, const void* k, const void* v, void* o, float* S,
                                                     int n, int H, int d, int dv, long long q_stride,
                                                     long long k_stride, long long v_stride, long long o_stride,
                                                     const float* log_decay, float scale, const int* slots,
                                                     int n_slots, kata_dtype_t dtype, void* stream) {
  kata_status_t s = check_shape(0, H, d, dv, n, dtype, 0);
  if (s != KATA_OK) return s;
  if ((long long)n * H * (dv / 32) > 0x7fffffffll) return KATA_ERR_UNSUPPORTED;
  if (slots && (long long)n * n * H * (dv / 32) > kMaxStepSearch) return KATA_ERR_UNSUPPORTED;
  if (n_slots < 0 || (!slots && n_slots < n)) return KATA_ERR_INVALID_ARG;
  if (n == 0) return KATA_OK;
  if (!q || !k || !v || !o || (!S && n_slots > 0) || !log_decay) return KATA_ERR_INVALID_ARG;
  for (const void* p : {q, k, v, (const void*)o, (const void*)S})
    if (!aligned(p, 16)) return KATA_ERR_MISALIGNED;
  if (!aligned(log_decay, 4) || !aligned(slots, 4)) return KATA_ERR_MISALIGNED;
  const int unit = dtype == KATA_BF16 ? 8 : 4;
  if ((s = check_stride(q_stride, H, d, unit)) != KATA_OK || (s = check_stride(k_stride, H, d, unit)) != KATA_OK ||
      (s = check_stride(v_stride, H, dv, unit)) != KATA_OK || (s = check_stride(o_stride, H, dv, unit)) != KATA_OK)
    return s;
  return from_cuda(launch_decay_step(q, k, v, o, S, n, H, d, dv, q_stride, k_stride, v_stride, o_stride, log_decay,
                                     scale, slots, n_slots, dtype, wait_ctl(), static_cast<cudaStream_t>(stream)));
}

static kata_status_t check_q8(const void* S, const void* z, const void* cache, const void* scale, const void* z_cache,
                              int n_slots, int n_entries, const int* slots, const int* entries, int n, int H, int rows,
                              int dv) {
  if (n < 0 || n_slots < 0 || n_entries < 0 || H < 1 || rows < 1) return KATA_ERR_INVALID_ARG;
  if (dv != 16 && dv != 64 && dv != 128) return KATA_ERR_UNSUPPORTED;
  // one grid row per pair, and tiles of 64 or more of the H * rows rows along the other axis
  if (n > 65535 || (long long)H * rows > (1ll << 30)) return KATA_ERR_UNSUPPORTED;
  if ((z == nullptr) != (z_cache == nullptr)) return KATA_ERR_INVALID_ARG;
  if ((!slots && n > n_slots) || (!entries && n > n_entries)) return KATA_ERR_INVALID_ARG;
  if (n == 0) return KATA_OK;
  if ((!S && n_slots > 0) || ((!cache || !scale) && n_entries > 0)) return KATA_ERR_INVALID_ARG;
  if (!aligned(S, 16) || !aligned(cache, 4)) return KATA_ERR_MISALIGNED;
  for (const void* p : {z, scale, z_cache, (const void*)slots, (const void*)entries})
    if (!aligned(p, 4)) return KATA_ERR_MISALIGNED;
  return KATA_OK;
}

KATA_API kata_status_t kata_state_store_q8(const float* S, const float* z, int n_slots, signed char* cache,
                                           float* scale, float* z_cache, int n_entries, const int* slots,
                                           const int* entries, int n, int H, int rows, int dv, void* stream) {
  const kata_status_t s = check_q8(S, z, cache, scale, z_cache, n_slots, n_entries, slots, entries, n, H, rows, dv);
  if (s != KATA_OK || n == 0) return s;
  return from_cuda(launch_state_store_q8(S, z, n_slots, cache, scale, z_cache, n_entries, slots, entries, n,
                                         (long long)H * rows, dv, wait_ctl(), static_cast<cudaStream_t>(stream)));
}

KATA_API kata_status_t kata_state_load_q8(const signed char* cache, const float* scale, const float* z_cache,
                                          int n_entries, float* S, float* z, int n_slots, const int* entries,
                                          const int* slots, int n, int H, int rows, int dv, void* stream) {
  const kata_status_t s = check_q8(S, z, cache, scale, z_cache, n_slots, n_entries, slots, entries, n, H, rows, dv);
  if (s != KATA_OK || n == 0) return s;
  return from_cuda(launch_state_load_q8(cache, scale, z_cache, n_entries, S, z, n_slots, entries, slots, n,
                                        (long long)H * rows, dv, wait_ctl(), static_cast<cudaStream_t>(stream)));
}
