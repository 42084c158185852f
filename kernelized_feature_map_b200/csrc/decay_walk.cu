// decay_walk.cu -- linear attention with a per-head decay over packed
// sequences, token by token: the plainest form of the walk (kata_internal.h).
//
// One CTA per sequence, head and walk; the state is in registers, 16 x 16
// threads with a (d1/16) x (d2/16) tile each.
#include "decay_common.cuh"
#include "kata_internal.h"

namespace kata {
namespace {

constexpr int kThreads = 256;

template <int D1, int D2>
__global__ void __launch_bounds__(kThreads) decay_walk_kernel(const DecayWalk w, const DecayShape sh, int* status) {
  constexpr int R = D1 / 16, C = D2 / 16;
  __shared__ float sa[D1], sb[D1], sc[D2];
  __shared__ float red[16][D2];
  __shared__ int found[8];
  const int tid = threadIdx.x, lane = tid & 31, tr = tid / 16, tc = tid % 16;
  const int h = blockIdx.x % sh.H, n = blockIdx.x / sh.H;
  if (tid < 32) {
    bool valid;
    const Segment g = find_segment(sh.cu, sh.N, sh.T, max(sh.T, 1), n, lane, valid);
    const int row =
        w.init || w.fin ? pool_row(sh.slots, g.seq, sh.n_slots, w.fin != nullptr, lane, status) : -1;
    if (tid == 0) {
      if (!valid) report_status(status, kStatusInvalidArg);
      found[0] = g.s0;
      found[1] = g.s1;
      found[2] = row;
    }
  }
  __syncthreads();
  const int s0 = found[0], s1 = found[1], row = found[2];
  float hi, lo;
  decay_factor(used_log_decay(sh.log_decay[h], status), hi, lo);
  const bool entered = w.init && row >= 0 && (!sh.resume || sh.resume[n]);
  const long long base = ((long long)row * sh.H + h) * D1 * D2;
  float S[R][C];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int r = tr * R + i, c = tc * C + j;
      S[i][j] = entered ? w.init[base + (w.init_transposed ? c * D1 + r : r * D2 + c)] : 0.f;
    }
  using B = __nv_bfloat16;
  // forward: out = scale * A S, the state unscaled; reversed: the state is the
  // gradient R, whose terms carry the scale and whose entering value does not
  const float s_in = w.reverse ? sh.scale : 1.f, s_out = w.reverse ? 1.f : sh.scale;
  for (int x = 0; x < s1 - s0; ++x) {
    const long long t = w.reverse ? s1 - 1 - x : s0 + x;
    if (tid < D1) {
      sa[tid] = Elem<B>::load(static_cast<const B*>(w.a) + t * w.a_stride + h * D1 + tid);
      sb[tid] = Elem<B>::load(static_cast<const B*>(w.b) + t * w.b_stride + h * D1 + tid);
    }
    if (tid < D2) sc[tid] = Elem<B>::load(static_cast<const B*>(w.c) + t * w.c_stride + h * D2 + tid);
    __syncthreads();
    // reversed, the entering state is already that of the last token
    const float keep = w.reverse && x == 0 ? 1.f : hi, rest = w.reverse && x == 0 ? 0.f : lo;
    float acc[C] = {};
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < C; ++j) {
        S[i][j] = fmaf(keep, S[i][j], fmaf(rest, S[i][j], s_in * sb[tr * R + i] * sc[tc * C + j]));
        acc[j] = fmaf(sa[tr * R + i], S[i][j], acc[j]);
      }
#pragma unroll
    for (int j = 0; j < C; ++j) red[tr][tc * C + j] = acc[j];
    __syncthreads();
    if (tid < D2) {
      float o = 0.f;
      for (int i = 0; i < 16; ++i) o += red[i][tid];
      Elem<B>::store(static_cast<B*>(w.out) + t * w.out_stride + h * D2 + tid, s_out * o);
    }
  }
  if (w.fin && row >= 0) {
    const float last = w.reverse && s1 > s0 ? hi : 1.f;  // to before the first token
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < C; ++j) w.fin[base + (tr * R + i) * D2 + tc * C + j] = last * S[i][j];
  }
  if (sh.zero_outside) {
    const long long t0 = n == 0 ? 0 : s1, t1 = n == 0 ? s0 : s1;
    for (long long t = t0; t < t1; ++t)
      if (tid < D2) Elem<B>::store(static_cast<B*>(w.out) + t * w.out_stride + h * D2 + tid, 0.f);
    if (n == sh.N - 1)
      for (long long t = s1; t < sh.T; ++t)
        if (tid < D2) Elem<B>::store(static_cast<B*>(w.out) + t * w.out_stride + h * D2 + tid, 0.f);
  }
}

}  // namespace

size_t decay_workspace_bytes(int T, int H, int d1, int d2, int N, int walks) { return 0; }

cudaError_t launch_decay_walks(const DecayWalk* walks, int n, const DecayShape& sh, void* ws, const WaitCtl& wc,
                               cudaStream_t st) {
  for (int i = 0; i < n; ++i) {
    const DecayWalk& w = walks[i];
    const unsigned grid = (unsigned)sh.N * sh.H;
    if (w.d1 == 64 && w.d2 == 64) decay_walk_kernel<64, 64><<<grid, kThreads, 0, st>>>(w, sh, wc.status);
    else if (w.d1 == 64) decay_walk_kernel<64, 128><<<grid, kThreads, 0, st>>>(w, sh, wc.status);
    else if (w.d2 == 64) decay_walk_kernel<128, 64><<<grid, kThreads, 0, st>>>(w, sh, wc.status);
    else decay_walk_kernel<128, 128><<<grid, kThreads, 0, st>>>(w, sh, wc.status);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// Sequences of no tokens at all: T = 0 makes every range empty.
cudaError_t launch_decay_empty(const DecayWalk& w, const DecayShape& sh, const WaitCtl& wc, cudaStream_t st) {
  return w.fin ? launch_decay_walks(&w, 1, sh, nullptr, wc, st) : cudaSuccess;
}

}  // namespace kata
