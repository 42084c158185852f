// decay_step.cu -- one token of linear attention with a per-head decay:
//
//   S <- a S + k v^T,   o = scale * q^T S        (S [d, dv] fp32, in place)
//
// Bound by HBM: the state is read and written once, 8 d dv bytes per stream
// and head, against 5 d dv operations.  The value columns are independent of
// one another, so a CTA takes a slab of 32 columns (rows of 128 bytes, one
// DRAM line) of one stream and head: a single stream of 16 heads with
// dv = 128 is 64 CTAs, and a large batch keeps ~16 CTAs of 128 threads with
// all of their slab's loads in flight on every SM.  Eight lanes cover a row
// of the slab with 16-byte vectors; the sum over rows that gives o goes
// through shuffles and one shared-memory pass.
//
// Measured (other pools in between): 512 streams, 16 heads, d = dv = 128 1.07 GB in
// 160 us, 6.7 TB/s (as a plain copy); 64 streams 23.2 us, 5.8 TB/s; 333 streams, 8
// heads, d = 64, fp32 29.1 us, 5.8 TB/s; a single stream 2.7 us, a launch's latency
// (4.4 to 4.9 us a call, the host's part).
#include "decay_common.cuh"
#include "kata_internal.h"

namespace kata {
namespace {

constexpr int kThreads = 128;
constexpr int kSlab = 32;                      // value columns of a CTA
constexpr int kLanes = kSlab / 4;              // lanes per row
constexpr int kRowsPerPass = kThreads / kLanes;  // 16

struct StepArgs {
  const void *q, *k, *v;
  void* o;
  float* S;
  int H, dv, n_slots;
  long long q_stride, k_stride, v_stride, o_stride;  // elements
  const float* log_decay;
  float scale;
  const int* slots;
  int* status;
};

template <typename Tin, int D>
__global__ void __launch_bounds__(kThreads) decay_step_kernel(const StepArgs a) {
  constexpr int kPasses = D / kRowsPerPass;
  __shared__ float sq[D], sk[D];
  __shared__ float4 red[kThreads / 32][kLanes];
  griddep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slabs = a.dv / kSlab;
  const int slab = blockIdx.x % slabs, h = blockIdx.x / slabs % a.H, i = blockIdx.x / slabs / a.H;
  const int cg = tid % kLanes, r0 = tid / kLanes;
  const int col = slab * kSlab + 4 * cg;
  Tin* o = static_cast<Tin*>(a.o) + i * a.o_stride + (long long)h * a.dv + col;

  const int slot = pool_row(a.slots, i, a.n_slots, true, lane, a.status);
  if (slot < 0) {
    if (tid < kLanes)
#pragma unroll
      for (int e = 0; e < 4; ++e) Elem<Tin>::store(o + e, 0.f);
    return;
  }
  float4* Sb = reinterpret_cast<float4*>(a.S + ((long long)slot * a.H + h) * D * a.dv + col);
  const int ld = a.dv / 4;
  float4 s[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) s[p] = __ldcs(Sb + (r0 + p * kRowsPerPass) * ld);
  const Tin* q = static_cast<const Tin*>(a.q) + i * a.q_stride + (long long)h * D;
  const Tin* k = static_cast<const Tin*>(a.k) + i * a.k_stride + (long long)h * D;
  const Tin* v = static_cast<const Tin*>(a.v) + i * a.v_stride + (long long)h * a.dv + col;
  if (tid < D) {
    sq[tid] = Elem<Tin>::load(q + tid);
    sk[tid] = Elem<Tin>::load(k + tid);
  }
  float hi, lo;
  decay_factor(used_log_decay(a.log_decay[h], a.status), hi, lo);
  const float4 vv = make_float4(Elem<Tin>::load(v), Elem<Tin>::load(v + 1), Elem<Tin>::load(v + 2),
                                Elem<Tin>::load(v + 3));
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int r = r0 + p * kRowsPerPass;
    const float kr = sk[r], qr = sq[r];
    float4 n;
    n.x = fmaf(hi, s[p].x, fmaf(lo, s[p].x, kr * vv.x));
    n.y = fmaf(hi, s[p].y, fmaf(lo, s[p].y, kr * vv.y));
    n.z = fmaf(hi, s[p].z, fmaf(lo, s[p].z, kr * vv.z));
    n.w = fmaf(hi, s[p].w, fmaf(lo, s[p].w, kr * vv.w));
    __stcs(Sb + r * ld, n);
    acc.x = fmaf(qr, n.x, acc.x);
    acc.y = fmaf(qr, n.y, acc.y);
    acc.z = fmaf(qr, n.z, acc.z);
    acc.w = fmaf(qr, n.w, acc.w);
  }
#pragma unroll
  for (int m = kLanes; m < 32; m <<= 1) {
    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, m);
    acc.y += __shfl_xor_sync(0xffffffffu, acc.y, m);
    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, m);
    acc.w += __shfl_xor_sync(0xffffffffu, acc.w, m);
  }
  if (lane < kLanes) red[warp][lane] = acc;
  __syncthreads();
  if (tid < kLanes) {
    float4 t = red[0][tid];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) {
      t.x += red[w][tid].x;
      t.y += red[w][tid].y;
      t.z += red[w][tid].z;
      t.w += red[w][tid].w;
    }
    Elem<Tin>::store(o, a.scale * t.x);
    Elem<Tin>::store(o + 1, a.scale * t.y);
    Elem<Tin>::store(o + 2, a.scale * t.z);
    Elem<Tin>::store(o + 3, a.scale * t.w);
  }
}

}  // namespace

cudaError_t launch_decay_step(const void* q, const void* k, const void* v, void* o, float* S, int n, int H, int d,
                              int dv, long long q_stride, long long k_stride, long long v_stride, long long o_stride,
                              const float* log_decay, float scale, const int* slots, int n_slots, kata_dtype_t dt,
                              const WaitCtl& wc, cudaStream_t st) {
  const StepArgs a{q, k, v, o, S, H, dv, n_slots, q_stride, k_stride, v_stride, o_stride, log_decay, scale, slots,
                   wc.status};
  const unsigned grid = (unsigned)n * H * (dv / kSlab);
  auto run = [&](auto kernel) { return launch_pdl(kernel, dim3(grid), dim3(kThreads), 0, st, a); };
  if (dt == KATA_BF16) return d == 64 ? run(decay_step_kernel<__nv_bfloat16, 64>) : run(decay_step_kernel<__nv_bfloat16, 128>);
  return d == 64 ? run(decay_step_kernel<float, 64>) : run(decay_step_kernel<float, 128>);
}

}  // namespace kata
