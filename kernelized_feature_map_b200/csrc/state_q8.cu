// state_q8.cu -- pools of fp32 states to and from an 8-bit cache.
//
// A state row x (dv values) is held as integers c_j in [-127, 127] and one
// fp32 scale = max|x| / 127:  c_j = round(x_j / scale), ties to even.  The
// error of a value is at most scale / 2, the same over the whole row, which
// for the rows of accumulated products (values of like size) is nearer than
// a 3-bit mantissa holds them.
//
// Both directions are bound by HBM: 4 bytes one way and 1 the other per
// value.  A row is covered by dv/4 consecutive lanes with one 16-byte vector
// each, so a warp's load is 512 contiguous bytes of the pool and its store
// 128 of the cache; a thread has kUnroll of them in flight before it uses
// the first.  The slots of one index pair are contiguous (H * rows rows), so
// a CTA takes one pair and kTileRows of its rows.
//
// Measured (16 heads of [128 x 128], other pools in between): 256 pairs 338 MB,
// store 55 us, 6.1 TB/s, load 52 us, 6.4 TB/s (94 and 99% of a plain copy's rate);
// 48 pairs 63 MB 13.5 and 12.3 us (one wave and a half of CTAs, whose start and end
// count); one pair 3.3 and 2.9 us, a launch's latency.
#include <float.h>

#include "decay_common.cuh"
#include "kata_internal.h"

namespace kata {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 8;

template <int DV>
struct Q8 {
  static constexpr int kLanes = DV / 4;                              // lanes per row
  static constexpr int kRowsPerPass = kThreads / kLanes;
  static constexpr int kTileRows = kRowsPerPass * kUnroll;
};

// max / 127 rounded to nearest, for the scale of a row.  s0 = max * RN(1/127) is
// within one unit of the quotient and max - 127 s0 is exact, so one more step
// rounds correctly (P. Markstein, IBM J. Res. Dev. 34, 1990); a general division
// in every lane cost a third of the kernel.
__device__ __forceinline__ float row_scale(float max) {
  constexpr float kInv = 1.f / 127.f;
  const float s0 = max * kInv;
  return fmaf(fmaf(-127.f, s0, max), kInv, s0);
}

// The integers nearest to x / s, ties to even, in the low bytes of t, for
// |x| <= 127 s (1 + 2^-24) and s >= 2^-126.  Added to 1.5 2^23, x / s (times an
// approximate 1 / s) is rounded to an integer q; the remainder x - q s has no
// more than 24 bits, so the fma gives it exactly, and below s / 2 it proves q the
// nearest.  Otherwise, next to a border, q is one off or x / s a tie.  Twice the
// remainder is compared with s: half of an odd s below 2^-125 is no fp32 value.
constexpr float kMagic = 12582912.f;
struct Rounded {
  float t, r2;  // r2: twice the remainder
  __device__ __forceinline__ Rounded(float x, float s, float inv) {
    t = fmaf(x, inv, kMagic);
    r2 = 2.f * fmaf(-(t - kMagic), s, x);
  }
  __device__ __forceinline__ void settle(float s) {
    const float a = fabsf(r2);
    if (a > s || (a == s && (__float_as_uint(t) & 1u))) t += r2 > 0.f ? 1.f : -1.f;
  }
};

// Largest of m over the kLanes lanes of this lane's row.
template <int kLanes>
__device__ __forceinline__ unsigned row_max(unsigned m) {
  if constexpr (kLanes == 32) return __reduce_max_sync(0xffffffffu, m);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// The pair of this CTA: pool row and cache entry, false when it is skipped.
__device__ __forceinline__ bool find_pair(const int* src_idx, int n_src, const int* dst_idx, int n_dst, int i,
                                          int* status, int& src, int& dst) {
  __shared__ int found[2];
  if (threadIdx.x < 32) {
    const int a = pool_row(src_idx, i, n_src, false, threadIdx.x, status);
    const int b = pool_row(dst_idx, i, n_dst, true, threadIdx.x, status);
    if (threadIdx.x == 0) {
      found[0] = a;
      found[1] = b;
    }
  }
  __syncthreads();
  src = found[0];
  dst = found[1];
  return src >= 0 && dst >= 0;
}

template <int DV>
__global__ void __launch_bounds__(kThreads)
    state_store_q8_kernel(const float* __restrict__ S, const float* __restrict__ z, int n_slots,
                          int8_t* __restrict__ cache, float* __restrict__ scale, float* __restrict__ z_cache,
                          int n_entries, const int* __restrict__ slots, const int* __restrict__ entries,
                          long long rows, int* status) {
  using Q = Q8<DV>;
  griddep_wait();
  int slot, entry;
  if (!find_pair(slots, n_slots, entries, n_entries, blockIdx.y, status, slot, entry)) return;
  const int sub = threadIdx.x % Q::kLanes;
  const long long row0 = (long long)blockIdx.x * Q::kTileRows + threadIdx.x / Q::kLanes;
  const float4* src = reinterpret_cast<const float4*>(S + (long long)slot * rows * DV);
  float4 x[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long r = row0 + u * Q::kRowsPerPass;
    x[u] = r < rows ? __ldcs(src + r * Q::kLanes + sub) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  unsigned* dst = reinterpret_cast<unsigned*>(cache + (long long)entry * rows * DV);
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long r = row0 + u * Q::kRowsPerPass;
    // as unsigned integers the magnitudes order like the values, NaN above infinity
    unsigned m = max(max(__float_as_uint(fabsf(x[u].x)), __float_as_uint(fabsf(x[u].y))),
                     max(__float_as_uint(fabsf(x[u].z)), __float_as_uint(fabsf(x[u].w))));
    m = row_max<Q::kLanes>(m);
    float s = row_scale(__uint_as_float(m));
    const bool held = m < 0x7f800000u && s >= FLT_MIN;
    const float inv = __frcp_rn(held ? s : 1.f);
    Rounded v[4] = {{x[u].x, s, inv}, {x[u].y, s, inv}, {x[u].z, s, inv}, {x[u].w, s, inv}};
    const float worst = fmaxf(fmaxf(fabsf(v[0].r2), fabsf(v[1].r2)), fmaxf(fabsf(v[2].r2), fabsf(v[3].r2)));
    if (__any_sync(0xffffffffu, worst >= s)) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e].settle(s);
    }
    unsigned c = __byte_perm(__byte_perm(__float_as_uint(v[0].t), __float_as_uint(v[1].t), 0x0040),
                             __byte_perm(__float_as_uint(v[2].t), __float_as_uint(v[3].t), 0x0040), 0x5410);
    if (!held) {
      c = 0u;
      s = m >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : 0.f;
    }
    if (r < rows) {
      dst[r * Q::kLanes + sub] = c;
      if (sub == 0) {
        scale[entry * rows + r] = s;
        if (z) z_cache[entry * rows + r] = z[slot * rows + r];
      }
    }
  }
}

template <int DV>
__global__ void __launch_bounds__(kThreads)
    state_load_q8_kernel(const int8_t* __restrict__ cache, const float* __restrict__ scale,
                         const float* __restrict__ z_cache, int n_entries, float* __restrict__ S,
                         float* __restrict__ z, int n_slots, const int* __restrict__ entries,
                         const int* __restrict__ slots, long long rows, int* status) {
  using Q = Q8<DV>;
  griddep_wait();
  int entry, slot;
  if (!find_pair(entries, n_entries, slots, n_slots, blockIdx.y, status, entry, slot)) return;
  const int sub = threadIdx.x % Q::kLanes;
  const long long row0 = (long long)blockIdx.x * Q::kTileRows + threadIdx.x / Q::kLanes;
  const char4* src = reinterpret_cast<const char4*>(cache + (long long)entry * rows * DV);
  char4 c[kUnroll];
  float s[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long r = row0 + u * Q::kRowsPerPass;
    c[u] = r < rows ? src[r * Q::kLanes + sub] : make_char4(0, 0, 0, 0);
    s[u] = r < rows ? scale[entry * rows + r] : 0.f;
  }
  float4* dst = reinterpret_cast<float4*>(S + (long long)slot * rows * DV);
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long r = row0 + u * Q::kRowsPerPass;
    if (r < rows) {
      dst[r * Q::kLanes + sub] = make_float4((float)c[u].x * s[u], (float)c[u].y * s[u], (float)c[u].z * s[u],
                                             (float)c[u].w * s[u]);
      if (z && sub == 0) z[slot * rows + r] = z_cache[entry * rows + r];
    }
  }
}

template <int DV>
dim3 q8_grid(long long rows, int n) {
  return dim3((unsigned)((rows + Q8<DV>::kTileRows - 1) / Q8<DV>::kTileRows), (unsigned)n);
}

}  // namespace

cudaError_t launch_state_store_q8(const float* S, const float* z, int n_slots, signed char* cache, float* scale,
                                  float* z_cache, int n_entries, const int* slots, const int* entries, int n,
                                  long long rows, int dv, const WaitCtl& wc, cudaStream_t st) {
  auto run = [&](auto width) {
    constexpr int DV = decltype(width)::value;
    return launch_pdl(state_store_q8_kernel<DV>, q8_grid<DV>(rows, n), dim3(kThreads), 0, st, S, z, n_slots,
                      reinterpret_cast<int8_t*>(cache), scale, z_cache, n_entries, slots, entries, rows, wc.status);
  };
  if (dv == 16) return run(std::integral_constant<int, 16>());
  if (dv == 64) return run(std::integral_constant<int, 64>());
  return run(std::integral_constant<int, 128>());
}

cudaError_t launch_state_load_q8(const signed char* cache, const float* scale, const float* z_cache, int n_entries,
                                 float* S, float* z, int n_slots, const int* entries, const int* slots, int n,
                                 long long rows, int dv, const WaitCtl& wc, cudaStream_t st) {
  auto run = [&](auto width) {
    constexpr int DV = decltype(width)::value;
    return launch_pdl(state_load_q8_kernel<DV>, q8_grid<DV>(rows, n), dim3(kThreads), 0, st,
                      reinterpret_cast<const int8_t*>(cache), scale, z_cache, n_entries, S, z, n_slots, entries, slots,
                      rows, wc.status);
  };
  if (dv == 16) return run(std::integral_constant<int, 16>());
  if (dv == 64) return run(std::integral_constant<int, 64>());
  return run(std::integral_constant<int, 128>());
}

}  // namespace kata
