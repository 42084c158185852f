// decay_walk_sm100.cu -- linear attention with a per-head decay over packed
// sequences, chunk by chunk on tcgen05 / TMEM.
//
// One walk (kata_internal.h) computes out_t = scale * sum_{s<=t} a^(t-s)
// (A_t . B_s) C_s plus the reach of the entering state, or the same over
// s >= t, backwards.  A sequence is walked in chunks of 128 tokens with the
// state S [d1, d2] in between.  For a chunk of r tokens (rows i, j; forward):
//   P     = A B^T                              [128 x 128]
//   W_ij  = a^(i-j) P_ij for j <= i, else 0    rounded to bf16
//   out_i = scale (sum_j W_ij C_j + a^(i+1) A_i S)
//   U     = sum_j (a^(r-1-j) B_j) C_j^T,   S <- a^r S + U
// and backwards, where the entering state already belongs to the chunk's last
// token: W_ij = a^(j-i) P_ij for j >= i, the reach of S is a^(r-1-i) and B_j
// enters with a^(j+1), times the scale (S is then the gradient itself, which
// the entering gradient joins unscaled).
//
// Roundings.  S is fp32, in TMEM for the whole walk.  The tensor cores truncate
// as they accumulate, so U is summed for itself, smallest part first, and added
// to S by the CUDA cores; a^128 is held as the sum of two fp32 values.  A scaled
// key enters U as two bf16 values (it loses up to 2^-16), as three (2^-24) where
// the chunk is still an 1/16 or more of the state that leaves.  Of tokens of like
// magnitude that state then agrees with fp32 arithmetic (1e-7 to 3e-7 of it in the
// mean square, at any length).  Which it is goes by the decay alone: where the last
// tokens' keys are zero or small, the state is made of keys of two values, and off
// by up to 9e-6 (4.8e-6 measured; with three everywhere 131072 tokens take 935 us
// instead of 760, 8192 in 13 sequences 89 instead of 82).  W and the copy of S that
// A is multiplied with are rounded to bf16 once, as operands of the tensor cores:
// they reach only out, which is rounded as far itself.  Out's error is 0.0024 in
// the mean square, of which its own rounding is 0.0017; a second value of each
// would be eight products more, and a second copy of S has no room beside two
// stages at d = dv = 128.
//
// One CTA per segment of a sequence, head and walk (1 CTA per SM: 512 TMEM
// columns, 26 warps of 72 registers):
//   0-7    S: a^r S + U, its bf16 copy for A S, and A S times the reach; the state
//          that leaves
//   8-15   W from P, over it; then out, through the chunk's C tile
//   16-23  keys: rest or hi in place over B once P is done, lo over A once A has
//          met S; rows past the sequence's end cleared in B and C, so that nothing
//          of the next sequence (NaN included) gets in
//   24     MMA issue (whole warp, one elected lane)
//   25     TMA: A, B, C tiles in, out
// Warps 8-23 also bring the state that enters.  A role has at least one warp per
// TMEM lane quarter.  MMA order per chunk: P; A S; the keys' parts; W C onto A S.
// An A and a B tile are loaded again once every product of the chunk is done, a C
// tile once out, written over it, has left.
//
// TMEM columns: P (W over it) 128 | A S, W C d2 | U d2 | S d2.  With d1 = 64 the
// state product still has 128 rows: its A operand reads the 64 columns twice
// (leading offset 0), so lanes 64-127 hold a second copy of S, and the two
// halves of the warps write one half of the bf16 copy each.
//
// Long sequences with few heads do not fill the SMs: they are cut into segments
// of L tokens.  decay_walk_kernel<.., true> first sums each segment from a zero
// state (the one walked last excepted); a walk then starts from the sums before
// its segment, which it adds up itself, or for 16 segments and more
// decay_scan_kernel does (plan below).
//
// What bounds it.  A chunk's critical path is work of CUDA cores on tiles (S and
// its copy, then keys and W side by side, then A S, then out) with four short
// products between: 5500 cycles a chunk at d = dv = 128, of which the tensor pipe
// works 38%; its tiles cross shared memory in 4700 cycles, and at 148 SMs its
// bytes HBM in 5500.  The sums, of which no chunk waits for another, are bound by
// the loads in flight (three stages 4.6 TB/s, two 3.7).  Measured: 131072 tokens,
// 16 heads, d = dv = 128 730 us, 2.9 TB/s of q, k, v and o (650 to 780 us by the
// clocks that the power cap leaves); a quarter of it are the segments' sums, which
// read k and v once more.  8192 tokens in 13 sequences: 83 us.  75 tokens, d = dv
// = 64: 8.3 us, a launch and one chunk's path.  Gradients, 8 x 2048 tokens, 16
// heads, d = dv = 128: 195 us.  Tried and not faster: fewer warps with more
// registers each, out by warps of its own, two accumulators for out, A S ahead of
// P, W in blocks of 32 columns (spills), S with its next columns on their way, a
// quarter of S by the warps of W.
#include <cuda.h>

#include <algorithm>
#include <atomic>

#include "decay_common.cuh"
#include "kata_internal.h"
#include "sm100.cuh"

namespace kata {
namespace {

using namespace sm100;

constexpr int kChunk = 128;
constexpr int kThreads = 832, kSumThreads = 768;
constexpr int kMaxWalks = 3;
constexpr uint32_t kTmemCols = 512;

struct WalkParams {
  CUtensorMap a, b, c, o;
  __nv_bfloat16* out;
  long long out_stride;
  const float* init;
  float* fin;
  float* rec;            // records of this walk's split sequences, [segment][H][d1][d2]
  int swapped;           // this walk has (d1, d2) of the kernel exchanged
  int reverse, init_transposed;
  float s_intra, s_inter, s_key;
};

struct Params {
  WalkParams w[kMaxWalks];
  const int* cu;
  const float* log_decay;
  const int* slots;
  const unsigned char* resume;
  int n_walks, T, H, N, L, n_slots, zero_outside, folded, max_records;
  WaitCtl wc;
};

template <int D1, int D2>
struct Cfg {
  static constexpr int kA = kChunk * D1 * 2, kC = kChunk * D2 * 2;  // tile bytes
  static constexpr int kStage = 2 * kA + kC;                         // [A | B | C]
  static constexpr int kCopy = D1 * D2 * 2;
  static constexpr int kFit = (224 * 1024 - kCopy) / kStage;
  static constexpr int kStages = kFit > 4 ? 4 : kFit;                // 2 (128, 128) .. 4 (64, 64)
  static constexpr int offStage = 0;
  static constexpr int offCopy = kStages * kStage;
  // the sum: stages [B | C], then lo
  static constexpr int kSumStage = kA + kC;
  static constexpr int kSumStages = (224 * 1024 - kA) / kSumStage >= 4 ? 4 : 3;  // 3 (128, 128), else 4
  static constexpr int offLo = kSumStages * kSumStage;
  static constexpr int kBytes =
      (offCopy + kCopy > offLo + kA ? offCopy + kCopy : offLo + kA) + 1024;  // + alignment slack
  static constexpr uint32_t colP = 0, colE = 128, colU = 128 + D2, colS = 128 + 2 * D2;
  static constexpr uint32_t colSumU = 0, colSumS = 2 * D2;  // the sum: two accumulators, and the sum
};
constexpr int kMaxStages = 4;

// What a CTA sets up while it looks for its segment, the same for all widths.
constexpr int kWeights = 178;  // 18 banks on: the two copies' reads share no bank
struct Shared {
  // s_intra times the weights a^|y| of y = j - i, 0 on the side that is not kept, twice, the second
  // time one entry on, so that the pair at any lane's j is aligned in one of them
  float weight[2 * kWeights];
  uint64_t full[kMaxStages];    // A and B landed (the sum: B and C)
  uint64_t late[kMaxStages];    // C landed
  uint64_t staged[kMaxStages];  // out in shared memory (256)
  uint64_t done[kMaxStages];    // every product of the chunk complete
  uint64_t scaled[kMaxStages];  // the sum's scaled keys written (256)
  uint64_t lo_free[2];          // the sum's lo read, of even and odd chunks
  uint64_t p_full;              // P in TMEM
  uint64_t w_full;              // W written (256)
  uint64_t s_init;              // the state that enters in TMEM (512)
  uint64_t s_copied;            // S copied to shared memory (256)
  uint64_t a_done;              // A has met B and S: its tile takes lo, and A S can be scaled
  uint64_t e_ready;             // A S scaled (256)
  uint64_t hi_full;             // hi, or rest before it, written, rows past the end cleared (256)
  uint64_t lo_full;             // lo written (256)
  uint64_t rest_done;           // rest has met C: its tile takes hi (the sum: lo)
  uint64_t last_full;           // hi (the sum: lo) written after rest (256)
  uint64_t o_full;              // out complete
  uint64_t o_free;              // and read (256)
  uint64_t u_done;              // the chunk's sum complete
  uint64_t sum_done[2];         // the sum's chunk sums complete, of even and odd chunks
  uint64_t sum_free[2];         // and read (128)
  uint64_t mma_done;            // every MMA issued has completed
  float keep[2];                // a^128, its rounded value and what that leaves out
  float keep_segment;           // a^L
  uint32_t tmem;
  int abort;
};
constexpr int kMaxShared = 227 * 1024 - (int)sizeof(Shared) - 64;
static_assert(Cfg<128, 128>::kStages >= 2 && Cfg<128, 128>::kBytes <= kMaxShared, "shared memory");
static_assert(Cfg<128, 64>::kBytes <= kMaxShared && Cfg<64, 128>::kBytes <= kMaxShared, "shared memory");
static_assert(Cfg<64, 64>::kBytes <= kMaxShared, "shared memory");

struct Found {
  int seq, s0, s1, seg, n_seg, t0, t1, rec, row, resumed;
};

// 16-byte unit u (8 values) of row r in a tile of 128-byte swizzled rows, `rows` to a 64-column atom
__device__ __forceinline__ uint32_t unit_offset(int rows, int r, int u) {
  return (uint32_t)((u >> 3) * rows * 128 + r * 128 + (((u & 7) ^ (r & 7)) << 4));
}

// Shared memory by its 32-bit address: a store whose pointer may also be a global
// one, as those of out, is compiled to a generic store, which takes twice as long.
__device__ __forceinline__ void sts128(uint32_t to, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(to), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t from) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(from));
  return v;
}
__device__ __forceinline__ uint64_t lds64(uint32_t from) {
  uint64_t v;
  asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(from));
  return v;
}

// Bounded wait as mbar_wait_w of sm100.cuh, in less code: a walk has more than
// twenty of them, and written out in full they, with other loops unrolled, came
// to 92 KB, more than an SM's instruction cache keeps.  The abort flag is the
// CTA's; the limit and the status word are the call's.
__device__ __forceinline__ bool wait_on(const WaitCtl& wc, int* abort_flag, uint64_t* bar, uint32_t parity) {
  bool ok = mbar_test_wait(bar, parity);
  if (!ok) {
    const long long t0 = clock64();
    do {
      if (*(volatile int*)abort_flag) break;
      if (clock64() - t0 >= wc.limit) {
        *(volatile int*)abort_flag = 1;
        report_status(wc.status, kErrTimeout);
        break;
      }
      ok = mbar_try_wait_sleep(bar, parity);
    } while (!ok);
  }
  return __all_sync(0xffffffffu, ok);
}

// one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}

// Of 16 values in bf16 pairs, those up to the last-th (from the
// first-th on); the others become 0 whatever they are.
__device__ __forceinline__ void keep_up_to(uint32_t (&x)[8], int last) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] &= __funnelshift_rc(0xffffffffu, 0u, (uint32_t)max(0, 16 - 16 * (last - 2 * e)));
}
__device__ __forceinline__ void keep_from(uint32_t (&x)[8], int first) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] &= __funnelshift_lc(0u, 0xffffffffu, (uint32_t)max(0, 16 * (first - 2 * e)));
}

// Column and row of a lane: with d1 = 64 lanes 64-127 hold a second copy of the
// state, and each half of the lanes handles one half of the columns in memory.
template <int D1, int D2>
struct StateLane {
  int row, own0, own1;
  __device__ __forceinline__ StateLane(int quarter, int lane)
      : row((quarter * 32 + lane) % D1),
        own0(D1 == 64 && quarter >= 2 ? D2 / 2 : 0),
        own1(D1 == 64 && quarter < 2 ? D2 / 2 : D2) {}
};

__device__ __forceinline__ void store_32b(void* to, const uint32_t* z) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(z[0]), "r"(z[1]), "r"(z[2]),
               "r"(z[3]), "r"(z[4]), "r"(z[5]), "r"(z[6]), "r"(z[7])
               : "memory");
}

// 8 values, a whole sector where they start on one
__device__ __forceinline__ void store_8(float* to, const uint32_t* x, bool wide) {
  if (wide) {
    store_32b(to, x);
  } else {
    *reinterpret_cast<uint4*>(to) = make_uint4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<uint4*>(to + 4) = make_uint4(x[4], x[5], x[6], x[7]);
  }
}

// D columns of TMEM times a factor of the lane: 16 at a time, and the next 16 on their way
template <int D>
__device__ __forceinline__ void scale_columns(uint32_t col, float factor) {
  const uint64_t f2 = f32x2(__float_as_uint(factor), __float_as_uint(factor));
  uint32_t r[2][16];
  auto put = [&](uint32_t at, uint32_t (&x)[16]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint64_t v = f32x2_mul(f32x2(x[2 * k], x[2 * k + 1]), f2);
      x[2 * k] = (uint32_t)v;
      x[2 * k + 1] = (uint32_t)(v >> 32);
    }
    tmem_st16(at, x);
  };
  tmem_ld16(col, r[0]);
#pragma unroll 1
  for (int at = 0; at < D; at += 32) {
    tmem_wait_ld();
    tmem_ld16(col + at + 16, r[1]);
    put(col + at, r[0]);
    tmem_wait_ld();
    if (at + 32 < D) tmem_ld16(col + at + 32, r[0]);
    put(col + at + 16, r[1]);
  }
}

// A key times its factor, f k, as the sum of three bf16 values: hi = f1 k with f1
// the factor rounded, lo = (f1 k - hi) + f2 k with f2 what f1 leaves out (the
// parenthesis is a bf16 value), and rest what these leave out, from the product
// in fp32.  Up to 2^-24 of f k is lost, as in fp32 arithmetic; hi and lo alone
// would lose 2^-16 (4e-6 of the state in the mean square).  Rows past the end
// (another sequence's, or nothing) count as zeros, and are cleared in the tiles.
struct KeyFactor {
  __nv_bfloat162 f1, f2;
  uint64_t f;
  __device__ __forceinline__ explicit KeyFactor(float x) {
    const __nv_bfloat16 a = __float2bfloat16_rn(x), b = __float2bfloat16_rn(x - __bfloat162float(a));
    f1 = __halves2bfloat162(a, a);
    f2 = __halves2bfloat162(b, b);
    f = f32x2(__float_as_uint(x), __float_as_uint(x));
  }
  static __device__ __forceinline__ __nv_bfloat162 pair(uint32_t x) {
    return *reinterpret_cast<const __nv_bfloat162*>(&x);
  }
  static __device__ __forceinline__ uint32_t bits(__nv_bfloat162 x) { return *reinterpret_cast<const uint32_t*>(&x); }
  static __device__ __forceinline__ uint64_t wide(uint32_t x) { return f32x2(x << 16, x & 0xffff0000u); }
  __device__ __forceinline__ uint32_t high(uint32_t k) const { return bits(__hmul2(pair(k), f1)); }
  __device__ __forceinline__ uint32_t low(uint32_t k) const {
    return bits(__hfma2(pair(k), f2, __hfma2(pair(k), f1, __hneg2(__hmul2(pair(k), f1)))));
  }
  __device__ __forceinline__ uint32_t rest(uint32_t k) const {
    const uint64_t minus = f32x2(0xbf800000u, 0xbf800000u);
    uint64_t d = f32x2_fma(wide(high(k)), minus, f32x2_mul(wide(k), f));
    d = f32x2_fma(wide(low(k)), minus, d);
    return pack_bf16x2(f32x2_lo(d), f32x2_hi(d));
  }
};

// The first unit of one half of a row of D values; unit u is at this ^ 16 u (tiles
// are 1024-byte aligned).
template <int D>
__device__ __forceinline__ uint32_t half_row(uint32_t tile, int j, int half) {
  return tile + unit_offset(kChunk, j, half * (D / 16));
}
// One half of a row from its tile
template <int D>
__device__ __forceinline__ void read_half(uint32_t tile, int j, int half, uint32_t (&x)[D / 4]) {
  const uint32_t row = half_row<D>(tile, j, half);
#pragma unroll
  for (int u = 0; u < D / 16; ++u) {
    const uint4 v = lds128(row ^ 16 * u);
    x[4 * u] = v.x;
    x[4 * u + 1] = v.y;
    x[4 * u + 2] = v.z;
    x[4 * u + 3] = v.w;
  }
}
// What is computed from x before and after this is computed twice, not kept in
// registers (x, hi, lo and rest together are 128).
template <int N>
__device__ __forceinline__ void compute_again(uint32_t (&x)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) asm volatile("" : "+r"(x[e]));
}
// and, through a function of each pair, to one
template <int D, typename F>
__device__ __forceinline__ void write_half(uint32_t tile, int j, int half, const uint32_t (&x)[D / 4], F of) {
  const uint32_t row = half_row<D>(tile, j, half);
#pragma unroll
  for (int u = 0; u < D / 16; ++u)
    sts128(row ^ 16 * u, of(x[4 * u]), of(x[4 * u + 1]), of(x[4 * u + 2]),
           of(x[4 * u + 3]));
}
// a half row of zeros
template <int D>
__device__ __forceinline__ void clear_half(uint32_t tile, int j, int half) {
  const uint32_t row = half_row<D>(tile, j, half);
#pragma unroll
  for (int u = 0; u < D / 16; ++u) sts128(row ^ 16 * u, 0u, 0u, 0u, 0u);
}

// descriptors of the state's products: scaled keys (M-major), and the C tile (N-major)
template <int D1>
__device__ __forceinline__ uint64_t key_desc(uint32_t tile) {
  return smem_desc(tile, D1 == 128 ? 16384u : 0u, 1024, kSw128);
}

// the segment that is walked last: no sum of it is needed, its record holds what enters the sequence
__device__ __forceinline__ int last_walked(const WalkParams& w, const Found& f) {
  return w.reverse ? 0 : f.n_seg - 1;
}

// Whether a state still holds a 16th or more of what entered it `tokens` ago.  If
// not, what rest would add to it is below 2^-20 of the size it entered with, and hi
// and lo do: 2^-20 of the state where later tokens are as large as earlier ones.
__device__ __forceinline__ bool remembered(float g, int tokens) { return g * (float)tokens >= -2.7725887f; }

// a^tokens as a rounded value and what that leaves out: a state is multiplied by it
// once a chunk (a scanned one: once a segment), for as long as it remembers, and
// what rounding leaves out, up to 2^-25, would add up, the same every time (147
// segments: 2e-6 of the state).
__device__ __forceinline__ void power_of(float g, int tokens, float& hi, float& lo) {
  const double x = exp((double)g * tokens);
  hi = (float)x;
  lo = (float)(x - (double)hi);
}

// y of the first weight
__device__ __forceinline__ int first_weight(bool reverse) { return reverse ? -32 : -128; }

template <int D1, int D2>
__device__ void walk(const Params& p, const WalkParams& w, int h, float g, uint8_t* smem, Shared& sh, const Found& f) {
  using C = Cfg<D1, D2>;
  constexpr int kStages = C::kStages;
  uint64_t *full = sh.full, *late = sh.late, *staged = sh.staged, *done = sh.done;
  uint64_t *s_init = &sh.s_init, *p_full = &sh.p_full, *w_full = &sh.w_full, *s_copied = &sh.s_copied, *e_ready = &sh.e_ready;
  uint64_t *a_done = &sh.a_done, *hi_full = &sh.hi_full, *rest_done = &sh.rest_done, *lo_full = &sh.lo_full;
  uint64_t *last_full = &sh.last_full, *o_full = &sh.o_full;
  uint64_t *o_free = &sh.o_free, *u_done = &sh.u_done, *mma_done = &sh.mma_done;
  const uint32_t weight = smem_u32(sh.weight);
  const uint32_t tmem = sh.tmem;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool rev = w.reverse != 0, split = f.n_seg > 1;
  const int n_chunks = (f.t1 - f.t0 + kChunk - 1) / kChunk;
  // c-th chunk walked: its first token and its tokens
  auto chunk_t = [&](int c) { return f.t0 + (rev ? n_chunks - 1 - c : c) * kChunk; };
  auto chunk_n = [&](int c) { return min(kChunk, f.t1 - chunk_t(c)); };
  // chunks whose keys enter with their rest: those that the state which leaves remembers
  const bool leaves = w.fin && f.row >= 0 && f.seg == last_walked(w, f);
  auto precise = [&](int c) { return leaves && remembered(g, rev ? chunk_t(c) - f.s0 : f.s1 - chunk_t(c) - kChunk); };
  // tiles of a chunk (one thread): A and B as soon as the chunk before it in the
  // stage has been multiplied, C once that chunk's out, which leaves through its
  // C tile, has left
  auto load = [&](int c) {
    const int st = c % kStages, t = chunk_t(c);
    uint8_t* base = smem + C::offStage + st * C::kStage;
    mbar_arrive_expect_tx(full + st, 2 * C::kA);
#pragma unroll
    for (int x = 0; x < D1 / 64; ++x) {
      tma_load_3d(base + x * 16384, &w.a, full + st, 64 * x, h, t);
      tma_load_3d(base + C::kA + x * 16384, &w.b, full + st, 64 * x, h, t);
    }
  };
  auto load_late = [&](int c) {
    const int st = c % kStages, t = chunk_t(c);
    uint8_t* base = smem + C::offStage + st * C::kStage;
    mbar_arrive_expect_tx(late + st, C::kC);
#pragma unroll
    for (int x = 0; x < D2 / 64; ++x) tma_load_3d(base + 2 * C::kA + x * 16384, &w.c, late + st, 64 * x, h, t);
  };

  const int y0 = first_weight(rev);
  auto power = [&](int x) { return expf(g * (float)x); };  // a^x
  auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_on(p.wc, &sh.abort, bar, parity); };

  // The state that enters, to TMEM, by the warps of W, out and B, a quarter of the
  // columns each; 32 (16) columns' loads are in flight.  A cut sequence's segment
  // starts from its scanned record, or sums those before it by itself, from the
  // copy of what enters the sequence (which the last one may be overwriting).
  constexpr int size = D1 * D2;
  if (warp >= 8 && warp < 24 && n_chunks > 0) {
    constexpr int kCols = D2 / 4;
    const int m = warp % 4 * 32 + lane, row = m % D1, at = (warp / 4 - 2) * kCols;
    const float* src = nullptr;
    if (split)
      src = w.rec + ((long long)(f.rec + (p.folded ? last_walked(w, f) : f.seg)) * p.H + h) * size;
    else if (w.init && f.row >= 0 && f.resumed)
      src = w.init + ((long long)f.row * p.H + h) * size;
    const bool transposed = w.init_transposed && !split;
    if (split) griddep_wait();  // the sums, scanned or not
    float r[kCols];
#pragma unroll
    for (int e = 0; e < kCols; ++e) r[e] = 0.f;
    auto row_of = [&](const float* from, float (&x)[kCols]) {
#pragma unroll
      for (int e = 0; e < kCols; e += 4) {
        const float4 v = *reinterpret_cast<const float4*>(from + row * D2 + at + e);
        x[e] = v.x;
        x[e + 1] = v.y;
        x[e + 2] = v.z;
        x[e + 3] = v.w;
      }
    };
    if (src && transposed) {
#pragma unroll
      for (int e = 0; e < kCols; ++e) r[e] = src[(at + e) * D1 + row];
    } else if (src) {
      row_of(src, r);
    }
    if (split && p.folded) {
      const int before = rev ? f.n_seg - 1 - f.seg : f.seg;
#pragma unroll 1
      for (int s = 0; s < before; ++s) {
        const int seg = rev ? f.n_seg - 1 - s : s;
        const int tokens = min(p.L, f.s1 - f.s0 - seg * p.L);
        const float keep = tokens == p.L ? sh.keep_segment : expf(g * (float)tokens);
        float x[kCols];
        row_of(w.rec + ((long long)(f.rec + seg) * p.H + h) * size, x);
#pragma unroll
        for (int e = 0; e < kCols; ++e) r[e] = fmaf(keep, r[e], x[e]);
      }
    }
    const uint32_t to = tmem + ((uint32_t)(warp % 4 * 32) << 16) + C::colS + at;
#pragma unroll
    for (int e = 0; e < kCols; e += 16) {
      uint32_t z[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) z[k] = __float_as_uint(r[e + k]);
      tmem_st16(to + e, z);
    }
    tmem_wait_st();
    tc_fence_before();
    mbar_arrive(s_init);
  }

  if (warp < 8) {
    // --------------------------------------------------------------- S
    const int quarter = warp % 4;
    const StateLane<D1, D2> l(quarter, lane);
    // half of the lane's columns
    const int c0 = l.own0 + warp / 4 * ((l.own1 - l.own0) / 2), c1 = c0 + (l.own1 - l.own0) / 2;
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16) + C::colS;
    // the lane's row of the copy: its columns are of one atom, unit u of it at copy ^ 16 u
    const uint32_t copy = smem_u32(smem + C::offCopy) + unit_offset(D1, l.row, c0 / 64 * 8);
    float* dst = w.fin && f.row >= 0 && f.seg == (rev ? 0 : f.n_seg - 1)
                     ? w.fin + ((long long)f.row * p.H + h) * size
                     : nullptr;
    const bool wide = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;
    bool ok = n_chunks == 0 || wait(s_init, 0);
#pragma unroll 1
    for (int c = 0; ok && c <= n_chunks && n_chunks > 0; ++c) {
      // The state before chunk c (c = n_chunks: the one that leaves): a^n S + U of
      // the chunk before, added in fp32 (the tensor core's accumulation truncates:
      // onto S it would cost 6e-7 of it every chunk).  16 columns at a time.
      float k0 = 1.f, k1 = 0.f;
      const bool add = c > 0, last = c == n_chunks;
      if (add) {
        if (!wait(u_done, (c - 1) & 1)) break;
        if (last && !dst) break;
        const int n = chunk_n(c - 1);
        k0 = n == kChunk ? sh.keep[0] : power(n);
        k1 = n == kChunk ? sh.keep[1] : 0.f;
      }
      tc_fence_after();
      const uint64_t keep = f32x2(__float_as_uint(k0), __float_as_uint(k0));
      const uint64_t more = f32x2(__float_as_uint(k1), __float_as_uint(k1));
#pragma unroll 1
      for (int at = c0; at < c1; at += 16) {
        uint32_t r[16], u[16];
        tmem_ld16(lane_base + at, r);
        tmem_ld16(lane_base - C::colS + C::colU + at, u);  // before the first chunk: not used
        tmem_wait_ld();
        if (add) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint64_t x = f32x2(r[2 * k], r[2 * k + 1]);
            const uint64_t v = f32x2_fma(x, keep, f32x2_fma(x, more, f32x2(u[2 * k], u[2 * k + 1])));
            r[2 * k] = (uint32_t)v;
            r[2 * k + 1] = (uint32_t)(v >> 32);
          }
          if (!last) tmem_st16(lane_base + at, r);
        }
        if (last) {
          store_8(dst + l.row * D2 + at, r, wide);
          store_8(dst + l.row * D2 + at + 8, r + 8, wide);
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t z[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              z[k] = pack_bf16x2(__uint_as_float(r[8 * e + 2 * k]), __uint_as_float(r[8 * e + 2 * k + 1]));
            sts128(copy ^ 16 * ((at / 8 + e) & 7), z[0], z[1], z[2], z[3]);
          }
        }
      }
      if (last) break;
      tmem_wait_st();
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(s_copied);
      // A S times a^reach: the product of W and C is added to it
      const int i = quarter * 32 + lane, n = chunk_n(c);
      const float reach = w.s_inter * power(rev ? max(n - 1 - i, 0) : i + 1);
      if (!wait(a_done, c & 1)) break;
      tc_fence_after();
      scale_columns<D2 / 2>(lane_base - C::colS + C::colE + warp / 4 * (D2 / 2), reach);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(e_ready);
    }
    if (n_chunks == 0 && dst) {  // an empty sequence leaves what it starts from
      const float* src = w.init && f.resumed ? w.init + ((long long)f.row * p.H + h) * size : nullptr;
      for (int j = c0; j < c1; ++j)
        dst[l.row * D2 + j] = src ? src[w.init_transposed ? j * D1 + l.row : l.row * D2 + j] : 0.f;
    }
    griddep_wait();  // a grid ends after those it was launched behind
  } else if (warp < 16) {
    // --------------------------------------------------------------- W and out
    const int quarter = warp % 4, half = warp >= 12 ? 1 : 0;
    const int i = quarter * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
    // Of the four blocks of 32 columns of a row, one warp takes the outer two and
    // the other the inner two.
#pragma unroll 1
    for (int c = 0; c < n_chunks; ++c) {
      const int n = chunk_n(c);
      if (!wait(p_full, c & 1)) break;
      tc_fence_after();
#pragma unroll 1
      for (int y = 0; y < 4; ++y) {
        const int bb = half ? 1 + (y >> 1) : 3 * (y >> 1), j0 = 32 * bb + 16 * (y & 1);  // columns j0 .. j0 + 15
        uint32_t x[8];
        if (rev ? bb < quarter : bb > quarter) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = 0u;
        } else {
          uint32_t r[16];
          tmem_ld16(lane_base + C::colP + j0, r);
          tmem_wait_ld();
          const int at = j0 - i - y0;
          const uint32_t t = weight + 4 * (at & 1 ? kWeights + at - 1 : at);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint64_t v = f32x2_mul(f32x2(r[2 * e], r[2 * e + 1]), lds64(t + 8 * e));
            x[e] = pack_bf16x2(f32x2_lo(v), f32x2_hi(v));
          }
          // what a weight of 0 does not remove if it is NaN or infinite: beyond the
          // diagonal, and backwards columns past the end, another sequence's rows
          if (bb == quarter) {
            if (rev)
              keep_from(x, i - j0);
            else
              keep_up_to(x, i - j0);
          }
          if (rev && j0 + 16 > n) keep_up_to(x, n - 1 - j0);
        }
        tmem_st8(lane_base + C::colP + 32 * bb + 8 * (y & 1), x);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(w_full);
      // out, through the C tile, which every product has read by now; a copy of a
      // tile that is not full would reach into the next sequence
      if (!wait(o_full, c & 1)) break;
      tc_fence_after();
#pragma unroll 1
      for (int at = half * (D2 / 2); at < (half + 1) * (D2 / 2); at += 32) {
        uint32_t x[32];
        tmem_ld32(lane_base + C::colE + at, x);
        tmem_wait_ld();
        if (at + 32 == (half + 1) * (D2 / 2)) {
          tc_fence_before();
          mbar_arrive(o_free);
        }
        uint32_t z[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) z[e] = pack_bf16x2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
        if (n == kChunk) {
          const uint32_t orow = smem_u32(smem + C::offStage) + c % kStages * C::kStage + 2 * C::kA +
                                unit_offset(kChunk, i, half * (D2 / 16) & ~7);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sts128(orow ^ 16 * ((at / 8 + e) & 7), z[4 * e], z[4 * e + 1], z[4 * e + 2], z[4 * e + 3]);
        } else if (i < n) {
          uint4* orow =
              reinterpret_cast<uint4*>(w.out + (long long)(chunk_t(c) + i) * w.out_stride + (long long)h * D2 + at);
#pragma unroll
          for (int e = 0; e < 4; ++e) orow[e] = make_uint4(z[4 * e], z[4 * e + 1], z[4 * e + 2], z[4 * e + 3]);
        }
      }
      if (n == kChunk) fence_proxy_async_smem();
      mbar_arrive(staged + c % kStages);
    }
  } else if (warp == 25) {
    // --------------------------------------------------------------- copies: tiles in, out
    int loaded = min(kStages, n_chunks), loaded_late = loaded;
    if (lane == 0) {
#pragma unroll 1
      for (int c = 0; c < loaded; ++c) {
        load(c);
        load_late(c);
      }
    }
    __syncwarp();
#pragma unroll 1
    for (int c = 0; c < n_chunks; ++c) {
      const int st = c % kStages;
      if (!wait(done + st, (c / kStages) & 1)) break;
      if (loaded < n_chunks) {
        if (lane == 0) load(loaded);
        ++loaded;
        __syncwarp();
      }
      if (!wait(staged + st, (c / kStages) & 1)) break;
      if (lane == 0) {
        if (chunk_n(c) == kChunk) {
#pragma unroll
          for (int x = 0; x < D2 / 64; ++x)
            tma_store_3d(&w.o, smem + C::offStage + st * C::kStage + 2 * C::kA + x * 16384, 64 * x, h, chunk_t(c));
          bulk_commit_group();
          bulk_wait_read_all();
        }
        if (loaded_late < n_chunks) load_late(loaded_late);
      }
      if (loaded_late < n_chunks) ++loaded_late;
      __syncwarp();
    }
    // every copy that was issued ends before the CTA does
    if (lane == 0) bulk_wait_all();
#pragma unroll 1
    for (int c = max(loaded - kStages, 0); c < loaded; ++c) mbar_wait_drain(full + c % kStages, (c / kStages) & 1);
#pragma unroll 1
    for (int c = max(loaded_late - kStages, 0); c < loaded_late; ++c)
      mbar_wait_drain(late + c % kStages, (c / kStages) & 1);
  } else if (warp == 24) {
    // --------------------------------------------------------------- MMA
    constexpr uint32_t id_p = idesc_bf16(128, 128, false, false);  // A, B both K-major
    constexpr uint32_t id_o = idesc_bf16(128, D2, false, true);    // A or W, and C or the copy of S (N-major)
    constexpr uint32_t id_s = idesc_bf16(128, D2, true, true);     // B^T (M-major), C (N-major)
    const uint32_t sStage = smem_u32(smem + C::offStage);
    const uint64_t dcopy = smem_desc(smem_u32(smem + C::offCopy), D1 * 128, 1024, kSw128);
    int rests = 0;
#pragma unroll 1
    for (int c = 0; c < n_chunks; ++c) {
      const int st = c % kStages;
      const uint32_t sA = sStage + st * C::kStage, sB = sA + C::kA, sC = sB + C::kA;
      const uint64_t dA = smem_desc(sA, 16, 1024, kSw128), dB = smem_desc(sB, 16, 1024, kSw128);
      const uint64_t dC = smem_desc(sC, 16384, 1024, kSw128);
      const uint64_t kB = key_desc<D1>(sB), kA = key_desc<D1>(sA);
      // U (+)= K^T C, K scaled keys in the B or the A tile
      auto add_keys = [&](uint64_t keys, bool first, uint64_t* done) {
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < kChunk / 16; ++ks)
            mma_ss(tmem + C::colU, desc_add(keys, ks * 2048), desc_add(dC, ks * 2048), id_s, !first || ks > 0);
          if (done) mma_commit(done);
        }
        __syncwarp();
      };
      if (!wait(full + st, (c / kStages) & 1)) break;
      tc_fence_after();
      // over W of the chunk before only after its product, which was issued before
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < D1 / 16; ++ks) {
          const uint32_t off = (ks >> 2) * 16384 + (ks & 3) * 32;
          mma_ss(tmem + C::colP, desc_add(dA, off), desc_add(dB, off), id_p, ks > 0);
        }
        mma_commit(p_full);
      }
      __syncwarp();
      // the copy of S, and with it U read
      if (!wait(s_copied, c & 1)) break;
      if (c > 0 && !wait(o_free, (c - 1) & 1)) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < D1 / 16; ++ks)
          mma_ss(tmem + C::colE, desc_add(dA, (ks >> 2) * 16384 + (ks & 3) * 32), desc_add(dcopy, ks * 2048), id_o,
                 ks > 0);
        mma_commit(a_done);
      }
      __syncwarp();
      // rest, lo, hi: what the accumulation truncates is a part of what is there; hi, lo without a rest
      const bool all = precise(c);
      if (!wait(late + st, (c / kStages) & 1)) break;
      if (!wait(hi_full, c & 1)) break;
      tc_fence_after();
      add_keys(kB, true, all ? rest_done : nullptr);
      if (!wait(lo_full, c & 1)) break;
      tc_fence_after();
      add_keys(kA, false, all ? nullptr : u_done);
      if (all) {
        if (!wait(last_full, rests & 1)) break;
        tc_fence_after();
        add_keys(kB, false, u_done);
        ++rests;
      }
      if (!wait(w_full, c & 1)) break;
      if (!wait(e_ready, c & 1)) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < kChunk / 16; ++ks)  // keys 16 ks ..: at the start of the 32 columns they came from
          mma_ts(tmem + C::colE, tmem + C::colP + (ks >> 1) * 32 + (ks & 1) * 8, desc_add(dC, ks * 2048), id_o, 1);
        mma_commit(o_full);
        mma_commit(done + st);
      }
      __syncwarp();
    }
    // every MMA that was issued ends before the CTA does
    mma_commit_w(mma_done);
    mbar_wait_drain(mma_done, 0);
  } else {
    // --------------------------------------------------------------- B
    const int j = (warp & 3) * 32 + lane, half = warp >= 20 ? 1 : 0;  // token of the chunk, half of its row
    int rests = 0;
#pragma unroll 1
    for (int c = 0; c < n_chunks; ++c) {
      const int st = c % kStages, n = chunk_n(c);
      const bool live = j < n;
      const uint32_t tA = smem_u32(smem + C::offStage) + st * C::kStage;
      const KeyFactor kf(live ? w.s_key * power(rev ? j + 1 : n - 1 - j) : 0.f);
      uint32_t x[D1 / 4];
      if (!wait(full + st, (c / kStages) & 1)) break;
      if (n < kChunk && !wait(late + st, (c / kStages) & 1)) break;
      if (!live) {  // of P only what W drops comes from these rows
        clear_half<D1>(tA + C::kA, j, half);
        clear_half<D2>(tA + 2 * C::kA, j, half);
      }
      read_half<D1>(tA + C::kA, j, half, x);
      if (!wait(p_full, c & 1)) break;
      if (precise(c)) {
        write_half<D1>(tA + C::kA, j, half, x, [&](uint32_t k) { return kf.rest(k); });
        fence_proxy_async_smem();
        mbar_arrive(hi_full);
        compute_again(x);
        if (!wait(a_done, c & 1)) break;
        write_half<D1>(tA, j, half, x, [&](uint32_t k) { return kf.low(k); });
        fence_proxy_async_smem();
        mbar_arrive(lo_full);
        compute_again(x);
        if (!wait(rest_done, rests & 1)) break;
        write_half<D1>(tA + C::kA, j, half, x, [&](uint32_t k) { return kf.high(k); });
        fence_proxy_async_smem();
        mbar_arrive(last_full);
        ++rests;
      } else {
        write_half<D1>(tA + C::kA, j, half, x, [&](uint32_t k) { return kf.high(k); });
        fence_proxy_async_smem();
        mbar_arrive(hi_full);
        compute_again(x);
        // lo, while A meets S
#pragma unroll
        for (int e = 0; e < D1 / 4; ++e) {
          x[e] = kf.low(x[e]);
        }
        if (!wait(a_done, c & 1)) break;
        write_half<D1>(tA, j, half, x, [](uint32_t k) { return k; });
        fence_proxy_async_smem();
        mbar_arrive(lo_full);
      }
    }
  }
}

// The sum of one segment of a sequence that is cut, from a zero state:
//   sum_t a^(tokens of the segment after t) B_t C_t^T   (backwards: a^(tokens before t, and t))
// With each key scaled for the segment's end nothing is carried from chunk to
// chunk, so no product waits for another: bound by the loads of B and C.
// Warps: 0 MMA, 1 TMA, 4-19 scale the keys in two groups, a chunk each, 20-23
// add the chunks' sums.
template <int D1, int D2>
__device__ void sum_segment(const Params& p, const WalkParams& w, int h, float g, uint8_t* smem, Shared& sh,
                            const Found& f) {
  using C = Cfg<D1, D2>;
  constexpr int kStages = C::kSumStages;
  uint64_t *full = sh.full, *empty = sh.done, *scaled = sh.scaled, *lo_free = sh.lo_free, *mma_done = &sh.mma_done;
  const uint32_t tmem = sh.tmem;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_chunks = (f.t1 - f.t0 + kChunk - 1) / kChunk;
  const uint32_t sStage = smem_u32(smem), sLo = sStage + C::offLo;
  auto precise = [&](int c) {
    const int t = f.t0 + c * kChunk;
    return w.fin && remembered(g, w.reverse ? t - f.s0 : f.s1 - t - kChunk);
  };
  auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_on(p.wc, &sh.abort, bar, parity); };
  if (warp == 0) {
    constexpr uint32_t id_s = idesc_bf16(128, D2, true, true);
    int rests = 0;
#pragma unroll 1
    for (int c = 0; c < n_chunks; ++c) {
      const int st = c % kStages;
      const uint32_t sB = sStage + st * C::kSumStage;
      const uint64_t dC = smem_desc(sB + C::kA, 16384, 1024, kSw128);
      if (!wait(full + st, (c / kStages) & 1)) break;
      if (!wait(scaled + st, (c / kStages) & 1)) break;
      tc_fence_after();
      if (c > 1 && !wait(sh.sum_free + (c & 1), ((c >> 1) - 1) & 1)) break;
      tc_fence_after();
      // smallest first, into an accumulator of the chunk's own
      auto add = [&](uint32_t keys, bool first) {
        const uint64_t dK = key_desc<D1>(keys);
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < kChunk / 16; ++ks)
            mma_ss(tmem + C::colSumU + (c & 1) * D2, desc_add(dK, ks * 2048), desc_add(dC, ks * 2048), id_s,
                   !first || ks > 0);
        }
        __syncwarp();
      };
      const bool all = precise(c);
      add(sLo, true);  // rest where there is one
      if (all) {
        mma_commit_w(&sh.rest_done);
        if (!wait(&sh.last_full, rests & 1)) break;
        tc_fence_after();
        add(sLo, false);
        ++rests;
      }
      add(sB, false);
      mma_commit_w(sh.sum_done + (c & 1));
      mma_commit_w(empty + st);
      mma_commit_w(lo_free + (c & 1));
    }
    mma_commit_w(mma_done);
    mbar_wait_drain(mma_done, 0);
  } else if (warp == 1) {
    int issued = 0;
#pragma unroll 1
    for (int c = 0; c < n_chunks; ++c, ++issued) {
      const int st = c % kStages, t = f.t0 + c * kChunk;
      if (!wait(empty + st, ((c / kStages) & 1) ^ 1)) break;
      if (lane != 0) continue;
      uint8_t* base = smem + st * C::kSumStage;
      mbar_arrive_expect_tx(full + st, C::kSumStage);
#pragma unroll
      for (int x = 0; x < D1 / 64; ++x) tma_load_3d(base + x * 16384, &w.b, full + st, 64 * x, h, t);
#pragma unroll
      for (int x = 0; x < D2 / 64; ++x) tma_load_3d(base + C::kA + x * 16384, &w.c, full + st, 64 * x, h, t);
    }
    // every copy that was issued ends before the CTA does
#pragma unroll 1
    for (int c = max(issued - kStages, 0); c < issued; ++c) mbar_wait_drain(full + c % kStages, (c / kStages) & 1);
    __syncwarp();
  } else if (warp >= 20) {
    // the chunks' sums, added in fp32
    const int quarter = warp % 4;
    const StateLane<D1, D2> l(quarter, lane);
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
    float* dst = w.rec + ((long long)(f.rec + f.seg) * p.H + h) * (D1 * D2);
    const bool wide = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;
#pragma unroll 1
    for (int c = 0; c < n_chunks; ++c) {
      if (!wait(sh.sum_done + (c & 1), (c >> 1) & 1)) break;
      tc_fence_after();
#pragma unroll 1
      for (int at = 0; at < D2; at += 8) {
        uint32_t r[8], u[8];
        tmem_ld8(lane_base + C::colSumU + (c & 1) * D2 + at, u);
        tmem_ld8(lane_base + C::colSumS + at, r);
        tmem_wait_ld();
        if (c > 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e) u[e] = __float_as_uint(__uint_as_float(r[e]) + __uint_as_float(u[e]));
        }
        if (c + 1 < n_chunks)
          tmem_st8(lane_base + C::colSumS + at, u);
        else if (at >= l.own0 && at < l.own1)
          store_8(dst + l.row * D2 + at, u, wide);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(sh.sum_free + (c & 1));
    }
  } else if (warp >= 4) {
    // two groups of eight warps, a chunk each, half a row a thread
    const int j = (warp & 3) * 32 + lane, half = warp >> 2 & 1;
    // No wait is a phase ahead: a group that waits for chunk c + 2 has seen the
    // products of chunk c - 1 complete (lo_free), the last that used its stage.
    static_assert(kStages >= 3, "stages");
    int rests = 0;  // of the chunks before c
#pragma unroll 1
    for (int c = 0; c < n_chunks; ++c) {
      const bool all = precise(c);
      if ((c & 1) != (warp >= 12 ? 1 : 0)) {
        rests += all;
        continue;
      }
      const int st = c % kStages, t = f.t0 + c * kChunk, n = min(kChunk, f.t1 - t);
      const uint32_t sB = sStage + st * C::kSumStage;
      const float fac =
          j < n ? w.s_key * expf(g * (float)(w.reverse ? t + j + 1 - f.t0 : f.t1 - 1 - t - j)) : 0.f;
      const KeyFactor kf(fac);
      uint32_t x[D1 / 4];
      if (!wait(full + st, (c / kStages) & 1)) break;
      if (j >= n) {
        clear_half<D1>(sB, j, half);
        clear_half<D2>(sB + C::kA, j, half);
      }
      read_half<D1>(sB, j, half, x);
      write_half<D1>(sB, j, half, x, [&](uint32_t k) { return kf.high(k); });
      compute_again(x);
      if (!all) {
#pragma unroll
        for (int e = 0; e < D1 / 4; ++e) x[e] = kf.low(x[e]);
      }
      if (c > 0 && !wait(lo_free + ((c - 1) & 1), ((c - 1) >> 1) & 1)) break;
      if (all) {
        write_half<D1>(sLo, j, half, x, [&](uint32_t k) { return kf.rest(k); });
        fence_proxy_async_smem();
        mbar_arrive(scaled + st);
        compute_again(x);
        if (!wait(&sh.rest_done, rests & 1)) break;
        write_half<D1>(sLo, j, half, x, [&](uint32_t k) { return kf.low(k); });
        fence_proxy_async_smem();
        mbar_arrive(&sh.last_full);
        ++rests;
        continue;
      }
      write_half<D1>(sLo, j, half, x, [](uint32_t k) { return k; });
      fence_proxy_async_smem();
      mbar_arrive(scaled + st);
    }
  }
}

// what enters the sequence, as [d1][d2], to the record of the segment walked last
__device__ __noinline__ void copy_init(const WalkParams& w, const Found& f, int H, int h, int d1, int d2) {
  const int size = d1 * d2;
  const float* src = w.init && f.row >= 0 && f.resumed ? w.init + ((long long)f.row * H + h) * size : nullptr;
  float* dst = w.rec + ((long long)(f.rec + f.seg) * H + h) * size;
  for (int x = threadIdx.x; x < size; x += kSumThreads)
    dst[x] = !src ? 0.f : src[w.init_transposed ? x % d2 * d1 + x / d2 : x];
}

// DA, DB: the widths (d1, d2) of the walks; a `swapped` walk has them exchanged.
template <int DA, int DB, bool kSum>
__global__ void __launch_bounds__(kSum ? kSumThreads : kThreads, 1) decay_walk_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Shared sh;
  __shared__ Found found;
  if (kSum || p.max_records == 0) griddep_wait();  // the first kernel of the call
  if constexpr (kSum) griddep_launch_dependents();
  const int wi = blockIdx.x % p.n_walks, h = blockIdx.x / p.n_walks % p.H, item = blockIdx.x / p.n_walks / p.H;
  const WalkParams& w = p.w[wi];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float g = used_log_decay(p.log_decay[h], p.wc.status);
  if (warp == 0) {
    bool valid;
    // Sequences that are not cut first: they are walked while the others' sums are taken.
    const int whole = kSum || p.L >= p.T ? 0 : count_whole(p.cu, p.N, p.T, p.L, lane);
    const FindWhat what = !kSum && p.L >= p.T     ? kSegments
                          : !kSum && item < whole ? kWholeSequences
                                                  : kSplitSegments;
    const Segment s = find_segment(p.cu, p.N, p.T, p.L, what, what == kSplitSegments ? item - whole : item, lane, valid);
    const bool last = kSum && s.seg == (w.reverse ? 0 : s.n_seg - 1), states = !kSum || last;
    const bool resumed = states && s.seq >= 0 && (!p.resume || p.resume[s.seq]);
    const int row = states && s.seq >= 0 && (w.init || w.fin)
                        ? pool_row(p.slots, s.seq, p.n_slots, w.fin != nullptr, lane, p.wc.status)
                        : -1;
    if (lane == 0) {
      if (!valid) report_status(p.wc.status, kStatusInvalidArg);
      found = Found{s.seq, s.s0, s.s1, s.seg, s.n_seg, s.t0, s.t1, s.rec, row,
                    resumed ? 1 : 0};
    }
  } else if (warp == 1) {
    tmem_alloc(&sh.tmem, kTmemCols);
  } else if (warp == 2) {
    if (lane == 0) {
      for (int s = 0; s < kMaxStages; ++s) {
        mbar_init(sh.full + s, 1);
        mbar_init(sh.late + s, 1);
        mbar_init(sh.staged + s, 256);
        mbar_init(sh.done + s, 1);
        mbar_init(sh.scaled + s, 256);
      }
      for (uint64_t* b : {&sh.p_full, &sh.a_done, &sh.rest_done, &sh.o_full, &sh.u_done, &sh.mma_done, sh.lo_free,
                          sh.lo_free + 1, sh.sum_done, sh.sum_done + 1})
        mbar_init(b, 1);
      for (uint64_t* b : {sh.sum_free, sh.sum_free + 1}) mbar_init(b, 128);
      mbar_init(&sh.s_init, 512);
      for (uint64_t* b : {&sh.s_copied, &sh.e_ready, &sh.w_full, &sh.hi_full, &sh.lo_full, &sh.last_full, &sh.o_free}) mbar_init(b, 256);
      sh.abort = 0;
      fence_barrier_init();
      fence_proxy_async_smem();
    }
  } else if (warp == 3) {
    if (lane == 0) {
      prefetch_tmap(&w.a);
      prefetch_tmap(&w.b);
      prefetch_tmap(&w.c);
      prefetch_tmap(&w.o);
      power_of(g, kChunk, sh.keep[0], sh.keep[1]);
      // rounded: up to 15 segments come to 3e-7 of the state in the mean square (what it leaves out, added here too,
      // takes 1% of a packed batch's time)
      sh.keep_segment = (float)exp((double)g * p.L);
    }
  } else if constexpr (!kSum) {
    for (int x = threadIdx.x - 128; x < 2 * kWeights; x += kThreads - 128) {
      const int y = first_weight(w.reverse) + x % kWeights + x / kWeights;
      sh.weight[x] = (w.reverse ? y >= 0 : y <= 0) ? w.s_intra * expf(g * fabsf((float)y)) : 0.f;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (found.seq >= 0) {
    auto run = [&](auto d1, auto d2) {
      if constexpr (kSum)
        sum_segment<decltype(d1)::value, decltype(d2)::value>(p, w, h, g, smem, sh, found);
      else
        walk<decltype(d1)::value, decltype(d2)::value>(p, w, h, g, smem, sh, found);
    };
    using A = std::integral_constant<int, DA>;
    using B = std::integral_constant<int, DB>;
    if (kSum && found.seg == last_walked(w, found))
      copy_init(w, found, p.H, h, w.swapped ? DB : DA, w.swapped ? DA : DB);
    else if (DA != DB && w.swapped)
      run(B(), A());
    else
      run(A(), B());
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(sh.tmem, kTmemCols);
  }
  // rows of out outside every sequence
  if (!kSum && p.zero_outside && found.seq >= 0) {
    const int units = (w.swapped ? DA : DB) / 8;
    auto clear = [&](int t0, int t1) {
#pragma unroll 1
      for (int t = t0 + (int)threadIdx.x / units; t < t1; t += kThreads / units)
        if ((int)threadIdx.x < kThreads / units * units)
          *reinterpret_cast<uint4*>(w.out + t * w.out_stride + (long long)h * units * 8 + threadIdx.x % units * 8) =
              make_uint4(0u, 0u, 0u, 0u);
    };
    if (found.seq == 0 && found.seg == 0) clear(0, found.s0);
    if (found.seq == p.N - 1 && found.seg == found.n_seg - 1) clear(found.s1, p.T);
  }
}

// The sums of a split sequence's segments become the states that enter them:
// E_first = init, E_next = a^(tokens) E + sum, in walking order.  One thread
// per four values; the sums of up to kAhead segments are in flight at once.
constexpr int kScanThreads = 256, kAhead = 8;

__global__ void __launch_bounds__(kScanThreads) decay_scan_kernel(const __grid_constant__ Params p, int d_a, int d_b) {
  __shared__ Found found;
  griddep_launch_dependents();
  const int part = d_a * d_b / 4 / kScanThreads, y = blockIdx.x / part;
  const int wi = y % p.n_walks, h = y / p.n_walks % p.H, item = y / p.n_walks / p.H;
  const WalkParams& w = p.w[wi];
  if (threadIdx.x < 32) {
    bool valid;
    const Segment g = find_segment(p.cu, p.N, p.T, p.L, kSplitSequences, item, threadIdx.x, valid);
    const int row = g.seq >= 0 && w.init
                        ? pool_row(p.slots, g.seq, p.n_slots, w.fin != nullptr, threadIdx.x, p.wc.status)
                        : -1;
    if (threadIdx.x == 0)
      found = Found{g.seq, g.s0, g.s1, g.seg, g.n_seg, g.t0, g.t1, g.rec, row,
                    g.seq >= 0 && (!p.resume || p.resume[g.seq]) ? 1 : 0};
  }
  __syncthreads();
  const Found f = found;
  if (f.seq < 0) {
    griddep_wait();  // a grid ends after those it was launched behind
    return;
  }
  const bool rev = w.reverse != 0;
  const int d1 = w.swapped ? d_b : d_a, d2 = w.swapped ? d_a : d_b;
  const int size4 = d1 * d2 / 4, x = blockIdx.x % part * kScanThreads + threadIdx.x;
  const float g = used_log_decay(p.log_decay[h], p.wc.status);
  float4 e = make_float4(0.f, 0.f, 0.f, 0.f);
  if (f.row >= 0 && f.resumed) {
    const float* src = w.init + ((long long)f.row * p.H + h) * (4ll * size4);
    if (w.init_transposed) {
      const int r = 4 * x / d2, c = 4 * x % d2;
      e = make_float4(src[c * d1 + r], src[(c + 1) * d1 + r], src[(c + 2) * d1 + r], src[(c + 3) * d1 + r]);
    } else {
      e = reinterpret_cast<const float4*>(src)[x];
    }
  }
  griddep_wait();
  auto at = [&](int s) {  // s-th segment walked
    const int seg = rev ? f.n_seg - 1 - s : s;
    return reinterpret_cast<float4*>(w.rec) + ((long long)(f.rec + seg) * p.H + h) * size4 + x;
  };
  float full, rest;
  power_of(g, p.L, full, rest);
  for (int s0 = 0; s0 < f.n_seg; s0 += kAhead) {
    float4 sum[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (s0 + u < f.n_seg - 1) sum[u] = *at(s0 + u);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (s0 + u >= f.n_seg) break;
      *at(s0 + u) = e;
      if (s0 + u < f.n_seg - 1) {
        const int seg = rev ? f.n_seg - 1 - s0 - u : s0 + u, tokens = min(p.L, f.s1 - f.s0 - seg * p.L);
        const float k = tokens == p.L ? full : expf(g * (float)tokens), r = tokens == p.L ? rest : 0.f;
        e = make_float4(fmaf(k, e.x, fmaf(r, e.x, sum[u].x)), fmaf(k, e.y, fmaf(r, e.y, sum[u].y)),
                        fmaf(k, e.z, fmaf(r, e.z, sum[u].z)), fmaf(k, e.w, fmaf(r, e.w, sum[u].w)));
      }
    }
  }
}

// fin = init or zero, for sequences without tokens (T = 0); the states of many
// heads are more tiles than a grid has rows
constexpr int kEmptyThreads = 256, kMaxGridRows = 65535;

__global__ void __launch_bounds__(kEmptyThreads) decay_empty_kernel(const float* init, float* fin, const int* slots,
                                                                    int n_slots, const unsigned char* resume,
                                                                    long long size4, int* status) {
  const int n = blockIdx.x;
  const int row = pool_row(slots, n, n_slots, true, threadIdx.x & 31, status);
  if (row < 0) return;
  const bool entered = init && (!resume || resume[n]);
  for (long long x = (long long)blockIdx.y * kEmptyThreads + threadIdx.x; x < size4;
       x += (long long)gridDim.y * kEmptyThreads)
    reinterpret_cast<float4*>(fin)[row * size4 + x] =
        entered ? reinterpret_cast<const float4*>(init)[row * size4 + x] : make_float4(0.f, 0.f, 0.f, 0.f);
}

// [T][H][width] with `stride` elements between tokens, box [128 tokens][1 head][64 values], 128-byte swizzle
bool make_tmap(CUtensorMap* map, const void* base, int width, int H, int T, long long stride) {
  typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                               const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const EncodeFn enc = []() -> EncodeFn {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &qr) != cudaSuccess ||
        qr != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<EncodeFn>(fn);
  }();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)H, (cuuint64_t)T};
  const cuuint64_t strides[2] = {(cuuint64_t)width * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, 1, kChunk};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How sequences are cut.  The lengths are on the device; the plan knows T, N,
// the heads and the walks, and takes the length of segments that would be best
// for sequences of equal length: a CTA per segment, waves of 148.  In units of
// half a chunk's walk (measured: 1.6 us at d = dv = 128; a chunk's sum takes
// one): kStart for a CTA's start and end, and where anything is cut kCut for
// two more launches, with the sums.  Segments are not shorter than an even
// share of the whole, so that of sequences that differ only those are cut that
// would outlast the rest; and several short sequences (up to kUncut chunks
// together) never, as even two more launches that find nothing to do cost
// 6 us (a call of 1337 tokens in 5 sequences 37 us instead of 27).
//
// kUncut measured, cut against not, calls of 2, 5 and 12 sequences of very unequal
// lengths, 2 to 24 heads, us: 10 chunks together, two sequences of 2 and 8 heads at
// d = dv = 64 19.4 and 19.8 against 20.3 and 20.6 (gradients of 2 heads 17.4, 18.8),
// all others lose by cutting, up to 60% (128, 24 heads, gradients: 43.8, 27.2).
// 12 chunks: two sequences 20.7
// against 24.8 (d = dv = 64) and 34.8 against 34.4 (128), five 19.9 against 15.9
// and 28.7 against 22.0.  14 chunks: two 24.1 against 38.1 and 41.6 against 51.8,
// five 22.3 against 26.8 and 35.5 against 37.0, twelve 18.8 against 15.8 and 30.5
// against 21.7.  What decides is the longest sequence (cutting pays from 8 chunks
// on at 64, from 9 at 128, if few heads leave SMs free), which the plan does not
// know.
struct Plan {
  int L;              // tokens per segment, a multiple of 128
  int max_segments;   // of all sequences together
  int max_records;    // of split sequences
};

// Up to kFold segments of a sequence a walk sums the records before its own
// itself (each costs it about half a microsecond, the scan a launch of 7 us).
constexpr int kSMs = 148, kMinSegment = 2, kUncut = 12, kStart = 4, kCut = 5, kFold = 16;

Plan make_plan(int T, int H, int N, int walks) {
  const long long heads = (long long)H * walks;
  const long long chunks = ((long long)T + kChunk - 1) / kChunk;
  const long long len = std::max(((long long)T / N + kChunk - 1) / kChunk, 1ll);  // chunks of an even sequence
  long long best = -1, k_best = 1;
  for (long long k = len; k >= 1; k = k > 64 ? k - k / 32 : k - 1) {
    const long long segs = (len + k - 1) / k, waves = (segs * N * heads + kSMs - 1) / kSMs;
    const long long cost = waves * (2 * k + kStart) + (segs > 1 ? waves * k + kCut : 0);
    if (best < 0 || cost < best) {
      best = cost;
      k_best = k;
    }
  }
  long long k = std::max(k_best, (long long)kMinSegment);
  if (N > 1) k = std::max(k, chunks <= kUncut ? chunks : (chunks + N) * heads / kSMs);
  Plan pl;
  pl.L = (int)std::min(k * kChunk, 1ll << 30);
  pl.max_segments = N + T / pl.L;
  pl.max_records = T > pl.L ? T / pl.L + std::min(N, T / pl.L) : 0;
  return pl;
}

// The kernel's dynamic shared memory, set once per context (it took 1 us of every call).
template <int DA, int DB, bool kSum>
cudaError_t allow_shared(int bytes) {
  static std::atomic<void*> set{nullptr};
  void* ctx = current_context();
  if (ctx && set.load(std::memory_order_acquire) == ctx) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(decay_walk_kernel<DA, DB, kSum>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) set.store(current_context(), std::memory_order_release);
  return e;
}

template <int DA, int DB>
cudaError_t launch(const Params& p, const Plan& pl, cudaStream_t st) {
  constexpr int bytes = Cfg<DA, DB>::kBytes > Cfg<DB, DA>::kBytes ? Cfg<DA, DB>::kBytes : Cfg<DB, DA>::kBytes;
  cudaError_t e = allow_shared<DA, DB, false>(bytes);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)pl.max_segments * p.H * p.n_walks);
  auto walks = [&] { return launch_pdl(decay_walk_kernel<DA, DB, false>, grid, dim3(kThreads), (size_t)bytes, st, p); };
  if (pl.max_records == 0) return walks();
  if ((e = allow_shared<DA, DB, true>(bytes)) != cudaSuccess) return e;
  e = launch_pdl(decay_walk_kernel<DA, DB, true>, dim3((unsigned)pl.max_records * p.H * p.n_walks), dim3(kSumThreads),
                 (size_t)bytes, st, p);
  if (e != cudaSuccess) return e;
  if (p.folded) return walks();
  const dim3 scan(DA * DB / 4 / kScanThreads * (unsigned)std::min(p.N, p.T / pl.L) * p.H * p.n_walks);
  e = launch_pdl(decay_scan_kernel, scan, dim3(kScanThreads), 0, st, p, DA, DB);
  if (e != cudaSuccess) return e;
  return walks();
}

}  // namespace

size_t decay_workspace_bytes(int T, int H, int d1, int d2, int N, int walks) {
  return (size_t)walks * make_plan(T, H, N, walks).max_records * H * d1 * d2 * sizeof(float);
}

cudaError_t launch_decay_walks(const DecayWalk* walks, int n, const DecayShape& sh, void* ws, const WaitCtl& wc,
                               cudaStream_t st) {
  if (n < 1 || n > kMaxWalks) return cudaErrorInvalidValue;
  const Plan pl = make_plan(sh.T, sh.H, sh.N, n);
  Params p{};
  const int da = walks[0].d1, db = walks[0].d2;
  for (int i = 0; i < n; ++i) {
    const DecayWalk& x = walks[i];
    WalkParams& w = p.w[i];
    if (!make_tmap(&w.a, x.a, x.d1, sh.H, sh.T, x.a_stride) || !make_tmap(&w.b, x.b, x.d1, sh.H, sh.T, x.b_stride) ||
        !make_tmap(&w.c, x.c, x.d2, sh.H, sh.T, x.c_stride) ||
        !make_tmap(&w.o, x.out, x.d2, sh.H, sh.T, x.out_stride))
      return cudaErrorInvalidValue;
    w.out = static_cast<__nv_bfloat16*>(x.out);
    w.out_stride = x.out_stride;
    w.init = x.init;
    w.fin = x.fin;
    w.rec = static_cast<float*>(ws) + (size_t)i * pl.max_records * sh.H * x.d1 * x.d2;
    w.swapped = x.d1 != da;
    w.reverse = x.reverse;
    w.init_transposed = x.init_transposed;
    w.s_intra = sh.scale;
    w.s_inter = x.reverse ? 1.f : sh.scale;
    w.s_key = x.reverse ? sh.scale : 1.f;
  }
  p.cu = sh.cu;
  p.log_decay = sh.log_decay;
  p.slots = sh.slots;
  p.resume = sh.resume;
  p.n_walks = n;
  p.T = sh.T;
  p.H = sh.H;
  p.N = sh.N;
  p.L = pl.L;
  p.folded = sh.T / pl.L < kFold;
  p.max_records = pl.max_records;
  p.n_slots = sh.n_slots;
  p.zero_outside = sh.zero_outside;
  p.wc = wc;
  if (da == 64 && db == 64) return launch<64, 64>(p, pl, st);
  if (da == 128 && db == 128) return launch<128, 128>(p, pl, st);
  if (da == 64) return launch<64, 128>(p, pl, st);
  return launch<128, 64>(p, pl, st);
}

cudaError_t launch_decay_empty(const DecayWalk& w, const DecayShape& sh, const WaitCtl& wc, cudaStream_t st) {
  if (!w.fin) return cudaSuccess;
  const long long size4 = (long long)sh.H * w.d1 * w.d2 / 4;
  const long long tiles = std::min((size4 + kEmptyThreads - 1) / kEmptyThreads, (long long)kMaxGridRows);
  decay_empty_kernel<<<dim3((unsigned)sh.N, (unsigned)tiles), kEmptyThreads, 0, st>>>(
      w.init, w.fin, sh.slots, sh.n_slots, sh.resume, size4, wc.status);
  return cudaGetLastError();
}

}  // namespace kata
