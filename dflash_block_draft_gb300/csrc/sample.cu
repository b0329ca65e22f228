// sample.cu -- a token of every row of logits by temperature, top-k, top-p and min-p, with
// given random numbers, and the filtered distribution itself where it is wanted (sm_103a).
//
// Per row, with m the largest logit and w_i = exp((l_i - m) / T): the tokens in the order
// of their logits, equal ones in the order of their numbers; the first top_k of them; of
// those the shortest beginning with a sum of at least top_p of theirs; of those the ones
// with w_i >= min_p.  What is kept is then everything down to one place of that order (the
// "cut", a logit and a token's number), and the token is the first one, in the order of the
// numbers, whose running sum of kept weights exceeds u times the whole.
//
// A cluster of 1 to 8 CTAs takes a row and holds it in shared memory: the logits are
// read from memory once.  There
//   the largest logit;
//   top-k: a histogram of counts over 2048 equal steps of the logit, from the largest one
//     down to the smallest of the threads' maxima (as many tokens as there are threads lie
//     above it), merged through distributed shared memory; the tokens in the step where
//     the count is reached go into a list (at most 256; else the step is divided again, by the
//     bits of logit and number, so that ties divide too), whose order is found by comparing
//     all pairs;
//   top-p: the same with weights instead of counts, over the steps down to where weights
//     end (31.2 T);
//   the kept weights' sums by runs of tokens, one exchange, and the run that passes u times
//     the whole once more, a few tokens a thread.
//
// Weights are whole steps of 2^-44 of the largest one, added up as 64-bit integers, so that
// no sum depends on the order, the number of CTAs or the threads' timing, and the cut and the
// token are those of the real numbers unless a border lies within about 2^-38 of the
// sum (fp32 sums would draw another token in every fiftieth row of a vocabulary of
// 131072).  A weight costs 23 packed fp32 instructions for two tokens and about 15 integer
// ones for each: l - m as two floats, times log2(e) / T as two floats; 2^y from a table of
// 2^(j / 128) and a polynomial of degree 4, in fixed point from there on.  64-bit
// floating point runs at a hundredth of that rate here.
#include <cooperative_groups.h>
#include <limits.h>
#include <math.h>
#include <stddef.h>

#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace dflash {
namespace {

namespace cg = cooperative_groups;
typedef unsigned long long u64;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;       // of a histogram: 4 a thread
constexpr int kList = 256;        // tokens whose order is found by comparing all pairs
constexpr int kMaxCluster = 8;
constexpr int kIndexBits = 19;    // of a token's number
constexpr uint32_t kIndexMask = (1u << kIndexBits) - 1;
constexpr int kChunkMax = 49152;  // logits a CTA can hold
static_assert(DFLASH_SAMPLE_MAX_V <= kMaxCluster * kChunkMax && DFLASH_SAMPLE_MAX_V <= (int)kIndexMask + 1, "vocabulary");
static_assert(kBins == 4 * kThreads && kThreads >= 2 * kList, "thread layout");
constexpr float kTop = 3.402823466e+38f;  // the largest finite logit; +inf counts as that

// ------------------------------------------------------------------ weights
// 2^(j / 128) in steps of 2^-45.
struct Powers {
  u64 at[128];
};
constexpr Powers make_powers() {
  Powers p = {};
  for (int j = 0; j < 128; ++j) {
    // the series of e^x: its terms fall below 2^-60 of the sum
    const long double x = 0.693147180559945309417232121458L * j / 128;
    long double t = 1, s = 1;
    for (int k = 1; k < 30; ++k) {
      t = t * x / k;
      s += t;
    }
    p.at[j] = (u64)(s * 35184372088832.0L + 0.5L);
  }
  return p;
}
__device__ constexpr Powers kPowers = make_powers();

struct Scale {
  float m, ch, cl;  // the largest logit; log2(e) / T as ch + cl
};

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// From the bits of the three sums below: 2^y in steps of 2^-44, rounded, y = raw / 128 + z.
__device__ __forceinline__ u64 power(const u64* tab, int raw, int zi, int rest) {
  const u64 t = tab[raw & 127];
  const int n = -(raw >> 7);
  // 2^z - 1 in steps of 2^-39: z ln 2 exactly enough, and the rest of the series
  const int s = (int)(((long long)zi * 1488522236) >> 16) + rest;  // (ln 2 * 2^31)
  const u64 w = t + (u64)(((long long)(int)(t >> 15) * s) >> 24);
  return ((w >> (n & 63)) + 1) >> 1;
}

// Weights of two logits.  What lies more than 45 powers of two below m, or is no number,
// gives anything: the caller looks at the logit.
__device__ __forceinline__ void weights(const Scale& c, const u64* tab, float2 l, u64& w0, u64& w1) {
  const float2 neg = both(-1.f), nm = both(-c.m), ch = both(c.ch);
  // l - m = d + err exactly (the two-sum of Moller and Knuth)
  const float2 d = __fadd2_rn(l, nm), bb = __ffma2_rn(l, neg, d);
  const float2 err = __fadd2_rn(__ffma2_rn(__ffma2_rn(bb, neg, d), neg, l), __ffma2_rn(bb, neg, nm));
  // y = -np + e
  const float2 np = __fmul2_rn(d, both(-c.ch));
  const float2 e = __ffma2_rn(err, ch, __ffma2_rn(d, both(c.cl), __ffma2_rn(d, ch, np)));
  // whole steps of 1/128 by the adder's bits, and what remains, r = -rn
  const float big = 0x1.8p16f;
  const float2 t1 = __ffma2_rn(np, neg, both(big));
  const float2 rn = __fadd2_rn(np, __fadd2_rn(t1, both(-big)));
  const float2 z = __ffma2_rn(rn, neg, e);
  // r in steps of 2^-24, and the tail
  const float half = 0.75f;
  const float2 t2 = __ffma2_rn(rn, neg, both(half));
  const float2 tail = __ffma2_rn(__fadd2_rn(rn, __fadd2_rn(t2, both(-half))), neg, e);
  // 2^z - 1 - r ln 2: the tail's part and z^2 (c2 + z (c3 + z c4)), in steps of 2^-39
  const float tiny = 0x1.8p-16f;
  const float2 q = __ffma2_rn(__ffma2_rn(z, both(9.618129107e-3f), both(5.550410867e-2f)), z, both(2.402265070e-1f));
  const float2 t3 = __ffma2_rn(q, __fmul2_rn(z, z), __ffma2_rn(tail, both(0.6931471806f), both(tiny)));
  const int b1 = __float_as_int(big), b2 = __float_as_int(half), b3 = __float_as_int(tiny);
  w0 = power(tab, __float_as_int(t1.x) - b1, __float_as_int(t2.x) - b2, __float_as_int(t3.x) - b3);
  w1 = power(tab, __float_as_int(t1.y) - b1, __float_as_int(t2.y) - b2, __float_as_int(t3.y) - b3);
}

// The weight as a float, for the distribution: 2^(fraction) times the power of two.
__device__ __forceinline__ float weight_f32(const Scale& c, float l) {
  const float d = l - c.m, p = d * c.ch;
  const float n = rintf(p);
  const float f = fmaf(d, c.cl, fmaf(d, c.ch, -n));
  return n < -140.f ? 0.f : ldexpf(exp2f(f), (int)n);
}

// ------------------------------------------------------------------ order
// A token's place in the order, the larger the earlier: the logit's bits, made to ascend,
// then the number.  (x + 0 turns -0 into +0: equal logits are equal here.)
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t b = __float_as_uint(l + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
__device__ __forceinline__ u64 place_of(uint32_t key, int i) { return ((u64)key << kIndexBits) | (kIndexMask - (uint32_t)i); }

// Everything down to token i of logit v is kept.
struct Cut {
  float v;
  int i;
  __device__ __forceinline__ bool keeps(float l, int k) const { return l > v || (l == v && k <= i); }
};

// ------------------------------------------------------------------ a row in shared memory
template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
};
// The N logits of one 16-byte vector.
__device__ __forceinline__ void unpack(const uint4& v, float (&x)[4]) {
  x[0] = __uint_as_float(v.x);
  x[1] = __uint_as_float(v.y);
  x[2] = __uint_as_float(v.z);
  x[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
// NaN becomes -inf, +inf the largest finite value of the type.
__device__ __forceinline__ uint32_t tidy(uint32_t w, float) {
  return __float_as_uint(fminf(fmaxf(__uint_as_float(w), -INFINITY), kTop));
}
__device__ __forceinline__ uint32_t tidy(uint32_t w, __nv_bfloat16) {
  __nv_bfloat162 x = *reinterpret_cast<__nv_bfloat162*>(&w);
  const __nv_bfloat16 lo = __ushort_as_bfloat16(0xFF80), hi = __ushort_as_bfloat16(0x7F7F);
  x = __hmin2(__hmax2(x, __nv_bfloat162(lo, lo)), __nv_bfloat162(hi, hi));
  return *reinterpret_cast<uint32_t*>(&x);
}

struct Row {
  // what a CTA tells the others
  float max, low;     // largest logit; smallest of the threads' maxima
  int groups;         // threads that have logits
  int best;           // the first token with the row's largest logit (greedy)
  int listed;         // tokens of the range
  uint32_t key_lo, key_hi;  // their keys
  u64 sum;            // kept weights
  u64 list[kList];
  // its own
  alignas(16) uint32_t lo[kBins];  // counts, or the weights' lower
  alignas(16) uint32_t hi[kBins];  // and upper halves
  u64 tab[128];
  u64 scan[kWarps];
  u64 all[kList], all_w[kList];
  float f[kWarps], g[kWarps];
  u64 found_before;
  int found;
  u64 cut;
  Scale scale;
  float ends, least;  // no weight below `ends`; min-p's bound
  double bar;
};

static_assert(offsetof(Row, lo) % 16 == 0 && offsetof(Row, hi) % 16 == 0, "histograms are read in 16-byte pieces");

template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Exclusive sum over the block's threads; *total is the whole.
__device__ __forceinline__ u64 block_scan(u64 v, u64* scratch, u64* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 c = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 u = __shfl_up_sync(0xffffffffu, c, o);
    if (lane >= o) c += u;
  }
  __syncthreads();  // scratch of an earlier call has been read
  if (lane == 31) scratch[warp] = c;
  __syncthreads();
  u64 before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    before += w < warp ? scratch[w] : 0;
    all += scratch[w];
  }
  *total = all;
  return before + c - v;
}

template <typename T>
struct Pass {
  static constexpr int N = Vec<T>::N;
  const uint4* chunk;
  int run;    // logits of a warp's run
  int first;  // number of the chunk's first token
  // body(x, i): N logits, the first of which is token i's, for the whole warp at a time
  template <typename Body>
  __device__ __forceinline__ void each(Body body) const {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int k = lane * N; k < run; k += 32 * N) {
      float x[N];
      unpack(chunk[(warp * run + k) / N], x);
      body(x, first + warp * run + k);
    }
  }
};

// The cut of top-k (WEIGHTS false; target: k) or top-p (true; target from `share` of the
// whole): the token of `prior`'s in which the running count or weight reaches the target.
// The first division is by equal steps of the logit from m down to `bound`; without a
// bound it is by the bits.  Returns prior where there are fewer tokens than k.
template <bool WEIGHTS, typename T>
__device__ __forceinline__ Cut select(const Pass<T>& pass, Row& s, cg::cluster_group& cluster, const Cut& prior,
                                      const Scale sc, float bound, float range, u64 target, double share) {
  constexpr int N = Vec<T>::N;
  const int tid = threadIdx.x, lane = tid & 31, ranks = (int)cluster.num_blocks();
  const float m = sc.m;
  u64 before = 0;             // count or weight in front of the range
  int bin = -1;               // the step that the range is, -1: none (the places below say)
  u64 lo = 0, hi = ~0ull;     // the range's places
  bool linear = range > 0.f;
  const float step = linear ? kBins / range : 0.f;
  auto bin_of = [&](float l) { return min(kBins - 1, (int)((m - l) * step)); };
  bool divide = WEIGHTS || linear;
  int shift = 0;
  for (;;) {
    if (divide) {
      // ---- a histogram of the range
      *reinterpret_cast<uint4*>(&s.lo[4 * tid]) = make_uint4(0, 0, 0, 0);
      if (WEIGHTS) *reinterpret_cast<uint4*>(&s.hi[4 * tid]) = make_uint4(0, 0, 0, 0);
      __syncthreads();
      pass.each([&](const float (&x)[N], int i) {
        bool in[N];
        bool any = false;
#pragma unroll
        for (int k = 0; k < N; ++k) {
          in[k] = x[k] >= bound && prior.keeps(x[k], i + k);
          if (!linear && in[k]) {
            const u64 p = place_of(key_of(x[k]), i + k);
            in[k] = p >= lo && p <= hi;
          }
          any |= in[k];
        }
        if (!any) return;
#pragma unroll
        for (int k = 0; k < N; k += 2) {
          u64 w[2] = {0, 0};
          if (WEIGHTS && (in[k] || in[k + 1])) weights(sc, s.tab, make_float2(x[k], x[k + 1]), w[0], w[1]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (!in[k + e]) continue;
            const int b = linear ? bin_of(x[k + e]) : (int)((hi - place_of(key_of(x[k + e]), i + k + e)) >> shift);
            if (WEIGHTS) {
              const uint32_t wl = (uint32_t)w[e];
              const uint32_t wh = (uint32_t)(w[e] >> 32) + (atomicAdd(&s.lo[b], wl) + wl < wl);
              if (wh) atomicAdd(&s.hi[b], wh);
            } else {
              atomicAdd(&s.lo[b], 1u);
            }
          }
        }
      });
      cluster.sync();
      // ---- merged, every CTA for itself
      u64 v[4] = {0, 0, 0, 0};
      for (int c = 0; c < ranks; ++c) {
        const uint4 a = *reinterpret_cast<const uint4*>(cluster.map_shared_rank(&s.lo[4 * tid], c));
        uint4 b = make_uint4(0, 0, 0, 0);
        if (WEIGHTS) b = *reinterpret_cast<const uint4*>(cluster.map_shared_rank(&s.hi[4 * tid], c));
        v[0] += ((u64)b.x << 32) + a.x;
        v[1] += ((u64)b.y << 32) + a.y;
        v[2] += ((u64)b.z << 32) + a.z;
        v[3] += ((u64)b.w << 32) + a.w;
      }
      u64 total;
      u64 at = before + block_scan(v[0] + v[1] + v[2] + v[3], s.scan, &total);
      if (WEIGHTS && target == 0) target = max(1ull, min(total, (u64)__dmul_ru(share, (double)total)));
      if (!WEIGHTS && before + total < target) return prior;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (at < target && target <= at + v[k]) {  // one thread
          s.found = 4 * tid + k;
          s.found_before = at;
        }
        at += v[k];
      }
      __syncthreads();
      bin = s.found;
      before = s.found_before;
      if (!linear) {
        hi -= (u64)bin << shift;
        lo = max(lo, hi - ((1ull << shift) - 1));
      }
    }
    // ---- the range's tokens, as far as there is room for them
    if (tid == 0) {
      s.listed = 0;
      s.key_lo = ~0u;
      s.key_hi = 0;
    }
    __syncthreads();
    uint32_t klo = ~0u, khi = 0;
    pass.each([&](const float (&x)[N], int i) {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if (!(x[k] >= bound && prior.keeps(x[k], i + k))) continue;
        const uint32_t key = key_of(x[k]);
        const u64 p = place_of(key, i + k);
        if (linear && bin >= 0 ? bin_of(x[k]) != bin : p < lo || p > hi) continue;
        klo = min(klo, key);
        khi = max(khi, key);
        const int at = atomicAdd(&s.listed, 1);
        if (at < kList) s.list[at] = p;
      }
    });
    klo = __reduce_min_sync(0xffffffffu, klo);
    khi = __reduce_max_sync(0xffffffffu, khi);
    if (lane == 0 && khi) {
      atomicMin(&s.key_lo, klo);
      atomicMax(&s.key_hi, khi);
    }
    cluster.sync();
    int n = 0, owner = -1, slot = 0;
    klo = ~0u;
    khi = 0;
    for (int c = 0; c < ranks; ++c) {
      const int k = *cluster.map_shared_rank(&s.listed, c);
      klo = min(klo, *cluster.map_shared_rank(&s.key_lo, c));
      khi = max(khi, *cluster.map_shared_rank(&s.key_hi, c));
      if (tid >= n && tid < n + k) {
        owner = c;
        slot = tid - n;
      }
      n += k;
    }
    if (n == 0) return prior;  // (a row without weights, or with fewer tokens than k)
    if (n <= kList) {
      u64 mine = 0;
      if (tid < n) {
        mine = cluster.map_shared_rank(s.list, owner)[slot];
        s.all[tid] = mine;
        if (WEIGHTS) {
          u64 w0, w1;
          const float l = logit_of((uint32_t)(mine >> kIndexBits));
          weights(sc, s.tab, both(l), w0, w1);
          s.all_w[tid] = w0;
        }
      }
      __syncthreads();
      // two threads a token
      const int i = tid >> 1;
      u64 sum = 0;
      if (i < n) {
        const u64 p = s.all[i];
        for (int j = tid & 1; j < n; j += 2)
          if (s.all[j] > p) sum += WEIGHTS ? s.all_w[j] : 1ull;
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      if (i < n) {
        const u64 at = before + sum, w = WEIGHTS ? s.all_w[i] : 1ull;
        if (at < target && target <= at + w) s.cut = s.all[i];
        // fewer than k tokens in all: down to the last one
        if (!WEIGHTS && before + n < target && sum == n - 1ull) s.cut = s.all[i];
      }
      __syncthreads();
      const u64 p = s.cut;
      return Cut{logit_of((uint32_t)(p >> kIndexBits)), (int)(kIndexMask - (uint32_t)(p & kIndexMask))};
    }
    // ---- too many: the range between its keys is divided again
    hi = min(hi, place_of(khi, 0));
    lo = max(lo, (u64)klo << kIndexBits);
    shift = max(0, 64 - __clzll((long long)(hi - lo)) - 11);
    linear = false;
    divide = true;
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a) {
  constexpr int N = Vec<T>::N;
  extern __shared__ __align__(16) uint4 chunk[];
  __shared__ __align__(16) Row s;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int r = blockIdx.x / ranks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* row = static_cast<const T*>(a.x) + r * a.xs;
  Pass<T> pass;
  pass.chunk = chunk;
  pass.run = a.chunk / kWarps;
  pass.first = rank * a.chunk;
  const float temp = a.temp ? a.temp[r] : 1.f;
  const float top_p = a.top_p ? a.top_p[r] : 1.f, min_p = a.min_p ? a.min_p[r] : 0.f, u = a.u[r];
  const int top_k = a.top_k ? a.top_k[r] : 0;

  // ---- the row comes in
  float mine = -INFINITY;
  bool have = false;
#pragma unroll 4
  for (int k = lane * N; k < pass.run; k += 32 * N) {
    const int at = warp * pass.run + k, i = pass.first + at;
    uint4 v;
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
    if (VEC) {
      constexpr uint32_t none = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;
      v = make_uint4(none, none, none, none);
      if (i < a.V) v = __ldcs(reinterpret_cast<const uint4*>(row + i));
    } else {
      alignas(16) T e[N];
#pragma unroll
      for (int j = 0; j < N; ++j) e[j] = i + j < a.V ? row[i + j] : from_f32<T>(-INFINITY);
      v = *reinterpret_cast<uint4*>(e);
    }
    have |= i < a.V;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = tidy(w[j], T());
    chunk[at / N] = v;
    float x[N];
    unpack(v, x);
#pragma unroll
    for (int j = 0; j < N; ++j) mine = fmaxf(mine, x[j]);
  }
  if (tid < 128) s.tab[tid] = kPowers.at[tid];
  {
    float hi = mine, lo = have ? mine : INFINITY;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    }
    if (lane == 0) {
      s.f[warp] = hi;
      s.g[warp] = lo;
    }
  }
  const int groups = __syncthreads_count(have);
  if (tid == 0) {
    float hi = s.f[0], lo = s.g[0];
    for (int w = 1; w < kWarps; ++w) {
      hi = fmaxf(hi, s.f[w]);
      lo = fminf(lo, s.g[w]);
    }
    s.max = hi;
    s.low = lo;
    s.groups = groups;
  }
  cluster.sync();
  float m = -INFINITY, low = INFINITY;
  int threads = 0;
  for (int c = 0; c < ranks; ++c) {
    m = fmaxf(m, *cluster.map_shared_rank(&s.max, c));
    low = fminf(low, *cluster.map_shared_rank(&s.low, c));
    threads += *cluster.map_shared_rank(&s.groups, c);
  }
  const bool bad = !(temp >= 0.f) || isinf(temp);
  const bool none = bad || m == -INFINITY;  // nothing to choose from
  int token = -1;                           // known to one thread of the cluster
  Cut cut = {-kTop, (int)kIndexMask};
  u64 total = 0;
  if (none) {
    if (rank == 0 && tid == 0) {
      record_error(a.err, DFLASH_ERR_INVALID);
      token = 0;
    }
    cut.v = INFINITY;
  } else if (temp == 0.f) {
    // ---- the first of the largest
    if (tid == 0) s.best = INT_MAX;
    __syncthreads();
    int best = INT_MAX;
    pass.each([&](const float (&x)[N], int i) {
#pragma unroll
      for (int k = N - 1; k >= 0; --k)
        if (x[k] == m) best = min(best, i + k);
    });
    best = (int)__reduce_min_sync(0xffffffffu, (unsigned)best);
    if (lane == 0) atomicMin(&s.best, best);
    cluster.sync();
    best = INT_MAX;
    for (int c = 0; c < ranks; ++c) best = min(best, *cluster.map_shared_rank(&s.best, c));
    if (rank == 0 && tid == 0) token = best;
    cut.v = m;
    cut.i = best;
  } else {
    if (tid == 0) {
      const double t = fmax((double)temp, 0x1p-100), c = 1.4426950408889634074 / t;
      s.scale.m = m;
      s.scale.ch = (float)c;
      s.scale.cl = (float)(c - (double)(float)c);
      // 45 powers of two below m weights are less than half a step
      s.ends = __double2float_ru((double)m - 31.191623125 * t);
      s.least = min_p > 0.f ? __double2float_ru((double)m + log(min((double)min_p, 1.0)) * t) : -kTop;
    }
    __syncthreads();
    const Scale sc = s.scale;
    const float ends = fmaxf(s.ends, -kTop), least = s.least;
    if (top_k > 0 && top_k < a.V) {
      const bool known = top_k <= threads && low > -INFINITY;
      const float bound = known ? low : -kTop;
      cut = select<false, T>(pass, s, cluster, cut, sc, bound, known ? fminf(fmaxf(m - low, 1e-30f), kTop) : 0.f, top_k, 0.);
    }
    if (top_p < 1.f) {
      const float bound = fmaxf(ends, cut.v);
      if (top_k > 0) cluster.sync();  // the other CTAs have read this one's list and histogram
      cut = select<true, T>(pass, s, cluster, cut, sc, bound, fminf(fmaxf(m - bound, 1e-30f), kTop), 0,
                            (double)top_p);
    }
    if (least > cut.v) {
      cut.v = least;
      cut.i = (int)kIndexMask;
    }
    // ---- the kept weights
    u64 sum = 0;
    pass.each([&](const float (&x)[N], int i) {
      bool in[N];
      bool any = false;
#pragma unroll
      for (int k = 0; k < N; ++k) any |= in[k] = x[k] >= ends && cut.keeps(x[k], i + k);
      if (!any) return;
#pragma unroll
      for (int k = 0; k < N; k += 2) {
        u64 w0, w1;
        weights(sc, s.tab, make_float2(x[k], x[k + 1]), w0, w1);
        sum += (in[k] ? w0 : 0) + (in[k + 1] ? w1 : 0);
      }
    });
    sum = warp_sum(sum);
    __syncthreads();  // scan of an earlier pass has been read
    if (lane == 0) s.scan[warp] = sum;
    __syncthreads();
    u64 own = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) own += s.scan[w];
    if (tid == 0) s.sum = own;
    cluster.sync();
    u64 before = 0;
    for (int c = 0; c < ranks; ++c) {
      const u64 x = *cluster.map_shared_rank(&s.sum, c);
      before += c < rank ? x : 0;
      total += x;
    }
    // sums are whole numbers: one exceeds u * total where it exceeds its floor
    const u64 bar = (u64)__dmul_rd((double)fminf(fmaxf(u, 0.f), 0x1.fffffep-1f), (double)total);
    if (before <= bar && bar < before + own) {  // one CTA
      int w = 0;
      while (before + s.scan[w] <= bar) before += s.scan[w++];
      // the warp's run once more, a few tokens in a row a thread
      const int per = (pass.run + kThreads - 1) / kThreads;
      const T* logits = reinterpret_cast<const T*>(chunk) + w * pass.run;
      const int at = tid * per, i = pass.first + w * pass.run + at;
      auto weight = [&](int k) -> u64 {
        if (at + k >= pass.run) return 0;
        const float l = to_f32(logits[at + k]);
        u64 w0, w1;
        weights(sc, s.tab, both(l), w0, w1);
        return l >= ends && cut.keeps(l, i + k) ? w0 : 0;
      };
      u64 sum = 0, all;
      for (int k = 0; k < per; ++k) sum += weight(k);
      u64 c = before + block_scan(sum, s.scan, &all);
      if (c <= bar && bar < c + sum)  // one thread
        for (int k = 0; token < 0; ++k) {
          c += weight(k);
          if (c > bar) token = i + k;
        }
    }
  }
  if (token >= 0) a.tokens[r] = token;
  if (a.probs) {
    float* out = a.probs + r * a.ps;
    const Scale sc = none || temp == 0.f ? Scale{0.f, 0.f, 0.f} : s.scale;
    float inv = 1.f;
    if (total) {
      __syncthreads();
      if (tid == 0) s.bar = 0x1p44 / (double)total;
      __syncthreads();
      inv = (float)s.bar;
    }
    pass.each([&](const float (&x)[N], int i) {
      float p[N];
#pragma unroll
      for (int k = 0; k < N; ++k) p[k] = cut.keeps(x[k], i + k) ? weight_f32(sc, x[k]) * inv : 0.f;
      if (a.probs_vec) {
#pragma unroll
        for (int k = 0; k < N; k += 4)
          if (i + k < a.V) __stcs(reinterpret_cast<float4*>(out + i + k), make_float4(p[k], p[k + 1], p[k + 2], p[k + 3]));
      } else {
#pragma unroll
        for (int k = 0; k < N; ++k)
          if (i + k < a.V) out[i + k] = p[k];
      }
    });
  }
  cluster.sync();  // no CTA leaves while another may still read what it tells
}

template <typename T, bool VEC>
cudaError_t run(const SampleArgs& a, int ranks, size_t smem, cudaStream_t stream) {
  auto kernel = sample_kernel<T, VEC>;
  static std::atomic<uint64_t> ready{0};  // devices whose kernel has its shared memory's size
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev >= 64 || !(ready.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(kChunkMax * sizeof(T)));
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)ranks;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)a.N * ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, a);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_sample(SampleArgs a, bool bf16, cudaStream_t stream) {
  const int esz = bf16 ? 2 : 4, n = 16 / esz;
  const bool vec = a.V % n == 0 && ((uintptr_t)a.x & 15u) == 0 && (a.N == 1 || a.xs % n == 0);
  a.probs_vec = a.V % 4 == 0 && ((uintptr_t)a.probs & 15u) == 0 && (a.N == 1 || a.ps % 4 == 0);
  // CTAs a row: as few as hold a share of 64 KB (two CTAs an SM, so that one row comes in
  // while another is worked on), more while the launch stays within one wave.
  auto chunk_of = [&](int ranks) {
    const int unit = kThreads * n;
    return ((a.V + ranks - 1) / ranks + unit - 1) / unit * unit;
  };
  int ranks = 1;
  while (ranks < kMaxCluster && chunk_of(ranks) * esz > 65536) ranks *= 2;
  while (ranks < kMaxCluster && (long long)a.N * ranks * 2 <= 2 * 152 && chunk_of(ranks) > kThreads * n) ranks *= 2;
  a.chunk = chunk_of(ranks);
  const size_t smem = (size_t)a.chunk * esz;
  if (bf16) return vec ? run<__nv_bfloat16, true>(a, ranks, smem, stream) : run<__nv_bfloat16, false>(a, ranks, smem, stream);
  return vec ? run<float, true>(a, ranks, smem, stream) : run<float, false>(a, ranks, smem, stream);
}

}  // namespace dflash
