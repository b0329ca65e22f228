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
// One CTA, or a cluster of 2 to 8, takes a row and holds it in shared memory: the logits are
// read from memory once, by 16 bytes a thread.  Then
//   the largest logit, and the maxima of 512 groups of threads (one exchange);
//   top-k up to 160: a bound that k of the groups reach, found by halving, so that at least k
//     tokens lie above it and about k + k^2 / 1000 more; they go into a list of 256 whose order
//     comes from comparing all pairs, and everything else is worked out from the list;
//   larger k: the tokens above a bound counted in 4096 equal steps of the logit, the counts
//     merged through distributed shared memory, and the step in which k is reached listed (or,
//     where it holds too many, divided by the bits of logit and number, so that ties divide too);
//   top-p: the weights' approximate masses in 4096 equal steps say between which logits the
//     cut must lie; the exact pass over all tokens adds up what is in front of them and lists
//     what is between, and the exact border falls in the list (or, where that holds too
//     many, is looked for by the bits of logit and number);
//   the sums of kept weights by runs of tokens, one exchange, and the run that passes u times
//     the whole once more, a few tokens a thread.
//
// Bound by instructions and as much by a row's phases, which wait for one another (46 to 62 % of
// the issue slots, 8 to 17 % of the memory's rate): a weight costs some 21 instructions, a look at
// a logit 2 to 15, and what a row costs besides (barriers, exchanges, the list) is as much as 8000
// tokens of a CTA.  Two CTAs of 512 threads an SM, one row's wait under the other's work.  Measured:
// 64 rows of 131072 bf16 logits with temperature alone 20.8 us; 1664 rows of 32000 with top-k 40 in
// most of them 77; 128 rows of 131072 fp32 with top-p and the distributions written 126; 4 rows of
// 32000 9.4.
// (With a histogram of all weights for top-p and a second exact pass, 128 rows took 251 us;
// top-k by a histogram of everything above the least of the threads' maxima, 4 rows 17.)  The
// kernel runs once through most of its code, which was 190 KB where loops were copied and
// functions inlined: 4 rows then took 29 us.
//
// Weights are whole steps of 2^-44 of the largest one, added up as integers, so that no sum
// depends on the order, the number of CTAs or the threads' timing.  A pair of weights takes 16
// packed fp32 instructions in bf16 and 22 in fp32, and each some 13 others: l - m, times
// log2(e) / T as two floats; 2^y from a table of 2^(j / 128) in two floats and a polynomial of
// degree 3; the bits of sums with 2.5 and 1.5 2^-21 count the steps, as in verify.cu.  (Four packed
// instructions fewer a pair took 64 rows from 24.6 us to 22.7 where eight copies of the table
// without bank conflicts, or shuffles in its place, changed nothing.)  The
// weights' errors, 2^-33.5 rms, are each other's by chance and add up to a border's as their
// root: of a vocabulary of 131072 every 10^7th row would draw another token than the real numbers
// (every 50th with fp32 sums of weights that are off in one direction).  Twice the instructions
// for 2^-40 took 1.5 times as long, and neither differed from 64-bit sums in 25000 rows; 64-bit
// floating point runs at a hundredth of fp32's rate.
#include <cooperative_groups.h>
#include <limits.h>
#include <math.h>
#include <stddef.h>

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace dflash {
namespace {

namespace cg = cooperative_groups;
typedef unsigned long long u64;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 4096;       // of the masses
constexpr int kCoarse = kBins / kThreads;  // bins that a thread looks at together
constexpr int kParts = 512;       // of a range whose border is looked for: one a thread
constexpr int kPartBits = 9;
constexpr int kList = 256;        // tokens whose order is found by comparing all pairs
constexpr int kDirect = 160;      // top-k up to here: the tokens above the k-th of 512 groups' maxima, some 190, fit the list
constexpr int kMaxCluster = 8;
constexpr int kIndexBits = 19;    // of a token's number
constexpr uint32_t kIndexMask = (1u << kIndexBits) - 1;
constexpr int kChunkBytes = 196608;  // of logits that a CTA can hold
static_assert(DFLASH_SAMPLE_MAX_V <= kMaxCluster * kChunkBytes / 4 && DFLASH_SAMPLE_MAX_V <= (int)kIndexMask + 1, "vocabulary");
static_assert(kCoarse == 8 && kParts == kThreads && kThreads >= 2 * kList, "thread layout");
constexpr float kTop = 0x1p126f;  // logits above count as it, those below -kTop are no choice: differences are finite
// Masses of top-p's first look: a weight within its bin, linear from 1 to e^(-31.2 / 4096), in
// 1 / kMass, the finest unit in which all tokens that a CTA can hold fit one 32-bit bin (equal
// logits, or a high temperature).
constexpr float kBinRatio = 0.99241175f;  // e^(-31.2 / 4096)
constexpr uint32_t kMass = 43690;
constexpr uint32_t kMassSlope = (uint32_t)(kMass * 128 * (1.0 - 0.99241175) + 0.5);  // a 512th of a bin, in 2^-16
static_assert((u64)kMass * (kChunkBytes / 2) < 1ull << 32, "a bin holds every token of a CTA");
// Margin of the masses, on either side of the comparison: they are off by less than 2.7e-5 (bins
// linear within 7.2e-6, masses rounded 1.2e-5, fp32 distances, powers and sums 7e-6).
constexpr float kOver = 1.00008f;

// ------------------------------------------------------------------ weights
// 2^(j / 128) as a float and what it lacks.
struct Powers {
  float hi[128], lo[128];
};
constexpr Powers make_powers() {
  Powers p = {};
  for (int j = 0; j < 128; ++j) {
    // the series of e^x, x = j ln 2 / 128, whose terms fall below 2^-60 of the sum; the 24 bits
    // of hi leave 29 of the sum's 53 for lo
    const double x = 0.69314718055994530942 * j / 128;
    double t = 1, s = 0;
    for (int k = 1; k < 25; ++k) {
      t = t * x / k;
      s += t;
    }
    p.hi[j] = (float)(1 + s);
    p.lo[j] = (float)(s - ((double)p.hi[j] - 1));
  }
  return p;
}
__device__ constexpr Powers kPowers = make_powers();

struct Scale {
  float m, ch, cl;  // the largest logit; log2(e) / T as ch + cl
};

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// A weight in steps: hi of 2^-22, lo (signed) of 2^-44, or sums of them.
struct Steps44 {
  int hi, lo;
  __device__ __forceinline__ u64 joined() const { return (u64)(((long long)hi << 22) + lo); }
};
constexpr float kHi = 2.5f, kLo = 0x1.8p-21f;  // sums with these have their last bits at 2^-22 and 2^-44

// The powers' table in shared memory.
struct Table {
  float hi[128], lo[128];
};

// Weights of two logits that are at most 45 powers of two below the largest one; 0 where !in.
// Off by at most 2^-31 of themselves (2^-33.5 rms), and by half a step (small ones by one).  In fp32 l - m is
// taken as two floats; of two bf16 values it fits one, but where one of them is below
// 2^-16 of the other.
template <typename T>
__device__ __forceinline__ void weights(const Scale& c, const Table& tab, float2 l, bool in0, bool in1, Steps44& w0,
                                        Steps44& w1) {
  const float2 neg = both(-1.f), nm = both(-c.m), ch = both(c.ch);
  l = make_float2(in0 ? l.x : c.m, in1 ? l.y : c.m);
  const float2 d = __fadd2_rn(l, nm);
  // y = log2(e) / T d = raw / 128 + z, the whole steps by the adder's bits
  const float big = 0x1.8p16f;  // (its own bits are 0 in the lower half)
  const float2 t1 = __ffma2_rn(d, ch, both(big));
  float2 z = __ffma2_rn(d, ch, __ffma2_rn(t1, neg, both(big)));
  if (sizeof(T) == 4) {  // l - m = d + err exactly (the two-sum of Moller and Knuth)
    const float2 bb = __ffma2_rn(l, neg, d);
    const float2 err = __fadd2_rn(__ffma2_rn(__ffma2_rn(bb, neg, d), neg, l), __ffma2_rn(bb, neg, nm));
    z = __ffma2_rn(err, ch, z);
  }
  z = __ffma2_rn(d, both(c.cl), z);
  const int raw0 = __float_as_int(t1.x), raw1 = __float_as_int(t1.y);
  // 2^(raw / 128) = p (th + tl)
  const float2 th = make_float2(tab.hi[raw0 & 127], tab.hi[raw1 & 127]);
  const float2 tl = make_float2(tab.lo[raw0 & 127], tab.lo[raw1 & 127]);
  const int p0 = (raw0 * 65536 + 0x3F800000) & 0xFF800000, p1 = (raw1 * 65536 + 0x3F800000) & 0xFF800000;
  const float2 p = make_float2(in0 ? __int_as_float(p0) : 0.f, in1 ? __int_as_float(p1) : 0.f);
  // s = 2^z - 1, and (th + tl) (1 + s) = hi + lo
  const float2 q = __ffma2_rn(z, both(5.55041087e-2f), both(0.240226507f));
  const float2 s = __fmul2_rn(z, __ffma2_rn(q, z, both(0.693147182f)));
  const float2 hi = __ffma2_rn(th, s, th);
  const float2 lo = __fadd2_rn(__ffma2_rn(th, s, __ffma2_rn(hi, neg, th)), tl);
  // in steps
  const float2 x = __ffma2_rn(hi, p, both(kHi));
  const float2 y = __ffma2_rn(lo, p, __ffma2_rn(hi, p, __ffma2_rn(x, neg, both(kHi + kLo))));
  w0 = Steps44{__float_as_int(x.x) - __float_as_int(kHi), __float_as_int(y.x) - __float_as_int(kLo)};
  w1 = Steps44{__float_as_int(x.y) - __float_as_int(kHi), __float_as_int(y.y) - __float_as_int(kLo)};
}
template <typename T>
__device__ __forceinline__ u64 weight(const Scale& c, const Table& tab, float l, bool in) {
  Steps44 w0, w1;
  weights<T>(c, tab, both(l), in, in, w0, w1);
  return w0.joined();
}

// The weight as a float, for the distribution, whose values are fp32 anyway: off by 2^-22 where the
// rounding of the result alone is 2^-24.  (The draw takes the weights in steps.)
__device__ __forceinline__ float weight_f32(const Scale& c, float l) {
  const float d = l - c.m, n = rintf(d * c.ch);
  const float f = fmaf(d, c.cl, fmaf(d, c.ch, -n));
  return n < -126.f ? 0.f : ptx::ex2(f) * __int_as_float(((int)n + 127) << 23);
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
// The larger of two, number for number (NaN loses), of what a 32-bit word holds.
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b, float) {
  return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
}
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b, __nv_bfloat16) {
  const __nv_bfloat162 m = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}
template <typename T>
__device__ __forceinline__ uint32_t largest(const uint4& v) {
  return larger(larger(v.x, v.y, T()), larger(v.z, v.w, T()), T());
}
__device__ __forceinline__ float value_of(uint32_t w, float) { return __uint_as_float(w); }
__device__ __forceinline__ float value_of(uint32_t w, __nv_bfloat16) {
  return fmaxf(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// A bit for each logit of a 32-bit word that lies from lo to hi (bf16: two, by borders in bf16).
template <typename T>
struct Between;
template <>
struct Between<float> {
  float lo, hi;
  __device__ __forceinline__ Between(float lo_, float hi_) : lo(lo_), hi(hi_) {}
  __device__ __forceinline__ unsigned operator()(uint32_t w) const {
    return __uint_as_float(w) >= lo && __uint_as_float(w) <= hi;
  }
};
template <>
struct Between<__nv_bfloat16> {
  __nv_bfloat162 lo, hi;
  __device__ __forceinline__ Between(float lo_, float hi_)
      : lo(__bfloat162bfloat162(__float2bfloat16_ru(lo_))), hi(__bfloat162bfloat162(__float2bfloat16_rd(hi_))) {}
  __device__ __forceinline__ unsigned operator()(uint32_t w) const {
    const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w);
    const unsigned both = __hge2_mask(x, lo) & __hle2_mask(x, hi);
    return (both & 1u) | (both >> 15 & 2u);
  }
};

struct Row {
  // what a CTA tells the others
  float coarse[kThreads];          // masses of kCoarse bins each
  float top[kThreads];             // largest logit of 1 to 8 neighbouring threads, 512 in the cluster
  alignas(8) float2 low;           // smallest of the threads' maxima; threads that have logits
  alignas(16) int4 listed;         // tokens of the range; the smallest and the largest of their keys
  alignas(16) ulonglong2 weight;   // weights in front of the bracket, and all
  u64 sum;                         // kept weights
  int best;                        // the first token with the row's largest logit (greedy)
  u64 list[kList];
  alignas(16) uint32_t lo[kBins];  // counts, masses, or the weights' lower
  uint32_t hi[kParts];             // and upper halves
  // its own
  Table tab;
  u64 scan[kWarps];
  float scan_f[kWarps], coarse_before[kThreads];
  u64 all[kList], all_w[kList];
  u64 ranked[kMaxCluster];         // kept weights of the bracket, each CTA's
  uint32_t keys[kWarps];
  u64 found_before;
  int found, b1, b2;
  u64 cut, bar;
  double log_min_p;
  int first;          // the first token that is kept (a random number of 0)
  Scale scale;
  float ends, least, inv;  // no weight below `ends`; min-p's bound; 1 / kept weights
};

static_assert(offsetof(Row, lo) % 16 == 0 && offsetof(Row, listed) % 16 == 0 && offsetof(Row, weight) % 16 == 0 &&
                  offsetof(Row, low) % 8 == 0, "read in pieces of 16 and 8 bytes");
static_assert(sizeof(Row) + kChunkBytes <= 232448, "shared memory budget");

// Adds to a 64-bit sum in shared memory, the halves by themselves.
__device__ __forceinline__ void add64(u64* to, u64 w) {
  uint32_t* h = reinterpret_cast<uint32_t*>(to);
  const uint32_t lo = (uint32_t)w, hi = (uint32_t)(w >> 32) + (atomicAdd(h, lo) + lo < lo);
  if (hi) atomicAdd(h + 1, hi);
}

template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The smallest value of the block's threads.
__device__ __noinline__ uint32_t block_least(Row& s, uint32_t v) {
  v = __reduce_min_sync(0xffffffffu, v);
  __syncthreads();  // the values of an earlier call have been read
  if ((threadIdx.x & 31) == 0) s.keys[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_min_sync(0xffffffffu, s.keys[threadIdx.x % kWarps]);
}

// Exclusive sum over the block's threads; *total is the whole.  (The kernel runs through most
// of its code once a row: its size is time, so what is used in several places is called.)
template <typename V>
__device__ __noinline__ V block_scan(V v, V* scratch, V* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  V c = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V u = __shfl_up_sync(0xffffffffu, c, o);
    if (lane >= o) c += u;
  }
  __syncthreads();  // scratch of an earlier call has been read
  if (lane == 31) scratch[warp] = c;
  __syncthreads();
  V w = lane < kWarps ? scratch[lane] : 0;
  const V own = w;
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1) {
    const V u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  *total = __shfl_sync(0xffffffffu, w, kWarps - 1);
  return __shfl_sync(0xffffffffu, w - own, warp) + c - v;
}

// The CTA's logits, 4 at a time.
template <typename T>
struct Pass {
  T* chunk;
  int run;    // logits of a warp's run
  int first;  // number of the chunk's first token
  __device__ __forceinline__ void load(int at, float (&x)[4]) const {
    if constexpr (sizeof(T) == 4) {
      const float4 v = *reinterpret_cast<const float4*>(chunk + at);
      x[0] = v.x;
      x[1] = v.y;
      x[2] = v.z;
      x[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(chunk + at);
      x[0] = __uint_as_float(v.x << 16);
      x[1] = __uint_as_float(v.x & 0xFFFF0000u);
      x[2] = __uint_as_float(v.y << 16);
      x[3] = __uint_as_float(v.y & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ float logit(int at) const { return to_f32(chunk[at]); }
  // body(x, at): the logits at .. at + 3 of the chunk, the whole warp together
  template <typename Body>
  __device__ __forceinline__ void each(Body body) const {
    const int at = (threadIdx.x >> 5) * run + (threadIdx.x & 31) * 4;
#pragma unroll 1
    for (int k = 0; k < run; k += 128) {
      float x[4];
      load(at + k, x);
      body(x, at + k);
    }
  }
  // body(l, at) for every logit that is `bound` at least: few of them
  template <typename Body>
  __device__ __forceinline__ void some(float bound, Body body) const {
    const uint4* v = reinterpret_cast<const uint4*>(chunk + (threadIdx.x >> 5) * run) + (threadIdx.x & 31);
#pragma unroll 2
    for (int k = 0; k < run; k += 32 * Vec<T>::N, v += 32) {
      if (value_of(largest<T>(*v), T()) >= bound) {
        const int at = (int)(reinterpret_cast<const T*>(v) - chunk);
        const uint32_t w[4] = {v->x, v->y, v->z, v->w};
        unsigned mask = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (sizeof(T) == 4) {
            mask |= (unsigned)(__uint_as_float(w[e]) >= bound) << e;
          } else {
            mask |= (unsigned)(__uint_as_float(w[e] << 16) >= bound) << (2 * e);
            mask |= (unsigned)(__uint_as_float(w[e] & 0xFFFF0000u) >= bound) << (2 * e + 1);
          }
        }
#pragma unroll 1
        for (; mask; mask &= mask - 1) {
          const int e = at + __ffs(mask) - 1;
          body(logit(e), e);
        }
      }
    }
  }
  // body(l, at) for every logit from `lo` to `hi`: few of them
  template <typename Body>
  __device__ __forceinline__ void range(float lo, float hi, Body body) const {
    constexpr int N = Vec<T>::N;
    const uint4* v = reinterpret_cast<const uint4*>(chunk + (threadIdx.x >> 5) * run) + (threadIdx.x & 31);
    const Between<T> in(lo, hi);
#pragma unroll 2
    for (int k = 0; k < run; k += 32 * N, v += 32) {
      const uint4 w = *v;
      unsigned mask = in(w.x) | in(w.y) << (N / 4) | in(w.z) << (N / 2) | in(w.w) << (3 * N / 4);
#pragma unroll 1
      for (const int at = (int)(reinterpret_cast<const T*>(v) - chunk); mask; mask &= mask - 1) {
        const int e = at + __ffs(mask) - 1;
        body(logit(e), e);
      }
    }
  }
};

// A logit's distance from the largest one in 2^21 steps of a range, by the adder's
// bits.  Never falls as the logit falls.
struct Steps {
  float m, mul;
  __device__ __forceinline__ Steps(float m_, float range) : m(m_), mul(0x1p21f / range) {}
  __device__ __forceinline__ int at(float l) const {
    return __float_as_int(fmaf(m - l, mul, 0x1.8p23f)) - __float_as_int(0x1.8p23f);
  }
};
constexpr int kStepBits = 9;  // steps of a bin of the masses
static_assert(kBins << kStepBits == 1 << 21, "steps");

// An empty list, and a cut in front of every token for the search in it.
__device__ __forceinline__ void clear_list(Row& s) {
  if (threadIdx.x == 0) {
    s.listed = make_int4(0, -1, 0, 0);
    s.cut = (u64)key_of(INFINITY) << kIndexBits;
  }
}
// Puts a token into the CTA's list, as far as there is room, and its key into the thread's range.
__device__ __forceinline__ void enlist(Row& s, float l, int i, uint32_t& klo, uint32_t& khi) {
  const uint32_t key = key_of(l);
  klo = min(klo, key);
  khi = max(khi, key);
  const int at = atomicAdd(&s.listed.x, 1);
  if (at < kList) s.list[at] = place_of(key, i);
}
__device__ __forceinline__ void tell_keys(Row& s, uint32_t klo, uint32_t khi) {
  klo = __reduce_min_sync(0xffffffffu, klo);
  khi = __reduce_max_sync(0xffffffffu, khi);
  if ((threadIdx.x & 31) == 0 && khi) {
    atomicMin(reinterpret_cast<uint32_t*>(&s.listed.y), klo);
    atomicMax(reinterpret_cast<uint32_t*>(&s.listed.z), khi);
  }
}
// A row's CTAs.  ONE: a single one, and none of the cluster's barriers and reads (1664 rows of
// 32000 took 92 us with them, 78 without).
template <bool ONE>
struct Team {
  static constexpr int kMost = ONE ? 1 : kMaxCluster;
  static __device__ __forceinline__ int size() { return ONE ? 1 : (int)cg::this_cluster().num_blocks(); }
  static __device__ __forceinline__ int rank() { return ONE ? 0 : (int)cg::this_cluster().block_rank(); }
  static __device__ __forceinline__ void sync() {
    if constexpr (ONE) __syncthreads();
    else cg::this_cluster().sync();
  }
  // sync() in two halves, which whole warps come to
  static __device__ __forceinline__ void arrive() {
    if constexpr (!ONE) {
      __syncwarp();
      asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }
  }
  static __device__ __forceinline__ void wait() {
    if constexpr (ONE) {
      __syncthreads();
    } else {
      __syncwarp();
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
  }
  // what a CTA has at the place of `p`
  template <typename V>
  static __device__ __forceinline__ const V* peer(const V* p, int rank) {
    if constexpr (ONE) return p;
    else return cg::this_cluster().map_shared_rank(p, rank);
  }
  // what all of them have there, 0 beyond the team (all reads in flight at once)
  template <typename V>
  static __device__ __forceinline__ void all(const V* p, V (&out)[kMost]) {
    const int ranks = size();
#pragma unroll
    for (int c = 0; c < kMost; ++c) out[c] = *peer(p, c & (ranks - 1));
#pragma unroll
    for (int c = 0; c < kMost; ++c) out[c] = c < ranks ? out[c] : V(0);
  }
};
// All CTAs' lists into s.all and their weights into s.all_w, if they are kList at most, and the
// range of their keys.  Returns their number.  (After a sync; a block barrier follows.)
template <typename T, bool ONE>
__device__ __noinline__ int join_lists(Row& s, uint32_t* klo, uint32_t* khi) {
  using G = Team<ONE>;
  const int tid = threadIdx.x, lane = tid & 31, ranks = G::size();
  int4 v = make_int4(0, -1, 0, 0);
  if (lane < ranks) v = *G::peer(&s.listed, lane);
  *klo = __reduce_min_sync(0xffffffffu, (uint32_t)v.y);
  *khi = __reduce_max_sync(0xffffffffu, (uint32_t)v.z);
  int upto = v.x;
#pragma unroll
  for (int o = 1; o < G::kMost; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += u;
  }
  const int n = __shfl_sync(0xffffffffu, upto, G::kMost - 1);
  if (n <= kList) {
    int owner = 0, before = 0;  // of entry tid
#pragma unroll
    for (int c = 0; c < G::kMost - 1; ++c) {
      const int u = __shfl_sync(0xffffffffu, upto, c);
      if (tid >= u) {
        owner = c + 1;
        before = u;
      }
    }
    if (tid < n) {
      const u64 p = G::peer(s.list, owner)[tid - before];
      s.all[tid] = p;
      const float l = logit_of((uint32_t)(p >> kIndexBits));
      s.all_w[tid] = weight<T>(s.scale, s.tab, l, l >= s.ends);
    }
  }
  __syncthreads();
  return n;
}
// For token i = tid / g of the n listed ones, g threads each (a power of two up to 32): how many
// places of the list lie in front of its own, and their weight.
__device__ __forceinline__ int group_of(int n) { return n <= 16 ? 32 : n <= 32 ? 16 : n <= 64 ? 8 : n <= 128 ? 4 : 2; }
__device__ __noinline__ u64 in_front(const Row& s, int n, int g, int i, int* rank) {
  u64 sum = 0;
  int count = 0;
  if (i < n) {
    const u64 p = s.all[i];
#pragma unroll 2
    for (int j = threadIdx.x & (g - 1); j < n; j += g)
      if (s.all[j] > p) {
        sum += s.all_w[j];
        ++count;
      }
  }
  for (int o = g >> 1; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    count += __shfl_xor_sync(0xffffffffu, count, o);
  }
  *rank = count;
  return sum;
}
__device__ __forceinline__ Cut cut_at(u64 place) {
  return Cut{logit_of((uint32_t)(place >> kIndexBits)), (int)(kIndexMask - (uint32_t)(place & kIndexMask))};
}

// The listed token in which the running count or weight, `before` in front of the list, reaches the target
// (none: a cut that keeps nothing).
template <bool WEIGHTS>
__device__ __forceinline__ Cut cut_in_list(Row& s, int n, u64 before, u64 target) {
  const int g = group_of(n), i = threadIdx.x / g;
  int rank;
  const u64 sum = in_front(s, n, g, i, &rank);
  if (i < n) {
    const u64 at = before + (WEIGHTS ? sum : rank), w = WEIGHTS ? s.all_w[i] : 1;
    if (at < target && target <= at + w) s.cut = s.all[i];
  }
  __syncthreads();
  return cut_at(s.cut);
}

// The bins of s.lo in which a running sum over all CTAs' bins passes a border.  A bin's sum is its
// content times 2^(-slope b) (ratio: 2^-slope); b1: the first bin whose running sum times `over`
// reaches share times the whole, or `least`; b2: the first one whose running sum reaches `over` times that.
// b1 < 0: the whole is below `least`.  before: the sum in front of b1, where b1 = b2.
struct Border {
  int b1, b2;
  float before;
};
template <bool ONE>
__device__ __forceinline__ Border border(Row& s, float slope, float ratio, float over, float share, float least) {
  using G = Team<ONE>;
  const int tid = threadIdx.x, lane = tid & 31;
  {
    const uint4* bins = reinterpret_cast<const uint4*>(&s.lo[kCoarse * tid]);
    const uint4 x = bins[0], y = bins[1];
    const uint32_t v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    float mass = 0.f;
#pragma unroll
    for (int k = 7; k >= 0; --k) mass = fmaf(mass, ratio, (float)v[k]);
    s.coarse[tid] = mass * ptx::ex2(-slope * (float)(kCoarse * tid));  // (at the first bin's beginning)
  }
  if (tid == 0) {
    s.b1 = kThreads;
    s.b2 = -1;
  }
  G::sync();
  clear_list(s);
  // ---- merged: eight bins together, then those that the border lies in by themselves
  float part[G::kMost];
  G::all(&s.coarse[tid], part);
  float v = 0.f;
#pragma unroll
  for (int c = 0; c < G::kMost; ++c) v += part[c];
  float all;
  const float c0 = block_scan(v, s.scan_f, &all), c1 = c0 + v;
  const float want = fmaxf(share * all, least);
  if (all < least) return Border{-1, -1, 0.f};
  // (rounding can show two threads the same border, or none: then the bracket is the wider one)
  s.coarse_before[tid] = c0;
  if (c1 * over >= want && !(c0 * over >= want)) atomicMin(&s.b1, tid);
  if (c1 >= want * over && !(c0 >= want * over)) atomicMax(&s.b2, tid);
  __syncthreads();
  const int lo8 = s.b1 == kThreads ? 0 : s.b1, hi8 = s.b2 < 0 ? kThreads - 1 : s.b2;
  int b1 = lo8 * kCoarse, b2 = hi8 * kCoarse + kCoarse - 1;
  float before = 0.f;
  if (hi8 - lo8 < 4) {  // 32 bins at most: every warp for itself
    const int bin = min(kBins - 1, b1 + lane);
    uint32_t w[G::kMost];
    G::all(&s.lo[bin], w);
    float mass = 0.f;
#pragma unroll
    for (int c = 0; c < G::kMost; ++c) mass += (float)w[c];
    mass *= ptx::ex2(-slope * (float)bin);
    float upto = mass;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float u = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += u;
    }
    upto += s.coarse_before[lo8];
    const unsigned may = __ballot_sync(0xffffffffu, upto * over >= want), must = __ballot_sync(0xffffffffu, upto >= want * over);
    // (where none of these bins reaches it, rounding hid the border: the last one)
    const int end = (hi8 - lo8 + 1) * kCoarse - 1, e1 = may ? min(__ffs(may) - 1, end) : end;
    b2 = b1 + (must ? min(__ffs(must) - 1, end) : end);
    b1 += e1;
    before = __shfl_sync(0xffffffffu, upto - mass, e1);
  }
  return Border{b1, b2, before};
}

// The border's bins as logits, which take one comparison each: what is above `first` lies in an
// earlier bin, what is below `last` in a later one (steps are rounded, and off by a quarter besides:
// two more).
struct Bracket {
  float first, last;
};
__device__ __forceinline__ Bracket logits_of(const Border& b, float m, float range) {
  const float step = range * 0x1p-21f;
  return Bracket{__fmaf_ru(-(float)((b.b1 << kStepBits) - 2), step, m),
                 b.b2 < kBins - 1 ? __fmaf_rd(-(float)(((b.b2 + 1) << kStepBits) + 2), step, m) : -INFINITY};
}
__device__ __forceinline__ void clear_bins(Row& s) {
  uint4* bins = reinterpret_cast<uint4*>(&s.lo[kCoarse * threadIdx.x]);
  bins[0] = bins[1] = make_uint4(0, 0, 0, 0);
  __syncthreads();
}

// The cut of top-k (WEIGHTS false; target: k) or top-p (true): the token, of those that
// `prior` keeps and whose keys lie in [klo, khi], in which the running count or weight, `before` in
// front of the range, reaches the target.  The range is divided by places, from the largest
// key to the smallest, into 512 parts.  Returns prior where there are fewer tokens than k, a cut that
// keeps nothing where the target does not lie in the range.
template <bool WEIGHTS, bool ONE, typename T>
__device__ __forceinline__ Cut select(const Pass<T>& pass, Row& s, const Cut& prior, const Scale& sc, uint32_t klo,
                                      uint32_t khi, u64 before, u64 target) {
  using G = Team<ONE>;
  const int tid = threadIdx.x;
  u64 lo = (u64)klo << kIndexBits, hi = place_of(khi, 0);  // the range's places
  int shift;
  float under, over;  // and its logits
  auto divide = [&]() {
    shift = max(0, 64 - __clzll((long long)(hi - lo)) - kPartBits);
    under = logit_of((uint32_t)(lo >> kIndexBits));
    over = logit_of((uint32_t)(hi >> kIndexBits));
  };
  divide();
  auto part_of = [&](float l, int i) -> int {
    if (!prior.keeps(l, i)) return -1;
    const u64 p = place_of(key_of(l), i);
    return p < lo || p > hi ? -1 : (int)((hi - p) >> shift);
  };
#pragma unroll 1
  for (;;) {
    // ---- a histogram of the range
    s.lo[tid] = 0;
    if (WEIGHTS) s.hi[tid] = 0;
    if (tid == 0) s.found = -1;
    __syncthreads();
    pass.range(under, over, [&](float l, int at) {
      const int part = part_of(l, pass.first + at);
      if (part < 0) return;
      if (WEIGHTS) {
        const u64 w = weight<T>(sc, s.tab, l, true);
        const uint32_t wl = (uint32_t)w;
        const uint32_t wh = (uint32_t)(w >> 32) + (atomicAdd(&s.lo[part], wl) + wl < wl);
        if (wh) atomicAdd(&s.hi[part], wh);
      } else {
        atomicAdd(&s.lo[part], 1u);
      }
    });
    G::sync();
    clear_list(s);  // (every CTA has read the lists of an earlier range)
    // ---- merged, every CTA for itself
    u64 v = 0;
    uint32_t part_lo[G::kMost], part_hi[G::kMost] = {};
    G::all(&s.lo[tid], part_lo);
    if (WEIGHTS) G::all(&s.hi[tid], part_hi);
#pragma unroll
    for (int c = 0; c < G::kMost; ++c) v += ((u64)part_hi[c] << 32) + part_lo[c];
    u64 total;
    const u64 at = before + block_scan(v, s.scan, &total);
    if (!WEIGHTS && before + total < target) return prior;
    if (at < target && target <= at + v) {  // one thread
      s.found = tid;
      s.found_before = at;
    }
    __syncthreads();
    const int part = s.found;
    if (part < 0) return Cut{INFINITY, (int)kIndexMask};
    before = s.found_before;
    // ---- the part's tokens
    klo = ~0u;
    khi = 0;
    pass.range(under, over, [&](float l, int at) {
      if (part_of(l, pass.first + at) == part) enlist(s, l, pass.first + at, klo, khi);
    });
    tell_keys(s, klo, khi);
    G::sync();
    const int n = join_lists<T, ONE>(s, &klo, &khi);
    if (n <= kList) return cut_in_list<WEIGHTS>(s, n, before, target);
    // ---- too many: what lies between the part's keys is divided
    hi -= (u64)part << shift;
    lo = max(lo, hi - ((1ull << shift) - 1));
    hi = min(hi, place_of(khi, 0));
    lo = max(lo, (u64)klo << kIndexBits);
    divide();
  }
}

// log2(e) / T in two floats (2^-47), and where weights end: 45 powers of two below m they are less
// than half a step.
__device__ __forceinline__ Scale scale_of(float m, float t, float* ends) {
  const float e = 1.44269502f, c = e / t;                             // log2(e) = e + 1.9259630e-8
  const float left = fmaf(-c, t, e) + 1.92596299e-8f;
  *ends = fmaxf(__fmaf_ru(-31.1916f, t, m), -kTop);
  return Scale{m, c, left / t};
}
// (64-bit floating point is slow here: one thread, while the others wait for the row.)
__device__ __noinline__ double log_of(float min_p) { return log(min((double)min_p, 1.0)); }

// floor(x * whole) for x in [0, 1), exactly, and whether that is less than the product.
__device__ __forceinline__ u64 times(float x, u64 whole, bool* more) {
  const uint32_t b = __float_as_uint(x);
  const uint32_t e = b >> 23;
  const u64 mantissa = e ? (b & 0x7FFFFFu) | 0x800000u : b;
  const int shift = 150 - (int)max(e, 1u);  // x = mantissa 2^-shift, 24 <= shift <= 149
  const u64 lo = mantissa * whole, hi = __umul64hi(mantissa, whole);
  *more = shift >= 128 ? (lo | hi) != 0 : shift >= 64 ? lo != 0 || (hi & ((1ull << (shift - 64)) - 1)) != 0
                                                      : (lo & ((1ull << shift) - 1)) != 0;
  return shift >= 128 ? 0 : shift >= 64 ? hi >> (shift - 64) : hi << (64 - shift) | lo >> shift;
}
// The weight that a nucleus has to reach: at least one step.  *exact: a whole number of steps, which
// weights of less than half a step, counted as none, put out of reach of those that meet it.
__device__ __forceinline__ u64 share_of(float top_p, u64 whole, bool* exact) {
  bool more;
  const u64 x = times(fmaxf(top_p, 0.f), whole, &more);
  *exact = !more && x > 0;
  return max(1ull, x + more);
}
// The bar of the draw: sums are whole numbers, and one exceeds u * whole where it exceeds its floor.
__device__ __forceinline__ u64 draw_bar(float u, u64 whole) {
  bool more;
  return times(fminf(fmaxf(u, 0.f), 0x1.fffffep-1f), whole, &more);
}

template <typename T, bool VEC, bool ONE>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a) {
  constexpr int N = Vec<T>::N;
  extern __shared__ __align__(16) uint4 chunk[];
  __shared__ __align__(16) Row s;
  using G = Team<ONE>;
  const int rank = G::rank(), ranks = G::size();
  const int r = blockIdx.x / ranks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* row = static_cast<const T*>(a.x) + r * a.xs;
  Pass<T> pass;
  pass.chunk = reinterpret_cast<T*>(chunk);
  pass.run = a.chunk / kWarps;
  pass.first = rank * a.chunk;
  const float temp = a.temp ? a.temp[r] : 1.f;
  const float top_p = a.top_p ? a.top_p[r] : 1.f, min_p = a.min_p ? a.min_p[r] : 0.f, u = a.u[r];
  const int top_k = a.top_k ? a.top_k[r] : 0;

  // ---- the row comes in
  constexpr uint32_t kNone = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;  // -inf
  uint32_t best = kNone;
  bool have = false;
#pragma unroll 4
  for (int k = lane * N; k < pass.run; k += 32 * N) {
    const int at = warp * pass.run + k, i = pass.first + at;
    uint4 v;
    if (VEC) {
      v = make_uint4(kNone, kNone, kNone, kNone);
      if (i < a.V) v = __ldcs(reinterpret_cast<const uint4*>(row + i));
    } else {
      alignas(16) T e[N];
#pragma unroll
      for (int j = 0; j < N; ++j) e[j] = i + j < a.V ? row[i + j] : from_f32<T>(-INFINITY);
      v = *reinterpret_cast<uint4*>(e);
    }
    have |= i < a.V;
    best = larger(best, largest<T>(v), T());
    chunk[at / N] = v;
  }
  const float mine = value_of(best, T());
  // ---- the largest logit
  if (tid < 128) {
    s.tab.hi[tid] = kPowers.hi[tid];
    s.tab.lo[tid] = kPowers.lo[tid];
  }
  clear_list(s);
  {
    float hi = mine;
    for (int o = 1; o < ranks; o <<= 1) hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    if (tid % ranks == 0) s.top[tid / ranks] = hi;
    if (top_k > kThreads) {
      const uint32_t least = block_least(s, have ? key_of(mine) : ~0u);
      const int threads = __syncthreads_count(have);
      if (tid == 0) s.low = make_float2(logit_of(least), (float)threads);
    }
  }
  G::arrive();
  if (tid == kThreads - 32 && min_p > 0.f) s.log_min_p = log_of(min_p);
  G::wait();
  float top = G::peer(s.top, tid * ranks / kThreads)[tid % (kThreads / ranks)];
  float m = logit_of(~block_least(s, ~key_of(top)));
  if (m > kTop) {
    m = kTop;
    top = fminf(top, kTop);
    pass.some(kTop, [&](float, int at) { pass.chunk[at] = from_f32<T>(kTop); });
    __syncthreads();
  }
  const bool bad = !(temp >= 0.f) || isinf(temp);
  const bool none = bad || !(m >= -kTop);  // nothing to choose from
  int token = -1;                           // known to one thread of the cluster
  Cut cut = {-kTop, (int)kIndexMask};
  u64 total = 0;
  if (none) {
    cut.v = INFINITY;
  } else if (temp == 0.f) {
    // ---- the first of the largest
    if (tid == 0) s.best = INT_MAX;
    __syncthreads();
    pass.some(m, [&](float, int at) { atomicMin(&s.best, pass.first + at); });
    G::sync();
    const int best = lane < ranks ? *G::peer(&s.best, lane) : INT_MAX;
    cut.v = m;
    cut.i = (int)__reduce_min_sync(0xffffffffu, (unsigned)best);
    if (rank == 0 && tid == 0) token = cut.i;
  } else {
    const float t = fmaxf(temp, 0x1p-100f);
    float ends, least = -kTop;
    const Scale sc = scale_of(m, t, &ends);
    if (tid == 0) {
      s.scale = sc;
      s.ends = ends;
      // the smallest logit whose weight is min_p at least
      if (min_p > 0.f) s.least = __double2float_ru((double)m + s.log_min_p * (double)t);
    }
    __syncthreads();
    if (min_p > 0.f) least = s.least;
    int n = 0;  // tokens of s.all, where those are all that top-k leaves
    const bool limited = top_k > 0 && top_k < a.V;
    if (limited) {
      float bound, range;
      bool tight = true;  // few tokens lie above the bound
      if (top_k <= __syncthreads_count(top >= -kTop)) {
        // ---- k groups reach this far: their maxima, halved towards the k-th
        bound = logit_of(block_least(s, top >= -kTop ? key_of(top) : ~0u));
        float over = m;
#pragma unroll 1
        for (int i = 0; i < 12 && over > bound; ++i) {
          const float mid = 0.5f * bound + 0.5f * over;
          const int reach = __syncthreads_count(top >= mid);
          if (reach >= top_k) bound = mid;
          else over = mid;
          if (reach >= top_k && reach <= top_k + top_k / 8) break;
        }
        range = 1.001f * (m - bound);
        if (top_k <= kDirect) {
          // ---- the tokens above: some more than k
          uint32_t klo = ~0u, khi = 0;
          pass.some(bound, [&](float l, int at) { enlist(s, l, pass.first + at, klo, khi); });
          tell_keys(s, klo, khi);
          G::sync();
          n = join_lists<T, ONE>(s, &klo, &khi);
          if (n > kList) n = 0;
        }
      } else {
        const float2 v = lane < ranks ? *G::peer(&s.low, lane) : make_float2(INFINITY, 0.f);
        const float low = logit_of(__reduce_min_sync(0xffffffffu, key_of(v.x)));
        // as many tokens as threads lie above the least of the threads' maxima; else down to where weights end
        const bool known = top_k > kThreads && top_k <= (int)warp_sum(v.y) && low >= -kTop;
        bound = known ? low : ends;
        range = known ? 1.001f * (m - low) : 31.2f * t;
        tight = false;
      }
      if (n == 0) {
        // ---- counts in 4096 steps from the largest logit to the bound, and the k-th's step's tokens
        range = fmaxf(range, 1e-30f);
        const Steps steps(m, range);
        clear_bins(s);
        auto bin_of = [&](float l) { return min(kBins - 1, steps.at(l) >> kStepBits); };
        if (tight)
          pass.some(bound, [&](float l, int) { atomicAdd(&s.lo[bin_of(l)], 1u); });
        else
          pass.each([&](const float (&x)[4], int) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (x[k] >= bound) atomicAdd(&s.lo[bin_of(x[k])], 1u);
          });
        __syncthreads();
        const Border at = border<ONE>(s, 0.f, 1.f, 1.f, 0.f, (float)top_k);
        uint32_t klo = ~0u, khi = 0;
        u64 before = 0;
        int listed = kList + 1;
        if (at.b1 >= 0) {
          const Bracket in = logits_of(at, m, range);
          pass.range(fmaxf(in.last, bound), in.first, [&](float l, int i) {
            if (bin_of(l) == at.b1) enlist(s, l, pass.first + i, klo, khi);
          });
          tell_keys(s, klo, khi);
          before = (u64)at.before;
        } else {  // the k-th has no weight: among all tokens
          klo = key_of(-kTop);
          khi = key_of(m);
        }
        G::sync();
        if (at.b1 >= 0) listed = join_lists<T, ONE>(s, &klo, &khi);
        if (listed <= kList) cut = cut_in_list<false>(s, listed, before, top_k);
        else cut = select<false, ONE, T>(pass, s, cut, sc, klo, khi, before, top_k);
      }
    }
    if (n > 0) {
      // ---- all from the list
      const int g = group_of(n), i = tid / g;
      int rank_of;
      const u64 at = in_front(s, n, g, i, &rank_of);
      const u64 place = i < n ? s.all[i] : 0, w = i < n ? s.all_w[i] : 0;
      const bool lead = i < n && (tid & (g - 1)) == 0;
      if (top_p < 1.f || min_p > 0.f) {
        if (tid == 0) s.cut = ~0ull;
        const int lost = __syncthreads_or(lead && rank_of < top_k && w == 0);
        if (lead && rank_of == top_k - 1) {
          bool exact = false;
          s.bar = top_p < 1.f ? share_of(top_p, at + w, &exact) : ~0ull;  // of K's weight
          if (exact && lost) ++s.bar;
        }
        __syncthreads();
        const bool keep = rank_of < top_k && at < s.bar && logit_of((uint32_t)(place >> kIndexBits)) >= least;
        if (keep && lead) atomicMin(&s.cut, place);
      } else if (lead && rank_of == top_k - 1) {
        s.cut = place;
      }
      __syncthreads();
      const u64 edge = s.cut;
      cut = cut_at(edge);
      // kept weights by rising numbers
      const u64 turned = place & kIndexMask;
      u64 upto = 0, whole = 0;
      int earlier = 0;
#pragma unroll 2
      for (int j = tid & (g - 1); j < n; j += g) {
        const u64 x = s.all[j], y = x >= edge ? s.all_w[j] : 0;
        whole += y;
        if ((x & kIndexMask) >= turned) upto += y;
        earlier += x >= edge && (x & kIndexMask) > turned;
      }
      for (int o = g >> 1; o > 0; o >>= 1) {
        upto += __shfl_xor_sync(0xffffffffu, upto, o);
        whole += __shfl_xor_sync(0xffffffffu, whole, o);
        earlier += __shfl_xor_sync(0xffffffffu, earlier, o);
      }
      total = whole;
      const u64 bar = draw_bar(u, whole);
      // (0 draws the first token that is kept, however little it weighs)
      if (rank == 0 && lead && place >= edge && (u > 0.f ? upto - w <= bar && bar < upto : earlier == 0))
        token = (int)(kIndexMask - (uint32_t)turned);
    } else {
      if (limited) {
        // tokens that top-k's cut divides from their equals: from here on the logit alone says who is left
        pass.some(cut.v, [&](float l, int at) {
          if (l == cut.v && pass.first + at > cut.i) pass.chunk[at] = from_f32<T>(-INFINITY);
        });
        __syncthreads();  // (other lanes read them next)
        cut.i = (int)kIndexMask;
      }
      bool nucleus = top_p < 1.f;
      float first_in = INFINITY, last_in = -INFINITY;  // logits of the bracket in which top-p's cut lies
      const Steps steps(m, 31.2f * t);
      float floor = fmaxf(ends, cut.v);
      if (nucleus) {
        // ---- where top-p's cut can lie: the weights' masses in 4096 steps
        if (limited) G::sync();  // the other CTAs have read this one's histogram
        clear_bins(s);
        pass.each([&](const float (&x)[4], int) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int q = steps.at(x[k]);
            const uint32_t mass = ((kMass << 16) + 32768u - kMassSlope * (q & 511)) >> 16;
            if (x[k] >= floor) atomicAdd(&s.lo[min(kBins - 1, q >> kStepBits)], mass);
          }
        });
        __syncthreads();
        const Border at = border<ONE>(s, 0.0109892786f, kBinRatio, kOver, fmaxf(top_p, 1e-6f), 0.f);  // 31.2 / 4096 log2(e)
        const Bracket in = logits_of(at, m, 31.2f * t);
        first_in = in.first;
        last_in = in.last;
        // min-p ends in front of the bracket: top-p takes nothing away
        if (least >= ends && least > first_in) nucleus = false;
      }
      if (!nucleus && least > cut.v) {
        cut.v = least;
        cut.i = (int)kIndexMask;
        floor = fmaxf(ends, least);
      }
      // ---- the weights: those in front of the bracket are kept, and those in it come to the list
      uint32_t klo = ~0u, khi = 0;
      Steps44 kept = {0, 0}, rest = {0, 0};  // (192 tokens a thread at most)
      pass.each([&](const float (&x)[4], int at) {
        if (!__any_sync(0xffffffffu, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) >= floor)) return;
        Steps44 w[4];
        weights<T>(sc, s.tab, make_float2(x[0], x[1]), x[0] >= floor, x[1] >= floor, w[0], w[1]);
        weights<T>(sc, s.tab, make_float2(x[2], x[3]), x[2] >= floor, x[3] >= floor, w[2], w[3]);
        if (!nucleus) {
          kept.hi += w[0].hi + w[1].hi + w[2].hi + w[3].hi;
          kept.lo += w[0].lo + w[1].lo + w[2].lo + w[3].lo;
          return;
        }
        unsigned mask = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          Steps44& to = x[k] > first_in ? kept : rest;
          to.hi += w[k].hi;
          to.lo += w[k].lo;
          mask |= (unsigned)(x[k] <= first_in && x[k] >= fmaxf(floor, last_in)) << k;
        }
#pragma unroll 1
        for (; mask; mask &= mask - 1) {
          const int k = at + __ffs(mask) - 1;
          enlist(s, pass.logit(k), pass.first + k, klo, khi);
        }
      });
      u64 sum = kept.joined();
      u64 own_sums = 0;   // lane c: kept weights of CTA c
      bool told = false;  // known already, the runs' in s.scan
      if (nucleus) {
        // ---- top-p's cut
        tell_keys(s, klo, khi);
        sum = warp_sum(sum);
        const u64 behind = warp_sum(rest.joined());
        if (lane == 0) {
          s.scan[warp] = sum;
          s.all_w[warp] = behind;
        }
        if (lane > 0) sum = 0;  // (the warp's sum is one lane's from here on)
        __syncthreads();
        if (warp == 0) {
          const u64 x = warp_sum(lane < kWarps ? s.scan[lane] : 0), y = warp_sum(lane < kWarps ? s.all_w[lane] : 0);
          if (lane == 0) s.weight = make_ulonglong2(x, x + y);
        }
        if (tid < kMaxCluster) s.ranked[tid] = 0;
        G::sync();
        ulonglong2 v = make_ulonglong2(0, 0);
        if (lane < ranks) v = *G::peer(&s.weight, lane);
        const u64 before = warp_sum((u64)v.x), whole = warp_sum((u64)v.y);
        bool exact;
        u64 target = share_of(top_p, whole, &exact);
        const int n = join_lists<T, ONE>(s, &klo, &khi);
        if (exact) {
          // (a share of a half does it in every other row, others hardly ever)
          bool lost = false;
          pass.some(fmaxf(cut.v, -kTop), [&](float l, int) { lost |= l < ends; });
          lost = __syncthreads_or(lost);
          if (tid == 0) s.best = lost;
          G::sync();
          target += __any_sync(0xffffffffu, lane < ranks && *G::peer(&s.best, lane)) ? 1 : 0;
        }
        if (n <= kList) {
          const int g = group_of(n), i = tid / g;
          int unused;
          const u64 at = before + in_front(s, n, g, i, &unused);
          if (i < n && at < target && target <= at + s.all_w[i]) s.cut = s.all[i];
          __syncthreads();
          cut = cut_at(s.cut);
          if (least > cut.v) cut = Cut{least, (int)kIndexMask};
          // what is kept of the bracket joins the CTAs' and the runs' sums
          if (tid < n) {
            const u64 p = s.all[tid];
            const int k = (int)(kIndexMask - (uint32_t)(p & kIndexMask));
            const u64 w = s.all_w[tid];
            if (cut.keeps(logit_of((uint32_t)(p >> kIndexBits)), k)) {
              const int c = k / a.chunk;
              add64(s.ranked + c, w);
              if (c == rank) add64(s.scan + (k - pass.first) / pass.run, w);
            }
          }
          __syncthreads();
          told = true;
          own_sums = (lane < ranks ? v.x + s.ranked[lane] : 0);
        } else {
          const float over = logit_of(khi);
          cut = select<true, ONE, T>(pass, s, cut, sc, klo, khi, before, target);
          if (least > cut.v) cut = Cut{least, (int)kIndexMask};
          const float from = fmaxf(ends, cut.v);
          pass.range(from, over, [&](float l, int at) {
            sum += weight<T>(sc, s.tab, l, cut.keeps(l, pass.first + at));
          });
        }
      }
      // ---- the token
      if (!told) {
        sum = warp_sum(sum);
        __syncthreads();  // scan of an earlier pass has been read
        if (lane == 0) s.scan[warp] = sum;
        __syncthreads();
        const u64 own = warp_sum(lane < kWarps ? s.scan[lane] : 0);
        if (tid == 0) s.sum = own;
        G::sync();
        own_sums = lane < ranks ? *G::peer(&s.sum, lane) : 0;
      }
      total = warp_sum(own_sums);
      u64 before = warp_sum(lane < rank ? own_sums : 0);
      const u64 own = __shfl_sync(0xffffffffu, own_sums, rank);
      if (!(u > 0.f)) {  // the first token that is kept, however little it weighs
        if (tid == 0) s.first = INT_MAX;
        __syncthreads();
        pass.some(cut.v, [&](float l, int at) {
          if (cut.keeps(l, pass.first + at)) atomicMin(&s.first, pass.first + at);
        });
        G::sync();
        const int first = lane < ranks ? *G::peer(&s.first, lane) : INT_MAX;
        if (rank == 0) {
          const int best = (int)__reduce_min_sync(0xffffffffu, (unsigned)first);
          if (tid == 0) token = best;
        }
      }
      const u64 bar = draw_bar(u, total);
      if (u > 0.f && before <= bar && bar < before + own) {  // one CTA
        // the first run whose end passes the bar
        u64 upto = lane < kWarps ? s.scan[lane] : 0;
#pragma unroll
        for (int o = 1; o < kWarps; o <<= 1) {
          const u64 x = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += x;
        }
        const int w = __ffs(__ballot_sync(0xffffffffu, before + upto > bar)) - 1;
        if (w > 0) before += __shfl_sync(0xffffffffu, upto, w - 1);
        // the warp's run once more, a few tokens in a row a thread
        const int per = (pass.run + kThreads - 1) / kThreads;
        const int at = tid * per, i = w * pass.run + at;
        auto weight_at = [&](int k) -> u64 {
          if (at + k >= pass.run) return 0;
          const float l = pass.logit(i + k);
          return weight<T>(sc, s.tab, l, l >= ends && cut.keeps(l, pass.first + i + k));
        };
        u64 sum = 0, all;
#pragma unroll 1
        for (int k = 0; k < per; ++k) sum += weight_at(k);
        u64 c = before + block_scan(sum, s.scan, &all);
        if (c <= bar && bar < c + sum)  // one thread
#pragma unroll 1
          for (int k = 0; token < 0; ++k) {
            c += weight_at(k);
            if (c > bar) token = pass.first + i + k;
          }
      }
    }
  }
  if (cut.v == INFINITY) {  // nothing is kept
    total = 0;
    token = rank == 0 && tid == 0 ? 0 : -1;
    if (token == 0) record_error(a.err, DFLASH_ERR_INVALID);
  }
  if (token >= 0) a.tokens[r] = token;
  if (a.probs) {
    // ---- the distribution
    float* out = a.probs + r * a.ps;
    const Scale sc = none || temp == 0.f ? Scale{0.f, 0.f, 0.f} : s.scale;
    float inv = 1.f;
    if (total) {
      if (tid == 0) s.inv = (float)(0x1p44 / (double)total);
      __syncthreads();
      inv = s.inv;
    }
    // few are kept, or one of the lowest logit divides its equals: zeros first, then those
    const bool sparse = cut.v > -kTop || cut.i < (int)kIndexMask;
    pass.each([&](const float (&x)[4], int at) {
      const int i = pass.first + at;
      float p[4] = {0.f, 0.f, 0.f, 0.f};
      unsigned mask = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        mask |= (unsigned)(x[k] >= cut.v) << k;
        if (!sparse && x[k] >= cut.v) p[k] = weight_f32(sc, x[k]) * inv;
      }
      if (a.probs_vec) {
        if (i < a.V) __stcs(reinterpret_cast<float4*>(out + i), make_float4(p[0], p[1], p[2], p[3]));
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (i + k < a.V) out[i + k] = p[k];
      }
      if (sparse)
#pragma unroll 1
        for (; mask; mask &= mask - 1) {
          const int k = __ffs(mask) - 1;
          const float l = pass.logit(at + k);
          if (cut.keeps(l, i + k)) out[i + k] = weight_f32(sc, l) * inv;
        }
    });
  }
  // ---- the end
  G::sync();  // no CTA leaves while another may still read what it tells
}

template <typename T, bool VEC, bool ONE>
cudaError_t run(const SampleArgs& a, int ranks, size_t smem, cudaStream_t stream) {
  auto kernel = sample_kernel<T, VEC, ONE>;
  static std::atomic<uint64_t> ready{0};  // devices whose kernel has its shared memory's size
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev >= 64 || !(ready.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kChunkBytes);
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
  cfg.numAttrs = ONE ? 0 : 1;
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
  // CTAs a row.  What a row costs besides its tokens is every CTA's, and a single one waits for no
  // other: one where a row fits, else as many as bring two CTAs an SM (64 KB each, so that one row comes
  // in while another is worked on).  600 rows of 98304 bf16 logits take 107 us with one CTA (temperature alone;
  // top-k 40: 51; top-p 0.9: 248), 137 (100, 286) with four; 1000 of 32000 fp32 92 (66, 150), 98 (80, 168) with
  // two; 128 of 131072 fp32 with top-p 128 with eight, 142 with four.  While there is an SM for each,
  // more CTAs share a long row: 38 rows of 50257 bf16 17.3 (14.5, 30.9) with four and 20.7 (14.4, 51.3)
  // with one, but 60 of 8192 fp32 10.3 (10.4, 14.5) with two and 8.3 (8.3, 12.5) with one; 16384 are
  // the same either way.
  auto chunk_of = [&](int ranks) {
    const int unit = kThreads * n;
    return ((a.V + ranks - 1) / ranks + unit - 1) / unit * unit;
  };
  int ranks = 1;
  if (chunk_of(1) * esz > kChunkBytes)
    while (ranks < kMaxCluster && chunk_of(ranks) * esz > 65536) ranks *= 2;
  if (a.V > 16384)
    while (ranks < kMaxCluster && (long long)a.N * ranks * 2 <= 152) ranks *= 2;
  a.chunk = chunk_of(ranks);
  const size_t smem = (size_t)a.chunk * esz;
  auto pick = [&](auto one) {
    constexpr bool ONE = decltype(one)::value;
    if (bf16)
      return vec ? run<__nv_bfloat16, true, ONE>(a, ranks, smem, stream) : run<__nv_bfloat16, false, ONE>(a, ranks, smem, stream);
    return vec ? run<float, true, ONE>(a, ranks, smem, stream) : run<float, false, ONE>(a, ranks, smem, stream);
  };
  return ranks == 1 ? pick(std::true_type()) : pick(std::false_type());
}

}  // namespace dflash
