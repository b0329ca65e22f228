// verify.cu -- verification of drafted tokens against the target's probabilities
// with given random numbers (sm_103a).
//
// Per request: the first drafted token with not (u q(x) < p(x)) is replaced by
// the smallest i with w_0 + .. + w_i > s (w_0 + .. + w_{V-1}), w = max(p - q, 0)
// (p itself behind the last token, or where w is all zero).
//
// What has to be read is one row of p and one of q, 8 bytes for each entry of the
// vocabulary, so large batches are bound by memory and small ones by the chain of
// dependent steps.  A cluster of 1 to 8 CTAs takes a request: every CTA finds the
// rejected position for itself (a few gathered values, cheaper than a round trip
// through the cluster), adds up its share of the row, and one exchange of the
// sums through distributed shared memory tells all of them which CTA holds the
// drawn entry.  Its warps' sums, and the sums of the up to 32 segments of the
// warp that holds it, narrow it down to one segment, which that warp walks once
// more (in L2 by now).  One launch, no workspace.
//
// Sums are exact: a weight is held in whole steps of 2^-45, and those are added up
// as integers (a row of a distribution sums to about 2^45), so that neither the
// order of the sum nor the number of CTAs changes the result, and an entry next
// to the border is decided as in the real numbers up to 2^-46 a weight.  (fp32
// sums would draw another entry in every few hundredth row of a large vocabulary;
// fp64 adds run at a fraction of the integer rate.)  The steps come from the adder:
// the bits of 1 + p count steps of 2^-23, what that addition lost is exact in fp32,
// and the bits of its sum with 1.5 2^-22 count steps of 2^-45.  Nine instructions an
// entry in packed fp32; 64-bit conversions took 85 us for 128 rows of 131072,
// shifts of the fraction 47 us; this takes 28, of which the reads are 20 and the
// chain of dependent steps the rest.
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace dflash {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxCluster = 8;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kStep = 128;    // entries a warp reads at once: a float4 a lane
constexpr int kUnroll = 2;    // such reads in flight (28 us; 29 with four, 31 with eight); segments are multiples of kStep * kUnroll
constexpr int kSegments = 32; // most segments of a warp's run

// Weights of two entries, max(p - q, 0), as steps of 2^-23 and of 2^-45 (signed) that
// belong together.  No weight where p > q does not hold, NaN included.
constexpr float kBias = 0x1.8p-22f;  // sums with it lie in [2^-22, 2^-21): their last bit is 2^-45
__device__ __forceinline__ void add_weights(float2 p, float2 q, int& hi, int& lo) {
  const float2 one = make_float2(1.f, 1.f), none = make_float2(-1.f, -1.f), neg = make_float2(-1.f, -1.f);
  const float2 tp = __fadd2_rn(p, one), tq = __fadd2_rn(q, one);
  // p - (tp - 1) and the same of q: exact; their difference, at most 2^-23, is rounded once
  const float2 rp = __ffma2_rn(__fadd2_rn(tp, none), neg, p), rq = __ffma2_rn(__fadd2_rn(tq, none), neg, q);
  const float2 t = __fadd2_rn(__ffma2_rn(rq, neg, rp), make_float2(kBias, kBias));
  if (p.x > q.x) {
    hi += __float_as_int(tp.x) - __float_as_int(tq.x);
    lo += __float_as_int(t.x) - __float_as_int(kBias);
  }
  if (p.y > q.y) {
    hi += __float_as_int(tp.y) - __float_as_int(tq.y);
    lo += __float_as_int(t.y) - __float_as_int(kBias);
  }
}
__device__ __forceinline__ unsigned long long join(int hi, int lo) {
  return (unsigned long long)(((long long)hi << 22) + lo);
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// How the row's weights are made: p and q, p without one entry, or p alone.
struct Row {
  const float *p, *q;  // q nullable
  int skip;            // entry with weight 0 (-1: none)
};

// Four entries of p and q at i; those at and beyond `end`, and the one without
// weight, are 0.
struct Four {
  float4 p, q;
};
template <bool VEC, bool Q>
__device__ __forceinline__ Four load4(const Row& r, int i, int end) {
  Four f;
  f.p = f.q = make_float4(0.f, 0.f, 0.f, 0.f);
  if (VEC) {
    if (i < end) {
      f.p = *reinterpret_cast<const float4*>(r.p + i);
      if (Q) f.q = *reinterpret_cast<const float4*>(r.q + i);
    }
  } else {
    if (i < end) f.p.x = r.p[i];
    if (i + 1 < end) f.p.y = r.p[i + 1];
    if (i + 2 < end) f.p.z = r.p[i + 2];
    if (i + 3 < end) f.p.w = r.p[i + 3];
    if (Q) {
      if (i < end) f.q.x = r.q[i];
      if (i + 1 < end) f.q.y = r.q[i + 1];
      if (i + 2 < end) f.q.z = r.q[i + 2];
      if (i + 3 < end) f.q.w = r.q[i + 3];
    }
  }
  if (!Q && (unsigned)r.skip - (unsigned)i < 4u) {
    if (r.skip == i) f.p.x = 0.f;
    if (r.skip == i + 1) f.p.y = 0.f;
    if (r.skip == i + 2) f.p.z = 0.f;
    if (r.skip == i + 3) f.p.w = 0.f;
  }
  return f;
}

// Sum of [lo, hi) (lo a multiple of 4), over the whole warp.
template <bool VEC, bool Q>
__device__ __forceinline__ unsigned long long segment_sum(const Row& r, int lo, int hi, int lane) {
  unsigned long long s = 0;
  for (int i0 = lo + 4 * lane; i0 - 4 * lane < hi; i0 += kStep * kUnroll) {
    Four f[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) f[k] = load4<VEC, Q>(r, i0 + k * kStep, hi);
    int h = 0, l = 0;  // 8 entries: at most 2^26 and 2^25
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      add_weights(make_float2(f[k].p.x, f[k].p.y), make_float2(f[k].q.x, f[k].q.y), h, l);
      add_weights(make_float2(f[k].p.z, f[k].p.w), make_float2(f[k].q.z, f[k].q.w), h, l);
    }
    s += join(h, l);
  }
  return warp_sum(s);
}

template <bool VEC>
__global__ void __launch_bounds__(kThreads, 4) verify_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ int s_acc;
  __shared__ unsigned long long s_warp[kWarps], s_seg[kWarps][kSegments];
  __shared__ unsigned long long s_total[2];  // this CTA's sums: weights, and p alone where those are all zero
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int r = blockIdx.x / ranks;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = a.offsets[r], t1 = a.offsets[r + 1];
  const float sample = a.s[r];  // needed last, read while the offsets are
  const int n = t1 - t0;
  int* out = a.out + (long long)r * (a.max_draft + 1);
  // (t1 < t0 by itself: of offsets far apart the difference wraps); the same in every CTA of the cluster
  if (t0 < 0 || t1 < t0 || t1 > a.total || n > a.max_draft) {
    if (rank == 0) {
      for (int j = threadIdx.x; j <= a.max_draft; j += kThreads) out[j] = -1;
      if (threadIdx.x == 0) {
        a.acc[r] = 0;
        record_error(a.err, DFLASH_ERR_INVALID);
      }
    }
    return;
  }
  const float* target = a.p + ((long long)t0 + r) * a.ps;
  if (warp == 0) {
    int acc = n;
    for (int j0 = 0; j0 < n; j0 += 32) {
      const int j = j0 + lane;
      bool reject = false;
      if (j < n) {
        const int x = a.tokens[t0 + j];
        if (x < 0 || x >= a.V) {
          reject = true;
          if (rank == 0) record_error(a.err, DFLASH_ERR_INVALID);
        } else {
          const double q = a.q ? (double)a.q[(t0 + j) * a.qs + x] : 1.0;
          reject = !((double)a.u[t0 + j] * q < (double)target[j * a.ps + x]);
        }
      }
      const unsigned m = __ballot_sync(0xffffffffu, reject);
      if (m) {
        acc = j0 + __ffs(m) - 1;
        break;
      }
    }
    if (lane == 0) s_acc = acc;
  }
  __syncthreads();
  const int acc = s_acc;
  Row row;
  row.p = target + acc * a.ps;
  row.q = acc < n && a.q ? a.q + (t0 + acc) * a.qs : nullptr;
  row.skip = acc < n && !a.q ? a.tokens[t0 + acc] : -1;
  // Runs: the vocabulary in equal pieces, one a warp, multiples of 4 entries; a run in
  // up to kSegments segments.
  const int piece = (a.V + 4 * ranks * kWarps - 1) / (4 * ranks * kWarps) * 4;
  const int span = (piece + kSegments * kStep * kUnroll - 1) / (kSegments * kStep * kUnroll) * (kStep * kUnroll);
  const int lo = (int)min((long long)a.V, (long long)(rank * kWarps + warp) * piece), hi = min(a.V, lo + piece);

  unsigned long long before = 0, total = 0, mine = 0;
  for (int pass = 0; pass < 2; ++pass) {
    mine = 0;
    for (int g = 0; lo + g * span < hi; ++g) {
      const int i0 = lo + g * span, i1 = min(hi, i0 + span);
      const unsigned long long s =
          row.q ? segment_sum<VEC, true>(row, i0, i1, lane) : segment_sum<VEC, false>(row, i0, i1, lane);
      if (lane == 0) s_seg[warp][g] = s;
      mine += s;
    }
    if (lane == 0) s_warp[warp] = mine;
    __syncthreads();
    if (threadIdx.x == 0) {
      unsigned long long s = 0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) s += s_warp[i];
      s_total[pass] = s;
      if (rank == 0) out[acc] = 0;  // stays where no entry is found (sums of rows that are no distribution may wrap)
    }
    cluster.sync();
    before = total = 0;
    for (int c = 0; c < ranks; ++c) {
      const unsigned long long s = *cluster.map_shared_rank(&s_total[pass], c);
      before += c < rank ? s : 0ull;
      total += s;
    }
    if (total > 0 || (!row.q && row.skip < 0)) break;  // the same in every CTA
    row.q = nullptr;  // nothing of p lies above q: p itself
    row.skip = -1;
    __syncthreads();  // s_warp has been read
  }
  for (int i = 0; i < warp; ++i) before += s_warp[i];
  if (total > 0) {
    // z is the first entry whose running sum exceeds s * total; sums are whole
    // numbers, so it exceeds floor(s * total), which a product rounded down keeps.
    const float u = fminf(fmaxf(sample, 0.f), 0x1.fffffep-1f);
    const unsigned long long bar = (unsigned long long)__dmul_rd((double)u, (double)total);
    if (before <= bar && bar < before + mine) {  // one warp of the cluster
      unsigned long long at = before;
      int g = 0;
      while (lo + (g + 1) * span < hi && at + s_seg[warp][g] <= bar) at += s_seg[warp][g++];
      const int end = min(hi, lo + (g + 1) * span);
#pragma unroll 4
      for (int i0 = lo + g * span; i0 < end; i0 += kStep) {
        const int i = i0 + 4 * lane;
        const Four f = row.q ? load4<VEC, true>(row, i, end) : load4<VEC, false>(row, i, end);
        const float p4[4] = {f.p.x, f.p.y, f.p.z, f.p.w}, q4[4] = {f.q.x, f.q.y, f.q.z, f.q.w};
        unsigned long long w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          int h = 0, l = 0;
          add_weights(make_float2(p4[e], 0.f), make_float2(q4[e], 0.f), h, l);
          w[e] = join(h, l);
        }
        const unsigned long long s = w[0] + w[1] + w[2] + w[3];
        unsigned long long c = s;  // inclusive scan over the lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned long long v = __shfl_up_sync(0xffffffffu, c, o);
          if (lane >= o) c += v;
        }
        const unsigned m = __ballot_sync(0xffffffffu, at + c > bar);
        if (m) {
          if (lane == __ffs(m) - 1) {
            unsigned long long k = at + c - s;
            int e = 0;
#pragma unroll
            for (int f = 0; f < 4; ++f) {
              if (k <= bar) e = f;  // entries up to the one that passes the bar
              k += w[f];
            }
            out[acc] = i + e;
          }
          break;
        }
        at += __shfl_sync(0xffffffffu, c, 31);
      }
    }
  } else if (rank == 0 && threadIdx.x == 0) {
    record_error(a.err, DFLASH_ERR_INVALID);
  }
  if (rank == 0) {
    for (int j = threadIdx.x; j <= a.max_draft; j += kThreads)
      if (j != acc) out[j] = j < acc ? a.tokens[t0 + j] : -1;
    if (threadIdx.x == 0) a.acc[r] = acc;
  }
  cluster.sync();  // no CTA leaves while another may still read its sums
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t stream) {
  const bool vec = a.V % 4 == 0 && a.ps % 4 == 0 && ((uintptr_t)a.p & 15u) == 0 &&
                   (!a.q || (a.qs % 4 == 0 && ((uintptr_t)a.q & 15u) == 0));
  // As many CTAs a request as keep the launch within one wave of four CTAs an SM: a
  // second wave repeats the chain of dependent steps, and fewer, larger shares
  // read as fast.  (128 rows of 131072 entries: 28 us with 4, 33 with 8, 57 with one; 4
  // rows of 32000: 5.8 us with 8, 12 with one.)
  int ranks = kMaxCluster;
  while (ranks > 1 && (long long)a.R * ranks > 4 * 152) ranks >>= 1;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)ranks;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)a.R * ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, vec ? verify_kernel<true> : verify_kernel<false>, a);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

}  // namespace dflash
