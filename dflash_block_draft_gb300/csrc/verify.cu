// verify.cu -- verification of drafted tokens against the target's probabilities
// with given random numbers (sm_103a).
//
// Per request: the first drafted token with not (u q(x) < p(x)) is replaced by
// the smallest i with w_0 + .. + w_i > s (w_0 + .. + w_{V-1}), w = max(p - q, 0)
// (p itself behind the last token, or where w is all zero).
//
// What has to be read is one row of p and one of q, 8 bytes for each entry of the
// vocabulary, so large batches are bound by memory and small ones by the chain of
// dependent steps.  A cluster of 8 CTAs takes a request: every CTA finds the
// rejected position for itself (a few gathered values, cheaper than a round trip
// through the cluster), adds up its eighth of the row, and one exchange of the 8
// sums through distributed shared memory tells all of them which CTA holds the
// drawn entry.  That one narrows it down to a warp's run from the warps' sums,
// and the warp walks its run (in L2 by now) once more.  One launch, no workspace.
//
// Sums are exact: every weight is an integer multiple of 2^-50, held in 64-bit
// integers (a row of a distribution sums to about 2^50).  So neither the order of
// the sum nor the number of CTAs changes the result, and an entry next to the
// border is decided as in the real numbers up to 2^-50 a weight; fp32 sums
// (2^-24) would draw another entry in every few hundredth row of a large
// vocabulary, and fp64 adds run at a fraction of the integer rate.
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace dflash {
namespace {

namespace cg = cooperative_groups;

constexpr int kCluster = 8;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kStep = 128;  // entries a warp reads at once: a float4 a lane

// A probability in steps of 2^-50; outside [0, 1] clamped, NaN counts as 0.
__device__ __forceinline__ unsigned long long fixed50(float p) {
  return __float2ull_rn(fminf(fmaxf(p, 0.f), 1.f) * 0x1p50f);
}

__device__ __forceinline__ unsigned long long weight(float p, float q) {
  const unsigned long long a = fixed50(p), b = fixed50(q);
  return a > b ? a - b : 0ull;
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

// Weights of the four entries at i (i + 3 may lie beyond `end`: weight 0).
template <bool VEC>
__device__ __forceinline__ void weights4(const Row& r, long long i, long long end, unsigned long long* w) {
  float p[4], q[4] = {0.f, 0.f, 0.f, 0.f};
  if (VEC) {
    const float4 a = i < end ? *reinterpret_cast<const float4*>(r.p + i) : make_float4(0.f, 0.f, 0.f, 0.f);
    p[0] = a.x; p[1] = a.y; p[2] = a.z; p[3] = a.w;
    if (r.q && i < end) {
      const float4 b = *reinterpret_cast<const float4*>(r.q + i);
      q[0] = b.x; q[1] = b.y; q[2] = b.z; q[3] = b.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      p[e] = i + e < end ? r.p[i + e] : 0.f;
      if (r.q) q[e] = i + e < end ? r.q[i + e] : 0.f;
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = i + e == r.skip ? 0ull : weight(p[e], q[e]);
}

// Sum of the warp's run [lo, hi) (lo a multiple of 4).
template <bool VEC>
__device__ __forceinline__ unsigned long long run_sum(const Row& r, long long lo, long long hi, int lane) {
  unsigned long long s = 0;
#pragma unroll 4
  for (long long i = lo + 4 * lane; i < hi; i += kStep) {
    unsigned long long w[4];
    weights4<VEC>(r, i, hi, w);
    s += w[0] + w[1] + w[2] + w[3];
  }
  return warp_sum(s);
}

template <bool VEC>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    verify_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ int s_acc;
  __shared__ unsigned long long s_warp[kWarps];
  __shared__ unsigned long long s_total[2];  // this CTA's sums: weights, and p alone where those are all zero
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int r = blockIdx.x / kCluster;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = a.offsets[r], t1 = a.offsets[r + 1];
  const int n = t1 - t0;
  int* out = a.out + (long long)r * (a.max_draft + 1);
  if (t0 < 0 || n < 0 || t1 > a.total || n > a.max_draft) {  // the same in every CTA of the cluster
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
  // Runs: the vocabulary in kCluster * kWarps equal pieces, multiples of 4 entries.
  const long long piece = ((long long)a.V + 4 * kCluster * kWarps - 1) / (4 * kCluster * kWarps) * 4;
  const long long lo = min((long long)a.V, (rank * kWarps + warp) * piece), hi = min((long long)a.V, lo + piece);

  unsigned long long before = 0, total = 0, mine = 0;
  for (int pass = 0; pass < 2; ++pass) {
    mine = run_sum<VEC>(row, lo, hi, lane);
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
    for (int c = 0; c < kCluster; ++c) {
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
    // numbers, so it exceeds floor(s * total).
    const float u = fminf(fmaxf(a.s[r], 0.f), 0x1.fffffep-1f);
    const unsigned long long bar = (unsigned long long)((double)u * (double)total);
    if (before <= bar && bar < before + mine) {  // one warp of the cluster
      unsigned long long at = before;
      for (long long i0 = lo; i0 < hi; i0 += kStep) {
        const long long i = i0 + 4 * lane;
        unsigned long long w[4];
        weights4<VEC>(row, i, hi, w);
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
            out[acc] = (int)(i + e);
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
  const unsigned grid = (unsigned)a.R * kCluster;
  if (vec) verify_kernel<true><<<grid, kThreads, 0, stream>>>(a);
  else verify_kernel<false><<<grid, kThreads, 0, stream>>>(a);
  count_launch();
  return cudaGetLastError();
}

}  // namespace dflash
