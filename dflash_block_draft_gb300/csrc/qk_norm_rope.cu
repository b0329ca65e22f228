// qk_norm_rope.cu -- RMS norm and position rotation of query and key heads, the
// same on the way into a paged cache, and the backward pass (sm_103a).
//
//   y = x (mean x^2 + eps)^-1/2 w,   out = Rot(pos) y
//   backward: g = Rot(pos)^T dout, dw = sum g x^, dx = r (g w - x^ mean(g w x^))
//
// All of it is bound by memory: ten to twenty operations a component against 4
// (bf16, in and out) to 12 bytes.  A head lies in the registers of a group of 8, 16
// or 32 lanes, 8 components a lane: with planes (i, i + rot/2) the 4 components
// at 4 c and the 4 at rot/2 + 4 c, so that every plane is whole inside a lane and
// its 4 cosines and sines serve both; with planes (2 i, 2 i + 1) eight in a row.
// Only the mean goes through shuffles.  (A first form with 16-byte vectors and the
// partner components by shuffle needed twice the cosines and 8 shuffles a head.)
// Head shapes whose planes cut through these vectors (rot % 8 != 0), and
// misaligned tensors, run on a plain kernel with a warp for each head (32768 tokens of
// 40 heads of 128: 518 us where the others take 116; backward 1949 and 183).
//
// Measured, bf16, heads of 128: forward of 32768 x 40 heads 116 us, 5.9 TB/s; backward
// 183 us, 5.6 TB/s (a mix of reads and writes that a copy moves at 6.8); the same in
// fp32 283 us, 4.8 TB/s, and 318, 6.4; appending
// 64 blocks of 16 tokens with their queries 6.6 us, 31000 tokens' keys and values
// 42 us, 6.0 TB/s.
#include <float.h>
#include <limits.h>

#include "common.cuh"
#include "internal.h"

namespace dflash {
namespace {

constexpr int kThreads = 256;

// Four components as they lie in memory; in registers they are pairs, for the
// packed fp32 instructions (these kernels issue about as long as they load).
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint2 v;
  __device__ __forceinline__ void unpack(float2* x) const {
    x[0] = make_float2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u));
    x[1] = make_float2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
  }
  __device__ __forceinline__ void pack(const float2* x) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0].x, x[0].y), b = __floats2bfloat162_rn(x[1].x, x[1].y);
    v.x = *reinterpret_cast<const uint32_t*>(&a);
    v.y = *reinterpret_cast<const uint32_t*>(&b);
  }
};
template <>
struct Raw<float> {
  float4 v;
  __device__ __forceinline__ void unpack(float2* x) const {
    x[0] = make_float2(v.x, v.y);
    x[1] = make_float2(v.z, v.w);
  }
  __device__ __forceinline__ void pack(const float2* x) { v = make_float4(x[0].x, x[0].y, x[1].x, x[1].y); }
};

// A lane's 8 components of a head: 4 at `a`, 4 at `b`; angles ang .. ang + 3.
struct LanePart {
  int a, b, ang;
  bool in, turned;
};
__device__ __forceinline__ LanePart lane_part(const RopeArgs& r, int c) {
  LanePart p;
  p.in = 8 * c < r.D;
  p.turned = 8 * c < r.rot;
  p.ang = 4 * c;
  const bool split = p.turned && !r.interleaved;
  p.a = split ? 4 * c : 8 * c;
  p.b = split ? 4 * c + (r.rot >> 1) : 8 * c + 4;
  return p;
}

template <typename T>
struct Part {
  Raw<T> a, b;
  __device__ __forceinline__ void load(const T* head, const LanePart& p) {
    a = *reinterpret_cast<const Raw<T>*>(head + p.a);
    b = *reinterpret_cast<const Raw<T>*>(head + p.b);
  }
  __device__ __forceinline__ void store(T* head, const LanePart& p) const {
    *reinterpret_cast<Raw<T>*>(head + p.a) = a;
    *reinterpret_cast<Raw<T>*>(head + p.b) = b;
  }
  __device__ __forceinline__ void unpack(float2* x) const {
    a.unpack(x);
    b.unpack(x + 2);
  }
  __device__ __forceinline__ void pack(const float2* x) {
    a.pack(x);
    b.pack(x + 2);
  }
};

// x := x rotated; with the sines' signs turned, rotated back.  cs, sn: the lane's
// four angles in pairs.
__device__ __forceinline__ void rotate8(float2* x, const float2* cs, const float2* sn, int interleaved) {
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float c = e & 1 ? cs[e / 2].y : cs[e / 2].x, s = e & 1 ? sn[e / 2].y : sn[e / 2].x;
      const float2 u = x[e];
      x[e] = __ffma2_rn(make_float2(u.y, u.x), make_float2(-s, s), __fmul2_rn(u, make_float2(c, c)));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float2 u = x[e], v = x[2 + e], neg = make_float2(-sn[e].x, -sn[e].y);
      x[e] = __ffma2_rn(v, neg, __fmul2_rn(u, cs[e]));
      x[2 + e] = __ffma2_rn(u, sn[e], __fmul2_rn(v, cs[e]));
    }
  }
}

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o, LANES);
  return v;
}

// Where a token goes: its position and, for a paged call, the element offsets of
// its cache rows.
struct Place {
  int ok, pos;
  long long krow, vrow;
};

// The rest of token t's placement, where r is the last request to begin at or before it (negative:
// none does) and len its length.  What has no place is recorded, but for tokens that no request
// holds behind the last offset, `end`.
__device__ __forceinline__ Place place_in(const RopeArgs& a, int t, int r, int len, int end) {
  Place pl = {0, 0, 0, 0};
  if (r < 0) {
    if (t < end) record_error(a.err, DFLASH_ERR_INVALID);
    return pl;
  }
  const int q0 = a.q_off[r], q1 = a.q_off[r + 1];
  const long long p = (long long)len - (q1 - q0) + (t - q0);
  if (q0 < 0 || q0 > t || q1 <= t || q1 > a.T || p < 0 || p >= (long long)a.max_pages * a.P ||
      (a.rot > 0 && p >= a.max_pos)) {
    if (q1 > t || t < end) record_error(a.err, DFLASH_ERR_INVALID);
    return pl;
  }
  const int pp = (int)p, page = a.table[(long long)r * a.max_pages + pp / a.P];
  if (page < 0 || page >= a.num_pages) {
    record_error(a.err, DFLASH_ERR_INVALID);
    return pl;
  }
  const long long row = (long long)(pp % a.P) * a.Hkv * a.D;
  pl.ok = 1;
  pl.pos = pp;
  pl.krow = page * a.kps + row;
  pl.vrow = page * a.vps + row;
  return pl;
}

__device__ __forceinline__ bool disordered(const RopeArgs& a, int q0, int q1) { return q0 < 0 || q1 < q0 || q1 > a.T; }

// Records offsets out of order, the grid's threads sharing the requests: where tokens are found
// by search, nobody else looks at all of them.
__device__ __forceinline__ void check_offsets(const RopeArgs& a) {
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < a.R; i += (long long)gridDim.x * kThreads)
    if (disordered(a, a.q_off[i], a.q_off[i + 1])) record_error(a.err, DFLASH_ERR_INVALID);
}

// Whole warp: lane i < n places token t0 + i (ok = 0 elsewhere).  The request of t0,
// the last one that begins at or before it, is found 32 offsets at a time; the
// next tokens' requests follow from the 32 offsets behind it, or, where more
// requests than that end among them (empty ones), by a search of the lane's own.
__device__ __forceinline__ Place place_tokens(const RopeArgs& a, long long t0, int n) {
  const int lane = threadIdx.x & 31;
  const long long t = t0 + lane;
  const int end = a.q_off[a.R];
  int lo = 0, len = a.R;  // it lies in [lo, lo + len)
  while (len > 1) {
    const int step = (len + 31) / 32;
    const int at = lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, at < len && a.q_off[lo + at] <= t0);
    const int k = m ? 31 - __clz(m) : 0;
    lo += k * step;
    len = min(step, len - k * step);
  }
  const int next = lo + 1 + lane < a.R ? a.q_off[lo + 1 + lane] : INT_MAX;
  int r = lo;
  for (int i = 0; i < n; ++i) {
    const int c = __popc(__ballot_sync(0xffffffffu, next <= t0 + i));
    if (lane == i) r = min(lo + c, a.R - 1);
  }
  if (lane < n && t < a.T) {
    if (r - lo == 32) {
      int hi = a.R;
      while (hi - r > 1) {
        const int mid = (r + hi) >> 1;
        if (a.q_off[mid] <= t) r = mid;
        else hi = mid;
      }
    }
    return place_in(a, (int)t, r, a.kv_lens[r], end);
  }
  return Place{0, 0, 0, 0};
}

// The same by a whole block where it has a thread for every request: each looks whether
// its request has tokens among t0 .. t0 + n - 1, so that offsets and lengths are read at
// once.  It claims the first of them; a token belongs to the last claim at or before it.
// claims: n words of shared memory; the result is in the first warp's lanes.
__device__ __forceinline__ Place place_claimed(const RopeArgs& a, long long t0, int n, unsigned long long* claims) {
  const int i = threadIdx.x;
  const bool have = i < a.R;
  const int q0 = have ? a.q_off[i] : 0, q1 = have ? a.q_off[i + 1] : 0, len = have ? a.kv_lens[i] : 0;
  const int end = a.q_off[a.R];
  if (i < n) claims[i] = 0;
  __syncthreads();
  if (q1 > q0 && q1 > t0 && q0 < t0 + n)
    atomicMax(&claims[max((long long)q0, t0) - t0], (unsigned long long)(i + 1) << 32 | (unsigned)len);
  if (have && disordered(a, q0, q1)) record_error(a.err, DFLASH_ERR_INVALID);
  __syncthreads();
  if (i >= 32) return Place{0, 0, 0, 0};
  unsigned long long c = i < n ? claims[i] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long v = __shfl_up_sync(0xffffffffu, c, o);
    if (i >= o) c = max(c, v);
  }
  const long long t = t0 + i;
  if (i >= n || t >= a.T) return Place{0, 0, 0, 0};
  return place_in(a, (int)t, (int)(c >> 32) - 1, (int)(unsigned)c, end);
}

__device__ __forceinline__ Place place_position(const RopeArgs& a, int t) {
  Place pl = {0, 0, 0, 0};
  pl.pos = a.rot > 0 ? a.pos[t] : 0;
  pl.ok = a.rot <= 0 || (pl.pos >= 0 && pl.pos < a.max_pos);
  if (!pl.ok) record_error(a.err, DFLASH_ERR_INVALID);
  return pl;
}

// Forward.  A block takes HPG query heads, key heads or (paged) value heads of one
// token a group: all loads of a group go out together, before the tokens' places
// are found, and what differs between kinds of heads is the same in a whole block.
// Blocks count [tokens][chunk]; chunks below nq are query heads, below nq + nk key
// heads.  (A block that took all heads of its tokens, with the table rows in shared
// memory, spent more instructions on which head is whose than on the heads: 205 for
// every two heads, and 215 us against 117 for 32768 tokens of 40 heads.)
template <typename T, int LANES, int HPG, bool PAGED>
__global__ void __launch_bounds__(kThreads)
    rope_fwd_kernel(const __grid_constant__ RopeArgs a, int nq, int nk, int nchunk) {
  constexpr int kGroups = kThreads / LANES;
  __shared__ Place s_place[PAGED ? kGroups : 1];
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES, lane32 = threadIdx.x & 31;
  const int chunk = blockIdx.x % nchunk;
  const long long t0 = (long long)(blockIdx.x / nchunk) * kGroups, t = t0 + group;
  const bool is_q = chunk < nq, is_v = PAGED && chunk >= nq + nk;
  const int H = is_q ? a.Hq : a.Hkv;
  const int h0 = (chunk - (is_q ? 0 : is_v ? nq + nk : nq)) * HPG, nh = min(HPG, H - h0);
  const LanePart lp = lane_part(a, lane);
  const bool mine = lp.in && t < a.T;
  Part<T> x[HPG];
  if (mine) {
    const T* src = static_cast<const T*>(is_q ? a.q : is_v ? a.v : a.k) + t * (is_q ? a.qs : is_v ? a.vs : a.ks) +
                   h0 * a.D;
#pragma unroll
    for (int j = 0; j < HPG; ++j)
      if (j < nh) x[j].load(src + j * a.D, lp);
  }
  const T* w = static_cast<const T*>(is_q ? a.wq : a.wk);
  float2 wv[4];
  if (w && lp.in && !is_v) {
    Part<T> wr;
    wr.load(w, lp);
    wr.unpack(wv);
  }
  Place pl = {0, 0, 0, 0};
  if (PAGED) {
    // (64 blocks of 16 tokens: 6.6 us, 6.8 by the search; 250 requests of 100 to 200 tokens 52.4
    // and 53.7)
    if (a.R <= kThreads) {
      __shared__ unsigned long long claims[PAGED ? kGroups : 1];
      const Place p = place_claimed(a, t0, kGroups, claims);
      if (threadIdx.x < kGroups) s_place[threadIdx.x] = p;
    } else {
      if (threadIdx.x < 32) {
        const Place p = place_tokens(a, t0, kGroups);
        if (lane32 < kGroups) s_place[lane32] = p;
      }
      check_offsets(a);
    }
    __syncthreads();
    pl = s_place[group];
  } else if (t < a.T) {
    pl = place_position(a, (int)t);
  }
  if (!is_v) {
    float2 cs[2], sn[2];
    if (pl.ok && lp.turned) {
      const float* row = a.cs + (long long)pl.pos * a.rot + lp.ang;
      const float4 c = *reinterpret_cast<const float4*>(row), s = *reinterpret_cast<const float4*>(row + (a.rot >> 1));
      cs[0] = make_float2(c.x, c.y);
      cs[1] = make_float2(c.z, c.w);
      sn[0] = make_float2(s.x, s.y);
      sn[1] = make_float2(s.z, s.w);
    }
    const float inv_d = 1.f / (float)a.D;
#pragma unroll
    for (int j = 0; j < HPG; ++j) {
      if (j >= nh) break;  // the whole block's
      float2 y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = make_float2(0.f, 0.f);
      if (mine) x[j].unpack(y);
      if (w) {
        float2 s2 = __fmul2_rn(y[0], y[0]);
#pragma unroll
        for (int e = 1; e < 4; ++e) s2 = __ffma2_rn(y[e], y[e], s2);
        const float r = rsqrtf(group_sum<LANES>(s2.x + s2.y) * inv_d + a.eps);
        const float2 r2 = make_float2(r, r);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = __fmul2_rn(__fmul2_rn(y[e], r2), wv[e]);
      }
      if (lp.turned) rotate8(y, cs, sn, a.interleaved);
      x[j].pack(y);
    }
  }
  if (mine && pl.ok) {
    T* dst = is_q     ? static_cast<T*>(a.qo) + (t * a.Hq + h0) * a.D
             : !PAGED ? static_cast<T*>(a.ko) + (t * a.Hkv + h0) * a.D
             : is_v   ? static_cast<T*>(a.vc) + pl.vrow + h0 * a.D
                      : static_cast<T*>(a.kc) + pl.krow + h0 * a.D;
#pragma unroll
    for (int j = 0; j < HPG; ++j)
      if (j < nh) x[j].store(dst + j * a.D, lp);
  }
}

// Backward.  A block keeps to one chunk of hpg query heads or hpg key heads and
// walks the tokens, a group a token: the weight and this lane's share of its
// gradient stay in registers all along.  The block adds its groups' shares up in
// shared memory and writes one row of partial sums, so the order of the sums is
// fixed.  Blocks count [row of blocks][chunk]; chunks below nq are query heads.
template <typename T, int LANES>
__global__ void __launch_bounds__(kThreads, 4)
    rope_bwd_kernel(const __grid_constant__ RopeArgs a, int hpg, int nq, int nchunk) {
  constexpr int kGroups = kThreads / LANES;
  // Heads in flight a group.  Two (one in fp32) with four blocks an SM: 184 us for 32768
  // tokens of 40 heads; four with two blocks 191; the next heads' loads ahead of
  // the arithmetic, with two blocks, 183.
  constexpr int kBatch = sizeof(T) == 2 ? 2 : 1;
  __shared__ float red[kGroups][LANES * 8];
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const int chunk = blockIdx.x % nchunk, brow = blockIdx.x / nchunk, brows = gridDim.x / nchunk;
  const bool is_q = chunk < nq;
  const int H = is_q ? a.Hq : a.Hkv;
  const int h0 = (is_q ? chunk : chunk - nq) * hpg, h1 = min(H, h0 + hpg);
  const T* w = static_cast<const T*>(is_q ? a.wq : a.wk);
  const T* src = static_cast<const T*>(is_q ? a.q : a.k);
  const T* dsrc = static_cast<const T*>(is_q ? a.dqo : a.dko);
  T* dst = static_cast<T*>(is_q ? a.qo : a.ko);
  const long long stride = is_q ? a.qs : a.ks;
  const bool normed = w != nullptr;
  const LanePart lp = lane_part(a, lane);
  float2 wv[4], dw[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) wv[e] = dw[e] = make_float2(0.f, 0.f);
  if (normed && lp.in) {
    Part<T> wr;
    wr.load(w, lp);
    wr.unpack(wv);
  }
  const float inv_d = 1.f / (float)a.D;
  const int step = brows * kGroups;
  int t = brow * kGroups + group;  // T + step fits: the host bounds T
  int pos = a.rot > 0 && t < a.T ? a.pos[t] : 0;
  for (int base = brow * kGroups; base < a.T; base += step, t += step) {
    const bool ok = t < a.T && (a.rot <= 0 || (pos >= 0 && pos < a.max_pos));
    if (t < a.T && !ok) record_error(a.err, DFLASH_ERR_INVALID);
    const bool have = ok && lp.in;
    float2 cs[2] = {make_float2(1.f, 1.f), make_float2(1.f, 1.f)}, sn[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    if (ok && lp.turned) {
      const float* row = a.cs + (long long)pos * a.rot + lp.ang;
      const float4 c = *reinterpret_cast<const float4*>(row), s = *reinterpret_cast<const float4*>(row + (a.rot >> 1));
      cs[0] = make_float2(c.x, c.y);
      cs[1] = make_float2(c.z, c.w);
      sn[0] = make_float2(-s.x, -s.y);
      sn[1] = make_float2(-s.z, -s.w);
    }
    if (a.rot > 0 && t + step < a.T) pos = a.pos[t + step];
    const long long row_in = t * stride, row_out = (long long)t * H * a.D;
    for (int hb = h0; hb < h1; hb += kBatch) {
      Part<T> xr[kBatch], gr[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (have && hb + j < h1) {
          gr[j].load(dsrc + row_out + (hb + j) * a.D, lp);
          if (normed) xr[j].load(src + row_in + (hb + j) * a.D, lp);
        }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (hb + j >= h1) break;  // the whole block's
        float2 g[4], x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) g[e] = x[e] = make_float2(0.f, 0.f);
        if (have) {
          gr[j].unpack(g);
          if (normed) xr[j].unpack(x);
        }
        if (lp.turned) rotate8(g, cs, sn, a.interleaved);
        if (normed) {
          float2 gw[4], s2 = __fmul2_rn(x[0], x[0]), d2;
          gw[0] = __fmul2_rn(g[0], wv[0]);
          d2 = __fmul2_rn(gw[0], x[0]);
#pragma unroll
          for (int e = 1; e < 4; ++e) {
            gw[e] = __fmul2_rn(g[e], wv[e]);
            s2 = __ffma2_rn(x[e], x[e], s2);
            d2 = __ffma2_rn(gw[e], x[e], d2);
          }
          const float r = rsqrtf(group_sum<LANES>(s2.x + s2.y) * inv_d + a.eps);
          // r times mean(g w x^) r, the factor of x
          const float c = -group_sum<LANES>(d2.x + d2.y) * r * r * inv_d * r;
          const float2 r2 = make_float2(r, r), c2 = make_float2(c, c);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            dw[e] = __ffma2_rn(g[e], __fmul2_rn(x[e], r2), dw[e]);
            g[e] = __ffma2_rn(x[e], c2, __fmul2_rn(gw[e], r2));
          }
        }
        if (have) {
          gr[j].pack(g);
          gr[j].store(dst + row_out + (hb + j) * a.D, lp);
        }
      }
    }
  }
  if (lp.in) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      red[group][lp.a + e] = e & 1 ? dw[e / 2].y : dw[e / 2].x;
      red[group][lp.b + e] = e & 1 ? dw[2 + e / 2].y : dw[2 + e / 2].x;
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < a.D; d += kThreads) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) s += red[i][d];
    a.dw_part[(long long)blockIdx.x * a.D + d] = s;
  }
}

// Sums the blocks' rows: 8 columns a block, 128 threads down each column, whose five
// loads go out together (one thread a column of 32 took as long as a short call's
// gradients).  Row b belongs to the query weight where b % nchunk < nq, else to
// the key weight.
constexpr int kDwCols = 8, kDwRows = 128;
__global__ void __launch_bounds__(kDwCols* kDwRows)
    rope_dw_kernel(const float* part, int blocks, int nq, int nchunk, int D, float* dwq, float* dwk) {
  __shared__ float red[kDwRows / 4][kDwCols];
  const int c = threadIdx.x % kDwCols, y = threadIdx.x / kDwCols;
  const int d = blockIdx.x * kDwCols + c, w = blockIdx.y;
  float* dst = w ? dwk : dwq;
  if (!dst) return;
  const int first = w ? nq : 0, n = w ? nchunk - nq : nq;  // this weight's chunks of every row of blocks
  const int rows = n > 0 ? blocks / nchunk * n : 0;
  float s = 0.f;
#pragma unroll 8
  for (int i = y; i < rows; i += kDwRows) s += part[((long long)(i / n) * nchunk + first + i % n) * D + d];
  s += __shfl_xor_sync(0xffffffffu, s, 8);  // a warp's four rows
  s += __shfl_xor_sync(0xffffffffu, s, 16);
  if (y % 4 == 0) red[y / 4][c] = s;
  __syncthreads();
  if (y == 0) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kDwRows / 4; ++i) sum += red[i][c];
    dst[d] = sum;
  }
}

// ---------------------------------------------------------------- plain kernels
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float warp_sum(float v) { return group_sum<32>(v); }

// Component d of row y (shared memory) rotated (dir = 1) or rotated back (dir = -1).
__device__ __forceinline__ float turn_one(const RopeArgs& a, const float* y, const float* row, int d, float dir) {
  if (d >= a.rot) return y[d];
  const int h = a.rot >> 1;
  const int ang = a.interleaved ? d >> 1 : (d < h ? d : d - h);
  const bool first = a.interleaved ? (d & 1) == 0 : d < h;
  const int mate = a.interleaved ? d ^ 1 : (first ? d + h : d - h);
  return fmaf(y[d], row[ang], dir * (first ? -y[mate] : y[mate]) * row[h + ang]);
}

template <typename T, bool PAGED>
__global__ void __launch_bounds__(kThreads) rope_fwd_plain_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float rows[kWarps][DFLASH_PAGED_MAX_D];
  const int lane = threadIdx.x & 31;
  float* y = rows[threadIdx.x >> 5];
  const int heads = a.Hq + (PAGED ? 2 : 1) * a.Hkv;
  const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (PAGED) check_offsets(a);
  if (unit >= (long long)a.T * heads) return;
  const int t = (int)(unit / heads), h = (int)(unit % heads);
  Place pl;
  if (PAGED) {
    pl = place_tokens(a, t, 1);  // in lane 0
    pl.ok = __shfl_sync(0xffffffffu, pl.ok, 0);
    pl.pos = __shfl_sync(0xffffffffu, pl.pos, 0);
    pl.krow = __shfl_sync(0xffffffffu, pl.krow, 0);
    pl.vrow = __shfl_sync(0xffffffffu, pl.vrow, 0);
  } else {
    pl = place_position(a, t);
  }
  if (!pl.ok) return;
  const bool is_q = h < a.Hq, is_v = PAGED && h >= a.Hq + a.Hkv;
  const T* src;
  T* dst;
  if (is_q) {
    src = static_cast<const T*>(a.q) + t * a.qs + (long long)h * a.D;
    dst = static_cast<T*>(a.qo) + ((long long)t * a.Hq + h) * a.D;
  } else if (!is_v) {
    src = static_cast<const T*>(a.k) + t * a.ks + (long long)(h - a.Hq) * a.D;
    dst = PAGED ? static_cast<T*>(a.kc) + pl.krow + (long long)(h - a.Hq) * a.D
                : static_cast<T*>(a.ko) + ((long long)t * a.Hkv + (h - a.Hq)) * a.D;
  } else {
    src = static_cast<const T*>(a.v) + t * a.vs + (long long)(h - a.Hq - a.Hkv) * a.D;
    dst = static_cast<T*>(a.vc) + pl.vrow + (long long)(h - a.Hq - a.Hkv) * a.D;
    for (int d = lane; d < a.D; d += 32) dst[d] = src[d];
    return;
  }
  const T* w = static_cast<const T*>(is_q ? a.wq : a.wk);
  float ss = 0.f;
  for (int d = lane; d < a.D; d += 32) {
    y[d] = to_f32(src[d]);
    ss = fmaf(y[d], y[d], ss);
  }
  const float r = rsqrtf(warp_sum(ss) / (float)a.D + a.eps);
  if (w)
    for (int d = lane; d < a.D; d += 32) y[d] = y[d] * r * to_f32(w[d]);
  __syncwarp();
  const float* row = a.cs + (long long)pl.pos * a.rot;
  for (int d = lane; d < a.D; d += 32) dst[d] = from_f32<T>(turn_one(a, y, row, d, 1.f));
}

template <typename T>
__global__ void __launch_bounds__(kThreads) rope_bwd_plain_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float rows[kWarps][DFLASH_PAGED_MAX_D];
  __shared__ float acc[kWarps][2][DFLASH_PAGED_MAX_D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* y = rows[warp];
  const int heads = a.Hq + a.Hkv;
  for (int d = lane; d < 2 * DFLASH_PAGED_MAX_D; d += 32) (&acc[warp][0][0])[d] = 0.f;  // queries, then keys
  const long long units = (long long)a.T * heads;
  for (long long unit = (long long)blockIdx.x * kWarps + warp; unit < units; unit += (long long)gridDim.x * kWarps) {
    const int t = (int)(unit / heads), h = (int)(unit % heads);
    const Place pl = place_position(a, t);
    if (!pl.ok) continue;
    const bool is_q = h < a.Hq;
    const long long at = is_q ? ((long long)t * a.Hq + h) * a.D : ((long long)t * a.Hkv + (h - a.Hq)) * a.D;
    const T* src = is_q ? static_cast<const T*>(a.q) + t * a.qs + (long long)h * a.D
                        : static_cast<const T*>(a.k) + t * a.ks + (long long)(h - a.Hq) * a.D;
    const T* dsrc = static_cast<const T*>(is_q ? a.dqo : a.dko) + at;
    const T* w = static_cast<const T*>(is_q ? a.wq : a.wk);
    T* dst = static_cast<T*>(is_q ? a.qo : a.ko) + at;
    const float* row = a.cs + (long long)pl.pos * a.rot;
    __syncwarp();
    for (int d = lane; d < a.D; d += 32) y[d] = to_f32(dsrc[d]);
    __syncwarp();
    float ss = 0.f, dot = 0.f;
    if (w)
      for (int d = lane; d < a.D; d += 32) {
        const float x = to_f32(src[d]);
        ss = fmaf(x, x, ss);
        dot = fmaf(turn_one(a, y, row, d, -1.f) * to_f32(w[d]), x, dot);
      }
    const float r = rsqrtf(warp_sum(ss) / (float)a.D + a.eps);
    const float c = warp_sum(dot) * r * r / (float)a.D;
    for (int d = lane; d < a.D; d += 32) {
      const float g = turn_one(a, y, row, d, -1.f);
      if (w) {
        const float x = to_f32(src[d]);
        acc[warp][is_q ? 0 : 1][d] += g * x * r;
        dst[d] = from_f32<T>(r * (g * to_f32(w[d]) - x * c));
      } else {
        dst[d] = from_f32<T>(g);
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.D; i += kThreads) {
    const int w = i / a.D, d = i % a.D;
    float s = 0.f;
    for (int k = 0; k < kWarps; ++k) s += acc[k][w][d];
    a.dw_part[((long long)blockIdx.x * 2 + w) * a.D + d] = s;  // even rows the query weight, odd rows the key weight
  }
}

// ---------------------------------------------------------------- host side
constexpr int kBwdBlocks = 608;  // 152 SMs x 4 blocks of 256 threads

bool on(const void* p, size_t bytes) { return ((uintptr_t)p % bytes) == 0; }

// Whether planes and addresses suit the four-component vectors.
bool vectors(const RopeArgs& a, bool bf16, bool paged, bool bwd) {
  const size_t b = bf16 ? 8 : 16;
  bool ok = a.rot % 8 == 0 && (a.rot == 0 || on(a.cs, 16));
  if (a.Hq > 0) ok = ok && on(a.q, b) && a.qs % 4 == 0 && on(a.qo, b) && on(a.wq, b);
  if (a.Hkv > 0) ok = ok && on(a.k, b) && a.ks % 4 == 0 && on(a.ko, b) && on(a.wk, b);
  if (paged) ok = ok && on(a.v, b) && a.vs % 4 == 0 && on(a.kc, b) && on(a.vc, b) && a.kps % 4 == 0 && a.vps % 4 == 0;
  if (bwd) ok = ok && on(a.dqo, b) && on(a.dko, b);
  return ok;
}

template <typename T, int LANES, int HPG, bool PAGED>
cudaError_t run_fwd(const RopeArgs& a, cudaStream_t s) {
  constexpr int groups = kThreads / LANES;
  const int nq = (a.Hq + HPG - 1) / HPG, nk = (a.Hkv + HPG - 1) / HPG, nchunk = nq + (PAGED ? 2 : 1) * nk;
  const long long blocks = ((long long)a.T + groups - 1) / groups * nchunk;
  if (blocks >= (1ll << 31)) return cudaErrorInvalidConfiguration;
  rope_fwd_kernel<T, LANES, HPG, PAGED><<<(unsigned)blocks, kThreads, 0, s>>>(a, nq, nk, nchunk);
  count_launch();
  return cudaGetLastError();
}

// Heads a group: as many as still give every SM two blocks.  The vectors of 8 (bf16)
// or 4 (fp32) heads are 128 bytes a lane in flight.  16 tokens of 40 heads take 2.1 us
// (3.5 with 8 heads a group), 32768 take 116 (217 with one).  Appending 1024 tokens of
// 48 heads: 6.6 us so, 7.4 us with four blocks an SM asked for, 10.8 with one head.
template <typename T, int LANES, bool PAGED>
cudaError_t pick_fwd(const RopeArgs& a, cudaStream_t s) {
  constexpr int most = sizeof(T) == 2 ? 8 : 4;
  const long long rows = ((long long)a.T + kThreads / LANES - 1) / (kThreads / LANES);
  const long long want = 152 * 2, heads = a.Hq + (PAGED ? 2 : 1) * a.Hkv;
  if (rows * heads / most >= want) return run_fwd<T, LANES, most, PAGED>(a, s);
  if (rows * heads / 4 >= want) return run_fwd<T, LANES, 4, PAGED>(a, s);
  if (rows * heads / 2 >= want) return run_fwd<T, LANES, 2, PAGED>(a, s);
  return run_fwd<T, LANES, 1, PAGED>(a, s);
}

template <typename T, bool PAGED>
cudaError_t type_fwd(const RopeArgs& a, cudaStream_t s) {
  if (vectors(a, sizeof(T) == 2, PAGED, false)) {
    if (a.D <= 64) return pick_fwd<T, 8, PAGED>(a, s);
    if (a.D <= 128) return pick_fwd<T, 16, PAGED>(a, s);
    return pick_fwd<T, 32, PAGED>(a, s);
  }
  const int heads = a.Hq + (PAGED ? 2 : 1) * a.Hkv;
  const long long blocks = ((long long)a.T * heads + kWarps - 1) / kWarps;
  if (blocks >= (1ll << 31)) return cudaErrorInvalidConfiguration;
  rope_fwd_plain_kernel<T, PAGED><<<(unsigned)blocks, kThreads, 0, s>>>(a);
  count_launch();
  return cudaGetLastError();
}

// How the partial norm gradients lie in the workspace.
struct DwRows {
  int blocks, nq, nchunk;
};

template <typename T, int LANES>
DwRows run_bwd(const RopeArgs& a, cudaStream_t s) {
  constexpr int groups = kThreads / LANES;
  // Heads a chunk: as many as still leave a full grid of blocks with work (32768 tokens
  // of 40 heads: 183 us with 8, 190 with 4, 270 with one).
  int hpg = 8;
  auto chunks = [&](int h) { return (h + hpg - 1) / hpg; };
  while (hpg > 1 &&
         ((long long)a.T + groups - 1) / groups * (chunks(a.Hq) + chunks(a.Hkv)) < kBwdBlocks)
    hpg >>= 1;
  while (chunks(a.Hq) + chunks(a.Hkv) > kBwdBlocks) hpg *= 2;
  DwRows d;
  d.nq = chunks(a.Hq);
  d.nchunk = d.nq + chunks(a.Hkv);
  const long long need = ((long long)a.T + groups - 1) / groups, most = kBwdBlocks / d.nchunk;
  d.blocks = (int)(need < most ? need : most) * d.nchunk;
  rope_bwd_kernel<T, LANES><<<d.blocks, kThreads, 0, s>>>(a, hpg, d.nq, d.nchunk);
  return d;
}

template <typename T>
cudaError_t type_bwd(const RopeArgs& a, float* dwq, float* dwk, cudaStream_t s) {
  DwRows d;
  if (vectors(a, sizeof(T) == 2, false, true)) {
    d = a.D <= 64 ? run_bwd<T, 8>(a, s) : a.D <= 128 ? run_bwd<T, 16>(a, s) : run_bwd<T, 32>(a, s);
  } else {
    const long long need = ((long long)a.T * (a.Hq + a.Hkv) + kWarps - 1) / kWarps;
    const int blocks = (int)(need < kBwdBlocks / 2 ? need : kBwdBlocks / 2);
    rope_bwd_plain_kernel<T><<<blocks, kThreads, 0, s>>>(a);
    d = {2 * blocks, 1, 2};
  }
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (!dwq && !dwk)) return e;
  rope_dw_kernel<<<dim3(a.D / kDwCols, 2), kDwCols * kDwRows, 0, s>>>(a.dw_part, d.blocks, d.nq, d.nchunk, a.D, dwq, dwk);
  count_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs& a, bool bf16, bool paged, cudaStream_t stream) {
  if (paged) return bf16 ? type_fwd<__nv_bfloat16, true>(a, stream) : type_fwd<float, true>(a, stream);
  return bf16 ? type_fwd<__nv_bfloat16, false>(a, stream) : type_fwd<float, false>(a, stream);
}

size_t rope_bwd_workspace_bytes(int D) { return sizeof(float) * (size_t)kBwdBlocks * D; }

cudaError_t launch_qk_norm_rope_bwd(RopeArgs a, bool bf16, float* dwq, float* dwk, cudaStream_t stream) {
  // Groups without a token take part with x = 0: with eps = 0 their r would be infinite, and
  // 0 times that reach dw.  (Telling them apart in the kernel: 186 us for 184.)
  if (a.eps < FLT_MIN) a.eps = FLT_MIN;
  return bf16 ? type_bwd<__nv_bfloat16>(a, dwq, dwk, stream) : type_bwd<float>(a, dwq, dwk, stream);
}

}  // namespace dflash
