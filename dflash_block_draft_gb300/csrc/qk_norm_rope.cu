// qk_norm_rope.cu -- RMS norm and position rotation of query and key heads, the
// same on the way into a paged cache, and the backward pass (sm_103a).
//
//   y = x (mean x^2 + eps)^-1/2 w,   out = Rot(pos) y
//   backward: g = Rot(pos)^T dout, dw = sum g x^, dx = r (g w - x^ mean(g w x^))
//
// All of it is bound by memory: about ten operations a component against 4 (bf16,
// in and out) to 12 bytes.  So a head is held in the registers of a group of 8,
// 16 or 32 lanes, each with one or two 16-byte vectors of it: the mean is a
// shuffle reduction inside the group, the partner component of a plane in the
// other half of the head comes by one shuffle, and nothing goes through shared
// memory.  A group takes several heads of ONE token, so that the token's cosines
// and sines (as many bytes in fp32 as two bf16 heads) are read once and stay in
// registers, and the heads' loads are in flight together.
// Head shapes whose planes cut through the vectors, and misaligned tensors, run
// on a plain kernel with a warp for each head and its row in shared memory.
#include "common.cuh"
#include "internal.h"

namespace dflash {
namespace {

constexpr int kThreads = 256;

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Vec {
  T e[VEC];
};

template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float* x) {
  const Vec<T, VEC> v = *reinterpret_cast<const Vec<T, VEC>*>(p);
#pragma unroll
  for (int i = 0; i < VEC; ++i) x[i] = to_f32(v.e[i]);
}

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float* x) {
  Vec<T, VEC> v;
#pragma unroll
  for (int i = 0; i < VEC; ++i) v.e[i] = from_f32<T>(x[i]);
  *reinterpret_cast<Vec<T, VEC>*>(p) = v;
}

// Where a token goes: its position and, for a paged call, the element offsets of
// its cache rows.  False: the token is skipped.
struct Place {
  int pos;
  long long krow, vrow;
};

template <bool PAGED>
__device__ __forceinline__ bool place_token(const RopeArgs& a, int t, Place* pl) {
  if (!PAGED) {
    pl->pos = a.rot > 0 ? a.pos[t] : 0;
    if (a.rot > 0 && (pl->pos < 0 || pl->pos >= a.max_pos)) {
      record_error(a.err, DFLASH_ERR_INVALID);
      return false;
    }
    return true;
  }
  if (t >= a.q_off[a.R]) return false;  // padding behind the last request
  int lo = 0, hi = a.R;
  while (hi - lo > 1) {  // the last request that begins at or before t
    const int mid = (lo + hi) >> 1;
    if (a.q_off[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int q0 = a.q_off[lo], q1 = a.q_off[lo + 1];
  const long long p = (long long)a.kv_lens[lo] - (q1 - q0) + (t - q0);
  if (q0 < 0 || q0 > t || q1 <= t || q1 > a.T || p < 0 || p >= (long long)a.max_pages * a.P ||
      (a.rot > 0 && p >= a.max_pos)) {
    record_error(a.err, DFLASH_ERR_INVALID);
    return false;
  }
  const int page = a.table[(long long)lo * a.max_pages + p / a.P];
  if (page < 0 || page >= a.num_pages) {
    record_error(a.err, DFLASH_ERR_INVALID);
    return false;
  }
  pl->pos = (int)p;
  const long long row = (p % a.P) * (long long)a.Hkv * a.D;
  pl->krow = page * a.kps + row;
  pl->vrow = page * a.vps + row;
  return true;
}

// A lane's components of a head: VPL vectors of VEC, vector j at chunk lane + LANES j.
template <int VEC, int LANES, int VPL>
struct Rotor {
  float cos[VPL][VEC], sin[VPL][VEC];  // sin carries the sign of the component
  int mate[VPL];                       // chunk that holds the partner components (half-split planes)
  bool turned[VPL];

  __device__ __forceinline__ void load(const RopeArgs& a, int pos, int lane, bool active) {
    const int h = a.rot >> 1;
    const float* row = a.cs + (long long)pos * a.rot;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int d = (lane + LANES * j) * VEC;
      turned[j] = active && d < a.rot;
      const bool second = !a.interleaved && d >= h;
      mate[j] = !turned[j] || a.interleaved ? lane + LANES * j : (second ? d - h : d + h) / VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int ang = a.interleaved ? (d + e) >> 1 : (second ? d - h : d) + e;
        cos[j][e] = turned[j] ? row[ang] : 1.f;
        const float sn = turned[j] ? row[h + ang] : 0.f;
        const bool first = a.interleaved ? (e & 1) == 0 : !second;
        sin[j][e] = first ? -sn : sn;
      }
    }
  }

  // x := x rotated (dir = 1) or rotated back (dir = -1).  Whole warp.
  __device__ __forceinline__ void apply(float (&x)[VPL][VEC], int interleaved, float dir) const {
    float y[VPL][VEC];
    if (interleaved) {
#pragma unroll
      for (int j = 0; j < VPL; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) y[j][e] = x[j][e ^ 1];
    } else {
#pragma unroll
      for (int j = 0; j < VPL; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          if (VPL == 1) {
            y[j][e] = __shfl_sync(0xffffffffu, x[0][e], mate[0], LANES);
          } else {
            const float y0 = __shfl_sync(0xffffffffu, x[0][e], mate[j] % LANES, LANES);
            const float y1 = __shfl_sync(0xffffffffu, x[VPL - 1][e], mate[j] % LANES, LANES);
            y[j][e] = mate[j] < LANES ? y0 : y1;
          }
        }
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (turned[j]) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[j][e] = fmaf(x[j][e], cos[j][e], dir * y[j][e] * sin[j][e]);
      }
  }
};

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o, LANES);
  return v;
}

// A group of LANES takes HPG heads of one token.  Heads count q, then k, then
// (paged) v.  Work units are [token][head chunk].
template <typename T, int VEC, int LANES, int VPL, int HPG, bool PAGED>
__global__ void __launch_bounds__(kThreads) rope_fwd_kernel(const __grid_constant__ RopeArgs a, int nchunk) {
  const int lane = threadIdx.x % LANES;
  const long long unit = (long long)blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
  const int t = (int)min(unit / nchunk, (long long)a.T);
  const int h0 = (int)(unit % nchunk) * HPG;
  const int heads = a.Hq + (PAGED ? 2 : 1) * a.Hkv;
  Place pl = {0, 0, 0};
  const bool ok = t < a.T && place_token<PAGED>(a, t, &pl);
  bool in[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) in[j] = ok && (lane + LANES * j) * VEC < a.D;
  float x[HPG][VPL][VEC];
#pragma unroll
  for (int u = 0; u < HPG; ++u) {
    const int h = h0 + u;
    const T* src;
    if (h < a.Hq) src = static_cast<const T*>(a.q) + t * a.qs + (long long)h * a.D;
    else if (!PAGED || h < a.Hq + a.Hkv) src = static_cast<const T*>(a.k) + t * a.ks + (long long)(h - a.Hq) * a.D;
    else src = static_cast<const T*>(a.v) + t * a.vs + (long long)(h - a.Hq - a.Hkv) * a.D;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[u][j][e] = 0.f;
      if (in[j] && h < heads) load_vec<T, VEC>(src + (lane + LANES * j) * VEC, x[u][j]);
    }
  }
  Rotor<VEC, LANES, VPL> rot;
  rot.load(a, pl.pos, lane, ok);
#pragma unroll
  for (int u = 0; u < HPG; ++u) {
    const int h = h0 + u;
    const bool is_q = h < a.Hq, is_v = PAGED && h >= a.Hq + a.Hkv;
    if (__any_sync(0xffffffffu, h < heads && !is_v)) {
      const T* w = static_cast<const T*>(is_q ? a.wq : a.wk);
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < VPL; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss = fmaf(x[u][j][e], x[u][j][e], ss);
      ss = group_sum<LANES>(ss);
      const float r = rsqrtf(ss / (float)a.D + a.eps);
      float y[VPL][VEC];
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        float wv[VEC];
        const bool normed = w != nullptr && in[j];
        if (normed) load_vec<T, VEC>(w + (lane + LANES * j) * VEC, wv);
#pragma unroll
        for (int e = 0; e < VEC; ++e) y[j][e] = normed ? x[u][j][e] * r * wv[e] : x[u][j][e];
      }
      rot.apply(y, a.interleaved, 1.f);
      if (!is_v) {
#pragma unroll
        for (int j = 0; j < VPL; ++j)
#pragma unroll
          for (int e = 0; e < VEC; ++e) x[u][j][e] = y[j][e];
      }
    }
    if (h >= heads) continue;
    T* dst;
    if (is_q) dst = static_cast<T*>(a.qo) + ((long long)t * a.Hq + h) * a.D;
    else if (!PAGED) dst = static_cast<T*>(a.ko) + ((long long)t * a.Hkv + (h - a.Hq)) * a.D;
    else if (!is_v) dst = static_cast<T*>(a.kc) + pl.krow + (long long)(h - a.Hq) * a.D;
    else dst = static_cast<T*>(a.vc) + pl.vrow + (long long)(h - a.Hq - a.Hkv) * a.D;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (in[j]) store_vec<T, VEC>(dst + (lane + LANES * j) * VEC, x[u][j]);
  }
}

// Backward: groups walk the units with the grid's stride and keep their share of
// the norm gradients in registers; a block adds its groups up in shared memory
// and writes one row of partial sums, so that the order of the sums is fixed.
template <typename T, int VEC, int LANES, int VPL>
__global__ void __launch_bounds__(kThreads)
    rope_bwd_kernel(const __grid_constant__ RopeArgs a, int nchunk, int hpg) {
  constexpr int kGroups = kThreads / LANES;
  __shared__ float red[kGroups][VPL * LANES * VEC];
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const int heads = a.Hq + a.Hkv;
  float dw[2][VPL][VEC];
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int j = 0; j < VPL; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) dw[w][j][e] = 0.f;
  const long long units = (long long)a.T * nchunk;
  for (long long base = (long long)blockIdx.x * kGroups; base < units; base += (long long)gridDim.x * kGroups) {
    const long long unit = base + group;
    const int t = (int)min(unit / nchunk, (long long)a.T);
    const int h0 = (int)(unit % nchunk) * hpg;
    Place pl = {0, 0, 0};
    const bool ok = t < a.T && place_token<false>(a, t, &pl);
    bool in[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) in[j] = ok && (lane + LANES * j) * VEC < a.D;
    Rotor<VEC, LANES, VPL> rot;
    rot.load(a, pl.pos, lane, ok);
#pragma unroll 2
    for (int u = 0; u < hpg; ++u) {
      const int h = h0 + u;
      const bool is_q = h < a.Hq, have = h < heads;
      const long long at = is_q ? ((long long)t * a.Hq + h) * a.D : ((long long)t * a.Hkv + (h - a.Hq)) * a.D;
      const T* w = static_cast<const T*>(is_q ? a.wq : a.wk);
      const bool normed = w != nullptr;
      const T* src = is_q ? static_cast<const T*>(a.q) + t * a.qs + (long long)h * a.D
                          : static_cast<const T*>(a.k) + t * a.ks + (long long)(h - a.Hq) * a.D;
      const T* dsrc = static_cast<const T*>(is_q ? a.dqo : a.dko) + at;
      float x[VPL][VEC], g[VPL][VEC], wv[VPL][VEC];
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[j][e] = g[j][e] = wv[j][e] = 0.f;
        if (in[j] && have) {
          const int d = (lane + LANES * j) * VEC;
          load_vec<T, VEC>(dsrc + d, g[j]);
          if (normed) {
            load_vec<T, VEC>(src + d, x[j]);
            load_vec<T, VEC>(w + d, wv[j]);
          }
        }
      }
      rot.apply(g, a.interleaved, -1.f);
      float ss = 0.f, dot = 0.f;
#pragma unroll
      for (int j = 0; j < VPL; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          ss = fmaf(x[j][e], x[j][e], ss);
          dot = fmaf(g[j][e] * wv[j][e], x[j][e], dot);
        }
      ss = group_sum<LANES>(ss);
      dot = group_sum<LANES>(dot);
      const float r = rsqrtf(ss / (float)a.D + a.eps);
      const float c = dot * r * r / (float)a.D;  // mean(g w x^) r, the factor of x inside the bracket
      if (have) {
        T* dst = static_cast<T*>(is_q ? a.qo : a.ko) + at;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float gx = normed ? g[j][e] * x[j][e] * r : 0.f;
            dw[0][j][e] += is_q ? gx : 0.f;
            dw[1][j][e] += is_q ? 0.f : gx;
            if (normed) g[j][e] = r * (g[j][e] * wv[j][e] - x[j][e] * c);
          }
          if (in[j]) store_vec<T, VEC>(dst + (lane + LANES * j) * VEC, g[j]);
        }
      }
    }
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < VPL; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) red[group][(lane + LANES * j) * VEC + e] = dw[w][j][e];
    __syncthreads();
    for (int d = threadIdx.x; d < a.D; d += kThreads) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) s += red[i][d];
      a.dw_part[((long long)blockIdx.x * 2 + w) * a.D + d] = s;
    }
  }
}

// Sums the blocks' rows: 32 columns a block, 32 threads down each column.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* part, int blocks, int D, float* dwq, float* dwk) {
  __shared__ float red[32][33];
  const int c = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int d = blockIdx.x * 32 + c, w = blockIdx.y;
  float* dst = w ? dwk : dwq;
  if (!dst) return;
  float s = 0.f;
  if (d < D)
    for (int b = y; b < blocks; b += 32) s += part[((long long)b * 2 + w) * D + d];
  red[y][c] = s;
  __syncthreads();
  if (y == 0 && d < D) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += red[i][c];
    dst[d] = sum;
  }
}

// ---------------------------------------------------------------- plain kernels
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float warp_sum(float v) { return group_sum<32>(v); }

// Component d of the rotation of row y (shared memory), dir as in Rotor::apply.
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
  if (unit >= (long long)a.T * heads) return;
  const int t = (int)(unit / heads), h = (int)(unit % heads);
  Place pl = {0, 0, 0};
  if (!place_token<PAGED>(a, t, &pl)) return;
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
  for (int d = lane; d < 2 * DFLASH_PAGED_MAX_D; d += 32) (&acc[warp][0][0])[d] = 0.f;
  const long long units = (long long)a.T * heads;
  for (long long unit = (long long)blockIdx.x * kWarps + warp; unit < units; unit += (long long)gridDim.x * kWarps) {
    const int t = (int)(unit / heads), h = (int)(unit % heads);
    Place pl = {0, 0, 0};
    if (!place_token<false>(a, t, &pl)) continue;
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
    a.dw_part[((long long)blockIdx.x * 2 + w) * a.D + d] = s;
  }
}

// ---------------------------------------------------------------- host side
constexpr int kBwdBlocks = 608;  // 152 SMs x 4 resident blocks

bool on(const void* p, size_t bytes) { return ((uintptr_t)p % bytes) == 0; }

// Widest vector (elements) that the shape and the addresses allow; 0: the plain kernels.
int vector_width(const RopeArgs& a, bool bf16, bool paged, bool bwd) {
  const size_t esz = bf16 ? 2 : 4;
  for (int vec = bf16 ? 8 : 4; vec >= 4; vec -= 4) {
    const size_t b = vec * esz;
    const int plane = a.interleaved ? a.rot : a.rot / 2;
    bool ok = a.D % vec == 0 && plane % vec == 0;
    if (a.Hq > 0) ok = ok && (!a.q || (on(a.q, b) && a.qs % vec == 0)) && on(a.qo, b) && on(a.wq, b);
    if (a.Hkv > 0) ok = ok && (!a.k || (on(a.k, b) && a.ks % vec == 0)) && on(a.ko, b) && on(a.wk, b);
    if (paged) ok = ok && on(a.v, b) && a.vs % vec == 0 && on(a.kc, b) && on(a.vc, b) && a.kps % vec == 0 && a.vps % vec == 0;
    if (bwd) ok = ok && on(a.dqo, b) && on(a.dko, b);
    if (ok) return vec;
  }
  return 0;
}

template <typename T, int VEC, int LANES, int VPL, int HPG, bool PAGED>
cudaError_t run_fwd(const RopeArgs& a, cudaStream_t s) {
  const int heads = a.Hq + (PAGED ? 2 : 1) * a.Hkv;
  const int nchunk = (heads + HPG - 1) / HPG, groups = kThreads / LANES;
  const long long blocks = ((long long)a.T * nchunk + groups - 1) / groups;
  if (blocks >= (1ll << 31)) return cudaErrorInvalidConfiguration;
  rope_fwd_kernel<T, VEC, LANES, VPL, HPG, PAGED><<<(unsigned)blocks, kThreads, 0, s>>>(a, nchunk);
  count_launch();
  return cudaGetLastError();
}

// Four heads a group once the groups still fill the machine (152 SMs x 2048
// threads); with fewer tokens one head a group, which shortens the call.
template <typename T, int VEC, int LANES, int VPL, bool PAGED>
cudaError_t pick_fwd(const RopeArgs& a, cudaStream_t s) {
  const long long lanes = (long long)a.T * (a.Hq + (PAGED ? 2 : 1) * a.Hkv) * LANES;
  return lanes / 4 >= 152ll * 2048 ? run_fwd<T, VEC, LANES, VPL, 4, PAGED>(a, s)
                                   : run_fwd<T, VEC, LANES, VPL, 1, PAGED>(a, s);
}

template <typename T, int VEC, bool PAGED>
cudaError_t width_fwd(const RopeArgs& a, cudaStream_t s) {
  const int chunks = a.D / VEC;
  if (chunks <= 8) return pick_fwd<T, VEC, 8, 1, PAGED>(a, s);
  if (chunks <= 16) return pick_fwd<T, VEC, 16, 1, PAGED>(a, s);
  if (chunks <= 32) return pick_fwd<T, VEC, 32, 1, PAGED>(a, s);
  return pick_fwd<T, VEC, 32, 2, PAGED>(a, s);
}

template <typename T, bool PAGED>
cudaError_t type_fwd(const RopeArgs& a, cudaStream_t s) {
  const int vec = vector_width(a, sizeof(T) == 2, PAGED, false);
  if (vec == 8) return width_fwd<T, sizeof(T) == 2 ? 8 : 4, PAGED>(a, s);
  if (vec == 4) return width_fwd<T, 4, PAGED>(a, s);
  const int heads = a.Hq + (PAGED ? 2 : 1) * a.Hkv;
  const long long blocks = ((long long)a.T * heads + kWarps - 1) / kWarps;
  if (blocks >= (1ll << 31)) return cudaErrorInvalidConfiguration;
  rope_fwd_plain_kernel<T, PAGED><<<(unsigned)blocks, kThreads, 0, s>>>(a);
  count_launch();
  return cudaGetLastError();
}

template <typename T, int VEC, int LANES, int VPL>
void run_bwd(const RopeArgs& a, int* blocks, cudaStream_t s) {
  constexpr int groups = kThreads / LANES;
  const int heads = a.Hq + a.Hkv;
  // heads a group: as many as leave every group of the full grid at least one unit
  int hpg = 8;
  while (hpg > 1 && (long long)a.T * ((heads + hpg - 1) / hpg) < (long long)kBwdBlocks * groups) hpg >>= 1;
  const int nchunk = (heads + hpg - 1) / hpg;
  const long long need = ((long long)a.T * nchunk + groups - 1) / groups;
  *blocks = (int)(need < kBwdBlocks ? need : kBwdBlocks);
  rope_bwd_kernel<T, VEC, LANES, VPL><<<*blocks, kThreads, 0, s>>>(a, nchunk, hpg);
}

template <typename T, int VEC>
void width_bwd(const RopeArgs& a, int* blocks, cudaStream_t s) {
  const int chunks = a.D / VEC;
  if (chunks <= 8) run_bwd<T, VEC, 8, 1>(a, blocks, s);
  else if (chunks <= 16) run_bwd<T, VEC, 16, 1>(a, blocks, s);
  else if (chunks <= 32) run_bwd<T, VEC, 32, 1>(a, blocks, s);
  else run_bwd<T, VEC, 32, 2>(a, blocks, s);
}

template <typename T>
cudaError_t type_bwd(const RopeArgs& a, float* dwq, float* dwk, cudaStream_t s) {
  const int vec = vector_width(a, sizeof(T) == 2, false, true);
  int blocks = 0;
  if (vec == 8) {
    width_bwd<T, sizeof(T) == 2 ? 8 : 4>(a, &blocks, s);
  } else if (vec == 4) {
    width_bwd<T, 4>(a, &blocks, s);
  } else {
    const long long need = ((long long)a.T * (a.Hq + a.Hkv) + kWarps - 1) / kWarps;
    blocks = (int)(need < kBwdBlocks ? need : kBwdBlocks);
    rope_bwd_plain_kernel<T><<<blocks, kThreads, 0, s>>>(a);
  }
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (!dwq && !dwk)) return e;
  rope_dw_kernel<<<dim3((a.D + 31) / 32, 2), 1024, 0, s>>>(a.dw_part, blocks, a.D, dwq, dwk);
  count_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs& a, bool bf16, bool paged, cudaStream_t stream) {
  if (paged) return bf16 ? type_fwd<__nv_bfloat16, true>(a, stream) : type_fwd<float, true>(a, stream);
  return bf16 ? type_fwd<__nv_bfloat16, false>(a, stream) : type_fwd<float, false>(a, stream);
}

size_t rope_bwd_workspace_bytes(int D) { return sizeof(float) * 2 * (size_t)kBwdBlocks * D; }

cudaError_t launch_qk_norm_rope_bwd(const RopeArgs& a, bool bf16, float* dwq, float* dwk, cudaStream_t stream) {
  return bf16 ? type_bwd<__nv_bfloat16>(a, dwq, dwk, stream) : type_bwd<float>(a, dwq, dwk, stream);
}

}  // namespace dflash
