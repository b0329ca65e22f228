// attn_paged.cu -- attention of new tokens over a paged key/value cache on the
// CUDA cores (fp32, and the bf16 shapes the tensor-core kernel does not take),
// and the kernel that merges the pieces of divided row tiles (sm_103a).
//
// Per row (token i of its request, query head) over the positions p it sees:
//   x_p = q . k_p scale log2 e,  out = sum_p 2^(x_p - m) v_p / l,  l = sum_p 2^(x_p - m)
// in one pass over the keys, the output rescaled by 2^(m_old - m_new) where the
// running maximum m rises.
//
// A CTA holds a row tile's queries in shared memory, walks its key tiles of 64
// positions (K, then V through one buffer) and multiplies in fp32: each thread
// has 4 rows of the scores and of the output in registers, so that one 16-byte
// shared-memory read feeds 4 to 16 multiply-adds.  Tiles of 64 rows, or of 16
// where no request has more rows than that (single tokens and short blocks with
// few heads a group, where 64-row tiles would multiply mostly padding).
// Rates: see the table of cases in the tests' companion benchmark; fp32 needs
// 4 D multiply-adds for each row and 8 D bytes of a position, so it is bound by
// the multiply-adds from about 10 rows on and by memory below.
#include <math.h>
#include <stdlib.h>
#include <string.h>

#include "paged.cuh"

namespace dflash {
namespace paged {

constexpr int kSimtBN = 64;
constexpr int kSimtThreads = 256;
constexpr int kSms = 152;
constexpr int kSimtMaxGrid = 2 * kSms;

namespace {

template <typename T>
struct alignas(16) Vec16 {
  T e[16 / sizeof(T)];
};

template <int BM, int DMAX>
struct SimtSmem {
  static constexpr int kStride = DMAX + 4;      // floats from row to row of Q, K and V
  static constexpr int kPStride = kSimtBN + 4;  // and of the scores
  float q[BM * kStride];
  float kv[kSimtBN * kStride];
  float p[BM * kPStride];
  float m[BM], l[BM], alpha[BM];
  int lim[BM];
  long long koff[kSimtBN], voff[kSimtBN];  // element offsets of the tile's rows; -1: zeros
  Range range;
  long long scratch[kSimtThreads / 32 + 1];
};

// Copies n rows of D elements to fp32 rows of shared memory (zeros where off < 0).
template <typename T, int STRIDE>
__device__ __forceinline__ void load_rows(float* dst, const T* base, const long long* off, int n, int D) {
  constexpr int VEC = 16 / sizeof(T);
  const int per = D / VEC;
  for (int i = threadIdx.x; i < n * per; i += kSimtThreads) {
    const int r = i / per, c = (i - r * per) * VEC;
    float x[VEC];
    const long long o = off[r];
    if (o >= 0) {
      const Vec16<T> v = *reinterpret_cast<const Vec16<T>*>(base + o + c);
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[e] = to_f32(v.e[e]);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < VEC; e += 4)
      *reinterpret_cast<float4*>(dst + r * STRIDE + c + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
  }
}

template <typename T, int BM, int DMAX>
__global__ void __launch_bounds__(kSimtThreads) paged_simt_kernel(const __grid_constant__ PagedArgs a) {
  constexpr int BN = kSimtBN;
  constexpr int TY = BM / 4, TX = kSimtThreads / TY;  // threads down the rows and across
  constexpr int CT = BN / TX;                         // scores a thread and row
  constexpr int NC = DMAX / TX;                       // output columns a thread and row
  constexpr int VW = NC < 4 ? NC : 4, U = NC / VW;
  static_assert(CT >= 1 && NC >= 1, "thread layout");
  using S = SimtSmem<BM, DMAX>;
  extern __shared__ __align__(16) uint8_t raw[];
  S& s = *reinterpret_cast<S*>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ty = tid / TX, tx = tid % TX;
  const int D = a.D;
  find_range<BN, kSimtThreads>(a, &s.range, s.scratch);
  Walker<BN> walk(a, s.range);
  Piece pc;
  int4 meta = make_int4(0, 0, 0, 0);
  while (walk.next(&pc)) {
    const int f0 = pc.rt * BM;  // first row of the tile within (request, key/value head)
    const int nrow = min(BM, pc.q.n * a.G - f0);
    __syncthreads();  // the previous piece is done with shared memory
    if (tid < BM) {
      s.m[tid] = -INFINITY;
      s.l[tid] = 0.f;
      const int tok = (f0 + tid) / a.G;
      s.lim[tid] = tid >= nrow ? 0 : a.causal ? max(0, pc.q.kv - pc.q.n + tok + 1) : pc.q.kv;
      if (tid < BN) {  // BM <= BN: the queries' offsets use the keys' table once
        const int g = (f0 + tid) % a.G;
        s.koff[tid] = tid < nrow ? ((long long)(pc.q.q0 + tok) * a.Hq + pc.h * a.G + g) * D : -1;
      }
    }
    __syncthreads();
    load_rows<T, S::kStride>(s.q, static_cast<const T*>(a.q), s.koff, BM, D);
    float o[4][NC];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < NC; ++c) o[i][c] = 0.f;
    for (int kt = pc.kt0; kt < pc.kt1; ++kt) {
      const int k0 = kt * BN;
      __syncthreads();  // the queries' offsets, or the previous tile, are done with
      if (tid < BN) {
        const int p = k0 + tid;
        long long ko = -1, vo = -1;
        if (p < pc.q.kv) {
          const int page = a.table[(long long)pc.r * a.max_pages + p / a.P];
          if (page < 0 || page >= a.num_pages) {
            record_error(a.err, DFLASH_ERR_INVALID);
          } else {
            const long long row = ((long long)(p % a.P) * a.Hkv + pc.h) * D;
            ko = page * a.kps + row;
            vo = page * a.vps + row;
          }
        }
        s.koff[tid] = ko;
        s.voff[tid] = vo;
      }
      __syncthreads();
      load_rows<T, S::kStride>(s.kv, static_cast<const T*>(a.kc), s.koff, BN, D);
      __syncthreads();
      // scores: rows 4 ty .., columns tx + TX j
      float x[4][CT];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < CT; ++j) x[i][j] = 0.f;
#pragma unroll 2
      for (int d = 0; d < D; d += 4) {
        float4 kk[CT];
#pragma unroll
        for (int j = 0; j < CT; ++j) kk[j] = *reinterpret_cast<const float4*>(s.kv + (tx + TX * j) * S::kStride + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 qq = *reinterpret_cast<const float4*>(s.q + (4 * ty + i) * S::kStride + d);
#pragma unroll
          for (int j = 0; j < CT; ++j)
            x[i][j] = fmaf(qq.x, kk[j].x, fmaf(qq.y, kk[j].y, fmaf(qq.z, kk[j].z, fmaf(qq.w, kk[j].w, x[i][j]))));
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < CT; ++j) s.p[(4 * ty + i) * S::kPStride + tx + TX * j] = x[i][j];
      __syncthreads();
      load_rows<T, S::kStride>(s.kv, static_cast<const T*>(a.vc), s.voff, BN, D);
      // softmax: a warp takes whole rows, two columns a lane
#pragma unroll
      for (int i = 0; i < BM / 8; ++i) {
        const int row = warp + 8 * i;
        float* pr = s.p + row * S::kPStride;
        const int lim = s.lim[row] - k0;
        const float x0 = lane < lim ? pr[lane] : -INFINITY;
        const float x1 = lane + 32 < lim ? pr[lane + 32] : -INFINITY;
        float mx = fmaxf(x0, x1);
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
        const float m0 = s.m[row];
        const float m1 = fmaxf(m0, mx * a.scale_log2);
        const float mm = m1 == -INFINITY ? 0.f : m1;
        // scaled and moved in one rounding: of large scores only the difference is rounded
        const float p0 = exp2f(fmaf(x0, a.scale_log2, -mm)), p1 = exp2f(fmaf(x1, a.scale_log2, -mm));
        pr[lane] = p0;
        pr[lane + 32] = p1;
        float sum = p0 + p1;
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
        if (lane == 0) {
          const float al = exp2f(m0 - mm);
          s.alpha[row] = al;
          s.l[row] = s.l[row] * al + sum;
          s.m[row] = m1;
        }
        __syncwarp();
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float al = s.alpha[4 * ty + i];
#pragma unroll
        for (int c = 0; c < NC; ++c) o[i][c] *= al;
      }
#pragma unroll 2
      for (int k = 0; k < BN; k += 4) {
        float pp[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 v = *reinterpret_cast<const float4*>(s.p + (4 * ty + i) * S::kPStride + k);
          pp[i][0] = v.x; pp[i][1] = v.y; pp[i][2] = v.z; pp[i][3] = v.w;
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int c0 = (tx + TX * u) * VW;
            float vv[VW];
#pragma unroll
            for (int e = 0; e < VW; ++e) vv[e] = 0.f;
            if (c0 < D) {
              const float* vp = s.kv + (k + kk) * S::kStride + c0;
              if constexpr (VW == 4) {
                const float4 v = *reinterpret_cast<const float4*>(vp);
                vv[0] = v.x; vv[1] = v.y; vv[2] = v.z; vv[3] = v.w;
              } else if constexpr (VW == 2) {
                const float2 v = *reinterpret_cast<const float2*>(vp);
                vv[0] = v.x; vv[1] = v.y;
              } else {
                vv[0] = *vp;
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int e = 0; e < VW; ++e) o[i][u * VW + e] = fmaf(pp[i][kk], vv[e], o[i][u * VW + e]);
          }
      }
    }
    // the piece's rows: finished, or left for the merge
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 4 * ty + i;
      if (row >= nrow) continue;
      const float l = s.l[row];
      if (pc.slot < 0) {
        const int tok = (f0 + row) / a.G, head = pc.h * a.G + (f0 + row) % a.G;
        const float inv = l > 0.f ? 1.f / l : 0.f;
        T* dst = static_cast<T*>(a.out) + ((long long)(pc.q.q0 + tok) * a.Hq + head) * D;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e = 0; e < VW; ++e) {
            const int c = (tx + TX * u) * VW + e;
            if (c < D) dst[c] = from_f32<T>(o[i][u * VW + e] * inv);
          }
        if (a.lse && tx == 0)
          a.lse[(long long)head * a.total_q + pc.q.q0 + tok] =
              l > 0.f ? (s.m[row] + log2f(l)) * 0.6931471805599453f : -INFINITY;
      } else {
        const long long at = (long long)pc.slot * a.rows + row;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e = 0; e < VW; ++e) {
            const int c = (tx + TX * u) * VW + e;
            if (c < D) a.part_o[at * D + c] = o[i][u * VW + e];
          }
        if (tx == 0) a.part_ml[at] = make_float2(s.m[row], l);
      }
    }
    if (pc.slot >= 0 && pc.shared) meta = pack_meta(pc);
  }
  if (tid == 0) a.meta[blockIdx.x] = meta;
}

// Merges the pieces of the row tile that CTA blockIdx.x began and left cut.  A warp
// takes a row, its lanes the columns.
template <typename T>
__global__ void __launch_bounds__(128) paged_merge_kernel(const __grid_constant__ PagedArgs a) {
  const int4 m = a.meta[blockIdx.x];
  if (m.x == 0) return;
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.y * 4 + (threadIdx.x >> 5);
  const Req q = load_request(a, m.y, false);
  const int f = m.w * a.rows + row;
  if (row >= a.rows || f >= q.n * a.G) return;
  const int first = 2 * blockIdx.x + 1;
  // slots first, first + 1, first + 3, ...: piece i > 0 continues the tile in CTA blockIdx.x + i
  auto slot = [&](int i) { return (long long)(i == 0 ? first : 2 * (blockIdx.x + i)) * a.rows + row; };
  float mx = -INFINITY;
  for (int i = lane; i < m.x; i += 32) mx = fmaxf(mx, a.part_ml[slot(i)].x);
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
  const float mm = mx == -INFINITY ? 0.f : mx;
  float l = 0.f;
  float o[DFLASH_PAGED_MAX_D / 32];
#pragma unroll
  for (int c = 0; c < DFLASH_PAGED_MAX_D / 32; ++c) o[c] = 0.f;
#pragma unroll 4
  for (int i = 0; i < m.x; ++i) {
    const long long at = slot(i);
    const float2 ml = a.part_ml[at];
    const float w = exp2f(ml.x - mm);
    l += w * ml.y;
    if (w > 0.f) {
#pragma unroll
      for (int c = 0; c < DFLASH_PAGED_MAX_D / 128; ++c) {
        const int d = 4 * lane + 128 * c;
        if (d < a.D) {
          const float4 v = *reinterpret_cast<const float4*>(a.part_o + at * a.D + d);
          o[4 * c] = fmaf(w, v.x, o[4 * c]);
          o[4 * c + 1] = fmaf(w, v.y, o[4 * c + 1]);
          o[4 * c + 2] = fmaf(w, v.z, o[4 * c + 2]);
          o[4 * c + 3] = fmaf(w, v.w, o[4 * c + 3]);
        }
      }
    }
  }
  const int tok = f / a.G, head = m.z * a.G + f % a.G;
  const float inv = l > 0.f ? 1.f / l : 0.f;
  T* dst = static_cast<T*>(a.out) + ((long long)(q.q0 + tok) * a.Hq + head) * a.D;
#pragma unroll
  for (int c = 0; c < DFLASH_PAGED_MAX_D / 128; ++c) {
    const int d = 4 * lane + 128 * c;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (d + e < a.D) dst[d + e] = from_f32<T>(o[4 * c + e] * inv);
  }
  if (a.lse && lane == 0)
    a.lse[(long long)head * a.total_q + q.q0 + tok] = l > 0.f ? (mx + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

template <typename T, int BM, int DMAX>
cudaError_t run_simt(const PagedArgs& a, int sms, int* grid, cudaStream_t s) {
  const size_t smem = sizeof(SimtSmem<BM, DMAX>);
  auto kernel = paged_simt_kernel<T, BM, DMAX>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  // two CTAs an SM where two fit, so that one loads while the other multiplies
  *grid = sms * (2 * (smem + 1024) <= 228 * 1024 ? 2 : 1);
  kernel<<<*grid, kSimtThreads, smem, s>>>(a);
  count_launch();
  return cudaGetLastError();
}

template <typename T, int BM>
cudaError_t pick_simt(const PagedArgs& a, int sms, int* grid, cudaStream_t s) {
  if (a.D <= 64) return run_simt<T, BM, 64>(a, sms, grid, s);
  if (a.D <= 128) return run_simt<T, BM, 128>(a, sms, grid, s);
  return run_simt<T, BM, 256>(a, sms, grid, s);
}

int simt_rows(int G, int max_q) { return (long long)G * max_q <= 16 ? 16 : 64; }

// DFLASH_FORCE_SIMT=1 (tests) routes every call to the CUDA-core kernel.
bool use_tensor_cores(bool bf16, int G, int D, int P) {
  const char* v = getenv("DFLASH_FORCE_SIMT");
  return bf16 && paged_tc_supported(G, D, P) && !(v && v[0] && strcmp(v, "0") != 0);
}

// Workspace: [meta | (m, l) | O], for the most CTAs a launch has.
struct PagedPlan {
  bool tc;
  int rows, max_grid;
  size_t ml, o, total;
};
PagedPlan plan_of(bool bf16, int Hq, int Hkv, int D, int max_q, int P) {
  PagedPlan p;
  const int G = Hq / Hkv;
  p.tc = use_tensor_cores(bf16, G, D, P);
  p.rows = p.tc ? paged_tc_rows(G, max_q) : simt_rows(G, max_q);
  p.max_grid = p.tc ? kSms : kSimtMaxGrid;
  const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t slots = 2 * (size_t)p.max_grid * p.rows;
  p.ml = up(kSimtMaxGrid * sizeof(int4));
  p.o = p.ml + up(slots * sizeof(float2));
  p.total = p.o + up(slots * D * sizeof(float));
  return p;
}

}  // namespace
}  // namespace paged

using namespace paged;

size_t paged_workspace_bytes(bool bf16, int Hq, int Hkv, int D, int max_q, int P) {
  return plan_of(bf16, Hq, Hkv, D, max_q, P).total;
}

cudaError_t launch_attn_paged(PagedArgs a, bool bf16, void* ws, cudaStream_t stream) {
  int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  if (sms > kSms) sms = kSms;
  const PagedPlan p = plan_of(bf16, a.Hq, a.Hkv, a.D, a.max_q, a.P);
  a.rows = p.rows;
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.meta = reinterpret_cast<int4*>(w);
  a.part_ml = reinterpret_cast<float2*>(w + p.ml);
  a.part_o = reinterpret_cast<float*>(w + p.o);
  int grid = sms;
  cudaError_t e;
  // Without a page there is no tensor to describe to TMA: the CUDA-core kernel with
  // its small row tiles (2 x 152 CTAs x 16 rows fit the 152 x 65 or more planned).
  if (p.tc && a.num_pages > 0) {
    e = launch_paged_tc(a, grid, stream);
  } else {
    if (p.tc) a.rows = 16;
    if (a.rows == 16)
      e = bf16 ? pick_simt<__nv_bfloat16, 16>(a, sms, &grid, stream) : pick_simt<float, 16>(a, sms, &grid, stream);
    else
      e = bf16 ? pick_simt<__nv_bfloat16, 64>(a, sms, &grid, stream) : pick_simt<float, 64>(a, sms, &grid, stream);
  }
  if (e != cudaSuccess) return e;
  const dim3 mg(grid, (a.rows + 3) / 4);
  if (bf16) paged_merge_kernel<__nv_bfloat16><<<mg, 128, 0, stream>>>(a);
  else paged_merge_kernel<float><<<mg, 128, 0, stream>>>(a);
  count_launch();
  return cudaGetLastError();
}

}  // namespace dflash
