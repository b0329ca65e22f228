// attn_paged.cu -- attention of new tokens over a paged key/value cache on the
// CUDA cores (fp32, and the bf16 shapes the tensor-core kernel does not take),
// and the kernel that merges the pieces of divided row tiles (sm_103a).
//
// Per row (token i of its request, query head) over the positions p it sees:
//   x_p = q . k_p scale log2 e,  out = sum_p 2^(x_p - m) v_p / l,  l = sum_p 2^(x_p - m)
// in one pass over the keys, the output rescaled by 2^(m_old - m_new) where the
// running maximum m rises.
//
// A CTA holds a row tile's queries in shared memory and walks its key tiles of 64
// positions (fp32 up to D = 64, 64-row tiles) or 32, which arrive by 16-byte
// asynchronous copies two tiles deep; the rows' offsets (page table and page row) are
// worked out one tile ahead of the copies.
// Each thread has 4 rows of the scores and of the output in registers, and all
// threads of a row lie in one warp, so that the softmax needs shuffles only and a
// key tile two block barriers.  Row tiles of 64 rows with 256 threads, or of 16 with
// 128 where no request has more rows (single tokens and short blocks with few
// heads a group, where 64-row tiles would multiply mostly padding; the smaller
// CTAs also put more copies in flight): 6 requests of up to 16 tokens with 16 fp32
// heads of 64, behind 300 to 4000 positions, take 30 us, 42 with 64-row tiles; 16
// single tokens of 16 heads of 128 take 107 us (3.8 TB/s), 156 with them.  fp32 needs
// 2 D multiply-adds for each row and 8 D bytes of a position, so it is bound by the
// multiply-adds, and by the shared memory that feeds them, from a few rows on and
// by memory below.  So are the bf16 shapes that come here: with D = 256 and 32 heads in 8
// groups, 16 single tokens behind 1000 to 8000 positions take 176 us (68 to read the keys and
// values), blocks of 16 tokens 766, and 512 tokens behind 8192 positions 3540, 40 TFLOP/s;
// with D = 128 and pages of 7 the last two take 406 and 1850.
#include <math.h>
#include <stdlib.h>
#include <string.h>

#include "paged.cuh"

namespace dflash {
namespace paged {

constexpr int kSms = 152;
// CTAs of a launch at most: 4 an SM with 16-row tiles, 2 with 64-row tiles.
constexpr int kSimtPerSm16 = 4, kSimtPerSm64 = 2;
constexpr int kSimtMaxGrid = kSimtPerSm16 * kSms;

namespace {

__device__ __forceinline__ void copy16(void* dst, const void* src, bool have) {  // zeros where !have
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src), "r"(have ? 16u : 0u)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                     __uint_as_float(v.y & 0xFFFF0000u));
}
__device__ __forceinline__ float2 load2(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 load2(const __nv_bfloat16* p) {
  const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

template <typename T, int BM, int DMAX>
struct Simt {
  // Positions of a key tile: two stages of K and V for two CTAs an SM, four of 16-row tiles
  // (bf16 with D = 128 and 64-row tiles: 160 us with 32, 172 with 64; fp32 with D = 64:
  // 64-row tiles 167 and 149, 16-row tiles 29 and 33).
  static constexpr int BN = sizeof(T) == 4 && DMAX <= 64 && BM == 64 ? 64 : 32;
  static constexpr int kThreads = BM == 16 ? 128 : 256;
  // CTAs an SM that the registers are kept to, where shared memory has room for them (bf16
  // 16-row tiles with D = 128: 63 us so, 113 with three and a grid of four)
  static constexpr int kPerSm = BM == 64 ? (DMAX <= 128 ? 2 : 1) : DMAX <= 64 || (sizeof(T) == 2 && DMAX <= 128) ? 4 : 1;
  static constexpr int kVec = 16 / sizeof(T);
  static constexpr int kStride = DMAX + kVec;  // elements from row to row of K and V
  static constexpr int kQStride = DMAX + 4;
  static constexpr int kPStride = BN + 4;
  struct Smem {
    T k[2][BN * kStride], v[2][BN * kStride];
    float q[BM * kQStride];
    float p[BM * kPStride];
    long long koff[3][BN], voff[3][BN];  // element offsets of the rows of tiles kt, kt + 1, kt + 2; -1: zeros
    Range range;
    long long scratch[kThreads / 32 + 1];
  };
};

template <typename T, int BM, int DMAX, bool TREE>
__global__ void __launch_bounds__(Simt<T, BM, DMAX>::kThreads, Simt<T, BM, DMAX>::kPerSm)
    paged_simt_kernel(const __grid_constant__ PagedArgs a) {
  using C = Simt<T, BM, DMAX>;
  constexpr int BN = C::BN, kThreads = C::kThreads, VEC = C::kVec;
  constexpr int TY = BM / 4, TX = kThreads / TY;  // threads down the rows and across
  constexpr int CT = BN / TX;                     // scores a thread and row
  constexpr int NC = DMAX / TX;                   // output columns a thread and row
  constexpr int VW = NC < 4 ? NC : 4, U = NC / VW;
  static_assert(CT >= 1 && NC >= 2 && TX <= 32, "thread layout");
  extern __shared__ __align__(16) uint8_t raw[];
  typename C::Smem& s = *reinterpret_cast<typename C::Smem*>(raw);
  const int tid = threadIdx.x;
  const int ty = tid / TX, tx = tid % TX;
  const int D = a.D;
  // copies: 16-byte piece tid % kPer of rows tid / kPer, + kRows, ...
  constexpr int kPer = DMAX / VEC, kRows = kThreads / kPer;
  static_assert(kRows >= 1 && BN % kRows == 0, "copy layout");
  find_range<BN, kThreads>(a, tid, &s.range, s.scratch, [] { __syncthreads(); });
  __syncthreads();
  Walker<BN> walk(a, s.range);
  Piece pc;
  Meta meta = no_meta();
  while (walk.next(&pc)) {
    const int f0 = pc.rt * BM;  // first row of the tile within (request, key/value head)
    const int nrow = min(BM, pc.q.n * a.G - f0);
    // offsets of key tile kt's row `tid` (threads below BN); the page's load is left in flight
    auto page_of = [&](int kt) {
      const int p = kt * BN + tid;
      return tid < BN && kt < pc.kt1 && p < pc.q.kv ? a.table[(long long)pc.r * a.max_pages + p / a.P] : -2;
    };
    auto put_offsets = [&](int kt, int page) {
      if (tid >= BN) return;
      long long ko = -1, vo = -1;
      if (page >= 0 && page < a.num_pages) {
        const long long row = ((long long)((kt * BN + tid) % a.P) * a.Hkv + pc.h) * D;
        ko = page * a.kps + row;
        vo = page * a.vps + row;
      } else if (page != -2 || (kt < pc.kt1 && kt * BN + tid < pc.q.kv)) {
        record_error(a.err, DFLASH_ERR_INVALID);
      }
      s.koff[kt % 3][tid] = ko;
      s.voff[kt % 3][tid] = vo;
    };
    auto fetch = [&](int kt) {  // its offsets are in place
      if (kt < pc.kt1) {
        const int c = tid % kPer * VEC;
        if (c < D) {
#pragma unroll
          for (int i = 0; i < BN / kRows; ++i) {
            const int r = tid / kPer + i * kRows;
            const long long ko = s.koff[kt % 3][r], vo = s.voff[kt % 3][r];
            copy16(&s.k[kt & 1][r * C::kStride + c], static_cast<const T*>(a.kc) + max(ko, 0ll) + c, ko >= 0);
            copy16(&s.v[kt & 1][r * C::kStride + c], static_cast<const T*>(a.vc) + max(vo, 0ll) + c, vo >= 0);
          }
        }
      }
      copy_commit();
    };
    put_offsets(pc.kt0, page_of(pc.kt0));
    put_offsets(pc.kt0 + 1, page_of(pc.kt0 + 1));
    for (int i = tid; i < BM * (D / 4); i += kThreads) {
      const int r = i / (D / 4), c = (i - r * (D / 4)) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < nrow) {
        const int f = f0 + r;
        x = load4(static_cast<const T*>(a.q) + ((long long)(pc.q.q0 + f / a.G) * a.Hq + pc.h * a.G + f % a.G) * D + c);
      }
      *reinterpret_cast<float4*>(s.q + r * C::kQStride + c) = x;
    }
    const int base = pc.q.kv - pc.q.n;  // position of the first new token
    int lim[4];
    float m[4], l[4];
    float2 o[4][NC / 2];  // in pairs of columns, for the packed multiply-adds
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 4 * ty + i;
      lim[i] = row >= nrow ? 0 : a.causal && !TREE ? max(0, base + (f0 + row) / a.G + 1) : pc.q.kv;
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < NC / 2; ++c) o[i][c] = make_float2(0.f, 0.f);
    }
    const bool idle = 32 / TX * 4 * (tid / 32) >= nrow;  // none of the warp's rows exists: it only copies
    __syncthreads();
    fetch(pc.kt0);
    for (int kt = pc.kt0; kt < pc.kt1; ++kt) {
      fetch(kt + 1);
      const int page = page_of(kt + 2);
      copy_wait<1>();
      __syncthreads();  // tile kt has landed
      const T* ks = s.k[kt & 1];
      const T* vs = s.v[kt & 1];
      const int k0 = kt * BN;
      if (!idle) {
        // scores: rows 4 ty .., columns tx + TX j
        float x[4][CT];
        float2 x2[4][CT];  // sums over the even and the odd components, for the packed multiply-adds
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < CT; ++j) x2[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
          float4 kk[CT];
#pragma unroll
          for (int j = 0; j < CT; ++j) kk[j] = load4(ks + (tx + TX * j) * C::kStride + d);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 qq = load4(s.q + (4 * ty + i) * C::kQStride + d);
#pragma unroll
            for (int j = 0; j < CT; ++j)
              x2[i][j] = __ffma2_rn(make_float2(qq.x, qq.y), make_float2(kk[j].x, kk[j].y),
                                    __ffma2_rn(make_float2(qq.z, qq.w), make_float2(kk[j].z, kk[j].w), x2[i][j]));
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < CT; ++j) x[i][j] = x2[i][j].x + x2[i][j].y;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float mx = -INFINITY;
          TreeBits<1> vis = {{~0ull}};
          if (TREE && k0 + BN > base)  // new tokens lie in this tile
            vis = tree_bits<1>(a.parents + pc.q.q0, min((f0 + 4 * ty + i) / a.G, pc.q.n - 1), base - k0);
#pragma unroll
          for (int j = 0; j < CT; ++j) {
            if (k0 + tx + TX * j >= lim[i] || (TREE && !((vis.w[0] >> (tx + TX * j)) & 1))) x[i][j] = -INFINITY;
            mx = fmaxf(mx, x[i][j]);
          }
#pragma unroll
          for (int w = TX / 2; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w, TX));
          const float m1 = fmaxf(m[i], mx * a.scale_log2);
          const float mm = m1 == -INFINITY ? 0.f : m1;
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < CT; ++j) {
            // scaled and moved in one rounding: of large scores only the difference is rounded
            const float e = exp2f(fmaf(x[i][j], a.scale_log2, -mm));
            s.p[(4 * ty + i) * C::kPStride + tx + TX * j] = e;
            sum += e;
          }
#pragma unroll
          for (int w = TX / 2; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w, TX);
          const float al = exp2f(m[i] - mm);
          l[i] = l[i] * al + sum;
          m[i] = m1;
#pragma unroll
          for (int c = 0; c < NC / 2; ++c) o[i][c] = __fmul2_rn(o[i][c], make_float2(al, al));
        }
        __syncwarp();  // the rows' weights, written by this warp alone
#pragma unroll 2
        for (int k = 0; k < BN; k += 4) {
          float pp[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 w = load4(s.p + (4 * ty + i) * C::kPStride + k);
            pp[i][0] = w.x; pp[i][1] = w.y; pp[i][2] = w.z; pp[i][3] = w.w;
          }
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const int c0 = (tx + TX * u) * VW;
              float2 vv[VW / 2];
#pragma unroll
              for (int e = 0; e < VW / 2; ++e) vv[e] = make_float2(0.f, 0.f);
              if (c0 < D) {
                const T* vp = vs + (k + kk) * C::kStride + c0;
                if constexpr (VW == 4) {
                  const float4 w = load4(vp);
                  vv[0] = make_float2(w.x, w.y);
                  vv[1] = make_float2(w.z, w.w);
                } else {
                  vv[0] = load2(vp);
                }
              }
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < VW / 2; ++e) {
                  float2& at = o[i][u * (VW / 2) + e];
                  at = __ffma2_rn(make_float2(pp[i][kk], pp[i][kk]), vv[e], at);
                }
            }
        }
      }
      put_offsets(kt + 2, page);
      __syncthreads();  // this stage's buffers may be filled again; the offsets are in place
    }
    copy_wait<0>();
    // the piece's rows: finished, or left for the merge
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 4 * ty + i;
      if (row >= nrow) continue;
      if (pc.slot < 0) {
        const int tok = (f0 + row) / a.G, head = pc.h * a.G + (f0 + row) % a.G;
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
        T* dst = static_cast<T*>(a.out) + ((long long)(pc.q.q0 + tok) * a.Hq + head) * D;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e = 0; e < VW; ++e) {
            const int c = (tx + TX * u) * VW + e;
            const float2 oo = o[i][(u * VW + e) / 2];
            if (c < D) dst[c] = from_f32<T>((e & 1 ? oo.y : oo.x) * inv);
          }
        if (a.lse && tx == 0)
          a.lse[(long long)head * a.total_q + pc.q.q0 + tok] =
              l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * 0.6931471805599453f;
      } else {
        const long long at = (long long)pc.slot * a.rows + row;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e = 0; e < VW; ++e) {
            const int c = (tx + TX * u) * VW + e;
            const float2 oo = o[i][(u * VW + e) / 2];
            if (c < D) a.part_o[at * D + c] = e & 1 ? oo.y : oo.x;
          }
        if (tx == 0) a.part_ml[at] = make_float2(m[i], l[i]);
      }
    }
    if (begins_cut(pc)) meta = meta_of(a, s.range, pc);
  }
  if (tid == 0) a.meta[blockIdx.x] = meta;
}

// Adds pieces i0 .. i0 + N - 1 of one row to (mx, l, o): a lane has CD float4 of columns, 4 LANES
// columns apart.
template <int N, int LANES, int CD, typename Slot>
__device__ __forceinline__ void merge_pieces(const PagedArgs& a, int i0, int count, Slot slot, int lane, float& mx,
                                             float& l, float4 (&o)[CD]) {
  float2 ml[N];
  float4 v[N][CD];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    ml[i] = make_float2(-INFINITY, 0.f);
    if (i0 + i < count) {
      const long long at = slot(i0 + i);
      ml[i] = a.part_ml[at];
#pragma unroll
      for (int c = 0; c < CD; ++c)
        if (4 * (lane + LANES * c) < a.D)
          v[i][c] = *reinterpret_cast<const float4*>(a.part_o + at * a.D + 4 * (lane + LANES * c));
    }
  }
  float top = mx;
#pragma unroll
  for (int i = 0; i < N; ++i) top = fmaxf(top, ml[i].x);
  const float mm = top == -INFINITY ? 0.f : top;
  const float al = exp2f(mx - mm);
  mx = top;
  l *= al;
#pragma unroll
  for (int c = 0; c < CD; ++c) o[c] = make_float4(o[c].x * al, o[c].y * al, o[c].z * al, o[c].w * al);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float w = exp2f(ml[i].x - mm);
    // not a piece that does not exist, saw nothing or vanishes beside the others; what is NaN (m
    // infinite or l NaN, from scores that are no numbers) stays NaN
    if (w != 0.f || ml[i].y != ml[i].y) {
      l = fmaf(w, ml[i].y, l);
#pragma unroll
      for (int c = 0; c < CD; ++c) {
        o[c].x = fmaf(w, v[i][c].x, o[c].x);
        o[c].y = fmaf(w, v[i][c].y, o[c].y);
        o[c].z = fmaf(w, v[i][c].z, o[c].z);
        o[c].w = fmaf(w, v[i][c].w, o[c].w);
      }
    }
  }
}

// Merges the pieces of the row tile that CTA blockIdx.x began and left cut.  LANES lanes take
// a row, two pieces at a time or, of more than four (long contexts, few rows; whole
// warps), eight, four where D > 128: two memory latencies in all, the meta data's and the pieces'.
template <typename T, int LANES, int CD>
__global__ void __launch_bounds__(128) paged_merge_kernel(const __grid_constant__ PagedArgs a) {
  const Meta m = a.meta[blockIdx.x];
  const int lane = threadIdx.x % LANES, row = blockIdx.y * (128 / LANES) + threadIdx.x / LANES;
  if (m.shared == 0 || row >= m.rows) return;
  // piece 0 lies in slot 2c + 1, piece i > 0, which continues the tile in CTA c + i, in slot 2 (c + i)
  auto slot = [&](int i) { return (long long)(i == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + i)) * a.rows + row; };
  float mx = -INFINITY, l = 0.f;
  float4 o[CD];
#pragma unroll
  for (int c = 0; c < CD; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (LANES < 32 || m.shared <= 4)
    for (int i = 0; i < m.shared; i += 2) merge_pieces<2, LANES>(a, i, m.shared, slot, lane, mx, l, o);
  if constexpr (LANES == 32) {
    constexpr int kBatch = CD == 1 ? 8 : 4;
    if (m.shared > 4)
      for (int i = 0; i < m.shared; i += kBatch) merge_pieces<kBatch, LANES>(a, i, m.shared, slot, lane, mx, l, o);
  }
  const int f = m.f0 + row, tok = f / a.G, head = m.head + f % a.G;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* dst = static_cast<T*>(a.out) + ((long long)(m.q0 + tok) * a.Hq + head) * a.D;
#pragma unroll
  for (int c = 0; c < CD; ++c) {
    const int d = 4 * (lane + LANES * c);
    if (d < a.D) {  // D is a multiple of 8: all four columns exist
      if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(dst + d) = make_float4(o[c].x * inv, o[c].y * inv, o[c].z * inv, o[c].w * inv);
      } else {
        const __nv_bfloat162 b0 = __floats2bfloat162_rn(o[c].x * inv, o[c].y * inv);
        const __nv_bfloat162 b1 = __floats2bfloat162_rn(o[c].z * inv, o[c].w * inv);
        uint2 w;
        w.x = *reinterpret_cast<const uint32_t*>(&b0);
        w.y = *reinterpret_cast<const uint32_t*>(&b1);
        *reinterpret_cast<uint2*>(dst + d) = w;
      }
    }
  }
  if (a.lse && lane == 0)
    a.lse[(long long)head * a.total_q + m.q0 + tok] = l == 0.f ? -INFINITY : (mx + log2f(l)) * 0.6931471805599453f;
}

// Eight lanes a row for pairs of tensor-core row tiles (more than 128 rows): with a warp a
// row, most of what it issues is the same in all lanes.  (Requests of 33 to 48 tokens 45.4 us in
// all, 49.8 with whole warps, 45.7 with 16 lanes and 45.6 with 4; 4 chunks of 512 tokens 84
// to 89, 96, 89 and 84 to 90.)
template <typename T>
void run_merge(const PagedArgs& a, int grid, cudaStream_t s) {
  constexpr int kLanes = sizeof(T) == 2 ? 8 : 32;  // only bf16 has such row tiles
  const long long most = (long long)a.max_q * a.G;
  const int rows = most < a.rows ? (int)most : a.rows, per = 128 / kLanes;
  if (a.D > 128) paged_merge_kernel<T, 32, 2><<<dim3(grid, (rows + 3) / 4), 128, 0, s>>>(a);
  else if (rows <= 128) paged_merge_kernel<T, 32, 1><<<dim3(grid, (rows + 3) / 4), 128, 0, s>>>(a);
  else paged_merge_kernel<T, kLanes, 32 / kLanes><<<dim3(grid, (rows + per - 1) / per), 128, 0, s>>>(a);
  count_launch();
}

template <typename T, int BM, int DMAX, bool TREE>
cudaError_t run_simt(const PagedArgs& a, int sms, int most, int* grid, cudaStream_t s) {
  using C = Simt<T, BM, DMAX>;
  const size_t smem = sizeof(typename C::Smem);
  static_assert(sizeof(typename C::Smem) <= 232448, "shared memory budget");
  auto kernel = paged_simt_kernel<T, BM, DMAX, TREE>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  // as many CTAs an SM as fit, so that some copy while others multiply
  int per_sm = (int)(228 * 1024 / (smem + 1024));
  if (per_sm > (BM == 16 ? kSimtPerSm16 : kSimtPerSm64)) per_sm = BM == 16 ? kSimtPerSm16 : kSimtPerSm64;
  *grid = sms * per_sm < most ? sms * per_sm : most;
  kernel<<<*grid, C::kThreads, smem, s>>>(a);
  count_launch();
  return cudaGetLastError();
}

template <typename T, int BM, bool TREE>
cudaError_t pick_simt(const PagedArgs& a, int sms, int most, int* grid, cudaStream_t s) {
  if (a.D <= 64) return run_simt<T, BM, 64, TREE>(a, sms, most, grid, s);
  if (a.D <= 128) return run_simt<T, BM, 128, TREE>(a, sms, most, grid, s);
  return run_simt<T, BM, 256, TREE>(a, sms, most, grid, s);
}
template <bool TREE>
cudaError_t pick_simt(const PagedArgs& a, bool bf16, int sms, int most, int* grid, cudaStream_t s) {
  if (a.rows == 16)
    return bf16 ? pick_simt<__nv_bfloat16, 16, TREE>(a, sms, most, grid, s) : pick_simt<float, 16, TREE>(a, sms, most, grid, s);
  return bf16 ? pick_simt<__nv_bfloat16, 64, TREE>(a, sms, most, grid, s) : pick_simt<float, 64, TREE>(a, sms, most, grid, s);
}

int simt_rows(int G, int max_q) { return (long long)G * max_q <= 16 ? 16 : 64; }

// bf16 runs on the tensor cores wherever their kernel takes the shape, single tokens
// too: 19 us for 8 of them behind 500 to 4096 positions, 33 on the CUDA cores.
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
  p.max_grid = p.tc ? kSms : p.rows == 16 ? kSimtMaxGrid : kSimtPerSm64 * kSms;
  const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  size_t slots = 2 * (size_t)p.max_grid * p.rows;
  // a tensor-core call on a cache without pages runs on the CUDA cores
  if (p.tc && slots < 2 * 2 * (size_t)kSms * 16) slots = 2 * 2 * (size_t)kSms * 16;
  p.ml = up(kSimtMaxGrid * sizeof(Meta));
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
  a.meta = reinterpret_cast<Meta*>(w);
  a.part_ml = reinterpret_cast<float2*>(w + p.ml);
  a.part_o = reinterpret_cast<float*>(w + p.o);
  int grid = sms;
  cudaError_t e;
  // Without a page there is no tensor to describe to TMA: the CUDA-core kernel with
  // its small row tiles.
  if (p.tc && a.num_pages > 0) {
    if (a.parents) a.tiles = (float)a.R * a.Hkv * (((long long)a.max_q * a.G + a.rows - 1) / a.rows);
    e = launch_paged_tc(a, grid, stream);
  } else {
    const int most = p.tc ? 2 * kSms : p.max_grid;
    if (p.tc) a.rows = 16;
    if (a.num_pages == 0) a.kc = a.vc = a.q;  // every copy is one of no bytes, from an address that exists
    e = a.parents ? pick_simt<true>(a, bf16, sms, most, &grid, stream) : pick_simt<false>(a, bf16, sms, most, &grid, stream);
  }
  if (e != cudaSuccess) return e;
  // (As a programmatic dependent launch the merge measured no faster, and 3 us slower with
  // an early trigger: its blocks find no room beside the attention kernel's.)
  if (bf16) run_merge<__nv_bfloat16>(a, grid, stream);
  else run_merge<float>(a, grid, stream);
  return cudaGetLastError();
}

}  // namespace dflash
