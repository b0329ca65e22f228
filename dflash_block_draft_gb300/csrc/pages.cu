// pages.cu -- the pages of a paged cache handed out, shared and taken back on the
// device (sm_103a).  refs[g] counts the table rows that hold page g; a page with 0 is
// free.  No free list: the lowest free pages are taken, in the order in which they are
// asked for, so that the result does not depend on the order in which threads run,
// and giving back what was taken restores the state exactly.
//
// One launch of one cluster of 8 CTAs.  Every CTA adds up all requests' needs for
// itself (a strip a thread and a scan, while the cluster waits for what is given back), reads the
// counts of an eighth of the pages, up to 64 a thread as a bit mask, and learns from one
// exchange through distributed shared memory how many free pages lie before its own.  The free
// pages go into a list in the workspace by their rank; the requests read their run of it.
// Pages beyond 262144 are looked at in further rounds, while pages are still wanted.
//
// Bound by the chain of dependent steps: lengths, table, counts, exchange, list, table, and three
// barriers of the cluster at some 2000 cycles each.  256 requests of up to 8000 positions that
// grow or shrink by up to 64, 30705 pages of 16: 7.3 us (8.4 with a warp a request, the needs
// added up behind the barrier and the counts written before it; a prompt of 125 pages given back
// four times and forked four times 16.4, 25.7 with eight lanes a request whatever their number).
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace dflash {
namespace {

namespace cg = cooperative_groups;

constexpr int kCluster = 8;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kStrip = 64;  // most pages a thread looks at in a round
constexpr int kRowWords = DFLASH_POOL_MAX_ROWS / 32;

// Exclusive sum over the block's threads; *total is the whole sum.
__device__ __forceinline__ int block_scan(int v, int* scratch /* [kWarps] */, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int c = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, c, o);
    if (lane >= o) c += u;
  }
  __syncthreads();  // scratch of an earlier call has been read
  if (lane == 31) scratch[warp] = c;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    before += w < warp ? scratch[w] : 0;
    all += scratch[w];
  }
  *total = all;
  return before + c - v;
}

struct Shared {
  int scan[kWarps];
  int at[kThreads];  // where the pages of a strip's askers begin among all that are wanted
  int free;          // free pages of this CTA in the round
};

// Items (rows of the table, or forks) in strips, of one where there are no more than 512: a strip
// a thread in every CTA to add them up, and a strip a group of the cluster's threads, at least 8
// and as many as there are for it, to work on their pages.
struct Strips {
  int len, items;
  int mine, sub, width;  // this thread's strip as one of a group (below 512), its number in it, the group's size
  __device__ __forceinline__ Strips(int n, int rank) : items(n) {
    len = (n + kThreads - 1) / kThreads;
    const int strips = len ? (n + len - 1) / len : 0;
    width = 8;
    while (2 * width * strips <= kCluster * kThreads && width < kThreads) width *= 2;
    const int t = rank * kThreads + (int)threadIdx.x;
    mine = t / width;
    sub = t % width;
  }
  __device__ __forceinline__ int lo(int strip) const { return min((long long)items, (long long)strip * len); }
  __device__ __forceinline__ int hi(int strip) const { return min((long long)items, (long long)(strip + 1) * len); }
};

// Adds up what the askers want, need(i) pages each, the same in every CTA.  Returns the whole.
template <typename Need>
__device__ __forceinline__ int plan(const Strips& st, Shared& s, Need need) {
  int mine = 0, wanted;
  for (int i = st.lo(threadIdx.x); i < st.hi(threadIdx.x); ++i) mine += need(i);
  s.at[threadIdx.x] = block_scan(mine, s.scan, &wanted);
  __syncthreads();
  return wanted;
}

// Takes pages for the askers in their order: put(i, j, page) is called for the j-th of asker
// i, page -1 where none is left.  Returns the number of pages that were missing.
template <typename Need, typename Put>
__device__ __forceinline__ int take(const PoolArgs& a, const Strips& st, int wanted, Shared& s,
                                    cg::cluster_group& cluster, Need need, Put put) {
  const int rank = (int)cluster.block_rank(), tid = threadIdx.x, lane = tid & 31;
  // the counts, as far as pages are wanted; the free pages by rank go to the workspace
  int found = 0;
  const int per = min(kStrip, ((a.num_pages + kCluster * kThreads - 1) / (kCluster * kThreads) + 3) & ~3);
  for (long long p0 = 0; p0 < a.num_pages && found < wanted; p0 += (long long)per * kThreads * kCluster) {
    const long long b = p0 + ((long long)rank * kThreads + tid) * per;
    unsigned long long mask = 0;
    if (b < a.num_pages) {
      const int end = (int)min((long long)per, a.num_pages - b);
      int j = 0;
      if (a.refs_vec)
        for (; j + 4 <= end; j += 4) {
          const int4 c = __ldcg(reinterpret_cast<const int4*>(a.refs + b + j));
          mask |= (unsigned long long)((c.x == 0) | (c.y == 0) << 1 | (c.z == 0) << 2 | (c.w == 0) << 3) << j;
        }
      for (; j < end; ++j) mask |= (unsigned long long)(__ldcg(a.refs + b + j) == 0) << j;
    }
    int here;
    int k = block_scan(__popcll(mask), s.scan, &here);
    if (tid == 0) s.free = here;
    cluster.sync();
    const int v = lane < kCluster ? *cluster.map_shared_rank(&s.free, lane & (kCluster - 1)) : 0;
    k += found + __reduce_add_sync(0xffffffffu, lane < rank ? v : 0);
    for (; mask && k < wanted; mask &= mask - 1, ++k) a.ws[k] = (int)b + __ffsll((long long)mask) - 1;
    found += __reduce_add_sync(0xffffffffu, v);
    cluster.sync();  // s.free has been read, the list is written
  }
  int at = s.at[st.mine];
  for (int i = st.lo(st.mine); i < st.hi(st.mine); ++i) {
    const int want = need(i);
#pragma unroll 4
    for (int j = st.sub; j < want; j += st.width) {
      const int page = at + j < found ? __ldcg(a.ws + at + j) : -1;
      if (page >= 0) a.refs[page] = 1;
      put(i, j, page);
    }
    at += want;
  }
  return max(0, wanted - found);
}

__device__ __forceinline__ int pages_of(int len, int P) { return (int)(((unsigned)len + P - 1) / (unsigned)P); }

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    resize_kernel(const __grid_constant__ PoolArgs a, const int32_t* __restrict__ old_lens,
                  const int32_t* __restrict__ new_lens) {
  __shared__ Shared s;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const long long most = (long long)a.max_pages * a.P;
  // pages that request r has and is to have; a request with a length out of range keeps its own
  auto load = [&](int r, int& had, int& want) {
    const int x = old_lens[r], y = new_lens[r];
    const bool bad = x < 0 || y < 0 || x > most || y > most;
    had = bad ? 0 : pages_of(x, a.P);
    want = bad ? 0 : pages_of(y, a.P);
    return bad;
  };
  const Strips st(a.R, rank);
  for (int r = st.lo(st.mine); r < st.hi(st.mine); ++r) {
    int had, want;
    if (load(r, had, want) && st.sub == 0) record_error(a.err, DFLASH_ERR_INVALID);
    int32_t* row = a.table + (long long)r * a.max_pages;
    for (int j = want + st.sub; j < had; j += st.width) {
      const int page = row[j];
      row[j] = -1;
      if (page == -1) continue;  // none was left when the request grew
      if (page < 0 || page >= a.num_pages) {
        record_error(a.err, DFLASH_ERR_INVALID);
      } else if (atomicSub(a.refs + page, 1) <= 0) {  // it was free: the count stays at 0
        atomicAdd(a.refs + page, 1);
        record_error(a.err, DFLASH_ERR_INVALID);
      }
    }
  }
  auto need = [&](int r) {
    int had, want;
    load(r, had, want);
    return max(0, want - had);
  };
  // the counts after everything that was given back; what is wanted meanwhile (whole warps come to both halves)
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  const int wanted = plan(st, s, need);
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  const int missing = take(a, st, wanted, s, cluster, need, [&](int r, int j, int page) {
    a.table[(long long)r * a.max_pages + pages_of(old_lens[r], a.P) + j] = page;
  });
  if (rank == 0 && threadIdx.x == 0) a.missing[0] = missing;
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    fork_kernel(const __grid_constant__ PoolArgs a, const __grid_constant__ ForkArgs f) {
  __shared__ Shared s;
  __shared__ unsigned s_dst[kRowWords], s_twice[kRowWords], s_src[kRowWords];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), tid = threadIdx.x, lane = tid & 31;
  const long long most = (long long)a.max_pages * a.P;
  // rows that are a fork's, two forks' or a source; every CTA finds them for itself
  for (int i = tid; i < (a.R + 31) / 32; i += kThreads) s_dst[i] = s_twice[i] = s_src[i] = 0;
  __syncthreads();
  for (int i = tid; i < f.n; i += kThreads) {
    const int x = f.src[i], y = f.dst[i];
    if (x >= 0 && x < a.R) atomicOr(&s_src[x >> 5], 1u << (x & 31));
    if (y >= 0 && y < a.R && (atomicOr(&s_dst[y >> 5], 1u << (y & 31)) >> (y & 31) & 1u))
      atomicOr(&s_twice[y >> 5], 1u << (y & 31));
  }
  __syncthreads();
  auto bit = [](const unsigned* m, int i) { return (m[i >> 5] >> (i & 31)) & 1u; };
  // positions of fork i's source, -1 where the fork is refused (lens[dst] is looked at apart)
  auto length = [&](int i) {
    const int x = f.src[i], y = f.dst[i];
    if (x < 0 || x >= a.R || y < 0 || y >= a.R || bit(s_twice, y) || bit(s_src, y)) return -1;
    const int n = __ldcg(f.lens + x);
    return n < 0 || n > most ? -1 : n;
  };
  // (No fork's row is a source or another fork's: what one fork reads no other one writes.)
  for (int i = rank * kWarps + (tid >> 5); i < f.n; i += kCluster * kWarps) {
    const int n = length(i);
    const bool ok = n >= 0 && __ldcg(f.lens + f.dst[i]) == 0;
    __syncwarp();  // read by all lanes before one of them writes it
    const int full = ok ? n / a.P : 0, rest = ok ? n % a.P : 0;
    const int32_t* from = a.table + (long long)(ok ? f.src[i] : 0) * a.max_pages;
    int32_t* to = a.table + (long long)(ok ? f.dst[i] : 0) * a.max_pages;
    for (int j = lane; j < full; j += 32) {
      const int page = from[j];
      to[j] = page;
      if (page >= 0 && page < a.num_pages) atomicAdd(a.refs + page, 1);
      else record_error(a.err, DFLASH_ERR_INVALID);
    }
    if (lane == 0) {
      if (ok) f.lens[f.dst[i]] = n;
      else record_error(a.err, DFLASH_ERR_INVALID);
      f.copy_rows[i] = rest;
      const int last = rest ? from[full] : -1;
      if (rest && (last < 0 || last >= a.num_pages)) record_error(a.err, DFLASH_ERR_INVALID);
      f.copy_src[i] = last;
      f.copy_dst[i] = -1;
    }
  }
  cluster.sync();
  auto need = [&](int i) { return __ldcg(f.copy_rows + i) > 0 ? 1 : 0; };
  const Strips st(f.n, rank);
  const int missing = take(a, st, plan(st, s, need), s, cluster, need, [&](int i, int, int page) {
    a.table[(long long)f.dst[i] * a.max_pages + length(i) / a.P] = page;
    f.copy_dst[i] = page;
  });
  if (rank == 0 && tid == 0) a.missing[0] = missing;
}

}  // namespace

size_t pool_workspace_bytes(int num_pages) { return sizeof(int32_t) * (size_t)num_pages; }

cudaError_t launch_pages_resize(const PoolArgs& a, const int32_t* old_lens, const int32_t* new_lens,
                                cudaStream_t stream) {
  resize_kernel<<<kCluster, kThreads, 0, stream>>>(a, old_lens, new_lens);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_pages_fork(const PoolArgs& a, const ForkArgs& f, cudaStream_t stream) {
  fork_kernel<<<kCluster, kThreads, 0, stream>>>(a, f);
  count_launch();
  return cudaGetLastError();
}

}  // namespace dflash
