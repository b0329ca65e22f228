// cache_move.cu -- rows and pages of a paged cache moved within it (sm_103a): the
// accepted nodes of a tree moved together (compact), and pages copied (copy), in the
// keys and values of all layers at once.
//
// Both read and write what they move once, and are bound by memory where that is
// much and by the chain of dependent reads (lengths, path, page table, rows) where it
// is little, which is the rule: a tree's accepted nodes are a few rows of a few KB.  Walk and
// compaction together: 5.8 us on the device for one request and four layers, 8.8 for 128 requests
// and eight layers (12 MB moved, 1.7 us of it memory).  64 copied last pages of up to 32
// positions of 4 KB, eight layers, keys and values: 141 MB, 18 us with cold caches.
#include "common.cuh"
#include "internal.h"

namespace dflash {
namespace {

constexpr int kThreads = 128;
constexpr int kBatch = 8;          // rows a thread has in flight
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;       // 16-byte vectors a thread copies

// One CTA: one request, one layer, keys or values.  A thread takes a 16-byte column of
// the rows and moves its rows in the path's order, kBatch at a time, loads before
// stores.  The path ascends, so path[j] >= j, and a row that is written (j) is not read
// any more: later rows are read from behind it, and those of its batch have been read.
__global__ void __launch_bounds__(kThreads) compact_kernel(const __grid_constant__ CompactArgs a) {
  __shared__ long long s_from[kThreads], s_to[kThreads];
  const int r = blockIdx.x, tid = threadIdx.x;
  const bool values = blockIdx.y & 1;
  const int layer = blockIdx.y >> 1;
  const int q0 = a.q_off[r], q1 = a.q_off[r + 1], kv = a.kv_lens[r], count = a.count[r];
  const int32_t* path = a.path + (long long)r * a.max_path;
  const int n = q1 - q0, base = kv - n;
  bool bad = q0 < 0 || q1 < q0 || q1 > a.total_q || kv < n || kv > (long long)a.max_pages * a.P || count < 0 ||
             count > n || count > a.max_path;
  const int nodes = bad ? 0 : count;
  for (int j = tid; j < nodes; j += kThreads) bad |= path[j] < j || path[j] >= n || (j > 0 && path[j - 1] >= path[j]);
  bad = __syncthreads_or(bad);
  if (blockIdx.y == 0 && tid == 0) {
    if (bad) record_error(a.err, DFLASH_ERR_INVALID);
    a.new_lens[r] = bad ? kv : base + count;
  }
  if (bad) return;
  const long long page_stride = values ? a.vps : a.kps;  // 16-byte vectors
  uint4* cache = static_cast<uint4*>(values ? a.vc : a.kc) + layer * (values ? a.vls : a.kls);
  // first vector of a position's row, -1 where it has no page
  auto row_of = [&](int p) -> long long {
    const int page = a.table[(long long)r * a.max_pages + p / a.P];
    if (page < 0 || page >= a.num_pages) {
      record_error(a.err, DFLASH_ERR_INVALID);
      return -1;
    }
    return page * page_stride + (long long)(p % a.P) * a.row;
  };
  for (int j0 = 0; j0 < count; j0 += kThreads) {
    if (j0 > 0) __syncthreads();  // the rows before have been moved
    const int j = j0 + tid;
    if (j < count) {
      const int k = path[j];
      const bool moves = k != j;
      s_from[tid] = moves ? row_of(base + k) : -1;
      s_to[tid] = moves ? row_of(base + j) : -1;
    }
    __syncthreads();
    const int rows = min(kThreads, count - j0);
    for (int c = tid; c < a.row; c += kThreads)
      for (int i0 = 0; i0 < rows; i0 += kBatch) {
        uint4 x[kBatch];
        bool live[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          live[i] = i0 + i < rows && s_from[i0 + i] >= 0 && s_to[i0 + i] >= 0;
          if (live[i]) x[i] = cache[s_from[i0 + i] + c];
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (live[i]) cache[s_to[i0 + i] + c] = x[i];
      }
  }
}

// One CTA: a run of kCopyThreads * kCopyVecs vectors of one copy, one layer, keys or values.
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyArgs a) {
  const int i = blockIdx.x;
  const bool values = blockIdx.y & 1;
  const int layer = blockIdx.y >> 1;
  const int src = a.src[i], dst = a.dst[i], rows = a.rows ? a.rows[i] : a.P;
  const bool none = src == -1 || dst == -1;
  if (!none && (src < 0 || src >= a.num_pages || dst < 0 || dst >= a.num_pages || rows < 0 || rows > a.P)) {
    if (threadIdx.x == 0) record_error(a.err, DFLASH_ERR_INVALID);
    return;
  }
  if (none || src == dst) return;
  const long long page_stride = values ? a.vps : a.kps;
  uint4* cache = static_cast<uint4*>(values ? a.vc : a.kc) + layer * (values ? a.vls : a.kls);
  const uint4* from = cache + src * page_stride;
  uint4* to = cache + dst * page_stride;
  const long long vecs = (long long)rows * a.row;
  for (long long c0 = (long long)blockIdx.z * (kCopyThreads * kCopyVecs) + threadIdx.x; c0 < vecs;
       c0 += (long long)gridDim.z * (kCopyThreads * kCopyVecs)) {
    uint4 x[kCopyVecs];
#pragma unroll
    for (int k = 0; k < kCopyVecs; ++k)
      if (c0 + k * kCopyThreads < vecs) x[k] = from[c0 + k * kCopyThreads];
#pragma unroll
    for (int k = 0; k < kCopyVecs; ++k)
      if (c0 + k * kCopyThreads < vecs) to[c0 + k * kCopyThreads] = x[k];
  }
}

}  // namespace

cudaError_t launch_cache_compact(const CompactArgs& a, cudaStream_t stream) {
  compact_kernel<<<dim3(a.R, 2 * a.layers), kThreads, 0, stream>>>(a);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_cache_copy(const CopyArgs& a, cudaStream_t stream) {
  const long long pieces = ((long long)a.P * a.row + kCopyThreads * kCopyVecs - 1) / (kCopyThreads * kCopyVecs);
  copy_kernel<<<dim3(a.n, 2 * a.layers, (unsigned)(pieces < 65535 ? pieces : 65535)), kCopyThreads, 0, stream>>>(a);
  count_launch();
  return cudaGetLastError();
}

}  // namespace dflash
