// paged.cuh -- how the paged-attention kernels deal their work out (sm_103a).
//
// A row tile is `rows` consecutive rows (token, head of the group; token-major) of
// one request and one key/value head; it needs the key tiles up to its last
// token's limit.  Its length is its key tiles plus kSetup for what it costs besides
// (queries in, results out: 3.3 us measured, 2.3 key tiles' worth; without them a
// CTA with 15 row tiles of a ragged batch took 455 us, one with two 407).  All row
// tiles, in the order request, key/value head, row tile, form one line of length T,
// and every CTA takes the next T / G of it, the first T mod G one more (G CTAs, at
// most T; further ones have none): equal work whatever the lengths, one long
// request or many short ones, without a host that knows the lengths.  A row tile's
// set-up lies before its first key tile; a CTA whose part of it ends there has none
// of it.  A row tile whose key tiles one CTA holds is finished by it; of one that is
// cut, every CTA leaves a partial result (running maximum, sum, unnormalised
// output) in the workspace: slot 2c for the piece that continues a row tile begun
// by an earlier CTA, slot 2c + 1 for the piece that begins one and is cut by the
// range's end.  The CTA that begins a cut row tile writes down in meta[c] how many
// CTAs share it, and the merge kernel adds the pieces up in that order.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace dflash {
namespace paged {

constexpr int kSetup = 2;

// One request as the kernels see it.
struct Req {
  int q0, n, kv;  // first packed row, new tokens, positions
  int nrt;        // row tiles of one key/value head (0: nothing to do)
};

__device__ __forceinline__ Req load_request(const PagedArgs& a, int r, bool report) {
  Req q;
  q.q0 = a.q_off[r];
  const int q1 = a.q_off[r + 1];
  q.n = q1 - q.q0;
  q.kv = a.kv_lens[r];
  // (q1 < q0 by itself: of offsets far apart the difference wraps)
  const bool bad = q.q0 < 0 || q1 < q.q0 || q1 > a.total_q || q.n > a.max_q || q.kv < 0 ||
                   q.kv > (long long)a.max_pages * a.P;
  if (bad && report) record_error(a.err, DFLASH_ERR_INVALID);
  // rows of a request fit 31 bits (the host bounds max_q * G)
  q.nrt = bad ? 0 : (unsigned)(q.n * a.G + a.rows - 1) / (unsigned)a.rows;
  return q;
}

// Positions that the last token of row tile rt sees; every row tile has one key
// tile at least, so that rows that see nothing are written too.
__device__ __forceinline__ int tile_limit(const PagedArgs& a, const Req& q, int rt) {
  if (!a.causal) return q.kv;
  const unsigned end = min((rt + 1) * a.rows, q.n * a.G);
  return max(0, q.kv - q.n + (int)((end - 1) / (unsigned)a.G) + 1);
}
template <int BN>
__device__ __forceinline__ int key_tiles(const PagedArgs& a, const Req& q, int rt) {
  return max(1, (tile_limit(a, q, rt) + BN - 1) / BN);
}
// Length of the first m row tiles of one key/value head, m <= nrt.  In closed form
// where the tokens of a row tile divide BN or BN divides them: with k = BN / tokens
// a row tile ends one k-th of a key tile after the one before.
template <int BN>
__device__ __forceinline__ long long length_of(const PagedArgs& a, const Req& q, int m) {
  if (m == 0) return 0;
  if (!a.causal) return (long long)m * (kSetup + key_tiles<BN>(a, q, 0));
  const unsigned tokens = (unsigned)a.rows / (unsigned)a.G;
  const int base = q.kv - q.n;
  long long s = 0;
  int full = min(m, q.nrt - 1);  // the last row tile may hold fewer tokens
  if (base >= 0 && tokens * a.G == a.rows && BN % tokens == 0) {
    const unsigned k = BN / tokens, first = (base + tokens - 1) / tokens;
    auto sum = [&](unsigned x) {  // of ceil(j / k), j = 1 .. x
      const unsigned c = x / k;
      return (long long)k * c * (c + 1) / 2 + (long long)(x - c * k) * (c + 1);
    };
    s = sum(first + full) - sum(first);
  } else if (base >= 0 && tokens * a.G == a.rows && tokens % BN == 0) {
    s = full * (long long)((base + BN - 1) / BN) + (long long)(tokens / BN) * full * (full + 1) / 2;
  } else {
    for (int rt = 0; rt < full; ++rt) s += key_tiles<BN>(a, q, rt);
  }
  s += (long long)kSetup * m;
  return m > full ? s + key_tiles<BN>(a, q, full) : s;
}

// a / b for a >= 0, b > 0, in 32 bits where both fit (64-bit divisions are long).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return (unsigned long long)(a | b) >> 32 ? a / b : (long long)((unsigned)a / (unsigned)b);
}

// A CTA's share of one row tile: key tiles [kt0, kt1) of nt.
struct Piece {
  int r, h, rt;
  Req q;
  int kt0, kt1, nt;
  int slot;            // partial slot, -1: the row tile is whole
  long long end;       // where the row tile ends
};

// A CTA's range, found once by a block's threads and kept in shared memory: its part
// of the line and its first piece.
struct Range {
  long long t1;       // end of its part
  long long share;    // T / G
  int more;           // T mod G: CTAs with one more
  int any;            // whether there is a piece
  long long t;        // place behind the first piece
  Piece first;
};

// Walks the pieces of a CTA's range.  Every role of a kernel keeps its own; the
// first piece is worked out once (the code is cold then, and it cost a microsecond).
template <int BN>
struct Walker {
  const PagedArgs& a;
  long long t, t1;  // next place, end
  long long at;     // where the current row tile begins
  Req q;
  int r, h, rt;
  int state;        // 0: the current row tile is next, 1: it is done with, 2: the first piece lies in `first`
  const Piece* first;

  __device__ __forceinline__ Walker(const PagedArgs& a_, const Range& rg) : a(a_) {
    t = rg.t;
    t1 = rg.t1;
    state = rg.any ? 2 : 0;
    if (!rg.any) t = t1;
    first = &rg.first;
  }
  __device__ __forceinline__ Walker(const PagedArgs& a_, long long t_, long long t1_, long long at_, const Req& q_, int r_,
                                    int h_, int rt_)
      : a(a_), t(t_), t1(t1_), at(at_), q(q_), r(r_), h(h_), rt(rt_), state(0), first(nullptr) {}

  __device__ __forceinline__ bool next(Piece* p) {
    if (state == 2) {
      *p = *first;
      r = p->r;
      h = p->h;
      rt = p->rt;
      q = p->q;
      at = p->end;
      state = 1;
      return true;
    }
    while (t < t1) {
      if (state == 1) {  // the next row tile, head or request with work
        if (++rt == q.nrt) {
          rt = 0;
          if (++h == a.Hkv) {
            h = 0;
            do q = load_request(a, ++r, false);
            while (q.nrt == 0 && r + 1 < a.R);
          }
        }
      }
      p->r = r;
      p->h = h;
      p->rt = rt;
      p->q = q;
      p->nt = key_tiles<BN>(a, q, rt);
      p->end = at + kSetup + p->nt;
      const long long end = min(p->end, t1);
      p->kt0 = max(0, (int)(t - at) - kSetup);
      p->kt1 = max(0, (int)(end - at) - kSetup);
      const int me = blockIdx.x;
      p->slot = p->kt0 > 0 ? 2 * me : p->kt1 < p->nt ? 2 * me + 1 : -1;
      t = end;
      at = p->end;
      state = 1;
      if (p->kt1 > p->kt0) return true;  // else the range ends in the row tile's set-up
    }
    return false;
  }
};

// kThreads threads, numbered tid: every thread adds up a strip of requests, a scan over
// the strips gives T and finds the strip, and its thread the first piece, of the CTA's
// part.  sync() is a barrier among them; the result is there after one more.
template <int BN, int kThreads, typename Sync>
__device__ __forceinline__ void find_range(const PagedArgs& a, int tid, Range* out,
                                           long long* scratch /* [kThreads/32] */, Sync sync) {
  const int lane = tid & 31, warp = tid >> 5;
  const int strip = (a.R + kThreads - 1) / kThreads;
  const int lo = min(a.R, tid * strip), hi = min(a.R, lo + strip);
  long long mine = 0, per = 0;
  Req q;
  for (int r = lo; r < hi; ++r) {
    q = load_request(a, r, blockIdx.x == 0);
    per = length_of<BN>(a, q, q.nrt);  // of one head
    mine += a.Hkv * per;
  }
  long long c = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, c, o);
    if (lane >= o) c += v;
  }
  if (lane == 31) scratch[warp] = c;
  if (tid == 0) out->any = 0;
  sync();
  long long base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    base += w < warp ? scratch[w] : 0;
    total += scratch[w];
  }
  const long long before = base + c - mine;
  const int ctas = (int)min((long long)gridDim.x, total), me = blockIdx.x;
  const long long share = ctas > 0 ? quotient(total, ctas) : 0;
  const int more = (int)(total - share * ctas);
  const long long t0 = me < ctas ? share * me + min(me, more) : total;
  const long long t1 = me < ctas ? t0 + share + (me < more) : total;
  if (tid == 0) {
    out->t1 = t1;
    out->share = share;
    out->more = more;
  }
  if (before <= t0 && t0 < before + mine) {  // one thread at most
    long long s = before;
    int r = hi - 1;
    if (hi - lo > 1) {
      for (r = lo; r < hi; ++r) {
        q = load_request(a, r, false);
        per = length_of<BN>(a, q, q.nrt);
        if (t0 < s + a.Hkv * per) break;
        s += a.Hkv * per;
      }
    }
    const int h = (int)quotient(t0 - s, per);
    s += h * per;
    // the last row tile that begins at or before t0
    const long long want = t0 - s;
    int x = 0, n = q.nrt;
    while (n > 1) {
      const int half = n >> 1;
      if (length_of<BN>(a, q, x + half) <= want) {
        x += half;
        n -= half;
      } else {
        n = half;
      }
    }
    Walker<BN> walk(a, t0, t1, s + length_of<BN>(a, q, x), q, r, h, x);
    Piece pc;
    if (walk.next(&pc)) {
      out->first = pc;
      out->t = walk.t;
      out->any = 1;
    }
  }
}

// CTA that holds place t of the line.
__device__ __forceinline__ int owner_of(long long t, const Range& rg) {
  const long long wide = (rg.share + 1) * rg.more;  // parts of the CTAs with one more
  return (int)(t < wide ? quotient(t, rg.share + 1) : rg.more + quotient(t - wide, rg.share));
}

// What the merge kernel needs about CTA c: the row tile that it begins and leaves cut.
struct Meta {
  int shared;     // CTAs that share it (0: none is cut)
  int q0;         // its request's first packed row
  int head;       // its group's first query head
  int f0, rows;   // its first row within (request, key/value head), and rows
};
__device__ __forceinline__ Meta no_meta() { return Meta{0, 0, 0, 0, 0}; }
// Whether this piece begins a row tile that is cut.
__device__ __forceinline__ bool begins_cut(const Piece& p) { return p.slot >= 0 && (p.slot & 1); }
__device__ __forceinline__ Meta meta_of(const PagedArgs& a, const Range& rg, const Piece& p) {
  const int f0 = p.rt * a.rows;
  return Meta{owner_of(p.end - 1, rg) - (int)blockIdx.x + 1, p.q.q0, p.h * a.G, f0, min(a.rows, p.q.n * a.G - f0)};
}

// The tensor-core kernel (attn_paged_tc.cu): which shapes it takes, the rows of its
// row tiles, and its launch over `grid` CTAs.
bool paged_tc_supported(int G, int D, int P);
int paged_tc_rows(int G, int max_q);
cudaError_t launch_paged_tc(const PagedArgs& a, int grid, cudaStream_t stream);

}  // namespace paged
}  // namespace dflash
