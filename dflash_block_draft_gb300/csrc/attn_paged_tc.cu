// attn_paged_tc.cu -- tensor-core (tcgen05 + TMEM + TMA) attention of new tokens
// over a paged key/value cache, bf16 (sm_103a).
//
// A row tile is up to 128 rows (token, head of the group; token-major: row =
// token * G + head) of one request and one key/value head, so that all G query
// heads of a group read each key and value once.  Per 128-position key tile
//   S = Q K^T   tcgen05 SS MMA, fp32 in TMEM
//   P = 2^(S scale log2 e - m), bf16, written over S   softmax warpgroup, a row a thread
//   O += P V    tcgen05 TS MMA
// with a running reference m that moves only when a maximum exceeds it by 2^8.
//
// Two forms of one kernel, both with two score tiles and two output accumulators
// in TMEM (2 x 128 + 2 x D columns) and two softmax warpgroups ("halves"), so that
// one half's MMAs run during the other half's softmax:
//   PAIR   the halves are two adjacent row tiles and share every key tile: prefill
//          chunks, bound by the tensor cores and the softmax between them;
//   SPLIT  the halves are the even and the odd key tiles of one row tile, and
//          are added up at the end of a piece: single tokens and draft blocks,
//          bound by memory, where a second row tile would be padding.  Row tiles of
//          up to 64 rows have two query buffers, so that the next one's queries are
//          there in time.
//
// The form is the launch's, from the bound on the requests' tokens: beside a chunk, or
// under a bound that is too loose, single tokens run as pairs whose second half is padding.
// 63 single tokens behind 1000 to 8000 positions take 186 us, 233 with a bound of 2048; in one
// call with 2048 tokens behind 8192 456 us, the two calls by themselves 186 and 238.
//
// Pages: a 128-position tile arrives as 128 / b boxes of b = gcd(page_size, 128)
// positions, one TMA load for each box and 64 components, lane by lane; a tile may
// so begin and end anywhere in a page.  Boxes of 8 positions of 128 components bring
// both halves of the components at once (their 1 KB blocks then lie next to each
// other): 64 loads a tile took 733 us where 32 take 478.  Positions behind the
// request's length are masked in S; of V their rows are set to zero in shared memory
// before P V reads them, since what an unfinished page holds there may be NaN.  A
// page that does not exist is loaded from behind the tensor's end, which TMA fills
// with zeros.
// Head dimensions below 64 or 128 are padded with zeros the same way.
//
// Warp roles (384 threads): warp 0 loads keys and values, warp 3 the queries (so that
// the next row tile's keys do not wait for the queries' buffer), warps 1 and 2 issue
// the MMAs of halves 0 and 1, warps 4..7 and 8..11 are the softmax and epilogue of
// halves 0 and 1.
// The grid is one CTA an SM; work is dealt as paged.cuh says.  Every mbarrier
// wait is bounded (DFLASH_ERR_TIMEOUT, CTA abort flag, wind-down).
//
// TREE: of the new tokens a row sees itself and its ancestors alone.  Tiles in front of the
// tree are unmasked, and of a tile with new tokens a row's thread follows its chain of
// parents into 128 bits while S is being computed; one test a tile decides whether bits are
// applied.  (Trees of 40 to 64 nodes of 32 requests behind 1024 to 32768 positions 257 us, the
// causal form 249; 272 with a second test of the causal limit in every tile.)
//
// Roundings: S, the softmax's statistics and O are fp32; P is rounded to bf16, the type
// that the MMA takes beside V, while its sum l is taken before that rounding; the
// results are rounded once.  (Against 64 bits the results' error is 2.2e-3 to 2.4e-3 of their
// size; rounding them alone makes 1.7e-3 of it.  With l from the rounded P it is 1.9e-3 where
// few keys matter and no less elsewhere, and a chunk takes 946 us.)
//
// Measured with 32 query heads in 8 groups, D = 128 (a block of 16 tokens, 64 requests
// of 1 to 33 thousand positions: 2.9 GB of keys and values): 432 to 443 us, 6.5 to
// 6.7 TB/s, as fast as a copy.  A chunk of 2048 tokens behind 32768: 800 to 825 us,
// 1.37 to 1.42 PFLOP/s; a key tile of a pair costs 3280 cycles, of which the MMAs of
// both halves take 2110 and one half's chain QK, softmax, PV the rest (P lies over S,
// so QK of the next tile waits for PV).  Scores issued 64 keys at a time into
// what P leaves free shorten that to 2950, but N = 64 MMAs then fill the tensor pipe
// and the clock falls with the power: 804 us, and 4 chunks of 512 tokens took
// 101 us against 90.
#include <math.h>

#include <atomic>

#include "paged.cuh"
#include "ptx.cuh"
#include "tc_common.cuh"

namespace dflash {
namespace paged {
namespace {

using tc::Ctl;
using tc::kWaitBudgetNs;
using tc::max64;
using tc::range_bits;

constexpr int kBM = 128, kBN = 128;
constexpr uint32_t kPanel = kBM * 128;  // 128 rows x 128 bytes (64 bf16)
constexpr int kThreads = 384;
constexpr int kLaunchRegs = 168;  // 65536 / 384, rounded down to a multiple of 8
constexpr uint32_t kCtlRegs = 120, kSoftmaxRegs = 192;
static_assert(128 * kCtlRegs + 256 * kSoftmaxRegs == kThreads * kLaunchRegs, "register split");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;  // S_i at kColS + 128 i, O_i at kColO + 128 i

// NP: 64-component panels of a head (1: D <= 64, 2: D <= 128).
template <int NP, bool PAIR>
struct Cfg {
  static constexpr uint32_t kSlot = NP * kPanel;  // a ring slot holds one K or V tile
  static constexpr uint32_t kQBytes = (PAIR ? 2 : 1) * NP * kPanel;
  // As many slots as fit the 227 KB: 5 or 6 of 32 KB, 12 of 16 KB.  SPLIT: one ring
  // for each half.  (A slot's uses have to belong to one consumer: a wait for a
  // phase while the phase before it is still open passes at once, and that phase is
  // known to be closed only by who waited for it.)
  static constexpr uint32_t kRings = PAIR ? 1 : 2;
  static constexpr uint32_t kRing = (14 * kPanel - kQBytes) / kSlot / kRings;
  static constexpr uint32_t kSlots = kRings * kRing;
  // Slot and phase parity of load c of ring r (tile m of the ring: K is load 2 m, V is 2 m + 1).
  static __device__ __forceinline__ uint32_t slot(uint32_t r, uint32_t c) { return r * kRing + c % kRing; }
  static __device__ __forceinline__ uint32_t parity(uint32_t c) { return (c / kRing) & 1u; }
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffRing = kQBytes;
  static constexpr uint32_t kOffBar = kOffRing + kSlots * kSlot;
  enum : int {
    Q_FULL = 0,   // 2 (one buffer each)
    Q_EMPTY = 2,  // 2
    RING_FULL = 4,
    RING_EMPTY = RING_FULL + (int)kSlots,
    S_FULL = RING_EMPTY + (int)kSlots,
    P_LO = S_FULL + 2,     // P of keys 0-63 written
    P_HI = P_LO + 2,       // P of keys 64-127 written
    PV_LO = P_HI + 2,      // PV of keys 0-63 completed
    QK_TURN = PV_LO + 2,   // PAIR: QK_i issued
    O_FULL = QK_TURN + 2,
    ML = O_FULL + 2,       // SPLIT: both halves' maxima and sums written
    EPI = ML + 1,          // SPLIT: both halves' accumulators read
    DRAIN = EPI + 1,
    kBars = DRAIN + 1
  };
  static constexpr uint32_t kOffTmem = kOffBar + 8 * kBars;
  static constexpr uint32_t kOffAbort = kOffTmem + 4;
  static constexpr uint32_t kOffRange = (kOffAbort + 4 + 7) / 8 * 8;
  static constexpr uint32_t kOffScratch = kOffRange + (sizeof(Range) + 7) / 8 * 8;
  static constexpr uint32_t kOffMl = kOffScratch + 8 * 8;
  static constexpr uint32_t kSmem = kOffMl + (PAIR ? 0 : 2 * kBM * 8);
  static_assert(kSmem <= 232448, "shared memory budget");
};

struct TcPagedArgs {
  PagedArgs a;
  int tokens;  // tokens of a tile of up to 128 rows: 128 / G, or all that a request can have
  int box;     // positions of a TMA box
  int dual;    // boxes hold both panels
  uint32_t panel, group;  // bytes from panel to panel and from 8 rows to the next 8 of a K or V tile
  int q_bufs;  // 2: row tiles of up to 64 rows, the second buffer in the first one's rows 64 ..
  int out_v8;  // output rows may be written in 32-byte pieces
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1),
      "r"(c2), "r"(c3)
      : "memory");
}

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2,
                                            int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1),
      "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}

// Hides the columns c0 + i (i < 64) at and beyond `lim` of the tile.
__device__ __forceinline__ void hide64(float* x, int c0, int lim) {
  if (lim >= c0 + 64) return;
  const uint64_t vis = range_bits(0, lim - c0);
  const uint32_t lo = (uint32_t)vis, hi = (uint32_t)(vis >> 32);
#pragma unroll
  for (int c = 0; c < 32; ++c) {
    x[c] = (lo >> c) & 1u ? x[c] : -INFINITY;
    x[32 + c] = (hi >> c) & 1u ? x[32 + c] : -INFINITY;
  }
}

// Hides the columns (64 from c0 on) whose bit of `vis` is not set.
__device__ __forceinline__ void hide_bits(float* x, uint64_t vis) {
  const uint32_t lo = (uint32_t)vis, hi = (uint32_t)(vis >> 32);
#pragma unroll
  for (int c = 0; c < 32; ++c) {
    x[c] = (lo >> c) & 1u ? x[c] : -INFINITY;
    x[32 + c] = (hi >> c) & 1u ? x[32 + c] : -INFINITY;
  }
}

template <int NP, bool PAIR, bool TREE>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tc_kernel(const __grid_constant__ TcPagedArgs ta, const __grid_constant__ CUtensorMap tmQ,
                    const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
  using C = Cfg<NP, PAIR>;
  constexpr int DP = 64 * NP;  // padded head dimension
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = ptx::smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedArgs& a = ta.a;
  if (sbase & 1023u) {  // the swizzled tiles need it; dynamic shared memory starts there
    if (threadIdx.x == 0) {
      a.meta[blockIdx.x] = no_meta();
      record_error(a.err, DFLASH_ERR_CUDA);
    }
    return;
  }
  Ctl ctl;
  ctl.bar0 = sbase + C::kOffBar;
  ctl.abort = reinterpret_cast<volatile int*>(smem + C::kOffAbort);
  ctl.err = a.err;
  ctl.budget = a.wait_ns;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffTmem);
  Range& range = *reinterpret_cast<Range*>(smem + C::kOffRange);
  float2* ml = reinterpret_cast<float2*>(smem + C::kOffMl);

  if (threadIdx.x == 0) {
    const uint32_t users = PAIR ? 2 : 1;  // MMA issuers that read a ring slot
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(ctl.bar(C::Q_FULL + b), 1);
      ptx::mbar_init(ctl.bar(C::Q_EMPTY + b), 2);
    }
    for (uint32_t s = 0; s < C::kSlots; ++s) {
      ptx::mbar_init(ctl.bar(C::RING_FULL + s), 1);
      ptx::mbar_init(ctl.bar(C::RING_EMPTY + s), users);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(ctl.bar(C::S_FULL + i), 1);
      ptx::mbar_init(ctl.bar(C::P_LO + i), 128);
      ptx::mbar_init(ctl.bar(C::P_HI + i), 128);
      ptx::mbar_init(ctl.bar(C::PV_LO + i), 1);
      ptx::mbar_init(ctl.bar(C::QK_TURN + i), 1);
      ptx::mbar_init(ctl.bar(C::O_FULL + i), 1);
    }
    ptx::mbar_init(ctl.bar(C::ML), 256);
    ptx::mbar_init(ctl.bar(C::EPI), 256);
    ptx::mbar_init(ctl.bar(C::DRAIN), 2);
    *ctl.abort = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  if (warp == 3 && lane == 0) {
    ptx::prefetch_tmap(&tmQ);
    ptx::prefetch_tmap(&tmK);
    ptx::prefetch_tmap(&tmV);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), kTmemCols);
    ptx::tmem_relinquish();
  }
  // the softmax warps look at the requests, while the others set the barriers and TMEM up
  if (warp >= 4)
    find_range<kBN, 256>(a, threadIdx.x - 128, &range, reinterpret_cast<long long*>(smem + C::kOffScratch),
                         [] { ptx::named_barrier(1, 256); });
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t ring = sbase + C::kOffRing;
  const int tile_rows = ta.tokens * a.G;  // rows of one half's tile
  // Buffer and phase parity of the n-th row tile's queries.
  const uint32_t q_two = ta.q_bufs == 2;
  auto q_buf = [&](uint32_t n) { return n & q_two; };
  auto q_parity = [&](uint32_t n) { return (n >> q_two) & 1u; };
  if (warp < 4) ptx::setmaxnreg_dec<kCtlRegs>();

  if (warp == 0) {
    // ------------------------------------------------------------ keys and values (whole warp)
    Walker<kBN> walk(a, range);
    Piece pc = {};
    uint32_t g = 0;                 // key tiles loaded
    uint32_t load0 = 0, load1 = 0;  // of each ring
    bool stop = false;
    const int boxes = kBN / ta.box;                     // boxes of a panel
    const int my_box = lane % boxes, my_pn = lane / boxes;  // this lane's box
    const bool mine = lane < (ta.dual ? boxes : boxes * NP);
    const uint32_t my_dst = ta.dual ? lane * 2048u : my_pn * kPanel + my_box * ta.box * 128u;
    // Page id of this lane's box of key tile kt; the load is left in flight.
    auto page_of = [&](int kt) {
      const int p0 = kt * kBN + my_box * ta.box;
      return mine && kt < pc.kt1 && p0 < pc.q.kv ? __ldg(a.table + (long long)pc.r * a.max_pages + p0 / a.P)
                                                : a.num_pages;
    };
    while (!stop && walk.next(&pc)) {
      int page_next = page_of(pc.kt0);
      if ((int)blockIdx.x == a.stall_cta) break;  // timeout test: this piece's key tiles never arrive
      for (int kt = pc.kt0; kt < pc.kt1 && !stop; ++kt, ++g) {
        // this lane's box: its page (one that does not exist lies behind the tensor's end) and row
        const int p0 = kt * kBN + my_box * ta.box, row = p0 % a.P;
        int page = page_next;
        page_next = page_of(kt + 1);
        if (page < 0 || page >= a.num_pages) {
          if (mine && p0 < pc.q.kv) record_error(a.err, DFLASH_ERR_INVALID);
          page = a.num_pages;
        }
        const uint32_t r = PAIR ? 0u : g & 1u;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const uint32_t c = r ? load1 : load0;
          const uint32_t s = C::slot(r, c);
          if (!__all_sync(0xffffffffu, ctl.wait(C::RING_EMPTY + s, C::parity(c) ^ 1u))) {
            stop = true;
            break;
          }
          load0 += r ? 0u : 1u;
          load1 += r;
          if (lane == 0) ptx::mbar_arrive_expect_tx(ctl.bar(C::RING_FULL + s), C::kSlot);
          __syncwarp();
          if (mine) {
            const uint32_t dst = ring + s * C::kSlot + my_dst, full = ctl.bar(C::RING_FULL + s);
            const CUtensorMap* map = kv ? &tmV : &tmK;
            if (ta.dual) tma_load_5d(dst, map, full, 0, row, 0, pc.h, page);
            else tma_load_4d(dst, map, full, 64 * my_pn, pc.h, row, page);
          }
        }
      }
    }
    // Wind-down (also after a timeout): every load lands before the CTA exits.
    for (uint32_t r = 0; r < C::kRings; ++r) {
      const uint32_t c = r ? load1 : load0;
      for (uint32_t i = c > C::kRing ? c - C::kRing : 0u; i < c; ++i)
        ctl.wait_landed(C::RING_FULL + C::slot(r, i), C::parity(i));
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ queries
    if (lane == 0) {
      Walker<kBN> walk(a, range);
      Piece pc;
      const uint32_t q_bytes = (uint32_t)tile_rows * 128u;  // bytes of a box
      uint32_t n = 0;
      while (walk.next(&pc)) {
        const uint32_t b = q_buf(n), full = ctl.bar(C::Q_FULL + b);
        if (!ctl.wait(C::Q_EMPTY + b, q_parity(n) ^ 1u)) break;
        ptx::mbar_arrive_expect_tx(full, q_bytes * (PAIR ? 2 : 1) * NP);
        for (int i = 0; i < (PAIR ? 2 : 1); ++i)
          for (int pn = 0; pn < NP; ++pn)
            ptx::tma_load_3d(sbase + C::kOffQ + (i * NP + pn) * kPanel + b * (kPanel / 2), &tmQ, full, 64 * pn,
                             pc.h * a.G, pc.q.q0 + (pc.rt * (PAIR ? 2 : 1) + i) * ta.tokens);
        ++n;
      }
      // the last load of each buffer
      for (uint32_t i = n > q_two ? n - 1 - q_two : 0u; i < n; ++i)
        ctl.wait_landed(C::Q_FULL + q_buf(i), q_parity(i));
    }
  } else if (warp == 1 || warp == 2) {
    // ------------------------------------------------------------ MMA issuers
    if (lane == 0) {
      const int i = warp - 1;
      const uint32_t kIdescQK = ptx::idesc_bf16_f32(kBM, kBN, 0, 0);  // Q, K both K-major
      const uint32_t kIdescPV = ptx::idesc_bf16_f32(kBM, DP, 0, 1);   // P from TMEM, V MN-major
      const uint64_t dq = ptx::smem_desc(sbase + C::kOffQ + (PAIR ? i * NP * kPanel : 0u), 16, 1024);
      const uint64_t dK = ptx::smem_desc(ring, 16, ta.group);
      const uint64_t dV = ptx::smem_desc(ring, ta.panel, ta.group);
      const uint32_t d_s = tmem + kColS + 128u * i;  // S_i; P_i aliases its head
      const uint32_t d_o = tmem + kColO + 128u * i;
      const uint32_t r = PAIR ? 0u : (uint32_t)i;  // this half's ring
      uint32_t g = 0, mine = 0, n_q = 0;  // tiles of the CTA, tiles of this half, row tiles
      auto full = [&](uint32_t c) { return ctl.wait(C::RING_FULL + C::slot(r, c), C::parity(c)); };
      auto release = [&](uint32_t c) { ptx::tc_commit(ctl.bar(C::RING_EMPTY + C::slot(r, c))); };
      // m: this half's tile number
      auto issue_qk = [&](uint32_t m, uint32_t buf) {
        const uint64_t k = dK + ((C::slot(r, 2 * m) * C::kSlot) >> 4);
        const uint64_t q = dq + ((buf * (kPanel / 2)) >> 4);
#pragma unroll
        for (int ks = 0; ks < 4 * NP; ++ks) {
          const uint32_t sub = (uint32_t)(ks & 3) * 32u, pn = (uint32_t)(ks >> 2);
          ptx::mma_ss(d_s, q + ((pn * kPanel + sub) >> 4), k + ((pn * ta.panel + sub) >> 4), kIdescQK, ks > 0);
        }
        ptx::tc_commit(ctl.bar(C::S_FULL + i));
        release(2 * m);
      };
      auto issue_pv = [&](uint32_t m, bool first, int ks0) {
        const uint64_t v = dV + ((C::slot(r, 2 * m + 1) * C::kSlot) >> 4);
#pragma unroll
        for (int ks = ks0; ks < ks0 + 4; ++ks)  // 16 keys: 8 packed P columns, two groups of 8 V rows
          ptx::mma_ts(d_o, d_s + (uint32_t)ks * 8u, v + (((uint32_t)ks * 2u * ta.group) >> 4), kIdescPV,
                      !(first && ks == 0));
      };
      // PV: keys 0-63 once that half of P is written, then the rest.
      auto pv = [&](uint32_t m, bool first) -> bool {
        if (!full(2 * m + 1) || !ctl.wait(C::P_LO + i, m & 1u)) return false;
        ptx::tc_fence_after();
        issue_pv(m, first, 0);
        ptx::tc_commit(ctl.bar(C::PV_LO + i));
        if (!ctl.wait(C::P_HI + i, m & 1u)) return false;
        ptx::tc_fence_after();
        issue_pv(m, false, 4);
        release(2 * m + 1);
        return true;
      };
      Walker<kBN> walk(a, range);
      Piece pc;
      bool stop = false;
      while (!stop && walk.next(&pc)) {
        const uint32_t buf = q_buf(n_q);
        if (!ctl.wait(C::Q_FULL + buf, q_parity(n_q))) break;
        ++n_q;
        bool any = false, first_pv = true;
        for (int kt = pc.kt0; kt < pc.kt1; ++kt, ++g) {
          if (!PAIR && (int)(g & 1u) != i) continue;
          if (!full(2 * mine)) {
            stop = true;
            break;
          }
          if (any) {
            if (!pv(mine - 1, first_pv)) {
              stop = true;
              break;
            }
            first_pv = false;
          }
          // PAIR: the halves' QKs take turns, so that S_1 lands one QK after S_0 and the
          // softmax warpgroups run staggered.
          if (PAIR &&
              (i == 1 ? !ctl.wait(C::QK_TURN + 0, g & 1u) : (g > 0 && !ctl.wait(C::QK_TURN + 1, (g - 1) & 1u)))) {
            stop = true;
            break;
          }
          ptx::tc_fence_after();
          issue_qk(mine, buf);
          if (PAIR) ptx::mbar_arrive(ctl.bar(C::QK_TURN + i));
          any = true;
          ++mine;
        }
        if (stop) break;
        ptx::tc_commit(ctl.bar(C::Q_EMPTY + buf));  // every QK of this half has been issued
        if (any) {
          if (!pv(mine - 1, first_pv)) break;
          ptx::tc_commit(ctl.bar(C::O_FULL + i));
        }
      }
      // Drain: every MMA this thread issued has finished before TMEM is released.
      ptx::tc_commit(ctl.bar(C::DRAIN));
      const uint64_t t0 = ptx::globaltimer();
      while (!ptx::mbar_try_wait(ctl.bar(C::DRAIN), 0)) {
        if (ptx::globaltimer() - t0 > kWaitBudgetNs) {
          record_error(ctl.err, DFLASH_ERR_TIMEOUT);
          break;
        }
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax + epilogue (warps 4..11)
    ptx::setmaxnreg_inc<kSoftmaxRegs>();
    const int half = (warp - 4) >> 2;
    const int row = (warp & 3) * 32 + lane;  // TMEM lane = row of the tile
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lane_off + kColS + 128u * half;
    const uint32_t o_col = tmem + lane_off + kColO + 128u * half;
    const uint32_t o_base = tmem + lane_off + kColO;
    const float c2 = a.scale_log2;
    Walker<kBN> walk(a, range);
    Piece pc;
    Meta meta = no_meta();
    uint32_t g = 0, mine = 0, n_epi = 0;  // tiles of the CTA, tiles of this half, pieces finished
    uint32_t n_full[2] = {0, 0};          // accumulators finished, each half
    bool stop = false;
    while (!stop && walk.next(&pc)) {
      const int f = pc.rt * a.rows + (PAIR ? half * tile_rows : 0) + row;  // row within (request, key/value head)
      const bool row_ok = row < tile_rows && f < pc.q.n * a.G;
      const int tok = f / a.G;
      const int base = pc.q.kv - pc.q.n;  // position of the first new token
      const int lim = !row_ok ? 0 : a.causal ? max(0, base + tok + 1) : pc.q.kv;  // (not TREE)
      const bool warp_ok = __any_sync(0xffffffffu, row_ok);
      float m_used = -INFINITY, l = 0.f;
      bool had[2] = {PAIR, PAIR};
      for (int kt = pc.kt0; kt < pc.kt1; ++kt, ++g) {
        if (!PAIR) {
          had[0] |= (g & 1u) == 0;
          had[1] |= (g & 1u) == 1;
          if ((int)(g & 1u) != half) continue;
        }
        const int k0 = kt * kBN;
        if (k0 + kBN > pc.q.kv) {
          // the request ends in this tile: its rows of V behind the end become zeros
          const uint32_t c = 2 * mine + 1, s = C::slot(PAIR ? 0u : (uint32_t)half, c);
          if (!__all_sync(0xffffffffu, ctl.wait(C::RING_FULL + s, C::parity(c)))) {
            stop = true;
            break;
          }
          if (k0 + row >= pc.q.kv) {
            uint8_t* at = smem + C::kOffRing + s * C::kSlot + (row >> 3) * ta.group + (row & 7) * 128;
#pragma unroll
            for (int pn = 0; pn < NP; ++pn)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                reinterpret_cast<uint4*>(at + pn * ta.panel)[e] = make_uint4(0u, 0u, 0u, 0u);
          }
          ptx::fence_proxy_async_smem();
        }
        // TREE: what the row sees of a tile with new tokens in it, while S is on its way
        const bool hides = TREE && (k0 + kBN > base || !row_ok);
        TreeBits<2> vis;
        if (hides) vis = tree_bits<2>(a.parents + pc.q.q0, row_ok ? tok : -1, base - k0);
        if (!__all_sync(0xffffffffu, ctl.wait(C::S_FULL + half, mine & 1u))) {
          stop = true;
          break;
        }
        ptx::tc_fence_after();
        float2 lsum = make_float2(0.f, 0.f);
        // (unrolled: chunks 815 -> 801 us; decode, where code is fetched anew for every
        // short piece, runs 4 % slower so)
#pragma unroll(PAIR ? 2 : 1)
        for (int hh = 0; hh < 2; ++hh) {
          if (warp_ok) {  // a warp without a row leaves its lanes of P as they are: they reach no other row
            float x[64];
            ptx::tmem_ld32(s_col + 64u * hh, reinterpret_cast<uint32_t*>(x));
            ptx::tmem_ld32(s_col + 64u * hh + 32u, reinterpret_cast<uint32_t*>(x) + 32);
            ptx::tmem_wait_ld();
            if (!TREE) hide64(x, 64 * hh, lim - k0);
            else if (hides) hide_bits(x, hh ? vis.w[1] : vis.w[0]);
            const float mh = max64(x) * c2;
            const bool raise = mh > m_used + 8.0f;  // also when m is still -inf and this half sees a key
            const bool scale_o = raise && m_used != -INFINITY;
            if (__any_sync(0xffffffffu, scale_o)) {
              const float alpha = scale_o ? ptx::ex2(m_used - mh) : 1.f;
              // second half: PV of keys 0-63 may still be adding to O
              if (hh == 1 && !__all_sync(0xffffffffu, ctl.wait(C::PV_LO + half, mine & 1u))) stop = true;
              ptx::tc_fence_after();
#pragma unroll 1
              for (int cc = 0; cc < DP; cc += 32) {
                uint32_t o[32];
                ptx::tmem_ld32(o_col + cc, o);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                ptx::tmem_st32(o_col + cc, o);
              }
              ptx::tmem_wait_st();
              l *= alpha;
              lsum.x *= alpha;
              lsum.y *= alpha;
            }
            if (raise) m_used = mh;
            const float msub = m_used == -INFINITY ? 0.f : m_used;
            const float2 mul2 = make_float2(c2, c2), neg2 = make_float2(-msub, -msub);
            uint32_t pk[32];
#pragma unroll
            for (int c = 0; c < 64; c += 2) {
              const float2 arg = __ffma2_rn(make_float2(x[c], x[c + 1]), mul2, neg2);
              const float2 pp = make_float2(ptx::ex2(arg.x), ptx::ex2(arg.y));
              lsum = __fadd2_rn(lsum, pp);
              pk[c / 2] = ptx::pack_bf16x2(pp.x, pp.y);
            }
            ptx::tmem_st32(s_col + 32u * hh, pk);
            ptx::tmem_wait_st();
          }
          ptx::tc_fence_before();
          ptx::mbar_arrive(ctl.bar((hh == 0 ? C::P_LO : C::P_HI) + half));
        }
        if (stop) break;
        l += lsum.x + lsum.y;
        ++mine;
      }
      if (stop) break;
      // ---- the piece's end: out = O / l, or (O, m, l) for the merge
      const long long part = pc.slot >= 0 ? (long long)pc.slot * a.rows + (PAIR ? half * tile_rows : 0) + row : 0;
      const int head = pc.h * a.G + (row_ok ? f % a.G : 0);
      const long long token = (long long)pc.q.q0 + tok;
      // SPLIT: both halves' accumulators are added up, each half taking half of the
      // columns, or one half alone had tiles and finishes them by itself, while the
      // other goes on to the next piece.
      const bool both = !PAIR && had[0] && had[1];
      float w0 = 1.f, w1 = 1.f, m = m_used;
      if (both) {
        ml[half * kBM + row] = make_float2(m_used, l);
        ptx::mbar_arrive(ctl.bar(C::ML));
        if (!__all_sync(0xffffffffu, ctl.wait(C::ML, n_epi & 1u))) break;
        const float2 a0 = ml[row], a1 = ml[kBM + row];
        m = fmaxf(a0.x, a1.x);
        const float mm = m == -INFINITY ? 0.f : m;
        w0 = ptx::ex2(a0.x - mm);
        w1 = ptx::ex2(a1.x - mm);
        l = w0 * a0.y + w1 * a1.y;
      }
      bool landed = true;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (both || (had[i] && i == half)) landed = ctl.wait(C::O_FULL + i, n_full[i] & 1u) && landed;
      if (!__all_sync(0xffffffffu, landed)) break;
#pragma unroll
      for (int i = 0; i < 2; ++i) n_full[i] += had[i];
      ptx::tc_fence_after();
      const float inv = pc.slot >= 0 ? 1.f : l == 0.f ? 0.f : 1.f / l;
      w0 *= inv;
      w1 *= inv;
      if (warp_ok && (half ? had[1] : had[0])) {
        const int c0 = both ? half * (DP / 2) : 0, c1 = both ? c0 + DP / 2 : DP;
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + (token * a.Hq + head) * a.D;
        float* pdst = a.part_o + part * a.D;
#pragma unroll 1
        for (int cc = c0; cc < c1; cc += 32) {
          uint32_t o[32];
          __syncwarp();  // the TMEM reads take the whole warp
          ptx::tmem_ld32(both ? o_base + cc : o_col + cc, o);
          if (!PAIR && both) {
            uint32_t o1[32];
            ptx::tmem_ld32(o_base + 128u + cc, o1);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = __float_as_uint(fmaf(__uint_as_float(o1[e]), w1, __uint_as_float(o[e]) * w0));
          } else {
            ptx::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
          }
          if (!row_ok) {
          } else if (pc.slot >= 0) {
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              if (cc + e < a.D) ptx::st_global_v8(pdst + cc + e, o + e);
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 16) {
              uint32_t b[8];
#pragma unroll
              for (int u = 0; u < 8; ++u)
                b[u] = ptx::pack_bf16x2(__uint_as_float(o[e + 2 * u]), __uint_as_float(o[e + 2 * u + 1]));
              const int col = cc + e;
              if (ta.out_v8 && col + 16 <= a.D) {
                ptx::st_global_v8(dst + col, b);
              } else {
                if (col < a.D) *reinterpret_cast<uint4*>(dst + col) = make_uint4(b[0], b[1], b[2], b[3]);
                if (col + 8 < a.D) *reinterpret_cast<uint4*>(dst + col + 8) = make_uint4(b[4], b[5], b[6], b[7]);
              }
            }
          }
        }
        if (row_ok && !(both && half == 1)) {
          if (pc.slot >= 0) a.part_ml[part] = make_float2(m, l);
          else if (a.lse)
            a.lse[(long long)head * a.total_q + token] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        }
      }
      if (both) {
        // neither half's next PV may overwrite an accumulator that the other still reads
        ptx::tc_fence_before();
        ptx::mbar_arrive(ctl.bar(C::EPI));
        if (!__all_sync(0xffffffffu, ctl.wait(C::EPI, n_epi & 1u))) break;
        ptx::tc_fence_after();
        ++n_epi;
      }
      if (begins_cut(pc)) meta = meta_of(a, range, pc);
    }
    if (warp == 4 && lane == 0) a.meta[blockIdx.x] = meta;
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

int gcd(int x, int y) {
  while (y) {
    const int t = x % y;
    x = y;
    y = t;
  }
  return x;
}

template <int NP, bool PAIR, bool TREE>
cudaError_t run_tc(const TcPagedArgs& ta, int grid, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                   cudaStream_t s) {
  auto kernel = paged_tc_kernel<NP, PAIR, TREE>;
  // Once a device: the shared memory's size, and the registers.  The setmaxnreg
  // split assumes the kernel launches with exactly kLaunchRegs registers a thread;
  // any other count would make setmaxnreg.inc wait forever.
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev >= 64 || !(ready.load(std::memory_order_acquire) & bit)) {
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, kernel) != cudaSuccess || fa.numRegs != kLaunchRegs)
      return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<NP, PAIR>::kSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  kernel<<<grid, kThreads, Cfg<NP, PAIR>::kSmem, s>>>(ta, q, k, v);
  count_launch();
  return cudaGetLastError();
}

template <bool TREE>
cudaError_t pick_tc(const TcPagedArgs& ta, bool pair, int grid, const CUtensorMap& q, const CUtensorMap& k,
                    const CUtensorMap& v, cudaStream_t s) {
  if (ta.a.D <= 64) return pair ? run_tc<1, true, TREE>(ta, grid, q, k, v, s) : run_tc<1, false, TREE>(ta, grid, q, k, v, s);
  return pair ? run_tc<2, true, TREE>(ta, grid, q, k, v, s) : run_tc<2, false, TREE>(ta, grid, q, k, v, s);
}

}  // namespace

bool paged_tc_supported(int G, int D, int P) { return D <= 128 && D % 8 == 0 && G <= kBM && P % 8 == 0; }

// A second row tile where some request has more rows than one holds: 808 us against 881
// for 2048 tokens behind 32768, 45 against 55 for 16 requests of 33 to 48 tokens (4
// heads a group), 21 and 21 where 4 requests of 30 to 100 tokens leave few row tiles.
static bool paired(int G, int max_q) { return max_q > kBM / G; }

// Tokens of a tile of up to 128 rows.
static int tile_tokens(int G, int max_q) { return max_q < kBM / G ? max_q : kBM / G; }

int paged_tc_rows(int G, int max_q) { return tile_tokens(G, max_q) * G * (paired(G, max_q) ? 2 : 1); }

cudaError_t launch_paged_tc(const PagedArgs& a, int grid, cudaStream_t stream) {
  TcPagedArgs ta;
  ta.a = a;
  ta.tokens = tile_tokens(a.G, a.max_q);
  ta.box = gcd(a.P, kBN);
  ta.dual = ta.box == 8 && a.D == 128;
  ta.panel = ta.dual ? 1024 : kPanel;
  ta.group = ta.dual ? 2048 : 1024;
  const bool pair = paired(a.G, a.max_q);
  // (26 us for 64 blocks with contexts of up to 200 positions, 27 with one buffer)
  ta.q_bufs = !pair && ta.tokens * a.G <= kBM / 2 ? 2 : 1;
  ta.out_v8 = ((uintptr_t)a.out & 31u) == 0 && a.D % 16 == 0;
  typedef unsigned long long u64;
  CUtensorMap mq, mk, mv;
  const u64 dq[3] = {(u64)a.D, (u64)a.Hq, (u64)a.total_q};
  const u64 sq[2] = {2ull * a.D, 2ull * a.D * a.Hq};
  const unsigned bq[3] = {64, (unsigned)a.G, (unsigned)ta.tokens};
  if (!make_map_3d_box(&mq, a.q, dq, sq, bq)) return cudaErrorInvalidValue;
  // A row of one head is 2 D bytes among the other heads' rows: L2 is not to fetch
  // beyond it, since the neighbours' turn is another CTA's (rows of 128 bytes fetched
  // in 256 took 369 us for the block step with D = 64).
  const int l2 = 2 * a.D % 256 == 0 ? 256 : 2 * a.D % 128 == 0 ? 128 : 64;
  const u64 head = 2ull * a.D, token = head * a.Hkv;
  bool ok = true;
  for (int v = 0; v < 2; ++v) {
    CUtensorMap* m = v ? &mv : &mk;
    const void* base = v ? a.vc : a.kc;
    const u64 page = 2ull * (u64)(v ? a.vps : a.kps);
    if (ta.dual) {
      const u64 d[5] = {64, (u64)a.P, 2, (u64)a.Hkv, (u64)a.num_pages}, s[4] = {token, 128, head, page};
      const unsigned b[5] = {64, 8, 2, 1, 1};
      ok = ok && make_map_box(m, base, 5, d, s, b, l2);
    } else {
      const u64 d[4] = {(u64)a.D, (u64)a.Hkv, (u64)a.P, (u64)a.num_pages}, s[3] = {head, token, page};
      const unsigned b[4] = {64, 1, (unsigned)ta.box, 1};
      ok = ok && make_map_box(m, base, 4, d, s, b, l2);
    }
  }
  if (!ok) return cudaErrorInvalidValue;
  return a.parents ? pick_tc<true>(ta, pair, grid, mq, mk, mv, stream) : pick_tc<false>(ta, pair, grid, mq, mk, mv, stream);
}

}  // namespace paged
}  // namespace dflash
