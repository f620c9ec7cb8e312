// Attention of one new token per sequence over a paged K/V cache (no selection): query heads in groups
// of 1..64 per key head, pages of any multiple of 16 rows, lengths on the device, an optional window.
//
// Per sequence, key head and query head of its group, over the keys j in [max(0, len - window), len):
//   out = softmax(scale q.k_j) V,   lse = log sum_j exp(scale q.k_j)
//
// Bound by HBM: K and V are read once (4 G flops per byte of a bf16 cache at a group of G heads), so the
// design keeps TMA loads in flight and everything else off their path. Two CTAs per SM, each a TMA
// warp, an MMA warp and four softmax warps around one ring of 16 KB tiles:
//   S = Q K^T      tcgen05, M = 64 (the group's heads, zero-padded), N = the tile's keys
//   P = exp2(S c - m_tile)   the lanes that hold a head's row (two per row), to shared memory
//   O_tile = P V   tcgen05, a fresh accumulator per tile
//   acc = acc 2^(m - m') + O_tile 2^(m_tile - m'),  m' = max(m, m_tile)   32-bit registers
// P is relative to its own tile's maximum, so it keeps its precision however far that maximum lies
// below the row's (a cache with one dominant key).
//
// An e4m3 cache goes to the tensor core as it is (kind::f8f6f4; nothing is widened). The 16-bit
// operand beside it is split into two 8-bit terms whose products accumulate in the same accumulator.
// P (scaled by 256): hi = e4m3(x), lo = e4m3(x - hi), 4 + 4 significant bits, as many as a bf16 has. Q, scaled
// per head by a power of two so that its largest element lies in [2^10, 2^11): hi = e5m2(x), lo =
// e4m3(x - hi). The first term leaves a multiple of 0 .. 16 of a bf16's last bit, which four bits hold, so an element
// is exact down to 2^-12 of the largest, and off by 2^-20 of that at most below (e4m3 for both terms:
// exact to 2^-9, off by 2^-17, which the logsumexp of a few keys showed: 7e-7 of it against 4e-8).
//
// The tiles of all (sequence, key head) pairs form one line that is cut into ranges of equal cost, one per
// CTA, from the lengths on the device (a captured launch serves any lengths). A pair that lies in one
// CTA's range is finished there; the others leave (m, l, acc) records that a second kernel joins in
// the order of the ranges, so results do not vary from run to run. Calls whose page table has room for short sequences
// only take clusters instead (cluster_size).
//
// Measured against 6.56 TB/s, the memory's rate for a copy, in passes one after the other: 8 sequences of
// 256k tokens, 64 heads on one key head, 171 us (6.3 TB/s; 183 us when a long run holds the clocks at the
// power limit); 48 of up to 8k, 32 heads on 8 in pages of 16, 96 us (6.1; 99); e4m3 codes, 8 of up to 256k, 70 us
// (4.7; 81 us at the power limit). There the tensor cores are 60% busy (M = 64 runs at half their rate, and
// both operands have two terms), and the softmax warps' chain from scores to P is as long as a tile's
// load. About 10 us of the long cases are start and end: the first tiles' way, the last tiles' chain, the join. Windows
// of 128 keys of 64 sequences, 64 heads on 8 in pages of 16, take 22 us for 5 us of bytes: a pair's two or three tiles are
// little but its start and end. The line's kernels spill 4 to 48 bytes a thread (168 registers, two CTAs an SM).
// Tried and slower: eight softmax warps of half the columns with their maxima exchanged (140 us for 118 at
// 8 x 256k of e4m3); a part of the exponentials on the FMA pipe (114 for 110); the products of a row kept
// in tensor memory with the row rescaled when its maximum moves (bf16 1% faster at 16k, e4m3 3% slower, or
// less exact where one key outweighs the rest).
#include <type_traits>

#include "host_util.h"
#include "tc.cuh"

namespace hs2 {
namespace pattn {

constexpr int NT = 192;   // TMA warp, MMA warp, four softmax warps
constexpr int MH = 64;    // MMA rows
constexpr int kNoPage = -2147483647 - 1;
constexpr int MIN_TILES = 2;  // a CTA's share of the line at least: a record costs about as much as a tile
constexpr int OV = 2;         // what starting and ending a pair costs, in tiles

struct Params {
  const __nv_bfloat16* q;  // [B, Hq, D]
  __nv_bfloat16* out;      // [B, Hq, D]
  float* lse;              // [B, Hq] or NULL
  const int32_t *ptab, *lens;
  int B, Hk, G, page, box, max_pages, n_pages, window;
  float c;       // scale log2(e), times K's scale
  float oscale;  // V's scale
  int W;         // CTAs of the grid at most in use; of a cluster
  int4* cuts;    // [W] of the cut before each CTA's range: pair, its first CTA, its segments (0: no cut in a pair)
  float* po;     // [W][2][G][D] records
  float2* pml;   // [G][W][2] their maxima and sums (a row's side by side: the join reads them a line at a time)
  long long wait_ns;
  DevStatus* st;
};

constexpr int MAX_NR = 5;
constexpr int MAX_CS = 8;  // CTAs of a cluster at most
constexpr int FEW = 256;   // keys: above, the roundings of P average out (and two terms cost a tenth of the time)
struct Shared {
  uint64_t r_full[MAX_NR], r_empty[MAX_NR], q_ready, s_full, s_free, p_ready, o_full, drained;
  uint32_t tmem_base;
  volatile int abort_flag;
  int warp_sum[NT / 32], start[6];
};

// CL: the clusters of short sequences. Where a head sees few keys they hold P in two bf16 terms (e4m3 has two
// anyway), 16 significant bits, for one rounding of each to bf16 shows there (a head with two keys: 0.0027 of the
// output instead of 0.0016; from 256 keys on 0.0019 and less).
template <int D, bool F8, bool CL>
struct Lay {
  static constexpr int TILE = F8 || D == 64 ? 128 : 64;       // keys of a tile: 16 KB of K
  static constexpr int EB = F8 ? 1 : 2;
  static constexpr int NKB = D * EB / 128;                    // 128-byte column blocks of a cache row
  static constexpr int SLOT = TILE * D * EB;
  static constexpr int Q_BYTES = MH * D * 2;                  // (e4m3: hi and lo terms)
  static constexpr int P_BYTES = MH * TILE * 2;               // one term of P (e4m3: both)
  static constexpr bool TWO = CL && !F8;
  static constexpr int NB = TWO && D == 64 ? 1 : 2, PB = P_BYTES * (TWO ? 2 : 1);  // buffers of P, one's bytes
  static constexpr int NR = F8 || D == 64 || CL ? 4 : 5;      // ring slots
  static constexpr int OFF_P = Q_BYTES, OFF_R = OFF_P + NB * PB;
  static constexpr int REC = D * 4 + 16;  // a row's accumulators in a cluster's join (16 bytes apart: banks)
  static_assert(MH * (REC + 8) <= NR * SLOT, "a cluster's records lie in the ring");
  // the barriers lie behind the ring and nothing is declared beside it: 1,024-byte aligned without
  // slack, so that two CTAs with a fifth slot fit an SM
  static constexpr int OFF_B = OFF_R + NR * SLOT;
  static constexpr int BYTES = OFF_B + (int)sizeof(Shared);
};

__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, long long limit, volatile int* abort_flag,
                                         DevStatus* st, unsigned where) {
  const uint32_t a = smem_u32(bar);
  if (mbar_try_wait(a, parity)) return true;
  const long long t0 = globaltimer_ns();
  while (true) {
    if (mbar_try_wait(a, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > limit) {
      *abort_flag = 1;
      report_status(st, kStatusTimeout, where);
      return false;
    }
  }
}
// the whole warp waits and gets one answer
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, long long limit, volatile int* abort_flag,
                                          DevStatus* st, unsigned where) {
  if (__all_sync(0xffffffffu, mbar_try_wait(smem_u32(bar), parity))) return true;
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = wait_bar(bar, parity, limit, abort_flag, st, where) ? 1 : 0;
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// A in e4m3, or in e5m2; B in e4m3
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, int a_mn, int b_mn, int a_e5m2) {
  return (1u << 4) | ((uint32_t)(a_e5m2 & 1) << 7) | ((uint32_t)(a_mn & 1) << 15) | ((uint32_t)(b_mn & 1) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);  // D = f32; formats: e4m3 0, e5m2 1
}
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::
          "r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// two values (the first in the low half) as f16x2 -> their hi and lo e4m3 codes (the first in the low byte)
__device__ __forceinline__ void split_e4m3(uint32_t x, uint32_t& hi, uint32_t& lo) {
  uint16_t h, l;
  uint32_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h) : "r"(x));
  asm("{.reg .b32 w;\n\tcvt.rn.f16x2.e4m3x2 w, %1;\n\tsub.rn.f16x2 %0, %2, w;}" : "=r"(r) : "h"(h), "r"(x));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(l) : "r"(r));
  hi = h;
  lo = l;
}

// the same with the first term in e5m2
__device__ __forceinline__ void split_e5m2(uint32_t x, uint32_t& hi, uint32_t& lo) {
  uint16_t h, l;
  uint32_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(h) : "r"(x));
  asm("{.reg .b32 w;\n\tcvt.rn.f16x2.e5m2x2 w, %1;\n\tsub.rn.f16x2 %0, %2, w;}" : "=r"(r) : "h"(h), "r"(x));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(l) : "r"(r));
  hi = h;
  lo = l;
}

// A sequence's tiles: from the one that holds its first visible key to the one that holds its last.
// A length that the page table cannot hold counts as none.
template <int TILE>
__device__ __forceinline__ int seq_tiles(const Params& p, int b, int& len, int& t0, bool* bad = nullptr) {
  len = p.lens[b];
  if (len < 0 || (long long)len > (long long)p.max_pages * p.page) {
    if (bad) *bad = true;
    len = 0;
  }
  const int first = p.window > 0 && len > p.window ? len - p.window : 0;
  t0 = first / TILE;
  return len > 0 ? (len + TILE - 1) / TILE - t0 : 0;
}

// A pair's length on the line: its tiles and OV more in front of them, so that a CTA whose range holds many
// short pairs gets fewer tiles.
__device__ __forceinline__ int pair_len(int n) { return n > 0 ? n + OV : 0; }

// The segments of a range [pos, end) of the line: runs of tiles of one (sequence, key head).
template <int TILE>
struct Walk {
  int b, base, len, t0, n;  // the sequence, its start on the line, its length, first tile, tiles per head
  int pos, end;
  int next_hk, at;          // the head that pos lies in, and its start on the line
  int hk, off, cnt;         // the segment: key head, first tile within the head's run, tiles
  __device__ __forceinline__ bool next(const Params& p) {
    while (pos < end) {
      const int m = pair_len(n);
      if (m > 0 && pos < base + p.Hk * m) {
        const int x = pos - at, y = min(m, x + end - pos);
        pos += y - x;
        hk = next_hk;
        if (y == m) { at += m; ++next_hk; }
        off = max(x - OV, 0);
        cnt = y - OV - off;
        if (cnt > 0) return true;
        continue;
      }
      base += p.Hk * m;
      at = base;
      next_hk = 0;
      ++b;
      if (b >= p.B) return false;
      n = seq_tiles<TILE>(p, b, len, t0);
    }
    return false;
  }
  __device__ __forceinline__ int first_key(const Params& p) const {
    return p.window > 0 && len > p.window ? len - p.window : 0;
  }
};

// The ranges of N tiles: the first N % W CTAs take one tile more than the others (one 32-bit division; a
// 64-bit w N / W cost the join as much as its records).
struct Split {
  int W, q, r;
  __device__ __forceinline__ Split(int N, int most, int least) {
    W = min(most, max((N + least - 1) / least, 1));
    q = N / W;
    r = N - q * W;
  }
  __device__ __forceinline__ int start(int w) const { return w * q + min(w, r); }
  __device__ __forceinline__ int owner(int tile) const {  // the CTA whose range holds it
    const int cut = r * (q + 1);
    return tile < cut ? tile / (q + 1) : r + (tile - cut) / q;
  }
};

// The one segment of a cluster's CTA.
template <int TILE>
struct One {
  int b, hk, len, t0, n, off, cnt;
  bool left;
  __device__ __forceinline__ bool next(const Params&) {
    const bool now = left;
    left = false;
    return now;
  }
  __device__ __forceinline__ int first_key(const Params& p) const {
    return p.window > 0 && len > p.window ? len - p.window : 0;
  }
};

// CL: short sequences. A cluster of p.W CTAs works on one (sequence, key head), its tiles shared out evenly,
// and joins its accumulators through distributed shared memory: no line, no records, no second kernel.
template <int D, bool F8, bool CL>
__global__ void __launch_bounds__(NT, 2) paged_attn_kernel(const __grid_constant__ CUtensorMap tmK,
                                                           const __grid_constant__ CUtensorMap tmV, Params p) {
  using L = Lay<D, F8, CL>;
  constexpr int TILE = L::TILE, NR = L::NR, NKB = L::NKB, SLOT = L::SLOT;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *sQ = smem, *sP = smem + L::OFF_P, *sR = smem + L::OFF_R;
  Shared& sh = *reinterpret_cast<Shared*>(smem + L::OFF_B);
  uint64_t *r_full = sh.r_full, *r_empty = sh.r_empty;
  uint64_t &q_ready = sh.q_ready, &s_full = sh.s_full, &s_free = sh.s_free, &p_ready = sh.p_ready, &o_full = sh.o_full,
           &drained = sh.drained;
  uint32_t& tmem_base = sh.tmem_base;
  volatile int& abort_flag = sh.abort_flag;
  int *warp_sum = sh.warp_sum, *s_start = sh.start;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nact = (p.G + 15) / 16;  // softmax warps with heads
  const long long limit = p.wait_ns;
  if (smem_u32(smem) & 1023) {  // (the tiles' swizzle needs it; nothing is declared that could move it)
    if (tid == 0) report_status(p.st, kStatusBounds, 700);
    return;
  }

  if (tid == 0) {
    for (int i = 0; i < NR; ++i) { mbar_init(&r_full[i], 1); mbar_init(&r_empty[i], 1); }
    mbar_init(&q_ready, nact); mbar_init(&s_full, 1); mbar_init(&s_free, nact);
    mbar_init(&p_ready, nact); mbar_init(&o_full, 1); mbar_init(&drained, 1);
    abort_flag = 0;
    s_start[0] = -1;
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  // rows of Q and P without a head stay zero
  for (int i = tid; i < L::OFF_R / 16; i += NT) st_shared_v4(smem_u32(smem) + i * 16, 0u, 0u, 0u, 0u);
  fence_async_smem();
  griddep_wait();
  // (a kernel before this one may still be about to take its tensor memory until the wait ends)
  if (warp == 1) { tmem_alloc(&tmem_base, 256); tmem_relinquish(); }
  griddep_launch_dependents();

  const int cta = blockIdx.x;
  int r0 = 0;  // the start of this CTA's range on the line
  Split split(1, 1, 1);
  std::conditional_t<CL, One<TILE>, Walk<TILE>> wk;
  if constexpr (CL) {
    const int rank = (int)cluster_ctarank(), pair = cta / p.W;
    bool bad = false;
    wk.b = pair / p.Hk; wk.hk = pair % p.Hk;
    wk.n = seq_tiles<TILE>(p, wk.b, wk.len, wk.t0, &bad);
    split = Split(wk.n, p.W, 1);
    wk.off = rank < split.W ? split.start(rank) : 0;
    wk.cnt = rank < split.W ? split.start(rank + 1) - wk.off : 0;
    wk.left = wk.cnt > 0;
    if (bad && rank == 0 && tid == 0) report_status(p.st, kStatusBounds, 701);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  } else {
    // ---- the line of tiles: each thread sums a run of sequences
    const int per = (p.B + NT - 1) / NT;
    int mine = 0;
    bool bad = false;
    for (int i = 0; i < per; ++i) {
      const int b = tid * per + i;
      int len, t0;
      if (b < p.B) mine += pair_len(seq_tiles<TILE>(p, b, len, t0, &bad));
    }
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int before = x - mine, all = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      const int s = warp_sum[w];
      if (w < warp) before += s;
      all += s;
    }
    const int N = all * p.Hk;
    split = Split(N, p.W, MIN_TILES);
    r0 = cta < split.W ? split.start(cta) : N;
    const int r1 = cta < split.W ? split.start(cta + 1) : N;
    if (r0 < r1 && before * p.Hk <= r0 && r0 < (before + mine) * p.Hk) {
      int at = before * p.Hk;
      for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        int len, t0;
        const int n = pair_len(seq_tiles<TILE>(p, b, len, t0));
        if (r0 < at + n * p.Hk) {
          const int hk = (r0 - at) / n;
          s_start[0] = b; s_start[1] = at; s_start[2] = len; s_start[3] = t0; s_start[4] = hk; s_start[5] = at + hk * n;
          break;
        }
        at += n * p.Hk;
      }
    }
    if (bad && cta == 0) report_status(p.st, kStatusBounds, 701);
    __syncthreads();
    wk.pos = r0; wk.end = s_start[0] >= 0 ? r1 : r0;
    wk.b = s_start[0]; wk.base = s_start[1]; wk.len = s_start[2]; wk.t0 = s_start[3];
    wk.next_hk = s_start[4]; wk.at = s_start[5];
    wk.n = wk.len > 0 ? (wk.len + TILE - 1) / TILE - wk.t0 : 0;
  }
  const uint32_t tmem = tmem_base, tS = 0, tO = 128;
  const bool two = L::TWO && wk.len - wk.first_key(p) <= FEW;  // P in two terms

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer: lane x loads
    // rows x * box .. of a tile (one page's), K and V of a tile from the same page ids
    const uint64_t once = policy_evict_first();
    const int n_box = TILE / p.box;
    uint32_t ri = 0;
    bool ok = true;
    auto load = [&](const CUtensorMap* m, int pg, int row, int hk) -> bool {
      const int s = ri % NR;
      if (!warp_wait(&r_empty[s], ((ri / NR) & 1) ^ 1, limit, &abort_flag, p.st, 702)) return false;
      if (lane == 0) mbar_expect_tx(&r_full[s], SLOT);
      __syncwarp();
      if (lane < n_box) {
        uint8_t* dst = sR + s * SLOT + lane * p.box * 128;
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) {
          asm volatile(
              "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, "
              "{%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst + kb * (TILE * 128))),
              "l"(m), "r"(smem_u32(&r_full[s])), "r"(kb * 64), "r"(row), "r"(hk), "r"(pg), "l"(once)
              : "memory");
        }
      }
      ++ri;
      return true;
    };
    while (ok && wk.next(p)) {
      const int first = wk.first_key(p);
      const int32_t* row_ids = p.ptab + (size_t)wk.b * p.max_pages;
      // the page of this lane's rows of tile t: one past the pool (which reads zeros) where no key of
      // them is visible or the id is not one of the pool's
      auto page_of = [&](int t) -> int {
        const int k0 = t * TILE + lane * p.box;
        if (lane >= n_box || k0 >= wk.len || k0 + p.box <= first) return kNoPage;
        const int pg = row_ids[k0 / p.page];
        return pg == kNoPage ? -1 : pg;
      };
      auto checked = [&](int pg) -> int {
        if (pg >= 0 && pg < p.n_pages) return pg;
        if (pg != kNoPage) report_status(p.st, kStatusBounds, 703);
        return p.n_pages;
      };
      const int t_lo = wk.t0 + wk.off, t_hi = t_lo + wk.cnt;
      int pg_next = page_of(t_lo), pg_v = 0, row_v = 0;
      for (int t = t_lo; t < t_hi && ok; ++t) {
        const int raw = pg_next, row = (t * TILE + lane * p.box) % p.page;
        if (t + 1 < t_hi) pg_next = page_of(t + 1);
        int pg = checked(raw);
        ok = load(&tmK, pg, row, wk.hk);
        if (ok && t > t_lo) ok = load(&tmV, pg_v, row_v, wk.hk);
        pg_v = pg;
        row_v = row;
      }
      if (ok) ok = load(&tmV, pg_v, row_v, wk.hk);
    }
    if (!ok)  // let the copies already issued land before the CTA exits
      for (uint32_t i = ri > NR ? ri - NR : 0; i < ri; ++i) mbar_wait(&r_full[i % NR], (i / NR) & 1, limit);
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer (one thread); before
    // the first tile can arrive the warp writes what the join has to know, and the rows of sequences without a key
    auto zero = [&](size_t row0, int rows) {
      uint4* dst = reinterpret_cast<uint4*>(p.out + row0 * D);
      for (int i = lane; i < rows * (D / 8); i += 32) dst[i] = make_uint4(0u, 0u, 0u, 0u);
      if (p.lse)
        for (int i = lane; i < rows; i += 32) p.lse[row0 + i] = -INFINITY;
    };
    if constexpr (CL) {
      if (wk.n == 0 && cta % p.W == 0) zero((size_t)(cta / p.W) * p.G, p.G);
    } else {
      if (lane == 1) {
        int4 c = make_int4(0, 0, 0, 0);
        if (s_start[0] >= 0) {
          const int s = wk.at + OV;
          if (r0 > s) {
            c.x = wk.b * p.Hk + wk.next_hk;
            c.y = split.owner(s);
            c.z = split.owner(s + wk.n - 1) + 1 - c.y;
          }
        }
        p.cuts[cta] = c;
      }
      for (int b = cta; b < p.B; b += gridDim.x) {
        int len, t0;
        if (seq_tiles<TILE>(p, b, len, t0) == 0) zero((size_t)b * p.Hk * p.G, p.Hk * p.G);
      }
    }
    __syncwarp();
    if (lane == 0) {
      uint32_t ri = 0, js = 0, jp = 0, nq = 0;
      bool ok = true;
      const uint64_t qa = sdesc(smem_u32(sQ), 16, 1024), pa = sdesc(smem_u32(sP), 16, 1024);
      auto issue_s = [&]() -> bool {
        const int s = ri % NR;
        if (!wait_bar(&r_full[s], (ri / NR) & 1, limit, &abort_flag, p.st, 711)) return false;
        if (!wait_bar(&s_free, (js & 1) ^ 1, limit, &abort_flag, p.st, 712)) return false;
        tc_fence_after();
        const uint64_t ka = sdesc(smem_u32(sR + s * SLOT), 16, 1024);
        if constexpr (F8) {
#pragma unroll
          for (int h = 0; h < 2; ++h)  // Q's hi and lo terms
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
              umma_f8(tmem + tS, sdesc_at(qa, h * (MH * 128) + kk * 32), sdesc_at(ka, kk * 32),
                      idesc_f8(MH, TILE, 0, 0, h == 0), h + kk > 0);
        } else {
          constexpr uint32_t ID = idesc_bf16(MH, TILE, 0, 0);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_ss(tmem + tS, sdesc_at(qa, (kk / 4) * (MH * 128) + (kk % 4) * 32),
                    sdesc_at(ka, (kk / 4) * (TILE * 128) + (kk % 4) * 32), ID, kk > 0);
        }
        umma_commit(&s_full);
        umma_commit(&r_empty[s]);
        ++ri;
        ++js;
        return true;
      };
      auto issue_pv = [&]() -> bool {
        const int s = ri % NR;
        if (!wait_bar(&r_full[s], (ri / NR) & 1, limit, &abort_flag, p.st, 713)) return false;
        // P is in shared memory (and the accumulator of the tile before it has been read)
        if (!wait_bar(&p_ready, jp & 1, limit, &abort_flag, p.st, 714)) return false;
        tc_fence_after();
        const uint32_t pb = L::NB == 2 ? (jp & 1) * L::PB : 0;
        if constexpr (F8) {
          constexpr uint32_t ID = idesc_f8(MH, D, 0, 1, 0);
          const uint64_t va = sdesc(smem_u32(sR + s * SLOT), TILE * 128, 1024);
#pragma unroll
          for (int h = 0; h < 2; ++h)  // P's hi and lo terms
#pragma unroll
            for (int kk = 0; kk < TILE / 32; ++kk)
              umma_f8(tmem + tO, sdesc_at(pa, pb + h * (MH * 128) + kk * 32), sdesc_at(va, kk * 4096), ID, h + kk > 0);
        } else {
          constexpr uint32_t ID = idesc_bf16(MH, D, 0, 1);
          const uint64_t va = sdesc(smem_u32(sR + s * SLOT), TILE * 128, 1024);
#pragma unroll
          for (int h = 0; h < (L::TWO ? 2 : 1); ++h)
            if (h == 0 || two)
#pragma unroll
            for (int kk = 0; kk < TILE / 16; ++kk)
              umma_ss(tmem + tO, sdesc_at(pa, pb + h * L::P_BYTES + (kk / 4) * (MH * 128) + (kk % 4) * 32),
                      sdesc_at(va, kk * 2048), ID, h + kk > 0);
        }
        umma_commit(&o_full);
        umma_commit(&r_empty[s]);
        ++ri;
        ++jp;
        return true;
      };
      while (ok && wk.next(p)) {
        ok = wait_bar(&q_ready, nq & 1, limit, &abort_flag, p.st, 710);
        ++nq;
        for (int i = 0; i < wk.cnt && ok; ++i) {
          ok = issue_s();
          if (ok && i > 0) ok = issue_pv();
        }
        if (ok) ok = issue_pv();
      }
      if (!ok) {  // no MMA may still be running when the CTA gives its tensor memory back
        umma_commit(&drained);
        mbar_wait(&drained, 0, limit);
      }
    }
  } else if ((warp & 3) < nact) {
    // ------------------------------------------------------------------ softmax: lanes l and l + 16 of
    // warp quarter qd share head row 16 qd + l (TMEM keeps the rows of an M = 64 accumulator in the
    // first 16 lanes of each quarter); the first takes a tile's lower keys and the head's lower
    // columns, the second the upper ones
    const int qd = warp & 3, row = qd * 16 + (lane & 15), lh = lane >> 4;
    const uint32_t tq = tmem + ((uint32_t)(qd * 32) << 16);
    constexpr int SC = TILE / 2, OC = D / 2;  // columns of a lane
    constexpr int NL = SC / 32, NO = OC / 32;
    const int s0 = lh * SC, o0 = lh * OC;     // the first ones
    uint32_t js = 0, jp = 0, ring = 0;
    bool ok = true;
    // a pair's query row -> shared memory (once its last pair's score products are done); the
    // factor from its scores to exponents
    auto load_q = [&](int pair) -> float {
      float c = p.c;
      const __nv_bfloat16* src = p.q + ((size_t)pair * p.G + row) * D;
      if constexpr (F8) {
        uint4 w[D / 16];
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          w[i] = row < p.G ? reinterpret_cast<const uint4*>(src + o0)[i] : make_uint4(0u, 0u, 0u, 0u);
        float am = 0.f, nan = 0.f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint32_t a[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float v0 = __uint_as_float(a[k] << 16), v1 = __uint_as_float(a[k] & 0xFFFF0000u);
            am = fmaxf(am, fmaxf(fabsf(v0), fabsf(v1)));
            nan += (v0 - v0) + (v1 - v1);  // NaN when an element is infinite or NaN
          }
        }
        am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 16));
        nan += __shfl_xor_sync(0xffffffffu, nan, 16);
        // am 2^e in [2^10, 2^11)
        int e = 137 - (int)(__float_as_uint(am) >> 23);  // 127 + 10 - biased exponent
        e = am > 0.f ? (e < -120 ? -120 : e > 120 ? 120 : e) : 0;
        const float up = __uint_as_float((uint32_t)(127 + e) << 23);
        c = p.c * __uint_as_float((uint32_t)(127 - e) << 23) + nan;
#pragma unroll
        for (int i = 0; i < D / 16; i += 2) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4& ww = w[i + k / 2];
            const uint32_t a = k % 2 ? ww.z : ww.x, b2 = k % 2 ? ww.w : ww.y;
            uint32_t h0, l0, h1, l1;
            // (a bf16 element times that power of two is an f16 value, or too small to matter)
            split_e5m2(pack_f16x2(__uint_as_float(a << 16) * up, __uint_as_float(a & 0xFFFF0000u) * up), h0, l0);
            split_e5m2(pack_f16x2(__uint_as_float(b2 << 16) * up, __uint_as_float(b2 & 0xFFFF0000u) * up), h1, l1);
            hi[k] = h0 | (h1 << 16);
            lo[k] = l0 | (l1 << 16);
          }
          const uint32_t dst = smem_u32(sQ) + sw128_off(row, o0 / 16 + i / 2);
          st_shared_v4(dst, hi[0], hi[1], hi[2], hi[3]);
          st_shared_v4(dst + MH * 128, lo[0], lo[1], lo[2], lo[3]);
        }
      } else {
        uint4 w[OC / 8];
#pragma unroll
        for (int i = 0; i < OC / 8; ++i)
          w[i] = row < p.G ? reinterpret_cast<const uint4*>(src + o0)[i] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < OC / 8; ++i) {
          const int ch = o0 / 8 + i;
          st_shared_v4(smem_u32(sQ) + (ch / 8) * (MH * 128) + sw128_off(row, ch % 8), w[i].x, w[i].y, w[i].z, w[i].w);
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_ready);
      return c;
    };
    bool more = wk.next(p);
    float c = more ? load_q(wk.b * p.Hk + wk.hk) : 0.f;
    while (more) {
      float m_run = -INFINITY, l_run = 0.f, al = 1.f, be = 0.f;  // al, be: factors of the last tile's O
      float acc[OC];
#pragma unroll
      for (int k = 0; k < OC; ++k) acc[k] = 0.f;
      // acc = acc al + O be for the tile whose PV was issued last
      auto add_o = [&]() -> bool {
        if (!warp_wait(&o_full, jp & 1, limit, &abort_flag, p.st, 721)) return false;
        ++jp;
        tc_fence_after();
        const bool grown = __any_sync(0xffffffffu, al != 1.f);  // a row's maximum moved: rare after its first tiles
        float o[OC];
#pragma unroll
        for (int j = 0; j < NO; ++j) tmem_ld16x2_32<OC>(tq + tO + j * 32, *reinterpret_cast<float(*)[32]>(o + j * 32));
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < OC; k += 2) {
          if (grown) fmul2(acc[k], acc[k + 1], acc[k], acc[k + 1], al, al);
          ffma2(acc[k], acc[k + 1], o[k], o[k + 1], be, be, acc[k], acc[k + 1]);
        }
        tc_fence_before();
        return true;
      };
      const int first = wk.first_key(p), len = wk.len, cnt = wk.cnt, t_lo = wk.t0 + wk.off;
      const int pair = wk.b * p.Hk + wk.hk;
      const bool whole = wk.cnt == wk.n, begins = wk.off == 0;
      for (int i = 0; i < cnt; ++i) {
        const int key0 = (t_lo + i) * TILE;
        const int lo = max(first - key0, 0), hi = min(len - key0, TILE);  // visible keys of the tile
        if (!warp_wait(&s_full, js & 1, limit, &abort_flag, p.st, 720)) { ok = false; break; }
        ++js;
        float sv[SC];
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < NL; ++j) tmem_ld16x2_32<SC>(tq + tS + j * 32, *reinterpret_cast<float(*)[32]>(sv + j * 32));
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free);
        if (lo > 0 || hi < TILE) {
          const int a = lo - s0, b2 = hi - s0;
#pragma unroll
          for (int k = 0; k < SC; ++k) sv[k] = k >= a && k < b2 ? sv[k] : -INFINITY;
        }
        float rx[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
        for (int k = 4; k < SC; k += 8)
#pragma unroll
          for (int y = 0; y < 4; ++y) rx[y] = k + 4 < SC ? fmaxf(rx[y], fmaxf(sv[k + y], sv[k + 4 + y])) : fmaxf(rx[y], sv[k + y]);
        float rm = fmaxf(fmaxf(rx[0], rx[1]), fmaxf(rx[2], rx[3]));
        rm = fmaxf(rm, __shfl_xor_sync(0xffffffffu, rm, 16));
        const float mt = rm * c;
        const float neg = mt == -INFINITY ? 0.f : F8 ? 8.f - mt : -mt;
        float la = 0.f, lb = 0.f;
        // P -> shared memory, K-major, 16 bytes of codes as soon as they are there
        const uint32_t pb = smem_u32(sP) + (L::NB == 2 ? ((js - 1) & 1) * L::PB : 0);
        if (L::NB == 1 && i > 0 && !add_o()) { ok = false; break; }  // (the last product reads it)
        auto probabilities = [&](auto two_) {
          constexpr bool TT = decltype(two_)::value;
          constexpr int CK = F8 ? 16 : 8;  // keys of a chunk
#pragma unroll
          for (int k0 = 0; k0 < SC; k0 += CK) {
            uint32_t pk[TT ? CK : CK / 2];  // bf16 pairs, their rests; e4m3: hi codes of four keys, then lo codes
#pragma unroll
            for (int k = 0; k < CK; k += 4) {
              float e[4];
              const float* v = sv + k0 + k;
              ffma2(e[0], e[1], v[0], v[1], c, c, neg, neg);
              ffma2(e[2], e[3], v[2], v[3], c, c, neg, neg);
#pragma unroll
              for (int y = 0; y < 4; ++y) e[y] = fast_exp2(e[y]);
              fadd2(la, lb, la, lb, e[0], e[1]);
              fadd2(la, lb, la, lb, e[2], e[3]);
              if constexpr (F8) {
                uint32_t h0, l0, h1, l1;
                split_e4m3(pack_f16x2(e[0], e[1]), h0, l0);
                split_e4m3(pack_f16x2(e[2], e[3]), h1, l1);
                pk[k / 4] = h0 | (h1 << 16);
                pk[CK / 4 + k / 4] = l0 | (l1 << 16);
              } else {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  if constexpr (TT) {
                    // the first term cut off, not rounded: the rest is positive, and no zero (2^-126 at least), so that
                    // its product with an infinite value is that infinity again
                    const uint32_t h0 = __float_as_uint(e[2 * y]) & 0xFFFF0000u;
                    const uint32_t h1 = __float_as_uint(e[2 * y + 1]) & 0xFFFF0000u;
                    pk[k / 2 + y] = (h0 >> 16) | h1;
                    uint32_t r = pack_bf16x2(e[2 * y] - __uint_as_float(h0), e[2 * y + 1] - __uint_as_float(h1));
                    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(r) : "r"(0x00800080u));
                    pk[CK / 2 + k / 2 + y] = r;
                  } else {
                    pk[k / 2 + y] = pack_bf16x2(e[2 * y], e[2 * y + 1]);
                  }
                }
              }
            }
            const int ch = (s0 + k0) / CK;
            const uint32_t dst = pb + (ch / 8) * (MH * 128) + sw128_off(row, ch % 8);
            st_shared_v4(dst, pk[0], pk[1], pk[2], pk[3]);
            if constexpr (F8) st_shared_v4(dst + MH * 128, pk[4], pk[5], pk[6], pk[7]);
            if constexpr (TT) st_shared_v4(dst + L::P_BYTES, pk[4], pk[5], pk[6], pk[7]);
          }
        };
        if (two) probabilities(std::integral_constant<bool, L::TWO>{});
        else probabilities(std::false_type{});
        // the last tile's product before this tile's may overwrite it
        if (L::NB == 2 && i > 0 && !add_o()) { ok = false; break; }
        // factors of this tile's product
        const float mn = fmaxf(m_run, mt);
        al = m_run == mn ? 1.f : m_run == -INFINITY ? 0.f : fast_exp2(m_run - mn);
        be = mt == -INFINITY ? 0.f : (F8 ? 0.00390625f : 1.f) * fast_exp2(mt - mn);
        l_run = l_run * al + (la + lb) * be;
        m_run = mn;
        if (lo > 0 || hi < TILE) {
          // rows of V that no key is in may hold anything, and 0 times an infinity or a NaN is not 0
          const uint32_t vi = ring + (i == cnt - 1 ? 2 * cnt - 1 : 2 * i + 2);
          if (!warp_wait(&r_full[vi % NR], (vi / NR) & 1, limit, &abort_flag, p.st, 722)) { ok = false; break; }
          const uint32_t v = smem_u32(sR + (vi % NR) * SLOT);
          for (int ch = qd * 32 + lane; ch < SLOT / 16; ch += nact * 32) {
            const int r = (ch / 8) % TILE;
            if (r < lo || r >= hi) st_shared_v4(v + ch * 16, 0u, 0u, 0u, 0u);
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready);
      }
      if (!ok) break;
      ring += 2 * cnt;
      // the next pair's queries while the last product runs (its score products are done)
      more = wk.next(p);
      const float c_next = more ? load_q(wk.b * p.Hk + wk.hk) : 0.f;
      if (!add_o()) break;
      l_run += __shfl_xor_sync(0xffffffffu, l_run, 16);
      if (whole && row < p.G) {
        const size_t head = (size_t)pair * p.G + row;
        const float inv = l_run == 0.f ? 0.f : p.oscale / l_run;
        uint4* dst = reinterpret_cast<uint4*>(p.out + head * D + o0);
#pragma unroll
        for (int k = 0; k < OC; k += 8)
          dst[k / 8] = make_uint4(pack_bf16x2(acc[k] * inv, acc[k + 1] * inv), pack_bf16x2(acc[k + 2] * inv, acc[k + 3] * inv),
                                  pack_bf16x2(acc[k + 4] * inv, acc[k + 5] * inv),
                                  pack_bf16x2(acc[k + 6] * inv, acc[k + 7] * inv));
        if (p.lse && lh == 0) p.lse[head] = (m_run + log2f(l_run)) * 0.69314718055994531f;
      } else if (!whole) {
        if constexpr (CL) {  // the ring is done with: its last product has been read
          float4* dst = reinterpret_cast<float4*>(sR + row * L::REC + o0 * 4);
#pragma unroll
          for (int k = 0; k < OC; k += 4) dst[k / 4] = make_float4(acc[k], acc[k + 1], acc[k + 2], acc[k + 3]);
          if (lh == 0) reinterpret_cast<float2*>(sR + MH * L::REC)[row] = make_float2(m_run, l_run);
        } else {
          // a record: slot 1 where the segment begins its pair, else slot 0. 128 bytes of a row at a time, through
          // the warp's own rows of the two P buffers (a lane's 16 bytes of its row each cost a line: 2 us at the end)
          const size_t rec = (size_t)cta * 2 + (begins ? 1 : 0);
#pragma unroll
          for (int j = 0; j < NO; ++j) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<float4*>(sP + lh * L::P_BYTES + sw128_off(row, k)) =
                  make_float4(acc[j * 32 + 4 * k], acc[j * 32 + 4 * k + 1], acc[j * 32 + 4 * k + 2], acc[j * 32 + 4 * k + 3]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int h = i / 4, r = qd * 16 + (i % 4) * 4 + lane / 8, ch = lane % 8;
              const float4 v = *reinterpret_cast<const float4*>(sP + h * L::P_BYTES + sw128_off(r, ch));
              if (r < p.G) *reinterpret_cast<float4*>(p.po + (rec * p.G + r) * D + h * OC + j * 32 + ch * 4) = v;
            }
            __syncwarp();
          }
          if (row < p.G && lh == 0) p.pml[(size_t)row * (2 * p.W) + rec] = make_float2(m_run, l_run);
        }
      }
      c = c_next;
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) { tc_fence_after(); tmem_dealloc(tmem, 256); }
  if constexpr (CL) {
    if (split.W == 1) return;  // (of the whole cluster)
    __syncwarp();
    cluster_sync_all();  // every CTA's accumulators are in its shared memory
    // rows rank, rank + W, .. : a warp a row, every CTA's record of it asked for at once
    constexpr int VL = D / 32;
    const int rank = (int)cluster_ctarank();
    for (int row = rank + p.W * warp; row < p.G; row += p.W * (NT / 32)) {
      const uint32_t rec = smem_u32(sR) + row * L::REC + lane * (VL * 4), ml = smem_u32(sR) + MH * L::REC + row * 8;
      float o[MAX_CS][VL], m[MAX_CS], l[MAX_CS];
#pragma unroll
      for (int i = 0; i < MAX_CS; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int v = 0; v < VL; ++v) o[i][v] = 0.f;
        if (i < split.W) {
          const uint32_t ra = dsmem_addr(rec, i), ma = dsmem_addr(ml, i);
          m[i] = ld_dsmem_f32(ma);
          l[i] = ld_dsmem_f32(ma + 4);
          if constexpr (VL == 4) {
            const float4 x = ld_dsmem_v4(ra);
            o[i][0] = x.x; o[i][1] = x.y; o[i][2] = x.z; o[i][3] = x.w;
          } else {
            o[i][0] = ld_dsmem_f32(ra);
            o[i][1] = ld_dsmem_f32(ra + 4);
          }
        }
      }
      float M = m[0], acc[VL], ls = 0.f;
#pragma unroll
      for (int i = 1; i < MAX_CS; ++i) M = fmaxf(M, m[i]);
#pragma unroll
      for (int v = 0; v < VL; ++v) acc[v] = 0.f;
#pragma unroll
      for (int i = 0; i < MAX_CS; ++i) {
        const float w = m[i] == -INFINITY ? 0.f : fast_exp2(m[i] - M);
        ls += l[i] * w;
#pragma unroll
        for (int v = 0; v < VL; ++v) acc[v] += o[i][v] * w;
      }
      const size_t head = (size_t)(wk.b * p.Hk + wk.hk) * p.G + row;
      const float inv = ls == 0.f ? 0.f : p.oscale / ls;
      uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + head * D + lane * VL);
#pragma unroll
      for (int v = 0; v < VL; v += 2) dst[v / 2] = pack_bf16x2(acc[v] * inv, acc[v + 1] * inv);
      if (lane == 0 && p.lse) p.lse[head] = (M + log2f(ls)) * 0.69314718055994531f;
    }
    cluster_sync_all();  // nothing reads another CTA's memory after this
  }
}

// Joins the records of the (sequence, key head) pairs that several CTAs worked on, in the order of
// their ranges. A pair cut into cnt segments has cnt - 1 cuts inside it, and the JX blocks of each such cut share
// the pair's units, whole head rows or 32 columns of one (where there are more blocks than rows: one sequence of
// 256k tokens has 64 rows of 296 records), so all blocks have about as much to read however the line is
// cut. What bounds it is the chain of dependent reads, each a microsecond's third from L2: the main
// kernel leaves what a cut's blocks have to know in one 16-byte word, and a unit's maxima, sums and
// accumulators are asked for together. Warps that a block has to spare share a unit's records.
constexpr int JT = 256, JW = JT / 32, JX = 2;
// A unit: 4 LR columns of a head row; LR lanes read a record, 32 / LR records at a time.
template <int D, int LR>
__device__ __forceinline__ void join_units(const Params& p, int pair, int w0, int cnt, int first, int step,
                                           float (*s_acc)[D]) {
  constexpr int RPL = 32 / LR, C = D / (4 * LR), U = 4, ML = 5;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane / LR, li = lane % LR;
  const int units = p.G * C, mine = first < units ? (units - first + step - 1) / step : 0;
  const int split = mine >= 8 ? 1 : mine >= 4 ? 2 : mine >= 2 ? 4 : 8, sub = warp % split;
  for (int k0 = 0; k0 < mine; k0 += JW / split) {
    const int k = k0 + warp / split, unit = first + k * step, row = unit / C, col = (unit % C) * (4 * LR) + li * 4;
    const bool on = k < mine;
    // the first segment begins its pair (record 1 of its CTA), the others begin their CTA's range
    auto rec = [&](int i) { return (w0 + i) * 2 + (i == 0 ? 1 : 0); };
    const float2* ml = p.pml + (size_t)row * (2 * p.W);
    float acc[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f, M = -INFINITY;
    auto weight = [&](float x, float to) { return x == -INFINITY ? 0.f : fast_exp2(x - to); };
    if (on) {
      float4 o[U];
      float m[U];
      auto load = [&](int i0) {  // this lane's records i0, i0 + split * RPL, ..
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u * (split * RPL);
          m[u] = -INFINITY;
          o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i < cnt) {
            const int r = rec(i);
            o[u] = __ldcg(reinterpret_cast<const float4*>(p.po + ((size_t)r * p.G + row) * D + col));
            m[u] = __ldcg(&ml[r].x);
          }
        }
      };
      const int i_first = sub * RPL + g;
      load(i_first);
      // maxima and sums, ML records a lane at a time
      for (int i0 = lane; i0 - lane < cnt; i0 += 32 * ML) {
        float2 x[ML];
        float top = M;
#pragma unroll
        for (int j = 0; j < ML; ++j)
          x[j] = i0 + 32 * j < cnt ? __ldcg(ml + rec(i0 + 32 * j)) : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int j = 0; j < ML; ++j) top = fmaxf(top, x[j].x);
        l *= weight(M, top);
#pragma unroll
        for (int j = 0; j < ML; ++j) l += x[j].y * weight(x[j].x, top);
        M = top;
      }
      float top = M;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      l *= weight(M, top);
      M = top;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
      for (int i0 = i_first;;) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float w = weight(m[u], M);
          acc[0] += o[u].x * w; acc[1] += o[u].y * w; acc[2] += o[u].z * w; acc[3] += o[u].w * w;
        }
        i0 += U * split * RPL;
        if (i0 - g >= cnt) break;  // (the same for every lane)
        load(i0);
      }
#pragma unroll
      for (int d = 16; d >= LR; d >>= 1)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[v] += __shfl_xor_sync(0xffffffffu, acc[v], d);
    }
    if (split > 1) {
      __syncthreads();
      if (g == 0) *reinterpret_cast<float4*>(&s_acc[warp][li * 4]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      __syncthreads();
      if (sub == 0 && g == 0)
        for (int j = 1; j < split; ++j) {
          const float4 x = *reinterpret_cast<const float4*>(&s_acc[warp + j][li * 4]);
          acc[0] += x.x; acc[1] += x.y; acc[2] += x.z; acc[3] += x.w;
        }
    }
    if (on && sub == 0 && g == 0) {
      const size_t head = (size_t)pair * p.G + row;
      const float inv = l == 0.f ? 0.f : p.oscale / l;
      *reinterpret_cast<uint2*>(p.out + head * D + col) =
          make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
      if (col == 0 && p.lse) p.lse[head] = (M + log2f(l)) * 0.69314718055994531f;
    }
  }
}
template <int D>
__global__ void __launch_bounds__(JT, 4) paged_join_kernel(Params p) {
  __shared__ __align__(16) float s_acc[JW][D];
  const int cut = blockIdx.x + 1;
  griddep_wait();
  griddep_launch_dependents();
  const int4 c = __ldcg(p.cuts + cut);
  const int pair = c.x, w0 = c.y, cnt = c.z;
  if (cnt == 0) return;  // not between two tiles of a pair
  const int step = JX * (cnt - 1), first = (cut - w0 - 1) * JX + blockIdx.y;
  if (step > 2 * p.G) join_units<D, 8>(p, pair, w0, cnt, first, step, s_acc);
  else join_units<D, D / 4>(p, pair, w0, cnt, first, step, s_acc);
}

// -------------------------------------------------------------------------------------- host
constexpr size_t kStatusBytes = 256;
static size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

static size_t carve(Params* p, void* ws, int G, int D, int W) {
  uint8_t* base = (uint8_t*)ws;
  size_t off = kStatusBytes;
  if (p) { p->st = (DevStatus*)base; p->cuts = (int4*)(base + off); }
  off = up256(off + (size_t)W * sizeof(int4));
  if (p) p->pml = (float2*)(base + off);
  off = up256(off + (size_t)W * 2 * G * sizeof(float2));
  if (p) p->po = (float*)(base + off);
  return up256(off + (size_t)W * 2 * G * D * sizeof(float));
}

static int gcd(int a, int b) { return b == 0 ? a : gcd(b, a % b); }

template <int D, bool F8>
static cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const Params& p, cudaStream_t st) {
  using L = Lay<D, F8, false>;
  const auto k = paged_attn_kernel<D, F8, false>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
  if (e != cudaSuccess) return e;
  {
    LaunchScope ls("paged_attn", st);
    e = launch_k(k, dim3(p.W), dim3(NT), L::BYTES, st, true, tk, tv, p);
  }
  if (e != cudaSuccess || p.W == 1) return e;
  LaunchScope ls("paged_join", st);
  return launch_k(paged_join_kernel<D>, dim3(p.W - 1, JX), dim3(JT), 0, st, true, p);
}
template <int D, bool F8>
static cudaError_t launch_clusters(const CUtensorMap& tk, const CUtensorMap& tv, const Params& p, cudaStream_t st) {
  using L = Lay<D, F8, true>;
  const auto k = paged_attn_kernel<D, F8, true>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
  if (e != cudaSuccess) return e;
  LaunchScope ls("paged_attn_cluster", st);
  return launch_clusters_k(k, dim3(p.B * p.Hk * p.W), dim3(NT), L::BYTES, st, true, p.W, tk, tv, p);
}

// CTAs of a cluster for `pairs` (sequence, key head) of at most n tiles each; 0: the line of tiles.
// n comes from the page table's width (and the window): the lengths are on the device, so short sequences in a table for
// long ones take the line (one of 1,000 tokens 11.3 us instead of 8.9, in e4m3 12.2 instead of 9.0).
// Clusters spare the records and the second kernel, about five tiles' time, but share a pair's tiles among 8
// CTAs at most, and a ragged batch's short pairs leave theirs idle (three quarters of the line's share
// is what a batch of mixed lengths has to gain by). Measured, clusters and line: 64 heads on one key head, one
// sequence of 1,000 tokens 8.3 and 10.8 us, of 4,096 13.3 and 10.5 us; 250 sequences of up to 1,000 tokens 21 and
// 27 us, 16 of 8,192 24 and 21 us. Clusters of 16 gain nothing where these lose, and 16 of them take two waves.
static int cluster_size(long long pairs, long long n, int sms) {
  if (pairs > 2 * sms) return 0;
  int cs = MAX_CS;
  while (cs > 1 && (pairs * cs > 2 * sms || cs / 2 >= n)) cs /= 2;
  const long long share = pairs * (n + OV) / (2 * sms);
  return 4 * n <= cs * (20 + 3 * share) ? cs : 0;
}

}  // namespace pattn
}  // namespace hs2

using namespace hs2;

extern "C" {

static bool pattn_sizes_ok(int B, int Hq, int Hk) {
  return B >= 0 && Hk >= 1 && Hq >= Hk && Hq % Hk == 0 && (long long)B * Hq <= 0x3FFFFFFFll;
}

size_t hs2_paged_attn_workspace_bytes(int B, int Hq, int Hk, int d) {
  if (!pattn_sizes_ok(B, Hq, Hk) || Hq / Hk > pattn::MH || (d != 64 && d != 128)) return 0;
  const int sms = num_sms() > 0 ? num_sms() : 148;
  return pattn::carve(nullptr, nullptr, Hq / Hk, d, 2 * sms);
}

hs2_status hs2_paged_attn(const hs2_bf16* Q, const void* K_pages, const void* V_pages, const long long* k_page_strides,
                          const long long* v_page_strides, int n_pages, int page_size, const int32_t* page_table,
                          int max_pages, const int32_t* lens, int B, int Hq, int Hk, int d, int e4m3, float k_scale,
                          float v_scale, float scale, int window, hs2_bf16* out, float* lse, void* workspace,
                          size_t workspace_bytes, hs2_stream stream) {
  if (!pattn_sizes_ok(B, Hq, Hk) || !K_pages || !V_pages || !k_page_strides || !v_page_strides ||
      (B > 0 && (!Q || !page_table || !lens || !out)) || n_pages < 1 || page_size < 1 || max_pages < 1 || window < 0 ||
      (long long)max_pages * page_size > 0x3FFFFFFFll || !(scale > 0.f && scale < INFINITY) || !aligned16(Q) ||
      !aligned16(K_pages) || !aligned16(V_pages) || !aligned16(out))
    return HS2_ERR_INVALID_ARG;
  if (!pool_strides_ok(k_page_strides, e4m3) || !pool_strides_ok(v_page_strides, e4m3)) return HS2_ERR_INVALID_ARG;
  if (e4m3 && !(cache_scale_ok(k_scale) && cache_scale_ok(v_scale))) return HS2_ERR_INVALID_ARG;
  const int G = Hq / Hk;
  if (G > pattn::MH || page_size % 16 != 0 || (d != 128 && (d != 64 || e4m3)) || !device_is_sm100())
    return HS2_ERR_UNSUPPORTED_SHAPE;
  if (!workspace || !aligned16(workspace) || workspace_bytes < hs2_paged_attn_workspace_bytes(B, Hq, Hk, d))
    return HS2_ERR_WORKSPACE;
  if (B == 0) return HS2_OK;
  const int tile = e4m3 || d == 64 ? 128 : 64;
  pattn::Params p{};
  p.q = (const __nv_bfloat16*)Q; p.out = (__nv_bfloat16*)out; p.lse = lse;
  p.ptab = page_table; p.lens = lens;
  p.B = B; p.Hk = Hk; p.G = G; p.page = page_size; p.box = pattn::gcd(page_size, tile);
  p.max_pages = max_pages; p.n_pages = n_pages; p.window = window;
  p.c = scale * 1.4426950408889634f * (e4m3 ? k_scale : 1.f);
  p.oscale = e4m3 ? v_scale : 1.f;
  p.wait_ns = wait_limit_ns();
  // tiles that the batch can have at most: one line of 32-bit tile numbers
  const long long span = (long long)max_pages * page_size;
  const long long n_max = window > 0 && window < span ? (window - 1) / tile + 2 : (span + tile - 1) / tile;  // of one pair
  const long long most = (long long)B * Hk * (n_max + pattn::OV);
  if (most > 0x3FFFFFFFll) return HS2_ERR_UNSUPPORTED_SHAPE;
  p.W = 2 * num_sms();
  pattn::carve(&p, workspace, G, d, p.W);
  const int cs = pattn::cluster_size((long long)B * Hk, n_max, num_sms());
  if (cs > 0) p.W = cs;
  else if (most < p.W) p.W = (int)most;
  CUtensorMap tk, tv;
  if (!make_tmap_pool(&tk, K_pages, d, page_size, Hk, n_pages, k_page_strides[0], k_page_strides[1], k_page_strides[2],
                      p.box, e4m3 != 0) ||
      !make_tmap_pool(&tv, V_pages, d, page_size, Hk, n_pages, v_page_strides[0], v_page_strides[1], v_page_strides[2],
                      p.box, e4m3 != 0))
    return HS2_ERR_CUDA;
  const cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  if (cs > 0)
    e = e4m3 ? pattn::launch_clusters<128, true>(tk, tv, p, st)
             : d == 128 ? pattn::launch_clusters<128, false>(tk, tv, p, st) : pattn::launch_clusters<64, false>(tk, tv, p, st);
  else
    e = e4m3 ? pattn::launch<128, true>(tk, tv, p, st)
             : d == 128 ? pattn::launch<128, false>(tk, tv, p, st) : pattn::launch<64, false>(tk, tv, p, st);
  return e == cudaSuccess ? HS2_OK : HS2_ERR_CUDA;
}

}  // extern "C"
