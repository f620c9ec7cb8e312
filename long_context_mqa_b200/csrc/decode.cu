// Decode step of the full-attention + selection layer (one query token per sequence, the
// query at position t = N_b - 1 of sequence b's N_b-token K/V cache; the N_b may differ), as one
// persistent kernel.
//
// The score of a key is sum_h p_h = sum_h exp(s_h - lse_h): each head's logsumexp over the whole
// row is needed before any score is final. Instead of a full first pass over K for it, phase 1
// estimates it from a sample of the tiles, phase 2 streams K and V once against that reference,
// and the selection is made exact with bounds and a re-score of the few keys near the threshold:
//
//   phase 1  every st-th tile of each sequence (about 64 tiles), K only.
//            S^T = K_tile Q^T on tcgen05 (M = 128 keys in TMEM lanes, N = 64 heads); the two
//            softmax warpgroups split the heads (32 each); every thread owns one key lane and
//            keeps, per head, a reference r and a sum l of exp2(s*c - r) (r moves only when a
//            value exceeds it by 2^64); one reduce-scatter merge per segment -> (m, l) records.
//   grid barrier (bounded).
//   phase 2  K and V, each CTA's range backwards. The sequence's sampled lse2' per head from all
//            its records; S^T again; p' = exp2(s*c - lse2') (no rescaling, p' >= p); the head
//            sum score' is an in-thread reduction; P'^T (bf16) goes to shared memory as an
//            MN-major operand and O'^T += V^T P'^T accumulates in TMEM; a warp reduce-scatter of
//            p' accumulates the per-head totals L'_h = sum_j p'_jh. Scores go to a global buffer
//            and a 2048-bin histogram of their bits 30..20. The two warpgroups take alternate
//            tiles.
//   tail     the last CTA to finish a sequence forms the exact lse = lse2' + log2 L' (out is
//            sum O' / L' in the combine), and since score = sum_h p'_h / L'_h lies within
//            [score' / max L', score' / min L'], it turns the bin of the k-th score' into a bin
//            above which keys are certainly selected and one below which they certainly are
//            not. select.cu collects the band between them, re-scores it exactly and selects.
//
// A sequence whose p' reaches 2^64 (a key far more probable than everything sampled) is flagged
// and redone with every tile (the reference is then the exact lse) by a second
// launch of this kernel, which leaves at once when nothing is flagged.
//
// The grid is one CTA per SM, launched cooperatively (all CTAs co-resident). Warp roles
// (320 threads): warp 0 = TMA producer (Q per segment; K and V tiles through one 5-slot ring,
// in the order the tensor core consumes them), warp 1 = tcgen05 issuer and TMEM owner,
// warps 2..5 and 6..9 = softmax warpgroups 0 and 1 (warp w reads TMEM lanes 32*(w%4)..+31).
// Every wait is bounded; on timeout the kernel records it in the status word and unwinds with
// its barrier sequence intact.
//
// FP8 cache (F8, 448 threads): K and V arrive as e4m3 tiles (16 KB, half the bytes) through an
// 8-slot ring, and a fourth warpgroup (warps 10..13) widens them exactly to f16: a K row into
// TMEM, where the S MMA reads its A operand (each thread writes its own key's row: lane = key),
// a V row into the f16 tile in shared memory that the next PV MMA reads; it also rewrites each
// segment's query in place as f16, and P is packed as f16, so every MMA is f16 x f16 with fp32
// accumulation. The softmax warps keep each row's p' per head in TMEM and sum the rows once per
// segment. The cache's scales are folded into the logit factor c and the output combine. f16 P
// holds values below 65504: the references are offset (p' = 4 p'' in the sampled pass, 2^12 p in
// the exact redo, both cancelling in O / L') and a key whose head sum passes 65504 is flagged
// for the redo.
#include "decode.h"
#include "host_util.h"
#include "tc.cuh"

namespace hs2 {
namespace dec {

constexpr int TILE = 128;
constexpr int NTHREADS = 320;     // bf16 cache
constexpr int NTHREADS_F8 = 448;  // FP8 cache: + a warpgroup that widens the e4m3 tiles
constexpr int CONV_WARP0 = 10;    // its first warp
constexpr int SM_WG0 = 2;  // first warp of softmax warpgroup 0
constexpr int RING = 5;    // K/V tile slots
constexpr int RING8 = 8;   // e4m3 K/V tile slots (FP8 cache)
constexpr float F8_MAX_SCORE = 65504.f;  // largest f16: a bound on each p' of a key
constexpr float F8_OFF_SAMPLED = 2.f;    // log2 offsets of the p' reference (FP8 cache)
constexpr float F8_OFF_EXACT = 12.f;
constexpr int NBINS = 2048;
constexpr float REF_SLACK = 64.f;

__device__ __forceinline__ void named_bar(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// bounded wait that also gives up when another role already aborted
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
// Warp-collective form: every lane gets the same answer, so the warp-synchronous tcgen05.ld that
// follows is never reached by only part of the warp. A phase that has already completed is seen
// by all lanes at once, without a divergent branch (the FP8 kernel's widening warps wait on two
// barriers per ring item: 2.7% off its time); otherwise lane 0 waits, bounded, and passes it on.
__device__ __forceinline__ bool warp_wait_bar(uint64_t* bar, uint32_t parity, long long limit,
                                              volatile int* abort_flag, DevStatus* st, unsigned where) {
  if (__all_sync(0xffffffffu, mbar_try_wait(smem_u32(bar), parity))) return true;
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = wait_bar(bar, parity, limit, abort_flag, st, where) ? 1 : 0;
  ok = __shfl_sync(0xffffffffu, ok, 0);
  return ok != 0;
}
// (m, l) <- merge of two (max, sum of exp2(x - max)) pairs
__device__ __forceinline__ void merge_ml(float& m, float& l, float m2, float l2) {
  const float mx = fmaxf(m, m2);
  const float a1 = m == -INFINITY ? 0.f : fast_exp2(m - mx);
  const float a2 = m2 == -INFINITY ? 0.f : fast_exp2(m2 - mx);
  l = l * a1 + l2 * a2;
  m = mx;
}

// Page ids of a run of n tiles lt0, lt0 + step, ... of sequence b from a page table
// [B][max_pages] (a contiguous cache: no table, every id -1). Each id is read 4 tiles before the
// producer needs it, so the table's latency hides behind the ring's waits.
struct PageRun {
  const int32_t* row;
  int lt, step, left, v0, v1, v2, v3;
  __device__ __forceinline__ int load(int k) const {
    return row && k < left ? row[lt + k * step] : -1;
  }
  __device__ __forceinline__ void start(const int32_t* ptab, int max_pages, int b, int lt0, int st, int n) {
    row = ptab ? ptab + (size_t)b * max_pages : nullptr;
    lt = lt0; step = st; left = n;
    v0 = load(0); v1 = load(1); v2 = load(2); v3 = load(3);
  }
  __device__ __forceinline__ int next() {
    const int r = v0;
    v0 = v1; v1 = v2; v2 = v3;
    v3 = load(4);
    lt += step;
    --left;
    return r;
  }
};

// the first phase-1 (sampled) tile at or after local tile lt
__device__ __forceinline__ int first_sample(int lt, int st) { return (lt + st - 1) / st * st; }
// phase 1 of sequence b takes every st-th tile: about `target` tiles (every tile when target is
// 0), and at most an eighth of the sequence's tiles (at least 4): a short sequence of a ragged
// batch sampled in full would give the CTAs covering it most of the first pass while every other
// CTA waits at the grid barrier
__device__ __forceinline__ int sample_stride(const Sched& S, int b, int target) {
  const int tiles = (int)(S.seq_start[b + 1] - S.seq_start[b]);
  if (target > 0 && target > tiles / 8) target = tiles / 8 > 4 ? tiles / 8 : 4;
  return target > 0 && tiles / target > 1 ? tiles / target : 1;
}

template <int H, int D, bool F8>
__global__ void __launch_bounds__(F8 ? NTHREADS_F8 : NTHREADS, 1)
    dec_fused_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmQ, DecParams p) {
  static_assert(H == 64 && D == 128, "the decode kernel is instantiated for 64 heads x 128");
  constexpr int KT_BYTES = TILE * D * 2;
  constexpr int Q_BYTES = H * D * 2;
  constexpr int P_BYTES = TILE * H * 2;
  constexpr int NKB = D / 64;
  constexpr int HW = H / 2;  // heads per warpgroup in phase 1
  constexpr int NR = F8 ? RING8 : RING;                // ring slots
  constexpr int SLOT_BYTES = F8 ? TILE * D : KT_BYTES;  // one K or V tile as it arrives
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sQ = smem;                     // Q of the current segment
  uint8_t* sR = sQ + Q_BYTES;             // NR tiles (K or V)
  uint8_t* sV = sR + NR * SLOT_BYTES;     // FP8 cache: the f16 V tile of the next PV
  uint8_t* sP = sV + (F8 ? KT_BYTES : 0);  // P^T of warpgroup 0 / 1
  uint32_t* shist = (uint32_t*)(sP + 2 * P_BYTES);
  __shared__ __align__(8) uint64_t r_full[NR], r_empty[NR], s_full[2], s_empty[2], p_full[2], p_empty[2], q_full,
      q_empty, o_full, o_empty;
  // FP8 cache: the f16 K rows in TMEM and the f16 V tiles (filled by the widening warps,
  // emptied by the S and PV MMAs) and the query rewritten as f16
  __shared__ __align__(8) uint64_t ka_full[2], ka_empty[2], v16_full, v16_empty, q16_full;
  __shared__ uint32_t tmem_base;
  __shared__ volatile int abort_flag;
  __shared__ __align__(16) float slse[H];
  __shared__ __align__(16) float red[8][H][2];  // merge scratch (phase-1 view: [2][4][HW][2])
  __shared__ int s_last;
  __shared__ unsigned s_wtot[8];
  __shared__ unsigned s_cnt2[8][2];
  __shared__ float s_lmm[2][2];
  __shared__ int s_band[3];

  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;
  const Sched& S = p.sch;  // in parameter space (its start table is indexed at run time)
  const long long limit = p.wait_ns;
  const uint32_t tS = 0, tO = 2 * H;  // TMEM columns: S buffers 0..2H-1, O^T 2H..3H-1
  constexpr uint32_t tKA = 256;       // FP8 cache: f16 K tiles 256..319, 320..383 (D / 2 columns each)
  constexpr uint32_t tLA = 384;       // FP8 cache: per-row sums of p' of warpgroup 0 / 1 (H columns each)
  constexpr uint32_t TMEM_COLS = F8 ? 512 : 256;
  // launched as a programmatic dependent: nothing before this point touches global memory
  griddep_wait();
  // the exact redo runs only if the sampled launch before it flagged a sequence (every CTA reads
  // the same final count, so the whole grid leaves together, before any barrier)
  if (p.fallback && *(volatile const int*)&p.ovf[p.B] == 0) return;
  // in the redo, only flagged sequences are processed (every role skips the same segments)
  auto skip_seq = [&](int b) -> bool { return p.fallback && *(volatile const int*)&p.ovf[b] == 0; };

  for (int i = threadIdx.x; i < NBINS; i += (F8 ? NTHREADS_F8 : NTHREADS)) shist[i] = 0;
  if (threadIdx.x == 0) {
    // FP8 cache: a slot is released by the 4 widening warps; bf16: by the MMA that read it
    for (int i = 0; i < NR; ++i) { mbar_init(&r_full[i], 1); mbar_init(&r_empty[i], F8 ? 4 : 1); }
    if (F8) {
      for (int i = 0; i < 2; ++i) { mbar_init(&ka_full[i], 4); mbar_init(&ka_empty[i], 1); }
      mbar_init(&v16_full, 4); mbar_init(&v16_empty, 1);
      mbar_init(&q16_full, 4);
    }
    for (int i = 0; i < 2; ++i) {
      // phase 1: all 8 softmax warps release an S buffer; phase 2: the 4 warps of its owner, x2
      mbar_init(&s_full[i], 1); mbar_init(&s_empty[i], 8);
      mbar_init(&p_full[i], 4); mbar_init(&p_empty[i], 1);
    }
    mbar_init(&q_full, 1); mbar_init(&q_empty, 1);
    mbar_init(&o_full, 1); mbar_init(&o_empty, 4);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) { tmem_alloc(&tmem_base, TMEM_COLS); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      tma_prefetch_desc(&tmK); tma_prefetch_desc(&tmV); tma_prefetch_desc(&tmQ);
      const uint64_t keep = policy_evict_last(), once = policy_evict_first();
      uint32_t ri = 0, nq = 0;
      bool ok = true;
      auto load_q = [&](int b) -> bool {
        if (!wait_bar(&q_empty, (nq & 1) ^ 1, limit, &abort_flag, p.st, 201)) return false;
        mbar_expect_tx(&q_full, Q_BYTES);
        for (int kb = 0; kb < NKB; ++kb) tma_load_3d(sQ + kb * (H * 128), &tmQ, &q_full, kb * 64, 0, b);
        ++nq;
        return true;
      };
      // tile lt of sequence b: rows lt*128.. of its cache, or (paged cache) page `pg`, whose 128
      // rows are the third tensor-map coordinate's slice (an id outside the pool reads zeros)
      auto load_tile = [&](const CUtensorMap* m, int lt, int b, uint64_t pol, int pg) -> bool {
        const int s = ri % NR;
        if (!wait_bar(&r_empty[s], ((ri / NR) & 1) ^ 1, limit, &abort_flag, p.st, 202)) return false;
        mbar_expect_tx(&r_full[s], SLOT_BYTES);
        if (p.ptab && (pg < 0 || pg >= p.n_pages)) report_status(p.st, kStatusBounds, 203);  // reads zeros
        const int c1 = p.ptab ? 0 : lt * TILE, c2 = p.ptab ? pg : b;
        if constexpr (F8) {  // one 128-byte row per key: a single swizzled box
          tma_load_3d_hint(sR + s * SLOT_BYTES, m, &r_full[s], 0, c1, c2, pol);
        } else {
          for (int kb = 0; kb < NKB; ++kb)
            tma_load_3d_hint(sR + s * KT_BYTES + kb * (TILE * 128), m, &r_full[s], kb * 64, c1, c2, pol);
        }
        ++ri;
        return true;
      };
      // page ids of a run of tiles lt0, lt0 + step, ... (count n), read 4 ahead of their use
      PageRun pr;
      for (int g = 0; g < S.n_groups && ok; ++g) {
        long long t0, t1;
        S.range(g, cta, t0, t1);
        for (long long t = t0; t < t1 && ok;) {  // phase 1: K, ascending
          const int b = S.seq_of(t);
          const long long seg_end = t1 < (long long)S.seq_start[b + 1] ? t1 : (long long)S.seq_start[b + 1];
          if (skip_seq(b)) { t = seg_end; continue; }
          if (!load_q(b)) { ok = false; break; }
          const int st = sample_stride(S, b, p.sample_tiles), lt_hi = (int)(seg_end - (long long)S.seq_start[b]);
          const int lt0 = first_sample((int)(t - (long long)S.seq_start[b]), st);
          pr.start(p.ptab, p.max_pages, b, lt0, st, lt0 < lt_hi ? (lt_hi - 1 - lt0) / st + 1 : 0);
          for (int lt = lt0; lt < lt_hi && ok; lt += st)
            if (!load_tile(&tmK, lt, b, keep, pr.next())) ok = false;
          t = seg_end;
        }
        for (long long t = t1 - 1; t >= t0 && ok;) {  // phase 2: descending
          const int b = S.seq_of(t);
          const long long seg_lo = t0 > (long long)S.seq_start[b] ? t0 : (long long)S.seq_start[b];
          if (skip_seq(b)) { t = seg_lo - 1; continue; }
          if (!load_q(b)) { ok = false; break; }
          // in the order the tensor core consumes them: S of a tile needs its K, then the PV of
          // the tile before it (the next higher one) needs that tile's V
          const long long seg_hi = t;
          pr.start(p.ptab, p.max_pages, b, (int)(seg_hi - (long long)S.seq_start[b]), -1, (int)(seg_hi - seg_lo + 1));
          int pg_prev = -1;  // the page of tile lt + 1 (its V follows this tile's K)
          for (; t >= seg_lo; --t) {
            const int lt = (int)(t - (long long)S.seq_start[b]);
            const int pg = pr.next();
            if (!load_tile(&tmK, lt, b, once, pg)) { ok = false; break; }
            if (t < seg_hi && !load_tile(&tmV, lt + 1, b, once, pg_prev)) { ok = false; break; }
            pg_prev = pg;
          }
          if (ok && !load_tile(&tmV, (int)(seg_lo - (long long)S.seq_start[b]), b, once, pg_prev)) { ok = false; break; }
        }
      }
      if (!ok) {  // let the copies already issued land before the CTA exits
        for (uint32_t x = (ri > NR ? ri - NR : 0); x < ri; ++x) mbar_wait(&r_full[x % NR], (x / NR) & 1, limit);
        if (nq > 0) mbar_wait(&q_full, (nq - 1) & 1, limit);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ tcgen05 issuer
    if (lane == 0) {
      constexpr uint32_t IDESC_S = F8 ? idesc_f16(128, H, 0, 0) : idesc_bf16(128, H, 0, 0);
      constexpr uint32_t IDESC_O = F8 ? idesc_f16(D, H, 1, 1) : idesc_bf16(D, H, 1, 1);
      uint64_t* const qready = F8 ? &q16_full : &q_full;  // the query as the MMAs read it
      // js counts S tiles (the TMEM S buffer is js & 1), jp phase-2 tiles (their P buffer / owner)
      uint32_t ri = 0, js = 0, jp = 0, nq = 0, seg2 = 0;
      uint32_t npu[2] = {0, 0};  // PV uses of each P buffer
      uint32_t npv = 0;          // PVs issued (FP8 cache: uses of the f16 V buffer)
      bool ok = true;
      auto issue_s = [&](uint32_t kidx) -> bool {
        const int s = kidx % NR, buf = js & 1;
        if constexpr (F8) {  // the tile's f16 K rows, written to TMEM by the softmax warps
          if (!wait_bar(&ka_full[buf], (js >> 1) & 1, limit, &abort_flag, p.st, 217)) return false;
        } else {
          if (!wait_bar(&r_full[s], (kidx / NR) & 1, limit, &abort_flag, p.st, 211)) return false;
        }
        if (!wait_bar(&s_empty[buf], ((js >> 1) & 1) ^ 1, limit, &abort_flag, p.st, 212)) return false;
        tc_fence_after();
        const uint64_t qa = sdesc(smem_u32(sQ), 16, 1024);
        if constexpr (F8) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t bq = sdesc_at(qa, (kk / 4) * (H * 128) + (kk % 4) * 32);
            umma_ts(tmem + tS + buf * H, tmem + tKA + buf * (D / 2) + kk * 8, bq, IDESC_S, kk > 0);
          }
          umma_commit(&s_full[buf]);
          umma_commit(&ka_empty[buf]);
        } else {
          const uint64_t ka = sdesc(smem_u32(sR + s * KT_BYTES), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t a = sdesc_at(ka, (kk / 4) * (TILE * 128) + (kk % 4) * 32);
            const uint64_t bq = sdesc_at(qa, (kk / 4) * (H * 128) + (kk % 4) * 32);
            umma_ss(tmem + tS + buf * H, a, bq, IDESC_S, kk > 0);
          }
          umma_commit(&s_full[buf]);
          umma_commit(&r_empty[s]);
        }
        ++js;
        return true;
      };
      auto issue_pv = [&](uint32_t jj, uint32_t vidx, bool first) -> bool {
        const int buf = jj & 1, s = vidx % NR;
        if (!wait_bar(&p_full[buf], npu[buf] & 1, limit, &abort_flag, p.st, 214)) return false;
        if constexpr (F8) {  // the tile's f16 V (one buffer: one use per PV)
          if (!wait_bar(&v16_full, npv & 1, limit, &abort_flag, p.st, 218)) return false;
        } else {
          if (!wait_bar(&r_full[s], (vidx / NR) & 1, limit, &abort_flag, p.st, 215)) return false;
        }
        if (first && !wait_bar(&o_empty, (seg2 & 1) ^ 1, limit, &abort_flag, p.st, 216)) return false;
        tc_fence_after();
        const uint64_t va = sdesc(smem_u32(F8 ? sV : sR + s * KT_BYTES), TILE * 128, 1024);
        const uint64_t pa = sdesc(smem_u32(sP + buf * P_BYTES), TILE * 128, 1024);
#pragma unroll
        for (int kk = 0; kk < TILE / 16; ++kk) {
          const uint64_t a = sdesc_at(va, kk * 2048);
          const uint64_t bb = sdesc_at(pa, kk * 2048);
          umma_ss(tmem + tO, a, bb, IDESC_O, (first && kk == 0) ? 0u : 1u);
        }
        umma_commit(&p_empty[buf]);
        umma_commit(F8 ? &v16_empty : &r_empty[s]);
        npu[buf]++;
        ++npv;
        return true;
      };
      for (int g = 0; g < S.n_groups && ok; ++g) {
        long long t0, t1;
        S.range(g, cta, t0, t1);
        for (long long t = t0; t < t1 && ok;) {  // phase 1
          const int b = S.seq_of(t);
          const long long seg_end = t1 < (long long)S.seq_start[b + 1] ? t1 : (long long)S.seq_start[b + 1];
          if (skip_seq(b)) { t = seg_end; continue; }
          if (!wait_bar(qready, nq & 1, limit, &abort_flag, p.st, 210)) { ok = false; break; }
          const int st = sample_stride(S, b, p.sample_tiles), lt_hi = (int)(seg_end - (long long)S.seq_start[b]);
          for (int lt = first_sample((int)(t - (long long)S.seq_start[b]), st); lt < lt_hi && ok; lt += st)
            if (!issue_s(ri++)) ok = false;
          t = seg_end;
          if (!ok) break;
          umma_commit(&q_empty);
          ++nq;
        }
        for (long long t = t1 - 1; t >= t0 && ok;) {  // phase 2
          const int b = S.seq_of(t);
          const long long seg_lo = t0 > (long long)S.seq_start[b] ? t0 : (long long)S.seq_start[b];
          if (skip_seq(b)) { t = seg_lo - 1; continue; }
          const uint32_t n = (uint32_t)(t - seg_lo + 1), base = ri;
          // S of a tile, then PV of the tile before it
          if (!wait_bar(qready, nq & 1, limit, &abort_flag, p.st, 213)) { ok = false; break; }
          for (uint32_t x = 0; x < n; ++x, ++jp) {
            if (!issue_s(base + (x == 0 ? 0u : 2 * x - 1))) { ok = false; break; }
            if (x > 0 && !issue_pv(jp - 1, base + 2 * x, x == 1)) { ok = false; break; }
          }
          if (!ok) break;
          umma_commit(&q_empty);
          ++nq;
          if (!issue_pv(jp - 1, base + 2 * n - 1, n == 1)) { ok = false; break; }
          umma_commit(&o_full);
          ++seg2;
          ri = base + 2 * n;
          t = seg_lo - 1;
        }
      }
    }
  } else if (F8 && warp >= CONV_WARP0) {
    // ------------------------------------------------------------------ e4m3 widening (FP8 cache)
    // Takes every ring item in order: the query of a segment (rewritten in place as f16), a K
    // tile (each thread its key row, f16, into the TMEM buffer of the tile's S MMA), a V tile
    // (each thread its key row into the f16 V buffer of the tile's PV MMA, zeros past the
    // sequence). It runs up to two tiles ahead of the MMAs, bounded by those buffers.
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;                 // key within the tile == TMEM lane
    const int ctid = (warp - CONV_WARP0) * 32 + lane;    // 0..127
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    uint32_t ri = 0, js = 0, jp = 0, nq = 0;
    uint32_t nv = 0;  // V tiles widened into the f16 buffer
    bool ok = true;
    auto widen_q = [&]() -> bool {
      if (!warp_wait_bar(&q_full, nq & 1, limit, &abort_flag, p.st, 226)) return false;
      for (int i = ctid; i < Q_BYTES / 16; i += 128) {
        const uint32_t a = smem_u32(sQ) + i * 16;
        const uint4 w = ld_shared_v4(a);
        st_shared_v4(a, bf16x2_to_f16x2(w.x), bf16x2_to_f16x2(w.y), bf16x2_to_f16x2(w.z), bf16x2_to_f16x2(w.w));
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q16_full);
      return true;
    };
    auto widen_k = [&](uint32_t item, uint32_t jsx) -> bool {
      const int slot = (int)(item % NR), kb = (int)(jsx & 1);
      if (!warp_wait_bar(&r_full[slot], (item / NR) & 1, limit, &abort_flag, p.st, 227)) return false;
      if (!warp_wait_bar(&ka_empty[kb], ((jsx >> 1) & 1) ^ 1, limit, &abort_flag, p.st, 228)) return false;
      tc_fence_after();
      const uint32_t src = smem_u32(sR + slot * SLOT_BYTES);
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        uint32_t w[32];
#pragma unroll
        for (int c4 = 0; c4 < 4; ++c4) {
          const uint4 x = ld_shared_v4(src + sw128_off(row, hh * 4 + c4));
          e4m3x4_to_f16x4(x.x, w[c4 * 8 + 0], w[c4 * 8 + 1]);
          e4m3x4_to_f16x4(x.y, w[c4 * 8 + 2], w[c4 * 8 + 3]);
          e4m3x4_to_f16x4(x.z, w[c4 * 8 + 4], w[c4 * 8 + 5]);
          e4m3x4_to_f16x4(x.w, w[c4 * 8 + 6], w[c4 * 8 + 7]);
        }
        tmem_st32(tmem + lane_base + tKA + kb * (D / 2) + hh * 32, w);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) { mbar_arrive(&ka_full[kb]); mbar_arrive(&r_empty[slot]); }
      return true;
    };
    // a V tile in two steps: the row's 8 chunks into registers (the e4m3 slot is then free), and
    // later, once the previous PV has read the f16 buffer, widened into it
    auto load_v = [&](uint32_t item, bool valid_row, uint4 (&x)[D / 16]) -> bool {
      const int slot = (int)(item % NR);
      if (!warp_wait_bar(&r_full[slot], (item / NR) & 1, limit, &abort_flag, p.st, 229)) return false;
      const uint32_t src = smem_u32(sR + slot * SLOT_BYTES);
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
        x[c] = valid_row ? ld_shared_v4(src + sw128_off(row, c)) : make_uint4(0u, 0u, 0u, 0u);
      __syncwarp();
      if (lane == 0) mbar_arrive(&r_empty[slot]);
      return true;
    };
    auto store_v = [&](const uint4 (&x)[D / 16]) -> bool {
      if (!warp_wait_bar(&v16_empty, (nv & 1) ^ 1, limit, &abort_flag, p.st, 232)) return false;
      const uint32_t dst = smem_u32(sV);
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        uint32_t h[8];
        e4m3x4_to_f16x4(x[c].x, h[0], h[1]);
        e4m3x4_to_f16x4(x[c].y, h[2], h[3]);
        e4m3x4_to_f16x4(x[c].z, h[4], h[5]);
        e4m3x4_to_f16x4(x[c].w, h[6], h[7]);
        const uint32_t o = dst + (c / 4) * (TILE * 128);
        st_shared_v4(o + sw128_off(row, (2 * c) % 8), h[0], h[1], h[2], h[3]);
        st_shared_v4(o + sw128_off(row, (2 * c + 1) % 8), h[4], h[5], h[6], h[7]);
      }
      fence_async_smem();  // read by the tensor core
      __syncwarp();
      if (lane == 0) mbar_arrive(&v16_full);
      ++nv;
      return true;
    };
    for (int g = 0; g < S.n_groups; ++g) {
      long long t0, t1;
      S.range(g, cta, t0, t1);
      for (long long t = t0; t < t1;) {  // phase 1: the query, then the sampled K tiles
        const int b = S.seq_of(t);
        const long long seg_end = t1 < (long long)S.seq_start[b + 1] ? t1 : (long long)S.seq_start[b + 1];
        if (skip_seq(b)) { t = seg_end; continue; }
        if (ok && !widen_q()) ok = false;
        ++nq;
        const int st = sample_stride(S, b, p.sample_tiles), lt_hi = (int)(seg_end - (long long)S.seq_start[b]);
        for (int lt = first_sample((int)(t - (long long)S.seq_start[b]), st); lt < lt_hi; lt += st, ++ri, ++js)
          if (ok && !widen_k(ri, js)) ok = false;
        t = seg_end;
      }
      for (long long t = t1 - 1; t >= t0;) {  // phase 2: the query, then K(0) K(1) V(0) K(2) V(1) ...
        const int b = S.seq_of(t);
        const long long seg_lo = t0 > (long long)S.seq_start[b] ? t0 : (long long)S.seq_start[b];
        if (skip_seq(b)) { t = seg_lo - 1; continue; }
        if (ok && !widen_q()) ok = false;
        ++nq;
        const uint32_t n = (uint32_t)(t - seg_lo + 1), base = ri;
        const int n_b = S.seq_len[b];
        auto v_valid = [&](uint32_t x) {  // row of tile x (descending from t) inside the sequence
          return (t - (long long)x - (long long)S.seq_start[b]) * TILE + row < (long long)n_b;
        };
        // ring items K(0) K(1) V(0) K(2) V(1) ... K(n-1) V(n-2) V(n-1), taken in that order; V(x)
        // is widened after K(x + 2), so that the wait for PV(x - 1) overlaps a K tile's work
        if (ok && !widen_k(base, js)) ok = false;
        if (ok && n > 1 && !widen_k(base + 1, js + 1)) ok = false;
        for (uint32_t x = 0; x < n && ok; ++x) {
          uint4 vr[D / 16];
          if (!load_v(x == n - 1 ? base + 2 * n - 1 : base + 2 * x + 2, v_valid(x), vr)) { ok = false; break; }
          if (x + 2 < n && !widen_k(base + 2 * x + 3, js + x + 2)) { ok = false; break; }
          if (!store_v(vr)) { ok = false; break; }
        }
        ri = base + 2 * n;
        js += n;
        jp += n;
        t = seg_lo - 1;
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax warpgroups
    const int wg = (warp - SM_WG0) / 4;
    const int wq = (warp - SM_WG0) % 4;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;            // key within the tile == TMEM lane == P^T row
    const int all_tid = wg * 128 + wq * 32 + lane;  // 0..255 over both warpgroups
    const int swarp = all_tid >> 5;                 // 0..7
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const float c = p.c;
    float(*red1)[4][HW][2] = reinterpret_cast<float(*)[4][HW][2]>(&red[0][0][0]);
    // state the selection accumulates into, cleared before this CTA's first grid-barrier arrival
    if (cta == 0) {
      for (int i = all_tid; i < p.B * NBINS; i += 256)
        if (!skip_seq(i / NBINS)) p.hist[i] = 0u;
      for (int i = all_tid; i < p.B; i += 256)
        if (!skip_seq(i)) p.seq_done[i] = 0;
      if (!p.fallback)
        for (int i = all_tid; i <= p.B; i += 256) p.ovf[i] = 0;
    }
    if (!p.fallback) {  // the selection bitmap (the collect kernel sets bits after this kernel)
      const long long total = (long long)p.B * p.words;
      const long long per = (total + S.G - 1) / S.G;
      const long long w0 = per * cta, w1 = w0 + per < total ? w0 + per : total;
      for (long long i = w0 + all_tid; i < w1; i += 256) p.bitmap[i] = 0u;
    }
    uint32_t js = 0, jp = 0, ri = 0, npu = 0, seg2 = 0;  // as in the tcgen05 issuer
    bool ok = true;
    // after a failed wait every later wait returns at once: the loop and named-barrier
    // structure stays identical across all 8 warps, only the work is skipped
    for (int g = 0; g < S.n_groups; ++g) {
      long long t0, t1;
      S.range(g, cta, t0, t1);
      // ---------------------------------------------------------------- phase 1 (sampled tiles)
      uint32_t n1 = 0;  // K tiles phase 1 took through the ring
      for (long long t = t0; t < t1;) {
        const int b = S.seq_of(t);
        const long long seg_end = t1 < (long long)S.seq_start[b + 1] ? t1 : (long long)S.seq_start[b + 1];
        if (skip_seq(b)) { t = seg_end; continue; }  // uniform: every softmax warp skips it
        bool first = true;
        float r[HW], l[HW];
#pragma unroll
        for (int h = 0; h < HW; ++h) { r[h] = -INFINITY; l[h] = 0.f; }
        const int st = sample_stride(S, b, p.sample_tiles), lt_hi = (int)(seg_end - (long long)S.seq_start[b]);
        for (int lt = first_sample((int)(t - (long long)S.seq_start[b]), st); lt < lt_hi; lt += st) {
          const uint32_t jt = js++;
          ++n1;
          if (!ok) continue;
          const int buf = jt & 1;
          if (!warp_wait_bar(&s_full[buf], (jt >> 1) & 1, limit, &abort_flag, p.st, 221)) { ok = false; continue; }
          tc_fence_after();
          float v[HW];
          tmem_ld32(tmem + lane_base + tS + buf * H + wg * HW, v);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[buf]);
          const bool valid = lt * TILE + row < S.seq_len[b];
          if (first) {
            // a lane's first key of the segment sets its references (invalid lanes only occur in
            // a sequence's partial last tile, which then is the segment's last sampled tile)
            first = false;
#pragma unroll
            for (int h = 0; h < HW; ++h) {
              r[h] = valid ? v[h] * c : -INFINITY;
              l[h] = valid ? 1.f : 0.f;
            }
            continue;
          }
          float dmax = -INFINITY;
#pragma unroll
          for (int h = 0; h < HW; ++h) {
            v[h] = valid ? fmaf(v[h], c, -r[h]) : -INFINITY;  // exponent relative to the reference
            dmax = fmaxf(dmax, v[h]);
          }
          if (__any_sync(0xffffffffu, dmax > REF_SLACK)) {
            // rare: move the reference of the heads that outgrew it
#pragma unroll
            for (int h = 0; h < HW; ++h) {
              const float d = v[h];
              if (d > REF_SLACK) {
                l[h] = l[h] * fast_exp2(-d) + 1.f;
                r[h] = r[h] + d;
              } else {
                l[h] += fast_exp2(d);
              }
            }
          } else {
#pragma unroll
            for (int h = 0; h < HW; ++h) l[h] += fast_exp2(v[h]);
          }
        }
        t = seg_end;
        // merge the 128 lanes of each warpgroup. Within a warp a reduce-scatter: at each step a
        // lane keeps half of its heads and merges in its partner's copy of that half, so after
        // 16 + 8 + 4 + 2 + 1 exchanges lane i holds head i of the warpgroup's 32. Then the 4
        // warps through shared memory.
#pragma unroll
        for (int half = 16; half >= 1; half >>= 1) {
          const bool up = (lane & half) != 0;
#pragma unroll
          for (int i = 0; i < half; ++i) {
            const float sm = up ? r[i] : r[i + half], sl = up ? l[i] : l[i + half];
            float km = up ? r[i + half] : r[i], kl = up ? l[i + half] : l[i];
            merge_ml(km, kl, __shfl_xor_sync(0xffffffffu, sm, half), __shfl_xor_sync(0xffffffffu, sl, half));
            r[i] = km;
            l[i] = kl;
          }
        }
        red1[wg][wq][lane][0] = r[0];
        red1[wg][wq][lane][1] = l[0];
        named_bar(3, 256);
        if (all_tid < H) {
          const int hg = all_tid / HW, hh = all_tid % HW;
          float mm = red1[hg][0][hh][0], ll = red1[hg][0][hh][1];
          for (int w = 1; w < 4; ++w) merge_ml(mm, ll, red1[hg][w][hh][0], red1[hg][w][hh][1]);
          const size_t sl = (size_t)S.slot(b, cta, S.cta_of(g, (long long)S.seq_start[b]));
          p.ml[sl * 2 * H + all_tid] = mm;
          p.ml[sl * 2 * H + H + all_tid] = ll;
        }
        named_bar(3, 256);
      }
      ri += n1;  // the phase-1 K items of the ring
      // ---------------------------------------------------------------- grid barrier
      // gbar[0] counts arrivals over the step's launches: zero when the sampled launch starts (a
      // zero-filled workspace, then re-armed by the collect kernel after both launches)
      named_bar(3, 256);
      if (all_tid == 0) {
        __threadfence();
        const unsigned target = (unsigned)S.G * (unsigned)(g + 1 + (p.fallback ? S.n_groups : 0));
        const unsigned arrived = atomicAdd(&p.gbar[0], 1u);
        if (arrived >= target) {  // a count left over: the workspace was not zero-filled
          abort_flag = 1;
          report_status(p.st, kStatusBounds, 231);
        }
        const long long tw = globaltimer_ns();
        while (!abort_flag && *(volatile unsigned*)&p.gbar[0] < target) {
          if (globaltimer_ns() - tw > limit) {
            abort_flag = 1;
            report_status(p.st, kStatusTimeout, 230);
          }
        }
        __threadfence();
      }
      named_bar(3, 256);
      // every CTA of this grid is resident: the next grid on the stream may start launching
      // (earlier, its CTAs could take SMs this grid still needs)
      if (g == 0) griddep_launch_dependents();
      if (abort_flag) ok = false;
      // ---------------------------------------------------------------- phase 2
      for (long long t = t1 - 1; t >= t0;) {
        const int b = S.seq_of(t);
        const long long seg_lo = t0 > (long long)S.seq_start[b] ? t0 : (long long)S.seq_start[b];
        if (skip_seq(b)) { t = seg_lo - 1; continue; }  // uniform: every softmax warp skips it
        int sg, c_lo, c_hi;
        S.covering(b, sg, c_lo, c_hi);
        const int n_b = S.seq_len[b], ncand = n_b - p.W > 0 ? n_b - p.W : 0;  // this sequence's
        {  // the sequence's lse from every phase-1 partial of it: 16 threads per partial record
           // (4 heads each), 16 records per round, then a shuffle and a shared-memory merge
          const int q4 = all_tid & 15;
          float M[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, L[4] = {0.f, 0.f, 0.f, 0.f};
          const float* rec = p.ml + (size_t)S.slot(b, c_lo, c_lo) * 2 * H + 4 * q4;
          const int n_rec = c_hi - c_lo + 1;
#pragma unroll 4
          for (int i = all_tid >> 4; i < n_rec; i += 16) {
            const float4 m4 = __ldcg(reinterpret_cast<const float4*>(rec + (size_t)i * 2 * H));
            const float4 l4 = __ldcg(reinterpret_cast<const float4*>(rec + (size_t)i * 2 * H + H));
            merge_ml(M[0], L[0], m4.x, l4.x);
            merge_ml(M[1], L[1], m4.y, l4.y);
            merge_ml(M[2], L[2], m4.z, l4.z);
            merge_ml(M[3], L[3], m4.w, l4.w);
          }
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            merge_ml(M[x], L[x], __shfl_xor_sync(0xffffffffu, M[x], 16), __shfl_xor_sync(0xffffffffu, L[x], 16));
            if (lane < 16) { red[swarp][4 * q4 + x][0] = M[x]; red[swarp][4 * q4 + x][1] = L[x]; }
          }
          named_bar(3, 256);
          if (all_tid < H) {
            const int h = all_tid;
            float mm = red[0][h][0], ll = red[0][h][1];
            for (int w = 1; w < 8; ++w) merge_ml(mm, ll, red[w][h][0], red[w][h][1]);
            const float lse2 = mm + log2f(ll);
            // of the sampled tiles only: the reference of p' = exp2(s*c - lse2); FP8 cache: less
            // an offset that keeps p' well inside the f16 range of P
            slse[h] = F8 ? lse2 - (p.fallback ? F8_OFF_EXACT : F8_OFF_SAMPLED) : lse2;
          }
          named_bar(3, 256);
        }
        const uint32_t n = (uint32_t)(t - seg_lo + 1), base = ri;
        float la = 0.f, lb = 0.f;  // sums of p' over this warp's keys for heads 2*lane, 2*lane + 1
        bool lsum_started = false;  // FP8 cache: this warpgroup's TMEM sums hold a tile of the segment
        for (uint32_t x = 0; x < n; ++x, --t, ++jp, ++js) {
          if ((int)(jp & 1) != wg || !ok) continue;  // the other warpgroup's tile, or unwinding
          const int lt = (int)(t - (long long)S.seq_start[b]);
          const int buf = jp & 1;   // == wg: this warpgroup's P buffer
          const int sbi = js & 1;   // the TMEM S buffer of this tile
          const int key = lt * TILE + row;
          const bool valid = key < n_b;
          if (!warp_wait_bar(&s_full[sbi], (js >> 1) & 1, limit, &abort_flag, p.st, 222)) { ok = false; continue; }
          tc_fence_after();
          float v[H];
#pragma unroll
          for (int cc = 0; cc < H / 32; ++cc) {
            float tmp[32];
            tmem_ld32(tmem + lane_base + tS + sbi * H + cc * 32, tmp);
#pragma unroll
            for (int x2 = 0; x2 < 32; ++x2) v[cc * 32 + x2] = tmp[x2];
          }
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cnt(&s_empty[sbi], 2);
          float sa = 0.f, sb = 0.f;
          uint32_t pk[H / 2];
#pragma unroll
          for (int h = 0; h < H; h += 4) {
            const float4 ls = *reinterpret_cast<const float4*>(&slse[h]);
            float e0, e1, e2, e3;
            ffma2(e0, e1, v[h], v[h + 1], c, c, -ls.x, -ls.y);
            ffma2(e2, e3, v[h + 2], v[h + 3], c, c, -ls.z, -ls.w);
            const float p0 = valid ? fast_exp2(e0) : 0.f, p1 = valid ? fast_exp2(e1) : 0.f;
            const float p2 = valid ? fast_exp2(e2) : 0.f, p3 = valid ? fast_exp2(e3) : 0.f;
            fadd2(sa, sb, sa, sb, p0, p1);
            fadd2(sa, sb, sa, sb, p2, p3);
            pk[h / 2] = F8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
            pk[h / 2 + 1] = F8 ? pack_f16x2(p2, p3) : pack_bf16x2(p2, p3);
            v[h] = p0; v[h + 1] = p1; v[h + 2] = p2; v[h + 3] = p3;
          }
          const float score = sa + sb;
          // p' above 2^64 (or not finite): the sampled reference was far too low for this
          // sequence; flag it for the exact redo (the sum is above 2^64 iff a term is). FP8
          // cache: the head sum above the f16 range (a sufficient test for every term's fit)
          if (__any_sync(0xffffffffu, valid && !(score <= (F8 ? F8_MAX_SCORE : 1.8446744e19f))) && lane == 0) {
            if (atomicExch(&p.ovf[b], 1) == 0) atomicAdd(&p.ovf[p.B], 1);
          }
          if (!warp_wait_bar(&p_empty[buf], (npu & 1) ^ 1, limit, &abort_flag, p.st, 223)) { ok = false; continue; }
          if (!F8 && (lt + 1) * TILE > n_b) {
            // the sequence's last tile, partial: its V rows past the sequence hold whatever the
            // caller's buffer holds there (rows of a longer sequence's slot in a ragged batch).
            // P is 0 for them, but 0 * inf is NaN in the PV product: zero those rows first. The
            // tile's V item cannot be overwritten before this warpgroup's P releases its PV.
            const uint32_t vi = x == n - 1 ? base + 2 * n - 1 : base + 2 * x + 2;
            const int vs = (int)(vi % NR);
            if (!warp_wait_bar(&r_full[vs], (vi / NR) & 1, limit, &abort_flag, p.st, 225)) { ok = false; continue; }
            if (!valid) {
              const uint32_t vrow = smem_u32(sR + vs * KT_BYTES);
#pragma unroll
              for (int ch = 0; ch < D / 8; ++ch)
                st_shared_v4(vrow + (ch / 8) * (TILE * 128) + sw128_off(row, ch % 8), 0u, 0u, 0u, 0u);
            }
            fence_async_smem();  // the zeros are read by the tensor core
          }
          const uint32_t prow = smem_u32(sP + buf * P_BYTES);
#pragma unroll
          for (int ch = 0; ch < H / 8; ++ch)
            st_shared_v4(prow + sw128_off(row, ch), pk[4 * ch], pk[4 * ch + 1], pk[4 * ch + 2], pk[4 * ch + 3]);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[buf]);
          ++npu;
          if constexpr (F8) {
            // this key row's p' per head added into the warpgroup's TMEM sums (lane = row); the
            // sums over the rows are formed once, at the end of the segment
            const uint32_t la_addr = tmem + lane_base + tLA + wg * H;
#pragma unroll
            for (int hb = 0; hb < H / 16; ++hb) {
              float acc[16];
              if (lsum_started) {
                tmem_ld16(la_addr + hb * 16, acc);
                tmem_ld_wait();
              } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[i] = 0.f;
              }
#pragma unroll
              for (int i = 0; i < 16; i += 2)
                fadd2(acc[i], acc[i + 1], acc[i], acc[i + 1], v[hb * 16 + i], v[hb * 16 + i + 1]);
              tmem_st16(la_addr + hb * 16, acc);
            }
            tmem_st_wait();
            lsum_started = true;
          } else {
            // per-head sums over the warp's 32 keys by a reduce-scatter: at each step a lane keeps
            // half of its values and adds its partner's copy of that half; at the end lane L holds
            // heads 2L and 2L + 1
#pragma unroll
            for (int stp = 0; stp < 5; ++stp) {
              const int cnt = 64 >> stp, dist = 16 >> stp;
              const bool up = (lane & dist) != 0;
#pragma unroll
              for (int i = 0; i < cnt / 2; ++i) {
                const float send = up ? v[i] : v[i + cnt / 2];
                const float keep = up ? v[i + cnt / 2] : v[i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, send, dist);
              }
            }
            la += v[0];
            lb += v[1];
            if (p.blk_part) {  // the warp's 32-key sums per head (exact block scores of HySparse v1)
              float* grp = p.blk_part + ((size_t)b * p.blk_groups + (size_t)lt * 4 + quarter) * H;
              reinterpret_cast<float2*>(grp)[lane] = make_float2(v[0], v[1]);
            }
          }
          const bool is_cand = valid && key < ncand;
          if (is_cand) p.sc[(size_t)b * p.sc_stride + key] = score;
          const unsigned bin = (__float_as_uint(score) >> 20) & (NBINS - 1);
          const unsigned act = __ballot_sync(0xffffffffu, is_cand);
          if (is_cand) {
            const unsigned peers = __match_any_sync(act, bin);
            if ((int)(__ffs(peers) - 1) == lane) atomicAdd(&shist[bin], (unsigned)__popc(peers));
          }
        }
        ri = base + 2 * n;
        if constexpr (F8) {
          // the warpgroup's TMEM sums over its rows: one reduce-scatter per segment (lane L ends
          // with heads 2L and 2L + 1 of its warp's 32 rows)
          if (lsum_started && ok) {
            float v[H];
#pragma unroll
            for (int hb = 0; hb < H / 32; ++hb) {
              float tmp[32];
              tmem_ld32(tmem + lane_base + tLA + wg * H + hb * 32, tmp);
#pragma unroll
              for (int i = 0; i < 32; ++i) v[hb * 32 + i] = tmp[i];
            }
            tmem_ld_wait();
#pragma unroll
            for (int stp = 0; stp < 5; ++stp) {
              const int cnt = 64 >> stp, dist = 16 >> stp;
              const bool up = (lane & dist) != 0;
#pragma unroll
              for (int i = 0; i < cnt / 2; ++i) {
                const float send = up ? v[i] : v[i + cnt / 2];
                const float keep = up ? v[i + cnt / 2] : v[i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, send, dist);
              }
            }
            la = v[0];
            lb = v[1];
          }
        }
        {  // this segment's per-head sums of p' over its keys: one record per (sequence, CTA)
          float* rr = &red[0][0][0];  // [8 warps][64 heads]
          rr[swarp * H + 2 * lane] = la;
          rr[swarp * H + 2 * lane + 1] = lb;
          named_bar(3, 256);
          if (all_tid < H) {
            float L = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) L += rr[w * H + all_tid];
            p.lp[(size_t)S.slot(b, cta, c_lo) * H + all_tid] = L;
          }
        }
        // segment done: warpgroup 0 fetches O^T (lane = output column d, one TMEM column per head)
        if (wg == 0 && ok) {
          if (!warp_wait_bar(&o_full, seg2 & 1, limit, &abort_flag, p.st, 224)) ok = false;
          if (ok) {
            tc_fence_after();
            float* dst = p.opart + (size_t)S.slot(b, cta, c_lo) * H * D;
#pragma unroll
            for (int cc = 0; cc < H / 32; ++cc) {
              float o[32];
              tmem_ld32(tmem + lane_base + tO + cc * 32, o);
              tmem_ld_wait();
#pragma unroll
              for (int x2 = 0; x2 < 32; ++x2) dst[(cc * 32 + x2) * D + row] = o[x2];
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_empty);
          }
        }
        ++seg2;
        // flush this sequence's histogram (both warpgroups are done with the segment)
        named_bar(3, 256);
        for (int i = all_tid; i < NBINS; i += 256) {
          const uint32_t cnt = shist[i];
          if (cnt) { atomicAdd(&p.hist[(size_t)b * NBINS + i], cnt); shist[i] = 0; }
        }
        __threadfence();
        named_bar(3, 256);
        // the last CTA to finish this sequence finds the bin of its k-th largest score
        if (all_tid == 0) s_last = atomicAdd(&p.seq_done[b], 1) == c_hi - c_lo;
        named_bar(3, 256);
        if (s_last) {
          // The last CTA of the sequence: exact per-head totals L'_h = sum_j p'_jh give the exact
          // lse (lse2 = lse2' + log2 L'); the true score of key j is sum_h p'_jh / L'_h, so
          // score'_j / max L' <= score_j <= score'_j / min L'. With rho = min L' / max L', a key
          // whose score' is above (upper edge of the k-th score' bin) / rho is certainly chosen,
          // one below rho * (lower edge) certainly not; the keys in between (the band) are
          // re-scored exactly (sel_rescore) and the top "need" of them by exact score taken.
          __threadfence();
          int* meta = p.meta + b * 8;
          const int K = p.K_sel;
          {  // L'_h over the sequence's records: 4 threads per head, their loads issued together
            float(*tl)[H] = reinterpret_cast<float(*)[H]>(&red[0][0][0]);
            const float* rec = p.lp + (size_t)S.slot(b, c_lo, c_lo) * H + (all_tid & (H - 1));
            float L4 = 0.f;
#pragma unroll 8
            for (int i = all_tid / H; i <= c_hi - c_lo; i += 256 / H) L4 += __ldcg(rec + (size_t)i * H);
            tl[all_tid / H][all_tid & (H - 1)] = L4;
          }
          named_bar(3, 256);
          if (all_tid < H) {
            const float(*tl)[H] = reinterpret_cast<const float(*)[H]>(&red[0][0][0]);
            const float L = (tl[0][all_tid] + tl[1][all_tid]) + (tl[2][all_tid] + tl[3][all_tid]);
            const float lse2 = slse[all_tid] + log2f(L);
            p.lse_out[b * H + all_tid] = lse2 * 0.69314718055994531f;
            p.lse2x[b * H + all_tid] = lse2;
            p.lsum[b * H + all_tid] = L;
            float mn = L, mx = L;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
              mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            }
            if (lane == 0) { s_lmm[swarp][0] = mn; s_lmm[swarp][1] = mx; }
          }
          named_bar(3, 256);
          if (ncand <= K || K == 0) {
            if (all_tid == 0) {
              meta[0] = K == 0 ? NBINS : -1;  // every older token above bin -1, or none above NBINS
              meta[1] = K == 0 ? 0 : ncand;
              meta[2] = 0;
              meta[3] = NBINS + 1;            // empty band
              meta[4] = 0; meta[5] = 0;
            }
          } else {
            // thread i owns bins hi..hi-7 (descending); block-inclusive scan of their counts
            const int hi = NBINS - 1 - 8 * all_tid;
            unsigned cnt8[8], local = 0;
#pragma unroll
            for (int x = 0; x < 8; ++x) { cnt8[x] = __ldcg(&p.hist[(size_t)b * NBINS + hi - x]); local += cnt8[x]; }
            unsigned incl = local;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const unsigned nb = __shfl_up_sync(0xffffffffu, incl, o);
              if (lane >= o) incl += nb;
            }
            if (lane == 31) s_wtot[swarp] = incl;
            named_bar(3, 256);
            unsigned add = 0;
            for (int x = 0; x < swarp; ++x) add += s_wtot[x];
            incl += add;
            const unsigned excl = incl - local;
            if (excl < (unsigned)K && incl >= (unsigned)K) {
              unsigned run = excl;
              for (int x = 0; x < 8; ++x) {
                if (run + cnt8[x] >= (unsigned)K) { s_band[2] = hi - x; break; }
                run += cnt8[x];
              }
            }
            named_bar(3, 256);
            if (all_tid == 0) {
              const float rho = fminf(s_lmm[0][0], s_lmm[1][0]) / fmaxf(s_lmm[0][1], s_lmm[1][1]);
              const unsigned beta = (unsigned)s_band[2];
              // score' of the k-th key lies in [lo, hi) of bin beta; slack for rounding of the sums
              const float lo = __uint_as_float(beta << 20), up_e = __uint_as_float((beta + 1) << 20);
              const float lower = rho * lo * (1.f - 3e-5f);
              const float upper = up_e / rho * (1.f + 3e-5f);
              const int b_lo = (int)((__float_as_uint(lower) >> 20) & (NBINS - 1));
              int b_hi = (int)(__float_as_uint(upper) >> 20);
              b_hi = b_hi > NBINS - 1 ? NBINS - 1 : b_hi;
              s_band[0] = b_lo;
              s_band[1] = b_hi;
            }
            named_bar(3, 256);
            const int b_lo = s_band[0], b_hi = s_band[1];
            unsigned above = 0, band = 0;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              const int bin = hi - x;
              if (bin > b_hi) above += cnt8[x];
              else if (bin >= b_lo) band += cnt8[x];
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
              above += __shfl_xor_sync(0xffffffffu, above, off);
              band += __shfl_xor_sync(0xffffffffu, band, off);
            }
            if (lane == 0) { s_cnt2[swarp][0] = above; s_cnt2[swarp][1] = band; }
            named_bar(3, 256);
            if (all_tid == 0) {
              unsigned ab = 0, bd = 0;
              for (int w = 0; w < 8; ++w) { ab += s_cnt2[w][0]; bd += s_cnt2[w][1]; }
              meta[0] = b_hi;             // bins above: chosen outright
              meta[1] = (int)ab;
              meta[2] = K - (int)ab;      // to take from the band by exact score
              meta[3] = b_lo;             // bins b_lo..b_hi: the band
              meta[4] = 0;                // band keys collected so far
              meta[5] = (int)bd;          // band size expected
            }
          }
        }
        named_bar(3, 256);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) { tc_fence_after(); tmem_dealloc(tmem, TMEM_COLS); }
}

// ------------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------------
size_t fused_smem_bytes(int H, int D, bool f8) {
  const size_t ring = f8 ? RING8 * (size_t)TILE * D + (size_t)TILE * D * 2 : RING * (size_t)TILE * D * 2;
  return 1024 + (size_t)H * D * 2 + ring + 2 * (size_t)TILE * H * 2 + NBINS * 4;
}

cudaError_t launch_decode_attn(const CUtensorMap& tmK, const CUtensorMap& tmV, const CUtensorMap& tmQ,
                               const DecParams& p, bool f8, cudaStream_t stream) {
  constexpr int H = 64, D = 128;
  static bool configured[2] = {false, false};
  auto* kern = f8 ? dec_fused_kernel<H, D, true> : dec_fused_kernel<H, D, false>;
  if (!configured[f8]) {
    cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)fused_smem_bytes(H, D, f8));
    configured[f8] = true;
  }
  // the sampled launch, then the exact redo of any sequence it flagged (normally none: the redo's
  // CTAs read the flag count and leave at once). Every CTA waits for all others at the grid
  // barrier, so both launches are cooperative; both are also programmatic dependents of the
  // work before them (their CTAs wait in griddepcontrol.wait), so the launch overlaps it.
  for (int pass = 0; pass < 2; ++pass) {
    DecParams q = p;
    if (pass == 1) {
      q.fallback = 1;
      q.sample_tiles = 0;  // every tile: the reference is the exact lse
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.sch.G);
    cfg.blockDim = dim3(f8 ? NTHREADS_F8 : NTHREADS);
    cfg.dynamicSmemBytes = fused_smem_bytes(H, D, f8);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e;
    {
      LaunchScope ls(pass == 0 ? "dec_fused" : "dec_redo", stream);
      e = cudaLaunchKernelEx(&cfg, kern, tmK, tmV, tmQ, q);
    }
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

}  // namespace dec
}  // namespace hs2
