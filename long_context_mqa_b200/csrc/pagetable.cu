// Page tables, slots and positions of one serving step from the requests' lengths.
//
// Request b holds lens[b] cached tokens and gains delta[b] (negative: its cache is cut back), so it
// holds ceil(lens/page) pages and wants ceil((lens + delta)/page). Free pages wait in a ring: the
// requests' new pages are taken from its head in request order (an exclusive prefix sum of the pages
// that each lacks), pages given back are appended behind its tail, and the two ranges never meet
// because the ring has room for every page of the pool. A granted request's new tokens, packed in
// request order, get a position each (lens[b], lens[b] + 1, ..) and a slot (page * page_size + row). A request that the
// free pages or the packed rows do not suffice for, or whose pages the ring cannot take back, is left as it was.
//
// The work is a prefix sum over at most 4,096 requests and then independent items: one per token row
// and one per returned page, each finding its request by a binary search in the sums. Every block
// computes the sums for itself (16 KB of lengths from L2, three scans in step), which costs less than a
// second launch or a grid-wide wait, and takes its share of the items. The token that is the first of
// its page writes the table entry. Latency bounds it: two reads that depend on one another, the
// scan between them (replayed from a graph 2.8 us for 32 requests with one token each, 5.1 us for 511 with 105,000
// rows; called one after the other 5.1 and 6.0 us).
#include "host_util.h"
#include "tc.cuh"

namespace hs2 {
namespace ptab {

constexpr int NT = 512;
constexpr int MAX_B = 4096;

struct Params {
  int32_t* table;
  const int32_t *lens, *delta;
  int32_t* ring;
  const int32_t* state;  // {head, count}
  int32_t *lens_out, *state_out, *cu, *pos, *slots;
  int B, width, cap, page, T;
  unsigned* done;  // blocks that have read the inputs; zero between calls
  DevStatus* st;
};

// Sums of counts stop below 2^30 (for counts >= 0 this addition is associative too), so that no request's
// numbers, however wrong, wrap a sum around; row indices stay below 2^30.
constexpr int MOST = (1 << 30) - 1;
__device__ __forceinline__ int sat_add(int a, int b) { return min(a + b, MOST); }

// the request whose range [off[b], off[b + 1]) holds i (ranges may be empty)
__device__ __forceinline__ int find(const int* off, int n, int i) {
  int lo = 0, hi = n;  // off[lo] <= i < off[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// PER: requests of a thread
template <int PER>
__global__ void __launch_bounds__(NT) page_table_kernel(Params p) {
  extern __shared__ int sm[];
  int* tok = sm;               // [B + 1] first packed row of each request
  int* add = tok + p.B + 1;    // [B] its first new page, counted from the ring's head; -1: not granted
  int* back = add + p.B;       // [B + 1] its first returned page
  int* held_len = back + p.B + 1;  // [B] its length; of one that gives pages back, how many it keeps
  __shared__ int warp_sum[3][NT / 32], s_used, s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) s_used = 0;
  griddep_wait();
  griddep_launch_dependents();
  const int head = p.state[0], count = p.state[1];
  // what each request adds: token rows, pages it lacks, pages it gives back
  int len[PER], rows[PER], grow[PER], gone[PER], want_len[PER], sum[3] = {0, 0, 0};
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * PER + i;
    len[i] = b < p.B ? p.lens[b] : 0;
    rows[i] = b < p.B ? p.delta[b] : 0;
  }
  const bool state_ok = head >= 0 && head < p.cap && count >= 0 && count <= p.cap;
  bool bad = !state_ok;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int n = len[i], x = rows[i], b = tid * PER + i;
    const long long m = (long long)n + x;
    int keep = n;
    grow[i] = gone[i] = 0;
    rows[i] = x > 0 ? min(x, MOST) : 0;
    // a length or an end outside the table: the request is left as it is
    if (n < 0 || m < 0 || n > (long long)p.width * p.page || m > (long long)p.width * p.page) {
      bad = true;
      want_len[i] = n;
      grow[i] = -1;
    } else {
      want_len[i] = (int)m;
      const int held = (n + p.page - 1) / p.page, want = (int)((m + p.page - 1) / p.page);
      grow[i] = want > held ? want - held : 0;
      gone[i] = held > want ? held - want : 0;
      if (gone[i] > 0) keep = want;
    }
    if (b < p.B) held_len[b] = keep;
    sum[0] = sat_add(sum[0], rows[i]);
    sum[1] = sat_add(sum[1], max(grow[i], 0));
    sum[2] = sat_add(sum[2], gone[i]);
  }
  // the three exclusive prefix sums over the block (saturating: every value is >= 0), and their totals
  int at[3], all[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    int x = sum[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x = sat_add(x, y);
    }
    if (lane == 31) warp_sum[k][warp] = x;
    const int prev = __shfl_up_sync(0xffffffffu, x, 1);
    at[k] = lane == 0 ? 0 : prev;
  }
  __syncthreads();
  // the inputs have been read; the block that is the last to say so writes the new lengths and the
  // ring's state at its end, so that they may be updated in place
  if (gridDim.x > 1 && tid == NT - 1) {
    __threadfence();
    s_last = atomicAdd(p.done, 1u) == gridDim.x - 1;
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    int x = lane < NT / 32 ? warp_sum[k][lane] : 0;
#pragma unroll
    for (int o = 1; o < NT / 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x = sat_add(x, y);
    }
    all[k] = __shfl_sync(0xffffffffu, x, NT / 32 - 1);
    const int before = __shfl_sync(0xffffffffu, x, warp > 0 ? warp - 1 : 0);
    if (warp > 0) at[k] = sat_add(before, at[k]);
  }
  const int rows_all = all[0], back_all = all[2];
  const int avail = state_ok ? count : 0;
  // more pages than the ring holds with those given back (the caller's lists disagree): none is
  const bool room = state_ok && (long long)count + back_all <= p.cap;
  if (!room && back_all > 0) bad = true;
  int used = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * PER + i;
    // its rows have to lie within the packed ones, all of them (a page is entered by the token that is its first);
    // those of every later request with new tokens lie behind them
    bool granted = grow[i] >= 0 && (rows[i] == 0 || at[0] + rows[i] <= p.T);
    if (granted && grow[i] > 0) {
      granted = at[1] <= avail && grow[i] <= avail - at[1];  // in request order, while they last
      if (granted) used = at[1] + grow[i];
      else bad = true;
    }
    if (b < p.B) {
      tok[b] = at[0];
      back[b] = at[2];
      add[b] = granted ? at[1] : -1;
    }
    at[0] = sat_add(at[0], rows[i]);
    at[1] = sat_add(at[1], max(grow[i], 0));
    at[2] = sat_add(at[2], gone[i]);
    if (!granted || (gone[i] > 0 && !room)) want_len[i] = len[i];
  }
  used = __reduce_max_sync(0xffffffffu, used);
  if (lane == 0 && used > 0) atomicMax(&s_used, used);
  if (tid == 0) {
    tok[p.B] = rows_all;
    back[p.B] = back_all;
  }
  if (rows_all > p.T) bad = true;
  const bool any_bad = __syncthreads_or(bad);
  if (any_bad && blockIdx.x == 0 && tid == 0) report_status(p.st, kStatusBounds, 601);

  auto wrap = [&](unsigned i) { return i >= (unsigned)p.cap ? i - (unsigned)p.cap : i; };  // i < 2 cap
  const unsigned items = (unsigned)p.T + (unsigned)(room ? back_all : 0);  // (both below 2^30)
  for (unsigned i0 = blockIdx.x * NT + tid; i0 < items; i0 += gridDim.x * NT) {
    const int it = (int)i0;
    if (it < p.T) {
      int pos = -1;
      long long slot = -1;
      if (it < rows_all) {
        const int b = find(tok, p.B, it), n = held_len[b], first = add[b];
        pos = n + it - tok[b];
        if (first >= 0) {
          const int j = pos / p.page, r = pos - j * p.page, held = (n + p.page - 1) / p.page;
          int pg;
          if (j < held) {
            pg = p.table[(size_t)b * p.width + j];
          } else {
            pg = p.ring[wrap((unsigned)head + (unsigned)(first + j - held))];
            if (r == 0) p.table[(size_t)b * p.width + j] = pg;
          }
          slot = (long long)pg * p.page + r;
          if (pg < 0 || slot > 0x7FFFFFFFll) {  // no page's id
            slot = -1;
            report_status(p.st, kStatusBounds, 602);
          }
        }
      }
      p.pos[it] = pos;
      p.slots[it] = (int)slot;
    } else {
      const int i = it - p.T, b = find(back, p.B, i);
      const int pg = p.table[(size_t)b * p.width + held_len[b] + i - back[b]];
      if (pg < 0 || (long long)pg * p.page > 0x7FFFFFFFll) report_status(p.st, kStatusBounds, 603);
      p.ring[wrap((unsigned)head + (unsigned)(count + i))] = pg;
    }
  }
  if (blockIdx.x == 0)
    for (int b = tid; b <= p.B; b += NT) p.cu[b] = tok[b];
  if (gridDim.x > 1) {
    __syncthreads();
    if (!s_last) return;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * PER + i;
    if (b < p.B) p.lens_out[b] = want_len[i];
  }
  if (tid == 0) {
    if (gridDim.x > 1) *p.done = 0;
    const int u = s_used;
    p.state_out[0] = state_ok ? (int)wrap((unsigned)head + (unsigned)u) : head;
    p.state_out[1] = state_ok ? count - u + (room ? back_all : 0) : count;
  }
}

constexpr size_t kStatusBytes = 256;
constexpr size_t kDoneOffset = 128;

}  // namespace ptab
}  // namespace hs2

using namespace hs2;

extern "C" {

size_t hs2_page_table_update_workspace_bytes(void) { return ptab::kStatusBytes; }

hs2_status hs2_page_table_update(int32_t* page_table, int B, int max_pages, const int32_t* lens, const int32_t* delta,
                                 int32_t* free_ring, int ring_size, const int32_t* free_state, int page_size,
                                 int max_tokens, int32_t* lens_out, int32_t* free_state_out, int32_t* cu_tokens,
                                 int32_t* positions, int32_t* slots, void* workspace, size_t workspace_bytes,
                                 hs2_stream stream) {
  if (!page_table || !lens || !delta || !free_ring || !free_state || !lens_out || !free_state_out || !cu_tokens ||
      B < 1 || max_pages < 1 || ring_size < 1 || page_size < 1 || max_tokens < 0 ||
      (long long)max_pages * page_size > ptab::MOST || max_tokens > ptab::MOST || (max_tokens > 0 && (!positions || !slots)))
    return HS2_ERR_INVALID_ARG;
  if (B > ptab::MAX_B || !device_is_sm100()) return HS2_ERR_UNSUPPORTED_SHAPE;
  if (!workspace || !aligned16(workspace) || workspace_bytes < ptab::kStatusBytes) return HS2_ERR_WORKSPACE;
  ptab::Params p{page_table, lens, delta, free_ring, free_state, lens_out, free_state_out, cu_tokens, positions, slots,
                 B, max_pages, ring_size, page_size, max_tokens,
                 (unsigned*)((uint8_t*)workspace + ptab::kDoneOffset), (DevStatus*)workspace};
  // a row a thread, while there are threads: a decode step is one block's work (a row waits for a page id from
  // L2 or HBM, so rows in turn cost that each: 511 requests with 105,000 rows 9.9 us at four rows a thread)
  const long long blocks = ((long long)max_tokens + ptab::NT - 1) / ptab::NT, most = 2ll * num_sms();
  const int grid = (int)(blocks < 1 ? 1 : blocks > most ? most : blocks);
  const size_t smem = (size_t)(4 * B + 2) * sizeof(int);
  const cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  if (B <= ptab::NT) {
    LaunchScope ls("page_table", st);
    e = launch_k(ptab::page_table_kernel<1>, dim3(grid), dim3(ptab::NT), smem, st, true, p);
  } else {
    e = cudaFuncSetAttribute(ptab::page_table_kernel<ptab::MAX_B / ptab::NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)((4 * ptab::MAX_B + 2) * sizeof(int)));
    if (e != cudaSuccess) return HS2_ERR_CUDA;
    LaunchScope ls("page_table", st);
    e = launch_k(ptab::page_table_kernel<ptab::MAX_B / ptab::NT>, dim3(grid), dim3(ptab::NT), smem, st, true, p);
  }
  return e == cudaSuccess ? HS2_OK : HS2_ERR_CUDA;
}

}  // extern "C"
