// Page tables, slots and positions of one serving step from the requests' lengths.
//
// Request b holds lens[b] cached tokens and gains delta[b] (negative: its cache is cut back), so it
// holds ceil(lens/page) pages and wants ceil((lens + delta)/page). Free pages wait in a ring: the
// requests' new pages are taken from its head in request order (an exclusive prefix sum of the pages
// that each lacks), pages given back are appended behind its tail, and the two ranges never meet
// because the ring has room for every page of the pool. A granted request's new tokens, packed in
// request order, get a position each (lens[b], lens[b] + 1, ..) and a slot (page * page_size + row).
//
// The work is a prefix sum over at most 4,096 requests and then independent items: one per token row
// and one per returned page, each finding its request by a binary search in the sums. Every block
// computes the sums for itself (16 KB of lengths from L2, three block scans), which costs less than a
// second launch or a grid-wide wait, and takes its share of the items. The token that is the first of
// its page writes the table entry. The last block to have read the inputs writes the new lengths and
// the ring's state, so that both may be updated in place.
#include "host_util.h"
#include "tc.cuh"

namespace hs2 {
namespace ptab {

constexpr int NT = 512;
constexpr int MAX_B = 4096;
constexpr int PER = MAX_B / NT;  // requests of a thread at most

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

// exclusive prefix sum of one value per thread (0 .. MOST) over the block, and its total
__device__ __forceinline__ int block_scan(int v, int* total, int* warp_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x = sat_add(x, y);
  }
  __syncthreads();
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const int s = warp_sum[w];
    if (w < warp) before = sat_add(before, s);
    all = sat_add(all, s);
  }
  *total = all;
  const int prev = __shfl_up_sync(0xffffffffu, x, 1);
  return lane == 0 ? before : sat_add(before, prev);
}

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

__global__ void __launch_bounds__(NT) page_table_kernel(Params p) {
  extern __shared__ int sm[];
  int* tok = sm;               // [B + 1] first packed row of each request
  int* add = tok + p.B + 1;    // [B] its first new page, counted from the ring's head; -1: not granted
  int* back = add + p.B;       // [B + 1] its first returned page
  __shared__ int warp_sum[NT / 32];
  __shared__ int s_used, s_last;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  const int head = p.state[0], count = p.state[1];
  const bool state_ok = head >= 0 && head < p.cap && count >= 0 && count <= p.cap;
  const int per = (p.B + NT - 1) / NT;
  if (tid == 0) s_used = 0;
  // what each request adds: token rows, pages it lacks, pages it gives back
  int len[PER], rows[PER], grow[PER], gone[PER], want_len[PER];
  int sr = 0, sg = 0, sb = 0;
  bool bad = !state_ok;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    len[i] = rows[i] = grow[i] = gone[i] = want_len[i] = 0;
    const int b = tid * per + i;
    if (i < per && b < p.B) {
      const int n = p.lens[b], x = p.delta[b];
      const long long m = (long long)n + x;
      len[i] = n;
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
      }
      sr = sat_add(sr, rows[i]);
      sg = sat_add(sg, max(grow[i], 0));
      sb = sat_add(sb, gone[i]);
    }
  }
  int rows_all, grow_all, back_all;
  int r0 = block_scan(sr, &rows_all, warp_sum);
  int g0 = block_scan(sg, &grow_all, warp_sum);
  int b0 = block_scan(sb, &back_all, warp_sum);
  const int avail = state_ok ? count : 0;
  int used = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * per + i;
    if (i < per && b < p.B) {
      tok[b] = r0;
      back[b] = b0;
      r0 = sat_add(r0, rows[i]);
      b0 = sat_add(b0, gone[i]);
      bool granted = grow[i] >= 0;
      if (grow[i] > 0) {
        granted = g0 <= avail && grow[i] <= avail - g0;  // in request order, while they last
        if (granted) used = g0 + grow[i];
        else bad = true;
      }
      add[b] = granted ? g0 : -1;
      g0 = sat_add(g0, max(grow[i], 0));
      if (!granted) want_len[i] = len[i];
    }
  }
  if (used > 0) atomicMax(&s_used, used);
  if (tid == 0) {
    tok[p.B] = rows_all;
    back[p.B] = back_all;
  }
  // more pages than the ring holds with those given back: the caller's lists disagree
  const bool room = state_ok && (long long)count + back_all <= p.cap;
  if (!room && back_all > 0) bad = true;
  if (rows_all > p.T) bad = true;
  const bool any_bad = __syncthreads_or(bad);
  if (any_bad && blockIdx.x == 0 && tid == 0) report_status(p.st, kStatusBounds, 601);

  const long long items = (long long)p.T + (room ? back_all : 0);
  const long long step = (long long)gridDim.x * NT;
  for (long long it = (long long)blockIdx.x * NT + tid; it < items; it += step) {
    if (it < p.T) {
      const int row = (int)it;
      int pos = -1;
      long long slot = -1;
      if (row < rows_all) {
        const int b = find(tok, p.B, row);
        const int n = p.lens[b], first = add[b];
        pos = n + row - tok[b];
        if (first >= 0) {
          const int j = pos / p.page, r = pos - j * p.page, held = (n + p.page - 1) / p.page;
          int pg;
          if (j < held) {
            pg = p.table[(size_t)b * p.width + j];
          } else {
            pg = p.ring[((long long)head + first + j - held) % p.cap];
            if (r == 0) p.table[(size_t)b * p.width + j] = pg;
          }
          slot = (long long)pg * p.page + r;
          if (pg < 0 || slot > 0x7FFFFFFFll) slot = -1;
        }
      }
      p.pos[row] = pos;
      p.slots[row] = (int)slot;
    } else {
      const int i = (int)(it - p.T);
      const int b = find(back, p.B, i);
      const int want = (p.lens[b] + p.delta[b] + p.page - 1) / p.page;
      p.ring[((long long)head + count + i) % p.cap] = p.table[(size_t)b * p.width + want + i - back[b]];
    }
  }
  if (blockIdx.x == 0)
    for (int b = tid; b <= p.B; b += NT) p.cu[b] = tok[b];
  // the last block to get here has seen every other one read the inputs
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    s_last = atomicAdd(p.done, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * per + i;
    if (i < per && b < p.B) p.lens_out[b] = want_len[i];
  }
  if (tid == 0) {
    *p.done = 0;
    const int u = s_used;
    p.state_out[0] = state_ok ? (int)(((long long)head + u) % p.cap) : head;
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
  // one block per 2,048 rows: a decode step is one block's work, a prompt's rows spread over the GPU
  int grid = (max_tokens + 2047) / 2048;
  if (grid < 1) grid = 1;
  if (grid > num_sms()) grid = num_sms();
  const size_t smem = (size_t)(3 * B + 2) * sizeof(int);
  if (smem > 48000 && cudaFuncSetAttribute(ptab::page_table_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)((3 * ptab::MAX_B + 2) * sizeof(int))) != cudaSuccess)
    return HS2_ERR_CUDA;
  LaunchScope ls("page_table", (cudaStream_t)stream);
  return launch_k(ptab::page_table_kernel, dim3(grid), dim3(ptab::NT), smem, (cudaStream_t)stream, true, p) == cudaSuccess
             ? HS2_OK
             : HS2_ERR_CUDA;
}

}  // extern "C"
