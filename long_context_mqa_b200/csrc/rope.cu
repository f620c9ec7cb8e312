// Norm and position rotation of query and key heads in one pass, its backward pass, and the
// serving form that also writes the rotated keys and the values into the pages of a cache.
//
// Per row x of d elements (one head of one token), with the head weight w and position t:
//   n = x * rsqrt(mean(x^2) + eps) * w           (no weight: n = x)
//   (a, b) -> m (a cos - b sin, b cos + a sin)   for each pair of the first `rot` elements, the
//   angle t * inv_freq[i]; pair i is (i, i + rot/2), or (2i, 2i + 1) when interleaved.
// Backward, g the upstream gradient rotated back (by -angle, times m), u = g w, r = rsqrt(..):
//   dx = r (u - x r^2 mean(u x)),   dw = sum over rows of g x r.
//
// All of it is bound by HBM (a few flops per byte; the kernels read each row once and write it
// once), so the layout serves the memory system: a lane owns 8 consecutive elements (one 16-byte
// access), d/8 lanes a row, and a warp works on the rows of ONE token, so the token's cosines and
// sines stay in registers over its heads. They are computed once per (warp, token): each lane takes
// a share of the angles, in 64 bits as turns t * f / 2 pi reduced to [-1/2, 1/2] (a 32-bit angle of
// position 10^6 is off by 0.06), and the lanes read theirs back from shared memory. A row's mean is
// a shuffle reduction over its lanes, and in the half layout the partner of an element sits rot/16
// lanes away. Loads of several rows are issued before the first is used. All arithmetic is in 32
// bits, rounded once at the store.
#include "host_util.h"
#include "tc.cuh"

namespace hs2 {
namespace rope {

constexpr int NT = 256, NW = NT / 32;
constexpr int MAX_HALF = 64;  // rot / 2 at most

struct Params {
  const __nv_bfloat16 *q, *k, *v;
  long long q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;  // token and head strides in elements
  const int32_t* pos;
  const double* inv_freq;
  const void *qw, *kw;  // NULL: no norm
  int w_f32;
  int T, Hq, Hk, rot;
  int rows;    // rows of a token: Hq + Hk, + Hk values in the paged form
  int parts;   // warps that share a token's rows
  float eps, mscale;
  __nv_bfloat16 *q_out, *k_out;  // contiguous [T, Hq, D], [T, Hk, D]
  // paged form
  const int32_t* slots;
  void *k_pages, *v_pages;
  long long kp_ps, kp_rs, kp_hs, vp_ps, vp_rs, vp_hs;  // page, row and head strides in elements
  int page, n_pages;
  float k_inv, v_inv;  // 1 / scale of an e4m3 cache
  DevStatus* st;
  // backward
  const __nv_bfloat16* dq_out;
  const void* dk_out;
  __nv_bfloat16 *dq, *dk;
  float* part;  // [grid][2][D] weight gradients of each block
};

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(a[i] << 16);
    x[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
// two floats -> e4m3 codes (the first in the low byte), rounded to nearest even, saturating at 448
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8]) {
  return make_uint2(pack_e4m3x2(x[0], x[1]) | (pack_e4m3x2(x[2], x[3]) << 16),
                    pack_e4m3x2(x[4], x[5]) | (pack_e4m3x2(x[6], x[7]) << 16));
}
__device__ __forceinline__ void load_w8(const void* w, int f32, int at, float (&x)[8]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 1.f;
  } else if (f32) {
    const float4 a = __ldg((const float4*)((const float*)w + at)), b = __ldg((const float4*)((const float*)w + at) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    unpack8(__ldg((const uint4*)((const __nv_bfloat16*)w + at)), x);
  }
}

// The rotation of one token as a lane applies it: element e of the lane's 8 belongs to pair
// pair_of(e); cs[] holds that pair's cosine and sine times m (half layout: 8 pairs, interleaved: 4).
template <int D, bool INTER>
struct Rot {
  static constexpr int LPR = D / 8;            // lanes of a row
  static constexpr int NP = INTER ? 4 : 8;     // pairs a lane meets
  float c[NP], s[NP];
  int partner;   // the lane that holds the other half of this lane's pairs (half layout)
  bool on;       // this lane's elements are rotated

  __device__ __forceinline__ void init(int lane, int rot) {
    const int li = lane % LPR, hl = rot / 16;
    on = li * 8 < rot;
    partner = !on ? lane : li < hl ? lane + hl : lane - hl;
  }
  // the whole warp: token position t; `sc` is this warp's [MAX_HALF] buffer
  __device__ __forceinline__ void angles(int t, const double* inv_freq, int rot, float mscale, int lane, float2* sc) {
    const int half = rot / 2;
    __syncwarp();
    for (int i = lane; i < half; i += 32) {
      const double turns = (double)t * __ldg(inv_freq + i) * 0.15915494309189533577;  // 1 / (2 pi)
      float sn, cn;
      sincospif((float)(2.0 * (turns - rint(turns))), &sn, &cn);
      sc[i] = make_float2(cn * mscale, sn * mscale);
    }
    __syncwarp();
    const int li = lane % LPR;
    if (on) {
      const int first = INTER ? li * 4 : (li * 8 < half ? li * 8 : li * 8 - half);
      const float sg = !INTER && li * 8 < half ? -1.f : 1.f;  // first half: a cos - b sin
#pragma unroll
      for (int e = 0; e < NP; ++e) {
        const float2 x = sc[first + e];
        c[e] = x.x;
        s[e] = x.y * sg;
      }
    }
  }
  // x -> its rotation (dir = 1) or the transpose (dir = -1); every lane of the warp takes part
  __device__ __forceinline__ void apply(float (&x)[8], float dir) const {
    if (INTER) {
      if (on) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = x[2 * i], b = x[2 * i + 1], sn = s[i % NP] * dir;
          x[2 * i] = a * c[i % NP] - b * sn;
          x[2 * i + 1] = b * c[i % NP] + a * sn;
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float o = __shfl_sync(0xffffffffu, x[e], partner);
        if (on) x[e] = x[e] * c[e % NP] + o * (s[e % NP] * dir);
      }
    }
  }
};

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One warp per (token, part): the part's rows in passes of 32 / LPR rows, U passes in flight.
template <int D, bool INTER, bool PAGED, bool F8>
__global__ void __launch_bounds__(NT) rope_fwd_kernel(Params p) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, U = 4;
  __shared__ float2 sc[NW][MAX_HALF];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int li = lane % LPR, sub = lane / LPR;
  const long long item = (long long)blockIdx.x * NW + warp;
  griddep_wait();
  griddep_launch_dependents();
  const int t = (int)(item / p.parts), part = (int)(item % p.parts);
  if (t >= p.T) return;
  int slot = 0;
  if (PAGED) {
    slot = __ldg(p.slots + t);
    if (slot < 0) return;  // a padding row: nothing of it is read or written
  }
  Rot<D, INTER> rot;
  rot.init(lane, p.rot);
  rot.angles(__ldg(p.pos + t), p.inv_freq, p.rot, p.mscale, lane, sc[warp]);
  long long kc = -1, vc = -1;  // the cache rows of this token
  if (PAGED) {
    const int pg = slot / p.page, r = slot - pg * p.page;
    if (pg < p.n_pages) {
      kc = pg * p.kp_ps + r * p.kp_rs;
      vc = pg * p.vp_ps + r * p.vp_rs;
    } else if (part == 0 && lane == 0) {
      report_status(p.st, kStatusBounds, 501);
    }
  }
  const int n_pass = (p.rows + RPW - 1) / RPW;
  const int per = (n_pass + p.parts - 1) / p.parts;
  const int p1 = min(n_pass, (part + 1) * per);
  float wq[8], wk[8];
  load_w8(p.qw, p.w_f32, li * 8, wq);
  load_w8(p.kw, p.w_f32, li * 8, wk);
  for (int p0 = part * per; p0 < p1; p0 += U) {
    uint4 x4[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = (p0 + u) * RPW + sub;
      x4[u] = make_uint4(0u, 0u, 0u, 0u);
      if (p0 + u < p1 && row < p.rows) {
        const __nv_bfloat16* src = row < p.Hq            ? p.q + t * p.q_ts + row * p.q_hs
                                   : row < p.Hq + p.Hk ? p.k + t * p.k_ts + (row - p.Hq) * p.k_hs
                                                       : p.v + t * p.v_ts + (row - p.Hq - p.Hk) * p.v_hs;
        x4[u] = __ldg(reinterpret_cast<const uint4*>(src) + li);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (p0 + u >= p1) break;  // (warp-uniform)
      const int row = (p0 + u) * RPW + sub;
      const bool is_q = row < p.Hq, is_k = !is_q && row < p.Hq + p.Hk;
      float x[8];
      unpack8(x4[u], x);
      float y[8];
      if (p.qw) {  // (both weights are given, or neither)
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
        const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + p.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[e] * r * (is_q ? wq[e] : wk[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[e];
      }
      rot.apply(y, 1.f);
      if (row >= p.rows) continue;
      if (is_q) {
        reinterpret_cast<uint4*>(p.q_out + ((long long)t * p.Hq + row) * D)[li] = pack8(y);
      } else if (!PAGED) {
        reinterpret_cast<uint4*>(p.k_out + ((long long)t * p.Hk + row - p.Hq) * D)[li] = pack8(y);
      } else if (kc >= 0) {
        const int h = is_k ? row - p.Hq : row - p.Hq - p.Hk;
        const long long at = (is_k ? kc + h * p.kp_hs : vc + h * p.vp_hs) + li * 8;
        void* pool = is_k ? p.k_pages : p.v_pages;
        if (F8) {
          const float inv = is_k ? p.k_inv : p.v_inv;
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = (is_k ? y[e] : x[e]) * inv;
          *reinterpret_cast<uint2*>((uint8_t*)pool + at) = pack8_e4m3(y);
        } else {
          *reinterpret_cast<uint4*>((__nv_bfloat16*)pool + at) = is_k ? pack8(y) : x4[u];
        }
      }
    }
  }
}

// Backward: warps stride over (token, part) items and keep the weight gradients of their 8 elements
// in registers; a block adds its warps' in a fixed order and writes one record (rope_dw_kernel adds
// the records, also in a fixed order: the result does not vary from run to run).
template <int D, bool INTER, bool GK32>
__global__ void __launch_bounds__(NT) rope_bwd_kernel(Params p) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, U = 2;
  __shared__ float2 sc[NW][MAX_HALF];
  __shared__ float red[NW][2][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int li = lane % LPR, sub = lane / LPR;
  griddep_wait();
  griddep_launch_dependents();
  Rot<D, INTER> rot;
  rot.init(lane, p.rot);
  float wq[8], wk[8], aq[8], ak[8];
  load_w8(p.qw, p.w_f32, li * 8, wq);
  load_w8(p.kw, p.w_f32, li * 8, wk);
#pragma unroll
  for (int e = 0; e < 8; ++e) aq[e] = ak[e] = 0.f;
  const int n_pass = (p.rows + RPW - 1) / RPW;
  const int per = (n_pass + p.parts - 1) / p.parts;
  const long long items = (long long)p.T * p.parts;
  for (long long item = (long long)blockIdx.x * NW + warp; item < items; item += (long long)gridDim.x * NW) {
    const int t = (int)(item / p.parts), part = (int)(item % p.parts);
    const int p1 = min(n_pass, (part + 1) * per);
    if (part * per >= p1) continue;
    rot.angles(__ldg(p.pos + t), p.inv_freq, p.rot, p.mscale, lane, sc[warp]);
    for (int p0 = part * per; p0 < p1; p0 += U) {
      uint4 x4[U], g4[U], h4[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int row = (p0 + u) * RPW + sub;
        x4[u] = g4[u] = h4[u] = make_uint4(0u, 0u, 0u, 0u);
        if (p0 + u < p1 && row < p.rows) {
          if (row < p.Hq) {
            if (p.qw) x4[u] = __ldg(reinterpret_cast<const uint4*>(p.q + t * p.q_ts + row * p.q_hs) + li);
            g4[u] = __ldg(reinterpret_cast<const uint4*>(p.dq_out + ((long long)t * p.Hq + row) * D) + li);
          } else {
            const long long at = ((long long)t * p.Hk + row - p.Hq) * D;
            if (p.qw) x4[u] = __ldg(reinterpret_cast<const uint4*>(p.k + t * p.k_ts + (row - p.Hq) * p.k_hs) + li);
            if (GK32) {
              g4[u] = __ldg(reinterpret_cast<const uint4*>((const float*)p.dk_out + at) + 2 * li);
              h4[u] = __ldg(reinterpret_cast<const uint4*>((const float*)p.dk_out + at) + 2 * li + 1);
            } else {
              g4[u] = __ldg(reinterpret_cast<const uint4*>((const __nv_bfloat16*)p.dk_out + at) + li);
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (p0 + u >= p1) break;  // (warp-uniform)
        const int row = (p0 + u) * RPW + sub;
        const bool is_q = row < p.Hq;
        float x[8], g[8];
        unpack8(x4[u], x);
        if (GK32 && !is_q) {
          const uint32_t a[8] = {g4[u].x, g4[u].y, g4[u].z, g4[u].w, h4[u].x, h4[u].y, h4[u].z, h4[u].w};
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] = __uint_as_float(a[e]);
        } else {
          unpack8(g4[u], g);
        }
        rot.apply(g, -1.f);
        if (p.qw) {
          float ss = 0.f, ux = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            ss += x[e] * x[e];
            ux += g[e] * (is_q ? wq[e] : wk[e]) * x[e];
          }
          const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + p.eps);
          const float m = row_sum<LPR>(ux) * (1.f / D) * r * r;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float gw = g[e] * x[e] * r;
            if (is_q) aq[e] += gw;
            else ak[e] += gw;
            g[e] = r * (g[e] * (is_q ? wq[e] : wk[e]) - x[e] * m);
          }
        }
        if (row < p.rows) {
          __nv_bfloat16* dst = is_q ? p.dq + ((long long)t * p.Hq + row) * D : p.dk + ((long long)t * p.Hk + row - p.Hq) * D;
          reinterpret_cast<uint4*>(dst)[li] = pack8(g);
        }
      }
    }
  }
  if (!p.qw) return;
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      aq[e] += __shfl_xor_sync(0xffffffffu, aq[e], o);
      ak[e] += __shfl_xor_sync(0xffffffffu, ak[e], o);
    }
  if (sub == 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      red[warp][0][li * 8 + e] = aq[e];
      red[warp][1][li * 8 + e] = ak[e];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += NT) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) s += (&red[w][0][0])[i];
    p.part[(size_t)blockIdx.x * 2 * D + i] = s;
  }
}

// dw[c] = the sum of n records' column c: 32 columns a block, 32 strips of records
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* part, int n, int D, float* dqw, float* dkw) {
  __shared__ float s[32][33];
  griddep_wait();
  griddep_launch_dependents();
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), strip = threadIdx.x >> 5;
  float a = 0.f;
#pragma unroll 4
  for (int i = strip; i < n; i += 32) a += __ldcg(part + (size_t)i * 2 * D + c);
  s[strip][threadIdx.x & 31] = a;
  __syncthreads();
  if (strip == 0) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += s[i][threadIdx.x];
    if (c < D) dqw[c] = t;
    else if (dkw) dkw[c - D] = t;
  }
}

// -------------------------------------------------------------------------------------- host
// Warps that share a token: one when there are tokens enough to fill the GPU's warps (the angles are
// computed once per token), else as many as it takes, down to one pass of rows a warp.
static int parts_of(int T, int rows, int rpw, int sms) {
  const int passes = (rows + rpw - 1) / rpw;
  const long long want = ((long long)sms * 32 + T - 1) / T;
  return (int)(want < 1 ? 1 : want > passes ? passes : want);
}

template <int D>
static cudaError_t launch_fwd(const Params& p, bool inter, bool paged, bool f8, cudaStream_t st) {
  const long long items = (long long)p.T * p.parts;
  const dim3 grid((unsigned)((items + NW - 1) / NW));
  LaunchScope ls(paged ? "rope_paged" : "rope", st);
  if (paged) {
    if (f8) return inter ? launch_k(rope_fwd_kernel<D, true, true, true>, grid, dim3(NT), 0, st, true, p)
                         : launch_k(rope_fwd_kernel<D, false, true, true>, grid, dim3(NT), 0, st, true, p);
    return inter ? launch_k(rope_fwd_kernel<D, true, true, false>, grid, dim3(NT), 0, st, true, p)
                 : launch_k(rope_fwd_kernel<D, false, true, false>, grid, dim3(NT), 0, st, true, p);
  }
  return inter ? launch_k(rope_fwd_kernel<D, true, false, false>, grid, dim3(NT), 0, st, true, p)
               : launch_k(rope_fwd_kernel<D, false, false, false>, grid, dim3(NT), 0, st, true, p);
}
template <int D>
static cudaError_t launch_bwd(const Params& p, int grid, bool inter, bool gk32, cudaStream_t st) {
  LaunchScope ls("rope_bwd", st);
  if (gk32) return inter ? launch_k(rope_bwd_kernel<D, true, true>, dim3(grid), dim3(NT), 0, st, true, p)
                         : launch_k(rope_bwd_kernel<D, false, true>, dim3(grid), dim3(NT), 0, st, true, p);
  return inter ? launch_k(rope_bwd_kernel<D, true, false>, dim3(grid), dim3(NT), 0, st, true, p)
               : launch_k(rope_bwd_kernel<D, false, false>, dim3(grid), dim3(NT), 0, st, true, p);
}

constexpr size_t kStatusBytes = 256;
// Blocks of the backward: every warp of the GPU busy (the weight gradients are one record a block)
static int bwd_grid(int T, int rows, int rpw, int sms, int& parts) {
  parts = parts_of(T, rows, rpw, sms);
  const long long blocks = ((long long)T * parts + NW - 1) / NW;
  return (int)(blocks < sms * 4ll ? blocks : sms * 4ll);
}

static bool strides_ok(const void* p, long long ts, long long hs) {
  return aligned16(p) && ts >= 0 && hs >= 0 && ts % 8 == 0 && hs % 8 == 0;
}
static bool shape_ok(int d, int rot) { return (d == 64 || d == 128) && rot >= 16 && rot <= d && rot % 16 == 0; }
static bool sizes_ok(int T, int Hq, int Hk) {
  return T >= 0 && Hq >= 1 && Hk >= 0 && Hq <= 1024 && Hk <= 1024;
}
static bool weights_ok(const void* qw, const void* kw, int Hk) {
  return aligned16(qw) && aligned16(kw) && (qw != nullptr || kw == nullptr) && (qw == nullptr || Hk == 0 || kw != nullptr);
}

}  // namespace rope
}  // namespace hs2

using namespace hs2;

extern "C" {

hs2_status hs2_qk_norm_rope(const hs2_bf16* Q, const hs2_bf16* K, long long q_token_stride, long long q_head_stride,
                            long long k_token_stride, long long k_head_stride, const int32_t* positions,
                            const double* inv_freq, int T, int Hq, int Hk, int d, int rot, int interleaved,
                            float mscale, float eps, const void* q_weight, const void* k_weight, int weight_fp32,
                            hs2_bf16* q_out, hs2_bf16* k_out, hs2_stream stream) {
  if (!rope::sizes_ok(T, Hq, Hk) || !Q || !positions || !inv_freq || !q_out || !aligned16(q_out) ||
      !rope::strides_ok(Q, q_token_stride, q_head_stride) || !rope::weights_ok(q_weight, k_weight, Hk))
    return HS2_ERR_INVALID_ARG;
  if (Hk > 0 && (!K || !k_out || !aligned16(k_out) || !rope::strides_ok(K, k_token_stride, k_head_stride)))
    return HS2_ERR_INVALID_ARG;
  if (!rope::shape_ok(d, rot) || !device_is_sm100()) return HS2_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return HS2_OK;
  rope::Params p{};
  p.q = (const __nv_bfloat16*)Q; p.k = (const __nv_bfloat16*)K;
  p.q_ts = q_token_stride; p.q_hs = q_head_stride; p.k_ts = k_token_stride; p.k_hs = k_head_stride;
  p.pos = positions; p.inv_freq = inv_freq;
  p.qw = q_weight; p.kw = k_weight ? k_weight : q_weight; p.w_f32 = weight_fp32;
  p.T = T; p.Hq = Hq; p.Hk = Hk; p.rot = rot; p.rows = Hq + Hk;
  p.parts = rope::parts_of(T, p.rows, 256 / d, num_sms());
  p.eps = eps; p.mscale = mscale;
  p.q_out = (__nv_bfloat16*)q_out; p.k_out = (__nv_bfloat16*)k_out;
  const cudaError_t e = d == 128 ? rope::launch_fwd<128>(p, interleaved != 0, false, false, (cudaStream_t)stream)
                                 : rope::launch_fwd<64>(p, interleaved != 0, false, false, (cudaStream_t)stream);
  return e == cudaSuccess ? HS2_OK : HS2_ERR_CUDA;
}

size_t hs2_qk_norm_rope_paged_workspace_bytes(void) { return rope::kStatusBytes; }

hs2_status hs2_qk_norm_rope_paged(const hs2_bf16* Q, const hs2_bf16* K, const hs2_bf16* V, long long q_token_stride,
                                  long long q_head_stride, long long k_token_stride, long long k_head_stride,
                                  long long v_token_stride, long long v_head_stride, const int32_t* positions,
                                  const int32_t* slots, const double* inv_freq, int T, int Hq, int Hk, int d, int rot,
                                  int interleaved, float mscale, float eps, const void* q_weight,
                                  const void* k_weight, int weight_fp32, hs2_bf16* q_out, void* k_pages, void* v_pages,
                                  const long long* k_page_strides, const long long* v_page_strides, int n_pages,
                                  int page_size, int e4m3, float k_scale, float v_scale, void* workspace,
                                  size_t workspace_bytes, hs2_stream stream) {
  if (!rope::sizes_ok(T, Hq, Hk) || Hk < 1 || !Q || !K || !V || !positions || !slots || !inv_freq || !q_out ||
      !k_pages || !v_pages || !k_page_strides || !v_page_strides || n_pages < 1 || page_size < 1 ||
      (long long)n_pages * page_size > 0x7FFFFFFFll || !aligned16(q_out) || !aligned16(k_pages) ||
      !aligned16(v_pages) || !rope::strides_ok(Q, q_token_stride, q_head_stride) ||
      !rope::strides_ok(K, k_token_stride, k_head_stride) || !rope::strides_ok(V, v_token_stride, v_head_stride) ||
      !rope::weights_ok(q_weight, k_weight, Hk))
    return HS2_ERR_INVALID_ARG;
  if (!pool_strides_ok(k_page_strides, e4m3) || !pool_strides_ok(v_page_strides, e4m3)) return HS2_ERR_INVALID_ARG;
  if (e4m3 && !(k_scale > 0.f && k_scale < INFINITY && v_scale > 0.f && v_scale < INFINITY)) return HS2_ERR_INVALID_ARG;
  if (!rope::shape_ok(d, rot) || !device_is_sm100()) return HS2_ERR_UNSUPPORTED_SHAPE;
  if (!workspace || !aligned16(workspace) || workspace_bytes < rope::kStatusBytes) return HS2_ERR_WORKSPACE;
  if (T == 0) return HS2_OK;
  rope::Params p{};
  p.q = (const __nv_bfloat16*)Q; p.k = (const __nv_bfloat16*)K; p.v = (const __nv_bfloat16*)V;
  p.q_ts = q_token_stride; p.q_hs = q_head_stride; p.k_ts = k_token_stride; p.k_hs = k_head_stride;
  p.v_ts = v_token_stride; p.v_hs = v_head_stride;
  p.pos = positions; p.inv_freq = inv_freq; p.slots = slots;
  p.qw = q_weight; p.kw = k_weight; p.w_f32 = weight_fp32;
  p.T = T; p.Hq = Hq; p.Hk = Hk; p.rot = rot; p.rows = Hq + 2 * Hk;
  p.parts = rope::parts_of(T, p.rows, 256 / d, num_sms());
  p.eps = eps; p.mscale = mscale;
  p.q_out = (__nv_bfloat16*)q_out; p.k_pages = k_pages; p.v_pages = v_pages;
  p.kp_ps = k_page_strides[0]; p.kp_rs = k_page_strides[1]; p.kp_hs = k_page_strides[2];
  p.vp_ps = v_page_strides[0]; p.vp_rs = v_page_strides[1]; p.vp_hs = v_page_strides[2];
  p.page = page_size; p.n_pages = n_pages;
  p.k_inv = e4m3 ? 1.f / k_scale : 1.f; p.v_inv = e4m3 ? 1.f / v_scale : 1.f;
  p.st = (DevStatus*)workspace;
  const cudaError_t e = d == 128 ? rope::launch_fwd<128>(p, interleaved != 0, true, e4m3 != 0, (cudaStream_t)stream)
                                 : rope::launch_fwd<64>(p, interleaved != 0, true, e4m3 != 0, (cudaStream_t)stream);
  return e == cudaSuccess ? HS2_OK : HS2_ERR_CUDA;
}

size_t hs2_qk_norm_rope_bwd_workspace_bytes(int T, int Hq, int Hk, int d) {
  if (!rope::sizes_ok(T, Hq, Hk) || (d != 64 && d != 128)) return 0;
  const int sms = num_sms() > 0 ? num_sms() : 148;
  int parts = 1;
  const int grid = T > 0 ? rope::bwd_grid(T, Hq + Hk, 256 / d, sms, parts) : 0;
  return rope::kStatusBytes + (size_t)grid * 2 * d * sizeof(float);
}

hs2_status hs2_qk_norm_rope_bwd(const hs2_bf16* Q, const hs2_bf16* K, long long q_token_stride,
                                long long q_head_stride, long long k_token_stride, long long k_head_stride,
                                const int32_t* positions, const double* inv_freq, int T, int Hq, int Hk, int d,
                                int rot, int interleaved, float mscale, float eps, const void* q_weight,
                                const void* k_weight, int weight_fp32, const hs2_bf16* dq_out, const void* dk_out,
                                int dk_out_fp32, hs2_bf16* dQ, hs2_bf16* dK, float* dq_weight, float* dk_weight,
                                void* workspace, size_t workspace_bytes, hs2_stream stream) {
  if (!rope::sizes_ok(T, Hq, Hk) || !Q || !positions || !inv_freq || !dq_out || !dQ || !aligned16(dq_out) ||
      !aligned16(dQ) || !rope::strides_ok(Q, q_token_stride, q_head_stride) ||
      !rope::weights_ok(q_weight, k_weight, Hk))
    return HS2_ERR_INVALID_ARG;
  if (Hk > 0 && (!K || !dk_out || !dK || !aligned16(dk_out) || !aligned16(dK) ||
                 !rope::strides_ok(K, k_token_stride, k_head_stride)))
    return HS2_ERR_INVALID_ARG;
  if (q_weight && (!dq_weight || (Hk > 0 && !dk_weight))) return HS2_ERR_INVALID_ARG;
  if (!rope::shape_ok(d, rot) || !device_is_sm100()) return HS2_ERR_UNSUPPORTED_SHAPE;
  if (!workspace || !aligned16(workspace) || workspace_bytes < hs2_qk_norm_rope_bwd_workspace_bytes(T, Hq, Hk, d))
    return HS2_ERR_WORKSPACE;
  const cudaStream_t st = (cudaStream_t)stream;
  rope::Params p{};
  p.q = (const __nv_bfloat16*)Q; p.k = (const __nv_bfloat16*)K;
  p.q_ts = q_token_stride; p.q_hs = q_head_stride; p.k_ts = k_token_stride; p.k_hs = k_head_stride;
  p.pos = positions; p.inv_freq = inv_freq;
  p.qw = q_weight; p.kw = k_weight ? k_weight : q_weight; p.w_f32 = weight_fp32;
  p.T = T; p.Hq = Hq; p.Hk = Hk; p.rot = rot; p.rows = Hq + Hk;
  p.eps = eps; p.mscale = mscale;
  p.dq_out = (const __nv_bfloat16*)dq_out; p.dk_out = dk_out;
  p.dq = (__nv_bfloat16*)dQ; p.dk = (__nv_bfloat16*)dK;
  p.part = (float*)((uint8_t*)workspace + rope::kStatusBytes);
  int grid = 0;
  if (T > 0) {
    grid = rope::bwd_grid(T, p.rows, 256 / d, num_sms(), p.parts);
    const cudaError_t e = d == 128 ? rope::launch_bwd<128>(p, grid, interleaved != 0, dk_out_fp32 != 0, st)
                                   : rope::launch_bwd<64>(p, grid, interleaved != 0, dk_out_fp32 != 0, st);
    if (e != cudaSuccess) return HS2_ERR_CUDA;
  }
  if (q_weight) {
    LaunchScope ls("rope_dw", st);
    if (launch_k(rope::rope_dw_kernel, dim3(2 * d / 32), dim3(1024), 0, st, true, (const float*)p.part, grid, d,
                 dq_weight, Hk > 0 ? dk_weight : (float*)nullptr) != cudaSuccess)
      return HS2_ERR_CUDA;
  }
  return HS2_OK;
}

}  // extern "C"
