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
// All of it is bound by HBM (a few flops per byte; each row is read once and written once), and next to
// that by the issue slots, so the layout spares instructions. A lane owns two groups of 4 elements
// (8-byte accesses; d/8 lanes a row) chosen so that it holds both elements of its pairs: in the half
// layout groups 4 i and rot/2 + 4 i, interleaved 8 i and 8 i + 4; no element moves between lanes, only
// the row's sums do. The head weight is folded into the lane's cosines and sines,
//   y = r (x C + partner S),   C = m w cos, S = -+ m w_partner sin,
// 16 registers that stay over a token's heads (a warp works on the rows of ONE token), and products run
// two to an instruction (f32x2). The angles are computed once per (warp, token), shared out over the
// lanes, in 64 bits as turns t * f / 2 pi reduced to [-1/2, 1/2] (a 32-bit angle of position 10^6 is off
// by 0.06), while the token's first rows are on their way. Loads of several rows are issued before the
// first is used. All arithmetic is in 32 bits, rounded once at the store.
//
// Measured against a copy's 6.56 TB/s: 32k tokens of 64 + 1 heads of 128, 184 us (5.9 TB/s; 196 us when a
// long run holds the clocks at the power limit), their gradient 298 us (5.5; 304); 4,099 tokens of 32 + 8 heads
// into e4m3 pages 19.4 us (4.7): one wave of warps, each waiting for six batches of rows in turn. From 500 to 6,000 tokens a
// warp has a few such batches and little else: 1,000 tokens 9.9 us for 5.1 us of bytes, 3,000 24.0 for 15.2; their
// gradients, whose last passes run one at a time, 17.2 for 7.6 and 41.4 for 22.9. (Spills: up to 56 bytes a thread in the
// forward's kernels, 32 in the gradient's.) Tried
// and slower: rings in shared memory filled by cp.async for the gradient (368 us; it is the sums' chain that
// waits), more and smaller batches at a higher occupancy (492), L2 prefetch of a warp's rows (211 for the
// forward), streaming cache hints (no difference).
#include <type_traits>

#include "host_util.h"
#include "tc.cuh"

namespace hs2 {
namespace rope {

constexpr int NT = 128, NW = NT / 32;
constexpr int MAX_HALF = 64;  // rot / 2 at most

// What the cache holds: bf16, or e4m3 codes of x / scale, rounded once: where both scales are powers of two (E4M3_EXACT)
// the product with the reciprocal is the quotient, else codes8 looks twice.
enum Cache { BF16, E4M3_EXACT, E4M3 };

struct Params {
  const __nv_bfloat16 *q, *k, *v;
  long long q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;  // token and head strides in elements
  const int32_t* pos;
  const double* inv_freq;
  const void *qw, *kw;  // NULL: no norm
  int w_f32;
  int T, Hq, Hk, rot;
  int parts;   // warps that share a token's rows
  float eps, mscale;
  __nv_bfloat16 *q_out, *k_out;  // contiguous [T, Hq, D], [T, Hk, D]
  // paged form
  const int32_t* slots;
  void *k_pages, *v_pages;
  long long kp_ps, kp_rs, kp_hs, vp_ps, vp_rs, vp_hs;  // page, row and head strides in elements
  int page, n_pages;
  float k_inv, v_inv;  // reciprocals of an e4m3 cache's scales
  DevStatus* st;
  // backward
  const __nv_bfloat16* dq_out;
  union {  // (288 bytes in all: at 248, 256 and 296 a launch takes the host 0.3 us longer)
    const void* dk_out;
    struct { float k_scale, v_scale; };  // paged form
  };
  __nv_bfloat16 *dq, *dk;
  float* part;  // [grid][2][D] weight gradients of each block
};

// 8 values of a lane: x[0..3] its first group, x[4..7] its second
struct V8 {
  float x[8];
};
__device__ __forceinline__ void unpack4(const uint2& w, float* x) {
  x[0] = __uint_as_float(w.x << 16);
  x[1] = __uint_as_float(w.x & 0xFFFF0000u);
  x[2] = __uint_as_float(w.y << 16);
  x[3] = __uint_as_float(w.y & 0xFFFF0000u);
}
__device__ __forceinline__ uint2 pack4(const float* x) { return make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])); }
// four floats -> e4m3 codes (the first in the low byte), rounded to nearest even, saturating at 448
__device__ __forceinline__ uint32_t pack4_e4m3(const float* x) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[1]), "f"(x[0]));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[3]), "f"(x[2]));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
// d = a * b + c and d = a * b, elementwise
__device__ __forceinline__ void fma8(V8& d, const V8& a, const V8& b, const V8& c) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) ffma2(d.x[i], d.x[i + 1], a.x[i], a.x[i + 1], b.x[i], b.x[i + 1], c.x[i], c.x[i + 1]);
}
__device__ __forceinline__ void mul8(V8& d, const V8& a, const V8& b) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) fmul2(d.x[i], d.x[i + 1], a.x[i], a.x[i + 1], b.x[i], b.x[i + 1]);
}
__device__ __forceinline__ void scale8(V8& d, const V8& a, float b) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) fmul2(d.x[i], d.x[i + 1], a.x[i], a.x[i + 1], b, b);
}
__device__ __forceinline__ float dot8(const V8& a, const V8& b) {
  float s = 0.f, t = 0.f;
#pragma unroll
  for (int i = 0; i < 8; i += 2) ffma2(s, t, a.x[i], a.x[i + 1], b.x[i], b.x[i + 1], s, t);
  return s + t;
}

// Eight quotients x / s as e4m3 codes, each rounded once. Two products, 2^-20 of the quotient below and above it, nearly
// always have one code, the quotient's. Where they have not, a border between two codes lies within 2^-19 of the
// product with the reciprocal, and so does t, the nearest number of five significant bits, as all borders are; the sign
// of x - t s (one rounding: exact) tells the quotient's side of t, and any number there up to the next one has its code.
// 4,099 tokens of 32 + 8 heads: 19.4 us with powers of two, 20.5 us with other scales (22.7 with 0.03, whose quotients of one
// bf16 significand in 128 lie on a border).
template <Cache C>
__device__ __forceinline__ uint2 codes8(const V8& x, float s, float inv) {
  auto product = [&](float by) {
    V8 y;
    scale8(y, x, by);
    return make_uint2(pack4_e4m3(y.x), pack4_e4m3(y.x + 4));
  };
  if constexpr (C == E4M3_EXACT) return product(inv);
  uint2 code = product(inv * (1.f - 0x1p-20f));
  const uint2 high = product(inv * (1.f + 0x1p-20f));
  if ((code.x ^ high.x) | (code.y ^ high.y)) {
    V8 y;
    scale8(y, x, inv);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const unsigned t = (__float_as_uint(y.x[i]) + 0x40000u) & 0xFFF80000u;
      const float r = fmaf(-__uint_as_float(t), s, x.x[i]);
      if (r == 0.f) y.x[i] = __uint_as_float(t);
      else if (r == r) y.x[i] = __uint_as_float((int)(__float_as_uint(r) ^ t) < 0 ? t - 1 : t + 1);  // (no number: as it is)
    }
    code = make_uint2(pack4_e4m3(y.x), pack4_e4m3(y.x + 4));
  }
  return code;
}

// Which elements a lane owns, and its pairs: half layout, group one's element i with group two's;
// interleaved, elements 2 i and 2 i + 1 of each group. Lanes past the rotated part own two adjacent
// groups that pass.
template <int D, bool INTER>
struct Lane {
  static constexpr int LPR = D / 8;  // lanes of a row
  int a, b;                          // first element of each group
  bool on;                           // its elements are rotated
  __device__ __forceinline__ Lane(int lane, int rot) {
    const int li = lane % LPR;
    on = li * 8 < rot;
    a = INTER || !on ? li * 8 : li * 4;
    b = INTER || !on ? a + 4 : rot / 2 + li * 4;
  }
  __device__ __forceinline__ static V8 swap(const V8& x) {  // each element's partner
    V8 y;
#pragma unroll
    for (int i = 0; i < 8; ++i) y.x[i] = x.x[INTER ? i ^ 1 : i ^ 4];
    return y;
  }
  // cosines, and sines signed as the rotation applies them (y = x c + partner s), both times m
  __device__ __forceinline__ void read(const float2* sc, V8& c, V8& s) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = on ? sc[INTER ? a / 2 + i / 2 : a + i % 4] : make_float2(1.f, 0.f);
      const bool first = INTER ? i % 2 == 0 : i < 4;
      c.x[i] = v.x;
      s.x[i] = first ? -v.y : v.y;
    }
  }
  __device__ __forceinline__ void weights(const void* w, int f32, V8& v) const {
    if (!w) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v.x[i] = 1.f;
    } else if (f32) {
      const float4 p = __ldg((const float4*)((const float*)w + a)), q = __ldg((const float4*)((const float*)w + b));
      v.x[0] = p.x; v.x[1] = p.y; v.x[2] = p.z; v.x[3] = p.w;
      v.x[4] = q.x; v.x[5] = q.y; v.x[6] = q.z; v.x[7] = q.w;
    } else {
      unpack4(__ldg((const uint2*)((const __nv_bfloat16*)w + a)), v.x);
      unpack4(__ldg((const uint2*)((const __nv_bfloat16*)w + b)), v.x + 4);
    }
  }
};

// The whole warp: cosines and sines of position t, times m, into the warp's buffer
__device__ __forceinline__ void angles(int t, const double* inv_freq, int half, float mscale, int lane, float2* sc) {
  __syncwarp();
  for (int i = lane; i < half; i += 32) {
    const double turns = (double)t * __ldg(inv_freq + i) * 0.15915494309189533577;  // 1 / (2 pi)
    float sn, cn;
    sincospif((float)(2.0 * (turns - rint(turns))), &sn, &cn);
    sc[i] = make_float2(cn * mscale, sn * mscale);
  }
  __syncwarp();
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One warp per (token, part): a part is a run of the token's passes, a pass 32 / LPR rows: first the
// passes of the queries, then the keys', then (paged) the values'.
template <int D, bool INTER, bool PAGED, Cache C>
__global__ void __launch_bounds__(NT, 8) rope_fwd_kernel(Params p) {
  constexpr bool F8 = C != BF16;
  constexpr int LPR = D / 8, RPW = 32 / LPR, U = 4;
  __shared__ float2 sc[NW][MAX_HALF];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / LPR;
  const long long item = (long long)blockIdx.x * NW + warp;
  griddep_wait();
  griddep_launch_dependents();
  const int t = (int)(item / p.parts), part = (int)(item % p.parts);
  if (t >= p.T) return;
  const int pos = p.pos[t];
  int slot = 0;
  if (PAGED) {
    slot = p.slots[t];
    if (slot < 0) return;  // a padding row: nothing of it is read or written
  }
  const Lane<D, INTER> own(lane, p.rot);
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
  const int nq = (p.Hq + RPW - 1) / RPW, nk = (p.Hk + RPW - 1) / RPW;  // passes
  const int n_pass = nq + (PAGED ? 2 : 1) * nk;
  const int per = (n_pass + p.parts - 1) / p.parts;
  const int p0 = part * per, p1 = min(n_pass, p0 + per);
  if (p0 >= p1) return;
  bool fresh = false;  // the warp's angles are computed (while its first rows are on their way)

  // rows sub, sub + RPW, .. of passes [i0, i1) of H heads: x -> y -> put
  auto rows = [&](int i0, int i1, int H, const __nv_bfloat16* src, long long hs, const void* w, auto put) {
    V8 C, S;
    for (int i = i0; i < i1; i += U) {
      uint2 xa[U], xb[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = (i + u) * RPW + sub;
        xa[u] = xb[u] = make_uint2(0u, 0u);
        if (i + u < i1 && h < H) {
          xa[u] = *reinterpret_cast<const uint2*>(src + h * hs + own.a);
          xb[u] = *reinterpret_cast<const uint2*>(src + h * hs + own.b);
        }
      }
      if (i == i0) {
        V8 c, s, wv;
        own.weights(w, p.w_f32, wv);
        if (!fresh) angles(pos, p.inv_freq, p.rot / 2, p.mscale, lane, sc[warp]);
        fresh = true;
        own.read(sc[warp], c, s);
        mul8(C, wv, c);
        mul8(S, Lane<D, INTER>::swap(wv), s);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i + u >= i1) break;  // (warp-uniform)
        const int h = (i + u) * RPW + sub;
        V8 x, y;
        unpack4(xa[u], x.x);
        unpack4(xb[u], x.x + 4);
        mul8(y, x, C);
        if (own.on) fma8(y, Lane<D, INTER>::swap(x), S, y);
        if (w) scale8(y, y, rsqrtf(row_sum<LPR>(dot8(x, x)) * (1.f / D) + p.eps));
        if (h < H) put(h, y);
      }
    }
  };
  if (p0 < nq)
    rows(p0, min(p1, nq), p.Hq, p.q + t * p.q_ts, p.q_hs, p.qw, [&](int h, const V8& y) {
      __nv_bfloat16* dst = p.q_out + ((long long)t * p.Hq + h) * D;
      *reinterpret_cast<uint2*>(dst + own.a) = pack4(y.x);
      *reinterpret_cast<uint2*>(dst + own.b) = pack4(y.x + 4);
    });
  if (p1 > nq && p0 < nq + nk)
    rows(max(p0, nq) - nq, min(p1, nq + nk) - nq, p.Hk, p.k + t * p.k_ts, p.k_hs, p.kw, [&](int h, V8& y) {
      if (!PAGED) {
        __nv_bfloat16* dst = p.k_out + ((long long)t * p.Hk + h) * D;
        *reinterpret_cast<uint2*>(dst + own.a) = pack4(y.x);
        *reinterpret_cast<uint2*>(dst + own.b) = pack4(y.x + 4);
      } else if (kc >= 0) {
        const long long at = kc + h * p.kp_hs;
        if (F8) {
          const uint2 code = codes8<C>(y, p.k_scale, p.k_inv);
          *reinterpret_cast<uint32_t*>((uint8_t*)p.k_pages + at + own.a) = code.x;
          *reinterpret_cast<uint32_t*>((uint8_t*)p.k_pages + at + own.b) = code.y;
        } else {
          *reinterpret_cast<uint2*>((__nv_bfloat16*)p.k_pages + at + own.a) = pack4(y.x);
          *reinterpret_cast<uint2*>((__nv_bfloat16*)p.k_pages + at + own.b) = pack4(y.x + 4);
        }
      }
    });
  if (PAGED && vc >= 0) {  // the values as they are, 8 adjacent elements a lane, U passes on their way at once
    const int li8 = (lane % LPR) * 8;
    const __nv_bfloat16* src = p.v + t * p.v_ts + li8;
    for (int i = max(p0, nq + nk); i < p1; i += U) {
      uint4 w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = (i + u - nq - nk) * RPW + sub;
        if (i + u < p1 && h < p.Hk) w[u] = *reinterpret_cast<const uint4*>(src + h * p.v_hs);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = (i + u - nq - nk) * RPW + sub;
        if (i + u >= p1 || h >= p.Hk) continue;
        const long long at = vc + h * p.vp_hs + li8;
        if (F8) {
          V8 x;
          unpack4(make_uint2(w[u].x, w[u].y), x.x);
          unpack4(make_uint2(w[u].z, w[u].w), x.x + 4);
          *reinterpret_cast<uint2*>((uint8_t*)p.v_pages + at) = codes8<C>(x, p.v_scale, p.v_inv);
        } else {
          *reinterpret_cast<uint4*>((__nv_bfloat16*)p.v_pages + at) = w[u];
        }
      }
    }
  }
}

// Backward: warps stride over (token, part) items and keep the weight gradients of their 8 elements
// in registers; a block adds its warps' in a fixed order and writes one record (rope_dw_kernel adds
// the records, also in a fixed order: the result does not vary from run to run).
template <int D, bool INTER, bool GK32>
__global__ void __launch_bounds__(NT, 4) rope_bwd_kernel(Params p) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, U = 4;
  __shared__ float2 sc[NW][MAX_HALF];
  __shared__ float red[NW][2][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / LPR;
  griddep_wait();
  griddep_launch_dependents();
  const Lane<D, INTER> own(lane, p.rot);
  V8 aq, ak;  // weight gradients
#pragma unroll
  for (int e = 0; e < 8; ++e) aq.x[e] = ak.x[e] = 0.f;
  const int nq = (p.Hq + RPW - 1) / RPW, nk = (p.Hk + RPW - 1) / RPW, n_pass = nq + nk;  // passes
  const int per = (n_pass + p.parts - 1) / p.parts;
  const long long items = (long long)p.T * p.parts;

  // passes [i0, i1) of H heads with the gradients g (bf16, or fp32) of [H, D]; steps of U passes
  // without a row missing first, as in the forward pass
  V8 c, s;
  int pos = 0, t = -1;
  bool fresh = false;  // the token's angles are computed (while its first rows are on their way)
  auto rows = [&](int i0, int i1, int H, const __nv_bfloat16* src, long long hs, const void* w, const void* g, auto g32,
                  __nv_bfloat16* dst, V8& acc) {
    constexpr bool G32 = decltype(g32)::value;
    constexpr int GB = G32 ? 4 : 2;
    V8 wv;
    own.weights(w, p.w_f32, wv);
    const __nv_bfloat16 *xa = src + (i0 * RPW + sub) * hs + own.a, *xb = xa + (own.b - own.a);
    const long long step = RPW * hs;
    const char *ga = (const char*)g + ((i0 * RPW + sub) * D + own.a) * GB, *gb = ga + (own.b - own.a) * GB;
    __nv_bfloat16 *da = dst + (i0 * RPW + sub) * D + own.a, *db = da + (own.b - own.a);
    auto run = [&](int i, auto n_, auto full_) {
      constexpr int N = decltype(n_)::value;
      constexpr bool FULL = decltype(full_)::value;
      const bool on = FULL || i * RPW + sub < H;
      uint2 va[N], vb[N];
      V8 gv[G32 ? N : 1];
      uint2 ha[N], hb[N];
#pragma unroll
      for (int u = 0; u < N; ++u) {
        va[u] = vb[u] = ha[u] = hb[u] = make_uint2(0u, 0u);
        if (w && on) {
          va[u] = *reinterpret_cast<const uint2*>(xa);
          vb[u] = *reinterpret_cast<const uint2*>(xb);
        }
        xa += step;
        xb += step;
        if constexpr (G32) {
          const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
          const float4 q0 = on ? *reinterpret_cast<const float4*>(ga + u * (RPW * D * GB)) : z;
          const float4 q1 = on ? *reinterpret_cast<const float4*>(gb + u * (RPW * D * GB)) : z;
          gv[u].x[0] = q0.x; gv[u].x[1] = q0.y; gv[u].x[2] = q0.z; gv[u].x[3] = q0.w;
          gv[u].x[4] = q1.x; gv[u].x[5] = q1.y; gv[u].x[6] = q1.z; gv[u].x[7] = q1.w;
        } else if (on) {
          ha[u] = *reinterpret_cast<const uint2*>(ga + u * (RPW * D * GB));
          hb[u] = *reinterpret_cast<const uint2*>(gb + u * (RPW * D * GB));
        }
      }
      if (!fresh) {
        angles(pos, p.inv_freq, p.rot / 2, p.mscale, lane, sc[warp]);
        own.read(sc[warp], c, s);
        s = Lane<D, INTER>::swap(s);  // the transpose: n = y c + partner s, with the partner's s
        fresh = true;
      }
#pragma unroll
      for (int u = 0; u < N; ++u) {
        V8 y, n;
        if constexpr (G32) {
          y = gv[u];
        } else {
          unpack4(ha[u], y.x);
          unpack4(hb[u], y.x + 4);
        }
        mul8(n, y, c);
        if (own.on) fma8(n, Lane<D, INTER>::swap(y), s, n);
        if (w) {
          V8 x, u8, gx;
          unpack4(va[u], x.x);
          unpack4(vb[u], x.x + 4);
          mul8(u8, n, wv);
          mul8(gx, n, x);
          const float r = rsqrtf(row_sum<LPR>(dot8(x, x)) * (1.f / D) + p.eps);
          const float m = row_sum<LPR>(dot8(u8, x)) * (1.f / D) * r * r * r;
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            ffma2(acc.x[e], acc.x[e + 1], gx.x[e], gx.x[e + 1], r, r, acc.x[e], acc.x[e + 1]);
            fmul2(u8.x[e], u8.x[e + 1], u8.x[e], u8.x[e + 1], r, r);
            ffma2(n.x[e], n.x[e + 1], x.x[e], x.x[e + 1], -m, -m, u8.x[e], u8.x[e + 1]);
          }
        }
        if (on) {
          *reinterpret_cast<uint2*>(da + u * (RPW * D)) = pack4(n.x);
          *reinterpret_cast<uint2*>(db + u * (RPW * D)) = pack4(n.x + 4);
        }
      }
      ga += N * (RPW * D * GB); gb += N * (RPW * D * GB);
      da += N * (RPW * D); db += N * (RPW * D);
    };
    const int full = min(i1, H / RPW);
    int i = i0;
    for (; i + U <= full; i += U) run(i, std::integral_constant<int, U>{}, std::true_type{});
    for (; i < i1; ++i) run(i, std::integral_constant<int, 1>{}, std::false_type{});
  };
  for (long long item = (long long)blockIdx.x * NW + warp; item < items; item += (long long)gridDim.x * NW) {
    const int part = (int)(item % p.parts);
    t = (int)(item / p.parts);
    const int p0 = part * per, p1 = min(n_pass, p0 + per);
    if (p0 >= p1) continue;
    pos = p.pos[t];
    fresh = false;
    if (p0 < nq)
      rows(p0, min(p1, nq), p.Hq, p.q + t * p.q_ts, p.q_hs, p.qw, p.dq_out + (long long)t * p.Hq * D, std::false_type{},
           p.dq + (long long)t * p.Hq * D, aq);
    if (p1 > nq)
      rows(max(p0, nq) - nq, p1 - nq, p.Hk, p.k + t * p.k_ts, p.k_hs, p.kw,
           (const char*)p.dk_out + (long long)t * p.Hk * D * (GK32 ? 4 : 2), std::integral_constant<bool, GK32>{},
           p.dk + (long long)t * p.Hk * D, ak);
  }
  if (!p.qw) return;
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      aq.x[e] += __shfl_xor_sync(0xffffffffu, aq.x[e], o);
      ak.x[e] += __shfl_xor_sync(0xffffffffu, ak.x[e], o);
    }
  if (sub == 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int at = e < 4 ? own.a + e : own.b + e - 4;
      red[warp][0][at] = aq.x[e];
      red[warp][1][at] = ak.x[e];
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
  constexpr int U = 19;  // records in flight: one round of reads for the 592 there are at most on 148 SMs
  for (int i = strip; i < n; i += 32 * U) {
    float v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = i + 32 * u < n ? __ldcg(part + (size_t)(i + 32 * u) * 2 * D + c) : 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) a += v[u];
  }
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
// Passes of a token: 256 / d rows at a time of the queries, and of the keys (and values) n times
static int passes_of(int Hq, int Hk, int n, int d) {
  const int rpw = 256 / d;
  return (Hq + rpw - 1) / rpw + n * ((Hk + rpw - 1) / rpw);
}
// Warps that share a token: what takes the fewest steps, in waves of the `warps` that the GPU holds at
// once, with a start (position, angles: about ANGLE passes) for each of them. Measured against as many as
// fill the GPU, rounded up: 700 tokens of 64 + 1 heads 8.1 and 9.6 us, 6,000 tokens 43.2 and 46.7 us.
constexpr int ANGLE = 8;
static int parts_of(int T, int passes, int warps) {
  long long best = 0;
  int parts = 1;
  for (int n = 1;;) {  // the fewest warps for each number of passes a warp
    const int per = (passes + n - 1) / n;
    const long long waves = ((long long)T * n + warps - 1) / warps, cost = waves * (per + ANGLE);
    if (n == 1 || cost < best) { best = cost; parts = n; }
    if (per == 1) break;
    n = (passes + per - 2) / (per - 1);
  }
  return parts;
}

template <int D, bool PAGED, Cache C>
static cudaError_t launch_fwd(const Params& p, bool inter, cudaStream_t st) {
  const long long items = (long long)p.T * p.parts;
  const dim3 grid((unsigned)((items + NW - 1) / NW));
  LaunchScope ls(PAGED ? "rope_paged" : "rope", st);
  return inter ? launch_k(rope_fwd_kernel<D, true, PAGED, C>, grid, dim3(NT), 0, st, true, p)
               : launch_k(rope_fwd_kernel<D, false, PAGED, C>, grid, dim3(NT), 0, st, true, p);
}
template <int D>
static cudaError_t launch_paged(const Params& p, bool inter, Cache c, cudaStream_t st) {
  return c == BF16 ? launch_fwd<D, true, BF16>(p, inter, st)
         : c == E4M3 ? launch_fwd<D, true, E4M3>(p, inter, st) : launch_fwd<D, true, E4M3_EXACT>(p, inter, st);
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
static int bwd_grid(int T, int passes, int sms, int& parts) {
  parts = parts_of(T, passes, sms * 4 * NW);
  const long long blocks = ((long long)T * parts + NW - 1) / NW;
  return (int)(blocks < sms * 4ll ? blocks : sms * 4ll);
}

static bool power_of_two(float s) { return (1.f / s) * (double)s == 1.0; }
static bool strides_ok(const void* p, long long ts, long long hs) {
  return aligned16(p) && ts >= 0 && hs >= 0 && ts % 8 == 0 && hs % 8 == 0;
}
static bool shape_ok(int d, int rot) { return (d == 64 || d == 128) && rot >= 16 && rot <= d && rot % 16 == 0; }
static bool numbers_ok(float mscale, float eps) { return fabsf(mscale) < INFINITY && eps >= 0.f && eps < INFINITY; }
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
  if (!rope::sizes_ok(T, Hq, Hk) || (T > 0 && (!Q || !positions || !q_out)) || !inv_freq || !aligned16(q_out) ||
      !rope::strides_ok(Q, q_token_stride, q_head_stride) || !rope::weights_ok(q_weight, k_weight, Hk) ||
      !rope::numbers_ok(mscale, eps))
    return HS2_ERR_INVALID_ARG;
  if (Hk > 0 && ((T > 0 && (!K || !k_out)) || !aligned16(k_out) || !rope::strides_ok(K, k_token_stride, k_head_stride)))
    return HS2_ERR_INVALID_ARG;
  if (!rope::shape_ok(d, rot) || !device_is_sm100()) return HS2_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return HS2_OK;
  rope::Params p{};
  p.q = (const __nv_bfloat16*)Q; p.k = (const __nv_bfloat16*)K;
  p.q_ts = q_token_stride; p.q_hs = q_head_stride; p.k_ts = k_token_stride; p.k_hs = k_head_stride;
  p.pos = positions; p.inv_freq = inv_freq;
  p.qw = q_weight; p.kw = k_weight ? k_weight : q_weight; p.w_f32 = weight_fp32;
  p.T = T; p.Hq = Hq; p.Hk = Hk; p.rot = rot;
  p.parts = rope::parts_of(T, rope::passes_of(Hq, Hk, 1, d), num_sms() * 32);
  p.eps = eps; p.mscale = mscale;
  p.q_out = (__nv_bfloat16*)q_out; p.k_out = (__nv_bfloat16*)k_out;
  const cudaError_t e = d == 128 ? rope::launch_fwd<128, false, rope::BF16>(p, interleaved != 0, (cudaStream_t)stream)
                                 : rope::launch_fwd<64, false, rope::BF16>(p, interleaved != 0, (cudaStream_t)stream);
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
  if (!rope::sizes_ok(T, Hq, Hk) || Hk < 1 || (T > 0 && (!Q || !K || !V || !positions || !slots || !q_out)) || !inv_freq ||
      !rope::numbers_ok(mscale, eps) || !k_pages || !v_pages || !k_page_strides || !v_page_strides || n_pages < 1 || page_size < 1 ||
      (long long)n_pages * page_size > 0x7FFFFFFFll || !aligned16(q_out) || !aligned16(k_pages) ||
      !aligned16(v_pages) || !rope::strides_ok(Q, q_token_stride, q_head_stride) ||
      !rope::strides_ok(K, k_token_stride, k_head_stride) || !rope::strides_ok(V, v_token_stride, v_head_stride) ||
      !rope::weights_ok(q_weight, k_weight, Hk))
    return HS2_ERR_INVALID_ARG;
  if (!pool_strides_ok(k_page_strides, e4m3) || !pool_strides_ok(v_page_strides, e4m3)) return HS2_ERR_INVALID_ARG;
  if (e4m3 && !(cache_scale_ok(k_scale) && cache_scale_ok(v_scale))) return HS2_ERR_INVALID_ARG;
  if (!rope::shape_ok(d, rot) || !device_is_sm100()) return HS2_ERR_UNSUPPORTED_SHAPE;
  if (!workspace || !aligned16(workspace) || workspace_bytes < rope::kStatusBytes) return HS2_ERR_WORKSPACE;
  if (T == 0) return HS2_OK;
  rope::Params p{};
  p.q = (const __nv_bfloat16*)Q; p.k = (const __nv_bfloat16*)K; p.v = (const __nv_bfloat16*)V;
  p.q_ts = q_token_stride; p.q_hs = q_head_stride; p.k_ts = k_token_stride; p.k_hs = k_head_stride;
  p.v_ts = v_token_stride; p.v_hs = v_head_stride;
  p.pos = positions; p.inv_freq = inv_freq; p.slots = slots;
  p.qw = q_weight; p.kw = k_weight; p.w_f32 = weight_fp32;
  p.T = T; p.Hq = Hq; p.Hk = Hk; p.rot = rot;
  p.parts = rope::parts_of(T, rope::passes_of(Hq, Hk, 2, d), num_sms() * 32);
  p.eps = eps; p.mscale = mscale;
  p.q_out = (__nv_bfloat16*)q_out; p.k_pages = k_pages; p.v_pages = v_pages;
  p.kp_ps = k_page_strides[0]; p.kp_rs = k_page_strides[1]; p.kp_hs = k_page_strides[2];
  p.vp_ps = v_page_strides[0]; p.vp_rs = v_page_strides[1]; p.vp_hs = v_page_strides[2];
  p.page = page_size; p.n_pages = n_pages;
  rope::Cache cache = rope::BF16;
  if (e4m3) {
    p.k_scale = k_scale; p.v_scale = v_scale;
    p.k_inv = 1.f / k_scale; p.v_inv = 1.f / v_scale;
    cache = rope::power_of_two(k_scale) && rope::power_of_two(v_scale) ? rope::E4M3_EXACT : rope::E4M3;
  }
  p.st = (DevStatus*)workspace;
  const cudaError_t e = d == 128 ? rope::launch_paged<128>(p, interleaved != 0, cache, (cudaStream_t)stream)
                                 : rope::launch_paged<64>(p, interleaved != 0, cache, (cudaStream_t)stream);
  return e == cudaSuccess ? HS2_OK : HS2_ERR_CUDA;
}

size_t hs2_qk_norm_rope_bwd_workspace_bytes(int T, int Hq, int Hk, int d) {
  if (!rope::sizes_ok(T, Hq, Hk) || (d != 64 && d != 128)) return 0;
  const int sms = num_sms() > 0 ? num_sms() : 148;
  int parts = 1;
  const int grid = T > 0 ? rope::bwd_grid(T, rope::passes_of(Hq, Hk, 1, d), sms, parts) : 0;
  return rope::kStatusBytes + (size_t)grid * 2 * d * sizeof(float);
}

hs2_status hs2_qk_norm_rope_bwd(const hs2_bf16* Q, const hs2_bf16* K, long long q_token_stride,
                                long long q_head_stride, long long k_token_stride, long long k_head_stride,
                                const int32_t* positions, const double* inv_freq, int T, int Hq, int Hk, int d,
                                int rot, int interleaved, float mscale, float eps, const void* q_weight,
                                const void* k_weight, int weight_fp32, const hs2_bf16* dq_out, const void* dk_out,
                                int dk_out_fp32, hs2_bf16* dQ, hs2_bf16* dK, float* dq_weight, float* dk_weight,
                                void* workspace, size_t workspace_bytes, hs2_stream stream) {
  if (!rope::sizes_ok(T, Hq, Hk) || (T > 0 && (!Q || !positions || !dq_out || !dQ)) || !inv_freq || !aligned16(dq_out) ||
      !aligned16(dQ) || !rope::strides_ok(Q, q_token_stride, q_head_stride) ||
      !rope::weights_ok(q_weight, k_weight, Hk) || !rope::numbers_ok(mscale, eps))
    return HS2_ERR_INVALID_ARG;
  if (Hk > 0 && ((T > 0 && (!K || !dk_out || !dK)) || !aligned16(dk_out) || !aligned16(dK) ||
                 !rope::strides_ok(K, k_token_stride, k_head_stride)))
    return HS2_ERR_INVALID_ARG;
  if (q_weight && (!dq_weight || (Hk > 0 && !dk_weight))) return HS2_ERR_INVALID_ARG;
  if (!rope::shape_ok(d, rot) || !device_is_sm100()) return HS2_ERR_UNSUPPORTED_SHAPE;
  if (q_weight && (!workspace || !aligned16(workspace) || workspace_bytes < hs2_qk_norm_rope_bwd_workspace_bytes(T, Hq, Hk, d)))
    return HS2_ERR_WORKSPACE;
  const cudaStream_t st = (cudaStream_t)stream;
  rope::Params p{};
  p.q = (const __nv_bfloat16*)Q; p.k = (const __nv_bfloat16*)K;
  p.q_ts = q_token_stride; p.q_hs = q_head_stride; p.k_ts = k_token_stride; p.k_hs = k_head_stride;
  p.pos = positions; p.inv_freq = inv_freq;
  p.qw = q_weight; p.kw = k_weight ? k_weight : q_weight; p.w_f32 = weight_fp32;
  p.T = T; p.Hq = Hq; p.Hk = Hk; p.rot = rot;
  p.eps = eps; p.mscale = mscale;
  p.dq_out = (const __nv_bfloat16*)dq_out; p.dk_out = dk_out;
  p.dq = (__nv_bfloat16*)dQ; p.dk = (__nv_bfloat16*)dK;
  p.part = q_weight ? (float*)((uint8_t*)workspace + rope::kStatusBytes) : nullptr;
  int grid = 0;
  if (T > 0) {
    grid = rope::bwd_grid(T, rope::passes_of(Hq, Hk, 1, d), num_sms(), p.parts);
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
