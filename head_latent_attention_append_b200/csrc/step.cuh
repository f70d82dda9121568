// What a ragged serving step runs around the attention: the plan of its page
// tables and slots, the norms of the two latents with the paged write, and
// the norms and rotation of the query heads.
//
// The pages cache one latent and one position key per token ("Latent
// Attention Meets RoPE", "Two small, telling details") and leave open how
// tokens find their cache rows and whether the latents are normalised; the
// norms here are RMS norms, y = x / sqrt(mean(x^2) + eps) * gamma, and the
// rotation is the library's (interleaved pairs, angle pos * theta_i).
#pragma once
#include "common.cuh"
#include "sm100.cuh"

namespace mla {
namespace step {

// ------------------------------------------------------------------- plan
// Requests are admitted in order while their new tokens fit the row budget
// and their new pages the free list, so the admitted ones are a prefix and
// two running sums decide everything:
//   tok[b] = sum_{b' <= b} new[b'],
//   pg[b]  = sum_{b' <= b} (ceil((past + new) / 64) - ceil(past / 64)).
// The work is latency: 8 bytes in and 12 out per request, 16 out per row.  So
// it is one launch, in which every CTA repeats the two sums over all requests
// (a few microseconds up to thousands of requests, from L2) instead of one
// kernel making them and a second one waiting for it; then each CTA writes
// its share of requests, new pages and rows, each row finding its request by
// a binary search in shared memory.
constexpr int PLAN_THREADS = 512;
constexpr int PLAN_MAX_B = 16384;  // the two sums of every request sit in shared memory

struct PlanArgs {
  const int32_t* new_len;     // [B]
  const int32_t* past_len;    // [B]
  const int32_t* free_pages;  // [n_free]
  int32_t* page_table;        // [B][max_pages]
  int32_t* q_start;           // [B+1]
  int32_t* kv_len;            // [B]
  int32_t* seq_idx;           // [rows]
  int32_t* pos;               // [rows]
  int64_t* slot;              // [rows]
  int32_t* counts;            // [3]
  int32_t* err;               // or null
  int B, n_free, max_pages, num_pages, rows;
};

// Sums that stop at `cap` (< 2^31), which keeps them associative and in 32
// bits whatever the lengths are.
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b, uint32_t cap) { return min(a + b, cap); }

// A request's new tokens, cached pages and new pages; one whose lengths are
// negative or pass its page table counts as empty.
struct PlanReq {
  int n, have, need;
  bool ok;
};
__device__ __forceinline__ PlanReq plan_req(const PlanArgs& a, int b) {
  const int n = a.new_len[b], p = a.past_len[b];
  const long long end = (long long)n + p;
  PlanReq r{0, 0, 0, n >= 0 && p >= 0 && end <= (long long)a.max_pages * 64};
  if (r.ok) {
    r.n = n;
    r.have = (int)(((long long)p + 63) >> 6);
    r.need = (int)((end + 63) >> 6) - r.have;
  }
  return r;
}

// Largest i in [0, n) with s[i] <= x (s non-decreasing, s[0] <= x).
__device__ __forceinline__ int plan_find(const uint32_t* s, int n, uint32_t x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(PLAN_THREADS) plan_kernel(const PlanArgs a) {
  extern __shared__ uint32_t plan_smem[];
  uint32_t* const qs = plan_smem;             // [B+1] first row of each request
  uint32_t* const pg = plan_smem + a.B + 1;   // [B+1] first new page of each request
  __shared__ uint32_t wt[PLAN_THREADS / 32], wp[PLAN_THREADS / 32];
  __shared__ uint32_t admitted, rows_used, pages_used;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const uint32_t cap_t = (uint32_t)a.rows + 1, cap_p = (uint32_t)a.n_free + 1;
  if (tid == 0) admitted = rows_used = pages_used = 0;

  // This thread's requests are consecutive; its sums, then the block's.
  const int chunk = ceil_div(a.B, PLAN_THREADS);
  const int lo = min(a.B, tid * chunk), hi = min(a.B, lo + chunk);
  uint32_t st = 0, sp = 0;
  for (int b = lo; b < hi; ++b) {
    const PlanReq r = plan_req(a, b);
    if (!r.ok && blockIdx.x == 0) flag_error(a.err, kErrBounds);
    st = sat_add(st, r.n, cap_t);
    sp = sat_add(sp, r.need, cap_p);
  }
  uint32_t it = st, ip = sp;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t yt = __shfl_up_sync(0xffffffffu, it, o), yp = __shfl_up_sync(0xffffffffu, ip, o);
    if (lane >= o) {
      it = sat_add(it, yt, cap_t);
      ip = sat_add(ip, yp, cap_p);
    }
  }
  if (lane == 31) {
    wt[wid] = it;
    wp[wid] = ip;
  }
  uint32_t et = __shfl_up_sync(0xffffffffu, it, 1), ep = __shfl_up_sync(0xffffffffu, ip, 1);
  if (lane == 0) et = ep = 0;
  __syncthreads();
  for (int i = 0; i < wid; ++i) {
    et = sat_add(et, wt[i], cap_t);
    ep = sat_add(ep, wp[i], cap_p);
  }
  uint32_t my_adm = 0, my_rows = 0, my_pages = 0;
  for (int b = lo; b < hi; ++b) {
    const PlanReq r = plan_req(a, b);
    qs[b] = et;
    pg[b] = ep;
    et = sat_add(et, r.n, cap_t);
    ep = sat_add(ep, r.need, cap_p);
    if (et < cap_t && ep < cap_p) {  // fits, and so does every request before it
      ++my_adm;
      my_rows = et;
      my_pages = ep;
    }
  }
  if (my_adm) {
    atomicAdd(&admitted, my_adm);
    atomicMax(&rows_used, my_rows);
    atomicMax(&pages_used, my_pages);
  }
  __syncthreads();
  const uint32_t nr = rows_used, np = pages_used, adm = admitted;
  // A refused request starts where the admitted ones end, so it has no rows.
  for (int b = lo; b < hi; ++b) {
    qs[b] = min(qs[b], nr);
    pg[b] = min(pg[b], np);
  }
  if (tid == 0) {
    qs[a.B] = nr;
    pg[a.B] = np;
  }
  __syncthreads();

  const int g = blockIdx.x * PLAN_THREADS + tid, step = gridDim.x * PLAN_THREADS;
  for (int b = g; b <= a.B; b += step) {
    a.q_start[b] = (int)qs[b];
    if (b == a.B) break;
    const PlanReq r = plan_req(a, b);
    // A refused request keeps its cached tokens; lengths that make no sense count as an empty cache.
    a.kv_len[b] = r.ok ? a.past_len[b] + (b < (int)adm ? r.n : 0) : 0;
  }
  if (g == 0) {
    a.counts[0] = (int)adm;
    a.counts[1] = (int)nr;
    a.counts[2] = (int)np;
  }
  for (int i = g; i < (int)np; i += step) {
    const int b = plan_find(pg, a.B, i);
    const int have = plan_req(a, b).have;
    a.page_table[(long long)b * a.max_pages + have + (i - (int)pg[b])] = a.free_pages[i];
  }
  for (int t = g; t < a.rows; t += step) {
    int seq = -1, p = 0;
    long long s = -1;
    if (t < (int)nr) {
      seq = plan_find(qs, a.B, t);
      const int past = a.past_len[seq];
      p = past + (t - (int)qs[seq]);
      const int j = p >> 6, have = (int)(((long long)past + 63) >> 6);
      // A new page comes from the free list itself: its table entry is being written by some other thread.
      const int page = j < have ? a.page_table[(long long)seq * a.max_pages + j] : a.free_pages[(int)pg[seq] + j - have];
      if (page >= 0 && page < a.num_pages) s = (long long)page * 64 + (p & 63);
      else flag_error(a.err, kErrBounds);
    }
    a.seq_idx[t] = seq;
    a.pos[t] = p;
    a.slot[t] = s;
  }
}

// ---------------------------------------------------------- norms, rotation
// 16-byte vectors where every row starts on a 16-byte boundary and every
// width is whole vectors (VE elements each), else single elements.
template <typename T, bool kVec>
struct Vec {
  static constexpr int VE = kVec ? 16 / (int)sizeof(T) : 1;
  uint4 u;  // as it is stored: half the registers of its values in 32 bits
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kVec) u = *reinterpret_cast<const uint4*>(p);
    else u.x = __float_as_uint(to_f32(*p));
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kVec) *reinterpret_cast<uint4*>(p) = u;
    else *p = from_f32<T>(__uint_as_float(u.x));
  }
  __device__ __forceinline__ void get(float (&f)[VE]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (kVec && sizeof(T) == 2) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[q]));
        f[2 * q] = v.x;
        f[2 * q + 1] = v.y;
      }
    } else {
#pragma unroll
      for (int q = 0; q < VE; ++q) f[q] = __uint_as_float(w[q]);
    }
  }
  __device__ __forceinline__ void set(const float (&f)[VE]) {
    if constexpr (kVec && sizeof(T) == 2) {
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * q], f[2 * q + 1]);
        w[q] = *reinterpret_cast<const uint32_t*>(&h);
      }
      u = make_uint4(w[0], w[1], w[2], w[3]);
    } else if constexpr (kVec) {
      u = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    } else {
      u.x = __float_as_uint(f[0]);
    }
  }
  // Adds the squares of the values times `by` to `ss`.
  __device__ __forceinline__ void squares(float& ss, float by = 1.f) const {
    float f[VE];
    get(f);
#pragma unroll
    for (int e = 0; e < VE; ++e) ss = fmaf(f[e] * by, f[e] * by, ss);
  }
  // The normalised values: x * inv * gamma, rounded once.
  __device__ __forceinline__ void norm(float inv, const Vec& g) {
    float f[VE], h[VE];
    get(f);
    g.get(h);
#pragma unroll
    for (int e = 0; e < VE; ++e) f[e] = f[e] * inv * h[e];
    set(f);
  }
};

struct Rope {
  double turns[32];  // theta_i / (2 pi): the turns that pair i makes per position
  int half;          // pairs of one key, d_r / 2
};

// Cosine and sine of pair i's angle at `pos`.  The turns are formed and
// reduced to [-1/2, 1/2] in 64 bits (a far position makes tens of thousands
// of them), and the sine and cosine of the reduced angle taken in 32.
__device__ __forceinline__ float2 rope_cs(const Rope& r, int pos, int i) {
  const double t = (double)pos * r.turns[i];
  float s, c;
  sincospif(2.0f * (float)(t - rint(t)), &s, &c);
  return make_float2(c, s);
}

// Lanes of one row (G of them, a power of two) add up their squares and return
// 1 / sqrt(sum / n + eps).  `sum(by)` is a lane's sum of (by x)^2: where the
// plain sum passes the range of 32 bits it is taken again with by = 2^-64.
template <class Sum>
__device__ __forceinline__ float row_rms(Sum sum, int n, float eps, int G) {
  auto all = [&](float ss) {
    for (int o = G >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    return ss;
  };
  float ss = all(sum(1.f));
  if (__any_sync(0xffffffffu, isinf(ss))) {
    const float small = all(sum(0x1p-64f));
    if (isinf(ss)) return rsqrtf(small / (float)n + eps * 0x1p-64f * 0x1p-64f) * 0x1p-64f;
  }
  return rsqrtf(ss / (float)n + eps);
}

// RMS norm of one row of n elements by one warp: out = x rsqrt(mean(x^2) +
// eps) gamma, in 32 bits and rounded once (a null gamma copies the row).  Up
// to NV vectors per lane stay in registers; a longer row is read a second
// time, from L1 or L2.  `x` and `out` may be the same row.
constexpr int NV = 8;
template <typename T, bool kVec>
__device__ __forceinline__ void warp_rms_row(const T* x, const T* gamma, T* out, int n, float eps, int lane) {
  using V = Vec<T, kVec>;
  const int nv = n / V::VE;
  V v[NV], g[NV];  // gamma is asked for before the sum is known
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (lane + 32 * i < nv) v[i].load(x + (lane + 32 * i) * V::VE);
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (gamma && lane + 32 * i < nv) g[i].load(gamma + (lane + 32 * i) * V::VE);
  const float inv = row_rms([&](float by) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane + 32 * i < nv) v[i].squares(ss, by);
    for (int i = lane + 32 * NV; i < nv; i += 32) {
      V u;
      u.load(x + i * V::VE);
      u.squares(ss, by);
    }
    return ss;
  }, n, eps, 32);
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (lane + 32 * i < nv) {
      if (gamma) v[i].norm(inv, g[i]);
      v[i].store(out + (lane + 32 * i) * V::VE);
    }
  for (int i = lane + 32 * NV; i < nv; i += 32) {
    V u, w;
    u.load(x + i * V::VE);
    if (gamma) {
      w.load(gamma + i * V::VE);
      u.norm(inv, w);
    }
    u.store(out + i * V::VE);
  }
}

// The two adjacent elements of a pair: one load or store in the vector form.
template <typename T, bool kVec>
__device__ __forceinline__ float2 load_pair(const T* p) {
  if constexpr (!kVec) return make_float2(to_f32(p[0]), to_f32(p[1]));
  else if constexpr (sizeof(T) == 2) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
  else return *reinterpret_cast<const float2*>(p);
}
template <typename T, bool kVec>
__device__ __forceinline__ void put_pair(T* p, float a, float b) {
  if constexpr (kVec) {
    store_pair(p, a, b);
  } else {
    p[0] = from_f32<T>(a);
    p[1] = from_f32<T>(b);
  }
}

// --------------------------------------------------- normalised append
// One warp per row and latent: warps of even index take the cache row
// [rms(c) gamma | RoPE(k_R)], the others c_Q (when there is one).  Each
// element is read and written once, so it is bound by memory (by latency at
// decode sizes); a warp's whole row is in flight at once.
struct NormAppendArgs {
  const void* kv;        // [T][kv_stride]: [c (d_c) | k_R]
  const void* kv_gamma;  // [d_c] or null
  const void* cq;        // [T][cq_stride] or null
  const void* cq_gamma;  // [d_cq] or null
  void* cq_out;
  const int32_t* pos;
  const int64_t* slot;
  void* cache;
  int32_t* err;
  long long kv_stride, cq_stride, cq_out_stride, num_slots;
  int T, d_c, d_cr, d_cq;
  float eps;
  Rope rope;
};
constexpr int NORM_THREADS = 128;

template <typename T, bool kVec>
__global__ void __launch_bounds__(NORM_THREADS) norm_append_kernel(const NormAppendArgs a) {
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * (NORM_THREADS / 32) + (threadIdx.x >> 5);
  const int parts = a.cq ? 2 : 1;
  const long long t = w / parts;
  if (t >= a.T) return;
  if (w - t * parts == 1) {
    warp_rms_row<T, kVec>(static_cast<const T*>(a.cq) + t * a.cq_stride, static_cast<const T*>(a.cq_gamma),
                          static_cast<T*>(a.cq_out) + t * a.cq_out_stride, a.d_cq, a.eps, lane);
    return;
  }
  const long long slot = a.slot[t];
  if (slot < 0 || slot >= a.num_slots) {
    if (slot != -1 && lane == 0) flag_error(a.err, kErrBounds);
    return;
  }
  const T* const x = static_cast<const T*>(a.kv) + t * a.kv_stride;
  T* const row = static_cast<T*>(a.cache) + slot * a.d_cr;
  const int pos = a.pos[t], half = a.rope.half, pairs = (a.d_cr - a.d_c) / 2;
  float2 k = make_float2(0.f, 0.f);  // the shared key is at most one pair per lane
  if (lane < pairs) k = load_pair<T, kVec>(x + a.d_c + 2 * lane);
  const float2 cs = lane < half ? rope_cs(a.rope, pos, lane) : make_float2(1.f, 0.f);
  warp_rms_row<T, kVec>(x, static_cast<const T*>(a.kv_gamma), row, a.d_c, a.eps, lane);
  for (int i = lane;; i += 32) {
    // With a key per head, pair i belongs to head i / half; its angle's sine and cosine sit in lane i % half.
    const int own = i % half;
    const float c = __shfl_sync(0xffffffffu, cs.x, own), s = __shfl_sync(0xffffffffu, cs.y, own);
    if (i < pairs) put_pair<T, kVec>(row + a.d_c + 2 * i, k.x * c - k.y * s, k.x * s + k.y * c);
    if (i - lane + 32 >= pairs) break;  // the same in every lane
    if (i + 32 < pairs) k = load_pair<T, kVec>(x + a.d_c + 2 * (i + 32));
  }
}

// --------------------------------------------------- query norm, rotation
// A block takes `hpb` heads of one token.  A head's content is normalised by a
// group of G lanes (the power of two that holds it as 16-byte vectors, so a
// warp works on 32 / G heads at once); the position parts of a block's heads
// share one table of sines and cosines and are walked as one array.  Bound by
// memory: every element is read and written once.
struct QueryArgs {
  const void* q;       // [T][n_h] rows [q_C (d_h) | q_R (d_r)], q_stride per token
  const void* gamma;   // [d_h] or null
  void* qc;            // content out, strides per token and head
  void* qr;            // position part out
  const int32_t* pos;
  long long q_stride, qc_ts, qc_hs, qr_ts, qr_hs;
  int T, n_h, d_h, d_r, hpb, group;
  float eps;
  Rope rope;
};
constexpr int QUERY_THREADS = 256;
constexpr int QNV = 4;  // vectors of a head's content that a lane keeps

template <typename T, bool kVec>
__global__ void __launch_bounds__(QUERY_THREADS) query_norm_rope_kernel(const QueryArgs a) {
  using V = Vec<T, kVec>;
  __shared__ float2 cs[32];
  const int tid = threadIdx.x, lane = tid & 31;
  const long long t = blockIdx.x;
  const int h0 = blockIdx.y * a.hpb, h1 = min(a.n_h, h0 + a.hpb);
  const int dq = a.d_h + a.d_r, G = a.group, sub = lane & (G - 1);
  const T* const x = static_cast<const T*>(a.q) + t * a.q_stride;
  const T* const gamma = static_cast<const T*>(a.gamma);
  if (tid < a.rope.half) cs[tid] = rope_cs(a.rope, a.pos[t], tid);

  const int nv = a.d_h / V::VE;
  V g[QNV];
#pragma unroll
  for (int i = 0; i < QNV; ++i)
    if (gamma && sub + G * i < nv) g[i].load(gamma + (sub + G * i) * V::VE);
  const int per = QUERY_THREADS / G;  // heads at a time
  for (int hb = h0; hb < h1; hb += per) {
    const int h = hb + tid / G;
    const bool live = h < h1;
    const T* const xc = x + (long long)h * dq;
    T* const out = static_cast<T*>(a.qc) + t * a.qc_ts + h * a.qc_hs;
    V v[QNV];
#pragma unroll
    for (int i = 0; i < QNV; ++i)
      if (live && sub + G * i < nv) v[i].load(xc + (sub + G * i) * V::VE);
    const float inv = row_rms([&](float by) {
      float ss = 0.f;
      if (!live) return ss;
#pragma unroll
      for (int i = 0; i < QNV; ++i)
        if (sub + G * i < nv) v[i].squares(ss, by);
      for (int i = sub + G * QNV; i < nv; i += G) {
        V u;
        u.load(xc + i * V::VE);
        u.squares(ss, by);
      }
      return ss;
    }, a.d_h, a.eps, G);
    if (!live) continue;
#pragma unroll
    for (int i = 0; i < QNV; ++i)
      if (sub + G * i < nv) {
        if (gamma) v[i].norm(inv, g[i]);
        v[i].store(out + (sub + G * i) * V::VE);
      }
    for (int i = sub + G * QNV; i < nv; i += G) {
      V u, w;
      u.load(xc + i * V::VE);
      if (gamma) {
        w.load(gamma + i * V::VE);
        u.norm(inv, w);
      }
      u.store(out + i * V::VE);
    }
  }
  __syncthreads();
  // Position parts: vectors of whole pairs (single pairs without them).
  constexpr int PE = kVec ? V::VE : 2;
  const int nr = a.d_r / PE, total = (h1 - h0) * nr;
  for (int i = tid; i < total; i += QUERY_THREADS) {
    const int h = h0 + i / nr, e0 = (i % nr) * PE;
    const T* const xr = x + (long long)h * dq + a.d_h + e0;
    T* const out = static_cast<T*>(a.qr) + t * a.qr_ts + h * a.qr_hs + e0;
    if constexpr (kVec) {
      V v;
      float f[V::VE];
      v.load(xr);
      v.get(f);
#pragma unroll
      for (int e = 0; e < V::VE; e += 2) {
        const float2 c = cs[(e0 + e) >> 1];
        const float x0 = f[e], x1 = f[e + 1];
        f[e] = x0 * c.x - x1 * c.y;
        f[e + 1] = x0 * c.y + x1 * c.x;
      }
      v.set(f);
      v.store(out);
    } else {
      const float2 c = cs[e0 >> 1];
      const float x0 = to_f32(xr[0]), x1 = to_f32(xr[1]);
      out[0] = from_f32<T>(x0 * c.x - x1 * c.y);
      out[1] = from_f32<T>(x0 * c.y + x1 * c.x);
    }
  }
}

}  // namespace step
}  // namespace mla
