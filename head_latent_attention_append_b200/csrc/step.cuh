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

// The calls of a step are short and follow one another, so each is launched
// while the kernel before it ends (sm100.cuh, programmatic dependent launch),
// which takes about 1.5 us off every one.
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
// a binary search in shared memory.  3.2 us for 64 requests of one token, 4.3
// for 1024 requests and 21,600 rows (device time; the launch takes the host 3).
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
  sm100::pdl_wait();
  sm100::pdl_trigger();
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
// width is whole vectors (VE elements each), else single elements.  The values
// are worked on two at a time (packed 32-bit multiplies and FMAs): these calls
// move every byte once and would be bound by issued instructions otherwise.
template <typename T, bool kVec>
struct Vec {
  static constexpr int VE = kVec ? 16 / (int)sizeof(T) : 1;
  static constexpr int NP = kVec ? VE / 2 : 1;  // pairs (a single element is one with 0)
  uint4 u;  // as it is stored: half the registers of its values in 32 bits
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kVec) u = *reinterpret_cast<const uint4*>(p);
    else u.x = __float_as_uint(to_f32(*p));
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kVec) *reinterpret_cast<uint4*>(p) = u;
    else *p = from_f32<T>(__uint_as_float(u.x));
  }
  __device__ __forceinline__ void get(float2 (&f)[NP]) const {
    if constexpr (!kVec) {
      f[0] = make_float2(__uint_as_float(u.x), 0.f);
    } else if constexpr (sizeof(T) == 2) {
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) f[q] = make_float2(__uint_as_float(w[q] << 16), __uint_as_float(w[q] & 0xffff0000u));
    } else {
      f[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
      f[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
    }
  }
  __device__ __forceinline__ void set(const float2 (&f)[NP]) {
    if constexpr (!kVec) {
      u.x = __float_as_uint(f[0].x);
    } else if constexpr (sizeof(T) == 2) {
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const __nv_bfloat162 h = __float22bfloat162_rn(f[q]);
        w[q] = *reinterpret_cast<const uint32_t*>(&h);
      }
      u = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      u = make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
    }
  }
  // Adds the squares of the values (times `by`, where it is not 1) to `ss`.
  template <bool kScaled>
  __device__ __forceinline__ void squares(float2& ss, float by) const {
    float2 f[NP];
    get(f);
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      if constexpr (kScaled) f[e] = __fmul2_rn(f[e], make_float2(by, by));
      ss = __ffma2_rn(f[e], f[e], ss);
    }
  }
  // Times a power of two (exact, but for results below the type's normal range).
  __device__ __forceinline__ void scale(float by) {
    float2 f[NP];
    get(f);
#pragma unroll
    for (int e = 0; e < NP; ++e) f[e] = __fmul2_rn(f[e], make_float2(by, by));
    set(f);
  }
  // The normalised values: x * inv * gamma, rounded once.
  __device__ __forceinline__ void norm(float inv, const Vec& g) {
    float2 f[NP], h[NP];
    get(f);
    g.get(h);
#pragma unroll
    for (int e = 0; e < NP; ++e) f[e] = __fmul2_rn(__fmul2_rn(f[e], make_float2(inv, inv)), h[e]);
    set(f);
  }
};

struct Rope {
  double turns[32];  // theta_i / (2 pi): the turns that pair i makes per position
  int half;          // pairs of one key, d_r / 2
};

// Cosine and sine of pair i's angle at `pos`.  The turns are formed and
// reduced to [-1/2, 1/2] in 64 bits (a far position makes tens of thousands
// of them), and the sine and cosine of the reduced angle taken in 32, which
// leaves rotated values off by 5e-8 of their pair's length (2-norm).
__device__ __forceinline__ float2 rope_cs(const Rope& r, int pos, int i) {
  const double t = (double)pos * r.turns[i];
  float s, c;
  sincospif(2.0f * (float)(t - rint(t)), &s, &c);
  return make_float2(c, s);
}
__device__ __forceinline__ float2 turn(float2 x, float2 cs) {
  return make_float2(x.x * cs.x - x.y * cs.y, x.x * cs.y + x.y * cs.x);
}

// The threads of one row add up their sums of squares: G neighbouring lanes (a
// power of two) of a warp in which every lane takes part,
template <int G>
struct LaneTotal {
  __device__ __forceinline__ float operator()(float ss) const {
#pragma unroll
    for (int o = G >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    return ss;
  }
  __device__ __forceinline__ bool any(bool b) const { return __any_sync(0xffffffffu, b); }
};
// or W whole warps, which share named barrier `bar` and two sets of W words of
// shared memory, used in turn so that one barrier is enough.  Every thread adds
// the words in the same order.
template <int W>
struct WarpsTotal {
  float* words;
  int warp, bar;
  int* flip;
  __device__ __forceinline__ float operator()(float ss) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    float* const w = words + *flip * W;
    *flip ^= 1;
    if ((threadIdx.x & 31) == 0) w[warp] = ss;
    sm100::named_bar_sync(bar, 32 * W);
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) ss += w[i];
    return ss;
  }
  __device__ __forceinline__ bool any(bool b) const { return b; }  // the same in every thread
};

// A thread's share of one row of n elements that `lanes` threads hold, this
// being number `lane`: NV vectors in registers; what a longer row has besides
// is read a second time, from L1 or L2.
template <typename T, bool kVec, int NV>
struct RowPart {
  using V = Vec<T, kVec>;
  V v[NV];
  __device__ __forceinline__ void load(const T* x, int nv, int lane, int lanes) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane + lanes * i < nv) v[i].load(x + (lane + lanes * i) * V::VE);
  }
  template <bool kScaled>
  __device__ __forceinline__ float squares(const T* x, int nv, int lane, int lanes, float by) const {
    float2 ss = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane + lanes * i < nv) v[i].template squares<kScaled>(ss, by);
    for (int i = lane + lanes * NV; i < nv; i += lanes) {
      V u;
      u.load(x + i * V::VE);
      u.template squares<kScaled>(ss, by);
    }
    return ss.x + ss.y;
  }
  // RMS norm: out = x / sqrt(mean(x^2) + eps) * gamma in 32 bits, rounded once;
  // a null gamma copies the row.  `x` and `out` may be the same row; `g` is
  // this thread's share of gamma.  Where the sum of squares passes the range
  // of 32 bits it is taken again of x 2^-96, so that no row of finite values
  // passes it (2^64 per value); 1 / sqrt(mean) is then as small as 2^-128,
  // below the normal range, so x takes 2^-64 of it and the factor the rest.
  // Where the squares fall below that range (and eps is too small to matter
  // less than they do) the same is done with 2^96, 2^64 and 2^32.
  // `live` is false in threads that only take part in the sums.
  template <class Total>
  __device__ __forceinline__ void norm(const RowPart& g, const T* x, const T* gamma, T* out, int nv, float inv_n,
                                       float eps, int lane, int lanes, bool live, const Total& total) {
    float inv = 1.f;
    float part = 1.f;
    bool far = false;
    if (gamma) {  // the same for every row
      const int own = live ? nv : 0;
      const float ss = total(squares<false>(x, own, lane, lanes, 1.f));
      const float mean = fmaf(ss, inv_n, eps);
      inv = rsqrtf(mean);
      far = isinf(ss) || mean < 0x1p-100f;
      if (total.any(far)) {
        const float by = isinf(ss) ? 0x1p-96f : 0x1p96f;
        const float again = total(squares<true>(x, own, lane, lanes, by));
        if (far) inv = rsqrtf(fmaf(again, inv_n, eps * by * by)) * (isinf(ss) ? 0x1p-32f : 0x1p32f);
        part = isinf(ss) ? 0x1p-64f : 0x1p64f;
      }
    }
    if (!live) return;
    if (far) {
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i].scale(part);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane + lanes * i < nv) {
        if (gamma) v[i].norm(inv, g.v[i]);
        v[i].store(out + (lane + lanes * i) * V::VE);
      }
    for (int i = lane + lanes * NV; i < nv; i += lanes) {
      V u, w;
      u.load(x + i * V::VE);
      if (gamma) {
        w.load(gamma + i * V::VE);
        if (far) u.scale(part);
        u.norm(inv, w);
      }
      u.store(out + i * V::VE);
    }
  }
};

// The two adjacent elements of a pair: one load or store in the vector form.
template <typename T, bool kVec>
__device__ __forceinline__ float2 load_pair(const T* p) {
  if constexpr (!kVec) return make_float2(to_f32(p[0]), to_f32(p[1]));
  else if constexpr (sizeof(T) == 2) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
  else return *reinterpret_cast<const float2*>(p);
}
template <typename T, bool kVec>
__device__ __forceinline__ void put_pair(T* p, float2 v) {
  if constexpr (kVec) {
    store_pair(p, v.x, v.y);
  } else {
    p[0] = from_f32<T>(v.x);
    p[1] = from_f32<T>(v.y);
  }
}

// --------------------------------------------------- normalised append
// With a query latent, a block per row: warp 0 takes the cache row
// [rms(c) gamma | RoPE(k_R)], the other three c_Q, which is about three times as
// long, so that every thread moves two to four vectors.  Without one, a warp per
// row.  Each element is read and written once: bound by memory, by latency at
// decode sizes.  So a warp walks several rows where there are many, keeps its
// share of gamma, and asks for the next row before it works on this one.
// 16,384 rows of 2112 bf16 values: 31.3 us, 4.4 TB/s, 0.68 of the measured copy
// rate (a block per row without walking 32.9, two rows ahead 38, eight vectors
// per lane and a warp for all of c_Q 77); neither memory nor issue is full then:
// a warp has one row on its way and waits at each row's sums.  64 rows: 2.4 us.
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

template <typename T, bool kVec, int NV>
__global__ void __launch_bounds__(NORM_THREADS, NV == 2 ? 8 : 4) norm_append_kernel(const NormAppendArgs a) {
  using Part = RowPart<T, kVec, NV>;
  constexpr int VE = Vec<T, kVec>::VE;
  __shared__ float words[6];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  sm100::pdl_wait();
  sm100::pdl_trigger();
  if (a.cq && warp > 0) {
    const int i = threadIdx.x - 32, nv = a.d_cq / VE;
    const T* const gamma = static_cast<const T*>(a.cq_gamma);
    const float inv_n = 1.f / (float)a.d_cq;
    int flip = 0;
    const WarpsTotal<3> total{words, warp - 1, 1, &flip};
    auto row = [&](int t) { return static_cast<const T*>(a.cq) + t * a.cq_stride; };
    Part cur, nxt, g;
    int t = blockIdx.x;
    if (t < a.T) cur.load(row(t), nv, i, 96);
    if (gamma) g.load(gamma, nv, i, 96);
    for (; t < a.T; t += gridDim.x) {
      if (t + (int)gridDim.x < a.T) nxt.load(row(t + gridDim.x), nv, i, 96);
      cur.norm(g, row(t), gamma, static_cast<T*>(a.cq_out) + t * a.cq_out_stride, nv, inv_n, a.eps, i, 96, true, total);
      cur = nxt;
    }
    return;
  }
  const int step = a.cq ? gridDim.x : gridDim.x * (NORM_THREADS / 32);
  const int nv = a.d_c / VE, half = a.rope.half, pairs = (a.d_cr - a.d_c) / 2;
  const T* const gamma = static_cast<const T*>(a.kv_gamma);
  const float inv_n = 1.f / (float)a.d_c;
  struct Row {
    Part c;
    float2 k;  // the shared key is at most one pair per lane
    long long slot;
    int pos;
  };
  auto src = [&](int t) { return static_cast<const T*>(a.kv) + t * a.kv_stride; };
  auto load = [&](Row& r, int t) {
    const T* const x = src(t);
    r.c.load(x, nv, lane, 32);
    if (lane < pairs) r.k = load_pair<T, kVec>(x + a.d_c + 2 * lane);
    r.slot = a.slot[t];
    r.pos = a.pos[t];
  };
  Row cur, nxt;
  Part g;
  int t = a.cq ? blockIdx.x : blockIdx.x * (NORM_THREADS / 32) + warp;
  if (t < a.T) load(cur, t);
  if (gamma) g.load(gamma, nv, lane, 32);
  for (; t < a.T; t += step) {
    if (t < a.T - step) load(nxt, t + step);
    if (cur.slot >= 0 && cur.slot < a.num_slots) {
      T* const dst = static_cast<T*>(a.cache) + cur.slot * a.d_cr;
      const float2 cs = lane < half ? rope_cs(a.rope, cur.pos, lane) : make_float2(1.f, 0.f);
      cur.c.norm(g, src(t), gamma, dst, nv, inv_n, a.eps, lane, 32, true, LaneTotal<32>{});
      if (pairs == half) {
        if (lane < pairs) put_pair<T, kVec>(dst + a.d_c + 2 * lane, turn(cur.k, cs));
      } else {
        // A key per head: pair i belongs to head i / half, and its angle's sine and cosine sit in lane i % half.
        for (int i0 = 0; i0 < pairs; i0 += 32) {
          const int i = i0 + lane, own = i % half;
          const float2 c = make_float2(__shfl_sync(0xffffffffu, cs.x, own), __shfl_sync(0xffffffffu, cs.y, own));
          if (i0 > 0 && i < pairs) cur.k = load_pair<T, kVec>(src(t) + a.d_c + 2 * i);
          if (i < pairs) put_pair<T, kVec>(dst + a.d_c + 2 * i, turn(cur.k, c));
        }
      }
    } else if (cur.slot != -1 && lane == 0) {
      flag_error(a.err, kErrBounds);
    }
    cur = nxt;
  }
}

// --------------------------------------------------- query norm, rotation
// A block takes some heads of one token.  A head's content is normalised by a
// group of G lanes (the power of two that holds it as 16-byte vectors, VPL of
// them per lane), two heads per group in a step; the position parts of a step's
// heads are turned by groups of 2^rope_shift lanes, so that a thread turns the
// same pairs of every head and keeps their sines and cosines, as it keeps its
// share of gamma.  Every element is read and written once.  What bounded the
// first versions was occupancy (two blocks an SM, 226 us for 4096 tokens of 128
// heads), then issued instructions (divisions by the group's size, one value
// at a time, 87 us); now memory: 74.5 us, 5.4 TB/s, 0.82 of the measured copy rate.
struct QueryArgs {
  const void* q;       // [T][n_h] rows [q_C (d_h) | q_R (d_r)], q_stride per token
  const void* gamma;   // [d_h] or null
  void* qc;            // content out, strides per token and head
  void* qr;            // position part out
  const int32_t* pos;
  long long q_stride, qc_ts, qc_hs, qr_ts, qr_hs;
  int T, n_h, d_h, d_r, hpb, rope_shift;  // hpb: heads per block, a multiple of a step's
  float eps;
  Rope rope;
};
constexpr int QUERY_THREADS = 128;

template <typename T, bool kVec, int G, int VPL>
__global__ void __launch_bounds__(QUERY_THREADS) query_norm_rope_kernel(const QueryArgs a) {
  using V = Vec<T, kVec>;
  using Part = RowPart<T, kVec, VPL>;
  constexpr int PER = QUERY_THREADS / G, STEP = 2 * PER;  // heads at a time and per step
  constexpr int PE = kVec ? V::VE : 2;                    // position parts: vectors of whole pairs, or single pairs
  __shared__ float2 cs[32];
  const int tid = threadIdx.x, sub = tid & (G - 1), grp = tid / G;
  const long long t = blockIdx.x;
  const int nv = a.d_h / V::VE, dq = a.d_h + a.d_r;
  const int h0 = blockIdx.y * a.hpb, h1 = min(a.n_h, h0 + a.hpb);
  const int e0 = (tid & ((1 << a.rope_shift) - 1)) * PE, rgrp = tid >> a.rope_shift, rper = QUERY_THREADS >> a.rope_shift;
  const bool turns = e0 < a.d_r;
  const T* const x = static_cast<const T*>(a.q) + t * a.q_stride;
  const T* const gamma = static_cast<const T*>(a.gamma);
  const float inv_n = 1.f / (float)a.d_h;

  struct Work {
    Part c[2];
    V r;         // the thread's first position part of the step
    float2 pair; // the same without vectors
  };
  auto load_turn = [&](Work& w, int h) {
    const T* const p = x + (long long)h * dq + a.d_h + e0;
    if constexpr (kVec) w.r.load(p);
    else w.pair = load_pair<T, false>(p);
  };
  auto load = [&](Work& w, int hb) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int h = hb + i * PER + grp;
      if (h < h1) w.c[i].load(x + (long long)h * dq, nv, sub, G);
    }
    if (turns && hb + rgrp < min(h1, hb + STEP)) load_turn(w, hb + rgrp);
  };
  sm100::pdl_wait();
  sm100::pdl_trigger();
  Work cur, nxt;
  load(cur, h0);
  Part g;
  if (gamma) g.load(gamma, nv, sub, G);
  if (tid < a.rope.half) cs[tid] = rope_cs(a.rope, a.pos[t], tid);
  __syncthreads();
  float2 c[PE / 2];
#pragma unroll
  for (int i = 0; i < PE / 2; ++i) c[i] = turns ? cs[e0 / 2 + i] : make_float2(1.f, 0.f);

  for (int hb = h0; hb < h1; hb += STEP) {
    if (hb + STEP < h1) load(nxt, hb + STEP);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int h = hb + i * PER + grp;
      cur.c[i].norm(g, x + (long long)h * dq, gamma, static_cast<T*>(a.qc) + t * a.qc_ts + h * a.qc_hs, nv, inv_n, a.eps,
                    sub, G, h < h1, LaneTotal<G>{});
    }
    const int he = min(h1, hb + STEP);
    if (turns)
      for (int h = hb + rgrp; h < he; h += rper) {
        if (h != hb + rgrp) load_turn(cur, h);
        T* const out = static_cast<T*>(a.qr) + t * a.qr_ts + h * a.qr_hs + e0;
        if constexpr (kVec) {
          float2 f[V::NP];
          cur.r.get(f);
#pragma unroll
          for (int i = 0; i < V::NP; ++i) f[i] = turn(f[i], c[i]);
          cur.r.set(f);
          cur.r.store(out);
        } else {
          put_pair<T, false>(out, turn(cur.pair, c[0]));
        }
      }
    cur = nxt;
  }
}

}  // namespace step
}  // namespace mla
