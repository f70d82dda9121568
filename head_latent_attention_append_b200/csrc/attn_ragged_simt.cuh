// Ragged attention on the CUDA cores: the 32-bit path, whose accuracy
// single-pass TF32 on the tensor cores would not keep.
//
// One CTA walks its worker's segments (ragged_sched.cuh) of up to 64 rows, 32
// keys at a time; warp w keeps rows w, w + 8, ... of them, with their whole
// softmax state, and works alone between the block's key tiles:
//   S = Q K^T: lane (cg, kx) multiplies 8 rows with keys kx, kx + 8, kx + 16,
//   kx + 24 over the columns 16 s + 4 cg ..; a reduce-scatter over the four
//   column groups leaves lane `key` with the 8 rows' scores of that key;
//   the online softmax takes all eight rows at once, four lanes each, by way of
//   the warp's own rows of P, and
//   O += P V has 8 rows x 4 NC columns (4 lane + 128 c) in a lane's registers.
// A 16-byte shared-memory load of a warp costs four cycles whatever it shares,
// so a tile of R x C values per lane is bound by FMAs only where R C >= 4 (R +
// C).  The scores' 8 x 4 is short of that by 1.5 and bound by shared memory (4 x
// 2 with 256 threads, or 2 x 2 with 512, are short by three and four and took
// 1.5 times as long); P V's 8 x 4 NC meets it from NC = 2 on.  FMAs are
// issued in pairs, which took 4% (d_c 512) to 9% (one tile per CTA) off.  A small
// batch is one tile per CTA and bound by latency, so all rows of a tile are
// copied asynchronously at once, the next 32 keys while these are worked on
// (where two buffers fit: rows of up to 432 values).  One bulk copy per row
// instead of sixteen bytes per thread: 5% faster at d_c 256 in large batches,
// 5% slower at 512 (registers), 1% slower in small ones.  400 tokens of 16 heads
// over up to 4000 keys run at 36 of 74 TFLOP/s; 39 tokens over up to 517 keys in
// 32 us, where 4.4 is their FMAs at that rate.
#pragma once
#include "ragged_sched.cuh"

namespace mla {
namespace ragged_simt {

constexpr int ROWS = 64, KT = 32, THREADS = 256, WARPS = THREADS / 32, PP = 36;

// Columns are padded with zeros to whole float4s, the latent and the position
// key separately, and the row to whole steps of 16; an odd number of float4s
// per row keeps the 8 rows of a quarter warp's load in different banks.
__host__ __device__ constexpr int pad4(int n) { return (n + 3) & ~3; }
__host__ __device__ constexpr int row_cols(int d_c, int d_r) { return (pad4(d_c) + pad4(d_r) + 15) & ~15; }
__host__ __device__ constexpr int pitch(int d_c, int d_r) { return row_cols(d_c, d_r) + 4; }
inline size_t smem_bytes(int d_c, int d_r, int buffers) {
  return sizeof(float) * ((size_t)(ROWS + buffers * KT) * pitch(d_c, d_r) + ROWS * PP) + 16;  // the last 16: the error word
}
constexpr size_t MAX_SMEM = 232448;
constexpr int kOwnMost = THREADS;  // requests and row blocks of a schedule that every CTA makes for itself
static_assert(sizeof(RaggedScratch<kOwnMost>) <= sizeof(float) * ((ROWS + KT) * 20 + ROWS * PP),
              "the schedule's sums fit the smallest rows' tiles");
inline int key_buffers(int d_c, int d_r) { return smem_bytes(d_c, d_r, 2) <= MAX_SMEM ? 2 : 1; }

// 16 bytes from global to shared memory without passing through registers, or
// zeros; both addresses 16-byte aligned.
__device__ __forceinline__ void copy16(float* dst, const float* src, bool zero) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm100::smem_u32(dst)), "l"(src), "r"(zero ? 0 : 16)
               : "memory");
}

struct Args {
  const float* q;            // row r of token t: q + t * q_ts + h * q_hs
  long long q_ts, q_hs;
  const float* cache;        // [num_pages][64][d_c + d_r]
  const int32_t* page_table; // [B][max_pages]
  int max_pages, num_pages, n_h, d_c, d_r;
  int buffers;               // key tiles in shared memory, 1 or 2
  float scale;               // softmax scale times log2 e
  RaggedSchedArgs sched;
  RaggedOut o;
};

// Where a segment's rows and keys are.
struct Ctx {
  float *Qs, *Kb, *Ps;  // [ROWS][P4], [buffers][KT][P4], [ROWS][PP]
  int* err;             // this CTA's error bits
  int d_cr, dcp, wq, P4;
  bool vec;
};

// A small batch runs this kernel's code once, so what is not an inner loop is
// kept small: the time of one tile was a third instruction misses while these
// copies and stores were unrolled with both of their forms.
//
// One row into shared memory by a warp: the latent at 0, the position key at
// dcp, zeros between and behind; not `live`: a row of zeros (src is then any
// address in bounds).
__device__ __noinline__ void put_row_any(float* dst, const float* src, bool live, int lane, int wq, int dcp, int d_c, int d_r) {
  for (int c = lane; c < wq; c += 32) {
    const int e = c < dcp ? (c < d_c ? c : -1) : (c - dcp < d_r ? d_c + c - dcp : -1);
    dst[c] = live && e >= 0 ? __ldg(src + e) : 0.f;
  }
}
__device__ __forceinline__ void put_row(const Args& a, const Ctx& x, float* dst, const float* src, bool live, int lane) {
  if (x.vec) {
#pragma unroll 1
    for (int v = lane; v < x.wq / 4; v += 32) {
      const bool in = 4 * v < x.d_cr;
      copy16(dst + 4 * v, in ? src + 4 * v : src, !live || !in);
    }
  } else {
    put_row_any(dst, src, live, lane, x.wq, x.dcp, a.d_c, a.d_r);
  }
}
__device__ __forceinline__ float4 at4(const float* p) { return *reinterpret_cast<const float4*>(p); }
// Four products as two pairs (even and odd columns).
__device__ __forceinline__ float2 dot4(float4 q, float4 k, float2 s) {
  s = __ffma2_rn(make_float2(q.x, q.y), make_float2(k.x, k.y), s);
  return __ffma2_rn(make_float2(q.z, q.w), make_float2(k.z, k.w), s);
}

// A segment of at most 8 MI rows.  MI is a constant so that the loops over a
// warp's rows leave no branches between loads and FMAs: with them the pipe was
// a quarter used.
template <int NC, int MI>
__device__ __forceinline__ void run_segment(const Args& a, const Ctx& x, const RSeg& g) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, kx = lane & 7, cg = lane >> 3, P4 = x.P4;
  const int k_begin = g.t_lo * 64, k_end = min(g.nkeys, g.t_hi * 64);
  const int32_t* const pages = a.page_table + (long long)g.seq * a.max_pages;
  // The page of keys k0 .. is known one tile ahead of its copy.
  int page_next = k_begin < k_end ? pages[k_begin / 64] : 0;
  auto fetch = [&](int k0, float* dst) {
    const int page = page_next;
    const bool ok = page >= 0 && page < a.num_pages;
    if (!ok && tid == 0) flag_error(x.err, kErrBounds);
    const float* const src = a.cache + ((long long)(ok ? page : 0) * 64 + k0 % 64) * x.d_cr;
#pragma unroll 1
    for (int r = warp; r < KT; r += WARPS)
      put_row(a, x, dst + r * P4, src + (long long)r * x.d_cr, ok && k0 + r < k_end, lane);
    if (k0 + KT < k_end) page_next = pages[(k0 + KT) / 64];
  };
  __syncthreads();  // the segment before is done with Qs and the key tiles
  // A block without keys needs no query rows either, and must not ask for them:
  // the key loop holds the only wait for the copies, and ones still in flight
  // could land on the next segment's rows.
  if (k_begin < k_end) {
#pragma unroll 1
    for (int i = 0; i < MI; ++i) {
      const int r = warp + WARPS * i, row = g.row0 + min(r, g.nrows - 1), t = row / a.n_h;
      put_row(a, x, x.Qs + r * P4, a.q + t * a.q_ts + (row - t * a.n_h) * a.q_hs, r < g.nrows, lane);
    }
    fetch(k_begin, x.Kb);
  }
  // The softmax state of the warp's rows: four lanes each, row lane / 4 (a warp
  // of fewer than eight rows leaves the others at no key).
  const int sr = lane >> 2, my_row = warp + WARPS * sr;
  const int lim = sr < MI && my_row < g.nrows ? min(max(g.base + (g.row0 + my_row) / a.n_h + 1, 0), g.nkeys) : 0;
  float m = -INFINITY, l = 0.f;
  float2 acc[MI][NC][2];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[i][c][0] = acc[i][c][1] = make_float2(0.f, 0.f);
  float* const Pr = x.Ps + warp * PP;
  int buf = 0;
  for (int k0 = k_begin; k0 < k_end; k0 += KT, buf ^= a.buffers - 1) {
    float* const Ks = x.Kb + buf * KT * P4;
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();  // this tile is there, and every thread is done with the one before
    if (a.buffers == 2 && k0 + KT < k_end) fetch(k0 + KT, x.Kb + (buf ^ 1) * KT * P4);
    float2 s2[MI][4];  // even and odd columns
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s2[i][j] = make_float2(0.f, 0.f);
    {
      const float* const kp = Ks + kx * P4 + 4 * cg;
      const float* const qp = x.Qs + warp * P4 + 4 * cg;
      for (int c = 0; c < x.wq; c += 16) {
        float4 k[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) k[j] = at4(kp + 8 * j * P4 + c);
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          const float4 q = at4(qp + WARPS * i * P4 + c);
#pragma unroll
          for (int j = 0; j < 4; ++j) s2[i][j] = dot4(q, k[j], s2[i][j]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      // The four column groups' sums: this lane is left with key kx + 8 cg = lane.
      const bool hi = cg & 2, odd = cg & 1;
      float s[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] = s2[i][j].x + s2[i][j].y;
      const float t0 = (hi ? s[2] : s[0]) + __shfl_xor_sync(0xffffffffu, hi ? s[0] : s[2], 16);
      const float t1 = (hi ? s[3] : s[1]) + __shfl_xor_sync(0xffffffffu, hi ? s[1] : s[3], 16);
      Pr[WARPS * i * PP + lane] = (odd ? t1 : t0) + __shfl_xor_sync(0xffffffffu, odd ? t0 : t1, 8);
    }
    __syncwarp();
    {
      // All rows at once: lane holds eight keys of row sr.
      float* const pr = Pr + WARPS * min(sr, MI - 1) * PP + 8 * (lane & 3);
      const float4 xa = at4(pr), xb = at4(pr + 4);
      float x[8] = {xa.x, xa.y, xa.z, xa.w, xb.x, xb.y, xb.z, xb.w};
      const int seen = lim - k0 - 8 * (lane & 3);  // of these eight
      float mx = -INFINITY;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = e < seen ? x[e] * a.scale : -INFINITY;
        mx = fmaxf(mx, x[e]);
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m, mx), ref = ref_max(mn), corr = exp2f(m - ref);
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = exp2f(x[e] - ref);
        sum += x[e];
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      l = fmaf(l, corr, sum);
      m = mn;
      __syncwarp();  // lanes of a row that does not exist read another's scores
      if (sr < MI) {
        *reinterpret_cast<float4*>(pr) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(pr + 4) = make_float4(x[4], x[5], x[6], x[7]);
      }
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const float ci = __shfl_sync(0xffffffffu, corr, 4 * i);
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int e = 0; e < 2; ++e) acc[i][c][e] = __fmul2_rn(acc[i][c][e], make_float2(ci, ci));
      }
    }
    __syncwarp();
    if (k0 + KT > g.kmin) {
      // Keys that only some of the rows see: a weight of 0 must not meet an
      // infinity or a NaN.  A row that does see one already has a NaN sum, or a
      // score of -inf there and with it no weight.
      __syncthreads();
      for (int r = max(0, g.kmin - k0) + warp; r < KT; r += WARPS)
        for (int c = lane; c < x.dcp; c += 32)
          if (!isfinite(Ks[r * P4 + c])) Ks[r * P4 + c] = 0.f;
      __syncthreads();
    }
    // A lane whose last columns lie behind the latent adds up what is there
    // (the position key or zeros) and does not store it.
#pragma unroll 1
    for (int k = 0; k < KT; k += 4) {
      float4 p[MI];
#pragma unroll
      for (int i = 0; i < MI; ++i) p[i] = at4(Pr + WARPS * i * PP + k);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float4 v = at4(Ks + (k + kk) * P4 + min(4 * lane + 128 * c, x.wq - 4));
#pragma unroll
          for (int i = 0; i < MI; ++i) {
            const float w = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
            acc[i][c][0] = __ffma2_rn(make_float2(w, w), make_float2(v.x, v.y), acc[i][c][0]);
            acc[i][c][1] = __ffma2_rn(make_float2(w, w), make_float2(v.z, v.w), acc[i][c][1]);
          }
        }
    }
    __syncwarp();  // Ps is the next tile's
    if (a.buffers == 1 && k0 + KT < k_end) {
      __syncthreads();
      fetch(k0 + KT, x.Kb);
    }
  }
  // A whole row block goes to out, a piece to its slot (rows of dcp columns);
  // where rows of `out` are not whole float4s, by way of this warp's own rows of
  // Qs.
  const bool wide = g.slot >= 0 || (a.d_c & 3) == 0;
  float* const base = wide ? (g.slot < 0 ? static_cast<float*>(a.o.out) + (long long)g.row0 * x.dcp
                                         : a.o.part_o + (long long)g.slot * ROWS * x.dcp)
                           : x.Qs;
  const int step = wide ? x.dcp : P4;
  if ((lane & 3) == 0 && sr < MI && my_row < g.nrows) {
    if (g.slot >= 0) a.o.part_ml[(long long)g.slot * ROWS + my_row] = make_float2(m, l);
    else if (a.o.lse) a.o.lse[(long long)g.row0 + my_row] = row_lse(ref_max(m), l);
  }
  const float row_factor = row_inv(l);
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int r = warp + WARPS * i;
    const float inv = __shfl_sync(0xffffffffu, row_factor, 4 * i);
    if (r >= g.nrows) continue;
    float* const dst = base + r * step + 4 * lane;
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (4 * lane + 128 * c < x.dcp)
        *reinterpret_cast<float4*>(dst + 128 * c) =
            make_float4(acc[i][c][0].x * inv, acc[i][c][0].y * inv, acc[i][c][1].x * inv, acc[i][c][1].y * inv);
  }
  if (!wide) {
    __syncwarp();
#pragma unroll 1
    for (int r = warp; r < g.nrows; r += WARPS)
      for (int c = lane; c < a.d_c; c += 32)
        static_cast<float*>(a.o.out)[((long long)g.row0 + r) * a.d_c + c] = x.Qs[r * P4 + c];
  }
}

template <int NC>
__global__ void __launch_bounds__(THREADS, 1) attn_ragged_simt_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(16) float sm[];
  Ctx x;
  x.d_cr = a.d_c + a.d_r;
  x.dcp = pad4(a.d_c);
  x.wq = row_cols(a.d_c, a.d_r);
  x.P4 = pitch(a.d_c, a.d_r);
  x.Qs = sm;
  x.Kb = x.Qs + ROWS * x.P4;
  x.Ps = x.Kb + a.buffers * KT * x.P4;
  x.vec = (a.d_c & 3) == 0 && (x.d_cr & 3) == 0 && ((a.q_ts | a.q_hs) & 3) == 0 &&
          ((reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.cache)) & 15) == 0;
  sm100::pdl_wait();
  sm100::pdl_trigger();
  x.err = reinterpret_cast<int*>(x.Ps + ROWS * PP);
  if (threadIdx.x == 0) *x.err = 0;
  __syncthreads();
  int2* const range = a.sched.s.range + blockIdx.x;
  if (a.sched.own) {
    ragged_schedule<kOwnMost>(a.sched, *reinterpret_cast<RaggedScratch<kOwnMost>*>(sm), blockIdx.x, range, x.err);
    __syncthreads();
  }
  const int seg_lo = range->x, seg_hi = range->y;
  RSeg g = a.sched.s.first[blockIdx.x];
  for (int si = seg_lo; si < seg_hi; ++si) {
    if (si > seg_lo) g = a.sched.s.segs[si];
    if (g.nrows <= 8) run_segment<NC, 1>(a, x, g);
    else if (g.nrows <= 16) run_segment<NC, 2>(a, x, g);
    else if (g.nrows <= 32) run_segment<NC, 4>(a, x, g);
    else run_segment<NC, 8>(a, x, g);
  }
  __syncthreads();
  if (threadIdx.x == 0) a.sched.s.worker_err[blockIdx.x] = *x.err;
}

}  // namespace ragged_simt
}  // namespace mla
