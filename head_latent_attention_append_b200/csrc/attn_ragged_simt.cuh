// Ragged attention on the CUDA cores: the 32-bit path, whose accuracy
// single-pass TF32 on the tensor cores would not keep.
//
// One CTA walks its worker's segments (ragged_sched.cuh) of up to 64 rows, 32
// keys at a time: S = Q K^T in registers (thread (ty, tx): rows ty + 16 i,
// keys tx + 16 j), the online softmax of a row among the 16 lanes that hold
// it, and O += P V with 4 rows x 4 NG columns of O in each thread's registers.
// A row's P is written and read by the same half-warp, so it costs no block
// barrier.  Bound by the FMA pipe (a 16-byte shared-memory load feeds 4 to 16
// FMAs); the loads of a key tile are about a tenth of its time, so there is
// one buffer.  Row groups past the block's rows are skipped.
#pragma once
#include "ragged_sched.cuh"

namespace mla {
namespace ragged_simt {

constexpr int ROWS = 64, KT = 32, THREADS = 256, PP = 36;

// Columns are padded with zeros to whole float4s, the latent and the position
// key separately; an odd number of float4s per row keeps the 16 rows of a
// score load in different banks.
__host__ __device__ constexpr int pad4(int n) { return (n + 3) & ~3; }
__host__ __device__ constexpr int pitch(int d_c, int d_r) { return 4 * (((pad4(d_c) + pad4(d_r)) / 4) | 1); }
inline size_t smem_bytes(int d_c, int d_r) { return sizeof(float) * ((size_t)(ROWS + KT) * pitch(d_c, d_r) + ROWS * PP); }

struct Args {
  const float* q;            // row r of token t: q + t * q_ts + h * q_hs
  long long q_ts, q_hs;
  const float* cache;        // [num_pages][64][d_c + d_r]
  const int32_t* page_table; // [B][max_pages]
  int max_pages, num_pages, n_h, d_c, d_r;
  float scale;               // softmax scale times log2 e
  RaggedSched sched;
  RaggedOut o;
  int* err;
};

template <int NG>
__global__ void __launch_bounds__(THREADS, 1) attn_ragged_simt_kernel(const Args a) {
  extern __shared__ float sm[];
  const int d_cr = a.d_c + a.d_r, dcp = pad4(a.d_c), wq = dcp + pad4(a.d_r), P4 = pitch(a.d_c, a.d_r);
  float* const Qs = sm;               // [ROWS][P4]
  float* const Ks = Qs + ROWS * P4;   // [KT][P4]
  float* const Ps = Ks + KT * P4;     // [ROWS][PP]
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, warp = tid >> 5, lane = tid & 31;
  sm100::pdl_wait();
  sm100::pdl_trigger();
  const int seg_lo = a.sched.worker_seg[blockIdx.x], seg_hi = a.sched.worker_seg[blockIdx.x + 1];
  const bool vec = (a.d_c & 3) == 0 && (d_cr & 3) == 0 && ((a.q_ts | a.q_hs) & 3) == 0 &&
                   ((reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.cache)) & 15) == 0;
  // One row into shared memory by a warp: the latent at 0, the position key
  // at dcp, zeros between and behind; a null source is a row of zeros.
  auto put_row = [&](float* dst, const float* src) {
    if (vec) {
      for (int v = lane; v < wq / 4; v += 32)
        reinterpret_cast<float4*>(dst)[v] =
            src && 4 * v < d_cr ? __ldg(reinterpret_cast<const float4*>(src) + v) : make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
      for (int c = lane; c < wq; c += 32) {
        const int e = c < dcp ? (c < a.d_c ? c : -1) : (c - dcp < a.d_r ? a.d_c + c - dcp : -1);
        dst[c] = src && e >= 0 ? __ldg(src + e) : 0.f;
      }
    }
  };

  for (int si = seg_lo; si < seg_hi; ++si) {
    const RSeg g = a.sched.segs[si];
    const int mi = ceil_div(g.nrows, 16);  // row groups that hold rows
    __syncthreads();
    for (int r = warp; r < 16 * mi; r += THREADS / 32) {
      const int row = g.row0 + r, t = row / a.n_h;
      put_row(Qs + r * P4, r < g.nrows ? a.q + t * a.q_ts + (row - t * a.n_h) * a.q_hs : nullptr);
    }
    int lim[4];
    float m[4], l[4], acc[4][NG][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty + 16 * i;
      lim[i] = r < g.nrows ? min(max(g.base + (g.row0 + r) / a.n_h + 1, 0), g.nkeys) : 0;
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < NG; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][c][e] = 0.f;
    }
    const int k_end = min(g.nkeys, g.t_hi * 64);
    for (int k0 = g.t_lo * 64; k0 < k_end; k0 += KT) {
      __syncthreads();
      {
        const int page = a.page_table[(long long)g.seq * a.max_pages + k0 / 64];
        const bool ok = page >= 0 && page < a.num_pages;
        if (!ok && tid == 0) flag_error(a.err, kErrBounds);
        const float* const src = a.cache + ((long long)(ok ? page : 0) * 64 + k0 % 64) * d_cr;
        for (int r = warp; r < KT; r += THREADS / 32)
          put_row(Ks + r * P4, ok && k0 + r < k_end ? src + (long long)r * d_cr : nullptr);
      }
      __syncthreads();
      float s[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i][0] = s[i][1] = 0.f;
      for (int c = 0; c < wq; c += 4) {
        const float4 ka = *reinterpret_cast<const float4*>(Ks + tx * P4 + c);
        const float4 kb = *reinterpret_cast<const float4*>(Ks + (tx + 16) * P4 + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < mi) {
            const float4 q = *reinterpret_cast<const float4*>(Qs + (ty + 16 * i) * P4 + c);
            s[i][0] = fmaf(q.x, ka.x, fmaf(q.y, ka.y, fmaf(q.z, ka.z, fmaf(q.w, ka.w, s[i][0]))));
            s[i][1] = fmaf(q.x, kb.x, fmaf(q.y, kb.y, fmaf(q.z, kb.z, fmaf(q.w, kb.w, s[i][1]))));
          }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < mi) {
          const float x0 = k0 + tx < lim[i] ? s[i][0] * a.scale : -INFINITY;
          const float x1 = k0 + tx + 16 < lim[i] ? s[i][1] * a.scale : -INFINITY;
          float mx = fmaxf(x0, x1);
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          const float mn = fmaxf(m[i], mx), ref = ref_max(mn);
          const float corr = exp2f(m[i] - ref), p0 = exp2f(x0 - ref), p1 = exp2f(x1 - ref);
          float sum = p0 + p1;
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          l[i] = fmaf(l[i], corr, sum);
          m[i] = mn;
          Ps[(ty + 16 * i) * PP + tx] = p0;
          Ps[(ty + 16 * i) * PP + tx + 16] = p1;
#pragma unroll
          for (int c = 0; c < NG; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][c][e] *= corr;
        }
      __syncwarp();
      if (k0 + KT > g.kmin) {
        // Keys that only some of the rows see: a weight of 0 must not meet an
        // infinity or a NaN.  A row that does see one already has a NaN sum.
        __syncthreads();
        for (int x = tid; x < KT * dcp; x += THREADS) {
          const int r = x / dcp, c = x - r * dcp;
          if (k0 + r >= g.kmin && !isfinite(Ks[r * P4 + c])) Ks[r * P4 + c] = 0.f;
        }
        __syncthreads();
      }
#pragma unroll 2
      for (int k = 0; k < KT; k += 4) {
        float4 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < mi) p[i] = *reinterpret_cast<const float4*>(Ps + (ty + 16 * i) * PP + k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
          for (int c = 0; c < NG; ++c) {
            if (4 * tx + 64 * c >= dcp) continue;
            const float4 v = *reinterpret_cast<const float4*>(Ks + (k + kk) * P4 + 4 * tx + 64 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (i < mi) {
                const float w = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
                acc[i][c][0] = fmaf(w, v.x, acc[i][c][0]);
                acc[i][c][1] = fmaf(w, v.y, acc[i][c][1]);
                acc[i][c][2] = fmaf(w, v.z, acc[i][c][2]);
                acc[i][c][3] = fmaf(w, v.w, acc[i][c][3]);
              }
          }
      }
    }
    // A whole row block goes to out, a piece to its slot (columns outermost).
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty + 16 * i;
      if (r >= g.nrows) continue;
      const float inv = row_inv(l[i]);
      float* const dst = g.slot < 0 ? static_cast<float*>(a.o.out) + ((long long)g.row0 + r) * a.d_c
                                    : a.o.part_o + (long long)g.slot * a.d_c * ROWS + r;
      const int step = g.slot < 0 ? 1 : ROWS;
#pragma unroll
      for (int c = 0; c < NG; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int col = 4 * tx + 64 * c + e;
          if (col < a.d_c) dst[(long long)col * step] = acc[i][c][e] * inv;
        }
      if (tx == 0) {
        if (g.slot >= 0) a.o.part_ml[(long long)g.slot * ROWS + r] = make_float2(m[i], l[i]);
        else if (a.o.lse) a.o.lse[(long long)g.row0 + r] = row_lse(ref_max(m[i]), l[i]);
      }
    }
  }
}

}  // namespace ragged_simt
}  // namespace mla
