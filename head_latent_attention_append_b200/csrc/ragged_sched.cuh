// Schedule of the ragged attention: any number of new tokens per request.
//
// The queries are walked as one matrix of rows, row = token * n_h + head, and
// a row block is up to `rows` consecutive rows of ONE request (they share its
// keys): 128 heads of one token, or eight tokens of a 16-head model, so that a
// model with few heads still fills the tensor cores' 128 rows.  Row r of
// token t sees the keys at positions 0 .. t + base, base = kv_len -
// q_start[b + 1]; a row block walks the 64-key tiles that its last row sees.
//
// Every worker takes an equal, contiguous share of all tiles in row-block
// order (a row block counts kBlockTiles more tiles for what it costs to change
// query rows), so a share may cut a row block into pieces, which
// ragged_combine_kernel merges.  All integer arithmetic: the cuts depend on
// the lengths alone.
#pragma once
#include "sched.cuh"
#include "sm100.cuh"

namespace mla {

constexpr int kRaggedMaxB = 16384;      // requests whose row-block offsets sit in shared memory
constexpr int kRaggedSmemInts = 56000;  // 4-byte words of shared memory the schedule may use

struct __align__(16) RSeg {
  int row0, nrows;  // the row block's rows
  int seq;          // its request
  int base;         // token t of the request is at position t + base
  int t_lo, t_hi;   // the tiles of this piece
  int slot;         // partial slot, or -1 for a whole row block
  int nkeys;        // keys that the last row sees
  int kmin;         // keys that the first row sees
  int pad[3];
};

struct RaggedSched {
  int* vs;          // [R+1] first (weighted) tile of each row block
  int* pc;          // [R+1] first segment of each row block
  int* worker_seg;  // [W+1] first segment of each worker
  RSeg* segs;       // [W+R]
  int* split;       // [1+W] count, then the first segment of each row block in pieces
};

struct RaggedSchedArgs {
  const int32_t* q_start;  // [B+1]
  const int32_t* kv_len;   // [B]
  int B, T, n_h, rows, W, max_pages, r_max, block_tiles;
  RaggedSched s;
  int* err;
  int smem_ints;           // words of dynamic shared memory
};

// Exclusive scan in place, with the total in 64 bits (data[] is meaningless
// if that does not fit in 32).
__device__ long long ragged_scan(int* data, int n) {
  __shared__ long long wide[32];
  const int T = blockDim.x, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int chunk = (n + T - 1) / T, lo = min(n, tid * chunk), hi = min(n, lo + chunk);
  long long s = 0;
  for (int i = lo; i < hi; ++i) s += data[i];
  long long x = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) wide[wid] = x;
  __syncthreads();
  long long before = 0, total = 0;
  for (int i = 0; i < (T >> 5); ++i) {
    if (i < wid) before += wide[i];
    total += wide[i];
  }
  int run = (int)(before + x - s);
  for (int i = lo; i < hi; ++i) {
    const int v = data[i];
    data[i] = run;
    run += v;
  }
  __syncthreads();
  return total;
}

__global__ void __launch_bounds__(1024) ragged_sched_kernel(const RaggedSchedArgs a) {
  extern __shared__ int rs_smem[];
  int* const bs = rs_smem;  // [B+1] first row block of each request
  const int tid = threadIdx.x, nt = blockDim.x;
  if (tid == 0) {
    *a.err = 0;
    a.s.split[0] = 0;
  }
  __syncthreads();
  // Starts that leave [0, T] or decrease leave nothing to compute; a length
  // outside its page table is clamped.
  int bad = 0;
  for (int b = tid; b < a.B; b += nt) {
    const int s0 = a.q_start[b], s1 = a.q_start[b + 1];
    if (s0 < 0 || s1 < s0 || s1 > a.T) bad = 1;
    const int n = bad ? 0 : s1 - s0, L = a.kv_len[b];
    if (n > 0 && (L < 0 || L > a.max_pages * 64LL)) flag_error(a.err, kErrBounds);
    bs[b] = (int)(((long long)n * a.n_h + a.rows - 1) / a.rows);
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) flag_error(a.err, kErrBounds);
    for (int w = tid; w <= a.W; w += nt) a.s.worker_seg[w] = 0;
    return;
  }
  const int R = (int)ragged_scan(bs, a.B);  // <= r_max: the starts are in order
  if (tid == 0) bs[a.B] = R;
  const bool in_smem = a.B + 1 + 2 * (R + 1) <= a.smem_ints;
  int* const vs = in_smem ? bs + a.B + 1 : a.s.vs;
  int* const pc = in_smem ? vs + R + 1 : a.s.pc;
  __syncthreads();

  auto block = [&](int rb) {
    RSeg g;
    const int b = find_le(bs, a.B, rb);
    const int s0 = a.q_start[b], s1 = a.q_start[b + 1];
    const int L = (int)min(max((long long)a.kv_len[b], 0LL), a.max_pages * 64LL);
    g.seq = b;
    g.row0 = s0 * a.n_h + (rb - bs[b]) * a.rows;
    g.nrows = min(a.rows, s1 * a.n_h - g.row0);
    g.base = L - s1;
    g.nkeys = max(0, g.base + (g.row0 + g.nrows - 1) / a.n_h + 1);
    g.kmin = max(0, g.base + g.row0 / a.n_h + 1);
    return g;
  };
  for (int rb = tid; rb < R; rb += nt) vs[rb] = max(1, ceil_div(block(rb).nkeys, 64)) + a.block_tiles;
  __syncthreads();
  const long long total64 = ragged_scan(vs, R);
  if (R == 0 || total64 > 0x7fffffffLL) {
    if (tid == 0 && R > 0) flag_error(a.err, kErrBounds);
    for (int w = tid; w <= a.W; w += nt) a.s.worker_seg[w] = 0;
    return;
  }
  const int total = (int)total64;
  if (tid == 0) vs[R] = total;
  const int W = min(a.W, total);  // every worker's share has at least one tile
  // The worker whose share [w total / W, (w + 1) total / W) holds tile x.
  auto owner = [&](int x) { return (int)((((long long)x + 1) * W - 1) / total); };
  __syncthreads();
  for (int rb = tid; rb < R; rb += nt) pc[rb] = owner(vs[rb + 1] - 1) - owner(vs[rb] + a.block_tiles) + 1;
  __syncthreads();
  const int nseg = (int)ragged_scan(pc, R);  // <= R + W
  if (tid == 0) pc[R] = nseg;
  __syncthreads();
  for (int s = tid; s < nseg; s += nt) {
    const int rb = find_le(pc, R, s), k = s - pc[rb], pieces = pc[rb + 1] - pc[rb];
    const int first = vs[rb] + a.block_tiles, w = owner(first) + k;
    RSeg g = block(rb);
    const long long lo = (long long)w * total / W, hi = (long long)(w + 1) * total / W;
    g.t_lo = (int)max(lo - first, 0LL);
    g.t_hi = (int)min(hi, (long long)vs[rb + 1]) - first;
    // Only the first and the last segment of a worker can be pieces.
    g.slot = pieces == 1 ? -1 : (k > 0 ? 2 * w : 2 * w + 1);
    g.pad[0] = g.pad[1] = g.pad[2] = 0;
    a.s.segs[s] = g;
    const int before = k > 0 ? w - 1 : (rb > 0 ? owner(vs[rb] - 1) : -1);  // the previous segment's worker
    for (int v = before + 1; v <= w; ++v) a.s.worker_seg[v] = s;
    if (s == nseg - 1)
      for (int v = w + 1; v <= a.W; ++v) a.s.worker_seg[v] = nseg;
    if (k == 0 && pieces > 1) a.s.split[1 + atomicAdd(&a.s.split[0], 1)] = s;
  }
}

// ------------------------------------------------------------------ combine
// What the attention kernels leave of a row block in pieces: in slot s, column
// by column, the piece's O / l (32 bits, rows contiguous, so that both sides
// move whole lines), and its (m, l) per row, in base 2:
//   m = max m_s,  l = sum 2^(m_s - m) l_s,  o = sum 2^(m_s - m) l_s N_s / l.
// One CTA merges 32 columns of a row block, its pieces in order.
// A row that sees no key of a piece (or none at all) has m = -inf and l = 0:
// its weights are taken relative to 0, its output is 0 and its lse -inf.  A
// NaN among its scores makes l, and with it the row, NaN.
__device__ __forceinline__ float ref_max(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ float row_inv(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float row_lse(float ref, float l) { return l == 0.f ? -INFINITY : ref + log2f(l); }

struct RaggedOut {
  void* out;       // [T * n_h][d_c]
  float* lse;      // [T * n_h] or null
  float* part_o;   // [2W][d_c][ROWS]
  float2* part_ml; // [2W][ROWS]
  int d_c;
};

constexpr int kCombineCols = 32, kCombineThreads = 256;

template <typename T, int ROWS>
__global__ void __launch_bounds__(kCombineThreads) ragged_combine_kernel(RaggedSched S, RaggedOut o, int W) {
  sm100::pdl_wait();
  sm100::pdl_trigger();
  constexpr int SUB = kCombineThreads / ROWS;   // threads per row
  constexpr int CPT = kCombineCols / SUB;       // columns per thread
  __shared__ int slots[2 * 160];
  __shared__ float tile[ROWS][kCombineCols + 1];
  if ((int)blockIdx.x >= S.split[0]) return;
  const int s0 = S.split[1 + blockIdx.x], nall = S.worker_seg[W];
  const RSeg g = S.segs[s0];
  const int tid = threadIdx.x;
  // The pieces of a row block follow one another, at most one per worker.
  int np = 0;
  for (int k0 = 0; k0 < W; k0 += kCombineThreads) {
    const int s = s0 + k0 + tid;
    const bool mine = s < nall && k0 + tid < W && S.segs[s].row0 == g.row0;
    if (mine) slots[k0 + tid] = S.segs[s].slot;
    np += __syncthreads_count(mine);
  }
  const int row = tid % ROWS, sub = tid / ROWS, c0 = blockIdx.y * kCombineCols + sub * CPT;
  float acc[CPT];
#pragma unroll
  for (int c = 0; c < CPT; ++c) acc[c] = 0.f;
  if (row < g.nrows) {
    float m = -INFINITY, l = 0.f;
    for (int k = 0; k < np; ++k) m = fmaxf(m, __ldcg(&o.part_ml[(long long)slots[k] * ROWS + row]).x);
    m = ref_max(m);
    for (int k = 0; k < np; ++k) {
      const float2 ml = __ldcg(&o.part_ml[(long long)slots[k] * ROWS + row]);
      const float w = exp2f(ml.x - m) * ml.y;
      const float* src = o.part_o + ((long long)slots[k] * o.d_c + c0) * ROWS + row;
#pragma unroll
      for (int c = 0; c < CPT; ++c)
        if (c0 + c < o.d_c) acc[c] = fmaf(w, __ldcg(src + c * ROWS), acc[c]);
      l += w;
    }
    const float inv = row_inv(l);
#pragma unroll
    for (int c = 0; c < CPT; ++c) acc[c] *= inv;
    if (o.lse && blockIdx.y == 0 && sub == 0) o.lse[(long long)g.row0 + row] = row_lse(m, l);
  }
#pragma unroll
  for (int c = 0; c < CPT; ++c) tile[row][sub * CPT + c] = acc[c];
  __syncthreads();
  const int cols = min(kCombineCols, o.d_c - (int)blockIdx.y * kCombineCols);
  T* const dst = static_cast<T*>(o.out) + (long long)g.row0 * o.d_c + blockIdx.y * kCombineCols;
  for (int i = tid; i < g.nrows * kCombineCols; i += kCombineThreads) {
    const int r = i / kCombineCols, c = i % kCombineCols;
    if (c < cols) dst[(long long)r * o.d_c + c] = from_f32<T>(tile[r][c]);
  }
}

}  // namespace mla
