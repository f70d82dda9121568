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
// order (a row block counts some more tiles for what it costs to change query
// rows), so a share may cut a row block into pieces, which
// ragged_combine_kernel merges.  All integer arithmetic: the cuts depend on
// the lengths alone.
#pragma once
#include "sched.cuh"
#include "sm100.cuh"

namespace mla {

constexpr int kRaggedMaxB = 16384;      // requests whose row-block offsets sit in shared memory
constexpr int kRaggedSmemInts = 47000;  // 4-byte words of dynamic shared memory the schedule may use

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
  int* wf;          // [R]   worker of that segment
  int2* range;      // [W] each worker's segments, [x, y); CTAs that make their own schedule: [CTAs], each its own copy
  RSeg* segs;       // [W+R]
  RSeg* first;      // [W]   a copy of each worker's first segment, which it reads beside its two numbers
  int4* split;      // [W] the row block whose first piece is this worker's last segment: first row, rows, -, pieces
                    // (one per worker from there on); 0 pieces: none
  int* worker_err;  // [CTAs of the attention kernel] each one's error bits
};

// The partial slot of piece k of a row block whose first piece is worker w0's:
// that one is its worker's last segment, the others are their workers' first.
__host__ __device__ __forceinline__ int ragged_slot(int w0, int k) { return k > 0 ? 2 * (w0 + k) : 2 * w0 + 1; }

struct RaggedSchedArgs {
  const int32_t* q_start;  // [B+1]
  const int32_t* kv_len;   // [B]
  int B, T, n_h, rows, W, max_pages, block_tiles;
  int keep_err;            // the error word is an earlier launch's too: do not zero it
  RaggedSched s;
  int* err;
  int own;                 // every attention CTA makes its worker's schedule, else ragged_sched_kernel all of it
  int one_go;              // the latter in one go
  int smem_ints;           // words of its dynamic shared memory
};

// Exclusive scan in place, with the total in 64 bits (data[] is meaningless
// if that does not fit in 32).  Out of line: the schedule is one pass over cold
// code, and a third of its time was instruction misses while this was in it
// three times.
__device__ __noinline__ long long ragged_scan(int* data, int n) {
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

// Exclusive scan of one value per thread (each below 2^25), with one barrier.
// `words`: two per warp, not used by another scan since the last barrier.
__device__ __forceinline__ int block_scan_once(int v, long long* words, long long* total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) words[wid] = x;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll 8
  for (int i = 0; i < warps; ++i) {
    const long long t = words[i];
    before += i < wid ? t : 0;
    all += t;
  }
  *total = all;
  return (int)before + x - v;
}

// Where row block `i` of the request whose rows start at token s0, end at s1
// and see L keys lies.
__device__ __forceinline__ RSeg ragged_block(const RaggedSchedArgs& a, int b, int i, int s0, int s1, int L) {
  RSeg g;
  g.seq = b;
  g.row0 = s0 * a.n_h + i * a.rows;
  g.nrows = min(a.rows, s1 * a.n_h - g.row0);
  g.base = L - s1;
  g.nkeys = max(0, g.base + (g.row0 + g.nrows - 1) / a.n_h + 1);
  g.kmin = max(0, g.base + g.row0 / a.n_h + 1);
  return g;
}
__device__ __forceinline__ int ragged_tiles(const RSeg& g) { return max(1, (g.nkeys + 63) >> 6); }

// The shares: worker w's starts at tile w len + min(w, rest).
struct RaggedShares {
  int total, W, len, rest, longer, block_tiles;
  __device__ __forceinline__ RaggedShares(int total_, int workers, int tiles)
      : total(total_), W(min(workers, total_)), block_tiles(tiles) {  // every share has at least one tile
    len = total / W;
    rest = total - len * W;
    longer = rest * (len + 1);
  }
  __device__ __forceinline__ int share(int w) const { return w * len + min(w, rest); }
  __device__ __forceinline__ int owner(int x) const {  // the worker whose share holds tile x
    const bool in = x < longer;
    return (in ? 0 : rest) + (x - (in ? 0 : longer)) / (in ? len + 1 : len);
  }
  // Segment s, piece k of `pieces` of the row block g whose (weighted) tiles
  // are [v0, v1), owned by worker w; `before`: the worker of
  // the segment before; `last`: the next one is another worker's.  `range`: where
  // the worker's segments are noted.
  __device__ __forceinline__ void emit(const RaggedSched& o, RSeg g, int s, int k, int pieces, int v0, int v1, int w,
                                       int before, bool last, int2* range) const {
    const int start = v0 + block_tiles;
    g.t_lo = max(share(w) - start, 0);
    g.t_hi = min(share(w + 1), v1) - start;
    // Only the first and the last segment of a worker can be pieces.
    g.slot = pieces == 1 ? -1 : ragged_slot(w - k, k);
    g.pad[0] = g.pad[1] = g.pad[2] = 0;
    o.segs[s] = g;
    if (before < w) {
      o.first[w] = g;
      range->x = s;
    }
    if (last) range->y = s + 1;
    if (k == 0 && pieces > 1) o.split[w] = make_int4(g.row0, g.nrows, 0, pieces);
  }
};

// Where a request's rows start and end and how many keys it sees; false for
// starts that leave [0, T] or decrease.  A length outside its page table is
// clamped and sets *range.
__device__ __forceinline__ bool ragged_request(const RaggedSchedArgs& a, int b, int& s0, int& s1, int& L, int& range) {
  s0 = a.q_start[b];
  s1 = a.q_start[b + 1];
  const long long len = a.kv_len[b], most = a.max_pages * 64LL;
  const bool ok = s0 >= 0 && s1 >= s0 && s1 <= a.T;
  if (ok && s1 > s0 && (len < 0 || len > most)) range = 1;
  L = (int)min(max(len, 0LL), most);
  return ok;
}
__device__ __forceinline__ int ragged_count(const RaggedSchedArgs& a, int s0, int s1) {
  return (int)(((long long)(s1 - s0) * a.n_h + a.rows - 1) / a.rows);
}

// The schedule in one go, for up to N requests and row blocks by N threads, with
// one barrier per sum.  `own`: the worker whose segments are kept, or -1 for all.
// Where an attention CTA has the threads, it does this for itself: one launch
// that does it for all, and the wait for it, cost 1 to 3 us (18.1 -> 17.0 for 8
// requests of one token, 49.0 -> 45.8 for 256; two of each per thread, 0.8 more).
// Behind that, up to 1024, the schedule kernel does (6 us less than its long way).
// Segment (row block, worker) has place row block + worker: along the schedule
// one of the two grows, so the places differ and a worker's are consecutive.
// `range`: worker max(own, 0)'s entry; the two CTAs of a pair note theirs apart, as
// one may be done while the other begins.  What else both write is the same.
// All threads of the block call it.
template <int N>
struct RaggedScratch {
  long long words[2][N / 32];
  int4 req[N];
  int bs[N];
};
template <int N>
__device__ __forceinline__ void ragged_schedule(const RaggedSchedArgs& a, RaggedScratch<N>& x, int own, int2* range,
                                                int* err) {
  const int tid = threadIdx.x, first = max(own, 0);  // tid: this thread's request and row block
  for (int w = first + tid; w < (own < 0 ? a.W : own + 1); w += N) {
    a.s.split[w] = make_int4(0, 0, 0, 0);
    range[w - first] = make_int2(0, 0);
  }
  int n = 0, bad = 0, clamped = 0;
  if (tid < a.B) {
    int4 q = make_int4(0, 0, 0, 0);
    if (ragged_request(a, tid, q.x, q.y, q.z, clamped)) n = ragged_count(a, q.x, q.y);
    else bad = 1;
    x.req[tid] = q;
  }
  const int none = __syncthreads_or(bad);
  if (clamped || (none && tid == 0)) flag_error(err, kErrBounds);
  if (none) return;
  long long sum;
  const int first_rb = block_scan_once(n, x.words[0], &sum);
  const int R = (int)sum;  // at most what the workspace holds: the starts are in order
  if (tid < a.B) x.bs[tid] = first_rb;
  __syncthreads();
  RSeg g{};
  int v = 0;
  if (tid < R) {
    const int b = find_le(x.bs, a.B, tid);
    const int4 q = x.req[b];
    g = ragged_block(a, b, tid - x.bs[b], q.x, q.y, q.z);
    v = ragged_tiles(g) + a.block_tiles;
  }
  const int v0 = block_scan_once(v, x.words[1], &sum), v1 = v0 + v;
  if (R == 0 || sum > 0x7fffffffLL) {
    if (tid == 0 && R > 0) flag_error(err, kErrBounds);
    return;
  }
  if (tid >= R) return;
  const RaggedShares sh((int)sum, a.W, a.block_tiles);
  const int w0 = sh.owner(v0 + a.block_tiles), w1 = sh.owner(v1 - 1);
  for (int w = own < 0 ? w0 : max(w0, own); w <= (own < 0 ? w1 : min(w1, own)); ++w) {
    const int before = w > w0 ? w - 1 : (v0 > 0 ? sh.owner(v0 - 1) : -1);
    const bool last = w < w1 || v1 == sh.total || sh.owner(v1 + a.block_tiles) > w;
    sh.emit(a.s, g, tid + w, w - w0, w1 - w0 + 1, v0, v1, w, before, last, range + (w - first));
  }
}

constexpr int kOneGoMost = 1024;

// The schedule of larger batches, in one launch for all workers.
__global__ void __launch_bounds__(1024) ragged_sched_kernel(const RaggedSchedArgs a) {
  extern __shared__ __align__(16) int rs_smem[];
  const int tid = threadIdx.x, nt = blockDim.x;
  sm100::pdl_wait();
  sm100::pdl_trigger();
  if (tid == 0 && !a.keep_err) *a.err = 0;
  if (a.one_go) {
    __syncthreads();  // the error word is zero
    ragged_schedule<kOneGoMost>(a, *reinterpret_cast<RaggedScratch<kOneGoMost>*>(rs_smem), -1, a.s.range, a.err);
    return;
  }
  for (int w = tid; w < a.W; w += nt) {
    a.s.split[w] = make_int4(0, 0, 0, 0);
    a.s.range[w] = make_int2(0, 0);
  }
  int* const off = rs_smem;  // [B+1] first row block of each request
  int bad = 0, range = 0;
  for (int b = tid; b < a.B; b += nt) {
    int s0, s1, L;
    const bool ok = ragged_request(a, b, s0, s1, L, range);
    if (!ok) bad = 1;
    off[b] = ok ? ragged_count(a, s0, s1) : 0;
  }
  const int none = __syncthreads_or(bad);
  if (range || (none && tid == 0)) flag_error(a.err, kErrBounds);
  if (none) return;

  const int R = (int)ragged_scan(off, a.B);  // at most what the workspace holds: the starts are in order
  if (tid == 0) off[a.B] = R;
  const bool in_smem = a.B + 1 + 3 * (R + 1) <= a.smem_ints;
  int* const vs = in_smem ? off + a.B + 1 : a.s.vs;
  int* const pc = in_smem ? vs + R + 1 : a.s.pc;
  int* const wf = in_smem ? pc + R + 1 : a.s.wf;
  __syncthreads();
  auto block = [&](int rb) {
    const int b = find_le(off, a.B, rb);
    int s0, s1, L, clamped;
    ragged_request(a, b, s0, s1, L, clamped);
    return ragged_block(a, b, rb - off[b], s0, s1, L);
  };
  for (int rb = tid; rb < R; rb += nt) vs[rb] = ragged_tiles(block(rb)) + a.block_tiles;
  __syncthreads();
  const long long total = ragged_scan(vs, R);
  if (R == 0 || total > 0x7fffffffLL) {
    if (tid == 0 && R > 0) flag_error(a.err, kErrBounds);
    return;
  }
  if (tid == 0) vs[R] = (int)total;
  const RaggedShares sh((int)total, a.W, a.block_tiles);
  __syncthreads();
  for (int rb = tid; rb < R; rb += nt) {
    wf[rb] = sh.owner(vs[rb] + a.block_tiles);
    pc[rb] = sh.owner(vs[rb + 1] - 1) - wf[rb] + 1;
  }
  __syncthreads();
  const int nseg = (int)ragged_scan(pc, R);  // <= R + W
  if (tid == 0) pc[R] = nseg;
  __syncthreads();
  for (int s = tid; s < nseg; s += nt) {
    const int rb = find_le(pc, R, s), k = s - pc[rb], w = wf[rb] + k;
    const int before = k > 0 ? w - 1 : (rb > 0 ? wf[rb - 1] + s - pc[rb - 1] - 1 : -1);
    sh.emit(a.s, block(rb), s, k, pc[rb + 1] - pc[rb], vs[rb], vs[rb + 1], w, before,
            s == nseg - 1 || k + 1 < pc[rb + 1] - pc[rb] || wf[rb + 1] > w, a.s.range + w);
  }
}

// ------------------------------------------------------------------ combine
// What the attention kernels leave of a row block in pieces: per slot s the
// piece's O / l in 32 bits and its (m, l) per row, in base 2:
//   m = max m_s,  l = sum 2^(m_s - m) l_s,  o = sum 2^(m_s - m) l_s N_s / l.
// The tensor-core kernel writes a slot column by column (rows contiguous, as
// its threads hold them), the CUDA-core kernel row by row (d_c padded to whole
// float4s), so that both move whole lines.
struct RaggedOut {
  void* out;       // [T * n_h][d_c]
  float* lse;      // [T * n_h] or null
  float* part_o;   // [2W][d_c][ROWS], or [2W][ROWS][d_c padded]
  float2* part_ml; // [2W][ROWS]
  int d_c;
};

// A row that sees no key of a piece (or none at all) has m = -inf and l = 0:
// its weights are taken relative to 0, its output is 0 and its lse -inf.  A
// NaN among its scores makes l, and with it the row, NaN.
__device__ __forceinline__ float ref_max(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ float row_inv(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float row_lse(float ref, float l) { return l == 0.f ? -INFINITY : ref + log2f(l); }

// One CTA merges kCombineCols columns of a row block, in order, kBatch pieces
// at a time: their O (16 bytes per load: four rows of a column, or four columns
// of a row) and (m, l) are asked for together, then the rows' maximum, weights
// and sum are brought up to date in shared memory as an online softmax does,
// and the batch is added.  Bound by latency (some pieces of a few hundred KB
// in all, from L2), hence one pass: about 4 us for eight row blocks of nine
// pieces.  The first CTA also gathers the attention CTAs' error bits into the
// call's error word (`keep_err`: beside what an earlier launch left there).
constexpr int kCombineCols = 16, kCombineThreads = 128, kBatch = 4;

template <typename T, int ROWS, bool kByColumn>
__global__ void __launch_bounds__(kCombineThreads) ragged_combine_kernel(RaggedSched S, RaggedOut o, int err_ctas, int* err,
                                                                         int keep_err) {
  sm100::pdl_wait();
  sm100::pdl_trigger();
  constexpr int QUADS = ROWS * kCombineCols / 4 / kCombineThreads;  // 16-byte items per thread
  static_assert(ROWS <= kCombineThreads && QUADS >= 1, "a thread keeps one row's state");
  __shared__ __align__(16) float coef[kBatch + 1][ROWS];  // weights of the batch, factor for what came before
  __shared__ float tile[kByColumn ? ROWS : 1][kCombineCols + 1];
  __shared__ float inv_of[ROWS];
  const int tid = threadIdx.x;
  const int4 e = S.split[blockIdx.x];
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid < 32) {
    int bits = 0;
    for (int i = tid; i < err_ctas; i += 32) bits |= S.worker_err[i];
    bits = __reduce_or_sync(0xffffffffu, bits);
    if (tid == 0) *err = bits | (keep_err ? *err : 0);
  }
  const int row0 = e.x, nrows = e.y, w0 = blockIdx.x, np = e.w;
  if (np == 0) return;
  const int col0 = blockIdx.y * kCombineCols, cols = min(kCombineCols, o.d_c - col0);
  const int pitch = kByColumn ? o.d_c : (o.d_c + 3) & ~3;
  const long long slot_elems = (long long)pitch * ROWS;
  // Items: quads of rows of a column (consecutive in the slot's column), or
  // quads of columns of a row.  pos: the row (of the first of the four), lane
  // of the item within it: the column.
  const int minor = kByColumn ? (nrows + 3) / 4 : (cols + 3) / 4;
  const int items = minor * (kByColumn ? cols : nrows);
  int row[QUADS], col[QUADS];
  float4 acc[QUADS];
#pragma unroll
  for (int i = 0; i < QUADS; ++i) {
    const int x = tid + i * kCombineThreads, major = x / minor, quad = 4 * (x - major * minor);
    row[i] = x < items ? (kByColumn ? quad : major) : -1;
    col[i] = col0 + (kByColumn ? major : quad);
    acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float m = -INFINITY, l = 0.f;  // of row `tid`
  for (int k0 = 0; k0 < np; k0 += kBatch) {
    float2 ml[kBatch];
    float4 v[QUADS][kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const long long slot = ragged_slot(w0, k0 + k);
      ml[k] = tid < nrows && k0 + k < np ? __ldcg(&o.part_ml[slot * ROWS + tid]) : make_float2(-INFINITY, 0.f);
    }
#pragma unroll
    for (int i = 0; i < QUADS; ++i)
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (row[i] >= 0 && k0 + k < np) {
          const long long off = kByColumn ? (long long)col[i] * ROWS + row[i] : (long long)row[i] * pitch + col[i];
          v[i][k] = __ldcg(reinterpret_cast<const float4*>(o.part_o + ragged_slot(w0, k0 + k) * slot_elems + off));
        }
    if (tid < nrows) {
      float mn = m;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) mn = fmaxf(mn, ml[k].x);
      const float ref = ref_max(mn), f = exp2f(m - ref);
      l *= f;
      coef[kBatch][tid] = f;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float w = exp2f(ml[k].x - ref) * ml[k].y;
        coef[k][tid] = w;
        l += w;
      }
      m = mn;
      inv_of[tid] = row_inv(l);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < QUADS; ++i) {
      if (row[i] < 0) continue;
      auto weights = [&](int k) {
        if constexpr (kByColumn) return *reinterpret_cast<const float4*>(&coef[k][row[i]]);
        const float c = coef[k][row[i]];
        return make_float4(c, c, c, c);
      };
      const float4 f = weights(kBatch);
      acc[i] = make_float4(acc[i].x * f.x, acc[i].y * f.y, acc[i].z * f.z, acc[i].w * f.w);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (k0 + k >= np) break;
        const float4 c = weights(k);
        acc[i].x = fmaf(c.x, v[i][k].x, acc[i].x);
        acc[i].y = fmaf(c.y, v[i][k].y, acc[i].y);
        acc[i].z = fmaf(c.z, v[i][k].z, acc[i].z);
        acc[i].w = fmaf(c.w, v[i][k].w, acc[i].w);
      }
    }
    __syncthreads();
  }
  if (o.lse && blockIdx.y == 0 && tid < nrows) o.lse[(long long)row0 + tid] = row_lse(ref_max(m), l);
  T* const dst = static_cast<T*>(o.out) + (long long)row0 * o.d_c;
  if constexpr (kByColumn) {
    // The rows behind nrows of a last group of four are never written to a
    // slot; what they leave in the tile is not stored.
#pragma unroll
    for (int i = 0; i < QUADS; ++i)
      if (row[i] >= 0) {
        const int c = col[i] - col0;
        tile[row[i]][c] = acc[i].x;
        tile[row[i] + 1][c] = acc[i].y;
        tile[row[i] + 2][c] = acc[i].z;
        tile[row[i] + 3][c] = acc[i].w;
      }
    __syncthreads();
    for (int x = tid; x < nrows * kCombineCols; x += kCombineThreads) {
      const int r = x / kCombineCols, c = x % kCombineCols;
      if (c < cols) dst[(long long)r * o.d_c + col0 + c] = from_f32<T>(tile[r][c] * inv_of[r]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < QUADS; ++i)
      if (row[i] >= 0) {
        const float f = inv_of[row[i]], w[4] = {acc[i].x, acc[i].y, acc[i].z, acc[i].w};
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (col[i] + c < o.d_c) dst[(long long)row[i] * o.d_c + col[i] + c] = from_f32<T>(w[c] * f);
      }
  }
}

}  // namespace mla
