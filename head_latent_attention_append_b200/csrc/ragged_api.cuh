// Host side of the ragged-step entry points (include/mla.h): argument checks,
// workspace layout and launches.  Part of mla_api.cu, whose helpers it uses.
#pragma once

namespace {

// Workers of the ragged attention: CTA pairs on the tensor cores, CTAs on the
// CUDA cores.  The caps size the partial slots.
constexpr int kRaggedPairs = 80, kRaggedCtas = 160;
// What changing query rows costs a worker, in tiles of 64 keys: the next rows'
// load and this block's output, about 6 us against 0.8 us a tile of a wide row
// on the tensor cores; small against a tile on the CUDA cores.  Measured on
// batches of 64 to 330 row blocks: with d_c = 512, 3, 6, 9 and 12 tiles gave 249,
// 238, 232 and 234 us; with d_c = 256, 35.0, 33.5, 35.1 and 36.5.  The widths 128
// and 384 take the line through these two points; they were not measured.
int block_tiles(const mla_dims& d) { return d.dtype == MLA_BF16 ? 3 + 3 * d.d_c / 256 : 1; }

struct RaggedPlan {
  size_t hdr, vs, pc, wf, range, segs, first, split, worker_err, part_o, part_ml, total;
  int rows, cap, r_max;
};
RaggedPlan make_ragged_plan(const mla_dims& d, int B, int T) {
  RaggedPlan P{};
  const bool tc = d.dtype == MLA_BF16;
  P.rows = tc ? ragged_tc::ROWS : ragged_simt::ROWS;
  P.cap = tc ? kRaggedPairs : kRaggedCtas;
  P.r_max = (int)((long long)T * d.n_h / P.rows) + std::min(B, T);
  size_t o = 256;
  P.vs = o;         o = align_up(o + sizeof(int) * ((size_t)P.r_max + 1), 256);
  P.pc = o;         o = align_up(o + sizeof(int) * ((size_t)P.r_max + 1), 256);
  P.wf = o;         o = align_up(o + sizeof(int) * ((size_t)P.r_max + 1), 256);
  P.range = o;      o = align_up(o + sizeof(int2) * 2 * (size_t)P.cap, 256);
  P.segs = o;       o = align_up(o + sizeof(RSeg) * ((size_t)P.cap + P.r_max), 256);
  P.first = o;      o = align_up(o + sizeof(RSeg) * (size_t)P.cap, 256);
  P.split = o;      o = align_up(o + sizeof(int4) * (size_t)P.cap, 256);
  P.worker_err = o; o = align_up(o + sizeof(int) * 2 * (size_t)P.cap, 256);
  P.part_o = o;     o = align_up(o + sizeof(float) * 2 * P.cap * P.rows * (size_t)align_up(d.d_c, 4), 256);
  P.part_ml = o;    o = align_up(o + sizeof(float2) * 2 * P.cap * P.rows, 256);
  P.total = o;
  return P;
}

mla_status check_ragged(const mla_dims* dims, int B, int T) {
  mla_status s = check_dims(dims);
  if (s != MLA_OK) return s;
  if (B <= 0 || T < 0) return MLA_ERR_INVALID_ARG;
  // One shared position key (a per-head one has no dense score product); row
  // and row-block counts in 32 bits.
  if (dims->rope_key_per_head || B > kRaggedMaxB || (long long)T * dims->n_h > INT_MAX - ragged_tc::ROWS)
    return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}

// Whether [a, a + na) and [b, b + nb) share a byte.
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na && nb && x < y + nb && y < x + na;
}

// The bytes of a tensor of rows: n groups s bytes apart, each of m rows of w
// bytes hs apart (rows do not overlap and come in order).
struct RowSet {
  uintptr_t p;
  long long n, s, m, hs, w;
  uintptr_t end;  // behind the last row (0 where there are no rows)
  RowSet(const void* p_, long long n_, long long s_, long long m_, long long hs_, long long w_)
      : p(reinterpret_cast<uintptr_t>(p_)), n(n_), s(s_), m(m_), hs(hs_), w(w_), end(n ? p + (n - 1) * s + extent() : 0) {}
  RowSet(const void* p_, long long bytes) : RowSet(p_, p_ && bytes ? 1 : 0, bytes, 1, bytes, bytes) {}
  long long extent() const { return (m - 1) * hs + w; }
};
bool same_rows(const RowSet& a, const RowSet& b) {
  return a.p == b.p && a.n == b.n && a.m == b.m && a.w == b.w && (a.n <= 1 || a.s == b.s) && (a.m <= 1 || a.hs == b.hs);
}
// Whether a group of `a` and one of `b` that starts `d` bytes behind it share a byte.
bool groups_meet(const RowSet& a, const RowSet& b, long long d) {
  for (long long i = 0, j = 0; i < a.m && j < b.m;) {
    const long long x = i * a.hs, y = d + j * b.hs;
    if (x < y + b.w && y < x + a.w) return true;
    if (x < y) ++i;
    else ++j;
  }
  return false;
}
// Whether two tensors with rows share a byte.  Interleaved ones (slices of one
// wider row) do not; they have one stride, for which a few groups tell of all.
__attribute__((noinline)) bool rows_cross(RowSet a, RowSet b) {
  const long long d = (long long)(b.p - a.p), ea = a.extent(), eb = b.extent();
  if (a.n == 1) a.s = b.s;
  if (b.n == 1) b.s = a.s;
  if (a.s == b.s) {
    // Group j of b against group j - k of a: d + k s bytes apart.
    const long long first = (-eb - d) / a.s - 1;
    for (long long k = std::max(1 - a.n, first); k < b.n && d + k * a.s < ea; ++k)
      if (d + k * a.s > -eb && groups_meet(a, b, d + k * a.s)) return true;
    return false;
  }
  for (long long i = 0, j = 0; i < a.n && j < b.n;) {
    const long long x = i * a.s, y = d + j * b.s;
    if (x < y + eb && y < x + ea && groups_meet(a, b, y - x)) return true;
    if (x + ea < y + eb) ++i;
    else ++j;
  }
  return false;
}
// The same for any two: tensors apart, the usual case, cost two comparisons
// (all of a call's together some tens of nanoseconds).
inline bool rows_meet(const RowSet& a, const RowSet& b) { return a.p < b.end && b.p < a.end && rows_cross(a, b); }

// RoPE frequencies as turns per position.
step::Rope rope_table(const mla_dims& d) {
  static thread_local step::Rope last;
  static thread_local float last_base = 0.f;
  if (last.half != d.d_r / 2 || last_base != d.rope_base) {
    last.half = d.d_r / 2;
    last_base = d.rope_base;
    for (int i = 0; i < last.half; ++i)
      last.turns[i] = pow((double)d.rope_base, -2.0 * i / d.d_r) / 6.283185307179586476925286766559;
  }
  return last;
}

template <int NPV>
cudaError_t launch_ragged_tc(const CUtensorMap& mapS, const CUtensorMap& mapV, const ragged_tc::Args& a, int W,
                             cudaStream_t st) {
  auto kfn = ragged_tc::attn_ragged_kernel<NPV>;
  cudaError_t e = set_smem_once(kfn, ragged_tc::SMEM_BYTES);
  if (e) return e;
  return launch_pdl(kfn, dim3(2 * W), dim3(ragged_tc::THREADS), ragged_tc::SMEM_BYTES, st, mapS, mapV, a);
}

template <int NC>
cudaError_t launch_ragged_simt(const ragged_simt::Args& a, int W, cudaStream_t st) {
  auto kfn = ragged_simt::attn_ragged_simt_kernel<NC>;
  const size_t sm = ragged_simt::smem_bytes(a.d_c, a.d_r, a.buffers);
  cudaError_t e = set_smem_once(kfn, ragged_simt::MAX_SMEM);
  if (e) return e;
  return launch_pdl(kfn, dim3(W), dim3(ragged_simt::THREADS), sm, st, a);
}

// Rows per block of the normalised append: one, until the blocks fill the GPU
// eight times over; then each walks several.
template <typename T>
cudaError_t launch_norm_append(const step::NormAppendArgs& a, bool vec, cudaStream_t st) {
  const int ve = vec ? 16 / (int)sizeof(T) : 1, per = a.cq ? 1 : step::NORM_THREADS / 32;
  const int grid = std::min(ceil_div(a.T, per), 8 * num_sms());
  const bool small = a.d_c <= 2 * 32 * ve && a.d_cq <= 2 * 96 * ve;  // two vectors a thread
  const dim3 threads(step::NORM_THREADS);
  if (!vec) return launch_pdl(step::norm_append_kernel<T, false, 4>, dim3(grid), threads, 0, st, a);
  if (small) return launch_pdl(step::norm_append_kernel<T, true, 2>, dim3(grid), threads, 0, st, a);
  return launch_pdl(step::norm_append_kernel<T, true, 4>, dim3(grid), threads, 0, st, a);
}

template <typename T, bool kVec, int G, int VPL>
cudaError_t launch_query(step::QueryArgs& a, cudaStream_t st) {
  // Heads per block: all of a token's, unless that leaves the GPU with fewer
  // than sixteen blocks an SM; then fewer, in whole steps.
  const int step_heads = 2 * (step::QUERY_THREADS / G), steps = ceil_div(a.n_h, step_heads);
  const int want = ceil_div(16 * num_sms(), a.T), parts = std::max(1, std::min(steps, want));
  a.hpb = step_heads * ceil_div(steps, parts);
  return launch_pdl(step::query_norm_rope_kernel<T, kVec, G, VPL>, dim3((unsigned)a.T, (unsigned)ceil_div(a.n_h, a.hpb)),
                    dim3(step::QUERY_THREADS), 0, st, a);
}
template <typename T>
cudaError_t launch_query(step::QueryArgs& a, bool vec, cudaStream_t st) {
  const int ve = 16 / (int)sizeof(T), parts = vec ? a.d_r / ve : a.d_r / 2;  // vectors or pairs of a position part
  for (a.rope_shift = 0; (1 << a.rope_shift) < parts;) ++a.rope_shift;
  if (!vec) return launch_query<T, false, 32, 4>(a, st);
  const int nv = a.d_h / ve;
  if (nv <= 4) return launch_query<T, true, 4, 1>(a, st);
  if (nv <= 8) return launch_query<T, true, 8, 1>(a, st);
  if (nv <= 16) return launch_query<T, true, 16, 1>(a, st);
  if (nv <= 32) return launch_query<T, true, 32, 1>(a, st);
  return launch_query<T, true, 32, 4>(a, st);
}

// Schedule (in the attention kernel, where the batch is small enough),
// attention, merge of the row blocks in pieces.  `err`: the error word, zeroed
// or written by the first launch here that reports, unless an earlier one of the
// call reports there too.
mla_status attend_ragged_impl(const mla_dims& d, const void* q, long long q_ts, long long q_hs, const int32_t* q_start,
                              const int32_t* kv_len, const int32_t* page_table, int B, int T, int max_pages,
                              int num_pages, const void* cache, void* out, float* lse, void* ws, const RaggedPlan& P,
                              int* err, bool keep_err, cudaStream_t st) {
  const bool tc = d.dtype == MLA_BF16;
  const int W = std::max(1, std::min(P.cap, tc ? num_sms() / 2 : num_sms()));
  const float scale =
      (float)((d.softmax_scale > 0.f ? (double)d.softmax_scale : 1.0 / sqrt((double)(d.d_h + d.d_r))) * kLog2e);
  const RaggedSched S{at<int>(ws, P.vs), at<int>(ws, P.pc), at<int>(ws, P.wf), at<int2>(ws, P.range),
                      at<RSeg>(ws, P.segs), at<RSeg>(ws, P.first), at<int4>(ws, P.split), at<int>(ws, P.worker_err)};
  const RaggedOut o{out, lse, at<float>(ws, P.part_o), at<float2>(ws, P.part_ml), d.d_c};
  cudaError_t e;
  // Who makes the schedule (ragged_schedule).
  const bool own = std::max(B, P.r_max) <= (tc ? ragged_tc::kOwnMost : ragged_simt::kOwnMost);
  const bool one_go = std::max(B, P.r_max) <= kOneGoMost;
  const int ints = one_go ? (int)(sizeof(RaggedScratch<kOneGoMost>) / sizeof(int))
                          : (int)std::min<long long>(B + 1 + 3LL * (P.r_max + 1), kRaggedSmemInts);
  const RaggedSchedArgs sa{q_start, kv_len, B, T, d.n_h, P.rows, W, max_pages, block_tiles(d), keep_err, S, err, own,
                           one_go, ints};
  if (!own) {
    if ((e = set_smem_once(ragged_sched_kernel, sizeof(int) * (size_t)kRaggedSmemInts))) return cuda_status(e);
    ++g_launches;
    if ((e = launch_pdl(ragged_sched_kernel, dim3(1), dim3(1024), sizeof(int) * (size_t)ints, st, sa)))
      return cuda_status(e);
  }
  ++g_launches;
  prof_mark(st, true);
  if (tc) {
    ragged_tc::Args a{static_cast<const __nv_bfloat16*>(q), q_ts, q_hs, page_table, max_pages, num_pages, d.n_h, d.d_c,
                      d.d_c + d.d_r, scale, q_hs == d.d_c + d.d_r && q_ts == d.n_h * q_hs, sa, o};
    // Score ring: 32-row boxes (one CTA's keys of a page); latent ring: 64-row boxes.
    CUtensorMap mapS, mapV;
    const long long rows = (long long)num_pages * d.page_size;
    if (!encode_cache_map(&mapS, cache, a.q_row, rows, 32) || !encode_cache_map(&mapV, cache, a.q_row, rows, 64))
      return MLA_ERR_CUDA;
    switch (d.d_c / 128) {
      case 1: e = launch_ragged_tc<1>(mapS, mapV, a, W, st); break;
      case 2: e = launch_ragged_tc<2>(mapS, mapV, a, W, st); break;
      case 3: e = launch_ragged_tc<3>(mapS, mapV, a, W, st); break;
      default: e = launch_ragged_tc<4>(mapS, mapV, a, W, st); break;
    }
  } else {
    ragged_simt::Args a{static_cast<const float*>(q), q_ts, q_hs, static_cast<const float*>(cache), page_table,
                        max_pages, num_pages, d.n_h, d.d_c, d.d_r, ragged_simt::key_buffers(d.d_c, d.d_r), scale, sa, o};
    if (d.d_c <= 128) e = launch_ragged_simt<1>(a, W, st);
    else if (d.d_c <= 256) e = launch_ragged_simt<2>(a, W, st);
    else e = launch_ragged_simt<4>(a, W, st);
  }
  if (e) return cuda_status(e);
  prof_mark(st, false);
  ++g_launches;
  const dim3 grid(W, ceil_div(d.d_c, kCombineCols));
  const int err_ctas = tc ? 2 * W : W, keep = keep_err || !own;  // the schedule kernel leaves bits there too
  if (tc)
    e = launch_pdl(ragged_combine_kernel<__nv_bfloat16, ragged_tc::ROWS, true>, grid, dim3(kCombineThreads), 0, st, S, o,
                   err_ctas, err, keep);
  else
    e = launch_pdl(ragged_combine_kernel<float, ragged_simt::ROWS, false>, grid, dim3(kCombineThreads), 0, st, S, o,
                   err_ctas, err, keep);
  return cuda_status(e);
}

// The whole ragged step from hidden states: the projections' scratch first
// (its header holds the error word), then the intermediates, then the ragged
// attention's workspace.
struct RaggedStepPlan {
  Plan base;  // hdr, counters, partial
  size_t cq, qc, qabs, obar, ragged, total;
  RaggedPlan attend;
};
RaggedStepPlan make_ragged_step_plan(const mla_dims& d, int B, int T) {
  RaggedStepPlan P{};
  const size_t e = esize(d), n = (size_t)T * d.n_h;
  P.base = make_plan(d, T, false);
  size_t o = P.base.total;
  P.cq = o;     o = align_up(o + e * (size_t)T * d.d_cq, 256);
  P.qc = o;     o = align_up(o + e * n * d.d_h, 256);
  P.qabs = o;   o = align_up(o + e * n * (d.d_c + d.d_r), 256);
  P.obar = o;   o = align_up(o + e * n * d.d_c, 256);
  P.ragged = o;
  P.attend = make_ragged_plan(d, B, T);
  P.total = o + P.attend.total;
  return P;
}

template <typename T>
mla_status ragged_step_impl(const mla_weights* w, const void* h, const int32_t* q_start, const int32_t* kv_len,
                            const int32_t* seq_idx, const int32_t* pos, const int32_t* page_table, int B, int T_,
                            int max_pages, int num_pages, void* cache, float* out, void* ws, const RaggedStepPlan& P,
                            cudaStream_t st) {
  const mla_dims& d = w->d;
  const int din = d_in(d), q_row = d.d_c + d.d_r;
  cudaError_t e;
  // (1) the new tokens' cache rows.
  mla_status s = append_impl<T>(w, h, seq_idx, pos, 0, B, page_table, max_pages, num_pages, cache, T_, ws, P.base, st,
                                nullptr, 0, kSplitKTileSplits, INT_MAX, true);
  if (s != MLA_OK) return s;
  // (2) query latent, (3) q_C and the rotated q_R, (4) absorption.  The scale
  // is the attention's, in 32 bits.
  const void* src = h;
  if (d.d_cq > 0) {
    EpiStore<T> epi{at<T>(ws, P.cq), d.d_cq, 0, 1.f};
    if ((e = gemm<T>(h, d.d_model, 0, w->dq, d.d_model, 0, T_, d.d_cq, d.d_model, 1, epi, ws, P.base, st)))
      return cuda_status(e);
    src = at<T>(ws, P.cq);
  }
  {
    EpiQProj<T> epi{};
    epi.qc = at<T>(ws, P.qc);
    epi.qabs = at<T>(ws, P.qabs);
    for (int i = 0; i < d.d_r / 2; ++i) epi.theta[i] = w->theta[i];
    epi.n_h = d.n_h; epi.d_h = d.d_h; epi.d_r = d.d_r; epi.d_c = d.d_c; epi.d_cr = q_row;
    epi.qabs_rows = d.n_h;
    epi.qr_scale = 1.f;
    epi.pos = pos;
    if ((e = gemm<T>(src, din, 0, w->uqr, din, 0, T_, d.n_h * (d.d_h + d.d_r), din, 1, epi, ws, P.base, st)))
      return cuda_status(e);
  }
  {
    EpiStore<T> epi{at<T>(ws, P.qabs), (long long)d.n_h * q_row, q_row, 1.f};
    if ((e = gemm<T>(at<T>(ws, P.qc), (long long)d.n_h * d.d_h, d.d_h, w->ukt, d.d_h, (long long)d.d_c * d.d_h, T_,
                     d.d_c, d.d_h, d.n_h, epi, ws, P.base, st)))
      return cuda_status(e);
  }
  // (5) attention on the latent cache, (6) o_h = W_UV,h obar_h.
  s = attend_ragged_impl(d, at<T>(ws, P.qabs), (long long)d.n_h * q_row, q_row, q_start, kv_len, page_table, B, T_,
                         max_pages, num_pages, cache, at<T>(ws, P.obar), nullptr, at<char>(ws, P.ragged), P.attend,
                         at<int>(ws, P.base.hdr), true, st);
  if (s != MLA_OK) return s;
  EpiStore<float> epi{out, (long long)d.n_h * d.d_v, d.d_v, 1.f};
  return cuda_status(gemm<T>(at<T>(ws, P.obar), (long long)d.n_h * d.d_c, d.d_c, w->uv, d.d_c,
                             (long long)d.d_v * d.d_c, T_, d.d_v, d.d_c, d.n_h, epi, ws, P.base, st));
}

}  // namespace

extern "C" {

mla_status mla_plan_step(const int32_t* new_len, const int32_t* past_len, int B, const int32_t* free_pages, int n_free,
                         int32_t* page_table, int max_pages, int num_pages, int32_t* q_start, int32_t* kv_len,
                         int32_t* seq_idx, int32_t* pos, int64_t* slot, int rows, int32_t* counts,
                         int32_t* device_error, cudaStream_t stream) {
  if (B <= 0 || n_free < 0 || max_pages <= 0 || num_pages <= 0 || rows < 0) return MLA_ERR_INVALID_ARG;
  if (!new_len || !past_len || !page_table || !q_start || !kv_len || !counts || (n_free > 0 && !free_pages) ||
      (rows > 0 && (!seq_idx || !pos || !slot)))
    return MLA_ERR_INVALID_ARG;
  if (!aligned(slot, 8) || !aligned(new_len, 4) || !aligned(past_len, 4) || !aligned(free_pages, 4) ||
      !aligned(page_table, 4) || !aligned(q_start, 4) || !aligned(kv_len, 4) || !aligned(seq_idx, 4) ||
      !aligned(pos, 4) || !aligned(counts, 4) || !aligned(device_error, 4))
    return MLA_ERR_INVALID_ARG;
  // Sums and positions in 32 bits.
  if (B > step::PLAN_MAX_B || rows > (1 << 30) || n_free > (1 << 30) || max_pages > INT_MAX / 64 - 1)
    return MLA_ERR_UNSUPPORTED;
  // Every CTA reads all lengths while others write: an output in their place
  // (kv_len for past_len, say) would be read half updated.
  const size_t i32 = sizeof(int32_t), nb = B * i32, nr = rows * i32;
  const struct { const void* p; size_t n; } in[] = {{new_len, nb}, {past_len, nb}, {free_pages, n_free * i32}},
      out[] = {{page_table, nb * (size_t)max_pages}, {q_start, nb + i32}, {kv_len, nb}, {seq_idx, nr}, {pos, nr},
               {slot, 2 * nr}, {counts, 3 * i32}};
  for (const auto& x : in)
    for (const auto& y : out)
      if (overlap(x.p, x.n, y.p, y.n)) return MLA_ERR_INVALID_ARG;
  const step::PlanArgs a{new_len, past_len, free_pages, page_table, q_start, kv_len,    seq_idx, pos,
                         slot,    counts,   device_error, B,        n_free,  max_pages, num_pages, rows};
  const size_t sm = sizeof(uint32_t) * 2 * ((size_t)B + 1);
  cudaError_t e = set_smem_once(step::plan_kernel, sizeof(uint32_t) * 2 * ((size_t)step::PLAN_MAX_B + 1));
  if (e) return cuda_status(e);
  g_launches = 1;
  const int ctas = std::min(num_sms(), ceil_div(std::max(rows, B + 1), step::PLAN_THREADS));
  return cuda_status(launch_pdl(step::plan_kernel, dim3(ctas), dim3(step::PLAN_THREADS), sm, stream, a));
}

mla_status mla_append_normed(const mla_dims* dims, const void* kv, int64_t kv_stride, const void* kv_gamma,
                             const void* cq, int64_t cq_stride, const void* cq_gamma, void* cq_out,
                             int64_t cq_out_stride, float eps, const int32_t* pos, const int64_t* slot, void* cache,
                             int num_pages, int T, int32_t* device_error, cudaStream_t stream) {
  mla_status s = check_dims(dims);
  if (s != MLA_OK) return s;
  const mla_dims& d = *dims;
  const int d_cr = cache_row(d);
  if (T < 0 || num_pages <= 0 || !(eps >= 0.f) || kv_stride < d_cr) return MLA_ERR_INVALID_ARG;
  if ((cq != nullptr) != (cq_out != nullptr) || (!cq && cq_gamma)) return MLA_ERR_INVALID_ARG;
  if (cq && (d.d_cq <= 0 || cq_stride < d.d_cq || cq_out_stride < d.d_cq)) return MLA_ERR_INVALID_ARG;
  if (T > (1 << 30)) return MLA_ERR_UNSUPPORTED;  // a warp's next row in 32 bits
  if (T == 0) return MLA_OK;
  if (!kv || !pos || !slot || !cache) return MLA_ERR_INVALID_ARG;
  const size_t e = esize(d);
  if (!aligned(kv, e) || !aligned(kv_gamma, e) || !aligned(cq, e) || !aligned(cq_gamma, e) || !aligned(cq_out, e) ||
      !aligned(pos, 4) || !aligned(slot, 8) || !aligned(cache, 16) || !aligned(device_error, 4))
    return MLA_ERR_INVALID_ARG;
  {
    // Other blocks still read their rows while this one writes: only a c_Q row
    // may be written over itself.
    const long long b = (long long)e;
    const RowSet rows(kv, T, kv_stride * b, 1, 0, d_cr * b), latent(cq, cq ? T : 0, cq_stride * b, 1, 0, d.d_cq * b),
        out(cq_out, cq ? T : 0, cq_out_stride * b, 1, 0, d.d_cq * b),
        pages(cache, (long long)num_pages * d.page_size * d_cr * b);
    const RowSet in[] = {rows, {kv_gamma, d.d_c * b}, {cq_gamma, d.d_cq * b}, {pos, 4LL * T}, {slot, 8LL * T}};
    for (const RowSet& x : in)
      if (rows_meet(x, pages) || rows_meet(x, out)) return MLA_ERR_INVALID_ARG;
    if (rows_meet(latent, pages) || rows_meet(out, pages) || (rows_meet(latent, out) && !same_rows(latent, out)))
      return MLA_ERR_INVALID_ARG;
  }
  step::NormAppendArgs a{};
  a.kv = kv; a.kv_gamma = kv_gamma; a.kv_stride = kv_stride;
  a.cq = cq; a.cq_gamma = cq_gamma; a.cq_stride = cq_stride;
  a.cq_out = cq_out; a.cq_out_stride = cq_out_stride;
  a.pos = pos; a.slot = slot; a.cache = cache; a.num_slots = (long long)num_pages * d.page_size;
  a.err = device_error;
  a.T = T; a.d_c = d.d_c; a.d_cr = d_cr; a.d_cq = cq ? d.d_cq : 0;
  a.eps = eps;
  a.rope = rope_table(d);
  // 16-byte accesses where every row and width allows them.
  const long long ve = 16 / (long long)e;
  bool vec = aligned(kv, 16) && aligned(kv_gamma, 16) && kv_stride % ve == 0 && d.d_c % ve == 0 && d_cr % ve == 0;
  if (cq)
    vec = vec && aligned(cq, 16) && aligned(cq_gamma, 16) && aligned(cq_out, 16) && cq_stride % ve == 0 &&
          cq_out_stride % ve == 0 && d.d_cq % ve == 0;
  g_launches = 1;
  return cuda_status(d.dtype == MLA_BF16 ? launch_norm_append<__nv_bfloat16>(a, vec, stream)
                                         : launch_norm_append<float>(a, vec, stream));
}

mla_status mla_query_norm_rope(const mla_dims* dims, const void* q, int64_t q_stride, const void* gamma, float eps,
                               const int32_t* pos, void* qc_out, int64_t qc_token_stride, int64_t qc_head_stride,
                               void* qr_out, int64_t qr_token_stride, int64_t qr_head_stride, int T,
                               cudaStream_t stream) {
  mla_status s = check_dims(dims);
  if (s != MLA_OK) return s;
  const mla_dims& d = *dims;
  if (T < 0 || !(eps >= 0.f) || q_stride < (long long)d.n_h * (d.d_h + d.d_r) || qc_head_stride < d.d_h ||
      qr_head_stride < d.d_r || qc_token_stride < (d.n_h - 1) * qc_head_stride + d.d_h ||
      qr_token_stride < (d.n_h - 1) * qr_head_stride + d.d_r)
    return MLA_ERR_INVALID_ARG;
  if (T == 0) return MLA_OK;
  if (!q || !pos || !qc_out || !qr_out) return MLA_ERR_INVALID_ARG;
  const size_t e = esize(d);
  if (!aligned(q, e) || !aligned(gamma, e) || !aligned(pos, 4) || !aligned(qc_out, e) || !aligned(qr_out, e))
    return MLA_ERR_INVALID_ARG;
  {
    // As in the append: a part of q may only be written over itself.
    const long long b = (long long)e, dq = (d.d_h + d.d_r) * b;
    const RowSet content(q, T, q_stride * b, d.n_h, dq, d.d_h * b),
        position(static_cast<const char*>(q) + d.d_h * b, T, q_stride * b, d.n_h, dq, d.d_r * b),
        qc(qc_out, T, qc_token_stride * b, d.n_h, qc_head_stride * b, d.d_h * b),
        qr(qr_out, T, qr_token_stride * b, d.n_h, qr_head_stride * b, d.d_r * b);
    const RowSet in[] = {{gamma, d.d_h * b}, {pos, 4LL * T}};
    for (const RowSet& x : in)
      if (rows_meet(x, qc) || rows_meet(x, qr)) return MLA_ERR_INVALID_ARG;
    if (rows_meet(qc, qr) || rows_meet(content, qr) || rows_meet(position, qc) ||
        (rows_meet(content, qc) && !same_rows(content, qc)) || (rows_meet(position, qr) && !same_rows(position, qr)))
      return MLA_ERR_INVALID_ARG;
  }
  const int ve = 16 / (int)e;
  const bool vec = aligned(q, 16) && aligned(gamma, 16) && aligned(qc_out, 16) && aligned(qr_out, 16) &&
                   d.d_h % ve == 0 && d.d_r % ve == 0 && q_stride % ve == 0 && qc_token_stride % ve == 0 &&
                   qc_head_stride % ve == 0 && qr_token_stride % ve == 0 && qr_head_stride % ve == 0;
  step::QueryArgs a{};
  a.q = q; a.gamma = gamma; a.qc = qc_out; a.qr = qr_out; a.pos = pos;
  a.q_stride = q_stride;
  a.qc_ts = qc_token_stride; a.qc_hs = qc_head_stride;
  a.qr_ts = qr_token_stride; a.qr_hs = qr_head_stride;
  a.T = T; a.n_h = d.n_h; a.d_h = d.d_h; a.d_r = d.d_r;
  a.eps = eps;
  a.rope = rope_table(d);
  g_launches = 1;
  return cuda_status(d.dtype == MLA_BF16 ? launch_query<__nv_bfloat16>(a, vec, stream)
                                         : launch_query<float>(a, vec, stream));
}

size_t mla_attend_ragged_workspace_bytes(const mla_dims* dims, int B, int T) {
  if (check_ragged(dims, B, T) != MLA_OK) return 0;
  return make_ragged_plan(*dims, B, T).total;
}

mla_status mla_attend_ragged(const mla_dims* dims, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                             const int32_t* q_start, const int32_t* kv_len, const int32_t* page_table, int max_pages,
                             int num_pages, const void* cache, void* out, float* lse, int B, int T, void* workspace,
                             size_t workspace_bytes, cudaStream_t stream) {
  mla_status s = check_ragged(dims, B, T);
  if (s != MLA_OK) return s;
  const mla_dims& d = *dims;
  if (max_pages <= 0 || num_pages <= 0 || num_pages > INT_MAX / 64 || max_pages > INT_MAX / 64 ||
      q_head_stride < d.d_c + d.d_r || q_token_stride < (d.n_h - 1) * q_head_stride + d.d_c + d.d_r)
    return MLA_ERR_INVALID_ARG;
  if (T == 0) return MLA_OK;
  if (!q || !q_start || !kv_len || !page_table || !cache || !out || !workspace) return MLA_ERR_INVALID_ARG;
  if (!aligned(workspace, 256) || !aligned(cache, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(q_start, 4) || !aligned(kv_len, 4) || !aligned(page_table, 4))
    return MLA_ERR_INVALID_ARG;
  // The tensor-core path reads query rows in 16-byte pieces.
  if (d.dtype == MLA_BF16 ? !aligned(q, 16) || q_token_stride % 8 || q_head_stride % 8 : !aligned(q, 4))
    return MLA_ERR_INVALID_ARG;
  const size_t e = esize(d);
  const size_t q_bytes = e * ((size_t)(T - 1) * q_token_stride + (size_t)(d.n_h - 1) * q_head_stride + d.d_c + d.d_r);
  if (overlap(q, q_bytes, out, e * (size_t)T * d.n_h * d.d_c)) return MLA_ERR_INVALID_ARG;
  const RaggedPlan P = make_ragged_plan(d, B, T);
  if (workspace_bytes < P.total) return MLA_ERR_WORKSPACE;
  g_launches = 0;
  return attend_ragged_impl(d, q, q_token_stride, q_head_stride, q_start, kv_len, page_table, B, T, max_pages, num_pages,
                            cache, out, lse, workspace, P, at<int>(workspace, P.hdr), false, stream);
}

size_t mla_ragged_step_workspace_bytes(const mla_dims* dims, int B, int T) {
  if (check_ragged(dims, B, T) != MLA_OK) return 0;
  return make_ragged_step_plan(*dims, B, T).total;
}

mla_status mla_ragged_step(const mla_weights* w, const void* h, const int32_t* q_start, const int32_t* kv_len,
                           const int32_t* seq_idx, const int32_t* pos, const int32_t* page_table, int max_pages,
                           int num_pages, void* cache, float* out, int B, int T, void* workspace,
                           size_t workspace_bytes, cudaStream_t stream) {
  if (!w) return MLA_ERR_INVALID_ARG;
  mla_status s = check_ragged(&w->d, B, T);
  if (s != MLA_OK) return s;
  if (max_pages <= 0 || num_pages <= 0 || num_pages > INT_MAX / 64 || max_pages > INT_MAX / 64)
    return MLA_ERR_INVALID_ARG;
  if (T == 0) return MLA_OK;
  if (!h || !q_start || !kv_len || !seq_idx || !pos || !page_table || !cache || !out || !workspace)
    return MLA_ERR_INVALID_ARG;
  if (!aligned(workspace, 256) || !aligned(h, 16) || !aligned(cache, 16) || !aligned(out, 16) ||
      !aligned(q_start, 4) || !aligned(kv_len, 4) || !aligned(seq_idx, 4) || !aligned(pos, 4) ||
      !aligned(page_table, 4))
    return MLA_ERR_INVALID_ARG;
  const RaggedStepPlan P = make_ragged_step_plan(w->d, B, T);
  if (workspace_bytes < P.total) return MLA_ERR_WORKSPACE;
  s = begin_call(workspace, stream, P.base);
  if (s != MLA_OK) return s;
  if (w->d.dtype == MLA_BF16)
    return ragged_step_impl<__nv_bfloat16>(w, h, q_start, kv_len, seq_idx, pos, page_table, B, T, max_pages, num_pages,
                                           cache, out, workspace, P, stream);
  return ragged_step_impl<float>(w, h, q_start, kv_len, seq_idx, pos, page_table, B, T, max_pages, num_pages, cache,
                                 out, workspace, P, stream);
}

}  // extern "C"
