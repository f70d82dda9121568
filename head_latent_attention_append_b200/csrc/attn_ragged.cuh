// Ragged absorbed attention on the sm_100a tensor cores: every request's new
// tokens over its paged latent cache.
//
// For 128 rows (row = token * n_h + head, all of one request; see
// ragged_sched.cuh) and every 64-key cache page
//   S = Q page^T,  P = exp2(scale log2e S - m),  O += P page[:, latent],
// as in attn_tc.cuh ("ai-decoupled-rope-mla", absorbed score and output
// equations), whose pipeline and operand layouts this kernel shares: a
// 2-CTA cluster issues cta_group::2 MMAs, each CTA owning 64 of the rows with
// their whole softmax state; the score ring, the latent ring, the TMEM and
// shared-memory maps and the barriers are the ones described there.  What
// differs:
//   - the 128 rows are a row block of a request, not the heads of one token, so
//     a 16-head model fills them with eight tokens, and any number of heads
//     works;
//   - each row has its own last key.  Only the pages behind the first row's
//     last key need a mask (at most 1 + ceil(d / 64) of a row block whose last
//     row sees d keys more than its first), and in those the latent rows are
//     cleared of what a weight of 0 must not meet: rows behind the block's last
//     key wholly, infinities and NaNs in rows that only some of the block's
//     rows see (a row that sees one has a NaN sum already, or a score of -inf
//     there and with it no weight);
//   - the softmax scale is applied to the scores in 32 bits (one FMA with the
//     running maximum), so the queries come as they are;
//   - a piece of a cut row block leaves its O in 32 bits, column by column, so
//     that a warp's store is one line without passing through shared memory,
//     and the merge adds no rounding.  P (bf16, as the MMA reads it) and the
//     output are the only roundings to fewer than 32 bits; the weights are
//     taken by the hardware's 2^x (2^-22 relative).  Against 64 bits the outputs
//     are off by 1.9e-3 to 2.1e-3 (2-norm), where rounding the exact output once
//     gives 1.7e-3.
//
// Bound by the tensor pipe's page loop (1480 cycles a page, 1244 of them MMAs)
// and, run back to back, by power: 862 tokens of 128 heads over up to 16,001
// keys take 2.47 ms, 1160 TFLOP/s, 0.84 of the sustained bf16 rate; a batch of
// 330 tokens over up to 4171 keys 271 us (234 in short runs, near full clock),
// 0.69 of it.  A change of query rows
// costs 12,000 cycles (the next rows' load, this block's output), which the
// schedule counts.  The page loop sits at the register limit: merging pieces
// here, calling its ends out of line or handing registers over made it 10 to 20%
// slower.
#pragma once
#include "attn_tc.cuh"
#include "ragged_sched.cuh"

namespace mla {
namespace ragged_tc {
using namespace sm100;
using attn_tc::CH_S;
using attn_tc::CH_V;
using attn_tc::cluster_rank;
using attn_tc::cluster_sync_all;
using attn_tc::desc_add;
using attn_tc::fast_exp2;
using attn_tc::KT;
using attn_tc::map_peer;
using attn_tc::MAX_NPV;
using attn_tc::MAX_TS;
using attn_tc::OFF_BAR;
using attn_tc::OFF_LS;
using attn_tc::OFF_MISC;
using attn_tc::OFF_MX;
using attn_tc::OFF_P;
using attn_tc::OFF_QS;
using attn_tc::OFF_SG;
using attn_tc::OFF_STG;
using attn_tc::OFF_VG;
using attn_tc::P_BYTES;
using attn_tc::pack_bf16x2;
using attn_tc::prefetch_l2;
using attn_tc::QS_BYTES;
using attn_tc::SG_BYTES;
using attn_tc::SGS;
using attn_tc::SMEM_BYTES;
using attn_tc::THREADS;
using attn_tc::TM_COLS;
using attn_tc::TM_O;
using attn_tc::TM_Q;
using attn_tc::TM_S;
using attn_tc::VG_BYTES;
using attn_tc::VGS;

constexpr int ROWS = 128;          // rows of a row block
constexpr int CROWS = ROWS / 2;    // rows per CTA
constexpr int kOwnMost = THREADS;  // requests and row blocks of a schedule that every CTA makes for itself
static_assert(sizeof(RaggedScratch<kOwnMost>) <= VGS * VG_BYTES, "the schedule's sums fit the latent ring");

struct Args {
  const __nv_bfloat16* q;      // row r of token t, head h: q + t * q_ts + h * q_hs, d_c + d_r values
  long long q_ts, q_hs;
  const int32_t* page_table;   // [B][max_pages]
  int max_pages, num_pages, n_h, d_c, q_row;
  float scale;                 // softmax scale times log2 e
  int q_dense;                 // the rows of q are contiguous
  RaggedSchedArgs sched;
  RaggedOut o;
};

// Walks a worker's segments page by page, the next page's id loaded one step
// ahead.
struct PageWalk {
  const RSeg* segs;
  const int32_t* page_table;
  int max_pages;
  int si, seg_hi, t;
  RSeg g, gn;
  bool more;
  int page_next;
  __device__ void start(int seg_lo, const RSeg& first) {
    si = seg_lo;
    more = si < seg_hi;
    if (!more) return;
    g = first;
    gn = si + 1 < seg_hi ? segs[si + 1] : g;
    t = g.t_lo;
    page_next = page_table[(long long)g.seq * max_pages + t];
  }
  __device__ int next(RSeg& cur, int& tile) {
    cur = g;
    tile = t;
    const int page = page_next;
    if (++t >= g.t_hi) {
      if (++si < seg_hi) {
        g = gn;
        if (si + 1 < seg_hi) gn = segs[si + 1];
        t = g.t_lo;
      } else {
        more = false;
      }
    }
    if (more) page_next = page_table[(long long)g.seq * max_pages + t];
    return page;
  }
};

// Pages whose latent rows the softmax threads touch before P*V reads them:
// the ones that reach past the first row's last key.
__device__ __forceinline__ bool edge_page(const RSeg& g, int t) { return (t + 1) * KT > g.kmin; }

template <int NPV>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    attn_ragged_kernel(const __grid_constant__ CUtensorMap mapS, const __grid_constant__ CUtensorMap mapV,
                       const Args a) {
  constexpr int NCH = 2 * NPV;                       // latent chunks of a row
  constexpr int NK = NCH + 1;                        // + the RoPE chunk
  constexpr int NTS = NK < MAX_TS ? NK : MAX_TS;     // chunks of Q in TMEM
  constexpr int NSS = NK - NTS;                      // chunks of Q in shared memory
  static_assert(NPV >= 1 && NPV <= MAX_NPV && NSS * CH_V <= QS_BYTES, "latent width");
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the same in every CTA: all leave before any barrier
    if (threadIdx.x == 0) a.sched.s.worker_err[blockIdx.x] = kErrLayout;
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint64_t* sg_full = bars;                // [SGS] both CTAs' score chunks landed (even CTA's)
  uint64_t* sg_empty = sg_full + SGS;      // [SGS] the page's score MMA is done (both CTAs)
  uint64_t* vg_full = sg_empty + SGS;      // [VGS] both CTAs' latent chunks landed (even CTA's)
  uint64_t* vg_empty = vg_full + VGS;      // [VGS] the page's P*V is done (both CTAs)
  uint64_t* vg_part = vg_empty + VGS;      // [VGS] this CTA's chunks of an edge page landed
  uint64_t* s_full = vg_part + VGS;        // [2] S of the page in buffer b is complete (both CTAs)
  uint64_t* p_ready = s_full + 2;          // [2] both CTAs' P of the page are in their P tiles (even CTA's)
  uint64_t* pv_done = p_ready + 2;         // [2] P*V of the page has completed (both CTAs)
  uint64_t* q_ready = pv_done + 2;         // a segment's Q rows are in place in both CTAs (even CTA's)
  uint64_t* o_free = q_ready + 1;          // both CTAs have read a segment's O (even CTA's)
  uint64_t* final_bar = o_free + 1;        // the MMA issuer's last commit
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC + 4);
  int* const err = reinterpret_cast<int*>(smem + OFF_MISC + 8);  // this CTA's error bits

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int w = blockIdx.x >> 1;

  if (tid == 32) {
    for (int i = 0; i < SGS; ++i) {
      mbar_init(&sg_full[i], 1);   // the even CTA's arrive.expect_tx + both CTAs' bytes
      mbar_init(&sg_empty[i], 1);  // commit of the score MMA
    }
    for (int i = 0; i < VGS; ++i) {
      mbar_init(&vg_full[i], 1);
      mbar_init(&vg_empty[i], 1);
      mbar_init(&vg_part[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_ready[i], 16);  // one arrive per softmax warp of both CTAs
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(q_ready, 16);
    mbar_init(o_free, 16);
    mbar_init(final_bar, 1);
    *abort_flag = 0;
    *err = 0;
    mbar_fence_init();
  }
  if (warp == 2) {
    tmem_alloc_pair(tmem_slot, TM_COLS);
    tmem_relinquish_pair();
  }
  if (tid == 0) {
    tma_prefetch_desc(&mapS);
    tma_prefetch_desc(&mapV);
  }
  __syncthreads();
  cluster_sync_all();  // the peer's barriers and TMEM exist before anyone signals them
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  // Everything above overlaps the kernel before this one.
  pdl_wait();
  pdl_trigger();
  const RSeg* segs = a.sched.s.segs;
  // The worker's segments pass through memory either way: handed over in
  // registers, they cost the page loop 2 to 4%.
  int2* const range = a.sched.s.range + (a.sched.own ? blockIdx.x : w);
  if (a.sched.own) {
    ragged_schedule<kOwnMost>(a.sched, *reinterpret_cast<RaggedScratch<kOwnMost>*>(smem + OFF_VG), w, range, err);
    fence_proxy_async_smem();  // the latent ring's copies land where the sums were
    __syncthreads();
  }
  const int seg_lo = range->x, seg_hi = range->y;

  if (warp == 0 || warp == 2) {
    // ---------------------------------------------------- TMA producers
    // Warp 0 fills the score ring (this CTA's 32 keys of every chunk), warp
    // 2 the latent ring (all 64 keys of this CTA's latent chunks); both
    // complete on the even CTA's barriers, except edge pages in the latent
    // ring, which land on a barrier of the CTA's own.
    const bool score_ring = warp == 0;
    const int nslots = score_ring ? SGS : VGS;
    uint64_t* full = score_ring ? sg_full : vg_full;
    uint64_t* empty = score_ring ? sg_empty : vg_empty;
    uint8_t* ring = smem + (score_ring ? OFF_SG : OFF_VG);
    const int slot_bytes = score_ring ? SG_BYTES : VG_BYTES;
    const uint32_t full_even = map_peer(smem_u32(full), 0);
    PageWalk pw{segs, a.page_table, a.max_pages, 0, seg_hi, 0, RSeg{}, RSeg{}, false, 0};
    pw.start(seg_lo, a.sched.s.first[w]);
    static_assert(VGS == 2, "two latent slots");
    uint32_t cnt = 0, part_cnt0 = 0, part_cnt1 = 0;  // edge loads per latent slot
    while (pw.more) {
      RSeg g;
      int t;
      int page = pw.next(g, t);
      const uint32_t s = cnt % nslots;
      if (!mbar_wait_warp(&empty[s], ((cnt / nslots) & 1) ^ 1, abort_flag, err)) break;
      if (page < 0 || page >= a.num_pages) {
        // A block that sees no key walks one page all the same, masked whole.
        if (g.nkeys > 0 && rank == 0 && score_ring && elect_one()) flag_error(err, kErrBounds);
        page = 0;
      }
      const bool edge = edge_page(g, t);
      uint8_t* dst = ring + s * slot_bytes;
      if (elect_one()) {
        if (score_ring) {
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * NK * CH_S);
          for (int c = 0; c < NK; ++c)
            tma_load_2d_pair(dst + c * CH_S, &mapS, 64 * c, page * KT + (int)rank * 32, full_even + 8 * s);
        } else if (!edge) {
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * NPV * CH_V);
          for (int q = 0; q < NPV; ++q)
            tma_load_2d_pair(dst + q * CH_V, &mapV, ((int)rank * NPV + q) * 64, page * KT, full_even + 8 * s);
        } else {
          mbar_arrive_expect_tx(&vg_part[s], NPV * CH_V);
          for (int q = 0; q < NPV; ++q)
            tma_load_2d(dst + q * CH_V, &mapV, ((int)rank * NPV + q) * 64, page * KT, &vg_part[s]);
          if (rank == 0) mbar_arrive(&full[s]);  // the phase still advances; p_ready covers the bytes
        }
      }
      __syncwarp();
      if (!score_ring && edge) {
        if (s == 0) ++part_cnt0;
        else ++part_cnt1;
      }
      ++cnt;
    }
    if (*abort_flag) {
      // Let every copy already issued land before the CTA can exit (the even
      // CTA's barriers count the odd CTA's bytes too).
      if (rank == 0)
        for (uint32_t q = 0; q < (uint32_t)nslots && q < cnt; ++q) {
          const uint32_t last = q + nslots * ((cnt - 1 - q) / nslots);
          mbar_wait_warp(&full[q], (last / nslots) & 1, abort_flag, nullptr, 50000000ull, false);
        }
      if (!score_ring)
        for (int q = 0; q < VGS; ++q) {
          const uint32_t n_q = q == 0 ? part_cnt0 : part_cnt1;
          if (n_q) mbar_wait_warp(&vg_part[q], (n_q - 1) & 1, abort_flag, nullptr, 50000000ull, false);
        }
    }
  } else if (warp == 1 && rank == 0) {
    // ------------------------------------------------------- MMA issuer
    const uint32_t tS = tbase + TM_S, tO = tbase + TM_O, tQ = tbase + TM_Q;
    const uint64_t dS0 = sdesc_sw128(smem_u32(smem + OFF_SG), 16, 1024);
    const uint64_t dQ0 = sdesc_sw128(smem_u32(smem + OFF_QS), 16, 1024);
    const uint64_t dP0 = sdesc_sw128(smem_u32(smem + OFF_P), 16, 1024);
    const uint64_t dV0 = sdesc_sw128(smem_u32(smem + OFF_VG), CH_V, 1024);  // MN-major: LBO = chunk stride
    const uint32_t idS = idesc_bf16(128, 64, 0, 0);
    const uint32_t idV2 = idesc_bf16(128, 256, 0, 1), idV1 = idesc_bf16(128, 128, 0, 1);
    bool ok = true;
    // P*V of page pj: waits for both CTAs' P (and, at a segment's first page,
    // for both CTAs to have read the previous segment's O).
    auto issue_pv = [&](uint32_t pj, bool first, uint32_t sk) -> bool {
      const uint32_t vs = pj % VGS;
      bool r_ok = mbar_wait(&vg_full[vs], (pj / VGS) & 1, abort_flag, err);
      if (r_ok && first && sk > 0) r_ok = mbar_wait(o_free, (sk - 1) & 1, abort_flag, err);
      if (r_ok) r_ok = mbar_wait(&p_ready[pj & 1], (pj >> 1) & 1, abort_flag, err);
      if (!__all_sync(0xffffffffu, r_ok)) return false;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t a0 = desc_add(dP0, (pj & 1) * P_BYTES);
        const uint64_t b0 = desc_add(dV0, vs * VG_BYTES);
#pragma unroll
        for (int k = 0; k < KT / 16; ++k) {
#pragma unroll
          for (int m = 0; m < (NPV + 1) / 2; ++m)
            mma_pair_ss(tO + m * 128, desc_add(a0, k * 32), desc_add(b0, m * 2 * CH_V + k * 2048),
                        (2 * m + 1 < NPV) ? idV2 : idV1, (first && k == 0) ? 0u : 1u);
        }
        tc_commit_pair(&pv_done[pj & 1], 3);
        tc_commit_pair(&vg_empty[vs], 3);
      }
      __syncwarp();
      return true;
    };
    uint32_t j = 0, seg_k = 0, prev_j = 0, prev_sk = 0;
    bool have_prev = false, prev_first = false;
    for (int si = seg_lo; si < seg_hi && ok; ++si, ++seg_k) {
      const int n = segs[si].t_hi - segs[si].t_lo;
      for (int i = 0; i < n; ++i, ++j) {
        if (i == 0) {
          // The previous segment's last P*V first, then this segment's Q.
          if (have_prev && !(ok = issue_pv(prev_j, prev_first, prev_sk))) break;
          have_prev = false;
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(q_ready, seg_k & 1, abort_flag, err)))) break;
        }
        const uint32_t gs = j % SGS;
        if (!(ok = mbar_wait_warp(&sg_full[gs], (j / SGS) & 1, abort_flag, err))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t d = tS + (j & 1) * 32;
          const uint64_t b0 = desc_add(dS0, gs * SG_BYTES);
#pragma unroll
          for (int c = 0; c < NK; ++c) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint64_t b = desc_add(b0, c * CH_S + k * 32);
              if (c < NTS)
                mma_pair_ts(d, tQ + c * 32 + k * 8, b, idS, (c | k) ? 1u : 0u);
              else
                mma_pair_ss(d, desc_add(dQ0, (c - NTS) * CH_V + k * 32), b, idS, (c | k) ? 1u : 0u);
            }
          }
          tc_commit_pair(&s_full[j & 1], 3);
          tc_commit_pair(&sg_empty[gs], 3);
        }
        __syncwarp();
        if (have_prev && !(ok = issue_pv(prev_j, prev_first, prev_sk))) break;
        have_prev = true;
        prev_j = j;
        prev_first = i == 0;
        prev_sk = seg_k;
      }
    }
    if (ok && have_prev) issue_pv(prev_j, prev_first, prev_sk);
    if (elect_one()) tc_commit_pair(final_bar, 1);
    __syncwarp();
    mbar_wait_warp(final_bar, 0, abort_flag, nullptr, 50000000ull, false);
  } else if (warp >= 4) {
    // ---------------------------------------------------------- softmax
    // Thread (lane quarter q4, column half ch) owns TMEM lane L = 32 q4 + lane:
    // row L mod 64 of this CTA, keys [32 (L div 64) + 16 ch, +16) of a page
    // and O columns [(L div 64) d_c/2 + ch d_c/4, +d_c/4).
    const int q4 = warp & 3, ch = (warp - 4) >> 2, grp = warp & 1;
    const int L = q4 * 32 + lane, hl = L & 63, kh = L >> 6, part = kh * 2 + ch;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t tS = tbase + lane_off + TM_S, tO = tbase + lane_off + TM_O, tQ = tbase + lane_off + TM_Q;
    const int crow0 = (int)rank * CROWS, my_row = crow0 + hl;
    float* mx = reinterpret_cast<float*>(smem + OFF_MX);    // [2][64][4]
    float* lsum = reinterpret_cast<float*>(smem + OFF_LS);  // [64][4]
    const uint32_t p_ready_even = map_peer(smem_u32(p_ready), 0);
    const uint32_t q_ready_even = map_peer(smem_u32(q_ready), 0);
    const uint32_t o_free_even = map_peer(smem_u32(o_free), 0);
    // A failed wait clears `ok` (warp-uniform) and the rest of the work is
    // skipped, but every thread still walks every page and every Q load so
    // that the named barriers always see all of their threads.
    bool ok = true;
    auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
      bool r_ok = mbar_wait(bar, parity, abort_flag, err);
      return __all_sync(0xffffffffu, r_ok);
    };
    auto signal_even = [&](uint32_t bar_even) {
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(bar_even);
    };
    // A segment's Q rows: q_issue() issues every global load into registers
    // before any store (thread tau takes 16-byte pieces tau and tau + 256 of
    // each 64-row x 128-byte chunk, eight threads per row segment); q_store()
    // writes chunks [0, NTS) into TMEM (lane L holds row L mod 64) and the rest
    // into shared memory.  Rows past the block's are zeros.
    uint4 pv[NK][2];
    auto q_issue = [&](const RSeg& g) {
      const int tau = tid - 128;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int pc = tau + 256 * h, r = crow0 + (pc >> 3), row = g.row0 + r, tok = row / a.n_h;
        const bool live = ok && r < g.nrows;
        const __nv_bfloat16* src = a.q + tok * a.q_ts + (row - tok * a.n_h) * a.q_hs + 8 * (pc & 7);
#pragma unroll
        for (int c = 0; c < NK; ++c)
          pv[c][h] = live && 64 * c + 8 * (pc & 7) < a.q_row ? __ldg(reinterpret_cast<const uint4*>(src + 64 * c))
                                                             : make_uint4(0, 0, 0, 0);
      }
    };
    auto q_store = [&]() {
      const int tau = tid - 128;
      // Chunks [NTS, NK) go straight to their shared-memory tiles.
#pragma unroll
      for (int s2 = 0; s2 < NSS; ++s2)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int pc = tau + 256 * h, r = pc >> 3, u = pc & 7;
          *reinterpret_cast<uint4*>(smem + OFF_QS + s2 * CH_V + r * 128 + ((u ^ (r & 7)) << 4)) = pv[NTS + s2][h];
        }
      // Chunks [0, NTS) pass through the staging tile, one at a time: thread
      // (L, ch) then stores columns [16 ch, 16 ch + 16) of the chunk for
      // TMEM lane L (both lane halves hold row L mod 64).
#pragma unroll
      for (int c = 0; c < NTS; ++c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int pc = tau + 256 * h, r = pc >> 3, u = pc & 7;
          *reinterpret_cast<uint4*>(smem + OFF_STG + r * 128 + ((u ^ (r & 7)) << 4)) = pv[c][h];
        }
        named_bar_sync(3, 256);
        uint32_t wv[16];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const uint4 x = *reinterpret_cast<const uint4*>(smem + OFF_STG + hl * 128 + (((4 * ch + v) ^ (hl & 7)) << 4));
          wv[4 * v + 0] = x.x;
          wv[4 * v + 1] = x.y;
          wv[4 * v + 2] = x.z;
          wv[4 * v + 3] = x.w;
        }
        if (ok) tmem_st16(tQ + 32 * c + 16 * ch, wv);
        named_bar_sync(3, 256);
      }
      if (ok) {
        fence_proxy_async_smem();  // the MMA (async proxy) reads what the threads wrote
        tmem_st_wait();
        tc_fence_before();
        signal_even(q_ready_even);
      }
    };
    // The next segment's Q rows are pulled into L2 a few pages before they
    // are loaded (an earlier prefetch would be evicted by the page stream).
    auto prefetch_q = [&](const RSeg& g) {
      if (tid == 128 && a.q_dense) {
        const int r0 = crow0, r1 = min(g.nrows, crow0 + CROWS);
        if (r1 > r0) prefetch_l2(a.q + ((long long)g.row0 + r0) * a.q_row, (uint32_t)((r1 - r0) * a.q_row * 2));
      }
    };

    uint32_t j = 0, part_par = 0;  // bit s: parity of the next edge load in latent slot s
    // The page loop keeps four numbers of its segment; the rest is read again at
    // its ends (three segments in registers were 4% slower, a ring of them in
    // shared memory 2%).
    if (seg_lo < seg_hi) {  // every softmax thread: q_store holds named barriers
      q_issue(a.sched.s.first[w]);
      q_store();
    }
    for (int si = seg_lo; si < seg_hi; ++si) {
      int t_lo, n, kmin, lim;
      {
        const RSeg g = segs[si];
        t_lo = g.t_lo;
        n = g.t_hi - g.t_lo;
        kmin = g.kmin;
        // Keys that this thread's row sees (none for a row past the block's).
        lim = my_row < g.nrows ? min(max(g.base + (g.row0 + my_row) / a.n_h + 1, 0), g.nkeys) : 0;
      }
      float m_used = -INFINITY, lt = 0.f;  // in base 2; O and the sums are relative to ref_max(m_used)
      for (int i = 0; i < n; ++i, ++j) {
        const int t = t_lo + i;
        const uint32_t b = j & 1;
        const bool edge = (t + 1) * KT > kmin;  // edge_page
        if (si + 1 < seg_hi && i == max(0, n - 6)) prefetch_q(segs[si + 1]);
        // S of page j is complete, and with it every earlier MMA: P*V of page
        // j - 2 (issued before S(j)) has released P tile b.
        ok = ok && wait_all(&s_full[b], (j >> 1) & 1);
        float s[16];
        if (ok) {
          tc_fence_after();
          uint32_t v[16];
          tmem_ld16(tS + b * 32 + ch * 16, v);
          tmem_ld_wait();
#pragma unroll
          for (int x = 0; x < 16; ++x) s[x] = __uint_as_float(v[x]);
        } else {
#pragma unroll
          for (int x = 0; x < 16; ++x) s[x] = 0.f;
        }
        const int k0 = kh * 32 + ch * 16;  // this thread's first key of the page
        if (edge) {
          const int rel = lim - t * KT - k0;
#pragma unroll
          for (int x = 0; x < 16; ++x)
            if (x >= rel) s[x] = -INFINITY;
        }
        float mt;
        {
          float m8[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) m8[x] = fmaxf(s[x], s[x + 8]);
#pragma unroll
          for (int w2 = 4; w2 >= 1; w2 >>= 1)
#pragma unroll
            for (int x = 0; x < w2; ++x) m8[x] = fmaxf(m8[x], m8[x + w2]);
          mx[(b * CROWS + hl) * 4 + part] = m8[0];
          named_bar_sync(1 + grp, 128);
          const float4 m4 = reinterpret_cast<const float4*>(mx)[b * CROWS + hl];
          mt = a.scale * fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w));
        }
        // Running max with lazy rescaling: O and the sums stay relative to
        // m_used until a page's max exceeds it by more than 2^8.  The four
        // threads of a row take the same decision from the same numbers.
        bool resc = false;
        float scale = 1.f;
        if (i == 0) {
          m_used = mt;
        } else if (mt > m_used + 8.f) {
          scale = fast_exp2(m_used - mt);
          m_used = mt;
          resc = true;
        }
        const float ref = ref_max(m_used);
        uint32_t pk[8];
        {
          float ps[4] = {0.f, 0.f, 0.f, 0.f};
          // The row sum adds the fp32 weights (not their bf16 roundings: the
          // difference is random, 2^-9 relative per key).
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const float e0 = fast_exp2(fmaf(s[2 * u], a.scale, -ref)), e1 = fast_exp2(fmaf(s[2 * u + 1], a.scale, -ref));
            ps[u & 3] += e0 + e1;
            pk[u] = pack_bf16x2(e0, e1);
          }
          lt = lt * scale + ((ps[0] + ps[1]) + (ps[2] + ps[3]));
        }
        // O is rescaled only after P*V of page j - 1 has completed.
        if (ok && __any_sync(0xffffffffu, resc)) {
          ok = wait_all(&pv_done[b ^ 1], ((j - 1) >> 1) & 1);
          if (ok) {
            tc_fence_after();
#pragma unroll
            for (int cc = 0; cc < NPV; ++cc) {
              uint32_t v[32];
              tmem_ld32(tO + ch * (NPV * 32) + cc * 32, v);
              tmem_ld_wait();
#pragma unroll
              for (int x = 0; x < 32; ++x) v[x] = __float_as_uint(__uint_as_float(v[x]) * scale);
              tmem_st32(tO + ch * (NPV * 32) + cc * 32, v);
            }
            tmem_st_wait();
          }
        }
        // P row hl, keys k0 .. k0 + 15: 16-byte pieces k0/8 and k0/8 + 1 of
        // the 128-byte-swizzled K-major tile.
        if (ok) {
          uint8_t* prow = smem + OFF_P + b * P_BYTES + hl * 128;
          const int u0 = k0 >> 3;
          *reinterpret_cast<uint4*>(prow + ((u0 ^ (hl & 7)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          *reinterpret_cast<uint4*>(prow + (((u0 + 1) ^ (hl & 7)) << 4)) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
        }
        if (ok && edge) {
          // 0 * NaN would poison O: rows behind the block's last key are
          // cleared, and in rows that only some of the block's rows see the
          // infinities and NaNs are (see the head of this file).
          const uint32_t vs = j % VGS;
          ok = wait_all(&vg_part[vs], (part_par >> vs) & 1);
          part_par ^= 1u << vs;
          if (ok) {
            uint8_t* vb = smem + OFF_VG + vs * VG_BYTES;
            const int first = max(0, kmin - t * KT), gone = min(KT, max(0, segs[si].nkeys - t * KT));
            const int rows = KT - first, units = rows * 8 * NPV;
            for (int x = tid - 128; x < units; x += 256) {
              const int qq = x / (rows * 8), rem = x - qq * rows * 8, r = first + rem / 8;
              uint4* const p = reinterpret_cast<uint4*>(vb + qq * CH_V + r * 128 + (rem % 8) * 16);
              if (r >= gone) {
                *p = make_uint4(0, 0, 0, 0);
              } else {
                uint4 v = *p;
                auto clean = [](uint32_t u) {  // zero where the exponent is all ones
                  if ((u & 0x7f80u) == 0x7f80u) u &= 0xffff0000u;
                  if ((u & 0x7f800000u) == 0x7f800000u) u &= 0xffffu;
                  return u;
                };
                const uint4 c = make_uint4(clean(v.x), clean(v.y), clean(v.z), clean(v.w));
                if (c.x != v.x || c.y != v.y || c.z != v.z || c.w != v.w) *p = c;
              }
            }
          }
        }
        if (ok) {
          fence_proxy_async_smem();  // the MMA (async proxy) reads P and the cleared rows
          tc_fence_before();
          signal_even(p_ready_even + 8 * b);
        }
        if (i + 1 < n) continue;

        // ---- end of the segment ----
        // The next segment's Q replaces this one's (its last score MMA is
        // complete); then O of this segment, once its last P*V is done.
        if (si + 1 < seg_hi) {  // every softmax thread: q_store holds named barriers
          q_issue(segs[si + 1]);
          q_store();
        }
        const RSeg g = segs[si];
        ok = ok && wait_all(&pv_done[b], (j >> 1) & 1);
        lsum[hl * 4 + part] = lt;
        named_bar_sync(1 + grp, 128);
        if (ok) tc_fence_after();
        const float4 l4 = reinterpret_cast<const float4*>(lsum)[hl];
        const float lrow = (l4.x + l4.y) + (l4.z + l4.w);
        const float inv = row_inv(lrow);
        if (g.slot >= 0) {
          // A piece of a cut row block: O / l in 32 bits, columns outermost,
          // straight from the registers (a warp's 32 rows are one line).
          const bool live = ok && my_row < g.nrows;
          float* const dst =
              a.o.part_o + ((long long)g.slot * a.d_c + kh * (a.d_c / 2) + ch * (NPV * 32)) * ROWS + my_row;
          if (live && part == 0) a.o.part_ml[(long long)g.slot * ROWS + my_row] = make_float2(m_used, lrow);
#pragma unroll 1
          for (int cc = 0; cc < NPV; ++cc) {
            uint32_t v[32];
            if (ok) {
              tmem_ld32(tO + ch * (NPV * 32) + cc * 32, v);
              tmem_ld_wait();
            }
            if (live) {
#pragma unroll
              for (int x = 0; x < 32; ++x) __stcg(dst + (cc * 32 + x) * ROWS, __uint_as_float(v[x]) * inv);
            }
          }
        } else {
          // A whole row block: normalised, rounded, and out through shared
          // memory (the P tiles and the staging tile, free now) so that the
          // global stores are coalesced: in round rho the threads with
          // part == rho write their d_c/4 columns of O into padded rows, then
          // all softmax threads store the 64 rows x d_c/4 columns.
          constexpr int PPR = 4 * NPV;          // 16-byte pieces per staged row
          constexpr int SROW = 16 * PPR + 16;   // padded row: consecutive rows start in different banks
          static_assert(CROWS * SROW <= 2 * P_BYTES + CH_V, "staged output fits the P and staging tiles");
          uint8_t* const so = smem + OFF_P;
          __nv_bfloat16* const obase = static_cast<__nv_bfloat16*>(a.o.out) + ((long long)g.row0 + crow0) * a.d_c;
          if (ok && part == 0 && my_row < g.nrows && a.o.lse)
            a.o.lse[(long long)g.row0 + my_row] = row_lse(ref_max(m_used), lrow);
#pragma unroll 1
          for (int rho = 0; rho < 4; ++rho) {
            if (ok && part == rho) {
#pragma unroll
              for (int cc = 0; cc < NPV; ++cc) {
                uint32_t v[32];
                tmem_ld32(tO + ch * (NPV * 32) + cc * 32, v);
                tmem_ld_wait();
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  uint4 o;
                  o.x = pack_bf16x2(__uint_as_float(v[8 * q + 0]) * inv, __uint_as_float(v[8 * q + 1]) * inv);
                  o.y = pack_bf16x2(__uint_as_float(v[8 * q + 2]) * inv, __uint_as_float(v[8 * q + 3]) * inv);
                  o.z = pack_bf16x2(__uint_as_float(v[8 * q + 4]) * inv, __uint_as_float(v[8 * q + 5]) * inv);
                  o.w = pack_bf16x2(__uint_as_float(v[8 * q + 6]) * inv, __uint_as_float(v[8 * q + 7]) * inv);
                  *reinterpret_cast<uint4*>(so + hl * SROW + (4 * cc + q) * 16) = o;
                }
              }
            }
            named_bar_sync(3, 256);
#pragma unroll
            for (int m = 0; m < NPV; ++m) {
              const int pc = (tid - 128) + 256 * m, r = pc / PPR, pp = pc - r * PPR;
              if (ok && crow0 + r < g.nrows)
                *reinterpret_cast<uint4*>(obase + (long long)r * a.d_c + rho * (NPV * 32) + 8 * pp) =
                    *reinterpret_cast<const uint4*>(so + r * SROW + 16 * pp);
            }
            named_bar_sync(3, 256);
          }
        }
        if (ok) {
          tc_fence_before();
          signal_even(o_free_even);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no CTA leaves while its peer may still use its shared memory or TMEM
  if (tid == 0) a.sched.s.worker_err[blockIdx.x] = *err;
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tbase, TM_COLS);
  }
}

}  // namespace ragged_tc
}  // namespace mla
