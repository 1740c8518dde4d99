// fa_paged_chunk_sm100.cuh -- paged attention of many new tokens (prompt chunks, alone or mixed
// with decoding steps), bf16: 256 rows (tokens x query heads of a group) per tile on tcgen05.
//
// Bound by the tensor cores and the exponentials, so the tile loop is the dense forward's
// (fa_fwd_sm100.cuh): two Q tiles of 128 rows, S and O in TMEM, P handed to the MMA warp through
// TMEM, K and V through separate TMA rings, one softmax thread per row.  What differs:
//   * The CTA is persistent: its share of the batch's line of key tiles (fa_paged.cuh) is a
//     sequence of pieces, and the roles run through all of them without meeting.  The MMA warp
//     starts the next piece's scores while the softmax warpgroups still write out the last one.
//   * Rows are tokens x heads of a group: one TMA box [tokens][G heads][64 columns] of the packed
//     queries is already the tile, so a K/V tile is read once for the whole group.  A piece of
//     few tokens (a decoding step in a mixed batch) takes a smaller box and one Q tile.
//   * A K/V tile of BN keys is one TMA box per page and 64 columns.  Pages that the table does not
//     name, or behind the last key, are read as an out-of-range page: zeros, without a read.
//   * Rows of the last page behind the last key may hold anything, and 0 * NaN is not 0: the
//     softmax warpgroups clear those V rows in shared memory before they hand over P.
// Key tiles: 128 keys at d = 128 (one CTA per SM), 64 at d = 64 (two CTAs per SM), as the forward.
// P is rounded to bf16 for P V, the type that the MMA takes beside a bf16 V (its row sum is taken
// before, in fp32); scores, statistics and sums are fp32.
// Measured: 2048 tokens over 32768 keys, 16 heads over 4: 440 us at d = 128 (1210 TFLOP/s; 470 to 530
// where the power limit holds the clock down), 392 at d = 64 (680); 8192 tokens of a causal prompt, d = 128: 265-280 us, where the dense forward of the
// same box takes 242-258.  The d = 64 tile is bound by the exponentials (62 % of the MUFU's issue
// slots) and their chain, as there; page sizes 16 to 256 measure alike.
#pragma once
#include "fa_paged.cuh"
#include "fa_paged_decode_sm100.cuh"

namespace fa {

enum : int {
  SITE_PCH_LOAD_EMPTY = 50, SITE_PCH_LOAD_DRAIN = 51, SITE_PCH_MMA_Q = 52, SITE_PCH_MMA_K = 53,
  SITE_PCH_MMA_V = 54, SITE_PCH_MMA_P = 55, SITE_PCH_MMA_FIN = 56, SITE_PCH_SM_S = 57,
  SITE_PCH_SM_O = 58, SITE_PCH_SM_V = 59
};

// One 32-byte sector per lane (the address 32-byte aligned): a warp whose lanes write a row each
// takes half as many store instructions as with 16-byte stores.
__device__ __forceinline__ void st_global_256(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d,
                                              uint32_t e, uint32_t f, uint32_t g, uint32_t h) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a), "r"(b), "r"(c),
               "r"(d), "r"(e), "r"(f), "r"(g), "r"(h)
               : "memory");
}

template <int D>
struct PagedChunkLayout {
  static constexpr int R = 256;
  static constexpr int BN = D == 64 ? 64 : 128;     // keys per tile
  static constexpr int C = 3;                       // an item's constant, in key tiles
  // key tiles that are worth a CTA: 128 tokens over 2048 keys, 16 heads over 4, d = 64 (128): 27 (23) us
  // with 1, 22 (26) with 4, 29 (36) with 8
  static constexpr int LEAST = BN == 64 ? 4 : 1;
  static constexpr int CTAS_PER_SM = BN == 64 ? 2 : 1;
  static constexpr int THREADS = 320;
  static constexpr int KST = BN == 64 ? 4 : 3;      // K ring depth
  static constexpr int VST = BN == 64 ? 4 : 2;      // V ring depth
  static constexpr int SUB = D / 64;                // 64-column (128-byte) sub-tiles
  static constexpr int Q_SUB = 256 * 128;           // bytes of 256 Q rows x 64 columns
  static constexpr int KV_SUB = BN * 128;
  static constexpr int KV_TILE = BN * D * 2;
  static constexpr int INFO = 8;                    // ring of per-tile page marks (see s_info)
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + SUB * Q_SUB;
  static constexpr int OFF_V = OFF_K + KST * KV_TILE;
  static constexpr int OFF_BAR = OFF_V + VST * KV_TILE;
  // q_full, q_empty, k_full[KST], k_empty[KST], v_full[VST], v_empty[VST], s_full[2], p_full[2],
  // o_done[2], p2_full[2], fin
  static constexpr int NBAR = 2 + 2 * KST + 2 * VST + 8 + 1;
  static constexpr int OFF_INFO = OFF_BAR + NBAR * 8;
  static constexpr int OFF_MISC = OFF_INFO + INFO * 4;
  static constexpr int OFF_SCHED = (OFF_MISC + 8 + 15) / 16 * 16;
  static constexpr int BYTES = OFF_SCHED + static_cast<int>(sizeof(PagedSched));
  static constexpr int SMEM_ALLOC = BYTES + 1024;   // slack for 1024-byte alignment
  static_assert(SMEM_ALLOC <= 232448 && CTAS_PER_SM * (SMEM_ALLOC + 1024) <= 233472, "shared memory");
  static constexpr bool SPLIT_P = BN == 128;        // P in two key halves, as the forward
  static constexpr uint32_t TMEM_COLS = 2 * BN + 2 * D <= 256 ? 256 : 512;
  static constexpr uint32_t O_COL0 = 2 * BN;
  static_assert(O_COL0 + 2 * D <= TMEM_COLS, "TMEM budget");
  // the load warp can be this many tiles ahead of a softmax warpgroup at most: P of tile t must
  // have been handed over before the scores of tile t + 2 can be issued
  static_assert(KST + 2 < INFO, "page marks are read before they are rewritten");
  __device__ static constexpr uint32_t s_col(int w) { return static_cast<uint32_t>(w) * BN; }
};

// What the roles need to know of a piece: key tiles [a, b) are in it, of which those below n0 (n1)
// hold a key that a row of Q tile 0 (1) may see.  Tiles from max(n0, n1) on (only the one tile of
// an item without keys) are passed over by all roles.
struct PagedChunkPiece {
  int rec, h, a, b;
  int n0, n1;
};

template <int BN>
__device__ __forceinline__ PagedChunkPiece paged_chunk_piece(const PagedParams& p, const PagedSched& s,
                                                             const PagedPiece& pc) {
  const PagedRec& rc = s.rec[pc.rec];
  PagedChunkPiece c = {pc.rec, pc.h, pc.a, pc.b, 0, 0};
  const int keys = paged_keys(p.causal, rc.kv, rc.pos0, rc.ntok);
  if (rc.ntok * p.G > 128) {
    c.n0 = (paged_keys(p.causal, rc.kv, rc.pos0, 127 / p.G + 1) + BN - 1) / BN;
    c.n1 = (keys + BN - 1) / BN;
  } else {
    c.n0 = (keys + BN - 1) / BN;
  }
  return c;
}

// Scores of the marked 16-key groups become -inf, in TMEM and before they are read, so that the
// rare case costs the loop one test (masking them in registers cost it 4 %).  The whole warp.
template <int BN>
__device__ __forceinline__ void paged_hide(uint32_t t_s, int marks) {
  uint32_t hidden[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) hidden[i] = __float_as_uint(-INFINITY);
  for (int g = 0; g < BN / 16; ++g)
    if ((marks >> g) & 1) tmem_st16(t_s + 16 * g, hidden);
  tmem_st_wait();
}

template <int D>
__global__ void __launch_bounds__(320, PagedChunkLayout<D>::CTAS_PER_SM)
fa_paged_chunk_sm100_kernel(const __grid_constant__ CUtensorMap tm_q,
                            const __grid_constant__ CUtensorMap tm_q_few,
                            const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const int few_tokens,
                            const PagedParams p) {
  using L = PagedChunkLayout<D>;
  constexpr int BN = L::BN, C = L::C;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bar_qf = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* bar_qe = bar_qf + 1;
  uint64_t* bar_kf = bar_qe + 1;
  uint64_t* bar_ke = bar_kf + L::KST;
  uint64_t* bar_vf = bar_ke + L::KST;
  uint64_t* bar_ve = bar_vf + L::VST;
  uint64_t* bar_sf = bar_ve + L::VST;
  uint64_t* bar_pf = bar_sf + 2;
  uint64_t* bar_od = bar_pf + 2;
  uint64_t* bar_p2 = bar_od + 2;
  uint64_t* bar_fin = bar_p2 + 2;
  // bits of 16-key groups of a tile whose page the table does not name; written before the tile's
  // K is awaited, read once its scores are there
  volatile int* s_info = reinterpret_cast<volatile int*>(smem + L::OFF_INFO);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  PagedSched& sched = *reinterpret_cast<PagedSched*>(smem + L::OFF_SCHED);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tpt = L::R / p.G;  // tokens per tile; G <= 256

  grid_dep_wait();  // launched to overlap the kernel before
  grid_dep_launch();
  const int cta = blockIdx.x;
  long long x, hi;
  PagedMine mine = {};
  if (!paged_share<BN, C, 320, L::LEAST>(p, tpt, sched, x, hi, mine)) return;
  if (threadIdx.x == 0) {
    mbar_init(bar_qf, 1);
    mbar_init(bar_qe, 1);
    for (int s = 0; s < L::KST; ++s) {
      mbar_init(&bar_kf[s], 1);
      mbar_init(&bar_ke[s], 1);
    }
    for (int s = 0; s < L::VST; ++s) {
      mbar_init(&bar_vf[s], 1);
      mbar_init(&bar_ve[s], 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&bar_sf[w], 1);
      mbar_init(&bar_pf[w], 128);
      mbar_init(&bar_p2[w], 128);
      mbar_init(&bar_od[w], 1);
    }
    mbar_init(bar_fin, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, L::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  bool ok = true;
  // running counts of each role: key tiles and pieces with keys (every role), S / PV per Q tile
  int it = 0, qn = 0, cnt0 = 0, cnt1 = 0;
  // MMA warp: the tile whose P V is still to be issued (0 flags: none)
  int prev_flags = 0, prev_vs = 0, prev_it = 0, prev_acc = 0;

  while (x < hi) {
    // (not the first list from `mine`: the loop then keeps more registers, 2.5 % at d = 128)
    paged_list<BN, C, 320>(p, tpt, x, hi, nullptr, sched);
    const long long stop = sched.stop;
    PagedPieces<C> pieces;
    pieces.start(p, sched, x);
    PagedPiece pc;
    if (warp == 8) {
      // ------------------------------------------------------------------ TMA producer
      // every lane keeps its page of a tile; the boxes of a tile are issued by one lane each
      const int box = min(1 << p.page_shift, BN);  // rows of a page in a tile
      const int np = BN / box;
      const int part = lane / (np * L::SUB);       // 0: K or V by turns, more: idle
      const int pg = lane / L::SUB % np, sub = lane % L::SUB;
      while (ok && pieces.next(p, sched, pc)) {
        const PagedChunkPiece c = paged_chunk_piece<BN>(p, sched, pc);
        const PagedRec rc = sched.rec[c.rec];
        bool first = true;
        const int32_t* table = p.table + rc.b * p.table_stride;
        const int keys = paged_keys(p.causal, rc.kv, rc.pos0, rc.ntok);
        const int h = c.h / p.splits, q0 = h * p.group + (c.h - h * p.splits) * p.G;
        auto page_id = [&](int j) -> int {
          const int k = j * BN + pg * box;
          return k < keys ? table[k >> p.page_shift] : -1;
        };
        int id = page_id(c.a);
        const int j_end = min(c.b, max(c.n0, c.n1));
        for (int j = c.a; j < j_end; ++j) {
          const int id_now = id;
          if (j + 1 < j_end) id = page_id(j + 1);
          const bool there = id_now >= 0 && id_now < p.num_pages;
          const bool behind = j * BN + pg * box >= keys;
          // groups of 16 keys whose page the table does not name
          const bool bad16 = __shfl_sync(0xffffffffu, !there && !behind, (16 * (lane & 7) / box % np) * L::SUB);
          const unsigned bad = __ballot_sync(0xffffffffu, lane < BN / 16 && bad16);
          const int row = (j * BN) & ((1 << p.page_shift) - 1);
          const int page = there ? id_now : p.num_pages;
          const int ks = it % L::KST, vs = it % L::VST;
          if (it >= L::KST)
            ok = __all_sync(0xffffffffu, mbar_wait(&bar_ke[ks], ((it / L::KST) - 1) & 1, abort_flag, SITE_PCH_LOAD_EMPTY));
          if (!ok) break;
          if (lane == 0) {
            s_info[it % L::INFO] = static_cast<int>(bad);
            mbar_arrive_expect_tx(&bar_kf[ks], L::KV_TILE);
          }
          __syncwarp();
          if (part == 0)
            tma_load_4d(smem + L::OFF_K + ks * L::KV_TILE + sub * L::KV_SUB + pg * box * 128, &tm_k,
                        &bar_kf[ks], sub * 64, row, h, page);
          // the piece's Q, once every S of the piece before has read its own
          if (first && ok) {
            first = false;
            if (qn > 0)
              ok = __all_sync(0xffffffffu, mbar_wait(bar_qe, (qn - 1) & 1, abort_flag, SITE_PCH_LOAD_EMPTY));
            if (ok) {
              if (lane == 0) {
                const bool few = rc.ntok <= few_tokens;
                mbar_arrive_expect_tx(bar_qf, L::SUB * (few ? few_tokens : tpt) * p.G * 128);
                for (int s = 0; s < L::SUB; ++s)
                  tma_load_3d(smem + L::OFF_Q + s * L::Q_SUB, few ? &tm_q_few : &tm_q, bar_qf, s * 64,
                              q0, rc.tok0);
              }
              ++qn;
            }
          }
          if (ok && it >= L::VST)
            ok = __all_sync(0xffffffffu, mbar_wait(&bar_ve[vs], ((it / L::VST) - 1) & 1, abort_flag, SITE_PCH_LOAD_EMPTY));
          if (!ok) {
            ++it;  // its K load is in flight; see the drain
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(&bar_vf[vs], L::KV_TILE);
          __syncwarp();
          if (part == 0)
            tma_load_4d(smem + L::OFF_V + vs * L::KV_TILE + sub * L::KV_SUB + pg * box * 128, &tm_v,
                        &bar_vf[vs], sub * 64, row, h, page);
          ++it;
          cnt0 = it;  // V tiles issued
        }
      }
    } else if (warp == 9) {
      // ------------------------------------------------------------------ MMA issuer
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, BN, false, false);
      constexpr uint32_t idesc_o = idesc_bf16_f32(128, D, false, true);
      const uint64_t q_desc = sdesc_sw128(smem_u32(smem + L::OFF_Q), 16, 1024);
      const uint64_t k_desc = sdesc_sw128(smem_u32(smem + L::OFF_K), 16, 1024);
      const uint64_t v_desc = sdesc_sw128(smem_u32(smem + L::OFF_V), L::KV_SUB, 1024);
      auto koff = [](int k, int sub) -> uint64_t {
        return static_cast<uint64_t>(((k >> 2) * sub + (k & 3) * 32) >> 4);
      };
      // O_w (+)= P_w V(vs), as in the forward; cnt: P_w tiles taken so far
      auto issue_pv = [&](int w, int vs, int& cnt, bool acc) -> bool {
        if (!mbar_wait_w(&bar_pf[w], cnt & 1, abort_flag, SITE_PCH_MMA_P)) return false;
        tc_fence_after();
        const uint32_t a_tmem = tmem + L::s_col(w);
        const uint32_t d_tmem = tmem + L::O_COL0 + w * D;
        const uint64_t vb = v_desc + static_cast<uint64_t>((vs * L::KV_TILE) >> 4);
#pragma unroll
        for (int kb = 0; kb < BN / 64; ++kb) {
          if (L::SPLIT_P && kb == 1) {
            if (!mbar_wait_w(&bar_p2[w], cnt & 1, abort_flag, SITE_PCH_MMA_P)) return false;
            tc_fence_after();
          }
          uint32_t a[4];
          uint64_t b[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int k = 4 * kb + i;
            a[i] = a_tmem + 8 * k;
            b[i] = vb + static_cast<uint64_t>((k * 2048) >> 4);
          }
          mma_ts_x4(d_tmem, a, b, idesc_o, (acc || kb > 0) ? 1u : 0u);
        }
        mma_commit_w(&bar_od[w]);
        ++cnt;
        return true;
      };
      auto issue_s = [&](int w, int ks) {
        const uint64_t qa = q_desc + static_cast<uint64_t>((w * 128 * 128) >> 4);
        const uint64_t kb0 = k_desc + static_cast<uint64_t>((ks * L::KV_TILE) >> 4);
#pragma unroll
        for (int kb = 0; kb < D / 64; ++kb) {
          uint64_t a[4], b[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a[i] = qa + koff(4 * kb + i, L::Q_SUB);
            b[i] = kb0 + koff(4 * kb + i, L::KV_SUB);
          }
          mma_ss_x4(tmem + L::s_col(w), a, b, idesc_s, kb > 0 ? 1u : 0u);
        }
        mma_commit_w(&bar_sf[w]);
      };
      // P V of the last tile, when no S follows it in the same piece
      auto flush_pv = [&]() {
        if (ok && prev_flags != 0) {
          ok = mbar_wait_w(&bar_vf[prev_vs], (prev_it / L::VST) & 1, abort_flag, SITE_PCH_MMA_V);
          if (ok) {
            tc_fence_after();
            if (prev_flags & 1) ok = issue_pv(0, prev_vs, cnt0, prev_acc & 1);
            if (ok && (prev_flags & 2)) ok = issue_pv(1, prev_vs, cnt1, (prev_acc & 2) != 0);
            if (ok) mma_commit_w(&bar_ve[prev_vs]);
          }
        }
        prev_flags = 0;
      };
      while (ok && pieces.next(p, sched, pc)) {
        const PagedChunkPiece c = paged_chunk_piece<BN>(p, sched, pc);
        bool first = true;
        int acc = 0;  // bit w: O_w of this piece has been started
        const int j_end = min(c.b, max(c.n0, c.n1));
        for (int j = c.a; ok && j < j_end; ++j) {
          const int f = (j < c.n0 ? 1 : 0) | (j < c.n1 ? 2 : 0);  // the Q tiles that see this tile
          const int ks = it % L::KST;
          if (first) {
            // the piece before ends here: its last P V must not wait for this piece's loads
            flush_pv();
            ok = ok && mbar_wait_w(bar_qf, qn & 1, abort_flag, SITE_PCH_MMA_Q);
            ++qn;
            first = false;
          }
          ok = ok && mbar_wait_w(&bar_kf[ks], (it / L::KST) & 1, abort_flag, SITE_PCH_MMA_K);
          if (ok && prev_flags != 0)
            ok = mbar_wait_w(&bar_vf[prev_vs], (prev_it / L::VST) & 1, abort_flag, SITE_PCH_MMA_V);
          if (!ok) break;
          tc_fence_after();
          // for w = 0 then 1: PV_w of the previous tile, then S_w of this tile
          if (prev_flags & 1) ok = issue_pv(0, prev_vs, cnt0, prev_acc & 1);
          if (ok && (f & 1)) issue_s(0, ks);
          if (ok && (prev_flags & 2)) ok = issue_pv(1, prev_vs, cnt1, (prev_acc & 2) != 0);
          if (ok && (f & 2)) issue_s(1, ks);
          if (!ok) break;
          mma_commit_w(&bar_ke[ks]);
          if (prev_flags != 0) mma_commit_w(&bar_ve[prev_vs]);
          prev_flags = f;
          prev_vs = it % L::VST;
          prev_it = it;
          prev_acc = acc;
          acc |= f;
          ++it;
        }
        if (ok && !first) mma_commit_w(bar_qe);  // every S of this piece has read Q
      }
      flush_pv();  // the softmax warpgroups finish the listed pieces before the next list
      if (stop >= hi) {
        // all MMAs issued by this warp have completed before TMEM is released
        mma_commit_w(bar_fin);
        mbar_wait_w(bar_fin, 0, abort_flag, SITE_PCH_MMA_FIN);
      }
    } else {
      // ------------------------------------------------------------------ softmax warpgroups
      const int w = warp >> 2, qw = warp & 3;
      const int r = 128 * w + 32 * qw + lane;  // this thread's row of the tile
      const uint32_t t_lane = static_cast<uint32_t>(32 * qw) << 16;
      const uint32_t t_s = tmem + t_lane + L::s_col(w);
      const uint32_t t_o = tmem + t_lane + L::O_COL0 + w * D;
      const float scale2 = p.scale2;
      const int my_tok = r / p.G, warp_tok = (128 * w + 32 * qw) / p.G;
      while (pieces.next(p, sched, pc)) {
        const PagedChunkPiece c = paged_chunk_piece<BN>(p, sched, pc);
        float m_ref = -INFINITY, l = 0.f;
        const int cnt_piece = cnt0;
        const int kv = sched.rec[c.rec].kv;
        int n_row, n_min;  // keys of this row, and of the warp's first row (the fewest)
        {
          const PagedRec& rc = sched.rec[c.rec];
          n_row = p.causal ? min(kv, rc.pos0 + my_tok + 1) : kv;
          n_min = p.causal ? min(kv, rc.pos0 + warp_tok + 1) : kv;
        }
        const int j_end = min(c.b, w == 0 ? c.n0 : c.n1);
        for (int j = c.a; j < j_end && ok; ++j) {
          const int my_it = it + (j - c.a);
          const bool got = mbar_wait(&bar_sf[w], cnt0 & 1, abort_flag, SITE_PCH_SM_S);
          if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
          tc_fence_after();
          constexpr int NC = BN / 32;
          if (const int bad = s_info[my_it % L::INFO]) paged_hide<BN>(t_s, bad);
          uint32_t rg[NC][32];
#pragma unroll
          for (int cc = 0; cc < NC; ++cc) tmem_ld32(t_s + 32 * cc, rg[cc]);
          const int k0 = j * BN;
          tmem_ld_wait();
#pragma unroll
          for (int cc = 0; cc < NC; ++cc) reg_fence(rg[cc]);
          if (k0 + BN > n_min) {
#pragma unroll
            for (int cc = 0; cc < NC; ++cc)
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (k0 + 32 * cc + i >= n_row) rg[cc][i] = __float_as_uint(-INFINITY);
          }
          float mc[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) mc[u] = -INFINITY;
#pragma unroll
          for (int k = 0; k < BN; k += 2)
            mc[(k >> 1) & 7] = fmax3(mc[(k >> 1) & 7], __uint_as_float(rg[k >> 5][k & 31]),
                                     __uint_as_float(rg[k >> 5][(k & 31) + 1]));
          const float mx = fmax3(fmax3(mc[0], mc[1], mc[2]), fmax3(mc[3], mc[4], mc[5]),
                                 fmaxf(mc[6], mc[7]));
          const float tmax = mx * scale2;
          float m_new = m_ref;
          if (tmax > m_ref + 8.0f) m_new = tmax;  // also taken when m_ref is still -inf
          const float alpha = (m_new == m_ref) ? 1.0f : ex2_approx(m_ref - m_new);
          const float neg_base = (m_new == -INFINITY) ? 0.0f : -m_new;
          const bool rescale = cnt0 != cnt_piece && (m_new != m_ref);
          m_ref = m_new;
          float ra[4] = {0.f, 0.f, 0.f, 0.f}, rb[4] = {0.f, 0.f, 0.f, 0.f};
          auto exp_chunk = [&](int cc) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int q = 16 * cc + i;
              float x0, x1, p0, p1;
              ffma2(x0, x1, __uint_as_float(rg[cc][2 * i]), __uint_as_float(rg[cc][2 * i + 1]), scale2,
                    scale2, neg_base, neg_base);
              p0 = ex2_approx(x0);
              p1 = ex2_approx(x1);
              fadd2(ra[q & 3], rb[q & 3], ra[q & 3], rb[q & 3], p0, p1);
              pk[i] = pack_bf16x2(p0, p1);
            }
            tmem_st16(t_s + 16 * cc, pk);
          };
          auto hand_over = [&](uint64_t* bar) {
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(bar);
          };
          auto rescale_o = [&]() {
            if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
              for (int cc = 0; cc < D / 32; ++cc) {
                uint32_t o[32];
                tmem_ld32(t_o + 32 * cc, o);
                tmem_ld_wait();
                reg_fence(o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                tmem_st32(t_o + 32 * cc, o);
              }
            }
          };
          // V rows behind the request's last key in its last page: cleared (both warpgroups write
          // the same zeros, each before its own P goes out)
          const int stale = kv - k0;
          if (stale < BN && (kv & ((1 << p.page_shift) - 1)) != 0) {
            const int vs = my_it % L::VST;
            const bool gv = mbar_wait(&bar_vf[vs], (my_it / L::VST) & 1, abort_flag, SITE_PCH_SM_V);
            if (!__all_sync(0xffffffffu, gv)) { ok = false; break; }
            const int page_end = ((kv >> p.page_shift) + 1) << p.page_shift;
            const int n = (min(BN, page_end - k0) - stale) * 8 * L::SUB;
            for (int e = 32 * qw + lane; e < n; e += 128) {
              const int row = stale + e / (8 * L::SUB), q = e % (8 * L::SUB);
              *reinterpret_cast<uint4*>(smem + L::OFF_V + vs * L::KV_TILE + (q >> 3) * L::KV_SUB +
                                        row * 128 + (q & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
          }
          constexpr int C1 = L::SPLIT_P ? NC / 2 : NC;
#pragma unroll
          for (int cc = 0; cc < C1; ++cc) exp_chunk(cc);
          rescale_o();
          hand_over(&bar_pf[w]);
          if constexpr (L::SPLIT_P) {
#pragma unroll
            for (int cc = C1; cc < NC; ++cc) exp_chunk(cc);
            hand_over(&bar_p2[w]);
          }
          l = alpha * l + ((ra[0] + ra[1]) + (ra[2] + ra[3]) + ((rb[0] + rb[1]) + (rb[2] + rb[3])));
          ++cnt0;
        }
        // ---------------------------------------------------------------- write the piece out
        it += max(0, min(c.b, max(c.n0, c.n1)) - c.a);
        const PagedRec rc = sched.rec[c.rec];
        const int rows = rc.ntok * p.G;
        const bool any = cnt0 != cnt_piece;
        const bool whole = c.a == 0 && c.b == rc.n;
        if (ok && 128 * w < rows) {
          if (any) {
            const bool got = mbar_wait(&bar_od[w], (cnt0 - 1) & 1, abort_flag, SITE_PCH_SM_O);
            ok = __all_sync(0xffffffffu, got);
            tc_fence_after();
          }
          const size_t slot = static_cast<size_t>(cta) * 2 + (c.a > 0 ? 0 : 1);
          const int qh = ok ? paged_row_head(p, c.h, r, rows) : -1;
          const long long row = static_cast<long long>(rc.tok0 + my_tok) * p.H + qh;
          const float inv = 1.0f / l;
#pragma unroll
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t o[32];
            if (any && ok) {
              tmem_ld32(t_o + 32 * cc, o);
              tmem_ld_wait();
              reg_fence(o);
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = 0u;
            }
            if (qh >= 0) {
              if (whole) {
                __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) + row * D + 32 * cc;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  uint32_t hh[8];
#pragma unroll
                  for (int e = 0; e < 8; ++e)
                    hh[e] = l == 0.f ? 0u
                                     : pack_bf16x2(__uint_as_float(o[16 * i + 2 * e]) * inv,
                                                   __uint_as_float(o[16 * i + 2 * e + 1]) * inv);
                  if (p.o_al32) {
                    st_global_256(dst + 16 * i, hh[0], hh[1], hh[2], hh[3], hh[4], hh[5], hh[6], hh[7]);
                  } else {
                    *reinterpret_cast<uint4*>(dst + 16 * i) = make_uint4(hh[0], hh[1], hh[2], hh[3]);
                    *reinterpret_cast<uint4*>(dst + 16 * i + 8) = make_uint4(hh[4], hh[5], hh[6], hh[7]);
                  }
                }
              } else {
                float* dst = p.ws_o + (slot * p.rows_cap + r) * p.ws_pitch + 32 * cc;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  st_global_256(dst + 8 * i, o[8 * i], o[8 * i + 1], o[8 * i + 2], o[8 * i + 3], o[8 * i + 4],
                                o[8 * i + 5], o[8 * i + 6], o[8 * i + 7]);
              }
            }
          }
          if (qh >= 0) {
            if (whole) p.lse[row] = paged_lse(m_ref, l);
            else p.ws_ml[slot * p.rows_cap + r] = make_float2(m_ref, l);
          }
          tc_fence_before();  // O has been read before this warpgroup's next P goes out
        }
        if (threadIdx.x == 0 && !whole) paged_header<C>(p, sched, rc, pc, cta);
      }
    }
    x = stop;
    __syncthreads();  // the list is rewritten
  }
  if (warp == 8) {
    // Never leave the CTA with a copy in flight (immediate in the normal path)
    if (qn > 0) mbar_wait_drain(bar_qf, (qn - 1) & 1, SITE_PCH_LOAD_DRAIN);
    for (int r = max(0, it - L::KST); r < it; ++r)
      mbar_wait_drain(&bar_kf[r % L::KST], (r / L::KST) & 1, SITE_PCH_LOAD_DRAIN);
    for (int r = max(0, cnt0 - L::VST); r < cnt0; ++r)
      mbar_wait_drain(&bar_vf[r % L::VST], (r / L::VST) & 1, SITE_PCH_LOAD_DRAIN);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, L::TMEM_COLS);
  }
}

}  // namespace fa
