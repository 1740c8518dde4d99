// fa_paged_decode_sm100.cuh -- paged attention of few new tokens (decoding), bf16: at most 16
// rows (tokens x query heads of a group) per tile, so that each key is used a few times only and
// the cache's bytes are what counts.
//
// Bound by HBM: K and V are read once.  The loop therefore is a stream: four producer warps keep a
// ring of 64-key K/V tiles filled by TMA (one box per page and 64 columns; 128-byte swizzle; a
// warp issues its boxes one after the other, so 16-row pages want several warps: 3.9 TB/s with
// one, 4.6 with two, 5.0 with four at d = 64), and eight consumer warps, in two groups that take
// alternate tiles, work on 16 keys each with warp-level m16n8k16 MMAs -- the 16 rows fill one such
// tile, where a tcgen05 tile would be 128 rows of which 112 are idle, and the S and P of a warp
// never leave its registers.  Each warp keeps its own running maximum and sum, so warps meet once
// per item, not per tile; the eight partial results are then added through shared memory in fp32.
// An SM has about 22 bytes of HBM per cycle, a 64-key tile (d = 128) takes 1490 cycles to arrive,
// and a group needs about 500 for it, so the stream, not the arithmetic, sets the pace.
// Measured: 64 requests of up to 16384 keys, 32 heads over 8, d = 128 (2.17 GB): 335 us, 6.5 TB/s,
// the rate of a copy; 16 requests of 8192 keys: 96 us, 5.6 TB/s (d = 128), 52 us, 5.2 TB/s (d = 64);
// one request of 2000 keys: 10 us with its join.
//
// Page ids are fetched 8 to 32 tiles ahead.  A page that the table does not name, or that lies behind
// the last key, is read as an out-of-range page, which TMA fills with zeros without reading.
// Rows of the last page behind the last key may hold anything: their scores are replaced and
// their V elements cleared in registers.
//
// P is rounded to bf16 for P V (its row sum is taken before, in fp32); scores, statistics and
// sums are fp32.
#pragma once
#include "fa_paged.cuh"

namespace fa {

enum : int { SITE_PDEC_EMPTY = 40, SITE_PDEC_FULL = 41, SITE_PDEC_DRAIN = 42 };

template <int D>
struct PagedDecodeLayout {
  static constexpr int R = 16, KT = 64;
  static constexpr int C = 1;                        // an item's constant, in key tiles
  static constexpr int WARPS = 8;                    // consumers
  static constexpr int PRODUCERS = 4;                // two for K, two for V
  static constexpr int THREADS = (WARPS + PRODUCERS) * 32;
  static constexpr int SUB = D / 64;                 // 64-column (128-byte) sub-tiles
  static constexpr int SUBTILE = KT * 128;           // bytes
  static constexpr int TILE = KT * D * 2;            // one K or V tile
  static constexpr int STAGE = 2 * TILE;
  // Ring depth (192 KB).  Even, so that a stage always belongs to the same group: a group that
  // took a stage only every other round could not tell "not yet loaded" from "loaded twice" by
  // the barrier's phase parity, whose loads may complete out of order.
  static constexpr int ST = D == 128 ? 6 : 12;
  static_assert(ST % 2 == 0, "a stage belongs to one group");
  static constexpr int PITCH = D + 8;                // floats per row of the join buffer
  static constexpr int OFF_Q = ST * STAGE;           // [16][D] bf16, swizzled
  static constexpr int OFF_O = OFF_Q + R * D * 2;    // [4 warps][8 rows][PITCH] fp32
  static constexpr int OFF_ML = OFF_O + WARPS / 2 * 8 * PITCH * 4;  // [8 warps][16 rows] (m, l)
  static constexpr int OFF_BAR = OFF_ML + WARPS * R * 8;        // full[ST], empty[ST]
  static constexpr int OFF_BAD = OFF_BAR + 2 * ST * 8;          // [ST] bits: bad 16-key groups
  static constexpr int OFF_ABORT = OFF_BAD + ST * 4;
  static constexpr int OFF_SCHED = (OFF_ABORT + 4 + 15) / 16 * 16;
  static constexpr int BYTES = OFF_SCHED + static_cast<int>(sizeof(PagedSched));
  static constexpr int SMEM_ALLOC = BYTES + 1024;    // slack for 1024-byte alignment
  static_assert(SMEM_ALLOC <= 232448, "shared memory per CTA");
};

__device__ __forceinline__ void tma_load_4d(void* smem_dst, const CUtensorMap* map, uint64_t* bar,
                                            int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// c += a b, 16 x 8 x 16, bf16 operands, fp32 sums
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
__global__ void __launch_bounds__(PagedDecodeLayout<D>::THREADS, 1)
fa_paged_decode_sm100_kernel(const __grid_constant__ CUtensorMap tm_k,
                             const __grid_constant__ CUtensorMap tm_v, const PagedParams p) {
  using L = PagedDecodeLayout<D>;
  constexpr int KT = L::KT, ST = L::ST, C = L::C;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bar_full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* bar_empty = bar_full + ST;
  volatile int* s_bad = reinterpret_cast<volatile int*>(smem + L::OFF_BAD);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_ABORT);
  PagedSched& sched = *reinterpret_cast<PagedSched*>(smem + L::OFF_SCHED);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tpt = L::R / p.G;  // G <= R

  if (tid == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&bar_full[s], L::PRODUCERS);
      mbar_init(&bar_empty[s], L::WARPS / 2);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  grid_dep_wait();  // launched to overlap the kernel before
  grid_dep_launch();
  const int cta = blockIdx.x;
  long long x, hi;
  PagedMine mine = {};
  if (!paged_share<KT, C, L::THREADS>(p, tpt, sched, x, hi, mine)) return;  // else: a barrier has passed
  int it = 0;      // tiles issued (producer) or passed (consumers) so far
  bool ok = true;

  paged_list<KT, C, L::THREADS>(p, tpt, x, hi, &mine, sched);
  while (true) {
    const long long stop = sched.stop;
    if (warp >= L::WARPS) {
      // ---------------------------------------------------------------- producers
      const int box = min(1 << p.page_shift, KT);  // rows of a page in a tile
      const int np = KT / box;                     // pages in a tile
      const int part = (warp - L::WARPS) & 1;      // 0: K, 1: V; two warps take its boxes by turns
      const bool issues = lane < np * L::SUB && (lane & 1) == ((warp - L::WARPS) >> 1);
      const int bytes = __popc(__ballot_sync(0xffffffffu, issues)) * box * 128;
      const int pg = lane / L::SUB % np, sub = lane % L::SUB;
      // The pages of 32 / np tiles from t0 on, one per lane (-1 behind the last key: not looked up).
      // Fetched a batch ahead: a tile of 16 KB (d = 64) arrives faster than a table entry.
      const int batch = 32 / np;
      auto pages_of = [&](const PagedPiece& q, int t0) -> int {
        const PagedRec& rc = sched.rec[q.rec];
        const int j = t0 * KT + lane * box;
        if (j >= paged_keys(p.causal, rc.kv, rc.pos0, rc.ntok)) return -1;
        return p.table[rc.b * p.table_stride + (j >> p.page_shift)];
      };
      PagedPieces<C> pieces;
      pieces.start(p, sched, x);
      PagedPiece pc, after;
      bool more = pieces.next(p, sched, pc);
      int ids = more ? pages_of(pc, pc.a) : 0;
      while (more && ok) {
        const PagedRec& rc = sched.rec[pc.rec];
        const int keys = paged_keys(p.causal, rc.kv, rc.pos0, rc.ntok), h = pc.h / p.splits;
        more = pieces.next(p, sched, after);
        for (int t0 = pc.a; t0 < pc.b && ok; t0 += batch) {
          int ids_next = 0;
          if (t0 + batch < pc.b) ids_next = pages_of(pc, t0 + batch);
          else if (more) ids_next = pages_of(after, after.a);
          const bool mine_bad = (ids < 0 || ids >= p.num_pages) && t0 * KT + lane * box < keys;
          const bool any_bad = __any_sync(0xffffffffu, mine_bad);
          for (int t = t0; t < min(pc.b, t0 + batch); ++t) {
            const int id = __shfl_sync(0xffffffffu, ids, (t - t0) * np + pg);
            unsigned bad = 0;  // groups of 16 keys whose page the table does not name
            if (any_bad) {
              const bool b16 = __shfl_sync(0xffffffffu, mine_bad, (t - t0) * np + 16 * (lane & 3) / box);
              bad = __ballot_sync(0xffffffffu, lane < KT / 16 && b16);
            }
            const int s = it % ST;
            if (it >= ST)
              ok = __all_sync(0xffffffffu, mbar_wait(&bar_empty[s], ((it / ST) - 1) & 1, abort_flag,
                                                     SITE_PDEC_EMPTY));
            if (!ok) break;
            if (lane == 0) {
              if (warp == L::WARPS) s_bad[s] = static_cast<int>(bad);
              if (bytes > 0) mbar_arrive_expect_tx(&bar_full[s], bytes);
              else mbar_arrive(&bar_full[s]);
            }
            __syncwarp();
            if (issues)
              tma_load_4d(smem + s * L::STAGE + part * L::TILE + sub * L::SUBTILE + pg * box * 128,
                          part == 0 ? &tm_k : &tm_v, &bar_full[s], sub * 64,
                          (t * KT) & ((1 << p.page_shift) - 1), h,
                          id >= 0 && id < p.num_pages ? id : p.num_pages);
            ++it;
          }
          ids = ids_next;
        }
        pc = after;
      }
    } else {
      // ---------------------------------------------------------------- consumers
      const int group = warp >> 2, w4 = warp & 3;
      const int g = lane >> 2, c = lane & 3;
      float2* s_ml = reinterpret_cast<float2*>(smem + L::OFF_ML);
      float* s_o = reinterpret_cast<float*>(smem + L::OFF_O);
      const uint32_t q_addr = smem_u32(smem + L::OFF_Q);
      PagedPieces<C> pieces;
      pieces.start(p, sched, x);
      PagedPiece pc;
      while (pieces.next(p, sched, pc)) {
        const PagedRec rc = sched.rec[pc.rec];
        const int rows = rc.ntok * p.G;
        const int keys = paged_keys(p.causal, rc.kv, rc.pos0, rc.ntok);
        // Q rows to shared memory: 16-byte chunk q of row r at chunk q ^ (r & 7)
        constexpr int CH = D / 8;
        for (int e = tid; e < L::R * CH; e += L::WARPS * 32) {
          const int r = e / CH, q = e % CH;
          const int qh = paged_row_head(p, pc.h, r, rows);
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (qh >= 0)
            v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                static_cast<long long>(rc.tok0 + r / p.G) * p.q_st +
                                                qh * p.q_sh + q * 8);
          *reinterpret_cast<uint4*>(smem + L::OFF_Q + r * (D * 2) + ((q ^ (r & 7)) * 16)) = v;
        }
        named_bar_sync(1, L::WARPS * 32);
        uint32_t qf[D / 16][4];
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          // matrices: rows 0-7 / 8-15 of columns 16k..16k+7, then of 16k+8..16k+15
          const int r = lane & 15, q = 2 * k + (lane >> 4);
          ldsm4(qf[k], q_addr + r * (D * 2) + ((q ^ (r & 7)) * 16));
        }
        float o[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // rows g and g + 8
        // keys that rows g and g + 8 see, and the first row (the fewest)
        const int n0 = p.causal ? min(keys, rc.pos0 + g / p.G + 1) : keys;
        const int n1 = p.causal ? min(keys, rc.pos0 + (g + 8) / p.G + 1) : keys;
        const int n_min = p.causal ? min(keys, rc.pos0 + 1) : keys;

        for (int t = pc.a; t < pc.b; ++t, ++it) {
          if ((it & 1) != group || !ok) continue;
          const int s = it % ST;
          ok = __all_sync(0xffffffffu, mbar_wait(&bar_full[s], (it / ST) & 1, abort_flag,
                                                 SITE_PDEC_FULL));
          if (!ok) continue;
          const uint32_t kb = smem_u32(smem + s * L::STAGE), vb = kb + L::TILE;
          const int k0 = t * KT + 16 * w4;  // this warp's keys
          const bool bad = (s_bad[s] >> w4) & 1;
          // ---- S = Q K^T, 16 rows x 16 keys
          float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
          {
            // matrices: keys 0-7 at columns 16k.., 16k+8.., then keys 8-15
            const int r = 16 * w4 + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const int q = 2 * k + ((lane >> 3) & 1);
              uint32_t b[4];
              ldsm4(b, kb + (q >> 3) * L::SUBTILE + r * 128 + (((q & 7) ^ (r & 7)) * 16));
              mma_16816(sa, qf[k], b[0], b[1]);
              mma_16816(sb, qf[k], b[2], b[3]);
            }
          }
          // ---- mask; columns of this lane: 2c, 2c+1 (sa) and 8 + 2c, 8 + 2c + 1 (sb)
          const bool edge = bad || k0 + 16 > n_min;
          if (edge) {
            const int j = k0 + 2 * c;
            const int a0 = bad ? 0 : n0, a1 = bad ? 0 : n1;
            if (j >= a0) sa[0] = -INFINITY;
            if (j + 1 >= a0) sa[1] = -INFINITY;
            if (j >= a1) sa[2] = -INFINITY;
            if (j + 1 >= a1) sa[3] = -INFINITY;
            if (j + 8 >= a0) sb[0] = -INFINITY;
            if (j + 9 >= a0) sb[1] = -INFINITY;
            if (j + 8 >= a1) sb[2] = -INFINITY;
            if (j + 9 >= a1) sb[3] = -INFINITY;
          }
          float x0 = fmaxf(fmaxf(sa[0], sa[1]), fmaxf(sb[0], sb[1]));
          float x1 = fmaxf(fmaxf(sa[2], sa[3]), fmaxf(sb[2], sb[3]));
          x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
          x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
          x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2)) * p.scale2;
          x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2)) * p.scale2;
          // the reference maximum moves only when it grows by more than 8 (2^8): P <= 256
          const bool up0 = x0 > m0 + 8.0f, up1 = x1 > m1 + 8.0f;
          if (__any_sync(0xffffffffu, up0 || up1)) {
            const float f0 = up0 ? ex2_approx(m0 - x0) : 1.0f;  // 0 when m0 was -inf
            const float f1 = up1 ? ex2_approx(m1 - x1) : 1.0f;
            if (up0) m0 = x0;
            if (up1) m1 = x1;
            l0 *= f0;
            l1 *= f1;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
              o[i][0] *= f0;
              o[i][1] *= f0;
              o[i][2] *= f1;
              o[i][3] *= f1;
            }
          }
          const float z0 = m0 == -INFINITY ? 0.f : -m0, z1 = m1 == -INFINITY ? 0.f : -m1;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            sa[i] = ex2_approx(fmaf(sa[i], p.scale2, z0));
            sb[i] = ex2_approx(fmaf(sb[i], p.scale2, z0));
            sa[2 + i] = ex2_approx(fmaf(sa[2 + i], p.scale2, z1));
            sb[2 + i] = ex2_approx(fmaf(sb[2 + i], p.scale2, z1));
          }
          l0 += (sa[0] + sa[1]) + (sb[0] + sb[1]);
          l1 += (sa[2] + sa[3]) + (sb[2] + sb[3]);
          const uint32_t pf[4] = {pack_bf16x2(sa[0], sa[1]), pack_bf16x2(sa[2], sa[3]),
                                  pack_bf16x2(sb[0], sb[1]), pack_bf16x2(sb[2], sb[3])};
          // ---- O += P V
          {
            // matrices (transposed): keys 0-7 and 8-15 at columns 16i.., then at 16i+8..
            const int r = 16 * w4 + (lane & 15);
            uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;  // V rows 2c, 2c+1 / 8+2c, 8+2c+1
            if (edge) {
              const int j = k0 + 2 * c;
              keep0 = (j < keys ? 0xffffu : 0u) | (j + 1 < keys ? 0xffff0000u : 0u);
              keep1 = (j + 8 < keys ? 0xffffu : 0u) | (j + 9 < keys ? 0xffff0000u : 0u);
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              const int q = 2 * i + (lane >> 4);
              uint32_t b[4];
              ldsm4_t(b, vb + (q >> 3) * L::SUBTILE + r * 128 + (((q & 7) ^ (r & 7)) * 16));
              mma_16816(o[2 * i], pf, b[0] & keep0, b[1] & keep1);
              mma_16816(o[2 * i + 1], pf, b[2] & keep0, b[3] & keep1);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_empty[s]);
        }
        // ---- the eight warps' results
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
        if (c == 0) {
          s_ml[warp * L::R + g] = make_float2(m0, l0);
          s_ml[warp * L::R + g + 8] = make_float2(m1, l1);
        }
        named_bar_sync(1, L::WARPS * 32);
        const bool whole = pc.a == 0 && pc.b == rc.n;
        const size_t slot = paged_slot(cta, pc);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (8 * half >= rows) break;
          {
            const int r = 8 * half + g;
            float mm = -INFINITY;
#pragma unroll
            for (int w = 0; w < L::WARPS; ++w) mm = fmaxf(mm, s_ml[w * L::R + r].x);
            const bool some = (half ? l1 : l0) != 0.f;  // this warp has keys of the row
            const float f = ex2_approx((half ? m1 : m0) - mm);
            // group 1 hands over, group 0 adds its own (the same thread's places), row by row
            float* dst = s_o + (w4 * 8 + g) * L::PITCH + 2 * c;
            if (group == 1) {
#pragma unroll
              for (int i = 0; i < D / 8; ++i)
                *reinterpret_cast<float2*>(dst + 8 * i) =
                    some ? make_float2(o[i][2 * half] * f, o[i][2 * half + 1] * f) : make_float2(0.f, 0.f);
            }
            named_bar_sync(1, L::WARPS * 32);
            if (group == 0 && some) {
#pragma unroll
              for (int i = 0; i < D / 8; ++i) {
                const float2 other = *reinterpret_cast<const float2*>(dst + 8 * i);
                *reinterpret_cast<float2*>(dst + 8 * i) =
                    make_float2(fmaf(o[i][2 * half], f, other.x), fmaf(o[i][2 * half + 1], f, other.y));
              }
            }
          }
          named_bar_sync(1, L::WARPS * 32);
          {
            // warp w finishes row 8 half + w
            const int r = 8 * half + warp;
            const int qh = paged_row_head(p, pc.h, r, rows);
            if (qh >= 0) {
              float mm = -INFINITY, ll = 0.f;
#pragma unroll
              for (int w = 0; w < L::WARPS; ++w) mm = fmaxf(mm, s_ml[w * L::R + r].x);
#pragma unroll
              for (int w = 0; w < L::WARPS; ++w) {
                const float2 ml = s_ml[w * L::R + r];
                if (ml.y != 0.f) ll = fmaf(ml.y, ex2_approx(ml.x - mm), ll);
              }
              constexpr int E = D / 32;  // columns of a lane
              float acc[E];
#pragma unroll
              for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
              for (int w = 0; w < L::WARPS / 2; ++w) {
                const float* src = s_o + (w * 8 + warp) * L::PITCH + lane * E;
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] += src[e];
              }
              if (whole) {
                const float inv = ll == 0.f ? 0.0f : 1.0f / ll;
                const long long row = static_cast<long long>(rc.tok0 + r / p.G) * p.H + qh;
                uint32_t* op = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) + row * D + lane * E);
#pragma unroll
                for (int e = 0; e < E / 2; ++e) op[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
                if (lane == 0) p.lse[row] = paged_lse(mm, ll);
              } else {
                float* op = p.ws_o + (slot * p.rows_cap + r) * p.ws_pitch + lane * E;
#pragma unroll
                for (int e = 0; e < E; ++e) op[e] = acc[e];
                if (lane == 0) p.ws_ml[slot * p.rows_cap + r] = make_float2(mm, ll);
              }
            }
          }
          named_bar_sync(1, L::WARPS * 32);  // s_o (and, after the last, s_ml and Q) may be rewritten
        }
        if (tid == 0 && !whole) paged_header<C>(p, sched, rc, pc, cta);
      }
    }
    x = stop;
    if (x >= hi) break;
    __syncthreads();  // the list is rewritten
    paged_list<KT, C, L::THREADS>(p, tpt, x, hi, nullptr, sched);
  }
  if (warp >= L::WARPS) {
    // no copy may be in flight when the CTA ends (immediate unless a wait gave up)
    for (int r = max(0, it - ST); r < it; ++r) mbar_wait_drain(&bar_full[r % ST], (r / ST) & 1, SITE_PDEC_DRAIN);
  }
}

}  // namespace fa
