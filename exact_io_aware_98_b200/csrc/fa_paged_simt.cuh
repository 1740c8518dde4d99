// fa_paged_simt.cuh -- paged attention on CUDA cores: fp32 inputs, fp32 products and sums.
//
// Warps in WR row groups x WK key groups, RW rows and 32 KPL keys per warp and key tile.  Lane =
// key for the scores (RW dot products per key of the lane, as packed pairs of products, Q rows
// broadcast from shared memory); for P V a lane has the columns lane, lane + 32, .. (NC of them,
// the head dimension over 32 rounded up, so that a head of 64 or 80 columns does not pay for
// 128).  K and V rows are padded so that 16-byte reads of 32 rows at one column spread over all
// banks.  K and V tiles come by 16-byte asynchronous copies, the K tile of step t+1 while P V of
// step t runs and the V tile while the scores are formed; the page of a key is looked up two
// tiles ahead.  The reference maximum of a row moves only when a score exceeds it by more than 8
// (in log2 units), which one vote finds; so most tiles need no reduction over lanes.
//   PagedSimtFew (8 rows, 128 keys a tile, 8 warps): few rows per K/V head (decoding); bound by
//     HBM, so many keys in flight and little to do per key.
//   PagedSimtChunk (32 rows, 64 keys a tile, 4 warps): each key is read once per 32 rows, where 8
//     rows would make every SM read 64 bytes of L2 a cycle.  Bound by FFMA and shared-memory
//     reads, which two keys per lane balance: a Q row is read once for both.
#pragma once
#include "fa_paged.cuh"

namespace fa {

struct PagedSimtFew {
  static constexpr int WR = 2, WK = 4, RW = 4, KPL = 1;
};
struct PagedSimtChunk {
  static constexpr int WR = 4, WK = 1, RW = 8, KPL = 2;
};

template <typename Shape>
struct PagedSimtLayout {
  static constexpr int WARPS = Shape::WR * Shape::WK, THREADS = 32 * WARPS;
  static constexpr int R = Shape::WR * Shape::RW, KT = 32 * Shape::WK * Shape::KPL;
  static constexpr int C = 1;  // an item's constant, in key tiles
  static constexpr int P = 32 * Shape::KPL * Shape::RW;  // P of a warp, floats
  static_assert(WARPS * Shape::RW <= KT, "the warps' sums fit the K tile");
  static_assert(2 * WARPS * Shape::RW <= WARPS * P, "the warps' statistics fit P");
  // row pitch in floats of a d-column tile: an odd number of 16-byte chunks
  __host__ __device__ static int pitch(int d) { return (((d + 3) / 4) | 1) * 4; }
  // Q [R], K [KT], V [KT] rows, P [warps], offsets of the keys' rows in k and v [3 tiles][2][KT];
  // the K tile later holds the warps' sums, P their statistics
  static size_t bytes(int d) {
    return (static_cast<size_t>(R + 2 * KT) * pitch(d) + WARPS * P) * 4 + 6 * KT * 8 + sizeof(PagedSched);
  }
  // CTAs per SM that registers are kept for
  __host__ __device__ static constexpr int ctas(int nc) { return Shape::WK > 1 ? (nc > 2 ? 1 : 2) : (nc == 4 ? 2 : 3); }
};

__device__ __forceinline__ void cp_async16(void* smem, const void* g) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(g) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <typename Shape, int NC>
__global__ void __launch_bounds__(PagedSimtLayout<Shape>::THREADS, PagedSimtLayout<Shape>::ctas(NC))
fa_paged_simt_kernel(const PagedParams p) {
  using L = PagedSimtLayout<Shape>;
  constexpr int R = L::R, KT = L::KT, C = L::C, NT = L::THREADS;
  constexpr int WK = Shape::WK, RW = Shape::RW, KPL = Shape::KPL;
  extern __shared__ __align__(16) uint8_t smem_simt[];
  const int d = p.d, pitch = L::pitch(d), dv = (d + 3) / 4;
  float* s_q = reinterpret_cast<float*>(smem_simt);
  float* s_k = s_q + R * pitch;
  float* s_v = s_k + KT * pitch;
  float* s_p = s_v + KT * pitch;
  long long* s_off = reinterpret_cast<long long*>(s_p + L::WARPS * L::P);
  PagedSched& sched = *reinterpret_cast<PagedSched*>(s_off + 6 * KT);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wr = warp / WK, wk = warp % WK;
  const int tpt = R / p.G;  // G <= R

  // zero the columns that pad d up to a multiple of 4 (read by the 16-byte accesses)
  for (int e = tid; e < (R + 2 * KT) * pitch; e += NT) s_q[e] = 0.f;
  grid_dep_wait();  // launched to overlap the kernel before
  grid_dep_launch();
  const int cta = blockIdx.x;
  long long x, hi;
  PagedMine mine = {};
  if (!paged_share<KT, C, NT>(p, tpt, sched, x, hi, mine)) return;
  float* my_p = s_p + warp * L::P;
  // this thread's first 16-byte chunk (or element) of a tile, and the step to its next
  const int per_row = p.vec ? dv : d;
  const int ld_r = tid / per_row, ld_c = tid % per_row, ld_dr = NT / per_row, ld_dc = NT % per_row;

  paged_list<KT, C, NT>(p, tpt, x, hi, &mine, sched);
  while (true) {
    PagedPieces<C> pieces;
    pieces.start(p, sched, x);
    PagedPiece pc;
    while (pieces.next(p, sched, pc)) {
      const PagedRec rc = sched.rec[pc.rec];
      const int rows = rc.ntok * p.G;
      const int keys = paged_keys(p.causal, rc.kv, rc.pos0, rc.ntok);
      const int32_t* table = p.table + rc.b * p.table_stride;
      const long long hrow = static_cast<long long>(pc.h / p.splits) << p.page_shift;
      // key tid of tile t: its page (-1: no such key, or the table does not name one) ...
      auto page_of = [&](int t) -> int {
        const int j = t * KT + tid;
        if (tid >= KT || j >= keys) return -1;
        return table[j >> p.page_shift];
      };
      // ... and, noted for the copies, where its rows start in k and v, or -1
      auto note = [&](int t, int pg) {
        if (tid >= KT) return;
        const bool there = pg >= 0 && pg < p.num_pages;
        const long long row = (hrow + ((t * KT + tid) & ((1 << p.page_shift) - 1))) * d;
        s_off[t % 3 * 2 * KT + tid] = there ? pg * p.k_page + row : -1;
        s_off[t % 3 * 2 * KT + KT + tid] = there ? pg * p.v_page + row : -1;
      };
      // missing keys become zero rows: a stale row may hold anything, and 0 times it is not 0
      auto load = [&](float* dst, const void* base, const long long* off) {
        const float* g = static_cast<const float*>(base);
        for (int r = ld_r, c = ld_c; r < KT;) {
          const long long o = off[r];
          if (p.vec) {
            if (o >= 0) cp_async16(dst + r * pitch + 4 * c, g + o + 4 * c);
            else *reinterpret_cast<float4*>(dst + r * pitch + 4 * c) = make_float4(0.f, 0.f, 0.f, 0.f);
          } else {
            dst[r * pitch + c] = o >= 0 ? g[o + c] : 0.f;
          }
          r += ld_dr;
          c += ld_dc;
          if (c >= per_row) {
            c -= per_row;
            ++r;
          }
        }
        cp_async_commit();
      };
      auto load_k = [&](int t) { load(s_k, p.k, s_off + t % 3 * 2 * KT); };
      auto load_v = [&](int t) { load(s_v, p.v, s_off + t % 3 * 2 * KT + KT); };
      __syncthreads();  // the previous piece's reads of every shared array are over
      for (int e = tid; e < R * d; e += NT) {
        const int r = e / d, c = e - r * d;
        const long long tok = rc.tok0 + r / p.G;
        const int qh = paged_row_head(p, pc.h, r, rows);
        s_q[r * pitch + c] =
            qh >= 0 ? static_cast<const float*>(p.q)[tok * p.q_st + qh * p.q_sh + c] : 0.f;
      }
      note(pc.a, page_of(pc.a));
      if (pc.a + 1 < pc.b) note(pc.a + 1, page_of(pc.a + 1));
      __syncthreads();
      load_k(pc.a);
      load_v(pc.a);

      float m[RW], l[RW], acc[RW][NC];
      int lim[RW];  // last key that the row sees
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[r][c] = 0.f;
        const int tok = (wr * RW + r) / p.G;
        lim[r] = p.causal ? rc.pos0 + tok : 0x7fffffff;
      }
      const float* q0 = s_q + wr * RW * pitch;
      const int key0 = wk * 32 * KPL;  // the warp's first key of a tile; the lane's: key0 + 32 k + lane
      for (int t = pc.a; t < pc.b; ++t) {
        const int pg_next = t + 2 < pc.b ? page_of(t + 2) : -1;
        cp_async_wait<1>();
        __syncthreads();  // K of this tile is in
        const float* kr = s_k + (key0 + lane) * pitch;
        float sa[KPL][RW], sb[KPL][RW];  // sums of the even and the odd products
#pragma unroll
        for (int k = 0; k < KPL; ++k)
#pragma unroll
          for (int r = 0; r < RW; ++r) sa[k][r] = sb[k][r] = 0.f;
        for (int c = 0; c < 4 * dv; c += 4) {
          float4 kv[KPL];
#pragma unroll
          for (int k = 0; k < KPL; ++k) kv[k] = *reinterpret_cast<const float4*>(kr + 32 * k * pitch + c);
#pragma unroll
          for (int r = 0; r < RW; ++r) {
            const float4 qv = *reinterpret_cast<const float4*>(q0 + r * pitch + c);
#pragma unroll
            for (int k = 0; k < KPL; ++k) {
              ffma2(sa[k][r], sb[k][r], qv.x, qv.y, kv[k].x, kv[k].y, sa[k][r], sb[k][r]);
              ffma2(sa[k][r], sb[k][r], qv.z, qv.w, kv[k].z, kv[k].w, sa[k][r], sb[k][r]);
            }
          }
        }
        bool there[KPL];
#pragma unroll
        for (int k = 0; k < KPL; ++k) there[k] = s_off[t % 3 * 2 * KT + key0 + 32 * k + lane] >= 0;
        const int j = t * KT + key0 + lane;
#pragma unroll
        for (int r = 0; r < RW; ++r) {
          float top = -INFINITY;
#pragma unroll
          for (int k = 0; k < KPL; ++k) {
            sa[k][r] = (there[k] && j + 32 * k <= lim[r]) ? (sa[k][r] + sb[k][r]) * p.scale2 : -INFINITY;
            top = fmaxf(top, sa[k][r]);
          }
          if (__any_sync(0xffffffffu, top > m[r] + 8.0f)) {
            float mn = fmaxf(m[r], top);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
            const float a = exp2f(m[r] - mn);
            l[r] *= a;
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[r][c] *= a;
            m[r] = mn;
          }
#pragma unroll
          for (int k = 0; k < KPL; ++k) {
            sa[k][r] = sa[k][r] == -INFINITY ? 0.f : exp2f(sa[k][r] - m[r]);
            l[r] += sa[k][r];
          }
        }
#pragma unroll
        for (int k = 0; k < KPL; ++k)
#pragma unroll
          for (int r = 0; r < RW; r += 4)
            *reinterpret_cast<float4*>(my_p + (32 * k + lane) * RW + r) =
                make_float4(sa[k][r], sa[k][r + 1], sa[k][r + 2], sa[k][r + 3]);
        if (t + 2 < pc.b) note(t + 2, pg_next);
        __syncthreads();  // K read, P written
        if (t + 1 < pc.b) load_k(t + 1);
        else cp_async_commit();
        cp_async_wait<1>();
        __syncthreads();  // V of this tile is in
        const float* vr = s_v + key0 * pitch + lane;
#pragma unroll 4
        for (int kk = 0; kk < 32 * KPL; ++kk) {
          float vv[NC];
#pragma unroll
          for (int c = 0; c < NC; ++c) vv[c] = 32 * c + lane < 4 * dv ? vr[kk * pitch + 32 * c] : 0.f;
#pragma unroll
          for (int r = 0; r < RW; r += 4) {
            const float4 pr = *reinterpret_cast<const float4*>(my_p + kk * RW + r);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              acc[r][c] = fmaf(pr.x, vv[c], acc[r][c]);
              acc[r + 1][c] = fmaf(pr.y, vv[c], acc[r + 1][c]);
              acc[r + 2][c] = fmaf(pr.z, vv[c], acc[r + 2][c]);
              acc[r + 3][c] = fmaf(pr.w, vv[c], acc[r + 3][c]);
            }
          }
        }
        __syncthreads();  // V and P read
        if (t + 1 < pc.b) load_v(t + 1);
        else cp_async_commit();
      }
      cp_async_wait<0>();
#pragma unroll
      for (int r = 0; r < RW; ++r)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);

      const bool whole = pc.a == 0 && pc.b == rc.n;
      const size_t slot = paged_slot(cta, pc);
      auto write = [&](int r, float mm, float ll, const float (&o)[NC]) {
        const int qh = paged_row_head(p, pc.h, r, rows);
        if (qh < 0) return;
        const float f = !whole ? 1.0f : (ll == 0.f ? 0.0f : 1.0f / ll);
        const long long row = static_cast<long long>(rc.tok0 + r / p.G) * p.H + qh;
        float* op = whole ? static_cast<float*>(p.o) + row * d : p.ws_o + (slot * p.rows_cap + r) * p.ws_pitch;
#pragma unroll
        for (int c = 0; c < NC; ++c)
          if (32 * c + lane < d) op[32 * c + lane] = o[c] * f;
        if (lane == 0) {
          if (whole) p.lse[row] = paged_lse(mm, ll);
          else p.ws_ml[slot * p.rows_cap + r] = make_float2(mm, ll);
        }
      };
      if constexpr (WK == 1) {
#pragma unroll
        for (int r = 0; r < RW; ++r) write(wr * RW + r, m[r], l[r], acc[r]);
      } else {
        // join the key groups: their sums through the K tile's memory, statistics through P's
        float2* s_ml = reinterpret_cast<float2*>(s_p);  // [warps][RW]
        if (lane == 0)
          for (int r = 0; r < RW; ++r) s_ml[warp * RW + r] = make_float2(m[r], l[r]);
        __syncthreads();
#pragma unroll
        for (int r = 0; r < RW; ++r) {
          float mm = -INFINITY;
          for (int w = 0; w < WK; ++w) mm = fmaxf(mm, s_ml[(wr * WK + w) * RW + r].x);
          const float a = m[r] == -INFINITY ? 0.f : exp2f(m[r] - mm);
#pragma unroll
          for (int c = 0; c < NC; ++c)  // never the padding columns, which stay zero
            if (32 * c + lane < d) s_k[(warp * RW + r) * pitch + 32 * c + lane] = acc[r][c] * a;
        }
        __syncthreads();
        for (int r = warp; r < R; r += L::WARPS) {
          const int first = r / RW * WK, in = r % RW;  // the row's warps, its row in them
          float mm = -INFINITY, ll = 0.f, o[NC];
          for (int w = 0; w < WK; ++w) mm = fmaxf(mm, s_ml[(first + w) * RW + in].x);
#pragma unroll
          for (int c = 0; c < NC; ++c) o[c] = 0.f;
          for (int w = 0; w < WK; ++w) {
            const float2 ml = s_ml[(first + w) * RW + in];
            if (ml.x != -INFINITY) ll = fmaf(ml.y, exp2f(ml.x - mm), ll);
#pragma unroll
            for (int c = 0; c < NC; ++c)
              if (32 * c + lane < d) o[c] += s_k[((first + w) * RW + in) * pitch + 32 * c + lane];
          }
          write(r, mm, ll, o);
        }
      }
      if (tid == 0 && pc.a == 0 && pc.b < rc.n) paged_header<C>(p, sched, rc, pc.h, cta);
    }
    x = sched.stop;
    if (x >= hi) break;
    __syncthreads();  // the list is rewritten
    paged_list<KT, C, NT>(p, tpt, x, hi, nullptr, sched);
  }
}

}  // namespace fa
