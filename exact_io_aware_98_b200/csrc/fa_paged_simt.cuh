// fa_paged_simt.cuh -- paged attention on CUDA cores: fp32 inputs, fp32 products and sums.
//
// 128 threads; warps in WR row groups x WK key groups, 8 rows and 32 keys per warp and key
// tile.  Lane = key for the scores (8 dot products per lane, Q rows broadcast from shared
// memory), lane = four columns for P V.  K and V rows are padded so that 16-byte reads of 32
// rows at one column spread over all banks.  K and V tiles come by 16-byte asynchronous copies,
// the K tile of step t+1 while P V of step t runs and the V tile while the scores are formed.
//   WR = 1, WK = 4 (8 rows, 128 keys a tile): few rows per K/V head (decoding).
//   WR = 4, WK = 1 (32 rows, 32 keys a tile): chunks; each key is read once per 32 rows, where
//   8 rows would make every SM read 64 bytes of L2 a cycle.
#pragma once
#include "fa_paged.cuh"

namespace fa {

template <int WR, int WK>
struct PagedSimtLayout {
  static constexpr int R = 8 * WR, KT = 32 * WK;
  static constexpr int C = 1;  // an item's constant, in key tiles
  // row pitch in floats of a d-column tile: an odd number of 16-byte chunks
  __host__ __device__ static int pitch(int d) { return (((d + 3) / 4) | 1) * 4; }
  // Q [R], K [KT], V [KT] rows, P [4 warps][32 keys][8 rows], row offsets 2 x [KT]; the K and V
  // tiles (KT * 2 * pitch floats) later hold the warps' sums [4][8][pitch] and statistics
  static size_t bytes(int d) {
    return (static_cast<size_t>(R + 2 * KT) * pitch(d) + 4 * 32 * 8) * 4 + 2 * KT * 8 +
           sizeof(PagedSched);
  }
};

__device__ __forceinline__ void cp_async16(void* smem, const void* g) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(g) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <typename T, int WR, int WK>
__global__ void __launch_bounds__(128) fa_paged_simt_kernel(const PagedParams p) {
  using L = PagedSimtLayout<WR, WK>;
  constexpr int R = L::R, KT = L::KT, RW = 8, C = L::C;
  static_assert(WR * WK == 4, "four warps");
  extern __shared__ __align__(16) uint8_t smem_simt[];
  const int d = p.d, pitch = L::pitch(d), dv = (d + 3) / 4;
  float* s_q = reinterpret_cast<float*>(smem_simt);
  float* s_k = s_q + R * pitch;
  float* s_v = s_k + KT * pitch;
  float* s_p = s_v + KT * pitch;                                   // [4][32][8]
  long long* s_off = reinterpret_cast<long long*>(s_p + 4 * 32 * 8);  // [2][KT]
  PagedSched& sched = *reinterpret_cast<PagedSched*>(s_off + 2 * KT);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wr = warp / WK, wk = warp % WK;
  const int tpt = R / p.G;  // G <= R

  grid_dep_launch();
  // zero the columns that pad d up to a multiple of 4 (read by the 16-byte accesses)
  for (int e = tid; e < (R + 2 * KT) * pitch; e += 128) s_q[e] = 0.f;
  const int cta = blockIdx.x;
  long long x, hi;
  if (!paged_share<KT, C, 128>(p, tpt, sched, x, hi)) return;
  float* my_p = s_p + warp * 32 * 8;

  while (x < hi) {
    paged_list<KT, C, 128>(p, tpt, x, hi, sched);
    PagedPieces<C> pieces;
    pieces.start(p, sched, x);
    PagedPiece pc;
    while (pieces.next(p, sched, pc)) {
      const PagedRec rc = sched.rec[pc.rec];
      const int rows = rc.ntok * p.G;
      const int keys = paged_keys(p.causal, rc.kv, rc.pos0, rc.ntok);
      const int32_t* table = p.table + rc.b * p.table_stride;
      const long long hrow = static_cast<long long>(pc.h / p.splits) << p.page_shift;
      // page << 32 | row within the page's heads, or -1: no such key
      auto row_offsets = [&](int t, int buf) {
        for (int e = tid; e < KT; e += 128) {
          const int j = t * KT + e;
          long long o = -1;
          if (j < keys) {
            const int pg = table[j >> p.page_shift];
            if (pg >= 0 && pg < p.num_pages)
              o = (static_cast<long long>(pg) << 32) |
                  static_cast<long long>((hrow + (j & ((1 << p.page_shift) - 1))));
          }
          s_off[buf * KT + e] = o;
        }
      };
      // missing keys become zero rows: a stale row may hold anything, and 0 times it is not 0
      auto load = [&](float* dst, const void* base, long long page_stride, int buf) {
        const long long* off = s_off + buf * KT;
        const T* g = static_cast<const T*>(base);
        if (sizeof(T) == 4 && p.vec) {
          for (int e = tid; e < KT * dv; e += 128) {
            const int r = e / dv, c = (e - r * dv) * 4;
            const long long o = off[r];
            if (o >= 0)
              cp_async16(dst + r * pitch + c, g + (o >> 32) * page_stride + (o & 0xffffffffll) * d + c);
            else
              *reinterpret_cast<float4*>(dst + r * pitch + c) = make_float4(0.f, 0.f, 0.f, 0.f);
          }
        } else {
          for (int e = tid; e < KT * d; e += 128) {
            const int r = e / d, c = e - r * d;
            const long long o = off[r];
            dst[r * pitch + c] =
                o >= 0 ? to_f<T>(g[(o >> 32) * page_stride + (o & 0xffffffffll) * d + c]) : 0.f;
          }
        }
        cp_async_commit();
      };
      __syncthreads();  // the previous piece's reads of every shared array are over
      for (int e = tid; e < R * d; e += 128) {
        const int r = e / d, c = e - r * d;
        const long long tok = rc.tok0 + r / p.G;
        const int qh = paged_row_head(p, pc.h, r, rows);
        s_q[r * pitch + c] =
            qh >= 0 ? to_f<T>(static_cast<const T*>(p.q)[tok * p.q_st + qh * p.q_sh + c]) : 0.f;
      }
      row_offsets(pc.a, pc.a & 1);
      __syncthreads();
      load(s_k, p.k, p.k_page, pc.a & 1);
      load(s_v, p.v, p.v_page, pc.a & 1);

      float m[RW], l[RW], acc[RW][4];
      int lim[RW];  // last key that the row sees
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
        acc[r][0] = acc[r][1] = acc[r][2] = acc[r][3] = 0.f;
        const int tok = (wr * RW + r) / p.G;
        lim[r] = p.causal ? rc.pos0 + tok : 0x7fffffff;
      }
      const float* q0 = s_q + wr * RW * pitch;
      for (int t = pc.a; t < pc.b; ++t) {
        const int buf = t & 1;
        cp_async_wait<1>();
        __syncthreads();  // K of this tile is in
        // ---- scores of key wk * 32 + lane
        const float* kr = s_k + (wk * 32 + lane) * pitch;
        float s[RW];
#pragma unroll
        for (int r = 0; r < RW; ++r) s[r] = 0.f;
        for (int c = 0; c < 4 * dv; c += 4) {
          const float4 kv = *reinterpret_cast<const float4*>(kr + c);
#pragma unroll
          for (int r = 0; r < RW; ++r) {
            const float4 qv = *reinterpret_cast<const float4*>(q0 + r * pitch + c);
            s[r] = fmaf(qv.x, kv.x, s[r]);
            s[r] = fmaf(qv.y, kv.y, s[r]);
            s[r] = fmaf(qv.z, kv.z, s[r]);
            s[r] = fmaf(qv.w, kv.w, s[r]);
          }
        }
        const int j = t * KT + wk * 32 + lane;
        const bool there = s_off[buf * KT + wk * 32 + lane] >= 0;
#pragma unroll
        for (int r = 0; r < RW; ++r) {
          const float v = (there && j <= lim[r]) ? s[r] * p.scale2 : -INFINITY;
          float mx = v;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          const float mn = fmaxf(m[r], mx);
          const float pe = v == -INFINITY ? 0.f : exp2f(v - mn);
          if (mn != m[r]) {  // the same for the whole warp
            const float a = exp2f(m[r] - mn);
            l[r] *= a;
            acc[r][0] *= a;
            acc[r][1] *= a;
            acc[r][2] *= a;
            acc[r][3] *= a;
            m[r] = mn;
          }
          l[r] += pe;
          my_p[lane * 8 + r] = pe;
        }
        if (t + 1 < pc.b) row_offsets(t + 1, buf ^ 1);
        __syncthreads();  // K read, P written, the next row offsets known
        if (t + 1 < pc.b) load(s_k, p.k, p.k_page, buf ^ 1);
        else cp_async_commit();
        cp_async_wait<1>();
        __syncthreads();  // V of this tile is in
        if (lane < dv) {
          const float* vr = s_v + wk * 32 * pitch + lane * 4;
#pragma unroll 4
          for (int kk = 0; kk < 32; ++kk) {
            const float4 vv = *reinterpret_cast<const float4*>(vr + kk * pitch);
            const float4 pa = *reinterpret_cast<const float4*>(my_p + kk * 8);
            const float4 pb = *reinterpret_cast<const float4*>(my_p + kk * 8 + 4);
            const float pr[8] = {pa.x, pa.y, pa.z, pa.w, pb.x, pb.y, pb.z, pb.w};
#pragma unroll
            for (int r = 0; r < RW; ++r) {
              acc[r][0] = fmaf(pr[r], vv.x, acc[r][0]);
              acc[r][1] = fmaf(pr[r], vv.y, acc[r][1]);
              acc[r][2] = fmaf(pr[r], vv.z, acc[r][2]);
              acc[r][3] = fmaf(pr[r], vv.w, acc[r][3]);
            }
          }
        }
        __syncthreads();  // V and P read
        if (t + 1 < pc.b) load(s_v, p.v, p.v_page, buf ^ 1);
        else cp_async_commit();
      }
      cp_async_wait<0>();
#pragma unroll
      for (int r = 0; r < RW; ++r)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);

      // ---- join the key groups (WK > 1) through the K tile's memory, then write
      float* s_ml = s_p;  // [4 warps][8 rows] (m, l)
      if (WK > 1) {
        if (lane == 0)
          for (int r = 0; r < RW; ++r) {
            s_ml[(warp * 8 + r) * 2] = m[r];
            s_ml[(warp * 8 + r) * 2 + 1] = l[r];
          }
        __syncthreads();
        float* so = s_k + warp * 8 * pitch;
#pragma unroll
        for (int r = 0; r < RW; ++r) {
          float mm = -INFINITY;
          for (int w = 0; w < 4; ++w) mm = fmaxf(mm, s_ml[(w * 8 + r) * 2]);
          const float a = m[r] == -INFINITY ? 0.f : exp2f(m[r] - mm);
#pragma unroll
          for (int c = 0; c < 4; ++c)  // never the padding columns, which stay zero
            if (lane * 4 + c < d) so[r * pitch + lane * 4 + c] = acc[r][c] * a;
        }
        __syncthreads();
      }
      const bool whole = pc.a == 0 && pc.b == rc.n;
      const size_t slot = paged_slot(cta, pc);
#pragma unroll
      for (int rr = 0; rr < (WK > 1 ? 2 : RW); ++rr) {
        // WK > 1: warp w finishes rows 2w, 2w+1; else each warp its own 8
        const int r = WK > 1 ? 2 * warp + rr : wr * RW + rr;
        const int qh = paged_row_head(p, pc.h, r, rows);
        if (qh < 0) continue;
        float mm, ll;
        float4 o4;
        if constexpr (WK > 1) {
          mm = -INFINITY;
          for (int w = 0; w < 4; ++w) mm = fmaxf(mm, s_ml[(w * 8 + r) * 2]);
          ll = 0.f;
          o4 = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int w = 0; w < 4; ++w) {
            const float mw = s_ml[(w * 8 + r) * 2];
            if (mw != -INFINITY) ll = fmaf(s_ml[(w * 8 + r) * 2 + 1], exp2f(mw - mm), ll);
            if (lane < dv) {
              const float4 a4 = *reinterpret_cast<const float4*>(s_k + (w * 8 + r) * pitch + lane * 4);
              o4.x += a4.x;
              o4.y += a4.y;
              o4.z += a4.z;
              o4.w += a4.w;
            }
          }
        } else {
          mm = m[rr];
          ll = l[rr];
          o4 = make_float4(acc[rr][0], acc[rr][1], acc[rr][2], acc[rr][3]);
        }
        if (whole) {
          const float inv = ll == 0.f ? 0.0f : 1.0f / ll;
          const long long row = static_cast<long long>(rc.tok0 + r / p.G) * p.H + qh;
          T* op = static_cast<T*>(p.o) + row * d;
          const float ov[4] = {o4.x, o4.y, o4.z, o4.w};
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (lane * 4 + c < d) op[lane * 4 + c] = from_f<T>(ov[c] * inv);
          if (lane == 0) p.lse[row] = paged_lse(mm, ll);
        } else {
          float* op = p.ws_o + (slot * p.rows_cap + r) * p.ws_pitch;
          const float ov[4] = {o4.x, o4.y, o4.z, o4.w};
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (lane * 4 + c < d) op[lane * 4 + c] = ov[c];
          if (lane == 0) p.ws_ml[slot * p.rows_cap + r] = make_float2(mm, ll);
        }
      }
      if (tid == 0 && pc.a == 0 && pc.b < rc.n) paged_header<C>(p, sched, rc, pc.h, cta);
    }
    x = sched.stop;
    __syncthreads();  // the list is rewritten
  }
}

}  // namespace fa
