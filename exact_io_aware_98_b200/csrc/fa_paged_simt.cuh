// fa_paged_simt.cuh -- paged attention on CUDA cores: fp32 inputs, fp32 products and sums.
//
// Two kernels, both with K and V tiles by 16-byte asynchronous copies (the K tile of step t+1 while
// P V of step t runs, the V tile while the scores are formed), the page of a key looked up two
// tiles ahead, and a reference maximum per row that moves only when a score exceeds it by more
// than 8 (in log2 units), which one vote finds; so most tiles need no reduction over lanes.  K and V
// rows are padded to an odd number of 16-byte chunks, which spreads reads of neighbouring rows at
// one column over all banks.
//   fa_paged_f32_few_kernel (8 rows, 128 keys a tile, 8 warps): few rows per K/V head (decoding).
//     Warps in 2 row groups x 4 key groups, 4 rows and 32 keys each; lane = key for the scores, for
//     P V a lane has the columns lane, lane + 32, ..  Bound by latency: with one K and one V tile a
//     copy starts only when the phase that reads its buffer is over, and with fewer than 5 rows the
//     second row group works on none.  16 requests of 8192 keys, 8 heads over 2, d 128: 100 us, 2.7
//     TB/s of a copy's 6.5.
//   fa_paged_f32_chunk_kernel (64 rows, 64 keys a tile, 256 threads): a thread forms 4 rows x 4 keys
//     of scores and 4 rows x 2 NC columns of O (in pairs: one 8-byte read of V, packed FMAs), so
//     that a value read from shared memory enters four products.  512 tokens over 8192 keys, 16
//     heads over 4, d 128: 1.00 ms, 33 TFLOP/s (single columns 16 apart: 1.07 ms; a lane per key
//     with Q broadcast, 32 rows a tile: 1.16 ms).  Neither FFMA (35 % of its slots) nor shared
//     memory (57 %) is full: with one or two blocks per SM, latencies between the phases of a tile
//     remain; unrolling the score loop or leaving its packed FMA out changed nothing.
#pragma once
#include "fa_paged.cuh"

namespace fa {

// row pitch in floats of a d-column tile in shared memory
__host__ __device__ inline int paged_f32_pitch(int d) { return (((d + 3) / 4) | 1) * 4; }

struct PagedF32Few {
  static constexpr int WARPS = 8, THREADS = 256;
  static constexpr int WK = 4, RW = 4;              // key groups, rows of a warp
  static constexpr int R = 8, KT = 128;
  static constexpr int C = 1;                       // an item's constant, in key tiles
  // Q [R], K [KT], V [KT] rows, P [8 warps][32 keys][4 rows], offsets of the keys' rows in k and v
  // [3 tiles][2][KT]; the K tile later holds the warps' sums, P their statistics
  static size_t bytes(int d) {
    return (static_cast<size_t>(R + 2 * KT) * paged_f32_pitch(d) + WARPS * 32 * RW) * 4 + 6 * KT * 8 +
           sizeof(PagedSched);
  }
  // CTAs per SM that registers are kept for; nc: 32-column groups of the head
  __host__ __device__ static constexpr int ctas(int nc) { return nc > 2 ? 1 : 2; }
};

struct PagedF32Chunk {
  static constexpr int THREADS = 256;
  static constexpr int R = 64, KT = 64;
  static constexpr int C = 1;
  static constexpr int P_PITCH = R + 4;             // floats per key of P
  // Q [R], K [KT], V [KT] rows, P [KT][P_PITCH], offsets as above
  static size_t bytes(int d) {
    return (static_cast<size_t>(R + 2 * KT) * paged_f32_pitch(d) + KT * P_PITCH) * 4 + 6 * KT * 8 +
           sizeof(PagedSched);
  }
  __host__ __device__ static constexpr int ctas(int nc) { return nc > 3 ? 1 : 2; }
};

__device__ __forceinline__ void cp_async16(void* smem, const void* g) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(g) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The K and V tiles of one piece: where their rows lie, and their copies.  One per piece; every thread
// of the block (NT) takes part.
template <int NT, int KT>
struct PagedF32Tiles {
  const PagedParams& p;
  long long* s_off;    // [3][2][KT]
  float *s_k, *s_v;
  const int32_t* table;
  long long hrow;      // row of the head in a page
  int keys;            // that any row of the piece can see
  int pitch, per_row;  // 16-byte chunks (or elements) of a row
  int r0, c0, dr, dc;  // this thread's first one, and the step to its next

  // key threadIdx.x of tile t: its page (-1: no such key, or the table does not name one) ...
  __device__ __forceinline__ int page_of(int t) const {
    const int j = t * KT + static_cast<int>(threadIdx.x);
    if (threadIdx.x >= KT || j >= keys) return -1;
    return table[j >> p.page_shift];
  }
  // ... and, noted for the copies, where its rows start in k and v, or -1
  __device__ __forceinline__ void note(int t, int pg) const {
    const int tid = threadIdx.x;
    if (tid >= KT) return;
    const bool there = pg >= 0 && pg < p.num_pages;
    const long long row = (hrow + ((t * KT + tid) & ((1 << p.page_shift) - 1))) * p.d;
    s_off[t % 3 * 2 * KT + tid] = there ? pg * p.k_page + row : -1;
    s_off[t % 3 * 2 * KT + KT + tid] = there ? pg * p.v_page + row : -1;
  }
  __device__ __forceinline__ bool there(int t, int key) const { return s_off[t % 3 * 2 * KT + key] >= 0; }
  // missing keys become zero rows: a stale row may hold anything, and 0 times it is not 0
  __device__ __forceinline__ void load(float* dst, const void* base, const long long* off) const {
    const float* g = static_cast<const float*>(base);
    for (int r = r0, c = c0; r < KT;) {
      const long long o = off[r];
      if (p.vec) {
        if (o >= 0) cp_async16(dst + r * pitch + 4 * c, g + o + 4 * c);
        else *reinterpret_cast<float4*>(dst + r * pitch + 4 * c) = make_float4(0.f, 0.f, 0.f, 0.f);
      } else {
        dst[r * pitch + c] = o >= 0 ? g[o + c] : 0.f;
      }
      r += dr;
      c += dc;
      if (c >= per_row) {
        c -= per_row;
        ++r;
      }
    }
    cp_async_commit();
  }
  __device__ __forceinline__ void load_k(int t) const { load(s_k, p.k, s_off + t % 3 * 2 * KT); }
  __device__ __forceinline__ void load_v(int t) const { load(s_v, p.v, s_off + t % 3 * 2 * KT + KT); }
};

// NC: 32-column groups of the head dimension.
template <int NC>
__global__ void __launch_bounds__(PagedF32Few::THREADS, PagedF32Few::ctas(NC))
fa_paged_f32_few_kernel(const PagedParams p) {
  using L = PagedF32Few;
  constexpr int R = L::R, KT = L::KT, C = L::C, NT = L::THREADS, WK = L::WK, RW = L::RW;
  extern __shared__ __align__(16) uint8_t smem_simt[];
  const int d = p.d, pitch = paged_f32_pitch(d), dv = (d + 3) / 4;
  float* s_q = reinterpret_cast<float*>(smem_simt);
  float* s_k = s_q + R * pitch;
  float* s_v = s_k + KT * pitch;
  float* s_p = s_v + KT * pitch;
  long long* s_off = reinterpret_cast<long long*>(s_p + L::WARPS * 32 * RW);
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
  float* my_p = s_p + warp * 32 * RW;
  const int per_row = p.vec ? dv : d;

  paged_list<KT, C, NT>(p, tpt, x, hi, &mine, sched);
  while (true) {
    PagedPieces<C> pieces;
    pieces.start(p, sched, x);
    PagedPiece pc;
    while (pieces.next(p, sched, pc)) {
      const PagedRec rc = sched.rec[pc.rec];
      const int rows = rc.ntok * p.G;
      const PagedF32Tiles<NT, KT> tiles = {p, s_off, s_k, s_v, p.table + rc.b * p.table_stride,
                                           static_cast<long long>(pc.h / p.splits) << p.page_shift,
                                           paged_keys(p.causal, rc.kv, rc.pos0, rc.ntok), pitch, per_row,
                                           tid / per_row, tid % per_row, NT / per_row, NT % per_row};
      __syncthreads();  // the previous piece's reads of every shared array are over
      for (int e = tid; e < R * d; e += NT) {
        const int r = e / d, c = e - r * d;
        const long long tok = rc.tok0 + r / p.G;
        const int qh = paged_row_head(p, pc.h, r, rows);
        s_q[r * pitch + c] =
            qh >= 0 ? static_cast<const float*>(p.q)[tok * p.q_st + qh * p.q_sh + c] : 0.f;
      }
      tiles.note(pc.a, tiles.page_of(pc.a));
      if (pc.a + 1 < pc.b) tiles.note(pc.a + 1, tiles.page_of(pc.a + 1));
      __syncthreads();
      tiles.load_k(pc.a);
      tiles.load_v(pc.a);

      float m[RW], l[RW], acc[RW][NC];
      int lim[RW];  // last key that the row sees
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[r][c] = 0.f;
        lim[r] = p.causal ? rc.pos0 + (wr * RW + r) / p.G : 0x7fffffff;
      }
      const float* q0 = s_q + wr * RW * pitch;
      const int key0 = wk * 32;  // the warp's first key of a tile; the lane's: key0 + lane
      for (int t = pc.a; t < pc.b; ++t) {
        const int pg_next = t + 2 < pc.b ? tiles.page_of(t + 2) : -1;
        cp_async_wait<1>();
        __syncthreads();  // K of this tile is in
        const float* kr = s_k + (key0 + lane) * pitch;
        float sa[RW], sb[RW];  // sums of the even and the odd products
#pragma unroll
        for (int r = 0; r < RW; ++r) sa[r] = sb[r] = 0.f;
        for (int c = 0; c < 4 * dv; c += 4) {
          const float4 kv = *reinterpret_cast<const float4*>(kr + c);
#pragma unroll
          for (int r = 0; r < RW; ++r) {
            const float4 qv = *reinterpret_cast<const float4*>(q0 + r * pitch + c);
            ffma2(sa[r], sb[r], qv.x, qv.y, kv.x, kv.y, sa[r], sb[r]);
            ffma2(sa[r], sb[r], qv.z, qv.w, kv.z, kv.w, sa[r], sb[r]);
          }
        }
        const bool there = tiles.there(t, key0 + lane);
        const int j = t * KT + key0 + lane;
#pragma unroll
        for (int r = 0; r < RW; ++r) {
          const float v = (there && j <= lim[r]) ? (sa[r] + sb[r]) * p.scale2 : -INFINITY;
          if (__any_sync(0xffffffffu, v > m[r] + 8.0f)) {
            float mn = fmaxf(m[r], v);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
            const float a = exp2f(m[r] - mn);
            l[r] *= a;
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[r][c] *= a;
            m[r] = mn;
          }
          sa[r] = v == -INFINITY ? 0.f : exp2f(v - m[r]);
          l[r] += sa[r];
        }
        *reinterpret_cast<float4*>(my_p + lane * RW) = make_float4(sa[0], sa[1], sa[2], sa[3]);
        if (t + 2 < pc.b) tiles.note(t + 2, pg_next);
        __syncthreads();  // K read, P written
        if (t + 1 < pc.b) tiles.load_k(t + 1);
        else cp_async_commit();
        cp_async_wait<1>();
        __syncthreads();  // V of this tile is in
        const float* vr = s_v + key0 * pitch + lane;
#pragma unroll 4
        for (int kk = 0; kk < 32; ++kk) {
          float vv[NC];
#pragma unroll
          for (int c = 0; c < NC; ++c) vv[c] = 32 * c + lane < 4 * dv ? vr[kk * pitch + 32 * c] : 0.f;
          const float4 pr = *reinterpret_cast<const float4*>(my_p + kk * RW);
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            acc[0][c] = fmaf(pr.x, vv[c], acc[0][c]);
            acc[1][c] = fmaf(pr.y, vv[c], acc[1][c]);
            acc[2][c] = fmaf(pr.z, vv[c], acc[2][c]);
            acc[3][c] = fmaf(pr.w, vv[c], acc[3][c]);
          }
        }
        __syncthreads();  // V and P read
        if (t + 1 < pc.b) tiles.load_v(t + 1);
        else cp_async_commit();
      }
      cp_async_wait<0>();
#pragma unroll
      for (int r = 0; r < RW; ++r)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);

      const bool whole = pc.a == 0 && pc.b == rc.n;
      // join the key groups: their sums through the K tile's memory, statistics through P's
      float2* s_ml = reinterpret_cast<float2*>(s_p);  // [warps][RW]
      if (lane == 0)
        for (int r = 0; r < RW; ++r) s_ml[warp * RW + r] = make_float2(m[r], l[r]);
      __syncthreads();
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        float mm = -INFINITY;
        for (int w = 0; w < WK; ++w) mm = fmaxf(mm, s_ml[(wr * WK + w) * RW + r].x);
        const float a = exp2f(m[r] - mm);
#pragma unroll
        for (int c = 0; c < NC; ++c)  // never the padding columns, which stay zero
          if (32 * c + lane < d)
            s_k[(warp * RW + r) * pitch + 32 * c + lane] = l[r] == 0.f ? 0.f : acc[r][c] * a;
      }
      __syncthreads();
      {
        const int r = warp;                             // one row per warp
        const int first = r / RW * WK, in = r % RW;     // the row's warps, its row in them
        const int qh = paged_row_head(p, pc.h, r, rows);
        if (qh >= 0) {
          const size_t slot = paged_slot(cta, pc);
          float mm = -INFINITY, ll = 0.f, o[NC];
          for (int w = 0; w < WK; ++w) mm = fmaxf(mm, s_ml[(first + w) * RW + in].x);
#pragma unroll
          for (int c = 0; c < NC; ++c) o[c] = 0.f;
          for (int w = 0; w < WK; ++w) {
            const float2 ml = s_ml[(first + w) * RW + in];
            if (ml.y != 0.f) ll = fmaf(ml.y, exp2f(ml.x - mm), ll);
#pragma unroll
            for (int c = 0; c < NC; ++c)
              if (32 * c + lane < d) o[c] += s_k[((first + w) * RW + in) * pitch + 32 * c + lane];
          }
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
        }
      }
      if (tid == 0 && !whole) paged_header<C>(p, sched, rc, pc, cta);
    }
    x = sched.stop;
    if (x >= hi) break;
    __syncthreads();  // the list is rewritten
    paged_list<KT, C, NT>(p, tpt, x, hi, nullptr, sched);
  }
}

// NC: 32-column groups of the head dimension; a thread has 2 NC columns of O.
template <int NC>
__global__ void __launch_bounds__(PagedF32Chunk::THREADS, PagedF32Chunk::ctas(NC))
fa_paged_f32_chunk_kernel(const PagedParams p) {
  using L = PagedF32Chunk;
  constexpr int R = L::R, KT = L::KT, C = L::C, NT = L::THREADS, CO = 2 * NC;
  extern __shared__ __align__(16) uint8_t smem_simt[];
  const int d = p.d, pitch = paged_f32_pitch(d), dv = (d + 3) / 4;
  float* s_q = reinterpret_cast<float*>(smem_simt);
  float* s_k = s_q + R * pitch;
  float* s_v = s_k + KT * pitch;
  float* s_p = s_v + KT * pitch;  // [key][row]; behind V, whose last row is read up to 32 NC columns
  long long* s_off = reinterpret_cast<long long*>(s_p + KT * L::P_PITCH);
  PagedSched& sched = *reinterpret_cast<PagedSched*>(s_off + 6 * KT);
  const int tid = threadIdx.x;
  const int tx = tid & 15, ty = tid >> 4;  // keys tx + 16 k, columns 32 c + 2 tx and the next; rows 4 ty + i
  const int tpt = R / p.G;  // G <= R

  // zero the columns that pad d up to a multiple of 4 (read by the 16-byte accesses)
  for (int e = tid; e < (R + 2 * KT) * pitch; e += NT) s_q[e] = 0.f;
  grid_dep_wait();  // launched to overlap the kernel before
  grid_dep_launch();
  const int cta = blockIdx.x;
  long long x, hi;
  PagedMine mine = {};
  if (!paged_share<KT, C, NT>(p, tpt, sched, x, hi, mine)) return;
  const int per_row = p.vec ? dv : d;

  paged_list<KT, C, NT>(p, tpt, x, hi, &mine, sched);
  while (true) {
    PagedPieces<C> pieces;
    pieces.start(p, sched, x);
    PagedPiece pc;
    while (pieces.next(p, sched, pc)) {
      const PagedRec rc = sched.rec[pc.rec];
      const int rows = rc.ntok * p.G;
      const PagedF32Tiles<NT, KT> tiles = {p, s_off, s_k, s_v, p.table + rc.b * p.table_stride,
                                           static_cast<long long>(pc.h / p.splits) << p.page_shift,
                                           paged_keys(p.causal, rc.kv, rc.pos0, rc.ntok), pitch, per_row,
                                           tid / per_row, tid % per_row, NT / per_row, NT % per_row};
      __syncthreads();  // the previous piece's reads of every shared array are over
      for (int e = tid; e < R * d; e += NT) {
        const int r = e / d, c = e - r * d;
        const long long tok = rc.tok0 + r / p.G;
        const int qh = paged_row_head(p, pc.h, r, rows);
        s_q[r * pitch + c] =
            qh >= 0 ? static_cast<const float*>(p.q)[tok * p.q_st + qh * p.q_sh + c] : 0.f;
      }
      tiles.note(pc.a, tiles.page_of(pc.a));
      if (pc.a + 1 < pc.b) tiles.note(pc.a + 1, tiles.page_of(pc.a + 1));
      __syncthreads();
      tiles.load_k(pc.a);
      tiles.load_v(pc.a);

      float m[4], l[4], acc[4][CO];
      int lim[4];  // last key that the row sees
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < CO; ++c) acc[i][c] = 0.f;
        lim[i] = p.causal ? rc.pos0 + (4 * ty + i) / p.G : 0x7fffffff;
      }
      for (int t = pc.a; t < pc.b; ++t) {
        const int pg_next = t + 2 < pc.b ? tiles.page_of(t + 2) : -1;
        cp_async_wait<1>();
        __syncthreads();  // K of this tile is in
        float sa[4][4], sb[4][4];  // [row][key]: sums of the even and the odd products
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) sa[i][k] = sb[i][k] = 0.f;
        for (int c = 0; c < 4 * dv; c += 4) {
          float4 kv[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            kv[k] = *reinterpret_cast<const float4*>(s_k + (tx + 16 * k) * pitch + c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 qv = *reinterpret_cast<const float4*>(s_q + (4 * ty + i) * pitch + c);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              ffma2(sa[i][k], sb[i][k], qv.x, qv.y, kv[k].x, kv[k].y, sa[i][k], sb[i][k]);
              ffma2(sa[i][k], sb[i][k], qv.z, qv.w, kv[k].z, kv[k].w, sa[i][k], sb[i][k]);
            }
          }
        }
        bool there[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) there[k] = tiles.there(t, tx + 16 * k);
        const int j = t * KT + tx;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float top = -INFINITY;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            sa[i][k] = (there[k] && j + 16 * k <= lim[i]) ? (sa[i][k] + sb[i][k]) * p.scale2 : -INFINITY;
            top = fmaxf(top, sa[i][k]);
          }
          if (__any_sync(0xffffffffu, top > m[i] + 8.0f)) {  // in either of the warp's two rows
            float mn = fmaxf(m[i], top);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
            const float a = m[i] == mn ? 1.0f : exp2f(m[i] - mn);
            l[i] *= a;
#pragma unroll
            for (int c = 0; c < CO; ++c) acc[i][c] *= a;
            m[i] = mn;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            sa[i][k] = sa[i][k] == -INFINITY ? 0.f : exp2f(sa[i][k] - m[i]);
            l[i] += sa[i][k];
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<float4*>(s_p + (tx + 16 * k) * L::P_PITCH + 4 * ty) =
              make_float4(sa[0][k], sa[1][k], sa[2][k], sa[3][k]);
        if (t + 2 < pc.b) tiles.note(t + 2, pg_next);
        __syncthreads();  // K read, P written
        if (t + 1 < pc.b) tiles.load_k(t + 1);
        else cp_async_commit();
        cp_async_wait<1>();
        __syncthreads();  // V of this tile is in
#pragma unroll 4
        for (int kk = 0; kk < KT; ++kk) {
          const float4 pr = *reinterpret_cast<const float4*>(s_p + kk * L::P_PITCH + 4 * ty);
          const float* vr = s_v + kk * pitch + 2 * tx;  // columns from d on: other values, never written out
#pragma unroll
          for (int c = 0; c < CO; c += 2) {
            const float2 v = *reinterpret_cast<const float2*>(vr + 16 * c);
            const float pi[4] = {pr.x, pr.y, pr.z, pr.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              ffma2(acc[i][c], acc[i][c + 1], pi[i], pi[i], v.x, v.y, acc[i][c], acc[i][c + 1]);
            }
          }
        }
        __syncthreads();  // V and P read
        if (t + 1 < pc.b) tiles.load_v(t + 1);
        else cp_async_commit();
      }
      cp_async_wait<0>();
      const bool whole = pc.a == 0 && pc.b == rc.n;
      const size_t slot = paged_slot(cta, pc);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
        const int r = 4 * ty + i;
        const int qh = paged_row_head(p, pc.h, r, rows);
        if (qh < 0) continue;
        const float f = !whole ? 1.0f : (l[i] == 0.f ? 0.0f : 1.0f / l[i]);
        const long long row = static_cast<long long>(rc.tok0 + r / p.G) * p.H + qh;
        float* op = whole ? static_cast<float*>(p.o) + row * d : p.ws_o + (slot * p.rows_cap + r) * p.ws_pitch;
#pragma unroll
        for (int c = 0; c < CO; ++c) {
          const int col = 16 * (c & ~1) + 2 * tx + (c & 1);
          if (col < d) op[col] = l[i] == 0.f ? 0.f : acc[i][c] * f;
        }
        if (tx == 0) {
          if (whole) p.lse[row] = paged_lse(m[i], l[i]);
          else p.ws_ml[slot * p.rows_cap + r] = make_float2(m[i], l[i]);
        }
      }
      if (tid == 0 && !whole) paged_header<C>(p, sched, rc, pc, cta);
    }
    x = sched.stop;
    if (x >= hi) break;
    __syncthreads();  // the list is rewritten
    paged_list<KT, C, NT>(p, tpt, x, hi, nullptr, sched);
  }
}

}  // namespace fa
