// fa_paged.cuh -- what the paged-attention kernels share: their parameters, the division of a
// ragged batch over the CTAs, and the kernel that joins partial results.
//
// The work.  Request b brings nq = cu_q[b+1] - cu_q[b] new tokens, the last of its kv_len[b]
// cached positions.  Token i of it sees the keys j < kv_len with, under a causal mask,
// j <= kv_len - nq + i.  The G = H / H_kv query heads that share a K/V head are rows of one
// tile: row r of a row tile is token r / G and head r % G, so that a tile of R rows holds
// R / G tokens (rounded down) and reads each key once for all of them.  A group of more than R
// heads is dealt out over several tiles of G <= R heads, each a K/V head of its own here
// ("tile head": H_kv * splits of them).
//
// The division.  An item is one (row tile, K/V head); its cost is the number n of key tiles its
// rows can see (at least 1, so that a row with no key gets its O = 0 and lse = -inf).  The items
// of the batch laid end to end form a line of W key tiles, which is cut into equal shares, one
// per CTA.  So a batch of any mix of lengths loads all SMs alike, a single long request is
// spread over all of them, and every CTA has at most one item that it continues for the CTA
// before it and at most one that it leaves unfinished.  Those two pieces go to the workspace as
// unnormalised fp32 sums with their row maximum and row sum; fa_paged_join_kernel adds them in
// the order of the keys.  Every other item is finished where it was computed.  The division
// depends on the lengths only, so results do not vary between runs.  Each CTA computes it from
// the lengths on its own: no host copy of the lengths, no extra launch, and a captured call
// follows lengths that change on the device.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "fa_paged_cache.cuh"
#include "fa_simt.cuh"
#include "ptx.cuh"

namespace fa {

struct PagedParams {
  const void *q, *k, *v;  // k, v: caches
  void* o;                // [T][H][d]
  float* lse;             // [T][H]
  const int32_t *table, *kv_len, *cu_q;
  long long table_stride;
  long long q_st, q_sh;        // q's token and head strides in elements
  long long k_page, v_page;    // page strides of the caches in elements
  int T, B, H, d;
  int group;                   // query heads per K/V head
  int G, splits;               // heads per tile, tiles per group (ceil(group / G))
  int Hv;                      // tile heads: H_kv * splits
  int vec;                     // rows and strides allow 16-byte copies
  int page_shift, num_pages, max_pages;
  int causal;
  float scale2;                // scale * log2(e)
  // workspace: headers [ctas], row statistics [ctas][2][rows_cap], sums [ctas][2][rows_cap][pitch]
  int4* ws_head;
  float2* ws_ml;
  float* ws_o;
  int rows_cap, ws_pitch;      // rows per part; floats per row (d rounded up to 4)
};

// One row tile of a request, as the CTAs pass it around.
struct PagedRec {
  long long lin;  // where its items start on the line of key tiles
  int b;          // request
  int tok0, ntok; // first row of q, number of tokens
  int pos0;       // cached position of the first token (negative: before the cache's start)
  int kv;         // cached keys of the request
  int n;          // key tiles of each of its Hv items (>= 1)
};

constexpr int PAGED_RECS = 32;  // row tiles a CTA lists at a time

struct PagedSched {
  long long tmp[33];
  PagedRec rec[PAGED_RECS];
  int n_rec;
  long long stop;  // end of the listed part of the CTA's share
};

// Row r of a tile of tile head h: its token within the tile and its query head (-1: the tile has
// no such row, or its group has no such head).
__device__ __forceinline__ int paged_row_head(const PagedParams& p, int h, int r, int rows) {
  const int kv = h / p.splits;
  const int i = (h - kv * p.splits) * p.G + r % p.G;
  return r < rows && i < p.group ? kv * p.group + i : -1;
}

struct PagedReq {
  int tok0, nq, kv, tiles_per;  // tiles_per: tokens per row tile
};

__device__ __forceinline__ PagedReq paged_req(const PagedParams& p, int b, int tpt) {
  PagedReq r;
  const int lo = min(max(p.cu_q[b], 0), p.T), hi = min(max(p.cu_q[b + 1], 0), p.T);
  const long long room = static_cast<long long>(p.max_pages) << p.page_shift;
  r.tok0 = lo;
  r.nq = max(hi - lo, 0);
  r.kv = static_cast<int>(min(static_cast<long long>(max(p.kv_len[b], 0)), room));
  r.tiles_per = tpt;
  return r;
}

// Keys that the tokens [t tpt, t tpt + ntok) of a request can see between them.
__device__ __forceinline__ int paged_keys(int causal, int kv, int pos0, int ntok) {
  if (!causal) return kv;
  const long long last = static_cast<long long>(pos0) + ntok;  // one past the last token
  return static_cast<int>(min(max(last, 0ll), static_cast<long long>(kv)));
}

// Key tiles of row tile t (KT keys each, at least one).
template <int KT>
__device__ __forceinline__ int paged_tiles(int causal, const PagedReq& r, int t) {
  const int ntok = min(r.tiles_per, r.nq - t * r.tiles_per);
  const int keys = paged_keys(causal, r.kv, r.kv - r.nq + t * r.tiles_per, ntok);
  return max(1, (keys + KT - 1) / KT);
}

// Key tiles of all row tiles of a request, for one K/V head.
template <int KT>
__device__ __forceinline__ long long paged_cost(const PagedParams& p, const PagedReq& r) {
  const int nt = (r.nq + r.tiles_per - 1) / r.tiles_per;
  if (!p.causal) return static_cast<long long>(nt) * max(1, (r.kv + KT - 1) / KT);
  long long c = 0;
  for (int t = 0; t < nt; ++t) c += paged_tiles<KT>(1, r, t);
  return c;
}

// The length W of the line.  Every thread of the block (NT) calls it.
template <int KT, int NT>
__device__ long long paged_total(const PagedParams& p, int tpt, PagedSched& s) {
  long long mine = 0, all;
  for (int b = threadIdx.x; b < p.B; b += NT) mine += paged_cost<KT>(p, paged_req(p, b, tpt));
  block_excl_scan<long long, NT>(mine, s.tmp, &all);
  return all * p.Hv;
}

// Lists the row tiles that [lo, hi) of the line touches, PAGED_RECS at most, and sets s.stop to
// where the listed part ends.  Every thread of the block calls it, lo < hi.
template <int KT, int NT>
__device__ void paged_list(const PagedParams& p, int tpt, long long lo, long long hi,
                           PagedSched& s) {
  if (threadIdx.x == 0) s.stop = hi;
  long long carry = 0;
  int listed = 0;
  for (int b0 = 0; b0 < p.B && carry < hi && listed < PAGED_RECS; b0 += NT) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    PagedReq r = {0, 0, 0, 1};
    if (b < p.B) r = paged_req(p, b, tpt);
    long long sum, lin = 0;
    const long long cost = b < p.B ? paged_cost<KT>(p, r) * p.Hv : 0;
    lin = carry + block_excl_scan<long long, NT>(cost, s.tmp, &sum);
    const int nt = (r.nq + r.tiles_per - 1) / r.tiles_per;
    int count = 0;
    const bool touch = cost > 0 && lin < hi && lin + cost > lo;
    if (touch) {
      long long x = lin;
      for (int t = 0; t < nt && x < hi; ++t) {
        const long long e = x + static_cast<long long>(paged_tiles<KT>(p.causal, r, t)) * p.Hv;
        if (e > lo) ++count;
        x = e;
      }
    }
    long long all;
    long long at = listed + block_excl_scan<long long, NT>(count, s.tmp, &all);
    if (count > 0 && at < PAGED_RECS) {
      long long x = lin;
      for (int t = 0; t < nt && x < hi && at < PAGED_RECS; ++t) {
        const int n = paged_tiles<KT>(p.causal, r, t);
        const long long e = x + static_cast<long long>(n) * p.Hv;
        if (e > lo) {
          PagedRec c;
          c.lin = x;
          c.b = b;
          c.tok0 = r.tok0 + t * r.tiles_per;
          c.ntok = min(r.tiles_per, r.nq - t * r.tiles_per);
          c.pos0 = r.kv - r.nq + t * r.tiles_per;
          c.kv = r.kv;
          c.n = n;
          s.rec[at] = c;
          if (at == PAGED_RECS - 1) s.stop = min(hi, e);
          ++at;
        }
        x = e;
      }
    }
    carry += sum;
    listed = static_cast<int>(min(listed + all, static_cast<long long>(PAGED_RECS)));
  }
  if (threadIdx.x == 0) s.n_rec = listed;
  __syncthreads();
}

// One piece: key tiles [a, b) of the item (record, tile head h).
struct PagedPiece {
  int rec, h, a, b;
  long long item_end;  // end of the whole item on the line
};

// The piece that starts at x of the line; `rec` is where the search starts (records are in
// order and x only grows).
__device__ __forceinline__ PagedPiece paged_piece(const PagedParams& p, const PagedSched& s,
                                                  long long x, int rec) {
  while (rec + 1 < s.n_rec && x >= s.rec[rec + 1].lin) ++rec;
  PagedPiece c;
  const int n = s.rec[rec].n;
  const long long off = x - s.rec[rec].lin;
  c.rec = rec;
  c.h = static_cast<int>(off / n);
  c.a = static_cast<int>(off - static_cast<long long>(c.h) * n);
  c.b = static_cast<int>(min(static_cast<long long>(n), c.a + (s.stop - x)));
  c.item_end = s.rec[rec].lin + static_cast<long long>(c.h + 1) * n;
  return c;
}

// The share of CTA c of `ctas` on a line of W >= ctas tiles.
__device__ __forceinline__ long long paged_cut(long long W, long long c, long long ctas) {
  return W * c / ctas;
}

// Where a piece's partial sums go: slot 0 continues an item, slot 1 leaves one unfinished.
__device__ __forceinline__ size_t paged_slot(int cta, const PagedPiece& c) {
  return static_cast<size_t>(cta) * 2 + (c.a > 0 ? 0 : 1);
}

// Header of a CTA that leaves the item of piece c unfinished: the CTAs from this one on that
// hold its parts, and where its rows go.  {parts, tile head, first token, tokens}.
__device__ __forceinline__ int4 paged_header(const PagedSched& s, const PagedPiece& c,
                                             long long W, long long ctas, int cta) {
  const long long last = (c.item_end * ctas + W - 1) / W - 1;  // the CTA that reaches its end
  return make_int4(static_cast<int>(last - cta + 1), c.h, s.rec[c.rec].tok0, s.rec[c.rec].ntok);
}

// Natural-log log-sum-exp of a row from its maximum (log2 units) and sum; -inf without keys.
__device__ __forceinline__ float paged_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// ---------------------------------------------------------------------------------- join
// Block (c, j) joins rows of the item that CTA c left unfinished: O = sum_i 2^(m_i - m) O_i / l,
// l = sum_i 2^(m_i - m) l_i, over the parts in key order.  WPR warps share a row: they take every
// WPR-th part, eight of them loaded at once, and add their sums in warp order.  WPR = 4 where
// items have few rows and many parts (decoding: 12.2 us for the call of one request of 2000 keys,
// against 19.7 us with a part's loads waiting for the one before), 1 where they have many rows.
// Bound by the launch and three dependent loads; launched to overlap the end of the kernel before.
constexpr int JOIN_WARPS = 8;

template <typename T, int WPR>
__global__ void __launch_bounds__(JOIN_WARPS * 32) fa_paged_join_kernel(const PagedParams p) {
  __shared__ float4 s_acc[JOIN_WARPS][32];
  __shared__ float s_l[JOIN_WARPS];
  grid_dep_wait();
  const int cta = blockIdx.x;
  const int4 head = p.ws_head[cta];
  if (head.x <= 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = head.w * p.G, parts = head.x;
  const size_t first = static_cast<size_t>(cta) * 2 + 1;
  constexpr int AT_ONCE = JOIN_WARPS / WPR;
  for (int r0 = blockIdx.y * AT_ONCE; r0 < rows; r0 += gridDim.y * AT_ONCE) {
    const int r = r0 + warp / WPR;
    const int qh = paged_row_head(p, head.y, r, rows);
    // part i: slot 1 of this CTA, then slot 0 of the ones after it
    auto stats = [&](int i) { return (i == 0 ? first : first + 2 * i - 1) * p.rows_cap + r; };
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);  // columns 4 lane ..
    if (qh >= 0) {
      for (int i = lane; i < parts; i += 32) m = fmaxf(m, p.ws_ml[stats(i)].x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      constexpr int DEPTH = 8;
      for (int i0 = warp % WPR; i0 < parts; i0 += DEPTH * WPR) {
        float4 part[DEPTH];
        float2 ml[DEPTH];
#pragma unroll
        for (int k = 0; k < DEPTH; ++k) {
          const int i = i0 + k * WPR;
          if (i >= parts) continue;
          ml[k] = p.ws_ml[stats(i)];
          const float* src = p.ws_o + stats(i) * p.ws_pitch + 4 * lane;
          part[k] = 4 * lane < p.d ? *reinterpret_cast<const float4*>(src) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int k = 0; k < DEPTH; ++k) {
          if (i0 + k * WPR >= parts || ml[k].x == -INFINITY) continue;
          const float w = exp2f(ml[k].x - m);
          l = fmaf(w, ml[k].y, l);
          acc.x = fmaf(w, part[k].x, acc.x);
          acc.y = fmaf(w, part[k].y, acc.y);
          acc.z = fmaf(w, part[k].z, acc.z);
          acc.w = fmaf(w, part[k].w, acc.w);
        }
      }
    }
    if constexpr (WPR > 1) {
      s_acc[warp][lane] = acc;
      if (lane == 0) s_l[warp] = l;
      __syncthreads();
      if (warp % WPR == 0) {
#pragma unroll
        for (int w = 1; w < WPR; ++w) {
          const float4 a = s_acc[warp + w][lane];
          acc.x += a.x;
          acc.y += a.y;
          acc.z += a.z;
          acc.w += a.w;
          l += s_l[warp + w];
        }
      }
      __syncthreads();  // s_acc is rewritten for the next rows
    }
    if (qh >= 0 && warp % WPR == 0) {
      const long long row = static_cast<long long>(head.z + r / p.G) * p.H + qh;
      const float inv = l == 0.f ? 0.f : 1.0f / l;
      T* op = static_cast<T*>(p.o) + row * p.d + 4 * lane;
      const float o[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (4 * lane + c < p.d) op[c] = from_f<T>(o[c]);
      if (lane == 0) p.lse[row] = paged_lse(m, l);
    }
  }
}

}  // namespace fa
