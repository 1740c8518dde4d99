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
// rows can see (at least 1, so that a row with no key gets its O = 0 and lse = -inf) plus a
// constant for its start and its output, in units of a tile (the kernels measure it: without it,
// the CTA that gets the short items of a causal prompt's beginning finished last, at twice the
// time of the others).  The items of the batch laid end to end form a line of length W, which is
// cut into equal shares, one per CTA; an item's constant lies behind its tiles, so a cut there
// leaves the item whole.  So a batch of any mix of lengths loads all SMs alike, a single long request is
// spread over all of them, and every CTA has at most one item that it continues for the CTA
// before it and at most one that it leaves unfinished.  Those two pieces go to the workspace as
// unnormalised fp32 sums with their row maximum and row sum; a join kernel adds them in the order of
// the keys.  Every other item is finished where it was computed.  The division
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
  int vec;                     // cache rows and strides allow 16-byte copies
  int o_al32;                  // o is 32-byte aligned
  int page_shift, num_pages, max_pages;
  int causal;
  float scale2;                // scale * log2(e)
  // workspace: headers [ctas][2], row statistics [ctas][2][rows_cap], sums [ctas][2][rows_cap][pitch]
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
  long long stop;        // end of the listed part of the CTA's share
  long long W, ctas;     // the line's length, the CTAs that share it
};

// Row r of a tile of tile head h: its token within the tile and its query head (-1: the tile has
// no such row, or its group has no such head).
__device__ __forceinline__ int paged_row_head(const PagedParams& p, int h, int r, int rows) {
  const int kv = h / p.splits;
  const int i = (h - kv * p.splits) * p.G + r % p.G;
  return r < rows && i < p.group ? kv * p.group + i : -1;
}

struct PagedReq {
  int tok0, nq, kv;
};

__device__ __forceinline__ PagedReq paged_req(const PagedParams& p, int b) {
  PagedReq r;
  const int lo = min(max(p.cu_q[b], 0), p.T), hi = min(max(p.cu_q[b + 1], 0), p.T);
  r.tok0 = lo;
  r.nq = max(hi - lo, 0);
  r.kv = min(max(p.kv_len[b], 0), p.max_pages << p.page_shift);  // at most 2^30
  return r;
}

// Keys that a tile's tokens can see between them, the first at position pos0.
__device__ __forceinline__ int paged_keys(int causal, int kv, int pos0, int ntok) {
  return causal ? min(max(pos0 + ntok, 0), kv) : kv;
}

// Key tiles (of KT keys, at least one) of row tile t of a request.
template <int KT>
__device__ __forceinline__ int paged_tiles(int causal, const PagedReq& r, int tpt, int t) {
  const int keys = causal ? r.kv - r.nq + min(r.nq, (t + 1) * tpt) : r.kv;
  return (max(keys, 1) + KT - 1) / KT;
}

// sum of (a j + b) / m (rounded down) over j in [0, n), a, b >= 0: the lattice points under a line, by
// the Euclidean recursion of floor sums (Graham, Knuth, Patashnik, Concrete Mathematics, section
// 3.5): take the whole parts of a / m and b / m out, then swap the axes.  Two rounds where a divides m
// or m divides a.  a n + b fits 32 bits.
__device__ __forceinline__ long long floor_sum(unsigned n, unsigned m, unsigned a, unsigned b) {
  long long s = 0;
  while (n > 0) {
    s += static_cast<long long>(n) * (n - 1) / 2 * (a / m) + static_cast<long long>(n) * (b / m);
    a %= m;
    b %= m;
    const unsigned y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const unsigned t = m;
    m = a;
    a = t;
  }
  return s;
}

// Length of the first t row tiles of a request for one tile head (t at most their number); C: an
// item's constant.  In closed form: a prompt has thousands of row tiles.
template <int KT, int C>
__device__ __forceinline__ long long paged_prefix(int causal, const PagedReq& r, int tpt, int t) {
  const long long each = static_cast<long long>(t) * C;
  if (!causal) return each + static_cast<long long>(t) * ((max(r.kv, 1) + KT - 1) / KT);
  const int base = r.kv - r.nq;  // keys before the request's tokens (negative: rows without keys)
  const int full = min(t, r.nq / tpt);                       // tiles of tpt tokens
  const int none = base < 0 ? min(full, -base / tpt) : 0;    // whose rows see no key: one key tile
  long long s = each + none;
  if (full > none)
    s += floor_sum(full - none, KT, tpt, base + (none + 1) * tpt + KT - 1);
  if (t > full) s += (max(r.kv, 1) + KT - 1) / KT;           // the last, shorter tile
  return s;
}

// This thread's request of a batch that has one per thread at most: loaded, costed and placed on the
// line once for the CTA's share and its first list.  (Later lists load again: few CTAs need one,
// and the registers would be held through the loop.)
struct PagedMine {
  PagedReq r;
  long long lin, cost;
};

// The length W of the line.  Every thread of the block (NT) calls it.
template <int KT, int C, int NT>
__device__ long long paged_total(const PagedParams& p, int tpt, PagedSched& s, PagedMine& mine) {
  long long sum = 0, all;
  for (int b = threadIdx.x; b < p.B; b += NT) {
    mine.r = paged_req(p, b);
    sum += paged_prefix<KT, C>(p.causal, mine.r, tpt, (mine.r.nq + tpt - 1) / tpt) * p.Hv;
  }
  mine.lin = block_excl_scan<long long, NT>(sum, s.tmp, &all);
  mine.cost = sum;
  return all;
}

// Lists the row tiles that [lo, hi) of the line touches, PAGED_RECS at most, and sets s.stop to
// where the listed part ends.  Every thread of the block calls it, lo < hi.
template <int KT, int C, int NT>
__device__ __forceinline__ void paged_list(const PagedParams& p, int tpt, long long lo, long long hi,
                                           const PagedMine* mine, PagedSched& s) {
  const bool known = mine != nullptr && p.B <= NT;
  if (threadIdx.x == 0) s.stop = hi;
  long long carry = 0;
  int listed = 0;
  for (int b0 = 0; b0 < p.B && carry < hi && listed < PAGED_RECS; b0 += NT) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    PagedReq r = {0, 0, 0};
    long long lin = 0, cost = 0, sum = hi;
    int nt = 0;
    if (known) {
      if (b < p.B) {
        r = mine->r;
        cost = mine->cost;
      }
      lin = mine->lin;
      nt = (r.nq + tpt - 1) / tpt;
    } else {
      if (b < p.B) r = paged_req(p, b);
      nt = (r.nq + tpt - 1) / tpt;
      cost = paged_prefix<KT, C>(p.causal, r, tpt, nt) * p.Hv;
      lin = carry + block_excl_scan<long long, NT>(cost, s.tmp, &sum);
    }
    // this request's first row tile that ends behind lo, where it starts, and how many from it
    // on (PAGED_RECS at most) start before hi
    int t0 = 0, count = 0;
    long long x0 = lin;
    if (cost > 0 && lin < hi && lin + cost > lo) {
      if (lin < lo) {
        int end = nt;  // the tile is in [t0, end)
        while (end - t0 > 1) {
          const int mid = (t0 + end) >> 1;
          if (lin + paged_prefix<KT, C>(p.causal, r, tpt, mid) * p.Hv <= lo) t0 = mid; else end = mid;
        }
        x0 = lin + paged_prefix<KT, C>(p.causal, r, tpt, t0) * p.Hv;
      }
      long long x = x0;
      for (int t = t0; t < nt && x < hi && count < PAGED_RECS; ++t, ++count)
        x += static_cast<long long>(paged_tiles<KT>(p.causal, r, tpt, t) + C) * p.Hv;
    }
    int all;
    int at = listed + block_excl_scan<int, NT>(count, reinterpret_cast<int*>(s.tmp), &all);
    for (int t = t0; t < t0 + count && at < PAGED_RECS; ++t, ++at) {
      PagedRec c;
      c.lin = x0;
      c.b = b;
      c.tok0 = r.tok0 + t * tpt;
      c.ntok = min(tpt, r.nq - t * tpt);
      c.pos0 = r.kv - r.nq + t * tpt;
      c.kv = r.kv;
      c.n = paged_tiles<KT>(p.causal, r, tpt, t);
      s.rec[at] = c;
      x0 += static_cast<long long>(c.n + C) * p.Hv;
      if (at == PAGED_RECS - 1) s.stop = min(hi, x0);
    }
    carry += sum;
    listed = min(listed + all, PAGED_RECS);
  }
  if (threadIdx.x == 0) s.n_rec = listed;
  __syncthreads();
}

// One piece: key tiles [a, b) of the item (record, tile head h), a < b.
struct PagedPiece {
  int rec, h, a, b;
};

// Walks over the pieces of the listed part of a CTA's share.
template <int C>
struct PagedPieces {
  long long x;  // where the next piece is looked for
  int rec, h, off;  // its item, and how far x is into it
  __device__ __forceinline__ void start(const PagedParams&, const PagedSched& s, long long x0) {
    x = x0;
    rec = 0;
    while (rec + 1 < s.n_rec && x >= s.rec[rec + 1].lin) ++rec;
    const int len = s.rec[rec].n + C;
    const long long d = x - s.rec[rec].lin;
    h = static_cast<int>(d / len);
    off = static_cast<int>(d - static_cast<long long>(h) * len);
  }
  __device__ __forceinline__ bool next(const PagedParams& p, const PagedSched& s, PagedPiece& c) {
    while (x < s.stop) {
      const int n = s.rec[rec].n;
      const int step = static_cast<int>(min(static_cast<long long>(n + C - off), s.stop - x));
      c.rec = rec;
      c.h = h;
      c.a = off;
      c.b = min(n, off + step);
      const bool some = off < n;
      x += step;
      off = 0;
      if (++h == p.Hv) {
        h = 0;
        ++rec;
      }
      if (some) return true;
    }
    return false;
  }
};

// Where a piece's partial sums go: slot 0 continues an item, slot 1 leaves one unfinished.
__device__ __forceinline__ size_t paged_slot(int cta, const PagedPiece& c) {
  return static_cast<size_t>(cta) * 2 + (c.a > 0 ? 0 : 1);
}

// Start of a CTA: its share [lo, hi) of the line, and empty headers.  false: nothing to do.
// Every thread of the block calls it.  LEAST: the least share that is worth a CTA, in key tiles.
template <int KT, int C, int NT, int LEAST = 1>
__device__ __forceinline__ bool paged_share(const PagedParams& p, int tpt, PagedSched& s, long long& lo,
                                            long long& hi, PagedMine& mine) {
  const long long W = paged_total<KT, C, NT>(p, tpt, s, mine);
  const long long ctas = min(static_cast<long long>(gridDim.x), (W + LEAST - 1) / LEAST);
  const int cta = blockIdx.x;
  if (threadIdx.x == 0) {
    s.W = W;
    s.ctas = ctas;
    p.ws_head[2 * cta] = p.ws_head[2 * cta + 1] = make_int4(0, 0, 0, 0);
  }
  if (cta >= ctas) return false;
  lo = W * cta / ctas;
  hi = W * (cta + 1) / ctas;
  return true;
}

// The CTA whose share holds place x of the line.
__device__ __forceinline__ int paged_cta_of(const PagedSched& s, long long x) {
  return static_cast<int>(((x + 1) * s.ctas + s.W - 1) / s.W) - 1;
}

// Header of a piece c that is not a whole item, in its slot: {first CTA of the item's parts, their
// number << 16 | tokens, tile head, first token}.  Called by the thread that wrote the empty one.
template <int C>
__device__ __forceinline__ void paged_header(const PagedParams& p, const PagedSched& s,
                                             const PagedRec& r, const PagedPiece& c, int cta) {
  const long long start = r.lin + static_cast<long long>(c.h) * (r.n + C);
  const int first = c.a == 0 ? cta : paged_cta_of(s, start);
  const int last = c.b == r.n ? cta : paged_cta_of(s, start + r.n - 1);
  p.ws_head[paged_slot(cta, c)] = make_int4(first, (last - first + 1) << 16 | r.ntok, c.h, r.tok0);
}

// Natural-log log-sum-exp of a row from its maximum (log2 units) and sum; -inf without keys.
//
// A sum is exactly 0 where a row saw no key, or only scores of -inf, and only there (else the key that
// set the maximum has added 1).  So "no key" is read from the sum, never from the maximum: a row
// whose scores are all NaN keeps the maximum -inf, which max passes NaN over, and its NaN is in the
// sum.  Where the sum is 0 the sums of P V count as 0 too, whatever they hold: 0 times a V that is
// not finite is NaN.
__device__ __forceinline__ float paged_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// ---------------------------------------------------------------------------------- join
// Rows of an item that several CTAs worked on: O = sum_i 2^(m_i - m) O_i / l,
// l = sum_i 2^(m_i - m) l_i, over the parts in key order; part 0 is slot 1 of the first CTA, part i
// slot 0 of the i-th behind it.  Bound by the launch, the dependent loads (the header, the parts)
// and, after chunks, by the parts' 39 MB in L2 (148 SMs x two 128 KB parts); launched to overlap
// the end of the kernel before.  Two forms:
//   few rows, many parts (decoding): the blocks of the first CTA have all of them; four warps share
//     a row, each takes every fourth part, eight of them loaded at once, and they meet in warp
//     order;
//   many rows (chunks): the blocks of each of an item's CTAs have an equal share of its rows, a row
//     per group of lanes, four parts loaded at once.  (All rows by the first CTA's blocks: 45 us
//     for 128 tokens over 2048 keys, 16 heads over 4, d = 64, whose items are in 9 parts; so 21.
//     Several rows in flight per lane cost registers and were slower.)
constexpr int JOIN_WARPS = 8;

// The item of a header.
struct PagedJoinItem {
  int first, parts, rows, h, tok0;  // the CTAs that hold its parts; rows = 0: no item
  __device__ __forceinline__ void get(const PagedParams& p, const int4& e) {
    first = e.x;
    parts = e.y >> 16;
    rows = (e.y & 0xffff) * p.G;
    h = e.z;
    tok0 = e.w;
  }
};

__device__ __forceinline__ size_t paged_part(int cta, int i) {
  return i == 0 ? static_cast<size_t>(cta) * 2 + 1 : static_cast<size_t>(cta + i) * 2;
}

// Running join of one row, four columns per lane.
struct PagedJoin {
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  __device__ __forceinline__ void raise(float to) {  // to >= m
    const float f = to == m ? 1.0f : exp2f(m - to);
    m = to;
    l *= f;
    acc.x *= f;
    acc.y *= f;
    acc.z *= f;
    acc.w *= f;
  }
  __device__ __forceinline__ void add(float2 ml, float4 a) {  // ml.x <= m
    if (ml.y == 0.f) return;  // no key
    const float w = exp2f(ml.x - m);  // (NaN or 0 beside a NaN sum, which stays NaN)
    l = fmaf(w, ml.y, l);
    acc.x = fmaf(w, a.x, acc.x);
    acc.y = fmaf(w, a.y, acc.y);
    acc.z = fmaf(w, a.z, acc.z);
    acc.w = fmaf(w, a.w, acc.w);
  }
  template <typename T>
  __device__ __forceinline__ void store(const PagedParams& p, long long row, int col) const {
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    const float o[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
    T* op = static_cast<T*>(p.o) + row * p.d + col;
    if (p.d % 4 == 0) {  // o is 16-byte aligned
      if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint2*>(op) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
      else
        *reinterpret_cast<float4*>(op) = make_float4(o[0], o[1], o[2], o[3]);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (col + c < p.d) op[c] = from_f<T>(o[c]);
    }
    if (col == 0) p.lse[row] = paged_lse(m, l);
  }
};

template <typename T>
__global__ void __launch_bounds__(JOIN_WARPS * 32) fa_paged_join_few_kernel(const PagedParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const int cta = blockIdx.x;
  constexpr int WPR = 4, DEPTH = 8;
  __shared__ float4 s_acc[JOIN_WARPS][32];
  __shared__ float2 s_ml[JOIN_WARPS];
  PagedJoinItem item;  // the one that the CTA leaves unfinished, if any
  item.get(p, p.ws_head[2 * cta + 1]);
  if (item.rows == 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = item.rows, parts = item.parts;
  for (int r0 = blockIdx.y * (JOIN_WARPS / WPR); r0 < rows; r0 += gridDim.y * (JOIN_WARPS / WPR)) {
    const int r = r0 + warp / WPR;
    const int qh = paged_row_head(p, item.h, r, rows);
    PagedJoin j;
    for (int i0 = qh >= 0 ? warp % WPR : parts; i0 < parts; i0 += DEPTH * WPR) {
      float4 part[DEPTH];
      float2 ml[DEPTH];
      float top = j.m;
#pragma unroll
      for (int k = 0; k < DEPTH; ++k) {
        const int i = i0 + k * WPR;
        ml[k] = make_float2(-INFINITY, 0.f);
        part[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i >= parts) continue;
        const size_t at = paged_part(cta, i) * p.rows_cap + r;
        ml[k] = p.ws_ml[at];
        if (4 * lane < p.d) part[k] = *reinterpret_cast<const float4*>(p.ws_o + at * p.ws_pitch + 4 * lane);
      }
#pragma unroll
      for (int k = 0; k < DEPTH; ++k) top = fmaxf(top, ml[k].x);
      j.raise(top);
#pragma unroll
      for (int k = 0; k < DEPTH; ++k) j.add(ml[k], part[k]);
    }
    s_acc[warp][lane] = j.acc;
    if (lane == 0) s_ml[warp] = make_float2(j.m, j.l);
    __syncthreads();
    if (warp % WPR == 0 && qh >= 0 && 4 * lane < p.d) {
      float top = j.m;
#pragma unroll
      for (int w = 1; w < WPR; ++w) top = fmaxf(top, s_ml[warp + w].x);
      j.raise(top);
#pragma unroll
      for (int w = 1; w < WPR; ++w) j.add(s_ml[warp + w], s_acc[warp + w][lane]);
      j.store<T>(p, static_cast<long long>(item.tok0 + r / p.G) * p.H + qh, 4 * lane);
    }
    __syncthreads();  // s_acc is rewritten for the next rows
  }
}

// LPR: lanes per row, 4 LPR >= d.
template <typename T, int LPR>
__global__ void __launch_bounds__(JOIN_WARPS * 32) fa_paged_join_rows_kernel(const PagedParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const int cta = blockIdx.x;
  constexpr int GROUPS = JOIN_WARPS * 32 / LPR, DEPTH = 4;
  PagedJoinItem item[2];
  int lo[2], n[2];  // this CTA's rows of the one item and of the other: n from lo on
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    item[i].get(p, p.ws_head[2 * cta + i]);
    const int rows = item[i].rows, parts = item[i].parts, at = cta - item[i].first;
    lo[i] = parts == 0 ? 0 : rows * at / parts;
    n[i] = parts == 0 ? 0 : rows * (at + 1) / parts - lo[i];
  }
  const int col = 4 * (threadIdx.x % LPR);
  for (int e = blockIdx.y * GROUPS + threadIdx.x / LPR; e < n[0] + n[1]; e += gridDim.y * GROUPS) {
    const bool second = e >= n[0];
    const PagedJoinItem it = second ? item[1] : item[0];
    const int row = second ? lo[1] + e - n[0] : lo[0] + e, first = it.first, parts = it.parts;
    PagedJoin j;
    for (int i0 = 0; i0 < parts; i0 += DEPTH) {
      float4 part[DEPTH];
      float2 ml[DEPTH];
      float top = j.m;
#pragma unroll
      for (int k = 0; k < DEPTH; ++k) {
        ml[k] = make_float2(-INFINITY, 0.f);
        part[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i0 + k >= parts) continue;
        const size_t at = paged_part(first, i0 + k) * p.rows_cap + row;
        ml[k] = p.ws_ml[at];
        if (col < p.d) part[k] = *reinterpret_cast<const float4*>(p.ws_o + at * p.ws_pitch + col);
      }
#pragma unroll
      for (int k = 0; k < DEPTH; ++k) top = fmaxf(top, ml[k].x);
      j.raise(top);
#pragma unroll
      for (int k = 0; k < DEPTH; ++k) j.add(ml[k], part[k]);
    }
    const int qh = paged_row_head(p, it.h, row, it.rows);
    if (qh >= 0 && col < p.d) j.template store<T>(p, static_cast<long long>(it.tok0 + row / p.G) * p.H + qh, col);
  }
}

}  // namespace fa
