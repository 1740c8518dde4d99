// fa_paged_cache.cuh -- the paged key/value cache around the attention: the plan of a batch
// (token offsets, positions, cache slots, block-table entries from the requests' lengths) and
// the append of new keys and values at those slots, with the rotary rotation of keys and
// queries.
//
// Cache layout: [page][H_kv][page_size][d]; token position p of a request lies in page
// block_table[request][p / page_size], row p % page_size, and its slot is the number
// page * page_size + row.
#pragma once
#include <cstdint>

#include "fa_rope.cuh"

namespace fa {

// ---------------------------------------------------------------------------------- block scan
// Exclusive prefix sum over the block's threads; *total gets the sum.  `tmp` is 33 entries of
// shared memory; every thread of the block calls it (two barriers).
template <typename T, int NT>
__device__ __forceinline__ T block_excl_scan(T v, T* tmp, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T up = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += up;
  }
  if (lane == 31) tmp[warp] = s;
  __syncthreads();
  T before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const T x = tmp[w];
    if (w < warp) before += x;
    all += x;
  }
  __syncthreads();  // tmp may be written again
  *total = all;
  return before + s - v;
}

// ---------------------------------------------------------------------------------- plan
struct PlanParams {
  const int32_t *ctx_len, *new_len, *free_pages, *cursor;
  int32_t* table;
  long long table_stride;
  int32_t *cu_q, *kv_len, *positions, *counts;
  long long* slots;
  int B, n_free, max_pages, max_tokens, page_shift;
};

constexpr int PLAN_THREADS = 256;

// Each block owns PLAN_THREADS tokens and scans the requests' lengths by itself, PLAN_THREADS
// requests at a time, until it has passed its tokens: no second launch and no order between
// blocks.  Bound by the latency of one launch, of the lengths' load, of a page id's load and of
// the stores; the scan of B requests costs B / 256 further steps.  A page is opened by exactly
// one token (the one at its first row), and that token's thread writes the table entry; block 0
// also writes the per-request outputs.  2.8 us for 256 requests of one token as for 64 of up to
// 1000, back to back.
__global__ void __launch_bounds__(PLAN_THREADS) fa_paged_plan_kernel(const PlanParams p) {
  __shared__ long long tmp[33];
  __shared__ int s_start[PLAN_THREADS + 1];  // first token of each request (clamped)
  __shared__ int s_ctx[PLAN_THREADS];
  __shared__ int s_base[PLAN_THREADS];       // its first new page's place in the free list
  const int tid = threadIdx.x;
  const int t0 = static_cast<int>(blockIdx.x) * PLAN_THREADS;
  const int tok = t0 + tid;
  const int t_end = min(t0 + PLAN_THREADS, p.max_tokens);
  const int page = 1 << p.page_shift;
  const bool lead = blockIdx.x == 0;
  grid_dep_wait();  // launched to overlap the kernel before, as the next one may overlap this
  grid_dep_launch();
  const long long cursor = p.cursor == nullptr ? 0 : max(0, *p.cursor);
  long long asked = 0, pages = 0;  // sums over the requests before this round's
  for (int b0 = 0; b0 < p.B; b0 += PLAN_THREADS) {
    const int b = b0 + tid;
    const long long ctx = b < p.B ? max(0, p.ctx_len[b]) : 0;
    const long long want = b < p.B ? max(0, p.new_len[b]) : 0;
    long long sum;
    const long long start = asked + block_excl_scan<long long, PLAN_THREADS>(want, tmp, &sum);
    // tokens beyond max_tokens are not part of the step
    const long long got = min(want, max(0ll, p.max_tokens - start));
    const long long first = (ctx + page - 1) >> p.page_shift;
    const long long last = min((ctx + got + page - 1) >> p.page_shift,
                               static_cast<long long>(p.max_pages));
    long long psum;
    const long long base =
        pages + block_excl_scan<long long, PLAN_THREADS>(max(0ll, last - first), tmp, &psum);
    if (lead && b < p.B) {
      p.cu_q[b] = static_cast<int>(min(start, static_cast<long long>(p.max_tokens)));
      p.kv_len[b] = static_cast<int>(min(ctx + got, 0x7fffffffll));
    }
    const long long here = min(asked, static_cast<long long>(p.max_tokens));
    const long long next = min(asked + sum, static_cast<long long>(p.max_tokens));
    if (here < t_end && next > t0) {
      s_start[tid] = static_cast<int>(min(start, static_cast<long long>(p.max_tokens)));
      s_ctx[tid] = static_cast<int>(ctx);
      s_base[tid] = static_cast<int>(min(base, 0x7fffffffll));
      __syncthreads();
      if (tok >= here && tok < next) {
        // the last request of this round that starts at or before the token (empty requests
        // share their start with the one that follows, which is later)
        int lo = 0, hi = min(PLAN_THREADS, p.B - b0);
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (s_start[mid] <= tok) lo = mid; else hi = mid;
        }
        const long long pos = static_cast<long long>(s_ctx[lo]) + (tok - s_start[lo]);
        const long long at = pos >> p.page_shift;
        const long long opened = (static_cast<long long>(s_ctx[lo]) + page - 1) >> p.page_shift;
        int id = -1;
        if (at < p.max_pages) {
          int32_t* entry = p.table + (b0 + lo) * p.table_stride + at;
          if (at >= opened) {
            const long long k = cursor + s_base[lo] + (at - opened);
            if (k < p.n_free) id = p.free_pages[k];
            if ((pos & (page - 1)) == 0) *entry = id;
          } else {
            id = *entry;
          }
        }
        p.positions[tok] = static_cast<int>(min(pos, 0x7fffffffll));
        p.slots[tok] = id < 0 ? -1ll
                              : (static_cast<long long>(id) << p.page_shift) + (pos & (page - 1));
      }
      __syncthreads();  // the shared arrays are rewritten in the next round
    }
    asked += sum;
    pages += psum;
    if (!lead && asked >= t_end) return;
  }
  // padding behind the last request
  if (tok < p.max_tokens && tok >= asked) {
    p.positions[tok] = 0;
    p.slots[tok] = -1;
  }
  if (lead && tid == 0) {
    const long long avail = max(0ll, p.n_free - cursor);
    const long long taken = min(pages, avail);
    p.cu_q[p.B] = static_cast<int>(min(asked, static_cast<long long>(p.max_tokens)));
    p.counts[0] = static_cast<int>(min(asked, 0x7fffffffll));
    p.counts[1] = static_cast<int>(taken);
    p.counts[2] = static_cast<int>(min(pages - taken, 0x7fffffffll));
    p.counts[3] = static_cast<int>(min(cursor + taken, 0x7fffffffll));
  }
}

// ---------------------------------------------------------------------------------- append
struct AppendParams {
  const void *q, *k, *v;
  void *q_out, *k_cache, *v_cache;
  const long long* slots;
  const int32_t* positions;  // or nullptr: no rotation (rot = 0)
  const double* inv_freq;
  long long qs[2], ks[2], vs[2], qos[2];  // token and head strides in elements
  long long k_page, v_page;               // page strides of the caches in elements
  long long n_slots;                      // num_pages * page_size
  int T, H, H_kv, d, rot;                 // H = 0 without queries
  int n_rot, n_units;
  RopeShape shape;
  int page_shift;
  float mag;
};

// The H + 2 H_kv head rows of a token: queries, keys, values.
template <typename T>
struct AppendRows {
  const AppendParams& p;
  const T *q, *k, *v;   // the token's first rows
  T *qo, *kc, *vc;      // where they go; kc = nullptr: the token is not stored
  __device__ __forceinline__ void prepare(int n) {
    q = static_cast<const T*>(p.q) + n * p.qs[0];
    qo = static_cast<T*>(p.q_out) + n * p.qos[0];
    k = static_cast<const T*>(p.k) + n * p.ks[0];
    v = static_cast<const T*>(p.v) + n * p.vs[0];
    const long long slot = p.slots[n];
    kc = vc = nullptr;
    if (slot >= 0 && slot < p.n_slots) {  // else padding, or no such slot
      const long long pg = slot >> p.page_shift, row = slot & ((1 << p.page_shift) - 1);
      kc = static_cast<T*>(p.k_cache) + pg * p.k_page + row * p.d;
      vc = static_cast<T*>(p.v_cache) + pg * p.v_page + row * p.d;
    }
  }
  __device__ __forceinline__ const T* src(int h) const {
    if (h < p.H) return q + h * p.qs[1];
    h -= p.H;
    return h < p.H_kv ? k + h * p.ks[1] : v + (h - p.H_kv) * p.vs[1];
  }
  __device__ __forceinline__ T* dst(int h) const {
    if (h < p.H) return qo + h * p.qos[1];
    h -= p.H;
    return h < p.H_kv ? kc + (static_cast<long long>(h) << p.page_shift) * p.d
                      : vc + (static_cast<long long>(h - p.H_kv) << p.page_shift) * p.d;
  }
  __device__ __forceinline__ bool stored(int h) const { return h < p.H || kc != nullptr; }
  __device__ __forceinline__ bool turned(int h) const { return h < p.H + p.H_kv; }
};

// One launch for all three tensors.  Bound by the launch and two dependent loads at a decode
// step's size (64 tokens, 32 + 16 heads, d = 128: 2.9 us back to back), by HBM at a prompt's (8201
// tokens, 16 + 8 heads, d = 64, 50 MB: 11.6 us from L2, 15.9 from HBM, 3.2 TB/s: 774 blocks at three
// per SM are 1.74 waves, the second three quarters full; 387 blocks, one wave, take 11.1).  fp32, 2000
// tokens, 32 + 16 heads, d = 128 (98 MB): 18.0 us, 5.5 TB/s.
template <typename T, int V, bool IL>
__global__ void __launch_bounds__(ROPE_THREADS, 3) fa_paged_append_kernel(const AppendParams p) {
  AppendRows<T> rows = {p, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr};
  rope_block<T, V, IL>(p.shape, p.T, p.H + 2 * p.H_kv, p.rot, p.n_rot, p.n_units, p.positions,
                       p.inv_freq, p.mag, 1.0f, rows);
}

}  // namespace fa
