// fa_paged_api.cuh -- host side of the rotary and paged-cache entry points: argument checks,
// the choice of kernel and launch shape, launches.  Included by fa_lib.cu behind fa_api.cu,
// whose helpers (fail, check_launch, set_smem, TimedLaunch, encode_fn) it uses.
#pragma once

namespace {

constexpr int kSms = 148;            // B200; grids and workspaces are sized by it

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int dtype_bytes(int dtype) { return dtype == FA_BF16 ? 2 : (dtype == FA_F32 ? 4 : 0); }

int log2_page(int page_size) {
  if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)) != 0) return -1;
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

// A launch that may overlap the kernel before it on the stream (programmatic dependent launch): every
// kernel launched so waits for that kernel before its first access to memory.  Back to back, the
// launch latency and the set-up of a kernel then hide behind the one before.
template <typename... Exp, typename... Act>
int launch_overlapped(const char* what, void (*kern)(Exp...), dim3 grid, unsigned block, size_t smem,
                      cudaStream_t s, Act&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, std::forward<Act>(args)...);
  if (e != cudaSuccess) return fail(FA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return check_launch(what);
}

// ---- rotary -----------------------------------------------------------------------------
// Vector width for rows of d columns of which `rot` turn: 16 bytes where every row start and
// every piece of a row allows it, else one element.
int rope_vec(int es, int d, int rot, bool rows16) {
  const int v = 16 / es;
  return rows16 && (rot / 2) % v == 0 && (d - rot) % v == 0 ? v : 1;
}

// Lays blocks over the work.  A thread walks over several heads where that still leaves every SM
// enough blocks; otherwise one head per thread, and so few tokens per block that the table of cos
// and sin is one entry per thread.  Measured (back to back in a graph, us) with 8 / 4 / 2 heads per
// thread and, at the least sizes, the small table; * the rule's choice:
//   rotation 16 x 16384 x 128             23.7* 27.5  42.7         1024 blocks of 8 heads
//   rotation 8 x 12 x 1024 x 64           10.6   7.6* 10.7          256
//   append 8201 tokens, 24 heads, d 64    11.1  11.7* 14.9          387
//   append 2048 tokens, 48 heads, d 128    9.7  13.4* 20.2          384
//   append  512 tokens, 48 heads, d 128    5.9   5.7   6.6   7.5*    96
//   append   64 tokens, 48 heads, d 128    5.7   4.6   4.1   2.9*    12
// So the two borders (6 blocks of 8 heads per SM, 3/2 of 4) lie on the safe side of the largest and the
// smallest sizes; between them, where blocks of 8 heads make one or two waves, up to a quarter is lost.
fa::RopeShape rope_shape(long long N, int heads, int B, int units, int pass, int half) {
  fa::RopeShape sh;
  sh.pass = pass;
  sh.uw = std::min(units, fa::ROPE_THREADS);
  sh.u_blocks = (units + sh.uw - 1) / sh.uw;
  const int rows = fa::ROPE_THREADS / sh.uw;
  auto place = [&](int tb, int hpt) {
    sh.tb = static_cast<int>(std::min<long long>(N, std::max(1, std::min(tb, rows))));
    sh.hs = std::min(heads, rows / sh.tb);
    sh.hpt = std::min(hpt, (heads + sh.hs - 1) / sh.hs);
    sh.h_blocks = (heads + sh.hs * sh.hpt - 1) / (sh.hs * sh.hpt);
    return (N + sh.tb - 1) / sh.tb * sh.h_blocks * sh.u_blocks * B;
  };
  if (place(rows, 2 * fa::ROPE_DEPTH) >= 6 * kSms) return sh;
  if (place(rows, fa::ROPE_DEPTH) >= 3 * kSms / 2) return sh;
  place(half > 0 ? fa::ROPE_THREADS / half : rows, 1);
  return sh;
}

template <typename T, int V>
void (*rope_kernel(bool il))(const fa::RopeParams) {
  return il ? fa::fa_rope_kernel<T, V, true> : fa::fa_rope_kernel<T, V, false>;
}
template <typename T, int V>
void (*append_kernel(bool il))(const fa::AppendParams) {
  return il ? fa::fa_paged_append_kernel<T, V, true> : fa::fa_paged_append_kernel<T, V, false>;
}

// ---- paged attention ----------------------------------------------------------------------
// One kernel variant: rows and keys of a tile and CTAs of the grid.
struct PagedShape {
  int rows, ctas;
};

size_t paged_ws_part(long long T, int group, int d, PagedShape v, int* rows_cap, size_t* off_ml,
                     size_t* off_o) {
  const int splits = (group + v.rows - 1) / v.rows;
  const int G = (group + splits - 1) / splits;
  const long long cap = std::min<long long>(v.rows, T * G);
  const size_t head = round256(static_cast<size_t>(v.ctas) * 2 * sizeof(int4));
  const size_t ml = round256(static_cast<size_t>(v.ctas) * 2 * cap * sizeof(float2));
  if (rows_cap != nullptr) {
    *rows_cap = static_cast<int>(cap);
    *off_ml = head;
    *off_o = head + ml;
  }
  return head + ml + round256(static_cast<size_t>(v.ctas) * 2 * cap * ((d + 3) / 4 * 4) * sizeof(float));
}

// CTAs of a CUDA-core variant: what shared memory lets an SM hold, up to what its registers are
// kept for.
template <typename L>
PagedShape f32_shape(int d) {
  const int per_sm = static_cast<int>(std::min<size_t>(L::ctas((d + 31) / 32), 233472 / (L::bytes(d) + 1024)));
  return {L::R, kSms * per_sm};
}

PagedShape decode_shape() { return {16, kSms}; }
PagedShape chunk_shape(int d) { return {256, kSms * (d == 64 ? fa::PagedChunkLayout<64>::CTAS_PER_SM : 1)}; }

size_t paged_ws_bytes(long long T, int group, int d) {
  size_t n = 0;
  for (const PagedShape v : {f32_shape<fa::PagedF32Few>(d), f32_shape<fa::PagedF32Chunk>(d), decode_shape(),
                             chunk_shape(d)})
    n = std::max(n, paged_ws_part(T, group, d, v, nullptr, nullptr, nullptr));
  return n;
}

// Sets the tile fields of a variant's parameters and lays its workspace out.
void paged_tiles(fa::PagedParams& p, PagedShape v, int H_kv, void* ws) {
  size_t off_ml = 0, off_o = 0;
  p.splits = (p.group + v.rows - 1) / v.rows;
  p.G = (p.group + p.splits - 1) / p.splits;
  p.Hv = H_kv * p.splits;
  p.ws_pitch = (p.d + 3) / 4 * 4;
  paged_ws_part(p.T, p.group, p.d, v, &p.rows_cap, &off_ml, &off_o);
  uint8_t* b = static_cast<uint8_t*>(ws);
  p.ws_head = reinterpret_cast<int4*>(b);
  p.ws_ml = reinterpret_cast<float2*>(b + off_ml);
  p.ws_o = reinterpret_cast<float*>(b + off_o);
}

// few: after the kernel of few rows per tile.
template <typename T>
int launch_join(const fa::PagedParams& p, int ctas, bool few, cudaStream_t s) {
  // blocks per CTA: two rows each, or eight per SM
  const int y = few ? (p.rows_cap + 1) / 2 : 8 * kSms / ctas;
  auto* kern = few ? fa::fa_paged_join_few_kernel<T>
                   : (p.d <= 64 ? fa::fa_paged_join_rows_kernel<T, 16> : fa::fa_paged_join_rows_kernel<T, 32>);
  return launch_overlapped("fa_paged_join_kernel", kern, dim3(ctas, y), fa::JOIN_WARPS * 32, 0, s, p);
}

template <typename L>
int launch_paged_f32(void (*kern)(fa::PagedParams), const fa::PagedParams& p, cudaStream_t s) {
  const size_t smem = L::bytes(p.d);
  const int rc = set_smem(kern, static_cast<int>(smem));
  if (rc != FA_OK) return rc;
  return launch_overlapped("fa_paged_f32_kernel", kern, dim3(f32_shape<L>(p.d).ctas), L::THREADS, smem, s, p);
}

// 4-D view [page][H_kv][page_size][d] bf16 of a cache, 128-byte swizzled boxes of 64 columns and
// box_rows rows of one page and head.  An out-of-range page reads as zeros.
int make_cache_map(CUtensorMap* map, const void* base, int pages, int H_kv, int page_size, int d,
                   long long page_stride, int box_rows, const char* name) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const long long page_elems = static_cast<long long>(H_kv) * page_size * d;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(page_size),
                              static_cast<cuuint64_t>(H_kv), static_cast<cuuint64_t>(pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(d) * 2,
                                 static_cast<cuuint64_t>(page_size) * d * 2,
                                 static_cast<cuuint64_t>(pages > 1 ? page_stride : page_elems) * 2};
  const cuuint32_t box[4] = {64u, static_cast<cuuint32_t>(box_rows), 1u, 1u};
  const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims,
                         strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FA_ERR_CUDA, "tensor map for %s failed (%d)", name, (int)r);
  return FA_OK;
}

template <int D>
int launch_paged_decode(const fa::PagedParams& p, int H_kv, int page_size, cudaStream_t s) {
  using L = fa::PagedDecodeLayout<D>;
  CUtensorMap mk, mv;
  const int box = std::min(page_size, L::KT);
  int rc;
  if ((rc = make_cache_map(&mk, p.k, p.num_pages, H_kv, page_size, D, p.k_page, box, "k_cache")) != FA_OK) return rc;
  if ((rc = make_cache_map(&mv, p.v, p.num_pages, H_kv, page_size, D, p.v_page, box, "v_cache")) != FA_OK) return rc;
  if ((rc = set_smem(fa::fa_paged_decode_sm100_kernel<D>, L::SMEM_ALLOC)) != FA_OK) return rc;
  TimedLaunch tl("fa_paged_decode_sm100_kernel", s);
  return launch_overlapped("fa_paged_decode_sm100_kernel", fa::fa_paged_decode_sm100_kernel<D>,
                           dim3(decode_shape().ctas), L::THREADS, L::SMEM_ALLOC, s, mk, mv, p);
}

// 3-D view [T][H][d] bf16 of the packed queries, 128-byte swizzled boxes of 64 columns, `heads`
// heads and `tokens` tokens.
int make_query_map(CUtensorMap* map, const fa::PagedParams& p, int heads, int tokens) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(p.d), static_cast<cuuint64_t>(p.H),
                              static_cast<cuuint64_t>(p.T)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(p.H > 1 ? p.q_sh : p.d) * 2,
                                 static_cast<cuuint64_t>(p.T > 1 ? p.q_st : p.d) * 2};
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(heads), static_cast<cuuint32_t>(tokens)};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p.q), dims,
                         strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FA_ERR_CUDA, "tensor map for q failed (%d)", (int)r);
  return FA_OK;
}

template <int D>
int launch_paged_chunk(const fa::PagedParams& p, int H_kv, int page_size, cudaStream_t s) {
  using L = fa::PagedChunkLayout<D>;
  CUtensorMap mq, mqf, mk, mv;
  const int box = std::min(page_size, L::BN);
  const int tpt = L::R / p.G, few = std::min(tpt, std::max(1, 32 / p.G));
  int rc;
  if ((rc = make_query_map(&mq, p, p.G, tpt)) != FA_OK) return rc;
  if ((rc = make_query_map(&mqf, p, p.G, few)) != FA_OK) return rc;
  if ((rc = make_cache_map(&mk, p.k, p.num_pages, H_kv, page_size, D, p.k_page, box, "k_cache")) != FA_OK) return rc;
  if ((rc = make_cache_map(&mv, p.v, p.num_pages, H_kv, page_size, D, p.v_page, box, "v_cache")) != FA_OK) return rc;
  if ((rc = set_smem(fa::fa_paged_chunk_sm100_kernel<D>, L::SMEM_ALLOC)) != FA_OK) return rc;
  TimedLaunch tl("fa_paged_chunk_sm100_kernel", s);
  return launch_overlapped("fa_paged_chunk_sm100_kernel", fa::fa_paged_chunk_sm100_kernel<D>,
                           dim3(chunk_shape(D).ctas), L::THREADS, L::SMEM_ALLOC, s, mq, mqf, mk, mv, few, p);
}

// Rows of a K/V head (new tokens x heads of its group) up to which the kernels of few rows per tile run.
//   bf16: 16 rows, one tile.  More rows read the cache once per tile: 16 requests of 8192 keys, 32
//   heads over 8, d 128, take 98 us with 16 rows (chunk kernel 112), 177 with 24 (112); 2 requests
//   of 2048 keys 16 us (17) and 19 (17).
//   fp32: 24 rows, three tiles of 8: 4 requests of 4096 keys, 8 heads over 4, d 128: 36 us with 8
//   rows (chunk kernel 83), 60 with 16 (84), 79 with 24 (85), 103 with 32 (86).
int few_rows(int dtype) { return dtype == FA_F32 ? 24 : 16; }

// The kernel of the batch and its join; rows: of a K/V head.
int paged_run_bf16(fa::PagedParams p, long long rows, int H_kv, int page_size, void* ws, cudaStream_t s) {
  const bool few = rows <= few_rows(FA_BF16);
  const PagedShape v = few ? decode_shape() : chunk_shape(p.d);
  paged_tiles(p, v, H_kv, ws);
  int rc;
  if (few) rc = p.d == 64 ? launch_paged_decode<64>(p, H_kv, page_size, s) : launch_paged_decode<128>(p, H_kv, page_size, s);
  else rc = p.d == 64 ? launch_paged_chunk<64>(p, H_kv, page_size, s) : launch_paged_chunk<128>(p, H_kv, page_size, s);
  return rc != FA_OK ? rc : launch_join<__nv_bfloat16>(p, v.ctas, few, s);
}

int paged_run_f32(fa::PagedParams p, long long rows, int H_kv, void* ws, cudaStream_t s) {
  using Kernel = void (*)(fa::PagedParams);
  const bool few = rows <= few_rows(FA_F32);
  const PagedShape v = few ? f32_shape<fa::PagedF32Few>(p.d) : f32_shape<fa::PagedF32Chunk>(p.d);
  paged_tiles(p, v, H_kv, ws);
  const Kernel few_kernels[4] = {fa::fa_paged_f32_few_kernel<1>, fa::fa_paged_f32_few_kernel<2>,
                                 fa::fa_paged_f32_few_kernel<3>, fa::fa_paged_f32_few_kernel<4>};
  const Kernel chunk_kernels[4] = {fa::fa_paged_f32_chunk_kernel<1>, fa::fa_paged_f32_chunk_kernel<2>,
                                   fa::fa_paged_f32_chunk_kernel<3>, fa::fa_paged_f32_chunk_kernel<4>};
  const int nc = (p.d - 1) / 32;
  const int rc = few ? launch_paged_f32<fa::PagedF32Few>(few_kernels[nc], p, s)
                     : launch_paged_f32<fa::PagedF32Chunk>(chunk_kernels[nc], p, s);
  return rc != FA_OK ? rc : launch_join<float>(p, v.ctas, few, s);
}

// Whether [a, a + an) and [b, b + bn) share a byte.
bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && x < y + bn && y < x + an;
}

// Whether [a, a + an) shares a byte with one of `rows` pieces of n bytes, `stride` >= n bytes apart.
bool overlap_rows(const void* a, size_t an, const void* b, size_t rows, size_t stride, size_t n) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  if (a == nullptr || b == nullptr || an == 0) return false;
  if (x < y) return y < x + an;
  const size_t r = (x - y) / stride, in = (x - y) % stride;  // the row at or before a
  return r < rows && (in < n || (r + 1 < rows && in + an > stride));
}

// Copies a packed call's arguments (which need not be aligned) after checking their size.
template <typename Args>
int unpack(const Args* packed, Args* a) {
  if (packed == nullptr) return fail(FA_ERR_INVALID, "null arguments");
  std::memcpy(&a->size, packed, sizeof(a->size));
  if (a->size != sizeof(Args))
    return fail(FA_ERR_INVALID, "packed arguments of %llu bytes, not %zu",
                static_cast<unsigned long long>(a->size), sizeof(Args));
  std::memcpy(a, packed, sizeof(Args));
  return FA_OK;
}

}  // namespace

extern "C" {

int fa_rope(const void* x, void* y, const int32_t* positions, const double* inv_freq, int B, int H,
            int N, int d, int rotary_dim, const int64_t* x_strides, const int64_t* y_strides,
            int64_t positions_stride, float magnitude, int options, int dtype, void* stream) {
  const int es = dtype_bytes(dtype);
  if (es == 0) return fail(FA_ERR_INVALID, "unknown dtype %d", dtype);
  if ((options & ~(FA_ROPE_INTERLEAVED | FA_ROPE_BACKWARD)) != 0)
    return fail(FA_ERR_INVALID, "unknown rotary options 0x%x", options);
  if (B < 0 || H < 1 || N < 0 || d < 1) return fail(FA_ERR_INVALID, "B, N >= 0 and H, d >= 1 required");
  if (d > 1024) return fail(FA_ERR_UNSUPPORTED, "d <= 1024 required, got %d", d);
  if (rotary_dim < 2 || rotary_dim > d || (rotary_dim & 1) != 0)
    return fail(FA_ERR_INVALID, "rotary_dim must be even and in [2, d], got %d", rotary_dim);
  if (!std::isfinite(magnitude)) return fail(FA_ERR_INVALID, "magnitude must be finite");
  if (x_strides == nullptr || y_strides == nullptr) return fail(FA_ERR_INVALID, "null strides");
  if (B == 0 || N == 0) return FA_OK;
  if (!x || !y || !inv_freq) return fail(FA_ERR_INVALID, "null tensor pointer");
  if (N > (1 << 24)) return fail(FA_ERR_UNSUPPORTED, "N too large");
  const int ext[3] = {B, H, N};
  bool rows16 = aligned_to(x, 16) && aligned_to(y, 16);
  for (int i = 0; i < 3; ++i) {
    if (ext[i] < 2) continue;
    if (y_strides[i] == 0) return fail(FA_ERR_INVALID, "the output's strides must not be 0");
    if (x == y && x_strides[i] != y_strides[i])
      return fail(FA_ERR_INVALID, "in place, input and output strides must be equal");
    rows16 = rows16 && (x_strides[i] * es) % 16 == 0 && (y_strides[i] * es) % 16 == 0;
  }
  if (!aligned_to(x, es) || !aligned_to(y, es) || !aligned_to(inv_freq, 8) ||
      !aligned_to(positions, 4))
    return fail(FA_ERR_ALIGN, "a pointer is not aligned to its elements");
  fa::RopeParams p;
  p.x = x;
  p.y = y;
  p.positions = positions;
  p.inv_freq = inv_freq;
  for (int i = 0; i < 3; ++i) {
    p.xs[i] = x_strides[i];
    p.ys[i] = y_strides[i];
  }
  p.pos_sb = positions_stride;
  p.B = B;
  p.H = H;
  p.N = N;
  p.rot = rotary_dim;
  const int V = rope_vec(es, d, rotary_dim, rows16);
  p.n_rot = rotary_dim / 2 / V;
  const int vecs = x == y ? 0 : (d - rotary_dim) / V;  // pass-through; in place, they stay
  const int pass = vecs % 2 == 0 ? 2 : 1;
  p.n_units = p.n_rot + vecs / pass;
  p.shape = rope_shape(N, H, B, p.n_units, pass, rotary_dim / 2);
  p.mag = magnitude;
  p.sgn = (options & FA_ROPE_BACKWARD) ? -1.0f : 1.0f;
  const long long gx = (N + p.shape.tb - 1ll) / p.shape.tb * p.shape.h_blocks * p.shape.u_blocks;
  if (gx > 0x7fffffffll) return fail(FA_ERR_UNSUPPORTED, "grid too large");
  const bool il = (options & FA_ROPE_INTERLEAVED) != 0;
  auto* kern = dtype == FA_BF16 ? (V > 1 ? rope_kernel<__nv_bfloat16, 8>(il) : rope_kernel<__nv_bfloat16, 1>(il))
                                : (V > 1 ? rope_kernel<float, 4>(il) : rope_kernel<float, 1>(il));
  const int by = std::min(B, 65535);
  if ((B + by - 1) / by > 65535) return fail(FA_ERR_UNSUPPORTED, "B too large");
  return launch_overlapped("fa_rope_kernel", kern, dim3(static_cast<unsigned>(gx), by, (B + by - 1) / by),
                           fa::ROPE_THREADS, 0, static_cast<cudaStream_t>(stream), p);
}

int fa_paged_plan(const int32_t* ctx_len, const int32_t* new_len, const int32_t* free_pages,
                  int n_free, const int32_t* cursor, int32_t* block_table, int64_t table_stride,
                  int B, int max_pages, int page_size, int max_tokens, int32_t* cu_q,
                  int32_t* kv_len, int32_t* positions, int64_t* slots, int32_t* counts,
                  void* stream) {
  const int shift = log2_page(page_size);
  if (shift < 0) return fail(FA_ERR_INVALID, "page_size must be a power of two in [16, 1024], got %d", page_size);
  if (B < 1 || max_pages < 1 || max_tokens < 1 || n_free < 0)
    return fail(FA_ERR_INVALID, "B, max_pages, max_tokens >= 1 and n_free >= 0 required");
  if (B > (1 << 24) || max_tokens > (1 << 24)) return fail(FA_ERR_UNSUPPORTED, "B or max_tokens too large");
  if (!ctx_len || !new_len || (!free_pages && n_free > 0) || !block_table || !cu_q || !kv_len ||
      !positions || !slots || !counts)
    return fail(FA_ERR_INVALID, "null pointer");
  if (B > 1 && table_stride < max_pages)
    return fail(FA_ERR_INVALID, "block-table rows overlap: stride %lld for %d pages",
                static_cast<long long>(table_stride), max_pages);
  if (!aligned_to(ctx_len, 4) || !aligned_to(new_len, 4) || !aligned_to(free_pages, 4) ||
      !aligned_to(cursor, 4) || !aligned_to(block_table, 4) || !aligned_to(cu_q, 4) ||
      !aligned_to(kv_len, 4) || !aligned_to(positions, 4) || !aligned_to(slots, 8) ||
      !aligned_to(counts, 4))
    return fail(FA_ERR_ALIGN, "a pointer is not aligned to its elements");
  {
    // blocks read the inputs while others write: an output must not be an input, nor another output
    const size_t b4 = static_cast<size_t>(B) * 4, t4 = static_cast<size_t>(max_tokens) * 4;
    const size_t row = static_cast<size_t>(max_pages) * 4;
    const size_t stride = B > 1 ? static_cast<size_t>(table_stride) * 4 : row;
    auto in_table = [&](const void* t, size_t n) { return overlap_rows(t, n, block_table, B, stride, row); };
    const struct {
      const void* p;
      size_t n;
    } in[4] = {{ctx_len, b4}, {new_len, b4}, {free_pages, static_cast<size_t>(n_free) * 4}, {cursor, 4}},
      out[5] = {{cu_q, b4 + 4}, {kv_len, b4}, {positions, t4}, {slots, 2 * t4}, {counts, 16}};
    for (const auto& i : in) {
      bool bad = in_table(i.p, i.n);
      for (const auto& o : out) bad = bad || (i.n > 0 && overlap(i.p, i.n, o.p, o.n));
      if (bad) return fail(FA_ERR_INVALID, "an output overlaps an input");
    }
    for (int i = 0; i < 5; ++i) {
      bool bad = in_table(out[i].p, out[i].n);
      for (int j = 0; j < i; ++j) bad = bad || overlap(out[i].p, out[i].n, out[j].p, out[j].n);
      if (bad) return fail(FA_ERR_INVALID, "two outputs overlap");
    }
  }
  fa::PlanParams p;
  p.ctx_len = ctx_len;
  p.new_len = new_len;
  p.free_pages = free_pages;
  p.cursor = cursor;
  p.table = block_table;
  p.table_stride = table_stride;
  p.cu_q = cu_q;
  p.kv_len = kv_len;
  p.positions = positions;
  p.counts = counts;
  p.slots = reinterpret_cast<long long*>(slots);
  p.B = B;
  p.n_free = n_free;
  p.max_pages = max_pages;
  p.max_tokens = max_tokens;
  p.page_shift = shift;
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(max_tokens) + fa::PLAN_THREADS - 1) / fa::PLAN_THREADS);
  return launch_overlapped("fa_paged_plan_kernel", fa::fa_paged_plan_kernel, dim3(grid), fa::PLAN_THREADS, 0,
                           static_cast<cudaStream_t>(stream), p);
}

int fa_paged_append(const void* q, const void* k, const void* v, void* q_out, void* k_cache,
                    void* v_cache, const int64_t* slots, const int32_t* positions,
                    const double* inv_freq, int T, int H, int H_kv, int d, int rotary_dim,
                    const int64_t* strides, int64_t k_page_stride, int64_t v_page_stride,
                    int page_size, int num_pages, float magnitude, int options, int dtype,
                    void* stream) {
  const int es = dtype_bytes(dtype);
  if (es == 0) return fail(FA_ERR_INVALID, "unknown dtype %d", dtype);
  if ((options & ~FA_ROPE_INTERLEAVED) != 0) return fail(FA_ERR_INVALID, "unknown append options 0x%x", options);
  const int shift = log2_page(page_size);
  if (shift < 0) return fail(FA_ERR_INVALID, "page_size must be a power of two in [16, 1024], got %d", page_size);
  if (T < 0 || H < 0 || H_kv < 1 || d < 1 || num_pages < 1)
    return fail(FA_ERR_INVALID, "T, H >= 0 and H_kv, d, num_pages >= 1 required");
  if (d > 1024) return fail(FA_ERR_UNSUPPORTED, "d <= 1024 required, got %d", d);
  if (strides == nullptr) return fail(FA_ERR_INVALID, "null strides");
  if (inv_freq == nullptr ? rotary_dim != 0
                          : (rotary_dim < 2 || rotary_dim > d || (rotary_dim & 1) != 0))
    return fail(FA_ERR_INVALID, "rotary_dim must be even and in [2, d], or 0 without inv_freq; got %d", rotary_dim);
  if (inv_freq != nullptr && positions == nullptr && T > 0)
    return fail(FA_ERR_INVALID, "a rotation needs positions");
  if (!std::isfinite(magnitude)) return fail(FA_ERR_INVALID, "magnitude must be finite");
  const long long page_elems = static_cast<long long>(H_kv) * page_size * d;
  if (num_pages > 1 && (k_page_stride < page_elems || v_page_stride < page_elems))
    return fail(FA_ERR_INVALID, "cache pages overlap");
  if (T == 0) return FA_OK;
  if (!k || !v || !k_cache || !v_cache || !slots || (H > 0 && (!q || !q_out)))
    return fail(FA_ERR_INVALID, "null tensor pointer");
  if (T > (1 << 24)) return fail(FA_ERR_UNSUPPORTED, "T too large");
  // strides: token and head of q, k, v, q_out
  bool rows16 = aligned_to(k, 16) && aligned_to(v, 16) && aligned_to(k_cache, 16) && aligned_to(v_cache, 16) &&
                (static_cast<long long>(d) * es) % 16 == 0 && (k_page_stride * es) % 16 == 0 &&
                (v_page_stride * es) % 16 == 0;
  bool elems = aligned_to(k, es) && aligned_to(v, es) && aligned_to(k_cache, es) && aligned_to(v_cache, es) &&
               aligned_to(slots, 8) && aligned_to(positions, 4) && aligned_to(inv_freq, 8);
  if (H > 0) {
    rows16 = rows16 && aligned_to(q, 16) && aligned_to(q_out, 16);
    elems = elems && aligned_to(q, es) && aligned_to(q_out, es);
  }
  const int heads[4] = {H, H_kv, H_kv, H};
  for (int i = H > 0 ? 0 : 1; i < (H > 0 ? 4 : 3); ++i) {
    if (T > 1) rows16 = rows16 && (strides[2 * i] * es) % 16 == 0;
    if (heads[i] > 1) rows16 = rows16 && (strides[2 * i + 1] * es) % 16 == 0;
  }
  if (H > 0 && ((T > 1 && strides[6] == 0) || (H > 1 && strides[7] == 0)))
    return fail(FA_ERR_INVALID, "the output's strides must not be 0");
  if (H > 0 && q == q_out && ((T > 1 && strides[0] != strides[6]) || (H > 1 && strides[1] != strides[7])))
    return fail(FA_ERR_INVALID, "in place, input and output strides must be equal");
  if (!elems) return fail(FA_ERR_ALIGN, "a pointer is not aligned to its elements");
  fa::AppendParams p;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_out = q_out;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.slots = reinterpret_cast<const long long*>(slots);
  p.positions = positions;
  p.inv_freq = inv_freq;
  for (int i = 0; i < 2; ++i) {
    p.qs[i] = strides[i];
    p.ks[i] = strides[2 + i];
    p.vs[i] = strides[4 + i];
    p.qos[i] = strides[6 + i];
  }
  p.k_page = k_page_stride;
  p.v_page = v_page_stride;
  p.n_slots = static_cast<long long>(num_pages) << shift;
  p.T = T;
  p.H = H;
  p.H_kv = H_kv;
  p.d = d;
  p.rot = rotary_dim;
  const int V = rope_vec(es, d, rotary_dim, rows16);
  p.n_rot = rotary_dim / 2 / V;
  const int vecs = (d - rotary_dim) / V, pass = vecs % 2 == 0 ? 2 : 1;
  p.n_units = p.n_rot + vecs / pass;
  p.page_shift = shift;
  p.mag = magnitude;
  const int rows = H + 2 * H_kv;
  p.shape = rope_shape(T, rows, 1, p.n_units, pass, rotary_dim / 2);
  const long long gx = (T + p.shape.tb - 1ll) / p.shape.tb * p.shape.h_blocks * p.shape.u_blocks;
  if (gx > 0x7fffffffll) return fail(FA_ERR_UNSUPPORTED, "grid too large");
  const bool il = (options & FA_ROPE_INTERLEAVED) != 0;
  auto* kern = dtype == FA_BF16 ? (V > 1 ? append_kernel<__nv_bfloat16, 8>(il) : append_kernel<__nv_bfloat16, 1>(il))
                                : (V > 1 ? append_kernel<float, 4>(il) : append_kernel<float, 1>(il));
  return launch_overlapped("fa_paged_append_kernel", kern, dim3(static_cast<unsigned>(gx)), fa::ROPE_THREADS, 0,
                           static_cast<cudaStream_t>(stream), p);
}

size_t fa_paged_workspace_size(int T, int B, int H, int H_kv, int d) {
  if (T < 1 || B < 1 || H < 1 || H_kv < 1 || H % H_kv != 0 || d < 1 || d > 128) return 0;
  return paged_ws_bytes(T, H / H_kv, d);
}

int fa_paged_fwd(const void* q, const void* k_cache, const void* v_cache,
                 const int32_t* block_table, const int32_t* kv_len, const int32_t* cu_q, void* o,
                 float* lse, int T, int B, int H, int H_kv, int d, int64_t q_token_stride,
                 int64_t q_head_stride, int64_t k_page_stride, int64_t v_page_stride,
                 int64_t table_stride, int page_size, int num_pages, int max_pages, int max_q,
                 float scale, int causal, int dtype, void* workspace, size_t workspace_bytes,
                 void* stream) {
  if (T < 0 || B < 1 || H < 1 || d < 1 || num_pages < 1 || max_pages < 1)
    return fail(FA_ERR_INVALID, "T >= 0 and B, H, d, num_pages, max_pages >= 1 required");
  int rc = check_groups(H, H_kv);
  if (rc != FA_OK) return rc;
  if (!(std::isfinite(scale) && scale > 0.f)) return fail(FA_ERR_INVALID, "scale must be finite and > 0");
  const int es = dtype_bytes(dtype);
  if (es == 0) return fail(FA_ERR_INVALID, "unknown dtype %d", dtype);
  if (dtype == FA_BF16 && d != 64 && d != 128)
    return fail(FA_ERR_UNSUPPORTED, "bf16 paged attention supports d in {64, 128}, got %d", d);
  if (d > 128) return fail(FA_ERR_UNSUPPORTED, "paged attention supports d <= 128, got %d", d);
  const int shift = log2_page(page_size);
  if (shift < 0) return fail(FA_ERR_INVALID, "page_size must be a power of two in [16, 1024], got %d", page_size);
  if (T > (1 << 24) || B > (1 << 24)) return fail(FA_ERR_UNSUPPORTED, "T or B too large");
  if ((static_cast<long long>(max_pages) << shift) > (1ll << 30))
    return fail(FA_ERR_UNSUPPORTED, "more than 2^30 positions per request");
  if (static_cast<long long>(H_kv) * num_pages > 0x7fffffffll || (static_cast<long long>(H_kv) << shift) > 0x7fffffffll)
    return fail(FA_ERR_UNSUPPORTED, "cache too large");
  if (B > 1 && table_stride < max_pages) return fail(FA_ERR_INVALID, "block-table rows overlap");
  const long long page_elems = static_cast<long long>(H_kv) * page_size * d;
  if (num_pages > 1 && (k_page_stride < page_elems || v_page_stride < page_elems))
    return fail(FA_ERR_INVALID, "cache pages overlap");
  if ((T > 1 && q_token_stride < 1) || (H > 1 && q_head_stride < 1))
    return fail(FA_ERR_INVALID, "q's strides must be positive");
  if (T == 0) return FA_OK;
  if (!q || !k_cache || !v_cache || !block_table || !kv_len || !cu_q || !o || !lse)
    return fail(FA_ERR_INVALID, "null tensor pointer");
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) || !aligned16(lse))
    return fail(FA_ERR_ALIGN, "tensor pointers must be 16-byte aligned");
  if (!aligned_to(block_table, 4) || !aligned_to(kv_len, 4) || !aligned_to(cu_q, 4))
    return fail(FA_ERR_ALIGN, "a pointer is not aligned to its elements");
  if (dtype == FA_BF16 &&
      ((T > 1 && q_token_stride % 8 != 0) || (H > 1 && q_head_stride % 8 != 0) ||
       (num_pages > 1 && (k_page_stride % 8 != 0 || v_page_stride % 8 != 0))))
    return fail(FA_ERR_ALIGN, "bf16 strides must be multiples of 8 elements");
  {
    const size_t rows_out = static_cast<size_t>(T) * H;
    const size_t q_bytes =
        (static_cast<size_t>(T - 1) * (T > 1 ? q_token_stride : 0) + static_cast<size_t>(H - 1) * (H > 1 ? q_head_stride : 0) + d) * es;
    if (overlap(o, rows_out * d * es, q, q_bytes) || overlap(lse, rows_out * 4, q, q_bytes) ||
        overlap(o, rows_out * d * es, lse, rows_out * 4))
      return fail(FA_ERR_INVALID, "o, lse and q overlap");
  }
  const size_t need = paged_ws_bytes(T, H / H_kv, d);
  if (workspace == nullptr || workspace_bytes < need)
    return fail(FA_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need, workspace_bytes);
  if (!aligned_to(workspace, 256)) return fail(FA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  fa::PagedParams p;
  p.q = q;
  p.k = k_cache;
  p.v = v_cache;
  p.o = o;
  p.lse = lse;
  p.table = block_table;
  p.kv_len = kv_len;
  p.cu_q = cu_q;
  p.table_stride = table_stride;
  p.q_st = q_token_stride;
  p.q_sh = q_head_stride;
  p.k_page = k_page_stride;
  p.v_page = v_page_stride;
  p.T = T;
  p.B = B;
  p.H = H;
  p.group = H / H_kv;
  p.d = d;
  p.vec = d % 4 == 0 && (num_pages == 1 || ((k_page_stride * es) % 16 == 0 && (v_page_stride * es) % 16 == 0));
  p.o_al32 = aligned_to(o, 32) ? 1 : 0;
  p.page_shift = shift;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.causal = causal ? 1 : 0;
  p.scale2 = scale * kLog2e;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // new tokens of a request: the caller's bound, or the mean
  const long long most = max_q > 0 ? std::min(max_q, T) : (static_cast<long long>(T) + B - 1) / B;
  const long long rows = most * p.group;
  return dtype == FA_BF16 ? paged_run_bf16(p, rows, H_kv, page_size, workspace, s)
                          : paged_run_f32(p, rows, H_kv, workspace, s);
}

int fa_rope_packed(const fa_rope_args* args) {
  fa_rope_args a;
  const int rc = unpack(args, &a);
  if (rc != FA_OK) return rc;
  return fa_rope(a.x, a.y, a.positions, a.inv_freq, a.B, a.H, a.N, a.d, a.rotary_dim, a.x_strides,
                 a.y_strides, a.positions_stride, a.magnitude, a.options, a.dtype, a.stream);
}

int fa_paged_plan_packed(const fa_paged_plan_args* args) {
  fa_paged_plan_args a;
  const int rc = unpack(args, &a);
  if (rc != FA_OK) return rc;
  return fa_paged_plan(a.ctx_len, a.new_len, a.free_pages, a.n_free, a.cursor, a.block_table,
                       a.table_stride, a.B, a.max_pages, a.page_size, a.max_tokens, a.cu_q, a.kv_len,
                       a.positions, a.slots, a.counts, a.stream);
}

int fa_paged_append_packed(const fa_paged_append_args* args) {
  fa_paged_append_args a;
  const int rc = unpack(args, &a);
  if (rc != FA_OK) return rc;
  return fa_paged_append(a.q, a.k, a.v, a.q_out, a.k_cache, a.v_cache, a.slots, a.positions,
                         a.inv_freq, a.T, a.H, a.H_kv, a.d, a.rotary_dim, a.strides,
                         a.k_page_stride, a.v_page_stride, a.page_size, a.num_pages, a.magnitude,
                         a.options, a.dtype, a.stream);
}

int fa_paged_fwd_packed(const fa_paged_fwd_args* args) {
  fa_paged_fwd_args a;
  const int rc = unpack(args, &a);
  if (rc != FA_OK) return rc;
  return fa_paged_fwd(a.q, a.k_cache, a.v_cache, a.block_table, a.kv_len, a.cu_q, a.o, a.lse, a.T,
                      a.B, a.H, a.H_kv, a.d, a.q_token_stride, a.q_head_stride, a.k_page_stride,
                      a.v_page_stride, a.table_stride, a.page_size, a.num_pages, a.max_pages, a.max_q,
                      a.scale, a.causal, a.dtype, a.workspace, a.workspace_bytes, a.stream);
}

}  // extern "C"
