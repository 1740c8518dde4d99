// fa_rope.cuh -- rotary positions: the rotation kernel (forward and its transpose) and the
// rotation helpers that the cache append shares.
//
// A token at position p turns the pair (x1, x2) of frequency f by the angle a = p f:
//     y1 = m (x1 cos a - x2 sin a),   y2 = m (x2 cos a + x1 sin a),
// m a constant magnitude (1 unless the frequencies are scaled by parts).  The pairs of the
// first `rot` columns are (i, i + rot/2) or, interleaved, (2i, 2i + 1); the other columns pass
// through.  The map is m times an orthogonal matrix, so its gradient is the same kernel with
// the angle's sign turned.
//
// Angles: p f reaches 10^6 radians and more, where fp32 has lost the angle.  The number of
// quarter turns p f 2/pi is formed and reduced to [-1/2, 1/2] in fp64 (absolute error below
// 10^-9 up to p f = 10^6), and only the remainder goes to fp32.
//
// What bounds it: HBM -- one read and one write of the tensor -- and at small sizes the launch.
// A thread keeps one 16-byte pair of columns of one token and walks over heads: its cos and sin
// stay in registers, no index is divided in the loop, and the loads of four heads are in flight
// at once, the first of them already while the block's table of cos and sin is being made.
// Measured, inputs not in L2: 16 heads x 16384 tokens, d = 128, bf16 (134 MB): 25 us, 5.3 TB/s;
// 8 x 12 x 1024, d = 64 (25 MB): 9 us; one thread per element with its own cos and sin: 88 and 17.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "fa_simt.cuh"

namespace fa {

// cos and sin of p f, times `mag` (the sign of sin times `sgn`).  Quarter turns in fp64, then
// the Taylor polynomials of sin and cos on [-pi/4, pi/4]: remainders below 2e-9 (x^11 / 11!)
// and 2e-10 (x^12 / 12!), under half an fp32 ulp of the larger of the two.
__device__ __forceinline__ float2 rope_cos_sin(int pos, double f, float mag, float sgn) {
  constexpr double kTwoOverPi = 0.63661977236758134308;
  constexpr float kHalfPi = 1.57079632679489661923f;
  constexpr double kRound = 6755399441055744.0;  // 1.5 * 2^52: adding it rounds to an integer
  const double turns = static_cast<double>(pos) * (f * kTwoOverPi);
  const double shifted = turns + kRound;
  const float x = static_cast<float>(turns - (shifted - kRound)) * kHalfPi;
  const int quad = __double2loint(shifted) & 3;   // whose low bits are then the integer's
  const float x2 = x * x;
  float s = fmaf(x2, 2.7557319e-6f, -1.9841270e-4f);
  s = fmaf(s, x2, 8.3333333e-3f);
  s = fmaf(s, x2, -1.6666667e-1f);
  s = fmaf(s * x2, x, x);
  float c = fmaf(x2, -2.7557319e-7f, 2.4801587e-5f);
  c = fmaf(c, x2, -1.3888889e-3f);
  c = fmaf(c, x2, 4.1666667e-2f);
  c = fmaf(c, x2, -0.5f);
  c = fmaf(c, x2, 1.0f);
  const float cs = (quad & 1) ? s : c;
  const float sn = (quad & 1) ? c : s;
  return make_float2(((quad == 1 || quad == 2) ? -cs : cs) * mag,
                     ((quad >= 2) ? -sn : sn) * (mag * sgn));
}

// V consecutive elements as one load or store: one element, or 16 bytes held as 32-bit words (two
// bf16 to a word, the first in the low half).
template <typename T, int V>
struct RopeVec {
  T e[V];
  __device__ __forceinline__ float get(int i) const { return to_f<T>(e[i]); }
  __device__ __forceinline__ void set2(int i, float x, float y) {  // elements i, i + 1
    e[i] = from_f<T>(x);
    e[i + 1] = from_f<T>(y);
  }
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (V == 1) {
      e[0] = *p;
    } else {
      const float4 v = *reinterpret_cast<const float4*>(p);
      e[0] = v.x, e[1] = v.y, e[2] = v.z, e[3] = v.w;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (V == 1) *p = e[0];
    else *reinterpret_cast<float4*>(p) = make_float4(e[0], e[1], e[2], e[3]);
  }
};
template <>
struct RopeVec<__nv_bfloat16, 8> {
  uint4 w;
  __device__ __forceinline__ uint32_t word(int i) const {
    return i == 0 ? w.x : (i == 1 ? w.y : (i == 2 ? w.z : w.w));
  }
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float((i & 1) ? word(i >> 1) & 0xffff0000u : word(i >> 1) << 16);
  }
  __device__ __forceinline__ void set2(int i, float x, float y) {
    const uint32_t v = pack_bf16x2(x, y);
    if (i == 0) w.x = v;
    else if (i == 2) w.y = v;
    else if (i == 4) w.z = v;
    else w.w = v;
  }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = w; }
};

// One pair; the rounding of each product is spelled out, so that every path (layouts, vector
// widths, the cache append) gives the same bits.
__device__ __forceinline__ void rope_pair(float x1, float x2, float2 w, float& y1, float& y2) {
  y1 = fmaf(x1, w.x, -__fmul_rn(x2, w.y));
  y2 = fmaf(x2, w.x, __fmul_rn(x1, w.y));
}

// Turns the pairs held in (a, b): half layout pairs a[i] with b[i]; interleaved pairs
// neighbours inside a and inside b (V = 1: a with b).  cs points at the V (cos, sin) entries.
template <typename T, int V, bool IL>
__device__ __forceinline__ void rope_turn(RopeVec<T, V>& a, RopeVec<T, V>& b,
                                          const float2* __restrict__ cs) {
  if constexpr (V == 1) {
    float y1, y2;
    rope_pair(a.get(0), b.get(0), cs[0], y1, y2);
    a.e[0] = from_f<T>(y1);
    b.e[0] = from_f<T>(y2);
  } else if constexpr (!IL) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      float y1, y2, z1, z2;
      rope_pair(a.get(i), b.get(i), cs[i], y1, y2);
      rope_pair(a.get(i + 1), b.get(i + 1), cs[i + 1], z1, z2);
      a.set2(i, y1, z1);
      b.set2(i, y2, z2);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      float y1, y2;
      rope_pair(a.get(i), a.get(i + 1), cs[i / 2], y1, y2);
      a.set2(i, y1, y2);
      rope_pair(b.get(i), b.get(i + 1), cs[V / 2 + i / 2], y1, y2);
      b.set2(i, y1, y2);
    }
  }
}

// A head row is cut into units: unit u < n_rot covers two vectors of V elements and V
// frequencies (starting at u V); the units after that cover two pass-through vectors, or one
// where their number is odd.
template <int V, bool IL>
__device__ __forceinline__ void rope_unit(int u, int n_rot, int rot, int pass, int& c0, int& c1) {
  if (u < n_rot) {
    c0 = IL ? 2 * u * V : u * V;
    c1 = IL ? c0 + V : c0 + rot / 2;
  } else {
    c0 = rot + (u - n_rot) * pass * V;
    c1 = pass == 2 ? c0 + V : -1;
  }
}

// How a block is laid over (units, tokens, heads), chosen by the host: `uw` units of a head row
// x `tb` tokens x `hs` heads are its threads, and each thread walks over `hpt` heads, hs apart.
struct RopeShape {
  int uw, tb, hs, hpt;
  int pass;                // pass-through vectors per unit: 1 or 2
  int u_blocks, h_blocks;  // blocks along the units and the heads
};

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_TABLE = 2048;  // (cos, sin) entries: tb * rot / 2 at most
constexpr int ROPE_DEPTH = 4;     // heads loaded at once

// The block's work.  `rows` gives the head rows of this thread's token, after prepare(token): where
// head h is read and written, whether it is stored at all and whether it is turned.
template <typename T, int V, bool IL, typename Rows>
__device__ __forceinline__ void rope_block(const RopeShape& sh, int N, int n_heads, int rot, int n_rot,
                                           int n_units, const int32_t* __restrict__ pos,
                                           const double* __restrict__ inv_freq, float mag, float sgn,
                                           Rows& rows) {
  __shared__ float2 table[ROPE_TABLE];
  using Vec = RopeVec<T, V>;
  grid_dep_wait();  // launched to overlap the kernel before, as the next one may overlap this
  grid_dep_launch();
  const int half = rot / 2;
  int blk = blockIdx.x;
  const int ub = blk % sh.u_blocks;
  blk /= sh.u_blocks;
  const int hb = blk % sh.h_blocks, tb0 = blk / sh.h_blocks * sh.tb;
  const int tid = threadIdx.x;
  const int u = ub * sh.uw + tid % sh.uw;
  const int r = tid / sh.uw;
  const int t = r % sh.tb, slot = r / sh.tb;
  const int n = tb0 + t;
  const bool active = slot < sh.hs && n < N && u < n_units;
  const int h_end = min(n_heads, (hb + 1) * sh.hs * sh.hpt);
  int h = hb * sh.hs * sh.hpt + slot;
  int c0 = 0, c1 = -1;
  rope_unit<V, IL>(u, n_rot, rot, sh.pass, c0, c1);
  if (active) rows.prepare(n);
  Vec va[ROPE_DEPTH], vb[ROPE_DEPTH];
  auto load = [&]() {
#pragma unroll
    for (int k = 0; k < ROPE_DEPTH; ++k) {
      const int hk = h + k * sh.hs;
      if (active && hk < h_end) {  // a row that is not stored is read all the same: no wait for its slot
        const T* src = rows.src(hk);
        va[k].load(src + c0);
        if (c1 >= 0) vb[k].load(src + c1);
      }
    }
  };
  load();
  float2 cs[V];
  if (half > 0) {
    const int nt = min(sh.tb, N - tb0);
    for (int e = tid; e < nt * half; e += ROPE_THREADS) {
      const int tt = e / half, i = e - tt * half;
      table[e] = rope_cos_sin(pos == nullptr ? tb0 + tt : pos[tb0 + tt], inv_freq[i], mag, sgn);
    }
    __syncthreads();
    if (active && u < n_rot) {
#pragma unroll
      for (int i = 0; i < V; ++i) cs[i] = table[t * half + u * V + i];
    }
  }
  if (!active) return;
  while (true) {
#pragma unroll
    for (int k = 0; k < ROPE_DEPTH; ++k) {
      const int hk = h + k * sh.hs;
      if (hk >= h_end || !rows.stored(hk)) continue;
      T* dst = rows.dst(hk);
      if (c1 >= 0) {
        if (u < n_rot && rows.turned(hk)) rope_turn<T, V, IL>(va[k], vb[k], cs);
        vb[k].store(dst + c1);
      }
      va[k].store(dst + c0);
    }
    h += ROPE_DEPTH * sh.hs;
    if (h >= h_end) break;
    load();
  }
}

struct RopeParams {
  const void* x;
  void* y;
  const int32_t* positions;  // or nullptr: 0 .. N-1
  const double* inv_freq;    // [rot/2]
  long long xs[3], ys[3];    // strides of batch, head, token in elements
  long long pos_sb;          // positions' batch stride
  int B, H, N, rot;
  int n_rot, n_units;        // rotated units, all units of a head row
  RopeShape shape;
  float mag, sgn;
};

template <typename T>
struct RopeRows {
  const T* x;
  T* y;
  long long xh, yh, xn, yn;
  __device__ __forceinline__ void prepare(int n) {
    x += n * xn;
    y += n * yn;
  }
  __device__ __forceinline__ const T* src(int h) const { return x + h * xh; }
  __device__ __forceinline__ T* dst(int h) const { return y + h * yh; }
  __device__ __forceinline__ bool stored(int) const { return true; }
  __device__ __forceinline__ bool turned(int) const { return true; }
};

template <typename T, int V, bool IL>
__global__ void __launch_bounds__(ROPE_THREADS, 3) fa_rope_kernel(const RopeParams p) {
  const int b = blockIdx.y + gridDim.y * blockIdx.z;
  if (b >= p.B) return;
  RopeRows<T> rows = {static_cast<const T*>(p.x) + b * p.xs[0], static_cast<T*>(p.y) + b * p.ys[0],
                      p.xs[1], p.ys[1], p.xs[2], p.ys[2]};
  rope_block<T, V, IL>(p.shape, p.N, p.H, p.rot, p.n_rot, p.n_units,
                       p.positions == nullptr ? nullptr : p.positions + b * p.pos_sb, p.inv_freq,
                       p.mag, p.sgn, rows);
}

}  // namespace fa
