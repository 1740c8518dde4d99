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
// What bounds it: HBM -- one read and one write of the tensor.  A block takes a few tokens and
// many heads, so one table of cos and sin in shared memory (a few fp64 operations and two short
// polynomials per entry) serves all of a token's heads, and each thread keeps up to four pairs
// of 16-byte loads in flight.
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
  const double turns = static_cast<double>(pos) * (f * kTwoOverPi);
  const double whole = rint(turns);
  const float x = static_cast<float>(turns - whole) * kHalfPi;
  // the quadrant, from the low bits of the (possibly large) integer
  const int quad = static_cast<int>(static_cast<long long>(whole) & 3ll);
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

// V consecutive elements of T as one load or store (V * sizeof(T) is 16 bytes, or one element).
template <typename T, int V>
struct alignas(V * sizeof(T)) RopeVec {
  T e[V];
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
  float y1, y2;
  if constexpr (!IL || V == 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      rope_pair(to_f<T>(a.e[i]), to_f<T>(b.e[i]), cs[i], y1, y2);
      a.e[i] = from_f<T>(y1);
      b.e[i] = from_f<T>(y2);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      rope_pair(to_f<T>(a.e[2 * i]), to_f<T>(a.e[2 * i + 1]), cs[i], y1, y2);
      a.e[2 * i] = from_f<T>(y1);
      a.e[2 * i + 1] = from_f<T>(y2);
      rope_pair(to_f<T>(b.e[2 * i]), to_f<T>(b.e[2 * i + 1]), cs[V / 2 + i], y1, y2);
      b.e[2 * i] = from_f<T>(y1);
      b.e[2 * i + 1] = from_f<T>(y2);
    }
  }
}

// A head row is cut into units: unit u < n_rot covers two vectors of V elements and V
// frequencies (starting at u V); the units after that cover one pass-through vector each.
template <int V, bool IL>
__device__ __forceinline__ void rope_unit(int u, int n_rot, int rot, int& c0, int& c1) {
  if (u < n_rot) {
    c0 = IL ? 2 * u * V : u * V;
    c1 = IL ? c0 + V : c0 + rot / 2;
  } else {
    c0 = rot + (u - n_rot) * V;
    c1 = -1;
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
  int tb, hc, n_hchunks;     // tokens and heads per block, blocks along the heads
  int heads_inner;           // consecutive threads walk heads before tokens
  float mag, sgn;
};

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_TABLE = 4096;  // (cos, sin) entries per block: tb * rot / 2 at most

template <typename T, int V, bool IL>
__global__ void __launch_bounds__(ROPE_THREADS) fa_rope_kernel(const RopeParams p) {
  __shared__ float2 table[ROPE_TABLE];
  const int half = p.rot / 2;
  const int tblk = static_cast<int>(blockIdx.x) / p.n_hchunks;
  const int hblk = static_cast<int>(blockIdx.x) - tblk * p.n_hchunks;
  const int n0 = tblk * p.tb, h0 = hblk * p.hc;
  const int nt = min(p.tb, p.N - n0), nh = min(p.hc, p.H - h0);
  const int total = nt * nh * p.n_units;
  using Vec = RopeVec<T, V>;
  for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
    const int32_t* pos = p.positions == nullptr ? nullptr : p.positions + b * p.pos_sb;
    for (int e = threadIdx.x; e < nt * half; e += ROPE_THREADS) {
      const int t = e / half, i = e - t * half;
      table[e] = rope_cos_sin(pos == nullptr ? n0 + t : pos[n0 + t], p.inv_freq[i], p.mag, p.sgn);
    }
    __syncthreads();
    const T* xb = static_cast<const T*>(p.x) + b * p.xs[0];
    T* yb = static_cast<T*>(p.y) + b * p.ys[0];
    constexpr int DEPTH = 4;
    for (int e0 = threadIdx.x; e0 < total; e0 += DEPTH * ROPE_THREADS) {
      Vec va[DEPTH], vb[DEPTH];
      int c0[DEPTH], c1[DEPTH], tt[DEPTH], uu[DEPTH];
      long long yo[DEPTH];
#pragma unroll
      for (int k = 0; k < DEPTH; ++k) {
        const int e = e0 + k * ROPE_THREADS;
        if (e >= total) break;
        const int r = e / p.n_units;
        uu[k] = e - r * p.n_units;
        int h;
        if (p.heads_inner) {
          tt[k] = r / nh;
          h = r - tt[k] * nh;
        } else {
          h = r / nt;
          tt[k] = r - h * nt;
        }
        rope_unit<V, IL>(uu[k], p.n_rot, p.rot, c0[k], c1[k]);
        const T* row = xb + (h0 + h) * p.xs[1] + (n0 + tt[k]) * p.xs[2];
        yo[k] = (h0 + h) * p.ys[1] + (n0 + tt[k]) * p.ys[2];
        va[k] = *reinterpret_cast<const Vec*>(row + c0[k]);
        if (c1[k] >= 0) vb[k] = *reinterpret_cast<const Vec*>(row + c1[k]);
      }
#pragma unroll
      for (int k = 0; k < DEPTH; ++k) {
        if (e0 + k * ROPE_THREADS >= total) break;
        if (c1[k] >= 0) {
          rope_turn<T, V, IL>(va[k], vb[k], table + tt[k] * half + uu[k] * V);
          *reinterpret_cast<Vec*>(yb + yo[k] + c1[k]) = vb[k];
        }
        *reinterpret_cast<Vec*>(yb + yo[k] + c0[k]) = va[k];
      }
    }
    __syncthreads();  // the table is rewritten for the next batch entry
  }
}

}  // namespace fa
