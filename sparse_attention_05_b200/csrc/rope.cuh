// rope.cuh -- rotary positions on a part of every head.
//
// Pair i of the rotated part (dims (2i, 2i + 1) of it, or (i, i + rot/2) in the half
// layout) is turned by the angle position * freq_i and scaled by `magnitude`:
//   (a, b) -> magnitude * (a cos - b sin, a sin + b cos)
// and by the transposed matrix (sin -> -sin) in the backward pass. MLA gives 64 of a
// query's dims to it (DeepSeek-V3.2-Exp technical report, Appendix A: the rope part).
//
// The kernel moves 2 x (row bytes) and computes three flops a dim, so memory bounds it.
// The angle is formed in fp64 turns and reduced to [-1/2, 1/2] before it becomes fp32:
// at position 10^6 an fp32 product would be off by 0.06 rad. That costs one fp64
// multiplication per (row, pair); every head of the row reads the sine and cosine from
// shared memory.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace dsa {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxRows = 32;     // rows of one block
constexpr int kRopeMaxRot = 512;     // rotated dims of a head
constexpr int kRopeTable = 2048;     // (row, pair) entries of one block's table, 16 KB

struct RopeParams {
  const void* x;
  void* out;
  const int32_t* positions;  // [rows]
  const double* freqs;       // [half] radians per position
  int64_t x_row, x_head, o_row, o_head;  // strides in elements
  int64_t rows;
  int32_t heads, half, rot_begin, dim;
  int32_t rows_per_block, heads_per_block;
  int32_t copy;              // dims outside the rotated part are copied
  float magnitude, sign;     // sign = -1: transposed
};

// cos and sin of pos * freq, times magnitude.
__device__ __forceinline__ float2 rope_turn(int32_t pos, double freq, float magnitude) {
  double turns = (double)pos * (freq * 0.15915494309189533577);
  turns -= rint(turns);
  float s, c;
  sincospif(2.0f * (float)turns, &s, &c);
  return make_float2(c * magnitude, s * magnitude);
}

template <typename T> __device__ __forceinline__ float rope_to_float(T v);
template <> __device__ __forceinline__ float rope_to_float(float v) { return v; }
template <> __device__ __forceinline__ float rope_to_float(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float rope_to_float(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <typename T> __device__ __forceinline__ T rope_from_float(float v);
template <> __device__ __forceinline__ float rope_from_float(float v) { return v; }
template <> __device__ __forceinline__ __half rope_from_float(float v) {
  return __float2half_rn(v);
}
template <> __device__ __forceinline__ __nv_bfloat16 rope_from_float(float v) {
  return __float2bfloat16_rn(v);
}

// V elements moved as one access (16 bytes, or one element).
template <typename T, int V>
struct alignas(V * sizeof(T)) RopeVec {
  T v[V];
};

// A unit is what one thread does at once: V dims of the rotated part with their
// partners (interleaved: one run of max(V, 2) dims; half layout: two runs of V), or V
// dims to copy.
template <typename T, int V, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  using Vec = RopeVec<T, V>;
  constexpr int kPairs = kInterleaved ? (V > 1 ? V / 2 : 1) : V;
  __shared__ float2 table[kRopeTable];
  const int64_t row0 = (int64_t)blockIdx.x * p.rows_per_block;
  const int nrows = (int)min((int64_t)p.rows_per_block, p.rows - row0);
  const int h0 = blockIdx.y * p.heads_per_block;
  const int nheads = min(p.heads_per_block, p.heads - h0);
  for (int i = threadIdx.x; i < nrows * p.half; i += kRopeThreads) {
    const int r = i / p.half, j = i - r * p.half;
    float2 t = rope_turn(__ldg(p.positions + row0 + r), __ldg(p.freqs + j), p.magnitude);
    t.y *= p.sign;
    table[i] = t;
  }
  __syncthreads();
  const int rot_units = p.half / kPairs;
  const int units = rot_units + (p.copy ? (p.dim - 2 * p.half) / V : 0);
  const int total = nrows * nheads * units;
  const T* x = reinterpret_cast<const T*>(p.x);
  T* out = reinterpret_cast<T*>(p.out);
  for (int i = threadIdx.x; i < total; i += kRopeThreads) {
    const int rh = i / units, u = i - rh * units;
    const int r = rh / nheads, h = h0 + rh - r * nheads;
    const T* xs = x + (row0 + r) * p.x_row + h * p.x_head;
    T* os = out + (row0 + r) * p.o_row + h * p.o_head;
    if (u >= rot_units) {
      int d = (u - rot_units) * V;
      if (d >= p.rot_begin) d += 2 * p.half;
      *reinterpret_cast<Vec*>(os + d) = *reinterpret_cast<const Vec*>(xs + d);
      continue;
    }
    const float2* t = table + r * p.half + u * kPairs;
    if constexpr (kInterleaved) {
      const int d = p.rot_begin + u * 2 * kPairs;
      T e[2 * kPairs];
      if constexpr (V > 1) {
        *reinterpret_cast<Vec*>(e) = *reinterpret_cast<const Vec*>(xs + d);
      } else {
        e[0] = xs[d];
        e[1] = xs[d + 1];
      }
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        const float a = rope_to_float(e[2 * j]), b = rope_to_float(e[2 * j + 1]);
        e[2 * j] = rope_from_float<T>(a * t[j].x - b * t[j].y);
        e[2 * j + 1] = rope_from_float<T>(a * t[j].y + b * t[j].x);
      }
      if constexpr (V > 1) {
        *reinterpret_cast<Vec*>(os + d) = *reinterpret_cast<const Vec*>(e);
      } else {
        os[d] = e[0];
        os[d + 1] = e[1];
      }
    } else {
      const int d = p.rot_begin + u * V;
      Vec lo = *reinterpret_cast<const Vec*>(xs + d);
      Vec hi = *reinterpret_cast<const Vec*>(xs + d + p.half);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float a = rope_to_float(lo.v[j]), b = rope_to_float(hi.v[j]);
        lo.v[j] = rope_from_float<T>(a * t[j].x - b * t[j].y);
        hi.v[j] = rope_from_float<T>(a * t[j].y + b * t[j].x);
      }
      *reinterpret_cast<Vec*>(os + d) = lo;
      *reinterpret_cast<Vec*>(os + d + p.half) = hi;
    }
  }
}

}  // namespace dsa
