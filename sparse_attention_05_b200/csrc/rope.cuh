// rope.cuh -- rotary positions on a part of every head.
//
// Pair i of the rotated part (dims (2i, 2i + 1) of it, or (i, i + rot/2) in the half
// layout) is turned by the angle position * freq_i and scaled by `magnitude`:
//   (a, b) -> magnitude * (a cos - b sin, a sin + b cos)
// and by the transposed matrix (sin -> -sin) in the backward pass. MLA gives 64 of a
// query's dims to it (DeepSeek-V3.2-Exp technical report, Appendix A: the rope part).
//
// The kernel moves 2 x (row bytes) and computes three flops a dim, so memory bounds it.
// The angle, its sine and its cosine are formed in fp64: at position 10^6 an fp32 product
// would be off by 0.06 rad. A thread owns one unit (a run of dims with their partners, or as
// many dims to copy) of one row and takes it through several heads with its sines and cosines
// in registers; the block forms each of them once, in shared memory, while the first loads
// are on their way. What is left is bytes in flight: five blocks an SM whose threads have two
// runs of 16 B under way each carry 8192 rows of 64 bf16 heads (half of 128 dims rotated) in
// 51 us (55 with runs unpacked as they arrived; then four blocks with four runs took 63, three
// 67).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace dsa {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxRot = 512;     // rotated dims of a head
constexpr int kRopeMaxDim = 32768;

struct RopeParams {
  const void* x;
  void* out;
  const int32_t* positions;  // [rows]
  const double* freqs;       // [half] radians per position
  int64_t x_row, x_head, o_row, o_head;  // strides in elements
  int64_t rows;
  int32_t heads, half, rot_begin;
  int32_t copied;            // dims of a head to copy (0 in place)
  int32_t rot_units, units;  // of a head: rotated, and with those to copy
  int32_t row_blocks;        // blocks that share a row's units (1: a block takes whole rows)
  int32_t block_rows;        // rows of a block (row_blocks = 1)
  int32_t block_units;       // (row, unit) pairs of a block; kRopeThreads / block_units heads
                             // go side by side
  int32_t turns;             // heads of a thread
  float magnitude, sign;     // sign = -1: transposed
};

// cos and sin of pos * freq, times magnitude, in fp64 and rounded to fp32 once. Less than an
// eighth of a turn is left after the quarters (q); the Taylor series to x^13 and x^14 are
// within 2^-45 there. (65536 appended tokens take 39 us with them, 41 with the library's pair.)
__device__ __forceinline__ float2 rope_turn(int32_t pos, double freq, float magnitude) {
  double turns = (double)pos * (freq * 0.15915494309189533577);
  turns = 4.0 * (turns - rint(turns));
  const double q = rint(turns);
  const double x = (turns - q) * 1.57079632679489661923, y = -x * x;
  double s = 1.0 / 6227020800.0, c = 1.0 / 87178291200.0;
  s = fma(s, y, 1.0 / 39916800.0), c = fma(c, y, 1.0 / 479001600.0);
  s = fma(s, y, 1.0 / 362880.0), c = fma(c, y, 1.0 / 3628800.0);
  s = fma(s, y, 1.0 / 5040.0), c = fma(c, y, 1.0 / 40320.0);
  s = fma(s, y, 1.0 / 120.0), c = fma(c, y, 1.0 / 720.0);
  s = fma(s, y, 1.0 / 6.0), c = fma(c, y, 1.0 / 24.0);
  s = fma(s, y, 1.0), c = fma(c, y, 0.5);
  s *= x, c = fma(c, y, 1.0);
  const int quarter = (int)q & 3;
  const float fs = (float)((quarter & 1 ? c : s) * magnitude);
  const float fc = (float)((quarter & 1 ? s : c) * magnitude);
  return make_float2(quarter == 1 || quarter == 2 ? -fc : fc, quarter >= 2 ? -fs : fs);
}

// A pair turned: the products and their sum are rounded to fp32 one by one, not contracted, so
// that a rotated value has the same bits wherever it is formed (an appended key's scale and
// codes hang on the last bit of its largest value).
__device__ __forceinline__ float2 rope_pair(float a, float b, float2 cs) {
  return make_float2(__fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y)),
                     __fadd_rn(__fmul_rn(a, cs.y), __fmul_rn(b, cs.x)));
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

// A unit of a head: one run of V dims (interleaved, V > 1), else two runs of V dims, `gap`
// apart. Rotated: a run of pairs, or the firsts and seconds of V pairs.
template <typename T, int V, bool kInterleaved>
struct RopeUnit {
  static constexpr bool kTwo = !kInterleaved || V == 1;
  static constexpr int kPairs = kTwo ? V : V / 2;
  RopeVec<T, V> lo, hi;
  __device__ __forceinline__ void load(const T* x, int gap, bool two) {
    lo = *reinterpret_cast<const RopeVec<T, V>*>(x);
    if (kTwo && two) hi = *reinterpret_cast<const RopeVec<T, V>*>(x + gap);
  }
  __device__ __forceinline__ void store(T* out, int gap, bool two) const {
    *reinterpret_cast<RopeVec<T, V>*>(out) = lo;
    if (kTwo && two) *reinterpret_cast<RopeVec<T, V>*>(out + gap) = hi;
  }
  // The runs as they were loaded: 16-bit elements are not unpacked before this point, where
  // they would take twice the registers.
  __device__ __forceinline__ void packed() {
    if constexpr (sizeof(lo) == 16) {
      auto tie = [](RopeVec<T, V>& v) {
        uint4 w = *reinterpret_cast<uint4*>(&v);
        asm volatile("" : "+r"(w.x), "+r"(w.y), "+r"(w.z), "+r"(w.w));
        v = *reinterpret_cast<RopeVec<T, V>*>(&w);
      };
      tie(lo);
      if (kTwo) tie(hi);
    }
  }
  __device__ __forceinline__ void turn(const float2 (&t)[kPairs]) {
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      T& first = kTwo ? lo.v[j] : lo.v[(2 * j) % V];
      T& second = kTwo ? hi.v[j] : lo.v[(2 * j + 1) % V];
      const float2 r = rope_pair(rope_to_float(first), rope_to_float(second), t[j]);
      first = rope_from_float<T>(r.x);
      second = rope_from_float<T>(r.y);
    }
  }
};

template <typename T, int V, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, 5) rope_kernel(const RopeParams p) {
  using Unit = RopeUnit<T, V, kInterleaved>;
  constexpr int kPairs = Unit::kPairs;
  constexpr int kRun = Unit::kTwo ? 2 * V : V;     // dims of a unit
  constexpr int kHeads = Unit::kTwo ? 1 : 2;       // in flight: two runs of a thread
  const int slot = threadIdx.x / p.block_units, c = threadIdx.x - slot * p.block_units;
  const int slots = kRopeThreads / p.block_units;
  int64_t row;
  int u;
  if (p.row_blocks == 1) {
    const int r = c / p.units;
    row = (int64_t)blockIdx.x * p.block_rows + r;
    u = c - r * p.units;
  } else {
    row = blockIdx.x / p.row_blocks;
    u = (int)(blockIdx.x - row * p.row_blocks) * p.block_units + c;
  }
  int h = (int)blockIdx.y * p.turns * slots + slot;
  const int end = min(p.heads, h - slot + p.turns * slots);
  const bool active = slot < slots && row < p.rows && u < p.units && h < end;
  const bool turned = active && u < p.rot_units;
  int d, gap;
  bool two = true;
  if (turned) {
    d = p.rot_begin + u * (kInterleaved ? kRun : V);
    gap = kInterleaved ? 1 : p.half;
  } else {  // dims to copy, numbered without the rotated part: a run of each half of them
    const int e = (u - p.rot_units) * V, next = e + (p.units - p.rot_units) * V;
    auto dim = [&](int i) { return i < p.rot_begin ? i : i + 2 * p.half; };
    d = dim(e);
    gap = dim(next) - d;
    two = next < p.copied;
  }
  const T* x = reinterpret_cast<const T*>(p.x) + row * p.x_row + d;
  T* out = reinterpret_cast<T*>(p.out) + row * p.o_row + d;
  Unit e[kHeads];
  auto load = [&] {
#pragma unroll
    for (int j = 0; j < kHeads; ++j)
      if (h + j * slots < end) e[j].load(x + (h + j * slots) * p.x_head, gap, two);
  };
  if (active) load();
  // block_rows * half <= kRopeThreads * kPairs entries: a row has half / kPairs units or more
  __shared__ float2 table[kRopeThreads * kPairs];
  const int64_t row0 = p.row_blocks == 1 ? (int64_t)blockIdx.x * p.block_rows : row;
  const int entries = (int)min((int64_t)p.block_rows, p.rows - row0) * p.half;
  for (int i = threadIdx.x; i < entries; i += kRopeThreads) {
    const int r = i / p.half;
    float2 t = rope_turn(__ldg(p.positions + row0 + r), __ldg(p.freqs + i - r * p.half),
                         p.magnitude);
    t.y *= p.sign;
    table[i] = t;
  }
  __syncthreads();
  if (!active) return;
#pragma unroll
  for (int j = 0; j < kHeads; ++j) e[j].packed();
  float2 t[kPairs];
  if (turned) {
#pragma unroll
    for (int j = 0; j < kPairs; ++j) t[j] = table[(int)(row - row0) * p.half + u * kPairs + j];
  }
  while (true) {
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      if (h + j * slots < end) {
        if (turned) e[j].turn(t);
        e[j].store(out + (h + j * slots) * p.o_head, gap, two);
      }
    }
    h += kHeads * slots;
    if (h >= end) break;
    load();
  }
}

}  // namespace dsa
