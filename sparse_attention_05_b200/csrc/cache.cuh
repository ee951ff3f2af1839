// cache.cuh -- new tokens into the two per-token caches, and the tokens that stay
// moved together.
//
// Append: the caches hold what the path reads: the latent row [512 latent | 64 rope
// dims, rotated] in bf16, and the 128-d indexer key in E4M3 with one fp32 scale per
// token (the two caches of "DeepSeek-V3.2开源技术报告", DSA principle section). The key is
// quantized from its fp32 rotated value:
//   s = max(amax |k|, 2^-120) / 448,  code = E4M3(k / s)
// (round to nearest even), the rule the indexer applies to its queries. Both divisions
// are IEEE fp32: a reciprocal would move codes at the rounding borders. A token is 1408 B
// read and 1284 B written, so memory bounds the large calls and one round trip the small
// ones. One warp a token: lane l owns pair l of the 32 rotated pairs of both rows, so
// each lane forms one sine and cosine.
//
// Compact: slot i of the destination takes slot kept[i] of the source.
#pragma once

#include <cuda_bf16.h>

#include "ptx.cuh"
#include "rope.cuh"
#include "rows.cuh"

namespace dsa {

constexpr int kAppendWarps = 4;

struct AppendParams {
  const __nv_bfloat16* latent;  // [T] rows of 576, stride latent_stride
  const __nv_bfloat16* keys;    // [T] rows of 128, stride key_stride
  const int32_t* positions;     // [T] or nullptr (the slot)
  const double* freqs;          // [32]
  uint8_t* kv;                  // latent cache rows of 1152 B
  uint8_t* k_idx;               // key rows of 128 B
  float* k_scale;
  const int32_t* block_table;
  const int32_t* seqlens;
  const int32_t* q_start;
  int64_t latent_stride, key_stride, window_rows;
  int32_t max_ctx, q_per_seq, num_q, row_begin, row_count;
  int32_t paged, page_size, max_pages, num_pages;
  int32_t latent_interleaved, key_rotated, key_interleaved;
  float magnitude;
};

__global__ void __launch_bounds__(kAppendWarps * 32) cache_append_kernel(const AppendParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t local = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  if (local >= p.window_rows) return;
  const int b = (int)(local / p.row_count);
  const int qi = p.row_begin + (int)(local - (int64_t)b * p.row_count);
  const SeqRows R = seq_rows(p.q_start, p.seqlens, b, p.q_per_seq, p.num_q, p.max_ctx);
  if (!R.ok) {
    if (lane == 0) report_error(kErrBounds);
    return;
  }
  if (qi >= R.q_len) return;
  const int64_t t = R.t0 + qi;
  const int slot = R.seqlen - R.q_len + qi;
  int64_t row = (int64_t)b * p.max_ctx + slot;
  if (p.paged) {
    const int pg = __ldg(p.block_table + (int64_t)b * p.max_pages + slot / p.page_size);
    if (pg < 0 || pg >= p.num_pages) {
      if (lane == 0) report_error(kErrBounds);
      return;
    }
    row = (int64_t)pg * p.page_size + slot % p.page_size;
  }
  const __nv_bfloat16* lat = p.latent + t * p.latent_stride;
  const __nv_bfloat16* key = p.keys + t * p.key_stride;
  uint4* dst = reinterpret_cast<uint4*>(p.kv + row * 1152);
  const uint4 n0 = __ldg(reinterpret_cast<const uint4*>(lat) + lane);
  const uint4 n1 = __ldg(reinterpret_cast<const uint4*>(lat) + 32 + lane);
  // the lane's pair of each rotated part, and its two plain key dims
  const int l0 = p.latent_interleaved ? 2 * lane : lane, l1 = p.latent_interleaved ? l0 + 1 : lane + 32;
  const int k0 = p.key_interleaved ? 2 * lane : lane, k1 = p.key_interleaved ? k0 + 1 : lane + 32;
  const float la = __bfloat162float(lat[512 + l0]), lb = __bfloat162float(lat[512 + l1]);
  float ka = __bfloat162float(key[k0]), kb = __bfloat162float(key[k1]);
  const float2 kc = __bfloat1622float2(
      *reinterpret_cast<const __nv_bfloat162*>(key + 64 + 2 * lane));
  const float2 cs = rope_turn(p.positions ? __ldg(p.positions + t) : slot, __ldg(p.freqs + lane),
                              p.magnitude);
  dst[lane] = n0;
  dst[32 + lane] = n1;
  __nv_bfloat16* rope = reinterpret_cast<__nv_bfloat16*>(dst) + 512;
  const float2 l = rope_pair(la, lb, cs);
  rope[l0] = __float2bfloat16_rn(l.x);
  rope[l1] = __float2bfloat16_rn(l.y);
  if (p.key_rotated) {
    const float2 k = rope_pair(ka, kb, cs);
    ka = k.x, kb = k.y;
  }
  // the largest magnitude by its bits: a NaN anywhere makes the scale a NaN
  auto bits = [](float v) { return __float_as_uint(v) & 0x7fffffffu; };
  const uint32_t m = __reduce_max_sync(0xffffffffu, max(max(bits(ka), bits(kb)),
                                                        max(bits(kc.x), bits(kc.y))));
  const float amax = __uint_as_float(m);
  const float scale = __fdiv_rn(amax < 0x1p-120f ? 0x1p-120f : amax, 448.0f);
  const uint16_t rot = cvt_e4m3x2(__fdiv_rn(ka, scale), __fdiv_rn(kb, scale));
  uint8_t* codes = p.k_idx + row * 128;
  codes[k0] = (uint8_t)rot;
  codes[k1] = (uint8_t)(rot >> 8);
  *reinterpret_cast<uint16_t*>(codes + 64 + 2 * lane) =
      cvt_e4m3x2(__fdiv_rn(kc.x, scale), __fdiv_rn(kc.y, scale));
  if (lane == 0) p.k_scale[row] = scale;
}

// ---- compact ---------------------------------------------------------------------------
// Moving in place: kept is ascending, so kept[i] >= i, and a chunk's destinations lie
// below every later chunk's sources. A cluster of CTAs takes a column slice of a sequence
// through its chunks in order: it loads a chunk into shared memory, waits at the cluster's
// barrier until all its CTAs have theirs, and stores it, while the next chunk's loads are under
// way or done. The slices are independent of each other: nine of 128 B of the latent
// row, one of the key row, one of scale and mass.
// Into other pages the rows need no order: a warp takes up to 16 of them whole, four at a time
// (1280 B of latent and key in 16-byte pieces, ten of a lane in flight): 48 sequences of 8192
// kept tokens take 156 us, and 186 in slices, which touch every row's DRAM page nine times.
constexpr int kCompactThreads = 256;
constexpr int kCompactBlock = kCompactThreads + 32;  // in place: and a warp for the barriers
constexpr int kCompactSlices = 11;
// A CTA's chunk in place: 256 or 512 rows (one or two entries of a lane), two or three of them
// in shared memory.
constexpr int kCompactRows = kCompactThreads;
constexpr int compact_smem_bytes(int entries, int buffers) {
  return buffers * entries * kCompactRows * 128;
}

struct CompactParams {
  const uint8_t* kv;
  const uint8_t* k_idx;
  const float* k_scale;
  const float* mass;           // or nullptr
  uint8_t* to_kv;
  uint8_t* to_k_idx;
  float* to_k_scale;
  float* to_mass;
  const int32_t* kept;         // [batch][keep]
  const int32_t* new_lens;     // [batch]
  const int32_t* seqlens;      // [batch] or nullptr
  const int32_t* table;        // paged source
  const int32_t* to_table;     // paged destination
  int64_t mass_ld, to_mass_ld;
  int32_t keep, splits;        // splits: CTAs of one slice (the cluster's), or of a sequence
  int32_t steps;               // into other pages: steps of a warp
  int32_t max_ctx, page_size, max_pages, num_pages;
  int32_t to_max_ctx, to_page_size, to_max_pages, to_num_pages;
};

// Row of the cache arrays that holds a slot, -1 for a page outside the cache.
__device__ __forceinline__ int cache_row(const int32_t* table, int b, int slot, int max_ctx,
                                         int page_size, int max_pages, int num_pages) {
  if (!table) return b * max_ctx + slot;
  const int pg = __ldg(table + (int64_t)b * max_pages + slot / page_size);
  if (pg < 0 || pg >= num_pages) return -1;
  return pg * page_size + slot % page_size;
}

// Sequence b's old and new length; false (reported) where they are out of range.
__device__ __forceinline__ bool compact_lengths(const CompactParams& p, int b, int& len, int& n) {
  len = p.seqlens ? __ldg(p.seqlens + b) : p.max_ctx;
  n = __ldg(p.new_lens + b);
  const bool ok = len >= 0 && len <= p.max_ctx && n >= 0 && n <= p.keep && n <= len &&
                  n <= p.to_max_ctx;
  if (!ok && threadIdx.x == 0) report_error(kErrBounds);
  return ok;
}

constexpr int kMoveWarps = kCompactThreads / 32;
constexpr int kMoveRows = 4;      // of a warp at a time
constexpr int kMoveSteps = 4;     // such steps of a warp, at most
static_assert(kMoveRows * kMoveSteps <= 32, "a lane for every row");
__global__ void __launch_bounds__(kCompactThreads, 3) cache_move_kernel(const CompactParams p) {
  const int b = blockIdx.x / p.splits, rank = blockIdx.x % p.splits;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int len, n;
  if (!compact_lengths(p, b, len, n)) return;
  const int rows = p.steps * kMoveRows;  // of this warp: a lane has the places of one
  const int64_t i = ((int64_t)rank * kMoveWarps + warp) * rows + lane;
  int slot = 0, from = -1, to = -1;
  if (lane < rows && i < n) {
    slot = __ldg(p.kept + (int64_t)b * p.keep + i);
    if (slot >= 0 && slot < len)
      from = cache_row(p.table, b, slot, p.max_ctx, p.page_size, p.max_pages, p.num_pages);
    to = cache_row(p.to_table, b, (int)i, p.to_max_ctx, p.to_page_size, p.to_max_pages, p.to_num_pages);
    if (from < 0 || to < 0) {
      report_error(kErrBounds);
      from = to = -1;
    }
  }
  if (__any_sync(0xffffffffu, from >= 0)) {
    constexpr int kPieces = 1280 / 16, kEach = kMoveRows * kPieces / 32;
    // this lane's j-th piece of the rows from r0 on, nullptr where there is none
    auto piece = [&](auto* latent, auto* keys, int row_of, int r0, int j) {
      const int c = j * 32 + lane, r = c / kPieces, at = (c - r * kPieces) * 16;
      const int64_t row = __shfl_sync(0xffffffffu, row_of, r0 + r);
      auto* to = at < 1152 ? latent + row * 1152 + at : keys + row * 128 + (at - 1152);
      return row < 0 ? nullptr : to;
    };
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += kMoveRows) {
      uint4 v[kEach];
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const uint8_t* src = piece(p.kv, p.k_idx, from, r0, j);
        if (src) v[j] = *reinterpret_cast<const uint4*>(src);
      }
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        uint8_t* dst = piece(p.to_kv, p.to_k_idx, to, r0, j);
        if (dst) *reinterpret_cast<uint4*>(dst) = v[j];
      }
    }
    if (from >= 0) {
      p.to_k_scale[to] = p.k_scale[from];
      if (p.mass) p.to_mass[(int64_t)b * p.to_mass_ld + i] = p.mass[(int64_t)b * p.mass_ld + slot];
    }
  }
  if (p.mass)
    for (int64_t z = n + (int64_t)rank * kCompactThreads + threadIdx.x; z < min(len, p.to_max_ctx);
         z += (int64_t)p.splits * kCompactThreads)
      p.to_mass[(int64_t)b * p.to_mass_ld + z] = 0.f;
}

// What has to be ordered is one CTA's loads of a chunk before another's stores to the same
// slots, which takes a release and an acquire. A release also waits for the stores before it, so
// it is given for chunk c + 1 before chunk c is stored: then the stores before it are chunk
// c - 1's, long done (8 paged sequences of 16384 kept tokens 79 us; 84 where a CTA arrives for
// a chunk right before it stores it). The last warp, which moves nothing, gives it for its CTA,
// whose other warps have met it at the block's barrier (contiguous, 74 us, 80 with a release by
// every warp, and 68 with none: what the order costs). A cluster of one CTA needs the block's
// barrier alone.
__device__ __forceinline__ void chunk_loaded(bool mover, int splits) {
  __syncthreads();
  if (splits == 1) return;
  if (mover)
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  else
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void chunk_loaded_by_all(int splits) {
  if (splits > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// kBuffers: with three the loads of chunk c + 2 are issued before chunk c is stored, else after.
template <int kEntries, int kBuffers>
__global__ void __launch_bounds__(kCompactBlock) cache_compact_kernel(const CompactParams p) {
  extern __shared__ uint4 compact_smem[];
  const int b = blockIdx.x / p.splits, rank = blockIdx.x % p.splits;
  const int slice = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool mover = tid < kCompactThreads;
  int len, n;
  if (!compact_lengths(p, b, len, n)) return;
  const int32_t* kept = p.kept + (int64_t)b * p.keep;
  const int step = p.splits * kEntries * kCompactRows;
  // this lane's e-th entry of chunk c, whose row its warp moves
  auto entry = [&](int c, int e) {
    return c * step + (rank * kEntries + e) * kCompactRows + tid;
  };
  // its source row; -1: none, already in its place, or the warp that moves nothing
  auto source = [&](int i, int& slot) {
    if (i >= n || !mover) return -1;
    slot = __ldg(kept + i);
    const bool ok = slot >= i && slot < len && (i == 0 || slot > __ldg(kept + i - 1));
    if (ok && slot == i) return -1;
    const int row = ok ? cache_row(p.table, b, slot, p.max_ctx, p.page_size, p.max_pages,
                                   p.num_pages) : -1;
    if (row < 0) report_error(kErrBounds);
    return row;
  };
  auto destination = [&](int i) {
    const int row = cache_row(p.to_table, b, i, p.to_max_ctx, p.to_page_size, p.to_max_pages,
                              p.to_num_pages);
    if (row < 0) report_error(kErrBounds);
    return row;
  };
  const int chunks = (n + step - 1) / step;
  if (slice < 10) {  // 128 B a row; a warp instruction moves four rows, eight lanes a row
    const int piece = lane & 7, sub = lane >> 3;
    const int64_t pitch = slice < 9 ? 1152 : 128;
    const uint8_t* from = (slice < 9 ? p.kv + slice * 128 : p.k_idx) + piece * 16;
    uint8_t* to = (slice < 9 ? p.to_kv + slice * 128 : p.to_k_idx) + piece * 16;
    // a lane's pieces in shared memory: + 32 a group of four rows, + kCompactRows * 8 an entry
    uint4* mine = compact_smem + (warp * 32 + sub) * 8 + piece;
    auto buffer = [&](int c) { return mine + (c % kBuffers) * kEntries * kCompactRows * 8; };
    auto load = [&](int c, int (&row)[kEntries]) {
#pragma unroll
      for (int e = 0; e < kEntries; ++e) {
        int slot;
        row[e] = c < chunks ? source(entry(c, e), slot) : -1;
      }
#pragma unroll
      for (int e = 0; e < kEntries; ++e) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = __shfl_sync(0xffffffffu, row[e], j * 4 + sub);
          if (r >= 0)
            cp_async_16(smem_u32(buffer(c) + e * kCompactRows * 8 + j * 32), from + r * pitch, 16u);
        }
      }
      cp_async_commit();
    };
    int row[kEntries], next[kEntries], far[kEntries] = {}, dst[kEntries];
    load(0, row);
    load(1, next);
    cp_async_wait_group<1>();
    if (chunks > 0) chunk_loaded(mover, p.splits);
    for (int c = 0; c < chunks; ++c) {
      if (kBuffers == 3) load(c + 2, far);
#pragma unroll
      for (int e = 0; e < kEntries; ++e) dst[e] = row[e] >= 0 ? destination(entry(c, e)) : -1;
      cp_async_wait_group<kBuffers - 2>();  // this thread's part of chunk c + 1
      chunk_loaded_by_all(p.splits);
      if (c + 1 < chunks) chunk_loaded(mover, p.splits);
#pragma unroll
      for (int e = 0; e < kEntries; ++e) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = __shfl_sync(0xffffffffu, dst[e], j * 4 + sub);
          if (r >= 0)
            *reinterpret_cast<uint4*>(to + r * pitch) = buffer(c)[e * kCompactRows * 8 + j * 32];
        }
        row[e] = next[e], next[e] = far[e];
      }
      if (kBuffers == 2) load(c + 2, next);
    }
    return;
  }
  // scale and mass, 4 B each
  float* mine = reinterpret_cast<float*>(compact_smem) + tid;
  auto buffer = [&](int c, int e) { return mine + ((c % kBuffers) * kEntries + e) * 2 * kCompactThreads; };
  auto load = [&](int c, int (&row)[kEntries]) {
#pragma unroll
    for (int e = 0; e < kEntries; ++e) {
      int slot;
      row[e] = c < chunks ? source(entry(c, e), slot) : -1;
      if (row[e] >= 0) {
        cp_async_4(smem_u32(buffer(c, e)), p.k_scale + row[e], 4u);
        if (p.mass)
          cp_async_4(smem_u32(buffer(c, e) + kCompactThreads), p.mass + (int64_t)b * p.mass_ld + slot, 4u);
      }
    }
    cp_async_commit();
  };
  int row[kEntries], next[kEntries], far[kEntries] = {};
  load(0, row);
  load(1, next);
  cp_async_wait_group<1>();
  if (chunks > 0) chunk_loaded(mover, p.splits);
  for (int c = 0; c < chunks; ++c) {
    if (kBuffers == 3) load(c + 2, far);
    int dst[kEntries];
#pragma unroll
    for (int e = 0; e < kEntries; ++e) dst[e] = row[e] >= 0 ? destination(entry(c, e)) : -1;
    cp_async_wait_group<kBuffers - 2>();
    chunk_loaded_by_all(p.splits);
    if (c + 1 < chunks) chunk_loaded(mover, p.splits);
#pragma unroll
    for (int e = 0; e < kEntries; ++e) {
      if (dst[e] >= 0) {
        p.to_k_scale[dst[e]] = *buffer(c, e);
        if (p.mass)
          p.to_mass[(int64_t)b * p.to_mass_ld + entry(c, e)] = buffer(c, e)[kCompactThreads];
      }
      row[e] = next[e], next[e] = far[e];
    }
    if (kBuffers == 2) load(c + 2, next);
  }
  if (p.mass && mover)
    for (int i = n + rank * kCompactThreads + tid; i < min(len, p.to_max_ctx);
         i += p.splits * kCompactThreads)
      p.to_mass[(int64_t)b * p.to_mass_ld + i] = 0.f;
}

}  // namespace dsa
