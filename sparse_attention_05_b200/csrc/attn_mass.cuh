// attn_mass.cuh -- the attention weight every cached token received, accumulated.
//
// For query row t and its listed entries s (the sparse MLA's S_t, DeepSeek-V3.2-Exp
// technical report §1 Eq. 2) with the forward's per-head log-sum-exp,
//   p(t, s) = 1/128 sum_h exp(scale q_{t,h} . c_s - LSE_{t,h}),   mass[b][s] += sum_t p(t, s).
// The head mean is the main attention's distribution of the report's §2.1.
//
// Per listed entry 1152 B gathered and 147456 flops: 128 flops a byte, below the ~253
// at which this part's BF16 rate and HBM rate meet, so rows gathered from HBM are bound
// by the gather; rows that L2 holds by the L2 -> SM gather and the tensor core alike.
// One persistent CTA per SM walks (row, 128-entry tile) items: with few rows an equal run
// of all rows' tiles each (a row may be shared by several CTAs), with many every
// gridDim-th row whole, which spreads the short rows evenly.
// The row's Q (128 heads x 576) stays in shared memory as nine 128-B-swizzled chunks of 64
// dims, the listed latent rows stream through a ring of 64-dim chunks, and
// D[entry][head] = K_tile (128 x 576) . Q^T lands in one of two TMEM accumulators, entries
// on the lanes, so that the sum over heads stays inside a thread. The next row's Q chunk c
// travels with its first tile's chunk c: the ring stage it takes is free only once the
// last row's products with chunk c are done (the ring is shorter than a tile).
// Tiles without a single valid entry are passed over by every role alike.
//
// Warp roles (288 threads): 0-3 epilogue (thread = entry), 4 TMEM and MMA issue, 5-8
// producers (a warp's cp.async covers four whole 128-B lines, eight lanes a line; one
// line a lane would take eight times the tag lookups). Entries are read two tiles ahead
// and their pages one tile ahead.
//
// The sums over the rows are the same for every order of execution:
//   few rows a sequence: p goes to the workspace, and one CTA a sequence adds its rows
//     one after another (equal entries of one row carry equal p, so their order is free);
//   many rows: p is added as a 64-bit integer in units of 2^-40, which commutes, and a
//     second kernel turns the sums into fp32. 2^-41 is the most an entry is off.
#pragma once

#include <cuda_bf16.h>

#include "ptx.cuh"
#include "rows.cuh"

namespace dsa {

constexpr int kMassHeads = 128;
constexpr int kMassDqk = 576;
constexpr int kMassChunks = kMassDqk / 64;
constexpr int kMassTile = 128;
constexpr int kMassStages = 5;
constexpr int kMassThreads = 288;
constexpr int kMassChunkBytes = 128 * 128;
constexpr int kMassSmemBytes = 1024 + (kMassChunks + kMassStages) * kMassChunkBytes +
                               2 * kMassHeads * 4 + 24 * 8 + 16;
static_assert(kMassStages <= kMassChunks, "a Q chunk must be free when its ring stage is");
static_assert(kMassSmemBytes <= 232448, "attention mass shared memory exceeds the per-CTA limit");
constexpr float kMassUnit = 1099511627776.0f;             // 2^40 units of fixed point
constexpr float kMassMaxP = 64.0f;                        // a larger p is not a weight
constexpr unsigned long long kMassNan = 1ull << 63;       // set, never added

struct MassParams {
  const uint8_t* kv;           // latent cache rows of 1152 B
  const __nv_bfloat16* q;      // [T][128][576]
  const int32_t* idx;          // [T][k]
  const float* lse;            // [T][128]
  const int32_t* block_table;
  const int32_t* seqlens;
  const int32_t* q_start;
  float* p_out;                // [batch * row_count][k], or nullptr
  unsigned long long* sums;    // [batch][max_ctx], or nullptr
  float* mass;                 // [batch][mass_ld]
  int64_t mass_ld;
  int32_t k, batch, max_ctx, q_per_seq, num_q;
  int32_t row_begin, row_count;
  int32_t paged, page_size, max_pages, num_pages;
  int32_t whole_rows;          // CTAs take whole rows instead of runs of tiles
  float scale_log2;
  uint64_t timeout_ns;
};

// The (row, tile) items of one CTA, in order.
struct MassItems {
  int64_t row, end;    // window row, and the end (rows, or the CTA's last item)
  int tile, b, pos;
  int64_t t;           // global query row, -1: the sequence does not have it
  bool live;           // there is an item

  __device__ __forceinline__ void start(const MassParams& p) {
    const int ntiles = (p.k + kMassTile - 1) / kMassTile;
    const int64_t rows = (int64_t)p.batch * p.row_count;
    tile = 0;
    if (p.whole_rows) {
      row = blockIdx.x;
      end = rows;
      live = row < end;
    } else {
      const int64_t first = rows * ntiles * blockIdx.x / gridDim.x;
      end = rows * ntiles * (blockIdx.x + 1) / gridDim.x;
      live = first < end;
      row = first / ntiles;
      tile = (int)(first - row * ntiles);
    }
    if (live) find(p);
  }
  __device__ __forceinline__ void find(const MassParams& p) {
    b = (int)(row / p.row_count);
    const int qi = p.row_begin + (int)(row - (int64_t)b * p.row_count);
    const SeqRows R = seq_rows(p.q_start, p.seqlens, b, p.q_per_seq, p.num_q, p.max_ctx);
    t = R.ok && qi < R.q_len ? R.t0 + qi : -1;
    pos = R.seqlen - R.q_len + qi;
    if (!R.ok) report_error(kErrBounds);
  }
  __device__ __forceinline__ void next(const MassParams& p) {
    const int ntiles = (p.k + kMassTile - 1) / kMassTile;
    if (t >= 0 && ++tile < ntiles) {
      live = p.whole_rows || row * ntiles + tile < end;
      return;
    }
    tile = 0;
    row += p.whole_rows ? gridDim.x : 1;
    live = p.whole_rows ? row < end : row * ntiles < end;
    if (live) find(p);
  }
  // Entry e of the tile: its slot, or -1.
  __device__ __forceinline__ int entry(const MassParams& p, int e) const {
    const int i = tile * kMassTile + e;
    if (!live || t < 0 || i >= p.k) return -1;
    const int sel = __ldg(p.idx + t * p.k + i);
    return sel <= pos ? max(sel, -1) : -1;
  }
};

// Whether any of a tile's 128 entries is one, told from four per lane.
__device__ __forceinline__ bool mass_tile_used(const int (&sel)[4]) {
  return __any_sync(0xffffffffu, (sel[0] & sel[1] & sel[2] & sel[3]) >= 0);
}

__global__ void __launch_bounds__(kMassThreads, 1)
    attn_mass_kernel(const __grid_constant__ MassParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + kMassChunks * kMassChunkBytes;
  float* sLse2 = reinterpret_cast<float*>(sK + kMassStages * kMassChunkBytes);  // [2][128]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sLse2 + 2 * kMassHeads);
  uint64_t* kfull = bars;                    // [stages] the chunk (and its Q chunk) landed
  uint64_t* kempty = kfull + kMassStages;    // [stages] its products are done
  uint64_t* tfull = kempty + kMassStages;    // [2] accumulator ready
  uint64_t* tempty = tfull + 2;              // [2] read
  uint64_t* mdone = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(mdone + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kMassStages; ++i) {
      mbar_init(smem_u32(&kfull[i]), 128);
      mbar_init(smem_u32(&kempty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&tfull[i]), 1);
      mbar_init(smem_u32(&tempty[i]), 128);
    }
    mbar_init(smem_u32(mdone), 1);
    *abort_flag = 0;
    fence_mbarrier_init_cluster();
  }
  if (warp == 4) {
    tmem_alloc(smem_u32(tmem_holder), 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const uint64_t TO = p.timeout_ns;
  int drain_dummy = 0;
  volatile int* no_abort = &drain_dummy;

  if (warp >= 5) {
    // ------------------------------------------------------------ producers
    const int pw = warp - 5, piece = lane & 7, sub = lane >> 3;
    auto load_entries = [&](const MassItems& m, int (&sel)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) sel[i] = m.entry(p, i * 32 + lane);
    };
    // the page of this lane's own entry (entry pw * 32 + lane of the tile)
    auto own = [&](const int (&sel)[4]) {
      return pw == 0 ? sel[0] : pw == 1 ? sel[1] : pw == 2 ? sel[2] : sel[3];
    };
    auto load_page = [&](const MassItems& m, int s) {
      return p.paged && s >= 0
                 ? __ldg(p.block_table + (int64_t)m.b * p.max_pages + s / p.page_size) : 0;
    };
    MassItems cur, ahead, far;  // this tile's, one and two tiles ahead
    int s0[4], s1[4], s2[4];
    cur.start(p);
    load_entries(cur, s0);
    ahead = cur;
    if (ahead.live) ahead.next(p);
    load_entries(ahead, s1);
    far = ahead;
    int page0 = load_page(cur, own(s0));
    int64_t q_row = -1;  // the query row whose Q is in shared memory
    uint32_t it = 0;
    bool ok = true;
    while (cur.live && ok) {
      const int page1 = load_page(ahead, own(s1));
      if (far.live) far.next(p);
      load_entries(far, s2);
      if (mass_tile_used(s0)) {
        const int sel = own(s0);
        int row = -1;
        if (sel >= 0) {
          if (!p.paged)
            row = cur.b * p.max_ctx + sel;
          else if (page0 >= 0 && page0 < p.num_pages)
            row = page0 * p.page_size + sel % p.page_size;
          else
            report_error(kErrBounds);
        }
        int rows[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) rows[i] = __shfl_sync(0xffffffffu, row, i * 4 + sub);
        const bool new_q = cur.t != q_row;
        q_row = cur.t;
        const uint8_t* q = reinterpret_cast<const uint8_t*>(p.q + cur.t * kMassHeads * kMassDqk);
#pragma unroll 1
        for (int c = 0; c < kMassChunks; ++c, ++it) {
          const int st = it % kMassStages;
          if (!warp_wait(smem_u32(&kempty[st]), ((it / kMassStages) & 1) ^ 1, TO, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t dst = smem_u32(sK + st * kMassChunkBytes);
          const int off = c * 128 + piece * 16;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            cp_async_16(dst + sw128_offset(pw * 32 + i * 4 + sub, piece),
                        p.kv + (int64_t)max(rows[i], 0) * (kMassDqk * 2) + off,
                        rows[i] >= 0 ? 16u : 0u);
          if (new_q) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int h = pw * 32 + i * 4 + sub;
              cp_async_16(smem_u32(sQ + c * kMassChunkBytes) + sw128_offset(h, piece),
                          q + h * (kMassDqk * 2) + off, 16u);
            }
          }
          cp_async_mbar_arrive(smem_u32(&kfull[st]));
        }
      }
      cur = ahead;
      ahead = far;
      page0 = page1;
#pragma unroll
      for (int i = 0; i < 4; ++i) s0[i] = s1[i], s1[i] = s2[i];
    }
    cp_async_wait_all();
  } else if (warp == 4) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t idesc = instr_desc(1 /*bf16*/, 0, 0, 128, 128);
    uint32_t it = 0, tiles = 0;
    bool ok = true;
    MassItems m;
    m.start(p);
    int sel[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sel[i] = m.entry(p, i * 32 + lane);
    while (m.live && ok) {
      const bool used = mass_tile_used(sel);
      m.next(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) sel[i] = m.entry(p, i * 32 + lane);  // the next tile's
      if (!used) continue;
      const int ab = tiles & 1;
      if (lane == 0) {
        ok = mbar_wait(smem_u32(&tempty[ab]), ((tiles >> 1) & 1) ^ 1, TO, abort_flag);
        tc_fence_after();
        const uint32_t d = tmem_base + ab * 128;
        for (int c = 0; c < kMassChunks && ok; ++c, ++it) {
          const int st = it % kMassStages;
          ok = mbar_wait(smem_u32(&kfull[st]), (it / kMassStages) & 1, TO, abort_flag);
          if (!ok) break;
          tc_fence_after();
          fence_proxy_async_smem();  // cp.async (generic proxy) writes -> tensor-core reads
          const uint32_t ka = smem_u32(sK + st * kMassChunkBytes);
          const uint32_t qa = smem_u32(sQ + c * kMassChunkBytes);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_bf16_ss(d, smem_desc_sw128(ka + kk * 32, 16, 1024),
                        smem_desc_sw128(qa + kk * 32, 16, 1024), idesc, (c > 0 || kk > 0) ? 1u : 0u);
          mma_commit(smem_u32(&kempty[st]));
        }
        if (ok) mma_commit(smem_u32(&tfull[ab]));
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      ++tiles;
    }
    if (lane == 0) {
      mma_commit(smem_u32(mdone));
      mbar_wait(smem_u32(mdone), 0, TO, no_abort);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    uint32_t tiles = 0;
    int lse_buf = 0;
    int64_t lse_row = -1;
    MassItems m;
    m.start(p);
    int sel[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sel[i] = m.entry(p, i * 32 + lane);
    while (m.live) {
      const bool used = mass_tile_used(sel);
      const int slot = warp == 0 ? sel[0] : warp == 1 ? sel[1] : warp == 2 ? sel[2] : sel[3];
      const MassItems now = m;
      m.next(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) sel[i] = m.entry(p, i * 32 + lane);
      float w = 0.f;
      if (used) {
        if (now.t != lse_row) {  // double-buffered: the four warps are at most a barrier apart
          lse_row = now.t;
          lse_buf ^= 1;
          sLse2[lse_buf * kMassHeads + tid] =
              __ldg(p.lse + now.t * kMassHeads + tid) * 1.4426950408889634f;
        }
        const int ab = tiles & 1;
        const bool got = warp_wait(smem_u32(&tfull[ab]), (tiles >> 1) & 1, TO, abort_flag);
        if (!named_barrier_and(1, 128, got)) break;
        tc_fence_after();
        const float* lse2 = sLse2 + lse_buf * kMassHeads;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float z[32];
          tmem_ld32(tmem_base + ab * 128 + c * 32 + lane_off, z);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) w += ex2_approx(z[i] * p.scale_log2 - lse2[c * 32 + i]);
        }
        tc_fence_before();
        mbar_arrive(smem_u32(&tempty[ab]));
        ++tiles;
      }
      w *= 1.0f / kMassHeads;
      const int e = now.tile * kMassTile + tid;
      if (p.sums) {
        if (slot >= 0) {
          unsigned long long* s = p.sums + (int64_t)now.b * p.max_ctx + slot;
          if (w <= kMassMaxP)
            atomicAdd(s, (unsigned long long)__float2ll_rn(w * kMassUnit));
          else
            atomicOr(s, kMassNan);
        }
      } else if (now.t >= 0 && e < p.k) {
        p.p_out[now.row * p.k + e] =
            slot < 0 ? 0.f : w <= kMassMaxP ? w : __int_as_float(0x7fffffff);
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 256);
  }
}

// Few rows: one CTA adds a sequence's rows in order.
__global__ void __launch_bounds__(512) mass_add_rows_kernel(const __grid_constant__ MassParams p) {
  const int b = blockIdx.x;
  const SeqRows R = seq_rows(p.q_start, p.seqlens, b, p.q_per_seq, p.num_q, p.max_ctx);
  if (!R.ok) return;
  const int last = min(p.row_begin + p.row_count, R.q_len);
  float* mass = p.mass + (int64_t)b * p.mass_ld;
  for (int qi = p.row_begin; qi < last; ++qi) {
    const int pos = R.seqlen - R.q_len + qi;
    const int32_t* idx = p.idx + (R.t0 + qi) * p.k;
    const float* w = p.p_out + ((int64_t)b * p.row_count + qi - p.row_begin) * p.k;
    for (int e = threadIdx.x; e < p.k; e += blockDim.x) {
      const int sel = __ldg(idx + e);
      if (sel >= 0 && sel <= pos) atomicAdd(mass + sel, w[e]);
    }
    __syncthreads();
  }
}

// Many rows: the integer sums of one sequence's slots to fp32, added to its mass.
__global__ void __launch_bounds__(256) mass_add_sums_kernel(const __grid_constant__ MassParams p) {
  const int b = blockIdx.y;
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= p.max_ctx) return;
  const unsigned long long s = p.sums[(int64_t)b * p.max_ctx + i];
  if (s == 0) return;
  float* m = p.mass + (int64_t)b * p.mass_ld + i;
  *m = s & kMassNan ? __int_as_float(0x7fffffff)
                    : *m + (float)((double)s * (1.0 / (double)kMassUnit));
}

}  // namespace dsa
