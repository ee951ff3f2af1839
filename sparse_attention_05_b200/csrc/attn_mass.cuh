// attn_mass.cuh -- the attention weight every cached token received, accumulated.
//
// For query row t and its listed entries s (the sparse MLA's S_t, DeepSeek-V3.2-Exp
// technical report §1 Eq. 2) with the forward's per-head log-sum-exp,
//   p(t, s) = 1/128 sum_h exp(scale q_{t,h} . c_s - LSE_{t,h}),   mass[b][s] += sum_t p(t, s).
// The head mean is the main attention's distribution of the report's §2.1.
//
// Per listed entry 1152 B gathered and 147456 flops: 128 flops a byte, below the ~253
// at which this part's BF16 rate and HBM rate meet, so the gather bounds the kernel:
// rows in HBM come at 5.2-6.4 TB/s with 112-200 KB of loads in flight per SM and 4.3 with
// 80 KB, rows in L2 at up to 15 TB/s (measured, loads alone). Hence Q does not take shared
// memory: the first 512 dims of the row's Q (128 heads x 576) are the A operand in tensor
// memory (256 columns), only the last 64 stay in shared memory, and the rest of that is a
// ring of six 32-KB stages for the listed latent rows, 64 dims of up to 256 rows each.
// D[head][entry] = Q . K_tile^T takes the other 256 columns: a product with N = 256 costs
// the tensor core little more than one with N = 128, so a wide tile is nearly free.
//
// One persistent CTA per SM walks (row, tile) items: with few rows an equal run of all
// rows' tiles each (a row may be shared by several CTAs), with many every gridDim-th row
// whole, which spreads the short rows evenly. A row's Q travels through the ring as nine
// stages before its first tile. Tiles without a valid entry are passed over by every role.
//
// Warp roles (640 threads):
//   warps 0-15  epilogue: warp w has heads 32 (w % 4) .. + 31 and columns 64 (w / 4) .. + 63.
//               It empties the accumulator into registers (there is one: the tensor core
//               waits for no more than that), four heads of a column in a thread, takes the
//               exponentials and sums a column in the thread and over the eight lanes that
//               share it (with one head a lane the sums took 31 exchanges for 32 columns,
//               not 7, and 512 rows 215 us, not 199); the four partial sums of a column
//               meet in shared memory
//   warp 16     TMEM, and the issue of the copies of Q into it and of the products
//   warps 17-19 producers: a warp's cp.async covers four whole 128-B lines, eight lanes a
//               line (one line a lane would take eight times the tag lookups). Entries are
//               read two tiles ahead and their pages one tile ahead. Where the list has
//               no entry the cache's first row is copied and its column dropped (a copy
//               with a zero-fill operand takes 1.6 times as long to issue).
//
// The sums over the rows are the same for every order of execution:
//   one row a sequence: p is added to the mass where it is computed (equal entries of one
//     row carry equal p, so their order is free);
//   few rows a sequence: p goes to the workspace, and one CTA a sequence adds its rows
//     one after another;
//   many rows: p is added as a 64-bit integer, which commutes, and a second kernel turns the
//     sums into fp32. The unit is the smallest in which the rows' largest weights add up below
//     2^62 (2^-47 for 512 rows); half of it is the most an entry is off.
#pragma once

#include <cuda_bf16.h>

#include "ptx.cuh"
#include "rows.cuh"

namespace dsa {

constexpr int kMassHeads = 128;
constexpr int kMassDqk = 576;
constexpr int kMassChunks = kMassDqk / 64;
constexpr int kMassMaxTile = 256;                  // entries of a tile (MMA N), at most
constexpr int kMassQuarter = kMassMaxTile / 4;     // columns of an epilogue warp
constexpr int kMassStages = 6;
constexpr int kMassStageBytes = kMassMaxTile * 128;
constexpr int kMassEpilogue = 512, kMassProducers = 96;
constexpr int kMassThreads = kMassEpilogue + 32 + kMassProducers;
constexpr int kMassQCols = 256;                    // tensor memory columns of Q's chunks 0-7
constexpr int kMassQBytes = kMassHeads * 128;      // its last chunk, in shared memory
constexpr int kMassSmemBytes = 1024 + kMassStages * kMassStageBytes + kMassQBytes +
                               2 * 4 * kMassMaxTile * 4 /*partial sums*/ + 24 * 8 + 16;
static_assert(kMassSmemBytes <= 232448, "attention mass shared memory exceeds the per-CTA limit");
static_assert(kMassQCols + kMassMaxTile <= 512, "tensor memory");
static_assert(kMassStages < kMassChunks, "Q's last chunk is free once its place in the ring is");
constexpr float kMassMaxP = 64.0f;                        // a larger p is not a weight
// The tensor core truncates its running sums: after the 36 dependent steps of a logit z it is
// short of about 2^-21 z, and the weight off by as much. The scale makes up for the mean of it.
// Against exp(scale q.c - LSE) for the LSE as it is given, rows whose weights' mean logit is
// 2.2, 5.9, -1.3 and 19.8 are off by 2e-8, -3e-7, 1e-8 and -8e-7 of their weight, and by
// -1.0e-6, -3.0e-6, 6e-7 and -9.7e-6 without. (The forward's LSE has truncated logits of its
// own, in sums of 18 steps: its rows add up to 1 within 1e-6 either way.) Where partial sums
// cancel, what is lost goes with them and no factor helps: 1.4e-5 with sums up to 29.
constexpr double kMassUntruncate = 1.0 + 1.0 / 2097152.0;
constexpr unsigned long long kMassNan = 1ull << 63;       // set, never added

struct MassParams {
  const uint8_t* kv;           // latent cache rows of 1152 B
  const __nv_bfloat16* q;      // [T][128][576]
  const int32_t* idx;          // [T][k]
  const float* lse;            // [T][128]
  const int32_t* block_table;
  const int32_t* seqlens;
  const int32_t* q_start;
  // where the weights go: one of these, else to the mass itself
  float* p_out;                // [batch * row_count][k], or nullptr
  unsigned long long* sums;    // [batch][max_ctx], or nullptr
  float* mass;                 // [batch][mass_ld]
  int64_t mass_ld;
  int32_t k, batch, max_ctx, q_per_seq, num_q;
  int32_t row_begin, row_count;
  int32_t paged, page_size, max_pages, num_pages;
  int32_t tile;                // entries of a tile: a multiple of 16, at most 256
  int32_t ntiles;              // of a row
  int32_t whole_rows;          // CTAs take whole rows instead of runs of tiles
  float scale;
  float units;                 // of the integer sums in 1: a power of two
  uint64_t timeout_ns;
};

// The (row, tile) items of one CTA, in order. (Rows, and one CTA's items, are below 2^31.)
struct MassItems {
  int row;             // window row
  int left;            // items after this one (runs of tiles)
  int tile, b, pos;
  int t;               // global query row, -1: the sequence does not have it
  bool live;           // there is an item

  __device__ __forceinline__ void start(const MassParams& p) {
    const int64_t rows = (int64_t)p.batch * p.row_count;
    tile = 0;
    if (p.whole_rows) {
      row = blockIdx.x;
      left = 0;
      live = row < rows;
    } else {
      const int ntiles = p.ntiles;
      const int64_t first = rows * ntiles * blockIdx.x / gridDim.x;
      left = (int)(rows * ntiles * (blockIdx.x + 1) / gridDim.x - first) - 1;
      live = left >= 0;
      row = (int)(first / ntiles);
      tile = (int)(first - (int64_t)row * ntiles);
    }
    if (live) find(p);
  }
  __device__ __forceinline__ void find(const MassParams& p) {
    b = row / p.row_count;
    const int qi = p.row_begin + row - b * p.row_count;
    const SeqRows R = seq_rows(p.q_start, p.seqlens, b, p.q_per_seq, p.num_q, p.max_ctx);
    t = R.ok && qi < R.q_len ? (int)R.t0 + qi : -1;
    pos = R.seqlen - R.q_len + qi;
    if (!R.ok) report_error(kErrBounds);
  }
  __device__ __forceinline__ void next(const MassParams& p) {
    const int ntiles = p.ntiles;
    if (t >= 0 && tile + 1 < ntiles) {
      ++tile;
      live = p.whole_rows || --left >= 0;
      return;
    }
    if (p.whole_rows) {
      live = (int64_t)row + gridDim.x < (int64_t)p.batch * p.row_count;
      row += gridDim.x;
    } else {
      left -= ntiles - tile;  // the rest of a row that the sequence does not have
      live = left >= 0;
      ++row;
    }
    tile = 0;
    if (live) find(p);
  }
  // Entry e of the tile as it is listed, -1 past the list. Nothing here waits for the load.
  __device__ __forceinline__ int listed(const MassParams& p, int e) const {
    const int i = tile * p.tile + e;
    return live && t >= 0 && e < p.tile && i < p.k ? __ldg(p.idx + (int64_t)t * p.k + i) : -1;
  }
  __device__ __forceinline__ bool valid(int sel) const { return sel >= 0 && sel <= pos; }
  // Columns of the tile's MMA: its entries, to a multiple of 16.
  __device__ __forceinline__ int columns(const MassParams& p) const {
    return (min(p.tile, p.k - tile * p.tile) + 15) & ~15;
  }
};

// Whether a tile has an entry at all. Only a row that sees fewer keys than the list is long
// can have a tile without one (or one that lists keys twice, which it may compute in vain).
__device__ __forceinline__ bool mass_used(const MassParams& p, const MassItems& m, int lane) {
  if (!m.live || m.t < 0) return false;
  if (m.pos + 1 >= p.k) return true;
  bool any = false;
#pragma unroll
  for (int i = 0; i < kMassMaxTile / 32; ++i) any |= m.valid(m.listed(p, i * 32 + lane));
  return __any_sync(0xffffffffu, any);
}

// 128 rows of 32 bytes from shared memory (descriptor as an MMA operand's) to the 128 lanes
// of eight tensor memory columns, ordered before the products issued after it.
__device__ __forceinline__ void tmem_copy_128x32(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.128x256b [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Place in the ring: stage and the parity of its round.
struct MassRing {
  int stage = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void next() {
    if (++stage == kMassStages) stage = 0, round ^= 1;
  }
};

// 16 lanes x 32 columns of tensor memory: register 4 j + 2 r + c of a thread holds
// lane l / 4 + 8 r, column 8 j + 2 (l % 4) + c (l: the thread's lane).
__device__ __forceinline__ void tmem_ld_16x256b(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// Waits for this thread's tensor memory loads; ties the registers to the wait.
template <int N>
__device__ __forceinline__ void tmem_wait_ld_tie(uint32_t (&r)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// A block of 32 columns of a warp's 32 heads: this thread's logits of heads l / 4 and + 8
// (lo), + 16 and + 24 (hi).
struct MassBlock {
  uint32_t lo[16], hi[16];
  __device__ __forceinline__ void load(uint32_t taddr) {
    tmem_ld_16x256b(taddr, lo);
    tmem_ld_16x256b(taddr + (16u << 16), hi);
  }
  __device__ __forceinline__ void wait() {
    tmem_wait_ld_tie(lo);
    tmem_wait_ld_tie(hi);
  }
  // The weights, summed over the warp's heads: four in the thread, then halving exchanges
  // over the eight lanes that share its columns. Every column is summed in the same order.
  // Lane l gets column 16 b4 + 8 b3 + b2 + 2 (l % 4) by its bits.
  // The difference scale z - LSE is rounded as such: with log2 e inside both terms a weight
  // would also lose what their size costs.
  __device__ __forceinline__ float sum(float scale, const float (&lse)[4], int lane) const {
    auto weight = [&](uint32_t z, int r) {
      return ex2_approx(1.4426950408889634f * fmaf(__uint_as_float(z), scale, -lse[r]));
    };
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
        v[2 * j + c] = (weight(lo[4 * j + c], 0) + weight(lo[4 * j + 2 + c], 1)) +
                       (weight(hi[4 * j + c], 2) + weight(hi[4 * j + 2 + c], 3));
    }
#pragma unroll
    for (int n = 4, o = 16; n > 0; n >>= 1, o >>= 1) {
      const bool up = lane & o;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float keep = up ? v[i + n] : v[i], give = up ? v[i] : v[i + n];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
    }
    return v[0];
  }
};

// kFull: every tile has 256 entries, so the copies need no test of how many there are (512 rows
// of 2048, calls in a graph: 174 us with it, 187 without).
template <bool kFull>
__global__ void __launch_bounds__(kMassThreads, 1)
    attn_mass_kernel(const __grid_constant__ MassParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sQ = ring + kMassStages * kMassStageBytes;        // Q's last chunk
  float* sPart = reinterpret_cast<float*>(sQ + kMassQBytes);  // [2][4][256]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sPart + 2 * 4 * kMassMaxTile);
  uint64_t* kfull = bars;                    // [stages] the stage's copies are complete
  uint64_t* kempty = kfull + kMassStages;    // [stages] it was read
  uint64_t* tfull = kempty + kMassStages;    // the accumulator is ready
  uint64_t* tempty = tfull + 1;              // it is in registers
  uint64_t* mdone = tempty + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(mdone + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kMassStages; ++i) {
      mbar_init(smem_u32(&kfull[i]), kMassProducers);
      mbar_init(smem_u32(&kempty[i]), 1);
    }
    mbar_init(smem_u32(tfull), 1);
    mbar_init(smem_u32(tempty), kMassEpilogue / 32);
    mbar_init(smem_u32(mdone), 1);
    *abort_flag = 0;
    fence_mbarrier_init_cluster();
  }
  if (warp == 16) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_q = *tmem_holder, tmem_d = tmem_q + kMassQCols;
  const uint64_t TO = p.timeout_ns;
  int drain_dummy = 0;
  volatile int* no_abort = &drain_dummy;

  if (warp >= 17) {
    // ------------------------------------------------------------ producers
    const int pw = warp - 17, piece = lane & 7, sub = lane >> 3;
    // rows of this warp: per from pw * per on, a multiple of four
    const int per = (p.tile / 4 + 2) / 3 * 4;
    constexpr int kGroups = (kMassMaxTile / 4 + 2) / 3;  // of four rows
    constexpr int kLastGroups = kMassMaxTile / 4 - 2 * kGroups;  // the last warp's, of a full tile
    // this lane's entries pw * per + lane, + 32 and + 64 of the tile
    auto own_entries = [&](const MassItems& m, int (&own)[3]) {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        own[i] = lane + 32 * i < per ? m.listed(p, pw * per + lane + 32 * i) : -1;
    };
    auto load_page = [&](const MassItems& m, int s) {
      return p.paged && m.valid(s)
                 ? __ldg(p.block_table + (int64_t)m.b * p.max_pages + s / p.page_size) : 0;
    };
    auto cache_row_of = [&](const MassItems& m, int s, int page) {
      if (!m.valid(s)) return 0;
      if (!p.paged) return m.b * p.max_ctx + s;
      if (page >= 0 && page < p.num_pages) return page * p.page_size + s % p.page_size;
      report_error(kErrBounds);
      return 0;
    };
    MassRing at;
    bool ok = true;
    auto acquire = [&] {
      const uint32_t bar = smem_u32(&kempty[at.stage]);
      if (!__all_sync(0xffffffffu, mbar_test_wait(bar, at.round ^ 1)))
        ok = warp_wait(bar, at.round ^ 1, TO, abort_flag);
      return ok;
    };
    // where this lane's 16 bytes of a four-row group lie in a stage: rows alternate between
    // two phases of the swizzle
    const uint32_t even = sw128_offset(pw * per + sub, piece);
    const uint32_t odd = sw128_offset(pw * per + 4 + sub, piece) - 512;
    MassItems cur, ahead, far;  // this tile's, one and two tiles ahead
    int own0[3], own1[3], own2[3], page0[3], page1[3];
    cur.start(p);
    own_entries(cur, own0);
    ahead = cur;
    if (ahead.live) ahead.next(p);
    own_entries(ahead, own1);
    far = ahead;
#pragma unroll
    for (int i = 0; i < 3; ++i) page0[i] = load_page(cur, own0[i]);
    int q_row = -1;  // the query row whose Q went through the ring last
    while (cur.live && ok) {
#pragma unroll
      for (int i = 0; i < 3; ++i) page1[i] = load_page(ahead, own1[i]);
      if (far.live) far.next(p);
      own_entries(far, own2);
      if (mass_used(p, cur, lane)) {
        if (cur.t != q_row) {
          q_row = cur.t;
          const uint8_t* q =
              reinterpret_cast<const uint8_t*>(p.q + (int64_t)q_row * kMassHeads * kMassDqk) + piece * 16;
#pragma unroll 1
          for (int c = 0; c < kMassChunks && ok; ++c) {
            if (!acquire()) break;
            // (the products that read the last chunk are done: two stages of this Q are read)
            const uint32_t dst = smem_u32(c < kMassChunks - 1 ? ring + at.stage * kMassStageBytes
                                                              : sQ);
#pragma unroll
            for (int i = 0; i < 11; ++i) {
              const int h = (pw * 11 + i) * 4 + sub;
              if (h < kMassHeads)
                cp_async_16(dst + sw128_offset(h, piece), q + h * (kMassDqk * 2) + c * 128, 16u);
            }
            cp_async_mbar_arrive(smem_u32(&kfull[at.stage]));
            at.next();
          }
        }
        int mine[3];
        const uint8_t* rows[kGroups];
#pragma unroll
        for (int i = 0; i < 3; ++i) mine[i] = cache_row_of(cur, own0[i], page0[i]);
#pragma unroll
        for (int i = 0; i < kGroups; ++i)
          rows[i] = p.kv + piece * 16 + (int64_t)(kMassDqk * 2) *
                    __shfl_sync(0xffffffffu, mine[i / 8], (i * 4 + sub) & 31);
        const int groups = min(per, max(0, cur.columns(p) - pw * per)) / 4;
#pragma unroll
        for (int c = 0; c < kMassChunks; ++c) {
          if (!acquire()) break;
          const uint32_t dst = smem_u32(ring + at.stage * kMassStageBytes);
          const uint32_t dst_even = dst + even, dst_odd = dst + odd;
#pragma unroll
          for (int i = 0; i < kGroups; ++i)
            if (kFull ? i < kLastGroups || pw < 2 : i < groups)
              cp_async_16((i & 1 ? dst_odd : dst_even) + i * 512, rows[i] + c * 128, 16u);
          cp_async_mbar_arrive(smem_u32(&kfull[at.stage]));
          at.next();
        }
      }
      cur = ahead;
      ahead = far;
#pragma unroll
      for (int i = 0; i < 3; ++i) own0[i] = own1[i], own1[i] = own2[i], page0[i] = page1[i];
    }
    cp_async_wait_all();
  } else if (warp == 16) {
    // ------------------------------------------------------------ MMA issuer
    MassRing at;
    uint32_t tiles = 0;
    bool ok = true;
    int q_row = -1;
    MassItems m;
    m.start(p);
    while (m.live && ok) {
      const MassItems now = m;
      const bool used = mass_used(p, m, lane);
      m.next(p);
      if (!used) continue;
      const bool new_q = now.t != q_row;
      q_row = now.t;
      const uint32_t idesc = instr_desc(1 /*bf16*/, 0, 0, 128, now.columns(p));
      if (lane == 0) {
        // the accumulator was read, so all products before are done, and Q may be replaced
        ok = mbar_wait(smem_u32(tempty), (tiles & 1) ^ 1, TO, abort_flag);
        tc_fence_after();
        const int stages = (new_q ? 2 : 1) * kMassChunks;
        MassRing st = at;
        for (int i = 0; i < stages && ok; ++i, st.next()) {
          ok = mbar_wait(smem_u32(&kfull[st.stage]), st.round, TO, abort_flag);
          if (!ok) break;
          tc_fence_after();
          fence_proxy_async_smem();  // cp.async (generic proxy) writes -> tensor-core reads
          const uint32_t src = smem_u32(ring + st.stage * kMassStageBytes);
          const int c = stages - i <= kMassChunks ? i - (stages - kMassChunks) : -1;
          if (c < 0) {  // a chunk of Q; the products that follow see it
            if (i < kMassChunks - 1) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                tmem_copy_128x32(tmem_q + i * 32 + kk * 8, smem_desc_sw128(src + kk * 32, 16, 1024));
            }
          } else if (c < kMassChunks - 1) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16_ts(tmem_d, tmem_q + c * 32 + kk * 8, smem_desc_sw128(src + kk * 32, 16, 1024),
                          idesc, (c > 0 || kk > 0) ? 1u : 0u);
          } else {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16_ss(tmem_d, smem_desc_sw128(smem_u32(sQ) + kk * 32, 16, 1024),
                          smem_desc_sw128(src + kk * 32, 16, 1024), idesc, 1u);
          }
          mma_commit(smem_u32(&kempty[st.stage]));
        }
        if (ok) mma_commit(smem_u32(tfull));
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      for (int i = 0; i < (new_q ? 2 : 1) * kMassChunks; ++i) at.next();
      ++tiles;
    }
    if (lane == 0) {
      mma_commit(smem_u32(mdone));
      mbar_wait(smem_u32(mdone), 0, TO, no_abort);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int quad = warp & 3, quarter = warp >> 2;
    const int head = quad * 32 + (lane >> 2);  // and + 8, + 16, + 24
    const int column = (lane & 16) + (lane & 8) + ((lane >> 2) & 1) + 2 * (lane & 3);
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    uint32_t tiles = 0;
    MassItems m;
    m.start(p);
    float next_lse[4] = {0.f, 0.f, 0.f, 0.f};
    auto load_lse = [&](const MassItems& i) {
      if (!i.live || i.t < 0) return;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        next_lse[r] = __ldg(p.lse + (int64_t)i.t * kMassHeads + head + 8 * r);
    };
    int sel = m.listed(p, tid);
    load_lse(m);
    while (m.live) {
      const MassItems now = m;
      float lse[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) lse[r] = next_lse[r];
      const bool now_used = mass_used(p, m, lane);
      const int slot = m.valid(sel) ? sel : -1;
      m.next(p);
      sel = m.listed(p, tid);
      if (m.t != now.t) load_lse(m);
      float w = 0.f;
      if (now_used) {
        // Warp 0 alone polls; the others sleep at the named barrier
        const bool got = warp != 0 || warp_wait(smem_u32(tfull), tiles & 1, TO, abort_flag);
        if (!named_barrier_and(1, kMassEpilogue, got)) break;
        tc_fence_after();
        MassBlock za, zb;
        const uint32_t col = tmem_d + lane_off + quarter * kMassQuarter;
        za.load(col);
        zb.load(col + 32);
        za.wait();
        zb.wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(tempty));
        const int n = now.columns(p) - quarter * kMassQuarter;
        float* part = sPart + ((tiles & 1) * 4 + quad) * kMassMaxTile + quarter * kMassQuarter;
        if (n > 0) part[column] = za.sum(p.scale, lse, lane);
        if (n > 32) part[32 + column] = zb.sum(p.scale, lse, lane);
        named_barrier_sync(2, kMassEpilogue);
        if (tid < kMassMaxTile) {
          const float* all = sPart + (tiles & 1) * 4 * kMassMaxTile + tid;
          w = (all[0] + all[kMassMaxTile]) + (all[2 * kMassMaxTile] + all[3 * kMassMaxTile]);
        }
        ++tiles;
      }
      w *= 1.0f / kMassHeads;
      const int e = now.tile * p.tile + tid;
      const float weight = w <= kMassMaxP ? w : __int_as_float(0x7fffffff);
      if (p.p_out) {
        if (now.t >= 0 && tid < p.tile && e < p.k)
          p.p_out[(int64_t)now.row * p.k + e] = slot < 0 ? 0.f : weight;
      } else if (slot >= 0) {
        unsigned long long* s = p.sums + (int64_t)now.b * p.max_ctx + slot;
        if (!p.sums)
          atomicAdd(p.mass + (int64_t)now.b * p.mass_ld + slot, weight);
        else if (w <= kMassMaxP)
          atomicAdd(s, (unsigned long long)__float2ll_rn(w * p.units));
        else
          atomicOr(s, kMassNan);
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem_q, 512);
  }
}

// Few rows: one CTA adds a sequence's rows in order, four entries of a thread at a time; the
// next ones are loaded before the barrier between two rows.
constexpr int kMassAddThreads = 512;
__global__ void __launch_bounds__(kMassAddThreads)
    mass_add_rows_kernel(const __grid_constant__ MassParams p) {
  const int b = blockIdx.x;
  const SeqRows R = seq_rows(p.q_start, p.seqlens, b, p.q_per_seq, p.num_q, p.max_ctx);
  if (!R.ok) return;
  const int last = min(p.row_begin + p.row_count, R.q_len);
  float* mass = p.mass + (int64_t)b * p.mass_ld;
  int sel[4];
  float w[4];
  auto load = [&](int qi, int e0) {
    const int32_t* idx = p.idx + (R.t0 + qi) * p.k;
    const float* row = p.p_out + ((int64_t)b * p.row_count + qi - p.row_begin) * p.k;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = e0 + j * kMassAddThreads + threadIdx.x;
      sel[j] = qi < last && e < p.k ? __ldg(idx + e) : -1;
      w[j] = qi < last && e < p.k ? __ldg(row + e) : 0.f;
    }
  };
  load(p.row_begin, 0);
  for (int qi = p.row_begin; qi < last; ++qi) {
    const int pos = R.seqlen - R.q_len + qi;
    for (int e0 = 0; e0 < p.k;) {
      int s[4];
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] = sel[j], v[j] = w[j];
      e0 += 4 * kMassAddThreads;
      e0 < p.k ? load(qi, e0) : load(qi + 1, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (s[j] >= 0 && s[j] <= pos) atomicAdd(mass + s[j], v[j]);
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
                    : *m + (float)((double)s / (double)p.units);
}

}  // namespace dsa
