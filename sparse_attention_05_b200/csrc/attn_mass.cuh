// attn_mass.cuh -- the attention weight every cached token received, accumulated.
//
// For query row t and its listed entries s (the sparse MLA's S_t, DeepSeek-V3.2-Exp
// technical report §1 Eq. 2) with the forward's per-head log-sum-exp,
//   p(t, s) = 1/128 sum_h exp(scale q_{t,h} . c_s - LSE_{t,h}),   mass[b][s] += sum_t p(t, s).
// The head mean is the main attention's distribution of the report's §2.1.
//
// Per listed entry 1152 B gathered and 147456 flops: 128 flops a byte, below the ~253
// at which this part's BF16 rate and HBM rate meet, so rows gathered from HBM are bound
// by the gather and rows that L2 holds by the tensor core. One CTA a query row: the row's
// Q (128 heads x 576) stays in shared memory as nine 128-B-swizzled chunks of 64 dims, the
// listed latent rows stream through a ring of 64-dim chunks, and
// D[entry][head] = K_tile (128 x 576) . Q^T lands in one of two TMEM accumulators, entries
// on the lanes, so that the sum over heads stays inside a thread.
//
// Warp roles (288 threads): 0-3 epilogue (thread = entry), 4 TMEM and MMA issue, 5-8
// producers (a warp's cp.async covers four whole 128-B lines, eight lanes a line; one
// line a lane would take eight times the tag lookups).
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
                               kMassHeads * 4 + 24 * 8 + 16;
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
  float scale_log2;
  uint64_t timeout_ns;
};

__global__ void __launch_bounds__(kMassThreads, 1)
    attn_mass_kernel(const __grid_constant__ MassParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + kMassChunks * kMassChunkBytes;
  float* sLse2 = reinterpret_cast<float*>(sK + kMassStages * kMassChunkBytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sLse2 + kMassHeads);
  uint64_t* kfull = bars;
  uint64_t* kempty = kfull + kMassStages;
  uint64_t* tfull = kempty + kMassStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* qfull = tempty + 2;
  uint64_t* mdone = qfull + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(mdone + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t local = blockIdx.x;
  const int b = (int)(local / p.row_count);
  const int qi = p.row_begin + (int)(local - (int64_t)b * p.row_count);
  const SeqRows R = seq_rows(p.q_start, p.seqlens, b, p.q_per_seq, p.num_q, p.max_ctx);
  if (!R.ok || qi >= R.q_len) {
    if (tid == 0 && !R.ok) report_error(kErrBounds);
    return;
  }
  const int64_t t = R.t0 + qi;
  const int pos = R.seqlen - R.q_len + qi;
  const int ntiles = (p.k + kMassTile - 1) / kMassTile;

  if (tid == 0) {
    for (int i = 0; i < kMassStages; ++i) {
      mbar_init(smem_u32(&kfull[i]), 128);
      mbar_init(smem_u32(&kempty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&tfull[i]), 1);
      mbar_init(smem_u32(&tempty[i]), 128);
    }
    mbar_init(smem_u32(qfull), 256);
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
    const uint8_t* qrow = reinterpret_cast<const uint8_t*>(p.q + t * kMassHeads * kMassDqk);
#pragma unroll 1
    for (int c = 0; c < kMassChunks; ++c) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int h = pw * 32 + i * 4 + sub;
        cp_async_16(smem_u32(sQ + c * kMassChunkBytes) + sw128_offset(h, piece),
                    qrow + h * (kMassDqk * 2) + c * 128 + piece * 16, 16u);
      }
    }
    sLse2[tid - 160] = __ldg(p.lse + t * kMassHeads + tid - 160) * 1.4426950408889634f;
    mbar_arrive(smem_u32(qfull));           // the LSE row
    cp_async_mbar_arrive(smem_u32(qfull));  // Q, once it has landed
    uint32_t it = 0;
    bool ok = true;
    for (int tile = 0; tile < ntiles && ok; ++tile) {
      const int e = tile * kMassTile + pw * 32 + lane;
      const int sel = e < p.k ? __ldg(p.idx + t * p.k + e) : -1;
      int row = -1;
      if (sel >= 0 && sel <= pos) {
        if (!p.paged) {
          row = b * p.max_ctx + sel;
        } else {
          const int pg = __ldg(p.block_table + (int64_t)b * p.max_pages + sel / p.page_size);
          if (pg >= 0 && pg < p.num_pages)
            row = pg * p.page_size + sel % p.page_size;
          else
            report_error(kErrBounds);
        }
      }
      int rows[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) rows[i] = __shfl_sync(0xffffffffu, row, i * 4 + sub);
#pragma unroll 1
      for (int c = 0; c < kMassChunks; ++c, ++it) {
        const int st = it % kMassStages;
        if (!warp_wait(smem_u32(&kempty[st]), ((it / kMassStages) & 1) ^ 1, TO, abort_flag)) {
          ok = false;
          break;
        }
        const uint32_t dst = smem_u32(sK + st * kMassChunkBytes);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          cp_async_16(dst + sw128_offset(pw * 32 + i * 4 + sub, piece),
                      p.kv + (int64_t)max(rows[i], 0) * (kMassDqk * 2) + c * 128 + piece * 16,
                      rows[i] >= 0 ? 16u : 0u);
        cp_async_mbar_arrive(smem_u32(&kfull[st]));
      }
    }
    cp_async_wait_all();
  } else if (warp == 4) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t idesc = instr_desc(1 /*bf16*/, 0, 0, 128, 128);
      uint32_t it = 0;
      bool ok = mbar_wait(smem_u32(qfull), 0, TO, abort_flag);
      for (int tile = 0; tile < ntiles && ok; ++tile) {
        const int ab = tile & 1;
        if (!mbar_wait(smem_u32(&tempty[ab]), ((tile >> 1) & 1) ^ 1, TO, abort_flag)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + ab * 128;
        for (int c = 0; c < kMassChunks; ++c, ++it) {
          const int st = it % kMassStages;
          if (!mbar_wait(smem_u32(&kfull[st]), (it / kMassStages) & 1, TO, abort_flag)) {
            ok = false;
            break;
          }
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
      mma_commit(smem_u32(mdone));
      mbar_wait(smem_u32(mdone), 0, TO, no_abort);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    bool ok = warp_wait(smem_u32(qfull), 0, TO, abort_flag);
    for (int tile = 0; tile < ntiles && ok; ++tile) {
      const int ab = tile & 1;
      const int e = tile * kMassTile + warp * 32 + lane;
      const int sel = e < p.k ? __ldg(p.idx + t * p.k + e) : -1;
      ok = warp_wait(smem_u32(&tfull[ab]), (tile >> 1) & 1, TO, abort_flag);
      if (!ok) break;
      tc_fence_after();
      float w = 0.f;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        float z[32];
        tmem_ld32(tmem_base + ab * 128 + c * 32 + lane_off, z);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) w += ex2_approx(z[i] * p.scale_log2 - sLse2[c * 32 + i]);
      }
      tc_fence_before();
      mbar_arrive(smem_u32(&tempty[ab]));
      const bool valid = sel >= 0 && sel <= pos;
      w *= 1.0f / kMassHeads;
      if (p.sums) {
        if (valid) {
          unsigned long long* s = p.sums + (int64_t)b * p.max_ctx + sel;
          if (w <= kMassMaxP)
            atomicAdd(s, (unsigned long long)__float2ll_rn(w * kMassUnit));
          else
            atomicOr(s, kMassNan);
        }
      } else if (e < p.k) {
        p.p_out[local * p.k + e] = !valid ? 0.f : w <= kMassMaxP ? w : __int_as_float(0x7fffffff);
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
