// evict.cuh -- which cached tokens stay when a sequence's caches are trimmed.
//
// Of a sequence of n tokens the first `sink` and the last `recent` stay, and of those
// between them the keep - sink - recent with the most accumulated attention mass (ties
// to the lower slot). The order is that of the mass's bits made monotone; -0 counts as
// +0 and a NaN ranks below every number.
//
// Radix select over 11 + 11 + 10 bits of the key. The mass is 4 B a slot; what a call waits
// for is a chain of short steps, so a cluster of up to eight CTAs takes a sequence, each a run
// of its slots (the keys held in shared memory where they fit), and only two steps look at
// every key: the first histogram, and a sweep that turns the keys above the border bin and
// those in it into two bitmaps. The later digits look at the second bitmap's slots alone, and
// the slots are written from the bitmaps in order. Where the border bin holds nothing but
// zeros (the slots no query ever chose), there are no later digits: 128 x 131072 slots, nine
// in ten of them zero, half kept, take 62 us, not 116.
// A cluster's histograms meet through 16 partial sums per CTA: one warp of each CTA finds
// the group of 128 bins that holds the border and then loads just that group from the
// other CTAs (the whole histograms would be 56 KB a CTA over distributed shared memory). The
// same loads tell a CTA how many kept slots lie in the CTAs before it.
#pragma once

#include <type_traits>

#include "ptx.cuh"

namespace dsa {

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictBins = 2048;
constexpr int kEvictGroup = kEvictBins / kEvictWarps;  // bins of one partial sum
constexpr int kEvictLoads = 16;           // of a thread, in flight
constexpr int kEvictStage = 1024 + 32;    // slots of 32 words, an element apart every 32 (banks)
constexpr int kEvictRest = 4;             // and at the end of its run
// Members of a bitmap word up to which its own thread takes them.
constexpr int kEvictSparse = 16;
constexpr int kEvictMaxSplits = 8;
constexpr int kEvictMaxKeys = 45056;      // keys a CTA holds in shared memory (176 KB)
constexpr int kEvictPairKeys = 18432;     // and each of two CTAs on an SM
constexpr int kEvictRunBits = 262144;     // slots whose two bitmaps each of two CTAs holds
constexpr int kEvictMaxCtx = 1 << 22;     // two bits a slot fit in shared memory up to here
constexpr int kEvictMaxDynamic = kEvictMaxKeys * 4 + kEvictMaxKeys / 4;
static_assert(2 * (kEvictPairKeys * 4 + kEvictPairKeys / 4 + 35840 + 1024) <= 228 * 1024 &&
                  2 * (kEvictRunBits / 4 + 35840 + 1024) <= 228 * 1024,
              "two CTAs an SM");
static_assert(kEvictMaxCtx / kEvictMaxSplits / 4 + 64 <= kEvictMaxDynamic, "bitmaps do not fit");

struct EvictShared {
  union {
    int hist[4][kEvictBins];      // of the three digits; [3]: the first digit's odd lanes
    uint16_t stage[kEvictWarps][kEvictStage];  // at the end: a warp's slots, in order
  };
  int sums[3][kEvictWarps];     // of each group of bins, from the top down
  int scan[2][kEvictWarps];
  int zeros;                    // of this CTA's slots
  int found[5];
};

struct EvictParams {
  const float* mass;         // [batch][ld]
  const int32_t* seqlens;    // [batch] or nullptr
  int32_t* kept;             // [batch][keep]
  int32_t* new_lens;         // [batch]
  int64_t ld;
  int32_t max_ctx, keep, sink, recent;
  int32_t splits;            // CTAs of a sequence's cluster
  int32_t run;               // most slots of one CTA, a multiple of 32
};

constexpr uint32_t kEvictZero = 0x80000000u;  // evict_key(0)

__device__ __forceinline__ uint32_t evict_key(float m) {
  if (m != m) return 0u;
  const uint32_t u = __float_as_uint(m + 0.0f);  // -0 + 0 = +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int4 ld_cluster_v4(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ int ld_cluster(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// One more in a bin, by a predicate: no branch around each key's.
__device__ __forceinline__ void count_if(uint32_t bin, bool counts) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %1, 0;\n\t@p red.shared.add.u32 [%0], 1;\n\t}" ::"r"(bin),
      "r"((int)counts)
      : "memory");
}

__device__ __forceinline__ int warp_inclusive(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// The cluster's barrier in two halves.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// After every CTA's histogram `pass`: the digit at which the count from the top reaches
// `left`, and what is left of it inside that bin; of the CTAs before this one, the keys above
// that bin and in it; and after the first whether that bin holds zeros only (all in sh.found).
__device__ __forceinline__ void evict_digit(EvictShared& sh, int pass, int left, int rank,
                                            int splits) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  {  // group `warp` from the top: bins 2047 - 128 warp downwards
    const int at = kEvictBins - kEvictGroup * (warp + 1) + 4 * lane;
    int4 c = *reinterpret_cast<const int4*>(&sh.hist[pass][at]);
    if (pass == 0) {
      const int4 odd = *reinterpret_cast<const int4*>(&sh.hist[3][at]);
      c.x += odd.x, c.y += odd.y, c.z += odd.z, c.w += odd.w;
      *reinterpret_cast<int4*>(&sh.hist[0][at]) = c;
    }
    const int s = __reduce_add_sync(0xffffffffu, c.x + c.y + c.z + c.w);
    if (lane == 0) sh.sums[pass][warp] = s;
  }
  cluster_sync_all();
  if (warp == 0) {
    // lane l: group l of all CTAs (half of the lanes have none)
    const uint32_t sums = smem_u32(&sh.sums[pass][lane & (kEvictWarps - 1)]);
    int v[kEvictMaxSplits];
#pragma unroll
    for (int r = 0; r < kEvictMaxSplits; ++r) v[r] = r < splits ? ld_cluster(mapa_shared(sums, r)) : 0;
    int zeros = 0;  // every lane: of all CTAs
    if (pass == 0)
      zeros = __reduce_add_sync(0xffffffffu, lane < splits ? ld_cluster(mapa_shared(smem_u32(&sh.zeros), lane)) : 0);
    int all = 0, mine = 0;
#pragma unroll
    for (int r = 0; r < kEvictMaxSplits; ++r) all += v[r], mine += r < rank ? v[r] : 0;
    int upto = warp_inclusive(all, lane);
    const int group = __ffs(__ballot_sync(0xffffffffu, upto >= left)) - 1;
    const int above = __shfl_sync(0xffffffffu, upto - all, group);
    // lane l: four bins of that group, the highest first
    const int first = kEvictBins - kEvictGroup * group - 4 * (lane + 1);
    const uint32_t addr = smem_u32(&sh.hist[pass][first]);
    int4 c[kEvictMaxSplits];
#pragma unroll
    for (int r = 0; r < kEvictMaxSplits; ++r)
      c[r] = r < splits ? ld_cluster_v4(mapa_shared(addr, r)) : make_int4(0, 0, 0, 0);
    int4 sum = make_int4(0, 0, 0, 0), part = make_int4(0, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < kEvictMaxSplits; ++r) {
      sum.x += c[r].x, sum.y += c[r].y, sum.z += c[r].z, sum.w += c[r].w;
      if (r < rank) part.x += c[r].x, part.y += c[r].y, part.z += c[r].z, part.w += c[r].w;
    }
    const int down[4] = {sum.w, sum.z, sum.y, sum.x}, ours[4] = {part.w, part.z, part.y, part.x};
    const int four = down[0] + down[1] + down[2] + down[3];
    int before = above + warp_inclusive(four, lane) - four;
    mine = lane < group ? mine : 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int next = before + down[j];
      if (before < left && next >= left) {
        sh.found[0] = first + 3 - j;
        sh.found[1] = left - before;
        sh.found[3] = ours[j];
        sh.found[4] = down[j] == zeros && pass == 0 && sh.found[0] == (int)(kEvictZero >> 21);
      }
      if (next < left) mine += ours[j];
      before = next;
    }
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0) sh.found[2] = mine;
  }
  __syncthreads();
}

// kHold: the keys stay in shared memory.
template <bool kHold>
__global__ void __launch_bounds__(kEvictThreads, 2)
    evict_select_kernel(const EvictParams p) {
  extern __shared__ uint32_t evict_smem[];
  __shared__ __align__(16) EvictShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / p.splits, rank = blockIdx.x % p.splits;
  int n = p.seqlens ? __ldg(p.seqlens + b) : p.max_ctx;
  int32_t* kept = p.kept + (int64_t)b * p.keep;
  const int gtid = rank * kEvictThreads + tid, gthreads = p.splits * kEvictThreads;
  if (n < 0 || n > p.max_ctx) {
    if (gtid == 0) report_error(kErrBounds);
    n = 0;
  }
  if (gtid == 0) p.new_lens[b] = min(n, p.keep);
  if (n <= p.keep) {
    for (int64_t i = gtid; i < p.keep; i += gthreads) kept[i] = i < n ? (int)i : -1;  // keep + a stride: past 2^31
    return;
  }
  const int want = p.keep - p.sink - p.recent;  // of [sink, n - recent), which holds more
  for (int i = gtid; i < p.sink; i += gthreads) kept[i] = i;
  for (int i = gtid; i < p.recent; i += gthreads) kept[p.sink + want + i] = n - p.recent + i;
  if (want == 0) return;
  // this CTA's run of the middle, a multiple of 32 slots but for the end
  const int middle = n - p.recent - p.sink;
  const int run = ((middle + p.splits - 1) / p.splits + 31) & ~31;
  const int begin = min(p.sink + rank * run, n - p.recent);
  const int count = min(run, n - p.recent - begin), words = (count + 31) >> 5;
  const float* mass = p.mass + (int64_t)b * p.ld + begin;
  uint32_t* bits_above = evict_smem;                  // [run / 32]
  uint32_t* bits_at = bits_above + (p.run >> 5);      // [run / 32]
  uint32_t* keys = bits_at + (p.run >> 5);            // [run] where they are held
  auto key_at = [&](int i) { return kHold ? keys[i] : evict_key(__ldg(mass + i)); };
  if (tid == 0) sh.zeros = 0;
  for (int i = tid; i < 4 * kEvictBins; i += kEvictThreads) (&sh.hist[0][0])[i] = 0;
  __syncthreads();
  // The slots no query ever chose share one key; a thread counts its own of them.
  int zeros = 0;
  auto add = [&](int pass, int digit, uint32_t key, bool member) {
    if (member && key == kEvictZero) ++zeros;
    count_if(smem_u32(&sh.hist[pass][digit]), member && key != kEvictZero);
  };
  auto add_zeros = [&](int pass, int digit) {
    zeros = __reduce_add_sync(0xffffffffu, zeros);
    if (lane == 0 && zeros) {
      atomicAdd(&sh.hist[pass][digit], zeros);
      if (pass == 0) atomicAdd(&sh.zeros, zeros);
    }
    zeros = 0;
  };
  // f over the warp's slots: many loads at a time while they are whole, few after
  auto sweep = [&](auto f) {
    for (int i0 = warp * 32; i0 < count; i0 += kEvictThreads * kEvictLoads) {
      if (i0 + kEvictThreads * (kEvictLoads - 1) + 32 <= count) {
        f(i0, std::true_type{});
      } else {
#pragma unroll 1
        for (int i = i0; i < count; i += kEvictThreads * kEvictRest)
          f(i, std::false_type{});
      }
    }
  };
  const int first = lane & 1 ? 3 : 0;
  auto histogram = [&](int i0, auto whole) {  // whole: all of the warp's slots are the CTA's
    constexpr bool kWhole = decltype(whole)::value;
    constexpr int kLoads = kWhole ? kEvictLoads : kEvictRest;
    float m[kLoads];  // in flight at once
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int i = i0 + j * kEvictThreads + lane;
      m[j] = kWhole || i < count ? __ldg(mass + i) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int i = i0 + j * kEvictThreads + lane;
      const uint32_t key = evict_key(m[j]);
      if (kHold && (kWhole || i < count)) keys[i] = key;
      add(first, key >> 21, key, kWhole || i < count);
    }
  };
  sweep(histogram);
  add_zeros(0, kEvictZero >> 21);
  evict_digit(sh, 0, want, rank, p.splits);
  const uint32_t top = sh.found[0];
  int left = sh.found[1];
  int g = sh.found[2];  // keys above the border in the CTAs before this one
  int e = sh.found[3];  // and at it
  const bool decided = sh.found[4];
  // the bitmaps, and the second digit of the keys in the border bin (zeros only: nothing left
  // to decide but their slots)
  auto border = [&](int i0, auto whole) {
    constexpr bool kWhole = decltype(whole)::value;
    constexpr int kLoads = kWhole ? kEvictLoads : kEvictRest;
    uint32_t key[kLoads];
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int i = i0 + j * kEvictThreads + lane;
      key[j] = kWhole || i < count ? key_at(i) : 0u;
    }
    uint32_t above = 0, at = 0;  // lane j: the word of the j-th load
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const bool in = kWhole || i0 + j * kEvictThreads + lane < count;
      const uint32_t digit = key[j] >> 21;
      const uint32_t a = __ballot_sync(0xffffffffu, in && digit > top);
      const uint32_t e = __ballot_sync(0xffffffffu, in && digit == top);
      if (lane == j) above = a, at = e;
      if (e) add(1, (key[j] >> 10) & 2047, key[j], in && digit == top);
    }
    const int w = (i0 >> 5) + lane * kEvictWarps;
    if (lane < kLoads && w < words) bits_above[w] = above, bits_at[w] = at;
  };
  sweep(border);
  add_zeros(1, 0);
  // The slots of the second bitmap against a digit: above it, or still at it. A thread takes
  // a word (or several, for as many loads in flight), from another bit on than its neighbours
  // (the keys then lie in different banks); where words are dense, the warp takes them one by
  // one.
  auto refine = [&](int shift, uint32_t mask, uint32_t digit, bool next) {
    constexpr int kWords = kHold ? 1 : 4;
    for (int w0 = warp * 32; w0 < words; w0 += kWords * kEvictThreads) {
      uint32_t todo[kWords], most = 0;
#pragma unroll
      for (int k = 0; k < kWords; ++k) {
        const int w = w0 + k * kEvictThreads + lane;
        const uint32_t members = w < words ? bits_at[w] : 0u;
        most = max(most, (uint32_t)__popc(members));
        todo[k] = __funnelshift_r(members, members, lane);
      }
      if (__reduce_max_sync(0xffffffffu, most) <= kEvictSparse) {
        uint32_t above[kWords] = {}, at[kWords] = {};
        bool more;
        do {
          uint32_t key[kWords];
          int bit[kWords];
#pragma unroll
          for (int k = 0; k < kWords; ++k) {
            bit[k] = (__ffs(todo[k]) - 1 + lane) & 31;
            key[k] = todo[k] ? key_at((w0 + k * kEvictThreads + lane) * 32 + bit[k]) : 0u;
          }
          more = false;
#pragma unroll
          for (int k = 0; k < kWords; ++k) {
            const uint32_t d = (key[k] >> shift) & mask;
            const bool equal = todo[k] && d == digit;
            if (todo[k] && d > digit) above[k] |= 1u << bit[k];
            if (equal) at[k] |= 1u << bit[k];
            if (next) add(2, key[k] & 1023, key[k], equal);
            todo[k] &= todo[k] - 1;
            more |= todo[k] != 0;
          }
        } while (more);
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
          const int w = w0 + k * kEvictThreads + lane;
          if (w < words) bits_above[w] |= above[k], bits_at[w] = at[k];
        }
        continue;
      }
#pragma unroll 1
      for (int w1 = w0; w1 < min(words, w0 + kWords * kEvictThreads); w1 += kEvictThreads) {
        const int w = w1 + lane;
        const uint32_t members = w < words ? bits_at[w] : 0u;
        uint32_t above = 0, at = 0;
        constexpr int kLoads = 8;
#pragma unroll 1
        for (int j0 = 0; j0 < 32; j0 += kLoads) {
          uint32_t key[kLoads];
          bool in[kLoads];
#pragma unroll
          for (int j = 0; j < kLoads; ++j) {
            in[j] = (__shfl_sync(0xffffffffu, members, j0 + j) >> lane) & 1;
            key[j] = key_at(min((w1 + j0 + j) * 32 + lane, count - 1));
          }
#pragma unroll
          for (int j = 0; j < kLoads; ++j) {
            const uint32_t d = (key[j] >> shift) & mask;
            const uint32_t a = __ballot_sync(0xffffffffu, in[j] && d > digit);
            const uint32_t e = __ballot_sync(0xffffffffu, in[j] && d == digit);
            if (lane == j0 + j) above = a, at = e;
            if (next) add(2, key[j] & 1023, key[j], in[j] && d == digit);
          }
        }
        if (w < words) bits_above[w] |= above, bits_at[w] = at;
      }
    }
    if (next) add_zeros(2, 0);
  };
  if (!decided) {
    evict_digit(sh, 1, left, rank, p.splits);
    const uint32_t second = sh.found[0];
    left = sh.found[1];
    g += sh.found[2];
    refine(10, 2047, second, true);
    evict_digit(sh, 2, left, rank, p.splits);
  }
  cluster_arrive();  // nothing of another CTA is read from here on
  if (!decided) {
    const uint32_t third = sh.found[0];
    left = sh.found[1];
    g += sh.found[2];
    e = sh.found[3];
    refine(0, 1023, third, false);
  }
  __syncthreads();
  // The slots in order, all those above and of those at the border the first `left`: each
  // warp its share of the words, after those of the warps before it.
  const int share = ((words + kEvictWarps - 1) / kEvictWarps + 31) & ~31;
  const int w_end = min(words, (warp + 1) * share);
  int ng = 0, ne = 0;
  for (int w = warp * share + lane; w < w_end; w += 32) {
    ng += __popc(bits_above[w]);
    ne += __popc(bits_at[w]);
  }
  ng = __reduce_add_sync(0xffffffffu, ng);
  ne = __reduce_add_sync(0xffffffffu, ne);
  if (lane == 0) sh.scan[0][warp] = ng, sh.scan[1][warp] = ne;
  cluster_wait();  // no CTA reads this one's histograms any more
  __syncthreads();
#pragma unroll
  for (int v = 0; v < kEvictWarps; ++v) {
    const int a = sh.scan[0][v], c = sh.scan[1][v];
    if (v < warp) g += a, e += c;
  }
  uint16_t* stage = sh.stage[warp];
  for (int w0 = warp * share; w0 < w_end; w0 += 32) {
    const int w = w0 + lane;
    const uint32_t above = w < w_end ? bits_above[w] : 0u;
    uint32_t at = w < w_end ? bits_at[w] : 0u;
    const int ng = __popc(above), ne = __popc(at);
    const int ig = warp_inclusive(ng, lane), ie = warp_inclusive(ne, lane);
    const int be = e + ie - ne, take = left - be;
    if (take <= 0) at = 0;
    for (int over = ne - take; take > 0 && over > 0; --over) at &= ~(0x80000000u >> __clz(at));
    // the warp's slots go through shared memory to consecutive places
    const uint32_t word = above | at;
    const int place = p.sink + g + ig - ng + min(be, left);
    const int to = __shfl_sync(0xffffffffu, place, 0);
    const int total = __shfl_sync(0xffffffffu, place + __popc(word), 31) - to;
    int i = place - to;
    for (uint32_t todo = word; todo; todo &= todo - 1, ++i)
      stage[i + (i >> 5)] = (uint16_t)(lane * 32 + __ffs(todo) - 1);
    __syncwarp();
    const int slot0 = begin + w0 * 32;
#pragma unroll 4
    for (int i = lane; i < total; i += 32) kept[to + i] = slot0 + stage[i + (i >> 5)];
    __syncwarp();
    g += __shfl_sync(0xffffffffu, ig, 31);
    e += __shfl_sync(0xffffffffu, ie, 31);
  }
}

}  // namespace dsa
