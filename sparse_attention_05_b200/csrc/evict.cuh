// evict.cuh -- which cached tokens stay when a sequence's caches are trimmed.
//
// Of a sequence of n tokens the first `sink` and the last `recent` stay, and of those
// between them the keep - sink - recent with the most accumulated attention mass (ties
// to the lower slot). The order is that of the mass's bits made monotone; -0 counts as
// +0 and a NaN ranks below every number.
//
// Radix select over 11 + 11 + 10 bits of the key. The mass is 4 B a slot, read once; what
// a call waits for is a chain of short steps, so a cluster of up to eight CTAs takes a
// sequence, each a run of its slots with the keys held in shared memory, and only two
// steps look at every key: the first histogram, and a sweep that turns the keys above the
// border bin and those in it into two bitmaps. The later digits look at the second
// bitmap's slots alone, and the slots are written from the bitmaps in order.
// A cluster's histograms meet through 16 partial sums per CTA: one warp of each CTA finds
// the group of 128 bins that holds the border and then loads just that group from the
// other CTAs (the whole histograms would be 56 KB a CTA over distributed shared memory).
#pragma once

#include <type_traits>

#include "ptx.cuh"

namespace dsa {

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictBins = 2048;
constexpr int kEvictGroup = kEvictBins / kEvictWarps;  // bins of one partial sum
constexpr int kEvictLoads = 16;           // of a thread, in flight
// Slots of a bitmap word up to which its own thread writes them: the stores of a warp's
// threads lie apart, but there are few. Denser words are written by the whole warp, a word at
// a time. (128 x 131072, keeping an eighth: 81 us by threads, 85 by warps; half of tied masses:
// 240 and 133.)
constexpr int kEvictSparse = 16;
constexpr int kEvictMaxSplits = 8;
constexpr int kEvictMaxKeys = 45056;      // keys a CTA holds in shared memory (176 KB)
constexpr int kEvictMaxCtx = 1 << 22;     // two bits a slot fit in shared memory up to here
constexpr int kEvictMaxDynamic = kEvictMaxKeys * 4 + kEvictMaxKeys / 4;
static_assert(kEvictMaxCtx / kEvictMaxSplits / 4 + 64 <= kEvictMaxDynamic, "bitmaps do not fit");

struct EvictShared {
  int hist[4][kEvictBins];      // of the three digits; [3]: the first digit's odd lanes
  int sums[3][kEvictWarps];     // of each group of bins, from the top down
  int scan[2][kEvictWarps];
  int counts[2];                // this CTA's slots above and at the border
  int found[2];
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
  int32_t hold;              // its keys stay in shared memory
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

__device__ __forceinline__ int2 ld_cluster_v2(uint32_t addr) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ int warp_inclusive(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// After every CTA's histogram `pass`: the digit at which the count from the top reaches
// `left`, and what is left of it inside that bin (in sh.found).
__device__ __forceinline__ void evict_digit(EvictShared& sh, int pass, int left, int splits) {
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
    // lane: four groups of one CTA
    int4 s = make_int4(0, 0, 0, 0);
    if ((lane >> 2) < splits)
      s = ld_cluster_v4(mapa_shared(smem_u32(&sh.sums[pass][4 * (lane & 3)]), lane >> 2));
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
      s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
      s.z += __shfl_xor_sync(0xffffffffu, s.z, o);
      s.w += __shfl_xor_sync(0xffffffffu, s.w, o);
    }
    // every lane: the sums of all groups above its own four, then the group of the border
    const int mine = s.x + s.y + s.z + s.w;
    int before = 0;
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      const int v = __shfl_sync(0xffffffffu, mine, q);
      if (q < (lane & 3)) before += v;
    }
    const int part[4] = {s.x, s.y, s.z, s.w};
    int group = -1, above = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (before < left && before + part[j] >= left) {
        group = 4 * (lane & 3) + j;
        above = before;
      }
      before += part[j];
    }
    const int owner = __ffs(__ballot_sync(0xffffffffu, group >= 0)) - 1;
    group = __shfl_sync(0xffffffffu, group, owner);
    above = __shfl_sync(0xffffffffu, above, owner);
    // lane l: four bins of that group, the highest first
    const int first = kEvictBins - kEvictGroup * group - 4 * (lane + 1);
    const uint32_t addr = smem_u32(&sh.hist[pass][first]);
    int4 c[kEvictMaxSplits];
#pragma unroll
    for (int r = 0; r < kEvictMaxSplits; ++r)
      c[r] = r < splits ? ld_cluster_v4(mapa_shared(addr, r)) : make_int4(0, 0, 0, 0);
#pragma unroll
    for (int r = 1; r < kEvictMaxSplits; ++r)
      c[0].x += c[r].x, c[0].y += c[r].y, c[0].z += c[r].z, c[0].w += c[r].w;
    const int down[4] = {c[0].w, c[0].z, c[0].y, c[0].x};
    const int sum = down[0] + down[1] + down[2] + down[3];
    before = above + warp_inclusive(sum, lane) - sum;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (before < left && before + down[j] >= left) {
        sh.found[0] = first + 3 - j;
        sh.found[1] = left - before;
      }
      before += down[j];
    }
  }
  __syncthreads();
}

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
    for (int i = gtid; i < p.keep; i += gthreads) kept[i] = i < n ? i : -1;
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
  auto key_at = [&](int i) { return p.hold ? keys[i] : evict_key(__ldg(mass + i)); };
  for (int i = tid; i < 4 * kEvictBins; i += kEvictThreads) (&sh.hist[0][0])[i] = 0;
  __syncthreads();
  // The slots no query ever chose share one key; a thread counts its own of them.
  int zeros = 0;
  auto add = [&](int* hist, int digit, uint32_t key, bool member) {
    if (member && key == kEvictZero) ++zeros;
    if (member && key != kEvictZero) atomicAdd(hist + digit, 1);
  };
  auto add_zeros = [&](int* bin) {
    zeros = __reduce_add_sync(0xffffffffu, zeros);
    if (lane == 0 && zeros) atomicAdd(bin, zeros);
    zeros = 0;
  };
  int* first = sh.hist[lane & 1 ? 3 : 0];
  auto histogram = [&](int i0, auto whole) {  // whole: all of the warp's slots are the CTA's
    constexpr bool kWhole = decltype(whole)::value;
    float m[kEvictLoads];  // in flight at once
#pragma unroll
    for (int j = 0; j < kEvictLoads; ++j) {
      const int i = i0 + j * kEvictThreads + lane;
      m[j] = kWhole || i < count ? __ldg(mass + i) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kEvictLoads; ++j) {
      const int i = i0 + j * kEvictThreads + lane;
      const uint32_t key = evict_key(m[j]);
      if (p.hold && (kWhole || i < count)) keys[i] = key;
      add(first, key >> 21, key, kWhole || i < count);
    }
  };
  for (int i0 = warp * 32; i0 < count; i0 += kEvictThreads * kEvictLoads) {
    if (i0 + kEvictThreads * (kEvictLoads - 1) + 32 <= count)
      histogram(i0, std::true_type{});
    else
      histogram(i0, std::false_type{});
  }
  add_zeros(&sh.hist[0][kEvictZero >> 21]);
  evict_digit(sh, 0, want, p.splits);
  const uint32_t top = sh.found[0];
  int left = sh.found[1];
  // the bitmaps, and the second digit of the keys in the border bin
#pragma unroll 4
  for (int i0 = warp * 32; i0 < count; i0 += kEvictThreads) {
    const bool in = i0 + lane < count;
    const uint32_t key = in ? key_at(i0 + lane) : 0u, digit = key >> 21;
    const uint32_t above = __ballot_sync(0xffffffffu, in && digit > top);
    const bool at = in && digit == top;
    const uint32_t equal = __ballot_sync(0xffffffffu, at);
    if (lane == 0) {
      bits_above[i0 >> 5] = above;
      bits_at[i0 >> 5] = equal;
    }
    if (equal) add(sh.hist[1], (key >> 10) & 2047, key, at);
  }
  add_zeros(&sh.hist[1][0]);
  // the slots of the second bitmap against a digit: above it, or still at it. A thread
  // takes whole words, each from another bit on (the keys then lie in different banks).
  auto refine = [&](int shift, uint32_t mask, uint32_t digit, bool next) {
    for (int w = tid; w < words; w += kEvictThreads) {
      uint32_t todo = __funnelshift_r(bits_at[w], bits_at[w], lane), above = 0, at = 0;
      while (todo) {
        const int bit = (__ffs(todo) - 1 + lane) & 31;
        todo &= todo - 1;
        const uint32_t key = key_at(w * 32 + bit), d = (key >> shift) & mask;
        if (d > digit) {
          above |= 1u << bit;
        } else if (d == digit) {
          at |= 1u << bit;
          if (next) add(sh.hist[2], key & 1023, key, true);
        }
      }
      bits_above[w] |= above;
      bits_at[w] = at;
    }
    if (next) add_zeros(&sh.hist[2][0]);
  };
  evict_digit(sh, 1, left, p.splits);
  const uint32_t second = sh.found[0];
  left = sh.found[1];
  refine(10, 2047, second, true);
  evict_digit(sh, 2, left, p.splits);
  const uint32_t third = sh.found[0];
  left = sh.found[1];
  refine(0, 1023, third, false);
  __syncthreads();
  // what lies before this CTA's slots
  int g = 0, e = 0;
  for (int w = tid; w < words; w += kEvictThreads) {
    g += __popc(bits_above[w]);
    e += __popc(bits_at[w]);
  }
  g = __reduce_add_sync(0xffffffffu, g);
  e = __reduce_add_sync(0xffffffffu, e);
  if (lane == 0) sh.scan[0][warp] = g, sh.scan[1][warp] = e;
  __syncthreads();
  if (tid == 0) {
    g = e = 0;
    for (int w = 0; w < kEvictWarps; ++w) g += sh.scan[0][w], e += sh.scan[1][w];
    sh.counts[0] = g, sh.counts[1] = e;
  }
  cluster_sync_all();
  g = e = 0;
  for (int r = 0; r < rank; ++r) {
    const int2 v = ld_cluster_v2(mapa_shared(smem_u32(&sh.counts[0]), r));
    g += v.x, e += v.y;
  }
  // the slots in order: all those above, and of those at the border the first `left`
  for (int w0 = 0; w0 < words; w0 += kEvictThreads) {
    const int w = w0 + tid;
    const uint32_t above = w < words ? bits_above[w] : 0u;
    uint32_t at = w < words ? bits_at[w] : 0u;
    const int ng = __popc(above), ne = __popc(at);
    const int ig = warp_inclusive(ng, lane), ie = warp_inclusive(ne, lane);
    if (lane == 31) sh.scan[0][warp] = ig, sh.scan[1][warp] = ie;
    __syncthreads();
    int bg = g + ig - ng, be = e + ie - ne;
    for (int v = 0; v < kEvictWarps; ++v) {
      const int a = sh.scan[0][v], c = sh.scan[1][v];
      if (v < warp) bg += a, be += c;
      g += a, e += c;
    }
    for (int over = ne - max(0, left - be); over > 0 && at; --over) at &= ~(0x80000000u >> __clz(at));
    const uint32_t word = above | at;
    int place = p.sink + bg + min(be, left);
    if (__reduce_max_sync(0xffffffffu, (uint32_t)__popc(word)) <= kEvictSparse) {
      for (uint32_t todo = word; todo; todo &= todo - 1)
        kept[place++] = begin + w * 32 + __ffs(todo) - 1;
    } else {
#pragma unroll 4
      for (int j = 0; j < 32; ++j) {
        const uint32_t m = __shfl_sync(0xffffffffu, word, j);
        const int to = __shfl_sync(0xffffffffu, place, j);
        if ((m >> lane) & 1)
          kept[to + __popc(m & ((1u << lane) - 1))] = begin + (w0 + warp * 32 + j) * 32 + lane;
      }
    }
    __syncthreads();
  }
  cluster_sync_all();  // no CTA leaves while another still reads its shared memory
}

}  // namespace dsa
