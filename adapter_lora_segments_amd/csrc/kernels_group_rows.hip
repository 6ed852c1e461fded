// Stable grouping of rows by id on the device: offsets of the groups and the
// order of the rows, the counting sort of mlora_plan_from_ids for ids that
// only the device holds.
//
// Position of row i = (rows in lower groups) + (earlier rows of its group).
// Every wave owns a contiguous run of rows.  A first pass counts each wave's
// rows per group; sums over the groups and over the earlier waves give every
// (wave, group) its first position; a second pass walks the wave's rows 64 at
// a time: the lanes that hold one id are found with one ballot per id bit,
// a row's rank is the number of such lanes below it, and the lowest of them
// advances the group's position.  Counts are integers and every position has
// one owner, so the result depends on the ids alone.
// Bound by latency: 32 rows 4.0 us in one launch; 262144 rows in 64 groups 3.4 us
// (count) and 9.7 us (place) for 2 MB moved by 64 workgroups: before it places
// its 256 rows a wave, place zeroes its counters, counts its rows again and sums
// the counts of all parts.
#include "device_common.hpp"
#include "experts.hpp"

namespace mlora {

namespace {

constexpr int kWaves = 16;                 // waves per workgroup (1024 threads)
constexpr int kMaxLds = 64 * 1024;         // bytes of LDS a launch takes

// Waves that place rows on their own: as many as their counters (and `extra`
// more rows of n_groups counters) fit into LDS.
__host__ __device__ __forceinline__ int place_waves(int n_groups, int extra) {
  int w = kWaves;
  while (w > 1 && 256 + (w + extra) * n_groups * 4 > kMaxLds) w >>= 1;
  return w;
}
__host__ __device__ __forceinline__ int lds_bytes(int n_groups, int extra) {
  return 256 + (place_waves(n_groups, extra) + extra) * n_groups * 4;
}

// Lanes of the wave whose `id` equals this lane's (id < 2^bits).
__device__ __forceinline__ uint64_t match_any(int id, bool on, int bits) {
  uint64_t m = __ballot(on);
  for (int b = 0; b < bits; ++b) {
    const uint64_t s = __ballot((id >> b) & 1);
    m &= ((id >> b) & 1) ? s : ~s;
  }
  return m;
}

// Exclusive sums of v over the workgroup's threads (1024), and the total.
__device__ __forceinline__ int block_exclusive(int v, int* wsum, int& total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int inc = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(inc, d);
    if (lane >= d) inc += u;
  }
  if (lane == 63) wsum[w] = inc;
  __syncthreads();
  int before = 0, all = 0;
  for (int j = 0; j < kWaves; ++j) {
    const int x = wsum[j];
    before += j < w ? x : 0;
    all += x;
  }
  __syncthreads();
  total = all;
  return before + inc - v;
}

// One workgroup's rows [r0, r1): per-wave counts cnt[cw][n_groups] in LDS.
__device__ __forceinline__ void count_rows(const int32_t* ids, int64_t r0, int64_t r1, int G, int cw, int64_t per,
                                           int* cnt) {
  for (int i = threadIdx.x; i < cw * G; i += 1024) cnt[i] = 0;
  __syncthreads();
  // every thread counts for the wave that will place the row
  for (int64_t i = r0 + threadIdx.x; i < r1; i += 1024) {
    const int id = ids[i];
    if ((unsigned)id < (unsigned)G) atomicAdd(&cnt[((int)(i - r0) / (int)per) * G + id], 1);
  }
  __syncthreads();
}

// Second pass: wave w < cw places rows [r0 + w per, r0 + (w + 1) per); base
// [cw][G] holds each wave's first position per group.
__device__ __forceinline__ void place_rows(const int32_t* ids, int64_t r0, int64_t r1, int G, int cw, int64_t per,
                                           int bits, int* base, int32_t* order) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  if (w >= cw) return;
  int* mine = base + w * G;
  const int64_t lo = r0 + w * per, hi = min(r1, lo + per);
  int next = lo + lane < hi ? ids[lo + lane] : -1;
  for (int64_t i = lo; i < hi; i += 64) {
    const int id = next;
    next = i + 64 + lane < hi ? ids[i + 64 + lane] : -1;     // in flight during this step
    const bool on = (unsigned)id < (unsigned)G;
    const uint64_t same = match_any(on ? id : 0, on, bits);
    const int rank = __popcll(same & (((uint64_t)1 << lane) - 1));
    if (on) order[mine[id] + rank] = (int32_t)(i + lane);
    // LDS reads above come before the leaders' writes: a wave runs in order
    __builtin_amdgcn_wave_barrier();
    if (on && rank == 0) mine[id] += __popcll(same);
    __builtin_amdgcn_wave_barrier();
  }
}

// Offsets from the groups' totals, and every wave's first positions in place
// of its counts.  tot(g): rows of group g in all workgroups; pre(g): those of
// earlier workgroups.
template <class TOT, class PRE>
__device__ __forceinline__ int bases(int G, int cw, int* cnt, int* wsum, int32_t* offsets, TOT tot, PRE pre) {
  int before = 0;
  for (int g0 = 0; g0 < G; g0 += 1024) {
    const int g = g0 + threadIdx.x;
    const int v = g < G ? tot(g) : 0;
    int all;
    const int ex = before + block_exclusive(v, wsum, all);
    if (g < G) {
      if (offsets) offsets[g] = ex;
      int p = ex + pre(g);
      for (int w = 0; w < cw; ++w) {
        const int c = cnt[w * G + g];
        cnt[w * G + g] = p;
        p += c;
      }
    }
    before += all;
  }
  if (offsets && threadIdx.x == 0) offsets[G] = before;
  __syncthreads();
  return before;
}

}  // namespace

// All rows by one workgroup: one launch, for the rows of a decode step.
__global__ __launch_bounds__(1024) void k_group_rows_one(const int32_t* ids, int64_t rows, int G, int bits,
                                                         int32_t* offsets, int32_t* order) {
  extern __shared__ int lds[];
  int* wsum = lds;
  int* cnt = lds + 64;
  const int cw = place_waves(G, 0);
  const int64_t per = max((int64_t)1, (rows + cw - 1) / cw);
  count_rows(ids, 0, rows, G, cw, per, cnt);
  auto tot = [&](int g) {
    int s = 0;
    for (int w = 0; w < cw; ++w) s += cnt[w * G + g];
    return s;
  };
  const int end = bases(G, cw, cnt, wsum, offsets, tot, [](int) { return 0; });
  place_rows(ids, 0, rows, G, cw, per, bits, cnt, order);
  for (int64_t i = end + threadIdx.x; i < rows; i += 1024) order[i] = -1;
}

// Part b's counts per group.
__global__ __launch_bounds__(1024) void k_group_count(const int32_t* ids, int64_t rows, int64_t part, int G,
                                                      int32_t* counts) {
  extern __shared__ int lds[];
  const int64_t r0 = blockIdx.x * part, r1 = min(rows, r0 + part);
  count_rows(ids, r0, r1, G, 1, part, lds);
  for (int g = threadIdx.x; g < G; g += 1024) counts[(int64_t)blockIdx.x * G + g] = lds[g];
}

// Part b's rows placed: every workgroup sums the parts' counts by itself.
__global__ __launch_bounds__(1024) void k_group_place(const int32_t* ids, int64_t rows, int64_t part, int G, int bits,
                                                      const int32_t* counts, int32_t* offsets, int32_t* order) {
  extern __shared__ int lds[];
  int* wsum = lds;
  int* tot = lds + 64;
  int* pre = tot + G;
  const int cw = place_waves(G, 2);
  int* cnt = pre + G;
  const int64_t r0 = blockIdx.x * part, r1 = min(rows, r0 + part);
  const int64_t per = max((int64_t)1, (part + cw - 1) / cw);
  for (int g = threadIdx.x; g < 2 * G; g += 1024) tot[g] = 0;
  count_rows(ids, r0, r1, G, cw, per, cnt);
  // threads share the (part, group) pairs; the sums are integers
  const int parts = gridDim.x;
  const int lanes = max(1, 1024 / G);                 // parts summed side by side per group
  for (int i = threadIdx.x; i < G * lanes; i += 1024) {
    const int g = i % G, l = i / G;
    int all = 0, before = 0;
    for (int p = l; p < parts; p += lanes) {
      const int c = counts[(int64_t)p * G + g];
      all += c;
      before += p < (int)blockIdx.x ? c : 0;
    }
    atomicAdd(&tot[g], all);
    atomicAdd(&pre[g], before);
  }
  __syncthreads();
  const int end = bases(G, cw, cnt, wsum, blockIdx.x == 0 ? offsets : nullptr, [&](int g) { return tot[g]; },
                        [&](int g) { return pre[g]; });
  place_rows(ids, r0, r1, G, cw, per, bits, cnt, order);
  // positions behind the last group, shared by the workgroups
  for (int64_t i = end + (int64_t)blockIdx.x * 1024 + threadIdx.x; i < rows; i += (int64_t)parts * 1024) order[i] = -1;
}

void launch_group_rows(const int32_t* ids, int64_t rows, int32_t n_groups, int32_t* offsets, int32_t* order,
                       int32_t* counts, hipStream_t s) {
  int bits = 0;
  while ((1 << bits) < n_groups) ++bits;
  if (rows <= kGroupOneLaunch) {
    hipLaunchKernelGGL(k_group_rows_one, dim3(1), dim3(1024), lds_bytes(n_groups, 0), s, ids, rows, n_groups, bits, offsets, order);
    return;
  }
  const int64_t part = group_part_rows(rows);
  const unsigned parts = (unsigned)((rows + part - 1) / part);
  hipLaunchKernelGGL(k_group_count, dim3(parts), dim3(1024), (size_t)n_groups * 4, s, ids, rows, part, n_groups,
                     counts);
  hipLaunchKernelGGL(k_group_place, dim3(parts), dim3(1024), lds_bytes(n_groups, 2), s, ids, rows, part, n_groups,
                     bits, counts, offsets, order);
}

}  // namespace mlora
