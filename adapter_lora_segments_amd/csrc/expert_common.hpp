// Device pieces shared by the grouped expert products: which rows a tile
// owns, where a grouped row lies, the order of the tiles, and E2M1 decoding.
#pragma once

#include "device_common.hpp"
#include "experts.hpp"

namespace mlora {

// The kernel's ExpertArgs (its only parameter) read from the kernel argument
// segment where they are used.  Kept in scalar registers across a loop over
// tiles they would push the loop's own scalars out; the empty asm hides that
// two calls give the same pointer.
__device__ __forceinline__ const ExpertArgs& kernel_args() {
  auto p = (const __attribute__((address_space(4))) ExpertArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const ExpertArgs*)p;
}

// n / d for 0 <= n < 2^31 (div_by; mul is 0 for d = 1).
__device__ __forceinline__ uint32_t div_fast(uint32_t n, const DivBy& d) {
  return (__umulhi(n, d.mul) >> d.shift) + (d.mul ? 0u : n);
}

// Order entry `v` as a row to read: an entry that names no row reads row 0.
__device__ __forceinline__ uint32_t read_row(int v, int rows) { return (unsigned)v < (unsigned)rows ? (uint32_t)v : 0u; }

// Source row of grouped row s.
__device__ __forceinline__ int64_t source_row(const ExpertArgs& a, const RowMap& m, int s) {
  return m.by_order ? (int64_t)div_fast(read_row(a.order[s], a.rows), m.div) : (int64_t)s;
}

// Group e's rows [lo, hi), clamped to the buffers.
__device__ __forceinline__ void group_rows(const ExpertArgs& a, int e, int& lo, int& hi) {
  if (!a.offsets) {
    lo = 0;
    hi = a.rows;
    return;
  }
  lo = min(max(a.offsets[e], 0), a.rows);
  hi = max(lo, min(a.offsets[e + 1], a.rows));
}

// A tile in the rows form: rows [row0, row0 + mrows) of expert e,
// column tile tn.  mrows = 0: nothing to do.
struct RowTile {
  int e, row0, mrows, tn;
};

// The row tiles of BM rows that the groups' sizes give (known on the device
// only; a grid covers their upper bound).  Lane l sums the tiles of group
// 64 c + l in chunk c, so a router of up to 64 experts costs one pair of loads
// and one wave scan.  Tile b belongs to XCD b mod 8 (a workgroup's, and
// b + gridDim.x's when the grid is a multiple of 8); each XCD takes a
// contiguous run of the actual tiles, and tiles go down GM row tiles before
// moving along N, so tiles that run together share rows and columns in the
// XCD's L2.
template <int BM, int GM>
struct RowTiles {
  int E, nN, TM;
  int lo, hi, cnt, inc;   // this lane's group of chunk 0: rows, tiles, tiles up to and with it

  __device__ __forceinline__ void group(const ExpertArgs& a, int c, int& l, int& h, int& n, int& sum) const {
    const int lane = threadIdx.x & 63;
    l = h = 0;
    if (c + lane < E) group_rows(a, c + lane, l, h);
    n = pieces_of(h - l, BM);
    sum = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int u = __shfl_up(sum, d);
      if (lane >= d) sum += u;
    }
  }
  __device__ __forceinline__ RowTiles(const ExpertArgs& a, int n_tiles) : nN(n_tiles) {
    E = a.offsets ? a.n_experts : 1;
    group(a, 0, lo, hi, cnt, inc);
    TM = __builtin_amdgcn_readlane(inc, 63);
    for (int c = 64; c < E; c += 64) {
      int l2, h2, c2, i2;
      group(a, c, l2, h2, c2, i2);
      TM += __builtin_amdgcn_readlane(i2, 63);
    }
  }
  // Tile b; mrows = 0 past the last one.
  __device__ __forceinline__ RowTile at(const ExpertArgs& a, int b) const {
    const int T = TM * nN, xcd = b & 7, q = b >> 3, per = T >> 3, rem = T & 7;
    RowTile t{0, 0, 0, 0};
    if (q >= per + (xcd < rem ? 1 : 0)) return t;
    const int L = xcd * per + min(xcd, rem) + q;
    const int fm = L / (GM * nN) * GM, gm = min(GM, TM - fm);
    const int within = L - fm * nN;
    const int tm = fm + within % gm;
    t.tn = within / gm;
    // the group whose tiles hold tm
    int l1 = lo, h1 = hi, n1 = cnt, i1 = inc;
    for (int c = 0, before = 0; c < E; c += 64) {
      if (c > 0) group(a, c, l1, h1, n1, i1);
      const uint64_t past = __ballot(before + i1 > tm);
      if (past != 0) {
        const int l = __builtin_ctzll(past);
        const int first = before + __builtin_amdgcn_readlane(i1 - n1, l);
        t.e = c + l;
        t.row0 = __builtin_amdgcn_readlane(l1, l) + (tm - first) * BM;
        t.mrows = min(BM, __builtin_amdgcn_readlane(h1, l) - t.row0);
        break;
      }
      before += __builtin_amdgcn_readlane(i1, 63);
    }
    t.e = __builtin_amdgcn_readfirstlane(t.e);
    t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
    t.mrows = __builtin_amdgcn_readfirstlane(t.mrows);
    t.tn = __builtin_amdgcn_readfirstlane(t.tn);
    return t;
  }
};

// The chunks of C rows that the groups' rows are cut into (one at least, so a
// group without rows gets its zeros), and where a chunk's sums go: straight to
// the group's dW when it has one chunk, else to a slot of its own.
struct DwChunk {
  int e, row0, rows, slot;  // slot -1: the only chunk; rows < 0: past the last chunk
};
struct DwChunks {
  int E, C, total, room;  // room: slots there are, for offsets that are not ordered

  __device__ __forceinline__ void group(const ExpertArgs& a, int c, int& lo, int& hi, int& n, int& sum, int& slots) const {
    const int lane = threadIdx.x & 63;
    lo = hi = n = 0;
    if (c + lane < E) {
      group_rows(a, c + lane, lo, hi);
      n = max(1, pieces_of(hi - lo, C));
    }
    sum = n;
    slots = n > 1 ? n : 0;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int u = __shfl_up(sum, d), v = __shfl_up(slots, d);
      if (lane >= d) {
        sum += u;
        slots += v;
      }
    }
  }
  __device__ __forceinline__ explicit DwChunks(const ExpertArgs& a) {
    E = a.offsets ? a.n_experts : 1;
    C = a.chunk;
    total = 0;
    room = (int)(2 * (int64_t)a.rows / C);
    for (int c = 0; c < E; c += 64) {
      int lo, hi, n, sum, slots;
      group(a, c, lo, hi, n, sum, slots);
      total += __builtin_amdgcn_readlane(sum, 63);
    }
  }
  __device__ __forceinline__ DwChunk at(const ExpertArgs& a, int i) const {
    DwChunk r{0, 0, -1, -1};
    if (i >= total) return r;
    for (int c = 0, before = 0, used = 0; c < E; c += 64) {
      int lo, hi, n, sum, slots;
      group(a, c, lo, hi, n, sum, slots);
      const uint64_t past = __ballot(before + sum > i);
      if (past != 0) {
        const int l = __builtin_ctzll(past);
        const int k = i - before - __builtin_amdgcn_readlane(sum - n, l);    // chunk of the group
        const int many = __builtin_amdgcn_readlane(n, l);
        r.e = c + l;
        r.row0 = __builtin_amdgcn_readlane(lo, l) + k * C;
        r.rows = min(C, __builtin_amdgcn_readlane(hi, l) - r.row0);
        r.slot = many > 1 ? used + __builtin_amdgcn_readlane(slots, l) - many + k : -1;
        if (r.slot >= room) r.rows = -1;
        break;
      }
      before += __builtin_amdgcn_readlane(sum, 63);
      used += __builtin_amdgcn_readlane(slots, 63);
    }
    return r;
  }
  // Chunks of group e and the first one's slot (if it has several).
  __device__ __forceinline__ void of_group(const ExpertArgs& a, int e, int& many, int& first) const {
    many = first = 0;
    for (int c = 0, used = 0; c < E; c += 64) {
      int lo, hi, n, sum, slots;
      group(a, c, lo, hi, n, sum, slots);
      if (e < c + 64) {
        many = __builtin_amdgcn_readlane(n, e - c);
        first = used + __builtin_amdgcn_readlane(slots, e - c) - many;
        if (first + many > room) many = 0;
        break;
      }
      used += __builtin_amdgcn_readlane(slots, 63);
    }
  }
};

// Eight E2M1 codes (one word) times 2^(x - 127) -> eight bf16, exact.
__device__ __forceinline__ u32x4 bf16_of_e2m1(uint32_t w, float scale) {
  u32x4 o;
  o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
  o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
  o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
  o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  return o;
}

}  // namespace mlora
