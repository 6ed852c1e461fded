// Device pieces shared by the grouped expert products: which rows a tile
// owns, where a grouped row lies, the order of the tiles, and E2M1 decoding.
#pragma once

#include "device_common.hpp"
#include "experts.hpp"

namespace mlora {

// n / d for 0 <= n < 2^31 (div_by).
__device__ __forceinline__ uint32_t div_fast(uint32_t n, const DivBy& d) {
  return d.mul ? __umulhi(n, d.mul) >> d.shift : n;
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

// A workgroup's tile in the rows form: rows [row0, row0 + mrows) of expert e,
// column tile tn.  mrows = 0: nothing to do.
struct RowTile {
  int e, row0, mrows, tn;
};

// The tile of workgroup blockIdx.x among the row tiles of BM rows that the
// groups' sizes give (known on the device only; the grid covers their upper
// bound).  Lane l sums the tiles of group 64 c + l in chunk c, so a router of
// up to 64 experts costs one pair of loads and one wave scan.  Workgroup b
// runs on XCD b mod 8; each XCD takes a contiguous run of the actual tiles,
// and tiles go down GM row tiles before moving along N, so tiles that run
// together share rows and columns in the XCD's L2.
template <int BM, int GM>
__device__ __forceinline__ RowTile row_tile(const ExpertArgs& a, int nN) {
  const int lane = threadIdx.x & 63;
  const int E = a.offsets ? a.n_experts : 1;
  auto tiles_of = [&](int e, int& lo, int& hi) {
    lo = hi = 0;
    if (e < E) group_rows(a, e, lo, hi);
    return (hi - lo + BM - 1) / BM;
  };
  auto scan = [&](int v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int u = __shfl_up(v, d);
      if (lane >= d) v += u;
    }
    return v;
  };
  int lo, hi;
  int cnt = tiles_of(lane, lo, hi);        // chunk 0's; the search below starts with it
  int inc = scan(cnt);
  int TM = __builtin_amdgcn_readlane(inc, 63);
  for (int c = 64; c < E; c += 64) {
    int lo2, hi2;
    TM += __builtin_amdgcn_readlane(scan(tiles_of(c + lane, lo2, hi2)), 63);
  }
  const int T = TM * nN, b = blockIdx.x;
  const int xcd = b & 7, q = b >> 3, per = T >> 3, rem = T & 7;
  if (q >= per + (xcd < rem ? 1 : 0)) return RowTile{0, 0, 0, 0};
  const int L = xcd * per + min(xcd, rem) + q;
  const int grp = L / (GM * nN), fm = grp * GM, gm = min(GM, TM - fm);
  const int within = L - fm * nN;
  const int tm = fm + within % gm;
  RowTile t;
  t.tn = within / gm;
  t.e = t.row0 = t.mrows = 0;
  // the group whose tiles hold tm
  for (int c = 0, before = 0; c < E; c += 64) {
    if (c > 0) {
      cnt = tiles_of(c + lane, lo, hi);
      inc = scan(cnt);
    }
    const uint64_t past = __ballot(before + inc > tm);
    if (past != 0) {
      const int l = __builtin_ctzll(past);
      const int first = before + __builtin_amdgcn_readlane(inc - cnt, l);
      t.e = c + l;
      t.row0 = __builtin_amdgcn_readlane(lo, l) + (tm - first) * BM;
      t.mrows = min(BM, __builtin_amdgcn_readlane(hi, l) - t.row0);
      break;
    }
    before += __builtin_amdgcn_readlane(inc, 63);
  }
  t.e = __builtin_amdgcn_readfirstlane(t.e);
  t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
  t.mrows = __builtin_amdgcn_readfirstlane(t.mrows);
  t.tn = __builtin_amdgcn_readfirstlane(t.tn);
  return t;
}

// Eight E2M1 codes (one word) times 2^(x - 127) -> eight bf16, exact.
__device__ __forceinline__ u32x4 bf16_of_e2m1(uint32_t w, float scale) {
  u32x4 o;
  o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
  o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
  o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
  o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  return o;
}

// Largest number of row tiles that `rows` rows in at most `experts` groups
// can make.
inline int64_t max_row_tiles(int64_t rows, int64_t experts, int bm) {
  return rows / bm + (experts < rows ? experts : rows);
}

}  // namespace mlora
