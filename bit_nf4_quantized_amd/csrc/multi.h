// Rows grouped by adapter: what the route kernel leaves for the kernels of the
// multi-adapter linear (multi.hip, dense_gemm.hip).
#pragma once

#include "common.h"

namespace qlora {

// perm [M]: the rows in a stable order by adapter, rows without one (id
// outside [0, A)) last. Segment k < count[0] is the k-th adapter that has
// rows: adapter[k], rows perm[start[k] .. start[k+1]); start[count[0]] is the
// number of rows with an adapter.
struct RouteView {
  const int32_t* perm;
  const int32_t* start;
  const int32_t* adapter;
  const int32_t* count;
};

// Pieces of at most `len` rows, none across segments. Piece s of segment k has
// the number start[k] / len + k + s: numbers of different segments never
// meet, since a segment has at most end / len - start / len + 1 pieces, and
// all are below M / len + segments, which a launch can use as its grid before
// the segments are known. Called by whole waves; empty numbers give hi <= lo.
struct RoutePiece {
  int k, lo, hi;
};

__device__ __forceinline__ RoutePiece route_piece(const RouteView& r, int t, int len) {
  const int lane = threadIdx.x & 63;
  const int n = r.count[0];
  int below = 0;
  for (int base = 0; base < n; base += 64) {
    const int k = base + lane;
    below += __popcll(__ballot(k < n && r.start[k < n ? k : 0] / len + k <= t));
  }
  below = __builtin_amdgcn_readfirstlane(below);
  if (below == 0) return RoutePiece{0, 0, 0};
  const int k = below - 1;
  const int s0 = r.start[k], s1 = r.start[k + 1];
  const int lo = s0 + (t - (s0 / len + k)) * len;
  return RoutePiece{k, lo, lo + len < s1 ? lo + len : s1};
}

// Segments that meet sorted rows [m0, m1): [lo, hi). Called by whole waves.
struct RouteRange {
  int lo, hi;
};

__device__ __forceinline__ RouteRange route_range(const RouteView& r, int m0, int m1) {
  const int lane = threadIdx.x & 63;
  const int n = r.count[0];
  int before = 0, begun = 0;
  for (int base = 0; base < n; base += 64) {
    const int k = base + lane;
    const bool in = k < n;
    before += __popcll(__ballot(in && r.start[in ? k + 1 : 0] <= m0));
    begun += __popcll(__ballot(in && r.start[in ? k : 0] < m1));
  }
  return RouteRange{__builtin_amdgcn_readfirstlane(before), __builtin_amdgcn_readfirstlane(begun)};
}

// A product cut into S reduction slices: C = bf16(part[0] + part[1] + ...).
struct SplitSum {
  const float* part;   // [S][values]
  uint16_t* C;
  int64_t values;      // a multiple of 8
  int S;
};

// Its values 8 i .. 8 i + 8.
__device__ __forceinline__ void split_sum_body(const SplitSum& s, int64_t i) {
  i *= 8;
  if (i >= s.values) return;
  f32x4_t a = {0.0f, 0.0f, 0.0f, 0.0f}, b = a;
  int z = 0;
  for (; z + 2 <= s.S; z += 2) {
    const float* q = s.part + (int64_t)z * s.values + i;
    const f32x4_t a0 = *reinterpret_cast<const f32x4_t*>(q), b0 = *reinterpret_cast<const f32x4_t*>(q + 4);
    const f32x4_t a1 = *reinterpret_cast<const f32x4_t*>(q + s.values), b1 = *reinterpret_cast<const f32x4_t*>(q + s.values + 4);
    a += a0; b += b0;
    a += a1; b += b1;
  }
  if (z < s.S) {
    a += *reinterpret_cast<const f32x4_t*>(s.part + (int64_t)z * s.values + i);
    b += *reinterpret_cast<const f32x4_t*>(s.part + (int64_t)z * s.values + i + 4);
  }
  *reinterpret_cast<u32x4_t*>(s.C + i) =
      u32x4_t{pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y), pack_bf16x2(b.z, b.w)};
}

}  // namespace qlora
