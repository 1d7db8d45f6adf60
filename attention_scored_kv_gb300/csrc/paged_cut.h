// How the paged attends' work is measured out: tiles of 128 cached tokens, in plain C++ so
// that the sizes can be checked on the host.
//
// A unit is what a CTA computes at a time for one KV head: for single tokens a request, for
// prompts a group of `per` query tokens of a request.  All KV heads' units are alike, so a
// request's cost is one sum, which passes 32 bits: 1.5 M tokens at 4 a unit are 2.2e9 tiles.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define KVS_HD __host__ __device__ __forceinline__
#else
#define KVS_HD inline
#endif

namespace kvs {
namespace cut {

constexpr int kTokens = 16, kTileBlocks = 8;   // of a block; blocks of a tile
constexpr int kSetup = 3;                      // what a prompt unit's start costs, in tiles

KVS_HD int at_least(int a, int b) { return a > b ? a : b; }

// The blocks that query tokens i0 .. i0 + cnt - 1 of a request see any of, the first of its tokens being at position p0.
struct Unit {
  int i0, cnt;           // first query token of the request, tokens
  int b0, nb, tiles;     // first block, blocks, tiles (one at least)
  KVS_HD int cost() const { return tiles + kSetup; }
};
KVS_HD Unit unit_of(int p0, int n, int window, int qg, int per) {
  Unit u;
  u.i0 = qg * per;
  u.cnt = n - u.i0 < per ? n - u.i0 : per;
  const int hi = at_least(p0 + u.i0 + u.cnt, 0);
  const int lo = window > 0 ? at_least(p0 + u.i0 + 1 - window, 0) : 0;
  u.b0 = lo / kTokens;
  u.nb = at_least((hi + kTokens - 1) / kTokens - u.b0, 0);
  u.tiles = at_least((u.nb + kTileBlocks - 1) / kTileBlocks, 1);
  return u;
}

// Cost of a request's units lane, lane + lanes, ...
KVS_HD long long lane_cost(int p0, int n, int window, int per, int lane, int lanes) {
  long long sum = 0;
  for (int qg = lane; qg * (long long)per < n; qg += lanes) sum += unit_of(p0, n, window, qg, per).cost();
  return sum;
}

// The largest share that a CTA can have of a call: a CTA counts its own in 32 bits.
inline bool share_fits(long long units, int table_stride, int hkv, int ctas) {
  const long long most = table_stride / kTileBlocks + 2 + kSetup;
  return (double)units * most * hkv / ctas < 2147483647.0;
}

}  // namespace cut
}  // namespace kvs
