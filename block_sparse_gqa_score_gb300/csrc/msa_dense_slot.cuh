// msa_dense_slot.cuh -- dense decode's assignment of a batch's (request, tile of
// kTile tokens, KV head) units to CTAs, by their visible blocks.
#pragma once

#include "msa_device.cuh"
#include "msa_launch.h"

namespace msa {

// dense decode with fewer (request, tile, KV head) units than CTAs and split
// parts: the CTAs are shared out in the kernel among up to this many
// (request, tile) units in proportion to their blocks
constexpr int kBalancedTiles = 256;

// Blocks a dense-decode unit (request, tile) attends: up to its last token's
// current block (0 for a padding request or a tile of padding rows).
template <int kTile>
__device__ __forceinline__ int dense_tile_blocks(const AttendParams& p, int tu, int ntiles) {
  const int b = tu / ntiles, tile = tu - b * ntiles;
  const int L = p.seq_lens[b];
  const bool seq_ok = L >= 0 && (L == 0 || (L - 1) / kPage < p.S);
  const int tok = min(kTile * tile + kTile - 1, p.Q - 1);
  const int pos = seq_ok ? L - p.Q + tok : -1;
  return pos >= 0 ? pos / kPage + 1 : 0;
}

struct DenseSlot {
  int unit;    // (request, tile, KV head) unit, in blockIdx.x order of the plain grid; -1: none
  int part;    // which of its equal block ranges
  int nparts;  // how many ranges the unit is cut into
};

// Dense decode's work for CTA (or cluster of CTAs) c of C along x.  With a
// grid of one CTA per unit and split that is (c, blockIdx.y, gridDim.y).  With
// more CTAs than units (one per SM or more) the units share them out by their
// blocks: unit u (n_u blocks) takes z_u = min(ceil(n_u / T), splits) CTAs (at
// least one) for the smallest T at which every unit's CTAs fit the grid, so that
// no CTA holds much more than its share of the batch's pages; the CTAs go to the
// units in order, a unit's KV heads in turn, each head's ranges in turn.  Every
// CTA computes the same assignment from seq_lens (one warp, every lane the same
// result); CTAs past the last unit's get none.
template <int kTile>
__device__ DenseSlot dense_slot(const AttendParams& p, int ntiles, int C, int c, int lane) {
  const int NT = p.B * ntiles, H = p.Hkv, Z = p.splits;
  if (C <= NT * H)
    return DenseSlot{c, static_cast<int>(blockIdx.y), static_cast<int>(gridDim.y)};
  // Lane l holds (request, tile) unit l; the units past the 32nd, if any, are read
  // again where they are needed.  Loops, not unrolled: this code runs once, and its
  // instructions cost more to fetch than to execute.
  const int n0 = lane < NT ? dense_tile_blocks<kTile>(p, lane, ntiles) : 0;
  auto blocks = [&](int k) {
    return k == 0 ? n0 : k + lane < NT ? dense_tile_blocks<kTile>(p, k + lane, ntiles) : 0;
  };
  int total = 0;
#pragma unroll 1
  for (int k = 0; k < NT; k += 32)
    total += static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(blocks(k))));
  // ceil(n / T) as floor((n + T - 1/2) / T): the quotient is at least 1 / (2 T) off an
  // integer and the float product at most (n + T) / T * 2^-22 off the quotient
  // (n + T < 2^20)
  auto parts = [&](int k, float rT, float Th) {
    return k + lane < NT ? min(max(__float2int_rz((static_cast<float>(blocks(k)) + Th) * rT), 1), Z)
                         : 0;
  };
  // the smallest T with sum z_u <= C / H: T = total / (C / H - NT) has it, since z_u is
  // at most n / T + 1 (and so has T = total, one CTA a unit)
  const int per = C / H;
  int lo = 1, hi = (total + per - NT) / max(per - NT, 1) + 1;
#pragma unroll 1
  while (lo < hi) {
    const int T = (lo + hi) >> 1;
    const float rT = 1.f / static_cast<float>(T), Th = static_cast<float>(T) - 0.5f;
    int sum = 0;
#pragma unroll 1
    for (int k = 0; k < NT; k += 32)
      sum += static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(parts(k, rT, Th))));
    if (sum <= per) hi = T;
    else lo = T + 1;
  }
  const float rT = 1.f / static_cast<float>(lo), Th = static_cast<float>(lo) - 0.5f;
  int run = 0;   // CTAs of the units before this group of 32
#pragma unroll 1
  for (int k = 0; k < NT; k += 32) {
    const int zc = parts(k, rT, Th);
    int incl = zc * H;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += t;
    }
    const int start = run + incl - zc * H;
    const unsigned hit = __ballot_sync(0xffffffffu, zc > 0 && c >= start && c < start + zc * H);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const int st = __shfl_sync(0xffffffffu, start, src);
      const int z = __shfl_sync(0xffffffffu, zc, src);
      const int rel = c - st;
      return DenseSlot{(k + src) * H + rel / z, rel % z, z};
    }
    run += __shfl_sync(0xffffffffu, incl, 31);
  }
  return DenseSlot{-1, 0, 1};
}

}  // namespace msa
