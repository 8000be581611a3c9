// msa_score_prefill.cu -- the block scorer of prefill batches: for every (KV head, query
// token, block) the largest visible scaled q.k over the head group and the block's keys.
//
// Operation (msa_score_prefill in include/msa.h): scores[g, i, n] = max over the 16 heads
// of g and the keys t <= pos(i) of block n of sm_scale * k_scale * ks[page] * q.K_t;
// -inf where the token sees no key of the block.
//
// What bounds it: the tensor cores, 2 * 128 * 16 products a key, token and KV head
// against a key's 128 bytes shared by the chunk's tokens, and the shared memory that feeds
// them.  The product is S = Q K^T with the query rows (16 tokens x 16 heads, two M = 128
// halves) as A and two pages of keys as B, so that a thread's tensor-memory lane is one
// query row: the largest of a page's 128 columns is 64 three-input maxima without an
// exchange, and a token's 16 heads are 16 lanes.  (Two pages, N = 256: A is read once for
// both, 12 KiB of operands in 128 cycles; with a page at a time, 8 KiB in 64 cycles, shared
// memory was the limit and there were twice the products to issue: 340 us where two take 251.)
// A bf16 query is two exact e4m3 parts (two products a half, which cost what
// one bf16 product would, and the keys need no conversion), an fp8 query is one.  Each half
// has its 256 columns of tensor memory: while one is searched the other is multiplied.  One
// CTA an SM, each an equal share of all pages (msa_prefill.cuh); the next unit's query tile
// is prepared while the current one is worked on.
// Measured: four chunks of up to 1k tokens over 4k .. 16k, 64/4 heads, page scales 252 us,
// 1950 TFLOP/s (the tensor core is active in 87 % of the cycles); with an fp8 query on a K-only
// cache 196 us (its products need 128: each half's search, four loads from tensor memory in turn,
// is no longer hidden behind them); four chunks of some 200 tokens over 2k .. 8k on it 35.6 us (16),
// with a bf16 query 49.5 (32); eight prompts of 1024 tokens 114 us (36: units of 4.5 pages pay
// for their query tiles); three chunks of some 40 tokens on one KV head 13.7 us, of which 2 are
// products.  With the query tiles' split in line (118 KiB of code, the warps waited for
// instructions) the four chunks took 277 us.
//   warp 0       page look-ups, TMA of K tiles
//   warp 1       products (owns tensor memory)
//   warps 2, 3   segments and query tiles, a token each in turn (behind a short unit: warps
//                4..19, a token each)
//   warps 4..19  maxima and scores, four warps a half and page
#include <cstddef>

#include "msa_device.cuh"
#include "msa_launch.h"
#include "msa_prefill.cuh"
#include "msa_tcgen05.cuh"

namespace msa {

namespace {

using namespace prefill;

constexpr int kThreads = 640;
constexpr int kPairs = 3;                       // pairs of K tiles in flight
constexpr int kInfo = 8;                        // pairs' factors in flight
constexpr int kExtra = 4;                       // a unit's query tile, in pages
constexpr int kMinSteps = 1;
constexpr int kShort = 10;                      // pages of a unit too few to hide the next one's query tile
constexpr int kQTile = 4 * kHalfTile;           // two halves, hi and lo parts
constexpr int kOffK = 2 * kQTile;
constexpr int kOffTail = kOffK + kPairs * 2 * kHalfTile;
constexpr int kTmemCols = 512;                  // [half] of 256 columns, a page 128

struct Tail {
  uint64_t k_full[kPairs], k_empty[kPairs];
  uint64_t s_full[2], s_empty[2];               // by half
  uint64_t info_full[kInfo];
  uint64_t seg_full[2], seg_empty[2];
  uint64_t q_full[2];
  uint64_t q_part;                              // warps 4..19 <-> 2, 3: their tokens of a tile
  uint64_t finish;
  uint32_t tmem_base;
  float info[kInfo][2];                         // ks, or 0: no key of the page counts
  Segment seg[2];
  float zs[2][kTile];
  WalkScratch scratch;
};

constexpr int kSmemBytes = kOffTail + static_cast<int>(sizeof(Tail)) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

// Token x of a segment's query tile.  Not in line: its registers are not the search's.
__device__ __noinline__ void load_token(const PrefillParams& p, const Segment* sg, int x, uint8_t* tile,
                                        float* zs) {
  (void)load_query_tile<1, 4>(p, *sg, x, kTile, tile, zs, threadIdx.x & 31, [] { return true; });
}

__global__ void __launch_bounds__(kThreads, 1)
    score_prefill_kernel(const __grid_constant__ CUtensorMap kv_map,
                         const __grid_constant__ PrefillParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Tail* tail = reinterpret_cast<Tail*>(smem + kOffTail);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int parts = p.q8 ? 1 : 2;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < kPairs; ++s) {
      mbar_init(&tail->k_full[s], 1);
      mbar_init(&tail->k_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&tail->s_full[s], 1);
      mbar_init(&tail->s_empty[s], 8);
      mbar_init(&tail->seg_full[s], 1);
      mbar_init(&tail->seg_empty[s], 1 + 1 + 1 + 16);   // warps 0, 1, 3 and 4..19
      mbar_init(&tail->q_full[s], 2);
    }
    for (int s = 0; s < kInfo; ++s) mbar_init(&tail->info_full[s], 1);
    mbar_init(&tail->q_part, 16);
    mbar_init(&tail->finish, 1 + 1 + 2 + 16);
    fence_barrier_init();
    prefetch_tensormap(&kv_map);
  } else if (warp == 1) {
    tc::tmem_alloc(&tail->tmem_base, kTmemCols);
    tc::tmem_relinquish();
  }
  pdl_wait();   // lengths, tables and queries may be an earlier kernel's
  const bool bad = plan_walk<kThreads>(p, kExtra, kMinSteps, &tail->scratch);
  if (threadIdx.x == 0) {
    bool cut;
    int n;
    tail->seg[0] = next_segment(p, tail->scratch.walk, kExtra, cut, n);
  }
  tc::fence_before_thread_sync();
  __syncthreads();
  tc::fence_after_thread_sync();
  const uint32_t tmem = tail->tmem_base;
  fill_uncovered(p, bad, [&](int i) {
    for (int g = 0; g < p.Hkv; ++g)
      for (int n = threadIdx.x; n < p.S; n += kThreads)
        p.scores[(static_cast<int64_t>(g) * p.T + i) * p.S + n] = -INFINITY;
  });
  bool ok = true;

  if (warp == 0) {
    // ---- K tiles -----------------------------------------------------------------------------
    int t = 0, s = 0;    // pairs so far; the next one's place
    unsigned par = 0;    // its phase
    for (int i = 0; ok; ++i) {
      ok = __all_sync(0xffffffffu, wait_for(&tail->seg_full[i & 1], (i >> 1) & 1));
      if (!ok) break;
      const Segment sg = tail->seg[i & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&tail->seg_empty[i & 1]);
      if (sg.ntok == 0) break;
      const int32_t* trow = p.block_table + static_cast<int64_t>(sg.b) * p.S;
      for (int n0 = sg.n0; n0 < sg.n1 && ok; n0 += 32) {
        // 32 pages' entries and scales at once, a lane each
        const int n = n0 + lane;
        int page = 0;
        float ks = 0.f;
        if (n < sg.n1) {
          page = trow[n];
          ks = 1.f;
          if (page < 0 || static_cast<int64_t>(page) >= p.num_blocks) {
            flag_error(p.err, MSA_ERR_PAGE_RANGE);
            page = 0;
            ks = 0.f;
          } else if (p.kv_scales) {
            ks = p.kv_scales[(static_cast<int64_t>(page) * p.Hkv + sg.g) * p.scale_sides];
            if (!page_scale_ok(ks)) {
              flag_error(p.err, MSA_ERR_SCALE);
              ks = 0.f;
            }
          }
        }
        const int have = min(32, sg.n1 - n0);
        for (int x = 0; x < have; x += 2, ++t) {
          ok = t < kPairs || wait_for(&tail->k_empty[s], par ^ 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const int y = lane - x;              // this lane's page of the pair
          if ((y == 0 || y == 1) && lane < have) tail->info[t % kInfo][y] = ks;
          __syncwarp();
          if (y == 0) {
            mbar_arrive(&tail->info_full[t % kInfo]);
            mbar_arrive_expect_tx(&tail->k_full[s], x + 1 < have ? 2 * kHalfTile : kHalfTile);
          }
          __syncwarp();
          if ((y == 0 || y == 1) && lane < have)
            tma_load_2d(smem + kOffK + (2 * s + y) * kHalfTile, &kv_map, 0, (page * p.Hkv + sg.g) * kPage,
                        &tail->k_full[s]);
          __syncwarp();
          if (++s == kPairs) {
            s = 0;
            par ^= 1;
          }
        }
      }
    }
    if (lane == 0) {
      if (!ok) flag_error(p.err, MSA_ERR_TIMEOUT);
      for (int x = max(0, t - kPairs); x < t; ++x)
        (void)wait_for(&tail->k_full[x % kPairs], (x / kPairs) & 1);
      pdl_trigger();
      mbar_arrive(&tail->finish);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---- S = Q K^T ---------------------------------------------------------------------------
    const uint64_t q0 = tc::sw128_kmajor_desc(smem_u32(smem));
    const uint64_t k0 = tc::sw128_kmajor_desc(smem_u32(smem + kOffK));
    const bool leader = tc::elect_one();
    // (the vote makes it the same for the compiler as well)
    auto wait = [&](uint64_t* bar, unsigned parity) {
      return __all_sync(0xffffffffu, wait_for(bar, parity)) != 0;
    };
    int s = 0;                 // place of the next pair
    unsigned k_par = 0;
    int n_0 = 0, n_1 = 0;      // pairs multiplied, by half
    auto scores = [&](int h, int qbuf, int& n, uint32_t idesc) {
      if (n >= 1 && !wait(&tail->s_empty[h], (n - 1) & 1)) return false;
      tc::fence_after_thread_sync();
      if (leader) {
        const uint64_t bk = k0 + static_cast<uint64_t>(s) * (2 * kHalfTile >> 4);
        const uint64_t aq = q0 + static_cast<uint64_t>(qbuf) * (kQTile >> 4) +
                            static_cast<uint64_t>(h) * (2 * kHalfTile >> 4);
        const uint32_t d = tmem + 256 * h;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) tc::mma_e4m3(d, aq + 2 * ks, bk + 2 * ks, idesc, ks > 0);
        if (parts == 2) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            tc::mma_e4m3(d, aq + (kHalfTile >> 4) + 2 * ks, bk + 2 * ks, idesc, 1);
        }
        tc::commit(&tail->s_full[h]);
      }
      __syncwarp();
      ++n;
      return true;
    };
    for (int i = 0; ok; ++i) {
      ok = wait(&tail->seg_full[i & 1], (i >> 1) & 1);
      if (!ok) break;
      const int ntok = __reduce_max_sync(0xffffffffu, tail->seg[i & 1].ntok);
      const int pages = __reduce_max_sync(0xffffffffu, tail->seg[i & 1].n1 - tail->seg[i & 1].n0);
      if (ntok == 0) break;
      ok = wait(&tail->q_full[i & 1], (i >> 1) & 1);
      // Behind a unit of two halves, the pages of a unit of one: nothing else holds them back
      // until the other half's warps have read their last pair and its factors, whose places
      // (and phases) come round.
      if (ok && ntok <= kHalfTokens && n_1 > 0) ok = wait(&tail->s_empty[1], (n_1 - 1) & 1);
      for (int x = 0; x < pages && ok; x += 2) {
        const uint32_t idesc = x + 1 < pages ? tc::idesc_e4m3_f32(128, 2 * kPage) : tc::idesc_e4m3_f32(128, kPage);
        ok = wait(&tail->k_full[s], k_par);
        if (!ok) break;
        ok = scores(0, i & 1, n_0, idesc);
        if (ok && ntok > kHalfTokens) ok = scores(1, i & 1, n_1, idesc);
        if (leader) tc::commit(&tail->k_empty[s]);
        __syncwarp();
        if (++s == kPairs) {
          s = 0;
          k_par ^= 1;
        }
      }
      if (leader) tc::commit(&tail->seg_empty[i & 1]);      // the query tile has been read
      __syncwarp();
    }
    if (leader) {
      if (!ok) flag_error(p.err, MSA_ERR_TIMEOUT);
      tc::commit(&tail->finish);
    }
    __syncwarp();
    (void)mbar_wait(&tail->finish, 0);
    tc::fence_after_thread_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  } else if (warp < 4) {
    // ---- segments and query tiles ------------------------------------------------------------
    const int h = warp - 2;
    int last_pages = 0, parted = 0;   // pages of the segment before; tiles of warps 4..19
    for (int i = 0;; ++i) {
      ok = __all_sync(0xffffffffu, i < 2 || wait_for(&tail->seg_empty[i & 1], ((i >> 1) - 1) & 1));
      if (!ok) break;
      if (h == 0) {
        if (lane == 0) {
          bool cut;
          int n;
          if (i > 0) tail->seg[i & 1] = next_segment(p, tail->scratch.walk, kExtra, cut, n);
          mbar_arrive(&tail->seg_full[i & 1]);
        }
        __syncwarp();
      } else {
        ok = __all_sync(0xffffffffu, wait_for(&tail->seg_full[i & 1], (i >> 1) & 1));
        if (!ok) break;
      }
      const Segment sg = tail->seg[i & 1];
      if (sg.ntok > 0 && last_pages < kShort) {
        // the tile is prepared by warps 4..19
        ok = __all_sync(0xffffffffu, wait_for(&tail->q_part, parted & 1));
        if (!ok) break;
        ++parted;
      } else if (sg.ntok > 0)
        (void)load_query_tile<kTile / 2, 4>(p, sg, h, 2, smem + (i & 1) * kQTile, tail->zs[i & 1], lane,
                                         [] { return true; });
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&tail->q_full[i & 1]);
        if (h == 1) mbar_arrive(&tail->seg_empty[i & 1]);
      }
      if (sg.ntok == 0) break;
      last_pages = sg.n1 - sg.n0;
    }
    if (lane == 0) {
      if (!ok) flag_error(p.err, MSA_ERR_TIMEOUT);
      mbar_arrive(&tail->finish);
    }
    __syncwarp();
  } else {
    // ---- maxima of half h, page pg of each pair ----------------------------------------------
    const int h = (warp - 4) >> 3, pg = ((warp - 4) >> 2) & 1, quarter = warp & 3;
    const uint32_t at = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + 256 * h + 128 * pg;
    const int j = kHalfTokens * h + 2 * quarter + (lane >> 4);   // this lane's token of the tile
    int t = 0, mine = 0;      // pairs so far, and those of this half
    int last_pages = 0;       // of the segment before
    for (int i = 0; ok; ++i) {
      ok = __all_sync(0xffffffffu, wait_for(&tail->seg_full[i & 1], (i >> 1) & 1));
      if (!ok) break;
      const Segment sg = tail->seg[i & 1];
      if (sg.ntok == 0) break;
      if (last_pages < kShort) {
        // at the start, or behind a unit in whose time two warps could not have: a token a warp
        load_token(p, &tail->seg[i & 1], warp - 4, smem + (i & 1) * kQTile, tail->zs[i & 1]);
        if (lane == 0) mbar_arrive(&tail->q_part);
        __syncwarp();
      }
      last_pages = sg.n1 - sg.n0;
      ok = __all_sync(0xffffffffu, wait_for(&tail->q_full[i & 1], (i >> 1) & 1));
      if (!ok) break;
      const float zs = tail->zs[i & 1][j];
      __syncwarp();
      if (lane == 0) mbar_arrive(&tail->seg_empty[i & 1]);
      if (h == 1 && sg.ntok <= kHalfTokens) {
        t += (sg.n1 - sg.n0 + 1) / 2;
        continue;
      }
      const int pos = sg.pos0 + j;
      float* row = p.scores + (static_cast<int64_t>(sg.g) * p.T + sg.tok0 + j) * p.S;
      const bool there = j < sg.ntok;
      float keep = 0.f;                   // the score of block n with n % 16 == lane % 16
      for (int n = sg.n0 + pg; n < sg.n1 + pg; n += 2, ++t, ++mine) {
        // (the products first: a half that skipped units may be many pages early, and
        // info_full's phases come round; it is never late, see the products)
        ok = wait_for(&tail->s_full[h], mine & 1) && wait_for(&tail->info_full[t % kInfo], (t / kInfo) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const bool one = n >= sg.n1;      // the last pair has one page, not this warp's
        const float ks = one ? 0.f : tail->info[t % kInfo][pg];
        tc::fence_after_thread_sync();
        const int lim = pos - n * kPage;  // keys <= lim are visible
        const bool edge = __any_sync(0xffffffffu, lim < kPage - 1);
        float m = -INFINITY;
        if (!one) {
#pragma unroll
          for (int c = 0; c < kPage; c += 32) {
            uint32_t v[32];
            tc::ld_32x32b_x32(at + c, v);
            tc::wait_ld();
            if (edge) {
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = c + e <= lim ? v[e] : 0xFF800000u;
            }
            float a[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              a[k] = fmaxf(__uint_as_float(v[k]), __uint_as_float(v[k + 2]));
#pragma unroll
              for (int e = k + 4; e < 32; e += 4)
                a[k] = fmax3f(a[k], __uint_as_float(v[e]), __uint_as_float(v[e + 2]));
            }
            m = c == 0 ? fmaxf(a[0], a[1]) : fmax3f(m, a[0], a[1]);   // (NaN only where all are)
          }
          tc::fence_before_thread_sync();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&tail->s_empty[h]);
        if (one) continue;
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float sc = ks > 0.f && lim >= 0 ? m * (zs * ks) : -INFINITY;
        if ((n & 15) == (lane & 15)) keep = sc;
        if ((n & 15) >= 14 || n + 2 >= sg.n1) {
          // this warp's eight of 16 neighbouring blocks, of two tokens
          const int at_n = (n & ~15) + (lane & 15);
          if (there && at_n >= sg.n0 && at_n <= n && ((at_n ^ n) & 1) == 0) row[at_n] = keep;
        }
      }
      if (!ok) break;
      // behind the unit's last page: blocks that none of its tokens sees
      const int last = (sg.pos0 + sg.ntok - 1) / kPage;
      if (sg.n1 > last && there)
        for (int n = last + 1 + pg * 16 + (lane & 15); n < p.S; n += 32) row[n] = -INFINITY;
    }
    if (lane == 0) {
      if (!ok) flag_error(p.err, MSA_ERR_TIMEOUT);
      mbar_arrive(&tail->finish);
    }
    __syncwarp();
  }
}

}  // namespace

cudaError_t launch_score_prefill(const CUtensorMap& kv_map, const PrefillParams& p,
                                 cudaStream_t stream, bool pdl) {
  static std::atomic<unsigned long long> attr_done{0};
  const cudaError_t e = once_per_device(attr_done, [&] {
    return cudaFuncSetAttribute(score_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSmemBytes);
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(score_prefill_kernel, dim3(static_cast<unsigned>(p.ctas)), dim3(kThreads),
                    kSmemBytes, stream, pdl, kv_map, p);
}

}  // namespace msa
