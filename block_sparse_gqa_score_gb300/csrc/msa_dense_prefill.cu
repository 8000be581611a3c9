// msa_dense_prefill.cu -- dense attention of a chunk of new tokens over the paged cache:
// the model's dense layers in prefill and chunked prefill.
//
// Operation (msa_dense_prefill in include/msa.h): query token j of request b, at pos =
// seq_lens[b] - q_len + j, attends every key t <= pos of its request:
//   out[i, h] = sum_t softmax_t(sm_scale K_t . q[i, h]) V_t.
// With z the logit in log2 units, vs the page's V scale and u = z + log2(vs),
//   out = v_scale sum_t 2^(u_t - M) V8_t / sum_t 2^(u_t - M) / vs[page(t)],
// so that the product takes weights relative to what a key contributes (without page
// scales vs = 1).
//
// What bounds it: the tensor cores, 4 * 128 * 16 products a key, token and KV head
// against a key's 256 bytes shared by the chunk's tokens.  A unit is 16 tokens x 16 heads,
// two halves of M = 128 query rows; a step is a page of 128 keys:
//   S = Q K^T    e4m3 x e4m3: the keys as stored; a bf16 query is two exact e4m3 parts
//                (two products at twice the rate of a bf16 one, and no conversion of K)
//   softmax      a query row is a tensor-memory lane and a thread: no exchange at all
//   O += P V     fp16 x fp16 with P from tensor memory, where it takes the place of its
//                half's S; the values are converted to fp16 (exact) by four warps, once
//                for both halves.  (P in e4m3 parts would save the conversion and cost the
//                softmax warps, which have more to do, two conversions for each element.)
// While one half's softmax runs, the other half's products do: the tensor core issues
// O(j) and S(j + 1) of one half, then of the other.  S(j + 1) may overwrite P(j) because
// the products of a thread execute in the order they are issued.
//
// P = 2^(u - M + kShift) is relative to a running reference M of the row, the largest u
// rounded up when M is set; M stays until 64 P sum to more than kMost (fp16 holds 65504), so
// that O is rescaled in a row's first pages and then hardly ever, by a power of two, and what
// was made of the page so far with it.  No maximum is taken on the way: S is read 64 columns at
// a time, and only a unit's first piece and one whose sum says so are searched (and, the
// latter, done again).  With the maximum of every piece the four chunks below took 697 us.
// P is rounded to fp16: 2^-11 of itself down to 2^-21 of the row's largest, and at most
// 2^-32 of that below.  Sums are of the unrounded P, in fp32, page by page.
//
// A value row that a token does not see must not reach it even as NaN (0 times NaN): keys
// past the tile's last token are 0 for all, and of those that only some of its tokens see
// NaN codes are set to 0 and put back at the end into the rows that see them.
//
//   warp 0        page look-ups, TMA of K and V tiles
//   warp 1        products (owns tensor memory)
//   warps 2, 3    segments (warp 2); query tiles: tokens 8..15, warps 12..15 two of the others each
//   warps 4..11   softmax and output, four warps a half
//   warps 12..15  values to fp16
// One CTA an SM, each an equal share of all pages (msa_prefill.cuh); what several CTAs
// work on is merged by a second kernel from their parts, in the order of the pages.
//
// Measured, 64/4 heads: four chunks of up to 1k tokens over 4k .. 16k 678 us (1455 TFLOP/s),
// with an fp8 query 635 (the products of both need 512 and 384); one chunk of 1050 tokens over
// 128k on one KV head with page scales 741 us (1515 TFLOP/s); eight prompts of 1024 tokens 241 us
// (72: units of 4.5 pages, whose query tiles, outputs and masked last pages take longer than the
// pages); two chunks of 18 and 27 tokens over 2k .. 3k on one KV head 22.4 us, at most two
// pages a CTA and the rest latency: two launches, the first tiles, each loop's first run, the merge.
// A page takes some 2950 cycles, of which the products alone need 2250 (2048 at the tensor
// core's rate): the rest is the round of one half, S 900 cycles, softmax 1300 (the two halves'
// warps share the issue slots), P handed on 300, O 500, of which the other half's products
// hide most but not all.  S ahead of P would break the round, but two S and a P for each half
// beside O do not fit 512 columns, and with S of 64 keys at a time, where they do, the products
// take as long as those of 128 (856 us for the four chunks).  Slower were too: sixteen softmax
// warps with two threads a row (registers spill), a product warp for each half, pieces of 32
// columns, P handed on in halves.  The warps' code
// has to stay small: seven different loops share the SM's instruction cache, and with the query
// tiles' split and the converter in line (191 KiB) short units took half as long again.
#include <cstddef>

#include "msa_device.cuh"
#include "msa_launch.h"
#include "msa_prefill.cuh"
#include "msa_tcgen05.cuh"

namespace msa {

namespace {

using namespace prefill;

constexpr int kThreads = 512;
constexpr int kSlots = 3;                       // K tiles in flight
constexpr int kVSlots = 2;                      // V tiles as stored, in flight
constexpr int kInfo = 16;                       // pages' factors in flight
constexpr int kSegs = 4;                        // segments known at a time
// A unit's query and output, in pages' time: an fp8 query is copied, a bf16 one split (the four
// chunks above with 4: 693 us; 5: 696, 6: 700, 7: 702).
__device__ __forceinline__ int extra_steps(const PrefillParams& p) { return p.q8 ? 3 : 4; }
constexpr int kMinSteps = 2;
constexpr int kRows = kGroup * kTile;           // query rows of a unit
constexpr int kQTile = 4 * kHalfTile;           // two halves, hi and lo parts
constexpr int kVTile = 2 * kHalfTile;           // a page's values in fp16
constexpr int kOffK = kQTile;
constexpr int kOffV8 = kOffK + kSlots * kHalfTile;
constexpr int kOffV = kOffV8 + kVSlots * kHalfTile;
constexpr int kOffTail = kOffV + 2 * kVTile;
constexpr int kLoaders = 6;                     // warps that prepare query tiles
constexpr int kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;      // [half] of 128 columns each

constexpr float kShift = 8.f;                   // P = 2^kShift at the largest u when M is set
constexpr float kMost = 60000.f;                // M moves when 64 P sum to more
constexpr float kTiny = 0x1p-108f;              // 2^-40 of it is not 0, and 2^40 leaves every logit 0

struct PageInfo {
  float k, lv, iv;      // K scale, log2 and reciprocal of the V scale
  int block;            // logical block; -1: no key of the page is attended
};

struct Tail {
  uint64_t k_full[kSlots], k_empty[kSlots];
  uint64_t v8_full[kVSlots], v8_empty[kVSlots];
  uint64_t v_full[2], v_empty[2];               // fp16 values
  uint64_t s_full[2], p_full[2], o_full[2], o_empty[2];   // by half
  uint64_t info_full[kInfo];
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t q_full, q_empty;
  uint64_t finish;
  uint32_t tmem_base;
  int nan_seen[kSegs];                          // by segment: NaN codes were set to 0
  alignas(16) PageInfo info[kInfo];
  Segment seg[kSegs];
  float zs[kSegs][kTile];
  WalkScratch scratch;
};

constexpr int kSmemBytes = kOffTail + static_cast<int>(sizeof(Tail)) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

// Four e4m3 codes (a word) -> four fp16 (exact).
__device__ __forceinline__ uint2 e4m3x4_to_f16x4(uint32_t w) {
  uint2 r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(w));
  return r;
}

// 0x80 in each byte of w that is an e4m3 NaN (0x7F or 0xFF).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

__device__ __forceinline__ void add2(float& d0, float& d1, float b0, float b1) {
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%0, %1};\n\t"
      "mov.b64 y, {%2, %3};\n\t"
      "add.rn.f32x2 x, x, y;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "+f"(d0), "+f"(d1)
      : "f"(b0), "f"(b1));
}
// (a0, a1) * b + c
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b, float c) {
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%2, %3};\n\t"
      "mov.b64 y, {%4, %4};\n\t"
      "mov.b64 z, {%5, %5};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b), "f"(c));
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Four lanes' rows of four 16-byte pieces turned: lane k of a group of four gets piece k of
// each of its rows, so that a store of the group is 64 bytes of one row.  (A thread's row
// stored by itself, 16 bytes a line, took 4.5 us a unit.)
__device__ __forceinline__ void turn4(uint4 (&v)[4], int lane) {
  auto trade = [&](uint4& a, uint4& b, bool up, int x) {   // up: a goes, else b
    uint4 g = up ? a : b;
    g.x = __shfl_xor_sync(0xffffffffu, g.x, x);
    g.y = __shfl_xor_sync(0xffffffffu, g.y, x);
    g.z = __shfl_xor_sync(0xffffffffu, g.z, x);
    g.w = __shfl_xor_sync(0xffffffffu, g.w, x);
    if (up) a = g;
    else b = g;
  };
  const bool b0 = lane & 1, b1 = lane & 2;
  trade(v[0], v[1], b0, 1);
  trade(v[2], v[3], b0, 1);
  trade(v[0], v[2], b1, 2);
  trade(v[1], v[3], b1, 2);
}

__global__ void __launch_bounds__(kThreads, 1)
    dense_prefill_kernel(const __grid_constant__ CUtensorMap kv_map, const PrefillParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Tail* tail = reinterpret_cast<Tail*>(smem + kOffTail);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int parts = p.q8 ? 1 : 2;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&tail->k_full[s], 1);
      mbar_init(&tail->k_empty[s], 1);
    }
    for (int s = 0; s < kVSlots; ++s) {
      mbar_init(&tail->v8_full[s], 1);
      mbar_init(&tail->v8_empty[s], 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&tail->v_full[s], 4);
      mbar_init(&tail->v_empty[s], 1);
      mbar_init(&tail->s_full[s], 1);
      mbar_init(&tail->p_full[s], 4);
      mbar_init(&tail->o_full[s], 1);
      mbar_init(&tail->o_empty[s], 4);
    }
    for (int s = 0; s < kSegs; ++s) {
      mbar_init(&tail->seg_full[s], 1);
      mbar_init(&tail->seg_empty[s], 1 + 1 + 1 + 8 + 4);   // warps 0, 1, 3, 4..11, 12..15
    }
    for (int s = 0; s < kInfo; ++s) mbar_init(&tail->info_full[s], 1);
    mbar_init(&tail->q_full, kLoaders);
    mbar_init(&tail->q_empty, 1);
    mbar_init(&tail->finish, 1 + 1 + 2 + 8 + 4);
    fence_barrier_init();
    prefetch_tensormap(&kv_map);
  } else if (warp == 1) {
    tc::tmem_alloc(&tail->tmem_base, kTmemCols);
    tc::tmem_relinquish();
  }
  pdl_wait();   // lengths, tables and queries may be an earlier kernel's
  const bool bad = plan_walk<kThreads>(p, extra_steps(p), kMinSteps, &tail->scratch);
  bool any_cut = false;          // (warp 2's first lane, which goes on with the segments)
  if (threadIdx.x == 64) {
    int n;
    tail->seg[0] = next_segment(p, tail->scratch.walk, extra_steps(p), any_cut, n);
    tail->nan_seen[0] = 0;
    if (any_cut) p.cut[blockIdx.x] = make_int4(n, tail->seg[0].tok0, tail->seg[0].ntok, tail->seg[0].g);
  }
  tc::fence_before_thread_sync();
  __syncthreads();
  tc::fence_after_thread_sync();
  const uint32_t tmem = tail->tmem_base;
  fill_uncovered(p, bad, [&](int i) {
    uint4* row = reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(i) * p.Hq * kHeadDim);
    for (int x = threadIdx.x; x < p.Hq * kHeadDim / 8; x += kThreads) row[x] = make_uint4(0u, 0u, 0u, 0u);
  });
  bool ok = true;
  // The first query tile: nobody but warp 0, which loads the first pages, has anything else
  // to do yet.
  if (warp > 0 && tail->seg[0].ntok > 0 && tail->seg[0].n0 < tail->seg[0].n1) {
    (void)load_query_tile<2, 2>(p, tail->seg[0], warp - 1, 15, smem, tail->zs[0], lane, [] { return true; });
    named_barrier(1, 32 * 15);
  }

  if (warp < 4) {
    if (warp == 0) {
      // ---- K and V tiles -----------------------------------------------------------------------
      int t = 0;    // pages so far
      for (int i = 0; ok; ++i) {
        ok = __all_sync(0xffffffffu, wait_for(&tail->seg_full[i & 3], (i >> 2) & 1));
        if (!ok) break;
        const Segment sg = tail->seg[i & 3];
        __syncwarp();
        if (lane == 0) mbar_arrive(&tail->seg_empty[i & 3]);
        if (sg.ntok == 0) break;
        const int32_t* trow = p.block_table + static_cast<int64_t>(sg.b) * p.S;
        for (int n0 = sg.n0; n0 < sg.n1 && ok; n0 += 32) {
          // 32 pages' entries and scales at once, a lane each
          const int n = n0 + lane;
          int page = 0;
          PageInfo info{1.f, 0.f, 1.f, -1};
          if (n < sg.n1) {
            page = trow[n];
            if (page < 0 || static_cast<int64_t>(page) >= p.num_blocks) {
              flag_error(p.err, MSA_ERR_PAGE_RANGE);
              page = 0;
            } else {
              info.block = n;
              if (p.kv_scales) {
                const PageScale sc = make_page_scale(load_page_scale(p.kv_scales, page, p.Hkv, sg.g));
                if (sc.bad != 0.f) flag_error(p.err, MSA_ERR_SCALE);
                info = PageInfo{sc.k, sc.lv, sc.iv, sc.bad != 0.f ? -1 : n};
              }
            }
          }
          const int have = min(32, sg.n1 - n0);
          for (int x = 0; x < have; ++x, ++t) {
            const int s = t % kSlots, sv = t % kVSlots;
            ok = t < kSlots || wait_for(&tail->k_empty[s], ((t / kSlots) - 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const int row = (page * p.Hkv + sg.g) * kPage;
            if (lane == x) {
              tail->info[t % kInfo] = info;
              mbar_arrive(&tail->info_full[t % kInfo]);
              mbar_arrive_expect_tx(&tail->k_full[s], kHalfTile);
              tma_load_2d(smem + kOffK + s * kHalfTile, &kv_map, 0, row, &tail->k_full[s]);
            }
            ok = t < kVSlots || wait_for(&tail->v8_empty[sv], ((t / kVSlots) - 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (ok && lane == x) {
              mbar_arrive_expect_tx(&tail->v8_full[sv], kHalfTile);
              tma_load_2d(smem + kOffV8 + sv * kHalfTile, &kv_map, kHeadDim, row, &tail->v8_full[sv]);
            }
            __syncwarp();
            if (!ok) {      // this page's K tile is on its way, its V tile is not
              if (lane == 0) (void)wait_for(&tail->k_full[s], (t / kSlots) & 1);
              break;
            }
          }
        }
      }
      if (lane == 0) {
        if (!ok) flag_error(p.err, MSA_ERR_TIMEOUT);
        // the loads still in flight land before shared memory can be released
        for (int x = max(0, t - kSlots); x < t; ++x)
          (void)wait_for(&tail->k_full[x % kSlots], (x / kSlots) & 1);
        for (int x = max(0, t - kVSlots); x < t; ++x)
          (void)wait_for(&tail->v8_full[x % kVSlots], (x / kVSlots) & 1);
        pdl_trigger();
        mbar_arrive(&tail->finish);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---- products ----------------------------------------------------------------------------
      const uint64_t q0 = tc::sw128_kmajor_desc(smem_u32(smem));
      const uint64_t k0 = tc::sw128_kmajor_desc(smem_u32(smem + kOffK));
      const uint64_t v0 = tc::sw128_mnmajor16_desc(smem_u32(smem + kOffV), kHalfTile);
      constexpr uint32_t idesc_s = tc::idesc_e4m3_f32(128, kPage);
      constexpr uint32_t idesc_o = tc::idesc_f16_f32_bmn(128, kHeadDim);
      const bool leader = tc::elect_one();
      // (the vote makes it the same for the compiler as well)
      auto wait = [&](uint64_t* bar, unsigned parity) {
        return __all_sync(0xffffffffu, wait_for(bar, parity)) != 0;
      };
      int t = 0, s = 0;          // pages whose S is issued; its slot
      unsigned k_par = 0;
      int n_p0 = 0, n_p1 = 0;    // pages whose O is issued, by half
      int n_o0 = 0, n_o1 = 0;    // units whose O was begun, by half
      // S of half h against the K tile in slot s
      auto scores = [&](int h) {
        if (leader) {
          const uint64_t bk = k0 + static_cast<uint64_t>(s) * (kHalfTile >> 4);
          const uint64_t aq = q0 + static_cast<uint64_t>(h) * (2 * kHalfTile >> 4);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            tc::mma_e4m3(tmem + kColS + 128 * h, aq + 2 * ks, bk + 2 * ks, idesc_s, ks > 0);
          if (parts == 2) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              tc::mma_e4m3(tmem + kColS + 128 * h, aq + (kHalfTile >> 4) + 2 * ks, bk + 2 * ks, idesc_s, 1);
          }
          tc::commit(&tail->s_full[h]);
        }
        __syncwarp();
      };
      // O of half h with the values of page tv (of all pages)
      auto output = [&](int h, int tv, bool begin, int& n_p, int& n_o) {
        if (!wait(&tail->p_full[h], n_p & 1)) return false;
        if (!wait(&tail->v_full[tv & 1], (tv >> 1) & 1)) return false;
        if (begin) {             // the unit before has been read out of O
          if (n_o > 0 && !wait(&tail->o_empty[h], (n_o - 1) & 1)) return false;
          ++n_o;
        }
        ++n_p;
        tc::fence_after_thread_sync();
        if (leader) {
          const uint64_t bv = v0 + static_cast<uint64_t>(tv & 1) * (kVTile >> 4);
          // 16 keys each: 8 columns of P, two 8-row groups of V
          tc::mma_f16_tmem(tmem + kColO + 128 * h, tmem + kColS + 128 * h, bv, idesc_o, !begin);
#pragma unroll
          for (int ks = 1; ks < 8; ++ks)
            tc::mma_f16_tmem(tmem + kColO + 128 * h, tmem + kColS + 128 * h + 8 * ks,
                             bv + static_cast<uint64_t>(ks) * (2048 >> 4), idesc_o, 1);
        }
        __syncwarp();
        return true;
      };
      for (int i = 0; ok; ++i) {
        ok = wait(&tail->seg_full[i & 3], (i >> 2) & 1);
        if (!ok) break;
        const int ntok = __reduce_max_sync(0xffffffffu, tail->seg[i & 3].ntok);
        const int pages = __reduce_max_sync(0xffffffffu, tail->seg[i & 3].n1 - tail->seg[i & 3].n0);
        if (leader) mbar_arrive(&tail->seg_empty[i & 3]);
        __syncwarp();
        if (ntok == 0) break;
        if (pages == 0) continue;
        const bool both = ntok > kHalfTokens;
        ok = wait(&tail->q_full, n_o0 & 1);
        for (int x = 0; x <= pages && ok; ++x) {
          if (x > 0) {
            ok = output(0, t - 1, x == 1, n_p0, n_o0);
            if (!ok) break;
            if (leader) {
              if (!both) tc::commit(&tail->v_empty[(t - 1) & 1]);
              if (x == pages) tc::commit(&tail->o_full[0]);
            }
            __syncwarp();
          }
          if (x < pages) {
            ok = wait(&tail->k_full[s], k_par);
            if (!ok) break;
            tc::fence_after_thread_sync();
            scores(0);
          }
          if (both) {
            if (x > 0) {
              ok = output(1, t - 1, x == 1, n_p1, n_o1);
              if (!ok) break;
              if (leader) {
                tc::commit(&tail->v_empty[(t - 1) & 1]);
                if (x == pages) tc::commit(&tail->o_full[1]);
              }
              __syncwarp();
            }
            if (x < pages) scores(1);
          }
          if (x < pages) {
            if (leader) {
              tc::commit(&tail->k_empty[s]);
              if (x == pages - 1) tc::commit(&tail->q_empty);   // the query tile has been read
            }
            __syncwarp();
            ++t;
            if (++s == kSlots) {
              s = 0;
              k_par ^= 1;
            }
          }
        }
      }
      if (leader) {
        if (!ok) flag_error(p.err, MSA_ERR_TIMEOUT);
        tc::commit(&tail->finish);
      }
      __syncwarp();
      (void)mbar_wait(&tail->finish, 0);
      tc::fence_after_thread_sync();
      tc::tmem_dealloc(tmem, kTmemCols);
    } else {
      // ---- segments and query tiles --------------------------------------------------------------
      const int h = warp - 2;
      int tiles = 0;         // query tiles so far
      bool more = true;      // warp 2: the last segment is not known yet
      for (int i = 0;; ++i) {
        if (h == 0) {
          // up to two segments ahead, so that their queries can be on their way
          for (int a = i == 0 ? 0 : i + 2; a <= i + 2 && more; ++a) {
            ok = __all_sync(0xffffffffu, a < kSegs || wait_for(&tail->seg_empty[a & 3], ((a >> 2) - 1) & 1));
            if (!ok) break;
            if (lane == 0) {
              if (a > 0) {
                bool cut;
                int n;
                const Segment next = next_segment(p, tail->scratch.walk, extra_steps(p), cut, n);
                tail->seg[a & 3] = next;
                tail->nan_seen[a & 3] = 0;
                if (cut) p.cut[blockIdx.x] = make_int4(n, next.tok0, next.ntok, next.g);
                any_cut |= cut;
              }
              mbar_arrive(&tail->seg_full[a & 3]);
            }
            __syncwarp();
            more = tail->seg[a & 3].ntok > 0;
          }
          if (!ok) break;
        } else {
          ok = __all_sync(0xffffffffu, wait_for(&tail->seg_full[i & 3], (i >> 2) & 1));
          if (!ok) break;
        }
        const Segment sg = tail->seg[i & 3];
        if (h == 0) {
          // a part without pages (of the unit's extra steps alone) is empty
          if (sg.ntok > 0 && sg.slot >= 0 && sg.n0 == sg.n1)
            for (int x = lane; x < kRows; x += 32)
              p.part_ml[static_cast<int64_t>(sg.slot) * kRows + x] = make_float2(-INFINITY, 0.f);
        }
        if (sg.ntok > 0 && sg.n0 < sg.n1) {
          // tokens 8 + h, 10 + h, .. (warps 12..15 take the first eight)
          if (i > 0)
            ok = load_query_tile<4, 2>(p, sg, kHalfTokens + h, 2, smem, tail->zs[i & 3], lane, [&] {
              return __all_sync(0xffffffffu, tiles == 0 || wait_for(&tail->q_empty, (tiles - 1) & 1)) != 0;
            });
          if (!ok) break;
          ++tiles;
          if (lane == 0) mbar_arrive(&tail->q_full);
        }
        __syncwarp();
        if (lane == 0 && h == 1) mbar_arrive(&tail->seg_empty[i & 3]);
        if (sg.ntok == 0) break;
      }
      if (lane == 0) {
        if (h == 0 && !any_cut) p.cut[blockIdx.x] = make_int4(0, 0, 0, 0);
        if (!ok) flag_error(p.err, MSA_ERR_TIMEOUT);
        mbar_arrive(&tail->finish);
      }
      __syncwarp();
    }
  } else if (warp < 12) {
    // ---- softmax of one half -------------------------------------------------------------------
    const int h = (warp - 4) >> 2, quarter = warp & 3;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
    const uint32_t s_at = lane_addr + kColS + 128 * h, o_at = lane_addr + kColO + 128 * h;
    const int row = 32 * quarter + lane;                 // of the half
    const int j = kHalfTokens * h + row / kGroup;        // this row's token of the tile
    int t = 0, mine = 0, units = 0;
    for (int i = 0; ok; ++i) {
      ok = __all_sync(0xffffffffu, wait_for(&tail->seg_full[i & 3], (i >> 2) & 1));
      if (!ok) break;
      const Segment sg = tail->seg[i & 3];
      if (sg.ntok == 0) break;
      const int pages = sg.n1 - sg.n0;
      if (pages == 0 || (h == 1 && sg.ntok <= kHalfTokens)) {
        t += pages;
        __syncwarp();
        if (lane == 0) mbar_arrive(&tail->seg_empty[i & 3]);
        continue;
      }
      const int pos = sg.pos0 + j;
      float zs = 0.f;
      float M = -INFINITY;      // the reference, -inf until the row has seen a key
      float l = 0.f;
      for (int n = sg.n0; n < sg.n1; ++n, ++t, ++mine) {
        ok = wait_for(&tail->s_full[h], mine & 1) &&
             wait_for(&tail->info_full[t % kInfo], (t / kInfo) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const PageInfo in = tail->info[t % kInfo];
        if (n == sg.n0) zs = fmaxf(tail->zs[i & 3][j], kTiny);   // (0 times a masked -inf is NaN)
        tc::fence_after_thread_sync();
        const int lim = in.block < 0 ? -1 : pos - n * kPage;  // keys <= lim are visible
        const bool edge = __any_sync(0xffffffffu, lim < kPage - 1);
        const float zt = zs * in.k;
        // (no reference yet, of a row that has seen no key: every P comes out as infinity or NaN)
        float nl = M == -INFINITY ? INFINITY : in.lv - M + kShift;
        float lp = 0.f;           // the page's sum
#pragma unroll 1
        for (int c = 0; c < kPage; c += 64) {
          uint32_t w[32];
          float sum = INFINITY;
#pragma unroll 1
          for (bool known = n > sg.n0 || c > 0, last = false;; known = last = true) {
            if (known) {
              float a0 = 0.f, a1 = 0.f, b0 = 0.f, b1 = 0.f;
              float s[64];
              {
                uint32_t v[2][32];
                tc::ld_32x32b_x32(s_at + c, v[0]);
                tc::ld_32x32b_x32(s_at + c + 32, v[1]);
                tc::wait_ld();
#pragma unroll
                for (int e = 0; e < 64; ++e) s[e] = __uint_as_float(v[e >> 5][e & 31]);
              }
              if (edge) {
                const int to = lim - c;
#pragma unroll
                for (int e = 0; e < 64; ++e) s[e] = e <= to ? s[e] : -INFINITY;
              }
#pragma unroll
              for (int e = 0; e < 64; e += 4) {
                float x0, x1, x2, x3;
                fma2(x0, x1, s[e], s[e + 1], zt, nl);
                fma2(x2, x3, s[e + 2], s[e + 3], zt, nl);
                x0 = ex2(x0), x1 = ex2(x1), x2 = ex2(x2), x3 = ex2(x3);
                add2(a0, a1, x0, x1);
                add2(b0, b1, x2, x3);
                w[e / 2] = pack_f16x2(x0, x1);
                w[e / 2 + 1] = pack_f16x2(x2, x3);
              }
              sum = (a0 + a1) + (b0 + b1);
              if (last || __all_sync(0xffffffffu, sum <= kMost)) break;
            }
            // the first piece, or some P may have passed fp16: M moves to the row's largest
            float top = -INFINITY;          // -inf: no visible key
#pragma unroll 1
            for (int k = c; k < c + 64; k += 32) {
              uint32_t v[32];
              tc::ld_32x32b_x32(s_at + k, v);
              tc::wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (k + e <= lim) top = fmaxf(top, __uint_as_float(v[e]));
            }
            const float u = fmaf(top, zt, in.lv);
            const bool move = u > M && !(sum <= kMost);
            const float to = move ? ceilf(u) : M;
            const float al = move ? ex2(M - to) : 1.f;         // a power of two; 0 at the first
            M = to;
            nl = M == -INFINITY ? 0.f : in.lv - M + kShift;
            l *= al;
            lp *= al;
            // this page's P so far
            tc::wait_st();
#pragma unroll 1
            for (int k = 0; k < c / 2; k += 8) {
              uint32_t v[8];
              tc::ld_32x32b_x8(s_at + k, v);
              tc::wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[e]));
                v[e] = pack_f16x2(f.x * al, f.y * al);
              }
              tc::st_32x32b_x8(s_at + k, v);
            }
            if (n > sg.n0) {
              // the products so far are complete: S(n) was issued behind them
#pragma unroll 1
              for (int k = 0; k < kHeadDim; k += 8) {
                uint32_t v[8];
                tc::ld_32x32b_x8(o_at + k, v);
                tc::wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * al);
                tc::st_32x32b_x8(o_at + k, v);
              }
            }
          }
          lp += sum;
          tc::st_32x32b_x32(s_at + c / 2, w);    // over columns that have been read
        }
        l = fmaf(lp, in.iv, l);
        tc::wait_st();
        tc::fence_before_thread_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tail->p_full[h]);
      }
      if (!ok) break;
      // ---- the row's output
      ok = __all_sync(0xffffffffu, wait_for(&tail->o_full[h], units & 1));
      if (!ok) break;
      ++units;
      tc::fence_after_thread_sync();
      const bool nan_seen = tail->nan_seen[i & 3] != 0;
      const bool there = j < sg.ntok;
      // (P was 2^kShift times the weights; a row with a NaN logit is NaN altogether)
      float inv = l > 0.f ? __fdividef(p.v_scale, l) : 0.f;
      if (l != l) inv = l;
      const bool whole = sg.slot < 0;
      // rows are written four at a time, 64 bytes of each by a group of four lanes
      const int row4 = 128 * h + 32 * quarter + (lane & ~3), piece = lane & 3;
#pragma unroll 1
      for (int c = 0; c < kHeadDim; c += 32) {
        uint32_t v[32];
        tc::ld_32x32b_x32(o_at + c, v);
        tc::wait_ld();
        if (nan_seen) {
          // value rows that only some of the tile's tokens see: back to NaN for this one
          for (int key = sg.pos0 + 1; key <= pos && there; ++key) {
            const int n = key / kPage;
            if (n < sg.n0 || n >= sg.n1) continue;
            const int page = p.block_table[static_cast<int64_t>(sg.b) * p.S + n];
            if (page < 0 || static_cast<int64_t>(page) >= p.num_blocks) continue;
            if (p.kv_scales &&
                make_page_scale(load_page_scale(p.kv_scales, page, p.Hkv, sg.g)).bad != 0.f)
              continue;
            const uint8_t* val = p.kv + ((static_cast<int64_t>(page) * p.Hkv + sg.g) * kPage + key % kPage) *
                                 kRowBytes + kHeadDim + c;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if ((val[e] & 0x7F) == 0x7F) v[e] = 0x7FFFFFFFu;
          }
        }
        if (whole) {
          uint4 q[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              o[e] = pack_bf16x2(__uint_as_float(v[8 * x + 2 * e]) * inv,
                                 __uint_as_float(v[8 * x + 2 * e + 1]) * inv);
            q[x] = make_uint4(o[0], o[1], o[2], o[3]);
          }
          turn4(q, lane);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int r = row4 + x;
            if (r / kGroup < sg.ntok)
              *reinterpret_cast<uint4*>(
                  p.out + (static_cast<int64_t>(sg.tok0 + r / kGroup) * p.Hq + sg.g * kGroup + r % kGroup) *
                              kHeadDim + c + 8 * piece) = q[x];
          }
        } else {
#pragma unroll
          for (int y = 0; y < 32; y += 16) {
            uint4 q[4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
              q[x] = make_uint4(v[y + 4 * x], v[y + 4 * x + 1], v[y + 4 * x + 2], v[y + 4 * x + 3]);
            turn4(q, lane);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int r = row4 + x;
              if (r / kGroup < sg.ntok)
                *reinterpret_cast<uint4*>(p.part_o + (static_cast<int64_t>(sg.slot) * kRows + r) * kHeadDim +
                                          c + y + 4 * piece) = q[x];
            }
          }
        }
      }
      if (!whole && there)
        p.part_ml[static_cast<int64_t>(sg.slot) * kRows + 128 * h + row] = make_float2(M, l);
      tc::fence_before_thread_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&tail->o_empty[h]);
        mbar_arrive(&tail->seg_empty[i & 3]);
      }
    }
    if (lane == 0) {
      if (!ok) flag_error(p.err, MSA_ERR_TIMEOUT);
      mbar_arrive(&tail->finish);
    }
    __syncwarp();
  } else {
    // ---- values to fp16 ------------------------------------------------------------------------
    // eight lanes take 16-byte chunks 0..3 of an even key's row and 4..7 of the next one's
    // (then the other way round), so that neither side has bank conflicts
    const int w4 = warp - 12;
    int t = 0, tiles = 0;
    // tokens 2 w4 and 2 w4 + 1 of the next query tile, asked for a segment ahead
    QueryRows rows[2];
    for (int i = 0; ok; ++i) {
      ok = __all_sync(0xffffffffu, wait_for(&tail->seg_full[i & 3], (i >> 2) & 1));
      if (!ok) break;
      const Segment sg = tail->seg[i & 3];
      if (sg.ntok == 0) break;
      if (sg.n0 < sg.n1) {
        if (i > 0) {
          float z[2];
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (2 * w4 + k < sg.ntok) z[k] = rows[k].split<2>(p);
          ok = __all_sync(0xffffffffu, tiles == 0 || wait_for(&tail->q_empty, (tiles - 1) & 1));
          if (!ok) break;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int j = 2 * w4 + k;
            if (j < sg.ntok) {
              rows[k].store(p, kGroup * j, smem, smem + kHalfTile, lane);
            } else {
              zero_query_rows(kGroup * j, smem, lane);
              if (!p.q8) zero_query_rows(kGroup * j, smem + kHalfTile, lane);
            }
            if (lane == 0) tail->zs[i & 3][j] = j < sg.ntok ? z[k] : 0.f;
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
        }
        ++tiles;
        if (lane == 0) mbar_arrive(&tail->q_full);
        __syncwarp();
      }
      ok = __all_sync(0xffffffffu, wait_for(&tail->seg_full[(i + 1) & 3], ((i + 1) >> 2) & 1));
      if (!ok) break;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (2 * w4 + k < tail->seg[(i + 1) & 3].ntok)
          rows[k].load(p, tail->seg[(i + 1) & 3].tok0 + 2 * w4 + k, tail->seg[(i + 1) & 3].g, lane);
      for (int n = sg.n0; n < sg.n1; ++n, ++t) {
        const int sv = t % kVSlots, b = t & 1;
        ok = wait_for(&tail->v8_full[sv], (t / kVSlots) & 1) &&
             wait_for(&tail->info_full[t % kInfo], (t / kInfo) & 1) &&
             (t < 2 || wait_for(&tail->v_empty[b], ((t >> 1) - 1) & 1));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const bool none = tail->info[t % kInfo].block < 0;
        // keys <= all: seen by every token of the tile; keys > last: by none
        const int all = none ? -1 : sg.pos0 - n * kPage;
        const int last = none ? -1 : all + sg.ntok - 1;
        const uint8_t* from = smem + kOffV8 + sv * kHalfTile;
        uint8_t* to = smem + kOffV + b * kVTile;
        bool nan = false;
        // chunk x of this lane: which key of the page and which 16 bytes of its row
        auto key_of = [&](int x) { return 32 * w4 + 8 * (x >> 1) + 2 * (lane >> 3) + ((lane >> 2) & 1); };
        auto piece_of = [&](int x) { return (lane & 3) + 4 * (((lane >> 2) & 1) ^ (x & 1)); };
        auto convert = [&](const uint4& r, int key, int c) {
          const uint2 f0 = e4m3x4_to_f16x4(r.x), f1 = e4m3x4_to_f16x4(r.y);
          const uint2 f2 = e4m3x4_to_f16x4(r.z), f3 = e4m3x4_to_f16x4(r.w);
          uint8_t* half = to + (c >> 2) * kHalfTile;
          *reinterpret_cast<uint4*>(half + sw128(key, 2 * (c & 3))) = make_uint4(f0.x, f0.y, f1.x, f1.y);
          *reinterpret_cast<uint4*>(half + sw128(key, 2 * (c & 3) + 1)) = make_uint4(f2.x, f2.y, f3.x, f3.y);
        };
        if (all >= kPage - 1) {
#pragma unroll 4
          for (int x = 0; x < 8; ++x)
            convert(*reinterpret_cast<const uint4*>(from + sw128(key_of(x), piece_of(x))), key_of(x), piece_of(x));
        } else {
#pragma unroll 1
          for (int x = 0; x < 8; ++x) {
            const int key = key_of(x), c = piece_of(x);
            uint4 r = *reinterpret_cast<const uint4*>(from + sw128(key, c));
            if (key > last) {
              r = make_uint4(0u, 0u, 0u, 0u);
            } else if (key > all) {
              uint32_t* q = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t m = nan_bytes(q[e]);
                nan |= m != 0;
                q[e] &= ~((m >> 7) * 0xFFu);
              }
            }
            convert(r, key, c);
          }
        }
        if (nan) tail->nan_seen[i & 3] = 1;
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&tail->v8_empty[sv]);
          mbar_arrive(&tail->v_full[b]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&tail->seg_empty[i & 3]);
    }
    if (lane == 0) {
      if (!ok) flag_error(p.err, MSA_ERR_TIMEOUT);
      mbar_arrive(&tail->finish);
    }
    __syncwarp();
  }
}

// ---- merge of shared units: blockIdx.x's unit, a warp a query row ------------------------------
constexpr int kMergeWarps = 8;

__global__ void __launch_bounds__(kMergeWarps * 32) merge_kernel(const PrefillParams p) {
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 cut = p.cut[blockIdx.x];    // parts, first token, tokens, KV head
  const int row = blockIdx.y * kMergeWarps + warp;
  if (cut.x == 0 || row >= kGroup * cut.z) return;
  const int64_t c = blockIdx.x;
  auto place = [&](int k) { return (k == 0 ? 2 * c + 1 : 2 * (c + k)) * kRows + row; };
  float M = -INFINITY;
  for (int k = lane; k < cut.x; k += 32) {
    const float2 ml = p.part_ml[place(k)];
    if (ml.y != 0.f) M = fmaxf(M, ml.x);
  }
  M = warp_max_f32(M);
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < cut.x; k0 += 32) {
    // lane k: the weight of part k0 + k, 0 where it is empty
    const float2 ml = k0 + lane < cut.x ? p.part_ml[place(k0 + lane)] : make_float2(0.f, 0.f);
    const float mine = ml.y == 0.f ? 0.f : ml.x == -INFINITY ? 1.f : ex2(ml.x - M);   // (no reference: NaN)
    const int have = min(32, cut.x - k0);
    for (int k = 0; k < have; k += 4) {
      float4 v[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const bool some = __shfl_sync(0xffffffffu, ml.y, (k + x) & 31) != 0.f && k + x < have;
        v[x] = some ? *reinterpret_cast<const float4*>(p.part_o + place(k0 + k + x) * kHeadDim + 4 * lane)
                    : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float w = k + x < have ? __shfl_sync(0xffffffffu, mine, (k + x) & 31) : 0.f;
        // (a weight that vanishes does not keep a NaN out; an empty part is zeros)
        l = fmaf(w, __shfl_sync(0xffffffffu, ml.y, (k + x) & 31), l);
        o.x = fmaf(w, v[x].x, o.x);
        o.y = fmaf(w, v[x].y, o.y);
        o.z = fmaf(w, v[x].z, o.z);
        o.w = fmaf(w, v[x].w, o.w);
      }
    }
  }
  float inv = l > 0.f ? __fdividef(p.v_scale, l) : 0.f;
  if (l != l) inv = l;
  uint2 w;
  w.x = f32_to_bf16_bits(o.x * inv) | (f32_to_bf16_bits(o.y * inv) << 16);
  w.y = f32_to_bf16_bits(o.z * inv) | (f32_to_bf16_bits(o.w * inv) << 16);
  uint16_t* out = p.out + (static_cast<int64_t>(cut.y + row / kGroup) * p.Hq + cut.w * kGroup +
                           row % kGroup) * kHeadDim;
  *reinterpret_cast<uint2*>(out + 4 * lane) = w;
}

}  // namespace

size_t dense_prefill_workspace(int ctas) {
  return static_cast<size_t>(ctas) * (2 * kRows * (kHeadDim * sizeof(float) + sizeof(float2)) + sizeof(int4));
}

cudaError_t launch_dense_prefill(const CUtensorMap& kv_map, const PrefillParams& p,
                                 cudaStream_t stream, bool pdl) {
  static std::atomic<unsigned long long> attr_done{0};
  cudaError_t e = once_per_device(attr_done, [&] {
    return cudaFuncSetAttribute(dense_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSmemBytes);
  });
  if (e != cudaSuccess) return e;
  e = launch_pdl(dense_prefill_kernel, dim3(static_cast<unsigned>(p.ctas)), dim3(kThreads), kSmemBytes,
                 stream, pdl, kv_map, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(merge_kernel, dim3(static_cast<unsigned>(p.ctas), kRows / kMergeWarps),
                    dim3(kMergeWarps * 32), 0, stream, true, p);
}

}  // namespace msa
