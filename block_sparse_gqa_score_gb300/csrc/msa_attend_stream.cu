// msa_attend_stream.cu -- the attend on lists and page scales for batches of more
// (token, KV head) rows than CTAs fit the GPU: prefill and large decode batches.
//
// Operation and products as msa_attend_scaled.cu with one token a tile; here a CTA
// stays and takes row after row (row blockIdx.x + i * gridDim.x), and its roles run
// ahead of each other across rows: while the softmax is in a row's last pages the
// producer has looked up the next row's list, pages and scales and loads its K tiles,
// and the query's parts are built as soon as the row's last S^T product is done.  With
// a CTA a row the look-ups, the query and the output (8000 of 36000 cycles for 16
// pages) were in line with the pages: 334 us for 1536 prefill tokens of 64/4 heads
// over 8k-32k tokens.
//   warp 0       lists, scales, query parts, TMA of K tiles
//   warp 1       S^T products (and owns tensor memory)
//   warp 2       TMA of V tiles; sets the value rows that the token does not see to 0
//   warp 3       O^T products
//   warps 4..11  softmax and output, two groups of four warps, eight heads each
// A row is an item; an item's pages and scales are in one of two places, filled by
// warp 0 and freed by its readers: the softmax and warps 2 and 3 (a row without pages has
// no product that would show them to be past it), warp 1 by the end of its products.
// Pages, batches of pages and items are counted on across rows, each role for itself, and
// give every barrier's slot and phase.  Two CTAs an SM.  (The products are issued by code
// that one lane alone runs: issued from a branch inside a loop of the whole warp, the
// query descriptor that reached the tensor core was wrong.)
//
// Measured: 273 us for those 1536 tokens, 11.9 TB/s of pages out of L2; what bounds it are
// the softmax warps, 16 of them an SM: 61 % of the issue slots, the rest their chain of
// waits, and no pipe: without the loads it takes 5 % less.
#include <cstddef>

#include "msa_device.cuh"
#include "msa_launch.h"
#include "msa_page_softmax.cuh"
#include "msa_tcgen05.cuh"

namespace msa {

namespace {

using namespace paged;

constexpr int kSlots = 3;                       // of the K ring and of the V ring
constexpr int kBatch = Groups<1>::kBatch;
constexpr int kH = Groups<1>::kHeads, kCount = Groups<1>::kCount;
constexpr int kThreads = Groups<1>::kThreads;
constexpr int kPBlock = 8 * 32, kPBuf = kPage * 32;
constexpr int kOffV = kSlots * kHalfTile;
constexpr int kOffQ = 2 * kOffV;
constexpr int kOffP = kOffQ + 32 * 128;
constexpr int kOffTail = kOffP + kBatch * kPBuf;
constexpr int kTmemCols = 256;

struct Item {
  PageInfo info[kTopK];
  int pages[kTopK];
  int n_pages, pos;
  int current;              // the token's own block is listed (and so the first page)
  float zs;                 // logit scale (log2 units) times 2^e of the query split
};

struct Tail {
  uint64_t k_full[kSlots], k_empty[kSlots];   // TMA <-> S^T
  uint64_t v_full[kSlots], v_empty[kSlots];   // TMA <-> O^T
  uint64_t v_land;                  // TMA -> warp 2: a V tile with rows to be zeroed
  uint64_t s_full[2], s_empty[2];   // S^T <-> softmax, a batch a buffer
  uint64_t p_full, o_done;          // softmax <-> O^T, a batch at a time
  uint64_t q_free;                  // an item's S^T products complete
  uint64_t item_full[2];            // pages, scales and the query's tile are there
  uint64_t item_empty[2];           // the softmax and warps 2 and 3 are through with the item
  uint64_t finish;
  uint32_t tmem_base;
  alignas(16) Item item[2];
  alignas(16) float mx[kCount][kH][4];
  alignas(16) float lsum[kCount][kH][4];
};
static_assert(offsetof(Tail, item) % 16 == 0 && sizeof(Item) % 16 == 0 &&
              offsetof(Tail, mx) % 16 == 0 && offsetof(Tail, lsum) % 16 == 0, "float4 access");

constexpr int kSmemBytes = kOffTail + static_cast<int>((sizeof(Tail) + 15) / 16 * 16) + 1024;
static_assert(kOffQ % 1024 == 0 && kOffP % 1024 == 0 && kOffTail % 16 == 0, "operand alignment");
static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs an SM");

template <bool kFp8Q, bool kVarlen>
__global__ void __launch_bounds__(kThreads, 2)
    stream_attend_kernel(const __grid_constant__ CUtensorMap kv_map, const AttendParams p) {
  constexpr int kSCols = kFp8Q ? kGroup : 2 * kGroup;   // columns of one page's S^T
  constexpr uint32_t kColAcc = 2 * kBatch * kSCols;
  static_assert(kColAcc + 2 * kGroup <= kTmemCols, "tensor memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Tail* tail = reinterpret_cast<Tail*>(smem + kOffTail);
  uint8_t* qtile = smem + kOffQ;
  uint8_t* pbuf = smem + kOffP;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tokens = kVarlen ? p.T : p.B * p.Q;
  const int64_t units = static_cast<int64_t>(tokens) * p.Hkv;   // head by head, its tokens in turn

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&tail->k_full[s], 1);
      mbar_init(&tail->k_empty[s], 1);
      mbar_init(&tail->v_full[s], 1);
      mbar_init(&tail->v_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&tail->s_full[s], 1);
      mbar_init(&tail->s_empty[s], 4 * kCount);
      mbar_init(&tail->item_full[s], 1);
      mbar_init(&tail->item_empty[s], 4 * kCount + 2);
    }
    mbar_init(&tail->p_full, 4 * kCount);
    mbar_init(&tail->o_done, 1);
    mbar_init(&tail->v_land, 1);
    mbar_init(&tail->q_free, 1);
    mbar_init(&tail->finish, 4 + 4 * kCount);
    fence_barrier_init();
    prefetch_tensormap(&kv_map);
  } else if (warp == 1) {
    tc::tmem_alloc(&tail->tmem_base, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_thread_sync();
  __syncthreads();
  tc::fence_after_thread_sync();
  const uint32_t tmem = tail->tmem_base;
  bool ok = true;

  if (warp == 0) {
    // ---- lists, scales, query parts, K tiles --------------------------------------------------------------
    pdl_wait();   // the lists may be the previous kernel's; so may what its readers still need
    int t = 0;    // pages so far
    int i = 0;
    for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x, ++i) {
      const int g = static_cast<int>(u / tokens), tok = static_cast<int>(u - static_cast<int64_t>(g) * tokens);
      int n = lane < kTopK ? p.topk[(static_cast<int64_t>(tok) * p.Hkv + g) * kTopK + lane] : -1;
      int b, j, qlen;
      bool tok_ok = true;
      if constexpr (kVarlen) {
        tok_ok = varlen_token(p.cu_q, p.B, tok, lane, b, j, qlen);
      } else {
        b = tok / p.Q;
        j = tok - b * p.Q;
        qlen = p.Q;
      }
      const int32_t* trow = p.block_table + static_cast<int64_t>(b) * p.S;
      const int L = p.seq_lens[b];
      // a prefill request's tokens are the last qlen of its sequence
      const bool seq_ok = tok_ok && L >= 0 && (L == 0 || (L - 1) / kPage < p.S) &&
                          (!kVarlen || L >= qlen);
      if (!seq_ok && lane == 0) flag_error(p.err, MSA_ERR_SEQ_RANGE);
      const int pos = seq_ok ? L - qlen + j : -1;
      const int cur = pos >= 0 ? pos / kPage : -1;
      bool valid = lane < kTopK && pos >= 0 && n != -1;
      if (valid && (n < 0 || n > cur)) {
        flag_error(p.err, MSA_ERR_TOPK_RANGE);
        valid = false;
      }
      // a block listed again at a later slot is dropped
      const unsigned same = __match_any_sync(0xffffffffu, valid ? n : -2 - lane);
      if (valid && (same & ((1u << lane) - 1u))) {
        flag_error(p.err, MSA_ERR_TOPK_DUP);
        valid = false;
      }
      int page = -1;
      if (valid) {
        page = trow[n];
        if (page < 0 || static_cast<int64_t>(page) >= p.num_blocks) {
          flag_error(p.err, MSA_ERR_PAGE_RANGE);
          valid = false;
        }
      }
      // page order: the current block first, then the others by slot
      const unsigned vm = __ballot_sync(0xffffffffu, valid);
      const bool front = valid && n == cur;
      const unsigned fm = __ballot_sync(0xffffffffu, front);
      const int k = front ? 0 : __popc(vm & ~fm & ((1u << lane) - 1u)) + (fm ? 1 : 0);
      const int np = __popc(vm);
      uint4 raw[8];
      if constexpr (!kFp8Q)
        load_query_rows(p.q + (static_cast<int64_t>(tok) * p.Hq + g * kGroup) * kHeadDim, lane, raw);
      const float2 sc = valid ? load_page_scale(p.kv_scales, page, p.Hkv, g) : make_float2(1.f, 1.f);
      Item* it = &tail->item[i & 1];
      if (i >= 2 && !wait_for(&tail->item_empty[i & 1], ((i >> 1) - 1) & 1)) ok = false;
      if (valid) {
        it->pages[k] = page;
        it->info[k] = page_info(p, sc, n);
      }
      // the query's tile, once the last item's products with it are complete
      if (i >= 1 && !wait_for(&tail->q_free, (i - 1) & 1)) ok = false;
      const int64_t row = static_cast<int64_t>(tok) * p.Hq + g * kGroup;
      float zs;
      if constexpr (kFp8Q) {
        store_query_rows_fp8(p.q8 + row * kHeadDim, 0, qtile, lane);
        zs = p.logit_scale * p.q_scale;
      } else {
        zs = p.logit_scale * exp2i(store_query_e4m3(raw, 0, qtile, qtile + kGroup * 128, lane));
      }
      tc::fence_proxy_async_smem();   // the tile is read by the tensor core
      if (lane == 0) {
        it->n_pages = np;
        it->pos = pos;
        it->current = fm != 0;
        it->zs = zs;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&tail->item_full[i & 1]);
      for (int x = 0; x < np && ok; ++x, ++t) {
        const int s = t % kSlots;
        if (t >= kSlots && !wait_for(&tail->k_empty[s], ((t / kSlots) - 1) & 1)) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&tail->k_full[s], kHalfTile);
          tma_load_2d(smem + s * kHalfTile, &kv_map, 0, (it->pages[x] * p.Hkv + g) * kPage,
                      &tail->k_full[s]);
        }
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    if (lane == 0) {
      if (!ok) flag_error(p.err, MSA_ERR_TIMEOUT);
      // the loads still in flight land before shared memory can be released
      for (int x = max(0, t - kSlots); x < t; ++x)
        (void)wait_for(&tail->k_full[x % kSlots], (x / kSlots) & 1);
      mbar_arrive(&tail->finish);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---- S^T = K Q^T -----------------------------------------------------------------------------
    if (lane == 0) {
      const uint64_t a0 = tc::sw128_kmajor_desc(smem_u32(smem));
      const uint64_t bq = tc::sw128_kmajor_desc(smem_u32(qtile));
      constexpr uint32_t idesc = tc::idesc_e4m3_f32(128, kSCols);
      int t = 0, nb = 0, i = 0;   // pages, batches, items so far
      for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x, ++i) {
        ok = wait_for(&tail->item_full[i & 1], (i >> 1) & 1);
        const int np = ok ? tail->item[i & 1].n_pages : 0;
        for (int x = 0; x < np && ok; x += kBatch, ++nb) {
          const int buf = nb & 1;
          ok = nb < 2 || wait_for(&tail->s_empty[buf], ((nb >> 1) - 1) & 1);
          for (int y = x; y < min(x + kBatch, np) && ok; ++y, ++t) {
            const int s = t % kSlots;
            ok = wait_for(&tail->k_full[s], (t / kSlots) & 1);
            if (!ok) break;
            tc::fence_after_thread_sync();
            const uint64_t a = a0 + static_cast<uint64_t>(s) * (kHalfTile >> 4);
            const uint32_t d = tmem + kSCols * (kBatch * buf + y - x);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) tc::mma_e4m3(d, a + 2 * ks, bq + 2 * ks, idesc, ks > 0);
            tc::commit(&tail->k_empty[s]);
          }
          if (ok) tc::commit(&tail->s_full[buf]);
        }
        tc::commit(&tail->q_free);
      }
      if (!ok) flag_error(p.err, MSA_ERR_TIMEOUT);
      tc::commit(&tail->finish);
    }
    __syncwarp();
    // free tensor memory once every role is done with it
    (void)mbar_wait(&tail->finish, 0);
    tc::fence_after_thread_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  } else if (warp == 2) {
    // ---- V tiles -----------------------------------------------------------------------------------
    int t = 0, i = 0, edges = 0;
    for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x, ++i) {
      const int g = static_cast<int>(u / tokens);
      const Item* it = &tail->item[i & 1];
      ok = __all_sync(0xffffffffu, wait_for(&tail->item_full[i & 1], (i >> 1) & 1));
      const int np = ok ? it->n_pages : 0;
      // the first page is the one that may end past the token's position
      const int lim = np > 0 ? it->pos - (it->pos / kPage) * kPage : 0;
      const bool edge = np > 0 && it->current && lim < kPage - 1;
      for (int x = 0; x < np && ok; ++x) {
        const int s = t % kSlots;
        ok = __all_sync(0xffffffffu, t < kSlots || wait_for(&tail->v_empty[s], ((t / kSlots) - 1) & 1));
        if (!ok) break;
        if (lane == 0) {
          uint64_t* full = edge && x == 0 ? &tail->v_land : &tail->v_full[s];
          mbar_arrive_expect_tx(full, kHalfTile);
          tma_load_2d(smem + kOffV + s * kHalfTile, &kv_map, kHeadDim,
                      (it->pages[x] * p.Hkv + g) * kPage, full);
        }
        ++t;
        // (not before the next load is on its way)
        if (edge && (x == 1 || np == 1)) {
          const int s0 = (t - 1 - x) % kSlots;
          ok = __all_sync(0xffffffffu, wait_for(&tail->v_land, edges & 1));
          ++edges;
          if (!ok) break;
          zero_value_rows(smem + kOffV + s0 * kHalfTile, lim, lane);
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tail->v_full[s0]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&tail->item_empty[i & 1]);
    }
    if (lane == 0) {
      if (!ok) flag_error(p.err, MSA_ERR_TIMEOUT);
      for (int x = max(0, t - kSlots); x < t; ++x)
        (void)wait_for(&tail->v_full[x % kSlots], (x / kSlots) & 1);
      pdl_trigger();
      mbar_arrive(&tail->finish);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ---- O^T += V^T P^T ------------------------------------------------------------------------------
    if (lane == 0) {
      const uint64_t a0 = tc::sw128_mnmajor_desc(smem_u32(smem + kOffV));
      const uint64_t b0 = tc::interleave_mnmajor_desc(smem_u32(pbuf), kPBlock, 128);
      constexpr uint32_t idesc = tc::idesc_e4m3_f32_mn(128, 2 * kGroup);
      int t = 0, nb = 0, i = 0;
      uint32_t acc = 0;   // the item has had a product
      for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x, ++i) {
        ok = wait_for(&tail->item_full[i & 1], (i >> 1) & 1);
        const int np = ok ? tail->item[i & 1].n_pages : 0;
        for (int x = 0; x < np && ok; x += kBatch, ++nb) {
          // (read before the wait: behind it, the load cost 7 us of 290)
          bool bad[kBatch];
#pragma unroll
          for (int y = 0; y < kBatch; ++y) bad[y] = tail->item[i & 1].info[(x + y) % kTopK].block < 0;
          ok = wait_for(&tail->p_full, nb & 1);
          if (x == 0) acc = 0;
#pragma unroll
          for (int y1 = 0; y1 < kBatch; ++y1) {
            const int y = x + y1;
            if (y >= np || !ok) break;
            const int s = t % kSlots;
            ok = wait_for(&tail->v_full[s], (t / kSlots) & 1);
            if (!ok) break;
            ++t;
            tc::fence_after_thread_sync();
            const uint64_t a = a0 + static_cast<uint64_t>(s) * (kHalfTile >> 4);
            const uint64_t bp = b0 + static_cast<uint64_t>(((y - x) * kPBuf) >> 4);
            if (!bad[y1]) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                tc::mma_e4m3(tmem + kColAcc, a + 256 * kk, bp + ((4 * kPBlock) >> 4) * kk, idesc, acc);
                acc = 1;
              }
            }
            tc::commit(&tail->v_empty[s]);
          }
          if (ok) tc::commit(&tail->o_done);
        }
        mbar_arrive(&tail->item_empty[i & 1]);
      }
      if (!ok) flag_error(p.err, MSA_ERR_TIMEOUT);
      tc::commit(&tail->finish);
    }
    __syncwarp();
  } else {
    // ---- group gi: kH heads ------------------------------------------------------------------------------
    const int gi = (warp - 4) >> 2;
    const int h0 = kH * gi;
    const int quarter = warp & 3;
    const int key = 32 * quarter + lane;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
    PageSoftmax<1, kSCols, kSCols, kPBuf> sm;
    sm.gi = gi;
    sm.quarter = quarter;
    sm.lane = lane;
    sm.key = key;
    sm.s_addr = lane_addr + h0;
    sm.acc_addr = lane_addr + kColAcc + h0;
    sm.pj = pbuf + (key >> 3) * kPBlock + (key & 7) * 16 + h0;
    sm.mx = tail->mx[gi];
    sm.lsum = tail->lsum[gi];
    sm.ok = true;
    int nb = 0, i = 0;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x, ++i) {
      Item* it = &tail->item[i & 1];
      if (sm.ok) sm.ok = wait_for(&tail->item_full[i & 1], (i >> 1) & 1);
      // a group goes on together: the number of an item's steps, and so of its barriers,
      // is known to all its warps
      if (group_or<1>(gi, !sm.ok)) {
        sm.ok = false;
        break;
      }
      const int np = it->n_pages, pos = it->pos;
      const float zs = it->zs;
      sm.begin();
      for (int x = 0; x < np; x += kBatch, ++nb) {
        const int buf = nb & 1, have = min(kBatch, np - x);
        sm.step(buf, &tail->s_full[buf], (nb >> 1) & 1, &tail->s_empty[buf], &it->info[x], have, zs,
                pos, &tail->o_done, (nb - 1) & 1, nb == 0, &tail->p_full);
      }
      float o[kH];
      sm.finish(np > 0, &tail->o_done, (nb - 1) & 1, o);
      const int g = static_cast<int>(u / tokens), tok = static_cast<int>(u - static_cast<int64_t>(g) * tokens);
      if (sm.ok)
        sm.write(p.out, static_cast<int64_t>(tok) * p.Hq + g * kGroup + h0, p.v_scale, o);
      __syncwarp();
      if (lane == 0) mbar_arrive(&tail->item_empty[i & 1]);
    }
    if (!sm.ok && lane == 0) flag_error(p.err, MSA_ERR_TIMEOUT);
    __syncwarp();
    if (lane == 0) mbar_arrive(&tail->finish);
  }
}

template <bool kFp8Q, bool kVarlen>
cudaError_t launch(const CUtensorMap& kv_map, const AttendParams& p, dim3 grid, cudaStream_t stream,
                   bool pdl) {
  auto* k = stream_attend_kernel<kFp8Q, kVarlen>;
  static std::atomic<unsigned long long> attr_done{0};
  cudaError_t e = once_per_device(attr_done, [&] {
    cudaError_t r = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (r != cudaSuccess) return r;
    return cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout,
                                static_cast<int>(cudaSharedmemCarveoutMaxShared));
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(k, grid, dim3(kThreads), kSmemBytes, stream, pdl, kv_map, p);
}

}  // namespace

cudaError_t launch_attend_stream(const CUtensorMap& kv_map, const AttendParams& p,
                                 cudaStream_t stream, bool pdl) {
  const int64_t units = static_cast<int64_t>(p.cu_q ? p.T : p.B * p.Q) * p.Hkv;
  const int64_t slots = 2 * static_cast<int64_t>(p.sms);
  const dim3 grid(static_cast<unsigned>(units < slots ? units : slots));
  if (p.cu_q)
    return p.q8 ? launch<true, true>(kv_map, p, grid, stream, pdl)
                : launch<false, true>(kv_map, p, grid, stream, pdl);
  return p.q8 ? launch<true, false>(kv_map, p, grid, stream, pdl)
              : launch<false, false>(kv_map, p, grid, stream, pdl);
}

}  // namespace msa
