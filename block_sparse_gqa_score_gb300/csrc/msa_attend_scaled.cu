// msa_attend_scaled.cu -- the attend on a cache with page scales: sparse decode
// and prefill on lists (given, or selected in the prologue), and dense decode.
//
// Operation (msa_*_scaled in include/msa.h): for each query row the keys of its
// listed (dense decode: all) pages up to its position, with K = K8 ks[page] and
// V = V8 vs[page] per KV head; an empty key set gives 0.
//
// The mathematics is msa_page_softmax.cuh's.
//
// Layout: as the attend for one scale per tensor.  One CTA per (tile of kNT
// tokens of one request, KV head, part); the tile's 16 kNT query rows are the N
// of two transposed tensor-core products per page, S^T = K Q^T (the bf16 query
// as exact fp8 hi and lo parts; an fp8 query as it is) and O^T += V^T P^T (P's hi
// and lo parts, N = 32 per token), so that the page's 128 keys, then its 128 value
// dims, fill M, and fp8 pages are operands as stored.  O^T stays in tensor memory
// over all pages.  kNT = 1 (lists, and dense decode of single tokens): two CTAs an
// SM; kNT = 4 (dense decode of two or more tokens a request): one CTA an SM, each
// page loaded once for four tokens.  K and V tiles have rings of their own (three
// or five slots each): a K tile is free once its S^T is there, long before the V
// tile's product.
//   warp 0       page lists, scales, TMA of K tiles
//   warp 1       S^T products (and owns tensor memory)
//   warp 2       TMA of V tiles; sets the value rows that a token does not see to 0
//   warp 3       O^T products
//   warps 4..    softmax and output, four a group: a thread owns one key, a group
//                a token's 16 heads (kNT = 4) or half of them (kNT = 1).  A step
//                takes a page (kNT = 4) or two.
//
// The pages of a short call are cut over the CTAs of a cluster (kNT = 1), which merge
// their parts through distributed shared memory, so that a small batch needs neither
// a workspace nor a second kernel.
//
// What bounds it, measured (64 query heads, 4 KV heads): lists of batch 16, 4 tokens,
// 8k-32k: 24 us, 4.6 TB/s of its pages; start, lists and pages one behind the other, a
// call of 2 rows already takes 9 us.  Dense decode of one token over 262144: 54 us,
// 5.0 TB/s; the first tile is asked for after 4.5 us, behind the assignment.  Dense
// decode of batch 16, 4 tokens, 8k-32k: 97 us, 3.5 TB/s: the softmax warps' chain of
// waits, 1.2 us a page, on the CTA with the most pages (84, the average is 67).
#include <cstddef>

#include "msa_dense_slot.cuh"
#include "msa_device.cuh"
#include "msa_launch.h"
#include "msa_page_softmax.cuh"
#include "msa_select.cuh"
#include "msa_tcgen05.cuh"

namespace msa {

namespace {

using namespace paged;

constexpr int kChunk = 32;                    // dense decode: pages looked up at once, one a lane
constexpr int kSelectCap = 8000;              // selector keys in K slots 1 and 2, then its slots
constexpr int kMaxCluster = 8;
constexpr int kTableCopy = 512;               // block-table entries copied to shared memory

enum Mode { kLists, kSelect, kDense };

template <int kNT>
struct Tail {
  static constexpr int kSlots = kNT == 1 ? 3 : 5;   // of the K ring and of the V ring
  static constexpr int kHeads = Groups<kNT>::kHeads, kCount = Groups<kNT>::kCount;
  uint64_t k_full[kSlots];  // TMA -> S^T
  uint64_t k_empty[kSlots]; // S^T -> TMA
  uint64_t v_full[kSlots];  // TMA -> O^T
  uint64_t v_land[2];       // TMA -> warp 2: a V tile with rows that not every token sees
  uint64_t v_edges;         // warp 2 is through with those
  uint64_t v_empty[kSlots]; // O^T -> TMA
  uint64_t s_full[2];       // a batch's S^T ready -> softmax
  uint64_t s_empty[2];      // softmax has read a batch's S^T
  uint64_t p_full;          // a batch's P^T written -> O^T
  uint64_t o_done;          // a batch's O^T complete (the P^T buffer free)
  uint64_t info_full[2];    // a chunk's scales and blocks are in its half of `info`
  uint64_t finish;          // every role done and every product complete
  uint32_t tmem_base;
  int n_pages;
  int edge;                 // list modes: page 0's V tile lands on v_land
  int ok;                   // 0: some softmax warp gave up on a wait
  int pos[kNT];             // token positions, -1: none
  float zs[kNT];            // logit scale (log2 units) times 2^e of each token's query split
  int pages[kTopK];         // list modes: this CTA's pages
  uint32_t nan[kNT][4];     // kNT > 1: value dims with a NaN that the token sees (nan_values)
  PageInfo info[2 * kChunk];
  alignas(16) float mx[kCount][kHeads][4];    // batch maxima by quarter
  alignas(16) float lsum[kCount][kHeads][4];  // running sums by quarter
  float ml[kGroup][2];          // cluster merge: (m, l) of this CTA's part
};
// read and written as float4
static_assert(alignof(Tail<1>) == 16 && offsetof(Tail<1>, mx) % 16 == 0 &&
              offsetof(Tail<1>, lsum) % 16 == 0 && offsetof(Tail<1>, info) % 16 == 0, "float4 access");
static_assert(alignof(Tail<4>) == 16 && offsetof(Tail<4>, mx) % 16 == 0 &&
              offsetof(Tail<4>, lsum) % 16 == 0 && offsetof(Tail<4>, info) % 16 == 0, "float4 access");

// K ring, V ring, query tile, P^T of a batch, Tail.
template <int kNT>
struct Smem {
  static constexpr int kSlots = Tail<kNT>::kSlots;
  static constexpr int kPBlock = 8 * 32 * kNT;   // P^T: 8 keys x (hi, lo) of each token
  static constexpr int kPBuf = kPage * 32 * kNT; // one page's
  static constexpr int kV = kSlots * kHalfTile;
  static constexpr int kQ = 2 * kV;
  static constexpr int kP = kQ + 32 * kNT * 128;
  static constexpr int kTail = kP + Groups<kNT>::kBatch * kPBuf;
  static constexpr int kBytes = kTail + static_cast<int>((sizeof(Tail<kNT>) + 15) / 16 * 16) + 1024;
  static_assert(kQ % 1024 == 0 && kP % 1024 == 0 && kTail % 16 == 0,
                "operand tiles need 1024-byte alignment");
};
static_assert(4 * kSelectCap + 4 * kTopK <= 2 * kHalfTile && Smem<1>::kSlots >= 3,
              "selector scratch fits K slots 1 and 2");
static_assert(2 * (Smem<1>::kBytes + 1024) <= 228 * 1024, "two CTAs an SM");
static_assert(Smem<4>::kBytes <= 227 * 1024, "one CTA an SM");
static_assert(kGroup * kHeadDim * 4 <= Smem<1>::kV, "a CTA's part fits the K ring");
static_assert(4 * kTableCopy <= Groups<1>::kBatch * Smem<1>::kPBuf, "the block-table copy fits the P^T buffer");
static_assert(kChunk % 2 == 0, "a batch's pages are of one chunk");

// Warps 0 and 2 of the list modes' prologue (before the groups use their barriers).
__device__ __forceinline__ void table_barrier() {
  __syncwarp();
  asm volatile("barrier.cta.sync.aligned 1, 64;" ::: "memory");
}

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A 32-bit load from the same place in the shared memory of cluster CTA `rank`.
__device__ __forceinline__ float ld_peer(const float* own, uint32_t rank) {
  float v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %1, %2;\n\t"
      "ld.shared::cluster.f32 %0, [a];\n\t}"
      : "=f"(v)
      : "r"(smem_u32(own)), "r"(rank)
      : "memory");
  return v;
}

// A warp: the value rows first_lim < r <= lim of block `blk`, which the tile's later
// tokens see and the earlier ones do not.  A NaN there would reach the others' columns
// of the product too: it is set to 0, and its dim goes into `nan` of the tokens that see
// the row.  At most three rows; a row's 16-byte chunk c lies at c ^ (row & 7).
template <int kNT>
__device__ __forceinline__ void nan_values(uint8_t* tile, int first_lim, int lim, int blk,
                                           Tail<kNT>* tail, int lane) {
  static_assert(kNT <= 5, "eight lanes a row");
  const int r = first_lim + 1 + (lane >> 3), c = lane & 7;
  if (r < 0 || r > min(lim, kPage - 1)) return;
  uint32_t* w = reinterpret_cast<uint32_t*>(tile + r * 128 + 16 * c);
  uint32_t dims = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t x = w[e], m = __vcmpeq4(x & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
    w[e] = x & ~m;
    dims |= (((m & 0x08040201u) * 0x01010101u) >> 24) << (4 * e);   // a bit a byte
  }
  if (dims == 0) return;
  const int at = c ^ (r & 7);
#pragma unroll
  for (int j = 0; j < kNT; ++j)
    if (tail->pos[j] >= blk * kPage + r) atomicOr(&tail->nan[j][at >> 1], dims << (16 * (at & 1)));
}

// kNT tokens a tile; kCluster: the pages of a part are cut over a cluster's CTAs.
template <int kNT, Mode kMode, bool kFp8Q, bool kVarlen, bool kCluster>
__global__ void __launch_bounds__(Groups<kNT>::kThreads, kNT == 1 ? 2 : 1)
    scaled_attend_kernel(const __grid_constant__ CUtensorMap kv_map, const AttendParams p) {
  using Sm = Smem<kNT>;
  constexpr int kSlots = Sm::kSlots;
  constexpr int kBatch = Groups<kNT>::kBatch;
  // A bf16 query's tile: the hi rows of all tokens, then the lo rows.  One token: both
  // in one product, N = 32, added by the softmax.  More: two products into the same
  // columns, which takes the tensor core as long (N = 64 twice for 128 once) and
  // halves what the softmax reads of tensor memory.
  constexpr bool kFold = kNT > 1 && !kFp8Q;
  constexpr int kSCols = kFp8Q || kFold ? kGroup : 2 * kGroup;   // S^T columns of one token
  constexpr int kSN = kSCols * kNT;                        // columns of one page's S^T
  constexpr uint32_t kColAcc = 2 * kBatch * kSN;           // O^T behind two batches of S^T
  constexpr int kTmemCols = kNT == 1 ? 256 : 512;
  static_assert(kColAcc + 2 * kGroup * kNT <= kTmemCols, "tensor memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Tail<kNT>* tail = reinterpret_cast<Tail<kNT>*>(smem + Sm::kTail);
  uint8_t* qtile = smem + Sm::kQ;
  uint8_t* pbuf = smem + Sm::kP;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- this CTA's work: token tile, KV head, part of nparts, cluster rank ----------
  uint32_t cs = 1, rank = 0;
  if constexpr (kCluster) {
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cs));
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  }
  const int cx = kCluster ? static_cast<int>(blockIdx.x / cs) : static_cast<int>(blockIdx.x);
  const int ntiles = kMode == kDense ? (p.Q + kNT - 1) / kNT : 1;
  int b = 0, tok0 = 0, qlen = p.Q, g, split, nsplit;   // tok0: first token of the tile
  int64_t row_tok = 0;                                 // its row among the batch's tokens
  bool tok_ok = true;
  if constexpr (kMode == kDense) {
    const DenseSlot ds = dense_slot<kNT>(p, ntiles, static_cast<int>(kCluster ? gridDim.x / cs : gridDim.x),
                                         cx, lane);
    if (ds.unit < 0) return;   // the whole cluster: no unit left for it
    g = ds.unit % p.Hkv;
    tok0 = kNT * ((ds.unit / p.Hkv) % ntiles);
    b = ds.unit / (p.Hkv * ntiles);
    split = ds.part;
    nsplit = ds.nparts;
    row_tok = static_cast<int64_t>(b) * p.Q + tok0;
  } else {
    g = static_cast<int>(blockIdx.y);
    split = static_cast<int>(blockIdx.z);
    nsplit = p.splits;
    row_tok = cx;
    if constexpr (kVarlen) {
      tok_ok = varlen_token(p.cu_q, p.B, cx, lane, b, tok0, qlen);
    } else {
      b = cx / p.Q;
      tok0 = cx - b * p.Q;
    }
  }
  const int32_t* trow = p.block_table + static_cast<int64_t>(b) * p.S;
  const int ncopy = p.S < kTableCopy ? p.S : kTableCopy;
  int32_t* table_s = reinterpret_cast<int32_t*>(pbuf);   // prologue only
  const int L = p.seq_lens[b];
  // a prefill request's tokens are the last qlen of its sequence
  const bool seq_ok = tok_ok && L >= 0 && (L == 0 || (L - 1) / kPage < p.S) &&
                      (!kVarlen || L >= qlen);
  auto token_pos = [&](int j) -> int {
    return seq_ok && tok0 + j < qlen ? L - qlen + tok0 + j : -1;
  };
  int last_pos = -1, valid_toks = 0;
#pragma unroll
  for (int j = 0; j < kNT; ++j) {
    const int q = token_pos(j);
    if (q >= 0) {
      last_pos = q;
      ++valid_toks;
    }
  }
  // dense decode: this CTA's blocks [lo, hi)
  int lo = 0, hi = 0;
  if constexpr (kMode == kDense) {
    const int nblk = last_pos >= 0 ? last_pos / kPage + 1 : 0;
    const int64_t of = static_cast<int64_t>(nsplit) * cs, at = static_cast<int64_t>(split) * cs + rank;
    lo = static_cast<int>(nblk * at / of);
    hi = static_cast<int>(nblk * (at + 1) / of);
  }

  const int first_pos = last_pos - max(valid_toks - 1, 0);
  // 0 or 1, the number of v_land: block `blk` (at most the last token's) has rows that
  // not every token sees; -1: none
  auto edge_of = [&](int blk) {
    return blk * kPage + kPage - 1 > first_pos ? blk - first_pos / kPage : -1;
  };

  // ---- prologue ----------------------------------------------------------------------
  // warp 0: the lane's page, its block (-1: none) and scales (dense decode: of the next chunk)
  int pg_next = 0, blk_next = -1;
  int slot = lane;   // list modes: the lane's page's place in this CTA's order
  float2 sc_next = make_float2(1.f, 1.f);
  // one lane: the K or V tile of page `page`, the t-th, into its slot
  auto load_k = [&](int t, int page) {
    const int s = t % kSlots;
    mbar_arrive_expect_tx(&tail->k_full[s], kHalfTile);
    tma_load_2d(smem + s * kHalfTile, &kv_map, 0, (page * p.Hkv + g) * kPage, &tail->k_full[s]);
  };
  auto load_v = [&](int t, int page, int e) {   // e: edge_of the page's block
    const int s = t % kSlots;
    uint64_t* full = e < 0 ? &tail->v_full[s] : &tail->v_land[e];
    mbar_arrive_expect_tx(full, kHalfTile);
    tma_load_2d(smem + Sm::kV + s * kHalfTile, &kv_map, kHeadDim, (page * p.Hkv + g) * kPage, full);
  };
  // dense decode: the lane's page of slot t (a bad table entry: page 0 instead,
  // attended by no key), then its scales
  auto look_up = [&](int t) {
    pg_next = 0;
    blk_next = -1;
    if (lo + t < hi) {
      const int pg = trow[lo + t];
      if (pg >= 0 && static_cast<int64_t>(pg) < p.num_blocks) {
        pg_next = pg;
        blk_next = lo + t;
      } else {
        flag_error(p.err, MSA_ERR_PAGE_RANGE);
      }
    }
  };
  auto look_up_scales = [&] {
    sc_next = load_page_scale(p.kv_scales, pg_next, p.Hkv, g);
  };
  auto next_info = [&]() -> PageInfo {
    return blk_next >= 0 ? page_info(p, sc_next, blk_next) : PageInfo{1.f, 0.f, 1.f, -1};
  };
  int n_list = -1;
  if (kMode == kLists && warp == 0) {
    pdl_wait();   // the lists may be the previous kernel's
    if (lane < kTopK) n_list = p.topk[(row_tok * p.Hkv + g) * kTopK + lane];
  }
  if (kMode != kDense && warp == 2) {
    // the request's block-table row (its first kTableCopy entries), all loads in
    // flight while the list is fetched
    int32_t v[kTableCopy / 32];
#pragma unroll
    for (int k = 0; k < kTableCopy / 32; ++k) v[k] = 32 * k + lane < ncopy ? trow[32 * k + lane] : 0;
#pragma unroll
    for (int k = 0; k < kTableCopy / 32; ++k)
      if (32 * k + lane < ncopy) table_s[32 * k + lane] = v[k];
    table_barrier();
  }
  if (warp == 0) {
    if (!seq_ok && lane == 0 && split == 0 && rank == 0) flag_error(p.err, MSA_ERR_SEQ_RANGE);
    const int cur = last_pos >= 0 ? last_pos / kPage : -1;
    const int part = split * static_cast<int>(cs) + static_cast<int>(rank);
    const int nparts = nsplit * static_cast<int>(cs);
    int pre_page = -1;   // select mode: the current block's page, always listed, first
    if (kMode == kSelect && cur >= 0 && part == 0) {
      const int pg = trow[cur];
      if (pg >= 0 && static_cast<int64_t>(pg) < p.num_blocks) pre_page = pg;
    }
    if (lane == 0) {
      const unsigned warps =
          4u * Groups<kNT>::kPerToken * (kNT == 1 ? 1u : static_cast<unsigned>(max(valid_toks, 1)));
      for (int s = 0; s < kSlots; ++s) {
        mbar_init(&tail->k_full[s], 1);
        mbar_init(&tail->k_empty[s], 1);
        mbar_init(&tail->v_full[s], 1);
        mbar_init(&tail->v_empty[s], 1);
      }
      for (int s = 0; s < 2; ++s) {
        mbar_init(&tail->s_full[s], 1);
        mbar_init(&tail->s_empty[s], warps);
        mbar_init(&tail->info_full[s], 1);
      }
      mbar_init(&tail->p_full, warps);
      mbar_init(&tail->o_done, 1);
      mbar_init(&tail->v_land[0], 1);
      mbar_init(&tail->v_land[1], 1);
      mbar_init(&tail->v_edges, 1);
      mbar_init(&tail->finish, 4 + 4 * Groups<kNT>::kCount);
      fence_barrier_init();
      prefetch_tensormap(&kv_map);
      tail->ok = 1;
      tail->edge = 0;
      for (int j = 0; j < kNT; ++j) tail->pos[j] = token_pos(j);
      if (kNT > 1)
        for (int e = 0; e < 4 * kNT; ++e) tail->nan[e >> 2][e & 3] = 0;
      if (pre_page >= 0) {
        load_k(0, pre_page);
        load_v(0, pre_page, edge_of(cur));
      }
    }
    __syncwarp();
    int np = 0;
    if constexpr (kMode == kDense) {
      np = hi - lo;
      look_up(lane);
      look_up_scales();
      if (lane < min(np, kSlots)) {
        load_k(lane, pg_next);
        load_v(lane, pg_next, edge_of(lo + lane));
      }
    } else {
      const int64_t list = (row_tok * p.Hkv + g) * kTopK;
      int n = n_list;
      if constexpr (kMode == kSelect) {
        pdl_wait();   // the scores are the previous kernel's
        bool nan = false;
        uint8_t* scratch = smem + kHalfTile;     // K slots 1 and 2, not yet loaded
        n = last_pos >= 0
                ? select::select_row<16>(p.scores + g * p.s_stride_h + row_tok * p.s_stride_t,
                                         p.s_stride_n, last_pos, lane,
                                         reinterpret_cast<uint32_t*>(scratch), kSelectCap,
                                         reinterpret_cast<int*>(scratch + 4 * kSelectCap), nan)
                : -1;
        if (lane < kTopK && part == 0) p.topk_out[list + lane] = n;
        if (__any_sync(0xffffffffu, nan) && lane == 0) flag_error(p.err, MSA_ERR_SCORE_NAN);
        tc::fence_proxy_async_smem();            // scratch writes before TMA loads into it
        __syncwarp();
      }
      bool valid = lane < kTopK && last_pos >= 0 && n != -1;
      if (valid && (n < 0 || n > cur)) {
        flag_error(p.err, MSA_ERR_TOPK_RANGE);
        valid = false;
      }
      if constexpr (kMode == kLists) {   // a block listed again at a later slot is dropped
        const unsigned same = __match_any_sync(0xffffffffu, valid ? n : -2 - lane);
        if (valid && (same & ((1u << lane) - 1u))) {
          flag_error(p.err, MSA_ERR_TOPK_DUP);
          valid = false;
        }
      }
      int page = -1;
      table_barrier();
      if (valid) {
        page = n < ncopy ? table_s[n] : trow[n];
        if (page < 0 || static_cast<int64_t>(page) >= p.num_blocks) {
          flag_error(p.err, MSA_ERR_PAGE_RANGE);
          valid = false;
        }
      }
      // page order: the current block first, then the others by slot
      const unsigned vm = __ballot_sync(0xffffffffu, valid);
      const bool front = valid && n == cur;
      const unsigned fm = __ballot_sync(0xffffffffu, front);
      const int idx = front ? 0 : __popc(vm & ~fm & ((1u << lane) - 1u)) + (fm ? 1 : 0);
      const bool mine = valid && idx % nparts == part;
      const int k = idx / nparts;
      np = __popc(__ballot_sync(0xffffffffu, mine));
      // the scales are asked for before the pages: behind the first pages of all
      // CTAs they came two microseconds later
      if (mine) {
        pg_next = page;
        blk_next = n;
        slot = k;
        look_up_scales();
        tail->pages[k] = page;
        if (k < kSlots && !(k == 0 && pre_page >= 0)) {
          load_k(k, page);
          load_v(k, page, edge_of(n));
        }
        if (k == 0) tail->edge = edge_of(n) >= 0;
      }
    }
    if (lane == 0) tail->n_pages = np;
  } else if (warp == 1) {
    tc::tmem_alloc(&tail->tmem_base, kTmemCols);
    tc::tmem_relinquish();
  } else if (warp >= 4 && (warp - 4) % (4 * Groups<kNT>::kPerToken) == 0) {
    // token j's query rows (hi, then lo; an fp8 query's as they are)
    const int j = (warp - 4) / (4 * Groups<kNT>::kPerToken);
    if (tok0 + j < qlen || kNT == 1) {
      const int64_t row = (row_tok + j) * p.Hq + g * kGroup;
      if constexpr (kFp8Q) {
        store_query_rows_fp8(p.q8 + row * kHeadDim, kGroup * j, qtile, lane);
        if (lane == 0) tail->zs[j] = p.logit_scale * p.q_scale;
      } else {
        const int e = prepare_query_e4m3(p.q + row * kHeadDim, kGroup * j, qtile,
                                         qtile + kGroup * kNT * 128, lane);
        if (lane == 0) tail->zs[j] = p.logit_scale * exp2i(e);
      }
    } else {
      zero_query_rows(kGroup * j, qtile, lane);
      if (!kFp8Q) zero_query_rows(kGroup * (kNT + j), qtile, lane);
      if (lane == 0) tail->zs[j] = 0.f;
    }
    tc::fence_proxy_async_smem();   // the tile is read by the tensor core
  }
  if (kMode == kDense && warp == 2) look_up(lane);   // the V producer's own pages
  if (kNT > 1 && warp >= 4) {
    // a token that is not there has P = 0: written once, read on every page
    const int j = (warp - 4) / (4 * Groups<kNT>::kPerToken);
    if (token_pos(j) < 0) {
      const int key = 32 * (warp & 3) + lane;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        uint8_t* pk = pbuf + i * Sm::kPBuf + 256 * j + (key >> 3) * Sm::kPBlock + (key & 7) * 16;
        *reinterpret_cast<uint4*>(pk) = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(pk + 128) = make_uint4(0u, 0u, 0u, 0u);
      }
      tc::fence_proxy_async_smem();
    }
  }
  tc::fence_before_thread_sync();
  __syncthreads();
  tc::fence_after_thread_sync();
  const int n_pages = tail->n_pages;
  const uint32_t tmem = tail->tmem_base;

  if (warp < 4) {
    // kNT = 4: 32 registers a thread from these four warps to 8 of each softmax thread
    // (96 at launch; the sum stays): 115 us -> 101 for batch 16 over 8k-32k
    if constexpr (kNT > 1) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 0 || warp == 2) {
      // ---- TMA producers: K tiles (warp 0, with the scales), V tiles (warp 2) ----------------
      const bool is_k = warp == 0;
      uint64_t* full = is_k ? tail->k_full : tail->v_full;
      uint64_t* empty = is_k ? tail->k_empty : tail->v_empty;
      if (is_k) {
        // the first pages' scales, which the softmax waits for, have arrived meanwhile
        if (kMode == kDense || blk_next >= 0) tail->info[slot] = next_info();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tail->info_full[0]);
      }
      int issued = min(n_pages, kSlots);
      bool ok = true;
      // dense decode, chunk by chunk: a chunk's pages are looked up when the one before
      // it begins and their scales when it is half through
      int pg = pg_next;
      // warp 2: tile t, of block blk, has landed on v_land[e]
      auto settle = [&](int e, int t, int blk) {
        bool known = true, attended = true;
        if constexpr (kNT > 1) {
          // (a page that is not attended may be any page in the place of a bad table
          // entry's; its info is there long before its tile's turn)
          known = wait_for(&tail->info_full[(t / kChunk) & 1], (t / (2 * kChunk)) & 1);
          attended = tail->info[t % (2 * kChunk)].block >= 0;
        }
        const bool landed = __all_sync(0xffffffffu, wait_for(&tail->v_land[e], 0) && known);
        ok = ok && landed;
        if (!landed) return;
        uint8_t* tile = smem + Sm::kV + t % kSlots * kHalfTile;
        if (kNT > 1 && attended)
          nan_values(tile, first_pos - blk * kPage, last_pos - blk * kPage, blk, tail, lane);
        zero_value_rows(tile, last_pos - blk * kPage, lane);
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tail->v_full[t % kSlots]);
      };
      if (kMode != kDense && !is_k && tail->edge) settle(0, 0, last_pos / kPage);
      if (kMode == kDense && kChunk < n_pages) look_up(kChunk + lane);
      for (int t = kSlots; t < n_pages && ok; ++t) {
        int page;
        if constexpr (kMode == kDense) {
          if (is_k && t % kChunk == kChunk / 2) look_up_scales();
          if (t % kChunk == 0) {
            pg = pg_next;
            if (is_k) {
              // its half of `info` was last read two chunks ago: the K slots passed on
              // since say that the softmax is past it
              tail->info[t % (2 * kChunk) + lane] = next_info();
              __syncwarp();
              if (lane == 0) mbar_arrive(&tail->info_full[(t / kChunk) & 1]);
            }
            if (t + kChunk < n_pages) look_up(t + kChunk + lane);
          }
          page = __shfl_sync(0xffffffffu, pg, t % kChunk);
        } else {
          page = tail->pages[t];
        }
        if (!wait_for(&empty[t % kSlots], ((t / kSlots) - 1) & 1)) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
          if (lane == 0) {
            if (is_k) load_k(t, page);
            else load_v(t, page, kMode == kDense ? edge_of(lo + t) : -1);
          }
          issued = t + 1;
        }
      }
      if (kMode == kDense && !is_k) {
        // the last tiles, all loads of this CTA on their way
        for (int e = 0; e < 2; ++e) {
          const int blk = first_pos / kPage + e, t = blk - lo;
          if (t >= 0 && t < issued && edge_of(blk) == e) settle(e, t, blk);
        }
      }
      if (lane == 0) {
        if (kNT > 1 && !is_k) mbar_arrive(&tail->v_edges);
        if (!ok) flag_error(p.err, MSA_ERR_TIMEOUT);
        // the loads still in flight land before shared memory can be released
        for (int t = max(0, issued - kSlots); t < issued; ++t)
          (void)wait_for(&full[t % kSlots], (t / kSlots) & 1);
        if (!is_k) pdl_trigger();
        mbar_arrive(&tail->finish);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---- S^T = K Q^T, a batch of pages a buffer --------------------------------------------
      if (lane == 0) {
        const uint64_t a0 = tc::sw128_kmajor_desc(smem_u32(smem));
        const uint64_t bq = tc::sw128_kmajor_desc(smem_u32(qtile));
        constexpr uint32_t idesc = tc::idesc_e4m3_f32(128, kSN);
        bool ok = true;
        for (int t0 = 0, n = 0; t0 < n_pages && ok; t0 += kBatch, ++n) {
          const int buf = n & 1;
          ok = n < 2 || wait_for(&tail->s_empty[buf], ((n >> 1) - 1) & 1);
          for (int t = t0; t < min(t0 + kBatch, n_pages) && ok; ++t) {
            const int s = t % kSlots;
            ok = wait_for(&tail->k_full[s], (t / kSlots) & 1);
            if (!ok) break;
            tc::fence_after_thread_sync();
            const uint64_t a = a0 + static_cast<uint64_t>(s) * (kHalfTile >> 4);
            const uint32_t d = tmem + kSN * (kBatch * buf + t - t0);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) tc::mma_e4m3(d, a + 2 * ks, bq + 2 * ks, idesc, ks > 0);
            if constexpr (kFold) {
              constexpr uint64_t kLo = (kGroup * kNT * 128) >> 4;   // the lo rows
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                tc::mma_e4m3(d, a + 2 * ks, bq + kLo + 2 * ks, idesc, 1);
            }
            tc::commit(&tail->k_empty[s]);
          }
          if (ok) tc::commit(&tail->s_full[buf]);
        }
        if (!ok) flag_error(p.err, MSA_ERR_TIMEOUT);
        tc::commit(&tail->finish);
      }
      __syncwarp();
      // free tensor memory once every role is done with it
      (void)mbar_wait(&tail->finish, 0);
      tc::fence_after_thread_sync();
      tc::tmem_dealloc(tmem, kTmemCols);
    } else {
      // ---- O^T += V^T P^T ----------------------------------------------------------------------
      if (lane == 0) {
        const uint64_t a0 = tc::sw128_mnmajor_desc(smem_u32(smem + Sm::kV));
        // B: each token's 16 hi heads, then its 16 lo ones 128 bytes further; 8-key
        // blocks kPBlock apart
        const uint64_t b0 = tc::interleave_mnmajor_desc(smem_u32(pbuf), Sm::kPBlock, 128);
        constexpr uint32_t idesc = tc::idesc_e4m3_f32_mn(128, 32 * kNT);
        bool ok = true;
        uint32_t acc = 0;   // there has been a product
        for (int t0 = 0, n = 0; t0 < n_pages && ok; t0 += kBatch, ++n) {
          // pages of bad scales have no product (read before the wait for P)
          if (t0 % kChunk == 0) ok = wait_for(&tail->info_full[(t0 / kChunk) & 1], (t0 / (2 * kChunk)) & 1);
          bool bad[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) bad[i] = tail->info[(t0 + i) % (2 * kChunk)].block < 0;
          ok = ok && wait_for(&tail->p_full, n & 1);
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int t = t0 + i, s = t % kSlots;
            if (t >= n_pages || !ok) break;
            ok = wait_for(&tail->v_full[s], (t / kSlots) & 1);
            if (!ok) break;
            tc::fence_after_thread_sync();
            const uint64_t a = a0 + static_cast<uint64_t>(s) * (kHalfTile >> 4);
            const uint64_t bp = b0 + static_cast<uint64_t>(((t - t0) * Sm::kPBuf) >> 4);
            if (!bad[i]) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                tc::mma_e4m3(tmem + kColAcc, a + 256 * kk, bp + ((4 * Sm::kPBlock) >> 4) * kk, idesc, acc);
                acc = 1;
              }
            }
            tc::commit(&tail->v_empty[s]);
          }
          if (ok) tc::commit(&tail->o_done);
        }
        if (!ok) flag_error(p.err, MSA_ERR_TIMEOUT);
        tc::commit(&tail->finish);
      }
      __syncwarp();
    }
  } else {
    if constexpr (kNT > 1) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    // ---- group gi: kH heads of token j ------------------------------------------------------
    constexpr int kH = Groups<kNT>::kHeads;
    const int gi = (warp - 4) >> 2;
    const int j = gi / Groups<kNT>::kPerToken;
    const int h0 = kH * (gi % Groups<kNT>::kPerToken);   // the group's first head
    const int quarter = warp & 3;
    const int key = 32 * quarter + lane;   // key of the page; value dim at the end
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
    PageSoftmax<kNT, kSCols, kSN, Sm::kPBuf> sm;
    sm.gi = gi;
    sm.quarter = quarter;
    sm.lane = lane;
    sm.key = key;
    sm.s_addr = lane_addr + kSCols * j + h0;
    sm.acc_addr = lane_addr + kColAcc + 32 * j + h0;
    sm.pj = pbuf + 256 * j + (key >> 3) * Sm::kPBlock + (key & 7) * 16 + h0;
    sm.mx = tail->mx[gi];
    sm.lsum = tail->lsum[gi];
    sm.ok = true;
    sm.begin();
    const float zs = tail->zs[j];
    const int pos = tail->pos[j];
    const int n_steps = pos >= 0 ? (n_pages + kBatch - 1) / kBatch : 0;
    for (int n = 0; n < n_steps; ++n) {
      const int buf = n & 1, k0 = kBatch * n;
      // the pages' scales and blocks
      if (k0 % kChunk == 0 && sm.ok)
        sm.ok = wait_for(&tail->info_full[(k0 / kChunk) & 1], (k0 / (2 * kChunk)) & 1);
      sm.step(buf, &tail->s_full[buf], (n >> 1) & 1, &tail->s_empty[buf],
              &tail->info[k0 % (2 * kChunk)], min(kBatch, n_pages - k0), zs, pos, &tail->o_done,
              (n - 1) & 1, n == 0, &tail->p_full);
    }

    // ---- output: this thread's value dim of each head ---------------------------------------
    float o[kH];
    sm.finish(n_steps > 0, &tail->o_done, (n_steps - 1) & 1, o);
    const float lv = sm.lv;
    float (&l)[kH] = sm.l;
    float (&nl)[kH] = sm.nl;
    if (!sm.ok && lane == 0) {
      flag_error(p.err, MSA_ERR_TIMEOUT);
      tail->ok = 0;
    }
    group_sync<kNT>(gi);   // tail->ok
    if constexpr (kNT > 1) {
      if (sm.ok) sm.ok = wait_for(&tail->v_edges, 0);   // nan
      if (tail->nan[j][key >> 5] >> lane & 1) {
#pragma unroll
        for (int h = 0; h < kH; ++h) o[h] = __uint_as_float(0x7FFFFFFFu);
      }
    }
    const int64_t row0 = (row_tok + j) * p.Hq + g * kGroup;
    const int64_t rows = static_cast<int64_t>(kVarlen ? p.T : p.B * p.Q) * p.Hq;
    const int64_t base = static_cast<int64_t>(split) * rows + row0;
    if (kMode == kDense) pdl_wait();   // the outputs may be the previous kernel's inputs
    if constexpr (kCluster) {
      // this CTA's part into its K ring (every load has landed and every product is
      // complete), then each CTA merges its share of the heads
      float* po = reinterpret_cast<float*>(smem);
#pragma unroll
      for (int h = 0; h < kH; ++h) po[(h0 + h) * kHeadDim + key] = l[h] > 0.f ? o[h] : 0.f;
#pragma unroll
      for (int h = 0; h < kH; ++h)
        if (h == key) {
          tail->ml[h0 + h][0] = lv - nl[h];   // M
          tail->ml[h0 + h][1] = tail->ok ? l[h] : 0.f;
        }
    } else if (tail->ok && (kNT == 1 || tok0 + j < qlen)) {
      if (p.splits == 1) {
        sm.write(p.out, row0 + h0, p.v_scale, o);
      } else {
#pragma unroll
        for (int h = 0; h < kH; ++h)
          p.part_o[(base + h0 + h) * kHeadDim + key] = o[h] * p.v_scale;
#pragma unroll
        for (int h = 0; h < kH; ++h)
          if (h == key) {
            p.part_ml[(base + h0 + h) * 2] = lv - nl[h];
            p.part_ml[(base + h0 + h) * 2 + 1] = l[h];
          }
      }
    }
    if (kMode == kDense && !kCluster && split == 0 && key < kH && (kNT == 1 || tok0 + j < qlen)) {
      // a unit cut into fewer ranges than the workspace's parts marks the rest empty
      for (int s2 = nsplit; s2 < p.splits; ++s2) {
        const int64_t at = (static_cast<int64_t>(s2) * rows + row0 + h0 + key) * 2;
        p.part_ml[at] = -INFINITY;
        p.part_ml[at + 1] = 0.f;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&tail->finish);
    if constexpr (kCluster) {
      cluster_sync();
      const int per = kGroup / static_cast<int>(cs);   // heads of this CTA, the groups in turn
      for (int i = gi; i < per; i += Groups<kNT>::kCount) {
        const int h = per * static_cast<int>(rank) + i;
        float m[kMaxCluster], lr[kMaxCluster], v[kMaxCluster];
        float M = -INFINITY;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          m[r] = -INFINITY;
          lr[r] = v[r] = 0.f;
          if (r < static_cast<int>(cs)) {
            m[r] = ld_peer(&tail->ml[h][0], r);
            lr[r] = ld_peer(&tail->ml[h][1], r);
            v[r] = ld_peer(reinterpret_cast<float*>(smem) + h * kHeadDim + key, r);
          }
          if (lr[r] > 0.f) M = fmaxf(M, m[r]);
        }
        float den = 0.f, acc = 0.f;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          const float w = lr[r] > 0.f ? ex2(m[r] - M) : 0.f;
          den = fmaf(w, lr[r], den);
          acc = fmaf(w, v[r], acc);
        }
        if (p.splits == 1) {
          const float rr = den > 0.f ? acc * (p.v_scale / den) : 0.f;
          p.out[(row0 + h) * kHeadDim + key] = static_cast<uint16_t>(f32_to_bf16_bits(rr));
        } else {
          p.part_o[(base + h) * kHeadDim + key] = acc * p.v_scale;
          if (key == 0) {
            p.part_ml[(base + h) * 2] = M;
            p.part_ml[(base + h) * 2 + 1] = den;
          }
          if (kMode == kDense && split == 0 && key == 0)
            for (int s2 = nsplit; s2 < p.splits; ++s2) {
              p.part_ml[(static_cast<int64_t>(s2) * rows + row0 + h) * 2] = -INFINITY;
              p.part_ml[(static_cast<int64_t>(s2) * rows + row0 + h) * 2 + 1] = 0.f;
            }
        }
      }
      cluster_sync();   // no CTA ends while another reads its part
    }
  }
  if constexpr (kCluster) {
    if (warp < 4) {
      cluster_sync();
      cluster_sync();
    }
  }
}

}  // namespace

namespace {

template <int kNT, Mode kMode, bool kFp8Q, bool kVarlen, bool kCluster>
cudaError_t launch(const CUtensorMap& kv_map, const AttendParams& p, dim3 grid, int cs,
                   cudaStream_t stream, bool pdl) {
  auto* k = scaled_attend_kernel<kNT, kMode, kFp8Q, kVarlen, kCluster>;
  static std::atomic<unsigned long long> attr_done{0};
  cudaError_t e = once_per_device(attr_done, [&] {
    cudaError_t r = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Smem<kNT>::kBytes);
    if (r != cudaSuccess) return r;
    // all of the unified L1 / shared storage as shared memory: two CTAs per SM
    return cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout,
                                static_cast<int>(cudaSharedmemCarveoutMaxShared));
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(Groups<kNT>::kThreads);
  cfg.dynamicSmemBytes = Smem<kNT>::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  if (kCluster) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = static_cast<unsigned>(cs);
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs++].val.clusterDim.z = 1;
  }
  if (pdl) {   // as launch_pdl
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  return cudaLaunchKernelEx(&cfg, k, kv_map, p);
}

template <Mode kMode, bool kFp8Q>
cudaError_t launch_lists(const CUtensorMap& kv_map, const AttendParams& p, dim3 grid, int cs,
                         cudaStream_t stream, bool pdl) {
  if (p.cu_q)
    return cs > 1 ? launch<1, kMode, kFp8Q, true, true>(kv_map, p, grid, cs, stream, pdl)
                  : launch<1, kMode, kFp8Q, true, false>(kv_map, p, grid, cs, stream, pdl);
  return cs > 1 ? launch<1, kMode, kFp8Q, false, true>(kv_map, p, grid, cs, stream, pdl)
                : launch<1, kMode, kFp8Q, false, false>(kv_map, p, grid, cs, stream, pdl);
}

template <bool kFp8Q>
cudaError_t launch_dense(const CUtensorMap& kv_map, const AttendParams& p, dim3 grid, int cs,
                         cudaStream_t stream, bool pdl) {
  if (p.Q > 1) return launch<4, kDense, kFp8Q, false, false>(kv_map, p, grid, cs, stream, pdl);
  return cs > 1 ? launch<1, kDense, kFp8Q, false, true>(kv_map, p, grid, cs, stream, pdl)
                : launch<1, kDense, kFp8Q, false, false>(kv_map, p, grid, cs, stream, pdl);
}

}  // namespace

cudaError_t launch_attend_scaled(const CUtensorMap& kv_map, const AttendParams& p,
                                 cudaStream_t stream, bool pdl) {
  const bool dense = p.dense_span > 0;
  const int sms = p.sms;
  const int ntile = p.Q > 1 && dense ? 4 : 1;                  // tokens a tile
  const int64_t slots = ntile == 1 ? 2 * sms : sms;            // CTAs resident at once
  const int tiles = (p.Q + ntile - 1) / ntile;
  const int64_t units = dense ? static_cast<int64_t>(p.B) * tiles * p.Hkv
                              : static_cast<int64_t>(p.cu_q ? p.T : p.B * p.Q) * p.Hkv;
  // The CTAs of a cluster cut a unit's part where that puts more CTAs to use and leaves
  // each a page or more (lists: 16 pages a row).  Clusters count on one CTA an SM: a
  // cluster that has to go second on its SMs starts 3.7 us later, a plain CTA 1.5 us (lists
  // of 32 requests, 4 KV heads: 128 CTAs 20.5 us, 128 clusters of two 24.6; dense decode of
  // 32768 tokens, 4 KV heads: 21.7 against 26.6; of 131072, one KV head: 26.4 against 26.0).
  const int pages = dense ? p.S : kTopK;
  int cs = 1;
  if (ntile == 1 && (dense || p.splits == 1)) {
    int64_t best = 0;
    for (int c = 1; c <= kMaxCluster && c <= pages; c *= 2) {
      const int64_t parts = (c > 1 ? sms : slots) / c / units;   // clusters a unit can have
      const int64_t used = units * c * (parts < p.splits ? parts : p.splits);
      if (used > best) {
        best = used;
        cs = c;
      }
    }
  }
  // rows for more than one wave of CTAs: CTAs that stay, each row's start and end hidden
  // behind others' pages
  if (!dense && !p.scores && p.splits == 1 && units > slots)
    return launch_attend_stream(kv_map, p, stream, pdl);
  dim3 grid;
  if (!dense) {
    grid = dim3(static_cast<unsigned>(units / p.Hkv * cs), p.Hkv, p.splits);
    if (p.scores)
      return p.q8 ? launch_lists<kSelect, true>(kv_map, p, grid, cs, stream, pdl)
                  : launch_lists<kSelect, false>(kv_map, p, grid, cs, stream, pdl);
    return p.q8 ? launch_lists<kLists, true>(kv_map, p, grid, cs, stream, pdl)
                : launch_lists<kLists, false>(kv_map, p, grid, cs, stream, pdl);
  }
  // dense decode: fewer units than slots share the slots out by their blocks
  // (dense_slot), up to `splits` parts a unit; else one part a unit
  if (p.splits > 1 && units < slots && p.B * tiles <= kBalancedTiles)
    grid = dim3(static_cast<unsigned>((cs > 1 ? sms : slots) / cs * cs));
  else
    grid = dim3(static_cast<unsigned>(units * cs), p.splits);
  return p.q8 ? launch_dense<true>(kv_map, p, grid, cs, stream, pdl)
              : launch_dense<false>(kv_map, p, grid, cs, stream, pdl);
}

}  // namespace msa
