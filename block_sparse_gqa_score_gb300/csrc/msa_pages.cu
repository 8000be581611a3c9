// msa_pages.cu -- the cache's pages: the next step's rows of a block table forked,
// reordered, freed and grown (msa_fork_pages), the pages of a pool moved together
// (msa_compact_pages), and the copies of pages that both ask for (msa_copy_pages).
//
// A pool is its counts alone: refs[page] rows hold a page, 0 of them make it free.  Both
// plans are one launch of one cluster of eight CTAs, which share out the counts by page
// ranges; a thread holds a run of neighbouring pages, so that one scan over the CTA and
// the eight CTAs' totals (exchanged through distributed shared memory) rank every free or
// live page in the order of the pages.  The ranks are the whole plan:
//   fork:    the k-th page that the rows need is the k-th free page; the thread that
//            holds that page finds the row by a search in the rows' prefix sums and writes
//            the entry, so there is no list of free pages and no scratch memory.
//   compact: L pages are live; the k-th live page at or past L goes to the k-th hole
//            below L.  Either side of move k is written by the thread that holds the page.
// The order of pages fixes every result; the only atomics are sums of whole numbers.
#include <climits>

#include "msa_device.cuh"
#include "msa_launch.h"

namespace msa {

namespace {

constexpr int kThreads = 1024;
constexpr int kCluster = 8;       // the largest portable cluster

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// The cluster's CTAs have all started, behind the wait: only then may another CTA's shared
// memory be touched.  (Arrived at first thing and waited for just ahead of the first store
// over there, so that it runs beside the reads of the counts.)
__device__ __forceinline__ void cluster_started_arrive() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_started_wait() {
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// All of the cluster's threads: what any of them wrote, to shared or global memory, is
// seen by all behind it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// `v` into the same shared variable of CTA `rank` of the cluster.
__device__ __forceinline__ void store_remote(int* at, unsigned rank, int v) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.b32 [a], %2;\n\t}" ::"r"(smem_u32(at)),
      "r"(rank), "r"(v)
      : "memory");
}

__device__ __forceinline__ int pages_of(int64_t tokens) {
  return static_cast<int>((tokens + kPage - 1) / kPage);
}

// Sum of the threads' values before this thread's; the CTA's sum in `total`.  `part`:
// 33 ints of shared memory, free again once every thread has passed another barrier.
__device__ __forceinline__ int block_scan(int v, int* part, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) part[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = part[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    __syncwarp();
    part[lane] = w;
  }
  __syncthreads();
  total = part[31];
  return x - v + (warp ? part[warp - 1] : 0);
}

struct Shared {
  int scan_a[32], scan_b[32];
  int total[kCluster];      // each CTA's pages counted
  int below;                // compact: live pages below L
};

// ---------------------------------------------------------------------------
// fork

__device__ __forceinline__ int row_tokens(const int32_t* lens, int row, int S, bool& bad) {
  const int L = lens[row];
  if (L >= 0 && (L == 0 || (L - 1) / kPage < S)) return L;
  bad = true;
  return 0;
}

// Row b of the next step: n tokens are taken over from the parent row.
struct ForkRow {
  int parent;     // -1: none
  int n, grow;
  __device__ __forceinline__ bool copied(const int* first, int b) const {
    // the parent's begun page goes to another row or stays with other holders: entry held()
    // is a copy
    return n % kPage != 0 && first[parent] != b;
  }
  // entries taken over from the parent (all but a page to be copied), and entries of the row
  __device__ __forceinline__ int held(bool copy) const { return pages_of(n) - (copy ? 1 : 0); }
  __device__ __forceinline__ int want() const { return pages_of(static_cast<int64_t>(n) + grow); }
};

__device__ __forceinline__ ForkRow load_fork_row(const ForkParams& p, int b, unsigned& bad) {
  ForkRow r{p.parents[b], 0, p.grow ? p.grow[b] : 0};
  if (r.parent < -1 || r.parent >= p.B) {
    bad |= MSA_ERR_ROW_RANGE;
    return ForkRow{-1, 0, 0};
  }
  bool seq = false;
  if (r.parent >= 0) r.n = row_tokens(p.lens, r.parent, p.S, seq);
  if (r.grow < 0 || r.n + static_cast<int64_t>(r.grow) > static_cast<int64_t>(p.S) * kPage ||
      r.n > INT_MAX - r.grow) {
    seq = true;
    r.grow = 0;
  }
  if (seq) bad |= MSA_ERR_SEQ_RANGE;
  return r;
}

__global__ void __launch_bounds__(kThreads) __cluster_dims__(kCluster)
    fork_kernel(const ForkParams p) {
  extern __shared__ int dyn[];
  __shared__ Shared sh;
  int* first = dyn;                 // [B] the lowest row that follows this one; -1: its begun
                                    // page has other holders, and is taken over by nobody
  int* children = first + p.B;      // [B] how many do
  int* before = children + p.B;     // [rows + 1] pages that the rows before need
  ForkRow* facts = reinterpret_cast<ForkRow*>(before + p.rows + 1);   // [rows]
  const int tid = threadIdx.x, lane = tid & 31;
  const unsigned cta = cluster_rank();
  cluster_started_arrive();
  pdl_trigger();
  pdl_wait();

  // a run of `run` neighbouring pages a thread
  const int threads = kCluster * kThreads;
  const int run = (p.num_blocks - 1) / threads + 1;
  const int64_t lo64 = static_cast<int64_t>(cta * kThreads + tid) * run;
  const int lo = static_cast<int>(min(lo64, static_cast<int64_t>(p.num_blocks)));
  const int hi = static_cast<int>(min(lo64 + run, static_cast<int64_t>(p.num_blocks)));
  int mine = 0;
  for (int i = lo; i < hi; ++i) {
    const int r = p.refs[i];
    p.refs_out[i] = r;
    mine += r == 0;
  }
  // (the last threads' first: with few rows they are not the threads that load the new rows)
  for (int b = kThreads - 1 - tid; b < p.B; b += kThreads) {
    bool seq = false;
    const int n = row_tokens(p.lens, b, p.S, seq);
    bool others = false;
    if (n % kPage != 0) {
      const int page = p.table[static_cast<int64_t>(b) * p.S + n / kPage];
      others = page >= 0 && page < p.num_blocks && p.refs[page] > 1;
    }
    first[b] = others ? -1 : INT_MAX;
    children[b] = 0;
  }
  // `each` neighbouring rows a thread
  unsigned bad = 0;
  const int each = (p.rows + kThreads - 1) / kThreads;
  const int r0 = min(tid * each, p.rows), r1 = min(r0 + each, p.rows);
  for (int b = r0; b < r1; ++b) facts[b] = load_fork_row(p, b, bad);
  int cta_free;
  const int at = block_scan(mine, sh.scan_a, cta_free);
  cluster_started_wait();
  if (tid < kCluster) store_remote(&sh.total[cta], tid, cta_free);
  for (int b = r0; b < r1; ++b) {
    const int q = facts[b].parent;
    if (q >= 0) {
      atomicMin(&first[q], b);
      atomicAdd(&children[q], 1);
    }
  }
  __syncthreads();
  int need = 0;
  for (int b = r0; b < r1; ++b) {
    const ForkRow r = facts[b];
    before[b] = need;
    need += r.want() - r.held(r.copied(first, b));
  }
  int total_need;
  const int sum = block_scan(need, sh.scan_b, total_need);
  for (int b = r0; b < r1; ++b) before[b] += sum;
  if (tid == 0) before[p.rows] = total_need;
  // the totals of all CTAs, and refs_out as a copy of refs, before the changes to it
  cluster_sync();
  int free_before = at, total_free = 0;
#pragma unroll
  for (unsigned c = 0; c < kCluster; ++c) {
    if (c < cta) free_before += sh.total[c];
    total_free += sh.total[c];
  }
  const bool fits = total_need <= total_free;
  if (!fits) bad |= MSA_ERR_NO_PAGES;

  // the free pages that are needed, to their rows
  if (fits && mine > 0 && free_before < total_need) {
    int k = free_before;
    for (int i = lo; i < hi && k < total_need; ++i) {
      if (p.refs[i] != 0) continue;
      int x = 0, y = p.rows;        // the last row whose pages begin at or before k
      while (y - x > 1) {
        const int m = (x + y) >> 1;
        if (before[m] <= k) x = m;
        else y = m;
      }
      const ForkRow r = facts[x];
      const bool copy = r.copied(first, x);
      const int e = r.held(copy) + k - before[x];
      p.table_out[static_cast<int64_t>(x) * p.S + e] = i;
      p.refs_out[i] = 1;
      if (copy && k == before[x]) {
        int src = p.table[static_cast<int64_t>(r.parent) * p.S + e], tokens = r.n % kPage, dst = i;
        if (src < 0 || src >= p.num_blocks) {
          bad |= MSA_ERR_PAGE_RANGE;
          src = dst = -1;
          tokens = 0;
        }
        p.copies[3 * static_cast<int64_t>(x)] = src;
        p.copies[3 * static_cast<int64_t>(x) + 1] = dst;
        p.copies[3 * static_cast<int64_t>(x) + 2] = tokens;
      }
      ++k;
    }
  }
  // the rows: what they take over, and -1 behind their last page; a warp a row
  const int warps = threads / 32, warp = static_cast<int>(cta) * (kThreads / 32) + tid / 32;
  for (int b = warp; b < p.rows; b += warps) {
    const ForkRow r = facts[b];
    const bool copy = r.copied(first, b);
    int32_t* to = p.table_out + static_cast<int64_t>(b) * p.S;
    const int32_t* from = p.table + static_cast<int64_t>(max(r.parent, 0)) * p.S;
    const int held = fits ? r.held(copy) : 0, want = fits ? r.want() : 0;
    for (int e = lane; e < p.S; e += 32) {
      if (e >= held && e < want) continue;
      int page = -1;
      if (e < held) {
        page = from[e];
        if (page < 0 || page >= p.num_blocks) {
          bad |= MSA_ERR_PAGE_RANGE;
          page = -1;
        }
      }
      to[e] = page;
    }
    if (lane == 0) p.lens_out[b] = fits ? r.n + r.grow : 0;
    if (lane < 3 && !(fits && copy)) p.copies[3 * static_cast<int64_t>(b) + lane] = lane < 2 ? -1 : 0;
  }
  // the counts of the pages that were held: one row fewer, children[b] more
  for (int b = warp; b < p.B && fits; b += warps) {
    bool seq = false;
    const int n = row_tokens(p.lens, b, p.S, seq), c = children[b];
    if (seq) bad |= MSA_ERR_SEQ_RANGE;
    const int32_t* from = p.table + static_cast<int64_t>(b) * p.S;
    const int all = pages_of(n), full = n / kPage;
    for (int e = lane; e < all; e += 32) {
      // the begun page goes to one child, or to none
      const int more = e < full ? c - 1 : (first[b] < 0 ? 0 : min(c, 1)) - 1;
      if (more == 0) continue;
      const int page = from[e];
      if (page < 0 || page >= p.num_blocks) {
        bad |= MSA_ERR_PAGE_RANGE;
        continue;
      }
      if (p.refs[page] < 1) bad |= MSA_ERR_REFS;
      atomicAdd(&p.refs_out[page], more);
    }
  }
  bad = __reduce_or_sync(0xffffffffu, bad);
  if (bad && lane == 0) flag_error(p.err, bad);
}

// ---------------------------------------------------------------------------
// compact

__global__ void __launch_bounds__(kThreads) __cluster_dims__(kCluster)
    compact_kernel(const CompactParams p) {
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31;
  const unsigned cta = cluster_rank();
  cluster_started_arrive();
  pdl_trigger();
  pdl_wait();
  const int threads = kCluster * kThreads;
  const int run = (p.num_blocks - 1) / threads + 1;
  const int64_t lo64 = static_cast<int64_t>(cta * kThreads + tid) * run;
  const int lo = static_cast<int>(min(lo64, static_cast<int64_t>(p.num_blocks)));
  const int hi = static_cast<int>(min(lo64 + run, static_cast<int64_t>(p.num_blocks)));
  int mine = 0;
  for (int i = lo; i < hi; ++i) mine += p.refs[i] != 0;
  int cta_live;
  const int at = block_scan(mine, sh.scan_a, cta_live);
  cluster_started_wait();
  if (tid < kCluster) store_remote(&sh.total[cta], tid, cta_live);
  if (tid == 0) sh.below = 0;
  cluster_sync();
  int before = at, live = 0;     // live pages before this thread's, and in all
#pragma unroll
  for (unsigned c = 0; c < kCluster; ++c) {
    if (c < cta) before += sh.total[c];
    live += sh.total[c];
  }
  if (lo <= live && live < hi) {
    int below = before;
    for (int i = lo; i < live; ++i) below += p.refs[i] != 0;
    for (unsigned c = 0; c < kCluster; ++c) store_remote(&sh.below, c, below);
  }
  cluster_sync();
  const int below = live < p.num_blocks ? sh.below : live;
  const int moves = live - below;
  // either side of each move; refs_out of a page that moves holds its move's number
  int rank = before;
  for (int i = lo; i < hi; ++i) {
    const int r = p.refs[i];
    if (i < live) {
      if (r != 0) {
        p.refs_out[i] = r;
      } else {
        int32_t* c = p.copies + 3 * static_cast<int64_t>(i - rank);
        c[1] = i;
        c[2] = kPage;
      }
    } else {
      p.refs_out[i] = r != 0 ? rank - below : 0;
      if (r != 0) p.copies[3 * static_cast<int64_t>(rank - below)] = i;
    }
    rank += r != 0;
  }
  const int t = static_cast<int>(cta) * kThreads + tid;
  for (int k = moves + t; k < p.num_blocks / 2; k += threads) {
    int32_t* c = p.copies + 3 * static_cast<int64_t>(k);
    c[0] = c[1] = -1;
    c[2] = 0;
  }
  cluster_sync();
  // (what is read back is checked: outputs that share memory must not lead out of the pool)
  unsigned bad = 0;
  for (int k = t; k < moves; k += threads) {
    const int32_t* c = p.copies + 3 * static_cast<int64_t>(k);
    const int src = __ldcg(c), dst = __ldcg(c + 1);
    if (src >= 0 && src < p.num_blocks && dst >= 0 && dst < p.num_blocks) p.refs_out[dst] = p.refs[src];
    else bad |= MSA_ERR_REFS;
  }
  const int warps = threads / 32;
  for (int b = t / 32; b < p.B; b += warps) {
    bool seq = false;
    const int n = pages_of(row_tokens(p.lens, b, p.S, seq));
    if (seq) bad |= MSA_ERR_SEQ_RANGE;
    const int64_t row = static_cast<int64_t>(b) * p.S;
    for (int e = lane; e < p.S; e += 32) {
      int page = -1;
      if (e < n) {
        page = p.table[row + e];
        if (page < 0 || page >= p.num_blocks) {
          bad |= MSA_ERR_PAGE_RANGE;
          page = -1;
        } else if (p.refs[page] == 0) {   // held, yet free: its place may have been given away
          bad |= MSA_ERR_REFS;
          page = -1;
        } else if (page >= live) {
          const int k = __ldcg(p.refs_out + page);
          if (k >= 0 && k < moves) {
            page = __ldcg(p.copies + 3 * static_cast<int64_t>(k) + 1);
          } else {
            bad |= MSA_ERR_REFS;
            page = -1;
          }
        }
      }
      p.table_out[row + e] = page;
    }
  }
  bad = __reduce_or_sync(0xffffffffu, bad);
  if (bad && lane == 0) flag_error(p.err, bad);
  cluster_sync();
  for (int i = max(lo, live); i < hi; ++i) p.refs_out[i] = 0;
}

// ---------------------------------------------------------------------------
// copies

constexpr int kCopyThreads = 256;
constexpr int kFlight = 8;        // 16-byte loads a thread has in flight

// bytes [from, to) of one run of bytes, a warp's lanes side by side
template <typename V>
__device__ __forceinline__ void copy_span(uint8_t* dst, const uint8_t* src, int64_t bytes, int t,
                                          int threads) {
  const int64_t n = bytes / static_cast<int64_t>(sizeof(V));
  const V* s = reinterpret_cast<const V*>(src);
  V* d = reinterpret_cast<V*>(dst);
  int64_t i = t;
  for (; i + (kFlight - 1) * static_cast<int64_t>(threads) < n; i += kFlight * static_cast<int64_t>(threads)) {
    V v[kFlight];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) v[k] = __ldcs(s + i + k * static_cast<int64_t>(threads));
#pragma unroll
    for (int k = 0; k < kFlight; ++k) d[i + k * static_cast<int64_t>(threads)] = v[k];
  }
  for (; i < n; i += threads) d[i] = s[i];
}

// Copy blockIdx.x + k gridDim.x; blockIdx.y of gridDim.y shares of it, by units.
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyParams p) {
  pdl_trigger();
  pdl_wait();
  for (int64_t k = blockIdx.x; k < p.n; k += gridDim.x) {
    const int src = p.copies[3 * k], dst = p.copies[3 * k + 1];
    const int rows = p.copies[3 * k + 2];
    if (src == -1 && dst == -1) continue;
    if (src < 0 || src >= p.num_blocks || dst < 0 || dst >= p.num_blocks || rows < 0 || rows > kPage) {
      if (threadIdx.x == 0) flag_error(p.err, MSA_ERR_PAGE_RANGE);
      continue;
    }
    if (src == dst || rows == 0) continue;
    int share = 0;
    for (int c = 0; c < p.caches; ++c) {
      const CopyCache& h = p.cache[c];
      const int64_t unit = static_cast<int64_t>(h.rows) * h.row_bytes;
      const uint8_t* s = h.base + src * unit * h.units;
      uint8_t* d = h.base + dst * unit * h.units;
      if (h.rows == 1) {                   // no token rows: the page's bytes, by 4
        if (share++ % gridDim.y == blockIdx.y)
          copy_span<uint32_t>(d, s, unit * h.units, threadIdx.x, kCopyThreads);
        continue;
      }
      for (int u = 0; u < h.units; ++u)
        if (share++ % gridDim.y == blockIdx.y)
          copy_span<uint4>(d + u * unit, s + u * unit, static_cast<int64_t>(rows) * h.row_bytes,
                           threadIdx.x, kCopyThreads);
    }
  }
}

}  // namespace

cudaError_t launch_fork(const ForkParams& p, cudaStream_t stream, bool pdl) {
  const size_t smem = (2 * static_cast<size_t>(p.B) + p.rows + 1) * sizeof(int) + p.rows * sizeof(ForkRow);
  static std::atomic<unsigned long long> attr_done{0};
  const cudaError_t e = once_per_device(attr_done, [&] {
    return cudaFuncSetAttribute(fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (3 * kMaxForkRows + 1) * static_cast<int>(sizeof(int)) +
                                    kMaxForkRows * static_cast<int>(sizeof(ForkRow)));
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(fork_kernel, dim3(kCluster), dim3(kThreads), smem, stream, pdl, p);
}

cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream, bool pdl) {
  return launch_pdl(compact_kernel, dim3(kCluster), dim3(kThreads), 0, stream, pdl, p);
}

cudaError_t launch_copy(const CopyParams& p, cudaStream_t stream, bool pdl) {
  int units = 0;
  for (int c = 0; c < p.caches; ++c) units += p.cache[c].rows == 1 ? 1 : p.cache[c].units;
  // CTAs for eight an SM; each copy in four shares at least (one share each for 2170 moves of
  // 192 KiB left the SMs uneven: 90 us, 87 with four; a share a unit, ten: 109)
  const int x = p.n < 4096 ? p.n : 4096;
  const int fill = (8 * p.sms + x - 1) / x;
  int y = fill > 4 ? fill : 4;
  y = y < units ? y : units;
  return launch_pdl(copy_kernel, dim3(static_cast<unsigned>(x), static_cast<unsigned>(y)),
                    dim3(kCopyThreads), 0, stream, pdl, p);
}

}  // namespace msa
