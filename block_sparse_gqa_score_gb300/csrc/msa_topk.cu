// msa_topk.cu -- stage 2, the block selector.
//
// For each (token, KV head) row: keep the current block cur = pos/128 and the
// 15 best earlier blocks in the order (score descending, block index
// ascending); write the kept ids ascending, -1 padded (the vLLM test file's
// _make_topk layout); all -1 for a padding row.  Scores are read through
// arbitrary element strides, as TensorRT-LLM PR #17171's selector takes the
// scorer's [head, token, block] buffer through a transposed view.  One warp
// per row.
//
// What bounds it: the issue slots, some 650 instructions a row (its scores are a few hundred
// floats).  The kept blocks are found from the lanes' own maxima: L, the 15th largest of
// the 32, has at least 15 keys at or above it, and few keys are above it (some 20 of 256
// random ones).  If fewer than 15 are, they are kept with the first keys equal to L; else
// the 15 are chosen among them alone, each compared with all of them in shared memory.
// 5980 tokens of 4 heads over up to 512 blocks: 24 us, 1.1 TB/s of scores.  (A search bit by
// bit, 31 rounds of a count over the warp, took 83 us; several heads of a token in one
// warp, with the next row's scores on their way, 26 to 28.)  A row with more than 64 keys above L (they would have to lie in few lanes) is
// left to the search of msa_select.cuh, as are rows of more than 2048 blocks.
#include "msa_device.cuh"
#include "msa_launch.h"
#include "msa_select.cuh"

namespace msa {

namespace {

constexpr int kWarps = 4;
constexpr int kShort = 512;   // blocks of a row that the short form takes
constexpr int kAbove = 64;    // keys above L that are compared with each other

// select::order_key in fewer steps: -0 becomes 0 by the addition.
__device__ __forceinline__ uint32_t key_of(float x, bool& nan) {
  const bool bad = x != x;
  nan |= bad;
  const uint32_t u = __float_as_uint(x + 0.f);
  return bad ? 0x007FFFFFu : u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

// The kept blocks of a row of 16 .. 32 NK candidates, as select::select_row returns them;
// false where it has to do it.  above: shared scratch of this warp, 2 kAbove words.
template <int NK>
__device__ __forceinline__ bool select_by_maxima(const float* __restrict__ srow, int64_t stride_n,
                                                 int cur, int lane, uint32_t* above, int* slots,
                                                 bool& nan, int& kept) {
  constexpr unsigned kAll = 0xffffffffu;
  constexpr int kSel = select::kSel;
  uint32_t k[NK];
  uint32_t m = 0;
  {
    float f[NK];
#pragma unroll
    for (int e = 0; e < NK; ++e) f[e] = lane + 32 * e < cur ? srow[(lane + 32 * e) * stride_n] : 0.f;
#pragma unroll
    for (int e = 0; e < NK; ++e) {
      k[e] = lane + 32 * e < cur ? key_of(f[e], nan) : 0u;   // 0 ranks below every real key
      m = max(m, k[e]);
    }
  }
  // L: the smallest of the maxima that fewer than 15 are larger than
  int larger = 0;
#pragma unroll
  for (int o = 1; o < 32; ++o) larger += __shfl_xor_sync(kAll, m, o) > m;
  const uint32_t low = __reduce_min_sync(kAll, larger < kSel ? m : kAll);
  // the keys above L and their blocks, in ascending order
  const unsigned lt = (1u << lane) - 1u;
  uint32_t* block = above + kAbove;
  int n = 0;
#pragma unroll
  for (int e = 0; e < NK; ++e) {
    const bool over = k[e] > low;
    const unsigned b = __ballot_sync(kAll, over);
    const int at = n + __popc(b & lt);
    if (over && at < kAbove) {
      above[at] = k[e];
      block[at] = lane + 32 * e;
    }
    n += __popc(b);
  }
  if (n > kAbove) return false;
  __syncwarp();
  if (n >= kSel) {
    // tau: the smallest of them that fewer than 15 are larger than; all larger ones are kept, and
    // of its equals as many of the first as there is room for
    const uint32_t a = lane < n ? above[lane] : 0u, b = 32 + lane < n ? above[32 + lane] : 0u;
    int a_gt = 0, b_gt = 0;
    for (int j = 0; j < n; j += 4) {      // (words at and past n: not counted)
      const uint4 v = *reinterpret_cast<const uint4*>(above + j);
      const uint32_t x[4] = {v.x, j + 1 < n ? v.y : 0u, j + 2 < n ? v.z : 0u, j + 3 < n ? v.w : 0u};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a_gt += x[i] > a;
        b_gt += x[i] > b;
      }
    }
    const uint32_t tau = __reduce_min_sync(kAll, min(a_gt < kSel ? a : kAll, b != 0u && b_gt < kSel ? b : kAll));
    const unsigned gt_a = __ballot_sync(kAll, a > tau), gt_b = __ballot_sync(kAll, b > tau);
    const unsigned eq_a = __ballot_sync(kAll, a == tau), eq_b = __ballot_sync(kAll, b == tau);
    const int need = kSel - __popc(gt_a) - __popc(gt_b);
    const bool take_a = a > tau || (a == tau && __popc(eq_a & lt) < need);
    const bool take_b = b > tau || (b == tau && __popc(eq_a) + __popc(eq_b & lt) < need);
    const unsigned t_a = __ballot_sync(kAll, take_a), t_b = __ballot_sync(kAll, take_b);
    if (take_a) slots[__popc(t_a & lt)] = block[lane];
    if (take_b) slots[__popc(t_a) + __popc(t_b & lt)] = block[32 + lane];
  } else {
    // all keys above L, and of those equal to it the first
    const int need = kSel - n;
    int written = 0, ties = 0;
#pragma unroll
    for (int e = 0; e < NK; ++e) {
      const bool eq = k[e] == low;             // (L is a real key: not 0)
      const unsigned be = __ballot_sync(kAll, eq);
      const bool take = k[e] > low || (eq && ties + __popc(be & lt) < need);
      const unsigned bs = __ballot_sync(kAll, take);
      if (take) slots[written + __popc(bs & lt)] = lane + 32 * e;
      ties += __popc(be);
      written += __popc(bs);
    }
  }
  if (lane == 0) slots[kSel] = cur;
  __syncwarp();
  kept = lane < kTopK ? slots[lane] : -1;
  return true;
}

// kVarlen: a prefill-style batch, the tokens' requests looked up in cu_q.  kLong: rows may
// have more than kShort blocks; without it a warp has 64 registers and 2 KiB, with it 168 and
// 8 KiB, and the GPU holds half as many.
template <bool kVarlen, bool kLong>
__global__ void __launch_bounds__(kWarps * 32) topk_kernel(const TopkParams p) {
  constexpr int kCache = kLong ? 2048 : kShort;   // candidates cached per warp
  __shared__ __align__(16) uint32_t s_keys[kWarps][kCache];
  __shared__ int s_slots[kWarps][kTopK];
  pdl_trigger();
  pdl_wait();  // scores come from the previous kernel; topk may still be read by one
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int T = kVarlen ? p.T : p.B * p.Q;
  if (row >= static_cast<int64_t>(T) * p.Hkv) return;
  const int i = static_cast<int>(row / p.Hkv), g = static_cast<int>(row - static_cast<int64_t>(i) * p.Hkv);
  int b, j, qlen;
  bool tok_ok = true;
  if constexpr (kVarlen) {
    tok_ok = varlen_token(p.cu_q, p.B, i, lane, b, j, qlen);
  } else {
    b = i / p.Q;
    j = i - b * p.Q;
    qlen = p.Q;
  }
  int32_t* out = p.topk + row * kTopK;

  const int L = p.seq_lens[b];
  // a prefill request's tokens are the last qlen of its sequence
  const bool seq_ok = tok_ok && L >= 0 && (L == 0 || (L - 1) / kPage < p.S) && (!kVarlen || L >= qlen);
  if (!seq_ok && lane == 0 && (kVarlen || j == 0) && g == 0) flag_error(p.err, MSA_ERR_SEQ_RANGE);
  const int pos = seq_ok ? L - qlen + j : -1;
  if (pos < 0) {
    if (lane < kTopK) out[lane] = -1;
    return;
  }
  const float* srow = p.scores + g * p.stride_h + static_cast<int64_t>(i) * p.stride_t;
  bool nan = false;
  const int cur = pos / kPage;
  int v;
  bool done = false;
  if (cur >= kTopK && cur <= 32 * 8)
    done = select_by_maxima<8>(srow, p.stride_n, cur, lane, s_keys[warp], s_slots[warp], nan, v);
  else if (cur >= kTopK && cur <= 32 * 16)
    done = select_by_maxima<16>(srow, p.stride_n, cur, lane, s_keys[warp], s_slots[warp], nan, v);
  else if (kLong && cur > 32 * 16 && cur <= 32 * 32)
    done = select_by_maxima<32>(srow, p.stride_n, cur, lane, s_keys[warp], s_slots[warp], nan, v);
  else if (kLong && cur > 32 * 32 && cur <= 32 * 64)
    done = select_by_maxima<64>(srow, p.stride_n, cur, lane, s_keys[warp], s_slots[warp], nan, v);
  if (!done)
    v = select::select_row<kLong ? 64 : 16>(srow, p.stride_n, pos, lane, s_keys[warp], kCache,
                                            s_slots[warp], nan);
  if (lane < kTopK) out[lane] = v;
  if (__any_sync(0xffffffffu, nan) && lane == 0) flag_error(p.err, MSA_ERR_SCORE_NAN);
}

}  // namespace

cudaError_t launch_topk(const TopkParams& p, cudaStream_t stream, bool pdl) {
  const int64_t rows = static_cast<int64_t>(p.cu_q ? p.T : p.B * p.Q) * p.Hkv;
  const int64_t grid = (rows + kWarps - 1) / kWarps;
  const bool varlen = p.cu_q != nullptr;
  auto* k = p.S > kShort ? (varlen ? topk_kernel<true, true> : topk_kernel<false, true>)
                         : (varlen ? topk_kernel<true, false> : topk_kernel<false, false>);
  return launch_pdl(k, dim3(static_cast<unsigned>(grid)), dim3(kWarps * 32), 0, stream, pdl, p);
}

}  // namespace msa
