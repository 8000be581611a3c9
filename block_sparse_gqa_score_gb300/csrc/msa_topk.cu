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
// What bounds it: the issue slots, some 720 instructions a row (its scores are a few hundred
// floats).  The kept blocks are found from the lanes' own maxima: L, the 15th largest of
// the 32, has at least 15 scores at or above it, and few are above it (some 20 of 256
// random ones).  If fewer than 15 are, they are kept with the first scores equal to L; else
// the 15 are chosen among them alone, each compared with all of them in shared memory.  A row
// with more than 64 scores above L (they would have to lie in few lanes) is left to the search
// of msa_select.cuh.  Rows of up to 2048 blocks are held in registers, longer ones read again.
// 5999 tokens of 4 heads over up to 512 blocks: 18.6 us, 1.4 TB/s of scores; the same rows in
// a table of more than 512 columns, which the long form takes, 29.8; over 1024 .. 2048 blocks
// 91.8.  (A search bit by bit, 31 rounds of a count over the warp, took 83 us for the first;
// several heads of a token in one warp, with the next row's scores on their way, was slower.)
// A decode step's 256 rows of 2000 blocks 7.6 us (bit by bit 31), 32 rows of 4000 13.3 (106);
// rows whose best scores all lie in three lanes, which are searched after all, 31.8 and 126
// (31 and 116).
#include "msa_device.cuh"
#include "msa_launch.h"
#include "msa_select.cuh"

namespace msa {

namespace {

constexpr int kWarps = 4;
constexpr int kShort = 512;   // blocks of a row that the short form takes
constexpr int kAbove = 64;    // scores above L that are compared with each other

// Smallest of a float across the warp, NaN ignored.
__device__ __forceinline__ float warp_min_f32(float x) {
  float r;
  asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// The kept blocks of a row of 16 .. 32 NK candidates, as select::select_row returns them;
// false where it has to do it.  Scores are compared as they are (-0 equals 0); a NaN score
// counts as -inf, and a NaN of this function's own stands for no block at all: no
// comparison holds with it.  NK 0: rows of any length, read again in place of being held.
// scratch: shared words of this warp, at most 1024.
template <int NK>
__device__ __forceinline__ bool select_by_maxima(const float* __restrict__ srow, int64_t stride_n,
                                                 int cur, int lane, uint32_t* scratch, int* slots,
                                                 bool& nan, int& kept) {
  constexpr unsigned kAll = 0xffffffffu;
  constexpr int kSel = select::kSel;
  const float none = __uint_as_float(0x7FFFFFFFu);
  constexpr int kRoom = NK > 0 && NK <= 16 ? 32 * NK : kAbove;   // scores above L that are kept
  constexpr int kUnroll = NK > 0 ? NK : 8;
  const int groups = NK > 0 ? NK : (cur + 31) / 32;
  float* above = reinterpret_cast<float*>(scratch);
  uint32_t* block = scratch + kRoom;
  float f[kUnroll];
  // the score of block lane + 32 e
  auto load = [&](int e) {
    return 32 * e < cur - lane ? __ldg(srow + (lane + 32 * static_cast<int64_t>(e)) * stride_n) : none;
  };
  float m = none;
  if constexpr (NK > 0) {
    const float* at = srow + lane * stride_n;
    const int64_t step = 32 * stride_n;
#pragma unroll
    for (int e = 0; e < NK; ++e, at += step) f[e] = 32 * e < cur - lane ? __ldg(at) : none;
#pragma unroll
    for (int e = 0; e < NK; ++e) {
      const bool bad = f[e] != f[e] && 32 * e < cur - lane;
      nan |= bad;
      f[e] = bad ? -INFINITY : f[e];
      m = fmaxf(m, f[e]);
    }
  } else {
    for (int e0 = 0; e0 < groups; e0 += kUnroll) {
#pragma unroll
      for (int e = 0; e < kUnroll; ++e) f[e] = load(e0 + e);
#pragma unroll
      for (int e = 0; e < kUnroll; ++e) {
        const bool bad = f[e] != f[e] && 32 * (e0 + e) < cur - lane;
        nan |= bad;
        m = fmaxf(m, bad ? -INFINITY : f[e]);
      }
    }
  }
  auto value = [&](int e) {
    if constexpr (NK > 0) return f[e];
    const float x = load(e);
    return x != x && 32 * e < cur - lane ? -INFINITY : x;
  };
  // L: the smallest of the lanes' maxima that fewer than 15 are larger than
  above[lane] = m;
  __syncwarp();
  int larger = 0;
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    const float4 v = *reinterpret_cast<const float4*>(above + j);
    larger += (v.x > m) + (v.y > m) + (v.z > m) + (v.w > m);
  }
  const float low = warp_min_f32(larger < kSel ? m : none);
  __syncwarp();
  // the scores above L and their blocks, in ascending order of the blocks
  const unsigned lt = (1u << lane) - 1u;
  int n = 0;
#pragma unroll kUnroll
  for (int e = 0; e < groups; ++e) {
    const float x = value(e);
    const bool over = x > low;
    const unsigned b = __ballot_sync(kAll, over);
    const int k = n + __popc(b & lt);
    if (over && (kRoom == 32 * NK || k < kRoom)) {
      above[k] = x;
      block[k] = lane + 32 * e;
    }
    n += __popc(b);
  }
  __syncwarp();     // (ahead of the return too: who searches the row writes the same words)
  if (n > kAbove) return false;
  if (n >= kSel) {
    // tau: the smallest of them that fewer than 15 are larger than; all larger ones are kept, and
    // of its equals as many of the first as there is room for
    const bool two = n > 32;
    const float a = lane < n ? above[lane] : none, b = 32 + lane < n ? above[32 + lane] : none;
    int a_gt = 0, b_gt = 0;
    for (int j = 0; j < n; j += 4) {
      float4 v = *reinterpret_cast<const float4*>(above + j);
      if (j + 4 > n) {                     // (what lies past the n-th is not counted)
        v.y = j + 1 < n ? v.y : none;
        v.z = j + 2 < n ? v.z : none;
        v.w = none;
      }
      a_gt += (v.x > a) + (v.y > a) + (v.z > a) + (v.w > a);
      if (two) b_gt += (v.x > b) + (v.y > b) + (v.z > b) + (v.w > b);
    }
    const float tau = warp_min_f32(fminf(a_gt < kSel ? a : none, two && b_gt < kSel ? b : none));
    const unsigned gt_a = __ballot_sync(kAll, a > tau), eq_a = __ballot_sync(kAll, a == tau);
    const unsigned gt_b = __ballot_sync(kAll, b > tau), eq_b = __ballot_sync(kAll, b == tau);
    const int need = kSel - __popc(gt_a) - __popc(gt_b);
    const bool take_a = a > tau || (a == tau && __popc(eq_a & lt) < need);
    const bool take_b = b > tau || (b == tau && __popc(eq_a) + __popc(eq_b & lt) < need);
    const unsigned t_a = __ballot_sync(kAll, take_a), t_b = __ballot_sync(kAll, take_b);
    if (take_a) slots[__popc(t_a & lt)] = block[lane];
    if (take_b) slots[__popc(t_a) + __popc(t_b & lt)] = block[32 + lane];
  } else {
    // all scores above L, and of those equal to it the first
    const int need = kSel - n;
    int written = 0, ties = 0;
#pragma unroll kUnroll
    for (int e = 0; e < groups; ++e) {
      const float x = value(e);
      const bool eq = x == low;
      const unsigned be = __ballot_sync(kAll, eq);
      const bool take = x > low || (eq && ties + __popc(be & lt) < need);
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
// have more than kShort blocks; without it a thread has 48 or 56 registers and a warp 4 KiB,
// with it 154 and 8 KiB, and an SM holds 12 warps in place of 36.
template <bool kVarlen, bool kLong>
__global__ void __launch_bounds__(kWarps * 32) topk_kernel(const TopkParams p) {
  constexpr int kCache = kLong ? 2048 : 1024;     // words of shared memory a warp
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
  else if (kLong && cur > 32 * 64)
    done = select_by_maxima<0>(srow, p.stride_n, cur, lane, s_keys[warp], s_slots[warp], nan, v);
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
