// msa_topk.cu -- stage 2, the block selector.
//
// For each (token, KV head) row: keep the current block cur = pos/128 and the
// 15 best earlier blocks in the order (score descending, block index
// ascending); write the kept ids ascending, -1 padded (the vLLM test file's
// _make_topk layout); all -1 for a padding row.  Scores are read through
// arbitrary element strides, as TensorRT-LLM PR #17171's selector takes the
// scorer's [head, token, block] buffer through a transposed view.  One warp
// per row; the per-row algorithm is in msa_select.cuh.
#include "msa_device.cuh"
#include "msa_launch.h"
#include "msa_select.cuh"

namespace msa {

namespace {

constexpr int kWarps = 4;
constexpr int kCache = 2048;  // candidates cached per warp (8 KiB)

// kVarlen: a prefill-style batch, the tokens' requests looked up in cu_q.
template <bool kVarlen>
__global__ void __launch_bounds__(kWarps * 32) topk_kernel(const TopkParams p) {
  __shared__ uint32_t s_keys[kWarps][kCache];
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
  const int v = select::select_row<64>(srow, p.stride_n, pos, lane, s_keys[warp], kCache,
                                   s_slots[warp], nan);
  if (lane < kTopK) out[lane] = v;
  if (__any_sync(0xffffffffu, nan) && lane == 0) flag_error(p.err, MSA_ERR_SCORE_NAN);
}

}  // namespace

cudaError_t launch_topk(const TopkParams& p, cudaStream_t stream, bool pdl) {
  const int64_t rows = static_cast<int64_t>(p.cu_q ? p.T : p.B * p.Q) * p.Hkv;
  const int64_t grid = (rows + kWarps - 1) / kWarps;
  return launch_pdl(p.cu_q ? topk_kernel<true> : topk_kernel<false>,
                    dim3(static_cast<unsigned>(grid)), dim3(kWarps * 32), 0, stream, pdl, p);
}

}  // namespace msa
