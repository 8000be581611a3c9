// msa_append.cu -- the cache append: a step's new keys and values rotated by
// their positions, quantised to fp8 and written to their rows of the paged
// cache, and the step's queries rotated in the same launch.
//
// Operation (msa_append_kv in include/msa.h): token j of request b is at pos =
// seq_lens[b] - Q + j; a rotated pair is (a cos - b sin, b cos + a sin) with the
// table's row of pos; a code is e4m3(x / scale), scale the tensor's or, with page
// scales, the smallest power of two that holds the page's largest magnitude.
//
// What bounds it: bytes.  A token of 64/4 heads reads 18 KiB of q, k and v and
// its table row and writes 16 KiB of q (8 as fp8) and 1 KiB of codes, against
// a few instructions an element.  So every element is read once and written
// once: a half warp holds one head's row, 16 bytes a lane, the rotation's
// partner comes from a lane 8 to 64 elements away by shuffle (or is the
// neighbour in the lane), and the lane's table entries serve all the rows it
// rotates.
//
// One scale per tensor: a warp takes rows of one token, eight at a time, four
// 16-byte loads a lane in flight (eight with more than one task a warp).  Page
// scales need the largest magnitude of all of the page's new rows before the
// first code: in decode the rows of one (page, KV head, side), at most 16, stay in
// one warp's registers between the maximum and the quantisation; in prefill the
// CTA's eight warps read the page's up to 128 rows a second time, from L1 (held
// in registers they halved the CTAs an SM, which the query rows of the same
// launch paid for: 313 us for 28779 tokens of 64/4 heads).
//
// Measured (64/4 heads): 28779 tokens with page scales 181 us, 5.7 TB/s, 85 % of a copy's
// rate; 6000 tokens with one scale 39 us, 81 %; 128 single tokens 5 us, launch and four
// dependent loads.
#include "msa_device.cuh"
#include "msa_launch.h"

namespace msa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTokenRows = 8;     // rows of one token a warp takes
constexpr int kPasses = 8;        // page scales: two rows a warp and pass
constexpr int kDecodeRows = 2 * kPasses;   // tokens a request with one warp per unit

// A lane's share of a head's row: elements 8 c .. 8 c + 7 of it, c = lane % 16.
// The rotation as y = x * c + x' * s, x' the pair's other element.
struct Rotation {
  float c[8], s[8];
  int partner;      // lane that holds x' (halves), or -1: x' is the neighbour here
  bool on;          // this lane's elements are rotated

  __device__ __forceinline__ void load(const AppendParams& p, int pos, int lane) {
    const int ch = lane & 15, half = p.rot_dim >> 4;   // chunks of half the rotated dims
    on = ch < 2 * half;
    partner = -1;
    if (!on) return;
    const float* row = p.cos_sin + static_cast<int64_t>(pos) * p.rot_dim;
    if (p.interleaved) {
      const float4 cv = __ldg(reinterpret_cast<const float4*>(row + 4 * ch));
      const float4 sv = __ldg(reinterpret_cast<const float4*>(row + 8 * half + 4 * ch));
      const float ca[4] = {cv.x, cv.y, cv.z, cv.w}, sa[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        c[2 * e] = c[2 * e + 1] = ca[e];
        s[2 * e] = -sa[e];
        s[2 * e + 1] = sa[e];
      }
    } else {
      const bool first = ch < half;
      const int f = first ? ch : ch - half;
      const float sign = first ? -1.f : 1.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float4 cv = __ldg(reinterpret_cast<const float4*>(row + 8 * f + 4 * k));
        const float4 sv = __ldg(reinterpret_cast<const float4*>(row + 8 * half + 8 * f + 4 * k));
        c[4 * k] = cv.x, c[4 * k + 1] = cv.y, c[4 * k + 2] = cv.z, c[4 * k + 3] = cv.w;
        s[4 * k] = sign * sv.x, s[4 * k + 1] = sign * sv.y;
        s[4 * k + 2] = sign * sv.z, s[4 * k + 3] = sign * sv.w;
      }
    }
  }

  // The lane of the half warp that holds x' (its own when nothing is exchanged);
  // the same for every token, so every lane can take part in the shuffles.
  static __device__ __forceinline__ int source(const AppendParams& p, int lane) {
    const int ch = lane & 15, half = p.rot_dim >> 4;
    if (p.interleaved || ch >= 2 * half) return lane;
    return (lane & 16) | (ch < half ? ch + half : ch - half);
  }
};

__device__ __forceinline__ void unpack8(const uint4& r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = bf16_bits_to_f32(w[e] & 0xFFFF);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}

// The lane's eight elements of a row, rotated (`turn`: this row is rotated at
// all).  Every lane of the warp calls it.
__device__ __forceinline__ void rotate8(const AppendParams& p, const Rotation& rot, int src,
                                        bool turn, const uint4& raw, float (&y)[8]) {
  unpack8(raw, y);
  if (p.rot_dim == 0) return;
  float x[8];
  if (p.interleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = y[e ^ 1];
  } else {
    uint4 o;
    o.x = __shfl_sync(0xffffffffu, raw.x, src);
    o.y = __shfl_sync(0xffffffffu, raw.y, src);
    o.z = __shfl_sync(0xffffffffu, raw.z, src);
    o.w = __shfl_sync(0xffffffffu, raw.w, src);
    unpack8(o, x);
  }
  if (turn && rot.on) {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = fmaf(y[e], rot.c[e], x[e] * rot.s[e]);
  }
}

__device__ __forceinline__ uint2 to_e4m3x8(const float (&y)[8], float f) {
  return make_uint2(f32x4_to_e4m3x4(y[0] * f, y[1] * f, y[2] * f, y[3] * f),
                    f32x4_to_e4m3x4(y[4] * f, y[5] * f, y[6] * f, y[7] * f));
}

__device__ __forceinline__ bool seq_len_ok(const AppendParams& p, int L) {
  return L >= 0 && (L == 0 || (L - 1) / kPage < p.S);
}

// ----------------------------------------------------------------------------
// Rows of one token by one warp: query rows, and with one scale per tensor the
// K and V rows, eight a task.  A token's first ceil(Hq / 8) tasks are query rows
// 8 t .. 8 t + 7, the rest K and V rows.  A warp takes `per` consecutive tasks of
// one token, the next task's loads in flight while one is rotated and written:
// the token's position and table row, four dependent loads away in a prefill
// batch, are then fetched once for many rows.

template <bool kScaled>
struct TokenTasks {
  int gq, all;
  __host__ __device__ explicit TokenTasks(const AppendParams& p) {
    gq = (p.Hq + kTokenRows - 1) / kTokenRows;
    all = gq + (kScaled ? 0 : (p.sides * p.Hkv + kTokenRows - 1) / kTokenRows);
  }
};

template <bool kVarlen, bool kScaled>
__device__ __forceinline__ void token_rows(const AppendParams& p, int64_t work, int per, int lane) {
  const TokenTasks<kScaled> tasks(p);
  const int parts = (tasks.all + per - 1) / per;
  const int i = static_cast<int>(work / parts);
  const int first = static_cast<int>(work - static_cast<int64_t>(i) * parts) * per;
  if (i >= p.T) return;
  const int last = min(first + per, tasks.all);
  const int ch = lane & 15, odd = lane >> 4;
  const int kv_rows = p.sides * p.Hkv;
  auto load = [&](int t, uint4 (&raw)[kTokenRows / 2]) {
    const bool is_q = t < tasks.gq;
    const int r0 = kTokenRows * (is_q ? t : t - tasks.gq) + odd;
    const int nrows = is_q ? p.Hq : kv_rows;
#pragma unroll
    for (int k = 0; k < kTokenRows / 2; ++k) {
      const int r = r0 + 2 * k;
      raw[k] = make_uint4(0u, 0u, 0u, 0u);
      if (r < nrows) {
        const uint16_t* src = is_q ? p.q + i * p.q_stride + r * kHeadDim
                              : r < p.Hkv ? p.k + i * p.k_stride + r * kHeadDim
                                          : p.v + i * p.v_stride + (r - p.Hkv) * kHeadDim;
        raw[k] = *reinterpret_cast<const uint4*>(src + 8 * ch);
      }
    }
  };
  uint4 raw[kTokenRows / 2];
  load(first, raw);
  int b, j, qlen;
  bool ok = true;
  if constexpr (kVarlen) {
    ok = varlen_token(p.cu_q, p.B, i, lane, b, j, qlen);
  } else {
    b = i / p.Q;
    j = i - b * p.Q;
    qlen = p.Q;
  }
  const int L = p.seq_lens[b];
  ok = ok && seq_len_ok(p, L) && (!kVarlen || L >= qlen);
  if (!ok && lane == 0) flag_error(p.err, MSA_ERR_SEQ_RANGE);
  int pos = ok ? L - qlen + j : -1;
  if (pos >= p.max_pos) {
    if (lane == 0) flag_error(p.err, MSA_ERR_POS_RANGE);
    pos = -1;
  }
  Rotation rot;
  rot.on = false;
  if (p.rot_dim > 0 && pos >= 0) rot.load(p, pos, lane);
  const int src = Rotation::source(p, lane);
  for (int t = first; t < last; ++t) {
    uint4 next[kTokenRows / 2] = {};
    if (t + 1 < last) load(t + 1, next);
    if (t < tasks.gq) {
      const int r0 = kTokenRows * t + odd;
#pragma unroll
      for (int k = 0; k < kTokenRows / 2; ++k) {
        const int r = r0 + 2 * k;
        if (pos < 0) raw[k] = make_uint4(0u, 0u, 0u, 0u);
        float y[8];
        rotate8(p, rot, src, true, raw[k], y);
        if (r >= p.Hq) continue;
        const int64_t at = (static_cast<int64_t>(i) * p.Hq + r) * kHeadDim + 8 * ch;
        if (p.q_fp8) {
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.q_out) + at) = to_e4m3x8(y, p.inv_q);
        } else {
          uint4 o;
          o.x = f32_to_bf16_bits(y[0]) | (f32_to_bf16_bits(y[1]) << 16);
          o.y = f32_to_bf16_bits(y[2]) | (f32_to_bf16_bits(y[3]) << 16);
          o.z = f32_to_bf16_bits(y[4]) | (f32_to_bf16_bits(y[5]) << 16);
          o.w = f32_to_bf16_bits(y[6]) | (f32_to_bf16_bits(y[7]) << 16);
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.q_out) + at) = o;
        }
      }
    } else if (!kScaled && pos >= 0) {
      const int page = p.block_table[static_cast<int64_t>(b) * p.S + pos / kPage];
      if (page < 0 || static_cast<int64_t>(page) >= p.num_blocks) {
        if (lane == 0) flag_error(p.err, MSA_ERR_PAGE_RANGE);
      } else {
        const int row_bytes = kHeadDim * p.sides;
        uint8_t* dst = p.kv + (static_cast<int64_t>(page) * p.Hkv * kPage + pos % kPage) * row_bytes;
        const int r0 = kTokenRows * (t - tasks.gq) + odd;
#pragma unroll
        for (int k = 0; k < kTokenRows / 2; ++k) {
          const int r = r0 + 2 * k;
          const bool is_k = r < p.Hkv;
          float y[8];
          rotate8(p, rot, src, is_k, raw[k], y);
          if (r < kv_rows)
            *reinterpret_cast<uint2*>(dst +
                                      static_cast<int64_t>(is_k ? r : r - p.Hkv) * kPage * row_bytes +
                                      (is_k ? 0 : kHeadDim) + 8 * ch) =
                to_e4m3x8(y, is_k ? p.inv_k : p.inv_v);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kTokenRows / 2; ++k) raw[k] = next[k];
  }
}

// ----------------------------------------------------------------------------
// Page scales.

// The smallest power of two s >= 2^-40 with amax <= 448 s, at most 2^40 (amax
// finite, >= 0): 448 = 1.75 * 2^8, so for amax = m 2^x it is 2^(x - 8), or twice
// that when m > 1.75.
__device__ __forceinline__ float page_scale_for(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = max(-40, min(40, e));
  return exp2i(e);
}

// Slots of the requests before request r in a prefill batch: a request of n
// tokens touches at most n / 128 + 2 pages (rounded down), which
// floor(end / 128) - floor(start / 128) + 2 is not below.
__device__ __forceinline__ int slots_before(const int32_t* cu_q, int r) {
  return cu_q[r] / kPage + 2 * r;
}

// One unit: the new rows of one (page, KV head, side), by kW warps (`w`: the
// calling warp's number among them).  kW = 1: at most 16 rows.
template <bool kVarlen, int kW>
__device__ __forceinline__ void page_unit(const AppendParams& p, int64_t unit, int w, int lane,
                                          float* red) {
  const int heads = p.Hkv * p.sides;
  const int64_t slot = unit / heads;
  const int hs = static_cast<int>(unit - slot * heads);
  const int g = hs / p.sides, side = hs - g * p.sides;
  int b, part, start, qlen;
  if constexpr (kVarlen) {
    // the request whose slots hold this one: the last with slots_before <= slot
    int lo = 0, hi = p.B;
    while (lo < hi) {
      const int step = (hi - lo + 31) >> 5;
      const int r = lo + (lane + 1) * step - 1;
      const bool before = r < hi && slots_before(p.cu_q, r + 1) <= slot;
      const int k = __popc(__ballot_sync(0xffffffffu, before));
      lo += k * step;
      hi = min(hi, lo + step - 1);
    }
    if (lo >= p.B) return;
    b = lo;
    start = p.cu_q[b];
    const int end = p.cu_q[b + 1];
    part = static_cast<int>(slot - slots_before(p.cu_q, b));
    if (start < 0 || end < start || end > p.T || part < 0) {
      if (lane == 0) flag_error(p.err, MSA_ERR_SEQ_RANGE);
      return;
    }
    qlen = end - start;
    if (qlen == 0) return;
  } else {
    const int per = p.Q > 1 ? 2 : 1;   // Q <= 32 tokens touch at most two pages
    b = static_cast<int>(slot / per);
    part = static_cast<int>(slot - static_cast<int64_t>(b) * per);
    if (b >= p.B) return;
    start = b * p.Q;
    qlen = p.Q;
  }
  const int L = p.seq_lens[b];
  if (!seq_len_ok(p, L) || (kVarlen && L < qlen)) {
    if (lane == 0) flag_error(p.err, MSA_ERR_SEQ_RANGE);
    return;
  }
  const int pos0 = max(L - qlen, 0);               // the request's first position written
  const int n = pos0 / kPage + part;               // logical page
  if (n > (L - 1) / kPage || L == 0) return;
  const int first = max(pos0, n * kPage), r0 = first - n * kPage;
  int last = min(L, (n + 1) * kPage);              // one past the last position here
  if (last > p.max_pos) {
    if (lane == 0) flag_error(p.err, MSA_ERR_POS_RANGE);
    last = p.max_pos;
  }
  const int rows = last - first;
  if (rows <= 0) return;
  const int page = p.block_table[static_cast<int64_t>(b) * p.S + n];
  if (page < 0 || static_cast<int64_t>(page) >= p.num_blocks) {
    if (lane == 0) flag_error(p.err, MSA_ERR_PAGE_RANGE);
    return;
  }
  float* scale = p.kv_scales + (static_cast<int64_t>(page) * p.Hkv + g) * p.sides + side;
  const float old = *scale;
  // token of position `first`
  const int64_t tok0 = start + (first - (L - qlen));
  const uint16_t* src_rows = side == 0 ? p.k + tok0 * p.k_stride + g * kHeadDim
                                       : p.v + tok0 * p.v_stride + g * kHeadDim;
  const int64_t stride = side == 0 ? p.k_stride : p.v_stride;
  constexpr int kHeld = kW == 1 ? kPasses : kPasses / 4;   // passes in registers at once
  const int ch = lane & 15, odd = lane >> 4;
  const float inv = side == 0 ? p.inv_k : p.inv_v;
  const int shsrc = Rotation::source(p, lane);
  // rows 2 (kW k + w) + odd, k = k0 .. k0 + n - 1, rotated and over the tensor's scale
  auto fetch = [&](int k0, auto& y) {
    constexpr int n = sizeof(y) / sizeof(y[0]);
    uint4 raw[n];
#pragma unroll
    for (int k = 0; k < n; ++k) {
      const int r = 2 * (kW * (k0 + k) + w) + odd;
      raw[k] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows) raw[k] = *reinterpret_cast<const uint4*>(src_rows + r * stride + 8 * ch);
    }
#pragma unroll
    for (int k = 0; k < n; ++k) {
      const int r = 2 * (kW * (k0 + k) + w) + odd;
      Rotation rot;
      rot.on = false;
      if (side == 0 && p.rot_dim > 0 && r < rows) rot.load(p, first + r, lane);
      if (side == 0) rotate8(p, rot, shsrc, true, raw[k], y[k]);
      else unpack8(raw[k], y[k]);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[k][e] *= inv;
    }
  };
  float amax = 0.f;
  auto largest = [&](const auto& y) {
    constexpr int n = sizeof(y) / sizeof(y[0]);
#pragma unroll
    for (int k = 0; k < n; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = fabsf(y[k][e]);
        amax = a < INFINITY ? fmaxf(amax, a) : amax;   // finite values only
      }
  };
  float kept[kHeld][8];
  if constexpr (kW == 1) {
    fetch(0, kept);
    largest(kept);
  } else {
#pragma unroll 1
    for (int k0 = 0; k0 < kPasses; k0 += kHeld) {
      fetch(k0, kept);
      largest(kept);
    }
  }
  amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
  if constexpr (kW > 1) {
    if (lane == 0) red[w] = amax;
    __syncthreads();     // every thread of the CTA works on this unit
#pragma unroll
    for (int k = 0; k < kW; ++k) amax = fmaxf(amax, red[k]);
  }
  float s = page_scale_for(amax);
  if (r0 > 0) {
    if (!page_scale_ok(old)) {
      if (lane == 0) flag_error(p.err, MSA_ERR_SCALE);
      return;
    }
    s = fmaxf(s, old);
  }
  const int row_bytes = kHeadDim * p.sides;
  uint8_t* dst = p.kv + (static_cast<int64_t>(page) * p.Hkv + g) * kPage * row_bytes + side * kHeadDim;
  const float f = 1.f / s;
  auto write = [&](int k0, const auto& y) {
    constexpr int n = sizeof(y) / sizeof(y[0]);
#pragma unroll
    for (int k = 0; k < n; ++k) {
      const int r = 2 * (kW * (k0 + k) + w) + odd;
      if (r < rows)
        *reinterpret_cast<uint2*>(dst + static_cast<int64_t>(r0 + r) * row_bytes + 8 * ch) =
            to_e4m3x8(y[k], f);
    }
  };
  if constexpr (kW == 1) {
    write(0, kept);
  } else {
#pragma unroll 1
    for (int k0 = 0; k0 < kPasses; k0 += kHeld) {
      fetch(k0, kept);
      write(k0, kept);
    }
  }
  if (r0 > 0 && s > old) {
    // the scale grew: the rows before the new ones, requantised
    const float ratio = old / s;
    for (int x = 32 * w + lane; x < 8 * r0; x += 32 * kW) {
      uint4* at = reinterpret_cast<uint4*>(dst + static_cast<int64_t>(x >> 3) * row_bytes + 16 * (x & 7));
      uint4 c = *at;
      uint32_t* cw = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t a = e4m3x2_to_f16x2(cw[e] & 0xFFFF), d = e4m3x2_to_f16x2(cw[e] >> 16);
        const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&a));
        const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&d));
        cw[e] = f32x4_to_e4m3x4(lo.x * ratio, lo.y * ratio, hi.x * ratio, hi.y * ratio);
      }
      *at = c;
    }
  }
  // every lane has read the old scale (the other warps before the maximum)
  __syncwarp();
  if (w == 0 && lane == 0) *scale = s;
}

// Page-scale units in the first unit_blocks CTAs, then the tokens' rows.
template <bool kVarlen, bool kScaled, int kW>
__global__ void __launch_bounds__(kThreads, kScaled && kW == 1 ? 2 : 3)
    append_kernel(const AppendParams p, int unit_blocks, int per) {
  __shared__ float red[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();   // cache rows, scales and outputs may be the previous kernel's
  if (kVarlen && blockIdx.x == 0 && threadIdx.x == 0 &&
      (p.cu_q[0] != 0 || p.cu_q[p.B] != p.T))
    flag_error(p.err, MSA_ERR_SEQ_RANGE);
  if (kScaled && static_cast<int>(blockIdx.x) < unit_blocks) {
    if constexpr (kW == 1)
      page_unit<kVarlen, 1>(p, static_cast<int64_t>(blockIdx.x) * kWarps + warp, 0, lane, red);
    else
      page_unit<kVarlen, kW>(p, blockIdx.x, warp, lane, red);
    return;
  }
  token_rows<kVarlen, kScaled>(
      p, (static_cast<int64_t>(blockIdx.x) - unit_blocks) * kWarps + warp, per, lane);
}

// Nothing: stands between an append and a call that may start early (see launch_append).
__global__ void order_kernel() {}

}  // namespace

cudaError_t launch_append(const AppendParams& p, cudaStream_t stream, bool pdl) {
  const bool scaled = p.kv_scales != nullptr, varlen = p.cu_q != nullptr;
  // one warp a unit holds 16 rows; longer queries take a CTA a unit
  const bool narrow = !varlen && p.Q <= kDecodeRows;
  int64_t unit_blocks = 0;
  if (scaled) {
    const int64_t slots = varlen ? p.T / kPage + 2 * static_cast<int64_t>(p.B)
                                 : static_cast<int64_t>(p.B) * (p.Q > 1 ? 2 : 1);
    const int64_t units = slots * p.Hkv * p.sides;
    unit_blocks = narrow ? (units + kWarps - 1) / kWarps : units;
  }
  // Tasks of one token a warp takes: one while that leaves the GPU's warps idle
  // (decode: latency), all of a token's when there is a wave of such warps (6000
  // tokens of 64/4 heads: 9 tasks a warp 41.1 us, 3 41.9, 1 58.4), in equal shares.
  const int tasks = scaled ? TokenTasks<true>(p).all : TokenTasks<false>(p).all;
  const int64_t wave = static_cast<int64_t>(p.sms) * 24;   // three CTAs an SM
  const int64_t fit = static_cast<int64_t>(p.T) * tasks / wave;
  int per = tasks == 0 ? 1 : static_cast<int>(fit < 1 ? 1 : fit > tasks ? tasks : fit);
  const int shares = (tasks + per - 1) / per;
  if (shares > 0) per = (tasks + shares - 1) / shares;
  const int64_t warps = static_cast<int64_t>(p.T) * ((tasks + per - 1) / per);
  const int64_t blocks = unit_blocks + (warps + kWarps - 1) / kWarps;
  if (blocks == 0) return cudaSuccess;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks)), block(kThreads);
  const int ub = static_cast<int>(unit_blocks);
  cudaError_t e =
      !scaled ? (varlen ? launch_pdl(append_kernel<true, false, 1>, grid, block, 0, stream, pdl, p, ub, per)
                        : launch_pdl(append_kernel<false, false, 1>, grid, block, 0, stream, pdl, p, ub, per))
      : varlen ? launch_pdl(append_kernel<true, true, kWarps>, grid, block, 0, stream, pdl, p, ub, per)
      : narrow ? launch_pdl(append_kernel<false, true, 1>, grid, block, 0, stream, pdl, p, ub, per)
               : launch_pdl(append_kernel<false, true, kWarps>, grid, block, 0, stream, pdl, p, ub, per);
  // With input overlap on, the next call's first kernel reads the cache and
  // the query before it waits for the kernel just before it.  An empty kernel
  // that starts only after this one has finished stands between them.
  if (e == cudaSuccess && pdl)
    e = launch_pdl(order_kernel, dim3(1), dim3(1), 0, stream, false);
  return e;
}

}  // namespace msa
