// msa_page_softmax.cuh -- the softmax of the attends on a cache with page scales: what
// one group of four warps does with the S^T of a batch of pages.
//
// Mathematics.  With z the logit in log2 units and u = z + log2(vs[page]),
//
//   out = sum_t 2^(u_t - M) V8_t / sum_t 2^(u_t - M) / vs[page(t)],
//
// so the fp8 product takes weights P = 2^(u - M) that are relative to what a
// page contributes, and the running sum divides each page's by vs again.  u is
// one FFMA from the raw dot product: factor ks * sm_scale * log2(e) * 2^e (2^e
// of the query split), addend log2(vs) - M.  M is a running reference, not the
// running maximum: P = 2^(kPShift) at the largest u when M is set, and M stays
// until some P would pass 2^kPTop (e4m3 holds 448).  Whether it does is one vote
// a step: the largest of a thread's u against the bound, or-ed over the
// token's four warps by one barrier; only then are the exact maxima of the 16
// heads formed and exchanged and the sums and the accumulator rescaled.  (With
// exact maxima on every page a warp issued about 650 instructions a page; the
// vote leaves about 200.)
//
// P is two e4m3 parts, hi = P rounded and lo = 2^4 (P - hi) rounded (at most 16 * 16),
// in columns of their own that meet at the end, lo times 2^-4.  They carry P to 2^-8 of
// itself down to 2^-5; below that lo's step is 2^-13 absolutely, 2^-19.5 of the row's
// largest term (kPShift).  A tail of 10^5 keys under that step can hold half of a row's
// weight, and the running sum counts it, so lo is rounded with an offset of up to half a
// step that differs from key to key of a page (split_offset): of many equal small P the
// right share is stored as the step above and the rest as the one below.  Worked out from
// these roundings for 2048 to 262144 keys, equal or spread by a nat, beside a key of 0.1 to
// 0.97 of the weight, outputs are off by at most 0.0017 of sum p |v| (0.9 with lo on hi's
// grid, 0.9 without the offset).  It costs 1536 prefill tokens 4 of 271 us, the
// other attends nothing that could be measured.
#pragma once

#include "msa_device.cuh"
#include "msa_tcgen05.cuh"

namespace msa {
namespace paged {

constexpr float kPShift = 6.5f;               // P = 2^kPShift at the largest u when M is set
constexpr float kPTop = 8.5f;                 // M moves when some P would pass 2^kPTop

struct alignas(16) PageInfo {
  float k, lv, iv;   // as PageScale
  int block;         // logical block, -1: no key of this page is attended
};

// Softmax groups of four warps, each with kHeads heads of one token, behind four
// warps of other roles.
template <int kNT>
struct Groups {
  static constexpr int kHeads = kNT == 1 ? 8 : 16;
  static constexpr int kPerToken = kGroup / kHeads;
  static constexpr int kCount = kNT * kPerToken;
  static constexpr int kThreads = 32 * (4 + 4 * kCount);
  static constexpr int kBatch = kNT == 1 ? 2 : 1;   // pages a group takes at once
};

// mbar_wait with one try before the clock is read: most waits here find their phase
// complete.
__device__ __forceinline__ bool wait_for(uint64_t* bar, unsigned parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
  while (!mbar_try_wait_sleep(bar, parity, 1000000u))
    if (global_ns() - t0 > kWaitLimitNs) return false;
  return true;
}

// Barriers 1 .. 4 of the groups (named in the instruction: a kernel that computes the
// number is given all 16 of a CTA), with the or of a predicate or plain.
template <int kId>
__device__ __forceinline__ bool barrier_or_id(bool pred) {
  unsigned r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "barrier.cta.red.or.aligned.pred p, %2, 128, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(pred ? 1u : 0u), "n"(kId)
      : "memory");
  return r != 0;
}

template <int kId>
__device__ __forceinline__ void barrier_id() {
  asm volatile("barrier.cta.sync.aligned %0, 128;" ::"n"(kId) : "memory");
}

// Value rows that no token sees have P = 0, but their bytes may be anything (an fp8 NaN
// times 0 is NaN).  A page whose scales are bad has no product at all; in a page that
// ends past the (first) token's position the unseen rows are set to 0 by the warp that
// loads the V tiles, before it hands the tile on: such a tile lands on a barrier of its
// own.  In the softmax warps the same cost 9 us of 291 (1536 prefill tokens).
__device__ __forceinline__ void zero_value_rows(uint8_t* tile, int lim, int lane) {
  for (int x = 8 * max(lim + 1, 0) + lane; x < 8 * kPage; x += 32)
    reinterpret_cast<uint4*>(tile)[x] = make_uint4(0u, 0u, 0u, 0u);
}

template <int kNT>
__device__ __forceinline__ bool group_or(int gi, bool pred) {
  __syncwarp();
  if (gi == 0) return barrier_or_id<1>(pred);
  if (Groups<kNT>::kCount == 2 || gi == 1) return barrier_or_id<2>(pred);
  return gi == 2 ? barrier_or_id<3>(pred) : barrier_or_id<4>(pred);
}

template <int kNT>
__device__ __forceinline__ void group_sync(int gi) {
  __syncwarp();
  if (gi == 0) barrier_id<1>();
  else if (Groups<kNT>::kCount == 2 || gi == 1) barrier_id<2>();
  else if (gi == 2) barrier_id<3>();
  else barrier_id<4>();
}

__device__ __forceinline__ PageInfo page_info(const AttendParams& p, float2 scales, int block) {
  const PageScale s = make_page_scale(scales);
  if (s.bad != 0.f) flag_error(p.err, MSA_ERR_SCALE);
  return PageInfo{s.k, s.lv, s.iv, s.bad != 0.f ? -1 : block};
}

// Columns of this thread's tensor-memory lane.
__device__ __forceinline__ void ld_cols(uint32_t a, uint32_t (&r)[8]) { tc::ld_32x32b_x8(a, r); }
__device__ __forceinline__ void ld_cols(uint32_t a, uint32_t (&r)[16]) { tc::ld_32x32b_x16(a, r); }
__device__ __forceinline__ void st_cols(uint32_t a, const uint32_t (&r)[8]) { tc::st_32x32b_x8(a, r); }
__device__ __forceinline__ void st_cols(uint32_t a, const uint32_t (&r)[16]) { tc::st_32x32b_x16(a, r); }

__device__ __forceinline__ void store_p(uint8_t* at, const uint32_t (&w)[2]) {
  *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_p(uint8_t* at, const uint32_t (&w)[4]) {
  *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
}

// lo's rounding offset of a key, in [-1/2, 1/2) of its smallest step (2^-9), twice as
// fp16.  A page's keys take 128 evenly spaced offsets, neighbours far apart (bits
// reversed), and the next page's are turned by the golden ratio.  It depends on the
// key's place in the sequence alone.  An offset by itself rounds to 0, so P = 0 stays 0.
__device__ __forceinline__ uint32_t split_offset(uint32_t key_reversed, int block) {
  const int x = static_cast<int>(key_reversed + static_cast<uint32_t>(block) * 0x9E3779B9u);
  const float d = static_cast<float>(x) * exp2i(-41);
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %1;" : "=r"(r) : "f"(d));
  return r;
}

constexpr float kLoUnit = 0.0625f;   // 2^-4: lo counts these

// Four probabilities (0 <= P <= 448) -> their e4m3 parts, first in the low byte:
// hi = P rounded, lo = 16 times the remainder of P as fp16 (exact), plus the key's
// offset, rounded.  Converting hi from fp32 and packing in one block of PTX takes 57
// cycles for 16 values of a warp (without the offset), pair by pair through fp16 82.
__device__ __forceinline__ void split_p(float a, float b, float c, float d, uint32_t offset,
                                        uint32_t& hi, uint32_t& lo) {
  asm("{\n\t.reg .b16 p, q, r, s;\n\t.reg .b32 x, y, u, v;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 p, %3, %2;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 q, %5, %4;\n\t"
      "mov.b32 %0, {p, q};\n\t"
      "cvt.rn.f16x2.f32 x, %3, %2;\n\t"
      "cvt.rn.f16x2.f32 y, %5, %4;\n\t"
      "cvt.rn.f16x2.e4m3x2 u, p;\n\t"
      "cvt.rn.f16x2.e4m3x2 v, q;\n\t"
      "sub.rn.f16x2 u, x, u;\n\t"
      "sub.rn.f16x2 v, y, v;\n\t"
      "fma.rn.f16x2 u, u, %6, %7;\n\t"
      "fma.rn.f16x2 v, v, %6, %7;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 r, u;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 s, v;\n\t"
      "mov.b32 %1, {r, s};\n\t}"
      : "=&r"(hi), "=r"(lo)
      : "f"(a), "f"(b), "f"(c), "f"(d), "r"(0x4C004C00u), "r"(offset));   // 16, 16
}

// a + b and a * b + c of two neighbouring values in one instruction, each rounded as by
// the scalar one (the warps' issue slots are 60 % taken: 278 -> 269 us for 1536 prefill
// tokens).
__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%2, %3};\n\t"
      "mov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b, float c0,
                                     float c1) {
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%2, %3};\n\t"
      "mov.b64 y, {%4, %4};\n\t"
      "mov.b64 z, {%5, %6};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
}

// One thread's share of a group's softmax: key (and at the end value dim) `key` of kH
// heads.  kSCols: S^T columns of one token, 32 where the query's hi and lo parts are
// added here; page_cols: columns of one page's S^T, page_p: bytes of its P^T.
template <int kNT, int kSCols, int page_cols, int page_p>
struct PageSoftmax {
  static constexpr int kH = Groups<kNT>::kHeads, kBatch = Groups<kNT>::kBatch;
  int gi, quarter, lane, key;
  uint32_t s_addr, acc_addr;   // this thread's lane of the group's S^T and O^T columns
  uint8_t* pj;                 // its P^T bytes
  float (*mx)[4];              // [kH][4]: batch maxima by quarter
  float (*lsum)[4];            // [kH][4]: running sums by quarter
  // nl: log2(vs) - M per head, the addend of u - M (0 until the token has seen a
  // key); lv: the log2(vs) in it.  l: this key slot's share of the running sums.
  float nl[kH], l[kH];
  float lv;
  bool unset;
  // Once a wait has run out the warp waits for nothing any more but still takes
  // part in the group's barriers, so that its other warps get past them.
  bool ok;

  __device__ __forceinline__ void begin() {
    lv = 0.f;
    unset = true;
#pragma unroll
    for (int h = 0; h < kH; ++h) nl[h] = l[h] = 0.f;
  }

  // A batch of `have` pages (1 .. kBatch): S^T in buffer s_buf, complete at s_full's
  // phase s_par; P^T, free when o_done's phase o_par is complete (at once: first), is
  // announced on p_full.  zs: the token's logit scale; pos: its position.
  __device__ __forceinline__ void step(int s_buf, uint64_t* s_full, unsigned s_par,
                                       uint64_t* s_empty, const PageInfo* info, int have, float zs,
                                       int pos, uint64_t* o_done, unsigned o_par, bool first,
                                       uint64_t* p_full) {
    if (ok) ok = wait_for(s_full, s_par);
    tc::fence_after_thread_sync();
    float t[kBatch][kH], iv[kBatch];
    int lim[kBatch];   // keys <= lim are visible
    {
      uint32_t sv[kBatch][kH];
      const uint32_t at = s_addr + page_cols * kBatch * s_buf;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) ld_cols(at + page_cols * i, sv[i]);
      if constexpr (kSCols == 2 * kGroup) {
        uint32_t sl[kBatch][kH];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) ld_cols(at + page_cols * i + kGroup, sl[i]);
        tc::wait_ld();
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
#pragma unroll
          for (int h = 0; h < kH; h += 2)
            add2(t[i][h], t[i][h + 1], __uint_as_float(sv[i][h]), __uint_as_float(sv[i][h + 1]),
                 __uint_as_float(sl[i][h]), __uint_as_float(sl[i][h + 1]));
      } else {
        tc::wait_ld();
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
#pragma unroll
          for (int h = 0; h < kH; ++h) t[i][h] = __uint_as_float(sv[i][h]);
      }
    }
    tc::fence_before_thread_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(s_empty);
    // u - M + kPShift: the raw dot products times zt, plus nl
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const PageInfo in = info[i];
      const bool there = i < have;   // (the columns of an odd last page hold anything)
      const float zt = zs * in.k;
      if (there && in.lv != lv) {    // the same in every thread
        const float d = in.lv - lv;
#pragma unroll
        for (int h = 0; h < kH; h += 2) add2(nl[h], nl[h + 1], nl[h], nl[h + 1], d, d);
        lv = in.lv;
      }
      iv[i] = there ? in.iv : 0.f;
      lim[i] = !there || in.block < 0 ? -1 : pos - in.block * kPage;
#pragma unroll
      for (int h = 0; h < kH; h += 2)
        fma2(t[i][h], t[i][h + 1], t[i][h], t[i][h + 1], zt, nl[h], nl[h + 1]);
      if (lim[i] < kPage - 1 && key > lim[i]) {
#pragma unroll
        for (int h = 0; h < kH; ++h) t[i][h] = -INFINITY;
      }
#pragma unroll
      for (int h = 0; h < kH; h += 2) top = fmax3f(top, t[i][h], t[i][h + 1]);
    }
    bool stored = false, free_p = first;
    if (group_or<kNT>(gi, unset ? top > -INFINITY : top > kPTop)) {
      // set or move the references: the heads' maxima over the batch's keys
#pragma unroll
      for (int h = 0; h < kH; ++h) {
        const float m = warp_max_f32(fmaxf(t[0][h], t[kBatch - 1][h]));
        if (lane == h) mx[h][quarter] = m;
      }
      group_sync<kNT>(gi);
      // lane h (and h + kH ..): kPShift - the maximum where head h's reference moves, else 0
      float d_h, al_h;
      {
        const float4 m4 = *reinterpret_cast<const float4*>(mx[lane & (kH - 1)]);
        const float m = fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w));
        d_h = (unset || m > kPTop) && fabsf(m) < INFINITY ? kPShift - m : 0.f;
        al_h = ex2(d_h);
      }
#pragma unroll
      for (int h = 0; h < kH; ++h) {
        const float d = __shfl_sync(0xffffffffu, d_h, h);
        nl[h] += d;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) t[i][h] += d;
      }
      if (!unset) {
#pragma unroll
        for (int h = 0; h < kH; ++h) l[h] *= __shfl_sync(0xffffffffu, al_h, h);
        // the earlier products are relative to the old references (a token that
        // has seen no key has only zeros there): once they are complete, and
        // before this batch's, whose P is not written yet
        if (ok && !first) ok = wait_for(o_done, o_par);
        free_p = true;
        tc::fence_after_thread_sync();
#pragma unroll
        for (int c = 0; c < 2 * kH; c += 8) {   // the hi columns, then the lo ones
          const uint32_t at = acc_addr + c % kH + kGroup * (c / kH);
          uint32_t av[8];
          ld_cols(at, av);
          tc::wait_ld();
#pragma unroll
          for (int h = 0; h < 8; ++h)
            av[h] = __float_as_uint(__uint_as_float(av[h]) * __shfl_sync(0xffffffffu, al_h, c % kH + h));
          st_cols(at, av);
        }
        tc::wait_st();
        stored = true;
      }
      unset = false;
    }
    uint32_t hw[kBatch][kH / 4], lw[kBatch][kH / 4];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const uint32_t offset = split_offset(__brev(key), info[i].block);
#pragma unroll
      for (int q4 = 0; q4 < kH / 4; ++q4) {
        float* e = &t[i][4 * q4];
#pragma unroll
        for (int h = 0; h < 4; ++h) e[h] = ex2(e[h]);   // P; 0 for an invisible key
#pragma unroll
        for (int h = 0; h < 4; h += 2) {
          float* lh = &l[4 * q4 + h];
          fma2(lh[0], lh[1], e[h], e[h + 1], iv[i], lh[0], lh[1]);
        }
        split_p(e[0], e[1], e[2], e[3], offset, hw[i][q4], lw[i][q4]);
      }
    }
    // the P^T buffer was last read by the batch before
    if (ok && !free_p) ok = wait_for(o_done, o_par);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      store_p(pj + i * page_p, hw[i]);
      store_p(pj + i * page_p + 128, lw[i]);
    }
    tc::fence_proxy_async_smem();
    if (stored) tc::fence_before_thread_sync();   // the rescale before O^T
    __syncwarp();
    if (lane == 0) mbar_arrive(p_full);
  }

  // The token's sums (in l, every thread) and outputs o of value dim `key`, not yet
  // divided; any: it had pages, and o_done's phase o_par is its last product.
  __device__ __forceinline__ void finish(bool any, uint64_t* o_done, unsigned o_par,
                                         float (&o)[kH]) {
    // Running sums: 32 key slots a warp.  Each step halves the heads a lane keeps
    // (those whose index agrees with the lane in the step's bit), then the lanes
    // left with one head are summed.
    {
      float part[kH];
#pragma unroll
      for (int h = 0; h < kH; ++h) part[h] = l[h];
#pragma unroll
      for (int n = kH / 2; n >= 1; n >>= 1) {
        const bool up = (lane & n) != 0;
#pragma unroll
        for (int h = 0; h < n; ++h) {
          const float keep = up ? part[h + n] : part[h], give = up ? part[h] : part[h + n];
          part[h] = keep + __shfl_xor_sync(0xffffffffu, give, n);
        }
      }
#pragma unroll
      for (int off = kH; off < 32; off <<= 1)
        part[0] += __shfl_xor_sync(0xffffffffu, part[0], off);
      if (lane < kH) lsum[lane][quarter] = part[0];
    }
#pragma unroll
    for (int h = 0; h < kH; ++h) o[h] = 0.f;
    if (any) {
      if (ok) ok = wait_for(o_done, o_par);
      tc::fence_after_thread_sync();
      uint32_t ah[kH], al[kH];
      ld_cols(acc_addr, ah);
      ld_cols(acc_addr + kGroup, al);
      tc::wait_ld();
      tc::fence_before_thread_sync();
#pragma unroll
      for (int h = 0; h < kH; ++h) o[h] = fmaf(__uint_as_float(al[h]), kLoUnit, __uint_as_float(ah[h]));
    }
    group_sync<kNT>(gi);
#pragma unroll
    for (int h = 0; h < kH; ++h) {
      const float4 l4 = *reinterpret_cast<const float4*>(lsum[h]);
      l[h] = (l4.x + l4.y) + (l4.z + l4.w);
      if (l[h] != l[h]) {   // a NaN logit: the whole row, whatever it is merged with
        l[h] = 1.f;
        o[h] = __uint_as_float(0x7FFFFFFFu);
      }
    }
  }

  // out[h] of the kH rows from `row` (rows of kHeadDim).
  __device__ __forceinline__ void write(uint16_t* out, int64_t row, float v_scale,
                                        const float (&o)[kH]) const {
#pragma unroll
    for (int h = 0; h < kH; ++h) {
      const float r = l[h] > 0.f ? o[h] * __fdividef(v_scale, l[h]) : 0.f;
      out[(row + h) * kHeadDim + key] = static_cast<uint16_t>(f32_to_bf16_bits(r));
    }
  }
};

}  // namespace paged
}  // namespace msa
