// msa_prefill.cuh -- what the kernels over every visible page of a prefill batch share
// (dense attention, the block scorer): how the work is cut over the CTAs, and the query
// tiles.
//
// A unit is a tile of 16 query tokens of one request and one KV head, 256 query rows that
// see the pages 0 .. pos / 128 of the tile's last token.  A unit's work is its pages (and
// kExtra steps for its query and its output); the units of all requests, in the order
// (request, KV head, tile), make one line of steps, and every CTA takes the same share of
// the line, whatever the lengths are: a unit that a share's end cuts is worked on by
// several CTAs, a range of its pages each.  A request's steps are a closed form of its
// lengths (tiles lie 16 tokens apart and pages 128 long, so the pages of tile t are
// floor((a + t) / 8) + 1), so a CTA finds its place by one scan over the requests and a
// search over one request's tiles, and nothing is planned on the host.
#pragma once

#include "msa_device.cuh"
#include "msa_launch.h"
#include "msa_tcgen05.cuh"

namespace msa {
namespace prefill {

constexpr int kTile = 16;               // query tokens of a unit
constexpr int kHalfTokens = 8;          // query tokens of one 128-row half

// mbar_wait with one try before the clock is read: most waits here find their phase
// complete.
__device__ __forceinline__ bool wait_for(uint64_t* bar, unsigned parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
  while (!mbar_try_wait_sleep(bar, parity, 1000000u))
    if (global_ns() - t0 > kWaitLimitNs) return false;
  return true;
}

// A request's query tokens, and whether they can be worked on.
struct Request {
  int start, ql, L;
  bool bad;
  __device__ __forceinline__ int ctx() const { return L - ql; }
  __device__ __forceinline__ int tiles() const { return (ql + kTile - 1) / kTile; }
};

__device__ __forceinline__ Request load_request(const PrefillParams& p, int b) {
  Request r;
  const int c0 = p.cu_q[b], c1 = p.cu_q[b + 1];
  r.L = p.seq_lens[b];
  r.start = c0;
  r.bad = c0 < 0 || c1 < c0 || c1 > p.T || r.L < 0 || (r.L > 0 && (r.L - 1) / kPage >= p.S) ||
          r.L < c1 - c0;
  r.ql = r.bad ? 0 : c1 - c0;
  return r;
}

// sum over u < y of floor(u / 8)
__device__ __forceinline__ int64_t eighths(int64_t y) {
  const int64_t q = y >> 3;
  return 4 * q * (q - 1) + (y & 7) * q;
}

// Pages that tile t of the request sees.
__device__ __forceinline__ int tile_pages(const Request& r, int t) {
  return (r.ctx() + min(kTile * (t + 1), r.ql) - 1) / kPage + 1;
}

// Steps of the request's first x tiles for one KV head.
__device__ __forceinline__ int64_t tile_steps(const Request& r, int x, int extra) {
  const int full = min(x, r.ql / kTile);       // tiles of 16 tokens
  const int64_t a = (r.ctx() + kTile - 1) / kTile;
  int64_t s = full + eighths(a + full) - eighths(a) + static_cast<int64_t>(extra) * x;
  if (x > full) s += (r.L - 1) / kPage + 1;
  return s;
}

// (a b - minus) / c of numbers that are not negative, by 32-bit division where they fit.
__device__ __forceinline__ int64_t scaled(int64_t a, int64_t b, int64_t c, int minus = 0) {
  if (a < (1 << 22) && b < 512 && c < (1ll << 31))
    return static_cast<uint32_t>(a * b - minus) / static_cast<uint32_t>(c);
  return (a * b - minus) / c;
}

// What one CTA works on next: pages n0 .. n1 - 1 of a unit.
struct Segment {
  int b, g;
  int tok0, ntok;       // the tile's first token and how many it has (0: no more segments)
  int pos0;             // position of the first token
  int n0, n1;
  int slot;             // where this part of a shared unit goes; -1: the unit is whole
};

// The CTA's share of the line of steps and its place in it.
struct Walk {
  int64_t w, w1;        // the steps [w, w1) are still to do
  int64_t total;
  int active;           // CTAs that have a share
  int b, g, t;
  int64_t s;            // steps of the current unit that lie before w
  Request r;
};

struct WalkScratch {
  int64_t part[32];
  Walk walk;
};

// Sets up scratch->walk for this CTA; every thread of the block calls it, and may use
// the scratch behind it.  min_steps: CTAs have shares of at least this many steps (fewer
// CTAs take part in little work).  Returns whether some request's lengths are bad.
template <int kThreads>
__device__ __forceinline__ bool plan_walk(const PrefillParams& p, int extra, int min_steps,
                                          WalkScratch* scratch) {
  constexpr int kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool bad = false;
  int64_t total = 0;
  // the line's length; a batch of at most kThreads requests is read once
  Request r;
  int64_t steps = 0, before = 0;
  auto scan = [&](int b) {     // steps of request b, of those before it in the chunk; chunk total
    r.ql = 0;
    r.bad = false;
    if (b < p.B) r = load_request(p, b);
    bad |= r.bad;
    steps = r.ql > 0 ? p.Hkv * tile_steps(r, r.tiles(), extra) : 0;
    int64_t x = steps;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();           // the scratch of the last chunk has been read
    if (lane == 31) scratch->part[warp] = x;
    __syncthreads();
    before = x - steps;
    int64_t all = 0;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const int64_t y = scratch->part[k];
      if (k < warp) before += y;
      all += y;
    }
    return all;
  };
  for (int b0 = 0; b0 < p.B; b0 += kThreads) total += scan(b0 + tid);
  int64_t active = total / min_steps;
  active = active < 1 ? 1 : (active < gridDim.x ? active : static_cast<int64_t>(gridDim.x));
  const int64_t c = blockIdx.x;
  const int64_t w0 = c < active ? scaled(total, c, active) : total;
  const int64_t w1 = c < active ? scaled(total, c + 1, active) : total;
  if (tid == 0) {
    scratch->walk.w = w0;
    scratch->walk.w1 = w1;
    scratch->walk.total = total;
    scratch->walk.active = static_cast<int>(active);
  }
  if (w0 < w1) {
    int64_t base = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
      const int64_t all = p.B > kThreads ? scan(b0 + tid) : total;
      const int64_t at = base + before;
      if (steps > 0 && w0 >= at && w0 < at + steps) {
        Walk& k = scratch->walk;
        const int64_t per_head = tile_steps(r, r.tiles(), extra);
        k.b = b0 + tid;
        k.r = r;
        k.g = static_cast<int>(scaled(w0 - at, 1, per_head));
        const int64_t in = w0 - at - k.g * per_head;
        int x = 0, y = r.tiles();        // the last tile that begins at or before `in`
        while (y - x > 1) {
          const int m = (x + y) >> 1;
          if (tile_steps(r, m, extra) <= in) x = m;
          else y = m;
        }
        k.t = x;
        k.s = in - tile_steps(r, x, extra);
      }
      base += all;
    }
  }
  return __syncthreads_or(bad);
}

// The next segment of the walk (one thread, or a warp alike); ntok 0 when the share is
// done.  first_cut: the unit starts here and other CTAs end it; `parts` of them in all,
// this one among them.
__device__ __forceinline__ Segment next_segment(const PrefillParams& p, Walk& k, int extra,
                                                bool& first_cut, int& parts) {
  Segment s;
  first_cut = false;
  parts = 0;
  s.ntok = 0;
  if (k.w >= k.w1) return s;
  const int np = tile_pages(k.r, k.t);
  const int64_t steps = np + extra;
  const int64_t s0 = k.s, s1 = min(steps, s0 + (k.w1 - k.w));
  s.b = k.b;
  s.g = k.g;
  s.tok0 = k.r.start + kTile * k.t;
  s.ntok = min(kTile, k.r.ql - kTile * k.t);
  s.pos0 = k.r.ctx() + kTile * k.t;
  // the extra steps come first
  s.n0 = static_cast<int>(max(s0 - extra, static_cast<int64_t>(0)));
  s.n1 = static_cast<int>(max(s1 - extra, static_cast<int64_t>(0)));
  s.slot = s0 == 0 && s1 == steps ? -1 : 2 * static_cast<int>(blockIdx.x) + (s0 == 0 ? 1 : 0);
  if (s0 == 0 && s1 < steps) {
    first_cut = true;
    // the CTA that has the unit's last step: the largest c with total c / active <= it
    const int64_t last = k.w + steps - 1;
    parts = static_cast<int>(scaled(last + 1, k.active, k.total, 1)) - static_cast<int>(blockIdx.x) + 1;
  }
  k.w += s1 - s0;
  k.s = s1;
  if (s1 == steps) {
    k.s = 0;
    if (++k.t == k.r.tiles()) {
      k.t = 0;
      if (++k.g == p.Hkv) {
        k.g = 0;
        if (k.w < k.w1)
          do {
            k.r = load_request(p, ++k.b);
          } while (k.r.ql == 0 && k.b + 1 < p.B);
      }
    }
  }
  return s;
}

// Rows that no unit writes, a CTA in turn: `fill(token)` for the tokens before the first
// and behind the last request's, and those of requests with bad lengths.  Every thread of
// the block calls it (and fill); `bad` as plan_walk returned it.
template <typename Fill>
__device__ __forceinline__ void fill_uncovered(const PrefillParams& p, bool bad, Fill&& fill) {
  const int first = p.B > 0 ? p.cu_q[0] : p.T, last = p.B > 0 ? p.cu_q[p.B] : p.T;
  const bool ends = first > 0 || last < p.T;
  if (!bad && !ends) return;
  if (threadIdx.x == 0) flag_error(p.err, MSA_ERR_SEQ_RANGE);
  for (int i = blockIdx.x; i < min(first, p.T); i += gridDim.x) fill(i);
  for (int64_t i = static_cast<int64_t>(max(last, 0)) + blockIdx.x; i < p.T; i += gridDim.x)
    fill(static_cast<int>(i));
  if (!bad) return;
  for (int b = 0; b < p.B; ++b) {
    if (!load_request(p, b).bad) continue;
    const int c0 = max(p.cu_q[b], 0), c1 = min(p.cu_q[b + 1], p.T);
    for (int64_t i = static_cast<int64_t>(c0) + blockIdx.x; i < c1; i += gridDim.x)
      fill(static_cast<int>(i));
  }
}

// One token's 16 query rows in a tile of 128-byte rows (swizzled): fp8 rows as stored, or
// bf16 rows as hi and lo parts, the parts and the factor 2^e those of store_query_e4m3.  A
// warp a token; a lane holds 8 elements of every other row (four of them with fp8 rows), so
// that loads and stores are whole lines.
struct QueryRows {
  uint4 v[8];

  __device__ __forceinline__ void load(const PrefillParams& p, int tok, int g, int lane) {
    const int64_t row = static_cast<int64_t>(tok) * p.Hq + g * kGroup;
    if (p.q8) {
      const uint8_t* at = p.q8 + row * kHeadDim + 16 * lane;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = __ldg(reinterpret_cast<const uint4*>(at + 512 * k));
    } else {
      const uint16_t* at = p.q + row * kHeadDim + 8 * lane;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = __ldg(reinterpret_cast<const uint4*>(at + 256 * k));
    }
  }

  // Eight bf16 values times sd: hi and lo parts.
  static __device__ __forceinline__ uint4 parts(uint4 v, float sd) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t h[2], l[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const float f[4] = {bf16_bits_to_f32(w[2 * x] & 0xFFFF) * sd,
                          __uint_as_float(w[2 * x] & 0xFFFF0000u) * sd,
                          bf16_bits_to_f32(w[2 * x + 1] & 0xFFFF) * sd,
                          __uint_as_float(w[2 * x + 1] & 0xFFFF0000u) * sd};
      split_e4m3x4(f, h[x], l[x]);
    }
    return make_uint4(h[0], h[1], l[0], l[1]);
  }

  // A bf16 row's values to their parts, in place: v[k].x, .y hi and .z, .w lo of the lane's eight
  // elements.  Returns the dot products' factor.
  template <int kTurn>
  __device__ __forceinline__ float split(const PrefillParams& p) {
    if (p.q8) return p.logit_scale * p.q_scale;
    uint32_t m = 0;                       // the largest magnitudes as bf16 bits, two at a time
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      m = __vmaxu2(m, v[k].x & 0x7FFF7FFFu);
      m = __vmaxu2(m, v[k].y & 0x7FFF7FFFu);
      m = __vmaxu2(m, v[k].z & 0x7FFF7FFFu);
      m = __vmaxu2(m, v[k].w & 0x7FFF7FFFu);
    }
    const unsigned top = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
    const int biased = static_cast<int>(top >> 7);
    int e = (biased == 0 || biased == 0xFF) ? 0 : biased - 127 - 7;   // largest in [2^7, 2^8)
    e = e < -100 ? -100 : (e > 100 ? 100 : e);
    const float sd = exp2i(-e);
    // (in a loop, the array turned by kTurn at a time: in line it was 6 KiB of code a token, and the
    // warps of these kernels wait for instructions when their parts do not fit the SM's cache)
#pragma unroll 1
    for (int k = 0; k < 8; k += kTurn) {
      uint4 r[kTurn];
#pragma unroll
      for (int x = 0; x < kTurn; ++x) r[x] = parts(v[x], sd);
#pragma unroll
      for (int x = 0; x < 8; ++x) v[x] = x + kTurn < 8 ? v[x + kTurn] : r[x + kTurn - 8];
    }
    return p.logit_scale * exp2i(e);
  }

  // Into rows row0 .. row0 + 15 of `hi` (and `lo`).
  __device__ __forceinline__ void store(const PrefillParams& p, int row0, uint8_t* hi, uint8_t* lo,
                                        int lane) const {
    if (p.q8) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<uint4*>(hi + sw128(row0 + 4 * k + (lane >> 3), lane & 7)) = v[k];
      return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int off = sw128(row0 + 2 * k + (lane >> 4), (lane & 15) >> 1) + 8 * (lane & 1);
      *reinterpret_cast<uint2*>(hi + off) = make_uint2(v[k].x, v[k].y);
      *reinterpret_cast<uint2*>(lo + off) = make_uint2(v[k].z, v[k].w);
    }
  }
};

// Tokens first, first + step .. of a unit's query tile (two halves of 8 tokens, hi and lo
// parts, kHalfTile bytes each; rows of tokens that are not there are 0) and their dot
// products' factors zs[16].  One warp, which takes at most kMost tokens; wait() returns,
// false to give up, when the tile's last readers are through: the rows are loaded and split
// by then.
template <int kMost, int kTurn, typename Wait>
__device__ __forceinline__ bool load_query_tile(const PrefillParams& p, const Segment& sg, int first,
                                                int step, uint8_t* tile, float* zs, int lane,
                                                Wait&& wait) {
  constexpr int kAhead = kMost < 2 ? kMost : 2;    // tokens in registers at a time
  QueryRows rows[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (first + k * step < sg.ntok) rows[k].load(p, sg.tok0 + first + k * step, sg.g, lane);
#pragma unroll 1
  for (int j0 = first; j0 < kTile; j0 += kAhead * step) {
    float z[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (j0 + k * step < sg.ntok) z[k] = rows[k].split<kTurn>(p);
    if (j0 == first && !wait()) return false;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int j = j0 + k * step;
      if (j >= kTile) break;
      uint8_t* hi = tile + (j / kHalfTokens) * (2 * kHalfTile);
      uint8_t* lo = hi + kHalfTile;
      const int row0 = kGroup * (j % kHalfTokens);
      if (j < sg.ntok) {
        rows[k].store(p, row0, hi, lo, lane);
        if (lane == 0) zs[j] = z[k];
        if (kMost > kAhead && j + kAhead * step < sg.ntok)
          rows[k].load(p, sg.tok0 + j + kAhead * step, sg.g, lane);
      } else if (j < kHalfTokens || sg.ntok > kHalfTokens) {   // (a half without tokens is not read)
        zero_query_rows(row0, hi, lane);
        if (!p.q8) zero_query_rows(row0, lo, lane);
        if (lane == 0) zs[j] = 0.f;
      }
    }
  }
  tc::fence_proxy_async_smem();   // read by the tensor core
  __syncwarp();
  return true;
}

}  // namespace prefill
}  // namespace msa
