// glq_step.hip -- what a serving step does around the compressed linears and the
// paged cache (gfx950), and its entry points of the C ABI.
//
// Kernels:
//   kv_plan_k        request lengths -> pages taken, slots, positions, offsets
//   qk_norm_rope_k   norms of query and key heads, rotation, write into the cache
//   route_pick_k     router scores -> each token's experts and weights
//   route_group_k    for very many tokens: counts of groups of workgroups
//   route_place_k    rows in the experts' order, for more tokens than one workgroup takes
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "glq.h"
#include "glq_cache.h"
#include "glq_fwht.h"

namespace glq {
namespace {

// Largest of x over the 64 lanes of a wave, in every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  x = row_max<32>(x);
  const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return r[0] > r[1] ? r[0] : r[1];
}

// Sum of x over LPR lanes (8, 16, 32 or 64 of them in a row), in every one of them.
template <int LPR> __device__ __forceinline__ float lanes_sum(float x) {
  auto moved = [](float v, auto ctrl) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), decltype(ctrl)::value, 0xF, 0xF, false));
  };
  x += moved(x, std::integral_constant<int, 0xB1>());          // quad_perm: lane ^ 1, lane ^ 2
  x += moved(x, std::integral_constant<int, 0x4E>());
  x += moved(x, std::integral_constant<int, 0x141>());         // half row mirror: the other four
  if constexpr (LPR >= 16) x += moved(x, std::integral_constant<int, 0x140>());   // row mirror
  if constexpr (LPR >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (LPR == 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return x;
}

// ------------------------------------------------------------ pages and slots

struct PlanArgs {
  const int32_t *lens, *added, *free_pages;
  int32_t *table, *new_lens, *cu_q, *slots, *positions, *cu_k, *read_slots, *used;
  int64_t batch, max_pages, num_free, num_pages, max_tokens, max_read;
  int32_t page_shift;
  uint32_t q_tiles, r_tiles, p_groups;     // workgroups of the three lists
};

constexpr int kPlanThreads = 256, kPlanChunk = 1024;

enum PlanList { kNew, kRead, kPages };
// entries of a workgroup's tile: one page a thread, whose writes are scattered, eight tokens
constexpr int kPlanEach = 8, kPlanPages = kPlanThreads, kPlanTokens = kPlanEach * kPlanThreads;

// Sums that stop at 2^31 - 1: no list is longer, and what begins there is past its end.
__device__ __forceinline__ int32_t capped(int32_t x, int32_t y) {
  const uint32_t s = (uint32_t)x + (uint32_t)y;
  return s < 0x7FFFFFFFu ? (int32_t)s : INT32_MAX;
}
__device__ __forceinline__ int32_t capped_scan(int32_t x) {    // inclusive, over the lanes of a wave
  x = capped(x, __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false));    // row_shr 1, 2, 4, 8
  x = capped(x, __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false));
  x = capped(x, __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false));
  x = capped(x, __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false));
  x = capped(x, __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false));    // row_bcast 15 into rows 1 and 3
  x = capped(x, __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false));    // row_bcast 31 into rows 2 and 3
  return x;
}

struct PlanShared {
  int32_t begin[kPlanChunk], taken[kPlanChunk];      // entries of the list and pages before a request
  int32_t len[kPlanChunk], held[kPlanChunk];
  int32_t wave_sum[2][kPlanThreads / 64];
};

// Every workgroup writes one tile of one of three lists: the new tokens' slots
// and positions, all cached tokens' slots, the pages taken. It sums up the requests'
// counts itself (1024 requests at a time), which costs less than a launch that would do it for all; an
// entry finds its request by bisection in LDS. A page taken in this call is read from the list of free pages,
// never from the table, so no workgroup waits for another. In a tile of up to 1024 entries threads take one at a time; in a fuller one a
// thread has 8 neighbouring entries, found by one bisection and a few steps, their pages asked for together (300 and 1024
// requests with one new token 4.3 and 6.1 us one at a time, 6.2 and 6.6 by eights; 32 requests of 4096 new tokens in all
// and 64 of 16384, all read back, 8.4 and 9.8 against 5.7 and 6.0).
// Bound by latency: launch, lengths, sums and bisection, pages: 3.2 us for 32 requests with one new token, 6.0 for 64 with 16384
// new tokens and all of 145,000 read back.
// Returns the number of entries that the list has in all (the tokens lists: counted as far as the tile).
template <PlanList LIST>
__device__ __forceinline__ int32_t plan_tile(const PlanArgs &a, PlanShared &sh, int64_t tile, bool first) {
  auto &begin = sh.begin, &taken = sh.taken, &len = sh.len, &held = sh.held;
  auto &wave_sum = sh.wave_sum;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int32_t most = LIST == kNew ? (int32_t)a.max_tokens : LIST == kRead ? (int32_t)a.max_read : INT32_MAX;
  constexpr int TILE = LIST == kPages ? kPlanPages : kPlanTokens;
  const int32_t t0 = tile < INT32_MAX / TILE ? (int32_t)tile * TILE : INT32_MAX;
  const int32_t t1 = most - t0 < TILE ? (most > t0 ? most : t0) : t0 + TILE;
  const int32_t page = 1 << a.page_shift, max_pages = (int32_t)a.max_pages, num_free = (int32_t)a.num_free;
  auto pages_of = [&](int64_t tokens) {
    const int64_t p = (tokens + page - 1) >> a.page_shift;
    return p < max_pages ? (int32_t)p : max_pages;
  };
  int32_t before = 0, pages_before = 0;                        // of the chunks behind
  for (int64_t c = 0; c < a.batch; c += kPlanChunk) {
    if (LIST != kPages && !first && before >= t1) break;       // uniform
    const int n_here = a.batch - c < kPlanChunk ? (int)(a.batch - c) : kPlanChunk;
    int32_t n[4], p[4], l[4], h[4], nsum = 0, psum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = 4 * tid + i;
      const int32_t x = at < n_here ? a.lens[c + at] : 0, y = at < n_here ? a.added[c + at] : 0;
      l[i] = x > 0 ? x : 0;
      n[i] = y > 0 ? y : 0;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int32_t ph = pages_of(l[i]), pt = pages_of((int64_t)l[i] + n[i]), all = capped(l[i], n[i]);
      if (LIST == kNew && first && 4 * tid + i < n_here) a.new_lens[c + 4 * tid + i] = all;
      const int32_t mine = LIST == kNew ? n[i] : LIST == kRead ? all : pt - ph;
      h[i] = ph;
      p[i] = psum, n[i] = nsum;
      psum = capped(psum, pt - ph), nsum = capped(nsum, mine);
    }
    const int32_t nup = capped_scan(nsum), pup = capped_scan(psum);
    // (sums up to the lane before: the cap is never taken off)
    const int32_t nlow = __builtin_amdgcn_update_dpp(0, nup, 0x138, 0xF, 0xF, false);    // wave_shr 1
    const int32_t plow = __builtin_amdgcn_update_dpp(0, pup, 0x138, 0xF, 0xF, false);
    __syncthreads();                                           // the chunk before is done with LDS
    if (lane == 63) wave_sum[0][wave] = nup, wave_sum[1][wave] = pup;
    __syncthreads();
    int32_t nbase = before, pbase = pages_before, ntotal = before, ptotal = pages_before;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 64; ++w) {
      if (w < wave) nbase = capped(nbase, wave_sum[0][w]), pbase = capped(pbase, wave_sum[1][w]);
      ntotal = capped(ntotal, wave_sum[0][w]), ptotal = capped(ptotal, wave_sum[1][w]);
    }
    nbase = capped(nbase, nlow), pbase = capped(pbase, plow);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = 4 * tid + i;
      const int32_t start = capped(nbase, n[i]);
      begin[at] = at < n_here ? start : INT32_MAX;
      taken[at] = capped(pbase, p[i]);
      len[at] = l[i];
      held[at] = h[i];
      if (LIST != kPages && first && at < n_here) (LIST == kNew ? a.cu_q : a.cu_k)[c + at] = start < most ? start : most;
    }
    __syncthreads();
    const int32_t from = t0 > before ? t0 : before, end = ntotal < t1 ? ntotal : t1;
    int top = 1;                                               // a power of two that holds the requests
    while (top < n_here) top <<= 1;
    auto entry = [&](auto per, int32_t i0) {                   // entries i0 .. i0 + PER - 1 within from .. end
      constexpr int PER = decltype(per)::value;
      int at = 0;                                              // the last request that begins at the first of them or before
      const int32_t i1 = i0 > from ? i0 : from;
      for (int s = top >> 1; s; s >>= 1)
        if (begin[at + s] <= i1) at += s;
      // what the request is, read again only where the next one begins
      int32_t b0, b1, ln, hd, tk;
      auto look = [&] { b0 = begin[at], b1 = at + 1 < n_here ? begin[at + 1] : INT32_MAX, ln = len[at], hd = held[at], tk = taken[at]; };
      look();
      const int32_t *src[PER];
      int32_t pg[PER], in[PER];
      bool is[PER];
#pragma unroll
      for (int x = 0; x < PER; ++x) {
        const int32_t i = i0 + x;
        if constexpr (PER > 1)
          while (b1 <= i && at + 1 < n_here) ++at, look();
        const int32_t nth = i - b0;
        if constexpr (LIST == kPages) {
          if (i >= from && i < end) a.table[(c + at) * a.max_pages + hd + nth] = i < num_free ? a.free_pages[i] : -1;
        } else {
          const int64_t t = LIST == kNew ? (int64_t)ln + nth : nth, e = t >> a.page_shift, f = tk + e - hd;
          in[x] = t < INT32_MAX ? (int32_t)t : INT32_MAX;
          const bool here = i >= from && i < end, old = e < hd;
          is[x] = here && (old || (e < max_pages && f < num_free));
          src[x] = !is[x] ? a.lens : old ? a.table + (c + at) * a.max_pages + e : a.free_pages + f;   // (some word, not used)
        }
      }
      if constexpr (LIST != kPages) {
#pragma unroll
        for (int x = 0; x < PER; ++x) pg[x] = *src[x];         // all in flight together
#pragma unroll
        for (int x = 0; x < PER; ++x) pg[x] = is[x] ? pg[x] : -1;
      }
      if constexpr (LIST != kPages) {
        int32_t slot[PER];
#pragma unroll
        for (int x = 0; x < PER; ++x)
          slot[x] = pg[x] >= 0 && pg[x] < a.num_pages ? (pg[x] << a.page_shift) + (in[x] & (page - 1)) : -1;
        int32_t *list = LIST == kNew ? a.slots : a.read_slots;
        const bool whole = PER == kPlanEach && i0 >= from && i0 + PER <= end &&
                           ((reinterpret_cast<uintptr_t>(list) | (LIST == kNew ? reinterpret_cast<uintptr_t>(a.positions) : 0)) & 15) == 0;
        if constexpr (PER == kPlanEach) {
          if (whole) {
#pragma unroll
            for (int x = 0; x < PER; x += 4) {
              *reinterpret_cast<int4 *>(list + i0 + x) = make_int4(slot[x], slot[x + 1], slot[x + 2], slot[x + 3]);
              if constexpr (LIST == kNew)
                *reinterpret_cast<int4 *>(a.positions + i0 + x) = make_int4(in[x], in[x + 1], in[x + 2], in[x + 3]);
            }
          }
        }
        if (!whole)
#pragma unroll
          for (int x = 0; x < PER; ++x)
            if (i0 + x >= from && i0 + x < end) {
              list[i0 + x] = slot[x];
              if constexpr (LIST == kNew) a.positions[i0 + x] = in[x];
            }
      }
    };
    if (LIST == kPages || end - from <= 4 * kPlanThreads) {
      for (int32_t i = from + tid; i < end; i += kPlanThreads) entry(std::integral_constant<int, 1>(), i);
    } else {
      entry(std::integral_constant<int, kPlanEach>(), t0 + kPlanEach * tid);
    }
    before = ntotal;
    pages_before = ptotal;
  }
  if constexpr (LIST == kPages) {
    if (first && tid == 0) *a.used = before;
  } else {
    if (first && tid == 0) (LIST == kNew ? a.cu_q : a.cu_k)[a.batch] = before < most ? before : most;
    for (int32_t i = (t0 > before ? t0 : before) + tid; i < t1; i += kPlanThreads) {   // behind the last token
      if constexpr (LIST == kNew) a.slots[i] = -1, a.positions[i] = 0;
      else a.read_slots[i] = -1;
    }
  }
  return before;
}

__global__ void __launch_bounds__(kPlanThreads) kv_plan_k(PlanArgs a) {
  __shared__ PlanShared sh;
  const uint32_t g = blockIdx.x;
  if (g < a.q_tiles) {
    plan_tile<kNew>(a, sh, g, g == 0);
  } else if (g < a.q_tiles + a.r_tiles) {
    plan_tile<kRead>(a, sh, g - a.q_tiles, g == a.q_tiles);
  } else {
    // one tile each where no more than max_tokens are new; the lengths alone say how many pages there are
    const int64_t mine = g - a.q_tiles - a.r_tiles;
    for (int64_t tile = mine;; tile += a.p_groups)
      if (plan_tile<kPages>(a, sh, tile, tile == 0) <= (tile + a.p_groups) * kPlanPages) break;     // (ends: entries are below 2^31)
  }
}

// ------------------------------------------------------------ head norms and rotation

struct NormArgs {
  const void *q, *k;
  void *q_out, *k_out;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;
  const float *q_weight, *k_weight, *rotary;
  const int32_t *positions;
  int64_t max_positions;
  uint32_t groups, units;            // groups of D / 8 lanes, of which a token has `units`
  int32_t q_heads, rot;
  float eps;
  KvIo io;                           // the cache, and v as its dense[1]
};

constexpr int kNoCache = -1;

// Lanes hold 8 elements of a head's row each, D / 8 lanes a row: the mean of squares is a
// sum over those lanes, the partner of an element i of a half rotation (i + rot / 2) is
// in the lane rot / 16 further, that of a pair rotation in the same lane. Values are float32
// until the one rounding to the operands' type; the cache gets the rounded key, as
// if it were appended afterwards. The lanes of a row take HB heads of one kind (queries, keys or values) of a token, whose
// loads are in flight together and share the angles and the weights. 8192 tokens, 32 on 8 heads of 128 in bf16 with the write into a
// bf16 cache: 48 us from tensors that no cache holds, 4.7 TB/s, bound by what it reads and writes; 39 on the same tensors again, where the VALU is 94%
// busy. 32 tokens 4.2 us, launch and two loads one after the other.
template <int FMT, int D, bool F32, bool PAIRS, int HB>
__global__ void __launch_bounds__(256) qk_norm_rope_k(NormArgs a) {
  constexpr int LPR = D / 8, ES = F32 ? 4 : 2;
  const uint32_t g = (blockIdx.x * 256u + threadIdx.x) / LPR;
  if (g >= a.groups) return;                          // whole rows leave together
  const int at = threadIdx.x % LPR, kv_heads = a.io.heads;
  const int64_t token = g / a.units;
  const int u = (int)(g - (uint32_t)token * a.units);
  const int q_units = (a.q_heads + HB - 1) / HB, kv_units = (kv_heads + HB - 1) / HB;
  const int which = u < q_units ? 0 : u < q_units + kv_units ? 1 : 2;                // query, key, value
  const int h0 = (which == 0 ? u : which == 1 ? u - q_units : u - q_units - kv_units) * HB;
  const int heads = (which == 0 ? a.q_heads : kv_heads) - h0;                        // the unit has min(this, HB)
  const uint8_t *from = reinterpret_cast<const uint8_t *>(which == 0 ? a.q : which == 1 ? a.k : a.io.dense[1]) +
                        ES * (token * (which == 0 ? a.q_stride : which == 1 ? a.k_stride : a.io.stride[1]) + (int64_t)h0 * D + 8 * at);
  float x[HB][8];
#pragma unroll
  for (int i = 0; i < HB; ++i) load8<F32>(from + ES * D * (i < heads ? i : 0), x[i]);
  if (which < 2) {
    const float *weight = which == 0 ? a.q_weight : a.k_weight;
    const bool in = 8 * at < a.rot;
    const int half = a.rot / 16;                      // lanes of one half
    const bool upper = at >= half;
    constexpr int ANGLES = PAIRS ? 4 : 8;
    float cs[ANGLES], sn[ANGLES], w[8];
    if (a.rot > 0) {
      int64_t p = a.positions[token];
      p = p < 0 ? 0 : p < a.max_positions ? p : a.max_positions - 1;
      const float *row = a.rotary + p * a.rot + (!in ? 0 : PAIRS ? 4 * at : 8 * (upper ? at - half : at));
#pragma unroll
      for (int i = 0; i < ANGLES; i += 4) {
        const float4 c = *reinterpret_cast<const float4 *>(row + i), s = *reinterpret_cast<const float4 *>(row + a.rot / 2 + i);
        cs[i] = c.x, cs[i + 1] = c.y, cs[i + 2] = c.z, cs[i + 3] = c.w;
        sn[i] = s.x, sn[i + 1] = s.y, sn[i + 2] = s.z, sn[i + 3] = s.w;
      }
#pragma unroll
      for (int i = 0; i < ANGLES; ++i) {
        cs[i] = in ? cs[i] : 1.0f;                    // (lanes past the rotated dimensions)
        sn[i] = !in ? 0.0f : PAIRS || upper ? sn[i] : -sn[i];
      }
    }
    if (weight) load8<true>(weight + 8 * at, w);
#pragma unroll
    for (int i = 0; i < HB; ++i) {
      if (weight) {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(x[i][j], x[i][j], s);
        s = lanes_sum<LPR>(s);
        const float r = 1.0f / sqrtf(s / (float)D + a.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[i][j] *= w[j] * r;
      }
      if (a.rot > 0) {
        if constexpr (PAIRS) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float c = x[i][2 * j], d = x[i][2 * j + 1];
            x[i][2 * j] = in ? c * cs[j] - d * sn[j] : c;
            x[i][2 * j + 1] = in ? d * cs[j] + c * sn[j] : d;
          }
        } else {
          float y[8];
          if (a.rot == D) {                           // the lane half a row away, without a trip through LDS
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = lane_xor(x[i][j], LPR / 2);
          } else {
            const int other = in ? (upper ? threadIdx.x - half : threadIdx.x + half) : threadIdx.x;
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = __shfl(x[i][j], other & 63);
          }
          // (selected, not multiplied by cos = 1 and sin = 0: what is not finite in lanes past the rotation stays as it is)
#pragma unroll
          for (int j = 0; j < 8; ++j) x[i][j] = in ? x[i][j] * cs[j] + y[j] * sn[j] : x[i][j];
        }
      }
      if constexpr (!F32) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const uint32_t two = pack_bf16(x[i][j], x[i][j + 1]);
          x[i][j] = bf16_lo(two), x[i][j + 1] = bf16_hi(two);
        }
      }
    }
    uint8_t *to = reinterpret_cast<uint8_t *>(which == 0 ? a.q_out : a.k_out);
    if (to) {
      to += ES * (token * (which == 0 ? a.q_out_stride : a.k_out_stride) + (int64_t)h0 * D + 8 * at);
#pragma unroll
      for (int i = 0; i < HB; ++i)
        if (i < heads) store8<F32>(to + ES * D * i, x[i]);
    }
  }
  if constexpr (FMT != kNoCache) {
    if (which > 0) {
      KvPart<D> part;
      part.slot = (uint32_t)a.io.slots[token];
      if (part.slot < a.io.capacity) {
        const uint32_t pg = part.slot >> a.io.page_shift, in_page = part.slot & ((1u << a.io.page_shift) - 1);
#pragma unroll
        for (int i = 0; i < HB; ++i) {
          if (i >= heads) break;
          part.cached = (((int64_t)pg * kv_heads + h0 + i) << a.io.page_shift) + in_page;
          append_row<FMT, D>(a.io, part, which - 1, at, x[i]);
        }
      }
    }
  }
}

// ------------------------------------------------------------ routing

struct RouteArgs {
  const void *logits;
  int64_t tokens, blocks, groups;                  // groups of blocks that counts are summed up for, 0: none
  int32_t experts, top, each;                      // tokens a block
  int32_t normalize;
  float *weights;
  int32_t *ids, *pos, *src, *offsets, *counts;     // counts [blocks][experts], then [groups][experts], workspace
};

// Tokens a workgroup, a multiple of its waves. Up to 64 tokens take one workgroup, with as few a wave as they need (16 of 64 experts' tokens
// 4.0 us, in the form for 64 7.4). Beyond, few tokens each make the choice short and more counts to add up: 8 of 128
// experts, choice and rows for 16, 32 and 64 tokens each: 500 tokens 9.3, 10.7 and 15.7 us, 2048: 9.8, 11.4 and 15.8, 4096 of 1024 experts:
// 34, 31 and 40, 8192 of 128: 19.2, 13.5 and 16.6. Adding up all counts in each workgroup grows with the square of
// the tokens (32768: 137, 54 and 33), so past 512 workgroups groups of 256 of them are added up first, in a launch between.
constexpr int kRouteAlone = 64, kRouteThreads = 1024, kRouteMost = 1024, kRouteGroup = 256;
constexpr int64_t kRouteShort = 2048, kRouteMiddle = 16384, kRoutePlain = 512;
inline int route_each(int64_t tokens) {
  if (tokens <= kRouteAlone) return tokens <= 16 ? 16 : tokens <= 32 ? 32 : 64;
  return tokens <= kRouteShort ? 16 : tokens <= kRouteMiddle ? 32 : 64;
}
inline int64_t route_blocks(int64_t tokens) {
  const int each = route_each(tokens);
  return tokens < each ? 1 : (tokens + each - 1) / each;
}
inline int64_t route_groups(int64_t tokens) {
  return route_blocks(tokens) <= kRoutePlain ? 0 : (route_blocks(tokens) + kRouteGroup - 1) / kRouteGroup;
}

// Order of scores as unsigned numbers, 0 for those that choose nothing (-inf, NaN); both zeros are one.
__device__ __forceinline__ uint32_t score_order(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  if (!(x > -INFINITY)) return 0u;
  return (int32_t)u < 0 ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float score_of(uint32_t order) {    // (order > 0)
  return __uint_as_float((int32_t)order < 0 ? order & 0x7FFFFFFFu : ~order);
}

// Exclusive sums of one number a thread over the workgroup's threads; total in *sum.
__device__ __forceinline__ int32_t group_before(int32_t x, int32_t *sum) {
  __shared__ int32_t part[kRouteThreads / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t up = wave_scan<false>(x);
  if (lane == 63) part[wave] = up;
  __syncthreads();
  int32_t base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kRouteThreads / 64; ++w) {
    if (w < wave) base += part[w];
    all += part[w];
  }
  *sum = all;
  return base + up - x;
}

// A wave takes a token, its lanes experts lane, lane + 64, ...: `top` times the largest
// score left, the lowest index among equals. Up to 64 tokens a workgroup: who chose an
// expert is a mask of 64 bits in LDS (or-ed in any order, the same whatever it is), so
// a choice's place among the workgroup's is the number of lower bits, and nothing
// depends on which wave comes first. One workgroup alone (up to 64 tokens) goes on
// to the rows itself: one launch. Bound by the VALU work of `top` maxima over the wave, each of lane exchanges and a ballot: 4.5 us
// for a token a wave with 8 of 128 experts, 7.7 for two, of which the launch and the scores are 2.5; 10^6 tokens 430 us,
// 1.3 TB/s of scores and choices.
template <int NV, bool F32, int TOKENS>
__global__ void __launch_bounds__(kRouteThreads) route_pick_k(RouteArgs a) {
  __shared__ unsigned long long chose[kRouteMost];
  __shared__ int32_t first[kRouteMost];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e < a.experts; e += kRouteThreads) chose[e] = 0;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * TOKENS;
  constexpr int WAVES = kRouteThreads / 64, PER = TOKENS / WAVES;        // tokens wave, wave + WAVES, ...
  // The tokens of a wave side by side, so that their chains of maxima overlap. A score that is not chosen yet is its order.
  int32_t mine[PER];                                           // lane j: the token's choice j
  float value[PER], peak[PER];                                 // its score; the largest one
  uint32_t order[PER][NV];
  float x[PER][NV];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int64_t t = t0 + wave + i * WAVES;
    mine[i] = -1, value[i] = -INFINITY, peak[i] = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = lane + 64 * v;
      x[i][v] = -INFINITY;
      if (e < a.experts && t < a.tokens) {
        const size_t o = (size_t)t * a.experts + e;
        x[i][v] = F32 ? reinterpret_cast<const float *>(a.logits)[o]
                      : __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(a.logits)[o] << 16);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)
#pragma unroll
    for (int v = 0; v < NV; ++v) order[i][v] = score_order(x[i][v]);
  for (int j = 0; j < a.top; ++j) {
    uint32_t best[PER], any = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      best[i] = 0;
#pragma unroll
      for (int v = 0; v < NV; ++v) best[i] = order[i][v] > best[i] ? order[i][v] : best[i];
      best[i] = wave_max(best[i]);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      best[i] = __builtin_amdgcn_readfirstlane((int)best[i]);
      any |= best[i];
    }
    if (any == 0) break;                                       // uniform: nothing left of any token
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      int e = -1;                                              // the lowest index among equals: first v, then lane
#pragma unroll
      for (int v = NV - 1; v >= 0; --v) {
        const unsigned long long hit = __ballot(order[i][v] == best[i]);
        e = hit ? 64 * v + __ffsll((long long)hit) - 1 : e;
      }
      if (best[i] == 0) continue;                              // uniform: nothing left of this one
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (lane + 64 * v == e) order[i][v] = 0;
      const float s = score_of(best[i]);
      if (j == 0) peak[i] = s;
      if (lane == j) mine[i] = e, value[i] = s;
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int in = wave + i * WAVES;
    const int64_t t = t0 + in;
    if (t >= a.tokens) continue;                               // uniform
    const float w = mine[i] >= 0 ? expf(value[i] - peak[i]) : 0.0f;
    float sum = w;
    if (!a.normalize) {                                        // the others
#pragma unroll
      for (int v = 0; v < NV; ++v) sum += order[i][v] ? expf(score_of(order[i][v]) - peak[i]) : 0.0f;
    }
    sum = lanes_sum<64>(sum);
    if (lane < a.top) {
      a.weights[t * a.top + lane] = mine[i] >= 0 ? w / sum : 0.0f;
      a.ids[t * a.top + lane] = mine[i];
    }
    if (mine[i] >= 0) atomicOr(&chose[mine[i]], 1ull << in);
  }
  __syncthreads();
  const bool alone = gridDim.x == 1;
  int32_t total = 0;
  if (alone) {
    const int32_t count = tid < a.experts ? __popcll(chose[tid]) : 0;
    const int32_t before = group_before(count, &total);
    if (tid < a.experts) {
      first[tid] = before;
      a.offsets[tid] = before;
    }
    if (tid == 0) a.offsets[a.experts] = total;
    __syncthreads();
  } else {
    for (int e = tid; e < a.experts; e += kRouteThreads)
      a.counts[(size_t)blockIdx.x * a.experts + e] = __popcll(chose[e]);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int in = wave + i * WAVES;
    const int64_t t = t0 + in;
    if (t >= a.tokens || lane >= a.top) continue;
    int32_t at = -1;
    if (mine[i] >= 0) {
      at = __popcll(chose[mine[i]] & ((1ull << in) - 1));
      if (alone) {
        at += first[mine[i]];
        a.src[at] = (int32_t)t;
      }
    }
    a.pos[t * a.top + lane] = at;
  }
  if (alone)
    for (int64_t r = total + tid; r < a.tokens * a.top; r += kRouteThreads) a.src[r] = -1;
}

// Counts of kRouteGroup workgroups: their sum, and in place of each the sum of those before it in the group. The threads
// of an expert take a run of workgroups each, twice over.
__global__ void __launch_bounds__(kRouteThreads) route_group_k(RouteArgs a) {
  __shared__ int32_t sums[kRouteThreads];
  const int tid = threadIdx.x;
  int width = 1;                                               // experts up to a power of two
  while (width < a.experts) width <<= 1;
  const int parts = kRouteThreads / width, e = tid & (width - 1), part = tid / width;
  const int64_t first = (int64_t)blockIdx.x * kRouteGroup, left = a.blocks - first, n = left < kRouteGroup ? left : kRouteGroup;
  const int64_t b0 = first + n * part / parts, b1 = first + n * (part + 1) / parts;
  int32_t sum = 0;
  if (e < a.experts)
    for (int64_t b = b0; b < b1; ++b) sum += a.counts[b * a.experts + e];
  sums[tid] = sum;
  __syncthreads();
  if (e >= a.experts) return;
  int32_t before = 0, all = 0;
  for (int p = 0; p < parts; ++p) {
    const int32_t s = sums[e + p * width];
    all += s;
    if (p < part) before += s;
  }
  for (int64_t b = b0; b < b1; ++b) {
    const int32_t c = a.counts[b * a.experts + e];
    a.counts[b * a.experts + e] = before;
    before += c;
  }
  if (part == 0) a.counts[(a.blocks + blockIdx.x) * a.experts + e] = all;
}

// Rows of one workgroup's tokens: those of earlier workgroups and of earlier experts come
// before. Every workgroup adds up all counts, or those of the groups (256 by 128 of them for 8192 tokens and
// 128 experts, from L2), instead of a launch between the two that would.
__global__ void __launch_bounds__(kRouteThreads) route_place_k(RouteArgs a) {
  __shared__ int32_t sums[2][kRouteThreads];                   // before this workgroup's, and all
  __shared__ int32_t first[kRouteMost];
  const int tid = threadIdx.x;
  int width = 1;                                               // experts up to a power of two
  while (width < a.experts) width <<= 1;
  const int parts = kRouteThreads / width, e = tid & (width - 1), part = tid / width;
  const int32_t *counts = a.groups ? a.counts + a.blocks * a.experts : a.counts;
  const int64_t many = a.groups ? a.groups : a.blocks, mine = a.groups ? blockIdx.x / kRouteGroup : blockIdx.x;
  int32_t before = 0, all = 0;
  if (e < a.experts) {
    int64_t b = part;
    for (; b + 7 * parts < many; b += 8 * parts) {             // eight loads in flight
      int32_t n[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) n[i] = counts[(b + i * parts) * a.experts + e];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        all += n[i];
        if (b + i * parts < mine) before += n[i];
      }
    }
    for (; b < many; b += parts) {
      const int32_t n = counts[b * a.experts + e];
      all += n;
      if (b < mine) before += n;
    }
    if (a.groups && part == 0) before += a.counts[(int64_t)blockIdx.x * a.experts + e];      // of the group, before this one
  }
  sums[0][tid] = before, sums[1][tid] = all;
  __syncthreads();
  if (tid < width) {
    before = all = 0;
    for (int p = 0; p < parts; ++p) before += sums[0][tid + p * width], all += sums[1][tid + p * width];
  } else {
    before = all = 0;
  }
  int32_t total;
  const int32_t start = group_before(all, &total);
  if (tid < a.experts) {
    first[tid] = start + before;
    if (blockIdx.x == 0) a.offsets[tid] = start;
  }
  if (blockIdx.x == 0 && tid == 0) a.offsets[a.experts] = total;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * a.each;
  const int64_t n = (a.tokens - t0 < a.each ? a.tokens - t0 : a.each) * a.top;
  for (int64_t i = tid; i < n; i += kRouteThreads) {
    const int64_t o = t0 * a.top + i;
    const int32_t id = a.ids[o];
    if (id < 0) continue;
    const int32_t at = a.pos[o] + first[id];
    a.pos[o] = at;
    a.src[at] = (int32_t)(o / a.top);
  }
  for (int64_t r = total + (int64_t)blockIdx.x * kRouteThreads + tid; r < a.tokens * a.top;
       r += (int64_t)gridDim.x * kRouteThreads)
    a.src[r] = -1;
}

// ------------------------------------------------------------ argument checks and launches

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

template <int FMT, int D, bool F32, bool PAIRS, int HB>
int launch_norm_heads(NormArgs a, int64_t tokens, hipStream_t st) {
  const int64_t units = (a.q_heads + HB - 1) / HB + (FMT == kNoCache ? 1 : 2) * ((a.io.heads + HB - 1) / HB);
  const int64_t blocks = (tokens * units * (D / 8) + 255) / 256;
  if (blocks > kMaxGroups) return GLQ_ERR_UNSUPPORTED;
  a.units = (uint32_t)units, a.groups = (uint32_t)(tokens * units);
  hipLaunchKernelGGL((qk_norm_rope_k<FMT, D, F32, PAIRS, HB>), dim3((unsigned)blocks), dim3(256), 0, st, a);
  return hip_status(hipGetLastError(), "qk_norm_rope_k");
}

template <int FMT, int D, bool F32>
int launch_norm(const NormArgs &a, int64_t tokens, bool pairs, hipStream_t st) {
  // Several heads a row of lanes where four would leave every CU eight waves; two where rows become codes, whose maxima take
  // registers, and of float32, which has twice the loads in flight. One, two and four heads (us a call in a graph, three or four sets of
  // tensors in turn; 32 on 8 heads of 128, those of 16 on 4 of 256 are within 5% of them):
  //   bf16     8192 tokens without a cache 50.1, 44.3, 41.1, into bf16 60.8, 51.5, 50.6, int8 63.4, 51.5, 54.7, int4 62.7, 54.0, 53.2
  //            1024 tokens (the first with several) 9.2, 8.2, 8.6, and 10.0, 9.8, 10.0, and 10.8, 10.6, 12.3, and 10.8, 10.5, 12.4
  //            512 tokens (the last with one) 5.3, 5.5, 5.8, and 6.4, 6.4, 7.0, and 6.8, 7.1, 8.9, and 6.6, 7.2, 8.8
  //   float32  8192 tokens 69.9, 66.0, 67.8, into bf16 79.1, 77.2, 80.3, int8 80.1, 76.4, 79.4, int4 78.5, 75.1, 78.2
  //            1024 tokens 11.8, 11.7, 12.2, and 13.4, 12.8, 13.5, and 13.5, 13.6, 15.7, and 13.6, 13.5, 15.7
  // Heads of 64 gain later (32 on 8, bf16: 2048 tokens 9.1, 8.1, 8.6, into int8 10.7, 11.3, 12.6; 8192 24.9, 22.8, 21.2 and 34.7, 31.3, 34.2;
  // 16 on 2 of 64, float32 into int8, 8192 tokens: 19.4, 22.0, 20.2, the most that the rule loses).
  constexpr int HB = F32 || FMT == GLQ_KV_INT8 || FMT == GLQ_KV_INT4 ? 2 : 4;
  const int64_t heads = a.q_heads + (FMT == kNoCache ? 1 : 2) * a.io.heads;
  if (tokens * heads * (D / 8) >= (int64_t)256 * 8 * 64 * 4)
    return pairs ? launch_norm_heads<FMT, D, F32, true, HB>(a, tokens, st) : launch_norm_heads<FMT, D, F32, false, HB>(a, tokens, st);
  return pairs ? launch_norm_heads<FMT, D, F32, true, 1>(a, tokens, st) : launch_norm_heads<FMT, D, F32, false, 1>(a, tokens, st);
}

template <int FMT>
int launch_norm_dim(const NormArgs &a, int64_t tokens, int d, glq_dtype dt, bool pairs, hipStream_t st) {
  if (dt == GLQ_F32)
    return d == 64 ? launch_norm<FMT, 64, true>(a, tokens, pairs, st) : d == 128 ? launch_norm<FMT, 128, true>(a, tokens, pairs, st)
                                                                         : launch_norm<FMT, 256, true>(a, tokens, pairs, st);
  return d == 64 ? launch_norm<FMT, 64, false>(a, tokens, pairs, st) : d == 128 ? launch_norm<FMT, 128, false>(a, tokens, pairs, st)
                                                                        : launch_norm<FMT, 256, false>(a, tokens, pairs, st);
}

int check_route(int64_t tokens, int32_t experts, int32_t top) {
  if (tokens < 0 || experts < 1 || top < 1 || top > experts) return GLQ_ERR_ARG;
  if (experts > kRouteMost || top > 64 || tokens > 0x7FFFFFFF / 64) return GLQ_ERR_UNSUPPORTED;
  return GLQ_OK;
}

template <int NV, bool F32>
void launch_pick_tokens(const RouteArgs &a, hipStream_t st) {
  const dim3 grid((unsigned)a.blocks), block(kRouteThreads);
  if (a.each == 64) hipLaunchKernelGGL((route_pick_k<NV, F32, 64>), grid, block, 0, st, a);
  else if (a.each == 32) hipLaunchKernelGGL((route_pick_k<NV, F32, 32>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((route_pick_k<NV, F32, 16>), grid, block, 0, st, a);
}

template <int NV>
void launch_pick(const RouteArgs &a, glq_dtype dt, hipStream_t st) {
  if (dt == GLQ_F32) launch_pick_tokens<NV, true>(a, st);
  else launch_pick_tokens<NV, false>(a, st);
}

}  // namespace
}  // namespace glq

using namespace glq;

extern "C" int glq_kv_plan(const glq_plan *P, void *hip_stream) {
  if (!P || P->batch < 0 || P->max_pages < 1 || P->num_pages < 1 || P->num_free < 0 || P->max_tokens < 0 || P->max_read < 0)
    return GLQ_ERR_ARG;
  if (P->page_size < 16 || P->page_size > 1024 || (P->page_size & (P->page_size - 1))) return GLQ_ERR_ARG;
  const bool read = P->max_read > 0 || P->read_slots || P->cu_k;
  if (!P->cu_q || !P->used || (P->batch > 0 && (!P->lens || !P->added || !P->page_table || !P->new_lens))) return GLQ_ERR_ARG;
  if (P->num_free > 0 && !P->free_pages) return GLQ_ERR_ARG;
  if (P->max_tokens > 0 && (!P->slots || !P->positions)) return GLQ_ERR_ARG;
  if (read && (!P->cu_k || (P->max_read > 0 && !P->read_slots))) return GLQ_ERR_ARG;
  const void *const words[] = {P->lens, P->added, P->free_pages, P->page_table, P->new_lens, P->cu_q,
                               P->slots, P->positions, P->cu_k, P->read_slots, P->used};
  for (const void *p : words)
    if (!aligned4(p)) return GLQ_ERR_ARG;
  if (P->batch > 0 && (P->new_lens == P->lens || P->new_lens == P->added)) return GLQ_ERR_ARG;
  // (a tile's entries, and what lies a tile further, are numbered in 32 bits)
  constexpr int64_t most = 0x7FFFFFFF - 2 * kPlanTokens;
  if (P->num_pages > 0x7FFFFFFF / P->page_size || P->max_pages > 0x7FFFFFFF / P->page_size || P->max_tokens > most ||
      P->max_read > most || P->num_free > 0x7FFFFFFF || P->batch > most || (P->batch > 0 && P->max_pages > most / P->batch))
    return GLQ_ERR_UNSUPPORTED;
  auto tiles = [](int64_t n, int64_t each) { return (uint32_t)((n + each - 1) / each); };
  PlanArgs a = {P->lens, P->added, P->free_pages, P->page_table, P->new_lens, P->cu_q, P->slots, P->positions, P->cu_k,
                P->read_slots, P->used, P->batch, P->max_pages, P->num_free, P->num_pages, P->max_tokens, P->max_read,
                log2_of(P->page_size), 1, 0, 0};
  if (P->max_tokens > 0) a.q_tiles = tiles(P->max_tokens, kPlanTokens);
  if (read) a.r_tiles = P->max_read > 0 ? tiles(P->max_read, kPlanTokens) : 1;
  // pages that max_tokens new ones can take, as far as the table has room; without any, the workgroup that writes *used
  const int64_t taken = P->max_tokens / P->page_size + P->batch, room = P->batch * P->max_pages, pages = taken < room ? taken : room;
  a.p_groups = pages > 0 ? tiles(pages, kPlanPages) : 1;
  const int64_t groups = (int64_t)a.q_tiles + a.r_tiles + a.p_groups;
  if (groups > kMaxGroups) return GLQ_ERR_UNSUPPORTED;
  hipLaunchKernelGGL(kv_plan_k, dim3((unsigned)groups), dim3(kPlanThreads), 0, reinterpret_cast<hipStream_t>(hip_stream), a);
  return hip_status(hipGetLastError(), "kv_plan_k");
}

extern "C" int glq_qk_norm_rope(const glq_qk *N, const glq_kv_cache *C, uint32_t flags, void *hip_stream) {
  if (!N || (flags & ~(uint32_t)GLQ_ROPE_PAIRS) || !valid_dtype(N->dt) || N->tokens < 0) return GLQ_ERR_ARG;
  if (N->q_heads < 1 || N->kv_heads < 1 || N->rotary_dim < 0 || N->rotary_dim > N->head_dim) return GLQ_ERR_ARG;
  if (!std::isfinite(N->eps) || N->eps < 0.0f) return GLQ_ERR_ARG;
  if (!valid_dim(N->head_dim) || N->rotary_dim % 16 || N->q_heads > 65536 || N->kv_heads > 65536) return GLQ_ERR_UNSUPPORTED;
  if (C) {
    const int rc = check_cache(C);
    if (rc) return rc;
    if (C->kv_heads != N->kv_heads || C->head_dim != N->head_dim) return GLQ_ERR_ARG;
  }
  if (N->tokens == 0) return GLQ_OK;
  const int d = N->head_dim;
  if (!valid_rows(N->q, N->q_stride, N->q_heads, d, N->dt) || !valid_rows(N->q_out, N->q_out_stride, N->q_heads, d, N->dt) ||
      !valid_rows(N->k, N->k_stride, N->kv_heads, d, N->dt))
    return GLQ_ERR_ARG;
  if ((N->k_out || !C) && !valid_rows(N->k_out, N->k_out_stride, N->kv_heads, d, N->dt)) return GLQ_ERR_ARG;
  if ((N->q_out == N->q && N->q_out_stride != N->q_stride) || (N->k_out == N->k && N->k_out_stride != N->k_stride))
    return GLQ_ERR_ARG;
  if (C && (!valid_rows(N->v, N->v_stride, N->kv_heads, d, N->dt) || !N->slots || !aligned4(N->slots))) return GLQ_ERR_ARG;
  if (!aligned16(N->q_weight) || !aligned16(N->k_weight)) return GLQ_ERR_ARG;
  if (N->rotary_dim > 0 && (!N->positions || !aligned4(N->positions) || !N->rotary || !aligned16(N->rotary) || N->max_positions < 1))
    return GLQ_ERR_ARG;
  const int64_t heads = (int64_t)N->q_heads + N->kv_heads * (C ? 2 : 1);
  if (N->tokens > (int64_t(1) << 40) / heads) return GLQ_ERR_UNSUPPORTED;
  NormArgs a = {N->q, N->k, N->q_out, N->k_out, N->q_stride, N->k_stride, N->q_out_stride, N->k_out_stride,
                N->q_weight, N->k_weight, N->rotary, N->positions, N->max_positions, 0, 0, N->q_heads, N->rotary_dim, N->eps, {}};
  a.io.heads = N->kv_heads;
  const glq_dtype dt = (glq_dtype)N->dt;
  const bool pairs = flags & GLQ_ROPE_PAIRS;
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  if (!C) return launch_norm_dim<kNoCache>(a, N->tokens, d, dt, pairs, st);
  a.io.cache[0] = C->k, a.io.cache[1] = C->v;
  a.io.scale[0] = C->k_scale, a.io.scale[1] = C->v_scale;
  a.io.dense[1] = const_cast<void *>(N->v), a.io.stride[1] = N->v_stride;
  a.io.slots = N->slots;
  a.io.page_shift = log2_of(C->page_size), a.io.capacity = (uint32_t)(C->num_pages * C->page_size);
  switch (C->format) {
    case GLQ_KV_BF16: return launch_norm_dim<GLQ_KV_BF16>(a, N->tokens, d, dt, pairs, st);
    case GLQ_KV_INT8: return launch_norm_dim<GLQ_KV_INT8>(a, N->tokens, d, dt, pairs, st);
    default: return launch_norm_dim<GLQ_KV_INT4>(a, N->tokens, d, dt, pairs, st);
  }
}

extern "C" size_t glq_route_workspace(int64_t tokens, int32_t experts, int32_t top_k) {
  if (check_route(tokens, experts, top_k)) return 0;
  // (one workgroup needs none; a size of 0 says that the call would be refused; fewer tokens can have more workgroups)
  int64_t most = 0;
  for (const int64_t t : {tokens, tokens < kRouteShort ? tokens : kRouteShort, tokens < kRouteMiddle ? tokens : kRouteMiddle}) {
    const int64_t need = route_blocks(t) > 1 ? route_blocks(t) + route_groups(t) : 0;
    most = need > most ? need : most;
  }
  return 256 + (size_t)most * experts * 4;
}

extern "C" int glq_route(const void *logits, glq_dtype dt, int64_t tokens, int32_t experts, int32_t top_k, uint32_t flags,
                         float *weights, int32_t *ids, int32_t *pos, int32_t *src, int32_t *offsets, void *workspace,
                         size_t ws_bytes, void *hip_stream) {
  if (!valid_dtype(dt) || (flags & ~(uint32_t)GLQ_ROUTE_NORMALIZE)) return GLQ_ERR_ARG;
  const int rc = check_route(tokens, experts, top_k);
  if (rc) return rc;
  if (!offsets || !aligned4(offsets) || (tokens > 0 && (!logits || !weights || !ids || !pos || !src))) return GLQ_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(logits) & (dt == GLQ_F32 ? 3 : 1)) || !aligned4(weights) || !aligned4(ids) || !aligned4(pos) ||
      !aligned4(src))
    return GLQ_ERR_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || ws_bytes < glq_route_workspace(tokens, experts, top_k))
    return GLQ_ERR_WORKSPACE;
  RouteArgs a = {logits, tokens, route_blocks(tokens), route_groups(tokens), experts, top_k, route_each(tokens),
                 (flags & GLQ_ROUTE_NORMALIZE) ? 1 : 0, weights, ids, pos, src, offsets, reinterpret_cast<int32_t *>(workspace)};
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  if (experts <= 64) launch_pick<1>(a, dt, st);
  else if (experts <= 128) launch_pick<2>(a, dt, st);
  else if (experts <= 256) launch_pick<4>(a, dt, st);
  else if (experts <= 512) launch_pick<8>(a, dt, st);
  else launch_pick<16>(a, dt, st);
  int rc2 = hip_status(hipGetLastError(), "route_pick_k");
  if (rc2 || a.blocks == 1) return rc2;
  if (a.groups) {
    hipLaunchKernelGGL(route_group_k, dim3((unsigned)a.groups), dim3(kRouteThreads), 0, st, a);
    const int rc3 = hip_status(hipGetLastError(), "route_group_k");
    if (rc3) return rc3;
  }
  hipLaunchKernelGGL(route_place_k, dim3((unsigned)a.blocks), dim3(kRouteThreads), 0, st, a);
  return hip_status(hipGetLastError(), "route_place_k");
}
