// glq_attn.hip -- paged key-value cache and attention (gfx950) and their
// entry points of the C ABI: what a model runs between its compressed q, k, v
// projections and its output projection.
//
// Kernels:
//   kv_append_k     tokens' keys and values -> bf16, 8-bit or 4-bit rows
//   kv_read_k       cached rows -> dense keys and values
//   attn_decode_k   one new token per sequence over the paged cache
//   attn_prompt_bf16  packed prompts, bf16 matrix instructions
//   attn_prompt_f32   packed prompts, float32 matrix instructions
#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <type_traits>

#include "glq.h"
#include "glq_cache.h"

namespace glq {
namespace {

#define INLINED __attribute__((always_inline))   // lambdas on register arrays

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

template <int FMT, int D, bool F32>
__global__ void __launch_bounds__(256) kv_append_k(KvIo io) {
  KvPart<D> p;
  if (!p.place(io) || p.slot >= io.capacity) return;
  const int at = threadIdx.x % (D / 8);
  float x[2][8];
#pragma unroll
  for (int w = 0; w < 2; ++w)
    load8<F32>(reinterpret_cast<const uint8_t *>(io.dense[w]) + (F32 ? 4 : 2) * (p.dense[w] + 8 * at), x[w]);
#pragma unroll
  for (int w = 0; w < 2; ++w) append_row<FMT, D>(io, p, w, at, x[w]);
}

// The other way: a slot outside the cache gives zeros. Bound by the memory: 50,001
// tokens of 8 heads of 128 from 8 bits to bf16 in 57 us, 5.4 TB/s, over several sets of tensors in
// turn (the same set again, whose codes the 256 MB cache then holds: 45); with stores that stay in
// the caches 64.5, 4.8 TB/s, what a large copy reaches. To float32 3.5 TB/s: a lane's 32 bytes
// go out in two stores, half a line of the row each.
template <int FMT, int D, bool F32>
__global__ void __launch_bounds__(256) kv_read_k(KvIo io) {
  constexpr int WORDS = row_bytes<FMT>(D) / (D / 8) / 4;       // dwords a lane
  KvPart<D> p;
  if (!p.place(io)) return;
  const int at = threadIdx.x % (D / 8);
  const bool in = p.slot < io.capacity;
  uint32_t word[2][WORDS];
  float scale[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int64_t row = in ? p.cached : 0;
    load_words<WORDS>(reinterpret_cast<const uint8_t *>(io.cache[w]) + row * row_bytes<FMT>(D) + 4 * WORDS * at, word[w]);
    scale[w] = FMT == GLQ_KV_BF16 ? 1.0f : io.scale[w][row];
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (FMT == GLQ_KV_BF16) x[i] = (i & 1) ? bf16_hi(word[w][i / 2]) : bf16_lo(word[w][i / 2]);
      else if constexpr (FMT == GLQ_KV_INT8) x[i] = (float)(int8_t)(word[w][i / 4] >> (8 * (i % 4))) * scale[w];
      else x[i] = (float)((int)((word[w][0] >> (4 * i)) & 15u) - 8) * scale[w];
      x[i] = in ? x[i] : 0.0f;
    }
    store8<F32, true>(reinterpret_cast<uint8_t *>(io.dense[w]) + (F32 ? 4 : 2) * (p.dense[w] + 8 * at), x);
  }
}

// ------------------------------------------------------------ one new token

constexpr int64_t kCus = 256;                        // of an MI355X; only how work is shared out hangs on it
constexpr int decode_per_cu(int dim, bool f32) {
  return dim == 256 ? 1 : dim == 128 ? (f32 ? 1 : 2) : f32 ? 2 : 3;
}

struct DecodeArgs {
  const void *k, *v;
  const float *ks, *vs;
  const void *q;
  void *out;
  int64_t q_stride, out_stride;
  const int32_t *table, *lens;
  int64_t max_pages, max_len;
  int32_t heads, group, row_tiles, page_shift, num_pages;
  float abs_scale2, q_sign;    // |scale| log2(e) and the sign; for a scale of 0, 1 and 0
  int32_t batch, part_floats;  // floats of one workgroup's sums
  int32_t whole;               // no unit is split
  int32_t even_groups;         // workgroups that are enough where they get even shares
  unsigned int *tickets;       // [workgroups], zero between calls
  float *part;                 // [workgroups][part_floats]
};

// The wave works on tiles of 32 cached tokens, two 16-token halves. Scores
// are taken transposed, S^T = K Q^T (16x16x32 products, A = 16 tokens, B = the
// group's query heads padded to 16): lane (g, n) = (lane >> 4, lane & 15) then
// holds head n's scores of tokens 4 g .. 4 g + 3 of each half, which is the B
// operand of O^T = V^T P^T as it stands if its 8 k-slots mean those 8 tokens.
// V^T's A operand wants the same 8 tokens of one dimension a lane: the lane
// loads D / 16 neighbouring dimensions of each of its 8 tokens (whole rows per
// load) and puts pairs of tokens together in registers, so nothing passes
// through LDS until the waves join.
template <int FMT, int D> struct Tile {
  static constexpr int RB = row_bytes<FMT>(D);
  static constexpr int KW = RB / 16;                 // dwords of K per lane and half
  static constexpr int VB = RB / 16;                 // bytes of V per lane and token
  static constexpr int VW = VB < 4 ? 1 : VB / 4;
  uint32_t k[2][KW], v[8][VW];
  float ks[8], vs[8];
  uint32_t gone;                                     // bit s: half s lies on a page outside the cache
};

// dimension of element e of k-step c in quarter g (the order in which a lane's K
// bytes come out; Q is loaded in the same order)
template <int FMT, int D> __device__ __forceinline__ int k_dim(int c, int g, int e) {
  if constexpr (FMT == GLQ_KV_BF16) return 32 * c + 8 * g + e;
  if constexpr (FMT == GLQ_KV_INT8) return 64 * (c >> 1) + 16 * g + 8 * (c & 1) + e;
  const int o = (e >> 1) + 4 * (e & 1);              // pairs of nibbles 4 apart
  if constexpr (D == 64) return 16 * g + 8 * c + o;
  return 128 * (c >> 2) + 32 * g + 8 * (c & 3) + o;
}

// what no kernel of this call writes: read by scalar loads where the address is uniform
typedef __attribute__((address_space(4))) const int32_t *scalar_ints;

// The pages of a tile's two halves (a half past the end repeats the first). A plan that found no free page
// writes one outside the cache, and what lies in any page inside is another request's: the tokens of
// such a half are loaded from kNowhere, and their scores become -inf. Loaded from a page inside, their values would need a mask
// too, whatever they are: in every tile, not the last alone, that took 64 registers (30,000 tokens in bf16 43.5 us, 29.6 so, and 29.5 where no
// page was looked at).
struct Pages { uint32_t p[2], gone; };
struct Nowhere {
  uint8_t row[16 * 512];                             // 16 tokens of the longest rows
  float scale[16];
};
// (chosen between as global addresses: of generic ones the compiler makes flat loads: 32 of up to 4096 in 8 bits 43.8 us, 39.2 so)
typedef __attribute__((address_space(1))) const uint8_t *global_bytes;
template <class T> __device__ __forceinline__ const T *either(bool one, const T *x, const T *y) {
  const global_bytes a = (global_bytes)(uintptr_t)x, b = (global_bytes)(uintptr_t)y;
  return (const T *)(const uint8_t *)(one ? a : b);
}
__device__ const Nowhere kNowhere __attribute__((aligned(16))) = {{}, {1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1}};
__device__ __forceinline__ Pages pages_of(const DecodeArgs &a, scalar_ints table, int t, int end) {
  Pages x;
  x.gone = 0;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int32_t page = table[(t + 16 * s < end ? t + 16 * s : t) >> a.page_shift];
    x.p[s] = page < 0 ? 0u : page < a.num_pages ? (uint32_t)page : (uint32_t)a.num_pages - 1;
    x.gone |= x.p[s] != (uint32_t)page ? 1u << s : 0u;
  }
  return x;
}

template <int FMT, int D>
__device__ __forceinline__ void load_tile(const DecodeArgs &a, const Pages &pages, int h, int lane, int t, int end,
                                          Tile<FMT, D> &x) {
  using T = Tile<FMT, D>;
  const int g = lane >> 4, n = lane & 15;
  const uint8_t *kp = reinterpret_cast<const uint8_t *>(a.k), *vp = reinterpret_cast<const uint8_t *>(a.v);
  x.gone = pages.gone;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int ts = t + 16 * s < end ? t + 16 * s : t;
    const int64_t row = (((int64_t)pages.p[s] * a.heads + h) << a.page_shift) + (ts & ((1 << a.page_shift) - 1));
    const bool gone = pages.gone >> s & 1;           // uniform
    static_assert(16 * T::RB <= sizeof kNowhere.row, "rows of a half");
    const uint8_t *kr = either(gone, kNowhere.row, kp + row * T::RB) + n * T::RB;
    if constexpr (T::RB >= 64) {
#pragma unroll
      for (int i = 0; i < T::RB / 64; ++i) load_words<4>(kr + 64 * i + 16 * g, &x.k[s][4 * i]);
    } else {
      load_words<2>(kr + 8 * g, x.k[s]);
    }
    const uint8_t *vr = either(gone, kNowhere.row, vp + row * T::RB) + 4 * g * T::RB + n * T::VB;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if constexpr (T::VB == 2) x.v[4 * s + r][0] = *reinterpret_cast<const uint16_t *>(vr + r * T::RB);
      else load_words<T::VW>(vr + r * T::RB, x.v[4 * s + r]);
    }
    if constexpr (FMT != GLQ_KV_BF16) {
      const float4 u = *reinterpret_cast<const float4 *>(either(gone, kNowhere.scale, a.ks + row) + 4 * g);
      const float4 w = *reinterpret_cast<const float4 *>(either(gone, kNowhere.scale, a.vs + row) + 4 * g);
      x.ks[4 * s] = u.x, x.ks[4 * s + 1] = u.y, x.ks[4 * s + 2] = u.z, x.ks[4 * s + 3] = u.w;
      x.vs[4 * s] = w.x, x.vs[4 * s + 1] = w.y, x.vs[4 * s + 2] = w.z, x.vs[4 * s + 3] = w.w;
    }
  }
}

// nibble j of each 16-bit half as bf16 16 + code + 8: the code's 4 bits go
// into the top of the mantissa of 16
struct Nibbles {
  uint32_t mask = 0x00780078u, sixteen = 0x41804180u;
  // kept in registers: v_and_or_b32 takes no literals, and as literals they cost an instruction more
  __device__ __forceinline__ Nibbles() { asm("" : "+v"(mask), "+v"(sixteen)); }
};
__device__ __forceinline__ uint32_t nibbles(uint32_t x, int j, const Nibbles &c) {
  const uint32_t y = j == 0 ? x << 3 : x >> (4 * j - 3);
  return (y & c.mask) | c.sixteen;
}
constexpr float kBias4 = 24.0f;                      // what nibbles() adds to a code
// the same pair as the codes themselves (float32 path: the biased sums would
// cost it a decimal digit)
__device__ __forceinline__ uint32_t nibbles_unbiased(uint32_t x, int j) {
  return pack_high((float)((x >> (4 * j)) & 15u) - 8.0f, (float)((x >> (16 + 4 * j)) & 15u) - 8.0f);
}
template <bool BIASED> __device__ __forceinline__ uint32_t nibble_pair(uint32_t x, int j, const Nibbles &c) {
  if constexpr (BIASED) return nibbles(x, j, c);
  else return nibbles_unbiased(x, j);
}

template <int FMT, int D, bool BIASED>
__device__ __forceinline__ bf16x8 k_operand(const Tile<FMT, D> &x, int s, int c, const Nibbles &nib) {
  uint4 u;
  if constexpr (FMT == GLQ_KV_BF16) {
    u = make_uint4(x.k[s][4 * c], x.k[s][4 * c + 1], x.k[s][4 * c + 2], x.k[s][4 * c + 3]);
  } else if constexpr (FMT == GLQ_KV_INT8) {
    const uint32_t a = x.k[s][2 * c], b = x.k[s][2 * c + 1];
    u.x = pack_high((float)(int8_t)a, (float)(int8_t)(a >> 8));
    u.y = pack_high((float)(int8_t)(a >> 16), (float)(int8_t)(a >> 24));
    u.z = pack_high((float)(int8_t)b, (float)(int8_t)(b >> 8));
    u.w = pack_high((float)(int8_t)(b >> 16), (float)(int8_t)(b >> 24));
  } else {
    const uint32_t a = x.k[s][c];
    u = make_uint4(nibble_pair<BIASED>(a, 0, nib), nibble_pair<BIASED>(a, 1, nib), nibble_pair<BIASED>(a, 2, nib),
                   nibble_pair<BIASED>(a, 3, nib));
  }
  return __builtin_bit_cast(bf16x8, u);
}

// dimension n D / 16 + i of the lane's 8 tokens
template <int FMT, int D, bool BIASED>
__device__ __forceinline__ bf16x8 v_operand(const Tile<FMT, D> &x, int i, const Nibbles &nib) {
  uint32_t u[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    if constexpr (FMT == GLQ_KV_BF16) {
      u[p] = __builtin_amdgcn_perm(x.v[2 * p + 1][i >> 1], x.v[2 * p][i >> 1], (i & 1) ? 0x07060302u : 0x05040100u);
    } else if constexpr (FMT == GLQ_KV_INT8) {
      const int sh = 8 * (i & 3);
      u[p] = pack_high((float)(int8_t)(x.v[2 * p][i >> 2] >> sh), (float)(int8_t)(x.v[2 * p + 1][i >> 2] >> sh));
    } else {
      const uint32_t w = __builtin_amdgcn_perm(x.v[2 * p + 1][i >> 3], x.v[2 * p][i >> 3],
                                               (i & 4) ? 0x07060302u : 0x05040100u);
      u[p] = nibble_pair<BIASED>(w, i & 3, nib);
    }
  }
  return __builtin_bit_cast(bf16x8, make_uint4(u[0], u[1], u[2], u[3]));
}

// 8 floats as NP bf16 operands whose sum they are (1: rounded to nearest even; 2:
// 16 bits; 3: all 24). The cache is what this kernel waits for, so the weights of
// the bf16 path take two parts as well: few tokens, or a few that outweigh
// the rest, would show the 2^-8 of one.
template <int NP>
__device__ __forceinline__ void split8(const float *x, bf16x8 *o) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[i] = pack_bf16(r[2 * i], r[2 * i + 1]);
      if (p + 1 < NP) r[2 * i] -= bf16_lo(u[i]), r[2 * i + 1] -= bf16_hi(u[i]);
    }
    o[p] = __builtin_bit_cast(bf16x8, make_uint4(u[0], u[1], u[2], u[3]));
  }
}

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// max or sum over the four lanes of one column (lane & 15)
__device__ __forceinline__ float column_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float column_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// written through to, and read from, the memory side that the eight XCDs share (sc1)
__device__ __forceinline__ void store_shared(__amdgpu_buffer_rsrc_t r, int at, f32x4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, 4 * at, 0, 16);
}
__device__ __forceinline__ f32x4 load_shared(__amdgpu_buffer_rsrc_t r, int at) {
  return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, 4 * at, 0, 16));
}

// The running maxima are taken this much too high (in base 2), so that a row's weights, each
// at most 2^8 of the largest one's base, add up to no more than 1/2: the sum of weights
// times values is then no larger than the largest value, and a mean of finite values stays
// finite. It costs nothing (one multiply-add where a multiplication was) and takes its bits from
// where weights and values vanish. By the sequence's own number of keys, not the call's bound on
// it, on which a result should not depend. `extra`: for operands larger than the values they stand for.
__device__ __forceinline__ float headroom_of(int keys, int extra = 0) {
  return (float)(9 + extra + (keys > 1 ? 32 - __builtin_clz((unsigned)(keys - 1)) : 0));
}

// A part of a row's sums: values, their maximum and total
struct Sums {
  float o[8], top, total;
};
__device__ __forceinline__ void merge(Sums &s, const float *o, float top, float total) {
  const float mn = fmaxf(s.top, top), base = mn == -INFINITY ? 0.0f : mn;
  const float f = __builtin_amdgcn_exp2f(s.top - base), g = __builtin_amdgcn_exp2f(top - base);
  s.top = mn;
  s.total = s.total * f + total * g;
#pragma unroll
  for (int i = 0; i < 8; ++i) s.o[i] = s.o[i] * f + o[i] * g;
}

// What a workgroup does: one part of one unit (a sequence, a kept head and up to
// 16 of its query heads; 128-token tiles).
struct Place {
  int b, unit, part, parts;    // unit within the sequence; of `parts` (0: nothing to do)
  int len, tiles;              // of the sequence; tiles of the unit
};

__device__ __forceinline__ int length_of(const DecodeArgs &a, int b) {
  const int len = ((scalar_ints)(uintptr_t)a.lens)[b];
  return len < 0 ? 0 : len > a.max_len ? (int)a.max_len : len;
}

// Parts of a unit of `tiles` tiles where a part should have 1 / inv of them.
// Splitting costs a workgroup what some tiles take (its sums' way to memory, the
// ticket, and their way back), so a unit that is no more than `spare` tiles
// longer stays whole. Where there is a unit for every CU the memory is busy
// anyway and the cost is paid in full, so that there the difference is 8 tiles, and 5 otherwise. 32
// heads on 8 of 128, 8 bits but where said: one sequence of 256 6.8 us whole, 8.7 in parts; eight of 640
// 10.2 and 12.3; 32 of 1024 in 4 bits 13.1 and 15.7; one of 1024 (8 tiles) 12.1 and 9.9. Against it:
// heads of 256 would gain from 5 tiles on (one of 640 17.3 and 11.4).
// Any value from 1 on is right; every workgroup computes the same one (the multiply-add is written
// out, so that each copy of this rounds alike: find_place's last loop ends by it).
__device__ __forceinline__ int parts_of(int tiles, float inv, int spare) {
  return tiles == 0 ? 0 : (float)(tiles - spare) * inv <= 1.0f ? 1 : (int)__builtin_fmaf((float)tiles, inv, 0.999f);
}

// The smallest share for which the launch has workgroups enough for all parts,
// found by every workgroup alike: up to 64 sequences, one a lane, by bisection;
// beyond, by parts <= tiles / share + 1.
__device__ __forceinline__ Place find_place(const DecodeArgs &a, int lane) {
  const int each = (a.batch + 63) / 64, units = a.heads * a.row_tiles, at = blockIdx.x;
  Place p = {0, 0, 0, 0, 0, 0};
  if (a.whole) {
    p.b = at / units;
    p.unit = at - p.b * units;
    p.len = length_of(a, p.b);
    p.tiles = (p.len + 127) >> 7;
    p.parts = p.tiles > 0 ? 1 : 0;
    return p;
  }
  const int64_t groups = gridDim.x;
  const int spare = (int64_t)a.batch * units >= kCus ? 8 : 5;
  float inv;
  int mine = 0;
  int len = 0;                                       // of the lane's sequence
  if (each == 1) {
    len = lane < a.batch ? length_of(a, lane) : 0;
    const int t = (len + 127) >> 7;
    const int most = __builtin_amdgcn_readlane(wave_scan<true>(t), 63);
    const int total = __builtin_amdgcn_readlane(wave_scan<false>(t), 63);
    // One workgroup a CU streams as fast as two and splits less (heads of 128, one sequence of
    // 8192, 8 bits: 11.7 us, 16.6 with two), unless that leaves the shares uneven (32 of up
    // to 4096: 37.9 us, 33.4 with two). Only rows of 8 bits and more of heads of 128 (even_groups):
    // 4 bits want the second one's VALU (two of up to 131,072: 56.7 us, 62.1 with one a CU; one of
    // 8192, though, 14.3 and 11.0), heads of 64 have three (the same two in 8 bits 45.9 and 48.3, in
    // 4 bits 39.4 and 50.7; one of 100,000 in bf16 44.1 and 37.9), heads of 256 have one.
    for (int64_t limit = min((int64_t)a.even_groups, groups);; limit = groups) {
      int lo = 0, hi = max(1, most);                 // shares: too small, large enough
      while (hi - lo > 1) {
        const int share = (lo + hi) >> 1;
        const int count = __builtin_amdgcn_readlane(wave_scan<false>(parts_of(t, __builtin_amdgcn_rcpf((float)share), spare)), 63);
        if ((int64_t)count * units <= limit) hi = share;
        else lo = share;
      }
      inv = __builtin_amdgcn_rcpf((float)hi);
      if (limit == groups || (float)hi * (float)limit <= 1.15f * (float)total * (float)units) break;
    }
    mine = parts_of(t, inv, spare);
  } else {
    int64_t total = 0;
    for (int b = lane; b < a.batch; b += 64) total += (length_of(a, b) + 127) >> 7;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) total += __shfl_xor(total, s);
    inv = 1.0f / (float)(total * units / (groups - (int64_t)a.batch * units) + 2);
    for (int b = lane * each; b < min(a.batch, (lane + 1) * each); ++b) mine += parts_of((length_of(a, b) + 127) >> 7, inv, spare);
  }
  const int upto = wave_scan<false>(mine);
  const uint64_t here = __builtin_amdgcn_ballot_w64((upto - mine) * units <= at && at < upto * units);
  if (!here) return p;
  const int from = __builtin_ctzll(here);
  int base = __builtin_amdgcn_readlane(upto - mine, from) * units;
  p.b = from * each;
  while (true) {                                     // ends: the part is of one of the lane's sequences
    p.len = each == 1 ? __builtin_amdgcn_readlane(len, from) : length_of(a, p.b);
    p.tiles = (p.len + 127) >> 7;
    p.parts = __builtin_amdgcn_readfirstlane(parts_of(p.tiles, inv, spare));
    if (at < base + p.parts * units) break;
    base += p.parts * units;
    ++p.b;
  }
  p.unit = (at - base) / p.parts;
  p.part = (at - base) - p.unit * p.parts;
  return p;
}

// The waves of a workgroup take every fourth 32-token tile, the next tile's
// loads in flight while one is worked on. A unit of several parts: each leaves
// its sums in the workspace and takes a ticket; the one with the last ticket
// joins them, in the order of the tiles. Workgroups per CU: what the registers
// of two tiles leave room for.
template <int FMT, int D, bool F32>
__global__ void __launch_bounds__(256, (decode_per_cu(D, F32))) attn_decode_k(DecodeArgs a) {
  constexpr int NP = F32 ? 3 : 1, KS = D / 32, DT = D / 16;
  constexpr int WP = F32 ? 3 : 2;                    // bf16 parts of a weight
  constexpr bool BIASED = FMT == GLQ_KV_INT4 && !F32;
  // float32 heads of 256 over bf16 rows: two tiles would not fit the registers
  constexpr bool AHEAD = !(F32 && D == 256 && FMT == GLQ_KV_BF16);
  // [4][16] rows of sums, [4][16] maxima, [4][16] totals; rows a float4 longer than
  // D, so that the 16 lanes of a column write to different banks
  constexpr int P = D + 4;
  extern __shared__ float shm[];
  float *so = shm, *sm = shm + 4 * 16 * P, *sl = sm + 64;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, n = lane & 15;
  const int64_t esize = F32 ? 4 : 2;
  // sequences without tokens: zeros (last, so that no load waits for it)
  auto zero_rows = [&]() INLINED {
    for (int b = blockIdx.x; b < a.batch; b += gridDim.x)
      if (length_of(a, b) == 0)
        for (int e = threadIdx.x; e < a.heads * a.group * (D / 8); e += 256) {
          const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
          store8<F32>(reinterpret_cast<uint8_t *>(a.out) + esize * (b * a.out_stride + 8 * (int64_t)e), zero);
        }
  };

  const Place at = find_place(a, lane);
  if (at.parts == 0) return zero_rows();
  const int rt = at.unit % a.row_tiles, h = at.unit / a.row_tiles;
  const int head0 = h * a.group + 16 * rt, rows = min(16, a.group - 16 * rt);
  const int64_t b = at.b;
  const scalar_ints table = (scalar_ints)(uintptr_t)(a.table + b * a.max_pages);
  const int tile0 = (int)((int64_t)at.tiles * at.part / at.parts);
  const int tile1 = (int)((int64_t)at.tiles * (at.part + 1) / at.parts);
  const int t0 = 128 * tile0 + 32 * wave, end = min(at.len, 128 * tile1);
  {
    Tile<FMT, D> tile;
    Pages next = {{0, 0}, 0};
    if (t0 < end) {
      const Pages first = pages_of(a, table, t0, end);
      next = pages_of(a, table, t0 + 128 < end ? t0 + 128 : t0, end);
      load_tile<FMT, D>(a, first, h, lane, t0, end, tile);
    }

    bf16x8 q[NP][KS];
    float qsum = 0.0f;
#pragma unroll
    for (int c = 0; c < KS; ++c) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint8_t *p = reinterpret_cast<const uint8_t *>(a.q) +
                           esize * (b * a.q_stride + (int64_t)(head0 + (n < rows ? n : 0)) * D + k_dim<FMT, D>(c, g, e));
        x[e] = F32 ? *reinterpret_cast<const float *>(p) : bf16_lo(*reinterpret_cast<const uint16_t *>(p));
        x[e] = a.q_sign == 0.0f ? 0.0f : x[e] * a.q_sign;
        qsum += x[e];
      }
      bf16x8 o[NP];
      split8<NP>(x, o);
#pragma unroll
      for (int p = 0; p < NP; ++p) q[p][c] = o[p];
    }
    const float s0 = BIASED ? -kBias4 * column_sum(qsum) : 0.0f;

    // (4-bit operands carry a bias of kBias4 on codes of up to 7)
    const float headroom = headroom_of(at.len, BIASED ? 3 : 0);
    float m = -INFINITY, base = 0.0f, l = 0.0f;
    f32x4 acc[DT];
#pragma unroll
    for (int i = 0; i < DT; ++i) acc[i] = (f32x4){0, 0, 0, 0};

    const Nibbles nib;
    auto work = [&](Tile<FMT, D> &x, int t) INLINED {
      float s[8];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        f32x4 c4 = {s0, s0, s0, s0};
#pragma unroll
        for (int c = 0; c < KS; ++c) {
          const bf16x8 kk = k_operand<FMT, D, BIASED>(x, half, c, nib);
#pragma unroll
          for (int p = 0; p < NP; ++p) c4 = mfma16(kk, q[p][c], c4);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
          s[4 * half + r] = FMT == GLQ_KV_BF16 ? c4[r] : c4[r] * x.ks[4 * half + r];
      }
      if (x.gone) {                                  // uniform
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = x.gone >> (j >> 2) & 1 ? -INFINITY : s[j];
      }
      if (t + 32 > end) {                            // tokens past the end: no weight, and values that are 0
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bool in = t + 16 * (j >> 2) + 4 * g + (j & 3) < end;
          s[j] = in ? s[j] : -INFINITY;
          if constexpr (FMT == GLQ_KV_BF16) {
#pragma unroll
            for (int w = 0; w < Tile<FMT, D>::VW; ++w) x.v[j][w] = in ? x.v[j][w] : 0u;
          } else {
            x.vs[j] = in ? x.vs[j] : 0.0f;
          }
        }
      }
      float mt = s[0];
#pragma unroll
      for (int j = 1; j < 8; ++j) mt = fmaxf(mt, s[j]);
      mt = fmaf(column_max(mt), a.abs_scale2, headroom);
      // the running maximum follows only where it is outgrown by 2^8: weights of
      // up to 2^8 lose nothing, and the sums are rarely rescaled
      if (__any(mt > m + 8.0f)) {
        // nothing summed yet: known by the row's maximum, as l is this lane's tokens only, and acc
        // all four lanes'
        const bool none = m == -INFINITY;
        m = fmaxf(m, mt);
        const float now = m == -INFINITY ? 0.0f : m;
        const float alpha = none ? 0.0f : __builtin_amdgcn_exp2f(base - now);
        base = now;
        l *= alpha;
#pragma unroll
        for (int i = 0; i < DT; ++i) acc[i] *= alpha;
      }
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        w[j] = __builtin_amdgcn_exp2f(fmaf(s[j], a.abs_scale2, -base));
        l += w[j];
        if constexpr (FMT != GLQ_KV_BF16) w[j] *= x.vs[j];
      }
      bf16x8 pw[WP];
      split8<WP>(w, pw);
      const uint32_t nb = 0xC1C0C1C0u;               // -kBias4 twice
      const bf16x8 bias = __builtin_bit_cast(bf16x8, make_uint4(nb, nb, nb, nb));
#pragma unroll
      for (int i = 0; i < DT; ++i) {
        const bf16x8 vv = v_operand<FMT, D, BIASED>(x, i, nib);
#pragma unroll
        for (int p = 0; p < WP; ++p) {
          // the 4-bit operand's bias leaves at once, tile by tile: over a long
          // cache the biased sums would outgrow the result they hide
          if constexpr (BIASED) acc[i] = mfma16(bias, pw[p], acc[i]);
          acc[i] = mfma16(vv, pw[p], acc[i]);
        }
      }
    };
    // The page numbers are read one tile further ahead than the tiles. No branch
    // lies between a tile's loads and its use but those that skip the use: where
    // paths with and without newer loads met, the wait for the older ones would
    // be a wait for all.
    auto ahead = [&](int t, Tile<FMT, D> &x) INLINED {
      const Pages now = next;
      next = pages_of(a, table, t + 128 < end ? t + 128 : t, end);
      load_tile<FMT, D>(a, now, h, lane, t, end, x);
    };
    if (t0 < end) {
      int t = t0;
      if constexpr (AHEAD && D == 256) {             // no registers for two copies of the work
        for (; t + 128 < end; t += 128) {
          Tile<FMT, D> x;
          ahead(t + 128, x);
          __builtin_amdgcn_sched_barrier(0);
          work(tile, t);
          tile = x;
        }
        work(tile, t);
      } else if constexpr (AHEAD) {
        Tile<FMT, D> tile2;
        while (true) {                               // two tiles in turn: a copy would wait for the loads
          if (t + 128 >= end) {
            work(tile, t);
            break;
          }
          ahead(t + 128, tile2);
          __builtin_amdgcn_sched_barrier(0);         // the loads go out before the work
          work(tile, t);
          t += 128;
          if (t + 128 >= end) {
            work(tile2, t);
            break;
          }
          ahead(t + 128, tile);
          __builtin_amdgcn_sched_barrier(0);
          work(tile2, t);
          t += 128;
        }
      } else {
        for (; t + 128 < end; t += 128) {
          work(tile, t);
          ahead(t + 128, tile);
        }
        work(tile, t);
      }
    }
    l = column_sum(l);

    // join the waves
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int i = 0; i < DT; i += 4)
        *reinterpret_cast<float4 *>(so + (wave * 16 + n) * P + (4 * g + r) * DT + i) =
            make_float4(acc[i][r], acc[i + 1][r], acc[i + 2][r], acc[i + 3][r]);
    if (g == 0) sm[16 * wave + n] = l == 0.0f ? -INFINITY : base, sl[16 * wave + n] = l;
    __syncthreads();
    const int items = rows * (D / 8);
    auto finish = [&](int e, const Sums &x) {
      const int row = e / (D / 8), d0 = 8 * (e % (D / 8));
      const float inv = x.total == 0.0f ? 0.0f : 1.0f / x.total;
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = x.o[i] * inv;
      store8<F32>(reinterpret_cast<uint8_t *>(a.out) + esize * (b * a.out_stride + (int64_t)(head0 + row) * D + d0), o);
    };
    const int first = blockIdx.x - at.part, count = at.parts;
    const __amdgpu_buffer_rsrc_t mine = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(a.part + (int64_t)blockIdx.x * a.part_floats), 0, 4 * a.part_floats, 0x00020000);
    for (int e = threadIdx.x; e < items; e += 256) {
      const int row = e / (D / 8), d0 = 8 * (e % (D / 8));
      Sums x = {{0, 0, 0, 0, 0, 0, 0, 0}, -INFINITY, 0.0f};
#pragma unroll
      for (int w = 0; w < 4; ++w) merge(x, &so[(16 * w + row) * P + d0], sm[16 * w + row], sl[16 * w + row]);
      if (count == 1) {
        finish(e, x);
      } else {
        store_shared(mine, 8 * e, (f32x4){x.o[0], x.o[1], x.o[2], x.o[3]});
        store_shared(mine, 8 * e + 4, (f32x4){x.o[4], x.o[5], x.o[6], x.o[7]});
        if (d0 == 0) store_shared(mine, rows * D + 4 * row, (f32x4){x.top, x.total, 0, 0});
      }
    }
    if (count > 1) {
      __builtin_amdgcn_s_waitcnt(0);                 // the sums are at the memory side
      __syncthreads();
      int *flag = reinterpret_cast<int *>(sm);
      if (threadIdx.x == 0)
        *flag = (int)__hip_atomic_fetch_add(a.tickets + first, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __syncthreads();
      if (*flag == count - 1) {
        if (threadIdx.x == 0) __hip_atomic_store(a.tickets + first, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        // few items: slices of the threads take every slices-th part, and meet in LDS
        const int slices = items >= 256 ? 1 : 256 / items;
        const __amdgpu_buffer_rsrc_t all =
            __builtin_amdgcn_make_buffer_rsrc((void *)(a.part + (int64_t)first * a.part_floats), 0,
                                              4 * a.part_floats * count, 0x00020000);
        for (int e0 = 0; e0 < items; e0 += 256) {
          const int e = slices == 1 ? e0 + threadIdx.x : threadIdx.x % items;
          const int slice = slices == 1 ? 0 : threadIdx.x / items;
          Sums x = {{0, 0, 0, 0, 0, 0, 0, 0}, -INFINITY, 0.0f};
          // Parts a thread has in flight: 8 where that is all of them, since loads past the last cost as
          // much as others (four sequences of up to 3000, 32 heads on 8 of 128, bf16: 12.4 us, 16.2 with
          // 16; one of 1000, float32: 10.0, 12.5 with 24), and as many as the registers hold otherwise (24
          // parts, 8 heads on 1 of 256: 15.6 us with 24, 16.3 with 8). Heads of 64, three workgroups a CU,
          // have registers for 8 (one of 8192: 11.9 us, 18.5 with 16).
          if (e < items && slice < slices) {
            const int row = e / (D / 8);
            auto take = [&](auto fly) INLINED {
              constexpr int FLY = decltype(fly)::value;                      // parts whose loads are in flight
              for (int c0 = slice; c0 < count; c0 += FLY * slices) {
                f32x4 lo[FLY], hi[FLY], mt[FLY];
#pragma unroll
                for (int j = 0; j < FLY; ++j) {      // past the last: the last, unused
                  const int p = min(c0 + j * slices, count - 1) * a.part_floats;
                  lo[j] = load_shared(all, p + 8 * e), hi[j] = load_shared(all, p + 8 * e + 4);
                  mt[j] = load_shared(all, p + rows * D + 4 * row);
                }
                __builtin_amdgcn_sched_barrier(0);   // all of them go out before the first is used
#pragma unroll
                for (int j = 0; j < FLY; ++j) {
                  const bool in = c0 + j * slices < count;
                  float o[8];
#pragma unroll
                  for (int i = 0; i < 4; ++i) o[i] = in ? lo[j][i] : 0.0f, o[4 + i] = in ? hi[j][i] : 0.0f;
                  merge(x, o, in ? mt[j][0] : -INFINITY, in ? mt[j][1] : 0.0f);
                }
              }
            };
            if (D == 64 || count <= 8 * slices) take(std::integral_constant<int, 8>());
            else take(std::integral_constant<int, D == 64 ? 8 : F32 || D == 256 ? 24 : 16>());
            if (slices == 1) finish(e, x);
          }
          if (slices == 1) continue;
          __syncthreads();                           // everyone has read the flag
#pragma unroll
          for (int i = 0; i < 8; ++i) shm[10 * threadIdx.x + i] = x.o[i];
          shm[10 * threadIdx.x + 8] = x.top, shm[10 * threadIdx.x + 9] = x.total;
          __syncthreads();
          if ((int)threadIdx.x < items) {
            for (int s = 1; s < slices; ++s) {
              const float *y = shm + 10 * (s * items + threadIdx.x);
              merge(x, y, y[8], y[9]);
            }
            finish(e, x);
          }
        }
      }
    }
  }
  zero_rows();
}

// ------------------------------------------------------------ prompts

struct PromptArgs {
  const void *q, *k, *v;
  void *out;
  int64_t q_stride, k_stride, v_stride, out_stride, total_q, total_k;
  const int32_t *cu_q, *cu_k;
  int64_t max_q;
  int32_t q_heads, kv_heads, batch, causal;
  float scale2;                // scale * log2(e)
  float abs_scale2;            // bf16 path: its magnitude, the sign in q_xor; for a
  uint32_t q_and, q_xor;       // scale of 0, 1 and queries of 0 (q_and)
};

__device__ __forceinline__ int clamped(int x, int64_t top) { return x < 0 ? 0 : x > top ? (int)top : x; }

template <bool F32> __device__ __forceinline__ float4 load4(const void *p, int64_t at) {
  if constexpr (F32) return *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(p) + at);
  const uint2 u = *reinterpret_cast<const uint2 *>(reinterpret_cast<const uint16_t *>(p) + at);
  return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
}

// A weight of 0 times a value that is not finite is NaN, and would reach
// queries that do not see the key. In a tile with such pairs the values that
// are not finite become 0, and the queries that do see one get NaN.
template <int CT, class Acc>
__device__ __forceinline__ void keep_unseen_out(float4 &x, const bool (&seen)[CT][4], int r, Acc acc) {
  float v[4] = {x.x, x.y, x.z, x.w};
  bool bad = false;
#pragma unroll
  for (int c = 0; c < 4; ++c) bad |= !(fabsf(v[c]) < INFINITY);
  if (!__any(bad)) return;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const bool b = !(fabsf(v[c]) < INFINITY);
    v[c] = b ? 0.0f : v[c];
#pragma unroll
    for (int t = 0; t < CT; ++t) {
      const f32x4 hit = __builtin_amdgcn_mfma_f32_16x16x4f32(b ? 1.0f : 0.0f, seen[t][r] ? 1.0f : 0.0f,
                                                             (f32x4){0, 0, 0, 0}, 0, 0, 0);
      f32x4 &o = acc(t)[c];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = hit[e] > 0.0f ? NAN : o[e];
    }
  }
  x = make_float4(v[0], v[1], v[2], v[3]);
}

// Rows of attention in float32: a wave takes CT tiles of 16 rows against every
// `step`-th 16 keys from `first` on, with float32 16x16x4 products, transposed as
// in the decode kernel: S^T = K Q^T leaves lane (g, n) row n's scores of keys 4 g +
// r, the B operand of the r-th step of O^T = V^T P^T. k-slot g of step 4 i + r of
// the scores means dimension 16 i + 4 g + r, row n of value tile (i, c) means
// dimension 64 i + 4 n + c: both are 16-byte loads. Row x is head head0 + x % group
// of query x / group. The next keys' loads are in flight while these are worked on.
// Bound by issue: these products and the VALU do not run at once (0 cycles of both by
// the counters), a tile's 32 products (heads of 64) take 1024 cycles and the rest, about
// 110 instructions, 450. So addresses are stepped, masks only where keys end, sums
// rescaled when a maximum rises by more than 8: 146 us against 153 for eight prompts of
// 333 on 1000, 16 heads on 2 of 64 (in tiles of 32 rows); 8 heads of 128, three prompts of
// 200 on 500: 38.2 against 44.9.
struct RowJob {
  int head0, group, kvh, row0, rows;   // rows: of the sequence (queries * group)
  int q0, k0, lk, shift;               // first query and key row, keys, keys ahead of the queries
};
template <int D, int CT> struct RowSums {
  f32x4 acc[CT][D / 16];
  float m[CT], l[CT];                  // maximum and this lane's part of the total
};
template <int D> struct KvRows {
  float4 k[D / 16], v[4][D / 64];
};

// a lane's element of its key row and of its four value rows of the keys from j0 on
// (rows past the last one: that one)
struct RowsAt { int64_t k, v[4]; };
__device__ __forceinline__ RowsAt rows_at(const PromptArgs &a, const RowJob &w, int lane, int D, int j0) {
  const int g = lane >> 4, n = lane & 15;
  RowsAt p;
  p.k = (w.k0 + min(j0 + n, w.lk - 1)) * a.k_stride + (int64_t)w.kvh * D + 4 * g;
#pragma unroll
  for (int r = 0; r < 4; ++r) p.v[r] = (w.k0 + min(j0 + 4 * g + r, w.lk - 1)) * a.v_stride + (int64_t)w.kvh * D + 4 * n;
  return p;
}

template <int D, bool F32>
__device__ __forceinline__ void load_rows(const PromptArgs &a, const RowsAt &p, KvRows<D> &x) {
#pragma unroll
  for (int i = 0; i < D / 16; ++i) x.k[i] = load4<F32>(a.k, p.k + 16 * i);
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int i = 0; i < D / 64; ++i) x.v[r][i] = load4<F32>(a.v, p.v[r] + 64 * i);
}

template <int D, bool F32, int CT>
__device__ __forceinline__ void attend_rows(const PromptArgs &a, const RowJob &w, int lane, int first, int step,
                                            RowSums<D, CT> &o) {
  const int g = lane >> 4, n = lane & 15;
  float4 q[CT][D / 16];
  int last[CT];                                      // this lane's rows' last keys
#pragma unroll
  for (int t = 0; t < CT; ++t) {
    const int row = min(w.row0 + 16 * t + n, w.rows - 1), query = row / w.group;
    last[t] = a.causal ? query + w.shift : w.lk - 1;
    const int64_t at = (int64_t)(w.q0 + query) * a.q_stride + (int64_t)(w.head0 + row - query * w.group) * D + 4 * g;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) q[t][i] = load4<F32>(a.q, at + 16 * i);
    o.m[t] = -INFINITY, o.l[t] = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o.acc[t][i] = (f32x4){0, 0, 0, 0};
  }
  // keys that all rows of the wave see, and that any of them sees
  const int all = a.causal ? w.row0 / w.group + w.shift : w.lk - 1;
  const int top = min(w.row0 + 16 * CT, w.rows) - 1;
  const int end = min(w.lk, a.causal ? top / w.group + w.shift + 1 : w.lk);
  if (first >= end) return;
  const float headroom = headroom_of(w.lk);
  auto work = [&](KvRows<D> &x, int j0) INLINED {
    const bool masked = j0 + 15 > all || j0 + 16 > w.lk;
    f32x4 s[CT];
    bool seen[CT][4];
#pragma unroll
    for (int t = 0; t < CT; ++t) {
      s[t] = (f32x4){0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        s[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(x.k[i].x, q[t][i].x, s[t], 0, 0, 0);
        s[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(x.k[i].y, q[t][i].y, s[t], 0, 0, 0);
        s[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(x.k[i].z, q[t][i].z, s[t], 0, 0, 0);
        s[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(x.k[i].w, q[t][i].w, s[t], 0, 0, 0);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) s[t][r] *= a.scale2;
      if (masked)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = j0 + 4 * g + r;
          seen[t][r] = j <= last[t] && j < w.lk;
          s[t][r] = seen[t][r] ? s[t][r] : -INFINITY;
        }
      const float mt = column_max(fmaxf(fmaxf(s[t][0], s[t][1]), fmaxf(s[t][2], s[t][3]))) + headroom;
      if (__any(mt > o.m[t] + 8.0f)) {               // weights of up to 2^8 go with the old base
        const float mn = fmaxf(o.m[t], mt);
        const float alpha = o.m[t] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(o.m[t] - mn);
        o.m[t] = mn;
        o.l[t] *= alpha;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o.acc[t][i] *= alpha;
      }
      const float base = o.m[t] == -INFINITY ? 0.0f : o.m[t];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        s[t][r] = __builtin_amdgcn_exp2f(s[t][r] - base);
        o.l[t] += s[t][r];
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        float4 v = x.v[r][i];
        if (masked) {
          if (j0 + 4 * g + r >= w.lk) v = make_float4(0, 0, 0, 0);
          keep_unseen_out<CT>(v, seen, r, [&](int t) { return &o.acc[t][4 * i]; });
        }
#pragma unroll
        for (int t = 0; t < CT; ++t) {
          o.acc[t][4 * i] = __builtin_amdgcn_mfma_f32_16x16x4f32(v.x, s[t][r], o.acc[t][4 * i], 0, 0, 0);
          o.acc[t][4 * i + 1] = __builtin_amdgcn_mfma_f32_16x16x4f32(v.y, s[t][r], o.acc[t][4 * i + 1], 0, 0, 0);
          o.acc[t][4 * i + 2] = __builtin_amdgcn_mfma_f32_16x16x4f32(v.z, s[t][r], o.acc[t][4 * i + 2], 0, 0, 0);
          o.acc[t][4 * i + 3] = __builtin_amdgcn_mfma_f32_16x16x4f32(v.w, s[t][r], o.acc[t][4 * i + 3], 0, 0, 0);
        }
      }
  };
  KvRows<D> x;
  int j0 = first;
  if constexpr (!F32) {                              // (the bf16 kernel's way out: registers, not haste)
    for (; j0 < end; j0 += step) {
      load_rows<D, F32>(a, rows_at(a, w, lane, D, j0), x);
      work(x, j0);
    }
    return;
  }
  KvRows<D> y;
  RowsAt p = rows_at(a, w, lane, D, j0);
  const int64_t k_step = step * a.k_stride, v_step = step * a.v_stride;
  auto next = [&](KvRows<D> &to) INLINED {
    if (j0 + step + 16 > w.lk) {
      p = rows_at(a, w, lane, D, j0 + step);
    } else {
      p.k += k_step;
#pragma unroll
      for (int r = 0; r < 4; ++r) p.v[r] += v_step;
    }
    load_rows<D, F32>(a, p, to);
    __builtin_amdgcn_sched_barrier(0);               // the loads go out before the work
  };
  load_rows<D, F32>(a, p, x);
  while (j0 + step < end) {
    next(y);
    work(x, j0);
    j0 += step;
    x = y;
  }
  work(x, j0);
}

// row x's values of a lane to memory, divided by the row's total
template <int D, bool F32>
__device__ __forceinline__ void store_row(const PromptArgs &a, const RowJob &w, int row, int d, float4 v) {
  const int query = row / w.group;
  const int64_t at = (int64_t)(w.q0 + query) * a.out_stride + (int64_t)(w.head0 + row - query * w.group) * D + d;
  if constexpr (F32) *reinterpret_cast<float4 *>(reinterpret_cast<float *>(a.out) + at) = v;
  else *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(a.out) + at) =
           make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}

// one wave, all keys, 16 rows: the bf16 kernel's way out where values are not finite
template <int D>
__device__ __forceinline__ void rows_alone(const PromptArgs &a, const RowJob &w, int lane) {
  RowSums<D, 1> o;
  attend_rows<D, false, 1>(a, w, lane, 0, 16, o);
  const float l = column_sum(o.l[0]), inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int g = lane >> 4, row = w.row0 + (lane & 15);
  if (row >= w.rows) return;
#pragma unroll
  for (int i = 0; i < D / 64; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      store_row<D, false>(a, w, row, 64 * i + 4 * (4 * g + r),
                          make_float4(o.acc[0][4 * i][r] * inv, o.acc[0][4 * i + 1][r] * inv,
                                      o.acc[0][4 * i + 2][r] * inv, o.acc[0][4 * i + 3][r] * inv));
}

// a sequence: its first query and key row and their numbers
struct Span { int q0, lq, k0, lk; };
__device__ __forceinline__ Span span_of(const PromptArgs &a, int64_t b) {
  const int q0 = clamped(a.cu_q[b], a.total_q), q1 = clamped(a.cu_q[b + 1], a.total_q);
  const int k0 = clamped(a.cu_k[b], a.total_k), k1 = clamped(a.cu_k[b + 1], a.total_k);
  return {q0, q1 - q0, k0, k1 - k0 > 0 ? k1 - k0 : 0};
}

// Workgroups of a sequence of lq queries (R rows each: queries times the heads of a
// kept head); more queries than the launch was made for are not done
template <int R> __device__ __forceinline__ int tiles_of(const PromptArgs &a, int lq) {
  const int64_t n = lq < a.max_q ? lq : a.max_q;
  return n > 0 ? (int)((n * (a.q_heads / a.kv_heads) + R - 1) / R) : 0;
}

// The sequence and tile of a kept head's at-th workgroup. In a causal prompt the
// last tiles see the most keys and come first, over all sequences (up to 64 of
// them, one a lane: the highest tile for which few enough come before it, by
// bisection on counts; beyond, sequence by sequence). Workgroups without a tile are the
// last: between the others they would hold their places up (one prompt of 2048 among 11
// empty ones took 115 us instead of 52).
struct Spot { Span span; int tile; };                // tile < 0: none
template <int R> __device__ __forceinline__ Spot find_tile(const PromptArgs &a, int lane, int at) {
  const Spot none = {{0, 0, 0, 0}, -1};
  if (a.batch <= 64) {
    Span mine = {0, 0, 0, 0};
    if (lane < a.batch) mine = span_of(a, lane);
    const int tiles = tiles_of<R>(a, mine.lq);
    auto from = [&](int tile) INLINED {              // workgroups of tiles from `tile` on
      return __builtin_amdgcn_readlane(wave_scan<false>(max(tiles - tile, 0)), 63);
    };
    if (at >= from(0)) return none;
    int lo = 0, hi = __builtin_amdgcn_readlane(wave_scan<true>(tiles), 63), after = 0;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1, n = from(mid);
      if (n > at) lo = mid;
      else hi = mid, after = n;
    }
    const uint64_t in = __builtin_amdgcn_ballot_w64(tiles > lo);
    const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(in >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)in, 0u));
    const int b = __builtin_ctzll(__builtin_amdgcn_ballot_w64(tiles > lo && before == at - after));
    return {{__builtin_amdgcn_readlane(mine.q0, b), __builtin_amdgcn_readlane(mine.lq, b),
             __builtin_amdgcn_readlane(mine.k0, b), __builtin_amdgcn_readlane(mine.lk, b)}, lo};
  }
  const int each = (a.batch + 63) / 64;
  int mine = 0;
  for (int b = lane * each; b < min(a.batch, (lane + 1) * each); ++b) mine += tiles_of<R>(a, span_of(a, b).lq);
  const int upto = wave_scan<false>(mine);
  const uint64_t here = __builtin_amdgcn_ballot_w64(upto - mine <= at && at < upto);
  if (!here) return none;
  const int lane_of = __builtin_ctzll(here);
  int base = __builtin_amdgcn_readlane(upto - mine, lane_of);
  for (int b = lane_of * each; b < min(a.batch, (lane_of + 1) * each); ++b) {  // the tile is of one of the lane's sequences
    const Span s = span_of(a, b);
    const int n = __builtin_amdgcn_readfirstlane(tiles_of<R>(a, s.lq));
    if (at < base + n)
      return {{__builtin_amdgcn_readfirstlane(s.q0), __builtin_amdgcn_readfirstlane(s.lq),
               __builtin_amdgcn_readfirstlane(s.k0), __builtin_amdgcn_readfirstlane(s.lk)}, n - 1 - (at - base)};
    base += n;
  }
  return none;
}

// The float32 path. A workgroup takes 16 CT rows (queries times the heads that
// share a kept head), its waves a quarter of the keys each; they join in LDS.
template <int D, int CT>
__global__ void __launch_bounds__(256, (D < 256 ? 2 : 1)) attn_prompt_f32(PromptArgs a) {
  extern __shared__ float shm[];                     // [4][16 CT][D] sums, [4][16 CT] maxima, [4][16 CT] totals
  constexpr int R = 16 * CT;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kvh = blockIdx.x % a.kv_heads, group = a.q_heads / a.kv_heads;
  const Spot spot = find_tile<R>(a, lane, blockIdx.x / a.kv_heads);
  if (spot.tile < 0) return;
  const Span s = spot.span;
  const int row0 = R * spot.tile, rows = (int)min((int64_t)s.lq, a.max_q) * group;
  const RowJob w = {kvh * group, group, kvh, row0, rows, s.q0, s.k0, s.lk, s.lk - s.lq};
  RowSums<D, CT> o;
  attend_rows<D, true, CT>(a, w, lane, 16 * wave, 64, o);
  const int g = lane >> 4, n = lane & 15;
  float *so = shm, *sm = shm + 4 * R * D, *sl = sm + 4 * R;
#pragma unroll
  for (int t = 0; t < CT; ++t) {
    const float l = column_sum(o.l[t]);
#pragma unroll
    for (int i = 0; i < D / 64; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *reinterpret_cast<float4 *>(so + (R * wave + 16 * t + n) * D + 64 * i + 4 * (4 * g + r)) =
            make_float4(o.acc[t][4 * i][r], o.acc[t][4 * i + 1][r], o.acc[t][4 * i + 2][r], o.acc[t][4 * i + 3][r]);
    if (g == 0) sm[R * wave + 16 * t + n] = l == 0.0f ? -INFINITY : o.m[t], sl[R * wave + 16 * t + n] = l;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < R * (D / 4); e += 256) {
    const int row = e / (D / 4), d = 4 * (e % (D / 4));
    if (row0 + row >= w.rows) break;
    float top = -INFINITY, total = 0.0f;
    float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int x = 0; x < 4; ++x) top = fmaxf(top, sm[R * x + row]);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float f = top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(sm[R * x + row] - top);
      const float4 u = *reinterpret_cast<const float4 *>(so + (R * x + row) * D + d);
      total += f * sl[R * x + row];
      v.x += f * u.x, v.y += f * u.y, v.z += f * u.z, v.w += f * u.w;
    }
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    store_row<D, true>(a, w, row0 + row, d, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
  }
}

// The bf16 path. A workgroup mostly takes 128 rows (queries times the heads that share a
// kept head), 32 a wave, against tiles of 64 keys that its waves share in LDS.
// 32x32x16 products, transposed: S^T = K Q^T leaves lane (h, n) = (lane >> 5, lane
// & 31) 16 of the scores of row n per 32 keys (keys 8 i + 4 h + r), so a softmax step
// is within a lane up to one exchange with lane ^ 32, and its weights are the B
// operand of O^T = V^T P^T as they stand if k-slot 4 i + r of half h means key 8 i +
// 4 h + r. V^T's A operand in that order is two transposing LDS reads of 4 keys
// each.
//
// Weights are rounded to bf16 for that product (8 bits; their total is summed before): the second
// part that the decode kernel gives them would double one of the two products of a kernel that
// waits for the matrix cores. Error against 64 bits: 0.0021 of the result's size, 0.0016 with
// float32 weights, which is the result's own rounding.
//
// The products of a tile (1024 cycles of the matrix cores) and its softmax step (about
// 980 of the VALU) are phases of their own; two workgroups share a CU and are rarely
// in the same one. Measured level or slower: eight waves in two groups half a tile
// apart, with barriers between the phases (4096 tokens, 24 heads, no mask: 219
// us against 204, for the coarser workgroups), and the softmax step spread
// between the products of one wave (207; 8192 tokens, 32 heads, causal 519
// against 493): the clock falls by as much as the overlap gains (1.8 GHz).
//
// Few rows (a chunk of a prompt, or drafted tokens, on a long prefix) take 32 a workgroup
// instead, all waves the same ones: each goes through its share of the keys alone, with a
// tile of K and one of V of its own and no barriers, and they join their sums at the end.
// There the loads bound it: 128 KiB a CU in flight or in use, 82 GB/s a CU out of L2.
//
// Queries and sums pass LDS on their way too: rows in whole lines (12 packed prompts of up to
// 2048 tokens, 32 heads on 8: 184 us, 195 with each lane's 16 and 8 bytes straight from
// and to its row). A workgroup's start and end are still about six tiles' time.
//
// The tiles go from memory to LDS without passing registers, 16 bytes a lane;
// chunk c of a row lies at chunk c ^ swizzle(row), which spreads both the 16
// rows of a K read and the 4 rows x 64 bytes of a V read over all banks.
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;

template <int D> __host__ __device__ constexpr int swizzle(int row) {
  return D == 64 ? ((row >> 1) & 1) << 2 | ((row >> 2) & 3) : (row & 3) << 2 | ((row >> 2) & 3);
}

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ float across32(float x) {   // the value of lane ^ 32
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(threadIdx.x & 32 ? r[0] : r[1]);
}

constexpr int kKeys = 64;                            // keys of a tile

// 64 rows of D bf16 values from src (rows stride_bytes apart, `rows` of them
// there: the rest is not read) into LDS at dst, RUNS KiB by each wave. Written
// as instructions: these loads have no result registers, and the compiler,
// which cannot tell the tile they fill from the ones being read, would wait for
// them before the next LDS read. The wait is the caller's, before the barrier
// that publishes the tile.
template <int RUNS>
__device__ __forceinline__ void stage_tile(const uint8_t *src, int stride_bytes, int rows, uint32_t dst, int wave,
                                           const int *voff) {
  const uint64_t at = reinterpret_cast<uintptr_t>(src);
  const int lo = __builtin_amdgcn_readfirstlane((int)at), hi = __builtin_amdgcn_readfirstlane((int)(at >> 32));
  const int bytes = __builtin_amdgcn_readfirstlane(rows * stride_bytes);
#pragma unroll
  for (int i = 0; i < RUNS; ++i)
    asm volatile(
        "s_mov_b32 s84, %0\n\ts_mov_b32 s85, %1\n\ts_mov_b32 s86, %2\n\ts_mov_b32 s87, 0x20000\n\t"   // a raw buffer
        "s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %4, s[84:87], 0 offen lds"
        :
        : "s"(lo), "s"(hi), "s"(bytes), "s"(__builtin_amdgcn_readfirstlane((int)(dst + 1024 * (RUNS * wave + i)))),
          "v"(voff[i])
        : "memory", "s84", "s85", "s86", "s87");
}

// The barrier of a step: LDS reads of before are done where their products are, and none
// of after may move up
__device__ __forceinline__ void tile_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void staged_tiles_landed() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Few rows: waves that each hold a tile of K and one of V in LDS
template <int D> constexpr int few_waves() { return D == 256 ? 2 : 4; }

// A workgroup's 32 rows from its waves' sums over their keys, 32 / NW rows a wave
template <int D>
__device__ __forceinline__ void join_few(const PromptArgs &a, RowJob w, int lane, int wave, const f32x16 (&acc)[D / 32],
                                         float base, float l) {
  constexpr int NW = few_waves<D>(), RS = D + 4;     // (4 more: rows start in other banks)
  extern __shared__ float shm[];                     // [NW][32][RS] sums, [NW][32] bases, [NW][32] totals
  float *sb = shm + NW * 32 * RS, *sl = sb + NW * 32;
  const int h = lane >> 5, n = lane & 31;
  __syncthreads();                                   // the tiles' places are free
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; r += 4)
      *reinterpret_cast<float4 *>(shm + (32 * wave + n) * RS + 32 * i + 2 * r + 4 * h) =
          make_float4(acc[i][r], acc[i][r + 1], acc[i][r + 2], acc[i][r + 3]);
  if (h == 0) sb[32 * wave + n] = l == 0.0f ? -INFINITY : base, sl[32 * wave + n] = l;
  __syncthreads();
  constexpr int OWN = 32 / NW, LANES = 64 / OWN, PARTS = D / (4 * LANES);   // a wave's rows, a row's lanes
  const int at = OWN * wave + lane / LANES, row = w.row0 + at, d0 = 4 * (lane % LANES);
  float top = -INFINITY, total = 0.0f, f[NW];
#pragma unroll
  for (int x = 0; x < NW; ++x) top = fmaxf(top, sb[32 * x + at]);
#pragma unroll
  for (int x = 0; x < NW; ++x) {
    f[x] = top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(sb[32 * x + at] - top);
    total += f[x] * sl[32 * x + at];
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  bool bad = false;
  float4 v[PARTS];
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    v[i] = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int x = 0; x < NW; ++x) {
      const float4 u = *reinterpret_cast<const float4 *>(shm + (32 * x + at) * RS + 4 * LANES * i + d0);
      v[i].x += f[x] * u.x, v[i].y += f[x] * u.y, v[i].z += f[x] * u.z, v[i].w += f[x] * u.w;
    }
    v[i].x *= inv, v[i].y *= inv, v[i].z *= inv, v[i].w *= inv;
    bad |= !(fabsf(v[i].x) < INFINITY && fabsf(v[i].y) < INFINITY && fabsf(v[i].z) < INFINITY &&
             fabsf(v[i].w) < INFINITY);
  }
  w.row0 += OWN * wave;
  w.rows = min(w.rows, w.row0 + OWN);
  if (w.row0 >= w.rows) return;
  if (__any(bad)) {                                  // as in the kernel below, for the wave's rows
    rows_alone<D>(a, w, lane);
  } else if (row < w.rows) {
#pragma unroll
    for (int i = 0; i < PARTS; ++i) store_row<D, false>(a, w, row, 4 * LANES * i + d0, v[i]);
  }
}

template <int D, bool FEW>
__global__ void __launch_bounds__(FEW ? 64 * few_waves<D>() : 256, FEW || D == 256 ? 1 : 2)
    attn_prompt_bf16(PromptArgs a) {
  constexpr int KS = D / 16, DT = D / 32, RB = 2 * D, TB = kKeys * RB, NW = FEW ? few_waves<D>() : 4;
  constexpr int RUNS = TB / 1024 / (FEW ? 1 : NW);
  constexpr int R = FEW ? 32 : 32 * NW;              // rows of a workgroup
  // Two steps a turn of the loop, each with its tiles' places in the reads' offsets, or
  // one, and the addresses change: 16 VALU instructions more (prompts of 8192, 32 heads
  // on 8 of 128: 517 us, 510 with two), but two steps of heads of 256 spill registers
  // (4096, 16 on 2: 208 us, 179 with one).
  constexpr bool TWO = !FEW && D < 256;
  // LDS: K tiles at 0 and TB, V tiles at 2 TB and 3 TB; FEW: a wave's K at 2 TB wave, its V TB further
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 5, n = lane & 31;
  const int kvh = blockIdx.x % a.kv_heads, group = a.q_heads / a.kv_heads;
  const Spot spot = find_tile<R>(a, lane, blockIdx.x / a.kv_heads);
  if (spot.tile < 0) return;
  const Span sp = spot.span;
  const int row_wg = R * spot.tile, rows = (int)min((int64_t)sp.lq, a.max_q) * group;
  const int row0 = row_wg + (FEW ? 0 : 32 * wave);
  // A row's query and its place in q or out, from the tile's first query on; rows past the
  // last one: that one's. (x is the row and 1/2, over a group of up to 2^16 and below that
  // and 128: the float32 quotient is never off by as much as the half.)
  const int query_wg = row_wg / group, rem = row_wg - query_wg * group;
  const float per_group = __builtin_amdgcn_rcpf((float)group), last_x = (float)(rows - 1 - row_wg + rem) + 0.5f;
  const float x_wave = (float)(row0 - row_wg + rem) + 0.5f;
  auto element_of = [&](float x, int64_t stride) INLINED {
    x = fminf(x, last_x);
    const int query = (int)(x * per_group);
    return query * stride + ((int)x - query * group) * D;
  };
  const int64_t q_wg = sp.q0 + query_wg;
  const int query = query_wg + (int)(fminf(x_wave + (float)n, last_x) * per_group);
  const int shift = sp.lk - sp.lq;
  const int last = a.causal ? query + shift : sp.lk - 1;        // this lane's last key
  // keys up to first_wave are seen by all rows of the wave
  const int first_wave = a.causal ? row0 / group + shift : sp.lk - 1;
  const int end = (a.causal ? min(row_wg + R, rows) - 1 : 0) / group + (a.causal ? shift : sp.lk - 1) + 1;
  const int tiles = end > 0 ? (end + kKeys - 1) / kKeys : 0;

  // staging: lane i of run r of a wave writes LDS chunk 64 r + i of the wave's
  // part; the chunk of the row that belongs there is fetched
  int koff[RUNS], voff[RUNS];
#pragma unroll
  for (int i = 0; i < RUNS; ++i) {
    const int chunk = 64 * ((FEW ? 0 : RUNS * wave) + i) + lane, r = chunk / (RB / 16), c = chunk % (RB / 16);
    const int from = (c ^ swizzle<D>(r)) * 16;
    koff[i] = r * (int)(2 * a.k_stride) + from;
    voff[i] = r * (int)(2 * a.v_stride) + from;
  }
  const uint8_t *kp = reinterpret_cast<const uint8_t *>(a.k) + 2 * ((int64_t)sp.k0 * a.k_stride + (int64_t)kvh * D);
  const uint8_t *vp = reinterpret_cast<const uint8_t *>(a.v) + 2 * ((int64_t)sp.k0 * a.v_stride + (int64_t)kvh * D);
  const int k_step = (int)(2 * a.k_stride), v_step = (int)(2 * a.v_stride);
  auto stage_k = [&](int t) INLINED {
    stage_tile<RUNS>(kp + (int64_t)kKeys * t * k_step, k_step, min(kKeys, sp.lk - kKeys * t),
                     FEW ? 2 * TB * wave : (t & 1) * TB, FEW ? 0 : wave, koff);
  };
  auto stage_v = [&](int t) INLINED {
    stage_tile<RUNS>(vp + (int64_t)kKeys * t * v_step, v_step, min(kKeys, sp.lk - kKeys * t),
                     FEW ? 2 * TB * wave + TB : (2 + (t & 1)) * TB, FEW ? 0 : wave, voff);
  };

  // A wave's 32 queries come by way of the V tiles' places, rows in whole lines (straight into
  // registers, an instruction would fetch 32 bytes of each of 32 rows); sums leave likewise by
  // way of the K tiles'.
  constexpr int ROW_RUNS = 32 * RB / 1024;
  const uint32_t q_place = FEW ? 2 * TB * wave + TB : 2 * TB + 32 * RB * wave, out_place = 32 * RB * wave;
  auto stage_q = [&]() INLINED {
#pragma unroll
    for (int i = 0; i < ROW_RUNS; ++i) {
      const int chunk = 64 * i + lane, r = chunk / (RB / 16), c = chunk % (RB / 16);
      const uint16_t *from = reinterpret_cast<const uint16_t *>(a.q) + (q_wg * a.q_stride + (int64_t)kvh * group * D) +
                             (element_of(x_wave + (float)r, a.q_stride) + 8 * (c ^ swizzle<D>(r)));
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                   :
                   : "s"(__builtin_amdgcn_readfirstlane((int)(q_place + 1024 * i))), "v"(from)
                   : "memory");
    }
  };
  const int tile0 = FEW ? wave : 0;
  if (tile0 < tiles) {
    stage_k(tile0);
    stage_q();
  }
  __builtin_amdgcn_sched_barrier(0);                 // on their way while the rest is set up

  // LDS addresses of the reads: of K's k-steps and of V's dimension tiles (keys 4 h
  // on and 8 further), in the first of the two places
  const int al = lane & 15, gg = (lane >> 4) & 1, vrow = 4 * h + (al >> 2);
  uint32_t k_at[KS], v_at[DT][2];
#pragma unroll
  for (int i = 0; i < KS; ++i) k_at[i] = (FEW ? 2 * TB * wave : 0) + n * RB + (((2 * i + h) ^ swizzle<D>(n)) << 4);
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = vrow + 8 * e;
      v_at[i][e] = (FEW ? 2 * TB * wave + TB : 2 * TB) + r * RB + (((4 * i + 2 * gg + ((al & 3) >> 1)) ^ swizzle<D>(r)) << 4) + 8 * (al & 1);
    }
  typedef __attribute__((address_space(3))) const bf16x8 lds_bf16x8;
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  typedef short s16x8 __attribute__((ext_vector_type(8)));

  bf16x8 q[KS];
  auto read_q = [&]() INLINED {
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      const uint32_t at = q_place + n * RB + (((2 * i + h) ^ swizzle<D>(n)) << 4);
      uint4 u = __builtin_bit_cast(uint4, *reinterpret_cast<lds_bf16x8 *>((uintptr_t)at));
      u.x = (u.x & a.q_and) ^ a.q_xor, u.y = (u.y & a.q_and) ^ a.q_xor;
      u.z = (u.z & a.q_and) ^ a.q_xor, u.w = (u.w & a.q_and) ^ a.q_xor;
      q[i] = __builtin_bit_cast(bf16x8, u);
    }
    // in registers before the place is another tile's
#pragma unroll
    for (int i = 0; i < KS; ++i) asm volatile("" : "+v"(q[i]));
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  };

  f32x16 acc[DT], s[2];
  bf16x8 p[4];
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[i][r] = 0.0f;
  const float headroom = headroom_of(sp.lk);
  float m = -INFINITY, base = 0.0f, l = 0.0f;

  // Products FROM .. TO - 1 of a tile's NV + NS: O^T += V^T P^T of a tile, then S^T =
  // K Q^T of the next. The LDS reads are kept AHEAD products before their use, by
  // hand: left to itself the compiler reads late and a product waits for every
  // operand, or reads all at once.
  constexpr int NV = 4 * DT, NS = 2 * KS, AHEAD = 6;
  auto operand = [&](int j, int kv, int kk) INLINED {
    if (j >= NV) {
      const int i = (j - NV) >> 1, u = j & 1;
      return *reinterpret_cast<lds_bf16x8 *>((uintptr_t)(k_at[i] + 32 * RB * u + TB * kk));
    }
    const int w = j / DT, i = j % DT, at = 16 * RB * w + TB * kv;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(uintptr_t)(v_at[i][0] + at));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(uintptr_t)(v_at[i][1] + at));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  // the V tile is in place VP, the K tile in the other (!TWO: where the addresses say)
  auto products = [&](auto from, auto to, auto vp) INLINED {
    constexpr int F = decltype(from)::value, T = decltype(to)::value, VP = decltype(vp)::value;
    constexpr int KP = TWO ? 1 - VP : 0;
    bf16x8 ring[AHEAD];
#pragma unroll
    for (int j = F; j < F + AHEAD; ++j) ring[(j - F) % AHEAD] = operand(j, VP, KP);
    __builtin_amdgcn_sched_barrier(0);
#pragma clang loop unroll(full)
    for (int j = F; j < T; ++j) {
      const bf16x8 x = ring[(j - F) % AHEAD];
      if (j < NV) {
        acc[j % DT] = mfma32(x, p[j / DT], acc[j % DT]);
      } else {
        const int i = (j - NV) >> 1, u = j & 1;
        f32x16 zero;
#pragma unroll
        for (int r = 0; r < 16; ++r) zero[r] = 0.0f;
        s[u] = mfma32(x, q[i], i == 0 ? zero : s[u]);
      }
      if (j + AHEAD < T) ring[(j - F) % AHEAD] = operand(j + AHEAD, VP, KP);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto next_tiles = [&](bool v) INLINED {            // !TWO: the reads go on in the other place
    if constexpr (TWO) return;
#pragma unroll
    for (int i = 0; i < KS; ++i) k_at[i] ^= TB;
#pragma unroll
    for (int i = 0; i < DT; ++i) v_at[i][0] ^= v ? TB : 0, v_at[i][1] ^= v ? TB : 0;
  };
  typedef std::integral_constant<int, 0> first_t;
  typedef std::integral_constant<int, NV> mid_t;
  typedef std::integral_constant<int, 0> place0_t;
  typedef std::integral_constant<int, 1> place1_t;
  typedef std::integral_constant<int, NV + NS> all_t;
  auto softmax = [&](int t) INLINED {
    const int j0 = kKeys * t;
    if (j0 + kKeys - 1 > first_wave) {               // some row does not see some key of the tile
      const int rel = last - j0 - 4 * h;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[u][r] = 32 * u + 8 * (r >> 2) + (r & 3) <= rel ? s[u][r] : -INFINITY;
    }
    float mt = s[0][0];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 16; ++r) mt = fmaxf(mt, s[u][r]);
    mt = fmaf(fmaxf(mt, across32(mt)), a.abs_scale2, headroom);
    // the running maximum follows only where it is outgrown by 2^8: weights of
    // up to 2^8 lose nothing, and the sums are rarely rescaled
    if (__any(mt > m + 8.0f)) {
      // nothing summed yet: known by the row's maximum, as l is this half's keys only, and acc both
      // halves'
      const bool none = m == -INFINITY;
      m = fmaxf(m, mt);
      const float now = m == -INFINITY ? 0.0f : m;
      const float alpha = none ? 0.0f : __builtin_amdgcn_exp2f(base - now);
      base = now;
      l *= alpha;
#pragma unroll
      for (int i = 0; i < DT; ++i) acc[i] *= alpha;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[u][r] = __builtin_amdgcn_exp2f(fmaf(s[u][r], a.abs_scale2, -base));
        l += s[u][r];
      }
#pragma unroll
      for (int w = 0; w < 2; ++w)
        p[2 * u + w] = __builtin_bit_cast(
            bf16x8, make_uint4(pack_bf16(s[u][8 * w], s[u][8 * w + 1]), pack_bf16(s[u][8 * w + 2], s[u][8 * w + 3]),
                               pack_bf16(s[u][8 * w + 4], s[u][8 * w + 5]), pack_bf16(s[u][8 * w + 6], s[u][8 * w + 7])));
    }
    // done here: put off, the sum would keep all 32 weights in registers, and the
    // packing would go into the products' phase
    asm volatile("" : "+v"(l), "+v"(p[0]), "+v"(p[1]), "+v"(p[2]), "+v"(p[3]));
  };

  // Step t: the softmax step of tile t, then the values of tile t and the scores of tile
  // t + 1. Asked for before the products of step t - 1: K(t + 1) and V(t), whose places
  // were last read in step t - 2; the barrier between softmax step and products
  // finds them landed. Every wave goes through every tile of the workgroup: those
  // that see less would only wait, and one path keeps the sums in one place.
  auto ask = [&](int t) INLINED {
    if (t + 1 < tiles) stage_k(t + 1);
    if (t < tiles) stage_v(t);
  };
  if constexpr (FEW) {
    // every wave for itself, over every NW-th tile: the next K is asked for where the last
    // one's products end, and so is the next V
    auto landed = [&](bool more) INLINED {           // all, or all but the tile asked for last
      __builtin_amdgcn_sched_barrier(0);
      if (more) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(RUNS) : "memory");
      else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    };
    if (wave < tiles) {
      landed(false);
      read_q();
      stage_v(wave);
      products(mid_t(), all_t(), place0_t());
      if (wave + NW < tiles) stage_k(wave + NW);
      for (int t = wave;; t += NW) {
        const bool more = t + NW < tiles;
        softmax(t);
        landed(more);
        products(first_t(), mid_t(), place0_t());
        if (!more) break;
        stage_v(t + NW);
        landed(true);
        products(mid_t(), all_t(), place0_t());
        if (t + 2 * NW < tiles) stage_k(t + 2 * NW);
      }
    }
    join_few<D>(a, {kvh * group, group, kvh, row0, rows, sp.q0, sp.k0, sp.lk, shift}, lane, wave, acc, base,
                l + across32(l));
    return;
  }
  if (tiles > 0) {
    staged_tiles_landed();
    read_q();
    tile_barrier();
    ask(0);
    __builtin_amdgcn_sched_barrier(0);
    products(mid_t(), all_t(), std::integral_constant<int, TWO>());   // (K in place 0)
    next_tiles(false);
    auto step = [&](int t, auto vp) INLINED {
      softmax(t);
      staged_tiles_landed();
      tile_barrier();
      ask(t + 1);
      __builtin_amdgcn_sched_barrier(0);
      products(first_t(), all_t(), vp);
      next_tiles(true);
    };
    int t = 0;
    if constexpr (TWO)
      for (; t + 2 < tiles; t += 2) {
        step(t, place0_t());
        step(t + 1, place1_t());
      }
    for (; t + 1 < tiles; ++t) step(t, place0_t());  // (TWO: the last one, if their number is even)
    softmax(t);
    staged_tiles_landed();
    tile_barrier();
    if (TWO && (t & 1)) products(first_t(), mid_t(), place1_t());
    else products(first_t(), mid_t(), place0_t());
  }
  if (row0 >= rows) return;
  l += across32(l);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  float nans[4] = {0, 0, 0, 0};                      // 0, or NaN for a value that is not finite
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      acc[i][r] *= inv;
      nans[r & 3] = fmaf(acc[i][r], 0.0f, nans[r & 3]);
    }
  const float nan = (nans[0] + nans[1]) + (nans[2] + nans[3]);
  RowJob w = {kvh * group, group, kvh, row0, rows, sp.q0, sp.k0, sp.lk, shift};
  // a weight of 0 times an infinity or a NaN that the row does not see: such a
  // wave is done over, pair by pair
  if (__any(nan != nan)) {
    for (; w.row0 < min(row0 + 32, rows); w.row0 += 16) rows_alone<D>(a, w, lane);
    return;
  }
  // (the K tiles were last read before the last barrier)
  typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
  typedef __attribute__((address_space(3))) u32x2 lds_u32x2;
  typedef __attribute__((address_space(3))) const u32x4 lds_u32x4;
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      *reinterpret_cast<lds_u32x2 *>((uintptr_t)(out_place + n * RB + (((4 * i + r) ^ swizzle<D>(n)) << 4) + 8 * h)) =
          (u32x2){pack_bf16(acc[i][4 * r], acc[i][4 * r + 1]), pack_bf16(acc[i][4 * r + 2], acc[i][4 * r + 3])};
#pragma unroll
  for (int i = 0; i < ROW_RUNS; ++i) {
    const int chunk = 64 * i + lane, r = chunk / (RB / 16), c = chunk % (RB / 16);
    const u32x4 u = *reinterpret_cast<lds_u32x4 *>((uintptr_t)(out_place + r * RB + ((c ^ swizzle<D>(r)) << 4)));
    if (row0 + r < rows)
      *reinterpret_cast<u32x4 *>(reinterpret_cast<uint16_t *>(a.out) + (q_wg * a.out_stride + (int64_t)kvh * group * D) +
                                 (element_of(x_wave + (float)r, a.out_stride) + 8 * c)) = u;
  }
}

// ------------------------------------------------------------ argument checks

constexpr float kLog2e = 1.4426950408889634f;
bool valid_scale(float scale) { return std::isfinite(scale * kLog2e); }      // the kernels' exponentials are of base 2

template <bool READ, int FMT, int D>
int launch_kv(const KvIo &io, glq_dtype dt, hipStream_t st) {
  const uint64_t blocks = ((uint64_t)io.rows * (D / 8) + 255) / 256;
  auto kern = READ ? (dt == GLQ_F32 ? kv_read_k<FMT, D, true> : kv_read_k<FMT, D, false>)
                   : (dt == GLQ_F32 ? kv_append_k<FMT, D, true> : kv_append_k<FMT, D, false>);
  hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(256), 0, st, io);
  return hip_status(hipGetLastError(), READ ? "kv_read_k" : "kv_append_k");
}

template <bool READ, int FMT>
int launch_kv_dim(const KvIo &io, int d, glq_dtype dt, hipStream_t st) {
  return d == 64 ? launch_kv<READ, FMT, 64>(io, dt, st) : d == 128 ? launch_kv<READ, FMT, 128>(io, dt, st)
                                                                  : launch_kv<READ, FMT, 256>(io, dt, st);
}

template <bool READ>
int kv_io(const glq_kv_cache *C, void *k, void *v, glq_dtype dt, int64_t k_stride, int64_t v_stride,
          const int32_t *slots, int64_t tokens, void *hip_stream) {
  const int rc = check_cache(C);
  if (rc) return rc;
  if (!valid_dtype(dt) || tokens < 0) return GLQ_ERR_ARG;
  if (tokens == 0) return GLQ_OK;
  if (!valid_rows(k, k_stride, C->kv_heads, C->head_dim, dt) || !valid_rows(v, v_stride, C->kv_heads, C->head_dim, dt) ||
      !slots || (reinterpret_cast<uintptr_t>(slots) & 3))
    return GLQ_ERR_ARG;
  // threads are numbered in 32 bits
  if (tokens > 0x7FFFFFFF / ((int64_t)C->kv_heads * (C->head_dim / 8))) return GLQ_ERR_UNSUPPORTED;
  const KvIo io = {{C->k, C->v}, {C->k_scale, C->v_scale}, {k, v}, {k_stride, v_stride}, slots,
                   (uint32_t)(tokens * C->kv_heads), C->kv_heads,
                   log2_of(C->page_size), (uint32_t)(C->num_pages * C->page_size)};
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  switch (C->format) {
    case GLQ_KV_BF16: return launch_kv_dim<READ, GLQ_KV_BF16>(io, C->head_dim, dt, st);
    case GLQ_KV_INT8: return launch_kv_dim<READ, GLQ_KV_INT8>(io, C->head_dim, dt, st);
    default: return launch_kv_dim<READ, GLQ_KV_INT4>(io, C->head_dim, dt, st);
  }
}

int check_decode(const glq_kv_cache *C, int64_t batch, int32_t q_heads, int64_t max_len) {
  const int rc = check_cache(C);
  if (rc) return rc;
  if (batch < 0 || q_heads < 1 || q_heads % C->kv_heads || max_len < 0) return GLQ_ERR_ARG;
  if (max_len > 0x7FFFFFFF - 4096 || q_heads > 65536) return GLQ_ERR_UNSUPPORTED;
  const int64_t tiles = (q_heads / C->kv_heads + 15) / 16;
  if (batch > kMaxGroups / ((int64_t)C->kv_heads * tiles)) return GLQ_ERR_UNSUPPORTED;
  return GLQ_OK;
}

// Workgroups of a launch: as many as run at once, or half of that more than
// there are units where these are many; the units' parts are made to fit. Past
// the ticket counters (one a workgroup) units are not split.
constexpr int64_t kTickets = GLQ_ATTN_CTRL_BYTES / 4;
struct DecodePlan { int64_t units, groups, part_floats, ws_bytes; bool whole; };
DecodePlan decode_plan(const glq_kv_cache *C, int dt, int64_t batch, int32_t q_heads, int64_t max_len) {
  const int64_t group = q_heads / C->kv_heads, rows = group < 16 ? group : 16;
  const int64_t units = batch * C->kv_heads * ((group + 15) / 16), tiles = (max_len + 127) / 128;
  const int64_t once = kCus * decode_per_cu(C->head_dim, dt == GLQ_F32);
  DecodePlan p;
  p.units = units;
  p.groups = once > units + once / 2 ? once : units + once / 2;
  p.whole = p.groups > kTickets || tiles <= 1;
  if (p.whole) p.groups = units;
  else if (batch <= 64 && p.groups > units * tiles) p.groups = units * tiles;   // a part is a tile at least
  p.part_floats = rows * (C->head_dim + 4);
  p.ws_bytes = GLQ_ATTN_CTRL_BYTES + (p.whole ? 0 : p.groups * p.part_floats * 4);
  return p;
}

// Dynamic LDS above the default limit of 64 KiB, asked for once per kernel and device
template <auto Kernel> int allow_lds(size_t bytes) {
  if (bytes <= 64 * 1024) return GLQ_OK;
  static std::atomic<uint64_t> allowed{0};
  int dev = 0;
  const int rc = hip_status(hipGetDevice(&dev), "hipGetDevice");
  if (rc) return rc;
  if (dev < 64 && (allowed.load(std::memory_order_relaxed) >> dev & 1)) return GLQ_OK;
  const int rc2 = hip_status(hipFuncSetAttribute(reinterpret_cast<const void *>(Kernel),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes),
                             "hipFuncSetAttribute");
  if (rc2 == GLQ_OK && dev < 64) allowed.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  return rc2;
}

template <int FMT, int D, bool F32>
int launch_decode_kernel(const DecodeArgs &a, int64_t groups, hipStream_t st) {
  constexpr size_t shm = (4 * 16 * (D + 4) + 128) * sizeof(float);
  const int rc = allow_lds<attn_decode_k<FMT, D, F32>>(shm);
  if (rc) return rc;
  hipLaunchKernelGGL((attn_decode_k<FMT, D, F32>), dim3((unsigned)groups), dim3(256), shm, st, a);
  return hip_status(hipGetLastError(), "attn_decode_k");
}

template <int FMT, int D>
int launch_decode(const DecodeArgs &a, glq_dtype dt, int64_t groups, hipStream_t st) {
  return dt == GLQ_F32 ? launch_decode_kernel<FMT, D, true>(a, groups, st)
                       : launch_decode_kernel<FMT, D, false>(a, groups, st);
}

template <int FMT>
int launch_decode_dim(const DecodeArgs &a, int d, glq_dtype dt, int64_t groups, hipStream_t st) {
  return d == 64 ? launch_decode<FMT, 64>(a, dt, groups, st) : d == 128 ? launch_decode<FMT, 128>(a, dt, groups, st)
                                                                      : launch_decode<FMT, 256>(a, dt, groups, st);
}

template <auto Kernel>
int launch_rows(const PromptArgs &a, int64_t groups, int threads, size_t shm, hipStream_t st, const char *name) {
  if (groups > kMaxGroups) return GLQ_ERR_UNSUPPORTED;
  const int rc = allow_lds<Kernel>(shm);
  if (rc) return rc;
  hipLaunchKernelGGL(Kernel, dim3((unsigned)groups), dim3((unsigned)threads), shm, st, a);
  return hip_status(hipGetLastError(), name);
}

// workgroups of R rows that a launch can need: no sequence has more than max_q
// queries, and all together no more than total_q (no overflow: batch and rows are below 2^31, heads
// below 2^17, and the smaller of the two counts is below 2^46)
int64_t prompt_groups(const PromptArgs &a, int R) {
  const int64_t group = a.q_heads / a.kv_heads, one = (a.max_q * group + R - 1) / R;
  const int64_t all = (a.total_q * group) / R + a.batch;
  return (a.batch * one < all ? a.batch * one : all) * a.kv_heads;
}

template <int D>
int launch_prompt(const PromptArgs &a, bool f32, hipStream_t st) {
  if (!f32) {
    // Few rows, with the keys over the waves, where the card holds all workgroups of 32
    // rows at once (by LDS: one a CU, two with heads of 64) and sequences have more than two
    // tiles of keys on average. Us with workgroups of 128 rows and of 32, 32 heads on 8
    // of 128, causal: 64 tokens on 2000 39.3 and 22.5, on 30000 471 and 190, on 192
    // 10.3 and 9.3, on 64 8.3 and 9.0; four times 64 on 448 14.8 and 11.6, seven times (448
    // workgroups) 15.8 and 21.3. 16 heads on 2 of 64, 64 on 2000: 28.2 and 15.1; 8 on 1 of
    // 256: 77.2 and 53.1.
    constexpr int lds = 4 * kKeys * 2 * D, few_lds = few_waves<D>() * lds / 2;
    const int64_t few = prompt_groups(a, 32);
    if (few <= (D == 64 ? 2 : 1) * kCus && a.total_k > 2 * kKeys * a.batch)
      return launch_rows<attn_prompt_bf16<D, true>>(a, few, 64 * few_waves<D>(), few_lds, st, "attn_prompt_bf16");
    return launch_rows<attn_prompt_bf16<D, false>>(a, prompt_groups(a, 128), 256, lds, st, "attn_prompt_bf16");
  }
  // Heads of 64: 32 rows a workgroup where that leaves many for every CU, 16 otherwise: 12
  // prompts of 400, 32 heads on 32 (4,992 workgroups of 32) 124 us and 138, eight of 333 on
  // 1000, 16 on 2 (1,332) 148 and 141, 64 on 2000 48.5 and 29.9. Larger heads: two tiles'
  // sums and queries leave one workgroup a CU (eight of 333 on 1000, 16 on 4 of 128: 233 us and 184)
  const int64_t groups = prompt_groups(a, 32);
  constexpr size_t shm = 4 * 16 * (D + 2) * sizeof(float);
  if constexpr (D == 64)
    if (groups >= 8 * kCus) return launch_rows<attn_prompt_f32<D, 2>>(a, groups, 256, 2 * shm, st, "attn_prompt_f32");
  return launch_rows<attn_prompt_f32<D, 1>>(a, prompt_groups(a, 16), 256, shm, st, "attn_prompt_f32");
}

}  // namespace
}  // namespace glq

using namespace glq;

extern "C" int glq_kv_append(const glq_kv_cache *C, const void *k, const void *v, glq_dtype dt, int64_t k_stride,
                             int64_t v_stride, const int32_t *slots, int64_t tokens, void *hip_stream) {
  return kv_io<false>(C, const_cast<void *>(k), const_cast<void *>(v), dt, k_stride, v_stride, slots, tokens,
                      hip_stream);
}

extern "C" int glq_kv_read(const glq_kv_cache *C, const int32_t *slots, int64_t tokens, void *k, void *v,
                           glq_dtype dt, int64_t k_stride, int64_t v_stride, void *hip_stream) {
  return kv_io<true>(C, k, v, dt, k_stride, v_stride, slots, tokens, hip_stream);
}

extern "C" size_t glq_attn_decode_workspace(const glq_kv_cache *C, int64_t batch, int32_t q_heads, int64_t max_len) {
  if (check_decode(C, batch, q_heads, max_len)) return 0;
  // the need grows with the batch as long as units are split, and is the control words alone
  // beyond: the largest batch up to this one that is split needs most
  const int64_t each = (int64_t)C->kv_heads * ((q_heads / C->kv_heads + 15) / 16);
  int64_t bytes = 0;
  for (const int dt : {GLQ_F32, GLQ_BF16}) {
    const int64_t split = (kTickets - kCus * decode_per_cu(C->head_dim, dt == GLQ_F32) / 2) / each;
    for (const int64_t b : {batch, batch < split ? batch : split}) {
      const int64_t need = decode_plan(C, dt, b, q_heads, max_len).ws_bytes;
      bytes = need > bytes ? need : bytes;
    }
  }
  return (size_t)bytes;
}

extern "C" int glq_attn_decode(const glq_kv_cache *C, const void *q, glq_dtype dt, int64_t q_stride, int64_t batch,
                               int32_t q_heads, const int32_t *page_table, int64_t max_pages, const int32_t *lens,
                               int64_t max_len, float scale, void *out, int64_t out_stride, void *workspace,
                               size_t ws_bytes, void *hip_stream) {
  const int rc = check_decode(C, batch, q_heads, max_len);
  if (rc) return rc;
  if (!valid_dtype(dt) || !valid_scale(scale) || max_pages < 0) return GLQ_ERR_ARG;
  if (batch == 0) return GLQ_OK;
  if (max_len > (max_pages < 0x7FFFFFFF ? max_pages : 0x7FFFFFFF) * C->page_size) return GLQ_ERR_ARG;
  if (!valid_rows(q, q_stride, q_heads, C->head_dim, dt) || !valid_rows(out, out_stride, q_heads, C->head_dim, dt) ||
      !lens || (!page_table && max_len > 0) || (reinterpret_cast<uintptr_t>(lens) & 3) ||
      (reinterpret_cast<uintptr_t>(page_table) & 3))
    return GLQ_ERR_ARG;
  const DecodePlan p = decode_plan(C, dt, batch, q_heads, max_len);
  if (!workspace || ws_bytes < (size_t)p.ws_bytes ||
      (reinterpret_cast<uintptr_t>(workspace) & 255))
    return GLQ_ERR_WORKSPACE;
  const int32_t group = q_heads / C->kv_heads, tiles = (group + 15) / 16;
  const float scale2 = scale * kLog2e;
  const DecodeArgs a = {C->k, C->v, C->k_scale, C->v_scale, q, out, q_stride, out_stride, page_table, lens, max_pages,
                        max_len, C->kv_heads, group, tiles, log2_of(C->page_size), (int32_t)C->num_pages,
                        scale2 == 0.0f ? 1.0f : fabsf(scale2), scale2 == 0.0f ? 0.0f : copysignf(1.0f, scale2),
                        (int32_t)batch, (int32_t)p.part_floats,
                        p.whole ? 1 : 0,
                        // (where, and why: find_place)
                        C->head_dim == 128 && C->format != GLQ_KV_INT4 && p.groups >= kCus && p.units <= kCus
                            ? (int32_t)kCus : (int32_t)p.groups,
                        reinterpret_cast<unsigned int *>(workspace),
                        reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(workspace) + GLQ_ATTN_CTRL_BYTES)};
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  switch (C->format) {
    case GLQ_KV_BF16: return launch_decode_dim<GLQ_KV_BF16>(a, C->head_dim, dt, p.groups, st);
    case GLQ_KV_INT8: return launch_decode_dim<GLQ_KV_INT8>(a, C->head_dim, dt, p.groups, st);
    default: return launch_decode_dim<GLQ_KV_INT4>(a, C->head_dim, dt, p.groups, st);
  }
}

extern "C" int glq_attn_prompt(const glq_prompt *P, uint32_t flags, void *hip_stream) {
  if (!P || (flags & ~1u) || !valid_dtype(P->dt) || !valid_scale(P->scale)) return GLQ_ERR_ARG;
  if (P->q_heads < 1 || P->kv_heads < 1 || P->q_heads % P->kv_heads) return GLQ_ERR_ARG;
  if (P->total_q < 0 || P->total_k < 0 || P->batch < 0 || P->max_q < 0) return GLQ_ERR_ARG;
  if (!valid_dim(P->head_dim) || P->q_heads > 65536) return GLQ_ERR_UNSUPPORTED;
  if (P->total_q > 0x7FFFFFFF || P->total_k > 0x7FFFFFFF) return GLQ_ERR_UNSUPPORTED;
  // byte offsets within a tile of 64 rows are 32 bits wide
  if (P->k_stride > (1 << 22) || P->v_stride > (1 << 22)) return GLQ_ERR_UNSUPPORTED;
  if (P->batch == 0 || P->total_q == 0 || P->max_q == 0) return GLQ_OK;
  if (!P->cu_q || !P->cu_k || (reinterpret_cast<uintptr_t>(P->cu_q) & 3) || (reinterpret_cast<uintptr_t>(P->cu_k) & 3))
    return GLQ_ERR_ARG;
  if (!valid_rows(P->q, P->q_stride, P->q_heads, P->head_dim, P->dt) ||
      !valid_rows(P->out, P->out_stride, P->q_heads, P->head_dim, P->dt))
    return GLQ_ERR_ARG;
  if (P->total_k > 0 && (!valid_rows(P->k, P->k_stride, P->kv_heads, P->head_dim, P->dt) ||
                         !valid_rows(P->v, P->v_stride, P->kv_heads, P->head_dim, P->dt)))
    return GLQ_ERR_ARG;
  const int64_t most = P->max_q < P->total_q ? P->max_q : P->total_q;
  const bool f = P->dt == GLQ_F32;
  if (P->batch >= 0x7FFFFFFF || most * P->q_heads > 0x7FFFFFFF - 64) return GLQ_ERR_UNSUPPORTED;
  const float scale2 = P->scale * kLog2e;
  const PromptArgs a = {P->q, P->k, P->v, P->out, P->q_stride, P->k_stride, P->v_stride, P->out_stride, P->total_q,
                        P->total_k, P->cu_q, P->cu_k, most, P->q_heads, P->kv_heads, (int32_t)P->batch,
                        (flags & GLQ_ATTN_CAUSAL) ? 1 : 0,
                        scale2, scale2 == 0.0f ? 1.0f : fabsf(scale2), scale2 == 0.0f ? 0u : 0xFFFFFFFFu,
                        scale2 < 0.0f ? 0x80008000u : 0u};
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  switch (P->head_dim) {
    case 64: return launch_prompt<64>(a, f, st);
    case 128: return launch_prompt<128>(a, f, st);
    default: return launch_prompt<256>(a, f, st);
  }
}
