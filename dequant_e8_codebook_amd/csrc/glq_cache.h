// glq_cache.h -- the paged key-value cache's rows (library-internal): conversions,
// the write of a token's head, and the argument checks and error text of the calls on it. Included
// by the attention calls (glq_attn.hip), those of the step around them (glq_step.hip) and, for
// the checks and conversions, by those of the experts (glq_experts.hip).
#pragma once
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>

#include "glq.h"

namespace glq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

// The error text of this thread: glq_last_error()'s 256-byte buffer.
int hip_status(hipError_t e, const char *where = "launch") {
  if (e == hipSuccess) return GLQ_OK;
  snprintf(const_cast<char *>(glq_last_error()), 256, "%s: %s (%d)", where, hipGetErrorString(e), (int)e);
  return GLQ_ERR_HIP;
}

// two floats to packed bf16 (round to nearest even), one v_cvt_pk_bf16_f32
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}
// the high halves of two floats: exact where both are bf16 values
__device__ __forceinline__ uint32_t pack_high(float a, float b) {
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// 8 elements at p (16-byte aligned) as floats
template <bool F32>
__device__ __forceinline__ void load8(const void *p, float *x) {
  if constexpr (F32) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    x[0] = bf16_lo(u.x), x[1] = bf16_hi(u.x), x[2] = bf16_lo(u.y), x[3] = bf16_hi(u.y);
    x[4] = bf16_lo(u.z), x[5] = bf16_hi(u.z), x[6] = bf16_lo(u.w), x[7] = bf16_hi(u.w);
  }
}
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
template <bool STREAM> __device__ __forceinline__ void store16(void *p, u32x4 v) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(p));
  else *reinterpret_cast<u32x4 *>(p) = v;
}
// STREAM: written once, past the caches
template <bool F32, bool STREAM = false>
__device__ __forceinline__ void store8(void *p, const float *x) {
  if constexpr (F32) {
    store16<STREAM>(p, __builtin_bit_cast(u32x4, (f32x4){x[0], x[1], x[2], x[3]}));
    store16<STREAM>(reinterpret_cast<uint8_t *>(p) + 16, __builtin_bit_cast(u32x4, (f32x4){x[4], x[5], x[6], x[7]}));
  } else {
    store16<STREAM>(p, (u32x4){pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])});
  }
}

template <int N> __device__ __forceinline__ void load_words(const uint8_t *p, uint32_t *w) {
  if constexpr (N >= 4) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 u = reinterpret_cast<const uint4 *>(p)[i];
      w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
    }
  } else if constexpr (N == 2) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    w[0] = u.x, w[1] = u.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t *>(p);
  }
}

// ------------------------------------------------------------ cache write / read

template <int FMT> __host__ __device__ constexpr int row_bytes(int d) {
  return FMT == GLQ_KV_BF16 ? 2 * d : FMT == GLQ_KV_INT8 ? d : d / 2;
}

struct KvIo {
  void *cache[2];              // keys, values
  float *scale[2];
  void *dense[2];              // [tokens][heads][d], rows stride[] elements apart
  int64_t stride[2];
  const int32_t *slots;
  uint32_t rows;               // tokens * heads
  int32_t heads, page_shift;
  uint32_t capacity;           // slots in the cache
};

// Blocks go to the eight XCDs in turn; 16 neighbouring ones, which share the cache lines of
// a page's scales, go to the same one here (the prefix of 50,001 tokens below: 64.8 us, 67.0
// without: its lines came into all eight L2s).
__device__ __forceinline__ uint32_t near_block() {
  const uint32_t b = blockIdx.x;
  return b < (gridDim.x & ~127u) ? (b & ~127u) | (b & 7u) << 4 | ((b >> 3) & 15u) : b;
}

// One lane holds 8 elements of one (token, head) row of the keys and of the values,
// d / 8 lanes a row.
template <int D> struct KvPart {
  uint32_t slot;
  int64_t cached, dense[2];    // row of the cache, first element of the row in the dense operands
  __device__ __forceinline__ bool place(const KvIo &io) {
    const uint32_t row = (near_block() * 256u + threadIdx.x) / (D / 8);
    if (row >= io.rows) return false;                // whole rows leave together
    const uint32_t token = row / (uint32_t)io.heads;
    const int h = (int)(row - token * (uint32_t)io.heads);
    slot = (uint32_t)io.slots[token];
    // rows of the cache are [page][head][token of the page]
    const uint32_t page = slot >> io.page_shift, in_page = slot & ((1u << io.page_shift) - 1);
    cached = (((int64_t)page * io.heads + h) << io.page_shift) + in_page;
    dense[0] = token * io.stride[0] + (int64_t)h * D, dense[1] = token * io.stride[1] + (int64_t)h * D;
    return true;
  }
};

// the largest of x over the d / 8 lanes of a row
template <int LPR> __device__ __forceinline__ uint32_t row_max(uint32_t x) {
  auto with = [](uint32_t a, int b) { return a > (uint32_t)b ? a : (uint32_t)b; };
  x = with(x, __builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xF, 0xF, false));      // quad_perm: lane ^ 1, lane ^ 2
  x = with(x, __builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xF, 0xF, false));
  x = with(x, __builtin_amdgcn_mov_dpp((int)x, 0x141, 0xF, 0xF, false));     // half row mirror: the other four
  if constexpr (LPR >= 16) x = with(x, __builtin_amdgcn_mov_dpp((int)x, 0x140, 0xF, 0xF, false));   // row mirror
  if constexpr (LPR == 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = r[0] > r[1] ? r[0] : r[1];
  }
  return x;
}

// a = max |x| is taken on the bit patterns, so a NaN is the largest and reaches
// the scale. The quotient x Q / a comes from a's reciprocal r: y = xQ r, then y + (xQ
// - y a) r, which is the correctly rounded quotient where r is the correctly
// rounded reciprocal (Markstein); one division a lane instead of eight (16 ->
// 11 us for 8192 tokens of 8 heads of 128 into 4 bits, the same ones again). What is left:
// the launch for few tokens, and otherwise the memory's latency, with one row of a lane in flight:
// those 8192 in 13.9 us from tensors that no cache holds (3.1 TB/s; 15.9, 4.2, to bf16), 50,001 in 59
// (4.4; 76, 5.4).
template <int FMT, int D>
__device__ __forceinline__ void append_row(const KvIo &io, const KvPart<D> &p, int which, int at, const float *x) {
  uint8_t *out = reinterpret_cast<uint8_t *>(io.cache[which]) + p.cached * row_bytes<FMT>(D);
  if constexpr (FMT == GLQ_KV_BF16) {
    store8<false>(out + 16 * at, x);
  } else {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = __float_as_uint(x[i]) & 0x7FFFFFFFu;
      top = b > top ? b : top;
    }
    top = row_max<D / 8>(top);
    constexpr float Q = FMT == GLQ_KV_INT8 ? 127.0f : 7.0f;
    const float a = __uint_as_float(top);
    const bool codes = top > 0 && top < 0x7F800000u;  // a = 0, inf and NaN have codes 0
    // a moved away from the ends of the range by a power of two: exact, but for
    // elements that have code 0 anyway
    const float pre = a > 0x1p64f ? 0x1p-96f : a < 0x1p-64f ? 0x1p96f : 1.0f;
    const float b = codes ? a * pre : 1.0f, r = 1.0f / b, preq = codes ? pre * Q : 0.0f;
    int q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float n = codes ? x[i] * preq : 0.0f, y = n * r;
      q[i] = __float2int_rn(fmaf(fmaf(-y, b, n), r, y));
    }
    if constexpr (FMT == GLQ_KV_INT8) {
      uint32_t lo = 0, hi = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo |= (uint32_t)(q[i] & 255) << (8 * i);
        hi |= (uint32_t)(q[4 + i] & 255) << (8 * i);
      }
      *reinterpret_cast<uint2 *>(out + 8 * at) = make_uint2(lo, hi);
    } else {
      uint32_t w = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) w |= (uint32_t)(q[i] + 8) << (4 * i);
      *reinterpret_cast<uint32_t *>(out + 4 * at) = w;
    }
    // NaN for an infinity too: with a scale of inf, the codes of 0 would count on a score's sum being
    // exactly 0 to give NaN, and the 4-bit operands' is 0 up to rounding
    if (at == 0) io.scale[which][p.cached] = top < 0x7F800000u ? a / Q : NAN;
  }
}

// inclusive sum, or maximum of values from 0 on, over the lanes up to each (DPP
// row shifts and broadcasts; the whole wave's in lane 63)
template <bool MAX> __device__ __forceinline__ int wave_scan(int x) {
  auto with = [](int a, int b) { return MAX ? (a > b ? a : b) : a + b; };
  x = with(x, __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false));   // row_shr 1, 2, 4, 8
  x = with(x, __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false));
  x = with(x, __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false));
  x = with(x, __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false));
  x = with(x, __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false));   // row_bcast 15 into rows 1 and 3
  x = with(x, __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false));   // row_bcast 31 into rows 2 and 3
  return x;
}

// ------------------------------------------------------------ argument checks

bool valid_dtype(int dt) { return dt == GLQ_F32 || dt == GLQ_BF16; }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool valid_dim(int d) { return d == 64 || d == 128 || d == 256; }
// workgroups of 256 that a launch can have: its threads are counted in 32 bits
constexpr int64_t kMaxGroups = 0xFFFFFFFFu / 256;
int log2_of(int x) { return 31 - __builtin_clz((unsigned)x); }

int check_cache(const glq_kv_cache *C) {
  if (!C || C->format < GLQ_KV_BF16 || C->format > GLQ_KV_INT4) return GLQ_ERR_ARG;
  if (C->kv_heads < 1 || C->num_pages < 1) return GLQ_ERR_ARG;
  if (C->page_size < 16 || C->page_size > 1024 || (C->page_size & (C->page_size - 1))) return GLQ_ERR_ARG;
  if (!C->k || !C->v || !aligned16(C->k) || !aligned16(C->v)) return GLQ_ERR_ARG;
  if (C->format != GLQ_KV_BF16 && (!C->k_scale || !C->v_scale || !aligned16(C->k_scale) || !aligned16(C->v_scale)))
    return GLQ_ERR_ARG;
  if (!valid_dim(C->head_dim) || C->kv_heads > 65536) return GLQ_ERR_UNSUPPORTED;
  if (C->num_pages > 0x7FFFFFFF / C->page_size) return GLQ_ERR_UNSUPPORTED;
  return GLQ_OK;
}

// pointer and row stride (elements) of a [rows][heads][d] operand
bool valid_rows(const void *p, int64_t stride, int64_t heads, int64_t d, int dt) {
  const int64_t esize = dt == GLQ_F32 ? 4 : 2;
  return p && aligned16(p) && stride >= heads * d && stride < (int64_t(1) << 40) && (stride * esize) % 16 == 0;
}

}  // namespace
}  // namespace glq
