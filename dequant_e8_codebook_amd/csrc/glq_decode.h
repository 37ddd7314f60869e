// glq_decode.h -- device functions that rebuild E8 codebook weights inside a
// product (library-internal): the decode tables in LDS, the walk from stored
// indices to MFMA operands, index loads and conversions. Included by the
// kernels of single layers (glq_kernels.hip) and of grouped experts
// (glq_experts.hip).
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "glq.h"
#include "glq_tables.h"

namespace glq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------- LDS tables
// LDS layout of the decode tables: [RT][HT][R3 at 3 bpw]
constexpr uint32_t kLdsRt = 0;
constexpr uint32_t kLdsHt = kLdsRt + kRtBytes;
constexpr uint32_t kLdsR3 = kLdsHt + kHtBytes;

template <int BPW> struct TabCfg;
template <> struct TabCfg<2> { static constexpr uint32_t ht = kHtBf16Off, r3_bytes = 0; };
template <> struct TabCfg<3> { static constexpr uint32_t ht = kHtTOff, r3_bytes = kR3Bytes; };
template <> struct TabCfg<4> { static constexpr uint32_t ht = kHtTOff, r3_bytes = 0; };

template <int BPW>
constexpr uint32_t lds_table_bytes() { return kLdsR3 + TabCfg<BPW>::r3_bytes; }

// blob offset of LDS table byte pos
template <int BPW>
__device__ __forceinline__ uint32_t table_src(uint32_t pos) {
  return pos < kLdsHt ? kRtOff + pos : pos < kLdsR3 ? TabCfg<BPW>::ht + (pos - kLdsHt) : kR3Off + (pos - kLdsR3);
}

typedef __attribute__((address_space(3))) void lds_void_t;
typedef __attribute__((address_space(1))) void glb_void_t;

// Copy RT + the value table of this bit width (+ R3 at 3 bpw) into LDS (bytes
// 0 .. lds_table_bytes) with global-to-LDS loads: no registers held, nothing
// waited for here. Run r (1 KiB of the LDS image) is copied by wave r mod the
// wave count, lane i writing its bytes 16 i .. 16 i + 15. The caller waits
// with tables_landed() before the barrier that publishes the tables.
template <int BPW, int NT = 256>
__device__ __forceinline__ void load_tables(uint8_t *, const uint8_t *blob) {
  constexpr uint32_t total = lds_table_bytes<BPW>();
  constexpr uint32_t runs = total / 1024;
  static_assert(total % 1024 == 0 && kLdsHt % 1024 == 0 && kLdsR3 % 1024 == 0, "LDS table runs");
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (uint32_t r = wave; r < runs; r += NT / 64) {
    const uint32_t pos = 1024 * r + 16 * lane;
    __builtin_amdgcn_global_load_lds((glb_void_t *)(blob + table_src<BPW>(pos)), (lds_void_t *)(uintptr_t)(1024 * r),
                                     16, 0, 0);
  }
}

// wait for this wave's vector-memory loads, the table copies included
__device__ __forceinline__ void tables_landed() { __builtin_amdgcn_s_waitcnt(0x0F70); }   // vmcnt(0)

// LDS pointers built from absolute addresses. Every kernel that decodes uses
// dynamic LDS only (no static __shared__), so its dynamic region starts at
// offset 0 and the table offsets are compile-time constants that fold into
// the DS instructions' offset field (a pointer to the extern array would add
// its link-time base with a VALU add on every lookup).
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) const uint16_t lds_u16;
typedef __attribute__((address_space(3))) const u32x2_t lds_u64;
typedef __attribute__((address_space(3))) const u32x4_t lds_u128;
typedef __attribute__((address_space(3))) const uint32_t lds_u32;
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  return *reinterpret_cast<lds_u16 *>(static_cast<uintptr_t>(addr));
}
__device__ __forceinline__ uint32_t lds_rd32(uint32_t addr) {
  return *reinterpret_cast<lds_u32 *>(static_cast<uintptr_t>(addr));
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  const u32x2_t v = *reinterpret_cast<lds_u64 *>(static_cast<uintptr_t>(addr));
  return make_uint2(v.x, v.y);
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  const u32x4_t v = *reinterpret_cast<lds_u128 *>(static_cast<uintptr_t>(addr));
  return make_uint4(v.x, v.y, v.z, v.w);
}

typedef __attribute__((address_space(3))) uint16_t lds_u16_w;
typedef __attribute__((address_space(3))) float lds_f32_w;
__device__ __forceinline__ void lds_st16(uint32_t addr, uint32_t v) {
  *reinterpret_cast<lds_u16_w *>(static_cast<uintptr_t>(addr)) = static_cast<uint16_t>(v);
}
__device__ __forceinline__ void lds_stf(uint32_t addr, float v) {
  *reinterpret_cast<lds_f32_w *>(static_cast<uintptr_t>(addr)) = v;
}

// i' = i - 1 (mod 2^16) for the two 16-bit indices packed in a word.
__device__ __forceinline__ uint32_t pk_dec16(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(u16x2, w) - (u16x2)(1));
}

// Byte offsets (inside HT) of the low and high half-vectors of index i',
// from the record of its chunk (glq_tables.h): the low window is
// bfe(i', 0, t_lo) with t_lo in bits 0-4 of the record, the high window
// bfe(i', T, 2) with T in bits 0-4 of rec >> 16, and (rec >> 16) >> 2 is 8 HI.
__device__ __forceinline__ void rec_offsets(uint32_t ip, uint32_t rec, uint32_t &lo, uint32_t &hi) {
  lo = (rec & 0xFFE0u) + (__builtin_amdgcn_ubfe(ip, 0, rec) << 3);
  const uint32_t wh = rec >> 16;
  hi = (wh >> 2) + (__builtin_amdgcn_ubfe(ip, wh, 2) << 3);
}

// record of index i' = i - 1 mod 2^16 (RT entry i' >> 2 at byte i' & ~3)
__device__ __forceinline__ uint32_t rec_of(uint32_t ip) { return lds_rd32(kLdsRt + (ip & 0xFFFCu)); }

__device__ __forceinline__ uint32_t pk_add16(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(u16x2, a) + __builtin_bit_cast(u16x2, b));
}

// Stage-1 and stage-2 halves into operand form: 16-bit lanes M * a + b
// (mod 2^16), M = 2 at 3 bpw and 4 at 4 bpw (one packed multiply-add).
// MAD: the multiplier is hidden from the optimiser (an empty asm), which then
// emits one v_pk_mad_u16 instead of a shift and an add (the decode-GEMM with
// partial x~ tiles keeps the shift and add: there the one-instruction form
// cost registers)
template <uint16_t M, bool MAD = true>
__device__ __forceinline__ uint32_t pk_comb(uint32_t a, uint32_t b) {
  uint32_t mm = (uint32_t)M * 0x10001u;
  if constexpr (MAD) asm("" : "+s"(mm));
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(u16x2, a) * __builtin_bit_cast(u16x2, mm) +
                                          __builtin_bit_cast(u16x2, b));
}

// Decode one group into 8 x 16-bit operand values, coordinate t in half t of
// the result (uint4 = 8 halves). 2 bpw: bf16 of v. 3/4 bpw: bf16 of 192 + u
// with u = 4 v (3 bpw) or 8 v (4 bpw). ip1 = i1 - 1 mod 2^16; at 4 bpw
// a2 = i2 - 1 mod 2^16 too, at 3 bpw a2 = i2 (a direct table row).
template <int BPW>
__device__ __forceinline__ uint4 decode_ip(uint32_t ip1, uint32_t a2) {
  uint32_t lo, hi;
  rec_offsets(ip1, rec_of(ip1), lo, hi);
  const uint2 a = lds64(kLdsHt + lo);
  const uint2 b = lds64(kLdsHt + hi);
  if constexpr (BPW == 2) {
    (void)a2;
    return make_uint4(a.x, a.y, b.x, b.y);
  } else if constexpr (BPW == 3) {
    const uint4 r = lds128(kLdsR3 + (a2 << 4));
    return make_uint4(pk_comb<2>(a.x, r.x), pk_comb<2>(a.y, r.y), pk_comb<2>(b.x, r.z), pk_comb<2>(b.y, r.w));
  } else {
    uint32_t lo2, hi2;
    rec_offsets(a2, rec_of(a2), lo2, hi2);
    const uint2 c = lds64(kLdsHt + lo2);
    const uint2 d = lds64(kLdsHt + hi2);
    return make_uint4(pk_comb<4>(a.x, c.x), pk_comb<4>(a.y, c.y), pk_comb<4>(b.x, d.x), pk_comb<4>(b.y, d.y));
  }
}

// Same, from plain indices (i1, and i2 of its plane).
template <int BPW>
__device__ __forceinline__ uint4 decode_group(uint32_t i1, uint32_t i2, const uint8_t *) {
  return decode_ip<BPW>((i1 - 1u) & 0xFFFFu, BPW == 4 ? ((i2 - 1u) & 0xFFFFu) : i2);
}

// Decode of 8 groups split into phases, so that the LDS reads of one phase
// are in flight together: p1 the chunk records (and the direct residual rows
// at 3 bpw), p2 the half-vector offsets and reads, p3 the combine into
// operand form (as decode_ip). Each phase takes a range [G0, G1) of the
// groups, so a caller can stagger them. q1 / q2 hold the indices as
// decode_ip takes them.
template <int BPW, bool MAD = true>
struct Dec8 {
  uint32_t R1[8], R2[8];
  uint4 r3[8];
  uint2 va[8], vb[8], vc[8], vd[8];

  template <int G0 = 0, int G1 = 8>
  __device__ __forceinline__ void p1(const uint32_t (&q1)[8], const uint32_t (&q2)[8]) {
#pragma unroll
    for (int g = G0; g < G1; ++g) {
      R1[g] = rec_of(q1[g]);
      if constexpr (BPW == 4) R2[g] = rec_of(q2[g]);
      if constexpr (BPW == 3) r3[g] = lds128(kLdsR3 + (q2[g] << 4));
    }
  }
  template <int G0 = 0, int G1 = 8>
  __device__ __forceinline__ void p2(const uint32_t (&q1)[8], const uint32_t (&q2)[8]) {
#pragma unroll
    for (int g = G0; g < G1; ++g) {
      uint32_t lo, hi;
      rec_offsets(q1[g], R1[g], lo, hi);
      va[g] = lds64(kLdsHt + lo);
      vb[g] = lds64(kLdsHt + hi);
      if constexpr (BPW == 4) {
        uint32_t lo2, hi2;
        rec_offsets(q2[g], R2[g], lo2, hi2);
        vc[g] = lds64(kLdsHt + lo2);
        vd[g] = lds64(kLdsHt + hi2);
      }
    }
  }
  template <int G0 = 0, int G1 = 8>
  __device__ __forceinline__ void p3(uint4 (&out)[8]) {
#pragma unroll
    for (int g = G0; g < G1; ++g) {
      if constexpr (BPW == 2) out[g] = make_uint4(va[g].x, va[g].y, vb[g].x, vb[g].y);
      else if constexpr (BPW == 3)
        out[g] = make_uint4(pk_comb<2, MAD>(va[g].x, r3[g].x), pk_comb<2, MAD>(va[g].y, r3[g].y),
                            pk_comb<2, MAD>(vb[g].x, r3[g].z), pk_comb<2, MAD>(vb[g].y, r3[g].w));
      else
        out[g] = make_uint4(pk_comb<4, MAD>(va[g].x, vc[g].x), pk_comb<4, MAD>(va[g].y, vc[g].y),
                            pk_comb<4, MAD>(vb[g].x, vd[g].x), pk_comb<4, MAD>(vb[g].y, vd[g].y));
    }
  }
  // all phases at once
  __device__ __forceinline__ void run(const uint32_t (&q1)[8], const uint32_t (&q2)[8], uint4 (&out)[8]) {
    p1(q1, q2);
    p2(q1, q2);
    p3(out);
  }
};

// value of one decoded 16-bit operand as the exact float32 v
template <int BPW>
__device__ __forceinline__ float operand_value(uint32_t h16) {
  const float f = __uint_as_float(h16 << 16);
  if constexpr (BPW == 2) return f;
  else if constexpr (BPW == 3) return (f - kBiasValue) * 0.25f;
  else return (f - kBiasValue) * 0.125f;
}

// epilogue factors: z = post * (acc - bias * rowsum(x~)) with post = s (2 bpw),
// s/4 (3 bpw), s/8 (4 bpw) and bias = 0 / 192 / 192
template <int BPW> struct Epi;
template <> struct Epi<2> { static constexpr float bias = 0.0f, mul = 1.0f; };
template <> struct Epi<3> { static constexpr float bias = kBiasValue, mul = 0.25f; };
template <> struct Epi<4> { static constexpr float bias = kBiasValue, mul = 0.125f; };

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// bf16 bit patterns of two floats (a in bits 0-15), round to nearest even:
// one v_cvt_pk_bf16_f32 on gfx950
__device__ __forceinline__ uint32_t bf16x2_rne(float a, float b) {
  const f32x2_t v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

__device__ __forceinline__ uint16_t f32_to_bf16_rne(float f) { return (uint16_t)bf16x2_rne(f, 0.0f); }

__device__ __forceinline__ void store_out(void *y, glq_dtype dt, size_t off, float v) {
  if (dt == GLQ_F32) reinterpret_cast<float *>(y)[off] = v;
  else reinterpret_cast<uint16_t *>(y)[off] = f32_to_bf16_rne(v);
}

__device__ __forceinline__ uint32_t load_idx2(const void *idx2, size_t off, int bpw) {
  if (bpw == 3) return reinterpret_cast<const uint8_t *>(idx2)[off];
  return reinterpret_cast<const uint16_t *>(idx2)[off];
}

// Index loads of 8 consecutive groups of one weight row, kept as loaded so
// that nothing waits for them until gv_unpack (a computation on a loaded
// value placed right after its load would stall the wave there).
struct GvRaw { uint4 a, b; };

template <int BPW, bool G8>
__device__ __forceinline__ GvRaw gv_load_raw(const uint16_t *idx1, const void *idx2, int64_t row, int64_t G,
                                             int64_t g0) {
  // row is clamped to the layer; groups past G are clamped (they meet zero weight operands)
  GvRaw r;
  if constexpr (G8) {
    const int64_t off = row * G + min(g0, G - 8);
    r.a = *reinterpret_cast<const uint4 *>(idx1 + off);
    if constexpr (BPW == 3) {
      const uint2 b = *reinterpret_cast<const uint2 *>(reinterpret_cast<const uint8_t *>(idx2) + off);
      r.b = make_uint4(b.x, b.y, 0u, 0u);
    } else if constexpr (BPW == 4) {
      r.b = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(idx2) + off);
    } else {
      r.b = make_uint4(0u, 0u, 0u, 0u);
    }
  } else {
    uint32_t w1[8], w2[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int64_t o = row * G + min(g0 + u, G - 1);
      w1[u] = idx1[o];
      w2[u] = BPW == 2 ? 0u : load_idx2(idx2, o, BPW);
    }
    r.a = make_uint4(w1[0] | (w1[1] << 16), w1[2] | (w1[3] << 16), w1[4] | (w1[5] << 16), w1[6] | (w1[7] << 16));
    if constexpr (BPW == 3)
      r.b = make_uint4(w2[0] | (w2[1] << 8) | (w2[2] << 16) | (w2[3] << 24),
                       w2[4] | (w2[5] << 8) | (w2[6] << 16) | (w2[7] << 24), 0u, 0u);
    else
      r.b = make_uint4(w2[0] | (w2[1] << 16), w2[2] | (w2[3] << 16), w2[4] | (w2[5] << 16), w2[6] | (w2[7] << 16));
  }
  return r;
}

// i1 = i' = i - 1 mod 2^16 of stage 1; i2 = i' of stage 2 at 4 bpw, the plain
// residual row at 3 bpw
template <int BPW>
__device__ __forceinline__ void gv_unpack(const GvRaw &r, uint32_t (&i1)[8], uint32_t (&i2)[8]) {
  const uint32_t w[4] = {pk_dec16(r.a.x), pk_dec16(r.a.y), pk_dec16(r.a.z), pk_dec16(r.a.w)};
#pragma unroll
  for (int u = 0; u < 4; ++u) { i1[2 * u] = w[u] & 0xFFFFu; i1[2 * u + 1] = w[u] >> 16; }
  if constexpr (BPW == 3) {
#pragma unroll
    for (int u = 0; u < 4; ++u) { i2[u] = (r.b.x >> (8 * u)) & 0xFFu; i2[4 + u] = (r.b.y >> (8 * u)) & 0xFFu; }
  } else if constexpr (BPW == 4) {
    const uint32_t x[4] = {pk_dec16(r.b.x), pk_dec16(r.b.y), pk_dec16(r.b.z), pk_dec16(r.b.w)};
#pragma unroll
    for (int u = 0; u < 4; ++u) { i2[2 * u] = x[u] & 0xFFFFu; i2[2 * u + 1] = x[u] >> 16; }
  } else {
#pragma unroll
    for (int u = 0; u < 8; ++u) i2[u] = 0u;
  }
}

// stored indices -> decode inputs of groups u = 0..3 (as decode_ip takes them)
template <int BPW>
__device__ __forceinline__ void g8_split(uint2 i1, uint2 i2, uint32_t (&q1)[8], uint32_t (&q2)[8]) {
  const uint2 d1 = make_uint2(pk_dec16(i1.x), pk_dec16(i1.y));
  const uint2 d2 = BPW == 4 ? make_uint2(pk_dec16(i2.x), pk_dec16(i2.y)) : i2;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    q1[u] = ((u < 2 ? d1.x : d1.y) >> (16 * (u & 1))) & 0xFFFFu;
    if constexpr (BPW == 3) q2[u] = (d2.x >> (8 * u)) & 0xFFu;
    else if constexpr (BPW == 4) q2[u] = ((u < 2 ? d2.x : d2.y) >> (16 * (u & 1))) & 0xFFFFu;
    else q2[u] = 0u;
  }
}

// Issue pattern of one run of N MFMAs: after each, up to D LDS reads, V VALU operations,
// W LDS writes and M global loads.
template <int N, int V, int D, int W = 0, int M = 0>
__device__ __forceinline__ void gm_interleave() {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (D > 0) __builtin_amdgcn_sched_group_barrier(0x100, D, 0);
    if constexpr (V > 0) __builtin_amdgcn_sched_group_barrier(0x002, V, 0);
    if constexpr (W > 0) __builtin_amdgcn_sched_group_barrier(0x200, W, 0);
    if constexpr (M > 0) __builtin_amdgcn_sched_group_barrier(0x020, M, 0);
  }
}

}  // namespace
}  // namespace glq
