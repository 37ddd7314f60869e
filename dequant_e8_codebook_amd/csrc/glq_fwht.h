// glq_fwht.h -- the Walsh-Hadamard transform of a workgroup's elements in registers,
// lane exchanges and one LDS transpose (library-internal). Included by the kernels of single
// layers (glq_kernels.hip) and of grouped experts (glq_experts.hip); its lane exchange also by
// glq_step.hip.
#pragma once
#include <hip/hip_runtime.h>

namespace glq {
namespace {

// v of lane (lane ^ mask) within the wave, mask a power of two <= 32 known at
// compile time: DPP moves for masks below 16 (quad_perm for 1 and 2; a half-row
// mirror (lane ^ 7) then quad_perm [3,2,1,0] (lane ^ 3) for 4; a row mirror
// (lane ^ 15) then a half-row mirror for 8); for 16 and 32 the gfx950 lane
// swaps, VALU operations that need no trip through the LDS unit.
// v_permlane16_swap(a, b) exchanges the odd 16-lane rows of a with the even
// rows of b, v_permlane32_swap(a, b) the upper half of a with the lower half
// of b; with a = b = v, lane l finds v of lane l ^ 16 (l ^ 32) in the second
// result where bit 4 (bit 5) of l is clear and in the first where it is set.
#define GLQ_DPP(v, ctrl) __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), ctrl, 0xF, 0xF, false))
__device__ __forceinline__ float lane_xor(float v, int mask) {
  switch (mask) {
    case 1: return GLQ_DPP(v, 0xB1);
    case 2: return GLQ_DPP(v, 0x4E);
    case 4: return GLQ_DPP(GLQ_DPP(v, 0x141), 0x1B);
    case 8: return GLQ_DPP(GLQ_DPP(v, 0x140), 0x141);
    case 16: {
      const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
      return __uint_as_float((threadIdx.x & 16) ? r[0] : r[1]);
    }
    default: {
      const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
      return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
    }
  }
}
#undef GLQ_DPP

// Block FWHT over bits 0 .. logb - 1 of the flat index of 64 NW E elements
// (E = 1, 2, 4, 8, 16 per thread, NW = 4, 8 or 16 waves; 2^logb <= 64 NW E)
// held E per thread. On entry thread t holds elements E t + i in v[i]. The low
// L = log2 E + 6 bits are transformed in registers and across the lanes of the
// wave; when logb > L the values pass once through LDS (buf, 64 NW E + 64
// floats; a pad of 4 floats per 2^L elements keeps the reads conflict-free)
// and the remaining log2 NW bits are transformed the same way. Afterwards
// thread t holds element ly_elem<E, NW>(t, i, transposed) in v[i]: with
// e = lo + 2^L hi, either (E < NW) LPC = NW / E lanes share a column lo, lane
// sub of them holding hi = sub E + i, or (E >= NW) a thread holds the NW
// elements of each of its E / NW columns lo = t + 64 NW c, i = NW c + hi.
// Unscaled: (a, b) -> (a + b, a - b) at every stage.
template <int E, int NW = 16> struct LyF {
  static constexpr int LE = E == 1 ? 0 : E == 2 ? 1 : E == 4 ? 2 : E == 8 ? 3 : 4;
  static constexpr int L = LE + 6;
  static constexpr int WB = NW == 1 ? 0 : NW == 2 ? 1 : NW == 4 ? 2 : NW == 8 ? 3 : 4;
  static constexpr int LPC = E < NW ? NW / E : 1;  // lanes per column after the transpose
  static constexpr int CPT = E < NW ? 1 : E / NW;  // columns per thread after the transpose
};

template <int E, int NW = 16>
__device__ __forceinline__ int ly_elem(int tid, int i, bool transposed) {
  using F = LyF<E, NW>;
  if (!transposed) return E * tid + i;
  if constexpr (E < NW) {
    const int lo = tid / F::LPC, sub = tid % F::LPC;
    return lo + ((sub * E + i) << F::L);
  } else {
    return tid + 64 * NW * (i / NW) + ((i % NW) << F::L);
  }
}

template <int E>
__device__ __forceinline__ void ly_stage_regs(float (&v)[E], int s) {
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (!(i & (1 << s))) {
      const float a = v[i], b = v[i + (1 << s)];
      v[i] = a + b;
      v[i + (1 << s)] = a - b;
    }
}

// one butterfly stage across lane pairs (lane, lane ^ mask): the lower lane
// keeps a + b, the upper one a - b, as o + (+-1) v in one exact fma
template <int E>
__device__ __forceinline__ void ly_stage_lanes(float (&v)[E], int mask, bool upper) {
  const float sg = upper ? -1.0f : 1.0f;
#pragma unroll
  for (int i = 0; i < E; ++i) v[i] = fmaf(v[i], sg, lane_xor(v[i], mask));
}

// One butterfly stage across lane bit 4 (R16) or lane bit 5 for register
// pairs (a, b): the lane swap (16-lane rows, or 32-lane halves) exchanges the
// odd rows of a with the even rows of b, after which every lane holds both
// members of one butterfly pair in its two results (a pair of a in the even
// rows, a pair of b in the odd ones). The butterflies run in registers, and
// the same swap of the sums and differences puts every result back in place:
// four operations per two elements instead of a copy, a swap, a select and an
// fma per element.
template <int E, bool R16>
__device__ __forceinline__ void ly_stage_swap(float (&v)[E]) {
  static_assert(E >= 2 && E % 2 == 0, "register pairs");
#pragma unroll
  for (int p = 0; p < E; p += 2) {
    const auto r = R16 ? __builtin_amdgcn_permlane16_swap(__float_as_uint(v[p]), __float_as_uint(v[p + 1]), false, false)
                       : __builtin_amdgcn_permlane32_swap(__float_as_uint(v[p]), __float_as_uint(v[p + 1]), false, false);
    const float a = __uint_as_float(r[0]), b = __uint_as_float(r[1]);
    const float sum = a + b, dif = a - b;
    const auto t = R16 ? __builtin_amdgcn_permlane16_swap(__float_as_uint(sum), __float_as_uint(dif), false, false)
                       : __builtin_amdgcn_permlane32_swap(__float_as_uint(sum), __float_as_uint(dif), false, false);
    v[p] = __uint_as_float(t[0]);
    v[p + 1] = __uint_as_float(t[1]);
  }
}

// The stages above the wave (labels L .. logb - 1, logb > L): an LDS transpose
// to the layout of ly_elem(., ., true), then the butterflies there.
template <int E, int NW>
__device__ __forceinline__ void ly_fwht_cross(float (&v)[E], float *buf, int logb, int tid) {
  using F = LyF<E, NW>;
  constexpr int LE = F::LE, L = F::L;
  {
    float *w = buf + E * tid + 4 * (tid >> 6);         // element E tid + i at e + 4 (e >> L)
    if constexpr (E >= 4) {
#pragma unroll
      for (int i = 0; i < E; i += 4) *reinterpret_cast<float4 *>(w + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) w[i] = v[i];
    }
  }
  __syncthreads();
  if constexpr (E < NW) {
    const int lo = tid / F::LPC, sub = tid % F::LPC;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int hi = sub * E + i;
      v[i] = buf[lo + (hi << L) + 4 * hi];
    }
#pragma unroll
    for (int h = 0; h < F::WB; ++h) {
      if (L + h >= logb) break;
      if (h < LE) ly_stage_regs<E>(v, h);
      else ly_stage_lanes<E>(v, 1 << (h - LE), (sub >> (h - LE)) & 1);
    }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int hi = i % NW;
      v[i] = buf[tid + 64 * NW * (i / NW) + (hi << L) + 4 * hi];
    }
#pragma unroll
    for (int h = 0; h < F::WB; ++h) {
      if (L + h >= logb) break;
      ly_stage_regs<E>(v, h);
    }
  }
}

// FULL: the block is all 64 NW E elements (logb = L + log2 NW), so that every
// stage runs and none is tested at run time.
template <int E, int NW = 16, bool FULL = false>
__device__ __forceinline__ bool ly_fwht(float (&v)[E], float *buf, int logb_rt, int tid) {
  using F = LyF<E, NW>;
  constexpr int LE = F::LE, L = F::L;
  const int logb = FULL ? L + F::WB : logb_rt;
  const int lane = tid & 63;
#pragma unroll
  for (int s = 0; s < LE; ++s)
    if (s < logb) ly_stage_regs<E>(v, s);
#pragma unroll
  for (int s = 0; s < 6; ++s) {
    if (LE + s < logb) {
      if constexpr (E >= 2) {
        if (s == 4) { ly_stage_swap<E, true>(v); continue; }
        if (s == 5) { ly_stage_swap<E, false>(v); continue; }
      }
      ly_stage_lanes<E>(v, 1 << s, (lane >> s) & 1);
    }
  }
  if (logb <= L) return false;
  ly_fwht_cross<E, NW>(v, buf, logb, tid);
  return true;
}

// The lane stages of rb_fwht_wave pair lanes l and l ^ m for m = 1, 2, 7, 8:
// each partner read is a single DPP permutation (quad_perm for 1 and 2, the
// half-row mirror for 7, a rotation by 8 within 16-lane rows for 8), folded
// into one fused multiply-add per element. Stage j transforms bit j of
// rb_ell(l) (its pairs differ in exactly that bit), which makes the four
// stages the Hadamard transform over element bits 3..6. The lower member of
// a pair (bit j of rb_ell(l) clear) keeps a + b, the upper one a - b instead
// of b - a: the upper lane's value is then the negated result, a factor
// rb_sgn(l) = (-1)^popcount(rb_ell(l) & 15) that every later stage carries
// along unchanged (partners share it) and the output scale removes.
__device__ __forceinline__ int rb_ell(int l) { return l ^ (((l >> 2) & 1) * 3); }
__device__ __forceinline__ float rb_sgn(int l) { return (__popc(rb_ell(l) & 15) & 1) ? -1.0f : 1.0f; }
__device__ __forceinline__ int rb_elem(int p) {
  return (p & ~1023) | (p & 7) | (((p >> 3) & 1) << 9) | (rb_ell((p >> 4) & 63) << 3);
}

// One lane stage on 16 registers: v[i] += s * v[i] of the partner lane, the
// partner read by the DPP control CTRL of a v_fmac_f32_dpp (one VALU
// operation per element; the compiler does not fold a DPP move into a
// multiply-add). The leading s_nop gives the two wait states a DPP read needs
// after a VALU write of its source, which the compiler cannot see through the
// asm; inside the block each instruction reads its own register only.
#define RB_FMAC16(CTRL, S)                                                                                  \
  asm volatile("s_nop 1\n\t"                                                                                \
               "v_fmac_f32_dpp %0, %0, %16 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                          \
               "v_fmac_f32_dpp %1, %1, %16 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                          \
               "v_fmac_f32_dpp %2, %2, %16 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                          \
               "v_fmac_f32_dpp %3, %3, %16 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                          \
               "v_fmac_f32_dpp %4, %4, %16 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                          \
               "v_fmac_f32_dpp %5, %5, %16 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                          \
               "v_fmac_f32_dpp %6, %6, %16 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                          \
               "v_fmac_f32_dpp %7, %7, %16 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                          \
               "v_fmac_f32_dpp %8, %8, %16 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                          \
               "v_fmac_f32_dpp %9, %9, %16 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                          \
               "v_fmac_f32_dpp %10, %10, %16 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                        \
               "v_fmac_f32_dpp %11, %11, %16 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                        \
               "v_fmac_f32_dpp %12, %12, %16 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                        \
               "v_fmac_f32_dpp %13, %13, %16 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                        \
               "v_fmac_f32_dpp %14, %14, %16 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                        \
               "v_fmac_f32_dpp %15, %15, %16 " CTRL " row_mask:0xf bank_mask:0xf"                            \
               : "+v"(v[0]), "+v"(v[1]), "+v"(v[2]), "+v"(v[3]), "+v"(v[4]), "+v"(v[5]), "+v"(v[6]),         \
                 "+v"(v[7]), "+v"(v[8]), "+v"(v[9]), "+v"(v[10]), "+v"(v[11]), "+v"(v[12]), "+v"(v[13]),     \
                 "+v"(v[14]), "+v"(v[15])                                                                    \
               : "v"(S))

// The FWHT over a wave's 1024 labels (E = 16 registers a lane): registers,
// then the four DPP lane stages, then lane bits 4 and 5 by lane swaps.
// Lane bits 4 and 5 (element bits 7 and 8) without the swap back: register
// pairs (p, p + 8) trade lane bit 4, then lane bit 5, for register bit 3, and
// the butterfly results stay where the trade left them. Afterwards register
// bit 3 holds element bit 8, lane bit 5 element bit 7 and lane bit 4 element
// bit 9 (rb_elem_out); register bits 0..2 are still element bits 0..2, so a
// lane's 8 registers of one half are 8 consecutive elements.
template <bool R16>
__device__ __forceinline__ void rb_stage_swap_keep(float (&v)[16]) {
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const auto r = R16 ? __builtin_amdgcn_permlane16_swap(__float_as_uint(v[p]), __float_as_uint(v[p + 8]), false, false)
                       : __builtin_amdgcn_permlane32_swap(__float_as_uint(v[p]), __float_as_uint(v[p + 8]), false, false);
    const float a = __uint_as_float(r[0]), b = __uint_as_float(r[1]);
    v[p] = a + b;
    v[p + 8] = a - b;
  }
}

// element of register i of lane l after rb_fwht_wave<., true>
__device__ __forceinline__ int rb_elem_out(int l, int i) {
  return (i & 7) | ((rb_ell(l) & 15) << 3) | (((l >> 5) & 1) << 7) | (((i >> 3) & 1) << 8) | (((l >> 4) & 1) << 9);
}

template <int FIRST = 0, bool KEEP = false>
__device__ __forceinline__ void rb_fwht_wave(float (&v)[16], int lane) {
  // FIRST = 1: the caller has done register stage 0 (element bit 0);
  // KEEP: the last two stages leave the layout of rb_elem_out
#pragma unroll
  for (int s = FIRST; s < 4; ++s) ly_stage_regs<16>(v, s);
  const int ell = rb_ell(lane);
  const float s0 = (ell & 1) ? -1.0f : 1.0f, s1 = (ell & 2) ? -1.0f : 1.0f;
  const float s2 = (ell & 4) ? -1.0f : 1.0f, s3 = (ell & 8) ? -1.0f : 1.0f;
  RB_FMAC16("quad_perm:[1,0,3,2]", s0);   // lane ^ 1
  RB_FMAC16("quad_perm:[2,3,0,1]", s1);   // lane ^ 2
  RB_FMAC16("row_half_mirror", s2);       // lane ^ 7
  RB_FMAC16("row_ror:8", s3);             // lane ^ 8
  asm volatile("s_nop 1" ::);
  if constexpr (KEEP) {
    rb_stage_swap_keep<true>(v);
    rb_stage_swap_keep<false>(v);
  } else {
    ly_stage_swap<16, true>(v);
    ly_stage_swap<16, false>(v);
  }
}
#undef RB_FMAC16

}  // namespace
}  // namespace glq
