// glq_experts.hip -- compressed linears of experts on ragged groups of rows
// (gfx950), and their entry points of the C ABI.
//
// With the rows in the experts' order, row r of expert e: y_r = U_e^T (s_e W^_e) (V_e x_r),
// a layer as in glq_kernels.hip for each expert, all of them in three launches:
//   xp_in_k, xp_in_blk_k     x~_r = V_e x_r, rows gathered from their tokens
//   xp_gemm_k                z_r = W^_e x~_r, the weights rebuilt inside the product
//   xp_out_k, xp_out_blk_k   y_r = U_e^T (s_e z_r), or a token's weighted sum of them
// (_blk_k: rows of whole blocks of 1024 to 16384 elements; the others any multiple of 8). How many rows an expert has
// is known on the device only: launches are sized by the most there can be, and a workgroup without rows ends at once.
//
// What bounds them (times of the kernels on their own): 8192 rows, 1024 an expert, of 4096 through 4096 x 4096 at 2 bits: input
// transform 44 us (3.0 TB/s of rows read and x~ written; VALU 78% busy), product 250 us (1.10 PFLOP/s; the bf16 product of one
// layer of that size reaches the same), output transform 34.5 us (3.9 TB/s; VALU 72%). Few rows: 64 experts of 1024 x 2048 at 2 bits,
// 24 rows each: 8, 22.5 (1.5 TB/s of indices; the LDS unit is busy 45% of it, two thirds of that conflicts of the table lookups) and 4.8 us, of which
// about 4 each are the launch, the chain of dependent loads (offsets, rows, data) and in the product the copy of the tables.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <type_traits>

#include "glq.h"
#include "glq_cache.h"
#include "glq_decode.h"
#include "glq_fwht.h"

namespace glq {
namespace {

constexpr int kMaxExperts = 1024;
constexpr uint32_t kCus = 256;                       // of an MI355X; only how work is shared out hangs on it

// ------------------------------------------------------------ rows and experts

__device__ __forceinline__ int32_t bounded(int32_t x, int32_t most) { return x < 0 ? 0 : x < most ? x : most; }

// Expert of row r (0 <= r < the last offset): the number of experts that end at r or before. Every wave for itself.
__device__ __forceinline__ int expert_of(const int32_t *offsets, int count, int32_t r) {
  int e = 0;
  for (int c = threadIdx.x & 63; c < count; c += 64) e += __popcll(__ballot(offsets[c + 1] <= r));
  e = __builtin_amdgcn_readfirstlane(e);
  return e < count ? e : count - 1;
}

// ------------------------------------------------------------ row transforms

struct XpRows {
  const void *x;
  void *y;
  const int32_t *offsets, *src, *pos;
  const float *weights;
  const int8_t *sign_k, *sign_n;
  uint16_t *xt;                // [planes][rows][kp] bf16: x~, or three parts that add up to it; zeros from k on
  float *rowsum;               // [1 + ks][rows] sums of x~, whole and of each part along k (bf16 path)
  float *row_factor;           // [rows] what z's row is to be multiplied by, but for the transform's 1 / sqrt(block) and
  int32_t *row_expert;         // [rows] the power of two in the upper half of this (put_factor); the lower half: the expert
  int32_t *row_parts;          // [rows] parts along k of the row's tile (0: it had none) and 16 times its first part's row of zs
  const void *z;               // [rows][n] of rows in one part: float32 or float16, both without row_factor
  const float *zs;             // rows of n of those in several: part p's is zs_step rows times p further
  const float *scale, *row_scale;
  float unit;                  // of the operands: 1, 1/4 or 1/8 of a weight at 2, 3 or 4 bits
  int64_t k, kp, n, x_rows, out_rows;    // kp: k up to a multiple of 128
  int32_t count, rows, top, ks, zs_step;
  int log_k, log_n;            // Hadamard blocks
};

// The product's steps of 64 inputs, and the first one of part `part` of `parts`: steps come in pairs
constexpr int kGemmK = 64, kSplitSteps = 256;        // rows of more steps (16384 inputs) are not split
__device__ __forceinline__ int part_begin(int64_t steps, int part, int parts) { return 2 * (int)(steps / 2 * part / parts); }

// The transform of up to 64 NW E elements held E a thread, block 2^logb, each thread
// with its own elements again afterwards.
template <int E, int NW>
__device__ __forceinline__ void row_fwht(float (&v)[E], float *buf, int logb) {
  using F = LyF<E, NW>;
  const int tid = threadIdx.x;
  if (!ly_fwht<E, NW>(v, buf, logb, tid)) return;
  __syncthreads();                                   // buf is read
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int p = ly_elem<E, NW>(tid, i, true);
    buf[p + 4 * (p >> F::L)] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < E; ++i) v[i] = buf[E * tid + 4 * ((E * tid) >> F::L) + i];
}

__device__ __forceinline__ void load_signs8(const int8_t *p, float *s) {
  const uint2 u = *reinterpret_cast<const uint2 *>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = (float)(int8_t)((i < 4 ? u.x : u.y) >> (8 * (i & 3)));
}

// Between the product and U^T z is float32, and for many rows with x and y in bf16 float16, 11 bits, rounded once: that
// (2^-11 relative at most) adds 1% to the roundings of x~ and y (2^-8 each, at random and added in squares), and halves what is moved. Parts
// along k are float32 always, as sums are. So that any row fits its range, a row's x is taken
// times 2^-e, e = row_exponent, from the start, and z times 2^e at the end: with M the largest |x| and 2^c >= sqrt(k),
// the vector x 2^-e is at most 2 long, and so is x~; a weight row in units of the operands (8 v at 4 bits) is
// at most 8 * 1.25 sqrt(12) sqrt(k / 8) = 12.3 sqrt(k) long, so |z| < 24.6 sqrt(k), below 65504 up to k = 2^21 (35,600).
// At the other end, a row of k equal elements has its z around 8 and the most uneven one around 8 / sqrt(k): far above
// 2^-14 either way. The sums of the biased operands stay far from float32's ends as well.
__device__ __forceinline__ int row_exponent(uint32_t top, int64_t k) {
  if (top == 0 || top >= 0x7F800000u) return 0;
  int c = 0;
  while ((int64_t(1) << (2 * c)) < k) ++c;
  const int e = (int)(top >> 23);                    // (0: below the normal numbers, as 2^-126)
  return (e ? e - 127 : -126) + c;
}

// z's row is to be multiplied by scale 2^shift, which may leave float32's range where y does not: shift reaches 138, and a
// row of one large element has a z and a y far below M sqrt(k). So it is kept as a factor between 2^-60 and 2^60 and the
// power of two that is left, which z takes before its transform: with z 2^rest = y / factor, neither comes near the range's ends.
__device__ __forceinline__ void put_factor(const XpRows &a, int32_t r, int expert, float scale, int shift) {
  const int e = (int)(__float_as_uint(scale) >> 23 & 255u) - 127, all = e + shift, within = all < -60 ? -60 : all > 60 ? 60 : all;
  a.row_factor[r] = ldexpf(scale, within - e);
  a.row_expert[r] = (all - within) * 65536 + expert;
  a.row_parts[r] = 0;                                // (decreasing offsets: rows no tile is for)
}
static_assert(kMaxExperts <= 65536, "an expert's number in 16 bits");

// x times the signs, 8 elements at a time, or zeros
template <bool F32>
__device__ __forceinline__ void load_signed8(const XpRows &a, bool in, int64_t from, const int8_t *signs, int64_t o, float *v) {
  if (in && o < a.k) {
    float s[8];
    load8<F32>(reinterpret_cast<const uint8_t *>(a.x) + (F32 ? 4 : 2) * (from * a.k + o), v);
    load_signs8(signs + o, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= s[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  }
}

// One workgroup a row. bf16: x~ (times 2^-e) rounded to bf16, what the matrix cores take, and the sum of the
// rounded values, which the biased operands at 3 and 4 bits need. float32: x~ as three bf16 parts, which
// hold all of its 24 bits.
template <int E, int NW, bool F32>
__global__ void __launch_bounds__(64 * NW) xp_in_k(XpRows a) {
  extern __shared__ __attribute__((aligned(16))) float buf[];       // 64 NW E + 64
  __shared__ float part[NW];
  __shared__ uint32_t tops[NW];
  __shared__ float step_sum[F32 ? 1 : kSplitSteps];
  constexpr int SEG = 64 * NW * E;
  const int tid = threadIdx.x;
  const int32_t r = blockIdx.x;
  if (r < bounded(a.offsets[0], a.rows) || r >= bounded(a.offsets[a.count], a.rows)) return;
  const int e = expert_of(a.offsets, a.count, r);
  const int64_t from = a.src ? a.src[r] : r;
  const bool in = from >= 0 && from < a.x_rows;
  const int8_t *signs = a.sign_k + (int64_t)e * a.k;
  float v[E], inv = 1.0f / sqrtf((float)(1 << a.log_k)), sum = 0.0f;
  int shift = 0;
  for (int64_t s0 = F32 || a.kp <= SEG ? 0 : a.kp / SEG * SEG; s0 >= 0; s0 -= SEG) {     // (the first segment stays in v)
#pragma unroll
    for (int h = 0; h < E; h += 8) load_signed8<F32>(a, in, from, signs, s0 + E * tid + h, v + h);
    if constexpr (F32) break;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int m = (int)(__float_as_uint(v[i]) & 0x7FFFFFFFu);
      shift = shift > m ? shift : m;
    }
  }
  if constexpr (!F32) {
    uint32_t top = row_max<32>((uint32_t)shift);
    const auto both = __builtin_amdgcn_permlane32_swap(top, top, false, false);
    top = both[0] > both[1] ? both[0] : both[1];
    if constexpr (NW > 1) {
      if ((tid & 63) == 0) tops[tid >> 6] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < NW; ++w) top = top > tops[w] ? top : tops[w];
    }
    shift = row_exponent(top, a.k);
  }
  if (tid == 0) put_factor(a, r, e, a.scale[e] * a.unit, shift);
  for (int64_t s0 = 0; s0 < a.kp; s0 += SEG) {
    if (s0) {
#pragma unroll
      for (int h = 0; h < E; h += 8) load_signed8<F32>(a, in, from, signs, s0 + E * tid + h, v + h);
      __syncthreads();
    }
    if constexpr (!F32) {
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = ldexpf(v[i], -shift);
    }
    row_fwht<E, NW>(v, buf, a.log_k);
    float here = 0.0f;
#pragma unroll
    for (int h = 0; h < E; h += 8) {
      const int64_t o = s0 + E * tid + h;
      if (o >= a.kp) continue;                       // (from k on: zeros, as blocks end there)
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = v[h + i] * inv;
#pragma unroll
      for (int p = 0; p < (F32 ? 3 : 1); ++p) {
        uint16_t *to = a.xt + ((int64_t)p * a.rows + r) * a.kp + o;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          w[i / 2] = pack_bf16(x[i], x[i + 1]);
          const float lo = bf16_lo(w[i / 2]), hi = bf16_hi(w[i / 2]);
          if constexpr (F32) x[i] -= lo, x[i + 1] -= hi;
          else here += lo + hi;
        }
        *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    if constexpr (!F32) {
      sum += here;
      if (a.ks > 1) {                                // sums of steps: 64 / E lanes each
#pragma unroll
        for (int m = 1; m < 64 / E; m <<= 1) here += lane_xor(here, m);
        const int64_t o = s0 + E * tid;
        if (o % kGemmK == 0 && o < a.kp) step_sum[o / kGemmK] = here;
      }
    }
  }
  if constexpr (!F32) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) sum += lane_xor(sum, m);
    if ((tid & 63) == 0) part[tid >> 6] = sum;
    __syncthreads();
    if (tid == 0) {
      float all = 0.0f;
      for (int w = 0; w < NW; ++w) all += part[w];
      a.rowsum[r] = all;
    }
    if (a.ks > 1 && tid < a.ks) {
      const int64_t steps = a.kp / kGemmK;
      float some = 0.0f;
      for (int s = part_begin(steps, tid, a.ks); s < part_begin(steps, tid + 1, a.ks); ++s) some += step_sum[s];
      a.rowsum[(1 + tid) * (int64_t)a.rows + r] = some;
    }
  }
}

// 8 float16 values at p (16-byte aligned)
__device__ __forceinline__ void load_f16(const uint16_t *p, float *x) {
  typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
  const f16x8 v = *reinterpret_cast<const f16x8 *>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = (float)v[i];
}

// 8 floats from any multiple of 4 bytes on, as row scales may lie
__device__ __forceinline__ void load_words8(const float *p, float *x) {
  typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
  const f32x4_any a = reinterpret_cast<const f32x4_any *>(p)[0], b = reinterpret_cast<const f32x4_any *>(p)[1];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = a[i], x[4 + i] = b[i];
}

// One workgroup a row of y: a row's U^T z, or with `pos` the sum of a token's rows, each with its weight, in
// the order of its choices, in float32. Z16: z in float16. Parts along k are added up here.
template <int E, int NW, bool F32, bool Z16>
__global__ void __launch_bounds__(64 * NW) xp_out_k(XpRows a) {
  extern __shared__ __attribute__((aligned(16))) float buf[];
  const int tid = threadIdx.x;
  const int64_t row_y = blockIdx.x;
  const int32_t first = bounded(a.offsets[0], a.rows), end = bounded(a.offsets[a.count], a.rows);
  if (!a.pos && (row_y < first || row_y >= end)) return;
  const float inv = 1.0f / sqrtf((float)(1 << a.log_n));
  bool again = false;
  for (int64_t s0 = 0; s0 < a.n; s0 += 64 * NW * E) {
    float acc[E];
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = 0.0f;
    for (int j = 0; j < a.top; ++j) {
      const int32_t r = a.pos ? a.pos[row_y * a.top + j] : (int32_t)row_y;
      if (r < first || r >= end) continue;           // uniform
      const int expert = a.row_expert[r], e = expert & 0xFFFF, rest = expert >> 16;
      const int where = a.row_parts[r], parts = where & 15;
      const float w = (a.pos ? a.weights[row_y * a.top + j] * inv : inv) * a.row_factor[r];
      const int8_t *signs = a.sign_n + (int64_t)e * a.n;
      float v[E];
#pragma unroll
      for (int h = 0; h < E; h += 8) {
        const int64_t o = s0 + E * tid + h;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[h + i] = 0.0f;
        if (o >= a.n) continue;
        if (parts == 1) {
          if constexpr (Z16) load_f16(reinterpret_cast<const uint16_t *>(a.z) + (int64_t)r * a.n + o, v + h);
          else load8<true>(reinterpret_cast<const float *>(a.z) + (int64_t)r * a.n + o, v + h);
        } else {
          for (int p = 0; p < parts; ++p) {
            float x[8];
            load8<true>(a.zs + ((where >> 4) + (int64_t)p * a.zs_step) * a.n + o, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[h + i] += x[i];
          }
        }
        if (a.row_scale) {
          float x[8];
          load_words8(a.row_scale + (int64_t)e * a.n + o, x);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[h + i] *= x[i];
        }
      }
      if (rest)                                      // uniform, and rare
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = ldexpf(v[i], rest);
      if (again) __syncthreads();
      again = true;
      row_fwht<E, NW>(v, buf, a.log_n);
#pragma unroll
      for (int h = 0; h < E; h += 8) {
        const int64_t o = s0 + E * tid + h;
        if (o >= a.n) continue;
        float s[8];
        load_signs8(signs + o, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[h + i] = fmaf(v[h + i] * s[i], w, acc[h + i]);
      }
    }
#pragma unroll
    for (int h = 0; h < E; h += 8) {
      const int64_t o = s0 + E * tid + h;
      if (o < a.n) store8<F32>(reinterpret_cast<uint8_t *>(a.y) + (F32 ? 4 : 2) * (row_y * a.n + o), acc + h);
    }
  }
}

// ------------------------------------------------------------ rows of whole blocks of 1024 to 16384

// The same two transforms for rows of at most 16 waves of 1024 elements each, 16 a lane, NW waves a block. The wave's
// part is that of the single layers' block kernel (registers, one multiply-add a DPP lane stage, lane swaps that keep their
// layout); the waves of a block then exchange all their values through LDS, four at a time, each summing up its own
// signs of them: no transpose back, two barriers a row. Workgroups take runs of rows, whose next
// one is in flight while one is transformed. 8192 rows of 4096: in 44 us, out 34.5, and 67 and 52 by the general kernels
// above; one token's two rows 4.6 and 5.8 us.

constexpr int kRowWaves = 16;                        // most waves a row

// Transform over the waves of a block: v of wave w (in its block) becomes the sum over waves j of (-1)^|w & j| v_j.
// buf: 4 KiB a wave. A barrier lies between the callers' last use of buf and this.
template <int NW>
__device__ __forceinline__ void cross_waves(float (&v)[16], float4 *buf, int wave, int lane) {
  auto put = [&] {
#pragma unroll
    for (int q = 0; q < 4; ++q) buf[(4 * wave + q) * 64 + lane] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
  };
  auto add = [&](int from, float s) {                // v + s times the other's
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 f = buf[(4 * from + q) * 64 + lane];
      v[4 * q] = fmaf(f.x, s, v[4 * q]), v[4 * q + 1] = fmaf(f.y, s, v[4 * q + 1]);
      v[4 * q + 2] = fmaf(f.z, s, v[4 * q + 2]), v[4 * q + 3] = fmaf(f.w, s, v[4 * q + 3]);
    }
  };
  auto onto = [&](int from, float s) {               // s v + the other's
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 f = buf[(4 * from + q) * 64 + lane];
      v[4 * q] = fmaf(v[4 * q], s, f.x), v[4 * q + 1] = fmaf(v[4 * q + 1], s, f.y);
      v[4 * q + 2] = fmaf(v[4 * q + 2], s, f.z), v[4 * q + 3] = fmaf(v[4 * q + 3], s, f.w);
    }
  };
  auto sign = [&](int bit) { return wave & bit ? -1.0f : 1.0f; };
  auto four = [&](int b) {                           // bits b and 2 b of the wave's number
    const float s1 = sign(b), s2 = sign(2 * b);
    onto(wave ^ 3 * b, s1 * s2);
    add(wave ^ b, s2);
    add(wave ^ 2 * b, s1);
  };
  if constexpr (NW == 1) return;
  put();
  __syncthreads();
  if constexpr (NW == 2) onto(wave ^ 1, sign(1));
  else four(1);
  if constexpr (NW >= 8) {
    __syncthreads();
    put();
    __syncthreads();
    if constexpr (NW == 8) onto(wave ^ 4, sign(4));
    else four(4);
  }
}

// rows [r0, r1) of n from `first` on that workgroup b of `groups` takes
__device__ __forceinline__ void my_run(int64_t first, int64_t n, int32_t &r0, int32_t &r1) {
  r0 = (int32_t)(first + n * blockIdx.x / gridDim.x);
  r1 = (int32_t)(first + n * (blockIdx.x + 1) / gridDim.x);
}

template <int NW, bool F32>
__global__ void __launch_bounds__(64 * kRowWaves) xp_in_blk_k(XpRows a) {
  extern __shared__ __attribute__((aligned(16))) float4 cross[];
  __shared__ uint32_t tops[2][F32 ? 1 : kRowWaves];  // of this row and the one before, which waves of other blocks may still read
  __shared__ float sums[2][F32 ? 1 : kSplitSteps];   // of the steps of 64 elements, of this row and the one before
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
  // A workgroup for each row there can be: its row is known before the offsets are, and so are its loads.
  const bool each = gridDim.x == (uint32_t)a.rows;   // uniform
  int32_t sources = each && a.src ? a.src[blockIdx.x] : 0;
  const int32_t first = bounded(a.offsets[0], a.rows), end = bounded(a.offsets[a.count], a.rows);
  int32_t r0 = blockIdx.x, r1 = r0 + 1;
  if (!each) my_run(first, end > first ? end - first : 0, r0, r1);
  const int el = 1024 * wave + 8 * rb_ell(lane), eo = 1024 * wave + rb_elem_out(lane, 0);    // elements read, written (+ 512, + 256)
  constexpr int RAW = F32 ? 4 : 2;
  uint4 raw[RAW];
  auto load = [&](int64_t from, uint4 (&to)[RAW]) {
    if (from >= 0 && from < a.x_rows) {
      const uint4 *p = reinterpret_cast<const uint4 *>(reinterpret_cast<const uint8_t *>(a.x) + (F32 ? 4 : 2) * (from * a.k + el));
      if constexpr (F32) {
        to[0] = p[0], to[1] = p[1], to[2] = p[128], to[3] = p[129];
      } else {
        to[0] = p[0], to[1] = p[64];
      }
    } else {
#pragma unroll
      for (int i = 0; i < RAW; ++i) to[i] = make_uint4(0, 0, 0, 0);
    }
  };
  auto fetch = [&](int32_t r) {
    if (a.src && !each && ((r - r0) & 63) == 0) sources = r + lane < r1 ? a.src[r + lane] : -1;
    load(a.src ? __builtin_amdgcn_readlane(sources, (r - r0) & 63) : r, raw);
  };
  if (r0 < r1) fetch(r0);                            // (of any row there is room for)
  if (r0 >= r1 || r0 < first || r0 >= end) return;
  int e = 0;
  float scale = 0.0f;
  int32_t until = r0;                                // rows of e end here
  // float32: sign bits of the elements, two a word. bf16: (s0, s1) of a word's two elements, whose product with the word is the first
  // sum of the transform; that with (s0, -s1) is the first difference
  uint32_t flip[8];
  const int64_t steps = a.kp / kGemmK;
  const float inv = rb_sgn(lane) / sqrtf((float)(1 << a.log_k));
  // The sums of row r, once all its waves have written theirs: eight lanes of the first wave a part along k, then all parts
  auto finish = [&](int32_t r) {
    if (wave) return;
    const int p = lane >> 3;
    float some = 0.0f;
    if (p < a.ks)
      for (int s = part_begin(steps, p, a.ks) + (lane & 7); s < part_begin(steps, p + 1, a.ks); s += 8) some += sums[r & 1][s];
    some += lane_xor(some, 1);
    some += lane_xor(some, 2);
    some += lane_xor(some, 4);
    if (a.ks > 1 && p < a.ks && (lane & 7) == 0) a.rowsum[(1 + p) * (int64_t)a.rows + r] = some;
    some += lane_xor(some, 8);
    some += lane_xor(some, 16);
    some += lane_xor(some, 32);
    if (lane == 0) a.rowsum[r] = some;
  };
  for (int32_t r = r0; r < r1; ++r) {
    if (r >= until) {
      e = expert_of(a.offsets, a.count, r);
      until = bounded(a.offsets[e + 1], a.rows);
      scale = a.scale[e] * a.unit;
      const int8_t *signs = a.sign_k + (int64_t)e * a.k + el;
      const uint2 s0 = *reinterpret_cast<const uint2 *>(signs), s1 = *reinterpret_cast<const uint2 *>(signs + 512);
      const uint32_t s[4] = {s0.x, s0.y, s1.x, s1.y};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t two = s[i / 2] >> (16 * (i & 1));
        flip[i] = ((two & 0x80u) << 8 | (two & 0x8000u) << 16) | (F32 ? 0u : 0x3F803F80u);
      }
    }
    float v[16];
    uint32_t top = 0;
    if constexpr (F32) {
      const uint32_t w[16] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w,
                              raw[2].x, raw[2].y, raw[2].z, raw[2].w, raw[3].x, raw[3].y, raw[3].z, raw[3].w};
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(w[i] ^ (i & 1 ? flip[i / 2] & 0x80000000u : flip[i / 2] << 16));
    } else {
      uint32_t w[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
      u16x2 most = (u16x2)(0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, w[i] & 0x7FFF7FFFu));
        const bf16x2_t x2 = __builtin_bit_cast(bf16x2_t, w[i]);
        v[2 * i] = __builtin_amdgcn_fdot2_f32_bf16(x2, __builtin_bit_cast(bf16x2_t, flip[i]), 0.0f, false);
        v[2 * i + 1] = __builtin_amdgcn_fdot2_f32_bf16(x2, __builtin_bit_cast(bf16x2_t, flip[i] ^ 0x80000000u), 0.0f, false);
      }
      top = most.x > most.y ? most.x : most.y;
      top = row_max<32>(top);
      const auto both = __builtin_amdgcn_permlane32_swap(top, top, false, false);
      top = both[0] > both[1] ? both[0] : both[1];
      if (lane == 0) tops[r & 1][wave] = top;
    }
    if (r + 1 < r1) fetch(r + 1);
    if (waves > 1) __syncthreads();                  // tops; the exchange and the sums of the row before are through
    int shift = 0, before = 0;
    if constexpr (!F32) {
      if (r > r0) finish(r - 1);
      for (int w = 0; w < waves; ++w) top = top > tops[r & 1][w] ? top : tops[r & 1][w];
      shift = row_exponent(top << 16, a.k);
      // 2^-shift waits for the end, where it costs nothing, unless sums of 16384 could leave float32's range before: such rows
      // are read again, as their first sums are among those
      if (shift > 100 || shift < -100) {             // uniform, and rare
        before = -shift;
        uint4 again[RAW];
        load(a.src ? a.src[r] : r, again);
        const uint32_t w[8] = {again[0].x, again[0].y, again[0].z, again[0].w, again[1].x, again[1].y, again[1].z, again[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t u = w[i] ^ (flip[i] & 0x80008000u);
          const float lo = ldexpf(bf16_lo(u), before), hi = ldexpf(bf16_hi(u), before);
          v[2 * i] = lo + hi, v[2 * i + 1] = lo - hi;
        }
      }
    }
    if (tid == 0) put_factor(a, r, e, scale, shift);
    rb_fwht_wave<F32 ? 0 : 1, true>(v, lane);
    cross_waves<NW>(v, cross, wave, lane);
    const float scaled = ldexpf(inv, -shift - before);
    float here[2] = {0.0f, 0.0f};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = v[8 * h + i] * scaled;
#pragma unroll
      for (int p = 0; p < (F32 ? 3 : 1); ++p) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          w[i / 2] = pack_bf16(x[i], x[i + 1]);
          if constexpr (F32) x[i] -= bf16_lo(w[i / 2]), x[i + 1] -= bf16_hi(w[i / 2]);
          else here[h] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, w[i / 2]),
                                                         __builtin_bit_cast(bf16x2_t, 0x3F803F80u), here[h], false);
        }
        *reinterpret_cast<uint4 *>(a.xt + ((int64_t)p * a.rows + r) * a.kp + eo + 256 * h) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    if constexpr (!F32) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {                  // eight neighbouring lanes have a step's 64 elements
        here[h] += lane_xor(here[h], 1);
        here[h] += lane_xor(here[h], 2);
        here[h] += lane_xor(here[h], 4);
        if ((lane & 7) == 0) sums[r & 1][(eo + 256 * h) / kGemmK] = here[h];
      }
    }
  }
  if constexpr (!F32) {
    __syncthreads();
    finish(r1 - 1);
  }
}

// Items are rows of z: the rows themselves, or each token's choices. A wave's lanes look up 64 items at a time (row, expert,
// factor), so the chain of loads behind a choice is gone through once for them all. With few tokens a workgroup has several sets
// of waves (blockDim over the row's waves): set s takes choices s, s + sets, ... and the sets' sums meet in LDS, always in
// the same order.
template <int NW, bool F32, bool Z16>
__global__ void __launch_bounds__(64 * kRowWaves) xp_out_blk_k(XpRows a) {
  extern __shared__ __attribute__((aligned(16))) float4 cross[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int waves = (int)(a.n >> 10), sets = (int)(blockDim.x >> 6) / waves, set = wave / waves;
  const int32_t first = bounded(a.offsets[0], a.rows), end = bounded(a.offsets[a.count], a.rows);
  int32_t y0, y1;
  my_run(a.pos ? 0 : first, a.pos ? a.out_rows : end > first ? end - first : 0, y0, y1);
  if (y0 >= y1) return;
  const int el = 1024 * (wave - set * waves) + 8 * rb_ell(lane), eo = 1024 * (wave - set * waves) + rb_elem_out(lane, 0);
  const float inv = 1.0f / sqrtf((float)(1 << a.log_n));
  constexpr int RAW = Z16 ? 2 : 4;
  const int turns = (a.top + sets - 1) / sets;       // items of a token that a set has
  const int64_t items = (int64_t)(y1 - y0) * turns;
  int32_t row = -1, expert = 0, where = 0;           // of item base + lane
  float factor = 0.0f;
  int64_t base = -64;
  struct Item { int32_t row, where, expert; float factor; uint4 raw[RAW]; uint2 sign[2]; };
  auto load_row = [&](const float *row, uint4 (&raw)[4]) {
    const uint4 *z = reinterpret_cast<const uint4 *>(row + el);
    raw[0] = z[0], raw[1] = z[1], raw[2] = z[128], raw[3] = z[129];
  };
  auto part = [&](int p, const Item &it) { return a.zs + ((it.where >> 4) + (int64_t)p * a.zs_step) * a.n; };
  auto fetch = [&](int64_t i, Item &it) {
    if (i >= base + 64) {
      base = i;
      row = -1;
      const int64_t mine = i + lane, y = mine / turns;
      const int j = (int)(mine - y * turns) * sets + set;
      if (mine < items && j < a.top) {
        row = a.pos ? a.pos[(y0 + y) * a.top + j] : (int32_t)(y0 + y);
        if (row < first || row >= end) row = -1;
        factor = inv;
        if (a.pos) factor *= a.weights[(y0 + y) * a.top + j];
      }
      if (row >= 0) {
        expert = a.row_expert[row], where = a.row_parts[row];
        factor *= a.row_factor[row];
        if (where == 0) row = -1;
      }
    }
    const int at = (int)(i - base);
    it.row = __builtin_amdgcn_readlane(row, at);
    if (it.row < 0) return;
    it.where = __builtin_amdgcn_readlane(where, at);
    it.factor = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(factor), at));
    it.expert = __builtin_amdgcn_readlane(expert, at);
    if constexpr (Z16) {                             // (parts, of a launch's last units, are asked for when their turn comes)
      if ((it.where & 15) == 1) {                    // uniform
        const uint4 *z = reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(a.z) + (int64_t)it.row * a.n + el);
        it.raw[0] = z[0], it.raw[1] = z[64];
      }
    } else {                                         // (one address and no branch: where paths with other loads met, they were waited for)
      const float *whole = reinterpret_cast<const float *>(a.z) + (int64_t)it.row * a.n;
      load_row((it.where & 15) == 1 ? whole : part(0, it), it.raw);
    }
    const int8_t *signs = a.sign_n + (int64_t)(it.expert & 0xFFFF) * a.n + eo;
    it.sign[0] = *reinterpret_cast<const uint2 *>(signs), it.sign[1] = *reinterpret_cast<const uint2 *>(signs + 256);
  };
  typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
  auto spread = [&](const uint4 (&raw)[4], float (&x)[16]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      x[4 * q] = __uint_as_float(raw[q].x), x[4 * q + 1] = __uint_as_float(raw[q].y);
      x[4 * q + 2] = __uint_as_float(raw[q].z), x[4 * q + 3] = __uint_as_float(raw[q].w);
    }
  };
  float acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
  Item next;
  fetch(0, next);
  int turn = 0;
  int32_t y = y0;
  for (int64_t i = 0; i < items; ++i) {
    const Item it = next;
    if (i + 1 < items) fetch(i + 1, next);
    float v[16];
    if (it.row >= 0) {
      const int parts = it.where & 15;
      if constexpr (Z16) {
        if (parts > 1) {
          uint4 raw[4];
          load_row(part(0, it), raw);
          spread(raw, v);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const f16x8 f = __builtin_bit_cast(f16x8, it.raw[h]);
#pragma unroll
            for (int q = 0; q < 8; ++q) v[8 * h + q] = (float)f[q];
          }
        }
      } else {
        spread(it.raw, v);
      }
      for (int p = 1; p < parts; ++p) {
        uint4 raw[4];
        float x[16];
        load_row(part(p, it), raw);
        spread(raw, x);
#pragma unroll
        for (int q = 0; q < 16; ++q) v[q] += x[q];
      }
      if (a.row_scale) {
        const int64_t e = it.expert & 0xFFFF;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x[8];
          load_words8(a.row_scale + e * a.n + el + 512 * h, x);
#pragma unroll
          for (int q = 0; q < 8; ++q) v[8 * h + q] *= x[q];
        }
      }
      if (it.expert >> 16)                           // uniform, and rare (put_factor)
#pragma unroll
        for (int q = 0; q < 16; ++q) v[q] = ldexpf(v[q], it.expert >> 16);
      rb_fwht_wave<0, true>(v, lane);
    } else if (sets > 1) {                           // (the other sets may have a row: the exchange's barriers are all waves')
#pragma unroll
      for (int q = 0; q < 16; ++q) v[q] = 0.0f;
    }
    if (it.row >= 0 || sets > 1) {
      cross_waves<NW>(v, cross, wave, lane);
      if (it.row >= 0) {
        // the factor with each output sign put in its place
        const float f = it.factor * rb_sgn(lane);
        const uint32_t turn = f < 0.0f ? 0x80808080u : 0u;
        const uint32_t s[4] = {it.sign[0].x ^ turn, it.sign[0].y ^ turn, it.sign[1].x ^ turn, it.sign[1].y ^ turn};
#pragma unroll
        for (int q = 0; q < 16; ++q)
          acc[q] = fmaf(v[q], copysignf(f, __uint_as_float(s[q / 4] << (24 - 8 * (q & 3)))), acc[q]);
      }
      if constexpr (NW > 1) __syncthreads();         // the exchange is read
    }
    if (++turn == turns) {
      if (sets > 1) {
        if (set > 0)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            cross[(4 * wave + q) * 64 + lane] = make_float4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]);
        __syncthreads();
        if (set == 0)
          for (int s = 1; s < sets; ++s)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float4 f = cross[(4 * (wave + s * waves) + q) * 64 + lane];
              acc[4 * q] += f.x, acc[4 * q + 1] += f.y, acc[4 * q + 2] += f.z, acc[4 * q + 3] += f.w;
            }
        __syncthreads();
      }
      if (set == 0)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          store8<F32>(reinterpret_cast<uint8_t *>(a.y) + (F32 ? 4 : 2) * ((int64_t)y * a.n + eo + 256 * h), acc + 8 * h);
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[q] = 0.0f;
      turn = 0;
      ++y;
    }
  }
}

// ------------------------------------------------------------ the product

struct XpProduct {
  const uint16_t *idx1, *xt;
  const void *idx2;
  const uint8_t *cb;
  const float *rowsum;
  const int32_t *offsets;
  int32_t *row_parts;
  void *z;                     // [rows][n], and the parts' sums beside: as in XpRows
  float *zs;
  int64_t n, k, kp;
  int32_t count, rows;
  int32_t zs_step;             // `rows`, or with zs_own the rows of a tile
  bool zs_own;                 // each unit has rows of zs to itself
  bool z16;                    // z in float16
  uint32_t n_groups;           // of 256 weight rows
  uint32_t likely;             // workgroups that very likely have a tile
  int32_t ks;                  // parts along k, at most, of the rows that are split
};

// biased operands (bf16 of 192 + u) to bf16 of u, exact
__device__ __forceinline__ uint4 unbiased(uint4 w) {
  auto two = [](uint32_t u) { return pack_high(bf16_lo(u) - kBiasValue, bf16_hi(u) - kBiasValue); };
  return make_uint4(two(w.x), two(w.y), two(w.z), two(w.w));
}

// ------------------------------------------------------------ 256 by 256 tiles

typedef float f32x16 __attribute__((ext_vector_type(16)));

// A tile: rows row0 .. row1 - 1 of expert e, its weight rows from 256 group on, part `part` of `parts` along k.
// zs: row of part 0's sums of row0.
struct XpTile { int e; int32_t row0, row1; uint32_t group; int part, parts; int32_t zs; };

// The launch's tiles, numbered. Units are groups of tm rows of an expert, whole ones first, then the experts'
// remainders, which are shorter. Where the last round on the card has few enough tiles, its units are split along k, into as many of up
// to ks parts as find a CU each: their parts' z lie in planes of their own that the output's transform adds up, so no part
// waits for another (see xp_parts for figures). Numbers 8 i + x are for XCD x, in runs of neighbouring tiles (the
// weight rows of one unit).
struct XpTiles {
  const XpProduct &a;
  const int tm, lane;
  int32_t lo, have;                                  // rows of expert `lane`: begin, number
  uint32_t whole, rest, lead, first, parts, blocks, all;

  __device__ __forceinline__ void rows_of(int x, int32_t &l, int32_t &n) const {
    l = x < a.count ? bounded(a.offsets[x], a.rows) : 0;
    const int32_t hi = x < a.count ? bounded(a.offsets[x + 1], a.rows) : 0;
    n = hi > l ? hi - l : 0;
  }
  __device__ __forceinline__ XpTiles(const XpProduct &product, int rows) : a(product), tm(rows), lane(threadIdx.x & 63) {
    whole = rest = 0;
    rows_of(lane, lo, have);
    for (int c = 0; c < a.count; c += 64) {
      int32_t l = lo, n = have;
      if (c) rows_of(c + lane, l, n);
      whole += (uint32_t)__builtin_amdgcn_readlane(wave_scan<false>(n / tm), 63);
      rest += __popcll(__ballot(n % tm != 0));
    }
    lead = whole + rest;                             // units that are not split
    parts = 1;
    const uint32_t tail = (lead * a.n_groups % kCus + a.n_groups - 1) / a.n_groups;      // those of the last round
    while (2 * parts <= (uint32_t)a.ks && 2 * parts * tail * a.n_groups <= kCus) parts *= 2;
    if (parts > 1) lead -= tail;
    first = lead * a.n_groups, blocks = (first + 7) / 8 * 8;
    all = blocks + ((whole + rest - lead) * a.n_groups * parts + 7) / 8 * 8;
  }
  // tile b < all; false where the runs leave a gap
  __device__ __forceinline__ bool find(uint32_t b, XpTile &tile) const {
    auto spread = [](uint32_t i, uint32_t n) {       // i-th number -> tile, in runs of an XCD; n: none
      const uint32_t run = (n + 7) / 8, t = (i % 8) * run + i / 8;
      return i / 8 < run && t < n ? t : n;
    };
    tile.part = 0, tile.parts = 1, tile.zs = 0;
    uint32_t u;
    if (b < blocks) {
      const uint32_t t = spread(b, first);
      if (t >= first) return false;
      u = t / a.n_groups, tile.group = t % a.n_groups;
    } else {
      const uint32_t n = (whole + rest - lead) * a.n_groups * parts, t = spread(b - blocks, n);
      if (t >= n) return false;
      u = t / (a.n_groups * parts);
      const uint32_t in = t - u * a.n_groups * parts;
      tile.zs = (int32_t)(u * parts) * tm;
      u += lead;
      tile.part = (int)(in / a.n_groups), tile.parts = (int)parts, tile.group = in % a.n_groups;
    }
    const bool is_rest = u >= whole;
    if (is_rest) u -= whole;
    uint32_t before = 0;
    for (int c = 0; c < a.count; c += 64) {
      int32_t l = lo, n = have;
      if (c) rows_of(c + lane, l, n);
      const uint32_t mine = is_rest ? (n % tm != 0 ? 1u : 0u) : (uint32_t)(n / tm), up = (uint32_t)wave_scan<false>((int)mine);
      const uint32_t at_first = before + up - mine;
      const unsigned long long hit = __ballot(mine > 0 && at_first <= u && u < at_first + mine);
      if (hit) {
        const int at = __ffsll((long long)hit) - 1;
        tile.e = c + at;
        const int32_t begin = __builtin_amdgcn_readlane(l, at), end = begin + __builtin_amdgcn_readlane(n, at);
        tile.row0 = is_rest ? begin + (end - begin) / tm * tm
                            : begin + (int32_t)(u - (uint32_t)__builtin_amdgcn_readlane((int)at_first, at)) * tm;
        tile.row1 = end - tile.row0 < tm ? end : tile.row0 + tm;
        if (!a.zs_own) tile.zs = tile.row0;
        return true;
      }
      before += (uint32_t)__builtin_amdgcn_readlane((int)up, 63);
    }
    return false;
  }
};

// Tiles of so few rows read x~ from memory straight into operands, which takes that load off the LDS unit and costs the vector
// memory path 2 lines a row and load. Products through LDS and so: 16 experts of 4096 x 4096 with 4 rows each, at 4 bits 60.5 and
// 54.0 us, at 3 bits 50.7 and 47.7; 8 of them with one row at 4 bits 33.4 and 30.4; 64 of 1024 x 2048 at 2 bits with 1, 3, 8
// and 24 rows 22.8, 22.5, 22.2 and 22.3, and 21.4, 22.4, 24.4 and 34; parts of 4 steps (4 of 1024 x 1024, 4 rows) 8.7 and 9.2.
constexpr int kDirectRows = 4;
constexpr int kGemmThreads = 512, kGemmLda = kGemmK + 8;
// rows of x~ in LDS, of which there are two tiles: 256 of bf16 x~, 64 of each part of float32 x~
constexpr int gemm_rows(bool f32) { return f32 ? 192 : 256; }
constexpr size_t gemm_lds(size_t tables, bool f32) { return tables + 2 * sizeof(uint16_t) * gemm_rows(f32) * kGemmLda; }

// One tile's loop over k and its end, for 32 MB rows or fewer (row0 .. row1 - 1) and P parts of x~.
//
// A wave owns 32 weight rows for all rows of the tile: MFMA 32x32x16 with x~ from LDS (double-buffered, one
// barrier a step) and its weights rebuilt straight into the other operand a step ahead,
// so each weight is rebuilt once a workgroup. The step's MFMAs come in runs; the walk of the
// next step's indices (records, halves, combination) and the tile's loads and writes are spread over them.
// A step is 64 inputs, or 128 where the tile has few rows: lane half p then has the groups 8 p .. 8 p + 7 of 8 inputs, 16 bytes
// of indices in one load. Few rows are bound by the LDS unit: of 226 passes a wave and step at 2 bits 162 are the lookups (random banks) and
// 64 the operands of x~ (64 experts of 1024 x 2048, 24 rows: 22.4 us, in steps of 64 23.7). What did not help there: indices asked for four
// steps ahead, records looked up a step ahead (24.7), lanes of rows that are not there masked out of the reads (24.2), 16 waves.
// DIRECT: x~ of the few rows from memory straight into operands, asked for a step ahead; no tiles, no barrier.
template <int BPW, bool G4, int MB, int P, bool DIRECT = false>
__device__ __forceinline__ void gemm_tile(const XpProduct &a, uint8_t *lds, const XpTile &tile, int64_t n0) {
  const int tid = threadIdx.x;
  const int32_t row0 = tile.row0, row1 = tile.row1;
  const int64_t e = tile.e;
  constexpr bool F32 = P == 3;
  constexpr int TPH = MB < 4 ? MB : 4, HB = MB / TPH;          // MFMA tiles of a run, runs of one of the 4 k-steps
  constexpr int KS = MB * P <= 3 ? 2 : 1;                      // 64s of inputs in a step
  constexpr int RP = 32 * MB;                                  // rows of a part in LDS
  constexpr int PIECES = RP * KS / 64, LDA = KS * kGemmK + 8;  // loads of 16 bytes a thread, a part; a row in LDS
  uint16_t *As0 = reinterpret_cast<uint16_t *>(lds + lds_table_bytes<BPW>());
  uint16_t *As1 = As0 + gemm_rows(F32) * kGemmLda;
  const int lane = tid & 63, c = lane & 31, p = lane >> 5;
  const int64_t G = a.k / 8, steps = a.kp / kGemmK;
  const int64_t begin = part_begin(steps, tile.part, tile.parts) / KS;
  const int64_t S = part_begin(steps, tile.part + 1, tile.parts) / KS - begin;  // steps of this part
  const int64_t left = a.n - n0, rows_w = left < 0 ? 0 : left < 32 ? left : 32, wrow = e * a.n + (rows_w ? n0 : 0);
  __amdgpu_buffer_rsrc_t xa[P];
#pragma unroll
  for (int q = 0; q < P; ++q)
    xa[q] = __builtin_amdgcn_make_buffer_rsrc((void *)(a.xt + ((int64_t)q * a.rows + row0) * a.kp), 0,
                                              (int)((row1 - row0) * a.kp * 2), 0x00020000);
  const __amdgpu_buffer_rsrc_t r1 =
      __builtin_amdgcn_make_buffer_rsrc((void *)(a.idx1 + wrow * G), 0, (int)(rows_w * G * 2), 0x00020000);
  const __amdgpu_buffer_rsrc_t r2 = __builtin_amdgcn_make_buffer_rsrc(
      BPW == 2 ? (void *)a.idx1 : (void *)(reinterpret_cast<const uint8_t *>(a.idx2) + wrow * G * (BPW == 4 ? 2 : 1)), 0,
      (int)(BPW == 2 ? 0 : rows_w * G * (BPW == 4 ? 2 : 1)), 0x00020000);
  const int row_t = tid / (8 * KS), chunk_t = tid % (8 * KS);
  const uint32_t va = (uint32_t)(row_t * a.kp * 2 + 16 * chunk_t);
  const uint32_t vi = (uint32_t)(c * G + 4 * KS * p);          // this lane's first index of step 0
  const int sa = (int)(64 / KS * a.kp * 2);
  auto load_a = [&](int64_t s, uint4 (&ra)[P * PIECES]) {
#pragma unroll
    for (int q = 0; q < P; ++q)
#pragma unroll
      for (int u = 0; u < PIECES; ++u)
        ra[q * PIECES + u] = __builtin_bit_cast(
            uint4, __builtin_amdgcn_raw_buffer_load_b128(xa[q], va, (int)(2 * KS * kGemmK * (begin + s)) + u * sa, 0));
  };
  auto store_a = [&](uint16_t *As, const uint4 (&ra)[P * PIECES]) {
#pragma unroll
    for (int i = 0; i < P * PIECES; ++i)
      *reinterpret_cast<uint4 *>(As + (row_t + 64 / KS * i) * LDA + 8 * chunk_t) = ra[i];
  };
  // indices of step s as stored, 4 KS of them; those past a row's end meet zeros of x~
  struct Indices { uint2 i1[KS], i2[KS]; };
  auto load_idx = [&](int64_t step, Indices &x) {
    const int at = (int)(8 * KS * (begin + step));             // in indices
    if constexpr (G4 && KS == 1) {
      x.i1[0] = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(r1, 2 * vi, 2 * at, 0));
      if constexpr (BPW == 3) x.i2[0].x = __builtin_amdgcn_raw_buffer_load_b32(r2, vi, at, 0);
      if constexpr (BPW == 4) x.i2[0] = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(r2, 2 * vi, 2 * at, 0));
    } else if constexpr (G4) {
      const uint4 w = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r1, 2 * vi, 2 * at, 0));
      x.i1[0] = make_uint2(w.x, w.y), x.i1[KS - 1] = make_uint2(w.z, w.w);
      if constexpr (BPW == 3) {
        const uint2 v = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(r2, vi, at, 0));
        x.i2[0].x = v.x, x.i2[KS - 1].x = v.y;
      }
      if constexpr (BPW == 4) {
        const uint4 v = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r2, 2 * vi, 2 * at, 0));
        x.i2[0] = make_uint2(v.x, v.y), x.i2[KS - 1] = make_uint2(v.z, v.w);
      }
    } else {
      // Rows begin at any multiple of 2 bytes (1): whole words from the one that a lane's first index lies in, shifted into place. (A
      // wave's rows begin at multiples of 16 and 8 bytes and end there, so the words are the rows' own.)
      auto words = [&](const __amdgpu_buffer_rsrc_t &r, uint32_t byte, int step_bytes, uint32_t (&w)[2 * KS + 1]) {
        const uint32_t from = byte & ~3u;
        if constexpr (KS == 1) {
          const uint2 x = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(r, from, step_bytes, 0));
          w[0] = x.x, w[1] = x.y;
        } else {
          const uint4 x = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, from, step_bytes, 0));
          w[0] = x.x, w[1] = x.y, w[2] = x.z, w[2 * KS - 1] = x.w;
        }
        w[2 * KS] = __builtin_amdgcn_raw_buffer_load_b32(r, from, step_bytes + 8 * KS, 0);
      };
      auto pairs = [&](const __amdgpu_buffer_rsrc_t &r, uint2 (&to)[KS]) {
        uint32_t w[2 * KS + 1];
        words(r, 2 * vi, 2 * at, w);
        const uint32_t shift = 16 * (vi & 1);
#pragma unroll
        for (int h = 0; h < KS; ++h)
          to[h] = make_uint2(__builtin_amdgcn_alignbit(w[2 * h + 1], w[2 * h], shift), __builtin_amdgcn_alignbit(w[2 * h + 2], w[2 * h + 1], shift));
      };
      pairs(r1, x.i1);
      if constexpr (BPW == 4) pairs(r2, x.i2);
      if constexpr (BPW == 3) {
        const uint32_t from = vi & ~3u, shift = 8 * (vi & 3);
        const uint2 w = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(r2, from, at, 0));
        x.i2[0].x = __builtin_amdgcn_alignbit(w.y, w.x, shift);
        if constexpr (KS == 2)
          x.i2[KS - 1].x = __builtin_amdgcn_alignbit(__builtin_amdgcn_raw_buffer_load_b32(r2, from, at + 8, 0), w.y, shift);
      }
    }
  };
  auto split = [&](const Indices &x, uint32_t (&q1)[8], uint32_t (&q2)[8]) {
#pragma unroll
    for (int h = 0; h < KS; ++h) {
      uint32_t p1[8], p2[8];
      g8_split<BPW>(x.i1[h], BPW == 2 ? make_uint2(0u, 0u) : x.i2[h], p1, p2);
#pragma unroll
      for (int u = 0; u < 4; ++u) q1[4 * h + u] = p1[u], q2[4 * h + u] = p2[u];
    }
  };
  auto load_x = [&](int64_t s, uint4 (&x)[8]) {
#pragma unroll
    for (int u = 0; u < 8; ++u)
      x[u] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(xa[0], (uint32_t)(c * a.kp * 2 + 128 * p),
                                                                             (int)(256 * (begin + s)) + 16 * u, 0));
  };
  auto upto = [&](int64_t s) { return s < S ? s : S - 1; };
  uint4 ra[P * PIECES], X0[8], X1[8];
  if constexpr (DIRECT) load_x(0, X0);
  else load_a(0, ra);
  float row_sum = 0.0f;                                        // thread t: of row row0 + t
  if constexpr (!F32 && BPW > 2)
    if (tid < 256 && tid < row1 - row0) {
      const float *sums = a.rowsum + row0 + tid;
      if (tile.parts == 1) row_sum = sums[0];
      else                                                     // (there are ks sums, some for each part)
        for (int i = a.ks / tile.parts, at = 1 + tile.part * i; i > 0; --i, ++at) row_sum += sums[at * (int64_t)a.rows];
    }
  Indices now, next;
  load_idx(0, now);
  tables_landed();                                             // and the first tile and indices
  load_idx(upto(1), next);
  if constexpr (!DIRECT) {
    store_a(As0, ra);
    load_a(upto(1), ra);
  }
  __syncthreads();                                             // of all waves
  f32x16 acc[MB];
#pragma unroll
  for (int t = 0; t < MB; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[t][i] = 0.f;
  uint4 B0[8], B1[8];                                          // groups u = 0 .. 4 KS - 1 used
  auto plain = [](uint4 w) { return F32 && BPW > 2 ? unbiased(w) : w; };
  {
    uint32_t q1[8], q2[8];
    split(now, q1, q2);
#pragma unroll
    for (int u = 0; u < 4 * KS; ++u) B0[u] = plain(decode_ip<BPW>(q1[u], q2[u]));
  }
  uint4 H0[P * TPH], H1[P * TPH];                              // operands of even and odd runs
  auto read_a = [&](const uint16_t *As, int run, uint4 (&h)[P * TPH]) {
    const int u = run / HB, t0 = TPH * (run % HB);
#pragma unroll
    for (int q = 0; q < P; ++q)
#pragma unroll
      for (int t = 0; t < TPH; ++t)
        h[q * TPH + t] = *reinterpret_cast<const uint4 *>(As + (q * RP + 32 * (t0 + t) + c) * LDA + 32 * KS * p + 8 * u);
  };
  if constexpr (!DIRECT) read_a(As0, 0, H0);
  auto kstep = [&](int64_t s, const uint4 (&bc)[8], uint4 (&bn)[8]) {
    const uint16_t *Acur = (s & 1) ? As1 : As0;
    uint16_t *Anext = (s & 1) ? As0 : As1;
    uint32_t q1[8], q2[8];
    split(next, q1, q2);                                       // of step s + 1
    load_idx(upto(s + 2), next);
    auto run = [&](int h, const uint4 (&av)[P * TPH], uint4 (&an)[P * TPH]) {
      if (h + 1 < 4 * KS * HB) read_a(Acur, h + 1, an);
      else read_a(Anext, 0, an);
      const int u = h / HB, t0 = TPH * (h % HB);
#pragma unroll
      for (int q = 0; q < P; ++q)
#pragma unroll
        for (int t = 0; t < TPH; ++t)
          acc[t0 + t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, av[q * TPH + t]),
                                                                __builtin_bit_cast(bf16x8, bc[u]), acc[t0 + t], 0, 0, 0);
    };
    constexpr int NW = BPW == 4 ? 2 : 1;                       // table walks a group
    Dec8<BPW, true> D;
    D.template p1<0, 4 * KS>(q1, q2);
    if constexpr (HB == 2) {                                   // the eight runs and their mix as in gemm8_bf16
      run(0, H0, H1);
      gm_interleave<4, 3, (4 * NW + (BPW == 3 ? 4 : 0) + 4 + 3) / 4>();
      __builtin_amdgcn_sched_barrier(0);
      D.template p2<0, 2>(q1, q2);
      run(1, H1, H0);
      gm_interleave<4, (14 * NW + 3) / 4, (4 * NW + 4 + 3) / 4>();
      __builtin_amdgcn_sched_barrier(0);
      D.template p2<2, 4>(q1, q2);
      run(2, H0, H1);
      gm_interleave<4, (14 * NW + 3) / 4, (4 * NW + 4 + 3) / 4>();
      __builtin_amdgcn_sched_barrier(0);
      D.template p3<0, 2>(bn);
      run(3, H1, H0);
      gm_interleave<4, 2, 1>();
      __builtin_amdgcn_sched_barrier(0);
      D.template p3<2, 4>(bn);
      store_a(Anext, ra);
      run(4, H0, H1);
      gm_interleave<4, 2, 1, 1>();
      __builtin_amdgcn_sched_barrier(0);
      load_a(upto(s + 2), ra);
      run(5, H1, H0);
      gm_interleave<4, 0, 1, 0, 1>();
      __builtin_amdgcn_sched_barrier(0);
      run(6, H0, H1);
      __builtin_amdgcn_sched_barrier(0);
      __syncthreads();
      run(7, H1, H0);
      __builtin_amdgcn_sched_barrier(0);
    } else if constexpr (KS == 2) {
      run(0, H0, H1);
      run(1, H1, H0);
      __builtin_amdgcn_sched_barrier(0);
      D.template p2<0, 4>(q1, q2);
      run(2, H0, H1);
      D.template p2<4, 8>(q1, q2);
      run(3, H1, H0);
      __builtin_amdgcn_sched_barrier(0);
      store_a(Anext, ra);
      load_a(upto(s + 2), ra);
      run(4, H0, H1);
      run(5, H1, H0);
      D.template p3<0, 8>(bn);
#pragma unroll
      for (int u = 0; u < 8; ++u) bn[u] = plain(bn[u]);
      run(6, H0, H1);
      __syncthreads();
      run(7, H1, H0);
    } else {
      run(0, H0, H1);
      __builtin_amdgcn_sched_barrier(0);
      D.template p2<0, 4>(q1, q2);
      run(1, H1, H0);
      __builtin_amdgcn_sched_barrier(0);
      store_a(Anext, ra);
      load_a(upto(s + 2), ra);
      run(2, H0, H1);
      D.template p3<0, 4>(bn);
#pragma unroll
      for (int u = 0; u < 4; ++u) bn[u] = plain(bn[u]);
      __syncthreads();
      run(3, H1, H0);
    }
  };
  auto dstep = [&](int64_t s, const uint4 (&bc)[8], uint4 (&bn)[8], const uint4 (&xc)[8], uint4 (&xn)[8]) {
    uint32_t q1[8], q2[8];
    split(next, q1, q2);                                       // of step s + 1
    load_idx(upto(s + 2), next);
    load_x(upto(s + 1), xn);
    auto mfma = [&](int u) {
      acc[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, xc[u]), __builtin_bit_cast(bf16x8, bc[u]), acc[0],
                                                       0, 0, 0);
    };
    Dec8<BPW, true> D;
    D.template p1<0, 8>(q1, q2);
    mfma(0);
    mfma(1);
    __builtin_amdgcn_sched_barrier(0);
    D.template p2<0, 4>(q1, q2);
    mfma(2);
    D.template p2<4, 8>(q1, q2);
    mfma(3);
    __builtin_amdgcn_sched_barrier(0);
    mfma(4);
    mfma(5);
    D.template p3<0, 8>(bn);
    mfma(6);
    mfma(7);
  };
  int64_t s = 0;
  for (; s + 1 < S; s += 2) {
    if constexpr (DIRECT) {
      dstep(s, B0, B1, X0, X1);
      dstep(s + 1, B1, B0, X1, X0);
    } else {
      kstep(s, B0, B1);
      kstep(s + 1, B1, B0);
    }
  }
  if (s < S) {
    if constexpr (DIRECT) dstep(s, B0, B1, X0, X1);
    else kstep(s, B0, B1);
  }
  if (n0 == 0 && tile.part == 0 && lane < 32)
#pragma unroll
    for (int t = 0; t < MB; ++t)
      if (row0 + 32 * t + lane < row1)
        a.row_parts[row0 + 32 * t + lane] = tile.parts == 1 ? 1 : tile.parts | (tile.zs + 32 * t + lane) << 4;
  // Lane (c, p) holds rows 8 (i >> 2) + 4 p + (i & 3) of weight row n0 + c. z goes out through the wave's own piece of LDS, 32 rows
  // at a time, so that a lane stores 16 bytes of a row: element by element, with a load of the row's sum for each,
  // the end of a tile took 15 of 141 us.
  constexpr bool BIAS = !F32 && BPW > 2;
  const uint32_t sums = lds_table_bytes<BPW>();
  __syncthreads();                                             // the tiles of x~ are done with
  if constexpr (BIAS) {
    if (tid < 256) lds_stf(sums + 4 * tid, row_sum);
    __syncthreads();
  }
  typedef __attribute__((address_space(3))) _Float16 lds_f16_w;
  auto leave = [&](auto wide) {
    constexpr bool W = decltype(wide)::value;                  // float32, or float16
    constexpr int ES = W ? 4 : 2, SB = 32 * ES + 16, CPR = 32 * ES / 16;        // bytes of an element and of a row, chunks a row
    const uint32_t mine = sums + 1024 + (uint32_t)__builtin_amdgcn_readfirstlane(tid >> 6) * 32 * SB;
    uint8_t *to = reinterpret_cast<uint8_t *>(tile.parts == 1 ? a.z : a.zs) +
                  (int64_t)(tile.parts == 1 ? row0 : tile.zs + tile.part * a.zs_step) * a.n * ES;
#pragma unroll
    for (int t = 0; t < MB; ++t) {
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint4 s = make_uint4(0, 0, 0, 0);
        if constexpr (BIAS) s = lds128(sums + 4 * (32 * t + 8 * g + 4 * p));
        const float bias[4] = {__uint_as_float(s.x), __uint_as_float(s.y), __uint_as_float(s.z), __uint_as_float(s.w)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float v = BIAS ? fmaf(-Epi<BPW>::bias, bias[i], acc[t][4 * g + i]) : acc[t][4 * g + i];
          const uint32_t at = mine + (8 * g + 4 * p + i) * SB + c * ES;
          if constexpr (W) lds_stf(at, v);
          else *reinterpret_cast<lds_f16_w *>((uintptr_t)at) = (_Float16)v;
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // other lanes of the wave read it
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < 32 * CPR / 64; ++i) {
        const int chunk = 64 * i + lane, rl = chunk / CPR, pc = chunk % CPR;
        const uint4 v = lds128(mine + rl * SB + pc * 16);
        const int32_t r = 32 * t + rl;
        const int64_t col = n0 + pc * (16 / ES);
        if (row0 + r < row1 && col < a.n)                      // (n is a multiple of 8)
          *reinterpret_cast<uint4 *>(to + (r * a.n + col) * ES) = v;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
  };
  static_assert(1024 + 8 * 32 * (32 * 4 + 16) <= 2 * sizeof(uint16_t) * gemm_rows(F32) * kGemmLda, "a wave's piece");
  if constexpr (F32) {
    leave(std::true_type());
  } else {
    if (a.z16 && tile.parts == 1) leave(std::false_type());
    else leave(std::true_type());
  }
}

// A workgroup a tile, one a CU at a time. (Workgroups that stay and take tile after tile from queues of their XCDs, with one
// copy of the tables each: level, 282 against 273 us for 512 tiles, and 2 us more where every CU has one tile.) The copy of the tables is
// under way while the tile is looked for, except in the last workgroups of the launch, which may have none.
template <int BPW, bool G4, bool F32>
__global__ void __launch_bounds__(kGemmThreads, 1) xp_gemm_k(XpProduct a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  if (blockIdx.x < a.likely) load_tables<BPW, kGemmThreads>(lds, a.cb);
  const XpTiles tiles(a, F32 ? 64 : 256);
  XpTile tile;
  if (blockIdx.x >= tiles.all || !tiles.find(blockIdx.x, tile)) {
    tables_landed();                                 // LDS loads in flight must not outlive their workgroup
    return;
  }
  if (blockIdx.x >= a.likely) load_tables<BPW, kGemmThreads>(lds, a.cb);
  const int64_t n0 = (int64_t)tile.group * 256 + 32 * __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t rows = tile.row1 - tile.row0;
  if constexpr (F32) {
    if (rows > 32) gemm_tile<BPW, G4, 2, 3>(a, lds, tile, n0);
    else gemm_tile<BPW, G4, 1, 3>(a, lds, tile, n0);
  } else {
    if (rows > 128) gemm_tile<BPW, G4, 8, 1>(a, lds, tile, n0);
    else if (rows > 64) gemm_tile<BPW, G4, 4, 1>(a, lds, tile, n0);
    else if (rows > 32) gemm_tile<BPW, G4, 2, 1>(a, lds, tile, n0);
    else if (rows > kDirectRows) gemm_tile<BPW, G4, 1, 1>(a, lds, tile, n0);
    else gemm_tile<BPW, G4, 1, 1, true>(a, lds, tile, n0);
  }
}

// ------------------------------------------------------------ launches and argument checks

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

bool aligned_to(const void *p, int a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int64_t up128(int64_t v) { return (v + 127) & ~int64_t(127); }
int64_t up256(int64_t v) { return (v + 255) & ~int64_t(255); }

int log_block(int64_t len) {
  int lb = 0;
  while (!(len >> lb & 1)) ++lb;
  return lb;
}

template <int E, int NW, bool OUT, bool F32, bool Z16>
int launch_transform_k(const XpRows &a, int64_t groups, hipStream_t st) {
  constexpr size_t shm = sizeof(float) * (64 * NW * E + 64);
  if constexpr (OUT) {
    const int rc = allow_lds<xp_out_k<E, NW, F32, Z16>>(shm);
    if (rc) return rc;
    hipLaunchKernelGGL((xp_out_k<E, NW, F32, Z16>), dim3((unsigned)groups), dim3(64 * NW), shm, st, a);
    return hip_status(hipGetLastError(), "xp_out_k");
  } else {
    const int rc = allow_lds<xp_in_k<E, NW, F32>>(shm);
    if (rc) return rc;
    hipLaunchKernelGGL((xp_in_k<E, NW, F32>), dim3((unsigned)groups), dim3(64 * NW), shm, st, a);
    return hip_status(hipGetLastError(), "xp_in_k");
  }
}

template <int NW, bool OUT, bool F32, bool Z16>
int launch_blocks_k(const XpRows &a, int64_t most, hipStream_t st) {
  const int waves = (int)((OUT ? a.n : a.k) / 1024);
  // the output's sets of waves: as many as choices and a workgroup take, where there are no more tokens than CUs (32 tokens of 8
  // choices, rows of 2048: 5.3 us, by one set 8.7; one token of two, rows of 4096: 7.1 and 10.3)
  int sets = 1;
  if (OUT && most <= kCus)
    while (2 * sets * waves <= kRowWaves && sets < a.top) sets *= 2;
  const size_t shm = NW > 1 || sets > 1 ? (size_t)waves * sets * 4096 : 0;
  // no more workgroups than run at once, by the registers of the kernels (waves a SIMD): more would leave some CUs a second
  // run of rows. NW = 4, 2048 and 8192 rows: in 14.5 and 44 us, with 6 waves a SIMD 16.7 and 49; out 11.1 and 34.5, and 12.7 and 36
  constexpr int resident = 4 * (OUT ? 4 : NW == 1 ? 8 : NW == 2 ? 6 : 5);
  const int per = resident / (waves * sets);
  const int64_t once = (int64_t)kCus * (per > 1 ? per : 1), groups = most < once ? most : once;
  if constexpr (OUT) {
    const int rc = allow_lds<xp_out_blk_k<NW, F32, Z16>>(shm + 2048);          // (and the static part)
    if (rc) return rc;
    hipLaunchKernelGGL((xp_out_blk_k<NW, F32, Z16>), dim3((unsigned)groups), dim3(64 * waves * sets), shm, st, a);
    return hip_status(hipGetLastError(), "xp_out_blk_k");
  } else {
    const int rc = allow_lds<xp_in_blk_k<NW, F32>>(shm + 2048);
    if (rc) return rc;
    hipLaunchKernelGGL((xp_in_blk_k<NW, F32>), dim3((unsigned)groups), dim3(64 * waves), shm, st, a);
    return hip_status(hipGetLastError(), "xp_in_blk_k");
  }
}

template <bool OUT, bool F32, bool Z16>
int launch_blocks(const XpRows &a, int64_t most, hipStream_t st) {
  switch (OUT ? a.log_n : a.log_k) {
    case 10: return launch_blocks_k<1, OUT, F32, Z16>(a, most, st);
    case 11: return launch_blocks_k<2, OUT, F32, Z16>(a, most, st);
    case 12: return launch_blocks_k<4, OUT, F32, Z16>(a, most, st);
    case 13: return launch_blocks_k<8, OUT, F32, Z16>(a, most, st);
    default: return launch_blocks_k<16, OUT, F32, Z16>(a, most, st);
  }
}

// 8 elements a thread, as many waves as the row (or 8192 of it at a time) takes; whole blocks of 16384 need 16 a thread.
template <bool OUT, bool F32, bool Z16 = false>
int launch_transform(const XpRows &a, int64_t groups, hipStream_t st) {
  const int64_t len = OUT ? a.n : a.k;
  if ((OUT ? a.log_n : a.log_k) >= 10 && len <= 1024 * kRowWaves) return launch_blocks<OUT, F32, Z16>(a, groups, st);
  if ((OUT ? a.log_n : a.log_k) == 14) return launch_transform_k<16, 16, OUT, F32, Z16>(a, groups, st);
  if (len <= 512) return launch_transform_k<8, 1, OUT, F32, Z16>(a, groups, st);
  if (len <= 1024) return launch_transform_k<8, 2, OUT, F32, Z16>(a, groups, st);
  if (len <= 2048) return launch_transform_k<8, 4, OUT, F32, Z16>(a, groups, st);
  if (len <= 4096) return launch_transform_k<8, 8, OUT, F32, Z16>(a, groups, st);
  return launch_transform_k<8, 16, OUT, F32, Z16>(a, groups, st);
}

template <int BPW, bool G4, bool F32>
int launch_gemm(XpProduct a, hipStream_t st) {
  constexpr int TM = F32 ? 64 : 256;
  a.n_groups = (uint32_t)((a.n + 255) / 256);
  // no more tiles than this, whatever the offsets are, parts of no more than fill the card, and up to 7 numbers to fill the XCDs'
  // runs of each kind
  const int64_t tiles = (a.rows / TM + (a.count < a.rows ? a.count : a.rows)) * a.n_groups, more = tiles * (a.ks - 1);
  const int64_t most = tiles + (more < kCus ? more : kCus) + 16;
  constexpr size_t shm = gemm_lds(lds_table_bytes<BPW>(), F32);
  static_assert(shm <= 160 * 1024, "LDS of a CU");
  const int rc = allow_lds<xp_gemm_k<BPW, G4, F32>>(shm);
  if (rc) return rc;
  if (most > 0xFFFFFFFFll / kGemmThreads) return GLQ_ERR_UNSUPPORTED;
  // (half of the experts with a remainder; where units are split depends on the card's share of the last round)
  a.likely = (uint32_t)((a.rows / TM + (a.count < a.rows ? a.count : a.rows) / 2) * a.n_groups);
  hipLaunchKernelGGL((xp_gemm_k<BPW, G4, F32>), dim3((unsigned)most), dim3(kGemmThreads), shm, st, a);
  return hip_status(hipGetLastError(), "xp_gemm_k");
}

template <int BPW>
int launch_product(const XpProduct &a, bool f32, hipStream_t st) {
  // rows of indices begin at multiples of 4 of them, or anywhere (5 experts of 1000 x 328 at 4 bits, 14 rows: 10.2 us by shifted words, 15.0
  // index by index, 9.5 for k = 320)
  if (a.k % 32 == 0) return f32 ? launch_gemm<BPW, true, true>(a, st) : launch_gemm<BPW, true, false>(a, st);
  return f32 ? launch_gemm<BPW, false, true>(a, st) : launch_gemm<BPW, false, false>(a, st);
}

int check_experts(const glq_experts *E) {
  if (!E || E->count < 1 || E->n < 1 || E->n % 8 || E->k < 8 || E->k % 8) return GLQ_ERR_ARG;
  if (E->bpw != 2 && E->bpw != 3 && E->bpw != 4) return GLQ_ERR_ARG;
  if ((E->bpw == 3 && E->resid_shift != 1) || (E->bpw == 4 && E->resid_shift != 2)) return GLQ_ERR_ARG;
  if (!E->scale || !E->idx1 || (E->bpw > 2 && !E->idx2) || !E->sign_k || !E->sign_n || !E->cb) return GLQ_ERR_ARG;
  if (!aligned_to(E->scale, 4) || !aligned_to(E->row_scale, 4) || !aligned_to(E->idx1, 16) || !aligned_to(E->idx2, 16) ||
      !aligned_to(E->sign_k, 8) || !aligned_to(E->sign_n, 8) || !aligned_to(E->cb, 16))
    return GLQ_ERR_ARG;
  if (E->count > kMaxExperts || E->n > (1 << 21) || E->k > (1 << 21) || log_block(E->k) > 14 || log_block(E->n) > 14)
    return GLQ_ERR_UNSUPPORTED;
  return GLQ_OK;
}

// Most parts along k of the units that are split (XpTiles): two, four where bf16 rows are long, and four or
// eight as many as give each CU one for the most tiles there can be; none under 4 steps, which would not pay for the
// transforms' reading more sums. 2 of 8 experts of 4096 x 4096 at 4 bits, a row each, 32 tiles: product 14 us in 8 parts,
// 32 in 2. 8192 rows over 8 experts of that size at 3 bits, 576 tiles: the call 343 us with its last 4 units in 4 parts,
// 353 with 20 in 2; of 4096 x 1024 (16 steps) at 2 bits 133 and 126.
int xp_parts(int64_t count, int64_t n, int64_t k, int64_t rows, bool f32) {
  const int64_t steps = up128(k) / kGemmK, most = (rows / (f32 ? 64 : 256) + (count < rows ? count : rows)) * ((n + 255) / 256);
  if (steps > kSplitSteps || steps < 8) return 1;
  int ks = f32 || steps < 32 ? 2 : 4;
  while (ks < 8 && most * 2 * ks <= kCus && steps / (2 * ks) >= 4) ks *= 2;
  return ks;
}

// Rows of the parts' sums (zs) in tiles of tm rows: ks times the rows, or, where that is less, the tiles' own: no more than a
// tile a CU is split (XpTiles).
int64_t zs_rows(int64_t n, int64_t rows, int ks, int tm) {
  const int64_t own = (int64_t)tm * (kCus / ((n + 255) / 256));
  return ks == 1 ? 0 : rows * ks < own ? rows * ks : own;
}
// As many at least, for up to this many rows of either type.
int64_t zs_most(int64_t n, int64_t k, int64_t rows) {
  const int64_t steps = up128(k) / kGemmK;
  return steps > kSplitSteps || steps < 8 ? 0 : zs_rows(n, rows, 8, 256);
}

struct XpLayout { int64_t xt, rowsum, row_factor, row_expert, row_parts, z, zs, total; };
XpLayout xp_layout(const glq_experts *E, int64_t rows) {
  XpLayout w;
  w.xt = 0;
  w.rowsum = w.xt + up256(rows * up128(E->k) * 6);    // float32 rows: three parts of 2 bytes
  w.row_factor = w.rowsum + up256(rows * 4 * 9);        // whole, and eight parts at most
  w.row_expert = w.row_factor + up256(rows * 4);
  w.row_parts = w.row_expert + up256(rows * 4);
  w.z = w.row_parts + up256(rows * 4);
  w.zs = w.z + up256(rows * E->n * 4);
  w.total = w.zs + up256(zs_most(E->n, E->k, rows) * E->n * 4);
  return w;
}

int check_rows(const glq_experts *E, int64_t rows) {
  const int rc = check_experts(E);
  if (rc) return rc;
  if (rows < 0) return GLQ_ERR_ARG;
  if (rows > 0x7FFFFFFF / 512) return GLQ_ERR_UNSUPPORTED;
  return GLQ_OK;
}

}  // namespace
}  // namespace glq

using namespace glq;

extern "C" size_t glq_expert_linear_workspace(const glq_experts *E, int64_t rows) {
  if (check_rows(E, rows)) return 0;
  return (size_t)xp_layout(E, rows < 1 ? 1 : rows).total;
}

extern "C" int glq_expert_linear(const glq_experts *E, const glq_expert_rows *R, void *workspace, size_t ws_bytes,
                                 void *hip_stream) {
  if (!R) return GLQ_ERR_ARG;
  int rc = check_rows(E, R->rows);
  if (rc) return rc;
  if (!valid_dtype(R->x_dt) || !valid_dtype(R->y_dt) || R->x_rows < 0 || R->tokens < 0) return GLQ_ERR_ARG;
  const int64_t out = R->pos ? R->tokens : R->rows;
  if (out == 0) return GLQ_OK;
  if (R->pos && (R->top_k < 1 || !R->weights || !aligned_to(R->pos, 4) || !aligned_to(R->weights, 4))) return GLQ_ERR_ARG;
  if (!R->src && R->x_rows < R->rows) return GLQ_ERR_ARG;
  if (!R->y || !aligned_to(R->y, 16) || !R->offsets || !aligned_to(R->offsets, 4) || !aligned_to(R->src, 4)) return GLQ_ERR_ARG;
  if (R->x_rows > 0 && R->rows > 0 && (!R->x || !aligned_to(R->x, 16))) return GLQ_ERR_ARG;
  if (R->x_rows > (int64_t(1) << 31) || out > 0x7FFFFFFF / 512 || (R->pos && R->top_k > 1024)) return GLQ_ERR_UNSUPPORTED;
  if (!workspace || !aligned_to(workspace, 256) || ws_bytes < glq_expert_linear_workspace(E, R->rows)) return GLQ_ERR_WORKSPACE;
  uint8_t *ws = reinterpret_cast<uint8_t *>(workspace);
  const XpLayout l = xp_layout(E, R->rows);
  const bool f32 = R->x_dt == GLQ_F32;
  const int ks = xp_parts(E->count, E->n, E->k, R->rows, f32), tm = f32 ? 64 : 256;
  // z in float16 where both ends are bfloat16 and in float32 it would be more than the 32 MB that the L2s hold. In float16 and float32,
  // rows of 4096 through 8 experts of 4096 x 4096 at 2 bits: 1024 rows 98 and 100 us, 2048: 118 and 122, 4096: 182 and 190,
  // 8192: 320 and 332; 65,536 rows, 64 of 2048 x 1024: 432 and 518; 2048 rows, 8 of 1024 x 1024: 35 and 35
  const bool z16 = !f32 && R->y_dt == GLQ_BF16 && R->rows * E->n >= (int64_t(1) << 23);
  XpRows a = {};
  a.x = R->x, a.y = R->y, a.offsets = R->offsets, a.src = R->src, a.pos = R->pos, a.weights = R->weights;
  a.sign_k = E->sign_k, a.sign_n = E->sign_n, a.scale = E->scale, a.row_scale = E->row_scale;
  a.unit = E->bpw == 2 ? Epi<2>::mul : E->bpw == 3 ? Epi<3>::mul : Epi<4>::mul;
  a.xt = reinterpret_cast<uint16_t *>(ws + l.xt), a.rowsum = reinterpret_cast<float *>(ws + l.rowsum);
  a.row_factor = reinterpret_cast<float *>(ws + l.row_factor), a.row_expert = reinterpret_cast<int32_t *>(ws + l.row_expert);
  a.row_parts = reinterpret_cast<int32_t *>(ws + l.row_parts), a.z = ws + l.z, a.zs = reinterpret_cast<float *>(ws + l.zs);
  const bool zs_own = zs_rows(E->n, R->rows, ks, tm) < R->rows * ks;
  a.zs_step = zs_own ? tm : (int32_t)R->rows;
  a.k = E->k, a.kp = up128(E->k), a.n = E->n, a.x_rows = R->x_rows, a.out_rows = out;
  a.count = (int32_t)E->count, a.rows = (int32_t)R->rows, a.top = R->pos ? R->top_k : 1, a.ks = ks;
  a.log_k = log_block(E->k), a.log_n = log_block(E->n);
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  if (R->rows > 0) {
    rc = f32 ? launch_transform<false, true>(a, R->rows, st) : launch_transform<false, false>(a, R->rows, st);
    if (rc) return rc;
    const XpProduct p = {E->idx1, a.xt, E->idx2, reinterpret_cast<const uint8_t *>(E->cb), a.rowsum, a.offsets,
                         a.row_parts, ws + l.z, reinterpret_cast<float *>(ws + l.zs), E->n, E->k, a.kp, a.count, a.rows,
                         a.zs_step, zs_own, z16, 0, 0, ks};
    rc = E->bpw == 2 ? launch_product<2>(p, f32, st) : E->bpw == 3 ? launch_product<3>(p, f32, st) : launch_product<4>(p, f32, st);
    if (rc) return rc;
  }
  if (R->y_dt == GLQ_F32) return launch_transform<true, true>(a, out, st);
  return z16 ? launch_transform<true, false, true>(a, out, st) : launch_transform<true, false>(a, out, st);
}
