// glq_experts.hip -- compressed linears of experts on ragged groups of rows
// (gfx950), and their entry points of the C ABI.
//
// With the rows in the experts' order, row r of expert e: y_r = U_e^T (s_e W^_e) (V_e x_r),
// a layer as in glq_kernels.hip for each expert, all of them in three launches:
//   xp_in_k     x~_r = V_e x_r, rows gathered from their tokens
//   xp_rows_k   z_r = s_e W^_e x~_r, the weights rebuilt inside the product
//   xp_out_k    y_r = U_e^T z_r, or a token's weighted sum of them
// How many rows an expert has is known on the device only: launches are sized by
// the most there can be, and a workgroup without rows ends at once.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdio>

#include "glq.h"
#include "glq_cache.h"
#include "glq_decode.h"
#include "glq_fwht.h"

namespace glq {
namespace {

constexpr int kMaxExperts = 1024;

// ------------------------------------------------------------ rows and experts

__device__ __forceinline__ int32_t bounded(int32_t x, int32_t most) { return x < 0 ? 0 : x < most ? x : most; }

// Expert of row r (0 <= r < the last offset): the number of experts that end at r or before. Every wave for itself.
__device__ __forceinline__ int expert_of(const int32_t *offsets, int count, int32_t r) {
  int e = 0;
  for (int c = threadIdx.x & 63; c < count; c += 64) e += __popcll(__ballot(offsets[c + 1] <= r));
  e = __builtin_amdgcn_readfirstlane(e);
  return e < count ? e : count - 1;
}

// Unit u of the row groups, tm rows of one expert each (the last of an expert may be shorter):
// expert and rows [row0, row1), or false where there are fewer units. Every wave for itself.
__device__ __forceinline__ bool find_unit(const int32_t *offsets, int count, int32_t rows, uint32_t u, int tm, int &e,
                                          int32_t &row0, int32_t &row1) {
  const int lane = threadIdx.x & 63;
  uint32_t before = 0;
  for (int c = 0; c < count; c += 64) {
    const int x = c + lane;
    const int32_t lo = x < count ? bounded(offsets[x], rows) : 0, hi = x < count ? bounded(offsets[x + 1], rows) : 0;
    const uint32_t mine = hi > lo ? (uint32_t)((hi - lo - 1) / tm + 1) : 0u;
    uint32_t up = mine;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const uint32_t y = __shfl_up(up, s);
      if (lane >= s) up += y;
    }
    const uint32_t first = before + up - mine;
    const unsigned long long hit = __ballot(mine > 0 && first <= u && u < first + mine);
    if (hit) {
      const int at = __ffsll((long long)hit) - 1;
      e = c + at;
      row0 = __builtin_amdgcn_readlane(lo, at) + (int32_t)(u - (uint32_t)__builtin_amdgcn_readlane((int)first, at)) * tm;
      const int32_t end = __builtin_amdgcn_readlane(hi, at);
      row1 = end - row0 < tm ? end : row0 + tm;
      return true;
    }
    before += (uint32_t)__builtin_amdgcn_readlane((int)up, 63);
  }
  return false;
}

// ------------------------------------------------------------ row transforms

struct XpRows {
  const void *x;
  void *y;
  const int32_t *offsets, *src, *pos;
  const float *weights;
  const int8_t *sign_k, *sign_n;
  uint16_t *xt;                // [planes][rows][kp] bf16: x~, or three parts that add up to it; zeros from k on
  float *rowsum, *z;           // [rows] sums of x~ (bf16 path), [rows][n]
  int32_t *row_expert;         // [rows]
  int64_t k, kp, n, x_rows;    // kp: k up to a multiple of 64
  int32_t count, rows, top;
  int log_k, log_n;            // Hadamard blocks
};

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

// One workgroup a row. bf16: x~ rounded to bf16, what the matrix cores take, and the sum of the
// rounded values, which the biased operands at 3 and 4 bits need. float32: x~ as three bf16 parts,
// which hold all of its 24 bits.
template <int E, int NW, bool F32>
__global__ void __launch_bounds__(64 * NW) xp_in_k(XpRows a) {
  extern __shared__ __attribute__((aligned(16))) float buf[];       // 64 NW E + 64
  __shared__ float part[NW];
  const int tid = threadIdx.x;
  const int32_t r = blockIdx.x;
  if (r < bounded(a.offsets[0], a.rows) || r >= bounded(a.offsets[a.count], a.rows)) return;
  const int e = expert_of(a.offsets, a.count, r);
  if (tid == 0) a.row_expert[r] = e;
  const int64_t from = a.src ? a.src[r] : r;
  const bool in = from >= 0 && from < a.x_rows;
  const int8_t *signs = a.sign_k + (int64_t)e * a.k;
  const float inv = 1.0f / sqrtf((float)(1 << a.log_k));
  float sum = 0.0f;
  for (int64_t s0 = 0; s0 < a.kp; s0 += 64 * NW * E) {
    float v[E];
#pragma unroll
    for (int h = 0; h < E; h += 8) {
      const int64_t o = s0 + E * tid + h;
      float s[8];
      if (in && o < a.k) {
        load8<F32>(reinterpret_cast<const uint8_t *>(a.x) + (F32 ? 4 : 2) * (from * a.k + o), v + h);
        load_signs8(signs + o, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[h + i] *= s[i];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[h + i] = 0.0f;
      }
    }
    if (s0) __syncthreads();
    row_fwht<E, NW>(v, buf, a.log_k);
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
          else sum += lo + hi;
        }
        *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
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
  }
}

// One workgroup a row of y: a row's U^T z, or with `pos` the sum of a token's rows, each with its weight, in
// the order of its choices, in float32.
template <int E, int NW, bool F32>
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
      const float w = a.pos ? a.weights[row_y * a.top + j] * inv : inv;
      const int8_t *signs = a.sign_n + (int64_t)a.row_expert[r] * a.n;
      float v[E];
#pragma unroll
      for (int h = 0; h < E; h += 8) {
        const int64_t o = s0 + E * tid + h;
        if (o < a.n) {
          load8<true>(a.z + (int64_t)r * a.n + o, v + h);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[h + i] = 0.0f;
        }
      }
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

// ------------------------------------------------------------ the product

struct XpProduct {
  const uint16_t *idx1, *xt;
  const void *idx2;
  const uint8_t *cb;
  const float *scale, *row_scale, *rowsum;
  const int32_t *offsets;
  float *z;
  int64_t n, k, kp;
  int32_t count, rows;
  uint32_t n_groups;           // of 128 weight rows, or of 256
};

// biased operands (bf16 of 192 + u) to bf16 of u, exact
__device__ __forceinline__ uint4 unbiased(uint4 w) {
  auto two = [](uint32_t u) { return pack_high(bf16_lo(u) - kBiasValue, bf16_hi(u) - kBiasValue); };
  return make_uint4(two(w.x), two(w.y), two(w.z), two(w.w));
}

// Workgroup: 64 rows of an expert by 128 of its weight rows, a wave 16 of those. As in the small-batch product
// of a layer: a chunk is 32 groups of 8 inputs, lane (j, q) rebuilds groups 8 q .. 8 q + 7 of it for weight
// row j, and step s of the matrix products takes group 8 q + s.
template <int BPW, bool G8, bool F32>
__global__ void __launch_bounds__(512) xp_rows_k(XpProduct a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  constexpr int P = F32 ? 3 : 1;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, j = lane & 15, q = lane >> 4;
  int e;
  int32_t row0, row1;
  if (!find_unit(a.offsets, a.count, a.rows, blockIdx.x / a.n_groups, 64, e, row0, row1)) return;
  load_tables<BPW, 512>(lds, a.cb);
  tables_landed();
  __syncthreads();
  const int64_t n0 = (int64_t)(blockIdx.x % a.n_groups) * 128 + 16 * wave, G = a.k / 8;
  if (n0 >= a.n) return;
  const int tiles = (row1 - row0 + 15) / 16;
  const int64_t row = (int64_t)e * a.n + (n0 + j < a.n ? n0 + j : a.n - 1);
  f32x4 acc[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int64_t c = 0; 32 * c < G; ++c) {
    const int64_t g0 = 32 * c + 8 * q;
    const GvRaw raw = gv_load_raw<BPW, G8>(a.idx1, a.idx2, row, G, g0);
    uint32_t i1[8], i2[8];
    gv_unpack<BPW>(raw, i1, i2);
    Dec8<BPW> D;
    uint4 bv[8];
    D.run(i1, i2, bv);
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      if constexpr (F32 && BPW > 2) bv[s] = unbiased(bv[s]);
      if (g0 + s >= G) bv[s] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t >= tiles) break;
      const int32_t r = row0 + 16 * t + j < row1 ? row0 + 16 * t + j : row1 - 1;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const uint16_t *x = a.xt + ((int64_t)p * a.rows + r) * a.kp;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const uint4 av = *reinterpret_cast<const uint4 *>(x + 8 * (g0 + s < G ? g0 + s : G - 1));
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, av), __builtin_bit_cast(bf16x8, bv[s]),
                                                           acc[t], 0, 0, 0);
        }
      }
    }
  }
  if (n0 + j >= a.n) return;
  float post = a.scale[e] * Epi<BPW>::mul;
  if (a.row_scale) post *= a.row_scale[row];
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int32_t r = row0 + 16 * t + 4 * q + i;
      if (r >= row1) continue;
      const float bias = F32 || BPW == 2 ? 0.0f : Epi<BPW>::bias * a.rowsum[r];
      a.z[(int64_t)r * a.n + n0 + j] = post * (acc[t][i] - bias);
    }
}

// ------------------------------------------------------------ many rows: 256 by 256 tiles

typedef float f32x16 __attribute__((ext_vector_type(16)));

// Workgroup b's tile of 256 (TM) rows of an expert by 256 of its weight rows, or false. Whole
// groups of TM rows come before the experts' remainders, which are shorter, so those fill
// the end of the launch. Neighbouring tiles (the weight rows of one group of rows) run on one XCD:
// blocks go to the eight in turn.
__device__ __forceinline__ bool find_tile(const int32_t *offsets, int count, int32_t rows, uint32_t b, uint32_t n_groups, int tm,
                                          int &e, int32_t &row0, int32_t &row1, uint32_t &group) {
  const int lane = threadIdx.x & 63;
  uint32_t whole = 0, rest = 0;
  for (int c = 0; c < count; c += 64) {
    const int x = c + lane;
    const int32_t lo = x < count ? bounded(offsets[x], rows) : 0, hi = x < count ? bounded(offsets[x + 1], rows) : 0;
    const int32_t mine = hi > lo ? hi - lo : 0;
    uint32_t w = (uint32_t)(mine / tm);
#pragma unroll
    for (int s = 32; s; s >>= 1) w += __shfl_xor(w, s);
    whole += (uint32_t)__builtin_amdgcn_readfirstlane((int)w);
    rest += __popcll(__ballot(mine % tm != 0));
  }
  const uint32_t first = whole * n_groups, all = first + rest * n_groups;
  auto spread = [](uint32_t i, uint32_t n) {         // i-th block of n -> tile, in runs of an XCD; n: none
    const uint32_t run = (n + 7) / 8, t = (i % 8) * run + i / 8;
    return i / 8 < run && t < n ? t : n;
  };
  const uint32_t lead = (first + 7) / 8 * 8;         // blocks of the whole groups
  const bool is_rest = b >= lead;
  const uint32_t n = is_rest ? all - first : first, t = spread(is_rest ? b - lead : b, n);
  if (t >= n) return false;
  const uint32_t u = t / n_groups;
  group = t % n_groups;
  uint32_t before = 0;
  for (int c = 0; c < count; c += 64) {
    const int x = c + lane;
    const int32_t lo = x < count ? bounded(offsets[x], rows) : 0, hi = x < count ? bounded(offsets[x + 1], rows) : 0;
    const int32_t have = hi > lo ? hi - lo : 0;
    const uint32_t mine = is_rest ? (have % tm != 0 ? 1u : 0u) : (uint32_t)(have / tm);
    uint32_t up = mine;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const uint32_t y = __shfl_up(up, s);
      if (lane >= s) up += y;
    }
    const uint32_t at_first = before + up - mine;
    const unsigned long long hit = __ballot(mine > 0 && at_first <= u && u < at_first + mine);
    if (hit) {
      const int at = __ffsll((long long)hit) - 1;
      e = c + at;
      const int32_t begin = __builtin_amdgcn_readlane(lo, at), end = __builtin_amdgcn_readlane(hi, at);
      row0 = is_rest ? begin + (end - begin) / tm * tm
                     : begin + (int32_t)(u - (uint32_t)__builtin_amdgcn_readlane((int)at_first, at)) * tm;
      row1 = end - row0 < tm ? end : row0 + tm;
      return true;
    }
    before += (uint32_t)__builtin_amdgcn_readlane((int)up, 63);
  }
  return false;
}

constexpr int kGemmThreads = 512, kGemmK = 64, kGemmLda = kGemmK + 8;
// rows of x~ in LDS, of which there are two tiles: 256 of bf16 x~, 64 of each part of float32 x~
constexpr int gemm_rows(bool f32) { return f32 ? 192 : 256; }
constexpr size_t gemm_lds(size_t tables, bool f32) { return tables + 2 * sizeof(uint16_t) * gemm_rows(f32) * kGemmLda; }

// One tile's loop over k and its end, for 32 MB rows or fewer (row0 .. row1 - 1) and P parts of x~.
//
// A wave owns 32 weight rows for all rows of the tile: MFMA 32x32x16 with x~ from LDS (double-buffered, one
// barrier a step of 64 inputs) and its weights rebuilt straight into the other operand a step ahead,
// so each weight is rebuilt once a workgroup. The step's MFMAs come in runs; the walk of the
// next step's indices (records, halves, combination) and the tile's loads and writes are spread over them.
template <int BPW, bool G4, int MB, int P>
__device__ __forceinline__ void gemm_tile(const XpProduct &a, uint8_t *lds, int e, int32_t row0, int32_t row1, int64_t n0) {
  constexpr bool F32 = P == 3;
  constexpr int TPH = MB < 4 ? MB : 4, HB = MB / TPH;          // MFMA tiles of a run, runs of one of the 4 k-steps
  constexpr int RP = MB < 2 ? 64 : 32 * MB;                    // rows of a part in LDS
  constexpr int PIECES = RP / 64;                              // of 64 rows, a part
  uint16_t *As0 = reinterpret_cast<uint16_t *>(lds + lds_table_bytes<BPW>());
  uint16_t *As1 = As0 + gemm_rows(F32) * kGemmLda;
  const int lane = threadIdx.x & 63, c = lane & 31, p = lane >> 5;
  const int64_t G = a.k / 8, S = a.kp / kGemmK;
  const int64_t left = a.n - n0, rows_w = left < 0 ? 0 : left < 32 ? left : 32, wrow = (int64_t)e * a.n + (rows_w ? n0 : 0);
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
  const uint32_t va = (uint32_t)((threadIdx.x >> 3) * a.kp * 2 + 16 * (threadIdx.x & 7));
  const uint32_t vi = (uint32_t)(c * G + 4 * p);               // this lane's first index of step 0
  const int sa = (int)(64 * a.kp * 2);
  auto load_a = [&](int64_t s, uint4 (&ra)[P * PIECES]) {
#pragma unroll
    for (int q = 0; q < P; ++q)
#pragma unroll
      for (int u = 0; u < PIECES; ++u)
        ra[q * PIECES + u] = __builtin_bit_cast(
            uint4, __builtin_amdgcn_raw_buffer_load_b128(xa[q], va, (int)(2 * kGemmK * s) + u * sa, 0));
  };
  auto store_a = [&](uint16_t *As, const uint4 (&ra)[P * PIECES]) {
#pragma unroll
    for (int i = 0; i < P * PIECES; ++i)
      *reinterpret_cast<uint4 *>(As + ((threadIdx.x >> 3) + 64 * i) * kGemmLda + 8 * (threadIdx.x & 7)) = ra[i];
  };
  // indices of step s as stored; those past a row's end meet zeros of x~
  auto load_idx = [&](int64_t s, uint2 &i1, uint2 &i2) {
    i2 = make_uint2(0u, 0u);
    if constexpr (G4) {
      i1 = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(r1, 2 * vi, (int)(16 * s), 0));
      if constexpr (BPW == 3) i2.x = __builtin_amdgcn_raw_buffer_load_b32(r2, vi, (int)(8 * s), 0);
      if constexpr (BPW == 4) i2 = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(r2, 2 * vi, (int)(16 * s), 0));
    } else {
      uint32_t w[4], v[4] = {0, 0, 0, 0};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        w[u] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r1, 2 * vi, (int)(16 * s + 2 * u), 0);
        if constexpr (BPW == 3) v[u] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(r2, vi, (int)(8 * s + u), 0);
        if constexpr (BPW == 4) v[u] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r2, 2 * vi, (int)(16 * s + 2 * u), 0);
      }
      i1 = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
      if constexpr (BPW == 3) i2.x = v[0] | v[1] << 8 | v[2] << 16 | v[3] << 24;
      if constexpr (BPW == 4) i2 = make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
    }
  };
  uint4 ra[P * PIECES];
  load_a(0, ra);
  uint2 i1, i2, j1, j2;
  load_idx(0, i1, i2);
  tables_landed();                                             // and the first tile and indices
  store_a(As0, ra);
  load_idx(S > 1 ? 1 : 0, j1, j2);
  load_a(S > 1 ? 1 : 0, ra);
  __syncthreads();
  f32x16 acc[MB];
#pragma unroll
  for (int t = 0; t < MB; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[t][i] = 0.f;
  uint4 B0[8], B1[8];                                          // groups u = 0 .. 3 used
  auto plain = [](uint4 w) { return F32 && BPW > 2 ? unbiased(w) : w; };
  {
    uint32_t q1[8], q2[8];
    g8_split<BPW>(i1, i2, q1, q2);
#pragma unroll
    for (int u = 0; u < 4; ++u) B0[u] = plain(decode_ip<BPW>(q1[u], q2[u]));
  }
  i1 = j1;
  i2 = j2;
  uint4 H0[P * TPH], H1[P * TPH];                              // operands of even and odd runs
  auto read_a = [&](const uint16_t *As, int run, uint4 (&h)[P * TPH]) {
    const int u = run / HB, t0 = TPH * (run % HB);
#pragma unroll
    for (int q = 0; q < P; ++q)
#pragma unroll
      for (int t = 0; t < TPH; ++t)
        h[q * TPH + t] = *reinterpret_cast<const uint4 *>(As + (q * RP + 32 * (t0 + t) + c) * kGemmLda + 32 * p + 8 * u);
  };
  read_a(As0, 0, H0);
  auto kstep = [&](int64_t s, const uint4 (&bc)[8], uint4 (&bn)[8]) {
    const uint16_t *Acur = (s & 1) ? As1 : As0;
    uint16_t *Anext = (s & 1) ? As0 : As1;
    uint32_t q1[8], q2[8];
    g8_split<BPW>(i1, i2, q1, q2);                             // of step s + 1
    load_idx(s + 2 < S ? s + 2 : S - 1, i1, i2);
    auto run = [&](int h, const uint4 (&av)[P * TPH], uint4 (&an)[P * TPH]) {
      if (h + 1 < 4 * HB) read_a(Acur, h + 1, an);
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
    D.template p1<0, 4>(q1, q2);
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
      load_a(s + 2 < S ? s + 2 : S - 1, ra);
      run(5, H1, H0);
      gm_interleave<4, 0, 1, 0, 1>();
      __builtin_amdgcn_sched_barrier(0);
      run(6, H0, H1);
      __builtin_amdgcn_sched_barrier(0);
      __syncthreads();
      run(7, H1, H0);
      __builtin_amdgcn_sched_barrier(0);
    } else {
      run(0, H0, H1);
      __builtin_amdgcn_sched_barrier(0);
      D.template p2<0, 4>(q1, q2);
      run(1, H1, H0);
      __builtin_amdgcn_sched_barrier(0);
      store_a(Anext, ra);
      load_a(s + 2 < S ? s + 2 : S - 1, ra);
      run(2, H0, H1);
      D.template p3<0, 4>(bn);
#pragma unroll
      for (int u = 0; u < 4; ++u) bn[u] = plain(bn[u]);
      __syncthreads();
      run(3, H1, H0);
    }
  };
  int64_t s = 0;
  for (; s + 1 < S; s += 2) {
    kstep(s, B0, B1);
    kstep(s + 1, B1, B0);
  }
  if (s < S) kstep(s, B0, B1);
  // lane (c, p) holds rows 8 (i >> 2) + 4 p + (i & 3) of weight row n0 + c: whole lines of z a half-wave
  if (c >= rows_w) return;
  float post = a.scale[e] * Epi<BPW>::mul;
  if (a.row_scale) post *= a.row_scale[wrow + c];
#pragma unroll
  for (int t = 0; t < MB; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int32_t r = row0 + 32 * t + 8 * (i >> 2) + 4 * p + (i & 3);
      if (r >= row1) continue;
      const float bias = F32 || BPW == 2 ? 0.0f : Epi<BPW>::bias * a.rowsum[r];
      a.z[(int64_t)r * a.n + n0 + c] = post * (acc[t][i] - bias);
    }
}

template <int BPW, bool G4, bool F32>
__global__ void __launch_bounds__(kGemmThreads, 1) xp_gemm_k(XpProduct a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  int e;
  int32_t row0, row1;
  uint32_t group;
  if (!find_tile(a.offsets, a.count, a.rows, blockIdx.x, a.n_groups, F32 ? 64 : 256, e, row0, row1, group)) return;
  load_tables<BPW, kGemmThreads>(lds, a.cb);         // (only now: LDS loads in flight must not outlive their workgroup)
  const int64_t n0 = (int64_t)group * 256 + 32 * __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t rows = row1 - row0;
  if constexpr (F32) {
    if (rows > 32) gemm_tile<BPW, G4, 2, 3>(a, lds, e, row0, row1, n0);
    else gemm_tile<BPW, G4, 1, 3>(a, lds, e, row0, row1, n0);
  } else {
    if (rows > 128) gemm_tile<BPW, G4, 8, 1>(a, lds, e, row0, row1, n0);
    else if (rows > 64) gemm_tile<BPW, G4, 4, 1>(a, lds, e, row0, row1, n0);
    else if (rows > 32) gemm_tile<BPW, G4, 2, 1>(a, lds, e, row0, row1, n0);
    else gemm_tile<BPW, G4, 1, 1>(a, lds, e, row0, row1, n0);
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
int64_t up64(int64_t v) { return (v + 63) & ~int64_t(63); }
int64_t up256(int64_t v) { return (v + 255) & ~int64_t(255); }

int log_block(int64_t len) {
  int lb = 0;
  while (!(len >> lb & 1)) ++lb;
  return lb;
}

template <int E, int NW, bool OUT, bool F32>
int launch_transform_k(const XpRows &a, int64_t groups, hipStream_t st) {
  constexpr size_t shm = sizeof(float) * (64 * NW * E + 64);
  if constexpr (OUT) {
    const int rc = allow_lds<xp_out_k<E, NW, F32>>(shm);
    if (rc) return rc;
    hipLaunchKernelGGL((xp_out_k<E, NW, F32>), dim3((unsigned)groups), dim3(64 * NW), shm, st, a);
    return hip_status(hipGetLastError(), "xp_out_k");
  } else {
    const int rc = allow_lds<xp_in_k<E, NW, F32>>(shm);
    if (rc) return rc;
    hipLaunchKernelGGL((xp_in_k<E, NW, F32>), dim3((unsigned)groups), dim3(64 * NW), shm, st, a);
    return hip_status(hipGetLastError(), "xp_in_k");
  }
}

// 8 elements a thread, as many waves as the row (or 8192 of it at a time) takes; whole blocks of 16384 need 16 a thread.
template <bool OUT, bool F32>
int launch_transform(const XpRows &a, int64_t groups, hipStream_t st) {
  const int64_t len = OUT ? a.n : a.k;
  if ((OUT ? a.log_n : a.log_k) == 14) return launch_transform_k<16, 16, OUT, F32>(a, groups, st);
  if (len <= 512) return launch_transform_k<8, 1, OUT, F32>(a, groups, st);
  if (len <= 1024) return launch_transform_k<8, 2, OUT, F32>(a, groups, st);
  if (len <= 2048) return launch_transform_k<8, 4, OUT, F32>(a, groups, st);
  if (len <= 4096) return launch_transform_k<8, 8, OUT, F32>(a, groups, st);
  return launch_transform_k<8, 16, OUT, F32>(a, groups, st);
}

template <int BPW, bool G8, bool F32>
int launch_rows(XpProduct a, hipStream_t st) {
  a.n_groups = (uint32_t)((a.n + 127) / 128);
  // units of 64 rows: no more than this, whatever the offsets are
  const int64_t groups = (a.rows / 64 + (a.count < a.rows ? a.count : a.rows)) * a.n_groups;
  if (groups > 0xFFFFFFFFll / 512) return GLQ_ERR_UNSUPPORTED;
  constexpr size_t shm = lds_table_bytes<BPW>();
  const int rc = allow_lds<xp_rows_k<BPW, G8, F32>>(shm);
  if (rc) return rc;
  hipLaunchKernelGGL((xp_rows_k<BPW, G8, F32>), dim3((unsigned)groups), dim3(512), shm, st, a);
  return hip_status(hipGetLastError(), "xp_rows_k");
}

template <int BPW, bool G4, bool F32>
int launch_gemm(XpProduct a, hipStream_t st) {
  constexpr int TM = F32 ? 64 : 256;
  a.n_groups = (uint32_t)((a.n + 255) / 256);
  // whole groups of rows and remainders: no more than this, whatever the offsets are; up to 7 blocks to fill the XCDs' runs of each
  const int64_t groups = (a.rows / TM + (a.count < a.rows ? a.count : a.rows)) * a.n_groups + 16;
  if (groups > 0xFFFFFFFFll / kGemmThreads) return GLQ_ERR_UNSUPPORTED;
  constexpr size_t shm = gemm_lds(lds_table_bytes<BPW>(), F32);
  const int rc = allow_lds<xp_gemm_k<BPW, G4, F32>>(shm);
  if (rc) return rc;
  hipLaunchKernelGGL((xp_gemm_k<BPW, G4, F32>), dim3((unsigned)groups), dim3(kGemmThreads), shm, st, a);
  return hip_status(hipGetLastError(), "xp_gemm_k");
}

template <int BPW>
int launch_product(const XpProduct &a, bool f32, hipStream_t st) {
  if (a.rows >= 32 * (int64_t)a.count) {
    if (a.k % 32 == 0) return f32 ? launch_gemm<BPW, true, true>(a, st) : launch_gemm<BPW, true, false>(a, st);
    return f32 ? launch_gemm<BPW, false, true>(a, st) : launch_gemm<BPW, false, false>(a, st);
  }
  if (a.k % 64 == 0) return f32 ? launch_rows<BPW, true, true>(a, st) : launch_rows<BPW, true, false>(a, st);
  return f32 ? launch_rows<BPW, false, true>(a, st) : launch_rows<BPW, false, false>(a, st);
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

struct XpLayout { int64_t xt, rowsum, row_expert, z, total; };
XpLayout xp_layout(const glq_experts *E, int64_t rows) {
  XpLayout w;
  w.xt = 0;
  w.rowsum = w.xt + up256(rows * up64(E->k) * 6);          // float32 rows: three parts of 2 bytes
  w.row_expert = w.rowsum + up256(rows * 4);
  w.z = w.row_expert + up256(rows * 4);
  w.total = w.z + up256(rows * E->n * 4);
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
  const XpRows a = {R->x, R->y, R->offsets, R->src, R->pos, R->weights, E->sign_k, E->sign_n,
                    reinterpret_cast<uint16_t *>(ws + l.xt), reinterpret_cast<float *>(ws + l.rowsum),
                    reinterpret_cast<float *>(ws + l.z), reinterpret_cast<int32_t *>(ws + l.row_expert), E->k, up64(E->k), E->n, R->x_rows,
                    (int32_t)E->count, (int32_t)R->rows, R->pos ? R->top_k : 1, log_block(E->k), log_block(E->n)};
  const bool f32 = R->x_dt == GLQ_F32;
  hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
  if (R->rows > 0) {
    rc = f32 ? launch_transform<false, true>(a, R->rows, st) : launch_transform<false, false>(a, R->rows, st);
    if (rc) return rc;
    const XpProduct p = {E->idx1, a.xt, E->idx2, reinterpret_cast<const uint8_t *>(E->cb), E->scale, E->row_scale, a.rowsum,
                         a.offsets, a.z, E->n, E->k, a.kp, a.count, a.rows, 0};
    rc = E->bpw == 2 ? launch_product<2>(p, f32, st) : E->bpw == 3 ? launch_product<3>(p, f32, st) : launch_product<4>(p, f32, st);
    if (rc) return rc;
  }
  return R->y_dt == GLQ_F32 ? launch_transform<true, true>(a, out, st) : launch_transform<true, false>(a, out, st);
}
