// msa_rope.cu — what lies between a layer's projections and its attention: per-head norm and
// rotary positions on the queries (cast to E4M3) and on the new keys (quantised straight into
// their cache pages), and the read-back of cached rows.
//
// ("vLLM ofrece soporte en día 0 para MiniMax-M3.1-Flash", "QKV GEMM + norm + RoPE + KV inserción
// fusión".) Sixteen lanes own one 128-element row, eight elements a lane, so that the norm's sum and the
// NVFP4 scale are shuffles inside the half warp; a query row's elements lie as the rotation pairs them up,
// a cache row's in order (its codes and scales are groups of neighbours) and its partners come by shuffles. The
// cosines and sines of a token are computed once per CTA (they are the same for all its heads).
// What bounds them: the queries their bytes where a lane's pieces are neighbours (8,192 x 64 f16 rows, interleaved pairs:
// 35.4 us, 5.69 TB/s); in the half layout they are apart, and loads and stores touch sectors twice (bf16, normalised: 48 us,
// 4.2 TB/s). The append and the read-back their instructions (16,383 tokens from fp32 rows: 23 and 14 us, where their bytes
// take 13 and 4.4; 8,192 from bf16 rows: 12 us, 3.6).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "msa.h"
#include "msa_device.cuh"
#include "msa_host.h"

namespace msa {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsAtOnce = kThreads / 16;
// Resident CTAs an SM: the kernels wait for memory, then for their angles (8,192 x 64 f16 rows: 35.7 us
// with six, 37.2 with five; six leave 40 registers, and four rows of 16 bits spill 32 bytes). The insert by tokens
// holds four rows (16,383 tokens and their read-back: 34.6 us with four, where fp32 rows spill 16 bytes, 36.7 with
// three, 43.2 with five, which spills more).
constexpr int kCtas = 6, kInsertCtas = 5, kTokenCtas = 4;

// i / d by a product and a shift: d_inv = 2^22 / d rounded up, exact where i d < 2^22 (a division is some
// twenty instructions, and these stand on every row's and every angle's path).
__host__ __device__ constexpr uint32_t inverse(uint32_t d) { return ((1u << 22) + d - 1) / d; }
__device__ __forceinline__ uint32_t quotient(uint32_t i, uint32_t d_inv) { return i * d_inv >> 22; }

struct Rope {
  const double* inv_freq;
  int rot, layout;
  float scale;
  uint32_t half_inv;  // inverse(rot / 2)
};

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// Eight elements of a row as loaded (a row waits in this form: four registers for a 16-bit type).
template <typename In>
struct Raw {
  uint4 v[sizeof(In) / 2];
  __device__ __forceinline__ void load(const In* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(In) / 2); ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(In) / 2); ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const;
};
template <>
__device__ __forceinline__ void Raw<float>::get(float (&x)[8]) const {
  x[0] = __uint_as_float(v[0].x); x[1] = __uint_as_float(v[0].y); x[2] = __uint_as_float(v[0].z); x[3] = __uint_as_float(v[0].w);
  x[4] = __uint_as_float(v[1].x); x[5] = __uint_as_float(v[1].y); x[6] = __uint_as_float(v[1].z); x[7] = __uint_as_float(v[1].w);
}
template <>
__device__ __forceinline__ void Raw<__nv_bfloat16>::get(float (&x)[8]) const {
  const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
template <>
__device__ __forceinline__ void Raw<__half>::get(float (&x)[8]) const {
  const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// Cosines and sines (times the scale) of tokens t0 .. t0 + nt - 1: cs[token][0][i], cs[token][1][i].
// The frequency as a fraction of a turn, in units of 2^-64, times the position wraps modulo one
// turn for free. Its top 32 bits are taken to the nearest quarter turn, and only what is left, at most an
// eighth of a turn either way, is rounded to fp32: off by 2^-27 half turns at most. (A whole turn in fp32,
// off by 2^-25, is 1 us faster for 8,192 x 64 rows, and changed bytes next to a tie.)
__device__ __forceinline__ void angle(double freq, int32_t pos, float scale, float* cos_out, float* sin_out) {
  double turn = freq * 0.15915494309189533577;  // 1 / (2 pi)
  turn -= floor(turn);
  const unsigned long long step = __double2ull_rn(turn * 18446744073709551616.0);
  const unsigned long long at = step * static_cast<unsigned long long>(static_cast<long long>(pos));
  const uint32_t hi = static_cast<uint32_t>((at + 0x80000000ull) >> 32), quarter = (hi + 0x20000000u) >> 30;
  float s, c;
  sincospif(static_cast<float>(static_cast<int>(hi - (quarter << 30))) * 4.656612873077392578125e-10f, &s, &c);  // 2^-31
  const float k = quarter & 2u ? -scale : scale;
  *cos_out = (quarter & 1u ? -s : c) * k;
  *sin_out = (quarter & 1u ? c : s) * k;
}
__device__ __forceinline__ void fill_angles(float (*cs)[2][64], const Rope& r, const int32_t* positions, int64_t t0,
                                            int nt) {
  const int half = r.rot >> 1;
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int t = static_cast<int>(quotient(i, r.half_inv)), j = i - t * half;  // i < 17 tokens x 64
    angle(r.inv_freq[j], positions[t0 + t], r.scale, &cs[t][0][j], &cs[t][1][j]);
  }
}

// x * rsqrt(mean(x^2) + eps) over the 16 lanes of a row; every lane of the warp calls it.
__device__ __forceinline__ float norm_factor(const float (&x)[8], float eps) {
  float s0 = 0.f, s1 = 0.f;
#pragma unroll
  for (int j = 0; j < 8; j += 2) fma_f32x2(x[j], x[j + 1], x[j], x[j + 1], s0, s1, s0, s1);
  float s = s0 + s1;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return rsqrtf(fmaf(s, 1.0f / kD, eps));
}

__device__ __forceinline__ void scale_row(float (&x)[8], float f, const float* weight) {
  float w[8];
  load8(weight, w);
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = x[j] * f * w[j];
}

// Rotate the row whose elements 8 l .. 8 l + 7 this lane (l = lane % 16) holds; every lane of the
// warp calls it (`on` false: shuffles only).
__device__ __forceinline__ void rotate(float (&x)[8], const float (*cs)[64], int rot, int layout, bool on) {
  const int l = threadIdx.x & 15, half = rot >> 1, d0 = 8 * l;
  if (layout == MSA_ROPE_HALF) {
    const bool low = d0 < half;
    const int partner = low ? l + (half >> 3) : l - (half >> 3);  // rot % 16 == 0: whole lanes
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = __shfl_sync(0xffffffffu, x[j], partner & 15, 16);
    if (on && d0 < rot) {
      const int j0 = low ? d0 : d0 - half;
      float c[8], s[8];
      load8(&cs[0][j0], c);
      load8(&cs[1][j0], s);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = fmaf(y[j], low ? -s[j] : s[j], x[j] * c[j]);
    }
  } else if (on && d0 < rot) {
    const float4 c4 = *reinterpret_cast<const float4*>(&cs[0][4 * l]), s4 = *reinterpret_cast<const float4*>(&cs[1][4 * l]);
    const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = fmaf(b, -s[i], a * c[i]);
      x[2 * i + 1] = fmaf(a, s[i], b * c[i]);
    }
  }
}

__device__ __forceinline__ uint2 to_e4m3(const float (&x)[8]) {
  return make_uint2(cvt_e4m3x2(x[0], x[1]) | (cvt_e4m3x2(x[2], x[3]) << 16),
                    cvt_e4m3x2(x[4], x[5]) | (cvt_e4m3x2(x[6], x[7]) << 16));
}

// The tokens and heads (or kinds) of a CTA's rows: row r0 + i = token t0 + (first + i) / per, head
// (first + i) % per. At most 2^22 x 1024 rows: r0 fits 32 bits, and so do all the divisions (with 64-bit
// ones 8,192 x 64 rows took 91 us).
struct Span {
  uint32_t r0, t0, first;
  int n;  // rows of this CTA
  __device__ Span(int64_t rows, int at_once, uint32_t per) {
    r0 = blockIdx.x * static_cast<uint32_t>(at_once);
    t0 = r0 / per;
    first = r0 - t0 * per;
    n = static_cast<int>(rows - r0 < at_once ? rows - r0 : at_once);
  }
};

// Eight elements of a row as the rotation pairs them up: two pieces of four, (i, i + rot / 2) in the half
// layout (lanes below rot / 8), neighbours everywhere else, so that no rotation leaves its lane.
struct Pieces {
  int d0, d1;
  __device__ __forceinline__ Pieces(int rot, int layout) {
    const int l = threadIdx.x & 15;
    const bool apart = layout == MSA_ROPE_HALF && l < rot >> 3;
    d0 = apart ? 4 * l : 8 * l;
    d1 = apart ? 4 * l + (rot >> 1) : 8 * l + 4;
    // in the half layout the lanes below rot / 8 hold all the rotated elements, the others the rest in order
  }
};
template <typename In>
struct Raw4 {
  uint32_t v[sizeof(In)];
  __device__ __forceinline__ void load(const In* p) {
    if constexpr (sizeof(In) == 4) {
      const uint4 a = *reinterpret_cast<const uint4*>(p);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    } else {
      const uint2 a = *reinterpret_cast<const uint2*>(p);
      v[0] = a.x; v[1] = a.y;
    }
  }
  __device__ __forceinline__ void get(float* x) const {
    if constexpr (std::is_same<In, float>::value) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if constexpr (std::is_same<In, __nv_bfloat16>::value) {
          x[2 * i] = __uint_as_float(v[i] << 16);
          x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[i]));
          x[2 * i] = f.x;
          x[2 * i + 1] = f.y;
        }
      }
    }
  }
};

// R rows a half warp: CTA c takes rows c * 16 R ..., row = token * heads + head. Dynamic shared
// memory: the angles of the tokens those rows touch.
template <typename In, int R>
__global__ void __launch_bounds__(kThreads, kCtas) k_rope_fp8(const In* __restrict__ x, int64_t rows, int32_t heads, uint32_t heads_inv,
                                                       int64_t tstride, int64_t hstride,
                                                       const int32_t* __restrict__ positions, const Rope rope,
                                                       const float* __restrict__ norm, float eps,
                                                       uint8_t* __restrict__ out) {
  extern __shared__ float4 smem4[];
  float (*cs)[2][64] = reinterpret_cast<float (*)[2][64]>(smem4);
  grid_dependency_wait();
  const Span sp(rows, kRowsAtOnce * R, static_cast<uint32_t>(heads));
  const int l = threadIdx.x & 15, w = threadIdx.x >> 4;
  const bool half = rope.layout == MSA_ROPE_HALF, turns = l < rope.rot >> 3;
  const Pieces at(rope.rot, rope.layout);
  Raw4<In> ra[R], rb[R];
  int tok[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int n = i * kRowsAtOnce + w;
    tok[i] = 0;
#pragma unroll
    for (int j = 0; j < static_cast<int>(sizeof(In)); ++j) ra[i].v[j] = rb[i].v[j] = 0u;
    if (n < sp.n) {
      const uint32_t k = sp.first + n;
      tok[i] = static_cast<int>(quotient(k, heads_inv));  // k < heads + 64
      const int64_t head = k - static_cast<uint32_t>(tok[i]) * static_cast<uint32_t>(heads);
      const In* p = x + (static_cast<int64_t>(sp.t0) + tok[i]) * tstride + head * hstride;
      if (half || sizeof(In) == 4) {
        ra[i].load(p + at.d0);
        rb[i].load(p + at.d1);
      } else {  // neighbours: one 16-byte load
        const uint4 a = *reinterpret_cast<const uint4*>(p + at.d0);
        ra[i].v[0] = a.x; ra[i].v[1] = a.y;
        rb[i].v[0] = a.z; rb[i].v[1] = a.w;
      }
    }
  }
  if (rope.rot > 0) fill_angles(cs, rope, positions, sp.t0, static_cast<int>(quotient(sp.first + sp.n - 1, heads_inv)) + 1);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int n = i * kRowsAtOnce + w;
    float v[8];
    ra[i].get(v);
    rb[i].get(v + 4);
    if (norm != nullptr) {
      const float f = norm_factor(v, eps);
      const float4 a = *reinterpret_cast<const float4*>(norm + at.d0), b = *reinterpret_cast<const float4*>(norm + at.d1);
      const float wt[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = v[j] * f * wt[j];
    }
    if (turns) {
      const float4 c4 = *reinterpret_cast<const float4*>(&cs[tok[i]][0][4 * l]),
                   s4 = *reinterpret_cast<const float4*>(&cs[tok[i]][1][4 * l]);
      const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
      if (half) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float a = v[j], b = v[4 + j];
          v[j] = fmaf(b, -s[j], a * c[j]);
          v[4 + j] = fmaf(a, s[j], b * c[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float a = v[2 * j], b = v[2 * j + 1];
          v[2 * j] = fmaf(b, -s[j], a * c[j]);
          v[2 * j + 1] = fmaf(a, s[j], b * c[j]);
        }
      }
    }
    if (n < sp.n) {
      uint8_t* o = out + (static_cast<int64_t>(sp.r0) + n) * kD;
      const uint2 e = to_e4m3(v);
      if (half) {
        *reinterpret_cast<uint32_t*>(o + at.d0) = e.x;
        *reinterpret_cast<uint32_t*>(o + at.d1) = e.y;
      } else {
        *reinterpret_cast<uint2*>(o + at.d0) = e;
      }
    }
  }
}

struct KvRows {
  const void *k, *v, *ik;
  int64_t kt, kh, vt, vh, it;
};

// Row kinds of a token: 0..3 K of head 0..3, 4..7 V of head 0..3, 8 the index key. A half warp a row.
template <typename In>
__global__ void __launch_bounds__(kThreads, kInsertCtas) k_rope_kv_insert(const KvRows src, int64_t rows, int32_t kinds,
                                                             const int32_t* __restrict__ positions,
                                                             const int64_t* __restrict__ slots, const Rope rope,
                                                             const float* __restrict__ k_norm,
                                                             const float* __restrict__ ik_norm, float eps,
                                                             uint8_t* __restrict__ kv_pages,
                                                             uint8_t* __restrict__ index_pages, int32_t index_dtype,
                                                             int32_t num_pages, uint32_t* status) {
  extern __shared__ float4 smem4[];
  float (*cs)[2][64] = reinterpret_cast<float (*)[2][64]>(smem4);
  grid_dependency_wait();
  const Span sp(rows, kRowsAtOnce, static_cast<uint32_t>(kinds));
  const int l = threadIdx.x & 15, w = threadIdx.x >> 4;
  const uint32_t inv = kinds == 8 ? inverse(8) : inverse(9);
  const bool in = w < sp.n;
  const int tok = in ? static_cast<int>(quotient(sp.first + w, inv)) : 0;
  const int kind = in ? static_cast<int>(sp.first) + w - tok * kinds : 4;
  const int64_t t = static_cast<int64_t>(sp.t0) + tok;
  const int64_t slot = in ? slots[t] : -1;
  const In* p = kind < 4 ? static_cast<const In*>(src.k) + t * src.kt + kind * src.kh
              : kind < 8 ? static_cast<const In*>(src.v) + t * src.vt + (kind - 4) * src.vh
                         : static_cast<const In*>(src.ik) + t * src.it;
  Raw<In> raw;
  if (in) raw.load(p + 8 * l);
  else raw.zero();
  if (rope.rot > 0) fill_angles(cs, rope, positions, sp.t0, static_cast<int>(quotient(sp.first + sp.n - 1, inv)) + 1);
  __syncthreads();
  const bool turns = kind < 4 || kind == 8;
  float v[8];
  raw.get(v);
  if (__any_sync(0xffffffffu, turns)) {  // a warp of two V rows has neither norm nor rotation
    const float* norm = kind < 4 ? k_norm : (kind == 8 ? ik_norm : nullptr);
    if (k_norm != nullptr || ik_norm != nullptr) {
      const float f = norm_factor(v, eps);
      if (norm != nullptr) scale_row(v, f, norm + 8 * l);
    }
    if (rope.rot > 0) rotate(v, cs[tok], rope.rot, rope.layout, turns);
  }
  uint32_t s;
  const uint32_t word = quantize_word(v, &s);
  if (slot == -1) return;
  if (slot < 0 || slot >= static_cast<int64_t>(num_pages) * kBS) {
    if (l == 0) set_status(status, MSA_ERR_DEVICE_FAULT);
    return;
  }
  const int64_t page = slot / kBS;
  const int prow = static_cast<int>(slot % kBS);
  if (kind == 8 && index_dtype == MSA_INDEX_FP8) {
    *reinterpret_cast<uint2*>(index_pages + page * kIdxPageFp8 + prow * kD + 8 * l) = to_e4m3(v);
    return;
  }
  uint8_t* region = kind < 8 ? kv_pages + page * kKvPage + ((kind & 3) * 2 + (kind >> 2)) * kRegion
                             : index_pages + page * kIdxPageNv;
  *reinterpret_cast<uint32_t*>(region + prow * kRowCodes + 4 * l) = word;
  if ((l & 1) == 0) region[kScaleOff + prow * kRowScales + l / 2] = static_cast<uint8_t>(s);
}

// The same for many tokens: a half warp takes a token's rows one after another (its slot, its place in the page
// and its angles once for all nine, V's without the steps it does not need), the next rows loaded meanwhile.
template <typename In>
__global__ void __launch_bounds__(kThreads, kTokenCtas) k_rope_kv_insert_tokens(
    const KvRows src, int64_t n, const int32_t* __restrict__ positions, const int64_t* __restrict__ slots, const Rope rope,
    const float* __restrict__ k_norm, const float* __restrict__ ik_norm, float eps, uint8_t* __restrict__ kv_pages,
    uint8_t* __restrict__ index_pages, int32_t index_dtype, int32_t num_pages, uint32_t* status) {
  __shared__ __align__(16) float cs[kRowsAtOnce][2][64];
  grid_dependency_wait();
  const int l = threadIdx.x & 15, w = threadIdx.x >> 4;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRowsAtOnce + w;
  const bool in = t < n;
  const int64_t slot = in ? slots[t] : -1;
  const In* const vp = static_cast<const In*>(src.v) + t * src.vt + 8 * l;
  Raw<In> raw[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    if (in) raw[h].load(static_cast<const In*>(src.k) + t * src.kt + h * src.kh + 8 * l);
    else raw[h].zero();
  }
  if (rope.rot > 0) {
    const int32_t pos = in ? positions[t] : 0;
    for (int j = l; j < rope.rot >> 1; j += 16) angle(rope.inv_freq[j], pos, rope.scale, &cs[w][0][j], &cs[w][1][j]);
    __syncwarp();
  }
  const bool live = slot >= 0 && slot < static_cast<int64_t>(num_pages) * kBS;
  if (!live && slot != -1 && l == 0) set_status(status, MSA_ERR_DEVICE_FAULT);
  const int64_t page = live ? slot / kBS : 0;
  const int prow = live ? static_cast<int>(slot % kBS) : 0;
  uint8_t* const kv = kv_pages + page * kKvPage;
  auto put = [&](uint8_t* region, const float (&v)[8]) {
    uint32_t s;
    const uint32_t word = quantize_word(v, &s);
    if (live) {
      *reinterpret_cast<uint32_t*>(region + prow * kRowCodes + 4 * l) = word;
      if ((l & 1) == 0) region[kScaleOff + prow * kRowScales + l / 2] = static_cast<uint8_t>(s);
    }
  };
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    float v[8];
    raw[h].get(v);
    if (in) raw[h].load(vp + h * src.vh);
    if (k_norm != nullptr) scale_row(v, norm_factor(v, eps), k_norm + 8 * l);
    if (rope.rot > 0) rotate(v, cs[w], rope.rot, rope.layout, true);
    put(kv + 2 * h * kRegion, v);
  }
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    float v[8];
    raw[h].get(v);
    if (h == 0 && in && src.ik != nullptr) raw[0].load(static_cast<const In*>(src.ik) + t * src.it + 8 * l);
    put(kv + (2 * h + 1) * kRegion, v);
  }
  if (src.ik != nullptr) {
    float v[8];
    raw[0].get(v);
    if (ik_norm != nullptr) scale_row(v, norm_factor(v, eps), ik_norm + 8 * l);
    if (rope.rot > 0) rotate(v, cs[w], rope.rot, rope.layout, true);
    if (index_dtype != MSA_INDEX_FP8) put(index_pages + page * kIdxPageNv, v);
    else if (live) *reinterpret_cast<uint2*>(index_pages + page * kIdxPageFp8 + prow * kD + 8 * l) = to_e4m3(v);
  }
}

// Half warp per cached row. The eight E4M3 values a scale gives (the dequantiser's table entry)
// are computed in registers: with two words a scale that is cheaper than a table in shared memory.
__global__ void __launch_bounds__(kThreads) k_kv_read(const int64_t* __restrict__ slots, int64_t n,
                                                      const uint8_t* __restrict__ kv_pages,
                                                      const uint8_t* __restrict__ index_pages, int32_t index_dtype,
                                                      int32_t num_pages, uint8_t* __restrict__ k,
                                                      uint8_t* __restrict__ v, uint8_t* __restrict__ ik,
                                                      uint32_t* status) {
  grid_dependency_wait();
  const uint32_t rows = static_cast<uint32_t>(n) * 9u;  // n <= 2^22
  const int64_t limit = static_cast<int64_t>(num_pages) * kBS;
  const int l = threadIdx.x & 15;
  for (uint32_t r = blockIdx.x * kRowsAtOnce + (threadIdx.x >> 4); r < rows; r += gridDim.x * kRowsAtOnce) {
    const int64_t t = r / 9u;
    const int kind = static_cast<int>(r % 9u);
    uint8_t* dst = kind < 4 ? k : (kind < 8 ? v : ik);
    if (dst == nullptr) continue;
    dst += (kind < 8 ? t * 4 + (kind & 3) : t) * kD + 8 * l;
    const int64_t slot = slots[t];
    uint32_t lo = 0, hi = 0;
    if (slot >= limit || slot < -1) {
      if (l == 0) set_status(status, MSA_ERR_DEVICE_FAULT);
    } else if (slot >= 0) {
      const int64_t page = slot / kBS;
      const int prow = static_cast<int>(slot % kBS);
      if (kind == 8 && index_dtype == MSA_INDEX_FP8) {
        const uint2 b = *reinterpret_cast<const uint2*>(index_pages + page * kIdxPageFp8 + prow * kD + 8 * l);
        lo = b.x;
        hi = b.y;
      } else {
        const uint8_t* region = kind < 8 ? kv_pages + page * kKvPage + ((kind & 3) * 2 + (kind >> 2)) * kRegion
                                         : index_pages + page * kIdxPageNv;
        const uint32_t word = *reinterpret_cast<const uint32_t*>(region + prow * kRowCodes + 4 * l);
        dq8(word, dequant_entry(region[kScaleOff + prow * kRowScales + l / 2]), lo, hi);
      }
    }
    *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
  }
}

msa_status check_rope(const msa_rope* r, Rope* out) {
  if (r == nullptr || r->rot_dim < 0 || r->rot_dim > kD || r->rot_dim % 16 != 0) return MSA_ERR_INVALID_ARG;
  if (r->layout != MSA_ROPE_HALF && r->layout != MSA_ROPE_INTERLEAVED) return MSA_ERR_INVALID_ARG;
  if (r->rot_dim > 0 && (r->inv_freq == nullptr || !msa_host::aligned(r->inv_freq, 8))) return MSA_ERR_INVALID_ARG;
  if (!isfinite(r->scale)) return MSA_ERR_INVALID_ARG;
  *out = Rope{r->inv_freq, r->rot_dim, r->layout, r->scale, r->rot_dim > 0 ? inverse(r->rot_dim / 2) : 0u};
  return MSA_OK;
}

bool rows_ok(const void* p, int32_t dtype, int64_t tstride, int64_t hstride) {
  const int64_t step = dtype == MSA_F32 ? 4 : 8;  // elements in 16 bytes
  return p != nullptr && msa_host::aligned(p, 16) && tstride % step == 0 && hstride % step == 0;
}

bool dtype_ok(int32_t dtype) { return dtype == MSA_F32 || dtype == MSA_BF16 || dtype == MSA_F16; }

// Many rows a half warp (64 bytes a lane: their loads in flight together, one set of angles for all) from where a row a
// half warp no longer fits the SMs at once, so that fewer rows spread over them. Where such a CTA's rows are more than 8
// tokens' (few heads), their angles are its work, and it pays from eight times as many rows or, past 16 tokens, not
// at all. us with many and with one: 64 normalised heads, half the row turned, 14,592 rows bf16 3.6 and 2.9, fp32
// 2.8 and 2.7; 16,000 rows bf16 3.6 and 3.6 (without norm 2.8 and 3.1), fp32 3.1 and 3.7; 32,768 rows bf16 5.3 and 6.2,
// fp32 6.4 and 6.6. 8 bf16 heads (8 tokens) 16,000 rows 4.1 and 3.7, 32,768 rows 6.0 and 6.3. 4 bf16 heads (16) 16,000
// rows 4.8 and 4.0, 65,536 rows 12.0 and 11.7, 262,144 rows 32.4 and 38.7. One fp32 head (32) 16,384 rows 8.0 and 7.6,
// 262,144 rows 80.1 and 79.0; one bf16 head (64) 9.5 and 7.6, 81.5 and 79.1.
template <typename In>
constexpr int kMany = 8 / sizeof(In);
template <typename In>
bool many_rows(int64_t rows, int32_t heads) {
  const int tokens = (kMany<In> * kRowsAtOnce + heads - 1) / heads;
  return tokens <= 16 && rows > static_cast<int64_t>(kCtas * kRowsAtOnce) * msa_host::kTunedSms * (tokens <= 8 ? 1 : 8);
}
// A half warp a token from one and a half such CTAs an SM on. us with a token and with a row a half warp, rows of a
// packed projection, normalised: bf16 2,200 tokens 6.1 and 5.5, 3,200 7.4 and 7.3, 3,648 7.7 and 8.0, 8,192 12.3 and 16.1;
// fp32 3,648 tokens 8.8 and 8.8, 4,096 9.0 and 9.5, 8,192 13.9 and 16.5 (no norm, the whole row turned, an FP8 index key:
// 3,648 9.0 and 8.4, 4,096 9.4 and 9.2, 8,192 14.7 and 15.9).
bool many_tokens(int64_t n) { return 2 * n >= static_cast<int64_t>(3 * kRowsAtOnce) * msa_host::kTunedSms; }

// Tokens that 16 R consecutive rows of `per` a token can touch, as bytes of angles.
size_t angle_bytes(const Rope& r, int rows, int per) {
  return r.rot > 0 ? static_cast<size_t>((rows + per - 2) / per + 1) * 2 * 64 * sizeof(float) : 0;
}

// The launches may start while the kernel before them on the stream ends: they wait for it first thing.
template <typename In>
cudaError_t launch_rope(const void* x, int64_t rows, int32_t heads, int64_t ts, int64_t hs, const int32_t* pos,
                        const Rope& r, const float* norm, float eps, uint8_t* out, cudaStream_t stream) {
  const bool many = many_rows<In>(rows, heads);
  const int per = many ? kMany<In> * kRowsAtOnce : kRowsAtOnce;
  return msa_host::launch_after_previous(many ? k_rope_fp8<In, kMany<In>> : k_rope_fp8<In, 1>,
                                         dim3(static_cast<unsigned>((rows + per - 1) / per)), dim3(kThreads),
                                         angle_bytes(r, per, heads), stream, static_cast<const In*>(x), rows, heads, inverse(heads), ts,
                                         hs, pos, r, norm, eps, out);
}

template <typename In>
cudaError_t launch_insert(const KvRows& src, int64_t rows, int kinds, const int32_t* pos, const int64_t* slots,
                          const Rope& r, const float* kn, const float* in, float eps, uint8_t* kv, uint8_t* ix,
                          int32_t ixt, int32_t pages, uint32_t* status, cudaStream_t stream) {
  const int64_t n = rows / kinds;
  if (many_tokens(n))
    return msa_host::launch_after_previous(k_rope_kv_insert_tokens<In>,
                                           dim3(static_cast<unsigned>((n + kRowsAtOnce - 1) / kRowsAtOnce)), dim3(kThreads),
                                           0, stream, src, n, pos, slots, r, kn, in, eps, kv, ix, ixt, pages, status);
  return msa_host::launch_after_previous(k_rope_kv_insert<In>,
                                         dim3(static_cast<unsigned>((rows + kRowsAtOnce - 1) / kRowsAtOnce)), dim3(kThreads),
                                         angle_bytes(r, kRowsAtOnce, kinds), stream, src, rows, kinds, pos, slots, r, kn, in,
                                         eps, kv, ix, ixt, pages, status);
}

}  // namespace
}  // namespace msa

using namespace msa;
using namespace msa_host;

extern "C" msa_status msa_rope_inv_freq(int32_t rot_dim, double theta, int32_t kind, double factor,
                                        double original_len, double slow, double fast, double* inv_freq, float* scale) {
  if (rot_dim < 16 || rot_dim > kD || rot_dim % 16 != 0 || inv_freq == nullptr || scale == nullptr)
    return MSA_ERR_INVALID_ARG;
  if (!(theta > 1.0) || !isfinite(theta) || kind < MSA_ROPE_PLAIN || kind > MSA_ROPE_BY_TURNS) return MSA_ERR_INVALID_ARG;
  if (kind != MSA_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor))) return MSA_ERR_INVALID_ARG;
  if (kind >= MSA_ROPE_BY_PARTS &&
      (!(original_len > 0.0) || !isfinite(original_len) || !(slow > 0.0) || !(fast > slow) || !isfinite(fast)))
    return MSA_ERR_INVALID_ARG;
  constexpr double kTwoPi = 6.283185307179586477;
  const int half = rot_dim / 2;
  *scale = kind == MSA_ROPE_BY_PARTS ? static_cast<float>(0.1 * log(factor) + 1.0) : 1.0f;
  // the pair index (a real number) that makes `turns` turns over original_len positions
  auto index_of = [&](double turns) { return half * log(original_len / (turns * kTwoPi)) / log(theta); };
  double lo = 0.0, hi = 0.0;
  if (kind == MSA_ROPE_BY_PARTS) {
    lo = fmax(floor(index_of(fast)), 0.0);
    hi = fmin(ceil(index_of(slow)), rot_dim - 1.0);
    if (hi <= lo) hi = lo + 0.001;
  }
  for (int i = 0; i < half; ++i) {
    const double f = pow(theta, -static_cast<double>(i) / half);
    double keep = 1.0;  // the share left as it is
    if (kind == MSA_ROPE_LINEAR) keep = 0.0;
    if (kind == MSA_ROPE_BY_PARTS) keep = 1.0 - fmin(fmax((i - lo) / (hi - lo), 0.0), 1.0);
    if (kind == MSA_ROPE_BY_TURNS) keep = fmin(fmax((original_len * f / kTwoPi - slow) / (fast - slow), 0.0), 1.0);
    inv_freq[i] = kind == MSA_ROPE_PLAIN ? f : keep * f + (1.0 - keep) * f / factor;
  }
  return MSA_OK;
}

extern "C" msa_status msa_rope_fp8(const void* x, int32_t dtype, int32_t T, int32_t heads, int64_t token_stride,
                                   int64_t head_stride, const int32_t* positions, const msa_rope* rope,
                                   const float* norm_weight, float eps, uint8_t* out, cudaStream_t stream) {
  Rope r;
  if (T < 0 || T > (1 << 22) || heads < 1 || heads > 1024 || !(eps >= 0.f) || !isfinite(eps)) return MSA_ERR_INVALID_ARG;
  if (!dtype_ok(dtype)) return MSA_ERR_UNSUPPORTED;
  msa_status st = check_rope(rope, &r);
  if (st != MSA_OK || T == 0) return st;
  if (!rows_ok(x, dtype, token_stride, head_stride) || out == nullptr || !aligned(out, 16) ||
      (norm_weight != nullptr && !aligned(norm_weight, 16)))
    return MSA_ERR_INVALID_ARG;
  if (r.rot > 0 && (positions == nullptr || !aligned(positions, 4))) return MSA_ERR_INVALID_ARG;
  const int64_t rows = static_cast<int64_t>(T) * heads;
  const auto go = dtype == MSA_F32 ? launch_rope<float> : (dtype == MSA_BF16 ? launch_rope<__nv_bfloat16> : launch_rope<__half>);
  if (go(x, rows, heads, token_stride, head_stride, positions, r, norm_weight, eps, out, stream) != cudaSuccess)
    return MSA_ERR_CUDA;
  return launch_status();
}

extern "C" msa_status msa_rope_kv_insert(const msa_kv_rows* rows, int64_t n, const int32_t* positions,
                                         const int64_t* slots, const msa_rope* rope, const float* k_norm,
                                         const float* ik_norm, float eps, uint8_t* kv_pages, uint8_t* index_pages,
                                         int32_t index_dtype, int32_t num_pages, uint32_t* status, cudaStream_t stream) {
  Rope r;
  if (rows == nullptr || n < 0 || n > (1 << 22) || num_pages < 0 || !(eps >= 0.f) || !isfinite(eps))
    return MSA_ERR_INVALID_ARG;
  if (!dtype_ok(rows->dtype)) return MSA_ERR_UNSUPPORTED;
  if (index_dtype != MSA_INDEX_NVFP4 && index_dtype != MSA_INDEX_FP8) return MSA_ERR_UNSUPPORTED;
  msa_status st = check_rope(rope, &r);
  if (st != MSA_OK || n == 0) return st;
  const bool ik = rows->ik != nullptr;
  if (!rows_ok(rows->k, rows->dtype, rows->k_token_stride, rows->k_head_stride) ||
      !rows_ok(rows->v, rows->dtype, rows->v_token_stride, rows->v_head_stride) ||
      (ik && (!rows_ok(rows->ik, rows->dtype, rows->ik_token_stride, 0) || index_pages == nullptr)))
    return MSA_ERR_INVALID_ARG;
  if (slots == nullptr || !aligned(slots, 8) || kv_pages == nullptr || !aligned(kv_pages, 256) ||
      !aligned(index_pages, 256) || !aligned(k_norm, 16) || !aligned(ik_norm, 16))
    return MSA_ERR_INVALID_ARG;
  if (r.rot > 0 && (positions == nullptr || !aligned(positions, 4))) return MSA_ERR_INVALID_ARG;
  const int kinds = ik ? 9 : 8;
  const KvRows src{rows->k, rows->v, rows->ik, rows->k_token_stride, rows->k_head_stride, rows->v_token_stride,
                   rows->v_head_stride, rows->ik_token_stride};
  const float* in = ik ? ik_norm : nullptr;
  const int64_t total = n * kinds;
  const auto go = rows->dtype == MSA_F32 ? launch_insert<float>
                                         : (rows->dtype == MSA_BF16 ? launch_insert<__nv_bfloat16> : launch_insert<__half>);
  if (go(src, total, kinds, positions, slots, r, k_norm, in, eps, kv_pages, index_pages, index_dtype, num_pages, status,
         stream) != cudaSuccess)
    return MSA_ERR_CUDA;
  return launch_status();
}

extern "C" msa_status msa_kv_read(const int64_t* slots, int64_t n, const uint8_t* kv_pages, const uint8_t* index_pages,
                                  int32_t index_dtype, int32_t num_pages, uint8_t* k, uint8_t* v, uint8_t* ik,
                                  uint32_t* status, cudaStream_t stream) {
  if (n < 0 || n > (1 << 22) || num_pages < 0) return MSA_ERR_INVALID_ARG;
  if (index_dtype != MSA_INDEX_NVFP4 && index_dtype != MSA_INDEX_FP8) return MSA_ERR_UNSUPPORTED;
  if (n == 0) return MSA_OK;
  if (slots == nullptr || !aligned(slots, 8) || !aligned(k, 8) || !aligned(v, 8) || !aligned(ik, 8))
    return MSA_ERR_INVALID_ARG;
  if ((k != nullptr || v != nullptr) && (kv_pages == nullptr || !aligned(kv_pages, 256))) return MSA_ERR_INVALID_ARG;
  if (ik != nullptr && (index_pages == nullptr || !aligned(index_pages, 256))) return MSA_ERR_INVALID_ARG;
  int64_t ctas = (n * 9 + kRowsAtOnce - 1) / kRowsAtOnce;
  if (ctas > kTunedSms * 64) ctas = kTunedSms * 64;
  if (launch_after_previous(k_kv_read, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, stream, slots, n, kv_pages,
                            index_pages, index_dtype, num_pages, k, v, ik, status) != cudaSuccess)
    return MSA_ERR_CUDA;
  return launch_status();
}
