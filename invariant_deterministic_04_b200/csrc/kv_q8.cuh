// The 8-bit paged KV store: rows quantised as they are written, and read back.
//
// A store row (page slot of one kv-head, D values) holds 8-bit values v and one fp32 scale
// s; it stands for v * s. From a bf16 row x with a = max |x|:
//   int8: s = a / 127 (one fp32 rounding), v = the integer nearest to 127 x / a, ties to even.
//     127 x has at most 15 significant bits, so it is exact in fp32 and v takes one rounded
//     division (divide8) and one rounding to an integer. Together they are exact: with x = mx 2^(j-d)
//     and a = ma 2^j (mx, ma < 2^8, ma >= 2^7) a quotient q >= 2^n that is no half-integer is
//     at least 2^-d / 255 > 2^(n-16) from the nearest one, and the division is off by 2^(n-24)
//     at most; a half-integer is representable, so the division gives it and the tie goes to even.
//   e4m3: s = 2^e, the least power of two with a <= 448 s; v = e4m3(x / s), nearest even. The
//     division by a power of two is exact.
//   a < 2^-100 (a row of zeros too): v = 0, s = 1. A row with a NaN or an infinity: v = 0,
//     s = NaN, so that it reads back, and enters attention, as NaN.
// Each element depends on its own row only.
//
// Floor: HBM. A row of D bf16 is read once (2 D bytes) and D + 4 bytes are written. Append is bound by
// instructions (it issues in 73 % of the cycles), read by the latency of its 8-byte loads. K and V of one
// (row, kv-head) go on the same D / 8 lanes, 16 bytes a lane of each. Appending 65536 rows of 8
// heads of 128 and reading them back moves 815 MB in 187 us, 4.4 TB/s (300 us with K and V on
// different lanes and a divide instruction sequence in place of divide8).
#pragma once

#include <cuda_fp8.h>

#include "attention.cuh"
#include "device.cuh"

namespace bi {
namespace kvq8 {

constexpr int PAGE = BI_PAGE_TOKENS;
constexpr int kThreads = 256;
constexpr uint32_t kEmptyBits = 0x0D80u;     // bf16 bits of 2^-100
constexpr uint32_t kLoudBits = 0x5F80u;      // bf16 bits of 2^64
constexpr uint32_t kNonFiniteBits = 0x7F80u; // bf16 bits of infinity

struct Store {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  int64_t num_pages;
  const int32_t* pt;
  int num_seqs, max_pages;
};

// Store row of (seq, pos) for kv-head g, or -1 (error recorded) if an id is out of range.
__device__ __forceinline__ int64_t slot_row(const Store& S, int seq, int pos, int g, int Hkv, bool report) {
  int pg = -1;
  if (seq >= 0 && seq < S.num_seqs && pos >= 0 && pos < S.max_pages * PAGE)
    pg = S.pt[(int64_t)seq * S.max_pages + pos / PAGE];
  if (pg < 0 || pg >= S.num_pages) {
    if (report) record_error(BI_ERR_DEVICE_INDEX);
    return -1;
  }
  return ((int64_t)pg * Hkv + g) * PAGE + pos % PAGE;
}

// D/8 lanes hold a row, 8 values each: the largest bit pattern of |x| over the row (bf16
// magnitudes order like integers, NaN above infinity above the finite ones).
template <int LANES>
__device__ __forceinline__ uint32_t row_max_bits(const uint4& x) {
  uint32_t m = 0;
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
#pragma unroll
  for (int off = LANES / 2; off >= 1; off >>= 1) m = max(m, __shfl_xor_sync(kFullMask, m, off));
  return m;
}

// The int8 values of 8 elements, rows below 2^64 given as they are and others at 2^-64 (num = 127 or
// 127 * 2^-64; a and its rounded reciprocal to match). The division is one step of a published
// correction (Markstein, IBM J. R&D 34, 1990): q0 = y r, q = q0 + (y - q0 a) r. The remainder is exact
// (y - q0 a is a multiple of ulp(q0) ulp(a) below 2^9 of it), so q is the quotient but for
// 2^-47 of it, rounded once: what the exactness above asks for. Adding 1.5 * 2^23 rounds to an
// integer, ties to even, whose low byte is the value.
__device__ __forceinline__ uint2 divide8(const uint4& x, float num, float a, float r) {
  float2 f[4];
  unpack8x2(x, f);
  const float2 n2 = make_float2(num, num), a2 = make_float2(-a, -a), r2 = make_float2(r, r);
  const float2 magic = make_float2(12582912.f, 12582912.f);
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = __fmul2_rn(n2, f[i]);
    const float2 q0 = __fmul2_rn(y, r2);
    const float2 q = __fadd2_rn(__ffma2_rn(__ffma2_rn(q0, a2, y), r2, q0), magic);
    v[i] = __byte_perm(__float_as_uint(q.x), __float_as_uint(q.y), 0x0040);
  }
  return make_uint2(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410));
}

template <int KIND>
__device__ __forceinline__ uint2 quantise8(const uint4& x, uint32_t amax_bits, float& scale) {
  const float a = __uint_as_float(amax_bits << 16);
  if (amax_bits < kEmptyBits || amax_bits >= kNonFiniteBits) {
    scale = amax_bits < kEmptyBits ? 1.f : __uint_as_float(0x7FC00000u);
    return make_uint2(0, 0);
  }
  if constexpr (KIND == BI_KV_INT8) {
    scale = __fdiv_rn(a, 127.f);
    // rows from 2^64 on are divided at 2^-64 of their size, where 127 x cannot overflow (elements
    // that this takes below the normal numbers are far below half a step)
    const bool loud = amax_bits >= kLoudBits;
    const float den = loud ? __fmul_rn(a, 0x1p-64f) : a;
    return divide8(x, loud ? 127.f * 0x1p-64f : 127.f, den, __frcp_rn(den));
  } else {
    float f[8];
    unpack8(x, f);
    // a = (1 + m / 128) 2^n: 448 = 1.75 * 2^8, so e = n - 8, one more where 1 + m / 128 > 1.75
    const int e = (int)(amax_bits >> 7) - 127 - 8 + ((amax_bits & 0x7Fu) > 0x60u ? 1 : 0);
    scale = __uint_as_float((uint32_t)(e + 127) << 23);
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
    uint16_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      h[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(f[2 * i], inv), __fmul_rn(f[2 * i + 1], inv)),
                                      __NV_SATFINITE, __NV_E4M3);
    return make_uint2((uint32_t)h[0] | (uint32_t)h[1] << 16, (uint32_t)h[2] | (uint32_t)h[3] << 16);
  }
}

// D/8 lanes take the K and the V row of one (row, kv-head); items is T * Hkv.
template <int KIND, int D>
__global__ void __launch_bounds__(kThreads) kv_append_q8_kernel(const uint16_t* __restrict__ kn,
                                                                const uint16_t* __restrict__ vn, int64_t ld_new,
                                                                const int32_t* __restrict__ q_seq,
                                                                const int32_t* __restrict__ q_pos, Store S,
                                                                uint32_t items, uint32_t Hkv) {
  constexpr uint32_t LANES = D / 8;
  const uint32_t item = blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
  const int j = (int)(threadIdx.x % LANES);
  pdl_wait();  // inputs written by the previous kernel on the stream are complete from here on
  pdl_trigger();
  const bool live = item < items;  // (the others keep the shuffles whole)
  const uint32_t it = live ? item : 0, t = it / Hkv, g = it - t * Hkv;
  const int64_t at = (int64_t)t * ld_new + (int64_t)g * D;
  const uint4 k = __ldg(reinterpret_cast<const uint4*>(kn + at) + j), v = __ldg(reinterpret_cast<const uint4*>(vn + at) + j);
  const int64_t row = slot_row(S, q_seq[t], q_pos[t], (int)g, (int)Hkv, live && j == 0);
  const uint32_t ka = row_max_bits<LANES>(k), va = row_max_bits<LANES>(v);
  if (!live || row < 0) return;
  float ks, vs;
  const uint2 k8 = quantise8<KIND>(k, ka, ks), v8 = quantise8<KIND>(v, va, vs);
  reinterpret_cast<uint2*>(S.k + row * D)[j] = k8;
  reinterpret_cast<uint2*>(S.v + row * D)[j] = v8;
  if (j == 0) {
    S.ks[row] = ks;
    S.vs[row] = vs;
  }
}

template <int KIND>
__device__ __forceinline__ void widen4(uint32_t w, float (&f)[4]) {
  if constexpr (KIND == BI_KV_INT8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = (float)(int8_t)(w >> (8 * i));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3);
      const float2 p = __half22float2(__half2(h));
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
}

template <int KIND>
__device__ __forceinline__ uint4 read8(const uint2& v, float s) {
  float f[4], h[4];
  widen4<KIND>(v.x, f);
  widen4<KIND>(v.y, h);
  return make_uint4(pack_bf16x2(__fmul_rn(f[0], s), __fmul_rn(f[1], s)), pack_bf16x2(__fmul_rn(f[2], s), __fmul_rn(f[3], s)),
                    pack_bf16x2(__fmul_rn(h[0], s), __fmul_rn(h[1], s)), pack_bf16x2(__fmul_rn(h[2], s), __fmul_rn(h[3], s)));
}

// The inverse: bf16(v * s) of the store rows at (q_seq[t], q_pos[t]); zeros where an id is bad.
template <int KIND, int D>
__global__ void __launch_bounds__(kThreads) kv_read_q8_kernel(uint16_t* __restrict__ ko, uint16_t* __restrict__ vo,
                                                              int64_t ld_out, const int32_t* __restrict__ q_seq,
                                                              const int32_t* __restrict__ q_pos, Store S, uint32_t items,
                                                              uint32_t Hkv) {
  constexpr uint32_t LANES = D / 8;
  const uint32_t item = blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
  const int j = (int)(threadIdx.x % LANES);
  pdl_wait();  // the store is complete from here on
  pdl_trigger();
  if (item >= items) return;
  const uint32_t t = item / Hkv, g = item - t * Hkv;
  const int64_t row = slot_row(S, q_seq[t], q_pos[t], (int)g, (int)Hkv, j == 0);
  uint4 k = make_uint4(0, 0, 0, 0), v = k;
  if (row >= 0) {
    const uint2 k8 = reinterpret_cast<const uint2*>(S.k + row * D)[j], v8 = reinterpret_cast<const uint2*>(S.v + row * D)[j];
    const float ks = S.ks[row], vs = S.vs[row];
    k = read8<KIND>(k8, ks);
    v = read8<KIND>(v8, vs);
  }
  const int64_t at = (int64_t)t * ld_out + (int64_t)g * D;
  reinterpret_cast<uint4*>(ko + at)[j] = k;
  reinterpret_cast<uint4*>(vo + at)[j] = v;
}

}  // namespace kvq8
}  // namespace bi
