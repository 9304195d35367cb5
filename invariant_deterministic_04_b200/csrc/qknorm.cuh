// Per-head RMSNorm of queries and keys with the rotary embedding in the same pass.
//
// For a head row x of D dims at position p, with r = rsqrt(mean x^2 + eps), n_i = x_i r w_i
// and (c, s) = table[p][i], i < D/2:
//   y_i = n_i c - n_{i+D/2} s,   y_{i+D/2} = n_{i+D/2} c + n_i s,
// all in fp32 and rounded to bf16 once (the norm and the rotation as two calls round n too).
//
// Reduction order of a head row (a function of D only): D/16 lanes share it, lane j owning
// dims 8j .. 8j+7 and D/2+8j .. D/2+8j+7 (a rotation pair never leaves its lane); a lane adds
// its 16 squares in that order in one FMA chain, then an xor butterfly over the D/16 lanes.
// So a row's bits depend on that row, its position and the weights only.
//
// Bound: HBM (each element read and written once; table and weights come from L1 / L2).
#pragma once

#include "device.cuh"

namespace bi {
namespace qknorm {

struct Part {  // queries or keys: rows t at x + t * ldx, written to y + t * ldy
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* w;
  uint16_t* y;
  int64_t ldy;
};

constexpr int kThreads = 256;

// One head row per D/16 lanes; heads 0 .. Hq-1 are queries, Hq .. Hq+Hkv-1 keys.
template <int D>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(Part q, Part k, int Hq, int H, int64_t nheads,
                                                                const int32_t* __restrict__ pos,
                                                                const float2* __restrict__ table, int max_pos,
                                                                float eps) {
  constexpr int LPH = D / 16;
  const int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t th = e / LPH;
  const int j = (int)(e % LPH);
  pdl_wait();  // inputs written by the previous kernel on the stream are complete from here on
  pdl_trigger();
  // lanes past the end redo the last head's work without storing (the butterfly needs whole warps)
  const bool live = th < nheads;
  const int64_t hh = live ? th : nheads - 1;
  const int64_t t = hh / H;
  const int h = (int)(hh - t * H);
  const bool is_q = h < Hq;
  const Part p = is_q ? q : k;
  const int64_t col = (int64_t)(is_q ? h : h - Hq) * D + 8 * j;
  float a[8], b[8];
  unpack8(*reinterpret_cast<const uint4*>(p.x + t * p.ldx + col), a);
  unpack8(*reinterpret_cast<const uint4*>(p.x + t * p.ldx + col + D / 2), b);
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = __fmaf_rn(a[i], a[i], ss);
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = __fmaf_rn(b[i], b[i], ss);
#pragma unroll
  for (int off = LPH / 2; off >= 1; off >>= 1) ss = __fadd_rn(ss, __shfl_xor_sync(kFullMask, ss, off));
  const float r = rsqrtf(__fadd_rn(__fdiv_rn(ss, (float)D), eps));
  const int ps = pos[t];
  if (!live) return;
  if (ps < 0 || ps >= max_pos) {
    if (j == 0) record_error(BI_ERR_DEVICE_INDEX);
    return;
  }
  float wa[8], wb[8], ya[8], yb[8];
  unpack8(__ldg(reinterpret_cast<const uint4*>(p.w + 8 * j)), wa);
  unpack8(__ldg(reinterpret_cast<const uint4*>(p.w + D / 2 + 8 * j)), wb);
  const float4* cs = reinterpret_cast<const float4*>(table + (int64_t)ps * (D / 2) + 8 * j);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 c = __ldg(cs + i);
    const float n0 = __fmul_rn(__fmul_rn(a[2 * i], r), wa[2 * i]), m0 = __fmul_rn(__fmul_rn(b[2 * i], r), wb[2 * i]);
    const float n1 = __fmul_rn(__fmul_rn(a[2 * i + 1], r), wa[2 * i + 1]);
    const float m1 = __fmul_rn(__fmul_rn(b[2 * i + 1], r), wb[2 * i + 1]);
    ya[2 * i] = __fmaf_rn(n0, c.x, -__fmul_rn(m0, c.y));
    yb[2 * i] = __fmaf_rn(m0, c.x, __fmul_rn(n0, c.y));
    ya[2 * i + 1] = __fmaf_rn(n1, c.z, -__fmul_rn(m1, c.w));
    yb[2 * i + 1] = __fmaf_rn(m1, c.z, __fmul_rn(n1, c.w));
  }
  uint16_t* y = p.y + t * p.ldy + col;
  *reinterpret_cast<uint4*>(y) = make_uint4(pack_bf16x2(ya[0], ya[1]), pack_bf16x2(ya[2], ya[3]),
                                            pack_bf16x2(ya[4], ya[5]), pack_bf16x2(ya[6], ya[7]));
  *reinterpret_cast<uint4*>(y + D / 2) = make_uint4(pack_bf16x2(yb[0], yb[1]), pack_bf16x2(yb[2], yb[3]),
                                                    pack_bf16x2(yb[4], yb[5]), pack_bf16x2(yb[6], yb[7]));
}

inline cudaError_t launch(const Part& q, const Part& k, int64_t T, int Hq, int Hkv, int D, const int32_t* pos,
                          const float2* table, int max_pos, float eps, cudaStream_t st) {
  const int64_t nheads = T * (Hq + Hkv);
  const unsigned grid = (unsigned)((nheads * (D / 16) + kThreads - 1) / kThreads);
  switch (D) {
    case 64:
      return launch_pdl(qk_norm_rope_kernel<64>, dim3(grid), dim3(kThreads), 0, st, q, k, Hq, Hq + Hkv, nheads, pos,
                        table, max_pos, eps);
    case 128:
      return launch_pdl(qk_norm_rope_kernel<128>, dim3(grid), dim3(kThreads), 0, st, q, k, Hq, Hq + Hkv, nheads, pos,
                        table, max_pos, eps);
    default:
      return launch_pdl(qk_norm_rope_kernel<256>, dim3(grid), dim3(kThreads), 0, st, q, k, Hq, Hq + Hkv, nheads, pos,
                        table, max_pos, eps);
  }
}

}  // namespace qknorm
}  // namespace bi
