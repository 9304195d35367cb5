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

// D/16 lanes take HPG heads of one token: j, j + J, j + 2 J, ... with J = ceil(H / HPG) groups of
// lanes a token (heads 0 .. Hq-1 are queries, Hq .. H-1 keys), so that the table row and
// the weights are read once for several heads and several heads' loads are in flight.
// groups is T * J.
template <int D, int HPG>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(Part q, Part k, uint32_t Hq, uint32_t H, uint32_t J,
                                                                uint32_t groups, const int32_t* __restrict__ pos,
                                                                const float2* __restrict__ table, int max_pos,
                                                                float eps) {
  constexpr uint32_t LPH = D / 16;
  const uint32_t group = blockIdx.x * (kThreads / LPH) + threadIdx.x / LPH;
  const int j = (int)(threadIdx.x % LPH);
  pdl_wait();  // inputs written by the previous kernel on the stream are complete from here on
  pdl_trigger();
  // lanes past the end redo the last group's work without storing (the butterfly needs whole warps)
  const uint32_t gr = min(group, groups - 1), t = gr / J, h0 = gr - t * J;
  uint4 x[HPG][2];
#pragma unroll
  for (int i = 0; i < HPG; ++i) {
    const uint32_t h = min(h0 + i * J, H - 1);
    const uint16_t* row = h < Hq ? q.x + (int64_t)t * q.ldx + (int64_t)h * D : k.x + (int64_t)t * k.ldx + (int64_t)(h - Hq) * D;
    x[i][0] = *reinterpret_cast<const uint4*>(row + 8 * j);
    x[i][1] = *reinterpret_cast<const uint4*>(row + D / 2 + 8 * j);
  }
  const int ps = pos[t];
  const bool ok = ps >= 0 && ps < max_pos;
  if (group < groups && !ok && j == 0) record_error(BI_ERR_DEVICE_INDEX);
  float4 cs[4];
  const float4* row_cs = reinterpret_cast<const float4*>(table + (int64_t)(ok ? ps : 0) * (D / 2) + 8 * j);
#pragma unroll
  for (int i = 0; i < 4; ++i) cs[i] = __ldg(row_cs + i);
#pragma unroll
  for (int i = 0; i < HPG; ++i) {
    const uint32_t h = h0 + i * J;
    float a[8], b[8];
    unpack8(x[i][0], a);
    unpack8(x[i][1], b);
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = __fmaf_rn(a[e], a[e], ss);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = __fmaf_rn(b[e], b[e], ss);
#pragma unroll
    for (int off = LPH / 2; off >= 1; off >>= 1) ss = __fadd_rn(ss, __shfl_xor_sync(kFullMask, ss, off));
    const float r = rsqrtf(__fadd_rn(__fmul_rn(ss, 1.f / D), eps));  // 1 / D is a power of two
    const bool is_q = h < Hq;
    const uint16_t* w = is_q ? q.w : k.w;
    float wa[8], wb[8], ya[8], yb[8];
    unpack8(__ldg(reinterpret_cast<const uint4*>(w + 8 * j)), wa);
    unpack8(__ldg(reinterpret_cast<const uint4*>(w + D / 2 + 8 * j)), wb);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float c = e & 1 ? cs[e / 2].z : cs[e / 2].x, s = e & 1 ? cs[e / 2].w : cs[e / 2].y;
      const float n = __fmul_rn(__fmul_rn(a[e], r), wa[e]), m = __fmul_rn(__fmul_rn(b[e], r), wb[e]);
      ya[e] = __fmaf_rn(n, c, -__fmul_rn(m, s));
      yb[e] = __fmaf_rn(m, c, __fmul_rn(n, s));
    }
    if (group >= groups || !ok || h >= H) continue;
    uint16_t* y = (is_q ? q.y + (int64_t)t * q.ldy + (int64_t)h * D : k.y + (int64_t)t * k.ldy + (int64_t)(h - Hq) * D) + 8 * j;
    *reinterpret_cast<uint4*>(y) = make_uint4(pack_bf16x2(ya[0], ya[1]), pack_bf16x2(ya[2], ya[3]),
                                              pack_bf16x2(ya[4], ya[5]), pack_bf16x2(ya[6], ya[7]));
    *reinterpret_cast<uint4*>(y + D / 2) = make_uint4(pack_bf16x2(yb[0], yb[1]), pack_bf16x2(yb[2], yb[3]),
                                                      pack_bf16x2(yb[4], yb[5]), pack_bf16x2(yb[6], yb[7]));
  }
}

template <int D, int HPG>
inline cudaError_t launch_hpg(const Part& q, const Part& k, int64_t T, int Hq, int H, const int32_t* pos,
                              const float2* table, int max_pos, float eps, cudaStream_t st) {
  const uint32_t J = (uint32_t)((H + HPG - 1) / HPG), groups = (uint32_t)(T * J);
  constexpr uint32_t per = kThreads / (D / 16);
  return launch_pdl(qk_norm_rope_kernel<D, HPG>, dim3(groups / per + (groups % per != 0)), dim3(kThreads), 0, st, q, k,
                    (uint32_t)Hq, (uint32_t)H, J, groups, pos, table, max_pos, eps);
}

// Four heads a group of lanes once one head each would give the SMs more than twice the threads
// they hold; below that more, shorter threads finish as soon or sooner. 32 + 8 heads of 128, one
// head against four: 64 rows 2.7 us and 3.4, 577 rows 4.6 and 4.4, 4096 rows 19.4 and 13.8, 32768
// rows 164 and 117 (671 MB: 5.7 TB/s).
template <int D>
inline cudaError_t launch_d(const Part& q, const Part& k, int64_t T, int Hq, int H, const int32_t* pos, const float2* table,
                            int max_pos, float eps, int sms, cudaStream_t st) {
  return T * H * (D / 16) > (int64_t)sms * 4096 ? launch_hpg<D, 4>(q, k, T, Hq, H, pos, table, max_pos, eps, st)
                                                : launch_hpg<D, 1>(q, k, T, Hq, H, pos, table, max_pos, eps, st);
}

inline cudaError_t launch(const Part& q, const Part& k, int64_t T, int Hq, int Hkv, int D, const int32_t* pos,
                          const float2* table, int max_pos, float eps, int sms, cudaStream_t st) {
  switch (D) {
    case 64: return launch_d<64>(q, k, T, Hq, Hq + Hkv, pos, table, max_pos, eps, sms, st);
    case 128: return launch_d<128>(q, k, T, Hq, Hq + Hkv, pos, table, max_pos, eps, sms, st);
    default: return launch_d<256>(q, k, T, Hq, Hq + Hkv, pos, table, max_pos, eps, sms, st);
  }
}

}  // namespace qknorm
}  // namespace bi
