// Attention over the 8-bit paged store (decode rows, and prefill rows with the same bits).
//
// For a query row (one token, one head) with visible keys 0 .. L-1 of its sequence:
//   s_t = scale q . (k_t sk_t),  out = sum_t e^(s_t) v_t sv_t / sum_t e^(s_t).
// In the base-2 domain with z_t = s_t log2 e + log2 sv_t and w_t = 2^(z_t - max z):
//   out = sum_t w_t v_t / sum_t (w_t / sv_t),
// so the value scale rides in the exponent, w_t lies in [0, 1] however far apart the rows'
// scales are, and both sums use the same w_t (an error of log2 sv_t is a common factor of a
// token's two terms).
//
// The products run on mma.sync m16n8k16 (f16 operands, fp32 sums). 8-bit keys and values are
// exact in f16. A query row is brought to |q| < 2^15 by a power of two (exact but for dims
// 2^28 below the row's largest, which lose bits below 2^-39 of it); 2^14 w_t is rounded to f16
// (half a step 2^-12 relative, and 2^-39 of the largest weight below 2^-28 of it), a finer
// rounding than the bf16 output's 2^-9. All sums and the softmax statistics are fp32.
// mma.sync takes its operands from registers, which is what this read pattern needs: decode
// has 1 to 16 query rows per kv-head, one MMA tile, and the 8-bit bytes go from HBM into the
// lane that widens them without a stop in shared memory.
//
// Per-row schedule (a function of the row's own L only, so decode, whole and chunked prefill,
// and any batch give the same bits):
//   * keys are cut into splits at absolute positions 0, 256, 512, ...; a split is folded page
//     by page (16 tokens, one MMA k-step of weights x values) with a running maximum;
//   * s_t is one chain of D/16 MMAs, dims in a fixed order; a lane sums its 4 tokens' w / sv of
//     each page in order, and the 4 lanes of a row are added by an xor tree at the split's end;
//   * splits are folded in ascending order: M' = max(M, m_s), X = X 2^(M-M') + x_s 2^(m_s-M').
// An MMA's output row depends on its own A row only, so it does not matter which rows share
// a tile. Tokens a row does not see get w = 0 exactly and stale value bytes are replaced by
// zeros; rows that see nothing give zeros.
#pragma once

#include "attention.cuh"
#include "kv_q8.cuh"

namespace bi {
namespace attnq8 {

using attn::PAGE;
using attn::PAGES_PER_SPLIT;
using attn::Rows;
using attn::SPLIT;

struct Cache {
  const uint8_t* k;
  const uint8_t* v;
  const float* ks;
  const float* vs;
  int64_t num_pages;
  const int32_t* pt;
};

// 2^x with results below 2^-126 flushed to 0 (they are under 2^-112 of the largest weight's 2^14).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Value scales are at least 2^-109, so neither they nor their reciprocals are flushed.
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint4 ldg16(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// d += A B with A 16 x 16 (rows = query rows), B 16 x 8, f16 operands.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The 8-bit values at bytes 0, 1 (lo) and 2, 3 (hi) of w as f16 pairs, exactly. int8: the
// byte v ^ 0x80 = v + 128 under the exponent byte 0x64 is the f16 number 1024 + v + 128.
template <int KIND>
__device__ __forceinline__ void widen(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (KIND == BI_KV_INT8) {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
    const uint32_t l = __byte_perm(u, 0x64646464u, 0x4140), h = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 dl = __hsub2(*reinterpret_cast<const __half2*>(&l), bias);
    const __half2 dh = __hsub2(*reinterpret_cast<const __half2*>(&h), bias);
    lo = *reinterpret_cast<const uint32_t*>(&dl);
    hi = *reinterpret_cast<const uint32_t*>(&dh);
  } else {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

// Lane layout (g = lane / 4, c = lane % 4, as in an MMA fragment):
//   queries: MMA rows g and g + 8; MMA step j covers dims 64 (j/4) + 16 c + 4 (j%4) + 0..3 of lane c;
//   keys: MMA column g of n-tile i is token 8 i + g; the lane loads dims 64 v + 16 c .. + 15;
//   scores: the lane holds tokens 2c, 2c+1, 2c+8, 2c+9 of rows g and g + 8, which is the A
//     fragment of weights x values as it stands;
//   values: the lane loads those four tokens' dims (D/8) g .. + D/8 - 1; MMA column g of n-tile i
//     is dim (D/8) g + i, so it holds output dims (D/4) c .. + D/4 - 1 of rows g and g + 8.
template <int D>
struct Page {
  uint4 k[2][D / 64];
  uint32_t v[4][D / 32];
  float ks[4], vs[4];  // of tokens 2c, 2c+1, 2c+8, 2c+9
};

template <int D>
__device__ __forceinline__ void load_page(Page<D>& P, const Cache& C, int64_t row0, int g, int c) {
  const uint8_t* kp = C.k + (row0 + g) * D + 16 * c;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int v = 0; v < D / 64; ++v) P.k[i][v] = ldg16(kp + i * 8 * D + 64 * v);
  const uint8_t* vp = C.v + (row0 + 2 * c) * D + (D / 8) * g;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint8_t* p = vp + ((i & 1) + (i >> 1) * 8) * D;
    if constexpr (D == 128) {
      const uint4 x = ldg16(p);
      P.v[i][0] = x.x; P.v[i][1] = x.y; P.v[i][2] = x.z; P.v[i][3] = x.w;
    } else {
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
      P.v[i][0] = x.x; P.v[i][1] = x.y;
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = __ldg(reinterpret_cast<const float2*>(C.ks + row0 + 8 * i + 2 * c));
    const float2 b = __ldg(reinterpret_cast<const float2*>(C.vs + row0 + 8 * i + 2 * c));
    P.ks[2 * i] = a.x; P.ks[2 * i + 1] = a.y;
    P.vs[2 * i] = b.x; P.vs[2 * i + 1] = b.y;
  }
}

// Query rows in A-fragment order. RH = 1: MMA rows 8 .. 15 are empty (groups of up to 8 heads).
template <int D, int RH>
struct Query {
  uint32_t a[D / 16][2 * RH];  // step j: (row g: dims +0,1 | +2,3), then row g + 8
  float c[RH];                 // scale log2(e) / the row's power of two; NaN if the row is not finite
};

// Loads one query row (nullptr: zeros) into half `r` of the fragment. All lanes of the warp call it.
template <int D, int RH>
__device__ __forceinline__ void load_query(Query<D, RH>& Q, int r, const uint16_t* row, int c, float scale_log2) {
  uint4 x[D / 64][2];
  uint32_t m = 0;
#pragma unroll
  for (int v = 0; v < D / 64; ++v)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[v][i] = row ? __ldg(reinterpret_cast<const uint4*>(row + 64 * v + 16 * c + 8 * i)) : make_uint4(0, 0, 0, 0);
      const uint32_t w[4] = {x[v][i].x, x[v][i].y, x[v][i].z, x[v][i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) m = max(m, max(w[e] & 0x7FFFu, (w[e] >> 16) & 0x7FFFu));
    }
  m = max(m, __shfl_xor_sync(kFullMask, m, 1));
  m = max(m, __shfl_xor_sync(kFullMask, m, 2));
  const int e = max((int)(m >> 7) - 127, -100);  // |q| < 2^(e+1); rows below 2^-100 are not scaled further
  const bool finite = m < kvq8::kNonFiniteBits;
  const float up = __uint_as_float((uint32_t)(127 + 14 - (finite ? e : 14)) << 23);
  const float down = __uint_as_float((uint32_t)(127 - 14 + (finite ? e : 14)) << 23);
  Q.c[r] = finite ? __fmul_rn(scale_log2, down) : __uint_as_float(0x7FC00000u);
#pragma unroll
  for (int j = 0; j < D / 16; ++j) {
    // 4 dims: elements 4 (j%4) .. + 3 of the 16 in x[j/4]
    const uint4 q = x[j / 4][(j % 4) / 2];
    const uint32_t w0 = (j & 1) ? q.z : q.x, w1 = (j & 1) ? q.w : q.y;
    Q.a[j][2 * r] = pack_f16x2(__fmul_rn(bf16lo(w0), up), __fmul_rn(bf16hi(w0), up));
    Q.a[j][2 * r + 1] = pack_f16x2(__fmul_rn(bf16lo(w1), up), __fmul_rn(bf16hi(w1), up));
  }
}

// Running state of a split: per row the maximum z, 2^14 sum w / sv over the lane's tokens,
// and 2^14 sum w v over the lane's output dims (pairs of rows g, g + 8 as the MMA gives them).
template <int D, int RH>
struct State {
  float m[RH], l[RH];
  float o[D / 8][2 * RH];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int r = 0; r < RH; ++r) m[r] = -INFINITY, l[r] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int e = 0; e < 2 * RH; ++e) o[i][e] = 0.f;
  }
};

template <int RH>
__device__ __forceinline__ void mma_rows(float (&d)[2 * RH], const uint32_t (&a)[2 * RH], uint32_t b0, uint32_t b1) {
  if constexpr (RH == 2) {
    const uint32_t A[4] = {a[0], a[2], a[1], a[3]};
    mma16816(d, A, b0, b1);
  } else {
    const uint32_t A[4] = {a[0], 0u, a[1], 0u};
    float t[4] = {d[0], d[1], 0.f, 0.f};
    mma16816(t, A, b0, b1);
    d[0] = t[0];
    d[1] = t[1];
  }
}

// Scores of one page: s[i] covers tokens 8 i + 2c, + 1 of row g (then of row g + 8).
template <int KIND, int D, int RH>
__device__ __forceinline__ void page_scores(const Query<D, RH>& Q, const Page<D>& P, float (&s)[2][2 * RH]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int e = 0; e < 2 * RH; ++e) s[i][e] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      const uint4 x = P.k[i][j / 4];
      const uint32_t w = (j % 4) == 0 ? x.x : (j % 4) == 1 ? x.y : (j % 4) == 2 ? x.z : x.w;
      uint32_t b0, b1;
      widen<KIND>(w, b0, b1);
      mma_rows<RH>(s[i], Q.a[j], b0, b1);
    }
  }
}

// Weights of one page from its scores: updates m, l and o's scaling, and gives 2^14 w as the
// A fragment of the value product. lg, ri: log2 and reciprocal of the lane's four tokens'
// value scales. MASKED: row half r sees the first nv[r] tokens only; otherwise all 16.
template <int D, int RH, bool MASKED>
__device__ __forceinline__ void page_weights(const Query<D, RH>& Q, const float (&s)[2][2 * RH], const float (&ks)[4],
                                             const float (&lg)[4], const float (&ri)[4], const int (&nv)[RH], int c,
                                             State<D, RH>& S, uint32_t (&w)[2 * RH]) {
  float z[RH][4];
  float alpha[RH];
  bool moved = false;
#pragma unroll
  for (int r = 0; r < RH; ++r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[r][i] = __fmaf_rn(s[i >> 1][2 * r + (i & 1)], __fmul_rn(ks[i], Q.c[r]), lg[i]);
      if (MASKED && 8 * (i >> 1) + 2 * c + (i & 1) >= nv[r]) z[r][i] = -INFINITY;
    }
    float mx = fmaxf(fmaxf(z[r][0], z[r][1]), fmaxf(z[r][2], z[r][3]));
    mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, 2));
    const float mn = fmaxf(S.m[r], mx);
    alpha[r] = mn == S.m[r] ? 1.f : ex2(__fsub_rn(S.m[r], mn));
    moved |= mn != S.m[r];
    S.m[r] = mn;
  }
  if (__any_sync(kFullMask, moved)) {  // x * 1 == x, so rows whose maximum stayed keep their bits
#pragma unroll
    for (int r = 0; r < RH; ++r) {
      S.l[r] = __fmul_rn(S.l[r], alpha[r]);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        S.o[i][2 * r] = __fmul_rn(S.o[i][2 * r], alpha[r]);
        S.o[i][2 * r + 1] = __fmul_rn(S.o[i][2 * r + 1], alpha[r]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < RH; ++r) {
    const float ref = S.m[r] == -INFINITY ? 0.f : __fsub_rn(S.m[r], 14.f);
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i] = ex2(__fsub_rn(z[r][i], ref));
      if (!MASKED || 8 * (i >> 1) + 2 * c + (i & 1) < nv[r]) S.l[r] = __fmaf_rn(p[i], ri[i], S.l[r]);
    }
    w[2 * r] = pack_f16x2(p[0], p[1]);
    w[2 * r + 1] = pack_f16x2(p[2], p[3]);
  }
}

// o += weights x values of one page. `seen`: tokens from there on are replaced by zeros.
template <int KIND, int D, int RH, bool MASKED>
__device__ __forceinline__ void page_values(const Page<D>& P, const uint32_t (&w)[2 * RH], int seen, int c,
                                            State<D, RH>& S) {
#pragma unroll
  for (int u = 0; u < D / 32; ++u) {
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = P.v[i][u];
      if (MASKED && 8 * (i >> 1) + 2 * c + (i & 1) >= seen) x[i] = 0;
    }
    // bytes (token 2c, token 2c+1) of dims 4u, 4u+1 | 4u+2, 4u+3, and the same of tokens 2c+8, 2c+9
    const uint32_t a0 = __byte_perm(x[0], x[1], 0x5140), a1 = __byte_perm(x[0], x[1], 0x7362);
    const uint32_t b0 = __byte_perm(x[2], x[3], 0x5140), b1 = __byte_perm(x[2], x[3], 0x7362);
    uint32_t f0, f1, f2, f3, h0, h1, h2, h3;
    widen<KIND>(a0, f0, f1);
    widen<KIND>(a1, f2, f3);
    widen<KIND>(b0, h0, h1);
    widen<KIND>(b1, h2, h3);
    mma_rows<RH>(S.o[4 * u], w, f0, h0);
    mma_rows<RH>(S.o[4 * u + 1], w, f1, h1);
    mma_rows<RH>(S.o[4 * u + 2], w, f2, h2);
    mma_rows<RH>(S.o[4 * u + 3], w, f3, h3);
  }
}

// Folds one page of which `seen` tokens exist for the tile and nv[r] for row half r.
template <int KIND, int D, int RH>
__device__ __forceinline__ void fold_page(const Query<D, RH>& Q, const Page<D>& P, const int (&nv)[RH], int seen, int c,
                                          State<D, RH>& S) {
  float s[2][2 * RH], lg[4], ri[4];
  uint32_t w[2 * RH];
  page_scores<KIND, D, RH>(Q, P, s);
#pragma unroll
  for (int i = 0; i < 4; ++i) lg[i] = lg2(P.vs[i]), ri[i] = rcp(P.vs[i]);
  bool all = true;
#pragma unroll
  for (int r = 0; r < RH; ++r) all &= nv[r] >= PAGE;
  if (__all_sync(kFullMask, all)) {
    page_weights<D, RH, false>(Q, s, P.ks, lg, ri, nv, c, S, w);
    page_values<KIND, D, RH, false>(P, w, seen, c, S);
  } else {
    page_weights<D, RH, true>(Q, s, P.ks, lg, ri, nv, c, S, w);
    page_values<KIND, D, RH, true>(P, w, seen, c, S);
  }
}

// The xor tree over a row's 4 lanes that ends a split.
__device__ __forceinline__ float row_sum(float l) {
  l = __fadd_rn(l, __shfl_xor_sync(kFullMask, l, 1));
  return __fadd_rn(l, __shfl_xor_sync(kFullMask, l, 2));
}

// One step of the fold over splits: (M, L, O) and split (m, l, o) -> weights of both.
__device__ __forceinline__ void join(float& M, float m, float& a, float& b) {
  const float mn = fmaxf(M, m);
  const float ref = mn == -INFINITY ? 0.f : mn;
  a = ex2(__fsub_rn(M, ref));
  b = ex2(__fsub_rn(m, ref));
  M = mn;
}

// ---------------------------------------------------------------------------
// Decode: one warp per (row, kv-head, split); the split's partial result goes to the workspace.
//
// Bound: HBM (4 (2 D + 8) L Hkv flops-free bytes per row against 4 L Hq D flops). Each lane
// copies the bytes that it will itself widen into its own places of a ring in shared memory
// (cp.async, 16 bytes each), kStages pages ahead across item boundaries, so that nothing but
// the 32 scales of a page crosses lanes and no barrier beyond the warp's is needed; a warp's
// reads back are contiguous, without bank conflicts.

constexpr int kWarps = 4;
constexpr int kStages = 4;
constexpr int kCoarse = 1024;  // entries of the split-count prefix that a CTA keeps

template <int D>
struct Ring {
  static constexpr int K_BYTES = PAGE * D;         // [n-tile][64-dim part][lane] 16 bytes
  static constexpr int V_BYTES = PAGE * D;         // [token of the lane's four][lane] D/8 bytes
  static constexpr int STAGE = K_BYTES + V_BYTES + 2 * PAGE * 4;  // and the page's scales
  static constexpr int WARP = kStages * STAGE;
  static constexpr int SMEM = kWarps * WARP + (kCoarse + 1) * 4;
};

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Starts the copies of one page (store rows row0 .. row0 + 15) into a ring stage.
template <int D>
__device__ __forceinline__ void copy_page(uint32_t stage, const Cache& C, int64_t row0, int lane) {
  using T = Ring<D>;
  const int g = lane >> 2, c = lane & 3;
  const uint8_t* kp = C.k + (row0 + g) * D + 16 * c;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int v = 0; v < D / 64; ++v)
      cp_async<16>(stage + ((i * (D / 64) + v) * 32 + lane) * 16, kp + i * 8 * D + 64 * v);
  const uint8_t* vp = C.v + (row0 + 2 * c) * D + (D / 8) * g;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    cp_async<D / 8>(stage + T::K_BYTES + (i * 32 + lane) * (D / 8), vp + ((i & 1) + (i >> 1) * 8) * D);
  if (lane < 8)
    cp_async<16>(stage + T::K_BYTES + T::V_BYTES + 16 * lane, (lane < 4 ? C.ks + row0 : C.vs + row0 - 16) + 4 * lane);
}

// The lane's part of a page from its ring stage.
template <int D>
__device__ __forceinline__ void read_page(Page<D>& P, uint32_t stage, int lane) {
  using T = Ring<D>;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int v = 0; v < D / 64; ++v) P.k[i][v] = ld_shared_v4(stage + ((i * (D / 64) + v) * 32 + lane) * 16);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = stage + T::K_BYTES + (i * 32 + lane) * (D / 8);
    if constexpr (D == 128) {
      const uint4 x = ld_shared_v4(a);
      P.v[i][0] = x.x; P.v[i][1] = x.y; P.v[i][2] = x.z; P.v[i][3] = x.w;
    } else {
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(P.v[i][0]), "=r"(P.v[i][1]) : "r"(a));
    }
  }
  const uint32_t sc = stage + T::K_BYTES + T::V_BYTES + 8 * (lane & 3);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(P.ks[2 * i]), "=f"(P.ks[2 * i + 1]) : "r"(sc + 32 * i));
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(P.vs[2 * i]), "=f"(P.vs[2 * i + 1]) : "r"(sc + 64 + 32 * i));
  }
}

// A work item: split s of row r for one kv-head; `page` is page `lane` of it (-1: unusable).
struct Item {
  int r, s, kh, seen, page;
};

template <int KIND, int D, int RH>
__global__ void __launch_bounds__(kWarps * 32, D == 128 ? 3 : 4)
    split_kernel(const uint16_t* __restrict__ q, int Hq, int Hkv, Cache C, Rows R, int nrows, int max_splits,
                 float* __restrict__ po, float2* __restrict__ pml, float scale_log2) {
  using T = Ring<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int32_t warp_sum[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int G = Hq / Hkv;
  int32_t* pre = reinterpret_cast<int32_t*>(smem + kWarps * T::WARP);  // pre[i]: splits of rows below i * per
  pdl_wait();  // the caller's inputs are complete from here on
  pdl_trigger();

  // the prefix of split counts, `per` rows an entry (1 up to kCoarse rows)
  const int per = (nrows + kCoarse - 1) / kCoarse, entries = (nrows + per - 1) / per;
  int base = 0;
  for (int e0 = 0; e0 < entries; e0 += kWarps * 32) {
    const int e = e0 + (int)threadIdx.x;
    int n = 0;
    if (e < entries)
      for (int r = e * per; r < min(nrows, (e + 1) * per); ++r) n += attn::num_splits(R, r);
    int x = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(kFullMask, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int before = base;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += warp_sum[w];
      base += warp_sum[w];
    }
    if (e < entries) pre[e] = before + x - n;
    __syncthreads();
  }
  const int total = base * Hkv;
  const int step = (int)gridDim.x * kWarps;

  auto fetch = [&](int item) {
    Item I;
    const int f = item / Hkv;
    I.kh = item - f * Hkv;
    int lo = 0, hi = entries;  // pre[lo] <= f < pre[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= f) lo = mid;
      else hi = mid;
    }
    I.s = f - pre[lo];
    I.r = lo * per;
    while (per > 1) {
      const int n = attn::num_splits(R, I.r);
      if (I.s < n) break;
      I.s -= n;
      ++I.r;
    }
    int pt_row;
    const int len = attn::row_len(R, I.r, pt_row);
    I.seen = min(SPLIT, len - I.s * SPLIT);
    I.page = -1;
    if (lane * PAGE < I.seen) {
      const int pg = C.pt[(int64_t)pt_row * R.max_pages + I.s * PAGES_PER_SPLIT + lane];
      if (pg >= 0 && pg < C.num_pages) I.page = pg;
      else record_error(BI_ERR_DEVICE_INDEX);
    }
    return I;
  };

  const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * T::WARP);
  int item = warp * (int)gridDim.x + (int)blockIdx.x;
  if (item >= total) return;
  Item cur = fetch(item), nxt = cur;
  bool ahead = false;            // the copies have gone on to nxt
  int pj = 0, issued = 0, used = 0;
  // starts the copy of the next page of the item stream, if it is known by now
  auto issue = [&] {
    if (!ahead && pj * PAGE >= cur.seen && item + step < total) {
      nxt = fetch(item + step);
      ahead = true;
      pj = 0;
    }
    const Item& I = ahead ? nxt : cur;
    if (pj * PAGE < I.seen) {
      const int pg = __shfl_sync(kFullMask, I.page, pj);
      if (pg >= 0) copy_page<D>(ring + (uint32_t)(issued % kStages) * T::STAGE, C, ((int64_t)pg * Hkv + I.kh) * PAGE, lane);
      ++pj;
      ++issued;
    }
    cp_commit();
  };
  for (int i = 0; i < kStages; ++i) issue();

  while (true) {
    Query<D, RH> Q;
#pragma unroll
    for (int h = 0; h < RH; ++h) {
      const int head = g + 8 * h;
      load_query<D, RH>(Q, h, head < G ? q + ((int64_t)cur.r * Hq + cur.kh * G + head) * D : nullptr, c, scale_log2);
    }
    State<D, RH> S;
    S.clear();
    for (int j = 0; j * PAGE < cur.seen; ++j) {
      // with the ring full the oldest copy group is the page wanted; otherwise (the stream's end,
      // or an item of few pages) wait for all of them
      if (issued - used == kStages) cp_wait<kStages - 1>();
      else cp_wait<0>();
      __syncwarp();
      if (__shfl_sync(kFullMask, cur.page, j) >= 0) {  // the tokens of an unusable page are not seen
        Page<D> P;
        read_page<D>(P, ring + (uint32_t)(used % kStages) * T::STAGE, lane);
        int nv[RH];
#pragma unroll
        for (int h = 0; h < RH; ++h) nv[h] = cur.seen - j * PAGE;
        fold_page<KIND, D, RH>(Q, P, nv, nv[0], c, S);
      }
      ++used;
      __syncwarp();  // every lane has read this page's scales: its stage may be refilled
      issue();
    }
#pragma unroll
    for (int h = 0; h < RH; ++h) {
      const float l = row_sum(S.l[h]);
      const int head = g + 8 * h;
      if (head >= G) continue;
      const int64_t slot = ((int64_t)cur.r * max_splits + cur.s) * Hq + cur.kh * G + head;
      float* dst = po + slot * D + (D / 4) * c;
#pragma unroll
      for (int i = 0; i < D / 8; i += 4) {
        *reinterpret_cast<float4*>(dst + i) =
            make_float4(S.o[i][2 * h], S.o[i + 1][2 * h], S.o[i + 2][2 * h], S.o[i + 3][2 * h]);
        *reinterpret_cast<float4*>(dst + D / 8 + i) =
            make_float4(S.o[i][2 * h + 1], S.o[i + 1][2 * h + 1], S.o[i + 2][2 * h + 1], S.o[i + 3][2 * h + 1]);
      }
      if (c == 0) pml[slot] = make_float2(S.m[h], l);
    }
    if (item + step >= total) break;
    item += step;
    if (!ahead) {  // nothing of the next item has been asked for yet
      cur = fetch(item);
      pj = 0;
    } else {
      cur = nxt;
      ahead = false;
    }
    for (int i = issued - used; i < kStages; ++i) issue();  // short items left the ring less than full
  }
}

// Folds a row's splits in ascending order; one warp per (row, query head, 32 * DPL output dims).
// The lanes take the splits' maxima 32 at a time: the running maximum before and after each
// split (a maximum is exact in any order) gives the weights of both sides of its fold step, and
// the fold itself is one chain per output dim in split order whatever DPL is. Partials are
// loaded U at a time.
template <int D, int DPL>
__global__ void __launch_bounds__(256) combine_kernel(const float* __restrict__ po, const float2* __restrict__ pml,
                                                      Rows R, int nrows, int max_splits, int Hq,
                                                      uint16_t* __restrict__ out) {
  constexpr int NG = D / (32 * DPL);  // warps per (row, head)
  constexpr int U = DPL == 1 ? 16 : 8;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  pdl_wait();  // the split partials are complete from here on
  pdl_trigger();
  if (w >= (int64_t)nrows * Hq * NG) return;
  const int64_t rh = w / NG;
  const int r = (int)(rh / Hq), h = (int)(rh - (int64_t)r * Hq);
  const int d0 = ((int)(w - rh * NG) * 32 + lane) * DPL;
  const int n = attn::num_splits(R, r);
  const int64_t slot0 = (int64_t)r * max_splits * Hq + h;
  const float* src = po + slot0 * D + d0;
  float M = -INFINITY, L = 0.f, O[DPL];
#pragma unroll
  for (int d = 0; d < DPL; ++d) O[d] = 0.f;
  for (int s0 = 0; s0 < n; s0 += 32) {
    const float2 ml = s0 + lane < n ? pml[slot0 + (int64_t)(s0 + lane) * Hq] : make_float2(-INFINITY, 0.f);
    float top = ml.x;  // the running maximum up to and with this lane's split
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const float y = __shfl_up_sync(kFullMask, top, d);
      if (lane >= d) top = fmaxf(top, y);
    }
    top = fmaxf(top, M);
    float prev = __shfl_up_sync(kFullMask, top, 1);
    if (lane == 0) prev = M;
    float a, b;
    join(prev, ml.x, a, b);
    M = __shfl_sync(kFullMask, top, 31);
    const int cnt = min(32, n - s0);
    for (int u0 = 0; u0 < cnt; u0 += U) {
      float v[U][DPL];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float* p = src + (int64_t)(s0 + min(u0 + u, cnt - 1)) * Hq * D;
        if constexpr (DPL == 4) {
          const float4 x = *reinterpret_cast<const float4*>(p);
          v[u][0] = x.x; v[u][1] = x.y; v[u][2] = x.z; v[u][3] = x.w;
        } else if constexpr (DPL == 2) {
          const float2 x = *reinterpret_cast<const float2*>(p);
          v[u][0] = x.x; v[u][1] = x.y;
        } else {
          v[u][0] = *p;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float ak = __shfl_sync(kFullMask, a, (u0 + u) & 31), bk = __shfl_sync(kFullMask, b, (u0 + u) & 31);
        const float lk = __shfl_sync(kFullMask, ml.y, (u0 + u) & 31);
        if (u0 + u < cnt) {
          L = __fmaf_rn(lk, bk, __fmul_rn(L, ak));
#pragma unroll
          for (int d = 0; d < DPL; ++d) O[d] = __fmaf_rn(v[u][d], bk, __fmul_rn(O[d], ak));
        }
      }
    }
  }
  float y[DPL];
#pragma unroll
  for (int d = 0; d < DPL; ++d) y[d] = L == 0.f ? 0.f : __fdiv_rn(O[d], L);
  uint16_t* dst = out + rh * D + d0;
  if constexpr (DPL == 1) {
    *dst = to_bf16_bits(y[0]);
  } else {
#pragma unroll
    for (int d = 0; d < DPL; d += 2) reinterpret_cast<uint32_t*>(dst)[d / 2] = pack_bf16x2(y[d], y[d + 1]);
  }
}

// ---------------------------------------------------------------------------
// Prefill: query rows of one sequence are taken in tiles of up to 16 MMA rows.

// A tile: rows first .. first + n - 1 (one sequence), the longest of their visible lengths.
struct Tile {
  int first, n, pt_row, len;
};

// tiles[0 .. *count - 1] over T rows: runs of rows of one sequence cut into tiles of `per`
// rows. One CTA of 1024 threads, each owning a contiguous stretch of rows.
__global__ void __launch_bounds__(1024) plan_kernel(Rows R, int T, int per, Tile* __restrict__ tiles,
                                                    int32_t* __restrict__ count) {
  __shared__ int32_t start[1024], sums[1024];
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  const int each = (T + 1023) / 1024;
  const int r0 = min(tid * each, T), r1 = min(r0 + each, T);
  // the start of the run that row r0 - 1 lies in, from the running maximum of run starts
  int last = -1;
  for (int r = r0; r < r1; ++r)
    if (r == 0 || R.q_seq[r] != R.q_seq[r - 1]) last = r;
  start[tid] = last;
  __syncthreads();
  for (int d = 1; d < 1024; d <<= 1) {
    const int v = tid >= d ? start[tid - d] : -1;
    __syncthreads();
    start[tid] = max(start[tid], v);
    __syncthreads();
  }
  const int before = tid ? start[tid - 1] : -1;
  int run = before, local = 0;
  for (int r = r0; r < r1; ++r) {
    if (r == 0 || R.q_seq[r] != R.q_seq[r - 1]) run = r;
    local += (r - run) % per == 0;
  }
  sums[tid] = local;
  __syncthreads();
  for (int d = 1; d < 1024; d <<= 1) {
    const int v = tid >= d ? sums[tid - d] : 0;
    __syncthreads();
    sums[tid] += v;
    __syncthreads();
  }
  int at = sums[tid] - local;
  run = before;
  for (int r = r0; r < r1; ++r) {
    if (r == 0 || R.q_seq[r] != R.q_seq[r - 1]) run = r;
    if ((r - run) % per) continue;
    Tile t{r, 0, 0, 0};
    while (t.n < per && r + t.n < T && R.q_seq[r + t.n] == R.q_seq[r]) {
      int pt_row;
      const int len = attn::row_len(R, r + t.n, pt_row);
      if (len > t.len) t.len = len, t.pt_row = pt_row;
      ++t.n;
    }
    tiles[at++] = t;
  }
  if (tid == 1023) *count = sums[1023];
}

constexpr int kTileWarps = 4;

template <int D>
constexpr int tile_smem_bytes() {
  return kTileWarps * 16 * D * 4;
}

// One warp per (tile, kv-head): MMA row i is query head i % G of token i / G. Splits are folded
// into running totals in shared memory (one float per lane, row half and output dim).
template <int KIND, int D>
__global__ void __launch_bounds__(kTileWarps * 32) tile_kernel(const uint16_t* __restrict__ q, int64_t ldq, int Hq, int Hkv, Cache C,
                                                               Rows R, const Tile* __restrict__ tiles,
                                                               const int32_t* __restrict__ count,
                                                               uint16_t* __restrict__ out, float scale_log2) {
  extern __shared__ float totals[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int G = Hq / Hkv;
  float* tot = totals + warp * 16 * D + lane;  // entry i at tot[32 i]
  pdl_wait();  // the plan (and the caller's q and store) are complete from here on
  pdl_trigger();
  const int64_t total = (int64_t)*count * Hkv;
  for (int64_t item = total - 1 - ((int64_t)warp * gridDim.x + blockIdx.x); item >= 0;
       item -= (int64_t)gridDim.x * kTileWarps) {
    const Tile t = tiles[item / Hkv];
    const int kh = (int)(item % Hkv);
    Query<D, 2> Q;
    int len[2];
    int64_t orow[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = g + 8 * h, tok = i / G, head = kh * G + i % G;
      const bool live = tok < t.n;
      int pt_row;
      len[h] = live ? attn::row_len(R, t.first + tok, pt_row) : 0;
      orow[h] = live ? ((int64_t)(t.first + tok) * Hq + head) * D : -1;
      load_query<D, 2>(Q, h, live ? q + (int64_t)(t.first + tok) * ldq + (int64_t)head * D : nullptr, c, scale_log2);
    }
    float M[2] = {-INFINITY, -INFINITY}, L[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 2; ++i) tot[32 * i] = 0.f;
    const int32_t* prow = C.pt + (int64_t)t.pt_row * R.max_pages;
    for (int t0 = 0; t0 < t.len; t0 += SPLIT) {
      State<D, 2> S;
      S.clear();
      const int t1 = min(t0 + SPLIT, t.len);
      for (int tp = t0; tp < t1; tp += PAGE) {
        const int pg = prow[tp / PAGE];
        if (pg < 0 || pg >= C.num_pages) {
          if (lane == 0) record_error(BI_ERR_DEVICE_INDEX);
          continue;
        }
        Page<D> P;
        load_page<D>(P, C, ((int64_t)pg * Hkv + kh) * PAGE, g, c);
        const int nv[2] = {len[0] - tp, len[1] - tp};
        fold_page<KIND, D, 2>(Q, P, nv, t.len - tp, c, S);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float a, b;
        const float l = row_sum(S.l[h]);
        join(M[h], S.m[h], a, b);
        L[h] = __fmaf_rn(l, b, __fmul_rn(L[h], a));
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float* x = tot + 32 * (4 * i + 2 * h + e);
            *x = __fmaf_rn(S.o[i][2 * h + e], b, __fmul_rn(*x, a));
          }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (orow[h] < 0) continue;
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < D / 8; i += 8) {
          float y[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const float x = tot[32 * (4 * (i + u) + 2 * h + e)];
            y[u] = L[h] == 0.f ? 0.f : __fdiv_rn(x, L[h]);
          }
          *reinterpret_cast<uint4*>(out + orow[h] + (D / 4) * c + e * (D / 8) + i) =
              make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                         pack_bf16x2(y[6], y[7]));
        }
    }
  }
}

}  // namespace attnq8
}  // namespace bi
