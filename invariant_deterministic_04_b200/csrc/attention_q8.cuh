// Attention over the 8-bit paged store (decode rows, and prefill rows with the same bits).
//
// For a query row (one token, one head) with visible keys 0 .. L-1 of its sequence:
//   s_t = scale q . (k_t sk_t),  out = sum_t e^(s_t) v_t sv_t / sum_t e^(s_t).
// In the base-2 domain with z_t = s_t log2 e, any m and any F > 0:
//   p_t = 2^(z_t - m),  l = sum_t p_t,  w_t = p_t F sv_t,  out = sum_t w_t v_t / (F l).
// m is the softmax's reference and follows the running maximum of z; F is the value product's and
// follows 2^7 / max (p_t sv_t), so the largest weight is near 2^7 whatever the rows' scales are. The two
// are apart because the token that carries the softmax and the one whose w is largest need not be the
// same: with one reference over z_t + log2 sv_t (and l summing w_t / sv_t) a faint row's share of l
// left fp32's range beside a loud row's w. Both follow lazily: they move, m to the maximum and F to
// 2^7 over it, when a w passes 2^15 or a lane's l 2^24, so most pages need neither a reduction over
// lanes nor a rescaling of the sums. A value row of zeros is stored with scale 1 and gives nothing to the
// value product: F passes it over (kNoScale), else a null token that holds much of the weight would
// leave the other rows' weights f16's last bits. Weights below 2^-126 of the row's largest p are zeros, and
// so are weights whose p_t sv_t is below 2^-146 times that.
//
// The products run on mma.sync m16n8k16 (f16 operands, fp32 sums), keys and values as the
// 16-row operand, 8 query rows as the other: scores^T = K Q^T, out^T = V^T W^T. Decode has 1 to
// 16 query rows per kv-head, so this wastes the least of the MMA, and the operands come from
// registers: the 8-bit bytes go from HBM to the lane that widens them. 8-bit keys and values
// are exact in f16. A query row is brought to |q| < 2^15 by a power of two (exact but for dims
// 2^28 below the row's largest, which lose bits below 2^-39 of it). w_t <= 2^15 is rounded
// to f16: half a step 2^-11 relative (the bf16 output's is 2^-8), and 2^-32 of the largest for
// weights 2^-21 below it. All sums and the softmax statistics are fp32.
//
// Per-row schedule (a function of the row's own L only, so decode, whole and chunked prefill,
// and any batch give the same bits):
//   * keys are cut into splits at absolute positions 0, 256, 512, ...; a split is folded page
//     by page (16 tokens, one MMA k-step of weights x values);
//   * s_t is one chain of D/16 MMAs, dims in a fixed order; lane t mod 8 sums p over its two
//     tokens of each page in order, and the 8 lanes are added by an xor tree at the split's end;
//   * whether m and F move at a page, and to what, depends on the row's own scores and value scales;
//   * a split ends with l brought into [1, 2) by a power of two that goes to m, and its sum of w v divided
//     by F and multiplied by that power and 2^-h, h = 2 + ceil(log2(the row's splits)), which keeps the
//     sum over splits below 2^127 for value rows of any size;
//   * splits are folded in ascending order: M' = max(M, m_s), X = X 2^(M-M') + x_s 2^(m_s-M').
// m and M are held as -m, which is added to z.
// An MMA's output column depends on its own column of query rows only, so it does not matter
// which rows share a tile. Tokens a row does not see get w = 0 exactly and stale value bytes are
// replaced by zeros; rows that see nothing give zeros.
#pragma once

#include "attention.cuh"
#include "gemm.cuh"
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

// 2^x with results below 2^-126 flushed to 0 (of a p: where the row's largest so far is at least 1).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float nan() { return __uint_as_float(0x7FC00000u); }
// 1 / x of a normal number (of a smaller one: infinity).
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^e for e <= 127, and 2^-126 below that.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(max(e, -126) + 127) << 23); }

// d += A B with A 16 x 16 (keys or values), B 16 x 8 (columns = query rows), f16 operands.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// d = A B.
__device__ __forceinline__ void mma16816_first(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, "
      "%10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Transposes an 8 x 8 matrix of 16-bit elements held two to a lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
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
//   keys: MMA rows g and g + 8 are tokens g and g + 8 of the page; step j covers dims
//     64 (j/4) + 16 c + 4 (j%4) + 0..3 of lane c, so the lane loads dims 64 v + 16 c .. + 15;
//   queries: column g of tile n is query row 8 n + g, same dims;
//   scores: the lane holds tokens g and g + 8 of query rows 8 n + 2c and + 1; transposed in 8 x 8
//     blocks they are the weights' operand, tokens 2c, 2c+1 (and + 8) of query row 8 n + g;
//   values: the lane loads tokens 2c, 2c+1, 2c+8, 2c+9, dims (D/8) g .. + D/8 - 1; rows g and g + 8
//     of tile i are dims (D/8) g + 2 i and + 1, so the lane ends with output dims
//     (D/8) g .. + D/8 - 1 of query rows 8 n + 2c and + 1.

// Four dims (one MMA step) of the keys of tokens g (x) and g + 8 (y).
template <int KIND>
__device__ __forceinline__ uint4 key_operand(uint32_t x, uint32_t y) {
  uint4 a;
  widen<KIND>(x, a.x, a.z);
  widen<KIND>(y, a.y, a.w);
  return a;
}

// Four dims (two tiles) of the values of tokens 2c, 2c+1, 2c+8, 2c+9.
template <int KIND>
__device__ __forceinline__ void value_operands(const uint32_t (&x)[4], uint4& a, uint4& b) {
  // bytes (token 2c, token 2c+1) of dims 0, 1 | 2, 3, and the same of tokens 2c+8, 2c+9
  widen<KIND>(__byte_perm(x[0], x[1], 0x5140), a.x, a.y);
  widen<KIND>(__byte_perm(x[2], x[3], 0x5140), a.z, a.w);
  widen<KIND>(__byte_perm(x[0], x[1], 0x7362), b.x, b.y);
  widen<KIND>(__byte_perm(x[2], x[3], 0x7362), b.z, b.w);
}

constexpr float kUnseen = 0x1p127f;  // -m of a row that has seen nothing: m is below its scores
constexpr float kMostL = 0x1p24f;    // a lane's l that moves the references
constexpr float kMostF = 0x1p120f;
constexpr float kNoScale = 0x1p-149f;  // value scale of a row of zeros, where F is found and after

// NT tiles of 8 query rows. A row that is not finite is taken as zeros and marked: its sum l becomes NaN
// if it saw a token. (A NaN in its scores would make pages that are not there count.)
template <int D, int NT>
struct Query {
  uint32_t b[NT][D / 16][2];
  float2 c[NT];  // of rows 8 n + 2c, + 1: scale log2(e) / the row's power of two
  uint32_t bad;  // bit 2 n + r: row 8 n + 2c + r is not finite
  __device__ __forceinline__ bool marked(int n, int r) const { return bad >> (2 * n + r) & 1u; }
};

// Loads query row g of tile n (nullptr: zeros). All lanes of the warp call it.
template <int D, int NT>
__device__ __forceinline__ void load_query(Query<D, NT>& Q, int n, const uint16_t* row, int lane, float scale_log2) {
  const int c = lane & 3;
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
  const float mine = finite ? __fmul_rn(scale_log2, down) : nan();
  const float c0 = __shfl_sync(kFullMask, mine, 8 * c), c1 = __shfl_sync(kFullMask, mine, 8 * c + 4);
  Q.bad = (n ? Q.bad : 0u) | (c0 != c0 ? 1u << (2 * n) : 0u) | (c1 != c1 ? 2u << (2 * n) : 0u);
  Q.c[n] = make_float2(c0 != c0 ? 0.f : c0, c1 != c1 ? 0.f : c1);
#pragma unroll
  for (int j = 0; j < D / 16; ++j) {
    // 4 dims: elements 4 (j%4) .. + 3 of the 16 in x[j/4]
    const uint4 q = x[j / 4][(j % 4) / 2];
    const uint32_t w0 = finite ? (j & 1) ? q.z : q.x : 0u, w1 = finite ? (j & 1) ? q.w : q.y : 0u;
    Q.b[n][j][0] = pack_f16x2(__fmul_rn(bf16lo(w0), up), __fmul_rn(bf16hi(w0), up));
    Q.b[n][j][1] = pack_f16x2(__fmul_rn(bf16lo(w1), up), __fmul_rn(bf16hi(w1), up));
  }
}

// Running state of a split: per query row -m, F and the sum of p over the lane's tokens, and
// sum w v over the lane's output dims (o[n][i]: dims 2i | 2i + 1 of rows 2c, 2c+1).
template <int D, int NT>
struct State {
  float2 m[NT], f[NT], l[NT];
  float o[NT][D / 16][4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n] = make_float2(kUnseen, kUnseen);
      f[n] = make_float2(1.f, 1.f);
      l[n] = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
    }
  }
};

// What the fold needs of the lane's tokens g and g + 8.
struct Tokens {
  float ks[2], sv[2], z0[2];  // key and value scale; added to z: 0, or -infinity where there is no value scale (0)
};

// Weights of one page from its scores s (which become z): moves m and F (and l and o with them) where
// it must, adds to l, and gives w as the operand of the value product. masked (the same for the
// whole warp): the lane's query row (n, r) sees the first nv(n, r) tokens only; otherwise all 16
// are seen.
// The weights are taken with the references in hand first, which most pages keep. A row that has one
// above 2^15, or an l above kMostL in some lane (infinite on the first page that it sees), moves m to its
// largest score and F to what the page then asks for, if that is less than F already is. Rows of zeros
// are found here: elsewhere their weights, 2^15 at most, meet zeros. set_tokens() gives the tokens
// (bit i: token i) whose value rows are not zeros.
// There is one line of code through the accumulators, with small blocks beside it for what is
// rare: a second, masked form of the whole page beside the plain one was slower for pages that never
// ran it (prefill of 4096 tokens 695 us against 635).
template <int D, int NT, typename Nv, typename Set>
__device__ __forceinline__ void page_weights(const Query<D, NT>& Q, float (&s)[NT][4], Tokens T, bool masked, Nv nv,
                                             Set set_tokens, int g, State<D, NT>& S, uint32_t (&w)[NT][2]) {
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const float2 z = __ffma2_rn(make_float2(s[n][2 * t], s[n][2 * t + 1]), __fmul2_rn(make_float2(T.ks[t], T.ks[t]), Q.c[n]),
                                  make_float2(T.z0[t], T.z0[t]));
      s[n][2 * t] = z.x;
      s[n][2 * t + 1] = z.y;
    }
  if (masked) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (g + 8 * (e >> 1) >= nv(n, e & 1)) s[n][e] = -INFINITY;
  }
  auto prob = [&](int n, int t) {  // p of query rows 2c, 2c + 1
    const float2 x = __fadd2_rn(make_float2(s[n][2 * t], s[n][2 * t + 1]), S.m[n]);
    return make_float2(ex2(x.x), ex2(x.y));
  };
  float2 l[NT];
  auto weigh = [&](int n) {  // w and l of tile n. (p F before sv: it stays in range where F sv need not)
    l[n] = S.l[n];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const float2 p = prob(n, t);
      l[n] = __fadd2_rn(l[n], p);
      const float2 x = __fmul2_rn(__fmul2_rn(p, S.f[n]), make_float2(T.sv[t], T.sv[t]));
      w[n][t] = pack_f16x2(x.x, x.y);
    }
  };
  auto most = [&](int n) { return __hmax2(*reinterpret_cast<__half2*>(&w[n][0]), *reinterpret_cast<__half2*>(&w[n][1])); };
  __half2 top;
  float sums = 0.f;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    weigh(n);
    top = n ? __hmax2(top, most(n)) : most(n);  // (a NaN is passed over, here and below: it moves nothing)
    sums = fmaxf(sums, fmaxf(l[n].x, l[n].y));
  }
  const __half2 limit = __halves2half2(__ushort_as_half(0x7800), __ushort_as_half(0x7800));  // 2^15
  if (__any_sync(kFullMask, !__hble2(top, limit) || sums > kMostL)) {
    if (__any_sync(kFullMask, T.sv[0] == 1.f || T.sv[1] == 1.f)) {  // the scale of a row of zeros, and of few others
      const uint32_t set = set_tokens();
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if (T.sv[t] == 1.f && !(set >> (g + 8 * t) & 1u)) T.sv[t] = kNoScale;
    }
    const uint32_t rows = 0x11111111u << (threadIdx.x & 3);  // the lanes of rows 2c, 2c + 1
    float to[NT][2], q[NT][2];                               // -m once moved, and the page's largest p sv then
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) to[n][r] = fmaxf(s[n][r], s[n][2 + r]);
#pragma unroll
    for (int d = 4; d < 32; d <<= 1)
#pragma unroll
      for (int i = 0; i < 2 * NT; ++i) to[i / 2][i % 2] = fmaxf(to[i / 2][i % 2], __shfl_xor_sync(kFullMask, to[i / 2][i % 2], d));
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        to[n][r] = fminf(r ? S.m[n].y : S.m[n].x, -to[n][r]);
        q[n][r] = fmaxf(__fmul_rn(ex2(__fadd_rn(s[n][r], to[n][r])), T.sv[0]),
                        __fmul_rn(ex2(__fadd_rn(s[n][2 + r], to[n][r])), T.sv[1]));
      }
#pragma unroll
    for (int d = 4; d < 32; d <<= 1)
#pragma unroll
      for (int i = 0; i < 2 * NT; ++i) q[i / 2][i % 2] = fmaxf(q[i / 2][i % 2], __shfl_xor_sync(kFullMask, q[i / 2][i % 2], d));
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const __half2 mine = most(n);
      float al[2], ao[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const bool up = __ballot_sync(kFullMask, (r ? __high2float(mine) : __low2float(mine)) > 32768.f ||
                                                     (r ? l[n].y : l[n].x) > kMostL) & rows;
        float& m = r ? S.m[n].y : S.m[n].x;
        float& f = r ? S.f[n].y : S.f[n].x;
        // o keeps its meaning, 2^m o / F: by 2^(m_old - m) and F / F_old. x * 1 == x: other rows keep their bits
        const float down = ex2(__fsub_rn(to[n][r], m));
        const float ft = fminf(fminf(__fmul_rn(f, ex2(__fsub_rn(m, to[n][r]))), __fmul_rn(128.f, rcp(q[n][r]))), kMostF);
        al[r] = up ? down : 1.f;
        ao[r] = up ? __fmul_rn(__fmul_rn(down, ft), rcp(f)) : 1.f;
        if (up) m = to[n][r], f = ft;
      }
      S.l[n] = __fmul2_rn(S.l[n], make_float2(al[0], al[1]));
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const float2 o = __fmul2_rn(make_float2(S.o[n][i][e], S.o[n][i][e + 1]), make_float2(ao[0], ao[1]));
          S.o[n][i][e] = o.x;
          S.o[n][i][e + 1] = o.y;
        }
      weigh(n);
    }
  }
  if (masked) {  // tokens that a row does not see have no weight, whatever their scales (their p is 0, w may be NaN)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int t = 0; t < 2; ++t)
        w[n][t] &= (g + 8 * t < nv(n, 0) ? 0xFFFFu : 0u) | (g + 8 * t < nv(n, 1) ? 0xFFFF0000u : 0u);
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    S.l[n] = l[n];
    w[n][0] = transpose8x8(w[n][0]);
    w[n][1] = transpose8x8(w[n][1]);
  }
}

// The xor tree over a query row's 8 lanes that ends a split.
__device__ __forceinline__ float row_sum(float l) {
#pragma unroll
  for (int d = 4; d < 32; d <<= 1) l = __fadd_rn(l, __shfl_xor_sync(kFullMask, l, d));
  return l;
}

// h of a row of n splits.
__device__ __forceinline__ int headroom(int n) { return 34 - __clz(n - 1); }

// The end of a split for query row (n, r), of a row of `splits` splits: -m and l as the fold over splits
// takes them, and the factor that its sums of w v are multiplied by (fp32 subnormal, with 18 bits or
// more, where all its p sv are below 2^-90 or so).
struct SplitEnd {
  float m, l, c;
  __device__ __forceinline__ float value(float o) const { return __fmul_rn(o, c); }
};
template <int D, int NT>
__device__ __forceinline__ SplitEnd split_end(const State<D, NT>& S, int n, int r, int splits) {
  const float l = row_sum(r ? S.l[n].y : S.l[n].x);
  const int e = (int)(__float_as_uint(l) >> 23) - 127;  // l = 0: -127, which changes neither l nor kUnseen
  return {__fsub_rn(r ? S.m[n].y : S.m[n].x, (float)e), __fmul_rn(l, pow2(-e)),
          __fmul_rn(pow2(-e - headroom(splits)), rcp(r ? S.f[n].y : S.f[n].x))};
}

// The output of a row of n splits from its folded sums.
__device__ __forceinline__ float row_out(float o, float l, int n) {
  return l == 0.f ? 0.f : __fmul_rn(__fdiv_rn(o, l), pow2(headroom(n)));
}

// One step of the fold over splits: -M and a split's -m -> the factors of both sides.
__device__ __forceinline__ void join(float& M, float m, float& a, float& b) {
  const float mn = fminf(M, m);
  a = ex2(__fsub_rn(mn, M));
  b = ex2(__fsub_rn(mn, m));
  M = mn;
}

// ---------------------------------------------------------------------------
// A page in shared memory: 16 key rows of D bytes, then 16 value rows, each swizzled as a TMA
// tile is (16-byte chunk i of row t at chunk i ^ (t % 8) for 128-byte rows, i ^ (t / 2 % 4) for
// 64-byte rows), and its 16 key and 16 value scales elsewhere. With 128-byte rows a lane's key
// reads meet one bank conflict in two and its value reads none.

template <int D>
constexpr int kPageBytes = 2 * PAGE * D;
constexpr int kScaleBytes = 2 * PAGE * 4;

// Byte offset of 16-byte chunk i of token t's row.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int t, int i) {
  return (uint32_t)(t * D + ((i ^ (D == 128 ? (t & 7) : ((t >> 1) & 3))) << 4));
}

// Scores of a page: tokens g and g + 8 of query rows 8 n + 2c and + 1, before any scale.
template <int KIND, int D, int NT>
__device__ __forceinline__ void page_scores(const Query<D, NT>& Q, uint32_t page, int lane, float (&s)[NT][4]) {
  const int g = lane >> 2, c = lane & 3;
  const uint32_t k0 = page + chunk_at<D>(g, c);  // chunk c + 4 of a 128-byte row: bit 6 flipped
#pragma unroll
  for (int v = 0; v < D / 64; ++v) {
    const uint4 x = ld_shared_v4(v ? k0 ^ 64u : k0);
    const uint4 y = ld_shared_v4((v ? k0 ^ 64u : k0) + 8 * D);
    const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const uint4 a = key_operand<KIND>(xw[b], yw[b]);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (v + b == 0) mma16816_first(s[n], a, Q.b[n][0][0], Q.b[n][0][1]);
        else mma16816(s[n], a, Q.b[n][4 * v + b][0], Q.b[n][4 * v + b][1]);
      }
    }
  }
}

// Folds a page whose scores are s. masked: `seen` of its tokens exist, query row (n, r) sees nv(n, r).
template <int KIND, int D, int NT, typename Nv>
__device__ __forceinline__ void fold_page(const Query<D, NT>& Q, float (&s)[NT][4], uint32_t page, uint32_t scales,
                                          bool masked, Nv nv, int seen, int lane, State<D, NT>& S) {
  const int g = lane >> 2, c = lane & 3;
  Tokens T;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    T.ks[t] = ld_shared_f32(scales + 4 * g + 32 * t);
    T.sv[t] = ld_shared_f32(scales + 64 + 4 * g + 32 * t);
    T.z0[t] = T.sv[t] == 0.f ? -INFINITY : 0.f;
  }
  uint32_t w[NT][2];
  auto set_tokens = [&] {  // lane c of four ORs its quarter of the rows of tokens g and g + 8
    uint32_t mine = 0;
#pragma unroll
    for (int t = 0; t < 16; t += 8) {
      uint32_t any = 0;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const uint4 y = ld_shared_v4(page + PAGE * D + chunk_at<D>(g + t, c * (D / 64) + i));
        any |= y.x | y.y | y.z | y.w;
      }
      if (any) mine |= 1u << (g + t);
    }
    return __reduce_or_sync(kFullMask, mine);
  };
  page_weights<D, NT>(Q, s, T, masked, nv, set_tokens, g, S, w);
  uint32_t x[4][D / 32];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = 2 * c + (i & 1);
    const uint32_t at = page + PAGE * D + (i >> 1) * 8 * D;
    if constexpr (D == 128) {
      const uint4 y = ld_shared_v4(at + chunk_at<D>(t, g));
      x[i][0] = y.x; x[i][1] = y.y; x[i][2] = y.z; x[i][3] = y.w;
    } else {
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                   : "=r"(x[i][0]), "=r"(x[i][1])
                   : "r"(at + chunk_at<D>(t, g >> 1) + 8 * (g & 1)));
    }
  }
  if (masked) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (2 * c + (i & 1) + 8 * (i >> 1) >= seen)
#pragma unroll
        for (int u = 0; u < D / 32; ++u) x[i][u] = 0;
  }
#pragma unroll
  for (int u = 0; u < D / 32; ++u) {
    uint4 a, b;
    const uint32_t xu[4] = {x[0][u], x[1][u], x[2][u], x[3][u]};
    value_operands<KIND>(xu, a, b);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      mma16816(S.o[n][2 * u], a, w[n][0], w[n][1]);
      mma16816(S.o[n][2 * u + 1], b, w[n][0], w[n][1]);
    }
  }
}

// ---------------------------------------------------------------------------
// Decode: one warp per (row, kv-head, split); the split's partial result goes to the workspace.
//
// Bound: HBM (Hkv (2 D + 8) bytes per token against 4 Hq D flops) where there are splits enough to
// go round: 64 int8 sequences of up to 32768 tokens (2.2 GB) take 424 us, 5.2 TB/s. A single
// short round is bound by one warp's 16 pages one after another (one sequence of 16921 tokens: 21 us).
// Each warp has a ring of kStages pages that one lane fills by TMA (two tiles and two 64-byte scale
// rows a page), ahead across item boundaries, and widens pages from it. The same ring filled by
// cp.async, lane by lane, took 0.50 ms for those 2.2 GB without any arithmetic; TMA takes that off
// the warps. Three stages: two took 406 us and four 415 where three took 394; deeper rings for the
// fewer warps of a short round gained nothing.

constexpr int kStages = 3;
constexpr int kCoarse = 512;  // entries of the split-count prefix that a CTA keeps

// W warps a CTA.
template <int D, int W>
struct Ring {
  static constexpr int SCALES = W * kStages * kPageBytes<D>;
  static constexpr int BARS = SCALES + W * kStages * kScaleBytes;
  static constexpr int PREFIX = BARS + W * kStages * 8;
  static constexpr int SMEM = 1024 + PREFIX + kCoarse * 4;  // pages start on a 1024-byte boundary
  static_assert(SMEM <= 227 * 1024, "shared memory");
};
// Warps that an SM's registers hold: 168 a thread with 16 query rows of 128 dims, else 128.
template <int D, int NT>
constexpr int kSmWarps = D * NT == 256 ? 12 : 16;

// Tensor map of a cache's rows [rows, D] of bytes, loaded a page (16 rows) at a time.
template <int D>
inline bool make_page_map(CUtensorMap* map, const void* ptr, int64_t rows) {
  gemm::EncodeTiledFn enc = gemm::encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)D};
  cuuint32_t box[2] = {(cuuint32_t)D, (cuuint32_t)PAGE};
  cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A work item: split s of row r (of `splits`) for one kv-head; `page` is page `lane` of it (-1: unusable).
struct Item {
  int r, s, kh, seen, page, splits;
};

template <int KIND, int D, int NT, int W>
__global__ void __launch_bounds__(W * 32, kSmWarps<D, NT> / W)
    split_kernel(const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm,
                 const uint16_t* __restrict__ q, int Hq, int Hkv, Cache C, Rows R, int nrows, int max_splits,
                 float* __restrict__ po, float2* __restrict__ pml, float scale_log2) {
  using T = Ring<D, W>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  __shared__ int32_t warp_sum[W];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int G = Hq / Hkv;
  int32_t* pre = reinterpret_cast<int32_t*>(smem + T::PREFIX);  // pre[i]: splits of rows below i * per
  const uint32_t base_u = smem_u32(smem);
  const uint32_t ring = base_u + (uint32_t)(warp * kStages * kPageBytes<D>);
  const uint32_t scales = base_u + (uint32_t)(T::SCALES + warp * kStages * kScaleBytes);
  const uint32_t bars = base_u + (uint32_t)(T::BARS + warp * kStages * 8);
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(bars + 8 * i, 1);
    fence_mbar_init();
  }
  __syncwarp();
  pdl_wait();  // the caller's inputs are complete from here on
  pdl_trigger();

  // the prefix of split counts, `per` rows an entry (1 up to kCoarse rows)
  const int per = (nrows + kCoarse - 1) / kCoarse, entries = (nrows + per - 1) / per;
  int base = 0;
  for (int e0 = 0; e0 < entries; e0 += W * 32) {
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
    for (int w = 0; w < W; ++w) {
      if (w < warp) before += warp_sum[w];
      base += warp_sum[w];
    }
    if (e < entries) pre[e] = before + x - n;
    __syncthreads();
  }
  const int total = base * Hkv;
  const int step = (int)gridDim.x * W;

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
    I.splits = (len + SPLIT - 1) / SPLIT;
    I.page = -1;
    if (lane * PAGE < I.seen) {
      const int pg = C.pt[(int64_t)pt_row * R.max_pages + I.s * PAGES_PER_SPLIT + lane];
      if (pg >= 0 && pg < C.num_pages) I.page = pg;
      else record_error(BI_ERR_DEVICE_INDEX);
    }
    return I;
  };

  int item = warp * (int)gridDim.x + (int)blockIdx.x;
  if (item >= total) return;
  Item cur = fetch(item), nxt = cur;
  bool ahead = false;            // the copies have gone on to nxt
  int pj = 0;
  uint32_t issued = 0, used = 0, filled = 0, ph_bits = 0;
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
      const uint32_t st = issued % kStages, bar = bars + 8 * st;
      if (lane == 0) {
        if (pg >= 0) {
          const int64_t row0 = ((int64_t)pg * Hkv + I.kh) * PAGE;
          note_fill(filled, ph_bits, (int)st, (issued / kStages) & 1u);
          fence_proxy_async_smem();
          mbar_arrive_expect_tx(bar, kPageBytes<D> + kScaleBytes);
          tma_load_2d(ring + st * kPageBytes<D>, &km, 0, (int)row0, bar);
          tma_load_2d(ring + st * kPageBytes<D> + PAGE * D, &vm, 0, (int)row0, bar);
          bulk_g2s(scales + st * kScaleBytes, C.ks + row0, PAGE * 4, bar);
          bulk_g2s(scales + st * kScaleBytes + PAGE * 4, C.vs + row0, PAGE * 4, bar);
        } else {
          mbar_arrive(bar);
        }
      }
      ++pj;
      ++issued;
    }
  };
  for (int i = 0; i < kStages; ++i) issue();

  while (true) {
    Query<D, NT> Q;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int head = g + 8 * n;
      load_query<D, NT>(Q, n, head < G ? q + ((int64_t)cur.r * Hq + cur.kh * G + head) * D : nullptr, lane, scale_log2);
    }
    State<D, NT> S;
    S.clear();
    const uint32_t usable = __ballot_sync(kFullMask, cur.page >= 0);
    // Two pages at a time: the second's scores are under way during the first's weights. A page that
    // is not there, or unusable, is one of whose tokens none is seen (whatever its stage holds).
    for (int j = 0; j * PAGE < cur.seen; j += 2) {
      const bool second = (j + 1) * PAGE < cur.seen;
      bool ok = mbar_wait(bars + 8 * (used % kStages), (used / kStages) & 1u);
      if (second) ok = ok && mbar_wait(bars + 8 * ((used + 1) % kStages), ((used + 1) / kStages) & 1u);
      if (!__all_sync(kFullMask, ok)) {
        // a copy never landed (recorded): let the others land, then leave
        if (lane == 0) drain_copies(bars, 8, filled, ph_bits);
        __syncwarp();
        return;
      }
      float s[2][NT][4];
      int seen[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        seen[u] = (usable >> (j + u)) & 1u ? cur.seen - (j + u) * PAGE : 0;
        if (NT == 1 || u == 0) page_scores<KIND, D, NT>(Q, ring + ((used + u) % kStages) * kPageBytes<D>, lane, s[u]);
      }
      const bool masked = seen[0] < PAGE || seen[1] < PAGE;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t st = (used + u) % kStages;
        if (NT > 1 && u == 1) page_scores<KIND, D, NT>(Q, ring + st * kPageBytes<D>, lane, s[u]);  // (no registers for both)
        fold_page<KIND, D, NT>(Q, s[u], ring + st * kPageBytes<D>, scales + st * kScaleBytes, masked,
                               [&](int, int) { return seen[u]; }, seen[u], lane, S);
      }
      __syncwarp();  // every lane has read these pages: their stages may be refilled
      used += second ? 2 : 1;
      issue();
      if (second) issue();
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const SplitEnd E = split_end(S, n, r, cur.splits);
        const int head = 8 * n + 2 * c + r;
        if (head >= G) continue;
        const int64_t slot = ((int64_t)cur.r * max_splits + cur.s) * Hq + cur.kh * G + head;
        float* dst = po + slot * D + (D / 8) * g;
#pragma unroll
        for (int i = 0; i < D / 16; i += 2)
          *reinterpret_cast<float4*>(dst + 2 * i) = make_float4(E.value(S.o[n][i][r]), E.value(S.o[n][i][2 + r]),
                                                                E.value(S.o[n][i + 1][r]), E.value(S.o[n][i + 1][2 + r]));
        if (g == 0) pml[slot] = make_float2(E.m, Q.marked(n, r) && E.l > 0.f ? nan() : E.l);
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
    for (uint32_t i = issued - used; i < kStages; ++i) issue();  // short items left the ring less than full
  }
}

// Folds a row's splits in ascending order; one warp per (row, query head, 32 * DPL output dims).
// The lanes take the splits' -m 32 at a time: the running minimum before and after each
// split (a minimum is exact in any order) gives the weights of both sides of its fold step, and
// the fold itself is one chain per output dim in split order whatever DPL is. The partial
// outputs come U at a time, the next U and the next 32 references asked for before these are folded.
template <int D, int DPL>
__global__ void __launch_bounds__(256) combine_kernel(const float* __restrict__ po, const float2* __restrict__ pml,
                                                      Rows R, int nrows, int max_splits, int Hq,
                                                      uint16_t* __restrict__ out) {
  constexpr int NG = D / (32 * DPL);  // warps per (row, head)
  constexpr int U = DPL == 1 ? 16 : 4;
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
  float M = kUnseen, L = 0.f, O[DPL];
#pragma unroll
  for (int d = 0; d < DPL; ++d) O[d] = 0.f;
  auto load = [&](int s0, float (&v)[U][DPL]) {  // splits s0 .. s0 + U - 1 (past n: the last again, unused)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float* p = src + (int64_t)min(s0 + u, n - 1) * Hq * D;
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
  };
  auto load_ml = [&](int s0) {
    return s0 + lane < n ? pml[slot0 + (int64_t)(s0 + lane) * Hq] : make_float2(kUnseen, 0.f);
  };
  if (n > 0) {
    float va[U][DPL], vb[U][DPL];
    float2 ml = load_ml(0), next = load_ml(32);
    load(0, va);
    float a = 0.f, b = 0.f;
    auto fold = [&](int s0, const float (&v)[U][DPL]) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = (s0 + u) & 31;
        const float ak = __shfl_sync(kFullMask, a, at), bk = __shfl_sync(kFullMask, b, at);
        const float lk = __shfl_sync(kFullMask, ml.y, at);
        if (s0 + u < n) {
          L = __fmaf_rn(lk, bk, __fmul_rn(L, ak));
#pragma unroll
          for (int d = 0; d < DPL; ++d) O[d] = __fmaf_rn(v[u][d], bk, __fmul_rn(O[d], ak));
        }
      }
    };
    for (int s0 = 0; s0 < n; s0 += 2 * U) {
      if (s0 + U < n) load(s0 + U, vb);
      if (s0 % 32 == 0) {
        if (s0) ml = next, next = load_ml(s0 + 32);
        float top = ml.x;  // the running minimum up to and with this lane's split
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const float y = __shfl_up_sync(kFullMask, top, d);
          if (lane >= d) top = fminf(top, y);
        }
        top = fminf(top, M);
        float prev = __shfl_up_sync(kFullMask, top, 1);
        if (lane == 0) prev = M;
        join(prev, ml.x, a, b);
        M = __shfl_sync(kFullMask, top, 31);
      }
      fold(s0, va);
      if (s0 + 2 * U < n) load(s0 + 2 * U, va);
      if (s0 + U < n) fold(s0 + U, vb);
    }
  }
  float y[DPL];
#pragma unroll
  for (int d = 0; d < DPL; ++d) y[d] = row_out(O[d], L, n);
  uint16_t* dst = out + rh * D + d0;
  if constexpr (DPL == 1) {
    *dst = to_bf16_bits(y[0]);
  } else {
#pragma unroll
    for (int d = 0; d < DPL; d += 2) reinterpret_cast<uint32_t*>(dst)[d / 2] = pack_bf16x2(y[d], y[d + 1]);
  }
}

// ---------------------------------------------------------------------------
// Prefill: rows of one sequence that follow one another in the batch are taken in tiles, and a
// tile and one kv-head run on one CTA. Query row i of a tile is query head i % G of token i / G.
//   * tile_kernel, tiles of up to 192 query rows: eight warps (twelve for D = 64) share out the
//     tiles of 8 query rows (three each at most; two), and four more widen keys and values once for
//     all of them into a ring of stages in shared memory, in fragment order (every access is 16
//     contiguous bytes a lane).
//   * few_kernel, tiles of up to kFewRows query rows (decode rows in a mixed batch, ends of
//     chunks, short chunks): every warp takes all the rows and one split at a time, reading pages as
//     decode does; a CTA, or a cluster of kFewCluster where there are few tiles, folds as many splits
//     as it has warps at a time.
// Either way a split is folded by one warp in the order above, and splits in ascending order.
// Bound: the latency of a folding warp's instructions. One prompt of 4096 tokens (32 heads over 8,
// D = 128, int8; 137 GFLOP) takes 0.593 ms, 232 TFLOP/s, where mma.sync itself gave 509 TFLOP/s on
// operands in registers; the schedulers issue in a third of the cycles, and what is left is the
// wait for one result after another with two (D = 64: three) folding warps on a scheduler, as
// many as the accumulators leave room for.
// (The figures below are from before the denominator had a reference of its own, which takes 6 to 8 %.)
//   * D = 128: 3 tiles on 8 warps; 2 on 12 has no room for the accumulators (695 us against 600 then).
//   * D = 64: 2 tiles on 12 warps (322 us for that prompt); 3 on 8 took 358, 3 on 12 403.
//   * A third tile's queries are read from shared memory for each page: the registers that this
//     frees are worth more than the reads (600 -> 583 us).
//   * The scores of a page are not issued ahead of the weights of the one before, which takes
//     registers for both (D = 64: 340 us with, 322 without; D = 128: no difference).

constexpr int kFewRows = 16;

// What the plan holds, at the front of the workspace.
struct Counts {
  int32_t tiles, few;   // first rows of tiles: list[0 .. tiles - 1], and of few-row tiles: list[T - few .. T - 1]
  int32_t next;         // the next work item of tile_kernel
};

// Cuts the runs of rows of one sequence into tiles of `per` tokens. One CTA of 1024 threads, each
// owning a contiguous stretch of rows. A tile whose run ends within `few` tokens is a few-row tile,
// and so is every tile if per == few.
__global__ void __launch_bounds__(1024) plan_kernel(const int32_t* __restrict__ q_seq, int T, int per, int few,
                                                    int32_t* __restrict__ list, Counts* __restrict__ counts) {
  __shared__ int32_t warp_last[32];
  __shared__ int2 warp_count[32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_trigger();
  const int each = (T + 1023) / 1024;
  const int r0 = (int)min((int64_t)tid * each, (int64_t)T), r1 = min(r0 + each, T);
  auto starts = [&](int r) { return r == 0 || q_seq[r] != q_seq[r - 1]; };
  // (every row up to r + few: with rows of sequences in turn, that one alone may be of the same sequence)
  auto is_few = [&](int r) {
    bool ends = per == few || r + few >= T;
    const int seq = q_seq[r];
    for (int i = 1; i <= few && !ends; ++i) ends = q_seq[r + i] != seq;
    return ends;
  };
  // the start of the run that row r0 - 1 lies in: the running maximum of run starts before this thread
  int last = -1;
  for (int r = r0; r < r1; ++r)
    if (starts(r)) last = r;
  int upto = last;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(kFullMask, upto, d);
    if (lane >= d) upto = max(upto, v);
  }
  if (lane == 31) warp_last[warp] = upto;
  __syncthreads();
  int before = __shfl_up_sync(kFullMask, upto, 1);
  if (lane == 0) before = -1;
  before = max(before, __reduce_max_sync(kFullMask, lane < warp ? warp_last[lane] : -1));
  int run = before, n0 = 0, n1 = 0;
  for (int r = r0; r < r1; ++r) {
    if (starts(r)) run = r;
    if ((r - run) % per) continue;
    if (is_few(r)) ++n1;
    else ++n0;
  }
  int2 sum = make_int2(n0, n1);  // up to and with this thread, first in its warp
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(kFullMask, sum.x, d), y = __shfl_up_sync(kFullMask, sum.y, d);
    if (lane >= d) sum.x += x, sum.y += y;
  }
  if (lane == 31) warp_count[warp] = sum;
  __syncthreads();
  const int2 w = lane < warp ? warp_count[lane] : make_int2(0, 0);
  sum.x += __reduce_add_sync(kFullMask, w.x);
  sum.y += __reduce_add_sync(kFullMask, w.y);
  int at0 = sum.x - n0, at1 = T - (sum.y - n1) - 1;
  run = before;
  for (int r = r0; r < r1; ++r) {
    if (starts(r)) run = r;
    if ((r - run) % per) continue;
    if (is_few(r)) list[at1--] = r;
    else list[at0++] = r;
  }
  if (tid == 1023) *counts = Counts{sum.x, sum.y, 0};
}

// Tokens of the tile that starts at row `first`: rows of its sequence that follow it, `per` at most.
__device__ __forceinline__ int tile_tokens(const int32_t* __restrict__ q_seq, int first, int T, int per, int lane) {
  const int seq = q_seq[first];
  int n = 0;
  while (n < per) {
    const int r = first + n + lane;
    const uint32_t same = __ballot_sync(kFullMask, r < T && n + lane < per && q_seq[r] == seq);
    if (same != kFullMask) return n + __ffs(~same) - 1;
    n += 32;
  }
  return per;
}

// Page i of a sequence that is seen up to `len`: its id, or -1 past the end or if it is unusable.
__device__ __forceinline__ int page_id(const Cache& C, const int32_t* prow, int i, int len) {
  if (i * PAGE >= len) return -1;
  const int pg = prow[i];
  if (pg >= 0 && pg < C.num_pages) return pg;
  record_error(BI_ERR_DEVICE_INDEX);
  return -1;
}

// The ids of a sequence's pages as a walk over its chunks needs them: 32 pages from a multiple of
// 32 on, one a lane, and the next 32 already asked for.
struct PageIds {
  int first, now, then;
  __device__ __forceinline__ void start(const Cache& C, const int32_t* prow, int len, int lane) {
    first = 0;
    now = page_id(C, prow, lane, len);
    then = page_id(C, prow, 32 + lane, len);
  }
  // Moves on to the 32 pages that page i is among (i never falls, nor rises by more than 32).
  __device__ __forceinline__ void at(const Cache& C, const int32_t* prow, int i, int len, int lane) {
    if (i < first + 32) return;
    first += 32;
    now = then;
    then = page_id(C, prow, first + 32 + lane, len);
  }
  __device__ __forceinline__ int operator[](int i) const { return __shfl_sync(kFullMask, now, i & 31); }
};

// cp.async of one page (store rows row0 .. + 15) by a warp, 16 contiguous bytes a lane.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <int D>
__device__ __forceinline__ void copy_page(uint32_t page, uint32_t scales, const Cache& C, int64_t row0, int lane) {
#pragma unroll
  for (int i = 0; i < PAGE * D / 512; ++i) {
    const int at = i * 32 + lane, t = at / (D / 16), chunk = at % (D / 16);
    cp_async16(page + chunk_at<D>(t, chunk), C.k + row0 * D + at * 16);
    cp_async16(page + PAGE * D + chunk_at<D>(t, chunk), C.v + row0 * D + at * 16);
  }
  if (lane < 8) cp_async16(scales + 16 * lane, (lane < 4 ? C.ks + row0 : C.vs + row0 - PAGE) + 4 * lane);
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// Writes a query row's dims (D/8) g .. + D/8 - 1.
template <int D>
__device__ __forceinline__ void store_row(uint16_t* dst, const float (&x)[D / 8], float L, int splits) {
#pragma unroll
  for (int i = 0; i < D / 8; i += 8) {
    float y[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) y[u] = row_out(x[i + u], L, splits);
    *reinterpret_cast<uint4*>(dst + i) = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                                    pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
  }
}

constexpr int kWidenWarps = 4;
constexpr int kRing = 4;

// Registers: the CTA starts with the SM's shared out evenly; the widening warps keep 56 each and
// the folding warps take the rest (D = 128: 128 * 56 + 256 * 224 = 384 * 168; D = 64:
// 128 * 56 + 384 * 152 = 512 * 128).
template <int D>
struct TileShape {
  static constexpr int NT = D == 128 ? 3 : 2;     // tiles of 8 query rows per folding warp, at most
  static constexpr int FOLD = D == 128 ? 8 : 12;  // folding warps
  static constexpr int WARPS = FOLD + kWidenWarps, THREADS = WARPS * 32;
  static constexpr int ROWS = FOLD * NT * 8;
  static constexpr int WIDEN_REGS = 56, FOLD_REGS = D == 128 ? 224 : 152, START_REGS = D == 128 ? 168 : 128;
  static_assert(kWidenWarps * WIDEN_REGS + FOLD * FOLD_REGS <= WARPS * START_REGS, "registers at launch");
};

template <int D>
struct TileSmem {
  using P = TileShape<D>;
  static constexpr int PAGES = 256 / D;                      // pages a stage: one part of each kind per widening warp
  static constexpr int OPERANDS = PAGES * 2 * PAGE * D * 2;  // f16 keys, then values
  static constexpr int STAGE = OPERANDS + PAGES * PAGE * 16;  // and {ks, vs, z0, -} per token
  static constexpr int TOTALS = kRing * STAGE;               // fp32 totals [row][D], lane by lane
  static constexpr int STATS = TOTALS + P::ROWS * D * 4;     // M and L, lane by lane
  static constexpr int LENS = STATS + P::FOLD * 32 * P::NT * 16;  // visible lengths, lane by lane
  static constexpr int BARS = LENS + P::FOLD * 32 * P::NT * 8;
  static constexpr int ARGS = BARS + kRing * 16;                   // two TileArgs
  static constexpr int MARKS = ARGS + 512;                         // the query rows that are not finite, lane by lane
  static constexpr int QUERY = MARKS + P::FOLD * 128;              // a third tile's queries, lane by lane
  static constexpr int BYTES = QUERY + (P::NT == 3 ? P::FOLD * (D / 32) * 512 : 0);
  static_assert(BYTES <= 227 * 1024, "shared memory");
};

// A lane's part of a stage on its way: key bytes of tokens g and g + 8 and value bytes of four
// tokens, of one page and 64 (8 of the lane's) dims each, and a token's scales.
struct Raw {
  uint4 k[2];
  uint2 v[4];
  float ks, vs;
};

// Loads the part of the stage at token tp that widening warp `warp` owns. Bytes of unusable pages,
// and of tokens from len on, are zeros.
template <int D>
__device__ __forceinline__ void load_raw(Raw& X, const Cache& C, const int32_t* prow, PageIds& ids, int tp, int len, int Hkv,
                                         int kh, int warp, int lane) {
  using M = TileSmem<D>;
  static_assert(M::PAGES * (D / 64) == kWidenWarps && M::PAGES * PAGE <= kWidenWarps * 32, "one part a warp");
  const int g = lane >> 2, c = lane & 3;
  ids.at(C, prow, tp / PAGE, len, lane);  // a stage lies within 32 pages
  const int page = warp / (D / 64), part = warp % (D / 64);
  const int t0 = tp + page * PAGE;
  const int pg = ids[t0 / PAGE];
  const bool ok = pg >= 0;
  const int64_t row0 = ok ? ((int64_t)pg * Hkv + kh) * PAGE : 0;
  const uint8_t* kp = C.k + (row0 + g) * D + 64 * part + 16 * c;
  X.k[0] = ok ? __ldg(reinterpret_cast<const uint4*>(kp)) : make_uint4(0, 0, 0, 0);
  X.k[1] = ok ? __ldg(reinterpret_cast<const uint4*>(kp + 8 * D)) : make_uint4(0, 0, 0, 0);
  const uint8_t* vp = C.v + (row0 + 2 * c) * D + (D / 8) * g + 8 * part;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = (i & 1) + 8 * (i >> 1);
    X.v[i] = ok && t0 + 2 * c + t < len ? __ldg(reinterpret_cast<const uint2*>(vp + t * D)) : make_uint2(0, 0);
  }
  X.ks = 0.f;
  X.vs = 0.f;
  if (warp * 32 < M::PAGES * PAGE) {
    const int tok = warp * 32 + lane, tpg = ids[(tp + tok) / PAGE];
    if (tpg >= 0 && tp + tok < len) {
      const int64_t r = ((int64_t)tpg * Hkv + kh) * PAGE + tok % PAGE;
      X.ks = __ldg(C.ks + r);
      X.vs = __ldg(C.vs + r);
    }
  }
}

// Widens a loaded part into a stage: keys [page][step][lane], values [page][tile][lane], tokens. A
// token without a value scale (0) has no weight.
template <int KIND, int D>
__device__ __forceinline__ void widen_raw(const Raw& X, uint32_t stage, int warp, int lane) {
  using M = TileSmem<D>;
  const int page = warp / (D / 64), part = warp % (D / 64);
  const uint32_t kb = stage + ((page * (D / 16) + 4 * part) * 32 + lane) * 16;
  const uint32_t xw[4] = {X.k[0].x, X.k[0].y, X.k[0].z, X.k[0].w}, yw[4] = {X.k[1].x, X.k[1].y, X.k[1].z, X.k[1].w};
#pragma unroll
  for (int b = 0; b < 4; ++b) st_shared_v4(kb + b * 512, key_operand<KIND>(xw[b], yw[b]));
  const uint32_t vb = kb + M::OPERANDS / 2;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = u ? X.v[i].y : X.v[i].x;
    uint4 a, b;
    value_operands<KIND>(w, a, b);
    st_shared_v4(vb + (2 * u) * 512, a);
    st_shared_v4(vb + (2 * u + 1) * 512, b);
  }
  if (warp * 32 < M::PAGES * PAGE) {
    const float4 t = make_float4(X.ks, X.vs, X.vs == 0.f ? -INFINITY : 0.f, 0.f);
    st_shared_v4(stage + M::OPERANDS + (warp * 32 + lane) * 16, *reinterpret_cast<const uint4*>(&t));
  }
}

// The CTA's barrier; its warps meet it in different places.
__device__ __forceinline__ void tile_sync() { asm volatile("barrier.cta.sync 0;" ::: "memory"); }

// A wait that, once one of this thread's has given up (recorded), is skipped: the CTA then runs to
// its end with wrong numbers instead of waiting again at every stage.
__device__ __forceinline__ void ring_wait(uint32_t bar, uint32_t parity, bool& dead) {
  if (!dead) dead = !mbar_wait(bar, parity);
}

// Scores of one page of a buffer for the warp's LIVE tiles, and a page's tokens.
template <int D, int LIVE>
__device__ __forceinline__ void wide_scores(const Query<D, LIVE>& Q, uint32_t buf, uint32_t third, int page, int lane,
                                            float (&s)[LIVE][4]) {
  const uint32_t kb = buf + (page * (D / 16) * 32 + lane) * 16;
  uint4 b;
#pragma unroll
  for (int j = 0; j < D / 16; ++j) {
    const uint4 a = ld_shared_v4(kb + j * 512);
#pragma unroll
    for (int n = 0; n < LIVE; ++n) {
      if (n == 2 && j % 2 == 0) b = ld_shared_v4(third + j * 256);
      const uint32_t b0 = n < 2 ? Q.b[n][j][0] : j % 2 ? b.z : b.x, b1 = n < 2 ? Q.b[n][j][1] : j % 2 ? b.w : b.y;
      if (j == 0) mma16816_first(s[n], a, b0, b1);
      else mma16816(s[n], a, b0, b1);
    }
  }
}
template <int D>
__device__ __forceinline__ Tokens wide_tokens(uint32_t buf, int page, int lane) {
  Tokens T;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const uint4 x = ld_shared_v4(buf + TileSmem<D>::OPERANDS + (page * PAGE + (lane >> 2) + 8 * t) * 16);
    T.ks[t] = __uint_as_float(x.x);
    T.sv[t] = __uint_as_float(x.y);
    T.z0[t] = __uint_as_float(x.z);
  }
  return T;
}
template <int D, int LIVE>
__device__ __forceinline__ void wide_values(uint32_t buf, int page, int lane, const uint32_t (&w)[LIVE][2],
                                            State<D, LIVE>& S) {
  const uint32_t vb = buf + TileSmem<D>::OPERANDS / 2 + (page * (D / 16) * 32 + lane) * 16;
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    const uint4 a = ld_shared_v4(vb + i * 512);
#pragma unroll
    for (int n = 0; n < LIVE; ++n) mma16816(S.o[n][i], a, w[n][0], w[n][1]);
  }
}

// Folds a page of a stage. masked: query row (n, r) sees the first nv(n, r) tokens.
template <int D, int LIVE, typename Nv>
__device__ __forceinline__ void fold_wide(const Query<D, LIVE>& Q, uint32_t stage, uint32_t third, int page, bool masked, Nv nv,
                                          int lane, State<D, LIVE>& S) {
  float s[LIVE][4];
  wide_scores<D, LIVE>(Q, stage, third, page, lane, s);
  const Tokens T = wide_tokens<D>(stage, page, lane);
  uint32_t w[LIVE][2];
  auto set_tokens = [&] {  // the lane ORs its dims of tokens 2c, 2c + 1, 2c + 8, 2c + 9, as f16 pairs
    const uint32_t vb = stage + TileSmem<D>::OPERANDS / 2 + (page * (D / 16) * 32 + lane) * 16;
    uint32_t lo = 0, hi = 0;
    for (int i = 0; i < D / 16; ++i) {
      const uint4 y = ld_shared_v4(vb + i * 512);
      lo |= y.x | y.y;
      hi |= y.z | y.w;
    }
    const uint32_t mine = (lo & 0xFFFFu ? 1u : 0u) | (lo >> 16 ? 2u : 0u) | (hi & 0xFFFFu ? 0x100u : 0u) | (hi >> 16 ? 0x200u : 0u);
    return __reduce_or_sync(kFullMask, mine << (2 * (lane & 3)));
  };
  page_weights<D, LIVE>(Q, s, T, masked, nv, set_tokens, lane >> 2, S, w);
  wide_values<D, LIVE>(stage, page, lane, w, S);
}

// What a warp needs of its tile.
struct TileArgs {
  const uint16_t* q;
  int64_t ldq;
  uint16_t* out;
  Cache C;
  Rows R;
  const int32_t* prow;
  int Hq, Hkv, G, first, rows, kh, len;
  float scale_log2;
};
static_assert(sizeof(TileArgs) <= 256, "room in shared memory");

// One tile for a folding warp with LIVE (or fewer) of its tiles of 8 query rows: the warp's n-th is
// tile 8 n + warp. Rows past the tile's end are zeros whose results go nowhere. `it` counts the
// ring's stages.
template <int KIND, int D, int LIVE>
__device__ __forceinline__ void fold_tile(const TileArgs& A, uint8_t* smem, uint32_t base, uint32_t bars, uint32_t& it,
                                          bool& dead, int warp, int lane) {
  using M = TileSmem<D>;
  using P = TileShape<D>;
  const int g = lane >> 2, c = lane & 3;
  constexpr int CHUNK = M::PAGES * PAGE;
  Query<D, LIVE> Q;
  int shortest = INT_MAX;
  // visible tokens of the lane's query rows, and running totals over splits, in places of this lane's own
  int2* lens = reinterpret_cast<int2*>(smem + M::LENS) + warp * 32 * P::NT + lane;               // entry n at [32 n]
  float* tot = reinterpret_cast<float*>(smem + M::TOTALS) + warp * (P::NT * 8) * D + lane;       // entry i at [32 i]
  float4* stats = reinterpret_cast<float4*>(smem + M::STATS) + warp * 32 * P::NT + lane;         // M and L, entry n at [32 n]
#pragma unroll
  for (int n = 0; n < LIVE; ++n) {
    const int i = (n * P::FOLD + warp) * 8 + g;
    load_query<D, LIVE>(Q, n,
                        i < A.rows ? A.q + (int64_t)(A.first + i / A.G) * A.ldq + (int64_t)(A.kh * A.G + i % A.G) * D : nullptr,
                        lane, A.scale_log2);
    int len[2] = {0, 0};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int k = (n * P::FOLD + warp) * 8 + 2 * c + r;
      if (k >= A.rows) continue;
      int pt_row;
      len[r] = attn::row_len(A.R, A.first + k / A.G, pt_row);
      shortest = min(shortest, len[r]);
    }
    lens[32 * n] = make_int2(len[0], len[1]);
  }
  const uint32_t third = base + M::QUERY + (warp * (D / 32) * 32 + lane) * 16;
  if constexpr (LIVE == 3) {
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
      st_shared_v4(third + j * 512, make_uint4(Q.b[2][2 * j][0], Q.b[2][2 * j][1], Q.b[2][2 * j + 1][0], Q.b[2][2 * j + 1][1]));
  }
  shortest = __reduce_min_sync(kFullMask, shortest);
#pragma unroll
  for (int n = 0; n < LIVE; ++n) stats[32 * n] = make_float4(kUnseen, kUnseen, 0.f, 0.f);
  uint32_t* marks = reinterpret_cast<uint32_t*>(smem + M::MARKS) + warp * 32 + lane;  // (no register for them in the loop)
  *marks = Q.bad;
#pragma unroll 8
  for (int i = 0; i < LIVE * D / 4; ++i) tot[32 * i] = 0.f;
#pragma unroll 1
  for (int t0 = 0; t0 < A.len; t0 += SPLIT) {
    State<D, LIVE> S;
    S.clear();
#pragma unroll 1
    for (int tp = t0; tp < min(t0 + SPLIT, A.len); tp += CHUNK, ++it) {
      const uint32_t stage = base + (it % kRing) * M::STAGE, full = bars + (it % kRing) * 16;
      ring_wait(full, (it / kRing) & 1u, dead);
#pragma unroll
      for (int p = 0; p < M::PAGES; ++p) {  // (pages that none of its rows sees too: a way round them costs more)
        const int at = tp + p * PAGE;
        fold_wide<D, LIVE>(Q, stage, third, p, at + PAGE > shortest,
                           [&](int n, int r) {
                             const int2 len = lens[32 * n];
                             return (r ? len.y : len.x) - at;
                           },
                           lane, S);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(full + 8);  // this warp has read the stage
    }
#pragma unroll
    for (int n = 0; n < LIVE; ++n) {
      float4 st = stats[32 * n];
      float a0, b0, a1, b1;
      const int2 len = lens[32 * n];
      const SplitEnd E0 = split_end(S, n, 0, (len.x + SPLIT - 1) / SPLIT), E1 = split_end(S, n, 1, (len.y + SPLIT - 1) / SPLIT);
      join(st.x, E0.m, a0, b0);
      join(st.y, E1.m, a1, b1);
      st.z = __fmaf_rn(E0.l, b0, __fmul_rn(st.z, a0));
      st.w = __fmaf_rn(E1.l, b1, __fmul_rn(st.w, a1));
      stats[32 * n] = st;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float* x = tot + 32 * (n * 2 * (D / 8) + 2 * i + e);  // and of row 2c + 1 at [32 (D / 8)]
          const float2 v = __fmul2_rn(make_float2(S.o[n][i][2 * e], S.o[n][i][2 * e + 1]), make_float2(E0.c, E1.c));
          const float2 y = __ffma2_rn(v, make_float2(b0, b1), __fmul2_rn(make_float2(x[0], x[32 * (D / 8)]), make_float2(a0, a1)));
          x[0] = y.x;
          x[32 * (D / 8)] = y.y;
        }
    }
  }
#pragma unroll
  for (int n = 0; n < LIVE; ++n)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int k = (n * P::FOLD + warp) * 8 + 2 * c + r;
      if (k >= A.rows) continue;
      const float4 st = stats[32 * n];
      float x[D / 8];
#pragma unroll
      for (int i = 0; i < D / 8; ++i) x[i] = tot[32 * ((n * 2 + r) * (D / 8) + i)];
      const int len = r ? lens[32 * n].y : lens[32 * n].x;
      float L = r ? st.w : st.z;
      if (L > 0.f && *marks >> (2 * n + r) & 1u) L = nan();
      store_row<D>(A.out + ((int64_t)(A.first + k / A.G) * A.Hq + A.kh * A.G + k % A.G) * D + (D / 8) * g, x, L,
                   (len + SPLIT - 1) / SPLIT);
    }
}

// One tile for a widening warp: its part of every stage. (The ring is what hides the loads: the
// widening warps are ahead of the folding ones by up to kRing stages.)
template <int KIND, int D>
__device__ __forceinline__ void widen_tile(const TileArgs& A, uint32_t base, uint32_t bars, uint32_t& it, bool& dead, int warp,
                                           int lane) {
  using M = TileSmem<D>;
  constexpr int CHUNK = M::PAGES * PAGE;
  if (A.len <= 0) return;
  PageIds ids;
  ids.start(A.C, A.prow, A.len, lane);
#pragma unroll 1
  for (int tp = 0; tp < A.len; tp += CHUNK, ++it) {
    const uint32_t stage = base + (it % kRing) * M::STAGE, full = bars + (it % kRing) * 16;
    Raw X;
    load_raw<D>(X, A.C, A.prow, ids, tp, A.len, A.Hkv, A.kh, warp, lane);
    if (it >= kRing) ring_wait(full + 8, (it / kRing - 1) & 1u, dead);
    widen_raw<KIND, D>(X, stage, warp, lane);
    __syncwarp();
    if (lane == 0) mbar_arrive(full);  // this warp's part is in place
  }
}

template <int KIND, int D>
__global__ void __launch_bounds__(TileShape<D>::THREADS, 1)
    tile_kernel(const uint16_t* __restrict__ q, int64_t ldq, int Hq, int Hkv, Cache C, Rows R, int T, int per,
                const int32_t* __restrict__ list, Counts* __restrict__ counts, uint16_t* __restrict__ out,
                float scale_log2) {
  using M = TileSmem<D>;
  using P = TileShape<D>;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(smem), bars = base + M::BARS;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(bars + 16 * i, kWidenWarps);     // a stage is complete
      mbar_init(bars + 16 * i + 8, P::FOLD);  // a stage has been read
    }
    fence_mbar_init();
  }
  pdl_wait();  // the plan (and the caller's q and store) are complete from here on
  pdl_trigger();
  uint32_t it = 0;
  bool dead = false;
  // What the tile in hand is, and the next one: the last warp looks the next one up once it has
  // widened this one's last stage, while the others still fold. rows < 0: there is none. Later rows
  // of a prompt see more keys: longest first.
  TileArgs* args = reinterpret_cast<TileArgs*>(smem + M::ARGS);
  auto look_up = [&](TileArgs& A) {
    int item = 0;
    if (lane == 0) item = counts->tiles * Hkv - 1 - atomicAdd(&counts->next, 1);  // all that this decides is who
    item = __shfl_sync(kFullMask, item, 0);
    if (item < 0) {
      if (lane == 0) A.rows = -1;
      return;
    }
    const int first = list[item / Hkv], n = tile_tokens(R.q_seq, first, T, per, lane);
    int len = 0, pt_row = 0;
    for (int i = lane; i < n; i += 32) {
      int row;
      const int x = attn::row_len(R, first + i, row);
      if (x > len) len = x, pt_row = row;
    }
    len = __reduce_max_sync(kFullMask, len);
    pt_row = __reduce_max_sync(kFullMask, pt_row);  // rows that see anything share it; the others gave 0
    if (lane == 0)
      A = TileArgs{q, ldq, out, C, R, C.pt + (int64_t)pt_row * R.max_pages, Hq, Hkv, Hq / Hkv, first, n * (Hq / Hkv),
                   item % Hkv, len, scale_log2};
  };
  int b = 0;
  if (warp >= P::FOLD) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(P::WIDEN_REGS));
    const bool looks = warp == P::FOLD + kWidenWarps - 1;
    if (looks) look_up(args[0]);
    for (tile_sync(); args[b].rows >= 0; b ^= 1, tile_sync()) {
      widen_tile<KIND, D>(args[b], base, bars, it, dead, warp - P::FOLD, lane);
      if (looks) look_up(args[b ^ 1]);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(P::FOLD_REGS));
    for (tile_sync(); args[b].rows >= 0; b ^= 1, tile_sync()) {
      const TileArgs& A = args[b];
      const int tiles = (A.rows + 7) / 8;  // of 8 query rows
      if (tiles > (P::NT - 1) * P::FOLD + warp) fold_tile<KIND, D, P::NT>(A, smem, base, bars, it, dead, warp, lane);
      else if (P::NT > 2 && tiles > P::FOLD + warp) fold_tile<KIND, D, 2>(A, smem, base, bars, it, dead, warp, lane);
      else fold_tile<KIND, D, 1>(A, smem, base, bars, it, dead, warp, lane);
    }
  }
}

constexpr int kFewWarps = 4;
constexpr int kFewStages = 3;
constexpr int kFewCluster = 8;

template <int D>
struct FewSmem {
  static constexpr int STAGE = kPageBytes<D> + kScaleBytes;
  static constexpr int RINGS = kFewWarps * kFewStages * STAGE;       // over which the partial results go
  static constexpr int PARTIALS = kFewWarps * kFewRows * D * 4;
  static constexpr int OVER = RINGS > PARTIALS ? RINGS : PARTIALS;
  static constexpr int BYTES = OVER + kFewWarps * kFewRows * 8 + kFewRows * D * 4;
};

// One tile of up to 8 NT query rows, by the CTAS CTAs of a cluster (1: this CTA alone).
template <int KIND, int D, int NT, int CTAS>
__device__ __forceinline__ void few_tile(const uint16_t* __restrict__ q, int64_t ldq, int Hq, int Hkv, int G, const Cache& C,
                                         const Rows& R, int first, int rows, int kh, uint16_t* __restrict__ out,
                                         float scale_log2, uint8_t* smem, int warp, int lane) {
  using M = FewSmem<D>;
  const int rank = CTAS > 1 ? (int)cluster_rank() : 0;
  auto sync = [&] {  // all that share the tile
    __syncwarp();
    if (CTAS > 1) cluster_barrier();
    else __syncthreads();
  };
  const int g = lane >> 2, c = lane & 3;
  const uint32_t base = smem_u32(smem);
  Query<D, NT> Q;
  int len[NT][2], longest = 0, shortest = INT_MAX / 2, pt_row = 0;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int i = 8 * n + g;
    load_query<D, NT>(Q, n, i < rows ? q + (int64_t)(first + i / G) * ldq + (int64_t)(kh * G + i % G) * D : nullptr,
                          lane, scale_log2);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int k = 8 * n + 2 * c + r;
      len[n][r] = INT_MAX / 2;  // no row: nothing to mask
      if (k < rows) {
        int row;
        len[n][r] = attn::row_len(R, first + k / G, row);
        longest = max(longest, len[n][r]);
        pt_row = max(pt_row, row);
      }
      shortest = min(shortest, len[n][r]);
    }
  }
  longest = __reduce_max_sync(kFullMask, longest);
  shortest = __reduce_min_sync(kFullMask, shortest);
  pt_row = __reduce_max_sync(kFullMask, pt_row);  // rows that see anything share it; the others gave 0
  const int32_t* prow = C.pt + (int64_t)pt_row * R.max_pages;
  // a split a warp at a time; then row k's four threads of each CTA fold them in order, D / CTAS dims a CTA
  const uint32_t ring = base + (uint32_t)(warp * kFewStages * kPageBytes<D>);
  const uint32_t scales = base + (uint32_t)(kFewWarps * kFewStages * kPageBytes<D> + warp * kFewStages * kScaleBytes);
  float* part = reinterpret_cast<float*>(smem);                                  // [warp][row][D]
  float2* pml = reinterpret_cast<float2*>(smem + M::OVER);                          // [warp][row]
  float* tot = reinterpret_cast<float*>(smem + M::OVER + kFewWarps * kFewRows * 8);      // [row][D]
  for (int i = threadIdx.x; i < rows * D; i += kFewWarps * 32) tot[i] = 0.f;
  constexpr int dims = D / 4 / CTAS;  // even
  const int frow = threadIdx.x >> 2, fd = (threadIdx.x & 3) * (D / 4) + rank * dims;
  float FM = kUnseen, FL = 0.f;
  for (int r0 = 0; r0 < longest; r0 += CTAS * kFewWarps * SPLIT) {
    const int t0 = r0 + (rank * kFewWarps + warp) * SPLIT, seen = min(SPLIT, longest - t0);
    State<D, NT> S;
    S.clear();
    const int np = seen > 0 ? (seen + PAGE - 1) / PAGE : 0;
    int page = -1;
    if (lane < np) page = page_id(C, prow, t0 / PAGE + lane, longest);
    auto issue = [&](int j) {
      if (j < np) {
        const int pg = __shfl_sync(kFullMask, page, j);
        const uint32_t st = (uint32_t)(j % kFewStages);
        if (pg >= 0)
          copy_page<D>(ring + st * kPageBytes<D>, scales + st * kScaleBytes, C, ((int64_t)pg * Hkv + kh) * PAGE, lane);
      }
      cp_commit();
    };
    for (int j = 0; j < kFewStages; ++j) issue(j);
    for (int j = 0; j < np; ++j) {
      cp_wait<kFewStages - 1>();
      __syncwarp();
      if (__shfl_sync(kFullMask, page, j) >= 0) {
        const int tp = t0 + j * PAGE;
        const uint32_t st = (uint32_t)(j % kFewStages), pg = ring + st * kPageBytes<D>;
        float s[NT][4];
        page_scores<KIND, D, NT>(Q, pg, lane, s);
        fold_page<KIND, D, NT>(Q, s, pg, scales + st * kScaleBytes, tp + PAGE > shortest,
                               [&](int n, int r) { return len[n][r] - tp; }, longest - tp, lane, S);
      }
      __syncwarp();
      issue(j + kFewStages);
    }
    cp_wait<0>();
    __syncthreads();  // the rings are free (and the totals cleared, or the last fold done)
    if (np > 0) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const SplitEnd E = split_end(S, n, r, (len[n][r] + SPLIT - 1) / SPLIT);
          const int k = 8 * n + 2 * c + r;
          if (k >= rows) continue;
          float* dst = part + (warp * kFewRows + k) * D + (D / 8) * g;
#pragma unroll
          for (int i = 0; i < D / 16; i += 2)
            *reinterpret_cast<float4*>(dst + 2 * i) = make_float4(E.value(S.o[n][i][r]), E.value(S.o[n][i][2 + r]),
                                                                  E.value(S.o[n][i + 1][r]), E.value(S.o[n][i + 1][2 + r]));
          if (g == 0) pml[warp * kFewRows + k] = make_float2(E.m, Q.marked(n, r) && E.l > 0.f ? nan() : E.l);
        }
    }
    sync();
    if (frow < rows) {
      for (int o = 0; o < CTAS && r0 + o * kFewWarps * SPLIT < longest; ++o) {  // the CTAs' splits, in order
        const int n = min(kFewWarps, (longest - r0 + SPLIT - 1) / SPLIT - o * kFewWarps);
        float fa[kFewWarps], fb[kFewWarps];
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) {
          fa[w] = 1.f;
          fb[w] = 0.f;
          if (w >= n) continue;
          const uint32_t at = base + M::OVER + (uint32_t)(w * kFewRows + frow) * 8;
          float m, l;
          if (CTAS > 1) {
            const uint32_t far = map_to_rank(at, (uint32_t)o);
            m = ld_cluster_f32(far);
            l = ld_cluster_f32(far + 4);
          } else {
            m = ld_shared_f32(at);
            l = ld_shared_f32(at + 4);
          }
          join(FM, m, fa[w], fb[w]);
          FL = __fmaf_rn(l, fb[w], __fmul_rn(FL, fa[w]));
        }
#pragma unroll 2
        for (int d = fd; d < fd + dims; ++d) {
          const uint32_t at = base + (uint32_t)(frow * D + d) * 4;
          const uint32_t far = CTAS > 1 ? map_to_rank(at, (uint32_t)o) : at;
          float v[kFewWarps];
#pragma unroll
          for (int w = 0; w < kFewWarps; ++w) {
            v[w] = 0.f;
            if (w < n) v[w] = CTAS > 1 ? ld_cluster_f32(far + w * kFewRows * D * 4) : ld_shared_f32(far + w * kFewRows * D * 4);
          }
          float x = tot[frow * D + d];
#pragma unroll
          for (int w = 0; w < kFewWarps; ++w)
            if (w < n) x = __fmaf_rn(v[w], fb[w], __fmul_rn(x, fa[w]));
          tot[frow * D + d] = x;
        }
      }
    }
    sync();  // the partial results are read: the rings may be refilled
  }
  __syncthreads();
  if (frow < rows) {
    uint16_t* dst = out + ((int64_t)(first + frow / G) * Hq + kh * G + frow % G) * D;
    const int splits = attn::num_splits(R, first + frow / G);
    for (int d = fd; d < fd + dims; d += 2)
      *reinterpret_cast<uint32_t*>(dst + d) =
          pack_bf16x2(row_out(tot[frow * D + d], FL, splits), row_out(tot[frow * D + d + 1], FL, splits));
  }
}

template <int KIND, int D>
__global__ void __launch_bounds__(kFewWarps * 32, 3)
    few_kernel(const uint16_t* __restrict__ q, int64_t ldq, int Hq, int Hkv, Cache C, Rows R, int T, int few,
               const int32_t* __restrict__ list, const Counts* __restrict__ counts, uint16_t* __restrict__ out,
               float scale_log2, bool clusters) {
  extern __shared__ __align__(1024) uint8_t smem_few[];  // pages' swizzle counts from 128-byte boundaries
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = Hq / Hkv;
  pdl_wait();  // the plan (and the caller's q and store) are complete from here on
  pdl_trigger();
  const int total = counts->few * Hkv;
  // A cluster a tile where that takes two rounds of clusters at most (a few rows of long contexts);
  // a CTA a tile otherwise, and where no row can have more splits than a CTA has warps. One decode row
  // at 32000 tokens 520 -> 99 us, 16 rows at 4000 151 -> 62 us (8 kv-heads of 128, e4m3).
  const bool together = clusters && total <= 2 * (int)gridDim.x / kFewCluster;
  const int ctas = together ? kFewCluster : 1;
  for (int item = (int)blockIdx.x / ctas; item < total; item += (int)gridDim.x / ctas) {
    const int first = list[T - 1 - item / Hkv], kh = item % Hkv;
    const int rows = tile_tokens(R.q_seq, first, T, few, lane) * G;
#define BI_FEW_TILE(NT, CTAS) \
  few_tile<KIND, D, NT, CTAS>(q, ldq, Hq, Hkv, G, C, R, first, rows, kh, out, scale_log2, smem_few, warp, lane)
    if (together) {
      if (rows <= 8) BI_FEW_TILE(1, kFewCluster);
      else BI_FEW_TILE(2, kFewCluster);
    } else {
      if (rows <= 8) BI_FEW_TILE(1, 1);
      else BI_FEW_TILE(2, 1);
    }
#undef BI_FEW_TILE
    __syncthreads();  // shared memory is free for the next tile
  }
}

}  // namespace attnq8
}  // namespace bi
