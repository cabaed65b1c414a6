// fa_score.cuh -- shaped scores: what the forward, the backward and the attention over a
// 4-bit cache share. A score is
//   t = cap * tanh(scale * q.k / cap) - slope_h * |i - j|   (either term may be off),
// and query i sees key j iff both lie in one document, i - wl <= j (wl >= 0), and
// j <= i + wr (wr >= 0; causal is wr = 0) or j lies in the document's prefix.
//
// Documents are runs of a row given by their offsets, so the keys that a query sees, and
// the queries that see a key, are intervals, and both ends of the interval grow with the
// row index. The kernels use that twice: the tiles that a block of rows walks are those
// from its first row's lower end to its last row's upper end, and a tile needs no element
// test where it lies between the last row's lower end and the first row's upper end.
#pragma once

#include "fa_ptx.cuh"

namespace fa {

// Bits of the kernels' kScore parameter (0: plain scores, nothing of this file is used).
constexpr int kScoreOn = 1;    // documents, prefix, shared K/V heads
constexpr int kScoreCap = 2;   // tanh cap
constexpr int kScoreBias = 4;  // distance bias
constexpr int kScoreFar = 8;   // with kScoreCap: a cap above kNearCap (see tanh_scores)

struct ScoreParams {
  const float* slopes;  // [H], or null
  const int* docs;      // [B, n_docs + 1] offsets, or null: one document [0, N)
  const int* prefix;    // [B, n_docs] prefix lengths, or null
  int n_docs;           // >= 1
  int H;                // query heads per batch entry
  int group;            // query heads that share a K/V head
  // tanh(x) = s * q(s^2) with x = s * scale / cap: the polynomial's coefficients with the
  // powers of scale / cap folded in, the same times c (what turns a tanh to a score in log2
  // units), and the bound on s^2 up to which it holds (see make_score)
  float q5[5], cq5[5];
  float lim5;
  float cap_in;       // scale / cap
  float cap_in2;      // 2 * log2(e) * scale / cap, for the form on the exponential; 0: no cap
  float slope_mul;    // a slope times this is in units of the scores before c (below)
};

// tanh(x) / x as a polynomial in x^2 for |x| <= 0.8: least squares at Chebyshev nodes with
// Lawson reweighting toward the minimax fit; largest relative error 1.0e-6.
constexpr double kTanhLimit5 = 0.8;
constexpr double kTanhQ5[5] = {0.9999989944, -0.3332537202, 0.1323056571, -0.04918014249,
                               0.01210013727};

// The form of tanh on the exponential is off by up to 6.3e-7, times the cap: up to this cap by 4e-5
// of a score, a twelfth of a rounding of its weight to f16.
constexpr float kNearCap = 64.0f;

struct Span {
  int lo, hi;
};

// The document of token i: the last m with offsets[m] <= i (so empty documents are passed
// over), or -1 in front of the first. n_docs: behind the last. Ends for any contents.
__host__ __device__ __forceinline__ int doc_of(const int* offsets, int n_docs, int i) {
  int a = -1, b = n_docs + 1;  // offsets[a] <= i < offsets[b], with -inf and +inf at the ends
  while (b - a > 1) {
    const int m = (a + b) >> 1;
    if (offsets[m] <= i) a = m; else b = m;
  }
  return a;
}

// Token i's document [s, e) within [0, N) and the end of its prefix; an empty document
// for padding. docs and prefix are the batch entry's own rows.
__host__ __device__ __forceinline__ void doc_span(const int* docs, const int* prefix, int n_docs,
                                                  int N, int i, int& s, int& e, int& ahead) {
  int m = 0;
  s = 0;
  e = N;
  if (docs != nullptr) {
    m = doc_of(docs, n_docs, i);
    if (m < 0 || m >= n_docs) {
      s = e = ahead = 0;
      return;
    }
    s = docs[m] < 0 ? 0 : docs[m];
    e = docs[m + 1] > N ? N : docs[m + 1];
    if (e < s) e = s;
  }
  int p = prefix != nullptr ? prefix[m] : 0;
  p = p < 0 ? 0 : (p > e - s ? e - s : p);
  ahead = s + p;
}

// Keys [lo, hi) that query i sees; empty for i >= N and for padding.
__host__ __device__ __forceinline__ Span keys_of_query(const int* docs, const int* prefix,
                                                       int n_docs, int N, int wl, int wr, int i) {
  if (i < 0 || i >= N) return Span{0, 0};
  int s, e, ahead;
  doc_span(docs, prefix, n_docs, N, i, s, e, ahead);
  Span k{s, e};
  if (wl >= 0 && i - wl > k.lo) k.lo = i - wl;
  if (wr >= 0) {
    const int r = i + wr + 1 > ahead ? i + wr + 1 : ahead;
    if (r < k.hi) k.hi = r;
  }
  if (k.hi < k.lo) k.hi = k.lo;
  return k;
}

// Queries [lo, hi) that see key j; empty for j >= N and for padding.
__host__ __device__ __forceinline__ Span queries_of_key(const int* docs, const int* prefix,
                                                        int n_docs, int N, int wl, int wr, int j) {
  if (j < 0 || j >= N) return Span{0, 0};
  int s, e, ahead;
  doc_span(docs, prefix, n_docs, N, j, s, e, ahead);
  Span q{s, e};
  if (wr >= 0 && j >= ahead && j - wr > q.lo) q.lo = j - wr;
  if (wl >= 0 && j + wl + 1 < q.hi) q.hi = j + wl + 1;
  if (q.hi < q.lo) q.hi = q.lo;
  return q;
}

// The first and last tokens of rows [r0, r1] that lie in a document (first > last if none).
__host__ __device__ __forceinline__ void real_rows(const int* docs, int n_docs, int N, int r0,
                                                   int r1, int& first, int& last) {
  first = r0;
  last = r1 < N - 1 ? r1 : N - 1;
  if (docs != nullptr) {
    if (docs[0] > first) first = docs[0];
    if (docs[n_docs] - 1 < last) last = docs[n_docs] - 1;
  }
}

// Rows [lo, hi) hold the tokens of documents; the others are padding. The bounds of tests that
// no row of a tile meets where there is no padding (rows from N on read as zeros).
__device__ __forceinline__ Span padding_bounds(const int* docs, int n_docs, int N) {
  if (docs == nullptr) return Span{0, 0x7fffffff};
  return Span{docs[0], docs[n_docs] >= N ? 0x7fffffff : docs[n_docs]};
}

// 128-wide tiles [lo, hi) that hold every key some query of rows [r0, r0 + 127] sees.
__host__ __device__ __forceinline__ Span key_tiles_of_rows(const int* docs, const int* prefix,
                                                           int n_docs, int N, int wl, int wr,
                                                           int r0) {
  int first, last;
  real_rows(docs, n_docs, N, r0, r0 + 127, first, last);
  if (first > last) return Span{0, 0};
  const Span a = keys_of_query(docs, prefix, n_docs, N, wl, wr, first);
  const Span b = keys_of_query(docs, prefix, n_docs, N, wl, wr, last);
  if (b.hi <= a.lo) return Span{0, 0};
  return Span{a.lo / 128, (b.hi + 127) / 128};
}

// 128-wide tiles [lo, hi) that hold every query that sees some key of rows [r0, r0 + 127].
__host__ __device__ __forceinline__ Span query_tiles_of_keys(const int* docs, const int* prefix,
                                                             int n_docs, int N, int wl, int wr,
                                                             int r0) {
  int first, last;
  real_rows(docs, n_docs, N, r0, r0 + 127, first, last);
  if (first > last) return Span{0, 0};
  const Span a = queries_of_key(docs, prefix, n_docs, N, wl, wr, first);
  const Span b = queries_of_key(docs, prefix, n_docs, N, wl, wr, last);
  if (b.hi <= a.lo) return Span{0, 0};
  return Span{a.lo / 128, (b.hi + 127) / 128};
}

// Rows of a tile in shared memory (D / 64 chunks of 128-byte rows, `first` the first row's
// token) that are padding, made zeros by one warp before the products that read them: the
// weights of padding are 0, but times a NaN there they would be NaN. Called by the warp that
// issues the products, once the tile has landed. Few tiles hold padding, and inlined into the
// issuer's loop these stores slowed every step of the backward (B1 H8 N16384 d128 by 3%, with
// no documents at all; B2 H16 Hkv4 N4096 in documents by 9%, as a call by 4%).
template <int D>
__device__ __noinline__ void zero_rows(uint8_t* tile, int chunk_bytes, int rows, int first, int lo,
                                       int hi) {
  for (int u = threadIdx.x & 31; u < rows * 8; u += 32) {
    const int at = first + u / 8;
    if (at < lo || at >= hi)
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
        *reinterpret_cast<uint4*>(tile + c * chunk_bytes + u * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  __syncwarp();
}
template <int D>
__device__ __forceinline__ void zero_padding(uint8_t* tile, int chunk_bytes, int rows, int first,
                                             const Span& real) {
  if (first < real.lo || first + rows > real.hi)
    zero_rows<D>(tile, chunk_bytes, rows, first, real.lo, real.hi);
}

// s * q(S) for a pair of scores, on the FMA pipe, with S = s * s.
template <int n>
__device__ __forceinline__ float2 odd_poly2(float2 S, const float (&q)[n]) {
  float2 r = make_float2(q[n - 1], q[n - 1]);
#pragma unroll
  for (int k = n - 2; k >= 0; --k) r = ffma2(r, S, make_float2(q[k], q[k]));
  return r;
}
template <int n>
__device__ __forceinline__ float odd_poly(float s, const float (&q)[n]) {
  const float S = s * s;
  float r = q[n - 1];
#pragma unroll
  for (int k = n - 2; k >= 0; --k) r = fmaf(r, S, q[k]);
  return s * r;
}

// A batch entry's offsets and prefixes copied to shared memory (room for `room` ints) by the
// whole CTA, where they fit: the searches above are chains of dependent loads. docs and prefix
// are moved to the copy. Every thread of the CTA calls it. In the backward, together with
// key tiles ordered by rank, it took forward and backward at B3 H8 Hkv2 N1531 d64 (5
// documents a row) from 128 to 122 us; the forward gained nothing by it and searches in place.
__device__ __forceinline__ void share_documents(int* shared, int room, int n_docs,
                                                const int*& docs, const int*& prefix) {
  const int n = (docs ? n_docs + 1 : 0) + (prefix ? n_docs : 0);
  if (docs == nullptr || n > room) return;
  for (int k = threadIdx.x; k < n; k += blockDim.x)
    shared[k] = k <= n_docs ? docs[k] : prefix[k - n_docs - 1];
  __syncthreads();
  docs = shared;
  if (prefix) prefix = shared + n_docs + 1;
}

// tanh of one score: 1 - 2 / (1 + e^2x), by the exponential and the reciprocal of the MUFU
// unit. Absolute error up to 6.3e-7, which the cap multiplies: fit where the polynomial does not
// reach, |x| > 0.8 (9.5e-7 of the result there at most).
__device__ __forceinline__ float tanh_exp(float s, float cap_in2) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + ex2_approx(s * cap_in2)));
  return fmaf(-2.0f, r, 1.0f);
}

// tanh in place of n scores held by this thread (n even). Which form is a warp's choice
// (the branch would diverge otherwise): the polynomial where every score of the warp's piece
// lies within its reach (capped models keep most well inside the cap), else the one on the
// exponential. That form's error is absolute, and would show in scores near 0 of other rows
// under a large cap; so above kNearCap (kFar) each score of such a piece takes the one or the
// other by its own size, relative error 1.05e-6 either way. Taken at all caps it spilled
// registers and cost every capped forward (B1 H8 N16384 d128 causal, cap 50: 711 -> 785 us).
template <int n, bool kFar>
__device__ __forceinline__ void tanh_scores(uint32_t* s, const ScoreParams& p) {
  float2 S[n / 2];
  float top = 0.0f;
#pragma unroll
  for (int k = 0; k < n / 2; ++k) {
    const float2 x = make_float2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1]));
    S[k] = fmul2(x, x);
    top = fmax3(top, S[k].x, S[k].y);
  }
  if (__any_sync(0xffffffffu, !(top <= p.lim5))) {
    if constexpr (kFar) {
      constexpr float q[5] = {static_cast<float>(kTanhQ5[0]), static_cast<float>(kTanhQ5[1]),
                              static_cast<float>(kTanhQ5[2]), static_cast<float>(kTanhQ5[3]),
                              static_cast<float>(kTanhQ5[4])};
      constexpr float kReach = static_cast<float>(kTanhLimit5 * kTanhLimit5);
#pragma unroll
      for (int k = 0; k < n / 2; ++k) {
        const float2 raw = make_float2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1]));
        const float2 x = fmul2(raw, make_float2(p.cap_in, p.cap_in)), X = fmul2(x, x);
        const float2 r = fmul2(x, odd_poly2(X, q));
        const float fx = tanh_exp(raw.x, p.cap_in2), fy = tanh_exp(raw.y, p.cap_in2);
        s[2 * k] = __float_as_uint(X.x <= kReach ? r.x : fx);
        s[2 * k + 1] = __float_as_uint(X.y <= kReach ? r.y : fy);
      }
    } else {
#pragma unroll
      for (int k = 0; k < n; ++k)
        s[k] = __float_as_uint(tanh_exp(__uint_as_float(s[k]), p.cap_in2));
    }
  } else {
#pragma unroll
    for (int k = 0; k < n / 2; ++k) {
      const float2 r =
          fmul2(make_float2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])),
                odd_poly2(S[k], p.q5));
      s[2 * k] = __float_as_uint(r.x);
      s[2 * k + 1] = __float_as_uint(r.y);
    }
  }
}

// Bits [lo, hi) of a word (any lo and hi), the visible columns of 32: one test of a constant
// bit per score instead of an addition and a comparison. (shl by 32 or more gives 0.)
__device__ __forceinline__ uint32_t span_bits(int lo, int hi) {
  uint32_t a, b;
  asm("shl.b32 %0, %1, %2;" : "=r"(a) : "r"(0xffffffffu), "r"(max(lo, 0)));
  asm("shl.b32 %0, %1, %2;" : "=r"(b) : "r"(0xffffffffu), "r"(max(hi, 0)));
  return a & ~b;
}

// Adds slope_neg * |d0 + k| to n scores of consecutive columns k, in place; d0 is the (whole)
// distance of column 0 from this thread's row. Where all distances of the warp have one sign
// the bias runs in pairs, from an exact start every 16 columns (distances below 2^24 are
// exact in 32 bits) by at most seven additions.
template <int n>
__device__ __forceinline__ void bias_scores(uint32_t (&s)[n], int d0, float slope_neg) {
  const bool right = d0 >= 0, left = d0 + n - 1 <= 0;
  if (__all_sync(0xffffffffu, right) || __all_sync(0xffffffffu, left)) {
    const float sl = right ? slope_neg : -slope_neg;
#pragma unroll
    for (int k = 0; k < n; k += 16) {
      const float f = static_cast<float>(d0 + k) * sl;
      float2 b = make_float2(f, f + sl);
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const float2 x = fadd2(b, make_float2(__uint_as_float(s[k + e]),
                                              __uint_as_float(s[k + e + 1])));
        s[k + e] = __float_as_uint(x.x);
        s[k + e + 1] = __float_as_uint(x.y);
        b = fadd2(b, make_float2(2.0f * sl, 2.0f * sl));
      }
    }
  } else {
    const float f0 = static_cast<float>(d0);
#pragma unroll
    for (int k = 0; k < n; ++k)
      s[k] = __float_as_uint(
          fmaf(slope_neg, fabsf(f0 + static_cast<float>(k)), __uint_as_float(s[k])));
  }
}

}  // namespace fa
