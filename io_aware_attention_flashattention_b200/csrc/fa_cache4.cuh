// fa_cache4.cuh -- a key/value cache held in 4 bits: appending rows, reading rows back,
// and the attention of single tokens and short drafts over it.
//
// A row (one token's K or V of one head, d values) is held as d codes of 4 bits and a pair
// (scale, zero) in the model's 16-bit type:
//   zero = min x, scale = (max x - min x) / 15, code = round((x - zero) / scale),
//   value = scale * code + zero.
// Rows lie in pages of `page` tokens: codes [n_pages, 2 (K, V), Hkv, page, d/2] bytes, the
// even channel of a pair in the low four bits; params [n_pages, 2, Hkv, page] words, the
// scale in the low half. Token t of sequence b is slot t % page of page
// table[b][t / page]. Pages hold whole groups of 16 tokens, so no group straddles two.
#pragma once

#include <type_traits>

#include "fa_ptx.cuh"
#include "fa_score.cuh"

namespace fa {
namespace cache4 {

struct Layout {
  uint8_t* codes;
  uint32_t* params;
  const int* table;  // [B, max_pages]
  long long n_pages;
  int max_pages;
  int Hkv;
  int page;   // tokens per page: a power of two from 16 to 256
  int shift;  // its logarithm
};

// Index of the first row (slot 0) of a page's K (which = 0) or V (1) of one head.
__host__ __device__ __forceinline__ long long page_row(long long id, int which, int hk, int Hkv,
                                                       int shift) {
  return ((id * 2 + which) * Hkv + hk) << shift;
}

// The page that holds token t of a sequence with this page table row; -1 if t lies outside
// the table or its entry outside the cache.
__host__ __device__ __forceinline__ long long page_of(const int* table_row, int max_pages,
                                                      long long n_pages, int shift, long long t) {
  if (t < 0) return -1;
  const long long at = t >> shift;
  if (at >= max_pages) return -1;
  const long long id = table_row[at];
  return id >= 0 && id < n_pages ? id : -1;
}

template <Elt E>
__device__ __forceinline__ float2 scale_zero(uint32_t w) {
  return unpack2<E>(w);
}

// Division of numbers below 2^31 by a number the host knows, as one product and a shift
// (Granlund and Montgomery, "Division by invariant integers using multiplication", 1994):
// with l = ceil(log2 n) and m = ceil(2^(31 + l) / n), x / n = x m >> (31 + l).
struct Divisor {
  uint32_t n, m;
  int s;
  __device__ __forceinline__ uint32_t quotient(uint32_t x) const {
    return static_cast<uint32_t>((static_cast<unsigned long long>(x) * m) >> s);
  }
};

// (w & mask) | bits in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(bits));
  return r;
}

// ------------------------------------------------------------------ append and read
//
// A row by D / 16 neighbouring lanes, 16 channels (32 bytes, 8 bytes of codes) each. The
// kernels move 2 D + D / 2 + 4 bytes per row and are bound by memory as long as a thread
// spends few enough instructions on its 16 channels: row indices by products instead of
// divisions, the quotient by a reciprocal (see quantise), codes to floats by the mantissa.
// B16 Hkv8 n2048 ragged d128 (130 MB each): the append 95 us with a division for each value,
// 58 us with one for those near a half, 36 us this way; the read 58 us with 64-bit divisions
// for the row, 37 us this way.

struct RowsParams {
  uint16_t* K;  // read by the append, written by the read
  uint16_t* V;
  Layout L;
  const int* positions;
  const int* counts;  // or null
  Divisor n, hkv;
  uint32_t rows;  // B * Hkv * n
};

// What a thread's row is: its batch entry's token t lies in `row` of the cache (-1: nowhere).
template <int D>
struct RowAt {
  uint32_t r;
  int lane, which;
  bool counted;
  long long row;
};

template <int D>
__device__ __forceinline__ RowAt<D> row_at(const RowsParams& p) {
  constexpr int G = D / 16;  // lanes of a row
  RowAt<D> a;
  a.r = blockIdx.x * (256u / G) + threadIdx.x / G;
  a.lane = threadIdx.x % G;
  a.which = blockIdx.y;
  a.row = -1;
  a.counted = false;
  if (a.r >= p.rows) return a;
  const uint32_t bh = p.n.quotient(a.r), b = p.hkv.quotient(bh);
  const int t = static_cast<int>(a.r - bh * p.n.n), hk = static_cast<int>(bh - b * p.hkv.n);
  a.counted = p.counts == nullptr || t < p.counts[b];
  if (!a.counted) return a;
  const long long pos = static_cast<long long>(p.positions[b]) + t;
  const long long id = page_of(p.L.table + static_cast<size_t>(b) * p.L.max_pages, p.L.max_pages,
                               p.L.n_pages, p.L.shift, pos);
  if (id < 0) {
    if (a.lane == 0) atomicOr(&g_status, kStatusBadPage);
    return a;
  }
  a.row = page_row(id, a.which, hk, p.L.Hkv, p.L.shift) + (pos & (p.L.page - 1));
  return a;
}

template <Elt E>
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (E == Elt::BF16)
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Codes round((x - lo) / scale), halves to even, of 16 values given as 8 pairs. With inv the
// correctly rounded reciprocal, q0 = d inv and r = d - q0 scale (exact), fma(r, inv, q0) is
// the correctly rounded quotient (Markstein, "Computation of elementary functions on the IBM
// RISC System/6000 processor", 1990), in pairs and without a branch: ties are common among
// 16-bit values, so a test for them sent most warps to a division each. Adding 1.5 * 2^23
// rounds and leaves the code in the low bits; the sum of the shifted bits holds a constant
// beside the codes. Where the scale is below the type's normal numbers (codes may pass 15, and
// the products may leave the normal range) or x - lo may pass 32 bits the quotients are formed
// one by one, of halves: 0.5 x - 0.5 lo stays in range, and halving is exact (16-bit values
// and their differences are multiples of 2^-133, 32 bits hold those of 2^-149).
template <Elt E>
__device__ __forceinline__ uint2 quantise(const uint32_t (&w)[8], float lo, float hi, float scale) {
  constexpr float kMagic = 12582912.0f;
  constexpr float kNormal = E == Elt::BF16 ? 1e-30f : 6.2e-5f;
  uint32_t code[2] = {0u, 0u};
  if (scale >= kNormal && hi - lo < 3.0e38f) {
    const float inv = __frcp_rn(scale);
    const float2 inv2 = make_float2(inv, inv), neg2 = make_float2(-scale, -scale);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 d = fadd2(unpack2<E>(w[k]), make_float2(-lo, -lo));
      const float2 q0 = fmul2(d, inv2);
      const float2 q = ffma2(ffma2(q0, neg2, d), inv2, q0);
      const float2 y = fadd2(q, make_float2(kMagic, kMagic));
      code[k / 4] += (__float_as_uint(y.x) << (8 * (k % 4))) +
                     (__float_as_uint(y.y) << (8 * (k % 4) + 4));
    }
    // the sum of 0x4B400000 << 4k over k = 0..7, modulo 2^32
    constexpr uint32_t kConstant = 0x4B400000u + (0x4B400000u << 4) + (0x4B400000u << 8) +
                                   (0x4B400000u << 12) + (0x4B400000u << 16) +
                                   (0x4B400000u << 20) + (0x4B400000u << 24) +
                                   (0x4B400000u << 28);
    code[0] -= kConstant;
    code[1] -= kConstant;
  } else if (scale > 0.0f) {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float2 x = unpack2<E>(w[k / 2]);
      const float d = __fsub_rn(0.5f * ((k & 1) ? x.y : x.x), 0.5f * lo);
      const float c = fminf(fmaxf(rintf(__fdiv_rn(d, 0.5f * scale)), 0.0f), 15.0f);
      code[k / 8] |= static_cast<uint32_t>(c) << (4 * (k % 8));
    }
  }
  return make_uint2(code[0], code[1]);
}

template <int D, Elt E>
__global__ void __launch_bounds__(256) append_kernel(const RowsParams p) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int G = D / 16;
  const RowAt<D> a = row_at<D>(p);
  if (a.row < 0) return;  // all lanes of a row alike
  const uint4* src = reinterpret_cast<const uint4*>((a.which ? p.V : p.K) +
                                                    static_cast<size_t>(a.r) * D) + 2 * a.lane;
  const uint4 w0 = src[0], w1 = src[1];
  const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
  // the least x and the least -x (NaN wins), of pairs, then of both halves as one pair
  uint32_t lows = w[0], highs = w[0] ^ 0x80008000u;
#pragma unroll
  for (int k = 1; k < 8; ++k) {
    lows = min2_nan<E>(lows, w[k]);
    highs = min2_nan<E>(highs, w[k] ^ 0x80008000u);
  }
  uint32_t both = min2_nan<E>(__byte_perm(lows, highs, 0x5410), __byte_perm(lows, highs, 0x7632));
  const unsigned group = ((1u << G) - 1u) << ((threadIdx.x & 31) / G * G);
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1)
    both = min2_nan<E>(both, __shfl_xor_sync(group, both, o));
  const float2 ends = unpack2<E>(both);
  const float lo = ends.x, hi = -ends.y;
  // The step rounded to 16 bits is the step that codes are made for and values read with;
  // the zero is one of the row's own values, so it needs no rounding. Each bound is divided
  // by itself: their difference may pass the largest bf16.
  constexpr float kFifteenth = 1.0f / 15.0f;
  const uint32_t sz = pack2<E>(__fsub_rn(__fmul_rn(hi, kFifteenth), __fmul_rn(lo, kFifteenth)), lo);
  const uint2 code = quantise<E>(w, lo, hi, scale_zero<E>(sz).x);
  reinterpret_cast<uint2*>(p.L.codes + a.row * (D / 2))[a.lane] = code;
  if (a.lane == 0) p.L.params[a.row] = sz;
}

// The same rows back as 16-bit values [B, Hkv, n, D]; rows behind a count are zeros.
template <int D, Elt E>
__global__ void __launch_bounds__(256) read_kernel(const RowsParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const RowAt<D> a = row_at<D>(p);
  if (a.r >= p.rows) return;
  uint32_t o[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
  if (a.row >= 0) {
    const uint2 code = reinterpret_cast<const uint2*>(p.L.codes + a.row * (D / 2))[a.lane];
    const float2 sz = scale_zero<E>(p.L.params[a.row]);
    const float2 s2 = make_float2(sz.x, sz.x), z2 = make_float2(sz.y, sz.y);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t c = (k < 4 ? code.x : code.y) >> (8 * (k % 4));
      // 2^23 + code, less 2^23
      const float2 v = fadd2(make_float2(__uint_as_float(and_or(c, 15u, 0x4B000000u)),
                                         __uint_as_float(and_or(c >> 4, 15u, 0x4B000000u))),
                             make_float2(-8388608.0f, -8388608.0f));
      const float2 x = ffma2(s2, v, z2);
      o[k] = pack2<E>(x.x, x.y);
    }
  }
  uint4* dst = reinterpret_cast<uint4*>((a.which ? p.V : p.K) + static_cast<size_t>(a.r) * D) +
               2 * a.lane;
  dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
  dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

// ------------------------------------------------------------------ attend
//
// One CTA of kWarps warps takes one K/V head of one sequence, up to 8 * NT query rows (the
// group's heads times the draft's tokens) and a piece of the sequence; every warp takes
// every kWarps-th step of 32 tokens of it and keeps its own running maximum, sum and
// output, joined at the end over the warps and then (by combine_kernel) over the pieces.
// Products on the tensor cores (mma.m16n8k16, fp32 accumulators) with tokens, then
// channels, as the 16 rows, so that up to 8 query rows cost one product:
//   S^T[16 tokens x 8 rows] = codes[16 x d] Q^T[d x 8]
//   O^T[d x 8] += V codes^T[d x 16] P^T[16 x 8]
// A step's codes and pairs (32 (d + 8) bytes) come through two buffers of shared memory of
// the warp's own, one step ahead by asynchronous copies, and leave them in the order
// that the products take them: a thread reads whole words of 8 codes, and any order of the
// summed index will do as long as both operands follow it. Two codes of a word become a
// pair of 16-bit floats c - 8 by a shift, one logical operation and one packed addition. (16 +
// c would save K the addition, at the price of a shift: no faster, and less exact.) With
// sum q = qs:
//   s = scale_k * (sum q (c - 8)) + (zero_k + 8 scale_k) qs
// and, with P' = P scale_v:
//   o = sum P' (c - 8) + sum P (zero_v + 8 scale_v).
// P' enters its product as a sum of two bf16, P' rounded and what that leaves (2^-17 of P'
// is lost): one bf16 alone put the output 2.4e-3 off in f16 (B1 H32 Hkv4 L131071 d128),
// ten times that type's own rounding. f16 would not do: scales times weights of long rows
// fall below its normal range. The reference maximum of a row moves only when a score
// passes it by more than 2^8, as in the forward.
// Bound by memory (d + 8 bytes per token and head, K and V), then by the instructions that
// unpack codes: shifts and logical operations issue at half rate, and their pipe is 57% busy, the
// issue slots 67%, at 2.9 TB/s (B64 H32 Hkv8 d128, 2048 to 8192 tokens, cap 50).

constexpr int kWarps = 4;
constexpr int kGroup = 16;  // tokens of one product: the rows that a page holds whole
constexpr int kStep = 32;   // tokens per step of a warp: two groups

struct AttendParams {
  const uint16_t* Q;  // [B, H, Nq, D]
  uint16_t* O;
  float* LSE;  // [B, H, Nq]
  const int* lengths;
  float* part_o;   // [B * H * Nq][n_pieces][D], pieces > 1 only
  float2* part_ml;  // [B * H * Nq][n_pieces] (maximum in log2 units, sum)
  Layout L;
  ScoreParams score;
  int H, Nq;
  int rows;      // query rows per K/V head: group * Nq
  Divisor nq;
  int row_tiles;  // CTAs they take
  int n_pieces;
  int piece;  // steps per piece, a multiple of kWarps
  int wl;     // < 0: no window
  float scale_log2;
};

template <Elt E>
__device__ __forceinline__ void mma_16n8k16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                            uint32_t b1) {
  if constexpr (E == Elt::BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The 8 x 8 matrix of 16-bit elements that a warp holds as an accumulator's half, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Nibbles j of both halves of a word as a pair of 16-bit floats code - 8: 128 + code (bf16) or
// 1024 + code (f16), the code being the mantissa's last bits, and one exact addition. The
// mantissa of f16 has room for the nibble four bits up as well: 1024 + 16 code, and one
// exact multiplication and addition, which spares the shift (f16 B1 H32 Hkv4 L131071 31.9 ->
// 31.5 us).
template <Elt E, int j>
__device__ __forceinline__ uint32_t centred(uint32_t w) {
  uint32_t r;
  if constexpr (E == Elt::BF16)
    asm("add.rn.bf16x2 %0, %1, %2;"
        : "=r"(r) : "r"(and_or(w >> (4 * j), 0x000F000Fu, 0x43004300u)), "r"(0xC308C308u));
  else if constexpr (j % 2 == 0)
    asm("add.rn.f16x2 %0, %1, %2;"
        : "=r"(r) : "r"(and_or(w >> (4 * j), 0x000F000Fu, 0x64006400u)), "r"(0xE408E408u));
  else  // / 16 - 72
    asm("fma.rn.f16x2 %0, %1, %2, %3;"
        : "=r"(r) : "r"(and_or(w >> (4 * j - 4), 0x00F000F0u, 0x64006400u)), "r"(0x2C002C00u),
                    "r"(0xD480D480u));
  return r;
}

__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool wide) {
  if (wide)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

template <int N>
__device__ __forceinline__ void shared_words(uint32_t (&r)[N], uint32_t at) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(at));
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r[0]) : "r"(at));
}

// The ring's place of one 16-byte unit of a row, units of K and V moved within 128 bytes so
// that the reads below meet no bank twice (K: rows g' of 8 lanes are 4 apart; V: the rows of
// 16 lanes are 1 apart and half read).
template <int D>
__host__ __device__ constexpr int ring_unit(int which, int row, int unit) {
  const int at = row * (D / 32) + unit;
  return which == 0 ? at ^ (((row >> 2) & 1) << 2)
                    : (D == 128 ? at ^ (((row >> 1) & 1) << 1) : at);
}

// kMods: kScoreCap, kScoreBias and kScoreFar.
template <int D, Elt E, int NT, int kMods>
__global__ void __launch_bounds__(kWarps * 32)
    attend_kernel(const AttendParams p) {
  constexpr int R = 8 * NT;      // query rows of the CTA
  constexpr int KS = D / 16;     // steps of the score product
  constexpr int MT = D / 16;     // 16-channel blocks of the output
  constexpr int kRow = D / 2;               // bytes of a row's codes
  constexpr int kHalf = kGroup * kRow;      // of a group's K or V codes
  constexpr int kPart = 2 * kHalf + 2 * kGroup * 4;  // of a group: codes, then the pairs
  constexpr int kRing = kWarps * 4 * kPart;
  constexpr int kJoin = kWarps * 8 * (D + 4 + 2) * 4;
  // the buffers, and after the loop the warps' results
  __shared__ __align__(128) uint8_t smem[kRing > kJoin ? kRing : kJoin];
  float (*const sm_o)[8][D + 4] = reinterpret_cast<float (*)[8][D + 4]>(smem);
  float (*const sm_m)[8] = reinterpret_cast<float (*)[8]>(smem + kWarps * 8 * (D + 4) * 4);
  float (*const sm_l)[8] = reinterpret_cast<float (*)[8]>(smem + kWarps * 8 * (D + 5) * 4);
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  unsigned at = blockIdx.x;
  const int piece = static_cast<int>(at % p.n_pieces);
  at /= p.n_pieces;
  const int rt = static_cast<int>(at % p.row_tiles);
  at /= p.row_tiles;
  const int hk = static_cast<int>(at % p.L.Hkv), b = static_cast<int>(at / p.L.Hkv);
  const int row0 = rt * R;
  const int n_rows = min(R, p.rows - row0);
  const int group = p.score.group;
  // row r of this K/V head: its head of the group and its token of the draft, and its row of
  // [B, H, Nq]
  auto head_of = [&](int r) -> int { return static_cast<int>(p.nq.quotient(r)); };
  auto out_row = [&](int r) -> size_t {
    const int h = head_of(r);
    return (static_cast<size_t>(b) * p.H + hk * group + h) * p.Nq + (r - h * p.Nq);
  };

  const long long room = static_cast<long long>(p.L.max_pages) << p.L.shift;
  int len = max(p.lengths[b], 0);
  if (len > room) {
    len = static_cast<int>(room);
    if (threadIdx.x == 0) atomicOr(&g_status, kStatusBadPage);
  }
  const int pos0 = len - p.Nq;  // of the draft's first token
  const int first = p.wl < 0 || p.wl >= pos0 ? 0 : pos0 - p.wl;
  const int g_hi = (len + kGroup - 1) / kGroup;                    // groups with tokens
  const int s_lo = first / kStep, s_hi = g_hi / 2 + (g_hi & 1);      // steps
  const int* table = p.L.table + static_cast<size_t>(b) * p.L.max_pages;

  // this warp's steps: s_lo + piece * p.piece + warp, every kWarps-th of the piece, then the
  // same of piece + n_pieces, ... (more than one only where a length passes the given bound)
  auto next = [&](int x, int& in) -> int {
    in += kWarps;
    x += kWarps;
    if (in >= p.piece) {
      in = 0;
      x += (p.n_pieces - 1) * p.piece;
    }
    return x;
  };

  // Copies of one group into part 2 * buffer + (0, 1) of the warp's ring: a thread's units of
  // the K and V codes (unit lane of each 512 bytes) and one of the 32 pairs. A group without
  // a page takes page 0 instead (the reads stay inside the cache) and is marked. So is a group in
  // front of every row's window, which is not looked up (its page may be gone): the first half
  // of step s_lo may be one, and no other, so only the first call looks for it.
  const uint32_t ring = smem_u32(smem) + warp * (4 * kPart);
  const unsigned page_groups = p.L.shift - 4;  // log2 of the groups per page
  const unsigned n_pages = static_cast<unsigned>(p.L.n_pages);
  const unsigned heads2 = 2 * p.L.Hkv, slots = p.L.page - 1;
  const size_t v_rows = static_cast<size_t>(p.L.Hkv) << p.L.shift;  // from K's rows to V's
  constexpr int kUnits = kHalf / 512;  // copies of a thread per half: 2 (D = 128) or 1
  constexpr int kPerRow = D / 32;      // units of a row
  const uint8_t* const codes_lane = p.L.codes + lane * 16;
  const uint32_t* const params_lane = p.L.params + (lane & 15) + (lane < 16 ? 0 : v_rows);
  uint32_t dst_k[kUnits], dst_v[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int unit = u * 32 + lane;
    dst_k[u] = ring + ring_unit<D>(0, unit / kPerRow, unit % kPerRow) * 16;
    dst_v[u] = ring + kHalf + ring_unit<D>(1, unit / kPerRow, unit % kPerRow) * 16;
  }
  unsigned bad = 0;  // bits of the parts whose group is not there; 4 up: because it lies in front
  // the step x; kFirst: its groups in front of `first` are marked
  auto issue = [&](int x, int buffer, auto kFirst) {
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const int grp = 2 * x + part, slot = 2 * buffer + part;
      if (decltype(kFirst)::value && grp < first / kGroup) {
        bad |= 0x11u << slot;
      } else if (grp < g_hi) {
        unsigned id = static_cast<unsigned>(table[grp >> page_groups]);
        bad &= ~(0x11u << slot);
        if (id >= n_pages) {
          bad |= 1u << slot;
          id = 0;
        }
        const size_t row = ((static_cast<size_t>(id) * heads2 + hk) << p.L.shift) +
                           ((grp << 4) & slots);
        const uint8_t* k = codes_lane + row * kRow;
        const uint8_t* v = k + v_rows * kRow;
        const uint32_t off = slot * kPart;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
          copy_async(dst_k[u] + off, k + u * 512, true);
          copy_async(dst_v[u] + off, v + u * 512, true);
        }
        copy_async(ring + 2 * kHalf + lane * 4 + off, params_lane + row, false);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // the queries, as the score product's second operand, and the sums of their channels
  uint4 qw[NT][D / 32];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = row0 + nt * 8 + g;
#pragma unroll
    for (int w = 0; w < D / 32; ++w)
      qw[nt][w] = r < p.rows ? *reinterpret_cast<const uint4*>(p.Q + out_row(r) * D +
                                                               t * (D / 4) + 8 * w)
                             : make_uint4(0u, 0u, 0u, 0u);
  }
  int use = s_lo + piece * p.piece + warp, use_in = 0;
  int ahead = use, ahead_in = 0;
  issue(ahead, 0, std::true_type{});
  ahead = next(ahead, ahead_in);
  uint32_t q[NT][KS][2];
  float qs[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      const uint4 x = qw[nt][w];
      const float2 f0 = unpack2<E>(x.x), f1 = unpack2<E>(x.y), f2 = unpack2<E>(x.z),
                   f3 = unpack2<E>(x.w);
      sum += ((f0.x + f0.y) + (f1.x + f1.y)) + ((f2.x + f2.y) + (f3.x + f3.y));
      q[nt][2 * w][0] = __byte_perm(x.x, x.z, 0x5410);      // channels 0, 4
      q[nt][2 * w][1] = __byte_perm(x.x, x.z, 0x7632);      // 1, 5
      q[nt][2 * w + 1][0] = __byte_perm(x.y, x.w, 0x5410);  // 2, 6
      q[nt][2 * w + 1][1] = __byte_perm(x.y, x.w, 0x7632);  // 3, 7
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    qs[nt][0] = __shfl_sync(0xffffffffu, sum, 8 * t);
    qs[nt][1] = __shfl_sync(0xffffffffu, sum, 8 * t + 4);
  }
  // this thread's rows of the products' results: 2t and 2t + 1 of each 8
  int pos[NT][2];
  float slope_neg[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = min(row0 + nt * 8 + 2 * t + e, p.rows - 1), h = head_of(r);
      pos[nt][e] = pos0 + (r - h * p.Nq);
      if constexpr ((kMods & kScoreBias) != 0)
        slope_neg[nt][e] =
            -p.score.slopes[hk * group + h] * p.score.slope_mul * p.scale_log2;
    }

  // Without a cap the scores are in log2 units from the start: c goes into scale and zero.
  const float c = p.scale_log2;
  const float c_in = (kMods & kScoreCap) ? 1.0f : c;
  // m: the reference maximum (0 before there is one: bound is -inf then); bound: where a
  // score moves it; l, z: this thread's parts of the sums of P and of P (zero_v + 8 scale_v)
  float m[NT][2], bound[NT][2], l[NT][2], z[NT][2], o[NT][MT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      bound[nt][e] = -INFINITY;
      m[nt][e] = l[nt][e] = z[nt][e] = 0.0f;
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nt][mt][e] = 0.0f;
  }
  const int own = (g >> 1) + (g & 1) * 4;  // the token of the products' row g; g + 8: own + 8
  const int edge_hi = pos0 - kGroup + 1, edge_lo = p.wl < 0 ? -1 : len - 1 - p.wl;
  // this thread's reads of a part
  uint32_t src_k[2], src_v[4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int byte = t * (D / 8);
    src_k[h] = ring + ring_unit<D>(0, own + 8 * h, byte / 16) * 16 + byte % 16;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int byte = g * (D / 16);
    src_v[i] = ring + kHalf + ring_unit<D>(1, 4 * i + t, byte / 16) * 16 + byte % 16;
  }
  const uint32_t src_p = ring + 2 * kHalf + own * 4;

  for (int buffer = 0; use < s_hi; buffer ^= 1) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();  // every lane's copies are in, and every lane is done with the other buffer
    issue(ahead, buffer ^ 1, std::false_type{});
    ahead = next(ahead, ahead_in);
    const int step = use;
    use = next(use, use_in);
#pragma unroll 1
    for (int part = 0; part < 2; ++part) {
      const int k0 = (2 * step + part) * kGroup, slot = 2 * buffer + part;
      if (k0 >= len) break;
      if ((bad >> slot) & 1u) {  // not there; noted if for want of a page
        if (lane == 0 && ((bad >> slot) & 0x10u) == 0u) atomicOr(&g_status, kStatusBadPage);
        continue;
      }
      const uint32_t off = slot * kPart;
      // scores: (token own + 8h, row 2t + e) is s[nt][2h + e]
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = 0.0f;
      {
        uint32_t k[2][D / 32];  // channels t * D / 4 on of the two tokens
#pragma unroll
        for (int h = 0; h < 2; ++h) shared_words(k[h], src_k[h] + off);
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          const uint32_t a0[4] = {centred<E, 0>(k[0][w]), centred<E, 0>(k[1][w]),
                                  centred<E, 1>(k[0][w]), centred<E, 1>(k[1][w])};
          const uint32_t a1[4] = {centred<E, 2>(k[0][w]), centred<E, 2>(k[1][w]),
                                  centred<E, 3>(k[0][w]), centred<E, 3>(k[1][w])};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_16n8k16<E>(s[nt], a0, q[nt][2 * w][0], q[nt][2 * w][1]);
            mma_16n8k16<E>(s[nt], a1, q[nt][2 * w + 1][0], q[nt][2 * w + 1][1]);
          }
        }
      }
      float2 ksz[2], vsz[2];  // scale, and zero + 8 scale
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w[1];
        shared_words(w, src_p + off + 32 * h);
        ksz[h] = unpack2<E>(w[0]);
        ksz[h].y = fmaf(8.0f, ksz[h].x, ksz[h].y) * c_in;
        ksz[h].x *= c_in;
        shared_words(w, src_p + off + 64 + 32 * h);
        vsz[h] = unpack2<E>(w[0]);
        vsz[h].y = fmaf(8.0f, vsz[h].x, vsz[h].y);
      }
      uint32_t u[4 * NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          u[4 * nt + e] =
              __float_as_uint(fmaf(ksz[e >> 1].x, s[nt][e], ksz[e >> 1].y * qs[nt][e & 1]));
      if constexpr ((kMods & kScoreCap) != 0) {
        tanh_scores<4 * NT, (kMods & kScoreFar) != 0>(u, p.score);
#pragma unroll
        for (int e = 0; e < 4 * NT; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * c);
      }
      if constexpr ((kMods & kScoreBias) != 0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            u[4 * nt + e] = __float_as_uint(
                fmaf(slope_neg[nt][e & 1],
                     static_cast<float>(pos[nt][e & 1] - (k0 + own + 8 * (e >> 1))),
                     __uint_as_float(u[4 * nt + e])));
      }
      // rows' keys are [pos - wl, pos]: tests only where the 16 tokens cross an edge
      if (k0 > edge_hi || k0 < edge_lo) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = k0 + own + 8 * h;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (key > pos[nt][e] || (p.wl >= 0 && pos[nt][e] - key > p.wl))
                u[4 * nt + 2 * h + e] = __float_as_uint(-INFINITY);
          // A row takes nothing of a token that it does not see, whatever the slot holds, but
          // its weight of 0 times a NaN would be one: so such a token counts as 0 here, and
          // makes NaN the rows that see it. (x - x is 0 unless x is an infinity or NaN; zero +
          // 8 scale is one of them if either part is.)
          if (vsz[h].y - vsz[h].y != 0.0f) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (__uint_as_float(u[4 * nt + 2 * h + e]) != -INFINITY) z[nt][e] = NAN;
            vsz[h] = make_float2(0.0f, 0.0f);
          }
        }
      }
      bool up = false;
      float top[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          s[nt][e] = __uint_as_float(u[4 * nt + e]);
          s[nt][2 + e] = __uint_as_float(u[4 * nt + 2 + e]);
          top[nt][e] = fmaxf(s[nt][e], s[nt][2 + e]);
          up = up || top[nt][e] > bound[nt][e];
        }
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float alpha[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = top[nt][e];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
            const float was = bound[nt][e] == -INFINITY ? -INFINITY : m[nt][e];
            const float now = fmaxf(was, x);
            alpha[e] = ex2_approx(was - (now == -INFINITY ? 0.0f : now));  // 0 at first
            m[nt][e] = now == -INFINITY ? 0.0f : now;
            bound[nt][e] = now + 8.0f;
            l[nt][e] *= alpha[e];
            z[nt][e] *= alpha[e];
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][mt][e] *= alpha[e & 1];
        }
      }
      uint32_t pb[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[e] = ex2_approx(s[nt][e] - m[nt][e & 1]);
          l[nt][e & 1] += w[e];
          z[nt][e & 1] = fmaf(w[e], vsz[e >> 1].y, z[nt][e & 1]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float a = w[2 * h] * vsz[h].x, b = w[2 * h + 1] * vsz[h].x;
          const uint32_t pk = pack_bf16x2(a, b);
          const float2 back = unpack2<Elt::BF16>(pk);
          pb[nt][h] = transpose8(pk);
          pb[nt][2 + h] = transpose8(pack_bf16x2(a - back.x, b - back.y));
        }
      }
      uint32_t v[4][D / 64];  // tokens t, 4 + t, 8 + t, 12 + t: channels g * D / 8 on
#pragma unroll
      for (int i = 0; i < 4; ++i) shared_words(v[i], src_v[i] + off);
#pragma unroll
      for (int w = 0; w < D / 64; ++w) {
        const uint32_t lo0 = __byte_perm(v[0][w], v[1][w], 0x5410);
        const uint32_t lo1 = __byte_perm(v[2][w], v[3][w], 0x5410);
        const uint32_t hi0 = __byte_perm(v[0][w], v[1][w], 0x7632);
        const uint32_t hi1 = __byte_perm(v[2][w], v[3][w], 0x7632);
        const uint32_t a[4][4] = {
            {centred<Elt::BF16, 0>(lo0), centred<Elt::BF16, 1>(lo0),
             centred<Elt::BF16, 0>(lo1), centred<Elt::BF16, 1>(lo1)},
            {centred<Elt::BF16, 2>(lo0), centred<Elt::BF16, 3>(lo0),
             centred<Elt::BF16, 2>(lo1), centred<Elt::BF16, 3>(lo1)},
            {centred<Elt::BF16, 0>(hi0), centred<Elt::BF16, 1>(hi0),
             centred<Elt::BF16, 0>(hi1), centred<Elt::BF16, 1>(hi1)},
            {centred<Elt::BF16, 2>(hi0), centred<Elt::BF16, 3>(hi0),
             centred<Elt::BF16, 2>(hi1), centred<Elt::BF16, 3>(hi1)}};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_16n8k16<Elt::BF16>(o[nt][4 * w + i], a[i], pb[nt][0], pb[nt][1]);
            mma_16n8k16<Elt::BF16>(o[nt][4 * w + i], a[i], pb[nt][2], pb[nt][3]);
          }
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");

  // The warps' rows joined, eight at a time: a warp's row 2t + e, channels g * D / 8 + 8w + 2i +
  // (0, 1), into shared memory, then D / 4 threads a row.
  constexpr int T = D / 4;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    __syncthreads();  // the ring, or the eight rows before, are free
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], d);
        z[nt][e] += __shfl_xor_sync(0xffffffffu, z[nt][e], d);
      }
      const int r = 2 * t + e;
      if (g == 0) {
        sm_m[warp][r] = bound[nt][e] == -INFINITY ? -INFINITY : m[nt][e];
        sm_l[warp][r] = l[nt][e];
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        *reinterpret_cast<float2*>(&sm_o[warp][r][g * (D / 8) + 2 * mt]) =
            make_float2(o[nt][mt][e] + z[nt][e], o[nt][mt][2 + e] + z[nt][e]);
    }
    __syncthreads();
    const int here = min(8, n_rows - 8 * nt);
    for (int r = threadIdx.x / T; r < here; r += kWarps * 32 / T) {
      const int ch = (threadIdx.x % T) * 4;
      float top = sm_m[0][r];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sm_m[w][r]);
      const float base = top == -INFINITY ? 0.0f : top;
      float sum = 0.0f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2_approx(sm_m[w][r] - base);
        const float4 v = *reinterpret_cast<const float4*>(&sm_o[w][r][ch]);
        sum = fmaf(f, sm_l[w][r], sum);
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z);
        acc.w = fmaf(f, v.w, acc.w);
      }
      const size_t row = out_row(row0 + 8 * nt + r);
      if (p.n_pieces > 1) {
        const size_t slot = row * p.n_pieces + piece;
        if (ch == 0) p.part_ml[slot] = make_float2(top, sum);
        if (sum > 0.0f || sum != sum) *reinterpret_cast<float4*>(p.part_o + slot * D + ch) = acc;
      } else {
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        *reinterpret_cast<uint2*>(p.O + row * D + ch) =
            make_uint2(pack2<E>(acc.x * inv, acc.y * inv), pack2<E>(acc.z * inv, acc.w * inv));
        if (ch == 0)
          p.LSE[row] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
      }
    }
  }
}

// A row's pieces joined by a CTA of kJoinThreads: each thread four channels of every
// (4 kJoinThreads / D)-th piece, the sums joined over shared memory. 512 threads: the reads of
// a hundred pieces are then a few loads deep (B1 H32 Hkv4 L131071, 103 pieces: attention and
// join 37.7 us with 128 threads, 31.4 us with 512).
constexpr int kJoinThreads = 512;

template <int D, Elt E>
__global__ void __launch_bounds__(kJoinThreads)
    combine_kernel(const float* part_o, const float2* part_ml, uint16_t* O, float* LSE,
                   int n_pieces) {
  constexpr int T = D / 4, S = kJoinThreads / T;  // threads of a piece, pieces at a time
  __shared__ float sm_top[kJoinThreads / 32], sm_sum[S];
  __shared__ float4 sm_o[S][T];
  pdl_wait();
  pdl_launch_dependents();
  const size_t row = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int at = threadIdx.x % T, first = threadIdx.x / T;
  const float2* ml = part_ml + row * n_pieces;
  float top = -INFINITY;
  for (int k = threadIdx.x; k < n_pieces; k += kJoinThreads) top = fmaxf(top, ml[k].x);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  if (lane == 0) sm_top[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) top = fmaxf(top, sm_top[w]);
  const float base = top == -INFINITY ? 0.0f : top;
  const float4* src = reinterpret_cast<const float4*>(part_o) + row * n_pieces * T + at;
  float sum = 0.0f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = first; k < n_pieces; k += S) {
    const float2 w = ml[k];
    if (w.y == 0.0f) continue;  // a piece without keys left its output unwritten
    const float4 v = src[static_cast<size_t>(k) * T];
    const float f = ex2_approx(w.x - base);
    sum = fmaf(f, w.y, sum);
    acc.x = fmaf(f, v.x, acc.x);
    acc.y = fmaf(f, v.y, acc.y);
    acc.z = fmaf(f, v.z, acc.z);
    acc.w = fmaf(f, v.w, acc.w);
  }
  sm_o[first][at] = acc;
  if (at == 0) sm_sum[first] = sum;
  __syncthreads();
  if (first != 0) return;
#pragma unroll 4
  for (int k = 1; k < S; ++k) {
    const float4 v = sm_o[k][at];
    sum += sm_sum[k];
    acc.x += v.x;
    acc.y += v.y;
    acc.z += v.z;
    acc.w += v.w;
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  reinterpret_cast<uint2*>(O + row * D)[at] =
      make_uint2(pack2<E>(acc.x * inv, acc.y * inv), pack2<E>(acc.z * inv, acc.w * inv));
  if (at == 0) LSE[row] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
}

}  // namespace cache4
}  // namespace fa
