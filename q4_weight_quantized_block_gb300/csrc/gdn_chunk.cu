// The gated delta rule over 64 rows at a time, on the tensor cores: chunks and prompts of fak_gdn_attn.
//
// With G_t = g_1 + .. + g_t since the chunk began, S the state before it, and
//   A_ts = beta_t exp(G_t - G_s) k_t.k_s (s < t),  P_ts = exp(G_t - G_s) q_t.k_s (s <= t),  T = (I + A)^-1,
// the rule's rows are
//   R = diag(beta) (V - diag(exp G) K S),   U = T R,   O = diag(exp G) Q S + (P T) R,
//   S' = exp(G_64) S + K^T diag(exp(G_64 - G)) U,
// so that what goes from chunk to chunk is three products: [K; Q] S, [T; P T] R (128 rows each) and K^T U.  T and P T
// depend on no state: a first kernel makes them for all chunks and heads (a record of 33 KB each, in a scratch), the second
// goes through a sequence's chunks.
//
// Precision.  The state is held in f32 registers; products keep 21 to 22 bits, and each is off by no more than that part of what its
// own row and column have: of a row's value, or of what the rows before brought to the column and the decays have left.
//   S, and U by the decays to the chunk's end, go as the sum of two f16 (q and k are f16 already), a value column scaled by one
// power of two: by m, the largest of exp(G_64) |S| and exp(G_64 - G) |V|, which goes to 2^6 .. 2^7.  With lengths of k of at most 1 and
// 0 <= beta <= 2 the U so decayed is at most 282 m and the S behind 140 m, below 2^15.2, and what f16 drops is below 2^-25, so 2^-31 m.
//   R is as large as a row's values, which differ at will.  It goes as two f16, the second times 2^11, where these hold what the
// column's rows need (halves_hold), T and P T times 2^14 in the same way; products with second parts have sums of their own.  A column
// of a million times a row's own value still goes so; where one does not, the warp takes the chunk's rows one by one in f32.
//   T and P T are made without their decays, by products of two f16 (|T| is at most 2 then; rows of P are by a power of two of a
// query of length 1 to 2) and multiplied by them at the end, so that their errors decay too.  Sums of decays are made in fixed
// point and kept as two f32, so that decays over neighbouring rows, differences of large sums, are off by 2^-22 only; those over a
// stretch of rows that are below 2^-126 are zeros.
//
// First kernel: a block takes a chunk and a key head, whose K K^T and Q K^T its value heads share, four warps: A and P;
// inverses of 16 x 16 blocks by substitution, joined to 32 and to 64, in place of A, and P T, in place of P, by m16n8k16
// instructions; both by their decays.  Steps that wait for one another on 64 x 64 matrices: 118 us for 128 chunks of 48 heads on 16 key
// heads, of which the records' 208 MB are 31 us; four blocks to an SM hide part of it.
//
// Second kernel: two CTAs to a head, 64 value columns each; a warp holds 16 columns, as S^T in the accumulators of m16n8k16 (64
// registers a thread).  Those are laid out as the next product's first operand is, so that S^T, R^T and U^T go from product
// to product in registers: S^T K^T, R^T T^T, U^T K.  A second warp to the same columns takes S^T and R^T as operands from shared
// memory and makes what only the output wants: S^T Q^T, R^T (P T)^T, the norm (its sums of squares from all eight such warps of
// the head, a chunk later), the gate, the store.  One more warp issues the copies of K, Q, V, z and the records.  316
// instructions of 8 cycles of the tensor cores for the state and 188 for the output, 4,032 cycles a chunk on each of an SM's four
// parts; a chunk takes 6,700 to 7,000 (3.5 to 3.6 us): one warp's way through three products, the splitting into f16 and the scales, and shared
// memory, whose operands a warp of 16 columns takes for itself alone.  (R, T and P T as two tf32 each, which hold any column: 521 us
// for a prompt's 128 chunks in place of 448.  Under one scale of the column's largest value, with no sums of their own for
// second parts and no look at what the rows need: 397, and rows beside one of 10^4 times their size lost digits.)
//
// What did not help (measured with R, T and P T as two f16 under one scale, which hold less; a chunk of 6,000 cycles then): the same products by tcgen05, 64 columns
// to a CTA (6,200 cycles a chunk: 128 rows of S, R or U go through shared memory for each of three products that wait for one
// another, some 700 cycles for a product and as many for its operand); one CTA to a head with eight warps that make their outputs
// too (12,700 for both halves of a head); two warps to the same columns, each with half of the keys and rows (6,400 to 7,000: what
// they exchange fills shared memory); several sequences' heads one behind the other in a CTA, split evenly (a chunk 7 % longer);
// records without the zeros above the diagonal (fewer bytes, yet 7 % more time of the second kernel for one prompt); records of the
// next 32 chunks beside the chunks of these (3 % less for one prompt of 8,192, at the price of the kernel twice).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "attn_device.cuh"
#include "fak.h"
#include "fak_device.cuh"
#include "fak_tc.cuh"
#include "gdn_device.cuh"
#include "kv_device.cuh"

namespace {

constexpr int kRows = 64;  // of a chunk
constexpr int kPrepThreads = 128;
constexpr int kLd = 20;  // f32 blocks of 16 x 16 in shared memory: rows of 80 bytes
constexpr int kPart = 16384;  // from a matrix's first parts to its second: 128 rows of 64 f16

// What a chunk's rows decay by, and their strengths: behind [T; P T], two parts, in a chunk's record for a head.
struct Decays {
  float keep[kRows];  // exp G_t
  float left[kRows];  // exp(G_64 - G_t)
  float beta[kRows];
  float up[kRows];    // what the rows of P T are times: powers of two
};
constexpr int kRecord = 2 * kPart + (int)sizeof(Decays);
static_assert(kRecord % 16 == 0, "bulk copies");

// Where records stand.  dense: chunk c of a sequence s, begin <= c < begin + length, at s * length + c - begin.  Else a sequence
// has its place behind those before it, chunk c at place + c, of which begin .. begin + length are there.  The place is told by
// the sequence's first row r0 (and by the sequences before it): r0 / 64 + s, or, where there are more sequences than rows make
// such chunks, r0 / kGdnFew, which rises by at least its chunks over a sequence of more than that many rows (no others have
// records).
// order: the sequences, those of many chunks first; null where all go at once.
struct Records {
  unsigned char* at;
  int begin, length;
  bool dense, by_row;
  int* order;
};
static_assert(kGdnFew <= 32, "a chunk and a row take two places");

FAK_DEV int place_of(const Records& r, int r0, int s) { return r.by_row ? r0 / kGdnFew : r0 / kRows + s; }

FAK_DEV int64_t record_of(const Records& r, const GdnSeq& d, int s, int c) {
  return r.dense ? (int64_t)s * r.length + (c - r.begin) : (int64_t)place_of(r, d.r0, s) + c - r.begin;
}

// A sequence's chunks in this launch.
FAK_DEV void chunks_of(const GdnParams& p, const Records& r, const GdnSeq& d, int s, int& begin, int& end) {
  const int rows = d.r1 - d.first;
  const int from = r.dense ? r.begin : r.begin - place_of(r, d.r0, s);
  begin = max(from, 0);
  end = !d.ok || (p.few && rows <= p.few) ? 0 : min((rows + kRows - 1) / kRows, from + r.length);
}

// Of the second kernel: NW warps of 16 columns, as many for their output, and the copies'.
constexpr int NW = 4;
struct C {
  static constexpr int cols = 16 * NW;                              // value columns of a CTA
  static constexpr int slices = kGdnDim / cols;                     // CTAs of a head
  static constexpr int threads = 64 * NW + 128;
  static constexpr int off_kq = 0;                                  // two stages of [K; Q]: two panels of 128 rows
  static constexpr int off_tp = off_kq + 2 * 32768;                 // two stages of [T; P T], two parts
  static constexpr int off_v = off_tp + 4 * kPart;                 // V: panels of 64 columns, 128 bytes
  static constexpr int off_frag = off_v + kRows * cols * 2;         // each warp's S (8) and R (4) as operands, two parts
  static constexpr int off_z = off_frag + NW * 12 * 1024;           // z: panels of 32 columns, 128 bytes
  static constexpr int off_out = off_z + kRows * cols * 4;          // the output, f32 or bf16: panels of 128 bytes
  static constexpr int off_dec = off_out + kRows * cols * 4;
  static constexpr int off_sum = off_dec + 2 * (int)sizeof(Decays);  // sums of squares [2][8][64], then 1 / norms [NW][64]
  static constexpr int off_down = off_sum + (2 * 8 + NW) * kRows * 4;  // one over the columns' scales
  static constexpr int off_by = off_down + cols * 4;                // the scales of R's columns, then the warps' ways
  static constexpr int off_bar = off_by + cols * 4 + 16;
  static constexpr int smem = off_bar + 128 + 1024;
  static_assert(smem <= 232448, "shared memory exceeds the 227 KB per-block limit");
};

constexpr int kRegs = 168;  // of a thread at launch

// Named barriers of a pair of warps (pair w: 3 w on).
enum Named { kBarS = 1, kBarR, kBarUsed };

enum Bars { kLand0, kLand1, kReady0, kReady1, kFree0, kFree1, kLandV, kVFree, kZ, kZFree, kSum0, kSum1, kOut, kOutFree, kBars };

FAK_DEV void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

FAK_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
FAK_DEV uint32_t rank_in_cluster() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
FAK_DEV uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
// A value into shared memory of a CTA of the cluster, its 4 bytes counted on a barrier there.
FAK_DEV void st_async(uint32_t addr, float x, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr),
               "r"(__float_as_uint(x)), "r"(bar)
               : "memory");
}

FAK_DEV bool try_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

FAK_DEV void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// Two f32 operations in one instruction.
FAK_DEV uint64_t pair_bits(float2 a) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a.x), "f"(a.y));
  return d;
}
FAK_DEV float2 bits_pair(uint64_t d) {
  float2 a;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(d));
  return a;
}
FAK_DEV float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair_bits(a)), "l"(pair_bits(b)));
  return bits_pair(d);
}
FAK_DEV float2 mul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair_bits(a)), "l"(pair_bits(b)));
  return bits_pair(d);
}
FAK_DEV float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(pair_bits(a)), "l"(pair_bits(b)), "l"(pair_bits(c)));
  return bits_pair(d);
}
FAK_DEV float2 both(float a) { return make_float2(a, a); }
FAK_DEV float2 bf16_pair(uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }

// Two f32 as the sum of two pairs of f16.
FAK_DEV void split_half(float x, float y, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(y), "f"(x));
  float a, b;  // x and y less their first parts: exact; f16 operands and -1 to an f32 sum (1 % of a prompt's time)
  asm("{\n .reg .b16 p, q, m;\n mov.b32 {p, q}, %2;\n mov.b16 m, 0xBC00;\n fma.rn.f32.f16 %0, p, m, %3;\n fma.rn.f32.f16 %1, q, m, %4;\n}"
      : "=f"(a), "=f"(b)
      : "r"(hi), "f"(x), "f"(y));
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(b), "f"(a));
}

// Two f32 as the sum of two pairs of f16, the second times 2^11: the second has f16's full exponents, and what both drop is below 2^-36.
FAK_DEV void split_wide(float2 x, uint32_t& hi, uint32_t& lo) {
  const float2 y = mul2(x, both(2048.0f));
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(x.y), "f"(x.x));
  float a, b;
  asm("{\n .reg .b16 p, q, m;\n mov.b32 {p, q}, %2;\n mov.b16 m, 0xE800;\n fma.rn.f32.f16 %0, p, m, %3;\n fma.rn.f32.f16 %1, q, m, %4;\n}"
      : "=f"(a), "=f"(b)
      : "r"(hi), "f"(y.x), "f"(y.y));
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(b), "f"(a));
}

// Columns of a row (from a multiple of 8 on) of a tile of f16 parts, its panels of 64 columns `panel` bytes apart, the
// second part `part` bytes behind the first.  Every value is made before the first is stored, so that none waits for a store's turn.
template <int N>
FAK_DEV void put_halves(unsigned char* tile, int panel, int part, int row, int col, const float2 (&x)[N / 2]) {
  uint32_t hi[N / 2], lo[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) split_half(x[i].x, x[i].y, hi[i], lo[i]);
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    const int c = col + i;
    unsigned char* at = tile + (c >> 6) * panel + row * 128 + ((((c >> 3) & 7) ^ (row & 7)) << 4);
    *reinterpret_cast<uint4*>(at) = make_uint4(hi[i / 2], hi[i / 2 + 1], hi[i / 2 + 2], hi[i / 2 + 3]);
    *reinterpret_cast<uint4*>(at + part) = make_uint4(lo[i / 2], lo[i / 2 + 1], lo[i / 2 + 2], lo[i / 2 + 3]);
  }
}

// Operands of m16n8k16, both parts, from a tile of rows of 64 f16.  A: rows r0 .. +15, columns c0 .. +15; B: the same rows,
// columns 8 j .. +7.
struct FragA {
  uint32_t hi[4], lo[4];
};
struct FragB {
  uint32_t hi[2], lo[2];
};
FAK_DEV void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
FAK_DEV void load_a(FragA& a, uint32_t tile, int r0, int c0, int lane) {
  const int row = r0 + (lane & 15);
  const uint32_t at = tile + row * 128 + ((((c0 >> 3) + (lane >> 4)) ^ (row & 7)) << 4);
  ldsm4(a.hi, at);
  ldsm4(a.lo, at + kPart);
}
FAK_DEV void load_b(FragB& b, uint32_t tile, int r0, int j, int lane) {
  const int row = r0 + (lane & 15);
  const uint32_t at = tile + row * 128 + ((j ^ (row & 7)) << 4) + (lane >> 4) * kPart;
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(b.hi[0]), "=r"(b.hi[1]), "=r"(b.lo[0]), "=r"(b.lo[1])
               : "r"(at)
               : "memory");
}
FAK_DEV void mma16(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// A product's 16 x 8 as an operand B.
FAK_DEV void turn_b(FragB& b, const float (&c)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t hi, lo;
    split_half(c[2 * i], c[2 * i + 1], hi, lo);
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(b.hi[i]) : "r"(hi));
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(b.lo[i]) : "r"(lo));
  }
}
// Two products' 16 x 8, beside each other, both parts, at rows r0 .. +15, columns 8 j .. +15 of a tile (WIDE: as split_wide has them).
template <bool WIDE>
FAK_DEV void put_tiles(uint32_t tile, int r0, int j, const float (&a)[4], const float (&b)[4], int lane) {
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float* x = (i < 2 ? a : b) + 2 * (i & 1);
    if constexpr (WIDE)
      split_wide(make_float2(x[0], x[1]), hi[i], lo[i]);
    else
      split_half(x[0], x[1], hi[i], lo[i]);
  }
  const int row = r0 + (lane & 15);
  const uint32_t at = tile + row * 128 + (((j + (lane >> 4)) ^ (row & 7)) << 4);
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3])
               : "memory");
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(at + kPart), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]),
               "r"(lo[3])
               : "memory");
}
// The same for one product.
FAK_DEV void put_block(unsigned char* tile, int r0, int j, const float (&c)[4], float sign, int lane) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = r0 + 8 * i + (lane >> 2);
    uint32_t hi, lo;
    split_half(sign * c[2 * i], sign * c[2 * i + 1], hi, lo);
    unsigned char* at = tile + row * 128 + ((j ^ (row & 7)) << 4) + 4 * (lane & 3);
    *reinterpret_cast<uint32_t*>(at) = hi;
    *reinterpret_cast<uint32_t*>(at + kPart) = lo;
  }
}

struct ChunkMaps {
  CUtensorMap k, q, v, z, out;
};

struct ChunkDebug {
  unsigned long long timeout_ns;
  int unreachable;  // a test's: 1 where K and Q are never to count as landed
};

FAK_DEV void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
FAK_DEV void stsm4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
FAK_DEV void mma16(float2 (&c)[2], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0].x), "+f"(c[0].y), "+f"(c[1].x), "+f"(c[1].y)
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two tiles of accumulators (16 x 8 each) as an operand A of 16 x 16, both parts.
FAK_DEV void split_a(uint32_t (&hi)[4], uint32_t (&lo)[4], const float2 (&x)[2], const float2 (&y)[2]) {
  split_half(x[0].x, x[0].y, hi[0], lo[0]);
  split_half(x[1].x, x[1].y, hi[1], lo[1]);
  split_half(y[0].x, y[0].y, hi[2], lo[2]);
  split_half(y[1].x, y[1].y, hi[3], lo[3]);
}
// A row of 128 bytes' 16-byte piece in a tile of 128-byte swizzle.
FAK_DEV uint32_t piece(int row, int at) { return row * 128 + ((at ^ (row & 7)) << 4); }

// 2^by for a column whose largest magnitude is m = 2^e 1.f, which goes to 2^6 1.f (zeros and infinities: as they are)
FAK_DEV int scale_by(float m) {
  const int e = (int)(__float_as_uint(m) >> 23);
  return e == 0 || e == 255 ? 0 : min(max(133 - e, -120), 120);
}
FAK_DEV float two_to(int by) { return __uint_as_float((uint32_t)(127 + by) << 23); }

// Whether f16 parts (split_wide's) hold a column of R, and its scale: m the largest of the column's |S| and |V|, `least` the least that a
// row of it goes by: its |V|, or what is left of rows before.  m goes to 2^10 .. 2^11, so that R, at most 25 m, stays below 2^15.7,
// and the parts drop 2^-46 m of it; of T, times 2^14, 2^-50.  `least` has to be 2^-22 m, for this to be no more than 2^-21 of it
// (a zero is not, but where all are), and m a number from 2^-100 on.
FAK_DEV bool halves_hold(float m, float least, int& by) {
  const int e = (int)(__float_as_uint(m) >> 23);
  by = m == 0.0f ? 0 : 137 - e;
  return m == 0.0f || (e >= 27 && e < 255 && least >= m * 2.384185791015625e-7f);
}

template <bool F32>
__global__ void __launch_bounds__(C::threads, 1) gdn_chunk_kernel(const __grid_constant__ GdnParams p,
                                                                  const __grid_constant__ ChunkMaps maps, Records records,
                                                                  ChunkDebug dbg, int* status) {
  extern __shared__ unsigned char raw[];
  unsigned char* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::off_bar);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::off_bar + 8 * kBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const int slice = blockIdx.x % C::slices, unit = blockIdx.x / C::slices;
  const int place = unit / p.nv, h = unit - place * p.nv, s = records.order ? records.order[place] : place;
  const KvSeq seq = kv_seq(p.c, s);
  const GdnSeq d = gdn_seq(p.c, seq, s);
  if (!d.ok) {
    if (threadIdx.x == 0) atomicCAS(status, 0, FAK_ERR_DEVICE);
    return;
  }
  const int rows = d.r1 - d.first;
  if (p.few && rows <= p.few) return;  // the steps' kernel's
  // Where starts fall, two sequences that are in range may have the same records: both are left out.
  if (!records.dense && p.c.n_seqs > 1) {
    bool falls = false, same = false;
    for (int i = threadIdx.x; i < p.c.n_seqs; i += C::threads) falls |= p.c.row_start[i + 1] < p.c.row_start[i];
    if (__syncthreads_or(falls)) {
      const int mine = place_of(records, d.r0, s), behind = mine + (rows + kRows - 1) / kRows;
      for (int i = threadIdx.x; i < p.c.n_seqs; i += C::threads) {
        const GdnSeq e = gdn_seq(p.c, kv_seq(p.c, i), i);
        const int n = e.r1 - e.first, at = place_of(records, e.r0, i);
        same |= i != s && e.ok && n > p.few && at < behind && mine < at + (n + kRows - 1) / kRows;
      }
      if (__syncthreads_or(same)) {
        if (threadIdx.x == 0) atomicCAS(status, 0, FAK_ERR_DEVICE);
        return;
      }
    }
  }
  const int col0 = slice * C::cols;
  int begin, end;
  chunks_of(p, records, d, s, begin, end);
  if (records.begin == 0)
    for (int row = d.r0 + (int)threadIdx.x / (C::cols / 4); row < d.first; row += C::threads / (C::cols / 4))
      gdn_put4(p.out, p.out_bf16, row * p.out_row + h * p.out_head + col0 + 4 * ((int)threadIdx.x % (C::cols / 4)), gdn_zero4());
  const int chunks = end - begin;  // counted from 0 below
  if (chunks <= 0) return;
  const int first_row = d.first + begin * kRows, rows_left = rows - begin * kRows;

  if (threadIdx.x == 0) {
    *abort = 0;
    for (int i = 0; i < kBars; ++i) mbar_init(&bar[i], i == kFree0 || i == kFree1 ? 2 * NW : i == kVFree || i == kZFree || i == kOut ? NW : 1);
    fence_mbar_init();
  }
  __syncthreads();
  cluster_sync();

  // One that runs out is recorded, and no wait of the block waits after it.
  auto wait = [&](int b, int phase) {
    bool done = mbar_try_wait(&bar[b], phase & 1) || *abort != 0;
    for (int i = 0; i < 512 && !done; ++i) done = mbar_try_wait(&bar[b], phase & 1);
    if (!done && !mbar_wait_bounded(&bar[b], phase & 1, abort, dbg.timeout_ns)) {
      if (!*abort) atomicCAS(status, 0, FAK_ERR_TIMEOUT);
      *abort = 1;
    }
    __syncwarp();
  };
  auto arrive = [&](int b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar[b]);
  };
  auto dead = [&]() { return __any_sync(0xffffffffu, *abort != 0); };

  // registers of a thread: 224 + 208 + 72 of the 3 * kRegs that the block has.  (The copies' warp wants more than 56, beside which
  // the others could have 232 and 208: 2 % longer for 8 chunks; 232 + 200 + 72: as long.)
  if (warp < NW)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
  else if (warp < 2 * NW)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  if (warp < NW) {
    // ------------------------------------------------------------------ 16 columns
    const int g = lane >> 2, q2 = 2 * (lane & 3);
    const uint32_t base = smem_u32(smem);
    // S^T: tile i, keys 8 i + q2 and the next; columns g and g + 8
    float* st = p.state + ((int64_t)d.slot * p.nv + h) * kGdnState + col0 + 16 * warp + g;
    const bool empty = d.fresh && begin == 0;
    float2 S[16][2];
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float* at = st + (8 * i + q2) * kGdnDim + 8 * u;
        S[i][u] = empty ? both(0.0f) : make_float2(at[0], at[kGdnDim]);
      }
    uint32_t v[4][4];  // of the next chunk: rows 16 i + q2 and the next, + 8; columns g, g + 8
    float most_v[2], least_v[2];  // of its columns: the largest and the smallest magnitude
    auto fetch_v = [&](int c) {
      wait(kLandV, c);
      const uint32_t tile = base + C::off_v + (warp >> 2) * kRows * 128;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        ldsm4_trans(v[i], tile + piece(16 * i + (lane & 7) + ((lane >> 4) << 3), (2 * warp + ((lane >> 3) & 1)) & 7));
      arrive(kVFree);
      const int have = rows_left - c * kRows;
      uint32_t hi[2] = {0, 0}, lo[2] = {0x7f807f80u, 0x7f807f80u};
      auto look = [&](uint32_t x, uint32_t y, int u) {  // two rows' magnitudes
        asm("max.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(hi[u]) : "r"(x));
        asm("min.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(lo[u]) : "r"(y));
      };
      if (have < kRows) {  // what stands behind the last row is another's, whatever it holds
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int row = 16 * i + 8 * (u >> 1) + q2;
            const uint32_t there = row + 1 < have ? 0xffffffffu : row < have ? 0xffffu : 0;
            v[i][u] &= there;
            look(v[i][u], v[i][u] | (~there & 0x7f807f80u), u & 1);
          }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int u = 0; u < 4; ++u) look(v[i][u], v[i][u], u & 1);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float2 a = bf16_pair(hi[u]), b = bf16_pair(lo[u]);
        most_v[u] = fmaxf(fabsf(a.x), fabsf(a.y));
        least_v[u] = fminf(fabsf(b.x), fabsf(b.y));
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          most_v[u] = fmaxf(most_v[u], __shfl_xor_sync(0xffffffffu, most_v[u], o));
          least_v[u] = fminf(least_v[u], __shfl_xor_sync(0xffffffffu, least_v[u], o));
        }
      }
    };
    auto most_of = [&](float& a, float& b) {  // over the four lanes of columns g and g + 8
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
      }
    };
    // the state's scale, column by column: S holds the state times 2^by
    float ms[2] = {};
    fetch_v(0);
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u) ms[u] = fmaxf(ms[u], fmaxf(fabsf(S[i][u].x), fabsf(S[i][u].y)));
    most_of(ms[0], ms[1]);
    int by[2];
    float down[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      by[u] = scale_by(ms[u]);
      down[u] = two_to(-by[u]);
#pragma unroll
      for (int i = 0; i < 16; ++i) S[i][u] = mul2(S[i][u], both(two_to(by[u])));
    }

    uint4* frag = reinterpret_cast<uint4*>(smem + C::off_frag) + warp * 24 * 32 + lane;
    float* downs = reinterpret_cast<float*>(smem + C::off_down) + 16 * warp;
    int *bys = reinterpret_cast<int*>(smem + C::off_by) + 16 * warp, *ways = reinterpret_cast<int*>(smem + C::off_by) + C::cols + warp;
    // Where a row's value alone is too little of its column (halves_hold): the values to the place of R, in the order of the output's
    // accumulators, and the decays of rows lane and lane + 32; then row by row by the least that value and what is left of those
    // before come to.
    auto look_closer = [&](int c, float (&by_row)[2]) {
      const int have = min(kRows, rows_left - c * kRows);
      const float* gates = p.g + (int64_t)(first_row + c * kRows) * p.nv + h;
#pragma unroll
      for (int i = 0; i < 2; ++i) by_row[i] = expf(gates[(int64_t)min(lane + 32 * i, have - 1) * p.nv]);
      float* o = reinterpret_cast<float*>(frag - lane + 16 * 32);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 a = bf16_pair(v[i >> 1][2 * (i & 1)]), b = bf16_pair(v[i >> 1][2 * (i & 1) + 1]);
        *reinterpret_cast<float4*>(o + i * 128 + 16 * g + 2 * q2) = make_float4(a.x, b.x, a.y, b.y);
      }
      __syncwarp();
      // column lane & 15
      const int from = 4 * (lane & 7), u = lane >> 3 & 1;
      const float s0 = __shfl_sync(0xffffffffu, ms[0] * down[0], from), s1 = __shfl_sync(0xffffffffu, ms[1] * down[1], from);
      const float v0 = __shfl_sync(0xffffffffu, most_v[0], from), v1 = __shfl_sync(0xffffffffu, most_v[1], from);
      float here = u ? s1 : s0, least = __uint_as_float(0x7f800000u);
      const float most = fmaxf(here, u ? v1 : v0);
#pragma unroll 4
      for (int t = 0; t < have; ++t) {
        const float e = __shfl_sync(0xffffffffu, t < 32 ? by_row[0] : by_row[1], t & 31);
        here = fmaxf(fabsf(o[(t >> 3) * 128 + 16 * (lane & 7) + 2 * (t & 7) + u]), e * here);
        least = fminf(least, here);
      }
      int by;
      return (bool)__all_sync(0xffffffffu, halves_hold(most, least, by));
    };
    // A chunk's rows one by one in f32, as gdn_step_kernel has them: where f16 parts do not hold R.  The rows' outputs go to their values'
    // places.  (22 us for 64 rows, whose way by f16 parts takes 3.6.)
    auto rows_one_by_one = [&](int c, const Decays* dec, const float (&by_row)[2]) {
      const int have = min(kRows, rows_left - c * kRows);
      const unsigned char* kq = smem + C::off_kq + (c & 1) * 32768;
      float* o = reinterpret_cast<float*>(frag - lane + 16 * 32) + 16 * g;
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) S[i][u] = mul2(S[i][u], both(down[u]));
#pragma unroll 1
      for (int t = 0; t < have; ++t) {
        float2* here = reinterpret_cast<float2*>(o + (t >> 3) * 128 + 2 * (t & 7));
        const float e = __shfl_sync(0xffffffffu, t < 32 ? by_row[0] : by_row[1], t & 31), beta = dec->beta[t];
        const float x[2] = {here->x, here->y};
        float2 k[16], y[2][2] = {};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          k[i] = __half22float2(*reinterpret_cast<const __half2*>(kq + (i >> 3) * 16384 + piece(t, i & 7) + 2 * q2));
#pragma unroll
          for (int u = 0; u < 2; ++u) y[u][i & 1] = fma2(k[i], S[i][u], y[u][i & 1]);
        }
        float a[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          a[u] = (y[u][0].x + y[u][0].y) + (y[u][1].x + y[u][1].y);
#pragma unroll
          for (int m = 1; m < 4; m <<= 1) a[u] += __shfl_xor_sync(0xffffffffu, a[u], m);
          a[u] = beta * (x[u] - e * a[u]);
          y[u][0] = y[u][1] = both(0.0f);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 q = __half22float2(*reinterpret_cast<const __half2*>(kq + 8192 + (i >> 3) * 16384 + piece(t, i & 7) + 2 * q2));
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            S[i][u] = fma2(k[i], both(a[u]), mul2(S[i][u], both(e)));
            y[u][i & 1] = fma2(q, S[i][u], y[u][i & 1]);
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          a[u] = (y[u][0].x + y[u][0].y) + (y[u][1].x + y[u][1].y);
#pragma unroll
          for (int m = 1; m < 4; m <<= 1) a[u] += __shfl_xor_sync(0xffffffffu, a[u], m);
        }
        if ((lane & 3) == 0) *here = make_float2(a[0], a[1]);  // (behind the shuffles: read by all four)
      }
      if (lane == 0) *ways = 1;
      asm volatile("bar.arrive %0, 64;" ::"r"(3 * warp + kBarR) : "memory");
      float most[2] = {};
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) most[u] = fmaxf(most[u], fmaxf(fabsf(S[i][u].x), fabsf(S[i][u].y)));
      most_of(most[0], most[1]);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        by[u] = scale_by(most[u]);
        down[u] = two_to(-by[u]);
#pragma unroll
        for (int i = 0; i < 16; ++i) S[i][u] = mul2(S[i][u], both(two_to(by[u])));
      }
    };
    for (int c = 0; c < chunks; ++c) {
      const Decays* dec = reinterpret_cast<const Decays*>(smem + C::off_dec) + (c & 1);
      const uint32_t kq = base + C::off_kq + (c & 1) * 32768, tp = base + C::off_tp + (c & 1) * 2 * kPart;
      wait(kReady0 + (c & 1), c >> 1);
      // S^T, as an operand, to the output's warp too; S^T K^T
      float2 ks[8][2] = {};
      ms[0] = ms[1] = 0.0f;
      // (beside the products: R's scales, and the state's next by what is left of S and of the rows' values)
      float left_most[2] = {}, ratio[2], uup[2], rup[2];
      int next[2];
      bool hold;
      if (c > 0) named_bar_sync(3 * warp + kBarUsed, 64);
      if ((lane & 3) == 0) {
        downs[g] = down[0];
        downs[g + 8] = down[1];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        uint32_t hi[4], lo[4];
        split_a(hi, lo, S[2 * k], S[2 * k + 1]);
        frag[2 * k * 32] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        frag[(2 * k + 1) * 32] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
#pragma unroll
        for (int u = 0; u < 2; ++u)
          ms[u] = fmaxf(fmaxf(fmaxf(ms[u], fabsf(S[2 * k][u].x)), fabsf(S[2 * k][u].y)),
                        fmaxf(fabsf(S[2 * k + 1][u].x), fabsf(S[2 * k + 1][u].y)));
        const float2 left = *reinterpret_cast<const float2*>(dec->left + 8 * k + q2);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float2 y = mul2(bf16_pair(v[k >> 1][2 * (k & 1) + u]), left);
          left_most[u] = fmaxf(fmaxf(left_most[u], fabsf(y.x)), fabsf(y.y));
        }
        if (k == 7) {
#pragma unroll
          for (int o = 1; o < 4; o <<= 1)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              ms[u] = fmaxf(ms[u], __shfl_xor_sync(0xffffffffu, ms[u], o));
              left_most[u] = fmaxf(left_most[u], __shfl_xor_sync(0xffffffffu, left_most[u], o));
            }
          const float all = dec->keep[kRows - 1];
          int rby[2];
          hold = true;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float most = ms[u] * down[u];
            hold &= halves_hold(fmaxf(most, most_v[u]), least_v[u], rby[u]);
            rup[u] = two_to(rby[u]);
            next[u] = scale_by(fmaxf(most * all, left_most[u]));
            ratio[u] = all * two_to(min(max(next[u] - by[u], -126), 127));
            uup[u] = two_to(min(max(next[u] - rby[u] - 14, -126), 127));  // (T is times 2^14)
          }
          if ((lane & 3) == 0) {
            bys[g] = rby[0];
            bys[g + 8] = rby[1];
          }
          if (lane == 0) *ways = 0;
          hold = __all_sync(0xffffffffu, hold);
        }
        const uint32_t panel = kq + (k >> 2) * 16384;
        const int at = 2 * (k & 3) + ((lane >> 3) & 1);
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
          uint32_t b[4], e[4];
          const int row = 8 * j + (lane & 7) + ((lane >> 4) << 3);
          ldsm4(b, panel + piece(row, at));
          ldsm4(e, panel + piece(row + 16, at));
          mma16(ks[j], lo, b[0], b[1]);
          mma16(ks[j + 1], lo, b[2], b[3]);
          mma16(ks[j + 2], lo, e[0], e[1]);
          mma16(ks[j + 3], lo, e[2], e[3]);
          mma16(ks[j], hi, b[0], b[1]);
          mma16(ks[j + 1], hi, b[2], b[3]);
          mma16(ks[j + 2], hi, e[0], e[1]);
          mma16(ks[j + 3], hi, e[2], e[3]);
        }
      }
      asm volatile("bar.arrive %0, 64;" ::"r"(3 * warp + kBarS) : "memory");
      // R^T = beta (V^T - exp(G) S^T K^T) by its columns' scales, as an operand
      if (!hold) {
        float by_row[2];
        if (!look_closer(c, by_row)) {
          rows_one_by_one(c, dec, by_row);
          if (c + 1 < chunks) fetch_v(c + 1);
          arrive(kFree0 + (c & 1));
          continue;
        }
        __syncwarp();
      }
      const float sup[2] = {down[0] * rup[0], down[1] * rup[1]};
      uint32_t rh[4][4], rl[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = 2 * i + e;
          const float2 keep = *reinterpret_cast<const float2*>(dec->keep + 8 * j + q2);
          const float2 beta = *reinterpret_cast<const float2*>(dec->beta + 8 * j + q2);
          const float2 bk = mul2(mul2(beta, both(-1.0f)), keep);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            ks[j][u] = fma2(mul2(bk, both(sup[u])), ks[j][u], mul2(bf16_pair(v[i][2 * e + u]), mul2(beta, both(rup[u]))));
            split_wide(ks[j][u], rh[i][2 * e + u], rl[i][2 * e + u]);
          }
        }
        frag[(16 + 2 * i) * 32] = make_uint4(rh[i][0], rh[i][1], rh[i][2], rh[i][3]);
        frag[(17 + 2 * i) * 32] = make_uint4(rl[i][0], rl[i][1], rl[i][2], rl[i][3]);
      }
      asm volatile("bar.arrive %0, 64;" ::"r"(3 * warp + kBarR) : "memory");
      if (c + 1 < chunks) fetch_v(c + 1);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        by[u] = next[u];
        down[u] = two_to(-next[u]);
      }
      // U^T = R^T T^T: rows 16 j .. of T by columns 16 i .., i <= j
      float2 ut[8][2] = {};
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        float2 low[4][2] = {};  // of the products with second parts, times 2^11
#pragma unroll
        for (int i = 0; i <= j + 1; ++i) {
          // two row blocks beside each other, where both have the columns
          uint32_t th[2][4], tl[2][4];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (i > j + u) continue;
            const int row = 16 * (j + u) + (lane & 7) + ((lane >> 4) << 3), at = 2 * i + ((lane >> 3) & 1);
            ldsm4(th[u], tp + piece(row, at));
            ldsm4(tl[u], tp + kPart + piece(row, at));
          }
#pragma unroll
          for (int w = 0; w < 3; ++w)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              if (i > j + u) continue;
              if (w == 0) {
                mma16(low[2 * u], rl[i], th[u][0], th[u][1]);
                mma16(low[2 * u + 1], rl[i], th[u][2], th[u][3]);
              } else if (w == 1) {
                mma16(low[2 * u], rh[i], tl[u][0], tl[u][1]);
                mma16(low[2 * u + 1], rh[i], tl[u][2], tl[u][3]);
              } else {
                mma16(ut[2 * (j + u)], rh[i], th[u][0], th[u][1]);
                mma16(ut[2 * (j + u) + 1], rh[i], th[u][2], th[u][3]);
              }
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int e = 0; e < 2; ++e) ut[2 * j + u][e] = fma2(low[u][e], both(1.0f / 2048.0f), ut[2 * j + u][e]);
      }
      // U^T diag(exp(G_64 - G)) in the next chunk's scale, as an operand
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 left = *reinterpret_cast<const float2*>(dec->left + 8 * j + q2);
#pragma unroll
        for (int u = 0; u < 2; ++u) ut[j][u] = mul2(ut[j][u], mul2(left, both(uup[u])));
      }
      uint32_t uh[4][4], ul[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) split_a(uh[i], ul[i], ut[2 * i], ut[2 * i + 1]);
      // S^T = exp(G_64) S^T + U^T K
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) S[i][u] = mul2(S[i][u], both(ratio[u]));
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          uint32_t b[4], e[4];
          const int row = 16 * i + (lane & 15), at = (j & 7) + (lane >> 4);
          const uint32_t panel = kq + (j >> 3) * 16384;
          ldsm4_trans(b, panel + piece(row, at));
          ldsm4_trans(e, panel + piece(row, at + 2));
          mma16(S[j], ul[i], b[0], b[1]);
          mma16(S[j + 1], ul[i], b[2], b[3]);
          mma16(S[j + 2], ul[i], e[0], e[1]);
          mma16(S[j + 3], ul[i], e[2], e[3]);
          mma16(S[j], uh[i], b[0], b[1]);
          mma16(S[j + 1], uh[i], b[2], b[3]);
          mma16(S[j + 2], uh[i], e[0], e[1]);
          mma16(S[j + 3], uh[i], e[2], e[3]);
        }
      arrive(kFree0 + (c & 1));
    }
    named_bar_sync(3 * warp + kBarUsed, 64);
    if (!*abort) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float* at = st + (8 * i + q2) * kGdnDim + 8 * u;
          at[0] = S[i][u].x * down[u];
          at[kGdnDim] = S[i][u].y * down[u];
        }
    }
  } else if (warp < 2 * NW) {
    // ------------------------------------------------------------------ their output
    const int w = warp - NW, g = lane >> 2, q2 = 2 * (lane & 3);
    const uint32_t base = smem_u32(smem);
    const int me = (int)rank_in_cluster();
    float* sums = reinterpret_cast<float*>(smem + C::off_sum);
    float* norms = sums + (2 * 8 + w) * kRows;
    float gain[2] = {1.0f, 1.0f};
    if (p.norm_w) {
      gain[0] = p.norm_w[col0 + 16 * w + g];
      gain[1] = p.norm_w[col0 + 16 * w + g + 8];
    }
    // The output of a chunk, o, is finished while the next chunk is on its way: the norm's sums come from the cluster's warps.
    float2 o[8][2];
    auto finish = [&](int c) {
      if (p.norm_w) {
        wait(kSum0 + (c & 1), c >> 1);
        try_cluster(&bar[kSum0 + (c & 1)], c >> 1 & 1);  // (an acquire of the others' stores)
        float2 y = both(0.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) y = add2(y, *reinterpret_cast<const float2*>(sums + ((c & 1) * 8 + i) * kRows + 2 * lane));
        __syncwarp();  // (the chunk before is done with the norms)
        *reinterpret_cast<float2*>(norms + 2 * lane) =
            make_float2(rsqrtf(fmaf(y.x, 1.0f / kGdnDim, p.eps)), rsqrtf(fmaf(y.y, 1.0f / kGdnDim, p.eps)));
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 r = *reinterpret_cast<const float2*>(norms + 8 * i + q2);
          o[i][0] = mul2(o[i][0], mul2(r, both(gain[0])));
          o[i][1] = mul2(o[i][1], mul2(r, both(gain[1])));
        }
      }
      if (p.z) {
        wait(kZ, c);
        const unsigned char* zs = smem + C::off_z + (w >> 1) * kRows * 128;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int at = 16 * (w & 1) + g + 8 * u;  // column of the panel
            const float a = *reinterpret_cast<const float*>(zs + piece(8 * i + q2, at >> 2) + 4 * (at & 3));
            const float b = *reinterpret_cast<const float*>(zs + piece(8 * i + q2 + 1, at >> 2) + 4 * (at & 3));
            o[i][u] = mul2(o[i][u], make_float2(gdn_silu(a), gdn_silu(b)));
          }
        arrive(kZFree);
      }
      if (c > 0) wait(kOutFree, c - 1);
      if constexpr (F32) {
        unsigned char* to = smem + C::off_out + (w >> 1) * kRows * 128;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int at = 16 * (w & 1) + g + 8 * u;
            *reinterpret_cast<float*>(to + piece(8 * i + q2, at >> 2) + 4 * (at & 3)) = o[i][u].x;
            *reinterpret_cast<float*>(to + piece(8 * i + q2 + 1, at >> 2) + 4 * (at & 3)) = o[i][u].y;
          }
      } else {
        const uint32_t to = base + C::off_out + (w >> 2) * kRows * 128;
#pragma unroll
        for (int i = 0; i < 8; i += 2)
          stsm4_trans(to + piece(8 * i + (lane & 7) + ((lane >> 4) << 3), (2 * w + ((lane >> 3) & 1)) & 7),
                      pack_bf16(o[i][0].x, o[i][0].y), pack_bf16(o[i][1].x, o[i][1].y), pack_bf16(o[i + 1][0].x, o[i + 1][0].y),
                      pack_bf16(o[i + 1][1].x, o[i + 1][1].y));
      }
      fence_async();
      arrive(kOut);
    };

    const uint4* frag = reinterpret_cast<const uint4*>(smem + C::off_frag) + w * 24 * 32 + lane;
    const float* downs = reinterpret_cast<const float*>(smem + C::off_down) + 16 * w;
    const int *bys = reinterpret_cast<const int*>(smem + C::off_by) + 16 * w, *ways = reinterpret_cast<const int*>(smem + C::off_by) + C::cols + w;
    for (int c = 0; c < chunks; ++c) {
      const Decays* dec = reinterpret_cast<const Decays*>(smem + C::off_dec) + (c & 1);
      const uint32_t kq = base + C::off_kq + (c & 1) * 32768, tp = base + C::off_tp + (c & 1) * 2 * kPart;
      if (c > 0) finish(c - 1);
      named_bar_sync(3 * w + kBarS, 64);
      // O^T = exp(G) S^T Q^T
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j][0] = o[j][1] = both(0.0f);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint4 x = frag[2 * k * 32], y = frag[(2 * k + 1) * 32];
        const uint32_t hi[4] = {x.x, x.y, x.z, x.w}, lo[4] = {y.x, y.y, y.z, y.w};
        const uint32_t panel = kq + 8192 + (k >> 2) * 16384;
        const int at = 2 * (k & 3) + ((lane >> 3) & 1);
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
          uint32_t b[4], e[4];
          const int row = 8 * j + (lane & 7) + ((lane >> 4) << 3);
          ldsm4(b, panel + piece(row, at));
          ldsm4(e, panel + piece(row + 16, at));
          mma16(o[j], lo, b[0], b[1]);
          mma16(o[j + 1], lo, b[2], b[3]);
          mma16(o[j + 2], lo, e[0], e[1]);
          mma16(o[j + 3], lo, e[2], e[3]);
          mma16(o[j], hi, b[0], b[1]);
          mma16(o[j + 1], hi, b[2], b[3]);
          mma16(o[j + 2], hi, e[0], e[1]);
          mma16(o[j + 3], hi, e[2], e[3]);
        }
      }
      // O^T += R^T (P T)^T, in the scales of R's columns and of P T's rows
      named_bar_sync(3 * w + kBarR, 64);
      if (*ways) {  // made row by row
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint4 x = frag[(16 + j) * 32];
          o[j][0] = make_float2(__uint_as_float(x.x), __uint_as_float(x.z));
          o[j][1] = make_float2(__uint_as_float(x.y), __uint_as_float(x.w));
#pragma unroll
          for (int u = 0; u < 2; ++u) o[j][u] = mul2(o[j][u], both(p.scale));
        }
        asm volatile("bar.arrive %0, 64;" ::"r"(3 * w + kBarUsed) : "memory");
      } else {
        const int rby[2] = {bys[g], bys[g + 8]};
        const float sc[2] = {downs[g] * two_to(rby[0] + 14), downs[g + 8] * two_to(rby[1] + 14)};
        const float rdown[2] = {p.scale * two_to(-14 - rby[0]), p.scale * two_to(-14 - rby[1])};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 keep = mul2(*reinterpret_cast<const float2*>(dec->keep + 8 * j + q2), *reinterpret_cast<const float2*>(dec->up + 8 * j + q2));
          o[j][0] = mul2(mul2(o[j][0], both(sc[0])), keep);
          o[j][1] = mul2(mul2(o[j][1], both(sc[1])), keep);
        }
        float2 low[8][2] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 x = frag[(16 + 2 * i) * 32], y = frag[(17 + 2 * i) * 32];
          const uint32_t rh[4] = {x.x, x.y, x.z, x.w}, rl[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int j = i; j < 4; ++j) {
            uint32_t ph[4], pl[4];
            const int row = 16 * j + (lane & 7) + ((lane >> 4) << 3), at = 2 * i + ((lane >> 3) & 1);
            ldsm4(ph, tp + 8192 + piece(row, at));
            ldsm4(pl, tp + kPart + 8192 + piece(row, at));
            mma16(low[2 * j], rl, ph[0], ph[1]);
            mma16(low[2 * j + 1], rl, ph[2], ph[3]);
            mma16(low[2 * j], rh, pl[0], pl[1]);
            mma16(low[2 * j + 1], rh, pl[2], pl[3]);
            mma16(o[2 * j], rh, ph[0], ph[1]);
            mma16(o[2 * j + 1], rh, ph[2], ph[3]);
          }
        }
        asm volatile("bar.arrive %0, 64;" ::"r"(3 * w + kBarUsed) : "memory");
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          // (one over a power of two)
          const float2 up = *reinterpret_cast<const float2*>(dec->up + 8 * j + q2);
          const float2 back = make_float2(__uint_as_float(0x7f000000u - __float_as_uint(up.x)), __uint_as_float(0x7f000000u - __float_as_uint(up.y)));
#pragma unroll
          for (int u = 0; u < 2; ++u)
            o[j][u] = mul2(mul2(fma2(low[j][u], both(1.0f / 2048.0f), o[j][u]), both(rdown[u])), back);
        }
      }
      arrive(kFree0 + (c & 1));
      // O, and its columns' share of the rows' sums of squares: to 8 rows' sums over 8 lanes, then one over the lanes' halves
      if (p.norm_w && !dead()) {
        if (w == 0 && lane == 0) mbar_arrive_expect_tx(&bar[kSum0 + (c & 1)], 8 * kRows * 4);
        float2 y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = fma2(o[j][0], o[j][0], mul2(o[j][1], o[j][1]));
        // lanes 16, then 8, then 4 apart: each keeps half of what it has, and adds the other's
#pragma unroll
        for (int m = 4; m >= 1; m >>= 1) {
          const bool high = lane & (4 * m);
#pragma unroll
          for (int j = 0; j < m; ++j) {
            const float2 mine = high ? y[j + m] : y[j], give = high ? y[j] : y[j + m];
            y[j].x = mine.x + __shfl_xor_sync(0xffffffffu, give.x, 4 * m);
            y[j].y = mine.y + __shfl_xor_sync(0xffffffffu, give.y, 4 * m);
          }
        }
        // tile of the lane: its bits 4, 3, 2
        const int row = 8 * ((lane >> 4 & 1) * 4 + (lane >> 3 & 1) * 2 + (lane >> 2 & 1)) + q2;
        const uint32_t at = smem_u32(sums + ((c & 1) * 8 + me * NW + w) * kRows + row), on = smem_u32(&bar[kSum0 + (c & 1)]);
#pragma unroll
        for (int i = 0; i < C::slices; ++i) {
          st_async(map_rank(at, i), y[0].x, map_rank(on, i));
          st_async(map_rank(at + 4, i), y[0].y, map_rank(on, i));
        }
      }
    }
    finish(chunks - 1);
  } else if (warp == 2 * NW) {
    // ------------------------------------------------------------------ the copies
    // A barrier takes a copy's bytes only when it is done with the copy before: after a wait that gave up no copy is issued,
    // and those that were are waited for before the block ends.
    const int hk = h / p.group;
    const unsigned char* record0 = records.at + (record_of(records, d, s, begin) * p.nv + h) * kRecord;
    int values = 0, copied = 0, gates = 0;  // chunks of which V, of which K, Q and the record, of which z was asked for
    auto load_v = [&](int c) {  // (which goes to registers amid the chunk before)
      if (c >= 1) wait(kVFree, c - 1);
      if (dead()) return;
      values = c + 1;
      if (elect_one()) {
        mbar_arrive_expect_tx(&bar[kLandV], kRows * C::cols * 2);
        tma_load_3d_tx(smem + C::off_v, &maps.v, col0, h, first_row + c * kRows, &bar[kLandV]);
      }
      __syncwarp();
    };
    auto load = [&](int c) {
      if (c >= 2) wait(kFree0 + (c & 1), (c - 2) >> 1);
      if (dead()) return;
      copied = c + 1;
      const int row = first_row + c * kRows;
      unsigned char* to = smem + C::off_kq + (c & 1) * 32768;
      if (elect_one()) {
        uint64_t* land = &bar[kLand0 + (c & 1)];
        mbar_arrive_expect_tx(land, 32768 + kRecord);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          tma_load_3d_tx(to + i * 16384, &maps.k, 64 * i, hk, row, land);
          tma_load_3d_tx(to + i * 16384 + 8192, &maps.q, 64 * i, hk, row, land);
        }
        const unsigned char* record = record0 + (int64_t)c * p.nv * kRecord;
        bulk_g2s_nohint(smem + C::off_tp + (c & 1) * 2 * kPart, record, 2 * kPart, land);
        bulk_g2s_nohint(smem + C::off_dec + (c & 1) * sizeof(Decays), record + 2 * kPart, sizeof(Decays), land);
      }
      __syncwarp();
    };
    auto landed = [&](int c) {
      wait(kLand0 + (c & 1), c >> 1);
      const int have = rows_left - c * kRows;
      unsigned char* to = smem + C::off_kq + (c & 1) * 32768;
      if (have < kRows)  // the rows behind the sequence's last: others', whatever they hold
        for (int i = lane; i < (kRows - have) * 32; i += 32) {
          const int row = have + (i >> 5), at = i & 31;
          *reinterpret_cast<uint4*>(to + (at >> 4) * 16384 + ((at >> 3) & 1) * 8192 + row * 128 + ((at & 7) << 4)) = make_uint4(0, 0, 0, 0);
        }
      if (!dbg.unreachable) arrive(kReady0 + (c & 1));
    };
    auto load_z = [&](int c) {
      if (!p.z) return;
      if (c >= 1) wait(kZFree, c - 1);
      if (dead()) return;
      gates = c + 1;
      unsigned char* zs = smem + C::off_z;
      const int first = c * kRows, have = min(kRows, rows_left - first);
      if (p.z_wide) {
        if (elect_one()) {
          mbar_arrive_expect_tx(&bar[kZ], kRows * C::cols * 4);
#pragma unroll
          for (int i = 0; i < C::cols / 32; ++i)
            tma_load_3d_tx(zs + i * kRows * 128, &maps.z, col0 + 32 * i, h, first_row + first, &bar[kZ]);
        }
        __syncwarp();
      } else {
        const float* z0 = p.z + (first_row + first) * p.z_row + h * p.z_head + col0;
#pragma unroll 8
        for (int u = 0; u < kRows * C::cols / 32; ++u) {
          const int at = u * 32 + lane, x = at / C::cols, cl = at % C::cols;
          if (x < have)
            *reinterpret_cast<float*>(zs + (cl >> 5) * kRows * 128 + piece(x, (cl >> 2) & 7) + 4 * (cl & 3)) = z0[x * p.z_row + cl];
        }
        arrive(kZ);
      }
    };
    auto store = [&](int c) {  // the output of chunk c
      wait(kOut, c);
      if (dead()) return;
      const int have = min(kRows, rows_left - c * kRows), row = first_row + c * kRows;
      constexpr int line = F32 ? 32 : 64;  // columns of a panel
      const unsigned char* from = smem + C::off_out;
      if (p.out_wide && have == kRows) {
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < C::cols / line; ++i)
            asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(&maps.out),
                         "r"(col0 + line * i), "r"(h), "r"(row), "r"(smem_u32(from + i * kRows * 128))
                         : "memory");
          asm volatile("cp.async.bulk.commit_group;\n cp.async.bulk.wait_group.read 0;" ::: "memory");
        }
        __syncwarp();
      } else {
        constexpr int pieces = C::cols * (F32 ? 4 : 2) / 16;  // of a row
        unsigned char* out = static_cast<unsigned char*>(p.out) + ((int64_t)row * p.out_row + h * p.out_head + col0) * (F32 ? 4 : 2);
        for (int i = lane; i < have * pieces; i += 32) {
          const int x = i / pieces, at = i % pieces;
          *reinterpret_cast<uint4*>(out + x * p.out_row * (F32 ? 4 : 2) + 16 * at) =
              *reinterpret_cast<const uint4*>(from + (at >> 3) * kRows * 128 + piece(x, at & 7));
        }
      }
      arrive(kOutFree);
    };
    load_v(0);
    load(0);
    load_z(0);
    landed(0);
    if (chunks > 1) {
      load_v(1);
      load(1);
    }
    for (int c = 0; c < chunks && !dead(); ++c) {
      if (c > 0) {
        store(c - 1);
        load_z(c);
      }
      if (c + 1 < chunks) landed(c + 1);
      if (c + 2 < chunks) {
        load_v(c + 2);
        load(c + 2);
      }
    }
    store(chunks - 1);
    if (elect_one()) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
    if (dead()) {
      auto drain = [&](int b, int phase) {
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait_suspend(&bar[b], phase & 1, 20000u) && globaltimer_ns() - t0 < 1000000000ull) {
        }
      };
      for (int c = max(0, copied - 2); c < copied; ++c) drain(kLand0 + (c & 1), c >> 1);
      if (values) drain(kLandV, values - 1);
      if (gates && p.z_wide) drain(kZ, gates - 1);
    }
  }
  __syncthreads();
  cluster_sync();  // (no CTA leaves while another may still store into it)
  if (*abort) {                                 // (and a store that nothing waited for lands within a microsecond)
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 50000) {
    }
  }
}

// ------------------------------------------------------------------ T and P T
// [K; Q], and in their place, once their products are in registers, [T; P]; A's blocks on the diagonal in f32; four heads' decays; one
// over the scales of P's rows
constexpr int kOffDiag = 2 * kPart, kOffHi = kOffDiag + 4 * 16 * kLd * 4, kHeadDecays = 7 * kRows;
constexpr int kOffScale = kOffHi + 4 * kHeadDecays * 4, kPrepSmem = kOffScale + kRows * 4 + 1024;

// The sequence and chunk whose record is x, the whole warp: false where there is none.
FAK_DEV bool find_chunk(const GdnParams& p, const Records& r, int x, int lane, GdnSeq& d, int& s, int& c) {
  auto has = [&](int i, GdnSeq& e) {  // sequence i's chunk at x, or -1
    e = gdn_seq(p.c, kv_seq(p.c, i), i);
    const int rows = e.r1 - e.first;
    if (!e.ok || rows == 0 || (p.few && rows <= p.few)) return -1;
    const int at = x + r.begin - (r.dense ? i * r.length : place_of(r, e.r0, i));
    return at < 0 || (r.dense && (at < r.begin || at >= r.begin + r.length)) || (int64_t)at * kRows >= rows ? -1 : at;
  };
  if (r.dense) {
    s = x / r.length;
    return (c = has(s, d)) >= 0;
  }
  // where the starts rise, 32 probes a round
  int lo = 0, hi = p.c.n_seqs;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, i = lo + lane * step;
    const unsigned b = __ballot_sync(0xffffffffu, i < hi && place_of(r, p.c.row_start[i], i) <= x + r.begin);
    const int n = __popc(b);
    if (n > 1) lo += (n - 1) * step;
    hi = min(lo + step, hi);
  }
  s = lo;
  if ((c = has(s, d)) >= 0) return true;
  // a place of none, unless starts are out of range or fall: then all sequences
  bool odd = false;
#pragma unroll 8
  for (int i = lane; i < p.c.n_seqs; i += 32) {
    const int r0 = p.c.row_start[i], r1 = p.c.row_start[i + 1];
    odd |= r0 < 0 || r1 < r0 || r1 > p.c.rows;
  }
  if (!__any_sync(0xffffffffu, odd)) return false;
#pragma unroll 1
  for (int base = 0; base < p.c.n_seqs; base += 32) {
    GdnSeq e{0, 0, 0, 0, false, false};
    const int at = base + lane < p.c.n_seqs ? has(base + lane, e) : -1;
    const unsigned any = __ballot_sync(0xffffffffu, at >= 0);
    if (!any) continue;
    s = base + __ffs(any) - 1;
    c = has(s, d);
    return true;
  }
  return false;
}

// A class of sequences by their chunks n: n itself, from 32 on eight classes to a doubling.
constexpr int kClasses = 32 + 8 * 27;
FAK_DEV int class_of(int n) {
  if (n < 32) return n;
  const int e = 31 - __clz(n);
  return 32 + 8 * (e - 5) + ((n >> (e - 3)) & 7);
}

// The order of the sequences, by one block: those of the highest classes first.  (CTAs start in that order, and those that start
// last are the shortest: 16 prompts of 1 to 2,048 rows and 16 heads take 8 % longer in the batch's order.)
FAK_DEV void make_order(const GdnParams& p, const Records& r, int* count) {
  auto of = [&](int i) {
    int begin, end;
    chunks_of(p, r, gdn_seq(p.c, kv_seq(p.c, i), i), i, begin, end);
    return class_of(max(end - begin, 0));
  };
  for (int i = threadIdx.x; i < kClasses; i += kPrepThreads) count[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < p.c.n_seqs; i += kPrepThreads)
    atomicAdd(&count[of(i)], 1);
  __syncthreads();
  if (threadIdx.x == 0)
    for (int i = kClasses - 1, sum = 0; i >= 0; --i) {
      const int n = count[i];
      count[i] = sum;
      sum += n;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < p.c.n_seqs; i += kPrepThreads)
    r.order[atomicAdd(&count[of(i)], 1)] = i;
}

// Block (x, h): record x, key head h; one more block for the order.
__global__ void __launch_bounds__(kPrepThreads, 4) gdn_prepare_kernel(const __grid_constant__ GdnParams p, Records records, int slots) {
  extern __shared__ unsigned char raw[];
  unsigned char* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q2 = 2 * (lane & 3);
  const int hk = blockIdx.y;
  GdnSeq d;
  int s, c;
  if (blockIdx.x == slots) {
    if (hk == 0) make_order(p, records, reinterpret_cast<int*>(smem));
    return;
  }
  if (!find_chunk(p, records, blockIdx.x, lane, d, s, c)) return;
  const int rows = d.r1 - d.first, first = c * kRows, have = min(kRows, rows - first);
  unsigned char* tp = smem;
  const uint32_t kqs = smem_u32(smem), tps = kqs;
  float* diag = reinterpret_cast<float*>(smem + kOffDiag);
  float* scales = reinterpret_cast<float*>(smem + kOffScale);

  // K and Q, 16 threads to a row of 256 bytes; zeros behind the last row
  {
    const int piece = threadIdx.x & 15, x0 = threadIdx.x >> 4;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const __half* src = m ? p.q + (int64_t)(d.first + first) * p.q_row + hk * p.q_head + 8 * piece
                            : p.k + (int64_t)(d.first + first) * p.k_row + hk * p.k_head + 8 * piece;
      const int64_t step = m ? p.q_row : p.k_row;
      const uint32_t dst = kqs + (piece >> 3) * 16384 + m * 8192 + (((piece & 7) ^ x0) << 4);
#pragma unroll
      for (int u = 0; u < kRows / 8; ++u) {
        const int x = 8 * u + x0;
        copy16(dst + x * 128, x < have ? src + x * step : src, x < have);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // Of K K^T and Q K^T, 16 rows by 16 columns at a time, on and below the diagonal: rows 16 w .. of the first (parts 0 .. w) and
  // 16 (3 - w) .. of the second (parts w + 1 .. 4), five to a warp.
  float dots[5][8] = {};
  auto place = [&](int i, int& m, int& tile, int& j) {  // part i: product, rows, columns
    m = i > w;
    tile = m ? 3 - w : w;
    j = m ? i - w - 1 : i;
  };
  for (int h0 = 0; h0 < p.group; h0 += 4) {
    const int heads = min(4, p.group - h0);
    if (w < heads) {
      // Sums of g log2(e), two rows to a lane, in units of 2^-40; a decay of 2^-150 and below is as good as none left (and
      // sums that grow are cut where 2^G is infinite by far).  A NaN stays one from its row on.
      const int h = hk * p.group + h0 + w;
      float b[2];
      long long x[2];
      bool odd[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int at = 2 * lane + j;
        const int64_t row = d.first + first + at;
        const float gate = at < have ? p.g[row * p.nv + h] : 0.0f;
        b[j] = at < have ? p.beta[row * p.nv + h] : 0.0f;
        odd[j] = gate != gate;
        const float y = fminf(fmaxf(gate, -104.0f), 5000.0f);  // -150 log(2)
        const float hi = y * 1.44269504f, lo = fmaf(y, 1.44269504f, -hi) + y * 1.92596299e-8f;
        x[j] = __float2ll_rn(hi * 1099511627776.0f) + __float2ll_rn(lo * 1099511627776.0f);
      }
      const unsigned any = __ballot_sync(0xffffffffu, odd[0] || odd[1]);
      long long sum = x[0] + x[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      const bool before = any & ((1u << lane) - 1);
      const long long G[2] = {sum - x[1], sum};
      float hi[2], lo[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const long long u = (G[j] + (1ll << 30)) >> 31;
        hi[j] = (float)(int)u * (1.0f / 512.0f);
        lo[j] = (float)(int)(G[j] - (u << 31)) * 9.094947017729282e-13f;  // 2^-40
        if (before || odd[0] || (j == 1 && odd[1])) lo[j] = __uint_as_float(0x7fffffffu);
      }
      const float hi_end = __shfl_sync(0xffffffffu, hi[1], 31), lo_end = __shfl_sync(0xffffffffu, lo[1], 31);
      // of a head: G as two f32, beta, exp(G_t - G of the last row before t's 16), exp(G of row 16 i - 1 - G_s), i = 1, 2, 3
      float* mine = reinterpret_cast<float*>(smem + kOffHi) + w * kHeadDecays + 2 * lane;
      float ref_hi[4], ref_lo[4];
#pragma unroll
      for (int i = 1; i < 4; ++i) {
        ref_hi[i] = __shfl_sync(0xffffffffu, hi[1], 8 * i - 1);
        ref_lo[i] = __shfl_sync(0xffffffffu, lo[1], 8 * i - 1);
        *reinterpret_cast<float2*>(mine + (3 + i) * kRows) =
            make_float2(exp2_approx((ref_hi[i] - hi[0]) + (ref_lo[i] - lo[0])), exp2_approx((ref_hi[i] - hi[1]) + (ref_lo[i] - lo[1])));
      }
      const int own = lane >> 3;
      const float rh = own == 1 ? ref_hi[1] : own == 2 ? ref_hi[2] : ref_hi[3], rl = own == 1 ? ref_lo[1] : own == 2 ? ref_lo[2] : ref_lo[3];
      *reinterpret_cast<float2*>(mine + 3 * kRows) = make_float2(exp2_approx((hi[0] - rh) + (lo[0] - rl)), exp2_approx((hi[1] - rh) + (lo[1] - rl)));
      *reinterpret_cast<float2*>(mine) = make_float2(hi[0], hi[1]);
      *reinterpret_cast<float2*>(mine + kRows) = make_float2(lo[0], lo[1]);
      *reinterpret_cast<float2*>(mine + 2 * kRows) = make_float2(b[0], b[1]);
      unsigned char* record = records.at + ((int64_t)blockIdx.x * p.nv + h) * kRecord + 2 * kPart + 8 * lane;
      *reinterpret_cast<float2*>(record) = make_float2(exp2_approx(hi[0] + lo[0]), exp2_approx(hi[1] + lo[1]));
      *reinterpret_cast<float2*>(record + 4 * kRows) =
          make_float2(exp2_approx((hi_end - hi[0]) + (lo_end - lo[0])), exp2_approx((hi_end - hi[1]) + (lo_end - lo[1])));
      *reinterpret_cast<float2*>(record + 8 * kRows) = make_float2(b[0], b[1]);
    }
    if (h0 == 0) {  // (the gates come while K and Q do)
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();
      float squares[8] = {};  // Q Q^T of the rows 16 (3 - w) ..
#pragma unroll 2
      for (int k = 0; k < 8; ++k) {
        auto at = [&](int row, int piece) { return kqs + (piece >> 3) * 16384 + row * 128 + (((piece & 7) ^ (row & 7)) << 4); };
        uint32_t ak[4], aq[4];
        ldsm4(ak, at(16 * w + (lane & 15), 2 * k + (lane >> 4)));
        ldsm4(aq, at(64 + 16 * (3 - w) + (lane & 15), 2 * k + (lane >> 4)));
#pragma unroll
        for (int i = 0; i < 5; ++i) {
          int m, tile, j;
          place(i, m, tile, j);
          uint32_t b[4], a[4];
          ldsm4(b, at(16 * j + (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
#pragma unroll
          for (int u = 0; u < 4; ++u) a[u] = m ? aq[u] : ak[u];
          const uint32_t b0[2] = {b[0], b[1]}, b1[2] = {b[2], b[3]};
          mma16(*reinterpret_cast<float(*)[4]>(dots[i]), a, b0);
          mma16(*reinterpret_cast<float(*)[4]>(dots[i] + 4), a, b1);
        }
        {
          uint32_t b[4];
          ldsm4(b, at(64 + 16 * (3 - w) + (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
          const uint32_t b0[2] = {b[0], b[1]}, b1[2] = {b[2], b[3]};
          mma16(*reinterpret_cast<float(*)[4]>(squares), aq, b0);
          mma16(*reinterpret_cast<float(*)[4]>(squares + 4), aq, b1);
        }
      }
      // Queries are as long as they are: each row of P, and of P T, goes by a power of two by which its query's length is 1 .. 2.
      {
        const int from = 4 * g + (g >> 1);  // the lane that has rows g's and g + 8's sums of squares
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float ss = __shfl_sync(0xffffffffu, g & 1 ? squares[6 * u + 1] : squares[6 * u], from);
          const int e = (int)(__float_as_uint(ss) >> 23);
          const float up = two_to(e == 0 || e == 255 ? 0 : -((e - 127) >> 1));
          if ((lane & 3) == 0) scales[16 * (3 - w) + g + 8 * u] = up;
#pragma unroll
          for (int i = 0; i < 5; ++i)
            if (i > w) {
#pragma unroll
              for (int x = 0; x < 8; ++x)
                if ((x >> 1 & 1) == u) dots[i][x] *= up;
            }
        }
      }
      __syncthreads();
      // T and P T are zero above their blocks on the diagonal, which nothing writes
      for (int i = threadIdx.x; i < 2 * kPart / 16; i += kPrepThreads) *reinterpret_cast<uint4*>(tp + 16 * i) = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    for (int hh = 0; hh < heads; ++hh) {
      const int h = hk * p.group + h0 + hh;
      const float* hi = reinterpret_cast<const float*>(smem + kOffHi) + hh * kHeadDecays;
      const float *lo = hi + kRows, *beta = hi + 2 * kRows;
      // A from K K^T and the strengths, and P, to the places of T and P T
#pragma unroll
      for (int i = 0; i < 5; ++i) {
        int m, tile, j;
        place(i, m, tile, j);
        const int row = 16 * tile + g;
        const float b0 = m ? 1.0f : beta[row], b1 = m ? 1.0f : beta[row + 8];
        float y[2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float* z = dots[i] + 4 * e;
          y[e][0] = b0 * z[0];
          y[e][1] = b0 * z[1];
          y[e][2] = b1 * z[2];
          y[e][3] = b1 * z[3];
        }
        if (j == tile) {
          const int last = m ? g : g - 1;  // of row g's own 16 columns; row g + 8's: 8 more
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int at = 8 * e + q2;
            // (a zero that masks is put there, not multiplied by: it must not meet an infinity)
            y[e][0] = at <= last ? y[e][0] : 0.0f;
            y[e][1] = at + 1 <= last ? y[e][1] : 0.0f;
            y[e][2] = at <= last + 8 ? y[e][2] : 0.0f;
            y[e][3] = at + 1 <= last + 8 ? y[e][3] : 0.0f;
            if (!m) {
              *reinterpret_cast<float2*>(diag + row * kLd + at) = make_float2(y[e][0], y[e][1]);
              *reinterpret_cast<float2*>(diag + (row + 8) * kLd + at) = make_float2(y[e][2], y[e][3]);
            }
          }
        }
        put_tiles<false>(tps, m * kRows + 16 * tile, 2 * j, y[0], y[1], lane);
      }
      __syncthreads();
      {
        // row lane % 16 of the inverse of the 16 x 16 block of I + A at 16 w
        const int row = lane & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = i == row ? 1.0f : 0.0f;
        const float* a = diag + 16 * w * kLd;
#pragma unroll
        for (int i = 15; i > 0; --i) {
          float y[16];
#pragma unroll
          for (int j = 0; j < i; j += 4) {
            const float4 u = *reinterpret_cast<const float4*>(a + i * kLd + j);
            y[j] = u.x;
            y[j + 1] = u.y;
            y[j + 2] = u.z;
            y[j + 3] = u.w;
          }
#pragma unroll
          for (int j = i - 1; j >= 0; --j) x[j] = fmaf(-x[i], y[j], x[j]);
        }
        float2 y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = make_float2(x[2 * i], x[2 * i + 1]);
        if (lane < 16) put_halves<16>(tp, 0, kPart, 16 * w + row, 16 * w, y);
      }
      __syncthreads();
      {
        // two blocks of 32: the lower left is -T22 (A21 T11), eight columns to a warp
        const int at = 32 * (w >> 1), j = (at >> 3) + (w & 1);
        float x[4] = {}, y[4] = {}, x1[4] = {}, y1[4] = {}, x2[4] = {}, y2[4] = {};  // (products that do not wait for each other)
        FragA a, u;
        FragB b;
        load_a(a, tps, at + 16, at, lane);
        load_a(u, tps, at + 16, at + 16, lane);
        load_b(b, tps, at, j, lane);
        mma16(x1, a.lo, b.hi);
        mma16(x2, a.hi, b.lo);
        mma16(x, a.hi, b.hi);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] += x1[i] + x2[i];
        turn_b(b, x);
        mma16(y1, u.lo, b.hi);
        mma16(y2, u.hi, b.lo);
        mma16(y, u.hi, b.hi);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] += y1[i] + y2[i];
        __syncthreads();  // (A21 is read)
        put_block(tp, at + 16, j, y, -1.0f, lane);
      }
      __syncthreads();
      {
        // the block of 64's, 32 x 32, eight columns to a warp
        float x[2][4] = {}, y[2][4] = {};
        FragA a[2];
        FragB b;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          load_b(b, tps, 16 * k, w, lane);
#pragma unroll
          for (int m = 0; m < 2; ++m) load_a(a[m], tps, 32 + 16 * m, 16 * k, lane);
#pragma unroll
          for (int m = 0; m < 2; ++m) mma16(x[m], a[m].lo, b.hi);
#pragma unroll
          for (int m = 0; m < 2; ++m) mma16(x[m], a[m].hi, b.lo);
#pragma unroll
          for (int m = 0; m < 2; ++m) mma16(x[m], a[m].hi, b.hi);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          turn_b(b, x[k]);
#pragma unroll
          for (int m = k; m < 2; ++m) load_a(a[m], tps, 32 + 16 * m, 32 + 16 * k, lane);
#pragma unroll
          for (int m = k; m < 2; ++m) mma16(y[m], a[m].lo, b.hi);
#pragma unroll
          for (int m = k; m < 2; ++m) mma16(y[m], a[m].hi, b.lo);
#pragma unroll
          for (int m = k; m < 2; ++m) mma16(y[m], a[m].hi, b.hi);
        }
        __syncthreads();  // (A21 is read)
#pragma unroll
        for (int m = 0; m < 2; ++m) put_block(tp, 32 + 16 * m, w, y[m], -1.0f, lane);
      }
      __syncthreads();
      {
        // P T, by blocks of 16 x 16 (m, j): sums over k = j .. m, five steps to a warp
        const unsigned mine = w == 0 ? 0xffff0030u : w == 1 ? 0xffff3231u : w == 2 ? 0xffff1020u : 0x11223321u;
        float y[4][2][4] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int m = mine >> (8 * i + 4) & 15, j = mine >> (8 * i) & 15;
          if (m == 15) break;
          for (int k = j; k <= m; ++k) {
            FragA a;
            FragB b[2];
            load_a(a, tps, kRows + 16 * m, 16 * k, lane);
            load_b(b[0], tps, 16 * k, 2 * j, lane);
            load_b(b[1], tps, 16 * k, 2 * j + 1, lane);
#pragma unroll
            for (int u = 0; u < 2; ++u) mma16(y[i][u], a.lo, b[u].hi);
#pragma unroll
            for (int u = 0; u < 2; ++u) mma16(y[i][u], a.hi, b[u].lo);
#pragma unroll
            for (int u = 0; u < 2; ++u) mma16(y[i][u], a.hi, b[u].hi);
          }
        }
        __syncthreads();  // (T and P are read)
        // T, and P T in P's place, by their decays and 2^14: within the rows' own 16 columns one exponential each, before them by way of
        // the last row before the 16
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int m = mine >> (8 * i + 4) & 15, j = mine >> (8 * i) & 15;
          if (m == 15) break;
          FragA a;
          load_a(a, tps, 16 * m, 16 * j, lane);
          float t[2][4];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int row = 16 * m + 8 * u + g;
            const float f = hi[3 * kRows + row] * 16384.0f, hr = hi[row], lr = lo[row];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int at = 8 * e + q2, col = 16 * j + at;
              float2 by;
              if (j < m) {
                by = mul2(*reinterpret_cast<const float2*>(hi + (3 + m) * kRows + col), both(f));
              } else {
                const float2 hc = *reinterpret_cast<const float2*>(hi + col), lc = *reinterpret_cast<const float2*>(lo + col);
                by = mul2(make_float2(exp2_approx((hr - hc.x) + (lr - lc.x)), exp2_approx((hr - hc.y) + (lr - lc.y))), both(16384.0f));
              }
              const float2 t1 = __half22float2(*reinterpret_cast<const __half2*>(&a.hi[2 * e + u]));
              const float2 t2 = __half22float2(*reinterpret_cast<const __half2*>(&a.lo[2 * e + u]));
              float2 x = mul2(add2(t1, t2), by), z = mul2(make_float2(y[i][e][2 * u], y[i][e][2 * u + 1]), by);
              // (a zero that masks is put there, not multiplied by: it must not meet an infinity)
              if (j == m && at > g + 8 * u) x.x = z.x = 0.0f;
              if (j == m && at + 1 > g + 8 * u) x.y = z.y = 0.0f;
              t[e][2 * u] = x.x;
              t[e][2 * u + 1] = x.y;
              y[i][e][2 * u] = z.x;
              y[i][e][2 * u + 1] = z.y;
            }
          }
          put_tiles<true>(tps, 16 * m, 2 * j, t[0], t[1], lane);
          put_tiles<true>(tps, kRows + 16 * m, 2 * j, y[i][0], y[i][1], lane);
        }
      }
      fence_async();
      __syncthreads();
      unsigned char* record = records.at + ((int64_t)blockIdx.x * p.nv + h) * kRecord;
      if (threadIdx.x < kRows) reinterpret_cast<Decays*>(record + 2 * kPart)->up[threadIdx.x] = scales[threadIdx.x];
      if (threadIdx.x == 0) {
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(record), "r"(tps), "r"(2 * kPart) : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      }
      __syncthreads();
    }
  }
  if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

std::mutex g_mu;
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

cudaError_t encoder() {
  std::lock_guard<std::mutex> lk(g_mu);
  if (g_encode) return cudaSuccess;
  cudaDriverEntryPointQueryResult q;
  void* fn = nullptr;
  const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
  if (e != cudaSuccess) return e;
  if (q != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
  g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  return cudaSuccess;
}

// Rows [row][head][128], boxes of 64 rows of one head's 128 bytes.  (A stride that is never taken may be anything.)
bool rows_map(CUtensorMap* map, const void* base, CUtensorMapDataType type, int64_t rows, int heads, int64_t row, int64_t head) {
  const cuuint64_t elem = type == CU_TENSOR_MAP_DATA_TYPE_FLOAT32 ? 4 : 2;
  const cuuint64_t dim[3] = {kGdnDim, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t by_head = heads > 1 ? (cuuint64_t)head * elem : kGdnDim * elem;
  const cuuint64_t stride[2] = {by_head, rows > 1 ? (cuuint64_t)row * elem : by_head * heads};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / elem), 1, kRows}, one[3] = {1, 1, 1};
  return g_encode(map, type, 3, const_cast<void*>(base), dim, stride,
                  box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool F32>
cudaError_t launch(const GdnParams& p, const ChunkMaps& maps, const Records& records, const ChunkDebug& dbg, int* status, int dev,
                   cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = kv_smem_limit(gdn_chunk_kernel<F32>, C::smem, dev, done);
  if (e != cudaSuccess) return e;
  static std::atomic<int> regs{0};  // (a query that fails is made again by the next call)
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes a;
    e = cudaFuncGetAttributes(&a, gdn_chunk_kernel<F32>);
    if (e != cudaSuccess) return e;
    regs.store(a.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) < kRegs) return cudaErrorNotSupported;  // (its warps would wait for registers that nobody gives back)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)p.c.n_seqs * p.nv * C::slices));
  cfg.blockDim = dim3(C::threads);
  cfg.dynamicSmemBytes = C::smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C::slices;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gdn_chunk_kernel<F32>, p, maps, records, dbg, status);
}

constexpr int64_t kScratch = 1LL << 30;  // most bytes of records at a time; more chunks than they hold go in several launches

}  // namespace

cudaError_t gdn_chunk_launch(const GdnParams& p, unsigned long long timeout_ns, int unreachable, int* status, int dev, int sms, cudaStream_t s) {
  cudaError_t e = encoder();
  if (e != cudaSuccess) return e;
  ChunkMaps maps;
  memset(&maps, 0, sizeof(maps));
  const int nk = p.nv / p.group;
  if (!rows_map(&maps.k, p.k, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, p.c.rows, nk, p.k_row, p.k_head) ||
      !rows_map(&maps.q, p.q, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, p.c.rows, nk, p.q_row, p.q_head) ||
      !rows_map(&maps.v, p.v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.c.rows, p.nv, p.v_row, p.v_head) ||
      (p.z && p.z_wide && !rows_map(&maps.z, p.z, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, p.c.rows, p.nv, p.z_row, p.z_head)) ||
      (p.out_wide && !rows_map(&maps.out, p.out, p.out_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, p.c.rows,
                               p.nv, p.out_row, p.out_head)))
    return cudaErrorInvalidValue;
  const ChunkDebug dbg{timeout_ns, unreachable};
  // Records of all chunks, where they are few enough; else of a stretch of every sequence at a time, or, where that would be short
  // (below 16 chunks), of a stretch of all places.
  const int64_t longest = (std::min<int64_t>(p.c.max_q, p.c.rows) + kRows - 1) / kRows, head = (int64_t)p.nv * kRecord;
  const int64_t by_seq = p.c.rows / kRows + p.c.n_seqs, by_row = p.few ? p.c.rows / kGdnFew + 1 : by_seq;
  const int64_t places = std::min(by_seq, by_row), most = std::max<int64_t>(1, kScratch / head);
  Records records{nullptr, 0, (int)std::min(places, most), false, by_row < by_seq, nullptr};
  int64_t slots = records.length, all = places;  // records of a launch; what begin goes up to
  if (places > most && most / p.c.n_seqs >= 16) {
    records.dense = true;
    records.length = (int)std::min(longest, most / p.c.n_seqs);
    slots = p.c.n_seqs * (int64_t)records.length;
    all = longest;
  }
  const int64_t bytes = slots * head;
  void* scratch = nullptr;
  const bool ordered = p.c.n_seqs > 1 && (int64_t)p.c.n_seqs * p.nv * C::slices > sms;
  e = fak_scratch_alloc(&scratch, (size_t)bytes + (ordered ? 4 * (size_t)p.c.n_seqs : 0), s);
  if (e != cudaSuccess) return cudaErrorMemoryAllocation;
  records.at = static_cast<unsigned char*>(scratch);
  if (ordered) records.order = reinterpret_cast<int*>(records.at + bytes);
  static std::atomic<uint64_t> done{0};
  e = kv_smem_limit(gdn_prepare_kernel, kPrepSmem, dev, done);
  for (; e == cudaSuccess && records.begin < all; records.begin += records.length) {
    gdn_prepare_kernel<<<dim3((unsigned)(slots + ordered), (unsigned)nk), kPrepThreads, kPrepSmem, s>>>(p, records, (int)slots);
    e = cudaGetLastError();
    if (e == cudaSuccess) e = p.out_bf16 ? launch<false>(p, maps, records, dbg, status, dev, s) : launch<true>(p, maps, records, dbg, status, dev, s);
  }
  const cudaError_t f = cudaFreeAsync(scratch, s);
  return e != cudaSuccess ? e : f;
}
