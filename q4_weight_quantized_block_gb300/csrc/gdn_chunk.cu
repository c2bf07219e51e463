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
// Precision.  The state is held in f32 registers, and its products keep 22 bits: the f32 operand goes as the sum of two
// f16, the other one is f16 already (q, k) or two f16 too (T, P T; the small parts' product is left out).  f16's exponents
// take them because a chunk's S, R and U are scaled by one power of two.  With m the largest of |S| and |V|, lengths of k
// of at most 1 and 0 <= beta <= 2: |R| <= 25 m, |U| <= 281 m, and the next chunk's |S| <= 140 m.  The scale goes by m of
// the chunk before (its own would hold all warps up at a barrier), so m goes to 2^-2 .. 2^-1, U stays below 2^15, and what
// f16 drops is below 2^-25, so 2^-23 m.  T and P T need no scale: |T|, and so P T, is at most 3.  Sums of decays are made in fixed point and
// kept as two f32, so that decays over neighbouring rows, differences of large sums, are off by 2^-22 only.
//
// First kernel: a block takes a chunk and a key head, whose K K^T and Q K^T its value heads share, four warps: decays into A
// and P; inverses of 16 x 16 blocks by substitution, joined to 32 and to 64, and P T, in place of A and P, by m16n8k16
// instructions.  (Made by four more warps of the second kernel, a chunk ahead, the same work took longer than a chunk's
// products, and once for each CTA of a head.)
//
// Second kernel: a cluster of two CTAs (one on an SM) holds one head of one sequence, a CTA 64 of its value columns, as two
// halves of 32 that go their own ways, so that one's products run while the other's operands are made: only the norm
// needs the whole row, and its sums of squares go to the other CTA by asynchronous stores.  Warps:
//   0 .. 7, 8 .. 15  a half each: a warp reads the accumulators' 32 lanes (w % 4) and 16 columns; lanes 0..63 are K's or T's
//                    rows (R, then U, to shared memory as f16), 64..127 Q's or P T's (the output); S's rows in all 128.
//                    (With 32 columns to a warp a step took twice as long: one warp issues an instruction in four cycles.)
//   16, 17           issue a half's products;  18  copies K, Q, V, z and the records.
// The products read their operands from shared memory at 128 bytes a cycle: a step of 16 takes 128 rows of A (4 KB) and
// B's columns, so B's two parts stand side by side as 64 columns, one read of A for both.
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
constexpr int kChainThreads = 512;
constexpr int kThreads = kChainThreads + 128;
constexpr int kPrepThreads = 128;
constexpr int kLd = 20;  // f32 blocks of 16 x 16 in shared memory: rows of 80 bytes
constexpr int kPart = 16384;  // from a matrix's first parts to its second: 128 rows of 64 f16

// What a chunk's rows decay by, and their strengths: behind [T; P T], two parts, in a chunk's record for a head.
struct Decays {
  float keep[kRows];  // exp G_t
  float left[kRows];  // exp(G_64 - G_t)
  float beta[kRows];
};
constexpr int kRecord = 2 * kPart + (int)sizeof(Decays);
static_assert(kRecord % 16 == 0, "bulk copies");

// Where records stand.  dense: chunk c of a sequence s, begin <= c < begin + length, at s * length + c - begin; else chunk c at
// r0 / 64 + s + c, r0 being the sequence's first row (such starts rise by at least the sequences' numbers of chunks).
struct Records {
  unsigned char* at;
  int begin, length, dense;
};

FAK_DEV int64_t record_of(const Records& r, const GdnSeq& d, int s, int c) {
  return r.dense ? (int64_t)s * r.length + (c - r.begin) : (int64_t)(d.r0 / kRows) + s + c;
}

constexpr int kSlices = 2;                // CTAs of a head
constexpr int kCols = kGdnDim / kSlices;  // value columns of a CTA
constexpr int kHalf = kCols / 2;          // of a half
constexpr int W = kHalf / 2;              // of a thread
constexpr int kOffKq = 0;                                   // two stages of [K; Q]: two panels of 128 rows
constexpr int kOffTpt = kOffKq + 2 * 32768;                 // two stages of [T; P T], two parts
constexpr int kOffS = kOffTpt + 4 * kPart;                  // S of each half: 128 rows of 32 columns' first parts, then second
constexpr int kOffU = kOffS + 2 * 16384;                    // R, then U, of each half: 64 rows
constexpr int kOffV = kOffU + 2 * 8192;                     // two stages of V
constexpr int kOffZ = kOffV + 2 * 8192;                     // z: panels of 32 columns, 128 bytes
constexpr int kOffDec = kOffZ + kRows * kCols * 4;
constexpr int kOffSum = kOffDec + 2 * (int)sizeof(Decays);  // sums of squares [2][kSlices * 4][64]
constexpr int kOffGain = kOffSum + 2 * kSlices * 4 * kRows * 4;
constexpr int kOffMax = kOffGain + kCols * 4;               // of each half [8]
constexpr int kOffBar = kOffMax + 64;
constexpr int kChunkSmem = kOffBar + 192 + 1024;
static_assert(kChunkSmem <= 232448, "shared memory exceeds the 227 KB per-block limit");
constexpr int kAccD1 = 0, kAccD2 = 64, kAccD3 = 128, kAccHalf = 192;  // TMEM columns
constexpr int kTmemCols = 512;

enum Bars { kLand0, kLand1, kReady0, kReady1, kD1, kD2 = kD1 + 2, kD3 = kD2 + 2, kZ = kD3 + 2, kZFree, kSum0, kSum1, kDrain, kBars = kDrain + 2 };

// Named barriers of the first half (the second's are kNamed further on), for waits where a polling warp would take issue slots
// from those that work (a try of an mbarrier gives up after some 60 cycles; with all waits so, half of all instructions were
// of such loops).  The products' warp polls, and lets the others go.
enum Named { kBarTurn = 1, kBarS, kBarR, kBarU, kBarD1, kBarD2, kBarD3, kNamed = 7 };

template <int M, int N, bool A_MN, bool B_MN>
constexpr uint32_t kIdesc = (1u << 4) | ((A_MN ? 1u : 0u) << 15) | ((B_MN ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
                            ((uint32_t)(M >> 4) << 24);

FAK_DEV void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}

// 128-byte swizzle with M or N running: 64 of them by 8 k atoms, the next 64 `lbo` bytes on, the next 8 k 1024 bytes on
FAK_DEV uint64_t desc_mn(uint32_t addr, uint32_t lbo) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

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
  const __half2 h = __floats2half2_rn(x, y);
  const float2 b = fma2(__half22float2(h), both(-1.0f), make_float2(x, y));
  const __half2 l = __floats2half2_rn(b.x, b.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
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

// The same for a tile of 32 columns, whose second parts stand behind the first in a row of 128 bytes.
template <int N>
FAK_DEV void put_sides(unsigned char* tile, int row, int col, const float2 (&x)[N / 2]) {
  uint32_t hi[N / 2], lo[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) split_half(x[i].x, x[i].y, hi[i], lo[i]);
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    const int at = row * 128 + ((((col + i) >> 3) ^ (row & 7)) << 4);
    *reinterpret_cast<uint4*>(tile + at) = make_uint4(hi[i / 2], hi[i / 2 + 1], hi[i / 2 + 2], hi[i / 2 + 3]);
    *reinterpret_cast<uint4*>(tile + (at ^ 64)) = make_uint4(lo[i / 2], lo[i / 2 + 1], lo[i / 2 + 2], lo[i / 2 + 3]);
  }
}

// The sums of two columns each, `apart` columns apart.
template <int N>
FAK_DEV void ld_sums(uint32_t addr, int apart, float2 (&x)[N / 2]) {
  uint32_t r[N], u[N];
  tmem_ld_cols<N>(addr, r);
  tmem_ld_cols<N>(addr + apart, u);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < N / 2; ++i)
    x[i] = add2(make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])),
                make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])));
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
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
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
// sign * a product's 16 x 8, both parts, at rows r0 .. +15, columns 8 j .. +7 of a tile
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
  CUtensorMap k, q, v, z;
};

struct ChunkDebug {
  unsigned long long timeout_ns;
  int unreachable;  // a test's: 1 where K and Q are never to count as landed
};

__global__ void __launch_bounds__(kThreads, 1) gdn_chunk_kernel(const __grid_constant__ GdnParams p,
                                                                 const __grid_constant__ ChunkMaps maps, Records records,
                                                                 ChunkDebug dbg, int* status) {
  extern __shared__ unsigned char raw[];
  unsigned char* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + kOffBar);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + kOffBar + 8 * kBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffBar + 8 * kBars + 4);
  float* gain = reinterpret_cast<float*>(smem + kOffGain);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const int slice = blockIdx.x % kSlices, unit = blockIdx.x / kSlices;
  const int s = unit / p.nv, h = unit - s * p.nv;
  const KvSeq seq = kv_seq(p.c, s);
  const GdnSeq d = gdn_seq(p.c, seq, s);
  if (!d.ok) {
    if (threadIdx.x == 0) atomicCAS(status, 0, FAK_ERR_DEVICE);
    return;
  }
  const int rows = d.r1 - d.first;
  if (p.few && rows <= p.few) return;  // the steps' kernel's
  const int col0 = slice * kCols;
  const int begin = records.begin, end = min((rows + kRows - 1) / kRows, begin + records.length);  // this launch's chunks
  if (begin == 0)
    for (int i = threadIdx.x; i < (d.first - d.r0) * (kCols / 4); i += kThreads) {
      const int row = d.r0 + i / (kCols / 4);
      gdn_put4(p.out, p.out_bf16, row * p.out_row + h * p.out_head + col0 + 4 * (i % (kCols / 4)), gdn_zero4());
    }
  const int chunks = end - begin;  // counted from 0 below
  if (chunks <= 0) return;
  const int first_row = d.first + begin * kRows, rows_left = rows - begin * kRows;

  if (threadIdx.x == 0) {
    *abort = 0;
    for (int i = 0; i < kBars; ++i) mbar_init(&bar[i], i == kZFree ? 8 : 1);
    fence_mbar_init();
  }
  if (threadIdx.x < 16) reinterpret_cast<unsigned*>(smem + kOffMax)[threadIdx.x] = 0;
  if (threadIdx.x < kCols) gain[threadIdx.x] = p.norm_w ? p.norm_w[col0 + threadIdx.x] : 1.0f;
  if (warp == 16) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_async();
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  // One that runs out is recorded, and no wait of the block waits after it: every warp goes through its chunks, without
  // results, so that the named barriers stay in step (nothing but such waits lies between two of them).
  auto wait = [&](int b, int phase) {
    bool done = mbar_try_wait(&bar[b], phase & 1) || *abort != 0;
    for (int i = 0; i < 512 && !done; ++i) done = mbar_try_wait(&bar[b], phase & 1);
    if (!done && !mbar_wait_bounded(&bar[b], phase & 1, abort, dbg.timeout_ns)) {
      if (!*abort) atomicCAS(status, 0, FAK_ERR_TIMEOUT);
      *abort = 1;
    }
    __syncwarp();
  };
  // The same for warps that may sleep meanwhile.
  auto doze = [&](int b, int phase) {
    for (int i = 0; i < 4096 && !*abort && !mbar_try_wait(&bar[b], phase & 1); ++i) __nanosleep(100);
    wait(b, phase);
  };
  // What the warp wrote to shared memory and read from TMEM comes before what waits on the barrier, MMAs too.
  auto give = [&](int named, int threads) {
    fence_async();
    tc_fence_before_sync();
    asm volatile("bar.arrive %0, %1;" ::"r"(named), "r"(threads + 32) : "memory");
  };
  auto take = [&](int named, int threads) {
    named_bar_sync(named, threads + 32);
    tc_fence_after_sync();
  };

  if (warp < 16) {
    // ------------------------------------------------------------------ a half's chain
    const int half = warp >> 3, named = half * kNamed;
    const int quarter = warp & 3, col = ((warp >> 2) & 1) * W;  // of the half's columns
    const uint32_t acc = tmem + ((uint32_t)quarter << 21) + half * kAccHalf + col;  // TMEM: lane 32 quarter
    const int key = 32 * quarter + lane;      // the row of S
    const bool top = quarter < 2;             // K's and T's rows, else Q's and P T's
    const int t = 32 * (quarter & 1) + lane;  // the row of the chunk
    unsigned char *ss = smem + kOffS + half * 16384, *us = smem + kOffU + half * 8192;
    float* st = p.state + (((int64_t)d.slot * p.nv + h) * kGdnDim + key) * kGdnDim + col0 + half * kHalf + col;
    unsigned* most = reinterpret_cast<unsigned*>(smem + kOffMax) + 8 * half;  // [4] of S, [4] of V: largest magnitudes, by chunk
    float2 S[W / 2];
#pragma unroll
    for (int i = 0; i < W / 2; i += 2) {
      const float4 x = d.fresh && begin == 0 ? gdn_zero4() : *reinterpret_cast<const float4*>(st + 2 * i);
      S[i] = make_float2(x.x, x.y);
      S[i + 1] = make_float2(x.z, x.w);
    }
    uint32_t v[W / 2];  // of the next chunk
    auto fetch_v = [&](int c) {
      wait(kReady0 + (c & 1), c >> 1);
      const unsigned char* src = smem + kOffV + (c & 1) * 8192 + t * 128;
      const bool there = c * kRows + t < rows_left;  // (what stands behind the last row is another's, whatever it holds)
#pragma unroll
      for (int i = 0; i < W / 8; ++i) {
        const uint4 x = *reinterpret_cast<const uint4*>(src + ((((half * kHalf + col) >> 3) + i) ^ (t & 7)) * 16);
        v[4 * i] = there ? x.x : 0;
        v[4 * i + 1] = there ? x.y : 0;
        v[4 * i + 2] = there ? x.z : 0;
        v[4 * i + 3] = there ? x.w : 0;
      }
    };
    auto tell = [&](int at, float m) {  // a warp's largest magnitude to the half's
      const unsigned u = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
      if (lane == 0) atomicMax(&most[at], u);
    };
    auto tell_state = [&](int c) {
      float ms[2] = {};
#pragma unroll
      for (int i = 0; i < W / 2; ++i) ms[i & 1] = fmaxf(fmaxf(ms[i & 1], fabsf(S[i].x)), fabsf(S[i].y));
      tell(c & 3, fmaxf(ms[0], ms[1]));
    };
    auto tell_values = [&](int c) {
      float ms[2] = {};
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        const float2 x = bf16_pair(v[i]);
        ms[i & 1] = fmaxf(fmaxf(ms[i & 1], fabsf(x.x)), fabsf(x.y));
      }
      tell(4 + (c & 3), fmaxf(ms[0], ms[1]));
    };
    float up = 1.0f, down = 1.0f;  // the chunk's power of two, and one over it
    // S, as it stands before chunk c, scaled and in two parts to shared memory.  The scale goes by the state one chunk
    // before, whose magnitudes every warp has told by now.
    auto put_state = [&](int c) {
      const int b = max(c - 1, 0);
      const float m = __uint_as_float(max(most[b & 3], max(most[4 + (b & 3)], most[4 + (c & 3)])));
      // m = 2^e 1.f goes to 2^-2 1.f (zeros and infinities: as they are); the inverse is a normal number too
      const int e = (int)(__float_as_uint(m) >> 23);
      const int by = e == 0 || e == 255 ? 0 : min(max(125 - e, -120), 120);
      up = __uint_as_float((uint32_t)(127 + by) << 23);
      down = __uint_as_float((uint32_t)(127 - by) << 23);
      float2 x[W / 2];
#pragma unroll
      for (int i = 0; i < W / 2; ++i) x[i] = mul2(S[i], both(up));
      put_sides<W>(ss, key, col, x);
    };
    const uint32_t sum_to = smem_u32(smem + kOffSum);
    const int me = (int)rank_in_cluster();
    tell_state(0);
    if (top) {
      fetch_v(0);
      tell_values(0);
    }
    named_bar_sync(named + kBarTurn, 256);
    put_state(0);
    give(named + kBarS, 256);

    // The output of a chunk, whose rows stand in o, is finished while the next chunk's products run, so that the state does
    // not wait for it: its norm and gate between the next chunk's first two products, its stores between the last two.  The
    // rows turn in S's place, which the first product is done with, so that stores are whole lines: a thread's own row would
    // be a line for every lane (3,000 cycles a chunk).
    float2 o[W / 2];
    auto finish = [&](int c) {
      float r = 1.0f;
      if (p.norm_w) {
        wait(kSum0 + (c & 1), c >> 1);
        try_cluster(&bar[kSum0 + (c & 1)], c >> 1 & 1);  // (an acquire of the others' stores)
        const float* sums = reinterpret_cast<const float*>(smem + kOffSum) + (c & 1) * kSlices * 4 * kRows + t;
        float y = 0.0f;
#pragma unroll
        for (int i = 0; i < 4 * kSlices; ++i) y += sums[i * kRows];
        r = rsqrtf(fmaf(y, 1.0f / kGdnDim, p.eps));
      }
#pragma unroll
      for (int i = 0; i < W / 2; i += 2) {
        const float4 w = *reinterpret_cast<const float4*>(gain + half * kHalf + col + 2 * i);
        o[i] = mul2(o[i], mul2(make_float2(w.x, w.y), both(r)));
        o[i + 1] = mul2(o[i + 1], mul2(make_float2(w.z, w.w), both(r)));
      }
      if (p.z) {
        wait(kZ, c);
        const unsigned char* zs = smem + kOffZ + half * kRows * 128 + t * 128;
#pragma unroll
        for (int i = 0; i < W / 2; i += 2) {
          const float4 z = *reinterpret_cast<const float4*>(zs + ((((col >> 2) + i / 2) ^ (t & 7)) << 4));
          o[i] = mul2(o[i], make_float2(gdn_silu(z.x), gdn_silu(z.y)));
          o[i + 1] = mul2(o[i + 1], make_float2(gdn_silu(z.z), gdn_silu(z.w)));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[kZFree]);
      }
      if (p.out_bf16) {
#pragma unroll
        for (int i = 0; i < W / 2; i += 4)
          *reinterpret_cast<uint4*>(ss + t * 64 + ((((col + 2 * i) >> 3) ^ ((t >> 1) & 3)) << 4)) =
              make_uint4(pack_bf16(o[i].x, o[i].y), pack_bf16(o[i + 1].x, o[i + 1].y), pack_bf16(o[i + 2].x, o[i + 2].y),
                         pack_bf16(o[i + 3].x, o[i + 3].y));
      } else {
#pragma unroll
        for (int i = 0; i < W / 2; i += 2)
          *reinterpret_cast<float4*>(ss + t * 128 + ((((col + 2 * i) >> 2) ^ (t & 7)) << 4)) =
              make_float4(o[i].x, o[i].y, o[i + 1].x, o[i + 1].y);
      }
    };
    auto store = [&](int c) {
      named_bar_sync(named + kBarTurn, 128);
      const int have = *abort ? 0 : min(kRows, rows_left - c * kRows), i0 = ((warp >> 2) & 1) * 64 + t;  // of 128
      const int64_t to = (int64_t)(first_row + c * kRows) * p.out_row + h * p.out_head + col0 + half * kHalf;
      if (p.out_bf16) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int at = i * 128 + i0, row = at >> 2, pc = at & 3;
          if (row < have)
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + to + row * p.out_row + 8 * pc) =
                *reinterpret_cast<const uint4*>(ss + row * 64 + ((pc ^ ((row >> 1) & 3)) << 4));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = i * 128 + i0, row = at >> 3, pc = at & 7;
          if (row < have)
            *reinterpret_cast<float4*>(static_cast<float*>(p.out) + to + row * p.out_row + 4 * pc) =
                *reinterpret_cast<const float4*>(ss + row * 128 + ((pc ^ (row & 7)) << 4));
        }
      }
    };
    for (int c = 0; c < chunks; ++c) {
      const Decays* dec = reinterpret_cast<const Decays*>(smem + kOffDec) + (c & 1);
      float2 x[W / 2];
      float all;
      if (top) {
        take(named + kBarD1, 128);
        const float keep = dec->keep[t], left = dec->left[t], beta = dec->beta[t], bu = beta * up, bk = -beta * keep;
        all = dec->keep[kRows - 1];
        ld_sums<W>(acc + kAccD1, kHalf, x);
#pragma unroll
        for (int i = 0; i < W / 2; ++i) x[i] = fma2(both(bk), x[i], mul2(bf16_pair(v[i]), both(bu)));
        put_sides<W>(us, t, col, x);
        give(named + kBarR, 128);
        if (c + 1 < chunks) {
          fetch_v(c + 1);
          tell_values(c + 1);
        }
        take(named + kBarD2, 128);
        ld_sums<W>(acc + kAccD2, kHalf, x);
#pragma unroll
        for (int i = 0; i < W / 2; ++i) x[i] = mul2(x[i], both(left));
        put_sides<W>(us, t, col, x);
        give(named + kBarU, 128);
      } else {
        wait(kD1 + half, c);
        tc_fence_after_sync();
        const float keep = dec->keep[t], by = down * p.scale;
        all = dec->keep[kRows - 1];
        float2 y[W / 2];
        ld_sums<W>(acc + kAccD1, kHalf, y);
        if (c > 0) finish(c - 1);
        wait(kD2 + half, c);
        tc_fence_after_sync();
        ld_sums<W>(acc + kAccD2, kHalf, x);
        float2 sq = both(0.0f);
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
          o[i] = mul2(fma2(both(keep), y[i], x[i]), both(by));
          sq = fma2(o[i], o[i], sq);
        }
        if (p.norm_w && !*abort) {
          // the row's sum of squares goes to all of the cluster
          if (warp == 2 && lane == 0) mbar_arrive_expect_tx(&bar[kSum0 + (c & 1)], kSlices * 4 * kRows * 4);
          const uint32_t at = sum_to + (((c & 1) * kSlices * 4 + me * 4 + (warp >> 2)) * kRows + t) * 4;
#pragma unroll
          for (int i = 0; i < kSlices; ++i) st_async(map_rank(at, i), sq.x + sq.y, map_rank(smem_u32(&bar[kSum0 + (c & 1)]), i));
        }
        if (c > 0) store(c - 1);
      }
      take(named + kBarD3, 256);
      ld_sums<W>(acc + kAccD3, kHalf, x);
#pragma unroll
      for (int i = 0; i < W / 2; ++i) S[i] = fma2(both(all), S[i], mul2(x[i], both(down)));
      if (c + 1 < chunks) {
        put_state(c + 1);
        give(named + kBarS, 256);
        tell_state(c + 1);
        if ((threadIdx.x & 255) == 0) most[(c + 3) & 3] = most[4 + ((c + 3) & 3)] = 0;  // (the chunk before this one's: read by all)
      }
    }
    if (!top) {
      finish(chunks - 1);
      store(chunks - 1);
    }
    if (!*abort) {
#pragma unroll
      for (int i = 0; i < W / 2; i += 2) *reinterpret_cast<float4*>(st + 2 * i) = make_float4(S[i].x, S[i].y, S[i + 1].x, S[i + 1].y);
    }
  } else if (warp < 18) {
    // ------------------------------------------------------------------ a half's products
    const int half = warp - 16, named = half * kNamed;
    const uint32_t kq = smem_u32(smem + kOffKq), tp = smem_u32(smem + kOffTpt), acc = tmem + half * kAccHalf;
    const uint64_t ss = desc_mn(smem_u32(smem + kOffS + half * 16384), 0), us = desc_mn(smem_u32(smem + kOffU + half * 8192), 0);
    for (int c = 0; c < chunks; ++c) {
      const uint32_t kqc = kq + (c & 1) * 32768, tpc = tp + (c & 1) * 2 * kPart;
      wait(kReady0 + (c & 1), c >> 1);
      take(named + kBarS, 256);
      if (elect_one()) {
        const uint64_t a = umma_desc_sw128(kqc);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_f16(acc + kAccD1, a + (k >> 2) * (16384 >> 4) + (k & 3) * 2, ss + k * (2048 >> 4), kIdesc<128, 64, false, true>, k > 0);
        umma_commit(&bar[kD1 + half]);
      }
      __syncwarp();
      wait(kD1 + half, c);
      give(named + kBarD1, 128);
      take(named + kBarR, 128);
      if (elect_one()) {
        const uint64_t a = umma_desc_sw128(tpc);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          mma_f16(acc + kAccD2, a + 2 * k, us + k * (2048 >> 4), kIdesc<128, 64, false, true>, k > 0);
          mma_f16(acc + kAccD2, a + (kPart >> 4) + 2 * k, us + k * (2048 >> 4), kIdesc<128, 64, false, true>, 1);
        }
        umma_commit(&bar[kD2 + half]);
      }
      __syncwarp();
      wait(kD2 + half, c);
      give(named + kBarD2, 128);
      take(named + kBarU, 128);
      if (elect_one()) {
        const uint64_t a = desc_mn(kqc, 16384);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_f16(acc + kAccD3, a + k * (2048 >> 4), us + k * (2048 >> 4), kIdesc<128, 64, true, true>, k > 0);
        umma_commit(&bar[kD3 + half]);
      }
      __syncwarp();
      wait(kD3 + half, c);
      give(named + kBarD3, 256);
    }
    if (__any_sync(0xffffffffu, *abort != 0)) {  // what was issued is done with before the TMEM goes
      if (elect_one()) {
        umma_commit(&bar[kDrain + half]);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait_suspend(&bar[kDrain + half], 0, 20000u) && globaltimer_ns() - t0 < 1000000000ull) {
        }
      }
      __syncwarp();
    }
  } else if (warp == 18) {
    // ------------------------------------------------------------------ K, Q, V, z and the records
    // A barrier takes a copy's bytes only when it is done with the copy before: after a wait that gave up no copy is issued,
    // and those that were are waited for before the block ends.
    const int hk = h / p.group;
    int copied = 0, gates = 0;  // chunks of which all but z, and of which z, was asked for
    auto dead = [&]() { return __any_sync(0xffffffffu, *abort != 0); };
    auto load_z = [&](int c) {
      if (!p.z) return;
      if (c >= 1) doze(kZFree, c - 1);
      if (dead()) return;
      gates = c + 1;
      unsigned char* zs = smem + kOffZ;
      const int first = c * kRows, have = min(kRows, rows_left - first);
      if (p.z_wide) {
        if (elect_one()) {
          mbar_arrive_expect_tx(&bar[kZ], kRows * kCols * 4);
#pragma unroll
          for (int i = 0; i < kCols / 32; ++i)
            tma_load_3d_tx(zs + i * kRows * 128, &maps.z, col0 + 32 * i, h, first_row + first, &bar[kZ]);
        }
        __syncwarp();
      } else {
        const float* z0 = p.z + (first_row + first) * p.z_row + h * p.z_head + col0;
#pragma unroll 8
        for (int u = 0; u < kRows * kCols / 32; ++u) {
          const int at = u * 32 + lane, x = at / kCols, cl = at % kCols;
          if (x < have)
            *reinterpret_cast<float*>(zs + (cl >> 5) * kRows * 128 + x * 128 + ((((cl >> 2) & 7) ^ (x & 7)) << 4) + 4 * (cl & 3)) =
                z0[x * p.z_row + cl];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[kZ]);
      }
    };
    for (int c = 0; c < chunks; ++c) {
      if (c >= 2) {
        doze(kD3, c - 2);
        doze(kD3 + 1, c - 2);
      }
      if (dead()) break;
      copied = c + 1;
      const int first = c * kRows, have = min(kRows, rows_left - first);
      unsigned char* to = smem + kOffKq + (c & 1) * 32768;
      if (elect_one()) {
        uint64_t* land = &bar[kLand0 + (c & 1)];
        mbar_arrive_expect_tx(land, 32768 + kRecord + kRows * kCols * 2);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          tma_load_3d_tx(to + i * 16384, &maps.k, 64 * i, hk, first_row + first, land);
          tma_load_3d_tx(to + i * 16384 + 8192, &maps.q, 64 * i, hk, first_row + first, land);
        }
        // (V of two chunks before is in registers since that chunk's state was made)
        tma_load_3d_tx(smem + kOffV + (c & 1) * 8192, &maps.v, col0, h, first_row + first, land);
        const unsigned char* record = records.at + (record_of(records, d, s, begin + c) * p.nv + h) * kRecord;
        bulk_g2s_nohint(smem + kOffTpt + (c & 1) * 2 * kPart, record, 2 * kPart, land);
        bulk_g2s_nohint(smem + kOffDec + (c & 1) * sizeof(Decays), record + 2 * kPart, sizeof(Decays), land);
      }
      __syncwarp();
      doze(kLand0 + (c & 1), c >> 1);
      if (have < kRows)  // the rows behind the sequence's last: others', whatever they hold
        for (int i = lane; i < (kRows - have) * 32; i += 32) {
          const int row = have + (i >> 5), at = i & 31;
          *reinterpret_cast<uint4*>(to + (at >> 4) * 16384 + ((at >> 3) & 1) * 8192 + row * 128 + ((at & 7) << 4)) = make_uint4(0, 0, 0, 0);
        }
      if (!dbg.unreachable) {
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[kReady0 + (c & 1)]);
      }
      if (c > 0) load_z(c - 1);  // (wanted when the next chunk is on its way)
    }
    load_z(chunks - 1);
    if (dead()) {
      auto drain = [&](int b, int phase) {
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait_suspend(&bar[b], phase & 1, 20000u) && globaltimer_ns() - t0 < 1000000000ull) {
        }
      };
      for (int c = max(0, copied - 2); c < copied; ++c) drain(kLand0 + (c & 1), c >> 1);
      if (gates && p.z_wide) drain(kZ, gates - 1);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();  // (no CTA leaves while another may still store into it)
  if (*abort) {    // (and a store that nothing waited for lands within a microsecond)
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 50000) {
    }
    __syncwarp();
  }
  if (warp == 16) {
    tc_fence_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// ------------------------------------------------------------------ T and P T
constexpr int kOffTp = 32768, kOffDiag = kOffTp + 2 * kPart, kOffHi = kOffDiag + 4 * 16 * kLd * 4;  // behind [K; Q]
constexpr int kPrepSmem = kOffHi + 4 * 3 * kRows * 4 + 1024;

// The sequence and chunk whose record is x, the whole warp: false where there is none.
FAK_DEV bool find_chunk(const GdnParams& p, const Records& r, int64_t x, int lane, GdnSeq& d, int& s, int& c) {
  auto has = [&](int i, GdnSeq& e) {  // sequence i's chunk at x, or -1
    e = gdn_seq(p.c, kv_seq(p.c, i), i);
    const int rows = e.r1 - e.first;
    if (!e.ok || rows == 0 || (p.few && rows <= p.few)) return -1;
    const int64_t at = x - (r.dense ? (int64_t)i * r.length - r.begin : (int64_t)(e.r0 / kRows) + i);
    return at < r.begin || at >= r.begin + r.length || at * kRows >= rows ? -1 : (int)at;
  };
  if (r.dense) {
    s = (int)(x / r.length);
    return (c = has(s, d)) >= 0;
  }
  // where the starts rise, 32 probes a round
  int lo = 0, hi = p.c.n_seqs;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, i = lo + lane * step;
    const unsigned b = __ballot_sync(0xffffffffu, i < hi && (int64_t)(p.c.row_start[i] / kRows) + i <= x);
    const int n = __popc(b);
    if (n > 1) lo += (n - 1) * step;
    hi = min(lo + step, hi);
  }
  s = lo;
  if ((c = has(s, d)) >= 0) return true;
  // where they may fall beside numbers that are out of range: all sequences, where any is
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

// Block (x, h): record x, key head h.
__global__ void __launch_bounds__(kPrepThreads, 3) gdn_prepare_kernel(const __grid_constant__ GdnParams p, Records records) {
  extern __shared__ unsigned char raw[];
  unsigned char* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q2 = 2 * (lane & 3);
  const int hk = blockIdx.y;
  GdnSeq d;
  int s, c;
  if (!find_chunk(p, records, blockIdx.x, lane, d, s, c)) return;
  const int rows = d.r1 - d.first, first = c * kRows, have = min(kRows, rows - first);
  unsigned char *kq = smem, *tp = smem + kOffTp;
  const uint32_t kqs = smem_u32(kq), tps = smem_u32(tp);
  float* diag = reinterpret_cast<float*>(smem + kOffDiag);

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
  // T and P T are zero above their blocks on the diagonal, which nothing writes
  for (int i = threadIdx.x; i < 2 * kPart / 16; i += kPrepThreads) *reinterpret_cast<uint4*>(tp + 16 * i) = make_uint4(0, 0, 0, 0);
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();

  // Rows 16 m .. of K K^T (m = w) and of Q K^T (m = 3 - w), ten tiles of 8 columns to a warp
  float kk[8][4] = {}, qk[8][4] = {};
  const int mk = w, mq = 3 - w;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    auto at = [&](int row, int piece) { return kqs + (piece >> 3) * 16384 + row * 128 + (((piece & 7) ^ (row & 7)) << 4); };
    uint32_t ak[4], aq[4];
    ldsm4(ak, at(16 * mk + (lane & 15), 2 * k + (lane >> 4)));
    ldsm4(aq, at(64 + 16 * mq + (lane & 15), 2 * k + (lane >> 4)));
#pragma unroll
    for (int j = 0; j < 8; j += 2) {  // rows 8 j .. +15 of K: two tiles
      if (j > 2 * max(mk, mq)) continue;
      uint32_t b[4];
      ldsm4(b, at(8 * j + (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
      const uint32_t b0[2] = {b[0], b[1]}, b1[2] = {b[2], b[3]};
      if (j <= 2 * mk) {
        mma16(kk[j], ak, b0);
        mma16(kk[j + 1], ak, b1);
      }
      if (j <= 2 * mq) {
        mma16(qk[j], aq, b0);
        mma16(qk[j + 1], aq, b1);
      }
    }
  }

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
      float* mine = reinterpret_cast<float*>(smem + kOffHi) + w * 3 * kRows + 2 * lane;
      *reinterpret_cast<float2*>(mine) = make_float2(hi[0], hi[1]);
      *reinterpret_cast<float2*>(mine + kRows) = make_float2(lo[0], lo[1]);
      *reinterpret_cast<float2*>(mine + 2 * kRows) = make_float2(b[0], b[1]);
      unsigned char* record = records.at + ((int64_t)blockIdx.x * p.nv + h) * kRecord + 2 * kPart + 8 * lane;
      *reinterpret_cast<float2*>(record) = make_float2(exp2_approx(hi[0] + lo[0]), exp2_approx(hi[1] + lo[1]));
      *reinterpret_cast<float2*>(record + 4 * kRows) =
          make_float2(exp2_approx((hi_end - hi[0]) + (lo_end - lo[0])), exp2_approx((hi_end - hi[1]) + (lo_end - lo[1])));
      *reinterpret_cast<float2*>(record + 8 * kRows) = make_float2(b[0], b[1]);
    }
    __syncthreads();
    for (int hh = 0; hh < heads; ++hh) {
      const int h = hk * p.group + h0 + hh;
      const float* hi = reinterpret_cast<const float*>(smem + kOffHi) + hh * 3 * kRows;
      const float *lo = hi + kRows, *beta = hi + 2 * kRows;
      // A and P from K K^T and Q K^T by the decays, to the places of T and P T
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int tile = m ? mq : mk, row = 16 * tile + g;
        const float h0r = hi[row], l0r = lo[row], h1r = hi[row + 8], l1r = lo[row + 8];
        const float b0 = m ? 1.0f : beta[row], b1 = m ? 1.0f : beta[row + 8];
        const int last0 = m ? row : row - 1, last1 = last0 + 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (j > 2 * tile + 1) continue;
          const int col = 8 * j + q2;
          const float2 hc = *reinterpret_cast<const float2*>(hi + col), lc = *reinterpret_cast<const float2*>(lo + col);
          const float* x = m ? qk[j] : kk[j];
          float y[4] = {b0 * exp2_approx((h0r - hc.x) + (l0r - lc.x)) * x[0], b0 * exp2_approx((h0r - hc.y) + (l0r - lc.y)) * x[1],
                        b1 * exp2_approx((h1r - hc.x) + (l1r - lc.x)) * x[2], b1 * exp2_approx((h1r - hc.y) + (l1r - lc.y)) * x[3]};
          // (a zero that masks is put there, not multiplied by: it must not meet an infinity)
          if (col > last0) y[0] = 0.0f;
          if (col + 1 > last0) y[1] = 0.0f;
          if (col > last1) y[2] = 0.0f;
          if (col + 1 > last1) y[3] = 0.0f;
          put_block(tp, m * kRows + 16 * tile, j, y, 1.0f, lane);
          if (!m && j >= 2 * tile) {
            *reinterpret_cast<float2*>(diag + row * kLd + (col & 15)) = make_float2(y[0], y[1]);
            *reinterpret_cast<float2*>(diag + (row + 8) * kLd + (col & 15)) = make_float2(y[2], y[3]);
          }
        }
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
        // P T in place of P, by blocks of 16 x 16 (m, j): sums over k = j .. m, five steps to a warp
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
        __syncthreads();  // (P is read)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int m = mine >> (8 * i + 4) & 15, j = mine >> (8 * i) & 15;
          if (m == 15) break;
#pragma unroll
          for (int u = 0; u < 2; ++u) put_block(tp, kRows + 16 * m, 2 * j + u, y[i][u], 1.0f, lane);
        }
      }
      fence_async();
      __syncthreads();
      if (threadIdx.x == 0) {
        unsigned char* record = records.at + ((int64_t)blockIdx.x * p.nv + h) * kRecord;
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

cudaError_t launch(const GdnParams& p, const ChunkMaps& maps, const Records& records, const ChunkDebug& dbg, int* status, int dev,
                   cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = kv_smem_limit(gdn_chunk_kernel, kChunkSmem, dev, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)p.c.n_seqs * p.nv * kSlices));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kChunkSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kSlices;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gdn_chunk_kernel, p, maps, records, dbg, status);
}

constexpr int64_t kScratch = 1LL << 30;  // most bytes of records at a time; more chunks than they hold go in several launches

}  // namespace

cudaError_t gdn_chunk_launch(const GdnParams& p, unsigned long long timeout_ns, int unreachable, int* status, int dev, cudaStream_t s) {
  cudaError_t e = encoder();
  if (e != cudaSuccess) return e;
  ChunkMaps maps;
  memset(&maps, 0, sizeof(maps));
  const int nk = p.nv / p.group;
  if (!rows_map(&maps.k, p.k, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, p.c.rows, nk, p.k_row, p.k_head) ||
      !rows_map(&maps.q, p.q, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, p.c.rows, nk, p.q_row, p.q_head) ||
      !rows_map(&maps.v, p.v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.c.rows, p.nv, p.v_row, p.v_head) ||
      (p.z && p.z_wide && !rows_map(&maps.z, p.z, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, p.c.rows, p.nv, p.z_row, p.z_head)))
    return cudaErrorInvalidValue;
  const ChunkDebug dbg{timeout_ns, unreachable};
  // records of all chunks, where they are few enough; else of a stretch of every sequence at a time
  const int longest = (int)((std::min<int64_t>(p.c.max_q, p.c.rows) + kRows - 1) / kRows);
  const int64_t head = (int64_t)p.nv * kRecord, all = (p.c.rows / kRows + p.c.n_seqs) * head;
  Records records{nullptr, 0, longest, 0};
  int64_t bytes = all;
  if (all > kScratch) {
    records.dense = 1;
    records.length = (int)std::min<int64_t>(longest, std::max<int64_t>(1, kScratch / (p.c.n_seqs * head)));
    bytes = (int64_t)p.c.n_seqs * records.length * head;
  }
  void* scratch = nullptr;
  e = fak_scratch_alloc(&scratch, (size_t)bytes, s);
  if (e != cudaSuccess) return cudaErrorMemoryAllocation;
  records.at = static_cast<unsigned char*>(scratch);
  static std::atomic<uint64_t> done{0};
  e = kv_smem_limit(gdn_prepare_kernel, kPrepSmem, dev, done);
  for (; e == cudaSuccess && records.begin < longest; records.begin += records.length) {
    const int64_t slots = records.dense ? (int64_t)p.c.n_seqs * records.length : p.c.rows / kRows + p.c.n_seqs;
    gdn_prepare_kernel<<<dim3((unsigned)slots, (unsigned)nk), kPrepThreads, kPrepSmem, s>>>(p, records);
    e = cudaGetLastError();
    if (e == cudaSuccess) e = launch(p, maps, records, dbg, status, dev, s);
  }
  const cudaError_t f = cudaFreeAsync(scratch, s);
  return e != cudaSuccess ? e : f;
}
