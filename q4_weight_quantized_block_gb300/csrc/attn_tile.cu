// Attention of blocks of rows over the paged KV cache on the 5th-generation tensor cores.
//
// A block holds up to 128 rows of one sequence and KV head (twice that in a pair of CTAs): whole tokens, a row for
// each of their query heads of the group, so grouped heads fill the block whether the sequence has one new token or
// thousands.  Per
// tile of 128 keys
//   S = Q K^T (f32 in TMEM),  P = exp2(c S - m) (bf16, in S's own TMEM columns),  O += P V (f32 in TMEM)
// with the running maximum m and sum of the softmax.  m moves only when a row's maximum passes it by 8: until then
// weights reach at most 2^8, which bf16 and f32 hold as well as 1, and O is not rescaled.
//
// Sequences of more than 128 rows take the paired form (cta_group::2, heads of 128 and 256): the two CTAs hold 128
// rows each, and of every tile of K half the keys and of V half the dims.  With a CTA to itself a tile of 128 rows and
// keys at dh 256 reads 192 KB and takes 128 KB of copies through shared memory in the 2048 cycles that its MMAs last,
// more than the 128 bytes a cycle that it has; the pair halves K's and V's part, and the L2 traffic with it.
//
// A CTA (a pair) works on one block after the other until none is left: it takes over blocks of the grid that have not
// started (cluster launch control), so the longest, which come first, are dealt out as CTAs get free, and a block's
// loads and first scores run while the block before it is still being finished.
//
//   warps 0-7      softmax and results: warp w and w + 4 share rows 32 (w % 4) .. +31, half of the keys each
//   warp 8         TMEM owner; in the first CTA the MMA issuer
//   warps 9, 10    TMA of Q and K, and of V, by pages, each into a ring of its own (one warp needs some 500 cycles for a
//                  stage), in the 128-byte-swizzled layouts the MMAs read: Q and K 64 dims wide with the dims
//                  running (K-major), V keys by dims as stored (MN-major)
//   warp 11        the next block: takes it, works out its rows and keys
//   warps 12-19    for an 8-bit cache, codes to bf16, four warps K's and four V's: the copies land in rings of their own
//                  and they fill the MMAs' rings from them (12-15, for a bf16 cache: V of the tiles that a mask cuts
//                  is mended)
// Weights are rounded to bf16, off by 2^-8 of themselves at most: that is V's type, and a weight is A to V's B.  (8-bit
// codes could be f16, which would keep weights to 2^-11 but wants a base that holds the values' scales, as few rows have.)
// S has two or three buffers, so the next tile's S = Q K^T runs while the softmax works.
// 8-bit codes become bf16 exactly; their scales multiply the scores' columns and the weights instead.
// A weight of zero times a value that is not finite would be NaN, so in the tiles that a mask cuts a bf16 V is
// mended in shared memory: keys past the last row's position are made zeros, and so are values that are not
// finite, which the rows that do see them get added at the end.  (Codes are always finite, and a weight of zero is not
// multiplied by a scale.)  Scores of masked keys are replaced, whatever they are.
//
// A prompt of 8,192 tokens, 24 query and 4 KV heads of 256, in bf16: 594 to 620 us, 1.33 to 1.39 PFLOP/s, under the power
// limit's clocks (527 us, 1.56, from a rest); 512 tokens after 7,680 keys 98 us.  Heads of 128 are bound by the softmax
// warps, whose phases (scores, maximum, exponents) follow one another; 8-bit codes by those warps' scales and the conversion
// beside them: 8 x 1,024 tokens after 4,001 keys in bf16 611 us, in e4m3 927, with no unit above 45% busy.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "attn_device.cuh"
#include "fak.h"
#include "fak_device.cuh"
#include "fak_tc.cuh"

namespace {

constexpr int kPanel = 16384;  // 64 dims of Q's 128 rows

template <int DH, int KIND, int CG>
struct Cfg {
  static constexpr bool quant = KIND != FAK_KV_BF16;
  static constexpr int dv = DH / CG;                 // dims of V a CTA holds
  static constexpr int stage = !quant && CG == 2 && DH == 256 ? 32768 : 16384;
  static constexpr int raw = stage / 2;              // bytes of a stage's codes
  static constexpr int chunks = 256 * dv / stage;    // stages of one tile of K or of V
  static constexpr int vkeys = kTileN / chunks;      // keys of one V stage
  static constexpr int panels = stage / 8192 < DH / 64 ? stage / 8192 : DH / 64;  // 64 dims in a K stage, by 64 keys
  static constexpr int khalves = stage / 8192 / panels;  // (dh 64: two halves of a tile's keys)
  static constexpr int sbufs = DH == 256 ? 2 : 3;    // S buffers: 512 TMEM columns, less O's
  // stages of K, of V, and of their codes on their way to bf16
  static constexpr int ks = stage == 32768 ? 2 : quant ? (DH == 256 ? 3 : 4) : DH == 256 ? 4 : 5;
  static constexpr int vs = ks;
  static constexpr int rs = quant ? 2 : 0;
  // tiles whose scales are held at once: a tile's are loaded when the stage rs + ks stages before its first is
  // done with, as that tile's K was loaded, so the softmax is at most sbufs tiles further back
  static constexpr int slots = 1 + (rs + ks + chunks - 1) / chunks + sbufs;
  static constexpr int warps = quant ? 20 : 16;
  static constexpr int threads = warps * 32;
  static constexpr int off_k = kTileM * DH * 2;
  static constexpr int off_v = off_k + ks * stage;
  static constexpr int off_rk = off_v + vs * stage;
  static constexpr int off_rv = off_rk + rs * raw;
  static constexpr int off_scales = off_rv + rs * raw;
  static constexpr int off_red = off_scales + (quant ? slots * 2 * kTileN * 4 : 0);
  static constexpr int off_turn = off_red + 2 * 2 * kTileM * 4;  // where results turn, 2 KB to a softmax warp
  static constexpr int off_bar = off_turn + 8 * 2048;
  static constexpr int smem = off_bar + 688 + 1024;
  static_assert(smem <= 232448 - 1024, "shared memory exceeds the 227 KB per-block limit");
};

// A block: the whole pair's keys, this CTA's rows.
struct Unit {
  int seq, head, split;                  // KV head, piece of the keys
  int row0, token, nrows;                // the sequence's first row, the CTA's first token, its rows
  int p0, p_lo, p_hi, own_lo, own_hi;    // positions: of the sequence's first row, of the block's rows, of the CTA's
  int n, begin, direct, stop;            // key tiles, the first of them; the keys are one piece; there is no block
  KeyTiles kt;
};

// kind::f16 descriptors: f32 accumulator, bf16 operands; B_MN: B runs along N
template <int M, int N, bool B_MN>
constexpr uint32_t kIdescAttn = (1u << 4) | (1u << 7) | (1u << 10) | ((B_MN ? 1u : 0u) << 16) |
                                ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);

template <int CG>
FAK_DEV void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
}

template <int CG>
FAK_DEV void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
  if constexpr (CG == 1)
    umma_f16_ts(d, a, b, id, acc);
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
}

// Arrives on `bar` when the MMAs issued so far are done; in a pair on both CTAs' barriers at that offset.
template <int CG>
FAK_DEV void commit(uint64_t* bar) {
  if constexpr (CG == 1)
    umma_commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

FAK_DEV uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// The address of this CTA's shared variable in CTA `rank` of the pair.
FAK_DEV uint32_t map_to(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}

// Arrives on CTA 0's barrier, for its MMA issuer.  What that reads was written to TMEM or through
// fence.proxy.async, which order it; a release at cluster scope would wait a thousand cycles for every other store.
template <int CG>
FAK_DEV void arrive_first(uint64_t* bar) {
  if constexpr (CG == 1)
    mbar_arrive(bar);
  else
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(map_to(bar, 0)) : "memory");
}

FAK_DEV void arrive_release_cluster(uint64_t* bar, uint32_t rank) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(map_to(bar, rank)) : "memory");
}

FAK_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A tensor copy whose bytes count on CTA 0's barrier.
template <int CG>
FAK_DEV void load_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar, bool local) {
  if (CG == 1 || local)
    tma_load_3d_tx(dst, map, c0, c1, c2, bar);
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
        "%4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(map_to(bar, 0))
        : "memory");
}

// 128-byte swizzle with N running: 64 n by 8 k atoms, the next 64 n `lbo` bytes on, the next 8 k 1024 bytes on
FAK_DEV uint64_t desc_mn(uint32_t addr, uint32_t lbo) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// two f32 operations in one instruction
FAK_DEV uint64_t two(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
FAK_DEV void of_two(float& a, float& b, uint64_t d) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d)); }
FAK_DEV void mul2(float& a, float& b, float x, float y) {  // a *= x, b *= y
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(two(a, b)), "l"(two(x, y)));
  of_two(a, b, d);
}
FAK_DEV void add2(float& a, float& b, float x, float y) {  // a += x, b += y
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(two(a, b)), "l"(two(x, y)));
  of_two(a, b, d);
}
FAK_DEV void fma2(float& a, float& b, float x, float y, float f, float c) {  // a = x f + c, b = y f + c
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(two(x, y)), "l"(two(f, f)), "l"(two(c, c)));
  of_two(a, b, d);
}

FAK_DEV bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, "
      "p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Bounded wait; the clock, which takes hundreds of cycles to read, only after 64 tries.
FAK_DEV bool wait_bounded(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t timeout_ns) {
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait_suspend(bar, parity, 20000u)) return true;
  return mbar_wait_bounded(bar, parity, abort, timeout_ns);
}

// The n lowest bits (none for n <= 0, all from 64 on).
FAK_DEV uint64_t first_bits(int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; }

FAK_DEV bool tile_cut(int p_lo, int p_hi, int tile, const AttnParams& p) {
  return keys_cut(p_lo, p_hi, tile * kTileN, tile * kTileN + kTileN - 1, p.window, p.sinks);
}

// The cluster of the grid that is taken over, if one had not started: its first CTA's coordinates.
FAK_DEV void take_over(void* answer, uint64_t* bar, bool pair) {
  if (pair)
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.multicast::cluster::all.b128 "
        "[%0], [%1];" ::"r"(smem_u32(answer)),
        "r"(smem_u32(bar))
        : "memory");
  else
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     smem_u32(answer)),
                 "r"(smem_u32(bar))
                 : "memory");
}

FAK_DEV bool taken_over(const void* answer, int& x, int& y, int& z) {
  uint32_t got, a = 0, b = 0, c = 0;
  asm volatile(
      "{\n .reg .pred p;\n .reg .b128 r;\n ld.shared.b128 r, [%4];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n selp.u32 %3, 1, 0, p;\n"
      " mov.u32 %0, 0;\n mov.u32 %1, 0;\n mov.u32 %2, 0;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, %1, %2, _}, r;\n}"
      : "=r"(a), "=r"(b), "=r"(c), "=r"(got)
      : "r"(smem_u32(answer))
      : "memory");
  x = (int)a;
  y = (int)b;
  z = (int)c;
  return got != 0;
}

// Block x's sequence: the one of the last s with r0(s) / block + s <= x.  These starts rise by at least the
// sequence's number of blocks, so every block of rows has an x, and some x have none.  False: nothing to do.
// (Starts that are out of range are passed over, so that they leave out their own sequences alone.)
FAK_DEV bool find_unit(const AttnParams& p, int x, int head, int split, int rank, int lane, Unit& u) {
  auto before = [&](int start, int i) { return (unsigned)start <= (unsigned)p.c.rows && p.by_block(start) + i <= x; };
  int lo;
  KvSeq sq;
  if (p.c.n_seqs < 32) {
    const int start = lane <= p.c.n_seqs ? p.c.row_start[lane] : 0;
    const int len = lane < p.c.n_seqs ? p.c.kv_len[lane] : 0;
    lo = max(31 - __clz(__ballot_sync(0xffffffffu, lane < p.c.n_seqs && before(start, lane))), 0);
    sq.r0 = __shfl_sync(0xffffffffu, start, lo);
    sq.r1 = __shfl_sync(0xffffffffu, start, lo + 1);
    sq.len = __shfl_sync(0xffffffffu, len, lo);
    sq.ok = kv_seq_ok(p.c, sq);
  } else {
    lo = 0;
    for (int hi = p.c.n_seqs;;) {
      const int step = (hi - lo + 31) / 32, i = lo + lane * step, start = i < hi ? p.c.row_start[i] : -1;
      const bool yes = before(start, i);
      const int n = 32 - __clz(__ballot_sync(0xffffffffu, yes)), from = lo + max(n - 1, 0) * step;
      const unsigned later = __ballot_sync(0xffffffffu, !yes && (unsigned)start <= (unsigned)p.c.rows) & ~first_bits(n);
      const int to = later ? lo + (__ffs(later) - 1) * step : hi;
      const bool stuck = from == lo && to == hi;  // (all starts but lo's are out of range: not worth a search)
      lo = from;
      hi = to;
      if (step == 1 || stuck) break;
    }
    sq = kv_seq(p.c, lo);
  }
  if (!sq.ok) return false;
  const int64_t first = (int64_t)(x - (p.by_block(sq.r0) + lo)) * p.block;  // token
  if (first < 0 || first >= sq.r1 - sq.r0) return false;
  const int t0 = (int)first, tokens = min(p.block, sq.r1 - sq.r0 - t0), own = min(kTileM / p.group, p.block);
  u.seq = lo;
  u.head = head;
  u.split = split;
  u.row0 = sq.r0;
  u.token = t0 + rank * own;
  const int mine = max(0, min(own, tokens - rank * own));
  u.nrows = mine * p.group;
  u.p0 = sq.len - (sq.r1 - sq.r0);
  u.p_lo = u.p0 + t0;
  u.p_hi = u.p0 + t0 + tokens - 1;
  u.own_lo = u.p0 + u.token;
  u.own_hi = u.own_lo + max(mine, 1) - 1;
  u.kt = key_tiles(u.p_lo, u.p_hi, p.window, p.sinks, 7);
  u.direct = p.splits == 1 || u.kt.n <= p.per_split;
  u.begin = u.direct ? 0 : split * p.per_split;
  u.n = (u.direct || split == p.splits - 1 ? u.kt.n : min(u.kt.n, u.begin + p.per_split)) - u.begin;
  u.stop = 0;
  // a block whose keys are one piece, or that sees nothing at all, is the first split's
  return u.direct ? split == 0 : u.n > 0;
}

template <int DH, int KIND, int CG>
__global__ void __launch_bounds__(Cfg<DH, KIND, CG>::threads, 1)
    attn_tile_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap qmap,
                     const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, int* status) {
  using C = Cfg<DH, KIND, CG>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  float* scales = reinterpret_cast<float*>(smem + C::off_scales);  // [slot][key, value][128]
  float* red = reinterpret_cast<float*>(smem + C::off_red);        // [parity][half][128]
  // in a pair the MMA issuer waits on CTA 0's: kfull, vfull, mended, pfull, ofree, qfull
  uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + C::off_bar);
  uint64_t* kempty = kfull + C::ks;
  uint64_t* vfull = kempty + C::ks;
  uint64_t* vempty = vfull + C::vs;
  uint64_t* clean = vempty + C::vs;  // bf16: the stage's V has landed and is to be mended
  uint64_t* mended = clean + (C::quant ? 0 : C::vs);
  uint64_t* rkfull = mended + (C::quant ? 0 : C::vs);  // codes
  uint64_t* rkempty = rkfull + C::rs;
  uint64_t* rvfull = rkempty + C::rs;
  uint64_t* rvempty = rvfull + C::rs;
  uint64_t* scfull = rvempty + C::rs;
  uint64_t* sfull = scfull + (C::quant ? C::slots : 0);
  uint64_t* pfull = sfull + 3;
  uint64_t* odone = pfull + 3;
  uint64_t* pair = odone + 2;
  uint64_t* qfull = pair + 4;
  uint64_t* qempty = qfull + 1;
  uint64_t* ofree = qempty + 1;  // the block's results have left TMEM
  uint64_t* pdone = ofree + 1;   // bf16: V has been mended where it had to be (two: one CTA may be a block ahead)
  uint64_t* ufull = pdone + 2;   // blocks: handed out, done with
  uint64_t* uempty = ufull + 2;
  uint64_t* asked = uempty + 2;  // take_over's answer, and that both CTAs have read it
  uint64_t* heard = asked + 1;
  uint64_t* last = heard + 1;  // a block's copies of K have all been asked for
  uint64_t* drain = last + 1;
  static_assert((2 * C::ks + (C::quant ? 2 : 4) * C::vs + 4 * C::rs + (C::quant ? C::slots : 0) + 25) * 8 <= 656,
                "barriers exceed their area");
  uint8_t* answer = smem + C::off_bar + 656;  // 16 bytes
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::off_bar + 672);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::off_bar + 676);
  volatile int* odd = reinterpret_cast<volatile int*>(smem + C::off_bar + 680);
  __shared__ Unit units[2];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CG == 1 ? 0 : (int)cta_rank();
  if (warp == 1 && lane == 0) {
    for (int s = 0; s < C::ks; ++s) {
      mbar_init(&kfull[s], C::quant ? 4 * CG : 1);
      mbar_init(&kempty[s], 1);
    }
    for (int s = 0; s < C::vs; ++s) {
      mbar_init(&vfull[s], C::quant ? 4 * CG : 1);
      mbar_init(&vempty[s], 1);
      if (!C::quant) {
        mbar_init(&clean[s], 1);
        mbar_init(&mended[s], 4 * CG);
      }
    }
    for (int s = 0; s < C::rs; ++s) {
      mbar_init(&rkfull[s], 1);
      mbar_init(&rkempty[s], 4);
      mbar_init(&rvfull[s], 1);
      mbar_init(&rvempty[s], 4);
    }
    for (int s = 0; s < (C::quant ? C::slots : 0); ++s) mbar_init(&scfull[s], 1);
    for (int s = 0; s < 3; ++s) {
      mbar_init(&sfull[s], 1);
      mbar_init(&pfull[s], 8 * CG);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&odone[s], 1);
      mbar_init(&pdone[s], 4 * CG);
      mbar_init(&ufull[s], 1);
      mbar_init(&uempty[s], 11 + C::warps - 12);
    }
    for (int s = 0; s < 4; ++s) mbar_init(&pair[s], 2);
    mbar_init(qfull, 1 + p.unreachable);
    mbar_init(qempty, 1);
    mbar_init(ofree, 8 * CG);
    mbar_init(asked, 1);
    mbar_init(heard, CG);
    mbar_init(last, 1);
    mbar_init(drain, 1);
    *abort = 0;
    *odd = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    if constexpr (CG == 1) {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                   "r"(512u)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                   "r"(512u)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
  }
  if (warp == 2 && (blockIdx.x | blockIdx.y | blockIdx.z) == 0) {
    bool bad = false;  // every sequence's numbers are looked at once, also those that no block finds
    for (int i = lane; i < p.c.n_seqs; i += 32) bad |= !kv_seq(p.c, i).ok;
    if (bad) attn_record(status, FAK_ERR_DEVICE);
  }
  __syncwarp();
  tc_fence_before_sync();
  if constexpr (CG == 2)
    cluster_sync();  // both CTAs' barriers and TMEM stand
  else
    __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  const uint32_t tmem_s = tmem + DH;  // O in columns [0, DH), then the S buffers
  const uint64_t tmo = p.timeout_ns;
  // a whole warp waits: it goes on or gives up as one
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool done = __all_sync(0xffffffffu, wait_bounded(bar, parity, abort, tmo));
    if (!done) {
      if (!*abort) attn_record(status, FAK_ERR_TIMEOUT);
      *abort = 1;
    }
    return done;
  };
  // block k of this CTA; a warp is done with it
  auto handed = [&](int k) { return wait(&ufull[k & 1], (k >> 1) & 1) && !units[k & 1].stop; };
  auto release = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&uempty[k & 1]);
  };

  // Twenty warps start with 96 registers each (61440 in all): 128 for the softmax, 80 for the conversion, 56 for the rest.
  if constexpr (C::quant) {
    if (warp < 8)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
    else if (warp < 12)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
  }
  if (warp < 8) {
    // ---------------- softmax
    const int half = warp >> 2, quarter = warp & 3, row = 32 * quarter + lane;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const int row_token = p.by_group(row), row_head = row - row_token * p.group;
    // running over the blocks: S buffer and its parity, slot of the scales, products so far, exchanges with the other half
    int sb = 0, sph = 0, slot = 0, scph = 0, done = 0, meets = 0;
    bool ok = true;
    for (int k = 0; ok && handed(k); ++k) {
      const Unit& u = units[k & 1];
      const int n = u.n;
      const bool live = 32 * quarter < u.nrows;
      const int token = u.token + row_token, pos = u.p0 + token;
      float m = -INFINITY, l = 0.0f;
      for (int i = 0; i < n; ++i) {
        const int tile = key_tile(u.kt, u.begin + i), j0 = tile * kTileN + 64 * half;
        if (!(ok = wait(&sfull[sb], sph))) break;
        if constexpr (C::quant)
          if (!(ok = wait(&scfull[slot], scph))) break;
        // The product two tiles back is done.  With it known before this tile's weights are handed over, a barrier of
        // `odone` is never two phases past one that is waited for.  (Two S buffers: it came before these scores.)
        if (C::sbufs == 3 && i > 1 && !(ok = wait(&odone[done & 1], ((done - 2) >> 1) & 1))) break;
        tc_fence_after_sync();
        const uint32_t scol = tmem_s + lanes + (uint32_t)(sb * kTileN + 64 * half);
        if (live) {
          float t[64];
          {
            uint32_t raw[2][32];
            tmem_ld_cols<32>(scol, raw[0]);
            tmem_ld_cols<32>(scol + 32, raw[1]);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 64; ++c) t[c] = __uint_as_float(raw[c >> 5][c & 31]);
          }
          const float* sc = scales + (C::quant ? slot * 2 * kTileN + 64 * half : 0);
          if constexpr (C::quant) {
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
              const float4 f = *reinterpret_cast<const float4*>(sc + c);
              mul2(t[c], t[c + 1], f.x, f.y);
              mul2(t[c + 2], t[c + 3], f.z, f.w);
            }
          }
          const bool cut = tile_cut(u.own_lo, u.own_hi, tile, p);
          if (cut) {
            // the keys c that the row sees: c <= pos - j0, and beyond the window's edge or before the sinks' end
            uint64_t seen = first_bits(pos - j0 + 1);
            if (p.window) seen &= ~first_bits(pos - p.window - j0 + 1) | first_bits(p.sinks - j0);
            const uint32_t bits[2] = {(uint32_t)seen, (uint32_t)(seen >> 32)};
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (!(bits[c >> 5] & (1u << (c & 31)))) t[c] = -INFINITY;
          }
          float mx = -INFINITY;
#pragma unroll
          for (int c = 0; c < 64; ++c) mx = fmaxf(mx, t[c]);
          float* mine = red + (meets & 1) * 2 * kTileM;
          mine[half * kTileM + row] = mx;
          __syncwarp();
          if (lane == 0) mbar_arrive(&pair[quarter]);
          if (!(ok = wait(&pair[quarter], meets & 1))) break;
          ++meets;
          mx = fmaxf(mx, mine[(half ^ 1) * kTileM + row]) * p.scale;
          // a new base when the maximum passed it by 8, or is the first one seen
          const bool up = mx > m + 8.0f;
          if (__any_sync(0xffffffffu, up)) {
            const float next = up ? mx : m;
            const float f = up ? exp2_approx(m - next) : 1.0f;
            m = next;
            l *= f;
            if (i > 0) {
              if (!(ok = wait(&odone[(done + 1) & 1], ((done - 1) >> 1) & 1))) break;  // the product before
              tc_fence_after_sync();
#pragma unroll 1
              for (int c = 0; c < DH / 2; c += 32) {
                uint32_t o[32];
                const uint32_t at = tmem + lanes + (uint32_t)(half * (DH / 2) + c);
                tmem_ld_cols<32>(at, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st32(at, o);
              }
            }
          }
          const float base = m == -INFINITY ? 0.0f : m;
          float sum[2] = {0.0f, 0.0f};
          uint32_t w[32];
          auto weights = [&](auto masked) {
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
              float e[4];
#pragma unroll
              for (int j = 0; j < 4; j += 2) {
                fma2(e[j], e[j + 1], t[c + j], t[c + j + 1], p.scale, -base);
                e[j] = exp2_approx(e[j]);
                e[j + 1] = exp2_approx(e[j + 1]);
                add2(sum[0], sum[1], e[j], e[j + 1]);
              }
              if constexpr (C::quant) {
                const float4 f = *reinterpret_cast<const float4*>(sc + kTileN + c);
                const float v[4] = {f.x, f.y, f.z, f.w};
                if constexpr (decltype(masked)::value) {
                  // a weight of zero stays zero, whatever scale stands at the place of a key that is not seen
#pragma unroll
                  for (int j = 0; j < 4; ++j) e[j] = e[j] == 0.0f ? 0.0f : e[j] * v[j];
                } else {
                  mul2(e[0], e[1], v[0], v[1]);
                  mul2(e[2], e[3], v[2], v[3]);
                }
              }
              w[c / 2] = pack_bf16(e[0], e[1]);
              w[c / 2 + 1] = pack_bf16(e[2], e[3]);
            }
          };
          if (C::quant && cut)
            weights(std::true_type());
          else
            weights(std::false_type());
          l += sum[0] + sum[1];
          tmem_st32(scol, w);
          tmem_wait_st();
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) arrive_first<CG>(&pfull[sb]);
        ++done;
        if (++sb == C::sbufs) {
          sb = 0;
          sph ^= 1;
        }
        if (++slot == C::slots) {
          slot = 0;
          scph ^= 1;
        }
      }
      // ---------------- the rows' results
      if (ok && n > 0) ok = wait(&odone[(done - 1) & 1], ((done - 1) >> 1) & 1);
      if constexpr (!C::quant) {
        if (ok) ok = wait(&pdone[k & 1], (k >> 1) & 1);
        if (CG == 2 && ok) (void)try_wait_cluster(&pdone[k & 1], (k >> 1) & 1);  // (done: for its acquire of `odd`)
      }
      if (ok && live && n > 0) {
        tc_fence_after_sync();
        float* mine = red + (meets & 1) * 2 * kTileM;
        mine[half * kTileM + row] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(&pair[quarter]);
        ok = wait(&pair[quarter], meets & 1);
        ++meets;
        l += mine[(half ^ 1) * kTileM + row];
      }
      auto freed = [&]() {  // O may be written again
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) arrive_first<CG>(ofree);
      };
      if (ok && !live && n > 0) freed();
      if (ok && live) {
        const int head = u.head * p.group + row_head;
        // a row that sees nothing is zeros; one whose scores are all -inf is NaN, as 0 / 0 is
        const float scale = u.direct ? 1.0f / l : 1.0f;
        const bool mine = row < u.nrows, zero = pos < 0 || n == 0;
        const int64_t grow = u.row0 + token;
        const int64_t place = ((int64_t)u.split * p.c.rows + grow) * p.nq + head;
        if (!u.direct && mine && half == 0) p.stat[place] = make_float2(m, l);
        // 16 dims at a time turn in shared memory, so that a row's are stored 32 bytes (as f32: 64) in a piece:
        // four lanes a row, eight rows a step.  The next dims leave TMEM meanwhile.
        const int64_t to = u.direct ? grow * p.out_row + head * p.out_head : place * DH;
        const int64_t from = p.gate ? grow * p.gate_row + head * p.gate_head : 0;
        float* turn = reinterpret_cast<float*>(smem + C::off_turn) + warp * 512;
        const int d1 = half * (DH / 2);
        const bool gated = p.gate && u.direct;
        int64_t at[4], gate_at[4];
        bool there[4], blank[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int rr = 8 * e + (lane >> 2);
          at[e] = __shfl_sync(0xffffffffu, to, rr) + d1 + 4 * (lane & 3);
          gate_at[e] = __shfl_sync(0xffffffffu, from, rr) + d1 + 4 * (lane & 3);
          blank[e] = __shfl_sync(0xffffffffu, (int)zero, rr);
          there[e] = 32 * quarter + rr < u.nrows;
        }
        uint32_t o[2][16] = {};
        if (n > 0) tmem_ld_cols<16>(tmem + lanes + (uint32_t)d1, o[0]);
#pragma unroll 2
        for (int c = 0; c < DH / 2; c += 16) {
          uint32_t(&x)[16] = o[(c >> 4) & 1];
          float4 gate[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (gated && there[e] && !blank[e]) gate[e] = *reinterpret_cast<const float4*>(p.gate + gate_at[e] + c);
          if (n > 0) {
            tmem_wait_ld();
            if (c + 16 < DH / 2)
              tmem_ld_cols<16>(tmem + lanes + (uint32_t)(d1 + c + 16), o[((c >> 4) & 1) ^ 1]);
            else
              freed();
          }
          if (!C::quant && mine && *odd) {
            // values that are not finite, in tiles where they were left out: added for the rows that see them
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
              const int tile = key_tile(u.kt, u.begin + i);
              if (!tile_cut(u.p_lo, u.p_hi, tile, p)) continue;
#pragma unroll 1
              for (int j = tile * kTileN; j < min((tile + 1) * kTileN, pos + 1); ++j) {
                if (!sees(pos, j, p.window, p.sinks)) continue;
                int64_t v_at = kv_place(p.c, u.seq, j, u.head);
                if (v_at < 0) v_at = -1 - v_at;
                const uint16_t* v = reinterpret_cast<const uint16_t*>(p.c.v) + v_at * DH + d1 + c;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  if ((v[e] & 0x7F80u) == 0x7F80u)
                    x[e] = __float_as_uint(__uint_as_float(x[e]) + __uint_as_float((uint32_t)v[e] << 16));
              }
            }
          }
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<float4*>(turn + lane * 16 + ((e ^ ((lane >> 1) & 3)) << 2)) =
                make_float4(__uint_as_float(x[4 * e]) * scale, __uint_as_float(x[4 * e + 1]) * scale,
                            __uint_as_float(x[4 * e + 2]) * scale, __uint_as_float(x[4 * e + 3]) * scale);
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int rr = 8 * e + (lane >> 2);
            if (!there[e]) continue;
            float4 y = *reinterpret_cast<const float4*>(turn + rr * 16 + (((lane & 3) ^ ((rr >> 1) & 3)) << 2));
            if (blank[e]) y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (!u.direct) {
              *reinterpret_cast<float4*>(p.part + at[e] + c) = y;
              continue;
            }
            if (gated && !blank[e]) {
              y.x = gated_by(y.x, gate[e].x);
              y.y = gated_by(y.y, gate[e].y);
              y.z = gated_by(y.z, gate[e].z);
              y.w = gated_by(y.w, gate[e].w);
            }
            *reinterpret_cast<uint2*>(p.out + at[e] + c) = make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
          }
        }
      }
      release(k);
    }
  } else if (warp == 8) {
    // ---------------- MMA issuer
    // K: one CTA takes a tile as twice 64 keys, since its panels are 64 keys high; a pair holds 64 keys each
    constexpr uint32_t id_s = kIdescAttn<kTileM * CG, 64 * CG, false>, id_o = kIdescAttn<kTileM * CG, DH, true>;
    const uint64_t kd0 = umma_desc_sw128(smem_u32(smem + C::off_k)), qd = umma_desc_sw128(smem_u32(smem));
    // a stage's V: panels of 64 dims by vrows keys, all dims of the first keys, then of the next
    const int vshift = C::quant ? 31 - __clz(C::vkeys) : min(p.c.page_shift, 31 - __clz(C::vkeys));
    const uint64_t vd0 = desc_mn(smem_u32(smem + C::off_v), 128u << vshift);
    int kst = 0, kph = 0, vst = 0, sq = 0, sp = 0, pph = 0, blocks = 0, done = 0;
    uint32_t fulls = 0, mends = 0;  // a V stage that is mended has a barrier of its own: the parities go by uses
    bool ok = true;
    auto scores = [&](bool last) {
      const uint32_t d = tmem_s + (uint32_t)(sq * kTileN);
#pragma unroll
      for (int c = 0; c < C::chunks; ++c) {
        if (!(ok = wait(&kfull[kst], kph))) return;
        tc_fence_after_sync();
        const uint64_t kd = kd0 + (uint64_t)(kst * (C::stage >> 4));
        if (elect_one()) {
#pragma unroll
          for (int x = 0; x < C::stage / 8192; ++x) {  // the stage's parts: 64 dims of 64 keys
            const int part = c * (C::stage / 8192) + x;  // of the tile: the first 64 keys' panels, then the others'
            const int panel = part % (DH / 64), half = part / (DH / 64);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ss<CG>(d + 64 * half, qd + (uint64_t)((panel * kPanel + 32 * k) >> 4),
                         kd + (uint64_t)((x * 8192 + 32 * k) >> 4), id_s, panel | k);
          }
          commit<CG>(&kempty[kst]);
          if (c == C::chunks - 1) {
            commit<CG>(&sfull[sq]);
            if (last) commit<CG>(qempty);
          }
        }
        __syncwarp();
        if (++kst == C::ks) {
          kst = 0;
          kph ^= 1;
        }
      }
      sq = sq + 1 == C::sbufs ? 0 : sq + 1;
    };
    for (int k = 0; ok && handed(k); ++k) {
      const Unit& u = units[k & 1];
      const int n = u.n;
      if (rank == 0 && n > 0) {
        ok = wait(qfull, blocks & 1);
        for (int i = 0; i < min(C::sbufs, n) && ok; ++i) scores(i == n - 1);
        for (int i = 0; i < n && ok; ++i) {
          const bool mend = !C::quant && tile_cut(u.p_lo, u.p_hi, key_tile(u.kt, u.begin + i), p);
          if (!(ok = wait(&pfull[sp], pph))) break;
          if (i == 0 && blocks > 0 && !(ok = wait(ofree, (blocks - 1) & 1))) break;
          const uint32_t a = tmem_s + (uint32_t)(sp * kTileN);
#pragma unroll
          for (int c = 0; c < C::chunks; ++c) {
            if (!(ok = wait(mend ? &mended[vst] : &vfull[vst], ((mend ? mends : fulls) >> vst) & 1))) break;
            (mend ? mends : fulls) ^= 1u << vst;
            tc_fence_after_sync();
            const uint64_t vd = vd0 + (uint64_t)(vst * (C::stage >> 4));
            if (elect_one()) {
#pragma unroll
              for (int e = 0; e < C::vkeys / 16; ++e) {
                const int key = c * C::vkeys + 16 * e;  // weights: 64 keys in 32 columns, twice
                const int box = 16 * e >> vshift, in = 16 * e & ((1 << vshift) - 1);
                mma_ts<CG>(tmem, a + (uint32_t)((key >> 6) * 64 + (key & 63) / 2),
                           vd + (uint64_t)(((box << vshift) * (C::dv * 2) + in * 128) >> 4), id_o, (i | key) != 0);
              }
              commit<CG>(&vempty[vst]);
              if (c == C::chunks - 1) commit<CG>(&odone[done & 1]);
            }
            __syncwarp();
            if (++vst == C::vs) vst = 0;
          }
          ++done;
          if (ok && i + C::sbufs < n) scores(i + C::sbufs == n - 1);
          if (++sp == C::sbufs) {
            sp = 0;
            pph ^= 1;
          }
        }
        ++blocks;
      }
      release(k);
    }
    if ((!ok || *abort) && rank == 0 && elect_one()) {
      // what was issued completes before TMEM is freed
      commit<CG>(drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(drain, 0))
        if (globaltimer_ns() - t0 > 200000000ull) break;
    }
    __syncwarp();
  } else if (warp == 9 || warp == 10) {
    // ---------------- TMA: warp 9 Q, K and the scales, warp 10 V
    const bool value = warp == 10;
    const int kshift = min(p.c.page_shift, 6), krows = 1 << kshift;  // the maps' boxes: keys of K, of V
    const int vshift = min(p.c.page_shift, 31 - __clz(C::vkeys)), vrows = 1 << vshift;
    const int kpanels = krows == 64 ? C::panels : 1;  // and panels of K, which stand 64 keys apart
    const int boxes = kTileN >> kshift;
    const int S = C::quant ? C::rs : value ? C::vs : C::ks;
    constexpr int kw = C::panels * 64;  // 8-bit: bytes of a K stage's row
    uint64_t* const free = C::quant ? (value ? rvempty : rkempty) : value ? vempty : kempty;
    uint64_t* const lands = C::quant ? (value ? rvfull : rkfull) : value ? vfull : kfull;
    uint8_t* const to = smem + (C::quant ? (value ? C::off_rv : C::off_rk) : value ? C::off_v : C::off_k);
    int st = 0, ph = 1;  // the stage, the parity of its `free` (the first round is free already)
    int blocks = 0, slot = 0;
    uint32_t uses = 0xffffffffu, mends = 0xffffffffu;  // the parity of each stage's last use of `lands`, of `clean`
    bool ok = true;
    for (int k = 0; ok && handed(k); ++k) {
      const Unit& u = units[k & 1];
      const int n = u.n, g = u.head;
      // lane l: the vector index of key l * krows of the tile; keys past the last that a row sees take its
      // page: what lies there is masked
      auto places = [&](int i) {
        const int j =
            min(key_tile(u.kt, u.begin + i) * kTileN + (min(lane, boxes - 1) << kshift), u.p_hi & ~(krows - 1));
        int64_t at = kv_place(p.c, u.seq, j, g);
        if (at < 0) {
          attn_record(status, FAK_ERR_DEVICE);
          at = -1 - at;
        }
        return (int)at;
      };
      int ahead = n > 0 ? places(0) : 0;  // the next tile's, looked up early
      if (!value && n > 0) {
        // Q: panels of 64 dims, the group's heads of a token after token; rows past the block's are other rows', or zeros
        if (blocks > 0) ok = wait(qempty, (blocks - 1) & 1);
        if (!ok) break;
        ++blocks;
        const int bytes = kTileM / p.group * p.group * 128;
        if (rank == 0 && elect_one()) mbar_arrive_expect_tx(qfull, CG * (DH / 64) * bytes);
        __syncwarp();
        for (int c = 0; c < DH / 64; ++c) {
          if (elect_one())
            load_3d<CG>(smem + c * kPanel, &qmap, c * 64, g * p.group, u.row0 + u.token, qfull, false);
          __syncwarp();
        }
      }
      for (int i = 0; i < n && ok; ++i) {
        const int at = ahead;
        if (i + 1 < n) ahead = places(i + 1);
        if (C::quant && !value) {
          float* sc = scales + slot * 2 * kTileN;
          // (its last tile is done with: the rings hold fewer tiles than there are slots)
          if (elect_one()) mbar_arrive_expect_tx(&scfull[slot], 2 * kTileN * 4);
          __syncwarp();
          if (lane < boxes) {
            bulk_g2s_nohint(sc + lane * krows, p.c.ks + at, krows * 4, &scfull[slot]);
            bulk_g2s_nohint(sc + kTileN + lane * krows, p.c.vs + at, krows * 4, &scfull[slot]);
          }
          __syncwarp();
          slot = slot + 1 == C::slots ? 0 : slot + 1;
        }
        const bool mend = !C::quant && value && tile_cut(u.p_lo, u.p_hi, key_tile(u.kt, u.begin + i), p);
#pragma unroll 1
        for (int c = 0; c < C::chunks; ++c) {
          if (!(ok = wait(&free[st], ph))) break;
          // a pair's bytes count on CTA 0's barrier, but for codes and for V that is to be mended
          const bool local = C::quant || mend;
          uint64_t* bar = mend ? &clean[st] : &lands[st];
          uint8_t* dst = to + st * (C::quant ? C::raw : C::stage);
          if ((local || rank == 0) && elect_one())
            mbar_arrive_expect_tx(bar, C::quant ? C::raw : local ? C::stage : C::stage * CG);
          __syncwarp();
          (mend ? mends : uses) ^= 1u << st;
          if (!value) {
            // parts of 64 dims by 64 keys; a pair's CTA has its half of the keys
            const int part = c * (C::stage / 8192), panel = part % (DH / 64);
            const int first = 64 * (CG == 2 ? rank : part / (DH / 64));
            for (int r = 0; r < 64 * C::khalves; r += krows) {
              const int row = __shfl_sync(0xffffffffu, at, (first + r) >> kshift);
              if constexpr (C::quant) {
                if (elect_one()) tma_load_2d_tx(dst + r * kw, &kmap, panel * 64, row, bar);
              } else {
                for (int x = 0; x < C::panels; x += kpanels)
                  if (elect_one()) load_3d<CG>(dst + x * 8192 + r * 128, &kmap, 0, row, panel + x, bar, false);
              }
              __syncwarp();
            }
          } else {
            for (int r = 0; r < C::vkeys; r += vrows) {
              const int key = c * C::vkeys + r, row = __shfl_sync(0xffffffffu, at, key >> kshift) + (key & (krows - 1));
              if (elect_one()) {
                if constexpr (C::quant)
                  tma_load_2d_tx(dst + r * C::dv, &vmap, rank * C::dv, row, bar);
                else
                  load_3d<CG>(dst + r * C::dv * 2, &vmap, 0, row, rank * (C::dv / 64), bar, mend);
              }
              __syncwarp();
            }
          }
          if (++st == S) {
            st = 0;
            ph ^= 1;
          }
        }
      }
      if (!value && lane == 0) mbar_arrive(last);
      release(k);
    }
    // copies in flight land before the CTA can end (one that ran to its end has used every copy)
    if (lane == 0 && *abort) {
      auto landed = [&](uint64_t* bar, uint32_t parity) {
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(bar, parity & 1))
          if (globaltimer_ns() - t0 > 200000000ull) break;
      };
      for (int q = 0; q < S; ++q) {
        landed(&lands[q], uses >> q);
        if (!C::quant && value) landed(&clean[q], mends >> q);
      }
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 1000000ull) {  // Q and scales: a few kilobytes, landed long before this
      }
    }
    __syncwarp();
  } else if (warp == 11) {
    // ---------------- the blocks
    int x = blockIdx.x, y = blockIdx.y, z = blockIdx.z, k = 0;
    bool ok = true;
    auto hand = [&](const Unit& u) {
      if (!(ok = wait(&uempty[k & 1], ((k >> 1) & 1) ^ 1))) return;
      if (lane == 0) {
        units[k & 1] = u;
        mbar_arrive(&ufull[k & 1]);
      }
      __syncwarp();
      ++k;
    };
    for (int asks = 0; ok; ++asks) {
      Unit u;
      if (find_unit(p, ((int)gridDim.x - 1 - x) / CG, y, z, rank, lane, u)) hand(u);
      if (!ok) break;
      // Ask for the next one when this one's last keys are on their way: a few tiles before it is needed, and late
      // enough that it is not one that another SM would have begun at once (asked for at the start, 16 sequences' 64
      // blocks of 32 tiles were done by some 45 pairs of CTAs: 112 us, and 70 as it is).
      if (rank == 0 && k > 0 && !(ok = wait(last, (k - 1) & 1))) break;
      if (rank == 0 && asks > 0 && !(ok = wait(heard, (asks - 1) & 1))) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(asked, 16);
        if (rank == 0) take_over(answer, asked, CG == 2);
      }
      __syncwarp();
      // (also after a failure: the answer must not arrive in a CTA that has ended)
      const bool came = wait(asked, asks & 1);
      ok = ok && came && !*abort;
      if (!ok) break;
      const bool more = taken_over(answer, x, y, z);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive_first<CG>(heard);
      if (!more) break;
    }
    Unit none;
    none.stop = 1;
    none.n = 0;
    if (ok) hand(none);
  } else if (warp >= 12) {
    // ---------------- codes to bf16, V of cut tiles
    constexpr int T = 128;
    bool ok = true;
    if constexpr (C::quant) {
      // warps 12-15 K's stages, 16-19 V's; 16 codes to a thread and step
      const bool value = warp >= 16;
      const int tid = threadIdx.x - (value ? 16 : 12) * 32;
      constexpr int kwidth = C::panels * 4, vwidth = C::dv / 16;
      const int width_shift = value ? 31 - __clz(vwidth) : 31 - __clz(kwidth);
      const int panel = value ? C::vkeys * 128 : 8192;
      uint64_t *const rfull = value ? rvfull : rkfull, *const rempty = value ? rvempty : rkempty;
      uint64_t *const free = value ? vempty : kempty, *const fills = value ? vfull : kfull;
      const uint32_t fills_first = CG == 1 ? smem_u32(fills) : map_to(fills, 0);
      const int stages = value ? C::vs : C::ks;
      const uint8_t* const raw = smem + (value ? C::off_rv : C::off_rk);
      uint8_t* const ring = smem + (value ? C::off_v : C::off_k);
      int rs = 0, rph = 0, st = 0, ph = 1;
      for (int k = 0; ok && handed(k); ++k) {
        const int count = units[k & 1].n * C::chunks;
        for (int i = 0; i < count; ++i) {
          if (!(ok = wait(&rfull[rs], rph))) break;
          const uint4* src = reinterpret_cast<const uint4*>(raw + rs * C::raw);
          uint8_t* dst = ring + st * C::stage;
          uint4 q[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) q[e] = src[tid + e * T];
          if (!(ok = wait(&free[st], ph))) break;
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            const int e = tid + f * T, key = e >> width_shift, d = (e & ((1 << width_shift) - 1)) * 16;
            uint4 a, b;
            codes_to_bf16<KIND>(q[f].x, a.x, a.y);
            codes_to_bf16<KIND>(q[f].y, a.z, a.w);
            codes_to_bf16<KIND>(q[f].z, b.x, b.y);
            codes_to_bf16<KIND>(q[f].w, b.z, b.w);
            uint8_t* line = dst + (d >> 6) * panel + key * 128;
            const int e16 = (d & 63) >> 3;
            *reinterpret_cast<uint4*>(line + ((e16 ^ (key & 7)) << 4)) = a;
            *reinterpret_cast<uint4*>(line + (((e16 + 1) ^ (key & 7)) << 4)) = b;
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            if constexpr (CG == 1)
              mbar_arrive(&fills[st]);
            else
              asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(fills_first + 8 * st) : "memory");
            mbar_arrive(&rempty[rs]);  // after the stores, which came after the loads
          }
          if (++rs == C::rs) {
            rs = 0;
            rph ^= 1;
          }
          if (++st == stages) {
            st = 0;
            ph ^= 1;
          }
        }
        release(k);
      }
    } else {
      const int tid = threadIdx.x - 12 * 32;
      uint32_t landed = 0;  // parity of each stage's next use of `clean`
      int before = 0;       // V's stages of the blocks before
      const int vshift = min(p.c.page_shift, 31 - __clz(C::vkeys));
      for (int k = 0; ok && handed(k); ++k) {
        const Unit& u = units[k & 1];
        for (int i = 0; i < u.n && ok; ++i) {
          const int tile = key_tile(u.kt, u.begin + i);
          if (!tile_cut(u.p_lo, u.p_hi, tile, p)) continue;
          for (int c = 0; c < C::chunks; ++c) {
            const int st = (before + i * C::chunks + c) % C::vs;
            if (!(ok = wait(&clean[st], (landed >> st) & 1))) break;
            landed ^= 1u << st;
            uint4* v = reinterpret_cast<uint4*>(smem + C::off_v + st * C::stage);
            bool bad = false;
#pragma unroll
            for (int f = 0; f < C::stage / 16 / T; ++f) {
              const int e = tid + f * T, box = e / (C::dv / 8) >> vshift;  // a box: dv dims of 2^vshift keys
              const int j = tile * kTileN + c * C::vkeys + (box << vshift) + ((e >> 3) & ((1 << vshift) - 1));
              bool change = false;
              uint4 y = v[e];
              y.x = finite2(y.x, change);
              y.y = finite2(y.y, change);
              y.z = finite2(y.z, change);
              y.w = finite2(y.w, change);
              if (j > u.p_hi)
                v[e] = make_uint4(0, 0, 0, 0);
              else if (change)
                v[e] = y;
              bad |= change && j <= u.p_hi;
            }
            if (bad) {
              *odd = 1;  // (stays: later blocks of this CTA look for such values too, and find none of theirs)
              if constexpr (CG == 2)  // the other CTA's rows have these dims too
                asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_to((const void*)odd, rank ^ 1)), "r"(1)
                             : "memory");
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) arrive_first<CG>(&mended[st]);
          }
        }
        before = (before + u.n * C::chunks) % C::vs;
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 1) {
            mbar_arrive(&pdone[k & 1]);
          } else {
            arrive_release_cluster(&pdone[k & 1], 0);
            arrive_release_cluster(&pdone[k & 1], 1);
          }
        }
        release(k);
      }
    }
  }
  __syncwarp();
  tc_fence_before_sync();
  if constexpr (CG == 2)
    cluster_sync();  // no CTA of a pair ends while the other may still signal it
  else
    __syncthreads();
  if (warp == 8) {
    tc_fence_after_sync();
    if constexpr (CG == 1)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
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

// The cache's codes.  bf16: [panel of 64 dims][vector][64], boxes of `panels` panels of `rows` vectors of
// one page; 8-bit: [vector][dh], boxes of `width` bytes of `rows` vectors.
bool code_map(CUtensorMap* map, void* base, bool quant, int dh, int64_t n_vec, int width, int rows, int panels) {
  memset(map, 0, sizeof(*map));
  const cuuint64_t dim[3] = {(cuuint64_t)(quant ? dh : 64), (cuuint64_t)n_vec, (cuuint64_t)(dh / 64)};
  const cuuint64_t stride[2] = {(cuuint64_t)dh * (quant ? 1 : 2), 128};
  const cuuint32_t box[3] = {(cuuint32_t)width, (cuuint32_t)rows, (cuuint32_t)panels}, one[3] = {1, 1, 1};
  return g_encode(map, quant ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, quant ? 2 : 3, base,
                  dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  quant ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries: [row][head][dh], boxes of 64 dims of a group's heads of as many whole tokens as 128 rows hold.
bool query_map(CUtensorMap* map, const AttnParams& p, int dh) {
  memset(map, 0, sizeof(*map));
  const cuuint64_t dim[3] = {(cuuint64_t)dh, (cuuint64_t)p.nq, (cuuint64_t)p.c.rows};
  // (a stride that is never taken may be anything)
  const cuuint64_t head = p.nq > 1 ? (cuuint64_t)p.q_head * 2 : (cuuint64_t)dh * 2;
  const cuuint64_t stride[2] = {head, p.c.rows > 1 ? (cuuint64_t)p.q_row * 2 : head * p.nq};
  const cuuint32_t box[3] = {64, (cuuint32_t)p.group, (cuuint32_t)(kTileM / p.group)}, one[3] = {1, 1, 1};
  return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(p.q), dim, stride, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DH, int KIND, int CG>
cudaError_t launch(const AttnParams& p, int page, int64_t n_vec, int64_t blocks, int* status, int dev, cudaStream_t s) {
  using C = Cfg<DH, KIND, CG>;
  cudaError_t e = encoder();
  if (e != cudaSuccess) return e;
  CUtensorMap qmap, kmap, vmap;
  const int krows = std::min(page, 64), vrows = std::min(page, C::vkeys);
  if (!query_map(&qmap, p, DH)) return cudaErrorInvalidValue;
  if (!code_map(&kmap, p.c.k, C::quant, DH, n_vec, C::quant ? C::panels * 64 : 64, krows, krows == 64 ? C::panels : 1) ||
      !code_map(&vmap, p.c.v, C::quant, DH, n_vec, C::quant ? C::dv : 64, vrows, C::dv / 64))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> done{0};
  e = kv_smem_limit(attn_tile_kernel<DH, KIND, CG>, C::smem, dev, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((unsigned)(blocks * CG), (unsigned)p.c.n_kv, (unsigned)p.splits);
  cfg.blockDim = dim3(C::threads);
  cfg.dynamicSmemBytes = C::smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 2 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, attn_tile_kernel<DH, KIND, CG>, p, qmap, kmap, vmap, status);
}

template <int DH, int CG>
cudaError_t by_kind(int kind, const AttnParams& p, int page, int64_t n_vec, int64_t blocks, int* status, int dev,
                    cudaStream_t s) {
  return kind == FAK_KV_BF16   ? launch<DH, FAK_KV_BF16, CG>(p, page, n_vec, blocks, status, dev, s)
         : kind == FAK_KV_E4M3 ? launch<DH, FAK_KV_E4M3, CG>(p, page, n_vec, blocks, status, dev, s)
                               : launch<DH, FAK_KV_I8, CG>(p, page, n_vec, blocks, status, dev, s);
}

}  // namespace

cudaError_t attn_tile_launch(int kind, int dh, int page, int64_t n_vec, const AttnParams& p, int64_t blocks,
                             int* status, int dev, cudaStream_t s) {
  if (p.block > kTileM / p.group)
    return dh == 128 ? by_kind<128, 2>(kind, p, page, n_vec, blocks, status, dev, s)
                     : by_kind<256, 2>(kind, p, page, n_vec, blocks, status, dev, s);
  return dh == 64    ? by_kind<64, 1>(kind, p, page, n_vec, blocks, status, dev, s)
         : dh == 128 ? by_kind<128, 1>(kind, p, page, n_vec, blocks, status, dev, s)
                     : by_kind<256, 1>(kind, p, page, n_vec, blocks, status, dev, s);
}
