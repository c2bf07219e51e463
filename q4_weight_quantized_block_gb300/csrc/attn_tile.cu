// Attention of blocks of rows over the paged KV cache on the 5th-generation tensor cores.
//
// A block holds 128 rows of one sequence and KV head (256 in a pair of CTAs); a row is a (token, query head of
// the group) pair, so grouped heads fill the block whether the sequence has one new token or thousands.  Per
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
//   warps 0-7      softmax: warp w and w + 4 share rows 32 (w % 4) .. +31, half of the keys each
//   warp 8         TMEM owner; in the first CTA the MMA issuer
//   warp 9         TMA: K and V by pages in 16 KB stages of a ring, in the order the MMAs take them
//                  (K 0, K 1, V 0, K 2, V 1, ...), in the 128-byte-swizzled layouts the MMAs read: Q and K
//                  64 dims wide with the dims running (K-major), V keys by dims as stored (MN-major)
//   warps 12-15    for an 8-bit cache, codes to bf16: the copies land in a ring of their own and these warps fill
//                  the MMAs' ring from it; for a bf16 cache, V of the tiles that a mask cuts
// S has two or three buffers, so the next tile's S = Q K^T runs while the softmax works.
// 8-bit codes become bf16 exactly; their scales multiply the scores' columns and the weights instead.
// A weight of zero times a value that is not finite would be NaN, so in the tiles that a mask cuts a bf16 V is
// mended in shared memory: keys past the last row's position are made zeros, and so are values that are not
// finite, which the rows that do see them get added at the end.  (Codes are always finite, and a weight of zero is not
// multiplied by a scale.)  Scores of masked keys are replaced, whatever they are.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "attn_device.cuh"
#include "fak.h"
#include "fak_device.cuh"
#include "fak_tc.cuh"

namespace {

constexpr int kStageBytes = 16384;
constexpr int kSlots = 16;  // tiles whose scales are held at once (8-bit caches): more than the rings hold
constexpr int kRawBytes = kStageBytes / 2;

template <int DH, int KIND, int CG>
struct Cfg {
  static constexpr bool quant = KIND != FAK_KV_BF16;
  static constexpr int dv = DH / CG;                 // dims of V a CTA holds
  static constexpr int chunks = dv / 64;             // stages of one tile of K or of V
  static constexpr int vkeys = 8192 / dv;            // keys of one V stage
  static constexpr int panels = DH == 64 ? 1 : 2;    // a K stage: 64 keys by this many 64 dims (dh 64: twice 64 keys)
  static constexpr int sbufs = DH == 256 ? 2 : 3;    // S buffers: 512 TMEM columns, less O's
  static constexpr int stages = quant ? (DH == 256 ? 6 : 8) : DH == 256 ? 9 : DH == 128 ? 11 : 12;
  static constexpr int raw = !quant ? 0 : DH == 64 ? 6 : 5;  // stages of codes on their way to bf16
  static constexpr int threads = 16 * 32;
  static constexpr int off_ring = kTileM * DH * 2;
  static constexpr int off_raw = off_ring + stages * kStageBytes;
  static constexpr int off_scales = off_raw + raw * kRawBytes;
  static constexpr int off_red = off_scales + (quant ? kSlots * 2 * kTileN * 4 : 0);
  static constexpr int off_bar = off_red + 2 * 2 * kTileM * 4;
  static constexpr int smem = off_bar + 656 + 1024;
  static_assert(smem <= 232448 - 1024, "shared memory exceeds the 227 KB per-block limit");
};

// A block of rows: the whole pair's keys, this CTA's rows.
struct Unit {
  int seq, row0, rbase, nrows, p0, p_lo, p_hi, own_lo, own_hi, n, begin, direct, skip;
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

FAK_DEV float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

FAK_DEV uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

FAK_DEV uint32_t hmul2_bf16(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
FAK_DEV uint32_t hsub2_bf16(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Four 8-bit codes as four bf16, exactly.  e4m3: its exponent and significand bits set as bf16's stand for the
// value times 2^-120 (subnormals too).  int8: 128 + the low seven bits, less 128 or, for the negative, 256.
template <int KIND>
FAK_DEV void codes_to_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (KIND == FAK_KV_E4M3) {
    const uint32_t a = prmt(w, 0, 0x1404), b = prmt(w, 0, 0x3424);
    lo = hmul2_bf16(((a >> 4) & 0x07F007F0u) | (a & 0x80008000u), 0x7B807B80u);
    hi = hmul2_bf16(((b >> 4) & 0x07F007F0u) | (b & 0x80008000u), 0x7B807B80u);
  } else {
    const uint32_t a = prmt(w, 0, 0x4140), b = prmt(w, 0, 0x4342);
    lo = hsub2_bf16((a & 0x007F007Fu) | 0x43004300u, (a & 0x00800080u) | 0x43004300u);
    hi = hsub2_bf16((b & 0x007F007Fu) | 0x43004300u, (b & 0x00800080u) | 0x43004300u);
  }
}

// bf16 pair with values that are not finite made zero; sets odd if there was one
FAK_DEV uint32_t finite2(uint32_t w, bool& odd) {
  uint32_t m = 0xffffffffu;
  if ((w & 0x7F80u) == 0x7F80u) m &= 0xffff0000u;
  if ((w & 0x7F800000u) == 0x7F800000u) m &= 0x0000ffffu;
  odd |= m != 0xffffffffu;
  return w & m;
}

// One lane of a converged warp, the same each time: the compiler keeps what the lanes share in uniform registers
// around it, where TMA and MMA instructions want their operands (a branch on the lane's number costs 100
// cycles a load or MMA more).
FAK_DEV bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
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

FAK_DEV bool sees(int pos, int j, int window, int sinks) {
  return j <= pos && (!window || j > pos - window || j < sinks);
}

// Whether some row at positions p_lo .. p_hi does not see some key of the tile.
FAK_DEV bool tile_cut(int p_lo, int p_hi, int tile, int window, int sinks) {
  const int j0 = tile * kTileN, j1 = j0 + kTileN - 1;
  return !(j1 <= p_lo && (!window || j0 > p_hi - window || j1 < sinks));
}

// Block x's sequence: the one of the last s with r0(s) * group / block + s <= x.  These starts rise by at
// least the sequence's number of blocks, so every block of rows has an x, and some x have none.
FAK_DEV void find_unit(const AttnParams& p, int64_t x, int split, int rank, int lane, Unit& u) {
  int lo = 0, hi = p.c.n_seqs;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, i = lo + lane * step;
    const unsigned b =
        __ballot_sync(0xffffffffu, i < hi && (int64_t)p.c.row_start[i] * p.group / p.block + i <= x);
    const int n = __popc(b);
    if (n > 1) lo += (n - 1) * step;
    hi = min(lo + step, hi);
  }
  const KvSeq sq = kv_seq(p.c, lo);
  u.seq = lo;
  u.skip = 1;
  if (!sq.ok) return;
  const int64_t first = (x - ((int64_t)sq.r0 * p.group / p.block + lo)) * p.block;
  const int64_t total = (int64_t)(sq.r1 - sq.r0) * p.group;
  if (first < 0 || first >= total) return;
  const int rows = (int)min((int64_t)p.block, total - first);
  u.row0 = sq.r0;
  u.rbase = (int)first + rank * kTileM;
  u.nrows = max(0, min(kTileM, rows - rank * kTileM));
  u.p0 = sq.len - (sq.r1 - sq.r0);
  u.p_lo = u.p0 + (int)first / p.group;
  u.p_hi = u.p0 + ((int)first + rows - 1) / p.group;
  u.own_lo = u.p0 + u.rbase / p.group;
  u.own_hi = u.p0 + (u.rbase + max(u.nrows, 1) - 1) / p.group;
  u.kt = key_tiles(u.p_lo, u.p_hi, p.window, p.sinks);
  u.direct = p.splits == 1 || u.kt.n <= p.per_split;
  u.begin = split * p.per_split;
  const int end = u.direct || split == p.splits - 1 ? u.kt.n : min(u.kt.n, u.begin + p.per_split);
  if (u.direct) u.begin = 0;
  u.n = end - u.begin;
  // a block whose keys are one piece, or that sees nothing at all, is the first split's
  u.skip = u.direct ? (split != 0) : (u.n <= 0);
}

template <int DH, int KIND, int CG>
__global__ void __launch_bounds__(Cfg<DH, KIND, CG>::threads, 1)
    attn_tile_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, int* status) {
  using C = Cfg<DH, KIND, CG>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  float* scales = reinterpret_cast<float*>(smem + C::off_scales);  // [slot][key, value][128]
  float* red = reinterpret_cast<float*>(smem + C::off_red);        // [parity][half][128]
  // in a pair the MMA issuer's own are those of CTA 0: full, mended, pfull, qfull
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::off_bar);
  uint64_t* empty = full + C::stages;
  uint64_t* clean = empty + C::stages;  // bf16: the stage's V has landed and is to be mended
  uint64_t* mended = clean + (C::quant ? 0 : C::stages);
  uint64_t* rfull = mended + (C::quant ? 0 : C::stages);
  uint64_t* rempty = rfull + C::raw;
  uint64_t* scfull = rempty + C::raw;
  uint64_t* sfull = scfull + (C::quant ? kSlots : 0);
  uint64_t* pfull = sfull + 3;
  uint64_t* odone = pfull + 3;
  uint64_t* pair = odone + 2;
  uint64_t* qfull = pair + 4;
  uint64_t* pdone = qfull + 1;
  uint64_t* drain = pdone + 1;
  uint64_t* tready = drain + 1;
  static_assert((C::quant ? 2 * C::stages + 2 * C::raw + kSlots : 4 * C::stages) * 8 + 16 * 8 <= 640,
                "barriers exceed their area");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::off_bar + 640);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::off_bar + 644);
  volatile int* odd = reinterpret_cast<volatile int*>(smem + C::off_bar + 648);
  __shared__ Unit unit;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CG == 1 ? 0 : (int)cta_rank();
  if (warp == 0) {
    Unit u;
    find_unit(p, (gridDim.x - 1 - blockIdx.x) / CG, blockIdx.z, rank, lane, u);
    if (lane == 0) unit = u;
  } else if (warp == 1 && lane == 0) {
    for (int s = 0; s < C::stages; ++s) {
      mbar_init(&full[s], C::quant ? 4 * CG : 1);
      mbar_init(&empty[s], 1);
      if (!C::quant) {
        mbar_init(&clean[s], 1);
        mbar_init(&mended[s], 4 * CG);
      }
    }
    for (int s = 0; s < C::raw; ++s) {
      mbar_init(&rfull[s], 1);
      mbar_init(&rempty[s], 4);
    }
    for (int s = 0; s < (C::quant ? kSlots : 0); ++s) mbar_init(&scfull[s], 1);
    for (int s = 0; s < 3; ++s) {
      mbar_init(&sfull[s], 1);
      mbar_init(&pfull[s], 8 * CG);
    }
    for (int s = 0; s < 2; ++s) mbar_init(&odone[s], 1);
    for (int s = 0; s < 4; ++s) mbar_init(&pair[s], 2);
    mbar_init(qfull, 15 * CG);
    mbar_init(pdone, 4 * CG);
    mbar_init(drain, 1);
    mbar_init(tready, 1);
    *abort = 0;
    *odd = 0;
    fence_mbar_init();
  }
  if (warp == 2 && (blockIdx.x | blockIdx.y | blockIdx.z) == 0) {
    bool bad = false;  // every sequence's numbers are looked at once, also those that no block finds
    for (int i = lane; i < p.c.n_seqs; i += 32) bad |= !kv_seq(p.c, i).ok;
    if (bad) attn_record(status, FAK_ERR_DEVICE);
  }
  __syncwarp();
  if constexpr (CG == 2)
    cluster_sync();  // both CTAs' barriers stand
  else
    __syncthreads();
  const Unit& u = unit;
  if (u.skip) return;  // (a pair's CTAs agree)
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
  const int n = u.n, g = blockIdx.y;
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
  if (warp != 9) {
    // Q: rows of the block, 64 dims to a 16 KB panel, by all warps but the TMA's; rows past the block's are zeros
    const int w = warp < 9 ? warp : warp - 1;
    constexpr int T = 15 * 32, total = kTileM * DH / 8;
    const int tid = w * 32 + lane;
    constexpr int each = (total + T - 1) / T;
    uint4 x[each];
#pragma unroll
    for (int k = 0; k < each; ++k) {
      const int e = k * T + tid, row = e / (DH / 8), c = e % (DH / 8), r = u.rbase + row;
      x[k] = make_uint4(0, 0, 0, 0);
      if (row < u.nrows)
        x[k] = *reinterpret_cast<const uint4*>(p.q + (int64_t)(u.row0 + r / p.group) * p.q_row +
                                               (int64_t)(g * p.group + r % p.group) * p.q_head + c * 8);
    }
#pragma unroll
    for (int k = 0; k < each; ++k) {
      const int e = k * T + tid, row = e / (DH / 8), c = e % (DH / 8);
      if (e < total)
        *reinterpret_cast<uint4*>(smem + (c >> 3) * kStageBytes + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = x[k];
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) arrive_first<CG>(qfull);
    if (warp == 8) {
      tc_fence_before_sync();
      if (lane == 0) mbar_arrive(tready);
    }
  }
  if (warp <= 8) {
    wait(tready, 0);
    tc_fence_after_sync();
  }
  const uint32_t tmem = warp <= 8 ? *reinterpret_cast<volatile uint32_t*>(tmem_slot) : 0;
  const uint32_t tmem_s = tmem + DH;  // O in columns [0, DH), then the S buffers

  if (warp < 8) {
    // ---------------- softmax
    const int half = warp >> 2, quarter = warp & 3, row = 32 * quarter + lane;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const bool live = 32 * quarter < u.nrows;
    const int r = u.rbase + row, pos = u.p0 + r / p.group;
    float m = -INFINITY, l = 0.0f;
    bool ok = true;
    for (int i = 0; i < n && ok; ++i) {
      const int b = i % C::sbufs;
      const int tile = key_tile(u.kt, u.begin + i), j0 = tile * kTileN + 64 * half;
      if (!(ok = wait(&sfull[b], (i / C::sbufs) & 1))) break;
      if constexpr (C::quant)
        if (!(ok = wait(&scfull[i % kSlots], (i / kSlots) & 1))) break;
      tc_fence_after_sync();
      const uint32_t scol = tmem_s + lanes + (uint32_t)(b * kTileN + 64 * half);
      if (live) {
        uint32_t raw[2][32];
        tmem_ld_cols<32>(scol, raw[0]);
        tmem_ld_cols<32>(scol + 32, raw[1]);
        tmem_wait_ld();
        float t[64];
        const float* ks = scales + (i % kSlots) * 2 * kTileN + 64 * half;
#pragma unroll
        for (int k = 0; k < 64; ++k) {
          t[k] = __uint_as_float(raw[k >> 5][k & 31]);
          if constexpr (C::quant) t[k] *= ks[k];
        }
        if (tile_cut(u.own_lo, u.own_hi, tile, p.window, p.sinks)) {
#pragma unroll
          for (int k = 0; k < 64; ++k)
            if (!sees(pos, j0 + k, p.window, p.sinks)) t[k] = -INFINITY;
        }
        float mx = -INFINITY;
#pragma unroll
        for (int k = 0; k < 64; ++k) mx = fmaxf(mx, t[k]);
        float* mine = red + (i & 1) * 2 * kTileM;
        mine[half * kTileM + row] = mx;
        __syncwarp();
        if (lane == 0) mbar_arrive(&pair[quarter]);
        if (!(ok = wait(&pair[quarter], i & 1))) break;
        mx = fmaxf(mx, mine[(half ^ 1) * kTileM + row]) * p.scale;
        // a new base when the maximum passed it by 8, or is the first one seen
        const bool up = mx > m + 8.0f;
        if (__any_sync(0xffffffffu, up)) {
          const float next = up ? mx : m;
          const float f = up ? exp2_approx(m - next) : 1.0f;
          m = next;
          l *= f;
          if (i > 0) {
            if (!(ok = wait(&odone[(i - 1) & 1], ((i - 1) >> 1) & 1))) break;
            tc_fence_after_sync();
#pragma unroll 1
            for (int c = 0; c < DH / 2; c += 32) {
              uint32_t o[32];
              const uint32_t at = tmem + lanes + (uint32_t)(half * (DH / 2) + c);
              tmem_ld_cols<32>(at, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st32(at, o);
            }
          }
        }
        const float base = m == -INFINITY ? 0.0f : m;
        float sum[2] = {0.0f, 0.0f};
        uint32_t w[32];
#pragma unroll
        for (int k = 0; k < 64; k += 2) {
          const float a = exp2_approx(fmaf(t[k], p.scale, -base));
          const float c = exp2_approx(fmaf(t[k + 1], p.scale, -base));
          sum[0] += a;
          sum[1] += c;
          if constexpr (C::quant) {
            // a weight of zero stays zero, whatever scale stands at its place
            const float va = ks[kTileN + k], vc = ks[kTileN + k + 1];
            w[k / 2] = pack_bf16(a == 0.0f ? 0.0f : a * va, c == 0.0f ? 0.0f : c * vc);
          } else {
            w[k / 2] = pack_bf16(a, c);
          }
        }
        l += sum[0] + sum[1];
        tmem_st32(scol, w);
        tmem_wait_st();
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive_first<CG>(&pfull[b]);
    }
    // ---------------- the row's result
    // (the same barrier's phase before first: three tiles' products may still be under way here, and a
    // phase two back looks like the one that is waited for)
    if (ok && n > 2) ok = wait(&odone[(n - 1) & 1], ((n - 3) >> 1) & 1);
    if (ok && n > 0) ok = wait(&odone[(n - 1) & 1], ((n - 1) >> 1) & 1);
    if (ok) ok = wait(pdone, 0);
    if (CG == 2 && ok) ok = try_wait_cluster(pdone, 0);  // (done: for its acquire of `odd`)
    if (ok && live) {
      tc_fence_after_sync();
      float* mine = red + (n & 1) * 2 * kTileM;
      mine[half * kTileM + row] = l;
      __syncwarp();
      if (lane == 0) mbar_arrive(&pair[quarter]);
      ok = wait(&pair[quarter], n & 1);
      l += mine[(half ^ 1) * kTileM + row];
    }
    if (ok && live) {
      const int64_t grow = u.row0 + r / p.group;
      const int head = g * p.group + r % p.group;
      const bool mine = row < u.nrows;
      const int64_t slot = ((int64_t)blockIdx.z * p.c.rows + grow) * p.nq + head;
      // a row that sees nothing is zeros; one whose scores are all -inf is NaN, as 0 / 0 is
      const float inv = pos < 0 ? 0.0f : 1.0f / l;
      if (!u.direct && mine && half == 0) p.stat[slot] = make_float2(m, l);
#pragma unroll 1
      for (int c = 0; c < DH / 2; c += 32) {
        const int d0 = half * (DH / 2) + c;
        uint32_t o[32];
        if (n > 0) {
          tmem_ld_cols<32>(tmem + lanes + (uint32_t)d0, o);
          tmem_wait_ld();
        }
        if (pos < 0 || n == 0) {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0;
        }
        if (!C::quant && mine && *odd) {
          // values that are not finite, in tiles where they were left out: added for the rows that see them
          for (int i = 0; i < n; ++i) {
            const int tile = key_tile(u.kt, u.begin + i);
            if (!tile_cut(u.p_lo, u.p_hi, tile, p.window, p.sinks)) continue;
            for (int j = tile * kTileN; j < min((tile + 1) * kTileN, pos + 1); ++j) {
              if (!sees(pos, j, p.window, p.sinks)) continue;
              int64_t at = kv_place(p.c, u.seq, j, g);
              if (at < 0) at = -1 - at;
              const uint16_t* v = reinterpret_cast<const uint16_t*>(p.c.v) + at * DH + d0;
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if ((v[k] & 0x7F80u) == 0x7F80u)
                  o[k] = __float_as_uint(__uint_as_float(o[k]) + __uint_as_float((uint32_t)v[k] << 16));
            }
          }
        }
        if (mine && !u.direct) {
          float4* dst = reinterpret_cast<float4*>(p.part + slot * DH + d0);
#pragma unroll
          for (int k = 0; k < 32; k += 4)
            dst[k / 4] = make_float4(__uint_as_float(o[k]), __uint_as_float(o[k + 1]), __uint_as_float(o[k + 2]),
                                     __uint_as_float(o[k + 3]));
        } else if (mine) {
        float y[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) y[k] = __uint_as_float(o[k]) * inv;
        if (p.gate && pos >= 0) {
          const float4* gp = reinterpret_cast<const float4*>(p.gate + grow * p.gate_row + head * p.gate_head + d0);
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            const float4 x = gp[k / 4];
            y[k] /= 1.0f + __expf(-x.x);
            y[k + 1] /= 1.0f + __expf(-x.y);
            y[k + 2] /= 1.0f + __expf(-x.z);
            y[k + 3] /= 1.0f + __expf(-x.w);
          }
        }
        uint4* dst = reinterpret_cast<uint4*>(p.out + grow * p.out_row + head * p.out_head + d0);
#pragma unroll
        for (int k = 0; k < 32; k += 8)
          dst[k / 8] = make_uint4(pack_bf16(y[k], y[k + 1]), pack_bf16(y[k + 2], y[k + 3]),
                                  pack_bf16(y[k + 4], y[k + 5]), pack_bf16(y[k + 6], y[k + 7]));
        }
        __syncwarp();
      }
    }
  } else if (warp == 8) {
    // ---------------- MMA issuer
    if (n > 0 && rank == 0) {
      // K: one CTA takes a tile as twice 64 keys, since its panels are 64 keys high; a pair holds 64 keys each
      constexpr uint32_t id_s = kIdescAttn<kTileM * CG, 64 * CG, false>, id_o = kIdescAttn<kTileM * CG, DH, true>;
      const uint64_t kd0 = umma_desc_sw128(smem_u32(smem + C::off_ring)), qd = umma_desc_sw128(smem_u32(smem));
      // a stage's V: panels of 64 dims by vrows keys, all dims of the first keys, then of the next
      const int vshift = C::quant ? 31 - __clz(C::vkeys) : min(p.c.page_shift, 31 - __clz(C::vkeys));
      const uint64_t vd0 = desc_mn(smem_u32(smem + C::off_ring), 128u << vshift);
      // a stage that is mended has a barrier of its own, so the parities of both go by their uses
      int st = 0;
      uint32_t fulls = 0, mends = 0;
      bool ok = wait(qfull, 0);
      auto take = [&](bool mend) {  // the next stage, once it is full
        ok = ok && wait(mend ? &mended[st] : &full[st], ((mend ? mends : fulls) >> st) & 1);
        (mend ? mends : fulls) ^= 1u << st;
        tc_fence_after_sync();
        return ok;
      };
      auto scores = [&](int sb) {
        const uint32_t d = tmem_s + (uint32_t)(sb * kTileN);
#pragma unroll
        for (int c = 0; c < C::chunks; ++c) {
          if (!take(false)) return;
          const uint64_t kd = kd0 + (uint64_t)(st * (kStageBytes >> 4));
          if (elect_one()) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {  // the stage's halves: 64 dims of 64 keys
              constexpr int per = DH / 128;  // stages of 64 keys
              const int half = CG == 2 ? 0 : DH == 64 ? x : c / (per ? per : 1);
              const int panel = DH == 64 ? 0 : (CG == 2 ? c : c % (per ? per : 1)) * 2 + x;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_ss<CG>(d + 64 * half, qd + (uint64_t)((panel * kStageBytes + 32 * k) >> 4),
                           kd + (uint64_t)((x * 8192 + 32 * k) >> 4), id_s, panel | k);
            }
            commit<CG>(&empty[st]);
            if (c == C::chunks - 1) commit<CG>(&sfull[sb]);
          }
          __syncwarp();
          st = st + 1 == C::stages ? 0 : st + 1;
        }
      };
      for (int i = 0; i < min(C::sbufs, n) && ok; ++i) scores(i);
      int sb = 0, ph = 0;
      for (int i = 0; i < n && ok; ++i) {
        const bool mend = !C::quant && tile_cut(u.p_lo, u.p_hi, key_tile(u.kt, u.begin + i), p.window, p.sinks);
        if (!(ok = wait(&pfull[sb], ph))) break;
        const uint32_t a = tmem_s + (uint32_t)(sb * kTileN);
#pragma unroll
        for (int c = 0; c < C::chunks; ++c) {
          if (!take(mend)) break;
          const uint64_t vd = vd0 + (uint64_t)(st * (kStageBytes >> 4));
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < C::vkeys / 16; ++k) {
              const int key = c * C::vkeys + 16 * k;  // weights: 64 keys in 32 columns, twice
              const int box = 16 * k >> vshift, in = 16 * k & ((1 << vshift) - 1);
              mma_ts<CG>(tmem, a + (uint32_t)((key >> 6) * 64 + (key & 63) / 2),
                         vd + (uint64_t)(((box << vshift) * (C::dv * 2) + in * 128) >> 4), id_o, (i | key) != 0);
            }
            commit<CG>(&empty[st]);
            if (c == C::chunks - 1) commit<CG>(&odone[i & 1]);
          }
          __syncwarp();
          st = st + 1 == C::stages ? 0 : st + 1;
        }
        if (ok && i + C::sbufs < n) scores(sb);
        if (++sb == C::sbufs) {
          sb = 0;
          ph ^= 1;
        }
      }
      if (!ok && elect_one()) {
        // what was issued completes before TMEM is freed
        commit<CG>(drain);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(drain, 0))
          if (globaltimer_ns() - t0 > 200000000ull) break;
      }
      __syncwarp();
    }
  } else if (warp == 9) {
    // ---------------- TMA
    const int kshift = min(p.c.page_shift, 6), krows = 1 << kshift;  // the maps' boxes: keys of K, of V
    const int vshift = min(p.c.page_shift, 31 - __clz(C::vkeys)), vrows = 1 << vshift;
    const int kpanels = krows == 64 ? C::panels : 1;  // and panels of K, which stand 64 keys apart
    const int boxes = kTileN >> kshift;
    constexpr int S = C::quant ? C::raw : C::stages;
    constexpr int kw = C::panels * 64;  // 8-bit: bytes of a K stage's row
    uint64_t* const free = C::quant ? rempty : empty;
    int st = 0, ph = 1, sc = 0;  // the stage, the parity of its `free` (the first round is free already)
    uint32_t fulls = 0xffffffffu, lands = 0xffffffffu;  // the parity of each stage's last use of `full`, of `clean`
    bool ok = true;
    // lane l: the vector index of key l * krows of the tile; keys past the last that a row sees take its
    // page: what lies there is masked
    auto places = [&](int i) {
      const int j = min(key_tile(u.kt, u.begin + i) * kTileN + (min(lane, boxes - 1) << kshift), u.p_hi & ~(krows - 1));
      int64_t at = kv_place(p.c, u.seq, j, g);
      if (at < 0) {
        attn_record(status, FAK_ERR_DEVICE);
        at = -1 - at;
      }
      return (int)at;
    };
    int ahead = n > 0 ? places(0) : 0;  // the next tile's, looked up early
    int held[4];                        // those of the tiles whose V is still to come
    auto next = [&]() {
      if (++st == S) {
        st = 0;
        ph ^= 1;
      }
    };
    // the next stage, once it is free; its bytes count on CTA 0's barrier, but for V that is to be mended
    auto stage = [&](bool mend, uint64_t*& bar, uint8_t*& dst) {
      if (!(ok = ok && wait(&free[st], ph))) return false;
      bar = C::quant ? &rfull[st] : mend ? &clean[st] : &full[st];
      dst = smem + (C::quant ? C::off_raw + st * kRawBytes : C::off_ring + st * kStageBytes);
      const bool local = C::quant || mend;
      if ((local || rank == 0) && elect_one())
        mbar_arrive_expect_tx(bar, C::quant ? kRawBytes : local ? kStageBytes : kStageBytes * CG);
      __syncwarp();
      (mend ? lands : fulls) ^= 1u << st;
      return true;
    };
    auto keys = [&](int i, int at) {
      if constexpr (C::quant) {
        const int slot = i % kSlots;
        float* to = scales + slot * 2 * kTileN;
        if (elect_one()) mbar_arrive_expect_tx(&scfull[slot], 2 * kTileN * 4);
        __syncwarp();
        if (lane < boxes) {
          bulk_g2s_nohint(to + lane * krows, p.c.ks + at, krows * 4, &scfull[slot]);
          bulk_g2s_nohint(to + kTileN + lane * krows, p.c.vs + at, krows * 4, &scfull[slot]);
        }
        __syncwarp();
        ++sc;
      }
      uint64_t* bar;
      uint8_t* dst;
#pragma unroll
      for (int c = 0; c < C::chunks; ++c) {
        if (!stage(false, bar, dst)) return;
        constexpr int per = DH / 128;  // stages of 64 keys
        const int half = CG == 2 ? rank : c / (per ? per : 1);  // dh 64: the stage has both halves
        const int panel = (CG == 2 ? c : c % (per ? per : 1)) * 2;
        for (int k = 0; k < (DH == 64 ? kTileN : 64); k += krows) {
          const int row = __shfl_sync(0xffffffffu, at, (half * 64 + k) >> kshift);
          if constexpr (C::quant) {
            if (elect_one()) tma_load_2d_tx(dst + k * kw, &kmap, panel * 64, row, bar);
          } else {
            for (int x = 0; x < C::panels; x += kpanels)
              if (elect_one()) load_3d<CG>(dst + x * 8192 + k * 128, &kmap, 0, row, panel + x, bar, false);
          }
          __syncwarp();
        }
        next();
      }
    };
    auto values = [&](int i, int at) {
      const bool mend = !C::quant && tile_cut(u.p_lo, u.p_hi, key_tile(u.kt, u.begin + i), p.window, p.sinks);
      uint64_t* bar;
      uint8_t* dst;
#pragma unroll
      for (int c = 0; c < C::chunks; ++c) {
        if (!stage(mend, bar, dst)) return;
        for (int r = 0; r < C::vkeys; r += vrows) {
          const int key = c * C::vkeys + r, row = __shfl_sync(0xffffffffu, at, key >> kshift) + (key & (krows - 1));
          if (elect_one()) {
            if constexpr (C::quant)
              tma_load_2d_tx(dst + r * C::dv, &vmap, rank * C::dv, row, bar);
            else
              load_3d<CG>(dst + r * C::dv * 2, &vmap, 0, row, rank * C::chunks, bar, mend);
          }
          __syncwarp();
        }
        next();
      }
    };
    auto step = [&](int i) {  // K of tile i, its places kept for V
#pragma unroll
      for (int k = 3; k > 0; --k) held[k] = held[k - 1];
      held[0] = ahead;
      if (i + 1 < n) ahead = places(i + 1);
      keys(i, held[0]);
    };
    // V i follows K i + sbufs - 1 (or the last K): its places were kept that many tiles ago
    const int lead = min(C::sbufs, n);
    for (int i = 0; i < lead && ok; ++i) step(i);
    for (int i = 0; i < n && ok; ++i) {
      const int back = min(lead, n - i) - 1;
      values(i, back == 2 ? held[2] : back == 1 ? held[1] : held[0]);
      if (ok && i + C::sbufs < n) step(i + C::sbufs);
    }
    // copies in flight land before the block can end (one that ran to its end has used every copy)
    if (lane == 0 && *abort) {
      auto landed = [&](uint64_t* bar, uint32_t parity) {
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(bar, parity & 1))
          if (globaltimer_ns() - t0 > 200000000ull) break;
      };
      for (int q = 0; q < S; ++q) {
        landed(C::quant ? &rfull[q] : &full[q], fulls >> q);
        if (!C::quant) landed(&clean[q], lands >> q);
      }
      for (int q = max(0, sc - kSlots); q < sc; ++q) landed(&scfull[q % kSlots], q / kSlots);
    }
    __syncwarp();
  } else if (warp >= 12) {
    // ---------------- codes to bf16, V of cut tiles
    constexpr int T = 128;
    const int tid = threadIdx.x - 12 * 32;
    bool ok = true;
    if constexpr (C::quant) {
      int rs = 0, rph = 0, st = 0, ph = 1;
      auto convert = [&](bool value) {
        // 16 codes to a thread and step
        constexpr int kwidth = C::panels * 4, vwidth = C::dv / 16;
        for (int c = 0; c < C::chunks; ++c) {
          ok = ok && wait(&rfull[rs], rph) && wait(&empty[st], ph);
          if (!ok) return;
          const uint4* src = reinterpret_cast<const uint4*>(smem + C::off_raw + rs * kRawBytes);
          uint8_t* dst = smem + C::off_ring + st * kStageBytes;
          uint4 q[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) q[k] = src[tid + k * T];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int e = tid + k * T;
            const int key = value ? e / vwidth : e / kwidth, d = (value ? e % vwidth : e % kwidth) * 16;
            uint4 a, b;
            codes_to_bf16<KIND>(q[k].x, a.x, a.y);
            codes_to_bf16<KIND>(q[k].y, a.z, a.w);
            codes_to_bf16<KIND>(q[k].z, b.x, b.y);
            codes_to_bf16<KIND>(q[k].w, b.z, b.w);
            uint8_t* line = dst + (d >> 6) * (value ? C::vkeys * 128 : 8192) + key * 128;
            const int e16 = (d & 63) >> 3;
            *reinterpret_cast<uint4*>(line + ((e16 ^ (key & 7)) << 4)) = a;
            *reinterpret_cast<uint4*>(line + (((e16 + 1) ^ (key & 7)) << 4)) = b;
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            arrive_first<CG>(&full[st]);
            mbar_arrive(&rempty[rs]);  // after the stores, which came after the loads
          }
          if (++rs == C::raw) {
            rs = 0;
            rph ^= 1;
          }
          if (++st == C::stages) {
            st = 0;
            ph ^= 1;
          }
        }
      };
      for (int i = 0; i < min(C::sbufs, n) && ok; ++i) convert(false);
      for (int i = 0; i < n && ok; ++i) {
        convert(true);
        if (ok && i + C::sbufs < n) convert(false);
      }
    } else {
      uint32_t landed = 0;  // parity of each stage's next use of `clean`
      const int vshift = min(p.c.page_shift, 31 - __clz(C::vkeys));
      for (int i = 0; i < n && ok; ++i) {
        const int tile = key_tile(u.kt, u.begin + i);
        if (!tile_cut(u.p_lo, u.p_hi, tile, p.window, p.sinks)) continue;
        int it = (i + min(C::sbufs + i, n)) * C::chunks;  // V i comes after that many tiles
        for (int c = 0; c < C::chunks && ok; ++c, ++it) {
          const int st = it % C::stages;
          if (!(ok = wait(&clean[st], (landed >> st) & 1))) break;
          landed ^= 1u << st;
          uint4* v = reinterpret_cast<uint4*>(smem + C::off_ring + st * kStageBytes);
          bool bad = false;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int e = tid + k * T, box = e / (C::dv / 8) >> vshift;  // a box: dv dims of 2^vshift keys
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
            *odd = 1;
            if constexpr (CG == 2)  // the other CTA's rows have these dims too
              asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_to((const void*)odd, rank ^ 1)), "r"(1)
                           : "memory");
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) arrive_first<CG>(&mended[st]);
        }
      }
    }
    __syncwarp();
    if (lane == 0) {
      if constexpr (CG == 1) {
        mbar_arrive(pdone);
      } else {
        arrive_release_cluster(pdone, 0);
        arrive_release_cluster(pdone, 1);
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

template <int DH, int KIND, int CG>
cudaError_t launch(const AttnParams& p, int page, int64_t n_vec, int64_t blocks, int* status, cudaStream_t s) {
  using C = Cfg<DH, KIND, CG>;
  cudaError_t e = encoder();
  if (e != cudaSuccess) return e;
  CUtensorMap kmap, vmap;
  const int krows = std::min(page, 64), vrows = std::min(page, C::vkeys);
  if (!code_map(&kmap, p.c.k, C::quant, DH, n_vec, C::quant ? C::panels * 64 : 64, krows, krows == 64 ? C::panels : 1) ||
      !code_map(&vmap, p.c.v, C::quant, DH, n_vec, C::quant ? C::dv : 64, vrows, C::chunks))
    return cudaErrorInvalidValue;
  e = cudaFuncSetAttribute(attn_tile_kernel<DH, KIND, CG>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem);
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
  return cudaLaunchKernelEx(&cfg, attn_tile_kernel<DH, KIND, CG>, p, kmap, vmap, status);
}

template <int DH, int CG>
cudaError_t by_kind(int kind, const AttnParams& p, int page, int64_t n_vec, int64_t blocks, int* status,
                    cudaStream_t s) {
  return kind == FAK_KV_BF16   ? launch<DH, FAK_KV_BF16, CG>(p, page, n_vec, blocks, status, s)
         : kind == FAK_KV_E4M3 ? launch<DH, FAK_KV_E4M3, CG>(p, page, n_vec, blocks, status, s)
                               : launch<DH, FAK_KV_I8, CG>(p, page, n_vec, blocks, status, s);
}

}  // namespace

cudaError_t attn_tile_launch(int kind, int dh, int page, int64_t n_vec, const AttnParams& p, int64_t blocks,
                             int* status, cudaStream_t s) {
  if (p.block == 2 * kTileM)
    return dh == 128 ? by_kind<128, 2>(kind, p, page, n_vec, blocks, status, s)
                     : by_kind<256, 2>(kind, p, page, n_vec, blocks, status, s);
  return dh == 64    ? by_kind<64, 1>(kind, p, page, n_vec, blocks, status, s)
         : dh == 128 ? by_kind<128, 1>(kind, p, page, n_vec, blocks, status, s)
                     : by_kind<256, 1>(kind, p, page, n_vec, blocks, status, s);
}
