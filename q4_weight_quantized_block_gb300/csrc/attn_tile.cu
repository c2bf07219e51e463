// Attention of blocks of rows over the paged KV cache on the 5th-generation tensor cores.
//
// A block holds 128 rows of one sequence and KV head; a row is a (token, query head of the group) pair, so
// grouped heads fill the block whether the sequence has one new token or thousands.  Per tile of 128 keys
//   S = Q K^T (f32 in TMEM),  P = exp2(c S - m) (bf16, in S's own TMEM columns),  O += P V (f32 in TMEM)
// with the running maximum m and sum of the softmax.  m moves only when a row's maximum passes it by 8: until then
// weights reach at most 2^8, which bf16 and f32 hold as well as 1, and O is not rescaled.
//
//   warps 0-7      softmax: warp w and w + 4 share rows 32 (w % 4) .. +31, half of the keys each
//   warp 8         MMA issuer and TMEM owner
//   warp 9         TMA: K and V by pages in 16 KB stages of a ring, in the order the MMAs take them
//                  (K 0, K 1, V 0, K 2, V 1, ...), in the 128-byte-swizzled layouts the MMAs read: Q and K
//                  64 dims wide with the dims running (K-major), V keys by dims as stored (MN-major)
//   warps 10-13    Q's rows; then, for an 8-bit cache, codes to bf16: the copies land in a ring of their own and
//                  these warps fill the MMAs' ring from it; for a bf16 cache, V of the tiles that a mask cuts
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

template <int DH, int KIND>
struct Cfg {
  static constexpr bool quant = KIND != FAK_KV_BF16;
  static constexpr int chunks = DH / 64;             // stages of one tile of K or of V
  static constexpr int vkeys = 8192 / DH;            // keys of one V stage
  static constexpr int sbufs = DH == 256 ? 2 : 3;    // S buffers: 512 TMEM columns, less O's
  static constexpr int stages = quant ? (DH == 256 ? 6 : 8) : DH == 256 ? 9 : DH == 128 ? 11 : 12;
  static constexpr int raw = !quant ? 0 : DH == 64 ? 6 : 5;  // stages of codes on their way to bf16
  static constexpr int threads = 14 * 32;
  static constexpr int off_ring = kTileM * DH * 2;
  static constexpr int off_raw = off_ring + stages * kStageBytes;
  static constexpr int off_scales = off_raw + raw * kRawBytes;
  static constexpr int off_red = off_scales + (quant ? kSlots * 2 * kTileN * 4 : 0);
  static constexpr int off_bar = off_red + 2 * 2 * kTileM * 4;
  static constexpr int smem = off_bar + 640 + 1024;
  static_assert(smem <= 232448 - 1024, "shared memory exceeds the 227 KB per-block limit");
};

struct Unit {
  int seq, row0, rbase, nrows, p0, p_lo, p_hi, n, begin, direct, skip;
  KeyTiles kt;
};

// kind::f16 descriptors: f32 accumulator, bf16 operands, M 128; the second has B running along N
template <int N, bool B_MN>
constexpr uint32_t kIdescAttn = (1u << 4) | (1u << 7) | (1u << 10) | ((B_MN ? 1u : 0u) << 16) |
                                ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kTileM >> 4) << 24);

FAK_DEV void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc)
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

FAK_DEV bool sees(int pos, int j, int window, int sinks) {
  return j <= pos && (!window || j > pos - window || j < sinks);
}

// Whether some row of the block does not see some key of the tile.
FAK_DEV bool tile_cut(const Unit& u, int tile, int window, int sinks) {
  const int j0 = tile * kTileN, j1 = j0 + kTileN - 1;
  return !(j1 <= u.p_lo && (!window || j0 > u.p_hi - window || j1 < sinks));
}

// Block x's sequence: the one of the last s with r0(s) * group / 128 + s <= x.  These starts rise by at
// least the sequence's number of blocks, so every block of rows has an x, and some x have none.
FAK_DEV void find_unit(const AttnParams& p, int64_t x, int split, int lane, Unit& u) {
  int lo = 0, hi = p.c.n_seqs;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, i = lo + lane * step;
    const unsigned b =
        __ballot_sync(0xffffffffu, i < hi && (int64_t)p.c.row_start[i] * p.group / kTileM + i <= x);
    const int n = __popc(b);
    if (n > 1) lo += (n - 1) * step;
    hi = min(lo + step, hi);
  }
  const KvSeq sq = kv_seq(p.c, lo);
  u.seq = lo;
  u.skip = 1;
  if (!sq.ok) return;
  const int64_t mt = x - ((int64_t)sq.r0 * p.group / kTileM + lo);
  const int64_t total = (int64_t)(sq.r1 - sq.r0) * p.group;
  if (mt < 0 || mt * kTileM >= total) return;
  u.row0 = sq.r0;
  u.rbase = (int)(mt * kTileM);
  u.nrows = (int)min((int64_t)kTileM, total - u.rbase);
  u.p0 = sq.len - (sq.r1 - sq.r0);
  u.p_lo = u.p0 + u.rbase / p.group;
  u.p_hi = u.p0 + (u.rbase + u.nrows - 1) / p.group;
  u.kt = key_tiles(u.p_lo, u.p_hi, p.window, p.sinks);
  u.direct = p.splits == 1 || u.kt.n <= p.per_split;
  u.begin = split * p.per_split;
  const int end = u.direct || split == p.splits - 1 ? u.kt.n : min(u.kt.n, u.begin + p.per_split);
  if (u.direct) u.begin = 0;
  u.n = end - u.begin;
  // a block whose keys are one piece, or that sees nothing at all, is the first split's
  u.skip = u.direct ? (split != 0) : (u.n <= 0);
}

template <int DH, int KIND>
__global__ void __launch_bounds__(Cfg<DH, KIND>::threads, 1)
    attn_tile_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, int* status) {
  using C = Cfg<DH, KIND>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* scales = reinterpret_cast<float*>(smem + C::off_scales);  // [slot][key, value][128]
  float* red = reinterpret_cast<float*>(smem + C::off_red);        // [parity][half][128]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::off_bar);
  uint64_t* empty = full + C::stages;
  uint64_t* clean = empty + C::stages;  // bf16: the stage's V has landed and is to be mended
  uint64_t* rfull = clean + (C::quant ? 0 : C::stages);
  uint64_t* rempty = rfull + C::raw;
  uint64_t* scfull = rempty + C::raw;
  uint64_t* sfull = scfull + (C::quant ? kSlots : 0);
  uint64_t* pfull = sfull + 3;
  uint64_t* odone = pfull + 3;
  uint64_t* pair = odone + 2;
  uint64_t* qfull = pair + 4;
  uint64_t* pdone = qfull + 1;
  uint64_t* drain = pdone + 1;
  static_assert((3 * C::stages + 2 * C::raw + kSlots + 3 + 3 + 2 + 4 + 3) * 8 <= 624, "barriers exceed their area");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::off_bar + 624);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::off_bar + 628);
  volatile int* odd = reinterpret_cast<volatile int*>(smem + C::off_bar + 632);
  __shared__ Unit unit;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    Unit u;
    find_unit(p, gridDim.x - 1 - (int64_t)blockIdx.x, blockIdx.z, lane, u);
    if (lane == 0) unit = u;
  } else if (warp == 1 && lane == 0) {
    for (int s = 0; s < C::stages; ++s) {
      mbar_init(&full[s], 4);
      mbar_init(&empty[s], 1);
      if (!C::quant) mbar_init(&clean[s], 1);
    }
    for (int s = 0; s < C::raw; ++s) {
      mbar_init(&rfull[s], 1);
      mbar_init(&rempty[s], 4);
    }
    for (int s = 0; s < (C::quant ? kSlots : 0); ++s) mbar_init(&scfull[s], 1);
    for (int s = 0; s < 3; ++s) {
      mbar_init(&sfull[s], 1);
      mbar_init(&pfull[s], 8);
    }
    for (int s = 0; s < 2; ++s) mbar_init(&odone[s], 1);
    for (int s = 0; s < 4; ++s) mbar_init(&pair[s], 2);
    mbar_init(qfull, 4);
    mbar_init(pdone, 4);
    mbar_init(drain, 1);
    *abort = 0;
    *odd = 0;
    fence_mbar_init();
  }
  if (warp == 2 && (blockIdx.x | blockIdx.y | blockIdx.z) == 0) {
    bool bad = false;  // every sequence's numbers are looked at once, also those that no block finds
    for (int i = lane; i < p.c.n_seqs; i += 32) bad |= !kv_seq(p.c, i).ok;
    if (bad) attn_record(status, FAK_ERR_DEVICE);
  }
  __syncthreads();
  const Unit& u = unit;
  if (u.skip) {
    return;
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tmem_s = tmem + DH;  // O in columns [0, DH), then the S buffers
  const int n = u.n, g = blockIdx.y;
  const uint64_t tmo = p.timeout_ns;
  auto wait_one = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_wait_bounded(bar, parity, abort, tmo)) return true;
    if (!*abort) attn_record(status, FAK_ERR_TIMEOUT);
    *abort = 1;
    return false;
  };
  // a whole warp waits: it goes on or gives up as one
  auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait_one(bar, parity)); };

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
        if (tile_cut(u, tile, p.window, p.sinks)) {
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
      if (lane == 0) mbar_arrive(&pfull[b]);
    }
    // ---------------- the row's result
    // (the same barrier's phase before first: three tiles' products may still be under way here, and a
    // phase two back looks like the one that is waited for)
    if (ok && n > 2) ok = wait(&odone[(n - 1) & 1], ((n - 3) >> 1) & 1);
    if (ok && n > 0) ok = wait(&odone[(n - 1) & 1], ((n - 1) >> 1) & 1);
    if (ok) ok = wait(pdone, 0);
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
            if (!tile_cut(u, tile, p.window, p.sinks)) continue;
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
    if (lane == 0 && n > 0) {
      constexpr uint32_t id_s = kIdescAttn<kTileN, false>, id_o = kIdescAttn<DH, true>;
      const uint32_t ring = smem_u32(smem + C::off_ring);
      const uint64_t qdesc = umma_desc_sw128(smem_u32(smem));
      int it = 0;
      bool ok = wait_one(qfull, 0);
      auto take = [&]() {  // the next stage, once it is full
        ok = ok && wait_one(&full[it % C::stages], (it / C::stages) & 1);
        tc_fence_after_sync();
        return ok;
      };
      auto scores = [&](int i) {
        const uint32_t d = tmem_s + (uint32_t)((i % C::sbufs) * kTileN);
        for (int c = 0; c < C::chunks; ++c, ++it) {
          if (!take()) return;
          const uint64_t kd = umma_desc_sw128(ring + (it % C::stages) * kStageBytes);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ss(d, qdesc + (uint64_t)((c * kStageBytes + 32 * k) >> 4), kd + (uint64_t)(2 * k), id_s, c | k);
          umma_commit(&empty[it % C::stages]);
        }
        umma_commit(&sfull[i % C::sbufs]);
      };
      for (int i = 0; i < min(C::sbufs, n) && ok; ++i) scores(i);
      for (int i = 0; i < n && ok; ++i) {
        if (!(ok = wait_one(&pfull[i % C::sbufs], (i / C::sbufs) & 1))) break;
        const uint32_t a = tmem_s + (uint32_t)((i % C::sbufs) * kTileN);
        for (int c = 0; c < C::chunks; ++c, ++it) {
          if (!take()) break;
          const uint64_t vd = desc_mn(ring + (it % C::stages) * kStageBytes, C::vkeys * 128);
#pragma unroll
          for (int k = 0; k < C::vkeys / 16; ++k) {
            const int key = c * C::vkeys + 16 * k;  // weights: 64 keys in 32 columns, twice
            umma_f16_ts(tmem, a + (uint32_t)((key >> 6) * 64 + (key & 63) / 2), vd + (uint64_t)(k * 2048 >> 4), id_o,
                        (i | key) != 0);
          }
          umma_commit(&empty[it % C::stages]);
        }
        if (!ok) break;
        umma_commit(&odone[i & 1]);
        if (i + C::sbufs < n) scores(i + C::sbufs);
      }
      if (!ok) {
        // what was issued completes before TMEM is freed
        umma_commit(drain);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(drain, 0))
          if (globaltimer_ns() - t0 > 200000000ull) break;
      }
    }
  } else if (warp == 9) {
    // ---------------- TMA: every lane waits; the lanes share a stage's boxes
    const int page = 1 << p.c.page_shift;
    const int krows = min(page, kTileN), vrows = min(page, C::vkeys);  // the maps' boxes
    const int kboxes = kTileN / krows, vsub = C::vkeys / vrows;
    int it = 0, sc = 0;
    bool ok = true;
    // the vector index of key j0 + lane * krows, at the tile's start; keys past the last that a row sees
    // take its page: what lies there is masked
    auto places = [&](int i) {
      const int j = min(key_tile(u.kt, u.begin + i) * kTileN + min(lane, kboxes - 1) * krows, u.p_hi & ~(krows - 1));
      int64_t at = kv_place(p.c, u.seq, j, g);
      if (at < 0) {
        attn_record(status, FAK_ERR_DEVICE);
        at = -1 - at;
      }
      return (int)at;
    };
    auto stage = [&](uint8_t*& dst, uint64_t*& bar, bool mend) {  // the next stage, once it is free
      constexpr int S = C::quant ? C::raw : C::stages;
      uint64_t* free = C::quant ? rempty : empty;
      const int st = it % S;
      if (it >= S) ok = ok && wait(&free[st], ((it / S) - 1) & 1);
      dst = smem + (C::quant ? C::off_raw + st * kRawBytes : C::off_ring + st * kStageBytes);
      bar = C::quant ? &rfull[st] : mend ? &clean[st] : &full[st];
      if (ok && lane == 0) mbar_arrive_expect_tx(bar, C::quant ? kRawBytes : kStageBytes);
      if (ok && !C::quant && !mend && lane > 0 && lane < 4) mbar_arrive(bar);  // in place of four mending warps
      __syncwarp();
    };
    constexpr int kw = C::quant ? 64 : 128;  // bytes of a K stage's row
    auto keys = [&](int i, int at) {
      uint8_t* dst;
      uint64_t* bar;
      if constexpr (C::quant) {
        const int slot = i % kSlots;
        float* to = scales + slot * 2 * kTileN + lane * krows;
        if (lane == 0) mbar_arrive_expect_tx(&scfull[slot], 2 * kTileN * 4);
        __syncwarp();
        if (lane < kboxes) {
          bulk_g2s_nohint(to, p.c.ks + at, krows * 4, &scfull[slot]);
          bulk_g2s_nohint(to + kTileN, p.c.vs + at, krows * 4, &scfull[slot]);
        }
        ++sc;
      }
      for (int c = 0; c < C::chunks && ok; ++c, ++it) {
        stage(dst, bar, false);
        if (!ok) return;
        if (lane < kboxes) tma_load_2d_tx(dst + lane * krows * kw, &kmap, c * 64, at, bar);
      }
    };
    auto values = [&](int i, int at) {
      const bool mend = !C::quant && tile_cut(u, key_tile(u.kt, u.begin + i), p.window, p.sinks);
      uint8_t* dst;
      uint64_t* bar;
      for (int c = 0; c < C::chunks && ok; ++c, ++it) {
        stage(dst, bar, mend);
        if (!ok) return;
        // box (d, r): 64 dims (bf16) or all (codes), keys c * vkeys + r * vrows .. + vrows - 1
        const int r = lane % vsub, d = lane / vsub, key = c * C::vkeys + r * vrows;
        const int row = __shfl_sync(0xffffffffu, at, key / krows) + (key & (krows - 1));
        if (C::quant) {
          if (d == 0) tma_load_2d_tx(dst + r * vrows * DH, &vmap, 0, row, bar);
        } else if (d < DH / 64) {
          tma_load_2d_tx(dst + d * C::vkeys * 128 + r * vrows * 128, &vmap, d * 64, row, bar);
        }
      }
    };
    // the places of a tile's keys stay in a register of each lane until its values are loaded
    int at[4];
    int ahead = n > 0 ? places(0) : 0;  // the next tile's, loaded early
    auto next_keys = [&](int i) {
      at[i & 3] = ahead;
      if (i + 1 < n) ahead = places(i + 1);
      keys(i, i & 2 ? (i & 1 ? at[3] : at[2]) : (i & 1 ? at[1] : at[0]));
    };
    for (int i = 0; i < min(C::sbufs, n) && ok; ++i) next_keys(i);
    for (int i = 0; i < n && ok; ++i) {
      values(i, i & 2 ? (i & 1 ? at[3] : at[2]) : (i & 1 ? at[1] : at[0]));
      if (ok && i + C::sbufs < n) next_keys(i + C::sbufs);
    }
    // copies in flight land before the block can end
    constexpr int S = C::quant ? C::raw : C::stages;
    for (int q = max(0, it - S); q < it; ++q) {
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(C::quant ? &rfull[q % S] : &full[q % S], (q / S) & 1))
        if (globaltimer_ns() - t0 > 200000000ull) break;
    }
    for (int q = max(0, sc - kSlots); q < sc; ++q) {
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(&scfull[q % kSlots], (q / kSlots) & 1))
        if (globaltimer_ns() - t0 > 200000000ull) break;
    }
  } else {
    // ---------------- Q, codes to bf16, V of cut tiles
    constexpr int T = 128;
    const int tid = threadIdx.x - 10 * 32;
    bool ok = true;
    // Q: rows of the block, 64 dims to a 16 KB panel; rows past the block's are zeros
    for (int k = tid; k < kTileM * DH / 8; k += T) {
      const int row = k / (DH / 8), c = k % (DH / 8);
      uint4 x = make_uint4(0, 0, 0, 0);
      if (row < u.nrows) {
        const int r = u.rbase + row;
        x = *reinterpret_cast<const uint4*>(p.q + (int64_t)(u.row0 + r / p.group) * p.q_row +
                                            (int64_t)(g * p.group + r % p.group) * p.q_head + c * 8);
      }
      *reinterpret_cast<uint4*>(smem + (c >> 3) * kStageBytes + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = x;
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) mbar_arrive(qfull);
    if constexpr (C::quant) {
      int it = 0;
      auto convert = [&](bool value) {
        const int width = value ? DH / 16 : 4;  // 16 codes to a thread and step
        for (int c = 0; c < C::chunks; ++c, ++it) {
          const int rs = it % C::raw, st = it % C::stages;
          ok = ok && wait(&rfull[rs], (it / C::raw) & 1);
          if (ok && it >= C::stages) ok = wait(&empty[st], ((it / C::stages) - 1) & 1);
          if (!ok) return;
          const uint4* src = reinterpret_cast<const uint4*>(smem + C::off_raw + rs * kRawBytes);
          uint8_t* dst = smem + C::off_ring + st * kStageBytes;
          uint4 q[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) q[k] = src[tid + k * T];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int e = tid + k * T, key = e / width, d = (e % width) * 16;
            uint4 a, b;
            codes_to_bf16<KIND>(q[k].x, a.x, a.y);
            codes_to_bf16<KIND>(q[k].y, a.z, a.w);
            codes_to_bf16<KIND>(q[k].z, b.x, b.y);
            codes_to_bf16<KIND>(q[k].w, b.z, b.w);
            uint8_t* line = dst + (value ? (d >> 6) * C::vkeys * 128 : 0) + key * 128;
            const int e16 = (d & 63) >> 3;
            *reinterpret_cast<uint4*>(line + ((e16 ^ (key & 7)) << 4)) = a;
            *reinterpret_cast<uint4*>(line + (((e16 + 1) ^ (key & 7)) << 4)) = b;
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&full[st]);
            mbar_arrive(&rempty[rs]);  // after the stores, which came after the loads
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
      for (int i = 0; i < n && ok; ++i) {
        const int tile = key_tile(u.kt, u.begin + i);
        if (!tile_cut(u, tile, p.window, p.sinks)) continue;
        int it = (i + min(C::sbufs + i, n)) * C::chunks;  // V i comes after that many tiles
        for (int c = 0; c < C::chunks && ok; ++c, ++it) {
          const int st = it % C::stages;
          if (!(ok = wait(&clean[st], (landed >> st) & 1))) break;
          landed ^= 1u << st;
          uint4* v = reinterpret_cast<uint4*>(smem + C::off_ring + st * kStageBytes);
          bool bad = false;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int e = tid + k * T, j = tile * kTileN + c * C::vkeys + (e >> 3) % C::vkeys;
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
          if (bad) *odd = 1;
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[st]);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(pdone);
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
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

// Codes as rows of dh values, one to a vector; boxes of `width` values and `rows` vectors of one page.
bool code_map(CUtensorMap* map, void* base, bool quant, int dh, int64_t n_vec, int width, int rows) {
  memset(map, 0, sizeof(*map));
  const cuuint64_t dim[2] = {(cuuint64_t)dh, (cuuint64_t)n_vec};
  const cuuint64_t stride[1] = {(cuuint64_t)dh * (quant ? 1 : 2)};
  const cuuint32_t box[2] = {(cuuint32_t)width, (cuuint32_t)rows}, one[2] = {1, 1};
  return g_encode(map, quant ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dim, stride,
                  box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, quant ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DH, int KIND>
cudaError_t launch(const AttnParams& p, int page, int64_t n_vec, int64_t blocks, int* status, cudaStream_t s) {
  using C = Cfg<DH, KIND>;
  cudaError_t e = encoder();
  if (e != cudaSuccess) return e;
  CUtensorMap kmap, vmap;
  if (!code_map(&kmap, p.c.k, C::quant, DH, n_vec, 64, std::min(page, kTileN)) ||
      !code_map(&vmap, p.c.v, C::quant, DH, n_vec, C::quant ? DH : 64, std::min(page, C::vkeys)))
    return cudaErrorInvalidValue;
  e = cudaFuncSetAttribute(attn_tile_kernel<DH, KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)blocks, (unsigned)p.c.n_kv, (unsigned)p.splits);
  attn_tile_kernel<DH, KIND><<<grid, C::threads, C::smem, s>>>(p, kmap, vmap, status);
  return cudaGetLastError();
}

template <int DH>
cudaError_t by_kind(int kind, const AttnParams& p, int page, int64_t n_vec, int64_t blocks, int* status,
                    cudaStream_t s) {
  return kind == FAK_KV_BF16   ? launch<DH, FAK_KV_BF16>(p, page, n_vec, blocks, status, s)
         : kind == FAK_KV_E4M3 ? launch<DH, FAK_KV_E4M3>(p, page, n_vec, blocks, status, s)
                               : launch<DH, FAK_KV_I8>(p, page, n_vec, blocks, status, s);
}

}  // namespace

cudaError_t attn_tile_launch(int kind, int dh, int page, int64_t n_vec, const AttnParams& p, int64_t blocks,
                             int* status, cudaStream_t s) {
  return dh == 64    ? by_kind<64>(kind, p, page, n_vec, blocks, status, s)
         : dh == 128 ? by_kind<128>(kind, p, page, n_vec, blocks, status, s)
                     : by_kind<256>(kind, p, page, n_vec, blocks, status, s);
}
