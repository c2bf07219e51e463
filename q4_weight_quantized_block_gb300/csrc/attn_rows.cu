// Attention of few rows over the paged KV cache: decode steps, where a sequence and KV head has at most 16 rows
// (token, query head of the group) and all that counts is reading K and V once, at the memory's rate.
//
// A warp takes 16 keys at a time, in the layouts of the m16n8k16 matrix instruction without any turning, with the keys
// and dims as its 16 and the rows as its 8 (6 rows of a group of 6 waste 2, not 10):
//   S^T = K Q^T      A = K: lane (g, t) loads 16 bytes of two keys, which are its dims of two (8-bit codes: four)
//                    instructions; the dims come in another order than they stand, the same for Q
//   O^T += V^T P^T   A = V^T: lane (g, t) loads 16 bytes of four keys and pairs up neighbouring keys' values; P^T from
//                    S^T by an 8 x 8 transpose within the warp
// Few rows leave the tensor cores idle whatever instruction is used, so the plain one does.
//
// K and V of 16 keys are consecutive in a page: they come by bulk copies into slots of the warp's own, each with a
// barrier of its own, one to four steps ahead.  (As asynchronous copies of 16 bytes by each lane the loads alone reached
// 4.9 TB/s, as bulk copies 6.6: 64 sequences of up to 8,191 bf16 keys of 256 took 258 us, then 212, and without bank
// conflicts 202.)  Four warps share a block's keys in tiles of 64 or 128 and add their sums at the end; a sequence's
// keys are cut over blocks, which the join kernel adds.  The product of a step runs beside the scores of the next,
// which do not depend on it.
//
// 8-bit codes are multiplied as f16, which holds both kinds exactly and takes one conversion for two e4m3 codes (as bf16
// they took twice as many instructions: 131,071 int8 keys of 128, 78 us, then 64).  Q goes in as f16 too, each row
// scaled by a power of two; weights are 2^(score + log2 of the value's scale), under a maximum of those exponents.  Their
// sum, which the values have no part in, has a base of its own in each lane.
//
// Bound: bf16 by memory, 64 x 8,191 keys in 202 us, 6.1 TB/s (the copies alone 189); 8-bit by the instructions of the
// conversion, the same in e4m3 130 us, 4.9 TB/s (the copies alone 104); few keys by the launches and one block's chain
// of loads.  9 to 16 rows (255 registers, two blocks an SM): 64 sequences' two tokens over 4,000 keys in 187 us in bf16,
// 5.6 TB/s, 173 in e4m3, 175 in int8, 3.1.
// Each row's maximum moves only when passed by 8, as in the blocks' kernel (attn_tile.cu).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_device.cuh"
#include "fak.h"
#include "fak_device.cuh"
#include "fak_tc.cuh"

namespace {

constexpr int kWarps = 4;

// d += A B, bf16 or (F16) f16.
template <bool F16>
FAK_DEV void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8-bit codes as f16, exactly.  e4m3: one conversion for two.  int8, with the sign bit turned over: 0x6400 + code is
// 1024 + code in f16, less 1152.
FAK_DEV uint32_t less_1152(uint32_t x) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(0x64806480u));
  return d;
}
FAK_DEV uint32_t e4m3_to_f16(uint32_t two) {
  uint32_t d;
  asm("{ .reg .b16 h;\n cvt.u16.u32 h, %1;\n cvt.rn.f16x2.e4m3x2 %0, h; }" : "=r"(d) : "r"(two));
  return d;
}

// The four codes of a word, in order.
template <int KIND>
FAK_DEV void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (KIND == FAK_KV_E4M3) {
    lo = e4m3_to_f16(w & 0xffffu);
    hi = e4m3_to_f16(w >> 16);
  } else {
    const uint32_t x = w ^ 0x80808080u;
    lo = less_1152(prmt(x, 0x64646464u, 0x4140));
    hi = less_1152(prmt(x, 0x64646464u, 0x4342));
  }
}

// Each code of v beside the same code of w.
template <int KIND>
FAK_DEV void pairs_to_f16(uint32_t v, uint32_t w, uint32_t (&d)[4]) {
  if constexpr (KIND == FAK_KV_E4M3) {
    uint32_t v0, v1, w0, w1;
    codes_to_f16<KIND>(v, v0, v1);
    codes_to_f16<KIND>(w, w0, w1);
    d[0] = prmt(v0, w0, 0x5410);
    d[1] = prmt(v0, w0, 0x7632);
    d[2] = prmt(v1, w1, 0x5410);
    d[3] = prmt(v1, w1, 0x7632);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      d[e] = less_1152((prmt(v, w, 0x4400u + 0x1111u * (uint32_t)e) & 0x00FF00FFu) ^ 0x64806480u);
  }
}

FAK_DEV uint32_t pack_f16(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// With m the exponents' maximum less 7, the largest weight (times its value's scale) is 2^7 to 2^15: f16 keeps 11 bits of
// those down to 2^-14, and half a step of 2^-24 below, 2^-32 of the largest.
// The logarithm puts a value's scale in its weight's exponent: off by 2^-22 at scales near 1, by 2^-18 at the exponent's
// ends, as the sum of the two is rounded there too.
FAK_DEV float log2_approx(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

FAK_DEV uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

FAK_DEV int key_of(int i) { return ((i >> 1) ^ (i & 1) << 1) * 4 + (i & 1); }

// A row's base before any score.  (Minus infinity would need a look at each exponent: minus infinity less itself is NaN.)
constexpr float kNone = -3.402823466e38f;

template <int DH, int KIND, int NT>
struct RCfg {
  static constexpr bool quant = KIND != FAK_KV_BF16;
  static constexpr int bytes = quant ? 1 : 2;
  static constexpr int ke = 16 / bytes;                        // dims of a lane's K load
  static constexpr int kb = DH / (4 * ke);                     // K loads of a key and lane
  static constexpr int ve = 16 / bytes < DH / 8 ? 16 / bytes : DH / 8;  // dims of a lane's V load
  static constexpr int vb = DH / (8 * ve);                     // V loads of a key and lane
  static constexpr int vw = ve * bytes / 4;                    // words of one
  static constexpr int groups = quant && DH <= 128 ? 2 : 1;  // 16 keys each, of a step
  // 16 keys come in four copies, 32 bytes apart in the banks, and index i of the instructions' 8 (and i + 8) is key
  // key_of(i) (and that + 2): what 8 lanes load at once, two neighbouring indices' 64 bytes of K or four's 32 bytes of
  // V (every other index), then lies in different banks
  static constexpr int row_bytes = DH * bytes, four = 4 * row_bytes + 32, part = 4 * four;
  static constexpr int half = groups * (part + (quant ? 128 : 0));     // of a half (with a group's scales)
  // blocks of four warps on an SM; a warp's slots, halves of a step in turn, K and V, as many as then have room
  static constexpr int blocks = rows_blocks(quant, DH, 8 * NT);
  static constexpr int room = (233472 / blocks - 1792) / kWarps;
  static constexpr int halves = room / half < 8 ? room / half : 8;
  static constexpr float above = quant ? 7.0f : 0.0f, reach = above + 8.0f;
  static constexpr int row = DH + 8;  // floats of a row where the warps' sums meet
  static constexpr int sums = kWarps * 8 * NT * row * 4;
  static constexpr int smem = kWarps * halves * half > sums ? kWarps * halves * half : sums;
  static_assert(halves >= 3, "a half is worked on while others come");
};

template <int DH, int KIND, int NT>
__global__ void __launch_bounds__(kWarps * 32, RCfg<DH, KIND, NT>::blocks)
    attn_rows_kernel(const __grid_constant__ AttnParams p, int* status) {
  using C = RCfg<DH, KIND, NT>;
  extern __shared__ __align__(16) uint8_t smem[];
  float* so = reinterpret_cast<float*>(smem);  // at the end: [warp][8 NT rows][C::row]
  __shared__ float sm[kWarps][8 * NT], sl[kWarps][8 * NT], sb[kWarps][8 * NT];  // bases of O, the weights' sums, theirs
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int seq = blockIdx.x, kvh = blockIdx.y;
  // (the join kernel may be scheduled from here on; it waits for this grid's end itself)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const KvSeq sq = kv_seq(p.c, seq);
  if (!sq.ok) {
    if (threadIdx.x == 0) attn_record(status, FAK_ERR_DEVICE);
    return;
  }
  const int nrows = (sq.r1 - sq.r0) * p.group;
  if (nrows == 0) return;
  const int p0 = sq.len - (sq.r1 - sq.r0), p_lo = p0, p_hi = sq.len - 1;
  constexpr int tile = kWarps * 16 * C::groups;  // keys of a tile: 64 or 128
  const KeyTiles kt = key_tiles(p_lo, p_hi, p.window, p.sinks, tile == 64 ? 6 : 7);
  const bool direct = p.splits == 1 || kt.n <= p.per_split;
  const int begin = direct ? 0 : (int)blockIdx.z * p.per_split;
  const int end = direct || (int)blockIdx.z == p.splits - 1 ? kt.n : min(kt.n, begin + p.per_split);
  if (direct ? blockIdx.z != 0 : begin >= end) return;

  // A warp's steps: its keys of one tile after the other, the sinks' tiles first.  Keys past the last that a row
  // sees take that one's page; what lies there is masked.
  auto next = [&](int& i, int& j0) {
    ++i;
    j0 = i >= end ? -1 : i == begin || i == kt.head ? key_tile(kt, i) * tile + 16 * C::groups * warp : j0 + tile;
  };
  auto place = [&](int j) {
    int64_t at = kv_place(p.c, seq, min(j, p_hi & ~15), kvh);
    if (at < 0) {
      attn_record(status, FAK_ERR_DEVICE);
      at = -1 - at;
    }
    return at;
  };
  uint8_t* const slots = smem + warp * (C::halves * C::half);
  __shared__ uint64_t bars[kWarps][C::halves];  // a slot's bytes are there
  if (lane == 0) {
#pragma unroll
    for (int h = 0; h < C::halves; ++h) mbar_init(&bars[warp][h], 1 + p.unreachable);
    fence_mbar_init();
  }
  __syncwarp();
  // fetched up to halves / 2 steps ahead of the one at work
  constexpr int G = C::groups, gpart = C::half / G;
  int fi = begin - 1, fj = 0;  // the step that is fetched
  next(fi, fj);
  int i = fi, j0 = fj;
  int64_t fat[G];
  auto places = [&]() {
    if (fj >= 0) {
#pragma unroll
      for (int x = 0; x < G; ++x) fat[x] = place(fj + 16 * x);
    }
  };
  places();
  auto fetch = [&](int slot, bool value) {  // a half, where what stood there has been read; nothing past the last step
    if (fj >= 0 && elect_one()) {
      uint64_t* const bar = &bars[warp][slot];
      mbar_arrive_expect_tx(bar, G * (16 * C::row_bytes + (C::quant && !value ? 128 : 0)));
#pragma unroll
      for (int x = 0; x < G; ++x) {
        uint8_t* const to = slots + slot * C::half + x * gpart;
        const uint8_t* const src = (value ? p.c.v : p.c.k) + fat[x] * C::row_bytes;
#pragma unroll
        for (int c = 0; c < 4; ++c) bulk_g2s_nohint(to + c * C::four, src + c * 4 * C::row_bytes, 4 * C::row_bytes, bar);
        if (C::quant && !value) {
          bulk_g2s_nohint(to + C::part, p.c.ks + fat[x], 64, bar);
          bulk_g2s_nohint(to + C::part + 64, p.c.vs + fat[x], 64, bar);
        }
      }
    }
    if (value) {
      next(fi, fj);
      places();
    }
  };
  constexpr bool oddly = C::halves % 2;  // then the half that comes into K's slot is V, and the other way round
#pragma unroll
  for (int h = 0; h < C::halves; ++h) fetch(h, h & 1);
  // Q: lane (g, t) holds row g's (and g + 8's) dims as K's loads bring them
  uint32_t q[NT][DH / 8];
  int pos[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = g + 8 * nt, token = p.by_group(r);
#pragma unroll
    for (int w = 0; w < DH / 32; ++w) {  // 16 bytes: 8 dims
      uint4 x = make_uint4(0, 0, 0, 0);
      const int d = C::quant ? (w >> 1) * 64 + t * 16 + (w & 1) * 8 : w * 32 + t * 8;
      if (r < nrows)
        x = *reinterpret_cast<const uint4*>(p.q + (int64_t)(sq.r0 + token) * p.q_row +
                                            (int64_t)(kvh * p.group + r - token * p.group) * p.q_head + d);
      q[nt][4 * w] = x.x;
      q[nt][4 * w + 1] = x.y;
      q[nt][4 * w + 2] = x.z;
      q[nt][4 * w + 3] = x.w;
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int rr = 2 * t + c + 8 * nt;
      pos[nt][c] = rr < nrows ? p0 + p.by_group(rr) : -1;
    }
  }
  // 8-bit: Q as f16, which holds a bf16's significand, each row by the power of two that brings its largest to 1 .. 2
  // (what is then below 2^-24 is lost, 2^-24 of the largest); its inverse goes into the scores
  float qf[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    uint32_t top = 0;
    if constexpr (C::quant) {
#pragma unroll
      for (int w = 0; w < DH / 8; ++w) top = max(top, max(q[nt][w] << 16 & 0x7fff0000u, q[nt][w] & 0x7fff0000u));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      top = min(max(top & 0x7f800000u, 0x00800000u), 0x7e800000u);  // the exponent alone, and one that has an inverse
      const float up = __uint_as_float(top), down = __uint_as_float(0x7f000000u - top);
#pragma unroll
      for (int w = 0; w < DH / 8; ++w)
        q[nt][w] = pack_f16(__uint_as_float(q[nt][w] << 16) * down, __uint_as_float(q[nt][w] & 0xffff0000u) * down);
      qf[nt][0] = __shfl_sync(0xffffffffu, up, 8 * t) * p.scale;      // rows 2t, 2t + 1 are lanes (2t, .), (2t + 1, .)
      qf[nt][1] = __shfl_sync(0xffffffffu, up, 8 * t + 4) * p.scale;
    } else {
      qf[nt][0] = qf[nt][1] = p.scale;
    }
  }
  float o[NT][DH / 16][4] = {};
  float m[NT][2], l[NT][2], lm[NT][2];  // lm: 8-bit, the base of l, this lane's own (8 above the score that set it)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      m[nt][c] = lm[nt][c] = kNone;
      l[nt][c] = 0.0f;
    }

  const int kg = key_of(g), krow = (kg >> 2) * C::four + (kg & 3) * C::row_bytes;
  const int vrow[2] = {t * C::four, (t ^ 2) * C::four + C::row_bytes};  // keys key_of(2t), key_of(2t + 1)
  float s[G][NT][4];  // s[x][nt][c + 2 h]: key 16 x + kg + 2 h, row 2t + c + 8 nt
  float kf[G][2], vl[G][2];  // 8-bit: the keys' scales, log2 of the values'
  uint32_t pb[G][NT][2];
  auto scores = [&](const uint8_t* from) {
#pragma unroll
    for (int x = 0; x < G; ++x)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[x][nt][c] = 0.0f;
#pragma unroll
    for (int b = 0; b < C::kb; ++b)
#pragma unroll
      for (int x = 0; x < G; ++x) {
        const uint4 x0 = *reinterpret_cast<const uint4*>(from + x * gpart + krow + b * 64 + t * 16);
        const uint4 x1 = *reinterpret_cast<const uint4*>(from + x * gpart + krow + 2 * C::row_bytes + b * 64 + t * 16);
        const uint32_t a0[4] = {x0.x, x0.y, x0.z, x0.w}, a1[4] = {x1.x, x1.y, x1.z, x1.w};
        if constexpr (C::quant) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t k0, k1, l0, l1;
            codes_to_f16<KIND>(a0[w], k0, k1);
            codes_to_f16<KIND>(a1[w], l0, l1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816<true>(s[x][nt], k0, l0, k1, l1, q[nt][8 * b + 2 * w], q[nt][8 * b + 2 * w + 1]);
          }
        } else {
#pragma unroll
          for (int w = 0; w < 4; w += 2)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816<false>(s[x][nt], a0[w], a1[w], a0[w + 1], a1[w + 1], q[nt][4 * b + w], q[nt][4 * b + w + 1]);
        }
      }
    if constexpr (C::quant) {
#pragma unroll
      for (int x = 0; x < G; ++x) {
        const float* f = reinterpret_cast<const float*>(from + x * gpart + C::part);
        kf[x][0] = f[kg];
        kf[x][1] = f[kg + 2];
        vl[x][0] = log2_approx(f[16 + kg]);
        vl[x][1] = log2_approx(f[16 + kg + 2]);
      }
    }
  };
  auto softmax = [&](int sj) {
    const bool scut = keys_cut(p_lo, p_hi, sj, sj + 16 * G - 1, p.window, p.sinks);
#pragma unroll
    for (int x = 0; x < G; ++x) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          s[x][nt][c] *= C::quant ? kf[x][c >> 1] * qf[nt][c & 1] : qf[nt][c & 1];
          if (scut && !sees(pos[nt][c & 1], sj + 16 * x + kg + 2 * (c >> 1), p.window, p.sinks))
            s[x][nt][c] = -INFINITY;
        }
    }
    // 8-bit: a value's scale is part of its weight, 2^(t + log2 scale - m), with m set by the largest of those
    // exponents, so that weights fit f16 whatever the scales are.  The sum is of 2^(t - lm): with m as its base it would
    // lose what came before a value 2^126 times as large, zeros too.
    auto heavy = [&](int x, int nt, int c) {
      if constexpr (C::quant) return s[x][nt][c] + vl[x][c >> 1];
      return s[x][nt][c];
    };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float top[2], own[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        top[c] = fmaxf(heavy(0, nt, c), heavy(0, nt, c + 2));
        if constexpr (G == 2) top[c] = fmaxf(top[c], fmaxf(heavy(G - 1, nt, c), heavy(G - 1, nt, c + 2)));
        if constexpr (C::quant) {
          own[c] = fmaxf(s[0][nt][c], s[0][nt][c + 2]);
          if constexpr (G == 2) own[c] = fmaxf(own[c], fmaxf(s[G - 1][nt][c], s[G - 1][nt][c + 2]));
        }
      }
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], x));
        top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], x));
      }
      const bool up0 = top[0] > m[nt][0] + C::reach, up1 = top[1] > m[nt][1] + C::reach;
      const bool on0 = C::quant && own[0] > lm[nt][0], on1 = C::quant && own[1] > lm[nt][1];
      if (__any_sync(0xffffffffu, up0 || up1 || on0 || on1)) {
        const float n0 = up0 ? top[0] - C::above : m[nt][0], n1 = up1 ? top[1] - C::above : m[nt][1];
        const float f0 = up0 ? exp2_approx(m[nt][0] - n0) : 1.0f, f1 = up1 ? exp2_approx(m[nt][1] - n1) : 1.0f;
        m[nt][0] = n0;
        m[nt][1] = n1;
        if constexpr (C::quant) {
          const float l0 = on0 ? own[0] + 8.0f : lm[nt][0], l1 = on1 ? own[1] + 8.0f : lm[nt][1];
          if (on0) l[nt][0] *= exp2_approx(lm[nt][0] - l0);
          if (on1) l[nt][1] *= exp2_approx(lm[nt][1] - l1);
          lm[nt][0] = l0;
          lm[nt][1] = l1;
        } else {
          l[nt][0] *= f0;
          l[nt][1] *= f1;
        }
#pragma unroll
        for (int d = 0; d < DH / 16; ++d) {
          o[nt][d][0] *= f0;
          o[nt][d][1] *= f1;
          o[nt][d][2] *= f0;
          o[nt][d][3] *= f1;
        }
      }
#pragma unroll
      for (int x = 0; x < G; ++x) {
        float w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          w[c] = exp2_approx(s[x][nt][c] - (C::quant ? lm : m)[nt][c & 1]);
          l[nt][c & 1] += w[c];
          if constexpr (C::quant) {
            w[c] = exp2_approx(s[x][nt][c] + vl[x][c >> 1] - m[nt][c & 1]);
            // (the scale of a key that is not seen may be anything)
            if (scut && s[x][nt][c] == -INFINITY) w[c] = 0.0f;
          }
        }
        pb[x][nt][0] = transpose8(C::quant ? pack_f16(w[0], w[1]) : pack_bf16(w[0], w[1]));
        pb[x][nt][1] = transpose8(C::quant ? pack_f16(w[2], w[3]) : pack_bf16(w[2], w[3]));
      }
    }
  };
  // e4m3: NaN codes of a value that some rows see and others do not would reach the others as 0 * NaN.  They are made
  // zeros where they stand, ahead of the product, and the rows that do see them get NaN.
  auto nan_codes = [&](uint8_t* from) {
    bool found = false;
#pragma unroll 1
    for (int w = lane; w < 4 * G * C::row_bytes; w += 32) {  // words: 4 row_bytes of a group's keys, in four parts
      uint32_t* const at = reinterpret_cast<uint32_t*>(from + w / (4 * C::row_bytes) * gpart +
                                                       w % (4 * C::row_bytes) / C::row_bytes * C::four) + w % C::row_bytes;
      const uint32_t nan = ((*at & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;  // bytes of 0x7f and 0xff
      if (nan) *at &= ~((nan >> 7) * 0xffu);
      found |= nan != 0;
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (the next copy there comes after these stores)
    if (!__any_sync(0xffffffffu, found)) return;
    __syncwarp();
#pragma unroll 1
    for (int j = j0; j < min(j0 + 16 * G, p_hi + 1); ++j) {
      const uint8_t* const v = p.c.v + (place(j & ~15) + (j & 15)) * DH;
#pragma unroll
      for (int d = 0; d < DH / 16; ++d) {
        // o[nt][d]: dims ve g + 2 (d % (ve / 2)), + 1 of block d / (ve / 2)
        const uint32_t y =
            *reinterpret_cast<const uint16_t*>(v + d / (C::ve / 2) * 8 * C::ve + g * C::ve + 2 * (d % (C::ve / 2)));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (sees(pos[nt][c], j, p.window, p.sinks)) {
              if ((y & 0x7Fu) == 0x7Fu) o[nt][d][c] = __uint_as_float(0x7fffffffu);
              if ((y & 0x7F00u) == 0x7F00u) o[nt][d][c + 2] = __uint_as_float(0x7fffffffu);
            }
      }
    }
  };
  auto product = [&](const uint8_t* from) {
    const bool cut = keys_cut(p_lo, p_hi, j0, j0 + 16 * G - 1, p.window, p.sinks);
    bool odd = false;
#pragma unroll
    for (int x = 0; x < G; ++x)
#pragma unroll
      for (int b = 0; b < C::vb; ++b) {
        uint32_t vx[4][C::vw];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint8_t* const at =
              from + x * gpart + vrow[k & 1] + (k >> 1) * 2 * C::row_bytes + (b * 8 + g) * C::vw * 4;
          if constexpr (C::vw == 4) {
            const uint4 y = *reinterpret_cast<const uint4*>(at);
            vx[k][0] = y.x;
            vx[k][1] = y.y;
            vx[k][2] = y.z;
            vx[k][3] = y.w;
          } else {
            const uint2 y = *reinterpret_cast<const uint2*>(at);
            vx[k][0] = y.x;
            vx[k][1] = y.y;
          }
        }
        if (C::quant && cut) {
          // codes that no row sees may be e4m3's NaN
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int j = j0 + 16 * x + key_of(2 * t + (k & 1)) + 2 * (k >> 1);
            const bool seen = j <= p_hi && (!p.window || j > p_lo - p.window || j < p.sinks);
#pragma unroll
            for (int w = 0; w < C::vw; ++w) vx[k][w] = seen ? vx[k][w] : 0u;
          }
        }
        if (!C::quant && cut) {
          // a weight of zero times a value that is not finite would be NaN: such values are left out of the
          // product, and added for the rows that do see them; keys past the last that is seen are zeros
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const bool past = j0 + key_of(2 * t + (k & 1)) + 2 * (k >> 1) > p_hi;
#pragma unroll
            for (int w = 0; w < C::vw; ++w) {
              bool change = false;
              const uint32_t y = finite2(vx[k][w], change);
              vx[k][w] = past ? 0u : y;
              odd |= change && !past;
            }
          }
        }
#pragma unroll
        for (int w = 0; w < C::vw; ++w) {
          // (key 2t, 2t + 1), (2t + 8, 2t + 9): each of the word's dims
          uint32_t y[C::quant ? 4 : 2][2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t v0 = vx[2 * k][w], v1 = vx[2 * k + 1][w];
            if constexpr (C::quant) {
              uint32_t d[4];
              pairs_to_f16<KIND>(v0, v1, d);
#pragma unroll
              for (int e = 0; e < 4; ++e) y[e][k] = d[e];
            } else {
              y[0][k] = prmt(v0, v1, 0x5410);
              y[1][k] = prmt(v0, v1, 0x7632);
            }
          }
#pragma unroll
          for (int h = 0; h < (C::quant ? 2 : 1); ++h) {
            const int d = b * (C::ve / 2) + w * (C::quant ? 2 : 1) + h;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816<C::quant>(o[nt][d], y[2 * h][0], y[2 * h + 1][0], y[2 * h][1], y[2 * h + 1][1],
                                 pb[x][nt][0], pb[x][nt][1]);
          }
        }
      }
    if (!C::quant && cut && __any_sync(0xffffffffu, odd)) {
      const int64_t at = place(j0);
#pragma unroll 1
      for (int j = 0; j < min(16, p_hi + 1 - j0); ++j)
#pragma unroll
        for (int d = 0; d < DH / 16; ++d) {
          // o[nt][d]: dims ve g + 2 (d % (ve / 2)), + 1 of block d / (ve / 2)
          const uint32_t y = *reinterpret_cast<const uint32_t*>(
              p.c.v + ((at + j) * DH + d / (C::ve / 2) * 8 * C::ve + g * C::ve + 2 * (d % (C::ve / 2))) * 2);
          const float lo = __uint_as_float(y << 16), hi = __uint_as_float(y & 0xffff0000u);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              if (sees(pos[nt][c], j0 + j, p.window, p.sinks)) {
                if ((y & 0x7F80u) == 0x7F80u) o[nt][d][c] += lo;
                if ((y & 0x7F800000u) == 0x7F800000u) o[nt][d][c + 2] += hi;
              }
        }
    }
  };
  int slot = 0;
  auto advance = [&]() { slot = slot + 1 == C::halves ? 0 : slot + 1; };
  uint32_t phases = 0;  // of the slots
  auto landed = [&](int h) {  // false: the limit ran out
    uint64_t* const bar = &bars[warp][h];
    const uint32_t parity = phases >> h & 1;
    phases ^= 1u << h;
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait_suspend(bar, parity, 20000u)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait_suspend(bar, parity, 20000u))
      if (globaltimer_ns() - t0 > p.timeout_ns) return false;
    return true;
  };
  // The product of a step runs beside the scores of the next, which do not depend on it.  What stands in a slot is read
  // whether it landed or not; before the slot is filled again the lanes agree on that.  (As a vote ahead of the scores
  // this took 1 to 3% longer.)
  bool ok = true;
  int used = 0;  // where the limit runs out: halves that were waited for before
  if (j0 >= 0) {
    const bool there = landed(0);
    scores(slots);
    ok = __all_sync(0xffffffffu, there);
    if (ok) {
      __syncwarp();
      fetch(0, oddly);
      advance();
      softmax(j0);
    }
  }
  while (ok && j0 >= 0) {
    int ni = i, nj = j0;
    next(ni, nj);
    const int kslot = slot + 1 == C::halves ? 0 : slot + 1;
    const bool there = landed(slot) && (nj < 0 || landed(kslot));
    // (here, not between the scores and the product: there it took 2 to 8% longer)
    if (KIND == FAK_KV_E4M3 && p_lo < p_hi && keys_cut(p_lo, p_hi, j0, j0 + 16 * G - 1, p.window, p.sinks))
      nan_codes(slots + slot * C::half);
    scores(slots + kslot * C::half);  // (past the last step: of what stood there, and not used)
    product(slots + slot * C::half);
    if (!(ok = __all_sync(0xffffffffu, there))) {
      used = 1 + 2 * (i - begin);
      break;
    }
    __syncwarp();
    fetch(slot, !oddly);
    fetch(kslot, oddly);
    if (nj >= 0) softmax(nj);
    advance();
    advance();
    i = ni;
    j0 = nj;
  }

  if (!ok) {
    // the limit ran out: the copies in flight land (or a fifth of a second passes), and the block ends without results
    if (lane == 0) attn_record(status, FAK_ERR_TIMEOUT);
    const uint64_t t0 = globaltimer_ns(), limit = p.timeout_ns < 200000000ull ? p.timeout_ns : 200000000ull;
    for (int n = used; n < min(used + C::halves, 2 * (end - begin)); ++n)
      while (!mbar_try_wait_suspend(&bars[warp][n % C::halves], n / C::halves & 1, 20000u))
        if (globaltimer_ns() - t0 > limit) break;
    __syncwarp();
  }
  if (__syncthreads_or(!ok)) return;  // (from here on the slots are the place where the sums meet)
  // the four warps' sums
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float b = C::quant ? lm[nt][c] : m[nt][c];
      if constexpr (C::quant) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, x));
        l[nt][c] *= exp2_approx(lm[nt][c] - b);
      }
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], x);
      const int r = 2 * t + c + 8 * nt;
      if (g == 0) {
        sm[warp][r] = m[nt][c];
        sb[warp][r] = b;
        sl[warp][r] = l[nt][c];
      }
#pragma unroll
      for (int d = 0; d < DH / 16; ++d)
        *reinterpret_cast<float2*>(so + (warp * 8 * NT + r) * C::row + d / (C::ve / 2) * 8 * C::ve + g * C::ve +
                                   2 * (d % (C::ve / 2))) = make_float2(o[nt][d][c], o[nt][d][c + 2]);
    }
  __syncthreads();
  for (int k = threadIdx.x; k < nrows * (DH / 4); k += kWarps * 32) {
    const int r = k / (DH / 4), d = k % (DH / 4) * 4, token = p.by_group(r);
    const int head = kvh * p.group + r - token * p.group;
    const int64_t row = sq.r0 + token;
    float top = kNone, sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sb[w][r]);
    const float base = top;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum = fmaf(exp2_approx(sb[w][r] - base), sl[w][r], sum);
    // what the sums are multiplied with.  8-bit: it goes into the factors of O, which holds the values' scales: these
    // factors are taken in two halves, as one may be beyond f32 where their product with O is not, and a piece has the
    // whole powers of two of its weights' sum in its base, which leaves a half to 1: it is no larger than its values
    float inv = 1.0f;
    if (direct) {
      inv = 1.0f / sum;
    } else if (C::quant && sum > 0.0f && sum < INFINITY) {  // (at least 2^-8 then)
      const uint32_t e = __float_as_uint(sum) & 0x7f800000u;
      inv = __uint_as_float(0x7e800000u - e);
      sum *= inv;
      top += (float)((int)(e >> 23) - 126);
    }
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 x = *reinterpret_cast<const float4*>(so + (w * 8 * NT + r) * C::row + d);
      if constexpr (C::quant) {
        const float f = exp2_approx(0.5f * (sm[w][r] - base)), h = f * inv;
        y.x = fmaf(x.x * f, h, y.x);
        y.y = fmaf(x.y * f, h, y.y);
        y.z = fmaf(x.z * f, h, y.z);
        y.w = fmaf(x.w * f, h, y.w);
      } else {
        const float f = exp2_approx(sm[w][r] - base);
        y.x = fmaf(f, x.x, y.x);
        y.y = fmaf(f, x.y, y.y);
        y.z = fmaf(f, x.z, y.z);
        y.w = fmaf(f, x.w, y.w);
      }
    }
    if (!direct) {
      const int64_t slot = ((int64_t)blockIdx.z * p.c.rows + row) * p.nq + head;
      *reinterpret_cast<float4*>(p.part + slot * DH + d) = y;
      if (d == 0) p.stat[slot] = make_float2(top, sum);
      continue;
    }
    // a row that sees nothing is zeros; one whose scores are all -inf is NaN, as 0 / 0 is
    float4 x = make_float4(INFINITY, INFINITY, INFINITY, INFINITY);
    const bool blank = p0 + token < 0;
    if (p.gate && !blank) x = *reinterpret_cast<const float4*>(p.gate + row * p.gate_row + head * p.gate_head + d);
    if constexpr (C::quant) inv = 1.0f;
    uint2 w = make_uint2(pack_bf16(gated_by(y.x * inv, x.x), gated_by(y.y * inv, x.y)),
                         pack_bf16(gated_by(y.z * inv, x.z), gated_by(y.w * inv, x.w)));
    if (blank) w = make_uint2(0, 0);
    *reinterpret_cast<uint2*>(p.out + row * p.out_row + head * p.out_head + d) = w;
  }
}

template <int DH, int KIND, int NT>
cudaError_t launch(const AttnParams& p, int* status, int dev, cudaStream_t s) {
  using C = RCfg<DH, KIND, NT>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = kv_smem_limit(attn_rows_kernel<DH, KIND, NT>, C::smem, dev, done);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)p.c.n_seqs, (unsigned)p.c.n_kv, (unsigned)p.splits);
  attn_rows_kernel<DH, KIND, NT><<<grid, kWarps * 32, C::smem, s>>>(p, status);
  return cudaGetLastError();
}

template <int DH, int KIND>
cudaError_t by_rows(const AttnParams& p, int* status, int dev, cudaStream_t s) {
  return p.c.max_q * p.group <= 8 ? launch<DH, KIND, 1>(p, status, dev, s) : launch<DH, KIND, 2>(p, status, dev, s);
}

template <int DH>
cudaError_t by_kind(int kind, const AttnParams& p, int* status, int dev, cudaStream_t s) {
  return kind == FAK_KV_BF16   ? by_rows<DH, FAK_KV_BF16>(p, status, dev, s)
         : kind == FAK_KV_E4M3 ? by_rows<DH, FAK_KV_E4M3>(p, status, dev, s)
                               : by_rows<DH, FAK_KV_I8>(p, status, dev, s);
}

}  // namespace

cudaError_t attn_rows_launch(int kind, int dh, const AttnParams& p, int* status, int dev, cudaStream_t s) {
  return dh == 64    ? by_kind<64>(kind, p, status, dev, s)
         : dh == 128 ? by_kind<128>(kind, p, status, dev, s)
                     : by_kind<256>(kind, p, status, dev, s);
}
