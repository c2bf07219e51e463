// What the attention kernels share: a call's parameters, the plan of its split over
// the keys, and the keys that a block of rows sees.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "kv_device.cuh"

// r / d for 0 <= r < 2^31, by a multiplication: mul = ceil(2^(31 + s) / d), s = ceil(log2 d), shift = s - 1; d = 1: mul 0.
struct Quotient {
  uint32_t mul;
  int shift;
  __device__ __forceinline__ int operator()(int r) const {
    return mul ? (int)(__umulhi((uint32_t)r, mul) >> shift) : r;
  }
};

static inline Quotient quotient(int d) {
  if (d <= 1) return Quotient{0, 0};
  int s = 1;
  while (s < 31 && (1 << s) < d) ++s;
  return Quotient{(uint32_t)(((1ull << (31 + s)) + d - 1) / d), s - 1};
}

struct AttnParams {
  KvView c;
  const __nv_bfloat16* q;
  const float* gate;
  __nv_bfloat16* out;
  int64_t q_row, q_head, gate_row, gate_head, out_row, out_head;
  float scale;  // times log2(e): scores are held in powers of two
  int nq, group, window, sinks;
  int block;       // tokens of a block
  int tile_shift;  // keys of a tile
  Quotient by_group, by_block;  // r / group, r / block
  // the keys of a block of rows are cut into at most `splits` pieces of `per_split` key tiles; a block with more
  // than one piece leaves, for each piece, row and head, the unnormalised sum (part, dh values) and its base and
  // weight sum (stat), which the join kernel adds up
  int splits, per_split;
  float* part;   // [splits][rows][nq][dh]
  float2* stat;  // [splits][rows][nq]
  unsigned long long timeout_ns;
  int unreachable;  // a test's: 1 where copies are never to count as landed
};

constexpr int kTileM = 128;  // rows (token, query head of the group) of a CTA
constexpr int kTileN = 128;  // keys of a tile of the blocks' kernel
constexpr int kRowsMax = 16;  // most rows of a sequence and KV head that the kernel for few rows takes
// its blocks on an SM, as registers allow (64 sequences of up to 4,000 bf16 keys of 128: three 64 us, two 66; of up to
// 8,191 e4m3 keys of 256: three 130, two 142, four, which spill, 160)
constexpr int rows_blocks(bool quant, int dh, int rows) { return rows > 8 || (!quant && dh > 128) ? 2 : 3; }
constexpr int kRowsN = 64;    // keys of its tiles (8-bit codes and dh up to 128: twice as many)

FAK_DEV int ceil_div(int a, int b) { return (a + b - 1) / b; }

// The key tiles (of 2^shift keys) that rows at positions p_lo .. p_hi see: those of the first few positions
// that lie before the window's tiles, then the window's.
struct KeyTiles {
  int n, head, first;  // tiles in all, tiles of the sinks, first tile of the window
};

FAK_DEV KeyTiles key_tiles(int p_lo, int p_hi, int window, int sinks, int shift) {
  KeyTiles t{0, 0, 0};
  if (p_hi < 0) return t;
  if (window) {
    const int low = max(0, max(0, p_lo) - window + 1);
    t.first = low >> shift;
    t.head = min((min(sinks, p_hi + 1) + (1 << shift) - 1) >> shift, t.first);
  }
  t.n = t.head + (p_hi >> shift) - t.first + 1;
  return t;
}

FAK_DEV int key_tile(const KeyTiles& t, int i) { return i < t.head ? i : t.first + i - t.head; }

FAK_DEV bool sees(int pos, int j, int window, int sinks) {
  return j <= pos && (!window || j > pos - window || j < sinks);
}

// Whether some row at positions p_lo .. p_hi does not see some key of j0 .. j1.
FAK_DEV bool keys_cut(int p_lo, int p_hi, int j0, int j1, int window, int sinks) {
  return !(j1 <= p_lo && (!window || j0 > p_hi - window || j1 < sinks));
}

// Weights' exponentials take one instruction, off by 2^-22 of the result, where rounding the weight to bf16 or f16 may
// be off by 2^-8 or 2^-11.  Results below 2^-126 are zero.
FAK_DEV float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// y * sigmoid(x); x = infinity: y.  The fast forms, off by some 2^-21, where the result is rounded to bf16 at once
// (below x = -87 a sigmoid of 2^-126 and less counts as zero).
FAK_DEV float gated_by(float y, float x) { return __fdividef(y, 1.0f + __expf(-x)); }

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

// Two 8-bit codes, spread to the halves of a word by prmt, as two bf16, exactly.
//   e4m3 (in the halves' upper bytes): its exponent and significand bits set as bf16's stand for the value times 2^-120,
//   subnormals too.  int8 (in the lower bytes): 128 + the low seven bits, less 128 or, for the negative, 256.
// The other bytes may hold anything.
template <int KIND>
FAK_DEV uint32_t spread_to_bf16(uint32_t a) {
  if constexpr (KIND == FAK_KV_E4M3)
    return hmul2_bf16(((a >> 4) & 0x07F007F0u) | (a & 0x80008000u), 0x7B807B80u);
  else
    return hsub2_bf16((a & 0x007F007Fu) | 0x43004300u, (a & 0x00800080u) | 0x43004300u);
}

// The four codes of a word, in order.
template <int KIND>
FAK_DEV void codes_to_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  lo = spread_to_bf16<KIND>(prmt(w, w, 0x1100));
  hi = spread_to_bf16<KIND>(prmt(w, w, 0x3322));
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

// Records a device-side error of the call (attn.cu's status word).
FAK_DEV void attn_record(int* status, int code) { atomicCAS(status, 0, code); }

// Host: launches of the kernels in the other files.
cudaError_t attn_tile_launch(int kind, int dh, int page, int64_t n_vec, const AttnParams& p, int64_t blocks,
                             int* status, int dev, cudaStream_t s);
cudaError_t attn_rows_launch(int kind, int dh, const AttnParams& p, int* status, int dev, cudaStream_t s);
