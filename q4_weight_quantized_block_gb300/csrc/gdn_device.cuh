// What the kernels of the Gated DeltaNet layers share: a ragged batch with its slots (seen through the paged cache's
// view of one: a slot is its table's only page, positions are not bounded), and the linear attention's parameters.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "kv_device.cuh"

constexpr int kGdnDim = 128;  // key and value dims of a head
constexpr int kGdnState = kGdnDim * kGdnDim;

// Most rows of a sequence that goes row by row.  48 heads of one sequence take 8.4 us for 6 rows and 28.2 for 28 that way, and 31.0
// by chunks of 64, however many of the 64 there are; of 16 sequences 33, 119 and 146 us, of 64 130, 429 and 465.
constexpr int kGdnFew = 28;

// A sequence's rows that are no padding [first, r1), its slot, whether it begins with an empty state.
struct GdnSeq {
  int r0, first, r1, slot;
  bool fresh, ok;
};

FAK_DEV GdnSeq gdn_seq(const KvView& c, const KvSeq& q, int s) {
  GdnSeq d;
  d.slot = c.table[s];
  d.ok = q.ok && (unsigned)d.slot < (unsigned)c.n_pages;
  d.r0 = q.r0;
  d.r1 = q.r1;
  d.first = q.r1 - min(q.len, q.r1 - q.r0);
  d.fresh = q.len <= q.r1 - q.r0;
  return d;
}

struct GdnParams {
  KvView c;
  const __half *q, *k;
  const __nv_bfloat16* v;
  const float *g, *beta, *norm_w, *z;
  float* state;
  void* out;
  int64_t q_row, q_head, k_row, k_head, v_row, v_head, z_row, z_head, out_row, out_head;
  float scale, eps;
  int nv, group;
  bool out_bf16, z_wide, out_wide;  // z_wide: every vector of z stands on a multiple of 16 bytes; both: strides that TMA takes
  int few;  // most rows of a sequence that goes through the steps' kernel
};

// x / (1 + exp(-x)) by the fast exponential and reciprocal: off by some 2^-21 of itself (below x = -88: zero).
FAK_DEV float gdn_silu(float x) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return x * r;
}

FAK_DEV float4 gdn_zero4() { return make_float4(0.0f, 0.0f, 0.0f, 0.0f); }

// Four neighbouring values, f32 or bf16.
FAK_DEV void gdn_put4(void* out, bool bf16, int64_t at, const float4& x) {
  if (bf16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = x;
  }
}

FAK_DEV float4 gdn_bf16x4(const uint2& w) {
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u));
}

FAK_DEV float4 gdn_gate4(const GdnParams& p, const float* z) {
  if (p.z_wide) return *reinterpret_cast<const float4*>(z);
  return make_float4(z[0], z[1], z[2], z[3]);
}

FAK_DEV float gdn_warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Host: the launch of the chunks' kernel (gdn_chunk.cu).
cudaError_t gdn_chunk_launch(const GdnParams& p, unsigned long long timeout_ns, int unreachable, int* status, int dev, int sms,
                             cudaStream_t s);
