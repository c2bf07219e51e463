// Attention of few rows over the paged KV cache: decode steps, where a sequence and KV head has at most 16 rows
// (token, query head of the group) and all that counts is reading K and V once, at the memory's rate.
//
// A warp takes 16 keys at a time straight from memory into registers, in the layouts of the m16n8k16 matrix
// instruction, with the keys and dims as its 16 and the rows as its 8 (6 rows of a group of 6 waste 2, not 10):
//   S^T = K Q^T      A = K: lane (g, t) loads 16 bytes of keys g and g + 8, which are its dims of two (8-bit codes:
//                    four) instructions; the dims come in another order than they stand, the same for Q
//   O^T += V^T P^T   A = V^T: lane (g, t) loads 16 bytes of keys 2t, 2t + 1, 2t + 8 and 2t + 9 and pairs up
//                    neighbouring keys' values; P^T from S^T by an 8 x 8 transpose within the warp
// The next keys' loads are issued as soon as the registers are free, K's before the softmax and V's after the
// product, so 8 warps keep 64 KB (8-bit: half) on their way on an SM.  Four warps share a block's keys in tiles
// of 64 and add their sums at the end; a sequence's keys are cut over blocks, which the join kernel adds.
// Each row's maximum moves only when passed by 8, as in the blocks' kernel (attn_tile.cu).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_device.cuh"
#include "fak.h"
#include "fak_device.cuh"

namespace {

constexpr int kWarps = 4;

FAK_DEV void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

FAK_DEV uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

FAK_DEV uint4 load_once(const void* p) {  // read once: not kept in L1
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
FAK_DEV uint2 load_once8(const void* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

template <int DH, int KIND, int NT>
struct RCfg {
  static constexpr bool quant = KIND != FAK_KV_BF16;
  static constexpr int bytes = quant ? 1 : 2;
  static constexpr int ke = 16 / bytes;                        // dims of a lane's K load
  static constexpr int kb = DH / (4 * ke);                     // K loads of a key and lane
  static constexpr int ve = 16 / bytes < DH / 8 ? 16 / bytes : DH / 8;  // dims of a lane's V load
  static constexpr int vb = DH / (8 * ve);                     // V loads of a key and lane
  static constexpr int vw = ve * bytes / 4;                    // words of one
  static constexpr int row = DH + 8;                           // floats of a row in shared memory
  static constexpr int smem = kWarps * 8 * NT * row * 4;
};

template <int DH, int KIND, int NT>
__global__ void __launch_bounds__(kWarps * 32, 2)
    attn_rows_kernel(const __grid_constant__ AttnParams p, int* status) {
  using C = RCfg<DH, KIND, NT>;
  extern __shared__ float so[];  // [warp][8 NT rows][C::row]
  __shared__ float sm[kWarps][8 * NT], sl[kWarps][8 * NT];
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
  const KeyTiles kt = key_tiles(p_lo, p_hi, p.window, p.sinks, 6);
  const bool direct = p.splits == 1 || kt.n <= p.per_split;
  const int begin = direct ? 0 : (int)blockIdx.z * p.per_split;
  const int end = direct || (int)blockIdx.z == p.splits - 1 ? kt.n : min(kt.n, begin + p.per_split);
  if (direct ? blockIdx.z != 0 : begin >= end) return;

  // this warp's 16 keys of tile i: their first, and its vector index; none of them seen: -1
  auto first_key = [&](int i) {
    if (i >= end) return -1;
    const int j0 = key_tile(kt, i) * kRowsN + 16 * warp;
    const bool none = j0 > p_hi || (p.window && j0 + 15 <= p_lo - p.window && j0 >= p.sinks);
    return none ? -1 : j0;
  };
  auto place = [&](int j0) {
    if (j0 < 0) return (int64_t)0;
    int64_t at = kv_place(p.c, seq, j0, kvh);
    if (at < 0) {
      attn_record(status, FAK_ERR_DEVICE);
      at = -1 - at;
    }
    return at;
  };
  uint4 kx[2][C::kb];
  float ksc[2] = {}, vsc[2] = {};
  uint32_t vx[4][C::vb][C::vw];
  auto load_k = [&](int64_t at) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t v = at + g + 8 * h;
#pragma unroll
      for (int b = 0; b < C::kb; ++b) kx[h][b] = load_once(p.c.k + (v * DH + b * 4 * C::ke + t * C::ke) * C::bytes);
      if constexpr (C::quant) {
        ksc[h] = p.c.ks[v];
        vsc[h] = p.c.vs[v];
      }
    }
  };
  auto load_v = [&](int64_t at) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t v = at + 2 * t + (k & 1) + 8 * (k >> 1);
#pragma unroll
      for (int b = 0; b < C::vb; ++b) {
        const uint8_t* src = p.c.v + (v * DH + b * 8 * C::ve + g * C::ve) * C::bytes;
        if constexpr (C::vw == 4) {
          const uint4 x = load_once(src);
          vx[k][b][0] = x.x;
          vx[k][b][1] = x.y;
          vx[k][b][2] = x.z;
          vx[k][b][3] = x.w;
        } else {
          const uint2 x = load_once8(src);
          vx[k][b][0] = x.x;
          vx[k][b][1] = x.y;
        }
      }
    }
  };
  int i = begin, j0 = first_key(i);
  while (j0 < 0 && i < end) j0 = first_key(++i);  // (a warp may have none at all)
  int64_t at = place(j0);
  if (j0 >= 0) {
    load_k(at);
    load_v(at);
  }

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
  float o[NT][DH / 16][4] = {};
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      m[nt][c] = -INFINITY;
      l[nt][c] = 0.0f;
    }

  while (j0 >= 0) {
    int ni = i + 1, nj = first_key(ni);
    while (nj < 0 && ni < end) nj = first_key(++ni);
    const int64_t nat = place(nj);
    // scores of 16 keys: s[nt][c + 2 h] of key g + 8 h, row 2t + c + 8 nt
    float s[NT][4] = {};
#pragma unroll
    for (int b = 0; b < C::kb; ++b) {
      const uint32_t a0[4] = {kx[0][b].x, kx[0][b].y, kx[0][b].z, kx[0][b].w};
      const uint32_t a1[4] = {kx[1][b].x, kx[1][b].y, kx[1][b].z, kx[1][b].w};
      if constexpr (C::quant) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t x0, x1, y0, y1;
          codes_to_bf16<KIND>(a0[w], x0, x1);
          codes_to_bf16<KIND>(a1[w], y0, y1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(s[nt], x0, y0, x1, y1, q[nt][8 * b + 2 * w], q[nt][8 * b + 2 * w + 1]);
        }
      } else {
#pragma unroll
        for (int w = 0; w < 4; w += 2)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816(s[nt], a0[w], a1[w], a0[w + 1], a1[w + 1], q[nt][4 * b + w], q[nt][4 * b + w + 1]);
      }
    }
    float kf[2] = {p.scale, p.scale}, vf[2];
    if constexpr (C::quant) {
      kf[0] *= ksc[0];
      kf[1] *= ksc[1];
      vf[0] = vsc[0];
      vf[1] = vsc[1];
    }
    const bool cut = keys_cut(p_lo, p_hi, j0, j0 + 15, p.window, p.sinks);
    if (nj >= 0) load_k(nat);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        s[nt][c] *= kf[c >> 1];
        if (cut && !sees(pos[nt][c & 1], j0 + g + 8 * (c >> 1), p.window, p.sinks)) s[nt][c] = -INFINITY;
      }
    uint32_t pb[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float top[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        top[c] = fmaxf(s[nt][c], s[nt][c + 2]);
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) top[c] = fmaxf(top[c], __shfl_xor_sync(0xffffffffu, top[c], x));
      }
      const bool up0 = top[0] > m[nt][0] + 8.0f, up1 = top[1] > m[nt][1] + 8.0f;
      if (__any_sync(0xffffffffu, up0 || up1)) {
        const float n0 = up0 ? top[0] : m[nt][0], n1 = up1 ? top[1] : m[nt][1];
        const float f0 = up0 ? exp2_approx(m[nt][0] - n0) : 1.0f, f1 = up1 ? exp2_approx(m[nt][1] - n1) : 1.0f;
        m[nt][0] = n0;
        m[nt][1] = n1;
        l[nt][0] *= f0;
        l[nt][1] *= f1;
#pragma unroll
        for (int d = 0; d < DH / 16; ++d) {
          o[nt][d][0] *= f0;
          o[nt][d][1] *= f1;
          o[nt][d][2] *= f0;
          o[nt][d][3] *= f1;
        }
      }
      float w[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float base = m[nt][c & 1] == -INFINITY ? 0.0f : m[nt][c & 1];
        w[c] = exp2_approx(s[nt][c] - base);
        l[nt][c & 1] += w[c];
        // a weight of zero stays zero, whatever scale stands at its place
        if constexpr (C::quant) w[c] = w[c] == 0.0f ? 0.0f : w[c] * vf[c >> 1];
      }
      pb[nt][0] = transpose8(pack_bf16(w[0], w[1]));
      pb[nt][1] = transpose8(pack_bf16(w[2], w[3]));
    }
    if (!C::quant && cut) {
      // a weight of zero times a value that is not finite would be NaN: such values are left out of the product, and
      // added for the rows that do see them; keys past the last that is seen are zeros
      bool odd = false;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool past = j0 + 2 * t + (k & 1) + 8 * (k >> 1) > p_hi;
#pragma unroll
        for (int b = 0; b < C::vb; ++b)
#pragma unroll
          for (int w = 0; w < C::vw; ++w) {
            bool change = false;
            const uint32_t y = finite2(vx[k][b][w], change);
            vx[k][b][w] = past ? 0u : y;
            odd |= change && !past;
          }
      }
      if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
        for (int j = 0; j < min(16, p_hi + 1 - j0); ++j)
#pragma unroll
          for (int d = 0; d < DH / 16; ++d) {
            // row sums of dims 8 (or ve) g + 2 (d % (ve / 2)), + 1 of block d / (ve / 2)
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
    }
#pragma unroll
    for (int b = 0; b < C::vb; ++b) {
#pragma unroll
      for (int w = 0; w < C::vw; ++w) {
        uint32_t x[4][2];  // key, pair of dims (bf16: one)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (C::quant)
            codes_to_bf16<KIND>(vx[k][b][w], x[k][0], x[k][1]);
          else
            x[k][0] = vx[k][b][w];
        }
#pragma unroll
        for (int h = 0; h < (C::quant ? 2 : 1); ++h) {
          const int d = b * (C::ve / 2) + w * (C::quant ? 2 : 1) + h;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816(o[nt][d], prmt(x[0][h], x[1][h], 0x5410), prmt(x[0][h], x[1][h], 0x7632),
                     prmt(x[2][h], x[3][h], 0x5410), prmt(x[2][h], x[3][h], 0x7632), pb[nt][0], pb[nt][1]);
        }
      }
    }
    if (nj >= 0) load_v(nat);
    i = ni;
    j0 = nj;
    at = nat;
  }

  // the four warps' sums
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], x);
      const int r = 2 * t + c + 8 * nt;
      if (g == 0) {
        sm[warp][r] = m[nt][c];
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
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w][r]);
    const float base = top == -INFINITY ? 0.0f : top;
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = exp2_approx(sm[w][r] - base);
      const float4 x = *reinterpret_cast<const float4*>(so + (w * 8 * NT + r) * C::row + d);
      sum = fmaf(f, sl[w][r], sum);
      y.x = fmaf(f, x.x, y.x);
      y.y = fmaf(f, x.y, y.y);
      y.z = fmaf(f, x.z, y.z);
      y.w = fmaf(f, x.w, y.w);
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
    const float inv = 1.0f / sum;
    uint2 w = make_uint2(pack_bf16(gated_by(y.x * inv, x.x), gated_by(y.y * inv, x.y)),
                         pack_bf16(gated_by(y.z * inv, x.z), gated_by(y.w * inv, x.w)));
    if (blank) w = make_uint2(0, 0);
    *reinterpret_cast<uint2*>(p.out + row * p.out_row + head * p.out_head + d) = w;
  }
}

template <int DH, int KIND, int NT>
cudaError_t launch(const AttnParams& p, int* status, cudaStream_t s) {
  using C = RCfg<DH, KIND, NT>;
  const cudaError_t e =
      cudaFuncSetAttribute(attn_rows_kernel<DH, KIND, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)p.c.n_seqs, (unsigned)p.c.n_kv, (unsigned)p.splits);
  attn_rows_kernel<DH, KIND, NT><<<grid, kWarps * 32, C::smem, s>>>(p, status);
  return cudaGetLastError();
}

template <int DH, int KIND>
cudaError_t by_rows(const AttnParams& p, int* status, cudaStream_t s) {
  return p.c.max_q * p.group <= 8 ? launch<DH, KIND, 1>(p, status, s) : launch<DH, KIND, 2>(p, status, s);
}

template <int DH>
cudaError_t by_kind(int kind, const AttnParams& p, int* status, cudaStream_t s) {
  return kind == FAK_KV_BF16   ? by_rows<DH, FAK_KV_BF16>(p, status, s)
         : kind == FAK_KV_E4M3 ? by_rows<DH, FAK_KV_E4M3>(p, status, s)
                               : by_rows<DH, FAK_KV_I8>(p, status, s);
}

}  // namespace

cudaError_t attn_rows_launch(int kind, int dh, const AttnParams& p, int* status, cudaStream_t s) {
  return dh == 64    ? by_kind<64>(kind, p, status, s)
         : dh == 128 ? by_kind<128>(kind, p, status, s)
                     : by_kind<256>(kind, p, status, s);
}
