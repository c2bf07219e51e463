// fak_residual_norm: the norm after a block, its gate and scale, the residual sum and the norm before the next block, in
// one pass: a block of threads holds a row in registers from its loads to its stores.  (Of rows of more than 16,384 values, or
// 8,192 on single values, 1,024 threads of 64 registers hold a part only; the rest goes through local memory: 2,048 rows of 32,768 take
// 195 us, floor 138, with a gate 468, floor 178; of 32,767 on single values 536 and 1,085.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "fak.h"
#include "fak_device.cuh"
#include "kv_device.cuh"

namespace {

struct NormParams {
  void *h, *n;
  const void* y;
  const float *w, *y_w, *gate;
  int64_t h_row, y_row, n_row, gate_row, gate_col;
  int64_t rows;
  float scale, eps, offset;
  int d;
  bool h_bf16, y_bf16, n_bf16, post, sigmoid;
};

// V neighbouring values (1, 2 or 4) of an f32 or bf16 row.
template <int V>
FAK_DEV void get(const void* p, bool bf16, int64_t at, float (&x)[V]) {
  if constexpr (V == 1) {
    x[0] = bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at]) : static_cast<const float*>(p)[at];
  } else if constexpr (V == 2) {
    if (bf16) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p) + at);
      x[0] = __uint_as_float(w << 16);
      x[1] = __uint_as_float(w & 0xffff0000u);
    } else {
      const float2 w = *reinterpret_cast<const float2*>(static_cast<const float*>(p) + at);
      x[0] = w.x;
      x[1] = w.y;
    }
  } else if (bf16) {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + at);
    x[0] = __uint_as_float(w.x << 16);
    x[1] = __uint_as_float(w.x & 0xffff0000u);
    x[2] = __uint_as_float(w.y << 16);
    x[3] = __uint_as_float(w.y & 0xffff0000u);
  } else {
    const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    x[0] = w.x;
    x[1] = w.y;
    x[2] = w.z;
    x[3] = w.w;
  }
}

template <int V>
FAK_DEV void put(void* p, bool bf16, int64_t at, const float (&x)[V]) {
  if constexpr (V == 1) {
    if (bf16)
      static_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(x[0]);
    else
      static_cast<float*>(p)[at] = x[0];
  } else if constexpr (V == 2) {
    if (bf16)
      *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p) + at) = __floats2bfloat162_rn(x[0], x[1]);
    else
      *reinterpret_cast<float2*>(static_cast<float*>(p) + at) = make_float2(x[0], x[1]);
  } else if (bf16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + at) = make_float4(x[0], x[1], x[2], x[3]);
  }
}

// The block's sum, the same in every thread; `red` is used once.
FAK_DEV float block_sum(float x, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  x = lane < warps ? red[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Block r: row r; thread t holds the values V (t + i * threads) .. + V - 1 for i < PER.  A row's loads are all asked for
// before the first is used.
// GATE: with a gate; its registers cost blocks on an SM (16,384 rows of 5,120 without one take 169 us, 177 with its registers).
template <int V, int PER, bool GATE>
__global__ void __launch_bounds__(1024) residual_norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float red[2][32];
  const int64_t row = blockIdx.x;
  float h[PER][V], y[PER][V], gate[GATE ? PER : 1][V];
  bool in[PER];
  int at[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    at[i] = V * (threadIdx.x + i * blockDim.x);
    in[i] = at[i] < p.d;
    if (!in[i]) continue;
    get<V>(p.h, p.h_bf16, row * p.h_row + at[i], h[i]);
    if (p.y) get<V>(p.y, p.y_bf16, row * p.y_row + at[i], y[i]);
    if (GATE && p.gate) {  // (tested again: without it the compiler spreads the loads, 256 us for 16,384 x 5,120 in place of 225)
      if (p.gate_col) {
        get<V>(p.gate, false, row * p.gate_row + at[i], gate[i]);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) gate[i][j] = p.gate[row * p.gate_row];
      }
    }
  }
  if (p.y) {
    float r = 1.0f;
    if (p.post) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (in[i])
#pragma unroll
          for (int j = 0; j < V; ++j) ss = fmaf(y[i][j], y[i][j], ss);
      r = rsqrtf(block_sum(ss, red[0]) / p.d + p.eps);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (!in[i]) continue;
      float w[V];
      const bool gain = p.post && p.y_w;
      if (gain) get<V>(p.y_w, false, at[i], w);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float x = y[i][j];
        if (p.post) x *= r;
        if (gain) x *= p.offset + w[j];
        if (GATE && p.gate) x *= p.sigmoid ? 1.0f / (1.0f + expf(-gate[i][j])) : gate[i][j];
        h[i][j] = fmaf(p.scale, x, h[i][j]);
      }
      put<V>(p.h, p.h_bf16, row * p.h_row + at[i], h[i]);
    }
  }
  if (!p.n) return;
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (in[i])
#pragma unroll
      for (int j = 0; j < V; ++j) ss = fmaf(h[i][j], h[i][j], ss);
  const float r = rsqrtf(block_sum(ss, red[1]) / p.d + p.eps);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (!in[i]) continue;
    float w[V], x[V];
    if (p.w) get<V>(p.w, false, at[i], w);
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = h[i][j] * r * (p.w ? p.offset + w[j] : 1.0f);
    put<V>(p.n, p.n_bf16, row * p.n_row + at[i], x);
  }
}

template <int V, int PER>
cudaError_t launch(const NormParams& p, cudaStream_t s) {
  const int units = (p.d + V - 1) / V;
  const int threads = ((units + PER - 1) / PER + 31) / 32 * 32;
  if (p.gate)
    residual_norm_kernel<V, PER, true><<<(unsigned)p.rows, threads, 0, s>>>(p);
  else
    residual_norm_kernel<V, PER, false><<<(unsigned)p.rows, threads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

extern "C" int fak_residual_norm(const fak_norm_args* a, fak_stream_t stream) {
  if (!a) return FAK_ERR_INVALID_ARG;
  for (const int t : {a->h_type, a->y_type, a->n_type})
    if (t != FAK_ROWS_F32 && t != FAK_ROWS_BF16) return FAK_ERR_INVALID_ARG;
  if (a->gate_kind != FAK_GATE_LINEAR && a->gate_kind != FAK_GATE_SIGMOID) return FAK_ERR_INVALID_ARG;
  if (a->d < 1 || a->d > 32768 || a->rows < 0 || a->rows > 0x7fffffff) return FAK_ERR_SHAPE;
  if (!(a->eps >= 0.0f) || !std::isfinite(a->eps) || !std::isfinite(a->scale) || !std::isfinite(a->gain_offset) || (a->gate_col != 0 && a->gate_col != 1))
    return FAK_ERR_INVALID_ARG;
  if (a->rows && !a->h) return FAK_ERR_INVALID_ARG;
  NormParams p;
  memset(&p, 0, sizeof(p));
  p.h_row = kv_stride(a->h_row, a->rows);
  p.y_row = kv_stride(a->y_row, a->rows);
  p.n_row = kv_stride(a->n_row, a->rows);
  p.gate_row = kv_stride(a->gate_row, a->rows);
  p.gate_col = a->gate_col;
  const bool hb = a->h_type == FAK_ROWS_BF16, yb = a->y_type == FAK_ROWS_BF16, nb = a->n_type == FAK_ROWS_BF16;
  const uintptr_t f32s = (uintptr_t)a->w | (uintptr_t)a->y_w | (uintptr_t)a->gate | (hb ? 0 : (uintptr_t)a->h) |
                         (yb ? 0 : (uintptr_t)a->y) | (nb ? 0 : (uintptr_t)a->n);
  const uintptr_t all = (uintptr_t)a->h | (uintptr_t)a->y | (uintptr_t)a->n;
  if ((f32s & 3) || (all & 1)) return FAK_ERR_ALIGN;
  // rows that are written over one another
  const auto meet = [&](int64_t row) { return a->rows > 1 && row > -(int64_t)a->d && row < a->d; };
  if ((a->h && a->y && meet(a->h_row)) || (a->n && meet(a->n_row))) return FAK_ERR_INVALID_ARG;
  if (a->rows == 0 || (!a->y && !a->n)) return FAK_OK;
  const int st = kv_device(nullptr, nullptr);
  if (st != FAK_OK) return st;
  p.h = a->h;
  p.y = a->y;
  p.n = a->n;
  p.w = a->w;
  p.y_w = a->y_w;
  p.gate = a->y ? a->gate : nullptr;
  p.rows = a->rows;
  p.scale = a->scale;
  p.eps = a->eps;
  p.offset = a->gain_offset;
  p.d = a->d;
  p.h_bf16 = hb;
  p.y_bf16 = yb;
  p.n_bf16 = nb;
  p.post = a->post_norm != 0;
  p.sigmoid = a->gate_kind == FAK_GATE_SIGMOID;
  // As many values at a time as every row of every operand stands on a multiple of: 4, 2 or 1.
  const auto by = [&](int v) {
    const auto rows = [&](const void* at, int64_t row, int elem) { return !at || (!((uintptr_t)at & (v * elem - 1)) && row % v == 0); };
    return a->d % v == 0 && rows(a->h, p.h_row, hb ? 2 : 4) && rows(a->y, p.y_row, yb ? 2 : 4) && rows(a->n, p.n_row, nb ? 2 : 4) &&
           rows(a->w, 0, 4) && rows(a->y_w, 0, 4) && (!p.gate_col || rows(p.gate, p.gate_row, 4));
  };
  // (16,384 rows of 1,500 on multiples of 8 bytes take 60 us by fours, 153 by ones; 3,451 of 7,510 77 us by twos, 100 by ones.)
  // Many rows: 16 values to a thread, so that several blocks are on an SM, by ones from 4,096 values on
  // and without a gate (3,451 of 7,511: 100 us, by 8 to a thread 189; 1,391 of 2,559: 21 and 18); few: the fewest values that
  // 1,024 threads allow, but by twos and ones no fewer than 4 and 8 above 2,048 and 1,024.
  // On both sides of the cut, by fours, 16 to a thread and the fewest: 304 rows of 8,192 8.4 and 9.6 us, of 5,120 6.6 and 6.0; 608 of 8,192
  // 14.4 and 15.7, of 5,120 10.4 and 9.9, of 1,024 3.7 and 2.6; 4,096 of 8,192 72 and 83, of 5,120 46.7 both, of 1,024 12.0 and 11.6.
  const bool many = a->rows >= 608 && a->d >= 1024 && a->d <= 16384;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  if (by(4))
    e = many             ? launch<4, 4>(p, s)
        : a->d <= 4096   ? launch<4, 1>(p, s)
        : a->d <= 8192   ? launch<4, 2>(p, s)
        : a->d <= 16384  ? launch<4, 4>(p, s)
                         : launch<4, 8>(p, s);
  else if (by(2))
    e = many || (a->d > 8192 && a->d <= 16384) ? launch<2, 8>(p, s)
        : a->d <= 2048                         ? launch<2, 1>(p, s)
        : a->d <= 8192                         ? launch<2, 4>(p, s)
                                               : launch<2, 16>(p, s);
  else
    e = a->d <= 1024                              ? launch<1, 1>(p, s)
        : a->d <= (many && !p.gate ? 4096 : 8192) ? launch<1, 8>(p, s)
        : a->d <= 16384                           ? launch<1, 16>(p, s)
                                                  : launch<1, 32>(p, s);
  return fak_cuda_status(e);
}
