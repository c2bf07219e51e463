// Softmax attention of new rows over the paged KV cache (fak_paged_attn).
//
// One warp per (row, query head): each lane holds dh / 32 neighbouring dims of q and
// of the output, a score is one warp sum, and the softmax runs along the keys with
// the running maximum and sum.  Only positions that the row sees are read.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "fak.h"
#include "fak_device.cuh"
#include "kv_device.cuh"

namespace {

__device__ int g_attn_status;

struct AttnParams {
  KvView c;
  const __nv_bfloat16* q;
  const float* gate;
  __nv_bfloat16* out;
  int64_t q_row, q_head, gate_row, gate_head, out_row, out_head;
  float scale;
  int nq, window, sinks;
};

template <int N, int KIND>
FAK_DEV void load_vector(const uint8_t* codes, const float* scales, int64_t at, int lane, float (&x)[N]) {
  if constexpr (KIND == FAK_KV_BF16) {
    const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(codes) + at * (32 * N) + lane * N;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __bfloat162float(p[i]);
  } else {
    const uint8_t* p = codes + at * (32 * N) + lane * N;
    const float s = scales[at];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (KIND == FAK_KV_E4M3)
        x[i] = half_bits_to_float(__nv_cvt_fp8_to_halfraw(p[i], __NV_E4M3).x) * s;
      else
        x[i] = (float)(int8_t)p[i] * s;
    }
  }
}

template <int DH, int KIND>
__global__ void __launch_bounds__(256) attn_kernel(const __grid_constant__ AttnParams p) {
  constexpr int N = DH / 32;
  const int lane = threadIdx.x & 31, h = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int64_t row = blockIdx.x;
  if (h >= p.nq) return;
  const int s = kv_find_seq(p.c, row, lane);
  const KvSeq sq = kv_seq(p.c, s);
  if (!sq.ok) {
    if (lane == 0) atomicCAS(&g_attn_status, 0, FAK_ERR_DEVICE);
    return;
  }
  if (row < sq.r0 || row >= sq.r1) return;
  const int pos = sq.len - (sq.r1 - (int)row), g = h / (p.nq / p.c.n_kv);
  float q[N], o[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    q[i] = __bfloat162float(p.q[row * p.q_row + h * p.q_head + lane * N + i]);
    o[i] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  const int low = p.window ? max(0, pos - p.window + 1) : 0;
  for (int j = min(p.sinks, low) ? 0 : low; j <= pos; ++j) {
    if (j < low && j >= p.sinks) j = low;
    int64_t at = kv_place(p.c, s, j, g);
    if (at < 0) {
      if (lane == 0) atomicCAS(&g_attn_status, 0, FAK_ERR_DEVICE);
      at = -1 - at;
    }
    float x[N], d = 0.0f;
    load_vector<N, KIND>(p.c.k, p.c.ks, at, lane, x);
#pragma unroll
    for (int i = 0; i < N; ++i) d = fmaf(q[i], x[i], d);
#pragma unroll
    for (int b = 16; b > 0; b >>= 1) d += __shfl_xor_sync(0xffffffffu, d, b);
    d *= p.scale;
    const float top = fmaxf(m, d), base = top == -INFINITY ? 0.0f : top;  // all scores so far -inf: weights 0
    const float was = expf(m - base), w = expf(d - base);
    l = l * was + w;
    load_vector<N, KIND>(p.c.v, p.c.vs, at, lane, x);
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = fmaf(w, x[i], o[i] * was);
    m = top;
  }
  const float r = pos < 0 ? 0.0f : 1.0f / l;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float y = o[i] * r;
    if (p.gate) y = y / (1.0f + expf(-p.gate[row * p.gate_row + h * p.gate_head + lane * N + i]));
    if (pos < 0) y = 0.0f;
    p.out[row * p.out_row + h * p.out_head + lane * N + i] = __float2bfloat16_rn(y);
  }
}

template <int DH>
cudaError_t launch_attn(int kind, const AttnParams& p, cudaStream_t s) {
  const dim3 grid((unsigned)p.c.rows, (unsigned)((p.nq + 7) / 8));
  if (kind == FAK_KV_BF16)
    attn_kernel<DH, FAK_KV_BF16><<<grid, 256, 0, s>>>(p);
  else if (kind == FAK_KV_E4M3)
    attn_kernel<DH, FAK_KV_E4M3><<<grid, 256, 0, s>>>(p);
  else
    attn_kernel<DH, FAK_KV_I8><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

int attn_shape(const fak_kv_cache* c, const fak_attn_args* a) {
  if (a->window < 0 || a->sinks < 0 || !(a->scale > 0.0f) || !std::isfinite(a->scale)) return FAK_ERR_INVALID_ARG;
  if (a->nq < 1 || a->nq % c->n_kv || a->nq / c->n_kv > 128 || a->rows < 0 || a->rows > 0x7fffffff || a->max_q < 0 ||
      a->max_kv < 0 || a->max_kv > 1 << 30 || a->nq > 65535)
    return FAK_ERR_SHAPE;
  return FAK_OK;
}

}  // namespace

extern "C" size_t fak_paged_attn_workspace_bytes(const fak_kv_cache* cache, const fak_kv_batch* batch,
                                                 const fak_attn_args* a) {
  if (!cache || !batch || !a) return 0;
  return 0;
}

extern "C" int fak_paged_attn(const fak_kv_cache* cache, const fak_kv_batch* batch, const fak_attn_args* a,
                              fak_stream_t stream) {
  AttnParams p;
  memset(&p, 0, sizeof(p));
  int st = kv_view(cache, batch, &p.c);
  if (st != FAK_OK) return st;
  if (!a || !a->q || !a->out) return FAK_ERR_INVALID_ARG;
  if ((st = attn_shape(cache, a)) != FAK_OK) return st;
  if ((((uintptr_t)a->q | (uintptr_t)a->out | (uintptr_t)a->gate) & 15) ||
      ((a->q_row | a->q_head | a->out_row | a->out_head) & 7) || (a->gate && ((a->gate_row | a->gate_head) & 3)) ||
      ((uintptr_t)a->workspace & 255))
    return FAK_ERR_ALIGN;
  const size_t need = fak_paged_attn_workspace_bytes(cache, batch, a);
  if (need && !a->workspace) return FAK_ERR_INVALID_ARG;
  if (a->workspace_bytes < need) return FAK_ERR_SHAPE;
  if (a->rows == 0 || batch->n_seqs == 0) return FAK_OK;
  int sms = 0;
  if ((st = kv_device(&sms)) != FAK_OK) return st;
  p.c.rows = a->rows;
  p.c.max_q = a->max_q;
  p.c.max_kv = a->max_kv;
  p.q = static_cast<const __nv_bfloat16*>(a->q);
  p.gate = a->gate;
  p.out = static_cast<__nv_bfloat16*>(a->out);
  p.q_row = a->q_row;
  p.q_head = a->q_head;
  p.gate_row = a->gate_row;
  p.gate_head = a->gate_head;
  p.out_row = a->out_row;
  p.out_head = a->out_head;
  p.scale = a->scale;
  p.nq = a->nq;
  p.window = a->window;
  p.sinks = a->window ? a->sinks : 0;
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = cache->dh == 64    ? launch_attn<64>(cache->kind, p, s)
                        : cache->dh == 128 ? launch_attn<128>(cache->kind, p, s)
                                           : launch_attn<256>(cache->kind, p, s);
  return fak_cuda_status(e);
}

int fak_attn_take_status() {
  int v = 0, zero = 0;
  const cudaError_t e = cudaMemcpyFromSymbol(&v, g_attn_status, sizeof(int));
  if (e != cudaSuccess) return fak_cuda_status(e);
  cudaMemcpyToSymbol(g_attn_status, &zero, sizeof(int));
  return v;
}
