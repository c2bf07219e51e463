// The paged KV cache's writes and reads: fak_kv_append (RMSNorm and RoPE of new
// rows, keys and values quantised into the cache, queries to bf16) and
// fak_kv_read (cached vectors back as rows).
//
// Both only move bytes.  A warp owns one head's vector: each lane holds dh / 32
// neighbouring values, so a vector's sum of squares or largest magnitude is one
// warp reduction, and the rotary partner (i, i + rot / 2) is a whole number of
// lanes away because rot is a multiple of 16.
//
// Bound by memory where rows are many: 8 chunks of 1,024 f32 rows of 24 + 4 + 4 heads of 256 written in 72 us as bf16,
// 5.6 TB/s, and in 83 us as e4m3, 4.6; 16 sequences of up to 8,192 int8 vectors of 4 + 4 heads read in 63 us, 6.2 TB/s.
// Every load of a warp is asked for before the first is used, and a block lives for one row: with blocks of two vectors
// a warp, or registers for more blocks, writes took 1 to 17% longer.  Few rows: bound by the launch.
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

constexpr int kKvThreads = 256;
constexpr int kKvWarps = kKvThreads / 32;

__device__ int g_kv_status;

FAK_DEV void kv_record() { atomicCAS(&g_kv_status, 0, FAK_ERR_DEVICE); }

// N neighbouring values of a row (16-byte aligned vectors; N = 2, 4, 8).
template <int N>
FAK_DEV void load_vals(const float* p, float (&x)[N]) {
  if constexpr (N == 2) {
    const float2 a = *reinterpret_cast<const float2*>(p);
    x[0] = a.x;
    x[1] = a.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 a = *reinterpret_cast<const float4*>(p + i);
      x[i] = a.x;
      x[i + 1] = a.y;
      x[i + 2] = a.z;
      x[i + 3] = a.w;
    }
  }
}

// N bytes * E (a power of two up to 32) as words.
template <int BYTES>
FAK_DEV void load_bytes(const void* p, uint32_t* w) {
  if constexpr (BYTES == 2) {
    w[0] = *reinterpret_cast<const uint16_t*>(p);
  } else if constexpr (BYTES == 4) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (BYTES == 8) {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    w[0] = a.x;
    w[1] = a.y;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    w[0] = a.x;
    w[1] = a.y;
    w[2] = a.z;
    w[3] = a.w;
  }
}

template <int BYTES>
FAK_DEV void store_bytes(void* p, const uint32_t* w) {
  if constexpr (BYTES == 2)
    *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
  else if constexpr (BYTES == 4)
    *reinterpret_cast<uint32_t*>(p) = w[0];
  else if constexpr (BYTES == 8)
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

FAK_DEV float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
FAK_DEV float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <int N>
FAK_DEV void load_vals(const __nv_bfloat16* p, float (&x)[N]) {
  uint32_t w[(N + 1) / 2];
  load_bytes<2 * N>(p, w);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}

template <int N>
FAK_DEV void store_bf16(void* p, const float (&x)[N]) {
  uint32_t w[(N + 1) / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&a);
  }
  store_bytes<2 * N>(p, w);
}

template <int KIND>
constexpr int kCodeBytes = KIND == FAK_KV_BF16 ? 2 : 1;

struct AppendParams {
  KvView c;
  const void *q, *k, *v;
  int64_t q_row, q_head, k_row, k_head, v_row, v_head;
  const float *qw, *kw;
  const uint64_t* rope;
  __nv_bfloat16* q_out;
  float eps;
  int nq, rot;
};

// Quantises a vector held by the warp and stores its codes and scale at vector index `at`.
template <int N, int KIND>
FAK_DEV void put_vector(uint8_t* codes, float* scales, int64_t at, const float (&x)[N], int lane) {
  uint8_t* dst = codes + (at * (32 * N) + lane * N) * kCodeBytes<KIND>;
  if constexpr (KIND == FAK_KV_BF16) {
    store_bf16<N>(dst, x);
  } else {
    // the largest magnitude, as bits: their order is the magnitudes', and NaN is above infinity
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    m = __reduce_max_sync(0xffffffffu, m);
    constexpr float top = KIND == FAK_KV_E4M3 ? 448.0f : 127.0f;
    const float a = __uint_as_float(m);
    const bool zero = m < 0x0d800000u, lost = m >= 0x7f800000u;  // below 2^-100; an infinity or NaN
    const float inv = zero || lost ? 0.0f : top * __frcp_rn(a);  // (as PyTorch divides a number by a tensor: the same codes)
    uint32_t w[(N + 3) / 4] = {};
    if (!lost) {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        uint32_t two;
        if constexpr (KIND == FAK_KV_E4M3) {
          two = __nv_cvt_float2_to_fp8x2(make_float2(x[i] * inv, x[i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
        } else {
          const int lo = __float2int_rn(x[i] * inv), hi = __float2int_rn(x[i + 1] * inv);
          two = (uint32_t)(lo & 0xff) | ((uint32_t)(hi & 0xff) << 8);
        }
        w[i / 4] |= two << (8 * (i % 4));
      }
    }
    store_bytes<N>(dst, w);
    if (lane == 0) scales[at] = lost ? __uint_as_float(0x7fffffffu) : (zero ? 0.0f : a / top);
  }
}

// Blocks on an SM, as many as the registers of a row's own path leave (0: as the compiler has it): the search that only
// bad numbers need must not take more.  (Left alone it takes 104 where 80 do at dh 256, and 8 ragged chunks of 1,024 rows
// 60 us, not 48; bf16 at dh 128 76.7 us, not 72.5; 8-bit at dh 64 is faster left alone, 51.4 us and 53.8.)
constexpr int append_blocks(int dh, int kind, int v, int bytes) {
  if (v == 1) return 0;
  if (dh == 256) return 3;
  if (dh == 128) return kind == FAK_KV_BF16 && bytes == 4 ? 5 : 4;
  return kind == FAK_KV_BF16 ? 7 : 0;
}

// Block (x, y): row x, vectors [y * 8 V, +8 V) of its nq queries, n_kv keys and n_kv values, V to a
// warp with all their loads in flight before the first is used.  The row's rotary sines and cosines
// are made once for the block, from 64-bit fractions of a turn: position * frequency wraps at whole
// turns by itself, so the angle is as good at position 2^30 as at 1.
template <int DH, int KIND, int V, typename T>
__global__ void __launch_bounds__(kKvThreads, append_blocks(DH, KIND, V, sizeof(T)))
    kv_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int N = DH / 32;
  __shared__ float2 cs[128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;
  const int total = p.nq + 2 * p.c.n_kv;
  const int first = (blockIdx.y * kKvWarps + warp) * V;
  float x[V][N];
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int h = first + u;
    if (h >= total) continue;
    const T* src = h < p.nq ? static_cast<const T*>(p.q) + row * p.q_row + h * p.q_head
                   : h < p.nq + p.c.n_kv
                       ? static_cast<const T*>(p.k) + row * p.k_row + (h - p.nq) * p.k_head
                       : static_cast<const T*>(p.v) + row * p.v_row + (h - p.nq - p.c.n_kv) * p.v_head;
    load_vals<N>(src + lane * N, x[u]);
  }
  int s;
  KvSeq q = kv_locate(p.c, row, lane, s);
  if (!__any_sync(0xffffffffu, kv_has(q, row))) {  // (all lanes or none)
    bool bad;
    q = kv_locate_all(p.c, row, lane, s, bad);
    if (bad && threadIdx.x == 0) kv_record();
    if (!q.ok) return;  // rows of no sequence
  }
  const int pos = q.len - (q.r1 - (int)row);
  if (pos < 0) return;  // padding
  const int half = p.rot / 2;
  if (threadIdx.x < half) {
    // the nearest quarter of a turn goes first, so that f32 rounds an eighth at most: 2^-27 half turns, and small sines
    // and cosines are as good at every quarter as at none
    const uint64_t turn = p.rope[threadIdx.x] * (uint64_t)pos;
    const uint64_t quarter = (turn + (1ull << 61)) >> 62;
    float sn, co;
    sincospif((float)(long long)(turn - (quarter << 62)) * 1.0842021724855044e-19f, &sn, &co);  // 2^-63: in half turns
    const float c = quarter & 1 ? -sn : co, s = quarter & 1 ? co : sn;
    cs[threadIdx.x] = quarter & 2 ? make_float2(-c, -s) : make_float2(c, s);
  }
  if (half) __syncthreads();
  // this lane's sines and cosines, and where its rotary partners are; the gains stay while the vectors are of one kind
  const int span = half / N;  // lanes of one half; N divides rot / 2
  const bool in = lane < 2 * span, low = lane < span;
  const int other = in ? (low ? lane + span : lane - span) : lane;
  float co[N], si[N], gain[N];
  if (in) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 c = cs[(low ? lane : other) * N + i];
      co[i] = c.x;
      si[i] = low ? -c.y : c.y;
    }
  }
  const float* held = nullptr;
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int h = first + u;
    if (h >= total) break;
    const bool isq = h < p.nq, isk = !isq && h < p.nq + p.c.n_kv;
    const float* w = isq ? p.qw : isk ? p.kw : nullptr;
    if (w) {
      if (w != held) load_vals<N>(w + lane * N, gain);
      held = w;
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) ss = fmaf(x[u][i], x[u][i], ss);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      // (rsqrtf is off by 2 units in the last place at most; a square root and a division take 40 instructions)
      const float r = rsqrtf(fmaf(ss, 1.0f / DH, p.eps));
#pragma unroll
      for (int i = 0; i < N; ++i) x[u][i] *= r * gain[i];
    }
    if (half && (isq || isk)) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float y = __shfl_sync(0xffffffffu, x[u][i], other);
        if (in) x[u][i] = fmaf(y, si[i], x[u][i] * co[i]);
      }
    }
    if (isq) {
      store_bf16<N>(p.q_out + (row * p.nq + h) * DH + lane * N, x[u]);
      continue;
    }
    const int g = isk ? h - p.nq : h - p.nq - p.c.n_kv;
    const int64_t at = kv_place(p.c, s, pos, g);
    if (at < 0) {
      if (lane == 0) kv_record();
      continue;
    }
    put_vector<N, KIND>(isk ? p.c.k : p.c.v, isk ? p.c.ks : p.c.vs, at, x[u], lane);
  }
}

struct ReadParams {
  KvView c;
  void *k, *v;
};

constexpr int kReadVec = 8;  // vectors of one row a warp reads at a time

// Warp (x, y): row x, vectors [8 y, +8) of its n_kv keys and n_kv values, all loads in flight at once.
template <int DH, int KIND, typename T>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const __grid_constant__ ReadParams p) {
  constexpr int N = DH / 32, E = kCodeBytes<KIND>;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kKvWarps + (threadIdx.x >> 5);
  if (row >= p.c.rows) return;
  int s;
  KvSeq q = kv_locate(p.c, row, lane, s);
  if (!__any_sync(0xffffffffu, kv_has(q, row))) {  // (all lanes or none)
    bool bad;
    q = kv_locate_all(p.c, row, lane, s, bad);
    if (bad && lane == 0) kv_record();
    if (!q.ok) return;
  }
  const int pos = q.len - (q.r1 - (int)row);
  int64_t base = 0;
  if (pos >= 0) {
    base = kv_place(p.c, s, pos, 0);
    if (base < 0) {
      if (lane == 0) kv_record();
      base = -1 - base;
    }
  }
  const int first = blockIdx.y * kReadVec, total = 2 * p.c.n_kv;
  uint32_t w[kReadVec][(N * E + 3) / 4];
  float sc[kReadVec];
#pragma unroll
  for (int u = 0; u < kReadVec; ++u) {
    const int h = first + u;
    if (h >= total || pos < 0) continue;
    const bool key = h < p.c.n_kv;
    const int64_t at = base + ((int64_t)(key ? h : h - p.c.n_kv) << p.c.page_shift);
    load_bytes<N * E>((key ? p.c.k : p.c.v) + (at * DH + lane * N) * E, w[u]);
    if constexpr (KIND != FAK_KV_BF16) sc[u] = (key ? p.c.ks : p.c.vs)[at];
  }
#pragma unroll
  for (int u = 0; u < kReadVec; ++u) {
    const int h = first + u;
    if (h >= total) break;
    const bool key = h < p.c.n_kv;
    T* out = static_cast<T*>(key ? p.k : p.v);
    if (!out) continue;
    float x[N];
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      if (pos < 0) {
        x[i] = x[i + 1] = 0.0f;
      } else if constexpr (KIND == FAK_KV_BF16) {
        x[i] = bf16_lo(w[u][i / 2]);
        x[i + 1] = bf16_hi(w[u][i / 2]);
      } else {
        const uint32_t two = (w[u][i / 4] >> (8 * (i % 4))) & 0xffffu;
        if constexpr (KIND == FAK_KV_E4M3) {
          const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
          x[i] = half_bits_to_float(hr.x) * sc[u];
          x[i + 1] = half_bits_to_float(hr.y) * sc[u];
        } else {
          x[i] = (float)(int8_t)(two & 0xff) * sc[u];
          x[i + 1] = (float)(int8_t)(two >> 8) * sc[u];
        }
      }
    }
    T* dst = out + (row * p.c.n_kv + (key ? h : h - p.c.n_kv)) * DH + lane * N;
    if constexpr (sizeof(T) == 2) {
      store_bf16<N>(dst, x);
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 2) *reinterpret_cast<float2*>(dst + i) = make_float2(x[i], x[i + 1]);
    }
  }
}

template <int DH, int KIND, typename T>
cudaError_t launch_append(const AppendParams& p, int sms, cudaStream_t s) {
  const int total = p.nq + 2 * p.c.n_kv;
  // four vectors to a warp share the row's sines and keep 4 KB in flight; with fewer rows than
  // SMs one vector to a warp spreads a row over more SMs instead
  if (p.c.rows < sms) {
    const dim3 grid((unsigned)p.c.rows, (unsigned)((total + kKvWarps - 1) / kKvWarps));
    kv_append_kernel<DH, KIND, 1, T><<<grid, kKvThreads, 0, s>>>(p);
  } else {
    const dim3 grid((unsigned)p.c.rows, (unsigned)((total + 4 * kKvWarps - 1) / (4 * kKvWarps)));
    kv_append_kernel<DH, KIND, 4, T><<<grid, kKvThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

template <int DH, typename T>
cudaError_t append_kind(int kind, const AppendParams& p, int sms, cudaStream_t s) {
  return kind == FAK_KV_BF16   ? launch_append<DH, FAK_KV_BF16, T>(p, sms, s)
         : kind == FAK_KV_E4M3 ? launch_append<DH, FAK_KV_E4M3, T>(p, sms, s)
                               : launch_append<DH, FAK_KV_I8, T>(p, sms, s);
}

template <int DH, typename T>
cudaError_t launch_read(int kind, const ReadParams& p, cudaStream_t s) {
  const dim3 grid((unsigned)((p.c.rows + kKvWarps - 1) / kKvWarps),
                  (unsigned)((2 * p.c.n_kv + kReadVec - 1) / kReadVec));
  if (kind == FAK_KV_BF16)
    kv_read_kernel<DH, FAK_KV_BF16, T><<<grid, kKvThreads, 0, s>>>(p);
  else if (kind == FAK_KV_E4M3)
    kv_read_kernel<DH, FAK_KV_E4M3, T><<<grid, kKvThreads, 0, s>>>(p);
  else
    kv_read_kernel<DH, FAK_KV_I8, T><<<grid, kKvThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

extern "C" int fak_rope_table(int rot, double theta, uint64_t* table) {
  if (!table) return FAK_ERR_INVALID_ARG;
  if (rot < 2 || rot > 256 || rot % 2) return FAK_ERR_SHAPE;
  if (!(theta >= 1.0) || !std::isfinite(theta)) return FAK_ERR_INVALID_ARG;
  // at most 1 / (2 pi) of a turn per position; 53 bits of it, so position p is off by p 2^-55 turns
  for (int i = 0; i < rot / 2; ++i)
    table[i] = (uint64_t)std::llround(std::pow(theta, -2.0 * i / rot) * 0.15915494309189535 * 4611686018427387904.0)
               << 2;
  return FAK_OK;
}

extern "C" int fak_kv_append(const fak_kv_cache* cache, const fak_kv_batch* batch, const fak_kv_rows* r,
                             fak_stream_t stream) {
  AppendParams p;
  memset(&p, 0, sizeof(p));
  int st = kv_view(cache, batch, &p.c);
  if (st != FAK_OK) return st;
  if (!r || (r->type != FAK_ROWS_F32 && r->type != FAK_ROWS_BF16)) return FAK_ERR_INVALID_ARG;
  if (r->nq < 0 || r->rows < 0 || r->rows > 0x7fffffff || r->rot < 0 || r->rot % 16 || r->rot > cache->dh ||
      (int64_t)r->nq + 2 * cache->n_kv > 65535 * kKvWarps)
    return FAK_ERR_SHAPE;
  if (r->rows && (!r->k || !r->v || (r->nq && (!r->q || !r->q_out)))) return FAK_ERR_INVALID_ARG;
  if (r->rot && !r->rope) return FAK_ERR_INVALID_ARG;
  if (!(r->eps >= 0.0f)) return FAK_ERR_INVALID_ARG;
  // vectors on 16-byte boundaries: 4 f32 or 8 bf16 elements
  const int64_t m = r->type == FAK_ROWS_F32 ? 3 : 7;
  p.q_row = kv_stride(r->q_row, r->rows);
  p.q_head = kv_stride(r->q_head, r->nq);
  p.k_row = kv_stride(r->k_row, r->rows);
  p.k_head = kv_stride(r->k_head, cache->n_kv);
  p.v_row = kv_stride(r->v_row, r->rows);
  p.v_head = kv_stride(r->v_head, cache->n_kv);
  const int64_t strides = p.k_row | p.k_head | p.v_row | p.v_head | (r->nq ? p.q_row | p.q_head : 0);
  const uintptr_t bits = (uintptr_t)r->k | (uintptr_t)r->v | (uintptr_t)r->q_norm_w | (uintptr_t)r->k_norm_w |
                         (r->nq ? (uintptr_t)r->q | (uintptr_t)r->q_out : 0);
  if ((strides & m) || (bits & 15) || ((uintptr_t)r->rope & 7)) return FAK_ERR_ALIGN;
  if (r->rows == 0 || batch->n_seqs == 0) return FAK_OK;
  int sms = 0;
  if ((st = kv_device(nullptr, &sms)) != FAK_OK) return st;
  p.c.rows = r->rows;
  p.q = r->q;
  p.k = r->k;
  p.v = r->v;
  p.qw = r->q_norm_w;
  p.kw = r->k_norm_w;
  p.rope = r->rope;
  p.q_out = static_cast<__nv_bfloat16*>(r->q_out);
  p.eps = r->eps;
  p.nq = r->nq;
  p.rot = r->rot;
  cudaStream_t s = (cudaStream_t)stream;
  const int kind = cache->kind;
  cudaError_t e;
  if (r->type == FAK_ROWS_F32)
    e = cache->dh == 64    ? append_kind<64, float>(kind, p, sms, s)
        : cache->dh == 128 ? append_kind<128, float>(kind, p, sms, s)
                           : append_kind<256, float>(kind, p, sms, s);
  else
    e = cache->dh == 64    ? append_kind<64, __nv_bfloat16>(kind, p, sms, s)
        : cache->dh == 128 ? append_kind<128, __nv_bfloat16>(kind, p, sms, s)
                           : append_kind<256, __nv_bfloat16>(kind, p, sms, s);
  return fak_cuda_status(e);
}

extern "C" int fak_kv_read(const fak_kv_cache* cache, const fak_kv_batch* batch, int64_t rows, int type, void* k_out,
                           void* v_out, fak_stream_t stream) {
  ReadParams p;
  memset(&p, 0, sizeof(p));
  int st = kv_view(cache, batch, &p.c);
  if (st != FAK_OK) return st;
  if ((type != FAK_ROWS_F32 && type != FAK_ROWS_BF16) || (rows && !k_out && !v_out)) return FAK_ERR_INVALID_ARG;
  if (rows < 0 || rows > 0x7fffffff || cache->n_kv > 65535 * (kReadVec / 2)) return FAK_ERR_SHAPE;
  if (((uintptr_t)k_out | (uintptr_t)v_out) & 15) return FAK_ERR_ALIGN;
  if (rows == 0 || batch->n_seqs == 0) return FAK_OK;
  if ((st = kv_device(nullptr, nullptr)) != FAK_OK) return st;
  p.c.rows = rows;
  p.k = k_out;
  p.v = v_out;
  cudaStream_t s = (cudaStream_t)stream;
  const int kind = cache->kind;
  cudaError_t e;
  if (type == FAK_ROWS_F32)
    e = cache->dh == 64    ? launch_read<64, float>(kind, p, s)
        : cache->dh == 128 ? launch_read<128, float>(kind, p, s)
                           : launch_read<256, float>(kind, p, s);
  else
    e = cache->dh == 64    ? launch_read<64, __nv_bfloat16>(kind, p, s)
        : cache->dh == 128 ? launch_read<128, __nv_bfloat16>(kind, p, s)
                           : launch_read<256, __nv_bfloat16>(kind, p, s);
  return fak_cuda_status(e);
}

int fak_kv_take_status() {
  int v = 0, zero = 0;
  const cudaError_t e = cudaMemcpyFromSymbol(&v, g_kv_status, sizeof(int));
  if (e != cudaSuccess) return fak_cuda_status(e);
  cudaMemcpyToSymbol(g_kv_status, &zero, sizeof(int));
  return v;
}
