// The Gated DeltaNet layers on ragged batches: the short causal convolution with what stands between it and the linear
// attention (fak_gdn_conv), and the gated delta rule row by row (fak_gdn_attn).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "fak.h"
#include "fak_device.cuh"
#include "gdn_device.cuh"
#include "kv_device.cuh"

namespace {

__device__ int g_gdn_status;

constexpr unsigned long long kGdnTimeout = 2000000000ull;
std::atomic<unsigned long long> g_gdn_timeout{kGdnTimeout};
std::atomic<int> g_gdn_unreachable{0};

FAK_DEV void gdn_record() { atomicCAS(&g_gdn_status, 0, FAK_ERR_DEVICE); }

// ------------------------------------------------------------------ the convolution
constexpr int kConvThreads = 256;
constexpr int kConvWarps = kConvThreads / 32;

struct ConvParams {
  KvView c;
  const void *x, *b, *a;
  int64_t x_row, b_row, a_row;
  const float *conv_w, *a_log, *dt_bias;
  float* state;
  __half *q, *k;
  __nv_bfloat16* v;
  float *g, *beta;
  float eps;
  int nk, nv;
};

FAK_DEV float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
FAK_DEV float4 load4(const __nv_bfloat16* p) { return gdn_bf16x4(*reinterpret_cast<const uint2*>(p)); }
FAK_DEV float load1(const float* p) { return *p; }
FAK_DEV float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
template <bool WIDE, typename T>
FAK_DEV float4 load_row4(const T* p) {
  if constexpr (WIDE) return load4(p);
  return make_float4(load1(p), load1(p + 1), load1(p + 2), load1(p + 3));
}

// Block (x, y): rows [R x, +R), heads [8 y, +8) of the nk queries, nk keys and nv values, one to a warp (a lane has four
// neighbouring channels, so that a head's sum of squares is one warp's), and behind them one for the rows' decays and
// strengths.  A block takes the rows of its range but those that stand second or third in a sequence that began before
// it; of a sequence that begins in it, it takes the first three rows even behind its range.  So a sequence's old state
// is read, and its new one written, by one block alone, the one that has its first row, and no other block waits.
template <int R, bool WIDE, typename T>
__global__ void __launch_bounds__(kConvThreads, R == 8 ? 3 : 4) gdn_conv_kernel(const __grid_constant__ ConvParams p) {
  const int lane = threadIdx.x & 31;
  const int head = blockIdx.y * kConvWarps + (threadIdx.x >> 5);
  const int heads = 2 * p.nk + p.nv;
  if (head > heads) return;
  const int64_t base = (int64_t)blockIdx.x * R;
  const int64_t end = min(base + R, p.c.rows);
  if (head == heads) {
    // numbers out of range are recorded even where no row is looked for with them (by the first block, for all sequences)
    if (base == 0) {
#pragma unroll 4
      for (int s = lane; s < p.c.n_seqs; s += 32)
        if (!gdn_seq(p.c, kv_seq(p.c, s), s).ok) gdn_record();
    }
    for (int64_t row = base; row < end; ++row) {
      int s;
      KvSeq q = kv_locate(p.c, row, lane, s);
      if (!__any_sync(0xffffffffu, kv_has(q, row))) {
        bool bad;
        q = kv_locate_all(p.c, row, lane, s, bad);
        if (!q.ok) continue;
      }
      const GdnSeq d = gdn_seq(p.c, q, s);
      if (!d.ok || row < d.first) continue;
      for (int h = lane; h < p.nv; h += 32) {
        const float b = load1(static_cast<const T*>(p.b) + row * p.b_row + h);
        const float u = load1(static_cast<const T*>(p.a) + row * p.a_row + h) + p.dt_bias[h];
        // softplus(u) = max(u, 0) + log(1 + exp(-|u|)): exp never overflows
        p.g[row * p.nv + h] = -expf(p.a_log[h]) * (fmaxf(u, 0.0f) + log1pf(expf(-fabsf(u))));
        p.beta[row * p.nv + h] = 1.0f / (1.0f + expf(-b));
      }
    }
    return;
  }
  const int64_t chans = (int64_t)heads * kGdnDim;
  const int64_t ch = (int64_t)head * kGdnDim + 4 * lane;
  const T* x = static_cast<const T*>(p.x) + ch;
  // the rows from three before the range on, all asked for at once (a single row: itself, which every way needs)
  constexpr int kIn = R == 1 ? 1 : R + 3;
  const bool inside = R == 1 || (base >= 3 && base + R <= p.c.rows);
  float4 in[kIn];
  if (inside) {
    const T* at = x + (R == 1 ? base : base - 3) * p.x_row;
#pragma unroll
    for (int i = 0; i < kIn; ++i, at += p.x_row) in[i] = load_row4<WIDE>(at);
  }
  float4 w[4];  // of the lane's four channels: the taps, oldest first
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = load4(p.conv_w + (ch + i) * 4);

  auto taps = [&](const float4& x0, const float4& x1, const float4& x2, const float4& x3) {
    float4 c;
    c.x = gdn_silu(fmaf(w[0].w, x3.x, fmaf(w[0].z, x2.x, fmaf(w[0].y, x1.x, w[0].x * x0.x))));
    c.y = gdn_silu(fmaf(w[1].w, x3.y, fmaf(w[1].z, x2.y, fmaf(w[1].y, x1.y, w[1].x * x0.y))));
    c.z = gdn_silu(fmaf(w[2].w, x3.z, fmaf(w[2].z, x2.z, fmaf(w[2].y, x1.z, w[2].x * x0.z))));
    c.w = gdn_silu(fmaf(w[3].w, x3.w, fmaf(w[3].z, x2.w, fmaf(w[3].y, x1.w, w[3].x * x0.w))));
    return c;
  };
  const bool value = head >= 2 * p.nk, key = head >= p.nk;
  __half* unit = (key ? p.k : p.q) + (int64_t)(head - (key ? p.nk : 0)) * kGdnDim + 4 * lane;  // of row 0, of a query or key
  auto put_unit = [&](int64_t row, const float4& c, float r) {
    const __half2 a = __floats2half2_rn(c.x * r, c.y * r), b = __floats2half2_rn(c.z * r, c.w * r);
    *reinterpret_cast<uint2*>(unit + row * p.nk * kGdnDim) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  };
  auto put_value = [&](int64_t row, const float4& c) {
    gdn_put4(p.v, true, (row * p.nv + head - 2 * p.nk) * kGdnDim + 4 * lane, c);
  };
  auto emit = [&](int64_t row, const float4& x0, const float4& x1, const float4& x2, const float4& x3) {
    const float4 c = taps(x0, x1, x2, x3);
    if (value)
      put_value(row, c);
    else
      put_unit(row, c, rsqrtf(gdn_warp_sum(fmaf(c.x, c.x, fmaf(c.y, c.y, fmaf(c.z, c.z, c.w * c.w)))) + p.eps));
  };

  if constexpr (R == 8) {
    // rows in the midst of a sequence: all of them together
    int s;
    const KvSeq q = kv_locate(p.c, base, lane, s);
    const GdnSeq e = gdn_seq(p.c, q, s);
    if (__all_sync(0xffffffffu, inside && e.ok && base >= e.first + 3 && base + R <= e.r1)) {
      float4 c[R];
#pragma unroll
      for (int i = 0; i < R; ++i) c[i] = taps(in[i], in[i + 1], in[i + 2], in[i + 3]);
      if (value) {
#pragma unroll
        for (int i = 0; i < R; ++i) put_value(base + i, c[i]);
        return;
      }
      // the rows' sums over the lanes: lanes 16, 8 and 4 apart each keep half of their rows and add the other's; then the
      // four lanes that have the same row
      float ss[R];
#pragma unroll
      for (int i = 0; i < R; ++i) ss[i] = fmaf(c[i].x, c[i].x, fmaf(c[i].y, c[i].y, fmaf(c[i].z, c[i].z, c[i].w * c[i].w)));
#pragma unroll
      for (int m = 4; m >= 1; m >>= 1) {
        const bool high = lane & (4 * m);
#pragma unroll
        for (int i = 0; i < m; ++i) {
          const float give = high ? ss[i] : ss[i + m];
          ss[i] = (high ? ss[i + m] : ss[i]) + __shfl_xor_sync(0xffffffffu, give, 4 * m);
        }
      }
      ss[0] += __shfl_xor_sync(0xffffffffu, ss[0], 2);
      ss[0] += __shfl_xor_sync(0xffffffffu, ss[0], 1);
      const float r = rsqrtf(ss[0] + p.eps);
#pragma unroll
      for (int i = 0; i < R; ++i) put_unit(base + i, c[i], __shfl_sync(0xffffffffu, r, 4 * i));
      return;
    }
  }

  GdnSeq d{0, 0, 0, 0, false, false};
  int64_t known = -1;  // d is that of the rows below
  const bool tells = head == 0 && lane == 0;
#pragma unroll 1
  for (int64_t row = base; row < end; ++row) {
    if (row >= known) {
      int s;
      KvSeq q = kv_locate(p.c, row, lane, s);
      if (!__any_sync(0xffffffffu, kv_has(q, row))) {  // (all lanes or none)
        bool bad;
        q = kv_locate_all(p.c, row, lane, s, bad);
        if (bad && tells) gdn_record();
        if (!q.ok) continue;  // rows of no sequence
      }
      d = gdn_seq(p.c, q, s);
      if (!d.ok && tells) gdn_record();
      known = d.r1;
    }
    if (!d.ok || row < d.first) continue;
    const int64_t at = row - d.first;
    const T* here = x + row * p.x_row;
    const float4 now = R == 1 ? in[0] : load_row4<WIDE>(here);
    if (at >= 3) {
      emit(row, load_row4<WIDE>(here - 3 * p.x_row), load_row4<WIDE>(here - 2 * p.x_row), load_row4<WIDE>(here - p.x_row), now);
      continue;
    }
    if (at > 0) continue;  // taken with the first
    float* st = p.state + (int64_t)d.slot * 3 * chans + ch;
    float4 h0 = gdn_zero4(), h1 = h0, h2 = h0;
    if (!d.fresh) {
      h0 = load4(st);
      h1 = load4(st + chans);
      h2 = load4(st + 2 * chans);
    }
    const int n = d.r1 - d.first;
    float4 y = now;
    emit(row, h0, h1, h2, y);
    for (int j = 1; j < min(n, 3); ++j) {
      h0 = h1;
      h1 = h2;
      h2 = y;
      y = load_row4<WIDE>(x + (row + j) * p.x_row);
      emit(row + j, h0, h1, h2, y);
    }
    if (n > 3) {
      h1 = load_row4<WIDE>(x + (int64_t)(d.r1 - 3) * p.x_row);
      h2 = load_row4<WIDE>(x + (int64_t)(d.r1 - 2) * p.x_row);
      y = load_row4<WIDE>(x + (int64_t)(d.r1 - 1) * p.x_row);
    }
    *reinterpret_cast<float4*>(st) = h1;
    *reinterpret_cast<float4*>(st + chans) = h2;
    *reinterpret_cast<float4*>(st + 2 * chans) = y;
  }
}

template <bool WIDE, typename T>
cudaError_t launch_conv(const ConvParams& p, int sms, cudaStream_t s) {
  const unsigned y = (unsigned)((2 * p.nk + p.nv + 1 + kConvWarps - 1) / kConvWarps);
  if (p.c.rows <= 4LL * sms)
    gdn_conv_kernel<1, WIDE, T><<<dim3((unsigned)p.c.rows, y), kConvThreads, 0, s>>>(p);
  else
    gdn_conv_kernel<8, WIDE, T><<<dim3((unsigned)((p.c.rows + 7) / 8), y), kConvThreads, 0, s>>>(p);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ the gated delta rule, row by row
constexpr int kStepThreads = 256;

// Block s * nv + h: value head h of sequence s.  A warp holds 16 rows of S, a lane four columns of them.  With the decay
// e, S_old^T k and S_old^T q give all of a row: u = beta (v - e S_old^T k), o = e S_old^T q + (q . k) u, S = e S_old + k u^T,
// so that a row takes one sum over the warps.
__global__ void __launch_bounds__(kStepThreads, 2) gdn_step_kernel(const __grid_constant__ GdnParams p) {
  __shared__ __align__(16) float kq[2][2][kGdnDim];
  __shared__ __align__(16) float4 red[2][8][2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = blockIdx.x / p.nv, h = blockIdx.x - s * p.nv;
  const KvSeq seq = kv_seq(p.c, s);
  const GdnSeq d = gdn_seq(p.c, seq, s);
  const int n = d.r1 - d.first;
  if (d.ok && n > p.few) return;  // the chunks' kernel's
  if (!d.ok) {
    if (h == 0 && threadIdx.x == 0) gdn_record();
    return;
  }
  for (int row = d.r0 + warp; row < d.first; row += 8)
    gdn_put4(p.out, p.out_bf16, row * p.out_row + h * p.out_head + 4 * lane, gdn_zero4());
  if (n == 0) return;

  float* st = p.state + (((int64_t)d.slot * p.nv + h) * kGdnDim + 16 * warp) * kGdnDim + 4 * lane;
  float4 S[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) S[i] = d.fresh ? gdn_zero4() : *reinterpret_cast<const float4*>(st + i * kGdnDim);

  const int hk = h / p.group;
  const __half* src = warp == 0 ? p.k + hk * p.k_head : p.q + hk * p.q_head;
  const int64_t src_row = warp == 0 ? p.k_row : p.q_row;
  auto fetch = [&](int row) { return *reinterpret_cast<const uint2*>(src + row * src_row + 4 * lane); };
  auto put = [&](int at, const uint2& w) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
    *reinterpret_cast<float4*>(&kq[at][warp][4 * lane]) = make_float4(a.x, a.y, b.x, b.y);
  };
  if (warp < 2) put(0, fetch(d.first));
  const float4 gain = p.norm_w ? *reinterpret_cast<const float4*>(p.norm_w + 4 * lane) : make_float4(1.0f, 1.0f, 1.0f, 1.0f);
  for (int t = 0; t < n; ++t) {
    const int row = d.first + t, at = t & 1;
    uint2 next = make_uint2(0, 0);
    if (warp < 2 && t + 1 < n) next = fetch(row + 1);
    const float4 v = gdn_bf16x4(*reinterpret_cast<const uint2*>(p.v + row * p.v_row + h * p.v_head + 4 * lane));
    const float e = expf(p.g[(int64_t)row * p.nv + h]), beta = p.beta[(int64_t)row * p.nv + h];
    const bool mine = (t & 7) == warp;  // whose warp's turn it is to write the row
    float4 z = gdn_zero4();
    if (mine && p.z) z = gdn_gate4(p, p.z + row * p.z_row + h * p.z_head + 4 * lane);
    __syncthreads();
    float4 a = gdn_zero4(), b = gdn_zero4();
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const float4 k = *reinterpret_cast<const float4*>(&kq[at][0][16 * warp + i]);
      const float4 q = *reinterpret_cast<const float4*>(&kq[at][1][16 * warp + i]);
      const float kk[4] = {k.x, k.y, k.z, k.w}, qq[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a.x = fmaf(kk[j], S[i + j].x, a.x);
        a.y = fmaf(kk[j], S[i + j].y, a.y);
        a.z = fmaf(kk[j], S[i + j].z, a.z);
        a.w = fmaf(kk[j], S[i + j].w, a.w);
        b.x = fmaf(qq[j], S[i + j].x, b.x);
        b.y = fmaf(qq[j], S[i + j].y, b.y);
        b.z = fmaf(qq[j], S[i + j].z, b.z);
        b.w = fmaf(qq[j], S[i + j].w, b.w);
      }
    }
    red[at][warp][0][lane] = a;
    red[at][warp][1][lane] = b;
    if (warp < 2 && t + 1 < n) put(1 - at, next);
    const float4 k4 = *reinterpret_cast<const float4*>(&kq[at][0][4 * lane]), q4 = *reinterpret_cast<const float4*>(&kq[at][1][4 * lane]);
    const float qk = gdn_warp_sum(fmaf(k4.x, q4.x, fmaf(k4.y, q4.y, fmaf(k4.z, q4.z, k4.w * q4.w))));
    __syncthreads();
    a = red[at][0][0][lane];
    b = red[at][0][1][lane];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      const float4 x = red[at][i][0][lane], y = red[at][i][1][lane];
      a = make_float4(a.x + x.x, a.y + x.y, a.z + x.z, a.w + x.w);
      b = make_float4(b.x + y.x, b.y + y.y, b.z + y.z, b.w + y.w);
    }
    const float4 u = make_float4(beta * (v.x - e * a.x), beta * (v.y - e * a.y), beta * (v.z - e * a.z), beta * (v.w - e * a.w));
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const float4 k = *reinterpret_cast<const float4*>(&kq[at][0][16 * warp + i]);
      const float kk[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        S[i + j] = make_float4(fmaf(kk[j], u.x, e * S[i + j].x), fmaf(kk[j], u.y, e * S[i + j].y),
                               fmaf(kk[j], u.z, e * S[i + j].z), fmaf(kk[j], u.w, e * S[i + j].w));
    }
    if (!mine) continue;
    float4 o = make_float4(p.scale * fmaf(qk, u.x, e * b.x), p.scale * fmaf(qk, u.y, e * b.y),
                           p.scale * fmaf(qk, u.z, e * b.z), p.scale * fmaf(qk, u.w, e * b.w));
    float r = 1.0f;
    if (p.norm_w)
      r = rsqrtf(fmaf(gdn_warp_sum(fmaf(o.x, o.x, fmaf(o.y, o.y, fmaf(o.z, o.z, o.w * o.w)))), 1.0f / kGdnDim, p.eps));
    o = make_float4(o.x * r * gain.x, o.y * r * gain.y, o.z * r * gain.z, o.w * r * gain.w);
    if (p.z) o = make_float4(o.x * gdn_silu(z.x), o.y * gdn_silu(z.y), o.z * gdn_silu(z.z), o.w * gdn_silu(z.w));
    gdn_put4(p.out, p.out_bf16, row * p.out_row + h * p.out_head + 4 * lane, o);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) *reinterpret_cast<float4*>(st + i * kGdnDim) = S[i];
}

// Host side: checks of the batch; fills the view.
int gdn_view(const fak_gdn_batch* b, int n_slots, KvView* w) {
  if (b->n_seqs < 0 || (b->n_seqs && n_slots < 1)) return FAK_ERR_SHAPE;
  if (b->n_seqs && (!b->row_start || !b->kv_len || !b->slot)) return FAK_ERR_INVALID_ARG;  // (an empty tensor has no address)
  if (((uintptr_t)b->row_start | (uintptr_t)b->kv_len | (uintptr_t)b->slot) & 3) return FAK_ERR_ALIGN;
  w->table = b->slot;
  w->row_start = b->row_start;
  w->kv_len = b->kv_len;
  w->n_seqs = b->n_seqs;
  w->n_pages = n_slots;
  w->max_pages = w->max_q = w->max_kv = 0x7fffffff;
  w->page_shift = 0;
  return FAK_OK;
}

}  // namespace

extern "C" int fak_gdn_conv(const fak_gdn_batch* batch, const fak_gdn_rows* r, fak_stream_t stream) {
  ConvParams p;
  memset(&p, 0, sizeof(p));
  if (!batch || !r) return FAK_ERR_INVALID_ARG;
  int st = gdn_view(batch, r->n_slots, &p.c);
  if (st != FAK_OK) return st;
  if (r->type != FAK_ROWS_F32 && r->type != FAK_ROWS_BF16) return FAK_ERR_INVALID_ARG;
  if (r->nk < 1 || r->nv < 1 || r->nk > (1 << 16) || r->nv > (1 << 16) || r->rows < 0 || r->rows > 0x7fffffff) return FAK_ERR_SHAPE;
  if (r->rows && (!r->x || !r->b || !r->a || !r->q || !r->k || !r->v || !r->g || !r->beta)) return FAK_ERR_INVALID_ARG;
  if (!r->conv_w || !r->a_log || !r->dt_bias || !r->conv_state || !(r->eps >= 0.0f) || !std::isfinite(r->eps)) return FAK_ERR_INVALID_ARG;
  const int elem = r->type == FAK_ROWS_F32 ? 4 : 2;
  p.x_row = kv_stride(r->x_row, r->rows);
  p.b_row = kv_stride(r->b_row, r->rows);
  p.a_row = kv_stride(r->a_row, r->rows);
  const uintptr_t bits = (uintptr_t)r->conv_w | (uintptr_t)r->conv_state | (uintptr_t)r->q | (uintptr_t)r->k | (uintptr_t)r->v;
  const uintptr_t words = (uintptr_t)r->a_log | (uintptr_t)r->dt_bias | (uintptr_t)r->g | (uintptr_t)r->beta;
  if ((bits & 15) || (words & 3) || (((uintptr_t)r->x | (uintptr_t)r->b | (uintptr_t)r->a) & (elem - 1))) return FAK_ERR_ALIGN;
  if (r->rows == 0 || batch->n_seqs == 0) return FAK_OK;
  int sms = 0;
  if ((st = kv_device(nullptr, &sms)) != FAK_OK) return st;
  p.c.rows = r->rows;
  p.x = r->x;
  p.b = r->b;
  p.a = r->a;
  p.conv_w = r->conv_w;
  p.a_log = r->a_log;
  p.dt_bias = r->dt_bias;
  p.state = r->conv_state;
  p.q = static_cast<__half*>(r->q);
  p.k = static_cast<__half*>(r->k);
  p.v = static_cast<__nv_bfloat16*>(r->v);
  p.g = r->g;
  p.beta = r->beta;
  p.eps = r->eps;
  p.nk = r->nk;
  p.nv = r->nv;
  cudaStream_t s = (cudaStream_t)stream;
  // four channels a load where every row stands on a multiple of four elements
  const bool wide = !((uintptr_t)r->x & (4 * elem - 1)) && !(p.x_row & 3);
  return fak_cuda_status(elem == 4 ? (wide ? launch_conv<true, float>(p, sms, s) : launch_conv<false, float>(p, sms, s))
                                   : (wide ? launch_conv<true, __nv_bfloat16>(p, sms, s) : launch_conv<false, __nv_bfloat16>(p, sms, s)));
}

extern "C" int fak_gdn_attn(const fak_gdn_batch* batch, const fak_gdn_args* a, fak_stream_t stream) {
  GdnParams p;
  memset(&p, 0, sizeof(p));
  if (!batch || !a) return FAK_ERR_INVALID_ARG;
  int st = gdn_view(batch, a->n_slots, &p.c);
  if (st != FAK_OK) return st;
  if (a->out_type != FAK_ROWS_F32 && a->out_type != FAK_ROWS_BF16) return FAK_ERR_INVALID_ARG;
  if (a->nk < 1 || a->nv < 1 || a->nv > 65535 || a->nv % a->nk || a->rows < 0 || a->rows > 0x7fffffff || a->max_q < 0 ||
      (int64_t)batch->n_seqs * a->nv > 0x3fffffff)
    return FAK_ERR_SHAPE;
  if (!(a->scale > 0.0f) || !std::isfinite(a->scale) || !(a->eps >= 0.0f) || !std::isfinite(a->eps)) return FAK_ERR_INVALID_ARG;
  if (a->rows && (!a->q || !a->k || !a->v || !a->g || !a->beta || !a->out)) return FAK_ERR_INVALID_ARG;
  if (!a->state) return FAK_ERR_INVALID_ARG;
  p.q_row = kv_stride(a->q_row, a->rows);
  p.q_head = kv_stride(a->q_head, a->nk);
  p.k_row = kv_stride(a->k_row, a->rows);
  p.k_head = kv_stride(a->k_head, a->nk);
  p.v_row = kv_stride(a->v_row, a->rows);
  p.v_head = kv_stride(a->v_head, a->nv);
  p.z_row = kv_stride(a->z_row, a->rows);
  p.z_head = kv_stride(a->z_head, a->nv);
  p.out_row = kv_stride(a->out_row, a->rows);
  p.out_head = kv_stride(a->out_head, a->nv);
  const uintptr_t bits = (uintptr_t)a->q | (uintptr_t)a->k | (uintptr_t)a->v | (uintptr_t)a->state | (uintptr_t)a->norm_w |
                         (uintptr_t)a->out;
  const int64_t two = p.q_row | p.q_head | p.k_row | p.k_head | p.v_row | p.v_head;  // strides of 16-bit rows
  const int64_t out = p.out_row | p.out_head;
  const auto fits = [](int64_t stride, int64_t n, int elem) { return n <= 1 || (stride > 0 && stride < (1LL << 40) / elem); };
  if (!fits(p.q_row, a->rows, 2) || !fits(p.q_head, a->nk, 2) || !fits(p.k_row, a->rows, 2) || !fits(p.k_head, a->nk, 2) ||
      !fits(p.v_row, a->rows, 2) || !fits(p.v_head, a->nv, 2))
    return FAK_ERR_INVALID_ARG;
  const auto meet = [](int64_t stride, int64_t n) { return n > 1 && stride > -kGdnDim && stride < kGdnDim; };  // vectors written over one another
  if (meet(a->out_row, a->rows) || meet(a->out_head, a->nv)) return FAK_ERR_INVALID_ARG;
  if ((bits & 15) || (two & 7) || (out & (a->out_type == FAK_ROWS_F32 ? 3 : 7)) || 
      (((uintptr_t)a->g | (uintptr_t)a->beta | (uintptr_t)a->z) & 3))
    return FAK_ERR_ALIGN;
  if (a->rows == 0 || batch->n_seqs == 0) return FAK_OK;
  int dev = 0, sms = 0;
  if ((st = kv_device(&dev, &sms)) != FAK_OK) return st;
  p.c.rows = a->rows;
  p.c.max_q = a->max_q;
  p.q = static_cast<const __half*>(a->q);
  p.k = static_cast<const __half*>(a->k);
  p.v = static_cast<const __nv_bfloat16*>(a->v);
  p.g = a->g;
  p.beta = a->beta;
  p.norm_w = a->norm_w;
  p.z = a->z;
  p.z_wide = !(((uintptr_t)a->z & 15) | ((p.z_row | p.z_head) & 3)) && fits(p.z_row, a->rows, 4) && fits(p.z_head, a->nv, 4);
  p.state = a->state;
  p.out = a->out;
  p.out_wide = fits(p.out_row, a->rows, 4) && fits(p.out_head, a->nv, 4);
  p.scale = a->scale;
  p.eps = a->eps;
  p.nv = a->nv;
  p.group = a->nv / a->nk;
  p.out_bf16 = a->out_type == FAK_ROWS_BF16;
  cudaStream_t s = (cudaStream_t)stream;
  // Sequences of more than kGdnFew rows go over chunks of 64, the others row by row.  (The chunks first: where their scratch
  // cannot be had, nothing is launched.)
  const bool few = std::min<int64_t>(a->max_q, a->rows) <= kGdnFew;
  if (few || batch->n_seqs > 1) p.few = kGdnFew;
  if (!few) {
    void* status = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&status, g_gdn_status);
    if (e != cudaSuccess) return fak_cuda_status(e);
    e = gdn_chunk_launch(p, g_gdn_timeout.load(std::memory_order_relaxed), g_gdn_unreachable.load(std::memory_order_relaxed),
                         static_cast<int*>(status), dev, sms, s);
    st = fak_cuda_status(e);
    if (e != cudaSuccess) return e == cudaErrorMemoryAllocation ? FAK_ERR_NOMEM : st;
  }
  if (p.few) gdn_step_kernel<<<(unsigned)(batch->n_seqs * a->nv), kStepThreads, 0, s>>>(p);
  return fak_cuda_status(cudaGetLastError());
}

extern "C" int fak_gdn_debug_wait(int64_t timeout_ns, int unreachable) {
  if (timeout_ns < 0 || (unreachable != 0 && unreachable != 1)) return FAK_ERR_INVALID_ARG;
  g_gdn_timeout = timeout_ns ? (unsigned long long)timeout_ns : kGdnTimeout;
  g_gdn_unreachable = unreachable;
  return FAK_OK;
}

int fak_gdn_take_status() {
  int v = 0, zero = 0;
  const cudaError_t e = cudaMemcpyFromSymbol(&v, g_gdn_status, sizeof(int));
  if (e != cudaSuccess) return fak_cuda_status(e);
  cudaMemcpyToSymbol(g_gdn_status, &zero, sizeof(int));
  return v;
}
