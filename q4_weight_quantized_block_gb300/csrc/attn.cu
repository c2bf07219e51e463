// Softmax attention of new rows over the paged KV cache (fak_paged_attn).
//
// The call's checks, the cut of its keys into pieces where there are few rows, and the kernel that
// joins the pieces.  The attention itself: attn_rows.cu for few rows (decode steps), attn_tile.cu for more.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "attn_device.cuh"
#include "fak.h"
#include "fak_device.cuh"

namespace {

__device__ int g_attn_status;

std::atomic<int64_t> g_wait_ns{0};       // fak_paged_attn_debug_wait's
std::atomic<int> g_unreachable{0};

constexpr int kPlanSms = 152;  // GB300's SMs: the workspace's size must not depend on the current device

// Adds up the pieces of the blocks of rows whose keys were cut: W warps (1, eight (row, query head)s to a block, or 16)
// to a (row, query head), each for every W-th piece.
//   out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i * sigmoid(gate),  M = max m_i
// in an order that the pieces' number alone sets, so the result does not depend on which finished first.
template <int DH, int W>
__global__ void __launch_bounds__(W == 1 ? 256 : 512) attn_join_kernel(const __grid_constant__ AttnParams p) {
  constexpr int N = DH / 32, kJoin = W == 1 ? 8 : 1;  // (row, query head)s of a block
  __shared__ float so[W][DH], sl[W];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = blockIdx.y * kJoin + warp / W;
  const int64_t row = blockIdx.x;
  int s;
  KvSeq sq = kv_locate(p.c, row, lane, s);
  bool bad;
  if (!kv_has(sq, row)) sq = kv_locate_all(p.c, row, lane, s, bad);
  // the pieces' kernel is done (every block waits: this grid must not end before that one)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!sq.ok) return;
  if (W == 1 && h >= p.nq) return;
  const int token = (int)(row - sq.r0);
  const int tokens = sq.r1 - sq.r0, base = token / p.block * p.block, last = base + min(p.block, tokens - base) - 1;
  const int p0 = sq.len - tokens, pos = p0 + token;
  const KeyTiles kt = key_tiles(p0 + base, p0 + last, p.window, p.sinks, p.tile_shift);
  if (kt.n <= p.per_split) return;  // one piece: the block wrote its result itself
  const int pieces = min(p.splits, ceil_div(kt.n, p.per_split));
  const int64_t slot = row * p.nq + h, step = p.c.rows * p.nq;
  float top = -INFINITY;
  for (int i = lane; i < pieces; i += 32) top = fmaxf(top, p.stat[slot + i * step].x);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  // (2^12 above the largest: there are fewer pieces, so pieces as large as f32 holds do not add up beyond it)
  const float zero = top == -INFINITY ? 0.0f : top + 12.0f;
  float o[N] = {}, l = 0.0f;
  constexpr int U = 4;  // pieces in flight
  for (int i0 = warp % W; i0 < pieces; i0 += U * W) {
    float2 st[U];
    float x[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = slot + (int64_t)(i0 + u * W) * step;
      st[u] = make_float2(-INFINITY, 0.0f);
      if (i0 + u * W < pieces) {
        st[u] = p.stat[at];
#pragma unroll
        for (int k = 0; k < N; ++k) x[u][k] = p.part[at * DH + lane + 32 * k];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u * W >= pieces) break;
      const float f = exp2_approx(st[u].x - zero);
      l = fmaf(f, st[u].y, l);
#pragma unroll
      for (int k = 0; k < N; ++k) o[k] = fmaf(f, x[u][k], o[k]);
    }
  }
  if constexpr (W > 1) {
#pragma unroll
    for (int k = 0; k < N; ++k) so[warp][lane + 32 * k] = o[k];
    if (lane == 0) sl[warp] = l;
    __syncthreads();
    if (warp >= N) return;
    o[0] = l = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      o[0] += so[w][warp * 32 + lane];
      l += sl[w];
    }
  }
#pragma unroll
  for (int k = 0; k < (W > 1 ? 1 : N); ++k) {
    const int d = lane + 32 * (W > 1 ? warp : k);
    float y = o[k] / l;
    if (p.gate) y = gated_by(y, p.gate[row * p.gate_row + h * p.gate_head + d]);
    p.out[row * p.out_row + h * p.out_head + d] = __float2bfloat16_rn(pos < 0 ? 0.0f : y);
  }
}

// How a call is cut.
struct Plan {
  bool few;                     // the kernel for few rows
  int64_t blocks;               // blocks of rows of one KV head, at most
  int block, tile;              // tokens of a block, keys of a tile
  int splits, per_split;
};

Plan make_plan(const fak_kv_cache* c, const fak_kv_batch* b, const fak_attn_args* a) {
  Plan pl;
  const int group = a->nq / c->n_kv;
  const int64_t rows = (int64_t)a->max_q * group;
  pl.few = rows <= kRowsMax;
  // whole tokens to a block; pairs of CTAs where sequences have more than one CTA holds (and half of V's dims are 64)
  const int own = kTileM / group, ctas = !pl.few && c->dh > 64 && a->max_q > own ? 2 : 1;
  pl.block = pl.few ? kRowsMax : own * ctas;
  pl.blocks = pl.few ? b->n_seqs : a->rows / pl.block + b->n_seqs;  // see find_unit
  pl.tile = !pl.few ? kTileN : c->kind == FAK_KV_BF16 || c->dh > 128 ? kRowsN : 2 * kRowsN;
  int64_t tiles = ((int64_t)a->max_kv + pl.tile - 1) / pl.tile;
  if (a->window && a->window < a->max_kv) {
    const int64_t span = pl.block;
    tiles = std::min<int64_t>(tiles, ((int64_t)a->window + span) / pl.tile + 2 +
                                         std::min<int64_t>((int64_t)a->sinks / pl.tile + 1, tiles));
  }
  tiles = std::max<int64_t>(tiles, 1);
  const int64_t each = pl.few ? 1 : (a->max_q + pl.block - 1) / pl.block;  // blocks of a sequence, at most
  const int64_t busy = std::max<int64_t>(1, std::min<int64_t>(pl.blocks, b->n_seqs * each) * ctas * c->n_kv);
  pl.splits = 1;
  pl.per_split = (int)tiles;
  if (pl.few) {
    // One sequence's pieces are all alike: as many as blocks fit at once.  Several sequences differ in length, which
    // smaller pieces even out: four times as many, of 512 keys or more.  (64 of up to 8,191 e4m3 keys of 256, in pieces
    // of 512 keys 157 us, of 1,024 130, of 2,048 144, whole 218; measured on this batch alone.)
    const int64_t places = rows_blocks(c->kind != FAK_KV_BF16, c->dh, (int)rows) * kPlanSms, least = 512 / pl.tile;
    const int64_t four = std::max<int64_t>(1, 4 * places / busy), one = std::max<int64_t>(1, places / busy);
    int64_t per = std::max<int64_t>(least, (tiles + four - 1) / four);
    if (b->n_seqs == 1 || (tiles + per - 1) / per * busy < places) per = (tiles + one - 1) / one;
    pl.per_split = (int)std::min(per, tiles);
    pl.splits = (int)((tiles + pl.per_split - 1) / pl.per_split);
    return pl;
  }
  // The cut that is over soonest if every block saw all `tiles`: waves of blocks over the SMs, each as long as a piece
  // and the time of about three tiles to begin and to end, seven where it leaves its sums in memory, and four more for
  // the join.  (512 rows after 8,191 keys of 256: whole 105 us, in two 127, in four 120; after 30,000: 313, 333, 277.
  // The three times are from this form alone, bf16 at dh 256; other forms' tiles take 0.8 to 1.3 times as long, and
  // theirs were not measured.)
  int64_t best = -1;
  for (int64_t s = 1; s <= 64 && s <= tiles; ++s) {
    const int64_t per = (tiles + s - 1) / s, n = (tiles + per - 1) / per;
    const int64_t cost = (busy * n + kPlanSms - 1) / kPlanSms * (per + (n > 1 ? 7 : 3)) + (n > 1 ? 4 : 0);
    if (best < 0 || cost < best) {
      best = cost;
      pl.splits = (int)n;
      pl.per_split = (int)per;
    }
  }
  return pl;
}

// Workspace: the pieces' sums, then their bases and weight sums.
size_t part_bytes(const fak_kv_cache* c, const fak_attn_args* a, const Plan& pl) {
  return pl.splits < 2 ? 0 : (size_t)pl.splits * a->rows * a->nq * c->dh * 4;
}
size_t stat_bytes(const fak_attn_args* a, const Plan& pl) {
  return pl.splits < 2 ? 0 : (size_t)pl.splits * a->rows * a->nq * 8;
}

template <int DH>
cudaError_t launch_join(const AttnParams& p, cudaStream_t s) {
  // 16 warps to a (row, query head) where pieces are many and the blocks run all at once (512 rows' nine pieces took
  // 16 warps 190 us longer than one)
  const bool many = p.splits > 8 && p.c.rows * p.nq <= 4 * kPlanSms;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((unsigned)p.c.rows, (unsigned)(many ? p.nq : (p.nq + 7) / 8));
  cfg.blockDim = dim3(many ? 512 : 256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return many ? cudaLaunchKernelEx(&cfg, attn_join_kernel<DH, 16>, p) : cudaLaunchKernelEx(&cfg, attn_join_kernel<DH, 1>, p);
}

int attn_shape(const fak_kv_cache* c, const fak_attn_args* a) {
  if (a->window < 0 || a->sinks < 0 || !(a->scale > 0.0f) || !std::isfinite(a->scale)) return FAK_ERR_INVALID_ARG;
  if (a->nq < 1 || a->nq % c->n_kv || a->nq / c->n_kv > 128 || a->rows < 0 || a->rows > 0x7fffffff || a->max_q < 0 ||
      a->max_kv < 0 || a->max_q > 1 << 28 || a->max_kv > 1 << 29 || a->nq > 65535 || a->rows * a->nq > 1LL << 40)
    return FAK_ERR_SHAPE;
  return FAK_OK;
}

}  // namespace

extern "C" size_t fak_paged_attn_workspace_bytes(const fak_kv_cache* cache, const fak_kv_batch* batch,
                                                 const fak_attn_args* a) {
  if (!cache || !batch || !a || cache->n_kv < 1 || batch->n_seqs < 0 || attn_shape(cache, a) != FAK_OK) return 0;
  const Plan pl = make_plan(cache, batch, a);
  return part_bytes(cache, a, pl) + stat_bytes(a, pl);
}

extern "C" int fak_paged_attn(const fak_kv_cache* cache, const fak_kv_batch* batch, const fak_attn_args* a,
                              fak_stream_t stream) {
  AttnParams p;
  memset(&p, 0, sizeof(p));
  int st = kv_view(cache, batch, &p.c);
  if (st != FAK_OK) return st;
  if (!a || (a->rows && (!a->q || !a->out))) return FAK_ERR_INVALID_ARG;
  if ((st = attn_shape(cache, a)) != FAK_OK) return st;
  p.q_row = kv_stride(a->q_row, a->rows);
  p.q_head = kv_stride(a->q_head, a->nq);
  p.out_row = kv_stride(a->out_row, a->rows);
  p.out_head = kv_stride(a->out_head, a->nq);
  p.gate_row = a->gate ? kv_stride(a->gate_row, a->rows) : 0;
  p.gate_head = a->gate ? kv_stride(a->gate_head, a->nq) : 0;
  // (a tensor map's strides are above zero and below 2^40 bytes)
  constexpr int64_t least = 1, most = 1LL << 38;
  if ((a->rows > 1 && (p.q_row < least || p.q_row > most)) || (a->nq > 1 && (p.q_head < least || p.q_head > most)))
    return FAK_ERR_SHAPE;
  if ((((uintptr_t)a->q | (uintptr_t)a->out | (uintptr_t)a->gate) & 15) ||
      ((p.q_row | p.q_head | p.out_row | p.out_head) & 7) || ((p.gate_row | p.gate_head) & 3) ||
      ((uintptr_t)a->workspace & 255))
    return FAK_ERR_ALIGN;
  const Plan pl = make_plan(cache, batch, a);
  const size_t parts = part_bytes(cache, a, pl), need = parts + stat_bytes(a, pl);
  if (need && !a->workspace) return FAK_ERR_INVALID_ARG;
  if (a->workspace_bytes < need) return FAK_ERR_SHAPE;
  if (pl.blocks > 0x3fffffff || cache->n_kv > 65535) return FAK_ERR_SHAPE;
  if (a->rows == 0 || batch->n_seqs == 0) return FAK_OK;
  int dev = 0;
  if ((st = kv_device(&dev, nullptr)) != FAK_OK) return st;
  static std::atomic<int*> words[64];  // the status word's address on each device
  int* st_word = words[dev].load(std::memory_order_relaxed);
  cudaError_t e = cudaSuccess;
  if (!st_word) {
    e = cudaGetSymbolAddress(reinterpret_cast<void**>(&st_word), g_attn_status);
    if (e != cudaSuccess) return fak_cuda_status(e);
    words[dev].store(st_word, std::memory_order_relaxed);
  }
  p.c.rows = a->rows;
  p.c.max_q = a->max_q;
  p.c.max_kv = a->max_kv;
  p.q = static_cast<const __nv_bfloat16*>(a->q);
  p.gate = a->gate;
  p.out = static_cast<__nv_bfloat16*>(a->out);
  p.scale = a->scale * 1.4426950408889634f;
  p.nq = a->nq;
  p.group = a->nq / cache->n_kv;
  p.block = pl.block;
  p.tile_shift = pl.tile == 64 ? 6 : 7;
  p.by_group = quotient(p.group);
  p.by_block = quotient(p.block);
  p.window = a->window >= a->max_kv ? 0 : a->window;  // (as wide as the longest sequence: none)
  p.sinks = p.window ? std::min(a->sinks, a->max_kv) : 0;
  p.splits = pl.splits;
  p.per_split = pl.per_split;
  p.part = static_cast<float*>(a->workspace);
  p.stat = reinterpret_cast<float2*>(static_cast<uint8_t*>(a->workspace) + parts);
  // (a wait may be for a whole block: 2 s, and 20 us for each of its tiles)
  const int64_t wait_ns = g_wait_ns.load(std::memory_order_relaxed);
  p.timeout_ns = wait_ns ? (unsigned long long)wait_ns : 2000000000ull + 20000ull * (unsigned)pl.per_split;
  p.unreachable = g_unreachable.load(std::memory_order_relaxed);
  cudaStream_t s = (cudaStream_t)stream;
  e = pl.few ? attn_rows_launch(cache->kind, cache->dh, p, st_word, dev, s)
             : attn_tile_launch(cache->kind, cache->dh, cache->page, cache->n_pages * cache->n_kv * cache->page, p,
                                pl.blocks, st_word, dev, s);
  if (e == cudaSuccess && pl.splits > 1)
    e = cache->dh == 64 ? launch_join<64>(p, s) : cache->dh == 128 ? launch_join<128>(p, s) : launch_join<256>(p, s);
  return fak_cuda_status(e);
}

extern "C" int fak_paged_attn_debug_wait(int64_t timeout_ns, int unreachable) {
  if (timeout_ns < 0 || (unreachable != 0 && unreachable != 1)) return FAK_ERR_INVALID_ARG;
  g_wait_ns.store(timeout_ns, std::memory_order_relaxed);
  g_unreachable.store(unreachable, std::memory_order_relaxed);
  return FAK_OK;
}

int fak_attn_take_status() {
  int v = 0, zero = 0;
  const cudaError_t e = cudaMemcpyFromSymbol(&v, g_attn_status, sizeof(int));
  if (e != cudaSuccess) return fak_cuda_status(e);
  cudaMemcpyToSymbol(g_attn_status, &zero, sizeof(int));
  return v;
}
