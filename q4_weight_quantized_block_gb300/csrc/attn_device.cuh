// What the attention kernels share: a call's parameters, the plan of its split over
// the keys, and the keys that a block of rows sees.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "kv_device.cuh"

struct AttnParams {
  KvView c;
  const __nv_bfloat16* q;
  const float* gate;
  __nv_bfloat16* out;
  int64_t q_row, q_head, gate_row, gate_head, out_row, out_head;
  float scale;  // times log2(e): scores are held in powers of two
  int nq, group, window, sinks;
  int block_shift;  // rows of a block: 128, or 256 in a pair of CTAs
  uint32_t group_mul;  // r / group = r group_mul / 2^(32 + group_shift) for 0 <= r < 2^31 (group 1: group_mul 0)
  int group_shift;
  // the keys of a block of rows are cut into at most `splits` pieces of `per_split` key tiles; a block with more
  // than one piece leaves, for each piece, row and head, the unnormalised sum (part, dh values) and its base and
  // weight sum (stat), which the join kernel adds up
  int splits, per_split;
  float* part;   // [splits][rows][nq][dh]
  float2* stat;  // [splits][rows][nq]
  unsigned long long timeout_ns;

  __device__ __forceinline__ int by_group(int r) const {
    return group_mul ? (int)(__umulhi((uint32_t)r, group_mul) >> group_shift) : r;
  }
};

constexpr int kTileM = 128;  // rows (token, query head of the group) of a CTA
constexpr int kTileN = 128;  // keys of a tile

FAK_DEV int ceil_div(int a, int b) { return (a + b - 1) / b; }

// The key tiles that rows at positions p_lo .. p_hi see: those of the first few positions that lie
// before the window's tiles, then the window's.
struct KeyTiles {
  int n, head, first;  // tiles in all, tiles of the sinks, first tile of the window
};

FAK_DEV KeyTiles key_tiles(int p_lo, int p_hi, int window, int sinks) {
  KeyTiles t{0, 0, 0};
  if (p_hi < 0) return t;
  if (window) {
    const int low = max(0, max(0, p_lo) - window + 1);
    t.first = low / kTileN;
    t.head = min(ceil_div(min(sinks, p_hi + 1), kTileN), t.first);
  }
  t.n = t.head + p_hi / kTileN - t.first + 1;
  return t;
}

FAK_DEV int key_tile(const KeyTiles& t, int i) { return i < t.head ? i : t.first + i - t.head; }

// Records a device-side error of the call (attn.cu's status word).
FAK_DEV void attn_record(int* status, int code) { atomicCAS(status, 0, code); }

// Host: launches of the kernels in the other files.
cudaError_t attn_tile_launch(int kind, int dh, int page, int64_t n_vec, const AttnParams& p, int64_t blocks,
                             int* status, cudaStream_t s);
