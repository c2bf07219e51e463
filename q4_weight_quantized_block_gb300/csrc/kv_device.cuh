// The paged KV cache as its kernels see it: the ragged batch, the places of
// positions, and the host-side checks shared by kv.cu and attn.cu.
#pragma once
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "fak.h"
#include "fak_device.cuh"

struct KvView {
  const int32_t* table;
  const int32_t* row_start;
  const int32_t* kv_len;
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  int64_t rows;
  int n_seqs, max_pages, n_kv, page_shift, n_pages;
  int max_q, max_kv;  // bounds of the call (append and read: none)
};

// One sequence's rows [r0, r1) and length; ok is false when its numbers are out of range.
struct KvSeq {
  int r0, r1, len;
  bool ok;
};

FAK_DEV bool kv_seq_ok(const KvView& c, const KvSeq& q) {
  return q.r0 >= 0 && q.r0 <= q.r1 && q.r1 <= c.rows && q.len >= 0 &&
         (int64_t)q.len <= ((int64_t)c.max_pages << c.page_shift) && q.r1 - q.r0 <= c.max_q && q.len <= c.max_kv;
}

FAK_DEV KvSeq kv_seq(const KvView& c, int s) {
  KvSeq q;
  q.r0 = c.row_start[s];
  q.r1 = c.row_start[s + 1];
  q.len = c.kv_len[s];
  q.ok = kv_seq_ok(c, q);
  return q;
}

// The last sequence whose rows begin at or before `row` (a whole warp calls): 32 probes a round.
FAK_DEV int kv_find_seq(const KvView& c, int64_t row, int lane) {
  int lo = 0, hi = c.n_seqs;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, i = lo + lane * step;
    const unsigned b = __ballot_sync(0xffffffffu, i < hi && c.row_start[i] <= row);
    const int n = __popc(b);
    if (n > 1) lo += (n - 1) * step;
    hi = min(lo + step, hi);
  }
  return lo;
}

// A row's sequence s and its numbers where the starts rise (a whole warp calls).  Up to 31 sequences' numbers are read at
// once, which saves a trip to memory.  What is found may not have the row: kv_has tells.
FAK_DEV KvSeq kv_locate(const KvView& c, int64_t row, int lane, int& s) {
  if (c.n_seqs < 32) {
    const int start = lane <= c.n_seqs ? c.row_start[lane] : 0x7fffffff;
    const int len = lane < c.n_seqs ? c.kv_len[lane] : 0;
    s = max(__popc(__ballot_sync(0xffffffffu, lane < c.n_seqs && start <= row)) - 1, 0);
    KvSeq q;
    q.r0 = __shfl_sync(0xffffffffu, start, s);
    q.r1 = __shfl_sync(0xffffffffu, start, s + 1);
    q.len = __shfl_sync(0xffffffffu, len, s);
    q.ok = kv_seq_ok(c, q);
    return q;
  }
  s = kv_find_seq(c, row, lane);
  return kv_seq(c, s);
}

FAK_DEV bool kv_has(const KvSeq& q, int64_t row) { return q.ok && q.r0 <= row && row < q.r1; }

// The same where they may fall, as they do beside numbers that are out of range: all sequences are looked at (a row that
// several have is one of theirs).  ok is false where none has the row; bad: some numbers are out of range.
FAK_DEV KvSeq kv_locate_all(const KvView& c, int64_t row, int lane, int& s, bool& bad) {
  bad = false;
#pragma unroll 1
  for (int base = 0; base < c.n_seqs; base += 32) {
    KvSeq q{0, 0, 0, true};
    if (base + lane < c.n_seqs) q = kv_seq(c, base + lane);
    bad |= __any_sync(0xffffffffu, !q.ok);
    const unsigned has = __ballot_sync(0xffffffffu, kv_has(q, row));
    if (!has) continue;
    const int src = 31 - __clz(has);
    s = base + src;
    q.r0 = __shfl_sync(0xffffffffu, q.r0, src);
    q.r1 = __shfl_sync(0xffffffffu, q.r1, src);
    q.len = __shfl_sync(0xffffffffu, q.len, src);
    q.ok = bad = true;  // (with rising starts it had been found)
    return q;
  }
  return KvSeq{0, 0, 0, false};
}

// The vector index (page, head, slot) of position `pos` of sequence s; -1 - that of page 0 when the
// table holds a page that is not there.  pos lies below max_pages * page.
FAK_DEV int64_t kv_place(const KvView& c, int s, int pos, int head) {
  const int pg = c.table[(int64_t)s * c.max_pages + (pos >> c.page_shift)];
  const int slot = pos & ((1 << c.page_shift) - 1);
  if ((unsigned)pg >= (unsigned)c.n_pages) return -1 - (((int64_t)head << c.page_shift) + slot);
  return (((int64_t)pg * c.n_kv + head) << c.page_shift) + slot;
}

// Host side: the stride of a dimension of n; one that is never taken may be anything.
static inline int64_t kv_stride(int64_t stride, int64_t n) { return n > 1 ? stride : 0; }

// Host side: checks of the cache and the batch; fills the view.
static inline int kv_view(const fak_kv_cache* c, const fak_kv_batch* b, KvView* w) {
  if (!c || !b) return FAK_ERR_INVALID_ARG;
  if (c->kind != FAK_KV_BF16 && c->kind != FAK_KV_E4M3 && c->kind != FAK_KV_I8) return FAK_ERR_INVALID_ARG;
  const bool quant = c->kind != FAK_KV_BF16;
  if (!c->k || !c->v || (quant && (!c->k_scale || !c->v_scale))) return FAK_ERR_INVALID_ARG;
  const bool none = b->n_seqs == 0;  // (an empty tensor has no address)
  if (!none && (!b->page_table || !b->row_start || !b->kv_len)) return FAK_ERR_INVALID_ARG;
  if ((c->dh != 64 && c->dh != 128 && c->dh != 256) || c->page < 16 || c->page > 256 || (c->page & (c->page - 1)))
    return FAK_ERR_SHAPE;
  if (c->n_kv < 1 || c->n_pages < 1 || c->n_pages >= (1LL << 31) || b->n_seqs < 0 || (!none && b->max_pages < 1))
    return FAK_ERR_SHAPE;
  if (c->n_kv >= (1LL << 31) / c->page / c->n_pages) return FAK_ERR_SHAPE;  // n_pages * n_kv * page < 2^31
  const uintptr_t bits = (uintptr_t)c->k | (uintptr_t)c->v;
  if (bits & 15) return FAK_ERR_ALIGN;
  if (quant && (((uintptr_t)c->k_scale | (uintptr_t)c->v_scale) & 15)) return FAK_ERR_ALIGN;
  if (((uintptr_t)b->page_table | (uintptr_t)b->row_start | (uintptr_t)b->kv_len) & 3) return FAK_ERR_ALIGN;
  w->table = b->page_table;
  w->row_start = b->row_start;
  w->kv_len = b->kv_len;
  w->k = static_cast<uint8_t*>(c->k);
  w->v = static_cast<uint8_t*>(c->v);
  w->ks = quant ? c->k_scale : nullptr;
  w->vs = quant ? c->v_scale : nullptr;
  w->n_seqs = b->n_seqs;
  w->max_pages = b->max_pages;
  w->n_kv = c->n_kv;
  w->page_shift = __builtin_ctz((unsigned)c->page);
  w->n_pages = (int)c->n_pages;
  w->max_q = w->max_kv = 0x7fffffff;
  return FAK_OK;
}

// FAK_OK when the current device is sm_103.  The device's number into *dev, its SM count into *sms (either may
// be null).  What a device is does not change: looked up once.
static inline int kv_device(int* dev_out, int* sms) {
  static std::atomic<int> known[64];  // 0: not looked up; SM count + 1, or -1 when it is another kind
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fak_cuda_status(e);
  if (dev < 0 || dev >= 64) return FAK_ERR_UNSUPPORTED;
  int k = known[dev].load(std::memory_order_relaxed);
  if (k == 0) {
    int major = 0, minor = 0, count = 0;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, dev);
    k = major == 10 && minor == 3 ? count + 1 : -1;
    known[dev].store(k, std::memory_order_relaxed);
  }
  if (k < 0) return FAK_ERR_UNSUPPORTED;
  if (dev_out) *dev_out = dev;
  if (sms) *sms = k - 1;
  return FAK_OK;
}

// Raises a kernel's shared memory limit on device `dev` at its first launch there.
template <typename K>
static inline cudaError_t kv_smem_limit(K* kernel, int bytes, int dev, std::atomic<uint64_t>& done) {
  if (done.load(std::memory_order_relaxed) >> dev & 1) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}
