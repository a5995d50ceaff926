// The paged key-value cache: host checks and device helpers shared by the page
// operators (tv_pages.cu) and the attention that reads pages (tv_paged_attn.cu).
#pragma once

#include "tv_common.cuh"

namespace tv {

constexpr int kMaxListed = 4096;     // sequences one call may list
constexpr int kListThreads = 256;    // block of the kernels that move rows and pages
constexpr int kMaxSeqs = 65536;      // rows of a sequence table (their marks fit a block's shared memory)

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// tokens per page: a power of two that whole tiles are made of
inline int check_pool(const tv_pool* p) {
  if (!p || !p->k || !p->v || !p->refs || !aligned16(p->k) || !aligned16(p->v) || !aligned16(p->refs)) return TV_E_ARG;
  if (p->n_layers < 1 || p->n_pages < 1 || p->n_kv_heads < 1) return TV_E_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return TV_E_UNSUPPORTED;
  if (p->page_size != 16 && p->page_size != 32 && p->page_size != 64 && p->page_size != 128) return TV_E_UNSUPPORTED;
  // the pool's rows are one tensor-map dimension, indexed by int32 coordinates
  unsigned long long rows = (unsigned long long)p->n_layers * (unsigned long long)p->n_pages;
  if (rows > 0x7fffffffull) return TV_E_UNSUPPORTED;
  rows *= (unsigned long long)p->n_kv_heads;
  if (rows > 0x7fffffffull || rows * (unsigned long long)p->page_size > 0x7fffffffull) return TV_E_UNSUPPORTED;
  return TV_OK;
}

// A pool of either kind as the calls that only move its bytes see it: every
// token's head is row_bytes of K and of V, a page of a layer one block of them.
struct PagePool : tv_pool {
  int32_t row_bytes;
};

inline PagePool page_pool(const tv_pool& p) {
  PagePool q;
  static_cast<tv_pool&>(q) = p;
  q.row_bytes = p.head_dim * 2;
  return q;
}

// in 4 bits: head_dim / 2 bytes of codes and a bf16 scale for every 32 of them
inline int row_bytes4(int head_dim) { return head_dim / 2 + head_dim / 32 * 2; }

inline int check_pool(const tv_pool4* p, PagePool* q) {
  if (!p) return TV_E_ARG;
  *q = PagePool{};
  q->k = reinterpret_cast<tv_bf16*>(p->k);
  q->v = reinterpret_cast<tv_bf16*>(p->v);
  q->refs = p->refs;
  q->n_layers = p->n_layers;
  q->n_pages = p->n_pages;
  q->n_kv_heads = p->n_kv_heads;
  q->page_size = p->page_size;
  q->head_dim = p->head_dim;
  q->row_bytes = row_bytes4(p->head_dim);
  return check_pool(q);
}

inline int check_seqs(const tv_seqs* s, const tv_pool* p) {
  if (!s || !s->pages || !s->lens || s->max_seqs < 1 || s->max_pages < 1) return TV_E_ARG;
  if (s->max_seqs > kMaxSeqs || (long long)s->max_pages * p->page_size > 0x7fffffffll) return TV_E_UNSUPPORTED;
  return TV_OK;
}

inline int check_listed(int n) { return n < 1 ? TV_E_ARG : (n > kMaxListed ? TV_E_UNSUPPORTED : TV_OK); }

// (a length may be near 2^31: nothing is added to it)
__device__ __forceinline__ int pages_of(int len, int page_size) { return len / page_size + (len % page_size != 0); }

// a sequence's length if its table row allows it, -1 otherwise
__device__ __forceinline__ int seq_len(const tv_seqs& t, int page_size, int s) {
  const int len = __ldcg(t.lens + s);
  return len >= 0 && len <= t.max_pages * page_size ? len : -1;
}

// what a block found wrong with its list; the lowest bit is reported, so that
// the code does not depend on the order of the threads
constexpr uint32_t kBadSeq = 1u, kBadCapacity = 2u, kBadPage = 4u;
__device__ __forceinline__ int bad_code(uint32_t bad) {
  return bad & kBadSeq ? TV_E_SEQ : (bad & kBadCapacity ? TV_E_CAPACITY : TV_E_PAGE);
}

// ---- rows into pages and out of them: what the kernels for either pool share ----
// Row r of listed sequence i (starts[i] <= r < starts[i + 1]) is token
// pos[i] + r - starts[i].
struct RowList {
  const int32_t *ids, *pos, *starts;
  int n, rows;
};

// Every block checks the whole list before it moves a row: true if it may.
// s_start: [n + 1]; s_mark (ONCE: a sequence may be listed once): a bit per
// table row.  All of the block's threads call it; they meet in it.
template <bool ONCE>
__device__ __forceinline__ bool look_over(const tv_seqs& t, int page_size, const RowList& l, int* s_start, uint32_t* s_mark,
                                          uint32_t* s_bad, int32_t* status) {
  const int tid = threadIdx.x;
  if (tid == 0) *s_bad = 0u;
  if (ONCE)
    for (int i = tid; i < (t.max_seqs + 31) / 32; i += kListThreads) s_mark[i] = 0u;
  __syncthreads();
  for (int i = tid; i <= l.n; i += kListThreads) {
    const int a = l.starts[i];
    s_start[i] = a;
    uint32_t bad = a < 0 || a > l.rows ? kBadSeq : 0u;
    if (i < l.n) {
      const int b = l.starts[i + 1], s = l.ids[i], at = l.pos[i];
      if (b < a || s < 0 || s >= t.max_seqs || at < 0) {
        bad = kBadSeq;
      } else {
        if (ONCE && (atomicOr(&s_mark[s >> 5], 1u << (s & 31)) >> (s & 31)) & 1u) bad = kBadSeq;
        const int len = seq_len(t, page_size, s);
        if (len < 0) bad = kBadSeq;
        else if ((long long)at + (b - a) > len) bad |= kBadCapacity;
      }
    }
    if (bad) atomicOr(s_bad, bad);
  }
  __syncthreads();
  if (*s_bad && tid == 0) status_set(status, bad_code(*s_bad));
  return *s_bad == 0u;
}

// the listed sequence of row r, starts[0] <= r < starts[n]
__device__ __forceinline__ int sequence_of(const int* s_start, int n, uint32_t r) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((uint32_t)s_start[mid] <= r) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// host checks of a call that moves rows, and the report of bad page entries
// behind its kernel (tv_pages.cu)
int check_rows(const tv_pool& pool, int layer, const tv_seqs* seqs, const RowList& l, const void* k, const void* v,
               size_t row_stride, size_t head_stride, const int32_t* status);
int launch_rows_report(const tv_pool& pool, const tv_seqs& seqs, const RowList& l, int sms, int32_t* status,
                       cudaStream_t st);

// ---- the page calls, for either pool (tv_pages.cu); the pool and seqs are checked ----
size_t pages_ws_bytes(const tv_pool& p);
int pages_release(const PagePool& pool, const tv_seqs* seqs, const int32_t* ids, const int32_t* keep, int n,
                  int32_t* dev_status, void* stream);
int pages_fork(const PagePool& pool, const tv_seqs* seqs, const int32_t* src, const int32_t* dst, int n,
               int32_t* dev_status, void* stream);
int pages_extend(const PagePool& pool, const tv_seqs* seqs, const int32_t* ids, const int32_t* add, int n,
                 void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream);
int pages_compact(const PagePool& pool, const tv_seqs* seqs, int32_t* remap, int32_t* n_used, void* workspace,
                  size_t workspace_bytes, int32_t* dev_status, void* stream);

}  // namespace tv
