// The paged key-value cache: host checks and device helpers shared by the page
// operators (tv_pages.cu) and the attention that reads pages (tv_paged_attn.cu).
#pragma once

#include "tv_common.cuh"

namespace tv {

constexpr int kMaxListed = 4096;     // sequences one call may list
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

}  // namespace tv
