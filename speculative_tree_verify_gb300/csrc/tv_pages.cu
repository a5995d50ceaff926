// Pages of a key-value cache: forking, extending with copy-on-write, releasing,
// compacting, and moving rows into and out of pages.
//
// The state is the caller's: refs[p] counts the sequences that hold page p (0 =
// free), a table row lists a sequence's pages in order, lens its tokens.  There
// is no free list to keep in step with the counts; pages are always taken
// lowest index first, which is found by scanning the counts (4 bytes a page,
// from L2), so the outcome is a function of the state alone.
//
// Every bookkeeping call checks its whole list before it changes anything: for
// short lists one block looks, meets and acts; for long ones a first kernel
// looks and the next act only while the status word is zero.
#include "tv_kernels.cuh"
#include "tv_pages.cuh"

namespace tv {
namespace {

constexpr int kSeqThreads = 1024;    // of those that follow a sequence's pages: few rounds of dependent loads
constexpr int kPlanThreads = 1024;   // the one block that allocates

// ---- releasing and forking ---------------------------------------------------
// Releasing (FORK = false: a = ids, b = keep) or forking (a = src, b = dst): one
// block per listed sequence.  A block is a chain of dependent loads (list,
// length, entries, counts), so the first entries, kPer a thread, are asked for
// with the length, and kPer counts are on their way at once.
constexpr int kPer = 4;
struct Entries {   // of places j0 + thread + kSeqThreads u of a table row
  int e[kPer];
  __device__ __forceinline__ void load(const int32_t* row, int j0, int end) {
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int j = j0 + (int)threadIdx.x + u * kSeqThreads;
      e[u] = j < end ? __ldcg(row + j) : -1;
    }
  }
  template <class F>
  __device__ __forceinline__ void each(int j0, int first, int last, F f) const {
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int j = j0 + (int)threadIdx.x + u * kSeqThreads;
      if (j >= first && j < last) f(u, j, e[u]);
    }
  }
};

// indexes, lengths and page entries in range, no index listed twice; forking:
// no target among the sources, every target empty
template <bool FORK>
__global__ void __launch_bounds__(kSeqThreads) list_check_kernel(tv_pool pool, tv_seqs t, const int32_t* a,
                                                                 const int32_t* b, int n, int32_t* status) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x, ps = pool.page_size;
  const int s = a[i], d = b[i];   // d: the target row, or the tokens kept
  int bad = 0;
  if (s < 0 || s >= t.max_seqs || (FORK && (d < 0 || d >= t.max_seqs))) {
    bad = TV_E_SEQ;
  } else {
    const int32_t* row = t.pages + (size_t)s * t.max_pages;
    Entries x;
    x.load(row, 0, t.max_pages);
    const int len = seq_len(t, ps, s), there = FORK ? __ldcg(t.lens + d) : 0;
    for (int j = threadIdx.x; j < n; j += kSeqThreads)
      if (FORK ? (j != i && b[j] == d) || a[j] == d : j != i && a[j] == s) bad = TV_E_SEQ;
    if (len < 0 || there != 0 || (!FORK && (d < 0 || d > len))) {
      bad = TV_E_SEQ;
    } else {
      const int first = FORK ? 0 : pages_of(d, ps), last = pages_of(len, ps);
      for (long long j0 = 0; j0 < last; j0 += kPer * kSeqThreads) {
        if (j0 > 0) x.load(row, (int)j0, last);
        int held[kPer];
        x.each((int)j0, 0, last, [&](int u, int, int p) {
          held[u] = p >= 0 && p < pool.n_pages ? __ldcg(pool.refs + p) : 0;
        });
        x.each((int)j0, first, last, [&](int u, int, int) {
          if (held[u] < 1) bad = TV_E_PAGE;
        });
      }
    }
  }
  if (bad) status_set(status, bad);
}

template <bool FORK>
__global__ void __launch_bounds__(kSeqThreads) list_apply_kernel(tv_pool pool, tv_seqs t, const int32_t* a,
                                                                 const int32_t* b, int n, int32_t* status) {
  pdl_wait();
  pdl_trigger();
  const int stop = status_get(status), ps = pool.page_size;
  const int s = a[blockIdx.x], d = b[blockIdx.x];
  const bool in = s >= 0 && s < t.max_seqs && (!FORK || (d >= 0 && d < t.max_seqs));   // false only where it stops
  Entries x;
  int len = 0;
  if (in) {
    x.load(t.pages + (size_t)s * t.max_pages, 0, t.max_pages);
    len = __ldcg(t.lens + s);
  }
  // Samples of one source stand next to each other: the first of a run counts
  // its pages for all of them.
  int count = 1;
  if (FORK) {
    const int i = blockIdx.x, lane = threadIdx.x & 31;
    if (i > 0 && a[i - 1] == s) count = 0;
    for (int j = i + 1; count > 0; j += 32) {
      const unsigned other = __ballot_sync(0xffffffffu, j + lane >= n || a[j + lane] != s);
      count += other ? __ffs(other) - 1 : 32;
      if (other) break;
    }
  }
  if (__syncthreads_or(stop != 0 || !in)) return;   // from here on every thread has the old length
  const int first = FORK ? 0 : pages_of(d, ps), last = pages_of(len, ps);
  for (long long j0 = 0; j0 < last; j0 += kPer * kSeqThreads) {
    if (j0 > 0) x.load(t.pages + (size_t)s * t.max_pages, (int)j0, last);
    x.each((int)j0, first, last, [&](int, int j, int p) {
      if (FORK) t.pages[(size_t)d * t.max_pages + j] = p;
      if (count > 0) atomicAdd(pool.refs + p, FORK ? count : -1);
    });
  }
  if (threadIdx.x == 0) t.lens[FORK ? d : s] = FORK ? len : d;
}

// The same by one block, a warp a listed sequence, which holds its table
// entries in registers between the look and the act.  Such a call is a chain of dependent
// loads (list, length and entries, counts), about 0.6 us each, and its
// launches, 2 to 3 us each; one SM's atomics are what it can run out of.  A
// pass of release, fork, extend, release took, by one block against two
// launches a call: 14.5 against 18.1 us for 8 sequences of 65 pages, but 24.0
// against 18.2 us for 8 of 494 and 40.3 against 23.6 us for 32 of 494.
constexpr int kBlockThreads = 1024;
constexpr int kWarpEntries = 512;     // table entries a warp's registers hold
constexpr int kBlockEntries = 1024;   // and those a block takes on
inline bool one_block(const tv_seqs& t, int n) {
  return n <= kBlockThreads / 32 && t.max_pages <= kWarpEntries && n * t.max_pages <= kBlockEntries;
}

template <bool FORK>
__global__ void __launch_bounds__(kBlockThreads) list_block_kernel(tv_pool pool, tv_seqs t, const int32_t* a,
                                                                   const int32_t* b, int n, int32_t* status) {
  const int lane = threadIdx.x & 31, i = threadIdx.x >> 5, ps = pool.page_size;
  pdl_wait();
  pdl_trigger();
  const bool skip = status_get(status) != 0;
  int bad = 0, s = 0, d = 0, len = 0, first = 0, last = 0;
  int e[kWarpEntries / 32];
  if (i < n) {
    s = __ldg(a + i);
    d = __ldg(b + i);   // forking: the target row; releasing: the tokens kept
    if (s < 0 || s >= t.max_seqs || (FORK && (d < 0 || d >= t.max_seqs))) {
      bad = TV_E_SEQ;
    } else {
      const int32_t* row = t.pages + (size_t)s * t.max_pages;
#pragma unroll
      for (int k = 0; k < kWarpEntries / 32; ++k)   // with the length on its way
        if (lane + 32 * k < t.max_pages) e[k] = __ldcg(row + lane + 32 * k);
      len = seq_len(t, ps, s);
      if (len < 0 || (FORK ? __ldcg(t.lens + d) != 0 : d < 0 || d > len)) bad = TV_E_SEQ;
    }
    if (!bad) {
      first = FORK ? 0 : pages_of(d, ps);
      last = pages_of(len, ps);
#pragma unroll
      for (int k = 0; k < kWarpEntries / 32; ++k) {
        const int j = lane + 32 * k;
        if (j >= first && j < last && (e[k] < 0 || e[k] >= pool.n_pages || __ldcg(pool.refs + e[k]) < 1)) bad = TV_E_PAGE;
      }
    }
  }
  // no row listed twice; forking: no target among the sources (n <= 32: a lane a sequence)
  if (i == 0) {
    const int sa = lane < n ? __ldg(a + lane) : -1 - lane, sb = lane < n ? __ldg(b + lane) : -1 - lane;
    const bool twice = __popc(__match_any_sync(0xffffffffu, FORK ? sb : sa)) > 1;
    bool among = false;
    for (int k = 0; k < n; ++k) among = among | (sb == __shfl_sync(0xffffffffu, sa, k));
    if (lane < n && (twice || (FORK && among))) bad = TV_E_SEQ;
  }
  if (bad && !skip) status_set(status, bad);
  if (__syncthreads_or(bad) || skip || i >= n) return;
  int32_t* to = t.pages + (size_t)d * t.max_pages;
#pragma unroll
  for (int k = 0; k < kWarpEntries / 32; ++k) {
    const int j = lane + 32 * k;
    if (j >= first && j < last) {
      if (FORK) {
        to[j] = e[k];
        atomicAdd(pool.refs + e[k], 1);
      } else {
        atomicSub(pool.refs + e[k], 1);
      }
    }
  }
  if (lane == 0) t.lens[FORK ? d : s] = FORK ? len : d;
}

// ---- extending -----------------------------------------------------------------
// exclusive sum over the block's threads; *total = the sum of all
__device__ __forceinline__ int block_scan(int v, int* s_warp, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();   // the last call's readers are done with s_warp
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  int w = lane < kPlanThreads / 32 ? s_warp[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const int before = warp ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
  return before + x - v;
}

struct ExtendWs {
  int32_t* free_list;   // [n_pages]
  int32_t* pair;        // [2 * kMaxListed]: the copy of listed sequence i, source and target page, or -1
};

// One block.  Listed sequence i needs ceil((len + add) / page) - ceil(len / page)
// new pages, and one more where its last page is partly filled and shared: that
// page is copied, so that the new tokens' rows go into a page of its own.  In
// list order the last holder of a page keeps it, which with m listed holders of
// a page with r references means: all m copy, except that the last in the list
// keeps it when m = r.  The holders of a page are counted by comparing along
// the list in shared memory (n comparisons for each listed holder of a shared
// page, 4 at a time).
//
// The call is a chain of dependent loads (list, length, last entry, its count)
// beside which the first counts are already on their way for the search of
// free pages; nothing is written before the last check.
struct ExtendSmem {   // of n listed sequences, and a mark for every table row
  int *last, *off, *row, *len;
  uint32_t* mark;
  static size_t bytes(int n, int max_seqs) {
    return (size_t)((n + 3) & ~3) * 16 + (size_t)((max_seqs + 127) / 128) * 16;
  }
};
__global__ void __launch_bounds__(kPlanThreads) extend_plan_kernel(tv_pool pool, tv_seqs t, const int32_t* ids,
                                                                   const int32_t* add, int n, ExtendWs ws,
                                                                   int32_t* status) {
  extern __shared__ __align__(16) int s_dyn[];
  __shared__ int s_warp[32];
  __shared__ uint32_t s_bad;
  __shared__ unsigned long long s_need;     // pages needed in all
  constexpr int kCow = 1 << 30;
  const int tid = threadIdx.x, ps = pool.page_size, n4 = (n + 3) & ~3;
  ExtendSmem sm;
  sm.last = s_dyn;              // shared partly filled page of listed sequence i, or -1
  sm.off = s_dyn + n4;          // its need, then the offset of its new pages; bit 30: it copies
  sm.row = s_dyn + 2 * n4;      // its table row
  sm.len = s_dyn + 3 * n4;      // its length
  sm.mark = reinterpret_cast<uint32_t*>(s_dyn + 4 * n4);
  for (int i = tid; i < (t.max_seqs + 31) / 32; i += kPlanThreads) sm.mark[i] = 0u;
  if (tid == 0) s_bad = 0u, s_need = 0;
  if (tid < n4 - n) sm.last[n + tid] = -1;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  auto counts = [&](int p0) {   // of pages p0 + 4 tid .. + 3; past the pool: held
    const int p = p0 + 4 * tid;
    int4 r = make_int4(1, 1, 1, 1);
    if (p + 3 < pool.n_pages) {
      r = __ldcg(reinterpret_cast<const int4*>(pool.refs + p));
    } else {
      if (p < pool.n_pages) r.x = __ldcg(pool.refs + p);
      if (p + 1 < pool.n_pages) r.y = __ldcg(pool.refs + p + 1);
      if (p + 2 < pool.n_pages) r.z = __ldcg(pool.refs + p + 2);
    }
    return r;
  };
  const int skip = status_get(status);
  int4 r = counts(0);
  for (int i = tid; i < n; i += kPlanThreads) {
    const int s = __ldg(ids + i), a = __ldg(add + i);
    uint32_t bad = 0u;
    int last = -1, len = 0;
    if (s < 0 || s >= t.max_seqs || (atomicOr(&sm.mark[s >> 5], 1u << (s & 31)) >> (s & 31)) & 1u) {
      bad = kBadSeq;
    } else {
      len = seq_len(t, ps, s);
      if (len < 0 || a < 0) bad = kBadSeq;
      else if (a > t.max_pages * ps - len) bad = kBadCapacity;
      else if (a > 0 && len % ps != 0) {
        const int p = __ldcg(t.pages + (size_t)s * t.max_pages + len / ps);
        const int held = p >= 0 && p < pool.n_pages ? __ldcg(pool.refs + p) : 0;
        if (held < 1) bad = kBadPage;
        else if (held > 1) last = p;
      }
    }
    sm.last[i] = last;
    sm.row[i] = s;
    sm.len[i] = len;
    if (bad) atomicOr(&s_bad, bad);
  }
  __syncthreads();
  for (int i = tid; i < n && !s_bad; i += kPlanThreads) {
    const int len = sm.len[i], p = sm.last[i];
    int need = pages_of(len + __ldg(add + i), ps) - pages_of(len, ps);   // below 2^28: a table row holds 2^31 - 1 tokens
    bool cow = false;
    if (p >= 0) {
      int holders = 0, after = 0;
      for (int k = 0; k < n4; k += 4) {
        const int4 q = *reinterpret_cast<const int4*>(sm.last + k);
        holders += (q.x == p) + (q.y == p) + (q.z == p) + (q.w == p);
        after += (q.x == p && k > i) + (q.y == p && k + 1 > i) + (q.z == p && k + 2 > i) + (q.w == p && k + 3 > i);
      }
      const int held = __ldcg(pool.refs + p);
      if (holders > held) atomicOr(&s_bad, kBadPage);   // more holders than references
      cow = holders < held || after > 0;
      need += cow;
    }
    atomicAdd(&s_need, (unsigned long long)need);
    sm.off[i] = need | (cow ? kCow : 0);
  }
  __syncthreads();
  if (s_bad || skip) {
    if (tid == 0 && !skip) status_set(status, bad_code(s_bad));
    return;
  }
  const bool fits = s_need <= (unsigned long long)pool.n_pages;
  const int total = fits ? (int)s_need : 0;
  int carry = 0;
  for (int i0 = 0; i0 < n && total > 0; i0 += kPlanThreads) {   // needs -> offsets
    const int i = i0 + tid;
    const int v = i < n ? sm.off[i] : 0;
    int sum;
    const int off = carry + block_scan(v & ~kCow, s_warp, &sum);
    if (i < n) sm.off[i] = off | (v & kCow);
    carry += sum;
  }
  // the lowest free pages, in order
  int found = 0;
  for (int p0 = 0; p0 < pool.n_pages && found < total; p0 += 4 * kPlanThreads) {
    if (p0 > 0) r = counts(p0);
    const int p = p0 + 4 * tid;
    int got;
    int at = found + block_scan((r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0), s_warp, &got);
    if (r.x == 0 && at < total) ws.free_list[at] = p;
    at += r.x == 0;
    if (r.y == 0 && at < total) ws.free_list[at] = p + 1;
    at += r.y == 0;
    if (r.z == 0 && at < total) ws.free_list[at] = p + 2;
    at += r.z == 0;
    if (r.w == 0 && at < total) ws.free_list[at] = p + 3;
    found += got;
  }
  if (!fits || total > found) {
    if (tid == 0) status_set(status, TV_E_CAPACITY);
    return;
  }
  __syncthreads();
  for (int f = tid; f < total; f += kPlanThreads) {
    int lo = 0, hi = n - 1;   // the last sequence whose first new page is at or before f
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((sm.off[mid] & ~kCow) <= f) lo = mid;
      else hi = mid - 1;
    }
    const int k = f - (sm.off[lo] & ~kCow), cow = (sm.off[lo] & kCow) ? 1 : 0;
    const int page = ws.free_list[f];
    t.pages[(size_t)sm.row[lo] * t.max_pages + pages_of(sm.len[lo], ps) + k - cow] = page;
    pool.refs[page] = 1;
  }
  for (int i = tid; i < n; i += kPlanThreads) {
    const bool cow = total > 0 && (sm.off[i] & kCow);
    ws.pair[2 * i] = cow ? sm.last[i] : -1;
    ws.pair[2 * i + 1] = cow ? ws.free_list[sm.off[i] & ~kCow] : -1;
    if (cow) atomicSub(pool.refs + sm.last[i], 1);
    t.lens[sm.row[i]] = sm.len[i] + __ldg(add + i);
  }
}

// One page of one layer's K or V is one contiguous block of memory.  bytes: a
// multiple of 16 (16 tokens are 2048 bytes or more in bf16, 576 or more in 4
// bits); eight 16-byte loads a thread are in flight before the first store.
__device__ __forceinline__ void copy_block(const uint8_t* from, uint8_t* to, uint32_t bytes) {
  const uint4* a = reinterpret_cast<const uint4*>(from);
  uint4* b = reinterpret_cast<uint4*>(to);
  const uint32_t n = bytes / 16;
  for (uint32_t i0 = 0; i0 < n; i0 += 8 * blockDim.x) {
    uint4 x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t i = i0 + u * blockDim.x + threadIdx.x;
      if (i < n) x[u] = __ldcg(a + i);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t i = i0 + u * blockDim.x + threadIdx.x;
      if (i < n) b[i] = x[u];
    }
  }
}
__device__ __forceinline__ void copy_page(const PagePool& pool, int layer, bool is_v, int src, int dst) {
  constexpr size_t kPiece = size_t(1) << 31;   // a page of very many heads passes 2^32 bytes
  const size_t bytes = (size_t)pool.n_kv_heads * pool.page_size * pool.row_bytes;
  uint8_t* base = reinterpret_cast<uint8_t*>(is_v ? pool.v : pool.k) + (size_t)layer * pool.n_pages * bytes;
  for (size_t at = 0; at < bytes; at += kPiece)
    copy_block(base + (size_t)src * bytes + at, base + (size_t)dst * bytes + at,
               (uint32_t)(bytes - at < kPiece ? bytes - at : kPiece));
}

// grid (listed sequences, 2 layers): the copies of extend_plan_kernel
__global__ void __launch_bounds__(kListThreads) extend_copy_kernel(PagePool pool, ExtendWs ws, int32_t* status) {
  pdl_wait();
  pdl_trigger();
  if (block_skip(status)) return;
  const int src = __ldcg(ws.pair + 2 * blockIdx.x), dst = __ldcg(ws.pair + 2 * blockIdx.x + 1);
  if (src < 0) return;
  for (int y = blockIdx.y; y < 2 * pool.n_layers; y += gridDim.y) copy_page(pool, y >> 1, y & 1, src, dst);
}

// ---- compacting ------------------------------------------------------------------
struct CompactWs {
  int32_t* src;     // [n_pages]
  int32_t* dst;     // [n_pages]
  int32_t* moves;   // [1]
};

// Block 0: with U pages used, the k-th used page at or past U moves to the
// k-th free page below U (as many of the one as of the other).  The other
// blocks check the live table entries.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(tv_pool pool, tv_seqs t, CompactWs ws,
                                                                    int32_t* status) {
  __shared__ int s_warp[32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  if (blockIdx.x > 0) {
    int bad = 0;
    for (int s = blockIdx.x - 1; s < t.max_seqs; s += gridDim.x - 1) {
      const int len = seq_len(t, pool.page_size, s);
      if (len < 0) {
        bad = TV_E_SEQ;
        continue;
      }
      const int32_t* row = t.pages + (size_t)s * t.max_pages;
      for (int j = tid; j < pages_of(len, pool.page_size); j += kPlanThreads) {
        const int p = __ldcg(row + j);
        if (p < 0 || p >= pool.n_pages || __ldcg(pool.refs + p) < 1) bad = TV_E_PAGE;
      }
    }
    if (bad) status_set(status, bad);
    return;
  }
  int mine = 0, bad = 0;
  for (int p = tid; p < pool.n_pages; p += kPlanThreads) {
    const int r = __ldcg(pool.refs + p);
    mine += r > 0;
    if (r < 0) bad = TV_E_PAGE;
  }
  if (bad) status_set(status, bad);
  int used;
  block_scan(mine, s_warp, &used);
  int n_src = 0, n_dst = 0;
  for (int p0 = 0; p0 < pool.n_pages; p0 += kPlanThreads) {
    const int p = p0 + tid;
    const bool in = p < pool.n_pages;
    const bool held = in && __ldcg(pool.refs + p) > 0;
    const bool move = held && p >= used, hole = in && !held && p < used;
    int got;
    // a page is one or the other, and below used only holes, past it only moves
    const int at = block_scan((move ? 1 : 0) | (hole ? 1 << 16 : 0), s_warp, &got);
    if (move) ws.src[n_src + (at & 0xffff)] = p;
    if (hole) ws.dst[n_dst + (at >> 16)] = p;
    n_src += got & 0xffff;
    n_dst += got >> 16;
  }
  if (tid == 0) {
    ws.moves[0] = n_src;
    ws.moves[1] = used;
  }
}

__global__ void __launch_bounds__(kListThreads) compact_remap_kernel(tv_pool pool, CompactWs ws, int32_t* remap,
                                                                     int32_t* n_used, int32_t* status) {
  pdl_wait();
  pdl_trigger();
  if (block_skip(status)) return;
  const int moves = __ldcg(ws.moves), used = __ldcg(ws.moves + 1);
  const int stride = gridDim.x * kListThreads;
  const int i0 = blockIdx.x * kListThreads + threadIdx.x;
  if (i0 == 0) *n_used = used;
  // pages below `used` that are held stay; holes and pages past it are free afterwards ...
  for (int p = i0; p < pool.n_pages; p += stride) {
    const bool held = __ldcg(pool.refs + p) > 0;
    if (!held || p < used) remap[p] = held ? p : -1;
  }
  // ... and the moves say where the held ones past it go
  for (int i = i0; i < moves; i += stride) remap[__ldcg(ws.src + i)] = __ldcg(ws.dst + i);
}

// The moves (no target is a source: targets lie below `used`, sources past it),
// the tables, then the counts of the moved pages.
__global__ void __launch_bounds__(kListThreads) compact_move_kernel(PagePool pool, tv_seqs t, CompactWs ws,
                                                                    const int32_t* remap, int32_t* status) {
  pdl_wait();
  pdl_trigger();
  if (block_skip(status)) return;
  const int moves = __ldcg(ws.moves);
  const long long items = (long long)moves * 2 * pool.n_layers;
  for (int s = blockIdx.x; s < t.max_seqs; s += gridDim.x) {
    const int np = pages_of(__ldcg(t.lens + s), pool.page_size);
    int32_t* row = t.pages + (size_t)s * t.max_pages;
    for (int j = threadIdx.x; j < np; j += kListThreads) row[j] = __ldcg(remap + __ldcg(row + j));
  }
  for (int i = blockIdx.x * kListThreads + threadIdx.x; i < moves; i += gridDim.x * kListThreads) {
    const int a = __ldcg(ws.src + i), b = __ldcg(ws.dst + i);
    pool.refs[b] = __ldcg(pool.refs + a);
    pool.refs[a] = 0;
  }
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int y = (int)(it / moves), i = (int)(it % moves);
    copy_page(pool, y >> 1, y & 1, __ldcg(ws.src + i), __ldcg(ws.dst + i));
  }
}

// ---- rows into pages and out of them ---------------------------------------------
// One warp per row; a row's K and V are each n_kv_heads pieces of head_dim
// values, contiguous per head on both sides.
//
// A bad page entry leaves out its rows alone.  Blocks that have yet to start
// would take the status it is reported by for an earlier call's and leave out
// theirs as well, so a call of more than one block reports by a kernel of its
// own behind the moves (rows_report_kernel).
template <bool WRITE>
__global__ void __launch_bounds__(kListThreads) rows_kernel(tv_pool pool, int layer, tv_seqs t, RowList list,
                                                            __nv_bfloat16* k, __nv_bfloat16* v, size_t row_stride,
                                                            size_t head_stride, int32_t* status) {
  __shared__ int s_start[kMaxListed + 1];
  __shared__ uint32_t s_bad;
  extern __shared__ uint32_t s_mark[];   // WRITE: a bit per table row
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, ps = pool.page_size;
  if (block_skip(status)) return;
  if (!look_over<WRITE>(t, ps, list, s_start, s_mark, &s_bad, status)) return;
  const int first = s_start[0], total = s_start[list.n];
  const int lane = tid & 31;
  const int pieces = pool.n_kv_heads * (pool.head_dim / 8);   // 16-byte pieces of a row's K
  const int dsh = pool.head_dim == 128 ? 4 : 3;
  const size_t page_elems = (size_t)pool.n_kv_heads * ps * pool.head_dim;
  __nv_bfloat16 *pk = reinterpret_cast<__nv_bfloat16*>(pool.k), *pv = reinterpret_cast<__nv_bfloat16*>(pool.v);
  // (unsigned: a count near 2^31 and a stride do not wrap)
  for (uint32_t r = first + blockIdx.x * (kListThreads / 32) + (tid >> 5); r < (uint32_t)total;
       r += gridDim.x * (kListThreads / 32)) {
    const int i = sequence_of(s_start, list.n, r);
    const int at = __ldg(list.pos + i) + (int)r - s_start[i];
    const int p = __ldcg(t.pages + (size_t)__ldg(list.ids + i) * t.max_pages + at / ps);
    if (p < 0 || p >= pool.n_pages) {
      if (gridDim.x == 1 && lane == 0) status_set(status, TV_E_PAGE);
      continue;
    }
    const size_t base = ((size_t)layer * pool.n_pages + p) * page_elems + (size_t)(at % ps) * pool.head_dim;
    for (int c0 = 0; c0 < pieces; c0 += 4 * 32) {
      uint4 x[8];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int c = c0 + u * 32 + lane;
        if (c < pieces) {
          const int h = c >> dsh, e = (c & ((1 << dsh) - 1)) * 8;
          const size_t in_page = base + (size_t)h * ps * pool.head_dim + e;
          const size_t in_rows = (size_t)r * row_stride + (size_t)h * head_stride + e;
          x[2 * u] = __ldcg(reinterpret_cast<const uint4*>(WRITE ? k + in_rows : pk + in_page));
          x[2 * u + 1] = __ldcg(reinterpret_cast<const uint4*>(WRITE ? v + in_rows : pv + in_page));
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int c = c0 + u * 32 + lane;
        if (c < pieces) {
          const int h = c >> dsh, e = (c & ((1 << dsh) - 1)) * 8;
          const size_t in_page = base + (size_t)h * ps * pool.head_dim + e;
          const size_t in_rows = (size_t)r * row_stride + (size_t)h * head_stride + e;
          *reinterpret_cast<uint4*>(WRITE ? pk + in_page : k + in_rows) = x[2 * u];
          *reinterpret_cast<uint4*>(WRITE ? pv + in_page : v + in_rows) = x[2 * u + 1];
        }
      }
    }
  }
}

// The entries of the rows of rows_kernel, looked at while it moves them: it
// triggers behind its own wait, so what it reads is there when this kernel
// starts.  Lists that it refuses reach no entry here that they name wrongly,
// and have set the status.
__global__ void __launch_bounds__(kListThreads) rows_report_kernel(int n_pages, int ps, tv_seqs t, RowList l,
                                                                   int32_t* status) {
  bool bad = false;
  for (int i = blockIdx.x; i < l.n; i += gridDim.x) {
    const int a = __ldcg(l.starts + i), b = __ldcg(l.starts + i + 1), s = __ldcg(l.ids + i), at = __ldcg(l.pos + i);
    if (a < 0 || b <= a || b > l.rows || s < 0 || s >= t.max_seqs || at < 0) continue;
    const int len = seq_len(t, ps, s);
    if ((long long)at + (b - a) > len) continue;
    const int last = (at + (b - a) - 1) / ps;
    for (int j = at / ps + (int)threadIdx.x; j <= last; j += kListThreads) {
      const int p = __ldcg(t.pages + (size_t)s * t.max_pages + j);
      bad = bad || p < 0 || p >= n_pages;
    }
  }
  pdl_wait();
  pdl_trigger();
  if (bad) status_set(status, TV_E_PAGE);   // (where the call was stopped, the word is set)
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

int rows_call(bool write, const tv_pool* pool, int layer, const tv_seqs* seqs, const RowList& l, void* k, void* v,
              size_t row_stride, size_t head_stride, int32_t* status, void* stream) {
  int rc = check_pool(pool);
  if (rc || (rc = check_rows(*pool, layer, seqs, l, k, v, row_stride, head_stride, status))) return rc;
  const int sms = num_sms();
  if (sms <= 0) return TV_E_CUDA;
  const int per = kListThreads / 32;
  const int want = (l.rows + per - 1) / per, most = sms * 8;
  const dim3 grid(want < 1 ? 1 : (want < most ? want : most));
  __nv_bfloat16 *kp = static_cast<__nv_bfloat16*>(k), *vp = static_cast<__nv_bfloat16*>(v);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const size_t smem = write ? (size_t)((seqs->max_seqs + 31) / 32) * 4 : 0;
  rc = launch_pdl(write ? rows_kernel<true> : rows_kernel<false>, grid, dim3(kListThreads), smem, st, *pool, layer, *seqs,
                  l, kp, vp, row_stride, head_stride, status);
  if (rc || grid.x == 1) return rc;
  return launch_rows_report(*pool, *seqs, l, sms, status, st);
}

}  // namespace

int check_rows(const tv_pool& pool, int layer, const tv_seqs* seqs, const RowList& l, const void* k, const void* v,
               size_t row_stride, size_t head_stride, const int32_t* status) {
  int rc = check_seqs(seqs, &pool);
  if (rc) return rc;
  if (!l.ids || !l.pos || !l.starts || !k || !v || !status || layer < 0 || layer >= pool.n_layers || l.rows < 0) return TV_E_ARG;
  if ((rc = check_listed(l.n))) return rc;
  // 16-byte pieces on both sides
  return !aligned16(k) || !aligned16(v) || row_stride % 8 != 0 || head_stride % 8 != 0 ? TV_E_ARG : TV_OK;
}

int launch_rows_report(const tv_pool& pool, const tv_seqs& seqs, const RowList& l, int sms, int32_t* status,
                       cudaStream_t st) {
  return launch_pdl(rows_report_kernel, dim3(l.n < sms ? l.n : sms), dim3(kListThreads), 0, st, pool.n_pages,
                    pool.page_size, seqs, l, status);
}

// extend: the free list and the pairs; compact: two page lists and two counts
size_t pages_ws_bytes(const tv_pool& p) {
  return align256((size_t)p.n_pages * 4) * 2 + align256(2 * kMaxListed * 4);
}

int pages_release(const PagePool& pool, const tv_seqs* seqs, const int32_t* ids, const int32_t* keep, int n,
                  int32_t* dev_status, void* stream) {
  int rc = check_seqs(seqs, &pool);
  if (rc) return rc;
  if (!ids || !keep || !dev_status) return TV_E_ARG;
  if ((rc = check_listed(n))) return rc;
  const tv_pool p = pool;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (one_block(*seqs, n))
    return launch_pdl(list_block_kernel<false>, dim3(1), dim3(kBlockThreads), 0, st, p, *seqs, ids, keep, n, dev_status);
  rc = launch_pdl(list_check_kernel<false>, dim3(n), dim3(kSeqThreads), 0, st, p, *seqs, ids, keep, n, dev_status);
  if (rc) return rc;
  return launch_pdl(list_apply_kernel<false>, dim3(n), dim3(kSeqThreads), 0, st, p, *seqs, ids, keep, n, dev_status);
}

int pages_fork(const PagePool& pool, const tv_seqs* seqs, const int32_t* src, const int32_t* dst, int n,
               int32_t* dev_status, void* stream) {
  int rc = check_seqs(seqs, &pool);
  if (rc) return rc;
  if (!src || !dst || !dev_status) return TV_E_ARG;
  if ((rc = check_listed(n))) return rc;
  const tv_pool p = pool;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (one_block(*seqs, n))
    return launch_pdl(list_block_kernel<true>, dim3(1), dim3(kBlockThreads), 0, st, p, *seqs, src, dst, n, dev_status);
  rc = launch_pdl(list_check_kernel<true>, dim3(n), dim3(kSeqThreads), 0, st, p, *seqs, src, dst, n, dev_status);
  if (rc) return rc;
  return launch_pdl(list_apply_kernel<true>, dim3(n), dim3(kSeqThreads), 0, st, p, *seqs, src, dst, n, dev_status);
}

int pages_extend(const PagePool& pool, const tv_seqs* seqs, const int32_t* ids, const int32_t* add, int n,
                 void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  int rc = check_seqs(seqs, &pool);
  if (rc) return rc;
  if (!ids || !add || !dev_status) return TV_E_ARG;
  if ((rc = check_listed(n))) return rc;
  if (!workspace || workspace_bytes < pages_ws_bytes(pool) || !aligned16(workspace)) return TV_E_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(workspace);
  ExtendWs ws;
  ws.free_list = reinterpret_cast<int32_t*>(w);
  ws.pair = reinterpret_cast<int32_t*>(w + 2 * align256((size_t)pool.n_pages * 4));
  static std::atomic<bool> attr[64];
  if (ensure_smem_limit(extend_plan_kernel, ExtendSmem::bytes(kMaxListed, kMaxSeqs), attr)) return TV_E_CUDA;
  rc = launch_pdl(extend_plan_kernel, dim3(1), dim3(kPlanThreads), ExtendSmem::bytes(n, seqs->max_seqs), st,
                  static_cast<const tv_pool&>(pool), *seqs, ids, add, n, ws, dev_status);
  if (rc) return rc;
  const int y = 2 * pool.n_layers < 65535 ? 2 * pool.n_layers : 65535;
  return launch_pdl(extend_copy_kernel, dim3(n, y), dim3(kListThreads), 0, st, pool, ws, dev_status);
}

int pages_compact(const PagePool& pool, const tv_seqs* seqs, int32_t* remap, int32_t* n_used, void* workspace,
                  size_t workspace_bytes, int32_t* dev_status, void* stream) {
  int rc = check_seqs(seqs, &pool);
  if (rc) return rc;
  if (!remap || !n_used || !dev_status) return TV_E_ARG;
  if (!workspace || workspace_bytes < pages_ws_bytes(pool) || !aligned16(workspace)) return TV_E_WORKSPACE;
  const int sms = num_sms();
  if (sms <= 0) return TV_E_CUDA;
  const tv_pool p = pool;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(workspace);
  CompactWs ws;
  ws.src = reinterpret_cast<int32_t*>(w);
  ws.dst = reinterpret_cast<int32_t*>(w + align256((size_t)pool.n_pages * 4));
  ws.moves = reinterpret_cast<int32_t*>(w + 2 * align256((size_t)pool.n_pages * 4));
  const int checks = seqs->max_seqs < sms - 1 ? seqs->max_seqs : sms - 1;
  rc = launch_pdl(compact_plan_kernel, dim3(1 + checks), dim3(kPlanThreads), 0, st, p, *seqs, ws, dev_status);
  if (rc) return rc;
  const int rb = (pool.n_pages + kListThreads - 1) / kListThreads;
  rc = launch_pdl(compact_remap_kernel, dim3(rb < sms ? rb : sms), dim3(kListThreads), 0, st, p, ws, remap, n_used,
                  dev_status);
  if (rc) return rc;
  return launch_pdl(compact_move_kernel, dim3(sms * 8), dim3(kListThreads), 0, st, pool, *seqs, ws,
                    (const int32_t*)remap, dev_status);
}

}  // namespace tv

using namespace tv;

extern "C" {

int tv_pages_workspace_size(const tv_pool* pool, const tv_seqs* seqs, size_t* bytes) {
  int rc = check_pool(pool);
  if (rc || (rc = check_seqs(seqs, pool))) return rc;
  if (!bytes) return TV_E_ARG;
  *bytes = pages_ws_bytes(*pool);
  return TV_OK;
}

int tv_pages_release(const tv_pool* pool, const tv_seqs* seqs, const int32_t* ids, const int32_t* keep, int n,
                     int32_t* dev_status, void* stream) {
  const int rc = check_pool(pool);
  return rc ? rc : pages_release(page_pool(*pool), seqs, ids, keep, n, dev_status, stream);
}

int tv_pages_fork(const tv_pool* pool, const tv_seqs* seqs, const int32_t* src, const int32_t* dst, int n,
                  int32_t* dev_status, void* stream) {
  const int rc = check_pool(pool);
  return rc ? rc : pages_fork(page_pool(*pool), seqs, src, dst, n, dev_status, stream);
}

int tv_pages_extend(const tv_pool* pool, const tv_seqs* seqs, const int32_t* ids, const int32_t* add, int n,
                    void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  const int rc = check_pool(pool);
  return rc ? rc : pages_extend(page_pool(*pool), seqs, ids, add, n, workspace, workspace_bytes, dev_status, stream);
}

int tv_pages_compact(const tv_pool* pool, const tv_seqs* seqs, int32_t* remap, int32_t* n_used, void* workspace,
                     size_t workspace_bytes, int32_t* dev_status, void* stream) {
  const int rc = check_pool(pool);
  return rc ? rc : pages_compact(page_pool(*pool), seqs, remap, n_used, workspace, workspace_bytes, dev_status, stream);
}

int tv_pages_write(const tv_pool* pool, int layer, const tv_seqs* seqs, const int32_t* ids, const int32_t* pos,
                   const int32_t* starts, int n, int rows, const tv_bf16* k, const tv_bf16* v, size_t row_stride,
                   size_t head_stride, int32_t* dev_status, void* stream) {
  return rows_call(true, pool, layer, seqs, RowList{ids, pos, starts, n, rows}, const_cast<tv_bf16*>(k),
                   const_cast<tv_bf16*>(v), row_stride, head_stride, dev_status, stream);
}

int tv_pages_read(const tv_pool* pool, int layer, const tv_seqs* seqs, const int32_t* ids, const int32_t* pos,
                  const int32_t* starts, int n, int rows, tv_bf16* k, tv_bf16* v, size_t row_stride,
                  size_t head_stride, int32_t* dev_status, void* stream) {
  return rows_call(false, pool, layer, seqs, RowList{ids, pos, starts, n, rows}, k, v, row_stride, head_stride,
                   dev_status, stream);
}

}  // extern "C"
