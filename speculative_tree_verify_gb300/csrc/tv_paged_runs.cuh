// What the attentions of one new token over pages share (bf16 pages:
// tv_paged_attn.cu; 4 bits: tv_paged4_attn.cu): the list of work and the runs
// of a CTA, the workspace and the kernel that joins partial results.
//
// The work is the list of 64-token tiles of every (sequence, KV head, block of
// 16 query heads) in that order, each such head block counted SEG_COST tiles
// more for what it costs to begin and end; CTA c takes an equal, contiguous
// range of it, whatever the lengths, so one long context among short ones and
// one sequence alone both fill every SM.  A head block cut by a range border
// leaves unnormalised partials that paged_merge_kernel joins in tile order: no
// atomics, the same bits every run.
//
// Through a window (WIN) a sequence's tiles are those that hold a visible
// token: tile t of the list is tile t of the sequence among the sinks, and
// t + skip behind them.
#pragma once

#include "tv_kernels.cuh"
#include "tv_pages.cuh"

namespace tv {

constexpr int kTile = 64;                        // tokens of a tile
constexpr int kRows = 16;                        // query heads of a block
constexpr int kMaxTokens = 2048;                 // sequences of one call: their places fit beside the stages
constexpr int kInfo = 640;                       // up to here their table rows and lengths do, too
constexpr int kMaxCtas = 256;                    // partial slots reserved: 2 a CTA
static_assert(kInfo * 12 <= kMaxTokens * 4, "rows and lengths in the places of more sequences");

struct PaWs {
  int4* cut;          // [CTAs]: the head block whose first tile but not the last is the CTA's:
                      // listed index, head block, last CTA with a tile of it; -1: none
  float* ml;          // [2 CTAs][kRows][2]: offset and sum
  float* o;           // [2 CTAs][kRows][D]
};

struct PaParams {
  tv_pool pool;
  tv_seqs seqs;
  const int32_t* ids;
  const __nv_bfloat16 *q, *k_new, *v_new;
  size_t q_stride, kv_stride;
  __nv_bfloat16* out;
  int32_t* status;
  PaWs ws;
  int layer, n, Hq, G, HB;   // G query heads a KV head, in HB blocks of kRows
  int window, sinks;
  float scale_log2;
};

__device__ __forceinline__ float ex2f(float x) {   // 2^x by the SFU, about 2^-22 relative, 2^-inf = 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// untiled copy: 16-byte aligned addresses, a multiple of 16 bytes
__device__ __forceinline__ void bulk_load(void* smem_dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               :
               : "r"(smem_u32(smem_dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ int tiles_of(int len) { return len / kTile + (len % kTile != 0); }

// A run: tiles [t0, t1) of one sequence and head block.  The CTA's runs in
// order; a range may begin or end within a head block's fixed cost.
struct Run {
  int i, s, len, T;     // listed index, table row, length, tiles of the head block
  int h, hb, t0, t1;    // KV head, block of its query heads
  uint32_t base;        // place of tile 0
  int lo, sink_tiles, skip;   // WIN: first token of the window (0: nothing is hidden), tiles of the sinks before it
                              // and tiles between the two
  template <bool WIN>
  __device__ __forceinline__ int tile(int t) const {   // of the sequence
    return WIN && t >= sink_tiles ? t + skip : t;
  }
};

// THREADS: of the block.  The arrays are shared memory: first [n + 1], and up
// to kInfo sequences row and len [n].
template <int THREADS, int SEG_COST, bool WIN>
struct RunList {
  const PaParams& p;
  uint32_t* first;
  int *row, *len;
  bool info;
  uint32_t all, lo, hi, chunk;   // places in all; the CTA's range

  __device__ __forceinline__ RunList(const PaParams& params, uint32_t* s_first)
      : p(params), first(s_first), row(reinterpret_cast<int*>(s_first + params.n + 1)), len(row + params.n),
        info(params.n <= kInfo) {}

  __device__ __forceinline__ void window(Run& g) const {
    const int tiles = tiles_of(g.len);
    g.lo = g.sink_tiles = g.skip = 0;
    if constexpr (WIN) {
      if (g.len > p.window && g.len - p.window > p.sinks) {
        g.lo = g.len - p.window;
        g.sink_tiles = min(tiles_of(p.sinks), g.lo / kTile);
        g.skip = g.lo / kTile - g.sink_tiles;
      }
    }
    g.T = tiles - g.skip;
  }
  // of one head block, its fixed cost included; the host has seen to it that all fit 31 bits
  __device__ __forceinline__ uint32_t head_tiles(int length) const {
    if (length <= 0) return 0u;
    Run g;
    g.len = length;
    window(g);
    return (uint32_t)(g.T + SEG_COST);
  }
  __device__ __forceinline__ int look(int i, int& s) const {   // length of listed sequence i, -1: refused
    s = __ldg(p.ids + i);
    return s >= 0 && s < p.seqs.max_seqs ? seq_len(p.seqs, p.pool.page_size, s) : -1;
  }

  // Every CTA reads the same lengths and finds the same list.  False: refused.
  // s_mark: a bit per table row, zeroed; s_part [THREADS / 32].
  __device__ __forceinline__ bool build(uint32_t* s_mark, uint32_t* s_part, int* s_bad) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, Hkv = p.pool.n_kv_heads;
    if (p.n <= 32) {   // one warp, one barrier
      if (warp == 0) {
        const bool stop = status_get(p.status) != 0;
        int s = -1 - lane, length = 0;
        if (lane < p.n) length = look(lane, s);
        const bool twice = __popc(__match_any_sync(0xffffffffu, lane < p.n ? s : -1 - lane)) > 1;
        const bool bad = __any_sync(0xffffffffu, length < 0 || (p.k_new && twice));   // two new tokens, one slot
        uint32_t x = head_tiles(length) * Hkv * p.HB;
        const uint32_t own = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        if (lane < p.n) {
          first[lane] = x - own;
          row[lane] = s;
          len[lane] = length;
        }
        if (lane == 31) first[p.n] = x;
        if (lane == 0) {
          if (bad && !stop) status_set(p.status, TV_E_SEQ);
          *s_bad = bad || stop;
        }
      }
      __syncthreads();
      if (*s_bad) return false;
      all = first[p.n];
    } else {
      int bad = status_get(p.status) != 0;
      const int per = (p.n + THREADS - 1) / THREADS;
      uint32_t sum = 0;
      for (int i = tid * per; i < min(p.n, (tid + 1) * per); ++i) {
        int s, length = look(i, s);
        if (length >= 0 && p.k_new && (atomicOr(&s_mark[s >> 5], 1u << (s & 31)) >> (s & 31)) & 1u) length = -1;
        if (length < 0) bad = TV_E_SEQ;
        if (info) {
          row[i] = s;
          len[i] = length;
        }
        first[i] = sum;
        sum += head_tiles(length) * Hkv * p.HB;
      }
      if (bad < 0) status_set(p.status, bad);
      uint32_t x = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) s_part[warp] = x;
      if (__syncthreads_or(bad)) return false;
      uint32_t before = x - sum;
      all = 0;
      for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += s_part[w];
        all += s_part[w];
      }
      for (int i = tid * per; i < min(p.n, (tid + 1) * per); ++i) first[i] += before;
      if (tid == 0) first[p.n] = all;
      __syncthreads();
    }
    return true;
  }
  __device__ __forceinline__ void range() {
    chunk = (all + gridDim.x - 1) / gridDim.x;
    lo = min(all, chunk * blockIdx.x), hi = min(all, lo + chunk);
  }

  __device__ __forceinline__ void sequence(Run& g, int i) const {
    g.i = i;
    g.s = info ? row[i] : __ldg(p.ids + i);
    g.len = info ? len[i] : __ldcg(p.seqs.lens + g.s);
    window(g);
  }
  __device__ __forceinline__ void bound(Run& g) const { g.t1 = hi > g.base ? (int)min((uint32_t)g.T, hi - g.base) : 0; }
  __device__ __forceinline__ bool next_run(Run& g) const {   // false: there is none
    if (g.base + g.T >= hi) return false;
    g.base += g.T + SEG_COST;
    if (++g.hb == p.HB) {
      g.hb = 0;
      if (++g.h == p.pool.n_kv_heads) {
        g.h = 0;
        int i = g.i + 1;
        while (first[i + 1] == first[i]) ++i;
        sequence(g, i);
        g.base = first[i] + SEG_COST;
      }
    }
    g.t0 = 0;
    bound(g);
    return g.t1 > 0;
  }
  __device__ __forceinline__ bool first_run(Run& g) const {
    int i = 0;   // the sequence of place lo: the last whose first place is at or before it
    for (int b = p.n - 1; i < b;) {
      const int mid = (i + b + 1) >> 1;
      if (first[mid] <= lo) i = mid;
      else b = mid - 1;
    }
    sequence(g, i);
    const uint32_t unit = g.T + SEG_COST, hh = (lo - first[i]) / unit;
    g.h = (int)(hh / p.HB);
    g.hb = (int)(hh % p.HB);
    g.base = first[i] + hh * unit + SEG_COST;
    g.t0 = lo > g.base ? (int)(lo - g.base) : 0;
    bound(g);
    return g.t0 < g.t1 || next_run(g);
  }
};

// ---- host (tv_paged_attn.cu) ---------------------------------------------------
size_t paged_workspace(int D, PaWs* ws, uint8_t* base);
int check_paged_heads(int n_q_heads, int n_kv_heads, int n);
// the arguments of a call over either pool, checked and put in p; *sms: the GPU's.
// seg_cost: the kernel's, which with the tiles has to fit the list's 31 bits
int fill_paged(PaParams& p, int seg_cost, const tv_pool& pool, int layer, const tv_seqs* seqs, const int32_t* ids, int n, int n_q_heads,
               int window, int sinks, const tv_bf16* q, size_t q_stride, const tv_bf16* k_new, const tv_bf16* v_new,
               size_t kv_stride, tv_bf16* out, void* workspace, size_t workspace_bytes, int32_t* dev_status, int* sms);
// joins what ctas CTAs left
int launch_paged_merge(const PaParams& p, int ctas, cudaStream_t st);

}  // namespace tv
