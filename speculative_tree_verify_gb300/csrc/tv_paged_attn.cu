// Attention of one new token per sequence over a paged cache:
//   o[i, h] = sum_{j < len} softmax_j(q[i, h] . k[j, g] / sqrt(D)) v[j, g],  g = h / (Hq / Hkv),
// after the new token's own K and V rows went into slot len - 1.
//
// What bounds it: every cached K and V byte is read once for at most 16 query
// heads, far below the tensor cores' rate, so the kernel is built as a stream
// over memory; how it is cut over the CTAs is in tv_paged_runs.cuh.
//
// In a CTA three warps look up pages (32 boxes' entries at a time, the next 32 on
// their way) and issue TMA loads (a page's tokens of one head are contiguous:
// boxes of min(page, 64) rows x 64 values, 128-byte swizzle) into a ring of
// stages, each every third tile; eight warps compute, tile t by warps
// 4 (t mod 2) .. + 3, 16 tokens each, with mma.sync m16n8k16: the query heads
// are the 16 rows (a KV head's 5 or so need no 128-row tile, and the tokens of
// a warp need no other warp until the head ends).  S = Q K^T leaves each
// thread with the P it needs as the A operand of O += P V; P goes in as two
// bf16 parts (within 2^-16 of it together), which costs 1 to 4 % of the time
// (128 x 8k tokens: 648 -> 652 us; one of 32k: 29.0 -> 30.1 us) and leaves the
// output's own rounding as the only one.  Offsets move only when a score
// passes them by 2^8.
//
// An infinity in a token's V is the result in its dimension, but the products
// have it times the second part of P, which may be zero or below it, and sums
// that are joined have it times a weight that may be zero: NaN.  So where an
// element is NaN and its row's sum is not, the run's V is looked over again,
// and the element is what the infinities and NaN there make of it.
//
// Through a window (WIN: tv_attend_paged_window) the tiles between the sinks
// and the window are no work at all, and boxes that hold nothing visible are
// not loaded; of the others the hidden tokens' scores are -inf and their V is
// emptied in shared memory, as that of the slots past the length.
#include <cmath>
#include <type_traits>

#include "tv_gemm.cuh"
#include "tv_paged_runs.cuh"

namespace tv {
namespace {

// Tiles in flight: 192 KB of the SM at D = 128.  Even, so that a stage always
// belongs to the same four warps: their waits then see every phase of its
// barrier, and a parity can not name the phase before last.
constexpr int kStages = 6;
static_assert(kStages % 2 == 0, "tile t: stage t mod kStages, warps 4 (t mod 2) .. + 3");
constexpr int kCompWarps = 8;
constexpr int kCompThreads = kCompWarps * 32;
// Each has every third tile, so that a stage (and a place of the queries) always
// belongs to the same warp: its waits then see every phase of the place's
// barrier, and a parity can not name the phase before last.
constexpr int kLoadWarps = 3;
static_assert(kStages % kLoadWarps == 0, "a stage always belongs to the same loading warp");
constexpr int kPaThreads = kCompThreads + 32 * kLoadWarps;
constexpr int kQueries = 8;                      // segments whose queries are loaded ahead, at most
// rows joined at a time when a head block ends: as many as there is room for
// (at D = 128 and up to 357 sequences 5 or 6, at D = 64 all 8; with four at a time
// 128 sequences of 1 to 8191, 40/8 heads, a window of 2047, took 63.9 us, now 56.6)
constexpr int kRedRows = 4, kMostRedRows = 8;
// What a head block costs besides its tiles, in tiles (its queries, its join).
// 48 sequences of 1 to 8191 tokens, 8/2 heads, with 2, 3, 5, 6 tiles: 14.7, 14.6,
// 13.7, 14.0 us; 128 of them, 40/8 heads: 82, 77, 74, 75 us.  It stays at 2 there: another
// cut sums in another order, and results keep their last bits.  Through a window few
// tiles are left to a head block (the 128, a window of 2047, with 2, 3, 4, 5, 6 tiles:
// 62, 58, 58, 56, 57 us).
constexpr int kSegCost = 2, kSegCostWin = 5;
constexpr float kMoveLog2 = 8.f;

template <int D>
struct PaSmem {
  static constexpr int SLAB = kTile * 128;                   // 64 dimensions of a tile
  static constexpr int HALF = (D / 64) * SLAB;               // a tile's K (or V)
  static constexpr int STAGE = 2 * HALF;
  static constexpr int OFF_ML = kStages * STAGE;
  static constexpr int Q_ROW = D * 2 + 16;          // rows 16 bytes apart in the banks: ldmatrix without conflicts
  // 2 kRows query rows: those of the next 2 to kQueries runs
  static constexpr int OFF_Q = OFF_ML + kCompWarps * kRows * 8;
  static constexpr int OFF_BAR = OFF_Q + 2 * kRows * Q_ROW;
  static constexpr int OFF_FIRST = OFF_BAR + 256;   // [n + 1]; up to kInfo sequences also their rows and lengths
  static constexpr int RED_ROW = kCompWarps * D * 4;
  static constexpr int MOST = 232448 - 64 - 1024;   // of a CTA, static arrays and alignment aside
  // [8 warps][red_rows][D] fp32 at the end; the marks of listed rows first
  __host__ __device__ static constexpr int off_red(int n) {
    return (OFF_FIRST + (n + 1) * 4 + (n <= kInfo ? n * 8 : 0) + 15) & ~15;
  }
  __host__ __device__ static constexpr int red_rows(int n) {
    const int fit = (MOST - off_red(n)) / RED_ROW;
    return fit < kMostRedRows ? fit : kMostRedRows;
  }
  static size_t bytes(int n) { return 1024 + (size_t)off_red(n) + red_rows(n) * RED_ROW; }
  static_assert(kRedRows * RED_ROW >= kMaxSeqs / 8, "a mark for every table row");
  static_assert(red_rows(kMaxTokens) >= kRedRows && red_rows(kInfo) >= kRedRows, "shared memory of one CTA");
};

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void comp_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kCompThreads) : "memory"); }

__device__ __forceinline__ void quad_sync(int quad) {
  asm volatile("bar.sync %0, %1;" ::"r"(2 + quad), "n"(kCompThreads / 2) : "memory");
}

// a barrier of n threads: true if v is true on any of them
__device__ __forceinline__ bool bar_any(bool v, int id, int n) {
  uint32_t out;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "bar.red.or.pred p, %2, %3, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(out)
      : "r"((uint32_t)v), "r"(id), "r"(n)
      : "memory");
  return out != 0;
}

// Rows r0 .. r0 + nr - 1 of a run's output (out) or partial result (part_o), an
// element of which is NaN: what is not finite among the run's V, by dimension,
// and where that is infinities of one sign, the infinity.  By 32 nw threads
// that meet on barrier bar; kinds: D words, ml: offsets and sums of the nw
// warps.  Out of line, since a call that has no use for it pays for its place
// in the join (us without it, out of line, inside: 256 short sequences x 16
// heads 49.4, 50.4, 52.2; one of 1k 9.33, 9.50, 9.65).  WIN: at and end count the
// tokens of the list's tiles.
template <int D, bool WIN>
__device__ __noinline__ void put_infinities(const PaParams& p, int i, int s, int len, Run g, uint32_t at, uint32_t end, int h,
                                            int nr, uint32_t* kinds, const float2* ml, int nw, int me, int bar,
                                            __nv_bfloat16* out, float* part_o) {
  const int ps = p.pool.page_size, c = 8 * (me % (D / 8));
  auto meet = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(32 * nw) : "memory"); };
  for (int d = me; d < D; d += 32 * nw) kinds[d] = 0u;   // 1: NaN, 2: +inf, 4: -inf
  meet();
  for (at += me / (D / 8); at < end; at += 32 * nw / (D / 8)) {   // (unsigned: lengths near 2^31)
    uint32_t tok = at;
    if constexpr (WIN) {
      if (at >= (uint32_t)g.sink_tiles * kTile) tok += (uint32_t)g.skip * kTile;
      if (tok >= (uint32_t)len || (tok < (uint32_t)g.lo && tok >= (uint32_t)p.sinks)) continue;
    }
    const __nv_bfloat16* v = p.v_new + (size_t)i * p.kv_stride + (size_t)h * D;   // the new row may not be in its page yet
    if (!p.v_new || tok != (uint32_t)len - 1) {
      const int page = __ldcg(p.seqs.pages + (size_t)s * p.seqs.max_pages + tok / ps);
      if (page < 0 || page >= p.pool.n_pages) continue;
      v = reinterpret_cast<const __nv_bfloat16*>(p.pool.v) +
          ((((size_t)p.layer * p.pool.n_pages + page) * p.pool.n_kv_heads + h) * ps + tok % ps) * D;
    }
    const uint4 x = __ldcg(reinterpret_cast<const uint4*>(v + c));
    const uint32_t q[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t b = q[u >> 1] >> (16 * (u & 1)) & 0xffffu;
      if ((b & 0x7f80u) == 0x7f80u) atomicOr(kinds + c + u, b & 0x7fu ? 1u : (b & 0x8000u ? 4u : 2u));
    }
  }
  meet();
  for (int e = me; e < nr * D; e += 32 * nw) {
    const int row = e / D;
    float M = -INFINITY, L = 0.f;
    for (int w = 0; w < nw; ++w) M = fmaxf(M, ml[w * kRows + row].x);
    for (int w = 0; w < nw; ++w) {
      const float2 x = ml[w * kRows + row];
      L += x.x == -INFINITY ? x.y : x.y * ex2f(x.x - M);
    }
    const uint32_t kind = kinds[e % D];
    if (!(L > 0.f && L < INFINITY) || (kind != 2u && kind != 4u)) continue;   // the row's own NaN, and both infinities, stay NaN
    const float x = kind == 2u ? INFINITY : -INFINITY;
    if (out) out[e] = __float2bfloat16_rn(x);
    else part_o[e] = x;
  }
  meet();
}

template <int D, bool WIN>
__global__ void __launch_bounds__(kPaThreads, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                      const __grid_constant__ PaParams p) {
  using L = PaSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* empty = full + kStages;
  uint64_t* q_full = empty + kStages;    // [kQueries] a segment's queries landed
  uint64_t* q_free = q_full + kQueries;  // [kQueries] all eight warps have seen them, those that compute it are done with them
  uint32_t* s_first = reinterpret_cast<uint32_t*>(smem + L::OFF_FIRST);
  const int red_rows = L::red_rows(p.n);
  float* s_red = reinterpret_cast<float*>(smem + L::off_red(p.n));
  float2* s_ml = reinterpret_cast<float2*>(smem + L::OFF_ML);
  uint32_t* s_mark = reinterpret_cast<uint32_t*>(s_red);
  __shared__ uint32_t s_part[kPaThreads / 32];
  __shared__ int s_bad;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ps = p.pool.page_size, Hkv = p.pool.n_kv_heads;
  // places of the query ring: short sequences need many runs ahead
  const int qrows = min(kRows, p.G), qslots = min(kQueries, 2 * kRows / qrows);

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 4);   // the four warps that compute its tile
    }
    for (int s = 0; s < kQueries; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_free[s], kCompWarps);
    }
    fence_mbar_init();
    prefetch_tmap(&map_k);
    prefetch_tmap(&map_v);
    s_bad = 0;
  }
  if (p.n > 32 && p.k_new)
    for (int i = tid; i < (p.seqs.max_seqs + 31) / 32; i += kPaThreads) s_mark[i] = 0u;
  __syncthreads();
  pdl_wait();
  pdl_trigger();

  RunList<kPaThreads, WIN ? kSegCostWin : kSegCost, WIN> runs(p, s_first);
  if (!runs.build(s_mark, s_part, &s_bad)) return;
  // sequences without a token: zeros
  for (int i = blockIdx.x; i < p.n; i += gridDim.x)
    if (s_first[i + 1] == s_first[i])
      for (int e = tid; e < p.Hq * D / 8; e += kPaThreads)
        reinterpret_cast<uint4*>(p.out + (size_t)i * p.Hq * D)[e] = make_uint4(0u, 0u, 0u, 0u);

  runs.range();
  if (tid == 0) p.ws.cut[blockIdx.x] = make_int4(-1, 0, 0, 0);
  if (runs.lo >= runs.hi) return;

  if (warp >= kCompWarps) {
    // ---------------- pages and loads ----------------
    const int mine = warp - kCompWarps;             // tiles with (count mod kLoadWarps) == mine, and places of queries
    const int R = ps < kTile ? ps : kTile;          // rows of a box
    const int nsh = 6 - (31 - __clz(R)), nb = 1 << nsh;   // boxes of a tile's K slab
    const int psh = 31 - __clz(ps), per = 32 >> nsh;      // tiles of 32 boxes
    constexpr int kPer = 2 * (D / 64);              // K and V slabs of a box
    const int box = lane / kPer, which = lane % kPer;
    const bool is_v = which >= D / 64;
    const int slab = which % (D / 64);
    const uint64_t pol = policy_evict_first();
    const int y0 = p.layer * p.pool.n_pages;   // the host has seen to it that a row of the pool is an int
    bool ok = true;
    int count = 0, segs = 0;   // tiles and runs so far, anyone's
    auto wait = [&](uint64_t* bar, uint32_t parity) { ok = __all_sync(0xffffffffu, mbar_wait(bar, parity & 1u)); };
    // a box of tokens tok .. tok + R - 1 holds something that is seen
    auto seen = [&](const Run& g, int tok) {
      return tok < g.len && (!WIN || tok >= g.lo - (R - 1) || tok < p.sinks);
    };
    auto entry = [&](const Run& g, int tb) {   // the page of this lane's box of tiles tb ..., -1: not seen
      const int t = tb + (lane >> nsh);
      if (t >= g.t1) return -1;
      const int tok = g.tile<WIN>(t) * kTile + (lane & (nb - 1)) * R;
      return seen(g, tok) ? __ldcg(p.seqs.pages + (size_t)g.s * p.seqs.max_pages + (tok >> psh)) : -1;
    };
    Run g;
    bool have = runs.first_run(g);
    int pages = have ? entry(g, g.t0) : -1;
    while (have && ok) {
      Run next = g;   // the next entries are on their way before this run's tiles
      const bool more = runs.next_run(next);
      const int qs = segs % qslots;
      if (qs % kLoadWarps == mine) {   // its queries
        if (segs >= qslots) wait(&q_free[qs], (uint32_t)(segs / qslots - 1));
        if (!ok) break;
        const int r0 = g.hb * kRows, nr = min(kRows, p.G - r0);
        if (lane == 0) mbar_arrive_expect_tx(&q_full[qs], (uint32_t)(nr * D * 2));
        __syncwarp();
        if (lane < nr)
          bulk_load(smem + L::OFF_Q + (qs * qrows + lane) * L::Q_ROW,
                    p.q + (size_t)g.i * p.q_stride + (size_t)(g.h * p.G + r0 + lane) * D, D * 2, &q_full[qs]);
        __syncwarp();
      }
      ++segs;
      for (int tb = g.t0; tb < g.t1 && ok; tb += per) {
        const int next_pages = tb + per < g.t1 ? entry(g, tb + per) : (more ? entry(next, next.t0) : -1);
        const int end = min(tb + per, g.t1);
        for (int t = tb + (mine + kLoadWarps - count % kLoadWarps) % kLoadWarps; t < end; t += kLoadWarps) {
          const int issued = count + (t - tb), st = issued % kStages;
          const int page = __shfl_sync(0xffffffffu, pages, ((t - tb) << nsh) + (box & (nb - 1)));
          const int tok = g.tile<WIN>(t) * kTile + box * R;
          const bool in = box < nb && seen(g, tok);
          const bool good = in && page >= 0 && page < p.pool.n_pages;
          if (in && !good) status_set(p.status, TV_E_PAGE);
          const int y = good ? (((y0 + page) * Hkv + g.h) << psh) + (tok & (ps - 1)) : 0;
          if (issued >= kStages) wait(&empty[st], (uint32_t)(issued / kStages - 1));
          if (!ok) break;
          const unsigned boxes = __ballot_sync(0xffffffffu, good);
          if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)__popc(boxes) * (uint32_t)(R * 128));
          __syncwarp();
          if (good)
            tma_load_2d(smem + st * L::STAGE + (is_v ? L::HALF : 0) + slab * L::SLAB + box * R * 128, is_v ? &map_v : &map_k,
                        &full[st], slab * 64, y, pol);
          __syncwarp();
        }
        count += end - tb;
        pages = next_pages;
      }
      g = next;
      have = more;
    }
    if (!ok && lane == 0) status_set(p.status, TV_E_TIMEOUT);
    // loads in flight land before the CTA leaves: each warp has armed the
    // barriers of its own, and what a timeout left unissued is not waited for
    for (int u = max(0, segs - qslots); ok && u < segs; ++u)
      if (u % qslots % kLoadWarps == mine) wait(&q_full[u % qslots], (uint32_t)(u / qslots));
    for (int u = max(0, count - kStages); ok && u < count; ++u)
      if (u % kLoadWarps == mine) wait(&full[u % kStages], (uint32_t)(u / kStages));
    return;
  }

  // ---------------- compute warps ----------------
  constexpr int KS = D / 16;                        // k steps of S, and pairs of n blocks of O
  const int quad = warp >> 2, sl = warp & 3;        // tiles with (count mod 2) == quad; tokens 16 sl .. + 15 of a tile
  const int g8 = lane >> 2, t4 = lane & 3;
  bool ok = true;
  // the next tile and queries of this CTA: places in the rings, parities
  int st = 0, qs = 0;
  uint32_t st_par = 0u, qs_par = 0u;
  // lane addresses inside a slab: K as [token][d] fragments, V transposed
  const int k_tok = 16 * sl + (lane & 7) + ((lane >> 4) << 3), k_ch = (lane >> 3) & 1;
  const int v_tok = 16 * sl + (lane & 15), v_ch = lane >> 4;
  Run g;
  for (bool have = runs.first_run(g); have; have = runs.next_run(g)) {
    const int h = g.h, r0 = g.hb * kRows;   // KV head, first query head of the block in the group
    const int nr = min(kRows, p.G - r0);
    if (g.T == 1 && (st & 1) != quad) {   // one tile, and the other four warps'
      // no further ahead than the queries, nor further behind than their place:
      // it is not loaded again before these warps, too, have seen this phase (a
      // wait that comes a round late names the phase before last, which a parity can not)
      if (ok && !mbar_wait(&q_full[qs], qs_par)) ok = false;
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_free[qs]);
      if (++st == kStages) st = 0, st_par ^= 1u;
      if (++qs == qslots) qs = 0, qs_par ^= 1u;
      continue;
    }
    uint32_t qf[KS][4];
    {
      if (ok && !mbar_wait(&q_full[qs], qs_par)) ok = false;
      // rows past the group's heads: the last one again, products nobody reads
      const uint32_t qa = smem_u32(smem + L::OFF_Q) + (qs * qrows + min(lane & 15, nr - 1)) * L::Q_ROW + (lane >> 4) * 16;
#pragma unroll
      for (int k = 0; k < KS; ++k) ldsm4(qa + k * 32, qf[k]);
    }
    float o[2 * KS][4];
#pragma unroll
    for (int k = 0; k < 2 * KS; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[k][e] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;   // rows g8 and g8 + 8; sums of this thread's tokens

    for (int t = g.t0; t < g.t1; ++t) {
      const int at = st;
      const uint32_t par = st_par;
      if (++st == kStages) st = 0, st_par ^= 1u;
      if ((at & 1) != quad) continue;   // an even number of stages: the place's parity is the tile's
      uint8_t* sk = smem + at * L::STAGE;
      uint8_t* sv = sk + L::HALF;
      if (ok && !mbar_wait(&full[at], par)) ok = false;
      const int tok0 = g.tile<WIN>(t) * kTile + 16 * sl;
      int valid = min(16, g.len - tok0);   // this warp's tokens
      int hide0 = 0, hide1 = 0;            // those from hide0 up to hide1 are hidden
      if constexpr (WIN) {
        hide0 = max(0, p.sinks - tok0);
        hide1 = min(16, g.lo - tok0);
        if (hide0 == 0 && hide1 >= valid) valid = 0;
      }
      if (valid > 0) {
        bool wrote = false;
        if (p.k_new && tok0 + valid == g.len) {
          // the new token: its rows into the tile and into the page
          const bool v = lane >= 16;
          const int c = lane & 15;
          if (c < D / 8) {
            const __nv_bfloat16* row = (v ? p.v_new : p.k_new) + (size_t)g.i * p.kv_stride + (size_t)h * D;
            const uint4 x = __ldcg(reinterpret_cast<const uint4*>(row) + c);
            *reinterpret_cast<uint4*>((v ? sv : sk) + (c >> 3) * L::SLAB + swz(16 * sl + valid - 1, c & 7)) = x;
            if (r0 == 0) {
              const int page = __ldcg(p.seqs.pages + (size_t)g.s * p.seqs.max_pages + (g.len - 1) / ps);
              if (page >= 0 && page < p.pool.n_pages) {
                const size_t e = ((((size_t)p.layer * p.pool.n_pages + page) * Hkv + h) * ps + (g.len - 1) % ps) * D;
                reinterpret_cast<uint4*>((v ? p.pool.v : p.pool.k) + e)[c] = x;
              }
            }
          }
          wrote = true;
        }
        if (valid < 16) {   // slots past the length: whatever they hold, 0 * V stays 0
          for (int e = lane; e < (16 - valid) * (D / 8); e += 32) {
            const int tk = 16 * sl + valid + e / (D / 8), c = e % (D / 8);
            *reinterpret_cast<uint4*>(sv + (c >> 3) * L::SLAB + swz(tk, c & 7)) = make_uint4(0u, 0u, 0u, 0u);
          }
          wrote = true;
        }
        if (WIN && hide0 < hide1) {   // nor do hidden ones
          for (int e = lane; e < (hide1 - hide0) * (D / 8); e += 32) {
            const int tk = 16 * sl + hide0 + e / (D / 8), c = e % (D / 8);
            *reinterpret_cast<uint4*>(sv + (c >> 3) * L::SLAB + swz(tk, c & 7)) = make_uint4(0u, 0u, 0u, 0u);
          }
          wrote = true;
        }
        __syncwarp();
        float c0[4] = {0.f, 0.f, 0.f, 0.f}, c1[4] = {0.f, 0.f, 0.f, 0.f};
        const uint32_t ka = smem_u32(sk), va = smem_u32(sv);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t b[4];
          ldsm4(ka + (k >> 2) * L::SLAB + swz(k_tok, ((2 * k) & 7) + k_ch), b);
          mma16816(c0, qf[k], b[0], b[1]);
          mma16816(c1, qf[k], b[2], b[3]);
        }
        // tokens 2 t4, 2 t4 + 1 (c0) and 8 more (c1) of rows g8 (elements 0, 1) and g8 + 8 (2, 3)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tk = 2 * t4 + (e & 1);
          const bool in0 = tk < valid && (!WIN || tk < hide0 || tk >= hide1);
          const bool in1 = tk + 8 < valid && (!WIN || tk + 8 < hide0 || tk + 8 >= hide1);
          c0[e] = in0 ? c0[e] * p.scale_log2 : -INFINITY;
          c1[e] = in1 ? c1[e] * p.scale_log2 : -INFINITY;
        }
        float x0 = fmaxf(fmaxf(c0[0], c0[1]), fmaxf(c1[0], c1[1])), x1 = fmaxf(fmaxf(c0[2], c0[3]), fmaxf(c1[2], c1[3]));
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
        if (__any_sync(0xffffffffu, x0 > m0 + kMoveLog2 || x1 > m1 + kMoveLog2)) {
          const float n0 = x0 > m0 + kMoveLog2 ? x0 : m0, n1 = x1 > m1 + kMoveLog2 ? x1 : m1;
          const float a0 = n0 == m0 ? 1.f : ex2f(m0 - n0), a1 = n1 == m1 ? 1.f : ex2f(m1 - n1);
          m0 = n0;
          m1 = n1;
          l0 *= a0;
          l1 *= a1;
#pragma unroll
          for (int k = 0; k < 2 * KS; ++k) {
            o[k][0] *= a0;
            o[k][1] *= a0;
            o[k][2] *= a1;
            o[k][3] *= a1;
          }
        }
        const float f0 = m0 == -INFINITY ? 0.f : m0, f1 = m1 == -INFINITY ? 0.f : m1;
        uint32_t pf[4], pl[4];   // P and what its rounding to bf16 left
        auto pack = [](float a, float b, float& l, uint32_t& lo) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
          const uint32_t u = *reinterpret_cast<const uint32_t*>(&v);
          const float ra = a - __uint_as_float(u << 16), rb = b - __uint_as_float(u & 0xffff0000u);
          const __nv_bfloat162 w = __floats2bfloat162_rn(ra, rb);
          lo = *reinterpret_cast<const uint32_t*>(&w);
          l += a + b;
          return u;
        };
        pf[0] = pack(ex2f(c0[0] - f0), ex2f(c0[1] - f0), l0, pl[0]);
        pf[1] = pack(ex2f(c0[2] - f1), ex2f(c0[3] - f1), l1, pl[1]);
        pf[2] = pack(ex2f(c1[0] - f0), ex2f(c1[1] - f0), l0, pl[2]);
        pf[3] = pack(ex2f(c1[2] - f1), ex2f(c1[3] - f1), l1, pl[3]);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t b[4];
          ldsm4t(va + (k >> 2) * L::SLAB + swz(v_tok, ((2 * k) & 7) + v_ch), b);
          mma16816(o[2 * k], pf, b[0], b[1]);
          mma16816(o[2 * k + 1], pf, b[2], b[3]);
          mma16816(o[2 * k], pl, b[0], b[1]);
          mma16816(o[2 * k + 1], pl, b[2], b[3]);
        }
        if (wrote) fence_async_smem();   // before the stage takes another TMA write
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[at]);
    }

    // ---- the head block's partial results into one ----
    // of all eight warps, or, where the head block is one tile, of the four
    // that had it: the other four go on to the next head block meanwhile
    const bool whole = g.t0 == 0 && g.t1 == g.T;
    // a CTA's first run may begin inside a head block, its last end inside one
    const size_t slot = (size_t)blockIdx.x * 2 + (g.t0 == 0 ? 1 : 0);
    auto join = [&](auto nw_c) {
      constexpr int NW = decltype(nw_c)::value;        // warps that take part, from w0 on
      const int w0 = NW == kCompWarps ? 0 : 4 * quad, me = tid - 32 * w0;
      auto meet = [&]() {
        if constexpr (NW == kCompWarps) comp_sync();
        else quad_sync(quad);
      };
      l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
      l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
      if (t4 == 0) {
        s_ml[warp * kRows + g8] = make_float2(m0, l0);
        s_ml[warp * kRows + g8 + 8] = make_float2(m1, l1);
      }
      meet();
      // The queries' place is given up here, not behind the loads: an arrival
      // does not wait for ldmatrix results that nothing has used yet.  (A warp
      // without a token in this run has not used them, and never will.)
      if (lane == 0) mbar_arrive(&q_free[qs]);
      bool lost = false;   // an element is NaN
#pragma unroll 1   // one copy of the code: most groups need one or two parts, and short sequences run it once a tile
      for (int row0 = 0; row0 < nr; row0 += red_rows) {   // rows row0 .. + red_rows - 1, a lane has one of them at most
        const bool upper = g8 < row0;
        const int row = g8 + (upper ? 8 : 0), mine = row - row0;
        if (mine >= 0 && mine < red_rows) {
          float2 ml[NW];
          float M = -INFINITY, L = 0.f;
#pragma unroll
          for (int w = 0; w < NW; ++w) {
            ml[w] = s_ml[(w0 + w) * kRows + row];
            M = fmaxf(M, ml[w].x);
          }
#pragma unroll
          for (int w = 0; w < NW; ++w) L += ml[w].x == -INFINITY ? ml[w].y : ml[w].y * ex2f(ml[w].x - M);
          const float own = upper ? m1 : m0;
          float f = own == -INFINITY ? 0.f : ex2f(own - M);
          if (whole) f /= L;
          else if (warp == w0 && t4 == 0 && row < nr)
            *reinterpret_cast<float2*>(p.ws.ml + (slot * kRows + row) * 2) = make_float2(M, L);
          // row r: groups of 8 values XOR r, no bank twice in four rows
          float* dst = s_red + (warp * red_rows + mine) * D + 2 * t4;
          float* at[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) at[k] = dst + ((8 * k) ^ ((mine & 3) * 8));
#pragma unroll
          for (int k = 0; k < 2 * KS; ++k)
            *reinterpret_cast<float2*>(at[k & 3] + 32 * (k >> 2)) =
                make_float2((upper ? o[k][2] : o[k][0]) * f, (upper ? o[k][3] : o[k][1]) * f);
        }
        meet();
        for (int e = me; e < min(red_rows, nr - row0) * (D / 2); e += 32 * NW) {
          const int r = e / (D / 2), d = 2 * (e % (D / 2)), row = r + row0;
          {
            float2 acc = make_float2(0.f, 0.f);
#pragma unroll
            for (int w = 0; w < NW; ++w) {
              const float2 v = *reinterpret_cast<const float2*>(s_red + ((w0 + w) * red_rows + r) * D + (d ^ ((r & 3) * 8)));
              acc.x += v.x;
              acc.y += v.y;
            }
            lost = lost || acc.x != acc.x || acc.y != acc.y;
            if (whole)
              *reinterpret_cast<__nv_bfloat162*>(p.out + ((size_t)g.i * p.Hq + h * p.G + r0 + row) * D + d) =
                  __floats2bfloat162_rn(acc.x, acc.y);
            else
              *reinterpret_cast<float2*>(p.ws.o + (slot * kRows + row) * D + d) = acc;
          }
        }
        if (row0 + red_rows < nr) meet();
      }
      const int bar = NW == kCompWarps ? 1 : 2 + quad;
      if (bar_any(lost, bar, 32 * NW))
        put_infinities<D, WIN>(p, g.i, g.s, g.len, g, (uint32_t)g.t0 * kTile,
                          !WIN && g.t1 == g.T ? g.len : (uint32_t)g.t1 * kTile, h, nr,
                          reinterpret_cast<uint32_t*>(s_red + w0 * red_rows * D), s_ml + w0 * kRows, NW, me, bar,
                          whole ? p.out + ((size_t)g.i * p.Hq + h * p.G + r0) * D : nullptr, p.ws.o + slot * kRows * D);
    };
    if (g.T > 1) join(std::integral_constant<int, kCompWarps>{});
    else join(std::integral_constant<int, kCompWarps / 2>{});
    if (++qs == qslots) qs = 0, qs_par ^= 1u;
    if (tid == 0 && g.t0 == 0 && !whole)   // the CTA's last run
      p.ws.cut[blockIdx.x] = make_int4(g.i, g.h * p.HB + g.hb, (int)((g.base + g.T - 1) / runs.chunk), 0);
  }
  if (!ok && lane == 0) status_set(p.status, TV_E_TIMEOUT);
}

// Block c joins the head block whose first tile CTA c had and whose last it had
// not: the partials of CTAs c (its slot 1) to the last one's (slot 0), in that
// order.  A warp a row for the weights, then every thread a pair of values.
constexpr int kMergeThreads = 512;
template <int D>
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const PaParams p) {
  __shared__ float s_w[kRows][kMaxCtas];   // 2^(m_c - M) / sum
  pdl_wait();
  pdl_trigger();
  const int4 cut = __ldcg(p.ws.cut + blockIdx.x);
  const int stop = status_get(p.status);
  if (cut.x < 0 || stop != 0) return;
  const int c0 = blockIdx.x, np = cut.z - c0 + 1, r0 = (cut.y % p.HB) * kRows, nr = min(kRows, p.G - r0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto slot = [&](int c) { return (size_t)(c0 + c) * 2 + (c == 0 ? 1 : 0); };
  auto partial = [&](int e, int c) {
    return __ldcg(reinterpret_cast<const float2*>(p.ws.o + (slot(c) * kRows + e / (D / 2)) * D + 2 * (e % (D / 2))));
  };
  constexpr int kEarly = 16;   // partials asked for before the weights are known
  float2 v[kEarly];
#pragma unroll
  for (int c = 0; c < kEarly; ++c)
    v[c] = threadIdx.x < nr * (D / 2) && c < np ? partial(threadIdx.x, c) : make_float2(0.f, 0.f);
  if (warp < nr) {
    float2 ml[kMaxCtas / 32];
    float M = -INFINITY, sum = 0.f;
#pragma unroll
    for (int k = 0; k < kMaxCtas / 32; ++k) {
      ml[k] = make_float2(-INFINITY, 0.f);
      if (32 * k + lane < np)
        ml[k] = __ldcg(reinterpret_cast<const float2*>(p.ws.ml + (slot(32 * k + lane) * kRows + warp) * 2));
      M = fmaxf(M, ml[k].x);
    }
    M = warp_max(M);
#pragma unroll
    for (int k = 0; k < kMaxCtas / 32; ++k) {
      const float w = ml[k].x == -INFINITY ? 0.f : ex2f(ml[k].x - M);
      sum += ml[k].x == -INFINITY ? ml[k].y : ml[k].y * w;
      ml[k].x = w;
    }
    sum = warp_sum(sum);
#pragma unroll
    for (int k = 0; k < kMaxCtas / 32; ++k)
      if (32 * k + lane < np) s_w[warp][32 * k + lane] = ml[k].x / sum;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < nr * (D / 2); e += kMergeThreads) {
    const int row = e / (D / 2), d = 2 * (e % (D / 2));
    float2 acc = make_float2(0.f, 0.f);
    auto add = [&](float2 x, float w) {
      acc.x = fmaf(x.x, w, acc.x);
      acc.y = fmaf(x.y, w, acc.y);
    };
    int c = 0;
    if (e < kMergeThreads) {
#pragma unroll
      for (int u = 0; u < kEarly; ++u)
        if (u < np) add(v[u], s_w[row][u]);
      c = kEarly;
    }
#pragma unroll 8
    for (; c < np; ++c) add(partial(e, c), s_w[row][c]);
    if (acc.x != acc.x || acc.y != acc.y) {   // again, with an infinity that weighs nothing as it is
      acc = make_float2(0.f, 0.f);
#pragma unroll 1
      for (c = 0; c < np; ++c) {
        const float2 x = partial(e, c);
        const float w = s_w[row][c];
        acc.x += w == 0.f && isinf(x.x) ? x.x : x.x * w;
        acc.y += w == 0.f && isinf(x.y) ? x.y : x.y * w;
      }
    }
    *reinterpret_cast<__nv_bfloat162*>(p.out + ((size_t)cut.x * p.Hq + (cut.y / p.HB) * p.G + r0 + row) * D + d) =
        __floats2bfloat162_rn(acc.x, acc.y);
  }
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

template <int D, bool WIN>
int launch_paged(const PaParams& p, int ctas, cudaStream_t st) {
  CUtensorMap mk, mv;
  const int rows = p.pool.n_layers * p.pool.n_pages * p.pool.n_kv_heads * p.pool.page_size;   // checked to fit
  const int R = p.pool.page_size < kTile ? p.pool.page_size : kTile;
  int rc = make_tmap_bf16(&mk, p.pool.k, D, rows, 64, R);
  if (rc || (rc = make_tmap_bf16(&mv, p.pool.v, D, rows, 64, R))) return rc;
  static std::atomic<bool> attr[64];
  if (ensure_smem_limit(paged_attn_kernel<D, WIN>, 1024 + PaSmem<D>::MOST, attr)) return TV_E_CUDA;
  rc = launch_pdl(paged_attn_kernel<D, WIN>, dim3(ctas), dim3(kPaThreads), PaSmem<D>::bytes(p.n), st, mk, mv, p);
  return rc ? rc : launch_paged_merge(p, ctas, st);
}

int attend_paged(bool win, const tv_pool* pool, int layer, const tv_seqs* seqs, const int32_t* ids, int n, int n_q_heads,
                 int window, int sinks, const tv_bf16* q, size_t q_stride, const tv_bf16* k_new, const tv_bf16* v_new,
                 size_t kv_stride, tv_bf16* out, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                 void* stream) {
  PaParams p;
  int sms;
  int rc = check_pool(pool);
  if (rc || (rc = fill_paged(p, win ? kSegCostWin : kSegCost, *pool, layer, seqs, ids, n, n_q_heads, window, sinks, q, q_stride, k_new, v_new, kv_stride,
                             out, workspace, workspace_bytes, dev_status, &sms)))
    return rc;
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (win) return pool->head_dim == 128 ? launch_paged<128, true>(p, ctas, st) : launch_paged<64, true>(p, ctas, st);
  return pool->head_dim == 128 ? launch_paged<128, false>(p, ctas, st) : launch_paged<64, false>(p, ctas, st);
}

}  // namespace

size_t paged_workspace(int D, PaWs* ws, uint8_t* base) {
  const size_t cut = align256((size_t)kMaxCtas * sizeof(int4)), ml = align256((size_t)2 * kMaxCtas * kRows * 2 * 4);
  const size_t o = align256((size_t)2 * kMaxCtas * kRows * D * 4);
  if (ws) {
    ws->cut = reinterpret_cast<int4*>(base);
    ws->ml = reinterpret_cast<float*>(base + cut);
    ws->o = reinterpret_cast<float*>(base + cut + ml);
  }
  return cut + ml + o;
}

int check_paged_heads(int n_q_heads, int n_kv_heads, int n) {
  if (n_q_heads < 1) return TV_E_ARG;
  if (n_q_heads % n_kv_heads != 0 || n_q_heads > 65536) return TV_E_UNSUPPORTED;
  return n < 1 ? TV_E_ARG : (n > kMaxTokens ? TV_E_UNSUPPORTED : TV_OK);
}

int fill_paged(PaParams& p, int seg_cost, const tv_pool& pool, int layer, const tv_seqs* seqs, const int32_t* ids, int n, int n_q_heads,
               int window, int sinks, const tv_bf16* q, size_t q_stride, const tv_bf16* k_new, const tv_bf16* v_new,
               size_t kv_stride, tv_bf16* out, void* workspace, size_t workspace_bytes, int32_t* dev_status, int* sms) {
  int rc = check_seqs(seqs, &pool);
  if (rc) return rc;
  if (!ids || !q || !out || !dev_status || !k_new != !v_new || layer < 0 || layer >= pool.n_layers) return TV_E_ARG;
  if (window < 1 || sinks < 0) return TV_E_ARG;
  if ((rc = check_paged_heads(n_q_heads, pool.n_kv_heads, n))) return rc;
  const size_t D = pool.head_dim;
  if (!aligned16(q) || !aligned16(out) || q_stride % 8 != 0 || q_stride < n_q_heads * D) return TV_E_ARG;
  if (k_new && (!aligned16(k_new) || !aligned16(v_new) || kv_stride % 8 != 0 || kv_stride < pool.n_kv_heads * D))
    return TV_E_ARG;
  p.G = n_q_heads / pool.n_kv_heads;
  p.HB = (p.G + kRows - 1) / kRows;
  // the places of n sequences of the longest kind
  const unsigned long long most =
      (((unsigned long long)seqs->max_pages * pool.page_size + kTile - 1) / kTile + seg_cost + 2) * pool.n_kv_heads * p.HB;
  if (most > 0x7fffffffull / (unsigned)n) return TV_E_UNSUPPORTED;
  uint8_t* base = static_cast<uint8_t*>(workspace);
  if (!workspace || !aligned16(workspace) || workspace_bytes < paged_workspace(pool.head_dim, &p.ws, base)) return TV_E_WORKSPACE;
  *sms = num_sms();
  if (*sms <= 0) return TV_E_CUDA;
  p.pool = pool;
  p.seqs = *seqs;
  p.ids = ids;
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.k_new = reinterpret_cast<const __nv_bfloat16*>(k_new);
  p.v_new = reinterpret_cast<const __nv_bfloat16*>(v_new);
  p.q_stride = q_stride;
  p.kv_stride = kv_stride;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.status = dev_status;
  p.layer = layer;
  p.n = n;
  p.Hq = n_q_heads;
  p.window = window;
  p.sinks = sinks;
  p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)pool.head_dim));
  return TV_OK;
}

int launch_paged_merge(const PaParams& p, int ctas, cudaStream_t st) {
  return p.pool.head_dim == 128 ? launch_pdl(paged_merge_kernel<128>, dim3(ctas), dim3(kMergeThreads), 0, st, p)
                                : launch_pdl(paged_merge_kernel<64>, dim3(ctas), dim3(kMergeThreads), 0, st, p);
}

}  // namespace tv

using namespace tv;

extern "C" {

int tv_attend_paged_workspace_size(const tv_pool* pool, int n_q_heads, int n, size_t* bytes) {
  int rc = check_pool(pool);
  if (rc || (rc = check_paged_heads(n_q_heads, pool->n_kv_heads, n))) return rc;
  if (!bytes) return TV_E_ARG;
  *bytes = paged_workspace(pool->head_dim, nullptr, nullptr);
  return TV_OK;
}

int tv_attend_paged(const tv_pool* pool, int layer, const tv_seqs* seqs, const int32_t* ids, int n, int n_q_heads,
                    const tv_bf16* q, size_t q_stride, const tv_bf16* k_new, const tv_bf16* v_new, size_t kv_stride,
                    tv_bf16* out, void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  return attend_paged(false, pool, layer, seqs, ids, n, n_q_heads, 0x7fffffff, 0, q, q_stride, k_new, v_new, kv_stride,
                      out, workspace, workspace_bytes, dev_status, stream);
}

int tv_attend_paged_window(const tv_pool* pool, int layer, const tv_seqs* seqs, const int32_t* ids, int n, int n_q_heads,
                           int window, int sinks, const tv_bf16* q, size_t q_stride, const tv_bf16* k_new,
                           const tv_bf16* v_new, size_t kv_stride, tv_bf16* out, void* workspace, size_t workspace_bytes,
                           int32_t* dev_status, void* stream) {
  return attend_paged(true, pool, layer, seqs, ids, n, n_q_heads, window, sinks, q, q_stride, k_new, v_new, kv_stride, out,
                      workspace, workspace_bytes, dev_status, stream);
}

}  // extern "C"
