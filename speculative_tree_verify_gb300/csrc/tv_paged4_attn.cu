// Attention of one new token per sequence over a paged cache in 4 bits (tv_pool4),
// through a window or not:
//   o[i, h] = sum_j softmax_j(q[i, h] . k[j, g] / sqrt(D)) v[j, g],  k, v = n s,
// n the codes less 8, s a scale of each token's 32 dimensions.
//
// What bounds it: 9/8 bytes a value of K and V together, so that instructions
// come near to memory: a block of 16 tokens of one head (2.3 KB of K and V at
// D = 128) is some 100 cycles of an SM's share of the bandwidth, and 128 sequences of
// 8k take 152 a block now (270 us; 4.5 TB/s): 374 instructions on four schedulers,
// everything counted (48 such sequences), and half of the time the pipe of masks and
// conversions is taken.  Hence:
// - The cache lies as the tensor cores' operands do (tv_pool4): a lane loads its
//   codes with 16-byte loads, no ldmatrix, no shuffle.
// - Codes become operands without arithmetic: bits masked out of 16 are a whole number
//   times the type's smallest subnormal.  K goes in as bf16, n' 2^-133 or 16 times that,
//   n' = n + 8 (q, which is bf16 as it stands, carries the 16th part).  The tensor cores
//   align products as if subnormals were the smallest normal value and keep 25 bits, so
//   that of a code's products 2^-18 of the largest q of 16 dimensions is kept (fp16: 2^-15).
//   V goes in as fp16, as do the weights: n' 2^-24, and 8 bits (n' + 16 n") 2^-24 of
//   neighbours, which come apart at the end: that saves a mask.
//   (e4m3 products, to which four bits are an operand as well, turn into
//   conversions and fp16 products on this architecture: 549 us instead of 346.)
// - Both products have the codes as the operand of 16 rows and 8 heads as columns
//   (S^T = K Q^T, O^T += V^T P^T): up to 8 heads a KV head cost half of what 16 do
//   (346 -> 292 us).  -8 sum q of a group of 32 dimensions is added to its sum, which
//   then takes the token's scale; V's codes become n 2^-9, normal values, by one packed
//   multiply-add (subtracted only, they lost what is 2^-15 of the heaviest of 16 tokens).
// - A token's V scale goes into its weight, four weights of fp16 a token (one a
//   group), so that V needs no product.  The weights are relative to the largest
//   scale so far, as they are to the offset: 2^15 at most, and 2^7 for the largest
//   weight times the largest scale where an offset is set, so that fp16 has its 11
//   bits down to 2^-20 of that and a step of 2^-24, 2^-30 of it or less, below.
//
// How the work is cut over CTAs is in tv_paged_runs.cuh.  In a CTA four warps look
// up pages (32 boxes' entries at a time, the next 32 on their way) and copy whole
// blocks into a ring of stages, each every fourth tile (one warp alone issued one
// in 1200 cycles: 549 -> 346 us); the others compute, tile t by warps
// 2 (t mod teams) and the next, 32 tokens each (16 each: 292 us instead of 271).
#include <cmath>
#include <type_traits>

#include <cuda_fp16.h>

#include "tv_paged_runs.cuh"
#include "tv_pages4.cuh"

namespace tv {
namespace {

constexpr int kStages = 12;                      // tiles in flight: 108 KB at D = 128
// Each has every fourth tile, so that a stage (and a place of the queries) always
// belongs to the same warp: its waits then see every phase of the place's
// barrier, and a parity can not name the phase before last.
constexpr int kLoadWarps = 4;
static_assert(kStages % kLoadWarps == 0, "a stage always belongs to the same loading warp");
constexpr int kQueries = 8;                      // runs whose queries are loaded ahead, at most
// What a head block costs besides its tiles, in tiles: its queries, the wait of
// all warps for the last one's, its join.  128 sequences of 1 to 8191 tokens, 40/8
// heads, with 1, 3, 5, 8 tiles: 98, 85, 72, 64 us.
constexpr int kSegCost = 8;
constexpr float kMoveLog2 = 8.f;                 // offsets move when a score passes them by this
constexpr float kFar = 1024.f;                   // a move by less rounds a score by 2^-14 at most

// HN: blocks of 8 heads
template <int D, int HN>
struct P4 {
  using B = Block4<D>;
  static constexpr int WARPS = HN == 1 ? 12 : 8;   // that compute; the accumulators of 16 heads need the other half's registers
  static constexpr int TEAMS = WARPS / 2;          // two warps a tile, two blocks of 16 tokens each
  static constexpr int THREADS = 32 * (WARPS + kLoadWarps);
  static constexpr int HEADS = 8 * HN;
  // registers: the launch's, and how its warpgroups divide them
  static constexpr int REGS = 65536 / THREADS / 8 * 8, LOAD_REGS = 72;
  static constexpr int COMP_REGS = (REGS * THREADS - LOAD_REGS * 32 * kLoadWarps) / (32 * WARPS) / 8 * 8;
  static_assert(COMP_REGS * 32 * WARPS + LOAD_REGS * 32 * kLoadWarps <= REGS * THREADS, "registers of the launch");
  static constexpr int HALF = kTile / 16 * B::BYTES;   // a tile's K (or V)
  static constexpr int STAGE = 2 * HALF;
  static constexpr int OFF_RED = kStages * STAGE;      // [WARPS][HEADS][D] fp32; the marks of listed rows first
  static constexpr int OFF_ML = OFF_RED + WARPS * HEADS * D * 4;
  static constexpr int Q_ROW = D * 2 + 16;
  static constexpr int OFF_Q = OFF_ML + WARPS * kRows * 8;
  static constexpr int OFF_BAR = OFF_Q + 2 * kRows * Q_ROW;
  static constexpr int OFF_FIRST = OFF_BAR + 512;
  static size_t bytes(int n) { return 128 + OFF_FIRST + (size_t)(n + 1) * 4 + (n <= kInfo ? (size_t)n * 8 : 0); }
  static_assert(kStages % TEAMS == 0, "a stage always belongs to the same two warps");
  static_assert((2 * kStages + 2 * kQueries) * 8 <= 512, "barriers");
  static_assert(WARPS * HEADS * D * 4 >= kMaxSeqs / 8, "a mark for every table row");
  static_assert(128 + OFF_FIRST + (kMaxTokens + 1) * 4 <= 232448 - 512, "shared memory of one CTA");
  static_assert(HALF % 16 == 0 && B::BYTES % 16 == 0, "bulk copies");
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1, float c0, float c1, float c2, float c3) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, float c0, float c1, float c2, float c3) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// two whole numbers times 2^-24, less `off` of them, to whole numbers times 2^-9
template <int OFF>
__device__ __forceinline__ uint32_t lift_f16(uint32_t a) {
  static_assert(OFF == 8 || OFF == 136, "");
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(0x78007800u), "r"(OFF == 8 ? 0xa400a400u : 0xb440b440u));   // 2^15, -OFF 2^-9
  return r;
}
// an 8 x 8 matrix of 16-bit values, a row to four lanes, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
// mbar_wait of warps with nothing to do meanwhile: asleep between looks, so that
// they do not take issue slots from those that compute
__device__ __forceinline__ bool mbar_sleep(uint64_t* bar, uint32_t parity) {
  for (uint32_t n = 0; n < (uint32_t)(kWaitLimitNs / 1000); ++n) {   // (a sleep is up to twice as long)
    if (mbar_test(bar, parity)) return true;
    __nanosleep(500);
  }
  return mbar_wait(bar, parity);
}
// G words of shared memory, 4 G bytes aligned
template <int G>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t (&w)[G]) {
  if constexpr (G == 4)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a) : "memory");
  else
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a) : "memory");
}

template <int D, int HN>
__global__ void __launch_bounds__(P4<D, HN>::THREADS, 1) paged4_attn_kernel(const __grid_constant__ PaParams p) {
  using L = P4<D, HN>;
  using B = Block4<D>;
  constexpr int G = B::G, NW = L::WARPS, NT = L::TEAMS, NS = 2;   // NS: blocks of 16 tokens of a warp's tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* empty = full + kStages;
  uint64_t* q_full = empty + kStages;    // [kQueries] a run's queries landed
  uint64_t* q_free = q_full + kQueries;  // [kQueries] all warps have seen them, those that compute it are done with them
  uint32_t* s_first = reinterpret_cast<uint32_t*>(smem + L::OFF_FIRST);
  float* s_red = reinterpret_cast<float*>(smem + L::OFF_RED);
  float2* s_ml = reinterpret_cast<float2*>(smem + L::OFF_ML);
  uint32_t* s_mark = reinterpret_cast<uint32_t*>(smem + L::OFF_RED);
  __shared__ uint32_t s_part[L::THREADS / 32];
  __shared__ int s_bad;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ps = p.pool.page_size, Hkv = p.pool.n_kv_heads;
  const int qrows = min(kRows, p.G), qslots = min(kQueries, 2 * kRows / qrows);

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 2);   // the two warps that compute its tile
    }
    for (int s = 0; s < kQueries; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_free[s], NW);
    }
    fence_mbar_init();
    s_bad = 0;
  }
  if (p.n > 32 && p.k_new)
    for (int i = tid; i < (p.seqs.max_seqs + 31) / 32; i += L::THREADS) s_mark[i] = 0u;
  __syncthreads();
  pdl_wait();
  pdl_trigger();

  RunList<L::THREADS, kSegCost, true> runs(p, s_first);
  if (!runs.build(s_mark, s_part, &s_bad)) return;
  // sequences without a token: zeros
  for (int i = blockIdx.x; i < p.n; i += gridDim.x)
    if (s_first[i + 1] == s_first[i])
      for (int e = tid; e < p.Hq * D / 8; e += L::THREADS)
        reinterpret_cast<uint4*>(p.out + (size_t)i * p.Hq * D)[e] = make_uint4(0u, 0u, 0u, 0u);
  runs.range();
  if (tid == 0) p.ws.cut[blockIdx.x] = make_int4(-1, 0, 0, 0);
  if (runs.lo >= runs.hi) return;

  if (warp >= NW) {
    // ---------------- pages and loads ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::LOAD_REGS));
    const int mine = warp - NW;                            // tiles with (count mod kLoadWarps) == mine, and places of queries
    const int R = ps < kTile ? ps : kTile;                 // tokens of a box
    const int nsh = 6 - (31 - __clz(R)), nb = 1 << nsh;    // boxes of a tile
    const int psh = 31 - __clz(ps), per = 32 >> nsh;       // tiles of 32 boxes
    const size_t head_bytes = (size_t)(ps / 16) * B::BYTES;
    bool ok = true;
    int count = 0, segs = 0;     // tiles and runs so far, anyone's
    auto wait = [&](uint64_t* bar, uint32_t parity) { ok = __all_sync(0xffffffffu, mbar_sleep(bar, parity & 1u)); };
    // blocks [a, b) of the box at tok hold tokens that are seen
    auto blocks = [&](const Run& g, int tok, int& a, int& b) {
      a = 0;
      b = (min(R, g.len - tok) + 15) >> 4;
      if (tok >= p.sinks) a = max(0, g.lo - tok) >> 4;
      else if (tok <= g.lo - R) b = min(b, (p.sinks - tok + 15) >> 4);   // (sinks and window in one box: all of it)
    };
    auto entry = [&](const Run& g, int tb) {   // the page of this lane's box of tiles tb ..., -1: not seen
      const int t = tb + (lane >> nsh);
      if (t >= g.t1) return -1;
      const int tok = g.tile<true>(t) * kTile + (lane & (nb - 1)) * R;
      if (tok >= g.len) return -1;
      int a, b;
      blocks(g, tok, a, b);
      return a < b ? __ldcg(p.seqs.pages + (size_t)g.s * p.seqs.max_pages + (tok >> psh)) : -1;
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
        for (int t = tb + ((mine - count) & (kLoadWarps - 1)); t < end; t += kLoadWarps) {
          const int issued = count + (t - tb), st = issued % kStages;
          // lane 2 b: K of box b, lane 2 b + 1: V
          const int box = lane >> 1;
          const int page = __shfl_sync(0xffffffffu, pages, ((t - tb) << nsh) + (box & (nb - 1)));
          const int tok = g.tile<true>(t) * kTile + box * R;
          int a = 0, b = 0;
          if (box < nb && tok < g.len) blocks(g, tok, a, b);
          const bool in = a < b, good = in && page >= 0 && page < p.pool.n_pages;
          if (in && !good) status_set(p.status, TV_E_PAGE);
          const uint32_t bytes = good ? (uint32_t)((b - a) * B::BYTES) : 0u;
          const uint32_t total = __reduce_add_sync(0xffffffffu, bytes);
          if (issued >= kStages) wait(&empty[st], (uint32_t)(issued / kStages - 1));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&full[st], total);
          __syncwarp();
          if (good) {
            const uint8_t* src = reinterpret_cast<const uint8_t*>(lane & 1 ? p.pool.v : p.pool.k) +
                                 (((size_t)p.layer * p.pool.n_pages + page) * Hkv + g.h) * head_bytes +
                                 (size_t)(((tok & (ps - 1)) >> 4) + a) * B::BYTES;
            bulk_load(smem + st * L::STAGE + (lane & 1) * L::HALF + (box * (R / 16) + a) * B::BYTES, src, bytes, &full[st]);
          }
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
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::COMP_REGS));
  const int team = warp >> 1, first = 32 * (warp & 1);   // tiles with (count mod NT) == team; tokens first .. + 31 of a tile
  const int g8 = lane >> 2, t4 = lane & 3;
  const uint32_t pick = g8 & 1 ? 0x3244u : 0x1044u;   // of a word of two bf16, token g8's as fp32
  auto meet = [&](int nw) {
    asm volatile("bar.sync %0, %1;" ::"r"(nw == NW ? 1 : 2 + team), "r"(32 * nw) : "memory");
  };
  bool ok = true;
  // this warp's next tile and the CTA's next queries: places in the rings, parities
  int st = team, qs = 0;
  uint32_t st_par = 0u, qs_par = 0u;
  int turn = team;   // tiles of the CTA until its next one
  Run g;
  for (bool have = runs.first_run(g); have; have = runs.next_run(g)) {
    const int h = g.h, r0 = g.hb * kRows;   // KV head, first query head of the block in the group
    const int nr = min(kRows, p.G - r0);
    if (ok && !mbar_wait(&q_full[qs], qs_par)) ok = false;
    if (g.T == 1 && turn > 0) {   // one tile, and another team's
      // (no further ahead than the queries, nor further behind than their place:
      // it is not loaded again before these warps, too, have seen this phase)
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_free[qs]);
      --turn;
      if (++qs == qslots) qs = 0, qs_par ^= 1u;
      continue;
    }
    // Queries, as columns: head g8 (and g8 + 8), dimensions 32 j + 8 t4 .. + 7 of
    // group j, q0 .. q7, relative to the row's exponent: (q0, q4), (q1, q5) / 16,
    // (q2, q6), (q3, q7) / 16: exact.
    uint32_t q[HN][G][4];
    // of heads 2 t4 and 2 t4 + 1: -8 sum q of a group; what a product of q and codes is worth
    float bias[HN][G][2], sc[HN][2];
#pragma unroll
    for (int b = 0; b < HN; ++b) {
      // rows past the group's heads: the last one again, products nobody reads
      const uint32_t row = smem_u32(smem) + L::OFF_Q + (qs * qrows + min(g8 + 8 * b, nr - 1)) * L::Q_ROW + t4 * 16;
      uint32_t x[G][4];
      uint32_t top = 0u;
#pragma unroll
      for (int j = 0; j < G; ++j) {
        lds_words<4>(row + j * 64, x[j]);
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[j][0] & 0x7fff7fffu, x[j][1] & 0x7fff7fffu),
                                     __vmaxu2(x[j][2] & 0x7fff7fffu, x[j][3] & 0x7fff7fffu)));
      }
      top = max(top & 0xffffu, top >> 16);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // the largest to 2^120 .. 2^121, by two factors that are normal
      const int e = max((int)(top >> 7), 1), up = 247 - e;   // 127 + exponent
      const float f = __uint_as_float((uint32_t)(127 + min(up, 127)) << 23), f2 = __uint_as_float((uint32_t)(127 + max(up - 127, 0)) << 23);
      const float worth = p.scale_log2 * __uint_as_float((uint32_t)min(e + 13, 254) << 23);   // 2^(133 - up)
      sc[b][0] = __shfl_sync(0xffffffffu, worth, 8 * t4);
      sc[b][1] = __shfl_sync(0xffffffffu, worth, 8 * t4 + 4);
#pragma unroll
      for (int j = 0; j < G; ++j) {
        float sum = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {   // dimensions u and u + 4: halves u % 2 of words u / 2 and u / 2 + 2
          const float k = u & 1 ? f2 * 0.0625f : f2;
          const uint32_t y = x[j][u >> 1], z = x[j][(u >> 1) + 2];
          const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(u & 1 ? y & 0xffff0000u : y << 16) * f * k,
                                                         __uint_as_float(u & 1 ? z & 0xffff0000u : z << 16) * f * k);
          const float2 r = __bfloat1622float2(v);
          q[b][j][u] = *reinterpret_cast<const uint32_t*>(&v);
          sum += (r.x + r.y) * (u & 1 ? 16.f : 1.f);
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sum *= -0x1p-65f;   // -8 * 2^-133
        sum *= 0x1p-65f;
        bias[b][j][0] = __shfl_sync(0xffffffffu, sum, 8 * t4);
        bias[b][j][1] = __shfl_sync(0xffffffffu, sum, 8 * t4 + 4);
      }
    }
    // O^T: o[8 heads][j][0 .. 3] rows 32 j + 4 g8, that and 16 times the next, heads 2 t4, 2 t4 + 1; [4 .. 7]: two rows more
    float o[HN][G][8];
    // Weights are 2^(score - off) and go up to 2^limit: off is the head's offset less
    // what lifts the weights to fp16's range beside the scales, limit = 15 - log2 vtop.
    float off[HN][2], l[HN][2];  // l: sums of this thread's tokens
    float vtop = 0x1p-80f;       // power of two above the scales of V so far; at least so much that
    float limit = 95.f;          // a sum of 2^30 weights, whose V may all be zero, stays below 2^128
#pragma unroll
    for (int b = 0; b < HN; ++b) {
      off[b][0] = off[b][1] = 0.f, l[b][0] = l[b][1] = 0.f;
#pragma unroll
      for (int j = 0; j < G; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) o[b][j][e] = 0.f;
    }

    bool fresh = true;           // no token so far
    int t = g.t0 + turn;
    uint32_t again = 0u;         // a tile for the second time: a bit for each head whose offset moved far, and one more
    while (t < g.t1) {
      uint8_t* sk = smem + st * L::STAGE + first / 16 * B::BYTES;
      uint8_t* sv = sk + L::HALF;
      if (ok && !mbar_wait(&full[st], st_par)) ok = false;
      const uint32_t ka = smem_u32(sk), va = ka + L::HALF;
      // All of the warp's tokens are seen but in a sequence's last tile, the
      // window's first and the sinks' last.
      const bool special = t == g.T - 1 || (g.lo > 0 && (t == g.sink_tiles || t == g.sink_tiles - 1));
      const int tok0 = special ? g.tile<true>(t) * kTile + first : 0;
      auto out = [&](int tok) { return tok >= g.len || (tok >= p.sinks && tok < g.lo); };
      bool wrote = false;
      if (special && p.k_new && tok0 < g.len && g.len - tok0 <= 32) {
        // the new token: its codes into the tile and into the page
        const bool is_v = lane >= 16;
        const int c = lane & 15, at = g.len - 1, tk = at & 15, half = tk % 2 * 2;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (c < D / 8)
          x = __ldcg(reinterpret_cast<const uint4*>((is_v ? p.v_new : p.k_new) + (size_t)g.i * p.kv_stride + (size_t)h * D) + c);
        uint32_t scale;
        const uint32_t w = round4(x, scale);
        const int page = __ldcg(p.seqs.pages + (size_t)g.s * p.seqs.max_pages + at / ps);
        if (c < D / 8) {
          auto put = [&](uint8_t* block) {
            if (is_v) {
              *reinterpret_cast<uint16_t*>(block + B::v_word(tk, 2 * c) + half) = (uint16_t)w;
              *reinterpret_cast<uint16_t*>(block + B::v_word(tk, 2 * c + 1) + half) = (uint16_t)(w >> 16);
            } else {
              *reinterpret_cast<uint32_t*>(block + B::k_word(tk, c)) = w;
            }
            if (c % 4 == 0) *reinterpret_cast<uint16_t*>(block + B::scale(tk, c / 4) + half) = (uint16_t)scale;
          };
          put((is_v ? sv : sk) + (at - tok0) / 16 * B::BYTES);
          if (r0 == 0 && page >= 0 && page < p.pool.n_pages)
            put(reinterpret_cast<uint8_t*>(is_v ? p.pool.v : p.pool.k) +
                ((((size_t)p.layer * p.pool.n_pages + page) * Hkv + h) * ps + at % ps / 16 * 16) / 16 * B::BYTES);
        }
        wrote = true;
        __syncwarp();
      }
      if (!special || __any_sync(0xffffffffu, !out(tok0 + lane))) {
        // Tokens of this thread, as rows of S^T: g8 (n = 0) and g8 + 8 (1) of each block.
        float x[NS][HN][2][2];   // [n][head]
        uint32_t sb[NS][2][G];   // scales of V: of g8 and its neighbour
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          uint32_t w[2][G], sa[2][G];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            lds_words<G>(ka + s * B::BYTES + (8 * n + g8) * (D / 2) + t4 * (D / 8), w[n]);
            lds_words<G>(ka + s * B::BYTES + B::OFF_SCALE + (n * 4 + (g8 >> 1)) * G * 4, sa[n]);
            lds_words<G>(va + s * B::BYTES + B::OFF_SCALE + (n * 4 + (g8 >> 1)) * G * 4, sb[s][n]);
          }
#pragma unroll
          for (int j = 0; j < G; ++j) {
            const uint32_t w0 = w[0][j], w1 = w[1][j];
            const uint32_t u0 = __byte_perm(w0, 0u, 0x4341), u1 = __byte_perm(w1, 0u, 0x4341);   // its second and fourth bytes
            const float s0 = __uint_as_float(__byte_perm(sa[0][j], 0u, pick)), s1 = __uint_as_float(__byte_perm(sa[1][j], 0u, pick));
#pragma unroll
            for (int b = 0; b < HN; ++b) {
              float c[4];
              mma_bf16(c, w0 & 0x000f000fu, w1 & 0x000f000fu, w0 & 0x00f000f0u, w1 & 0x00f000f0u, q[b][j][0], q[b][j][1],
                       0.f, 0.f, 0.f, 0.f);
              mma_bf16(c, u0 & 0x000f000fu, u1 & 0x000f000fu, u0 & 0x00f000f0u, u1 & 0x00f000f0u, q[b][j][2], q[b][j][3], c[0],
                       c[1], c[2], c[3]);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float(&y)[2][2] = x[s][b];
                y[0][e] = j == 0 ? (c[e] + bias[b][j][e]) * s0 : fmaf(c[e] + bias[b][j][e], s0, y[0][e]);
                y[1][e] = j == 0 ? (c[2 + e] + bias[b][j][e]) * s1 : fmaf(c[2 + e] + bias[b][j][e], s1, y[1][e]);
              }
            }
          }
        }
        if (special) {   // what is past the length or hidden: no score, and a scale of zero, whatever it holds
#pragma unroll
          for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const int tok = tok0 + 16 * s + 8 * n + (g8 & ~1);
              const bool even = out(tok), odd = out(tok + 1);
              if (g8 & 1 ? odd : even)
#pragma unroll
                for (int b = 0; b < HN; ++b) x[s][b][n][0] = x[s][b][n][1] = -INFINITY;
              const uint32_t keep = (even ? 0u : 0x0000ffffu) | (odd ? 0u : 0xffff0000u);
#pragma unroll
              for (int j = 0; j < G; ++j) sb[s][n][j] &= keep;
            }
        }
        // exponents; the offsets move when passed, as the largest scale does, hardly ever
        float most = -INFINITY;
        const uint32_t vt = __byte_perm(__float_as_uint(vtop), 0u, 0x3232);   // its upper half twice
        uint32_t top = vt;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
#pragma unroll
          for (int b = 0; b < HN; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float& z = x[s][b][e >> 1][e & 1];
              z = fmaf(z, sc[b][e & 1], -off[b][e & 1]);
              most = fmaxf(most, z);
            }
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int j = 0; j < G; j += 2) top = __vimax3_u16x2(top, sb[s][n][j], sb[s][n][j + 1]);
        }
        if (__any_sync(0xffffffffu, fresh || most > limit || top != vt || again != 0u)) {
          uint32_t far = 0u;
          // scales that are NaN say nothing of the others
          top = 0u;
#pragma unroll
          for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int j = 0; j < G; ++j) {
                const uint32_t a = sb[s][n][j] & 0xffffu, b = sb[s][n][j] >> 16;
                top = max(top, max(a < 0x7f80u ? a : 0u, b < 0x7f80u ? b : 0u));
              }
          top = __reduce_max_sync(0xffffffffu, top);
          float down = 0.f;   // log2 of vtop's growth
          if (__uint_as_float(top << 16) > vtop) {   // to the next power of two
            down = (float)((int)(top >> 7) + 1 - (int)(__float_as_uint(vtop) >> 23));
            vtop = __uint_as_float(((top >> 7) + 1u) << 23);
            limit -= down;
          }
#pragma unroll
          for (int b = 0; b < HN; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float y = -INFINITY;   // the largest, by the tokens of all lanes
#pragma unroll
              for (int s = 0; s < NS; ++s) y = fmaxf(y, fmaxf(x[s][b][0][e], x[s][b][1][e]));
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
              y -= down;
              // the offset to 2^kMoveLog2 above the largest, or as it was
              const uint32_t head = 1u << (2 * b + e);
              const float up = (fresh || y > limit || (again & head) != 0u ? y - (limit - kMoveLog2) : 0.f) + down;
              const float now = off[b][e] + up, move = now - off[b][e];   // (rounded, as the offset is)
              // 2^-move as a square: scales that grow from next to nothing take it beyond what
              // one factor can hold, and the weights so far are still the sum's
              const float a = ex2f(-0.5f * move);
              if (fabsf(move) >= kFar) far |= head;
              off[b][e] = now;
#pragma unroll
              for (int s = 0; s < NS; ++s) x[s][b][0][e] -= move, x[s][b][1][e] -= move;
              l[b][e] = fresh ? 0.f : l[b][e] * a * a;
#pragma unroll
              for (int j = 0; j < G; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[b][j][2 * i + e] = fresh ? 0.f : o[b][j][2 * i + e] * a * a;
            }
          fresh = false;
          // A score of kFar and more, less the offset from before a move by as much, has lost
          // places that matter behind the move: then the tile once more, so that tokens of equal
          // scores weigh the same wherever they are, and the offset by what is exact now.
          if (again == 0u && __any_sync(0xffffffffu, far != 0u)) {
            again = far | 0x100u;
            continue;
          }
        }
#pragma unroll
        for (int s = 0; s < NS; ++s) {
#pragma unroll
          for (int b = 0; b < HN; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float& y = x[s][b][e >> 1][e & 1];
              y = ex2f(y);
              l[b][e & 1] += y;
            }
          uint32_t vw[2][G];
#pragma unroll
          for (int n = 0; n < 2; ++n) lds_words<G>(va + s * B::BYTES + (n * 32 + lane) * G * 4, vw[n]);
#pragma unroll
          for (int j = 0; j < G; ++j) {
            // rows of V^T: dimensions 4 g8, that and 16 times the next, two more; columns: tokens 2 t4, 2 t4 + 1 and 8 more
            uint32_t a[4][2];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const uint32_t w = vw[n][j], u1 = __byte_perm(w, 0u, 0x4341);
              a[0][n] = lift_f16<8>(w & 0x000f000fu);
              a[1][n] = lift_f16<136>(w & 0x00ff00ffu);
              a[2][n] = lift_f16<8>(u1 & 0x000f000fu);
              a[3][n] = lift_f16<136>(u1);
            }
#pragma unroll
            for (int b = 0; b < HN; ++b) {
              uint32_t pw[2];   // weights of this group, columns now: tokens 2 t4, 2 t4 + 1 (and 8 more) of head g8
#pragma unroll
              for (int n = 0; n < 2; ++n) {
                const float y = __uint_as_float(__byte_perm(sb[s][n][j], 0u, pick));
                pw[n] = transpose8(pack_f16(x[s][b][n][0] * y, x[s][b][n][1] * y));
              }
              float(&lo)[4] = *reinterpret_cast<float(*)[4]>(&o[b][j][0]);
              float(&hi)[4] = *reinterpret_cast<float(*)[4]>(&o[b][j][4]);
              mma_f16(lo, a[0][0], a[1][0], a[0][1], a[1][1], pw[0], pw[1], lo[0], lo[1], lo[2], lo[3]);
              mma_f16(hi, a[2][0], a[3][0], a[2][1], a[3][1], pw[0], pw[1], hi[0], hi[1], hi[2], hi[3]);
              // less 8 (and 8 + 16 * 8) of every code
            }
          }
        }
        if (wrote) fence_async_smem();   // before the stage takes another copy
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
      if ((st += NT) >= kStages) st = team, st_par ^= 1u;
      again = 0u;
      t += NT;
    }
    turn = t - g.t1;

    // ---- the head block's partial results into one ----
    // of all warps, or, where the head block is one tile, of the two that had
    // it: the others go on to the next head block meanwhile
    const bool whole = g.t0 == 0 && g.t1 == g.T;
    const int nw = g.T > 1 ? NW : 2, w0 = g.T > 1 ? 0 : 2 * team, me = tid - 32 * w0;
    // a CTA's first run may begin inside a head block, its last end inside one
    const size_t slot = (size_t)blockIdx.x * 2 + (g.t0 == 0 ? 1 : 0);
    // the weights' lift, 2^7 / vtop, is the offset's again; what the offset's rounding drops stays in the weights
    const float lift = limit - kMoveLog2, unlift = __uint_as_float(__float_as_uint(vtop) - (7u << 23));
#pragma unroll
    for (int b = 0; b < HN; ++b) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float at = off[b][e] + lift, rest = ex2f(lift - (at - off[b][e]));
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[b][e] += __shfl_xor_sync(0xffffffffu, l[b][e], d);
        if (g8 == 0) s_ml[warp * kRows + 8 * b + 2 * t4 + e] = make_float2(fresh ? -INFINITY : at, l[b][e] * unlift * rest);
        // head 8 b + 2 t4 + e, dimensions 32 j + 4 g8 .. + 3: chunks turned by the head, no bank twice
        float* dst = s_red + ((size_t)warp * L::HEADS + 8 * b + 2 * t4 + e) * D + ((g8 + 2 * t4) & 7) * 4;
        const float worth = 4.f * vtop * rest, part = 0.25f * vtop * rest;   // what the codes' and the weights' factors leave
        if (8 * b + 2 * t4 + e < nr)
#pragma unroll
          for (int j = 0; j < G; ++j) {
            const float(&r)[8] = o[b][j];
            *reinterpret_cast<float4*>(dst + 32 * j) =
                make_float4(r[e] * worth, (r[2 + e] - r[e]) * part, r[4 + e] * worth, (r[6 + e] - r[4 + e]) * part);
          }
      }
    }
    meet(nw);
    if (lane == 0) mbar_arrive(&q_free[qs]);
    for (int e = me; e < nr * (D / 4); e += 32 * nw) {
      const int row = e / (D / 4), d = e % (D / 4);   // head, four dimensions
      float M = -INFINITY, sum = 0.f;
      for (int w = 0; w < nw; ++w) M = fmaxf(M, s_ml[(w0 + w) * kRows + row].x);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      const float* src = s_red + ((size_t)w0 * L::HEADS + row) * D + d / 8 * 32 + ((d + (row & 6)) & 7) * 4;
#pragma unroll 4
      for (int w = 0; w < nw; ++w) {
        const float2 x = s_ml[(w0 + w) * kRows + row];
        const float4 v = *reinterpret_cast<const float4*>(src + (size_t)w * L::HEADS * D);
        const float f = ex2f(x.x - M);
        sum = fmaf(x.y, f, sum);
        acc.x = fmaf(v.x, f, acc.x);
        acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z);
        acc.w = fmaf(v.w, f, acc.w);
      }
      if (whole) {
        const float f = 1.f / sum;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * f, acc.y * f), hi = __floats2bfloat162_rn(acc.z * f, acc.w * f);
        *reinterpret_cast<uint2*>(p.out + ((size_t)g.i * p.Hq + h * p.G + r0 + row) * D + 4 * d) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      } else {
        *reinterpret_cast<float4*>(p.ws.o + (slot * kRows + row) * D + 4 * d) = acc;
        if (d == 0) *reinterpret_cast<float2*>(p.ws.ml + (slot * kRows + row) * 2) = make_float2(M, sum);
      }
    }
    meet(nw);   // before the places of the sums are written again
    if (++qs == qslots) qs = 0, qs_par ^= 1u;
    if (tid == 0 && g.t0 == 0 && !whole)   // the CTA's last run
      p.ws.cut[blockIdx.x] = make_int4(g.i, g.h * p.HB + g.hb, (int)((g.base + g.T - 1) / runs.chunk), 0);
  }
  if (!ok && lane == 0) status_set(p.status, TV_E_TIMEOUT);
}

template <int D, int HN>
int launch_paged4(const PaParams& p, int ctas, cudaStream_t st) {
  static std::atomic<bool> attr[64];
  if (ensure_smem_limit(paged4_attn_kernel<D, HN>, P4<D, HN>::bytes(kMaxTokens), attr)) return TV_E_CUDA;
  // the split of the registers must not ask for more than the launch brings
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, paged4_attn_kernel<D, HN>) != cudaSuccess) return TV_E_CUDA;
    regs.store(fa.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) < P4<D, HN>::REGS) return TV_E_UNSUPPORTED;
  const int rc = launch_pdl(paged4_attn_kernel<D, HN>, dim3(ctas), dim3(P4<D, HN>::THREADS), P4<D, HN>::bytes(p.n), st, p);
  return rc ? rc : launch_paged_merge(p, ctas, st);
}

}  // namespace
}  // namespace tv

using namespace tv;

extern "C" {

int tv_attend_paged4_workspace_size(const tv_pool4* pool, int n_q_heads, int n, size_t* bytes) {
  PagePool q;
  int rc = check_pool(pool, &q);
  if (rc || (rc = check_paged_heads(n_q_heads, q.n_kv_heads, n))) return rc;
  if (!bytes) return TV_E_ARG;
  *bytes = paged_workspace(q.head_dim, nullptr, nullptr);
  return TV_OK;
}

int tv_attend_paged4(const tv_pool4* pool, int layer, const tv_seqs* seqs, const int32_t* ids, int n, int n_q_heads,
                     int window, int sinks, const tv_bf16* q, size_t q_stride, const tv_bf16* k_new, const tv_bf16* v_new,
                     size_t kv_stride, tv_bf16* out, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                     void* stream) {
  PagePool pages;
  PaParams p;
  int sms;
  int rc = check_pool(pool, &pages);
  if (rc || (rc = fill_paged(p, kSegCost, pages, layer, seqs, ids, n, n_q_heads, window, sinks, q, q_stride, k_new, v_new, kv_stride,
                             out, workspace, workspace_bytes, dev_status, &sms)))
    return rc;
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // up to 8 query heads a KV head take half of the products and registers of 16
  if (p.G <= 8) return pages.head_dim == 128 ? launch_paged4<128, 1>(p, ctas, st) : launch_paged4<64, 1>(p, ctas, st);
  return pages.head_dim == 128 ? launch_paged4<128, 2>(p, ctas, st) : launch_paged4<64, 2>(p, ctas, st);
}

}  // extern "C"
