// Causal attention of packed prompts, grouped heads:
//   o[t, h] = sum_{j <= t} softmax_j(q[t, h] . k[j, g] / sqrt(D)) v[j, g],  g = h / G,
// t and j rows of the same sequence.
//
// What bounds it: 4 D flops a (row, key) pair on the tensor cores, with one
// exponential a pair on the SFU beside them.  So both products run on tcgen05
// and the exponentials of one tile hide behind the products of another.
//
// A CTA takes two tiles of 128 query vectors of one KV head.  The vectors are
// (token, head of the group) pairs, T = 128 / G tokens a tile, so that K and V
// are read once for the whole group and a short prompt fills a tile with its
// heads.  Its keys come in windows of 128, the last first, so that what is
// masked (the corner of the CTA's own tokens, and what lies behind them) is in
// the first windows alone:
//   S_s  = Q_s K_w^T       tcgen05.mma 128 x 128 x D, operands in shared memory
//   P_s  = 2^(S_s c - m)   two threads a row, 64 keys each: scores from TMEM to
//                          registers, exponentials, bf16 back into the first
//                          half of the scores' columns
//   O_s += P_s V_w         tcgen05.mma 128 x D x 128, P from TMEM, V from its
//                          TMA layout (MN-major)
// The issue order PV_0(w) S_0(w + 1) PV_1(w) S_1(w + 1) keeps the tensor pipe
// on one tile while the other's softmax runs.  A row's offset m need not be its
// maximum, only near it; where it is not, O_s is rescaled in TMEM by the row's
// own threads (S_s(w) is committed after PV_s(w - 1), so O_s is at rest).  Sums add the
// rounded P, fp32 throughout.
//
// Five kinds of warps keep their own pace, each one place (a pair of tiles)
// after the other, and meet only on barriers in shared memory: softmax (16),
// products, loads, the next places, and the look at what is masked.  A CTA
// takes over the places of CTAs that have not started, three windows before
// it is done with its own.
//
// Measured (40/8 heads of 128, us; each step with the ones before it): 16k
// tokens 2866 as first built; 1984 with the issuing warp in step (its
// descriptors stay in uniform registers); 1838 with two threads a row; 1749
// with sums instead of maxima; 1690 taking over places; 1654 with headroom in
// the offsets; 1597 to 1684 now (box to box), 1630 to 1720 TFLOP/s: 86 to 91 %
// of what cuBLAS reaches in a burst, 95 to 100 % of its sustained rate.  4k:
// 109 (1.58 PFLOP/s); 24 prompts of 1 to 1531: 59 to 60; one of 1024: 16.5.
// With heads of 64: 16k 1280 (1070 TFLOP/s; the softmax, which does not halve
// with the products).
//
// Masked places: a key that a row may not see has weight zero, and its V may
// be anything.  0 * NaN would reach the row through the product, so the V rows
// past the CTA's first token are looked over in shared memory before they are
// used; what is not finite is taken out and noted (per dimension, the first
// such key), and put into the rows that do see it at the end.
//
// Through a window (WIN: tv_attend_prompt_window) row t sees keys (t - W, t]
// and the first K, the sinks.  Of the pair's keys, those from its first token's
// lowest come in windows of 128.  Where these leave room for the sinks, they are
// counted from the pair's last key down, and the sinks are loaded into the last
// one's lowest steps, below what any row sees (16k tokens, 40/8 heads, W = 1024, K =
// 4, in turn: 281 us with a window of the sinks' own, 273 so, 256 without sinks; the
// present code by itself 279, 274 to 288 a call); else the sinks have windows of
// their own behind the others.  So a pair costs about (W + 2T + 127) / 128 windows,
// whatever the length.  What is masked is now at both
// ends; the lower end's V (keys up to W before the pair's last token) is looked
// over as well, and a pair whose V held something not finite reads its keys again
// from memory at the end, each row those that it sees (put_back): which rows see
// a key is no longer told by one number.
#include <cmath>
#include <type_traits>

#include "tv_gemm.cuh"
#include "tv_kernels.cuh"
#include "tv_pages.cuh"

namespace tv {
namespace {

constexpr int kPrSoftWarps = 16;                 // 8 a query tile
constexpr int kPrSoftThreads = kPrSoftWarps * 32;
constexpr int kWarpMma = kPrSoftWarps, kWarpTma = kPrSoftWarps + 1;
constexpr int kWarpPlan = kPrSoftWarps + 2, kWarpLook = kPrSoftWarps + 3;
constexpr int kPrThreads = kPrSoftThreads + 128;  // a whole warpgroup for the four roles' registers
// 640 threads of 96 registers at launch; 512 x 104 + 128 x 64 is the same sum
constexpr int kSoftRegs = 104, kRoleRegs = 64;
static_assert(kPrSoftThreads * kSoftRegs + 128 * kRoleRegs <= kPrThreads * 96, "registers of the launch");
constexpr int kAtomP = 128 * 128;                // bytes of a 128-row x 128-byte swizzled slab
// offsets, in powers of two (see the softmax): the first one, how far beyond a
// maximum the next ones go, and the sums of 64 exponentials that an offset may have
constexpr float kFirst = 20.f, kAbove = 20.f, kHigh = 256.f, kLow = 8.27180613e-25f;   // 2^-80

template <int D>
struct PrSmem {
  static constexpr int TILE = (D / 64) * kAtomP;   // 128 rows
  static constexpr int OFF_Q = 0;                  // two tiles
  static constexpr int OFF_K = 2 * TILE;           // two stages
  static constexpr int OFF_V = OFF_K + 2 * TILE;   // two stages
  static constexpr int OFF_CNT = OFF_V + 2 * TILE; // tile pairs of every sequence, where there are more than 32
  static constexpr int OFF_BAD = OFF_CNT + kMaxListed * 4;   // [2 places][3][D] first key whose V is NaN, +inf, -inf
  static constexpr int OFF_TOP = OFF_BAD + 2 * 3 * D * 8;    // [2 tiles][2 halves][128 rows] maxima
  static constexpr int OFF_SUM = OFF_TOP + 2 * 2 * 128 * 4;  // and sums
  static constexpr int OFF_BAR = OFF_SUM + 2 * 2 * 128 * 4;
  static constexpr size_t BYTES = 1024 + OFF_BAR + 256;
  static_assert(BYTES <= 232448 - 256, "shared memory of one CTA");
};

struct PrParams {
  const int32_t* starts;
  __nv_bfloat16* out;
  int32_t* status;
  int n, rows, Hq, Hkv, G, T;
  int window, sinks;              // WIN
  const __nv_bfloat16* v;         // WIN: V once more, for put_back
  size_t kv_stride;
  int queued;   // the grid is larger than the GPU: CTAs may be waiting whose places can be taken over
  float scale_log2;
};

__device__ __forceinline__ float ex2p(float x) {   // 2^x by the SFU, about 2^-22 relative, 2^-inf = 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// n consecutive 32-bit TMEM columns of this thread's lane
__device__ __forceinline__ void ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
        "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// two fp32 values in a 64-bit register: one instruction for both
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// a += x, x the bits of a bf16
__device__ __forceinline__ void add_bf16(float& a, uint16_t x) {
  asm("add.rn.f32.bf16 %0, %1, %0;" : "+f"(a) : "h"(x));
}
__device__ __forceinline__ float max3(float a, float b, float c) {   // NaN inputs are ignored
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// the two warps of a pair: all have come; true if v is true on any thread
__device__ __forceinline__ void pair_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool pair_any(bool v, int id) {
  uint32_t out;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "bar.red.or.pred p, %2, 64, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(out)
      : "r"((uint32_t)v), "r"(id)
      : "memory");
  return out != 0;
}
__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The issuing warp runs as one (no branch on the lane), so that descriptors and
// loop counters stay in its uniform registers, where the MMA takes them from;
// the instructions themselves carry the elected lane's predicate.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r;
}
// D[tmem] (+)= A[smem desc] * B[smem desc]^T
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem desc]: A holds two bf16 of a row per 32-bit column
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void commit_by(uint64_t* bar, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(leader)
      : "memory");
}

// ---- cluster launch control: the index of a CTA that has not started, whose
// work this CTA takes over (16 bytes written to shared memory, counted on the
// barrier)
__device__ __forceinline__ void clc_ask(void* answer, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
               :
               : "r"(smem_u32(answer)), "r"(smem_u32(bar))
               : "memory");
}
// -1: every CTA has started
__device__ __forceinline__ int clc_answer(const void* answer) {
  uint32_t x, got;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\t.reg .b32 y, z, w;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %1, 1, 0, p;\n\t"
      "mov.b32 %0, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, w}, h;\n\t}"
      : "=r"(x), "=r"(got)
      : "r"(smem_u32(answer))
      : "memory");
  return got ? (int)x : -1;
}

// a * 0 + c of two bf16 each
__device__ __forceinline__ uint32_t times_zero(uint32_t a, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(0u), "r"(c));
  return r;
}

// 32 bytes of one thread, one sector
__device__ __forceinline__ void store32(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               :
               : "l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// WIN: what is not finite in V, of keys j0 .. j1 - 1 that row t sees, into n
// dimensions of its result (row; v: the same dimensions of key 0), added to what
// the products left.  Keys that the products had are added twice, which changes nothing.
__device__ __noinline__ void put_back(const __nv_bfloat16* v, size_t stride, int window, int sinks, int j0, int j1, int t,
                                      uint16_t* row, int n) {
  for (int j = j0; j < j1 && j <= t; ++j) {
    if (j <= t - window && j >= sinks) continue;
    const uint4* x = reinterpret_cast<const uint4*>(v + (size_t)j * stride);
    for (int c = 0; c < n; c += 8) {
      const uint4 y = __ldg(x + c / 8);
      const uint32_t q[4] = {y.x, y.y, y.z, y.w};
      for (int u = 0; u < 8; ++u) {
        const uint32_t b = q[u >> 1] >> (16 * (u & 1)) & 0xffffu;
        if ((b & 0x7f80u) != 0x7f80u) continue;
        const float was = __uint_as_float((uint32_t)*reinterpret_cast<volatile uint16_t*>(row + c + u) << 16);
        const float sum = was + __uint_as_float(b << 16);
        row[c + u] = sum != sum ? 0x7fc0 : (uint16_t)(__float_as_uint(sum) >> 16);
      }
    }
  }
}

// 1-D grid: KV heads fastest, then the places ordered by the tile index inside
// their sequence, highest first (the longest rows start first, so that what is
// left at the end is short).  A CTA that has issued its work's last loads asks for
// the place of one that has not started, so that the next queries, keys and
// first products are under way while it writes its output; set-up is paid once
// an SM.
template <bool WIN>
struct PrMaps {
  CUtensorMap q, k, v;
};
template <>
struct PrMaps<true> {
  CUtensorMap q, k, v, k16, v16;   // boxes of 128 rows of K and V, and of 16
};

template <int D, bool WIN>
__global__ void __launch_bounds__(kPrThreads, 1)
    prompt_attn_kernel(const __grid_constant__ PrMaps<WIN> maps, const PrParams p) {
  using L = PrSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned long long* s_bad = reinterpret_cast<unsigned long long*>(smem + L::OFF_BAD);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);   // [2] a query tile landed
  uint64_t* q_free = q_full + 2;                                         // [2] its products are done
  uint64_t* k_full = q_free + 2;                                         // [2]
  uint64_t* k_free = k_full + 2;                                         // [2] the products with it are done
  uint64_t* v_full = k_free + 2;                                         // [2]
  uint64_t* v_free = v_full + 2;                                         // [2]
  uint64_t* s_full = v_free + 2;                                         // [2] S_s done (and every product before it)
  uint64_t* p_full = s_full + 2;                                         // [2] P_s stored, O_s rescaled (8 warps)
  uint64_t* o_fin = p_full + 2;                                          // [2] the last product into O_s done
  // a window's V looked over: two barriers in turn, since the look may be a
  // window ahead of the products (not two: V has two stages)
  uint64_t* v_ok = o_fin + 2;
  uint64_t* w_full = v_ok + 2;                                           // [2] a place written down
  uint64_t* w_free = w_full + 2;                                         // [2] every role has read it
  uint64_t* drain = w_free + 2;                                          // after a timeout: every product issued is done
  uint64_t* clc_bar = drain + 1;
  uint64_t* want = clc_bar + 1;                                          // a place's end is near
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(want + 1);
  __shared__ __align__(16) uint4 s_clc;
  __shared__ int4 s_work[2];        // row0, length, first token, KV head; length 0: no more
  __shared__ unsigned s_anybad[2];  // the place (counted from 1) whose V held something not finite
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_free[s], 1);
      mbar_init(&k_full[s], 1);
      mbar_init(&k_free[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_free[s], 2);   // the products and the look
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], kPrSoftWarps / 2);
      mbar_init(&o_fin[s], 1);
      mbar_init(&v_ok[s], 1);
      mbar_init(&w_full[s], 1);
      mbar_init(&w_free[s], kPrSoftWarps + 3);
      s_anybad[s] = 0;
    }
    mbar_init(drain, 1);
    mbar_init(clc_bar, 1);
    mbar_init(want, 1);
    fence_mbar_init();
    prefetch_tmap(&maps.q);
    prefetch_tmap(&maps.k);
    prefetch_tmap(&maps.v);
    if constexpr (WIN) {
      prefetch_tmap(&maps.k16);
      prefetch_tmap(&maps.v16);
    }
  }
  for (int e = tid; e < 2 * 3 * D; e += kPrThreads) s_bad[e] = ~0ull;
  if (warp == kWarpMma) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  const uint32_t tmem = *tmem_slot;

  // a place as every role sees it
  struct Work {
    int row0, len, t0, h;   // first row and length of the sequence, first token, KV head
    int hi, nst, nwin, skip0;
    int lo, nlow;   // WIN: first key of the windows but for the sinks; windows from it on, the others hold sinks
    int ss;         // WIN: 16-row steps of the last window that hold sinks instead, below every key that is seen
    int up, down;   // WIN: windows before up hold keys above the pair's first token, those from down on keys that the
                    // lower end hides (or, sinks behind which a step is not full, are treated as if)
  };
  auto read_work = [&](int it, bool ok) {   // again and again until free_work
    Work w;
    const int4 x = ok ? s_work[it & 1] : make_int4(0, 0, 0, 0);
    w.row0 = __shfl_sync(0xffffffffu, x.x, 0);   // uniform values, and known to be
    w.len = __shfl_sync(0xffffffffu, x.y, 0);
    w.t0 = __shfl_sync(0xffffffffu, x.z, 0);
    w.h = __shfl_sync(0xffffffffu, x.w, 0);
    w.hi = min(w.len, w.t0 + 2 * p.T);                // one past the last key
    w.nst = w.t0 + p.T < w.len ? 2 : 1;               // query tiles
    w.lo = 0;
    if constexpr (WIN) {
      const int lo = w.t0 - p.window + 1;
      if (lo > p.sinks) w.lo = lo;
    }
    w.nlow = (w.hi - w.lo + 127) / 128;
    w.nwin = w.nlow;
    w.ss = 0;
    if (WIN && w.lo > 0 && p.sinks > 0 && ((p.sinks + 15) & ~15) <= 128 * w.nlow - (w.hi - w.lo)) {
      w.ss = (p.sinks + 15) >> 4;
      w.lo = w.hi - 128 * w.nlow;   // (may lie before the sequence)
    }
    if constexpr (WIN) {
      const bool apart = w.lo > 0 && w.ss == 0;   // (sinks < lo then)
      const int hidden = w.hi - p.window - w.lo;   // below 2 T, or 2 T + 128 where the sinks share the last window
      w.up = max(1, w.nlow - ((w.t0 + 1 - w.lo) >> 7));
      w.down = hidden > 0 ? w.nlow - ((hidden + 127) >> 7) : w.nlow;
      if (apart) w.nwin += (p.sinks + 127) / 128;
      if (hidden <= 0 && (!apart || (p.sinks & 15) == 0)) w.down = w.nwin;
    }
    w.skip0 = w.nst == 2 ? w.nlow - (w.t0 + p.T - w.lo + 127) / 128 : 0;   // tile 0 sees nothing of the first window (0 or 1)
    return w;
  };
  auto wait_work = [&](int it, bool& ok) {
    if (ok && !mbar_wait(&w_full[it & 1], (uint32_t)(it >> 1) & 1u)) ok = false;
  };
  auto free_work = [&](int it) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&w_free[it & 1]);
  };
  // first key of window w, the last keys first
  auto w_start = [](const Work& k, int w) {
    if constexpr (WIN) return w < k.nlow ? k.lo + 128 * (k.nlow - 1 - w) : 128 * (k.nwin - 1 - w);
    else return 128 * (k.nwin - 1 - w);
  };
  // 16-key steps of window w that tile s sees anything of: what lies behind
  // its last token is neither multiplied nor looked at
  auto steps = [&](const Work& k, int s, int w) {
    const int end = WIN && w >= k.nlow ? p.sinks : min(k.len, k.t0 + (s + 1) * p.T);
    return min(8, (end - w_start(k, w) + 15) >> 4);
  };
  // WIN: rows [x, y) of window w that are hidden from some row of the pair by
  // the window's lower end; in a window of sinks, those behind them in a step
  auto below = [&](const Work& k, int w) {
    const int start = w_start(k, w);
    if (w >= k.nlow) return make_int2(min(128, p.sinks - start), 16 * steps(k, 0, w));
    return make_int2(k.ss > 0 ? (w == k.nlow - 1 ? p.sinks : 0) : max(0, p.sinks - start), min(128, k.hi - p.window - start));
  };
  // window w holds keys that a row may not see (so does the first, if only as a rule)
  auto scrub = [&](const Work& k, int w) {
    if constexpr (WIN) return w < k.up || w >= k.down;
    else return w == 0 || w_start(k, w) + 127 > k.t0;
  };

  if (warp >= kPrSoftWarps) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRoleRegs));
  if (warp == kWarpPlan) {
    // ---------------- places ----------------
    // c_i = ceil(len_i / 2T) tile pairs of sequence i; N(l) = sum_i max(0, c_i - l) of them have an index >= l
    int* s_cnt = reinterpret_cast<int*>(smem + L::OFF_CNT);
    int a = 0, b = 0, mine = 0;   // n <= 32: the lane's sequence
    auto count = [&](int x, int y) { return x < 0 || y < x || y > p.rows ? -1 : (y - x + 2 * p.T - 1) / (2 * p.T); };
    const bool stop = status_get(p.status) != 0;
    int top = 0, low = 0;
    for (int i = lane; i < p.n; i += 32) {
      a = __ldg(p.starts + i);
      b = __ldg(p.starts + i + 1);
      mine = count(a, b);
      if (p.n > 32) s_cnt[i] = mine;
      top = max(top, mine);
      low = min(low, mine);
    }
    __syncwarp();
    top = __reduce_max_sync(0xffffffffu, top);
    const bool bad = __any_sync(0xffffffffu, low < 0);
    if (bad && !stop && lane == 0) status_set(p.status, TV_E_SEQ);
    auto at_least = [&](int l) {   // N(l)
      int x = 0;
      if (p.n <= 32) x = max(0, mine - l);
      else
        for (int i = lane; i < p.n; i += 32) x += max(0, s_cnt[i] - l);
      return __reduce_add_sync(0xffffffffu, x);
    };
    const int all = stop || bad ? 0 : at_least(0);
    auto find = [&](int block) {   // {row0, length, first token, KV head} of a block's place, length 0: none
      const int place = block / p.Hkv;
      int found = -1, lo = 0, fa = a, fb = b;
      if (p.n == 1) {   // one sequence: its pairs from the last to the first
        lo = top - 1 - place;
        if (place < all) found = 0;
      } else if (place < all) {
        int hi = top;   // the largest l with N(l) > place; N(top) = 0
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (at_least(mid) > place) lo = mid;
          else hi = mid;
        }
        int k = place - at_least(lo + 1);   // the k-th sequence with more than lo pairs
        for (int i0 = 0; i0 < p.n; i0 += 32) {
          const int i = i0 + lane;
          const unsigned m = __ballot_sync(0xffffffffu, i < p.n && (p.n <= 32 ? mine : s_cnt[i]) > lo);
          if (k < __popc(m)) {
            const unsigned at = __ballot_sync(0xffffffffu, (m >> lane & 1u) && __popc(m & ((1u << lane) - 1u)) == k);
            found = i0 + __ffs(at) - 1;
            break;
          }
          k -= __popc(m);
        }
      }
      if (p.n <= 32) {
        fa = __shfl_sync(0xffffffffu, a, found & 31);
        fb = __shfl_sync(0xffffffffu, b, found & 31);
      } else if (found >= 0) {
        fa = __ldg(p.starts + found);
        fb = __ldg(p.starts + found + 1);
      }
      return found >= 0 ? make_int4(fa, fb - fa, lo * 2 * p.T, block % p.Hkv) : make_int4(0, 0, 0, 0);
    };
    bool ok = true;
    int block = blockIdx.x;
    for (int it = 0, asked = 0;; ) {
      const int4 x = block >= 0 ? find(block) : make_int4(0, 0, 0, 0);
      if (x.y > 0 || block < 0 || all == 0 || !p.queued) {
        if (it >= 2 && ok && !mbar_wait(&w_free[it & 1], (uint32_t)((it - 2) >> 1) & 1u)) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          s_work[it & 1] = x;
          mbar_arrive(&w_full[it & 1]);
        }
        __syncwarp();
        ++it;
        if (x.y == 0) break;
        if (!p.queued) {
          block = -1;
          continue;
        }
        // not before this place's end is near: who is done first takes the next
        ok = __all_sync(0xffffffffu, mbar_wait(want, (uint32_t)(it - 1) & 1u));
        if (!ok) break;
      }
      if (lane == 0) {
        fence_async_smem();   // the last answer was read through the generic proxy
        mbar_arrive_expect_tx(clc_bar, 16);
        clc_ask(&s_clc, clc_bar);
      }
      __syncwarp();
      ok = __all_sync(0xffffffffu, mbar_wait(clc_bar, (uint32_t)asked & 1u));
      if (!ok) break;
      block = __shfl_sync(0xffffffffu, clc_answer(&s_clc), 0);
      ++asked;
    }
    if (!ok && lane == 0) status_set(p.status, TV_E_TIMEOUT);
  } else if (warp == kWarpTma) {
    // ---------------- loads ----------------
    const uint32_t qbytes = (uint32_t)((D / 64) * p.T * p.G * 128);
    bool ok = true;
    int kv = 0, nk = 0, nv = 0, nq[2] = {0, 0};   // windows before this place; loads issued
    for (int it = 0;; ++it) {
      wait_work(it, ok);
      const Work k = read_work(it, ok);
      free_work(it);
      if (k.len == 0) break;
      auto load_kv = [&](const CUtensorMap* map, const CUtensorMap* map16, uint64_t* full, uint64_t* free, int off, int w, int& issued) {
        const int i = kv + w;
        if (i >= 2) ok = ok && mbar_wait(&free[i & 1], (uint32_t)((i - 2) >> 1) & 1u);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        if (lane == 0) mbar_arrive_expect_tx(&full[i & 1], L::TILE);
        if (WIN && k.ss > 0 && w == k.nlow - 1) {   // the sinks, and what is left of the window above them
          __syncwarp();
          const int b = lane / (D / 64), a = lane % (D / 64);
          if (b < 8)
            tma_load_3d(smem + off + (i & 1) * L::TILE + a * kAtomP + b * 2048, map16, &full[i & 1], k.h * D + a * 64, 0,
                        k.row0 + 16 * b + (b < k.ss ? 0 : w_start(k, w)));
          __syncwarp();
        } else if (lane == 0) {
#pragma unroll
          for (int a = 0; a < D / 64; ++a)
            tma_load_3d(smem + off + (i & 1) * L::TILE + a * kAtomP, map, &full[i & 1], k.h * D + a * 64, 0,
                        k.row0 + w_start(k, w));
        }
        ++issued;
      };
      const CUtensorMap *k16 = nullptr, *v16 = nullptr;
      if constexpr (WIN) k16 = &maps.k16, v16 = &maps.v16;
      auto load_q = [&](int s) {
        if (nq[s] > 0) ok = ok && mbar_wait(&q_free[s], (uint32_t)(nq[s] - 1) & 1u);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        if (lane == 0) {
          mbar_arrive_expect_tx(&q_full[s], qbytes);
#pragma unroll
          for (int a = 0; a < D / 64; ++a)
            tma_load_3d(smem + L::OFF_Q + s * L::TILE + a * kAtomP, &maps.q, &q_full[s], a * 64, k.h * p.G,
                        k.row0 + k.t0 + s * p.T);
        }
        ++nq[s];
      };
      for (int w = 0; w < k.nwin && ok; ++w) {
        // some three windows (5 us) before its end, time to find the next place
        if (w == max(0, k.nwin - 3) && lane == 0) mbar_arrive(want);
        load_kv(&maps.k, k16, k_full, k_free, L::OFF_K, w, nk);
        if (w == 0 && ok) load_q(0);
        if (ok) load_kv(&maps.v, v16, v_full, v_free, L::OFF_V, w, nv);
        if (w == 0 && ok && k.nst == 2) load_q(1);
      }
      if (!ok) break;
      kv += k.nwin;
    }
    if (!ok && lane == 0) status_set(p.status, TV_E_TIMEOUT);
    // loads in flight land before the CTA leaves
    for (int s = 0; s < 2; ++s)
      if (nq[s] > 0) mbar_wait(&q_full[s], (uint32_t)(nq[s] - 1) & 1u);
    for (int i = nk > 2 ? nk - 2 : 0; i < nk; ++i) mbar_wait(&k_full[i & 1], (uint32_t)(i >> 1) & 1u);
    for (int i = nv > 2 ? nv - 2 : 0; i < nv; ++i) mbar_wait(&v_full[i & 1], (uint32_t)(i >> 1) & 1u);
  } else if (warp == kWarpMma) {
    // ---------------- products ----------------
    const uint32_t leader = elect_one();
    const uint32_t idesc_s = idesc_bf16_f32(128, 0);                // N, the keys, comes with the window
    const uint32_t idesc_o = idesc_bf16_f32(128, D) | (1u << 16);   // B = V: MN-major
    const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(smem), 0), tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t dq = sdesc_sw128(base + L::OFF_Q, 16, 1024), dk = sdesc_sw128(base + L::OFF_K, 16, 1024);
    const uint64_t dv = sdesc_sw128(base + L::OFF_V, kAtomP, 1024);
    bool ok = true;
    // before this place: windows, windows looked over, P and query tiles
    int kv = 0, looked = 0, np[2] = {0, 0}, nq[2] = {0, 0};
    auto wait = [&](uint64_t* bar, uint32_t parity) { ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity & 1u)); };
    for (int it = 0;; ++it) {
      wait_work(it, ok);
      const Work k = read_work(it, ok);
      free_work(it);
      if (k.len == 0) break;
      // S_s = Q_s K_w^T; K_w (the CTA's i-th window) has landed
      auto product_s = [&](int s, int w, int i, bool first) {
        if (first) wait(&q_full[s], (uint32_t)nq[s]++);
        if (!ok) return;
        tc_fence_after();
        const uint64_t a = dq + (uint64_t)(s * (L::TILE >> 4)), b = dk + (uint64_t)((i & 1) * (L::TILE >> 4));
        const uint32_t idesc = idesc_s | (uint32_t)steps(k, s, w) << 18;   // N >> 3, at bit 17
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const uint64_t off = (uint64_t)(((c >> 2) * kAtomP + (c & 3) * 32) >> 4);
          umma_ss(tm + s * 128, a + off, b + off, idesc, c > 0 ? 1u : 0u, leader);
        }
        commit_by(&s_full[s], leader);
        if (s == k.nst - 1) commit_by(&k_free[i & 1], leader);
        if (w == k.nwin - 1) commit_by(&q_free[s], leader);
      };
      const int i0 = __shfl_sync(0xffffffffu, kv, 0);
      wait(&k_full[i0 & 1], (uint32_t)(i0 >> 1));
      if (!k.skip0) product_s(0, 0, i0, true);
      if (k.nst == 2) product_s(1, 0, i0, true);
      for (int w = 0; w < k.nwin && ok; ++w) {
        const int i = __shfl_sync(0xffffffffu, kv + w, 0);   // uniform, and known to be
        // both loads before the first P: nothing between a P and its products then
        wait(&v_full[i & 1], (uint32_t)(i >> 1));
        if (w + 1 < k.nwin) wait(&k_full[(i + 1) & 1], (uint32_t)((i + 1) >> 1));
        bool look = scrub(k, w);
        int seen = min(8, max(0, k.t0 + 1 - w_start(k, w)) >> 4);   // steps whose keys every row sees
        int low = 0;   // WIN: the first of them
        if (WIN && w >= k.down) {
          low = (below(k, w).y + 15) >> 4;
          if (w >= k.nlow) seen = 8;
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (s >= k.nst || !ok) break;
          const int f = s == 0 ? k.skip0 : 0;
          if (w >= f) {   // O_s += P_s V_w
            wait(&p_full[s], (uint32_t)np[s]++);
            if (!ok) break;
            tc_fence_after();
            const uint64_t b = dv + (uint64_t)((i & 1) * (L::TILE >> 4));
            auto step = [&](int c) {   // 16 keys
              umma_ts(tm + 256 + s * D, tm + s * 128 + c * 8, b + (uint64_t)(c * (2048 >> 4)), idesc_o,
                      (w > f || c > 0) ? 1u : 0u, leader);
            };
            if (!look) {
              const int n = steps(k, s, w);
              if (n == 8) {
#pragma unroll
                for (int c = 0; c < 8; ++c) step(c);
              } else {
                for (int c = 0; c < n; ++c) step(c);
              }
            } else {   // what every row sees does not wait for the look at the rest
              const int n = steps(k, s, w), m = min(n, seen);
              // (the first window's first step is the one that overwrites O_s)
              const int l = WIN && w == f && low > 0 ? m : min(m, low);
              for (int c = l; c < m; ++c) step(c);
              wait(&v_ok[looked & 1], (uint32_t)(looked >> 1));
              ++looked;
              look = false;
              if (!ok) break;
              tc_fence_after();
              if constexpr (WIN)
                for (int c = 0; c < l; ++c) step(c);
              for (int c = m; c < n; ++c) step(c);
            }
            if (w == k.nwin - 1) commit_by(&o_fin[s], leader);
            if (s == k.nst - 1) commit_by(&v_free[i & 1], leader);
          }
          if (w + 1 < k.nwin && w + 1 >= f) product_s(s, w + 1, i + 1, w + 1 == f && f > 0);
        }
      }
      if (!ok) break;
      kv += k.nwin;
    }
    if (!ok) {   // what was issued is done before TMEM is given back: a commit covers every product before it
      if (leader) status_set(p.status, TV_E_TIMEOUT);
      commit_by(drain, leader);
      mbar_wait(drain, 0);
    }
  } else if (warp == kWarpLook) {
    // ---------------- V rows that a row may not see ----------------
    bool ok = true;
    int kv = 0, looked = 0;   // windows, windows looked over before this place
    for (int it = 0;; ++it) {
      wait_work(it, ok);
      const Work k = read_work(it, ok);
      free_work(it);
      if (k.len == 0) break;
      // An entry of `bad` is the place's complement and the key, so that the
      // smallest is the latest place's first key; what two places before left
      // behind is larger.
      unsigned long long* bad = s_bad + (it & 1) * 3 * D;
      const unsigned tag = (unsigned)it + 1u;
      for (int w = 0; w < k.nwin; ++w) {
        const int i = kv + w;
        ok = __all_sync(0xffffffffu, mbar_wait(&v_full[i & 1], (uint32_t)(i >> 1) & 1u));
        if (!ok) break;
        if (!scrub(k, w)) {   // nothing to look at; the stage is not filled again before this, so that no phase is missed
          if (lane == 0) mbar_arrive(&v_free[i & 1]);
          continue;
        }
        uint8_t* sv = smem + L::OFF_V + (i & 1) * L::TILE;
        // rows of this pair's tokens but the first are looked at, those behind
        // its last token in the same step emptied
        const int key0 = w_start(k, w);
        int first = max(0, k.t0 + 1 - key0), last = min(128, k.hi - key0);
        int empty = last, end = (last + 15) & ~15;
        int below0 = 0, below1 = 0;   // WIN: a second range of them
        if (WIN && w >= k.down) {   // and the rows that the lower end hides
          const int2 b = below(k, w);
          if (w >= k.nlow) {   // the sinks are seen, what is behind them in their last step is not
            first = last = empty = b.x;
            end = b.y;
          } else if (b.x < b.y) {
            if (first >= last) first = b.x, last = b.y;
            else if (first <= b.y) first = min(first, b.x);
            else below0 = b.x, below1 = b.y;   // what lies between is not touched: its steps do not wait for this look
          }
        }
        constexpr int CH = D / 8;   // 16-byte pieces of a row, 32 / CH rows a step
        bool wrote = empty < end;
        const int c = lane % CH;
        uint8_t* piece = sv + (c >> 3) * kAtomP;
        for (int row = empty + lane / CH; row < end; row += 32 / CH)
          *reinterpret_cast<uint4*>(piece + swz(row, c & 7)) = make_uint4(0u, 0u, 0u, 0u);
        // eight rows a round: their swizzles repeat, so that a round's addresses are the last's and 1024
        constexpr int PER = CH / 4, BATCH = 2 * PER;
#pragma unroll 1
        for (;;) {
          const uint8_t* at[PER];
#pragma unroll
          for (int u = 0; u < PER; ++u) at[u] = piece + swz(first + lane / CH + u * (32 / CH), c & 7);
          for (int r0 = first + lane / CH; r0 < last; r0 += 16) {
            uint4 y[BATCH];
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
              const int row = r0 + u * (32 / CH);
              y[u] = row < last ? *reinterpret_cast<const uint4*>(at[u % PER] + (u / PER) * 1024) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int u = 0; u < PER; ++u) at[u] += 2048;
            // 0 x, summed: NaN where an x is not finite
            uint32_t any[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
              any[0] = times_zero(y[u].x, any[0]);
              any[1] = times_zero(y[u].y, any[1]);
              any[2] = times_zero(y[u].z, any[2]);
              any[3] = times_zero(y[u].w, any[3]);
            }
            if (((any[0] | any[1]) | (any[2] | any[3])) & 0x7fff7fffu) {
#pragma unroll 1
              for (int row = r0; row < last && row < r0 + 16; row += 32 / CH) {
                uint16_t* x = reinterpret_cast<uint16_t*>(piece + swz(row, c & 7));
#pragma unroll 1
                for (int u = 0; u < 8; ++u) {
                  const uint32_t b = x[u];
                  if ((b & 0x7f80u) == 0x7f80u) {
                    const int kind = (b & 0x7fu) ? 0 : (b & 0x8000u ? 2 : 1);   // NaN, +inf, -inf
                    if (!WIN) atomicMin(&bad[kind * D + c * 8 + u], (unsigned long long)~tag << 32 | (unsigned)(key0 + row));
                    x[u] = 0;
                  }
                }
              }
              *reinterpret_cast<volatile unsigned*>(&s_anybad[it & 1]) = tag;
              wrote = true;
            }
          }
          if (!WIN || below0 >= below1) break;
          first = below0, last = below1, below1 = 0;
        }
        if (wrote) fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&v_ok[looked & 1]);
          mbar_arrive(&v_free[i & 1]);
        }
        ++looked;
      }
      if (!ok) break;
      kv += k.nwin;
    }
    if (!ok && lane == 0) status_set(p.status, TV_E_TIMEOUT);
  }
  } else {
    // ---------------- softmax: warps 8 s .. 8 s + 7 hold tile s, thread pairs a row ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int s = warp >> 3, hf = (warp >> 2) & 1, r = (warp & 3) * 32 + lane;   // tile, half of the keys, row
    const uint32_t lb = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t sS = tmem + s * 128 + lb, sO = tmem + 256 + s * D + hf * (D / 2) + lb;
    float* s_top = reinterpret_cast<float*>(smem + L::OFF_TOP) + s * 256;
    float* s_sum = reinterpret_cast<float*>(smem + L::OFF_SUM) + s * 256;
    const int pair = 1 + s * 4 + (warp & 3);   // named barrier of the two warps that share rows
    const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2);
    const int rt = r / p.G;                    // token of the row in its tile
    // the row's place in the output, from the tile pair's and group's first
    const int ot = (s * p.T + rt) * p.Hq + r % p.G;
    bool ok = true;
    int ns = 0, nf = 0;                        // score tiles, finished outputs before this place

    for (int it = 0;; ++it) {
      wait_work(it, ok);
      const Work k = read_work(it, ok);
      if (pair_any(k.len == 0, pair)) break;   // the two warps of a pair leave together, whatever happened
      const bool active = s < k.nst;
      const int f = s == 0 ? k.skip0 : 0;
      const int tmin = k.t0 + s * p.T, t = tmin + rt;
      // rows of the tile behind the last vector or token hold anything: an
      // infinite offset keeps them out of every decision
      const bool live = r < p.T * p.G && t < k.len;
      float m = live ? kFirst : INFINITY, l = 0.f;   // offset of the row; sum over this thread's keys

      // One window.  The exponentials are taken at the offset that the row has,
      // kFirst to begin with: what matters is that the offset lies within some
      // 80 powers of two of the scores, since P and the sums are floating-point
      // numbers.  A sum over this thread's 64 keys says whether it does: above
      // kHigh some score lies too far above it, and below kLow, where the row
      // sees its first keys, all of them lie too far below.  Then (hardly ever)
      // both threads of the row find its maximum, the offset goes kAbove beyond
      // it, and the exponentials are taken again, once: their sum is below kHigh
      // then, but for scores beyond some 2^16, whose maximum (as the offset) is
      // known only to half its last place: 2^3 at the end of what the call
      // allows, so that a sum stays below 2^26.  P stays in registers until both warps have read their scores,
      // because it goes where the scores are.
      // lim: the last visible one of this thread's keys; before: the first key
      // of the window before (rows before it have seen none); again: O_s holds
      // earlier windows.  WIN: of them, those above low or below sink are visible.
      // Two copies of the code: PLAIN for windows that hide nothing of rows that
      // have keys already, one for all the others (a place of one or two
      // windows spends as long fetching instructions as on them: with a third
      // for masked windows the packed prompts took 66 us instead of 64).
      auto window = [&](auto plain_c, bool masked, int lim, int before, bool again, int low, int sink) {
        constexpr bool PLAIN = decltype(plain_c)::value;
        if (ok && !mbar_wait(&s_full[s], (uint32_t)ns & 1u)) ok = false;
        ++ns;
        tc_fence_after();
        // Of a masked window's pieces of 32 keys, those that every row of the
        // warp sees need no mask, and those that none sees are not read.
        int all_see = 63, any_see = 63;
        if (!WIN && !PLAIN && masked) {
          all_see = __reduce_min_sync(0xffffffffu, live ? lim : 63);
          any_see = __reduce_max_sync(0xffffffffu, live ? lim : -1);
        }
        // WIN: a bit for each of a piece's keys that the row sees (bits 0 .. n of a word: upto(n))
        uint32_t sees[2] = {~0u, ~0u};
        if (WIN && !PLAIN && masked) {
          auto upto = [](int n) {
            uint32_t r;   // (a shift by 32 or more leaves nothing)
            asm("shl.b32 %0, %1, %2;" : "=r"(r) : "r"(~0u), "r"(max(n + 1, 0)));
            return ~r;
          };
#pragma unroll
          for (int c = 0; c < 2; ++c)
            sees[c] = upto(lim - 32 * c) & (~upto(low - 32 * c) | upto(sink - 1 - 32 * c));
        }
        auto unseen = [&](int c) {   // by every row of the warp
          if constexpr (WIN) return masked && !__any_sync(0xffffffffu, live && sees[c] != 0u);
          else return 32 * c > any_see;
        };
        auto scores = [&](int c, uint32_t (&x)[32]) {   // half of its scores
          ld32(sS + 64 * hf + 32 * c, x);
          tmem_ld_wait();
          if (WIN && !PLAIN) {
            const uint32_t see = c == 0 ? sees[0] : sees[1];
            if (masked && !__all_sync(0xffffffffu, !live || see == ~0u)) {
#pragma unroll
              for (int u = 0; u < 32; ++u)
                if (!(see >> u & 1u)) x[u] = 0xff800000u;
            }
          } else if (!PLAIN && 32 * c + 31 > all_see) {
#pragma unroll
            for (int u = 0; u < 32; ++u)
              if (32 * c + u > lim) x[u] = 0xff800000u;
          }
        };
        uint32_t pk[32];
        float sum;
        for (bool first = true;; first = false) {
          const uint64_t neg2 = pack2(-m, -m);
          float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (!PLAIN && unseen(c)) {
#pragma unroll
              for (int u = 0; u < 16; ++u) pk[16 * c + u] = 0u;
              continue;
            }
            uint32_t x[32];
            scores(c, x);
#pragma unroll
            for (int u = 0; u < 16; ++u) {
              float a, b;
              unpack2(fma2(pack2(__uint_as_float(x[2 * u]), __uint_as_float(x[2 * u + 1])), scale2, neg2), a, b);
              const __nv_bfloat162 v = __floats2bfloat162_rn(ex2p(a), ex2p(b));
              const uint32_t q = *reinterpret_cast<const uint32_t*>(&v);
              pk[16 * c + u] = q;
              add_bf16(part[2 * (u & 1)], (uint16_t)q);
              add_bf16(part[2 * (u & 1) + 1], (uint16_t)(q >> 16));
            }
          }
          sum = (part[0] + part[1]) + (part[2] + part[3]);
          const bool fresh = !PLAIN && before > t;   // the row's first keys, if it sees any
          const bool has = WIN ? (sees[0] | sees[1]) != 0u : lim >= 0;   // it sees some of them
          const bool off = sum > kHigh || (first && fresh && live && has && sum < kLow);
          tc_fence_before();
          const bool any = pair_any(off, pair);
          tc_fence_after();
          if (!any || !first) break;
          float y = -INFINITY, z = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t x[32];
            scores(c, x);
#pragma unroll
            for (int u = 0; u < 32; u += 4) {
              y = max3(y, __uint_as_float(x[u]), __uint_as_float(x[u + 1]));
              z = max3(z, __uint_as_float(x[u + 2]), __uint_as_float(x[u + 3]));
            }
          }
          y = fmaxf(y, z);
          s_top[hf * 128 + r] = y;
          pair_sync(pair);
          y = fmaxf(y, s_top[(hf ^ 1) * 128 + r]) * p.scale_log2;   // the row's maximum
          // above: 64 keys below m + 2 do not add up to more than kHigh
          const bool move = live && (y > m + 2.f || (fresh && y < m - kAbove && y > -INFINITY));
          const float next = y + kAbove;
          const float scale = move && !fresh ? ex2p(m - next) : 1.f;   // a row without keys has nothing to rescale
          if (move) m = next;
          l *= scale;
          if (again) {
#pragma unroll 1
            for (int c = 0; c < D / 2; c += 16) {
              uint32_t o[16];
              ld16(sO + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * scale);
              st16(sO + c, o);
            }
          }
        }
        l += sum;
        st32(sS + 32 * hf, pk);
        st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[s]);
      };

      if (active) {
        // the windows that hide something, or are the first
        int w = f;
        if constexpr (WIN) {
          const int last = min(k.len, tmin + p.T) - 1;   // the tile's last token
#pragma unroll 1
          for (; w < k.nwin; ++w) {
            const int start = w_start(k, w);
            const bool sinks = w >= k.nlow;
            const int before = w == f ? 0x7fffffff : (sinks ? 0 : start + 128);
            const bool masked = sinks ? p.sinks - start < 128
                                      : start + 127 > tmin || (start <= last - p.window && (k.ss > 0 || start + 127 >= p.sinks));
            const int at = start + 64 * hf;
            if (!masked && before <= tmin) window(std::true_type{}, false, 63, 0, true, -1, 0);
            else   // (one copy of the code for both)
              window(std::false_type{}, masked, sinks ? p.sinks - 1 - at : (masked ? t - at : 63), before, w > f,
                     masked && !sinks ? t - p.window - at : -1,
                     k.ss > 0 ? (w == k.nlow - 1 ? p.sinks - 64 * hf : 0) : p.sinks - at);
          }
        } else {
          for (; w < k.nwin; ++w) {
            const int start = w_start(k, w);
            const bool masked = start + 127 > tmin;
            // rows without a key: all in the first window, and those before a window that hid it all
            const int before = w == f ? 0x7fffffff : start + 128;
            if (w > f && !masked && before <= tmin) break;
            window(std::false_type{}, masked, masked ? t - start - 64 * hf : 63, before, w > f, -1, 0);
          }
          // and all the others
          for (; w < k.nwin; ++w) window(std::true_type{}, false, 63, 0, true, -1, 0);
        }
        if (ok && !mbar_wait(&o_fin[s], (uint32_t)nf & 1u)) ok = false;
        ++nf;
        s_sum[hf * 128 + r] = l;
        pair_sync(pair);
        const float inv = 1.f / (s_sum[r] + s_sum[128 + r]);
        tc_fence_after();
        const Work k = read_work(it, true);   // read once more: not held through the windows
        const int t = k.t0 + s * p.T + rt;
        const bool live = r < p.T * p.G && t < k.len;
        const unsigned tag = (unsigned)it + 1u;
        // Two lanes store 64 bytes of one row, then of the other's: a store
        // instruction takes the memory pipe a cycle for every 128-byte line that
        // it touches.
        const bool odd = lane & 1;
        const int mate = __shfl_xor_sync(0xffffffffu, ot, 1);
        const unsigned keep = __ballot_sync(0xffffffffu, ok && live);
        __nv_bfloat16* dst = p.out + ((size_t)(k.row0 + k.t0) * p.Hq + k.h * p.G) * D + hf * (D / 2) + (odd ? 16 : 0);
        __nv_bfloat16 *dst0 = dst + (size_t)(odd ? mate : ot) * D, *dst1 = dst + (size_t)(odd ? ot : mate) * D;
        const bool keep0 = keep >> (lane & 30) & 1u, keep1 = keep >> (lane | 1) & 1u;
#pragma unroll 1
        for (int c = 0; c < D / 2; c += 32) {
          uint32_t o[32];
          ld32(sO + c, o);
          tmem_ld_wait();
          uint32_t b0[8], b1[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const __nv_bfloat162 v =
                __floats2bfloat162_rn(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
            const __nv_bfloat162 w =
                __floats2bfloat162_rn(__uint_as_float(o[16 + 2 * e]) * inv, __uint_as_float(o[17 + 2 * e]) * inv);
            const uint32_t x = *reinterpret_cast<const uint32_t*>(&v), y = *reinterpret_cast<const uint32_t*>(&w);
            const uint32_t z = __shfl_xor_sync(0xffffffffu, odd ? x : y, 1);
            b0[e] = odd ? z : x;
            b1[e] = odd ? y : z;
          }
          if (keep0) store32(dst0 + c, b0);
          if (keep1) store32(dst1 + c, b1);
        }
        if (*reinterpret_cast<volatile unsigned*>(&s_anybad[it & 1]) == tag) {   // what of V is not finite
          const unsigned long long* first = s_bad + (it & 1) * 3 * D + hf * (D / 2);
          uint16_t* row = reinterpret_cast<uint16_t*>(dst - (odd ? 16 : 0)) + (size_t)ot * D;
          if constexpr (WIN) {
            __syncwarp();   // over what the other lane has stored
            const __nv_bfloat16* v = p.v + (size_t)k.row0 * p.kv_stride + (size_t)k.h * D + hf * (D / 2);
            if (ok && live)
              for (int w = 0; w < k.nlow; ++w)
                if (scrub(k, w)) put_back(v, p.kv_stride, p.window, p.sinks, max(0, w_start(k, w)), w_start(k, w) + 128, t, row, D / 2);
          } else {
          auto sees = [&](unsigned long long x) { return (unsigned)(x >> 32) == ~tag && (int)(unsigned)x <= t; };
          __syncwarp();   // over what the other lane has stored
          // Added to what the products left, which may be NaN or infinite
          // itself: by a key before the pair's own, by the row's scores.
#pragma unroll 1
          for (int c = 0; c < D / 2; ++c) {
            const bool n = sees(first[c]), pi = sees(first[D + c]), ni = sees(first[2 * D + c]);
            if ((n || pi || ni) && ok && live) {
              float x = __uint_as_float((uint32_t)*reinterpret_cast<volatile uint16_t*>(row + c) << 16);
              if (pi) x += INFINITY;
              if (ni) x -= INFINITY;
              row[c] = n || x != x ? 0x7fc0 : (uint16_t)(__float_as_uint(x) >> 16);
            }
          }
          }
        }
        tc_fence_before();   // the next place's products into O_s follow this warp's next arrival
      }
      free_work(it);
    }
    if (!ok && lane == 0) status_set(p.status, TV_E_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool WIN>
int launch_prompt(PrParams& p, const void* q, const void* k, const void* v, size_t q_stride, size_t kv_stride,
                  cudaStream_t st) {
  PrMaps<WIN> m;
  int rc = make_tmap_bf16_rows(&m.q, q, D, p.Hq, p.rows, q_stride, 64, p.G, p.T);
  if (rc || (rc = make_tmap_bf16_rows(&m.k, k, p.Hkv * D, 1, p.rows, kv_stride, 64, 1, 128)) ||
      (rc = make_tmap_bf16_rows(&m.v, v, p.Hkv * D, 1, p.rows, kv_stride, 64, 1, 128)))
    return rc;
  if constexpr (WIN)
    if ((rc = make_tmap_bf16_rows(&m.k16, k, p.Hkv * D, 1, p.rows, kv_stride, 64, 1, 16)) ||
        (rc = make_tmap_bf16_rows(&m.v16, v, p.Hkv * D, 1, p.rows, kv_stride, 64, 1, 16)))
      return rc;
  static std::atomic<bool> attr[64];
  if (ensure_smem_limit(prompt_attn_kernel<D, WIN>, PrSmem<D>::BYTES, attr)) return TV_E_CUDA;
  // the roles' register split must not ask for more than the launch brings
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, prompt_attn_kernel<D, WIN>) != cudaSuccess) return TV_E_CUDA;
    regs.store(fa.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) * kPrThreads < kPrSoftThreads * kSoftRegs + 128 * kRoleRegs)
    return TV_E_UNSUPPORTED;
  // at most rows / 2T whole pairs and one ragged pair a sequence
  const long long pairs = (long long)p.rows / (2 * p.T) + (p.n < p.rows ? p.n : p.rows);
  const int sms = num_sms();
  if (sms <= 0) return TV_E_CUDA;
  p.queued = pairs * p.Hkv > sms;
  return launch_pdl(prompt_attn_kernel<D, WIN>, dim3((unsigned)(pairs * p.Hkv)), dim3(kPrThreads), PrSmem<D>::BYTES, st, m,
                    p);
}

int attend_prompt(bool win, int n_q_heads, int n_kv_heads, int head_dim, int window, int sinks, const tv_bf16* q,
                  const tv_bf16* k, const tv_bf16* v, size_t q_stride, size_t kv_stride, const int32_t* starts,
                  int n_seqs, int rows, tv_bf16* out, int32_t* dev_status, void* stream) {
  if (n_q_heads < 1 || n_kv_heads < 1 || !q || !k || !v || !starts || !out || !dev_status || rows < 1) return TV_E_ARG;
  if (window < 1 || sinks < 0) return TV_E_ARG;
  int rc = check_listed(n_seqs);
  if (rc) return rc;
  if (head_dim != 64 && head_dim != 128) return TV_E_UNSUPPORTED;
  if (n_q_heads % n_kv_heads != 0 || n_q_heads / n_kv_heads > 128 || n_q_heads > 65536) return TV_E_UNSUPPORTED;
  const size_t D = head_dim;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || (reinterpret_cast<uintptr_t>(out) & 31u) != 0) return TV_E_ARG;
  if (q_stride % 8 != 0 || kv_stride % 8 != 0) return TV_E_ARG;
  if (q_stride < n_q_heads * D || kv_stride < n_kv_heads * D) return TV_E_ARG;
  PrParams p;
  p.starts = starts;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.status = dev_status;
  p.n = n_seqs;
  p.rows = rows;
  p.Hq = n_q_heads;
  p.Hkv = n_kv_heads;
  p.G = n_q_heads / n_kv_heads;
  p.T = 128 / p.G;
  p.window = window < rows ? window : rows;   // no length is above rows, and differences of the two stay in range
  p.sinks = sinks < rows ? sinks : rows;
  p.v = reinterpret_cast<const __nv_bfloat16*>(v);
  p.kv_stride = kv_stride;
  p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)head_dim));
  if (((long long)rows / (2 * p.T) + n_seqs) * n_kv_heads > 0x7fffffffll) return TV_E_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (win)
    return head_dim == 128 ? launch_prompt<128, true>(p, q, k, v, q_stride, kv_stride, st)
                           : launch_prompt<64, true>(p, q, k, v, q_stride, kv_stride, st);
  return head_dim == 128 ? launch_prompt<128, false>(p, q, k, v, q_stride, kv_stride, st)
                         : launch_prompt<64, false>(p, q, k, v, q_stride, kv_stride, st);
}

}  // namespace
}  // namespace tv

using namespace tv;

extern "C" {

int tv_attend_prompt(int n_q_heads, int n_kv_heads, int head_dim, const tv_bf16* q, const tv_bf16* k, const tv_bf16* v,
                     size_t q_stride, size_t kv_stride, const int32_t* starts, int n_seqs, int rows, tv_bf16* out,
                     int32_t* dev_status, void* stream) {
  return attend_prompt(false, n_q_heads, n_kv_heads, head_dim, 0x7fffffff, 0, q, k, v, q_stride, kv_stride, starts, n_seqs,
                       rows, out, dev_status, stream);
}

int tv_attend_prompt_window(int n_q_heads, int n_kv_heads, int head_dim, int window, int sinks, const tv_bf16* q,
                            const tv_bf16* k, const tv_bf16* v, size_t q_stride, size_t kv_stride,
                            const int32_t* starts, int n_seqs, int rows, tv_bf16* out, int32_t* dev_status,
                            void* stream) {
  return attend_prompt(true, n_q_heads, n_kv_heads, head_dim, window, sinks, q, k, v, q_stride, kv_stride, starts, n_seqs,
                       rows, out, dev_status, stream);
}

}  // extern "C"
