// Rows into the pages of a cache in 4 bits, and out of them; the layout and the
// rounding are those of tv_pool4 in tv.h.
//
// What bounds it: a value is 2 bytes on one side and 9/16 on the other, and
// little is computed, so both kernels are streams over memory.  A warp takes a
// pair of tokens (their V share words) and 2 U 16-byte pieces a lane, K and V
// of U heads of 128 or 2 U of 64.  What V's 16-byte pieces, 64 bytes apart, take
// besides: 32-byte sectors between SM and L2 are 1.5 times the pool's bytes in, 1.7
// out (10610 rows; 27.0 us both ways, 60 % of the copy rate).
#include "tv_kernels.cuh"
#include "tv_pages.cuh"
#include "tv_pages4.cuh"

namespace tv {
namespace {

constexpr int kBlocksPerSm = 3;    // of up to 85 registers a thread (10610 rows in and out, in turn: 26.3 us; of 64, four: 27.2)
constexpr int kMany = 4;           // U where there are rows enough for every warp

// One task: R packed rows (writing, U = 1: one row, else two) and U pieces of
// heads, of K and of V.  Lanes 0 .. 15 have the first row of a pair, 16 .. 31 the
// second; of 16 lanes each has 8 values of a head, of one head of 128 or two of 64.
//
// A warp keeps its heads and goes from rows to rows (Walk); where the next ones
// lie is looked up while these ones' values are on their way.
struct Walk {
  uint32_t group, slot, slot0, groups, slots, step_group, step_slot;
  __device__ __forceinline__ Walk(uint32_t all_groups, uint32_t all_slots) : groups(all_groups), slots(all_slots) {
    const uint32_t warps = gridDim.x * (kListThreads / 32), w = blockIdx.x * (kListThreads / 32) + (threadIdx.x >> 5);
    step_group = min(groups, warps);
    step_slot = warps / step_group;
    group = w % step_group;
    slot = slot0 = w / step_group;
    if (slot0 >= step_slot) group = groups;   // more warps than whole sets of them
    else if (slot >= slots) next();
  }
  __device__ __forceinline__ bool more() const { return group < groups; }
  __device__ __forceinline__ void next() {
    slot += step_slot;
    if (slot >= slots) group = slot0 < slots ? group + step_group : groups, slot = slot0;
  }
};

// Writing, a pair is tokens 2 m and 2 m + 1 of one sequence where both are
// listed, so that the words of V (two tokens) and the scales are written whole.
// A row is the first of its pair, or alone, if its token is even or it is its
// sequence's first; what is neither belongs to the row before it, which may be
// the previous task's.
template <int D, int U>
__global__ void __launch_bounds__(kListThreads, kBlocksPerSm)
    rows4_write_kernel(tv_pool pool, int layer, tv_seqs t, RowList list, const __nv_bfloat16* k, const __nv_bfloat16* v,
                       size_t row_stride, size_t head_stride, int32_t* status) {
  using B = Block4<D>;
  __shared__ int s_start[kMaxListed + 1];
  __shared__ uint32_t s_bad;
  extern __shared__ uint32_t s_mark[];   // a bit per table row
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, ps = pool.page_size, Hkv = pool.n_kv_heads;
  if (block_skip(status)) return;
  if (!look_over<true>(t, ps, list, s_start, s_mark, &s_bad, status)) return;
  const uint32_t first = s_start[0], total = s_start[list.n];
  constexpr int LH = D / 8;                         // lanes of a head
  constexpr int kHeads = U * (16 / LH);       // heads of a task
  const uint32_t groups = (Hkv + kHeads - 1) / kHeads;
  constexpr uint32_t R = U == 1 ? 1 : 2;
  uint8_t *pk = reinterpret_cast<uint8_t*>(pool.k), *pv = reinterpret_cast<uint8_t*>(pool.v);
  const int odd = lane >> 4, c = lane % LH, sub = (lane & 15) / LH;
  Walk w(groups, total > first ? (total - first + R - 1) / R : 0u);
  uint32_t nth = 0;          // the task's row
  struct Row {
    uint32_t r;
    int h0, at, p;           // first head, token, page
    bool any, first, two;    // there is a row; first of its pair; the second is listed, too
  };
  auto look = [&](Row& x) {
    x.any = w.more();
    x.first = x.two = false;
    if (!x.any) return;
    x.r = first + R * w.slot + nth;
    x.h0 = (int)w.group * kHeads;
    if (x.r < total) {
      const int i = sequence_of(s_start, list.n, x.r);
      const uint32_t s0 = s_start[i], s1 = s_start[i + 1];
      x.at = __ldg(list.pos + i) + (int)(x.r - s0);
      x.first = !(x.at & 1) || x.r == s0;            // else it is the second of the pair before it
      x.two = !(x.at & 1) && x.r + 1 < s1;
      if (x.first) x.p = __ldcg(t.pages + (size_t)__ldg(list.ids + i) * t.max_pages + x.at / ps);   // (a pair lies in one page)
    }
    if (++nth == R || x.two) nth = 0, w.next();
  };
  Row next;
  look(next);
#pragma unroll 1
  while (next.any) {
    const Row cur = next;
    {
      const int h0 = cur.h0, at = cur.at, p = cur.p;
      const uint32_t r = cur.r;
      const bool two = cur.two;
      if (!cur.first || p < 0 || p >= pool.n_pages) {
        if (cur.first && gridDim.x == 1 && lane == 0) status_set(status, TV_E_PAGE);
        look(next);
        continue;
      }
      const bool mine = two || !odd;                 // a row alone: the upper lanes have none
      const int tok = (at & 15) + (two ? odd : 0);
      const size_t block = ((((size_t)layer * pool.n_pages + p) * Hkv) * ps + at % ps / 16 * 16) / 16 * B::BYTES;
      const size_t per_head = (size_t)(ps / 16) * B::BYTES;
      uint4 x[2 * U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * (16 / LH) + sub;
        const size_t e = (size_t)(r + (two ? odd : 0)) * row_stride + (size_t)h * head_stride + c * 8;
        const bool in = mine && h < Hkv;
        x[2 * u] = in ? __ldcs(reinterpret_cast<const uint4*>(k + e)) : make_uint4(0u, 0u, 0u, 0u);
        x[2 * u + 1] = in ? __ldcs(reinterpret_cast<const uint4*>(v + e)) : make_uint4(0u, 0u, 0u, 0u);
      }
      look(next);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * (16 / LH) + sub;
        if (h0 + u * (16 / LH) >= Hkv) break;        // (the same on all lanes)
        uint32_t sk, sv;                             // scales, bf16
        const uint32_t wk = round4(x[2 * u], sk), wv = round4(x[2 * u + 1], sv);
        const uint32_t ov = __shfl_xor_sync(0xffffffffu, wv, 16);
        const uint32_t os_k = __shfl_xor_sync(0xffffffffu, sk, 16), os_v = __shfl_xor_sync(0xffffffffu, sv, 16);
        if (!mine || h >= Hkv) continue;
        uint8_t *bk = pk + block + (size_t)h * per_head, *bv = pv + block + (size_t)h * per_head;
        *reinterpret_cast<uint32_t*>(bk + B::k_word(tok, c)) = wk;
        if (two) {
          // each lane one word of both tokens: dimensions 8 c .. + 3 the lower, 8 c + 4 .. + 7 the upper
          const uint32_t w = odd ? (ov >> 16) | (wv & 0xffff0000u) : (wv & 0xffffu) | (ov << 16);
          *reinterpret_cast<uint32_t*>(bv + B::v_word(tok, 2 * c + odd)) = w;
          if (c % 4 == 0) {
            if (odd) *reinterpret_cast<uint32_t*>(bv + B::scale(tok, c / 4)) = os_v | sv << 16;
            else *reinterpret_cast<uint32_t*>(bk + B::scale(tok, c / 4)) = sk | os_k << 16;
          }
        } else {
          const int o = tok % 2 * 2;
          *reinterpret_cast<uint16_t*>(bv + B::v_word(tok, 2 * c) + o) = (uint16_t)wv;
          *reinterpret_cast<uint16_t*>(bv + B::v_word(tok, 2 * c + 1) + o) = (uint16_t)(wv >> 16);
          if (c % 4 == 0) {
            *reinterpret_cast<uint16_t*>(bk + B::scale(tok, c / 4) + o) = (uint16_t)sk;
            *reinterpret_cast<uint16_t*>(bv + B::scale(tok, c / 4) + o) = (uint16_t)sv;
          }
        }
      }
    }
  }
}

// Reading, each half warp has its own row; a V word of two tokens reaches both
// lanes that want it in one load.
template <int D, int U>
__global__ void __launch_bounds__(kListThreads, kBlocksPerSm)
    rows4_read_kernel(tv_pool pool, int layer, tv_seqs t, RowList list, __nv_bfloat16* k, __nv_bfloat16* v,
                      size_t row_stride, size_t head_stride, int32_t* status) {
  using B = Block4<D>;
  __shared__ int s_start[kMaxListed + 1];
  __shared__ uint32_t s_bad;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, ps = pool.page_size, Hkv = pool.n_kv_heads;
  if (block_skip(status)) return;
  if (!look_over<false>(t, ps, list, s_start, nullptr, &s_bad, status)) return;
  const uint32_t first = s_start[0], total = s_start[list.n];
  constexpr int LH = D / 8;
  constexpr int kHeads = U * (16 / LH);
  const uint32_t groups = (Hkv + kHeads - 1) / kHeads;
  const uint8_t *pk = reinterpret_cast<const uint8_t*>(pool.k), *pv = reinterpret_cast<const uint8_t*>(pool.v);
  const int odd = lane >> 4, c = lane % LH, sub = (lane & 15) / LH;
  Walk w(groups, total > first ? (total - first + 1) / 2 : 0u);
  struct Row {
    uint32_t r;
    int h0, at, p;   // first head, token, page (-1: none)
    bool any;
  };
  auto look = [&](Row& x) {
    x.any = w.more();
    x.p = -1;
    if (!x.any) return;
    x.r = first + 2 * w.slot + odd;
    x.h0 = (int)w.group * kHeads;
    if (x.r < total) {
      const int i = sequence_of(s_start, list.n, x.r);
      x.at = __ldg(list.pos + i) + (int)(x.r - (uint32_t)s_start[i]);
      x.p = __ldcg(t.pages + (size_t)__ldg(list.ids + i) * t.max_pages + x.at / ps);
      if (x.p < 0 || x.p >= pool.n_pages) {
        if (gridDim.x == 1) status_set(status, TV_E_PAGE);
        x.p = -1;
      }
    }
    w.next();
  };
  Row next;
  look(next);
#pragma unroll 1
  while (next.any) {
    const int h0 = next.h0, at = next.at, p = next.p;
    const uint32_t r = next.r;
    const int tok = at & 15;
    const size_t block = ((((size_t)layer * pool.n_pages + p) * Hkv) * ps + at % ps / 16 * 16) / 16 * B::BYTES;
    const size_t per_head = (size_t)(ps / 16) * B::BYTES;
    uint32_t wk[U], va[U], vb[U], sk[U], sv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * (16 / LH) + sub;
      if (p >= 0 && h < Hkv) {
        const uint8_t *bk = pk + block + (size_t)h * per_head, *bv = pv + block + (size_t)h * per_head;
        wk[u] = __ldcg(reinterpret_cast<const uint32_t*>(bk + B::k_word(tok, c)));
        va[u] = __ldcg(reinterpret_cast<const uint32_t*>(bv + B::v_word(tok, 2 * c)));
        vb[u] = __ldcg(reinterpret_cast<const uint32_t*>(bv + B::v_word(tok, 2 * c + 1)));
        sk[u] = __ldcg(reinterpret_cast<const uint32_t*>(bk + B::scale(tok, c / 4)));
        sv[u] = __ldcg(reinterpret_cast<const uint32_t*>(bv + B::scale(tok, c / 4)));
      }
    }
    look(next);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * (16 / LH) + sub;
      if (p >= 0 && h < Hkv) {
        const size_t e = (size_t)r * row_stride + (size_t)h * head_stride + c * 8;
        const bool hi = tok & 1;
        const uint32_t wv = hi ? (va[u] >> 16) | (vb[u] & 0xffff0000u) : (va[u] & 0xffffu) | (vb[u] << 16);
        __stcs(reinterpret_cast<uint4*>(k + e), value4(wk[u], scale_f(sk[u], hi)));
        __stcs(reinterpret_cast<uint4*>(v + e), value4(wv, scale_f(sv[u], hi)));
      }
    }
  }
}

template <int D, int U>
int launch_rows4(bool write, const tv_pool& pool, int layer, const tv_seqs& seqs, const RowList& l, __nv_bfloat16* k,
                 __nv_bfloat16* v, size_t row_stride, size_t head_stride, int sms, int32_t* status, cudaStream_t st) {
  const int heads = U * 128 / D, per = kListThreads / 32, rows = write && U == 1 ? 1 : 2;
  const long long tasks = ((long long)l.rows + rows - 1) / rows * ((pool.n_kv_heads + heads - 1) / heads);
  const long long want = (tasks + per - 1) / per;
  const int most = sms * kBlocksPerSm;
  const dim3 grid((unsigned)(want < 1 ? 1 : (want < most ? want : most)));
  const size_t smem = write ? (size_t)((seqs.max_seqs + 31) / 32) * 4 : 0;
  const int rc = write ? launch_pdl(rows4_write_kernel<D, U>, grid, dim3(kListThreads), smem, st, pool, layer, seqs, l,
                                    (const __nv_bfloat16*)k, (const __nv_bfloat16*)v, row_stride, head_stride, status)
                       : launch_pdl(rows4_read_kernel<D, U>, grid, dim3(kListThreads), smem, st, pool, layer, seqs, l, k, v,
                                    row_stride, head_stride, status);
  return rc || grid.x == 1 ? rc : launch_rows_report(pool, seqs, l, sms, status, st);
}

int rows4_call(bool write, const tv_pool4* pool, int layer, const tv_seqs* seqs, const RowList& l, void* k, void* v,
               size_t row_stride, size_t head_stride, int32_t* status, void* stream) {
  PagePool p;
  int rc = check_pool(pool, &p);
  if (rc || (rc = check_rows(p, layer, seqs, l, k, v, row_stride, head_stride, status))) return rc;
  const int sms = num_sms();
  if (sms <= 0) return TV_E_CUDA;
  __nv_bfloat16 *kp = static_cast<__nv_bfloat16*>(k), *vp = static_cast<__nv_bfloat16*>(v);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // Few rows: small tasks, for latency; many: as many bytes in flight as a warp has room for.
  const bool few = ((long long)l.rows + 1) / 2 * p.n_kv_heads * p.head_dim / 512 < (long long)sms * kBlocksPerSm * (kListThreads / 32);
  auto launch = few ? (p.head_dim == 128 ? launch_rows4<128, 1> : launch_rows4<64, 1>)
                    : (p.head_dim == 128 ? launch_rows4<128, kMany> : launch_rows4<64, kMany>);
  return launch(write, p, layer, *seqs, l, kp, vp, row_stride, head_stride, sms, status, st);
}

}  // namespace
}  // namespace tv

using namespace tv;

extern "C" {

int tv_pages4_workspace_size(const tv_pool4* pool, const tv_seqs* seqs, size_t* bytes) {
  PagePool p;
  int rc = check_pool(pool, &p);
  if (rc || (rc = check_seqs(seqs, &p))) return rc;
  if (!bytes) return TV_E_ARG;
  *bytes = pages_ws_bytes(p);
  return TV_OK;
}

int tv_pages4_release(const tv_pool4* pool, const tv_seqs* seqs, const int32_t* ids, const int32_t* keep, int n,
                      int32_t* dev_status, void* stream) {
  PagePool p;
  const int rc = check_pool(pool, &p);
  return rc ? rc : pages_release(p, seqs, ids, keep, n, dev_status, stream);
}

int tv_pages4_fork(const tv_pool4* pool, const tv_seqs* seqs, const int32_t* src, const int32_t* dst, int n,
                   int32_t* dev_status, void* stream) {
  PagePool p;
  const int rc = check_pool(pool, &p);
  return rc ? rc : pages_fork(p, seqs, src, dst, n, dev_status, stream);
}

int tv_pages4_extend(const tv_pool4* pool, const tv_seqs* seqs, const int32_t* ids, const int32_t* add, int n,
                     void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  PagePool p;
  const int rc = check_pool(pool, &p);
  return rc ? rc : pages_extend(p, seqs, ids, add, n, workspace, workspace_bytes, dev_status, stream);
}

int tv_pages4_compact(const tv_pool4* pool, const tv_seqs* seqs, int32_t* remap, int32_t* n_used, void* workspace,
                      size_t workspace_bytes, int32_t* dev_status, void* stream) {
  PagePool p;
  const int rc = check_pool(pool, &p);
  return rc ? rc : pages_compact(p, seqs, remap, n_used, workspace, workspace_bytes, dev_status, stream);
}

int tv_pages4_write(const tv_pool4* pool, int layer, const tv_seqs* seqs, const int32_t* ids, const int32_t* pos,
                    const int32_t* starts, int n, int rows, const tv_bf16* k, const tv_bf16* v, size_t row_stride,
                    size_t head_stride, int32_t* dev_status, void* stream) {
  return rows4_call(true, pool, layer, seqs, RowList{ids, pos, starts, n, rows}, const_cast<tv_bf16*>(k),
                    const_cast<tv_bf16*>(v), row_stride, head_stride, dev_status, stream);
}

int tv_pages4_read(const tv_pool4* pool, int layer, const tv_seqs* seqs, const int32_t* ids, const int32_t* pos,
                   const int32_t* starts, int n, int rows, tv_bf16* k, tv_bf16* v, size_t row_stride,
                   size_t head_stride, int32_t* dev_status, void* stream) {
  return rows4_call(false, pool, layer, seqs, RowList{ids, pos, starts, n, rows}, k, v, row_stride, head_stride,
                    dev_status, stream);
}

}  // extern "C"
