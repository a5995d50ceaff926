"""Python binding of the C ABI in include/tv.h -- argument marshalling only.

Every function here has the name of its C entry point and does nothing but
turn Python values (ints, torch tensors, lists of structs) into the C
arguments and call the CUDA library.  All computation happens in the
library's kernels.  If the library is missing the import of a function fails
loudly: there is no fallback of any kind.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtv.so")

TV_OK = 0
STATUS = {
    0: "TV_OK", -1: "TV_E_ARG", -2: "TV_E_ORDER", -3: "TV_E_DUP_SIBLING", -4: "TV_E_TOKEN",
    -5: "TV_E_CAPACITY", -6: "TV_E_ROWS", -7: "TV_E_UNIFORM", -8: "TV_E_TEMP", -9: "TV_E_WORKSPACE",
    -10: "TV_E_CUDA", -11: "TV_E_UNSUPPORTED", -12: "TV_E_TIMEOUT", -13: "TV_E_PATH", -14: "TV_E_CHAIN",
    -15: "TV_E_PROPOSAL", -16: "TV_E_SEQ", -17: "TV_E_PAGE",
}
CODES = {v: k for k, v in STATUS.items()}

# entry points declared in include/tv.h
SYMBOLS = ("tv_workspace_size", "tv_verify_tree", "tv_accept_greedy", "tv_accept_residual", "tv_commit_kv",
           "tv_profile_start", "tv_profile_stop", "tv_status_string", "tv_accept_residual_noalloc",
           "tv_sample_workspace_size", "tv_sample_filter", "tv_accept_single_draw", "tv_accept_gumbel",
           "tv_accept_rejection", "tv_dn_verify_tree", "tv_dn_commit", "tv_price_init", "tv_price_lookup",
           "tv_price_observe", "tv_staircut", "tv_packed_weight_bytes", "tv_pack_weight",
           "tv_accept_greedy_commit", "tv_stack_workspace_size", "tv_verify_stack", "tv_commit_stack",
           "tv_pages_workspace_size", "tv_pages_extend", "tv_pages_fork", "tv_pages_release", "tv_pages_compact",
           "tv_pages_write", "tv_pages_read", "tv_attend_paged_workspace_size", "tv_attend_paged",
           "tv_attend_prompt", "tv_attend_prompt_window", "tv_attend_paged_window", "tv_pages4_workspace_size",
           "tv_pages4_extend", "tv_pages4_fork", "tv_pages4_release", "tv_pages4_compact", "tv_pages4_write",
           "tv_pages4_read", "tv_attend_paged4_workspace_size", "tv_attend_paged4", "tv_rope_init", "tv_rope_rows")
PROFILE_STAGES = ("prologue+embed", "qkv_gemm", "qkv_finalize", "attention", "o_gemm", "o_finalize", "lm_head")


class TvDims(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("vocab", ctypes.c_int32), ("rope_theta", ctypes.c_float),
                ("rms_eps", ctypes.c_float)]


class TvModel(ctypes.Structure):
    _fields_ = [("embed", ctypes.c_void_p), ("ln1", ctypes.c_void_p), ("wqkv", ctypes.c_void_p),
                ("wo", ctypes.c_void_p), ("ln_f", ctypes.c_void_p), ("lm_head", ctypes.c_void_p),
                ("dims", TvDims), ("packed", ctypes.c_int32)]


class TvKv(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("ctx_len", ctypes.c_int32),
                ("capacity", ctypes.c_int32)]


class TvTree(ctypes.Structure):
    _fields_ = [("parent", ctypes.c_void_p), ("token", ctypes.c_void_p), ("n", ctypes.c_int32)]


TV_KIND_CHAIN, TV_KIND_TREE = 0, 1
PRICE_MAX_CLASSES, PRICE_MAX_ROWS = 16, 32
_PriceRows = ctypes.c_double * (PRICE_MAX_ROWS + 1)


class TvPriceTable(ctypes.Structure):
    _fields_ = [("n_classes", ctypes.c_int32), ("class_ctx", ctypes.c_int32 * PRICE_MAX_CLASSES),
                ("step_ms", ctypes.c_double), ("prior", _PriceRows * 2 * PRICE_MAX_CLASSES),
                ("live", _PriceRows * 2 * PRICE_MAX_CLASSES), ("offset", ctypes.c_double * 2 * PRICE_MAX_CLASSES)]


class TvDnDims(ctypes.Structure):
    _fields_ = [("n_k_heads", ctypes.c_int32), ("n_v_heads", ctypes.c_int32), ("d_k", ctypes.c_int32),
                ("d_v", ctypes.c_int32)]


TV_LAYER_ATTN, TV_LAYER_DN = 0, 1


class TvLayer(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("ln_mix", ctypes.c_void_p), ("w_mix_in", ctypes.c_void_p),
                ("w_mix_out", ctypes.c_void_p), ("dn_norm", ctypes.c_void_p), ("ln_mlp", ctypes.c_void_p),
                ("w_gate_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p)]


class TvStack(ctypes.Structure):
    _fields_ = [("dims", TvDims), ("dn", TvDnDims), ("intermediate", ctypes.c_int32), ("n_layers", ctypes.c_int32),
                ("layers", ctypes.POINTER(TvLayer)), ("embed", ctypes.c_void_p), ("ln_f", ctypes.c_void_p),
                ("lm_head", ctypes.c_void_p), ("packed", ctypes.c_int32)]


class TvPool(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("refs", ctypes.c_void_p), ("n_layers", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("head_dim", ctypes.c_int32)]


class TvPool4(ctypes.Structure):
    _fields_ = TvPool._fields_


NO_WINDOW = (1 << 31) - 1   # a window that hides nothing
TV_ROPE_PLAIN, TV_ROPE_LINEAR, TV_ROPE_BASE, TV_ROPE_BLEND = 0, 1, 2, 3
ROPE_MAX_PAIRS = 64


class TvRope(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("gain", ctypes.c_double),
                ("freq", ctypes.c_double * ROPE_MAX_PAIRS)]


class TvSeqs(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("max_seqs", ctypes.c_int32),
                ("max_pages", ctypes.c_int32)]


_lib = None


class LibraryMissing(RuntimeError):
    pass


def load():
    """Load libtv.so (built in-tree by speculative_tree_verify_gb300.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise LibraryMissing(f"CUDA library not built: {LIB_PATH} is missing "
                                 "(run speculative_tree_verify_gb300.build.build())")
        lib = ctypes.CDLL(LIB_PATH)
        P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        lib.tv_workspace_size.argtypes = [ctypes.POINTER(TvDims), I, I, ctypes.POINTER(Z)]
        lib.tv_verify_tree.argtypes = [ctypes.POINTER(TvModel), ctypes.POINTER(TvKv), ctypes.POINTER(TvTree), I,
                                       P, P, P, P, P, Z, P, P]
        lib.tv_accept_greedy.argtypes = [ctypes.POINTER(TvTree), I, P, P, P, P, P, P]
        lib.tv_accept_residual.argtypes = [ctypes.POINTER(TvTree), I, P, ctypes.c_int32, ctypes.c_float, P, I,
                                           P, P, P, P, P, P, Z, P]
        lib.tv_accept_residual_noalloc.argtypes = [ctypes.POINTER(TvTree), I, P, ctypes.c_int32, ctypes.c_float, P,
                                                   I, P, P, P, P, P, P]
        lib.tv_commit_kv.argtypes = [ctypes.POINTER(TvKv), ctypes.POINTER(TvDims), ctypes.POINTER(TvTree), I,
                                     P, P, P, P, P, P]
        lib.tv_accept_greedy_commit.argtypes = [ctypes.POINTER(TvKv), ctypes.POINTER(TvDims), ctypes.POINTER(TvTree),
                                                I, P, P, P, P, P, P, P, P]
        lib.tv_packed_weight_bytes.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(Z)]
        lib.tv_pack_weight.argtypes = [P, ctypes.c_int32, ctypes.c_int32, P, P]
        lib.tv_profile_start.argtypes = [I]
        lib.tv_profile_stop.argtypes = [ctypes.POINTER(ctypes.c_float), I, ctypes.POINTER(I), ctypes.POINTER(I)]
        lib.tv_sample_workspace_size.argtypes = [ctypes.c_int32, I, ctypes.POINTER(Z)]
        lib.tv_sample_filter.argtypes = [P, P, I, ctypes.c_int32, ctypes.c_float, ctypes.c_int32, ctypes.c_float,
                                         ctypes.c_float, P, P]
        lib.tv_accept_single_draw.argtypes = [ctypes.POINTER(TvTree), I, P, ctypes.c_int32, ctypes.c_float, P, P,
                                              P, P, P, P, P, Z, P]
        lib.tv_accept_gumbel.argtypes = [ctypes.POINTER(TvTree), I, P, ctypes.c_int32, ctypes.c_float,
                                         ctypes.POINTER(ctypes.c_uint64), ctypes.POINTER(ctypes.c_int32), P, P, P,
                                         P, P, P, Z, P]
        lib.tv_accept_rejection.argtypes = [ctypes.POINTER(TvTree), I, P, ctypes.c_int32, ctypes.c_float, P, P,
                                            P, P, P, P, P, P, Z, P]
        lib.tv_dn_verify_tree.argtypes = [ctypes.POINTER(TvDnDims), ctypes.POINTER(TvTree), I, ctypes.POINTER(P), P,
                                          P, P, P, P, P, P, P, P, P]
        lib.tv_dn_commit.argtypes = [ctypes.POINTER(TvDnDims), ctypes.POINTER(TvTree), I, I, ctypes.POINTER(P), P, P,
                                     P, P, P, P, P]
        lib.tv_stack_workspace_size.argtypes = [ctypes.POINTER(TvStack), ctypes.POINTER(Z)]
        lib.tv_verify_stack.argtypes = [ctypes.POINTER(TvStack), ctypes.POINTER(TvKv), ctypes.POINTER(P),
                                        ctypes.POINTER(TvTree), I, P, P, P, P, P, Z, P, P]
        lib.tv_commit_stack.argtypes = [ctypes.POINTER(TvStack), ctypes.POINTER(TvKv), ctypes.POINTER(P),
                                        ctypes.POINTER(TvTree), I, P, P, P, P, P, Z, P, P]
        PO, SQ = ctypes.POINTER(TvPool), ctypes.POINTER(TvSeqs)
        lib.tv_pages_workspace_size.argtypes = [PO, SQ, ctypes.POINTER(Z)]
        lib.tv_pages_extend.argtypes = [PO, SQ, P, P, I, P, Z, P, P]
        lib.tv_pages_fork.argtypes = [PO, SQ, P, P, I, P, P]
        lib.tv_pages_release.argtypes = [PO, SQ, P, P, I, P, P]
        lib.tv_pages_compact.argtypes = [PO, SQ, P, P, P, Z, P, P]
        lib.tv_pages_write.argtypes = [PO, I, SQ, P, P, P, I, I, P, P, Z, Z, P, P]
        lib.tv_pages_read.argtypes = [PO, I, SQ, P, P, P, I, I, P, P, Z, Z, P, P]
        lib.tv_attend_prompt.argtypes = [I, I, I, P, P, P, Z, Z, P, I, I, P, P, P]
        lib.tv_attend_paged_workspace_size.argtypes = [PO, I, I, ctypes.POINTER(Z)]
        lib.tv_attend_paged.argtypes = [PO, I, SQ, P, I, I, P, Z, P, P, Z, P, P, Z, P, P]
        lib.tv_attend_prompt_window.argtypes = [I, I, I, I, I, P, P, P, Z, Z, P, I, I, P, P, P]
        lib.tv_attend_paged_window.argtypes = [PO, I, SQ, P, I, I, I, I, P, Z, P, P, Z, P, P, Z, P, P]
        P4 = ctypes.POINTER(TvPool4)
        for name in ("workspace_size", "extend", "fork", "release", "compact", "write", "read"):   # as those of tv_pool
            getattr(lib, "tv_pages4_" + name).argtypes = [P4] + getattr(lib, "tv_pages_" + name).argtypes[1:]
        lib.tv_attend_paged4_workspace_size.argtypes = [P4, I, I, ctypes.POINTER(Z)]
        lib.tv_attend_paged4.argtypes = [P4] + lib.tv_attend_paged_window.argtypes[1:]
        D = ctypes.c_double
        lib.tv_rope_init.argtypes = [ctypes.POINTER(TvRope), I, I, D, I, D, ctypes.c_int32, D, D, D]
        lib.tv_rope_rows.argtypes = [ctypes.POINTER(TvRope), P, Z, P, Z, I, I, P, I, P, P]
        lib.tv_price_init.argtypes = [ctypes.POINTER(TvPriceTable)]
        lib.tv_price_lookup.argtypes = [ctypes.POINTER(TvPriceTable), ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                        ctypes.POINTER(D)]
        lib.tv_price_observe.argtypes = [ctypes.POINTER(TvPriceTable), ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, D]
        lib.tv_staircut.argtypes = [P, P, P, ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(TvPriceTable),
                                    ctypes.c_int32, D, D, D, P, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(D)]
        lib.tv_status_string.argtypes = [I]
        lib.tv_status_string.restype = ctypes.c_char_p
        _lib = lib
    return _lib


def _p(x) -> Optional[int]:
    """Device/host address of a tensor, an int, or None."""
    if x is None or isinstance(x, int):
        return x
    return x.data_ptr()


def _i32(x) -> int:
    """A count of rows: what no int32 holds is more than any sequence has, and ctypes would cut it to 32 bits."""
    return max(-(1 << 31), min(int(x), (1 << 31) - 1))


def _arr(ctype, items: Sequence):
    return (ctype * len(items))(*items)


def _stream(stream) -> Optional[int]:
    if stream is None:
        return None
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def tv_status_string(code: int) -> str:
    return load().tv_status_string(int(code)).decode()


def tv_workspace_size(dims: TvDims, max_rows: int, max_ctx: int) -> int:
    out = ctypes.c_size_t(0)
    rc = load().tv_workspace_size(ctypes.byref(dims), int(max_rows), int(max_ctx), ctypes.byref(out))
    if rc != TV_OK:
        raise ValueError(f"tv_workspace_size: {STATUS.get(rc, rc)}")
    return int(out.value)


def tv_accept_greedy_commit(kvs: Sequence[TvKv], dims: TvDims, trees: Sequence[TvTree], argmax, path, accept_len,
                            out_tokens, committed_src, new_ctx, dev_status, stream=None) -> int:
    return load().tv_accept_greedy_commit(_arr(TvKv, kvs), ctypes.byref(dims), _arr(TvTree, trees), len(trees),
                                          _p(argmax), _p(path), _p(accept_len), _p(out_tokens), _p(committed_src),
                                          _p(new_ctx), _p(dev_status), _stream(stream))


def tv_packed_weight_bytes(rows: int, cols: int) -> int:
    out = ctypes.c_size_t(0)
    rc = load().tv_packed_weight_bytes(int(rows), int(cols), ctypes.byref(out))
    if rc != TV_OK:
        raise ValueError(f"tv_packed_weight_bytes: {STATUS.get(rc, rc)}")
    return int(out.value)


def tv_pack_weight(w, rows: int, cols: int, packed, stream=None) -> int:
    return load().tv_pack_weight(_p(w), int(rows), int(cols), _p(packed), _stream(stream))


def tv_verify_tree(model: TvModel, kvs: Sequence[TvKv], trees: Sequence[TvTree], logits, argmax, top2_gap,
                   attn_out, workspace, workspace_bytes: int, dev_status, stream=None) -> int:
    return load().tv_verify_tree(ctypes.byref(model), _arr(TvKv, kvs), _arr(TvTree, trees), len(trees),
                                 _p(logits), _p(argmax), _p(top2_gap), _p(attn_out), _p(workspace),
                                 int(workspace_bytes), _p(dev_status), _stream(stream))


def tv_accept_greedy(trees: Sequence[TvTree], argmax, path, accept_len, out_tokens, dev_status, stream=None) -> int:
    return load().tv_accept_greedy(_arr(TvTree, trees), len(trees), _p(argmax), _p(path), _p(accept_len),
                                   _p(out_tokens), _p(dev_status), _stream(stream))


def tv_accept_residual(trees: Sequence[TvTree], logits, vocab: int, temperature: float, uniforms,
                       bonus_at_leaf: bool, path, accept_len, out_tokens, out_count, dev_status, workspace,
                       workspace_bytes: int, stream=None) -> int:
    return load().tv_accept_residual(_arr(TvTree, trees), len(trees), _p(logits), int(vocab), float(temperature),
                                     _p(uniforms), 1 if bonus_at_leaf else 0, _p(path), _p(accept_len),
                                     _p(out_tokens), _p(out_count), _p(dev_status), _p(workspace),
                                     int(workspace_bytes), _stream(stream))


def tv_accept_residual_noalloc(trees: Sequence[TvTree], logits, vocab: int, temperature: float, uniforms,
                               bonus_at_leaf: bool, path, accept_len, out_tokens, out_count, dev_status,
                               stream=None) -> int:
    """tv_accept_residual for callers that cannot provide a workspace (the
    statistics live in a fixed 272 KB array inside the library; vocab <= 262144)."""
    return load().tv_accept_residual_noalloc(_arr(TvTree, trees), len(trees), _p(logits), int(vocab),
                                             float(temperature), _p(uniforms), 1 if bonus_at_leaf else 0,
                                             _p(path), _p(accept_len), _p(out_tokens), _p(out_count),
                                             _p(dev_status), _stream(stream))


def tv_sample_workspace_size(vocab: int, max_rows: int):
    """(rc, bytes) of workspace the sampled entry points need."""
    z = ctypes.c_size_t(0)
    rc = load().tv_sample_workspace_size(int(vocab), int(max_rows), ctypes.byref(z))
    return rc, int(z.value)


def tv_sample_filter(logits, filtered, rows: int, vocab: int, temperature: float, top_k: int, top_p: float,
                     min_p: float, dev_status, stream=None) -> int:
    return load().tv_sample_filter(_p(logits), _p(filtered), int(rows), int(vocab), float(temperature), int(top_k),
                                   float(top_p), float(min_p), _p(dev_status), _stream(stream))


def tv_accept_single_draw(trees: Sequence[TvTree], logits, vocab: int, temperature: float, uniforms, row_tokens,
                          path, accept_len, out_tokens, dev_status, workspace, workspace_bytes: int,
                          stream=None) -> int:
    return load().tv_accept_single_draw(_arr(TvTree, trees), len(trees), _p(logits), int(vocab), float(temperature),
                                        _p(uniforms), _p(row_tokens), _p(path), _p(accept_len), _p(out_tokens),
                                        _p(dev_status), _p(workspace), int(workspace_bytes), _stream(stream))


def tv_accept_gumbel(trees: Sequence[TvTree], logits, vocab: int, temperature: float, seeds: Sequence[int],
                     positions: Sequence[int], row_tokens, path, accept_len, out_tokens, dev_status, workspace,
                     workspace_bytes: int, stream=None) -> int:
    sd = (ctypes.c_uint64 * len(trees))(*[int(x) & 0xFFFFFFFFFFFFFFFF for x in seeds])
    ps = (ctypes.c_int32 * len(trees))(*[int(x) for x in positions])
    return load().tv_accept_gumbel(_arr(TvTree, trees), len(trees), _p(logits), int(vocab), float(temperature), sd,
                                   ps, _p(row_tokens), _p(path), _p(accept_len), _p(out_tokens), _p(dev_status),
                                   _p(workspace), int(workspace_bytes), _stream(stream))


def tv_accept_rejection(trees: Sequence[TvTree], logits, vocab: int, temperature: float, proposals, uniforms,
                        path, accept_len, out_tokens, out_count, dev_status, workspace, workspace_bytes: int,
                        stream=None) -> int:
    return load().tv_accept_rejection(_arr(TvTree, trees), len(trees), _p(logits), int(vocab), float(temperature),
                                      _p(proposals), _p(uniforms), _p(path), _p(accept_len), _p(out_tokens),
                                      _p(out_count), _p(dev_status), _p(workspace), int(workspace_bytes),
                                      _stream(stream))


def _ptrs(states):
    return (ctypes.c_void_p * len(states))(*[_p(x) for x in states])


def tv_dn_verify_tree(dims: TvDnDims, trees: Sequence[TvTree], states, q, k, v, beta, g, o, u, gc, dev_status,
                      stream=None) -> int:
    """states: one device buffer (tensor or address) per request."""
    return load().tv_dn_verify_tree(ctypes.byref(dims), _arr(TvTree, trees), len(trees), _ptrs(states), _p(q), _p(k),
                                    _p(v), _p(beta), _p(g), _p(o), _p(u), _p(gc), _p(dev_status), _stream(stream))


def tv_dn_commit(dims: TvDnDims, trees: Sequence[TvTree], n_layers: int, states, k, u, gc, path, accept_len,
                 dev_status, stream=None) -> int:
    return load().tv_dn_commit(ctypes.byref(dims), _arr(TvTree, trees), len(trees), int(n_layers), _ptrs(states),
                               _p(k), _p(u), _p(gc), _p(path), _p(accept_len), _p(dev_status), _stream(stream))


def tv_stack_workspace_size(stack: TvStack):
    """(rc, bytes) of workspace tv_verify_stack / tv_commit_stack need."""
    z = ctypes.c_size_t(0)
    rc = load().tv_stack_workspace_size(ctypes.byref(stack), ctypes.byref(z))
    return rc, int(z.value)


def tv_verify_stack(stack: TvStack, kvs: Sequence[TvKv], dn_states, trees: Sequence[TvTree], logits, argmax,
                    top2_gap, x_taps, workspace, workspace_bytes: int, dev_status, stream=None) -> int:
    """kvs: [n_attn_layers * n_req] (layer-major); dn_states: one device buffer
    per request; x_taps: bf16 [2 n_layers + 1][rows][hidden] or None."""
    return load().tv_verify_stack(ctypes.byref(stack), _arr(TvKv, kvs) if kvs else None,
                                  _ptrs(dn_states) if dn_states else None, _arr(TvTree, trees), len(trees),
                                  _p(logits), _p(argmax), _p(top2_gap), _p(x_taps), _p(workspace),
                                  int(workspace_bytes), _p(dev_status), _stream(stream))


def tv_commit_stack(stack: TvStack, kvs: Sequence[TvKv], dn_states, trees: Sequence[TvTree], path, accept_len,
                    committed_src, new_ctx, workspace, workspace_bytes: int, dev_status, stream=None) -> int:
    return load().tv_commit_stack(ctypes.byref(stack), _arr(TvKv, kvs) if kvs else None, _ptrs(dn_states) if dn_states else None,
                                  _arr(TvTree, trees), len(trees), _p(path), _p(accept_len), _p(committed_src),
                                  _p(new_ctx), _p(workspace), int(workspace_bytes), _p(dev_status), _stream(stream))


def tv_pages_workspace_size(pool: TvPool, seqs: TvSeqs) -> int:
    out = ctypes.c_size_t(0)
    rc = load().tv_pages_workspace_size(ctypes.byref(pool), ctypes.byref(seqs), ctypes.byref(out))
    if rc != TV_OK:
        raise ValueError(f"tv_pages_workspace_size: {STATUS.get(rc, rc)}")
    return int(out.value)


def tv_pages_extend(pool: TvPool, seqs: TvSeqs, ids, add, n: int, workspace, workspace_bytes: int, dev_status,
                    stream=None) -> int:
    return load().tv_pages_extend(ctypes.byref(pool), ctypes.byref(seqs), _p(ids), _p(add), int(n), _p(workspace),
                                  int(workspace_bytes), _p(dev_status), _stream(stream))


def tv_pages_fork(pool: TvPool, seqs: TvSeqs, src, dst, n: int, dev_status, stream=None) -> int:
    return load().tv_pages_fork(ctypes.byref(pool), ctypes.byref(seqs), _p(src), _p(dst), int(n), _p(dev_status),
                                _stream(stream))


def tv_pages_release(pool: TvPool, seqs: TvSeqs, ids, keep, n: int, dev_status, stream=None) -> int:
    return load().tv_pages_release(ctypes.byref(pool), ctypes.byref(seqs), _p(ids), _p(keep), int(n), _p(dev_status),
                                   _stream(stream))


def tv_pages_compact(pool: TvPool, seqs: TvSeqs, remap, n_used, workspace, workspace_bytes: int, dev_status,
                     stream=None) -> int:
    return load().tv_pages_compact(ctypes.byref(pool), ctypes.byref(seqs), _p(remap), _p(n_used), _p(workspace),
                                   int(workspace_bytes), _p(dev_status), _stream(stream))


def tv_pages_write(pool: TvPool, layer: int, seqs: TvSeqs, ids, pos, starts, n: int, rows: int, k, v,
                   row_stride: int, head_stride: int, dev_status, stream=None) -> int:
    """Strides in elements: the K heads of projection rows, or a tv_kv cache (row_stride = head_dim)."""
    return load().tv_pages_write(ctypes.byref(pool), int(layer), ctypes.byref(seqs), _p(ids), _p(pos), _p(starts),
                                 int(n), int(rows), _p(k), _p(v), int(row_stride), int(head_stride), _p(dev_status),
                                 _stream(stream))


def tv_pages_read(pool: TvPool, layer: int, seqs: TvSeqs, ids, pos, starts, n: int, rows: int, k, v, row_stride: int,
                  head_stride: int, dev_status, stream=None) -> int:
    """As tv_pages_write, from the pages into k and v."""
    return load().tv_pages_read(ctypes.byref(pool), int(layer), ctypes.byref(seqs), _p(ids), _p(pos), _p(starts),
                                int(n), int(rows), _p(k), _p(v), int(row_stride), int(head_stride), _p(dev_status),
                                _stream(stream))


def tv_attend_prompt(n_q_heads: int, n_kv_heads: int, head_dim: int, q, k, v, q_stride: int, kv_stride: int, starts,
                     n_seqs: int, rows: int, out, dev_status, stream=None) -> int:
    """Strides in elements."""
    return load().tv_attend_prompt(int(n_q_heads), int(n_kv_heads), int(head_dim), _p(q), _p(k), _p(v), int(q_stride),
                                   int(kv_stride), _p(starts), int(n_seqs), int(rows), _p(out), _p(dev_status),
                                   _stream(stream))


def tv_attend_paged_workspace_size(pool: TvPool, n_q_heads: int, n: int) -> int:
    out = ctypes.c_size_t(0)
    rc = load().tv_attend_paged_workspace_size(ctypes.byref(pool), int(n_q_heads), int(n), ctypes.byref(out))
    if rc != TV_OK:
        raise ValueError(f"tv_attend_paged_workspace_size: {STATUS.get(rc, rc)}")
    return int(out.value)


def tv_attend_paged(pool: TvPool, layer: int, seqs: TvSeqs, ids, n: int, n_q_heads: int, q, q_stride: int, k_new,
                    v_new, kv_stride: int, out, workspace, workspace_bytes: int, dev_status, stream=None) -> int:
    """Strides in elements; k_new and v_new may be None."""
    return load().tv_attend_paged(ctypes.byref(pool), int(layer), ctypes.byref(seqs), _p(ids), int(n), int(n_q_heads),
                                  _p(q), int(q_stride), _p(k_new), _p(v_new), int(kv_stride), _p(out), _p(workspace),
                                  int(workspace_bytes), _p(dev_status), _stream(stream))


def tv_attend_prompt_window(n_q_heads: int, n_kv_heads: int, head_dim: int, window: int, sinks: int, q, k, v,
                            q_stride: int, kv_stride: int, starts, n_seqs: int, rows: int, out, dev_status,
                            stream=None) -> int:
    """Strides in elements."""
    return load().tv_attend_prompt_window(int(n_q_heads), int(n_kv_heads), int(head_dim), _i32(window), _i32(sinks),
                                          _p(q), _p(k), _p(v), int(q_stride), int(kv_stride), _p(starts), int(n_seqs),
                                          int(rows), _p(out), _p(dev_status), _stream(stream))


def tv_attend_paged_window(pool: TvPool, layer: int, seqs: TvSeqs, ids, n: int, n_q_heads: int, window: int,
                           sinks: int, q, q_stride: int, k_new, v_new, kv_stride: int, out, workspace,
                           workspace_bytes: int, dev_status, stream=None) -> int:
    """Strides in elements; k_new and v_new may be None."""
    return load().tv_attend_paged_window(ctypes.byref(pool), int(layer), ctypes.byref(seqs), _p(ids), int(n),
                                         int(n_q_heads), _i32(window), _i32(sinks), _p(q), int(q_stride), _p(k_new),
                                         _p(v_new), int(kv_stride), _p(out), _p(workspace), int(workspace_bytes),
                                         _p(dev_status), _stream(stream))


def tv_pages4_workspace_size(pool: TvPool4, seqs: TvSeqs) -> int:
    out = ctypes.c_size_t(0)
    rc = load().tv_pages4_workspace_size(ctypes.byref(pool), ctypes.byref(seqs), ctypes.byref(out))
    if rc != TV_OK:
        raise ValueError(f"tv_pages4_workspace_size: {STATUS.get(rc, rc)}")
    return int(out.value)


def tv_pages4_extend(pool: TvPool4, seqs: TvSeqs, ids, add, n: int, workspace, workspace_bytes: int, dev_status,
                     stream=None) -> int:
    return load().tv_pages4_extend(ctypes.byref(pool), ctypes.byref(seqs), _p(ids), _p(add), int(n), _p(workspace),
                                   int(workspace_bytes), _p(dev_status), _stream(stream))


def tv_pages4_fork(pool: TvPool4, seqs: TvSeqs, src, dst, n: int, dev_status, stream=None) -> int:
    return load().tv_pages4_fork(ctypes.byref(pool), ctypes.byref(seqs), _p(src), _p(dst), int(n), _p(dev_status),
                                 _stream(stream))


def tv_pages4_release(pool: TvPool4, seqs: TvSeqs, ids, keep, n: int, dev_status, stream=None) -> int:
    return load().tv_pages4_release(ctypes.byref(pool), ctypes.byref(seqs), _p(ids), _p(keep), int(n), _p(dev_status),
                                    _stream(stream))


def tv_pages4_compact(pool: TvPool4, seqs: TvSeqs, remap, n_used, workspace, workspace_bytes: int, dev_status,
                      stream=None) -> int:
    return load().tv_pages4_compact(ctypes.byref(pool), ctypes.byref(seqs), _p(remap), _p(n_used), _p(workspace),
                                    int(workspace_bytes), _p(dev_status), _stream(stream))


def tv_pages4_write(pool: TvPool4, layer: int, seqs: TvSeqs, ids, pos, starts, n: int, rows: int, k, v,
                    row_stride: int, head_stride: int, dev_status, stream=None) -> int:
    """As tv_pages_write, from bf16 rows into 4 bits."""
    return load().tv_pages4_write(ctypes.byref(pool), int(layer), ctypes.byref(seqs), _p(ids), _p(pos), _p(starts),
                                  int(n), int(rows), _p(k), _p(v), int(row_stride), int(head_stride), _p(dev_status),
                                  _stream(stream))


def tv_pages4_read(pool: TvPool4, layer: int, seqs: TvSeqs, ids, pos, starts, n: int, rows: int, k, v,
                   row_stride: int, head_stride: int, dev_status, stream=None) -> int:
    """As tv_pages_read, from 4 bits into bf16 rows."""
    return load().tv_pages4_read(ctypes.byref(pool), int(layer), ctypes.byref(seqs), _p(ids), _p(pos), _p(starts),
                                 int(n), int(rows), _p(k), _p(v), int(row_stride), int(head_stride), _p(dev_status),
                                 _stream(stream))


def tv_attend_paged4_workspace_size(pool: TvPool4, n_q_heads: int, n: int) -> int:
    out = ctypes.c_size_t(0)
    rc = load().tv_attend_paged4_workspace_size(ctypes.byref(pool), int(n_q_heads), int(n), ctypes.byref(out))
    if rc != TV_OK:
        raise ValueError(f"tv_attend_paged4_workspace_size: {STATUS.get(rc, rc)}")
    return int(out.value)


def tv_attend_paged4(pool: TvPool4, layer: int, seqs: TvSeqs, ids, n: int, n_q_heads: int, window: int, sinks: int, q,
                     q_stride: int, k_new, v_new, kv_stride: int, out, workspace, workspace_bytes: int, dev_status,
                     stream=None) -> int:
    """Strides in elements; k_new and v_new may be None."""
    return load().tv_attend_paged4(ctypes.byref(pool), int(layer), ctypes.byref(seqs), _p(ids), int(n),
                                   int(n_q_heads), _i32(window), _i32(sinks), _p(q), int(q_stride), _p(k_new), _p(v_new),
                                   int(kv_stride), _p(out), _p(workspace), int(workspace_bytes), _p(dev_status),
                                   _stream(stream))


def tv_rope_init(rot_dim: int, interleaved: bool = False, theta: float = 10000.0, scaling: int = TV_ROPE_PLAIN,
                 factor: float = 1.0, original_ctx: int = 1, low_turns: float = 1.0, high_turns: float = 32.0,
                 gain: float = 1.0) -> TvRope:
    rope = TvRope()
    if scaling == TV_ROPE_BLEND and int(original_ctx) >= 1 << 31:   # ctypes would cut it to 32 bits
        raise ValueError("tv_rope_init: TV_E_ARG")
    rc = load().tv_rope_init(ctypes.byref(rope), int(rot_dim), 1 if interleaved else 0, float(theta), int(scaling),
                             float(factor), int(original_ctx), float(low_turns), float(high_turns), float(gain))
    if rc != TV_OK:
        raise ValueError(f"tv_rope_init: {STATUS.get(rc, rc)}")
    return rope


def tv_rope_rows(rope: TvRope, x, x_stride: int, out, out_stride: int, n_heads: int, head_dim: int, positions,
                 rows: int, dev_status, stream=None) -> int:
    """Strides in elements; out may be x."""
    return load().tv_rope_rows(ctypes.byref(rope), _p(x), int(x_stride), _p(out), int(out_stride), int(n_heads),
                               int(head_dim), _p(positions), int(rows), _p(dev_status), _stream(stream))


def tv_price_init(table: TvPriceTable) -> int:
    return load().tv_price_init(ctypes.byref(table))


def tv_price_lookup(table: TvPriceTable, context: int, kind: int, rows: int):
    """(rc, ms)"""
    ms = ctypes.c_double(0.0)
    rc = load().tv_price_lookup(ctypes.byref(table), int(context), int(kind), int(rows), ctypes.byref(ms))
    return rc, ms.value


def tv_price_observe(table: TvPriceTable, context: int, kind: int, rows: int, ms: float) -> int:
    return load().tv_price_observe(ctypes.byref(table), int(context), int(kind), int(rows), float(ms))


def tv_staircut(parent, q, score, kind: int, table: TvPriceTable, context: int, draft_ms: float, commit_ms: float,
                rollback_ms: float = 0.0):
    """Host arrays (numpy int32 / float32).  Returns (rc, kept nodes, value)."""
    import numpy as np
    par = np.ascontiguousarray(parent, dtype=np.int32)
    qq = np.ascontiguousarray(q, dtype=np.float32)
    sc = np.ascontiguousarray(score, dtype=np.float32)
    n = int(par.shape[0])
    keep = np.zeros(max(n, 1), dtype=np.int32)
    nk, val = ctypes.c_int32(0), ctypes.c_double(0.0)
    rc = load().tv_staircut(par.ctypes.data, qq.ctypes.data, sc.ctypes.data, n, int(kind), ctypes.byref(table),
                            int(context), float(draft_ms), float(commit_ms), float(rollback_ms), keep.ctypes.data,
                            ctypes.byref(nk), ctypes.byref(val))
    return rc, keep[:nk.value].tolist(), val.value


def tv_commit_kv(kvs: Sequence[TvKv], dims: TvDims, trees: Sequence[TvTree], path, accept_len, committed_src,
                 new_ctx, dev_status, stream=None) -> int:
    return load().tv_commit_kv(_arr(TvKv, kvs), ctypes.byref(dims), _arr(TvTree, trees), len(trees), _p(path),
                               _p(accept_len), _p(committed_src), _p(new_ctx), _p(dev_status), _stream(stream))


def tv_profile_start(max_calls: int) -> int:
    return load().tv_profile_start(int(max_calls))


def tv_profile_stop():
    """-> (rc, {stage name: summed ms}, recorded calls)"""
    ms = (ctypes.c_float * len(PROFILE_STAGES))()
    ns, nc = ctypes.c_int(0), ctypes.c_int(0)
    rc = load().tv_profile_stop(ms, len(PROFILE_STAGES), ctypes.byref(ns), ctypes.byref(nc))
    return rc, {name: float(ms[i]) for i, name in enumerate(PROFILE_STAGES)}, int(nc.value)
