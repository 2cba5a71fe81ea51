"""Python binding of libspecverify.so: the C-ABI's entry points under the same names.

Argument marshalling only.  Array arguments are torch CUDA tensors (contiguous; their
device pointers are passed) or raw device addresses as ints; ``stream`` is a torch stream,
a raw hipStream_t as an int, or None for torch's current stream.  A non-zero status from
the library raises SpecVerifyError.  All computation happens in the library's kernels;
there is no fallback: if the library cannot be built or loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import build as _build

SPECVERIFY_F32 = 0
SPECVERIFY_BF16 = 1

SPECVERIFY_OK = 0
SPECVERIFY_EINVAL = -1
SPECVERIFY_EUNSUPPORTED = -2
SPECVERIFY_ENOMEM = -3
SPECVERIFY_EHIP = -4
SPECVERIFY_ECAPACITY = -5

SPECVERIFY_MAX_K = 63
SPECVERIFY_MAX_VOCAB = 1 << 20
SPECVERIFY_STATIC_SCRATCH_BYTES = 4 << 20
SPECVERIFY_MAX_CUT_N = 8192
SPECVERIFY_NUM_KERNELS = 7
SPECVERIFY_MAX_PAGES = 1 << 30
SPECVERIFY_MAX_SEQS = 1 << 20
SPECVERIFY_MAX_BLOCKS = 1 << 20
SPECVERIFY_MAX_POOLS = 1 << 16
SPECVERIFY_MAX_PAGE_BYTES = 1 << 30
SPECVERIFY_MAX_NODES = 64
SPECVERIFY_MAX_HEAD_DIM = 256
SPECVERIFY_MAX_ENTRIES = 1 << 16
SPECVERIFY_TEST_CHUNK_FALLBACK = 1
SPECVERIFY_TEST_EXACT_TWO_PASS = 2
KERNEL_NAMES = ("row_stats", "accept_draw", "row_argmax", "greedy_emit", "quantile_cut",
                "early_accept", "early_rest_stats")

_lib = None
_lock = threading.Lock()


class SpecVerifyFilter(ctypes.Structure):
    """Per-row parameters of a cut law: device tensors (or addresses), None for what cuts nothing.
    The tensors are held for as long as the filter lives."""
    _fields_ = [(name, ctypes.c_void_p) for name in ("temperature", "top_k", "top_p", "min_p")]

    def __init__(self, temperature=None, top_k=None, top_p=None, min_p=None):
        self.tensors = {"temperature": temperature, "top_k": top_k, "top_p": top_p, "min_p": min_p}
        super().__init__(*(_ptr(t) for t in self.tensors.values()))

    def check(self, count: int):
        """The tensors' types and sizes against a call of `count` rows or sequences."""
        for name, t in self.tensors.items():
            _arr(t, count, "i32" if name == "top_k" else "f32", name)


class SpecVerifyNodes(ctypes.Structure):
    """A step's nodes: device tensors (or addresses), None for what the library fills in (see the
    header).  The tensors are held for as long as the structure lives."""
    _fields_ = [(name, ctypes.c_void_p) for name in ("seqs", "starts", "counts", "parents")]

    def __init__(self, seqs=None, starts=None, counts=None, parents=None):
        self.tensors = {"seqs": seqs, "starts": starts, "counts": counts, "parents": parents}
        self.checked = None
        super().__init__(*(_ptr(t) for t in self.tensors.values()))

    def check(self, n: int, rows: int):
        """The tensors' types and sizes against a call of n entries and `rows` rows."""
        if self.checked != (n, rows):
            for name, t in self.tensors.items():
                _arr(t, rows if name == "parents" else n, "i32", name)
            self.checked = (n, rows)


class SpecVerifyRotation(ctypes.Structure):
    """The rotation of positions: inv_freq [dims / 2] float32 on the device, held while this lives."""
    _fields_ = [("inv_freq", ctypes.c_void_p), ("dims", ctypes.c_int), ("interleaved", ctypes.c_int)]

    def __init__(self, inv_freq, dims, interleaved=False):
        _arr(inv_freq, dims // 2, "f32", "inv_freq")
        self.tensor = inv_freq
        super().__init__(_ptr(inv_freq), dims, int(bool(interleaved)))


class SpecVerifyError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s (status %d)" % (where, specverify_strerror(status), status))


# Another build of the same sources may be loaded instead (the sanitizer run of the CPU tests
# builds the host code with AddressSanitizer and UndefinedBehaviorSanitizer).
_LIB_OVERRIDE = os.environ.get("SPECVERIFY_LIB")


def library_path() -> str:
    return _LIB_OVERRIDE or _build.LIB


def load():
    """Load libspecverify.so, building it first only if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not _LIB_OVERRIDE and not os.path.exists(_build.LIB):
            _build.build(force=True)
        lib = ctypes.CDLL(library_path())
        vp, i, f, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_int64
        lib.specverify_create.argtypes = [ctypes.POINTER(vp), i, i, i, i]
        lib.specverify_create.restype = i
        lib.specverify_workspace_bytes.argtypes = [vp]
        lib.specverify_workspace_bytes.restype = i64
        lib.specverify_run_sampling.argtypes = [vp, vp, i, i, i, i, f, vp, vp, vp, vp, vp, vp, vp]
        lib.specverify_run_sampling.restype = i
        lib.specverify_run_sampling_early_exit.argtypes = lib.specverify_run_sampling.argtypes
        lib.specverify_run_sampling_early_exit.restype = i
        lib.specverify_run_sampling_static.argtypes = [vp, i, i, i, i, f, vp, vp, vp, vp, vp, vp,
                                                       vp]
        lib.specverify_run_sampling_static.restype = i
        lib.specverify_run_contrastive.argtypes = [vp, vp, i, i, i, i, f, vp, vp, vp, vp, vp, vp,
                                                   vp]
        lib.specverify_run_contrastive.restype = i
        lib.specverify_run_contrastive_early_exit.argtypes = lib.specverify_run_contrastive.argtypes
        lib.specverify_run_contrastive_early_exit.restype = i
        lib.specverify_run_greedy.argtypes = [vp, vp, i, i, i, i, vp, vp, vp, vp]
        lib.specverify_run_greedy.restype = i
        lib.specverify_run_greedy_early_exit.argtypes = lib.specverify_run_greedy.argtypes
        lib.specverify_run_greedy_early_exit.restype = i
        lib.specverify_sample.argtypes = [vp, vp, i, i, i, f, vp, vp, vp, vp]
        lib.specverify_sample.restype = i
        lib.specverify_run_greedy_heads.argtypes = [vp, vp, i, i, i, i, i, vp, vp, vp, vp, vp]
        lib.specverify_run_greedy_heads.restype = i
        lib.specverify_quantile_cut.argtypes = [vp, vp, i, i, f, vp, vp, vp, vp]
        lib.specverify_quantile_cut.restype = i
        flt = ctypes.POINTER(SpecVerifyFilter)
        lib.specverify_sample_filtered.argtypes = [vp, vp, i, i, i, i64, flt, vp, vp, vp, vp]
        lib.specverify_run_sampling_filtered.argtypes = [vp, vp, i, i, i, i, flt, flt, vp, vp, vp,
                                                         vp, vp, vp, vp]
        lib.specverify_cache_create.argtypes = [ctypes.POINTER(vp), i, i, i, i, i, i, i64,
                                                ctypes.POINTER(vp), vp, vp, vp, vp]
        lib.specverify_cache_workspace_bytes.argtypes = [vp]
        lib.specverify_cache_workspace_bytes.restype = i64
        lib.specverify_cache_destroy.argtypes = [vp]
        lib.specverify_cache_reserve.argtypes = [vp, vp, i, vp, vp, vp]
        lib.specverify_cache_commit.argtypes = [vp, vp, i, vp, vp, vp]
        lib.specverify_cache_fork.argtypes = [vp, vp, i, vp, vp, vp]
        lib.specverify_cache_free.argtypes = [vp, vp, i, vp, vp]
        lib.specverify_cache_compact.argtypes = [vp, vp, vp, vp]
        lib.specverify_cache_copy.argtypes = [vp, vp, i, vp, vp, vp]
        lib.specverify_run_greedy_tree.argtypes = [vp, vp, i, i, i, i, i, vp, vp, vp, vp, vp, vp, vp]
        lib.specverify_cache_keep_path.argtypes = [vp, vp, i, i, vp, vp, vp, vp]
        nodes, rotation = ctypes.POINTER(SpecVerifyNodes), ctypes.POINTER(SpecVerifyRotation)
        lib.specverify_attn_create.argtypes = [ctypes.POINTER(vp), vp, i, i, i, i, i, i]
        lib.specverify_attn_workspace_bytes.argtypes = [vp]
        lib.specverify_attn_workspace_bytes.restype = i64
        lib.specverify_attn_destroy.argtypes = [vp]
        lib.specverify_attn_append.argtypes = [vp, vp, i, i, i, i, i, nodes, rotation, vp, i64, vp, i64,
                                               vp, i64, vp, i64, vp]
        lib.specverify_attn_attend.argtypes = [vp, vp, i, i, i, i, i, nodes, f, i, vp, i64, vp, i64, vp,
                                               vp]
        lib.specverify_set_test_flags.argtypes = [vp, ctypes.c_uint]
        lib.specverify_set_test_flags.restype = i
        lib.specverify_destroy.argtypes = [vp]
        lib.specverify_destroy.restype = i
        lib.specverify_strerror.argtypes = [i]
        lib.specverify_strerror.restype = ctypes.c_char_p
        lib.specverify_profile_begin.argtypes = [vp, i, ctypes.c_uint, i]
        lib.specverify_profile_begin.restype = i
        lib.specverify_profile_launches.argtypes = [vp, i, ctypes.POINTER(ctypes.c_float), i]
        lib.specverify_profile_launches.restype = i
        lib.specverify_profile_end.argtypes = [vp, ctypes.POINTER(ctypes.c_double),
                                               ctypes.POINTER(ctypes.c_int)]
        lib.specverify_profile_end.restype = i
        _lib = lib
        return lib


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        if not x.is_cuda:
            raise ValueError("expected a device tensor, got one on %s" % x.device)
        if not x.is_contiguous():
            raise ValueError("expected a contiguous tensor")
        return x.data_ptr()
    raise TypeError("expected a torch tensor, an int device address or None, got %r" % type(x))


_ITEMSIZE = {"i32": 4, "f32": 4, "u8": 1}


def _ptrs(*specs):
    """The pointers of a call's array arguments, each spec (x, count, kind, name): every tensor
    is first checked against the call's shape (_arr), then converted (_ptr)."""
    kinds, out = _KINDS or _kinds(), []
    for x, count, kind, name in specs:
        if x is None or type(x) is int:
            out.append(x)
            continue
        # what passes needs no second look; anything else is checked in order, for the right error
        try:
            fine = (x.is_cuda and x.dtype in kinds[kind][0] and x.numel() >= count
                    and x.is_contiguous())
        except (AttributeError, KeyError):
            fine = False
        if not fine:
            for y, n, k, what in specs:
                _arr(y, n, k, what)
            return tuple(_ptr(y) for y, _, _, _ in specs)
        out.append(x.data_ptr())
    return out


_KINDS = {}       # kind -> (accepted element types, their name), filled at the first tensor


def _kinds():
    import torch
    _KINDS.update({
        SPECVERIFY_F32: ((torch.float32,), "float32"),
        SPECVERIFY_BF16: ((torch.bfloat16, torch.int16, torch.uint16),
                          "bfloat16 (or its 16-bit patterns)"),
        "i32": ((torch.int32,), "int32"), "f32": ((torch.float32,), "float32"),
        "u8": ((torch.uint8, torch.bool), "uint8")})
    return _KINDS


def _arr(x, count: int, kind, name: str):
    """Check a tensor argument against the call's shape: its element type (kind: "i32", "f32",
    "u8", or a logits dtype SPECVERIFY_F32 / SPECVERIFY_BF16) and at least `count` elements,
    so that no kernel reads or writes past it.  Plain integer addresses are not checked: their
    extent is the caller's to guarantee."""
    if x is None or isinstance(x, int) or not hasattr(x, "data_ptr"):
        return
    # any other logits dtype is checked as bfloat16 and refused by the library
    kinds = _KINDS or _kinds()
    ok, what = kinds.get(kind) or kinds[SPECVERIFY_BF16 if isinstance(kind, int) else kind]
    if x.dtype not in ok:
        raise ValueError("%s: expected %s elements, got %s" % (name, what, x.dtype))
    if x.numel() < count:
        raise ValueError("%s: needs at least %d elements for this call, has %d"
                         % (name, count, x.numel()))


def _verify_args(dtype, B, K, V, target, draft, tokens, uniforms, acc, out, probs, draft_rows):
    """The pointers of a sampling or contrastive verify call, checked against B, K and V
    (draft_rows: K for sampling, K + 1 for contrastive)."""
    return _ptrs((target, B * (K + 1) * V, dtype, "target/expert logits"),
                 (draft, B * draft_rows * V, dtype, "draft/amateur logits"),
                 (tokens, B * K, "i32", "draft_tokens"),
                 (uniforms, B * (K + 1), "f32", "uniforms"),
                 (acc, B, "i32", "accepted_len"),
                 (out, B * (K + 1), "i32", "out_tokens"),
                 (probs, B * K * 2, "f32", "out_probs"))


def _stream(s):
    if isinstance(s, int):
        return s
    if s is None:
        import torch
        if torch.cuda.is_initialized():      # the same handle without a Stream object around it
            return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    return s.cuda_stream


def _check(status: int, where: str):
    if status != SPECVERIFY_OK:
        raise SpecVerifyError(status, where)


def specverify_strerror(status: int) -> str:
    return load().specverify_strerror(int(status)).decode()


def specverify_create(device: int, max_batch: int, max_k: int, max_vocab: int) -> int:
    """Returns the context handle (an int)."""
    h = ctypes.c_void_p()
    _check(load().specverify_create(ctypes.byref(h), device, max_batch, max_k, max_vocab),
           "specverify_create")
    return h.value


def specverify_workspace_bytes(ctx: int) -> int:
    return int(load().specverify_workspace_bytes(ctx))


def specverify_run_sampling(ctx, stream, dtype, B, K, V, temperature, target_logits,
                            draft_logits, draft_tokens, uniforms, accepted_len, out_tokens,
                            out_probs=None) -> None:
    ptrs = _verify_args(dtype, B, K, V, target_logits, draft_logits, draft_tokens, uniforms,
                        accepted_len, out_tokens, out_probs, K)
    _check(load().specverify_run_sampling(ctx, _stream(stream), dtype, B, K, V,
                                          float(temperature), *ptrs), "specverify_run_sampling")


def specverify_run_sampling_static(stream, dtype, B, K, V, temperature, target_logits,
                                   draft_logits, draft_tokens, uniforms, accepted_len, out_tokens,
                                   out_probs=None) -> None:
    ptrs = _verify_args(dtype, B, K, V, target_logits, draft_logits, draft_tokens, uniforms,
                        accepted_len, out_tokens, out_probs, K)
    _check(load().specverify_run_sampling_static(_stream(stream), dtype, B, K, V,
                                                 float(temperature), *ptrs),
           "specverify_run_sampling_static")


def specverify_run_sampling_early_exit(ctx, stream, dtype, B, K, V, temperature, target_logits,
                                       draft_logits, draft_tokens, uniforms, accepted_len,
                                       out_tokens, out_probs=None) -> None:
    ptrs = _verify_args(dtype, B, K, V, target_logits, draft_logits, draft_tokens, uniforms,
                        accepted_len, out_tokens, out_probs, K)
    _check(load().specverify_run_sampling_early_exit(ctx, _stream(stream), dtype, B, K, V,
                                                     float(temperature), *ptrs),
           "specverify_run_sampling_early_exit")


def specverify_run_contrastive(ctx, stream, dtype, B, K, V, tau, expert_logits, amateur_logits,
                               draft_tokens, uniforms, accepted_len, out_tokens,
                               out_probs=None) -> None:
    ptrs = _verify_args(dtype, B, K, V, expert_logits, amateur_logits, draft_tokens, uniforms,
                        accepted_len, out_tokens, out_probs, K + 1)
    _check(load().specverify_run_contrastive(ctx, _stream(stream), dtype, B, K, V, float(tau),
                                             *ptrs), "specverify_run_contrastive")


def specverify_run_contrastive_early_exit(ctx, stream, dtype, B, K, V, tau, expert_logits,
                                          amateur_logits, draft_tokens, uniforms, accepted_len,
                                          out_tokens, out_probs=None) -> None:
    ptrs = _verify_args(dtype, B, K, V, expert_logits, amateur_logits, draft_tokens, uniforms,
                        accepted_len, out_tokens, out_probs, K + 1)
    _check(load().specverify_run_contrastive_early_exit(ctx, _stream(stream), dtype, B, K, V,
                                                        float(tau), *ptrs),
           "specverify_run_contrastive_early_exit")


def specverify_run_greedy(ctx, stream, dtype, B, K, V, target_logits, proposals, accepted_len,
                          out_tokens) -> None:
    _check(load().specverify_run_greedy(
        ctx, _stream(stream), dtype, B, K, V,
        *_ptrs((target_logits, B * (K + 1) * V, dtype, "target_logits"),
               (proposals, B * K, "i32", "proposals"), (accepted_len, B, "i32", "accepted_len"),
               (out_tokens, B * (K + 1), "i32", "out_tokens"))), "specverify_run_greedy")


def specverify_run_greedy_early_exit(ctx, stream, dtype, B, K, V, target_logits, proposals,
                                     accepted_len, out_tokens) -> None:
    _check(load().specverify_run_greedy_early_exit(
        ctx, _stream(stream), dtype, B, K, V,
        *_ptrs((target_logits, B * (K + 1) * V, dtype, "target_logits"),
               (proposals, B * K, "i32", "proposals"), (accepted_len, B, "i32", "accepted_len"),
               (out_tokens, B * (K + 1), "i32", "out_tokens"))),
        "specverify_run_greedy_early_exit")


def specverify_sample(ctx, stream, dtype, N, V, temperature, logits, uniforms, out_tokens,
                      out_probs=None) -> None:
    _check(load().specverify_sample(
        ctx, _stream(stream), dtype, N, V, float(temperature),
        *_ptrs((logits, N * V, dtype, "logits"), (uniforms, N, "f32", "uniforms"),
               (out_tokens, N, "i32", "out_tokens"), (out_probs, N, "f32", "out_probs"))),
        "specverify_sample")


def specverify_run_greedy_heads(ctx, stream, dtype, B, K, H, V, logits, proposals, accepted_len,
                                out_tokens, next_proposals=None) -> None:
    _check(load().specverify_run_greedy_heads(
        ctx, _stream(stream), dtype, B, K, H, V,
        *_ptrs((logits, B * (K + 1) * max(H, 0) * V, dtype, "logits"),
               (proposals, B * K, "i32", "proposals"), (accepted_len, B, "i32", "accepted_len"),
               (out_tokens, B * (K + 1), "i32", "out_tokens"),
               (next_proposals, B * max(H - 1, 0), "i32", "next_proposals"))),
        "specverify_run_greedy_heads")


def specverify_quantile_cut(ctx, stream, P, N, alpha, scores, r_cut, keep, n_keep) -> None:
    _check(load().specverify_quantile_cut(
        ctx, _stream(stream), P, N, float(alpha),
        *_ptrs((scores, P * N, "f32", "scores"), (r_cut, P, "f32", "r_cut"),
               (keep, P * N, "u8", "keep"), (n_keep, P, "i32", "n_keep"))),
        "specverify_quantile_cut")


def _filter(f, count: int):
    if f is None:
        return None
    f.check(count)
    return ctypes.byref(f)


def specverify_sample_filtered(ctx, stream, dtype, N, V, row_stride, filter, logits, uniforms,
                               out_tokens, out_probs=None) -> None:
    """logits: a contiguous tensor, or an [N, V] tensor of unit column stride and row stride
    row_stride."""
    span = (N - 1) * row_stride + V if N > 0 else 0
    if hasattr(logits, "data_ptr") and not logits.is_contiguous():
        if logits.dim() != 2 or logits.stride() != (row_stride, 1) or logits.shape != (N, V):
            raise ValueError("logits: expected [%d, %d] with strides (%d, 1), got %s with strides %s"
                             % (N, V, row_stride, tuple(logits.shape), logits.stride()))
        _arr(logits, 0, dtype, "logits")
        if not logits.is_cuda:
            raise ValueError("expected a device tensor, got one on %s" % logits.device)
        x = logits.data_ptr()
    else:
        x, = _ptrs((logits, span, dtype, "logits"))
    _check(load().specverify_sample_filtered(
        ctx, _stream(stream), dtype, N, V, row_stride, _filter(filter, N), x,
        *_ptrs((uniforms, N, "f32", "uniforms"), (out_tokens, N, "i32", "out_tokens"),
               (out_probs, N, "f32", "out_probs"))), "specverify_sample_filtered")


def specverify_run_sampling_filtered(ctx, stream, dtype, B, K, V, target_filter, draft_filter,
                                     target_logits, draft_logits, draft_tokens, uniforms,
                                     accepted_len, out_tokens, out_probs=None) -> None:
    ptrs = _verify_args(dtype, B, K, V, target_logits, draft_logits, draft_tokens, uniforms,
                        accepted_len, out_tokens, out_probs, K)
    _check(load().specverify_run_sampling_filtered(ctx, _stream(stream), dtype, B, K, V,
                                                   _filter(target_filter, B),
                                                   _filter(draft_filter, B), *ptrs),
           "specverify_run_sampling_filtered")


_cache_pages = {}       # handle -> num_pages, which page maps are checked against


def specverify_cache_create(device, num_pages, page_tokens, num_seqs, max_blocks, page_bytes, pools,
                            refs, tables, blocks, lengths) -> int:
    """Returns the handle (an int).  pools: a sequence of device tensors (or addresses) of
    num_pages * page_bytes bytes each.  The caller keeps pools and state alive while the handle
    lives."""
    for p in pools:
        if hasattr(p, "data_ptr") and p.numel() * p.element_size() < num_pages * page_bytes:
            raise ValueError("pools: needs at least %d bytes, has %d"
                             % (num_pages * page_bytes, p.numel() * p.element_size()))
    state = _ptrs((refs, num_pages, "i32", "refs"), (tables, num_seqs * max_blocks, "i32", "tables"),
                  (blocks, num_seqs, "i32", "blocks"), (lengths, num_seqs, "i32", "lengths"))
    arr = (ctypes.c_void_p * max(len(pools), 1))(*(_ptr(p) for p in pools))
    h = ctypes.c_void_p()
    _check(load().specverify_cache_create(ctypes.byref(h), device, num_pages, page_tokens, num_seqs,
                                          max_blocks, len(pools), page_bytes, arr, *state),
           "specverify_cache_create")
    _cache_pages[h.value] = num_pages
    return h.value


def specverify_cache_workspace_bytes(cache: int) -> int:
    return int(load().specverify_cache_workspace_bytes(cache))


def specverify_cache_destroy(cache) -> None:
    _cache_pages.pop(cache, None)
    _check(load().specverify_cache_destroy(cache), "specverify_cache_destroy")


def _cache_call(name, cache, stream, n, *lists):
    _check(getattr(load(), name)(cache, _stream(stream), n, *_ptrs(*lists)), name)


def specverify_cache_reserve(cache, stream, n, seqs, counts, status=None) -> None:
    _cache_call("specverify_cache_reserve", cache, stream, n, (seqs, n, "i32", "seqs"),
                (counts, n, "i32", "counts"), (status, n, "i32", "status"))


def specverify_cache_commit(cache, stream, n, seqs, accepted_len, status=None) -> None:
    _cache_call("specverify_cache_commit", cache, stream, n, (seqs, n, "i32", "seqs"),
                (accepted_len, n, "i32", "accepted_len"), (status, n, "i32", "status"))


def specverify_cache_fork(cache, stream, n, parents, children, status=None) -> None:
    _cache_call("specverify_cache_fork", cache, stream, n, (parents, n, "i32", "parents"),
                (children, n, "i32", "children"), (status, n, "i32", "status"))


def specverify_cache_free(cache, stream, n, seqs=None, keep=None) -> None:
    _cache_call("specverify_cache_free", cache, stream, n, (seqs, n, "i32", "seqs"),
                (keep, n, "u8", "keep"))


def specverify_cache_compact(cache, stream, page_map=None, num_used=None) -> None:
    _check(load().specverify_cache_compact(cache, _stream(stream),
                                           *_ptrs((page_map, _cache_pages.get(cache, 0), "i32",
                                                   "page_map"),
                                                  (num_used, 1, "i32", "num_used"))),
           "specverify_cache_compact")


def specverify_cache_copy(cache, stream, n, src, dst, status=None) -> None:
    _cache_call("specverify_cache_copy", cache, stream, n, (src, n, "i32", "src"),
                (dst, n, "i32", "dst"), (status, n, "i32", "status"))


def specverify_run_greedy_tree(ctx, stream, dtype, B, T, V, depth, target_logits, tokens, parents,
                               counts, accepted_len, path, out_tokens) -> None:
    _check(load().specverify_run_greedy_tree(
        ctx, _stream(stream), dtype, B, T, V, depth,
        *_ptrs((target_logits, B * T * V, dtype, "target_logits"), (tokens, B * T, "i32", "tokens"),
               (parents, B * T, "i32", "parents"), (counts, B, "i32", "counts"),
               (accepted_len, B, "i32", "accepted_len"), (path, B * (depth + 1), "i32", "path"),
               (out_tokens, B * (depth + 1), "i32", "out_tokens"))), "specverify_run_greedy_tree")


def specverify_cache_keep_path(cache, stream, n, max_count, seqs, accepted_len, path,
                               status=None) -> None:
    _check(load().specverify_cache_keep_path(
        cache, _stream(stream), n, max_count,
        *_ptrs((seqs, n, "i32", "seqs"), (accepted_len, n, "i32", "accepted_len"),
               (path, n * max_count, "i32", "path"), (status, n, "i32", "status"))),
        "specverify_cache_keep_path")


_attn_shapes = {}       # handle -> (dtype, query row elements, key row elements, query heads)


def specverify_attn_create(cache, dtype, q_heads, kv_heads, head_dim, max_entries, max_nodes) -> int:
    """Returns the handle (an int).  The cache has to live while calls are made."""
    h = ctypes.c_void_p()
    _check(load().specverify_attn_create(ctypes.byref(h), cache, dtype, q_heads, kv_heads, head_dim,
                                         max_entries, max_nodes), "specverify_attn_create")
    _attn_shapes[h.value] = (dtype, q_heads * head_dim, kv_heads * head_dim, q_heads)
    return h.value


def specverify_attn_workspace_bytes(attn: int) -> int:
    return int(load().specverify_attn_workspace_bytes(attn))


def specverify_attn_destroy(attn) -> None:
    if _attn_shapes is not None:          # the module's names may be gone at the interpreter's end
        _attn_shapes.pop(attn, None)
    _check(load().specverify_attn_destroy(attn), "specverify_attn_destroy")


def _rows(x, dtype, rows, width, stride, name):
    """The pointer of a row array: `rows` rows of `width` elements, `stride` apart.  A tensor is
    contiguous, or its first dimension has that stride and the others lie side by side."""
    if x is None or isinstance(x, int) or not hasattr(x, "data_ptr"):
        return _ptr(x)
    if x.is_contiguous():
        return _ptrs((x, (rows - 1) * stride + width if rows > 0 else 0, dtype, name))[0]
    shape, steps, beside = x.shape, x.stride(), 1
    if (len(steps) == 2 and steps[1] == 1 and steps[0] == stride and shape[0] >= rows
            and shape[1] >= width and x.is_cuda and dtype in (0, 1)
            and x.dtype in (_KINDS or _kinds())[dtype][0]):
        return x.data_ptr()
    _arr(x, 0, dtype, name)
    for size, step in zip(shape[:0:-1], steps[:0:-1]):
        if size != 1 and step != beside:
            raise ValueError("%s: the elements of a row have to lie side by side" % name)
        beside *= size
    if len(shape) < 2 or shape[0] < rows or beside < width or (rows > 1 and steps[0] != stride):
        raise ValueError("%s: expected %d rows of %d elements, %d apart, got %s with strides %s"
                         % (name, rows, width, stride, tuple(x.shape), x.stride()))
    if not x.is_cuda:
        raise ValueError("expected a device tensor, got one on %s" % x.device)
    return x.data_ptr()


def _nodes(nodes, n, rows):
    if nodes is None:
        return None
    nodes.check(n, rows)
    return ctypes.byref(nodes)


def specverify_attn_append(attn, stream, key_pool, value_pool, n, max_count, rows, nodes, rotation,
                           keys, key_stride, values, value_stride, queries=None, query_stride=0,
                           rotated=None, rotated_stride=0, status=None) -> None:
    dtype, q, kv, _ = _attn_shapes.get(attn, (0, 0, 0, 0))
    status, = _ptrs((status, n, "i32", "status"))
    _check(load().specverify_attn_append(
        attn, _stream(stream), key_pool, value_pool, n, max_count, rows, _nodes(nodes, n, rows),
        None if rotation is None else ctypes.byref(rotation),
        _rows(keys, dtype, rows, kv, key_stride, "keys"), key_stride,
        _rows(values, dtype, rows, kv, value_stride, "values"), value_stride,
        _rows(queries, dtype, rows, q, query_stride, "queries"), query_stride,
        _rows(rotated, dtype, rows, q, rotated_stride, "rotated"), rotated_stride, status),
        "specverify_attn_append")


def specverify_attn_attend(attn, stream, key_pool, value_pool, n, max_count, rows, nodes, scale, window,
                           queries, query_stride, out, out_stride, lse=None, status=None) -> None:
    dtype, q, _, heads = _attn_shapes.get(attn, (0, 0, 0, 0))
    lse, status = _ptrs((lse, rows * heads, "f32", "lse"), (status, n, "i32", "status"))
    _check(load().specverify_attn_attend(
        attn, _stream(stream), key_pool, value_pool, n, max_count, rows, _nodes(nodes, n, rows),
        scale, window, _rows(queries, dtype, rows, q, query_stride, "queries"), query_stride,
        _rows(out, dtype, rows, q, out_stride, "out"), out_stride, lse, status),
        "specverify_attn_attend")


def specverify_set_test_flags(ctx, flags: int) -> None:
    """Test hook: SPECVERIFY_TEST_* bits forcing rarely reached draw paths (0 = normal)."""
    _check(load().specverify_set_test_flags(ctx, int(flags)), "specverify_set_test_flags")


def specverify_destroy(ctx) -> None:
    _check(load().specverify_destroy(ctx), "specverify_destroy")


def specverify_profile_begin(ctx, max_calls: int, kinds=None, stride: int = 1) -> None:
    """kinds: kernel names (from KERNEL_NAMES) to time, or None for all of them; stride: time
    every stride-th call (the first, then every stride-th after it)."""
    mask = 0
    for k in kinds or ():
        mask |= 1 << KERNEL_NAMES.index(k)
    _check(load().specverify_profile_begin(ctx, max_calls, mask, stride),
           "specverify_profile_begin")


def specverify_profile_launches(ctx, kind: str) -> list:
    """Durations in ms of the timed launches of kernel `kind` (a KERNEL_NAMES entry) since
    specverify_profile_begin, in call order."""
    lib = load()
    k = KERNEL_NAMES.index(kind)
    n = lib.specverify_profile_launches(ctx, k, None, 0)
    _check(min(n, 0), "specverify_profile_launches")
    ms = (ctypes.c_float * max(n, 1))()
    got = lib.specverify_profile_launches(ctx, k, ms, n)
    _check(min(got, 0), "specverify_profile_launches")
    return list(ms)[:min(n, got)]


def specverify_profile_end(ctx):
    """Returns ({kernel name: summed ms}, {kernel name: launches})."""
    ms = (ctypes.c_double * SPECVERIFY_NUM_KERNELS)()
    n = (ctypes.c_int * SPECVERIFY_NUM_KERNELS)()
    _check(load().specverify_profile_end(ctx, ms, n), "specverify_profile_end")
    return (dict(zip(KERNEL_NAMES, list(ms))), dict(zip(KERNEL_NAMES, list(n))))
