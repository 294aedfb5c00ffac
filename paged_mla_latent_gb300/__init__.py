"""Python binding of the GB300 paged latent-MLA decode library (argument marshalling only).

Every function here has the name of the C entry point it calls in
``include/paged_mla.h``; each converts torch tensors to ``mla_tensor_t`` descriptors
(pointer, dtype, shape, strides), through ctypes or, where calls take a few microseconds, in
a compiled module, and passes the current CUDA stream.  Calls run on the
device of their tensors, whichever one is current.  All arithmetic runs in the library's
CUDA kernels; there is no Python or CPU fallback: if the library cannot
be loaded, importing this package raises, and calls that go through the module raise
where it is missing.

The operation ("[Kimi-K3 MLA TP8] MLA performance", §2-§5; "Scaling Kimi K3 on AMD
Instinct MI355X", §1 and §4): absorbed MLA decode over a paged FP8 cache (one token a
page as captured, or pages of 2..1024 tokens with kv_indptr counting pages and
kv_last_page_lens the last page's fill), each query head scoring every 576-wide latent
row, softmax over the request's positions
(causal within draft tokens), 512-wide BF16 latent output plus optional FP32 lse, and the
softmax-weighted merge of split-KV or context-shard partials.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import struct

import torch

from . import build as _build

__all__ = [
    "MlaError", "mla_decode", "mla_decode_shared_prefix", "mla_decode_noalloc", "mla_merge_partials",
    "mla_validate", "mla_check_error", "mla_get_workspace_size", "mla_get_shared_prefix_workspace_size",
    "mla_status_string", "make_workspace", "library_path", "PreparedDecode", "mla_latent_to_v",
    "mla_selftest_bounded_wait", "mla_qk_rope_concat_and_cache", "mla_gqa_rope_and_cache",
    "mla_gqa_decode", "mla_get_gqa_decode_workspace_size", "make_gqa_decode_workspace",
    "mla_prompt_attention", "mla_get_prompt_workspace_size", "mla_build_page_table",
    "mla_gqa_block_append", "mla_gqa_block_gather", "mla_gqa_block_decode",
    "mla_get_gqa_block_decode_workspace_size", "make_gqa_block_decode_workspace",
]

MLA_DTYPE_FP8_E4M3FN = 1
MLA_DTYPE_BF16 = 2
MLA_DTYPE_FP32 = 3
MLA_DTYPE_INT32 = 4

STATUS_NAMES = {
    0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_UNSUPPORTED",
    3: "MLA_ERR_WORKSPACE_TOO_SMALL", 4: "MLA_ERR_CUDA", 5: "MLA_ERR_BAD_INDEX",
    6: "MLA_ERR_TIMEOUT", 7: "MLA_ERR_BAD_INPUT",
}


class MlaTensor(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("ndim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


class MlaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {STATUS_NAMES.get(self.status, self.status)}")


def _load() -> ctypes.CDLL:
    path = _build.build_library()   # no-op when the in-tree library is up to date
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER(MlaTensor)
    c_i32, c_sz, vp = ctypes.c_int32, ctypes.c_size_t, ctypes.c_void_p
    lib.mla_status_string.restype = ctypes.c_char_p
    lib.mla_status_string.argtypes = [ctypes.c_int]
    lib.mla_get_workspace_size.restype = ctypes.c_int
    lib.mla_get_workspace_size.argtypes = [c_i32, c_i32, c_i32, c_i32, c_i32, ctypes.POINTER(c_sz)]
    lib.mla_decode.restype = ctypes.c_int
    lib.mla_decode.argtypes = [P, P, P, P, P, P, P, c_i32, ctypes.c_float, P, P, c_i32, P, vp, c_sz, vp]
    lib.mla_get_shared_prefix_workspace_size.restype = ctypes.c_int
    lib.mla_get_shared_prefix_workspace_size.argtypes = [c_i32, c_i32, c_i32, c_i32, ctypes.POINTER(c_sz)]
    lib.mla_decode_shared_prefix.restype = ctypes.c_int
    lib.mla_decode_shared_prefix.argtypes = [P, P, P, P, P, P, P, c_i32, ctypes.c_float, P, P, c_i32, P,
                                             vp, c_sz, vp]
    lib.mla_decode_noalloc.restype = ctypes.c_int
    lib.mla_decode_noalloc.argtypes = [P, P, P, P, P, P, P, c_i32, ctypes.c_float, P, P, c_i32, P, vp, vp]
    lib.mla_merge_partials.restype = ctypes.c_int
    lib.mla_merge_partials.argtypes = [P, P, P, P, P, P, vp, vp]
    lib.mla_expand_shared_prefix_indices.restype = ctypes.c_int
    lib.mla_expand_shared_prefix_indices.argtypes = [P, P, P, P, P, vp, vp]
    lib.mla_validate.restype = ctypes.c_int
    lib.mla_validate.argtypes = [P, P, P, P, P, P, vp, c_sz, vp]
    lib.mla_check_error.restype = ctypes.c_int
    lib.mla_check_error.argtypes = [vp, c_sz, vp]
    lib.mla_latent_to_v.restype = ctypes.c_int
    lib.mla_latent_to_v.argtypes = [P, P, P, vp]
    lib.mla_qk_rope_concat_and_cache.restype = ctypes.c_int
    lib.mla_qk_rope_concat_and_cache.argtypes = [P, P, P, P, P, P, c_i32, P, P, P, P, P, vp, vp]
    lib.mla_gqa_rope_and_cache.restype = ctypes.c_int
    lib.mla_gqa_rope_and_cache.argtypes = [vp] * 5 + [c_i32] + [vp] * 9   # _packed() descriptors
    lib.mla_get_gqa_decode_workspace_size.restype = ctypes.c_int
    lib.mla_get_gqa_decode_workspace_size.argtypes = [c_i32, c_i32, c_i32, c_i32, c_i32,
                                                      ctypes.POINTER(c_sz)]
    lib.mla_gqa_decode.restype = ctypes.c_int
    lib.mla_gqa_decode.argtypes = [vp] * 7 + [ctypes.c_float] + [vp] * 4 + [c_sz, vp]
    lib.mla_prompt_attention.restype = ctypes.c_int
    lib.mla_prompt_attention.argtypes = [vp] * 6 + [ctypes.c_float] + [vp] * 3 + [c_sz, vp]
    lib.mla_get_prompt_workspace_size.restype = ctypes.c_int
    lib.mla_get_prompt_workspace_size.argtypes = [ctypes.c_int64, c_i32, c_i32, ctypes.POINTER(c_sz)]
    lib.mla_build_page_table.restype = ctypes.c_int
    lib.mla_build_page_table.argtypes = [vp] * 3 + [c_i32] + [vp] * 12
    lib.mla_gqa_block_append.restype = ctypes.c_int
    lib.mla_gqa_block_append.argtypes = [vp] * 5 + [c_i32] + [vp] * 12
    lib.mla_gqa_block_gather.restype = ctypes.c_int
    lib.mla_gqa_block_gather.argtypes = [vp] * 15
    lib.mla_get_gqa_block_decode_workspace_size.restype = ctypes.c_int
    lib.mla_get_gqa_block_decode_workspace_size.argtypes = [c_i32] * 5 + [ctypes.POINTER(c_sz)]
    lib.mla_gqa_block_decode.restype = ctypes.c_int
    lib.mla_gqa_block_decode.argtypes = [vp] * 10 + [c_i32, ctypes.c_float] + [vp] * 2 + [c_sz, vp]
    lib.mla_selftest_bounded_wait.restype = ctypes.c_int
    lib.mla_selftest_bounded_wait.argtypes = [vp, vp, ctypes.c_int64, vp]
    return lib


class _NoModule:
    """Stands for the call module where it cannot be loaded: the calls that need it raise."""

    def __init__(self, why):
        self._why = why

    def __getattr__(self, name):
        raise ImportError(f"{name} needs the call module {_build.NATIVE_PATH}: {self._why}")


def _load_native():
    """The module whose calls take torch tensors (built next to the library, which it links)."""
    try:
        spec = importlib.util.spec_from_file_location("pmla_native", _build.build_native())
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
    except (ImportError, OSError, RuntimeError) as e:
        return _NoModule(e)
    return module


_lib = _load()
_native = _load_native()


def library_path() -> str:
    return _build.LIB_PATH


_DTYPES = {
    torch.uint8: MLA_DTYPE_FP8_E4M3FN,           # raw e4m3fn codes
    torch.float8_e4m3fn: MLA_DTYPE_FP8_E4M3FN,
    torch.bfloat16: MLA_DTYPE_BF16,
    torch.float32: MLA_DTYPE_FP32,
    torch.int32: MLA_DTYPE_INT32,
}


_I64x4 = ctypes.c_int64 * 4
_PAD = ((), (0,), (0, 0), (0, 0, 0), (0, 0, 0, 0))


def _desc(t):
    """The mla_tensor_t of a torch tensor: pointer, dtype, shape and strides (elements)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    shape = t.shape
    n = len(shape)
    if n > 4:
        raise ValueError("at most 4 dimensions")
    try:
        code = _DTYPES[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}") from None
    pad = _PAD[4 - n]
    return MlaTensor(t.data_ptr() or None, n, code, _I64x4(*shape, *pad),
                     _I64x4(*t.stride(), *pad))


def _ref(d):
    return ctypes.byref(d) if d is not None else None


def _stream(stream, device):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


# the index of the current CUDA device, where the library launches and whose SMs it counts (a
# call's tensors may be on another; torch.cuda's own function checks its set-up each time)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(device, fn, *args):
    """A library call with CUDA device `device` (an index) as the current one."""
    if device < 0 or _current_device() == device:      # (CPU tensors: the library refuses them)
        return fn(*args)
    with torch.cuda.device(device):
        return fn(*args)


def _check(rc: int, where: str):
    if rc != 0:
        raise MlaError(rc, where)


def mla_status_string(status: int) -> str:
    return _lib.mla_status_string(int(status)).decode()


def mla_get_workspace_size(batch_size: int, num_heads: int, max_seqlen_q: int = 1,
                           num_kv_splits: int = 0, num_sms: int = 0) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.mla_get_workspace_size(batch_size, num_heads, max_seqlen_q, num_kv_splits,
                                       num_sms, ctypes.byref(out)), "mla_get_workspace_size")
    return int(out.value)


def mla_get_shared_prefix_workspace_size(batch_size: int, num_heads: int, max_seqlen_q: int = 1,
                                         num_sms: int = 0) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.mla_get_shared_prefix_workspace_size(batch_size, num_heads, max_seqlen_q, num_sms,
                                                     ctypes.byref(out)),
           "mla_get_shared_prefix_workspace_size")
    return int(out.value)


def make_workspace(batch_size: int, num_heads: int, max_seqlen_q: int = 1,
                   num_kv_splits: int = 0, device=None, shared_prefix: bool = False) -> torch.Tensor:
    """A zero-initialised device workspace large enough for such calls (shared_prefix:
    for mla_decode_shared_prefix)."""
    device = torch.device(device or "cuda")
    with torch.cuda.device(device):
        if shared_prefix:
            n = mla_get_shared_prefix_workspace_size(batch_size, num_heads, max_seqlen_q)
        else:
            n = mla_get_workspace_size(batch_size, num_heads, max_seqlen_q, num_kv_splits)
    return torch.zeros(n, dtype=torch.uint8, device=device)




def mla_decode(q, kv_buffer, o, qo_indptr, kv_indptr, kv_indices, kv_last_page_lens,
               max_seqlen_q, sm_scale, q_scale, kv_scale, num_kv_splits=0, lse_out=None,
               workspace=None, stream=None):
    """Enqueue one decode call (see include/paged_mla.h).  Returns the workspace used."""
    if workspace is None:
        workspace = make_workspace(len(kv_indptr) - 1, q.shape[1], max_seqlen_q,
                                   num_kv_splits, q.device)
    descs = [_desc(t) for t in (q, kv_buffer, o, qo_indptr, kv_indptr, kv_indices,
                                kv_last_page_lens, q_scale, kv_scale, lse_out)]
    dq, dkv, do, dqo, dkvp, didx, dlast, dqs, dks, dlse = descs
    rc = _call(
        q.get_device(), _lib.mla_decode,
        _ref(dq), _ref(dkv), _ref(do), _ref(dqo), _ref(dkvp), _ref(didx), _ref(dlast),
        int(max_seqlen_q), float(sm_scale), _ref(dqs), _ref(dks), int(num_kv_splits), _ref(dlse),
        ctypes.c_void_p(workspace.data_ptr()), workspace.numel() * workspace.element_size(),
        _stream(stream, q.device))
    _check(rc, "mla_decode")
    return workspace


def mla_decode_shared_prefix(q, kv_buffer, o, qo_indptr, kv_indptr, kv_indices,
                             kv_last_page_lens, max_seqlen_q, sm_scale, q_scale, kv_scale,
                             shared_prefix_len, lse_out=None, workspace=None, stream=None):
    """Decode a batch whose requests share their first shared_prefix_len cache positions
    (see include/paged_mla.h).  Returns the workspace used."""
    if workspace is None:
        workspace = make_workspace(len(kv_indptr) - 1, q.shape[1], max_seqlen_q, 0, q.device,
                                   shared_prefix=True)
    descs = [_desc(t) for t in (q, kv_buffer, o, qo_indptr, kv_indptr, kv_indices,
                                kv_last_page_lens, q_scale, kv_scale, lse_out)]
    dq, dkv, do, dqo, dkvp, didx, dlast, dqs, dks, dlse = descs
    rc = _call(
        q.get_device(), _lib.mla_decode_shared_prefix,
        _ref(dq), _ref(dkv), _ref(do), _ref(dqo), _ref(dkvp), _ref(didx), _ref(dlast),
        int(max_seqlen_q), float(sm_scale), _ref(dqs), _ref(dks), int(shared_prefix_len),
        _ref(dlse), ctypes.c_void_p(workspace.data_ptr()),
        workspace.numel() * workspace.element_size(), _stream(stream, q.device))
    _check(rc, "mla_decode_shared_prefix")
    return workspace


class PreparedDecode:
    """One mla_decode (or, with shared_prefix_len, mla_decode_shared_prefix) call whose
    argument descriptors are built once, for a caller that runs the same buffers every step
    (fresh data in the same tensors).  run() enqueues the call through the C ABI with no
    per-call argument marshalling.  The descriptors hold the tensors' addresses, shapes and
    strides as they were here: prepare again after reallocating or reshaping any of them.
    The object keeps the tensors alive.
    """

    def __init__(self, q, kv_buffer, o, qo_indptr, kv_indptr, kv_indices, kv_last_page_lens,
                 max_seqlen_q, sm_scale, q_scale, kv_scale, num_kv_splits=0, lse_out=None,
                 workspace=None, shared_prefix_len=None, stream=None, compact_page_table=None):
        """compact_page_table: optional (shared_indices, own_indptr, own_indices) device
        tensors; run() then first rebuilds kv_indptr / kv_indices from them with
        mla_expand_shared_prefix_indices (a caller that uploads its page table every step
        sends the shared pages once).  The expansion's device-side errors (an own_indptr
        that is not monotone, a table longer than kv_indices) go to the workspace's error
        word, where mla_check_error reports them with the decode's own."""
        shared = shared_prefix_len is not None
        if workspace is None:
            workspace = make_workspace(len(kv_indptr) - 1, q.shape[1], max_seqlen_q,
                                       0 if shared else num_kv_splits, q.device,
                                       shared_prefix=shared)
        self.workspace = workspace
        self._keep = (q, kv_buffer, o, qo_indptr, kv_indptr, kv_indices, kv_last_page_lens,
                      q_scale, kv_scale, lse_out, workspace)
        self._descs = [_desc(t) for t in self._keep[:10]]
        r = [_ref(d) for d in self._descs]
        tail = (ctypes.c_void_p(workspace.data_ptr()),
                ctypes.c_size_t(workspace.numel() * workspace.element_size()))
        if shared:
            self._fn, self._where = _lib.mla_decode_shared_prefix, "mla_decode_shared_prefix"
            self._args = (r[0], r[1], r[2], r[3], r[4], r[5], r[6], int(max_seqlen_q),
                          float(sm_scale), r[7], r[8], int(shared_prefix_len), r[9]) + tail
        else:
            self._fn, self._where = _lib.mla_decode, "mla_decode"
            self._args = (r[0], r[1], r[2], r[3], r[4], r[5], r[6], int(max_seqlen_q),
                          float(sm_scale), r[7], r[8], int(num_kv_splits), r[9]) + tail
        self._device, self._index = q.device, q.get_device()
        self._stream = None if stream is None else _stream(stream, q.device)
        self._expand = None
        if compact_page_table is not None:
            sh, optr, own = compact_page_table
            self._expand_keep = (sh, optr, own)
            self._expand_descs = [_desc(t) for t in (sh, optr, own)] + self._descs[4:6]
            self._expand = tuple(_ref(d) for d in self._expand_descs) + (
                ctypes.c_void_p(workspace.data_ptr()),)

    def run(self, stream=None):
        """Enqueue the call on `stream` (default: the stream given when prepared, else
        torch's current stream)."""
        st = _stream(stream, self._device) if stream is not None else (
            self._stream if self._stream is not None else _stream(None, self._device))
        if self._expand is not None:
            rc = _call(self._index, _lib.mla_expand_shared_prefix_indices, *self._expand, st)
            if rc != 0:
                raise MlaError(rc, "mla_expand_shared_prefix_indices")
        rc = _call(self._index, self._fn, *self._args, st)
        if rc != 0:
            raise MlaError(rc, self._where)
        return self.workspace


def mla_decode_noalloc(q, kv_buffer, o, qo_indptr, kv_indptr, kv_indices, kv_last_page_lens,
                       max_seqlen_q, sm_scale, q_scale, kv_scale, num_kv_splits=0, lse_out=None,
                       error_out=None, stream=None):
    """Decode without a workspace: scratch lives in the library's fixed device array.

    For callers that cannot allocate device memory.  error_out: optional int32 device
    tensor receiving the call's raw device error bits.  Raises MlaError on a host-side
    error, including MLA_ERR_WORKSPACE_TOO_SMALL when the call needs more scratch than
    the fixed array holds.
    """
    descs = [_desc(t) for t in (q, kv_buffer, o, qo_indptr, kv_indptr, kv_indices,
                                kv_last_page_lens, q_scale, kv_scale, lse_out)]
    dq, dkv, do, dqo, dkvp, didx, dlast, dqs, dks, dlse = descs
    if error_out is not None:
        # the library copies 4 bytes device-to-device into it after the decode is queued
        if not isinstance(error_out, torch.Tensor) or error_out.dtype != torch.int32 or \
                error_out.numel() < 1 or error_out.device != q.device:
            raise ValueError("error_out must be an int32 tensor of at least one element on "
                             f"{q.device}")
    ew = ctypes.c_void_p(error_out.data_ptr()) if error_out is not None else None
    rc = _call(
        q.get_device(), _lib.mla_decode_noalloc,
        _ref(dq), _ref(dkv), _ref(do), _ref(dqo), _ref(dkvp), _ref(didx), _ref(dlast),
        int(max_seqlen_q), float(sm_scale), _ref(dqs), _ref(dks), int(num_kv_splits), _ref(dlse),
        ew, _stream(stream, q.device))
    _check(rc, "mla_decode_noalloc")


def mla_expand_shared_prefix_indices(shared_indices, own_indptr, own_indices, kv_indptr,
                                     kv_indices, error_word=None, stream=None):
    """Build the full page table of a shared-prefix batch on the device from the shared page
    ids (once) and each request's own ids (see include/paged_mla.h)."""
    descs = [_desc(t) for t in (shared_indices, own_indptr, own_indices, kv_indptr, kv_indices)]
    if error_word is not None and (not isinstance(error_word, torch.Tensor) or
                                   error_word.dtype != torch.int32 or error_word.numel() < 1 or
                                   error_word.device != kv_indices.device):
        raise ValueError("error_word must be an int32 tensor on the page table's device")
    ew = ctypes.c_void_p(error_word.data_ptr()) if error_word is not None else None
    rc = _call(kv_indices.get_device(), _lib.mla_expand_shared_prefix_indices,
               *[_ref(d) for d in descs], ew, _stream(stream, kv_indices.device))
    _check(rc, "mla_expand_shared_prefix_indices")


def mla_merge_partials(o_parts, lse_parts, reduce_indptr, reduce_idx, o, lse_out=None,
                       error_word=None, stream=None):
    """Softmax-weighted merge of partials with a CSR reduce map (see include/paged_mla.h)."""
    descs = [_desc(t) for t in (o_parts, lse_parts, reduce_indptr, reduce_idx, o, lse_out)]
    ew = ctypes.c_void_p(error_word.data_ptr()) if error_word is not None else None
    rc = _call(o.get_device(), _lib.mla_merge_partials, *[_ref(d) for d in descs], ew,
               _stream(stream, o.device))
    _check(rc, "mla_merge_partials")


def mla_latent_to_v(o, w_uv, v, stream=None):
    """v[t, h, :] = o[t, h, :] @ w_uv[h]: the latent o mapped to v_head_dim (see
    include/paged_mla.h)."""
    descs = [_desc(t) for t in (o, w_uv, v)]
    rc = _call(v.get_device(), _lib.mla_latent_to_v, *[_ref(d) for d in descs],
               _stream(stream, v.device))
    _check(rc, "mla_latent_to_v")


def mla_qk_rope_concat_and_cache(q_nope, q_pe, kv_c, k_pe, positions, cos_sin, is_neox,
                                 slot_mapping, q_scale, kv_scale, q_out, kv_buffer,
                                 error_word, stream=None):
    """Rotate q's and the new keys' rope columns, quantise q to the decode's fp8 q_out and
    write each token's new 576-wide entry into kv_buffer at its slot (see
    include/paged_mla.h).  error_word: an int32 device tensor (>= 1 element)."""
    if not isinstance(error_word, torch.Tensor) or error_word.dtype != torch.int32 or \
            error_word.numel() < 1 or error_word.device != q_out.device:
        raise ValueError(f"error_word must be an int32 tensor on {q_out.device}")
    descs = [_desc(t) for t in (q_nope, q_pe, kv_c, k_pe, positions, cos_sin)]
    tail = [_desc(t) for t in (slot_mapping, q_scale, kv_scale, q_out, kv_buffer)]
    rc = _call(q_out.get_device(), _lib.mla_qk_rope_concat_and_cache,
               *[_ref(d) for d in descs], int(is_neox), *[_ref(d) for d in tail],
               ctypes.c_void_p(error_word.data_ptr()), _stream(stream, q_out.device))
    _check(rc, "mla_qk_rope_concat_and_cache")


# mla_tensor_t by number of dimensions: pointer, ndim and dtype as one word, shape[4], stride[4]
_FORMS = tuple(
    (struct.Struct(f"<QQ{n}q{8 * (4 - n)}x{n}q{8 * (4 - n)}x").pack,
     {dtype: n | code << 32 for dtype, code in _DTYPES.items()}) for n in range(5))


def _packed(t, device):
    """The mla_tensor_t of a torch tensor on CUDA device `device` (an index) as bytes, whose
    buffer ctypes passes as the pointer: an eighth of the time of filling the ctypes
    structure, which one-shot calls of a few microseconds notice."""
    if t is None:
        return None
    try:
        if t.get_device() == device:
            shape = t.shape
            pack, words = _FORMS[len(shape)]
            return pack(t.data_ptr(), words[t.dtype], *shape, *t.stride())
    except (AttributeError, IndexError, KeyError):
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if t.get_device() != device:
        raise ValueError(f"expected a tensor on CUDA device {device}, got one on {t.device}")
    if t.dim() > 4:
        raise ValueError("at most 4 dimensions")
    raise TypeError(f"unsupported dtype {t.dtype}")


def _cuda_index(t):
    """The CUDA device index of the tensor that says where a call runs."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    return t.get_device()


def _raw_stream(stream, device):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _error_word(error_word, device):
    if not isinstance(error_word, torch.Tensor) or error_word.dtype is not torch.int32 or \
            error_word.get_device() != device or error_word.numel() < 1:
        raise ValueError(f"error_word must be an int32 tensor on CUDA device {device}")
    return error_word.data_ptr()


def mla_gqa_rope_and_cache(q, k, v, positions, cos_sin, is_neox, slot_mapping, q_out, k_cache,
                           v_cache, error_word, k_scale=None, v_scale=None, k_out=None,
                           stream=None):
    """Rotate q's and the new keys' first cos_sin.shape[1] columns and write each token's keys
    and values into the per-head caches at its slot (see include/paged_mla.h).  q_out and
    k_out may be q and k; k_scale and v_scale belong to e4m3 caches.  error_word: an int32
    device tensor (>= 1 element)."""
    d = _cuda_index(q)
    if d != _current_device():
        with torch.cuda.device(d):
            return mla_gqa_rope_and_cache(q, k, v, positions, cos_sin, is_neox, slot_mapping, q_out,
                                          k_cache, v_cache, error_word, k_scale, v_scale, k_out,
                                          stream)
    ew = _error_word(error_word, d)
    rc = _lib.mla_gqa_rope_and_cache(
        _packed(q, d), _packed(k, d), _packed(v, d), _packed(positions, d), _packed(cos_sin, d),
        int(is_neox), _packed(slot_mapping, d), _packed(k_scale, d), _packed(v_scale, d),
        _packed(q_out, d), _packed(k_out, d), _packed(k_cache, d), _packed(v_cache, d), ew,
        _raw_stream(stream, d))
    _check(rc, "mla_gqa_rope_and_cache")


def mla_get_gqa_decode_workspace_size(batch_size: int, num_heads: int, num_kv_heads: int,
                                      head_dim: int, num_sms: int = 0) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.mla_get_gqa_decode_workspace_size(batch_size, num_heads, num_kv_heads, head_dim,
                                                  num_sms, ctypes.byref(out)),
           "mla_get_gqa_decode_workspace_size")
    return int(out.value)


def make_gqa_decode_workspace(batch_size: int, num_heads: int, num_kv_heads: int, head_dim: int,
                              device=None) -> torch.Tensor:
    """A zero-initialised device workspace for mla_gqa_decode calls of this shape."""
    device = torch.device(device or "cuda")
    with torch.cuda.device(device):
        n = mla_get_gqa_decode_workspace_size(batch_size, num_heads, num_kv_heads, head_dim)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def mla_gqa_decode(q, k_cache, v_cache, o, kv_indptr, kv_indices, kv_last_page_lens, sm_scale,
                   k_scale=None, v_scale=None, lse_out=None, workspace=None, stream=None):
    """Attention of one new token a request over paged per-head caches (see
    include/paged_mla.h).  Returns the workspace used."""
    d = _cuda_index(q)
    if d != _current_device():
        with torch.cuda.device(d):
            return mla_gqa_decode(q, k_cache, v_cache, o, kv_indptr, kv_indices, kv_last_page_lens,
                                  sm_scale, k_scale, v_scale, lse_out, workspace, stream)
    if workspace is None:
        with _on_stream(stream, q.device):      # made and zeroed on the stream that uses it
            workspace = make_gqa_decode_workspace(q.shape[0], q.shape[1], k_cache.shape[2],
                                                  q.shape[2], q.device)
    elif workspace.get_device() != d:
        raise ValueError(f"the workspace must be on CUDA device {d}")
    rc = _lib.mla_gqa_decode(
        _packed(q, d), _packed(k_cache, d), _packed(v_cache, d), _packed(o, d),
        _packed(kv_indptr, d), _packed(kv_indices, d), _packed(kv_last_page_lens, d),
        float(sm_scale), _packed(k_scale, d), _packed(v_scale, d), _packed(lse_out, d),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _raw_stream(stream, d))
    _check(rc, "mla_gqa_decode")
    return workspace


def mla_get_prompt_workspace_size(n_keys: int, v_head_dim: int, num_sms: int = 0) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.mla_get_prompt_workspace_size(n_keys, v_head_dim, num_sms, ctypes.byref(out)),
           "mla_get_prompt_workspace_size")
    return int(out.value)


def _on_stream(stream, device):
    """A context whose allocations belong to the stream a call runs on."""
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return torch.cuda.stream(stream)
    return torch.cuda.stream(torch.cuda.ExternalStream(int(stream), device=device))


def mla_prompt_attention(q, k, v, o, qo_indptr, kv_indptr, sm_scale, error_word, lse_out=None,
                         workspace=None, stream=None):
    """Causal attention of packed whole prompts (see include/paged_mla.h).  error_word: an
    int32 device tensor (>= 1 element).  workspace: a device tensor of
    mla_get_prompt_workspace_size bytes; without one the call takes it from torch's allocator
    on the call's stream (up to 40 MB; nothing where no request can be long enough to be cut
    between SMs)."""
    d = _cuda_index(q)
    if d != _current_device():
        with torch.cuda.device(d):
            return mla_prompt_attention(q, k, v, o, qo_indptr, kv_indptr, sm_scale, error_word, lse_out,
                                        workspace, stream)
    ew = _error_word(error_word, d)
    if workspace is None:
        n = mla_get_prompt_workspace_size(k.shape[0], v.shape[-1])
        if n and stream is None:
            workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
        elif n:
            with _on_stream(stream, q.device):
                workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    elif workspace.get_device() != d:
        raise ValueError(f"the workspace must be on CUDA device {d}")
    ws, n = (workspace.data_ptr(), workspace.numel() * workspace.element_size()) \
        if workspace is not None else (None, 0)
    rc = _lib.mla_prompt_attention(
        _packed(q, d), _packed(k, d), _packed(v, d), _packed(o, d), _packed(qo_indptr, d),
        _packed(kv_indptr, d), float(sm_scale), _packed(lse_out, d), ew, ws, n,
        _raw_stream(stream, d))
    _check(rc, "mla_prompt_attention")


def mla_build_page_table(seq_lens, new_lens, block_table, page_size, qo_indptr, key_indptr, kv_indptr,
                         kv_indices, kv_last_page_lens, error_word, positions=None, slot_mapping=None,
                         free_pages=None, free_count=None, free_count_out=None, stream=None):
    """Build a step's page lists, positions and cache slots on the device from the requests'
    lengths, taking pages for the new tokens from a stack of free ones (see
    include/paged_mla.h).  error_word: an int32 device tensor of two elements, zero before its
    first use.  free_count_out may be free_count."""
    d = _cuda_index(seq_lens)
    if d != _current_device():
        with torch.cuda.device(d):
            return mla_build_page_table(seq_lens, new_lens, block_table, page_size, qo_indptr,
                                        key_indptr, kv_indptr, kv_indices, kv_last_page_lens,
                                        error_word, positions, slot_mapping, free_pages, free_count,
                                        free_count_out, stream)
    if not isinstance(error_word, torch.Tensor) or error_word.numel() < 2:
        raise ValueError("error_word must be an int32 tensor of two elements")
    rc = _native.mla_build_page_table(
        d, seq_lens, new_lens, block_table, page_size, free_pages, free_count, free_count_out, qo_indptr,
        key_indptr, kv_indptr, kv_indices, kv_last_page_lens, positions, slot_mapping, error_word,
        _raw_stream(stream, d))
    _check(rc, "mla_build_page_table")


def mla_gqa_block_append(q, k, v, positions, cos_sin, is_neox, qo_indptr, kv_indptr, kv_indices,
                         kv_last_page_lens, q_out, k_cache, v_cache, k_scale, v_scale, error_word,
                         k_out=None, stream=None):
    """Rotate q's and the new keys' first cos_sin.shape[1] columns and write each request's new
    keys and values behind its cached ones, into e4m3 caches with a scale for each block and
    head (see include/paged_mla.h).  q_out and k_out may be q and k.  error_word: an int32
    device tensor (>= 1 element)."""
    d = _cuda_index(q)
    if d != _current_device():
        with torch.cuda.device(d):
            return mla_gqa_block_append(q, k, v, positions, cos_sin, is_neox, qo_indptr, kv_indptr,
                                        kv_indices, kv_last_page_lens, q_out, k_cache, v_cache,
                                        k_scale, v_scale, error_word, k_out, stream)
    rc = _native.mla_gqa_block_append(
        d, q, k, v, positions, cos_sin, is_neox, qo_indptr, kv_indptr, kv_indices, kv_last_page_lens,
        q_out, k_out, k_cache, v_cache, k_scale, v_scale, error_word, _raw_stream(stream, d))
    _check(rc, "mla_gqa_block_append")


def mla_gqa_block_gather(k_cache, v_cache, k_scale, v_scale, kv_indptr, kv_indices, kv_last_page_lens,
                         row_indptr, k_rows, v_rows, error_word, qo_indptr=None, k_new=None,
                         v_new=None, stream=None):
    """Requests' cached keys and values (and the step's own behind them) as packed bf16 rows for
    mla_prompt_attention (see include/paged_mla.h).  error_word: an int32 device tensor (>= 1
    element)."""
    d = _cuda_index(k_cache)
    if d != _current_device():
        with torch.cuda.device(d):
            return mla_gqa_block_gather(k_cache, v_cache, k_scale, v_scale, kv_indptr, kv_indices,
                                        kv_last_page_lens, row_indptr, k_rows, v_rows, error_word,
                                        qo_indptr, k_new, v_new, stream)
    rc = _native.mla_gqa_block_gather(
        d, k_cache, v_cache, k_scale, v_scale, kv_indptr, kv_indices, kv_last_page_lens, row_indptr,
        qo_indptr, k_new, v_new, k_rows, v_rows, error_word, _raw_stream(stream, d))
    _check(rc, "mla_gqa_block_gather")


def mla_get_gqa_block_decode_workspace_size(num_heads: int, num_kv_heads: int, head_dim: int,
                                            max_seqlen_q: int = 1, num_sms: int = 0) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.mla_get_gqa_block_decode_workspace_size(num_heads, num_kv_heads, head_dim, max_seqlen_q,
                                                        num_sms, ctypes.byref(out)),
           "mla_get_gqa_block_decode_workspace_size")
    return int(out.value)


def make_gqa_block_decode_workspace(num_heads: int, num_kv_heads: int, head_dim: int,
                                    max_seqlen_q: int = 1, device=None) -> torch.Tensor:
    """A zero-initialised device workspace for mla_gqa_block_decode calls of this shape."""
    device = torch.device(device or "cuda")
    with torch.cuda.device(device):
        n = mla_get_gqa_block_decode_workspace_size(num_heads, num_kv_heads, head_dim, max_seqlen_q)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def mla_gqa_block_decode(q, k_cache, v_cache, k_scale, v_scale, o, qo_indptr, kv_indptr, kv_indices,
                         kv_last_page_lens, max_seqlen_q, sm_scale, lse_out=None, workspace=None,
                         stream=None):
    """Attention of each request's newest tokens over paged e4m3 caches with a scale for each
    block and head (see include/paged_mla.h).  Returns the workspace used."""
    d = _cuda_index(q)
    if d != _current_device():
        with torch.cuda.device(d):
            return mla_gqa_block_decode(q, k_cache, v_cache, k_scale, v_scale, o, qo_indptr, kv_indptr,
                                        kv_indices, kv_last_page_lens, max_seqlen_q, sm_scale, lse_out,
                                        workspace, stream)
    if workspace is None:
        with _on_stream(stream, q.device):      # made and zeroed on the stream that uses it
            workspace = make_gqa_block_decode_workspace(q.shape[1], k_cache.shape[2], q.shape[2],
                                                        max_seqlen_q, q.device)
    elif workspace.get_device() != d or not workspace.is_contiguous():
        raise ValueError(f"the workspace must be a contiguous tensor on CUDA device {d}")
    rc = _native.mla_gqa_block_decode(
        d, q, k_cache, v_cache, k_scale, v_scale, o, qo_indptr, kv_indptr, kv_indices, kv_last_page_lens,
        max_seqlen_q, sm_scale, lse_out, workspace.data_ptr(), workspace.nbytes, _raw_stream(stream, d))
    _check(rc, "mla_gqa_block_decode")
    return workspace


def mla_selftest_bounded_wait(error_word, result, limit_ns, stream=None):
    """Run the library's bounded mbarrier wait on a barrier nothing arrives at (see
    include/paged_mla.h): error_word (1) and result (3) are int32 device tensors."""
    for t, n in ((error_word, 1), (result, 3)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.numel() < n or \
                not t.is_cuda:
            raise ValueError(f"expected an int32 CUDA tensor of at least {n} element(s)")
    rc = _call(result.get_device(), _lib.mla_selftest_bounded_wait,
               ctypes.c_void_p(error_word.data_ptr()), ctypes.c_void_p(result.data_ptr()),
               int(limit_ns), _stream(stream, result.device))
    _check(rc, "mla_selftest_bounded_wait")


def mla_validate(q, kv_buffer, qo_indptr, kv_indptr, kv_indices, kv_last_page_lens,
                 workspace, stream=None) -> int:
    """Device-side check of the index inputs; returns the status code (synchronises)."""
    descs = [_desc(t) for t in (q, kv_buffer, qo_indptr, kv_indptr, kv_indices, kv_last_page_lens)]
    return int(_call(q.get_device(), _lib.mla_validate, *[_ref(d) for d in descs],
                     ctypes.c_void_p(workspace.data_ptr()), workspace.numel(),
                     _stream(stream, q.device)))


def mla_check_error(workspace, stream=None) -> int:
    """First device-side error recorded in the workspace since the last check (clears it)."""
    return int(_call(workspace.get_device(), _lib.mla_check_error,
                     ctypes.c_void_p(workspace.data_ptr()), workspace.numel(),
                     _stream(stream, workspace.device)))
