"""ctypes binding of libmla_tree.so: same names as the C ABI, argument
marshalling only (torch tensors -> device pointers, the current stream).
Every step of the verify path runs in the library's kernels; when the
library is missing this module raises instead of computing anything."""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch

from . import build as _build

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libmla_tree.so")

MT_OK, MT_EINVAL, MT_EUNSUPPORTED, MT_EWORKSPACE, MT_ECUDA = 0, -1, -2, -3, -4
DEV_BAD_SLOT, DEV_BAD_PARENT, DEV_BAD_INDPTR, DEV_TREE_TOO_BIG, DEV_TIMEOUT = 1, 2, 4, 8, 16
DEV_MISMATCH, DEV_BAD_POSITION, DEV_BAD_TOKEN, DEV_NO_PAGES = 32, 64, 128, 256
PATH_AUTO, PATH_SIMT, PATH_TC = 0, 1, 2

EXPORTS = ["mla_tree_abi_version", "mla_tree_status_string", "mla_tree_draft_kv_scatter",
           "mla_tree_kv_indices_build", "tree_mask_pack", "tree_mask_pack_bits", "mla_tree_prepare",
           "mla_tree_verify_workspace_bytes", "mla_tree_verify_launch_count", "mla_tree_verify",
           "mla_tree_verify_bits", "mla_tree_verify_masked", "mla_tree_verify_validate_workspace_bytes",
           "mla_tree_verify_validate", "mla_tree_verify_noalloc", "mla_tree_test_wait_limits",
           "mla_paged_append", "mla_paged_decode_workspace_bytes", "mla_paged_decode",
           "mla_paged_decode_window", "mla_token_logprobs", "mla_tree_accept", "mla_paged_compact",
           "mla_pages_fork", "mla_pages_fit_workspace_bytes", "mla_pages_fit", "mla_pages_fit_lens",
           "mla_paged_copy"]
MT_ESCRATCH = -5
NOALLOC_SCRATCH_BYTES = 64 << 20

_lib = None
P = ctypes.c_void_p
I32, I64, SZ, F32 = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float


class MlaTreeError(RuntimeError):
    pass


def load():
    """Load the library once; fail loudly if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise MlaTreeError("libmla_tree.so is not built (%s); run __graft_entry__.build()" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    lib.mla_tree_abi_version.restype = I32
    lib.mla_tree_status_string.restype = ctypes.c_char_p
    lib.mla_tree_status_string.argtypes = [I32]
    lib.mla_tree_draft_kv_scatter.restype = I32
    lib.mla_tree_draft_kv_scatter.argtypes = [P, I64, P, I32, P, I64, P, P]
    lib.mla_tree_kv_indices_build.restype = I32
    lib.mla_tree_kv_indices_build.argtypes = [P, I64, P, P, P, I32, I32, P, I64, P, P, P]
    lib.tree_mask_pack.restype = I32
    lib.tree_mask_pack.argtypes = [P, P, P, I32, I32, P, P, I64, P, P]
    lib.tree_mask_pack_bits.restype = I32
    lib.tree_mask_pack_bits.argtypes = [P, P, P, I32, I32, P, P, I64, P, P]
    lib.mla_tree_prepare.restype = I32
    lib.mla_tree_prepare.argtypes = [P, I64, P, P, I64, P, P, P, I32, I32, P, I64, P, I64, P, P, P, I64,
                                     P, P]
    lib.mla_tree_verify_workspace_bytes.restype = SZ
    lib.mla_tree_verify_workspace_bytes.argtypes = [I32, I32, I32, I32]
    lib.mla_tree_verify_launch_count.restype = I32
    lib.mla_tree_verify_launch_count.argtypes = [I32, I32, I32, I64, I32, I32]
    lib.mla_tree_verify.restype = I32
    lib.mla_tree_verify.argtypes = [P, P, I64, P, I64, P, P, P, I64, P, I32, I32, I32, F32,
                                    P, P, P, SZ, I32, I32, P, P]
    lib.mla_tree_verify_bits.restype = I32
    lib.mla_tree_verify_bits.argtypes = [P, P, I64, P, I64, P, P, P, I64, P, I32, I32, I32, F32,
                                         P, P, P, SZ, I32, I32, P, P]
    lib.mla_tree_verify_masked.restype = I32
    lib.mla_tree_verify_masked.argtypes = [P, P, I64, P, I64, P, P, P, I64, P, I32, I32, I32, I32, F32,
                                           P, P, P, SZ, I32, I32, P, P]
    lib.mla_tree_verify_validate_workspace_bytes.restype = SZ
    lib.mla_tree_verify_validate_workspace_bytes.argtypes = [I32, I32, I32, I32]
    lib.mla_tree_verify_validate.restype = I32
    lib.mla_tree_verify_validate.argtypes = [P, P, I64, P, I64, P, P, P, I64, P, I32, I32, I32, F32,
                                             P, P, P, SZ, I32, F32, P, P, P]
    lib.mla_tree_test_wait_limits.restype = I32
    lib.mla_tree_test_wait_limits.argtypes = [I32, I64]
    lib.mla_tree_verify_noalloc.restype = I32
    lib.mla_tree_verify_noalloc.argtypes = [P, P, I64, P, I64, P, P, P, I64, P, I32, I32, I32, F32,
                                            P, P, I32, I32, P, P]
    lib.mla_paged_append.restype = I32
    lib.mla_paged_append.argtypes = [P, I64, P, I64, P, F32, P, I64, I64, P, I64, I64, I32, P, I64, I32,
                                     P, P, P, I32, I32, P, I64, I32, P, I64, I64, I32, P, P]
    lib.mla_paged_decode_workspace_bytes.restype = SZ
    lib.mla_paged_decode_workspace_bytes.argtypes = [I32, I32]
    lib.mla_paged_decode.restype = I32
    lib.mla_paged_decode.argtypes = [P, I64, I64, P, I64, I64, I32, P, I64, I32, P, I32, I32, F32,
                                     P, P, P, SZ, P, P]
    lib.mla_paged_decode_window.restype = I32
    lib.mla_paged_decode_window.argtypes = [P, I64, I64, P, I64, I64, I32, P, I64, I32, P, I32, I32, I32, I32, F32,
                                            P, P, P, SZ, P, P]
    lib.mla_token_logprobs.restype = I32
    lib.mla_token_logprobs.argtypes = [P, I32, I64, I32, I32, P, I64, I32, I32, P, P, P, P, P, P, P]
    lib.mla_tree_accept.restype = I32
    lib.mla_tree_accept.argtypes = [P, P, P, I64, P, P, P, I32, I32, I32, P, P, P, P, P, P]
    lib.mla_paged_compact.restype = I32
    lib.mla_paged_compact.argtypes = [P, I64, I32, P, P, I32, P, I64, I32, P, I64, I64, I32, I32, I64, P, P]
    lib.mla_pages_fork.restype = I32
    lib.mla_pages_fork.argtypes = [P, P, P, P, I64, I32, I32, P, I64, P, P, P, I64, I32, P, P]
    lib.mla_pages_fit_workspace_bytes.restype = SZ
    lib.mla_pages_fit_workspace_bytes.argtypes = [I32, I64]
    lib.mla_pages_fit.restype = I32
    lib.mla_pages_fit.argtypes = [P, P, P, P, I64, I32, I32, P, I64, I32, I32, I32, P, P, SZ, P, P]
    lib.mla_pages_fit_lens.restype = I32
    lib.mla_pages_fit_lens.argtypes = [P, P, P, P, I64, I32, I32, P, I64, I32, I32, I32, P, P, P, SZ, P, P]
    lib.mla_paged_copy.restype = I32
    lib.mla_paged_copy.argtypes = [P, I64, P, I64, I64, I32, I32, I64, P, P]
    _lib = lib
    return lib


def _check(rc, what):
    if rc != MT_OK:
        msg = load().mla_tree_status_string(rc).decode()
        raise MlaTreeError("%s failed: %d (%s)" % (what, rc, msg))


def _ptr(t, dtype=None, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise MlaTreeError("%s must be a CUDA tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise MlaTreeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise MlaTreeError("%s must be contiguous" % name)
    return t.data_ptr() if t.numel() else None


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def abi_version():
    return load().mla_tree_abi_version()


def mla_tree_draft_kv_scatter(src, out_cache_loc, kv_buf, status=None, stream=None):
    """kv_buf[out_cache_loc[t]] = src[t] for every draft token t."""
    if src.dim() != 2 or src.stride(1) != 1 or src.dtype != torch.bfloat16 or not src.is_cuda:
        raise MlaTreeError("src must be a CUDA bf16 [T, >=576] tensor with unit column stride")
    rc = load().mla_tree_draft_kv_scatter(src.data_ptr() if src.numel() else None, src.stride(0),
                                          _ptr(out_cache_loc, torch.int32, "out_cache_loc"),
                                          out_cache_loc.numel(), _ptr(kv_buf, torch.bfloat16, "kv_buf"),
                                          kv_buf.shape[0], _ptr(status, torch.int32, "status"),
                                          _stream(stream))
    _check(rc, "mla_tree_draft_kv_scatter")


def mla_tree_kv_indices_build(prefix_indices, prefix_indptr, out_cache_loc, qo_indptr,
                              kv_indices, kv_indptr, status=None, stream=None):
    """kv_indices = per request, prefix slots followed by draft slots."""
    batch = qo_indptr.numel() - 1
    rc = load().mla_tree_kv_indices_build(
        _ptr(prefix_indices, torch.int32, "prefix_indices"), prefix_indices.numel(),
        _ptr(prefix_indptr, torch.int32, "prefix_indptr"),
        _ptr(out_cache_loc, torch.int32, "out_cache_loc"), _ptr(qo_indptr, torch.int32, "qo_indptr"),
        batch, out_cache_loc.numel(), _ptr(kv_indices, torch.int32, "kv_indices"), kv_indices.numel(),
        _ptr(kv_indptr, torch.int32, "kv_indptr"), _ptr(status, torch.int32, "status"), _stream(stream))
    _check(rc, "mla_tree_kv_indices_build")


def tree_mask_pack(parents, qo_indptr, kv_indptr, mask_indptr, packed_mask, status=None, stream=None):
    """Ancestor-or-self tree mask, row stride prefix + draft, flat per request."""
    batch = qo_indptr.numel() - 1
    rc = load().tree_mask_pack(
        _ptr(parents, torch.int32, "parents"), _ptr(qo_indptr, torch.int32, "qo_indptr"),
        _ptr(kv_indptr, torch.int32, "kv_indptr"), batch, parents.numel(),
        _ptr(mask_indptr, torch.int64, "mask_indptr"), _ptr(packed_mask, torch.uint8, "packed_mask"),
        packed_mask.numel(), _ptr(status, torch.int32, "status"), _stream(stream))
    _check(rc, "tree_mask_pack")


def tree_mask_pack_bits(parents, qo_indptr, kv_indptr, mask_word_indptr, mask_words, status=None,
                        stream=None):
    """The same tree mask, one bit per (row, column): rows of ceil(L/32) uint32 words."""
    batch = qo_indptr.numel() - 1
    rc = load().tree_mask_pack_bits(
        _ptr(parents, torch.int32, "parents"), _ptr(qo_indptr, torch.int32, "qo_indptr"),
        _ptr(kv_indptr, torch.int32, "kv_indptr"), batch, parents.numel(),
        _ptr(mask_word_indptr, torch.int64, "mask_word_indptr"),
        _ptr(mask_words, torch.int32, "mask_words"), mask_words.numel(),
        _ptr(status, torch.int32, "status"), _stream(stream))
    _check(rc, "tree_mask_pack_bits")


def mla_tree_prepare(draft_kv, out_cache_loc, prefix_indices, prefix_indptr, qo_indptr, parents,
                     kv_buf, kv_indices, kv_indptr, mask_word_indptr, mask_words, status=None,
                     stream=None):
    """Draft-KV scatter, KV index marshaling and bit-form mask packing in one launch."""
    if (draft_kv.dim() != 2 or draft_kv.stride(1) != 1 or draft_kv.dtype != torch.bfloat16
            or not draft_kv.is_cuda):
        raise MlaTreeError("draft_kv must be a CUDA bf16 [T, >=576] tensor with unit column stride")
    batch = qo_indptr.numel() - 1
    rc = load().mla_tree_prepare(
        draft_kv.data_ptr() if draft_kv.numel() else None, draft_kv.stride(0),
        _ptr(out_cache_loc, torch.int32, "out_cache_loc"),
        _ptr(prefix_indices, torch.int32, "prefix_indices"), prefix_indices.numel(),
        _ptr(prefix_indptr, torch.int32, "prefix_indptr"), _ptr(qo_indptr, torch.int32, "qo_indptr"),
        _ptr(parents, torch.int32, "parents"), batch, out_cache_loc.numel(),
        _ptr(kv_buf, torch.bfloat16, "kv_buf"), kv_buf.shape[0],
        _ptr(kv_indices, torch.int32, "kv_indices"), kv_indices.numel(),
        _ptr(kv_indptr, torch.int32, "kv_indptr"),
        _ptr(mask_word_indptr, torch.int64, "mask_word_indptr"),
        _ptr(mask_words, torch.int32, "mask_words"), mask_words.numel(),
        _ptr(status, torch.int32, "status"), _stream(stream))
    _check(rc, "mla_tree_prepare")


def mla_tree_test_wait_limits(drop_item=-1, wait_limit_ns=0):
    """Test facility: bound every wait of the tensor-core kernel by
    wait_limit_ns (0 = the default) and make its copy engines issue nothing
    from work item drop_item on (-1 = off). Process-wide."""
    _check(load().mla_tree_test_wait_limits(int(drop_item), int(wait_limit_ns)),
           "mla_tree_test_wait_limits")


def mla_tree_verify_workspace_bytes(batch, total_q, heads, max_splits=0):
    return int(load().mla_tree_verify_workspace_bytes(batch, total_q, heads, max_splits))


def mla_tree_verify_launch_count(batch, total_q, heads, kv_indices_len, max_splits=0, path=PATH_AUTO):
    return int(load().mla_tree_verify_launch_count(batch, total_q, heads, kv_indices_len, max_splits, path))


def mla_tree_verify(q, kv_buf, kv_indices, kv_indptr, qo_indptr, packed_mask, mask_indptr,
                    sm_scale, out, lse, workspace, max_splits=0, path=PATH_AUTO, status=None,
                    stream=None):
    """Tree-verify attention: out [T, H, 512] bf16 and lse [T, H] fp32."""
    if q.dim() != 3 or q.shape[2] != 576:
        raise MlaTreeError("q must be [total_q, heads, 576]")
    total_q, heads = q.shape[0], q.shape[1]
    batch = qo_indptr.numel() - 1
    rc = load().mla_tree_verify(
        _ptr(q, torch.bfloat16, "q"), _ptr(kv_buf, torch.bfloat16, "kv_buf"), kv_buf.shape[0],
        _ptr(kv_indices, torch.int32, "kv_indices"), kv_indices.numel(),
        _ptr(kv_indptr, torch.int32, "kv_indptr"), _ptr(qo_indptr, torch.int32, "qo_indptr"),
        _ptr(packed_mask, torch.uint8, "packed_mask"), packed_mask.numel(),
        _ptr(mask_indptr, torch.int64, "mask_indptr"), batch, total_q, heads, float(sm_scale),
        _ptr(out, torch.bfloat16, "out"), _ptr(lse, torch.float32, "lse"),
        _ptr(workspace, torch.uint8, "workspace"), workspace.numel(), max_splits, path,
        _ptr(status, torch.int32, "status"), _stream(stream))
    _check(rc, "mla_tree_verify")


def mla_tree_verify_bits(q, kv_buf, kv_indices, kv_indptr, qo_indptr, mask_words, mask_word_indptr,
                         sm_scale, out, lse, workspace, max_splits=0, path=PATH_AUTO, status=None,
                         stream=None):
    """mla_tree_verify with the mask in the bit form of tree_mask_pack_bits
    (mask_words: int32 tensor holding the uint32 words)."""
    if q.dim() != 3 or q.shape[2] != 576:
        raise MlaTreeError("q must be [total_q, heads, 576]")
    total_q, heads = q.shape[0], q.shape[1]
    batch = qo_indptr.numel() - 1
    rc = load().mla_tree_verify_bits(
        _ptr(q, torch.bfloat16, "q"), _ptr(kv_buf, torch.bfloat16, "kv_buf"), kv_buf.shape[0],
        _ptr(kv_indices, torch.int32, "kv_indices"), kv_indices.numel(),
        _ptr(kv_indptr, torch.int32, "kv_indptr"), _ptr(qo_indptr, torch.int32, "qo_indptr"),
        _ptr(mask_words, torch.int32, "mask_words"), mask_words.numel(),
        _ptr(mask_word_indptr, torch.int64, "mask_word_indptr"), batch, total_q, heads,
        float(sm_scale), _ptr(out, torch.bfloat16, "out"), _ptr(lse, torch.float32, "lse"),
        _ptr(workspace, torch.uint8, "workspace"), workspace.numel(), max_splits, path,
        _ptr(status, torch.int32, "status"), _stream(stream))
    _check(rc, "mla_tree_verify_bits")


MASK_BITS = 1         # the mask is in the bit form (int32 tensor of uint32 words)
MASK_SKIP_PREFIX = 2  # prefix columns visible, their mask entries unread


def mla_tree_verify_masked(q, kv_buf, kv_indices, kv_indptr, qo_indptr, mask, mask_indptr,
                           mask_flags, sm_scale, out, lse, workspace, max_splits=0, path=PATH_AUTO,
                           status=None, stream=None):
    """mla_tree_verify with the mask form and options as flags (MASK_BITS,
    MASK_SKIP_PREFIX): mask is a uint8 byte mask, or int32 words with
    MASK_BITS."""
    if q.dim() != 3 or q.shape[2] != 576:
        raise MlaTreeError("q must be [total_q, heads, 576]")
    total_q, heads = q.shape[0], q.shape[1]
    batch = qo_indptr.numel() - 1
    mdt = torch.int32 if mask_flags & MASK_BITS else torch.uint8
    rc = load().mla_tree_verify_masked(
        _ptr(q, torch.bfloat16, "q"), _ptr(kv_buf, torch.bfloat16, "kv_buf"), kv_buf.shape[0],
        _ptr(kv_indices, torch.int32, "kv_indices"), kv_indices.numel(),
        _ptr(kv_indptr, torch.int32, "kv_indptr"), _ptr(qo_indptr, torch.int32, "qo_indptr"),
        _ptr(mask, mdt, "mask"), mask.numel(), _ptr(mask_indptr, torch.int64, "mask_indptr"),
        int(mask_flags), batch, total_q, heads, float(sm_scale), _ptr(out, torch.bfloat16, "out"),
        _ptr(lse, torch.float32, "lse"), _ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
        max_splits, path, _ptr(status, torch.int32, "status"), _stream(stream))
    _check(rc, "mla_tree_verify_masked")


def mla_tree_verify_validate_workspace_bytes(batch, total_q, heads, max_splits=0):
    return int(load().mla_tree_verify_validate_workspace_bytes(batch, total_q, heads, max_splits))


def mla_tree_verify_validate(q, kv_buf, kv_indices, kv_indptr, qo_indptr, packed_mask, mask_indptr,
                             sm_scale, out, lse, workspace, diff, tolerance=1e-2, max_splits=0,
                             status=None, stream=None):
    """Validate mode: the call computed by both kernels; out/lse get the
    tensor-core result, diff (fp32 [2] on the device) the max-abs output and
    max relative LSE differences, status MT_DEV_MISMATCH beyond tolerance."""
    if q.dim() != 3 or q.shape[2] != 576:
        raise MlaTreeError("q must be [total_q, heads, 576]")
    total_q, heads = q.shape[0], q.shape[1]
    batch = qo_indptr.numel() - 1
    rc = load().mla_tree_verify_validate(
        _ptr(q, torch.bfloat16, "q"), _ptr(kv_buf, torch.bfloat16, "kv_buf"), kv_buf.shape[0],
        _ptr(kv_indices, torch.int32, "kv_indices"), kv_indices.numel(),
        _ptr(kv_indptr, torch.int32, "kv_indptr"), _ptr(qo_indptr, torch.int32, "qo_indptr"),
        _ptr(packed_mask, torch.uint8, "packed_mask"), packed_mask.numel(),
        _ptr(mask_indptr, torch.int64, "mask_indptr"), batch, total_q, heads, float(sm_scale),
        _ptr(out, torch.bfloat16, "out"), _ptr(lse, torch.float32, "lse"),
        _ptr(workspace, torch.uint8, "workspace"), workspace.numel(), max_splits, float(tolerance),
        _ptr(diff, torch.float32, "diff"), _ptr(status, torch.int32, "status"), _stream(stream))
    _check(rc, "mla_tree_verify_validate")


def mla_tree_verify_noalloc(q, kv_buf, kv_indices, kv_indptr, qo_indptr, packed_mask, mask_indptr,
                            sm_scale, out, lse, max_splits=0, path=PATH_AUTO, status=None,
                            stream=None):
    """mla_tree_verify for callers that cannot allocate: the split scratch is
    the library's built-in static device buffer instead of a workspace."""
    if q.dim() != 3 or q.shape[2] != 576:
        raise MlaTreeError("q must be [total_q, heads, 576]")
    total_q, heads = q.shape[0], q.shape[1]
    batch = qo_indptr.numel() - 1
    rc = load().mla_tree_verify_noalloc(
        _ptr(q, torch.bfloat16, "q"), _ptr(kv_buf, torch.bfloat16, "kv_buf"), kv_buf.shape[0],
        _ptr(kv_indices, torch.int32, "kv_indices"), kv_indices.numel(),
        _ptr(kv_indptr, torch.int32, "kv_indptr"), _ptr(qo_indptr, torch.int32, "qo_indptr"),
        _ptr(packed_mask, torch.uint8, "packed_mask"), packed_mask.numel(),
        _ptr(mask_indptr, torch.int64, "mask_indptr"), batch, total_q, heads, float(sm_scale),
        _ptr(out, torch.bfloat16, "out"), _ptr(lse, torch.float32, "lse"), max_splits, path,
        _ptr(status, torch.int32, "status"), _stream(stream))
    _check(rc, "mla_tree_verify_noalloc")


ROPE_PAIRS, ROPE_HALVES = 0, 1

# The calls of a decoding loop run once per token or layer, where their own time shows: a
# compiled module (csrc/paged_call.cpp) checks the tensors and calls the
# library. What does not fit comes back as None and goes through the checks
# here, one by one, for its message.
_paged_call = None


def _load_paged_call():
    global _paged_call
    lib = load()
    path = _build.call_path()
    if not os.path.exists(path):
        raise MlaTreeError("the module for this torch and Python is not built (%s); run __graft_entry__.build()" % path)
    spec = importlib.util.spec_from_file_location("_paged_call", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.bind(*(ctypes.cast(f, P).value for f in (
        lib.mla_paged_append, lib.mla_paged_decode, lib.mla_paged_decode_window, lib.mla_token_logprobs, lib.mla_tree_accept,
        lib.mla_paged_compact, lib.mla_pages_fork, lib.mla_pages_fit_lens, lib.mla_paged_copy)))
    _paged_call = mod
    return mod


def _refuse(name, t, dtype, dim, dev, shape=None, whole=False, other="cache", any_stride=False):
    """Raises what is wrong with one tensor, if anything is."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise MlaTreeError("%s must be a CUDA tensor" % name)
    want = "%s must be %s" % (name, dtype)
    if t.dtype != dtype:
        raise MlaTreeError("%s, got %s" % (want, t.dtype))
    if dev is not None and t.get_device() != dev:
        raise MlaTreeError("%s is on %s, the %s on cuda:%d" % (name, t.device, other, dev))
    if t.dim() != dim or shape is not None and tuple(t.shape) != tuple(shape):
        raise MlaTreeError("%s %s, got %s" % (want, "of %d dimensions" % dim if shape is None else list(shape),
                                              list(t.shape)))
    if whole and not t.is_contiguous():
        raise MlaTreeError("%s must be contiguous" % name)
    if dim and t.shape[-1] > 1 and t.stride(-1) != 1 and not any_stride:
        raise MlaTreeError("%s must have unit stride in its last dimension" % name)


def _refuse_paged(cache, block_table, kv_lens):
    _refuse("cache", cache, torch.bfloat16, 3, None)
    dev = cache.get_device()
    if cache.shape[1] < 1 or cache.shape[2] != 576 or cache.shape[1] > 1 and cache.stride(1) != 576:
        raise MlaTreeError("cache must be [num_pages, page_size, 576] with a page's rows one after another")
    _refuse("block_table", block_table, torch.int32, 2, dev)
    _refuse("kv_lens", kv_lens, torch.int32, 1, dev, (block_table.shape[0],), True)
    return dev


def _refuse_append(latent, k_rope, qo_indptr, kv_lens, block_table, cache, rope_table, q_rope, q_out, positions,
                   norm_weight, status):
    dev = _refuse_paged(cache, block_table, kv_lens)
    bf16, i32 = torch.bfloat16, torch.int32
    _refuse("latent", latent, bf16, 2, dev)
    t = latent.shape[0]
    _refuse("latent", latent, bf16, 2, dev, (t, 512))
    _refuse("k_rope", k_rope, bf16, 2, dev, (t, 64))
    if qo_indptr is not None:
        _refuse("qo_indptr", qo_indptr, i32, 1, dev, (block_table.shape[0] + 1,), True)
    elif t != block_table.shape[0]:
        raise MlaTreeError("without qo_indptr every request has one token: %d tokens, %d requests"
                           % (t, block_table.shape[0]))
    _refuse("rope_table", rope_table, torch.float32, 2, dev)
    _refuse("rope_table", rope_table, torch.float32, 2, dev, (rope_table.shape[0], 64), True)
    if (q_rope is None) != (q_out is None):
        raise MlaTreeError("q_rope and q_out go together")
    if q_rope is not None:
        _refuse("q_rope", q_rope, bf16, 3, dev)
        _refuse("q_rope", q_rope, bf16, 3, dev, (t, q_rope.shape[1], 64))
        _refuse("q_out", q_out, bf16, 3, dev, q_rope.shape)
    if positions is not None:
        _refuse("positions", positions, i32, 1, dev, (t,), True)
    if norm_weight is not None:
        _refuse("norm_weight", norm_weight, bf16, 1, dev, (512,), True)
    if status is not None:
        _refuse("status", status, i32, status.dim() if isinstance(status, torch.Tensor) else 1, dev, None, True)
    raise MlaTreeError("unsupported arguments")


def _refuse_decode(q, cache, block_table, kv_lens, out, lse, workspace, status):
    dev = _refuse_paged(cache, block_table, kv_lens)
    _refuse("q", q, torch.bfloat16, 3, dev)
    batch, heads = block_table.shape[0], q.shape[1]
    _refuse("q", q, torch.bfloat16, 3, dev, (batch, heads, 576))
    _refuse("out", out, torch.bfloat16, 3, dev, (batch, heads, 512), True)
    _refuse("lse", lse, torch.float32, 2, dev, (batch, heads), True)
    _refuse("workspace", workspace, torch.uint8, 1, dev, None, True)
    if status is not None:
        _refuse("status", status, torch.int32, status.dim() if isinstance(status, torch.Tensor) else 1, dev, None, True)
    raise MlaTreeError("unsupported arguments")


def mla_paged_append(latent, k_rope, qo_indptr, kv_lens, block_table, cache, rope_table, q_rope=None,
                     q_out=None, positions=None, norm_weight=None, norm_eps=1e-6,
                     rope_style=ROPE_PAIRS, status=None, stream=None):
    """Append new tokens to a paged latent cache [num_pages, page_size, 576]:
    latent [T, 512] (RMS-normalised where norm_weight is given) and k_rope
    [T, 64] rotated to its position, at position kv_lens[b] - n_b + i of
    request b's pages block_table[b]; and q_out = q_rope [T, H, 64] rotated
    alike (q_out may be q_rope). rope_table: fp32 [positions, 64], cos | sin.
    qo_indptr None: token b is request b's only one, and left out with its
    query where kv_lens[b] is 0 (a slot of a fixed batch that holds no request).
    Runs on the cache's device, on stream or that device's current one."""
    rc = (_paged_call or _load_paged_call()).append(
        latent, k_rope, qo_indptr, kv_lens, block_table, cache, rope_table, q_rope, q_out, positions, norm_weight,
        norm_eps, rope_style, status, None if stream is None else stream.cuda_stream)
    if rc is None:
        _refuse_append(latent, k_rope, qo_indptr, kv_lens, block_table, cache, rope_table, q_rope, q_out, positions,
                       norm_weight, status)
    if rc != MT_OK:
        _check(rc, "mla_paged_append")


def mla_paged_decode_workspace_bytes(batch, heads):
    return int(load().mla_paged_decode_workspace_bytes(batch, heads))


def mla_paged_decode(q, cache, block_table, kv_lens, sm_scale, out, lse, workspace, status=None,
                     stream=None):
    """Attention of one new token per request over a paged latent cache: q
    [B, H, 576] over the first kv_lens[b] positions of request b's pages;
    out [B, H, 512] bf16 and lse [B, H] fp32. workspace: uint8, at least
    mla_paged_decode_workspace_bytes(B, H). Runs on the cache's device, on
    stream or that device's current one."""
    rc = (_paged_call or _load_paged_call()).decode(
        q, cache, block_table, kv_lens, sm_scale, out, lse, workspace, status,
        None if stream is None else stream.cuda_stream)
    if rc is None:
        _refuse_decode(q, cache, block_table, kv_lens, out, lse, workspace, status)
    if rc != MT_OK:
        _check(rc, "mla_paged_decode")


def mla_paged_decode_window(q, cache, block_table, kv_lens, window, sinks, sm_scale, out, lse, workspace, status=None,
                            stream=None):
    """mla_paged_decode where request b sees its last ``window`` positions and
    its first ``sinks`` alone. Table entries of pages that hold none of them are
    not read."""
    rc = (_paged_call or _load_paged_call()).decode_window(
        q, cache, block_table, kv_lens, window, sinks, sm_scale, out, lse, workspace, status,
        None if stream is None else stream.cuda_stream)
    if rc is None:
        _refuse_int("window", window)
        _refuse_int("sinks", sinks)
        _refuse_decode(q, cache, block_table, kv_lens, out, lse, workspace, status)
    if rc != MT_OK:
        _check(rc, "mla_paged_decode_window")


def _refuse_int(name, v):
    if not isinstance(v, int) or not -(1 << 31) <= v < 1 << 31:
        raise MlaTreeError("%s must be a 32-bit int, got %r" % (name, v))


def _refuse_status(status, dev, other):
    if status is not None:
        _refuse("status", status, torch.int32, status.dim() if isinstance(status, torch.Tensor) else 1, dev, None, True, other)
    raise MlaTreeError("unsupported arguments")


def _refuse_logprobs(logits, tokens, logprobs, lse, entropy, top_ids, top_logprobs, status):
    types = (torch.bfloat16, torch.float16, torch.float32)
    if isinstance(logits, torch.Tensor) and logits.dtype not in types:
        raise MlaTreeError("logits must be bf16, fp16 or fp32, got %s" % logits.dtype)
    _refuse("logits", logits, getattr(logits, "dtype", None), 2, None)
    dev, rows, on = logits.get_device(), logits.shape[0], "logits"
    if logits.shape[1] < 1:
        raise MlaTreeError("logits must have a vocabulary, got %s" % list(logits.shape))
    if (tokens is None) != (logprobs is None):
        raise MlaTreeError("tokens and logprobs go together")
    if tokens is not None:
        dim = 2 if isinstance(tokens, torch.Tensor) and tokens.dim() == 2 else 1
        _refuse("tokens", tokens, torch.int32, dim, dev, None, False, on, dim == 1)
        if tokens.shape[0] != rows:
            raise MlaTreeError("tokens must have the logits' %d rows, got %s" % (rows, list(tokens.shape)))
        _refuse("logprobs", logprobs, torch.float32, dim, dev, tokens.shape, True, on)
    for name, v in (("lse", lse), ("entropy", entropy)):
        if v is not None:
            _refuse(name, v, torch.float32, 1, dev, (rows,), True, on)
    if top_ids is None and top_logprobs is not None:
        raise MlaTreeError("top_logprobs needs top_ids")
    if top_ids is not None:
        _refuse("top_ids", top_ids, torch.int32, 2, dev, None, True, on)
        _refuse("top_ids", top_ids, torch.int32, 2, dev, (rows, top_ids.shape[1]), True, on)
        if top_logprobs is not None:
            _refuse("top_logprobs", top_logprobs, torch.float32, 2, dev, top_ids.shape, True, on)
    _refuse_status(status, dev, on)


def mla_token_logprobs(logits, tokens=None, logprobs=None, lse=None, entropy=None, top_ids=None, top_logprobs=None,
                       status=None, stream=None):
    """Rows of logits [T, V] (bf16, fp16 or fp32; any row stride): the log
    probabilities of tokens [T] or [T, G] (-1: none), the rows' log sums of exp
    and entropies [T], and their k <= 32 most likely tokens, top_ids [T, k] and
    top_logprobs, equal ones by the lower token. What is None is left out. Runs
    on the logits' device, on stream or that device's current one."""
    rc = (_paged_call or _load_paged_call()).logprobs(
        logits, tokens, logprobs, lse, entropy, top_ids, top_logprobs, status,
        None if stream is None else stream.cuda_stream)
    if rc is None:
        _refuse_logprobs(logits, tokens, logprobs, lse, entropy, top_ids, top_logprobs, status)
    if rc != MT_OK:
        _check(rc, "mla_token_logprobs")


def _refuse_accept(parents, tokens, targets, qo_indptr, kv_lens, path, counts, next_tokens, new_lens, first, status):
    i32, on = torch.int32, "parents"
    _refuse("parents", parents, i32, 1, None, None, True)
    dev, t = parents.get_device(), parents.shape[0]
    _refuse("path", path, i32, 2, dev, None, True, on)
    batch = path.shape[0]
    _refuse("tokens", tokens, i32, 1, dev, (t,), True, on)
    _refuse("targets", targets, i32, 1, dev, (t,), False, on, True)
    _refuse("qo_indptr", qo_indptr, i32, 1, dev, (batch + 1,), True, on)
    for name, v in (("kv_lens", kv_lens), ("counts", counts), ("next_tokens", next_tokens), ("new_lens", new_lens)):
        _refuse(name, v, i32, 1, dev, (batch,), True, on)
    if first is not None:
        _refuse("first", first, i32, 1, dev, (batch,), True, on)
    _refuse_status(status, dev, on)


def mla_tree_accept(parents, tokens, targets, qo_indptr, kv_lens, path, counts, next_tokens, new_lens, first=None,
                    status=None, stream=None):
    """Walks request b's draft tree (nodes qo_indptr[b] .., parents as for
    tree_mask_pack) along the tokens that the model chose: from the prefix, the
    lowest child whose tokens entry is wanted, then its targets entry is wanted.
    path [B, most] gets the nodes taken (-1 behind), counts [B] how many,
    next_tokens [B] the token to go on with, new_lens [B] kv_lens without the
    nodes that were not taken (new_lens may be kv_lens). targets may have any
    stride (a column of top_ids); first [B] is what the prefix wants, None the
    token of each request's node 0."""
    rc = (_paged_call or _load_paged_call()).accept(
        parents, tokens, targets, qo_indptr, kv_lens, path, counts, next_tokens, new_lens, first, status,
        None if stream is None else stream.cuda_stream)
    if rc is None:
        _refuse_accept(parents, tokens, targets, qo_indptr, kv_lens, path, counts, next_tokens, new_lens, first, status)
    if rc != MT_OK:
        _check(rc, "mla_tree_accept")


def _refuse_layers(cache):
    dim = 4 if isinstance(cache, torch.Tensor) and cache.dim() == 4 else 3
    _refuse("cache", cache, torch.bfloat16, dim, None)
    if cache.shape[-2] < 1 or cache.shape[-1] != 576 or cache.shape[-2] > 1 and cache.stride(-2) != 576:
        raise MlaTreeError("cache must be [num_pages, page_size, 576] or [layers, num_pages, page_size, 576] "
                           "with a page's rows one after another")
    return cache.get_device()


def _refuse_compact(path, counts, kv_lens, block_table, cache, status):
    dev = _refuse_layers(cache)
    _refuse("block_table", block_table, torch.int32, 2, dev)
    batch = block_table.shape[0]
    _refuse("path", path, torch.int32, 2, dev)
    _refuse("path", path, torch.int32, 2, dev, (batch, path.shape[1]))
    _refuse("counts", counts, torch.int32, 1, dev, (batch,), True)
    _refuse("kv_lens", kv_lens, torch.int32, 1, dev, (batch,), True)
    _refuse_status(status, dev, "cache")


def mla_paged_compact(path, counts, kv_lens, block_table, cache, status=None, stream=None):
    """Moves the rows of the nodes that mla_tree_accept took up behind the
    prefix, in a cache [num_pages, page_size, 576] or, for all layers at once,
    [layers, num_pages, page_size, 576]: position base + path[b, k] to base + k,
    base = kv_lens[b] - counts[b] (kv_lens: the new lengths)."""
    rc = (_paged_call or _load_paged_call()).compact(path, counts, kv_lens, block_table, cache, status,
                                                     None if stream is None else stream.cuda_stream)
    if rc is None:
        _refuse_compact(path, counts, kv_lens, block_table, cache, status)
    if rc != MT_OK:
        _check(rc, "mla_paged_compact")


def _refuse_rows(table, refs, names):
    _refuse("refs", refs, torch.int32, 1, None, None, True)
    dev, on = refs.get_device(), "refs"
    for name, v in zip(names, table):
        _refuse(name, v, torch.int32, 2, dev, None, False, on)
    return dev


def _refuse_fork(parents, kv_lens, held, block_table, refs, new_lens, new_held, new_table, status):
    i32, on = torch.int32, "refs"
    dev = _refuse_rows((block_table, new_table), refs, ("block_table", "new_table"))
    old, rows = block_table.shape[0], new_table.shape[0]
    _refuse("new_table", new_table, i32, 2, dev, (rows, block_table.shape[1]), False, on)
    for name, v, n in (("parents", parents, rows), ("kv_lens", kv_lens, old), ("held", held, old),
                       ("new_lens", new_lens, rows), ("new_held", new_held, rows)):
        _refuse(name, v, i32, 1, dev, (n,), True, on)
    _refuse_status(status, dev, on)


def mla_pages_fork(parents, kv_lens, held, block_table, refs, new_lens, new_held, new_table, status=None, stream=None):
    """Row r of new_table shares the pages of row parents[r] of block_table
    (-1: none), with its kv_lens and held; rows that are nobody's parent give
    their pages back. refs [num_pages] counts the holders of each page. The new
    tensors are others than the old ones."""
    rc = (_paged_call or _load_paged_call()).fork(parents, kv_lens, held, block_table, refs, new_lens, new_held, new_table,
                                                  status, None if stream is None else stream.cuda_stream)
    if rc is None:
        _refuse_fork(parents, kv_lens, held, block_table, refs, new_lens, new_held, new_table, status)
    if rc != MT_OK:
        _check(rc, "mla_pages_fork")


def _refuse_fit(kv_lens, want_lens, held, block_table, refs, page_size, copies, workspace, window, sinks, status, step_lens):
    i32, on = torch.int32, "refs"
    for name, v in (("page_size", page_size), ("window", window), ("sinks", sinks)):
        _refuse_int(name, v)
    dev = _refuse_rows((block_table,), refs, ("block_table",))
    batch = block_table.shape[0]
    for name, v in (("kv_lens", kv_lens), ("want_lens", want_lens), ("held", held)):
        _refuse(name, v, i32, 1, dev, (batch,), True, on)
    _refuse("copies", copies, i32, 2, dev, (batch, 3), True, on)
    _refuse("workspace", workspace, torch.uint8, 1, dev, None, True, on)
    if step_lens is not None:
        _refuse("step_lens", step_lens, i32, 1, dev, (batch,), True, on)
    _refuse_status(status, dev, on)


def mla_pages_fit_workspace_bytes(batch, num_pages):
    return int(load().mla_pages_fit_workspace_bytes(batch, num_pages))


def mla_pages_fit(kv_lens, want_lens, held, block_table, refs, page_size, copies, workspace, window=0, sinks=0,
                  status=None, stream=None, step_lens=None):
    """Gives each request pages of its own for positions kv_lens .. want_lens -
    1 and takes back those behind want_lens and, with a window, those that lie
    wholly between the first sinks positions and the window of position kv_lens.
    copies [B, 3] gets (source page, destination page, rows) where a shared page
    was replaced, for mla_paged_copy. Without enough free pages DEV_NO_PAGES is
    set and nothing changes: no position behind kv_lens may be written then.
    step_lens [B] says so to the calls that follow: want_lens, or 0 for a request
    that may not be written to. workspace: uint8, mla_pages_fit_workspace_bytes(B,
    num_pages)."""
    rc = (_paged_call or _load_paged_call()).fit(kv_lens, want_lens, held, block_table, refs, page_size, copies, workspace,
                                                 window, sinks, status, None if stream is None else stream.cuda_stream, step_lens)
    if rc is None:
        _refuse_fit(kv_lens, want_lens, held, block_table, refs, page_size, copies, workspace, window, sinks, status, step_lens)
    if rc != MT_OK:
        _check(rc, "mla_pages_fit")


def mla_paged_copy(copies, cache, status=None, stream=None):
    """Copies the first copies[i, 2] rows of page copies[i, 0] to page copies[i,
    1] (-1: none), in a cache [num_pages, page_size, 576] or in every layer of
    [layers, num_pages, page_size, 576]."""
    rc = (_paged_call or _load_paged_call()).copy(copies, cache, status, None if stream is None else stream.cuda_stream)
    if rc is None:
        dev = _refuse_layers(cache)
        _refuse("copies", copies, torch.int32, 2, dev)
        _refuse("copies", copies, torch.int32, 2, dev, (copies.shape[0], 3), True)
        _refuse_status(status, dev, "cache")
    if rc != MT_OK:
        _check(rc, "mla_paged_copy")
