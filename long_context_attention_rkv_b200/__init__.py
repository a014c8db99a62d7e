"""Python binding of librkv, the residual KV-cache compression library for B200.

Argument marshalling only: every function here forwards to the C ABI declared
in ``include/rkv.h`` (same names), and every step of the path runs in the
library's CUDA kernels.  PyTorch is used for device memory and streams.  If
``librkv.so`` has not been built the import of the library fails loudly; there
is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librkv.so")

RKV_DTYPE_BF16 = 0
RKV_DTYPE_F32 = 1
RKV_DTYPE_F16 = 2
RKV_KV8_INT8 = 0
RKV_KV8_E4M3 = 1
RKV_FLAG_SELECT_SIMT = 0x1
RKV_FLAG_DECODE_DIRECT = 0x2
RKV_FLAG_DECODE_SIMT = 0x4
RKV_IDX_UNUSED = 0xFFFF
RKV_CACHE_DESC_BYTES = 32768

STATUS = {0: "RKV_OK", 1: "RKV_ERR_INVALID_ARG", 2: "RKV_ERR_UNSUPPORTED", 3: "RKV_ERR_WORKSPACE",
          4: "RKV_ERR_CUDA", 5: "RKV_ERR_CORRUPT", 6: "RKV_ERR_TIMEOUT"}
STATUS_CODE = {v: k for k, v in STATUS.items()}

EXPORTED = ["rkv_abi_version", "rkv_status_string", "rkv_schedule", "rkv_cache_size", "rkv_cache_bind",
            "rkv_unit_view_get", "rkv_build_refs", "rkv_search", "rkv_encode", "rkv_compress", "rkv_decode_attn", "rkv_reconstruct",
            "rkv_read_device_error", "rkv_compress_noalloc", "rkv_decode_attn_sparse", "rkv_cache_set_lengths",
            "rkv_append", "rkv_set_coder", "rkv_selftest_wait_timeout", "rkv_prefill_attn", "rkv_blocks_extend",
            "rkv_blocks_release", "rkv_kv8_store", "rkv_kv8_workspace", "rkv_kv8_decode_attn"]


class RkvError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


class rkv_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("head_dim", "n_kv_heads", "n_q_heads", "k", "bits", "group",
                                              "stride0", "refs_per_phase", "in_dtype", "out_dtype", "batch",
                                              "max_len")] + [("flags", ctypes.c_uint32), ("ref_bits", ctypes.c_int32),
                                                             ("coder", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class rkv_unit_view(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n", "n_ref", "n_cmp", "k", "code_bytes", "n_groups", "ref_bits",
                                              "reserved")] + \
               [(n, ctypes.c_void_p) for n in ("ref_K", "ref_V", "ref_half_norm", "ref_pos", "codes_K", "codes_V",
                                               "scale_K", "scale_V", "idx", "ref_scale_K", "ref_scale_V")]


class rkv_prefill_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("head_dim", "n_kv_heads", "n_q_heads", "batch", "in_dtype", "out_dtype",
                                              "kv_padded")] + [("scale", ctypes.c_float)] + \
               [(n, ctypes.c_int64) for n in ("q_rows", "kv_rows", "q_row_stride", "q_head_stride", "kv_row_stride",
                                              "kv_head_stride", "kv_plane_stride", "out_row_stride",
                                              "out_head_stride")]


class rkv_blocks_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "max_blocks", "block_size", "n_blocks")]


class rkv_kv8_cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("head_dim", "n_kv_heads", "n_q_heads", "block_size", "n_blocks",
                                              "max_blocks", "batch", "code_type", "in_dtype", "out_dtype")] + \
               [("scale", ctypes.c_float), ("reserved", ctypes.c_int32)] + \
               [(n, ctypes.c_void_p) for n in ("codes_K", "codes_V", "scale_K", "scale_V", "device_status")]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded librkv.so (raises if it is not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"librkv.so is not built ({LIB_PATH}); run long_context_attention_rkv_b200/build.py")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, u64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64
        cfgp = ctypes.POINTER(rkv_config)
        L.rkv_abi_version.restype = i32
        L.rkv_status_string.argtypes = [ctypes.c_int]
        L.rkv_status_string.restype = ctypes.c_char_p
        L.rkv_schedule.argtypes = [cfgp, i32, vp, i64, ctypes.POINTER(i32)]
        L.rkv_cache_size.argtypes = [cfgp, vp, ctypes.POINTER(u64), ctypes.POINTER(u64)]
        L.rkv_cache_bind.argtypes = [cfgp, vp, vp, u64, vp]
        L.rkv_unit_view_get.argtypes = [vp, i32, i32, ctypes.POINTER(rkv_unit_view)]
        L.rkv_build_refs.argtypes = [vp, vp, vp, vp]
        L.rkv_search.argtypes = [vp, vp, vp, u64, vp]
        L.rkv_encode.argtypes = [vp, vp, vp, vp, u64, vp]
        L.rkv_compress.argtypes = [vp, vp, vp, vp, u64, vp]
        L.rkv_decode_attn.argtypes = [vp, vp, vp, vp, u64, vp]
        L.rkv_reconstruct.argtypes = [vp, i32, i32, vp, i64, vp, vp, i32, vp]
        L.rkv_read_device_error.argtypes = [vp, vp, ctypes.POINTER(i32)]
        L.rkv_compress_noalloc.argtypes = [vp, vp, vp, vp]
        L.rkv_decode_attn_sparse.argtypes = [vp, vp, vp, vp, i32, vp, vp, u64, vp]
        L.rkv_cache_set_lengths.argtypes = [vp, vp, vp]
        L.rkv_append.argtypes = [vp, vp, vp, vp, vp]
        L.rkv_set_coder.argtypes = [vp, vp]
        L.rkv_selftest_wait_timeout.argtypes = [vp, vp]
        L.rkv_prefill_attn.argtypes = [vp] * 11
        L.rkv_blocks_extend.argtypes = [vp] * 8 + [i64] + [vp] * 4
        L.rkv_blocks_release.argtypes = [vp] * 10
        L.rkv_kv8_store.argtypes = [vp, vp, vp, i64, i64, vp, i64, vp]
        L.rkv_kv8_workspace.argtypes = [vp, ctypes.POINTER(u64)]
        L.rkv_kv8_decode_attn.argtypes = [vp] * 6 + [u64, vp]
        for name in EXPORTED[2:]:
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def _check(status: int, where: str):
    if status != 0:
        raise RkvError(status, where)


def _ptr(x):
    if x is None:
        return None
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    return int(x)


def _stream(stream):
    if stream is None:
        import torch

        return torch.cuda.current_stream().cuda_stream
    if hasattr(stream, "cuda_stream"):
        return stream.cuda_stream
    return int(stream)


def _lengths(lengths):
    arr = np.ascontiguousarray(np.asarray(lengths, dtype=np.int32))
    return arr, arr.ctypes.data


class CacheDesc:
    """Host-side handle of a bound cache (the opaque rkv_cache_desc blob)."""

    def __init__(self):
        self.buf = ctypes.create_string_buffer(RKV_CACHE_DESC_BYTES)

    @property
    def ptr(self):
        return ctypes.addressof(self.buf)


def make_config(head_dim, n_kv_heads, n_q_heads, k, bits, stride0, batch, max_len, refs_per_phase=0,
                in_dtype=RKV_DTYPE_BF16, out_dtype=None, group=32, flags=0, ref_bits=0, coder=0) -> rkv_config:
    """ref_bits: 0 (or 16) bf16 reference rows; 4 the int4 reference store.  coder: 0 identity,
    1 the learned-coder shapes (weights bound with rkv_set_coder)."""
    return rkv_config(head_dim, n_kv_heads, n_q_heads, k, bits, group, stride0, refs_per_phase, in_dtype,
                      in_dtype if out_dtype is None else out_dtype, batch, max_len, flags, ref_bits, coder, 0)


def make_prefill_config(head_dim, n_kv_heads, n_q_heads, batch, q_rows, kv_rows, in_dtype=RKV_DTYPE_BF16,
                        out_dtype=None, kv_padded=False, scale=0.0, q_strides=None, kv_strides=None,
                        out_strides=None) -> rkv_prefill_config:
    """Strides in elements, contiguous layouts by default: q and out [q_rows][n_q_heads][head_dim] (row, head);
    K and V packed [kv_rows][n_kv_heads][head_dim] or, with kv_padded, [batch][n_kv_heads][kv_rows][head_dim],
    the layout of rkv_compress (row, head, plane)."""
    D = head_dim
    qs = (n_q_heads * D, D) if q_strides is None else q_strides
    os_ = (n_q_heads * D, D) if out_strides is None else out_strides
    if kv_strides is None:
        kv_strides = (D, max(1, kv_rows) * D, n_kv_heads * max(1, kv_rows) * D) if kv_padded else (n_kv_heads * D, D, 0)
    return rkv_prefill_config(D, n_kv_heads, n_q_heads, batch, in_dtype, in_dtype if out_dtype is None else out_dtype,
                              1 if kv_padded else 0, scale, q_rows, kv_rows, qs[0], qs[1], *kv_strides, *os_)


def make_blocks_config(batch, max_blocks, block_size, n_blocks) -> rkv_blocks_config:
    return rkv_blocks_config(batch, max_blocks, block_size, n_blocks)


def make_kv8_config(head_dim, n_kv_heads, n_q_heads, block_size, n_blocks, max_blocks, batch, code_type=RKV_KV8_INT8,
                    in_dtype=RKV_DTYPE_BF16, out_dtype=None, scale=0.0) -> rkv_kv8_cache:
    """Shape of an 8-bit block cache; KV8Cache fills in the buffers."""
    return rkv_kv8_cache(head_dim, n_kv_heads, n_q_heads, block_size, n_blocks, max_blocks, batch, code_type, in_dtype,
                         in_dtype if out_dtype is None else out_dtype, scale, 0)


# --- the C ABI, one function each ------------------------------------------------------

def rkv_abi_version() -> int:
    return lib().rkv_abi_version()


def rkv_status_string(status: int) -> str:
    return lib().rkv_status_string(status).decode()


def rkv_schedule(cfg: rkv_config, n: int) -> np.ndarray:
    cnt = ctypes.c_int32(0)
    _check(lib().rkv_schedule(ctypes.byref(cfg), n, None, 0, ctypes.byref(cnt)), "rkv_schedule")
    pos = np.empty(cnt.value, dtype=np.int32)
    _check(lib().rkv_schedule(ctypes.byref(cfg), n, pos.ctypes.data, cnt.value, ctypes.byref(cnt)), "rkv_schedule")
    return pos


def rkv_cache_size(cfg: rkv_config, lengths) -> tuple[int, int]:
    arr, p = _lengths(lengths)
    cb, wb = ctypes.c_uint64(0), ctypes.c_uint64(0)
    _check(lib().rkv_cache_size(ctypes.byref(cfg), p, ctypes.byref(cb), ctypes.byref(wb)), "rkv_cache_size")
    return cb.value, wb.value


def rkv_cache_bind(cfg: rkv_config, lengths, dev_buf, nbytes: int) -> CacheDesc:
    arr, p = _lengths(lengths)
    d = CacheDesc()
    _check(lib().rkv_cache_bind(ctypes.byref(cfg), p, _ptr(dev_buf), nbytes, d.ptr), "rkv_cache_bind")
    return d


def rkv_unit_view_get(desc: CacheDesc, seq: int, kv_head: int) -> rkv_unit_view:
    v = rkv_unit_view()
    _check(lib().rkv_unit_view_get(desc.ptr, seq, kv_head, ctypes.byref(v)), "rkv_unit_view_get")
    return v


def rkv_build_refs(desc: CacheDesc, K, V, stream=None):
    _check(lib().rkv_build_refs(desc.ptr, _ptr(K), _ptr(V), _stream(stream)), "rkv_build_refs")


def rkv_search(desc: CacheDesc, K, workspace, workspace_bytes: int, stream=None):
    _check(lib().rkv_search(desc.ptr, _ptr(K), _ptr(workspace), workspace_bytes, _stream(stream)), "rkv_search")


def rkv_encode(desc: CacheDesc, K, V, workspace, workspace_bytes: int, stream=None):
    _check(lib().rkv_encode(desc.ptr, _ptr(K), _ptr(V), _ptr(workspace), workspace_bytes, _stream(stream)),
           "rkv_encode")


def rkv_compress(desc: CacheDesc, K, V, workspace, workspace_bytes: int, stream=None):
    _check(lib().rkv_compress(desc.ptr, _ptr(K), _ptr(V), _ptr(workspace), workspace_bytes, _stream(stream)),
           "rkv_compress")


def rkv_compress_noalloc(desc: CacheDesc, K, V, stream=None):
    """rkv_compress with the library's own fixed scratch array instead of a workspace (for callers
    that cannot allocate); see include/rkv.h for its limit and sharing rules."""
    _check(lib().rkv_compress_noalloc(desc.ptr, _ptr(K), _ptr(V), _stream(stream)), "rkv_compress_noalloc")


def rkv_decode_attn(desc: CacheDesc, q, out, workspace, workspace_bytes: int, stream=None):
    _check(lib().rkv_decode_attn(desc.ptr, _ptr(q), _ptr(out), _ptr(workspace), workspace_bytes, _stream(stream)),
           "rkv_decode_attn")


def rkv_cache_set_lengths(desc: CacheDesc, lengths, stream=None):
    arr, p = _lengths(lengths)
    _check(lib().rkv_cache_set_lengths(desc.ptr, p, _stream(stream)), "rkv_cache_set_lengths")


def rkv_append(desc: CacheDesc, K_new, V_new, active=None, stream=None):
    act = None if active is None else (ctypes.c_uint8 * len(active))(*[1 if x else 0 for x in active])
    _check(lib().rkv_append(desc.ptr, _ptr(K_new), _ptr(V_new), act, _stream(stream)), "rkv_append")


def rkv_set_coder(desc: CacheDesc, weights):
    """weights: eight device bf16 tensors [D][D]: Wg, Wu, Wo, Wd of K, then of V."""
    assert len(weights) == 8
    arr = (ctypes.c_void_p * 8)(*[_ptr(w) for w in weights])
    _check(lib().rkv_set_coder(desc.ptr, arr), "rkv_set_coder")


def rkv_decode_attn_sparse(desc: CacheDesc, q, positions, counts, max_sel: int, out, workspace, workspace_bytes: int,
                           stream=None):
    _check(lib().rkv_decode_attn_sparse(desc.ptr, _ptr(q), _ptr(positions), _ptr(counts), max_sel, _ptr(out),
                                        _ptr(workspace), workspace_bytes, _stream(stream)), "rkv_decode_attn_sparse")


def rkv_reconstruct(desc: CacheDesc, seq: int, kv_head: int, positions, n_pos: int, K_out, V_out,
                    out_dtype: int, stream=None):
    _check(lib().rkv_reconstruct(desc.ptr, seq, kv_head, _ptr(positions), n_pos, _ptr(K_out), _ptr(V_out),
                                 out_dtype, _stream(stream)), "rkv_reconstruct")


def rkv_read_device_error(desc: CacheDesc, stream=None) -> int:
    v = ctypes.c_int32(0)
    _check(lib().rkv_read_device_error(desc.ptr, _stream(stream), ctypes.byref(v)), "rkv_read_device_error")
    return v.value


def rkv_selftest_wait_timeout(err_dev, stream=None):
    """Queues the bounded-wait self-test; after a stream synchronisation err_dev (a device int32
    tensor) holds RKV_ERR_TIMEOUT (about 2 s later)."""
    _check(lib().rkv_selftest_wait_timeout(_ptr(err_dev), _stream(stream)), "rkv_selftest_wait_timeout")


def _refuse(where: str, why: str):
    raise RkvError(STATUS_CODE["RKV_ERR_INVALID_ARG"], f"{where} ({why})")


_device = _raw = None          # torch's current device and its current stream as an address, once torch is there


def _torch_calls():
    global _device, _raw
    import torch

    _device, _raw = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _elsewhere(where, x, cur):
    _refuse(where, f"a tensor on {x.device}, not on cuda:{cur}")


def _local(where: str, tensors):
    """Device addresses of tensors (None and plain addresses pass) and the current device's ordinal; tensors of
    another device, whose streams the call would not follow, are refused."""
    if _device is None:
        _torch_calls()
    cur = _device()
    return [x if x is None or x.__class__ is int else x.data_ptr() if x.get_device() == cur else _elsewhere(where, x, cur)
            for x in tensors], cur


def _raw_stream(stream, cur: int) -> int:
    return _raw(cur) if stream is None else _stream(stream)


def rkv_prefill_attn(cfg: rkv_prefill_config, q, K, V, q_off, kv_off, kv_len, out, lse, device_status, stream=None):
    p, cur = _local("rkv_prefill_attn", (q, K, V, q_off, kv_off, kv_len, out, lse, device_status))
    _check(lib().rkv_prefill_attn(ctypes.addressof(cfg), *p, _raw_stream(stream, cur)), "rkv_prefill_attn")


def rkv_blocks_extend(cfg: rkv_blocks_config, lengths, new_counts, block_table, free_list, n_free, new_off, slot_map,
                      max_new: int, lengths_out, n_free_out, device_status, stream=None):
    p, cur = _local("rkv_blocks_extend", (lengths, new_counts, block_table, free_list, n_free, new_off, slot_map,
                                          max_new, lengths_out, n_free_out, device_status))
    _check(lib().rkv_blocks_extend(ctypes.addressof(cfg), *p, _raw_stream(stream, cur)), "rkv_blocks_extend")


def rkv_blocks_release(cfg: rkv_blocks_config, lengths, ended, block_table, free_list, n_free, lengths_out, n_free_out,
                       device_status, stream=None):
    p, cur = _local("rkv_blocks_release", (lengths, ended, block_table, free_list, n_free, lengths_out, n_free_out,
                                           device_status))
    _check(lib().rkv_blocks_release(ctypes.addressof(cfg), *p, _raw_stream(stream, cur)), "rkv_blocks_release")


def rkv_kv8_store(cache: rkv_kv8_cache, K_new, V_new, row_stride: int, head_stride: int, slot_map, n_rows: int,
                  stream=None):
    p, cur = _local("rkv_kv8_store", (K_new, V_new, row_stride, head_stride, slot_map, n_rows))
    _check(lib().rkv_kv8_store(ctypes.addressof(cache), *p, _raw_stream(stream, cur)), "rkv_kv8_store")


def rkv_kv8_workspace(cache: rkv_kv8_cache) -> int:
    n = ctypes.c_uint64(0)
    _check(lib().rkv_kv8_workspace(ctypes.addressof(cache), ctypes.byref(n)), "rkv_kv8_workspace")
    return n.value


def rkv_kv8_decode_attn(cache: rkv_kv8_cache, q, block_table, lengths, out, workspace, workspace_bytes: int,
                        stream=None):
    p, cur = _local("rkv_kv8_decode_attn", (q, block_table, lengths, out, workspace, workspace_bytes))
    _check(lib().rkv_kv8_decode_attn(ctypes.addressof(cache), *p, _raw_stream(stream, cur)), "rkv_kv8_decode_attn")


# --- buffers ---------------------------------------------------------------------------

class Layer:
    """One layer's compressed cache: torch-allocated cache and workspace buffers plus the bound handle."""

    def __init__(self, cfg: rkv_config, lengths, device="cuda", workspace=None):
        import torch

        self.cfg = cfg
        self.lengths = [int(x) for x in lengths]
        self.cache_bytes, self.ws_bytes = rkv_cache_size(cfg, self.lengths)
        self.cache = torch.empty(self.cache_bytes, dtype=torch.uint8, device=device)
        if workspace is None:
            workspace = torch.empty(max(256, self.ws_bytes), dtype=torch.uint8, device=device)
        if workspace is not False:           # False: no workspace (calls that need none)
            assert workspace.numel() >= self.ws_bytes
        self.workspace = workspace if workspace is not False else None
        self.desc = rkv_cache_bind(cfg, self.lengths, self.cache, self.cache_bytes)

    def build_refs(self, K, V, stream=None):
        rkv_build_refs(self.desc, K, V, stream)

    def search(self, K, stream=None):
        rkv_search(self.desc, K, self.workspace, self.workspace.numel(), stream)

    def encode(self, K, V, stream=None):
        rkv_encode(self.desc, K, V, self.workspace, self.workspace.numel(), stream)

    def compress(self, K, V, stream=None):
        rkv_compress(self.desc, K, V, self.workspace, self.workspace.numel(), stream)

    def decode(self, q, out, stream=None):
        rkv_decode_attn(self.desc, q, out, self.workspace, self.workspace.numel(), stream)

    def set_coder(self, weights):
        """Learned-coder weights (kept referenced here so they outlive the handle's use)."""
        self._coder_weights = list(weights)
        rkv_set_coder(self.desc, self._coder_weights)

    def set_lengths(self, lengths, stream=None):
        """Current lengths (<= the bound ones, which are the capacity)."""
        rkv_cache_set_lengths(self.desc, lengths, stream)

    def append(self, K_new, V_new, active=None, stream=None):
        """One new token per active sequence: K_new, V_new [batch, kv_heads, head_dim] on the device."""
        rkv_append(self.desc, K_new, V_new, active, stream)

    def decode_sparse(self, q, positions, counts, out, stream=None):
        """positions: int32 [n_units, max_sel] on the device, counts: int32 [n_units] on the device."""
        rkv_decode_attn_sparse(self.desc, q, positions, counts, positions.shape[-1], out, self.workspace,
                               self.workspace.numel(), stream)

    def reconstruct(self, seq, kv_head, positions, n_pos, K_out, V_out, out_dtype, stream=None):
        rkv_reconstruct(self.desc, seq, kv_head, positions, n_pos, K_out, V_out, out_dtype, stream)

    def device_error(self, stream=None) -> int:
        return rkv_read_device_error(self.desc, stream)

    def unit(self, seq: int, kv_head: int) -> rkv_unit_view:
        return rkv_unit_view_get(self.desc, seq, kv_head)


def _take_error(status) -> int:
    """Reads and clears a device status word (waits for the current stream)."""
    v = int(status.item())
    if v:
        status.zero_()
    return v


def _torch_dtype(code: int):
    import torch

    return {RKV_DTYPE_BF16: torch.bfloat16, RKV_DTYPE_F32: torch.float32, RKV_DTYPE_F16: torch.float16}.get(code)


def _need(where: str, name: str, x, n: int, dtype, strided=False):
    """Refuses a tensor of another type, or with fewer than n elements to reach from its first one: those of a
    contiguous tensor or, where the layout is described apart from it (strided), those of its storage."""
    if x.dtype is dtype:
        if x.is_contiguous():
            if x.numel() >= n:
                return
        elif strided and x.untyped_storage().nbytes() // x.element_size() - x.storage_offset() >= n:
            return
    _refuse(where, f"{name} must be {dtype}" + ("" if strided else ", contiguous") + f" and hold {n} elements")


def _need_width(where: str, name: str, x, width: int):
    """Refuses a tensor with rows of another width: the call steps over rows of `width` elements (a flat tensor has none)."""
    if x.dim() > 1 and x.shape[-1] != width:
        _refuse(where, f"{name} has rows of {x.shape[-1]} elements, not {width}")


def _need_heads(where: str, name: str, x, heads):
    """The same for rows of heads = (heads, channels), which may be one dimension or two."""
    if x.dim() > 2 and x.shape[-2:] != heads or x.dim() == 2 and x.shape[1] not in (heads[0] * heads[1], heads[1]):
        _refuse(where, f"{name} has rows of {tuple(x.shape[1:])} elements, not {heads}")


class Prefill:
    """Causal attention over packed prompts: a configuration and its device status word."""

    def __init__(self, cfg: rkv_prefill_config, device="cuda"):
        import torch

        c = self.cfg = rkv_prefill_config.from_buffer_copy(cfg)
        self._in, self._out, self._i32, self._f32 = (_torch_dtype(c.in_dtype), _torch_dtype(c.out_dtype), torch.int32,
                                                     torch.float32)

        def reach(rows, row, heads, head, planes=1, plane=0):
            return (rows - 1) * row + (heads - 1) * head + (planes - 1) * plane + c.head_dim if rows > 0 else 0

        self._offs = (c.batch + 1, c.batch if c.kv_padded else c.batch + 1, c.batch, c.q_rows * c.n_q_heads)
        self._q_reach = reach(c.q_rows, c.q_row_stride, c.n_q_heads, c.q_head_stride)
        self._out_reach = reach(c.q_rows, c.out_row_stride, c.n_q_heads, c.out_head_stride)
        self._kv_reach = reach(c.kv_rows, c.kv_row_stride, c.n_kv_heads, c.kv_head_stride,
                               c.batch if c.kv_padded else 1, c.kv_plane_stride)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def attend(self, q, K, V, q_off, out, kv_off=None, kv_len=None, lse=None, stream=None):
        """q_off, kv_off: int32 [batch + 1], kv_len: int32 [batch], lse: float32 [q_rows, q_heads], all on the device;
        q, K, V and out laid out as the configuration's strides say."""
        dt, kv = self._in, self._kv_reach
        if not (q.dtype is dt and K.dtype is dt and V.dtype is dt and out.dtype is self._out and q.is_contiguous() and
                K.is_contiguous() and V.is_contiguous() and out.is_contiguous() and q.numel() >= self._q_reach and
                K.numel() >= kv and V.numel() >= kv and out.numel() >= self._out_reach):
            # strided views, or one of them is refused
            where = "Prefill.attend"
            _need(where, "q", q, self._q_reach, dt, True)
            _need(where, "K", K, kv, dt, True)
            _need(where, "V", V, kv, dt, True)
            _need(where, "out", out, self._out_reach, self._out, True)
        n_off, n_kv_off, n_len, n_lse = self._offs
        _need("Prefill.attend", "q_off", q_off, n_off, self._i32)
        if kv_off is not None:
            _need("Prefill.attend", "kv_off", kv_off, n_kv_off, self._i32)
        if kv_len is not None:
            _need("Prefill.attend", "kv_len", kv_len, n_len, self._i32)
        if lse is not None:
            _need("Prefill.attend", "lse", lse, n_lse, self._f32)
            _need_width("Prefill.attend", "lse", lse, self.cfg.n_q_heads)
        rkv_prefill_attn(self.cfg, q, K, V, q_off, kv_off, kv_len, out, lse, self.status, stream)

    def device_error(self) -> int:
        return _take_error(self.status)


class BlockTables:
    """Block table, free stack and lengths of the requests of a block cache, kept on the device."""

    def __init__(self, batch, max_blocks, block_size, n_blocks, device="cuda"):
        import torch

        self.cfg = make_blocks_config(batch, max_blocks, block_size, n_blocks)
        i32 = dict(dtype=torch.int32, device=device)
        self.table = torch.full((batch, max_blocks), -1, **i32)
        self.free_list = torch.arange(n_blocks - 1, -1, -1, **i32)     # block 0 on top
        self.n_free = torch.full((1,), n_blocks, **i32)
        self.lengths = torch.zeros(batch, **i32)
        self.new_off = torch.zeros(batch + 1, **i32)
        self.status = torch.zeros(1, **i32)

    def extend(self, new_counts, slot_map, stream=None):
        """Room for new_counts[b] more tokens of each request; their slots go to slot_map (int32, -1 behind the
        last), their packed offsets to new_off, and lengths grows."""
        _need("BlockTables.extend", "new_counts", new_counts, self.cfg.batch, self.lengths.dtype)
        _need("BlockTables.extend", "slot_map", slot_map, 0, self.lengths.dtype)
        rkv_blocks_extend(self.cfg, self.lengths, new_counts, self.table, self.free_list, self.n_free, self.new_off,
                          slot_map, slot_map.numel(), self.lengths, self.n_free, self.status, stream)

    def release(self, ended, stream=None):
        """The blocks of the requests with a nonzero flag (int32) go back, their lengths become 0."""
        _need("BlockTables.release", "ended", ended, self.cfg.batch, self.lengths.dtype)
        rkv_blocks_release(self.cfg, self.lengths, ended, self.table, self.free_list, self.n_free, self.lengths,
                           self.n_free, self.status, stream)

    def device_error(self) -> int:
        return _take_error(self.status)


class KV8Cache:
    """One layer's 8-bit block cache: codes [n_blocks, kv_heads, block_size, head_dim] (int8 or float8_e4m3fn) and
    scales [n_blocks, kv_heads] (float32), allocated here unless given, and the decode's workspace."""

    def __init__(self, cfg: rkv_kv8_cache, codes_K=None, codes_V=None, scale_K=None, scale_V=None, device="cuda",
                 workspace=None):
        import torch

        self.ws_bytes = rkv_kv8_workspace(cfg)                         # refuses an impossible shape
        shape = (cfg.n_blocks, cfg.n_kv_heads, cfg.block_size, cfg.head_dim)
        kind = torch.int8 if cfg.code_type == RKV_KV8_INT8 else torch.float8_e4m3fn

        def buffer(x, shape, dtype, name):
            if x is None:
                return torch.zeros(shape, dtype=torch.uint8 if dtype is kind else dtype, device=device).view(dtype)
            if tuple(x.shape) != shape or x.dtype is not dtype or not x.is_contiguous():
                _refuse("KV8Cache", f"{name} must be a contiguous {dtype} tensor of shape {shape}")
            return x

        self.codes_K = buffer(codes_K, shape, kind, "codes_K")
        self.codes_V = buffer(codes_V, shape, kind, "codes_V")
        self.scale_K = buffer(scale_K, shape[:2], torch.float32, "scale_K")
        self.scale_V = buffer(scale_V, shape[:2], torch.float32, "scale_V")
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        if workspace is None:
            workspace = torch.empty(max(256, self.ws_bytes), dtype=torch.uint8, device=device)
        self.workspace = workspace
        if workspace.dtype is not torch.uint8 or not workspace.is_contiguous():
            _refuse("KV8Cache", "workspace must be a contiguous torch.uint8 tensor")
        _, self.device_index = _local("KV8Cache", (self.codes_K, self.codes_V, self.scale_K, self.scale_V, self.workspace,
                                                   self.status))
        self._in, self._out, self._i32 = _torch_dtype(cfg.in_dtype), _torch_dtype(cfg.out_dtype), torch.int32
        self._row = (cfg.n_kv_heads, cfg.head_dim)
        self._heads, self._width = (cfg.n_q_heads, cfg.head_dim), cfg.max_blocks
        self._sizes = (cfg.batch * cfg.n_q_heads * cfg.head_dim, cfg.batch * cfg.max_blocks, cfg.batch)
        self.c = rkv_kv8_cache.from_buffer_copy(cfg)
        for name in ("codes_K", "codes_V", "scale_K", "scale_V"):
            setattr(self.c, name, getattr(self, name).data_ptr())
        self.c.device_status = self.status.data_ptr()

    def store(self, K_new, V_new, slot_map, stream=None):
        """K_new, V_new: [rows, kv_heads, head_dim] with the same row and head strides and contiguous channels;
        slot_map: int32 [rows] (negative: the row is skipped)."""
        where, shape, strides, v_strides = "KV8Cache.store", K_new.shape, K_new.stride(), V_new.stride()
        if len(shape) == 3 and (shape[0] == 1 or shape[1] == 1):       # a dimension of one has no step
            heads, d = self._row
            strides, v_strides = ((s[0] if shape[0] > 1 else heads * d, s[1] if shape[1] > 1 else d, *s[2:])
                                  for s in (strides, v_strides)) if V_new.shape == shape else (strides, None)
        if len(shape) != 3 or shape[1:] != self._row or V_new.shape != shape or v_strides != strides or \
                strides[2] != 1 or K_new.dtype is not self._in or V_new.dtype is not self._in:
            _refuse(where, f"K_new and V_new must be {self._in} [rows, {self._row[0]}, {self._row[1]}] with equal strides "
                           "and contiguous channels")
        _need(where, "slot_map", slot_map, shape[0], self._i32)
        self._here(where)
        rkv_kv8_store(self.c, K_new, V_new, strides[0], strides[1], slot_map, shape[0], stream)

    def decode(self, q, block_table, lengths, out, stream=None):
        """q, out: [batch, q_heads, head_dim]; block_table: int32 [batch, max_blocks]; lengths: int32 [batch]; all
        contiguous.  One workspace: calls on several streams must not overlap."""
        n, n_table, n_len = self._sizes
        i32 = self._i32
        if not (q.dtype is self._in and out.dtype is self._out and block_table.dtype is i32 and lengths.dtype is i32 and
                q.numel() >= n and out.numel() >= n and block_table.numel() >= n_table and lengths.numel() >= n_len and
                block_table.shape[-1] == self._width and q.shape[1:] == self._heads and out.shape[1:] == self._heads and
                q.is_contiguous() and out.is_contiguous() and block_table.is_contiguous() and lengths.is_contiguous()):
            _need("KV8Cache.decode", "q", q, n, self._in)
            _need("KV8Cache.decode", "out", out, n, self._out)
            _need("KV8Cache.decode", "block_table", block_table, n_table, i32)
            _need_width("KV8Cache.decode", "block_table", block_table, self._width)
            _need("KV8Cache.decode", "lengths", lengths, n_len, i32)
            _need_heads("KV8Cache.decode", "q", q, self._heads)
            _need_heads("KV8Cache.decode", "out", out, self._heads)
        self._here("KV8Cache.decode")
        rkv_kv8_decode_attn(self.c, q, block_table, lengths, out, self.workspace, self.workspace.numel(), stream)

    def _here(self, where):
        """The cache's buffers go into calls as addresses: their device has to be the current one."""
        if _device() != self.device_index:
            _refuse(where, f"the cache is on cuda:{self.device_index}, which is not the current device")

    def device_error(self) -> int:
        return _take_error(self.status)
