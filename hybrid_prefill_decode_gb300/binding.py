"""Thin ctypes binding of the C ABI in ``include/pod_attn.h`` (argument marshalling only).

Every step of the computation runs in the CUDA kernels of ``libpod_attn.so``; this module only
converts Python/torch arguments to pointers and sizes. There is no fallback: if the library has
not been built, loading raises.
"""
from __future__ import annotations

import array
import ctypes
import functools
import os
import re
from typing import Optional, Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libpod_attn.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "pod_attn.h")

OK = 0
ERR_INVALID_ARG = -1
ERR_UNSUPPORTED = -2
ERR_WORKSPACE = -3
ERR_CUDA = -4
ERR_BAD_INDEX = -5
ERR_TIMEOUT = -6
ERR_NO_BLOCKS = -7

VARIANTS = {"fused": 0, "serial": 1, "streams": 2}
KV_TYPES = {"bf16": 0, "e4m3": 1, "e2m1": 2}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "llama3": 4, "custom": 5}
BLOCK = 16


class Problem(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_prefill_seqs", ctypes.c_int32), ("num_prefill_tokens", ctypes.c_int32),
                ("num_decode_seqs", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("max_blocks_per_seq", ctypes.c_int32), ("scale", ctypes.c_float)]


class Options(ctypes.Structure):
    _fields_ = [("num_sms", ctypes.c_int32), ("ctas_per_sm", ctypes.c_int32),
                ("max_prefill_ctas", ctypes.c_int32), ("decode_splits", ctypes.c_int32),
                ("prefill_splits", ctypes.c_int32), ("instrument", ctypes.c_int32),
                ("variant", ctypes.c_int32), ("non_causal", ctypes.c_int32),
                ("kv_fp8", ctypes.c_int32), ("kv_fp4", ctypes.c_int32)]


class PlanInfo(ctypes.Structure):
    _fields_ = [("num_prefill_items", ctypes.c_int32), ("num_decode_items", ctypes.c_int32),
                ("num_units", ctypes.c_int32), ("num_sms", ctypes.c_int32),
                ("ctas_per_sm", ctypes.c_int32), ("max_prefill_ctas", ctypes.c_int32),
                ("grid_fused", ctypes.c_int32), ("grid_prefill", ctypes.c_int32),
                ("grid_decode", ctypes.c_int32), ("smem_bytes", ctypes.c_int32),
                ("threads_per_cta", ctypes.c_int32), ("item_words", ctypes.c_int32),
                ("workspace_bytes", ctypes.c_uint64), ("est_prefill_flops", ctypes.c_double),
                ("est_prefill_bytes", ctypes.c_double), ("est_decode_bytes", ctypes.c_double),
                ("est_decode_flops", ctypes.c_double)]

    def as_dict(self):
        return {k: getattr(self, k) for k, _ in self._fields_}


class Bucket(ctypes.Structure):
    _fields_ = [("prefill_flops", ctypes.c_int64), ("read_bytes", ctypes.c_int64),
                ("prefill_ctas", ctypes.c_int32), ("decode_ctas", ctypes.c_int32),
                ("grid", ctypes.c_int32), ("smem_per_cta", ctypes.c_int32),
                ("tmem_cols_per_cta", ctypes.c_int32), ("bucket_flops", ctypes.c_int32),
                ("bucket_bytes", ctypes.c_int32), ("bucket_ctas", ctypes.c_int32),
                ("intensity", ctypes.c_double), ("kv_type", ctypes.c_int32)]


class ItemRecord(ctypes.Structure):
    _fields_ = [("smid", ctypes.c_int32), ("kind", ctypes.c_int32), ("item", ctypes.c_int32),
                ("cta", ctypes.c_int32), ("t_start", ctypes.c_uint64),
                ("t_end", ctypes.c_uint64)]


class KvCacheDesc(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class RopeConfig(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("scaling", ctypes.c_int32), ("theta", ctypes.c_double),
                ("factor", ctypes.c_double), ("original_max_position", ctypes.c_double),
                ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double),
                ("low_freq_factor", ctypes.c_double), ("high_freq_factor", ctypes.c_double),
                ("attention_factor", ctypes.c_double), ("h_inv_freq", ctypes.c_void_p)]


class BlockPool(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("block_bytes", ctypes.c_size_t)]


_lib = None


def declared_functions() -> list:
    """Names of the functions include/pod_attn.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(pod_attn_[a-z0-9_]+)\s*\(", text)))


def load():
    """Load libpod_attn.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    lib.pod_attn_plan.restype = I32
    lib.pod_attn_plan.argtypes = [ctypes.POINTER(Problem), P, P, ctypes.POINTER(Options),
                                  ctypes.POINTER(P)]
    lib.pod_attn_workspace_bytes.restype = SZ
    lib.pod_attn_workspace_bytes.argtypes = [P]
    lib.pod_attn_upload.restype = I32
    lib.pod_attn_upload.argtypes = [P, P, SZ, P]
    lib.pod_attn_run.restype = I32
    lib.pod_attn_run.argtypes = [P, P, P, P, P, P, P, P, P, P, P, SZ, P, P]
    lib.pod_attn_run_decode_fp8.restype = I32
    lib.pod_attn_run_decode_fp8.argtypes = [P, P, P, P, P, P, P, P, P, P, SZ, P]
    lib.pod_attn_append_fp8.restype = I32
    lib.pod_attn_append_fp8.argtypes = [P, P, P, P, P, P, P, P, P, SZ, P]
    lib.pod_attn_plan_bucket.restype = I32
    lib.pod_attn_plan_bucket.argtypes = [P, ctypes.POINTER(Bucket)]
    lib.pod_attn_run_append.restype = I32
    lib.pod_attn_run_append.argtypes = [P, P, P, P, P, P, P, P, P, P, P, P, P, SZ, P, P]
    lib.pod_attn_last_device_status.restype = I32
    lib.pod_attn_last_device_status.argtypes = [P, P, P]
    lib.pod_attn_get_plan_info.restype = I32
    lib.pod_attn_get_plan_info.argtypes = [P, ctypes.POINTER(PlanInfo)]
    lib.pod_attn_plan_items.restype = I32
    lib.pod_attn_plan_items.argtypes = [P, P, SZ, ctypes.POINTER(SZ)]
    lib.pod_attn_read_records.restype = I32
    lib.pod_attn_read_records.argtypes = [P, P, P, SZ, ctypes.POINTER(SZ), P]
    lib.pod_attn_plan_destroy.restype = None
    lib.pod_attn_plan_destroy.argtypes = [P]
    lib.pod_attn_status_string.restype = ctypes.c_char_p
    lib.pod_attn_status_string.argtypes = [I32]
    lib.pod_attn_selftest_timeout.restype = I32
    lib.pod_attn_selftest_timeout.argtypes = [P, I32, P]
    I64 = ctypes.c_int64
    lib.pod_attn_rope_create.restype = I32
    lib.pod_attn_rope_create.argtypes = [ctypes.POINTER(RopeConfig), ctypes.POINTER(P)]
    lib.pod_attn_rope_destroy.restype = None
    lib.pod_attn_rope_destroy.argtypes = [P]
    lib.pod_attn_rope_frequencies.restype = I32
    lib.pod_attn_rope_frequencies.argtypes = [P, P, ctypes.POINTER(ctypes.c_double)]
    lib.pod_attn_rope_append.restype = I32
    lib.pod_attn_rope_append.argtypes = [P, P, P, I64, P, I64, P, I64, ctypes.POINTER(KvCacheDesc),
                                         P, P, P, P, SZ, P]
    lib.pod_attn_run_decode_fp4.restype = I32
    lib.pod_attn_run_decode_fp4.argtypes = [P, P, ctypes.POINTER(KvCacheDesc), P, P, P, P, SZ, P]
    lib.pod_attn_expand_fp4.restype = I32
    lib.pod_attn_expand_fp4.argtypes = [P, ctypes.POINTER(KvCacheDesc), P, P, P, P, P, P, SZ, P]
    lib.pod_attn_copy_blocks.restype = I32
    lib.pod_attn_copy_blocks.argtypes = [P, I32, I32, P, I32, P]
    lib.pod_attn_pages_create.restype = I32
    lib.pod_attn_pages_create.argtypes = [I32, I32, I32, ctypes.POINTER(P)]
    lib.pod_attn_pages_destroy.restype = None
    lib.pod_attn_pages_destroy.argtypes = [P]
    lib.pod_attn_pages_grow.restype = I32
    lib.pod_attn_pages_grow.argtypes = [P, I32, I32, P, ctypes.POINTER(I32)]
    lib.pod_attn_pages_fork.restype = I32
    lib.pod_attn_pages_fork.argtypes = [P, I32, I32, I32]
    lib.pod_attn_pages_free.restype = I32
    lib.pod_attn_pages_free.argtypes = [P, I32]
    lib.pod_attn_pages_compact.restype = I32
    lib.pod_attn_pages_compact.argtypes = [P, P, I32, ctypes.POINTER(I32)]
    lib.pod_attn_pages_tables.restype = I32
    lib.pod_attn_pages_tables.argtypes = [P, P, I32, P, P]
    lib.pod_attn_pages_free_blocks.restype = I32
    lib.pod_attn_pages_free_blocks.argtypes = [P]
    _lib = lib
    return lib


class PodAttnError(RuntimeError):
    def __init__(self, code, where):
        super().__init__(f"{where}: {load().pod_attn_status_string(code).decode()} ({code})")
        self.code = code


def _check(code, where):
    if code != OK:
        raise PodAttnError(code, where)


def _fits_i32(what: str, values: Sequence[int]):
    """Refuse whole numbers that an int32 does not hold: ctypes would drop their upper bits."""
    if values and (min(values) < -(1 << 31) or max(values) >= 1 << 31):
        raise ValueError(f"{what}: {min(values)} to {max(values)} is beyond int32")


def _i32_array(values: Sequence[int]):
    _fits_i32("list", values)
    arr = (ctypes.c_int32 * max(1, len(values)))(*values)
    return arr


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if t.numel() == 0:
        return None
    assert t.is_contiguous()
    return t.data_ptr()


def _stream_ptr(stream) -> Optional[int]:
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


_torch = _current_device = _current_stream = None


def _load_torch():
    """torch, imported once (importing this module alone does not need it)."""
    global _torch, _current_device, _current_stream
    if _torch is None:
        import torch
        _torch = torch
        _current_device = torch._C._cuda_getDevice
        _current_stream = torch._C._cuda_getCurrentRawStream
    return _torch


# The helpers below run on every call of a serving loop's small operators, where the host's time is
# the call's time: they compare types by identity and devices by index.
def _stream_on(index: int, stream) -> Optional[int]:
    """The stream to launch on: the given one, else the current one of device `index`, which has to
    be the current device (the library launches on the current device)."""
    if _current_device() != index:
        raise ValueError(f"tensors on cuda:{index}, but the current device is "
                         f"cuda:{_current_device()}")
    if stream is None:
        return _current_stream(index)
    return _stream_ptr(stream)


def _arg(name, t, dtype, shape, index) -> Optional[int]:
    """Pointer of a contiguous tensor of this type, shape (a torch.Size) and device index."""
    if t is not None and t.dtype is dtype and t.shape == shape and t.get_device() == index and \
            t.is_contiguous():
        return t.data_ptr()
    if t is None and 0 in shape:
        return None
    got = "None" if t is None else f"{t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}"
    raise ValueError(f"{name}: want contiguous {dtype} {tuple(shape)} on cuda:{index}, got {got}")


def _workspace(t, index) -> int:
    if t.get_device() != index:
        raise ValueError(f"workspace: want it on cuda:{index}, got one on {t.device}")
    return t.data_ptr()


def _rows(name, t, shape, index):
    """(pointer, token stride in elements) of bf16 [tokens][heads][dim] rows, tokens any stride
    apart."""
    if t.dtype is _torch.bfloat16 and t.shape == shape and t.get_device() == index:
        token, head, channel = t.stride()
        if channel == 1 and (head == shape[2] or shape[1] == 1):
            return t.data_ptr(), token if shape[0] > 1 else shape[1] * shape[2]
    raise ValueError(f"{name}: want bfloat16 {tuple(shape)} on cuda:{index} with dense heads, got "
                     f"{t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")


class Rope:
    """Rotary frequencies (pod_attn_rope_create): `scaling` is one of ROPE_SCALINGS; "custom", and no
    other, takes `inv_freq`, one frequency per pair in radians per position. attention_factor 0: the
    default."""

    def __init__(self, rot_dim: int, theta: float = 10000.0, interleaved: bool = False,
                 scaling: str = "none", factor: float = 1.0, original_max_position: float = 0.0,
                 beta_fast: float = 32.0, beta_slow: float = 1.0, low_freq_factor: float = 1.0,
                 high_freq_factor: float = 4.0, attention_factor: float = 0.0,
                 inv_freq: Optional[Sequence[float]] = None):
        self.handle = None
        _fits_i32("rot_dim", (rot_dim,))
        freq = None
        if inv_freq is not None:
            if scaling != "custom":
                raise ValueError(f"inv_freq: scaling {scaling!r} computes its own; want \"custom\"")
            if len(inv_freq) != rot_dim // 2:
                raise ValueError(f"inv_freq: want {rot_dim // 2} values, got {len(inv_freq)}")
            freq = (ctypes.c_double * max(1, len(inv_freq)))(*[float(x) for x in inv_freq])
        cfg = RopeConfig(rot_dim, 1 if interleaved else 0, ROPE_SCALINGS[scaling], theta, factor,
                         original_max_position, beta_fast, beta_slow, low_freq_factor,
                         high_freq_factor, attention_factor,
                         ctypes.cast(freq, ctypes.c_void_p) if freq is not None else None)
        handle = ctypes.c_void_p()
        _check(load().pod_attn_rope_create(ctypes.byref(cfg), ctypes.byref(handle)),
               "pod_attn_rope_create")
        self.handle = handle
        self.rot_dim = rot_dim

    def __del__(self):
        if getattr(self, "handle", None) is not None and _lib is not None:
            _lib.pod_attn_rope_destroy(self.handle)
            self.handle = None

    def frequencies(self):
        """(frequencies in radians per position, attention factor)."""
        out, mag = (ctypes.c_double * (self.rot_dim // 2))(), ctypes.c_double()
        _check(load().pod_attn_rope_frequencies(self.handle, ctypes.cast(out, ctypes.c_void_p),
                                                ctypes.byref(mag)), "pod_attn_rope_frequencies")
        return list(out), mag.value


def fp4_pool_shape(num_blocks: int, num_kv_heads: int, head_dim: int):
    """Shape of a uint8 pool of the 4-bit cache: per (block, kv-head) the codes, then the scales."""
    return num_blocks, num_kv_heads, 9 * head_dim


class KvCache:
    """A paged cache's pools and scales (pod_attn_kv_cache), of `kind` "bf16", "e4m3" or "e2m1"; it
    keeps the tensors alive. e4m3 pools may be uint8 or float8_e4m3fn."""

    def __init__(self, kind: str, k_pool, v_pool, k_scale=None, v_scale=None):
        torch = _load_torch()
        nb, hkv = k_pool.shape[:2]
        types = {"bf16": (torch.bfloat16,), "e4m3": (torch.uint8, torch.float8_e4m3fn),
                 "e2m1": (torch.uint8,)}[kind]
        dim = k_pool.shape[-1] // (9 if kind == "e2m1" else 1)
        shape = fp4_pool_shape(nb, hkv, dim) if kind == "e2m1" else (nb, hkv, BLOCK, dim)
        scales = {"bf16": (None, None), "e4m3": ((hkv, dim), (nb, hkv, BLOCK)),
                  "e2m1": ((hkv,), (hkv,))}[kind]
        for name, t in (("k_pool", k_pool), ("v_pool", v_pool)):
            if (t.dtype not in types or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or
                    t.device != k_pool.device):
                raise ValueError(f"{name}: want contiguous {types[0]} {tuple(shape)} on "
                                 f"{k_pool.device}, got {t.dtype} {tuple(t.shape)} on {t.device}")
        if k_pool.device.type != "cuda":
            raise ValueError(f"k_pool: want a CUDA tensor, got one on {k_pool.device}")
        self.index = k_pool.get_device()
        ptrs = [_arg(name, t, torch.float32, want, self.index) if want else None
                for name, t, want in (("k_scale", k_scale, scales[0]),
                                      ("v_scale", v_scale, scales[1]))]
        self.kind, self.device = kind, k_pool.device
        self.num_blocks, self.num_kv_heads, self.head_dim = int(nb), int(hkv), int(dim)
        self.heads = (self.num_kv_heads, self.head_dim)
        self.tensors = [t for t in (k_pool, v_pool, k_scale, v_scale) if t is not None]
        self.desc = KvCacheDesc(KV_TYPES[kind], int(nb), k_pool.data_ptr(), v_pool.data_ptr(),
                                *ptrs)
        self.ref = ctypes.byref(self.desc)

    @property
    def pools(self):
        """The tensors with a row per block: what copy_blocks has to move."""
        n = 4 if self.kind == "e4m3" else 2
        return [t for t in self.tensors[:n] if t.shape[0] == self.num_blocks and t.dim() > 2]


def copy_blocks(pools, pairs, stream=None):
    """pod_attn_copy_blocks: copy block src to block dst in every tensor of `pools` ([num_blocks]
    [...], contiguous) for each (src, dst) of `pairs` (a CPU int32 tensor [n][2] or a sequence)."""
    torch = _load_torch()
    if not pools:
        return
    if not isinstance(pairs, torch.Tensor):
        pairs = torch.tensor(list(pairs), dtype=torch.int32).reshape(-1, 2)
    if pairs.dtype is not torch.int32 or pairs.dim() != 2 or pairs.shape[1] != 2 or \
            pairs.is_cuda or not pairs.is_contiguous():
        raise ValueError(f"pairs: want a contiguous int32 [n][2] on the CPU, got {pairs.dtype} "
                         f"{tuple(pairs.shape)} on {pairs.device}")
    nb, index = pools[0].shape[0], pools[0].get_device()
    flat = array.array("Q")  # (pointer, bytes per block) of every pool: pod_attn_block_pool
    for t in pools:
        if t.shape[0] != nb or t.get_device() != index or index < 0 or not t.is_contiguous():
            raise ValueError(f"pools: want contiguous CUDA tensors of {nb} blocks on one device, "
                             f"got {tuple(t.shape)} strides {t.stride()} on {t.device}")
        flat.append(t.data_ptr())
        flat.append(t.nbytes // nb if nb else 0)
    if pairs.shape[0] == 0:
        return
    code = load().pod_attn_copy_blocks(flat.buffer_info()[0], len(pools), nb, pairs.data_ptr(),
                                       pairs.shape[0], _stream_on(index, stream))
    if code:
        raise PodAttnError(code, "pod_attn_copy_blocks")


class Pages:
    """Host bookkeeping of a cache's blocks (pod_attn_pages_*). `grow` and `compact` return the
    (src, dst) pairs that copy_blocks has to make on every pool before the next append."""

    def __init__(self, num_blocks: int, max_seqs: int, max_blocks_per_seq: int):
        self.handle = None
        _fits_i32("num_blocks, max_seqs, max_blocks_per_seq",
                  (num_blocks, max_seqs, max_blocks_per_seq))
        handle = ctypes.c_void_p()
        _check(load().pod_attn_pages_create(num_blocks, max_seqs, max_blocks_per_seq,
                                            ctypes.byref(handle)), "pod_attn_pages_create")
        self.handle, self.max_blocks_per_seq = handle, max_blocks_per_seq

    def __del__(self):
        if getattr(self, "handle", None) is not None and _lib is not None:
            _lib.pod_attn_pages_destroy(self.handle)
            self.handle = None

    def grow(self, seq: int, kv_len: int):
        _fits_i32("seq, kv_len", (seq, kv_len))
        pair, n = (ctypes.c_int32 * 2)(), ctypes.c_int32()
        _check(load().pod_attn_pages_grow(self.handle, seq, kv_len,
                                          ctypes.cast(pair, ctypes.c_void_p), ctypes.byref(n)),
               "pod_attn_pages_grow")
        return [tuple(pair)] if n.value else []

    def fork(self, src: int, dst: int, kv_len: int):
        _fits_i32("src, dst, kv_len", (src, dst, kv_len))
        _check(load().pod_attn_pages_fork(self.handle, src, dst, kv_len), "pod_attn_pages_fork")

    def free(self, seq: int):
        _fits_i32("seq", (seq,))
        _check(load().pod_attn_pages_free(self.handle, seq), "pod_attn_pages_free")

    def compact(self):
        import torch
        n = ctypes.c_int32()
        _check(load().pod_attn_pages_compact(self.handle, None, 0, ctypes.byref(n)),
               "pod_attn_pages_compact")
        pairs = torch.empty((n.value, 2), dtype=torch.int32)
        if n.value:
            _check(load().pod_attn_pages_compact(self.handle, pairs.data_ptr(), n.value,
                                                 ctypes.byref(n)), "pod_attn_pages_compact")
        return pairs

    def tables(self, seqs: Sequence[int]):
        """(block tables int32 [n][max_blocks_per_seq], lengths int32 [n]) on the CPU."""
        import torch
        bt = torch.empty((len(seqs), self.max_blocks_per_seq), dtype=torch.int32)
        lens = torch.empty((len(seqs),), dtype=torch.int32)
        ids = _i32_array(list(seqs))
        _check(load().pod_attn_pages_tables(self.handle, ctypes.cast(ids, ctypes.c_void_p),
                                            len(seqs), bt.data_ptr() or None,
                                            lens.data_ptr() or None), "pod_attn_pages_tables")
        return bt, lens

    @property
    def free_blocks(self) -> int:
        return int(load().pod_attn_pages_free_blocks(self.handle))


class _Shapes:
    """The tensor shapes and types that a plan's problem asks for."""

    def __init__(self, p: Problem):
        torch = _load_torch()
        self.bf16, self.i32 = torch.bfloat16, torch.int32
        tp, nd, d = p.num_prefill_tokens, p.num_decode_seqs, p.head_dim
        n = p.num_prefill_seqs + nd
        self.heads = (p.num_kv_heads, d)
        size = torch.Size
        self.q, self.kv = size((tp + nd, p.num_q_heads, d)), size((tp + nd, p.num_kv_heads, d))
        self.q_prefill, self.q_decode = size((tp, p.num_q_heads, d)), size((nd, p.num_q_heads, d))
        self.tables, self.lens = size((n, p.max_blocks_per_seq)), size((n,))
        self.pool = size((p.num_blocks, p.num_kv_heads, BLOCK, d))


class Plan:
    """A planned hybrid batch (host side). Mirrors pod_attn_plan / pod_attn_plan_destroy."""

    def __init__(self, num_q_heads: int, num_kv_heads: int, cu_seqlens: Sequence[int],
                 kv_lens: Sequence[int], num_decode_seqs: int, num_blocks: int,
                 max_blocks_per_seq: int, scale: float, variant: str = "fused",
                 num_sms: int = 0, ctas_per_sm: int = 0, max_prefill_ctas: int = 0,
                 decode_splits: int = 0, prefill_splits: int = 0, instrument: bool = False,
                 non_causal: bool = False, head_dim: int = 128, kv_fp8: bool = False,
                 kv_fp4: bool = False):
        lib = load()
        np_ = len(cu_seqlens) - 1 if len(cu_seqlens) > 0 else 0
        _fits_i32("sizes and options",
                  (num_q_heads, num_kv_heads, num_decode_seqs, num_blocks, max_blocks_per_seq, num_sms,
                   ctas_per_sm, max_prefill_ctas, decode_splits, prefill_splits, head_dim))
        self.problem = Problem(num_q_heads, num_kv_heads, head_dim, 16, np_,
                               int(cu_seqlens[-1]) if np_ > 0 else 0, num_decode_seqs,
                               num_blocks, max_blocks_per_seq, scale)
        self.options = Options(num_sms, ctas_per_sm, max_prefill_ctas, decode_splits,
                               prefill_splits, 1 if instrument else 0, VARIANTS[variant],
                               1 if non_causal else 0, 1 if kv_fp8 else 0,
                               1 if kv_fp4 else 0)
        self.variant = variant
        cu = _i32_array(list(cu_seqlens) if np_ > 0 else [0])
        if len(kv_lens) < np_ + num_decode_seqs:  # the library reads one for each sequence
            raise ValueError(f"kv_lens: {len(kv_lens)} for {np_} prefill and {num_decode_seqs} decode "
                             "sequences")
        kv = _i32_array(list(kv_lens))
        handle = ctypes.c_void_p()
        code = lib.pod_attn_plan(ctypes.byref(self.problem), ctypes.cast(cu, ctypes.c_void_p),
                                 ctypes.cast(kv, ctypes.c_void_p), ctypes.byref(self.options),
                                 ctypes.byref(handle))
        _check(code, "pod_attn_plan")
        self.handle = handle

    @classmethod
    def for_batch(cls, batch, variant="fused", **kw) -> "Plan":
        kw.setdefault("non_causal", not getattr(batch, "causal", True))
        kw.setdefault("head_dim", int(batch.head_dim))
        return cls(batch.num_q_heads, batch.num_kv_heads, batch.host_cu_seqlens,
                   batch.host_kv_lens, batch.num_decode_seqs, batch.num_blocks,
                   batch.max_blocks_per_seq, batch.scale, variant=variant, **kw)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value and _lib is not None:
            _lib.pod_attn_plan_destroy(h)
            self.handle = None

    @property
    def workspace_bytes(self) -> int:
        return int(load().pod_attn_workspace_bytes(self.handle))

    def info(self) -> dict:
        inf = PlanInfo()
        _check(load().pod_attn_get_plan_info(self.handle, ctypes.byref(inf)), "plan_info")
        return inf.as_dict()

    @functools.cached_property
    def _shapes(self) -> _Shapes:
        return _Shapes(self.problem)

    def items(self):
        """(prefill items [n][8], decode items [n][8], units [n][4]) as lists of lists."""
        lib = load()
        count = ctypes.c_size_t()
        _check(lib.pod_attn_plan_items(self.handle, None, 0, ctypes.byref(count)), "items")
        buf = (ctypes.c_int32 * max(1, count.value))()
        _check(lib.pod_attn_plan_items(self.handle, ctypes.cast(buf, ctypes.c_void_p),
                                       count.value, ctypes.byref(count)), "items")
        inf = self.info()
        flat = list(buf)[:count.value]
        n_p, n_d = inf["num_prefill_items"] * 8, inf["num_decode_items"] * 8
        rows = lambda xs, w: [xs[i:i + w] for i in range(0, len(xs), w)]
        return rows(flat[:n_p], 8), rows(flat[n_p:n_p + n_d], 8), rows(flat[n_p + n_d:], 4)

    def alloc_workspace(self, device="cuda"):
        import torch
        n = max(256, self.workspace_bytes)
        return torch.empty(n, dtype=torch.uint8, device=device)

    def upload(self, workspace, stream=None):
        _check(load().pod_attn_upload(self.handle, workspace.data_ptr(), workspace.numel(),
                                      _stream_ptr(stream)), "pod_attn_upload")

    def run(self, q_prefill, q_decode, k_pool, v_pool, block_tables, cu_seqlens_q, kv_lens,
            o_prefill, o_decode, workspace, stream=None, stream2=None):
        code = load().pod_attn_run(
            self.handle, _ptr(q_prefill), _ptr(q_decode), _ptr(k_pool), _ptr(v_pool),
            _ptr(block_tables), _ptr(cu_seqlens_q), _ptr(kv_lens), _ptr(o_prefill),
            _ptr(o_decode), workspace.data_ptr(), workspace.numel(), _stream_ptr(stream),
            _stream_ptr(stream2) if stream2 is not None else None)
        _check(code, "pod_attn_run")

    def bucket(self) -> dict:
        """pod_attn_plan_bucket: the plan's resource features and buckets."""
        b = Bucket()
        _check(load().pod_attn_plan_bucket(self.handle, ctypes.byref(b)), "pod_attn_plan_bucket")
        return {name: getattr(b, name) for name, _ in Bucket._fields_}

    def run_append(self, q_prefill, q_decode, k_new, v_new, k_pool, v_pool, block_tables,
                   cu_seqlens_q, kv_lens, o_prefill, o_decode, workspace, stream=None,
                   stream2=None):
        """pod_attn_run_append: write the new tokens' K/V rows (`k_new`, `v_new`, bf16
        [T_p + Nd][Hkv][128]) into the pools, then run the attention."""
        code = load().pod_attn_run_append(
            self.handle, _ptr(q_prefill), _ptr(q_decode), _ptr(k_new), _ptr(v_new),
            _ptr(k_pool), _ptr(v_pool), _ptr(block_tables), _ptr(cu_seqlens_q), _ptr(kv_lens),
            _ptr(o_prefill), _ptr(o_decode), workspace.data_ptr(), workspace.numel(),
            _stream_ptr(stream), _stream_ptr(stream2) if stream2 is not None else None)
        _check(code, "pod_attn_run_append")

    def run_decode_fp8(self, q_decode, k_pool8, v_pool8, k_scale, v_scale, block_tables,
                       kv_lens, o_decode, workspace, stream=None):
        """pod_attn_run_decode_fp8: decode over an e4m3 cache with K / V scales."""
        code = load().pod_attn_run_decode_fp8(
            self.handle, _ptr(q_decode), _ptr(k_pool8), _ptr(v_pool8), _ptr(k_scale),
            _ptr(v_scale), _ptr(block_tables), _ptr(kv_lens), _ptr(o_decode),
            workspace.data_ptr(), workspace.numel(), _stream_ptr(stream))
        _check(code, "pod_attn_run_decode_fp8")

    def append_fp8(self, k_new, v_new, k_pool8, v_pool8, k_scale, v_scale, block_tables,
                   workspace, stream=None):
        """pod_attn_append_fp8: quantise one new token per decode into the e4m3 cache."""
        code = load().pod_attn_append_fp8(
            self.handle, _ptr(k_new), _ptr(v_new), _ptr(k_pool8), _ptr(v_pool8), _ptr(k_scale),
            _ptr(v_scale), _ptr(block_tables), workspace.data_ptr(), workspace.numel(),
            _stream_ptr(stream))
        _check(code, "pod_attn_append_fp8")

    def _check_cache(self, cache):
        s = self._shapes
        if cache.heads != s.heads:
            raise ValueError(f"cache of {cache.num_kv_heads} heads x {cache.head_dim}, plan of "
                             f"{s.heads[0]} x {s.heads[1]}")
        return s, cache.index

    def rope_append(self, rope, q, k_new, v_new, cache, block_tables, q_prefill, q_decode,
                    workspace, stream=None):
        """pod_attn_rope_append: rotate the new tokens' q and k rows (`rope` None: no rotation) and
        append k and v to `cache` (a KvCache). q [T][Hq][D], k_new, v_new [T][Hkv][D] bf16 may be
        views with any token stride that is a multiple of 8 elements; q None appends only."""
        s, dev = self._check_cache(cache)
        qp = op = od = None
        qs = 0
        if q is not None:
            qp, qs = _rows("q", q, s.q, dev)
            op = _arg("q_prefill", q_prefill, s.bf16, s.q_prefill, dev)
            od = _arg("q_decode", q_decode, s.bf16, s.q_decode, dev)
        kp, ks = _rows("k_new", k_new, s.kv, dev)
        vp, vs = _rows("v_new", v_new, s.kv, dev)
        code = _lib.pod_attn_rope_append(
            self.handle, None if rope is None else rope.handle, qp, qs, kp, ks, vp, vs, cache.ref,
            _arg("block_tables", block_tables, s.i32, s.tables, dev), op, od,
            _workspace(workspace, dev), workspace.numel(), _stream_on(dev, stream))
        if code:
            raise PodAttnError(code, "pod_attn_rope_append")

    def run_decode_fp4(self, q_decode, cache, block_tables, kv_lens, o_decode, workspace,
                       stream=None):
        """pod_attn_run_decode_fp4: decode over a 4-bit cache (a KvCache of type "e2m1")."""
        s, dev = self._check_cache(cache)
        code = _lib.pod_attn_run_decode_fp4(
            self.handle, _arg("q_decode", q_decode, s.bf16, s.q_decode, dev), cache.ref,
            _arg("block_tables", block_tables, s.i32, s.tables, dev),
            _arg("kv_lens", kv_lens, s.i32, s.lens, dev),
            _arg("o_decode", o_decode, s.bf16, s.q_decode, dev), _workspace(workspace, dev),
            workspace.numel(), _stream_on(dev, stream))
        if code:
            raise PodAttnError(code, "pod_attn_run_decode_fp4")

    def expand_fp4(self, cache, block_tables4, k_pool, v_pool, block_tables, kv_lens, workspace,
                   stream=None):
        """pod_attn_expand_fp4: the sequences' rows of a 4-bit cache into bf16 pools with block
        tables of their own (this plan's)."""
        s, dev = self._check_cache(cache)
        code = _lib.pod_attn_expand_fp4(
            self.handle, cache.ref, _arg("block_tables4", block_tables4, s.i32, s.tables, dev),
            _arg("k_pool", k_pool, s.bf16, s.pool, dev),
            _arg("v_pool", v_pool, s.bf16, s.pool, dev),
            _arg("block_tables", block_tables, s.i32, s.tables, dev),
            _arg("kv_lens", kv_lens, s.i32, s.lens, dev), _workspace(workspace, dev),
            workspace.numel(), _stream_on(dev, stream))
        if code:
            raise PodAttnError(code, "pod_attn_expand_fp4")

    def device_status(self, workspace, stream=None) -> int:
        return int(load().pod_attn_last_device_status(self.handle, workspace.data_ptr(),
                                                      _stream_ptr(stream)))

    def records(self, workspace, stream=None):
        lib = load()
        inf = self.info()
        n = inf["num_prefill_items"] + inf["num_decode_items"]
        buf = (ItemRecord * max(1, n))()
        count = ctypes.c_size_t()
        _check(lib.pod_attn_read_records(self.handle, workspace.data_ptr(),
                                         ctypes.cast(buf, ctypes.c_void_p), n,
                                         ctypes.byref(count), _stream_ptr(stream)), "records")
        return [dict(smid=r.smid, kind=r.kind, item=r.item, cta=r.cta, t_start=r.t_start,
                     t_end=r.t_end) for r in buf[:count.value]]


def run_batch(plan: Plan, batch, workspace, o_prefill=None, o_decode=None, stream=None,
              stream2=None):
    """Launch `plan` on the device tensors of `batch`; returns (o_prefill, o_decode)."""
    import torch
    if o_prefill is None:
        o_prefill = torch.empty_like(batch.q_prefill)
    if o_decode is None:
        o_decode = torch.empty_like(batch.q_decode)
    if plan.variant == "streams" and stream2 is None:
        stream2 = _side_stream(batch.q_decode.device)
    plan.run(batch.q_prefill, batch.q_decode, batch.k_pool, batch.v_pool, batch.block_tables,
             batch.cu_seqlens_q, batch.kv_lens, o_prefill, o_decode, workspace, stream=stream,
             stream2=stream2)
    return o_prefill, o_decode


_side = {}


def _side_stream(device):
    import torch
    key = str(device)
    if key not in _side:
        _side[key] = torch.cuda.Stream(device=device)
    return _side[key]


def hybrid_attention(batch, variant: str = "fused", check_status: bool = True, **plan_kw):
    """One-call helper: plan, allocate a workspace, upload, run; returns (o_prefill, o_decode).

    `batch` holds device tensors (see ``workloads.HybridBatch``)."""
    plan = Plan.for_batch(batch, variant=variant, **plan_kw)
    ws = plan.alloc_workspace(batch.k_pool.device)
    plan.upload(ws)
    out = run_batch(plan, batch, ws)
    if check_status:
        _check(plan.device_status(ws), "device status")
    return out


def selftest_timeout(workspace, timeout_us: int, stream=None) -> int:
    """Run the bounded-wait self-test kernel; returns the device status it leaves (expected
    ERR_TIMEOUT)."""
    lib = load()
    _check(lib.pod_attn_selftest_timeout(workspace.data_ptr(), int(timeout_us),
                                         _stream_ptr(stream)), "selftest_timeout")
    return int(lib.pod_attn_last_device_status(None, workspace.data_ptr(), _stream_ptr(stream)))


def decode_fp8(fb, workspace=None, stream=None, **plan_kw):
    """Run the FP8-cache decode on an ``workloads.Fp8DecodeBatch`` whose tensors are on the GPU;
    returns o_decode (bf16 [Nd][Hq][128])."""
    import torch
    plan = Plan(fb.num_q_heads, fb.num_kv_heads, [], list(fb.decode_kv_lens),
                fb.num_decode_seqs, fb.num_blocks, fb.max_blocks_per_seq, fb.scale, kv_fp8=True,
                **plan_kw)
    ws = workspace if workspace is not None else plan.alloc_workspace(fb.q_decode.device)
    plan.upload(ws, stream)
    out = torch.empty_like(fb.q_decode)
    plan.run_decode_fp8(fb.q_decode, fb.k8, fb.v8, fb.k_scale, fb.v_scale, fb.block_tables,
                        fb.kv_lens, out, ws, stream=stream)
    st = plan.device_status(ws, stream)
    if st != OK:
        raise PodAttnError(st, "pod_attn_run_decode_fp8 (device)")
    return out
