"""Thin Python binding of libhpcdecode.so (C ABI declared in include/hpc_decode.h).

This module only marshals arguments. It checks tensor dtypes and devices and passes
``data_ptr()`` and the current CUDA stream to the library. Every step of the decode path
runs in the library's kernels. If the library is missing, importing this module raises
``HpcError``: there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
from dataclasses import dataclass

import numpy as np
import torch

from .build import LIB

HPC_OK, HPC_ERR_ARG, HPC_ERR_SHAPE, HPC_ERR_DTYPE, HPC_ERR_ALIGN, HPC_ERR_CUDA, HPC_ERR_CAPACITY = range(7)
HPC_BF16, HPC_FP32, HPC_E4M3 = 0, 1, 2
HPC_HND, HPC_NHD = 0, 1
_LAYOUTS = {"HND": HPC_HND, "NHD": HPC_NHD}
DEV_STATUS = {"bad_seqlen": 0x1, "bad_page": 0x2, "capacity": 0x4, "timeout": 0x8, "bad_index": 0x10,
              "bad_probs": 0x20}
ITEM_DTYPE = np.dtype([("req", "<i4"), ("kv_head", "<i2"), ("flags", "<i2"),
                       ("tile_begin", "<i4"), ("tile_end", "<i4")])
ITEM_DIRECT, ITEM_SECOND_SLOT = 1, 2
RECORD_DTYPE = np.dtype([("unit_begin", "<i8"), ("unit_end", "<i8"), ("chunk", "<i8"), ("item_cost", "<i4"),
                         ("n_items", "<i4")])
ITEM_COST_DEFAULT, ITEM_COST_MAX = -1, 1024
E4M3_KERNELS = {"mma": 0, "tcgen05": 1}
MULTI_KERNELS = {"default": 0, "mma": 1, "tcgen05": 2}
TRACE_WORDS = 8
BUILD_TRACE = 1

EXPORTS = ("hpc_step_record_bytes", "hpc_build_flags", "hpc_plan_workspace_bytes", "hpc_plan_static_workspace_bytes", "hpc_decode_plan",
           "hpc_decode_plan_static", "hpc_plan_cpu", "hpc_partial_o_bytes", "hpc_partial_ml_bytes",
           "hpc_decode_attention", "hpc_merge_states", "hpc_decode_prologue", "hpc_attention_launch_info",
           "hpc_status_string", "hpc_last_error", "hpc_abi_version", "hpc_decode_step_noalloc",
           "hpc_decode_step", "hpc_decode_step_workspace_bytes", "hpc_decode_step_prologue",
           "hpc_decode_step_multi", "hpc_decode_step_multi_workspace_bytes", "hpc_decode_step_lse",
           "hpc_merge_lse", "hpc_wait_selftest", "hpc_merge_lse_gather", "hpc_gather_rows", "hpc_gather_pages",
           "hpc_prompt_prologue", "hpc_verify_drafts", "hpc_pages_resize", "hpc_pages_fork", "hpc_pages_compact",
           "hpc_pages_copy", "hpc_prompt_attention", "hpc_prompt_attention_paged",
           "hpc_prompt_attention_partial_bytes", "hpc_gather_tokens", "hpc_gather_prompt_tokens")


class HpcError(RuntimeError):
    pass


class CPlan(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("tile_len", ctypes.c_int32),
                ("num_ctas", ctypes.c_int32), ("max_items", ctypes.c_int32), ("merge_capacity", ctypes.c_int32),
                ("is_static", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("counts", ctypes.c_void_p), ("items", ctypes.c_void_p), ("cta_indptr", ctypes.c_void_p),
                ("merge_indptr", ctypes.c_void_p), ("merge_list", ctypes.c_void_p)]


class COptions(ctypes.Structure):
    _fields_ = [("item_cost", ctypes.c_int32), ("e4m3_kernel", ctypes.c_int32), ("record", ctypes.c_void_p),
                ("record_items", ctypes.c_int32), ("multi_kernel", ctypes.c_int32), ("trace", ctypes.c_void_p),
                ("seq_lens_ready", ctypes.c_int32)]


_path = LIB


def library_path() -> str:
    return _path


def _load(path=LIB):
    if not os.path.exists(path):
        raise HpcError(f"{path} is missing; build it with `python -m load_balanced_split_step_b200.build` "
                       "(there is no CPU fallback)")
    lib = ctypes.CDLL(path)
    i32, i64, vp, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
    fp = ctypes.c_float
    P = ctypes.POINTER(CPlan)
    O = ctypes.POINTER(COptions)
    sig = {
        "hpc_step_record_bytes": (sz, [i32, i32]),
        "hpc_build_flags": (ctypes.c_uint32, []),
        "hpc_plan_workspace_bytes": (sz, [i32, i32, i32]),
        "hpc_plan_static_workspace_bytes": (sz, [i32, i32, i32]),
        "hpc_decode_plan": (ctypes.c_int, [vp, i32, i32, i32, i32, i32, i32, vp, sz, P, vp, vp]),
        "hpc_decode_plan_static": (ctypes.c_int, [vp, i32, i32, i32, i32, i32, i32, vp, sz, P, vp, vp]),
        "hpc_plan_cpu": (ctypes.c_int, [vp, i32, i32, i32, i32, i32, i32, vp, sz, P, vp]),
        "hpc_partial_o_bytes": (sz, [P, i32, i32]),
        "hpc_partial_ml_bytes": (sz, [P, i32]),
        "hpc_decode_attention": (ctypes.c_int, [vp, vp, vp, ctypes.c_int, ctypes.c_int, vp, vp, i32, i32, i32, i32, i32,
                                                vp, i32, vp, P, fp, vp, vp, vp, ctypes.c_int, O, vp, vp]),
        "hpc_merge_states": (ctypes.c_int, [vp, vp, P, i32, i32, vp, ctypes.c_int, vp, vp]),
        "hpc_decode_prologue": (ctypes.c_int, [vp, vp, vp, fp, fp, vp, vp, vp, ctypes.c_int, ctypes.c_int, vp, vp, i32,
                                               i32, vp, i32, vp, i32, i32, i32, i32, vp, vp]),
        "hpc_attention_launch_info": (ctypes.c_int, [i32, ctypes.c_int, i32, i32, i32, i32, ctypes.POINTER(i32),
                                                     ctypes.POINTER(i32), ctypes.POINTER(i32)]),
        "hpc_decode_step_noalloc": (ctypes.c_int, [vp, vp, vp, ctypes.c_int, vp, vp, i32, i32, i32, i32, i32, vp,
                                                   i32, vp, i32, i32, i32, fp, vp, ctypes.c_int, vp, vp]),
        "hpc_decode_step_workspace_bytes": (sz, [i32, i32, i32, i32, i32]),
        "hpc_decode_step": (ctypes.c_int, [vp, vp, vp, ctypes.c_int, ctypes.c_int, vp, vp, i32, i32, i32, i32, i32, vp,
                                           i32, vp, i32, i32, i32, fp, vp, sz, vp, ctypes.c_int, O, vp, vp]),
        "hpc_decode_step_prologue": (ctypes.c_int, [vp, vp, vp, fp, fp, vp, vp, ctypes.c_int, ctypes.c_int, vp, vp,
                                                    i32, i32, i32, i32, i32, vp, i32, vp, i32, i32, i32, fp, vp, sz,
                                                    vp, ctypes.c_int, O, vp, vp]),
        "hpc_decode_step_multi_workspace_bytes": (sz, [i32, i32, i32, i32, i32, i32]),
        "hpc_decode_step_multi": (ctypes.c_int, [vp, i32, vp, vp, ctypes.c_int, ctypes.c_int, vp, vp, i32, i32, i32,
                                                 i32, i32, vp, i32, vp, i32, i32, i32, fp, vp, sz, vp, ctypes.c_int, O,
                                                 vp, vp]),
        "hpc_decode_step_lse": (ctypes.c_int, [vp, vp, vp, ctypes.c_int, ctypes.c_int, vp, vp, i32, i32, i32, i32, i32,
                                               vp, i32, vp, i32, i32, i32, fp, vp, sz, vp, ctypes.c_int, vp, O, vp, vp]),
        "hpc_merge_lse": (ctypes.c_int, [vp, vp, i32, ctypes.c_int64, i32, vp, vp, vp]),
        "hpc_wait_selftest": (ctypes.c_int, [ctypes.c_uint64, i32, vp, vp, vp]),
        "hpc_merge_lse_gather": (ctypes.c_int, [vp, vp, ctypes.c_int64, vp, i32, i32, i32, i32, vp, vp, vp, vp]),
        "hpc_gather_rows": (ctypes.c_int, [vp, ctypes.c_int64, ctypes.c_int64, vp, ctypes.c_int64, vp, vp, vp]),
        "hpc_gather_pages": (ctypes.c_int, [vp, i32, i32, vp, vp, i32, i32, vp, vp, vp]),
        "hpc_prompt_prologue": (ctypes.c_int, [vp, ctypes.c_int64, vp, i32, vp, vp, fp, fp, vp, vp, vp, vp, ctypes.c_int,
                                               ctypes.c_int, vp, vp, i32, i32, vp, i32, vp, i32, i32, i32, vp, vp]),
        "hpc_verify_drafts": (ctypes.c_int, [vp, vp, ctypes.c_int64, vp, ctypes.c_int64, ctypes.c_int, vp, vp, vp, i32,
                                             i32, i32, vp, vp, vp, vp, vp]),
        "hpc_pages_resize": (ctypes.c_int, [vp, vp, i32, i32, i32, vp, vp, vp, vp, i32, vp, i32, vp, vp, vp]),
        "hpc_pages_fork": (ctypes.c_int, [vp, vp, i32, vp, vp, vp, i32, i32, i32, vp, vp, i32, vp, i32, vp, vp, vp]),
        "hpc_pages_compact": (ctypes.c_int, [vp, vp, i32, i32, vp, vp, i32, vp, vp, i32, vp, vp, vp]),
        "hpc_pages_copy": (ctypes.c_int, [ctypes.POINTER(vp), i32, ctypes.c_int64, i32, vp, i32, vp, vp, vp]),
        "hpc_prompt_attention": (ctypes.c_int, [vp, i64, i64, vp, i64, i64, vp, i64, i64, i64, i64, vp, vp, i32, i32, i32,
                                                i32, i32, fp, vp, vp, vp, vp, sz, vp, vp]),
        "hpc_prompt_attention_partial_bytes": (sz, [i32]),
        "hpc_gather_tokens": (ctypes.c_int, [vp, vp, ctypes.c_int, ctypes.c_int, vp, vp, i32, i32, vp, i32, vp, i32, i32,
                                             i32, i64, vp, vp, vp, vp, vp]),
        "hpc_gather_prompt_tokens": (ctypes.c_int, [vp, vp, ctypes.c_int, ctypes.c_int, vp, vp, i32, i32, vp, i32, vp, vp,
                                                    i32, i32, i32, i64, vp, vp, vp, vp, vp]),
        "hpc_prompt_attention_paged": (ctypes.c_int, [vp, i64, i64, vp, vp, ctypes.c_int, ctypes.c_int, i32, i32, vp, i32,
                                                      vp, i64, vp, i32, i32, i32, i32, fp, vp, vp, vp, vp, sz, vp, vp]),
        "hpc_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "hpc_last_error": (ctypes.c_char_p, []),
        "hpc_abi_version": (ctypes.c_int, []),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    return lib


try:  # the short way in for calls in the common form; without it every call goes the long way
    from . import _fastcall as _fast
except ImportError:
    _fast = None
_status_word = None if _fast is None else _fast.status_word
_FAST_CALLS = ("hpc_prompt_prologue", "hpc_prompt_attention", "hpc_prompt_attention_paged", "hpc_verify_drafts",
               "hpc_pages_resize", "hpc_pages_fork", "hpc_pages_compact", "hpc_pages_copy",
               "hpc_prompt_attention_partial_bytes")


def _bind(lib):
    if _fast is not None:
        _fast.bind(_check, *(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in _FAST_CALLS))
    return lib


def use_library(path: str = LIB):
    """Switch this module to another build of the library (e.g. the HPC_TRACE build, see
    ``build.build(trace=True)``); ``use_library()`` goes back to the default build."""
    global _lib, _path
    _lib = _bind(_load(path))
    _path = path


def build_flags() -> int:
    return int(_lib.hpc_build_flags())


def status_string(code: int) -> str:
    return _lib.hpc_status_string(code).decode()


def _check(rc: int, what: str):
    if rc != HPC_OK:
        raise HpcError(f"{what}: {status_string(rc)} ({rc}): {_lib.hpc_last_error().decode()}")


_lib = _bind(_load())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(t, name, dtype=None, device=None, cuda=True):
    if not isinstance(t, torch.Tensor):
        raise HpcError(f"{name} must be a torch.Tensor")
    if cuda and not t.is_cuda:
        raise HpcError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise HpcError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise HpcError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise HpcError(f"{name} must be contiguous")


def new_status(device) -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device)


@dataclass
class Plan:
    """A plan bound to its workspace. ``raw`` is the C struct passed to the library."""

    raw: CPlan
    workspace: torch.Tensor
    host: bool = False

    @property
    def num_ctas(self) -> int:
        return int(self.raw.num_ctas)

    @property
    def max_items(self) -> int:
        return int(self.raw.max_items)

    def _view(self, ptr, dtype, count):
        base = self.workspace.data_ptr()
        off = int(ptr) - base
        nbytes = np.dtype(dtype).itemsize * count
        return self.workspace[off:off + nbytes]

    def to_numpy(self) -> dict:
        """Copy the plan to host: counts, the valid items, and the index arrays."""
        r = self.raw
        counts = self._view(r.counts, np.int64, 4).cpu().numpy().view(np.int64)
        n_items, n_merge = int(counts[0]), int(counts[1])
        items = self._view(r.items, ITEM_DTYPE, n_items).cpu().numpy().view(ITEM_DTYPE)
        segs = r.batch * r.kv_heads
        return {
            "n_items": n_items, "n_merge": n_merge, "n_units": int(counts[2]), "chunk": int(counts[3]),
            "items": items,
            "cta_indptr": self._view(r.cta_indptr, np.int32, r.num_ctas + 1).cpu().numpy().view(np.int32),
            "merge_indptr": self._view(r.merge_indptr, np.int32, segs + 1).cpu().numpy().view(np.int32),
            "merge_list": self._view(r.merge_list, np.int32, n_merge).cpu().numpy().view(np.int32),
        }


def plan(seq_lens: torch.Tensor, num_heads: int, kv_heads: int, tile_len: int, num_ctas: int | None = None,
         max_seq_len: int = 0, status: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> Plan:
    """Load-balanced per-step plan on the device (``hpc_decode_plan``)."""
    _need(seq_lens, "seq_lens", torch.int32)
    dev = seq_lens.device
    if num_ctas is None:
        num_ctas = torch.cuda.get_device_properties(dev).multi_processor_count
    B = seq_lens.numel()
    nbytes = _lib.hpc_plan_workspace_bytes(B, kv_heads, num_ctas)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    status = new_status(dev) if status is None else status
    raw = CPlan()
    with torch.cuda.device(dev):
        _check(_lib.hpc_decode_plan(_ptr(seq_lens), B, num_heads, kv_heads, tile_len, num_ctas, max_seq_len,
                                    _ptr(workspace), workspace.numel(), ctypes.byref(raw), _ptr(status),
                                    _stream(dev)), "hpc_decode_plan")
    return Plan(raw, workspace)


def plan_static(seq_lens: torch.Tensor, num_heads: int, kv_heads: int, tile_len: int, splits: int,
                max_seq_len: int = 0, status: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None) -> Plan:
    """Static split-k plan on the device (``hpc_decode_plan_static``)."""
    _need(seq_lens, "seq_lens", torch.int32)
    dev = seq_lens.device
    B = seq_lens.numel()
    nbytes = _lib.hpc_plan_static_workspace_bytes(B, kv_heads, splits)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    status = new_status(dev) if status is None else status
    raw = CPlan()
    with torch.cuda.device(dev):
        _check(_lib.hpc_decode_plan_static(_ptr(seq_lens), B, num_heads, kv_heads, tile_len, splits, max_seq_len,
                                           _ptr(workspace), workspace.numel(), ctypes.byref(raw), _ptr(status),
                                           _stream(dev)), "hpc_decode_plan_static")
    return Plan(raw, workspace)


def plan_host(seq_lens, num_heads: int, kv_heads: int, tile_len: int, num_ctas: int,
              max_seq_len: int = 0) -> tuple[Plan, int]:
    """Host twin of ``plan`` (``hpc_plan_cpu``). Returns (plan, status word)."""
    lens = torch.as_tensor(seq_lens, dtype=torch.int32).contiguous().cpu()
    B = lens.numel()
    nbytes = _lib.hpc_plan_workspace_bytes(B, kv_heads, num_ctas)
    # 256-byte aligned host buffer
    buf = torch.empty(nbytes + 256, dtype=torch.uint8)
    off = (-buf.data_ptr()) % 256
    ws = buf[off:off + nbytes]
    st = ctypes.c_uint32(0)
    raw = CPlan()
    _check(_lib.hpc_plan_cpu(_ptr(lens), B, num_heads, kv_heads, tile_len, num_ctas, max_seq_len, _ptr(ws),
                             nbytes, ctypes.byref(raw), ctypes.byref(st)), "hpc_plan_cpu")
    p = Plan(raw, ws, host=True)
    p._keep = buf
    return p, int(st.value)


def partial_buffers(p: Plan, num_heads: int, head_dim: int, device):
    no = _lib.hpc_partial_o_bytes(ctypes.byref(p.raw), num_heads, head_dim) // 4
    nml = _lib.hpc_partial_ml_bytes(ctypes.byref(p.raw), num_heads) // 4
    return (torch.empty(max(no, 4), dtype=torch.float32, device=device),
            torch.empty(max(nml, 4), dtype=torch.float32, device=device))


_KV_DTYPES = {"bf16": HPC_BF16, "e4m3": HPC_E4M3}


def _kv_code(kv_dtype: str, t: torch.Tensor) -> int:
    if kv_dtype not in _KV_DTYPES:
        raise HpcError(f"kv_dtype must be one of {list(_KV_DTYPES)}")
    want = (torch.bfloat16,) if kv_dtype == "bf16" else (torch.uint8, torch.float8_e4m3fn)
    if t.dtype not in want:
        raise HpcError(f"cache dtype {t.dtype} does not match kv_dtype {kv_dtype}")
    return _KV_DTYPES[kv_dtype]


def _geometry(k_pages, kv_layout):
    """(num_pages, kv_heads, page_size, head_dim, layout code) of a cache tensor."""
    if kv_layout not in _LAYOUTS:
        raise HpcError(f"kv_layout must be one of {list(_LAYOUTS)}")
    if k_pages.dim() != 4:
        raise HpcError("cache must be 4-D")
    if kv_layout == "HND":
        n, hkv, psz, d = k_pages.shape
    else:
        n, psz, hkv, d = k_pages.shape
    return n, hkv, psz, d, _LAYOUTS[kv_layout]


def _cache(k_pages, v_pages, kv_dtype, kv_layout, k_scale, v_scale, head_dim, dev):
    """Checks the two caches against each other, the query's head_dim and the device, and the
    E4M3 scales. Returns (dtype code, num_pages, kv_heads, page_size, layout code)."""
    _need(k_pages, "k_pages", device=dev)
    _need(v_pages, "v_pages", device=dev)
    code = _kv_code(kv_dtype, k_pages)
    _kv_code(kv_dtype, v_pages)
    num_pages, Hkv, P, D, lay = _geometry(k_pages, kv_layout)
    if tuple(v_pages.shape) != tuple(k_pages.shape):
        raise HpcError(f"v_pages {tuple(v_pages.shape)} and k_pages {tuple(k_pages.shape)} differ")
    if D != head_dim:
        raise HpcError(f"cache head_dim {D} does not match the query's {head_dim}")
    if code == HPC_E4M3:
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            _need(t, name, torch.float32, dev)
            if t.numel() != Hkv:
                raise HpcError(f"{name} must hold one scale per kv head ({Hkv})")
    return code, num_pages, Hkv, P, lay


def _tables(block_table, seq_lens, batch, dev):
    _need(block_table, "block_table", torch.int32, dev)
    _need(seq_lens, "seq_lens", torch.int32, dev)
    if block_table.dim() != 2 or block_table.shape[0] != batch or seq_lens.numel() != batch:
        raise HpcError(f"block_table [batch, pages] and seq_lens [batch] must match the batch of {batch}")


def _output(out, shape, out_dtype, dev):
    if out is None:
        return torch.empty(shape, dtype=out_dtype, device=dev)
    _need(out, "out", (torch.float32, torch.bfloat16), dev)
    if tuple(out.shape) != tuple(shape):
        raise HpcError(f"out has shape {tuple(out.shape)}, expected {tuple(shape)}")
    return out


def _out_code(out):
    return HPC_BF16 if out.dtype == torch.bfloat16 else HPC_FP32


def options(item_cost=None, e4m3_kernel="mma", record=None, record_items=0, trace=None, device=None, num_ctas=None,
            multi_kernel="default", seq_lens_ready=False):
    """A ``hpc_step_options`` struct, or None when every option has its default.
    item_cost: 1/16 tile per item start (None: the library's default). e4m3_kernel: "mma" or
    "tcgen05". record: uint8 device tensor of ``record_bytes(num_ctas, record_items)`` bytes.
    trace: int64 device tensor [num_ctas, TRACE_WORDS] (HPC_TRACE builds only).
    seq_lens_ready: the kernel launched just before on the stream does not write seq_lens, so the
    single-launch step may plan before waiting for it."""
    if e4m3_kernel not in E4M3_KERNELS:
        raise HpcError(f"e4m3_kernel must be one of {list(E4M3_KERNELS)}")
    if multi_kernel not in MULTI_KERNELS:
        raise HpcError(f"multi_kernel must be one of {list(MULTI_KERNELS)}")
    if (item_cost is None and e4m3_kernel == "mma" and record is None and trace is None and multi_kernel == "default"
            and not seq_lens_ready):
        return None
    o = COptions()
    o.seq_lens_ready = 1 if seq_lens_ready else 0
    o.item_cost = ITEM_COST_DEFAULT if item_cost is None else int(item_cost)
    o.e4m3_kernel = E4M3_KERNELS[e4m3_kernel]
    o.multi_kernel = MULTI_KERNELS[multi_kernel]
    if record is not None:
        _need(record, "record", torch.uint8, device)
        o.record, o.record_items = record.data_ptr(), int(record_items)
        if num_ctas is not None and record.numel() < record_bytes(num_ctas, record_items):
            raise HpcError(f"record holds {record.numel()} bytes, {record_bytes(num_ctas, record_items)} needed")
    if trace is not None:
        _need(trace, "trace", torch.int64, device)
        if num_ctas is not None and trace.numel() < num_ctas * TRACE_WORDS:
            raise HpcError(f"trace must hold num_ctas x {TRACE_WORDS} words")
        o.trace = trace.data_ptr()
    return o


def _opt_ref(o):
    return None if o is None else ctypes.byref(o)


def record_bytes(num_ctas: int, record_items: int) -> int:
    return int(_lib.hpc_step_record_bytes(num_ctas, record_items))


def read_record(record: torch.Tensor, num_ctas: int, record_items: int):
    """The per-CTA records of a single-launch step: (headers RECORD_DTYPE [G], items list of
    ITEM_DTYPE arrays, the first min(n_items, record_items) of each CTA)."""
    raw = record.cpu().numpy()
    stride = RECORD_DTYPE.itemsize + record_items * ITEM_DTYPE.itemsize
    heads = np.empty(num_ctas, dtype=RECORD_DTYPE)
    items = []
    for g in range(num_ctas):
        blk = raw[g * stride:(g + 1) * stride]
        heads[g] = blk[:RECORD_DTYPE.itemsize].view(RECORD_DTYPE)[0]
        n = min(int(heads[g]["n_items"]), record_items)
        items.append(blk[RECORD_DTYPE.itemsize:RECORD_DTYPE.itemsize + n * ITEM_DTYPE.itemsize].view(ITEM_DTYPE))
    return heads, items


def attention(q, k_pages, v_pages, block_table, seq_lens, p: Plan, *, kv_dtype="bf16", kv_layout="HND",
              k_scale=None, v_scale=None, sm_scale=None, out=None, out_dtype=torch.float32, partial_o=None,
              partial_ml=None, status=None, e4m3_kernel="mma", trace=None):
    """Persistent split-KV attention (``hpc_decode_attention``). Returns (out, partial_o, partial_ml)."""
    _need(q, "q", torch.bfloat16)
    dev = q.device
    B, Hq, D = q.shape
    code, num_pages, Hkv, P, lay = _cache(k_pages, v_pages, kv_dtype, kv_layout, k_scale, v_scale, D, dev)
    _tables(block_table, seq_lens, B, dev)
    out = _output(out, (B, Hq, D), out_dtype, dev)
    if partial_o is None or partial_ml is None:
        partial_o, partial_ml = partial_buffers(p, Hq, D, dev)
    status = new_status(dev) if status is None else status
    scale = 1.0 / math.sqrt(D) if sm_scale is None else float(sm_scale)
    opt = options(e4m3_kernel=e4m3_kernel, trace=trace, device=dev, num_ctas=p.num_ctas)
    with torch.cuda.device(dev):
        _check(_lib.hpc_decode_attention(
            _ptr(q), _ptr(k_pages), _ptr(v_pages), code, lay, _ptr(k_scale), _ptr(v_scale), num_pages, P, Hq, Hkv, D,
            _ptr(block_table), block_table.shape[1], _ptr(seq_lens), ctypes.byref(p.raw), scale, _ptr(partial_o),
            _ptr(partial_ml), _ptr(out), _out_code(out), _opt_ref(opt), _ptr(status), _stream(dev)),
            "hpc_decode_attention")
    return out, partial_o, partial_ml


def merge(p: Plan, partial_o, partial_ml, out, num_heads: int, status=None):
    """Log-sum-exp merge of split (request, kv head) pairs (``hpc_merge_states``)."""
    dev = out.device
    _need(partial_o, "partial_o", torch.float32, dev)
    _need(partial_ml, "partial_ml", torch.float32, dev)
    _need(out, "out", (torch.float32, torch.bfloat16), dev)
    status = new_status(dev) if status is None else status
    D = out.shape[-1]
    with torch.cuda.device(dev):
        _check(_lib.hpc_merge_states(_ptr(partial_o), _ptr(partial_ml), ctypes.byref(p.raw), num_heads, D, _ptr(out),
                                     HPC_BF16 if out.dtype == torch.bfloat16 else HPC_FP32, _ptr(status),
                                     _stream(dev)), "hpc_merge_states")
    return out


def prologue(qkv, q_norm_w, k_norm_w, k_pages, v_pages, block_table, seq_lens, num_heads, kv_heads, *,
             kv_dtype="bf16", kv_layout="HND", k_scale=None, v_scale=None, eps=1e-6, rope_theta=1e6, q_out=None,
             status=None):
    """Fused RMSNorm + RoPE + KV-page write of the new token (``hpc_decode_prologue``). Returns q_out."""
    _need(qkv, "qkv", torch.bfloat16)
    dev = qkv.device
    _need(q_norm_w, "q_norm_w", torch.float32, dev)
    _need(k_norm_w, "k_norm_w", torch.float32, dev)
    B, H, D = qkv.shape
    if H != num_heads + 2 * kv_heads:
        raise HpcError("qkv must hold num_heads + 2*kv_heads heads")
    if q_norm_w.numel() != D or k_norm_w.numel() != D:
        raise HpcError("norm weights must hold head_dim values")
    code, num_pages, Hkv, P, lay = _cache(k_pages, v_pages, kv_dtype, kv_layout, k_scale, v_scale, D, dev)
    if Hkv != kv_heads:
        raise HpcError(f"cache has {Hkv} kv heads, expected {kv_heads}")
    _tables(block_table, seq_lens, B, dev)
    if q_out is None:
        q_out = torch.empty((B, num_heads, D), dtype=torch.bfloat16, device=dev)
    _need(q_out, "q_out", torch.bfloat16, dev)
    if tuple(q_out.shape) != (B, num_heads, D):
        raise HpcError("q_out must be [batch, num_heads, head_dim]")
    status = new_status(dev) if status is None else status
    with torch.cuda.device(dev):
        _check(_lib.hpc_decode_prologue(
            _ptr(qkv), _ptr(q_norm_w), _ptr(k_norm_w), float(eps), float(rope_theta), _ptr(q_out), _ptr(k_pages),
            _ptr(v_pages), code, lay, _ptr(k_scale), _ptr(v_scale), num_pages, P, _ptr(block_table),
            block_table.shape[1], _ptr(seq_lens), B, num_heads, kv_heads, D, _ptr(status), _stream(dev)),
            "hpc_decode_prologue")
    return q_out


def step_workspace(batch, num_heads, kv_heads, head_dim, num_ctas, device):
    """Zeroed workspace for ``decode_step_fused`` (its merge tickets must start at zero)."""
    n = _lib.hpc_decode_step_workspace_bytes(batch, num_heads, kv_heads, head_dim, num_ctas)
    if n == 0:
        raise HpcError("bad shape for hpc_decode_step_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def _grid(num_ctas, dev):
    return torch.cuda.get_device_properties(dev).multi_processor_count if num_ctas is None else int(num_ctas)


def _workspace(ws, nbytes, dev):
    if ws is None:
        return torch.zeros(nbytes, dtype=torch.uint8, device=dev)
    _need(ws, "workspace", torch.uint8, dev)
    return ws


def decode_step_fused(q, k_pages, v_pages, block_table, seq_lens, num_heads, kv_heads, tile_len, *,
                      kv_dtype="bf16", kv_layout="HND", k_scale=None, v_scale=None, num_ctas=None, sm_scale=None,
                      out=None, out_dtype=torch.float32, status=None, workspace=None, item_cost=None,
                      e4m3_kernel="mma", record=None, record_items=0, trace=None, seq_lens_ready=False):
    """One decode step in a single launch (``hpc_decode_step``): in-kernel planning, attention
    and ticket merge. Returns (out, status, workspace); pass the workspace back on later calls.
    item_cost, e4m3_kernel, record / record_items, trace and seq_lens_ready are the call's
    options."""
    _need(q, "q", torch.bfloat16)
    dev = q.device
    B, Hq, D = q.shape
    if Hq != num_heads:
        raise HpcError(f"q has {Hq} heads, expected {num_heads}")
    code, num_pages, Hkv, P, lay = _cache(k_pages, v_pages, kv_dtype, kv_layout, k_scale, v_scale, D, dev)
    if Hkv != kv_heads:
        raise HpcError(f"cache has {Hkv} kv heads, expected {kv_heads}")
    _tables(block_table, seq_lens, B, dev)
    G = _grid(num_ctas, dev)
    out = _output(out, (B, Hq, D), out_dtype, dev)
    status = new_status(dev) if status is None else status
    workspace = _workspace(workspace, _lib.hpc_decode_step_workspace_bytes(B, Hq, Hkv, D, G), dev)
    scale = 1.0 / math.sqrt(D) if sm_scale is None else float(sm_scale)
    opt = options(item_cost, e4m3_kernel, record, record_items, trace, dev, G, seq_lens_ready=seq_lens_ready)
    with torch.cuda.device(dev):
        _check(_lib.hpc_decode_step(
            _ptr(q), _ptr(k_pages), _ptr(v_pages), code, lay, _ptr(k_scale), _ptr(v_scale), num_pages, P, Hq, Hkv, D,
            _ptr(block_table), block_table.shape[1], _ptr(seq_lens), B, tile_len, G, scale, _ptr(workspace),
            workspace.numel(), _ptr(out), _out_code(out), _opt_ref(opt), _ptr(status), _stream(dev)),
            "hpc_decode_step")
    return out, status, workspace


def decode_step_prologue(qkv, q_norm_w, k_norm_w, k_pages, v_pages, block_table, seq_lens, num_heads, kv_heads,
                         tile_len, *, kv_dtype="bf16", kv_layout="HND", k_scale=None, v_scale=None, eps=1e-6,
                         rope_theta=1e6, num_ctas=None, sm_scale=None, out=None, out_dtype=torch.float32,
                         status=None, workspace=None, item_cost=None, record=None, record_items=0, trace=None,
                         seq_lens_ready=False):
    """One decode step in a single launch with the prologue folded in
    (``hpc_decode_step_prologue``): the new token's K/V go into the cache and q is formed from
    qkv inside the attention kernel. Returns (out, status, workspace)."""
    _need(qkv, "qkv", torch.bfloat16)
    dev = qkv.device
    _need(q_norm_w, "q_norm_w", torch.float32, dev)
    _need(k_norm_w, "k_norm_w", torch.float32, dev)
    B, H, D = qkv.shape
    if H != num_heads + 2 * kv_heads:
        raise HpcError("qkv must hold num_heads + 2*kv_heads heads")
    if q_norm_w.numel() != D or k_norm_w.numel() != D:
        raise HpcError("norm weights must hold head_dim values")
    code, num_pages, Hkv, P, lay = _cache(k_pages, v_pages, kv_dtype, kv_layout, k_scale, v_scale, D, dev)
    if Hkv != kv_heads:
        raise HpcError(f"cache has {Hkv} kv heads, expected {kv_heads}")
    _tables(block_table, seq_lens, B, dev)
    G = _grid(num_ctas, dev)
    out = _output(out, (B, num_heads, D), out_dtype, dev)
    status = new_status(dev) if status is None else status
    workspace = _workspace(workspace, _lib.hpc_decode_step_workspace_bytes(B, num_heads, Hkv, D, G), dev)
    scale = 1.0 / math.sqrt(D) if sm_scale is None else float(sm_scale)
    opt = options(item_cost, "mma", record, record_items, trace, dev, G, seq_lens_ready=seq_lens_ready)
    with torch.cuda.device(dev):
        _check(_lib.hpc_decode_step_prologue(
            _ptr(qkv), _ptr(q_norm_w), _ptr(k_norm_w), float(eps), float(rope_theta), _ptr(k_pages), _ptr(v_pages),
            code, lay, _ptr(k_scale), _ptr(v_scale), num_pages, P, num_heads, Hkv, D, _ptr(block_table),
            block_table.shape[1], _ptr(seq_lens), B, tile_len, G, scale, _ptr(workspace), workspace.numel(),
            _ptr(out), _out_code(out), _opt_ref(opt), _ptr(status), _stream(dev)), "hpc_decode_step_prologue")
    return out, status, workspace


def multi_workspace(batch, q_len, num_heads, kv_heads, head_dim, num_ctas, device):
    """Zeroed workspace for ``decode_step_multi``."""
    n = _lib.hpc_decode_step_multi_workspace_bytes(batch, q_len, num_heads, kv_heads, head_dim, num_ctas)
    if n == 0:
        raise HpcError("bad shape for hpc_decode_step_multi_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def decode_step_multi(q, k_pages, v_pages, block_table, seq_lens, kv_heads, tile_len, *, kv_dtype="bf16",
                      kv_layout="HND", k_scale=None, v_scale=None, num_ctas=None, sm_scale=None, out=None,
                      out_dtype=torch.float32, status=None, workspace=None, item_cost=None, record=None,
                      record_items=0, trace=None, multi_kernel="default", seq_lens_ready=False):
    """q_len new tokens per request in one launch (``hpc_decode_step_multi``): q is
    [B, q_len, Hq, D]; query token t of request r sits at position L_r - q_len + t and
    attends causally. multi_kernel: "default", "mma" or "tcgen05". Returns (out [B, q_len, Hq, D],
    status, workspace)."""
    _need(q, "q", torch.bfloat16)
    dev = q.device
    B, T, Hq, D = q.shape
    code, num_pages, Hkv, P, lay = _cache(k_pages, v_pages, kv_dtype, kv_layout, k_scale, v_scale, D, dev)
    if Hkv != kv_heads:
        raise HpcError(f"cache has {Hkv} kv heads, expected {kv_heads}")
    _tables(block_table, seq_lens, B, dev)
    G = _grid(num_ctas, dev)
    out = _output(out, (B, T, Hq, D), out_dtype, dev)
    status = new_status(dev) if status is None else status
    workspace = _workspace(workspace, _lib.hpc_decode_step_multi_workspace_bytes(B, T, Hq, Hkv, D, G), dev)
    scale = 1.0 / math.sqrt(D) if sm_scale is None else float(sm_scale)
    opt = options(item_cost, "mma", record, record_items, trace, dev, G, multi_kernel, seq_lens_ready)
    with torch.cuda.device(dev):
        _check(_lib.hpc_decode_step_multi(
            _ptr(q), T, _ptr(k_pages), _ptr(v_pages), code, lay, _ptr(k_scale), _ptr(v_scale), num_pages, P, Hq, Hkv,
            D, _ptr(block_table), block_table.shape[1], _ptr(seq_lens), B, tile_len, G, scale, _ptr(workspace),
            workspace.numel(), _ptr(out), _out_code(out), _opt_ref(opt), _ptr(status), _stream(dev)),
            "hpc_decode_step_multi")
    return out, status, workspace


def decode_step_lse(q, k_pages, v_pages, block_table, seq_lens, num_heads, kv_heads, tile_len, *, kv_dtype="bf16",
                    kv_layout="HND", k_scale=None, v_scale=None, num_ctas=None, sm_scale=None, out=None, lse=None,
                    status=None, workspace=None, item_cost=None, e4m3_kernel="mma", seq_lens_ready=False):
    """``hpc_decode_step_lse``: the single-launch step, plus the natural-log log-sum-exp of
    every output row. Returns (out fp32 [B, Hq, D], lse fp32 [B, Hq], status, workspace)."""
    _need(q, "q", torch.bfloat16)
    dev = q.device
    B, Hq, D = q.shape
    if Hq != num_heads:
        raise HpcError(f"q has {Hq} heads, expected {num_heads}")
    code, num_pages, Hkv, P, lay = _cache(k_pages, v_pages, kv_dtype, kv_layout, k_scale, v_scale, D, dev)
    if Hkv != kv_heads:
        raise HpcError(f"cache has {Hkv} kv heads, expected {kv_heads}")
    _tables(block_table, seq_lens, B, dev)
    G = _grid(num_ctas, dev)
    out = _output(out, (B, Hq, D), torch.float32, dev)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=dev) if lse is None else lse
    _need(lse, "lse", torch.float32, dev)
    if tuple(lse.shape) != (B, Hq):
        raise HpcError("lse must be [batch, num_heads]")
    status = new_status(dev) if status is None else status
    workspace = _workspace(workspace, _lib.hpc_decode_step_workspace_bytes(B, Hq, Hkv, D, G), dev)
    scale = 1.0 / math.sqrt(D) if sm_scale is None else float(sm_scale)
    opt = options(item_cost, e4m3_kernel, device=dev, seq_lens_ready=seq_lens_ready)
    with torch.cuda.device(dev):
        _check(_lib.hpc_decode_step_lse(
            _ptr(q), _ptr(k_pages), _ptr(v_pages), code, lay, _ptr(k_scale), _ptr(v_scale), num_pages, P, Hq, Hkv, D,
            _ptr(block_table), block_table.shape[1], _ptr(seq_lens), B, tile_len, G, scale, _ptr(workspace),
            workspace.numel(), _ptr(out), _out_code(out), _ptr(lse), _opt_ref(opt), _ptr(status), _stream(dev)),
            "hpc_decode_step_lse")
    return out, lse, status, workspace


def merge_lse(outs, lses, out=None, lse_out=None):
    """``hpc_merge_lse``: outs fp32 [parts, rows..., D], lses fp32 [parts, rows...] -> (out, lse)."""
    _need(outs, "outs", torch.float32)
    dev = outs.device
    _need(lses, "lses", torch.float32, dev)
    parts, D = outs.shape[0], outs.shape[-1]
    rows = lses[0].numel()
    if outs[0].numel() != rows * D:
        raise HpcError("outs and lses disagree on the rows")
    out = torch.empty(outs.shape[1:], dtype=torch.float32, device=dev) if out is None else out
    lse_out = torch.empty(lses.shape[1:], dtype=torch.float32, device=dev) if lse_out is None else lse_out
    with torch.cuda.device(dev):
        _check(_lib.hpc_merge_lse(_ptr(outs), _ptr(lses), parts, rows, D, _ptr(out), _ptr(lse_out), _stream(dev)),
               "hpc_merge_lse")
    return out, lse_out


def merge_lse_gather(outs, lses, part_index, out=None, lse_out=None, status=None):
    """``hpc_merge_lse_gather``: outs fp32 [part_rows, Hq, D], lses fp32 [part_rows, Hq], part_index
    int32 [B, max_parts] (-1 unused) -> (out [B, Hq, D], lse [B, Hq])."""
    _need(outs, "outs", torch.float32)
    dev = outs.device
    _need(lses, "lses", torch.float32, dev)
    _need(part_index, "part_index", torch.int32, dev)
    rows, Hq, D = outs.shape
    if tuple(lses.shape) != (rows, Hq) or part_index.dim() != 2:
        raise HpcError("outs [rows, Hq, D], lses [rows, Hq] and part_index [B, max_parts] disagree")
    Bn, mp = part_index.shape
    out = torch.empty((Bn, Hq, D), dtype=torch.float32, device=dev) if out is None else out
    lse_out = torch.empty((Bn, Hq), dtype=torch.float32, device=dev) if lse_out is None else lse_out
    _need(out, "out", torch.float32, dev)
    _need(lse_out, "lse_out", torch.float32, dev)
    with torch.cuda.device(dev):
        _check(_lib.hpc_merge_lse_gather(_ptr(outs), _ptr(lses), rows, _ptr(part_index), mp, Bn, Hq, D, _ptr(out),
                                         _ptr(lse_out), _ptr(status), _stream(dev)), "hpc_merge_lse_gather")
    return out, lse_out


def gather_rows(src, index, out=None, status=None):
    """``hpc_gather_rows``: out[j] = src[index[j]] along the first dimension (rows a multiple of 16 bytes)."""
    _need(src, "src")
    dev = src.device
    _need(index, "index", torch.int32, dev)
    n = index.numel()
    out = torch.empty((n,) + tuple(src.shape[1:]), dtype=src.dtype, device=dev) if out is None else out
    _need(out, "out", src.dtype, dev)
    row_bytes = src[0].numel() * src.element_size() if src.shape[0] else out[0].numel() * out.element_size()
    with torch.cuda.device(dev):
        _check(_lib.hpc_gather_rows(_ptr(src), src.shape[0], row_bytes, _ptr(index), n, _ptr(out), _ptr(status),
                                    _stream(dev)), "hpc_gather_rows")
    return out


def gather_pages(block_table, req, col0, width=None, out=None, status=None):
    """``hpc_gather_pages``: out[i][j] = block_table[req[i]][col0[i] + j] (-1 past the table), the
    block-table view of a request-sharded rank's parts. Returns out int32 [n, width]."""
    _need(block_table, "block_table", torch.int32)
    dev = block_table.device
    _need(req, "req", torch.int32, dev)
    _need(col0, "col0", torch.int32, dev)
    if block_table.dim() != 2 or req.numel() != col0.numel():
        raise HpcError("block_table must be 2-D and req / col0 of equal length")
    n = req.numel()
    width = block_table.shape[1] if width is None else int(width)
    out = torch.empty((n, width), dtype=torch.int32, device=dev) if out is None else out
    _need(out, "out", torch.int32, dev)
    if tuple(out.shape) != (n, width):
        raise HpcError("out must be [n, width]")
    with torch.cuda.device(dev):
        _check(_lib.hpc_gather_pages(_ptr(block_table), block_table.shape[0], block_table.shape[1], _ptr(req),
                                     _ptr(col0), n, width, _ptr(out), _ptr(status), _stream(dev)), "hpc_gather_pages")
    return out


def _want(t, name, dtype, dev):
    """``_need`` with its common outcome first: these calls are a few microseconds long."""
    if not (type(t) is torch.Tensor and t.dtype is dtype and t.device == dev and t.is_contiguous()):
        _need(t, name, dtype, dev)


def _empty(shape, dtype, dev):
    n = len(shape)
    strides = (1,) if n == 1 else (shape[1], 1) if n == 2 else (shape[1] * shape[2], shape[2], 1)
    return torch.empty_strided(shape, strides, dtype=dtype, device=dev)


def _packed(cu_seqlens, dev, batch=None):
    """Checks the boundaries of packed prompts; returns the number of requests."""
    _want(cu_seqlens, "cu_seqlens", torch.int32, dev)
    n = cu_seqlens.numel() - 1
    if cu_seqlens.dim() != 1 or n < 1 or (batch is not None and n != batch):
        raise HpcError("cu_seqlens must be [batch + 1]" + ("" if batch is None else f" for a batch of {batch}"))
    return n


def _addr(t):
    return None if t is None else t.data_ptr()


def _status(status, dev):
    """The caller's status word, or a zeroed one: one of those that the short way zeroes 128 at a time, since a memset
    of its own for each call costs as much as a small kernel. A captured call zeroes its own word, at every
    replay."""
    if status is not None:
        _want(status, "status", torch.int32, dev)
        return status
    word = None if _status_word is None else _status_word(dev.index)
    return new_status(dev) if word is None else word


def _launch(name, dev, *args):
    """Calls a library function that ends in a stream, on the current stream of the tensors' device."""
    fn, stream = getattr(_lib, name), torch._C._cuda_getCurrentRawStream(dev.index)
    if torch.cuda.current_device() == dev.index:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, stream)
    if rc != HPC_OK:
        _check(rc, name)


def _buffer(t, name, shape, dtype, dev):
    """An output the caller may hand in."""
    if t is None:
        return _empty(shape, dtype, dev)
    _want(t, name, dtype, dev)
    if t.shape != shape:
        raise HpcError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def prompt_prologue(qkv, cu_seqlens, q_norm_w, k_norm_w, k_pages, v_pages, block_table, seq_lens, num_heads, kv_heads,
                    *, kv_dtype="bf16", kv_layout="HND", k_scale=None, v_scale=None, eps=1e-6, rope_theta=1e6,
                    q_out=None, k_out=None, status=None):
    """RMSNorm + RoPE + KV-page write of every token of packed prompts (``hpc_prompt_prologue``): qkv is
    [tokens, Hq + 2 Hkv, D], request r's tokens are rows cu_seqlens[r] .. cu_seqlens[r + 1] - 1 and the
    last of its seq_lens[r]. Returns (q_out [tokens, Hq, D], k_out [tokens, Hkv, D], status); rows of no
    request are left as they were."""
    if _fast is not None:
        r = _fast.prompt_prologue(qkv, cu_seqlens, q_norm_w, k_norm_w, k_pages, v_pages, block_table, seq_lens, num_heads,
                                  kv_heads, _KV_DTYPES.get(kv_dtype), _LAYOUTS.get(kv_layout), k_scale, v_scale, eps,
                                  rope_theta, q_out, k_out, status)
        if r is not None:
            return r
    _need(qkv, "qkv", torch.bfloat16)
    dev = qkv.device
    _want(q_norm_w, "q_norm_w", torch.float32, dev)
    _want(k_norm_w, "k_norm_w", torch.float32, dev)
    if qkv.dim() != 3 or qkv.shape[1] != num_heads + 2 * kv_heads:
        raise HpcError("qkv must be [tokens, num_heads + 2*kv_heads, head_dim]")
    n, _, D = qkv.shape
    if q_norm_w.numel() != D or k_norm_w.numel() != D:
        raise HpcError("norm weights must hold head_dim values")
    code, num_pages, Hkv, P, lay = _cache(k_pages, v_pages, kv_dtype, kv_layout, k_scale, v_scale, D, dev)
    if Hkv != kv_heads:
        raise HpcError(f"cache has {Hkv} kv heads, expected {kv_heads}")
    batch = _packed(cu_seqlens, dev)
    _tables(block_table, seq_lens, batch, dev)
    q_out = _buffer(q_out, "q_out", (n, num_heads, D), torch.bfloat16, dev)
    k_out = _buffer(k_out, "k_out", (n, kv_heads, D), torch.bfloat16, dev)
    status = _status(status, dev)
    _launch("hpc_prompt_prologue", dev, qkv.data_ptr(), n, cu_seqlens.data_ptr(), batch, q_norm_w.data_ptr(),
            k_norm_w.data_ptr(), float(eps), float(rope_theta), q_out.data_ptr(), k_out.data_ptr(),
            k_pages.data_ptr(), v_pages.data_ptr(), code, lay, _addr(k_scale), _addr(v_scale), num_pages, P,
            block_table.data_ptr(), block_table.shape[1], _addr(seq_lens), num_heads, kv_heads, D, status.data_ptr())
    return q_out, k_out, status


def _strided(t, name, dev):
    """A bf16 [tokens, heads, head_dim] tensor with contiguous heads; returns (token stride, head stride)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or (dev is not None and t.device != dev):
        raise HpcError(f"{name} must be a CUDA tensor" + ("" if dev is None else f" on {dev}"))
    if t.dtype != torch.bfloat16:
        raise HpcError(f"{name} has dtype {t.dtype}, expected {torch.bfloat16}")
    if t.dim() != 3 or t.stride(2) != 1:
        raise HpcError(f"{name} must be [tokens, heads, head_dim] with contiguous heads")
    n, H, D = t.shape
    return (t.stride(0) if n > 1 else H * D), (t.stride(1) if H > 1 else D)


def _lse(lse, return_lse, n, heads, dev):
    if lse is None and not return_lse:
        return None
    return _buffer(lse, "lse", (n, heads), torch.float32, dev)


PROMPT_WORK_WORDS, PROMPT_SPLIT_KEYS = 8, 1536


def _prompt_scratch(max_keys, head_dim, dev):
    """(work, partial, bytes) of one prompt attention call; partial only where sequences can be cut."""
    work = torch.zeros(PROMPT_WORK_WORDS, dtype=torch.int32, device=dev)
    if max_keys <= PROMPT_SPLIT_KEYS:
        return work, None, 0
    with torch.cuda.device(dev):
        nbytes = _lib.hpc_prompt_attention_partial_bytes(head_dim)
    return work, torch.empty(nbytes, dtype=torch.uint8, device=dev), nbytes


def prompt_attention(q, k, v, cu_seqlens, *, cu_seqlens_k=None, causal=True, sm_scale=None, out=None, lse=None,
                     return_lse=False, status=None):
    """Attention of packed prompts (``hpc_prompt_attention``): q [tokens, Hq, D], k / v [kv_tokens, Hkv, D] in
    bf16, possibly views into one qkv tensor; sequence r is rows cu_seqlens[r] .. cu_seqlens[r + 1] - 1 (of k and
    v: cu_seqlens_k, default the same), its queries the last of its keys. Returns (out bf16 [tokens, Hq, D],
    lse fp32 [tokens, Hq] or None, status); rows of no sequence are left as they were."""
    if _fast is not None:
        r = _fast.prompt_attention(q, k, v, cu_seqlens, cu_seqlens_k, causal, sm_scale, out, lse, return_lse, status)
        if r is not None:
            return r
    qs = _strided(q, "q", None)
    dev = q.device
    ks, vs = _strided(k, "k", dev), _strided(v, "v", dev)
    n, Hq, D = q.shape
    if tuple(v.shape) != tuple(k.shape) or k.shape[2] != D:
        raise HpcError(f"k {tuple(k.shape)} and v {tuple(v.shape)} must agree, with the query's head_dim {D}")
    batch = _packed(cu_seqlens, dev)
    if cu_seqlens_k is not None:
        _packed(cu_seqlens_k, dev, batch)
    out = _buffer(out, "out", (n, Hq, D), torch.bfloat16, dev)
    lse = _lse(lse, return_lse, n, Hq, dev)
    status = _status(status, dev)
    scale = 1.0 / math.sqrt(D) if sm_scale is None else float(sm_scale)
    work, partial, nbytes = _prompt_scratch(k.shape[0], D, dev)
    _launch("hpc_prompt_attention", dev, q.data_ptr(), *qs, k.data_ptr(), *ks, v.data_ptr(), *vs, n, k.shape[0],
            cu_seqlens.data_ptr(), _addr(cu_seqlens_k), batch, Hq, k.shape[1], D, 1 if causal else 0, scale,
            out.data_ptr(), _addr(lse), work.data_ptr(), _addr(partial), nbytes, status.data_ptr())
    return out, lse, status


def gather_tokens(k_pages, v_pages, block_table, seq_lens, kv_tokens, *, kv_dtype="bf16", kv_layout="HND", k_scale=None,
                  v_scale=None, k_out=None, v_out=None, cu_seqlens=None, status=None, cu_queries=None):
    """The cached tokens of every request as packed bf16 rows (``hpc_gather_tokens``), kv_tokens rows at most. Returns
    (k, v [kv_tokens, Hkv, D], cu_seqlens int32 [batch + 1], status); rows past cu_seqlens[batch] are left as
    they were. With cu_queries, the boundaries of queries that are the last of those tokens, a request with fewer cached
    tokens than queries is flagged and has no rows (``hpc_gather_prompt_tokens``)."""
    _need(k_pages, "k_pages")
    dev, D = k_pages.device, k_pages.shape[-1]
    code, num_pages, Hkv, P, lay = _cache(k_pages, v_pages, kv_dtype, kv_layout, k_scale, v_scale, D, dev)
    if kv_tokens < 0:
        raise HpcError("kv_tokens must be >= 0")
    _want(seq_lens, "seq_lens", torch.int32, dev)
    batch = seq_lens.numel()
    _tables(block_table, seq_lens, batch, dev)
    k_out = _buffer(k_out, "k_out", (int(kv_tokens), Hkv, D), torch.bfloat16, dev)
    v_out = _buffer(v_out, "v_out", (int(kv_tokens), Hkv, D), torch.bfloat16, dev)
    cu_seqlens = _buffer(cu_seqlens, "cu_seqlens", (batch + 1,), torch.int32, dev)
    queries = ()
    if cu_queries is not None:
        _packed(cu_queries, dev, batch)
        queries = (cu_queries.data_ptr(),)
    status = _status(status, dev)
    _launch("hpc_gather_prompt_tokens" if queries else "hpc_gather_tokens", dev, k_pages.data_ptr(), v_pages.data_ptr(), code,
            lay, _addr(k_scale), _addr(v_scale), num_pages, P, block_table.data_ptr(), block_table.shape[1],
            seq_lens.data_ptr(), *queries, batch, Hkv, D, int(kv_tokens), k_out.data_ptr(), v_out.data_ptr(),
            cu_seqlens.data_ptr(), status.data_ptr())
    return k_out, v_out, cu_seqlens, status


def prompt_attention_paged(q, k_pages, v_pages, block_table, seq_lens, cu_seqlens, *, kv_layout="HND", sm_scale=None,
                           out=None, lse=None, return_lse=False, status=None, kv_dtype="bf16", k_scale=None, v_scale=None,
                           kv_tokens=None):
    """Causal attention of packed prompts, or chunks of them, over the pages of the cache
    (``hpc_prompt_attention_paged``): the queries of request r are the last of its seq_lens[r] cached tokens.
    Returns (out bf16 [tokens, Hq, D], lse fp32 [tokens, Hq] or None, status).

    The kernel reads bf16 pages of 16, 32, 64 or 128 tokens. With kv_tokens, an upper bound of the sum of seq_lens
    (which is on the device), the cached tokens are read into packed rows first (``gather_tokens``): for E4M3 caches,
    which need it, and pages of any size. The rows are bf16: an E4M3 code times its scale is rounded (by 2^-8 of the value at
    most), where the decode steps use the codes as they are. A request that is flagged for its length, which the kernel leaves alone, gets
    zeros and -inf this way, and so does one that kv_tokens leaves out."""
    if kv_tokens is None and kv_dtype != "bf16":
        raise HpcError(f"prompt_attention_paged of a {kv_dtype} cache needs kv_tokens, a bound of the sum of seq_lens")
    if kv_tokens is not None:
        k, v, cu_k, status = gather_tokens(k_pages, v_pages, block_table, seq_lens, kv_tokens, kv_dtype=kv_dtype,
                                           kv_layout=kv_layout, k_scale=k_scale, v_scale=v_scale, status=status,
                                           cu_queries=cu_seqlens)
        return prompt_attention(q, k, v, cu_seqlens, cu_seqlens_k=cu_k, sm_scale=sm_scale, out=out, lse=lse,
                                return_lse=return_lse, status=status)
    if _fast is not None:
        r = _fast.prompt_attention_paged(q, k_pages, v_pages, block_table, seq_lens, cu_seqlens, _LAYOUTS.get(kv_layout),
                                         sm_scale, out, lse, return_lse, status)
        if r is not None:
            return r
    qs = _strided(q, "q", None)
    dev = q.device
    n, Hq, D = q.shape
    code, num_pages, Hkv, P, lay = _cache(k_pages, v_pages, "bf16", kv_layout, None, None, D, dev)
    batch = _packed(cu_seqlens, dev)
    _tables(block_table, seq_lens, batch, dev)
    out = _buffer(out, "out", (n, Hq, D), torch.bfloat16, dev)
    lse = _lse(lse, return_lse, n, Hq, dev)
    status = _status(status, dev)
    scale = 1.0 / math.sqrt(D) if sm_scale is None else float(sm_scale)
    work, partial, nbytes = _prompt_scratch(block_table.shape[1] * P, D, dev)
    _launch("hpc_prompt_attention_paged", dev, q.data_ptr(), *qs, k_pages.data_ptr(), v_pages.data_ptr(), code, lay,
            num_pages, P, block_table.data_ptr(), block_table.shape[1], _addr(seq_lens), n, cu_seqlens.data_ptr(),
            batch, Hq, Hkv, D, scale, out.data_ptr(), _addr(lse), work.data_ptr(), _addr(partial), nbytes, status.data_ptr())
    return out, lse, status


def _rows(t, name, shape, dtype, dev):
    """A [batch, steps, vocab] tensor whose rows are equally far apart; returns that distance."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != dev:
        raise HpcError(f"{name} must be a CUDA tensor on {dev}")
    if t.dtype != dtype:
        raise HpcError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise HpcError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    Bn, T, V = shape
    if V > 1 and t.stride(2) != 1:
        raise HpcError(f"{name} must be contiguous along the vocabulary")
    row = t.stride(1) if T > 1 else (t.stride(0) if Bn > 1 and T == 1 else V)
    if (Bn > 1 and T > 0 and t.stride(0) != T * row) or row < V:
        raise HpcError(f"{name} must have equally spaced rows")
    return row


def verify_drafts(draft_tokens, target_probs, draft_probs, uniforms, *, draft_lens=None, seq_lens=None,
                  out_tokens=None, accepted=None, new_lens=None, status=None):
    """Which drafted tokens stand, and the token after them (``hpc_verify_drafts``): draft_tokens int32
    [B, T], target_probs [B, T + 1, V] and draft_probs [B, T, V] (or None: one-hot drafts) in fp32 or bf16,
    uniforms fp32 [B, T + 1]. Rows may be padded (a view of a wider tensor). Returns (out_tokens [B, T + 1],
    accepted [B], new_lens [B] or None, status); new_lens needs seq_lens."""
    if _fast is not None:
        r = _fast.verify_drafts(draft_tokens, target_probs, draft_probs, uniforms, draft_lens, seq_lens, out_tokens,
                                accepted, new_lens, status)
        if r is not None:
            return r
    _need(draft_tokens, "draft_tokens", torch.int32)
    dev = draft_tokens.device
    if draft_tokens.dim() != 2 or not isinstance(target_probs, torch.Tensor) or target_probs.dim() != 3:
        raise HpcError("draft_tokens must be [batch, drafts] and target_probs [batch, drafts + 1, vocab]")
    Bn, T = draft_tokens.shape
    V = target_probs.shape[2]
    if target_probs.dtype not in (torch.float32, torch.bfloat16):
        raise HpcError(f"target_probs has dtype {target_probs.dtype}, expected float32 or bfloat16")
    p_row = _rows(target_probs, "target_probs", (Bn, T + 1, V), target_probs.dtype, dev)
    q_row = V
    if draft_probs is not None:
        q_row = _rows(draft_probs, "draft_probs", (Bn, T, V), target_probs.dtype, dev)
    _want(uniforms, "uniforms", torch.float32, dev)
    if tuple(uniforms.shape) != (Bn, T + 1):
        raise HpcError(f"uniforms must be [{Bn}, {T + 1}]")
    for name, t in (("draft_lens", draft_lens), ("seq_lens", seq_lens)):
        if t is not None:
            _want(t, name, torch.int32, dev)
            if t.numel() != Bn:
                raise HpcError(f"{name} must be [batch]")
    out_tokens = _buffer(out_tokens, "out_tokens", (Bn, T + 1), torch.int32, dev)
    accepted = _buffer(accepted, "accepted", (Bn,), torch.int32, dev)
    if seq_lens is not None:
        new_lens = _buffer(new_lens, "new_lens", (Bn,), torch.int32, dev)
    elif new_lens is not None:
        raise HpcError("new_lens needs seq_lens")
    status = _status(status, dev)
    _launch("hpc_verify_drafts", dev, draft_tokens.data_ptr(), target_probs.data_ptr(), p_row, _addr(draft_probs),
            q_row, HPC_FP32 if target_probs.dtype == torch.float32 else HPC_BF16, uniforms.data_ptr(),
            _addr(draft_lens), _addr(seq_lens), Bn, T, V, out_tokens.data_ptr(), accepted.data_ptr(), _addr(new_lens),
            status.data_ptr())
    return out_tokens, accepted, new_lens, status


@dataclass
class PageUpdate:
    """What ``resize_pages``, ``fork_pages`` or ``compact_pages`` leaves on the device. ``moves`` and
    ``n_moves`` go to ``copy_pages``, before the destination pages are read or written."""

    block_table: torch.Tensor
    ref_count: torch.Tensor
    moves: torch.Tensor  # int32 [capacity, 2], the first n_moves pairs (source, destination) valid
    n_moves: torch.Tensor  # int32 [1]
    status: torch.Tensor
    seq_lens: torch.Tensor | None = None  # fork_pages
    page_map: torch.Tensor | None = None  # compact_pages


def _pool(block_table, ref_count):
    """(device, rows, max_pages, num_pages) of a cache's table and reference counts."""
    _need(block_table, "block_table", torch.int32)
    dev = block_table.device
    _want(ref_count, "ref_count", torch.int32, dev)
    if block_table.dim() != 2 or ref_count.dim() != 1:
        raise HpcError("block_table must be [rows, max_pages] and ref_count [num_pages]")
    return dev, block_table.shape[0], block_table.shape[1], ref_count.numel()


def _moves(moves, n_moves, capacity, dev):
    if moves is None:
        moves = _empty((max(capacity, 1), 2), torch.int32, dev)
    _want(moves, "moves", torch.int32, dev)
    if moves.dim() != 2 or moves.shape[1] != 2:
        raise HpcError("moves must be [capacity, 2]")
    return moves, _buffer(n_moves, "n_moves", (1,), torch.int32, dev)


def resize_pages(block_table, old_lens, new_lens, ref_count, page_size, *, block_table_out=None, ref_count_out=None,
                 moves=None, n_moves=None, status=None) -> PageUpdate:
    """Requests change from old_lens to new_lens tokens (``hpc_pages_resize``): pages are released, taken,
    and copied on write where a part-filled page is shared. Without output buffers the update is a new
    table and new counts; handing the inputs in as outputs updates them in place."""
    if _fast is not None:
        r = _fast.resize_pages(block_table, old_lens, new_lens, ref_count, page_size, block_table_out, ref_count_out,
                               moves, n_moves, status)
        if r is not None:
            return PageUpdate(*r)
    dev, Bn, M, N = _pool(block_table, ref_count)
    for name, t in (("old_lens", old_lens), ("new_lens", new_lens)):
        _want(t, name, torch.int32, dev)
        if t.numel() != Bn:
            raise HpcError(f"{name} must be [batch]")
    table_out = _buffer(block_table_out, "block_table_out", (Bn, M), torch.int32, dev)
    ref_out = _buffer(ref_count_out, "ref_count_out", (N,), torch.int32, dev)
    moves, n_moves = _moves(moves, n_moves, Bn, dev)
    status = _status(status, dev)
    _launch("hpc_pages_resize", dev, block_table.data_ptr(), table_out.data_ptr(), Bn, M, int(page_size),
            old_lens.data_ptr(), _addr(new_lens), ref_count.data_ptr(), ref_out.data_ptr(), N, moves.data_ptr(),
            moves.shape[0], n_moves.data_ptr(), status.data_ptr())
    return PageUpdate(table_out, ref_out, moves, n_moves, status)


def fork_pages(block_table, seq_lens, ref_count, parents, page_size, *, block_table_out=None, seq_lens_out=None,
               ref_count_out=None, moves=None, n_moves=None, status=None) -> PageUpdate:
    """New row r is old row parents[r], -1 for none (``hpc_pages_fork``): full pages are shared, a
    part-filled last page is copied for every child but the first, rows without children are released."""
    if _fast is not None:
        r = _fast.fork_pages(block_table, seq_lens, ref_count, parents, page_size, block_table_out, seq_lens_out,
                             ref_count_out, moves, n_moves, status)
        if r is not None:
            return PageUpdate(*r)
    dev, rows_in, M, N = _pool(block_table, ref_count)
    _want(seq_lens, "seq_lens", torch.int32, dev)
    if seq_lens.numel() != rows_in:
        raise HpcError("seq_lens must be [rows]")
    _want(parents, "parents", torch.int32, dev)
    rows_out = parents.numel()
    table_out = _buffer(block_table_out, "block_table_out", (rows_out, M), torch.int32, dev)
    lens_out = _buffer(seq_lens_out, "seq_lens_out", (rows_out,), torch.int32, dev)
    ref_out = _buffer(ref_count_out, "ref_count_out", (N,), torch.int32, dev)
    moves, n_moves = _moves(moves, n_moves, rows_out, dev)
    status = _status(status, dev)
    _launch("hpc_pages_fork", dev, block_table.data_ptr(), _addr(seq_lens), rows_in, parents.data_ptr(),
            table_out.data_ptr(), lens_out.data_ptr(), rows_out, M, int(page_size), ref_count.data_ptr(),
            ref_out.data_ptr(), N, moves.data_ptr(), moves.shape[0], n_moves.data_ptr(), status.data_ptr())
    return PageUpdate(table_out, ref_out, moves, n_moves, status, seq_lens=lens_out)


def compact_pages(block_table, ref_count, *, block_table_out=None, ref_count_out=None, page_map=None, moves=None,
                  n_moves=None, status=None) -> PageUpdate:
    """The pages in use move to the lowest ids (``hpc_pages_compact``); page_map names every page's new id."""
    if _fast is not None:
        r = _fast.compact_pages(block_table, ref_count, block_table_out, ref_count_out, page_map, moves, n_moves, status)
        if r is not None:
            return PageUpdate(*r)
    dev, Bn, M, N = _pool(block_table, ref_count)
    table_out = _buffer(block_table_out, "block_table_out", (Bn, M), torch.int32, dev)
    ref_out = _buffer(ref_count_out, "ref_count_out", (N,), torch.int32, dev)
    page_map = _buffer(page_map, "page_map", (N,), torch.int32, dev)
    moves, n_moves = _moves(moves, n_moves, N // 2, dev)
    status = _status(status, dev)
    _launch("hpc_pages_compact", dev, block_table.data_ptr(), table_out.data_ptr(), Bn, M, ref_count.data_ptr(),
            ref_out.data_ptr(), N, page_map.data_ptr(), moves.data_ptr(), moves.shape[0], n_moves.data_ptr(),
            status.data_ptr())
    return PageUpdate(table_out, ref_out, moves, n_moves, status, page_map=page_map)


def copy_pages(caches, moves, n_moves, *, status=None):
    """Copies the listed pages in every cache (``hpc_pages_copy``): caches is a list of tensors
    [num_pages, ...] of one shape and element size, the K and V of every layer that shares the table.
    Returns status."""
    caches = list(caches)
    if _fast is not None:
        r = _fast.copy_pages(caches, moves, n_moves, status)
        if r is not None:
            return r
    _need(moves, "moves", torch.int32)
    dev = moves.device
    if moves.dim() != 2 or moves.shape[1] != 2:
        raise HpcError("moves must be [capacity, 2]")
    _want(n_moves, "n_moves", torch.int32, dev)
    if n_moves.numel() != 1:
        raise HpcError("n_moves must hold one count")
    status = _status(status, dev)
    if not caches:
        return status
    if not all(isinstance(t, torch.Tensor) for t in caches):
        raise HpcError("the caches must be tensors")
    shape, size = caches[0].shape, caches[0].element_size()
    for t in caches:
        _want(t, "cache", t.dtype, dev)
        if t.shape != shape or t.element_size() != size or len(shape) < 2:
            raise HpcError("the caches must be [num_pages, ...] tensors of one shape and element size")
    num_pages = shape[0]
    if num_pages == 0:
        raise HpcError("the caches hold no pages")
    page_bytes = caches[0].numel() // num_pages * size
    ptrs = (ctypes.c_void_p * len(caches))(*[t.data_ptr() for t in caches])
    _launch("hpc_pages_copy", dev, ptrs, len(caches), page_bytes, num_pages, moves.data_ptr(), moves.shape[0],
            n_moves.data_ptr(), status.data_ptr())
    return status


def wait_selftest(limit_ns: int, arrive: bool, device, status=None):
    """``hpc_wait_selftest``: the library's bounded wait on a barrier phase that completes at once
    (arrive) or never (not arrive). Returns (status word, waited ns), both device tensors."""
    dev = torch.device(device)
    status = new_status(dev) if status is None else status
    waited = torch.zeros(1, dtype=torch.int64, device=dev)
    with torch.cuda.device(dev):
        _check(_lib.hpc_wait_selftest(int(limit_ns), 1 if arrive else 0, _ptr(status), _ptr(waited), _stream(dev)),
               "hpc_wait_selftest")
    return status, waited


def decode_step(q, k_pages, v_pages, block_table, seq_lens, num_heads, kv_heads, tile_len, *, kv_dtype="bf16",
                kv_layout="HND", k_scale=None, v_scale=None, num_ctas=None, out=None, out_dtype=torch.float32,
                status=None, static_splits=None, e4m3_kernel="mma"):
    """plan -> attention -> merge (three launches) for one decode step; returns (out, plan, status)."""
    dev = q.device
    status = new_status(dev) if status is None else status
    max_seq = block_table.shape[1] * _geometry(k_pages, kv_layout)[2]
    if static_splits:
        p = plan_static(seq_lens, num_heads, kv_heads, tile_len, static_splits, max_seq, status)
    else:
        p = plan(seq_lens, num_heads, kv_heads, tile_len, num_ctas, max_seq, status)
    out, po, pml = attention(q, k_pages, v_pages, block_table, seq_lens, p, kv_dtype=kv_dtype, kv_layout=kv_layout,
                             k_scale=k_scale, v_scale=v_scale, out=out, out_dtype=out_dtype, status=status,
                             e4m3_kernel=e4m3_kernel)
    merge(p, po, pml, out, num_heads, status)
    return out, p, status


NOALLOC_SCRATCH_BYTES = 16 << 20


def decode_step_noalloc(q, k_pages, v_pages, block_table, seq_lens, num_heads, kv_heads, tile_len, *,
                        kv_dtype="bf16", k_scale=None, v_scale=None, num_ctas=None, sm_scale=None, out=None,
                        out_dtype=torch.float32, status=None):
    """One decode step through ``hpc_decode_step_noalloc``: the library keeps the plan and
    partial states in its own static device array, for callers that cannot allocate device
    memory. Returns (out, status). Calls that overlap on the GPU share that array; keep
    them on one stream. The cache is HND."""
    _need(q, "q", torch.bfloat16)
    dev = q.device
    B, Hq, D = q.shape
    if Hq != num_heads:
        raise HpcError(f"q has {Hq} heads, expected {num_heads}")
    code, num_pages, Hkv, P, _ = _cache(k_pages, v_pages, kv_dtype, "HND", k_scale, v_scale, D, dev)
    if Hkv != kv_heads:
        raise HpcError(f"cache has {Hkv} kv heads, expected {kv_heads}")
    _tables(block_table, seq_lens, B, dev)
    G = _grid(num_ctas, dev)
    out = _output(out, (B, Hq, D), out_dtype, dev)
    status = new_status(dev) if status is None else status
    _need(status, "status", torch.int32, dev)
    scale = 1.0 / math.sqrt(D) if sm_scale is None else float(sm_scale)
    with torch.cuda.device(dev):
        _check(_lib.hpc_decode_step_noalloc(
            _ptr(q), _ptr(k_pages), _ptr(v_pages), code, _ptr(k_scale), _ptr(v_scale), num_pages, P, Hq, Hkv, D,
            _ptr(block_table), block_table.shape[1], _ptr(seq_lens), B, tile_len, G, scale, _ptr(out),
            _out_code(out), _ptr(status), _stream(dev)), "hpc_decode_step_noalloc")
    return out, status


def launch_info(head_dim, kv_dtype, page_size, tile_len, ctas_per_sm=1, e4m3_kernel="mma"):
    st, sm, th = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _check(_lib.hpc_attention_launch_info(head_dim, _KV_DTYPES[kv_dtype], page_size, tile_len, ctas_per_sm,
                                          E4M3_KERNELS[e4m3_kernel], ctypes.byref(st), ctypes.byref(sm),
                                          ctypes.byref(th)), "hpc_attention_launch_info")
    return {"stages": st.value, "smem_bytes": sm.value, "threads": th.value}
