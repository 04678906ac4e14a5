"""ctypes binding of the C ABI in include/mla_verify.h, include/mla_ddtree.h,
include/mla_kvq.h, include/mla_kv8.h and include/mla_kv_tables.h.

Argument marshalling only: torch tensors give device pointers, sizes and
strides; every step of the computation runs in the CUDA library.  The library
is loaded on first use and a missing build raises -- there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct
from dataclasses import dataclass
from typing import Optional

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libmla_verify.so")

MLA_OK, MLA_ERR_INVALID_ARG, MLA_ERR_UNSUPPORTED, MLA_ERR_CUDA, MLA_ERR_WORKSPACE, \
    MLA_ERR_DEVICE_CHECK = range(6)
MLA_BF16, MLA_FP32 = 0, 1
ALGO = {"auto": 0, "simt": 1, "tc": 2}

DEVERR = {
    0x1: "PREFIX", 0x2: "INDPTR", 0x4: "SLOT", 0x8: "PARENT", 0x10: "PAGES",
    0x20: "CAPACITY", 0x40: "TIMEOUT", 0x80: "LAYOUT", 0x100: "DRAFT", 0x200: "NONFINITE",
}

# every symbol include/*.h declares
EXPORTS = ("mla_verify_workspace_size", "mla_verify_attn", "mla_verify_attn_noalloc", "mla_verify_noalloc_check",
           "mla_verify_build_meta", "mla_verify_check", "mla_verify_splits_used", "mla_status_str",
           "mla_verify_abi_version",
           "mla_verify_selftest_timeout", "mla_kv_compact", "mla_ddtree_build", "mla_ddtree_accept",
           "mla_kvq_write", "mla_kvq_read", "mla_kvq_attn", "mla_kvq_attn_workspace_size", "mla_kvq_check",
           "mla_kvq_selftest_timeout",
           "mla_kv8_write", "mla_kv8_read", "mla_kv8_attn", "mla_kv8_attn_workspace_size", "mla_kv8_check",
           "mla_kv8_selftest_timeout", "mla_kv_tables")
NOALLOC_SCRATCH_BYTES = 32 << 20
DDTREE_WORKSPACE_BYTES = 256
KVQ_ROW_BYTES = 416
KVQ_MAX_EXPONENT = 32
KVQ_WORKSPACE_BYTES = 16384
KV8_ROW_BYTES = 640
KV8_MAX_SCALE = 15
KV8_MAX_EXPONENT = 32
KV8_WORKSPACE_BYTES = 16384
KV_TABLES_WORKSPACE_BYTES = 16384


class MlaVerifyArgs(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int), ("Q", ctypes.c_int), ("H", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("q_lat", ctypes.c_void_p), ("q_pe", ctypes.c_void_p),
        ("kv_c", ctypes.c_void_p), ("k_pe", ctypes.c_void_p),
        ("kv_c_stride", ctypes.c_int64), ("k_pe_stride", ctypes.c_int64),
        ("pool_slots", ctypes.c_int64),
        ("page_size", ctypes.c_int),
        ("kv_indptr", ctypes.c_void_p), ("kv_indices", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p), ("max_pages", ctypes.c_int),
        ("prefix_lens", ctypes.c_void_p), ("tree_parent", ctypes.c_void_p),
        ("scale", ctypes.c_float),
        ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("algo", ctypes.c_int),
        ("profile_events", ctypes.c_void_p),
    ]


class MlaDdtreeBuildArgs(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int), ("L", ctypes.c_int), ("K", ctypes.c_int), ("budget", ctypes.c_int),
        ("root_token", ctypes.c_void_p), ("cand_token", ctypes.c_void_p), ("cand_logp", ctypes.c_void_p),
        ("tree_parent", ctypes.c_void_p), ("tree_token", ctypes.c_void_p),
        ("tree_depth", ctypes.c_void_p), ("tree_score", ctypes.c_void_p),
    ]


class MlaDdtreeAcceptArgs(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int), ("Q", ctypes.c_int),
        ("tree_parent", ctypes.c_void_p), ("tree_token", ctypes.c_void_p), ("target_token", ctypes.c_void_p),
        ("node_slot", ctypes.c_void_p),
        ("accept_len", ctypes.c_void_p), ("accept_nodes", ctypes.c_void_p), ("accept_slots", ctypes.c_void_p),
        ("next_token", ctypes.c_void_p),
    ]


class MlaKvqCache(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("slots", ctypes.c_int64),
                ("exponent", ctypes.c_int)]


class MlaKvqRows(ctypes.Structure):
    _fields_ = [
        ("n", ctypes.c_int64), ("dtype", ctypes.c_int),
        ("kv_c", ctypes.c_void_p), ("k_pe", ctypes.c_void_p),
        ("kv_c_stride", ctypes.c_int64), ("k_pe_stride", ctypes.c_int64),
        ("slots", ctypes.c_void_p),
    ]


class MlaKvqAttnArgs(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int), ("Q", ctypes.c_int), ("H", ctypes.c_int),
        ("cache", MlaKvqCache),
        ("q_lat", ctypes.c_void_p), ("q_pe", ctypes.c_void_p),
        ("page_size", ctypes.c_int),
        ("kv_indptr", ctypes.c_void_p), ("kv_indices", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p), ("max_pages", ctypes.c_int),
        ("prefix_lens", ctypes.c_void_p), ("tree_parent", ctypes.c_void_p),
        ("window", ctypes.c_int), ("sinks", ctypes.c_int),
        ("scale", ctypes.c_float),
        ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
    ]


class MlaKv8Cache(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("slots", ctypes.c_int64),
                ("scales", ctypes.c_void_p), ("block", ctypes.c_int), ("exponent", ctypes.c_int)]


class MlaKv8AttnArgs(ctypes.Structure):
    _fields_ = [(n, MlaKv8Cache if n == "cache" else t) for n, t in MlaKvqAttnArgs._fields_]


class MlaKvTablesArgs(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int), ("Q", ctypes.c_int),
        ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int), ("num_pages", ctypes.c_int),
        ("prefix_lens", ctypes.c_void_p), ("new_lens", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p), ("pages_held", ctypes.c_void_p),
        ("free_ring", ctypes.c_void_p), ("free_state", ctypes.c_void_p), ("ring", ctypes.c_int),
        ("slots", ctypes.c_void_p), ("slots_len", ctypes.c_int64),
        ("kv_indptr", ctypes.c_void_p),
        ("kv_indices", ctypes.c_void_p), ("indices_len", ctypes.c_int64),
        ("scales", ctypes.c_void_p), ("block", ctypes.c_int),
    ]


def _packer(cls):
    """The bytes of a struct from its fields' values (a nested struct's in their
    place): a third of the time that making a ctypes.Structure takes, which
    counts in a call of a few us."""
    code = {ctypes.c_void_p: "P", ctypes.c_int64: "q", ctypes.c_int: "i", ctypes.c_float: "f"}

    def flat(c):
        return "".join(code.get(t) or flat(t) for _, t in c._fields_)
    p = struct.Struct("@" + flat(cls) + "0q")
    assert p.size == ctypes.sizeof(cls)
    return p.pack


_pack_cache, _pack_rows, _pack_attn = _packer(MlaKvqCache), _packer(MlaKvqRows), _packer(MlaKvqAttnArgs)
_pack_cache8, _pack_attn8, _pack_tables = _packer(MlaKv8Cache), _packer(MlaKv8AttnArgs), _packer(MlaKvTablesArgs)


class MlaError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {status_str(status)}")


_lib = None


def load(path: Optional[str] = None):
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"CUDA library not built: {p} (run __graft_entry__.build())")
    lib = ctypes.CDLL(p)
    lib.mla_verify_workspace_size.restype = ctypes.c_size_t
    lib.mla_verify_workspace_size.argtypes = [ctypes.POINTER(MlaVerifyArgs), ctypes.c_int]
    lib.mla_verify_attn.restype = ctypes.c_int
    lib.mla_verify_attn.argtypes = [ctypes.POINTER(MlaVerifyArgs), ctypes.c_void_p, ctypes.c_size_t,
                                    ctypes.c_int, ctypes.c_void_p]
    lib.mla_verify_attn_noalloc.restype = ctypes.c_int
    lib.mla_verify_attn_noalloc.argtypes = [ctypes.POINTER(MlaVerifyArgs), ctypes.c_int, ctypes.c_void_p]
    lib.mla_verify_noalloc_check.restype = ctypes.c_int
    lib.mla_verify_noalloc_check.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_uint32)]
    lib.mla_verify_splits_used.restype = ctypes.c_int
    lib.mla_verify_splits_used.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(ctypes.c_int32)]
    lib.mla_verify_build_meta.restype = ctypes.c_int
    lib.mla_verify_build_meta.argtypes = [ctypes.POINTER(MlaVerifyArgs), ctypes.c_void_p, ctypes.c_size_t,
                                          ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                          ctypes.c_void_p]
    lib.mla_verify_selftest_timeout.restype = ctypes.c_int
    lib.mla_verify_selftest_timeout.argtypes = [ctypes.POINTER(MlaVerifyArgs), ctypes.c_void_p, ctypes.c_size_t,
                                                ctypes.c_uint64, ctypes.c_void_p]
    lib.mla_kv_compact.restype = ctypes.c_int
    lib.mla_kv_compact.argtypes = [ctypes.POINTER(MlaVerifyArgs), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                   ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                   ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
    lib.mla_ddtree_build.restype = ctypes.c_int
    lib.mla_ddtree_build.argtypes = [ctypes.POINTER(MlaDdtreeBuildArgs), ctypes.c_void_p, ctypes.c_size_t,
                                     ctypes.c_void_p]
    lib.mla_ddtree_accept.restype = ctypes.c_int
    lib.mla_ddtree_accept.argtypes = [ctypes.POINTER(MlaDdtreeAcceptArgs), ctypes.c_void_p, ctypes.c_size_t,
                                      ctypes.c_void_p]
    for f in (lib.mla_kvq_write, lib.mla_kvq_read):
        f.restype = ctypes.c_int
        f.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.mla_kvq_attn.restype = ctypes.c_int
    lib.mla_kvq_attn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.mla_kvq_selftest_timeout.restype = ctypes.c_int
    lib.mla_kvq_selftest_timeout.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint64,
                                             ctypes.c_void_p]
    lib.mla_kvq_attn_workspace_size.restype = ctypes.c_size_t
    lib.mla_kvq_attn_workspace_size.argtypes = [ctypes.POINTER(MlaKvqAttnArgs)]
    lib.mla_kvq_check.restype = ctypes.c_int
    lib.mla_kvq_check.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(ctypes.c_uint32)]
    for f in (lib.mla_kv8_write, lib.mla_kv8_read):
        f.restype = ctypes.c_int
        f.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    for f in (lib.mla_kv8_attn, lib.mla_kv_tables):
        f.restype = ctypes.c_int
        f.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.mla_kv8_selftest_timeout.restype = ctypes.c_int
    lib.mla_kv8_selftest_timeout.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint64,
                                             ctypes.c_void_p]
    lib.mla_kv8_attn_workspace_size.restype = ctypes.c_size_t
    lib.mla_kv8_attn_workspace_size.argtypes = [ctypes.POINTER(MlaKv8AttnArgs)]
    lib.mla_kv8_check.restype = ctypes.c_int
    lib.mla_kv8_check.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(ctypes.c_uint32)]
    lib.mla_verify_check.restype = ctypes.c_int
    lib.mla_verify_check.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(ctypes.c_uint32)]
    lib.mla_status_str.restype = ctypes.c_char_p
    lib.mla_status_str.argtypes = [ctypes.c_int]
    lib.mla_verify_abi_version.restype = ctypes.c_int
    if path is None:
        _lib = lib
    return lib


def status_str(s: int) -> str:
    return load().mla_status_str(int(s)).decode()


# ----------------------------------------------------------------------------
# torch marshalling
# ----------------------------------------------------------------------------
def _ptr(t) -> Optional[int]:
    return None if t is None else int(t.data_ptr())


@dataclass
class DeviceInputs:
    """Device tensors of one verify problem (see inputs.Problem)."""
    B: int
    Q: int
    H: int
    dtype: str
    scale: float
    q_lat: object
    q_pe: object
    kv_c: object            # [pool_slots, >=512] view (row stride = pool row)
    k_pe: object            # [pool_slots, >=64] view
    prefix_lens: object
    tree_parent: object
    page_size: int
    kv_indptr: object = None
    kv_indices: object = None
    block_table: object = None
    pool: object = None     # owning tensor of kv_c / k_pe

    @property
    def pool_slots(self) -> int:
        return int(self.kv_c.shape[0])

    def check(self):
        """What the C ABI cannot see from pointers: element types, shapes,
        layouts and the device of every tensor.  Raises ValueError."""
        self.check_layout()
        _on_cuda(**self.tensors())

    def tensors(self):
        return dict(q_lat=self.q_lat, q_pe=self.q_pe, kv_c=self.kv_c, k_pe=self.k_pe, prefix_lens=self.prefix_lens,
                    tree_parent=self.tree_parent, kv_indptr=self.kv_indptr, kv_indices=self.kv_indices,
                    block_table=self.block_table)

    def check_layout(self):
        import torch
        el = torch.bfloat16 if self.dtype == "bf16" else torch.float32
        B, Q, H = self.B, self.Q, self.H
        _need(self.q_lat, "q_lat", el, (B, Q, H, 512))
        _need(self.q_pe, "q_pe", el, (B, Q, H, 64))
        for t, name, w in ((self.kv_c, "kv_c", 512), (self.k_pe, "k_pe", 64)):
            if t is None or t.dtype != el or t.dim() != 2 or t.shape[1] != w or t.stride(1) != 1:
                raise ValueError(f"{name} must be a [slots][{w}] {el} view with unit column stride")
        if self.k_pe.shape[0] != self.kv_c.shape[0]:
            raise ValueError("kv_c and k_pe must cover the same pool slots")
        _need(self.prefix_lens, "prefix_lens", torch.int32, (B,))
        _need(self.tree_parent, "tree_parent", torch.int32, (B, Q))
        if self.page_size == 1:
            _need(self.kv_indptr, "kv_indptr", torch.int32, (B + 1,))
            if self.kv_indices is None or self.kv_indices.dtype != torch.int32 or self.kv_indices.dim() != 1 \
                    or not self.kv_indices.is_contiguous():
                raise ValueError("kv_indices must be a contiguous 1-D int32 tensor")
        else:
            if self.block_table is None or self.block_table.dtype != torch.int32 or self.block_table.dim() != 2 \
                    or self.block_table.shape[0] != B or not self.block_table.is_contiguous():
                raise ValueError("block_table must be a contiguous [B][max_pages] int32 tensor")


def device_inputs(problem, device="cuda", separate_pools: bool = False) -> DeviceInputs:
    """Copy a numpy inputs.Problem to the device (packed [slot][576] pool by
    default; separate kv_c / k_pe arrays with ``separate_pools``)."""
    import torch

    def t(x, dt=None):
        if x is None:
            return None
        a = np.ascontiguousarray(x)
        if a.dtype == np.uint16:
            return torch.from_numpy(a.view(np.int16)).to(device).view(torch.bfloat16)
        tt = torch.from_numpy(a).to(device)
        return tt if dt is None else tt.to(dt)

    pool = t(problem.pool)
    if separate_pools:
        kv_c = pool[:, :512].contiguous()
        k_pe = pool[:, 512:].contiguous()
        owner = None
    else:
        kv_c, k_pe, owner = pool[:, :512], pool[:, 512:], pool
    return DeviceInputs(
        B=problem.B, Q=problem.Q, H=problem.H, dtype=problem.dtype, scale=problem.scale,
        q_lat=t(problem.q_lat), q_pe=t(problem.q_pe), kv_c=kv_c, k_pe=k_pe,
        prefix_lens=t(problem.prefix_lens.astype(np.int32)),
        tree_parent=t(problem.tree_parent.astype(np.int32)),
        page_size=problem.page_size,
        kv_indptr=t(problem.kv_indptr), kv_indices=t(problem.kv_indices),
        block_table=t(problem.block_table), pool=owner)


def make_args(di: DeviceInputs, out=None, lse=None, algo: str = "auto",
              profile_events=None, check: bool = True) -> MlaVerifyArgs:
    if check:
        import torch
        di.check_layout()
        odt = torch.bfloat16 if di.dtype == "bf16" else torch.float32
        if out is not None:
            _need(out, "out", odt, (di.B, di.Q, di.H, 512))
        if lse is not None:
            _need(lse, "lse", torch.float32, (di.B, di.Q, di.H))
        _on_cuda(out=out, lse=lse, **di.tensors())
    a = MlaVerifyArgs()
    a.B, a.Q, a.H = di.B, di.Q, di.H
    a.dtype = MLA_BF16 if di.dtype == "bf16" else MLA_FP32
    a.q_lat, a.q_pe = _ptr(di.q_lat), _ptr(di.q_pe)
    a.kv_c, a.k_pe = _ptr(di.kv_c), _ptr(di.k_pe)
    a.kv_c_stride = int(di.kv_c.stride(0))
    a.k_pe_stride = int(di.k_pe.stride(0))
    a.pool_slots = di.pool_slots
    a.page_size = di.page_size
    a.kv_indptr, a.kv_indices = _ptr(di.kv_indptr), _ptr(di.kv_indices)
    a.block_table = _ptr(di.block_table)
    a.max_pages = 0 if di.block_table is None else int(di.block_table.shape[1])
    a.prefix_lens, a.tree_parent = _ptr(di.prefix_lens), _ptr(di.tree_parent)
    a.scale = di.scale
    a.out, a.lse = _ptr(out), _ptr(lse)
    a.algo = ALGO[algo]
    if profile_events is not None:
        # keep the pointer array alive as long as the struct
        a._ev = (ctypes.c_void_p * 2)(int(profile_events[0].cuda_event), int(profile_events[1].cuda_event))
        a.profile_events = ctypes.cast(a._ev, ctypes.c_void_p)
    return a


def workspace_size(di: DeviceInputs, num_splits: int = 0, algo: str = "auto") -> int:
    a = make_args(di, algo=algo, check=False)
    n = load().mla_verify_workspace_size(ctypes.byref(a), int(num_splits))
    if n == 0 and di.B > 0 and di.Q > 0:
        raise MlaError(MLA_ERR_INVALID_ARG, "mla_verify_workspace_size")
    return int(n)


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(int(stream.cuda_stream))


def alloc_workspace(nbytes: int, device="cuda"):
    import torch
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def verify_attn(di: DeviceInputs, out=None, lse=None, num_splits: int = 0, algo: str = "auto",
                workspace=None, stream=None, profile_events=None, check: bool = True):
    """Run mla_verify_attn; returns (out [B,Q,H,512], lse [B,Q,H] fp32).
    check=False skips the tensor checks (a loop that already passed them)."""
    import torch
    dev = di.q_lat.device
    odt = torch.bfloat16 if di.dtype == "bf16" else torch.float32
    if out is None:
        out = torch.empty((di.B, di.Q, di.H, 512), dtype=odt, device=dev)
    if lse is None:
        lse = torch.empty((di.B, di.Q, di.H), dtype=torch.float32, device=dev)
    a = make_args(di, out, lse, algo, profile_events, check)
    lib = load()
    need = lib.mla_verify_workspace_size(ctypes.byref(a), int(num_splits))
    if workspace is None:
        workspace = alloc_workspace(need, dev)
    st = lib.mla_verify_attn(ctypes.byref(a), ctypes.c_void_p(_ptr(workspace)),
                             ctypes.c_size_t(workspace.numel() * workspace.element_size()),
                             int(num_splits), _stream(stream))
    if st != MLA_OK:
        raise MlaError(st, "mla_verify_attn")
    return out, lse


def verify_attn_noalloc(di: DeviceInputs, out=None, lse=None, num_splits: int = 0, algo: str = "auto",
                        stream=None, check_device: bool = False):
    """Run mla_verify_attn_noalloc (library-held scratch, no workspace); returns
    (out, lse).  Output tensors are created here when not given -- the library
    call itself allocates nothing.  check_device=True synchronises the stream
    and raises MlaError(MLA_ERR_DEVICE_CHECK) when the device found bad table
    contents (noalloc_check)."""
    import torch
    dev = di.q_lat.device
    odt = torch.bfloat16 if di.dtype == "bf16" else torch.float32
    if out is None:
        out = torch.empty((di.B, di.Q, di.H, 512), dtype=odt, device=dev)
    if lse is None:
        lse = torch.empty((di.B, di.Q, di.H), dtype=torch.float32, device=dev)
    a = make_args(di, out, lse, algo)
    st = load().mla_verify_attn_noalloc(ctypes.byref(a), int(num_splits), _stream(stream))
    if st != MLA_OK:
        raise MlaError(st, "mla_verify_attn_noalloc")
    if check_device and noalloc_check(stream) != 0:
        raise MlaError(MLA_ERR_DEVICE_CHECK, "mla_verify_attn_noalloc")
    return out, lse


def noalloc_check(stream=None) -> int:
    """Synchronise and return the device error bits the last
    mla_verify_attn_noalloc call on the current device left."""
    bits = ctypes.c_uint32(0)
    st = load().mla_verify_noalloc_check(_stream(stream), ctypes.byref(bits))
    if st not in (MLA_OK, MLA_ERR_DEVICE_CHECK):
        raise MlaError(st, "mla_verify_noalloc_check")
    return int(bits.value)


def selftest_timeout(di: DeviceInputs, out, lse, workspace, hold_ns: int, stream=None):
    """Run mla_verify_selftest_timeout: the tensor-core call with one device
    wait that gives up after hold_ns; read the outcome with check()."""
    a = make_args(di, out, lse, "tc")
    st = load().mla_verify_selftest_timeout(ctypes.byref(a), ctypes.c_void_p(_ptr(workspace)),
                                            ctypes.c_size_t(workspace.numel() * workspace.element_size()),
                                            ctypes.c_uint64(int(hold_ns)), _stream(stream))
    if st != MLA_OK:
        raise MlaError(st, "mla_verify_selftest_timeout")


def kv_compact(di: DeviceInputs, dst_pool, dst_slot0: int = 0, workspace=None, stream=None):
    """Run mla_kv_compact into ``dst_pool`` ([slots][576] of the cache dtype:
    kv_c columns 0-511, k_pe 512-575); returns (new_kv_indices [sum N_b] int32,
    new_kv_indptr [B+1] int32, workspace)."""
    import torch
    dev = di.q_lat.device
    a = make_args(di)
    lib = load()
    need = lib.mla_verify_workspace_size(ctypes.byref(a), 1)
    if workspace is None:
        workspace = alloc_workspace(need, dev)
    total = int((di.prefix_lens.to(torch.int64) + di.Q).sum().item())
    new_idx = torch.full((max(total, 1),), -1, dtype=torch.int32, device=dev)
    new_indptr = torch.zeros((di.B + 1,), dtype=torch.int32, device=dev)
    kv_compact_into(di, dst_pool, new_idx, new_indptr, workspace, dst_slot0, stream)
    return new_idx[:total], new_indptr, workspace


def kv_compact_into(di: DeviceInputs, dst_pool, new_idx, new_indptr, workspace, dst_slot0: int = 0, stream=None):
    """mla_kv_compact with caller-provided output tables (no host synchronisation)."""
    a = make_args(di)
    lib = load()
    st = lib.mla_kv_compact(ctypes.byref(a), ctypes.c_void_p(_ptr(workspace)),
                            ctypes.c_size_t(workspace.numel() * workspace.element_size()),
                            ctypes.c_void_p(_ptr(dst_pool)), ctypes.c_void_p(_ptr(dst_pool[:, 512:])),
                            ctypes.c_int64(dst_pool.stride(0)), ctypes.c_int64(dst_pool.stride(0)),
                            ctypes.c_int64(dst_slot0), ctypes.c_int64(dst_pool.shape[0]),
                            ctypes.c_void_p(_ptr(new_idx)), ctypes.c_void_p(_ptr(new_indptr)), _stream(stream))
    if st != MLA_OK:
        raise MlaError(st, "mla_kv_compact")


def build_meta(di: DeviceInputs, workspace=None, stream=None):
    """Run mla_verify_build_meta; returns (anc [B,Q] uint64 as int64, slots [sum N_b] int32)."""
    import torch
    dev = di.q_lat.device
    a = make_args(di)
    lib = load()
    need = lib.mla_verify_workspace_size(ctypes.byref(a), 1)
    if workspace is None:
        workspace = alloc_workspace(need, dev)
    total = int((di.prefix_lens.to(torch.int64) + di.Q).sum().item())
    anc = torch.zeros((di.B, di.Q), dtype=torch.int64, device=dev)
    slots = torch.full((max(total, 1),), -7, dtype=torch.int32, device=dev)
    st = lib.mla_verify_build_meta(ctypes.byref(a), ctypes.c_void_p(_ptr(workspace)),
                                   ctypes.c_size_t(workspace.numel()), ctypes.c_void_p(_ptr(anc)),
                                   ctypes.c_void_p(_ptr(slots)), ctypes.c_int64(total), _stream(stream))
    if st != MLA_OK:
        raise MlaError(st, "mla_verify_build_meta")
    return anc, slots[:total], workspace


def check(workspace, stream=None) -> int:
    """Synchronise and return the device error bits of the last call on this workspace."""
    bits = ctypes.c_uint32(0)
    st = load().mla_verify_check(ctypes.c_void_p(_ptr(workspace)), _stream(stream), ctypes.byref(bits))
    if st not in (MLA_OK, MLA_ERR_DEVICE_CHECK):
        raise MlaError(st, "mla_verify_check")
    return int(bits.value)


def splits_used(workspace, stream=None) -> int:
    """Synchronise and return the split count the last verify_attn call on
    this workspace used (the library's choice when num_splits was 0)."""
    v = ctypes.c_int32(0)
    st = load().mla_verify_splits_used(ctypes.c_void_p(_ptr(workspace)), _stream(stream), ctypes.byref(v))
    if st != MLA_OK:
        raise MlaError(st, "mla_verify_splits_used")
    return int(v.value)



# ----------------------------------------------------------------------------
# DDTree construction and acceptance (include/mla_ddtree.h)
# ----------------------------------------------------------------------------
def _ws_bytes(workspace) -> int:
    return workspace.numel() * workspace.element_size()


def _need(t, name: str, dtype, shape):
    """The C ABI sees only a pointer: check what it cannot (dtype, shape,
    contiguity, device) before handing it over."""
    import torch
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _on_cuda(**tensors):
    for name, t in tensors.items():
        if t is not None and t.device.type != "cuda":
            raise ValueError(f"{name} must be a CUDA tensor")


def _check_build(root_token, cand_token, cand_logp, B, L, K, Q, tree_parent, tree_token, tree_depth, tree_score,
                 workspace):
    import torch
    _need(cand_logp, "cand_logp", torch.float32, (B, L, K))
    _need(cand_token, "cand_token", torch.int32, (B, L, K))
    _need(root_token, "root_token", torch.int32, (B,))
    for t, name in ((tree_parent, "tree_parent"), (tree_token, "tree_token")):
        _need(t, name, torch.int32, (B, Q))
    if tree_depth is not None:
        _need(tree_depth, "tree_depth", torch.int32, (B, Q))
    if tree_score is not None:
        _need(tree_score, "tree_score", torch.float32, (B, Q))
    _on_cuda(cand_logp=cand_logp, cand_token=cand_token, root_token=root_token, tree_parent=tree_parent,
             tree_token=tree_token, tree_depth=tree_depth, tree_score=tree_score, workspace=workspace)


def _check_accept(tree_parent, tree_token, target_token, accept_len, accept_nodes, next_token, node_slot,
                  accept_slots, workspace, B, Q):
    import torch
    for t, name in ((tree_parent, "tree_parent"), (tree_token, "tree_token"), (target_token, "target_token"),
                    (accept_nodes, "accept_nodes")):
        _need(t, name, torch.int32, (B, Q))
    for t, name in ((accept_len, "accept_len"), (next_token, "next_token")):
        _need(t, name, torch.int32, (B,))
    if node_slot is not None:
        _need(node_slot, "node_slot", torch.int32, (B, Q))
    if accept_slots is not None:
        _need(accept_slots, "accept_slots", torch.int32, (B, Q))
    _on_cuda(tree_parent=tree_parent, tree_token=tree_token, target_token=target_token, accept_nodes=accept_nodes,
             accept_len=accept_len, next_token=next_token, node_slot=node_slot, accept_slots=accept_slots,
             workspace=workspace)


def ddtree_build_into(root_token, cand_token, cand_logp, budget: int, tree_parent, tree_token, workspace,
                      tree_depth=None, tree_score=None, stream=None, check: bool = True):
    """mla_ddtree_build into caller-provided [B][budget+1] outputs (no host
    synchronisation).  check=False skips the tensor checks, for a loop that
    passes tensors it has already passed once with checking on."""
    if cand_logp.dim() != 3:
        raise ValueError("cand_logp must be [B][L][K]")
    B, L, K = cand_logp.shape
    Q = int(budget) + 1
    if check:
        _check_build(root_token, cand_token, cand_logp, B, L, K, Q, tree_parent, tree_token, tree_depth, tree_score,
                     workspace)
    a = MlaDdtreeBuildArgs()
    a.B, a.L, a.K, a.budget = B, L, K, int(budget)
    a.root_token, a.cand_token, a.cand_logp = _ptr(root_token), _ptr(cand_token), _ptr(cand_logp)
    a.tree_parent, a.tree_token = _ptr(tree_parent), _ptr(tree_token)
    a.tree_depth, a.tree_score = _ptr(tree_depth), _ptr(tree_score)
    st = load().mla_ddtree_build(ctypes.byref(a), ctypes.c_void_p(_ptr(workspace)),
                                 ctypes.c_size_t(_ws_bytes(workspace)), _stream(stream))
    if st != MLA_OK:
        raise MlaError(st, "mla_ddtree_build")


def ddtree_build(root_token, cand_token, cand_logp, budget: int, workspace=None, stream=None):
    """Build the draft trees; inputs are device tensors [B] int32, [B][L][K] int32,
    [B][L][K] float32.  Returns (parent, token, depth, score) [B][budget+1] and the workspace."""
    import torch
    dev = cand_logp.device
    B = cand_logp.shape[0]
    Q = int(budget) + 1
    if workspace is None:
        workspace = alloc_workspace(DDTREE_WORKSPACE_BYTES, dev)
    parent = torch.full((B, Q), -7, dtype=torch.int32, device=dev)
    token = torch.full((B, Q), -7, dtype=torch.int32, device=dev)
    depth = torch.full((B, Q), -7, dtype=torch.int32, device=dev)
    score = torch.full((B, Q), float("nan"), dtype=torch.float32, device=dev)
    ddtree_build_into(root_token, cand_token, cand_logp, budget, parent, token, workspace, depth, score, stream)
    return parent, token, depth, score, workspace


def ddtree_accept_into(tree_parent, tree_token, target_token, accept_len, accept_nodes, next_token, workspace,
                       node_slot=None, accept_slots=None, stream=None, check: bool = True):
    """mla_ddtree_accept into caller-provided outputs (no host synchronisation);
    check as for ddtree_build_into."""
    if tree_parent.dim() != 2:
        raise ValueError("tree_parent must be [B][Q]")
    B, Q = tree_parent.shape
    if check:
        _check_accept(tree_parent, tree_token, target_token, accept_len, accept_nodes, next_token, node_slot,
                      accept_slots, workspace, B, Q)
    a = MlaDdtreeAcceptArgs()
    a.B, a.Q = B, Q
    a.tree_parent, a.tree_token, a.target_token = _ptr(tree_parent), _ptr(tree_token), _ptr(target_token)
    a.node_slot = _ptr(node_slot)
    a.accept_len, a.accept_nodes, a.accept_slots = _ptr(accept_len), _ptr(accept_nodes), _ptr(accept_slots)
    a.next_token = _ptr(next_token)
    st = load().mla_ddtree_accept(ctypes.byref(a), ctypes.c_void_p(_ptr(workspace)),
                                  ctypes.c_size_t(_ws_bytes(workspace)), _stream(stream))
    if st != MLA_OK:
        raise MlaError(st, "mla_ddtree_accept")


def ddtree_accept(tree_parent, tree_token, target_token, node_slot=None, workspace=None, stream=None):
    """Greedy acceptance; inputs are device int32 tensors [B][Q].  Returns
    (accept_len [B], accept_nodes [B][Q], next_token [B], accept_slots [B][Q] or None, workspace)."""
    import torch
    dev = tree_parent.device
    B, Q = tree_parent.shape
    if workspace is None:
        workspace = alloc_workspace(DDTREE_WORKSPACE_BYTES, dev)
    n_len = torch.full((B,), -7, dtype=torch.int32, device=dev)
    nodes = torch.full((B, Q), -7, dtype=torch.int32, device=dev)
    nxt = torch.full((B,), -7, dtype=torch.int32, device=dev)
    slots = None if node_slot is None else torch.full((B, Q), -7, dtype=torch.int32, device=dev)
    ddtree_accept_into(tree_parent, tree_token, target_token, n_len, nodes, nxt, workspace, node_slot, slots, stream)
    return n_len, nodes, nxt, slots, workspace


# ----------------------------------------------------------------------------
# 4-bit latent cache (include/mla_kvq.h)
# ----------------------------------------------------------------------------
@dataclass
class QuantCache:
    """A pool of packed cache rows: ``rows`` is a uint8 [slots][416] tensor or
    view (row stride a multiple of 32 bytes), ``exponent`` the power of two its
    latents are scaled by."""
    rows: object
    exponent: int = 0

    def check(self):
        import torch
        r = self.rows
        if r is None or r.dtype != torch.uint8 or r.dim() != 2 or r.shape[1] != KVQ_ROW_BYTES or r.stride(1) != 1:
            raise ValueError(f"cache rows must be a [slots][{KVQ_ROW_BYTES}] uint8 view with unit column stride")
        if not -KVQ_MAX_EXPONENT <= self.exponent <= KVQ_MAX_EXPONENT:
            raise ValueError(f"cache exponent {self.exponent} outside +-{KVQ_MAX_EXPONENT}")

    def values(self):
        """The fields of an MlaKvqCache."""
        r = self.rows
        m = r.shape[0]
        # the row stride of a one-row tensor is whatever its maker left there
        return r.data_ptr(), r.stride()[0] if m > 1 else KVQ_ROW_BYTES, m, self.exponent

    def tensors(self):
        return dict(rows=self.rows)


def kvq_alloc(slots: int, exponent: int = 0, device="cuda") -> QuantCache:
    """A cache of ``slots`` rows that all stand for zeros."""
    import torch
    rows = torch.zeros((slots, KVQ_ROW_BYTES), dtype=torch.uint8, device=device)
    return QuantCache(rows, exponent)


def _one_device(workspace=None, **tensors):
    """Every tensor on the same CUDA device, the workspace in one piece."""
    tensors["workspace"] = workspace
    _on_cuda(**tensors)
    devs = {t.device for t in tensors.values() if t is not None}
    if len(devs) != 1:
        raise ValueError(f"tensors on different devices: {sorted(map(str, devs))}")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")


def _made_on(stream):
    """Where arrays that a call makes are allocated and filled: on its stream,
    so that the fill precedes the kernels and the memory, once released, is not
    given to another stream's work before they are done."""
    import torch
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _kvq_launch(what: str, f, dev, stream, *args):
    """Calls f(*args, stream) with the tensors' device current."""
    import torch
    index = dev.index
    if stream is not None:
        if stream.device != dev:
            raise ValueError(f"{what}: stream on {stream.device}, tensors on {dev}")
        raw = stream.cuda_stream
    else:
        raw = torch._C._cuda_getCurrentRawStream(index)
    if index == torch._C._cuda_getDevice():
        st = f(*args, raw)
    else:
        with torch.cuda.device(dev):
            st = f(*args, raw)
    if st != MLA_OK:
        raise MlaError(st, what)


def _cache_rows(what: str, f, cache, pack, kv_c, k_pe, slots, workspace, stream, check: bool):
    if check:
        import torch
        cache.check()
        if kv_c is None or kv_c.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("kv_c must be a bfloat16 or float32 tensor")
        for t, name, w in ((kv_c, "kv_c", 512), (k_pe, "k_pe", 64)):
            if t is None or t.dtype != kv_c.dtype or t.dim() != 2 or t.shape[1] != w or t.stride(1) != 1:
                raise ValueError(f"{name} must be a [n][{w}] {kv_c.dtype} view with unit column stride")
            if t.shape[0] > 1 and t.stride(0) < w:
                raise ValueError(f"{name}: rows overlap")
        if k_pe.shape[0] != kv_c.shape[0]:
            raise ValueError("kv_c and k_pe must have the same number of rows")
        _need(slots, "slots", torch.int32, (kv_c.shape[0],))
        _one_device(kv_c=kv_c, k_pe=k_pe, slots=slots, workspace=workspace, **cache.tensors())
    dev = cache.rows.device
    if workspace is None:
        with _made_on(stream):
            workspace = alloc_workspace(KVQ_WORKSPACE_BYTES, dev)
    n = kv_c.shape[0]
    c = pack(*cache.values())
    r = _pack_rows(n, MLA_BF16 if kv_c.element_size() == 2 else MLA_FP32, kv_c.data_ptr(), k_pe.data_ptr(),
                   kv_c.stride()[0] if n > 1 else 512, k_pe.stride()[0] if n > 1 else 64, slots.data_ptr())
    _kvq_launch(what, f, dev, stream, c, r, workspace.data_ptr(), workspace.nbytes)
    return workspace


def kvq_write(cache: QuantCache, kv_c, k_pe, slots, workspace=None, stream=None, check: bool = True):
    """Run mla_kvq_write: quantise row i of kv_c [n][512] and k_pe [n][64]
    (bf16 or fp32; rows 16-byte aligned, any such row stride) into pool slot
    slots[i] (int32; -1 skips, the others differ from each other).  Returns the
    workspace (kvq_check reads its error bits).  check=False skips
    the tensor checks, for a loop that already passed them."""
    return _cache_rows("mla_kvq_write", load().mla_kvq_write, cache, _pack_cache, kv_c, k_pe, slots, workspace, stream,
                       check)


def _cache_read(what: str, f, cache, pack, slots, dtype, kv_c, k_pe, workspace, stream, check: bool):
    if check:
        cache.check()
        if dtype not in ("bf16", "fp32"):
            raise ValueError(f'dtype {dtype!r}, expected "bf16" or "fp32"')
    if kv_c is None or k_pe is None:
        import torch
        dt = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype] if kv_c is None else kv_c.dtype
        with _made_on(stream):
            if kv_c is None:
                kv_c = torch.zeros((slots.shape[0], 512), dtype=dt, device=cache.rows.device)
            if k_pe is None:
                k_pe = torch.zeros((slots.shape[0], 64), dtype=dt, device=cache.rows.device)
    return kv_c, k_pe, _cache_rows(what, f, cache, pack, kv_c, k_pe, slots, workspace, stream, check)


def kvq_read(cache: QuantCache, slots, dtype: str = "bf16", kv_c=None, k_pe=None, workspace=None, stream=None,
             check: bool = True):
    """Run mla_kvq_read: the rows that pool slots ``slots`` stand for, exactly,
    as ``dtype`` ("bf16" or "fp32"; that of kv_c when given).  Rows with slot
    -1 keep what the given arrays hold (zeros in arrays made here, on
    ``stream``).  Returns (kv_c [n][512], k_pe [n][64], workspace)."""
    return _cache_read("mla_kvq_read", load().mla_kvq_read, cache, _pack_cache, slots, dtype, kv_c, k_pe, workspace,
                       stream, check)


@dataclass
class KvqInputs:
    """Device tensors of one attention call over a 4-bit cache.  tree_parent
    None: each node's parent is the node before it (decoding, a linear draft).
    prefix_lens[b] = -1 marks an unused sequence of a padded batch."""
    B: int
    Q: int
    H: int
    scale: float
    q_lat: object           # [B, Q, H, 512] bf16
    q_pe: object            # [B, Q, H, 64] bf16
    cache: QuantCache
    prefix_lens: object     # [B] int32
    page_size: int
    tree_parent: object = None   # [B, Q] int32
    kv_indptr: object = None     # [B + 1] int32    (page_size 1)
    kv_indices: object = None    # int32, not empty (page_size 1)
    block_table: object = None   # [B, max_pages] int32  (page_size > 1)
    window: int = 0
    sinks: int = 0

    def tensors(self):
        return dict(q_lat=self.q_lat, q_pe=self.q_pe, prefix_lens=self.prefix_lens, tree_parent=self.tree_parent,
                    kv_indptr=self.kv_indptr, kv_indices=self.kv_indices, block_table=self.block_table,
                    **self.cache.tensors())

    def check_layout(self):
        """What the C ABI cannot see from pointers.  Raises ValueError."""
        import torch
        B, Q, H = self.B, self.Q, self.H
        self.cache.check()
        for name in ("page_size", "window", "sinks"):
            if not -2 ** 31 <= getattr(self, name) < 2 ** 31:
                raise ValueError(f"{name} {getattr(self, name)} outside 32 bits")
        _need(self.q_lat, "q_lat", torch.bfloat16, (B, Q, H, 512))
        _need(self.q_pe, "q_pe", torch.bfloat16, (B, Q, H, 64))
        _need(self.prefix_lens, "prefix_lens", torch.int32, (B,))
        if self.tree_parent is not None:
            _need(self.tree_parent, "tree_parent", torch.int32, (B, Q))
        if self.page_size == 1:
            _need(self.kv_indptr, "kv_indptr", torch.int32, (B + 1,))
            if self.kv_indices is None or self.kv_indices.dtype != torch.int32 or self.kv_indices.dim() != 1 \
                    or not self.kv_indices.is_contiguous():
                raise ValueError("kv_indices must be a contiguous 1-D int32 tensor")
        elif self.block_table is None or self.block_table.dtype != torch.int32 or self.block_table.dim() != 2 \
                or self.block_table.shape[0] != B or not self.block_table.is_contiguous():
            raise ValueError("block_table must be a contiguous [B][max_pages] int32 tensor")

    def values(self, out=None, lse=None):
        """The fields of an MlaKvqAttnArgs in their order, the cache's in its place."""
        table, tree, paged = self.block_table, self.tree_parent, self.page_size > 1
        return (self.B, self.Q, self.H, *self.cache.values(),
                self.q_lat.data_ptr(), self.q_pe.data_ptr(), self.page_size,
                0 if paged or self.kv_indptr is None else self.kv_indptr.data_ptr(),
                0 if paged or self.kv_indices is None else self.kv_indices.data_ptr(),
                table.data_ptr() if paged and table is not None else 0,
                table.shape[1] if paged and table is not None else 0,
                self.prefix_lens.data_ptr(), 0 if tree is None else tree.data_ptr(), self.window, self.sinks,
                self.scale, 0 if out is None else out.data_ptr(), 0 if lse is None else lse.data_ptr())

    def c_args(self, out=None, lse=None) -> MlaKvqAttnArgs:
        v = self.values(out, lse)
        return MlaKvqAttnArgs(*v[:3], MlaKvqCache(*v[3:7]), *v[7:])


def _attn_workspace_size(what: str, f, ki) -> int:
    import torch
    a = ki.c_args()
    with torch.cuda.device(ki.q_lat.device):
        n = f(ctypes.byref(a))
    if n == 0:
        raise MlaError(MLA_ERR_INVALID_ARG, what)
    return int(n)


def kvq_workspace_size(ki: KvqInputs) -> int:
    return _attn_workspace_size("mla_kvq_attn_workspace_size", load().mla_kvq_attn_workspace_size, ki)


def _cache_attn(what: str, f, pack, size, ki, out, lse, workspace, stream, check: bool):
    dev = ki.q_lat.device
    if out is None or lse is None:
        import torch
        with _made_on(stream):
            if out is None:
                out = torch.zeros((ki.B, ki.Q, ki.H, 512), dtype=torch.bfloat16, device=dev)
            if lse is None:
                lse = torch.zeros((ki.B, ki.Q, ki.H), dtype=torch.float32, device=dev)
    if check:
        import torch
        ki.check_layout()
        _need(out, "out", torch.bfloat16, (ki.B, ki.Q, ki.H, 512))
        _need(lse, "lse", torch.float32, (ki.B, ki.Q, ki.H))
        _one_device(out=out, lse=lse, workspace=workspace, **ki.tensors())
    if workspace is None:
        with _made_on(stream):
            workspace = alloc_workspace(size(ki), dev)
    _kvq_launch(what, f, dev, stream, pack(*ki.values(out, lse)), workspace.data_ptr(), workspace.nbytes)
    return out, lse


def _attn_selftest(what: str, f, pack, ki, out, lse, workspace, hold_ns: int, stream):
    import torch
    ki.check_layout()
    _need(out, "out", torch.bfloat16, (ki.B, ki.Q, ki.H, 512))
    _need(lse, "lse", torch.float32, (ki.B, ki.Q, ki.H))
    _one_device(out=out, lse=lse, workspace=workspace, **ki.tensors())
    _kvq_launch(what, lambda args, ws, n, raw: f(args, ws, n, ctypes.c_uint64(int(hold_ns)), raw), ki.q_lat.device,
                stream, pack(*ki.values(out, lse)), workspace.data_ptr(), workspace.nbytes)


def _cache_check(what: str, f, workspace, stream) -> int:
    import torch
    bits = ctypes.c_uint32(0)
    with torch.cuda.device(workspace.device):
        st = f(ctypes.c_void_p(_ptr(workspace)), _stream(stream), ctypes.byref(bits))
    if st not in (MLA_OK, MLA_ERR_DEVICE_CHECK):
        raise MlaError(st, what)
    return int(bits.value)


def kvq_attn(ki: KvqInputs, out=None, lse=None, workspace=None, stream=None, check: bool = True):
    """Run mla_kvq_attn; returns (out [B,Q,H,512] bf16, lse [B,Q,H] fp32).
    Rows of unused sequences keep what the given arrays hold (zeros in arrays
    made here, on ``stream``).  kvq_check reads the call's error bits from a
    workspace that was given; one made here is gone with the call.  check=False
    skips the tensor checks (a loop that already passed them)."""
    return _cache_attn("mla_kvq_attn", load().mla_kvq_attn, _pack_attn, kvq_workspace_size, ki, out, lse, workspace,
                       stream, check)


def kvq_selftest_timeout(ki: KvqInputs, out, lse, workspace, hold_ns: int, stream=None):
    """Run mla_kvq_selftest_timeout: the attention call with its waits limited
    to hold_ns and one of its products held back; read the outcome with
    kvq_check()."""
    _attn_selftest("mla_kvq_selftest_timeout", load().mla_kvq_selftest_timeout, _pack_attn, ki, out, lse, workspace,
                   hold_ns, stream)


def kvq_check(workspace, stream=None) -> int:
    """Synchronise and return the device error bits that the last kvq call on
    this workspace left."""
    return _cache_check("mla_kvq_check", load().mla_kvq_check, workspace, stream)


# ----------------------------------------------------------------------------
# paged 8-bit latent cache (include/mla_kv8.h)
# ----------------------------------------------------------------------------
@dataclass
class BlockCache:
    """A pool of 8-bit cache rows under one scale per block of ``block`` slots:
    ``rows`` is a uint8 [slots][640] tensor or view (row stride a multiple of 32
    bytes), ``scales`` an int32 [ceil(slots / block)] tensor of scale words (0: the
    block holds no rows), ``exponent`` the power of two the latents are scaled by."""
    rows: object
    scales: object
    block: int = 64
    exponent: int = 0

    def check(self):
        import torch
        r, s = self.rows, self.scales
        if r is None or r.dtype != torch.uint8 or r.dim() != 2 or r.shape[1] != KV8_ROW_BYTES or r.stride(1) != 1:
            raise ValueError(f"cache rows must be a [slots][{KV8_ROW_BYTES}] uint8 view with unit column stride")
        if r.shape[0] > 1 and r.stride(0) < KV8_ROW_BYTES:
            raise ValueError("cache rows overlap")
        if not 1 <= self.block < 2 ** 31:
            raise ValueError(f"cache block {self.block}, expected at least one slot")
        _need(s, "scales", torch.int32, (-(-r.shape[0] // self.block),))
        if not -KV8_MAX_EXPONENT <= self.exponent <= KV8_MAX_EXPONENT:
            raise ValueError(f"cache exponent {self.exponent} outside +-{KV8_MAX_EXPONENT}")

    def values(self):
        """The fields of an MlaKv8Cache."""
        r = self.rows
        m = r.shape[0]
        # the row stride of a one-row tensor is whatever its maker left there
        return (r.data_ptr(), r.stride()[0] if m > 1 else KV8_ROW_BYTES, m, self.scales.data_ptr(), self.block,
                self.exponent)

    def tensors(self):
        return dict(rows=self.rows, scales=self.scales)


def kv8_alloc(slots: int, block: int = 64, exponent: int = 0, device="cuda") -> BlockCache:
    """An empty cache of ``slots`` rows.  Where kv_tables hands out its pages, ``block`` should divide
    their size: blocks that are not inside a page are never emptied, and their scales never fall."""
    import torch
    return BlockCache(torch.zeros((slots, KV8_ROW_BYTES), dtype=torch.uint8, device=device),
                      torch.zeros((-(-slots // block),), dtype=torch.int32, device=device), block, exponent)


def kv8_write(cache: BlockCache, kv_c, k_pe, slots, workspace=None, stream=None, check: bool = True):
    """Run mla_kv8_write: quantise row i of kv_c [n][512] and k_pe [n][64] (bf16 or
    fp32; rows 16-byte aligned, any such row stride) into pool slot slots[i] (int32;
    -1 skips, the others differ from each other), raising the scales of the blocks
    they go to as far as they need.  Returns the workspace (kv8_check reads its
    error bits).  check=False skips the tensor checks, for a loop that already
    passed them."""
    return _cache_rows("mla_kv8_write", load().mla_kv8_write, cache, _pack_cache8, kv_c, k_pe, slots, workspace,
                       stream, check)


def kv8_read(cache: BlockCache, slots, dtype: str = "bf16", kv_c=None, k_pe=None, workspace=None, stream=None,
             check: bool = True):
    """Run mla_kv8_read: the rows that pool slots ``slots`` stand for, as ``dtype``
    ("bf16" or "fp32"; that of kv_c when given).  Rows with slot -1 keep what the
    given arrays hold (zeros in arrays made here, on ``stream``).  Returns
    (kv_c [n][512], k_pe [n][64], workspace)."""
    return _cache_read("mla_kv8_read", load().mla_kv8_read, cache, _pack_cache8, slots, dtype, kv_c, k_pe, workspace,
                       stream, check)


@dataclass
class Kv8Inputs(KvqInputs):
    """Device tensors of one attention call over an 8-bit cache: the fields of
    KvqInputs with ``cache`` a BlockCache."""

    def c_args(self, out=None, lse=None) -> MlaKv8AttnArgs:
        v = self.values(out, lse)
        return MlaKv8AttnArgs(*v[:3], MlaKv8Cache(*v[3:9]), *v[9:])


def kv8_workspace_size(ki: Kv8Inputs) -> int:
    return _attn_workspace_size("mla_kv8_attn_workspace_size", load().mla_kv8_attn_workspace_size, ki)


def kv8_attn(ki: Kv8Inputs, out=None, lse=None, workspace=None, stream=None, check: bool = True):
    """Run mla_kv8_attn; returns (out [B,Q,H,512] bf16, lse [B,Q,H] fp32); as
    kvq_attn, with kv8_check for the error bits."""
    return _cache_attn("mla_kv8_attn", load().mla_kv8_attn, _pack_attn8, kv8_workspace_size, ki, out, lse, workspace,
                       stream, check)


def kv8_selftest_timeout(ki: Kv8Inputs, out, lse, workspace, hold_ns: int, stream=None):
    """Run mla_kv8_selftest_timeout, as kvq_selftest_timeout."""
    _attn_selftest("mla_kv8_selftest_timeout", load().mla_kv8_selftest_timeout, _pack_attn8, ki, out, lse, workspace,
                   hold_ns, stream)


def kv8_check(workspace, stream=None) -> int:
    """Synchronise and return the device error bits that the last kv8 or kv_tables
    call on this workspace left."""
    return _cache_check("mla_kv8_check", load().mla_kv8_check, workspace, stream)


# ----------------------------------------------------------------------------
# page tables of a step (include/mla_kv_tables.h)
# ----------------------------------------------------------------------------
@dataclass
class TableInputs:
    """Device tensors of the page tables: what the requests need (prefix_lens, and
    new_lens or Q) and the state that a call brings to it (block_table, pages_held,
    free_ring, free_state)."""
    page_size: int
    prefix_lens: object     # [B] int32, -1: unused row
    block_table: object     # [B, max_pages] int32
    pages_held: object      # [B] int32
    free_ring: object       # [ring] int32 page ids
    free_state: object      # [3] int64: head, tail, 0
    num_pages: int
    Q: int = 1              # new tokens of each request, where new_lens is None
    new_lens: object = None  # [B] int32

    def tensors(self):
        return dict(prefix_lens=self.prefix_lens, block_table=self.block_table, pages_held=self.pages_held,
                    free_ring=self.free_ring, free_state=self.free_state, new_lens=self.new_lens)

    def check_layout(self):
        """What the C ABI cannot see from pointers.  Raises ValueError."""
        import torch
        for name in ("page_size", "num_pages", "Q"):
            if not -2 ** 31 <= getattr(self, name) < 2 ** 31:
                raise ValueError(f"{name} {getattr(self, name)} outside 32 bits")
        t = self.block_table
        if t is None or t.dtype != torch.int32 or t.dim() != 2 or not t.is_contiguous():
            raise ValueError("block_table must be a contiguous [B][max_pages] int32 tensor")
        B = t.shape[0]
        _need(self.prefix_lens, "prefix_lens", torch.int32, (B,))
        _need(self.pages_held, "pages_held", torch.int32, (B,))
        if self.new_lens is not None:
            _need(self.new_lens, "new_lens", torch.int32, (B,))
        _need(self.free_state, "free_state", torch.int64, (3,))
        _flat(self.free_ring, "free_ring")


def kv_tables_alloc(B: int, max_pages: int, num_pages: int, page_size: int, device="cuda") -> TableInputs:
    """The tables of B rows that hold nothing, every page free; prefix_lens are -1."""
    import torch
    i32 = dict(dtype=torch.int32, device=device)
    return TableInputs(page_size=page_size, prefix_lens=torch.full((B,), -1, **i32),
                       block_table=torch.full((B, max_pages), -1, **i32), pages_held=torch.zeros((B,), **i32),
                       free_ring=torch.arange(num_pages, **i32),
                       free_state=torch.tensor([0, num_pages, 0], dtype=torch.int64, device=device),
                       num_pages=num_pages)


def _flat(t, name: str):
    import torch
    if t is None or t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 1-D int32 tensor")


def kv_tables(ti: TableInputs, slots=None, kv_indptr=None, kv_indices=None, cache: Optional[BlockCache] = None,
              workspace=None, stream=None, check: bool = True):
    """Run mla_kv_tables: bring block_table, pages_held and the ring of free pages to
    this step's lengths, in place, and fill the given outputs: ``slots`` of the new
    tokens ([B][Q] or flat; with new_lens any flat length, -1 behind the last),
    ``kv_indptr`` [B+1] and ``kv_indices``, the page-size-1 tables.  With ``cache`` the
    blocks that lie inside a page that is handed out become empty.  Returns the workspace
    (kv8_check reads its error bits)."""
    if check:
        import torch
        ti.check_layout()
        B = ti.block_table.shape[0]
        if slots is not None and (slots.dtype != torch.int32 or not slots.is_contiguous()
                                  or (ti.new_lens is None and slots.numel() != B * ti.Q)):
            raise ValueError("slots must be contiguous int32, of B * Q entries where new_lens is not given")
        if kv_indptr is not None:
            _need(kv_indptr, "kv_indptr", torch.int32, (B + 1,))
        if kv_indices is not None:
            _flat(kv_indices, "kv_indices")
        scales = None
        if cache is not None:
            cache.check()
            scales = cache.scales
            if cache.rows.shape[0] < ti.num_pages * ti.page_size:
                raise ValueError("the cache has fewer slots than the pages")
        _one_device(slots=slots, kv_indptr=kv_indptr, kv_indices=kv_indices, scales=scales, workspace=workspace,
                    **ti.tensors())
    t = ti.block_table
    dev = t.device
    if workspace is None:
        with _made_on(stream):
            workspace = alloc_workspace(KV_TABLES_WORKSPACE_BYTES, dev)

    def p(x):
        return 0 if x is None else x.data_ptr()
    args = _pack_tables(t.shape[0], ti.Q, ti.page_size, t.shape[1], ti.num_pages, p(ti.prefix_lens), p(ti.new_lens),
                        p(t), p(ti.pages_held), p(ti.free_ring), p(ti.free_state), ti.free_ring.shape[0],
                        p(slots), 0 if slots is None else slots.numel(), p(kv_indptr), p(kv_indices),
                        0 if kv_indices is None else kv_indices.shape[0], 0 if cache is None else p(cache.scales),
                        0 if cache is None else cache.block)
    _kvq_launch("mla_kv_tables", load().mla_kv_tables, dev, stream, args, workspace.data_ptr(), workspace.nbytes)
    return workspace
