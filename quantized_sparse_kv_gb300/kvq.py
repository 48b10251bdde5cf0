"""Thin Python binding of the kvq C ABI (``include/kvq.h``).

Argument marshalling only: every step of packing and attention runs in the
CUDA kernels of ``libkvq.so``. PyTorch provides device memory and the current
stream. There is no CPU fallback: if the library is missing or a call fails,
these functions raise.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

F32, BF16, MXFP8 = 0, 1, 2
DTYPES = {"f32": F32, "bf16": BF16, "mxfp8": MXFP8}
TORCH_OF = {F32: torch.float32, BF16: torch.bfloat16}

STATUS = {0: "KVQ_OK", 1: "KVQ_ERR_ARG", 2: "KVQ_ERR_ALIGN", 3: "KVQ_ERR_UNSUPPORTED",
          4: "KVQ_ERR_WORKSPACE", 5: "KVQ_ERR_CUDA"}
DEV_INDEX, DEV_DUP, DEV_TIMEOUT, DEV_BOUNDS = 1, 2, 4, 8
# columns of kv_attend_stats (include/kvq.h, KVQ_STAT_*)
STATS = ("entropy", "support", "top1", "top5", "top10", "zero", "p_zero", "p_tv", "p_sum",
         "qk_tv", "qk_agree")

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvq.so")
# the same library built with every kernel's access ranges checked (KVQ_DEBUG)
DEBUG_LIB_PATH = os.path.join(_HERE, "libkvq_debug.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "kvq.h")


class KvqError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)}")
        self.status = status


class KvqCacheStruct(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("n_tokens", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("recent", ctypes.c_int32),
        ("kwin_dtype", ctypes.c_int32), ("vwin_dtype", ctypes.c_int32),
        ("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
        ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
        ("k_window", ctypes.c_void_p), ("v_window", ctypes.c_void_p),
        ("k_window_e8m0", ctypes.c_void_p),
        ("header", ctypes.c_uint32 * 4),
        ("cap_groups", ctypes.c_int32), ("cap_window", ctypes.c_int32),
    ]


class KvqRopeScaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("factor", ctypes.c_double),
                ("original", ctypes.c_double), ("p0", ctypes.c_double), ("p1", ctypes.c_double)]


class KvqRopeTensor(ctypes.Structure):
    _fields_ = [("inp", ctypes.c_void_p), ("out", ctypes.c_void_p), ("heads", ctypes.c_int32),
                ("rotate", ctypes.c_int32), ("stride_b", ctypes.c_int64),
                ("stride_h", ctypes.c_int64), ("stride_t", ctypes.c_int64)]


class KvqSummary(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("block", ctypes.c_int32), ("cap_blocks", ctypes.c_int32)]


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libkvq.so (built in-tree by ``quantized_sparse_kv_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with quantized_sparse_kv_gb300.build.build()")
    lib = ctypes.CDLL(path)
    vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    cp = ctypes.POINTER(KvqCacheStruct)
    lib.kvq_cache_sizes.argtypes = [i32, i32, i32, i32, i32, i32, i32, ctypes.POINTER(sz)]
    lib.kvq_cache_sizes.restype = i32
    lib.kvq_cache_sizes_reserved.argtypes = [i32, i32, i32, i32, i32, i32, i32,
                                             ctypes.POINTER(sz)]
    lib.kvq_cache_sizes_reserved.restype = i32
    lib.kv_append.argtypes = [cp, vp, vp, i32, i32, i32, vp, vp]
    lib.kv_append.restype = i32
    lib.kv_attend_stats.argtypes = [cp, vp, i32, i32, i32, f32, vp, vp, vp, ctypes.POINTER(sz),
                                    vp, vp]
    lib.kv_attend_stats.restype = i32
    lib.kv_attend_candidates_topk.argtypes = [cp, vp, i32, i32, i32, vp, i32, i32, f32, vp, i32,
                                              vp, vp, vp]
    lib.kv_attend_candidates_topk.restype = i32
    lib.kv_attend_candidates_block.argtypes = [cp, vp, i32, i32, i32, vp, i32, i32, f32, vp, i32,
                                               vp, ctypes.POINTER(sz), vp, vp]
    lib.kv_attend_candidates_block.restype = i32
    lib.kv_attend_region_drop.argtypes = [cp, vp, i32, i32, i32, f32, ctypes.POINTER(i32), i32,
                                          ctypes.c_uint32, vp, i32, vp, ctypes.POINTER(sz), vp,
                                          vp]
    lib.kv_attend_region_drop.restype = i32
    lib.kvq_cache_bytes.argtypes = [i32, i32, i32, i32, i32, i32, i32]
    lib.kvq_cache_bytes.restype = sz
    lib.kv_pack.argtypes = [vp, vp, i32, cp, vp, vp]
    lib.kv_pack.restype = i32
    lib.kv_attend.argtypes = [cp, vp, i32, i32, i32, f32, vp, i32, ctypes.POINTER(i32), i32, vp,
                              vp, ctypes.POINTER(sz), vp, vp]
    lib.kv_attend.restype = i32
    lib.kv_attend_candidates.argtypes = [cp, vp, i32, i32, i32, vp, i32, i32, f32, vp, i32, vp,
                                         ctypes.POINTER(sz), vp, vp]
    lib.kv_attend_candidates.restype = i32
    lib.kvq_rope_turns.argtypes = [i32, ctypes.c_double, ctypes.POINTER(KvqRopeScaling),
                                   ctypes.POINTER(ctypes.c_uint64), ctypes.POINTER(f32)]
    lib.kvq_rope_turns.restype = i32
    lib.kv_rope.argtypes = [ctypes.POINTER(KvqRopeTensor), i32, i32, i32, i32, i32, i32, i32, vp,
                            f32, i32, vp, vp, vp]
    lib.kv_rope.restype = i32
    lib.kv_attend_tree.argtypes = [cp, vp, i32, i32, i32, vp, vp, i32, vp, f32, vp, i32, vp,
                                   ctypes.POINTER(sz), vp, vp]
    lib.kv_attend_tree.restype = i32
    sp = ctypes.POINTER(KvqSummary)
    lib.kv_block_summary.argtypes = [cp, sp, i32, vp, vp]
    lib.kv_block_summary.restype = i32
    lib.kv_block_values.argtypes = [cp, sp, i32, vp, vp, vp]
    lib.kv_block_values.restype = i32
    lib.kv_select_blocks.argtypes = [cp, sp, vp, i32, i32, i32, i32, i32, vp, vp,
                                     ctypes.POINTER(sz), vp, vp]
    lib.kv_select_blocks.restype = i32
    lib.kv_attend_blocks.argtypes = [cp, vp, i32, i32, i32, vp, i32, i32, f32, vp, i32, vp,
                                     ctypes.POINTER(sz), vp, vp]
    lib.kv_attend_blocks.restype = i32
    lib.kvq_last_launch_count.argtypes = []
    lib.kvq_last_launch_count.restype = i32
    lib.kvq_last_path.argtypes = []
    lib.kvq_last_path.restype = ctypes.c_char_p
    lib.kvq_debug_set.argtypes = [ctypes.c_uint32, i32]
    lib.kvq_debug_set.restype = None
    lib.kvq_debug_checks.argtypes = []
    lib.kvq_debug_checks.restype = i32
    _lib = lib
    return lib


def header_functions(path: str = HEADER) -> list[str]:
    """Names of the functions include/kvq.h declares."""
    text = open(path, encoding="utf-8").read()
    return re.findall(r"KVQ_API\s+[\w\s\*]+?\b(\w+)\s*\(", text)


def _check(status: int, what: str):
    if status != 0:
        raise KvqError(status, what)


def cache_sizes(batch, kv_heads, n_tokens, head_dim, recent, kwin=F32, vwin=F32) -> list[int]:
    lib = load_library()
    out = (ctypes.c_size_t * 8)()
    _check(lib.kvq_cache_sizes(batch, kv_heads, n_tokens, head_dim, recent, kwin, vwin, out),
           "kvq_cache_sizes")
    return list(out)


def cache_sizes_reserved(batch, kv_heads, head_dim, kwin, vwin, cap_groups, cap_window) -> list[int]:
    lib = load_library()
    out = (ctypes.c_size_t * 8)()
    _check(lib.kvq_cache_sizes_reserved(batch, kv_heads, head_dim, kwin, vwin, cap_groups,
                                        cap_window, out), "kvq_cache_sizes_reserved")
    return list(out)


def cache_bytes(batch, kv_heads, n_tokens, head_dim, recent, kwin=F32, vwin=F32) -> int:
    return int(load_library().kvq_cache_bytes(batch, kv_heads, n_tokens, head_dim, recent, kwin,
                                              vwin))


def _dtype(x) -> int:
    return DTYPES[x] if isinstance(x, str) else int(x)


def _stream() -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _one_device(*tensors) -> torch.device:
    """The CUDA device all the tensors (None left out) live on."""
    devs = {t.device for t in tensors if t is not None}
    if len(devs) != 1 or next(iter(devs)).type != "cuda":
        raise ValueError("all tensors must live on one CUDA device")
    return next(iter(devs))


_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda i: torch.cuda.current_stream(i).cuda_stream)


class _Prepared:
    """Base of the prepared calls below: ``run()`` issues them on the current
    stream of their tensors' device, with the arguments marshalled once (a
    decoding step is bound by the host as much as by the GPU) and, for calls
    over a cache, again by the first run after the cache has grown. A captured
    run replays with the cache's lengths at its capture. A prepared call has
    one workspace: runs that may overlap, on several streams or from captured
    graphs, each need an object of their own."""

    def run(self, *args, **kw):
        if torch.cuda.current_device() != self.device.index:
            with torch.cuda.device(self.device):
                return self._run(*args, **kw)
        return self._run(*args, **kw)

    def _raw_stream(self) -> int:
        # the handle without the Stream object around it, about 2 us a call cheaper
        return _current_raw_stream(self.device.index)

    def launches(self) -> int:
        return int(self.lib.kvq_last_launch_count())

    def _workspace(self, need: int):
        """Workspace of at least ``need`` bytes. A larger one (the cache grew)
        takes half as much again as the last, and the last stays: a graph
        captured before may still be replayed and write to it."""
        if self.ws is None or need > self.ws.numel():
            if self.ws is not None:
                self._kept.append(self.ws)
                need = max(need, self.ws.numel() * 3 // 2)
            self.ws = torch.empty(max(need, 256), dtype=torch.uint8, device=self.device)
        self.ws_bytes = ctypes.c_size_t(self.ws.numel())


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(t.data_ptr() if t is not None and t.numel() else None)


class PackedCache:
    """Device arrays of one packed cache plus the C descriptor pointing at them.

    ``reserve=(cap_groups, cap_window)`` lays the arrays out with room for
    kv_append: cap_groups K groups (32 per group V rows) and cap_window window
    rows per (sequence, head)."""

    def __init__(self, batch, kv_heads, n_tokens, head_dim, recent, kwin="f32", vwin="f32",
                 device="cuda", reserve=None):
        self.batch, self.kv_heads, self.n_tokens = batch, kv_heads, n_tokens
        self.head_dim, self.recent = head_dim, recent
        self.kwin, self.vwin = _dtype(kwin), _dtype(vwin)
        self.cut = n_tokens - recent
        self.gk = -(-self.cut // 32)
        self.reserve = tuple(reserve) if reserve else (0, 0)
        if reserve:
            cap_g, cap_w = self.reserve
            if cap_g < self.gk or cap_w < recent:
                raise ValueError("reserve is smaller than the cache")
            rows_g, rows_v, rows_w = cap_g, 32 * cap_g, cap_w
        else:
            rows_g, rows_v, rows_w = self.gk, self.cut, recent
        self.sizes = cache_sizes(batch, kv_heads, n_tokens, head_dim, recent, self.kwin, self.vwin)
        u8 = torch.uint8
        b, h, d = batch, kv_heads, head_dim
        self.k_codes = torch.empty((b, h, rows_g, 32, d // 2), dtype=u8, device=device)
        self.k_scales = torch.empty((b, h, rows_g, d), dtype=torch.float32, device=device)
        self.v_codes = torch.empty((b, h, rows_v, d // 2), dtype=u8, device=device)
        self.v_scales = torch.empty((b, h, rows_v, d // 32), dtype=torch.float32, device=device)
        kdt = u8 if self.kwin == MXFP8 else TORCH_OF[self.kwin]
        self.k_window = torch.empty((b, h, rows_w, d), dtype=kdt, device=device)
        self.v_window = torch.empty((b, h, rows_w, d), dtype=TORCH_OF[self.vwin], device=device)
        self.k_window_e8m0 = torch.empty((b, h, rows_w, d // 32) if self.kwin == MXFP8 else (0,),
                                         dtype=u8, device=device)
        self.struct = KvqCacheStruct(
            batch, kv_heads, n_tokens, head_dim, recent, self.kwin, self.vwin,
            _ptr(self.k_codes), _ptr(self.k_scales), _ptr(self.v_codes), _ptr(self.v_scales),
            _ptr(self.k_window), _ptr(self.v_window), _ptr(self.k_window_e8m0),
            (ctypes.c_uint32 * 4)(0, 0, 0, 0), self.reserve[0], self.reserve[1])
        self.ref = ctypes.byref(self.struct)

    def _sync_shape(self):
        """Take n_tokens and recent back from the descriptor (kv_append moves them)."""
        self.n_tokens, self.recent = int(self.struct.n_tokens), int(self.struct.recent)
        self.cut = self.n_tokens - self.recent
        self.gk = -(-self.cut // 32)
        self.sizes = cache_sizes(self.batch, self.kv_heads, self.n_tokens, self.head_dim,
                                 self.recent, self.kwin, self.vwin)

    def used(self) -> dict:
        """Views of the filled part of every array (the tight layout's content)."""
        return {"k_codes": self.k_codes[:, :, :self.gk], "k_scales": self.k_scales[:, :, :self.gk],
                "v_codes": self.v_codes[:, :, :self.cut], "v_scales": self.v_scales[:, :, :self.cut],
                "k_window": self.k_window[:, :, :self.recent],
                "v_window": self.v_window[:, :, :self.recent]}

    @property
    def header(self):
        return list(self.struct.header)

    def payload_bytes(self) -> int:
        return int(sum(self.sizes))


def new_status(device="cuda") -> torch.Tensor:
    return torch.zeros(4, dtype=torch.int32, device=device)


def read_status(status: torch.Tensor) -> int:
    """Synchronise on the current stream and return the device status word."""
    torch.cuda.current_stream().synchronize()
    return int(status[0].item())


def pack(k: torch.Tensor, v: torch.Tensor, recent: int, kwin="f32", vwin=None,
         status: torch.Tensor | None = None, out: PackedCache | None = None,
         reserve=None) -> PackedCache:
    """kv_pack: k, v (batch, kv_heads, N, D) fp32 or bf16 on the GPU.

    ``out`` reuses the arrays of an existing cache of the same shape;
    ``reserve=(cap_groups, cap_window)`` leaves room for kv_append."""
    if k.dtype not in (torch.float32, torch.bfloat16) or v.dtype != k.dtype:
        raise TypeError("k and v must both be float32 or bfloat16")
    k = k.contiguous()
    v = v.contiguous()
    b, h, n, d = k.shape
    if out is None:
        vw = vwin if vwin is not None else ("f32" if _dtype(kwin) == F32 else "bf16")
        out = PackedCache(b, h, n, d, recent, kwin, vw, device=k.device, reserve=reserve)
    in_dt = F32 if k.dtype == torch.float32 else BF16
    lib = load_library()
    _check(lib.kv_pack(_ptr(k), _ptr(v), in_dt, out.ref,
                       _ptr(status) if status is not None else None, _stream()), "kv_pack")
    return out


class Attend:
    """A prepared kv_attend call: output, region-mass, workspace and status
    buffers are allocated once; ``run()`` only re-issues the C call."""

    def __init__(self, cache: PackedCache, q: torch.Tensor, sm_scale: float = 0.0,
                 out_dtype=None, region_bounds=None, out=None):
        self.lib = load_library()
        self.cache = cache
        self.q = q.contiguous()
        if self.q.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("q must be float32 or bfloat16")
        b, hq, nq, d = self.q.shape
        if b != cache.batch or d != cache.head_dim:
            raise ValueError("q does not match the cache")
        self.q_dt = F32 if self.q.dtype == torch.float32 else BF16
        self.out_dt = _dtype(out_dtype) if out_dtype is not None else self.q_dt
        self.out = out if out is not None else torch.empty(
            (b, hq, nq, d), dtype=TORCH_OF[self.out_dt], device=self.q.device)
        self.hq, self.nq, self.sm_scale = hq, nq, float(sm_scale or 0.0)
        if region_bounds is not None:
            rb = [int(x) for x in region_bounds]
            self.n_regions = len(rb) - 1
            self.bounds = (ctypes.c_int32 * len(rb))(*rb)
            self.mass = torch.empty((b, hq, nq, self.n_regions), dtype=torch.float32,
                                    device=self.q.device)
        else:
            self.n_regions, self.bounds, self.mass = 0, None, None
        self.status = new_status(self.q.device)
        need = ctypes.c_size_t(0)
        self._call(None, need)
        self.ws = torch.empty(max(int(need.value), 256), dtype=torch.uint8, device=self.q.device)
        self.ws_bytes = ctypes.c_size_t(self.ws.numel())
        self.path = None

    def _call(self, ws, ws_bytes):
        st = self.lib.kv_attend(self.cache.ref, _ptr(self.q), self.q_dt, self.hq, self.nq,
                                self.sm_scale, _ptr(self.out), self.out_dt, self.bounds,
                                self.n_regions, _ptr(self.mass), ws, ctypes.byref(ws_bytes),
                                _ptr(self.status), _stream())
        _check(st, "kv_attend")

    def run(self):
        self._call(_ptr(self.ws), self.ws_bytes)
        self.path = self.lib.kvq_last_path().decode()
        return self.out

    def launches(self) -> int:
        return int(self.lib.kvq_last_launch_count())


def attend(cache: PackedCache, q: torch.Tensor, sm_scale: float = 0.0, out_dtype=None,
           region_bounds=None):
    """kv_attend; returns (out, region_mass or None, path)."""
    a = Attend(cache, q, sm_scale, out_dtype, region_bounds)
    a.run()
    return a.out, a.mass, a.path


class AttendCandidates:
    """A prepared kv_attend_candidates call (see Attend)."""

    def __init__(self, cache: PackedCache, q: torch.Tensor, idx: torch.Tensor,
                 sm_scale: float = 0.0, out_dtype=None, validate: bool = False, out=None):
        self.lib = load_library()
        self.cache = cache
        self.q = q.contiguous()
        self.idx = idx.to(torch.int32).contiguous()
        b, hq, nq, d = self.q.shape
        if tuple(self.idx.shape[:3]) != (b, hq, nq):
            raise ValueError("idx must be (batch, q_heads, n_q, C)")
        self.q_dt = F32 if self.q.dtype == torch.float32 else BF16
        self.out_dt = _dtype(out_dtype) if out_dtype is not None else self.q_dt
        self.out = out if out is not None else torch.empty(
            (b, hq, nq, d), dtype=TORCH_OF[self.out_dt], device=self.q.device)
        self.hq, self.nq, self.c = hq, nq, int(self.idx.shape[3])
        self.sm_scale, self.validate = float(sm_scale or 0.0), int(bool(validate))
        self.status = new_status(self.q.device)
        need = ctypes.c_size_t(0)
        self._call(None, need)
        self.ws = torch.empty(max(int(need.value), 256), dtype=torch.uint8, device=self.q.device)
        self.ws_bytes = ctypes.c_size_t(self.ws.numel())

    def _call(self, ws, ws_bytes):
        st = self.lib.kv_attend_candidates(self.cache.ref, _ptr(self.q), self.q_dt, self.hq,
                                           self.nq, _ptr(self.idx), self.c, self.validate,
                                           self.sm_scale, _ptr(self.out), self.out_dt, ws,
                                           ctypes.byref(ws_bytes), _ptr(self.status), _stream())
        _check(st, "kv_attend_candidates")

    def run(self):
        self._call(_ptr(self.ws), self.ws_bytes)
        return self.out

    def launches(self) -> int:
        return int(self.lib.kvq_last_launch_count())


def attend_candidates(cache: PackedCache, q: torch.Tensor, idx: torch.Tensor,
                      sm_scale: float = 0.0, out_dtype=None, validate: bool = False):
    """kv_attend_candidates; returns (out, status tensor)."""
    a = AttendCandidates(cache, q, idx, sm_scale, out_dtype, validate)
    a.run()
    return a.out, a.status


def debug_set(wait_limit_ns: int = 0, drop_item: int = -1):
    """Failure-test hook (see kvq_debug_set in include/kvq.h)."""
    load_library().kvq_debug_set(int(wait_limit_ns), int(drop_item))


def append(cache: PackedCache, k_new: torch.Tensor, v_new: torch.Tensor, window: int,
           status: torch.Tensor | None = None) -> PackedCache:
    """kv_append: k_new, v_new (batch, kv_heads, T, D) fp32 or bf16 on the GPU,
    added after the cache's tokens; the window keeps at least ``window`` tokens
    and whole 32-token groups move from its oldest end into int4."""
    if k_new.dtype not in (torch.float32, torch.bfloat16) or v_new.dtype != k_new.dtype:
        raise TypeError("k_new and v_new must both be float32 or bfloat16")
    k_new, v_new = k_new.contiguous(), v_new.contiguous()
    b, h, t, d = k_new.shape
    if (b, h, d) != (cache.batch, cache.kv_heads, cache.head_dim) or v_new.shape != k_new.shape:
        raise ValueError("new tokens do not match the cache")
    in_dt = F32 if k_new.dtype == torch.float32 else BF16
    lib = load_library()
    _check(lib.kv_append(cache.ref, _ptr(k_new), _ptr(v_new), in_dt, t, window,
                         _ptr(status) if status is not None else None, _stream()), "kv_append")
    cache._sync_shape()
    return cache


def attend_stats(cache: PackedCache, q: torch.Tensor, signs: torch.Tensor | None = None,
                 sm_scale: float = 0.0, status: torch.Tensor | None = None) -> torch.Tensor:
    """kv_attend_stats: observer statistics of the softmax rows of q over the
    cache; returns float32 (batch, q_heads, n_q, len(STATS)), columns STATS.
    ``signs`` (D,) of +-1 turns on the signed Hadamard rotation of the MXFP8
    Q/K path."""
    q = q.contiguous()
    if q.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("q must be float32 or bfloat16")
    b, hq, nq, d = q.shape
    out = torch.empty((b, hq, nq, len(STATS)), dtype=torch.float32, device=q.device)
    sg = None
    if signs is not None:
        sg = signs.to(device=q.device, dtype=torch.float32).contiguous()
        if sg.shape != (d,):
            raise ValueError("signs must have head_dim entries")
    lib = load_library()
    q_dt = F32 if q.dtype == torch.float32 else BF16
    need = ctypes.c_size_t(0)
    _check(lib.kv_attend_stats(cache.ref, _ptr(q), q_dt, hq, nq, float(sm_scale or 0.0), _ptr(sg),
                               _ptr(out), None, ctypes.byref(need), None, _stream()),
           "kv_attend_stats")
    ws = torch.empty(max(int(need.value), 256), dtype=torch.uint8, device=q.device)
    ws_bytes = ctypes.c_size_t(ws.numel())
    _check(lib.kv_attend_stats(cache.ref, _ptr(q), q_dt, hq, nq, float(sm_scale or 0.0), _ptr(sg),
                               _ptr(out), _ptr(ws), ctypes.byref(ws_bytes),
                               _ptr(status) if status is not None else None, _stream()),
           "kv_attend_stats")
    return out


def attend_candidates_topk(cache: PackedCache, q: torch.Tensor, idx: torch.Tensor, top_k: int,
                           sm_scale: float = 0.0, out_dtype=None):
    """kv_attend_candidates_topk: attend only the top_k of each row's listed
    keys by exact score. Returns (out, selected positions, status tensor)."""
    q = q.contiguous()
    if q.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("q must be float32 or bfloat16")
    idx = idx.to(torch.int32).contiguous()
    b, hq, nq, d = q.shape
    if tuple(idx.shape[:3]) != (b, hq, nq):
        raise ValueError("idx must be (batch, q_heads, n_q, C)")
    q_dt = F32 if q.dtype == torch.float32 else BF16
    out_dt = _dtype(out_dtype) if out_dtype is not None else q_dt
    out = torch.empty((b, hq, nq, d), dtype=TORCH_OF[out_dt], device=q.device)
    selected = torch.empty((b, hq, nq, top_k), dtype=torch.int32, device=q.device)
    status = new_status(q.device)
    lib = load_library()
    _check(lib.kv_attend_candidates_topk(cache.ref, _ptr(q), q_dt, hq, nq, _ptr(idx),
                                         idx.shape[3], top_k, float(sm_scale or 0.0), _ptr(out),
                                         out_dt, _ptr(selected), _ptr(status), _stream()),
           "kv_attend_candidates_topk")
    return out, selected, status


class AttendCandidatesBlock:
    """A prepared kv_attend_candidates_block call: rows [k*block_q, (k+1)*block_q)
    of a head attend over list k of idx (batch, q_heads, ceil(n_q / block_q), C)."""

    def __init__(self, cache: PackedCache, q: torch.Tensor, idx: torch.Tensor, block_q: int,
                 sm_scale: float = 0.0, out_dtype=None):
        self.lib = load_library()
        self.cache = cache
        self.q = q.contiguous()
        if self.q.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("q must be float32 or bfloat16")
        self.idx = idx.to(torch.int32).contiguous()
        b, hq, nq, d = self.q.shape
        if tuple(self.idx.shape[:3]) != (b, hq, -(-nq // block_q)):
            raise ValueError("idx must be (batch, q_heads, ceil(n_q / block_q), C)")
        self.block_q = block_q
        self.q_dt = F32 if self.q.dtype == torch.float32 else BF16
        self.out_dt = _dtype(out_dtype) if out_dtype is not None else self.q_dt
        self.out = torch.empty((b, hq, nq, d), dtype=TORCH_OF[self.out_dt], device=self.q.device)
        self.hq, self.nq, self.sm_scale = hq, nq, float(sm_scale or 0.0)
        self.status = new_status(self.q.device)
        need = ctypes.c_size_t(0)
        self._call(None, need)
        self.ws = torch.empty(max(int(need.value), 256), dtype=torch.uint8, device=self.q.device)
        self.ws_bytes = ctypes.c_size_t(self.ws.numel())
        self.path = None

    def _call(self, ws, ws_bytes):
        st = self.lib.kv_attend_candidates_block(
            self.cache.ref, _ptr(self.q), self.q_dt, self.hq, self.nq, _ptr(self.idx),
            self.idx.shape[3], self.block_q, self.sm_scale, _ptr(self.out), self.out_dt, ws,
            ctypes.byref(ws_bytes), _ptr(self.status), _stream())
        _check(st, "kv_attend_candidates_block")

    def run(self) -> torch.Tensor:
        self._call(_ptr(self.ws), self.ws_bytes)
        self.path = self.lib.kvq_last_path().decode()
        return self.out


class AttendRegionDrop:
    """A prepared kv_attend_region_drop call: attention over the keys of the
    regions not listed in ``drop`` (region r = [bounds[r], bounds[r + 1]))."""

    def __init__(self, cache: PackedCache, q: torch.Tensor, region_bounds, drop,
                 sm_scale: float = 0.0, out_dtype=None):
        self.lib = load_library()
        self.cache = cache
        self.q = q.contiguous()
        if self.q.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("q must be float32 or bfloat16")
        rb = [int(x) for x in region_bounds]
        self.n_regions = len(rb) - 1
        self.bounds = (ctypes.c_int32 * len(rb))(*rb)
        self.mask = 0
        for r in drop:
            self.mask |= 1 << int(r)
        b, hq, nq, d = self.q.shape
        self.q_dt = F32 if self.q.dtype == torch.float32 else BF16
        self.out_dt = _dtype(out_dtype) if out_dtype is not None else self.q_dt
        self.out = torch.empty((b, hq, nq, d), dtype=TORCH_OF[self.out_dt], device=self.q.device)
        self.hq, self.nq, self.sm_scale = hq, nq, float(sm_scale or 0.0)
        self.status = new_status(self.q.device)
        need = ctypes.c_size_t(0)
        self._call(None, need)
        self.ws = torch.empty(max(int(need.value), 256), dtype=torch.uint8, device=self.q.device)
        self.ws_bytes = ctypes.c_size_t(self.ws.numel())

    def _call(self, ws, ws_bytes):
        st = self.lib.kv_attend_region_drop(
            self.cache.ref, _ptr(self.q), self.q_dt, self.hq, self.nq, self.sm_scale, self.bounds,
            self.n_regions, self.mask, _ptr(self.out), self.out_dt, ws, ctypes.byref(ws_bytes),
            _ptr(self.status), _stream())
        _check(st, "kv_attend_region_drop")

    def run(self) -> torch.Tensor:
        self._call(_ptr(self.ws), self.ws_bytes)
        return self.out


# ------------------------------------------------------------------ rotary positions
TREE_MAX = 256   # KVQ_TREE_MAX
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
# scaling kinds and the keyword arguments that fill (original, p0, p1)
ROPE_SCALINGS = {"none": (0, ()), "linear": (1, ()), "base": (2, ()),
                 "ramp": (3, ("original", "fast", "slow")),
                 "bands": (4, ("original", "low", "high"))}


class RopePlan:
    """Frequency table of kv_rope on the device (kvq_rope_turns): made once per
    model. ``scaling``: none, linear, base (``factor``), ramp (``factor``,
    ``original``, ``fast``, ``slow``) or bands (``factor``, ``original``,
    ``low``, ``high``); see include/kvq.h."""

    def __init__(self, rotary_dim: int, base: float = 10000.0, layout: str = "half",
                 scaling: str = "none", factor: float = 1.0, device="cuda", **params):
        if layout not in ROPE_LAYOUTS or scaling not in ROPE_SCALINGS:
            raise ValueError("unknown layout or scaling")
        kind, names = ROPE_SCALINGS[scaling]
        if set(params) != set(names):
            raise TypeError(f"scaling {scaling!r} takes {('factor',) + names if kind else ()}")
        sc = KvqRopeScaling(kind, float(factor), *([float(params[n]) for n in names] or [0.0] * 3))
        self.rotary_dim, self.layout = int(rotary_dim), ROPE_LAYOUTS[layout]
        host = (ctypes.c_uint64 * max(1, self.rotary_dim // 2))()
        amp = ctypes.c_float(0.0)
        _check(load_library().kvq_rope_turns(self.rotary_dim, float(base), ctypes.byref(sc), host,
                                             ctypes.byref(amp)), "kvq_rope_turns")
        self.amplitude = float(amp.value)
        self.turns_host = list(host)
        signed = [x - (1 << 64) if x >> 63 else x for x in self.turns_host]
        self.turns = torch.tensor(signed, dtype=torch.int64, device=device)


def _integers(x: torch.Tensor, what: str):
    """Refuse a tensor whose conversion to int32 would cut fractions off."""
    if x.is_floating_point() or x.is_complex() or x.dtype == torch.bool:
        raise TypeError(f"{what} must be whole numbers (int32, or a type that converts to it)")


def _static(copies: list, x: torch.Tensor, dtype=None) -> torch.Tensor:
    """x itself when a prepared call can read it in place, else a dense buffer
    (of ``dtype``) that every run() fills from x again. The calls record no
    gradients, nor do these copies."""
    x = x.detach()
    y = x.to(dtype or x.dtype).contiguous()
    if y.data_ptr() % 16:
        y = y.clone()
    if y is not x:
        copies.append((y, x))
    return y


def _refresh(copies: list):
    for buf, src in copies:
        buf.copy_(src)


def _rope_view(copies: list, x: torch.Tensor) -> torch.Tensor:
    """x if kv_rope can read it in place (unit feature stride, 16-byte rows), else as _static."""
    unit = 16 // x.element_size()
    ok = (x.stride(3) == 1 and x.data_ptr() % 16 == 0 and
          all(s >= 0 and (s % unit == 0 or n == 1) for s, n in zip(x.stride()[:3], x.shape[:3])))
    return x if ok else _static(copies, x)


class Rope(_Prepared):
    """A prepared kv_rope call: q (batch, heads, n, D) and optionally k of the
    same batch, n and D, at any strides (views of a projection's rows are read
    in place when their rows start on 16 bytes); ``v`` is only copied to the
    dense layout. ``positions`` (batch, n): int32 ones are read in place, other
    integers converted by every run. ``run()`` returns the outputs, dense (batch,
    heads, n, D)."""

    def __init__(self, plan: RopePlan, q: torch.Tensor, k: torch.Tensor | None,
                 positions: torch.Tensor, v: torch.Tensor | None = None, inverse: bool = False,
                 out=None):
        self.lib = load_library()
        self.plan, self.inverse = plan, int(bool(inverse))
        _integers(positions, "positions")
        src = [x for x in (q, k, v) if x is not None]
        self.device = _one_device(plan.turns, positions, *src, *(out or ()))
        if any(x.dim() != 4 or x.dtype != q.dtype for x in src):
            raise TypeError("q, k and v must be (batch, heads, n, D) of one type")
        if q.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("q, k and v must be float32 or bfloat16")
        b, _, n, d = q.shape
        if any((x.shape[0], x.shape[2], x.shape[3]) != (b, n, d) for x in src):
            raise ValueError("q, k and v must have the same batch, tokens and head dim")
        if tuple(positions.shape) != (b, n):
            raise ValueError("positions must be (batch, n)")
        if plan.rotary_dim > d:
            raise ValueError("rotary_dim is larger than the head dim")
        self._copies = []
        self.src = [_rope_view(self._copies, x) for x in src]
        self.positions = _static(self._copies, positions, torch.int32)
        if out is None:
            out = [torch.empty(x.shape, dtype=x.dtype, device=x.device) for x in src]
        if len(out) != len(src) or any(o.shape != x.shape or o.dtype != x.dtype or
                                       not o.is_contiguous() for o, x in zip(out, src)):
            raise ValueError("out must hold one dense tensor per input")
        self.out = list(out)
        self.dt = F32 if q.dtype == torch.float32 else BF16
        self.b, self.n, self.d = b, n, d
        arr = (KvqRopeTensor * len(src))()
        for i, (x, o) in enumerate(zip(self.src, self.out)):
            st = [s if m > 1 else 0 for s, m in zip(x.stride()[:3], x.shape[:3])]
            arr[i] = KvqRopeTensor(_ptr(x), _ptr(o), x.shape[1],
                                   0 if v is not None and i == len(src) - 1 else 1,
                                   st[0], st[1], st[2])
        self.arr = arr
        self._args = (arr, len(src), self.dt, b, n, d, plan.rotary_dim, plan.layout,
                      _ptr(plan.turns), plan.amplitude, self.inverse, _ptr(self.positions), None)

    def _run(self):
        if self._copies:
            _refresh(self._copies)
        _check(self.lib.kv_rope(*self._args, self._raw_stream()), "kv_rope")
        return self.out


def rope(plan: RopePlan, q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor,
         v: torch.Tensor | None = None, inverse: bool = False):
    """kv_rope; returns the outputs (q, and k, v if given). ``inverse`` turns by
    the negated angle: the gradient of the call."""
    return Rope(plan, q, k, positions, v, inverse).run()


# ------------------------------------------------------------------ drafted tokens
class AttendTree(_Prepared):
    """A prepared kv_attend_tree call (see Attend): q (batch, q_heads, T, D),
    k_tree, v_tree (batch, kv_heads, T, D) of the drafted tokens, parents
    (batch, T): the drafted token a token follows, -1 for the cache's last
    token, -2 for no token (its output row stays as it was)."""

    def __init__(self, cache: PackedCache, q: torch.Tensor, k_tree: torch.Tensor,
                 v_tree: torch.Tensor, parents: torch.Tensor, sm_scale: float = 0.0,
                 out_dtype=None, out=None):
        self.lib = load_library()
        self.cache = cache
        _integers(parents, "parents")
        self.device = _one_device(cache.k_scales, q, k_tree, v_tree, parents, out)
        self._copies = []
        self.q, self.k, self.v = (_static(self._copies, x) for x in (q, k_tree, v_tree))
        if self.q.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("q must be float32 or bfloat16")
        if self.k.dtype not in (torch.float32, torch.bfloat16) or self.v.dtype != self.k.dtype:
            raise TypeError("k_tree and v_tree must both be float32 or bfloat16")
        b, hq, t, d = self.q.shape
        if b != cache.batch or d != cache.head_dim:
            raise ValueError("q does not match the cache")
        if tuple(self.k.shape) != (b, cache.kv_heads, t, d) or self.v.shape != self.k.shape:
            raise ValueError("k_tree and v_tree must be (batch, kv_heads, T, D)")
        if tuple(parents.shape) != (b, t):
            raise ValueError("parents must be (batch, T)")
        self.parents = _static(self._copies, parents, torch.int32)
        self.q_dt = F32 if self.q.dtype == torch.float32 else BF16
        self.t_dt = F32 if self.k.dtype == torch.float32 else BF16
        self.out_dt = (_dtype(out_dtype) if out_dtype is not None else
                       self.q_dt if out is None else
                       F32 if out.dtype == torch.float32 else BF16)
        # rows without a token are never written: zeros unless the caller gives the buffer
        self.out = out if out is not None else torch.zeros(
            (b, hq, t, d), dtype=TORCH_OF[self.out_dt], device=self.q.device)
        if (self.out.shape != self.q.shape or self.out.dtype != TORCH_OF[self.out_dt] or
                not self.out.is_contiguous()):
            raise ValueError("out must be a dense tensor of q's shape")
        self.hq, self.t, self.sm_scale = hq, t, float(sm_scale or 0.0)
        self.status = new_status(self.q.device)
        self.ws, self._kept = None, []
        self._reserve()

    def _reserve(self):
        """Workspace for the cache's present length (it grows with appends)."""
        args = (self.cache.ref, _ptr(self.q), self.q_dt, self.hq, self.t, _ptr(self.k),
                _ptr(self.v), self.t_dt, _ptr(self.parents), self.sm_scale, _ptr(self.out),
                self.out_dt)
        need = ctypes.c_size_t(0)
        with torch.cuda.device(self.device):
            _check(self.lib.kv_attend_tree(*args, None, ctypes.byref(need), None, None),
                   "kv_attend_tree")
        self._n = self.cache.n_tokens
        self._workspace(int(need.value))
        self._args = (*args, _ptr(self.ws), ctypes.byref(self.ws_bytes), _ptr(self.status))
        self.path = None

    def _run(self) -> torch.Tensor:
        if self.cache.n_tokens != self._n:
            self._reserve()
        if self._copies:
            _refresh(self._copies)
        _check(self.lib.kv_attend_tree(*self._args, self._raw_stream()), "kv_attend_tree")
        if self.path is None:
            self.path = self.lib.kvq_last_path().decode()
        return self.out


def attend_tree(cache: PackedCache, q: torch.Tensor, k_tree: torch.Tensor, v_tree: torch.Tensor,
                parents: torch.Tensor, sm_scale: float = 0.0, out_dtype=None):
    """kv_attend_tree; returns (out, status tensor)."""
    a = AttendTree(cache, q, k_tree, v_tree, parents, sm_scale, out_dtype)
    a.run()
    return a.out, a.status


# ------------------------------------------------------------------ block-sparse attention
class BlockSummary(_Prepared):
    """int8 mean keys of the blocks of ``block`` tokens of a cache's int4 part
    (kv_block_summary), with room for the blocks the cache can grow to."""

    def __init__(self, cache: PackedCache, block: int = 64):
        if block not in (32, 64, 128):
            raise ValueError("block must be 32, 64 or 128")
        self.lib = load_library()
        self.cache, self.block = cache, block
        groups = cache.reserve[0] or cache.gk
        self.cap_blocks = -(-groups * 32 // block)
        self.device = dev = _one_device(cache.k_scales)
        b, h, d = cache.batch, cache.kv_heads, cache.head_dim
        self.codes = torch.empty((b, h, self.cap_blocks, d), dtype=torch.int8, device=dev)
        self.scales = torch.empty((b, h, self.cap_blocks), dtype=torch.float32, device=dev)
        self.struct = KvqSummary(_ptr(self.codes), _ptr(self.scales), block, self.cap_blocks)
        self.ref = ctypes.byref(self.struct)

    # blocks [_from, ...) hold summaries of an int4 part of _cut tokens
    _from = _cut = 0

    @property
    def blocks(self) -> int:
        return -(-self.cache.cut // self.block)

    def update(self, first: int = 0) -> "BlockSummary":
        """Recompute the blocks from ``first`` on (all of them by default)."""
        self.run("update", first)
        self.filled(first)
        return self

    def filled(self, first: int = 0):
        """Take it that the blocks from ``first`` on hold the cache's summaries: for entries
        that came another way than by ``update`` (loaded, or kv_block_summary itself)."""
        if self.covers(first) or first >= self.blocks:
            return
        cut = self.cache.cut
        # what was there before still holds: all of it, or the blocks that were whole then
        end = self.blocks if cut == self._cut else min(cut, self._cut) // self.block
        if not self._from <= first <= end:
            self._from = first
        self._cut = cut

    def covers(self, first: int = 0) -> bool:
        """Whether the blocks from ``first`` on hold summaries of the int4 part as long as it is
        now. (A cache packed anew in place, at the same length, is not noticed.)"""
        return self._from <= first and self._cut == self.cache.cut

    def values(self, first: int = 0) -> torch.Tensor:
        """The mean keys the codes stand for, fp32 (batch, kv_heads, blocks - first, D)."""
        if not self.covers(first) and 0 <= first < self.blocks:
            raise ValueError("the summary does not cover the cache: update() it")
        return self.run("values", first)

    def _run(self, what: str, first: int):
        c = self.cache
        if what == "update":
            _check(self.lib.kv_block_summary(c.ref, self.ref, first, None, self._raw_stream()),
                   "kv_block_summary")
            return None
        out = torch.empty((c.batch, c.kv_heads, max(0, self.blocks - first), c.head_dim),
                          dtype=torch.float32, device=self.device)
        # (the address as an int: about 1 us a call cheaper than a ctypes pointer)
        _check(self.lib.kv_block_values(c.ref, self.ref, first, out.data_ptr() or None, None,
                                        self._raw_stream()), "kv_block_values")
        return out


class AttendBlocks(_Prepared):
    """A prepared pair of calls, kv_select_blocks and kv_attend_blocks: each
    query token of a KV head attends the ``top_k`` blocks its summary scores
    highest and the whole window. The summary is the caller's to keep up with the
    cache (``BlockSummary.update`` after appends that moved groups into the int4
    part; a run that would read blocks without a summary raises ValueError).
    ``selected`` (batch, kv_heads, n_q, top_k) holds the chosen blocks after
    ``run()``; ``select=False`` attends the lists already there (``selected`` may
    be passed)."""

    def __init__(self, cache: PackedCache, q: torch.Tensor, summary: BlockSummary | None,
                 top_k: int, n_sink: int = 0, sm_scale: float = 0.0, out_dtype=None, out=None,
                 selected: torch.Tensor | None = None, block: int | None = None):
        self.lib = load_library()
        self.cache, self.summary = cache, summary
        self.device = _one_device(cache.k_scales, q, out, selected)
        self._copies = []
        self.q = _static(self._copies, q)
        if self.q.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("q must be float32 or bfloat16")
        b, hq, nq, d = self.q.shape
        if b != cache.batch or d != cache.head_dim:
            raise ValueError("q does not match the cache")
        if summary is not None and summary.cache is not cache:
            raise ValueError("the summary is another cache's")
        if summary is None and (selected is None or block is None):
            raise ValueError("without a summary, selected and block are needed")
        self.block = summary.block if summary is not None else int(block)
        self.top_k, self.n_sink = int(top_k), int(n_sink)
        shape = (b, cache.kv_heads, nq, self.top_k)
        if selected is None:
            selected = torch.full(shape, -1, dtype=torch.int32, device=self.q.device)
        if (tuple(selected.shape) != shape or selected.dtype != torch.int32 or
                not selected.is_contiguous()):
            raise ValueError("selected must be int32 (batch, kv_heads, n_q, top_k), dense")
        self.selected = selected
        self.q_dt = F32 if self.q.dtype == torch.float32 else BF16
        self.out_dt = (_dtype(out_dtype) if out_dtype is not None else
                       self.q_dt if out is None else
                       F32 if out.dtype == torch.float32 else BF16)
        self.out = out if out is not None else torch.empty(
            (b, hq, nq, d), dtype=TORCH_OF[self.out_dt], device=self.q.device)
        if (self.out.shape != self.q.shape or self.out.dtype != TORCH_OF[self.out_dt] or
                not self.out.is_contiguous()):
            raise ValueError("out must be a dense tensor of q's shape")
        self.hq, self.nq, self.sm_scale = hq, nq, float(sm_scale or 0.0)
        self.status = new_status(self.q.device)
        self.ws, self._kept = None, []
        self._reserve()

    def _reserve(self):
        """Workspace for the cache's present length (it grows with appends)."""
        select = None
        need = ctypes.c_size_t(0)
        attend = (self.cache.ref, _ptr(self.q), self.q_dt, self.hq, self.nq, _ptr(self.selected),
                  self.top_k, self.block, self.sm_scale, _ptr(self.out), self.out_dt)
        with torch.cuda.device(self.device):
            _check(self.lib.kv_attend_blocks(*attend, None, ctypes.byref(need), None, None),
                   "kv_attend_blocks")
            most = int(need.value)
            if self.summary is not None:
                select = (self.cache.ref, self.summary.ref, _ptr(self.q), self.q_dt, self.hq,
                          self.nq, self.top_k, self.n_sink, _ptr(self.selected))
                _check(self.lib.kv_select_blocks(*select, None, ctypes.byref(need), None, None),
                       "kv_select_blocks")
                most = max(most, int(need.value))
        self._n = self.cache.n_tokens
        # the calls run one after the other and may share their workspace
        self._workspace(most)
        tail = (_ptr(self.ws), ctypes.byref(self.ws_bytes), _ptr(self.status))
        self._attend_args = (*attend, *tail)
        self._select_args = (*select, *tail) if select else None
        self.path = None

    def _run(self, select: bool = True) -> torch.Tensor:
        if (select and self._select_args and not self.summary.covers() and
                self.summary.blocks > self.top_k):  # (else every block is taken unread)
            raise ValueError("the summary does not cover the cache: update() it")
        if self.cache.n_tokens != self._n:
            self._reserve()
        if self._copies:
            _refresh(self._copies)
        stream = self._raw_stream()
        if select and self._select_args:
            _check(self.lib.kv_select_blocks(*self._select_args, stream), "kv_select_blocks")
        _check(self.lib.kv_attend_blocks(*self._attend_args, stream), "kv_attend_blocks")
        if self.path is None:
            self.path = self.lib.kvq_last_path().decode()
        return self.out


def attend_blocks(cache: PackedCache, q: torch.Tensor, summary: BlockSummary, top_k: int,
                  n_sink: int = 0, sm_scale: float = 0.0, out_dtype=None):
    """kv_select_blocks and kv_attend_blocks; returns (out, selected, status tensor)."""
    a = AttendBlocks(cache, q, summary, top_k, n_sink, sm_scale, out_dtype)
    a.run()
    return a.out, a.selected, a.status
