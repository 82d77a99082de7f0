"""Python binding of libredmoe.so (C ABI: include/redmoe.h).

Argument marshalling only: every step of the layer runs in the library's CUDA kernels.
torch provides device memory and streams. The binding never computes a result itself
and has no fallback: if the library is missing it raises.

Names match the C entry points (redmoe_forward, redmoe_router, redmoe_route_build,
redmoe_forward_stack, redmoe_forward_noalloc, redmoe_workspace_bytes,
redmoe_workspace_init, redmoe_check_timeout, redmoe_selftest_wait_limit,
redmoe_fill_shared_memory, redmoe_forward_cached, redmoe_expert_cache_slot_bytes,
redmoe_expert_cache_init, redmoe_forward_host_experts, redmoe_expert_cache_prefetch,
redmoe_norm_forward, redmoe_norm_backward, redmoe_norm_workspace_bytes, redmoe_forward_block,
redmoe_workspace_bytes_block, redmoe_balance_forward, redmoe_balance_backward,
redmoe_balance_workspace_bytes, redmoe_gemv, redmoe_status_string, redmoe_abi_version).

The calls around the layer (norms, block, balance, gemv) check their tensors' types, shapes,
contiguity and device (ValueError) and run on the tensors' device, by default on that device's
current stream.
"""

from __future__ import annotations

import ctypes as C
import os
import threading
from typing import Dict, Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libredmoe.so")
ABI_VERSION = 1
DTYPES = {"f32": 0, "bf16": 1, "int4g32": 2, "int2g32": 3}
STATUS = {0: "REDMOE_OK", 1: "REDMOE_ERR_INVALID_ARG", 2: "REDMOE_ERR_UNSUPPORTED", 3: "REDMOE_ERR_WORKSPACE",
          4: "REDMOE_ERR_CUDA", 5: "REDMOE_ERR_TIMEOUT"}
# entry points declared in include/redmoe.h
SYMBOLS = ("redmoe_abi_version", "redmoe_status_string", "redmoe_workspace_bytes", "redmoe_workspace_init",
           "redmoe_forward", "redmoe_router", "redmoe_route_build", "redmoe_forward_stack",
           "redmoe_check_timeout", "redmoe_forward_noalloc", "redmoe_selftest_wait_limit",
           "redmoe_fill_shared_memory", "redmoe_forward_cached", "redmoe_expert_cache_slot_bytes",
           "redmoe_expert_cache_init", "redmoe_forward_host_experts", "redmoe_expert_cache_prefetch",
           "redmoe_workspace_bytes_host", "redmoe_forward_host", "redmoe_forward_stack_host",
           "redmoe_norm_forward", "redmoe_norm_workspace_bytes", "redmoe_norm_backward",
           "redmoe_workspace_bytes_block", "redmoe_forward_block", "redmoe_balance_workspace_bytes",
           "redmoe_balance_forward", "redmoe_balance_backward", "redmoe_gemv")

_lock = threading.Lock()
_lib = None


class RedmoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {STATUS.get(self.status, self.status)} ({redmoe_status_string(self.status)})")


class _Layer(C.Structure):
    _fields_ = [
        ("hidden", C.c_int32), ("n_experts", C.c_int32), ("top_k", C.c_int32), ("inter", C.c_int32),
        ("shared_inter", C.c_int32), ("x_dtype", C.c_int32), ("router_dtype", C.c_int32),
        ("expert_dtype", C.c_int32),
        ("router_w", C.c_void_p), ("router_bias", C.c_void_p), ("shared_gate_w", C.c_void_p),
        ("w_gate", C.c_void_p), ("w_up", C.c_void_p), ("w_down", C.c_void_p),
        ("s_gate", C.c_void_p), ("s_up", C.c_void_p), ("s_down", C.c_void_p),
        ("sh_gate", C.c_void_p), ("sh_up", C.c_void_p), ("sh_down", C.c_void_p),
        ("sh_s_gate", C.c_void_p), ("sh_s_up", C.c_void_p), ("sh_s_down", C.c_void_p),
    ]


class _ExpertCache(C.Structure):
    _fields_ = [("n_slots", C.c_int32), ("slot_gate", C.c_void_p), ("slot_up", C.c_void_p), ("slot_down", C.c_void_p),
                ("slot_s_gate", C.c_void_p), ("slot_s_up", C.c_void_p), ("slot_s_down", C.c_void_p),
                ("slot_of", C.c_void_p), ("expert_in", C.c_void_p), ("hot", C.c_void_p), ("stats", C.c_void_p),
                ("fill", C.c_void_p)]


class _Norm(C.Structure):
    _fields_ = [("hidden", C.c_int32), ("h_dtype", C.c_int32), ("y_dtype", C.c_int32), ("x_dtype", C.c_int32),
                ("w_dtype", C.c_int32), ("post_norm", C.c_int32), ("gate_kind", C.c_int32), ("gate_act", C.c_int32),
                ("gate_dtype", C.c_int32), ("eps", C.c_float), ("w_offset", C.c_float), ("res_scale", C.c_float),
                ("block_scale", C.c_float), ("post_w", C.c_void_p), ("pre_w", C.c_void_p)]


class _Matrix(C.Structure):
    _fields_ = [("rows", C.c_int32), ("cols", C.c_int32), ("dtype", C.c_int32), ("w", C.c_void_p), ("s", C.c_void_p)]


class _RouteDebug(C.Structure):
    _fields_ = [("counts", C.c_void_p), ("offsets", C.c_void_p), ("perm", C.c_void_p)]


def load():
    """Load libredmoe.so (built in-tree). Raises if it has not been built."""
    global _lib
    if _lib is not None:  # set once, complete
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m sparse_moe_gemv_b200.build`")
        lib = C.CDLL(LIB_PATH)
        P, i32, sz = C.c_void_p, C.c_int32, C.c_size_t
        lib.redmoe_abi_version.restype = i32
        lib.redmoe_abi_version.argtypes = []
        lib.redmoe_status_string.restype = C.c_char_p
        lib.redmoe_status_string.argtypes = [i32]
        lib.redmoe_workspace_bytes.restype = sz
        lib.redmoe_workspace_bytes.argtypes = [P, i32]
        lib.redmoe_workspace_init.restype = i32
        lib.redmoe_workspace_init.argtypes = [P, sz, P]
        lib.redmoe_forward.restype = i32
        lib.redmoe_forward.argtypes = [P, P, i32, P, P, P, P, sz, P, P]
        lib.redmoe_router.restype = i32
        lib.redmoe_router.argtypes = [P, P, i32, P, P, P, P, P, sz, P]
        lib.redmoe_route_build.restype = i32
        lib.redmoe_route_build.argtypes = [P, i32, i32, i32, P, P, P, P, sz, P]
        lib.redmoe_forward_stack.restype = i32
        lib.redmoe_forward_stack.argtypes = [P, i32, P, i32, P, P, P, P, sz, P]
        lib.redmoe_check_timeout.restype = i32
        lib.redmoe_check_timeout.argtypes = [P, P]
        lib.redmoe_forward_noalloc.restype = i32
        lib.redmoe_forward_noalloc.argtypes = [P, P, i32, P, P, P, P]
        lib.redmoe_selftest_wait_limit.restype = i32
        lib.redmoe_selftest_wait_limit.argtypes = [P, sz, i32, C.c_uint64, P]
        lib.redmoe_forward_cached.restype = i32
        lib.redmoe_forward_cached.argtypes = [P, P, i32, P, P, P, P, C.c_float, P, sz, P]
        lib.redmoe_expert_cache_slot_bytes.restype = sz
        lib.redmoe_expert_cache_slot_bytes.argtypes = [P]
        lib.redmoe_expert_cache_init.restype = i32
        lib.redmoe_expert_cache_init.argtypes = [P, P, P]
        lib.redmoe_forward_host_experts.restype = i32
        lib.redmoe_forward_host_experts.argtypes = [P, P, i32, P, P, P, P, P, sz, P]
        lib.redmoe_expert_cache_prefetch.restype = i32
        lib.redmoe_expert_cache_prefetch.argtypes = [P, P, P, i32, P, sz, P]
        lib.redmoe_fill_shared_memory.restype = i32
        lib.redmoe_fill_shared_memory.argtypes = [C.c_uint32, P]
        lib.redmoe_workspace_bytes_host.restype = sz
        lib.redmoe_workspace_bytes_host.argtypes = [P, i32]
        lib.redmoe_forward_host.restype = i32
        lib.redmoe_forward_host.argtypes = [P, P, i32, P, P, P, P, sz, P]
        lib.redmoe_forward_stack_host.restype = i32
        lib.redmoe_forward_stack_host.argtypes = [P, i32, P, i32, P, P, P, P, sz, P]
        lib.redmoe_norm_forward.restype = i32
        lib.redmoe_norm_forward.argtypes = [P, P, P, P, i32, P, P, P]
        lib.redmoe_norm_workspace_bytes.restype = sz
        lib.redmoe_norm_workspace_bytes.argtypes = [P, i32]
        lib.redmoe_norm_backward.restype = i32
        lib.redmoe_norm_backward.argtypes = [P, P, P, P, P, P, i32, P, P, P, P, P, P, sz, P]
        lib.redmoe_workspace_bytes_block.restype = sz
        lib.redmoe_workspace_bytes_block.argtypes = [P, i32]
        lib.redmoe_forward_block.restype = i32
        lib.redmoe_forward_block.argtypes = [P, P, P, P, P, i32, P, P, P, P, P, sz, P]
        lib.redmoe_balance_workspace_bytes.restype = sz
        lib.redmoe_balance_workspace_bytes.argtypes = [i32, i32]
        lib.redmoe_balance_forward.restype = i32
        lib.redmoe_balance_forward.argtypes = [P, i32, P, P, i32, i32, i32, P, P, P, P, P, sz, P]
        lib.redmoe_balance_backward.restype = i32
        lib.redmoe_balance_backward.argtypes = [P, i32, P, i32, i32, i32, P, P, P, P, P]
        lib.redmoe_gemv.restype = i32
        lib.redmoe_gemv.argtypes = [P, P, i32, i32, P, i32, P]
        if lib.redmoe_abi_version() != ABI_VERSION:
            raise RuntimeError("libredmoe.so ABI version mismatch")
        _lib = lib
        return lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# The handles behind torch.cuda.current_stream() and current_device(), without the Python objects
# around them: measured 0.07 us a call against 3.2 us for the stream object. A torch without CUDA has
# neither; there the public calls say so when they are made.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _raw_stream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(status: int, where: str):
    if status != 0:
        raise RedmoeError(status, where)


class Layer:
    """A layer's device tensors plus its C descriptor.

    `tensors` uses the names of the C struct (router_w, router_bias, shared_gate_w,
    w_gate, w_up, w_down, s_gate, s_up, s_down, sh_gate, sh_up, sh_down, sh_s_gate,
    sh_s_up, sh_s_down); the tensors are kept alive by this object.
    """

    def __init__(self, tensors: Dict[str, Optional[torch.Tensor]], hidden: int, n_experts: int, top_k: int,
                 inter: int, shared_inter: int, x_dtype: str = "bf16", router_dtype: str = "bf16",
                 expert_dtype: str = "bf16"):
        self.tensors = dict(tensors)
        s = _Layer()
        s.hidden, s.n_experts, s.top_k, s.inter, s.shared_inter = hidden, n_experts, top_k, inter, shared_inter
        s.x_dtype, s.router_dtype, s.expert_dtype = DTYPES[x_dtype], DTYPES[router_dtype], DTYPES[expert_dtype]
        for name, _ in _Layer._fields_[8:]:
            setattr(s, name, _ptr(self.tensors.get(name)))
        self.struct = s
        self.hidden, self.n_experts, self.top_k = hidden, n_experts, top_k
        self.inter, self.shared_inter = inter, shared_inter
        self.x_dtype, self.router_dtype, self.expert_dtype = x_dtype, router_dtype, expert_dtype

    @classmethod
    def from_shape(cls, tensors, shape):
        """`shape` has attributes H, E, k, I, Is, x_dtype, router_dtype, expert_dtype."""
        return cls(tensors, shape.H, shape.E, shape.k, shape.I, shape.Is, shape.x_dtype, shape.router_dtype,
                   shape.expert_dtype)

    @property
    def ref(self):
        return C.byref(self.struct)


def redmoe_abi_version() -> int:
    return int(load().redmoe_abi_version())


def redmoe_status_string(status: int) -> str:
    return load().redmoe_status_string(int(status)).decode()


def redmoe_workspace_bytes(layer: Layer, T: int) -> int:
    return int(load().redmoe_workspace_bytes(layer.ref, int(T)))


def redmoe_workspace_init(workspace: Optional[torch.Tensor], stream=None) -> None:
    """Zero a workspace's control block; None: the allocation-free scratch of this device."""
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().redmoe_workspace_init(_ptr(workspace), nbytes, _stream(stream)), "redmoe_workspace_init")


def new_workspace(layer: Layer, T: int, device=None) -> torch.Tensor:
    """A zeroed workspace tensor of redmoe_workspace_bytes(layer, T) bytes."""
    n = redmoe_workspace_bytes(layer, T)
    if n == 0:
        raise ValueError("invalid layer or token count")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def redmoe_forward(layer: Layer, x: torch.Tensor, out: torch.Tensor, topk_ids: torch.Tensor, topk_w: torch.Tensor,
                   workspace: torch.Tensor, dbg: Optional[Sequence[torch.Tensor]] = None, stream=None,
                   T: Optional[int] = None) -> None:
    """out[T,H] fp32, topk_ids[T,k] int32, topk_w[T,k] fp32 <- layer(x[T,H])."""
    lib = load()
    dbg_s = None
    if dbg is not None:
        dbg_s = _RouteDebug(_ptr(dbg[0]), _ptr(dbg[1]), _ptr(dbg[2]))
    T = x.shape[0] if T is None else T
    st = lib.redmoe_forward(layer.ref, _ptr(x), int(T), _ptr(out), _ptr(topk_ids), _ptr(topk_w),
                            _ptr(workspace), workspace.numel() * workspace.element_size(),
                            None if dbg_s is None else C.byref(dbg_s), _stream(stream))
    _check(st, "redmoe_forward")


def redmoe_workspace_bytes_host(layer: Layer, T: int) -> int:
    return int(load().redmoe_workspace_bytes_host(layer.ref, int(T)))


def new_workspace_host(layer: Layer, T: int, device=None) -> torch.Tensor:
    """A zeroed workspace tensor of redmoe_workspace_bytes_host(layer, T) bytes."""
    n = redmoe_workspace_bytes_host(layer, T)
    if n == 0:
        raise ValueError("invalid layer or token count")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def redmoe_forward_host(layer: Layer, x_host: torch.Tensor, out_host: torch.Tensor, ids_host: torch.Tensor,
                        w_host: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    """redmoe_forward with x and the results in host memory (pinned for asynchronous
    copies, and for results stored straight from the kernel at T <= 4). The results are
    valid once `stream` has been synchronised."""
    T = x_host.shape[0]
    st = load().redmoe_forward_host(layer.ref, _ptr(x_host), int(T), _ptr(out_host), _ptr(ids_host), _ptr(w_host),
                                    _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "redmoe_forward_host")


def redmoe_forward_cached(layer: Layer, x: torch.Tensor, out: torch.Tensor, topk_ids: torch.Tensor,
                          topk_w: torch.Tensor, cached: torch.Tensor, lam: float, workspace: torch.Tensor,
                          stream=None) -> None:
    """redmoe_forward with the opt-in cache-aware routing bias: cached [E] uint8 device mask
    of experts resident in the caller's cache, lam >= 0 (0: plain routing)."""
    T = x.shape[0]
    st = load().redmoe_forward_cached(layer.ref, _ptr(x), int(T), _ptr(out), _ptr(topk_ids), _ptr(topk_w),
                                      _ptr(cached), float(lam), _ptr(workspace),
                                      workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "redmoe_forward_cached")


def redmoe_router(layer: Layer, x: torch.Tensor, topk_ids: torch.Tensor, topk_w: torch.Tensor,
                  shared_gate: torch.Tensor, workspace: torch.Tensor, logits: Optional[torch.Tensor] = None,
                  stream=None) -> None:
    st = load().redmoe_router(layer.ref, _ptr(x), int(x.shape[0]), _ptr(topk_ids), _ptr(topk_w), _ptr(shared_gate),
                              _ptr(logits), _ptr(workspace), workspace.numel() * workspace.element_size(),
                              _stream(stream))
    _check(st, "redmoe_router")


def redmoe_route_build(topk_ids: torch.Tensor, n_experts: int, counts: torch.Tensor, offsets: torch.Tensor,
                       perm: torch.Tensor, stream=None) -> None:
    T, k = topk_ids.shape
    st = load().redmoe_route_build(_ptr(topk_ids), int(T), int(k), int(n_experts), _ptr(counts), _ptr(offsets),
                                   _ptr(perm), None, 0, _stream(stream))
    _check(st, "redmoe_route_build")


def redmoe_forward_stack(layers: Sequence[Layer], xs: Sequence[torch.Tensor], outs: Sequence[torch.Tensor],
                         ids: Sequence[torch.Tensor], ws: Sequence[torch.Tensor], workspace: torch.Tensor,
                         stream=None) -> None:
    n = len(layers)
    arr = (_Layer * n)(*[l.struct for l in layers])
    P = C.c_void_p * n
    T = xs[0].shape[0] if n else 0
    st = load().redmoe_forward_stack(C.cast(arr, C.c_void_p), n, C.cast(P(*[_ptr(t) for t in xs]), C.c_void_p),
                                     int(T), C.cast(P(*[_ptr(t) for t in outs]), C.c_void_p),
                                     C.cast(P(*[_ptr(t) for t in ids]), C.c_void_p),
                                     C.cast(P(*[_ptr(t) for t in ws]), C.c_void_p), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "redmoe_forward_stack")


def redmoe_forward_stack_host(layers: Sequence[Layer], xs: Sequence[torch.Tensor], outs: Sequence[torch.Tensor],
                              ids: Sequence[torch.Tensor], ws: Sequence[torch.Tensor], workspace: torch.Tensor,
                              stream=None) -> None:
    """redmoe_forward_stack with every x and result in host memory (pinned for the
    copy-free one-launch path); valid once `stream` has been synchronised."""
    n = len(layers)
    arr = (_Layer * n)(*[l.struct for l in layers])
    P = C.c_void_p * n
    T = xs[0].shape[0] if n else 0
    st = load().redmoe_forward_stack_host(C.cast(arr, C.c_void_p), n, C.cast(P(*[_ptr(t) for t in xs]), C.c_void_p),
                                          int(T), C.cast(P(*[_ptr(t) for t in outs]), C.c_void_p),
                                          C.cast(P(*[_ptr(t) for t in ids]), C.c_void_p),
                                          C.cast(P(*[_ptr(t) for t in ws]), C.c_void_p), _ptr(workspace),
                                          workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "redmoe_forward_stack_host")


def redmoe_check_timeout(workspace: Optional[torch.Tensor], stream=None) -> None:
    """Raise REDMOE_ERR_TIMEOUT if a bounded in-kernel wait gave up; None: the
    allocation-free scratch of this device."""
    _check(load().redmoe_check_timeout(_ptr(workspace), _stream(stream)), "redmoe_check_timeout")


def redmoe_forward_noalloc(layer: Layer, x: torch.Tensor, out: torch.Tensor, topk_ids: torch.Tensor,
                           topk_w: torch.Tensor, stream=None) -> None:
    """redmoe_forward for 1..4 token rows without a workspace argument.

    For callers that cannot allocate device memory (a strict stream capture, a loop that
    must not touch the allocator, a plug-in without a memory budget of its own): the
    scratch is a fixed 1 MiB array inside the library, shared by every call on the
    device. Calls must not overlap on the GPU; the first call on a device must not be
    made inside a stream capture (it looks up the array's address). A bounded wait that
    gave up is reported by redmoe_check_timeout(None) and cleared by
    redmoe_workspace_init(None).
    """
    st = load().redmoe_forward_noalloc(layer.ref, _ptr(x), int(x.shape[0]), _ptr(out), _ptr(topk_ids),
                                       _ptr(topk_w), _stream(stream))
    _check(st, "redmoe_forward_noalloc")


def redmoe_selftest_wait_limit(workspace: Optional[torch.Tensor], withhold: int, limit_ns: int, stream=None) -> None:
    """Run the bounded-wait self-test: block `withhold` skips a grid barrier, the others
    give up after limit_ns and record a timeout (read it with redmoe_check_timeout)."""
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().redmoe_selftest_wait_limit(_ptr(workspace), nbytes, int(withhold), int(limit_ns), _stream(stream)),
           "redmoe_selftest_wait_limit")


NAN_PATTERN = 0x7FC00000


def redmoe_fill_shared_memory(pattern: int = NAN_PATTERN, stream=None) -> None:
    """Fill every SM's shared memory with a 32-bit pattern before the next launch."""
    _check(load().redmoe_fill_shared_memory(int(pattern) & 0xFFFFFFFF, _stream(stream)), "redmoe_fill_shared_memory")


class ExpertCache:
    """A bounded device cache of routed experts (redmoe_expert_cache): n_slots slots in the
    layer's expert dtype plus the directory; device tensors owned by this object."""

    def __init__(self, layer: "Layer", n_slots: int, device=None):
        dev = device or "cuda"
        H, I, E = layer.hidden, layer.inter, layer.n_experts
        dt = layer.expert_dtype
        per = {"bf16": 2.0, "f32": 4.0, "int4g32": 0.5, "int2g32": 0.25}[dt]

        def stack(n, k):
            return torch.empty(n_slots, int(n * k * per), dtype=torch.uint8, device=dev)

        t = {"slot_gate": stack(I, H), "slot_up": stack(I, H), "slot_down": stack(H, I)}
        if dt in ("int4g32", "int2g32"):
            t.update(slot_s_gate=torch.empty(n_slots, I * H // 32, dtype=torch.bfloat16, device=dev),
                     slot_s_up=torch.empty(n_slots, I * H // 32, dtype=torch.bfloat16, device=dev),
                     slot_s_down=torch.empty(n_slots, H * I // 32, dtype=torch.bfloat16, device=dev))
        t.update(slot_of=torch.empty(E, dtype=torch.int32, device=dev),
                 expert_in=torch.empty(n_slots, dtype=torch.int32, device=dev),
                 hot=torch.empty(E, dtype=torch.float32, device=dev),
                 stats=torch.empty(4, dtype=torch.int32, device=dev),
                 fill=torch.empty(257, dtype=torch.int32, device=dev))
        self.tensors = t
        st = _ExpertCache()
        st.n_slots = n_slots
        for name, _ in _ExpertCache._fields_[1:]:
            setattr(st, name, _ptr(t.get(name)))
        self.struct = st
        self.n_slots = n_slots

    @property
    def ref(self):
        return C.byref(self.struct)


def redmoe_expert_cache_slot_bytes(layer: Layer) -> int:
    return int(load().redmoe_expert_cache_slot_bytes(layer.ref))


def redmoe_expert_cache_init(layer: Layer, cache: ExpertCache, stream=None) -> None:
    _check(load().redmoe_expert_cache_init(layer.ref, cache.ref, _stream(stream)), "redmoe_expert_cache_init")


def redmoe_forward_host_experts(layer: Layer, x: torch.Tensor, out: torch.Tensor, topk_ids: torch.Tensor,
                                topk_w: torch.Tensor, cache: ExpertCache, workspace: torch.Tensor, stream=None) -> None:
    """One token through a layer whose routed experts may be in pinned host memory."""
    st = load().redmoe_forward_host_experts(layer.ref, _ptr(x), int(x.shape[0]), _ptr(out), _ptr(topk_ids),
                                            _ptr(topk_w), cache.ref, _ptr(workspace),
                                            workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "redmoe_forward_host_experts")


def redmoe_expert_cache_prefetch(layer: Layer, cache: ExpertCache, ids: torch.Tensor, workspace: torch.Tensor,
                                 stream=None) -> None:
    st = load().redmoe_expert_cache_prefetch(layer.ref, cache.ref, _ptr(ids), int(ids.numel()), _ptr(workspace),
                                             workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "redmoe_expert_cache_prefetch")


# ------------------------------------------------------------------ around the layer
TORCH_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_CODES = {torch.float32: 0, torch.bfloat16: 1}
GATES = {"none": 0, "token": 1, "channel": 2, "element": 3}
GATE_ACTS = {"linear": 0, "sigmoid": 1}


def _arg(t: Optional[torch.Tensor], name: str, shape, dtype: torch.dtype, dev: int):
    """The address of a tensor argument, checked; None stays None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor {list(shape)} on cuda:{dev}, got {t.dtype} "
                         f"{list(t.shape)} on {t.device}{'' if t.is_contiguous() else ', not contiguous'}")
    return t.data_ptr()


_INT32_MAX = 2**31 - 1


def _int32(n: int, name: str) -> int:
    """A size that the library takes as int32 (ctypes would cut a longer one silently)."""
    if not -2**31 <= n < 2**31:
        raise ValueError(f"{name} = {n} is beyond int32")
    return n


def _rows(t: torch.Tensor, name: str) -> int:
    """T of a tensor whose first dimension is the token rows (its shape is checked beside the others')."""
    shape = t.shape
    if not shape:
        raise ValueError(f"{name}: expected rows of tokens, got a scalar")
    return shape[0] if shape[0] <= _INT32_MAX else _int32(shape[0], "T")


def _device_of(t: torch.Tensor, name: str) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name}: expected a CUDA tensor, got one on {t.device}")
    return dev


def _work(workspace: Optional[torch.Tensor], dev: int):
    """(address, bytes) of a workspace tensor or (None, 0)."""
    if workspace is None:
        return None, 0
    if not workspace.is_contiguous() or workspace.get_device() != dev:
        raise ValueError(f"workspace: expected a contiguous tensor on cuda:{dev}, got one on {workspace.device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


# The calls below are short beside what Python adds to them, so each is written out: a call for another
# device than the current one starts over with that device current, and every attribute is read once.
def _elsewhere(dev: int, fn, *args, **kw) -> None:
    with torch.cuda.device(dev):
        fn(*args, **kw)


class Norm:
    """The step between blocks (redmoe_norm): u = N(y; post_w) or y, h_out = res_scale h +
    block_scale g u, x = N(h_out; pre_w), with N the RMS norm and g the gate.

    gate: "none", "token" [T], "channel" [H] or "element" [T, H]; gate_act: "linear" or
    "sigmoid". Weights are [H] in one dtype, or None (factor 1); post_norm defaults to whether
    post_w is given. The weights are kept alive by this object.
    """

    def __init__(self, hidden: int, h_dtype: str = "bf16", y_dtype: str = "f32", x_dtype: str = "bf16",
                 pre_w: Optional[torch.Tensor] = None, post_w: Optional[torch.Tensor] = None,
                 post_norm: Optional[bool] = None, gate: str = "none", gate_act: str = "linear",
                 gate_dtype: str = "bf16", eps: float = 1e-6, w_offset: float = 0.0, res_scale: float = 1.0,
                 block_scale: float = 1.0):
        if pre_w is not None and post_w is not None and pre_w.dtype is not post_w.dtype:
            raise ValueError(f"pre_w and post_w have one dtype: got {pre_w.dtype} and {post_w.dtype}")
        first = pre_w if pre_w is not None else post_w
        self.device = None
        if first is not None:
            if first.dtype not in _CODES:
                raise ValueError(f"norm weights are float32 or bfloat16: got {first.dtype}")
            self.device = _device_of(first, "pre_w" if pre_w is not None else "post_w")
        s = _Norm()
        s.hidden = _int32(hidden, "hidden")
        s.h_dtype, s.y_dtype, s.x_dtype = DTYPES[h_dtype], DTYPES[y_dtype], DTYPES[x_dtype]
        s.w_dtype = _CODES[first.dtype] if first is not None else 0
        s.post_norm = int(post_w is not None if post_norm is None else post_norm)
        s.gate_kind, s.gate_act, s.gate_dtype = GATES[gate], GATE_ACTS[gate_act], DTYPES[gate_dtype]
        s.eps, s.w_offset, s.res_scale, s.block_scale = eps, w_offset, res_scale, block_scale
        dt = first.dtype if first is not None else None
        s.pre_w = _arg(pre_w, "pre_w", (hidden,), dt, self.device)
        s.post_w = _arg(post_w, "post_w", (hidden,), dt, self.device)
        self.struct, self.ref = s, C.byref(s)
        self.hidden, self.gate = hidden, gate
        self.pre_w, self.post_w = pre_w, post_w
        self.h_torch, self.y_torch, self.x_torch, self.gate_torch = (TORCH_DTYPES[d] for d in
                                                                     (h_dtype, y_dtype, x_dtype, gate_dtype))

    def gate_shape(self, T: int):
        return {"none": (0,), "token": (T,), "channel": (self.hidden,), "element": (T, self.hidden)}[self.gate]

    def _dev(self, t: torch.Tensor, name: str) -> int:
        dev = _device_of(t, name)
        if self.device is not None and self.device != dev:
            raise ValueError(f"{name} is on cuda:{dev}, the norm's weights on cuda:{self.device}")
        return dev


def redmoe_norm_forward(norm: Norm, h: torch.Tensor, h_out: Optional[torch.Tensor] = None,
                        x: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                        gate: Optional[torch.Tensor] = None, stream=None) -> None:
    """x <- N(h) (no y), or h_out [T,H] (may be h) and, where given, x [T,H] <- the residual step on (h, y)."""
    dev = norm._dev(h, "h")
    if dev != _raw_device():  # a tensor on a device: CUDA is initialised
        return _elsewhere(dev, redmoe_norm_forward, norm, h, h_out, x, y, gate, stream)
    rows, ht = h.shape, norm.h_torch
    T = rows[0] if rows else 0
    if T > _INT32_MAX or rows != (T, norm.hidden):
        rows = (_int32(T, "T"), norm.hidden)
    st = (_lib or load()).redmoe_norm_forward(
        norm.ref, _arg(h, "h", rows, ht, dev), None if y is None else _arg(y, "y", rows, norm.y_torch, dev),
        None if gate is None else _arg(gate, "gate", norm.gate_shape(T), norm.gate_torch, dev), T,
        None if h_out is None else _arg(h_out, "h_out", rows, ht, dev),
        None if x is None else _arg(x, "x", rows, norm.x_torch, dev),
        _raw_stream(dev) if stream is None else _stream(stream))
    if st:
        raise RedmoeError(st, "redmoe_norm_forward")


def redmoe_norm_workspace_bytes(norm: Norm, T: int) -> int:
    return int(load().redmoe_norm_workspace_bytes(norm.ref, _int32(int(T), "T")))


def new_norm_workspace(norm: Norm, T: int, device=None) -> torch.Tensor:
    """A zeroed workspace tensor for redmoe_norm_backward at T rows."""
    n = redmoe_norm_workspace_bytes(norm, T)
    if n == 0:
        raise ValueError("invalid norm or token count")
    if device is None:
        device = "cuda" if norm.device is None else f"cuda:{norm.device}"
    return torch.zeros(n, dtype=torch.uint8, device=device)


def redmoe_norm_backward(norm: Norm, h_out: torch.Tensor, dh: torch.Tensor, workspace: Optional[torch.Tensor],
                         dh_out: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                         y: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                         dy: Optional[torch.Tensor] = None, dgate: Optional[torch.Tensor] = None,
                         dpost_w: Optional[torch.Tensor] = None, dpre_w: Optional[torch.Tensor] = None,
                         stream=None) -> None:
    """dh, dy, dgate, dpost_w and dpre_w (fp32 [H]) <- the gradients dh_out and dx that arrive at
    h_out and x. dgate is fp32 for a token or channel gate, the gate's dtype for an element gate."""
    dev = norm._dev(h_out, "h_out")
    if dev != _raw_device():
        return _elsewhere(dev, redmoe_norm_backward, norm, h_out, dh, workspace, dh_out, dx, y, gate, dy, dgate, dpost_w,
                          dpre_w, stream)
    T = _rows(h_out, "h_out")
    rows, cols, f32, ht = (T, norm.hidden), (norm.hidden,), torch.float32, norm.h_torch
    g = dg = None
    if gate is not None:
        g = _arg(gate, "gate", norm.gate_shape(T), norm.gate_torch, dev)
    if dgate is not None:
        dg = _arg(dgate, "dgate", norm.gate_shape(T), norm.gate_torch if norm.gate == "element" else f32, dev)
    ws, nbytes = _work(workspace, dev)
    st = (_lib or load()).redmoe_norm_backward(
        norm.ref, _arg(h_out, "h_out", rows, ht, dev), None if y is None else _arg(y, "y", rows, norm.y_torch, dev), g,
        None if dh_out is None else _arg(dh_out, "dh_out", rows, ht, dev),
        None if dx is None else _arg(dx, "dx", rows, norm.x_torch, dev), T, _arg(dh, "dh", rows, ht, dev),
        None if dy is None else _arg(dy, "dy", rows, norm.y_torch, dev), dg,
        None if dpost_w is None else _arg(dpost_w, "dpost_w", cols, f32, dev),
        None if dpre_w is None else _arg(dpre_w, "dpre_w", cols, f32, dev), ws, nbytes,
        _raw_stream(dev) if stream is None else _stream(stream))
    if st:
        raise RedmoeError(st, "redmoe_norm_backward")


def redmoe_workspace_bytes_block(layer: Layer, T: int) -> int:
    return int(load().redmoe_workspace_bytes_block(layer.ref, _int32(int(T), "T")))


def new_workspace_block(layer: Layer, T: int, device=None) -> torch.Tensor:
    """A zeroed workspace tensor of redmoe_workspace_bytes_block(layer, T) bytes."""
    n = redmoe_workspace_bytes_block(layer, T)
    if n == 0:
        raise ValueError("invalid layer or token count")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def redmoe_forward_block(layer: Layer, before: Norm, after: Norm, h: torch.Tensor, h_out: torch.Tensor,
                         topk_ids: torch.Tensor, topk_w: torch.Tensor, workspace: torch.Tensor,
                         x_next: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                         stream=None) -> None:
    """The residual block around the layer: x = N(h) by `before`, y = layer(x), then `after`'s step on
    (h, y) into h_out (may be h) and, where given, x_next."""
    dev = before._dev(h, "h")
    after._dev(h, "h")
    if dev != _raw_device():
        return _elsewhere(dev, redmoe_forward_block, layer, before, after, h, h_out, topk_ids, topk_w, workspace, x_next,
                          gate, stream)
    T = _rows(h, "h")
    for name, t in layer.tensors.items():
        if t is not None and t.get_device() != dev:
            raise ValueError(f"the layer's {name} is on {t.device}, h on cuda:{dev}")
    rows, picks = (T, layer.hidden), (T, layer.top_k)
    ws, nbytes = _work(workspace, dev)
    st = (_lib or load()).redmoe_forward_block(
        layer.ref, before.ref, after.ref, _arg(h, "h", rows, before.h_torch, dev),
        None if gate is None else _arg(gate, "gate", after.gate_shape(T), after.gate_torch, dev), T,
        _arg(h_out, "h_out", rows, after.h_torch, dev), _arg(x_next, "x_next", rows, after.x_torch, dev),
        _arg(topk_ids, "topk_ids", picks, torch.int32, dev), _arg(topk_w, "topk_w", picks, torch.float32, dev),
        ws, nbytes, _raw_stream(dev) if stream is None else _stream(stream))
    if st:
        raise RedmoeError(st, "redmoe_forward_block")


def redmoe_balance_workspace_bytes(T: int, n_experts: int) -> int:
    return int(load().redmoe_balance_workspace_bytes(_int32(int(T), "T"), _int32(int(n_experts), "n_experts")))


def new_balance_workspace(T: int, n_experts: int, device=None) -> torch.Tensor:
    """A zeroed workspace tensor for redmoe_balance_forward."""
    n = redmoe_balance_workspace_bytes(T, n_experts)
    if n == 0:
        raise ValueError("invalid token or expert count")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def _logits(logits: torch.Tensor):
    dev, code, shape = _device_of(logits, "logits"), _CODES.get(logits.dtype), logits.shape
    if code is None or len(shape) != 2 or not logits.is_contiguous():
        raise ValueError(f"logits: expected a contiguous float32 or bfloat16 [T, E] tensor, got {logits.dtype} "
                         f"{list(logits.shape)}")
    T, E = shape
    if T > _INT32_MAX or E > _INT32_MAX:
        _int32(max(T, E), "a size of logits")
    return dev, code, T, E


def _mask(mask: Optional[torch.Tensor], T: int, dev: int):
    if mask is not None and mask.dtype is torch.bool:
        return _arg(mask, "mask", (T,), torch.bool, dev)
    return _arg(mask, "mask", (T,), torch.uint8, dev)


def redmoe_balance_forward(logits: torch.Tensor, topk_ids: torch.Tensor, loss: torch.Tensor, counts: torch.Tensor,
                           prob: torch.Tensor, n_rows: torch.Tensor, workspace: torch.Tensor,
                           mask: Optional[torch.Tensor] = None, stream=None) -> None:
    """loss[2] fp32 (balance, z), counts[E] int32, prob[E] fp32, n_rows[1] int32 <- the rows of logits
    [T,E] and topk_ids [T,k] int32 whose mask byte [T] (uint8 or bool) is not zero."""
    dev, code, T, E = _logits(logits)
    if dev != _raw_device():
        return _elsewhere(dev, redmoe_balance_forward, logits, topk_ids, loss, counts, prob, n_rows, workspace, mask, stream)
    if topk_ids.dim() != 2:
        raise ValueError(f"topk_ids: expected [T, k], got {list(topk_ids.shape)}")
    k = _int32(topk_ids.shape[1], "k")
    f32, i32 = torch.float32, torch.int32
    ws, nbytes = _work(workspace, dev)
    st = (_lib or load()).redmoe_balance_forward(
        logits.data_ptr(), code, _arg(topk_ids, "topk_ids", (T, k), i32, dev),
        None if mask is None else _mask(mask, T, dev), T, E, k, _arg(loss, "loss", (2,), f32, dev),
        _arg(counts, "counts", (E,), i32, dev), _arg(prob, "prob", (E,), f32, dev),
        _arg(n_rows, "n_rows", (1,), i32, dev), ws, nbytes, _raw_stream(dev) if stream is None else _stream(stream))
    if st:
        raise RedmoeError(st, "redmoe_balance_forward")


def redmoe_balance_backward(logits: torch.Tensor, counts: torch.Tensor, n_rows: torch.Tensor, grad_loss: torch.Tensor,
                            dlogits: torch.Tensor, top_k: int, mask: Optional[torch.Tensor] = None,
                            stream=None) -> None:
    """dlogits [T,E] (the logits' dtype; may be logits) <- grad_loss[2] fp32, with the forward call's
    counts, n_rows and mask."""
    dev, code, T, E = _logits(logits)
    if dev != _raw_device():
        return _elsewhere(dev, redmoe_balance_backward, logits, counts, n_rows, grad_loss, dlogits, top_k, mask, stream)
    i32 = torch.int32
    st = (_lib or load()).redmoe_balance_backward(
        logits.data_ptr(), code, None if mask is None else _mask(mask, T, dev), T, E, _int32(top_k, "top_k"),
        _arg(counts, "counts", (E,), i32, dev), _arg(n_rows, "n_rows", (1,), i32, dev),
        _arg(grad_loss, "grad_loss", (2,), torch.float32, dev), _arg(dlogits, "dlogits", (T, E), logits.dtype, dev),
        _raw_stream(dev) if stream is None else _stream(stream))
    if st:
        raise RedmoeError(st, "redmoe_balance_backward")


class Matrix:
    """A dense matrix [rows, cols] in an expert weight format (redmoe_matrix): packed bytes w [rows, cols/2]
    and bf16 scales s [rows, cols/32], kept alive by this object."""

    def __init__(self, w: torch.Tensor, s: torch.Tensor, rows: int, cols: int, dtype: str = "int4g32"):
        self.device = _device_of(w, "w")
        if dtype == "int4g32":  # other formats are refused by the call
            _arg(w, "w", (rows, cols // 2), torch.uint8, self.device)
            _arg(s, "s", (rows, cols // 32), torch.bfloat16, self.device)
        _int32(rows, "rows"), _int32(cols, "cols")
        st = _Matrix()
        st.rows, st.cols, st.dtype, st.w, st.s = rows, cols, DTYPES[dtype], _ptr(w), _ptr(s)
        self.struct, self.ref = st, C.byref(st)
        self.rows, self.cols, self.w, self.s = rows, cols, w, s


def redmoe_gemv(matrix: Matrix, x: torch.Tensor, y: torch.Tensor, stream=None) -> None:
    """y[T, rows] (fp32 or bf16) <- x[T, cols] bf16 times the matrix's transpose, T = 0..32."""
    dev = matrix.device
    if dev != _raw_device():
        return _elsewhere(dev, redmoe_gemv, matrix, x, y, stream)
    xt, yt, T = x.dtype, y.dtype, _rows(x, "x")
    xc, yc = _CODES.get(xt), _CODES.get(yt)
    if xc is None or yc is None:
        raise ValueError(f"x and y are float32 or bfloat16: got {xt} and {yt}")
    st = (_lib or load()).redmoe_gemv(matrix.ref, _arg(x, "x", (T, matrix.cols), xt, dev), xc, T,
                                      _arg(y, "y", (T, matrix.rows), yt, dev), yc,
                                      _raw_stream(dev) if stream is None else _stream(stream))
    if st:
        raise RedmoeError(st, "redmoe_gemv")
