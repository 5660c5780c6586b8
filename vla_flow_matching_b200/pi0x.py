"""Python binding of libpi0x (include/pi0x.h) — argument marshalling only.

Every step of the denoising loop runs in the library's CUDA kernels; this module
only converts numpy arrays / torch tensors to pointers and checks status codes.
The paged-cache calls are marshalled in C (csrc/binding.c), the others by ctypes.
It raises if the shared library is missing: there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import numpy as np

try:
    import torch
except ImportError:  # the sampler itself takes numpy arrays
    torch = None

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libpi0x.so")

PI0X_OK, PI0X_EINVAL, PI0X_EUNSUPPORTED, PI0X_ENOMEM, PI0X_ECUDA, PI0X_ETIMEOUT, PI0X_EDEVICE = range(7)
PI0X_BF16, PI0X_FP32 = 0, 1
PI0X_DTYPE_BF16, PI0X_DTYPE_F32, PI0X_DTYPE_E4M3, PI0X_DTYPE_INT8 = range(4)

#: Every symbol include/pi0x.h declares.
EXPORTED = ["pi0x_create", "pi0x_sample", "pi0x_sync_status", "pi0x_launch_count",
            "pi0x_status_string", "pi0x_last_error", "pi0x_destroy", "pi0x_version",
            "pi0x_debug_gemm_bf16", "pi0x_debug_attention", "pi0x_profile_enable", "pi0x_profile_read",
            "pi0x_set_variant", "pi0x_attention_noalloc", "pi0x_uses_loop", "pi0x_debug_loop_stall",
            "pi0x_debug_set_loop", "pi0x_qk_norm_rope", "pi0x_cache_write", "pi0x_cache_read",
            "pi0x_cache_attention", "pi0x_cache_attention_workspace", "pi0x_sample_cache"]

#: time grids of pi0x_set_variant
PI0X_TIME_PI0 = 0
PI0X_TIME_LINSPACE = 1

#: kernel classes of pi0x_profile_read
K_CLASSES = ["prep", "embed", "gemm", "norm", "rope", "attn", "geglu", "final", "loop"]


class Pi0xError(RuntimeError):
    def __init__(self, status: int, what: str):
        lib = load()
        msg = lib.pi0x_status_string(status).decode()
        detail = lib.pi0x_last_error().decode()
        super().__init__(f"{what}: {msg} ({status}){': ' + detail if detail else ''}")
        self.status = status


class Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in
                ("width", "depth", "mlp_dim", "num_heads", "num_kv_heads", "head_dim",
                 "horizon", "action_dim", "state_dim", "precision")]


_LAYER_FIELDS = ("in_norm_w", "q_w", "k_w", "v_w", "o_w", "post_norm_w", "gate_w", "up_w", "down_w")


class LayerWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in _LAYER_FIELDS]


_TOP_FIELDS = ("state_proj_w", "state_proj_b", "action_in_w", "action_in_b", "time_in_w",
               "time_in_b", "time_out_w", "time_out_b", "action_out_w", "action_out_b",
               "final_norm_w")


class Weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in _TOP_FIELDS] + [
        ("layers", ctypes.POINTER(LayerWeights)), ("dtype", ctypes.c_int)]


class Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p)] + [
        (n, ctypes.c_int) for n in ("layers", "num_pages", "page_size", "kv_heads", "head_dim", "dtype")]


class Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class Rotation(ctypes.Structure):
    _fields_ = [("q_gain", ctypes.c_void_p), ("k_gain", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("rope_base", ctypes.c_float)]


_lib = None
_native = None  # the paged-cache calls' marshalling, csrc/binding.c


def _fail(status: int, what: str):
    raise Pi0xError(status, what)


def load() -> ctypes.CDLL:
    """Load libpi0x.so (built in-tree by vla_flow_matching_b200.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"{_LIB_PATH} is missing: run `python -m vla_flow_matching_b200.build`")
    lib = ctypes.CDLL(_LIB_PATH)
    lib.pi0x_create.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(Weights),
                                ctypes.POINTER(ctypes.c_void_p)]
    lib.pi0x_create.restype = ctypes.c_int
    lib.pi0x_sample.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p),
                                ctypes.POINTER(ctypes.c_void_p), ctypes.c_void_p, ctypes.c_int,
                                ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                ctypes.c_void_p, ctypes.c_void_p]
    lib.pi0x_sample.restype = ctypes.c_int
    lib.pi0x_set_variant.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int]
    lib.pi0x_set_variant.restype = ctypes.c_int
    lib.pi0x_sync_status.argtypes = [ctypes.c_void_p]
    lib.pi0x_sync_status.restype = ctypes.c_int
    lib.pi0x_launch_count.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int]
    lib.pi0x_launch_count.restype = ctypes.c_long
    lib.pi0x_status_string.argtypes = [ctypes.c_int]
    lib.pi0x_status_string.restype = ctypes.c_char_p
    lib.pi0x_last_error.argtypes = []
    lib.pi0x_last_error.restype = ctypes.c_char_p
    lib.pi0x_destroy.argtypes = [ctypes.c_void_p]
    lib.pi0x_destroy.restype = None
    lib.pi0x_version.argtypes = []
    lib.pi0x_version.restype = ctypes.c_int
    lib.pi0x_debug_gemm_bf16.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int,
                                         ctypes.c_int, ctypes.c_void_p, ctypes.c_int, ctypes.c_int,
                                         ctypes.c_void_p]
    lib.pi0x_debug_gemm_bf16.restype = ctypes.c_int
    lib.pi0x_debug_attention.argtypes = [ctypes.c_void_p] * 6 + [ctypes.c_int] * 5 + [ctypes.c_void_p] * 2
    lib.pi0x_debug_attention.restype = ctypes.c_int
    lib.pi0x_attention_noalloc.argtypes = [ctypes.c_void_p] * 6 + [ctypes.c_int] * 4 + [ctypes.c_void_p] * 2
    lib.pi0x_attention_noalloc.restype = ctypes.c_int
    lib.pi0x_uses_loop.argtypes = [ctypes.c_void_p, ctypes.c_int]
    lib.pi0x_uses_loop.restype = ctypes.c_int
    lib.pi0x_debug_loop_stall.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_ulonglong]
    lib.pi0x_debug_loop_stall.restype = ctypes.c_int
    lib.pi0x_debug_set_loop.argtypes = [ctypes.c_void_p, ctypes.c_int]
    lib.pi0x_debug_set_loop.restype = ctypes.c_int
    lib.pi0x_profile_enable.argtypes = [ctypes.c_void_p, ctypes.c_int]
    lib.pi0x_profile_enable.restype = ctypes.c_int
    lib.pi0x_profile_read.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(ctypes.c_long),
                                      ctypes.POINTER(ctypes.c_double)]
    lib.pi0x_profile_read.restype = ctypes.c_int
    ptr, cint, rows, cache = ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(Rows), ctypes.POINTER(Cache)
    lib.pi0x_qk_norm_rope.argtypes = [cint] * 6 + [rows, rows, ptr, ctypes.POINTER(Rotation), rows, rows, ptr]
    lib.pi0x_qk_norm_rope.restype = cint
    lib.pi0x_cache_write.argtypes = [cache, cint, cint, cint, cint, rows, rows, ptr, cint, ptr, ptr,
                                     ctypes.POINTER(Rotation), cint, rows, rows, ptr]
    lib.pi0x_cache_write.restype = cint
    lib.pi0x_cache_read.argtypes = [cache, cint, cint, cint, cint, ptr, cint, ptr, ptr, cint, ptr, ptr, ptr, ptr]
    lib.pi0x_cache_read.restype = cint
    lib.pi0x_cache_attention.argtypes = [cache, cint, cint, cint, rows, ptr, cint, ptr, ptr, cint, ctypes.c_float,
                                         ptr, ptr, ptr, ctypes.c_size_t, ptr]
    lib.pi0x_cache_attention.restype = cint
    lib.pi0x_cache_attention_workspace.argtypes = [cache, cint, cint, cint]
    lib.pi0x_cache_attention_workspace.restype = ctypes.c_size_t
    lib.pi0x_sample_cache.argtypes = [ptr, cache, cint, cint, ptr, cint, ptr, ptr, ptr, ptr, cint, ptr, ptr]
    lib.pi0x_sample_cache.restype = cint
    _lib = lib
    return lib


def load_binding():
    """Load libpi0x.so and the paged-cache calls' marshalling (_binding.so), which the first of those
    calls does by itself.  It needs a torch with DLPack's C exchange interface (2.11 has it);
    :class:`Sampler` does without."""
    global _native
    if _native is None:
        load()
        if torch is None:
            raise ImportError("the paged-cache calls take torch tensors, and torch cannot be imported")
        try:
            from . import _binding
            _binding.setup(torch, _fail)
        except ImportError as e:
            raise ImportError(f"the paged-cache calls need _binding.so, built by `python -m "
                              f"vla_flow_matching_b200.build --force` beside a torch like 2.11: {e}") from e
        _native = _binding
    return _native


def _ptr(a) -> int:
    """Data pointer of a numpy array (host) or a torch tensor (host or device)."""
    if a is None:
        return 0
    if hasattr(a, "data_ptr"):
        if not a.is_contiguous():
            raise ValueError("tensor must be contiguous")
        return int(a.data_ptr())
    if isinstance(a, np.ndarray):
        if not a.flags["C_CONTIGUOUS"]:
            raise ValueError("array must be C-contiguous")
        return int(a.ctypes.data)
    raise TypeError(f"unsupported array type {type(a)}")


def _check(status: int, what: str):
    if status != PI0X_OK:
        raise Pi0xError(status, what)


def debug_gemm_bf16(A, Bw, D, bn: int = 128, splits: int = 1, stream: int = 0):
    """D = A @ Bw.T with the library's tcgen05 GEMM (device torch tensors: bf16, bf16, fp32)."""
    M, K = A.shape
    N = Bw.shape[0]
    _check(load().pi0x_debug_gemm_bf16(_ptr(A), _ptr(Bw), M, N, K, _ptr(D), bn, splits,
                                       ctypes.c_void_p(stream)), "pi0x_debug_gemm_bf16")
    return D


def debug_attention(q, ks, vs, prefix_k, prefix_v, mask, B, H, P, step0, out, impl=1, stream: int = 0):
    """One layer of suffix attention with the library's kernels (device torch tensors)."""
    _check(load().pi0x_debug_attention(_ptr(q), _ptr(ks), _ptr(vs), _ptr(prefix_k), _ptr(prefix_v), _ptr(mask),
                                       B, H, P, int(step0), int(impl), _ptr(out), ctypes.c_void_p(stream)),
           "pi0x_debug_attention")
    return out


def attention_noalloc(q, ks, vs, prefix_k, prefix_v, mask, B, H, P, step0, out, stream: int = 0):
    """The same attention through pi0x_attention_noalloc (no device allocation;
    scratch in the library's static device array)."""
    _check(load().pi0x_attention_noalloc(_ptr(q), _ptr(ks), _ptr(vs), _ptr(prefix_k), _ptr(prefix_v), _ptr(mask),
                                         B, H, P, int(step0), _ptr(out), ctypes.c_void_p(stream)),
           "pi0x_attention_noalloc")
    return out


def qk_norm_rope(q, k=None, start=None, *, positions=None, q_gain=None, k_gain=None, eps: float = 1e-6,
                 rope_base: Optional[float] = 10000.0, q_out=None, k_out=None):
    """Per-head RMSNorm (where a gain is given: gain 1 + g) and rotate-half rotation of
    queries and keys in one pass (pi0x_qk_norm_rope).

    ``q`` (B, T, heads, D) and ``k`` (B, T, kv_heads, D) or None: bf16 or fp32 CUDA
    tensors, D 64, 128 or 256, any strides in whole 16 bytes with a contiguous last
    dimension.  Token t of sample b has position ``positions[b, t]``, or
    ``start[b] + t`` (start None: 0).  ``rope_base`` None: no rotation.  Returns
    (q_out, k_out), new tensors unless given; an output may be its own input.
    Runs on the current stream of the tensors' device.  For inference: no gradient
    flows back, also where an input requires one, and autograd does not see what is
    written in place.
    """
    if _native is None:
        load_binding()
    r = _native.qk_norm_rope(q, k, start, positions, q_gain, k_gain, eps, rope_base, q_out, k_out)
    if r is NotImplemented:
        with torch.cuda.device(q.device):
            return _native.qk_norm_rope(q, k, start, positions, q_gain, k_gain, eps, rope_base, q_out, k_out)
    return r


class KVCache:
    """A paged key-value cache (pi0x_cache) over torch tensors.

    ``k``, ``v``: (layers, num_pages, page_size, kv_heads, head_dim) contiguous pools of
    bfloat16, float8_e4m3fn or int8; ``k_scale``, ``v_scale``: (layers, num_pages,
    page_size, kv_heads) float32, for the 8-bit types.  :meth:`empty` makes them.
    Which pages a sample has is the caller's: every method takes ``table`` (B,
    max_pages) int32 page numbers; an entry outside the pool holds no keys.  Methods
    run on the current stream of the cache's device, and may be captured into a graph.
    For inference: no method has a backward pass, inputs that require gradients are
    taken as plain data, and autograd does not see writes to pools and given outputs.
    """

    def __init__(self, k, v, k_scale=None, v_scale=None):
        types = {torch.bfloat16: PI0X_DTYPE_BF16, torch.float8_e4m3fn: PI0X_DTYPE_E4M3, torch.int8: PI0X_DTYPE_INT8}
        if k.dtype not in types or k.dtype != v.dtype or k.dim() != 5 or k.shape != v.shape or \
                not k.is_contiguous() or not v.is_contiguous():
            raise ValueError("KVCache: k and v must be contiguous (layers, num_pages, page_size, kv_heads, head_dim) "
                             "tensors of one type: bfloat16, float8_e4m3fn or int8")
        scaled = k.dtype != torch.bfloat16
        if scaled != (k_scale is not None) or scaled != (v_scale is not None):
            raise ValueError("KVCache: 8-bit pools need k_scale and v_scale, bfloat16 pools take none")
        for s in (k_scale, v_scale):
            if s is not None and (s.dtype != torch.float32 or s.shape != k.shape[:4] or not s.is_contiguous()):
                raise ValueError("KVCache: scales must be contiguous float32 (layers, num_pages, page_size, kv_heads)")
        for t in (k, v, k_scale, v_scale):
            if t is not None and (not t.is_cuda or t.device != k.device):
                raise ValueError("KVCache: every pool must be on one CUDA device")
        self._pools = k, v, k_scale, v_scale
        self.layers, self.num_pages, self.page_size, self.kv_heads, self.head_dim = k.shape
        self.device = k.device
        self._index = k.device.index
        self._desc = Cache(k.data_ptr(), v.data_ptr(), _ptr(k_scale), _ptr(v_scale), *k.shape, types[k.dtype])
        self._address = ctypes.addressof(self._desc)
        load_binding()

    # The descriptor holds these tensors' addresses, so they stay the cache's for its life.
    k = property(lambda self: self._pools[0])
    v = property(lambda self: self._pools[1])
    k_scale = property(lambda self: self._pools[2])
    v_scale = property(lambda self: self._pools[3])

    @classmethod
    def empty(cls, layers: int, num_pages: int, page_size: int, kv_heads: int = 1, head_dim: int = 256,
              dtype: str = "bf16", device="cuda"):
        """A cache of zeros; ``dtype`` "bf16", "e4m3" or "int8"."""
        types = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
        if dtype not in types:
            raise ValueError(f"KVCache: dtype is one of {sorted(types)}")
        shape = (layers, num_pages, page_size, kv_heads, head_dim)
        pools = [torch.zeros(shape, dtype=types[dtype], device=device) for _ in range(2)]
        if dtype != "bf16":
            pools += [torch.zeros(shape[:4], dtype=torch.float32, device=device) for _ in range(2)]
        return cls(*pools)

    def _call(self, function, *args):
        """`function` of the native binding on this cache, with its device current."""
        r = function(self._address, self._index, *args)
        if r is NotImplemented:
            with torch.cuda.device(self._index):
                return function(self._address, self._index, *args)
        return r

    def write(self, layer: int, k, v, table, start, count=None, *, q=None, q_out=None, positions=None, q_gain=None,
              k_gain=None, eps: float = 1e-6, rope_base: Optional[float] = None):
        """Write T new tokens a sample into the pages of ``layer`` (pi0x_cache_write).

        ``k``, ``v`` (B, T, kv_heads, head_dim) bf16 or fp32; token t of sample b goes to
        slot ``start[b] + t``; those at t >= ``count[b]`` (None: T) are left out.  With
        ``rope_base`` or a gain, keys are normed and rotated first as by
        :func:`qk_norm_rope`, and so is ``q`` (B, T, heads, head_dim), in the same pass.
        Returns ``q_out`` (new unless given), or None without q.
        """
        return self._call(_native.cache_write, layer, k, v, table, start, count, q, q_out, positions, q_gain, k_gain,
                          eps, rope_base)

    def read(self, table, lens, length: int, *, mask=None, layer0: int = 0, layers: Optional[int] = None, dtype=None,
             k_out=None, v_out=None, mask_out=None):
        """Slots 0..length-1 of ``layers`` layers from ``layer0`` (None: to the last) as
        contiguous (layers, B, kv_heads, length, head_dim) keys and values of ``dtype``
        (bfloat16, the default, or float32), and a (B, length) uint8 mask of the slots
        that hold a key: below ``lens[b]``, on a page of the pool and, with ``mask`` (B,
        length), nonzero there.  The others come out as zeros (pi0x_cache_read).
        """
        n = self.layers - layer0 if layers is None else layers
        return self._call(_native.cache_read, table, lens, length, mask, layer0, n, dtype or torch.bfloat16, k_out,
                          v_out, mask_out)

    def attend(self, layer: int, q, table, lens, *, mask=None, scale: Optional[float] = None, out=None, lse=None):
        """Attention of one new token a sample over the pages of ``layer``
        (pi0x_cache_attention): ``q`` (B, heads, head_dim) bf16, heads a multiple of
        kv_heads; keys are the slots below ``lens[b]`` on pages of the pool and, with
        ``mask`` (B, length), below its length and nonzero there.  ``scale`` None:
        head_dim ** -0.5.  Returns (out, lse): (B, heads, head_dim) bf16 and (B, heads)
        fp32, zeros and -inf for a sample without keys.
        """
        return self._call(_native.cache_attention, layer, q, table, lens, mask,
                          self.head_dim ** -0.5 if scale is None else scale, out, lse)


def _is_floats(a, n: int, device) -> bool:
    """Whether `a` is n contiguous float32 values, a numpy array or a tensor on the host or `device`."""
    if isinstance(a, np.ndarray):
        return a.dtype == np.float32 and a.size == n and a.flags.c_contiguous
    return isinstance(a, torch.Tensor) and a.dtype == torch.float32 and a.numel() == n and a.is_contiguous() and \
        (a.device.type == "cpu" or a.device == device)


class Sampler:
    """A pi0x handle: expert weights on the device plus the loop's workspace.

    ``weights`` follows :func:`vla_flow_matching_b200.synth.make_weights`: a dict of
    arrays (bf16 bits as uint16, or float32) with a ``"layers"`` list.
    """

    def __init__(self, dims, weights: dict, precision: int = PI0X_BF16):
        lib = load()
        self._lib = lib
        self.dims = dims
        self.precision = precision
        cfg = Config(dims.width, dims.depth, dims.mlp_dim, dims.num_heads, dims.num_kv_heads,
                     dims.head_dim, dims.horizon, dims.action_dim, dims.state_dim, precision)
        first = weights["state_proj_w"]
        dtype = PI0X_DTYPE_BF16 if np.asarray(first).dtype == np.uint16 else PI0X_DTYPE_F32
        keep = []

        def arr(a):
            a = np.ascontiguousarray(a, dtype=np.uint16 if dtype == PI0X_DTYPE_BF16 else np.float32)
            keep.append(a)
            return _ptr(a)

        layers = (LayerWeights * dims.depth)()
        for i, lw in enumerate(weights["layers"]):
            for n in _LAYER_FIELDS:
                setattr(layers[i], n, arr(lw[n]))
        w = Weights(*[arr(weights[n]) for n in _TOP_FIELDS],
                    ctypes.cast(layers, ctypes.POINTER(LayerWeights)), dtype)
        h = ctypes.c_void_p()
        _check(lib.pi0x_create(ctypes.byref(cfg), ctypes.byref(w), ctypes.byref(h)), "pi0x_create")
        self._h = h

    def launch_count(self, B: int, P: int, num_steps: int) -> int:
        return int(self._lib.pi0x_launch_count(self._h, B, P, num_steps))

    def uses_loop(self, B: int) -> bool:
        """True if calls with batch B run the persistent small-batch loop kernel."""
        return bool(self._lib.pi0x_uses_loop(self._h, int(B)))

    def debug_set_loop(self, enable: bool):
        """Allow (True, default) or forbid (False) the persistent loop (see pi0x_debug.h)."""
        _check(self._lib.pi0x_debug_set_loop(self._h, int(bool(enable))), "pi0x_debug_set_loop")

    def debug_loop_stall(self, stage: int, wait_ns: int):
        """Make the next loop call stall at `stage` (test hook, see pi0x_debug.h)."""
        _check(self._lib.pi0x_debug_loop_stall(self._h, int(stage), int(wait_ns)), "pi0x_debug_loop_stall")

    def sample(self, prefix_k: Sequence, prefix_v: Sequence, mask, state, x1, num_steps: int,
               x0=None, stream: Optional[int] = None):
        """Enqueue one call; arrays may be torch tensors (host or device) or numpy arrays.

        Returns ``x0`` (the given output, or a new tensor/array like ``x1``).
        """
        if x0 is None:
            x0 = x1.new_empty(x1.shape) if hasattr(x1, "new_empty") else np.empty_like(x1)
        B, P = int(mask.shape[0]), int(mask.shape[1])
        L = self.dims.depth
        if len(prefix_k) != L or len(prefix_v) != L:
            raise ValueError("one prefix K and V per layer is required")
        pk = (ctypes.c_void_p * L)(*[_ptr(k) for k in prefix_k])
        pv = (ctypes.c_void_p * L)(*[_ptr(v) for v in prefix_v])
        if stream is None:
            stream = torch.cuda.current_stream().cuda_stream if torch and torch.cuda.is_available() else 0
        _check(self._lib.pi0x_sample(self._h, pk, pv, _ptr(mask), B, P, _ptr(state), _ptr(x1),
                                     int(num_steps), _ptr(x0), ctypes.c_void_p(stream)),
               "pi0x_sample")
        return x0

    def sample_cache(self, cache: KVCache, table, lens, length: int, state, x1, num_steps: int, mask=None, x0=None):
        """Enqueue one call whose prefix K/V are slots 0..length-1 of a paged cache, as
        :meth:`KVCache.read` reads them (pi0x_sample_cache).  Runs on the current stream
        of the cache's device."""
        B = int(table.shape[0])
        for name, t, dtypes, shape in (("table", table, (torch.int32,), (B, table.shape[-1])),
                                       ("lens", lens, (torch.int32,), (B,)),
                                       ("mask", mask, (torch.uint8, torch.bool), (B, length))):
            if t is not None and (t.device != cache.device or t.dtype not in dtypes or t.shape != shape or
                                  not t.is_contiguous()):
                raise ValueError(f"Sampler.sample_cache: {name} must be a contiguous {dtypes[0]} tensor of shape "
                                 f"{tuple(shape)} on {cache.device}")
        d = self.dims
        for name, a, n in (("state", state, B * d.state_dim), ("x1", x1, B * d.horizon * d.action_dim),
                           ("x0", x0, B * d.horizon * d.action_dim)):
            if (a is not None or name != "x0") and not _is_floats(a, n, cache.device):
                raise ValueError(f"Sampler.sample_cache: {name} must be {n} contiguous float32 values for a batch of "
                                 f"{B}, on the host or {cache.device}")
        if x0 is None:
            x0 = x1.new_empty(x1.shape) if hasattr(x1, "new_empty") else np.empty_like(x1)
        with torch.cuda.device(cache.device):
            _check(self._lib.pi0x_sample_cache(
                self._h, cache._desc, B, length, _ptr(table), int(table.shape[1]), _ptr(lens), _ptr(mask), _ptr(state),
                _ptr(x1), int(num_steps), _ptr(x0), torch.cuda.current_stream().cuda_stream), "pi0x_sample_cache")
        return x0

    def set_variant(self, time_grid: int = PI0X_TIME_PI0, x_prediction: bool = False,
                    causal_actions: bool = False):
        """Solver / convention variant for later calls (see pi0x_set_variant)."""
        _check(self._lib.pi0x_set_variant(self._h, int(time_grid), int(bool(x_prediction)),
                                          int(bool(causal_actions))), "pi0x_set_variant")

    def profile(self, on: bool = True):
        _check(self._lib.pi0x_profile_enable(self._h, int(on)), "pi0x_profile_enable")

    def profile_read(self) -> dict:
        """{class: (launches, total_ms)} of the most recent profiled call."""
        out = {}
        for i, name in enumerate(K_CLASSES):
            n, ms = ctypes.c_long(), ctypes.c_double()
            _check(self._lib.pi0x_profile_read(self._h, i, ctypes.byref(n), ctypes.byref(ms)),
                   "pi0x_profile_read")
            out[name] = (int(n.value), float(ms.value))
        return out

    def sync(self):
        _check(self._lib.pi0x_sync_status(self._h), "pi0x_sync_status")

    def close(self):
        if getattr(self, "_h", None):
            self._lib.pi0x_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
