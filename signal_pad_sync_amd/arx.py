"""ctypes binding of libarx.so (C ABI in include/arx.h, test aids in
include/arx_test.h).

Argument marshalling only: every step of the path runs in the library's HIP
kernels. torch provides device memory and streams; tensors are passed as
``data_ptr()`` and streams as ``torch.cuda.current_stream().cuda_stream``.
Importing this module raises if libarx.so is missing: there is no fallback.
"""
import atexit
import ctypes
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libarx.so")

OK, EINVAL, ESTATE, ENOMEM, EHIP, EPROXY, EORDER, ETIMEOUT = 0, -1, -2, -3, -4, -5, -6, -7
PROXY_LOCKSTEP, PROXY_RUNAHEAD, PROXY_MANUAL, PROXY_STRESS = 0, 1, 2, 3
SEM_RELAXED, SEM_ACQ_REL = 0, 1
BARRIER_LANES, BARRIER_SPLIT = 1, 2
MAX_WORLD, MAX_PAD_BLOCKS, MAX_N = 8, 1024, 1 << 30
NOALLOC_MAX_N = 1 << 20
BF16, F16, F32 = 0, 1, 2
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

# names of arx_debug_state's words, in order
STATE_WORDS = ["seq_dev", "cnt0", "cnt1", "go", "abort", "ctl_seq", "ctl_bytes0", "ctl_bytes1",
               "ctl_done", "ctl_err", "ctl_err_seq", "posted"]

_c = ctypes
_u64p = _c.POINTER(_c.c_uint64)
_vp, _sz = _c.c_void_p, _c.c_size_t

# (name, restype, argtypes) for every entry point of arx.h and arx_test.h
SIGNATURES = [
    ("arx_init", _c.c_int, [_c.c_int, _c.c_size_t]),
    ("arx_init_rank", _c.c_int, [_c.c_int, _c.c_size_t, _c.c_int]),
    ("arx_finalize", _c.c_int, []),
    ("arx_publish", _c.c_int, [_c.c_uint64]),
    ("arx_allreduce", _c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    ("arx_reduce", _c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_int, _c.c_void_p]),
    ("arx_barrier_blockwise", _c.c_int, [_c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_void_p, _c.c_void_p,
                                         _c.c_void_p]),
    ("arx_counter_barrier", _c.c_int, [_c.c_int, _c.c_int, _c.c_int, _c.c_void_p, _c.c_void_p, _c.c_void_p,
                                       _c.c_void_p]),
    ("arx_symm_allreduce", _c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_size_t, _c.c_int, _c.c_void_p]),
    ("arx_symm_allreduce_noalloc", _c.c_int, [_c.c_int, _c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_size_t, _c.c_int,
                                              _c.c_void_p, _c.c_void_p]),
    ("arx_barrier_max_blocks", _c.c_int, []),
    ("arx_sem_ptr", _c.c_void_p, [_c.c_int]),
    ("arx_epoch_ptr", _c.c_void_p, [_c.c_int]),
    ("arx_recv_ptr", _c.c_void_p, [_c.c_int, _c.c_int]),
    ("arx_send_ptr", _c.c_void_p, [_c.c_int]),
    ("arx_pad_ptr", _c.c_void_p, [_c.c_int]),
    ("arx_set_proxy_mode", _c.c_int, [_c.c_int]),
    ("arx_set_stress_source", _c.c_int, [_c.c_void_p, _c.c_int]),
    ("arx_set_timeout_us", _c.c_int, [_c.c_uint64]),
    ("arx_status", _c.c_int, [_u64p, _u64p, _u64p]),
    ("arx_debug_state", _c.c_int, [_u64p, _c.c_int]),
    ("arx_debug_set_seq", _c.c_int, [_c.c_uint64]),
    ("arx_debug_fail_proxy", _c.c_int, []),
    ("arx_test_round_bf16", _c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    ("arx_test_oneshot_shape", _c.c_int, [_c.c_size_t, _c.c_int, _c.c_int, _c.c_uint, _c.c_int,
                                          _c.POINTER(_c.c_int), _c.c_int]),
    ("arx_strerror", _c.c_char_p, [_c.c_int]),
    ("arx_max_n", _c.c_size_t, []),
    ("arx_world", _c.c_int, []),
    ("arx_rank", _c.c_int, []),
    ("arx_linear", _c.c_int, [_vp] * 6 + [_sz] * 8 + [_c.c_int] * 2 + [_vp, _sz, _vp]),
    ("arx_linear_workspace", _sz, [_sz] * 3 + [_c.c_int]),
    ("arx_linear_backward", _c.c_int, [_vp] * 7 + [_sz] * 9 + [_c.c_int] * 2 + [_vp, _sz, _vp]),
    ("arx_linear_backward_workspace", _sz, [_sz] * 3 + [_c.c_int] * 2),
    ("arx_layer_norm", _c.c_int, [_vp] * 6 + [_sz] * 4 + [_c.c_double] + [_c.c_int] * 2 + [_vp]),
    ("arx_layer_norm_backward", _c.c_int, [_vp] * 8 + [_sz] * 5 + [_c.c_int] * 2 + [_vp, _sz, _vp]),
    ("arx_dropout_add", _c.c_int, [_vp] * 4 + [_sz] * 5 + [_c.c_double] + [_c.c_uint64] * 2 + [_c.c_int, _vp]),
    ("arx_dropout_add_backward", _c.c_int, [_vp] * 3 + [_sz] * 4 + [_c.c_double] + [_c.c_uint64] * 2 +
     [_c.c_int, _vp, _sz, _vp]),
    ("arx_dropout_add_norm", _c.c_int, [_vp] * 9 + [_sz] * 6 + [_c.c_double] * 2 + [_c.c_uint64] * 2 +
     [_c.c_int] * 2 + [_vp]),
    ("arx_dropout_add_norm_backward", _c.c_int, [_vp] * 11 + [_sz] * 7 + [_c.c_double] + [_c.c_uint64] * 2 +
     [_c.c_int] * 2 + [_vp, _sz, _vp]),
    ("arx_rows_workspace", _sz, [_sz] * 2 + [_c.c_int]),
]


class ArxError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"arx error {code}: {msg}")
        self.code = code


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"libarx.so not found at {path}; build it with signal_pad_sync_amd/build.py")
    # One HIP runtime per process: torch's. The library receives torch's
    # device pointers and streams, which only that runtime knows. Loaded
    # first, libarx.so would bring in the system's runtime, and torch would
    # then load its own copy beside it (torch's libraries name the runtime
    # by another file name), and one of the two would see no device. torch
    # loaded first, libarx.so binds to its runtime by soname.
    import torch  # noqa: F401
    L = ctypes.CDLL(path)
    for name, res, args in SIGNATURES:
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    return L


lib = load()
import torch  # noqa: E402  (load() has imported it first)

_TYPES = {torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32}
_MATRIX_TYPES = {torch.bfloat16: BF16, torch.float16: F16}

# The current device and stream, as torch's own compiled code asks for them:
# torch.cuda.current_stream() costs a call 2.8 us of host time, this 0.1.
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)


@atexit.register
def _finalize_at_exit():
    if lib.arx_world() != 0:
        lib.arx_finalize()


def _check(rc):
    if rc < 0:
        raise ArxError(rc, lib.arx_strerror(rc).decode())
    return rc


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _buf(t, n: int, what: str, itemsize: int = 2):
    """Device address of tensor t, after checking that it is a contiguous GPU
    tensor of itemsize-byte elements holding at least n of them (the library
    sees only the address, so it cannot check the extent itself)."""
    if t is None:
        if n > 0:
            raise ArxError(EINVAL, f"{what} is None")
        return None
    if not getattr(t, "is_cuda", False):
        raise ArxError(EINVAL, f"{what} must be a GPU tensor")
    if t.element_size() != itemsize:
        raise ArxError(EINVAL, f"{what} must have {itemsize}-byte elements, not {t.dtype}")
    if not t.is_contiguous():
        raise ArxError(EINVAL, f"{what} must be contiguous")
    if t.numel() < n:
        raise ArxError(EINVAL, f"{what} holds {t.numel()} elements, fewer than {n}")
    return t.data_ptr()


def init(world: int, max_n: int, rank: int = 0):
    _check(lib.arx_init_rank(world, max_n, rank))


def finalize():
    _check(lib.arx_finalize())


def publish(seq: int):
    _check(lib.arx_publish(seq))


def allreduce(inp, out, n: int = None, stream=None):
    """One one-shot call: out[:n] = rank-ordered sum; inp/out bf16 tensors."""
    if n is None:
        n = inp.numel()
    _check(lib.arx_allreduce(_buf(inp, n, "inp"), _buf(out, n, "out"), n, _stream(stream)))


def reduce(inp, out, par: int, n: int = None, stream=None):
    if n is None:
        n = inp.numel()
    _check(lib.arx_reduce(_buf(inp, n, "inp"), _buf(out, n, "out"), n, par, _stream(stream)))


def _tag_bufs(tags, seen, rounds: int, nblocks: int):
    """Addresses of a tag check's buffers: tags u32 [W, rounds, nblocks] and
    seen u32 [W, rounds, nblocks, W], both given or neither."""
    if tags is None and seen is None:
        return None, None
    if tags is None or seen is None:
        raise ArxError(EINVAL, "tags and seen go together")
    W = world()
    return _buf(tags, W * rounds * nblocks, "tags", 4), _buf(seen, W * rounds * nblocks * W, "seen", 4)


def barrier_blockwise(nblocks: int, sem: int = SEM_ACQ_REL, rounds: int = 1, flags: int = 0, tags=None, seen=None,
                      stream=None):
    """W * nblocks workgroups (or nblocks with flags=BARRIER_LANES) pass the
    blockwise barrier `rounds` times; tags / seen: int32 device tensors for
    the tag check (arx.h, barrier tags)."""
    tp, sp = _tag_bufs(tags, seen, rounds, nblocks)
    _check(lib.arx_barrier_blockwise(nblocks, sem, rounds, flags, tp, sp, _stream(stream)))


def counter_barrier(nblocks: int, rounds: int = 1, flags: int = 0, epochs_seen=None, tags=None, seen=None,
                    stream=None):
    """epochs_seen: optional int32 device tensor [W, nblocks] receiving each
    rank's block's epoch; tags / seen as for barrier_blockwise."""
    ptr = None if epochs_seen is None else _buf(epochs_seen, world() * nblocks, "epochs_seen", 4)
    tp, sp = _tag_bufs(tags, seen, rounds, nblocks)
    _check(lib.arx_counter_barrier(nblocks, rounds, flags, ptr, tp, sp, _stream(stream)))


def symm_allreduce_noalloc(world_size: int, inputs, outputs, n: int, iters: int, status=None, stream=None):
    """The symmetric exchange with no allocation and no library instance:
    inputs / outputs bf16 device tensors [iters, W, ld]; status: optional
    int32 device tensor of one element, set to 1 on a timeout."""
    ld = inputs.shape[-1]
    if tuple(outputs.shape[-1:]) != (ld,):
        raise ArxError(EINVAL, "inputs and outputs must have the same last dimension")
    need = iters * world_size * ld
    sp = None if status is None else _buf(status, 1, "status", 4)
    _check(lib.arx_symm_allreduce_noalloc(world_size, _buf(inputs, need, "inputs"), _buf(outputs, need, "outputs"),
                                          n, ld, iters, sp, _stream(stream)))


def barrier_max_blocks() -> int:
    """Largest nblocks of a barrier launch with one workgroup per rank and block."""
    return _check(lib.arx_barrier_max_blocks())


def symm_allreduce(inputs, outputs, n: int, iters: int, stream=None):
    """inputs / outputs: bf16 device tensors [iters, W, ld] (ld >= n, ld % 8 == 0)."""
    ld = inputs.shape[-1]
    if tuple(outputs.shape[-1:]) != (ld,):
        raise ArxError(EINVAL, "inputs and outputs must have the same last dimension")
    need = iters * world() * ld
    _check(lib.arx_symm_allreduce(_buf(inputs, need, "inputs"), _buf(outputs, need, "outputs"), n, ld, iters,
                                  _stream(stream)))


def sem_view(rank: int):
    """int32 tensor viewing rank `rank`'s semaphores, shape [MAX_PAD_BLOCKS, 32]
    (flag in column 0, base in column 1; the split design's end-stage flag in
    column 16, its base in column 17)."""
    return _view(lib.arx_sem_ptr(rank), MAX_PAD_BLOCKS * 32, "<i4", None).view(MAX_PAD_BLOCKS, 32)


def epoch_view(rank: int):
    """int32 tensor viewing rank `rank`'s per-block epochs, shape [MAX_PAD_BLOCKS]."""
    return _view(lib.arx_epoch_ptr(rank), MAX_PAD_BLOCKS, "<i4", None)


def set_proxy_mode(mode: int):
    _check(lib.arx_set_proxy_mode(mode))


def set_stress_source(pool, sets: int):
    """pool: bf16 device tensor [sets, W, max_n] (kept alive by the caller);
    None (or sets 0) clears the source."""
    ptr = None if pool is None or sets == 0 else _buf(pool, max(sets, 0) * world() * max_n(), "pool")
    _check(lib.arx_set_stress_source(ptr, sets))


def set_timeout_us(us: int):
    _check(lib.arx_set_timeout_us(us))


def status():
    a, b, c = ctypes.c_uint64(), ctypes.c_uint64(), ctypes.c_uint64()
    _check(lib.arx_status(ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)))
    return a.value, b.value, c.value


def debug_state() -> dict:
    buf = (ctypes.c_uint64 * 32)()
    m = _check(lib.arx_debug_state(buf, 32))
    d = {name: buf[i] for i, name in enumerate(STATE_WORDS)}
    d["flags"] = [buf[i] for i in range(len(STATE_WORDS), m)]
    return d


def debug_set_seq(seq: int):
    _check(lib.arx_debug_set_seq(seq))


def debug_fail_proxy():
    _check(lib.arx_debug_fail_proxy())


def max_n() -> int:
    return lib.arx_max_n()


def world() -> int:
    return lib.arx_world()


def test_round_bf16(inp_u32, out_u16, stream=None):
    n = inp_u32.numel()
    _check(lib.arx_test_round_bf16(_buf(inp_u32, n, "inp_u32", 4), _buf(out_u16, n, "out_u16"), n,
                                   _stream(stream)))


def test_oneshot_shape(n, world=8, block=0, resident=257, in_place=False) -> dict:
    out = (_c.c_int * 8)()
    _check(lib.arx_test_oneshot_shape(n, world, block, resident, 1 if in_place else 0, out, 8))
    return dict(zip(("block", "grid", "launched", "ncopy", "one_pass", "early_go", "nt_copy", "nt_peer"), list(out)))


class _DevArray:
    """__cuda_array_interface__ view of library-owned device memory."""

    def __init__(self, ptr, n, typestr):
        self.__cuda_array_interface__ = {"shape": (n,), "typestr": typestr, "data": (ptr, False),
                                         "version": 2, "strides": None}


def _view(ptr, n, typestr, dtype):
    import torch
    if not ptr:
        raise ArxError(EINVAL, "null slot (library not initialised or index out of range)")
    t = torch.as_tensor(_DevArray(ptr, n, typestr), device="cuda")
    return t.view(dtype) if dtype is not None else t


def _slot_len(n):
    m = max_n()
    if n is None:
        return m
    if not 0 < n <= m:
        raise ArxError(EINVAL, f"a slot view holds 1 to max_n = {m} elements, not {n}")
    return n


def recv_view(par: int, src: int, n: int = None):
    """bf16 tensor viewing recv slot [par][src] (library memory, no copy)."""
    import torch
    return _view(lib.arx_recv_ptr(par, src), _slot_len(n), "<i2", torch.bfloat16)


def send_view(par: int, n: int = None):
    import torch
    return _view(lib.arx_send_ptr(par), _slot_len(n), "<i2", torch.bfloat16)


def pad_view(rank: int):
    """int32 tensor viewing virtual rank `rank`'s pad, shape [MAX_PAD_BLOCKS, W]."""
    W = world()
    return _view(lib.arx_pad_ptr(rank), MAX_PAD_BLOCKS * W, "<i4", None).view(MAX_PAD_BLOCKS, W)


# ---- layer operators ---------------------------------------------------------
#
# Planes are 2-D tensors whose rows are contiguous (stride(1) == 1, any row
# stride); vectors are contiguous. Outputs that the caller does not pass, and
# workspaces, come from torch's allocator on the stream of the call.


class _Call:
    """One call's first tensor, type, GPU and stream, and the checks of its
    other tensors. It costs host time on every call, so it asks each tensor
    as little as it can."""

    __slots__ = ("first", "dtype", "device", "code", "stream", "alloc")

    def __init__(self, first, what, dtypes, stream):
        if not getattr(first, "is_cuda", False):
            raise ArxError(EINVAL, f"{what} must be a GPU tensor")
        self.first, self.dtype, self.device = first, first.dtype, first.get_device()
        self.code = dtypes.get(self.dtype)
        if self.code is None:
            raise ArxError(EINVAL, f"{what} is {self.dtype}, not one of {[str(d) for d in dtypes]}")
        if self.device != _current_device():
            raise ArxError(EINVAL, f"{what} is on GPU {self.device}, not on the current one")
        if stream is None:
            self.stream, self.alloc = _current_stream(self.device), None
        else:
            self.stream = _stream(stream)
            self.alloc = torch.cuda.ExternalStream(self.stream)

    def plane(self, t, what, shape=None):
        """(address, row stride) of a 2-D tensor of the call's type."""
        if t is None:
            return None, 0
        if t.dtype != self.dtype:
            raise ArxError(EINVAL, f"{what} is {t.dtype}, not {self.dtype}")
        if t.get_device() != self.device:
            raise ArxError(EINVAL, f"{what} must be a tensor on the call's GPU")
        size, strides = t.shape, t.stride()
        if len(strides) != 2 or (shape is not None and size != shape):
            raise ArxError(EINVAL, f"{what} has shape {tuple(size)}, not " +
                           ("two dimensions" if shape is None else f"{tuple(shape)}"))
        rows, cols = size
        ld = strides[0]
        if (strides[1] != 1 and cols > 1) or (ld < cols and rows > 1):
            raise ArxError(EINVAL, f"{what} has strides {strides}: its rows must be contiguous and apart")
        return t.data_ptr(), ld if rows > 1 else max(ld, cols)

    def vector(self, t, what, n, dtype=None):
        """Address of a contiguous vector of n elements."""
        if t is None:
            return None
        if t.dtype != (dtype or self.dtype):
            raise ArxError(EINVAL, f"{what} is {t.dtype}, not {dtype or self.dtype}")
        if t.get_device() != self.device:
            raise ArxError(EINVAL, f"{what} must be a tensor on the call's GPU")
        size = t.shape
        if len(size) != 1 or size[0] != n or (n > 1 and t.stride(0) != 1):
            raise ArxError(EINVAL, f"{what} has shape {tuple(size)} and strides {t.stride()}, not ({n},) and (1,)")
        return t.data_ptr()

    def empty(self, shape, dtype=None):
        if self.alloc is None:
            return self.first.new_empty(shape, dtype=dtype)
        with torch.cuda.stream(self.alloc):   # its memory is reused in that stream's order
            return self.first.new_empty(shape, dtype=dtype)

    def workspace(self, nbytes):
        """(tensor, address); the tensor lives until the call has been queued."""
        if nbytes == 0:
            return None, None
        t = self.empty(nbytes, torch.uint8)
        return t, t.data_ptr()


def _norm_types(weight, shift, dtype):
    """Type and code of a norm's weight and shift: the rows' or float32."""
    given = weight if weight is not None else shift
    wdtype = dtype if given is None else given.dtype
    if wdtype != dtype and wdtype != torch.float32:
        raise ArxError(EINVAL, f"weight is {wdtype}, not {dtype} or torch.float32")
    return wdtype, _TYPES[wdtype]


def _act(act):
    if act not in ACTS:
        raise ArxError(EINVAL, f"act {act!r} is not one of {sorted(ACTS)}")
    return ACTS[act]


def _on_lines(p, ld):
    """Rows that all start on 16-byte boundaries (arx.h, arx_linear)."""
    return not p & 15 and not ld & 7 and ld < 1 << 22


def linear(x, w, bias=None, residual=None, act="none", save_z=False, out=None, stream=None):
    """y = act(z) + residual with z = x w^T + bias; x [m, k], w [n, k], bias
    [n], residual [m, n], all bf16 or all f16. Returns y, or (y, z) with
    save_z (what linear_backward needs unless act is "none"). out: a plane for
    y; residual itself will do."""
    c = _Call(x, "x", _MATRIX_TYPES, stream)
    kind = _act(act)
    xp, ldx = c.plane(x, "x")
    wp, ldw = c.plane(w, "w")
    m, k = x.shape
    n = w.shape[0]
    if w.shape[1] != k:
        raise ArxError(EINVAL, f"w has shape {tuple(w.shape)} for rows of {k}")
    rp, ldr = c.plane(residual, "residual", (m, n))
    if out is None:
        out = c.empty((m, n))
    yp, ldy = c.plane(out, "out", (m, n))
    z = c.empty((m, n)) if save_z else None
    space = lib.arx_linear_workspace(m, n, k, _on_lines(xp, ldx) and _on_lines(wp, ldw))
    hold, space_p = c.workspace(space)
    _check(lib.arx_linear(xp, wp, c.vector(bias, "bias", n), rp, yp, z.data_ptr() if save_z else None, m, n, k, ldx,
                          ldw, ldr, ldy, n, kind, c.code, space_p, space, c.stream))
    return (out, z) if save_z else out


def linear_backward(dy, x, w, z=None, act="none", dx=True, dw=True, dbias=False, stream=None):
    """Gradients of linear: (dx, dw, dbias), None for those not asked for. z
    is what linear gave with save_z. The residual's gradient is dy."""
    c = _Call(dy, "dy", _MATRIX_TYPES, stream)
    kind = _act(act)
    dyp, lddy = c.plane(dy, "dy")
    m, n = dy.shape
    xp, ldx = c.plane(x, "x")
    wp, ldw = c.plane(w, "w")
    k = w.shape[1]
    if x.shape != (m, k) or w.shape[0] != n:
        raise ArxError(EINVAL, f"dy {tuple(dy.shape)}, x {tuple(x.shape)} and w {tuple(w.shape)} do not belong together")
    if z is None and kind:
        raise ArxError(EINVAL, f"act {act!r} needs z")
    zp, ldz = c.plane(z, "z", (m, n)) if kind else (None, 0)
    gx = c.empty((m, k)) if dx else None
    gw = c.empty((n, k)) if dw else None
    gb = c.empty(n) if dbias else None
    space = lib.arx_linear_backward_workspace(
        m, n, k, kind, _on_lines(dyp, lddy) and _on_lines(xp, ldx) and _on_lines(wp, ldw))
    hold, space_p = c.workspace(space)
    _check(lib.arx_linear_backward(dyp, xp, wp, zp, _ptr(gx), _ptr(gw), _ptr(gb), m, n, k, lddy, ldx, ldw, ldz, k, k,
                                   kind, c.code, space_p, space, c.stream))
    return gx, gw, gb


def layer_norm(x, weight=None, shift=None, eps=1e-5, out=None, stream=None):
    """Layer norm over each row of x [rows, cols]: (y, mean, rstd), the last
    two float32 [rows] for layer_norm_backward. weight, shift [cols]: x's type
    or float32. out: a plane for y; x itself will do."""
    c = _Call(x, "x", _TYPES, stream)
    xp, ldx = c.plane(x, "x")
    rows, cols = x.shape
    wdtype, wcode = _norm_types(weight, shift, c.dtype)
    if out is None:
        out = c.empty((rows, cols))
    yp, ldy = c.plane(out, "out", (rows, cols))
    mean, rstd = c.empty((2, rows), torch.float32).unbind(0)
    _check(lib.arx_layer_norm(xp, c.vector(weight, "weight", cols, wdtype), c.vector(shift, "shift", cols, wdtype), yp,
                              mean.data_ptr(), rstd.data_ptr(), rows, cols, ldx, ldy, eps, c.code, wcode, c.stream))
    return out, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, weight=None, stream=None):
    """Gradients of layer_norm: (dx, dweight, dshift); the last two in
    weight's type, or dy's without one."""
    c = _Call(dy, "dy", _TYPES, stream)
    dyp, lddy = c.plane(dy, "dy")
    rows, cols = dy.shape
    xp, ldx = c.plane(x, "x", (rows, cols))
    wdtype, wcode = _norm_types(weight, None, c.dtype)
    dx = c.empty((rows, cols))
    dw, db = c.empty(cols, wdtype), c.empty(cols, wdtype)
    space = lib.arx_rows_workspace(rows, cols, 2)
    hold, space_p = c.workspace(space)
    _check(lib.arx_layer_norm_backward(dyp, xp, c.vector(mean, "mean", rows, torch.float32),
                                       c.vector(rstd, "rstd", rows, torch.float32),
                                       c.vector(weight, "weight", cols, wdtype), dx.data_ptr(), dw.data_ptr(),
                                       db.data_ptr(), rows, cols, lddy, ldx, cols, c.code, wcode, space_p, space,
                                       c.stream))
    return dx, dw, db


def _seed(seed, offset):
    if not 0 <= seed < 1 << 64 or not 0 <= offset < 1 << 64:
        raise ArxError(EINVAL, f"seed {seed} and offset {offset} must be unsigned 64-bit numbers")


def dropout_add(x, residual=None, bias=None, p=0.0, seed=0, offset=0, out=None, stream=None):
    """residual + dropout(x + bias), the mask drawn from (seed, offset) and the
    element's place (arx.h, arx_dropout_add) and never stored. out: a plane;
    x or residual itself will do."""
    c = _Call(x, "x", _TYPES, stream)
    xp, ldx = c.plane(x, "x")
    rows, cols = x.shape
    rp, ldr = c.plane(residual, "residual", (rows, cols))
    _seed(seed, offset)
    if out is None:
        out = c.empty((rows, cols))
    hp, ldh = c.plane(out, "out", (rows, cols))
    _check(lib.arx_dropout_add(xp, c.vector(bias, "bias", cols), rp, hp, rows, cols, ldx, ldr, ldh, p, seed, offset,
                               c.code, c.stream))
    return out


def dropout_add_backward(dh, p=0.0, seed=0, offset=0, dbias=False, stream=None):
    """Gradients of dropout_add: (dx, dbias), dbias None unless asked for. The
    residual's gradient is dh."""
    c = _Call(dh, "dh", _TYPES, stream)
    dhp, lddh = c.plane(dh, "dh")
    rows, cols = dh.shape
    _seed(seed, offset)
    dx = c.empty((rows, cols))
    db = c.empty(cols) if dbias else None
    space = lib.arx_rows_workspace(rows, cols, 1) if dbias else 0
    hold, space_p = c.workspace(space)
    _check(lib.arx_dropout_add_backward(dhp, dx.data_ptr(), _ptr(db), rows, cols, lddh, cols, p, seed, offset, c.code,
                                        space_p, space, c.stream))
    return dx, db


def dropout_add_norm(x, residual=None, weight=None, shift=None, bias=None, p=0.0, seed=0, offset=0, eps=1e-5,
                     out=None, stream=None):
    """h = residual + dropout(x + bias) and its layer norm in one pass:
    (h, y, mean, rstd). out: a plane for h; x or residual itself will do."""
    c = _Call(x, "x", _TYPES, stream)
    xp, ldx = c.plane(x, "x")
    rows, cols = x.shape
    rp, ldr = c.plane(residual, "residual", (rows, cols))
    wdtype, wcode = _norm_types(weight, shift, c.dtype)
    _seed(seed, offset)
    h = c.empty((rows, cols)) if out is None else out
    hp, ldh = c.plane(h, "out", (rows, cols))
    y = c.empty((rows, cols))
    mean, rstd = c.empty((2, rows), torch.float32).unbind(0)
    _check(lib.arx_dropout_add_norm(xp, c.vector(bias, "bias", cols), rp, c.vector(weight, "weight", cols, wdtype),
                                    c.vector(shift, "shift", cols, wdtype), hp, y.data_ptr(), mean.data_ptr(),
                                    rstd.data_ptr(), rows, cols, ldx, ldr, ldh, cols, eps, p, seed, offset, c.code,
                                    wcode, c.stream))
    return h, y, mean, rstd


def dropout_add_norm_backward(dy, dh, h, mean, rstd, weight=None, p=0.0, seed=0, offset=0, dbias=False, stream=None):
    """Gradients of dropout_add_norm from y's (dy) and from h's other users
    (dh, or None): (dx, dresidual, dbias, dweight, dshift), dbias None unless
    asked for."""
    c = _Call(dy, "dy", _TYPES, stream)
    dyp, lddy = c.plane(dy, "dy")
    rows, cols = dy.shape
    dhp, lddh = c.plane(dh, "dh", (rows, cols))
    hp, ldh = c.plane(h, "h", (rows, cols))
    wdtype, wcode = _norm_types(weight, None, c.dtype)
    _seed(seed, offset)
    dx, dr = c.empty((rows, cols)), c.empty((rows, cols))
    db = c.empty(cols) if dbias else None
    dw, ds = c.empty(cols, wdtype), c.empty(cols, wdtype)
    space = lib.arx_rows_workspace(rows, cols, 3)
    hold, space_p = c.workspace(space)
    _check(lib.arx_dropout_add_norm_backward(dyp, dhp, hp, c.vector(mean, "mean", rows, torch.float32),
                                             c.vector(rstd, "rstd", rows, torch.float32),
                                             c.vector(weight, "weight", cols, wdtype), dx.data_ptr(), dr.data_ptr(),
                                             _ptr(db), dw.data_ptr(), ds.data_ptr(), rows, cols, lddy, lddh, ldh, cols,
                                             cols, p, seed, offset, c.code, wcode, space_p, space, c.stream))
    return dx, dr, db, dw, ds
