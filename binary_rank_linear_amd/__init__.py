"""Python binding of libblr.so, the MI355X (gfx950) binary low-rank (`blr`)
linear layer (C ABI in include/blr.h).

Argument marshalling only: every step of the layer runs in the HIP kernels
behind the C ABI. PyTorch supplies device memory and the current stream.
There is no fallback: if the library is missing or the device is not
gfx950, the calls raise.

The functions carry the C names: `blr_expand_signs`, `blr_forward`,
`blr_forward_noalloc`, `blr_backward`, `blr_backward_signs`, `blr_plane_linear`, `blr_sumsq`, `blr_workspace_bytes`,
the token routing (`blr_route_sort`, `blr_route_gather`, `blr_route_combine`, `blr_route_combine_backward`) and the
low-rank adapters beside a layer (`blr_adapters_forward`, `blr_adapters_backward`), the norms around a block
(`blr_norm_forward`, `blr_norm_backward`), the gated feed-forward (`blr_gated_forward`, `blr_gated_backward`) and rows
kept in 8 bits (`blr_checkpoint_save`, `blr_checkpoint_load`), plus the profiling calls;
`all_finite` and `next_gscale` are the host side
of the finite check and the power-of-two loss scale.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libblr.so")
_lib = None


class BlrError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def load():
    """Load libblr.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m binary_rank_linear_amd.build`")
    # torch brings a HIP runtime of its own. The library has to find that one in the process: loaded first it would
    # bring the system's, and torch's streams and memory mean nothing to another runtime.
    with contextlib.suppress(ImportError):  # without torch there is one runtime, and the calls on sizes still work
        import torch  # noqa: F401
    lib = ctypes.CDLL(LIB_PATH)
    i64, p, i32, f32, sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.blr_status_string.argtypes = [i32]
    lib.blr_status_string.restype = ctypes.c_char_p
    lib.blr_device_supported.argtypes = [i32]
    lib.blr_device_supported.restype = i32
    lib.blr_workspace_bytes.argtypes = [i64, i64, i64, i64]
    lib.blr_workspace_bytes.restype = sz
    lib.blr_expand_signs.argtypes = [p, i64, i64, p, p, p]
    lib.blr_expand_signs.restype = i32
    lib.blr_forward.argtypes = [i64, i64, i64, i64, p, p, p, p, p, p, p, i32, p, p, p, sz, p]
    lib.blr_forward.restype = i32
    lib.blr_forward_noalloc.argtypes = [i64, i64, i64, i64, p, p, p, p, p, p, p, i32, p, p, p]
    lib.blr_forward_noalloc.restype = i32
    lib.blr_backward.argtypes = [i64, i64, i64, i64, p, p, p, p, p, p, p, p, p, f32, p, p, p, p, i32, p, sz, p]
    lib.blr_backward.restype = i32
    lib.blr_backward_signs.argtypes = [i64, i64, i64, i64, p, p, p, p, p, p, p, p, p, f32, p, p, p, p, i32, p, p, i32,
                                       p, sz, p]
    lib.blr_backward_signs.restype = i32
    lib.blr_workspace_bytes_paths.argtypes = [i64, i64, i64, i64, i64]
    lib.blr_workspace_bytes_paths.restype = sz
    lib.blr_forward_paths.argtypes = [i64, i64, i64, i64, i64, p, p, p, p, p, p, p, i32, p, p, sz, p]
    lib.blr_forward_paths.restype = i32
    lib.blr_backward_paths.argtypes = [i64, i64, i64, i64, i64, p, p, p, p, p, p, p, p, f32, p, p, p, p, i32, p, p,
                                       i32, p, sz, p]
    lib.blr_backward_paths.restype = i32
    lib.blr_plane_linear.argtypes = [i64, i64, i64, p, p, p, f32, p]
    lib.blr_plane_linear.restype = i32
    lib.blr_sumsq.argtypes = [p, i64, p, i32, p]
    lib.blr_sumsq.restype = i32
    lib.blr_route_workspace_bytes.argtypes = [i64, i64]
    lib.blr_route_workspace_bytes.restype = sz
    lib.blr_route_sort.argtypes = [i64, i64, p, p, p, p, p, sz, p]
    lib.blr_route_sort.restype = i32
    lib.blr_route_gather.argtypes = [i64, i64, i64, i64, i32, p, p, p, p, p]
    lib.blr_route_gather.restype = i32
    lib.blr_route_combine.argtypes = [i64, i64, i64, i64, i32, p, p, p, p, p, i32, p]
    lib.blr_route_combine.restype = i32
    lib.blr_route_combine_backward.argtypes = [i64, i64, i64, i64, i32, p, p, p, p, p, p, p, p]
    lib.blr_route_combine_backward.restype = i32
    lib.blr_adapters_workspace_bytes.argtypes = [i64, i64, i64, i64, i64]
    lib.blr_adapters_workspace_bytes.restype = sz
    lib.blr_adapters_forward_workspace_bytes.argtypes = [i64, i64, i64, i64, i64]
    lib.blr_adapters_forward_workspace_bytes.restype = sz
    lib.blr_adapters_forward.argtypes = [i64, i64, i64, i64, i64, i32, i32, p, p, p, p, p, p, p, i32, p, p, sz, p]
    lib.blr_adapters_forward.restype = i32
    lib.blr_adapters_backward.argtypes = [i64, i64, i64, i64, i64, i32, i32, p, p, p, p, p, p, p, p, p, p, i32, p, i32,
                                          p, sz, p]
    lib.blr_adapters_backward.restype = i32
    lib.blr_checkpoint_save.argtypes = [i64, i64, i32, p, p, p, p]
    lib.blr_checkpoint_save.restype = i32
    lib.blr_checkpoint_load.argtypes = [i64, i64, i32, p, p, p, p]
    lib.blr_checkpoint_load.restype = i32
    lib.blr_norm_forward.argtypes = [i64, i64, i32, i32, i32, p, p, i32, p, p, i32, i64, f32, f32, p, f32, p, p, p, p, p,
                                     p]
    lib.blr_norm_forward.restype = i32
    lib.blr_norm_workspace_bytes.argtypes = [i64, i64, i64]
    lib.blr_norm_workspace_bytes.restype = sz
    lib.blr_norm_backward.argtypes = [i64, i64, i32, i32, i32, p, p, p, p, p, i32, p, p, p, i32, p, p, i32, i64, f32,
                                      f32, p, p, p, p, p, p, p, i32, p, sz, p]
    lib.blr_norm_backward.restype = i32
    lib.blr_gated_forward.argtypes = [i64, i64, i64, i32, i32, p, p, p, i32, p, p, p, p]
    lib.blr_gated_forward.restype = i32
    lib.blr_gated_workspace_bytes.argtypes = [i64, i64, i64]
    lib.blr_gated_workspace_bytes.restype = sz
    lib.blr_gated_backward.argtypes = [i64, i64, i64, i32, i32, i32, p, p, p, p, p, p, i32, p, p, f32, p, i32, p, p, i32,
                                       p, sz, p]
    lib.blr_gated_backward.restype = i32
    lib.blr_profile_enable.argtypes = [i32]
    lib.blr_profile_enable.restype = i32
    lib.blr_profile_read.argtypes = [ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(i64),
                                     ctypes.POINTER(ctypes.c_double), i32]
    lib.blr_profile_read.restype = i32
    lib.blr_profile_reset.argtypes = []
    lib.blr_profile_reset.restype = i32
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().blr_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != 0:
        raise BlrError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t, name, dtypes, shape=None):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU device")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def _bits_dtypes():
    import torch
    return (torch.int32, getattr(torch, "uint32", torch.int32))


def device_supported(device: int = 0) -> bool:
    return bool(load().blr_device_supported(int(device)))


def blr_workspace_bytes(M: int, d_in: int, d_out: int, r: int) -> int:
    return int(load().blr_workspace_bytes(M, d_in, d_out, r))


def workspace(M: int, d_in: int, d_out: int, r: int, device=None):
    import torch
    n = blr_workspace_bytes(M, d_in, d_out, r)
    if n == 0:
        raise BlrError(-2, "blr_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def blr_expand_signs(bits, rows: int, r: int, plane=True, plane_t=True, stream=None):
    """Expand a sign bitmap [rows][ceil(r/32)] into f16 planes. `plane` /
    `plane_t` are output tensors (f16 [rows][r] / [r][rows]), True to
    allocate, or None to skip. Returns (plane, plane_t)."""
    import torch
    W = (r + 31) // 32
    _need(bits, "bits", _bits_dtypes(), (rows, W))
    if plane is True:
        plane = torch.empty((rows, r), dtype=torch.float16, device=bits.device)
    if plane_t is True:
        plane_t = torch.empty((r, rows), dtype=torch.float16, device=bits.device)
    if plane is not None:
        _need(plane, "plane", (torch.float16, torch.int16), (rows, r))
    if plane_t is not None:
        _need(plane_t, "plane_t", (torch.float16, torch.int16), (r, rows))
    _check(load().blr_expand_signs(_ptr(bits), rows, r, _ptr(plane), _ptr(plane_t), _stream(stream)),
           "blr_expand_signs")
    return plane, plane_t


def blr_forward(x, bits_u, bits_v, h, l, g, *, y=None, accumulate_y=False, tape_a=None, tape_c=None,
                keep_c=False, ws=None, stream=None):
    """Forward of one path. Returns (y, tape_a, tape_c); outputs not given
    are allocated. y is overwritten unless accumulate_y. The c tape is kept
    only when tape_c is given or keep_c is set; otherwise tape_c is None and
    blr_backward recomputes c."""
    import torch
    f32 = (torch.float32,)
    M, d_in = _need(x, "x", f32).shape
    d_out, r = _need(h, "h", f32).shape[0], _need(l, "l", f32).shape[0]
    _need(g, "g", f32, (d_in,))
    W = (r + 31) // 32
    _need(bits_u, "bits_u", _bits_dtypes(), (d_out, W))
    _need(bits_v, "bits_v", _bits_dtypes(), (d_in, W))
    dev = x.device
    y = torch.empty((M, d_out), dtype=torch.float32, device=dev) if y is None else _need(y, "y", f32, (M, d_out))
    tape_a = torch.empty((M, r), dtype=torch.float32, device=dev) if tape_a is None else \
        _need(tape_a, "tape_a", f32, (M, r))
    if tape_c is None and keep_c:
        tape_c = torch.empty((M, d_out), dtype=torch.float32, device=dev)
    if tape_c is not None:
        _need(tape_c, "tape_c", f32, (M, d_out))
    if ws is None:
        ws = workspace(M, d_in, d_out, r, dev)
    _check(load().blr_forward(M, d_in, d_out, r, _ptr(x), _ptr(bits_u), _ptr(bits_v), _ptr(h), _ptr(l), _ptr(g),
                              _ptr(y), int(bool(accumulate_y)), _ptr(tape_a), _ptr(tape_c), _ptr(ws), ws.numel(),
                              _stream(stream)), "blr_forward")
    return y, tape_a, tape_c


# bytes of the allocation-free forward's scratch (BLR_NOALLOC_SCRATCH_BYTES):
# it serves sizes with r * d_in / 8 up to this
NOALLOC_SCRATCH_BYTES = 4 << 20


def blr_forward_noalloc(x, bits_u, bits_v, h, l, g, y, tape_a, *, accumulate_y=False, tape_c=None, stream=None):
    """blr_forward without a workspace and without allocating: every output
    (y, tape_a, and tape_c if kept) is the caller's; the library's own
    per-GPU scratch holds the transposed bitmap. Calls that overlap on one
    GPU race. Returns (y, tape_a, tape_c)."""
    import torch
    f32 = (torch.float32,)
    M, d_in = _need(x, "x", f32).shape
    d_out, r = _need(h, "h", f32).shape[0], _need(l, "l", f32).shape[0]
    _need(g, "g", f32, (d_in,))
    W = (r + 31) // 32
    _need(bits_u, "bits_u", _bits_dtypes(), (d_out, W))
    _need(bits_v, "bits_v", _bits_dtypes(), (d_in, W))
    _need(y, "y", f32, (M, d_out))
    _need(tape_a, "tape_a", f32, (M, r))
    if tape_c is not None:
        _need(tape_c, "tape_c", f32, (M, d_out))
    _check(load().blr_forward_noalloc(M, d_in, d_out, r, _ptr(x), _ptr(bits_u), _ptr(bits_v), _ptr(h), _ptr(l),
                                      _ptr(g), _ptr(y), int(bool(accumulate_y)), _ptr(tape_a), _ptr(tape_c),
                                      _stream(stream)), "blr_forward_noalloc")
    return y, tape_a, tape_c


def blr_backward(x, dy, bits_u, bits_v, h, l, g, tape_a, tape_c, gscale: float, *, dh=None, dl=None, dg=None,
                 dx=None, accumulate_dx=False, ws=None, stream=None):
    """Backward of one path. dh/dl/dg accumulate (allocated as zeros when not
    given); dx is overwritten unless accumulate_dx. tape_c is the forward's
    c tape, or None when the forward kept none. Returns (dh, dl, dg, dx)."""
    import torch
    f32 = (torch.float32,)
    M, d_in = _need(x, "x", f32).shape
    d_out, r = _need(h, "h", f32).shape[0], _need(l, "l", f32).shape[0]
    _need(g, "g", f32, (d_in,))
    _need(dy, "dy", f32, (M, d_out))
    W = (r + 31) // 32
    _need(bits_u, "bits_u", _bits_dtypes(), (d_out, W))
    _need(bits_v, "bits_v", _bits_dtypes(), (d_in, W))
    _need(tape_a, "tape_a", f32, (M, r))
    if tape_c is not None:
        _need(tape_c, "tape_c", f32, (M, d_out))
    dev = x.device
    dh = torch.zeros(d_out, dtype=torch.float32, device=dev) if dh is None else _need(dh, "dh", f32, (d_out,))
    dl = torch.zeros(r, dtype=torch.float32, device=dev) if dl is None else _need(dl, "dl", f32, (r,))
    dg = torch.zeros(d_in, dtype=torch.float32, device=dev) if dg is None else _need(dg, "dg", f32, (d_in,))
    dx = torch.empty((M, d_in), dtype=torch.float32, device=dev) if dx is None else _need(dx, "dx", f32, (M, d_in))
    if ws is None:
        ws = workspace(M, d_in, d_out, r, dev)
    _check(load().blr_backward(M, d_in, d_out, r, _ptr(x), _ptr(dy), _ptr(bits_u), _ptr(bits_v), _ptr(h), _ptr(l),
                               _ptr(g), _ptr(tape_a), _ptr(tape_c), ctypes.c_float(gscale), _ptr(dh), _ptr(dl),
                               _ptr(dg), _ptr(dx), int(bool(accumulate_dx)), _ptr(ws), ws.numel(), _stream(stream)),
           "blr_backward")
    return dh, dl, dg, dx


def blr_backward_signs(x, dy, bits_u, bits_v, h, l, g, tape_a, tape_c, gscale: float, *, dh=None, dl=None, dg=None,
                       dx=None, accumulate_dx=False, grad_u=None, grad_v=None, accumulate_signs=False, ws=None,
                       stream=None):
    """blr_backward plus the sign gradients G_U [d_out][r] and G_V [d_in][r]
    (allocated when not given; overwritten unless accumulate_signs).
    Returns (dh, dl, dg, dx, grad_u, grad_v)."""
    import torch
    f32 = (torch.float32,)
    M, d_in = _need(x, "x", f32).shape
    d_out, r = _need(h, "h", f32).shape[0], _need(l, "l", f32).shape[0]
    _need(g, "g", f32, (d_in,))
    _need(dy, "dy", f32, (M, d_out))
    W = (r + 31) // 32
    _need(bits_u, "bits_u", _bits_dtypes(), (d_out, W))
    _need(bits_v, "bits_v", _bits_dtypes(), (d_in, W))
    _need(tape_a, "tape_a", f32, (M, r))
    if tape_c is not None:
        _need(tape_c, "tape_c", f32, (M, d_out))
    dev = x.device
    dh = torch.zeros(d_out, dtype=torch.float32, device=dev) if dh is None else _need(dh, "dh", f32, (d_out,))
    dl = torch.zeros(r, dtype=torch.float32, device=dev) if dl is None else _need(dl, "dl", f32, (r,))
    dg = torch.zeros(d_in, dtype=torch.float32, device=dev) if dg is None else _need(dg, "dg", f32, (d_in,))
    dx = torch.empty((M, d_in), dtype=torch.float32, device=dev) if dx is None else _need(dx, "dx", f32, (M, d_in))
    grad_u = torch.empty((d_out, r), dtype=torch.float32, device=dev) if grad_u is None else \
        _need(grad_u, "grad_u", f32, (d_out, r))
    grad_v = torch.empty((d_in, r), dtype=torch.float32, device=dev) if grad_v is None else \
        _need(grad_v, "grad_v", f32, (d_in, r))
    if ws is None:
        ws = workspace(M, d_in, d_out, r, dev)
    _check(load().blr_backward_signs(M, d_in, d_out, r, _ptr(x), _ptr(dy), _ptr(bits_u), _ptr(bits_v), _ptr(h),
                                     _ptr(l), _ptr(g), _ptr(tape_a), _ptr(tape_c), ctypes.c_float(gscale), _ptr(dh),
                                     _ptr(dl), _ptr(dg), _ptr(dx), int(bool(accumulate_dx)), _ptr(grad_u),
                                     _ptr(grad_v), int(bool(accumulate_signs)), _ptr(ws), ws.numel(),
                                     _stream(stream)), "blr_backward_signs")
    return dh, dl, dg, dx, grad_u, grad_v


def blr_workspace_bytes_paths(M: int, d_in: int, d_out: int, r: int, paths: int) -> int:
    return int(load().blr_workspace_bytes_paths(M, d_in, d_out, r, paths))


def _paths_shapes(x, bits_u, bits_v, h, l, g):
    import torch
    f32 = (torch.float32,)
    M, d_in = _need(x, "x", f32).shape
    P, d_out = _need(h, "h", f32).shape
    r = _need(l, "l", f32, (P, l.shape[1])).shape[1]
    _need(g, "g", f32, (P, d_in))
    W = (r + 31) // 32
    _need(bits_u, "bits_u", _bits_dtypes(), (P, d_out, W))
    _need(bits_v, "bits_v", _bits_dtypes(), (P, d_in, W))
    return M, d_in, d_out, r, P


def blr_forward_paths(x, bits_u, bits_v, h, l, g, *, y=None, accumulate_y=False, tape_a=None, ws=None, stream=None):
    """Forward of a layer of P paths, fused: bits_u [P][d_out][W], bits_v
    [P][d_in][W], h [P][d_out], l [P][r], g [P][d_in]. y (+)= sum_p h_p.c_p;
    the a tape is [M][P r]. Returns (y, tape_a)."""
    import torch
    f32 = (torch.float32,)
    M, d_in, d_out, r, P = _paths_shapes(x, bits_u, bits_v, h, l, g)
    dev = x.device
    y = torch.empty((M, d_out), dtype=torch.float32, device=dev) if y is None else _need(y, "y", f32, (M, d_out))
    tape_a = torch.empty((M, P * r), dtype=torch.float32, device=dev) if tape_a is None else \
        _need(tape_a, "tape_a", f32, (M, P * r))
    if ws is None:
        ws = workspace_paths(M, d_in, d_out, r, P, dev)
    _check(load().blr_forward_paths(M, d_in, d_out, r, P, _ptr(x), _ptr(bits_u), _ptr(bits_v), _ptr(h), _ptr(l),
                                    _ptr(g), _ptr(y), int(bool(accumulate_y)), _ptr(tape_a), _ptr(ws), ws.numel(),
                                    _stream(stream)), "blr_forward_paths")
    return y, tape_a


def blr_backward_paths(x, dy, bits_u, bits_v, h, l, g, tape_a, gscale: float, *, dh=None, dl=None, dg=None, dx=None,
                       accumulate_dx=False, signs=False, grad_u=None, grad_v=None, accumulate_signs=False, ws=None,
                       stream=None):
    """Backward of a layer of P paths (blr_forward_paths' tape). dh [P][d_out],
    dl [P][r], dg [P][d_in] accumulate (zeros when not given); dx is
    overwritten unless accumulate_dx. With signs (or grad_u / grad_v given)
    also the sign gradients [P][d_out][r] and [P][d_in][r]. Returns
    (dh, dl, dg, dx, grad_u, grad_v), the last two None without signs."""
    import torch
    f32 = (torch.float32,)
    M, d_in, d_out, r, P = _paths_shapes(x, bits_u, bits_v, h, l, g)
    _need(dy, "dy", f32, (M, d_out))
    _need(tape_a, "tape_a", f32, (M, P * r))
    dev = x.device
    dh = torch.zeros((P, d_out), dtype=torch.float32, device=dev) if dh is None else _need(dh, "dh", f32, (P, d_out))
    dl = torch.zeros((P, r), dtype=torch.float32, device=dev) if dl is None else _need(dl, "dl", f32, (P, r))
    dg = torch.zeros((P, d_in), dtype=torch.float32, device=dev) if dg is None else _need(dg, "dg", f32, (P, d_in))
    dx = torch.empty((M, d_in), dtype=torch.float32, device=dev) if dx is None else _need(dx, "dx", f32, (M, d_in))
    if signs or grad_u is not None or grad_v is not None:
        grad_u = torch.empty((P, d_out, r), dtype=torch.float32, device=dev) if grad_u is None else \
            _need(grad_u, "grad_u", f32, (P, d_out, r))
        grad_v = torch.empty((P, d_in, r), dtype=torch.float32, device=dev) if grad_v is None else \
            _need(grad_v, "grad_v", f32, (P, d_in, r))
    if ws is None:
        ws = workspace_paths(M, d_in, d_out, r, P, dev)
    _check(load().blr_backward_paths(M, d_in, d_out, r, P, _ptr(x), _ptr(dy), _ptr(bits_u), _ptr(bits_v), _ptr(h),
                                     _ptr(l), _ptr(g), _ptr(tape_a), ctypes.c_float(gscale), _ptr(dh), _ptr(dl),
                                     _ptr(dg), _ptr(dx), int(bool(accumulate_dx)), _ptr(grad_u), _ptr(grad_v),
                                     int(bool(accumulate_signs)), _ptr(ws), ws.numel(), _stream(stream)),
           "blr_backward_paths")
    return dh, dl, dg, dx, grad_u, grad_v


def workspace_paths(M: int, d_in: int, d_out: int, r: int, paths: int, device=None):
    import torch
    n = blr_workspace_bytes_paths(M, d_in, d_out, r, paths)
    if n == 0:
        raise BlrError(-2, "blr_workspace_bytes_paths")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def blr_plane_linear(x, plane, scale: float = 1.0, *, y=None, stream=None):
    """y [M][n] = (f16(x * scale) . plane^T) / scale with plane an f16 [n][k]
    tensor (float16 or its int16 bit patterns). Returns y."""
    import torch
    M, k = _need(x, "x", (torch.float32,)).shape
    n = _need(plane, "plane", (torch.float16, torch.int16)).shape[0]
    _need(plane, "plane", (torch.float16, torch.int16), (n, k))
    y = torch.empty((M, n), dtype=torch.float32, device=x.device) if y is None else \
        _need(y, "y", (torch.float32,), (M, n))
    _check(load().blr_plane_linear(M, n, k, _ptr(x), _ptr(plane), _ptr(y), ctypes.c_float(scale), _stream(stream)),
           "blr_plane_linear")
    return y


_dtypes = None


def _types():
    """(f32, i32, wide, bytes, codes): dtype tuples for the checks below, and
    the numbers in the C ABI of `wide`, the element types of rows and adapters."""
    global _dtypes
    if _dtypes is None:
        import torch
        wide = (torch.float32, torch.float16, torch.bfloat16)
        _dtypes = ((torch.float32,), (torch.int32,), wide, (torch.uint8,), {t: i for i, t in enumerate(wide)})
    return _dtypes


def _at(t, name, dtypes, shape, dev):
    """Address of t, a contiguous tensor of this shape on GPU number dev. The
    checks are _need's, in the order that costs least when all is well."""
    try:
        if t.dtype in dtypes and t.shape == shape and t.is_contiguous() and t.get_device() == dev >= 0:
            return t.data_ptr()
    except AttributeError:
        pass
    _need(t, name, dtypes, shape)
    raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")


def _shape(t, name, dims):
    """t's shape, of `dims` dimensions."""
    try:
        shape = t.shape
        if len(shape) == dims:
            return shape
    except (AttributeError, TypeError):
        raise TypeError(f"{name} must be a torch.Tensor") from None
    raise ValueError(f"{name} has shape {tuple(shape)}, expected {dims} dimensions")


_gpus = {}  # number of a GPU: (torch.empty, its device)


def _new(shape, dtype, dev, stream):
    """Memory for a call on `stream` (None: the current one): the allocator
    hands out and takes back a tensor in the order of the stream it was made
    on, so it is made on the one that the kernels run on."""
    at = _gpus.get(dev)
    if at is None:
        import torch
        at = _gpus[dev] = (torch.empty, torch.device("cuda", dev))
    if stream is None:
        return at[0](shape, dtype=dtype, device=at[1])
    import torch
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=at[1])


def _out(t, name, dtype, shape, dev, stream):
    """(t, its address), t allocated when it is None."""
    if t is None:
        t = _new(shape, dtype, dev, stream)
        return t, t.data_ptr()
    return t, _at(t, name, (dtype,), shape, dev)


def _ws(ws, need, name, dev, stream):
    """(ws, (its address, its bytes)), `need` bytes allocated when it is None."""
    u8 = _types()[3]
    if ws is None:
        if need == 0:
            raise BlrError(-2, name)
        ws = _new(need, u8[0], dev, stream)
        return ws, (ws.data_ptr(), need)
    shape = _shape(ws, "ws", 1)
    return ws, (_at(ws, "ws", u8, shape, dev), shape[0])


def _device(t, name, dtypes, stream):
    """The GPU that t is on, and stream too."""
    try:
        dev = t.get_device()
    except AttributeError:
        dev = -1
    if dev < 0:
        _need(t, name, dtypes)
    if stream is not None and stream.device.index != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{dev}")
    return dev


_current = None  # (stream of a GPU, number of the current GPU)


def _launch(name, dev, stream, *args):
    """The C call `name` on the tensors' own device, on its current stream
    unless one is given."""
    global _current
    if _current is None:
        import torch
        torch.cuda.current_device()  # starts torch's side of the device, which the calls below take for granted
        _current = (torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice)
    handle = _current[0](dev) if stream is None else stream.cuda_stream
    fn = getattr(_lib or load(), name)
    if _current[1]() == dev:
        status = fn(*args, handle)
    else:
        import torch
        with torch.cuda.device(dev):
            status = fn(*args, handle)
    if status != 0:
        raise BlrError(status, name)


# pairs that a sort places in one launch, without a workspace
ROUTE_ONE_LAUNCH = 8192


def workspace_route(pairs: int, experts: int, device=None):
    import torch
    n = int(load().blr_route_workspace_bytes(pairs, experts))
    if n == 0:
        raise BlrError(-2, "blr_route_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def blr_route_sort(ids, experts: int, *, offsets=None, order=None, slot=None, ws=None, stream=None):
    """Sort the pairs of ids [T] or [T][k] (int32) by expert; an id outside
    [0, experts) means none. Returns (offsets [experts + 1], order [T k], slot
    in the shape of ids): the plan that the gather, the combine and the
    adapters take."""
    i32 = _types()[1]
    dev = _device(ids, "ids", i32, stream)
    shape = ids.shape
    if len(shape) not in (1, 2):
        raise ValueError(f"ids has shape {tuple(shape)}, expected [T] or [T][k]")
    at_ids, n = _at(ids, "ids", i32, shape, dev), ids.numel()
    if not 1 <= experts <= 1024 or n < 1:
        raise BlrError(-2, "blr_route_sort")
    work = (None, 0)
    if ws is not None or n > ROUTE_ONE_LAUNCH:
        ws, work = _ws(ws, load().blr_route_workspace_bytes(n, experts), "blr_route_workspace_bytes", dev, stream)
    offsets, at_offsets = _out(offsets, "offsets", i32[0], (experts + 1,), dev, stream)
    order, at_order = _out(order, "order", i32[0], (n,), dev, stream)
    slot, at_slot = _out(slot, "slot", i32[0], shape, dev, stream)
    _launch("blr_route_sort", dev, stream, n, experts, at_ids, at_offsets, at_order, at_slot, *work)
    return offsets, order, slot


def _route_plan(offsets, slot, dev):
    """(T, k, experts, the two addresses)."""
    i32 = _types()[1]
    ends = _shape(offsets, "offsets", 1)
    if ends[0] < 2:
        raise ValueError(f"offsets has shape {tuple(ends)}, expected [experts + 1]")
    shape = _shape(slot, "slot", 1 if getattr(slot, "ndim", 2) == 1 else 2)
    return (shape[0], shape[1] if len(shape) == 2 else 1, ends[0] - 1, _at(offsets, "offsets", i32, ends, dev),
            _at(slot, "slot", i32, shape, dev))


def _rows(t, name, stream):
    """(number of t's element type, rows, width, GPU) of rows t, where stream
    is too."""
    _, _, wide, _, codes = _types()
    dev = _device(t, name, wide, stream)
    rows, width = _shape(t, name, 2)
    if t.dtype not in codes:
        _need(t, name, wide)
    return codes[t.dtype], rows, width, dev


def blr_route_gather(x, offsets, slot, *, rows=None, stream=None):
    """Rows by expert: rows[slot[t][j]] = x[t], zero where the pair is not
    placed. Returns rows [T k][d]. Its gradient is blr_route_combine without
    weights."""
    code, _, d, dev = _rows(x, "x", stream)
    T, k, E, at_offsets, at_slot = _route_plan(offsets, slot, dev)
    at_x = _at(x, "x", (x.dtype,), (T, d), dev)
    rows, at_rows = _out(rows, "rows", x.dtype, (T * k, d), dev, stream)
    _launch("blr_route_gather", dev, stream, T, k, E, d, code, at_x, at_offsets, at_slot, at_rows)
    return rows


def blr_route_combine(z, offsets, slot, weights=None, *, y=None, accumulate_y=False, stream=None):
    """Experts' rows back into tokens: y[t] (+)= sum_j w[t][j] z[slot[t][j]]
    over the placed pairs; weights [T][k] f32, or None for ones. y is
    overwritten unless accumulate_y. Returns y [T][d]."""
    code, _, d, dev = _rows(z, "z", stream)
    T, k, E, at_offsets, at_slot = _route_plan(offsets, slot, dev)
    at_z = _at(z, "z", (z.dtype,), (T * k, d), dev)
    at_weights = None if weights is None else _at(weights, "weights", _types()[0], slot.shape, dev)
    if y is None and accumulate_y:
        raise ValueError("accumulate_y needs y")
    y, at_y = _out(y, "y", z.dtype, (T, d), dev, stream)
    _launch("blr_route_combine", dev, stream, T, k, E, d, code, at_z, at_offsets, at_slot, at_weights, at_y,
            1 if accumulate_y else 0)
    return y


def blr_route_combine_backward(dy, z, offsets, slot, weights=None, *, dz=None, dw=None, stream=None):
    """Gradient of blr_route_combine: dz[slot[t][j]] = w[t][j] dy[t] and, with
    weights, dw[t][j] = dy[t] . z[slot[t][j]], both zero where the pair is not
    placed. Returns (dz [T k][d], dw [T][k]), dw None without weights (z may
    then be None)."""
    f32 = _types()[0]
    code, _, d, dev = _rows(dy, "dy", stream)
    T, k, E, at_offsets, at_slot = _route_plan(offsets, slot, dev)
    at_dy = _at(dy, "dy", (dy.dtype,), (T, d), dev)
    at_weights = at_dw = at_z = None
    if weights is not None:
        at_weights = _at(weights, "weights", f32, slot.shape, dev)
        dw, at_dw = _out(dw, "dw", f32[0], slot.shape, dev, stream)
    elif dw is not None:
        raise ValueError("dw needs weights")
    if z is not None or dw is not None:
        at_z = _at(z, "z", (dy.dtype,), (T * k, d), dev)
    dz, at_dz = _out(dz, "dz", dy.dtype, (T * k, d), dev, stream)
    _launch("blr_route_combine_backward", dev, stream, T, k, E, d, code, at_dy, at_z, at_offsets, at_slot, at_weights,
            at_dz, at_dw)
    return dz, dw


def workspace_adapters(M: int, d_in: int, d_out: int, r: int, adapters: int, device=None, forward: bool = False):
    """A workspace of both adapter calls; with `forward`, of the forward alone."""
    import torch
    name = "blr_adapters_forward_workspace_bytes" if forward else "blr_adapters_workspace_bytes"
    n = int(getattr(load(), name)(M, d_in, d_out, r, adapters))
    if n == 0:
        raise BlrError(-2, name)
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def _adapters(rows, name, down, up, offsets, order, scale, ws, query, stream):
    """Checks that both adapter calls share; `rows` is x or dy, `query` tells
    the size of a workspace. Returns (sizes and types, addresses of down ..
    scale, ws, its (address, bytes), GPU)."""
    f32, i32, wide, _, codes = _types()
    act, M, _, dev = _rows(rows, name, stream)
    E, r, d_in = _shape(down, "down", 3)
    d_out = _shape(up, "up", 3)[1]
    at = (_at(down, "down", wide, (E, r, d_in), dev), _at(up, "up", (down.dtype,), (E, d_out, r), dev),
          _at(offsets, "offsets", i32, (E + 1,), dev), None if order is None else _at(order, "order", i32, (M,), dev),
          None if scale is None else _at(scale, "scale", f32, (E,), dev))
    need = getattr(load(), query)(M, d_in, d_out, r, E) if ws is None else 0
    ws, work = _ws(ws, need, query, dev, stream)
    return (M, d_in, d_out, r, E, act, codes[down.dtype]), at, ws, work, dev


def blr_adapters_forward(x, down, up, offsets, order=None, scale=None, *, y=None, accumulate_y=False, tape_s=None,
                         keep_tape=False, ws=None, stream=None):
    """Low-rank adapters of many requests at once: y[t] (+)= scale_e (x[t]
    down[e]^T) up[e]^T for each row t with adapter e. x [M][d_in]; down
    [E][r][d_in]; up [E][d_out][r]; (offsets, order) of
    blr_route_sort(adapter of each row, E), order None when the rows lie by
    adapter already. Beside a shared projection give its result as y with
    accumulate_y. The tape x down[e]^T [M][r], which the backward reads, is
    kept when tape_s is given or keep_tape is set. Returns (y, tape_s)."""
    if y is None and accumulate_y:
        raise ValueError("accumulate_y needs y")
    sizes, at, ws, work, dev = _adapters(x, "x", down, up, offsets, order, scale, ws,
                                         "blr_adapters_forward_workspace_bytes", stream)
    M, d_in, d_out, r = sizes[:4]
    at_x = _at(x, "x", (x.dtype,), (M, d_in), dev)
    y, at_y = _out(y, "y", x.dtype, (M, d_out), dev, stream)
    at_tape = None
    if keep_tape or tape_s is not None:
        tape_s, at_tape = _out(tape_s, "tape_s", _types()[0][0], (M, r), dev, stream)
    _launch("blr_adapters_forward", dev, stream, *sizes, at_x, *at, at_y, 1 if accumulate_y else 0, at_tape, *work)
    return y, tape_s


def blr_adapters_backward(x, dy, down, up, offsets, order=None, scale=None, tape_s=None, *, grad_down=None,
                          grad_up=None, accumulate_grads=False, grads=True, dx=None, accumulate_dx=False,
                          need_dx=True, ws=None, stream=None):
    """Backward of blr_adapters_forward: dx, and the f32 gradients grad_down
    [E][r][d_in] and grad_up [E][d_out][r] of every adapter (zero for one
    without rows). grads=False forms dx alone (x and tape_s may then be None),
    need_dx=False the gradients alone. Outputs not given are allocated;
    overwritten unless accumulate_grads / accumulate_dx. Returns (grad_down,
    grad_up, dx), None for what was not formed."""
    if (accumulate_grads and (grad_down is None or grad_up is None)) or (accumulate_dx and dx is None):
        raise ValueError("what is accumulated into has to be given")
    if not grads and (grad_down is not None or grad_up is not None):
        raise ValueError("grad_down and grad_up are given, but grads is False")
    if not need_dx and dx is not None:
        raise ValueError("dx is given, but need_dx is False")
    sizes, at, ws, work, dev = _adapters(dy, "dy", down, up, offsets, order, scale, ws,
                                         "blr_adapters_workspace_bytes", stream)
    M, d_in, d_out, r, E = sizes[:5]
    f32 = _types()[0]
    at_dy = _at(dy, "dy", (dy.dtype,), (M, d_out), dev)
    at_x = _at(x, "x", (dy.dtype,), (M, d_in), dev) if grads or x is not None else None
    at_tape = _at(tape_s, "tape_s", f32, (M, r), dev) if grads or tape_s is not None else None
    at_down = at_up = at_dx = None
    if grads:
        grad_down, at_down = _out(grad_down, "grad_down", f32[0], (E, r, d_in), dev, stream)
        grad_up, at_up = _out(grad_up, "grad_up", f32[0], (E, d_out, r), dev, stream)
    if need_dx:
        dx, at_dx = _out(dx, "dx", dy.dtype, (M, d_in), dev, stream)
    _launch("blr_adapters_backward", dev, stream, *sizes, at_x, at_dy, *at, at_tape, at_down, at_up,
            1 if accumulate_grads else 0, at_dx, 1 if accumulate_dx else 0, *work)
    return grad_down, grad_up, dx


def _kept(t, name, shape, dev):
    """Addresses of a checkpoint (q, b) of rows of this shape."""
    import torch
    try:
        q, b = t
    except (TypeError, ValueError):
        raise TypeError(f"{name} must be a tensor of rows or a checkpoint (q, b)") from None
    return (_at(q, f"{name} (q)", (torch.int8,), shape, dev),
            _at(b, f"{name} (b)", (torch.uint8,), (*shape[:-1], shape[-1] // 32), dev))


def _new_kept(kept, shape, dev, stream):
    """(kept, its addresses), the pair allocated when it is True."""
    import torch
    if kept is True:
        kept = (_new(shape, torch.int8, dev, stream), _new((*shape[:-1], shape[-1] // 32), torch.uint8, dev, stream))
    return tuple(kept), _kept(kept, "kept", shape, dev)


def blr_checkpoint_save(x, *, kept=True, stream=None):
    """Rows x [M][d] in 8 bits: q [M][d] (int8) and b [M][d / 32] (uint8), each
    32 values sharing the step 2^(b - 133). Returns (q, b), the given pair when
    `kept` is one."""
    code, M, d, dev = _rows(x, "x", stream)
    if d % 32:
        raise BlrError(-2, "blr_checkpoint_save")
    at_x = _at(x, "x", (x.dtype,), (M, d), dev)
    kept, at = _new_kept(kept, (M, d), dev, stream)
    _launch("blr_checkpoint_save", dev, stream, M, d, code, at_x, *at)
    return kept


def blr_checkpoint_load(q, b, dtype, *, x=None, stream=None):
    """The rows that a checkpoint stands for, in `dtype`. Returns x [M][d]."""
    import torch
    codes = _types()[4]
    dev = _device(q, "q", (torch.int8,), stream)
    M, d = _shape(q, "q", 2)
    at = _kept((q, b), "kept", (M, d), dev)
    if dtype not in codes:
        raise TypeError(f"dtype is {dtype}, expected one of {_types()[2]}")
    x, at_x = _out(x, "x", dtype, (M, d), dev, stream)
    _launch("blr_checkpoint_load", dev, stream, M, d, codes[dtype], *at, at_x)
    return x


# how a gate opens
GATE_LINEAR, GATE_SIGMOID, GATE_SILU = 0, 1, 2


def _number(v, lo, hi, status, where):
    """v in lo .. hi: ctypes cuts what C's type does not hold to its low bits."""
    if not lo <= v <= hi:
        raise BlrError(status, where)


_SPAN = (1 << 63) - 1


def workspace_norm(M: int, d: int, span: int = 1, device=None):
    import torch
    _number(span, 1, _SPAN, -2, "blr_norm_workspace_bytes")
    n = int(load().blr_norm_workspace_bytes(M, d, span))
    if n == 0:
        raise BlrError(-2, "blr_norm_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def _norm_columns(d, w, w_after, gate, gate_rows, ft, dev):
    """Addresses of w, w_after and the gate [gate_rows][d]."""
    f32 = _types()[0]
    return (None if w is None else _at(w, "w", f32, (d,), dev),
            None if w_after is None else _at(w_after, "w_after", f32, (d,), dev),
            None if gate is None else _at(gate, "gate", (ft,), (gate_rows, d), dev))


def blr_norm_forward(x, f=None, w=None, *, norm_f=False, w_after=None, gate=None, gate_kind=GATE_LINEAR, span=1,
                     skip=1.0, scale=1.0, eps=1e-6, n_dtype=None, need_n=True, out=None, n=None, stats=None,
                     need_stats=True, keep=False, kept=None, stream=None):
    """The residual stream after a block and the next block's normed rows:
    out = skip x + scale phi(gate) v, v = f w_after (normed first with norm_f),
    n = out rstd w. Without f, n is x normed and out is None. gate
    [ceil(M / span)][d] in f's type: a row for every `span` rows. n has n_dtype
    (x's type when not given). stats [2][M] is what the backward reads. With
    `keep` (or a pair `kept` to write to) the checkpoint of out, or of x without
    f, is formed too. Returns (out, n, stats, kept), None for what was not
    formed."""
    _number(span, 1, _SPAN, -2, "blr_norm_forward")
    _number(gate_kind, GATE_LINEAR, GATE_SILU, -9, "blr_norm_forward")
    code, M, d, dev = _rows(x, "x", stream)
    f32, _, wide, _, codes = _types()
    at_x = _at(x, "x", (x.dtype,), (M, d), dev)
    at_f = at_out = at_n = at_stats = None
    ft = n_dtype if f is None else getattr(f, "dtype", None)
    n_dtype = n_dtype or x.dtype
    ft = ft or x.dtype
    if f is not None:
        at_f = _at(f, "f", wide, (M, d), dev)
    elif out is not None or gate is not None or w_after is not None or norm_f:
        raise ValueError("out, gate, w_after and norm_f need f")
    if n_dtype not in codes:
        raise TypeError(f"n_dtype is {n_dtype}, expected one of {wide}")
    at_w, at_after, at_gate = _norm_columns(d, w, w_after, gate, -(-M // span), ft, dev)
    if f is not None:
        out, at_out = _out(out, "out", x.dtype, (M, d), dev, stream)
    if need_n or n is not None:
        n, at_n = _out(n, "n", n_dtype, (M, d), dev, stream)
    if need_stats or stats is not None:
        stats, at_stats = _out(stats, "stats", f32[0], (2, M), dev, stream)
    at_kept = (None, None)
    if keep or kept is not None:
        if d % 32:
            raise BlrError(-2, "blr_norm_forward")
        kept, at_kept = _new_kept(True if kept is None else kept, (M, d), dev, stream)
    _launch("blr_norm_forward", dev, stream, M, d, code, codes[ft], codes[n_dtype], at_x, at_f, 1 if norm_f else 0,
            at_after, at_gate, gate_kind, span, skip, scale, at_w, eps, at_out, at_n, at_stats, *at_kept)
    return out, n, stats, kept


def blr_norm_backward(dn, dout, out, f=None, w=None, stats=None, *, has_f=None, f_dtype=None, x_dtype=None,
                      norm_f=False, w_after=None, gate=None, gate_kind=GATE_LINEAR, span=1, skip=1.0, scale=1.0,
                      dx=None, need_dx=True, df=None, need_df=True, dgate=None, dw=None, dw_after=None, grads=True,
                      accumulate_grads=False, ws=None, stream=None):
    """Gradients of blr_norm_forward, dn and dout those of n and of out (None: a
    zero, for one of them). out and f are rows or checkpoints (q, b); the types
    that neither they nor dout tell are x_dtype and f_dtype. f None: the forward
    had none (has_f=True: it had, but its values do not take part). With `grads`
    the gradients of w, w_after and gate are formed where these are given and
    take part; overwritten unless accumulate_grads (dgate of span 1 always is).
    Returns (dx, df, dgate, dw, dw_after), None for what was not formed."""
    _number(span, 1, _SPAN, -2, "blr_norm_backward")
    _number(gate_kind, GATE_LINEAR, GATE_SILU, -9, "blr_norm_backward")
    f32, _, wide, _, codes = _types()
    rows, name = (dout, "dout") if dn is None else (dn, "dn")
    code, M, d, dev = _rows(rows, name, stream)
    has_f = f is not None if has_f is None else has_f
    if not has_f and (f is not None or gate is not None or w_after is not None or norm_f):
        raise ValueError("f, gate, w_after and norm_f need has_f")
    if not grads and (dgate is not None or dw is not None or dw_after is not None):
        raise ValueError("gradients are given, but grads is False")
    if (dx is not None and not need_dx) or (df is not None and not (need_df and has_f)):
        raise ValueError("dx or df is given, but not to be formed")
    if (dw is not None and (w is None or dn is None)) or (dw_after is not None and w_after is None) or \
            (dgate is not None and gate is None):
        raise ValueError("dw needs w and dn, dw_after w_after, and dgate gate")
    nt = rows.dtype if dn is not None else None
    xt = dout.dtype if dout is not None else getattr(out, "dtype", None) or x_dtype
    ft = getattr(f, "dtype", None) or f_dtype or (xt if not has_f else None)
    if xt not in codes or ft not in codes:
        raise TypeError(f"the type of the stream is {xt}, that of f {ft}: give x_dtype and f_dtype, of {wide}")
    if xt != wide[0]:
        nt = nt or xt
    else:
        nt = nt or wide[0]
    shape = (M, d)

    def given(t, name, dtype):
        if t is None:
            return None, (None, None)
        if hasattr(t, "dtype"):
            return _at(t, name, (dtype,), shape, dev), (None, None)
        return None, _kept(t, name, shape, dev)

    at_dn = None if dn is None else _at(dn, "dn", (nt,), shape, dev)
    at_dout = None if dout is None else _at(dout, "dout", (xt,), shape, dev)
    at_o, at_okept = given(out, "out", xt)
    at_f, at_fkept = given(f, "f", ft)
    gate_rows = -(-M // span)
    at_w, at_after, at_gate = _norm_columns(d, w, w_after, gate, gate_rows, ft, dev)
    at_stats = None if stats is None else _at(stats, "stats", f32, (2, M), dev)
    form = dict(dgate=grads and gate is not None, dw=grads and w is not None and dn is not None,
                dw_after=grads and w_after is not None)
    if accumulate_grads and ((form["dw"] and dw is None) or (form["dw_after"] and dw_after is None) or
                             (form["dgate"] and span > 1 and dgate is None)):
        raise ValueError("what is accumulated into has to be given")
    at_dx = at_df = at_dgate = at_dw = at_dafter = None
    need = load().blr_norm_workspace_bytes(M, d, span) if ws is None else 0
    ws, work = _ws(ws, need, "blr_norm_workspace_bytes", dev, stream)
    if need_dx:
        dx, at_dx = _out(dx, "dx", xt, shape, dev, stream)
    if need_df and has_f:
        df, at_df = _out(df, "df", ft, shape, dev, stream)
    if form["dgate"]:
        dgate, at_dgate = _out(dgate, "dgate", ft if span == 1 else f32[0], (gate_rows, d), dev, stream)
    if form["dw"]:
        dw, at_dw = _out(dw, "dw", f32[0], (d,), dev, stream)
    if form["dw_after"]:
        dw_after, at_dafter = _out(dw_after, "dw_after", f32[0], (d,), dev, stream)
    _launch("blr_norm_backward", dev, stream, M, d, codes[xt], codes[ft], codes[nt], at_dn, at_dout, at_o, *at_okept,
            1 if has_f else 0, at_f, *at_fkept, 1 if norm_f else 0, at_after, at_gate, gate_kind, span, skip, scale,
            at_w, at_stats, at_dx, at_df, at_dgate, at_dw, at_dafter, 1 if accumulate_grads else 0, *work)
    return dx, df, dgate, dw, dw_after


# the gated feed-forward's activation
ACT_SILU, ACT_GELU = 0, 1


def workspace_gated(M: int, d: int, ff: int, device=None):
    import torch
    n = int(load().blr_gated_workspace_bytes(M, d, ff))
    if n == 0:
        raise BlrError(-2, "blr_gated_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def _gated_weights(w_gate, w_up, stream):
    """(ff, d, type, its number, GPU, the two addresses)."""
    code, ff, d, dev = _rows(w_gate, "w_gate", stream)
    t = w_gate.dtype
    if code == 0:
        raise BlrError(-9, "w_gate")
    return ff, d, t, code, dev, (_at(w_gate, "w_gate", (t,), (ff, d), dev), _at(w_up, "w_up", (t,), (ff, d), dev))


def _tape(tape, M, ff, dev):
    """Addresses of g and u kept in 8 bits: q [2][M][ff], b [2][M][ff / 32]."""
    return _kept(tape, "tape", (2, M, ff), dev)


def blr_gated_forward(x, w_gate, w_up, *, kind=ACT_SILU, h_dtype=None, h=None, keep=False, tape=None, stream=None):
    """h = act(x w_gate^T) * (x w_up^T) in one kernel: x [M][d], w_gate and w_up
    [ff][d], all f16 or all bf16; h [M][ff] of h_dtype, theirs or f32. With `keep`
    (or a pair `tape` to write to) the two projections are kept in 8 bits for
    the backward: tape = (q [2][M][ff], b [2][M][ff / 32]). Returns (h, tape),
    tape None when not kept."""
    _number(kind, ACT_SILU, ACT_GELU, -9, "blr_gated_forward")
    ff, d, t, code, dev, at_w = _gated_weights(w_gate, w_up, stream)
    codes = _types()[4]
    M = _shape(x, "x", 2)[0]
    at_x = _at(x, "x", (t,), (M, d), dev)
    h_dtype = h.dtype if h_dtype is None and h is not None else h_dtype or t
    if h_dtype not in codes:
        raise TypeError(f"h_dtype is {h_dtype}, expected one of {_types()[2]}")
    h, at_h = _out(h, "h", h_dtype, (M, ff), dev, stream)
    at_tape = (None, None)
    if keep or tape is not None:
        if ff % 32:
            raise BlrError(-2, "blr_gated_forward")
        tape, at_tape = _new_kept(True if tape is None else tape, (2, M, ff), dev, stream)
    _launch("blr_gated_forward", dev, stream, M, d, ff, code, codes[h_dtype], at_x, *at_w, kind, at_h, *at_tape)
    return h, tape


def blr_gated_backward(x, dh, w_gate, w_up, tape=None, *, kind=ACT_SILU, gscale=1.0, dx=None, need_dx=True,
                       accumulate_dx=False, dw_gate=None, dw_up=None, grads=True, grad_dtype=None,
                       accumulate_grads=False, ws=None, stream=None):
    """Gradients of blr_gated_forward from dh [M][ff] (of the weights' type, or
    f32). x is rows or a checkpoint (q, b); the two projections come from the
    tape, or are formed again without one. gscale: the power of two under which
    dg and du are rounded to the weights' type. dw_gate and dw_up have
    grad_dtype, the weights' type or f32. grads=False forms dx alone (x may then
    be None with a tape), need_dx=False the weights' gradients alone. Outputs
    not given are allocated; overwritten unless accumulate_dx /
    accumulate_grads. Returns (dx, dw_gate, dw_up), None for what was not
    formed."""
    _number(kind, ACT_SILU, ACT_GELU, -9, "blr_gated_backward")
    if (accumulate_grads and (dw_gate is None or dw_up is None)) or (accumulate_dx and dx is None):
        raise ValueError("what is accumulated into has to be given")
    if not grads and (dw_gate is not None or dw_up is not None):
        raise ValueError("dw_gate and dw_up are given, but grads is False")
    if not need_dx and dx is not None:
        raise ValueError("dx is given, but need_dx is False")
    ff, d, t, code, dev, at_w = _gated_weights(w_gate, w_up, stream)
    f32, _, wide, _, codes = _types()
    M = _shape(dh, "dh", 2)[0]
    at_dh = _at(dh, "dh", (t, *f32), (M, ff), dev)
    at_x, at_xkept = None, (None, None)
    if x is not None and hasattr(x, "dtype"):
        at_x = _at(x, "x", (t,), (M, d), dev)
    elif x is not None:
        at_xkept = _kept(x, "x", (M, d), dev)
    at_tape = (None, None) if tape is None else _tape(tape, M, ff, dev)
    grad_dtype = dw_gate.dtype if grad_dtype is None and dw_gate is not None else grad_dtype or t
    if grad_dtype not in codes:
        raise TypeError(f"grad_dtype is {grad_dtype}, expected one of {wide}")
    need = load().blr_gated_workspace_bytes(M, d, ff) if ws is None else 0
    ws, work = _ws(ws, need, "blr_gated_workspace_bytes", dev, stream)
    at_dx = at_gate = at_up = None
    if need_dx:
        dx, at_dx = _out(dx, "dx", t, (M, d), dev, stream)
    if grads:
        dw_gate, at_gate = _out(dw_gate, "dw_gate", grad_dtype, (ff, d), dev, stream)
        dw_up, at_up = _out(dw_up, "dw_up", grad_dtype, (ff, d), dev, stream)
    _launch("blr_gated_backward", dev, stream, M, d, ff, code, codes[dh.dtype], codes[grad_dtype], at_x, *at_xkept, at_dh,
            *at_w, kind, *at_tape, gscale, at_dx, 1 if accumulate_dx else 0, at_gate, at_up,
            1 if accumulate_grads else 0, *work)
    return dx, dw_gate, dw_up


def blr_sumsq(a, nparts: int = 64, stream=None) -> float:
    """Sum of squares of a float32 tensor: nparts device partials, added on
    the host in f64 (the page's `sumsq`). Synchronises the stream."""
    import torch
    _need(a, "a", (torch.float32,))
    parts = torch.empty(nparts, dtype=torch.float32, device=a.device)
    _check(load().blr_sumsq(_ptr(a), a.numel(), _ptr(parts), int(nparts), _stream(stream)), "blr_sumsq")
    return float(parts.double().sum().item())


def all_finite(*tensors, stream=None) -> bool:
    """True when every element of the float32 tensors is finite (each sum
    of squares is finite; an overflowing square also reads as not finite)."""
    import math
    return all(math.isfinite(blr_sumsq(t, stream=stream)) for t in tensors)


def next_gscale(gscale: float, finite: bool, lo: float = 1.0, hi: float = 2.0 ** 24) -> float:
    """Power-of-two gradient staging scale for the next step: double it after
    a step whose gradients were finite, halve it after one that overflowed,
    within [lo, hi]."""
    g = gscale * 2.0 if finite else gscale * 0.5
    return min(max(g, lo), hi)


def blr_profile_enable(max_launches: int):
    _check(load().blr_profile_enable(int(max_launches)), "blr_profile_enable")


def blr_profile_reset():
    _check(load().blr_profile_reset(), "blr_profile_reset")


def blr_profile_read(max_kinds: int = 64) -> dict[str, tuple[int, float]]:
    """{kernel name: (launches, total ms)} of the timed launches so far."""
    names = (ctypes.c_char_p * max_kinds)()
    counts = (ctypes.c_int64 * max_kinds)()
    tot = (ctypes.c_double * max_kinds)()
    n = load().blr_profile_read(names, counts, tot, max_kinds)
    if n < 0:
        raise BlrError(n, "blr_profile_read")
    return {names[i].decode(): (int(counts[i]), float(tot[i])) for i in range(min(n, max_kinds))}
