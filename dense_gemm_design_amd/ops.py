"""Operators around the product: block-scaled e4m3 operands and their product, layer norm and its
gradients, and the clipping of a list of gradients (C ABI in include/gemm_ops.h).

Every function takes torch tensors on one GPU, checks them (ValueError) before anything is
launched, and enqueues kernels on torch's current stream of that GPU; outputs and workspaces are
torch's, so the calls can be recorded into a HIP graph.
"""
import ctypes
from array import array

import torch

from . import _lib
from ._lib import GEMM_BF16, GEMM_F32, GEMM_OK, GemmError

GEMM_BLOCK_ROW, GEMM_BLOCK_TILE = 0, 1
BLOCK = 128
EXPORTS = ("gemm_block_quantize", "gemm_block_workspace", "gemm_block_run", "gemm_layer_norm",
           "gemm_layer_norm_backward_workspace", "gemm_layer_norm_backward",
           "gemm_grad_norm_workspace", "gemm_grad_norm", "gemm_clip_grad_norm")

_BLOCKS = {"row": GEMM_BLOCK_ROW, "tile": GEMM_BLOCK_TILE}
_TYPES = {torch.bfloat16: GEMM_BF16, torch.float32: GEMM_F32}
_OUT = {"bf16": torch.bfloat16, "f32": torch.float32}
_CODES = (torch.uint8, torch.float8_e4m3fn)


class GemmBlockDesc(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("lda", ctypes.c_int64), ("ldb", ctypes.c_int64),
                ("scale_lda", ctypes.c_int64), ("scale_ldb", ctypes.c_int64),
                ("block_b", ctypes.c_int32), ("pow2", ctypes.c_int32),
                ("dtype_c", ctypes.c_int32), ("dtype_source", ctypes.c_int32)]


class GemmTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("numel", ctypes.c_int64), ("dtype", ctypes.c_int64)]


_ops = None


def load():
    """libdgemm.so with the argument types of include/gemm_ops.h."""
    global _ops
    if _ops is not None:
        return _ops
    lib = _lib.load()
    vp, sz, i64, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64, ctypes.c_int32
    f32 = ctypes.c_float
    desc, psz = ctypes.POINTER(GemmBlockDesc), ctypes.POINTER(sz)
    lib.gemm_block_quantize.argtypes = [vp, i32, i64, i64, i64, i32, i32, vp, i64, vp, i64, vp,
                                        i64, vp, i64, vp]
    lib.gemm_block_workspace.argtypes = [desc, psz]
    lib.gemm_block_run.argtypes = [desc, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.gemm_layer_norm.argtypes = [vp, i32, i64, i64, i64, vp, vp, i32, f32, vp, vp, vp, vp]
    lib.gemm_layer_norm_backward_workspace.argtypes = [i64, i64, psz]
    lib.gemm_layer_norm_backward.argtypes = [vp, i64, vp, i64, i32, i64, i64, vp, i32, vp, vp, vp,
                                             vp, vp, vp, sz, vp]
    lib.gemm_grad_norm_workspace.argtypes = [vp, i64, psz]
    lib.gemm_grad_norm.argtypes = [vp, i64, vp, vp, sz, vp]
    lib.gemm_clip_grad_norm.argtypes = [vp, i64, f32, vp, vp, sz, vp]
    for name in EXPORTS:
        getattr(lib, name).restype = ctypes.c_int
    _ops = lib
    return lib


def _enqueue(device, where, fn, *args):
    """fn(*args, stream) on `device`'s current stream."""
    stream = torch._C._cuda_getCurrentRawStream(device)
    if torch._C._cuda_getDevice() == device:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, stream)
    if status != GEMM_OK:
        raise GemmError(status, where)


def _bytes(where, fn, *args):
    n = ctypes.c_size_t()
    status = fn(*args, ctypes.byref(n))
    if status != GEMM_OK:
        raise GemmError(status, where)
    return n.value


def _refuse(what, t, want):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{what} must be a torch tensor")
    raise ValueError(f"{what} must be {want}; got {t.dtype} {tuple(t.shape)} with strides "
                     f"{t.stride()}")


def _on_one_gpu(**tensors):
    """The GPU that all of them are on."""
    device = None
    for what, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{what} is on {t.device}; every operand must be on the GPU")
        at = t.get_device()
        if device is None:
            device = at
        elif at != device:
            raise ValueError(f"{what} is on GPU {at}, other operands on GPU {device}")
    return device


def _rows(what, t):
    """(rows, cols, elements from row to row) of a matrix whose rows are packed."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.dtype not in _TYPES:
        _refuse(what, t, "a float32 or bfloat16 matrix")
    rows, cols = t.shape
    stride, one = t.stride()
    if cols > 1 and one != 1:
        _refuse(what, t, "a matrix of packed rows (columns next to each other)")
    if rows <= 1:
        stride = cols
    elif 0 < stride < cols:
        _refuse(what, t, "a matrix whose rows do not overlap")
    return rows, cols, stride


def _vector(what, t, numel, dtypes):
    if (not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.dim() != 1
            or t.shape[0] != numel or not t.is_contiguous()):
        _refuse(what, t, f"a packed vector of {numel}, {' or '.join(map(str, dtypes))}")


# ---- block-scaled e4m3 ------------------------------------------------------------------------

class BlockScaled:
    """A matrix (rows, K) in e4m3 with one float32 scale per block of 128 of its values.

    data     uint8 codes, (rows, K rounded up to 16), zeros behind column K
    scales   (rows, K / 128) for block "row" -- one of 128 neighbours of a row -- or
             (rows / 128, K / 128) for block "tile" (128 x 128), rounded up; stored with the scales
             of one block column next to each other, i.e. the transpose of a packed matrix
    pow2     every scale is a power of two (or NaN): the product then leaves the scaling to the
             matrix instructions
    """
    __slots__ = ("data", "scales", "K", "block", "pow2")

    def __init__(self, data, scales, K, block, pow2=False):
        self.data, self.scales, self.K, self.block, self.pow2 = data, scales, K, block, pow2

    @property
    def values(self):
        """The codes as torch's float8 values, (rows, K)."""
        return self.data.view(torch.float8_e4m3fn)[:, :self.K]

    def __repr__(self):
        return (f"BlockScaled({self.data.shape[0]} x {self.K}, block={self.block!r}, "
                f"pow2={self.pow2}, {self.data.device})")


def _operand(what, q):
    """(rows, bytes from row to row, floats from block column to block column), checked."""
    if not isinstance(q, BlockScaled):
        raise ValueError(f"{what} must be a BlockScaled")
    data, scales, K = q.data, q.scales, q.K
    if q.block not in _BLOCKS:
        raise ValueError(f"{what}.block must be one of {sorted(_BLOCKS)}; got {q.block!r}")
    if (not isinstance(data, torch.Tensor) or data.dim() != 2 or data.dtype not in _CODES
            or data.shape[1] != -(-K // 16) * 16):
        _refuse(f"{what}.data", data, f"uint8 or float8_e4m3fn codes (rows, {-(-K // 16) * 16})")
    rows, width = data.shape
    pitch = data.stride(0) if rows > 1 and width else width
    if (width > 1 and data.stride(1) != 1) or pitch < width or pitch % 16:
        _refuse(f"{what}.data", data, "packed rows at multiples of 16 bytes")
    kb, sr = -(-K // BLOCK), rows if q.block == "row" else -(-rows // BLOCK)
    if (not isinstance(scales, torch.Tensor) or scales.dtype is not torch.float32
            or tuple(scales.shape) != (sr, kb)):
        _refuse(f"{what}.scales", scales, f"float32 ({sr}, {kb})")
    spitch = scales.stride(1) if kb > 1 else sr
    if (sr > 1 and scales.stride(0) != 1) or spitch < sr:
        _refuse(f"{what}.scales", scales, "stored with the scales of one block column next to "
                                          "each other (the transpose of a packed matrix)")
    return rows, pitch, spitch


def block_quantize(x, block="row", transposed=False, pow2=False):
    """x (rows, cols), float32 or bfloat16 with packed rows, as BlockScaled: of each block the
    scale amax / 448 (at least 2^-126; with pow2 the smallest power of two that is not below it;
    NaN where the block holds an infinity or a NaN), and the codes of x / scale, rounded to nearest
    even.  block: "row" (1 x 128) or "tile" (128 x 128).  transposed: False for x, True for its
    transpose (cols, rows), "both" for the pair of them from one read of x."""
    rows, cols, stride = _rows("x", x)
    if block not in _BLOCKS:
        raise ValueError(f"block must be one of {sorted(_BLOCKS)}; got {block!r}")
    if transposed not in (False, True, "both"):
        raise ValueError(f'transposed must be False, True or "both"; got {transposed!r}')
    device = _on_one_gpu(x=x)
    sides = []
    for wanted, r, c in ((transposed is not True, rows, cols), (transposed is not False, cols, rows)):
        if not wanted:
            sides.append(None)
            continue
        data = x.new_empty((r, -(-c // 16) * 16), dtype=torch.uint8)
        scales = x.new_empty((-(-c // BLOCK), r if block == "row" else -(-r // BLOCK)),
                             dtype=torch.float32)
        sides.append((data, scales, c))
    args = []
    for side in sides:
        if side is None:
            args += [None, 0, None, 0]
        else:
            args += [side[0].data_ptr(), side[0].shape[1], side[1].data_ptr(), side[1].shape[1]]
    if rows and cols:
        _enqueue(device, "gemm_block_quantize", load().gemm_block_quantize, x.data_ptr(),
                 _TYPES[x.dtype], rows, cols, stride, _BLOCKS[block], bool(pow2), *args)
    out = tuple(BlockScaled(s[0], s[1].t(), s[2], block, bool(pow2)) for s in sides if s)
    return out if len(out) > 1 else out[0]


def block_gemm(a, b, out_dtype="bf16", bias_col=None, source=None, out=None):
    """C (M, N) = A B^T + bias_col + source of BlockScaled operands a (M, K), scaled per row and
    block of 128, and b (N, K), scaled per row or per tile.  bias_col: N float32; source: (M, N)
    float32 or bfloat16, packed, possibly `out` itself.  out_dtype: "bf16" or "f32", or that of
    `out`, which is written where it is given.  Sums are float32, rounded once."""
    M, lda, scale_lda = _operand("a", a)
    N, ldb, scale_ldb = _operand("b", b)
    K = a.K
    if b.K != K:
        raise ValueError(f"a and b must have the same K; got {K} and {b.K}")
    if a.block != "row":
        raise ValueError('a must have block "row": one scale per row and 128 columns')
    if out is None:
        if out_dtype not in _OUT:
            raise ValueError(f"out_dtype must be one of {sorted(_OUT)}; got {out_dtype!r}")
    elif (not isinstance(out, torch.Tensor) or out.dtype not in _TYPES
          or tuple(out.shape) != (M, N) or not out.is_contiguous()):
        _refuse("out", out, f"a packed float32 or bfloat16 matrix ({M}, {N})")
    if bias_col is not None:
        _vector("bias_col", bias_col, N, (torch.float32,))
    if source is not None and (not isinstance(source, torch.Tensor) or source.dtype not in _TYPES
                               or tuple(source.shape) != (M, N) or not source.is_contiguous()):
        _refuse("source", source, f"a packed float32 or bfloat16 matrix ({M}, {N})")
    data = a.data
    device = _on_one_gpu(a=data, a_scales=a.scales, b=b.data, b_scales=b.scales,
                         bias_col=bias_col, source=source, out=out)
    if out is None:
        out = data.new_empty((M, N), dtype=_OUT[out_dtype])
    if M == 0 or N == 0:
        return out
    lib = load()
    desc = GemmBlockDesc(M, N, K, lda, ldb, scale_lda, scale_ldb, _BLOCKS[b.block],
                         bool(a.pow2 and b.pow2), _TYPES[out.dtype],
                         _TYPES[source.dtype] if source is not None else GEMM_F32)
    need = _bytes("gemm_block_workspace", lib.gemm_block_workspace, desc)
    workspace = data.new_empty(need, dtype=torch.uint8) if need else None
    _enqueue(device, "gemm_block_run", lib.gemm_block_run, desc, data.data_ptr(),
             a.scales.data_ptr(), b.data.data_ptr(), b.scales.data_ptr(), out.data_ptr(),
             bias_col.data_ptr() if bias_col is not None else None,
             source.data_ptr() if source is not None else None,
             workspace.data_ptr() if need else None, need)
    return out


# ---- layer norm -------------------------------------------------------------------------------

def layer_norm(x, weight, bias=None, eps=1e-5):
    """(y, mean, rstd) of x (rows, cols), float32 or bfloat16 with packed rows: each row less its
    mean, times rstd = 1 / sqrt(variance + eps), times weight, plus bias.  weight and bias (cols)
    are float32 or of x's type; y has x's type, mean and rstd are float32 (rows)."""
    rows, cols, stride = _rows("x", x)
    if cols == 0:
        raise ValueError("x has rows of no elements, which have no mean")
    dtype = x.dtype
    _vector("weight", weight, cols, (torch.float32, dtype))
    if bias is not None:
        _vector("bias", bias, cols, (weight.dtype,))
    device = _on_one_gpu(x=x, weight=weight, bias=bias)
    y = x.new_empty((rows, cols))
    mean, rstd = x.new_empty((2, rows), dtype=torch.float32).unbind(0)
    if rows:
        _enqueue(device, "gemm_layer_norm", load().gemm_layer_norm, x.data_ptr(), _TYPES[dtype],
                 rows, cols, stride, weight.data_ptr(),
                 bias.data_ptr() if bias is not None else None, _TYPES[weight.dtype], eps,
                 y.data_ptr(), mean.data_ptr(), rstd.data_ptr())
    return y, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd):
    """(dx, dweight, dbias) of layer_norm for the gradient dy of its y; mean and rstd are what it
    returned.  dx has x's type, dweight and dbias the weight's, summed over the rows in float32."""
    rows, cols, stride = _rows("x", x)
    drows, dcols, dstride = _rows("dy", dy)
    if cols == 0:
        raise ValueError("x has rows of no elements, which have no mean")
    dtype = x.dtype
    if (drows, dcols) != (rows, cols) or dy.dtype is not dtype:
        _refuse("dy", dy, f"{dtype} ({rows}, {cols}) like x")
    _vector("weight", weight, cols, (torch.float32, dtype))
    _vector("mean", mean, rows, (torch.float32,))
    _vector("rstd", rstd, rows, (torch.float32,))
    device = _on_one_gpu(dy=dy, x=x, weight=weight, mean=mean, rstd=rstd)
    lib = load()
    dx = x.new_empty((rows, cols))
    dw, db = weight.new_empty((cols,)), weight.new_empty((cols,))
    need = _bytes("gemm_layer_norm_backward_workspace", lib.gemm_layer_norm_backward_workspace,
                  rows, cols)
    workspace = x.new_empty(need, dtype=torch.uint8) if need else None
    _enqueue(device, "gemm_layer_norm_backward", lib.gemm_layer_norm_backward, dy.data_ptr(),
             dstride, x.data_ptr(), stride, _TYPES[dtype], rows, cols, weight.data_ptr(),
             _TYPES[weight.dtype], mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), dw.data_ptr(),
             db.data_ptr(), workspace.data_ptr() if need else None, need)
    return dx, dw, db


# ---- gradient clipping ------------------------------------------------------------------------

def _tensor_list(grads, out):
    """The list as an array of gemm_tensor, its length, and the GPU it is on."""
    flat, device = [], None
    for i, g in enumerate(grads):
        if not isinstance(g, torch.Tensor) or g.dtype not in _TYPES or not g.is_contiguous():
            _refuse(f"gradient {i}", g, "packed float32 or bfloat16")
        if not g.is_cuda:
            raise ValueError(f"gradient {i} is on {g.device}; every operand must be on the GPU")
        at, n = g.get_device(), g.numel()
        if device is None:
            device = at
        elif at != device:
            raise ValueError(f"gradient {i} is on GPU {at}, others on GPU {device}")
        o = g if out is None else out[i]
        if o is not g:
            if not isinstance(o, torch.Tensor) or o.dtype is not g.dtype or o.numel() != n \
                    or not o.is_contiguous():
                _refuse(f"out {i}", o, f"packed {g.dtype} of {n} elements")
            if not o.is_cuda or o.get_device() != device:
                raise ValueError(f"out {i} is on {o.device}, the gradients on GPU {device}")
        flat += (g.data_ptr(), o.data_ptr(), n, _TYPES[g.dtype])
    if device is None:
        raise ValueError("the list of gradients is empty")
    return array("Q", flat), len(flat) // 4, device


def grad_norm(grads):
    """The 2-norm of all elements of a list of gradients (float32 or bfloat16, packed, on one
    GPU), as a float32 tensor of no dimension.  Squares are summed in float64."""
    grads = list(grads)
    return _norm(grads, None, None)


def clip_grad_norm(grads, max_norm, out=None):
    """Scales a list of gradients by min(1, max_norm / (norm + 1e-6)), in place or into the tensors
    `out` (one of each gradient's type and size), and returns the norm before that, as grad_norm."""
    grads = list(grads)
    max_norm = float(max_norm)
    if not max_norm >= 0.0:
        raise ValueError(f"max_norm must not be negative; got {max_norm}")
    if out is not None:
        out = list(out)
        if len(out) != len(grads):
            raise ValueError(f"out has {len(out)} tensors for {len(grads)} gradients")
    return _norm(grads, out, max_norm)


def _norm(grads, out, max_norm):
    table, count, device = _tensor_list(grads, out)
    at = table.buffer_info()[0]
    lib = load()
    need = _bytes("gemm_grad_norm_workspace", lib.gemm_grad_norm_workspace, at, count)
    norm = grads[0].new_empty((), dtype=torch.float32)
    workspace = norm.new_empty(need, dtype=torch.uint8) if need else None
    ptr = workspace.data_ptr() if need else None
    if max_norm is None:
        _enqueue(device, "gemm_grad_norm", lib.gemm_grad_norm, at, count, norm.data_ptr(), ptr,
                 need)
    else:
        _enqueue(device, "gemm_clip_grad_norm", lib.gemm_clip_grad_norm, at, count, max_norm,
                 norm.data_ptr(), ptr, need)
    return norm
