"""Operators around the product: block-scaled e4m3 operands and their product, layer norm and its
gradients, and the clipping of a list of gradients (C ABI in include/gemm_ops.h).

Every function takes torch tensors on one GPU, checks them (ValueError) before anything is
launched, and enqueues kernels on torch's current stream of that GPU; outputs and workspaces are
torch's, so the calls can be recorded into a HIP graph.  They are plain kernels to autograd: results
carry no history, whether or not the arguments require gradients, so a backward pass calls them by itself
(in a torch.autograd.Function, or as examples/fp8_linear.py does); what is written in place or into
`out` counts as changed, so autograd refuses to use what it had saved of it.  The checks and calls are compiled
(csrc/binding.cpp); load() gives the C ABI itself through ctypes.
"""
import ctypes

from . import _lib

GEMM_BLOCK_ROW, GEMM_BLOCK_TILE = 0, 1
EXPORTS = ("gemm_block_quantize", "gemm_block_workspace", "gemm_block_run", "gemm_layer_norm",
           "gemm_layer_norm_backward_workspace", "gemm_layer_norm_backward",
           "gemm_grad_norm_workspace", "gemm_grad_norm", "gemm_clip_grad_norm")


class GemmBlockDesc(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("lda", ctypes.c_int64), ("ldb", ctypes.c_int64),
                ("scale_lda", ctypes.c_int64), ("scale_ldb", ctypes.c_int64),
                ("block_b", ctypes.c_int32), ("pow2", ctypes.c_int32),
                ("dtype_c", ctypes.c_int32), ("dtype_source", ctypes.c_int32),
                ("exact", ctypes.c_int32)]


class GemmTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("numel", ctypes.c_int64), ("dtype", ctypes.c_int64)]


_ops = _native = None


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


def _binding():
    """The compiled binding; raises if it is not built."""
    global _native
    if _native is None:
        load()   # the library it calls, and the HIP runtime that torch carries
        try:
            from . import _binding as native
        except ImportError as e:
            raise RuntimeError("dense_gemm_design_amd/_binding.so is not built; run "
                               "dense_gemm_design_amd/build.py (or __graft_entry__.build())") from e
        _native = native
    return _native


# ---- block-scaled e4m3 ------------------------------------------------------------------------

class BlockScaled:
    """A matrix (rows, K) in e4m3 with one float32 scale per block of 128 of its values.

    data     uint8 codes, (rows, K rounded up to 16), zeros behind column K
    scales   (rows, K / 128) for block "row" -- one of 128 neighbours of a row -- or
             (rows / 128, K / 128) for block "tile" (128 x 128), rounded up; stored with the scales
             of one block column next to each other, i.e. the transpose of a packed matrix
    pow2     every scale is a positive power of two, 2^-126 at least, or NaN: the product then leaves
             the scaling to the matrix instructions (which would read other scales as such)
    """
    __slots__ = ("data", "scales", "K", "block", "pow2")

    def __init__(self, data, scales, K, block, pow2=False):
        self.data, self.scales, self.K, self.block, self.pow2 = data, scales, K, block, pow2

    @property
    def values(self):
        """The codes as torch's float8 values, (rows, K)."""
        import torch
        return self.data.view(torch.float8_e4m3fn)[:, :self.K]

    def __repr__(self):
        return (f"BlockScaled({self.data.shape[0]} x {self.K}, block={self.block!r}, "
                f"pow2={self.pow2}, {self.data.device})")


def block_quantize(x, block="row", transposed=False, pow2=False):
    """x (rows, cols), float32 or bfloat16 with packed rows, as BlockScaled: of each block the
    scale amax / 448 (at least 2^-126; with pow2 the smallest power of two that is not below it;
    NaN where the block holds an infinity or a NaN), and the codes of x / scale, rounded to nearest
    even.  block: "row" (1 x 128) or "tile" (128 x 128).  transposed: False for x, True for its
    transpose (cols, rows), "both" for the pair of them from one read of x."""
    if transposed not in (False, True, "both"):
        raise ValueError(f'transposed must be False, True or "both"; got {transposed!r}')
    both, pow2 = transposed == "both", bool(pow2)
    data, scales, data_t, scales_t = _binding().block_quantize(
        x, block, both or not transposed, both or bool(transposed), pow2)
    rows, cols = x.shape
    one = BlockScaled(data, scales, cols, block, pow2) if data is not None else None
    other = BlockScaled(data_t, scales_t, rows, block, pow2) if data_t is not None else None
    return (one, other) if one and other else one or other


def block_gemm(a, b, out_dtype="bf16", bias_col=None, source=None, out=None, exact=False):
    """C (M, N) = A B^T + bias_col + source of BlockScaled operands a (M, K), scaled per row and
    block of 128, and b (N, K), scaled per row or per tile.  bias_col: N float32; source: (M, N)
    float32 or bfloat16, packed, possibly `out` itself (but not otherwise overlapping it).  out_dtype: "bf16" or "f32", or that of
    `out`, which is written where it is given.  Sums are float32, rounded once; for a bfloat16 C of
    more than 32 rows the matrix instructions keep 13 binary places of eight neighbouring products
    below the largest (1.5e-5 of C on normal data), for a float32 C 24.  exact: 24 for a bfloat16 C of
    any number of rows too, at about half the speed -- for sums whose terms cancel, and where a row is to have
    the places that it has in a smaller batch."""
    for what, q in (("a", a), ("b", b)):
        if not isinstance(q, BlockScaled):
            raise ValueError(f"{what} must be a BlockScaled")
    if a.K != b.K:
        raise ValueError(f"a and b must have the same K; got {a.K} and {b.K}")
    if out is None and out_dtype not in ("bf16", "f32"):
        raise ValueError(f'out_dtype must be "bf16" or "f32"; got {out_dtype!r}')
    return _binding().block_gemm(a.data, a.scales, a.block, b.data, b.scales, b.block, a.K,
                                 bool(a.pow2 and b.pow2), out_dtype == "f32", bias_col, source, out,
                                 bool(exact))


# ---- layer norm -------------------------------------------------------------------------------

def layer_norm(x, weight, bias=None, eps=1e-5):
    """(y, mean, rstd) of x (rows, cols), float32 or bfloat16 with packed rows: each row less its
    mean, times rstd = 1 / sqrt(variance + eps), times weight, plus bias.  weight and bias (cols)
    are float32 or of x's type; y has x's type, mean and rstd are float32 (rows)."""
    return _binding().layer_norm(x, weight, bias, eps)


def layer_norm_backward(dy, x, weight, mean, rstd):
    """(dx, dweight, dbias) of layer_norm for the gradient dy of its y; mean and rstd are what it
    returned.  dx has x's type, dweight and dbias the weight's, summed over the rows in float32."""
    return _binding().layer_norm_backward(dy, x, weight, mean, rstd)


# ---- gradient clipping ------------------------------------------------------------------------

def grad_norm(grads):
    """The 2-norm of all elements of a list of gradients (float32 or bfloat16, packed, on one
    GPU), as a float32 tensor of no dimension.  Squares are summed in float64."""
    return _binding().norm(grads, None, None)


def clip_grad_norm(grads, max_norm, out=None):
    """Scales a list of gradients by min(1, max_norm / (norm + 1e-6)), in place or into the tensors
    `out` (one of each gradient's type and size), and returns the norm before that, as grad_norm.  What
    is written for one gradient must not overlap another one (a gradient that is in the list twice)."""
    return _binding().norm(grads, out, max_norm)
