"""What the operators around the product refuse, on CPU tensors and through the C ABI with calls that
return before anything is enqueued; the header and its ctypes mirrors; the tests' own plain forms."""
import ctypes
import os
import re
import subprocess

import pytest

torch = pytest.importorskip("torch")

import dense_gemm_design_amd as dg  # noqa: E402
import ops_ref as R  # noqa: E402
from dense_gemm_design_amd import _lib as L  # noqa: E402
from dense_gemm_design_amd import ops as O  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16 = torch.bfloat16


def refused(match, fn, *a, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


def test_exports_and_layouts(tmp_path):
    text = open(os.path.join(ROOT, "include", "gemm_ops.h")).read()
    names = re.findall(r"^\s*int\s*(gemm_\w+)\s*\(", text, re.M)
    assert sorted(names) == sorted(O.EXPORTS)
    lib = O.load()
    for name in names:
        assert hasattr(lib, name), name
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "gemm_ops.h"', 'int main(void){']
    structs = {"gemm_block_desc": O.GemmBlockDesc, "gemm_tensor": O.GemmTensor}
    for c, py in structs.items():
        lines.append(f'printf("{c} %zu\\n", sizeof({c}));')
        lines += [f'printf("{c}.{f} %zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0;}"]))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)],
                   check=True)
    out = dict(s.split() for s in subprocess.run([str(exe)], capture_output=True, text=True,
                                                 check=True).stdout.splitlines())
    for c, py in structs.items():
        assert int(out[c]) == ctypes.sizeof(py)
        for f, _ in py._fields_:
            assert int(out[f"{c}.{f}"]) == getattr(py, f).offset


def test_quantize_refusals():
    x = torch.zeros(40, 200)
    refused("on cpu", dg.block_quantize, x)
    refused("must be a torch tensor", dg.block_quantize, [1.0])
    refused("float32 or bfloat16 matrix", dg.block_quantize, x.half())
    refused("float32 or bfloat16 matrix", dg.block_quantize, x[0])
    refused("packed rows", dg.block_quantize, x.t())
    refused("do not overlap", dg.block_quantize, torch.as_strided(x, (40, 100), (50, 1)))
    refused("block must be", dg.block_quantize, x, "column")
    refused("transposed must be", dg.block_quantize, x, transposed="yes")


def scaled(rows, K, block="row", pow2=False):
    sr = rows if block == "row" else R.up(rows, 128)
    return dg.BlockScaled(torch.zeros(rows, R.up(K, 16) * 16, dtype=torch.uint8),
                          torch.ones(R.up(K, 128), sr).t(), K, block, pow2)


def test_product_refusals():
    a, b = scaled(300, 200), scaled(150, 200, "tile")
    refused("on cpu", dg.block_gemm, a, b)
    refused("a must be a BlockScaled", dg.block_gemm, a.data, b)
    refused("the same K", dg.block_gemm, a, scaled(150, 201))
    refused('must have block "row"', dg.block_gemm, b, a)
    refused("out_dtype must be", dg.block_gemm, a, b, out_dtype="e4m3")
    refused("bias_col must be", dg.block_gemm, a, b, bias_col=torch.zeros(151))
    refused("bias_col must be", dg.block_gemm, a, b, bias_col=torch.zeros(150, dtype=BF16))
    refused("source must be", dg.block_gemm, a, b, source=torch.zeros(150, 300))
    refused("source must be", dg.block_gemm, a, b, source=torch.zeros(150, 300).t())
    refused("out must be", dg.block_gemm, a, b, out=torch.zeros(300, 150, dtype=torch.half))
    for field, value, match in (("block", "column", "block must be"),
                                ("data", a.data[:, :200], "codes"),
                                ("data", a.data.float(), "codes"),
                                ("scales", a.scales[:, :1], "scales must be"),
                                ("scales", a.scales.double(), "scales must be"),
                                ("scales", a.scales.contiguous(), "one block column"),
                                ("data", torch.zeros(208, 300, dtype=torch.uint8).t(), "packed rows"),
                                ("data", torch.zeros(300, 209, dtype=torch.uint8)[:, :208],
                                 "packed rows")):
        bad = scaled(300, 200)
        setattr(bad, field, value)
        refused(match, dg.block_gemm, bad, b)


def test_norm_refusals():
    x, w = torch.zeros(40, 200), torch.ones(200)
    m = torch.zeros(40)
    refused("on cpu", dg.layer_norm, x, w)
    refused("no elements", dg.layer_norm, x[:, :0], w[:0])
    refused("packed rows", dg.layer_norm, x.t(), torch.ones(40))
    refused("weight must be", dg.layer_norm, x, w[:199])
    refused("weight must be", dg.layer_norm, x, w.to(BF16))
    refused("weight must be", dg.layer_norm, x, torch.ones(400)[::2])
    refused("bias must be", dg.layer_norm, x.to(BF16), w, w.to(BF16))
    refused("on cpu", dg.layer_norm_backward, x, x, w, m, m)
    refused("dy must be", dg.layer_norm_backward, x[:39], x, w, m, m)
    refused("dy must be", dg.layer_norm_backward, x.to(BF16), x, w, m, m)
    refused("mean must be", dg.layer_norm_backward, x, x, w, m[:39], m)
    refused("rstd must be", dg.layer_norm_backward, x, x, w, m, m.to(BF16))


def test_clip_refusals():
    g = torch.zeros(10)
    refused("list of gradients is empty", dg.grad_norm, [])
    refused("gradient 0 is on cpu", dg.grad_norm, [g])
    refused("gradient 0 must be packed", dg.clip_grad_norm, [g.half()], 1.0)
    refused("gradient 0 must be packed", dg.clip_grad_norm, [torch.zeros(10, 4).t()], 1.0)
    refused("must be a torch tensor", dg.grad_norm, [1.0])
    refused("max_norm must not be", dg.clip_grad_norm, [g], -1.0)
    refused("max_norm must not be", dg.clip_grad_norm, [g], float("nan"))
    refused("out has 2 tensors for 1", dg.clip_grad_norm, [g], 1.0, out=[g, g])


P = 1 << 20   # an aligned address that no call here reads: each is refused first


def test_c_abi_refusals():
    lib = O.load()
    inv, ali, uns, wsp = (L.GEMM_ERR_INVALID_ARG, L.GEMM_ERR_ALIGNMENT, L.GEMM_ERR_UNSUPPORTED,
                          L.GEMM_ERR_WORKSPACE)
    f32, bf16 = L.GEMM_F32, L.GEMM_BF16
    q = lib.gemm_block_quantize

    def quant(x=P, dtype=f32, rows=30, cols=200, stride=200, block=0, codes=P, pitch=208, scales=P,
              sp=30, codes_t=P, pitch_t=32, scales_t=P, spt=200):
        return q(x, dtype, rows, cols, stride, block, 0, codes, pitch, scales, sp, codes_t, pitch_t,
                 scales_t, spt, None)

    for kw, want in ((dict(rows=-1), inv), (dict(dtype=1), inv), (dict(block=2), inv),
                     (dict(codes=None, codes_t=None), inv), (dict(x=None), inv),
                     (dict(scales=None), inv), (dict(scales_t=None), inv), (dict(stride=199), inv),
                     (dict(stride=-1), inv), (dict(pitch=200), inv), (dict(pitch=224), inv),
                     (dict(pitch=192), inv), (dict(pitch_t=16), inv), (dict(sp=29), inv),
                     (dict(x=P + 2), ali), (dict(codes=P + 8), ali), (dict(codes_t=P + 8), ali),
                     (dict(scales=P + 2), ali), (dict(rows=0), 0), (dict(cols=0), 0)):
        assert quant(**kw) == want, kw

    def product(A=P, C=P, ws=None, n=0, bias=None, source=None, **kw):
        d = dict(M=100, N=90, K=300, lda=304, ldb=304, scale_lda=100, scale_ldb=90, block_b=0,
                 pow2=0, dtype_c=f32, dtype_source=f32)
        d.update(kw)
        return lib.gemm_block_run(O.GemmBlockDesc(**d), A, P, P, P, C, bias, source, ws, n, None)

    for kw, want in ((dict(M=-1), inv), (dict(block_b=2), inv), (dict(dtype_c=1), inv),
                     (dict(dtype_source=1), inv), (dict(lda=299), inv), (dict(lda=300), inv),
                     (dict(scale_lda=99), inv), (dict(scale_ldb=89), inv), (dict(A=None), inv),
                     (dict(C=None), inv), (dict(A=P + 8), ali), (dict(C=P + 2), ali),
                     (dict(bias=P + 2), ali), (dict(source=P + 2), ali),
                     (dict(lda=1 << 23), uns), (dict(M=0), 0), (dict(N=0), 0),
                     (dict(K=9000, lda=9008, ldb=9008), wsp),
                     (dict(K=9000, lda=9008, ldb=9008, ws=P, n=1000), wsp),
                     (dict(K=9000, lda=9008, ldb=9008, ws=P + 4, n=1 << 40), ali)):
        assert product(**kw) == want, kw
    assert lib.gemm_block_run(None, P, P, P, P, P, None, None, None, 0, None) == inv
    assert lib.gemm_block_workspace(O.GemmBlockDesc(), None) == inv

    def norm(x=P, dtype=bf16, rows=5, cols=70, stride=70, w=P, b=P, wtype=f32, y=P, mean=P, rstd=P):
        return lib.gemm_layer_norm(x, dtype, rows, cols, stride, w, b, wtype, 1e-5, y, mean, rstd,
                                   None)

    for kw, want in ((dict(rows=-1), inv), (dict(cols=0), inv), (dict(dtype=1), inv),
                     (dict(dtype=f32, wtype=bf16), inv), (dict(stride=69), inv), (dict(x=None), inv),
                     (dict(w=None), inv), (dict(y=None), inv), (dict(mean=None), inv),
                     (dict(rstd=None), inv), (dict(x=P + 1), ali), (dict(w=P + 2), ali),
                     (dict(b=P + 2), ali), (dict(rows=0), 0)):
        assert norm(**kw) == want, kw

    def back(dy=P, ds=70, x=P, stride=70, dtype=bf16, rows=5, cols=70, w=P, wtype=f32, mean=P,
             dx=P, dw=P, ws=P, n=1 << 40):
        return lib.gemm_layer_norm_backward(dy, ds, x, stride, dtype, rows, cols, w, wtype, mean, P,
                                            dx, dw, P, ws, n, None)

    for kw, want in ((dict(rows=-1), inv), (dict(cols=0), inv), (dict(ds=69), inv),
                     (dict(stride=69), inv), (dict(dy=None), inv), (dict(x=None), inv),
                     (dict(mean=None), inv), (dict(dx=None), inv), (dict(dw=None), inv),
                     (dict(w=None), inv), (dict(dx=P + 1), ali), (dict(dw=P + 2), ali),
                     (dict(ws=None), wsp), (dict(n=100), wsp), (dict(ws=P + 4), ali)):
        assert back(**kw) == want, kw

    def clip(data=P, out=P, numel=50, dtype=f32, max_norm=1.0, norm=P, ws=P, n=1 << 40):
        t = O.GemmTensor(data, out, numel, dtype)
        return lib.gemm_clip_grad_norm(ctypes.byref(t), 1, max_norm, norm, ws, n, None)

    for kw, want in ((dict(data=None), inv), (dict(out=None), inv), (dict(numel=-1), inv),
                     (dict(dtype=1), inv), (dict(max_norm=-1.0), inv), (dict(norm=None), inv),
                     (dict(max_norm=float("nan")), inv), (dict(data=P + 2), ali),
                     (dict(numel=1 << 40), uns), (dict(ws=None), wsp), (dict(n=4), wsp),
                     (dict(ws=P + 4), ali)):
        assert clip(**kw) == want, kw
    assert lib.gemm_grad_norm(None, 3, P, P, 1 << 40, None) == inv


def test_c_abi_limits():
    """Sizes whose offsets or launches would pass 32 bits are refused."""
    lib = O.load()
    n = ctypes.c_size_t()
    uns = L.GEMM_ERR_UNSUPPORTED
    d = dict(M=1, N=1, K=16, lda=16, ldb=16, scale_lda=1, scale_ldb=1, dtype_c=2, dtype_source=2)
    for kw, want in ((dict(N=1 << 22), 0), (dict(N=(1 << 22) + 1), uns), (dict(M=(1 << 31) + 1), uns),
                     (dict(lda=(1 << 22) + 16), uns), (dict(M=1 << 30, N=1 << 21), uns)):
        assert lib.gemm_block_workspace(O.GemmBlockDesc(**{**d, **kw}), ctypes.byref(n)) == want, kw
    assert lib.gemm_layer_norm_backward_workspace(1, 1 << 24, ctypes.byref(n)) == 0
    assert lib.gemm_layer_norm_backward_workspace(1, (1 << 24) + 1, ctypes.byref(n)) == uns
    c = (1 << 24) + 1
    assert lib.gemm_layer_norm(P, 2, 1, c, c, P, P, 2, 1e-5, P, P, P, None) == uns
    assert lib.gemm_layer_norm_backward(P, c, P, c, 2, 1, c, P, 2, P, P, P, P, P, P, 1 << 50,
                                        None) == uns
    big = 1 << 20
    assert lib.gemm_block_quantize(P, 2, big * 128, big * 128, big * 128, 0, 0, P, big * 128, P,
                                   big * 128, None, 0, None, 0, None) == uns


def test_workspaces_cover_their_sums():
    lib = O.load()
    n = ctypes.c_size_t()
    for rows, cols in ((1, 1), (5, 70), (3000, 4096), (100000, 33), (10, 50000)):
        assert lib.gemm_layer_norm_backward_workspace(rows, cols, ctypes.byref(n)) == 0
        assert n.value % (8 * cols) == 0 and 1 <= n.value // (8 * cols) <= rows
    for sizes in ([0], [1], [16384], [16385], [1] * 129, [10 ** 9] * 3):
        arr = (O.GemmTensor * len(sizes))(*[O.GemmTensor(P, P, s, 2) for s in sizes])
        assert lib.gemm_grad_norm_workspace(arr, len(sizes), ctypes.byref(n)) == 0
        assert n.value <= 8 * sum(R.up(s, 2048) for s in sizes)
        assert (n.value == 0) == (sum(sizes) == 0)


def test_plain_quantiser_pins():
    """All codes survive, midpoints go to the even code, neighbours of midpoints to their side."""
    codes = torch.tensor([c for c in range(256) if c & 127 != 127], dtype=torch.uint8)
    v = R.decode(codes)
    assert torch.equal(R.encode(v), codes)
    assert torch.equal(v.float().to(torch.float8_e4m3fn).view(torch.uint8), codes)
    pos = v[:127]
    mids = (pos[1:] + pos[:-1]) / 2
    at = R.encode(mids).long()
    assert bool((at % 2 == 0).all()) and bool(((at == torch.arange(126)) |
                                               (at == torch.arange(1, 127))).all())
    assert torch.equal(R.encode(mids * (1 + 1e-12)).long(), torch.arange(1, 127))
    assert torch.equal(R.encode(mids * (1 - 1e-12)).long(), torch.arange(126))
    codes, scales = R.quantize(torch.tensor([[448.0, 1.0, 0.0, -224.0]]), "row", False)
    assert float(scales) == 1.0 and R.decode(codes)[0, :4].tolist() == [448.0, 1.0, 0.0, -224.0]
    for top, want in ((448.0, 1.0), (448.5, 2.0), (224.0, 0.5), (0.0, 2.0 ** -126)):
        assert float(R.quantize(torch.tensor([[top]]), "tile", True)[1]) == want
