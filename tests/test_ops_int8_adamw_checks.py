"""What the int8 operators and the AdamW step refuse, on CPU tensors and through the C ABI with calls that
return before anything is enqueued; their ctypes mirrors; the state of a list."""
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
P = 1 << 20   # an aligned address that no call here reads: each is refused first
INV, ALI, UNS, WSP = (L.GEMM_ERR_INVALID_ARG, L.GEMM_ERR_ALIGNMENT, L.GEMM_ERR_UNSUPPORTED,
                      L.GEMM_ERR_WORKSPACE)


def refused(match, fn, *a, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


def test_layouts(tmp_path):
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "gemm_ops.h"', 'int main(void){']
    structs = {"gemm_int8_desc": O.GemmInt8Desc, "gemm_adamw_tensor": O.GemmAdamwTensor,
               "gemm_adamw_desc": O.GemmAdamwDesc}
    for c, py in structs.items():
        lines.append(f'printf("{c} %zu\\n", sizeof({c}));')
        lines += [f'printf("{c}.{f} %zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0;}"]))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    out = dict(s.split() for s in subprocess.run([str(exe)], capture_output=True, text=True,
                                                 check=True).stdout.splitlines())
    for c, py in structs.items():
        assert int(out[c]) == ctypes.sizeof(py)
        for f, _ in py._fields_:
            assert int(out[f"{c}.{f}"]) == getattr(py, f).offset


def test_quantize_refusals():
    x = torch.zeros(40, 200)
    refused("on cpu", dg.int8_quantize, x)
    refused("must be a torch tensor", dg.int8_quantize, [1.0])
    refused("float32 or bfloat16 matrix", dg.int8_quantize, x.half())
    refused("float32 or bfloat16 matrix", dg.int8_quantize, x[0])
    refused("packed rows", dg.int8_quantize, x.t())
    refused("do not overlap", dg.int8_quantize, torch.as_strided(x, (40, 100), (50, 1)))
    refused("transposed must be", dg.int8_quantize, x, transposed="yes")
    refused("negated", dg.int8_quantize, torch._neg_view(x))
    refused("strided", dg.int8_quantize, torch.eye(40).to_sparse())


def scaled(rows, K):
    return dg.Int8Scaled(torch.zeros(rows, R.up(K, 16) * 16, dtype=torch.int8), torch.ones(rows), K)


def test_product_refusals():
    a, b = scaled(300, 200), scaled(150, 200)
    refused("on cpu", dg.int8_gemm, a, b)
    refused("a must be an Int8Scaled", dg.int8_gemm, a.data, b)
    refused("b must be an Int8Scaled", dg.int8_gemm, a, dg.BlockScaled(b.data, b.scales, 200, "row"))
    refused("the same K", dg.int8_gemm, a, scaled(150, 201))
    refused("out_dtype must be", dg.int8_gemm, a, b, out_dtype="e4m3")
    for what, value, match in (("data", a.data.to(torch.uint8), "a.data must be int8 codes"),
                               ("data", a.data[:, :199], "a.data must be int8 codes"),
                               ("data", a.data[0], "a.data must be int8 codes"),
                               ("data", torch.zeros(208, 300, dtype=torch.int8).t(), "packed rows"),
                               ("data", torch.zeros(300, 216, dtype=torch.int8)[:, :208], "multiples of 16"),
                               ("scales", torch.ones(299), "a.scales must be a packed vector of 300"),
                               ("scales", torch.ones(300).double(), "a.scales must be a packed vector"),
                               ("scales", torch.ones(600)[::2], "a.scales must be a packed vector"),
                               ("scales", torch._neg_view(a.scales), "negated")):
        bad = scaled(300, 200)
        setattr(bad, what, value)
        refused(match, dg.int8_gemm, bad, b)
    b.data = b.data.to("meta")
    refused("a is on cpu", dg.int8_gemm, a, b)


def test_state_of_a_list():
    params = [torch.zeros(5, 30), torch.zeros(0), torch.zeros(128, dtype=BF16), torch.zeros(129)]
    s = dg.adamw_state(params)
    assert s.m.shape == s.v.shape == (640,) and s.m.dtype == torch.float8_e4m3fn
    assert s.m_scales.shape == s.v_scales.shape == (5,)
    assert not bool(s.m.view(torch.uint8).any()) and not bool(s.v.view(torch.uint8).any())
    m, v = s.moments()
    assert m.dtype == v.dtype == torch.float32 and not bool(m.any()) and not bool(v.any())
    f = dg.adamw_state(iter(params), "f32")
    assert f.m.shape == (640,) and f.m.dtype == torch.float32 and f.m_scales is None
    assert f.moments()[1] is f.v
    refused("dtype must be", dg.adamw_state, params, "bf16")
    refused("empty", dg.adamw_state, [])


def test_step_refusals():
    p, d = torch.zeros(300), torch.zeros(300)
    s = dg.adamw_state([p])
    step = lambda *a, **kw: dg.adamw_step(*a, **kw)   # noqa: E731
    refused("parameter 0 is on cpu", step, [p], [d], s, 1, 1e-3)
    refused("parameter 0 is on cpu", step, (x for x in [p]), (x for x in [d]), s, 1, 1e-3)
    refused("list of parameters is empty", step, [], [], s, 1, 1e-3)
    refused("2 gradients for 1", step, [p], [d, d], s, 1, 1e-3)
    refused("1 gradients and 2 copies for 1", step, [p], [d], s, 1, 1e-3, copies=[None, None])
    refused("parameter 0 must be a torch tensor", step, [1.0], [d], s, 1, 1e-3)
    refused("gradient 0 must be a torch tensor", step, [p], [None], s, 1, 1e-3)
    refused("parameter 0 must be packed", step, [p.half()], [d], s, 1, 1e-3)
    refused("parameter 0 must be packed", step, [torch.zeros(10, 30).t()], [d], s, 1, 1e-3)
    refused("gradient 0 must be packed", step, [p], [d.half()], s, 1, 1e-3)
    refused("gradient 0 must be packed", step, [p], [d[:299]], s, 1, 1e-3)
    refused("gradient 0 must be packed", step, [p], [d.view(300, 1)], s, 1, 1e-3)
    refused("negated", step, [p], [torch._neg_view(d)], s, 1, 1e-3)
    refused("strided", step, [torch.eye(4).to_sparse()], [d], s, 1, 1e-3)
    refused("state must be an AdamWState", step, [p], [d], (s.m, s.v), 1, 1e-3)


def test_c_abi_refusals():
    lib = O.load()
    f32, bf16, e4m3 = L.GEMM_F32, L.GEMM_BF16, L.GEMM_FP8_E4M3

    def quant(x=P, dtype=f32, rows=30, cols=200, stride=200, codes=P, pitch=208, scales=P, codes_t=P,
              pitch_t=32, scales_t=P, ws=P, n=1 << 40):
        return lib.gemm_int8_quantize(x, dtype, rows, cols, stride, codes, pitch, scales, codes_t, pitch_t,
                                      scales_t, ws, n, None)

    for kw, want in ((dict(rows=-1), INV), (dict(cols=-1), INV), (dict(dtype=1), INV),
                     (dict(codes=None, codes_t=None), INV), (dict(x=None), INV), (dict(scales=None), INV),
                     (dict(scales_t=None), INV), (dict(stride=199), INV), (dict(stride=-1), INV),
                     (dict(pitch=200), INV), (dict(pitch=224), INV), (dict(pitch=192), INV),
                     (dict(pitch_t=16), INV), (dict(x=P + 2), ALI), (dict(codes=P + 8), ALI),
                     (dict(codes_t=P + 8), ALI), (dict(scales=P + 2), ALI), (dict(ws=P + 2), ALI),
                     (dict(rows=3000, pitch_t=3008, ws=None), WSP),
                     (dict(rows=3000, pitch_t=3008, n=100), WSP), (dict(rows=0), 0), (dict(cols=0), 0),
                     (dict(rows=1 << 31, cols=1 << 31, stride=1 << 31), UNS),
                     (dict(rows=1 << 23, codes_t=None, pitch=208), UNS)):
        assert quant(**kw) == want, kw
    # 30 x 200 fp32 at P, and what is written, each at a place of its own or on another's last bytes
    apart = dict(codes=P + (1 << 16), scales=P + (2 << 16), codes_t=P + (3 << 16), scales_t=P + (4 << 16),
                 ws=P + (5 << 16))
    if not torch.cuda.is_available():
        assert quant(**apart) == L.GEMM_ERR_HIP
    for kw in (dict(codes=P + 29 * 800 + 784), dict(codes=P - 30 * 208 + 16), dict(scales=P + 23996),
               dict(codes_t=P + 23984), dict(scales_t=P - 796), dict(codes_t=P + (1 << 16) + 29 * 208),
               dict(scales=P + (3 << 16) + 6396), dict(scales_t=P + (2 << 16) + 116)):
        assert quant(**{**apart, **kw}) == INV, kw
    assert quant(rows=3000, pitch_t=3008, **{**apart, "codes": P + (1 << 26), "ws": P + 30}) == ALI
    far = dict(codes=P + (1 << 26), scales=P + (2 << 26), codes_t=P + (3 << 26), scales_t=P + (4 << 26))
    assert quant(rows=3000, pitch_t=3008, ws=P + 2399996, **far) == INV   # x and the workspace
    n = ctypes.c_size_t()
    assert lib.gemm_int8_quantize_workspace(30, 200, 1, 0, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.gemm_int8_quantize_workspace(3000, 200, 1, 1, ctypes.byref(n)) == 0 and n.value > 0
    assert lib.gemm_int8_quantize_workspace(30, 200, 0, 0, ctypes.byref(n)) == INV
    assert lib.gemm_int8_quantize_workspace(30, 200, 1, 1, None) == INV

    far = 1 << 30

    def product(A=P, sa=P, B=P, sb=P, C=far, ws=None, n=0, bias=None, source=None, **kw):
        d = dict(M=100, N=90, K=300, lda=304, ldb=304, dtype_c=f32, dtype_source=f32)
        d.update(kw)
        return lib.gemm_int8_run(O.GemmInt8Desc(**d), A, sa, B, sb, C, bias, source, ws, n, None)

    for kw, want in ((dict(M=-1), INV), (dict(dtype_c=1), INV), (dict(dtype_source=1), INV),
                     (dict(lda=299), INV), (dict(lda=300), INV), (dict(A=None), INV), (dict(C=None), INV),
                     (dict(sa=None), INV), (dict(sb=None), INV), (dict(A=P + 8), ALI),
                     (dict(C=far + 2), ALI), (dict(sa=P + 2), ALI), (dict(bias=P + 2), ALI),
                     (dict(source=P + 2), ALI), (dict(lda=1 << 23), UNS), (dict(M=0), 0), (dict(N=0), 0),
                     (dict(K=1 << 18, lda=1 << 18, ldb=1 << 18), WSP),
                     (dict(K=1 << 18, lda=1 << 18, ldb=1 << 18, ws=P, n=1000), WSP),
                     (dict(ws=P + 4), ALI), (dict(source=far + 4), INV), (dict(bias=far), INV),
                     (dict(sa=far + 8), INV), (dict(sb=far + 100 * 90 * 4 - 4), INV),
                     (dict(A=far + 16), INV), (dict(source=far, dtype_source=bf16), INV)):
        assert product(**kw) == want, kw
    assert lib.gemm_int8_run(None, P, P, P, P, P, None, None, None, 0, None) == INV
    assert lib.gemm_int8_workspace(O.GemmInt8Desc(dtype_c=f32, dtype_source=f32), None) == INV

    a = [P + (i << 16) for i in range(8)]   # addresses that lie apart

    def step(param=a[0], grad=a[1], copy=a[2], numel=50, dtype=f32, dtype_grad=f32, count=1, **kw):
        t = O.GemmAdamwTensor(param, grad, copy, numel, dtype, dtype_grad)
        d = dict(m=a[3], v=a[4], m_scales=a[5], v_scales=a[6], step=1, lr=1e-3, beta1=0.9, beta2=0.99,
                 eps=1e-8, weight_decay=0.1, max_norm=1.0, dtype_state=e4m3)
        d.update(kw)
        return lib.gemm_adamw_step(ctypes.byref(t), count, ctypes.byref(O.GemmAdamwDesc(**d)), None)

    nan, inf = float("nan"), float("inf")
    for kw, want in ((dict(param=None), INV), (dict(grad=None), INV), (dict(numel=-1), INV),
                     (dict(dtype=1), INV), (dict(dtype_grad=1), INV), (dict(m=None), INV),
                     (dict(v=None), INV), (dict(m_scales=None), INV), (dict(v_scales=None), INV),
                     (dict(dtype_state=bf16), INV), (dict(count=-1), INV), (dict(step=0), INV),
                     (dict(lr=nan), INV), (dict(beta1=1.0), INV), (dict(beta2=-0.1), INV),
                     (dict(beta1=nan), INV), (dict(eps=-1.0), INV), (dict(eps=inf), INV),
                     (dict(weight_decay=nan), INV), (dict(norm=a[7], max_norm=-1.0), INV),
                     (dict(norm=a[7], max_norm=nan), INV), (dict(numel=1 << 40), UNS),
                     (dict(param=a[0] + 2), ALI), (dict(grad=a[1] + 2), ALI), (dict(copy=a[2] + 1), ALI),
                     (dict(m=a[3] + 4), ALI), (dict(v=a[4] + 2, dtype_state=f32), ALI),
                     (dict(m_scales=a[5] + 2), ALI), (dict(lr_at=a[7] + 2), ALI),
                     (dict(step_at=a[7] + 4), ALI), (dict(grad=a[0]), INV), (dict(copy=a[0] + 100), INV),
                     (dict(v=a[3] + 64), INV), (dict(v_scales=a[5]), INV), (dict(norm=a[0] + 8), INV),
                     (dict(lr_at=a[3]), INV), (dict(step_at=a[2] + 8), INV), (dict(count=0), 0),
                     (dict(numel=0), 0), (dict(numel=0, grad=a[0]), 0)):
        assert step(**kw) == want, kw
    assert lib.gemm_adamw_step(None, 1, ctypes.byref(O.GemmAdamwDesc()), None) == INV
    assert lib.gemm_adamw_step(None, 0, None, None) == INV


def test_long_sums_are_cut_at_any_size():
    """K past 130944 always goes to int32 pieces of at most that, whatever the number of tiles."""
    lib = O.load()
    n = ctypes.c_size_t()
    for K in (130945, 262144, 540000, 600000, 1000000, 2100000, 3000000, 1 << 22):
        pieces = -(-K // (1023 * 128))
        for M, N in ((1, 1), (32, 5000), (33, 64), (300, 300), (1900, 2000), (2048, 2048), (9000, 7000)):
            d = O.GemmInt8Desc(M=M, N=N, K=K, lda=1 << 22, ldb=1 << 22, dtype_c=2, dtype_source=2)
            assert lib.gemm_int8_workspace(ctypes.byref(d), ctypes.byref(n)) == 0
            assert n.value >= pieces * M * N * 4, (M, N, K)
    # what adds the pieces has a workgroup for 1024 elements, and a launch under 2^32 work-items
    d = O.GemmInt8Desc(M=1 << 16, N=1 << 16, K=1 << 18, lda=1 << 18, ldb=1 << 18, dtype_c=2, dtype_source=2)
    assert lib.gemm_int8_workspace(ctypes.byref(d), ctypes.byref(n)) == UNS
    d.K = d.lda = d.ldb = 1 << 16
    assert lib.gemm_int8_workspace(ctypes.byref(d), ctypes.byref(n)) == 0 and n.value == 0


@pytest.mark.parametrize("count", [2, 40])
def test_overlaps_in_any_order(count):
    """Tensors in any order of addresses; one that overlaps another anywhere in the list is found."""
    lib = O.load()
    g = torch.Generator().manual_seed(count)
    order = torch.randperm(3 * count, generator=g).tolist()
    state = P + (1 << 30)

    def step(change=None):
        at = [P + 4096 * i for i in order]
        ts = [O.GemmAdamwTensor(at[3 * i], at[3 * i + 1], at[3 * i + 2], 1000, 2, 2) for i in range(count)]
        if change:
            change(ts)
        d = O.GemmAdamwDesc(m=state, v=state + (1 << 20), step=1, lr=1e-3, beta1=0.9, beta2=0.99,
                            dtype_state=2)
        return lib.gemm_adamw_step((O.GemmAdamwTensor * count)(*ts), count, ctypes.byref(d), None)

    for change in (lambda t: setattr(t[-1], "param", t[0].param),
                   lambda t: setattr(t[-1], "param", t[0].grad + 3996),
                   lambda t: setattr(t[0], "copy", t[-1].copy + 1998),
                   lambda t: setattr(t[0], "copy", t[0].param),
                   lambda t: setattr(t[-1], "copy", state + 512 * count),
                   lambda t: setattr(t[0], "grad", t[-1].copy - 3996)):
        assert step(change) == INV
    # nothing there is refused in a list that lies apart; without a GPU its launch fails instead
    if not torch.cuda.is_available():
        assert step() == L.GEMM_ERR_HIP
        assert step(lambda t: setattr(t[-1], "grad", t[0].grad)) == L.GEMM_ERR_HIP   # read twice


def test_names_are_public():
    import dense_gemm_design_amd as pkg
    for name in ("int8_quantize", "int8_gemm", "Int8Scaled", "adamw_state", "adamw_step", "AdamWState"):
        assert getattr(pkg, name).__doc__
    text = open(os.path.join(ROOT, "include", "gemm_ops.h")).read()
    head = text[:text.index("#ifndef")]
    for name in re.findall(r"^int (gemm_\w+)\(", text, re.M):
        if not name.endswith("workspace"):
            assert name in head, name
