"""How the Python calls of the operators take their arguments (CPU: nothing here reaches a kernel)."""
import os
import subprocess
import sys

import pytest

np = pytest.importorskip("numpy")
torch = pytest.importorskip("torch")

import dense_gemm_design_amd as dg  # noqa: E402
from dense_gemm_design_amd import ops as O  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("transposed,sides", [(False, (True, False)), (True, (False, True)),
                                              ("both", (True, True)), (0, (True, False)),
                                              (1, (False, True)), (np.bool_(False), (True, False)),
                                              (np.bool_(True), (False, True))])
def test_quantise_takes_truth_values_of_any_type(monkeypatch, transposed, sides):
    """0, 1 and numpy's truth values ask for one side, as False and True do."""
    asked = []

    class Binding:
        @staticmethod
        def block_quantize(x, block, rows, cols, pow2):
            asked.append((rows, cols))
            return (x, x) * 2 if rows and cols else (x, x, None, None) if rows else (None, None, x, x)

    monkeypatch.setattr(O, "_binding", lambda: Binding)
    q = dg.block_quantize(torch.zeros(3, 5), transposed=transposed)
    assert asked == [sides] and all(type(s) is bool for s in asked[0])
    if sides == (True, True):
        assert isinstance(q, tuple) and (q[0].K, q[1].K) == (5, 3)
    else:
        assert isinstance(q, dg.BlockScaled) and q.K == (5 if sides[0] else 3)


@pytest.mark.parametrize("transposed", ["yes", "True", 2, None, (True,)])
def test_quantise_refuses_other_sides(transposed):
    with pytest.raises(ValueError, match="transposed must be"):
        dg.block_quantize(torch.zeros(3, 5), transposed=transposed)


def test_gradients_may_come_from_a_generator():
    """A generator can be read once: it gets as far as a list does, to the check of its tensors."""
    grads = [torch.zeros(3), torch.zeros(4)]
    for call in (lambda g: dg.grad_norm(g), lambda g: dg.clip_grad_norm(g, 1.0),
                 lambda g: dg.clip_grad_norm(g, 1.0, out=(t for t in grads))):
        for given in (grads, tuple(grads), (t for t in grads), iter(grads)):
            with pytest.raises(ValueError, match="gradient 0 is on cpu"):
                call(given)
    with pytest.raises(ValueError, match="out has 1 tensors for 2"):
        dg.clip_grad_norm((t for t in grads), 1.0, out=(t for t in grads[:1]))
    with pytest.raises(ValueError, match="the list of gradients is empty"):
        dg.grad_norm(t for t in grads[:0])
    with pytest.raises(TypeError, match="sequence of tensors"):
        dg.grad_norm(3)


def test_the_package_imports_without_torch():
    """Descriptors, constants and the build need no torch; what runs a kernel imports it by itself."""
    code = ("import sys; sys.modules['torch'] = None; import dense_gemm_design_amd as dg; "
            "print(dg.make_desc(256, 256, 256, dg.GEMM_BF16, dg.GEMM_F32).M, dg.BlockScaled.__name__)")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == ["256", "BlockScaled"]


def recorded_build(monkeypatch, torch_there, gxx_there):
    """The commands of a build, none of them run."""
    from dense_gemm_design_amd import build as B
    ran = []

    class Done:
        returncode = 0

    monkeypatch.setattr(B.subprocess, "run", lambda c, **kw: ran.append(c) or Done())
    monkeypatch.setattr(B.os, "replace", lambda a, b: None)
    monkeypatch.setattr(B.shutil, "which", lambda name: "/usr/bin/" + name if gxx_there else None)
    if not torch_there:
        monkeypatch.setitem(sys.modules, "torch", None)
    assert B.build() == B.LIB
    assert sum("-c" in c for c in ran) == len(B.SOURCES)
    return ran[len(B.SOURCES) + 1:]   # behind the library's link


@pytest.mark.parametrize("gxx_there", [True, False])
def test_the_library_builds_without_torch(monkeypatch, capsys, gxx_there):
    """hipcc alone makes the C library; only the Python binding needs torch's headers."""
    assert recorded_build(monkeypatch, False, gxx_there) == []
    assert "torch" in capsys.readouterr().out


@pytest.mark.parametrize("gxx_there", [True, False])
def test_the_binding_builds_without_gxx(monkeypatch, gxx_there):
    (cmd,) = recorded_build(monkeypatch, True, gxx_there)
    assert os.path.basename(cmd[0]) == ("g++" if gxx_there else "amdclang++")
    assert any(c.endswith("binding.cpp") for c in cmd)


def test_tensors_that_are_not_plain_memory_are_refused():
    """A lazily negated view holds the other sign in memory; a sparse tensor holds no rows."""
    x, w, m = torch.ones(40, 64), torch.ones(64), torch.ones(40)
    neg = lambda t: torch._neg_view(t)   # noqa: E731 -- what .imag of a conjugate is
    a = dg.BlockScaled(torch.zeros(40, 64, dtype=torch.uint8), torch.ones(1, 40).t(), 64, "row")
    calls = (lambda: dg.block_quantize(neg(x)), lambda: dg.layer_norm(neg(x), w),
             lambda: dg.layer_norm(x, neg(w)), lambda: dg.layer_norm(x, w, neg(w)),
             lambda: dg.layer_norm_backward(neg(x), x, w, m, m),
             lambda: dg.layer_norm_backward(x, x, w, neg(m), m), lambda: dg.grad_norm([neg(x)]),
             lambda: dg.clip_grad_norm([neg(x), x], 1.0),
             lambda: dg.block_gemm(a, a, source=neg(torch.ones(40, 40))),
             lambda: dg.block_gemm(a, a, out=neg(torch.ones(40, 40))),
             lambda: dg.block_gemm(dg.BlockScaled(a.data, neg(a.scales), 64, "row"), a))
    for call in calls:
        with pytest.raises(ValueError, match="negated"):
            call()
    sparse = torch.eye(40).to_sparse()
    for call in (lambda: dg.block_quantize(sparse), lambda: dg.layer_norm(sparse, m),
                 lambda: dg.grad_norm([sparse]), lambda: dg.block_gemm(a, a, source=sparse)):
        with pytest.raises(ValueError, match="strided"):
            call()
