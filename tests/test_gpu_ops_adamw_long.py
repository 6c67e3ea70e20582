"""The AdamW step of lists too long for the caches, which loads and stores past them, and with e4m3 states takes
chunks of twice the size: against its formula in 64 bits, computed on the GPU."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_design_amd as dg  # noqa: E402
import ops_ref as R  # noqa: E402
from test_gpu_ops import dev  # noqa: E402,F401

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U, HALF = R.U, R.HALF
LR, BETAS, EPS, DECAY = 3e-3, (0.9, 0.95), 1e-8, 0.1
PASSING, CHUNKS = 96 << 20, 4096 * 2048   # bytes and elements from which on the kernels go over


@pytest.fixture(scope="module", autouse=True)
def large_tensors_go_back():
    """What torch keeps of them for other tests' tensors would count as memory in use there."""
    yield
    torch.cuda.empty_cache()


def bytes_of(params, grads, copies, state):
    return sum(p.numel() * (2 * p.element_size() + g.element_size() + (4 if state == "e4m3" else 16)
                            + (2 if c is not None else 0)) for p, g, c in zip(params, grads, copies))


def within(got, want, bound, what):
    bad = ~((got.double() - want).abs() <= bound)
    if bool(bad.any()):
        i = int(bad.view(-1).nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {got.numel()} outside, first at {i}: "
                             f"{float(got[i])} for {float(want[i])} +- {float(bound[i])}")


def moments(state):
    """float64 (m, root of v)."""
    if state.m_scales is None:
        return state.m.double(), state.v.double().sqrt()
    return (c.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128)
            for c, s in ((state.m, state.m_scales), (state.v, state.v_scales)))


@pytest.mark.parametrize("state", ["e4m3", "f32"])
@pytest.mark.parametrize("large,grad,copied", [(BF16, BF16, False), (F32, BF16, True), (F32, F32, False),
                                               (BF16, F32, True)],
                         ids=["bf16-gbf16", "f32-gbf16-copies", "f32-gf32", "bf16-gf32-copies"])
@pytest.mark.parametrize("n", [4_400_003, 8_600_001, 13_000_001])
def test_long_lists(dev, n, large, grad, copied, state):
    """One tensor of n elements, which starts anywhere, and small ones beside it."""
    print(f"adamw {n} {large} {grad} {state}", flush=True)
    g = torch.Generator(device=dev).manual_seed(n)
    other = F32 if large == BF16 else BF16
    sizes = [(5, other), (n, large), (0, large), (2049, other), (127, large), (300_001, large)]
    params, grads, copies, held = [], [], [], []
    for i, (k, t) in enumerate(sizes):
        by = i % 4   # elements that the tensor starts behind a multiple of 16 bytes
        for kind, to, scale in ((t, params, 1.0), (grad, grads, 1e-2)):
            flat = torch.full((k + 64,), 3.0, dtype=kind, device=dev)
            flat[16 + by:16 + by + k] = torch.randn(k, generator=g, device=dev) * scale
            to.append(flat[16 + by:16 + by + k])
            held.append((flat, by, k))
        flat = torch.full((k + 64,), 3.0, dtype=BF16, device=dev)
        copies.append(flat[17 + by:17 + by + k] if copied and i != 3 else None)
        held.append((flat, by + 1, k if copied and i != 3 else 0))
    s = dg.adamw_state(params, state)
    for x in (s.m_scales, s.v_scales):
        if x is not None:   # a state in the middle of a run: of 1e-2 and less
            x.copy_(torch.exp(torch.randn(len(x), generator=g, device=dev)) * 1e-5)
    if state == "e4m3":
        s.m.view(torch.uint8).random_(0, 127, generator=g)
        s.v.view(torch.uint8).random_(1, 127, generator=g)
        assert n < CHUNKS or sum(k for k, _ in sizes) >= CHUNKS
    else:
        s.m.copy_(torch.randn(len(s.m), generator=g, device=dev) * 3e-3)
        s.v.copy_((torch.rand(len(s.v), generator=g, device=dev) * 1e-2).square())
    if n == 13_000_001:
        assert bytes_of(params, grads, copies, state) > PASSING
    m0, r0 = moments(s)
    raw = [x.clone().view(torch.uint8) for x in (s.m, s.v)]
    before = [p.double() for p in params]
    step = 7
    dg.adamw_step(params, grads, s, step, LR, betas=BETAS, eps=EPS, weight_decay=DECAY,
                  copies=copies if copied else None)
    m1, r1 = moments(s)
    b1, b2 = BETAS
    at = 0
    for i, (p, d, old) in enumerate(zip(params, grads, before)):
        k, d = p.numel(), d.double()
        blocks = R.up(k, 128)
        m, v = b1 * m0[at:at + k] + (1 - b1) * d, b2 * r0[at:at + k] ** 2 + (1 - b2) * d * d
        # in units of U: both factors and both products 4, decoding 1, m's fma one; v 16 as of a square of one more
        dm = U * ((b1 * m0[at:at + k]).abs() * 3 + ((1 - b1) * d).abs() * 3 + m.abs())
        root = v.sqrt()
        den = root / (1 - b2 ** step) ** 0.5 + EPS
        rate = LR / (1 - b1 ** step)
        way = rate * m / den
        want = old - (LR * DECAY * old + way)
        # the root 2 and half of v's 16, its factor 2, the sum 1, its reciprocal 2; the rate 2, two products 2;
        # the parameter's share of lr wd 4, its fma 1, the difference 1
        bound = 20 * U * way.abs() + rate * dm / den + U * (4 * LR * DECAY + 2) * old.abs() + 2 * U * want.abs()
        within(p, want, (bound + HALF[p.dtype] * want.abs()) * (1 + 2.0 ** -10) + 2.0 ** -140, f"parameter {i}")
        if copies[i] is not None:
            within(copies[i], want, (bound + HALF[BF16] * want.abs()) * (1 + 2.0 ** -10) + 2.0 ** -140, f"copy {i}")
        if state == "f32":
            within(m1[at:at + k], m, dm * (1 + 2.0 ** -10) + 2.0 ** -148, f"m {i}")
            within(r1[at:at + k] ** 2, v, U * 16 * v + 2.0 ** -148, f"v {i}")
        else:
            for x, dx, got, scales, least in ((m, dm, m1, s.m_scales, 0.5),
                                              (root, 10 * U * root, r1, s.v_scales, 1.0)):
                pad = torch.zeros(2, blocks * 128, dtype=torch.float64, device=dev)
                pad[0, :k], pad[1, :k] = x, dx
                top, slack = (t.view(-1, 128).abs().amax(1) for t in pad) if k else pad
                sc = scales[at // 128:at // 128 + blocks].double()
                # the scale: of the largest, off by what that is off, and its own rounding
                within(sc, (top / 448).clamp(min=2.0 ** -126), slack / 448 + 2 * U * top / 448, f"scales {i}")
                # half a step of e4m3, 2^-4 of a normal number and 2^-10 scales of others (a root that is not
                # zero may be moved to 2^-9); the quotient's own rounding shifts the border by 4 U
                each = sc.repeat_interleave(128)[:k]
                half = torch.maximum(x.abs() * 2.0 ** -4, each * 2.0 ** -9 * least)
                within(got[at:at + k], x, (half + dx) * (1 + 2.0 ** -18), f"codes {i}")
        # behind the tensor's end, which counts as zero: as it was, or zero
        for now, then in zip((s.m, s.v), raw):
            now, then = (x.view(len(s.m), -1)[at + k:at + blocks * 128] for x in (now.view(torch.uint8), then))
            assert bool(((now == then) | (now == 0)).all()), f"behind state {i}"
        at += blocks * 128
    for i, (flat, by, k) in enumerate(held):
        assert bool((flat[:16 + by] == 3).all()) and bool((flat[16 + by + k:] == 3).all()), f"beside tensor {i}"
