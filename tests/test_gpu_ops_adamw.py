"""The AdamW step of a list of parameters against its formula in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_design_amd as dg  # noqa: E402
import ops_ref as R  # noqa: E402
from test_gpu_ops import dev, gen, randn  # noqa: E402,F401

pytestmark = pytest.mark.gpu
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = R.U
KEYS = dict(lr=3e-3, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)


def blocks_of(params):
    return [R.up(p.numel(), 128) for p in params]


def make_state(g, params, dtype, dev, size=1e-2):
    """A state in the middle of a run."""
    s = dg.adamw_state(params, dtype)
    at = 0
    for p, b in zip(params, blocks_of(params)):
        n = p.numel()
        root = torch.exp(randn(g, n)) * size
        m = randn(g, n) * root * 0.5
        if dtype == "f32":
            s.m[at:at + n], s.v[at:at + n] = m.to(dev), root.square().to(dev)
        else:
            held = torch.zeros(2, b * 128)
            held[0, :n], held[1, :n] = m, root
            scale = (held.view(2, b, 128).abs().amax(2) / 448).clamp(min=2.0 ** -126)
            q = (held.view(2, b, 128) / scale[:, :, None]).to(E4M3).view(2, -1)
            for mine, codes, sc, k in ((s.m, q[0], scale[0], 2), (s.v, q[1], scale[1], 3)):
                mine[at:at + b * 128].view(torch.uint8).copy_(codes.view(torch.uint8))
                (s.m_scales if k == 2 else s.v_scales)[at // 128:at // 128 + b] = sc.to(dev)
        at += b * 128
    return s


def clone(state):
    return dg.AdamWState(*(None if t is None else t.clone() for t in
                           (state.m, state.v, state.m_scales, state.v_scales)))


def values(state):
    """float64 (m, v) of a state on the CPU."""
    if state.m_scales is None:
        return state.m.double().cpu(), state.v.double().cpu()
    m, r = (c.view(torch.uint8).cpu() for c in (state.m, state.v))
    ms, vs = (s.cpu().double().repeat_interleave(128) for s in (state.m_scales, state.v_scales))
    return R.decode(m) * ms, (R.decode(r) * vs) ** 2


def step_and_check(params, grads, state, step, what, norm=None, max_norm=None, copies=None, **keys):
    keys = {**KEYS, **keys}
    t, lr = int(step), float(keys["lr"])
    b1, b2 = keys["betas"]
    before = [p.detach().double().cpu() for p in params]
    m0, v0 = values(state)
    codes0 = clone(state)
    dg.adamw_step(params, grads, state, step, norm=norm, max_norm=max_norm, copies=copies, **keys)
    c = 1.0 if norm is None else min(1.0, max_norm / (float(norm) + 1e-6))
    m1, v1 = values(state)
    e4m3 = state.m_scales is not None
    at = 0
    for i, (p, g, old, b) in enumerate(zip(params, grads, before, blocks_of(params))):
        n = p.numel()
        g = c * g.double().cpu().view(-1)
        old = old.view(-1)
        m, v = b1 * m0[at:at + n] + (1 - b1) * g, b2 * v0[at:at + n] + (1 - b2) * g * g
        # in units of U: g' 4 (the norm's sum, quotient, max_norm, product), both factors and both products 4
        # more, m's fma one; decoding an e4m3 moment 1
        dm = U * ((b1 * m0[at:at + n]).abs() * 3 + ((1 - b1) * g).abs() * 7 + m.abs())
        dv = U * 16 * v + 2.0 ** -148
        root = v.sqrt()
        den = root / (1 - b2 ** t) ** 0.5 + keys["eps"]
        rate = lr / (1 - b1 ** t)
        way = rate * m / den
        want = old - (lr * keys["weight_decay"] * old + way)
        # the root 2 and half of v's 16, its factor 2, the sum 1, its reciprocal 2; the rate 2, two products 2;
        # the parameter's share of lr wd 4, its fma 1, the difference 1
        bound = 20 * U * way.abs() + rate * dm / den + U * (
            4 * lr * abs(keys["weight_decay"]) + 2) * old.abs() + U * want.abs() * 2
        R.within(p.detach().view(-1), want, (bound + R.HALF[p.dtype] * want.abs()) * (1 + 2.0 ** -10)
                 + 2.0 ** -140, f"{what}: parameter {i}")
        if copies is not None and copies[i] is not None:
            R.within(copies[i].view(-1), want, (bound + R.HALF[BF16] * want.abs()) * (1 + 2.0 ** -10)
                     + 2.0 ** -140, f"{what}: copy {i}")
        if not e4m3:
            R.within(state.m[at:at + n], m, dm * (1 + 2.0 ** -10) + 2.0 ** -148, f"{what}: m {i}")
            R.within(state.v[at:at + n], v, dv * (1 + 2.0 ** -10), f"{what}: v {i}")
        else:
            for x, dx, got, sc, floor in ((m, dm, R.decode(state.m.view(torch.uint8)), state.m_scales, 0.5),
                                          (root, 10 * U * root + 2.0 ** -74, R.decode(
                                              state.v.view(torch.uint8)), state.v_scales, 1.0)):
                pad = torch.zeros(2, b * 128, dtype=torch.float64)
                pad[0, :n], pad[1, :n] = x, dx
                top, slack = pad[0].view(b, 128).abs().amax(1), pad[1].view(b, 128).amax(1)
                s = sc[at // 128:at // 128 + b].cpu().double()
                # the scale: of the largest, off by what that is off, one product and 1 / 448's rounding
                R.within(s, (top / 448).clamp(min=2.0 ** -126), slack / 448 + 3 * U * top / 448,
                         f"{what}: scales {i}")
                q = got[at:at + n] * s.repeat_interleave(128)[:n]
                # half a step of e4m3, 2^-4 of a normal number and 2^-10 scales of others (a root that is
                # not zero may be moved to 2^-9); the quotient's own rounding shifts the border by 4 U
                each = s.repeat_interleave(128)[:n]
                half = torch.maximum(x.abs() * 2.0 ** -4, each * 2.0 ** -9 * floor)
                R.within(q, x, (half + dx) * (1 + 2.0 ** -18), f"{what}: codes {i}")
                if floor == 1.0:
                    assert torch.equal(q > 0, x > 0), f"{what}: roots {i}"
        # behind the tensor's end
        for mine, other in ((state.m, codes0.m), (state.v, codes0.v)):
            assert torch.equal(mine.view(torch.uint8).view(len(mine), -1)[at + n:at + b * 128],
                               other.view(torch.uint8).view(len(mine), -1)[at + n:at + b * 128]), what
        at += b * 128


SIZES = [[1], [7], [128], [127, 129, 1], [2048], [2047, 2049], [5, 0, 300], [16385, 33], [70000, 3, 4096]]


@pytest.mark.parametrize("state", ["e4m3", "f32"])
@pytest.mark.parametrize("grad", [BF16, F32], ids=["gbf16", "gf32"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "-".join(map(str, s)))
def test_step(dev, sizes, dtype, grad, state):
    print(f"adamw {sizes} {dtype} {grad} {state}", flush=True)
    g = gen(sum(sizes))
    params = [randn(g, n).to(dtype).to(dev) for n in sizes]
    s = make_state(g, params, state, dev)
    for k in range(2):
        grads = [(randn(g, n) * 1e-2).to(grad).to(dev) for n in sizes]
        step_and_check(params, grads, s, 3 + k, f"step {3 + k}")


@pytest.mark.parametrize("state", ["e4m3", "f32"])
def test_first_steps_from_nothing(dev, state):
    """From zeros: the first step moves every parameter by lr and its decay, whatever its gradient's size."""
    g = gen(2)
    params = [randn(g, 300).to(dev), randn(g, 40, 70).to(dev)]
    grads = [(randn(g, *p.shape) * torch.exp(randn(g, *p.shape) * 2)).to(dev) for p in params]
    grads[0][:5] = 0
    s = dg.adamw_state(params, state)
    before = [p.clone() for p in params]
    step_and_check(params, grads, s, 1, "first", weight_decay=0.0)
    for p, b, d in zip(params, before, grads):
        moved = (b - p).double()
        want = 3e-3 * torch.sign(d.double())
        # m / (1 - b1) and sqrt(v / (1 - b2)) are both |g|: 20 U of lr, and eps; the difference rounds to p
        assert bool(((moved - want).abs() <= 3e-3 * (30 * U + 1e-8 / d.abs().double().clamp(min=1e-12))
                     + 2 * U * b.abs()).all())
    for t in (2, 3, 4):
        step_and_check(params, grads, s, t, f"step {t}")


@pytest.mark.parametrize("state", ["e4m3", "f32"])
def test_mixed_types_copies_and_norm(dev, state):
    g = gen(3)
    kinds = [(F32, BF16), (BF16, BF16), (F32, F32), (BF16, F32)] * 2
    shapes = [(33, 70), (1000,), (5, 5, 5), (129,), (2049,), (16, 128), (1,), (300, 9)]
    params = [randn(g, *s).to(k[0]).to(dev) for s, k in zip(shapes, kinds)]
    grads = [(randn(g, *s) * 0.3).to(k[1]).to(dev) for s, k in zip(shapes, kinds)]
    copies = [torch.full(s, 9.0, dtype=BF16, device=dev) if k[0] == F32 else None
              for s, k in zip(shapes, kinds)]
    kept = [x.clone() for x in grads]
    norm = dg.grad_norm(grads)
    s = make_state(g, params, state, dev)
    assert float(norm) > 2.0
    step_and_check(params, grads, s, 7, "clipped", norm=norm, max_norm=2.0, copies=copies)
    step_and_check(params, grads, s, 8, "not clipped", norm=norm, max_norm=1e9)
    step_and_check(params, grads, s, 9, "to nothing", norm=norm, max_norm=0.0)
    for a, b in zip(grads, kept):
        assert torch.equal(a, b)


@pytest.mark.parametrize("state", ["e4m3", "f32"])
def test_clipping_on_the_way_is_clipping_before(dev, state):
    """Within roundings of the gradients: both ways against the same formula."""
    g = gen(4)
    params = [randn(g, 5000).to(dev)]
    grads = [randn(g, 5000).to(dev)]
    norm = dg.grad_norm(grads)
    s = make_state(g, params, state, dev)
    p2, s2 = [params[0].clone()], clone(s)
    step_and_check(params, grads, s, 5, "on the way", norm=norm, max_norm=1.0)
    dg.clip_grad_norm(grads, 1.0)
    step_and_check(p2, grads, s2, 5, "before")


@pytest.mark.parametrize("state", ["e4m3", "f32"])
@pytest.mark.parametrize("copies", [False, True])
@pytest.mark.parametrize("count", [88, 96, 97, 120, 121, 300])
def test_lists_of_many_tensors(dev, count, copies, state):
    """More tensors than a table holds."""
    g = gen(count)
    sizes = [1 + (i * 37) % 400 for i in range(count)]
    params = [randn(g, n).to(F32 if i % 3 else BF16).to(dev) for i, n in enumerate(sizes)]
    grads = [(randn(g, n) * 1e-2).to(F32 if i % 2 else BF16).to(dev) for i, n in enumerate(sizes)]
    also = [torch.zeros(n, dtype=BF16, device=dev) if p.dtype == F32 else None
            for n, p in zip(sizes, params)] if copies else None
    step_and_check(params, grads, make_state(g, params, state, dev), 11, f"{count} tensors", copies=also)


@pytest.mark.parametrize("state", ["e4m3", "f32"])
def test_any_alignment(dev, state):
    """Tensors that start anywhere in larger ones, whose other elements stay."""
    g = gen(6)
    for dtype, grad in ((BF16, BF16), (F32, BF16), (BF16, F32)):
        hp, hg = randn(g, 9000).to(dtype).to(dev), (randn(g, 9000) * 1e-2).to(grad).to(dev)
        kept = hp.clone()
        cuts = [(1, 130), (131, 2500), (2637, 4000), (6641, 2222)]
        params = [hp[a:a + n] for a, n in cuts]
        grads = [hg[a + 2:a + 2 + n] for a, n in cuts]
        copies = [torch.zeros(n + 3, dtype=BF16, device=dev)[3:] for _, n in cuts]
        step_and_check(params, grads, make_state(g, params, state, dev), 4, f"{dtype}", copies=copies)
        mask = torch.ones(9000, dtype=torch.bool, device=dev)
        for a, n in cuts:
            mask[a:a + n] = False
        assert torch.equal(hp[mask], kept[mask])


def test_moments_of_very_unequal_size(dev):
    """Within a block: small moments and roots under the smallest codes.  A root that is not zero stays so,
    and no parameter moves by more than its moments can say."""
    g = gen(7)
    n = 1024
    size = torch.logspace(-12, 1, n)
    params = [randn(g, n).to(dev)]
    s = dg.adamw_state(params)
    before = params[0].clone()
    for t in range(1, 6):
        grads = [(randn(g, n).sign() * size).to(dev)]
        step_and_check(params, grads, s, t, f"step {t}", weight_decay=0.0)
    # |m'| / sqrt(v') is at most 7.3 for these betas where v is as large as its gradients made it; a root is
    # never under half of what it was rounded from
    assert float((params[0] - before).abs().max()) < 5 * 3e-3 * 20


@pytest.mark.parametrize("state", ["e4m3", "f32"])
def test_eps_of_zero_and_large_gradients(dev, state):
    g = gen(8)
    params = [randn(g, 700).to(dev)]
    grads = [randn(g, 700).to(dev) * 1e15]
    step_and_check(params, grads, dg.adamw_state(params, state), 1, "large", eps=0.0)
    grads = [randn(g, 700).to(dev) * 1e-15]
    step_and_check(params, grads, dg.adamw_state(params, state), 1, "small", eps=0.0)
    step_and_check(params, grads, dg.adamw_state(params, state), 10 ** 9, "late")
    step_and_check(params, grads, dg.adamw_state(params, state), 1, "no memory", betas=(0.0, 0.0))


@pytest.mark.parametrize("state", ["e4m3", "f32"])
def test_what_is_not_finite(dev, state):
    """fp32: the element's own moments and parameter; e4m3: the moments of its 128, its own parameter."""
    params = [torch.ones(300, device=dev), torch.ones(128, device=dev)]
    grads = [torch.full((300,), 0.1, device=dev), torch.full((128,), 0.1, device=dev)]
    grads[0][130] = float("nan")
    s = dg.adamw_state(params, state)
    dg.adamw_step(params, grads, s, 1, **KEYS)
    assert params[0].isnan().nonzero().tolist() == [[130]] and not bool(params[1].isnan().any())
    m, v = s.moments()
    bad = m.isnan().nonzero().view(-1).tolist()
    assert bad == ([130] if state == "f32" else list(range(128, 256)))
    assert torch.equal(m.isnan(), v.isnan())
    # a norm that is not finite, as clip_grad_norm has it
    p = [torch.ones(300, device=dev)]
    d = [torch.ones(300, device=dev)]
    inf, nan = (torch.tensor(x, device=dev) for x in (float("inf"), float("nan")))
    dg.adamw_step(p, d, dg.adamw_state(p, state), 1, norm=inf, max_norm=1.0, **{**KEYS, "weight_decay": 0})
    assert bool((p[0] == 1).all())
    dg.adamw_step(p, d, dg.adamw_state(p, state), 1, norm=nan, max_norm=1.0, **KEYS)
    assert bool(p[0].isnan().all())


@pytest.mark.parametrize("state", ["e4m3", "f32"])
def test_graph_replays_step_on(dev, state):
    """The step's number, the rate, the norm and the gradients are read anew by each replay."""
    g = gen(9)
    sizes = [3000, 129]
    params = [randn(g, n).to(dev) for n in sizes]
    held = [torch.zeros(n, device=dev) for n in sizes]
    copies = [torch.zeros(n, dtype=BF16, device=dev) for n in sizes]
    s = make_state(g, params, state, dev)
    step = torch.zeros((), dtype=torch.int64, device=dev)
    lr = torch.tensor([3e-3], device=dev)
    at_start = [p.clone() for p in params], clone(s)

    def one(params, s, copies):
        norm = dg.grad_norm(held)
        step.add_(1)
        dg.adamw_step(params, held, s, step, lr, norm=norm, max_norm=1.0, copies=copies)
        return norm

    one([p.clone() for p in params], clone(s), None)
    step.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one(params, s, copies)
    ep, es = at_start
    for t in range(1, 5):
        lr.fill_(3e-3 / t)
        for h in held:
            h.copy_((randn(g, h.numel()) * t).to(dev))
        norm = dg.grad_norm(held)
        dg.adamw_step(ep, held, es, torch.tensor([t], device=dev), torch.tensor(3e-3 / t, device=dev),
                      norm=norm, max_norm=1.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(params, ep, copies):
            assert torch.equal(a, b) and torch.equal(c, b.to(BF16)), t
        for a, b in zip((s.m, s.v), (es.m, es.v)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), t
    assert int(step) == 4


@pytest.mark.parametrize("t", [1, 2, 1000, 10 ** 12])
def test_numbers_from_the_host_and_from_the_device(dev, t):
    """A step's number or a rate in device memory gives what the host's number gives, to the formula's bound."""
    for step in (t, torch.tensor(t, device=dev)):
        for lr in (3e-3, torch.tensor([3e-3], device=dev)):
            g = gen(10)
            params = [randn(g, 500).to(dev)]
            grads = [randn(g, 500).to(dev)]
            step_and_check(params, grads, make_state(g, params, "f32", dev), step, f"{step} {lr}", lr=lr)


def test_other_streams(dev):
    """Two lists on two streams at once, and each alone."""
    g = gen(12)
    lists = [[randn(g, 100000).to(dev), randn(g, 333).to(dev)] for _ in range(2)]
    grads = [[(randn(g, p.numel()) * 1e-2).to(dev) for p in ps] for ps in lists]
    states = [dg.adamw_state(ps) for ps in lists]
    want = [[p.clone() for p in ps] for ps in lists]
    for ps, gs in zip(want, grads):
        st = dg.adamw_state(ps)
        for t in (1, 2, 3):
            dg.adamw_step(ps, gs, st, t, **KEYS)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in lists]
    for t in (1, 2, 3):
        for s, ps, gs, st in zip(streams, lists, grads, states):
            with torch.cuda.stream(s):
                dg.adamw_step(ps, gs, st, t, **KEYS)
    torch.cuda.synchronize()
    for ps, ws in zip(lists, want):
        for p, w in zip(ps, ws):
            assert torch.equal(p, w)


def test_parameters_count_as_changed(dev):
    p = torch.ones(300, device=dev, requires_grad=True)
    y = (p * p).sum()
    dg.adamw_step([p], [torch.ones(300, device=dev)], dg.adamw_state([p]), 1, **KEYS)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_a_parameter_that_is_there_twice(dev):
    p, d = torch.ones(400, device=dev), torch.ones(400, device=dev)
    for params, kw in (([p, p], {}), ([p[:300], p[200:]], {}), ([p], dict(copies=[d.view(BF16)[:400]])),
                       ([p], dict(copies=[p.view(BF16)[:400]]))):
        grads = [d[:x.numel()] for x in params]
        s = dg.adamw_state(params)
        with pytest.raises(ValueError, match="overlaps"):
            dg.adamw_step(params, grads, s, 1, 1e-3, **kw)
    with pytest.raises(ValueError, match="overlaps"):
        dg.adamw_step([p], [p], dg.adamw_state([p]), 1, 1e-3)
    s = dg.adamw_state([p])
    s.v = s.m
    with pytest.raises(ValueError, match="overlaps"):
        dg.adamw_step([p], [d], s, 1, 1e-3)
    assert bool((p == 1).all())
    dg.adamw_step([p[:200], p[200:]], [d[:200], d[:200]], dg.adamw_state([p[:200], p[200:]]), 1, 1e-3)
    assert torch.equal(p[:200], p[200:])


def test_training_in_8_bits(dev):
    """The layer's step as a program makes it: int8 products with their gradients, the norm, the update with
    8-bit states and bf16 copies, new codes; and a token alone afterwards gets what it gets in the batch."""
    g = gen(13)
    x = randn(g, 300, 200).to(BF16).to(dev)
    w = (randn(g, 130, 200) * 0.1).to(dev)
    bias = torch.zeros(130, device=dev)
    copy = torch.empty(130, 200, dtype=BF16, device=dev)
    state = dg.adamw_state([w, bias])
    for t in (1, 2, 3):
        qx, qxt = dg.int8_quantize(x, transposed="both")
        qw, qwt = dg.int8_quantize(w, transposed="both")
        y = dg.int8_gemm(qx, qw, bias_col=bias)
        dy = (y.float() - 1.0).to(BF16) * (1 / 300)
        qd, qdt = dg.int8_quantize(dy, transposed="both")
        dx, dw = dg.int8_gemm(qd, qwt), dg.int8_gemm(qdt, qxt, out_dtype="f32")
        assert dx.shape == x.shape and bool(dx.isfinite().all())
        grads = [dw, dy.float().sum(0)]
        step_and_check([w, bias], grads, state, t, f"step {t}", norm=dg.grad_norm(grads), max_norm=1.0,
                       copies=[copy, None])
    qw = dg.int8_quantize(w)
    y = dg.int8_gemm(dg.int8_quantize(x), qw, bias_col=bias)
    for i in (0, 77):
        assert torch.equal(dg.int8_gemm(dg.int8_quantize(x[i:i + 1]), qw, bias_col=bias), y[i:i + 1])
