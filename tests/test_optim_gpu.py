"""AdamW over many tensors and the gradient norm against the float64 reference.

Tolerances (u = 2^-24, the unit roundoff of fp32):
* m: two products and a sum, |d| <= 3u (b1 |m| + (1 - b1) |g|), with g = coef
  grad rounded once more: 4u of the terms' sizes; v likewise with one more
  product: 6u.
* p: the update is formed in 8 roundings and two bias corrections rounded
  to fp32, on moments with the errors above: 24u of the terms' sizes;
  the sum p - update adds 2u |p|.
* 8-bit codes: the stored value is the reference's rounding of the fp32
  moment.  A moment whose fp32 error carries it over a rounding boundary lands
  one code away: probability at most 2 (6u) (terms) / step with step >= |x| / 16,
  some 1e-5 without cancellation; at most one code apart, and 1e-3 of the
  values (or one) are allowed.
* bf16 parameters, rounded by the dither: the same argument with steps of
  |p| / 256: one step apart, 1e-2 of the values (or one).
"""

import numpy as np
import pytest

from gpu_util import from_dev, torch_mod
from oracle import operators as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
SIZES = [0, 1, 2, 3, 255, 256, 257, 4095, 4096, 4097, 20001]


def f32(x):
    return float(np.float32(x))


HP = dict(lr=f32(1e-3), betas=(f32(0.9), f32(0.999)), eps=f32(1e-8))


def make(torch, sizes, pdt, gdt, misalign, seed, gscale=1.0):
    """Lists of parameter and gradient tensors; misalign: views that start one element into a buffer."""
    rng = np.random.default_rng([5, seed])
    dt = dict(f32=torch.float32, bf16=torch.bfloat16)
    off = 1 if misalign else 0

    def up(a, d):
        t = torch.zeros(a.size + 1, dtype=dt[d], device="cuda:0")
        t[off:off + a.size] = torch.from_numpy(a).to("cuda:0").to(dt[d])
        return t[off:off + a.size]
    p = [up((rng.standard_normal(n) * 0.05).astype(np.float32), pdt) for n in sizes]
    g = [up((rng.standard_normal(n) * 10.0 ** rng.uniform(-7, 0, n) * gscale).astype(np.float32), gdt) for n in sizes]
    for t in g:
        t[:2] = 0.0
    return p, g


def padded(arrays):
    """The tensors' values in the layout of the state arrays."""
    return np.concatenate([np.pad(a, (0, -a.size % O.BLOCK)) for a in arrays] or [np.zeros(0)])


def host(ts):
    return [from_dev(t) for t in ts]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pdt,gdt,copy,misalign", [("f32", "f32", False, False), ("f32", "bf16", True, False),
                                                   ("bf16", "bf16", False, False), ("f32", "f32", True, True),
                                                   ("bf16", "f32", False, True)])
def test_adamw_steps(bits, pdt, gdt, copy, misalign):
    torch = torch_mod()
    import orthogonal_reparameterized_poetx_amd as P
    p, g = make(torch, SIZES, pdt, gdt, misalign, bits)
    copies = [torch.zeros(t.numel() + misalign, dtype=torch.bfloat16, device="cuda:0")[misalign:] for t in p] \
        if copy else None
    lr_mul = [1.0, 0.25, 2.0] * 4
    decay = [0.0, 0.1, f32(0.01), 0.5] * 3
    lr_mul, decay = lr_mul[:len(SIZES)], decay[:len(SIZES)]
    opt = P.AdamW(p, g, lr_mul=lr_mul, weight_decay=[0.0, 0.125, 0.5, 0.0] * 2 + [0.25, 0.0, 0.125], copies=copies,
                  state_bits=bits, **HP)
    decay = [0.0, 0.125, 0.5, 0.0] * 2 + [0.25, 0.0, 0.125]
    b1, b2 = HP["betas"]
    coef = torch.tensor([0.625], device="cuda:0")
    mul = padded([np.full(n, x) for n, x in zip(SIZES, lr_mul)])
    wd = padded([np.full(n, x) for n, x in zip(SIZES, decay)])
    pos = np.arange(mul.size)
    real = padded([np.ones(n) for n in SIZES]) > 0
    for step in (1, 2, 3):
        if step > 1:
            for t in g:
                t.mul_(-0.75)
        st = {k: t.cpu().numpy() for k, t in opt.state().items()}
        if bits == 32:
            m0, v0 = st["m"].astype(np.float64), st["v"].astype(np.float64)
        else:
            m0, v0 = O.decode8(st["m"], st["m_exp"], True), O.decode8(st["v"], st["v_exp"], False)
        p0, g0 = padded(host(p)), padded(host(g)) * 0.625
        opt.step(coef=coef)
        torch.cuda.synchronize()
        pr, mr, vr = O.adamw(p0, g0, m0, v0, step, HP["lr"], b1, b2, HP["eps"], mul, wd)
        mt, vt = b1 * np.abs(m0) + (1 - b1) * np.abs(g0), vr
        den = np.sqrt(vr / (1 - b2 ** step)) + HP["eps"]
        ptol = 2 * U * np.abs(p0) + 24 * U * HP["lr"] * mul * (wd * np.abs(p0) + mt / (1 - b1 ** step) / den)
        got = padded(host(p))
        if pdt == "f32":
            assert np.all(np.abs(got - pr) <= ptol), np.max(np.abs(got - pr) - ptol)
        else:
            ref, unit = O.round_bf16_dither(pr, pos, step)
            d = np.abs(got - ref)
            assert np.all(d <= 2 * unit) and (d > 0).sum() <= max(1, 0.01 * d.size)
        if copy:
            for c, t in zip(copies, p):
                assert torch.equal(c, t.to(torch.bfloat16))
        mg, vg = host(opt.moments())
        if bits == 32:
            assert np.all(np.abs(mg - mr) <= 4 * U * mt) and np.all(np.abs(vg - vr) <= 6 * U * vt)
        else:
            st = {k: t.cpu().numpy() for k, t in opt.state().items()}
            for x, k, ref, signed in ((mg, "m", mr, True), (vg, "v", vr, False)):
                assert np.array_equal(x, O.decode8(st[k], st[k + "_exp"], signed))
                want, unit = O.round8(ref, pos, step, signed)
                d = np.abs(x - want)
                assert np.all(d <= unit * 1.0001)
                assert (d > 0).sum() <= max(1, 1e-3 * d.size), (k, (d > 0).sum())
                assert np.all(x[~real] == 0)
            assert np.all((vg > 0) == (vr > 1e-45))
    assert opt.steps == 3


@pytest.mark.parametrize("bits", [32, 8])
def test_coef_not_finite_leaves_everything(bits):
    torch = torch_mod()
    import orthogonal_reparameterized_poetx_amd as P
    p, g = make(torch, [1000, 7], "f32", "f32", False, 3)
    opt = P.AdamW(p, g, state_bits=bits, **HP)
    opt.step()
    before = [t.clone() for t in p] + [t.clone() for t in opt.state().values()]
    for bad in (float("nan"), float("inf")):
        opt.step(coef=torch.tensor([bad], device="cuda:0"))
    after = p + list(opt.state().values())
    assert all(torch.equal(a, b) for a, b in zip(before, after))


def test_gradients_not_finite_stay_in_their_place():
    torch = torch_mod()
    import orthogonal_reparameterized_poetx_amd as P
    for bits in (32, 8):
        p, g = make(torch, [1024, 300], "f32", "f32", False, 4)
        g[0][300] = float("nan")
        g[0][600] = float("inf")
        before = host(p)
        opt = P.AdamW(p, g, state_bits=bits, **HP)
        opt.step()
        m, v = host(opt.moments())
        after = host(p)
        assert np.isnan(after[0][300]) and np.isnan(after[0][600])     # inf / inf
        fine = np.ones(1024, bool)
        fine[[300, 600]] = False
        assert np.all(np.isfinite(after[0][fine])) and np.all(np.isfinite(after[1]))
        assert np.any(after[0][fine] != before[0][fine])
        # 32 bits: the elements; 8 bits: their blocks of 256 are marked
        bad = np.zeros(m.size, bool)
        if bits == 32:
            bad[[300, 600]] = True
            assert np.array_equal(~np.isfinite(m), bad) and np.array_equal(~np.isfinite(v), bad)
        else:
            bad[256:512] = bad[512:768] = True
            assert np.array_equal(np.isnan(m), bad) and np.array_equal(np.isnan(v), bad)


def test_zero_gradients_and_extreme_sizes_in_8_bits():
    torch = torch_mod()
    import orthogonal_reparameterized_poetx_amd as P
    # a block of zeros, one of the smallest and one of the largest squares that fp32 holds
    g0 = np.zeros(1024, np.float32)
    g0[256:512] = 1e-19
    g0[512:768] = 1e18
    g0[768:1024] = 10.0 ** np.linspace(-12, 3, 256)
    p = [torch.ones(1024, device="cuda:0")]
    opt = P.AdamW(p, [torch.from_numpy(g0).to("cuda:0")], state_bits=8, **HP)
    opt.step()
    m, v = host(opt.moments())
    x = from_dev(p[0])
    assert np.all(m[:256] == 0) and np.all(v[:256] == 0) and np.all(x[:256] == 1)
    assert np.all(np.isfinite(x)) and np.all(np.isfinite(m)) and np.all(np.isfinite(v))
    assert np.all(v[256:] > 0)      # never zero for a nonzero square
    # within the window of the exponents a code is off by less than a step: 1 / 8 of the value
    want = 1e-3 * np.square(g0[512:].astype(np.float64))
    ok = want >= want.reshape(2, 256).max(1).repeat(256) * 2.0 ** -29
    assert ok.sum() > 300 and np.all(np.abs(v[512:] / want - 1)[ok] <= 0.1251)
    opt.step()
    assert np.all(np.isfinite(from_dev(p[0])))


def test_dithered_second_moment_follows_its_mean():
    """Constant gradients after much larger ones: v decays to g^2 (0.999^4000 = 0.018 of a start four times as high
    is 7 %), which rounding to nearest would not allow (one step moves v by at most 0.3 % of itself, half a code is 3 % or
    more).  A code's own rounding averages out over 4096 values: 5 % are allowed beside the 5.5 % of the decay."""
    torch = torch_mod()
    import orthogonal_reparameterized_poetx_amd as P
    rng = np.random.default_rng(8)
    g = (np.exp(rng.uniform(-1, 1, 4096))).astype(np.float32)
    gd = torch.from_numpy(2 * g).to("cuda:0")
    opt = P.AdamW([torch.zeros(4096, device="cuda:0")], [gd], betas=(0.9, 0.0), state_bits=8)
    opt.step()                              # beta2 = 0: v is the square at once
    gd.mul_(0.5)
    opt.hyper.beta2 = 0.999
    for _ in range(4000):
        opt.step()
    _, v = host(opt.moments())
    ratio = v / np.square(g.astype(np.float64))
    assert abs(ratio.mean() - (1 + 3 * 0.999 ** 4000)) <= 0.05
    assert np.all((ratio > 0.7) & (ratio < 1.5))


@pytest.mark.parametrize("gdt", ["f32", "bf16"])
@pytest.mark.parametrize("misalign", [False, True])
def test_grad_norm(gdt, misalign):
    torch = torch_mod()
    import orthogonal_reparameterized_poetx_amd as P
    _, g = make(torch, SIZES + [3_000_001], "f32", gdt, misalign, 6)
    norm = P.GradNorm(g)
    want = O.grad_norm(host(g), 1.0)
    for max_norm in (1.0, 1e9, float("inf"), 1.0):
        n, c = norm(max_norm)
        got, clip = float(n), float(c)
        # exact squares summed in fp64, one rounding to fp32
        assert abs(got - want[0]) <= 2 * U * want[0]
        ref = min(1.0, max_norm / (want[0] + 1e-6))
        assert abs(clip - ref) <= 2 * U * ref
    a = [float(x) for x in norm(0.5)]
    assert a == [float(x) for x in norm(0.5)]


def test_grad_norm_many_groups_sizes_and_values():
    torch = torch_mod()
    import orthogonal_reparameterized_poetx_amd as P
    # more chunks than workgroups
    big = torch.full((2048 * 4096 * 2 + 77,), 0.5, device="cuda:0")
    n, c = P.GradNorm([big])(1.0)
    assert float(n) == np.float32(np.sqrt(big.numel() * 0.25))
    # squares beyond fp32
    n, c = P.GradNorm([torch.full((100,), 1e30, device="cuda:0")])(1.0)
    assert abs(float(n) - 1e31) <= 4 * U * 1e31 and abs(float(c) * 1e31 - 1) <= 1e-6
    # nothing but empty tensors
    n, c = P.GradNorm([torch.zeros(0, device="cuda:0")])(2.0)
    assert float(n) == 0.0 and float(c) == 1.0
    for bad in (float("nan"), float("inf"), -float("inf")):
        g = torch.ones(5000, device="cuda:0")
        g[4999] = bad
        norm = P.GradNorm([g])
        n, c = norm(1.0)
        assert not np.isfinite(float(n)) and np.isnan(float(c))
        g[4999] = 0.0
        n, c = norm(1.0)
        assert np.isfinite(float(n)) and abs(float(c) * np.sqrt(4999.0) - 1) <= 1e-5


def test_norm_and_step_in_a_replayed_graph_and_on_another_stream():
    torch = torch_mod()
    import orthogonal_reparameterized_poetx_amd as P
    p, g = make(torch, [5000, 333], "f32", "f32", False, 9)
    q = [t.clone() for t in p]
    one, two = P.AdamW(p, g, state_bits=8, **HP), P.AdamW(q, g, state_bits=8, **HP)
    stream = torch.cuda.Stream()
    one.grad_norm(1.0)          # its buffers are made at the first call
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        _, coef = one.grad_norm(1.0)
        one.step(coef=coef)
    for k in range(4):
        for t in g:
            t.add_(0.01 * k)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        two.steps = 0           # the graph holds step 1
        with torch.cuda.stream(stream):
            _, coef = two.grad_norm(1.0)
            two.step(coef=coef)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(p, q))
        assert all(torch.equal(a, b) for a, b in zip(one.state().values(), two.state().values()))


def test_refusals_of_the_classes():
    torch = torch_mod()
    import orthogonal_reparameterized_poetx_amd as P
    d = "cuda:0"
    a = torch.zeros(8, device=d)
    for bad in (lambda: P.GradNorm([]), lambda: P.GradNorm([a.cpu()]), lambda: P.GradNorm([a.double()]),
                lambda: P.GradNorm([torch.zeros(4, 4, device=d).t()[:, :2]]),
                lambda: P.AdamW([a], [torch.zeros(9, device=d)]), lambda: P.AdamW([a], [a, a]),
                lambda: P.AdamW([a], [a.clone()], copies=[torch.zeros(8, device=d)]),
                lambda: P.AdamW([a], [a.clone()], state_bits=16),
                lambda: P.AdamW([a], [a.clone()], state=dict(m=a, v=a)),
                lambda: P.AdamW([a], [a.clone()]).step(coef=torch.zeros(2, device=d))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(P.PoetxError):
        P.GradNorm([a])(0.0)
    with pytest.raises(P.PoetxError):
        P.AdamW([a], [a.clone()], betas=(1.0, 0.9)).step()
    with pytest.raises(P.PoetxError):
        P.AdamW([a], [a.clone()], copies=[None], eps=-1.0).step()


def test_first_gradient_norm_inside_a_capture():
    torch = torch_mod()
    import orthogonal_reparameterized_poetx_amd as P
    p, g = make(torch, [5000, 333], "f32", "f32", False, 15)
    opt = P.AdamW(p, g, **HP)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm, coef = opt.grad_norm(1.0)
    for k in range(3):
        g[0].add_(k)
        graph.replay()
        torch.cuda.synchronize()
        want = O.grad_norm(host(g), 1.0)
        assert abs(float(norm) - want[0]) <= 2 * U * want[0] and abs(float(coef) - want[1]) <= 2 * U * want[1]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("first", [0, 100])
def test_a_skipped_step_is_as_if_it_had_not_been(bits, first):
    """Steps whose coefficient is not finite write nothing; those after them take the numbers they would have had:
    bias correction and dither, bit for bit."""
    torch = torch_mod()
    import orthogonal_reparameterized_poetx_amd as P
    sizes = [5000, 7, 1025]
    p, g = make(torch, sizes, "bf16" if bits == 8 else "f32", "f32", False, 16)
    q = [t.clone() for t in p]
    one = P.AdamW(p, g, state_bits=bits, step=first, **HP)
    two = P.AdamW(q, g, state_bits=bits, step=first, **HP)
    good, bad = (torch.tensor([x], device="cuda:0") for x in (0.5, float("nan")))
    for k, skip in enumerate([True, False, True, True, False, False, True, False, True, True]):
        if skip:
            one.step(coef=bad if k % 3 else torch.tensor([float("inf")], device="cuda:0"))
            continue
        for t in g:
            t.mul_(-0.75)
        one.step(coef=good)
        two.step(coef=good)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(p, q)), k
        assert all(torch.equal(a, b) for a, b in zip(one.state().values(), two.state().values())), k
        assert one.steps == two.steps
    assert one.steps == first + 4
    # taken up again from what is saved
    three = P.AdamW(p, g, state_bits=bits, state=one.state(), step=one.steps, **HP)
    three.step(coef=good)
    two.step(coef=good)
    assert all(torch.equal(a, b) for a, b in zip(p, q))
    one.steps = 7
    assert one.steps == 7


def test_a_set_of_several_launches():
    """More chunks of 1024 values than one launch takes (2^23): every value takes its step, a skipped one is counted
    once.  In bf16 with 8-bit moments, 52 GB."""
    torch = torch_mod()
    import orthogonal_reparameterized_poetx_amd as P
    n = (2 ** 23 + 5) * 1024 + 77
    p, g = [torch.zeros(n, dtype=torch.bfloat16, device="cuda:0") for _ in range(2)]
    g.fill_(-1.0)
    opt = P.AdamW([p], [g], state_bits=8, lr=0.5)
    opt.step(coef=torch.tensor([float("nan")], device="cuda:0"))
    assert opt.steps == 0 and not bool(p.any())
    opt.step()
    assert opt.steps == 1
    # the first step is the learning rate, whatever the gradient
    for x in p.split(2 ** 30):
        assert bool(((x - 0.5).abs() <= 2.0 ** -8).all())
    # m and v are a tenth and a thousandth of g and g^2, to an eighth; zero past the tensor's end
    st = opt.state()
    for k, want in (("m", -0.1), ("v", 1e-3)):
        for lo in (0, 2 ** 30, 2 ** 33 - 512, 2 ** 33, 2 ** 33 + 4096):
            x = O.decode8(st[k][lo:lo + 512].cpu().numpy(), st[k + "_exp"][lo // 256:lo // 256 + 2].cpu().numpy(), k == "m")
            assert np.all(np.abs(x / want - 1) <= 0.125), (k, lo)
        assert not bool(st[k][n:].any())
        assert int(st[k + "_exp"].min()) > 40
    norm, _ = opt.grad_norm()
    assert abs(float(norm) - n ** 0.5) <= 2 * U * n ** 0.5


@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-22, 1e-15, 1e-8])
@pytest.mark.parametrize("bits", [32, 8])
def test_second_moments_below_the_normal_range(bits, eps):
    """Gradients whose squares are subnormal in fp32 and an eps that does not cover their root.  The first update is
    g / (|g| + eps) of the learning rate; v holds a multiple of 2^-149, so its root is off by at most 2^-150 / v of
    itself beside the roundings (8-bit moments: the update takes them before they are rounded)."""
    torch = torch_mod()
    import orthogonal_reparameterized_poetx_amd as P
    g0 = (2.0 ** np.linspace(-66, -40, 512)).astype(np.float32)
    g0[1::2] *= -1
    p = [torch.zeros(512, device="cuda:0")]
    opt = P.AdamW(p, [torch.from_numpy(g0).to("cuda:0")], betas=(0.5, 0.5), lr=1.0, eps=f32(eps), state_bits=bits)
    opt.step()
    got = from_dev(p[0])
    g = g0.astype(np.float64)
    assert np.all(np.isfinite(got))
    want = -g / (np.abs(g) + f32(eps))
    # v = g^2 / 2, rounded to fp32 twice (the square and its half): 2^-149 at most
    v_err = 2.0 ** -149 / (g * g / 2) / 2
    assert np.all(np.abs(got - want) <= np.abs(want) * (24 * U + v_err))


def test_no_gradient_yet_and_eps_zero():
    """0 / 0 is NaN by the formula, in that value alone."""
    torch = torch_mod()
    import orthogonal_reparameterized_poetx_amd as P
    g = torch.tensor([0.0, 0.5, 1.0], device="cuda:0")
    p = [torch.zeros(3, device="cuda:0")]
    P.AdamW(p, [g], lr=1.0, eps=0.0).step()
    got = from_dev(p[0])
    assert np.isnan(got[0]) and abs(got[2] + 1) <= 24 * U


def test_a_norm_past_the_range_of_fp32():
    """It reads as infinite; the coefficient is that of the norm itself, here subnormal (steps of 2^-149)."""
    torch = torch_mod()
    import orthogonal_reparameterized_poetx_amd as P
    g = [torch.full((4,), 3e38, device="cuda:0")]
    n, c = P.GradNorm(g)(2.0)
    want = 2.0 / (2 * float(np.float32(3e38)))
    assert np.isinf(float(n)) and abs(float(c) - want) <= 2.0 ** -149
