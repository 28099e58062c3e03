"""Low-rank adapters beside a shared projection against the float64 reference.

Tolerances, elementwise (u = 2^-24): a sum of K products in fp32 in any order
is off by at most K u times the sum of its terms' sizes.  With T = s A x and
its sizes T~ = s |A| |x| (U, U~ alike), w = 2^-16 for bf16 sets (T and U
enter the second product as two bf16 values, which keep 16 bits) and 0
for fp32, and v the rounding of the result (2^-8 for bf16, u for fp32):
  Y   v |Y| + ((n + r + 4) u + w) |B| T~
  dX  v |dX| + ((m + r + 4) u + w) |A|^T U~
  dA  ((m + N + 4) u + w) U~ |x|^T          (the sum over slots included)
  dB  ((n + N + 4) u + w) |dy| T~^T
These hold in the worst case; the errors of a sum in fact add like a random
walk, so the norm of the difference is held to 4e-3 (bf16 results) and 2e-5
(fp32 results) of the result's as well.
"""

import numpy as np
import pytest

from gpu_util import from_dev, to_dev, torch_mod
from oracle import operators as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


class Case:
    def __init__(self, m, n, ranks, seg_start, seg_adapter, N, dtype="bf16", seed=0, pad=(0, 0, 0), offset=0):
        """pad: extra elements between rows of X, Y (dY) and dX; offset: elements before each first row."""
        torch = torch_mod()
        rng = np.random.default_rng([11, seed])
        self.m, self.n, self.N, self.dtype, self.ranks = m, n, N, dtype, ranks
        self.tdt = torch.bfloat16 if dtype == "bf16" else torch.float32

        def mat(shape, sigma, extra=0):
            a = (rng.standard_normal(shape) * sigma).astype(np.float32)
            t = torch.full((shape[0] * (shape[1] + extra) + offset,), float("nan"), dtype=self.tdt, device="cuda:0")
            v = t[offset:].view(shape[0], shape[1] + extra)[:, :shape[1]]
            v.copy_(torch.from_numpy(a))
            return v
        self.A = [mat((r, n), n ** -0.5) for r in ranks]
        self.B = [mat((m, r), 0.1) for r in ranks]
        self.scale = [0.5 + 0.25 * (i % 5) for i in range(len(ranks))]
        self.X, self.Y, self.dX = mat((N, n), 1.0, pad[0]), mat((N, m), 1.0, pad[1]), mat((N, n), 1.0, pad[2])
        self.dY = mat((N, m), 1.0, pad[1])
        self.start, self.which = np.asarray(seg_start), np.asarray(seg_adapter)
        self.sd, self.wd = to_dev(self.start, "i32"), to_dev(self.which, "i32")

    def set(self, **kw):
        import orthogonal_reparameterized_poetx_amd as P
        return P.AdapterSet(self.m, self.n, self.A, self.B, self.scale, **kw)

    def host(self):
        return [from_dev(a) for a in self.A], [from_dev(b) for b in self.B]


def near(got, ref, tol, bf16, name):
    d = np.abs(got - ref)
    assert np.all(np.isfinite(got)), name
    assert np.all(d <= tol), (name, float(np.max(d - tol)), float(np.max(d)))
    norm = np.linalg.norm(ref)
    if norm > 0:
        rel = np.linalg.norm(d) / norm
        assert rel <= (4e-3 if bf16 else 2e-5), (name, rel)


def check_forward(c, aset=None, **kw):
    torch = torch_mod()
    A, B = c.host()
    X, Y0 = from_dev(c.X), from_dev(c.Y)
    aset = aset or c.set()
    aset.forward(c.X, c.Y, c.sd, c.wd, **kw)
    torch.cuda.synchronize()
    ref = O.adapters_forward(X, Y0, A, B, c.scale, c.start, c.which)
    size = O.adapters_forward(np.abs(X), np.zeros_like(Y0), [np.abs(a) for a in A], [np.abs(b) for b in B], c.scale,
                              c.start, c.which)
    bf = c.dtype == "bf16"
    tol = (2.0 ** -8 if bf else U) * np.abs(ref) + ((c.n + max(c.ranks) + 4) * U + (2.0 ** -16 if bf else 0)) * size
    got = from_dev(c.Y)
    near(got, ref, tol, bf, "Y")
    assert np.array_equal(got[size.sum(1) == 0], Y0[size.sum(1) == 0])      # other tokens untouched
    return got


def check_backward(c, aset=None, dx=True, accumulate=None, **kw):
    torch = torch_mod()
    A, B = c.host()
    X, dY, dX0 = from_dev(c.X), from_dev(c.dY), from_dev(c.dX)
    aset = aset or c.set()
    dA, dB = aset.backward(c.X, c.dY, c.sd, c.wd, dX=c.dX if dx else None, accumulate=accumulate is not None, **kw)
    torch.cuda.synchronize()
    dXr, dAr, dBr = O.adapters_backward(X, dY, dX0, A, B, c.scale, c.start, c.which)
    a = np.abs
    dXs, dAs, dBs = O.adapters_backward(a(X), a(dY), np.zeros_like(dX0), [a(x) for x in A], [a(x) for x in B],
                                        c.scale, c.start, c.which)
    bf = c.dtype == "bf16"
    w, r = (2.0 ** -16 if bf else 0), max(c.ranks)
    if dx:
        near(from_dev(c.dX), dXr, (2.0 ** -8 if bf else U) * a(dXr) + ((c.m + r + 4) * U + w) * dXs, bf, "dX")
    else:
        assert np.array_equal(from_dev(c.dX), dX0)
    for i in range(len(A)):
        if accumulate is not None:
            dAr[i], dBr[i] = dAr[i] + accumulate[0][i], dBr[i] + accumulate[1][i]
        near(from_dev(dA[i]), dAr[i], ((c.m + c.N + 4) * U + w) * dAs[i] + U * a(dAr[i]), False, "dA%d" % i)
        near(from_dev(dB[i]), dBr[i], ((c.n + c.N + 4) * U + w) * dBs[i] + U * a(dBr[i]), False, "dB%d" % i)
    return dA, dB


SHAPES = [
    # m, n, ranks, seg_start, seg_adapter, N
    (256, 256, [16], [0, 64], [0], 64),
    (256, 256, [16], [0, 1], [0], 1),
    (600, 520, [5, 12, 9], [0, 0, 70, 71, 200, 333], [2, 0, -1, 1, 0], 333),
    (512, 1024, [8, 16, 24, 40], [0, 31, 64, 96, 129, 300], [3, 0, 2, 1, 3], 300),
    (7, 9, [1], [0, 2, 5], [0, 0], 5),
    (1, 1, [3], [0, 40], [0], 40),
    (264, 2056, [64, 33], [10, 10, 100, 105, 290], [1, 0, 7, 1], 310),
    (300, 200, [100, 128], [0, 150, 257], [1, 0], 257),
    (136, 72, [256, 200, 1], [0, 33, 66, 99], [2, 0, 1], 99),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_shapes(shape, dtype):
    c = Case(*SHAPES[shape], dtype=dtype, seed=shape)
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,offset", [((8, 16, 24), 0), ((3, 1, 5), 0), ((0, 0, 0), 1), ((4, 0, 8), 4)])
def test_strides_and_alignment(pad, offset, dtype):
    c = Case(320, 256, [16, 8, 3], [0, 50, 50, 120, 200], [0, 1, 2, 0], 200, dtype=dtype, seed=20, pad=pad,
             offset=offset)
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("nseg", [63, 64, 65, 200, 5000])
def test_many_segments(nseg):
    rng = np.random.default_rng(nseg)
    lens = rng.integers(0, 3, nseg)
    lens[nseg // 2] = 100
    start = np.concatenate([[0], np.cumsum(lens)])
    c = Case(128, 192, [16] * 7, start, rng.integers(-1, 9, nseg), int(start[-1]), seed=nseg)
    check_forward(c)
    check_backward(c)


def test_one_token_of_each_request():
    # all of one adapter, and each of its own
    for which in (np.zeros(64, int), np.arange(64)):
        c = Case(768, 512, [16] * 64, np.arange(65), which, 64, seed=3)
        check_forward(c)


def test_large_batch():
    c = Case(2048, 1024, [16, 16, 8], np.arange(0, 8193, 512), np.arange(16) % 4 - 1, 8192, seed=4)
    check_forward(c)
    check_backward(c)


def test_rows_far_apart():
    """Offsets beyond 2^31 elements."""
    torch = torch_mod()
    c = Case(64, 64, [16], [0, 40], [0], 40, seed=5)
    ld = 1 << 26
    for name in ("X", "Y", "dX", "dY"):
        t = getattr(c, name)
        big = torch.empty(39 * ld + 64, dtype=c.tdt, device="cuda:0")
        v = big.as_strided((40, 64), (ld, 1))
        v.copy_(t)
        setattr(c, name, v)
    check_forward(c)
    check_backward(c)


def test_accumulate_and_without_dx():
    c = Case(256, 320, [16, 4], [0, 100, 130], [0, 1], 130, seed=6)
    aset = c.set()
    with pytest.raises(ValueError):
        aset.backward(c.X, c.dY, c.sd, c.wd, accumulate=True)
    first = check_backward(c, aset, dx=False)
    before = [from_dev(t) for t in first[0]], [from_dev(t) for t in first[1]]
    check_backward(c, aset, accumulate=before)


def test_nothing_to_do():
    torch = torch_mod()
    c = Case(64, 96, [16, 8], [0, 0], [0], 0, seed=7)
    aset = c.set()
    aset.forward(c.X, c.Y, c.sd, c.wd)
    dA, dB = aset.backward(c.X, c.dY, c.sd, c.wd, dX=c.dX)
    for t in dA + dB:
        t.fill_(7.0)
    aset.backward(c.X, c.dY, c.sd, c.wd, accumulate=True)
    assert all(bool((t == 7).all()) for t in dA + dB)
    aset.backward(c.X, c.dY, c.sd, c.wd)
    assert not any(bool(t.any()) for t in dA + dB)
    # tokens, but no segment; segments, but no adapter
    c = Case(64, 96, [16, 8], [0], np.zeros(0, int), 50, seed=8)
    check_forward(c)
    check_backward(c)
    c = Case(64, 96, [16, 8], [0, 20, 50], [-1, 2], 50, seed=8)
    check_forward(c)
    check_backward(c)
    torch.cuda.synchronize()


def test_nan_and_inf_stay_with_their_tokens_and_adapters():
    torch = torch_mod()
    c = Case(256, 256, [16, 16, 40], [0, 40, 75, 90, 120], [0, 1, -1, 0], 120, seed=9)
    clean = c.set()
    X, Y, dY, dX = (getattr(c, k).clone() for k in ("X", "Y", "dY", "dX"))
    clean.forward(X, Y, c.sd, c.wd)
    cA, cB = clean.backward(X, dY, c.sd, c.wd, dX=dX)
    # a token of adapter 1, tokens without one, an unused adapter
    c.X[50, 3] = float("nan")
    c.dY[50, 5] = float("inf")
    c.X[80:90] = float("nan")
    c.dY[75:90] = float("nan")
    c.A[2].fill_(float("nan"))
    c.B[2].fill_(float("inf"))
    aset = c.set()
    aset.forward(c.X, c.Y, c.sd, c.wd)
    dA, dB = aset.backward(c.X, c.dY, c.sd, c.wd, dX=c.dX)
    torch.cuda.synchronize()
    keep = torch.ones(120, dtype=torch.bool, device="cuda:0")
    keep[50] = False
    assert torch.equal(c.Y[keep], Y[keep]) and bool(torch.isnan(c.Y[50]).all())
    assert torch.equal(c.dX[keep], dX[keep]) and not bool(torch.isfinite(c.dX[50]).any())
    for i in (0, 2):
        assert torch.equal(dA[i], cA[i]) and torch.equal(dB[i], cB[i])
    assert bool(torch.isnan(dA[1][:, 3]).all()) and not bool(torch.isfinite(dB[1][5]).any())


def test_equal_bits_again_on_another_stream_and_in_a_replayed_graph():
    torch = torch_mod()
    c = Case(512, 640, [16, 8, 16], [0, 33, 300, 301, 700], [1, 0, 2, 0], 700, seed=10)
    aset = c.set()
    Y0, dX0 = c.Y.clone(), c.dX.clone()
    aset.forward(c.X, c.Y, c.sd, c.wd)
    dA, dB = aset.backward(c.X, c.dY, c.sd, c.wd, dX=c.dX)
    torch.cuda.synchronize()
    want = [t.clone() for t in [c.Y, c.dX] + dA + dB]
    stream = torch.cuda.Stream()
    Y, dX = Y0.clone(), dX0.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        aset.forward(c.X, Y, c.sd, c.wd)
        aset.backward(c.X, c.dY, c.sd, c.wd, dX=dX)
    for k in range(3):
        for t in dA + dB:
            t.zero_()
        Y.copy_(Y0)
        dX.copy_(dX0)
        torch.cuda.synchronize()
        if k == 1:
            aset.forward(c.X, Y, c.sd, c.wd, stream=stream)
            aset.backward(c.X, c.dY, c.sd, c.wd, dX=dX, stream=stream)
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, [Y, dX] + dA + dB)), k


@pytest.mark.parametrize("what", ["A", "B", "X"])
def test_gradients_against_differences(what):
    """L = <dY, Y> is linear in each of A, B and x alone, so (L(+E) - L(-E)) / 2 is the derivative along E up to
    rounding: errors of fp32 sums walk randomly, so Y is off by less than (n + r + 4) u |Y| (the worst case of its
    terms' sizes, which exceed |Y| by the root of their number)."""
    torch = torch_mod()
    c = Case(192, 160, [12, 16], [0, 45, 80, 130], [0, 1, 0], 130, dtype="f32", seed=12)
    aset = c.set()
    c.dX.zero_()
    dA, dB = aset.backward(c.X, c.dY, c.sd, c.wd, dX=c.dX)
    gen = torch.Generator(device="cuda:0").manual_seed(3)
    tensors, grads = dict(A=(c.A, dA), B=(c.B, dB), X=([c.X], [c.dX]))[what]
    E = [torch.randn(t.shape, generator=gen, device="cuda:0") * t.std() for t in tensors]
    keep = [t.clone() for t in tensors]
    vals, size = [], 0.0
    for sign in (1.0, -1.0):
        for t, k, e in zip(tensors, keep, E):
            t.copy_(k + sign * e)
        Y = torch.zeros_like(c.Y)
        aset.forward(c.X, Y, c.sd, c.wd)
        vals.append(float((c.dY.double() * Y.double()).sum()))
        size += float((c.dY.double().abs() * Y.double().abs()).sum())
    diff = (vals[0] - vals[1]) / 2
    along = sum(float((g.double() * e.double()).sum()) for g, e in zip(grads, E))
    assert abs(diff - along) <= size * (160 + 16 + 4) * U


def test_refusals():
    torch = torch_mod()
    import orthogonal_reparameterized_poetx_amd as P
    c = Case(64, 96, [16, 8], [0, 30, 50], [0, 1], 50, seed=13)
    aset = c.set()
    d = "cuda:0"
    bad = [lambda: P.AdapterSet(64, 96, [], [], []), lambda: P.AdapterSet(64, 96, c.A, c.B[:1], c.scale),
           lambda: P.AdapterSet(64, 95, c.A, c.B, c.scale), lambda: P.AdapterSet(64, 96, c.B, c.A, c.scale),
           lambda: P.AdapterSet(64, 96, [a.half() for a in c.A], [b.half() for b in c.B], c.scale),
           lambda: P.AdapterSet(64, 96, [a.cpu() for a in c.A], [b.cpu() for b in c.B], c.scale),
           lambda: c.set(dA=[torch.zeros(16, 96, device=d)]),
           lambda: c.set(dA=[torch.zeros(16, 96, dtype=torch.bfloat16, device=d)] * 2),
           lambda: aset.forward(c.X.float(), c.Y, c.sd, c.wd), lambda: aset.forward(c.X, c.Y[:49], c.sd, c.wd),
           lambda: aset.forward(c.X.t(), c.Y, c.sd, c.wd), lambda: aset.forward(c.X, c.Y, c.sd.long(), c.wd),
           lambda: aset.forward(c.X, c.Y, c.sd[:2], c.wd), lambda: aset.forward(c.X, c.Y, c.sd.cpu(), c.wd),
           lambda: aset.forward(c.X, c.Y.as_strided((50, 64), (32, 1)), c.sd, c.wd),
           lambda: aset.backward(c.X, c.dY, c.sd, c.wd, dX=c.dX[:, :64])]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    big = torch.zeros(257, 96, dtype=torch.bfloat16, device=d)
    with pytest.raises(P.PoetxError):
        P.AdapterSet(64, 96, [big], [torch.zeros(64, 257, dtype=torch.bfloat16, device=d)], [1.0])


@pytest.mark.parametrize("ranks", [[32, 29], [64, 33], [128, 61], [256, 100]])
def test_wide_waves_of_an_expand(ranks):
    """Tiles enough for waves of 64 columns at every rank; an odd rank beside a whole one, widths past whole chunks."""
    c = Case(2504, 600, ranks, [0, 2000, 2003, 5403], [0, -1, 1], 5403, seed=sum(ranks))
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,n", [(1, 9), (3, 5), (9, 2), (8, 33), (35, 1)])
def test_pieces_at_the_end_of_a_matrix(m, n, dtype):
    """Widths and ranks of a few elements: 16-byte pieces then span several rows and the matrix's end."""
    c = Case(m, n, [1, 2, 3, 7], [0, 3, 4, 40, 41], [0, 1, 2, 3], 41, dtype=dtype, seed=10 * m + n)
    check_forward(c)
    check_backward(c)
    c = Case(m, n, [33, 20], [0, 3, 41], [0, 1], 41, dtype=dtype, seed=10 * m + n + 1)
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ranks", [[32, 16, 8, 29], [64, 1, 47, 16], [100, 3, 80, 112]])
@pytest.mark.parametrize("m,n", [(512, 768), (515, 773)])
def test_rank_groups_in_the_padding(m, n, ranks, dtype):
    """Few tiles: the ranks are shared out in groups of 16, and those of an adapter whose rank is at least 16 below
    its padding (to a multiple of 32) end in a group without a rank."""
    start = [0, 32, 64, 97, 130, 131, 190, 220, 256]
    c = Case(m, n, ranks, start, [0, 1, 2, 3, 1, 0, 2, 1], 256, dtype=dtype, seed=m + sum(ranks))
    check_forward(c)
    check_backward(c)


def _fill_freed_memory(torch):
    """Tensors of many sizes, so that blocks that were given back are in use again, and hold NaN."""
    return [torch.full((1 << k,), float("nan"), device="cuda:0") for k in range(7, 22) for _ in range(6)]


def test_replay_after_a_larger_call():
    """A server's order: decode captured, a prompt in between that needs a larger workspace, replay."""
    torch = torch_mod()
    ranks = [64, 16, 61, 32]
    c = Case(2048, 1024, ranks, np.arange(49), np.arange(48) % 5 - 1, 48, seed=30)
    big = Case(2048, 1024, ranks, [0, 1000, 3001], [2, 0], 3001, seed=31)
    dA, dB = ([torch.zeros(t.shape, device="cuda:0") for t in ts] for ts in (c.A, c.B))
    aset = c.set(dA=dA, dB=dB)
    Y0, dX0 = c.Y.clone(), c.dX.clone()
    Y, dX = Y0.clone(), dX0.clone()
    aset.forward(c.X, Y, c.sd, c.wd)
    aset.backward(c.X, c.dY, c.sd, c.wd, dX=dX)
    torch.cuda.synchronize()
    want = [t.clone() for t in [Y, dX] + dA + dB]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        aset.forward(c.X, Y, c.sd, c.wd)
        aset.backward(c.X, c.dY, c.sd, c.wd, dX=dX)
    for _ in range(3):
        aset.forward(big.X, big.Y, big.sd, big.wd)
        aset.backward(big.X, big.dY, big.sd, big.wd, dX=big.dX)
        torch.cuda.synchronize()
        held = _fill_freed_memory(torch)
        Y.copy_(Y0)
        dX.copy_(dX0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, [Y, dX] + dA + dB))
        assert all(bool(torch.isnan(t).all()) for t in held)
        del held


def test_replay_after_the_first_backward():
    """A forward captured before the set has gradients."""
    torch = torch_mod()
    c = Case(512, 640, [16, 40], [0, 33, 100], [1, 0], 100, seed=32)
    aset = c.set()
    Y0 = c.Y.clone()
    aset.forward(c.X, c.Y, c.sd, c.wd)
    torch.cuda.synchronize()
    want = c.Y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        aset.forward(c.X, c.Y, c.sd, c.wd)
    check_backward(c, aset)
    held = _fill_freed_memory(torch)
    for _ in range(3):
        c.Y.copy_(Y0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.Y, want)
        check_backward(c, aset)
    del held


def test_first_backward_inside_a_capture():
    torch = torch_mod()
    c = Case(64, 96, [16], [0, 33], [0], 33, seed=33)
    aset = c.set()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.X.add_(0)
        with pytest.raises(RuntimeError):
            aset.backward(c.X, c.dY, c.sd, c.wd)
    graph.replay()
    check_backward(c, aset)


def test_growth_on_another_stream():
    """A first and a larger call on a stream of their own, while the current stream's queued work still writes
    memory that it has given back."""
    torch = torch_mod()
    small = Case(512, 640, [16, 40], [0, 33, 100], [1, 0], 100, seed=34)
    big = Case(512, 640, [16, 40], [0, 333, 2000], [1, 0], 2000, seed=34)
    side = torch.cuda.Stream()
    want = []
    for c in (small, big):      # (one set for both: the adapters of the larger case)
        Y = c.Y.clone()
        big.set().forward(c.X, Y, c.sd, c.wd)
        want.append(Y)
    x = torch.randn(4096, 4096, device="cuda:0")
    for handle in (side, side.cuda_stream):
        aset = big.set()
        for c, w in zip((small, big), want):
            Y = c.Y.clone()
            torch.cuda.synchronize()
            junk = [torch.empty(1 << k, dtype=torch.uint8, device="cuda:0") for k in range(12, 24)]
            for _ in range(20):
                x = (x @ x).clamp(-1, 1)                     # the current stream is busy
            for t in junk:
                t.fill_(255)
            where = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in junk]
            del junk, t
            aset.forward(c.X, Y, c.sd, c.wd, stream=handle)
            ws = aset.workspace(0, c.N, len(c.which))
            assert all(ws.data_ptr() + ws.numel() <= lo or hi <= ws.data_ptr() for lo, hi in where)
            torch.cuda.synchronize()
            assert torch.equal(Y, w)


def test_object_gone_while_its_stream_is_busy():
    torch = torch_mod()
    c = Case(512, 640, [16, 40], [0, 33, 1000], [1, 0], 1000, seed=35)
    Y, want = c.Y.clone(), c.Y.clone()
    c.set().forward(c.X, want, c.sd, c.wd)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    x = torch.randn(4096, 4096, device="cuda:0")
    torch.cuda.synchronize()
    aset = c.set()
    with torch.cuda.stream(side):
        for _ in range(20):
            x = (x @ x).clamp(-1, 1)
    aset.forward(c.X, Y, c.sd, c.wd, stream=side)
    del aset
    held = _fill_freed_memory(torch)                         # on the current stream, at once
    torch.cuda.synchronize()
    assert torch.equal(Y, want) and all(bool(torch.isnan(t).all()) for t in held)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("count,which,lens", [
    (300, [299, 0, -1, 31, 32, 299, 64, 63], [40, 33, 5, 0, 64, 1, 200, 31]),
    (40, [39, 17, 5], [700, 0, 650]),
    (5000, [4999, 2500, 300, 4096], [1, 1, 1, 1]),
    (3, [2], [500]),
])
def test_more_adapters_than_segments(count, which, lens, dtype):
    """Partial sums lie by an adapter's place among those with tokens; the others' gradients are zero."""
    start = np.concatenate([[0], np.cumsum(lens)])
    c = Case(72, 40, [1 + i % 17 for i in range(count)] if count < 1000 else [2] * count, start, which, int(start[-1]),
             dtype=dtype, seed=count)
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ranks", [[16, 8], [5, 40]])
def test_segment_starts_outside_the_batch(ranks, dtype):
    """Starts below 0 and past N are taken as 0 and N; they do not decrease."""
    N = 150
    for start in ([-50, -3, 10, 40, 90, 200], [-2 ** 31, 2 ** 31 - 1], [0, 149, 150, 150, 151, 9999], [-7, 0, 0, 33],
                  [160, 170, 180], [-9, -5, 0]):
        which = [(1, 0, -1, 1, 0)[i % 5] for i in range(len(start) - 1)]
        c = Case(136, 200, ranks, start, which, N, dtype=dtype, seed=len(start))
        c.start = np.clip(c.start, 0, N)        # (the oracle's; the device has the others)
        check_forward(c)
        check_backward(c)
