"""The orthogonalised update of weights against its definition in 64 bits.

The tolerance of the iteration.  The kernels keep every matrix to 22 bits and add products in fp32,
cutting what they add, in chains of at most 64 additions: an entry of a product P Q is off by at
most 2^-18 (|P| |Q|).  How far such errors reach depends on the matrix (a weak singular value grows
by `a` in every step, and the errors in its direction with it), so the oracle iterates in 64 bits
twice, once exactly and once with each product's entries off by 2^-18 (|P| |Q|) times a random
number in [-1, 1], and the kernels may be four times as far from the exact result as that, in the
Frobenius norm of each matrix.  The store adds half a step of the type, relative to each value.
"""

import math
import time
from concurrent.futures import ThreadPoolExecutor

import pytest

torch = pytest.importorskip("torch")

from spherical_disco_convolution_b200 import disco as D  # noqa: E402
from spherical_disco_convolution_b200 import muon  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16
NS = muon.COEFFICIENTS
P = 4096  # a pointer no call below gets to use


# ------------------------------------------------------------------ refusals (no GPU)

def _status(fn, *args):
    with pytest.raises(D.DiscoError) as e:
        fn(*args)
    return e.value.status


def _orth(groups=1, rows=4, cols=8, dtype=0, steps=5, coef=NS, eps=1e-7, ps=(P,), outs=(P,), ws=P, nb=1 << 40):
    D.disco_orthogonalize(groups, rows, cols, dtype, D.newton_schulz(steps, coef, eps), list(ps), list(outs), ws, nb, None)


def _muon(lr=0.1, momentum=0.9, wd=0.0, w=(P,), g=(P,), m=(P,), wo=(P,), mo=(P,), dtype=0):
    D.disco_muon(1, 4, 8, dtype, D.newton_schulz(5, NS, 1e-7), lr, momentum, True, wd, list(w), list(g), list(m),
                 list(wo), list(mo), P, 1 << 40, None)


@pytest.mark.parametrize("kw,want", [
    (dict(groups=0), 1), (dict(rows=0), 1), (dict(cols=-3), 1), (dict(dtype=2), 1), (dict(steps=0), 1),
    (dict(steps=33), 1), (dict(coef=(math.nan, 0, 0)), 1), (dict(coef=(1, 33, 0)), 1), (dict(coef=(1, 0, -math.inf)), 1),
    (dict(eps=0.0), 1), (dict(eps=-1.0), 1), (dict(eps=9e-31), 1), (dict(eps=math.inf), 1), (dict(eps=math.nan), 1), (dict(ps=(None,)), 1), (dict(outs=(None,)), 1),
    (dict(ps=(P + 2,)), 1), (dict(outs=(P + 1,), dtype=1), 1), (dict(ws=None, rows=200, cols=300), 1),
    (dict(ws=P + 128), 1), (dict(nb=64, rows=200, cols=300), 1), (dict(ps=(), outs=()), 1), (dict(groups=65536), 2), (dict(rows=32769), 2), (dict(cols=40000), 2),
])
def test_orthogonalize_refuses(kw, want):
    assert _status(lambda: _orth(**kw)) == want


@pytest.mark.parametrize("kw", [
    dict(lr=math.inf), dict(wd=math.nan), dict(momentum=1.0), dict(momentum=-0.1), dict(momentum=math.nan),
    dict(w=(None,)), dict(g=(None,)), dict(m=(None,)), dict(wo=(None,)), dict(mo=(None,)), dict(m=(P + 2,)),
    dict(mo=(P + 2,), dtype=1), dict(g=(P + 1,), dtype=1),
])
def test_muon_refuses(kw):
    assert _status(lambda: _muon(**kw)) == D.DISCO_ERR_INVALID_ARG


def test_null_rule_and_workspace_size():
    assert D.library().disco_orthogonalize(1, 1, 4, 8, 0, None, None, None, None, 0, None) == D.DISCO_ERR_INVALID_ARG
    assert D.library().disco_orthogonalize_workspace_size(1, 1, 4, 8, None) == D.DISCO_ERR_INVALID_ARG
    assert _status(D.disco_orthogonalize_workspace_size, 0, 1, 4, 8) == D.DISCO_ERR_INVALID_ARG
    assert D.disco_orthogonalize_workspace_size(2, 2, 64, 192) == 0
    assert D.disco_orthogonalize_workspace_size(2, 2, 200, 300) > 0


@pytest.mark.parametrize("rows,cols", [(200, 300), (300, 600), (512, 4608), (1000, 1000)])
def test_the_workspace_of_many_tensors_serves_the_last_few(rows, cols):
    # 64 tensors go into one set of launches
    size = [D.disco_orthogonalize_workspace_size(n, 1, rows, cols) for n in range(1, 130)]
    for n in range(65, 130):
        assert size[n - 1] >= max(size[63], size[n % 64 - 1] if n % 64 else 0)


def test_python_refuses():
    w = torch.zeros(4, 3, 5)
    for call in (lambda: muon.orthogonalize(w), lambda: muon.orthogonalize([]), lambda: muon.muon_update(w, w, w, 0.1),
                 lambda: muon.muon_update([w], [w, w], [w], 0.1),
                 lambda: muon.Muon([torch.nn.Parameter(torch.zeros(4))]),
                 lambda: muon.Muon([torch.nn.Parameter(w)], groups=3),
                 lambda: muon.Muon([torch.nn.Parameter(w.transpose(0, 1))])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        muon.Muon([torch.nn.Parameter(w.half())])
    opt = muon.Muon([torch.nn.Parameter(w)])
    with pytest.raises(ValueError):
        opt.add_param_group({"params": [torch.nn.Parameter(torch.zeros(4))]})
    assert len(opt.param_groups) == 1


def test_momentum_stays_fp32_through_a_checkpoint():
    p = torch.nn.Parameter(torch.zeros(4, 6, dtype=BF16))
    opt = muon.Muon([p])
    m = torch.arange(24, dtype=F32).reshape(4, 6) / 7
    opt.state[p]["momentum_buffer"] = m.clone()
    again = muon.Muon([torch.nn.Parameter(torch.zeros(4, 6, dtype=BF16))])
    again.load_state_dict(opt.state_dict())
    got = again.state[again.param_groups[0]["params"][0]]["momentum_buffer"]
    assert got.dtype == F32 and torch.equal(got, m) and got.data_ptr() != m.data_ptr()


def test_a_first_step_is_not_captured(monkeypatch):
    p = torch.nn.Parameter(torch.zeros(4, 6))
    p.grad = torch.ones(4, 6)
    opt = muon.Muon([p])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError, match="before a CUDA graph"):
        opt.step()
    assert "momentum_buffer" not in opt.state[p]


# ------------------------------------------------------------------ the GPU's results

gpu = pytest.mark.gpu


@pytest.fixture
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def iterate(u, steps, coef, eps, gen=None):
    """u (matrices, rows, cols) in 64 bits; with gen, each product's entries off at random."""
    def mul(p, q):
        d = p @ q
        if gen is None:
            return d
        xi = 2 * torch.rand(d.shape, generator=gen, device=d.device, dtype=d.dtype) - 1
        return d + 2.0 ** -18 * xi * (p.abs() @ q.abs())

    a, b, c = coef
    tr = u.shape[1] > u.shape[2]
    x = u.mT if tr else u
    x = x / (torch.linalg.matrix_norm(x)[:, None, None] + eps)
    for _ in range(steps):
        g = mul(x, x.mT)
        x = mul(a * torch.eye(x.shape[1], device=x.device, dtype=x.dtype) + b * g + c * mul(g, g), x)
    return x.mT if tr else x


def matrices(t, groups):
    return t.double().reshape(groups, t.shape[0] // groups, -1)


def oracle(u, groups=1, steps=5, coef=NS, eps=1e-7):
    """(exact result, tolerance in each matrix's Frobenius norm), as matrices."""
    m = matrices(u, groups)
    gen = torch.Generator(device=u.device).manual_seed(99)
    want = iterate(m, steps, coef, eps)
    return want, 4 * torch.linalg.matrix_norm(iterate(m, steps, coef, eps, gen) - want)


def check(got, want, tol, dtype, groups, what):
    store = torch.linalg.matrix_norm(want) * torch.finfo(dtype).eps / 2
    err = torch.linalg.matrix_norm(matrices(got, groups) - want)
    assert torch.isfinite(got).all(), what
    assert (err <= tol + store + 1e-30).all(), f"{what}: off by {err.tolist()[:4]}, allowed {(tol + store).tolist()[:4]}"


def update(shape, dtype, seed, dev, scale=1e-3, noise=0.5):
    """A few strong directions of falling size over noise."""
    g = torch.Generator(device=dev).manual_seed(seed)
    rows, cols = shape[0], math.prod(shape[1:])
    r = min(6, rows, cols)
    u, v = torch.randn((rows, r), generator=g, device=dev), torch.randn((r, cols), generator=g, device=dev)
    t = (u * 0.5 ** torch.arange(r, device=dev)) @ v + noise * torch.randn((rows, cols), generator=g, device=dev)
    return (scale * t).reshape(shape).to(dtype)


# one value, one row, one column, both orientations, sides around the tiles of 64 and 128, lengths
# past one chain of 512, squares, the workloads' weights
SHAPES = [((1, 1), 1), ((1, 7), 1), ((9, 1), 1), ((2, 2), 1), ((4, 4, 3), 1), ((3, 5, 7), 1), ((32, 32, 3), 1),
          ((64, 64, 3), 1), ((64, 4, 3), 1), ((65, 63), 1), ((63, 65), 1), ((127, 129), 1), ((128, 128), 1),
          ((129, 127), 1), ((128, 64, 9), 1), ((256, 64, 9), 4), ((12, 5, 3), 4), ((96, 257), 3), ((130, 511), 1),
          ((200, 200), 1), ((257, 70, 3), 1), ((640, 131), 1), ((100, 2000), 1), ((2000, 37), 1), ((256, 256, 9), 1),
          ((384, 128, 3), 3), ((300, 513), 1)]


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape,groups", SHAPES)
def test_orthogonalize_matches_the_definition(shape, groups, dtype, cuda):
    u = update(shape, dtype, 1, cuda)
    want, tol = oracle(u, groups)
    check(muon.orthogonalize(u, groups), want, tol, dtype, groups, f"{shape}")


@gpu
@pytest.mark.parametrize("steps", [1, 2, 3, 8])
@pytest.mark.parametrize("coef", [NS, (1.5, -0.5, 0.0), (1.875, -1.25, 0.375)])
def test_other_steps_and_polynomials(steps, coef, cuda):
    for shape in [(48, 100), (150, 260)]:
        u = update(shape, F32, 2, cuda)
        want, tol = oracle(u, 1, steps, coef)
        check(muon.orthogonalize(u, 1, steps, coef), want, tol, F32, 1, f"{shape}")


@gpu
@pytest.mark.parametrize("shape", [(40, 70), (70, 40), (140, 300)])
def test_scaled_permutations_follow_the_scalar_polynomial(shape, cuda):
    """One value per row and column: every sum has one term, so a result is the scalar iteration of
    its value.  With e = 2^-23 (an operand of 22 bits and sign, or a product cut to 24 bits): A is
    off by 4.5 e (two operands, lo lo left out, the cut, its own store), A A by 10.5 e, and B X adds
    B's store, X's, lo lo and a cut: below 16 e = 2^-19 of each step's terms.  What a step hands on
    is stretched by the polynomial's derivative at the value."""
    gen = torch.Generator(device=cuda).manual_seed(3)
    k = min(shape)
    vals = torch.exp(3 * torch.randn(k, generator=gen, device=cuda)).float()
    at = torch.randperm(max(shape), generator=gen, device=cuda)[:k]
    u = torch.zeros(k, max(shape), device=cuda)
    u[torch.arange(k, device=cuda), at] = vals
    if shape[0] > shape[1]:
        u = u.T.contiguous()
    got = muon.orthogonalize(u)
    assert ((got != 0) == (u != 0)).all()
    s = vals.double() / (vals.double().norm() + 1e-7)
    a, b, c = NS
    tol = 2.0 ** -22 * s
    for _ in range(5):
        grow = (a + 3 * b * s ** 2 + 5 * c * s ** 4).abs()
        terms = a * s + abs(b) * s ** 3 + c * s ** 5
        s = a * s + b * s ** 3 + c * s ** 5
        tol = grow * tol + 2.0 ** -19 * terms
    g = got.T if shape[0] > shape[1] else got
    err = (g[torch.arange(k, device=cuda), at].double() - s).abs()
    assert (err <= tol).all(), f"worst {float((err / tol).max())} tolerances"


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_tensors_and_mixed_shapes(dtype, cuda):
    """Over one set of launches' 64 tensors, of three shapes, with groups."""
    shapes = [(8, 6, 3), (12, 40), (8, 6, 3)] * 5 + [(8, 6, 3)] * 60
    us = [update(s, dtype, 10 + i, cuda) for i, s in enumerate(shapes)]
    outs = muon.orthogonalize(us, groups=4)
    assert len(outs) == len(us)
    for u, o in zip(us, outs):
        want, tol = oracle(u, 4)
        check(o, want, tol, dtype, 4, "one of many")
    assert torch.equal(outs[0], muon.orthogonalize(us[0], groups=4))


@gpu
@pytest.mark.parametrize("shape", [(16, 40), (200, 300)])
def test_scale_zeros_and_bad_values(shape, cuda):
    u = update(shape, F32, 4, cuda)
    for scale in (1e-3, 1e4, 1e30):  # squares beyond fp32's range too
        v = u * scale
        want, tol = oracle(v)
        check(muon.orthogonalize(v), want, tol, F32, 1, f"scale {scale}")
    # |U| far below eps: X starts near U / eps, at 1e-14, where the pairs' fixed last place shows: X is
    # held times 2^12 with lo times 2^11, lo's last place is 2^-24, so an entry is off by up to 2^-48 in
    # each of five steps, and grows by `a` in each step after; n entries add up as their root
    v = u * 1e-18
    want, tol = oracle(v)
    floor = 2.0 ** -48 * math.sqrt(u.numel()) * sum(NS[0] ** k for k in range(6))
    check(muon.orthogonalize(v), want, tol + floor, F32, 1, "tiny")
    assert (muon.orthogonalize(torch.zeros_like(u)) == 0).all()
    v = u.clone()
    v[3] = 0  # a dead channel
    want, tol = oracle(v)
    got = muon.orthogonalize(v)
    check(got, want, tol, F32, 1, "dead channel")
    assert (got[3] == 0).all()
    pair = [u, u.clone()]
    pair[1][2, 3] = math.nan
    a, b = muon.orthogonalize(pair)
    assert torch.equal(a, muon.orthogonalize(u)) and torch.isnan(b).any()
    g2 = torch.cat([u, u])
    g2[2, 3] = math.inf
    assert torch.equal(muon.orthogonalize(g2, groups=2)[shape[0]:], a)


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("shape,groups", [((4, 4, 3), 1), ((64, 64, 3), 1), ((256, 64, 9), 4), ((200, 30), 1),
                                          ((260, 300), 1), ((150, 8, 3), 1)])
def test_the_whole_step(shape, groups, dtype, nesterov, cuda):
    lr, mom, wd = 0.05, 0.9, 0.1
    w = torch.randn(shape, device=cuda).to(dtype)
    g, m = update(shape, dtype, 5, cuda), update(shape, F32, 6, cuda)
    w1, m1 = muon.muon_update(w, g, m, lr, mom, nesterov, wd, groups)
    md = mom * m.double() + g.double()
    # one multiply-add in fp32; U keeps the rounded m' and one more rounding, 2^-22 of the whole
    assert ((m1.double() - md).abs() <= 2.0 ** -23 * (m.double().abs() + g.double().abs())).all()
    u = g.double() + mom * md if nesterov else md
    want, tol = oracle(u, groups)
    rows, cols = shape[0] // groups, math.prod(shape[1:])
    rate = lr * math.sqrt(max(1.0, rows / cols))
    step = (1 - lr * wd) * matrices(w, groups) - rate * want
    check(w1, step, 2 * rate * tol + 2.0 ** -22 * torch.linalg.matrix_norm(matrices(w, groups)), dtype, groups, "w'")
    w2, m2 = w.clone(), m.clone()
    r = muon.muon_update(w2, g, m2, lr, mom, nesterov, wd, groups, inplace=True)
    assert r[0] is w2 and r[1] is m2 and torch.equal(w2, w1) and torch.equal(m2, m1)


@gpu
def test_step_refusals(cuda):
    w = torch.randn(8, 6, device=cuda)
    m = torch.zeros_like(w)
    with pytest.raises(ValueError):
        muon.muon_update([w, w], [w, w], [m, m.clone()], 0.1, inplace=True)
    with pytest.raises(ValueError):
        muon.muon_update(w, w[:4].contiguous(), m, 0.1)
    with pytest.raises(TypeError):
        muon.muon_update(w, w, m.to(BF16), 0.1)
    with pytest.raises(TypeError):
        muon.muon_update(w.to(BF16), w, m, 0.1)
    with pytest.raises(ValueError):
        muon.muon_update(w, w, m, 0.1, groups=3)
    with pytest.raises(ValueError):
        muon.orthogonalize(w.T)
    with pytest.raises(ValueError):
        muon.orthogonalize(torch.zeros(0, 4, device=cuda))
    with pytest.raises(D.DiscoError):
        muon.orthogonalize(w, steps=0)


@gpu
@pytest.mark.parametrize("shape", [(20, 50), (60, 12), (140, 260)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_bases_off_sixteen_bytes_and_neighbours_untouched(shape, dtype, cuda):
    n = math.prod(shape)
    u = update(shape, dtype, 7, cuda)
    want = muon.orthogonalize(u)
    buf = torch.full((n + 64,), 3.0, dtype=dtype, device=cuda)
    src = torch.zeros(n + 8, dtype=dtype, device=cuda)
    v = src[3:3 + n].view(shape).copy_(u)
    nb = D.disco_orthogonalize_workspace_size(1, 1, *shape)
    ws = torch.empty(nb + 256, dtype=torch.uint8, device=cuda)
    code = D.DISCO_F32 if dtype == F32 else D.DISCO_BF16
    D.disco_orthogonalize(1, *shape, code, D.newton_schulz(5, NS, 1e-7), [v.data_ptr()], [buf[31:].data_ptr()],
                          ws.data_ptr(), nb, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(buf[31:31 + n].view(shape), want)
    assert (buf[:31] == 3).all() and (buf[31 + n:] == 3).all()


@gpu
@pytest.mark.parametrize("shape", [(20, 50), (60, 12), (140, 260), (90, 1000)])
def test_the_result_may_replace_the_update(shape, cuda):
    u = update(shape, F32, 17, cuda)
    want = muon.orthogonalize(u)
    nb = D.disco_orthogonalize_workspace_size(1, 1, *shape)
    ws = torch.empty(nb + 256, dtype=torch.uint8, device=cuda)
    D.disco_orthogonalize(1, *shape, D.DISCO_F32, D.newton_schulz(5, NS, 1e-7), [u.data_ptr()], [u.data_ptr()],
                          ws.data_ptr(), nb, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(u, want)


@gpu
def test_least_eps_and_scalars_as_tensors(cuda):
    assert (muon.orthogonalize(torch.zeros(20, 50, device=cuda), eps=1e-30) == 0).all()
    assert (muon.orthogonalize(torch.zeros(200, 300, device=cuda), eps=1e-30) == 0).all()
    w, g, m = (torch.randn(12, 30, device=cuda) for _ in range(3))
    a = muon.muon_update(w, g, m, torch.tensor(0.1), momentum=torch.tensor(0.5), weight_decay=torch.tensor(0.25))
    b = muon.muon_update(w, g, m, 0.1, momentum=0.5, weight_decay=0.25)
    assert torch.allclose(a[0], b[0], rtol=1e-6) and torch.equal(a[1], b[1])


@gpu
def test_streams_graphs_and_the_same_bits(cuda):
    for shape in [(64, 192), (200, 700)]:
        u = update(shape, F32, 8, cuda)
        want = muon.orthogonalize(u)
        assert torch.equal(muon.orthogonalize(u), want)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            a = muon.orthogonalize(u)
        b = muon.orthogonalize(u)  # at the same time, with a workspace of its own
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(a, want) and torch.equal(b, want)
        graphs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                o = muon.orthogonalize(u)
            graphs.append((g, o))
        u.copy_(update(shape, F32, 9, cuda))
        want = muon.orthogonalize(u)
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for _, o in graphs)
    D.disco_sync_status(torch.cuda.current_stream().cuda_stream)


@gpu
@pytest.mark.parametrize("shape", [(12, 20), (64, 192), (200, 300)])
def test_captured_steps_go_on_from_each_other(shape, cuda):
    p = torch.nn.Parameter(update(shape, F32, 50, cuda))
    p.grad = update(shape, F32, 51, cuda)
    w, m = p.detach().clone(), torch.zeros(shape, device=cuda)
    opt = muon.Muon([p], lr=0.1)
    opt.step()
    w, m = muon.muon_update(w, p.grad, m, 0.1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        opt.step()
    for k in range(2):
        p.grad.copy_(update(shape, F32, 52 + k, cuda))
        g.replay()
        w, m = muon.muon_update(w, p.grad, m, 0.1)
        torch.cuda.synchronize()
        assert torch.equal(p.detach(), w) and torch.equal(opt.state[p]["momentum_buffer"], m)


@gpu
def test_a_step_in_place_is_seen_by_autograd(cuda):
    w = torch.nn.Parameter(torch.randn(8, 12, device=cuda))
    x = torch.randn(5, 8, device=cuda, requires_grad=True)
    y = (x @ w).sum()
    opt = muon.Muon([w])
    w.grad = torch.randn_like(w)
    opt.step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


@gpu
def test_two_threads_at_once(cuda):
    # sizes of one kernel each that differ in the shared memory they ask for
    for shapes in [((30, 60), (30, 1500)), ((60, 64), (60, 2000)), ((200, 300), (140, 900))]:
        us = [update(s, F32, 40 + i, cuda) for i, s in enumerate(shapes)]
        want = [muon.orthogonalize(u) for u in us]
        torch.cuda.synchronize()

        def work(i):
            with torch.cuda.stream(torch.cuda.Stream()):
                got = [muon.orthogonalize(us[i]) for _ in range(200)]
            torch.cuda.synchronize()
            return all(torch.equal(o, want[i]) for o in got)

        with ThreadPoolExecutor(2) as pool:
            assert all(pool.map(work, range(2)))


@gpu
def test_optimizer_steps_as_the_function_does(cuda):
    torch.manual_seed(0)
    ps = [torch.nn.Parameter(torch.randn(s, device=cuda).to(t)) for s, t in
          [((8, 6, 3), F32), ((8, 6, 3), F32), ((16, 5), BF16), ((24, 4, 3), F32)]]
    idle = torch.nn.Parameter(torch.randn(4, 4, device=cuda))
    opt = muon.Muon([{"params": ps[:3] + [idle]}, {"params": ps[3:], "groups": 4, "lr": 0.1}], lr=0.03, weight_decay=0.02)
    ws, ms = [p.detach().clone() for p in ps], [torch.zeros(p.shape, device=cuda) for p in ps]
    kept = idle.detach().clone()
    for k in range(3):
        for i, p in enumerate(ps):
            p.grad = update(p.shape, p.dtype, 20 + 7 * k + i, cuda)
        assert opt.step(lambda: 1.5) == 1.5
        for i, p in enumerate(ps):
            ws[i], ms[i] = muon.muon_update(ws[i], p.grad, ms[i], 0.1 if i == 3 else 0.03, weight_decay=0.02,
                                            groups=4 if i == 3 else 1)
            assert torch.equal(p.detach(), ws[i]) and torch.equal(opt.state[p]["momentum_buffer"], ms[i])
    assert torch.equal(idle.detach(), kept) and idle not in opt.state


@gpu
@pytest.mark.parametrize("dtype,fused", [(F32, False), (BF16, True)])
def test_a_block_trains_with_norm_and_update(dtype, fused, cuda):
    """Convolution, norm, convolution, loss, backward, update: the gradients agree with the formulas
    (the norm replaced by elementary operations), and the step moves every weight as muon_update says."""
    from spherical_disco_convolution_b200.conv import DiscreteContinuousConvS2
    from spherical_disco_convolution_b200.norm import LayerNormS2

    torch.manual_seed(1)
    kw = dict(kernel_shape=(3,), theta_cutoff=0.3, device=cuda, dtype=dtype, fused=fused)
    c1 = DiscreteContinuousConvS2(32, 64, (33, 64), (33, 64), **kw)
    c2 = DiscreteContinuousConvS2(64, 32, (33, 64), (33, 64), groups=2, **kw)
    ln = LayerNormS2(64, device=cuda, dtype=dtype)
    x = torch.randn(2, 32, 33, 64, device=cuda).to(dtype)
    v = torch.randn(2, 32, 33, 64, device=cuda).to(dtype)

    def plain_norm(y):
        y = y.float()
        d = y - y.mean(1, keepdim=True)
        o = d * ((d * d).mean(1, keepdim=True) + ln.eps).rsqrt()
        return (o * ln.weight.float().view(1, -1, 1, 1) + ln.bias.float().view(1, -1, 1, 1)).to(dtype)

    leaves = [c1.weight, c1.bias, ln.weight, ln.bias, c2.weight, c2.bias]
    grads = []
    for n in (ln, plain_norm):
        for p in leaves:
            p.grad = None
        c2(n(c1(x))).backward(v)
        grads.append([p.grad.double() for p in leaves])
    # between the two the field and its gradient are rounded once each to the type, from values that
    # differ by a few 32-bit roundings: most agree to the bit, the rest by one step
    for a, b in zip(*grads):
        assert torch.linalg.vector_norm(a - b) <= (2.0 ** -7 if dtype == BF16 else 2.0 ** -18) * torch.linalg.vector_norm(b)
    opt = muon.Muon([{"params": [c1.weight]}, {"params": [c2.weight], "groups": 2}], lr=0.02)
    for p in leaves:
        p.grad = None
    c2(ln(c1(x))).backward(v)
    want = [muon.muon_update(c.weight.detach(), c.weight.grad, torch.zeros(c.weight.shape, device=cuda), 0.02, groups=g)[0]
            for c, g in ((c1, 1), (c2, 2))]
    opt.step()
    assert torch.equal(c1.weight.detach(), want[0]) and torch.equal(c2.weight.detach(), want[1])
    assert torch.isfinite(c2(ln(c1(x)))).all()


def _independent(outs):
    """Results share neither memory nor a version: one changed in place leaves what autograd saved of
    another, and one kept or saved holds no memory of the others."""
    assert len({o.untyped_storage().data_ptr() for o in outs}) == len(outs)
    assert all(o.untyped_storage().nbytes() == o.numel() * o.element_size() for o in outs)
    w = outs[1].detach().requires_grad_()
    y = (w * outs[0]).sum()
    for o in outs[1:]:
        before = outs[0]._version
        with torch.no_grad():
            o.add_(1)
        assert outs[0]._version == before
    y.backward()


@pytest.mark.parametrize("shape", [(4, 6), (4, 8, 3), (3, 5)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_results_of_a_list_are_independent(shape, dtype):
    _independent(muon._outputs(torch.zeros(shape, dtype=dtype), 4))


@gpu
@pytest.mark.parametrize("shape", [(4, 8, 3), (3, 5), (64, 64)])
def test_results_of_calls_are_independent(shape, cuda):
    us = [update(shape, F32, 70 + i, cuda) for i in range(3)]
    _independent(muon.orthogonalize(us))
    ws, ms = muon.muon_update(us, us, [u.clone() for u in us], 0.1)
    _independent(ws)
    _independent(ms)


# ------------------------------------------------------------------ every form of the tiled products
#
# What each reaches (tiles of 128 or 256 rows; S parts of K for X X^T / A A / B X):
#   (1024, 1024, 9), (9216, 1024)  256, on pairs, with partial sums: 7 / 4 / 1, the second one transposed
#   (1200, 70, 60) in 4 groups, (1000, 4501), (4610, 1000)  256, padded, rows off 16 bytes, transposed
#   (512, 512, 9), (512, 1000), (512, 2000)   128: 8 / 8 / 1, 8 / 8 / 4 and 8 / 8 / 2
#   (400, 500), (500, 400)                    128: 8 / 8 / 8, the second one's store transposed
#   (1000, 512)                               128: the transposed store of a cluster of 4
# and sides of at most 32 that are too long for the fp32 form: (32, 4608), (24, 12000) on 64-row and
# 128-row tiles, (32, 9216), (6000, 20), (8, 20000).
TILED = [((1024, 1024, 9), 1), ((9216, 1024), 1), ((1200, 70, 60), 4), ((1000, 4501), 1), ((4610, 1000), 1), ((512, 512, 9), 1),
         ((512, 1000), 1), ((512, 2000), 1), ((400, 500), 1), ((500, 400), 1), ((1000, 512), 1), ((32, 4608), 1), ((24, 12000), 1),
         ((32, 9216), 1), ((6000, 20), 1), ((8, 20000), 1)]


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape,groups", TILED)
def test_tiled_forms_match_the_definition(shape, groups, dtype, cuda):
    u = update(shape, dtype, 80, cuda)
    want, tol = oracle(u, groups)
    got = muon.orthogonalize(u, groups)
    check(got, want, tol, dtype, groups, f"{shape}")
    assert torch.equal(muon.orthogonalize(u, groups), got)


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape,groups", [((1024, 512, 9), 1), ((4610, 1000), 1), ((1200, 70, 60), 4), ((512, 1000), 1),
                                          ((500, 400), 1), ((32, 9216), 1), ((6000, 20), 1), ((300, 513), 1)])
def test_tiled_steps_in_place(shape, groups, dtype, cuda):
    lr, mom, wd = 0.05, 0.9, 0.1
    w = torch.randn(shape, device=cuda).to(dtype)
    g, m = update(shape, dtype, 81, cuda), update(shape, F32, 82, cuda)
    w0, m0 = w.clone(), m.clone()
    w1, m1 = muon.muon_update(w, g, m, lr, mom, True, wd, groups)
    assert torch.equal(w, w0) and torch.equal(m, m0)
    md = mom * m.double() + g.double()
    assert ((m1.double() - md).abs() <= 2.0 ** -23 * (m.double().abs() + g.double().abs())).all()
    want, tol = oracle(g.double() + mom * md, groups)
    rate = lr * math.sqrt(max(1.0, shape[0] / groups / math.prod(shape[1:])))
    step = (1 - lr * wd) * matrices(w, groups) - rate * want
    check(w1, step, 2 * rate * tol + 2.0 ** -22 * torch.linalg.matrix_norm(matrices(w, groups)), dtype, groups, "w'")
    muon.muon_update(w, g, m, lr, mom, True, wd, groups, inplace=True)
    assert torch.equal(w, w1) and torch.equal(m, m1)


@gpu
@pytest.mark.parametrize("count,shape", [(8, (300, 70, 60)), (70, (200, 700)), (79, (200, 700)), (66, (300, 513)), (65, (140, 260)), (130, (150, 40))])
def test_many_tensors_in_tiled_forms(count, shape, cuda):
    """Several sets of 64 tensors through one workspace of the exact size, the last set on tiles and
    splits of its own; what lies behind workspace and results stays as it was."""
    us = [update(shape, F32, 83 + i, cuda) for i in range(count)]
    n = math.prod(shape)
    rows, cols = shape[0], n // shape[0]
    nb = D.disco_orthogonalize_workspace_size(count, 1, rows, cols)
    ws = torch.full((nb + 4096,), 0xff, dtype=torch.uint8, device=cuda)  # NaN in every type
    outs = [torch.full((n + 8,), 5.0, device=cuda) for _ in us]
    D.disco_orthogonalize(1, rows, cols, D.DISCO_F32, D.newton_schulz(5, NS, 1e-7), [u.data_ptr() for u in us],
                          [o.data_ptr() for o in outs], ws.data_ptr() if nb else None, nb, torch.cuda.current_stream().cuda_stream)
    assert (ws[nb:] == 0xff).all()
    for u, o in zip(us, outs):
        assert (o[n:] == 5).all()
        want, tol = oracle(u)
        check(o[:n].view(shape), want, tol, F32, 1, "one of many")
    assert all(torch.equal(a, o[:n].view(shape)) for a, o in zip(muon.orthogonalize(us), outs))


@gpu
@pytest.mark.parametrize("shape,groups", [((1200, 70, 60), 4), ((512, 1000), 1), ((24, 12000), 1)])
def test_bad_values_spread_over_their_own_matrix_only(shape, groups, cuda):
    us = [update(shape, F32, 90 + i, cuda) for i in range(2)]
    want = muon.orthogonalize(us, groups)
    bad = [us[0], us[1].clone()]
    bad[1][1, 2] = math.nan
    got = muon.orthogonalize(bad, groups)
    assert torch.equal(got[0], want[0]) and torch.isnan(got[1]).any()
    rows = shape[0] // groups
    assert torch.equal(got[1][rows:], want[1][rows:])


# ------------------------------------------------------------------ a wait that runs out

def test_the_wait_self_test_refuses():
    def call(limit=1000, rows=64, cols=192, w=(P,)):
        D.disco_muon_wait_selftest(limit, 1, rows, cols, 0, D.newton_schulz(5, NS, 1e-7), 0.1, 0.9, True, 0.0, list(w), [P],
                                   [P], list(w), [P], P, 1 << 40, None)

    assert _status(lambda: call(limit=0)) == D.DISCO_ERR_INVALID_ARG
    assert _status(lambda: call(limit=1000001)) == D.DISCO_ERR_INVALID_ARG
    assert _status(lambda: call(rows=32)) == D.DISCO_ERR_UNSUPPORTED
    assert _status(lambda: call(w=(None,))) == D.DISCO_ERR_INVALID_ARG


@gpu
@pytest.mark.parametrize("steps", [1, 5, 32])
@pytest.mark.parametrize("count,shape", [(1, (64, 192)), (3, (100, 2000)), (1, (140, 260)), (1, (512, 1000)), (1, (400, 500)),
                                         (1, (1024, 4608)), (66, (300, 513))])
def test_after_a_wait_that_ran_out_no_weight_is_written(count, shape, steps, cuda):
    """The first product withheld, waits of 1 ms: the call ends soon whatever the number of steps (each of
    its kernels may take the 2 ms in which copies land), says so once, and the weights stay."""
    n, st = count, torch.cuda.current_stream().cuda_stream
    ws = [torch.randn(shape, device=cuda) for _ in range(n)]
    gs, ms = [update(shape, F32, 95, cuda)] * n, [torch.zeros(shape, device=cuda) for _ in range(n)]
    want = muon.muon_update(ws, gs, ms, 0.1, steps=steps)
    w0 = [w.clone() for w in ws]
    nb = D.disco_orthogonalize_workspace_size(n, 1, *shape)
    work = torch.full((nb + 256,), 0xff, dtype=torch.uint8, device=cuda)
    wp, gp, mp = ([t.data_ptr() for t in ts] for ts in (ws, gs, ms))
    D.disco_sync_status(st)
    t0 = time.perf_counter()
    D.disco_muon_wait_selftest(1000, 1, *shape, D.DISCO_F32, D.newton_schulz(steps, NS, 1e-7), 0.1, 0.95, True, 0.0, wp, gp,
                               mp, wp, mp, work.data_ptr(), nb, st)
    with pytest.raises(D.DiscoError) as e:
        D.disco_sync_status(st)
    assert e.value.status == D.DISCO_ERR_TIMEOUT and time.perf_counter() - t0 < 2.0
    D.disco_sync_status(st)
    assert all(torch.equal(a, b) for a, b in zip(ws, w0)) and all(torch.equal(a, b) for a, b in zip(ms, want[1]))
    assert (work[nb:] == 0xff).all()
    got = muon.muon_update(ws, gs, [torch.zeros_like(m) for m in ms], 0.1, steps=steps)
    assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))
    D.disco_sync_status(st)


@gpu
@pytest.mark.parametrize("shape", [(4, 12), (16, 40), (30, 4000), (60, 300), (100, 2000), (200, 300), (300, 6000), (500, 40)])
@pytest.mark.parametrize("top", [1e38, 3e38])
def test_updates_near_the_largest_numbers(shape, top, cuda):
    """1 / |U| is below fp32's normal numbers here."""
    u = update(shape, F32, 96, cuda)
    u = (u.double() * (top / float(u.abs().max()))).float()  # the factor is beyond fp32
    want, tol = oracle(u)
    check(muon.orthogonalize(u), want, tol, F32, 1, f"{shape}")


@gpu
@pytest.mark.parametrize("shape", [(12, 30), (40, 70), (140, 300)])
def test_iterates_within_the_pairs_range(shape, cuda):
    """Coefficients that let X grow: singular values of up to 4 before a step, entries of B of up to 100."""
    u = update(shape, F32, 97, cuda)
    for steps, coef in ((3, (2.0, 0.0, 0.0)), (1, (32.0, 32.0, 32.0)), (2, (1.0, 1.0, 1.0))):
        want, tol = oracle(u, 1, steps, coef)
        check(muon.orthogonalize(u, 1, steps, coef), want, tol, F32, 1, f"{shape} {coef}")


@gpu
def test_nothing_is_written_where_one_tensor_is_refused(cuda):
    """A list of two shapes, the second beyond the library's sides: the first is left as it was."""
    ws = [torch.randn(8, 12, device=cuda), torch.randn(32769, 2, device=cuda)]
    gs, ms = [torch.randn_like(w) for w in ws], [torch.zeros_like(w) for w in ws]
    kept = [w.clone() for w in ws]
    with pytest.raises(D.DiscoError) as e:
        muon.muon_update(ws, gs, ms, 0.1, inplace=True)
    assert e.value.status == D.DISCO_ERR_UNSUPPORTED
    assert all(torch.equal(w, k) for w, k in zip(ws, kept)) and not ms[0].any()
    ps = [torch.nn.Parameter(w.clone()) for w in ws]
    for p, g in zip(ps, gs):
        p.grad = g
    opt = muon.Muon([{"params": [ps[0]]}, {"params": [ps[1]]}])
    with pytest.raises(D.DiscoError):
        opt.step()
    assert torch.equal(ps[0].detach(), ws[0])
