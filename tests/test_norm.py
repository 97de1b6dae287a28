"""Layer norm over the channels of a field: forward and backward against the formulas in 64 bits.

Tolerances, element by element, from the roundings of a 32-bit evaluation (u = 2^-24).  With r =
1 / deviation, A = max_c |x| r at a point and XH = max_c |xh|:
  * a sum over channels takes at most n = 40 additions in a row up to 512 channels, and n = 24 + C / 64
    above (64 rows of lanes, each over every 64th channel, then their sums), so the mean is off by
    at most n u max|x| and a difference x - mean by (n + 1) u max|x|; r then is off by a relative
    (n + 1) u A + n u, and |d xh| <= (n + 8) u (A + |xh| (1 + A));
  * dx = r (e - s1 - xh s2): with E = max_c |e| and xh off by at most 4 u (A + XH) (the statistics
    come in rounded to 32 bits), |d dx| <= u r E ((n + 8) (1 + XH^2) + 8 XH (A + XH));
  * dgain and dbias are sums of fewer than 128 additions in a row over partial sums, so they are off
    by at most 128 u sum |terms|, plus what xh is off in each term;
and the store rounds to the field's type, half a step relative to the value.
"""

import math
from concurrent.futures import ThreadPoolExecutor

import pytest

torch = pytest.importorskip("torch")

from spherical_disco_convolution_b200 import disco as D  # noqa: E402
from spherical_disco_convolution_b200 import norm  # noqa: E402

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


# ------------------------------------------------------------------ refusals (no GPU)

def _status(fn, *args):
    with pytest.raises(D.DiscoError) as e:
        fn(*args)
    return e.value.status


P = 4096  # a pointer no call below gets to use


@pytest.mark.parametrize("B,C,n,dtype,want", [
    (0, 4, 8, 0, D.DISCO_ERR_INVALID_ARG), (1, 0, 8, 0, D.DISCO_ERR_INVALID_ARG), (1, 4, 0, 0, D.DISCO_ERR_INVALID_ARG),
    (-1, 4, 8, 0, D.DISCO_ERR_INVALID_ARG), (1, 4, 8, 7, D.DISCO_ERR_INVALID_ARG),
    (1, 16385, 8, 0, D.DISCO_ERR_UNSUPPORTED), (1, 4, 2 ** 31, 0, D.DISCO_ERR_UNSUPPORTED),
])
def test_sizes_are_refused(B, C, n, dtype, want):
    assert _status(D.disco_norm, B, C, n, dtype, P, P, P, 1e-5, P, P, None) == want
    assert _status(D.disco_norm_backward, B, C, n, dtype, P, P, P, P, P, P, P, P, 1 << 40, None) == want
    assert _status(D.disco_norm_workspace_size, B, C, n, dtype) == want


def test_pointers_and_scalars_are_refused():
    inv = D.DISCO_ERR_INVALID_ARG
    assert _status(D.disco_norm, 1, 4, 8, 0, None, P, P, 1e-5, P, P, None) == inv
    assert _status(D.disco_norm, 1, 4, 8, 0, P, P, P, 1e-5, None, P, None) == inv
    for eps in (-1e-5, math.inf, math.nan):
        assert _status(D.disco_norm, 1, 4, 8, 0, P, P, P, eps, P, P, None) == inv
    assert _status(D.disco_norm, 1, 4, 8, 0, P + 2, P, P, 1e-5, P, P, None) == inv
    assert _status(D.disco_norm, 1, 4, 8, 1, P + 1, P, P, 1e-5, P, P, None) == inv
    need = D.disco_norm_workspace_size(1, 4, 8, 0)
    assert need > 0
    back = [1, 4, 8, 0, P, P, P, P, P, P, P, P, need, None]
    for i, v in [(4, None), (5, None), (6, None), (11, None), (12, need - 1), (4, P + 2), (6, P + 2), (11, P + 1)]:
        args = list(back)
        args[i] = v
        assert _status(D.disco_norm_backward, *args) == inv
    args = list(back)
    args[8] = args[9] = args[10] = None
    assert _status(D.disco_norm_backward, *args) == inv


def test_cpu_tensors_and_wrong_modules_are_refused():
    x = torch.zeros(2, 3, 4, 5)
    with pytest.raises(ValueError):
        norm.layer_norm(x)
    with pytest.raises(ValueError):
        norm.layer_norm_backward(x, x, torch.zeros(2, 2, 4, 5))
    with pytest.raises(ValueError):
        norm.LayerNormS2(0)
    with pytest.raises(TypeError):
        norm.LayerNormS2(4, dtype=torch.float16)
    with pytest.raises(ValueError):
        norm.LayerNormS2(4)(x)
    m = norm.LayerNormS2(3, affine=False)
    assert not list(m.parameters())
    assert [n for n, _ in norm.LayerNormS2(3, bias=False).named_parameters()] == ["weight"]


# ------------------------------------------------------------------ the GPU's results

gpu = pytest.mark.gpu


@pytest.fixture
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def field(shape, dtype, seed, dev, offset=0.5, spread=1.0):
    g = torch.Generator(device=dev).manual_seed(seed)
    B, C = shape[:2]
    ones = (1,) * (len(shape) - 2)
    mu = offset * torch.randn((B, C) + ones, generator=g, device=dev)
    sd = spread * (0.5 + torch.rand((B, C) + ones, generator=g, device=dev))
    return (mu + sd * torch.randn(shape, generator=g, device=dev)).to(dtype)


def col(v, x):
    return v.double().view((1, -1) + (1,) * (x.dim() - 2))


def check(got, want, tol, what):
    assert got.shape == want.shape, what
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol).nan_to_num(1e30).max()):.3g} tolerances"


def adds(x):
    return 40 if x.shape[1] <= 512 else 24 + x.shape[1] // 64


def half_step(t, dtype):
    return torch.finfo(dtype).eps / 2 * t.abs()


def oracle(x, gain, bias, eps):
    xd = x.double()
    mean = xd.mean(1, keepdim=True)
    d = xd - mean
    r = 1 / ((d * d).mean(1, keepdim=True) + eps).sqrt()
    xh = d * r
    out = xh * (1 if gain is None else col(gain, x)) + (0 if bias is None else col(bias, x))
    return out, mean, r, xh


def check_forward(x, gain, bias, eps):
    out, stats = norm.layer_norm(x, gain, bias, eps)
    want, mean, r, xh = oracle(x, gain, bias, eps)
    A = x.double().abs().amax(1, keepdim=True) * r
    ga = 1.0 if gain is None else col(gain, x).abs()
    bi = 0.0 if bias is None else col(bias, x).abs()
    n = adds(x)
    check(out, want, (n + 8) * U * (A + xh.abs() * (1 + A)) * ga + U * bi + half_step(want, x.dtype) * (1 + 2 ** -6) + 1e-37,
          "out")
    check(stats[0].unsqueeze(1), mean, (n + 1) * U * x.double().abs().amax(1, keepdim=True) + 1e-37, "mean")
    check(stats[1].unsqueeze(1), r, ((n + 1) * U * A + (n + 1) * U) * r, "1 / deviation")
    return stats


def check_backward(dout, x, gain, eps):
    _, mean, r, xh = oracle(x, gain, None, eps)
    stats = torch.cat([mean, r], 1).transpose(0, 1).float().contiguous()
    dx, dgain, dbias = norm.layer_norm_backward(dout, x, stats, gain)
    do = dout.double()
    e = do * (1 if gain is None else col(gain, x))
    want = r * (e - e.mean(1, keepdim=True) - xh * (e * xh).mean(1, keepdim=True))
    A, XH, E = (t.amax(1, keepdim=True) for t in (x.double().abs() * r, xh.abs(), e.abs()))
    check(dx, want, U * r * E * ((adds(x) + 8) * (1 + XH ** 2) + 8 * XH * (A + XH)) + half_step(want, x.dtype) * (1 + 2 ** -6) + 1e-37,
          "dx")
    dims = [0] + list(range(2, x.dim()))
    terms = do * xh
    want = terms.sum(dims)
    check(dgain, want, U * (128 * terms.abs() + 4 * do.abs() * (A + XH)).sum(dims) + half_step(want, x.dtype) * (1 + 2 ** -6)
          + 1e-37, "dgain")
    want = do.sum(dims)
    check(dbias, want, 128 * U * do.abs().sum(dims) + half_step(want, x.dtype) * (1 + 2 ** -6) + 1e-37, "dbias")


# one point, one channel, one value; points that end inside a vector, a tile, a plane; channel
# counts around each split of the rows; more channels than registers hold
SHAPES = [(1, 1, 1, 1), (1, 4, 1, 1), (3, 5, 1, 1), (700, 33, 1, 1), (1, 2, 3, 3), (2, 3, 7, 9), (1, 4, 17, 32),
          (2, 8, 5, 8), (1, 9, 4, 6), (3, 50, 61, 121), (2, 63, 12, 20), (2, 64, 12, 20), (1, 65, 9, 20),
          (1, 128, 33, 34), (1, 129, 16, 16), (2, 256, 19, 36), (1, 257, 8, 9), (1, 511, 6, 11), (1, 512, 16, 24),
          (1, 513, 6, 8), (2, 1500, 3, 5), (1, 64, 181, 360), (4, 32, 91, 180), (1, 77, 91, 181),
          (1, 1, 181, 424), (2, 5, 181, 424), (1, 8, 181, 424), (1, 8, 181, 423), (2, 13, 140, 300), (2, 16, 140, 300),
          (1, 30, 183, 426), (1, 128, 181, 360), (1, 130, 181, 361), (1, 256, 120, 180), (1, 300, 120, 180),
          (1, 512, 90, 120), (1, 700, 64, 128), (1, 1024, 32, 72), (1, 1025, 16, 20)]


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward_match_the_formulas(shape, dtype, cuda):
    x, dout = field(shape, dtype, 1, cuda), field(shape, dtype, 2, cuda, 0.1)
    g = torch.Generator(device=cuda).manual_seed(3)
    gain = (1 + 0.3 * torch.randn(shape[1], generator=g, device=cuda)).to(dtype)
    bias = torch.randn(shape[1], generator=g, device=cuda).to(dtype)
    check_forward(x, gain, bias, 1e-5)
    check_backward(dout, x, gain, 1e-5)


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_most_channels(dtype, cuda):
    x, dout = field((1, norm_channels(), 2, 3), dtype, 4, cuda), field((1, norm_channels(), 2, 3), dtype, 5, cuda)
    check_forward(x, None, None, 1e-5)
    check_backward(dout, x, None, 1e-5)


def norm_channels():
    return 16384


@gpu
@pytest.mark.parametrize("affine", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("shape", [(2, 5), (3, 7, 10), (2, 16, 3, 4, 5)])
def test_other_axes_and_missing_parameters(shape, affine, cuda):
    x, dout = field(shape, F32, 6, cuda), field(shape, F32, 7, cuda)
    gain = torch.randn(shape[1], device=cuda) if affine[0] else None
    bias = torch.randn(shape[1], device=cuda) if affine[1] else None
    check_forward(x, gain, bias, 1e-3)
    check_backward(dout, x, gain, 1e-3)


@gpu
@pytest.mark.parametrize("offset", [30.0, 1000.0])
def test_fields_far_from_zero(offset, cuda):
    """A deviation formed as a difference of large sums would lose what the tolerance allows."""
    x = field((1, 64, 9, 16), F32, 8, cuda, offset=0.0) + offset
    check_forward(x, None, None, 1e-5)
    check_backward(field(x.shape, F32, 9, cuda), x, None, 1e-5)


@gpu
def test_constant_channels_and_zero_eps(cuda):
    x = torch.full((1, 24, 3, 5), 3.25, device=cuda)
    out, stats = norm.layer_norm(x, None, torch.ones(24, device=cuda), 1e-5)
    assert (out == 1).all() and (stats[0] == 3.25).all()
    assert torch.allclose(stats[1], torch.full_like(stats[1], 1e-5 ** -0.5), rtol=1e-6)
    x = field((1, 24, 3, 5), F32, 10, cuda)
    check_forward(x, None, None, 0.0)


@gpu
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_bad_points_stay_their_own(bad, cuda):
    """NaN and infinities spoil their point's channels and no other point (and the parameters' sums)."""
    x, dout = field((2, 20, 6, 7), F32, 11, cuda), field((2, 20, 6, 7), F32, 12, cuda)
    y = x.clone()
    y[1, 3, 2, 4] = bad
    a, sa = norm.layer_norm(x)
    b, sb = norm.layer_norm(y)
    hit = torch.zeros(2, 1, 6, 7, dtype=torch.bool, device=cuda)
    hit[1, 0, 2, 4] = True
    assert torch.equal(a[~hit.expand_as(a)], b[~hit.expand_as(b)])
    assert torch.isnan(b[1, :, 2, 4]).any()
    da = norm.layer_norm_backward(dout, x, sa)[0]
    db = norm.layer_norm_backward(dout, y, sb)[0]
    assert torch.equal(da[~hit.expand_as(da)], db[~hit.expand_as(db)])


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shift", [1, 2, 3, 4])
def test_bases_off_sixteen_bytes(dtype, shift, cuda):
    """Dense tensors that start inside an allocation, at any element."""
    shape, n = (2, 12, 5, 16), 2 * 12 * 5 * 16

    def off(t, k):
        buf = torch.empty(n + 8, dtype=dtype, device=cuda)
        v = buf[k:k + n].view(shape)
        v.copy_(t)
        return v

    x, dout = off(field(shape, dtype, 13, cuda), shift), off(field(shape, dtype, 14, cuda), shift + 1)
    check_forward(x, None, None, 1e-5)
    check_backward(dout, x, None, 1e-5)


@gpu
def test_results_stay_inside_their_tensors(cuda):
    shape, n = (1, 6, 5, 7), 210
    x = field(shape, F32, 15, cuda)
    buf = torch.full((n + 64,), 7.0, device=cuda)
    out = buf[32:32 + n].view(shape)
    st = torch.cuda.current_stream().cuda_stream
    D.disco_norm(1, 6, 35, D.DISCO_F32, x.data_ptr(), None, None, 1e-5, out.data_ptr(), None, st)
    assert (buf[:32] == 7).all() and (buf[32 + n:] == 7).all()
    want, _ = norm.layer_norm(x)
    assert torch.equal(out, want)
    # in place, and the gradient over dout
    y = x.clone()
    D.disco_norm(1, 6, 35, D.DISCO_F32, y.data_ptr(), None, None, 1e-5, y.data_ptr(), None, st)
    assert torch.equal(y, want)
    _, stats = norm.layer_norm(x)
    d = field(shape, F32, 16, cuda)
    dx, _, _ = norm.layer_norm_backward(d, x, stats)
    D.disco_norm_backward(1, 6, 35, D.DISCO_F32, d.data_ptr(), x.data_ptr(), stats.data_ptr(), None, d.data_ptr(),
                          None, None, None, 0, st)
    assert torch.equal(d, dx)


@gpu
def test_only_what_is_needed(cuda):
    x, dout = field((2, 40, 9, 10), BF16, 17, cuda), field((2, 40, 9, 10), BF16, 18, cuda)
    _, stats = norm.layer_norm(x)
    every = norm.layer_norm_backward(dout, x, stats)
    for need in [(True, False, False), (False, True, False), (False, False, True), (False, True, True), (True, True, False)]:
        got = norm.layer_norm_backward(dout, x, stats, None, *need)
        for n, a, b in zip(need, got, every):
            assert (a is None) == (not n)
            assert a is None or torch.equal(a, b)
    assert norm.layer_norm_backward(dout, x, stats, None, False, False, False) == (None, None, None)


@gpu
def test_the_same_bits_every_time(cuda):
    x, dout = field((2, 64, 91, 180), BF16, 19, cuda), field((2, 64, 91, 180), BF16, 20, cuda)
    runs = []
    for _ in range(3):
        out, stats = norm.layer_norm(x)
        runs.append((out, stats, *norm.layer_norm_backward(dout, x, stats)))
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


@gpu
@pytest.mark.parametrize("C", [12, 30, 60, 64, 100])
def test_many_tiles_in_groups_out_of_step(C, cuda):
    # groups of 1 to 8 warps, each through hundreds of tiles, beside copies that slow some SMs
    for dtype in (F32, BF16):
        x, dout = field((1, C, 361, 720), dtype, 27, cuda), field((1, C, 361, 720), dtype, 28, cuda)
        check_forward(x, None, None, 1e-5)
        check_backward(dout, x, None, 1e-5)
        want = norm.layer_norm(x)
        want += norm.layer_norm_backward(dout, x, want[1])
        side = torch.cuda.Stream()
        other = torch.zeros(1 << 24, device=cuda)
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(20):
            with torch.cuda.stream(side):
                other.add_(1)
            got = norm.layer_norm(x)
            got += norm.layer_norm_backward(dout, x, got[1])
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        torch.cuda.current_stream().wait_stream(side)


@gpu
def test_shapes_types_and_devices_are_refused(cuda):
    x = torch.zeros(2, 4, 6, 8, device=cuda)
    stats = torch.zeros(2, 2, 6, 8, device=cuda)
    for bad in (torch.zeros(5, device=cuda), torch.zeros(4, 1, device=cuda)):
        with pytest.raises(ValueError):
            norm.layer_norm(x, bad)
        with pytest.raises(ValueError):
            norm.layer_norm(x, None, bad)
    with pytest.raises(TypeError):
        norm.layer_norm(x, torch.zeros(4, device=cuda, dtype=BF16))
    with pytest.raises(TypeError):
        norm.layer_norm(x.half())
    with pytest.raises(ValueError):
        norm.layer_norm(x.transpose(2, 3))
    with pytest.raises(ValueError):
        norm.layer_norm(torch.zeros(0, 4, 6, 8, device=cuda))
    with pytest.raises(ValueError):
        norm.layer_norm(torch.zeros(4, device=cuda))
    with pytest.raises(ValueError):
        norm.layer_norm_backward(x[:, :3].contiguous(), x, stats)
    with pytest.raises(ValueError):
        norm.layer_norm_backward(x, x, stats[:, :1].contiguous())
    with pytest.raises(ValueError):
        norm.layer_norm_backward(x, x, stats.double())
    with pytest.raises(ValueError):
        norm.layer_norm_backward(x, x, stats.cpu())


@gpu
@pytest.mark.parametrize("affine,bias", [(True, True), (True, False), (False, False)])
def test_module_gradients_against_differences(affine, bias, cuda):
    """Directional derivatives of sum(out * v) by central differences in 64 bits (of the formula),
    step 1e-4 in inputs of size one: the difference is good to 1e-7 relative, the 32-bit gradient
    to 1e-5 of the sum of its terms' sizes."""
    m = norm.LayerNormS2(10, affine=affine, bias=bias, device=cuda)
    x = field((2, 10, 6, 9), F32, 21, cuda).requires_grad_()
    v = field((2, 10, 6, 9), F32, 22, cuda)
    if affine:
        with torch.no_grad():
            m.weight.add_(0.3 * torch.randn(10, device=cuda))
    m(x).backward(v)
    leaves = [x] + list(m.parameters())
    gen = torch.Generator(device=cuda).manual_seed(23)
    for leaf in leaves:
        step = torch.randn(leaf.shape, generator=gen, device=cuda).double()

        def value(h):
            vals = [t.detach().double() + (h * step if t is leaf else 0) for t in leaves]
            ga, bi = (vals[1] if affine else None), (vals[2] if bias else None)
            return float((oracle(vals[0], ga, bi, m.eps)[0] * v.double()).sum())

        diff = (value(1e-4) - value(-1e-4)) / 2e-4
        mine = leaf.grad.double() * step
        assert abs(float(mine.sum()) - diff) <= 1e-5 * float(mine.abs().sum())


@gpu
def test_module_takes_any_strides_and_frozen_parameters(cuda):
    m = norm.LayerNormS2(12, device=cuda, dtype=BF16)
    x = field((2, 12, 10, 8), BF16, 24, cuda)
    want = m(x)
    assert torch.equal(m(x.to(memory_format=torch.channels_last)), want)
    assert torch.equal(m(x.transpose(2, 3)), want.transpose(2, 3))
    x.requires_grad_()
    m.weight.requires_grad_(False)
    out = m(x)
    out.sum().expand(3).sum().backward()
    assert m.weight.grad is None and m.bias.grad is not None and x.grad is not None
    with pytest.raises(RuntimeError):
        torch.autograd.grad(torch.autograd.grad(m(x).square().sum(), x, create_graph=True)[0].sum(), x)


@gpu
@pytest.mark.parametrize("shapes", [((1, 70, 60, 72), (1, 120, 60, 72)), ((1, 9000, 5, 5), (1, 16000, 5, 5))])
def test_two_threads_at_once(shapes, cuda):
    # channels of one kernel each that differ in the shared memory they ask for
    xs = [field(s, F32, 30 + i, cuda) for i, s in enumerate(shapes)]

    def call(x):
        out, stats = norm.layer_norm(x)
        return (out, stats, *norm.layer_norm_backward(x, x, stats))

    want = [call(x) for x in xs]
    torch.cuda.synchronize()

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            got = [call(xs[i]) for _ in range(100)]
        torch.cuda.synchronize()
        return all(torch.equal(a, b) for g in got for a, b in zip(g, want[i]))

    with ThreadPoolExecutor(2) as pool:
        assert all(pool.map(work, range(2)))


@gpu
def test_another_stream_and_a_captured_call(cuda):
    x, dout = field((1, 64, 60, 72), BF16, 25, cuda), field((1, 64, 60, 72), BF16, 26, cuda)
    want = norm.layer_norm(x)
    want += norm.layer_norm_backward(dout, x, want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = norm.layer_norm(x)
        got += norm.layer_norm_backward(dout, x, got[1])
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):  # two graphs, each with scratch of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = norm.layer_norm(x)
            got += norm.layer_norm_backward(dout, x, got[1])
        graphs.append((g, got))
    x.copy_(field((1, 64, 60, 72), BF16, 27, cuda))
    want = norm.layer_norm(x)
    want += norm.layer_norm_backward(dout, x, want[1])
    for g, got in graphs:
        g.replay()
    torch.cuda.synchronize()
    for g, got in graphs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
@pytest.mark.slow
def test_offsets_beyond_32_bits(cuda):
    """A bf16 field of more than 2^32 bytes (2^31 values): the last points against the formula."""
    B, C, n = 2, 8, 2 ** 27 + 40
    x = torch.empty((B, C, n), dtype=BF16, device=cuda)
    for b in range(B):
        for c in range(C):
            x[b, c].normal_()
    out, stats = norm.layer_norm(x)
    tail = x[:, :, -4096:]
    want, mean, r, xh = oracle(tail, None, None, 1e-5)
    A = tail.double().abs().amax(1, keepdim=True) * r
    check(out[:, :, -4096:], want, 48 * U * (A + xh.abs() * (1 + A)) + half_step(want, BF16) * (1 + 2 ** -6), "out")
    dx, _, dbias = norm.layer_norm_backward(x, x, stats, None, True, False, True)
    # e = x: dx = r (xh / r + mean - mean - xh mean(x xh)), and mean(x xh) = var r
    var = 1 / r ** 2 - 1e-5
    want = xh * (1 - var * r ** 2)
    E, XH = tail.double().abs().amax(1, keepdim=True), xh.abs().amax(1, keepdim=True)
    check(dx[:, :, -4096:], want, U * r * E * (48 + 48 * XH ** 2 + 8 * XH * (A + XH)) + half_step(want, BF16) * (1 + 2 ** -6),
          "dx")
    del out, dx
    want = torch.stack([sum(x[b, c].sum(dtype=torch.float64) for b in range(B)) for c in range(C)])
    size = torch.stack([sum(x[b, c].abs().sum(dtype=torch.float64) for b in range(B)) for c in range(C)])
    # a thread adds up to 2^28 / (2 * 148 * 32 lanes) of a channel's values in a row
    check(dbias, want, (2 ** 28 / (2 * 148 * 32) + 128) * U * size + half_step(want, BF16) * (1 + 2 ** -6), "dbias")


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("C", [8, 24, 64, 100, 128, 200, 500])
def test_a_tile_is_read_before_the_next_one_lands(C, dtype, cuda):
    """Calls that start together with another stream's kernel, behind work that empties the L2 cache:
    the same bits as a call alone (a tile overwritten while it was read showed up here)."""
    n = 2 ** 25 // C // 8 * 8
    x, dout = field((1, C, n), dtype, 63, cuda), field((1, C, n), dtype, 64, cuda)
    want = norm.layer_norm(x)
    want += norm.layer_norm_backward(dout, x, want[1])
    torch.cuda.synchronize()
    for _ in range(60):
        torch.randn(2 ** 25, device=cuda).mul_(2)
        side = torch.cuda.Stream()
        other = torch.zeros(1 << 24, device=cuda)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other.add_(1)
        got = norm.layer_norm(x)
        got += norm.layer_norm_backward(dout, x, got[1])
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------ every form of the kernels
#
# Planes of at least 64 points with few enough channels pass through tiles in shared memory, in boxes
# where rows start on 16 bytes and copied by their own lanes where they do not; the others stay in
# registers.  These shapes reach each: whole and partial last tiles, several tiles a CTA, one group of
# warps and many, rows of any phase in 16 bytes.
FORMS = [(1, 6, 5, 7), (3, 5, 1, 1), (1, 24, 3, 5), (2, 100, 5, 9), (1, 600, 8, 8), (2, 1500, 3, 5),
         (1, 1, 8, 8), (2, 5, 9, 8), (1, 24, 16, 16), (2, 24, 13, 17), (1, 48, 181, 360), (2, 64, 91, 181), (1, 100, 61, 121),
         (1, 130, 40, 72), (1, 300, 33, 40), (1, 513, 12, 20), (2, 1000, 9, 11)]


def far_adds(x):
    # additions in a row over deviations from one channel, as in `adds`
    return adds(x) + 8


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("value", [3.25, 1013.25, -9999.123, 300.1])
@pytest.mark.parametrize("shape", FORMS)
def test_equal_channels_leave_the_bias(shape, value, dtype, cuda):
    """Points whose channels are all equal (a fill value, say): their mean is the value and xh is 0, to
    the bit, however large 1 / deviation = 1 / sqrt(eps) is; dx = r (e - mean e)."""
    C = shape[1]
    x = torch.full(shape, value, device=cuda).to(dtype)
    gen = torch.Generator(device=cuda).manual_seed(60)
    gain, bias = (torch.randn(C, generator=gen, device=cuda).to(dtype) for _ in range(2))
    out, stats = norm.layer_norm(x, gain, bias, 1e-5)
    assert torch.equal(stats[0].unsqueeze(1), x[:, :1].float())
    assert torch.equal(out, bias.view((1, -1) + (1,) * (x.dim() - 2)).expand_as(x))
    assert torch.allclose(stats[1], torch.full_like(stats[1], 1e-5 ** -0.5), rtol=2 ** -22)
    dout = field(shape, dtype, 61, cuda)
    dx, dgain, _ = norm.layer_norm_backward(dout, x, stats, gain)
    assert (dgain == 0).all()
    e = dout.double() * col(gain, x)
    r = stats[1].double().unsqueeze(1)
    want = r * (e - e.mean(1, keepdim=True))
    check(dx, want, (adds(x) + 8) * U * r * e.abs().amax(1, keepdim=True) + half_step(want, dtype) * (1 + 2 ** -6) + 1e-37, "dx")


@gpu
@pytest.mark.parametrize("offset", [30.0, 1000.0, -9999.123])
@pytest.mark.parametrize("shape", FORMS)
def test_far_from_zero_only_the_mean_is_rounded(shape, offset, cuda):
    """With k the first channel of a row of lanes and D = max_c |x - k|: the row's mean is k plus the mean
    of the differences, rounded once to u |mean| besides n u D for the sums; the mean of the point is
    the first row's plus the mean of the rows' differences from it, rounded once more (in the register
    form up to 4 rows of a warp join in two steps before that): off by j u |mean| + n u D, j = 2 for
    tiles and 4 for registers.  x - mean then is off by u |x - mean|, so that
    |d xh| <= r (j u |mean| + n u D) + (n + 8) u |xh| (1 + r D)."""
    x = (field(shape, F32, 62, cuda, offset=0.0) + offset).to(F32)
    out, stats = norm.layer_norm(x)
    want, mean, r, xh = oracle(x, None, None, 1e-5)
    xd, n = x.double(), far_adds(x)
    D = (xd.amax(1, keepdim=True) - xd.amin(1, keepdim=True))
    j = 2 if x[0, 0].numel() >= 64 and x.shape[1] <= 1024 else 4
    off = j * U * mean.abs() + n * U * D
    check(stats[0].unsqueeze(1), mean, off, "mean")
    tol = r * off + (n + 8) * U * xh.abs() * (1 + r * D) + 1e-37
    check(out, want, tol, "out")
    # the backward pass's xh, from the statistics rounded to 32 bits
    dout = torch.zeros_like(x)
    at = [0] * (x.dim() - 2)
    dout[(0, slice(None), *at)] = 1.0
    _, dgain, _ = norm.layer_norm_backward(dout, x, stats, None, False, True, False)
    check(dgain, want[(0, slice(None), *at)], tol[(0, slice(None), *at)] + U * xh[(0, slice(None), *at)].abs(), "xh")


@gpu
@pytest.mark.parametrize("shape", [(1, 64, 721, 1440), (1, 64, 721, 1441), (1, 8, 721, 1440), (2, 256, 181, 360), (1, 12, 721, 1441),
                                   (100000, 16, 7), (4000, 520, 63), (3000, 1500, 9)])
def test_parameter_sums_over_many_points(shape, cuda):
    """The same value at every point, so that roundings do not cancel: xh = 1/3 (mean 0, r 1) and dout
    = 1/3.  In 32 bits are added: 4 points of a tile at most by a thread, 8 tiles at most, and the
    lanes of a channel (32, of which 3 to 5 additions are one behind the other; 8 lanes where a thread
    adds 4 points); all that follows is in 64 bits.  With the product's rounding and the result's
    those are 1 + 3 + 8 + 3 + 1 or 1 + 1 + 8 + 5 + 1, at most 16, each u relative to a sum of equal
    signs."""
    third = torch.tensor(1 / 3, device=cuda)
    x = third.expand(shape).contiguous()
    stats = torch.zeros((2, shape[0], *shape[2:]), device=cuda)
    stats[1] = 1.0
    _, dgain, dbias = norm.layer_norm_backward(x, x, stats, None, False, True, True)
    n, t = shape[0] * math.prod(shape[2:]), third.double()
    for got, want, what in ((dgain, n * t * t, "dgain"), (dbias, n * t, "dbias")):
        check(got, want.expand(shape[1]), 16 * U * want, what)


@gpu
@pytest.mark.parametrize("which", [(1, 1, 1), (0, 1, 0), (0, 0, 1), (1, 0, 0)])
def test_the_function_has_the_module_s_gradients(which, cuda):
    m = norm.LayerNormS2(10, device=cuda)
    with torch.no_grad():
        m.weight.add_(0.3 * torch.randn(10, device=cuda))
    x, v = field((2, 10, 6, 9), F32, 65, cuda), field((2, 10, 6, 9), F32, 66, cuda)
    a = x.clone().requires_grad_()
    m(a).backward(v)
    want = [a.grad, m.weight.grad, m.bias.grad]
    leaves = [t.detach().clone().requires_grad_(bool(w)) for t, w in zip((x, m.weight, m.bias), which)]
    out, stats = norm.layer_norm(*leaves, eps=m.eps)
    assert out.requires_grad and not stats.requires_grad
    out.backward(v)
    for t, w, g in zip(leaves, which, want):
        assert (t.grad is None) != bool(w)
        assert not w or torch.equal(t.grad, g)
    with torch.no_grad():
        assert not norm.layer_norm(*leaves, eps=m.eps)[0].requires_grad
    assert not norm.layer_norm(x)[0].requires_grad
    with pytest.raises(ValueError):
        norm.layer_norm(leaves[0].transpose(2, 3).requires_grad_() if not which[0] else leaves[0].transpose(2, 3), *leaves[1:])
    with pytest.raises(RuntimeError):
        torch.autograd.grad(torch.autograd.grad(norm.layer_norm(a)[0].square().sum(), a, create_graph=True)[0].sum(), a)


LONG = [s for s in FORMS if math.prod(s[2:]) >= 64]


@gpu
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", LONG)
def test_bad_points_of_long_planes_stay_their_own(shape, dtype, bad, cuda):
    x, dout = field(shape, dtype, 67, cuda), field(shape, dtype, 68, cuda)
    B, C, n = shape[0], shape[1], math.prod(shape[2:])
    y, e = x.clone().view(B, C, n), dout.clone().view(B, C, n)
    hit = torch.zeros(B, 1, n, dtype=torch.bool, device=cuda)
    for b, c, p in [(0, 0, 5), (B - 1, C - 1, n - 1), (B - 1, C // 2, n // 2 + 1)]:
        y[b, c, p] = bad
        e[b, C - 1 - c, (p + 17) % n] = bad
        hit[b, 0, p] = hit[b, 0, (p + 17) % n] = True
    hit = hit.expand(B, C, n).reshape(shape)
    y, e = y.view(shape), e.view(shape)
    a, sa = norm.layer_norm(x)
    b, sb = norm.layer_norm(y)
    assert torch.equal(a[~hit], b[~hit])
    assert torch.isnan(b.view(B, C, n)[B - 1, :, n - 1]).any()
    da = norm.layer_norm_backward(dout, x, sa)[0]
    db = norm.layer_norm_backward(e, y, sb)[0]
    assert torch.equal(da[~hit], db[~hit])


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shift", [0, 1, 2, 3, 4, 8])
@pytest.mark.parametrize("shape", LONG)
def test_any_base_guards_and_overlap(shape, shift, dtype, cuda):
    """Tensors at any element of an allocation, results between guards, workspace at its exact size;
    then in place, the input's gradient over dout, and over x."""
    B, C, n = shape[0], shape[1], math.prod(shape[2:])
    N, code, es = B * C * n, D.DISCO_F32 if dtype == F32 else D.DISCO_BF16, dtype.itemsize
    st = torch.cuda.current_stream().cuda_stream
    bufs = []

    def place(count, k, t=dtype, values=None):
        buf = torch.full((count + 64,), 7, dtype=t, device=cuda)
        v = buf[16 + k:16 + k + count]
        if values is not None:
            v.copy_(values.reshape(-1))
        bufs.append((buf, 16 + k, count))
        return v

    def guarded():
        return all((b[:o] == 7).all() and (b[o + c:] == 7).all() for b, o, c in bufs)

    x, dout = field(shape, dtype, 69, cuda), field(shape, dtype, 70, cuda)
    gain, bias = field((1, C), dtype, 71, cuda)[0], field((1, C), dtype, 72, cuda)[0]
    xs, ds = place(N, shift, values=x), place(N, (shift + 3) % 8, values=dout)
    ga, bi = place(C, 1, values=gain), place(C, 2, values=bias)
    out, dx, dg, db = place(N, (shift + 1) % 8), place(N, (shift + 2) % 8), place(C, 3), place(C, 1)
    stats = place(2 * B * n, shift, F32)
    nb = D.disco_norm_workspace_size(B, C, n, code)
    ws = place(nb // 4, 1, F32)
    D.disco_norm(B, C, n, code, xs.data_ptr(), ga.data_ptr(), bi.data_ptr(), 1e-5, out.data_ptr(), stats.data_ptr(), st)
    D.disco_norm_backward(B, C, n, code, ds.data_ptr(), xs.data_ptr(), stats.data_ptr(), ga.data_ptr(), dx.data_ptr(),
                          dg.data_ptr(), db.data_ptr(), ws.data_ptr(), nb, st)
    assert guarded()
    check_forward_at(out.view(shape), stats.view(2, B, *shape[2:]), x, gain, bias)
    e = dout.double() * col(gain, x)
    _, mean, r, xh = oracle(x, None, None, 1e-5)
    want = r * (e - e.mean(1, keepdim=True) - xh * (e * xh).mean(1, keepdim=True))
    A, XH, E = (t.amax(1, keepdim=True) for t in (x.double().abs() * r, xh.abs(), e.abs()))
    # the statistics are the forward pass's own here: xh off by up to (n + 8) u (A + XH (1 + A))
    k = adds(x) + 8
    tol = U * r * E * (k * (1 + XH ** 2) + 2 * k * (1 + XH) * (A + XH * (1 + A))) + half_step(want, dtype) * (1 + 2 ** -6) + 1e-37
    check(dx.view(shape), want, tol, "dx")
    keep = dx.clone()
    for over in (ds, xs):
        saved = over.clone()
        D.disco_norm_backward(B, C, n, code, ds.data_ptr(), xs.data_ptr(), stats.data_ptr(), ga.data_ptr(),
                              over.data_ptr(), None, None, None, 0, st)
        # another phase in 16 bytes may take another form, whose sums differ in their order
        check(over.view(shape), keep.view(shape).double(), 2 * tol, "dx over an input")
        over.copy_(saved)
    D.disco_norm(B, C, n, code, xs.data_ptr(), ga.data_ptr(), bi.data_ptr(), 1e-5, xs.data_ptr(), None, st)
    check_forward_at(xs.view(shape), None, x, gain, bias)
    assert guarded()


def check_forward_at(out, stats, x, gain, bias):
    want, mean, r, xh = oracle(x, gain, bias, 1e-5)
    A, n = x.double().abs().amax(1, keepdim=True) * r, adds(x)
    check(out, want, (n + 8) * U * (A + xh.abs() * (1 + A)) * col(gain, x).abs() + U * col(bias, x).abs()
          + half_step(want, x.dtype) * (1 + 2 ** -6) + 1e-37, "out")
    if stats is not None:
        check(stats[0].unsqueeze(1), mean, (n + 1) * U * x.double().abs().amax(1, keepdim=True) + 1e-37, "mean")
        check(stats[1].unsqueeze(1), r, ((n + 1) * U * A + (n + 1) * U) * r, "1 / deviation")


@gpu
@pytest.mark.parametrize("size", [3e18, 1e20, 1e33])
@pytest.mark.parametrize("shape", [s for s in FORMS if s[1] > 1])
def test_squares_beyond_fp32_leave_the_bias(shape, size, cuda):
    """Deviations whose squares overflow: the variance is infinite, r is 0 and out the bias in every
    form, as 1 / sqrt(inf) has it; at 3e18 squares and the sum over a few channels still fit.  (Above
    3e38 / C the sum of the channels itself may overflow.)"""
    x = field(shape, F32, 73, cuda) * size
    bias = field((1, shape[1]), F32, 74, cuda)[0]
    out, stats = norm.layer_norm(x, None, bias)
    over = ((x.double() - x.double().mean(1, keepdim=True)) ** 2).sum(1) > 1e39
    assert not stats.isnan().any() and not out.isnan().any()
    assert (stats[1][over] == 0).all()
    hit = over.unsqueeze(1).expand_as(out)
    assert torch.equal(out[hit], col(bias, x).float().expand_as(out)[hit])
    if size == 3e18 and shape[1] < 7:
        check_forward(x, None, bias, 1e-5)
    dx = norm.layer_norm_backward(field(shape, F32, 75, cuda), x, stats)[0]
    assert (dx[hit] == 0).all()
