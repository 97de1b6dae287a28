"""The measured operators of training a block of DISCO layers: the layer norm of a field over its channels,
forward and backward, and the Muon update of the layers' weights (the orthogonalised update alone, and the whole
step with momentum and weight decay).

Fields are (B, C, nlat, nlon), as the convolution takes and gives them; the norm is over the C channels of every
grid point.  Weights are (C_out, C_in / groups, K); each group's rows are one matrix of C_out / groups rows and
C_in / groups * K columns, which is what the update orthogonalises.

`run` computes an operator in its plain form (elementary torch operations in 32 bits, rounded once at the end)
while `own` is false, and by the framework's calls while it is true.
"""

import math

import torch

own = False

STEPS = 5
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
NS_EPS = 1e-7
NORM_EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "bf16": 2}


def listed():
    return [
        # the norm after the smallest layer of the workloads: latency alone
        dict(name="norm tiny f32", op="norm", dtype="f32", B=1, C=4, nlat=17, nlon=32),
        # an odd regional grid and channel count in fp32: no row of a channel starts on a 16-byte boundary
        dict(name="norm ragged f32", op="norm", dtype="f32", B=3, C=50, nlat=61, nlon=121),
        # the norm of the weather layer's output, 64 channels of a 0.25 degree field
        dict(name="norm weather bf16", op="norm", dtype="bf16", B=1, C=64, nlat=721, nlon=1440),
        # the backward pass after the mid-size fp32 layer, batch 4
        dict(name="grad mid f32", op="norm_grad", dtype="f32", B=4, C=32, nlat=91, nlon=180),
        # odd channels on an odd one-degree grid in bf16: rows start at any even byte
        dict(name="grad odd bf16", op="norm_grad", dtype="bf16", B=1, C=77, nlat=181, nlon=361),
        # the backward pass after the wide grouped layer, the largest field of the workloads
        dict(name="grad grouped bf16", op="norm_grad", dtype="bf16", B=2, C=256, nlat=361, nlon=720),
        # the update of the smallest layer's weight: latency alone
        dict(name="orth tiny f32", op="orth", dtype="f32", layers=1, C_out=4, C_in=4, K=3, groups=1),
        # eight downsampling layers' weights in one call
        dict(name="orth downsample x8 bf16", op="orth", dtype="bf16", layers=8, C_out=128, C_in=64, K=9, groups=1),
        # one very wide layer without groups, where the products dominate
        dict(name="orth wide f32", op="orth", dtype="f32", layers=1, C_out=1024, C_in=1024, K=9, groups=1),
        # the whole step of the weather layer's weight
        dict(name="muon weather f32", op="muon", dtype="f32", layers=1, C_out=64, C_in=64, K=3, groups=1),
        # twelve grouped layers' weights in one step, 48 matrices
        dict(name="muon grouped x12 bf16", op="muon", dtype="bf16", layers=12, C_out=256, C_in=256, K=9, groups=4),
        # four wide layers in one step
        dict(name="muon 512 x4 bf16", op="muon", dtype="bf16", layers=4, C_out=512, C_in=512, K=9, groups=1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "orth", "muon"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("norm", "norm_grad"):
        # from four channels on: over one or two the norm leaves nothing of the field but signs, and its gradient cancels
        B, C = rng.randint(1, 4), _log_int(rng, 4, 512)
        nlat = _log_int(rng, 5, 721)
        nlon = _log_int(rng, 8, 1440)
        while B * C * nlat * nlon > 60_000_000:  # at most the weather layer's field, about
            nlat = max(1, nlat // 2)
        return dict(op=op, dtype=dtype, B=B, C=C, nlat=nlat, nlon=nlon)
    groups = rng.choice([1, 1, 1, 2, 4])
    C_out, C_in = groups * _log_int(rng, 1, 640), groups * _log_int(rng, 1, 640)
    K = rng.choice([1, 3, 5, 7, 9])
    layers = _log_int(rng, 1, 12)
    case = dict(op=op, dtype=dtype, layers=layers, C_out=C_out, C_in=C_in, K=K, groups=groups)
    while work(case)["flops"] > 1e11:
        case["layers"] = 1 if case["layers"] < 3 else case["layers"] // 2
        case["C_in"] = groups * max(1, case["C_in"] // groups // 2)
    return case


def _matrix(case):
    return case["C_out"] // case["groups"], case["C_in"] // case["groups"] * case["K"]


def work(case):
    es = SIZES[case["dtype"]]
    if case["op"] in ("norm", "norm_grad"):
        pts = case["B"] * case["nlat"] * case["nlon"]
        n = pts * case["C"]
        if case["op"] == "norm":  # x in, out and two statistics a point out
            return {"bytes": 2 * n * es + 8 * pts + 2 * case["C"] * es, "flops": 8 * n}
        return {"bytes": 3 * n * es + 8 * pts + 3 * case["C"] * es, "flops": 14 * n}
    M, N = _matrix(case)
    mats = case["layers"] * case["groups"]
    r, l = min(M, N), max(M, N)
    # a symmetric product needs one half of its entries: X X^T and A A
    flops = mats * STEPS * (3 * r * r * l + r * r * r)
    n = mats * M * N
    # the update in and out; the step reads w, g, m and writes w, m (momentum in 32 bits)
    return {"bytes": 2 * n * es if case["op"] == "orth" else n * (3 * es + 8), "flops": flops}


def _updates(gen, case, scale):
    """Weight gradients as training gives them: a few strong directions of falling size over small noise."""
    M, N = _matrix(case)
    mats = case["layers"] * case["groups"]
    r = min(8, M, N)
    u = torch.randn((mats, M, r), generator=gen, device="cuda")
    v = torch.randn((mats, r, N), generator=gen, device="cuda")
    fall = 0.6 ** torch.arange(r, device="cuda", dtype=torch.float32)
    g = (u * fall) @ v + 0.5 * torch.randn((mats, M, N), generator=gen, device="cuda")
    return (g * scale).reshape(case["layers"], case["C_out"], case["C_in"] // case["groups"], case["K"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    if case["op"] in ("norm", "norm_grad"):
        B, C, shape = case["B"], case["C"], (case["B"], case["C"], case["nlat"], case["nlon"])
        mu = 0.5 * torch.randn((B, C, 1, 1), generator=gen, device="cuda")
        sd = 0.5 + 1.5 * torch.rand((B, C, 1, 1), generator=gen, device="cuda")
        x = (mu + sd * torch.randn(shape, generator=gen, device="cuda")).to(dt)
        state = dict(case=case, x=x, gain=(1 + 0.2 * torch.randn(C, generator=gen, device="cuda")).to(dt))
        if case["op"] == "norm":
            state["bias"] = (0.1 * torch.randn(C, generator=gen, device="cuda")).to(dt)
        else:
            state["dout"] = torch.randn(shape, generator=gen, device="cuda").to(dt)
            # what the forward pass kept for this one: mean and 1 / deviation of every point
            xd = x.double()
            var, mean = torch.var_mean(xd, dim=1, correction=0)
            state["stats"] = torch.stack([mean, (var + NORM_EPS).rsqrt()]).float()
        return state
    state = dict(case=case, groups=case["groups"])
    state["g"] = [t.clone() for t in _updates(gen, case, 1e-3).to(dt)]
    if case["op"] == "muon":
        state["m"] = [t.clone() for t in _updates(gen, case, 5e-3)]
        M, N = _matrix(case)
        w = torch.randn((case["layers"], case["C_out"], N // case["K"], case["K"]), generator=gen, device="cuda")
        state["w"] = [t.clone() for t in (w / math.sqrt(N)).to(dt)]
    return state


LR, MOMENTUM, DECAY = 0.02, 0.95, 0.01


def _newton_schulz(u, M, N):
    """u (matrices, M, N) in 32 bits: the odd polynomial a X + b X X^T X + c (X X^T)^2 X, STEPS times, from
    X = u / (|u|_F + eps); on the transposed matrix where that has fewer rows."""
    a, b, c = COEFFICIENTS
    x = u.transpose(1, 2) if M > N else u
    x = x / ((x * x).sum(dim=(1, 2), keepdim=True).sqrt() + NS_EPS)
    for _ in range(STEPS):
        g = x @ x.transpose(1, 2)
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.transpose(1, 2) if M > N else x


def run(state):
    case = state["case"]
    if own:
        return _run_own(state)
    if case["op"] == "norm":
        x, dt = state["x"].float(), state["x"].dtype
        mean = x.mean(dim=1, keepdim=True)
        d = x - mean
        rstd = 1 / ((d * d).mean(dim=1, keepdim=True) + NORM_EPS).sqrt()
        out = d * rstd * state["gain"].float().view(1, -1, 1, 1) + state["bias"].float().view(1, -1, 1, 1)
        return out.to(dt), torch.stack([mean[:, 0], rstd[:, 0]])
    if case["op"] == "norm_grad":
        dt = state["x"].dtype
        mean, rstd = state["stats"][0].unsqueeze(1), state["stats"][1].unsqueeze(1)
        xh = (state["x"].float() - mean) * rstd
        dy = state["dout"].float()
        dgain = (dy * xh).sum(dim=(0, 2, 3), dtype=torch.float64)
        dbias = dy.sum(dim=(0, 2, 3), dtype=torch.float64)
        e = dy * state["gain"].float().view(1, -1, 1, 1)
        dx = rstd * (e - e.mean(dim=1, keepdim=True) - xh * (e * xh).mean(dim=1, keepdim=True))
        return dx.to(dt), dgain.to(dt), dbias.to(dt)
    M, N = _matrix(case)
    dt = state["g"][0].dtype
    g = torch.stack(state["g"]).float()
    if case["op"] == "orth":
        o = _newton_schulz(g.reshape(-1, M, N), M, N)
        return list(o.reshape(g.shape).to(dt).unbind())
    m = MOMENTUM * torch.stack(state["m"]) + g
    u = g + MOMENTUM * m
    o = _newton_schulz(u.reshape(-1, M, N), M, N).reshape(g.shape)
    w = (1 - LR * DECAY) * torch.stack(state["w"]).float() - LR * math.sqrt(max(1.0, M / N)) * o
    return list(w.to(dt).unbind()), list(m.unbind())


def _run_own(state):
    from spherical_disco_convolution_b200 import muon, norm

    case = state["case"]
    if case["op"] == "norm":
        return norm.layer_norm(state["x"], state["gain"], state["bias"], eps=NORM_EPS)
    if case["op"] == "norm_grad":
        return norm.layer_norm_backward(state["dout"], state["x"], state["stats"], state["gain"])
    if case["op"] == "orth":
        return muon.orthogonalize(state["g"], groups=case["groups"], steps=STEPS, coefficients=COEFFICIENTS, eps=NS_EPS)
    return muon.muon_update(state["w"], state["g"], state["m"], lr=LR, momentum=MOMENTUM, nesterov=True,
                            weight_decay=DECAY, groups=case["groups"], steps=STEPS, coefficients=COEFFICIENTS,
                            eps=NS_EPS)


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "norm":
        x = state["x"].double()
        s1 = x.sum(dim=1) / case["C"]
        x -= s1.unsqueeze(1)
        s2 = torch.linalg.vector_norm(x, dim=1) ** 2 / case["C"]
        rstd = (s2 + NORM_EPS) ** -0.5
        x *= rstd.unsqueeze(1)
        x *= state["gain"].double()[None, :, None, None]
        x += state["bias"].double()[None, :, None, None]
        return x, torch.stack([s1, rstd])
    if case["op"] == "norm_grad":
        x, dy = state["x"].double(), state["dout"].double()
        x -= (x.sum(dim=1) / case["C"]).unsqueeze(1)
        rstd = (torch.linalg.vector_norm(x, dim=1) ** 2 / case["C"] + NORM_EPS) ** -0.5
        x *= rstd.unsqueeze(1)
        dgain, dbias = torch.einsum("bcij,bcij->c", dy, x), torch.einsum("bcij->c", dy)
        dy *= state["gain"].double()[None, :, None, None]
        along = torch.einsum("bcij,bcij->bij", dy, x) / case["C"]
        dy -= (dy.sum(dim=1) / case["C"]).unsqueeze(1)
        dy -= x * along.unsqueeze(1)
        return dy * rstd.unsqueeze(1), dgain, dbias
    M, N = _matrix(case)
    g = torch.stack(state["g"]).double()
    m = None
    if case["op"] == "muon":
        m = MOMENTUM * torch.stack(state["m"]).double() + g
        g = g + MOMENTUM * m
    # The polynomial acts on each singular value: with the eigenvalues t and vectors U of X X^T (or X^T X, the
    # smaller), the result is U q(t) U^T X, q the product over the steps of a + b t + c t^2 with t <- t (a + b t + c t^2)^2.
    x = g.reshape(-1, M, N)
    x = x / (torch.linalg.matrix_norm(x)[:, None, None] + NS_EPS)
    t, U = torch.linalg.eigh(x.mT @ x if M > N else x @ x.mT)
    t, q = t.clamp(min=0), torch.ones_like(t)
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        p = a + t * (b + c * t)
        q, t = q * p, t * p * p
    Q = (U * q.unsqueeze(1)) @ U.mT
    o = (x @ Q if M > N else Q @ x).reshape(g.shape)
    if case["op"] == "orth":
        return list(o.unbind())
    w = (1 - LR * DECAY) * torch.stack(state["w"]).double() - LR * max(1.0, M / N) ** 0.5 * o
    return list(w.unbind()), list(m.unbind())
