"""ix_layer_norm and its gradient against the formulas in 64 bits.

Tolerances, with u = 2^-24 (half a step of f32): a thread adds at most 32 values,
and the threads' sums meet in at most 10 steps, so a row's sum is at most 42u of
the sum of magnitudes off; with the products and quotients around it, 64u.  Then
 mean: 64u mean|x|;  rstd: 64u relative, and what the mean's error adds to the
 variance, (64u mean|x| rstd)^2;
 out: eps / 2 of it for its one rounding, 64u rstd mean|x| |gamma| for the mean,
 128u (|xhat gamma| + |beta|) for the rest;
 dx: eps / 2, and 128u rstd (|h| + mean|h| + |xhat| mean|h xhat|);
 dgamma, dbeta: (rows / parts + 64)u of the sum of the magnitudes, where at most
 `rows` values meet in one thread: (rows + 64)u, for few rows.
"""
import pytest
import torch

from _helpers import require_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float16, torch.float32]
COLS = [1, 2, 7, 32, 33, 100, 128, 129, 256, 500, 512, 513, 1000, 1024, 1025, 2048, 2050, 4096, 5001, 8192, 8200, 8201,
        16384, 20001, 32760, 32768]


@pytest.fixture(scope="module")
def dsix():
    require_gpu()
    import deepseek_v3_sparse_gb300 as m
    m.load_prep()
    m.ix_prep_device_status()
    return m


def half(t):
    return torch.finfo(t).eps / 2


def within(got, want, tol, what):
    d = (got.double() - want).abs()
    tiny = torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps
    assert bool((d <= tol + tiny).all()), f"{what}: off by {float((d - tol).max())} more than allowed"


def make(rows, cols, dtype, layout, seed, scale=1.5, shift=0.25):
    g = torch.Generator(device="cuda").manual_seed(seed)
    pad = {"plain": 0, "padded": 16, "odd": 3}[layout]
    x = (torch.randn(rows, cols + pad, generator=g, device="cuda") * scale + shift).to(dtype)
    return x[:, pad // 2:pad // 2 + cols] if layout == "odd" else x[:, :cols]


def weights(cols, dtype, kind, seed):
    g = torch.Generator(device="cuda").manual_seed(seed + 1000)
    if kind == "none":
        return None, None
    w = dtype if kind == "typed" else torch.float32
    return (1 + 0.3 * torch.randn(cols, generator=g, device="cuda")).to(w), \
        (0.2 * torch.randn(cols, generator=g, device="cuda")).to(w)


def forward_reference(x, gamma, beta, eps):
    x = x.double()
    g = torch.ones(x.shape[1], dtype=torch.float64, device="cuda") if gamma is None else gamma.double()
    b = torch.zeros(x.shape[1], dtype=torch.float64, device="cuda") if beta is None else beta.double()
    mean = x.mean(1)
    var = ((x - mean[:, None]) ** 2).mean(1)
    rstd = 1 / torch.sqrt(var + eps)
    xhat = (x - mean[:, None]) * rstd[:, None]
    return xhat * g + b, mean, rstd, xhat, g, b


def check_forward(dsix, x, gamma, beta, eps, out):
    rows = x.shape[0]
    mean, rstd = torch.full((rows,), 9.0, device="cuda"), torch.full((rows,), 9.0, device="cuda")
    kept = x.clone()
    dsix.ix_layer_norm(x, gamma, beta, eps, out, mean, rstd)
    y, m, r, xhat, g, b = forward_reference(kept, gamma, beta, eps)
    size = kept.double().abs().mean(1)
    within(mean, m, 64 * U * size, "mean")
    off = 64 * U * size * r
    within(rstd, r, r * (64 * U + off * off), "rstd")
    within(out, y, half(out.dtype) * y.abs() + (off * (1 + off))[:, None] * g.abs() +
           128 * U * ((xhat * g).abs() + b.abs()), "out")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("layout", ["plain", "padded", "odd"])
def test_forward(dsix, dtype, layout):
    for n, cols in enumerate(COLS):
        for rows in (1, 5, 37):
            x = make(rows, cols, dtype, layout, n)
            gamma, beta = weights(cols, dtype, ("f32", "typed", "none")[n % 3], n)
            check_forward(dsix, x, gamma, beta, 1e-5, torch.empty_like(x))
    assert dsix.ix_prep_device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
def test_forward_many_rows_in_place(dsix, dtype):
    for rows, cols in ((20011, 128), (3001, 513), (700, 4096)):
        x = make(rows, cols, dtype, "plain", rows)
        gamma, beta = weights(cols, dtype, "f32", 5)
        check_forward(dsix, x, gamma, beta, 1e-6, x)


def test_forward_without_cancellation(dsix):
    """A mean a thousand times the spread: the squares of the centred values keep
    the variance, which the difference of mean square and squared mean loses."""
    x = make(9, 1000, torch.float32, "plain", 3, scale=1.0, shift=1000.0)
    check_forward(dsix, x, *weights(1000, torch.float32, "f32", 1), 0.0, torch.empty_like(x))


def test_forward_constant_rows_and_special_values(dsix):
    x = torch.zeros(4, 128, device="cuda")
    x[1] = 3.0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    out = torch.empty_like(x)
    dsix.ix_layer_norm(x, None, None, 1e-6, out)
    assert bool((out[:2] == 0).all()) and bool(torch.isnan(out[2:]).all())


def check_backward(dsix, rows, cols, dtype, layout, kind, seed, in_place=False):
    x, dy = make(rows, cols, dtype, layout, seed), make(rows, cols, dtype, layout, seed + 50, 0.5, 0.05)
    gamma, _ = weights(cols, dtype, kind, seed)
    _, mean, rstd, _, g, _ = forward_reference(x, gamma, None, 1e-5)
    mean, rstd = mean.float(), rstd.float()
    d64 = dy.double()
    dx = dy if in_place else torch.empty_like(dy)
    dgamma, dbeta = torch.full((cols,), 9.0, device="cuda"), torch.full((cols,), 9.0, device="cuda")
    work = torch.empty(max(1, dsix.ix_layer_norm_bwd_workspace_size(rows, cols)), dtype=torch.uint8, device="cuda")
    work.fill_(255)  # NaN bits: nothing of the workspace's contents counts
    dsix.ix_layer_norm_bwd(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, work)
    xhat = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    h = d64 * g
    mh, mhx = h.mean(1, keepdim=True), (h * xhat).mean(1, keepdim=True)
    r = rstd.double()[:, None]
    want = r * (h - mh - xhat * mhx)
    within(dx, want, half(dtype) * want.abs() + 128 * U * r * (
        h.abs() + h.abs().mean(1, keepdim=True) + xhat.abs() * (h * xhat).abs().mean(1, keepdim=True)), "dx")
    terms = min(rows, 64 + rows // 64) + 64
    within(dgamma, (d64 * xhat).sum(0), terms * U * (d64 * xhat).abs().sum(0), "dgamma")
    within(dbeta, d64.sum(0), terms * U * d64.abs().sum(0), "dbeta")
    # the same call gives the same bits, and without the weights' gradients the same dx
    if not in_place:
        a, b, again = torch.empty_like(dgamma), torch.empty_like(dbeta), torch.empty_like(dx)
        dsix.ix_layer_norm_bwd(dy, x, gamma, mean, rstd, again, a, b, work)
        assert torch.equal(a, dgamma) and torch.equal(b, dbeta) and torch.equal(again, dx)
        again.zero_()
        dsix.ix_layer_norm_bwd(dy, x, gamma, mean, rstd, again)
        assert torch.equal(again, dx)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("layout", ["plain", "padded", "odd"])
def test_backward(dsix, dtype, layout):
    for n, cols in enumerate(COLS):
        for rows in (1, 3, 41):
            check_backward(dsix, rows, cols, dtype, layout, ("f32", "typed", "none")[n % 3], n)
    assert dsix.ix_prep_device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(20011, 128), (5003, 96), (3001, 513), (1500, 4096), (700, 20001)])
def test_backward_many_rows(dsix, dtype, rows, cols):
    check_backward(dsix, rows, cols, dtype, "plain", "f32", rows)
    check_backward(dsix, rows, cols, dtype, "plain", "typed", rows, in_place=True)


def test_backward_of_no_rows_is_zero(dsix):
    x = torch.empty(0, 100, device="cuda")
    e = torch.empty(0, device="cuda")
    dgamma, dbeta = torch.ones(100, device="cuda"), torch.ones(100, device="cuda")
    dsix.ix_layer_norm_bwd(x, x, None, e, e, torch.empty_like(x), dgamma, dbeta)
    assert not dgamma.any() and not dbeta.any()
    dsix.ix_layer_norm(x, None, None, 1e-5, torch.empty_like(x))


def test_backward_needs_its_workspace(dsix):
    x = torch.ones(4, 128, device="cuda")
    m = torch.zeros(4, device="cuda")
    d = torch.empty(128, device="cuda")
    with pytest.raises(dsix.DsixError, match="WORKSPACE"):
        dsix.ix_layer_norm_bwd(x, x, None, m, m, torch.empty_like(x), d, d.clone(), torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_gradients_against_differences(dsix):
    """Central differences of sum(w * layer_norm(x)) in 64 bits along random
    directions; their truncation is of the order h^2 = 1e-6 of the third
    derivative's size, here below 1e-4 of the gradient's norm."""
    g = torch.Generator(device="cuda").manual_seed(7)
    rows, cols, eps = 6, 200, 1e-5
    x, w = (torch.randn(rows, cols, generator=g, device="cuda") for _ in range(2))
    gamma, beta = weights(cols, torch.float32, "f32", 3)
    out, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dsix.ix_layer_norm(x, gamma, beta, eps, out, mean, rstd)
    dx, dgamma, dbeta = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(beta)
    work = torch.empty(dsix.ix_layer_norm_bwd_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")
    dsix.ix_layer_norm_bwd(w, x, gamma, mean, rstd, dx, dgamma, dbeta, work)

    def f(x, gamma, beta):
        return (w.double() * forward_reference(x, gamma, beta, eps)[0]).sum()

    at = [t.double() for t in (x, gamma, beta)]
    for i, grad in enumerate((dx, dgamma, dbeta)):
        for _ in range(4):
            v = torch.randn(at[i].shape, generator=g, device="cuda", dtype=torch.float64)
            up, down = list(at), list(at)
            up[i], down[i] = at[i] + 1e-3 * v, at[i] - 1e-3 * v
            quotient = (f(*up) - f(*down)) / 2e-3
            got = (grad.double() * v).sum()
            assert abs(float(got - quotient)) <= 1e-4 * float(grad.double().norm() * v.norm())


def test_graph_on_a_side_stream(dsix):
    x = make(300, 256, torch.bfloat16, "plain", 1)
    gamma, beta = weights(256, torch.bfloat16, "f32", 1)
    outs = [torch.empty_like(x), torch.empty(300, device="cuda"), torch.empty(300, device="cuda"), torch.empty_like(x),
            torch.empty(256, device="cuda"), torch.empty(256, device="cuda")]
    work = torch.empty(dsix.ix_layer_norm_bwd_workspace_size(300, 256), dtype=torch.uint8, device="cuda")

    def both(stream=None):
        dsix.ix_layer_norm(x, gamma, beta, 1e-6, *outs[:3], stream=stream)
        dsix.ix_layer_norm_bwd(x, x, gamma, outs[1], outs[2], *outs[3:], work, stream=stream)

    both()
    want = [o.clone() for o in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        both(side)
    torch.cuda.current_stream().wait_stream(side)
    for o in outs:
        o.zero_()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
