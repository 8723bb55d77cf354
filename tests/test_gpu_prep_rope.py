"""ix_rope_table and ix_rope against the formulas in 64 bits (the table's angles
in exact fractions).

Tolerances, with u = 2^-24 (half a step of f32 relative to the value): a rotated
value is two f32 products and a sum, at most 2u(|a c| + |b s|) off, then rounded
once to the type: eps / 2 relative, or half the smallest subnormal.  A table
entry: the angle's fraction of a quarter turn is rounded to f32 (u pi / 4), the
sine within 2 of its units (4u), the amplitude's product u: 8u of the
amplitude, and p 2^-62 turns from the frequency's fixed point.
"""
from fractions import Fraction
import math

import pytest
import torch

from _helpers import require_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
PI = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def dsix():
    require_gpu()
    import deepseek_v3_sparse_gb300 as m
    m.load_prep()
    m.ix_prep_device_status()
    return m


@pytest.mark.parametrize("first,n,rot,scaling", [
    (0, 1, 2, None), (0, 300, 64, None), (131000, 72, 64, "yarn"), (1 << 20, 33, 128, "ntk"), (7, 5, 256, "linear"),
    ((1 << 40) - 3, 3, 66, None),
])
def test_table(dsix, first, n, rot, scaling):
    inv = dsix.ix_rope_frequencies(rot, 10000.0, scaling, 40.0, 4096)
    got = torch.full((n, rot), 7.0, device="cuda")
    dsix.ix_rope_table(got, inv, first_position=first, amplitude=1.25)
    got = got.cpu()
    for r in range(n):
        for i in range(rot // 2):
            turn = (Fraction(inv[i]) * (first + r) / (2 * PI)) % 1
            angle = 2 * math.pi * float(turn)
            tol = 1.25 * (8 * U + 2 * math.pi * (first + r) * 2.0 ** -62)
            assert abs(float(got[r, i]) - 1.25 * math.cos(angle)) <= tol, (r, i)
            assert abs(float(got[r, rot // 2 + i]) - 1.25 * math.sin(angle)) <= tol, (r, i)


def test_table_of_any_frequency(dsix):
    # whole turns per position, a quarter, negative, more than a turn, zero
    inv = [2 * math.pi, math.pi / 2, -0.75, 100.0, 0.0, 3.0]
    got = torch.empty(1000, 12, device="cuda")
    dsix.ix_rope_table(got, inv)
    a = torch.arange(1000, dtype=torch.float64)[:, None] * torch.tensor(inv, dtype=torch.float64)
    want = torch.cat([a.cos(), a.sin()], 1)
    # the reference's angle is off by 2^-53 of at most 100000
    assert (got.cpu().double() - want).abs().max() <= 8 * U + 100000 * 2.0 ** -52


def reference(x, pos, table, offset, interleaved, inverse):
    """(the result, the sum of the magnitudes of its two products) in 64 bits."""
    x, row = x.double().cpu(), table.double().cpu()[pos.cpu()][:, None]
    half = row.shape[-1] // 2
    c, s = row[..., :half], row[..., half:]
    s = -s if inverse else s
    idx = torch.arange(half)
    ia = offset + (2 * idx if interleaved else idx)
    ib = ia + (1 if interleaved else half)
    out, size = x.clone(), torch.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, a * s + b * c
    size[..., ia], size[..., ib] = (a * c).abs() + (b * s).abs(), (a * s).abs() + (b * c).abs()
    return out, size


def close(got, want, size, rotated):
    t = got.dtype
    tol = torch.finfo(t).eps / 2 * want.abs() + 2 * U * (1 + torch.finfo(t).eps) * size + \
        torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2
    d = (got.double().cpu() - want).abs()
    assert bool((d <= tol).all()), f"off by {float((d - tol).max())} more than allowed"


def make(tokens, heads, dim, dtype, layout, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, heads, dim + 24, generator=g).to(dtype).cuda()
    if layout == "sliced":                       # strided rows of a wider projection
        return x[..., 8:8 + dim], torch.empty(tokens, heads, dim + 8, dtype=dtype, device="cuda")[..., :dim]
    if layout == "odd":                          # not even 4-byte aligned
        return x[..., 1:1 + dim], torch.empty(tokens, heads, dim + 3, dtype=dtype, device="cuda")[..., 3:]
    if layout == "heads first":                  # [H, T, D] seen as [T, H, D]
        return (x[..., :dim].transpose(0, 1).contiguous().transpose(0, 1),
                torch.empty(heads, tokens, dim, dtype=dtype, device="cuda").transpose(0, 1))
    return x[..., :dim].contiguous(), torch.empty(tokens, heads, dim, dtype=dtype, device="cuda")


SHAPES = [  # tokens, heads, dim, rot, offset
    (1, 1, 2, 2, 0), (1, 64, 128, 64, 0), (3, 5, 128, 128, 0), (7, 128, 192, 64, 128), (33, 1, 80, 40, 40),
    (5, 3, 77, 30, 11), (2, 6, 256, 256, 0), (9, 2, 72, 64, 8), (1030, 64, 128, 64, 0), (700, 67, 96, 32, 64),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("layout", ["plain", "sliced", "odd", "heads first"])
def test_rope(dsix, dtype, interleaved, layout):
    for n, (tokens, heads, dim, rot, offset) in enumerate(SHAPES):
        x, out = make(tokens, heads, dim, dtype, layout, n)
        out.fill_(9.0)
        table = torch.empty(500, rot, device="cuda")
        dsix.ix_rope_table(table, dsix.ix_rope_frequencies(rot), first_position=17)
        pos = torch.randint(0, 500, (tokens,), generator=torch.Generator().manual_seed(n)).cuda()
        inverse = n % 2 == 1
        dsix.ix_rope(x, pos, table, out, offset=offset, interleaved=interleaved, inverse=inverse)
        want, size = reference(x, pos, table, offset, interleaved, inverse)
        close(out, want, size, rot)
        kept = torch.ones(dim, dtype=torch.bool)
        kept[offset:offset + rot] = False
        assert torch.equal(out[..., kept].cpu(), x[..., kept].cpu())  # copied bit for bit
        # in place: the same bits
        y = x.clone() if layout != "sliced" else torch.empty(tokens, heads, dim + 8, dtype=dtype, device="cuda")[..., :dim]
        y.copy_(x)
        dsix.ix_rope(y, pos, table, y, offset=offset, interleaved=interleaved, inverse=inverse)
        assert torch.equal(y, out), (tokens, heads, dim)
    assert dsix.ix_prep_device_status() == 0


def test_two_tensors_and_a_broadcast_input(dsix):
    g = torch.Generator().manual_seed(3)
    table = torch.empty(64, 64, device="cuda")
    dsix.ix_rope_table(table, dsix.ix_rope_frequencies(64))
    for tokens in (1, 13, 2100):
        q = torch.randn(tokens, 64, 128, generator=g).bfloat16().cuda()
        k = torch.randn(tokens, 1, 128, generator=g).bfloat16().cuda().expand(tokens, 3, 128)  # stride 0 heads
        pos = torch.randint(0, 64, (tokens,), generator=g).cuda()
        oq, ok = torch.empty_like(q), torch.empty(tokens, 3, 128, dtype=q.dtype, device="cuda")
        dsix.ix_rope(q, pos, table, oq, x2=k, out2=ok)
        close(oq, *reference(q, pos, table, 0, False, False), 64)
        close(ok, *reference(k, pos, table, 0, False, False), 64)
        # one of the two in place, the other not
        k2 = k.contiguous()
        dsix.ix_rope(q, pos, table, oq, x2=k2, out2=k2)
        assert torch.equal(k2, ok)
    assert dsix.ix_prep_device_status() == 0


def test_the_inverse_is_the_gradient(dsix):
    """<R x, g> = <x, R^T g>, and the difference quotient of <R x, g> along v is
    <v, R^T g> (the map is linear, so it has no truncation error)."""
    g = torch.Generator().manual_seed(4)
    x, w, v = (torch.randn(50, 4, 96, generator=g).cuda() for _ in range(3))
    pos = torch.randint(0, 90, (50,), generator=g).cuda()
    table = torch.empty(90, 64, device="cuda")
    dsix.ix_rope_table(table, dsix.ix_rope_frequencies(64), amplitude=1.3)
    for inter in (False, True):
        turn = lambda a, inv=False: (lambda o: (dsix.ix_rope(a, pos, table, o, 32, inter, inv), o)[1])(torch.empty_like(a))  # noqa: E731
        f = lambda a: float((turn(a).double() * w.double()).sum())  # noqa: E731
        grad = turn(w, True).double()
        # each value is off by at most 3u of a magnitude below 1.3 * 12
        tol = 50 * 4 * 96 * 3 * U * 1.3 * 12 * 6
        assert abs(f(x) - float((x.double() * grad).sum())) <= tol
        quotient = (f(x + v) - f(x - v)) / 2
        assert abs(quotient - float((v.double() * grad).sum())) <= 2 * tol


def test_more_items_than_one_launch_indexes(dsix):
    """65536 heads of 128 values in single elements: a launch takes 1024 tokens, so
    1030 go out in two, the second at an offset past 2^32 elements.  The input is
    one token's, broadcast."""
    heads, dim, tokens = 65536, 128, 1030
    x = torch.randn(1, heads, dim, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    out = torch.empty(tokens, heads, dim, dtype=torch.bfloat16, device="cuda")
    table = torch.empty(tokens, 2, device="cuda")
    dsix.ix_rope_table(table, [0.01])
    pos = torch.arange(tokens, device="cuda").flip(0).contiguous()
    dsix.ix_rope(x.expand(tokens, heads, dim), pos, table, out, offset=3)
    assert dsix.ix_prep_device_status() == 0
    for t in (0, 1, 1022, 1023, 1024, 1025, 1029):
        want, size = reference(x, pos[t:t + 1], table, 3, False, False)
        close(out[t:t + 1], want, size, 2)


def test_bad_positions_are_skipped(dsix):
    table = torch.ones(8, 64, device="cuda")
    x = torch.randn(4, 3, 128, device="cuda")
    out = torch.full_like(x, 5.0)
    dsix.ix_rope(x, torch.tensor([0, -1, 8, 7], device="cuda"), table, out)
    assert dsix.ix_prep_device_status() == 32
    assert bool((out[1:3] == 5).all()) and not bool((out[[0, 3]] == 5).all())


def test_special_values_pass_through(dsix):
    table = torch.empty(4, 64, device="cuda")
    dsix.ix_rope_table(table, dsix.ix_rope_frequencies(64))
    x = torch.zeros(2, 1, 128, device="cuda")
    x[0, 0, 3], x[1, 0, 100] = float("nan"), float("inf")  # one rotated, one copied
    out = torch.empty_like(x)
    dsix.ix_rope(x, torch.tensor([1, 2], device="cuda"), table, out)
    bad = torch.isnan(out[0, 0]).nonzero().flatten().tolist()
    assert bad == [3, 35] and float(out[1, 0, 100]) == float("inf") and int(torch.isfinite(out[1]).sum()) == 127


def test_graph_on_a_side_stream(dsix):
    table = torch.empty(64, 64, device="cuda")
    dsix.ix_rope_table(table, dsix.ix_rope_frequencies(64))
    x = torch.randn(10, 4, 128, device="cuda").half()
    pos = torch.arange(10, device="cuda")
    out, again = torch.empty_like(x), torch.empty_like(x)
    dsix.ix_rope(x, pos, table, out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        dsix.ix_rope(x, pos, table, again, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph.replay()
    assert torch.equal(out, again)


def test_nothing_to_do(dsix):
    x = torch.empty(0, 4, 128, device="cuda")
    dsix.ix_rope(x, torch.empty(0, dtype=torch.int64, device="cuda"), torch.ones(4, 64, device="cuda"), x.clone())
    dsix.ix_rope_table(torch.empty(0, 64, device="cuda"), [0.1] * 32)
    assert dsix.ix_prep_device_status() == 0
