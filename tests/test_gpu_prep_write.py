"""ix_norm_rope_write_k against its definition in 64 bits.

With u = 2^-24: a normed and rotated value z is at most
E = 256u (|xhat gamma| + |beta| + rstd mean|x| |gamma|), over the two values of
its pair, off before it is coded (a row's sums: see the layer norm's tests).  The
scale is amax / 448, off by max E / 448 and two roundings; a code stands for its
value to half a step of e4m3: 2^-4 relative, or half its smallest subnormal,
2^-10, of the scale.
"""
import numpy as np
import pytest
import torch

from _helpers import require_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def dsix():
    require_gpu()
    import deepseek_v3_sparse_gb300 as m
    m.load()
    m.load_prep()
    m.ix_prep_device_status()
    return m


def reference(k, gamma, beta, eps, pos, table, offset, interleaved):
    """(z, its error bound before the coding) in 64 bits."""
    x, g, b = k.double().cpu(), gamma.double().cpu(), beta.double().cpu()
    mean = x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + eps)
    xhat = (x - mean) * rstd
    y = xhat * g + b
    e = 256 * U * ((xhat * g).abs() + b.abs() + rstd * x.abs().mean(1, keepdim=True) * g.abs())
    row = table.double().cpu()[pos.cpu()]
    half = row.shape[1] // 2
    c, s = row[:, :half], row[:, half:]
    i = torch.arange(half)
    ia = offset + (2 * i if interleaved else i)
    ib = ia + (1 if interleaved else half)
    z, ez = y.clone(), e.clone()
    z[:, ia], z[:, ib] = y[:, ia] * c - y[:, ib] * s, y[:, ia] * s + y[:, ib] * c
    ez[:, ia] = ez[:, ib] = (e[:, ia] + e[:, ib]) * 1.5
    return z, ez


def run(dsix, n, dtype, rot, offset, interleaved, seed=0, pad=0, eps=1e-6, max_pos=300, blocks=None, skip=0):
    g = torch.Generator().manual_seed(seed)
    k = (torch.randn(n, 128 + pad, generator=g) * 2 + 0.3).to(dtype).cuda()[:, pad // 2:pad // 2 + 128]
    gamma, beta = (1 + 0.3 * torch.randn(128, generator=g)).cuda(), (0.3 * torch.randn(128, generator=g)).cuda()
    table = torch.empty(max_pos, rot, device="cuda")
    dsix.ix_rope_table(table, dsix.ix_rope_frequencies(rot))
    pos = torch.randint(0, max_pos, (n,), generator=g).cuda()
    blocks = blocks or (n + 63) // 64 + 3
    slots = torch.randperm(blocks * 64, generator=g)[:n]
    if skip:
        slots[::skip] = -1
    cache = torch.full((blocks, 8448), 0xAB, dtype=torch.uint8, device="cuda")
    dsix.ix_norm_rope_write_k(k, gamma, beta, eps, pos, table, slots.cuda(), cache, rope_offset=offset,
                              interleaved=interleaved)
    assert dsix.ix_prep_device_status() == 0
    return k, gamma, beta, table, pos, slots, cache


def entries(cache):
    codes = cache[:, :8192].reshape(-1, 128).cpu()
    scales = cache[:, 8192:].contiguous().view(torch.float32).reshape(-1).cpu()
    return codes, scales


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rot,offset", [(64, 0), (64, 64), (32, 0), (32, 48), (16, 0), (16, 112), (96, 16), (48, 8), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_values(dsix, dtype, rot, offset, interleaved):
    for n, pad, skip in ((1, 0, 0), (2, 16, 0), (63, 64, 5), (1000, 0, 3)):
        k, gamma, beta, table, pos, slots, cache = run(dsix, n, dtype, rot, offset, interleaved, seed=n, pad=pad, skip=skip)
        z, e = reference(k, gamma, beta, 1e-6, pos, table, offset, interleaved)
        codes, scales = entries(cache)
        live = slots >= 0
        got = codes[slots[live]].view(torch.float8_e4m3fn).double()
        sc = scales[slots[live]].double()
        z, e = z[live], e[live]
        amax = z.abs().amax(1)
        assert bool(((sc - amax / 448).abs() <= e.amax(1) / 448 + 4 * U * amax / 448).all())
        d = (got * sc[:, None] - z).abs()
        assert bool((d <= 2.0 ** -4 * z.abs() * (1 + 2.0 ** -10) + 2.0 ** -10 * sc[:, None] + 2 * e).all())
        # what no token names stays as it was
        others = torch.ones(codes.shape[0], dtype=torch.bool)
        others[slots[live]] = False
        assert bool((codes[others] == 0xAB).all())


def test_agrees_with_the_separate_calls(dsix):
    """Norm and rotation in f32, then the plain write of the bf16 key: the two
    paths differ by the bf16 rounding alone, at most one e4m3 step of a value."""
    k, gamma, beta, table, pos, slots, cache = run(dsix, 500, torch.float32, 64, 0, False, seed=9)
    y = torch.empty(500, 128, device="cuda")
    dsix.ix_layer_norm(k, gamma, beta, 1e-6, y)
    dsix.ix_rope(y[:, None], pos, table, y[:, None])
    other = torch.full_like(cache, 0xAB)
    dsix.ix_quant_write_k(y.bfloat16(), slots.cuda(), other)
    a, sa = entries(cache)
    b, sb = entries(other)
    va = a[slots].view(torch.float8_e4m3fn).double() * sa[slots].double()[:, None]
    vb = b[slots].view(torch.float8_e4m3fn).double() * sb[slots].double()[:, None]
    step = 2.0 ** -3 * torch.maximum(va.abs(), vb.abs()) + 2.0 ** -9 * sa[slots].double()[:, None]
    assert bool(((va - vb).abs() <= step * (1 + 2.0 ** -7)).all())


def test_constant_and_special_rows(dsix):
    """A constant row norms to beta; beta = 0 leaves zeros under the smallest
    scale; a NaN makes its own row NaN and no other."""
    k = torch.zeros(4, 128, device="cuda")
    k[1] = 5.0
    k[2, 9] = float("nan")
    k[3] = torch.arange(128, device="cuda").float()
    gamma, beta = torch.ones(128, device="cuda"), torch.zeros(128, device="cuda")
    table = torch.empty(8, 64, device="cuda")
    dsix.ix_rope_table(table, dsix.ix_rope_frequencies(64))
    cache = torch.zeros(1, 8448, dtype=torch.uint8, device="cuda")
    dsix.ix_norm_rope_write_k(k, gamma, beta, 1e-6, torch.arange(4, device="cuda"), table, torch.arange(4, device="cuda"), cache)
    assert dsix.ix_prep_device_status() == 0
    codes, scales = entries(cache)
    assert not bool((codes[:2] & 0x7F).any()) and scales[:2].tolist() == [torch.finfo(torch.float32).tiny] * 2
    v = codes[:4].view(torch.float8_e4m3fn).float()
    assert bool(torch.isnan(v[2]).all()) and bool(torch.isfinite(v[3]).all()) and float(v[3].abs().max()) == 448


def test_bad_slots_and_positions_are_skipped(dsix):
    k = torch.randn(5, 128, device="cuda").bfloat16()
    one, zero = torch.ones(128, device="cuda"), torch.zeros(128, device="cuda")
    table = torch.ones(8, 64, device="cuda")
    cache = torch.full((2, 8448), 0xAB, dtype=torch.uint8, device="cuda")
    pos, slots = torch.tensor([0, -1, 8, 3, 99], device="cuda"), torch.tensor([0, 1, 2, 128, -1], device="cuda")
    dsix.ix_norm_rope_write_k(k, one, zero, 1e-6, pos, table, slots, cache)
    assert dsix.ix_prep_device_status() == 1 | 32  # a skipped token's position is not looked at
    codes, _ = entries(cache)
    assert bool((codes[1:] == 0xAB).all()) and not bool((codes[0] == 0xAB).all())


def test_graph_on_a_side_stream(dsix):
    k, gamma, beta, table, pos, slots, cache = run(dsix, 77, torch.bfloat16, 64, 0, False, seed=2)
    again = torch.full_like(cache, 0xAB)
    s = slots.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        dsix.ix_norm_rope_write_k(k, gamma, beta, 1e-6, pos, table, s, again, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph.replay()
    assert torch.equal(again, cache)


def test_no_tokens(dsix):
    e = torch.empty(0, dtype=torch.int64, device="cuda")
    w = torch.ones(128, device="cuda")
    cache = torch.zeros(1, 8448, dtype=torch.uint8, device="cuda")
    dsix.ix_norm_rope_write_k(torch.empty(0, 128, device="cuda"), w, w, 1e-6, e, torch.ones(8, 64, device="cuda"), e, cache)
    assert np.count_nonzero(cache.cpu().numpy()) == 0
