"""libdsix_prep's C ABI and binding (CPU only: no kernel is launched): the
exported functions are those include/dsix_prep.h declares, every host-side
argument check returns before anything touches a GPU, the binding refuses
inconsistent shapes before it takes a pointer, and the rotary frequencies (a
host function) follow their formulas."""
import ctypes
import math
import os
import re
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dsix_prep.h")

OK, NULL, SHAPE, UNSUPPORTED, ALIGN, WORKSPACE = 0, -1, -2, -3, -4, -5
P = ctypes.c_void_p
A = P(0x10000)       # aligned fake device address (no check dereferences it)
ODD = P(0x10001)

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and
                                not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")


@pytest.fixture(scope="module")
def dsix():
    from deepseek_v3_sparse_gb300 import build
    import deepseek_v3_sparse_gb300 as m
    build.build()
    m.load_prep()
    return m


@pytest.fixture(scope="module")
def lib(dsix):
    return dsix.load_prep()


def test_exports_match_header(lib):
    names = sorted(set(re.findall(r"IX_API\s+[\w\s\*]+?\b(\w+)\s*\(", open(HEADER).read())))
    out = subprocess.run(["nm", "-D", "--defined-only", lib._name], capture_output=True, text=True, check=True).stdout
    exported = sorted(l.split()[-1] for l in out.splitlines()
                      if l.split()[-2:-1] == ["T"] and not l.split()[-1].startswith("_"))
    assert exported == names and len(names) == 9


def test_missing_library_is_an_error(dsix, tmp_path):
    with pytest.raises(dsix.DsixError, match="missing"):
        dsix.load_prep(str(tmp_path / "none.so"))


def _plan(**kw):
    order = ["cached", "new", "batch", "bs", "free", "n_free", "table", "stride", "width", "ctx", "cu_new", "cu_ctx",
             "cu_blocks", "slots", "pos", "req", "len", "ks", "ke", "rows"]
    d = dict(cached=A, new=A, batch=4, bs=64, free=A, n_free=9, table=A, stride=8, width=8, ctx=A, cu_new=A, cu_ctx=A,
             cu_blocks=A, slots=A, pos=A, req=A, len=A, ks=A, ke=A, rows=16)
    d.update(kw)
    return [d[k] for k in order] + [None]


@pytest.mark.parametrize("kw,want", [
    (dict(batch=-1), SHAPE), (dict(rows=-1), SHAPE), (dict(n_free=-1), SHAPE), (dict(width=9), SHAPE),
    (dict(stride=-8, width=-8), SHAPE), (dict(bs=0), UNSUPPORTED), (dict(rows=2 ** 31), UNSUPPORTED),
    (dict(cached=None), NULL), (dict(new=None), NULL), (dict(free=None), NULL), (dict(table=None), NULL),
    (dict(ctx=None), NULL), (dict(cu_new=None), NULL), (dict(cu_ctx=None), NULL), (dict(cu_blocks=None), NULL),
    (dict(slots=None), NULL), (dict(pos=None), NULL), (dict(req=None), NULL), (dict(len=None), NULL),
    (dict(ks=None), NULL), (dict(ke=None), NULL), (dict(slots=P(0x10008)), ALIGN), (dict(ke=P(0x10004)), ALIGN),
    (dict(table=P(0x10002)), ALIGN),
])
def test_plan_refusals(lib, kw, want):
    assert lib.ix_plan_step(*_plan(**kw)) == want


def _rope_call(dsix, lib, side=None, side2=None, **kw):
    from deepseek_v3_sparse_gb300.prep import _RopeTensor
    d = dict(x=A, out=P(0x20000), heads=4, xt=512, xh=128, ot=512, oh=128)
    d.update(side or {})
    one = _RopeTensor(*[d[k] for k in ("x", "out", "heads", "xt", "xh", "ot", "oh")])
    two = None
    if side2 is not None:
        e = dict(d, x=P(0x30000), out=P(0x40000))
        e.update(side2)
        two = ctypes.byref(_RopeTensor(*[e[k] for k in ("x", "out", "heads", "xt", "xh", "ot", "oh")]))
    a = dict(dtype=0, tokens=3, dim=128, offset=0, pos=A, table=A, max_pos=9, rot=64, flags=0)
    a.update(kw)
    return lib.ix_rope(ctypes.byref(one), two, *[a[k] for k in ("dtype", "tokens", "dim", "offset", "pos", "table",
                                                               "max_pos", "rot", "flags")], None)


@pytest.mark.parametrize("side,side2,kw,want", [
    ({}, None, dict(dtype=3), UNSUPPORTED), ({}, None, dict(rot=0), UNSUPPORTED), ({}, None, dict(rot=63), UNSUPPORTED),
    (dict(ot=2048, oh=512), None, dict(rot=258, dim=512), UNSUPPORTED), ({}, None, dict(offset=65), UNSUPPORTED),
    ({}, None, dict(flags=4), UNSUPPORTED), ({}, None, dict(tokens=-1), SHAPE), ({}, None, dict(offset=-2), SHAPE),
    ({}, None, dict(max_pos=-1), SHAPE), (dict(heads=0), None, {}, SHAPE), (dict(xt=-512), None, {}, SHAPE),
    (dict(oh=64), None, {}, SHAPE), (dict(ot=128), None, {}, SHAPE), ({}, dict(ot=100), {}, SHAPE),
    (dict(out=A, ot=1024), None, {}, SHAPE),  # in place with other strides
    (dict(x=None), None, {}, NULL), ({}, dict(out=None), {}, NULL), ({}, None, dict(pos=None), NULL),
    ({}, None, dict(table=None), NULL), (dict(x=ODD), None, {}, ALIGN), ({}, None, dict(pos=P(0x10004)), ALIGN),
    ({}, None, dict(table=P(0x10002)), ALIGN), ({}, None, dict(tokens=0), OK),
])
def test_rope_refusals(dsix, lib, side, side2, kw, want):
    assert _rope_call(dsix, lib, side, side2, **kw) == want


def test_rope_table_refusals(lib):
    f = (ctypes.c_double * 32)(*[0.5] * 32)
    bad = (ctypes.c_double * 32)(*[float("nan")] * 32)
    assert lib.ix_rope_table(f, 63, 0, 4, 1.0, A, None) == UNSUPPORTED
    assert lib.ix_rope_table(f, 64, -1, 4, 1.0, A, None) == SHAPE
    assert lib.ix_rope_table(f, 64, 0, -4, 1.0, A, None) == SHAPE
    assert lib.ix_rope_table(f, 64, 2 ** 40, 1, 1.0, A, None) == UNSUPPORTED
    assert lib.ix_rope_table(f, 64, 2 ** 62, 2 ** 62, 1.0, A, None) == UNSUPPORTED
    assert lib.ix_rope_table(f, 64, 0, 4, float("inf"), A, None) == UNSUPPORTED
    assert lib.ix_rope_table(bad, 64, 0, 4, 1.0, A, None) == UNSUPPORTED
    assert lib.ix_rope_table((ctypes.c_double * 32)(*[2.0 ** 20] * 32), 64, 0, 4, 1.0, A, None) == UNSUPPORTED
    assert lib.ix_rope_table(None, 64, 0, 4, 1.0, A, None) == NULL
    assert lib.ix_rope_table(f, 64, 0, 4, 1.0, None, None) == NULL
    assert lib.ix_rope_table(f, 64, 0, 4, 1.0, P(0x10008), None) == ALIGN
    assert lib.ix_rope_table(f, 64, 0, 0, 1.0, None, None) == OK


def _norm(**kw):
    d = dict(x=A, xs=128, gamma=A, beta=A, wt=2, eps=1e-6, rows=4, cols=128, out=P(0x20000), os=128, mean=A, rstd=A,
             dtype=0)
    d.update(kw)
    return [d[k] for k in ("x", "xs", "gamma", "beta", "wt", "eps", "rows", "cols", "out", "os", "mean", "rstd",
                           "dtype")] + [None]


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), SHAPE), (dict(cols=0), SHAPE), (dict(xs=-1), SHAPE), (dict(os=127), SHAPE),
    (dict(out=A, os=256), SHAPE), (dict(cols=32769, xs=32769, os=32769), UNSUPPORTED), (dict(dtype=5), UNSUPPORTED),
    (dict(wt=1), UNSUPPORTED), (dict(eps=-1.0), UNSUPPORTED), (dict(eps=float("nan")), UNSUPPORTED),
    (dict(eps=float("inf")), UNSUPPORTED), (dict(x=None), NULL), (dict(out=None), NULL), (dict(mean=None), NULL),
    (dict(x=ODD), ALIGN), (dict(gamma=P(0x10008)), ALIGN), (dict(rstd=P(0x10002)), ALIGN), (dict(rows=0), OK),
])
def test_layer_norm_refusals(lib, kw, want):
    assert lib.ix_layer_norm(*_norm(**kw)) == want


def _norm_bwd(lib, **kw):
    d = dict(dy=A, dys=128, x=A, xs=128, gamma=A, wt=2, mean=A, rstd=A, rows=4, cols=128, dx=P(0x20000), dxs=128,
             dgamma=A, dbeta=A, dtype=0, ws=A, nb=None)
    d.update(kw)
    if d["nb"] is None:
        d["nb"] = lib.ix_layer_norm_bwd_workspace_size(d["rows"], d["cols"])
    return lib.ix_layer_norm_bwd(*[d[k] for k in ("dy", "dys", "x", "xs", "gamma", "wt", "mean", "rstd", "rows", "cols",
                                                  "dx", "dxs", "dgamma", "dbeta", "dtype", "ws", "nb")], None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), SHAPE), (dict(cols=0), SHAPE), (dict(dxs=1), SHAPE), (dict(dys=-1), SHAPE),
    (dict(dx=A, dxs=256), SHAPE), (dict(cols=32769, dxs=32769), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED),
    (dict(wt=1), UNSUPPORTED), (dict(dbeta=None), NULL), (dict(dy=None), NULL), (dict(mean=None), NULL),
    (dict(dx=None), NULL), (dict(dx=ODD), ALIGN), (dict(ws=None), WORKSPACE), (dict(nb=4), WORKSPACE),
    (dict(ws=P(0x10008)), ALIGN), (dict(rows=0, dgamma=None, dbeta=None), OK),
])
def test_layer_norm_bwd_refusals(lib, kw, want):
    assert _norm_bwd(lib, **kw) == want


def test_layer_norm_bwd_workspace_size(lib):
    f = lib.ix_layer_norm_bwd_workspace_size
    assert f(0, 128) == 0 and f(-1, 128) == 0 and f(4, 0) == 0
    assert f(1, 128) >= 2 * 128 * 4 and f(10 ** 9, 128) == f(10 ** 6, 128)


def _write(**kw):
    d = dict(k=A, ks=128, dtype=0, n=4, gamma=A, beta=A, eps=1e-6, pos=A, table=A, max_pos=9, rot=64, off=0, inter=0,
             slots=A, cache=A, nb=8, bs=64)
    d.update(kw)
    return list(d.values()) + [None]


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), SHAPE), (dict(nb=-1), SHAPE), (dict(ks=-128), SHAPE), (dict(max_pos=-1), SHAPE),
    (dict(dtype=4), UNSUPPORTED), (dict(bs=32), UNSUPPORTED), (dict(eps=-1.0), UNSUPPORTED),
    (dict(rot=0), UNSUPPORTED), (dict(rot=40), UNSUPPORTED), (dict(rot=8), UNSUPPORTED), (dict(off=4), UNSUPPORTED),
    (dict(off=72), UNSUPPORTED), (dict(rot=144), UNSUPPORTED), (dict(off=-16), UNSUPPORTED), (dict(k=None), NULL), (dict(gamma=None), NULL),
    (dict(slots=None), NULL), (dict(table=None), NULL), (dict(cache=None), NULL), (dict(ks=132), ALIGN),
    (dict(k=P(0x10008)), ALIGN), (dict(table=P(0x10004)), ALIGN), (dict(pos=P(0x10004)), ALIGN), (dict(n=0), OK),
])
def test_norm_rope_write_refusals(lib, kw, want):
    assert lib.ix_norm_rope_write_k(*_write(**kw)) == want


# --- the binding -----------------------------------------------------------

def _said(fn, *a, **kw):
    with pytest.raises(Exception) as e:
        fn(*a, **kw)
    return str(e.value)


def bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


def i64(*s):
    return torch.zeros(*s, dtype=torch.int64)


def f32(*s):
    return torch.zeros(*s)


def u8(*s):
    return torch.zeros(*s, dtype=torch.uint8)


CALLS = {
    "ix_plan_step": (["cached_lens", "new_lens", "free_blocks", "block_table", "context_lens", "cu_new", "cu_ctx",
                      "cu_blocks", "slot_mapping", "positions", "row_req", "row_len", "ks", "ke"],
                     lambda: [i32(3), i32(3), i32(5), i32(3, 4), i32(3), i32(4), i32(4), i32(4), i64(9), i64(9),
                              i32(9), i32(9), i32(9), i32(9)],
                     [(1, i32(2)), (3, i32(2, 4)), (3, i32(12)), (4, i32(2)), (5, i32(3)), (6, i32(3)), (7, i32(3)),
                      (9, i64(8)), (10, i32(8)), (11, i32(8)), (12, i32(8)), (13, i32(8))]),
    "ix_rope": (["x", "positions", "cos_sin", "out"], lambda: [bf(5, 4, 128), i64(5), f32(9, 64), bf(5, 4, 128)],
                [(0, bf(5, 128)), (0, bf(128, 4, 5).transpose(0, 2)), (1, i64(4)), (2, f32(64)), (3, bf(5, 3, 128)),
                 (3, bf(4, 4, 128)), (3, f32(5, 4, 128))]),
    "ix_layer_norm": (["x", "gamma", "beta", "eps", "out", "mean", "rstd"],
                      lambda: [bf(5, 128), f32(128), f32(128), 1e-6, bf(5, 128), f32(5), f32(5)],
                      [(0, bf(128)), (0, i32(5, 128)), (1, f32(127)), (1, i32(128)), (2, bf(128)), (2, f32(129)),
                       (4, bf(5, 127)), (4, f32(5, 128)), (5, f32(4)), (6, None)]),
    "ix_layer_norm_bwd": (["dy", "x", "gamma", "mean", "rstd", "dx", "dgamma", "dbeta", "workspace"],
                          lambda: [bf(5, 128), bf(5, 128), bf(128), f32(5), f32(5), bf(5, 128), f32(128), f32(128),
                                   u8(1 << 20)],
                          [(0, bf(4, 128)), (0, f32(5, 128)), (2, bf(120)), (3, f32(4)), (4, f32(4)), (5, bf(5, 64)),
                           (6, f32(127)), (7, None)]),
    "ix_norm_rope_write_k": (["k", "gamma", "beta", "eps", "positions", "cos_sin", "slot_mapping", "cache"],
                             lambda: [bf(5, 128), f32(128), f32(128), 1e-6, i64(5), f32(9, 64), i64(5), u8(3, 8448)],
                             [(0, bf(5, 64)), (0, i32(5, 128)), (1, f32(64)), (4, i64(4)), (5, f32(64)), (6, i64(4)),
                              (7, u8(3, 8000)), (7, u8(8448))]),
    "ix_rope_table": (["cos_sin", "inv_freq"], lambda: [f32(9, 64), [0.1] * 32], [(0, f32(64)), (1, [0.1] * 31)]),
}


@pytest.mark.parametrize("name", CALLS)
def test_binding_checks(dsix, name):
    """Consistent CPU tensors get as far as the device check; each inconsistent
    one is refused before it, by its name."""
    fn = getattr(dsix, name)
    names, make, bad = CALLS[name]
    assert "must be a CUDA tensor" in _said(fn, *make())
    for i, value in bad:
        a = make()
        a[i] = value
        said = _said(fn, *a)
        assert names[i].split("_")[0] in said and "CUDA tensor" not in said, (names[i], said)


def test_binding_checks_of_the_second_rope_tensor(dsix):
    a = [bf(5, 4, 128), i64(5), f32(9, 64), bf(5, 4, 128)]
    assert "must be a CUDA tensor" in _said(dsix.ix_rope, *a, x2=bf(5, 1, 128), out2=bf(5, 1, 128))
    for x2, out2 in ((bf(4, 1, 128), bf(4, 1, 128)), (bf(5, 1, 64), bf(5, 1, 64)), (bf(5, 1, 128), bf(5, 2, 128)),
                     (bf(5, 1, 128), None), (f32(5, 1, 128), f32(5, 1, 128))):
        said = _said(dsix.ix_rope, *a, x2=x2, out2=out2)
        assert "2" in said and "CUDA tensor" not in said


# --- the rotary frequencies ------------------------------------------------

@pytest.mark.parametrize("rot", [2, 6, 64, 256])
@pytest.mark.parametrize("scaling", [None, "linear", "ntk", "yarn"])
def test_rope_frequencies(dsix, rot, scaling):
    base, factor, original = 10000.0, 40.0, 4096
    got = dsix.ix_rope_frequencies(rot, base, scaling, factor, original)
    b = base * factor ** (rot / (rot - 2)) if scaling == "ntk" and rot > 2 else base
    plain = [b ** (-2 * i / rot) for i in range(rot // 2)]
    want = plain
    if scaling == "linear":
        want = [w / factor for w in plain]
    if scaling == "yarn":
        d = lambda turns: rot * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
        low, high = max(math.floor(d(32)), 0), min(math.ceil(d(1)), rot - 1)
        g = [min(max((i - low) / max(high - low, 0.001), 0), 1) for i in range(rot // 2)]
        want = [w * (1 - x) + w / factor * x for w, x in zip(plain, g)]
        if rot == 64:  # fast pairs keep their frequency, slow ones are stretched
            assert got[0] == 1.0 and math.isclose(got[-1], plain[-1] / factor, rel_tol=1e-14)
    # a few roundings of 2^-53; the power amplifies that of its exponent by ln(base * factor) < 16
    assert len(got) == rot // 2 and all(math.isclose(x, y, rel_tol=64 * 2 ** -53) for x, y in zip(got, want))


def test_rope_frequencies_refusals(dsix):
    for kw in (dict(rot=3), dict(rot=0), dict(rot=258), dict(rot=64, base=1.0), dict(rot=64, base=float("inf")),
               dict(rot=64, scaling="linear", factor=0.5), dict(rot=64, scaling="yarn", factor=2.0),
               dict(rot=64, scaling="yarn", factor=2.0, original=4096, beta_fast=0.5),
               dict(rot=64, scaling="yarn", factor=2.0, original=4096, beta_slow=0.0), dict(rot=64, scaling="bent")):
        with pytest.raises(dsix.DsixError):
            dsix.ix_rope_frequencies(**kw)
