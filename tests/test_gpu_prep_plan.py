"""ix_plan_step against a plain loop over the requests: whole numbers, equal."""
import pytest
import torch

from _helpers import require_gpu

pytestmark = pytest.mark.gpu
BAD_BLOCK, BAD_RANGE, NO_BLOCK = 2, 8, 128
MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def dsix():
    require_gpu()
    import deepseek_v3_sparse_gb300 as m
    m.load_prep()
    m.ix_prep_device_status()
    return m


def plan_reference(cached, new, free, table, rows, bs):
    """The step, request by request; returns the outputs and the expected status bits."""
    status = 0
    cu_new, cu_ctx, cu_blocks, ctx = [0], [0], [0], []
    table = [list(r) for r in table]
    out = dict(slot_mapping=[], positions=[], row_req=[], row_len=[], ks=[], ke=[])

    def sat(x):
        nonlocal status
        if x >= MAX:
            status |= BAD_RANGE
        return min(x, MAX)

    for b, (c, n) in enumerate(zip(cached, new)):
        if c < 0 or n < 0:
            status |= BAD_RANGE
        c, n = max(c, 0), max(n, 0)
        have, need = -(-c // bs), -(-(c + n) // bs)
        for j in range(have, need):
            k = cu_blocks[-1] + j - have
            if j >= len(table[b]):
                status |= BAD_RANGE
                continue
            if k >= len(free):
                status |= NO_BLOCK
            table[b][j] = free[k] if k < len(free) else -1
        for p in range(c, c + n):
            if len(out["positions"]) == rows:
                break
            blk = table[b][p // bs] if p // bs < len(table[b]) else -1
            if p // bs < have and blk < 0 and p // bs < len(table[b]):
                status |= BAD_BLOCK
            if p // bs >= len(table[b]):
                status |= BAD_RANGE
            out["slot_mapping"].append(blk * bs + p % bs if blk >= 0 else -1)
            out["positions"].append(p)
            out["row_req"].append(b)
            out["row_len"].append(p + 1)
            out["ks"].append(cu_ctx[-1])
            out["ke"].append(cu_ctx[-1] + p + 1)
        ctx.append(c + n)
        cu_new.append(sat(cu_new[-1] + n))
        cu_ctx.append(sat(cu_ctx[-1] + c + n))
        cu_blocks.append(sat(cu_blocks[-1] + need - have))
    if cu_new[-1] > rows:
        status |= BAD_RANGE
    for name, v in out.items():
        v += [-1 if name == "slot_mapping" else 0] * (rows - len(v))
    out.update(block_table=table, context_lens=ctx, cu_new=cu_new, cu_ctx=cu_ctx, cu_blocks=cu_blocks)
    return out, status


def tensors(cached, new, free, table, rows, width):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    B = len(cached)
    e = lambda n, t=torch.int32: torch.full((n,), -77, dtype=t, device="cuda")  # noqa: E731
    return dict(cached_lens=i32(cached), new_lens=i32(new), free_blocks=i32(free),
                block_table=i32(table).reshape(B, width), context_lens=e(B), cu_new=e(B + 1), cu_ctx=e(B + 1),
                cu_blocks=e(B + 1), slot_mapping=e(rows, torch.int64), positions=e(rows, torch.int64), row_req=e(rows),
                row_len=e(rows), ks=e(rows), ke=e(rows))


def check(dsix, cached, new, rows=None, bs=64, free=None, width=None, spoil=None, table=None):
    B = len(cached)
    need = [-(-(max(c, 0) + max(n, 0)) // bs) for c, n in zip(cached, new)]
    have = [-(-max(c, 0) // bs) for c in cached]
    g = torch.Generator().manual_seed(len(cached) + sum(n for n in new if n > 0) % 1000)
    pool = torch.randperm(sum(need) + 9, generator=g).tolist()
    width = max(need + [1]) + 1 if width is None else width
    if table is None:
        table, at = [], 0
        for b in range(B):
            table.append((pool[at:at + have[b]] + [-5] * width)[:width])
            at += have[b]
    if spoil is not None:
        table[spoil[0]][spoil[1]] = -1
    free = pool[sum(have):] if free is None else free
    rows = sum(max(n, 0) for n in new) if rows is None else rows
    want, status = plan_reference(cached, new, free, table, rows, bs)
    t = tensors(cached, new, free, table, rows, width)
    for _ in range(2):  # the call can be repeated: the same lengths give the same table
        dsix.ix_plan_step(**t, block_size=bs)
        assert dsix.ix_prep_device_status() == status
        for name, v in want.items():
            assert t[name].flatten().tolist() == torch.tensor(v, dtype=torch.int64).flatten().tolist(), name
    return t


@pytest.mark.parametrize("bs", [64, 1, 48, 16])
@pytest.mark.parametrize("cached,new", [
    ([0], [1]), ([63], [1]), ([64], [1]), ([0], [0]), ([5, 0, 128], [0, 0, 0]), ([130, 64, 63, 0], [2, 2, 2, 2]),
    ([0, 100, 0, 64, 7], [300, 0, 0, 65, 1]), ([0, 0, 0], [0, 5, 0]),
])
def test_small(dsix, cached, new, bs):
    check(dsix, cached, new, bs=bs)


def test_no_requests(dsix):
    t = tensors([], [], [3], [], 5, 0)
    dsix.ix_plan_step(**t)
    assert dsix.ix_prep_device_status() == 0
    assert t["cu_new"].tolist() == t["cu_ctx"].tolist() == t["cu_blocks"].tolist() == [0]
    assert t["slot_mapping"].tolist() == [-1] * 5 and t["row_len"].tolist() == [0] * 5


@pytest.mark.parametrize("spare", [1, 2, 3, 4, 777])
def test_rows_padded_past_the_tokens(dsix, spare):
    check(dsix, [10, 64, 0], [3, 0, 70], rows=73 + spare)


@pytest.mark.parametrize("B,hi,seed", [(128, 2, 0), (37, 700, 1), (511, 9, 2), (512, 3, 3), (513, 3, 4), (2049, 5, 5),
                                       (4096, 3, 6), (4097, 3, 7), (9001, 2, 8)])
def test_ragged_batches(dsix, B, hi, seed):
    """Every size class of the scan: one pass and several, one launch and two."""
    g = torch.Generator().manual_seed(seed)
    new = torch.randint(0, hi + 1, (B,), generator=g).tolist()
    cached = torch.randint(0, 400, (B,), generator=g).tolist()
    check(dsix, cached, new)


@pytest.mark.parametrize("B", [1, 31, 32, 33, 256, 257, 511, 512, 513, 1023, 1024, 1025])
@pytest.mark.parametrize("hi", [1, 8, 9])
def test_steps_of_few_rows(dsix, B, hi):
    """Decode steps: a thread plans the rows of a request with up to eight; one request
    with more sends the step the other way."""
    g = torch.Generator().manual_seed(B + hi)
    new = torch.randint(0, hi + 1, (B,), generator=g).tolist()
    cached = torch.randint(0, 300, (B,), generator=g).tolist()
    new[B // 2] = hi
    check(dsix, cached, new, bs=16)
    check(dsix, cached, new, bs=64, rows=sum(new) + 300)
    check(dsix, cached, new, bs=3, rows=max(1, sum(new) // 2))


def test_long_contexts(dsix):
    # positions and slots of a cache past 2^31 keys: the slot is formed in 64 bits
    width = 5
    bs = 1 << 20
    table = [[7, 3000, -5, -5, -5], [2900, -5, -5, -5, -5]]
    t = check(dsix, [2 * bs - 1, 1], [3, 2], bs=bs, free=[4000, 4001], width=width, table=table)
    assert int(t["slot_mapping"][0]) == 3000 * bs + bs - 1 and int(t["slot_mapping"][1]) == 4000 * bs
    assert int(t["slot_mapping"][1]) > 2 ** 31


def test_what_does_not_fit_is_left_out(dsix):
    check(dsix, [0, 64, 10], [200, 5, 3], rows=150)             # more tokens than rows
    check(dsix, [0, 64, 10], [200, 5, 3], free=[11, 12])        # too few free blocks
    check(dsix, [0, 64, 10], [200, 5, 3], free=[])              # none
    check(dsix, [0, 64, 10], [200, 5, 3], width=2)              # a table too narrow
    check(dsix, [70, 64, 10], [5, 5, 3], spoil=(0, 1))          # a cached block that is missing
    check(dsix, [-3, 64, 10], [2, -5, 3])                       # negative lengths


def test_sums_saturate(dsix):
    big = 2 ** 30
    t = tensors([big, big, big], [1, 1, 0], [1, 2], [[1], [1], [1]], 2, 1)
    dsix.ix_plan_step(**t, block_size=2 ** 31 - 1)
    assert dsix.ix_prep_device_status() == BAD_RANGE
    assert t["cu_ctx"].tolist() == [0, big + 1, MAX, MAX] and t["context_lens"].tolist() == [big + 1, big + 1, big]
    assert t["positions"].tolist() == [big, big] and t["cu_new"].tolist() == [0, 1, 2, 2]


@pytest.mark.parametrize("shift", [2, 4])
def test_buffers_that_start_elsewhere(dsix, shift):
    """The 64-bit outputs on 16 and on 32 bytes (their stores differ), the others on 16."""
    g = torch.Generator().manual_seed(shift)
    new, cached = torch.randint(0, 90, (300,), generator=g).tolist(), torch.randint(0, 200, (300,), generator=g).tolist()
    t = check(dsix, cached, new)
    moved = dict(t)
    for name in ("slot_mapping", "positions", "row_req", "row_len", "ks", "ke"):
        n = shift if t[name].dtype is torch.int64 else 4
        moved[name] = torch.full((n + t[name].numel(),), -77, dtype=t[name].dtype, device="cuda")[n:]
    dsix.ix_plan_step(**moved)
    assert dsix.ix_prep_device_status() == 0
    assert all(torch.equal(moved[k], t[k]) for k in t)


def test_graph_and_side_stream(dsix):
    t = check(dsix, [10, 640], [3, 70])
    want = {k: v.clone() for k, v in t.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        dsix.ix_plan_step(**t, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    t["slot_mapping"].fill_(-9)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(t[k], want[k]) for k in t)
    # other lengths in the same buffers
    t["new_lens"].copy_(torch.tensor([1, 0], dtype=torch.int32))
    graph.replay()
    assert t["cu_new"].tolist() == [0, 1, 1] and t["slot_mapping"][1:].tolist() == [-1] * 72
