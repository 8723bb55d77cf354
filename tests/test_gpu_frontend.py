"""The front end and the calls behind it: prompts and decode steps planned on the
GPU, against the CPU oracle on the same cache and queries; the example."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle
from _helpers import check_logits_rows, check_topk_rows, require_gpu

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TOPK = 32


@pytest.fixture(scope="module")
def dsix():
    require_gpu()
    import deepseek_v3_sparse_gb300 as m
    m.load()
    m.load_prep()
    m.ix_device_status()
    m.ix_prep_device_status()
    return m


def make_front(dsix, rows, table, free, cache, max_pos=1024, interleaved=False):
    from deepseek_v3_sparse_gb300.frontend import FrontEnd
    g = torch.Generator(device="cuda").manual_seed(1)
    cos_sin = torch.empty(max_pos, 64, device="cuda")
    dsix.ix_rope_table(cos_sin, dsix.ix_rope_frequencies(64))
    return FrontEnd(rows=rows, block_table=table, free_blocks=free, cache=cache, eps=1e-6, cos_sin=cos_sin,
                    gamma=1 + 0.1 * torch.randn(128, generator=g, device="cuda"),
                    beta=0.1 * torch.randn(128, generator=g, device="cuda"), interleaved=interleaved)


def projections(rows, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    fused = torch.randn(rows, 65, 128, generator=g, device="cuda").bfloat16()  # the key beside the queries' heads
    return fused[:, 64], fused[:, :64], torch.rand(rows, 64, generator=g, device="cuda")


def test_prompts_then_decode_match_the_oracle(dsix):
    prompts, width = [130, 0, 64, 33], 4
    batch, total = len(prompts), sum(prompts)
    pool = torch.randperm(16, generator=torch.Generator().manual_seed(5)).int().cuda()
    table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    cache = torch.zeros(16, 8448, dtype=torch.uint8, device="cuda")
    lens = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    rows = total + 5  # padded: the last rows are empty
    front = make_front(dsix, rows, table, pool, cache)
    front.run(torch.zeros_like(lens), lens, *projections(rows, 2))
    assert front.cu_blocks.tolist() == [0, 3, 3, 4, 5] and front.slot_mapping[total:].tolist() == [-1] * 5
    k8, sc = torch.zeros(total, 128, dtype=torch.uint8, device="cuda"), torch.zeros(total, device="cuda")
    logits = torch.zeros(rows, 132, device="cuda")
    loc, glb = (torch.empty(rows, TOPK, dtype=torch.int32, device="cuda") for _ in range(2))
    dsix.ix_gather_k(cache, table, front.cu_ctx, k8, sc)
    dsix.ix_mqa_logits(front.q_fp8, front.w, k8, sc, front.ks, front.ke, logits)
    dsix.ix_topk_to_global(logits, front.row_len, front.row_req, table, TOPK, glb, loc)
    assert dsix.ix_device_status() == 0 and dsix.ix_prep_device_status() == 0
    row_len, row_req = front.row_len.cpu().numpy(), front.row_req.cpu().numpy()
    want = oracle.mqa_logits(front.q_fp8.cpu().numpy(), front.w.cpu().numpy(), k8.cpu().numpy(), sc.cpu().numpy(),
                             front.ks.cpu().numpy(), front.ke.cpu().numpy(), ld=132)
    bt = table.cpu().numpy()
    check_logits_rows(logits.cpu().numpy(), want, row_len, "prompt")
    live = np.flatnonzero(row_len)
    check_topk_rows(loc.cpu().numpy()[live], glb.cpu().numpy()[live], want[live], row_len[live], row_req[live], bt, 64,
                    TOPK, "prompt")
    # a decode token of every request: two of them take a block
    step = make_front(dsix, batch, table, pool[5:].contiguous(), cache)
    step.run(lens, torch.ones_like(lens), *projections(batch, 3))
    assert step.cu_blocks.tolist() == [0, 0, 1, 2, 2] and step.context_lens.tolist() == [131, 1, 65, 34]
    logits = torch.zeros(batch, 256, device="cuda")
    glb, loc = (torch.empty(batch, TOPK, dtype=torch.int32, device="cuda") for _ in range(2))
    work = torch.zeros(dsix.ix_topk_hist_workspace_size(batch), dtype=torch.uint8, device="cuda")
    dsix.ix_paged_mqa_logits_topk(step.q_fp8.view(batch, 1, 64, 128), step.w, cache, step.context_lens, table, logits,
                                  TOPK, glb, work, out_local=loc)
    assert dsix.ix_device_status() == 0 and dsix.ix_prep_device_status() == 0
    bt, ctx = table.cpu().numpy(), step.context_lens.cpu().numpy()
    want = oracle.paged_mqa_logits(step.q_fp8.cpu().numpy().reshape(batch, 1, 64, 128), step.w.cpu().numpy(),
                                   cache.cpu().numpy(), 64, ctx, np.maximum(bt, 0), ld=256)
    check_logits_rows(logits.cpu().numpy(), want, ctx, "decode")
    check_topk_rows(loc.cpu().numpy(), glb.cpu().numpy(), want, ctx, np.arange(batch), bt, 64, TOPK, "decode")


def test_a_prompt_in_one_step_or_token_by_token(dsix):
    """The cache, the queries and the weights do not depend on how a prompt is cut into steps."""
    n = 70
    k, q, w = projections(n, 4)
    results = []
    for cuts in ([n], [1] * n, [30, 34, 6]):
        table = torch.full((1, 2), -1, dtype=torch.int32, device="cuda")
        cache = torch.zeros(4, 8448, dtype=torch.uint8, device="cuda")
        at, q8, ws, free = 0, [], [], torch.tensor([2, 0], dtype=torch.int32, device="cuda")
        for c in cuts:
            taken = (at + 63) // 64
            front = make_front(dsix, c, table, free[taken:].contiguous(), cache, interleaved=True)
            i32 = lambda v: torch.tensor([v], dtype=torch.int32, device="cuda")  # noqa: E731
            front.run(i32(at), i32(c), k[at:at + c], q[at:at + c], w[at:at + c])
            q8.append(front.q_fp8)
            ws.append(front.w)
            at += c
        results.append((cache, torch.cat(q8), torch.cat(ws), table))
    assert dsix.ix_prep_device_status() == 0
    for other in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))


def test_example(dsix):
    spec = importlib.util.spec_from_file_location("serve_and_train", os.path.join(ROOT, "examples", "serve_and_train.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    chosen, counts = example.serve()
    assert counts == [370, 70, 199] and [int((r >= 0).sum()) for r in chosen] == [64, 64, 64]
    losses = example.train()
    assert losses[-1] < 0.5 * losses[0] and all(b < a for a, b in zip(losses, losses[1:]))
