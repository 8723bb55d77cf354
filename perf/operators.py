"""The operators around the indexer that a step needs before its logits, and the
key norm's training passes: what they are measured on.

  plan        block tables and slot maps from request lengths (ix_plan_step)
  rope_table  the rotary table of (scaled) frequencies (ix_rope_table)
  rope        rotary positions of a part of every head, forward or backward (ix_rope)
  norm        layer norm, forward or backward (ix_layer_norm, ix_layer_norm_bwd)
  write_k     layer norm + rotary positions + fp8 write of the indexer key into the
              paged cache (ix_norm_rope_write_k)

``run`` computes a case in elementary torch operations, or, where ``own`` is true,
through the package's entry points.
"""
import math

import torch

own = False

BLOCK = 64            # keys of a cache block
DIM = 128             # the indexer key's width
ENTRY = DIM + 4       # bytes of a key: its fp8 values and its f32 scale
TINY = torch.finfo(torch.float32).tiny
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # 128 requests that decode two tokens each at 4k to 32k keys: every step of a server
        {"name": "plan_decode", "op": "plan", "requests": 128, "new_lo": 2, "new_hi": 2, "old_lo": 4096,
         "old_hi": 32768, "spare": 0},
        # a thousand prompts, some of them empty, some with a cached prefix, admitted at once
        {"name": "plan_prompts", "op": "plan", "requests": 1024, "new_lo": 0, "new_hi": 2000, "old_lo": 0,
         "old_hi": 3000, "spare": 333},
        # the table of a model whose context was stretched from 4k to 128k
        {"name": "rope_table_128k", "op": "rope_table", "positions": 131072, "first": 0, "rot": 64, "scaling": "yarn",
         "base": 10000.0, "factor": 40.0, "original": 4096, "amplitude": 1.25},
        # the indexer's queries and keys of 128 requests with two rows each, half of every head rotated
        {"name": "rope_decode", "op": "rope", "type": "bf16", "tokens": 256, "heads": 64, "heads2": 1, "dim": 128,
         "rot": 64, "offset": 0, "interleaved": False, "inverse": False, "pad": 0, "max_pos": 32768},
        # the same of an 8k prompt chunk
        {"name": "rope_prefill", "op": "rope", "type": "bf16", "tokens": 8192, "heads": 64, "heads2": 1, "dim": 128,
         "rot": 64, "offset": 0, "interleaved": False, "inverse": False, "pad": 0, "max_pos": 8192},
        # the gradient of 128 attention heads whose last 64 of 192 values are rotated in pairs, ragged batch
        {"name": "rope_backward", "op": "rope", "type": "fp16", "tokens": 2047, "heads": 128, "heads2": 0, "dim": 192,
         "rot": 64, "offset": 128, "interleaved": True, "inverse": True, "pad": 8, "max_pos": 4096},
        # the key norm of a small decode batch
        {"name": "norm_decode", "op": "norm", "type": "bf16", "rows": 32, "cols": 128, "pad": 64, "backward": False},
        # a hidden state's norm over a training batch
        {"name": "norm_hidden", "op": "norm", "type": "bf16", "rows": 8192, "cols": 4096, "pad": 0, "backward": False},
        # the key norm's gradient over a long training batch
        {"name": "norm_key_backward", "op": "norm", "type": "bf16", "rows": 131071, "cols": 128, "pad": 0,
         "backward": True},
        # a wide norm's gradient in full precision, an odd width
        {"name": "norm_odd_backward", "op": "norm", "type": "fp32", "rows": 4099, "cols": 5001, "pad": 0,
         "backward": True},
        # the new keys of 128 requests with two rows each
        {"name": "write_k_decode", "op": "write_k", "type": "bf16", "tokens": 256, "rot": 64, "offset": 0,
         "interleaved": False, "pad": 64, "max_pos": 32768, "skip": 7},
        # the new keys of a long packed prompt batch
        {"name": "write_k_prefill", "op": "write_k", "type": "bf16", "tokens": 65521, "rot": 64, "offset": 0,
         "interleaved": False, "pad": 0, "max_pos": 65536, "skip": 0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "plan", "rope_table", "rope", "rope", "rope", "norm", "norm", "norm", "write_k", "write_k"])
    if op == "plan":
        requests = _log(rng, 1, 2048)
        most = max(1, min(4000, 1000000 // requests))
        hi = rng.choice([1, 2, _log(rng, 1, most)])
        old = _log(rng, 1, 32768 if requests <= 512 else 4096)
        return {"op": op, "requests": requests, "new_lo": rng.choice([0, hi // 2, hi]), "new_hi": hi,
                "old_lo": rng.choice([0, old // 2, old]), "old_hi": old, "spare": rng.choice([0, 1, 77])}
    if op == "rope_table":
        return {"op": op, "positions": _log(rng, 1, 131072), "first": rng.choice([0, 0, rng.randrange(1 << 20)]),
                "rot": 2 * rng.randint(1, 32) if rng.random() < 0.5 else 64, "scaling": rng.choice(["none", "linear", "ntk", "yarn"]),
                "base": rng.choice([10000.0, 500000.0]), "factor": rng.choice([2.0, 8.0, 40.0]), "original": 4096,
                "amplitude": rng.choice([1.0, 1.125])}
    if op == "rope":
        kind = rng.choice(list(TYPES))
        dim = rng.choice([64, 128, 192, 256, rng.randint(2, 256)])
        rot = min(dim, rng.choice([dim // 2 * 2, max(2, dim // 4 * 2), 64]))
        heads = rng.choice([1, 8, 64, 128, rng.randint(1, 128)])
        most = max(1, min(8192, 64 * 8192 * 128 * 2 // (heads * dim * BYTES[kind]) * 9 // 10))
        rot -= rot % 2
        return {"op": op, "type": kind, "tokens": _log(rng, 1, most), "heads": heads, "heads2": rng.choice([0, 1]),
                "dim": dim, "rot": rot, "offset": rng.choice([0, dim - rot]),
                "interleaved": rng.random() < 0.5, "inverse": rng.random() < 0.4, "pad": rng.choice([0, 0, 8, 64]),
                "max_pos": _log(rng, 64, 32768)}
    if op == "norm":
        kind = rng.choice(list(TYPES))
        cols = rng.choice([128, 512, 1024, 4096, 8192, _log(rng, 2, 16384), _log(rng, 2, 16384)])
        most = max(1, min(131072, 32 * 1024 * 1024 * 2 // (cols * BYTES[kind])))
        return {"op": op, "type": kind, "rows": _log(rng, 1, most), "cols": cols, "pad": rng.choice([0, 0, 64]),
                "backward": rng.random() < 0.5}
    rot = rng.choice([16, 32, 64, 128])
    return {"op": op, "type": rng.choice(list(TYPES)), "tokens": _log(rng, 1, 65536), "rot": rot,
            "offset": rng.choice([0, DIM - rot]), "interleaved": rng.random() < 0.5, "pad": rng.choice([0, 64]),
            "max_pos": _log(rng, 64, 65536), "skip": rng.choice([0, 0, 3, 11])}


# --- inputs ----------------------------------------------------------------

def _frequencies(c):
    """Radians per position of every pair, in 64 bits: base^(-2i/rot), stretched for long contexts."""
    rot, base = c["rot"], c["base"]
    if c["scaling"] == "ntk" and rot > 2:
        base = base * c["factor"] ** (rot / (rot - 2))
    i = torch.arange(rot // 2, dtype=torch.float64)
    inv = base ** (-2.0 * i / rot)
    if c["scaling"] == "linear":
        inv = inv / c["factor"]
    if c["scaling"] == "yarn":
        def pair(turns):  # the pair that makes so many turns over the original context
            return rot * math.log(c["original"] / (2 * math.pi * turns)) / (2 * math.log(base))
        low, high = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        inv = inv * (1 - ramp) + inv / c["factor"] * ramp
    return inv


def _table(positions, rot, dev):
    """cos and sin of plain frequencies, as a program has them from its start."""
    c = {"rot": rot, "base": 10000.0, "scaling": "none"}
    a = torch.arange(positions, dtype=torch.float64, device=dev)[:, None] * _frequencies(c).to(dev)
    return torch.cat([a.cos(), a.sin()], 1).float()


def _positions(tokens, max_pos, g, dev):
    """Runs of consecutive positions, as packed prompts and decode rows have them."""
    run = torch.randint(0, max_pos, ((tokens + 255) // 256, 1), generator=g, device=dev)
    return ((run + torch.arange(256, device=dev)) % max_pos).reshape(-1)[:tokens].contiguous()


class State:
    pass


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s, op = State(), case["op"]
    s.case = case

    def normal(*shape, scale=1.0, pad=0, kind="bf16", shift=0.0):
        """Normal values; with `pad`, a slice of a wider buffer (the last dimension but one is strided)."""
        wide = list(shape)
        wide[-1] += pad
        x = torch.randn(wide, generator=g, device=dev) * scale + shift
        return x.to(TYPES[kind])[..., :shape[-1]]

    if op == "plan":
        B = case["requests"]
        # lengths spread evenly over their range, in the seed's order: their sum, the rows of the step, stays the same
        order = torch.randperm(B, generator=g, device=dev)
        new = case["new_lo"] + (2 * order + 1) * (case["new_hi"] + 1 - case["new_lo"]) // (2 * B)
        old = torch.randint(case["old_lo"], case["old_hi"] + 1, (B,), generator=g, device=dev)
        width = (case["new_hi"] + case["old_hi"] + BLOCK - 1) // BLOCK + 1
        have, need = (old + BLOCK - 1) // BLOCK, (old + new + BLOCK - 1) // BLOCK
        tokens, used, taken = int(new.sum()), int(have.sum()), int((need - have).sum())
        pool = torch.randperm(used + taken + 64, generator=g, device=dev).int()
        s.table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
        col = torch.arange(width, device=dev)
        live = col < have[:, None]
        first = have.cumsum(0) - have
        s.table = torch.where(live, pool[(first[:, None] + col).clamp(max=used + taken + 63)], s.table).contiguous()
        s.free = pool[used:].contiguous()
        s.old, s.new = old.int(), new.int()
        s.tokens = max(1, tokens + case["spare"])
        i32 = dict(dtype=torch.int32, device=dev)
        s.context_lens = torch.empty(B, **i32)
        s.cu_new, s.cu_ctx, s.cu_blocks = (torch.empty(B + 1, **i32) for _ in range(3))
        s.slots, s.positions = (torch.empty(s.tokens, dtype=torch.int64, device=dev) for _ in range(2))
        s.row_req, s.row_len, s.ks, s.ke = (torch.empty(s.tokens, **i32) for _ in range(4))
    elif op == "rope_table":
        case = dict(case, amplitude=case["amplitude"] + (seed % 97) / 4096)
        s.case = case
        s.inv = _frequencies(case).tolist()
        s.table = torch.empty(case["positions"], case["rot"], device=dev)
    elif op == "rope":
        t, h, d, kind = case["tokens"], case["heads"], case["dim"], case["type"]
        s.x = normal(t, h, d, pad=case["pad"], kind=kind)
        s.out = torch.empty(t, h, d, dtype=TYPES[kind], device=dev)
        s.x2 = s.out2 = None
        if case["heads2"]:
            s.x2 = normal(t, case["heads2"], d, pad=case["pad"], kind=kind)
            s.out2 = torch.empty(t, case["heads2"], d, dtype=TYPES[kind], device=dev)
        s.table = _table(case["max_pos"], case["rot"], dev)
        s.positions = _positions(t, case["max_pos"], g, dev)
    elif op == "norm":
        r, c, kind = case["rows"], case["cols"], case["type"]
        s.x = normal(r, c, pad=case["pad"], kind=kind, scale=1.5, shift=0.25)
        s.gamma = 1 + 0.1 * torch.randn(c, generator=g, device=dev)
        s.beta = 0.1 * torch.randn(c, generator=g, device=dev)
        s.eps = 1e-6
        s.out = torch.empty(r, c, dtype=TYPES[kind], device=dev)
        s.mean, s.rstd = torch.empty(r, device=dev), torch.empty(r, device=dev)
        if case["backward"]:
            s.dy = normal(r, c, kind=kind, scale=0.125)
            var, mean = torch.var_mean(s.x.double(), 1, correction=0)
            s.mean, s.rstd = mean.float(), (var + s.eps).rsqrt().float()
            s.dgamma, s.dbeta = torch.empty(c, device=dev), torch.empty(c, device=dev)
            s.work = None
    else:
        n = case["tokens"]
        s.k = normal(n, DIM, pad=case["pad"], kind=case["type"], scale=2.0, shift=0.125)
        s.gamma = 1 + 0.1 * torch.randn(DIM, generator=g, device=dev)
        s.beta = 0.1 * torch.randn(DIM, generator=g, device=dev)
        s.eps = 1e-6
        s.table = _table(case["max_pos"], case["rot"], dev)
        s.positions = _positions(n, case["max_pos"], g, dev)
        blocks = 2 * ((n + BLOCK - 1) // BLOCK) + 4
        # a pool that holds other requests' keys, and one block behind it that nothing reads
        codes = torch.randn(blocks + 1, BLOCK * DIM, generator=g, device=dev).to(torch.float8_e4m3fn).view(torch.uint8)
        scales = torch.rand(blocks + 1, BLOCK, generator=g, device=dev).view(torch.uint8)
        s.pool = torch.cat([codes, scales], 1)
        s.cache = s.pool[:blocks]
        order = torch.randperm(blocks, generator=g, device=dev)[:(n + BLOCK - 1) // BLOCK]
        s.slots = (order[:, None] * BLOCK + torch.arange(BLOCK, device=dev)).reshape(-1)[:n].contiguous()
        if case["skip"]:
            s.slots[::case["skip"]] = -1
    return s


# --- one pass --------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


def _planned(s):
    return {"table": s.table, "context_lens": s.context_lens, "cu_new": s.cu_new, "cu_ctx": s.cu_ctx,
            "cu_blocks": s.cu_blocks, "slots": s.slots, "positions": s.positions, "row_req": s.row_req,
            "row_len": s.row_len, "ks": s.ks, "ke": s.ke}


def _cache_values(cache):
    return {"values": cache[:, :BLOCK * DIM].view(torch.float8_e4m3fn),
            "scales": cache[:, BLOCK * DIM:].view(torch.float32)}


def _run_own(s):
    import deepseek_v3_sparse_gb300 as dsix

    c, op = s.case, s.case["op"]
    if op == "plan":
        dsix.ix_plan_step(s.old, s.new, s.free, s.table, s.context_lens, s.cu_new, s.cu_ctx, s.cu_blocks, s.slots,
                          s.positions, s.row_req, s.row_len, s.ks, s.ke)
        return _planned(s)
    if op == "rope_table":
        dsix.ix_rope_table(s.table, s.inv, first_position=c["first"], amplitude=c["amplitude"])
        return s.table
    if op == "rope":
        dsix.ix_rope(s.x, s.positions, s.table, s.out, offset=c["offset"], interleaved=c["interleaved"],
                     inverse=c["inverse"], x2=s.x2, out2=s.out2)
        return {"out": s.out, "out2": s.out2}
    if op == "norm" and not c["backward"]:
        dsix.ix_layer_norm(s.x, s.gamma, s.beta, s.eps, s.out, s.mean, s.rstd)
        return {"out": s.out, "mean": s.mean, "rstd": s.rstd}
    if op == "norm":
        if s.work is None:  # a workspace that a training loop keeps
            size = dsix.ix_layer_norm_bwd_workspace_size(c["rows"], c["cols"])
            s.work = torch.empty(size, dtype=torch.uint8, device=s.x.device)
        dsix.ix_layer_norm_bwd(s.dy, s.x, s.gamma, s.mean, s.rstd, s.out, s.dgamma, s.dbeta, s.work)
        return {"dx": s.out, "dgamma": s.dgamma, "dbeta": s.dbeta}
    dsix.ix_norm_rope_write_k(s.k, s.gamma, s.beta, s.eps, s.positions, s.table, s.slots, s.cache,
                              rope_offset=c["offset"], interleaved=c["interleaved"])
    return _cache_values(s.cache)


def _rotate(x, cos, sin, offset, interleaved):
    """Rotates the pairs of x[..., offset:offset + rot] (f32); cos and sin: [..., rot / 2]."""
    half = cos.shape[-1]
    head, part, tail = x[..., :offset], x[..., offset:offset + 2 * half], x[..., offset + 2 * half:]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = part[..., :half], part[..., half:]
        part = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([head, part, tail], -1)


def _run_plain(s):
    c, op = s.case, s.case["op"]
    if op == "plan":
        return _plan_plain(s)
    if op == "rope_table":
        at = torch.arange(c["first"], c["first"] + c["positions"], dtype=torch.float64, device=s.table.device)
        a = at[:, None] * torch.tensor(s.inv, dtype=torch.float64, device=s.table.device)
        return (torch.cat([a.cos(), a.sin()], 1) * c["amplitude"]).float()
    if op == "rope":
        row = s.table[s.positions]
        half = c["rot"] // 2
        cos, sin = row[:, None, :half], row[:, None, half:]
        sin = -sin if c["inverse"] else sin
        turned = [None if x is None else _rotate(x.float(), cos, sin, c["offset"], c["interleaved"]).to(x.dtype)
                  for x in (s.x, s.x2)]
        return {"out": turned[0], "out2": turned[1]}
    if op == "norm" and not c["backward"]:
        x = s.x.float()
        mean = x.mean(1)
        centred = x - mean[:, None]
        rstd = ((centred * centred).mean(1) + s.eps).rsqrt()
        return {"out": (centred * rstd[:, None] * s.gamma + s.beta).to(s.x.dtype), "mean": mean, "rstd": rstd}
    if op == "norm":
        dy = s.dy.float()
        xhat = (s.x.float() - s.mean[:, None]) * s.rstd[:, None]
        g = dy * s.gamma
        dx = (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)) * s.rstd[:, None]
        return {"dx": dx.to(s.x.dtype), "dgamma": (dy * xhat).sum(0), "dbeta": dy.sum(0)}
    x = s.k.float()
    centred = x - x.mean(1, keepdim=True)
    y = centred * ((centred * centred).mean(1, keepdim=True) + s.eps).rsqrt() * s.gamma + s.beta
    row, half = s.table[s.positions], c["rot"] // 2
    y = _rotate(y, row[:, :half], row[:, half:], c["offset"], c["interleaved"])
    scale = (y.abs().amax(1) / 448.0).clamp(min=TINY)
    codes = (y / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    spare = s.pool.shape[0] - 1  # where the tokens without a slot go
    block = torch.where(s.slots < 0, spare, s.slots // BLOCK)
    row = s.slots.clamp(min=0) % BLOCK
    s.pool[:, :BLOCK * DIM].view(-1, BLOCK, DIM)[block, row] = codes
    s.pool[:, BLOCK * DIM:].view(torch.float32)[block, row] = scale
    return _cache_values(s.cache)


def _plan_plain(s):
    dev = s.old.device
    B, old, new = s.old.shape[0], s.old.long(), s.new.long()
    zero = torch.zeros(1, dtype=torch.int64, device=dev)
    have, context = (old + BLOCK - 1) // BLOCK, old + new
    cu_new = torch.cat([zero, new.cumsum(0)])
    cu_ctx = torch.cat([zero, context.cumsum(0)])
    cu_blocks = torch.cat([zero, ((context + BLOCK - 1) // BLOCK - have).cumsum(0)])
    # each request's new blocks come from the free list, in the order of the requests
    col = torch.arange(s.table.shape[1], device=dev)
    take = cu_blocks[:-1, None] + col - have[:, None]
    fresh = (col >= have[:, None]) & (take < cu_blocks[1:, None])
    s.table.copy_(torch.where(fresh, s.free[take.clamp(0, s.free.shape[0] - 1)], s.table))
    # a token's request: how many requests begin at or before it
    begins = torch.zeros(s.tokens + 1, dtype=torch.int64, device=dev)
    begins.index_add_(0, cu_new[:-1].clamp(max=s.tokens), torch.ones_like(new))
    t = torch.arange(s.tokens, device=dev)
    live = t < cu_new[-1]
    req = torch.where(live, begins[:-1].cumsum(0) - 1, 0)
    pos = torch.where(live, old[req] + t - cu_new[req], 0)
    slots = torch.where(live, s.table[req, pos // BLOCK].long() * BLOCK + pos % BLOCK, -1)
    length = torch.where(live, pos + 1, 0)
    ks = torch.where(live, cu_ctx[req], 0)
    return {"table": s.table, "context_lens": context.int(), "cu_new": cu_new.int(), "cu_ctx": cu_ctx.int(),
            "cu_blocks": cu_blocks.int(), "slots": slots, "positions": pos, "row_req": req.int(),
            "row_len": length.int(), "ks": ks.int(), "ke": (ks + length).int()}


# --- what a pass cannot do without -----------------------------------------

def work(case):
    op = case["op"]
    if op == "plan":
        B, new = case["requests"], (case["new_lo"] + case["new_hi"]) / 2
        tokens = B * new + case["spare"]
        # the lengths, a table entry and a free block for each block of new tokens; 32 bytes for each token
        return {"bytes": B * (8 + 4 + 12) + 8 * B * (new / BLOCK + 1) + 32 * tokens, "flops": 0}
    if op == "rope_table":
        return {"bytes": 4 * case["positions"] * case["rot"], "flops": 8 * case["positions"] * case["rot"]}
    if op == "rope":
        values = case["tokens"] * (case["heads"] + case["heads2"])
        rows = min(case["tokens"], case["max_pos"])
        return {"bytes": 2 * values * case["dim"] * BYTES[case["type"]] + 8 * case["tokens"] + 4 * rows * case["rot"],
                "flops": 3 * values * case["rot"]}
    if op == "norm":
        r, c, b = case["rows"], case["cols"], BYTES[case["type"]]
        if case["backward"]:
            return {"bytes": 3 * r * c * b + 8 * r + 12 * c, "flops": 13 * r * c}
        return {"bytes": 2 * r * c * b + 8 * r + 8 * c, "flops": 8 * r * c}
    n = case["tokens"]
    rows = min(n, case["max_pos"])
    return {"bytes": n * (DIM * BYTES[case["type"]] + 16 + ENTRY) + 4 * rows * case["rot"] + 8 * DIM,
            "flops": n * (12 * DIM + 3 * case["rot"])}


# --- the definitions in 64 bits --------------------------------------------

def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None
    s = prepare(case, seed)
    if op == "rope_table":
        n, first = case["positions"], case["first"]
        turns = torch.outer(torch.arange(n, dtype=torch.float64, device="cuda") + first,
                            torch.as_tensor(s.inv, dtype=torch.float64, device="cuda"))
        return s.case["amplitude"] * torch.cat((torch.cos(turns), torch.sin(turns)), dim=1)
    if op == "rope":
        # a pair as a complex number, multiplied by that of its angle
        angle = torch.complex(s.table[:, :case["rot"] // 2].double(), s.table[:, case["rot"] // 2:].double())[s.positions]
        return {"out": _exact_rotation(s.x.double(), angle, case, case["inverse"]),
                "out2": None if s.x2 is None else _exact_rotation(s.x2.double(), angle, case, case["inverse"])}
    if op == "norm":
        x = s.x.double()
        if not case["backward"]:
            var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
            rstd = 1 / torch.sqrt(var + s.eps)
            return {"out": (x - mean) * rstd * s.gamma.double() + s.beta.double(), "mean": mean[:, 0], "rstd": rstd[:, 0]}
        h = (x - s.mean.double()[:, None]) * s.rstd.double()[:, None]
        dy = s.dy.double()
        g = dy * s.gamma.double()
        n = x.shape[1]
        along = (g * h).sum(1, keepdim=True) / n
        dx = s.rstd.double()[:, None] * (g - g.sum(1, keepdim=True) / n - h * along)
        return {"dx": dx, "dgamma": torch.einsum("rc,rc->c", dy, h), "dbeta": dy.sum(0)}
    x = s.k.double()
    var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
    y = (x - mean) / torch.sqrt(var + s.eps) * s.gamma.double() + s.beta.double()
    angle = torch.complex(s.table[:, :case["rot"] // 2].double(), s.table[:, case["rot"] // 2:].double())[s.positions]
    y = _exact_rotation(y[:, None], angle, case, False)[:, 0]
    scale = (y.abs().max(dim=1).values / 448).clamp_min(TINY)
    blocks = s.cache.shape[0]
    now = _cache_values(s.cache)
    values = now["values"].reshape(blocks * BLOCK, DIM).to(torch.float64)
    scales = now["scales"].reshape(blocks * BLOCK).to(torch.float64)
    kept = s.slots >= 0
    values[s.slots[kept]] = (y / scale[:, None])[kept]
    scales[s.slots[kept]] = scale[kept]
    return {"values": values.reshape(blocks, BLOCK * DIM), "scales": scales.reshape(blocks, BLOCK)}


def _exact_rotation(x, angle, case, inverse):
    lo, rot = case["offset"], case["rot"]
    part = x[..., lo:lo + rot]
    if case["interleaved"]:
        pairs = torch.view_as_complex(part.reshape(*part.shape[:-1], rot // 2, 2).contiguous())
    else:
        pairs = torch.complex(part[..., :rot // 2].contiguous(), part[..., rot // 2:].contiguous())
    pairs = pairs * (angle.conj() if inverse else angle)[:, None]
    y = x.clone()
    if case["interleaved"]:
        y[..., lo:lo + rot] = torch.view_as_real(pairs).flatten(-2)
    else:
        y[..., lo:lo + rot] = torch.cat([pairs.real, pairs.imag], -1)
    return y
