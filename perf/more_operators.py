"""Long contexts over pages: page tables from request lengths, rotary positions of several axes, and attention over the
blocks of tokens that a cheap score selects. The cases these operators are measured on, their plain forms in
elementary torch operations, and their values in 64 bits.

kinds of case
  pages   pages_update: sequences grow (pages from a stack of free ones, slots of the new tokens) and shrink again
  turn    rope_apply_axes: q (or k) rows turned by positions of several axes (time, height, width)
  store   kv_append_axes: k turned and v appended at their slots of a paged cache, q turned on the way
  bounds  kv_block_bounds: the largest and smallest value of every column of the keys, for each block of tokens, in 8 bits
  select  block_select: the blocks a query attends to, by the bounds' score
  attend  decode_blocks: attention of new tokens over the listed blocks

Bounds (`codes` int8 [n, blocks, Hkv, 2, D], `scales` float32 [n, blocks, Hkv]) of a block's keys: a = max |k|, scale =
a / 127, codes[0] = ceil(max_t k / scale), codes[1] = floor(min_t k / scale), in [-127, 127]. A query row's codes are
round(q / (max |q| / 127)); a block's score for it is the sum over columns of code * codes[0] where code > 0, else
code * codes[1], times the row's scale; a KV head takes the largest over its group, times the block's scale.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a check of 5 drafted tokens for every sequence of a batch, taken back again
        {"name": "pages_draft", "kind": "pages", "B": 64, "page": 16, "blocks": 160, "held": 2400, "grow": 5, "fixed": True, "short": 0.0},
        # ragged prompts admitted and released, a few more than the pool holds
        {"name": "pages_prompts", "kind": "pages", "B": 256, "page": 64, "blocks": 65, "held": 0, "grow": 4096, "fixed": False, "short": 0.1},
        # the image patches of a vision tower, a third of the pairs to each axis, fp32 rows of 80 columns
        {"name": "turn_image", "kind": "turn", "tokens": 1031, "heads": 16, "D": 80, "sections": "8 16 16", "order": "blocks",
         "per_axis": True, "interleaved": True, "base": 10000.0, "factor": 1.0, "start": 0, "dtype": "f32"},
        # a long video's queries
        {"name": "turn_video", "kind": "turn", "tokens": 65536, "heads": 32, "D": 128, "sections": "16 24 24", "order": "blocks",
         "per_axis": False, "interleaved": False, "base": 1000000.0, "factor": 1.0, "start": 1200, "dtype": "bf16"},
        # the step of a grouped-query layer behind images: text positions far below the cache's
        {"name": "store_step", "kind": "store", "tokens": 64, "Hq": 32, "Hkv": 8, "D": 128, "sections": "16 24 24", "order": "blocks",
         "per_axis": False, "interleaved": False, "base": 1000000.0, "factor": 1.0, "start": 700, "page": 16, "pages": 8192, "live": 1.0},
        # packed prompts of text and video in a buffer with unused rows at its end, the axes' pairs dealt in turn
        {"name": "store_video", "kind": "store", "tokens": 50021, "Hq": 32, "Hkv": 8, "D": 128, "sections": "24 20 20",
         "order": "dealt", "per_axis": False, "interleaved": False, "base": 500000.0, "factor": 4.0, "start": 60000, "page": 64,
         "pages": 1024, "live": 0.9},
        # a chunk of 512 prompt tokens for each of 8 sequences
        {"name": "bounds_chunk", "kind": "bounds", "B": 8, "Hkv": 8, "D": 128, "block": 64, "page": 64, "held": 30000, "new": 512},
        # the caches of whole prompts
        {"name": "bounds_prompts", "kind": "bounds", "B": 32, "Hkv": 8, "D": 128, "block": 64, "page": 0, "held": 0, "new": 8192},
        # one sequence of 131,072 tokens
        {"name": "select_one", "kind": "select", "B": 1, "T": 1, "Hq": 32, "Hkv": 8, "D": 128, "block": 64, "page": 64, "K": 64,
         "lo": 131072, "hi": 131072, "first": 1, "last": 2},
        # a batch of long sequences in small blocks
        {"name": "select_batch", "kind": "select", "B": 32, "T": 1, "Hq": 32, "Hkv": 8, "D": 128, "block": 32, "page": 64, "K": 128,
         "lo": 16384, "hi": 131072, "first": 1, "last": 4},
        # one sequence's step
        {"name": "attend_one", "kind": "attend", "B": 1, "T": 1, "Hq": 32, "Hkv": 8, "D": 128, "block": 64, "page": 64, "K": 32,
         "lo": 65536, "hi": 65536},
        # a batch's step: 4,096 of 16,384 tokens
        {"name": "attend_batch", "kind": "attend", "B": 64, "T": 1, "Hq": 32, "Hkv": 8, "D": 128, "block": 64, "page": 64, "K": 64,
         "lo": 8192, "hi": 16384},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _draw_axes(rng, c):
    half = rng.choice([c["D"] // 2, c["D"] // 2, c["D"] // 32 * 8])
    n = rng.choice([1, 2, 3, 3, 4])
    c["per_axis"] = rng.random() < 0.4
    if c["per_axis"]:  # each axis a multiple of 8 pairs
        n = min(n, half // 8)
        cuts = sorted(rng.sample(range(1, half // 8), n - 1))
        sizes = [8 * (b - a) for a, b in zip([0] + cuts, cuts + [half // 8])]
    else:
        cuts = sorted(rng.sample(range(1, half), n - 1))
        sizes = [b - a for a, b in zip([0] + cuts, cuts + [half])]
    c["sections"] = " ".join(map(str, sizes))
    c["order"] = rng.choice(["blocks", "dealt"])
    c["interleaved"] = rng.random() < 0.4
    c["base"] = rng.choice([10000.0, 500000.0, 1000000.0])
    c["factor"] = rng.choice([1.0, 1.0, 4.0])
    c["start"] = _log_int(rng, 1, 1 << 20) - 1


def draw(rng):
    kind = rng.choice(["pages", "turn", "store", "bounds", "select", "attend"])
    c = {"kind": kind}
    if kind == "pages":
        c["B"] = _log_int(rng, 1, 256)
        c["page"] = rng.choice([16, 32, 64, 128])
        c["fixed"] = rng.random() < 0.5
        c["grow"] = _log_int(rng, 1, 64 if c["fixed"] else 4096)
        c["held"] = _log_int(rng, 1, 4096) - 1
        c["blocks"] = -(-(c["held"] + c["grow"]) // c["page"]) + rng.randint(0, 3)
        c["short"] = rng.choice([0.0, 0.0, 0.2, 0.9])
    elif kind == "turn":
        c["D"] = rng.choice([64, 80, 128, 256])
        c["heads"] = rng.choice([1, 8, 16, 32, rng.randint(1, 48)])
        c["tokens"] = _log_int(rng, 1, 65536 * 32 * 128 // (c["heads"] * c["D"]) // 2)
        _draw_axes(rng, c)
        c["dtype"] = rng.choice(["bf16", "f32"])
    elif kind == "store":
        c["D"] = rng.choice([64, 128, 256])
        c["Hkv"] = rng.choice([1, 4, 8, rng.randint(1, 40)])
        c["Hq"] = c["Hkv"] * rng.choice([1, 2, 4, 8])
        c["tokens"] = _log_int(rng, 1, 50021 * 48 * 128 // ((c["Hq"] + 2 * c["Hkv"]) * c["D"]))
        _draw_axes(rng, c)
        c["page"] = rng.choice([16, 32, 64, 128])
        c["pages"] = -(-c["tokens"] // c["page"]) + rng.randint(1, 40)
        c["live"] = rng.choice([1.0, 1.0, 0.9, 0.3])
    elif kind == "bounds":
        c["D"] = rng.choice([64, 128, 256])
        c["Hkv"] = rng.choice([1, 4, 8, rng.randint(1, 40)])
        c["block"] = rng.choice([16, 32, 64, 128])
        c["page"] = rng.choice([0, c["block"], 128])
        c["new"] = _log_int(rng, 1, 8192)
        c["held"] = rng.choice([0, _log_int(rng, 1, 8192)])
        most = 32 * 8 * 8192 * 128 // (c["Hkv"] * c["D"] * (c["new"] + c["held"]))
        c["B"] = _log_int(rng, 1, max(1, min(64, most)))
    else:
        c["T"] = rng.choice([1, 1, 1, rng.randint(2, 8)])
        c["D"] = rng.choice([64, 128, 256])
        c["Hkv"] = rng.choice([1, 2, 8, rng.randint(1, 16)])
        c["Hq"] = c["Hkv"] * rng.choice([1, 4, 8, rng.randint(1, 48)])
        c["block"] = rng.choice([16, 32, 64, 128])
        c["page"] = rng.choice([0, c["block"], 128])
        wide = max(1, c["T"] * c["Hq"] // c["Hkv"] // 8)
        if kind == "select":
            c["first"], c["last"] = rng.randint(0, 2), rng.randint(1, 4)
            c["K"] = c["first"] + c["last"] + _log_int(rng, 1, 250)
            c["hi"] = _log_int(rng, c["T"], min(16384 * c["block"], 1 << 20))
            most = 32 * 8 * 2048 * 128 // (c["Hkv"] * -(-c["hi"] // c["block"]) * c["D"] * wide)
        else:
            c["K"] = _log_int(rng, 1, 256)
            c["hi"] = _log_int(rng, c["T"], 65536)
            most = 64 * 8 * 4096 * 128 // (c["Hkv"] * c["T"] * min(c["hi"], c["K"] * c["block"]) * c["D"] * wide)
            most = min(most, 64 * 8 * 16384 * 128 // (c["Hkv"] * c["hi"] * c["D"]))
        c["lo"] = max(1, int(c["hi"] * rng.choice([0.0, 0.25, 1.0])))
        c["B"] = _log_int(rng, 1, max(1, min(128, most)))
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2 + 1)
    return g


def _randint(lo, hi, shape, g):
    """Whole numbers lo .. hi."""
    return torch.randint(lo, hi + 1, shape, generator=g, device=DEV)


def _sections(c):
    """Pairs of each axis."""
    return [int(n) for n in c["sections"].split()]


def _axis_of_pairs(c):
    """The axis that each pair's position comes from."""
    left = _sections(c)
    if c["order"] == "blocks":
        return [a for a, n in enumerate(left) for _ in range(n)]
    out, a = [], 0
    while sum(left):
        if left[a]:
            out.append(a)
            left[a] -= 1
        a = (a + 1) % len(left)
    return out


def _frequencies(c):
    """Radians a position of each pair: of its place among all pairs, or among its axis' own."""
    axes, sizes = _axis_of_pairs(c), _sections(c)
    seen, w = [0] * len(sizes), []
    for i, a in enumerate(axes):
        share = seen[a] / sizes[a] if c["per_axis"] else i / len(axes)
        seen[a] += 1
        w.append(c["base"] ** -share / c["factor"])
    return w


def _grid_positions(c, n, g):
    """[axes, n]: stretches of text, whose axes agree, and of frames, rows and columns, from `start` on."""
    A = len(_sections(c))
    i = torch.arange(n, device=DEV)
    side = 24
    grid = torch.stack([i // (side * side), i // side % side, i % side, i % 7])[:A]
    text = (i // 512) % 3 == 0
    return (c["start"] + torch.where(text, i // 9, grid)).int().contiguous()


def _table(pages, B, nb, g):
    return torch.randperm(pages, generator=g, device=DEV)[:B * nb].view(B, nb).int()


def _rows(shape, g):
    """Key or value rows: normal draws, one row in a hundred eight times as large."""
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    big = torch.rand(shape[:-1] + (1,), generator=g, device=DEV) < 0.01
    return torch.where(big, 8 * x, x)


def prepare(case, seed):
    g = _gen(seed)
    c, st = case, {"case": case}
    kind = c["kind"]
    if kind == "pages":
        B, P, nb = c["B"], c["page"], c["blocks"]
        lens = _randint(0, c["held"], (B,), g)
        grow = torch.full((B,), c["grow"], device=DEV) if c["fixed"] else _randint(1, c["grow"], (B,), g)
        st["lens"], st["want"] = lens.int(), (lens + grow).int()
        st["back"] = st["lens"].clone()
        held, need = ((x + P - 1) // P for x in (lens, lens + grow))
        pages = B * nb + 7
        perm = torch.randperm(pages, generator=g, device=DEV).int()
        j = torch.arange(nb, device=DEV)
        mine = j < held[:, None]
        st["table"] = torch.where(mine, perm[:B * nb].view(B, nb), -1)
        # the free pages on the stack, as many as are wanted or a share fewer; the places above them hold old numbers
        used = torch.cat([mine.flatten(), torch.zeros(7, dtype=torch.bool, device=DEV)])
        st["free"] = perm[torch.sort(used.int(), stable=True).indices].contiguous()
        wanted = int((need - held).sum())
        st["count"] = torch.tensor([wanted - int(wanted * c["short"])], device=DEV, dtype=torch.int32)
        n = B * c["grow"]
        st["pos"], st["offsets"] = torch.zeros(B, device=DEV, dtype=torch.int32), torch.zeros(B + 1, device=DEV, dtype=torch.int32)
        st["slots"], st["positions"] = (torch.zeros(n, device=DEV, dtype=torch.int32) for _ in range(2))
    elif kind == "turn":
        N, H, D = c["tokens"], c["heads"], c["D"]
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        st["x"] = torch.randn(N, H, D, generator=g, device=DEV, dtype=dt)
        st["positions"] = _grid_positions(c, N, g)
        st["out"] = torch.empty_like(st["x"])
    elif kind == "store":
        N, Hq, Hkv, D = c["tokens"], c["Hq"], c["Hkv"], c["D"]
        qkv = torch.randn(N, (Hq + 2 * Hkv) * D, generator=g, device=DEV, dtype=torch.bfloat16)  # one fused projection's rows
        st["q"] = qkv[:, :Hq * D].view(N, Hq, D)
        st["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(N, Hkv, D)
        st["v"] = qkv[:, (Hq + Hkv) * D:].view(N, Hkv, D)
        st["positions"] = _grid_positions(c, N, g)
        # tokens in order through pages in no order, the buffer's unused rows without a slot
        order = torch.randperm(c["pages"], generator=g, device=DEV)
        i = torch.arange(N, device=DEV)
        slots = order[i // c["page"]] * c["page"] + i % c["page"]
        st["slots"] = torch.where(i < max(1, int(N * c["live"])), slots, -1).int()
        st["q_out"] = torch.zeros(N, Hq, D, device=DEV, dtype=torch.bfloat16)
        st["kp"] = torch.zeros(c["pages"], c["page"], Hkv, D, device=DEV, dtype=torch.bfloat16)
        st["vp"] = torch.zeros_like(st["kp"])
    elif kind == "bounds":
        B, Hkv, D, blk = c["B"], c["Hkv"], c["D"], c["block"]
        st["from"] = _randint(c["held"] // 2, c["held"], (B,), g).int()
        st["lens"] = st["from"] + c["new"]
        step = c["page"] or blk
        S = -(-(c["held"] + c["new"]) // step) * step
        st["table"] = None
        n = B
        if c["page"]:
            n = B * (S // step) + 3
            st["table"] = _table(n, B, S // step, g)
            st["k"] = _rows((n, step, Hkv, D), g)
        else:
            st["k"] = _rows((B, S, Hkv, D), g)
        st["S"] = S
        st["codes"] = torch.zeros(n, (step if c["page"] else S) // blk, Hkv, 2, D, device=DEV, dtype=torch.int8)
        st["scales"] = torch.zeros(st["codes"].shape[:3], device=DEV)
    else:
        B, T, Hq, Hkv, D, blk = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["block"]
        st["lens"] = _randint(c["lo"], c["hi"], (B,), g).int()
        st["q"] = torch.randn(B, T, Hq, D, generator=g, device=DEV, dtype=torch.bfloat16)
        step = c["page"] or blk
        S = st["S"] = -(-c["hi"] // step) * step
        st["table"], n, per = None, B, S
        if c["page"]:
            n, per = B * (S // step) + 3, step
            st["table"] = _table(n, B, S // step, g)
        if kind == "select":
            # columns' extremes over a block, as shares of the block's largest value
            shape = (n, per // blk, Hkv, 2, D)
            x = 40 + 87 * torch.rand(shape, generator=g, device=DEV)
            x[..., 1, :] *= -1
            st["codes"] = x.round().to(torch.int8)
            st["scales"] = (0.015 + 0.015 * torch.rand(shape[:3], generator=g, device=DEV)).contiguous()
            st["blocks"] = torch.empty(B, T, Hkv, c["K"], device=DEV, dtype=torch.int32)
        else:
            st["k"], st["v"] = (_rows((n, per, Hkv, D), g) for _ in range(2))
            # every query token's last block and others before it, in order; -1 where there are fewer
            nb = S // blk
            seen = st["lens"].long().view(B, 1) - T + 1 + torch.arange(T, device=DEV)
            have = ((seen + blk - 1) // blk).clamp_min(0).view(B, T, 1, 1)
            j = torch.arange(nb, device=DEV)
            r = torch.rand(B, T, Hkv, nb, generator=g, device=DEV)
            r = torch.where(j < have, torch.where(j == have - 1, 2.0, r), -1.0)
            top = r.topk(min(c["K"], nb), -1)
            pick = torch.where(top.values < 0, nb, top.indices).sort(-1).values
            pick = torch.where(pick == nb, -1, pick)
            if c["K"] > nb:
                pick = torch.cat([pick, torch.full((B, T, Hkv, c["K"] - nb), -1, device=DEV)], -1)
            st["blocks"] = pick.int().contiguous()
            st["out"] = torch.empty_like(st["q"])
            st["lse"] = torch.empty(B, T, Hq, device=DEV)
    if own:  # what a program that uses the framework keeps beside its tensors
        import kv_cache_decode_gb300 as kvd
        if kind in ("turn", "store"):
            st["rope"] = kvd.RopeAxes(_sections(c), base=c["base"], order=c["order"], per_axis=c["per_axis"],
                                      scaling="linear" if c["factor"] > 1 else "none", factor=c["factor"],
                                      interleaved=c["interleaved"], device=DEV)
        if kind in ("select", "attend"):
            n = (kvd.block_select_plan(c["B"], c["T"], c["Hkv"], st["S"], c["block"]) if kind == "select" else
                 kvd.decode_blocks_plan(c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["K"], c["block"]))
            st["ws"] = torch.empty(max(n, 1), device=DEV, dtype=torch.uint8)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _resize(st, want, outputs):
    """Every sequence from its length to `want`: pages back to the stack and from it, in order of sequence and block."""
    c = st["case"]
    P, nb = c["page"], c["blocks"]
    old, want = st["lens"].long(), want.long()
    j = torch.arange(nb, device=DEV)
    ob, wb = (old + P - 1) // P, (want + P - 1) // P
    F = st["count"].long()
    gone = (j >= wb[:, None]) & (j < ob[:, None])
    R = gone.sum()
    r = gone.flatten().cumsum(0) - 1
    pages = st["free"].numel()
    stack = torch.cat([st["free"], st["free"][:1]])  # a place for what goes nowhere
    stack.scatter_(0, torch.where(gone.flatten(), F + R - 1 - r, pages), st["table"].flatten())
    F = F + R
    need = (wb - ob).clamp_min(0)
    given = (need == 0) | (need.cumsum(0) <= F)
    new = torch.where(given, want, old)
    more = (j >= ob[:, None]) & (j < ((new + P - 1) // P)[:, None])
    i = (more.flatten().cumsum(0) - 1).view_as(more)
    table = torch.where(more, stack[(F - 1 - i).clamp(0, pages - 1)], torch.where(gone, -1, st["table"]))
    st["free"].copy_(stack[:-1])
    st["count"].copy_(F - more.sum())
    st["table"].copy_(table)
    st["lens"].copy_(new)
    if outputs:
        st["pos"].copy_(old)
        ends = (new - old).clamp_min(0).cumsum(0)
        st["offsets"][1:].copy_(ends)
        n = torch.arange(st["slots"].numel(), device=DEV)
        b = torch.searchsorted(ends, n, right=True).clamp_max(c["B"] - 1)
        t = old[b] + n - st["offsets"].long()[b]
        live = n < ends[-1]
        page = table[b, (t // P).clamp(0, nb - 1)].long()
        st["slots"].copy_(torch.where(live, page * P + t % P, -1))
        st["positions"].copy_(torch.where(live, t, -1))


def _turned(c, x, positions):
    """Rows x [N, H, D] turned by positions [axes, N]: angles in 64 bits, the rotation in 32, rounded once."""
    axes = torch.tensor(_axis_of_pairs(c), device=x.device)
    w = torch.tensor(_frequencies(c), dtype=torch.float64, device=x.device)
    angle = positions.double()[axes].T * w
    cos, sin = (t.float().unsqueeze(1) for t in (angle.cos(), angle.sin()))
    R = 2 * axes.numel()
    r, rest = x[..., :R].float(), x[..., R:]
    if c["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :R // 2], r[..., R // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y.to(x.dtype), rest], -1)


def _bounds(st):
    """The bounds of the blocks that are full now and were not, in place."""
    c = st["case"]
    B, Hkv, D, blk = c["B"], c["Hkv"], c["D"], c["block"]
    nb = st["S"] // blk
    if st["table"] is None:
        k = st["k"].view(B, nb, blk, Hkv, D)
        where = torch.arange(B * nb, device=DEV).view(B, nb)
    else:
        per = c["page"] // blk
        where = (st["table"].long().unsqueeze(-1) * per + torch.arange(per, device=DEV)).view(B, nb)
        k = st["k"].view(-1, blk, Hkv, D)[where]
    k = k.float()
    hi, lo = k.amax(2), k.amin(2)                                  # [B, nb, Hkv, D]
    a = torch.maximum(hi.abs(), lo.abs()).amax(-1, keepdim=True)
    s = a / torch.full_like(a, 127.0)  # (a division by a Python number would multiply by its rounded reciprocal)
    one = torch.where(s > 0, s, 1.0)
    codes = torch.stack([(hi / one).ceil(), (lo / one).floor()], -2).clamp(-127, 127)
    end = (torch.arange(nb, device=DEV) + 1) * blk
    fresh = (end <= st["lens"].view(B, 1)) & (end > st["from"].view(B, 1))
    flat, scales = st["codes"].view(-1, Hkv, 2, D), st["scales"].view(-1, Hkv)
    flat[where] = torch.where(fresh.view(B, nb, 1, 1, 1), codes.to(torch.int8), flat[where])
    scales[where] = torch.where(fresh.view(B, nb, 1), s[..., 0], scales[where])


def _select(st):
    c = st["case"]
    B, T, Hq, Hkv, D, blk, K = (c[n] for n in ("B", "T", "Hq", "Hkv", "D", "block", "K"))
    nb = st["S"] // blk
    if st["table"] is None:
        codes, scales = st["codes"], st["scales"]
    else:
        codes, scales = (x[st["table"].long()].view((B, nb) + x.shape[2:]) for x in (st["codes"], st["scales"]))
    q = st["q"].float()
    sq = q.abs().amax(-1, keepdim=True)
    sq = sq / torch.full_like(sq, 127.0)
    qc = (q / torch.where(sq > 0, sq, 1.0)).round()
    both = torch.cat([qc.clamp_min(0), qc.clamp_max(0)], -1).view(B, T, Hkv, Hq // Hkv, 2 * D)
    both = both.permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, 2 * D)
    s = torch.matmul(both, codes.flatten(-2).float().permute(0, 2, 3, 1))  # whole numbers below 2^24: exact
    s = s.view(B, Hkv, T, Hq // Hkv, nb) * sq.view(B, T, Hkv, -1, 1).transpose(1, 2)
    s = (s.amax(3) * scales.permute(0, 2, 1).unsqueeze(2)).transpose(1, 2)  # [B, T, Hkv, nb]
    seen = (st["lens"].long().view(B, 1) - T + 1 + torch.arange(T, device=DEV)).clamp_min(0)
    have = ((seen + blk - 1) // blk).view(B, T, 1, 1)
    j = torch.arange(nb, device=DEV)
    s = torch.where((j < c["first"]) | (j >= have - c["last"]), math.inf, s)
    s = torch.where(j < have, s, -math.inf)
    k = min(K, nb)
    pick = s.sort(dim=-1, descending=True, stable=True).indices[..., :k]
    pick = torch.where(torch.arange(k, device=DEV) < have, pick, nb).sort(-1).values
    st["blocks"].fill_(-1)
    st["blocks"][..., :k] = torch.where(pick == nb, -1, pick)


def _tokens(st):
    """(rows of the flat cache [B, T, Hkv, K * block], which of them count) of the listed blocks."""
    c = st["case"]
    B, T, blk = c["B"], c["T"], c["block"]
    t = (st["blocks"].long().unsqueeze(-1) * blk + torch.arange(blk, device=DEV)).flatten(-2)
    seen = (st["lens"].long().view(B, 1) - T + 1 + torch.arange(T, device=DEV)).view(B, T, 1, 1)
    live = (t >= 0) & (t < seen)
    t = torch.where(live, t, 0)
    b = torch.arange(B, device=DEV).view(B, 1, 1, 1)
    if st["table"] is None:
        return b * st["S"] + t, live
    return st["table"].long()[b, t // c["page"]] * c["page"] + t % c["page"], live


def _attend(st):
    c = st["case"]
    B, T, Hq, Hkv, D = (c[n] for n in ("B", "T", "Hq", "Hkv", "D"))
    row, live = _tokens(st)
    h = torch.arange(Hkv, device=DEV).view(1, 1, Hkv, 1)
    k = st["k"].view(-1, Hkv, D)[row, h].float()
    s = torch.matmul(st["q"].float().view(B, T, Hkv, -1, D), k.transpose(-1, -2)) * (D ** -0.5)
    del k
    s = s.masked_fill(~live.unsqueeze(-2), -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    v = st["v"].view(-1, Hkv, D)[row, h].float()
    o = torch.matmul(p, v) / torch.where(l > 0, l, torch.ones_like(l))
    return o.view(B, T, Hq, D).bfloat16(), (m + torch.log(l)).view(B, T, Hq)


def run(st):
    c = st["case"]
    kind = c["kind"]
    if own:
        import kv_cache_decode_gb300 as kvd
        if kind == "pages":
            kvd.pages_update(st["table"], st["free"], st["count"], st["lens"], st["want"], c["page"], pos=st["pos"],
                             row_offsets=st["offsets"], slots=st["slots"], positions=st["positions"])
            kvd.pages_update(st["table"], st["free"], st["count"], st["lens"], st["back"], c["page"])
        elif kind == "turn":
            kvd.rope_apply_axes(st["rope"], st["x"], st["positions"], st["out"])
        elif kind == "store":
            kvd.kv_append_axes(st["rope"], st["kp"], st["vp"], st["k"], st["v"], st["slots"], st["positions"], q=st["q"],
                               q_out=st["q_out"])
        elif kind == "bounds":
            kvd.kv_block_bounds(st["k"], st["codes"], st["scales"], st["lens"], c["new"], c["block"], from_lens=st["from"],
                                block_table=st["table"])
        elif kind == "select":
            kvd.block_select(st["q"], st["codes"], st["scales"], st["lens"], st["S"], c["block"], st["blocks"], n_first=c["first"],
                             n_last=c["last"], block_table=st["table"], workspace=st["ws"])
        else:
            kvd.decode_blocks(st["q"], st["k"], st["v"], st["blocks"], st["lens"], c["block"], c["D"] ** -0.5, st["out"],
                              block_table=st["table"], workspace=st["ws"], lse=st["lse"])
    elif kind == "pages":
        _resize(st, st["want"], True)
        _resize(st, st["back"], False)
    elif kind == "turn":
        st["out"] = _turned(c, st["x"], st["positions"])
    elif kind == "store":
        st["q_out"].copy_(_turned(c, st["q"], st["positions"]))
        # rows without a slot go to a place that is dropped
        for name, new in (("kp", _turned(c, st["k"], st["positions"])), ("vp", st["v"])):
            flat = st[name].view(-1, c["Hkv"], c["D"])
            room = torch.cat([flat, flat[:1]])
            room[torch.where(st["slots"] < 0, flat.shape[0], st["slots"].long())] = new
            flat.copy_(room[:-1])
    elif kind == "bounds":
        _bounds(st)
    elif kind == "select":
        _select(st)
    else:
        st["out"], st["lse"] = _attend(st)
    if kind == "pages":
        return [st[n] for n in ("slots", "positions", "offsets", "pos", "lens", "table", "free", "count")]
    if kind == "turn":
        return st["out"]
    if kind == "store":
        return st["q_out"], st["kp"], st["vp"]
    if kind == "bounds":  # the values that the codes stand for
        return st["codes"] * st["scales"][..., None, None], st["scales"]
    if kind == "select":
        return st["blocks"]
    return st["out"], st["lse"]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c, kind = case, case["kind"]
    if kind == "pages":  # lengths in and out of both calls; pages, table entries and slots of the new tokens
        rows = c["B"] * (c["grow"] if c["fixed"] else (1 + c["grow"]) / 2) * (1 - c["short"])
        pages = rows / c["page"] + (c["B"] / 2 if c["held"] else 0)
        return {"bytes": 2 * c["B"] * 12 + c["B"] * 8 + 8 * rows + 2 * 8 * pages, "flops": 8 * rows}
    D = c["D"]
    if kind in ("turn", "store"):
        R, A = 2 * sum(_sections(c)), len(_sections(c))
        if kind == "turn":
            n = c["tokens"] * c["heads"] * D
            return {"bytes": 2 * n * (2 if c["dtype"] == "bf16" else 4) + 4 * A * c["tokens"], "flops": 3 * n * R / D}
        n = c["tokens"] * (c["Hq"] + c["live"] * 2 * c["Hkv"]) * D
        return {"bytes": 4 * n + c["tokens"] * 4 * (A + 1), "flops": 3 * c["tokens"] * (c["Hq"] + c["live"] * c["Hkv"]) * R}
    if kind == "bounds":
        blocks = c["B"] * c["Hkv"] * c["new"] / c["block"]
        return {"bytes": blocks * (c["block"] * D * 2 + 2 * D + 4), "flops": blocks * c["block"] * D * 2}
    tokens = c["B"] * c["T"] * (c["lo"] + c["hi"]) / 2
    if kind == "select":
        n = tokens * c["Hkv"] / c["block"]
        return {"bytes": n / c["T"] * (2 * D + 4) + c["B"] * c["T"] * (c["Hq"] * D * 2 + c["Hkv"] * c["K"] * 4),
                "flops": n * c["Hq"] / c["Hkv"] * 4 * D}
    n = min(tokens, c["B"] * c["T"] * c["K"] * c["block"])
    return {"bytes": n * c["Hkv"] * 4 * D + c["B"] * c["T"] * (c["Hq"] * (4 * D + 4) + c["Hkv"] * c["K"] * 4),
            "flops": n * c["Hq"] * D * 4}


# ---------------------------------------------------------------------------
# values in 64 bits
# ---------------------------------------------------------------------------

def _spin(case, x, positions):
    """Rows x [N, H, D], in float64, as complex pairs times exp(i angle); positions [axes, N]."""
    sections = [int(n) for n in case["sections"].split()]
    half = sum(sections)
    axis = np.repeat(np.arange(len(sections)), sections)
    if case["order"] == "dealt":  # pairs sorted by their number within the axis, then by axis
        axis = axis[np.lexsort((axis, np.concatenate([np.arange(n) for n in sections])))]
    place = np.arange(half) / half
    if case["per_axis"]:
        for a, n in enumerate(sections):
            place[axis == a] = np.arange(n) / n
    w = np.exp(-np.log(case["base"]) * place) / case["factor"]
    y = x.double()
    R = 2 * half
    for at in range(0, len(x), 8192):
        part = y[at:at + 8192]
        angle = positions[:, at:at + 8192].cpu().numpy().astype(np.float64)[axis].T * w
        turn = torch.from_numpy(np.exp(1j * angle)).to(x.device).unsqueeze(1)
        a, b = (part[..., 0:R:2], part[..., 1:R:2]) if case["interleaved"] else (part[..., :half], part[..., half:R])
        z = torch.complex(a.contiguous(), b.contiguous()) * turn
        a.copy_(z.real)
        b.copy_(z.imag)
    return y


def _exact_pages(case, st):
    P = case["page"]
    lens, table = st["lens"].tolist(), st["table"].tolist()
    buffer, F = st["free"].tolist(), int(st["count"])
    slots, positions = ([-1] * st["slots"].numel() for _ in range(2))
    offsets, first = [0], list(lens)
    starts = list(lens)
    denied = False
    for b, want in enumerate(st["want"].tolist()):  # growth: from the top of the stack, until one does not fit
        have, need = -(-lens[b] // P), -(-want // P) - -(-lens[b] // P)
        n = 0
        if need == 0 or (not denied and need <= F):
            for j in range(have, have + need):
                F -= 1
                table[b][j] = buffer[F]
            n, lens[b] = want - lens[b], want
        else:
            denied = True
        for i in range(n):
            t = starts[b] + i
            slots[offsets[-1] + i] = table[b][t // P] * P + t % P
            positions[offsets[-1] + i] = t
        offsets.append(offsets[-1] + n)
    gone = []
    for b, want in enumerate(st["back"].tolist()):  # and back: the first released page ends on top
        for j in range(-(-want // P), -(-lens[b] // P)):
            gone.append(table[b][j])
            table[b][j] = -1
        lens[b] = want
    for page in reversed(gone):
        buffer[F] = page
        F += 1
    return [np.array(x) for x in (slots, positions, offsets, first, lens, table, buffer, [F])]


def exact(case, seed):
    c, kind = case, case["kind"]
    if kind == "pages":
        if c["B"] * c["grow"] > 1 << 22:
            return None
        return _exact_pages(c, prepare(c, seed))
    D = c["D"]
    if kind == "turn":
        if c["tokens"] * c["heads"] * D > 1 << 29:
            return None
        st = prepare(c, seed)
        return _spin(c, st["x"], st["positions"])
    if kind == "store":
        if c["tokens"] * (c["Hq"] + c["Hkv"]) * D > 1 << 29 or c["pages"] * c["page"] * c["Hkv"] * D > 1 << 29:
            return None
        st = prepare(c, seed)
        kp, vp = st["kp"].double(), st["vp"].double()
        on = torch.nonzero(st["slots"] >= 0).flatten()
        at = st["slots"].long()[on]
        kp[at // c["page"], at % c["page"]] = _spin(c, st["k"], st["positions"])[on]
        vp[at // c["page"], at % c["page"]] = st["v"].double()[on]
        return _spin(c, st["q"], st["positions"]), kp, vp
    if kind == "bounds":
        if c["B"] * c["Hkv"] * c["new"] * D > 1 << 29:
            return None
        st = prepare(c, seed)
        blk = c["block"]
        value, scales = np.zeros(st["codes"].shape), np.zeros(st["scales"].shape)
        table = None if st["table"] is None else st["table"].cpu().numpy()
        for b, (lo, hi) in enumerate(zip(st["from"].tolist(), st["lens"].tolist())):
            for j in range(lo // blk, hi // blk):
                n, sub = (b, j) if table is None else (table[b, j * blk // c["page"]], j * blk % c["page"] // blk)
                rows = st["k"][n, sub * blk:(sub + 1) * blk].float().cpu().numpy()  # [block, Hkv, D]
                s = np.abs(rows).max((0, 2)) / np.float32(127)                      # float32 by definition
                up, down = np.ceil(rows.max(0) / s[:, None]), np.floor(rows.min(0) / s[:, None])
                value[n, sub] = np.clip(np.stack([up, down], 1), -127, 127) * s.astype(np.float64)[:, None, None]
                scales[n, sub] = s
        return value, scales
    if kind == "select":
        return _exact_select(c, seed)
    st = prepare(c, seed)
    if int(st["blocks"].numel()) * c["block"] * D > 1 << 30:
        return None
    B, T, Hq, Hkv = c["B"], c["T"], c["Hq"], c["Hkv"]
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64, device=DEV)
    rows, live = _tokens(st)
    G = Hq // Hkv
    k, v = (st[n].view(-1, Hkv, D) for n in ("k", "v"))
    for b in range(B):
        for i in range(T):
            keep = live[b, i].unsqueeze(1)                              # [Hkv, 1, n]
            at = rows[b, i]
            h = torch.arange(Hkv, device=DEV).unsqueeze(1)
            s = torch.einsum("hgd,hnd->hgn", st["q"][b, i].double().view(Hkv, G, D), k[at, h].double()) / math.sqrt(D)
            s = torch.where(keep, s, -math.inf)
            z = torch.logsumexp(s, -1)
            w = torch.where(keep, torch.exp(s - torch.where(z > -math.inf, z, 0.0).unsqueeze(-1)), 0.0)
            out[b, i] = torch.einsum("hgn,hnd->hgd", w, v[at, h].double()).reshape(Hq, D)
            lse[b, i] = z.flatten()
    return out, lse


def _exact_select(c, seed):
    """Scores in whole numbers, and the two roundings of their scales to float32 that the definition has."""
    if c["B"] * c["Hkv"] * c["T"] * (c["Hq"] // c["Hkv"]) * -(-c["hi"] // c["block"]) * c["D"] > 1 << 29:
        return None
    st = prepare(c, seed)
    q, lens = st["q"].float().cpu().numpy(), st["lens"].tolist()
    codes, scales = st["codes"].cpu().numpy(), st["scales"].cpu().numpy()
    table = None if st["table"] is None else st["table"].cpu().numpy()
    G, blk, K = c["Hq"] // c["Hkv"], c["block"], c["K"]
    out = np.full((c["B"], c["T"], c["Hkv"], K), -1)
    for b, L in enumerate(lens):
        cb, sb = (x[b] if table is None else x[table[b]].reshape((-1,) + x.shape[2:]) for x in (codes, scales))
        cb = cb.astype(np.float64)  # whole numbers below 2^24
        for i in range(c["T"]):
            n = max(0, -(-(L - c["T"] + 1 + i) // blk))
            for h in range(c["Hkv"]):
                best = np.full(n, -np.inf, np.float32)
                for row in q[b, i, h * G:(h + 1) * G]:
                    s = np.abs(row).max() / np.float32(127)
                    code = np.rint(row / s).astype(np.float64)
                    whole = cb[:n, h, 0] @ np.maximum(code, 0) + cb[:n, h, 1] @ np.minimum(code, 0)
                    best = np.maximum(best, whole.astype(np.float32) * s)
                best = best * sb[:n, h]
                j = np.arange(n)
                best[(j < c["first"]) | (j >= n - c["last"])] = np.inf
                pick = np.sort(np.lexsort((j, -best))[:K])
                out[b, i, h, :len(pick)] = pick
    return out
