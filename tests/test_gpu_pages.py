"""Page tables from request lengths, and rows turned and stored by their slots, on
the GPU: tables, stacks, slots and cached bits exactly; the rotation against
float64 phases (its cosines and sines are off by 1.1e-7 at most, products and sum in float32: 3e-7 of a pair's length, and
half a step of bf16 output: 8 significant bits, so 2^-8 of the value at most)."""
import numpy as np
import pytest

import blocks_ref as ref
from gpu_helpers import bf16_tensor_bits, cuda_or_skip, to_dev_bf16
from workloads import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu


class Device:
    """The device's side of blocks_ref.Pages."""

    def __init__(self, model, dev):
        import torch
        t = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
        self.dev, self.model = dev, model
        self.table, self.free, self.count, self.lens = t(model.table), t(model.stack), t([model.count]), t(model.lens)

    def update(self, new, rows, misalign=0):
        import torch
        import kv_cache_decode_gb300 as kvd
        B = len(new)
        i32 = dict(dtype=torch.int32, device=self.dev)
        pos, off = torch.full((B,), 99, **i32), torch.full((B + 1,), 99, **i32)
        buf = torch.full((2, rows + 16), 99, **i32)
        slots, positions = buf[0, misalign:misalign + rows], buf[1, misalign:misalign + rows]
        status = torch.zeros(1, **i32)
        kvd.pages_update(self.table, self.free, self.count, self.lens, torch.tensor(new, **i32), self.model.page, pos=pos,
                         row_offsets=off, slots=slots, positions=positions, status=status)
        torch.cuda.synchronize()
        assert bool((buf[:, :misalign] == 99).all()) and bool((buf[:, misalign + rows:] == 99).all())
        return [x.tolist() for x in (pos, off, slots, positions)], int(status.item())

    def check(self):
        m = self.model
        assert self.table.tolist() == m.table and self.lens.tolist() == m.lens and self.count.tolist() == [m.count]
        assert self.free.tolist() == m.stack


def _model(r, B, max_blocks, page, num_pages):
    return ref.Pages(B, max_blocks, page, num_pages, r.permutation(num_pages).tolist())


def _step(d, new, rows, misalign=0):
    import kv_cache_decode_gb300 as kvd
    pos, off, slots, positions, refused = d.model.update(new)
    got, st = d.update(new, rows, misalign)
    cut = len(slots) > rows > 0  # (empty tensors are as none given)
    bad = any(not 0 <= n <= d.model.max_blocks * d.model.page for n in new)
    pad = lambda x: (x + [-1] * rows)[:rows]  # noqa: E731
    assert got == [pos, off, pad(slots), pad(positions)]
    assert st == (kvd.STATUS_NO_PAGES if refused else 0) | (2 if cut or bad else 0)
    d.check()


@pytest.mark.parametrize("B,max_blocks,page,num_pages", [(1, 1, 16, 1), (1, 40, 16, 40), (7, 9, 64, 50), (64, 12, 16, 500), (600, 5, 32, 1500),
                                                        (513, 3, 128, 2000)])
def test_pages_random_walk(B, max_blocks, page, num_pages):
    dev = cuda_or_skip()
    r = np.random.default_rng(B)
    d = Device(_model(r, B, max_blocks, page, num_pages), dev)
    cap = max_blocks * page
    for step in range(12):
        kind = step % 4
        lens = np.array(d.model.lens)
        if kind == 0:      # some admitted, some finished, some left
            new = np.where(r.random(B) < 0.4, r.integers(0, cap + 1, B), lens)
        elif kind == 1:    # one token each
            new = lens + 1
        elif kind == 2:    # drafted tokens, some taken back, a length that the table cannot hold
            new = np.clip(lens + r.integers(-7, 8, B), 0, None)
            new[r.integers(B)] = r.choice([-1, cap + 1, 2 ** 31 - 1])
        else:              # most finish
            new = np.where(r.random(B) < 0.8, 0, lens)
        rows = int(r.choice([0, 1, 7, B, 3 * B + 5, B * cap]))
        _step(d, new.tolist(), rows, misalign=int(r.integers(0, 4)))


def test_pages_large():
    """8,192 sequences, and rows for a cluster of CTAs."""
    dev = cuda_or_skip()
    r = np.random.default_rng(3)
    d = Device(_model(r, 8192, 4, 16, 20000), dev)
    _step(d, r.integers(0, 65, 8192).tolist(), 300000)
    _step(d, r.integers(0, 65, 8192).tolist(), 100000)
    d = Device(_model(r, 24, 80, 64, 1500), dev)
    _step(d, r.integers(1, 4097, 24).tolist(), 24 * 4096, misalign=3)
    _step(d, [0] * 24, 0)


def test_pages_rollback_restores():
    """A shrink right behind a growth leaves table and stack as they were; with nothing asked for, nothing changes."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    r = np.random.default_rng(4)
    d = Device(_model(r, 33, 20, 16, 400), dev)
    _step(d, r.integers(0, 150, 33).tolist(), 5000)
    before = [x.clone() for x in (d.table, d.free, d.count, d.lens)]
    kvd.pages_update(d.table, d.free, d.count, d.lens, d.lens + 40, 16)
    assert not torch.equal(d.table, before[0])
    kvd.pages_update(d.table, d.free, d.count, d.lens, before[3], 16)
    kvd.pages_update(d.table, d.free, d.count, d.lens, d.lens.clone(), 16)
    for x, y in zip((d.table, d.free, d.count, d.lens), before):
        assert torch.equal(x, y)


def test_pages_without_sequences():
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    i32 = dict(dtype=torch.int32, device=dev)
    free, count = torch.arange(5, **i32), torch.tensor([5], **i32)
    none, off, slots, positions = torch.empty(0, **i32), torch.full((1,), 9, **i32), torch.full((7,), 9, **i32), torch.full((7,), 9, **i32)
    kvd.pages_update(torch.empty(0, 3, **i32), free, count, none, none.clone(), 16, pos=none.clone(), row_offsets=off, slots=slots,
                     positions=positions)
    assert off.tolist() == [0] and slots.tolist() == [-1] * 7 and positions.tolist() == [-1] * 7
    assert free.tolist() == list(range(5)) and count.tolist() == [5]


def test_pages_bad_state():
    """Counts and lengths out of range, entries and stack places that name no page: flagged, in bounds, the rest served."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    i32 = dict(dtype=torch.int32, device=dev)

    def run(table, free, count, lens, new, rows):
        t = [torch.tensor(x, **i32) for x in (table, free, count, lens, new)]
        slots, st = torch.full((rows,), 99, **i32), torch.zeros(1, **i32)
        kvd.pages_update(*t, 16, slots=slots, status=st)
        torch.cuda.synchronize()
        return [x.tolist() for x in t[:4]] + [slots.tolist()], int(st.item())
    # a count past the pool is taken as the whole stack
    (table, _, count, lens, slots), st = run([[-1, -1]], [1, 0, 2], [77], [0], [17], 18)
    assert st == kvd.STATUS_BAD_PAGE and table == [[2, 0]] and count == [1] and lens == [17]
    assert slots == [32 + i for i in range(16)] + [0, -1]
    # a negative count: no page
    (table, _, count, lens, _), st = run([[-1, -1]], [1, 0, 2], [-4], [0], [17], 0)
    assert st == kvd.STATUS_BAD_PAGE | kvd.STATUS_NO_PAGES and table == [[-1, -1]] and count == [0] and lens == [0]
    # a length before past the table is clamped to it
    (table, free, count, lens, _), st = run([[0, 1]], [2, 9, 9], [1], [2 ** 31 - 1], [0], 0)
    assert st == kvd.STATUS_SEQ_LEN_CLAMPED and table == [[-1, -1]] and free == [2, 1, 0] and count == [3] and lens == [0]
    # a place of the stack that names no page is handed on, without slots
    (table, _, _, lens, slots), st = run([[-1, -1]], [5, 1, 2], [1], [0], [3], 4)
    assert st == kvd.STATUS_BAD_PAGE and table == [[5, -1]] and lens == [3] and slots == [-1] * 4
    # more pages come back than the pool has
    (table, free, count, _, _), st = run([[0, 1], [1, 2]], [0, 1, 2], [2], [32, 32], [0, 0], 0)
    assert st == kvd.STATUS_BAD_PAGE and count == [3] and table == [[-1, -1], [-1, -1]]


# ---------------------------------------------------------------------------
# rotary positions of several axes
# ---------------------------------------------------------------------------

def _rope(kvd, dev, sections, **kw):
    rope = kvd.RopeAxes(sections, device=dev, **kw)
    t = {k: v for k, v in kw.items() if k != "interleaved"}
    turns, axes, factor = kvd.rope_axes_table(sections, **t)
    return rope, turns, axes, factor


def _positions(r, A, N):
    p = r.integers(0, 100000, (A, N))
    p[:, r.random(N) < 0.1] = 2 ** 31 - 1
    p[0, r.random(N) < 0.1] = -2 ** 31
    return p.astype(np.int32)


def _check_turn(got, x, pos, turns, axes, factor, interleaved, bf16_out):
    want = ref.turn_exact(x.astype(np.float64), pos, turns, axes, factor, interleaved)
    R = 2 * len(turns)
    assert np.array_equal(got[..., R:], x[..., R:].astype(np.float64))
    length = np.abs(x[..., :R]).max(-1, keepdims=True) * np.sqrt(2) * factor
    tol = 3e-7 * length + (np.abs(want[..., :R]) * 2.0 ** -8 * 1.001 if bf16_out else 0)
    assert (np.abs(got - want)[..., :R] <= tol).all()


@pytest.mark.parametrize("sections,kw", [((16, 24, 24), {}), ((24, 20, 20), dict(order="dealt", base=5e5)), ((8,), {}),
                                         ((8, 16, 8), dict(per_axis=True, interleaved=True)), ((1, 2, 3, 2), dict(order="dealt", interleaved=True)),
                                         ((16, 16), dict(scaling="parts", factor=8.0, original_len=4096.0)), ((64, 32, 32), {})])
@pytest.mark.parametrize("N,H,D", [(1, 1, 64), (5, 32, 128), (700, 3, 80), (30000, 1, 128), (129, 8, 256), (20000, 2, 64), (3, 5, 264)])
def test_turn(sections, kw, N, H, D):
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    if 2 * sum(sections) > D:
        pytest.skip("the rotary columns exceed the head")
    r = np.random.default_rng(N + D)
    rope, turns, axes, factor = _rope(kvd, dev, sections, **kw)
    assert np.array_equal(axes, ref.axes_of(sections, kw.get("order") == "dealt"))
    pos = _positions(r, len(sections), N)
    x = r.standard_normal((N, H, D)).astype(np.float32)
    inter = kw.get("interleaved", False)
    pd = torch.from_numpy(pos).to(dev)
    xd = torch.from_numpy(x).to(dev)
    out = torch.empty_like(xd)
    kvd.rope_apply_axes(rope, xd, pd, out)
    _check_turn(out.cpu().numpy().astype(np.float64), x, pos, turns, axes, factor, inter, False)
    # bf16, in place, slices of a wider buffer
    wide = torch.full((N, H * D + 16), 7.0, dtype=torch.bfloat16, device=dev)
    rows = wide[:, 8:8 + H * D].view(N, H, D)
    bits = f32_to_bf16_bits(x)
    rows.copy_(to_dev_bf16(bits, dev))
    kvd.rope_apply_axes(rope, rows, pd, rows)
    got = bf16_bits_to_f32(bf16_tensor_bits(rows)).astype(np.float64)
    _check_turn(got, bf16_bits_to_f32(bits), pos, turns, axes, factor, inter, True)
    assert bool((wide[:, :8] == 7).all()) and bool((wide[:, 8 + H * D:] == 7).all())
    # bf16 to fp32 gives what rounds to that
    out = torch.empty(N, H, D, device=dev)
    kvd.rope_apply_axes(rope, to_dev_bf16(bits, dev), pd, out)
    assert torch.equal(out.bfloat16(), rows)


def test_turn_one_axis_is_rope_apply():
    """Where all axes have the same positions the rotation is the one-axis one, bit for bit; positions of a wider buffer."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    x = torch.randn(40, 6, 128, device=dev, dtype=torch.bfloat16)
    p = torch.randint(-2 ** 31, 2 ** 31 - 1, (40,), device=dev).int()
    want, got = torch.empty_like(x), torch.empty_like(x)
    kvd.rope_apply(kvd.RopeTable(128, device=dev), x, p, want)
    wide = torch.zeros(3, 100, device=dev, dtype=torch.int32)
    wide[:, 20:60] = p
    kvd.rope_apply_axes(kvd.RopeAxes((16, 24, 24), device=dev), x, wide[:, 20:60], got)
    assert torch.equal(got, want)
    kvd.rope_apply_axes(kvd.RopeAxes((64,), device=dev), x.view(4, 10, 6, 128), p.view(1, 4, 10), got.view(4, 10, 6, 128))
    assert torch.equal(got, want)


@pytest.mark.parametrize("form", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("N,Hq,Hkv,D", [(1, 8, 1, 128), (64, 32, 8, 128), (37, 6, 3, 64), (300, 8, 8, 256), (30000, 2, 1, 64)])
def test_append(form, N, Hq, Hkv, D):
    """The rows that rope_apply_axes gives, stored by the plain appends, bit for bit; slots of no row and past the cache."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    r = np.random.default_rng(N)
    page, pages = 16, -(-N // 16) + 4
    rope = kvd.RopeAxes((8, 4, 12), base=5e5, order="dealt", device=dev)
    qkv = torch.randn(N, (Hq + 2 * Hkv) * D, device=dev, dtype=torch.bfloat16)
    q, k, v = qkv[:, :Hq * D].view(N, Hq, D), qkv[:, Hq * D:(Hq + Hkv) * D].view(N, Hkv, D), qkv[:, (Hq + Hkv) * D:].view(N, Hkv, D)
    pos = torch.from_numpy(_positions(r, 3, N)).to(dev)
    slots = r.permutation(pages * page)[:N].astype(np.int32)
    drop = r.random(N) < 0.2
    over = ~drop & (r.random(N) < 0.1)
    slots[drop] = r.choice([-1, -2 ** 31], drop.sum())
    slots[over] = r.choice([pages * page, 2 ** 31 - 1], over.sum())
    quant = form != "bf16"
    dt = {"bf16": torch.bfloat16, "int8": torch.int8, "fp8": torch.uint8}[form]

    def empty():
        c = [torch.full((pages, page, Hkv, D), 3, dtype=dt, device=dev) for _ in range(2)]
        return c, [torch.full((pages, page, Hkv), 9.0, device=dev) for _ in range(2)] if quant else [None, None]
    (kc, vc), (ks, vs) = empty()
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    q_out = torch.empty(N, Hq, D, device=dev, dtype=torch.bfloat16)
    kvd.kv_append_axes(rope, kc, vc, k, v, torch.from_numpy(slots).to(dev), pos, q=q, q_out=q_out, k_scales=ks, v_scales=vs, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == (kvd.STATUS_POS_OUT_OF_RANGE if over.any() else 0)
    want_q, kt = torch.empty_like(q_out), torch.empty(N, Hkv, D, device=dev, dtype=torch.bfloat16)
    kvd.rope_apply_axes(rope, q, pos, want_q)
    kvd.rope_apply_axes(rope, k, pos, kt)
    assert torch.equal(q_out, want_q)
    (kw, vw), (ksw, vsw) = empty()
    on = np.nonzero(~drop & ~over)[0]
    one = torch.from_numpy(slots[on] // page).to(dev), torch.from_numpy((slots[on] % page).astype(np.int32)).to(dev)
    if len(on):
        flat = lambda c: c.view(1, pages * page, Hkv, D)  # noqa: E731
        if quant:  # each row as a sequence of its own, whose page is the one that the slot lies on
            f = kvd.kv_append_q8_paged if form == "int8" else kvd.kv_append_fp8_paged
            f(kw, vw, ksw, vsw, kt[on].contiguous(), v[on].contiguous(), one[0].int().view(-1, 1).contiguous(), one[1])
        else:
            flat(kw)[0, torch.from_numpy(slots[on]).to(dev).long()] = kt[on]
            flat(vw)[0, torch.from_numpy(slots[on]).to(dev).long()] = v[on]
    assert torch.equal(kc, kw) and torch.equal(vc, vw)
    if quant:
        assert torch.equal(ks, ksw) and torch.equal(vs, vsw)
    # without queries, in place, a contiguous cache
    (k2, v2), (ks2, vs2) = empty()
    kvd.kv_append_axes(rope, k2, v2, k, v, torch.from_numpy(slots).to(dev), pos, k_scales=ks2, v_scales=vs2, paged=False)
    assert torch.equal(k2, kw) and torch.equal(v2, vw)


def test_turn_negative_turns_back():
    """The rotation by minus the positions undoes it (fp32: two roundings of each, 4e-7 of a pair's length together with the
    cosines' and sines')."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    x = torch.randn(333, 4, 128, device=dev)
    p = torch.randint(0, 1 << 20, (3, 333), device=dev).int()
    rope = kvd.RopeAxes((16, 24, 24), device=dev)
    y, z = torch.empty_like(x), torch.empty_like(x)
    kvd.rope_apply_axes(rope, x, p, y)
    kvd.rope_apply_axes(rope, y, -p, z)
    assert float((z - x).abs().max()) <= 6e-7 * float(x.abs().max()) * 2 ** 0.5


@pytest.mark.parametrize("what", ["turn", "append", "pages", "bounds", "select", "decode"])
def test_other_stream(what):
    """Each call on a stream of its own, whose inputs that stream makes, gives what it gives on the current one."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    i32 = dict(dtype=torch.int32, device=dev)
    q, k = torch.randn(4, 8, 64, generator=g, device=dev).bfloat16(), torch.randn(4, 512, 2, 64, generator=g, device=dev).bfloat16()
    lens, rope = torch.tensor([512, 77, 300, 16], **i32), kvd.RopeAxes((8, 24), device=dev)
    p = torch.randint(0, 1000, (2, 4), generator=g, device=dev).int()
    side = torch.cuda.Stream()

    def run(stream):
        on = stream or torch.cuda.current_stream()
        with torch.cuda.stream(on):
            torch.cuda._sleep(200000)
            qq, kk, ll, pp = q * 1, k * 1, lens * 1, p * 1
            codes, scales = kvd.alloc_block_bounds(kk, 16)
            if what == "turn":
                res = torch.empty_like(qq)
            elif what == "append":
                res = kk.clone()
                new, slots = qq[:, :2].contiguous(), torch.tensor([3, 600, -1, 2047], **i32)
            elif what == "pages":
                table, free, count = torch.full((4, 40), -1, **i32), torch.arange(150, **i32), torch.tensor([150], **i32)
                old, res = torch.zeros(4, **i32), torch.empty(905, **i32)
            elif what == "decode":
                res, blocks = torch.empty_like(qq), (torch.arange(4 * 2 * 5, **i32) % 32).view(4, 2, 5)
            elif what == "select":
                codes.copy_(torch.arange(codes.numel(), device=dev).view_as(codes) % 127)
                scales.fill_(0.5)
                res, ws = torch.empty(4, 2, 5, **i32), torch.empty(1 << 16, dtype=torch.uint8, device=dev)
        if what == "turn":
            kvd.rope_apply_axes(rope, qq, pp, res, stream=stream)
        elif what == "append":
            kvd.kv_append_axes(rope, res, kk, new, new.clone(), slots, pp, paged=False, stream=stream)
        elif what == "pages":
            kvd.pages_update(table, free, count, old, ll, 16, slots=res, stream=stream)
        elif what == "bounds":
            kvd.kv_block_bounds(kk, codes, scales, ll, 512, 16, stream=stream)
            res = codes
        elif what == "select":
            kvd.block_select(qq, codes, scales, ll, 512, 16, res, workspace=ws, stream=stream)
        else:
            kvd.decode_blocks(qq, kk, kk, blocks, ll, 16, 0.125, res, stream=stream)
        torch.cuda.synchronize()
        return res
    torch.cuda.synchronize()
    assert torch.equal(run(None), run(side))


# ---------------------------------------------------------------------------
# a serving loop
# ---------------------------------------------------------------------------

def _serve(kvd, torch, dev, graph):
    """Prompts admitted and appended, then steps of one token: pages, turned appends, bounds, selection, attention."""
    g = torch.Generator(device=dev)
    g.manual_seed(5)
    B, Hq, Hkv, D, page, block, K, steps = 5, 8, 2, 64, 32, 16, 6, 40
    max_blocks, pages, N = 12, 50, 700
    i32 = dict(dtype=torch.int32, device=dev)
    rope = kvd.RopeAxes((8, 12, 12), device=dev)
    kp, vp = (torch.full((pages, page, Hkv, D), float("nan"), dtype=torch.bfloat16, device=dev) for _ in range(2))
    codes, scales = kvd.alloc_block_bounds(kp, block)
    table, free, count = torch.full((B, max_blocks), -1, **i32), torch.randperm(pages, generator=g, device=dev).int(), torch.tensor([pages], **i32)
    lens, pos, off = torch.zeros(B, **i32), torch.zeros(B, **i32), torch.zeros(B + 1, **i32)
    ws = torch.empty(kvd.block_select_plan(B, 1, Hkv, max_blocks * page, block), dtype=torch.uint8, device=dev)
    blocks, out, lse = torch.empty(B, Hkv, K, **i32), torch.empty(B, Hq, D, device=dev), torch.empty(B, Hq, device=dev)
    status = torch.zeros(1, **i32)

    def tokens(n):
        return torch.randn(n, (Hq + 2 * Hkv) * D, generator=g, device=dev).bfloat16()

    def step(new, qkv, slots, positions, q_out, most):
        n = qkv.shape[0]
        q, k, v = qkv[:, :Hq * D].view(n, Hq, D), qkv[:, Hq * D:(Hq + Hkv) * D].view(n, Hkv, D), qkv[:, (Hq + Hkv) * D:].view(n, Hkv, D)
        kvd.pages_update(table, free, count, lens, new, page, pos=pos, row_offsets=off, slots=slots, positions=positions, status=status)
        kvd.kv_append_axes(rope, kp, vp, k, v, slots, positions.expand(3, n).contiguous(), q=q, q_out=q_out, status=status)
        kvd.kv_block_bounds(kp, codes, scales, lens, most, block, from_lens=pos, block_table=table, status=status)

    def attend(q):
        kvd.block_select(q, codes, scales, lens, max_blocks * page, block, blocks, n_first=1, n_last=2, block_table=table, workspace=ws,
                         status=status)
        kvd.decode_blocks(q, kp, vp, blocks, lens, block, D ** -0.5, out, block_table=table, lse=lse, status=status)
    buf = [torch.zeros(N, **i32) for _ in range(2)]
    prompts = torch.tensor([200, 1, 57, 128, 300], **i32)
    first = tokens(N)
    step(prompts, first, *buf, torch.empty(N, Hq, D, dtype=torch.bfloat16, device=dev), 300)
    feed = [tokens(B) for _ in range(steps)]
    qkv, q_out = torch.empty_like(feed[0]), torch.empty(B, Hq, D, dtype=torch.bfloat16, device=dev)
    sb = [torch.zeros(B, **i32) for _ in range(2)]

    def whole():
        step(lens + 1, qkv, *sb, q_out, 1)
        attend(q_out)
    results = []
    if graph:
        keep = [x.clone() for x in (table, free, count, lens, kp, vp, codes, scales)]
        qkv.copy_(feed[0])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            whole()
        torch.cuda.current_stream().wait_stream(side)
        G = torch.cuda.CUDAGraph()
        with torch.cuda.graph(G):
            whole()
        for x, y in zip((table, free, count, lens, kp, vp, codes, scales), keep):
            x.copy_(y)
    for x in feed:
        qkv.copy_(x)
        G.replay() if graph else whole()
        results.append((blocks.clone(), out.clone(), lse.clone(), lens.clone(), q_out.clone()))
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return results, (table.cpu().numpy(), kp.clone(), vp.clone(), page, block, K, Hkv, D)


def test_serving_loop():
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    eager, (table, kp, vp, page, block, K, Hkv, D) = _serve(kvd, torch, dev, False)
    graph, _ = _serve(kvd, torch, dev, True)
    for a, b in zip(eager, graph):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    # the last step against the definitions, from the cache alone
    blocks, out, lse, lens, q = (x.cpu() for x in eager[-1])
    for b, L in enumerate(lens.tolist()):
        rows = [table[b, t // page] * page + t % page for t in range(L)]
        k, v = (x.view(-1, Hkv, D)[rows].float().cpu().numpy() for x in (kp, vp))
        assert np.isfinite(k).all()
        G = q.shape[1] // Hkv
        for h in range(Hkv):
            qq = q[b, h * G:(h + 1) * G].float().numpy()
            nb = -(-L // block)
            s = np.zeros(nb, np.float32)
            for j in range(L // block):
                c, sc = ref.bounds(k[j * block:(j + 1) * block])
                s[j] = ref.score(qq, c[h:h + 1], sc[h:h + 1])[0]
            want = ref.select(s, K, 1, 2)
            assert blocks[b, h].tolist() == want
            o, l, _ = ref.attend(qq.astype(np.float64), k[:, h].astype(np.float64), v[:, h].astype(np.float64), want, L, block, D ** -0.5)
            assert np.abs(out[b, h * G:(h + 1) * G].double().numpy() - o).max() < 1e-4 and np.abs(lse[b, h * G:(h + 1) * G].double().numpy() - l).max() < 1e-4
