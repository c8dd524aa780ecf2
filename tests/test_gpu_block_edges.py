"""Edges of the page tables, the appends by slots and the attention over selected blocks on the GPU: what parts a warp's
threads, states that do not hold together, caches shorter than a block, steps in which not every sequence grows."""
import os
import re

import numpy as np
import pytest

import blocks_ref as ref
from gpu_helpers import bf16_tensor_bits, cuda_or_skip, to_dev_bf16
from test_gpu_blocks import Cache, _close, _codes, _normal, _run, _select, _select_want, _want
from test_gpu_pages import _check_turn, _positions, _rope, test_append as _append
from workloads import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,T", [(1, 1), (2, 1), (1, 9), (8, 2), (8, 4), (8, 6), (8, 11), (12, 5)])
def test_select_pages_missing_anywhere(D, G, T):
    """Lanes of one tile of 16 blocks that go different ways: entries without a page here and there, sequences that end
    inside a tile, every number of query rows scored at once, in one round and several."""
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    r = np.random.default_rng(1000 + D + G + T)
    Hkv, block, page, nb = 2, 16, 32, 150
    lens = [16 * 300 - 5, 16 * 257 + 3, 16 * 130, 16 * 9 + 1, 40]
    B = len(lens)
    n = B * nb + 2
    bt = r.permutation(n)[:B * nb].reshape(B, nb).astype(np.int32)
    bt[r.random(bt.shape) < 0.2] = -1
    bt[r.random(bt.shape) < 0.1] = 2 ** 31 - 1
    codes = _codes(r, (n, page // block, Hkv, D))
    scales = r.uniform(0.01, 0.03, (n, page // block, Hkv)).astype(np.float32)
    q = _normal(r, (B, T, G * Hkv, D))
    for K, first, last in ((8, 1, 2), (100, 0, 1)):
        got, st = _select(dev, q, codes, scales, lens, nb * page, block, K, first, last, bt)
        assert st == kvd.STATUS_BAD_PAGE
        assert np.array_equal(got, _select_want(q, codes, scales, lens, block, K, first, last, bt, page)), K


@pytest.mark.parametrize("block,page", [(16, 16), (32, 32), (64, 0)])
@pytest.mark.parametrize("Hq,D", [(4, 64), (16, 128), (48, 64), (40, 256)])
def test_attention_every_tail(Hq, D, block, page):
    """Stages that end at every token, for teams of one warp and of several: the scores past the end are masked by lane."""
    dev = cuda_or_skip()
    r = np.random.default_rng(Hq + D + block)
    c = Cache(r, list(range(1, 70)), 1, D, page, dev)
    q = _normal(r, (c.B, 1, Hq, D))
    x = np.tile(r.permutation(-(-c.S // block)).astype(np.int32), (c.B, 1, 1, 1))
    for dtype in ("bf16", "f32"):
        got = _run(c, q, x, block, dev, dtype)
        assert got[2] == 0
        _close(got[:2], _want(c, q, x, block), dtype)


@pytest.mark.parametrize("Hq,Hkv,D,block,K,lens", [(8, 1, 128, 128, 256, [32768]), (1, 1, 64, 16, 700, [11111]),
                                                   (48, 1, 256, 64, 128, [9000, 4097])])
def test_attention_of_several_clusters_flags_nothing(Hq, Hkv, D, block, K, lens):
    dev = cuda_or_skip()
    r = np.random.default_rng(K)
    c = Cache(r, lens, Hkv, D, 16, dev)
    q = _normal(r, (c.B, 1, Hq, D))
    x = r.integers(0, -(-c.S // block), (c.B, 1, Hkv, K)).astype(np.int32)
    for dtype in ("f32", "bf16"):
        got = _run(c, q, x, block, dev, dtype)
        assert got[2] == 0
        _close(got[:2], _want(c, q, x, block), dtype)


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("B", [7, 8, 14, 15, 16, 36, 37, 74, 75, 76, 77])
def test_attention_where_waves_end(B, D):
    """Numbers of pairs at which clusters of one size fill the machine, and one more."""
    dev = cuda_or_skip()
    r = np.random.default_rng(B + D)
    c = Cache(r, r.integers(0, 700, B), 1, D, 32, dev)
    q = _normal(r, (B, 1, 8, D))
    x = r.integers(0, -(-c.S // 32), (B, 1, 1, 40)).astype(np.int32)
    got = _run(c, q, x, 32, dev, "f32")
    assert got[2] == 0
    _close(got[:2], _want(c, q, x, 32), "f32")


def test_plans_for_this_device():
    """A plan for 152 multiprocessors is what a device of 152 says of itself."""
    import torch
    import kv_cache_decode_gb300 as kvd
    cuda_or_skip()
    if torch.cuda.get_device_properties(0).multi_processor_count != 152:
        pytest.skip("another number of multiprocessors")
    some = 0
    for D in (64, 128, 256):
        for B in (1, 2, 3, 5, 7, 8, 14, 15, 16):
            for K in (1, 16, 128, 1024):
                n = kvd.decode_blocks_plan(B, 1, 8, 1, D, K, 64, num_sms=152)
                assert kvd.decode_blocks_plan(B, 1, 8, 1, D, K, 64) == n
                some += n > 0
    assert some > 10


@pytest.mark.parametrize("S,block", [(20, 32), (1, 16), (40, 4096)])
def test_caches_shorter_than_a_block(S, block):
    """No bounds, one block that every token sees: bounds, selection and attention as over any cache."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    r = np.random.default_rng(S)
    c = Cache(r, [S, 0, 1, (S + 1) // 2], 2, 64, 0, dev, S=S)
    codes, scales = kvd.alloc_block_bounds(c.kd, block)
    assert codes.numel() == 0
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    kvd.kv_block_bounds(c.kd, codes, scales, c.lens_d, S, block, status=status)
    q = _normal(r, (4, 1, 8, 64))
    got, st = _select(dev, q, codes.cpu().numpy(), scales.cpu().numpy(), c.lens.tolist(), S, block, 3, 1, 2)
    assert st == 0 and int(status.item()) == 0
    assert got.tolist() == [[[[0 if L else -1, -1, -1]] * 2] for L in c.lens.tolist()]
    o, l, st = _run(c, q, got, block, dev, "f32")
    assert st == 0
    _close((o, l), _want(c, q, got, block), "f32")


# ---------------------------------------------------------------------------
# page tables
# ---------------------------------------------------------------------------

def _pages(dev, table, free, count, lens, new, page, rows):
    import torch
    import kv_cache_decode_gb300 as kvd
    i32 = dict(dtype=torch.int32, device=dev)
    t = [x if torch.is_tensor(x) else torch.tensor(x, **i32) for x in (table, free, count, lens, new)]
    off, slots, st = torch.full((len(new) + 1,), 99, **i32), torch.full((rows,), 99, **i32), torch.zeros(1, **i32)
    kvd.pages_update(*t, page, row_offsets=off, slots=slots, status=st)
    torch.cuda.synchronize()
    return t[:4] + [off.tolist(), slots.tolist()], int(st.item())


def test_pages_no_more_than_the_pool_has():
    """Lengths that claim more pages than there are: what comes back fills the stack, and no more is given out than it holds."""
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    none = [-1] * 4
    held = [[0, 1, -1, -1], [1, 2, -1, -1]]
    # 1 free and 4 that come back are taken for 3: four pages are not there
    (table, free, count, lens, off, slots), st = _pages(dev, held + [none], [0, 1, 2], [1], [32, 32, 0], [0, 0, 64], 16, 5)
    assert st == kvd.STATUS_BAD_PAGE | kvd.STATUS_NO_PAGES
    assert table.tolist() == [none] * 3 and count.tolist() == [3] and lens.tolist() == [0, 0, 0]
    assert off == [0] * 4 and slots == [-1] * 5
    # three are
    (table, free, count, lens, off, slots), st = _pages(dev, held + [none], [0, 1, 2], [1], [32, 32, 0], [0, 0, 48], 16, 49)
    assert st == kvd.STATUS_BAD_PAGE and count.tolist() == [0] and lens.tolist() == [0, 0, 48] and off == [0, 0, 0, 48]
    want = free.tolist()[::-1]
    assert table.tolist() == [none] * 2 + [want + [-1]] and slots == [p * 16 + t for p in want for t in range(16)] + [-1]


def test_pages_sums_past_32_bits():
    """Tokens that lengths of this size would add up to pass 2^32: refused, since the pool cannot hold them."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    i32 = dict(dtype=torch.int32, device=dev)
    table = torch.full((10, 1 << 18), -1, **i32)
    (table, free, count, lens, off, slots), st = _pages(dev, table, torch.zeros(1, **i32), [1], [1 << 30] * 5 + [0] * 5, [0] * 5 + [1 << 30] * 5, 4096,
                                                        1000)
    assert st == kvd.STATUS_BAD_PAGE | kvd.STATUS_NO_PAGES
    assert lens.tolist() == [0] * 10 and off == [0] * 11 and slots == [-1] * 1000 and bool((table == -1).all())


# ---------------------------------------------------------------------------
# rotary positions of several axes
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("order,interleaved", [("blocks", False), ("dealt", False), ("blocks", True)])
@pytest.mark.parametrize("sections,N,H,D", [((20, 20), 300, 16, 80), ((22, 21, 21), 77, 8, 128), ((8, 28, 28), 20000, 1, 128),
                                            ((9, 15), 9, 3, 64), ((31, 33), 30000, 2, 256)])
def test_turn_by_tables_of_each_axis(sections, N, H, D, order, interleaved):
    """Sections that end inside a thread's eight pairs, each with frequencies of its own table."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    r = np.random.default_rng(sum(sections))
    rope, turns, axes, factor = _rope(kvd, dev, sections, per_axis=True, order=order, interleaved=interleaved)
    pos = _positions(r, len(sections), N)
    x = r.standard_normal((N, H, D)).astype(np.float32)
    bits = f32_to_bf16_bits(x)
    xd, xb, pd = torch.from_numpy(x).to(dev), to_dev_bf16(bits, dev), torch.from_numpy(pos).to(dev)
    kvd.rope_apply_axes(rope, xd, pd, xd)
    _check_turn(xd.cpu().numpy().astype(np.float64), x, pos, turns, axes, factor, interleaved, False)
    kvd.rope_apply_axes(rope, xb, pd, xb)
    _check_turn(bf16_bits_to_f32(bf16_tensor_bits(xb)).astype(np.float64), bf16_bits_to_f32(bits), pos, turns, axes, factor, interleaved, True)


@pytest.mark.parametrize("form,N,Hq,Hkv,D", [
    ("bf16", 5, 4, 2, 80), ("bf16", 30000, 2, 1, 80), ("bf16", 7, 2, 1, 264), ("bf16", 30000, 2, 1, 264), ("bf16", 30000, 2, 1, 128),
    ("bf16", 30000, 1, 1, 256), ("int8", 30000, 2, 1, 128), ("int8", 30000, 1, 1, 256), ("fp8", 30000, 2, 1, 128),
    ("fp8", 30000, 1, 1, 256)])
def test_append_every_width(form, N, Hq, Hkv, D):
    """Heads of any width, and tokens of few heads, several to a warp, of every width: as test_gpu_pages.py's appends."""
    _append(form, N, Hq, Hkv, D)


# ---------------------------------------------------------------------------
# steps in which not every sequence grows
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("graph", [False, True])
def test_readme_step(graph):
    """The README's step as it stands there, for sequences that grow, pause, finish and find no page: every key and value in
    its own sequence, and the answers of those that grew against the definitions."""
    import torch
    import kv_cache_decode_gb300 as kvd
    dev = cuda_or_skip()
    readme = open(os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "README.md")).read()
    code, = [x for x in re.findall(r"```python\n(.*?)```", readme, re.S) if "RopeAxes" in x]
    at = code.index("kvd.pages_update")
    g = torch.Generator(device=dev)
    g.manual_seed(11)
    B, Hq, Hkv, D, max_blocks, pages = 6, 8, 2, 128, 4, 9
    i32 = dict(dtype=torch.int32, device=dev)

    def rows(*shape):
        return torch.randn(*shape, generator=g, device=dev).bfloat16()
    env = dict(torch=torch, kvd=kvd, B=B, Hq=Hq, Hkv=Hkv, D=D, max_len=64 * max_blocks, seq_lens=torch.zeros(B, **i32),
               new_lens=torch.zeros(B, **i32), old=torch.zeros(B, **i32), slots=torch.zeros(B, **i32), offsets=torch.zeros(B + 1, **i32),
               table=torch.full((B, max_blocks), -1, **i32), free=torch.arange(pages, **i32), count=torch.tensor([pages], **i32),
               positions=torch.zeros(3, B, **i32), blocks=torch.zeros(B, Hkv, 64, **i32), status=torch.zeros(1, **i32),
               out=torch.zeros(B, Hq, D, device=dev), q=rows(B, Hq, D), k_new=rows(B, Hkv, D), v_new=rows(B, Hkv, D),
               k_pool=rows(pages, 64, Hkv, D), v_pool=rows(pages, 64, Hkv, D))
    exec(code[:at], env)
    step = compile(code[at:], "README.md", "exec")
    # lengths before: pages 2 + 1 + 1 + 2 + 1 + 1 = 8 of 9
    lens = [65, 1, 63, 128, 30, 64]
    kvd.pages_update(env["table"], env["free"], env["count"], env["seq_lens"], torch.tensor(lens, **i32), 64)
    assert int(env["count"]) == 1
    keep = {n: x.clone() for n, x in env.items() if torch.is_tensor(x)}
    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            exec(step, env)
        torch.cuda.current_stream().wait_stream(side)
        G = torch.cuda.CUDAGraph()
        with torch.cuda.graph(G):
            exec(step, env)
        for n, x in keep.items():
            env[n].copy_(x)
    # sequence 3 takes the last page, 5 finds none; 1 pauses, 4 finishes (its page comes back first: 5 gets it in the next step)
    steps = [([66, 1, 64, 129, 30, 65], [66, 1, 64, 129, 30, 64], True), ([67, 2, 64, 130, 0, 65], [67, 2, 64, 130, 0, 65], False),
             ([67, 3, 65, 131, 1, 66], [67, 3, 64, 131, 0, 66], True)]
    have = [dict() for _ in range(B)]  # what each sequence's tokens hold, by position: those of these steps
    for want, got, refused in steps:
        env["new_lens"].copy_(torch.tensor(want, **i32))
        for n in ("q", "k_new", "v_new"):
            env[n].copy_(rows(*env[n].shape))
        env["positions"].copy_(torch.randint(0, 5000, (3, B), generator=g, device=dev))
        env["status"].zero_()
        kt, qt = torch.empty_like(env["k_new"]), torch.empty_like(env["q"])
        kvd.rope_apply_axes(env["rope"], env["k_new"], env["positions"], kt)
        kvd.rope_apply_axes(env["rope"], env["q"], env["positions"], qt)
        vt = env["v_new"].clone()
        G.replay() if graph else exec(step, env)
        torch.cuda.synchronize()
        assert env["seq_lens"].tolist() == got and int(env["status"]) == (kvd.STATUS_NO_PAGES if refused else 0)
        grown = [b for b in range(B) if got[b] > lens[b]]
        for b in range(B):
            have[b] = {t: x for t, x in have[b].items() if t < got[b]}
            if b in grown:
                have[b][got[b] - 1] = kt[b].clone(), vt[b].clone()
        table = env["table"].tolist()
        kf, vf = env["k_pool"].view(-1, Hkv, D), env["v_pool"].view(-1, Hkv, D)
        for b in range(B):
            for t, (k, v) in have[b].items():
                row = table[b][t // 64] * 64 + t % 64
                assert torch.equal(kf[row], k) and torch.equal(vf[row], v), (b, t)
        assert torch.equal(env["q"], qt)
        for b in grown:  # (fewer blocks than 64: all of them)
            at_rows = [table[b][t // 64] * 64 + t % 64 for t in range(got[b])]
            k, v = (x[at_rows].double().cpu().numpy() for x in (kf, vf))
            for h in range(Hkv):
                o, _, spread = ref.attend(qt[b, 4 * h:4 * h + 4].double().cpu().numpy(), k[:, h], v[:, h], list(range(4)), got[b], 64,
                                          D ** -0.5)
                tol = 1e-4 * np.maximum(1, spread) + 2 * 2.0 ** -16 / (1 - 2.0 ** -16) * spread  # (test_gpu_blocks.py's, float32)
                assert (np.abs(env["out"][b, 4 * h:4 * h + 4].double().cpu().numpy() - o) <= tol).all()
        lens = got
