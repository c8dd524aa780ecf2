"""Edges of the page tables, the appends by slots and the attention over selected blocks on the GPU: what parts a warp's
threads, states that do not hold together, caches shorter than a block, steps in which not every sequence grows."""
import numpy as np
import pytest

import blocks_ref as ref
from gpu_helpers import cuda_or_skip
from test_gpu_blocks import Cache, _close, _codes, _normal, _run, _select, _select_want, _want

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
