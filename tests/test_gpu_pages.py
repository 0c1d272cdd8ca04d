"""Page operations against a host model: allocation order, release, forks in
place (any parent map), compaction, record copies, and their error codes."""
import numpy as np
import pytest
import torch

from bit_kv_cache_quantize_gb300 import inputs as I
from bit_kv_cache_quantize_gb300 import kvarn as K
from bit_kv_cache_quantize_gb300.cache import PagedCache

from gpu_helpers import device
from serving_ref import Pages

pytestmark = pytest.mark.gpu
T = D = 128


def make(lens, extra=0, h=2, dtype="f16", kb=4, vb=2, columns=0):
    dev = device()
    w = I.Workload("pages", len(lens), 2 * h, h, dtype, lens, seed=400, max_tokens=max(lens) + 1, block_perm=True,
                   k_bits=kb, v_bits=vb)
    c = PagedCache(w, dev, extra_blocks=extra)
    if columns:
        more = torch.full((len(lens), columns), -1, dtype=torch.int32, device=dev)
        c.table = torch.cat([c.table, more], 1).contiguous()
        c.max_blocks += columns
    c.pool.random_(0, 256, generator=torch.Generator(device=dev).manual_seed(1))
    c.tail.view(torch.int16).random_(-30000, 30000, generator=torch.Generator(device=dev).manual_seed(2))
    return c, Pages(c.table.cpu().numpy(), c.num_blocks, c.lens.cpu().numpy())


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def same(c, m, lens=None):
    torch.cuda.synchronize()
    assert (c.table.cpu().numpy() == m.table).all()
    assert (c.refs.cpu().numpy() == m.refs).all()
    if lens is not None:
        assert (lens.cpu().numpy() == m.lens).all()


def test_alloc_takes_the_lowest_free_ids_in_order():
    c, m = make([300, 129, 0, 640, 1000], extra=9, columns=7)
    c.refs
    end = [9, 2, 1, 5, 8]
    c.alloc(ints([0, 2, 0, 5, 8]), ints(end))        # two empty ranges
    assert not m.alloc([0, 2, 0, 5, 8], end)
    same(c, m)
    assert c.check_error() == 0
    c.alloc(ints([0] * 5), ints([c.max_blocks] * 5))  # more than the pool has
    assert m.alloc([0] * 5, [c.max_blocks] * 5)
    same(c, m)
    assert c.check_error() == K.KVARN_DEV_ERR_POOL_FULL


def test_alloc_over_many_sequences_and_blocks():
    """More sequences than threads, ids across many slabs of the counts."""
    c, m = make([1] * 1500, extra=9001, h=1, columns=5)
    rng = np.random.default_rng(0)
    drop = (rng.random(1500) < 0.5).astype(np.int32)
    c.free(ints([0] * 1500), ints(drop))
    m.free([0] * 1500, drop)
    same(c, m)
    end = rng.integers(0, 7, 1500).astype(np.int32)
    c.alloc(ints([0] * 1500), ints(end))
    m.alloc([0] * 1500, end)
    same(c, m)
    assert c.check_error() == 0


def test_range_and_count_errors():
    c, m = make([300, 129, 500], extra=3)
    c.refs
    c.free(ints([0, -1, 0]), ints([1, 1, 1]))         # a bad range: that sequence is skipped
    m.free([0, 0, 0], [1, 0, 1])
    same(c, m)
    assert c.check_error() == K.KVARN_DEV_ERR_TOKEN_RANGE
    c.err.zero_()
    c.alloc(ints([0, 0, 0]), ints([1, c.max_blocks + 1, 1]))
    m.alloc([0, 0, 0], [1, 0, 1])
    same(c, m)
    assert c.check_error() == K.KVARN_DEV_ERR_TOKEN_RANGE
    c.err.zero_()
    blk = int(c.table[2, 1])
    c.refs[blk] = 0                                   # a count that was lost
    c.free(ints([0, 0, 1]), ints([0, 0, 2]))
    torch.cuda.synchronize()
    assert c.check_error() == K.KVARN_DEV_ERR_REF_COUNT
    assert int(c.refs[blk]) == 0 and int(c.table[2, 1]) == -1
    c.err.zero_()
    c.table[2, 2] = c.num_blocks + 5
    c.free(ints([0, 0, 2]), ints([0, 0, 3]))
    torch.cuda.synchronize()
    assert c.check_error() == K.KVARN_DEV_ERR_BLOCK_RANGE and int(c.table[2, 2]) == -1


def same_bits(a, b):
    """16-bit tiles of random bits hold NaNs: compare the bits."""
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


def tails_after(tail, lens, parent):
    want = tail.clone()
    for b, p in enumerate(parent):
        if p >= 0 and p != b:
            r = int(lens[p]) % T
            want[b, :, :, :r] = tail[p, :, :, :r]
    return want


@pytest.mark.parametrize("group,batch", [(1, 3), (2, 6), (3, 10), (4, 8), (5, 5), (7, 17), (16, 32), (64, 40),
                                         (100, 230), (1024, 300)])
@pytest.mark.parametrize("kind", ["random", "cycle", "first", "drop"])
def test_fork_any_map_in_place(group, batch, kind):
    rng = np.random.default_rng(group + batch)
    lens = rng.integers(0, 700, batch).tolist()
    c, m = make(lens, h=1 if batch > 50 else 2, dtype="bf16")
    base = np.arange(batch) // group * group
    size = np.minimum(group, batch - base)
    at = np.arange(batch) - base
    parent = {"random": base + rng.integers(0, 1 << 30, batch) % size, "cycle": base + (at + 1) % size, "first": base,
              "drop": np.where(at % 3 == 1, -1, base + rng.integers(0, 1 << 30, batch) % size)}[kind]
    tail, lens_d = c.tail.clone(), c.lens.clone()
    c.refs
    c.fork(ints(parent), group)
    m.fork(parent)
    same(c, m, c.lens)
    assert c.check_error() == 0
    assert same_bits(c.tail, tails_after(tail, lens_d.cpu(), parent))


def test_fork_errors_keep_the_slot():
    c, m = make([300, 200, 500, 129])
    c.refs
    tail = c.tail.clone()
    c.fork(ints([2, 0, 2, 1]), 2)                     # slots 0 and 3 name parents of the other group
    m.fork([0, 0, 2, 3])
    same(c, m, c.lens)
    assert c.check_error() == K.KVARN_DEV_ERR_SLOT_RANGE
    assert same_bits(c.tail, tails_after(tail, [300, 200, 500, 129], [0, 0, 2, 3]))
    c.err.zero_()
    c.lens[2] = -5
    c.fork(ints([0, 0, 2, 2]), 4)
    torch.cuda.synchronize()
    assert c.check_error() == K.KVARN_DEV_ERR_TOKEN_RANGE
    assert (c.table.cpu().numpy() == m.table).all() and int(c.lens[3]) == 129


@pytest.mark.parametrize("kb,vb", [(4, 2), (2, 2), (4, 4)])
@pytest.mark.parametrize("batch", [1, 5, 40])
def test_compact_moves_records_and_names(kb, vb, batch):
    rng = np.random.default_rng(batch)
    c, m = make(rng.integers(1, 900, batch).tolist(), extra=7, h=3, kb=kb, vb=vb)
    c.refs
    if batch > 1:                                     # shared blocks move once
        parent = np.arange(batch)
        parent[1] = 0
        c.fork(ints(parent), batch)
        m.fork(parent)
    for step in range(3):
        begin = np.zeros(batch, np.int32)
        end = np.where(rng.random(batch) < 0.4, c.max_blocks, 0).astype(np.int32)
        c.free(ints(begin), ints(end))
        m.free(begin, end)
        pool = c.pool.clone().reshape(c.num_blocks, -1)
        counts = c.compact()
        live, src, dst = m.compact()
        same(c, m)
        assert c.check_error() == 0
        assert counts.tolist() == [live, len(src)]
        pool[dst] = pool[src]
        assert torch.equal(c.pool.reshape(c.num_blocks, -1), pool)
        assert (m.refs[:live] > 0).all() and not m.refs[live:].any()
        tiles = rng.integers(0, 3, batch).astype(np.int32)
        tiles = np.minimum(tiles, c.max_blocks)
        c.alloc(ints(begin), ints(tiles))
        m.alloc(begin, tiles)
        same(c, m)


def test_compact_many_blocks_and_none():
    """Ids over several chunks of the prefix sum; an empty pool."""
    c, m = make([1] * 9500, h=1)
    rng = np.random.default_rng(3)
    end = (rng.random(9500) < 0.6).astype(np.int32)
    c.free(ints([0] * 9500), ints(end))
    m.free([0] * 9500, end)
    counts = c.compact()
    live, src, dst = m.compact()
    same(c, m)
    assert counts.tolist() == [live, len(src)]
    c.free(ints([0] * 9500), ints([1] * 9500))
    counts = c.compact()
    torch.cuda.synchronize()
    assert counts.tolist() == [0, 0] and not c.refs.any() and c.check_error() == 0


def test_compact_reports_a_block_without_count():
    c, m = make([128] * 6)
    c.refs
    top = int((c.table == c.num_blocks - 1).nonzero()[0, 0])
    c.refs[c.num_blocks - 1] = 0
    c.compact()
    torch.cuda.synchronize()
    assert c.check_error() == K.KVARN_DEV_ERR_REF_COUNT and int(c.table[top, 0]) == c.num_blocks - 1


@pytest.mark.parametrize("n", [1, 3, 50, 700])
@pytest.mark.parametrize("h,kb,vb", [(1, 2, 2), (3, 4, 2), (8, 4, 4)])
def test_copy_between_pools(n, h, kb, vb):
    dev = device()
    cfg = K.make_config(h, h, n + 5, k_bits=kb, v_bits=vb)
    size = K.kvarn_block_bytes(cfg)
    g = torch.Generator(device=dev).manual_seed(n)
    src = torch.randint(0, 256, (n + 9, size), dtype=torch.uint8, device=dev, generator=g)
    dst = torch.randint(0, 256, (n + 5, size), dtype=torch.uint8, device=dev, generator=g)
    a = torch.randperm(n + 9, device=dev, generator=g)[:n].to(torch.int32)
    b = torch.randperm(n + 5, device=dev, generator=g)[:n].to(torch.int32)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    want = dst.clone()
    want[b.long()] = src[a.long()]
    K.kvarn_copy_blocks(cfg, src, n + 9, a, dst, b, n, None, err)
    torch.cuda.synchronize()
    assert int(err) == 0 and torch.equal(dst, want)
    # a device count: fewer than n, then more
    for count in (n // 2, -4, n + 100):
        dst.zero_()
        m = min(n, max(0, count))
        want = torch.zeros_like(dst)
        want[b[:m].long()] = src[a[:m].long()]
        K.kvarn_copy_blocks(cfg, src, n + 9, a, dst, b, n, torch.tensor([count], dtype=torch.int32, device=dev), err)
        torch.cuda.synchronize()
        assert int(err) == 0 and torch.equal(dst, want)
    # ids out of range are skipped and reported
    bad = a.clone()
    bad[n // 2] = n + 9
    bad[n - 1] = -1 if n > 1 else n + 9
    want = torch.zeros_like(dst)
    keep = torch.ones(n, dtype=torch.bool, device=dev)
    keep[n // 2] = False
    keep[n - 1] = False
    want[b[keep].long()] = src[a[keep].long()]
    dst.zero_()
    K.kvarn_copy_blocks(cfg, src, n + 9, bad, dst, b, n, None, err)
    torch.cuda.synchronize()
    assert int(err) == K.KVARN_DEV_ERR_BLOCK_RANGE and torch.equal(dst, want)


def test_compact_reports_a_low_block_without_count():
    """A block below the live ones' end that a table entry names but no count
    holds: it may be given away as a hole, so it has to be reported."""
    c, m = make([128] * 6)
    c.refs[0] = 0
    c.compact()
    torch.cuda.synchronize()
    assert c.check_error() == K.KVARN_DEV_ERR_REF_COUNT


@pytest.mark.parametrize("batch,columns", [(128, (1 << 24) - 1), (2 ** 31 - 1, 1)])
def test_alloc_at_the_largest_tables(batch, columns):
    """Tables of 2^31 - 128 and 2^31 - 1 entries, open ones at both ends."""
    dev = device()
    cfg = K.make_config(1, 1, 9, "f16")
    table = torch.zeros(batch, columns, dtype=torch.int32, device=dev)
    refs = torch.tensor([7, 0, 1, 0, 0, 1, 0, 0, 1], dtype=torch.int32, device=dev)
    table[0, 0] = table[-1, -1] = table[batch // 2, columns // 2] = -1
    begin = torch.zeros(batch, dtype=torch.int32, device=dev)
    end = torch.full((batch,), columns, dtype=torch.int32, device=dev)
    need = K.kvarn_pages_workspace_bytes(cfg, batch)
    ws, err = torch.empty(need, dtype=torch.uint8, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    K.kvarn_alloc_blocks(cfg, table, columns, batch, begin, end, refs, ws, need, err)
    torch.cuda.synchronize()
    assert int(err) == 0
    assert [int(table[0, 0]), int(table[batch // 2, columns // 2]), int(table[-1, -1])] == [1, 3, 4]
    assert refs.tolist() == [7, 1, 1, 1, 1, 1, 0, 0, 1]
    table[0, 0] = table[-1, -1] = table[batch // 2, columns // 2] = 0
    assert not table.any()
