"""Refusals and sizes of the window, tree, commit and page calls: all found on
the host, before any launch (no GPU is needed)."""
import pytest
import torch

from bit_kv_cache_quantize_gb300 import build as B
from bit_kv_cache_quantize_gb300 import inputs as I
from bit_kv_cache_quantize_gb300 import kvarn as K
from bit_kv_cache_quantize_gb300.cache import PagedCache

INV, UNS = K.KVARN_ERR_INVALID, K.KVARN_ERR_UNSUPPORTED
CFG = K.make_config(8, 64, 100, "f16")
BAD = K.make_config(8, 64, 100, "f16", k_bits=3)


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()


def window(cfg=CFG, q=16, nq=1, table=16, mb=40, lens=16, batch=2, window=200, sinks=4, pool=16, tail=16, out=16,
           kind=0, ws=16, size=None):
    if size is None:
        size = 1 << 40
    return K.kvarn_window_attention(cfg, q, nq, table, mb, lens, batch, window, sinks, pool, tail, 0.1, out, kind, ws,
                                    size, 16, stream=0, check=False)


@pytest.mark.parametrize("change,status", [
    (dict(cfg=BAD), UNS), (dict(nq=0), INV), (dict(nq=4097), INV), (dict(mb=0), INV), (dict(mb=1 << 24), INV),
    (dict(batch=-1), INV), (dict(batch=65536), INV), (dict(window=0), INV), (dict(window=-5), INV),
    (dict(sinks=-1), INV), (dict(kind=2), INV), (dict(kind=-1), INV), (dict(q=None), INV), (dict(q=8), INV),
    (dict(table=None), INV), (dict(lens=None), INV), (dict(pool=None), INV), (dict(pool=24), INV),
    (dict(tail=None), INV), (dict(tail=8), INV), (dict(out=None), INV), (dict(out=4), INV), (dict(ws=None), INV),
    (dict(ws=8), INV), (dict(size=0), INV), (dict(nq=4096, batch=65535), UNS), (dict(batch=0, q=None), 0),
])
def test_window_refusals(change, status):
    assert window(**change) == status


def test_window_workspace():
    def size(**kw):
        a = dict(batch=2, mb=40, nq=1, w=200, s=4, cfg=CFG)
        a.update(kw)
        return K.kvarn_window_workspace_bytes(a["cfg"], a["batch"], a["mb"], a["nq"], a["w"], a["s"])
    # one query of a small call: clusters merge in shared memory
    assert size() == 16
    # a larger one: partial rows of 132 floats for 8 queries of each unit, per split and for the open tile
    splits, rest = divmod(size(batch=200, w=4096), 200 * 8 * 8 * 132 * 4)
    assert rest == 0 and 2 <= splits <= 6
    assert size(batch=200, w=2 ** 31 - 1, s=2 ** 31 - 1) == size(batch=200, w=128 * 40, s=0)  # no more than the table
    # 16 queries x 8 heads = one row block of up to 1 + (200 + 14) // 128 + 2 = 4 tiles
    splits, rest = divmod(size(nq=16), 2 * 8 * 128 * 132 * 4)
    assert rest == 0 and 2 <= splits <= 5
    for bad in (dict(w=0), dict(s=-1), dict(nq=0), dict(mb=0), dict(batch=-1), dict(cfg=BAD)):
        assert size(**bad) == 0
    assert window(size=size() - 1) == INV
    assert window(batch=200, window=4096, size=size(batch=200, w=4096) - 1) == INV
    assert window(nq=16, size=size(nq=16) - 1) == INV


def tree(cfg=CFG, q=16, k=16, v=16, mask=16, n=8, counts=None, table=16, mb=40, lens=16, batch=2, pool=16, tail=16,
         out=16, kind=1, ws=16, size=1 << 40):
    return K.kvarn_tree_attention(cfg, q, k, v, mask, n, counts, table, mb, lens, batch, pool, tail, 0.1, out, kind,
                                  ws, size, 16, stream=0, check=False)


@pytest.mark.parametrize("change,status", [
    (dict(cfg=BAD), UNS), (dict(n=0), INV), (dict(n=129), UNS), (dict(mb=0), INV), (dict(mb=1 << 24), INV),
    (dict(batch=-1), INV), (dict(batch=65536), INV), (dict(kind=3), INV), (dict(q=None), INV), (dict(k=None), INV),
    (dict(v=None), INV), (dict(mask=None), INV), (dict(mask=20), INV), (dict(k=8), INV), (dict(v=24), INV),
    (dict(table=None), INV), (dict(lens=None), INV), (dict(pool=None), INV), (dict(tail=None), INV),
    (dict(out=8), INV), (dict(ws=None), INV), (dict(size=0), INV), (dict(batch=0, q=None), 0),
])
def test_tree_refusals(change, status):
    assert tree(**change) == status


def test_tree_workspace():
    # partial rows of 132 floats: 128 per row block (16 nodes x 8 heads fill one) and KV head, for each split of the
    # 40 tiles (at least one, at most a tile each) and for the raw tokens
    for nodes, blocks in ((1, 1), (16, 1), (17, 2), (128, 8)):
        size = K.kvarn_tree_workspace_bytes(CFG, 2, 40, nodes)
        splits, rest = divmod(size, 2 * 8 * blocks * 128 * 132 * 4)
        assert rest == 0 and 2 <= splits <= 41
    for bad in ((BAD, 2, 40, 16), (CFG, -1, 40, 16), (CFG, 2, 0, 16), (CFG, 2, 40, 0), (CFG, 2, 40, 129)):
        assert K.kvarn_tree_workspace_bytes(*bad) == 0
    assert tree(n=16, size=K.kvarn_tree_workspace_bytes(CFG, 2, 40, 16) - 1) == INV


def commit(cfg=CFG, k=16, v=16, n=8, path=16, mp=5, plens=16, pos=16, table=16, mb=40, batch=2, tail=16, pool=16):
    return K.kvarn_commit_tokens(cfg, k, v, n, path, mp, plens, pos, table, mb, batch, tail, pool, 16, stream=0,
                                 check=False)


@pytest.mark.parametrize("change,status", [
    (dict(cfg=BAD), UNS), (dict(n=0), INV), (dict(mp=0), INV), (dict(mp=129), UNS), (dict(path=None, mp=9), INV),
    (dict(k=None), INV), (dict(v=8), INV), (dict(plens=None), INV), (dict(pos=None), INV), (dict(table=None), INV),
    (dict(tail=None), INV), (dict(pool=None), INV), (dict(pool=8), INV), (dict(mb=0), INV), (dict(batch=-1), INV),
    (dict(batch=1 << 28), INV), (dict(batch=0, k=None), 0),
])
def test_commit_refusals(change, status):
    assert commit(**change) == status


def test_pages_refusals():
    ws = K.kvarn_pages_workspace_bytes(CFG, 4)
    assert ws == 4 * 104 and K.kvarn_pages_workspace_bytes(BAD, 4) == 0 and K.kvarn_pages_workspace_bytes(CFG, -1) == 0

    def alloc(cfg=CFG, table=16, mb=40, batch=4, begin=16, end=16, refs=16, w=16, size=ws):
        return K.kvarn_alloc_blocks(cfg, table, mb, batch, begin, end, refs, w, size, 16, stream=0, check=False)
    for bad in (dict(table=None), dict(mb=0), dict(batch=-1), dict(begin=None), dict(end=None), dict(refs=None),
                dict(refs=8), dict(w=None), dict(w=8), dict(size=ws - 1), dict(batch=1 << 27), dict(mb=1 << 24)):
        assert alloc(**bad) == INV, bad
    assert alloc(cfg=BAD) == UNS and alloc(batch=0, table=None) == 0

    def free(table=16, mb=40, batch=4, begin=16, end=16, refs=16):
        return K.kvarn_free_blocks(CFG, table, mb, batch, begin, end, refs, 16, stream=0, check=False)
    for bad in (dict(table=None), dict(mb=0), dict(batch=-1), dict(begin=None), dict(end=None), dict(refs=None)):
        assert free(**bad) == INV, bad
    assert free(batch=0, refs=None) == 0

    def tails(parent=16, group=2, batch=4, lens=16, mb=40, tail=16):
        return K.kvarn_fork_tails(CFG, parent, group, batch, lens, mb, tail, 16, stream=0, check=False)
    for bad in (dict(parent=None), dict(group=0), dict(batch=-1), dict(lens=None), dict(mb=0), dict(tail=None),
                dict(tail=8)):
        assert tails(**bad) == INV, bad
    assert tails(group=1025) == UNS and tails(group=1, batch=65536) == UNS and tails(batch=0, tail=None) == 0

    def seqs(parent=16, group=2, batch=4, table=16, mb=40, lens=16, refs=16):
        return K.kvarn_fork_sequences(CFG, parent, group, batch, table, mb, lens, refs, 16, stream=0, check=False)
    for bad in (dict(parent=None), dict(group=0), dict(lens=None), dict(table=None), dict(refs=None), dict(mb=0)):
        assert seqs(**bad) == INV, bad
    assert seqs(group=1025) == UNS

    def compact(table=16, mb=40, batch=4, refs=16, src=16, dst=16, counts=16, w=16, size=ws):
        return K.kvarn_compact_blocks(CFG, table, mb, batch, refs, src, dst, counts, w, size, 16, stream=0,
                                      check=False)
    for bad in (dict(table=None), dict(refs=None), dict(src=None), dict(dst=None), dict(counts=None), dict(w=None),
                dict(size=ws - 1), dict(batch=0, refs=None)):
        assert compact(**bad) == INV, bad

    def copy(src=16, blocks=9, a=16, dst=16, b=16, n=3):
        return K.kvarn_copy_blocks(CFG, src, blocks, a, dst, b, n, None, 16, stream=0, check=False)
    for bad in (dict(src=None), dict(blocks=-1), dict(a=None), dict(dst=None), dict(b=None), dict(n=-1), dict(src=8),
                dict(dst=4)):
        assert copy(**bad) == INV, bad
    assert copy(n=0, a=None) == 0


def test_strided_tensors_are_refused():
    x = torch.zeros(4, 4, dtype=torch.int32).t()
    x = x[:, ::2]
    with pytest.raises(ValueError, match="contiguous"):
        K.kvarn_free_blocks(CFG, x, 2, 4, 16, 16, 16, 16, stream=0)


def test_tensors_of_another_type_or_on_the_host_are_refused():
    wide = torch.zeros(2, 4, dtype=torch.int64)
    with pytest.raises(ValueError, match="int32"):
        K.kvarn_free_blocks(CFG, wide, 4, 2, 16, 16, 16, 16, stream=0)
    host = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="on the GPU"):
        K.kvarn_free_blocks(CFG, host, 4, 2, 16, 16, 16, 16, stream=0)
    q = torch.zeros(2, 1, 64, 128, dtype=torch.float16)
    with pytest.raises(ValueError, match="on the GPU"):
        K.kvarn_window_attention(CFG, q, 1, 16, 40, 16, 2, 200, 4, 16, 16, 0.1, 16, 0, 16, 1 << 40, 16, stream=0)


def test_calls_of_many_shapes_share_workspaces():
    """A workspace is kept for good (a captured graph may hold its address),
    so a server's many chunk lengths must not make one each."""
    c = PagedCache(I.Workload("ws", 2, 8, 2, "f16", [300, 200], seed=1, max_tokens=301), "cpu")
    seen = {}
    for need in list(range(1000, 3000000, 7777)) + list(range(3000000, 1000, -9999)):
        ws = c._workspace("window", need)
        assert ws.numel() >= need
        seen[ws.data_ptr()] = ws.numel()
    assert len(seen) <= 8 and sum(seen.values()) <= 4 * 3000000
    assert c._workspace("window", 100).data_ptr() in seen
    big = c._workspace("tree", 1 << 20)
    assert big.data_ptr() not in seen and c._workspace("tree", 5).data_ptr() == big.data_ptr()


def test_pages_of_an_empty_pool_have_a_workspace():
    """Its one chunk count is stored as any other."""
    cfg = K.make_config(8, 64, 0, "f16")
    assert K.kvarn_pages_workspace_bytes(cfg, 4) == 16

    def compact(size):
        return K.kvarn_compact_blocks(cfg, 16, 40, 4, None, None, None, 16, 16, size, 16, stream=0, check=False)
    assert compact(0) == INV and compact(15) == INV


def test_what_a_call_makes_is_made_on_its_stream(monkeypatch):
    """Ranges, counts and workspaces that a call with stream= makes by torch
    are ordered with its kernels: made while that stream is the current one."""
    import contextlib
    active, made = [], []

    @contextlib.contextmanager
    def stream(s):
        active.append(s)
        yield
        active.pop()

    def noted(name):
        real = getattr(torch, name)

        def f(*a, **kw):
            made.append((name, active[-1] if active else None))
            return real(*a, **kw)
        return f
    w = I.Workload("streams", 2, 8, 2, "f16", [300, 200], seed=1, max_tokens=301)
    c = PagedCache(w, "cpu")
    q = torch.zeros(2, 3, 8, 128, dtype=torch.float16)
    kv = torch.zeros(2, 3, 2, 128, dtype=torch.float16)
    mask, parent = torch.zeros(2, 3, 1, dtype=torch.int64), torch.zeros(2, dtype=torch.int32)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    for name in ("full_like", "bincount", "zeros", "empty"):
        monkeypatch.setattr(torch, name, noted(name))
    for name in K.EXPORTS:
        if not name.endswith("_bytes"):
            monkeypatch.setattr(K, name, lambda *a, **kw: 0)
    s = object()
    for call in (lambda: c.free_behind_window(c.lens, 100, 4, stream=s), lambda: c.compact(stream=s),
                 lambda: c.window(q, 3, q, 100, stream=s), lambda: c.tree(q, kv, kv, mask, q, stream=s)):
        made.clear()
        call()
        assert made and all(at is s for _, at in made), made
    c._kept.clear()
    for call in (lambda: c.alloc(parent, parent, stream=s), lambda: c.fork(parent, 2, stream=s)):
        c._kept.pop("refs", None)
        made.clear()
        call()
        assert made and all(at is s for _, at in made), made


class Elsewhere:
    """Stands for an int32 tensor on the second GPU."""
    dtype, device, is_cuda, shape = torch.int32, torch.device("cuda:1"), True, (4,)

    def get_device(self):
        return 1

    def is_contiguous(self):
        return True

    def stride(self):
        return (1,)

    def data_ptr(self):
        return 16


CALLS = {  # arguments of each call; 16 stands for a device pointer
    "kvarn_window_attention": (16, 1, 16, 40, 16, 0, 200, 4, 16, 16, 0.1, 16, 0, 16, 1 << 40, 16),
    "kvarn_tree_attention": (16, 16, 16, 16, 8, 16, 16, 40, 16, 0, 16, 16, 0.1, 16, 1, 16, 1 << 40, 16),
    "kvarn_commit_tokens": (16, 16, 8, 16, 5, 16, 16, 16, 40, 0, 16, 16, 16),
    "kvarn_alloc_blocks": (16, 40, 0, 16, 16, 16, 16, 1 << 40, 16),
    "kvarn_free_blocks": (16, 40, 0, 16, 16, 16, 16),
    "kvarn_fork_tails": (16, 2, 0, 16, 40, 16, 16),
    "kvarn_fork_sequences": (16, 2, 0, 16, 40, 16, 16, 16),
    "kvarn_compact_blocks": (16, 40, 0, 16, 16, 16, 16, 16, 1 << 40, 16),
    "kvarn_copy_blocks": (16, 9, 16, 16, 16, 0, 16, 16),
}


@pytest.mark.parametrize("name", CALLS)
def test_every_tensor_has_to_lie_on_the_current_device(name, monkeypatch):
    monkeypatch.setattr(K, "_here", lambda: 0, raising=False)
    call, args = getattr(K, name), CALLS[name]
    assert call(BAD, *args, stream=0, check=False) == UNS  # (a configuration that the library refuses: no launch)
    for i, x in enumerate(args):
        if x == 16:
            with pytest.raises(ValueError, match="cuda:1, but the current device is cuda:0"):
                call(BAD, *args[:i], Elsewhere(), *args[i + 1:], stream=0, check=False)
    monkeypatch.setattr(K, "_here", lambda: 1, raising=False)
    assert call(BAD, *(Elsewhere() if x == 16 else x for x in args), stream=0, check=False) == UNS


def test_index_arrays_have_an_entry_per_sequence(monkeypatch):
    """A shorter array would be read past its end on the device."""
    for name in K.EXPORTS:
        if not name.endswith("_bytes"):
            monkeypatch.setattr(K, name, lambda *a, **kw: 0)
    c = PagedCache(I.Workload("short", 3, 8, 2, "f16", [300, 200, 1], seed=1, max_tokens=301), "cpu")
    q, kv = torch.zeros(3, 4, 8, 128, dtype=torch.float16), torch.zeros(3, 4, 2, 128, dtype=torch.float16)
    mask, path = torch.zeros(3, 4, 1, dtype=torch.int64), torch.zeros(3, 2, dtype=torch.int32)
    good = torch.zeros(3, dtype=torch.int32)
    calls = {
        "lens": [lambda x: c.window(q, 4, q, 100, lens=x), lambda x: c.tree(q, kv, kv, mask, q, lens=x),
                 lambda x: c.fork(good, 3, lens=x), lambda x: c.free_behind_window(x, 100)],
        "counts": [lambda x: c.tree(q, kv, kv, mask, q, counts=x)],
        "path_lens": [lambda x: c.commit(kv, kv, path, x, good)],
        "pos": [lambda x: c.commit(kv, kv, None, good, x)],
        "tile_begin": [lambda x: c.alloc(x, good), lambda x: c.free(x, good)],
        "tile_end": [lambda x: c.alloc(good, x), lambda x: c.free(good, x)],
        "parent": [lambda x: c.fork(x, 3)],
    }
    for name, each in calls.items():
        for call in each:
            call(good)
            for bad in (good[:2], torch.zeros(4, dtype=torch.int32), torch.zeros((), dtype=torch.int32)):
                with pytest.raises(ValueError, match=name):
                    call(bad)
    c.commit(kv, kv, path, good, good)
    with pytest.raises(ValueError, match="path"):
        c.commit(kv, kv, path[:2], good, good)


@pytest.mark.parametrize("window,n_sinks", [(0, 0), (-300, 0), (100, -1)])
def test_no_release_behind_an_impossible_window(window, n_sinks, monkeypatch):
    monkeypatch.setattr(K, "kvarn_free_blocks", lambda *a, **kw: 0)
    c = PagedCache(I.Workload("behind", 2, 8, 2, "f16", [300, 200], seed=1, max_tokens=301), "cpu")
    c.free_behind_window(c.lens, 100, 0)
    with pytest.raises(ValueError, match="window >= 1"):
        c.free_behind_window(c.lens, window, n_sinks)
