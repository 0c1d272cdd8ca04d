"""The serving operators write what they are asked to and nothing else: every
buffer a call may write lies between guard bytes, every one it only reads is
compared afterwards, workspaces have exactly the size asked for; and the
checked build (every access tested against its buffer) reports nothing and
gives the same bits."""
import numpy as np
import pytest
import torch

from bit_kv_cache_quantize_gb300 import build as B
from bit_kv_cache_quantize_gb300 import inputs as I
from bit_kv_cache_quantize_gb300 import kvarn as K
from bit_kv_cache_quantize_gb300.cache import PagedCache

from gpu_helpers import device
from serving_ref import normal16
from test_gpu_canaries import Guarded
from test_gpu_checked_build import library

pytestmark = pytest.mark.gpu
T = D = 128


def load(lens, dtype="f16", h=2, g=5, kb=4, vb=2, steps=0):
    return I.Workload("guards", len(lens), h * g, h, dtype, lens, seed=700, max_tokens=max(lens) + 1, block_perm=True,
                      k_bits=kb, v_bits=vb, decode_steps=steps)


LENS = [300, 130, 0, 255, 900]


def drafts(w, n, dev):
    mask = torch.full((w.batch, n, (n + 63) // 64), -1, dtype=torch.int64, device=dev)
    return (normal16(1, (w.batch, n, w.num_q_heads, D), w.dtype, dev),
            normal16(2, (w.batch, n, w.num_kv_heads, D), w.dtype, dev),
            normal16(3, (w.batch, n, w.num_kv_heads, D), w.dtype, dev), mask)


class Held:
    """Guarded copies of tensors a call writes; fingerprints of those it reads."""

    def __init__(self, dev):
        self.dev, self.guarded, self.read = dev, [], []

    def writes(self, x, name):
        g = Guarded(x.numel() * x.element_size(), self.dev)
        v = g.view(x.dtype).view(x.shape)
        v.copy_(x)
        self.guarded.append((g, name))
        return v

    def reads(self, x, name):
        self.read.append((x, x.clone(), name))
        return x

    def space(self, n):
        g = Guarded(n, self.dev)
        self.guarded.append((g, "workspace"))
        return g.view()

    def check(self, err):
        torch.cuda.synchronize()
        assert int(err[0]) == 0
        for g, name in self.guarded:
            g.check(name)
        for x, was, name in self.read:
            assert torch.equal(x.reshape(-1).view(torch.uint8), was.reshape(-1).view(torch.uint8)), f"{name} was written"


@pytest.mark.parametrize("n", [1, 5, 70])
@pytest.mark.parametrize("dtype,out16,kb,vb", [("f16", False, 4, 4), ("bf16", True, 2, 2)])
def test_attention_writes_its_rows_and_workspace(n, dtype, out16, kb, vb):
    dev = device()
    lens = [max(m, n) if m else 0 for m in LENS]
    w = load(lens, dtype, kb=kb, vb=vb)
    c = PagedCache(w, dev)
    c.prefill()
    q, k, v, mask = drafts(w, n, dev)
    kind = K.KVARN_OUT_16 if out16 else K.KVARN_OUT_F32
    h = Held(dev)
    for x, name in ((q, "q"), (k, "k_draft"), (v, "v_draft"), (mask, "mask"), (c.pool, "pool"), (c.tail, "tail"),
                    (c.table, "table"), (c.lens, "lens")):
        h.reads(x, name)
    err = h.writes(c.err, "dev_err")
    plain = torch.zeros(w.batch, n, w.num_q_heads, D, dtype=I.torch_dtype(dtype) if out16 else torch.float32, device=dev)
    for window, sinks in ((260, 130), (5, 0)):
        need = K.kvarn_window_workspace_bytes(c.cfg, w.batch, c.max_blocks, n, window, sinks)
        out = h.writes(plain, "window out")
        K.kvarn_window_attention(c.cfg, q, n, c.table, c.max_blocks, c.lens, w.batch, window, sinks, c.pool, c.tail,
                                 w.scale, out, kind, h.space(need), need, err)
    need = K.kvarn_tree_workspace_bytes(c.cfg, w.batch, c.max_blocks, n)
    out = h.writes(plain, "tree out")
    counts = h.reads(torch.tensor([n, 0, 1, n // 2, n], dtype=torch.int32, device=dev), "counts")
    K.kvarn_tree_attention(c.cfg, q, k, v, mask, n, counts, c.table, c.max_blocks, c.lens, w.batch, c.pool, c.tail,
                           w.scale, out, kind, h.space(need), need, err)
    h.check(err)
    assert not out[1].any() and not out[3, n // 2:].any()


def test_commit_and_pages_write_their_entries():
    dev = device()
    w = load(LENS, steps=130)
    c = PagedCache(w, dev, extra_blocks=6)
    c.prefill()
    n = 128
    _, k, v, _ = drafts(w, n, dev)
    h = Held(dev)
    for x, name in ((k, "k_draft"), (v, "v_draft")):
        h.reads(x, name)
    err, pool, tail = h.writes(c.err, "dev_err"), h.writes(c.pool, "pool"), h.writes(c.tail, "tail")
    path = h.reads(torch.arange(n, dtype=torch.int32, device=dev).repeat(w.batch, 1), "path")
    plens = h.reads(torch.tensor([128, 0, 127, 1, 5], dtype=torch.int32, device=dev), "path_lens")
    pos = h.reads(c.lens.clone(), "pos")
    K.kvarn_commit_tokens(c.cfg, k, v, n, path, n, plens, pos, h.reads(c.table, "table"), c.max_blocks, w.batch, tail,
                          pool, err)
    h.check(err)
    closed = {int(c.table[0, 2]), int(c.table[3, 1])}  # 300 + 128 and 255 + 1 pass a tile's end
    a, b = pool.view(c.num_blocks, -1), c.pool.view(c.num_blocks, -1)
    assert {i for i in range(c.num_blocks) if not torch.equal(a[i], b[i])} <= closed
    assert torch.equal(tail[1], c.tail[1])
    # pages: tails, table, counts and lengths between guards
    h = Held(dev)
    err, pool, tail = h.writes(c.err, "dev_err"), h.writes(c.pool, "pool"), h.writes(c.tail, "tail")
    table, refs, lens = h.writes(c.table, "table"), h.writes(c.refs, "refs"), h.writes(c.lens, "lens")
    parent = h.reads(torch.tensor([0, 0, 4, 4, 4], dtype=torch.int32, device=dev), "parent")
    K.kvarn_fork_tails(c.cfg, parent, 5, w.batch, lens, c.max_blocks, tail, err)
    K.kvarn_fork_sequences(c.cfg, parent, 5, w.batch, table, c.max_blocks, lens, refs, err)
    need = K.kvarn_pages_workspace_bytes(c.cfg, w.batch)
    begin = h.reads((lens // T).clone(), "begin")
    end = h.reads((lens // T + 1).clamp_max(c.max_blocks).clone(), "end")
    K.kvarn_alloc_blocks(c.cfg, table, c.max_blocks, w.batch, begin, end, refs, h.space(need), need, err)
    none = h.reads(torch.zeros(w.batch, dtype=torch.int32, device=dev), "tiles")
    one = h.reads(torch.tensor([1, 0, 1, 0, 1], dtype=torch.int32, device=dev), "tiles")
    K.kvarn_free_blocks(c.cfg, table, c.max_blocks, w.batch, none, one, refs, err)
    moves = [h.writes(torch.zeros(c.num_blocks, dtype=torch.int32, device=dev), "moves") for _ in range(2)]
    counts = h.writes(torch.zeros(2, dtype=torch.int32, device=dev), "counts")
    K.kvarn_compact_blocks(c.cfg, table, c.max_blocks, w.batch, refs, moves[0], moves[1], counts, h.space(need), need,
                           err)
    K.kvarn_copy_blocks(c.cfg, pool, c.num_blocks, moves[0], pool, moves[1], c.num_blocks, counts[1:], err)
    h.check(err)
    ids = table[table >= 0].cpu().numpy()
    assert (refs.cpu().numpy() == np.bincount(ids, minlength=c.num_blocks)).all()


def run_all(dtype, kb, vb, dev):
    """Every serving call once; all the bits it leaves."""
    lens = [300, 130, 0, 255, 900]
    w = load(lens, dtype, kb=kb, vb=vb, steps=130)
    c = PagedCache(w, dev, extra_blocks=4)
    c.prefill()
    c.refs
    bits = {}
    for n in (1, 9, 50):
        q, k, v, mask = drafts(w, n, dev)
        for t16 in (False, True):
            out = torch.zeros(w.batch, n, w.num_q_heads, D, dtype=I.torch_dtype(dtype) if t16 else torch.float32,
                              device=dev)
            c.tree(q, k, v, mask, out)
            bits["tree", n, t16] = out.clone()
            c.window(q, n, out, 200, 140)
            bits["window", n, t16] = out.clone()
    plens = torch.tensor([50, 0, 3, 1, 42], dtype=torch.int32, device=dev)
    c.commit(k, v, None, plens, c.lens)
    c.lens += plens
    c.fork(torch.tensor([0, 0, 2, 4, 4], dtype=torch.int32, device=dev), 5)
    c.alloc(c.lens // T, (c.lens // T + 1).clamp_max(c.max_blocks))
    c.free_behind_window(c.lens, 200, 140)
    bits["counts"] = c.compact().clone()
    bits.update(table=c.table.clone(), refs=c.refs.clone(), lens=c.lens.clone(), pool=c.pool.clone(), tail=c.tail.clone())
    torch.cuda.synchronize()
    assert c.check_error() == 0
    return bits


@pytest.mark.parametrize("dtype,kb,vb", [("f16", 4, 2), ("bf16", 4, 4), ("f16", 2, 2)])
def test_checked_build_reports_nothing_and_gives_the_same_bits(dtype, kb, vb):
    dev = device()
    plain = run_all(dtype, kb, vb, dev)
    with library(B.build_checked()):
        checked = run_all(dtype, kb, vb, dev)
    for key, x in plain.items():
        assert torch.equal(x.reshape(-1).view(torch.uint8), checked[key].reshape(-1).view(torch.uint8)), key


def test_compaction_of_an_empty_pool_stays_in_its_workspace():
    dev = device()
    cfg = K.make_config(2, 4, 0, "f16")
    h = Held(dev)
    err = h.writes(torch.zeros(1, dtype=torch.int32, device=dev), "dev_err")
    table = h.reads(torch.full((3, 5), -1, dtype=torch.int32, device=dev), "table")
    counts = h.writes(torch.full((2,), 7, dtype=torch.int32, device=dev), "counts")
    need = K.kvarn_pages_workspace_bytes(cfg, 3)
    K.kvarn_compact_blocks(cfg, table, 5, 3, None, None, None, counts, h.space(need), need, err)
    h.check(err)
    assert counts.tolist() == [0, 0]
