"""Every serving call with an explicit stream while torch's current stream is
busy: nothing a call makes or needs may wait for, or run ahead of, the wrong
stream.  Results equal those of the same calls on the current stream."""
import pytest
import torch

from bit_kv_cache_quantize_gb300 import inputs as I
from bit_kv_cache_quantize_gb300.cache import PagedCache

from gpu_helpers import device
from serving_ref import normal16

pytestmark = pytest.mark.gpu
T = D = 128


def calls(c, q, k, v, mask, after, outs, stream):
    """A step of every operator, each made for the first time; yields before each."""
    B, n = q.shape[:2]
    i32 = dict(dtype=torch.int32, device="cuda")
    plens, one, two = (torch.full((B,), x, **i32) for x in (n, 1, 2))
    begin, end = c.lens // T, after // T + 1
    parent = torch.tensor([1, 1, 3, 2] * (B // 4), **i32) + torch.arange(B, **i32) // 4 * 4
    q1 = q[:, :1].contiguous()
    torch.cuda.synchronize()
    yield
    c.alloc(begin, end, stream=stream)
    yield
    c.tree(q, k, v, mask, outs[0], stream=stream)
    yield
    c.commit(k, v, None, plens, c.lens, stream=stream)
    yield
    c.window(q, n, outs[1], 400, 3, lens=after, stream=stream)
    yield
    c.window(q1, 1, outs[2], 400, 3, lens=after, stream=stream)
    yield
    c.free_behind_window(after, 400, 3, stream=stream)
    yield
    c.fork(parent, 4, lens=after, stream=stream)
    yield
    c.free(one, two, stream=stream)
    yield
    c.compact(stream=stream)


def run(kind):
    dev = device()
    lens = [300, 1200, 77, 640] * 12
    w = I.Workload("streams", len(lens), 16, 8, "bf16", lens, seed=42, max_tokens=max(lens) + 9, block_perm=True,
                   decode_steps=140)
    c = PagedCache(w, dev, extra_blocks=200)
    c.prefill()
    for b, m in enumerate(lens):  # the tiles behind the contexts have no block yet
        c.table[b, m // T:] = -1
    n = 6
    q, k, v = (normal16(s, (w.batch, n, h, D), w.dtype) for s, h in ((1, 16), (2, 8), (3, 8)))
    mask = torch.full((w.batch, n, 1), 0b111111, dtype=torch.int64, device=dev)
    after = c.lens + n
    outs = [torch.zeros(w.batch, m, 16, D, dtype=torch.float32, device=dev) for m in (n, n, 1)]
    s = torch.cuda.Stream()
    stream = {"current": None, "stream": s, "handle": s.cuda_stream}[kind]
    a = torch.randn(8192, 8192, device=dev).bfloat16()
    other = torch.empty_like(a)
    for _ in calls(c, q, k, v, mask, after, outs, stream):
        if stream is not None:
            for _ in range(20):  # some 15 ms of work on the current stream
                torch.mm(a, a, out=other)
    if stream is not None:
        assert not torch.cuda.current_stream().query()  # still busy: nothing above waited for it
        s.synchronize()
    else:
        torch.cuda.synchronize()
    with torch.cuda.stream(s):
        left = [x.clone() for x in (*outs, c.table, c.refs, after, c.pool, c.tail, c.compact())]
        err = c.err.clone()
    torch.cuda.synchronize()
    assert int(err) == 0
    return left


@pytest.mark.parametrize("kind", ["stream", "handle"])
def test_calls_on_an_explicit_stream(kind):
    want = run("current")
    for i, (x, y) in enumerate(zip(want, run(kind))):
        assert torch.equal(x, y), i
