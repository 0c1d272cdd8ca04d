"""Rows that see nothing, and rows whose every score is NaN or -inf: the first
give zeros whatever their queries hold, the second NaN, as the formula says,
however the tokens are split over warps, CTAs and clusters."""
import numpy as np
import pytest
import torch

from bit_kv_cache_quantize_gb300 import inputs as I
from bit_kv_cache_quantize_gb300 import kvarn as K
from bit_kv_cache_quantize_gb300.cache import PagedCache

from gpu_helpers import device
from serving_ref import cache64, host64, normal16, tolerance
from test_gpu_tree import pack
from test_gpu_window import visible

pytestmark = pytest.mark.gpu
T = D = 128
NAN, INF = float("nan"), float("inf")


def load(lens, dtype="f16", h=1, g=4, kb=4, vb=2):
    return I.Workload("nonfinite", len(lens), h * g, h, dtype, lens, seed=900, max_tokens=max(lens), block_perm=True,
                      k_bits=kb, v_bits=vb)


def formula(q, Kc, Vc, see, scale):
    """attend64 with IEEE arithmetic throughout: a NaN or an infinity goes
    where the formula takes it; a row that sees nothing is zeros."""
    out = np.zeros_like(q)
    with np.errstate(invalid="ignore", over="ignore"):
        for r in range(q.shape[0]):
            idx = np.flatnonzero(see[r])
            if idx.size:
                s = (Kc[idx] * q[r]).sum(1) * scale
                p = np.exp(s - s.max())
                out[r] = (p[:, None] * Vc[idx]).sum(0) / p.sum()
    return out


def check(c, q, out, see_of, kd=None, vd=None):
    """Every row: NaN and infinities where the formula has them, its value elsewhere."""
    w, n = c.w, q.shape[1]
    torch.cuda.synchronize()
    assert c.check_error() == 0
    pool, tail, table = c.pool.cpu().numpy(), c.tail.cpu(), c.table.cpu().numpy()
    got = out.double().cpu().numpy()
    eps = 0.0 if out.dtype == torch.float32 else torch.finfo(out.dtype).eps
    single = out.dtype == torch.bfloat16 and (n > 1 or kd is not None)
    qh = host64(q, w.dtype).reshape(q.shape)
    for b in range(w.batch):
        m = w.seq_lens[b]
        see = see_of(b)
        for h in range(w.num_kv_heads):
            Kc, Vc = cache64(c, b, h, m, pool, tail, table) if m else (np.zeros((0, D)), np.zeros((0, D)))
            if kd is not None:
                Kc = np.concatenate([Kc, host64(kd, w.dtype).reshape(kd.shape)[b, :, h]])
                Vc = np.concatenate([Vc, host64(vd, w.dtype).reshape(vd.shape)[b, :, h]])
            for g in range(w.G):
                rows = qh[b, :, h * w.G + g]
                want = formula(rows, Kc, Vc, see, w.scale)
                have = got[b, :, h * w.G + g]
                for r in range(n):
                    if not see[r].any():
                        assert not have[r].any(), (b, h, g, r)
                        continue
                    fin = np.isfinite(want[r])
                    assert (np.isnan(have[r]) == np.isnan(want[r])).all(), (b, h, g, r)
                    assert (have[r][~fin & ~np.isnan(want[r])] == want[r][~fin & ~np.isnan(want[r])]).all(), (b, h, g, r)
                    if fin.any():
                        s1 = see[r:r + 1] & np.isfinite(Kc).all(1)[None]  # a weight of e^-inf adds nothing
                        tol = tolerance(rows[r:r + 1], Kc, Vc, s1, w.scale, eps, want[r:r + 1], single)
                        assert (np.abs(have[r] - want[r])[fin] <= np.broadcast_to(tol[0], (D,))[fin]).all(), (b, h, g, r)


def output(w, n, out16=False):
    return torch.full((w.batch, n, w.num_q_heads, D), 7.0, dtype=I.torch_dtype(w.dtype) if out16 else torch.float32,
                      device="cuda")


def filled(w, past=True):
    c = PagedCache(w, device())
    c.prefill()
    if past:  # slots behind each length hold NaN
        for b, m in enumerate(w.seq_lens):
            c.tail[b, :, :, m % T:] = NAN
    return c


@pytest.mark.parametrize("lens,n", [([0, 300, 0, 700], 1), ([0, 90, 1] * 40, 1),       # a cluster, a split over CTAs
                                    ([0, 100, 0, 128], 6), ([0, 300, 0, 700], 6)])     # one chunk, several
@pytest.mark.parametrize("dtype,out16", [("f16", False), ("bf16", True)])
def test_empty_slots_give_zeros_whatever_their_queries_hold(lens, n, dtype, out16):
    w = load([max(m, n) if m else 0 for m in lens], dtype, h=2 if len(lens) == 4 else 4, g=2)
    c = filled(w)
    need = K.kvarn_window_workspace_bytes(c.cfg, w.batch, c.max_blocks, n, 100, 4)
    if n > 1:  # a packed and a raw partial per unit where one chunk holds all tiles
        assert (need == 2 * w.batch * w.num_kv_heads * 128 * 132 * 4) == (max(lens) <= T)
    else:
        assert (need == 16) == (len(lens) == 4)
    q = I.multi_queries(w, n, device="cuda").reshape(w.batch, n, w.num_q_heads, D)
    q[0] = NAN
    q[2, :, :, 5] = INF
    out = output(w, n, out16)
    c.window(q, n, out, 100, 4)
    check(c, q, out, lambda b: visible(w.seq_lens[b], n, 100, 4) if w.seq_lens[b] else np.zeros((n, 0), bool))


@pytest.mark.parametrize("lens", [[0, 100], [0, 300]])  # one chunk; several
@pytest.mark.parametrize("dtype,out16", [("f16", True), ("bf16", False)])
def test_tree_rows_that_see_nothing_give_zeros_whatever_their_queries_hold(lens, dtype, out16):
    w, n = load(lens, dtype, h=2, g=2), 9
    c = filled(w)
    kd, vd = (normal16(s, (2, n, 2, D), dtype) for s in (1, 2))
    see = np.random.default_rng(3).random((2, n, n)) < 0.4
    see[0, [0, 4, 8]] = False
    see[0, 1, 1] = True
    q = I.multi_queries(w, n, device="cuda").reshape(2, n, 4, D)
    q[0, 4], q[0, 8, :, 3] = NAN, -INF
    out = output(w, n, out16)
    c.tree(q, kd, vd, pack(see).cuda(), out)
    assert not out[0, [0, 4, 8]].any()
    check(c, q, out, lambda b: np.concatenate([np.ones((n, lens[b]), bool), see[b]], 1), kd, vd)


@pytest.mark.parametrize("key", [NAN, -INF])
@pytest.mark.parametrize("dtype,out16", [("f16", False), ("bf16", True)])
@pytest.mark.parametrize("n,lens,window,at", [
    (1, [129, 257], 200, -1),        # the open tile holds the key alone: a cluster's last CTA
    (1, [129, 257] * 45, 200, -1),   # ... and a partial of its own in the workspace
    (1, [100, 200], 1, -1),          # the row sees nothing else
    (1, [50, 77], 60, -30),          # one of many tokens
    (2, [161, 33], 300, 32),         # the second half of a row group's tokens holds it alone
    (40, [161, 289], 300, 32),
    (3, [70, 200], 1, -1),           # the last row sees nothing else
])
def test_a_key_that_is_not_finite_reaches_every_row_that_sees_it(key, dtype, out16, n, lens, window, at):
    w = load(lens, dtype, h=1 if len(lens) == 2 else 4, g=4 if n < 40 else 1)
    c = filled(w)
    q = I.multi_queries(w, n, device="cuda").reshape(w.batch, n, w.num_q_heads, D)
    q[..., 11] = 1.0
    for b, m in enumerate(lens):
        c.tail[b, :, 0, at % (m % T), 11] = key
    out = output(w, n, out16)
    c.window(q, n, out, window, 0)
    check(c, q, out, lambda b: visible(lens[b], n, window, 0))


@pytest.mark.parametrize("key", [NAN, -INF])
@pytest.mark.parametrize("dtype,out16", [("f16", False), ("bf16", True)])
@pytest.mark.parametrize("lens", [[0, 100], [128, 200]])
def test_a_node_whose_key_is_not_finite_reaches_every_row_that_sees_it(key, dtype, out16, lens):
    """40 rows of one head: two warps share a row group, nodes 32 .. 39 fall to the second."""
    w, n = load(lens, dtype, h=1, g=1), 40
    c = filled(w)
    kd, vd = (normal16(s, (2, n, 1, D), dtype) for s in (1, 2))
    see = np.zeros((2, n, n), bool)
    see[:, :, 2] = see[:, :, 20] = True
    see[:, 33, 35] = True                    # alone in the second half, with others in the first
    see[:, 7] = False
    see[:, 7, 35] = True                     # alone
    see[:, 9, 30:40] = True                  # one of many
    kd[:, 35, 0, 11] = key
    q = I.multi_queries(w, n, device="cuda").reshape(2, n, 1, D)
    q[..., 11] = 1.0
    out = output(w, n, out16)
    c.tree(q, kd, vd, pack(see).cuda(), out)
    check(c, q, out, lambda b: np.concatenate([np.ones((n, lens[b]), bool), see[b]], 1), kd, vd)


@pytest.mark.parametrize("kind,n", [("window", 1), ("window", 5), ("tree", 5)])
@pytest.mark.parametrize("dtype,out16", [("f16", False), ("bf16", True)])
def test_a_query_that_is_not_finite_gives_nan_in_closed_tiles_alone(kind, n, dtype, out16):
    """Lengths of whole tiles: no raw part; the infinity's scores are of both signs."""
    w = load([128, 384], dtype, h=2, g=2)
    c = filled(w, past=False)
    q = I.multi_queries(w, n, device="cuda").reshape(2, n, 4, D)
    q[0, 0, 1, 7], q[1, n - 1, 2, 100] = NAN, INF
    kd, vd = (normal16(s, (2, n, 2, D), dtype) for s in (1, 2))
    out = output(w, n, out16)
    if kind == "tree":
        c.tree(q, kd, vd, torch.zeros(2, n, 1, dtype=torch.int64, device="cuda"), out)
    else:
        c.window(q, n, out, 1000, 0)
    torch.cuda.synchronize()
    assert c.check_error() == 0
    bad = torch.zeros(2, n, 4, dtype=torch.bool)
    bad[0, 0, 1] = bad[1, n - 1, 2] = True
    assert (torch.isnan(out).all(-1).cpu() == bad).all() and (torch.isfinite(out).all(-1).cpu() == ~bad).all()


@pytest.mark.parametrize("n,lens", [(1, [300, 129]), (1, [300, 129] * 45), (1, [127, 60]), (4, [300, 133]),
                                    (40, [300, 127])])
@pytest.mark.parametrize("dtype,out16", [("f16", False), ("bf16", True)])
def test_values_that_are_not_finite_reach_their_channel_of_the_rows_that_see_them(n, lens, dtype, out16):
    """Infinities stay infinities, both signs in one channel and NaNs give
    NaN, and the other channels keep their values."""
    w = load(lens, dtype, h=1 if len(lens) == 2 else 4, g=5 if n < 40 else 3)
    c = filled(w)
    for b, m in enumerate(lens):
        first = m - m % T
        for pos, channel, x in ((m - 1, 3, INF), (m - 1, 100, -INF), (m - 20, 0, NAN), (m - 33, 127, -INF),
                                (m - 40, 50, INF), (m - 41, 50, -INF)):
            if pos >= first:
                c.tail[b, :, 1, pos % T, channel] = x
    q = I.multi_queries(w, n, device="cuda").reshape(w.batch, n, w.num_q_heads, D)
    out = output(w, n, out16)
    for window in (1, 30, 200):
        c.window(q, n, out, window, 0)
        check(c, q, out, lambda b: visible(lens[b], n, window, 0))


@pytest.mark.parametrize("kind,n,batch", [("window", 1, 2), ("window", 1, 90), ("window", 4, 2), ("tree", 4, 2)])
@pytest.mark.parametrize("dtype,out16", [("f16", False), ("bf16", True)])
@pytest.mark.parametrize("near", [False, True])
def test_values_of_weight_zero_are_not_lost(kind, n, batch, dtype, out16, near):
    """A closed tile's scores (near: also those of two open-tile tokens) lie
    hundreds of powers of two above the open tile's, so those weights are 0 in
    fp32; what is not finite there still reaches the rows that see it (as 0
    times it: NaN)."""
    w = load([128 + 40] * batch, dtype, h=1 if batch == 2 else 4, g=2)
    c = PagedCache(w, device())
    u = torch.from_numpy(np.where(np.random.default_rng(1).random(D) < 0.5, 1.0, -1.0)).cuda()
    for b in range(batch):
        k = normal16(b, (168, w.num_kv_heads, D), dtype)
        k[:T] = (8 * u + 0.05 * k[:T]).to(k.dtype)
        k[T:] *= 0.01
        if near:
            k[T + 6] = k[T + 36] = (8 * u).to(k.dtype)
        c.quantize_sequence(b, k, normal16(b + 99, (168, w.num_kv_heads, D), dtype))
    c.tail[0, :, 1, 5, 9] = INF
    c.tail[1, :, 1, 35, 33] = NAN
    q = (8 * u).to(I.torch_dtype(dtype)).expand(batch, n, w.num_q_heads, D).contiguous()
    kd, vd = (normal16(s, (batch, n, w.num_kv_heads, D), dtype) for s in (1, 2))
    vd[1, 2 % n, :, 70] = -INF
    out = output(w, n, out16)
    if kind == "tree":
        c.tree(q, kd, vd, torch.full((batch, n, 1), -1, dtype=torch.int64, device="cuda"), out)
    else:
        c.window(q, n, out, 400, 0)
    torch.cuda.synchronize()
    assert c.check_error() == 0
    bad = torch.zeros(batch, D, dtype=torch.bool)
    bad[0, 9] = bad[1, 33] = True
    bad[1, 70] = kind == "tree"
    assert ((~torch.isfinite(out)).cpu() == bad[:, None, None].expand(out.shape)).all()
