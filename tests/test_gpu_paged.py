"""Block tables and slot maps, the cache write and windowed decode on the GPU
against the plain oracle: whole values equal, attention within the bounds that
its roundings give."""
import numpy as np
import pytest
import torch

import fia_inputs
from attention_fia_prefill_gb300 import _binding
from oracle import paged_oracle as po
from oracle.fia_oracle import f64

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ block tables and slots
def _tables(fia, ctx, new, bs, W=None, free=None, n_tokens=None, fill=-7):
    rng = np.random.default_rng(len(ctx) + bs)
    tot = [max(a, 0) + max(b, 0) for a, b in zip(ctx, new)]
    W = max([-(-t // bs) for t in tot] + [1]) if W is None else W
    need = sum(-(-t // bs) for t in tot)
    ids = rng.permutation(need + 5)
    table = np.full((len(ctx), W), fill, dtype=np.int64)
    at = 0
    for b, c in enumerate(ctx):
        n = min(-(-max(c, 0) // bs), W)
        table[b, :n] = ids[at:at + n]
        at += n
    free = list(ids[at:]) if free is None else free
    T = sum(max(a, 0) for a in new) if n_tokens is None else n_tokens
    ref = po.block_table_append(ctx, new, free, table, bs, T)
    dt = torch.from_numpy(table).int().to(DEV)
    got = fia.fia_block_table_append(i32(ctx), i32(new), i32(free), dt, block_size=bs, num_tokens=T)
    torch.cuda.synchronize()
    assert np.array_equal(dt.cpu().numpy(), ref[0])
    for g, r in zip(got, ref[1:]):
        assert g.cpu().tolist() == (list(r) if not isinstance(r, int) else [r])
    return got, dt


@pytest.mark.parametrize("bs", [1, 16, 100, 128])
def test_tables_ragged(fia, bs):
    _tables(fia, [0, 1, bs - 1, bs, bs + 1, 3 * bs, 1000], [1, 0, 1, 1, 2 * bs, bs + 3, 777], bs)


@pytest.mark.parametrize("B", [1, 3, 1023, 1024, 1025, 2500])
def test_tables_batch_sizes(fia, B):
    """Across the 1024-request chunk of the scan, tokens across CTAs."""
    r = np.random.default_rng(B)
    _tables(fia, r.integers(0, 90, B).tolist(), r.integers(0, 5, B).tolist(), 16)


def test_tables_one_long_request(fia):
    _tables(fia, [5, 17, 0], [0, 5000, 2], 16)


def test_tables_padding_and_undersized(fia):
    """More slots than tokens are -1; fewer: the rest of the tokens get nothing."""
    _tables(fia, [3, 9], [5, 7], 4, n_tokens=40)
    _tables(fia, [3, 9], [5, 7], 4, n_tokens=6)
    _tables(fia, [3, 9], [5, 7], 4, n_tokens=0)


def test_tables_short_list_and_narrow_table(fia):
    (_, _, _, blocks), _ = _tables(fia, [0, 4, 8], [9, 9, 9], 4, free=[11, 5, 3])
    assert blocks.item() > 3
    _tables(fia, [0, 4, 8], [9, 9, 9], 4, W=3)
    _tables(fia, [0, 4, 8], [9, 9, 9], 4, free=[])


def test_tables_negative_and_empty(fia):
    _tables(fia, [-3, 4], [2, -9], 4)
    got, _ = _tables(fia, [], [], 16, n_tokens=3)
    assert got[3].item() == 0


def test_tables_lengths_near_int32(fia):
    """A running position past 2^31 is clamped, not wrapped."""
    big = 2 ** 31 - 2
    s, kv, cu, nb = fia.fia_block_table_append(i32([big, 5]), i32([4, 2]), i32([7, 8]), i32([[0, 0], [1, 1]]),
                                               block_size=1 << 20, num_tokens=6)
    assert kv.tolist() == [2 ** 31 - 1, 7] and cu.tolist() == [4, 6]
    assert s.tolist() == [-1, -1, -1, -1, (1 << 20) + 5, (1 << 20) + 6]


# ------------------------------------------------------------------ cache write
@pytest.mark.parametrize("pool", ["BNBD", "BBH"])
@pytest.mark.parametrize("n2,d,dt,bs,T", [(8, 128, "bf16", 128, 300), (1, 64, "f16", 16, 1), (3, 72, "bf16", 5, 77),
                                          (2, 512, "f16", 64, 65), (5, 128, "bf16", 16, 1030)])
def test_write(fia, pool, n2, d, dt, bs, T):
    nb = 2 * (-(-T // bs)) + 1
    shape = (nb, n2, bs, d) if pool == "BNBD" else (nb, bs, n2 * d)
    kc, vc = (fia_inputs.normal(shape, dt, 70, i) for i in (1, 2))
    x = fia_inputs.normal((T, 4 * n2, d), dt, 71, 3)
    slots = np.random.default_rng(T).permutation(nb * bs)[:T]
    slots[T // 2::7] = -1
    slots[3::50] = nb * bs + 5      # past the pool: skipped
    xd = x.to(DEV)
    k, v = xd[:, n2:2 * n2], xd[:, 3 * n2:]   # slices of one projection
    a, b = kc.to(DEV), vc.to(DEV)
    got = fia.fia_cache_write(k, v, a, b, i32(slots.tolist()))
    assert got[0] is a and got[1] is b
    for y, c, z in ((x[:, n2:2 * n2], kc, a), (x[:, 3 * n2:], vc, b)):
        ref = po.cache_write(f64(y), f64(c), slots.tolist())
        assert np.array_equal(f64(z.cpu()), ref)


def test_write_latent_and_rope(fia):
    """Keys and values of different head dims (a latent cache and its rope part), and keys alone."""
    T, bs, nb = 50, 16, 8
    lat, rope = (fia_inputs.normal((T, 1, d), "bf16", 72, d).to(DEV) for d in (512, 64))
    cl, cr = torch.zeros(nb, bs, 512, dtype=torch.bfloat16, device=DEV), torch.zeros(nb, bs, 64, dtype=torch.bfloat16, device=DEV)
    slots = np.random.default_rng(1).permutation(nb * bs)[:T]
    fia.fia_cache_write(lat, rope, cl, cr, i32(slots.tolist()))
    assert torch.equal(cl.view(-1, 512)[slots], lat[:, 0]) and torch.equal(cr.view(-1, 64)[slots], rope[:, 0])
    only = torch.zeros_like(cl)
    fia.fia_cache_write(lat, None, only, None, i32(slots.tolist()))
    assert torch.equal(only, cl)


def test_write_e4m3(fia):
    T, bs = 9, 16
    x = torch.randn(T, 2, 64, device=DEV).to(torch.float8_e4m3fn)
    c = torch.zeros(3, 2, bs, 64, device=DEV).to(torch.float8_e4m3fn)
    fia.fia_cache_write(x, None, c, None, i32(list(range(20, 20 + T))))
    assert torch.equal(c.view(torch.uint8).transpose(1, 2).reshape(-1, 2, 64)[20:20 + T], x.view(torch.uint8))


# ------------------------------------------------------------------ windowed decode
def _window(fia, lens, n1, n2, D, pre, sink, Q=1, bs=128, dt="bf16", kv="BNBD", layout="BNSD", workload=80, evict=True):
    """A paged case whose unseen blocks are taken out of the tables (id -1 or far outside) and whose unseen rows are
    NaN: only what the tokens see may be read into the result."""
    c = fia_inputs.paged_decode_case(len(lens), n1, n2, D, lens, block_size=bs, dtype=dt, workload=workload, layout_kv=kv,
                                     q_tokens=Q)
    rows, table = [], c.block_table.clone()
    kp, vp = c.k_pool.clone(), c.v_pool.clone()
    for b, L in enumerate(lens):
        rows.append(tuple(po.cache_rows(f64(x), c.block_table[b], L, n2) for x in (c.k_pool, c.v_pool)))
        seen = po.window_see(Q, L, pre, sink).any(0) if L else np.zeros(0, bool)
        for i in range(-(-L // bs)):
            s = seen[i * bs:(i + 1) * bs]
            blk = int(c.block_table[b, i])
            for x in (kp, vp):
                y = x[blk] if x.dim() == 3 else x[blk].transpose(0, 1)
                y[:len(s)][torch.from_numpy(~s)] = float("nan")
            if evict and not s.any():
                table[b, i] = -1 if i % 2 else 2 ** 31 - 1
    q = c.q if layout == "BNSD" else c.q.transpose(1, 2).contiguous()
    q = q.flatten(2) if layout == "BSH" else q
    out, lse = fia.fia_decode_window(q.to(DEV), kp.to(DEV), vp.to(DEV), block_table=table.to(DEV), block_size=bs,
                                     actual_seq_kvlen=i32(lens), num_heads=n1, num_key_value_heads=n2, scale_value=c.scale,
                                     input_layout=layout, pre_tokens=pre, sink_tokens=sink, softmax_lse_flag=True)
    torch.cuda.synchronize()
    out = out.reshape(len(lens), Q, n1, D).transpose(1, 2) if layout != "BNSD" else out
    ref = po.decode(c.q, rows, lens, pre, sink, c.scale)
    po.assert_close(out, lse, ref)
    return out, lse


BIG = 2 ** 31 - 1


@pytest.mark.parametrize("pre,sink", [(0, 0), (0, 1), (15, 4), (16, 16), (100, 0), (127, 130), (1000, 3), (BIG, 0),
                                      (BIG, BIG), (40, BIG)])
def test_window_masks(fia, pre, sink):
    _window(fia, [1, 2, 16, 17, 300, 0, 513, 1999], 8, 2, 128, pre, sink)


@pytest.mark.parametrize("bs", [16, 32, 48, 64, 256])
@pytest.mark.parametrize("kv", ["BNBD", "BBH"])
def test_window_pages(fia, bs, kv):
    _window(fia, [1, 40, 333, 777], 8, 4, 128, 99, 5, bs=bs, kv="BNBD" if kv == "BNBD" else "BSH")


@pytest.mark.parametrize("n1,n2,Q", [(4, 4, 1), (6, 2, 3), (14, 2, 2), (16, 1, 1), (17, 1, 1), (32, 1, 1), (8, 2, 8), (33, 1, 1),
                                     (64, 1, 1), (8, 2, 16), (16, 1, 4), (5, 5, 16)])
def test_window_rows(fia, n1, n2, Q):
    """Units of 1..64 rows: one, two and four row tiles."""
    _window(fia, [max(Q, 1), 130, 555], n1, n2, 128, 70, 9, Q=Q, workload=81 + n1)


@pytest.mark.parametrize("dt,D", [("f16", 128), ("bf16", 64), ("f16", 64)])
@pytest.mark.parametrize("n1,Q", [(4, 1), (20, 1), (16, 4)])
def test_window_types(fia, dt, D, n1, Q):
    _window(fia, [64, 700, 18], n1, 1, D, 200, 4, Q=Q, dt=dt)


@pytest.mark.parametrize("layout", ["BSND", "BSH"])
def test_window_layouts(fia, layout):
    _window(fia, [12, 300], 8, 2, 128, 50, 2, Q=3, layout=layout)


def test_window_shorter_than_tokens(fia):
    """A length below Q_S: the tokens before the sequence's start see nothing."""
    out, lse = _window(fia, [0, 1, 3, 4, 90], 4, 2, 128, 30, 2, Q=4)
    assert torch.isposinf(lse[0]).all() and (out[0] == 0).all()


@pytest.mark.parametrize("B,n2", [(1, 1), (1, 8), (40, 8), (130, 4)])
def test_window_cluster_sizes(fia, B, n2):
    """Few to many units: clusters of 8 CTAs down to single CTAs; long spans, lengths from 0 up."""
    lens = [(i * 977) % 2600 for i in range(B)]
    lens[0] = 2600
    _window(fia, lens, 2 * n2, n2, 64, 2000, 20, bs=64, workload=95)


@pytest.mark.parametrize("layout", ["BNSD", "BSND", "BSH"])
def test_window_contiguous(fia, layout):
    B, n1, n2, S, D, Q = 3, 8, 2, 333, 128, 2
    q = fia_inputs.normal((B, n1, Q, D), "bf16", 82, 1)
    k, v = (fia_inputs.normal((B, n2, S, D), "bf16", 82, i) for i in (2, 3))
    scale = D ** -0.5
    lay = {"BNSD": lambda x: x, "BSND": lambda x: x.transpose(1, 2).contiguous(),
           "BSH": lambda x: x.transpose(1, 2).flatten(2).contiguous()}[layout]
    for lens in ([333, 2, 100], None):
        out, lse = fia.fia_decode_window(lay(q).to(DEV), lay(k).to(DEV), lay(v).to(DEV),
                                         actual_seq_kvlen=None if lens is None else i32(lens), num_heads=n1,
                                         num_key_value_heads=n2, scale_value=scale, input_layout=layout, pre_tokens=60,
                                         sink_tokens=7, softmax_lse_flag=True)
        if layout != "BNSD":
            out = out.reshape(B, Q, n1, D).transpose(1, 2)
        rows = [tuple(f64(x[b].transpose(0, 1)) for x in (k, v)) for b in range(B)]
        po.assert_close(out, lse, po.decode(q, rows, lens or [S] * B, 60, 7, scale))


def test_window_lengths_beyond_the_tables_are_clamped(fia):
    c = fia_inputs.paged_decode_case(1, 2, 1, 64, [96], block_size=32, workload=83, extra_table_cols=0)
    kw = dict(block_table=c.block_table.to(DEV), block_size=32, num_heads=2, num_key_value_heads=1, scale_value=c.scale,
              input_layout="BNSD")
    args = [x.to(DEV) for x in (c.q, c.k_pool, c.v_pool)]
    a, _ = fia.fia_decode_window(*args, actual_seq_kvlen=i32([96]), **kw)
    b, _ = fia.fia_decode_window(*args, actual_seq_kvlen=i32([2 ** 31 - 1]), **kw)
    z, _ = fia.fia_decode_window(*args, actual_seq_kvlen=i32([-5]), **kw)
    assert torch.equal(a, b) and (z == 0).all()


def test_window_without_window_equals_decode(fia):
    """No window: fia_decode on the same cache, to the rounding of both."""
    c = fia_inputs.paged_decode_case(5, 32, 8, 128, [1, 700, 2048, 33, 1500], workload=84)
    args = [x.to(DEV) for x in (c.q, c.k_pool, c.v_pool)]
    kw = dict(block_table=c.block_table.to(DEV), block_size=128, num_heads=32, num_key_value_heads=8, scale_value=c.scale,
              input_layout="BNSD", softmax_lse_flag=True)
    a, la = fia.fia_decode(*args, actual_seq_kvlen=c.kv_lens, **kw)
    b, lb = fia.fia_decode_window(*args, actual_seq_kvlen=i32(c.kv_lens), **kw)
    # each is off by at most half a step of the output and of the weights: |v| < 6 bounds sum w |v|
    assert (a.float() - b.float()).abs().max() <= 4 * 2 ** -8 * 6 and (la - lb).abs().max() < 1e-4
    again, _ = fia.fia_decode_window(*args, actual_seq_kvlen=i32(c.kv_lens), **kw)
    assert torch.equal(b, again)


def test_window_infinite_values_stay_where_they_are_seen(fia):
    """An infinity or NaN in a seen value row reaches the rows that see it and no others."""
    B, n1, D, S = 2, 2, 64, 200
    q, k, v = (fia_inputs.normal((B, n, s, D), "bf16", 85, i) for i, (n, s) in enumerate(((n1, 1), (n1, S), (n1, S))))
    v[0, 0, 150, 3] = float("inf")
    v[0, 1, 20, 5] = float("nan")     # behind the window
    out, _ = fia.fia_decode_window(*[x.to(DEV) for x in (q, k, v)], num_heads=n1, scale_value=0.125, input_layout="BNSD",
                                   pre_tokens=99, sink_tokens=2)
    assert torch.isposinf(out[0, 0, 0, 3]) and torch.isfinite(out[1]).all() and torch.isfinite(out[0, 1]).all()
    assert torch.isfinite(out[0, 0, 0, :3]).all()


# ------------------------------------------------------------------ windowed prefill
def _prefill(fia, ql, kl, n1, n2, D, pre, sink, layout="TND", dt="bf16", bs=0, kv="BNBD", workload=90, pad_q=0, pad_k=0,
             lens=True, extra_rows=0):
    """A window prefill against the oracle; returns (out, lse, the case's tensors)."""
    B, sq, sk = len(ql), max(ql) + pad_q, max(kl) + pad_k
    norm = fia_inputs.normal
    scale = D ** -0.5
    if layout == "TND":
        q = norm((sum(ql) + extra_rows, n1, D), dt, workload, 1)
        qs = list(torch.split(q[:sum(ql)], ql))
        dlq = i32(fia_inputs.cumsum_no_leading_zero(ql))
    else:
        q = norm((B, sq, n1, D), dt, workload, 1)
        qs = [q[b, :ql[b]] for b in range(B)]
        for b in range(B):
            q[b, ql[b]:] = float("nan")        # padding rows may hold anything
        dlq = i32(ql)
    table = None
    if bs:
        c = fia_inputs.paged_decode_case(B, n1, n2, D, kl, block_size=bs, dtype=dt, workload=workload + 1, layout_kv=kv)
        rows = [tuple(po.cache_rows(f64(x), c.block_table[b], kl[b], n2) for x in (c.k_pool, c.v_pool)) for b in range(B)]
        k, v, table, dlk = c.k_pool, c.v_pool, c.block_table.clone(), i32(kl)
        for b in range(B):
            seen = po.window_see(ql[b], kl[b], pre, sink).any(0) if ql[b] and kl[b] else np.zeros(kl[b], bool)
            for i in range(-(-kl[b] // bs)):
                if not seen[i * bs:(i + 1) * bs].any():
                    table[b, i] = -1 if i % 2 else 10 ** 9   # a block behind every row's window is gone
    elif layout == "TND":
        k, v = (norm((sum(kl), n2, D), dt, workload, i) for i in (2, 3))
        rows = [(f64(a), f64(b)) for a, b in zip(torch.split(k, kl), torch.split(v, kl))]
        dlk = i32(fia_inputs.cumsum_no_leading_zero(kl))
    else:
        k, v = (norm((B, sk, n2, D), dt, workload, i) for i in (2, 3))
        rows = [(f64(k[b, :kl[b]]), f64(v[b, :kl[b]])) for b in range(B)]
        for b in range(B):
            k[b, kl[b]:] = float("nan")
            v[b, kl[b]:] = float("nan")
        dlk = i32(kl)
    lay = {"TND": lambda x: x, "BSND": lambda x: x, "BNSD": lambda x: x.transpose(1, 2).contiguous(),
           "BSH": lambda x: x.flatten(2)}[layout]
    qd = lay(q).to(DEV)
    kd, vd = (x.to(DEV) if bs else lay(x).to(DEV) for x in (k, v))
    out = torch.full_like(qd, 7.0)
    lse = torch.full(((q.shape[0], n1, 1) if layout == "TND" else (B, n1, sq, 1)), 7.0, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    fia.fia_prefill_window(qd, kd, vd, actual_seq_qlen=dlq if lens else None, actual_seq_kvlen=dlk if lens else None,
                           block_table=None if table is None else table.to(DEV), block_size=bs, num_heads=n1,
                           num_key_value_heads=n2, scale_value=scale, input_layout=layout, pre_tokens=pre, sink_tokens=sink,
                           softmax_lse_flag=True, out=out, softmax_lse=lse, workspace=ws)
    assert fia.fia_device_status(ws) == 0
    back = {"TND": lambda x: x, "BSND": lambda x: x, "BNSD": lambda x: x.transpose(1, 2),
            "BSH": lambda x: x.reshape(B, sq, n1, D)}[layout]
    o, at = back(out), 0
    for b in range(B):
        n = ql[b]
        see = po.window_see(n, kl[b], pre, sink) if kl[b] else np.zeros((n, 0), bool)
        ref = po.attend(f64(qs[b]), rows[b][0], rows[b][1], see, scale)
        got = o[at:at + n] if layout == "TND" else o[b, :n]
        gl = lse[at:at + n, :, 0] if layout == "TND" else lse[b, :, :n, 0].T
        po.assert_close(got, gl, ref, f"batch {b}")
        at += n
        if layout != "TND":
            assert (o[b, n:] == 0).all() and torch.isposinf(lse[b, :, n:]).all()
    if layout == "TND":
        assert (out[sum(ql):] == 7).all() and (lse[sum(ql):] == 7).all()
    return out, lse, (qd, kd, vd)


@pytest.mark.parametrize("pre,sink", [(0, 0), (0, 3), (31, 4), (127, 0), (128, 128), (129, 129), (300, 1), (300, 200), (511, 513),
                                      (BIG, 0), (100, BIG)])
def test_prefill_window_masks(fia, pre, sink):
    _prefill(fia, [1, 700, 128, 0, 257], [1, 700, 128, 0, 257], 4, 2, 128, pre, sink)


@pytest.mark.parametrize("layout", ["BNSD", "BSND", "BSH"])
@pytest.mark.parametrize("dt,D", [("bf16", 128), ("f16", 64), ("bf16", 64)])
def test_prefill_window_padded(fia, layout, dt, D):
    """Ragged batches in padded layouts, more keys than rows and fewer; NaN in every padding row."""
    _prefill(fia, [300, 5, 0, 129], [700, 3, 40, 129], 6, 3, D, 150, 10, layout=layout, dt=dt, pad_q=60, pad_k=9)


def test_prefill_window_without_lengths(fia):
    _prefill(fia, [260, 260], [260, 260], 2, 1, 64, 70, 2, layout="BNSD", dt="f16", lens=False)


@pytest.mark.parametrize("bs,kv,layout", [(128, "BNBD", "TND"), (256, "BSH", "TND"), (512, "BNBD", "BNSD"), (128, "BSH", "BSND"),
                                          (384, "BNBD", "BSH")])
def test_prefill_window_paged(fia, bs, kv, layout):
    """Chunks against a cache whose blocks behind the windows are gone from the tables."""
    _prefill(fia, [200, 1, 300, 64], [1500, 901, 300, 64], 8, 2, 128, 260, 5, layout=layout, bs=bs, kv=kv)


def test_prefill_window_many_sequences(fia):
    """More sequences than a warp scans at once, empty ones among them, rows behind the last one untouched."""
    r = np.random.default_rng(3)
    ql = [int(x) for x in r.integers(0, 40, 75)]
    ql[70] = 600
    _prefill(fia, ql, ql, 2, 1, 64, 33, 2, extra_rows=37)


def test_prefill_window_fewer_keys_than_rows(fia):
    """Rows before position 0 see nothing, also where a whole 128-row tile lies there."""
    _prefill(fia, [400, 300], [90, 299], 2, 2, 128, 50, 3)


def test_prefill_window_equals_causal(fia):
    """Without a window: fia_prefill's causal mode, the same bits for one sequence."""
    ql = [640]
    out, lse, (q, k, v) = _prefill(fia, ql, ql, 4, 2, 128, BIG, 0)
    o2, l2 = fia.fia_prefill(q, k, v, num_heads=4, num_key_value_heads=2, scale_value=128 ** -0.5, input_layout="TND",
                             sparse_mode=3, actual_seq_qlen=ql, actual_seq_kvlen=ql, softmax_lse_flag=True)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_prefill_window_bad_lengths_stay_inside(fia):
    """Lengths outside the tensors are taken inside: nothing else is read or written."""
    q, k, v = (fia_inputs.normal((100, 2, 64), "bf16", 97, i).to(DEV) for i in (1, 2, 3))
    kw = dict(num_heads=2, scale_value=0.125, input_layout="TND", pre_tokens=20, sink_tokens=1)
    a, _ = fia.fia_prefill_window(q, k, v, actual_seq_qlen=i32([40, 100]), actual_seq_kvlen=i32([40, 100]), **kw)
    b, _ = fia.fia_prefill_window(q, k, v, actual_seq_qlen=i32([40, 10 ** 9]), actual_seq_kvlen=i32([40, 2 ** 31 - 1]), **kw)
    assert torch.equal(a, b)
    fia.fia_prefill_window(q, k, v, actual_seq_qlen=i32([-5, 70]), actual_seq_kvlen=i32([200, 3]), **kw)
    torch.cuda.synchronize()


def test_prefill_window_empty_keys(fia):
    q = fia_inputs.normal((2, 2, 5, 64), "bf16", 98, 1).to(DEV)
    k = torch.zeros(2, 2, 0, 64, dtype=torch.bfloat16, device=DEV)
    out, lse = fia.fia_prefill_window(q, k, k, num_heads=2, input_layout="BNSD", softmax_lse_flag=True)
    assert (out == 0).all() and torch.isposinf(lse).all()


# ------------------------------------------------------------------ shared prefix
def _prefix(fia, own_lens, P, n1, n2, D, Q=1, bs=128, dt="bf16", kv="BNBD", layout="BNSD", workload=100, totals=None):
    """own_lens: keys of each sequence behind the prefix; totals overrides whole lengths (sequences shorter than it)."""
    B, scale = len(own_lens), D ** -0.5
    lens = [P + n for n in own_lens] if totals is None else totals
    pages = P // bs
    c = fia_inputs.paged_decode_case(B, n1, n2, D, own_lens, block_size=bs, dtype=dt, workload=workload, layout_kv=kv,
                                     q_tokens=Q)
    r = np.random.default_rng(P + B)
    first = c.k_pool.shape[0] + r.permutation(pages)
    shape = (pages,) + tuple(c.k_pool.shape[1:])
    kp, vp = (torch.cat([x, fia_inputs.normal(shape, dt, workload, i)]) for i, x in ((7, c.k_pool), (8, c.v_pool)))
    table = torch.cat([torch.tensor(first, dtype=torch.int32).expand(B, pages), c.block_table], 1).contiguous()
    q = c.q if layout == "BNSD" else c.q.transpose(1, 2).contiguous()
    q = q.flatten(2) if layout == "BSH" else q
    kw = dict(block_table=table.to(DEV), block_size=bs, actual_seq_kvlen=i32(lens), num_heads=n1, num_key_value_heads=n2,
              scale_value=scale, input_layout=layout, softmax_lse_flag=True)
    args = [x.to(DEV) for x in (q, kp, vp)]
    out, lse = fia.fia_decode_shared_prefix(*args, shared_prefix_len=P, **kw)
    torch.cuda.synchronize()
    o = out.reshape(B, Q, n1, D).transpose(1, 2) if layout != "BNSD" else out
    pf, vf = f64(kp), f64(vp)
    rows = [tuple(po.cache_rows(x, table[b], lens[b], n2) for x in (pf, vf)) for b in range(B)]
    po.assert_close(o, lse, po.decode(c.q, rows, lens, 1 << 40, 0, scale))
    again, _ = fia.fia_decode_shared_prefix(*args, shared_prefix_len=P, **kw)
    assert torch.equal(out, again)
    for path in (1, 2):       # the prefix by a kernel of its own, and by every sequence's
        lib = _binding.load_library()
        lib.fia_debug_set_prefix_path(path)
        try:
            o, l = fia.fia_decode_shared_prefix(*args, shared_prefix_len=P, **kw)
        finally:
            lib.fia_debug_set_prefix_path(0)
        o = o.reshape(B, Q, n1, D).transpose(1, 2) if layout != "BNSD" else o
        po.assert_close(o, l, po.decode(c.q, rows, lens, 1 << 40, 0, scale))
    return out, lse, args, kw


@pytest.mark.parametrize("P", [128, 256, 384, 1152, 4096])
@pytest.mark.parametrize("B", [2, 5, 40])
def test_prefix_lengths(fia, P, B):
    _prefix(fia, [(i * 37) % 200 + 1 for i in range(B)], P, 8, 2, 128)


@pytest.mark.parametrize("bs", [16, 32, 64, 256])
@pytest.mark.parametrize("kv", ["BNBD", "BSH"])
def test_prefix_pages(fia, bs, kv):
    """Pages below a tile, prefixes that end inside one."""
    _prefix(fia, [1, bs, 3 * bs + 1], bs * (7 if bs < 128 else 3), 8, 2, 128, bs=bs, kv=kv, workload=101 + bs)


@pytest.mark.parametrize("n1,n2,Q,B", [(4, 4, 1, 300), (32, 8, 1, 33), (7, 1, 1, 40), (28, 4, 2, 12), (16, 1, 4, 5), (64, 1, 1, 3),
                                       (3, 3, 16, 20), (5, 1, 3, 9), (40, 8, 1, 26), (8, 8, 1, 130)])
def test_prefix_rows(fia, n1, n2, Q, B):
    """Row tiles of 128 / (heads x tokens) sequences: whole, part-filled, one to many tiles, odd groups."""
    _prefix(fia, [Q + (i * 13) % 60 for i in range(B)], 640, n1, n2, 64, Q=Q, bs=64, workload=103 + n1)


@pytest.mark.parametrize("dt,D", [("f16", 128), ("bf16", 64), ("f16", 64)])
@pytest.mark.parametrize("layout", ["BSND", "BSH"])
def test_prefix_types_and_layouts(fia, dt, D, layout):
    _prefix(fia, [3, 70, 40], 512, 8, 2, D, Q=3, dt=dt, layout=layout)


def test_prefix_short_and_empty_sequences(fia):
    """Lengths inside the prefix, at its end, zero and below the number of new tokens."""
    _prefix(fia, [1, 1, 1, 1, 1, 50], 256, 4, 2, 128, Q=2, totals=[0, 1, 100, 256, 257, 306])


def test_prefix_without_prefix_and_single_sequence(fia):
    out, lse, args, kw = _prefix(fia, [40, 300], 0, 8, 2, 128)
    w, l2 = fia.fia_decode_window(*args, **kw)
    assert torch.equal(out, w) and torch.equal(lse, l2)
    _prefix(fia, [77], 512, 8, 2, 128)


def test_prefix_reads_the_first_row_only(fia):
    """The prefix comes from the table's first row: other rows' entries of it are not looked at."""
    out, _, args, kw = _prefix(fia, [9, 30, 200], 384, 8, 2, 128)
    kw["block_table"][1:, :3] = -9
    o2, _ = fia.fia_decode_shared_prefix(*args, shared_prefix_len=384, **kw)
    assert torch.equal(out, o2)
    _binding.load_library().fia_debug_set_prefix_path(1)
    try:
        o3, _ = fia.fia_decode_shared_prefix(*args, shared_prefix_len=384, **kw)
        kw["block_table"][1:, :3] = kw["block_table"][0, :3]
        o4, _ = fia.fia_decode_shared_prefix(*args, shared_prefix_len=384, **kw)
    finally:
        _binding.load_library().fia_debug_set_prefix_path(0)
    assert torch.equal(o3, o4)


def test_prefix_status_and_workspace(fia):
    out, _, args, kw = _prefix(fia, [9, 30, 200], 384, 8, 2, 128)
    ws = torch.full((1 << 24,), 255, dtype=torch.uint8, device=DEV)
    o2, _ = fia.fia_decode_shared_prefix(*args, shared_prefix_len=384, workspace=ws, **kw)
    assert torch.equal(out, o2) and fia.fia_device_status(ws) == 0


# ------------------------------------------------------------------ the binding
def test_binding_checks(fia):
    """What the binding refuses, and the library's refusals as FIAError with the status."""
    q = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(2, 2, 50, 64, dtype=torch.bfloat16, device=DEV)
    kw = dict(num_heads=4, num_key_value_heads=2, input_layout="BNSD")
    with pytest.raises(ValueError, match="contiguous"):
        fia.fia_decode_window(q, k.transpose(2, 3), k, **kw)
    with pytest.raises(ValueError, match="CUDA"):
        fia.fia_decode_window(q, k.cpu(), k, **kw)
    with pytest.raises(TypeError, match="tensor"):
        fia.fia_decode_window(q, k, k, actual_seq_kvlen=[3, 4], **kw)
    with pytest.raises(TypeError, match="dtype"):
        fia.fia_decode_window(q.double(), k, k, **kw)
    with pytest.raises(fia.FIAError) as e:
        fia.fia_decode_window(q, k, k, pre_tokens=-1, **kw)
    assert e.value.status == 5 and "pre_tokens" in str(e.value)
    with pytest.raises(fia.FIAError):
        fia.fia_decode_window(q, k, k, actual_seq_kvlen=torch.zeros(2, dtype=torch.int64, device=DEV), **kw)
    with pytest.raises(ValueError, match="contiguous"):
        x = torch.zeros(4, 64, 2, dtype=torch.bfloat16, device=DEV).transpose(1, 2)
        fia.fia_cache_write(x, None, k, None, i32([0, 1, 2, 3]))
    z = i32([1, 2])
    with pytest.raises(ValueError, match="num_tokens"):
        fia.fia_block_table_append(z, z.clone(), z.clone(), torch.zeros(2, 2, dtype=torch.int32, device=DEV), block_size=4,
                                   num_tokens=5, slot_mapping=i32([0, 0]))
    with pytest.raises(fia.FIAError, match="overlap"):
        fia.fia_block_table_append(z, z.clone(), z.clone(), torch.zeros(2, 2, dtype=torch.int32, device=DEV), block_size=4,
                                   num_tokens=5, kv_lens=z)


def test_cache_write_refuses_repeated_tokens(fia):
    """A broadcast token has a stride of 0, which the C entry reads as "contiguous"."""
    pool = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16, device=DEV)
    one = torch.ones(1, 2, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="share memory"):
        fia.fia_cache_write(one.expand(4, 2, 64), None, pool, None, i32([0, 1, 2, 3]))
    fia.fia_cache_write(one.expand(1, 2, 64), None, pool, None, i32([3]))
    assert pool[0, :, 3].eq(1).all() and pool.sum() == 128


# ------------------------------------------------------------------ units of 17..64 rows
@pytest.mark.parametrize("pre,sink", [(0, 0), (0, 70), (15, 4), (64, 64), (100, 0), (127, 130), (1000, 3), (BIG, 0), (40, BIG)])
def test_wide_masks(fia, pre, sink):
    _window(fia, [1, 2, 63, 64, 65, 300, 0, 513, 1999], 40, 1, 128, pre, sink, workload=130)


@pytest.mark.parametrize("bs", [16, 32, 48, 64, 96, 256])
@pytest.mark.parametrize("kv", ["BNBD", "BSH"])
def test_wide_pages(fia, bs, kv):
    """Pages below a 64-key tile, that do not divide it, and above it; a window that starts inside a page."""
    _window(fia, [1, 8, 40, 333, 777], 16, 2, 128, 99, 70, Q=8, bs=bs, kv=kv, workload=131)


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("n1,n2,Q,lens,pre", [
    (32, 1, 1, [3000, 2049, 7, 0], 2500), (24, 1, 1, [2600, 64, 2047], BIG), (18, 2, 2, [2400, 2, 1], 2100),   # 32 rows, many keys
    (6, 2, 4, [1 + (i * 29) % 300 for i in range(90)], 270),                                                   # 180 units of 24 rows
    (64, 1, 1, [2900], BIG), (8, 1, 8, [900, 1, 64, 65, 128], 300), (44, 4, 5, [128] * 3, BIG)])               # 33..64 rows
def test_wide_units(fia, dt, D, n1, n2, Q, lens, pre):
    """Both layouts of the rows in TMEM, one to eight CTAs of a unit, CTAs without a tile."""
    _window(fia, lens, n1, n2, D, pre, 5, Q=Q, bs=64, dt=dt, workload=132 + n1)


@pytest.mark.parametrize("layout", ["BNSD", "BSND", "BSH"])
def test_wide_contiguous(fia, layout):
    """A cache whose last tile ends inside the tensor; NaN rows past a length; no keys at all."""
    B, n1, n2, S, D, Q = 2, 24, 2, 333, 64, 4
    q = fia_inputs.normal((B, n1, Q, D), "bf16", 133, 1)
    k, v = (fia_inputs.normal((B, n2, S, D), "bf16", 133, i) for i in (2, 3))
    lens, scale = [333, 70], D ** -0.5
    rows = [tuple(f64(x[b].transpose(0, 1)) for x in (k, v)) for b in range(B)]
    k[1, :, 70:] = float("nan")
    v[1, :, 70:] = float("nan")
    lay = {"BNSD": lambda x: x, "BSND": lambda x: x.transpose(1, 2).contiguous(),
           "BSH": lambda x: x.transpose(1, 2).flatten(2).contiguous()}[layout]
    kw = dict(num_heads=n1, num_key_value_heads=n2, scale_value=scale, input_layout=layout, softmax_lse_flag=True)
    out, lse = fia.fia_decode_window(lay(q).to(DEV), lay(k).to(DEV), lay(v).to(DEV), actual_seq_kvlen=i32(lens), pre_tokens=100,
                                     sink_tokens=3, **kw)
    out = out if layout == "BNSD" else out.reshape(B, Q, n1, D).transpose(1, 2)
    po.assert_close(out, lse, po.decode(q, [(a[:n], b[:n]) for (a, b), n in zip(rows, lens)], lens, 100, 3, scale))
    none = lay(k[:, :, :0]).to(DEV)
    out, lse = fia.fia_decode_window(lay(q).to(DEV), none, none, **kw)
    assert (out == 0).all() and torch.isposinf(lse).all()


def test_wide_empty_pool_reads_as_zeros(fia):
    """No block in the pool: every key and value of a length is 0, so out = 0 and lse = log(keys seen)."""
    q = fia_inputs.normal((2, 40, 1, 64), "bf16", 134, 1).to(DEV)
    pool = torch.zeros(0, 1, 32, 64, dtype=torch.bfloat16, device=DEV)
    table = torch.zeros(2, 4, dtype=torch.int32, device=DEV)
    out, lse = fia.fia_decode_window(q, pool, pool, actual_seq_kvlen=i32([100, 0]), block_table=table, block_size=32, num_heads=40,
                                     num_key_value_heads=1, input_layout="BNSD", softmax_lse_flag=True)
    assert (out == 0).all() and torch.isposinf(lse[1]).all() and (lse[0] - np.log(100)).abs().max() < 1e-5


@pytest.mark.parametrize("n1,n2,Q,B,own", [(64, 1, 1, 5, 700), (16, 2, 8, 4, 90), (48, 8, 4, 30, 300)])
def test_wide_behind_a_prefix(fia, n1, n2, Q, B, own):
    _prefix(fia, [Q + (i * 61) % own for i in range(B)], 512, n1, n2, 128, Q=Q, bs=128, workload=135 + n1)


def test_wide_timeout_leaves_nan(fia):
    """A wait that gives up leaves NaN in its unit's rows (there is no status word); the next call is right."""
    from attention_fia_prefill_gb300 import _binding as B
    lib = B.load_library()
    q, k, v = (fia_inputs.normal((4, n, s, 128), "bf16", 136, i).to(DEV) for i, (n, s) in enumerate(((64, 1), (1, 3000), (1, 3000))))
    kw = dict(num_heads=64, num_key_value_heads=1, scale_value=0.1, input_layout="BNSD")
    want, _ = fia.fia_decode_window(q, k, v, **kw)
    lib.fia_debug_set_wait_limit_ns(1)
    try:
        short, _ = fia.fia_decode_window(q, k, v, **kw)
        torch.cuda.synchronize()
    finally:
        lib.fia_debug_set_wait_limit_ns(0)
    gave_up = short.isnan().flatten(1).any(1)   # (a wait whose first try succeeds does not look at the limit)
    for b in range(4):
        assert short[b].isnan().all() if gave_up[b] else torch.equal(short[b], want[b])
    again, _ = fia.fia_decode_window(q, k, v, **kw)
    assert torch.equal(again, want)


@pytest.mark.parametrize("n1", [8, 64])
def test_prefix_read_by_every_sequence_reports_its_status(fia, n1):
    """Without a kernel of the prefix's own the decode kernels stamp the status word, and raise it."""
    q, k, v = (fia_inputs.normal(s, "bf16", 137, i).to(DEV) for i, s in enumerate(((2, n1, 1, 128), (40, 1, 64, 128), (40, 1, 64, 128))))
    table = torch.arange(40, dtype=torch.int32, device=DEV).view(2, 20)
    table[1, :8] = table[0, :8]
    kw = dict(block_table=table, block_size=64, actual_seq_kvlen=i32([1280, 1100]), shared_prefix_len=512, num_heads=n1,
              num_key_value_heads=1, scale_value=0.09, input_layout="BNSD")
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device=DEV)
    lib = _binding.load_library()
    want, _ = fia.fia_decode_shared_prefix(q, k, v, workspace=ws, **kw)
    assert fia.fia_device_status(ws) == 0
    lib.fia_debug_set_wait_limit_ns(1)
    try:
        short, _ = fia.fia_decode_shared_prefix(q, k, v, workspace=ws, **kw)
        status = fia.fia_device_status(ws)
    finally:
        lib.fia_debug_set_wait_limit_ns(0)
    assert (status == 10) == bool(short.isnan().any()) and (n1 == 64) >= (status == 10)
    again, _ = fia.fia_decode_shared_prefix(q, k, v, workspace=ws, **kw)
    assert fia.fia_device_status(ws) == 0 and torch.equal(again, want)
