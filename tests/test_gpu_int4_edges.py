"""Edges of the 4-bit cache on the GPU: values at the top of f16, factors of the scores at the ends of fp32, keys that a
token does not see with steps far above the others', and windows on evenly shared work."""
import numpy as np
import pytest
import torch

from oracle import int4_oracle as io
from oracle.fia_oracle import f64

from .test_gpu_int4 import DEV, DTYPES, i32, pools, slot_rows

pytestmark = pytest.mark.gpu
SHARED = 1 << 20     # keys of the tables' room that make a call of two units or more one of much work


def written(fia, k, v, G, bs=16, layout="BNBD", dt="bf16"):
    """Keys and values (B, L, N, D) -> pools and the tables of a sequence's own blocks."""
    B, L, n2, D = k.shape
    W = -(-L // bs)
    p = pools(B * W, n2, bs, D, G, layout, dt)
    slots = (torch.arange(B)[:, None] * (W * bs) + torch.arange(L)).reshape(-1)
    fia.fia_cache_write_int4(k.reshape(-1, n2, D).to(DTYPES[dt]).to(DEV), v.reshape(-1, n2, D).to(DTYPES[dt]).to(DEV), *p,
                             slots.to(torch.int32).to(DEV))
    return p, torch.arange(B * W, dtype=torch.int32).view(B, W)


def attend(fia, q, p, table, lens, bs=16, scale=1.0, room=0, **kw):
    """-> out, lse, the oracle's and (f16) its middles, of BNSD queries; room: keys that the tables have room for."""
    n1, n2 = q.shape[1], p[2].shape[1]
    wide = torch.zeros(table.shape[0], max(table.shape[1], room // bs), dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    out, lse = fia.fia_decode_window_int4(q.to(DEV), *p, actual_seq_kvlen=i32(lens), block_table=wide.to(DEV), block_size=bs,
                                          num_heads=n1, num_key_value_heads=n2, scale_value=scale, input_layout="BNSD",
                                          softmax_lse_flag=True, **kw)
    parts = [io.pool_parts(p[0], p[2]), io.pool_parts(p[1], p[3])]
    rows = [[io.rows(x, table[b].numpy(), n) for b, n in enumerate(lens)] for x in parts]
    span = kw.get("pre_tokens", 1 << 40), kw.get("sink_tokens", 0), scale
    middle = None
    if q.dtype == torch.float16:
        D = q.shape[-1]
        steps = np.repeat(f64(p[3]).transpose(0, 2, 1, 3, 4)[..., 0], D // p[3].shape[3], -1)
        steps = [io.rows((steps,), table[b].numpy(), n)[0] for b, n in enumerate(lens)]
        middle = io.middles(q, *rows, steps, lens, *span)
    return out, lse, io.decode(q, *rows, lens, *span), middle


# ------------------------------------------------------------------ the top of f16
def _groups_up_to(top, every):
    """A group of 64 for every (every-th) finite f16 low up to `top`: low, top, and values between them."""
    low = torch.arange(-32768, 32768).to(torch.int16).view(torch.float16)
    low = low[low.isfinite() & (low <= top)][::every].double()[:, None]
    u = torch.rand(low.shape[0], 64, generator=torch.Generator().manual_seed(int(top)), dtype=torch.float64)
    u[:, 5], u[:, 40] = 0.0, 1.0
    return (low + (top - low) * u).half()


@pytest.mark.parametrize("top,every", [(65504.0, 1), (65472.0, 5), (65440.0, 5), (65408.0, 5), (65376.0, 5)])
def test_f16_groups_at_the_top_of_the_type(fia, top, every):
    """Finite values read back finite, half a step off at most: the step is rounded down where code 15 would otherwise
    stand for more than the type holds."""
    x = _groups_up_to(top, every)
    x = torch.cat([x, x[:1].expand(-x.shape[0] % 16, -1)])[:, None]
    T, bs = x.shape[0], 16
    p = pools(T // bs, 1, bs, 64, 64, "BNBD", "f16")
    fia.fia_cache_write_int4(x.to(DEV), x.to(DEV), *p, torch.arange(T, dtype=torch.int32, device=DEV))
    k, v = fia.fia_cache_read_int4(*p, block_table=torch.arange(T // bs, dtype=torch.int32, device=DEV)[None], cu_kv_lens=i32([T]),
                                   num_tokens=T)
    assert k.isfinite().all() and torch.equal(k, v)
    step = f64(p[2])[..., 0, 0].reshape(-1, 1, 1)
    # the nearest code: what it stands for is at most |x| + step / 2 in magnitude, and is rounded to 24 bits, then to 11
    off = np.abs(f64(k) - f64(x)) - 2.0 ** -11 * (1 + 2.0 ** -10) * (np.abs(f64(x)) + step / 2) - 2.0 ** -25
    assert (off <= step / 2).all()
    code, want, low = io.quantise(x, 64)
    got_c, got_s = slot_rows(p[0], p[2])
    assert np.array_equal(got_c, io.pack(code)) and np.array_equal(f64(got_s), np.stack([want, low], -1))


@pytest.mark.parametrize("n1,D,G,room", [(1, 128, 32, 0), (4, 64, 32, 0), (8, 128, 128, SHARED), (16, 128, 64, 0), (32, 64, 64, 0),
                                         (64, 128, 128, 0), (40, 64, 64, SHARED), (64, 128, 32, SHARED)])
def test_f16_decode_at_the_top_of_the_type(fia, n1, D, G, room):
    """Outputs that are averages of values up to the type's largest are finite, and right."""
    B, L = 3, 90
    g = torch.Generator().manual_seed(n1 + D)
    k = torch.randn(B, L, 1, D, generator=g)
    v = torch.randn(B, L, 1, D, generator=g) * 30000
    v[..., ::4] = 65504.0
    v[..., 1::8] = -65504.0
    v[:, ::2, :, 2::8] = 65472.0
    v = v.clamp(-65504, 65504)
    p, table = written(fia, k, v, G, dt="f16")
    q = torch.randn(B, n1, 1, D, generator=g).half()
    q[0] = 0.0
    for lens in ([90, 1, 2], [77, 33, 16]):
        out, lse, ref, mid = attend(fia, q, p, table, lens, scale=D ** -0.5, room=room)
        assert out.isfinite().all()
        io.assert_close(out, lse, ref, 90, wide=n1 > 32 and G == D, middle=mid)
    # keys as large: scores of their size, but for small queries
    p, table = written(fia, v, k, G, dt="f16")
    out, lse, ref, mid = attend(fia, (q.float() * 1e-5).half(), p, table, [90, 1, 17], scale=0.125, room=room)
    io.assert_close(out, lse, ref, 90, wide=n1 > 32 and G == D, middle=mid)


# ------------------------------------------------------------------ the scores' factor
ROWS = [(1, 64, 32, 0), (4, 128, 128, 0), (8, 128, 32, SHARED), (16, 128, 64, 0), (32, 64, 64, SHARED), (64, 64, 64, 0),
        (48, 128, 128, SHARED), (64, 128, 32, 0)]    # rows of a unit, D, G, keys that the tables have room for


@pytest.mark.parametrize("n1,D,G,room", ROWS)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("scale", [1e-9, 2.0 ** -60, 2.0 ** -126])
def test_query_rows_of_zeros_and_small_scales(fia, n1, D, G, room, dt, scale):
    """A row of zeros (a padded one) averages the values it sees, whatever the scale."""
    g = torch.Generator().manual_seed(n1)
    k, v = torch.randn(3, 90, 1, D, generator=g), torch.randn(3, 90, 1, D, generator=g) + 2
    p, table = written(fia, k, v, G, dt=dt)
    q = torch.randn(3, n1, 1, D, generator=g).to(DTYPES[dt])
    q[0] = 0.0
    q[:, ::3] = 0.0
    q[:, 1::3] *= 2.0 ** -14
    out, lse, ref, mid = attend(fia, q, p, table, [90, 1, 17], scale=scale, room=room)
    assert out.isfinite().all()
    io.assert_close(out, lse, ref, 90, wide=n1 > 32 and G == D, middle=mid)


@pytest.mark.parametrize("n1,D,G,room", ROWS)
@pytest.mark.parametrize("at,scale", [(117, 0.125), (118, 0.125), (121, 0.125), (121, 2.0 ** 4), (-40, 2.0 ** 38), (-100, 2.0 ** 98),
                                      (-120, 2.0 ** 118), (-126, 2.0 ** 120)])
def test_queries_of_far_magnitudes(fia, n1, D, G, room, at, scale):
    """bf16 queries of 2^at: scores of a few units all the same (the keys are rows of one value)."""
    g = torch.Generator().manual_seed(n1 + at)
    unit = 2.0 ** (-at) / (D * scale)
    k = (torch.randn(3, 90, 1, 1, generator=g).double() * 3 * unit).expand(-1, -1, -1, D)
    v = torch.randn(3, 90, 1, D, generator=g)
    p, table = written(fia, k, v, G)
    q = ((1 + torch.rand(3, n1, 1, D, generator=g).double()) * 2.0 ** at).bfloat16()
    out, lse, ref, mid = attend(fia, q, p, table, [90, 1, 17], scale=scale, room=room)
    assert np.isfinite(ref[1]).all() and ref[4].max() < 40
    io.assert_close(out, lse, ref, 90, wide=n1 > 32 and G == D, middle=mid)


# ------------------------------------------------------------------ work shared evenly among the CTAs
@pytest.mark.parametrize("n1,Q,D,G", [(4, 1, 128, 128), (8, 2, 64, 32), (16, 4, 64, 64), (16, 4, 128, 32)])
def test_shares_that_begin_with_any_sequence(fia, n1, Q, D, G):
    """Shares whose first unit any lane finds, in the first 32 sequences and behind them, with nothing else to do and with
    much: the oracle's results, and the same bits on every run."""
    B, L = 200, 70
    g = torch.Generator().manual_seed(n1 + G)
    p, table = written(fia, *(torch.randn(4, L, 1, D, generator=g) for _ in range(2)), G)
    table = table[torch.arange(B) % 4]
    q = torch.randn(B, n1, Q, D, generator=g).bfloat16()
    for first, every in ((0, 1), (1, 7), (31, 33), (64, 2), (199, 1), (97, 50)):
        lens = [L - b % 9 if b >= first and (b - first) % every == 0 else 0 for b in range(B)]
        out, lse, ref, mid = attend(fia, q, p, table, lens, scale=D ** -0.5, room=SHARED)
        io.assert_close(out, lse, ref, L, wide=n1 * Q > 32 and G == D, middle=mid)
        wide = torch.nn.functional.pad(table, (0, SHARED // 16 - table.shape[1])).to(DEV)
        for _ in range(5):
            again = fia.fia_decode_window_int4(q.to(DEV), *p, actual_seq_kvlen=i32(lens), block_table=wide, block_size=16, num_heads=n1,
                                               num_key_value_heads=1, scale_value=D ** -0.5, input_layout="BNSD")
            assert torch.equal(again[0], out)


# ------------------------------------------------------------------ steps far above the others'
@pytest.mark.parametrize("room", [0, SHARED])
@pytest.mark.parametrize("n1,Q,D,dt", [(16, 4, 128, "bf16"), (9, 4, 64, "bf16"), (4, 16, 64, "bf16"), (16, 4, 128, "f16"), (4, 2, 64, "bf16"),
                                       (8, 4, 128, "bf16")])
@pytest.mark.parametrize("where", ["hidden", "light"])
def test_values_far_above_the_others(fia, n1, Q, D, dt, room, where):
    """A value row 2^40 times as wide as the others (f16: others 2^-9, it 2^14), that only the last token sees, or that
    every token sees with a weight of about e^-60: the others' digits stay.

    Weights times steps are rounded to 11 bits down to 2^-26 of their own largest, and to 2^-37 of it below; that is
    assert_close with the row's own largest where it takes the sequence's."""
    L = [61, 200]
    g = torch.Generator().manual_seed(n1 + D)
    k, v = (torch.randn(2, 200, 1, D, generator=g) for _ in range(2))
    big = 2.0 ** 40
    if dt == "f16":
        v, big = v * 2.0 ** -9, 2.0 ** 23
    q = torch.randn(2, n1, Q, D, generator=g)
    for b, n in enumerate(L):
        at = n - 1 if where == "hidden" else 20
        v[b, at] *= big
        if where == "light":
            q[b, :, :, 0], k[b, :, 0, 0], k[b, at, 0, 0] = 12.0, 0.0, -50.0 * D ** 0.5 / 10
    p, table = written(fia, k, v, D, dt=dt)
    out, lse, ref, mid = attend(fia, q.to(DTYPES[dt]), p, table, L, scale=D ** -0.5, room=room)
    ref = ref[:7] + (ref[6],)
    pick = slice(0, Q - 1) if where == "hidden" else slice(0, Q)
    io.assert_close(out[:, :, pick], lse[:, :, pick], tuple(x[:, :, pick] for x in ref), 200, wide=True, middle=None if mid is None else mid[:, :, pick])


def shared_evenly(fia, q, p, **kw):
    """Whether a call's work is shared evenly: then it needs a workspace, and refuses one of 256 bytes."""
    try:
        fia.fia_decode_window_int4(q, *p, workspace=torch.empty(256, dtype=torch.uint8, device=DEV), **kw)
    except fia.FIAError as e:
        assert "workspace" in str(e)
        return True
    return False


@pytest.mark.parametrize("n1,n2,Q,D,G,dt", [(4, 2, 1, 64, 32, "f16"), (6, 1, 1, 128, 128, "bf16"), (8, 2, 3, 128, 32, "bf16"),
                                            (10, 2, 5, 64, 64, "bf16"), (16, 2, 8, 128, 128, "bf16"), (16, 1, 4, 64, 64, "f16"),
                                            (8, 1, 8, 128, 64, "bf16")])
@pytest.mark.parametrize("pre,sink", [(1500, 20), (63, 300), (200, 0), (17, 5)])
def test_windows_on_evenly_shared_work(fia, n1, n2, Q, D, G, dt, pre, sink):
    """Windows that end in any chunk of a cut unit, gaps behind the sinks inside one; as many sequences as make the plan
    one of shares.  A share of them is compared."""
    bs, W = 16, 130
    span = min(W * bs, pre + sink + Q)
    rows = n1 // n2 * Q
    B = min(-(-(33 * 152 * 16 if rows <= 8 else 33 * 152 * 8 if rows <= 16 else 33 * 152 * 4 if rows <= 32 else 33 * 152 * 2) // (n2 * (span // 16))),
            100000)
    r = np.random.default_rng(pre + n1)
    lens = np.where(r.random(B) < min(0.5, 400 / B), r.integers(0, W * bs + 1, B), r.integers(0, 60, B))
    g = torch.Generator().manual_seed(pre + D)
    blocks = 400
    p, _ = written(fia, *(torch.randn(blocks, bs, n2, D, generator=g) for _ in range(2)), G, dt=dt)
    table = r.integers(0, blocks, (B, W)).astype(np.int32)
    q = torch.randn(B, n1, Q, D, generator=g).to(DTYPES[dt])
    kw = dict(actual_seq_kvlen=i32(lens.tolist()), block_table=torch.from_numpy(table).to(DEV), block_size=bs, num_heads=n1,
              num_key_value_heads=n2, scale_value=D ** -0.5, input_layout="BNSD", pre_tokens=pre, sink_tokens=sink, softmax_lse_flag=True)
    assert shared_evenly(fia, q.to(DEV), p, **kw)
    out, lse = fia.fia_decode_window_int4(q.to(DEV), *p, **kw)
    long = np.flatnonzero(lens >= 60)
    pick = np.concatenate([np.arange(10), r.choice(long, min(25, len(long)), False), r.integers(0, B, 15), np.arange(B - 5, B)])
    parts = [io.pool_parts(p[0], p[2]), io.pool_parts(p[1], p[3])]
    rows_ = [[io.rows(x, table[b], lens[b]) for b in pick] for x in parts]
    ref = io.decode(q[pick], *rows_, lens[pick], pre, sink, D ** -0.5)
    middle = None
    if dt == "f16":
        steps = np.repeat(f64(p[3]).transpose(0, 2, 1, 3, 4)[..., 0], G, -1)
        middle = io.middles(q[pick], *rows_, [io.rows((steps,), table[b], lens[b])[0] for b in pick], lens[pick], pre, sink, D ** -0.5)
    io.assert_close(out[pick], lse[pick], ref, W * bs, wide=rows > 32 and G == D, middle=middle)
    # and all of them against calls of a few sequences each, which clusters of CTAs take
    worst = 0.0
    for a in range(0, B, 96):
        few = dict(kw, actual_seq_kvlen=kw["actual_seq_kvlen"][a:a + 96], block_table=kw["block_table"][a:a + 96])
        some = fia.fia_decode_window_int4(q[a:a + 96].to(DEV), *p, **few)[0]
        worst = max(worst, (some.float() - out[a:a + 96].float()).abs().max().item())
    # (two results of averages of values below 8: their roundings, and those of P in 11 bits, twice)
    assert f64(p[3])[..., 1].min() > -8 and worst <= 2 * 8 * (torch.finfo(DTYPES[dt]).eps / 2 + 2.0 ** -10)


@pytest.mark.parametrize("n1,Q,D,G", [(10, 4, 64, 64), (16, 4, 128, 128), (4, 4, 64, 32), (2, 4, 128, 128)])
@pytest.mark.parametrize("at,pre", [(59, 200), (58, 200), (40, 18)])
@pytest.mark.parametrize("which", [0, 1])
def test_nan_keys_on_evenly_shared_work(fia, n1, Q, D, G, at, pre, which):
    """A NaN key or value reaches the tokens that see it, and no other: of its sequence, and of those behind it in a share."""
    bs, L, W = 16, 61, 16
    x = [torch.randn(1, 64, 1, D, generator=torch.Generator().manual_seed(i)) for i in (1, 2)]
    x[which][0, at, 0, 7] = float("nan")
    p, _ = written(fia, *x, G)
    B = 33 * 152 * (16 if n1 * Q <= 8 else 8 if n1 * Q <= 16 else 2) // (min(W * bs, pre + Q) // 16) + 1
    q = torch.randn(1, n1, Q, D, generator=torch.Generator().manual_seed(3)).bfloat16().expand(B, -1, -1, -1).contiguous()
    lens = torch.where(torch.arange(B) % 3 == 0, L, torch.arange(B) % 24).to(torch.int32).to(DEV)
    table = torch.arange(W, dtype=torch.int32).clamp(max=3).expand(B, W).contiguous().to(DEV)
    kw = dict(actual_seq_kvlen=lens, block_table=table, block_size=bs, num_heads=n1, num_key_value_heads=1, scale_value=0.1,
              input_layout="BNSD", pre_tokens=pre, softmax_lse_flag=True)
    assert shared_evenly(fia, q.to(DEV), p, **kw)
    out, lse = fia.fia_decode_window_int4(q.to(DEV), *p, **kw)
    i = np.arange(L - Q, L)
    see = torch.from_numpy((at <= i) & (at >= i - pre))
    assert see.any() and not see.all()
    group = slice(7 // G * G, 7 // G * G + G) if which else slice(0, D)
    bad = torch.zeros(n1, Q, D, dtype=torch.bool)
    bad[:, see, group] = True
    nan = out.isnan().cpu()
    assert (nan[::3] == bad).all() and not nan[1::3].any() and not nan[2::3].any()


def test_a_call_that_needs_a_workspace_records_no_error(fia):
    """The binding makes the workspace of a call with much work, and the last error stays that of the last call that failed."""
    from attention_fia_prefill_gb300 import _binding as B
    lib = B.load_library()
    g = torch.Generator().manual_seed(1)
    p, table = written(fia, *(torch.randn(2, 40, 1, 64, generator=g) for _ in range(2)), 64)
    q = torch.randn(2, 4, 1, 64, generator=g).bfloat16()
    with pytest.raises(fia.FIAError, match="in blocks of 16"):
        fia.fia_decode_window_int4(q.to(DEV), *p, actual_seq_kvlen=i32([1, 1]), block_table=table.to(DEV), block_size=-3, num_heads=4,
                                   num_key_value_heads=1, input_layout="BNSD")
    said = lib.fia_last_error()
    for room in (0, SHARED):
        attend(fia, q, p, table, [40, 3], room=room)
        assert lib.fia_last_error() == said
