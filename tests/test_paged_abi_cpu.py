"""The paged-serving entry points on the host, without a GPU: what they refuse
and with which status, before any CUDA call; and the plain oracle against
closed forms."""
import ctypes

import numpy as np
import pytest

from attention_fia_prefill_gb300 import _binding as B
from attention_fia_prefill_gb300 import build as fia_build
from oracle import paged_oracle as po

P = 1 << 20          # a fake, 16-byte aligned device address (never dereferenced)
F16, BF16, F32, I32, I64, E4M3 = B.DTYPE_F16, B.DTYPE_BF16, B.DTYPE_F32, B.DTYPE_I32, B.DTYPE_I64, B.DTYPE_F8E4M3


@pytest.fixture(scope="module")
def lib():
    fia_build.build()
    return B.load_library()


def t(shape, dtype=BF16, ptr=P):
    return bytes(B.raw_desc(ptr, dtype, shape))


def code(status):
    return B.STATUS_NAMES[status]


# ------------------------------------------------------------------ tables
def tables(lib, B_=4, F=8, W=6, T=10, bs=16, **kw):
    a = dict(ctx=t((B_,), I32, P), new=t((B_,), I32, P + 4096), free=t((F,), I32, P + 8192), table=t((B_, W), I32, P + 12288),
             slots=t((T,), I32, P + 16384), kv=t((B_,), I32, P + 20480), cu=t((B_,), I32, P + 24576),
             nb=t((1,), I32, P + 28672))
    a.update(kw)
    return code(lib.fia_block_table_append(a["ctx"], a["new"], a["free"], bs, a["table"], a["slots"], a["kv"], a["cu"],
                                           a["nb"], None))


@pytest.mark.parametrize("kw,status", [
    (dict(ctx=None), "FIA_ERR_NULL"), (dict(nb=None), "FIA_ERR_NULL"), (dict(table=None), "FIA_ERR_NULL"),
    (dict(ctx=t((4,), I32, None)), "FIA_ERR_NULL"),
    (dict(new=t((4,), I64)), "FIA_ERR_DTYPE"), (dict(table=t((4, 6), I64)), "FIA_ERR_DTYPE"),
    (dict(new=t((5,), I32)), "FIA_ERR_SHAPE"), (dict(kv=t((3,), I32)), "FIA_ERR_SHAPE"),
    (dict(slots=t((2, 5), I32)), "FIA_ERR_SHAPE"), (dict(nb=t((2,), I32)), "FIA_ERR_SHAPE"),
    (dict(table=t((5, 6), I32)), "FIA_ERR_BLOCK_TABLE"), (dict(bs=0), "FIA_ERR_BLOCK_TABLE"),
    (dict(bs=-16), "FIA_ERR_BLOCK_TABLE"), (dict(bs=2 ** 40), "FIA_ERR_BLOCK_TABLE"),
    (dict(free=t((8,), I32, P + 2)), "FIA_ERR_ALIGNMENT"), (dict(table=t((4, 6), I32, P + 12289)), "FIA_ERR_ALIGNMENT"),
    (dict(kv=t((4,), I32, P)), "FIA_ERR_UNSUPPORTED"),            # in place over context_lens
    (dict(cu=t((4,), I32, P + 20488)), "FIA_ERR_UNSUPPORTED"),    # over kv_lens
    (dict(slots=t((10,), I32, P + 8192 + 28)), "FIA_ERR_UNSUPPORTED"),
])
def test_tables_refusals(lib, kw, status):
    assert tables(lib, **kw) == status
    assert lib.fia_last_error()


# ------------------------------------------------------------------ cache write
def write(lib, T=10, n=2, d=64, nb=5, bs=16, ks=0, vs=0, **kw):
    a = dict(k=t((T, n, d)), v=t((T, n, d)), kc=t((nb, n, bs, d)), vc=t((nb, n, bs, d)), slots=t((T,), I32))
    a.update(kw)
    return code(lib.fia_cache_write(a["k"], ks, a["v"], vs, a["kc"], a["vc"], a["slots"], None))


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), "FIA_ERR_NULL"), (dict(kc=None), "FIA_ERR_NULL"), (dict(v=None), "FIA_ERR_NULL"),
    (dict(vc=None), "FIA_ERR_NULL"), (dict(slots=None), "FIA_ERR_NULL"),
    (dict(k=t((10, 2, 64), F32)), "FIA_ERR_DTYPE"), (dict(v=t((10, 2, 64), F16)), "FIA_ERR_DTYPE"),
    (dict(slots=t((10,), I64)), "FIA_ERR_DTYPE"),
    (dict(k=t((9, 2, 64))), "FIA_ERR_SHAPE"), (dict(k=t((10, 128))), "FIA_ERR_SHAPE"),
    (dict(kc=t((5, 3, 16, 64))), "FIA_ERR_SHAPE"), (dict(vc=t((6, 2, 16, 64))), "FIA_ERR_SHAPE"),
    (dict(vc=t((5, 2, 32, 64))), "FIA_ERR_SHAPE"), (dict(kc=t((5, 16, 64))), "FIA_ERR_SHAPE"),
    (dict(kc=t((5, 2))), "FIA_ERR_SHAPE"), (dict(k=t((10, 0, 64))), "FIA_ERR_SHAPE"),
    (dict(k=t((10, 2, 4)), v=t((10, 2, 4)), kc=t((5, 2, 16, 4)), vc=t((5, 2, 16, 4))), "FIA_ERR_UNSUPPORTED"),
    (dict(ks=64), "FIA_ERR_ALIGNMENT"), (dict(vs=132), "FIA_ERR_ALIGNMENT"), (dict(ks=-128), "FIA_ERR_ALIGNMENT"),
    (dict(k=t((10, 2, 64), BF16, P + 8)), "FIA_ERR_ALIGNMENT"), (dict(kc=t((5, 2, 16, 64), BF16, P + 2)), "FIA_ERR_ALIGNMENT"),
    (dict(kc=t((5, 2, 0, 64)), vc=t((5, 2, 0, 64))), "FIA_ERR_BLOCK_TABLE"),
])
def test_write_refusals(lib, kw, status):
    assert write(lib, **kw) == status


def test_write_without_tokens_or_blocks(lib):
    assert write(lib, T=0, k=t((0, 2, 64), BF16, None), v=t((0, 2, 64), BF16, None), slots=t((0,), I32, None)) == "FIA_OK"
    assert write(lib, nb=0, kc=t((0, 2, 16, 64), BF16, None), vc=t((0, 2, 16, 64), BF16, None)) == "FIA_OK"


@pytest.mark.parametrize("kw,names", [
    (dict(k=t((10, 2, 64), BF16, P)), "key or value"),                                   # key inside key_cache
    (dict(v=t((10, 2, 64), BF16, P + 5 * 2 * 16 * 64 * 2 - 16)), "key or value"),        # its last 16 bytes
    (dict(k=t((10, 2, 64), BF16, P - 9 * 1024 - 240), ks=512), "key or value"),          # a strided key's last row
    (dict(vc=t((5, 2, 16, 64), BF16, P + 4096)), "key_cache and value_cache"),
])
def test_write_refuses_overlaps(lib, kw, names):
    far = dict(k=t((10, 2, 64), BF16, P + (1 << 20)), v=t((10, 2, 64), BF16, P + (2 << 20)), vc=t((5, 2, 16, 64), BF16, P + (3 << 20)))
    assert write(lib, **{**far, **kw}) == "FIA_ERR_UNSUPPORTED"
    assert names in lib.fia_last_error().decode()


# ------------------------------------------------------------------ windowed decode
def window(lib, B_=2, n1=8, n2=2, Q=1, D=128, nb=9, bs=32, sink=4, prm=None, **kw):
    p = dict(num_heads=n1, num_key_value_heads=n2, input_layout="BNSD", block_size=bs, pre_tokens=100)
    p.update(prm or {})
    q = t((B_, n1, Q, D))
    a = dict(q=q, k=t((nb, n2, bs, D)), v=t((nb, n2, bs, D)), table=t((B_, 4), I32), lens=t((B_,), I32), out=q, lse=None)
    a.update(kw)
    return code(lib.fia_decode_window(a["q"], a["k"], a["v"], a["table"], a["lens"], ctypes.byref(B.Params(**p).p), sink,
                                      a["out"], a["lse"], None))


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), "FIA_ERR_NULL"), (dict(k=None), "FIA_ERR_NULL"), (dict(out=None), "FIA_ERR_NULL"),
    (dict(prm=dict(input_layout="XYZ")), "FIA_ERR_LAYOUT"), (dict(prm=dict(input_layout="TND")), "FIA_ERR_UNSUPPORTED"),
    (dict(k=t((9, 2, 32, 128), F16)), "FIA_ERR_DTYPE"), (dict(q=t((2, 8, 1, 128), F32)), "FIA_ERR_DTYPE"),
    (dict(out=t((2, 8, 1, 128), F16)), "FIA_ERR_DTYPE"), (dict(out=t((2, 8, 2, 128))), "FIA_ERR_SHAPE"),
    (dict(n1=7), "FIA_ERR_HEADS"), (dict(n1=130, n2=2), "FIA_ERR_HEADS"), (dict(Q=17), "FIA_ERR_UNSUPPORTED"),
    (dict(n1=64, n2=2, Q=3), "FIA_ERR_UNSUPPORTED"), (dict(D=192), "FIA_ERR_UNSUPPORTED"), (dict(D=96), "FIA_ERR_UNSUPPORTED"),
    (dict(bs=24), "FIA_ERR_BLOCK_TABLE"), (dict(bs=0), "FIA_ERR_BLOCK_TABLE"), (dict(table=t((3, 4), I32)), "FIA_ERR_BLOCK_TABLE"),
    (dict(table=t((2, 4), I64)), "FIA_ERR_BLOCK_TABLE"), (dict(table=t((2, 0), I32, None)), "FIA_ERR_BLOCK_TABLE"),
    (dict(table=t((2, 4), I32, P + 2)), "FIA_ERR_ALIGNMENT"),
    (dict(v=t((9, 2, 32, 64))), "FIA_ERR_SHAPE"), (dict(k=t((9, 4, 32, 128)), v=t((9, 4, 32, 128))), "FIA_ERR_SHAPE"),
    (dict(lens=None), "FIA_ERR_SEQLEN"), (dict(lens=t((3,), I32)), "FIA_ERR_SHAPE"), (dict(lens=t((2,), I64)), "FIA_ERR_DTYPE"),
    (dict(lens=t((2,), I32, P + 1)), "FIA_ERR_ALIGNMENT"), (dict(prm=dict(actual_seq_kvlen=[4, 4])), "FIA_ERR_SEQLEN"),
    (dict(prm=dict(scale_value=0.0)), "FIA_ERR_UNSUPPORTED"), (dict(prm=dict(scale_value=float("nan"))), "FIA_ERR_UNSUPPORTED"),
    (dict(prm=dict(pre_tokens=-1)), "FIA_ERR_UNSUPPORTED"), (dict(sink=-1), "FIA_ERR_UNSUPPORTED"),
    (dict(q=t((2, 8, 1, 128), BF16, P + 2)), "FIA_ERR_ALIGNMENT"), (dict(k=t((9, 2, 32, 128), BF16, P + 8)), "FIA_ERR_ALIGNMENT"),
    (dict(prm=dict(softmax_lse_flag=True)), "FIA_ERR_NULL"),
    (dict(prm=dict(softmax_lse_flag=True), lse=t((2, 8, 1), F32)), "FIA_ERR_SHAPE"),
    (dict(table=t((2, 2 ** 26), I32)), "FIA_ERR_SHAPE"),
    (dict(table=None, k=t((2, 3, 50, 128)), v=t((2, 3, 50, 128))), "FIA_ERR_HEADS"),
    (dict(table=None, k=t((3, 2, 50, 128)), v=t((3, 2, 50, 128))), "FIA_ERR_SHAPE"),
])
def test_window_refusals(lib, kw, status):
    assert window(lib, **kw) == status


def test_window_empty_query(lib):
    assert window(lib, B_=0, q=t((0, 8, 1, 128), BF16, None), out=t((0, 8, 1, 128), BF16, None)) == "FIA_OK"


# ------------------------------------------------------------------ the binding's own checks
def test_binding_refuses_before_the_library(lib):
    torch = pytest.importorskip("torch")
    import attention_fia_prefill_gb300 as fia
    x = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fia.fia_block_table_append(x, x, x, torch.zeros(4, 2, dtype=torch.int32), block_size=16, num_tokens=4)
    with pytest.raises(TypeError, match="tensor"):
        fia.fia_block_table_append([1, 2], x, x, x, block_size=16, num_tokens=4)
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fia.fia_cache_write(k, k, k, k, x)


# ------------------------------------------------------------------ the oracle
def test_oracle_window_counts():
    """Closed form: row p of L keys sees min(p, pre) + 1 keys of its window and the sinks before it."""
    for n, L, pre, sink in [(5, 9, 3, 2), (9, 9, 0, 0), (4, 4, 100, 100), (1, 30, 7, 12)]:
        see = po.window_see(n, L, pre, sink)
        for i in range(n):
            p = L - n + i
            lo = max(p - pre, 0)
            assert see[i].sum() == p - lo + 1 + min(sink, lo)


def test_oracle_attend_against_softmax():
    torch = pytest.importorskip("torch")
    g = np.random.default_rng(0)
    q, k, v = g.normal(size=(3, 4, 8)), g.normal(size=(11, 2, 8)), g.normal(size=(11, 2, 8))
    see = po.window_see(3, 11, 4, 2)
    out, lse, av, _ = po.attend(q, k, v, see, 0.3)
    for h in range(4):
        s = torch.tensor(0.3 * q[:, h] @ k[:, h // 2].T).masked_fill(torch.tensor(~see), -np.inf)
        assert np.allclose(out[:, h], torch.softmax(s, -1).numpy() @ v[:, h // 2], atol=1e-14)
        assert np.allclose(lse[:, h], torch.logsumexp(s, -1).numpy(), atol=1e-14)
        assert (av[:, h] >= np.abs(out[:, h]) - 1e-14).all()


def test_oracle_tables_invariants():
    """Every token has a slot of its own in a block of its request, and no block is handed out twice."""
    ctx, new, bs = [0, 3, 8, 5], [4, 0, 9, 7], 4
    table = np.full((4, 6), -7)
    used = iter(range(100))
    for b, c in enumerate(ctx):
        for i in range(-(-c // bs)):
            table[b, i] = next(used)
    tab, slots, kv, cu, n = po.block_table_append(ctx, new, list(range(50, 80)), table, bs, 20)
    assert kv == [4, 3, 17, 12] and cu == [4, 4, 13, 20] and n == 1 + 0 + 3 + 1
    assert len(set(slots)) == 20 and min(slots) >= 0
    ids = tab[tab >= 0]
    assert len(set(ids.tolist())) == len(ids) == 1 + 1 + 5 + 3
    at = 0
    for b in range(4):
        for i in range(new[b]):
            assert slots[at] == tab[b, (ctx[b] + i) // bs] * bs + (ctx[b] + i) % bs
            at += 1


# ------------------------------------------------------------------ windowed prefill
def prefill(lib, layout="TND", T=500, n1=8, n2=2, D=128, B_=3, bs=0, sink=4, prm=None, ws=P, wsb=256, size=False, **kw):
    p = dict(num_heads=n1, num_key_value_heads=n2, input_layout=layout, block_size=bs, pre_tokens=100)
    p.update(prm or {})
    if layout == "TND":
        q, k = t((T, n1, D)), t((T, n2, D))
    else:
        q, k = t((B_, n1, T, D)), t((B_, n2, T, D))
    if bs:
        k = t((20, n2, bs, D))
    a = dict(q=q, k=k, v=k, table=t((B_, 8), I32) if bs else None, ql=t((B_,), I32), kl=t((B_,), I32), out=q, lse=None)
    a.update(kw)
    args = [a["q"], a["k"], a["v"], a["table"], a["ql"], a["kl"], ctypes.byref(B.Params(**p).p), sink, a["out"], a["lse"]]
    n = ctypes.c_size_t(0)
    r = code(lib.fia_prefill_window_get_workspace_size(*args, ctypes.byref(n)))
    if size:
        return r, n.value
    # the execute call refuses the same
    return r if r == "FIA_OK" else (r, code(lib.fia_prefill_window(*args, ws, wsb, None)))


PREFILL_REFUSALS = [
    (dict(q=None), "FIA_ERR_NULL"), (dict(v=None), "FIA_ERR_NULL"), (dict(prm=dict(input_layout="NTD")), "FIA_ERR_LAYOUT"),
    (dict(k=t((500, 2, 128), F16)), "FIA_ERR_DTYPE"), (dict(out=t((500, 8, 128), F16)), "FIA_ERR_DTYPE"),
    (dict(ql=None), "FIA_ERR_SEQLEN"), (dict(kl=None), "FIA_ERR_SEQLEN"), (dict(ql=t((3,), I64)), "FIA_ERR_DTYPE"),
    (dict(ql=t((4097,), I32)), "FIA_ERR_SEQLEN"), (dict(kl=t((2,), I32)), "FIA_ERR_SHAPE"), (dict(ql=t((3, 1), I32)), "FIA_ERR_SHAPE"),
    (dict(prm=dict(actual_seq_qlen=[5])), "FIA_ERR_SEQLEN"), (dict(n1=6, n2=4), "FIA_ERR_HEADS"),
    (dict(n1=130, n2=2), "FIA_ERR_HEADS"), (dict(D=192), "FIA_ERR_UNSUPPORTED"), (dict(sink=-2), "FIA_ERR_UNSUPPORTED"),
    (dict(prm=dict(pre_tokens=-3)), "FIA_ERR_UNSUPPORTED"), (dict(prm=dict(scale_value=-1.0)), "FIA_ERR_UNSUPPORTED"),
    (dict(v=t((400, 2, 128))), "FIA_ERR_SHAPE"), (dict(out=t((500, 4, 128))), "FIA_ERR_SHAPE"),
    (dict(q=t((500, 8, 128), BF16, P + 4), out=t((500, 8, 128))), "FIA_ERR_ALIGNMENT"),
    (dict(prm=dict(softmax_lse_flag=True)), "FIA_ERR_NULL"),
    (dict(prm=dict(softmax_lse_flag=True), lse=t((500, 8, 2), F32)), "FIA_ERR_SHAPE"),
    (dict(bs=64), "FIA_ERR_BLOCK_TABLE"), (dict(bs=640), "FIA_ERR_BLOCK_TABLE"), (dict(bs=200), "FIA_ERR_BLOCK_TABLE"),
    (dict(bs=128, table=t((4, 8), I32)), "FIA_ERR_BLOCK_TABLE"), (dict(bs=128, kl=None), "FIA_ERR_SEQLEN"),
    (dict(bs=128, table=t((3, 0), I32, None)), "FIA_ERR_BLOCK_TABLE"),
    (dict(bs=128, k=t((20, 4, 128, 128)), v=t((20, 4, 128, 128))), "FIA_ERR_SHAPE"),
    (dict(layout="BNSD", ql=t((4,), I32)), "FIA_ERR_SHAPE"), (dict(layout="BNSD", k=t((2, 2, 500, 128)), v=t((2, 2, 500, 128))), "FIA_ERR_SHAPE"),
]


@pytest.mark.parametrize("kw,status", PREFILL_REFUSALS)
def test_prefill_window_refusals(lib, kw, status):
    assert prefill(lib, **kw) == (status, status)


def test_prefill_window_workspace(lib):
    assert prefill(lib, size=True) == ("FIA_OK", 256)
    assert prefill(lib, layout="BNSD", ql=None, kl=None, size=True) == ("FIA_OK", 256)
    q, k = t((500, 8, 128)), t((500, 2, 128))
    prm = B.Params(num_heads=8, num_key_value_heads=2, input_layout="TND")
    for ws, n, want in ((None, 256, "FIA_ERR_WORKSPACE"), (P, 255, "FIA_ERR_WORKSPACE"), (P + 8, 256, "FIA_ERR_ALIGNMENT")):
        r = lib.fia_prefill_window(q, k, k, None, t((3,), I32), t((3,), I32), ctypes.byref(prm.p), 0, q, None, ws, n, None)
        assert code(r) == want


# ------------------------------------------------------------------ shared prefix
def prefix(lib, B_=4, n1=8, n2=2, Q=1, D=128, nb=40, bs=128, cols=8, P_len=512, prm=None, ws=P, wsb=1 << 30, **kw):
    p = dict(num_heads=n1, num_key_value_heads=n2, input_layout="BNSD", block_size=bs)
    p.update(prm or {})
    q = t((B_, n1, Q, D))
    a = dict(q=q, k=t((nb, n2, bs, D)), v=t((nb, n2, bs, D)), table=t((B_, cols), I32), lens=t((B_,), I32), out=q, lse=None)
    a.update(kw)
    args = [a["q"], a["k"], a["v"], a["table"], a["lens"], ctypes.byref(B.Params(**p).p), P_len, a["out"], a["lse"]]
    n = ctypes.c_size_t(0)
    r = code(lib.fia_decode_shared_prefix_get_workspace_size(*args, ctypes.byref(n)))
    return (r, n.value) if r == "FIA_OK" else (r, code(lib.fia_decode_shared_prefix(*args, ws, wsb, None)))


@pytest.mark.parametrize("kw,status", [
    (dict(table=None), "FIA_ERR_SHAPE"), (dict(table=None, k=t((4, 2, 128, 128)), v=t((4, 2, 128, 128))), "FIA_ERR_BLOCK_TABLE"),
    (dict(P_len=100), "FIA_ERR_SEQLEN"), (dict(P_len=-128), "FIA_ERR_SEQLEN"), (dict(P_len=8 * 128 + 128), "FIA_ERR_SEQLEN"),
    (dict(bs=48, P_len=48), "FIA_ERR_BLOCK_TABLE"), (dict(bs=192, P_len=192), "FIA_ERR_BLOCK_TABLE"), (dict(lens=None), "FIA_ERR_SEQLEN"),
    (dict(q=None), "FIA_ERR_NULL"), (dict(D=192), "FIA_ERR_UNSUPPORTED"), (dict(n1=48, n2=1, Q=2), "FIA_ERR_UNSUPPORTED"),
    (dict(prm=dict(input_layout="TND")), "FIA_ERR_UNSUPPORTED"), (dict(v=t((40, 2, 64, 128))), "FIA_ERR_SHAPE"),
    (dict(k=t((40, 2, 128, 128), F16)), "FIA_ERR_DTYPE"), (dict(prm=dict(actual_seq_kvlen=[9])), "FIA_ERR_SEQLEN"),
])
def test_prefix_refusals(lib, kw, status):
    assert prefix(lib, **kw) == (status, status)


def test_prefix_workspace(lib):
    """One sequence, or no prefix: the status word; else whole splits of fp32 rows."""
    assert prefix(lib, B_=1) == ("FIA_OK", 256) and prefix(lib, P_len=0) == ("FIA_OK", 256)
    r, n = prefix(lib)
    one = 4 * 8 * (128 * 4 + 8)
    assert r == "FIA_OK" and n > 256 and 1 <= (n - 256) / one <= 4.1
    q, k = t((4, 8, 1, 128)), t((40, 2, 128, 128))
    prm = B.Params(num_heads=8, num_key_value_heads=2, input_layout="BNSD", block_size=128)
    for ws, have, want in ((None, n, "FIA_ERR_WORKSPACE"), (P, 256, "FIA_ERR_WORKSPACE"), (P + 8, n, "FIA_ERR_ALIGNMENT")):
        assert code(lib.fia_decode_shared_prefix(q, k, k, t((4, 8), I32), t((4,), I32), ctypes.byref(prm.p), 512, q, None, ws,
                                                 have, None)) == want


@pytest.mark.parametrize("scale", [1e-60, 1e-39, 1e300, float("inf")])
def test_scale_has_to_fit_fp32(lib, scale):
    """A factor that is 0 (or infinite) in fp32 times a hidden score of -inf is a NaN."""
    assert window(lib, prm=dict(scale_value=scale)) == "FIA_ERR_UNSUPPORTED"
    assert prefill(lib, prm=dict(scale_value=scale)) == ("FIA_ERR_UNSUPPORTED",) * 2
    assert prefix(lib, prm=dict(scale_value=scale)) == ("FIA_ERR_UNSUPPORTED",) * 2
