"""Calls whose bounded waits run out: what they leave behind.  A wait that looks
at a limit of 1 ns gives up; which waits do depends on timing, so the calls are
repeated and every outcome is held against what the header says of it."""
import pytest
import torch

import fia_inputs
from attention_fia_prefill_gb300 import _binding

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class short_waits:
    def __enter__(self):
        _binding.load_library().fia_debug_set_wait_limit_ns(1)

    def __exit__(self, *_):
        torch.cuda.synchronize()
        _binding.load_library().fia_debug_set_wait_limit_ns(0)


def dense(n1, n2, sq, skv, workload, B=1, D=128):
    return [fia_inputs.normal((B, n, s, D), "bf16", workload, i).to(DEV) for i, n, s in ((1, n1, sq), (2, n2, skv), (3, n2, skv))]


def prefix_args(n1, n2, B, P, own, bs=64, D=128, workload=150):
    """A batch behind a prefix of P keys, `own` keys of its own each."""
    pages, mine = P // bs, -(-own // bs)
    q = fia_inputs.normal((B, n1, 1, D), "bf16", workload, 1).to(DEV)
    k, v = (fia_inputs.normal((pages + B * mine, n2, bs, D), "bf16", workload, i).to(DEV) for i in (2, 3))
    table = torch.cat([torch.arange(pages).expand(B, pages), pages + torch.arange(B * mine).view(B, mine)], 1)
    kw = dict(block_table=table.int().to(DEV), block_size=bs, actual_seq_kvlen=i32([P + own] * B), shared_prefix_len=P,
              num_heads=n1, num_key_value_heads=n2, scale_value=D ** -0.5, input_layout="BNSD")
    return (q, k, v), kw


def calls(fia):
    """name -> one call; sizes whose CTAs load all their keys at once among them."""
    q, k, v = dense(8, 2, 1, 200, 140)
    d = dict(num_heads=8, num_key_value_heads=2, input_layout="BNSD", scale_value=0.09)
    few, many = dense(8, 2, 300, 200, 141), dense(8, 2, 700, 1500, 142)
    wq, wk, wv = dense(64, 1, 1, 100, 146, B=40)
    lq, lk, lv = dense(64, 1, 1, 3000, 147, B=4)
    w = dict(num_heads=64, num_key_value_heads=1, input_layout="BNSD", scale_value=0.09)
    pa, pk = prefix_args(16, 2, 40, 1024, 90)
    ea, ek = prefix_args(64, 1, 8, 256, 300)

    def apart(args, kw, path):
        lib = _binding.load_library()
        lib.fia_debug_set_prefix_path(path)
        try:
            return fia.fia_decode_shared_prefix(*args, **kw)[0]
        finally:
            lib.fia_debug_set_prefix_path(0)

    return {
        "prefill": lambda: fia.fia_prefill(*few, sparse_mode=2, **d)[0],
        "prefill many keys": lambda: fia.fia_prefill(*many, **d)[0],
        "decode": lambda: fia.fia_decode(q, k, v, **d)[0],
        "window prefill": lambda: fia.fia_prefill_window(*few, pre_tokens=60, sink_tokens=3, **d)[0],
        "window prefill many keys": lambda: fia.fia_prefill_window(*many, **d)[0],
        "window decode": lambda: fia.fia_decode_window(wq, wk, wv, **w)[0],
        "window decode many keys": lambda: fia.fia_decode_window(lq, lk, lv, **w)[0],
        "prefix apart": lambda: apart(pa, pk, 1),
        "prefix apart, wide": lambda: apart(ea, ek, 1),
        "prefix by every sequence": lambda: apart(ea, ek, 2),
    }


def test_calls_behind_ones_that_gave_up(fia):
    """Every copy and product of a CTA that gives up ends before the CTA does: whatever runs in its place next, with no
    pause in between, gives the bits that it gives alone."""
    ops = calls(fia)
    want = {n: f() for n, f in ops.items()}
    torch.cuda.synchronize()
    lib = _binding.load_library()
    for n, f in ops.items():
        for _ in range(3):
            lib.fia_debug_set_wait_limit_ns(1)
            try:
                for _ in range(5):
                    f()
            finally:
                lib.fia_debug_set_wait_limit_ns(0)   # (a call takes its limit when it is launched)
            got = {m: g() for m, g in ops.items()}
            torch.cuda.synchronize()
            for m, g in got.items():
                assert torch.equal(g, want[m]), (n, m)


def outcomes(call, want, tries=30):
    """(out, status) of short-limit calls, each on a workspace that no call has seen: `call` takes it.  The last call is
    a good one on the last workspace."""
    import attention_fia_prefill_gb300 as fia
    for fill in (0, 255):
        for _ in range(tries):
            ws = torch.full((1 << 24,), fill, dtype=torch.uint8, device=DEV)
            with short_waits():
                out = call(ws)
            yield out, fia.fia_device_status(ws)
        assert torch.equal(call(ws), want) and fia.fia_device_status(ws) == 0


def rows_right_or_nan(out, want):
    """Rows that are NaN (the others have to be right)."""
    o, w = out.reshape(-1, out.shape[-1]), want.reshape(-1, out.shape[-1])
    gone = o.isnan().any(1)
    assert o[gone].isnan().all() and torch.equal(o[~gone], w[~gone])
    return int(gone.sum())


@pytest.mark.parametrize("n1,B", [(64, 8), (24, 20), (40, 3)])
def test_prefix_by_every_sequence_raises_its_status(fia, n1, B):
    """Units of 17..64 rows on a workspace whose status word holds anything: rows that are NaN go with FIA_ERR_TIMEOUT."""
    args, kw = prefix_args(n1, 1, B, 256, 2100)
    lib = _binding.load_library()
    lib.fia_debug_set_prefix_path(2)
    try:
        want = fia.fia_decode_shared_prefix(*args, **kw)[0]
        gave_up = 0
        for out, status in outcomes(lambda ws: fia.fia_decode_shared_prefix(*args, workspace=ws, **kw)[0], want):
            n = rows_right_or_nan(out, want)
            gave_up += n > 0
            assert status == (10 if n else 0)
    finally:
        lib.fia_debug_set_prefix_path(0)
    assert gave_up > 0


def test_wide_window_decode_that_gives_up_leaves_nan(fia):
    """No workspace: NaN in the unit's rows, the others right."""
    q, k, v = dense(64, 1, 1, 3000, 149, B=40)
    kw = dict(num_heads=64, num_key_value_heads=1, scale_value=0.1, input_layout="BNSD")
    want = fia.fia_decode_window(q, k, v, **kw)[0]
    gave_up = 0
    for _ in range(30):
        with short_waits():
            out = fia.fia_decode_window(q, k, v, **kw)[0]
        gave_up += rows_right_or_nan(out, want) > 0
    assert gave_up > 0
    assert torch.equal(fia.fia_decode_window(q, k, v, **kw)[0], want)


@pytest.mark.parametrize("n1,n2,B,P", [(16, 2, 40, 1024), (4, 4, 300, 512), (64, 2, 9, 2048)])
def test_prefix_kernel_that_gives_up_leaves_nan(fia, n1, n2, B, P):
    """A prefix whose kernel gave up is not joined as whatever its workspace held: the rows are NaN, the status says so."""
    args, kw = prefix_args(n1, n2, B, P, 90)
    lib = _binding.load_library()
    lib.fia_debug_set_prefix_path(1)
    try:
        want = fia.fia_decode_shared_prefix(*args, **kw)[0]
        gave_up = 0
        for out, status in outcomes(lambda ws: fia.fia_decode_shared_prefix(*args, workspace=ws, **kw)[0], want):
            n = rows_right_or_nan(out, want)
            gave_up += n > 0
            assert status in (0, 10) and (n == 0 or status == 10)
    finally:
        lib.fia_debug_set_prefix_path(0)
    assert gave_up > 0


def test_window_prefill_that_gives_up_says_so(fia):
    """FIA_ERR_TIMEOUT for a call that left rows unwritten, on a workspace that held anything."""
    x = dense(8, 2, 700, 1500, 148)
    kw = dict(num_heads=8, num_key_value_heads=2, input_layout="BNSD", scale_value=0.09, pre_tokens=300, sink_tokens=4)
    want = fia.fia_prefill_window(*x, **kw)[0]
    gave_up = 0
    for out, status in outcomes(lambda ws: fia.fia_prefill_window(*x, workspace=ws, **kw)[0], want):
        assert status in (0, 10) and (status == 10 or torch.equal(out, want))
        gave_up += status == 10
    assert gave_up > 0
