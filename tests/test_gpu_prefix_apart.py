"""Decode behind a shared prefix with the prefix on a kernel of its own (the sizes
of these tests would have every sequence read it): steps, captured steps replayed
with new lengths, streams, calls that follow one another with nothing in between,
offsets past 2^31.  The decode kernel behind the prefix's reads lengths, tables,
queries and keys without waiting for it, so whatever wrote them has to be done."""
import numpy as np
import pytest
import torch

from attention_fia_prefill_gb300 import _binding
from oracle import paged_oracle as po
from oracle.fia_oracle import f64
from tests.test_gpu_paged_serving import Server, _prefix_case, check_decode

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.fixture(autouse=True)
def apart():
    lib = _binding.load_library()
    lib.fia_debug_set_prefix_path(1)
    yield
    lib.fia_debug_set_prefix_path(0)


# (rows of a unit 4, 8, 32 and 64: the decode kernel's three forms behind the prefix's)
UNITS = [(8, 2, 1), (8, 2, 2), (32, 2, 2), (64, 1, 1)]


def test_the_prefix_kernel_is_the_one_that_runs(fia):
    """Its partial results are in the workspace, and the other path's bits are not the same."""
    q, k, v, kw = _prefix_case(3)
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device=DEV)
    fia.fia_decode_shared_prefix(q, k, v, shared_prefix_len=512, workspace=ws, **kw)
    assert ws[256:].count_nonzero() > 0
    _binding.load_library().fia_debug_set_prefix_path(2)
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device=DEV)
    fia.fia_decode_shared_prefix(q, k, v, shared_prefix_len=512, workspace=ws, **kw)
    assert ws[256:].count_nonzero() == 0


@pytest.mark.parametrize("n1,n2,Q", UNITS)
def test_decode_steps(fia, n1, n2, Q):
    B = 6
    s = Server(fia, B, n1, n2, 128, 64, 60, 16, pre=0, sink=0, prefix=320)
    for step in range(70 // Q):   # past a page boundary of every sequence
        x = s.new_tokens(None, B * Q, seed=step)
        out = s.decode(i32([Q] * B), x.to(DEV), Q)
        refs = s.expect([Q] * B, x)
        if step in (0, 1, 31, 32, 64, 69):
            check_decode(out, refs, Q)


@pytest.mark.parametrize("n1,n2,Q", UNITS)
def test_captured_step_replays_with_new_lengths(fia, n1, n2, Q):
    B = 5
    s = Server(fia, B, n1, n2, 64, 32, 90, 24, pre=0, sink=0, prefix=256)
    x = torch.empty(B * Q, n1 + 2 * n2, 64, dtype=torch.bfloat16, device=DEV)
    new = i32([Q] * B)
    first = s.new_tokens(None, B * Q, seed=1)
    x.copy_(first)
    check_decode(s.decode(new, x, Q), s.expect([Q] * B, first), Q)     # eager, also loads the kernels
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = s.decode(new, x, Q)
    for step in range(30):
        tok = s.new_tokens(None, B * Q, seed=100 + step)
        x.copy_(tok)
        graph.replay()
        refs = s.expect([Q] * B, tok)
        if step % 13 == 0 or step == 29:
            torch.cuda.synchronize()
            check_decode(out, refs, Q)


def _call(fia, c, **more):
    q, k, v, kw = c
    return fia.fia_decode_shared_prefix(q, k, v, shared_prefix_len=512, **{**kw, **more})


def test_captured_lengths_shrink_and_grow(fia):
    """A replay reads the lengths of its own time: inside the prefix, none at all, and back; the same bits as eager."""
    c = _prefix_case(11)
    lens = c[3]["actual_seq_kvlen"]
    first = lens.clone()
    _call(fia, c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = _call(fia, c)
    r = np.random.default_rng(0)
    for step in range(12):
        new = first if step % 4 == 3 else i32([int(min(x, n)) for x, n in zip(r.integers(0, 700, len(first)), first.tolist())])
        lens.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        want, want_l = _call(fia, c)
        assert torch.equal(out, want) and torch.equal(lse, want_l)


def test_two_graphs_share_a_workspace(fia):
    """Replayed in turn on one stream, with nothing in between: each is through with it before the next begins."""
    a, b = _prefix_case(21), _prefix_case(22, B=7)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    want = [_call(fia, c)[0] for c in (a, b)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_call(fia, c, workspace=ws)[0])
        graphs.append(g)
    for _ in range(20):
        for o in outs:
            o.zero_()
        for g in graphs + graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    assert fia.fia_device_status(ws) == 0


def test_two_streams_at_once(fia):
    """Many calls in flight on two streams, among them the kernels that hold TMEM: the same bits as alone."""
    cases = [_prefix_case(i) for i in range(2)]
    wide = []
    for i in range(2):
        g = torch.Generator().manual_seed(40 + i)
        q, k, v, kw = _prefix_case(30 + i)
        q = torch.randn(q.shape[0], 64, 1, 128, generator=g).bfloat16().to(DEV)
        wide.append((q, k, v, {**kw, "num_heads": 64}))

    def calls(i):
        q, k, v, kw = wide[i]
        return [_call(fia, cases[i])[0], _call(fia, wide[i])[0], fia.fia_decode_window(q, k, v, pre_tokens=700, **kw)[0],
                fia.fia_prefill_window(cases[i][0].reshape(1, 8, -1, 128).contiguous(), k.reshape(1, 2, -1, 128),
                                       v.reshape(1, 2, -1, 128), num_heads=8, num_key_value_heads=2, input_layout="BNSD",
                                       pre_tokens=100, sink_tokens=1)[0], _call(fia, wide[i])[0]]

    alone = [calls(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        got = []
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got.append(calls(i))
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("n1", [8, 64])
def test_back_to_back_calls_see_each_others_writes(fia, n1):
    """Keys, lengths and queries rewritten between calls, with nothing waiting in between: every call sees the newest."""
    q, k, v, kw = _prefix_case(5)
    q = torch.randn(q.shape[0], n1, 1, 128, device=DEV).bfloat16()
    kw["num_heads"] = n1
    n, lens = k.shape[0] * 64, kw["actual_seq_kvlen"]
    rows = [torch.randn(n, 2, 128, device=DEV).bfloat16() for _ in range(4)]
    some = [lens - i for i in range(4)]
    slots, B = torch.arange(n, dtype=torch.int32, device=DEV), len(lens)
    spare = [torch.zeros(B, 64, dtype=torch.int32, device=DEV), i32([0])]

    def step(i, q):
        fia.fia_cache_write(rows[i], rows[i], k, v, slots)
        # the lengths come from a table update: some[i] held, none new
        fia.fia_block_table_append(some[i], torch.zeros_like(lens), spare[1], spare[0], block_size=64, num_tokens=0, kv_lens=lens)
        return fia.fia_decode_shared_prefix(q, k, v, shared_prefix_len=512, **kw)[0]

    want, x = [], q
    for i in range(4):
        x = step(i, x)
        torch.cuda.synchronize()
        want.append(x)
    for _ in range(5):
        got, x = [], q
        for i in range(4):
            x = step(i, x)      # a call's output is the next one's query
            got.append(x)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_events_around_the_prefix_kernel(fia):
    """fia_profile_next_call's events lie between the two kernels; the result is the same."""
    c = _prefix_case(9)
    want = _call(fia, c)[0]
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    for e in ev:
        e.record()
    _binding.profile_next_call(*ev)
    got = _call(fia, c)[0]
    torch.cuda.synchronize()
    assert torch.equal(want, got) and ev[0].elapsed_time(ev[1]) > 0


@pytest.mark.parametrize("n1", [16, 512])
def test_cache_past_32_bit_offsets(fia, n1):
    """Pools of 2.6e9 elements: the prefix and the sequences' own keys in their last blocks."""
    nblk, n2, bs, D, P = 20000, 8, 128, 128, 256
    kc, vc = (torch.empty(nblk, n2, bs, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    own = [300, 1, 129]
    lens, B = [P + n for n in own], len(own)
    g = torch.Generator().manual_seed(8)
    x = torch.randn(P + sum(own), 2 * n2, D, generator=g).bfloat16()
    free = torch.arange(nblk - 1, nblk - 41, -1, dtype=torch.int32, device=DEV)
    # the prefix as a request of its own, then the sequences' own keys behind P tokens held
    shared = torch.zeros(1, 2, dtype=torch.int32, device=DEV)
    slots, _, _, used = fia.fia_block_table_append(i32([0]), i32([P]), free, shared, block_size=bs, num_tokens=P)
    table = torch.zeros(B, 8, dtype=torch.int32, device=DEV)
    table[:, :2] = shared
    more, kv, _, _ = fia.fia_block_table_append(i32([P] * B), i32(own), free[int(used):].contiguous(), table, block_size=bs,
                                                num_tokens=sum(own))
    xd = x.to(DEV)
    fia.fia_cache_write(xd[:, :n2], xd[:, n2:], kc, vc, torch.cat([slots, more]))
    assert int(torch.cat([slots, more]).min()) > (nblk - 41) * bs
    q = torch.randn(B, n1, 1, D, generator=g).bfloat16()
    out, lse = fia.fia_decode_shared_prefix(q.to(DEV), kc, vc, block_table=table, block_size=bs, actual_seq_kvlen=kv,
                                            shared_prefix_len=P, num_heads=n1, num_key_value_heads=n2, scale_value=0.09,
                                            input_layout="BNSD", softmax_lse_flag=True)
    f, at, rows = f64(x), P, []
    for n in own:
        rows.append(tuple(np.concatenate([f[:P, c], f[at:at + n, c]]) for c in (slice(0, n2), slice(n2, 2 * n2))))
        at += n
    po.assert_close(out, lse, po.decode(q, rows, lens, 1 << 40, 0, 0.09))
