"""The paged-serving operators together, as a server runs them: lengths on the
GPU -> tables and slots -> write -> attention, step after step, eager and as
one captured step replayed with new lengths; streams, overlapping calls and the
device timeout path."""
import numpy as np
import pytest
import torch

import fia_inputs
from oracle import paged_oracle as po
from oracle.fia_oracle import f64

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Server:
    """Buffers of a small server.  step() grows tables, writes keys and values and attends, all with tensors that stay
    where they are, so that it can be captured; history() is what every sequence has seen, for the oracle."""

    def __init__(self, fia, B, n1, n2, D, bs, pool, cols, pre, sink, prefix=0, layout="BNBD", seed=0):
        self.fia, self.B, self.n1, self.n2, self.D, self.bs = fia, B, n1, n2, D, bs
        self.pre, self.sink, self.prefix = pre, sink, prefix
        shape = (pool, n2, bs, D) if layout == "BNBD" else (pool, bs, n2 * D)
        nan = float("nan")
        self.kc, self.vc = (torch.full(shape, nan, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        r = np.random.default_rng(seed)
        self.ids = i32(r.permutation(pool).tolist())
        self.used = torch.zeros(1, dtype=torch.int64, device=DEV)
        self.table = torch.full((B, cols), -1, dtype=torch.int32, device=DEV)
        self.ctx = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.scale = D ** -0.5
        self.keys, self.vals = ([np.zeros((0, n2, D)) for _ in range(B)] for _ in range(2))
        if prefix:   # one shared prompt: its blocks start every table
            k, v = (torch.randn(prefix, n2, D, device=DEV).bfloat16() for _ in range(2))
            n = prefix // bs
            slots, _, _, used = fia.fia_block_table_append(i32([0]), i32([prefix]), self.ids, torch.zeros(1, n, dtype=torch.int32, device=DEV),
                                                           block_size=bs, num_tokens=prefix)
            fia.fia_cache_write(k, v, self.kc, self.vc, slots)
            self.table[:, :n] = self.ids[:n]
            self.used += used
            self.ctx += prefix
            self.keys, self.vals = ([f64(x)] * B for x in (k, v))

    def new_tokens(self, lens, tokens, q_tokens=None, seed=0):
        """Random projections of a step's new tokens, one fused row each (query heads, key heads, value heads)."""
        g = torch.Generator().manual_seed(seed)
        return torch.randn(tokens, self.n1 + 2 * self.n2, self.D, generator=g).bfloat16()

    def append(self, new, x):
        free = self.ids[(self.used + torch.arange(64, device=DEV)).clamp(max=self.ids.shape[0] - 1)]
        slots, kv, cu, n = self.fia.fia_block_table_append(self.ctx, new, free, self.table, block_size=self.bs,
                                                           num_tokens=x.shape[0])
        self.used += n
        k, v = x[:, self.n1:self.n1 + self.n2], x[:, self.n1 + self.n2:]
        self.fia.fia_cache_write(k, v, self.kc, self.vc, slots)
        return kv, cu

    def decode(self, new, x, Q):
        """x: B * Q tokens, Q for each sequence."""
        kv, _ = self.append(new, x)
        q = x[:, :self.n1].reshape(self.B, Q, self.n1, self.D).contiguous()
        kw = dict(block_table=self.table, block_size=self.bs, actual_seq_kvlen=kv, num_heads=self.n1,
                  num_key_value_heads=self.n2, scale_value=self.scale, input_layout="BSND", softmax_lse_flag=True)
        if self.prefix:
            out = self.fia.fia_decode_shared_prefix(q, self.kc, self.vc, shared_prefix_len=self.prefix, **kw)
        else:
            out = self.fia.fia_decode_window(q, self.kc, self.vc, pre_tokens=self.pre, sink_tokens=self.sink, **kw)
        self.ctx.copy_(kv)
        return out

    def prefill(self, new, x):
        kv, cu = self.append(new, x)
        q = x[:, :self.n1].contiguous()
        out = self.fia.fia_prefill_window(q, self.kc, self.vc, block_table=self.table, block_size=self.bs, actual_seq_qlen=cu,
                                          actual_seq_kvlen=kv, num_heads=self.n1, num_key_value_heads=self.n2,
                                          scale_value=self.scale, input_layout="TND", pre_tokens=self.pre,
                                          sink_tokens=self.sink, softmax_lse_flag=True)
        self.ctx.copy_(kv)
        return out

    def expect(self, lens, x):
        """Adds the step's tokens to the history; the oracle's rows for them: a list by sequence of attend()'s."""
        x, at, refs = f64(x), 0, []
        for b, n in enumerate(lens):
            rows = x[at:at + n]
            at += n
            self.keys[b] = np.concatenate([self.keys[b], rows[:, self.n1:self.n1 + self.n2]])
            self.vals[b] = np.concatenate([self.vals[b], rows[:, self.n1 + self.n2:]])
            L = len(self.keys[b])
            pre, sink = (1 << 40, 0) if self.prefix else (self.pre, self.sink)
            refs.append(po.attend(rows[:, :self.n1], self.keys[b], self.vals[b], po.window_see(n, L, pre, sink), self.scale))
        return refs


def check_decode(out, refs, Q):
    o, l = out
    for b, ref in enumerate(refs):
        po.assert_close(o[b], l[b, :, :, 0].T, ref, f"sequence {b}")


@pytest.mark.parametrize("layout", ["BNBD", "BSH"])
def test_prefill_chunks_then_decode(fia, layout):
    """Prompts in two ragged chunks, then decode steps of one and of three tokens, through one cache."""
    B, n1, n2, D = 4, 8, 2, 64
    s = Server(fia, B, n1, n2, D, 128, 60, 12, pre=150, sink=4, layout=layout)
    for step, lens in enumerate(([200, 1, 70, 333], [40, 290, 0, 5])):
        T = sum(lens)
        x = s.new_tokens(lens, T, seed=step)
        o, l = s.prefill(i32(lens), x.to(DEV))
        at = 0
        for b, ref in enumerate(s.expect(lens, x)):
            po.assert_close(o[at:at + lens[b]], l[at:at + lens[b], :, 0], ref, f"chunk {step}, sequence {b}")
            at += lens[b]
    for step, Q in enumerate((1, 3, 1, 1, 3)):
        x = s.new_tokens(None, B * Q, seed=50 + step)
        out = s.decode(i32([Q] * B), x.to(DEV), Q)
        check_decode(out, s.expect([Q] * B, x), Q)


def test_shared_prefix_decode_steps(fia):
    """A batch drawing answers from one prompt."""
    B, Q = 6, 1
    s = Server(fia, B, 8, 2, 128, 64, 60, 16, pre=0, sink=0, prefix=320)
    for step in range(70):   # past a page boundary of every sequence
        x = s.new_tokens(None, B * Q, seed=step)
        out = s.decode(i32([Q] * B), x.to(DEV), Q)
        refs = s.expect([Q] * B, x)
        if step in (0, 1, 63, 64, 69):
            check_decode(out, refs, Q)


@pytest.mark.parametrize("prefix", [0, 256])
def test_captured_step_replays_with_new_lengths(fia, prefix):
    """One decode step in a graph, replayed: lengths, tables and slots follow on the device."""
    B, Q = 5, 2
    s = Server(fia, B, 8, 2, 64, 32, 90, 24, pre=60, sink=3, prefix=prefix)
    x = torch.empty(B * Q, s.n1 + 2 * s.n2, s.D, dtype=torch.bfloat16, device=DEV)
    new = i32([Q] * B)
    first = s.new_tokens(None, B * Q, seed=1)
    x.copy_(first)
    check_decode(s.decode(new, x, Q), s.expect([Q] * B, first), Q)     # eager, also loads the kernels
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = s.decode(new, x, Q)
    for step in range(40):
        tok = s.new_tokens(None, B * Q, seed=100 + step)
        x.copy_(tok)
        graph.replay()
        refs = s.expect([Q] * B, tok)
        if step % 13 == 0 or step == 39:
            torch.cuda.synchronize()
            check_decode(out, refs, Q)


def test_padded_batch_in_a_captured_step(fia):
    """Sequences that leave: new length 0, their slots -1, their rows 0 and +inf, the others as ever."""
    B, Q = 4, 1
    s = Server(fia, B, 4, 2, 64, 16, 60, 20, pre=40, sink=2)
    x = s.new_tokens(None, B, seed=3)
    s.decode(i32([1] * B), x.to(DEV), Q)
    s.expect([1] * B, x)
    # a batch of two live sequences, padded to four: tokens of the live ones first
    lens = [1, 1, 0, 0]
    y = s.new_tokens(None, B, seed=4)
    yd = y.to(DEV)
    kv, _ = s.append(i32(lens), yd)
    kv[2:] = 0
    q = yd[:, :s.n1].reshape(B, 1, s.n1, s.D).contiguous()
    out = s.fia.fia_decode_window(q, s.kc, s.vc, block_table=s.table, block_size=16, actual_seq_kvlen=kv, num_heads=4,
                                  num_key_value_heads=2, scale_value=s.scale, input_layout="BSND", pre_tokens=40, sink_tokens=2,
                                  softmax_lse_flag=True)
    refs = s.expect(lens, y[:2])
    for b in range(2):
        po.assert_close(out[0][b], out[1][b, :, :, 0].T, refs[b])
    assert (out[0][2:] == 0).all() and torch.isposinf(out[1][2:]).all()


# ------------------------------------------------------------------ streams, overlap, timeouts
def _prefix_case(seed, B=12):
    g = torch.Generator().manual_seed(seed)
    P, bs, n2, D = 512, 64, 2, 128
    own = [1 + (i * 31) % 180 for i in range(B)]
    pages = [-(-n // bs) for n in own]
    pool = P // bs + sum(pages)
    k, v = (torch.randn(pool, n2, bs, D, generator=g).bfloat16().to(DEV) for _ in range(2))
    q = torch.randn(B, 8, 1, D, generator=g).bfloat16().to(DEV)
    table = torch.zeros(B, P // bs + max(pages), dtype=torch.int32)
    table[:, :P // bs] = torch.arange(P // bs)
    at = P // bs
    for b, n in enumerate(pages):
        table[b, P // bs:P // bs + n] = torch.arange(at, at + n)
        at += n
    return q, k, v, dict(block_table=table.to(DEV), block_size=bs, actual_seq_kvlen=i32([P + n for n in own]), num_heads=8,
                         num_key_value_heads=n2, scale_value=D ** -0.5, input_layout="BNSD", softmax_lse_flag=True)


def test_calls_on_two_streams_at_once(fia):
    """Every attention call on two streams, many in flight: the same bits as alone (each has its workspace)."""
    cases = [_prefix_case(i) for i in range(2)]

    def calls(c):
        q, k, v, kw = c
        return [fia.fia_decode_shared_prefix(q, k, v, shared_prefix_len=512, **kw)[0],
                fia.fia_decode_window(q, k, v, pre_tokens=90, sink_tokens=4, **kw)[0],
                fia.fia_prefill_window(q.reshape(1, 8, -1, 128).contiguous(), k.reshape(1, 2, -1, 128), v.reshape(1, 2, -1, 128),
                                       num_heads=8, num_key_value_heads=2, input_layout="BNSD", pre_tokens=100, sink_tokens=1)[0]]

    alone = [calls(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(10):
        got = []
        for c, st in zip(cases, streams):
            with torch.cuda.stream(st):
                got.append(calls(c))
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_back_to_back_calls_see_each_others_writes(fia):
    """A cache rewritten between calls, with nothing waiting in between: every call sees the newest rows."""
    q, k, v, kw = _prefix_case(5)
    n = k.shape[0] * 64
    rows = [torch.randn(n, 2, 128, device=DEV).bfloat16() for _ in range(4)]
    slots = torch.arange(n, dtype=torch.int32, device=DEV)
    want = []
    for r in rows:
        fia.fia_cache_write(r, r, k, v, slots)
        torch.cuda.synchronize()
        want.append((fia.fia_decode_window(q, k, v, pre_tokens=300, **kw)[0],
                     fia.fia_decode_shared_prefix(q, k, v, shared_prefix_len=512, **kw)[0]))
        torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for r in rows:
            fia.fia_cache_write(r, r, k, v, slots)
            got.append((fia.fia_decode_window(q, k, v, pre_tokens=300, **kw)[0],
                        fia.fia_decode_shared_prefix(q, k, v, shared_prefix_len=512, **kw)[0]))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("op", ["prefill", "prefix"])
def test_timeout_path(fia, op):
    """Waits that give up under a 1 ns limit report FIA_ERR_TIMEOUT; the next call on the workspace is correct."""
    from attention_fia_prefill_gb300 import _binding as B
    lib = B.load_library()
    ws = torch.zeros(16 << 20, dtype=torch.uint8, device=DEV)
    q, k, v, kw = _prefix_case(7)

    def call():
        if op == "prefix":
            return fia.fia_decode_shared_prefix(q, k, v, shared_prefix_len=512, workspace=ws, **kw)[0]
        x = [fia_inputs.normal((1, n, 3000, 128), "bf16", 120, i).to(DEV) for i, n in ((1, 4), (2, 2), (3, 2))]
        return fia.fia_prefill_window(*x, num_heads=4, num_key_value_heads=2, input_layout="BNSD", pre_tokens=700,
                                      sink_tokens=9, workspace=ws)[0]

    good = call()
    assert fia.fia_device_status(ws) == 0
    lib.fia_debug_set_wait_limit_ns(1)
    try:
        call()
        status = fia.fia_device_status(ws)
    finally:
        lib.fia_debug_set_wait_limit_ns(0)
    assert status in (0, 10)     # a wait whose first try succeeds does not look at the limit
    again = call()
    assert fia.fia_device_status(ws) == 0 and torch.equal(good, again)


# ------------------------------------------------------------------ caches past 2^31 elements
def test_cache_past_32_bit_offsets(fia):
    """A pool of 2.6e9 elements (5.2 GB) each for keys and values: rows in its last blocks are written and attended to."""
    nblk, n2, bs, D, n1, B = 20000, 8, 128, 128, 16, 3
    kc, vc = (torch.empty(nblk, n2, bs, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    lens = [300, 129, 700]
    T = sum(lens)
    x = torch.randn(T, n1 + 2 * n2, D, generator=torch.Generator().manual_seed(9)).bfloat16()
    xd = x.to(DEV)
    free = torch.arange(nblk - 1, nblk - 41, -1, dtype=torch.int32, device=DEV)
    table = torch.zeros(B, 8, dtype=torch.int32, device=DEV)
    slots, kv, cu, _ = fia.fia_block_table_append(i32([0] * B), i32(lens), free, table, block_size=bs, num_tokens=T)
    assert int(slots.max()) >= (nblk - 1) * bs and int(table.max()) == nblk - 1
    k, v = xd[:, n1:n1 + n2], xd[:, n1 + n2:]
    fia.fia_cache_write(k, v, kc, vc, slots)
    f = f64(x)
    at, rows, ends = 0, [], []
    for n in lens:
        rows.append((f[at:at + n, n1:n1 + n2], f[at:at + n, n1 + n2:]))
        at += n
        ends.append(at - 1)
    kw = dict(block_table=table, block_size=bs, actual_seq_kvlen=kv, num_heads=n1, num_key_value_heads=n2, scale_value=0.09,
              softmax_lse_flag=True)
    q = xd[ends][:, :n1].reshape(B, n1, 1, D).contiguous()
    out, lse = fia.fia_decode_window(q, kc, vc, input_layout="BNSD", pre_tokens=200, sink_tokens=3, **kw)
    po.assert_close(out, lse, po.decode(q.cpu(), rows, lens, 200, 3, 0.09), "decode")
    out, lse = fia.fia_prefill_window(xd[:, :n1].contiguous(), kc, vc, input_layout="TND", actual_seq_qlen=cu, pre_tokens=200,
                                      sink_tokens=3, **kw)
    at = 0
    for b, n in enumerate(lens):
        ref = po.attend(f[at:at + n, :n1], *rows[b], po.window_see(n, n, 200, 3), 0.09)
        po.assert_close(out[at:at + n], lse[at:at + n, :, 0], ref, f"prefill {b}")
        at += n
    # the last sequence's first block as everybody's prefix
    shared = table.clone()
    shared[:, 0] = table[2, 0]
    kw["block_table"] = shared
    rows = [tuple(np.concatenate([rows[2][i][:bs], r[i][bs:]]) for i in (0, 1)) for r in rows]
    out, lse = fia.fia_decode_shared_prefix(q, kc, vc, input_layout="BNSD", shared_prefix_len=bs, **kw)
    po.assert_close(out, lse, po.decode(q.cpu(), rows, lens, 1 << 40, 0, 0.09), "prefix")


def test_no_keys_at_all(fia):
    """Contiguous keys of no rows, an empty pool, lengths of zero: zeros and +inf."""
    q = torch.randn(2, 4, 1, 64, device=DEV).bfloat16()
    k = torch.zeros(2, 2, 0, 64, dtype=torch.bfloat16, device=DEV)
    kw = dict(num_heads=4, num_key_value_heads=2, input_layout="BNSD", softmax_lse_flag=True)
    pool = torch.zeros(0, 2, 16, 64, dtype=torch.bfloat16, device=DEV)
    paged = dict(block_table=torch.zeros(2, 3, dtype=torch.int32, device=DEV), block_size=16, **kw)
    for out, lse in (fia.fia_decode_window(q, k, k, **kw), fia.fia_decode_window(q, pool, pool, actual_seq_kvlen=i32([20, 0]), **paged),
                     fia.fia_decode_shared_prefix(q, pool, pool, shared_prefix_len=16, actual_seq_kvlen=i32([20, 40]), **paged)):
        if lse is not None:
            assert torch.isfinite(out).all()
    out, lse = fia.fia_decode_window(q, k, k, **kw)
    assert (out == 0).all() and torch.isposinf(lse).all()
