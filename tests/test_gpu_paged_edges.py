"""Edges of the paged-serving operators, the shared prefix on both of its paths."""
import math

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


@pytest.fixture(params=[1, 2], ids=["apart", "every"])
def path(request):
    """The prefix by a kernel of its own, and by every sequence's."""
    lib = _binding.load_library()
    lib.fia_debug_set_prefix_path(request.param)
    yield request.param
    lib.fia_debug_set_prefix_path(0)


def batch(n1, n2, B, P, own, Q=1, bs=64, D=128, workload=160):
    """Query, pools, tables of a batch behind a prefix of P keys, with room for `own` keys of its own each."""
    pages, mine = P // bs, own // bs
    q = fia_inputs.normal((B, n1, Q, D), "bf16", workload, 1)
    k, v = (fia_inputs.normal((pages + B * mine, n2, bs, D), "bf16", workload, i) for i in (2, 3))
    table = torch.cat([torch.arange(pages).expand(B, pages), pages + torch.arange(B * mine).view(B, mine)], 1).int().contiguous()
    return q, k, v, table


def run(fia, q, k, v, table, lens, P, n2, scale=0.09):
    out, lse = fia.fia_decode_shared_prefix(q.to(DEV), k.to(DEV), v.to(DEV), block_table=table.to(DEV), block_size=k.shape[2],
                                            actual_seq_kvlen=i32(lens), shared_prefix_len=P, num_heads=q.shape[1],
                                            num_key_value_heads=n2, scale_value=scale, input_layout="BNSD", softmax_lse_flag=True)
    torch.cuda.synchronize()
    return out, lse


# ------------------------------------------------------------------ lengths past the tables
@pytest.mark.parametrize("Q", [1, 2, 16])
@pytest.mark.parametrize("n1,n2", [(4, 2), (4, 1)])
def test_prefix_lengths_past_the_tables(fia, path, Q, n1, n2):
    """Lengths are taken to the keys the tables have room for, the prefix being all of them: every token sees the cache up
    to itself."""
    P = 256
    lens = [P, P + 1, P + 5, P - 1, 2 ** 31 - 1, 3, P + Q]
    q, k, v, table = batch(n1, n2, len(lens), P, 0, Q=Q, workload=161)
    taken = [min(n, P) for n in lens]
    out, lse = run(fia, q, k, v, table, lens, P, n2)
    rows = [tuple(po.cache_rows(f64(x), table[b], n, n2) for x in (k, v)) for b, n in enumerate(taken)]
    po.assert_close(out, lse, po.decode(q, rows, taken, 1 << 40, 0, 0.09))


# ------------------------------------------------------------------ NaN scores
@pytest.mark.parametrize("n1", [4, 20, 64])
def test_nan_query_behind_a_prefix(fia, path, n1):
    """A query that is NaN gives NaN, also where the sequence has no key but the prefix's; its neighbours are as ever."""
    P, lens = 512, [512, 300, 700, 520, 0]
    q, k, v, table = batch(n1, 1, len(lens), P, 256, workload=162 + n1)
    want, want_l = run(fia, q, k, v, table, lens, P, 1)
    q[:3, 1] = float("nan")
    q[4, 1] = float("nan")     # (no keys: zeros and +inf whatever the query)
    out, lse = run(fia, q, k, v, table, lens, P, 1)
    assert out[:3, 1].isnan().all() and lse[:3, 1].isnan().all()
    others = [h for h in range(n1) if h != 1]
    assert torch.equal(out[:, others], want[:, others]) and torch.equal(lse[:, others], want_l[:, others])
    assert torch.equal(out[3:], want[3:]) and torch.equal(lse[3:], want_l[3:])


@pytest.mark.parametrize("n1", [4, 64])
@pytest.mark.parametrize("tiles", [range(8), [0], [7], [2, 3]])
def test_nan_keys_of_a_prefix(fia, path, n1, tiles):
    """Keys of the prefix that are NaN, whole 128-key tiles of it: NaN for every sequence that sees one."""
    P, lens = 1024, [1024, 1100, 1279, 1025]
    q, k, v, table = batch(n1, 1, len(lens), P, 256, bs=128, workload=164 + n1)
    k[list(tiles)] = float("nan")
    out, lse = run(fia, q, k, v, table, lens, P, 1)
    assert out.isnan().all() and lse.isnan().all()


# ------------------------------------------------------------------ block ids outside the pool
@pytest.mark.parametrize("n1", [4, 40])
def test_ids_outside_the_pool_read_as_zeros(fia, path, n1):
    """Negative ids and ids past the pool, in the prefix and behind it: what a block of zeros gives."""
    P, lens = 512, [512, 640, 700, 515]
    q, k, v, table = batch(n1, 1, len(lens), P, 256, workload=166 + n1)
    n = k.shape[0]
    k, v = (torch.cat([x, torch.zeros(1, *x.shape[1:], dtype=x.dtype)]) for x in (k, v))
    table[:, 2] = table[1, 9] = table[2, 8] = n
    want = run(fia, q, k, v, table, lens, P, 1)
    table[:, 2], table[1, 9], table[2, 8] = -1, 2 ** 31 - 1, -2 ** 31
    got = run(fia, q, k[:n], v[:n], table, lens, P, 1)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("kv", ["BNBD", "BSH"])
def test_prefill_ids_outside_the_pool_read_as_zeros(fia, kv):
    q = fia_inputs.normal((2, 4, 150, 64), "bf16", 167, 1).to(DEV)
    shape = (5, 2, 128, 64) if kv == "BNBD" else (5, 128, 128)
    k, v = (fia_inputs.normal(shape, "bf16", 167, i).to(DEV) for i in (2, 3))
    k[4] = v[4] = 0
    kw = dict(block_size=128, actual_seq_kvlen=i32([500, 300]), num_heads=4, num_key_value_heads=2, input_layout="BNSD",
              softmax_lse_flag=True, pre_tokens=200, sink_tokens=5)
    want = fia.fia_prefill_window(q, k, v, block_table=i32([[0, 4, 2, 4], [4, 1, 3, 0]]), **kw)
    got = fia.fia_prefill_window(q, k[:4], v[:4], block_table=i32([[0, -1, 2, 2 ** 31 - 1], [-2 ** 31, 1, 3, 0]]), **kw)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


# ------------------------------------------------------------------ pools without a block
@pytest.mark.parametrize("n1", [4, 40])
@pytest.mark.parametrize("P", [0, 64])
def test_prefix_empty_pool_reads_as_zeros(fia, path, n1, P):
    """As fia_decode_window: every key and value of a length is 0, so out = 0 and lse = log(keys seen)."""
    lens = [100, 0, 64, 1, 10 ** 6]
    q, _, _, _ = batch(n1, 1, len(lens), 0, 0, Q=1, workload=168)
    pool = torch.zeros(0, 1, 32, 128, dtype=torch.bfloat16)
    table = torch.zeros(len(lens), 4, dtype=torch.int32)
    out, lse = run(fia, q, pool, pool, table, lens, P, 1)
    o2, l2 = fia.fia_decode_window(q.to(DEV), pool.to(DEV), pool.to(DEV), block_table=table.to(DEV), block_size=32,
                                   actual_seq_kvlen=i32(lens), num_heads=n1, num_key_value_heads=1, scale_value=0.09,
                                   input_layout="BNSD", softmax_lse_flag=True)
    seen = torch.tensor([math.log(n) if n else math.inf for n in (100, 0, 64, 1, 128)]).view(-1, 1, 1, 1)
    for o, l in ((out, lse), (o2, l2)):
        assert (o == 0).all() and torch.isposinf(l[1]).all()
        live = [0, 2, 3, 4]
        # log2 of a sum of at most 128 ones and its product with ln 2, in fp32: 1e-5 is over ten steps of either
        assert (l.cpu()[live] - seen[live]).abs().max() < 1e-5


@pytest.mark.parametrize("kv", ["BNBD", "BSH"])
def test_prefill_empty_pool_reads_as_zeros(fia, kv):
    """Rows that see keys give 0 and log(keys seen), rows that see none 0 and +inf."""
    q = fia_inputs.normal((3, 2, 300, 64), "bf16", 169, 1).to(DEV)
    pool = torch.zeros((0, 1, 128, 64) if kv == "BNBD" else (0, 128, 64), dtype=torch.bfloat16, device=DEV)
    lens, pre, sink = [300, 500, 0], 99, 3
    out, lse = fia.fia_prefill_window(q, pool, pool, block_table=torch.zeros(3, 4, dtype=torch.int32, device=DEV), block_size=128,
                                      actual_seq_kvlen=i32(lens), num_heads=2, num_key_value_heads=1, input_layout="BNSD",
                                      softmax_lse_flag=True, pre_tokens=pre, sink_tokens=sink)
    assert (out == 0).all() and torch.isposinf(lse[2]).all()
    for b in (0, 1):
        n = po.window_see(300, lens[b], pre, sink).sum(1)
        assert np.abs(lse[b, :, :, 0].cpu().double().numpy() - np.log(n)).max() < 1e-5


# ------------------------------------------------------------------ the free list from step to step
def test_no_block_is_handed_out_twice(fia):
    """Steps that take the free list on by what the step before asked for: every block has one owner."""
    B, bs, r = 6, 16, np.random.default_rng(7)
    free = torch.from_numpy(r.permutation(200).astype(np.int32)).to(DEV)
    table = torch.full((B, 30), -1, dtype=torch.int32, device=DEV)
    ctx, held = i32([0] * B), 0
    for _ in range(12):
        new = [int(x) for x in r.integers(0, 40, B)]
        slots, kv, _, used = fia.fia_block_table_append(ctx, i32(new), free, table, block_size=bs, num_tokens=sum(new))
        free = free[int(used):]
        ctx.copy_(kv)
        held += int(used)
        owned = table[table >= 0]
        assert len(owned) == held == sum(-(-n // bs) for n in ctx.tolist()) and len(set(owned.tolist())) == held
        assert len(set(slots.tolist())) == sum(new) and int(slots.min()) >= 0
