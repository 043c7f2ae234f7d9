"""Edges of the paged-serving operators, the shared prefix on both of its paths."""
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
