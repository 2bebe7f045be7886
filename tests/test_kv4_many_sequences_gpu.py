"""Appends for more than 2^30 sequences, nearly all of them without new tokens: a token's sequence is found by bisection."""
import pytest
import torch

from output_centric_expert_gb300 import block_ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("turned", [False, True])
def test_more_than_2_30_sequences(turned):
    S, heads, dim = 2 ** 30 + 1000, 2, 64
    whose = [3, 2 ** 29 + 5, 2 ** 30 - 1, 2 ** 30 + 1, S - 1]  # the sequences with a new token
    cache = block_ops.Kv4Cache(len(whose), 16, heads, dim)
    table, lens = (torch.zeros(S, dtype=torch.int32, device="cuda") for _ in range(2))
    cu = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
    for i, s in enumerate(whose):
        cu[s + 1:] += 1
        table[s], lens[s] = i, i + 2
    table = table[:, None]
    q, k, v = (torch.randn(len(whose), heads, dim, device="cuda").to(torch.bfloat16) for _ in range(3))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    rope = block_ops.Rope(torch.zeros(16, dtype=torch.float64))
    if turned:
        block_ops.wd_kv4_rope_append(cache, rope, q.clone(), k, v, table, lens, cu_new=cu, err_flag=err)
    else:
        block_ops.wd_kv4_append(cache, k, v, table, lens, cu, err)
    assert int(err) == 0
    # the same tokens as five sequences of their own
    alone = block_ops.Kv4Cache(len(whose), 16, heads, dim)
    few = torch.arange(len(whose), dtype=torch.int32, device="cuda")
    block_ops.wd_kv4_append(alone, k, v, few[:, None].contiguous(), few + 2)
    assert all(torch.equal(a, b) for a, b in zip(cache.tensors, alone.tensors))
    got = [torch.empty(k.shape, device="cuda") for _ in range(4)]
    block_ops.wd_kv4_gather(cache, table, lens, got[0], got[1], cu, err)
    block_ops.wd_kv4_gather(alone, few[:, None].contiguous(), few + 2, got[2], got[3])
    assert int(err) == 0 and torch.equal(got[0], got[2]) and torch.equal(got[1], got[3])
