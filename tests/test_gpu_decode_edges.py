"""Edges of the receiver's decode calls on the GPU: places that do not exist, infinities and NaN
among keys and values, biases of the type's size, angles near a quarter turn.

The plain 64-bit evaluations and the tolerances derived beside them are those of
test_gpu_decode.
"""
import numpy as np
import pytest
import torch

from cross_model_attention_block_b200 import mapflow as mfb
from tests.test_gpu_decode import BF, F32, i32, near_rotated, pages, randn, slots

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("given", [False, True], ids=["new", "given"])
def test_queries_of_tokens_without_a_place_are_rotated(dt, given):
    """Pages outside the pool, and places past the table: the token's keys and values are skipped
    and reported, its query is that of its position; a padding sequence's stays as it was."""
    new, past = [20, 5, 9, 3], [10, 30, -2, 0]
    table, npages = pages([48, 48, 48, 48], 16, 90)
    c = mfb.KVCache(randn((npages, 16, 2, 64), dt, 91), randn((npages, 16, 2, 64), dt, 92), table)
    table[0, 1] = -1                                  # tokens 16 .. 29 of sequence 0
    table[1, 1:] = npages                             # 30, 31 and 32 .. 34 of sequence 1
    K0, V0 = c.K.clone(), c.V.clone()
    f, n = mfb.rope_freqs(64), sum(new)
    cu = i32(np.concatenate([[0], np.cumsum(new)]))
    x = randn((n, 4 + 2 + 2, 64), dt, 93)
    Qo = torch.full((n, 4, 64), 9.0, dtype=dt, device="cuda") if given else None
    q = mfb.kv_append(c, x[:, 4:6], x[:, 6:], i32(past), rope=mfb.Rope.from_freqs(f), Q=x[:, :4],
                      Q_out=Qo, cu_seqlens=cu)
    with pytest.raises(mfb.MapflowError) as e:
        mfb.sync_status()
    assert e.value.status == mfb.MF_ERR_INVALID_ARG
    live = torch.tensor([t for t in range(n) if not 25 <= t < 34], device="cuda")
    pos = torch.cat([torch.arange(10, 30), torch.arange(30, 35), torch.arange(3)])
    near_rotated(q[live], x[live][:, :4], pos, f, 64, False)
    if given:
        assert (q[25:34] == 9.0).all()
    at = torch.cat([slots(table, 16, 0, 10, 16), slots(table, 16, 3, 0, 3)])
    tok = torch.cat([torch.arange(6), torch.arange(34, 37)]).cuda()
    kf, vf = c.K.view(-1, 2, 64), c.V.view(-1, 2, 64)
    near_rotated(kf[at], x[tok][:, 4:6], torch.cat([torch.arange(10, 16), torch.arange(3)]), f, 64,
                 False)
    assert torch.equal(vf[at], x[tok][:, 6:])
    keep = torch.ones(npages * 16, dtype=torch.bool, device="cuda")
    keep[at] = False
    assert torch.equal(kf[keep], K0.view(-1, 2, 64)[keep])
    assert torch.equal(vf[keep], V0.view(-1, 2, 64)[keep])


def test_one_token_each_past_the_table():
    """Single tokens without cu_seqlens, one of them behind its table's last page."""
    table, npages = pages([32, 32], 16, 94)
    c = mfb.KVCache(randn((npages, 16, 1, 128), BF, 95), randn((npages, 16, 1, 128), BF, 96), table)
    Q, K = randn((2, 3, 128), BF, 97), randn((2, 1, 128), BF, 98)
    f = mfb.rope_freqs(128)
    q = mfb.kv_append(c, K, K, i32([32, 31]), rope=mfb.Rope.from_freqs(f), Q=Q)
    with pytest.raises(mfb.MapflowError):
        mfb.sync_status()
    near_rotated(q, Q, torch.tensor([32, 31]), f, 128, False)
