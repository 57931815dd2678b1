"""The single-token attention's division of work, its marshalling, and the rotation's launch
shapes on the GPU, where they can go wrong: rows cut between warps and blocks at every kind of
place, short tables, many sequences, logits that climb, captured calls whose lengths change.

The plain 64-bit evaluations and the tolerances derived beside them are those of
test_gpu_decode.
"""
import math

import numpy as np
import pytest
import torch

from cross_model_attention_block_b200 import mapflow as mfb
from tests.test_gpu_decode import (BF, F32, attend64, check_attention, filled_cache, i32,
                                   near_rotated, pages, randn, slots)

pytestmark = pytest.mark.gpu


def widened(c, width):
    """The same cache behind a table with room for `width` pages a sequence."""
    t = torch.full((c.nseq, width), -1, dtype=torch.int32, device="cuda")
    t[:, :c.max_pages] = c.page_table
    return mfb.KVCache(c.K, c.V, t)


def mixed(seed, n, hi):
    """Lengths: most short, some long, some empty."""
    r = np.random.default_rng(seed)
    x = np.exp(r.uniform(0, math.log(hi), n)).astype(int)
    x[r.random(n) < 0.1] = 0
    return x.tolist()


# ------------------------------------------------------------------ cuts

# head groups of every kernel variant: 1..4, 5..8 and 9..16 heads a group, and groups of groups
LAYOUTS = [(BF, 8, 8, 128), (BF, 12, 4, 64), (BF, 14, 2, 128), (BF, 16, 2, 64), (BF, 22, 2, 128),
           (BF, 16, 1, 64), (BF, 17, 1, 128), (BF, 64, 2, 64), (F32, 6, 6, 64), (F32, 8, 2, 128),
           (F32, 7, 1, 64), (F32, 16, 2, 128), (F32, 13, 1, 64), (F32, 33, 1, 128)]


@pytest.mark.parametrize("dt,Hq,Hkv,d", LAYOUTS)
@pytest.mark.parametrize("lengths", [mixed(1, 40, 3000), mixed(2, 300, 40), [9000, 1, 0, 16, 4097]],
                         ids=["spread", "many_short", "few_long"])
def test_rows_cut_anywhere(dt, Hq, Hkv, d, lengths):
    """Whole rows, rows over several warps, over several blocks; behind a table just wide enough
    and behind a wide one (another division of the work)."""
    c = filled_cache(lengths, 16, Hkv, d, dt, 50)
    Q = randn((len(lengths), Hq, d), dt, 51)
    for k in (c, widened(c, c.max_pages + 700)):
        O, lse = mfb.paged_attn(k, Q, i32(lengths))
        mfb.sync_status()
        check_attention(c, lengths, Q, O, lse, d ** -0.5)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("total", [1, 2, 31, 147, 148, 149, 295, 297, 1183, 1185])
def test_totals_around_the_numbers_of_blocks_and_warps(dt, total):
    """One long row, and two, of about as many 16-key units as there are blocks or warps."""
    for lengths in ([16 * total], [16 * total - 5, 16 * (total // 2) + 3]):
        c = filled_cache(lengths, 16, 1, 64, dt, 52)
        c = widened(c, c.max_pages + 40)
        Q = randn((len(lengths), 3, 64), dt, 53)
        O, lse = mfb.paged_attn(c, Q, i32(lengths))
        mfb.sync_status()
        check_attention(c, lengths, Q, O, lse, 64 ** -0.5)


@pytest.mark.parametrize("dt,Hq,Hkv,d,rows", [(BF, 16, 8, 64, 4), (BF, 64, 2, 128, 4),
                                              (F32, 33, 1, 128, 5), (F32, 8, 8, 64, 8)])
@pytest.mark.parametrize("few", [False, True], ids=["spread", "few_long"])
def test_lines_long_enough_for_more_blocks(dt, Hq, Hkv, d, rows, few):
    """Calls of 148 * 800 sixteens of keys (a row counts two besides) and more are cut for more
    blocks than fill the GPU; one sixteen fewer, and short ones behind the same table, are not."""
    need = 148 * 800 // rows  # sixteens and twos that each of a sequence's rows has to bring
    rest = [16 * (need - 3) // 2 - 16, 16 * (need + 1) // 4] if few else mixed(7, 150, 4000)
    used = sum((n + 15) // 16 + 2 for n in rest if n > 0)
    lengths = rest + [16 * (need - used - 2)]
    c = filled_cache(lengths, 16, Hkv, d, dt, 60)
    Q = randn((len(lengths), Hq, d), dt, 61)
    for last in (lengths[-1], lengths[-1] - 16, 5):
        lengths[-1] = last
        O, lse = mfb.paged_attn(c, Q, i32(lengths))
        mfb.sync_status()
        check_attention(c, lengths, Q, O, lse, d ** -0.5)
    lengths = [min(n, 40) for n in lengths]
    O, lse = mfb.paged_attn(c, Q, i32(lengths))
    mfb.sync_status()
    check_attention(c, lengths, Q, O, lse, d ** -0.5)


@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (8, 8), (8, 2), (16, 4), (20, 4), (32, 4), (36, 4),
                                    (9, 3), (15, 3), (48, 3)])
def test_heads_of_64_dims(Hq, Hkv):
    """Even and odd numbers of KV heads of 128 bytes a key, up to 16 query heads for two of them
    and more, narrow tables and wide ones (two KV heads at a time); NaN and infinities among the
    keys and values of one head stay in its own outputs."""
    lengths = [700, 1, 0, 16, 333, 2048, 47]
    c = filled_cache(lengths, 32, Hkv, 64, BF, 62)
    Q = randn((len(lengths), Hq, 64), BF, 63)
    for table in (c.page_table, widened(c, 900).page_table):
        O, lse = mfb.paged_attn(mfb.KVCache(c.K, c.V, table), Q, i32(lengths), window=500,
                                band_bias=-0.75, band_width=18)
        mfb.sync_status()
        check_attention(c, lengths, Q, O, lse, 0.125, -0.75, 18, 500)
        G = Hq // Hkv
        for bad in range(Hkv):
            k = mfb.KVCache(c.K.clone(), c.V.clone(), table)
            kh, vh = k.K.view(-1, Hkv, 64)[:, bad], k.V.view(-1, Hkv, 64)[:, bad]
            kh[:, 3], kh[::5, 7], vh[:, 5], vh[::3, 11] = math.nan, math.inf, -math.inf, math.nan
            O2, lse2 = mfb.paged_attn(k, Q, i32(lengths), window=500, band_bias=-0.75,
                                      band_width=18)
            mfb.sync_status()
            for h in range(Hkv):
                hs = slice(h * G, (h + 1) * G)
                if h == bad:
                    live = [s for s, n in enumerate(lengths) if n > 0]
                    assert O2[live][:, hs].isnan().all() and lse2[hs][:, live].isnan().all()
                else:
                    assert torch.equal(O2[:, hs], O[:, hs]) and torch.equal(lse2[hs], lse[hs])


@pytest.mark.parametrize("dt", [BF, F32])
def test_many_sequences(dt):
    """More sequences than a block has threads, empty ones among them, windows inside."""
    r = np.random.default_rng(3)
    lengths = r.integers(0, 60, 1500).tolist()
    for window in (0, 21):
        c = filled_cache(lengths, 16, 2, 64, dt, 54, window=window)
        Q = randn((len(lengths), 4, 64), dt, 55)
        O, lse = mfb.paged_attn(c, Q, i32(lengths), window=window, band_bias=1.5, band_width=9)
        mfb.sync_status()
        some = list(range(0, 1500, 37)) + [1499]
        for s in some:
            L = lengths[s]
            if L == 0:
                assert (O[s] == 0).all() and (lse[:, s] == -math.inf).all()
                continue
            at = slots(c.page_table, 16, s, 0, L)
            for h in range(2):
                K = c.K.view(-1, 2, 64)[at, h].double()
                V = c.V.view(-1, 2, 64)[at, h].double()
                if window:
                    K[:max(0, L - window)], V[:max(0, L - window)] = 0.0, 0.0
                o, e, tol, delta = attend64(Q[s, 2 * h:2 * h + 2].double(), K, V, 0.125, 1.5, 9,
                                            window)
                got = O[s, 2 * h:2 * h + 2].double()
                assert ((got - o).abs() <= tol + torch.finfo(dt).eps / 2 * o.abs()).all()
                err = (lse[2 * h:2 * h + 2, s].double() - e).abs()
                assert (err <= delta + 2.0 ** -22 * e.abs()).all()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("order", ["climbing", "falling", "steps"])
def test_logits_that_climb_and_fall(dt, order):
    """Logits that rise by more than the reference's slack again and again, fall, or jump: the
    sums are rescaled in the middle of a row, and pieces of very different size meet."""
    L, d, Hkv, G = 2500, 64, 2, 5
    c = filled_cache([L, 40], 16, Hkv, d, dt, 56)
    at = slots(c.page_table, 16, 0, 0, L)
    ramp = torch.linspace(0.0, 60.0, L, device="cuda")
    size = {"climbing": ramp, "falling": ramp.flip(0), "steps": torch.floor(ramp / 15) * 15}[order]
    Q = randn((2, Hkv * G, d), dt, 57).abs() + 0.1
    Q[:, :, 1:] *= 0.1
    c.K.view(-1, Hkv, d)[at, :, 0] = size[:, None].to(dt)
    O, lse = mfb.paged_attn(c, Q, i32([L, 40]), scale=1.0)
    mfb.sync_status()
    check_attention(c, [L, 40], Q, O, lse, 1.0)


def test_a_group_of_256_heads():
    lengths = [70, 0, 333]
    c = filled_cache(lengths, 16, 1, 128, BF, 58)
    Q = randn((3, 256, 128), BF, 59)
    O, lse = mfb.paged_attn(c, Q, i32(lengths))
    mfb.sync_status()
    check_attention(c, lengths, Q, O, lse, 128 ** -0.5)


@pytest.mark.parametrize("dt", [BF, F32])
def test_bad_pages_in_long_rows(dt):
    """Every third page of a row outside the pool: its other keys alone take part."""
    L, ps = 3000, 48
    c = filled_cache([L, 50], ps, 1, 64, dt, 60)
    good = c.page_table.clone()
    c.page_table[0, ::3] = c.npages + 5
    Q = randn((2, 4, 64), dt, 61)
    O, lse = mfb.paged_attn(c, Q, i32([L, 50]))
    with pytest.raises(mfb.MapflowError):
        mfb.sync_status()
    j = torch.arange(L, device="cuda")
    kept = slots(good, ps, 0, 0, L)[(j // ps) % 3 != 0]
    o, e, tol, delta = attend64(Q[0].double(), c.K.view(-1, 64)[kept].double(),
                                c.V.view(-1, 64)[kept].double(), 0.125, 0.0, 0, 0)
    assert ((O[0].double() - o).abs() <= tol + torch.finfo(dt).eps / 2 * o.abs()).all()
    assert ((lse[:, 0].double() - e).abs() <= delta + 2.0 ** -22 * e.abs()).all()
    c.page_table.fill_(-1)                                   # nothing left
    O, lse = mfb.paged_attn(c, Q, i32([L, 50]))
    with pytest.raises(mfb.MapflowError):
        mfb.sync_status()
    assert (O == 0).all() and (lse == -math.inf).all()


# ------------------------------------------------------------------ captured calls

@pytest.mark.parametrize("dt", [BF, F32])
def test_captured_call_follows_its_lengths(dt):
    """One captured call, replayed with other lengths and queries: from empty to the whole
    table, the cuts at other places each time; the bits of a call made outside a graph."""
    full = [4000, 17, 900, 2500]
    c = filled_cache(full, 16, 2, 64, dt, 62)
    Q, lens = randn((4, 8, 64), dt, 63), i32([0, 0, 0, 0])
    ws = torch.empty(8 << 20, dtype=torch.uint8, device="cuda")
    O, lse = mfb.paged_attn(c, Q, lens, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mfb.paged_attn(c, Q, lens, O=O, lse=lse, workspace=ws)
    for k, now in enumerate(([0, 0, 0, 0], [1, 17, 0, 33], full, [4000, 0, 0, 0], [15, 16, 17, 2500])):
        lens.copy_(i32(now))
        Q.copy_(randn((4, 8, 64), dt, 64 + k))
        O.fill_(7.0)
        graph.replay()
        got, got_lse = O.clone(), lse.clone()
        want = mfb.paged_attn(c, Q, lens)
        assert torch.equal(got, want[0]) and torch.equal(got_lse, want[1])
        check_attention(c, now, Q, got, got_lse, 0.125)
    mfb.sync_status()


def test_append_and_attention_overlap_their_launches():
    """A chain of small calls, each of which may be launched before the one ahead has ended,
    with a torch kernel between them now and then: the results of the same calls with a
    synchronization after each."""
    def run(wait):
        table, n = pages([540, 44, 108], 16, 70)
        kv = mfb.KVCache(randn((n, 16, 2, 128), BF, 70), randn((n, 16, 2, 128), BF, 76), table)
        lens, rp = i32([496, 0, 64]), mfb.Rope.make(128)
        x = randn((3, 8 + 4, 128), BF, 71)
        outs = []
        for k in range(40):
            q = mfb.kv_append(kv, x[:, 8:10], x[:, 10:], lens, rope=rp, Q=x[:, :8])
            if wait:
                torch.cuda.synchronize()
            O, lse = mfb.paged_attn(kv, q, lens, len_add=1)
            if wait:
                torch.cuda.synchronize()
            if k % 3 == 0:
                x = x.roll(1, 0)
            x[:, :8] = O
            lens.add_(1)
            outs += [O, lse]
        mfb.sync_status()
        return outs
    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ marshalling

def test_outputs_given_are_the_outputs_returned():
    lengths = [100, 37]
    c = filled_cache(lengths, 16, 2, 64, F32, 72)
    Q, L = randn((2, 4, 64), F32, 73), i32(lengths)
    O, lse = mfb.paged_attn(c, Q, L)
    O2, lse2, ws = torch.empty_like(O), torch.empty_like(lse), torch.empty(64, dtype=torch.uint8,
                                                                          device="cuda")
    a, b = mfb.paged_attn(c, Q, L, O=O2, lse=lse2, workspace=ws)   # too small: one is made
    assert a is O2 and b is lse2 and torch.equal(a, O) and torch.equal(b, lse)
    assert mfb.paged_attn(c, Q, L, scale=1)[0].shape == O.shape    # a whole number as scale
    rp = mfb.Rope.make(64)
    q = mfb.rope(rp, Q, start=L)
    q2, k2 = torch.empty_like(Q), torch.empty_like(Q)
    a, b = mfb.rope(rp, Q, Q, start=L, Q_out=q2, K_out=k2)
    assert a is q2 and b is k2 and torch.equal(q2, q) and torch.equal(k2, q)
    assert mfb.kv_append(c, Q[:, :2], Q[:, 2:], i32([0, 0])) is None
    q3 = torch.empty_like(Q)
    assert mfb.kv_append(c, Q[:, :2], Q[:, 2:], i32([0, 0]), rope=rp, Q=Q, Q_out=q3) is q3
    assert torch.equal(q3, mfb.rope(rp, Q, start=i32([0, 0])))


def refused(f, *a, **kw):
    with pytest.raises((mfb.MapflowError, ValueError)) as e:
        f(*a, **kw)
    assert str(e.value)


def test_refusals_with_tensors_on_the_gpu():
    c = filled_cache([40, 40], 16, 2, 64, F32, 74)
    Q, L = randn((2, 4, 64), F32, 75), i32([40, 40])
    refused(mfb.paged_attn, c, Q, L.long())
    refused(mfb.paged_attn, c, Q, L.cpu())
    refused(mfb.paged_attn, c, Q.bfloat16(), L)
    refused(mfb.paged_attn, c, Q[:, :3], L)
    refused(mfb.paged_attn, c, Q.transpose(1, 2), L)
    refused(mfb.paged_attn, c, Q, L, window=-1)
    refused(mfb.paged_attn, c, Q, L, window=1 << 40)
    refused(mfb.paged_attn, c, Q, L, len_add=-(1 << 40))
    refused(mfb.paged_attn, c, Q, L, scale=float("nan"))
    refused(mfb.paged_attn, c, Q, L, lse=torch.empty(2, 4, device="cuda"))
    refused(mfb.paged_attn, c, Q, L, O=torch.empty(2, 4, 64))
    refused(mfb.paged_attn, c, Q, L, workspace=torch.empty(8 << 20, dtype=torch.int8,
                                                           device="cuda"))
    refused(mfb.paged_attn, c, torch.empty(2, 514, 64, device="cuda"), L)
    rp = mfb.Rope.make(64)
    refused(mfb.rope, rp, Q)
    refused(mfb.rope, rp, Q, start=L[:1])
    refused(mfb.rope, rp, Q, start=L.cpu())
    refused(mfb.rope, rp, Q, Q.bfloat16(), start=L)
    refused(mfb.rope, rp, Q, start=L, K_out=Q)
    refused(mfb.rope, mfb.Rope.make(128), Q, start=L)
    refused(mfb.kv_append, c, Q, Q, L)
    refused(mfb.kv_append, c, Q[:, :2], Q[:, :2].bfloat16(), L)
    refused(mfb.kv_append, c, Q[:, :2], Q[:, 2:], L[:1])
    refused(mfb.kv_append, c, Q[:, :2], Q[:, 2:], L, rope=mfb.Rope.make(128))
    refused(mfb.kv_append, c, Q[:, :2], Q[:, 2:], i32([0]), cu_seqlens=i32([0, 2]))
    mfb.sync_status()                                        # nothing was launched


# ------------------------------------------------------------------ rotation

@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("ntok,Hq,Hk,d,rot", [(1, 1, 0, 64, 64), (3, 1, 1, 64, 32),
                                              (5, 3, 2, 128, 128), (148, 2, 1, 64, 64),
                                              (297, 1, 1, 64, 48), (3551, 4, 4, 64, 64),
                                              (3552, 4, 4, 64, 64), (20000, 1, 1, 64, 16),
                                              (40001, 2, 2, 128, 128), (2, 300, 1, 128, 20)])
def test_rope_launch_shapes(dt, ntok, Hq, Hk, d, rot):
    """Tokens that share a block or have one each, heads that fill half a step or many; the
    last block with fewer tokens."""
    f = mfb.rope_freqs(rot)
    seqs = [ntok // 3, 0, ntok - ntok // 3]
    start = [11, 5, 70000]
    pos = torch.cat([torch.arange(s, s + m) for s, m in zip(start, seqs)])
    Q = randn((ntok, Hq, d), dt, 80)
    K = randn((ntok, Hk, d), dt, 81) if Hk else None
    for inter in (False, True):
        out = mfb.rope(mfb.Rope.from_freqs(f, inter), Q, K, start=i32(start),
                       cu_seqlens=i32(np.concatenate([[0], np.cumsum(seqs)])))
        for x, y in zip((Q, K), out if Hk else (out,)):
            near_rotated(y, x, pos, f, rot, inter)


def test_append_padding_sequences_between_prompts():
    """Packed prompts with padding sequences among them: their tokens' rows stay as they were."""
    new, past = [20, 7, 33, 5], [3, -1, 0, -4]
    table, npages = pages([23, 7, 33, 5], 16, 82)
    c = mfb.KVCache(randn((npages, 16, 2, 64), BF, 83), randn((npages, 16, 2, 64), BF, 84), table)
    K0 = c.K.clone()
    cu = i32(np.concatenate([[0], np.cumsum(new)]))
    x = randn((sum(new), 4 + 2 + 2, 64), BF, 85)
    f = mfb.rope_freqs(64)
    Qo = torch.full((sum(new), 4, 64), 9.0, dtype=BF, device="cuda")
    mfb.kv_append(c, x[:, 4:6], x[:, 6:], i32(past), rope=mfb.Rope.from_freqs(f), Q=x[:, :4],
                  Q_out=Qo, cu_seqlens=cu)
    mfb.sync_status()
    live = torch.cat([torch.arange(20), torch.arange(27, 60)]).cuda()
    pos = torch.cat([torch.arange(3, 23), torch.arange(33)])
    near_rotated(Qo[live], x[live][:, :4], pos, f, 64, False)
    assert (Qo[20:27] == 9.0).all() and (Qo[60:] == 9.0).all()
    at = torch.cat([slots(table, 16, 0, 3, 23), slots(table, 16, 2, 0, 33)])
    near_rotated(c.K.view(-1, 2, 64)[at], x[live][:, 4:6], pos, f, 64, False)
    keep = torch.ones(npages * 16, dtype=torch.bool, device="cuda")
    keep[at] = False
    assert torch.equal(c.K.view(-1, 2, 64)[keep], K0.view(-1, 2, 64)[keep])


@pytest.mark.parametrize("dt", [BF, F32])
def test_tokens_behind_the_last_sequence(dt):
    """A captured append and rotation of a fixed batch whose sequences fill it less and less: the
    pools' other rows and the padding's rows of every output stay as they were."""
    ntok, nseq, Hq, Hkv, d = 40, 3, 4, 2, 128
    table, npages = pages([64] * nseq, 16, 86)
    c = mfb.KVCache(randn((npages, 16, Hkv, d), dt, 87), randn((npages, 16, Hkv, d), dt, 88), table)
    K0, V0 = c.K.clone(), c.V.clone()
    Q, K, V = (randn((ntok, h, d), dt, 89 + i) for i, h in enumerate((Hq, Hkv, Hkv)))
    f = mfb.rope_freqs(d)
    rp = mfb.Rope.from_freqs(f)
    past, cu = i32([3, 0, 20]), i32([0, 15, 15, 40])
    Qa, Qr, Kr = (torch.zeros((ntok, h, d), dtype=dt, device="cuda") for h in (Hq, Hq, Hkv))

    def run():
        mfb.kv_append(c, K, V, past, rope=rp, Q=Q, Q_out=Qa, cu_seqlens=cu)
        mfb.rope(rp, Q, K, start=past, cu_seqlens=cu, Q_out=Qr, K_out=Kr, backward=True)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for bounds in ([0, 15, 15, 40], [0, 15, 15, 39], [0, 7, 19, 20], [0, 0, 1, 1], [0, 0, 0, 0]):
        cu.copy_(i32(bounds))
        c.K.copy_(K0)
        c.V.copy_(V0)
        for x in (Qa, Qr, Kr):
            x.fill_(9.0)
        graph.replay()
        mfb.sync_status()
        n = bounds[-1]
        pos = torch.cat([torch.arange(p, p + b - a)
                         for p, a, b in zip((3, 0, 20), bounds, bounds[1:])])
        near_rotated(Qa[:n], Q[:n], pos, f, d, False)
        near_rotated(Qr[:n], Q[:n], pos, f, d, False, backward=True)
        near_rotated(Kr[:n], K[:n], pos, f, d, False, backward=True)
        for x in (Qa, Qr, Kr):
            assert (x[n:] == 9.0).all()
        at = torch.cat([slots(table, 16, s, p, p + b - a) for s, (p, a, b) in
                        enumerate(zip((3, 0, 20), bounds, bounds[1:]))])
        near_rotated(c.K.view(-1, Hkv, d)[at], K[:n], pos, f, d, False)
        assert torch.equal(c.V.view(-1, Hkv, d)[at], V[:n])
        keep = torch.ones(npages * 16, dtype=torch.bool, device="cuda")
        keep[at] = False
        for x, x0 in ((c.K, K0), (c.V, V0)):
            assert torch.equal(x.view(-1, Hkv, d)[keep], x0.view(-1, Hkv, d)[keep])


@pytest.mark.parametrize("dt", [BF, F32])
def test_a_pool_without_pages(dt):
    """No pages: sequences without tokens are empty rows, others have no key and are reported."""
    c = mfb.KVCache.make(0, 16, 2, 64, dt, torch.full((3, 4), -1, dtype=torch.int32, device="cuda"))
    Q = randn((3, 4, 64), dt, 92)
    O, lse = mfb.paged_attn(c, Q, i32([0, 0, 0]))
    mfb.sync_status()
    assert (O == 0).all() and (lse == -math.inf).all()
    O, lse = mfb.paged_attn(c, Q, i32([0, 30, 0]))
    with pytest.raises(mfb.MapflowError):
        mfb.sync_status()
    assert (O == 0).all() and (lse == -math.inf).all()
    mfb.sync_status()  # reported once
