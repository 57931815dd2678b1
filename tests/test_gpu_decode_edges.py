"""Edges of the receiver's decode calls on the GPU: places that do not exist, infinities and NaN
among keys and values, biases of the type's size, angles near a quarter turn.

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
from tests.test_gpu_decode_cuts import widened

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


# ------------------------------------------------------------------ angles

def test_angles_near_quarter_turns():
    """Cosines and sines near their zeros keep their digits.  An angle's distance from the nearest
    quarter turn is rounded to float32 (2^-24 of it, or 2^-34 turns where that is more); a sine
    of an eighth of a turn or less passes no more than that on, relative, and sincospif's 2 units
    (2^-23 each), and the cosine of so small an angle less: 2^-21 of the value and 2^-33 pi."""
    r, n = np.random.default_rng(11), 32
    off = [0, 1, -1, 1 << 30, -(1 << 30)] + [
        int(s * 2.0 ** e) for s, e in zip(r.choice([-1, 1], 123), r.uniform(28, 61, 123))]
    angles = [(q << 62) + d for d in off for q in range(4)]
    x = torch.zeros(1, 1, 2 * n, device="cuda")
    x[..., :n] = 1.0                                  # a pair's outputs: its cosine and its sine
    for k in range(0, len(angles), n):
        part = angles[k:k + n]
        phases = torch.from_numpy(np.array([a % 2 ** 64 for a in part], np.uint64).view(np.int64))
        y = mfb.rope(mfb.Rope(phases.cuda()), x, start=i32([1]))[0, 0].double().cpu()
        for i, a in enumerate(part):
            q, d = (a + (1 << 61)) >> 62, ((a + (1 << 61)) % (1 << 62)) - (1 << 61)
            co, si = math.cos(2 * math.pi * d / 2 ** 64), math.sin(2 * math.pi * d / 2 ** 64)
            want = [(co, si), (-si, co), (-co, -si), (si, -co)][q % 4]
            for got, w in zip((float(y[i]), float(y[n + i])), want):
                assert abs(got - w) <= 2.0 ** -21 * abs(w) + 2.0 ** -33 * math.pi, (a, got, w)


# ------------------------------------------------------------------ attention

# head groups of every kernel variant
LAYOUTS = [(BF, 8, 2, 128), (BF, 6, 1, 128), (BF, 24, 2, 128), (BF, 8, 2, 64), (BF, 28, 4, 64),
           (BF, 5, 1, 64), (BF, 12, 1, 64), (F32, 6, 2, 128), (F32, 7, 1, 64), (F32, 18, 2, 64)]


@pytest.mark.parametrize("dt,Hq,Hkv,d", LAYOUTS)
@pytest.mark.parametrize("L,low", [(2500, 2000), (60, 41), (9000, 8991)])
def test_values_behind_logits_of_minus_infinity(dt, Hq, Hkv, d, L, low):
    """Keys 0 .. low-1 of a row have logits of -inf, all keys of another row: a NaN or an infinity
    among their values is a NaN in that dim, wherever the row is cut (alone or in a batch, behind
    a tight table or a wide one), and the other dims are those of the keys that are left."""
    lengths, G = [L, L, 33, 700], Hq // Hkv
    c = filled_cache(lengths, 16, Hkv, d, dt, 100)
    kf, vf = c.K.view(-1, Hkv, d), c.V.view(-1, Hkv, d)
    Q = randn((4, Hq, d), dt, 101)
    Q[:, :, 0] = Q[:, :, 0].abs() + 0.5
    at = [slots(c.page_table, 16, s, 0, n) for s, n in enumerate(lengths)]
    kf[at[0][:low], :, 0] = -math.inf
    kf[at[1], :, 0] = -math.inf
    vf[at[0][low // 3], :, 5], vf[at[0][low // 2], :, 9] = math.nan, math.inf
    vf[at[1][L // 2], :, 3], vf[at[1][0], :, 7] = math.nan, -math.inf
    other = torch.ones(d, dtype=torch.bool, device="cuda")
    for n in (1, 2, 4):                               # sequences in the batch
        for table in (c.page_table, widened(c, c.max_pages + 600).page_table):
            k = mfb.KVCache(c.K, c.V, table[:n].contiguous())
            O, lse = mfb.paged_attn(k, Q[:n], i32(lengths[:n]))
            mfb.sync_status()
            other[:] = True
            other[[5, 9]] = False
            assert O[0][:, ~other].isnan().all()
            for h in range(Hkv):
                hs = slice(h * G, (h + 1) * G)
                o, e, tol, delta = attend64(Q[0, hs].double(), kf[at[0][low:], h].double(),
                                            vf[at[0][low:], h].double(), d ** -0.5, 0.0, 0, 0)
                tol = tol + torch.finfo(dt).eps / 2 * o.abs()
                assert ((O[0, hs].double() - o).abs() <= tol)[:, other].all()
                assert ((lse[hs, 0].double() - e).abs() <= delta + 2.0 ** -22 * e.abs()).all()
            if n > 1:
                other[:] = True
                other[[3, 7]] = False
                assert O[1][:, ~other].isnan().all() and (O[1][:, other] == 0).all()
                assert (lse[:, 1] == -math.inf).all()


@pytest.mark.parametrize("dt,Hq,Hkv,d", LAYOUTS)
@pytest.mark.parametrize("lengths", [[2500, 17, 700], [60, 1], [9000]], ids=len)
def test_infinities_among_values(dt, Hq, Hkv, d, lengths):
    """An infinity among the values makes its dim that infinity, both signs or a NaN make it NaN,
    in its own KV head alone; every other output keeps its bits.  Logits lie within 40 of one
    another, so that every weight is far from a float32's smallest."""
    n, G = len(lengths), Hq // Hkv
    c = filled_cache(lengths, 16, Hkv, d, dt, 110)
    Q = randn((n, Hq, d), dt, 111, 0.5)
    wide = widened(c, c.max_pages + 600).page_table
    plain = [mfb.paged_attn(mfb.KVCache(c.K, c.V, t), Q, i32(lengths))[0]
             for t in (c.page_table, wide)]
    want = [x.clone() for x in plain]
    vf, r = c.V.view(-1, Hkv, d), np.random.default_rng(7)
    for s, L in enumerate(lengths):
        at = slots(c.page_table, 16, s, 0, L)
        h, hit = s % Hkv, {}
        for dim in range(4, d, 5):
            j, kind = int(r.integers(L)), float(r.choice([math.inf, -math.inf, math.nan]))
            hit.setdefault(dim, []).append(kind)
            vf[at[j], h, dim] = kind
        if L > 1:                                     # both signs in one dim; one in every key
            vf[at[0], h, 1], vf[at[L - 1], h, 1] = math.inf, -math.inf
            vf[at, h, 2] = -math.inf
            hit[1], hit[2] = [math.nan], [-math.inf]
        for dim, kinds in hit.items():
            for x in want:
                x[s, h * G:(h + 1) * G, dim] = kinds[0]
    for t, x in zip((c.page_table, wide), want):
        O, lse = mfb.paged_attn(mfb.KVCache(c.K, c.V, t), Q, i32(lengths))
        mfb.sync_status()
        assert torch.equal(O.isnan(), x.isnan())
        assert torch.equal(O.nan_to_num(nan=0.0), x.nan_to_num(nan=0.0))
        assert lse.isfinite().all()


LOWEST = float(torch.finfo(F32).min)


@pytest.mark.parametrize("dt,Hq,Hkv,d", LAYOUTS[:1] + LAYOUTS[2:4] + LAYOUTS[7:9])
@pytest.mark.parametrize("bias", [LOWEST, -1e30, -3e4, 3e4, 2.3e38])
@pytest.mark.parametrize("window", [0, 64])
def test_band_bias_of_any_size(dt, Hq, Hkv, d, bias, window):
    """A row that lies inside the band, as all of a short sequence or of a short window does, has
    the weights of a row without one and a log-sum-exp further by the bias; a bias far below the
    logits masks the band's keys of a longer row."""
    lengths, band, G = [1, 40, 100, 101, 300, 9000], 100, Hq // Hkv
    c = filled_cache(lengths, 16, Hkv, d, dt, 120, window=window)
    Q = randn((len(lengths), Hq, d), dt, 121)
    for table in (c.page_table, widened(c, c.max_pages + 600).page_table):
        k = mfb.KVCache(c.K, c.V, table)
        O, lse = mfb.paged_attn(k, Q, i32(lengths), band_bias=bias, band_width=band, window=window)
        mfb.sync_status()
        for s, L in enumerate(lengths):
            lo, hi, shift = max(0, L - window) if window else 0, L, bias
            if lo < L - band:                         # longer than the band
                if bias > 0:
                    continue
                hi, shift = L - band, 0.0             # logits lie within 1e3 of zero
            at = slots(c.page_table, 16, s, lo, hi)
            for h in range(Hkv):
                hs = slice(h * G, (h + 1) * G)
                o, e, tol, delta = attend64(Q[s, hs].double(),
                                            c.K.view(-1, Hkv, d)[at, h].double(),
                                            c.V.view(-1, Hkv, d)[at, h].double(), d ** -0.5, 0.0, 0,
                                            0)
                tol = tol + torch.finfo(dt).eps / 2 * o.abs()
                assert ((O[s, hs].double() - o).abs() <= tol).all(), (s, L)
                e = e + shift
                # the sum with the bias rounds once more, at the bias's size
                err = (lse[hs, s].double() - e).abs()
                assert (err <= delta + 2.0 ** -22 * e.abs()).all(), (s, L)


@pytest.mark.parametrize("dt,Hq,Hkv,d", [(BF, 8, 2, 128), (F32, 4, 2, 64)])
def test_a_chunk_attends_through_repeated_table_rows(dt, Hq, Hkv, d):
    """Several new tokens of a sequence: one append, then one attention over a table with the
    sequence's row once a token, each token's own length."""
    past, n = [700, 0], [9, 21]
    table, npages = pages([p + m for p, m in zip(past, n)], 16, 140)
    c = mfb.KVCache(randn((npages, 16, Hkv, d), dt, 141), randn((npages, 16, Hkv, d), dt, 142),
                    table)
    x, cu = randn((30, Hq + 2 * Hkv, d), dt, 143), i32([0, 9, 30])
    Q = mfb.kv_append(c, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], i32(past), rope=mfb.Rope.make(d),
                      Q=x[:, :Hq], cu_seqlens=cu)
    rows = torch.repeat_interleave(torch.arange(2, device="cuda"), i32(n).long())
    each = mfb.KVCache(c.K, c.V, table[rows].contiguous())
    lengths = [p + 1 + i for p, m in zip(past, n) for i in range(m)]
    O, lse = mfb.paged_attn(each, Q, i32(lengths))
    mfb.sync_status()
    check_attention(each, lengths, Q, O, lse, d ** -0.5)


# ------------------------------------------------------------------ marshalling

def small_calls(dev="cuda"):
    """(function, arguments, keywords) of one valid call of each kind, and the cache."""
    with torch.cuda.device(dev):
        c = filled_cache([40, 17], 16, 2, 64, F32, 130)
        rp, lens, x = mfb.Rope.make(64), i32([40, 17]), randn((2, 8, 64), F32, 131)
        Q, K = x[:, :4], x[:, 4:6]
        return c, [(mfb.rope, (rp, Q, K), dict(start=lens)),
                   (mfb.rope, (rp, Q), dict(cu_seqlens=i32([0, 2]), backward=True)),
                   (mfb.kv_append, (c, K, x[:, 6:], i32([39, 16])), dict(rope=rp, Q=Q)),
                   (mfb.paged_attn, (c, Q, lens), dict(band_bias=1.0, band_width=3))]


def test_a_call_is_made_in_one_place(monkeypatch):
    """What the marshalling does not take is refused, never made some other way."""
    c, calls = small_calls()
    want = [f(*a, **kw) for f, a, kw in calls]
    K0, fast = c.K.clone(), mfb._fast

    class Refusing:
        def __getattr__(self, name):
            return fast.kv_cache if name == "kv_cache" else lambda *a: None

    monkeypatch.setattr(mfb, "_fast", Refusing())
    for f, a, kw in calls:
        with pytest.raises(mfb.MapflowError) as e:
            f(*a, **kw)
        assert e.value.status == mfb.MF_ERR_INVALID_ARG and str(e.value)
    assert torch.equal(c.K.view(torch.int32), K0.view(torch.int32))
    monkeypatch.undo()
    for (f, a, kw), w in zip(calls, want):
        got = f(*a, **kw)
        for x, y in zip(got, w) if isinstance(w, tuple) else ((got, w),):
            assert torch.equal(x, y)
    mfb.sync_status()


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_tensors_on_another_device_than_the_current_one():
    _, calls = small_calls("cuda:0")
    want = [f(*a, **kw) for f, a, kw in calls]
    _, calls = small_calls("cuda:1")
    for (f, a, kw), w in zip(calls, want):
        got = f(*a, **kw)
        assert torch.cuda.current_device() == 0
        for x, y in zip(got, w) if isinstance(w, tuple) else ((got, w),):
            assert x.device.index == 1 and torch.equal(x.cpu(), y.cpu())
