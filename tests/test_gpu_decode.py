"""Rotary positions, the paged key-value append and the single-token attention on the GPU,
against plain 64-bit evaluations of their formulas.

Tolerances.  A result is rounded once to its type: half a step, `finfo.eps / 2` of its size.
Before that:
* rotation: the angle is a float32 of half turns (2^-25 of a half turn: 9.4e-8 rad), sine and
  cosine are within 2 units (2 * 2^-24 each), the scale and the two products round once each:
  together below 5e-7 (|a| + |b|) |scale| for the pair (a, b);
* attention: a logit is a float32 sum of d products in any order: within
  (d + 8) 2^-24 sum_i |q_i k_i| |scale|, its exponent's scaling, bias and power of two within
  2^-22 (1 + |x|) more; with delta the largest of these over a row's keys plus 2^-16 (weights
  kept in two bf16 halves) plus L 2^-24 (the sums), the log-sum-exp is within delta (and one
  rounding) and O within 2 delta sum_j p_j |v_j|.
"""
import math

import numpy as np
import pytest
import torch

from cross_model_attention_block_b200 import mapflow as mfb
from cross_model_attention_block_b200 import synth

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, dt, seed, gain=1.5):
    return (torch.randn(shape, device="cuda", generator=gen(seed)) * gain).to(dt)


# --------------------------------------------------------------------- rotation

def rotate64(x, pos, f, rot, interleaved, scale=1.0, backward=False):
    """(rotated x, |a| + |b| of every element's pair), both float64."""
    y, pair = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    ang = pos.double().to(x.device)[:, None] * torch.as_tensor(f, device=x.device)[None]
    co, si = (ang.cos() * scale)[:, None], (ang.sin() * scale)[:, None]
    if backward:
        si = -si
    ia, ib = ((slice(0, rot, 2), slice(1, rot, 2)) if interleaved
              else (slice(0, rot // 2), slice(rot // 2, rot)))
    a, b = x[..., ia].double(), x[..., ib].double()
    y[..., ia], y[..., ib] = a * co - b * si, a * si + b * co
    pair[..., ia] = pair[..., ib] = a.abs() + b.abs()
    return y, pair


def near_rotated(got, x, pos, f, rot, interleaved, scale=1.0, backward=False):
    want, pair = rotate64(x, pos, f, rot, interleaved, scale, backward)
    tol = torch.finfo(x.dtype).eps / 2 * want.abs() + 5e-7 * abs(scale) * pair
    assert got.dtype == x.dtype
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), float((got.double() - want).abs().max()))
    assert torch.equal(got[..., rot:], x[..., rot:])


ROPES = [(128, 128, False), (128, 128, True), (128, 64, False), (128, 32, True), (64, 64, False),
         (64, 16, True), (64, 20, False), (128, 6, True), (64, 2, False), (128, 126, False)]


@pytest.mark.parametrize("d,rot,interleaved", ROPES)
@pytest.mark.parametrize("dt", [BF, F32])
def test_rope_packed(dt, d, rot, interleaved):
    """Ragged sequences (one empty, one of one token), starts, Q and K with their own head
    counts, forward and transposed."""
    lengths, start = [3, 0, 1, 70, 37], [0, 5, 100001, -3, 7]
    cu = i32(np.concatenate([[0], np.cumsum(lengths)]))
    n = sum(lengths)
    pos = torch.cat([torch.arange(s, s + m) for s, m in zip(start, lengths)])
    f = mfb.rope_freqs(rot)
    for Hq, Hk, backward, scale in ((5, 1, False, 1.0), (40, 40, True, 1.25), (3, 0, True, 1.0)):
        rp = mfb.Rope.from_freqs(f, interleaved, scale)
        Q = randn((n, Hq, d), dt, 1)
        K = randn((n, Hk, d), dt, 2) if Hk else None
        out = mfb.rope(rp, Q, K, start=i32(start), cu_seqlens=cu, backward=backward)
        outs = out if Hk else (out,)
        for x, y in zip((Q, K), outs):
            near_rotated(y, x, pos, f, rot, interleaved, scale, backward)


@pytest.mark.parametrize("ntok", [1, 2, 591, 593, 5000])
def test_rope_token_counts(ntok):
    """One token to many (the launch shape changes between), every token its own position."""
    f = mfb.rope_freqs(128)
    pos = torch.randint(0, 1 << 20, (ntok,), generator=torch.Generator().manual_seed(ntok))
    Q, K = randn((ntok, 32, 128), BF, 3), randn((ntok, 8, 128), BF, 4)
    q, k = mfb.rope(mfb.Rope.from_freqs(f), Q, K, start=i32(pos.tolist()))
    near_rotated(q, Q, pos, f, 128, False)
    near_rotated(k, K, pos, f, 128, False)


def test_rope_far_positions_keep_their_angle():
    """Positions to 2^31 - 1: the 64-bit oracle takes whole turns off exactly, in integers."""
    pos = [0, 1, 131071, 1 << 24, (1 << 24) + 1, 2 ** 31 - 1, -(2 ** 31)]
    f = mfb.rope_freqs(64)
    rp = mfb.Rope.from_freqs(f)
    ph = [int(x) % 2 ** 64 for x in rp.phases.tolist()]
    ang = torch.tensor([[(p * w) % 2 ** 64 / 2 ** 64 * 2 * math.pi for w in ph] for p in pos],
                       dtype=torch.float64, device="cuda")
    x = randn((len(pos), 2, 64), F32, 5)
    y = mfb.rope(rp, x, start=i32(pos))
    a, b = x[..., :32].double(), x[..., 32:].double()
    want = torch.cat([a * ang.cos()[:, None] - b * ang.sin()[:, None],
                      a * ang.sin()[:, None] + b * ang.cos()[:, None]], -1)
    pair = torch.cat([a.abs() + b.abs()] * 2, -1)
    assert ((y.double() - want).abs() <= 2 ** -24 * want.abs() + 5e-7 * pair).all()


@pytest.mark.parametrize("dt,rot", [(BF, 128), (F32, 48), (BF, 20)])
def test_rope_strided_offset_and_in_place(dt, rot):
    """Slices of a fused projection, odd storage offsets, and outputs that are their inputs."""
    n, f = 9, mfb.rope_freqs(rot)
    pos = torch.arange(11, 11 + n)
    rp = mfb.Rope.from_freqs(f)
    cu, st = i32([0, n]), i32([11])
    x = randn((n, 4 + 2 + 2, 128), dt, 6)
    q, k = mfb.rope(rp, x[:, :4], x[:, 4:6], start=st, cu_seqlens=cu)
    near_rotated(q, x[:, :4], pos, f, rot, False)
    near_rotated(k, x[:, 4:6], pos, f, rot, False)
    flat = randn((n * 4 * 128 + 3,), dt, 7)
    odd = flat[3:].view(n, 4, 128)                    # starts off a 16-byte boundary
    assert torch.equal(mfb.rope(rp, odd, start=st, cu_seqlens=cu),
                       mfb.rope(rp, odd.clone(), start=st, cu_seqlens=cu))
    y = x.clone()
    mfb.rope(rp, y[:, :4], y[:, 4:6], start=st, cu_seqlens=cu, Q_out=y[:, :4], K_out=y[:, 4:6])
    assert torch.equal(y[:, :4], q) and torch.equal(y[:, 4:6], k)
    assert torch.equal(y[:, 6:], x[:, 6:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient(interleaved):
    """The transposed call against the formula's gradient (autograd in 64 bits) and against
    central differences of the forward call."""
    n, H, d, rot, scale = 6, 3, 64, 32, 1.1
    f = mfb.rope_freqs(rot)
    rp = mfb.Rope.from_freqs(f, interleaved, scale)
    st = i32([0, 3, 77, 1000, 5, 123456])
    x, g = randn((n, H, d), F32, 8), randn((n, H, d), F32, 9)
    got = mfb.rope(rp, g, start=st, backward=True)
    z = x.double().requires_grad_()
    ang = st.double()[:, None] * torch.as_tensor(f, device="cuda")
    co, si = (ang.cos() * scale)[:, None], (ang.sin() * scale)[:, None]
    ia, ib = ((slice(0, rot, 2), slice(1, rot, 2)) if interleaved
              else (slice(0, rot // 2), slice(rot // 2, rot)))
    gg = g.double()
    loss = (gg[..., ia] * (z[..., ia] * co - z[..., ib] * si)).sum() \
        + (gg[..., ib] * (z[..., ia] * si + z[..., ib] * co)).sum() \
        + (gg[..., rot:] * z[..., rot:]).sum()
    loss.backward()
    near_rotated(got, g, st.cpu(), f, rot, interleaved, scale, backward=True)
    pair = rotate64(g, st.cpu(), f, rot, interleaved)[1]
    assert ((got.double() - z.grad).abs() <= 2 ** -24 * z.grad.abs() + 5e-7 * scale * pair).all()
    # differences along a direction u: <g, rope(x + u) - rope(x - u)> / 2 = <rope^T g, u>, as
    # the map is linear; the two forwards and the inputs x +- u round, each term as above
    u = randn((n, H, d), F32, 10)
    yp, ym = mfb.rope(rp, x + u, start=st), mfb.rope(rp, x - u, start=st)
    left = (gg * (yp.double() - ym.double())).sum() / 2
    right = (got.double() * u.double()).sum()
    size = (gg.abs() * (rotate64(x + u, st.cpu(), f, rot, interleaved)[1] + (x + u).abs())).sum()
    assert abs(float(left - right)) <= 2e-6 * scale * float(size)


# --------------------------------------------------------------------- paged cache

def pages(lengths, ps, seed, extra=2):
    """Page table with random pages (-1 where unused) and the pool's page count."""
    need = [-(-n // ps) for n in lengths]
    total = sum(need) + extra
    perm = np.random.default_rng(seed).permutation(total).astype(np.int32)
    t = np.full((len(lengths), max(need + [1])), -1, np.int32)
    k = 0
    for s, m in enumerate(need):
        t[s, :m] = perm[k:k + m]
        k += m
    return torch.from_numpy(t).cuda(), total


def slots(table, ps, s, lo, hi):
    """Pool rows of tokens lo .. hi-1 of sequence s."""
    j = torch.arange(lo, hi, device="cuda")
    return table[s].long()[j // ps] * ps + j % ps


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("ps,Hq,Hkv,d,rot,interleaved", [
    (16, 8, 2, 64, 64, False), (48, 5, 5, 128, 32, True), (16, 0, 3, 128, 128, False),
    (128, 32, 8, 128, 20, False)])
def test_append(dt, ps, Hq, Hkv, d, rot, interleaved):
    """Prompts and chunks of ragged sequences: every slot of the new tokens holds the rotated
    key and the value, every other slot of the pools what it held."""
    new, past = [17, 0, 1, 130, 33], [0, 4, 15, 31, 200]
    table, npages = pages([a + b for a, b in zip(new, past)], ps, 1)
    c = mfb.KVCache(randn((npages, ps, Hkv, d), dt, 1), randn((npages, ps, Hkv, d), dt, 2), table)
    K0, V0 = c.K.clone(), c.V.clone()
    n, f = sum(new), mfb.rope_freqs(rot)
    cu = i32(np.concatenate([[0], np.cumsum(new)]))
    x = randn((n, Hq + 2 * Hkv, d), dt, 3)
    Q, K, V = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    q = mfb.kv_append(c, K, V, i32(past), rope=mfb.Rope.from_freqs(f, interleaved),
                      Q=Q if Hq else None, cu_seqlens=cu)
    mfb.sync_status()
    pos = torch.cat([torch.arange(p, p + m) for p, m in zip(past, new)])
    if Hq:
        near_rotated(q, Q, pos, f, rot, interleaved)
    at = torch.cat([slots(table, ps, s, p, p + m) for s, (p, m) in enumerate(zip(past, new))])
    kf, vf = c.K.view(-1, Hkv, d), c.V.view(-1, Hkv, d)
    near_rotated(kf[at], K, pos, f, rot, interleaved)
    assert torch.equal(vf[at], V)
    keep = torch.ones(npages * ps, dtype=torch.bool, device="cuda")
    keep[at] = False
    assert torch.equal(kf[keep], K0.view(-1, Hkv, d)[keep])
    assert torch.equal(vf[keep], V0.view(-1, Hkv, d)[keep])


def test_append_single_tokens_without_rotation_and_padding():
    """One token per sequence, no rope; a negative length leaves its rows as they were."""
    past = [5, -1, 0, 31]
    table, npages = pages([6, 1, 1, 32], 16, 2)
    c = mfb.KVCache(randn((npages, 16, 2, 64), BF, 1), randn((npages, 16, 2, 64), BF, 2), table)
    K0 = c.K.clone()
    K, V, Q = randn((4, 2, 64), BF, 3), randn((4, 2, 64), BF, 4), randn((4, 6, 64), BF, 5)
    Qo = torch.full_like(Q, 9.0)
    mfb.kv_append(c, K, V, i32(past), Q=Q, Q_out=Qo)
    mfb.sync_status()
    live = [0, 2, 3]
    at = torch.cat([slots(table, 16, s, past[s], past[s] + 1) for s in live])
    assert torch.equal(c.K.view(-1, 2, 64)[at], K[live])
    assert torch.equal(c.V.view(-1, 2, 64)[at], V[live])
    assert torch.equal(Qo[live], Q[live]) and (Qo[1] == 9.0).all()
    keep = torch.ones(npages * 16, dtype=torch.bool, device="cuda")
    keep[at] = False
    assert torch.equal(c.K.view(-1, 2, 64)[keep], K0.view(-1, 2, 64)[keep])


def test_append_outside_the_table_or_pool_is_skipped_and_reported():
    table = i32([[0, 1], [9, -1], [2, -5]])
    c = mfb.KVCache(torch.zeros(4, 16, 1, 64, dtype=F32, device="cuda"),
                    torch.zeros(4, 16, 1, 64, dtype=F32, device="cuda"), table)
    K = torch.ones(3, 1, 64, device="cuda")
    for past, wrote in (([32, 0, 16], 0), ([31, 15, 15], 2), ([2 ** 31 - 1, 16, 0], 1)):
        c.K.zero_()
        mfb.kv_append(c, K, K, i32(past))
        with pytest.raises(mfb.MapflowError) as e:
            mfb.sync_status()
        assert e.value.status == mfb.MF_ERR_INVALID_ARG and "page" in str(e.value)
        assert int((c.K != 0).any(-1).sum()) == wrote
    mfb.kv_append(c, K, K, i32([0, -1, 3]))
    mfb.sync_status()                                       # reported once, then clear


# --------------------------------------------------------------------- attention

def attend64(q, K, V, scale, bias, band, window):
    """O, lse, and their tolerances before rounding, of one sequence and KV head in float64:
    q [G, d], K, V [L, d]."""
    L, d = K.shape
    back = L - 1 - torch.arange(L, device=q.device)
    x = (q @ K.t()) * scale + bias * (back < band)
    sums = (q.abs() @ K.abs().t()) * abs(scale)
    seen = back < window if window else torch.ones_like(back, dtype=torch.bool)
    x = x.masked_fill(~seen, -math.inf)
    p = torch.softmax(x, -1)
    delta = ((d + 8) * 2.0 ** -24 * sums + 2.0 ** -22 * (1 + x.abs()))[:, seen].amax(-1) \
        + 2.0 ** -16 + L * 2.0 ** -24
    V = V.masked_fill(~seen[:, None], 0.0)
    return p @ V, torch.logsumexp(x, -1), 2 * delta[:, None] * (p @ V.abs()), delta


def check_attention(c, lengths, Q, O, lse, scale, bias=0.0, band=0, window=0):
    Hq, G = Q.shape[1], Q.shape[1] // c.Hkv
    kf, vf = c.K.view(-1, c.Hkv, c.d), c.V.view(-1, c.Hkv, c.d)
    for s, L in enumerate(lengths):
        if L <= 0:
            assert (O[s] == 0).all() and (lse[:, s] == -math.inf).all()
            continue
        at = slots(c.page_table, c.page_size, s, 0, L)
        for h in range(c.Hkv):
            hs = slice(h * G, (h + 1) * G)
            K, V = kf[at, h].double(), vf[at, h].double()
            if window:  # what the window hides may hold anything
                K[:max(0, L - window)], V[:max(0, L - window)] = 0.0, 0.0
            o, e, tol, delta = attend64(Q[s, hs].double(), K, V, scale, bias, band, window)
            tol = tol + torch.finfo(O.dtype).eps / 2 * o.abs()
            err = (O[s, hs].double() - o).abs()
            assert (err <= tol).all(), (s, L, h, float(err.max()), float(tol.min()))
            err = (lse[hs, s].double() - e).abs()
            assert (err <= delta + 2.0 ** -22 * e.abs()).all(), (s, L, h, float(err.max()))


def filled_cache(lengths, ps, Hkv, d, dt, seed, holes=float("nan"), window=0):
    """A cache whose rows outside the sequences (and before their windows) hold `holes`."""
    table, npages = pages([max(n, 0) for n in lengths], ps, seed)
    c = mfb.KVCache.make(npages, ps, Hkv, d, dt, table)
    c.K.fill_(holes)
    c.V.fill_(holes)
    for s, n in enumerate(lengths):
        lo = max(0, n - window) if window else 0
        if n > 0:
            at = slots(table, ps, s, lo, n)
            c.K.view(-1, Hkv, d)[at] = randn((n - lo, Hkv, d), dt, 10 * seed + s)
            c.V.view(-1, Hkv, d)[at] = randn((n - lo, Hkv, d), dt, 10 * seed + s + 5, 1.0)
    return c


SHAPES = [(BF, 32, 8, 128), (BF, 4, 4, 128), (BF, 16, 1, 128), (BF, 10, 2, 64), (BF, 40, 2, 128),
          (BF, 24, 8, 64), (F32, 8, 2, 64), (F32, 3, 3, 128), (F32, 32, 2, 128), (F32, 20, 1, 64)]
LENGTHS = [[1], [0], [0, 16, 1, -1, 15, 17, 0], [127, 128, 129, 255, 257, 31, 33],
           [2049, 3, 700, 0, 1024, 1]]


@pytest.mark.parametrize("dt,Hq,Hkv,d", SHAPES)
@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda v: "x".join(map(str, v)))
def test_attention_lengths(dt, Hq, Hkv, d, lengths):
    """Every head layout at lengths around the tile sizes; everything outside the sequences is
    NaN."""
    c = filled_cache(lengths, 16, Hkv, d, dt, 3)
    Q = randn((len(lengths), Hq, d), dt, 4)
    O, lse = mfb.paged_attn(c, Q, i32(lengths))
    mfb.sync_status()
    check_attention(c, lengths, Q, O, lse, d ** -0.5)


@pytest.mark.parametrize("dt,d", [(BF, 128), (BF, 64), (F32, 64)])
@pytest.mark.parametrize("ps", [16, 48, 256])
@pytest.mark.parametrize("bias,band,window", [(2.0, 256, 0), (2.0, 1, 100), (-30.0, 50, 0),
                                              (0.0, 0, 1), (1.0, 5, 129), (0.0, 0, 5000)])
def test_attention_band_window_pages(dt, d, ps, bias, band, window):
    lengths = [600, 1, 129, 0, 2000, 100]
    c = filled_cache(lengths, ps, 2, d, dt, 5, holes=float("inf"), window=window)
    Q = randn((len(lengths), 10, d), dt, 6)
    O, lse = mfb.paged_attn(c, Q, i32(lengths), band_bias=bias, band_width=band, window=window)
    mfb.sync_status()
    check_attention(c, lengths, Q, O, lse, d ** -0.5, bias, band, window)


@pytest.mark.parametrize("dt", [BF, F32])
def test_attention_long_and_many(dt):
    """One sequence over the whole GPU, and more rows than the GPU runs at once; the same
    call twice gives the same bits."""
    for lengths in ([30011], [700] * 150 + [1, 0, 5000]):
        c = filled_cache(lengths, 16, 2, 128, dt, 7)
        Q = randn((len(lengths), 8, 128), dt, 8)
        O, lse = mfb.paged_attn(c, Q, i32(lengths))
        O2, lse2 = mfb.paged_attn(c, Q, i32(lengths))
        mfb.sync_status()
        assert torch.equal(O, O2) and torch.equal(lse, lse2)
        check_attention(c, lengths, Q, O, lse, 128 ** -0.5)


@pytest.mark.parametrize("dt", [BF, F32])
def test_attention_extreme_values(dt):
    """Logits far apart (one key takes all), equal logits, large scales, and len_add."""
    lengths = [300, 64, 17]
    c = filled_cache(lengths, 16, 2, 64, dt, 9)
    Q = randn((3, 4, 64), dt, 10)
    for scale in (0.0, 30.0, -1.0, 1e-3):
        O, lse = mfb.paged_attn(c, Q, i32([n - 2 for n in lengths]), len_add=2, scale=scale)
        mfb.sync_status()
        check_attention(c, lengths, Q, O, lse, scale)


@pytest.mark.parametrize("dt", [BF, F32])
def test_attention_nan_and_infinity_in_keys(dt):
    """A NaN among the keys a query sees reaches exactly its KV head's outputs; keys of -inf
    logits take no part; a row with nothing but -inf is an empty one."""
    c = filled_cache([200, 40, 40], 16, 2, 64, dt, 11)
    Q = randn((3, 4, 64), dt, 12).abs()
    c.K.view(-1, 2, 64)[slots(c.page_table, 16, 0, 0, 200)[77], 1, 3] = float("nan")
    low = slots(c.page_table, 16, 1, 0, 40)
    c.K.view(-1, 2, 64)[low[:39], :, 0] = -math.inf
    c.K.view(-1, 2, 64)[slots(c.page_table, 16, 2, 0, 40), :, 0] = -math.inf
    O, lse = mfb.paged_attn(c, Q, i32([200, 40, 40]))
    mfb.sync_status()
    assert O[0, 2:].isnan().all() and O[0, :2].isfinite().all()
    v = c.V.view(-1, 2, 64)[low[39]].repeat_interleave(2, 0)
    assert torch.equal(O[1], v)
    assert (O[2] == 0).all() and (lse[:, 2] == -math.inf).all()


def test_attention_strides_outputs_and_workspace():
    """Q from a fused projection, O into a wider buffer (the rest left alone), O over Q, a
    caller's workspace, padding rows."""
    lengths = [100, 37, -5]
    c = filled_cache(lengths, 16, 2, 128, BF, 13)
    x = randn((3, 8 + 4, 128), BF, 14)
    O, lse = mfb.paged_attn(c, x[:, :8], i32(lengths))
    check_attention(c, lengths, x[:, :8], O, lse, 128 ** -0.5)
    wide = torch.full((3, 12, 128), 7.0, dtype=BF, device="cuda")
    ws = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
    mfb.paged_attn(c, x[:, :8], i32(lengths), O=wide[:, :8], workspace=ws)
    assert torch.equal(wide[:, :8], O) and (wide[:, 8:] == 7.0).all()
    Q = x[:, :8].contiguous()
    mfb.paged_attn(c, Q, i32(lengths), O=Q)
    assert torch.equal(Q, O)


@pytest.mark.parametrize("dt", [BF, F32])
def test_attention_bad_pages_are_masked_and_reported(dt):
    """Pages outside the pool and lengths past the table: those keys take no part."""
    lengths = [40, 40]
    c = filled_cache(lengths, 16, 1, 64, dt, 15)
    Q = randn((2, 2, 64), dt, 16)
    good = c.page_table.clone()
    O, lse = mfb.paged_attn(c, Q, i32(lengths))
    mfb.sync_status()
    kept = torch.cat([slots(good, 16, 0, 0, 16), slots(good, 16, 0, 32, 40)])
    for bad in (-1, c.npages, 2 ** 31 - 1, -(2 ** 31)):
        c.page_table[0, 1] = bad
        O2, lse2 = mfb.paged_attn(c, Q, i32(lengths))
        with pytest.raises(mfb.MapflowError) as e:
            mfb.sync_status()
        assert e.value.status == mfb.MF_ERR_INVALID_ARG
        K, V = c.K.view(-1, 64)[kept].double(), c.V.view(-1, 64)[kept].double()
        o, l_, tol, delta = attend64(Q[0].double(), K, V, 64 ** -0.5, 0.0, 0, 0)
        assert ((O2[0].double() - o).abs() <= tol + torch.finfo(dt).eps / 2 * o.abs()).all()
        assert ((lse2[:, 0].double() - l_).abs() <= delta + 2.0 ** -22 * l_.abs()).all()
        assert torch.equal(O2[1], O[1]) and torch.equal(lse2[:, 1], lse[:, 1])
    c.page_table.copy_(good)
    O3, _ = mfb.paged_attn(c, Q, i32([40, 2 ** 31 - 1]))
    with pytest.raises(mfb.MapflowError):
        mfb.sync_status()
    assert torch.equal(O3[0], O[0])


def test_offsets_past_32_bits():
    """A pool of more than 2^31 elements: append to and attend over its last pages."""
    npages, ps, Hkv, d = (1 << 31) // (16 * 8 * 128) + 40, 16, 8, 128
    table = torch.arange(npages - 20, npages, dtype=torch.int32, device="cuda").flip(0)[None]
    c = mfb.KVCache.make(npages, ps, Hkv, d, BF, table.contiguous())
    assert c.K.numel() > 1 << 31
    K, V = randn((300, Hkv, d), BF, 17), randn((300, Hkv, d), BF, 18, 1.0)
    mfb.kv_append(c, K, V, i32([0]), cu_seqlens=i32([0, 300]))
    at = slots(c.page_table, ps, 0, 0, 300)
    assert torch.equal(c.K.view(-1, Hkv, d)[at], K) and torch.equal(c.V.view(-1, Hkv, d)[at], V)
    Q = randn((1, 32, d), BF, 19)
    O, lse = mfb.paged_attn(c, Q, i32([300]))
    mfb.sync_status()
    check_attention(c, [300], Q, O, lse, d ** -0.5)


# --------------------------------------------------------------------- together

class Plain:
    """The receiver's own tokens in float64, unpaged: histories of rotated keys and values
    rounded to the cache's type."""

    def __init__(self, nseq, f, dt):
        self.k, self.v, self.f, self.dt = [[] for _ in range(nseq)], [[] for _ in range(nseq)], f, dt

    def add(self, s, pos, K, V):
        y = rotate64(K, pos, self.f, 2 * len(self.f), False)[0]
        self.k[s].append(y.to(self.dt).double())
        self.v[s].append(V.double())


@pytest.mark.parametrize("dt,Hs,Hr,Hkv,d", [(BF, 8, 32, 8, 128), (F32, 4, 4, 2, 64)])
def test_prefill_then_decode(dt, Hs, Hr, Hkv, d):
    """A receiver's life: its prompt's keys and values go to pages (mf_kv_append), the mapped
    prefill reads that V pool (mf_mapped_av), then steps of append and attention; the
    steps captured into a graph and replayed give the eager steps' bits."""
    lengths, steps = [70, 129, 1], 4
    w, x = synth.small_case(lengths, Hs, Hr, Hkv, d, 64, 0.9,
                            dtype="bf16" if dt == BF else "f32")
    ctx = mfb.Context.make(lengths, Hs, d, 64, w.band_bias, w.band_width, dt)
    rp = mfb.Rope.make(d)
    sQ, sK = mfb.rope(rp, x.Q.cuda(), x.K.cuda(), cu_seqlens=ctx.cu_seqlens)
    lse, mass = mfb.block_stats(ctx, sQ, sK)
    cache = mfb.select_extract(ctx, sQ, sK, lse, mass, 0.9)
    V, W = x.V.cuda(), x.W.cuda()
    K = randn(V.shape, dt, 20)
    table, npages = pages([n + steps for n in lengths], 16, 21)
    kv = mfb.KVCache.make(npages, 16, Hkv, d, dt, table)
    kv.K.fill_(float("nan"))
    kv.V.fill_(float("nan"))
    mfb.kv_append(kv, K, V, rope=rp, cu_seqlens=ctx.cu_seqlens)
    O = mfb.mapped_av(cache, Hr, W, kv.V, Hkv, page_table=kv.page_table, page_size=16)
    assert torch.equal(O, mfb.mapped_av(cache, Hr, W, V, Hkv))
    mfb.sync_status()

    plain, t = Plain(3, mfb.rope_freqs(d), dt), 0
    for s, n in enumerate(lengths):
        plain.add(s, torch.arange(n), K[t:t + n], V[t:t + n])
        t += n
    lens = i32(lengths)
    xs = [randn((3, Hr + 2 * Hkv, d), dt, 30 + k) for k in range(steps)]
    xin, out, l_out = torch.empty_like(xs[0]), torch.empty((3, Hr, d), dtype=dt, device="cuda"), \
        torch.empty((Hr, 3), device="cuda")

    def step():
        q = mfb.kv_append(kv, xin[:, Hr:Hr + Hkv], xin[:, Hr + Hkv:], lens, rope=rp,
                          Q=xin[:, :Hr])
        mfb.paged_attn(kv, q, lens, len_add=1, O=out, lse=l_out)
        lens.add_(1)

    eager = []
    for k in range(steps):
        xin.copy_(xs[k])
        pos = lens.cpu()
        step()
        eager.append((out.clone(), l_out.clone()))
        for s in range(3):
            plain.add(s, pos[s:s + 1], xs[k][s:s + 1, Hr:Hr + Hkv], xs[k][s:s + 1, Hr + Hkv:])
            q = rotate64(xs[k][s:s + 1, :Hr], pos[s:s + 1], plain.f, d, False)[0].to(dt).double()
            kk, vv = torch.cat(plain.k[s]), torch.cat(plain.v[s])
            for h in range(Hkv):
                hs = slice(h * Hr // Hkv, (h + 1) * Hr // Hkv)
                o, e, tol, delta = attend64(q[0, hs], kk[:, h], vv[:, h], d ** -0.5, 0.0, 0, 0)
                # a key or query that the two sides round to neighbouring values of its type
                # moves its logit by a step of one product: counted as one step of each term
                step_x = torch.finfo(dt).eps * (q[0, hs].abs() @ kk[:, h].abs().t()).amax(-1) \
                    * d ** -0.5 / d
                size = tol / (2 * delta[:, None])
                tol = tol + 2 * step_x[:, None] * 4 * size + torch.finfo(dt).eps / 2 * o.abs()
                assert ((out[s, hs].double() - o).abs() <= tol).all()
    mfb.sync_status()

    lens.copy_(i32(lengths))
    xin.copy_(xs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    lens.copy_(i32(lengths))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    lens.copy_(i32(lengths))
    for k in range(steps):
        xin.copy_(xs[k])
        graph.replay()
        assert torch.equal(out, eager[k][0]) and torch.equal(l_out, eager[k][1])
    mfb.sync_status()


def test_two_streams_at_once():
    """Independent calls on two streams, each with its own workspace, do not disturb each
    other."""
    lengths = [3000, 17, 900]
    c = filled_cache(lengths, 16, 2, 128, BF, 22)
    Q = [randn((3, 8, 128), BF, 40 + k) for k in range(2)]
    L = i32(lengths)
    want = [mfb.paged_attn(c, q, L) for q in Q]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in Q]
    for _ in range(20):
        got = []
        for k, s in enumerate(st):
            with torch.cuda.stream(s):
                got.append(mfb.paged_attn(c, Q[k], L))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    mfb.sync_status()
