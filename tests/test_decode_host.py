"""Rotary frequencies and phases, and the refusals of the receiver's decode calls
(mf_rope, mf_kv_append, mf_paged_attn): host only, nothing here launches a kernel."""
import copy
import ctypes as C
import math
import pickle
from fractions import Fraction

import numpy as np
import pytest
import torch

from cross_model_attention_block_b200 import mapflow as mfb

P = C.c_void_p
BAD, UNSUP, WS, NOGPU = (mfb.MF_ERR_INVALID_ARG, mfb.MF_ERR_UNSUPPORTED, mfb.MF_ERR_WORKSPACE,
                         mfb.MF_ERR_CUDA)
needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                                  reason="made-up pointers must not reach a GPU")


# ------------------------------------------------------------- frequencies

def test_frequencies_follow_their_formulas(lib):
    r, base, c, L0, low, high = 96, 500000.0, 4.0, 8192.0, 1.0, 32.0
    i = np.arange(r // 2)
    plain = base ** (-2.0 * i / r)
    np.testing.assert_allclose(mfb.rope_freqs(r, base), plain, rtol=1e-14)
    np.testing.assert_allclose(mfb.rope_freqs(r, base, "linear", c), plain / c, rtol=1e-14)
    ntk = (base * c ** (r / (r - 2))) ** (-2.0 * i / r)
    np.testing.assert_allclose(mfb.rope_freqs(r, base, "ntk", c), ntk, rtol=1e-13)
    # its slowest pair turns factor times as slowly, its fastest as before
    assert math.isclose(ntk[-1], plain[-1] / c, rel_tol=1e-12) and ntk[0] == 1.0
    parts = mfb.rope_freqs(r, base, "parts", c, L0, low, high)
    turns = L0 * plain / (2 * math.pi)
    assert np.array_equal(parts[turns >= high], plain[turns >= high])
    np.testing.assert_allclose(parts[turns <= low], plain[turns <= low] / c, rtol=1e-14)
    mid = (turns > low) & (turns < high)
    assert mid.any() and (turns >= high).any() and (turns <= low).any()
    g = (turns - low) / (high - low)
    np.testing.assert_allclose(parts[mid], ((1 - g) * plain / c + g * plain)[mid], rtol=1e-13)


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=8, base=0.0),
                                dict(rot_dim=8, base=float("nan")),
                                dict(rot_dim=8, scaling="linear", factor=0.0),
                                dict(rot_dim=2, scaling="ntk", factor=2.0),
                                dict(rot_dim=8, scaling="parts", factor=2.0),
                                dict(rot_dim=8, scaling="parts", factor=2.0, original_length=10.0,
                                     low=4.0, high=4.0),
                                dict(rot_dim=8, scaling="other")])
def test_frequencies_refuse(lib, kw):
    with pytest.raises(mfb.MapflowError) as e:
        mfb.rope_freqs(**kw)
    assert e.value.status == BAD and str(e.value)


def test_phases_are_turns_modulo_one(lib):
    """2^64 f / 2 pi modulo 2^64, to the last bits of a 64-bit significand."""
    pi = Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
    f = np.array([1.0, 0.5, 1e-4, 6.0, 7.5, -0.25, 0.0, 123.456, 1e-300])
    got = mfb.Rope.from_freqs(f, device="cpu").phases.numpy().view(np.uint64)
    for x, g in zip(f, got):
        turns = Fraction(float(x)) / (2 * pi)
        want = round((turns - math.floor(turns)) * 2 ** 64) % 2 ** 64
        # the quotient is rounded to 64 bits: relative 2^-64 of the turns, and
        # half a unit of the last place
        off = min((int(g) - want) % 2 ** 64, (want - int(g)) % 2 ** 64)
        assert off <= 2 + 2 * abs(float(turns)), (x, off)


def test_phases_refuse(lib):
    with pytest.raises(mfb.MapflowError):
        mfb.Rope.from_freqs([1.0, float("inf")], device="cpu")
    assert lib.mf_rope_phases(None, 1, None) == BAD
    assert lib.mf_rope_phases(None, 0, None) == mfb.MF_OK
    assert lib.mf_rope_freqs(8, 1e4, 0, 1.0, 0.0, 1.0, 32.0, None) == BAD
    assert lib.mf_rope_freqs(8, 1e4, 9, 1.0, 0.0, 1.0, 32.0, P(16)) == BAD


# ------------------------------------------------------------- C ABI refusals

def rope_desc(**kw):
    return mfb.RopeDesc(*{**dict(rot_dim=64, interleaved=0, phases=256, scale=1.0), **kw}.values())


def batch(**kw):
    return mfb.TokenBatch(*{**dict(ntok=10, nseq=2, cu_seqlens=256, start=256), **kw}.values())


def cache(**kw):
    return mfb.KvCacheDesc(*{**dict(K=256, V=256, page_table=256, npages=8, page_size=16,
                                    max_pages_per_seq=4, nseq=2, Hkv=2, d=64, dt=mfb.MF_BF16),
                             **kw}.values())


def attn(**kw):
    return mfb.PagedAttnDesc(*{**dict(Hq=4, scale=0.125, band_bias=0.0, band_width=0, window=0,
                                      len_add=0), **kw}.values())


def call_rope(lib, r=None, b=None, d=64, dt=mfb.MF_BF16, Hq=4, Q=P(256), qs=256, Qo=P(256),
              qos=256, Hk=2, K=P(256), ks=128, Ko=P(256), kos=128):
    return lib.mf_rope(C.byref(r or rope_desc()), C.byref(b or batch()), d, dt, Hq, Q, qs, Qo, qos,
                       Hk, K, ks, Ko, kos, 0, None)


def call_append(lib, c=None, r=None, b=None, K=P(256), ks=128, V=P(256), vs=128, Hq=4, Q=P(256),
                qs=256, Qo=P(256), qos=256):
    return lib.mf_kv_append(C.byref(c or cache()), C.byref(r or rope_desc()),
                            C.byref(b or batch()), K, ks, V, vs, Hq, Q, qs, Qo, qos, None)


def call_attn(lib, c=None, a=None, lens=P(256), Q=P(256), qs=256, O=P(256), os_=256, ws=P(256),
              n=1 << 30):
    return lib.mf_paged_attn(C.byref(c or cache()), C.byref(a or attn()), lens, Q, qs, O, os_,
                             None, ws, n, None)


@needs_no_gpu
@pytest.mark.parametrize("kw,status", [
    (dict(r=rope_desc(rot_dim=0)), BAD), (dict(r=rope_desc(rot_dim=33)), BAD),
    (dict(r=rope_desc(rot_dim=66)), BAD), (dict(r=rope_desc(phases=None)), BAD),
    (dict(r=rope_desc(scale=float("inf"))), BAD), (dict(d=96), UNSUP), (dict(dt=7), BAD),
    (dict(b=batch(ntok=-1)), BAD), (dict(b=batch(nseq=0)), BAD),
    (dict(b=batch(cu_seqlens=None)), BAD), (dict(b=batch(ntok=1 << 31)), UNSUP),
    (dict(Hq=0), BAD), (dict(Hk=-1), BAD), (dict(Q=None), BAD), (dict(Qo=None), BAD),
    (dict(K=None), BAD), (dict(qs=255), BAD), (dict(qos=255), BAD), (dict(ks=127), BAD),
    (dict(kos=-1, Hk=2), BAD), (dict(Q=P(257)), BAD), (dict(Ko=P(257)), BAD),
])
def test_rope_refuses(lib, kw, status):
    assert call_rope(lib, **kw) == status and lib.mf_last_error().decode()


@needs_no_gpu
def test_rope_of_no_tokens_is_a_no_op(lib):
    b = batch(ntok=0, nseq=0)
    assert call_rope(lib, b=b, Q=None, Qo=None, K=None, Ko=None) == mfb.MF_OK
    assert lib.mf_rope(None, C.byref(b), 64, 0, 1, None, 64, None, 64, 0, None, 0, None, 0, 0,
                       None) == BAD
    assert lib.mf_rope(C.byref(rope_desc()), None, 64, 0, 1, None, 64, None, 64, 0, None, 0, None,
                       0, 0, None) == BAD


CACHE_REFUSALS = [
    (dict(dt=3), BAD), (dict(d=96), UNSUP), (dict(nseq=-1), BAD), (dict(Hkv=0), BAD),
    (dict(Hkv=257), UNSUP), (dict(npages=-1), BAD), (dict(max_pages_per_seq=-1), BAD),
    (dict(page_size=8), BAD), (dict(page_size=24), BAD), (dict(npages=1 << 28), UNSUP),
    (dict(max_pages_per_seq=1 << 27), UNSUP), (dict(K=None), BAD), (dict(V=None), BAD),
    (dict(page_table=None), BAD), (dict(K=264), BAD), (dict(V=258), BAD),
]


@needs_no_gpu
@pytest.mark.parametrize("kw,status", CACHE_REFUSALS)
def test_cache_refusals(lib, kw, status):
    c = cache(**kw)
    assert call_append(lib, c=c) == status and lib.mf_last_error().decode()
    assert call_attn(lib, c=c, a=attn(Hq=1028 if kw.get("Hkv") == 257 else 4)) == status
    assert lib.mf_paged_attn_workspace(C.byref(c), C.byref(attn())) == 0


@needs_no_gpu
@pytest.mark.parametrize("kw,status", [
    (dict(r=rope_desc(rot_dim=66)), BAD), (dict(b=batch(nseq=3)), BAD),
    (dict(b=batch(ntok=3, cu_seqlens=None)), BAD), (dict(K=None), BAD), (dict(V=None), BAD),
    (dict(ks=127), BAD), (dict(vs=0), BAD), (dict(Hq=-1), BAD), (dict(Q=None), BAD),
    (dict(Qo=None), BAD), (dict(qs=100), BAD), (dict(V=P(257)), BAD),
])
def test_append_refuses(lib, kw, status):
    assert call_append(lib, **kw) == status and lib.mf_last_error().decode()


@needs_no_gpu
def test_append_of_no_tokens_is_a_no_op_and_valid_calls_reach_the_device(lib):
    assert call_append(lib, c=cache(nseq=0), b=batch(ntok=0, nseq=0), K=None, V=None, Q=None,
                       Qo=None) == mfb.MF_OK
    assert call_append(lib) == NOGPU
    assert call_append(lib, Hq=0, Q=None, Qo=None) == NOGPU
    assert lib.mf_kv_append(None, None, C.byref(batch()), P(256), 128, P(256), 128, 0, None, 0,
                            None, 0, None) == BAD


@needs_no_gpu
@pytest.mark.parametrize("kw,status", [
    (dict(a=attn(Hq=0)), BAD), (dict(a=attn(Hq=5)), BAD), (dict(a=attn(Hq=258)), UNSUP),
    (dict(a=attn(scale=float("nan"))), BAD), (dict(a=attn(band_bias=float("inf"))), BAD),
    (dict(a=attn(band_width=-1)), BAD), (dict(a=attn(window=-1)), BAD), (dict(lens=None), BAD),
    (dict(Q=None), BAD), (dict(O=None), BAD), (dict(qs=255), BAD), (dict(os_=248), BAD),
    (dict(qs=257), BAD), (dict(Q=P(264)), BAD), (dict(O=P(258)), BAD), (dict(ws=None), WS),
    (dict(ws=P(128)), WS), (dict(n=10), WS),
])
def test_attention_refuses(lib, kw, status):
    assert call_attn(lib, **kw) == status and lib.mf_last_error().decode()


@needs_no_gpu
def test_attention_of_no_sequences_is_a_no_op(lib):
    assert call_attn(lib, c=cache(nseq=0), lens=None, Q=None, O=None) == mfb.MF_OK
    assert lib.mf_paged_attn(None, C.byref(attn()), *[P(256)] * 2, 256, P(256), 256, None, P(256),
                             1 << 30, None) == BAD
    assert lib.mf_paged_attn(C.byref(cache()), None, *[P(256)] * 2, 256, P(256), 256, None,
                             P(256), 1 << 30, None) == BAD


# ------------------------------------------------------------- binding refusals

def host_cache(nseq=2, maxp=3, dtype=torch.float32):
    return mfb.KVCache.make(6, 16, 2, 64, dtype, torch.zeros(nseq, maxp, dtype=torch.int32))


def refused(f, *a, **kw):
    with pytest.raises((mfb.MapflowError, ValueError)) as e:
        f(*a, **kw)
    assert str(e.value)


def test_binding_refuses_wrong_tensors(lib):
    rp = mfb.Rope.make(64, device="cpu")
    Q, K = torch.zeros(5, 4, 64), torch.zeros(5, 2, 64)
    st = torch.zeros(5, dtype=torch.int32)
    refused(mfb.rope, rp, Q)                                  # neither start nor cu_seqlens
    refused(mfb.rope, rp, Q, start=st.long())                 # index type
    refused(mfb.rope, rp, Q, start=st[:4])                    # one position each
    refused(mfb.rope, rp, Q[:, :, ::2], start=st)             # dims not adjacent
    refused(mfb.rope, rp, Q.transpose(0, 1), start=st[:4])    # heads not d apart
    refused(mfb.rope, rp, Q, K.bfloat16(), start=st)          # mixed types
    refused(mfb.rope, rp, Q, K[:4], start=st)                 # token counts differ
    refused(mfb.rope, rp, Q, start=st, K_out=K)               # K_out without K
    refused(mfb.rope, rp, Q.half(), start=st)                 # a type without kernels
    refused(mfb.rope, rp, Q, start=st)                        # not on a GPU
    refused(mfb.Rope, torch.zeros(4))                         # phases are 64-bit integers
    c, lens = host_cache(), torch.zeros(2, dtype=torch.int32)
    refused(mfb.KVCache, c.K, c.V[:5], c.page_table)
    refused(mfb.KVCache, c.K.transpose(1, 2), c.V.transpose(1, 2), c.page_table)
    refused(mfb.KVCache, c.K, c.V, c.page_table.long())
    refused(mfb.kv_append, c, K[:2], K[:2, :1], lens)
    refused(mfb.kv_append, c, K[:2].bfloat16(), K[:2], lens)
    refused(mfb.kv_append, c, K[:2], K[:2], lens, Q_out=Q[:2])
    refused(mfb.kv_append, c, K[:2], K[:2], lens)             # not on a GPU
    refused(mfb.paged_attn, c, Q[:3], lens)
    refused(mfb.paged_attn, c, Q[:2].bfloat16(), lens)
    refused(mfb.paged_attn, c, Q[:2, :3], lens)               # 3 heads over 2 KV heads
    refused(mfb.paged_attn, c, Q[:2], lens[:1])
    refused(mfb.paged_attn, c, Q[:2], lens, lse=torch.zeros(2, 4))
    refused(mfb.paged_attn, c, Q[:2], lens)                   # not on a GPU


def test_copies_describe_their_own_tensors(lib):
    """A deep copy or an unpickled one is of its own pools and phases; the tensors a description
    was made of cannot be exchanged behind it."""
    c = mfb.KVCache.make(5, 16, 2, 64, torch.float32, torch.arange(6, dtype=torch.int32).view(2, 3))
    c.K.fill_(1.0)
    rp = mfb.Rope.make(64, interleaved=True, scale=0.5, device="cpu")
    for again in (copy.deepcopy, lambda x: pickle.loads(pickle.dumps(x))):
        k = again(c)
        d = k._desc
        assert (d.K, d.V, d.page_table) == tuple(x.data_ptr() for x in (k.K, k.V, k.page_table))
        assert d.K != c.K.data_ptr() and torch.equal(k.K, c.K) and d.npages == 5
        assert torch.equal(k.page_table, c.page_table)
        r = again(rp)
        assert r._desc.phases == r.phases.data_ptr() != rp.phases.data_ptr()
        assert torch.equal(r.phases, rp.phases) and r.interleaved and r.scale == 0.5
    assert copy.copy(c)._desc.K == c.K.data_ptr()
    for x, name in ((c, "K"), (c, "V"), (c, "page_table"), (rp, "phases"), (rp, "scale")):
        with pytest.raises(AttributeError):
            setattr(x, name, getattr(x, name))
