"""What is measured of the serving-side operators: rotary positions (``mf.rope``), the append of
keys and values to a paged cache (``mf.kv_append``) and the attention of one new token over that
cache (``mf.paged_attn``).

``own`` false computes the plain form in elementary torch operations; true makes the calls a user
makes of the library.  Sizes are those of the framework's workloads (32 receiver heads over 8 KV
heads, 40 sender heads, 16-token pages, 32,768-token contexts, batches of 64 sequences with
log-uniform lengths in [1024, 16384], the float32 workload's 64-wide heads) and odd ones between.
"""
import math
import random

import torch

own = False

BF16, F32 = "bf16", "f32"
TYPES = {BF16: torch.bfloat16, F32: torch.float32}


# --------------------------------------------------------------------------- the cases

def listed():
    return [
        # a sender or receiver decoding one token of one sequence, far into a scaled context
        dict(name="rope_token", op="rope", seqs=1, lo=1, hi=1, start=30000, Hq=32, Hk=8, d=128,
             rot=128, dtype=BF16, interleaved=False, scaling="parts", backward=False, fused=True),
        # the 32K-token workload's sender layer: Q and K before the block statistics
        dict(name="rope_sender_32k", op="rope", seqs=1, lo=32768, hi=32768, start=0, Hq=40, Hk=40,
             d=128, rot=128, dtype=BF16, interleaved=False, scaling="none", backward=False,
             fused=False),
        # gradients of the rotated Q and K of a packed batch, float32 heads of 64
        dict(name="rope_grad_packed_f32", op="rope", seqs=13, lo=100, hi=2000, start=0, Hq=4, Hk=4,
             d=64, rot=64, dtype=F32, interleaved=True, scaling="linear", backward=True,
             fused=False),
        # a chunk of a batch whose sequences are already long; half of each head rotates
        dict(name="rope_chunk_partial", op="rope", seqs=7, lo=33, hi=1500, start=100000, Hq=32,
             Hk=8, d=128, rot=64, dtype=BF16, interleaved=True, scaling="ntk", backward=False,
             fused=True),
        # a decode step of 64 sequences: one new token each
        dict(name="append_token_64", op="append", seqs=64, lo=1, hi=1, past_lo=1024,
             past_hi=16383, Hq=32, Hkv=8, d=128, rot=128, page=16, dtype=BF16, interleaved=False,
             scaling="parts"),
        # prompts of a packed batch written to the cache, Q rotated in the same call
        dict(name="append_prompts", op="append", seqs=16, lo=1024, hi=16384, past_lo=0, past_hi=0,
             Hq=32, Hkv=8, d=128, rot=128, page=16, dtype=BF16, interleaved=False,
             scaling="none"),
        # chunks behind a cached prefix, float32, pages that the chunks begin and end inside
        dict(name="append_chunk_f32", op="append", seqs=5, lo=1, hi=700, past_lo=1, past_hi=999,
             Hq=4, Hkv=2, d=64, rot=32, page=48, dtype=F32, interleaved=True, scaling="linear"),
        # one token of one short sequence: latency
        dict(name="attn_token_1k", op="attn", seqs=1, lo=1009, hi=1009, Hq=32, Hkv=8, d=128,
             page=16, dtype=BF16, band=0, bias=0.0, window=0),
        # one token behind the 32K-token context
        dict(name="attn_token_32k", op="attn", seqs=1, lo=32768, hi=32768, Hq=32, Hkv=8, d=128,
             page=16, dtype=BF16, band=256, bias=2.0, window=0),
        # a decode step of the varlen batch: 64 sequences, log-uniform lengths
        dict(name="attn_varlen_64", op="attn", seqs=64, lo=1024, hi=16384, Hq=32, Hkv=8, d=128,
             page=16, dtype=BF16, band=0, bias=0.0, window=0),
        # few KV heads (16 query heads each), a sliding window, longer pages
        dict(name="attn_window_g16", op="attn", seqs=24, lo=1, hi=20000, Hq=32, Hkv=2, d=128,
             page=64, dtype=BF16, band=0, bias=0.0, window=4096),
        # float32, 64-wide heads, ragged lengths with empty and one-token sequences among them
        dict(name="attn_odd_f32", op="attn", seqs=11, lo=0, hi=5001, Hq=8, Hkv=2, d=64, page=16,
             dtype=F32, band=100, bias=2.0, window=0),
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], uniform over the logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn"])
    dtype = rng.choice([BF16, BF16, F32])
    d = rng.choice([64, 128])
    scaling = rng.choice(["none", "linear", "ntk", "parts"])
    interleaved = rng.choice([False, True])
    rot = rng.choice([d, d, d // 2, d // 4])
    if op == "rope":
        seqs = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, max(1, 16000 // seqs))
        Hq, Hk = rng.choice([(32, 8), (40, 40), (4, 4), (2, 2), (12, 3), (32, 0)])
        return dict(op=op, seqs=seqs, lo=max(1, hi // 7), hi=hi, start=rng.choice([0, 5, 77777]),
                    Hq=Hq, Hk=Hk, d=d, rot=rot, dtype=dtype, interleaved=interleaved,
                    scaling=scaling, backward=rng.choice([False, False, True]),
                    fused=rng.choice([False, True]))
    Hq, Hkv = rng.choice([(32, 8), (32, 4), (32, 16), (8, 8), (4, 2), (16, 1), (12, 4), (40, 2)])
    page = rng.choice([16, 16, 32, 48, 64, 128])
    if op == "append":
        seqs = _log_int(rng, 1, 64)
        hi = rng.choice([1, _log_int(rng, 1, max(1, 16000 // seqs))])
        past = _log_int(rng, 1, 4000)
        return dict(op=op, seqs=seqs, lo=max(1, hi // 7), hi=hi, past_lo=past // 3, past_hi=past,
                    Hq=Hq, Hkv=Hkv, d=d, rot=rot, page=page, dtype=dtype,
                    interleaved=interleaved, scaling=scaling)
    seqs = _log_int(rng, 1, 64)
    hi = _log_int(rng, 1, min(32768, 100000 // seqs))
    return dict(op=op, seqs=seqs, lo=hi // 9, hi=hi, Hq=Hq, Hkv=Hkv, d=d, page=page, dtype=dtype,
                band=rng.choice([0, 0, 256, 17]), bias=2.0, window=rng.choice([0, 0, 0, 1000]))


def _lengths(case, lo, hi, salt):
    """Ragged lengths of a case's sequences (of the case alone, so that work() knows them too)."""
    rng = random.Random(1000 * case["seqs"] + 7 * hi + salt)
    out = [_log_int(rng, max(lo, 1), max(hi, 1)) if hi > lo else hi for _ in range(case["seqs"])]
    if lo == 0 and hi > 0 and case["seqs"] > 2:
        out[1], out[2] = 0, 1
    return out


def _new(case):
    return _lengths(case, case["lo"], case["hi"], 1)


def _past(case):
    return _lengths(case, case["past_lo"], case["past_hi"], 2)


# --------------------------------------------------------------------------- inputs

def _frequencies(case):
    """Inverse frequencies of the pairs (float64, host), scaled for a context 8 times as long."""
    r, base, c = case["rot"], 10000.0, 8.0
    if case["scaling"] == "ntk" and r > 2:
        base *= c ** (r / (r - 2.0))
    f = base ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    if case["scaling"] == "linear":
        f = f / c
    if case["scaling"] == "parts":
        turns = 4096.0 * f / (2 * math.pi)
        g = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        f = (1 - g) * f / c + g * f
    return f, (0.1 * math.log(c) + 1.0 if case["scaling"] == "parts" else 1.0)


def _cu(lengths):
    c = [0]
    for n in lengths:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device="cuda")


def _pages(case, lengths, g):
    """A page table over a pool a little larger than needed: pages in random order, -1 where unused."""
    ps = case["page"]
    need = [-(-n // ps) for n in lengths]
    npages, width = sum(need) + 3, max(need + [1])
    order = torch.randperm(npages, generator=g, device="cuda").to(torch.int32)
    at = torch.full((len(lengths), width), -1, dtype=torch.int32, device="cuda")
    k = 0
    for s, n in enumerate(need):
        at[s, :n] = order[k:k + n]
        k += n
    return at, npages


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    dt, d = TYPES[case["dtype"]], case["d"]
    rand = lambda *shape, gain=1.5: torch.empty(shape, device="cuda").normal_(  # noqa: E731
        std=gain, generator=g).to(dt)
    s = dict(case=case)
    if case["op"] != "attn":
        f, scale = _frequencies(case)
        s["inv_freq"], s["scale"] = f.cuda(), scale
        if own:  # the handle that a user's program makes once
            from cross_model_attention_block_b200 import mapflow as mf
            s["rope"] = mf.Rope.from_freqs(f.numpy(), interleaved=case["interleaved"], scale=scale)
    if case["op"] == "rope":
        n = _new(case)
        ntok, Hq, Hk = sum(n), case["Hq"], case["Hk"]
        s["cu"] = _cu(n)
        s["start"] = torch.randint(case["start"] // 2, case["start"] + 1, (len(n),), generator=g,
                                   device="cuda", dtype=torch.int32)
        if case["fused"]:  # slices of one projection's output
            x = rand(ntok, Hq + 2 * Hk, d)
            s["Q"], s["K"] = x[:, :Hq], x[:, Hq:Hq + Hk]
        else:
            s["Q"], s["K"] = rand(ntok, Hq, d), rand(ntok, Hk, d)
        return s
    Hq, Hkv = case["Hq"], case["Hkv"]
    if case["op"] == "append":
        n, past = _new(case), _past(case)
        s["cu"] = _cu(n)
        s["lens"] = torch.tensor(past, dtype=torch.int32, device="cuda")
        s["table"], npages = _pages(case, [a + b for a, b in zip(n, past)], g)
        x = rand(sum(n), Hq + 2 * Hkv, d)
        s["Q"], s["K"], s["V"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    else:
        n = _new(case)
        s["lens"] = torch.tensor(n, dtype=torch.int32, device="cuda")
        s["table"], npages = _pages(case, n, g)
        s["Q"] = rand(len(n), Hq, d)
    s["K_pool"] = rand(npages, case["page"], Hkv, d)
    s["V_pool"] = rand(npages, case["page"], Hkv, d, gain=1.0)
    return s


# --------------------------------------------------------------------------- one pass

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _rope_own(s):
    from cross_model_attention_block_b200 import mapflow as mf
    K = s["K"] if s["case"]["Hk"] else None
    out = mf.rope(s["rope"], s["Q"], K, start=s["start"], cu_seqlens=s["cu"],
                  backward=s["case"]["backward"])
    return {"Q": out[0], "K": out[1]} if s["case"]["Hk"] else {"Q": out}


def _append_own(s):
    from cross_model_attention_block_b200 import mapflow as mf
    cache = mf.KVCache(s["K_pool"], s["V_pool"], s["table"])
    one = s["case"]["hi"] == 1
    Q = mf.kv_append(cache, s["K"], s["V"], s["lens"], rope=s["rope"], Q=s["Q"],
                     cu_seqlens=None if one else s["cu"])
    return {"Q": Q, "K_pool": s["K_pool"], "V_pool": s["V_pool"]}


def _attn_own(s):
    from cross_model_attention_block_b200 import mapflow as mf
    c = s["case"]
    cache = mf.KVCache(s["K_pool"], s["V_pool"], s["table"])
    O, lse = mf.paged_attn(cache, s["Q"], s["lens"], band_bias=c["bias"], band_width=c["band"],
                           window=c["window"])
    return {"O": O, "lse": lse}


def _rotate(x, pos, s):
    """x [ntok, H, d] rotated by positions [ntok] (angles in 64 bits, the rest in 32)."""
    c = s["case"]
    r, sign = c["rot"], -1.0 if c.get("backward") else 1.0
    angle = pos.double()[:, None] * s["inv_freq"][None, :]
    cos = (angle.cos() * s["scale"]).float()[:, None, :]
    sin = (angle.sin() * (s["scale"] * sign)).float()[:, None, :]
    y = x.float()
    if c["interleaved"]:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    else:
        a, b = y[..., :r // 2], y[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    return torch.cat([turned, y[..., r:]], dim=-1).to(x.dtype)


def _places(cu, start, ntok):
    """Sequence and position of every packed token."""
    t = torch.arange(ntok, device=cu.device)
    seq = torch.searchsorted(cu[1:].long(), t, right=True)
    return seq, t - cu.long()[seq] + start.long()[seq]


def _rope_plain(s):
    _, pos = _places(s["cu"], s["start"], s["Q"].shape[0])
    out = {"Q": _rotate(s["Q"], pos, s)}
    if s["case"]["Hk"]:
        out["K"] = _rotate(s["K"], pos, s)
    return out


def _append_plain(s):
    ps = s["case"]["page"]
    seq, pos = _places(s["cu"], s["lens"], s["Q"].shape[0])
    page = s["table"].long()[seq, pos // ps]
    s["K_pool"][page, pos % ps] = _rotate(s["K"], pos, s)
    s["V_pool"][page, pos % ps] = s["V"]
    return {"Q": _rotate(s["Q"], pos, s), "K_pool": s["K_pool"], "V_pool": s["V_pool"]}


def _attn_plain(s):
    c = s["case"]
    n, Hkv, d, G = c["seqs"], c["Hkv"], c["d"], c["Hq"] // c["Hkv"]
    at = s["table"].clamp(min=0).long()
    K = s["K_pool"][at].view(n, -1, Hkv, d).permute(0, 2, 1, 3).float()   # [n, Hkv, L, d]
    V = s["V_pool"][at].view(n, -1, Hkv, d).permute(0, 2, 1, 3).float()
    q = s["Q"].view(n, Hkv, G, d).float()
    x = (q @ K.transpose(-1, -2)) * (1.0 / math.sqrt(d))                  # [n, Hkv, G, L]
    back = s["lens"].long()[:, None] - 1 - torch.arange(x.shape[-1], device=x.device)[None, :]
    x = x + (c["bias"] * ((back >= 0) & (back < c["band"])))[:, None, None, :]
    seen = (back >= 0) & (back < (c["window"] or 1 << 40))
    x = x.masked_fill(~seen[:, None, None, :], float("-inf"))
    m = x.amax(-1, keepdim=True)
    p = (x - m.clamp(min=-3e38)).exp()
    total = p.sum(-1, keepdim=True)
    O = (p @ V) / total.clamp(min=1e-38)
    lse = (m + total.log()).masked_fill(total == 0, float("-inf"))
    return {"O": O.view(n, c["Hq"], d).to(s["Q"].dtype), "lse": lse.view(n, c["Hq"]).t().contiguous()}


_own = {"rope": _rope_own, "append": _append_own, "attn": _attn_own}
_plain = {"rope": _rope_plain, "append": _append_plain, "attn": _attn_plain}


# --------------------------------------------------------------------------- work, exact

def work(case):
    e, d = (2 if case["dtype"] == BF16 else 4), case["d"]
    if case["op"] == "rope":
        n, H = sum(_new(case)), case["Hq"] + case["Hk"]
        return {"bytes": 2 * n * H * d * e, "flops": 3 * n * H * case["rot"]}
    if case["op"] == "append":
        n, Hq, Hkv = sum(_new(case)), case["Hq"], case["Hkv"]
        return {"bytes": 2 * n * (Hq + 2 * Hkv) * d * e + 8 * case["seqs"],
                "flops": 3 * n * (Hq + Hkv) * case["rot"]}
    w = case["window"]
    n = sum(min(x, w) if w else x for x in _new(case))
    io = case["seqs"] * case["Hq"] * (2 * d * e + 4) + 4 * (case["seqs"] + n // case["page"])
    return {"bytes": 2 * n * case["Hkv"] * d * e + io, "flops": 4 * n * case["Hq"] * d}


def exact(case, seed):
    """The definition in 64 bits, sequence by sequence."""
    s = prepare(case, seed)
    if case["op"] == "attn":
        return _attn_exact(case, s)
    turn = torch.polar(torch.tensor(s["scale"], dtype=torch.float64, device="cuda"),
                       torch.zeros((), dtype=torch.float64, device="cuda"))
    first = s["start"] if case["op"] == "rope" else s["lens"]
    first, n, f = first.tolist(), _new(case), s["inv_freq"]
    p = torch.cat([torch.arange(a, a + m, dtype=torch.float64) for a, m in zip(first, n)]).cuda()
    unit = turn * torch.polar(torch.ones_like(p)[:, None].expand(-1, len(f)), p[:, None] * f)
    if case.get("backward"):
        unit = unit.conj()

    def rotated(x):
        y, r = x.double().clone(), case["rot"]
        a, b = (slice(0, r, 2), slice(1, r, 2)) if case["interleaved"] else \
            (slice(0, r // 2), slice(r // 2, r))
        z = torch.complex(y[..., a], y[..., b]) * unit[:, None, :]
        y[..., a], y[..., b] = z.real, z.imag
        return y

    if case["op"] == "rope":
        return {"Q": rotated(s["Q"]), **({"K": rotated(s["K"])} if case["Hk"] else {})}
    K, V, kp, vp = rotated(s["K"]), s["V"].double(), s["K_pool"].double(), s["V_pool"].double()
    flat_k, flat_v, ps, t = kp.view(-1, *kp.shape[2:]), vp.view(-1, *vp.shape[2:]), case["page"], 0
    for i, (a, m) in enumerate(zip(first, n)):
        j = torch.arange(a, a + m, device="cuda")
        slot = s["table"][i].long()[torch.div(j, ps, rounding_mode="floor")] * ps + j % ps
        flat_k[slot], flat_v[slot] = K[t:t + m], V[t:t + m]
        t += m
    return {"Q": rotated(s["Q"]), "K_pool": kp, "V_pool": vp}


def _attn_exact(case, s):
    G, d, ps = case["Hq"] // case["Hkv"], case["d"], case["page"]
    O = torch.zeros(case["seqs"], case["Hq"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((case["Hq"], case["seqs"]), -math.inf, dtype=torch.float64, device="cuda")
    for i, L in enumerate(_new(case)):
        lo = max(0, L - case["window"]) if case["window"] else 0
        if L == 0:
            continue
        j = torch.arange(lo, L, device="cuda")
        slot = s["table"][i].long()[torch.div(j, ps, rounding_mode="floor")] * ps + j % ps
        K = s["K_pool"].view(-1, case["Hkv"], d)[slot].double()
        V = s["V_pool"].view(-1, case["Hkv"], d)[slot].double()
        for h in range(case["Hkv"]):
            q = s["Q"][i, h * G:(h + 1) * G].double()
            x = torch.mm(q, K[:, h].t()) / math.sqrt(d)
            x[:, max(0, len(j) - case["band"]):] += case["bias"] if case["band"] else 0.0
            lse[h * G:(h + 1) * G, i] = torch.logsumexp(x, 1)
            O[i, h * G:(h + 1) * G] = torch.mm(torch.softmax(x, 1), V[:, h])
    return {"O": O, "lse": lse}
