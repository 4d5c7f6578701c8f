"""The prompt-attention and 4-bit-cache operators: real calls, their plain forms and their cost.

Five operators that a user of the tiered cache runs one after another: causal attention over
packed prompts, the attention weight each prompt token collects, the cache that holds keys and
values in 4 bits (written and read back), single-token attention over that cache, and the
eviction of all but the tokens of highest accumulated weight.

A 4-bit page holds 16 entries of one (sequence, kv head) unit in 20 D bytes, NG = D/32 groups:
K codes [16][4][NG] u32 (word (t, g), nibble j: element 32g + 8t + j), V codes [16][8][NG] u16
(half (r, g), nibble j: element 32g + 4r + j), K scales [16][NG] fp16, K zeros [16][NG] fp16,
V scales and V zeros [4][NG][2][2] fp16 at (t, g, hi, e) for entry i = 8 hi + 2 t + e. Per group
s = fp16(f32((max - min) / 15)), z = fp16(min), code = clamp(rint(f32(f32(x - z) / s)), 0, 15), 0 if s == 0.
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------


def listed():
    return [
        # a handful of very short requests that arrive together: launch latency counts
        dict(name="prompt_short", op="prompt", lens="5,33,1,64,17,2,48,30", Hq=8, Hkv=2, D=64, dtype="fp16"),
        # a serving batch: prompts of very different lengths, odd ones among them
        dict(name="prompt_ragged", op="prompt", lens="4001,129,2500,777,1,6143,1024,300", Hq=32, Hkv=8, D=128,
             dtype="bf16"),
        # one sequence of the 32K-context decode workload
        dict(name="prompt_long", op="prompt", lens="32768", Hq=32, Hkv=8, D=128, dtype="bf16"),
        # the weights of a batch of documents before their caches are cut down
        dict(name="mass_ragged", op="mass", lens="1500,333,4097,90", Hq=40, Hkv=8, D=128, dtype="fp16"),
        # the weights of one long prompt
        dict(name="mass_long", op="mass", lens="16384", Hq=32, Hkv=8, D=128, dtype="bf16"),
        # one decode step's new token per sequence
        dict(name="append_token", op="append", lens="1,1,1,1,1,1,1,1", held=2047, Hkv=8, D=128, dtype="bf16"),
        # a batch of prompts written to the 4-bit cache
        dict(name="append_prompt", op="append", lens="8192,4097,6001,1,12000,2477", held=0, Hkv=8, D=128,
             dtype="bf16"),
        # a single short conversation: latency
        dict(name="attend_small", op="attend", lens="509", Hq=8, Hkv=2, D=64, dtype="fp16", weigh=False),
        # a serving batch of very different context lengths, weights accumulated
        dict(name="attend_ragged", op="attend", lens="16000,31,8192,1,4095,12001,700,9000", Hq=40, Hkv=8, D=128,
             dtype="bf16", weigh=True),
        # the decode workload's batch of 32K contexts, weights accumulated
        dict(name="attend_long", op="attend", lens=",".join(["32768"] * 8), Hq=32, Hkv=8, D=128, dtype="bf16",
             weigh=True),
        # every sixteen decode steps: a full budget and sixteen new tokens, sixteen evicted
        dict(name="evict_step", op="evict", lens="2064,2064,2064,2064,2064,2064,2064,2064", budget=2048, recent=256,
             Hkv=8, D=128),
        # after the prompt: 32K contexts cut to 4K
        dict(name="evict_prompt", op="evict", lens=",".join(["32768"] * 8), budget=4096, recent=512, Hkv=8, D=128),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "mass", "append", "attend", "evict"])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    D = rng.choice([64, 128])
    c = dict(op=op, Hkv=Hkv, D=D)
    if op != "evict":
        c["dtype"] = rng.choice(["bf16", "fp16"])
    if op in ("prompt", "mass"):
        while G * Hkv > 40:
            G = max(1, G // 2)
        c["Hq"] = G * Hkv
        B = _spread(rng, 1, 24)
        top = _spread(rng, 8, 16000)
        lens, work = [], 0.0
        for _ in range(B):
            n = _spread(rng, max(1, top // 32), top)
            if work + float(n) * n * G * Hkv <= 16384.0 ** 2 * 32:
                work += float(n) * n * G * Hkv
                lens.append(n)
        lens = lens or [top // 2]
        if rng.random() < 0.3:
            lens.insert(rng.randrange(len(lens) + 1), 0)
    elif op == "append":
        B = _spread(rng, 1, 16)
        top = 1 if rng.random() < 0.25 else _spread(rng, 1, 8192)
        lens = [_spread(rng, max(1, top // 32), top) for _ in range(B)]
        while sum(lens) * Hkv * D > 32768 * 8 * 128:
            lens.pop()
        c["held"] = 0 if rng.random() < 0.3 else _spread(rng, 1, 4096)
    else:
        B = _spread(rng, 1, 16)
        top = _spread(rng, 16, 131072)
        lens, work = [], 0
        for _ in range(B):
            n = _spread(rng, max(1, top // 32), top)
            if (work + n) * Hkv * D <= 8 * 32768 * 8 * 128:
                work += n
                lens.append(n)
        if op == "attend":
            c["Hq"] = G * Hkv
            c["weigh"] = rng.random() < 0.6
            if rng.random() < 0.2:
                lens.insert(rng.randrange(len(lens) + 1), 0)
        else:
            c["budget"] = _spread(rng, 1, max(lens))
            c["recent"] = rng.randrange(0, c["budget"] + 1)
    c["lens"] = ",".join(str(n) for n in lens)
    return c


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


# ---------------------------------------------------------------------------------
# the plain 4-bit format
# ---------------------------------------------------------------------------------


def _quantise(x):
    """Codes [..., D] int64 and fp16 scales, zeros [..., D/32] of x [..., D]."""
    g = x.float().unflatten(-1, (-1, 32))
    mn, mx = g.amin(-1), g.amax(-1)
    s, z = ((mx - mn) / 15.0).half(), mn.half()
    sf, zf = s.float().unsqueeze(-1), z.float().unsqueeze(-1)
    q = torch.where(sf > 0, torch.round((g - zf) / torch.where(sf > 0, sf, torch.ones_like(sf))), torch.zeros_like(g))
    return q.clamp_(0, 15).flatten(-2).to(torch.uint8), s, z


def _values(codes, s, z):
    """The float32 values that codes [..., D] with scales and zeros [..., D/32] stand for."""
    return (codes.float().unflatten(-1, (-1, 32)) * s.float().unsqueeze(-1) + z.float().unsqueeze(-1)).flatten(-2)


def _order(D):
    """Where a page keeps what: for entry i, the bytes [16][20 D/16] of its K codes, V codes,
    K scales, K zeros, V scales, V zeros in the order of the elements and groups."""
    NG = D // 32
    idx = torch.empty(16, 20 * D // 16, dtype=torch.int64)
    for i in range(16):
        o = []
        for e in range(0, D, 2):  # K codes: element pairs in order
            g, t, j = e // 32, (e % 32) // 8, e % 8
            o.append(i * (D // 2) + (t * NG + g) * 4 + j // 2)
        for e in range(0, D, 2):
            g, r, j = e // 32, (e % 32) // 4, e % 4
            o.append(8 * D + i * (D // 2) + (r * NG + g) * 2 + j // 2)
        for part in (16, 17):
            o += [part * D + (i * NG + g) * 2 + b for g in range(NG) for b in (0, 1)]
        hi, t, e = i // 8, (i % 8) // 2, i % 2
        for part in (18, 19):
            o += [part * D + (((t * NG + g) * 2 + hi) * 2 + e) * 2 + b for g in range(NG) for b in (0, 1)]
        idx[i] = torch.tensor(o)
    return idx


def _pack(k, v):
    """Entry records [N][20 D/16] bytes of k, v [N][D], in the order of _order."""
    out = []
    meta = []
    for x in (k, v):
        c, s, z = _quantise(x)
        out.append(c[:, 0::2] | (c[:, 1::2] << 4))
        meta += [s.view(torch.uint8), z.view(torch.uint8)]
    return torch.cat(out + meta, 1)


def _unpack(rec, D):
    """Float32 values (k, v) [N][D] of entry records."""
    NG, h = D // 32, D // 2
    out = []
    for part in (0, 1):
        b = rec[:, part * h:(part + 1) * h]
        c = torch.stack([b & 15, b >> 4], -1).flatten(1)
        m = D + part * 4 * NG
        s = rec[:, m:m + 2 * NG].contiguous().view(torch.float16)
        z = rec[:, m + 2 * NG:m + 4 * NG].contiguous().view(torch.float16)
        out.append(_values(c, s, z))
    return out


def _slots(table, u, n, first=0):
    """Physical (page, slot) of entries first .. first + n - 1 of unit u."""
    i = torch.arange(first, first + n, device=table.device)
    return table[u, i // 16].long(), i % 16


def _put(pages, order, page, slot, rec):
    pages[page.unsqueeze(1), order[slot]] = rec


def _get(pages, order, page, slot):
    return pages[page.unsqueeze(1), order[slot]]


# ---------------------------------------------------------------------------------
# preparation
# ---------------------------------------------------------------------------------


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _tokens(gen, T, Hkv, D, dtype):
    """Keys or values [T][Hkv][D] with four outlier channels per kv head."""
    x = torch.randn((T, Hkv, D), generator=gen, device="cuda")
    ch = torch.rand((Hkv, D), generator=gen, device="cuda").argsort(1)[:, :4]
    gain = torch.ones((Hkv, D), device="cuda").scatter_(1, ch, 8.0)
    return (x * gain).to(dtype)


def _cu(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device="cuda")


def _empty_cache(gen, B, Hkv, D, capacity):
    """Buffers of a cache whose physical pages are scattered."""
    U, P = B * Hkv, max(1, -(-capacity // 16))
    perm = torch.rand(U * P, generator=gen, device="cuda").argsort().to(torch.int32)
    return dict(pages=torch.zeros((U * P, 20 * D), dtype=torch.uint8, device="cuda"),
                page_table=perm.view(U, P).contiguous(),
                counts=torch.zeros(U + B, dtype=torch.int32, device="cuda"),
                mass=torch.zeros((U * P, 16), device="cuda"),
                pos=torch.full((U * P, 16), -1, dtype=torch.int32, device="cuda"))


def _handle(buf, B, Hkv, D):
    from kv_cache_eviction_gqa_b200.binding import Int4Cache
    U, P = buf["page_table"].shape
    c = Int4Cache(B, Hkv, D, capacity=16 * P, device="cuda")
    for name in ("pages", "page_table", "counts", "mass", "pos"):
        getattr(c, name).copy_(buf[name])
    return c


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, lens, Hkv, D = case["op"], _lens(case), case["Hkv"], case["D"]
    B, T = len(lens), sum(lens)
    st = dict(op=op, lens=lens, B=B, T=T, Hkv=Hkv, D=D, dtype=_DT.get(case.get("dtype")))
    if op in ("prompt", "mass"):
        # a fused projection's output: queries, keys and values of a token side by side
        Hq = case["Hq"]
        qkv = torch.empty((T, Hq + 2 * Hkv, D), dtype=st["dtype"], device="cuda")
        qkv[:, :Hq] = _normal(gen, (T, Hq, D), st["dtype"])
        qkv[:, Hq:Hq + Hkv] = _tokens(gen, T, Hkv, D, st["dtype"])
        qkv[:, Hq + Hkv:] = _tokens(gen, T, Hkv, D, st["dtype"])
        st.update(Hq=Hq, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], cu=_cu(lens),
                  status=torch.zeros(2, dtype=torch.int32, device="cuda"))
        if op == "mass":
            st["lse"] = _plain_prompt(st, with_out=False)[1]
        return st
    U = B * Hkv
    if op == "append":
        held = case["held"]
        k, v = _tokens(gen, T, Hkv, D, st["dtype"]), _tokens(gen, T, Hkv, D, st["dtype"])
        buf = _empty_cache(gen, B, Hkv, D, held + max(lens))
        buf["counts"].fill_(held)
        st.update(k=k, v=v, cu=_cu(lens), held=held, new_mass=torch.rand((T, Hkv), generator=gen, device="cuda"),
                  first=torch.full((U,), held, dtype=torch.int32, device="cuda"))
    else:
        order = _order(D).cuda()
        buf = _empty_cache(gen, B, Hkv, D, max(lens) + (16 if op == "attend" else 0))
        for b, n in enumerate(lens):
            buf["counts"][U + b] = 2 * n
            if n == 0:
                continue
            k, v = _tokens(gen, n, Hkv, D, torch.bfloat16), _tokens(gen, n, Hkv, D, torch.bfloat16)
            for h in range(Hkv):
                u = b * Hkv + h
                buf["counts"][u] = n
                page, slot = _slots(buf["page_table"], u, n)
                _put(buf["pages"], order, page, slot, _pack(k[:, h], v[:, h]))
                # weights collected so far: heavy-tailed, with repeated values (zeros) among them
                w = torch.rand(n, generator=gen, device="cuda")
                buf["mass"][page, slot] = torch.where(w < 0.1, torch.zeros_like(w), w ** -0.5 - 1.0)
                # the entries that survived earlier evictions, in the order of their positions
                at = torch.rand(2 * n, generator=gen, device="cuda").argsort()[:n].sort().values
                buf["pos"][page, slot] = at.to(torch.int32)
        if op == "attend":
            st.update(Hq=case["Hq"], q=_normal(gen, (B, case["Hq"], D), st["dtype"]), weigh=case["weigh"])
        else:
            st.update(budget=case["budget"], recent=case["recent"])
            st["to"] = _empty_cache(gen, B, Hkv, D, case["budget"])
    st["buf"] = buf
    st["order"] = None if own else _order(D).cuda()
    if own:
        st["cache"] = _handle(buf, B, Hkv, D)
        if op == "evict":
            st["into"] = _handle(st["to"], B, Hkv, D)
            del st["to"]
        # what run restores before a pass is kept beside the cache
        st["buf"] = {n: buf[n] for n in ("counts", "mass")}
    return st


# ---------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------

_ROWS = 1024


def _plain_prompt(st, with_out=True):
    q, k, v, G, D = st["q"], st["k"], st["v"], st["Hq"] // st["Hkv"], st["D"]
    out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.empty(q.shape[:2], device=q.device)
    at = 0
    for n in st["lens"]:
        kf, vf = (x[at:at + n].float().transpose(0, 1) for x in (k, v))          # [Hkv][n][D]
        for r in range(0, n, _ROWS):
            m = min(_ROWS, n - r)
            qf = q[at + r:at + r + m].float().unflatten(1, (-1, G)).permute(1, 2, 0, 3).flatten(1, 2)
            s = qf @ kf[:, :r + m].transpose(1, 2) * (1.0 / math.sqrt(D))        # [Hkv][G m][r + m]
            row = torch.arange(r, r + m, device=q.device).repeat(G)
            s.masked_fill_(torch.arange(r + m, device=q.device) > row.unsqueeze(1), -math.inf)
            top = s.amax(-1, keepdim=True)
            e = torch.exp(s.sub_(top))
            l = e.sum(-1, keepdim=True)
            lse[at + r:at + r + m] = (top + torch.log(l)).view(-1, G, m).permute(2, 0, 1).flatten(1)
            if with_out:
                o = (e @ vf[:, :r + m]) / l
                out[at + r:at + r + m] = o.view(-1, G, m, D).permute(2, 0, 1, 3).flatten(1, 2).to(q.dtype)
        at += n
    return out, lse


def _plain_mass(st):
    q, k, lse, G, D = st["q"], st["k"], st["lse"], st["Hq"] // st["Hkv"], st["D"]
    mass = torch.zeros(k.shape[:2], device=q.device)
    at = 0
    for n in st["lens"]:
        kf = k[at:at + n].float().transpose(0, 1)
        for r in range(0, n, _ROWS):
            m = min(_ROWS, n - r)
            qf = q[at + r:at + r + m].float().unflatten(1, (-1, G)).permute(1, 2, 0, 3).flatten(1, 2)
            s = qf @ kf[:, :r + m].transpose(1, 2) * (1.0 / math.sqrt(D))
            row = torch.arange(r, r + m, device=q.device).repeat(G)
            s.masked_fill_(torch.arange(r + m, device=q.device) > row.unsqueeze(1), -math.inf)
            ls = lse[at + r:at + r + m].unflatten(1, (-1, G)).permute(1, 2, 0).flatten(1)
            mass[at:at + r + m] += torch.exp(s.sub_(ls.unsqueeze(-1))).sum(1).t()
        at += n
    return mass


def _plain_append(st):
    buf, Hkv, D, B = st["buf"], st["Hkv"], st["D"], st["B"]
    counts = buf["counts"].clone()
    rec = _pack(st["k"].flatten(0, 1), st["v"].flatten(0, 1)).view(st["T"], Hkv, -1)
    at = 0
    for b, n in enumerate(st["lens"]):
        for h in range(Hkv):
            u = b * Hkv + h
            page, slot = _slots(buf["page_table"], u, n, st["held"])
            _put(buf["pages"], st["order"], page, slot, rec[at:at + n, h])
            buf["mass"][page, slot] = st["new_mass"][at:at + n, h]
            buf["pos"][page, slot] = torch.arange(st["held"], st["held"] + n, device="cuda", dtype=torch.int32)
        counts[b * Hkv:(b + 1) * Hkv] += n
        counts[B * Hkv + b] += n
        at += n
    k, v = (x.view(st["T"], Hkv, D).to(st["dtype"]) for x in _unpack(rec.flatten(0, 1), D))
    return dict(k=k, v=v, counts=counts, mass=buf["mass"], pos=buf["pos"])


def _plain_attend(st):
    buf, Hkv, D, B, G = st["buf"], st["Hkv"], st["D"], st["B"], st["Hq"] // st["Hkv"]
    out = torch.zeros((B, st["Hq"], D), dtype=st["dtype"], device="cuda")
    mass = buf["mass"].clone() if st["weigh"] else None
    for b, n in enumerate(st["lens"]):
        for h in range(Hkv):
            if n == 0:
                continue
            page, slot = _slots(buf["page_table"], b * Hkv + h, n)
            k, v = _unpack(_get(buf["pages"], st["order"], page, slot), D)
            s = st["q"][b, h * G:(h + 1) * G].float() @ k.t() * (1.0 / math.sqrt(D))
            e = torch.exp(s - s.amax(-1, keepdim=True))
            p = e / e.sum(-1, keepdim=True)
            out[b, h * G:(h + 1) * G] = (p @ v).to(st["dtype"])
            if mass is not None:
                mass[page, slot] += p.sum(0)
    return (out, mass) if st["weigh"] else out


def _plain_evict(st):
    buf, to, Hkv, B = st["buf"], st["to"], st["Hkv"], st["B"]
    counts = torch.zeros_like(buf["counts"])
    counts[B * Hkv:] = buf["counts"][B * Hkv:]
    for b, n in enumerate(st["lens"]):
        for h in range(Hkv):
            u = b * Hkv + h
            page, slot = _slots(buf["page_table"], u, n)
            w, p = buf["mass"][page, slot], buf["pos"][page, slot]
            keep = torch.arange(n, device="cuda")
            if n > st["budget"]:
                newest = p >= buf["counts"][B * Hkv + b] - st["recent"]
                rank = torch.where(newest, torch.full_like(w, math.inf), w)
                keep = torch.sort(rank, descending=True, stable=True).indices[:st["budget"]].sort().values
            m = keep.numel()
            dp, ds = _slots(to["page_table"], u, m)
            _put(to["pages"], st["order"], dp, ds, _get(buf["pages"], st["order"], page[keep], slot[keep]))
            to["mass"][dp, ds] = w[keep]
            to["pos"][dp, ds] = p[keep]
            counts[u] = m
    return dict(pages=to["pages"], counts=counts, mass=to["mass"], pos=to["pos"])


# ---------------------------------------------------------------------------------
# a pass
# ---------------------------------------------------------------------------------


def run(st):
    op = st["op"]
    if not own:
        if op == "prompt":
            return _plain_prompt(st)
        return {"mass": _plain_mass, "append": _plain_append, "attend": _plain_attend, "evict": _plain_evict}[op](st)
    from kv_cache_eviction_gqa_b200 import binding as qe
    if op == "prompt":
        return qe.prompt_attend(st["q"], st["k"], st["v"], st["cu"], status=st["status"])[:2]
    if op == "mass":
        return qe.prompt_mass(st["q"], st["k"], st["lse"], st["cu"], status=st["status"])[0]
    cache = st["cache"]
    if op == "append":
        # the same tokens again: the counts go back to those before the call
        cache.counts.copy_(st["buf"]["counts"])
        cache.append(st["k"], st["v"], st["cu"], mass=st["new_mass"])
        k, v = cache.read(st["cu"], st["T"], first=st["first"], dtype=st["dtype"])
        return dict(k=k, v=v, counts=cache.counts, mass=cache.mass, pos=cache.pos)
    if op == "attend":
        if not st["weigh"]:
            return cache.attend(st["q"], accumulate=False)
        # the same step again: the weights go back to those before the call
        cache.mass.copy_(st["buf"]["mass"])
        return cache.attend(st["q"], accumulate=True), cache.mass
    into = st["into"]
    cache.evict(into, st["budget"], st["recent"])
    # the survivors' records move byte for byte
    return dict(pages=into.pages, counts=into.counts, mass=into.mass, pos=into.pos)


# ---------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------


def work(case):
    lens, Hkv, D = _lens(case), case["Hkv"], case["D"]
    T, B, op = sum(lens), len(lens), case["op"]
    rec = 20 * D // 16
    pairs = sum(n * (n + 1) / 2 for n in lens)
    if op == "prompt":
        return dict(bytes=T * (2 * case["Hq"] + 2 * Hkv) * D * 2 + T * case["Hq"] * 4,
                    flops=4.0 * D * case["Hq"] * pairs)
    if op == "mass":
        return dict(bytes=T * (case["Hq"] + Hkv) * D * 2 + T * case["Hq"] * 4 + T * Hkv * 4,
                    flops=2.0 * D * case["Hq"] * pairs)
    if op == "append":
        # tokens and weights in, entries out; entries in again and their values out
        return dict(bytes=T * Hkv * (8 * D + 2 * rec + 12), flops=8.0 * T * Hkv * 2 * D)
    if op == "attend":
        G = case["Hq"] // Hkv
        return dict(bytes=T * Hkv * (rec + (8 if case["weigh"] else 0)) + B * case["Hq"] * D * 4,
                    flops=4.0 * D * G * Hkv * T)
    kept = sum(min(n, case["budget"]) for n in lens)
    return dict(bytes=T * Hkv * 8 + kept * Hkv * (2 * rec + 8), flops=float(T * Hkv))


# ---------------------------------------------------------------------------------
# the definition in 64 bits, written apart from the plain forms
# ---------------------------------------------------------------------------------


def _pairs64(q, k, a, n, scale, r0, r1):
    """Causal scores in 64 bits of rows r0..r1 of the prompt at a: [heads][rows][r1]."""
    G = q.shape[1] // k.shape[1]
    kk = k[a:a + r1].double().repeat_interleave(G, dim=1)                        # [r1][Hq][D]
    s = torch.einsum("ihd,jhd->hij", q[a + r0:a + r1].double(), kk) * scale
    i = torch.arange(r0, r1, device=q.device)[:, None]
    j = torch.arange(r1, device=q.device)[None, :]
    return s, j <= i


def _exact_entries(pages, D, page, slot):
    """(k, v) [n][D] in 64 bits of entries at (page, slot), from the format's words."""
    NG = D // 32
    pg = pages[page]
    n = torch.arange(page.numel(), device=pages.device)
    dev = pages.device
    d = torch.arange(D, device=dev)
    g, w = d // 32, d % 32

    def half(base, idx):                                                          # fp16 at halfword index idx [n][D]
        b0 = pg[n[:, None], base + 2 * idx].int()
        b1 = pg[n[:, None], base + 2 * idx + 1].int()
        return (b0 | (b1 << 8)).to(torch.int16).view(torch.float16).double()

    kb = slot[:, None] * (D // 2) + ((w // 8) * NG + g) * 4 + (w % 8) // 2
    vb = 8 * D + slot[:, None] * (D // 2) + ((w // 4) * NG + g) * 2 + (w % 4) // 2
    kc = (pg[n[:, None], kb].int() >> (4 * (d % 2))) & 15
    vc = (pg[n[:, None], vb].int() >> (4 * (d % 2))) & 15
    mk = slot[:, None] * NG + g
    mv = ((((slot % 8) // 2)[:, None] * NG + g) * 2 + (slot // 8)[:, None]) * 2 + (slot % 2)[:, None]
    return (kc.double() * half(16 * D, mk) + half(17 * D, mk),
            vc.double() * half(18 * D, mv) + half(19 * D, mv))


def _exact_quantised(x):
    """Values of x [N][D] after quantisation: every step in 64 bits, rounded where the format rounds."""
    import numpy as np
    a = x.double().cpu().numpy().reshape(x.shape[0], -1, 32)
    lo, hi = a.min(2, keepdims=True), a.max(2, keepdims=True)
    f32 = lambda y: y.astype(np.float32).astype(np.float64)
    s = f32(f32(hi - lo) / 15.0).astype(np.float32).astype(np.float16).astype(np.float64)
    z = lo.astype(np.float16).astype(np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(s > 0, np.clip(np.rint(f32(f32(a - z) / s)), 0, 15), 0.0)
    return torch.from_numpy((c * s + z).reshape(x.shape)).to(x.device)


def exact(case, seed):
    global own
    kept_own, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept_own
    op, lens, Hkv, D = st["op"], st["lens"], st["Hkv"], st["D"]
    scale = 1.0 / math.sqrt(D)
    if op in ("prompt", "mass"):
        q, k, v, Hq = st["q"], st["k"], st["v"], st["Hq"]
        G = Hq // Hkv
        if sum(float(n) * n for n in lens) * Hq > 33000.0 ** 2 * 32:
            return None
        out = torch.empty(q.shape, dtype=torch.float64, device=q.device)
        lse = torch.empty(q.shape[:2], dtype=torch.float64, device=q.device)
        mass = torch.zeros((st["T"], Hkv), dtype=torch.float64, device=q.device)
        a = 0
        for n in lens:
            for r0 in range(0, n, 256):
                r1 = min(n, r0 + 256)
                s, see = _pairs64(q, k, a, n, scale, r0, r1)
                if op == "prompt":
                    lse[a + r0:a + r1] = torch.logsumexp(s.masked_fill(~see, -math.inf), -1).t()
                    p = torch.where(see, torch.exp(s - lse[a + r0:a + r1].t()[:, :, None]), 0.0)
                    vv = v[a:a + r1].double().repeat_interleave(G, dim=1)
                    out[a + r0:a + r1] = torch.einsum("hij,jhd->ihd", p, vv)
                else:
                    p = torch.where(see, torch.exp(s - st["lse"][a + r0:a + r1].double().t()[:, :, None]), 0.0)
                    mass[a:a + r1] += p.sum(1).view(Hkv, G, r1).sum(1).t()
            a += n
        return (out, lse) if op == "prompt" else mass
    buf, B = st["buf"], st["B"]
    if op == "append":
        mass, pos, counts = buf["mass"].clone(), buf["pos"].clone(), buf["counts"].clone()
        vals = [_exact_quantised(st[x].flatten(0, 1)).view(st["T"], Hkv, D) for x in ("k", "v")]
        a = 0
        for b, n in enumerate(lens):
            for h in range(Hkv):
                for_slot = torch.arange(n, device=mass.device) + int(counts[b * Hkv + h])
                pg = buf["page_table"][b * Hkv + h].long()[for_slot // 16]
                mass[pg, for_slot % 16] = st["new_mass"][a:a + n, h]
                pos[pg, for_slot % 16] = (torch.arange(n, device=mass.device) + int(buf["counts"][B * Hkv + b])).int()
                counts[b * Hkv + h] += n
            counts[B * Hkv + b] += n
            a += n
        return dict(k=vals[0], v=vals[1], counts=counts, mass=mass.double(), pos=pos)
    if op == "attend":
        G = st["Hq"] // Hkv
        out = torch.zeros((B, st["Hq"], D), dtype=torch.float64, device="cuda")
        mass = buf["mass"].double()
        for b, n in enumerate(lens):
            for h in range(Hkv):
                if n == 0:
                    continue
                at = torch.arange(n, device="cuda")
                pg = buf["page_table"][b * Hkv + h].long()[at // 16]
                k, v = _exact_entries(buf["pages"], D, pg, at % 16)
                p = torch.softmax(k @ st["q"][b, h * G:(h + 1) * G].double().t() * scale, 0)   # [n][G]
                out[b, h * G:(h + 1) * G] = p.t() @ v
                mass[pg, at % 16] += p.sum(1)
        return (out, mass) if st["weigh"] else out
    # eviction: an order on (newest, weight, lower index), cut at the budget
    to = st["to"]
    order = st["order"]
    counts = torch.zeros_like(buf["counts"])
    counts[B * Hkv:] = buf["counts"][B * Hkv:]
    for b, n in enumerate(lens):
        for h in range(Hkv):
            u = b * Hkv + h
            at = torch.arange(n, device="cuda")
            pg, sl = buf["page_table"][u].long()[at // 16], at % 16
            w, p = buf["mass"][pg, sl].double().cpu(), buf["pos"][pg, sl].cpu()
            cut = int(buf["counts"][B * Hkv + b]) - st["recent"]
            ranked = sorted(range(n), key=lambda i, w=w.tolist(), p=p.tolist(): (p[i] < cut, -w[i] if p[i] < cut else 0.0, i))
            keep = torch.tensor(sorted(ranked[:st["budget"]]), device="cuda")
            m = keep.numel()
            to_at = torch.arange(m, device="cuda")
            dp, ds = to["page_table"][u].long()[to_at // 16], to_at % 16
            to["pages"][dp.unsqueeze(1), order[ds]] = buf["pages"][pg[keep].unsqueeze(1), order[sl[keep]]]
            to["mass"][dp, ds] = buf["mass"][pg[keep], sl[keep]]
            to["pos"][dp, ds] = buf["pos"][pg[keep], sl[keep]]
            counts[u] = m
    return dict(pages=to["pages"], counts=counts, mass=to["mass"].double(), pos=to["pos"])
