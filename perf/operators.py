"""Measured cases of the serving operators: packed causal prefill attention and
the paged KV cache (append, decode attention, eviction by accumulated weight).

``run`` computes one pass of an operator, either in its plain form (elementary
torch operations in fp32) or, with ``own`` set, through the package's calls.
"""
from __future__ import annotations

import math
import random

import torch

own = False


# --------------------------------------------------------------------------- #
# cases
# --------------------------------------------------------------------------- #
def _prefill(lens_seed, batch, lo, hi, H, Hkv, d, q_rows=0):
    """batch sequences of lo..hi keys; q_rows = 0: every position is a query,
    else only the last q_rows positions are (a chunk of a longer prompt)."""
    return {"op": "prefill", "lens_seed": lens_seed, "batch": batch, "lo": lo, "hi": hi, "H": H, "Hkv": Hkv, "d": d,
            "q_rows": q_rows}


def _decode(lens_seed, batch, lo, hi, H, Hkv, d, page, weights):
    return {"op": "decode", "lens_seed": lens_seed, "batch": batch, "lo": lo, "hi": hi, "H": H, "Hkv": Hkv, "d": d,
            "page": page, "weights": weights}


def _append(lens_seed, batch, lo, hi, held, Hkv, d, page, keep):
    """Sequences that hold `held` entries get lo..hi tokens; keep = 0: all of
    them, else the `keep` selected ones of each KV head."""
    return {"op": "append", "lens_seed": lens_seed, "batch": batch, "lo": lo, "hi": hi, "held": held, "Hkv": Hkv,
            "d": d, "page": page, "keep": keep}


def _evict(lens_seed, batch, lo, hi, budget, recent, Hkv, d, page, step):
    """step: append one token, then evict back to the budget; else a cut of
    sequences of lo..hi entries down to the budget."""
    return {"op": "evict", "lens_seed": lens_seed, "batch": batch, "lo": lo, "hi": hi, "budget": budget,
            "recent": recent, "Hkv": Hkv, "d": d, "page": page, "step": step}


def listed():
    return [
        # a batch of short prompts on the small GQA layer: launch latency and raggedness
        {"name": "prefill short prompts", **_prefill(1, 16, 1, 512, 8, 2, 64)},
        # a serving batch of prompts of different lengths on the 32/8-head layer
        {"name": "prefill ragged batch", **_prefill(2, 8, 1024, 8192, 32, 8, 128)},
        # chunked prefill: the last 512 positions of four long prompts, 40/8 heads (groups of 5)
        {"name": "prefill chunk", **_prefill(3, 4, 8192, 32768, 40, 8, 128, 512)},
        # one long prompt
        {"name": "prefill 32K", **_prefill(4, 1, 32768, 32768, 32, 8, 128)},
        # one short sequence: the smallest decode step
        {"name": "decode short", **_decode(5, 1, 512, 512, 8, 2, 64, 16, False)},
        # a decode step of a ragged serving batch that also accumulates the attention weights
        {"name": "decode ragged batch", **_decode(6, 64, 1, 8192, 32, 8, 128, 16, True)},
        # decoding over caches compacted to a tenth of a 128K prompt, with weights for the eviction
        {"name": "decode compacted", **_decode(7, 8, 13107, 13107, 32, 8, 128, 64, True)},
        # one uncompressed 128K sequence, 40/8 heads
        {"name": "decode 128K", **_decode(8, 1, 131072, 131072, 40, 8, 128, 128, False)},
        # the new token of every sequence of a batch
        {"name": "append one token", **_append(9, 64, 1, 1, 1000, 8, 128, 16, 0)},
        # prompts compacted on their way into the cache: 1024 selected tokens per KV head
        {"name": "append selected", **_append(10, 8, 4096, 65536, 0, 8, 128, 64, 1024)},
        # a decode step's upkeep: one token in, one entry out, per KV head
        {"name": "evict one", **_evict(11, 64, 1024, 1024, 1024, 32, 8, 128, 16, True)},
        # a cut after the prompt: 32K entries down to 2048
        {"name": "evict to budget", **_evict(12, 4, 32768, 32768, 2048, 32, 8, 128, 64, False)},
    ]


def _spread(rng, lo, hi):
    """A whole number in lo..hi, spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    d = rng.choice((64, 128, 128))
    Hkv = rng.choice((1, 2, 3, 8))
    G = rng.choice((1, 2, 3, 4, 5, 7, 8))
    page = rng.choice((16, 32, 64, 128))
    seed = rng.randrange(1 << 20)
    op = rng.choice(("prefill", "decode", "append", "evict"))
    if op == "prefill":
        batch = _spread(rng, 1, 24)
        hi = _spread(rng, 8, 16384 // batch + 64)
        lo = rng.randint(1, hi)
        q_rows = rng.choice((0, 0, rng.randint(1, hi)))
        return _prefill(seed, batch, lo, hi, G * Hkv, Hkv, d, q_rows)
    if op == "decode":
        batch = _spread(rng, 1, 96)
        hi = _spread(rng, 16, max(17, 262144 // (batch * Hkv)))
        return _decode(seed, batch, rng.randint(1, hi), hi, G * Hkv, Hkv, d, page, rng.random() < 0.5)
    if op == "append":
        batch = _spread(rng, 1, 96)
        hi = _spread(rng, 1, 65536 // batch)
        keep = rng.choice((0, rng.randint(1, hi)))
        return _append(seed, batch, rng.randint(1, hi), hi, rng.randint(0, 300), Hkv, d, page, keep)
    batch = _spread(rng, 1, 48)
    budget = _spread(rng, 16, 131072 // (batch * 8))
    recent = rng.randint(0, budget // 4)
    if rng.random() < 0.5:
        return _evict(seed, batch, budget, budget, budget, recent, Hkv, d, page, True)
    hi = budget + _spread(rng, 1, 7 * budget)
    return _evict(seed, batch, rng.randint(max(1, budget // 2), hi), hi, budget, recent, Hkv, d, page, False)


def _lens(case):
    """The sequences' lengths: the longest given one first, the others spread."""
    r = random.Random(case["lens_seed"])
    lens = [_spread(r, case["lo"], case["hi"]) for _ in range(case["batch"])]
    lens[0] = case["hi"]
    r.shuffle(lens)
    return lens


def _q_lens(case, lens):
    return [min(n, case["q_rows"]) for n in lens] if case["q_rows"] else list(lens)


# --------------------------------------------------------------------------- #
# inputs
# --------------------------------------------------------------------------- #
def _cu(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def _qkv(g, n_q, n_k, H, Hkv, d, sinks):
    """bf16 queries, keys and values; the keys hold a few that every query of
    the group attends to (the sinks' rows and about one in 500 others)."""
    u = torch.randn(Hkv, d, generator=g, device="cuda")
    u /= u.norm(dim=1, keepdim=True)
    q = torch.randn(n_q, H, d, generator=g, device="cuda") + 2.0 * u.repeat_interleave(H // Hkv, 0)
    k = torch.randn(n_k, Hkv, d, generator=g, device="cuda")
    heavy = torch.rand(n_k, Hkv, generator=g, device="cuda") < 0.002
    if sinks is not None:
        heavy[sinks] = True
    k = torch.where(heavy[:, :, None], 2.0 * math.sqrt(d) * u + 0.1 * k, k)
    v = torch.randn(n_k, Hkv, d, generator=g, device="cuda")
    return q.bfloat16(), k.bfloat16(), v.bfloat16()


def _pages(g, case, lens, room):
    """A page pool with `lens` entries held per sequence and room for `room`
    more each, its pages in random order.  Entries are N(0, 1) with the heavy
    keys of _qkv; weights are what some steps of decoding leave behind."""
    B, Hkv, d, page = case["batch"], case["Hkv"], case["d"], case["page"]
    need = [-(-(n + room) // page) for n in lens]
    max_pages, num = max(need), sum(need) + 3
    order = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(B, max_pages, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    H = case.get("H", Hkv)
    q, k, v = _qkv(g, B, num * page, H, Hkv, d, None)
    k = k.view(num, page, Hkv, d).transpose(1, 2).contiguous()
    v = v.view(num, page, Hkv, d).transpose(1, 2).contiguous()
    weights = torch.rand(num, Hkv, page, generator=g, device="cuda").pow(4) * 3.0
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    pos = torch.zeros(num, Hkv, page, dtype=torch.int32, device="cuda")
    slot = torch.arange(max_pages * page, device="cuda", dtype=torch.int32)
    for b, n in enumerate(need):  # entry at slot s was token s
        pos[table[b, :n].long()] = slot[:n * page].view(n, 1, page).expand(n, Hkv, page)
    return {"q": q, "k_pages": k, "v_pages": v, "weights": weights, "pos": pos, "table": table,
            "seq_lens": lens_t, "next_pos": lens_t.clone(), "lens0": lens_t.clone(), "max_len": max(lens) + room}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    lens = _lens(case)
    B, Hkv, d = case["batch"], case["Hkv"], case["d"]
    s = {"case": dict(case), "lens": lens}
    if case["op"] == "prefill":
        ql = _q_lens(case, lens)
        s["q_lens"] = ql
        s["cu_q"], s["cu_k"] = _cu(ql), _cu(lens)
        s["q"], s["k"], s["v"] = _qkv(g, sum(ql), sum(lens), case["H"], Hkv, d, s["cu_k"][:-1].long())
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    elif case["op"] == "decode":
        s.update(_pages(g, case, lens, 1))
        s["out"] = torch.empty(B, case["H"], d, dtype=torch.float32, device="cuda")
        s["lse"] = torch.empty(B, case["H"], dtype=torch.float32, device="cuda")
    elif case["op"] == "append":
        kept = [min(n, case["keep"]) for n in lens] if case["keep"] else lens
        s.update(_pages(g, case, [case["held"]] * B, max(kept)))
        s["cu"], s["max_seqlen"] = _cu(lens), max(lens)
        _, s["k"], s["v"] = _qkv(g, 1, sum(lens), Hkv, Hkv, d, None)
        s["scores"] = s["idx"] = None
        if case["keep"]:
            s["scores"] = torch.rand(Hkv, sum(lens), generator=g, device="cuda").pow(6)
            idx = torch.full((B, Hkv, case["keep"]), -1, dtype=torch.int32, device="cuda")
            for b, n in enumerate(lens):
                pick = torch.rand(Hkv, n, generator=g, device="cuda").topk(kept[b], dim=1).indices
                idx[b, :, :kept[b]] = pick.sort(dim=1).values.to(torch.int32)
            s["idx"] = idx
    else:
        s.update(_pages(g, case, lens, 1))
        _, s["k"], s["v"] = _qkv(g, 1, B, Hkv, Hkv, d, None)
        s["weights0"], s["pos0"] = s["weights"].clone(), s["pos"].clone()
    return s


# --------------------------------------------------------------------------- #
# plain forms
# --------------------------------------------------------------------------- #
def _plain_prefill(s):
    c = s["case"]
    Hkv, G, d = c["Hkv"], c["H"] // c["Hkv"], c["d"]
    scale = 1.0 / math.sqrt(d)
    out, lse = s["out"], s["lse"]
    q0 = k0 = 0
    for lq, lk in zip(s["q_lens"], s["lens"]):
        k = s["k"][k0:k0 + lk].float().transpose(0, 1)  # [Hkv][lk][d]
        v = s["v"][k0:k0 + lk].float().transpose(0, 1)
        for r0 in range(0, lq, 1024):
            r1 = min(lq, r0 + 1024)
            end = r1 + lk - lq  # keys that the last of these rows sees
            q = s["q"][q0 + r0:q0 + r1].float().view(r1 - r0, Hkv, G, d).permute(1, 2, 0, 3).reshape(Hkv, -1, d)
            x = (q @ k[:, :end].transpose(1, 2)).view(Hkv, G, r1 - r0, end) * scale
            row = torch.arange(r0 + lk - lq, end, device="cuda")
            x.masked_fill_(torch.arange(end, device="cuda") > row[:, None], -math.inf)
            m = x.amax(-1, keepdim=True)
            x = (x - m).exp_()
            n = x.sum(-1, keepdim=True)
            o = (x.view(Hkv, -1, end) @ v[:, :end]).view(Hkv, G, r1 - r0, d) / n
            out[q0 + r0:q0 + r1] = o.permute(2, 0, 1, 3).reshape(r1 - r0, -1, d).to(out.dtype)
            lse[q0 + r0:q0 + r1] = (m + n.log()).squeeze(-1).permute(2, 0, 1).reshape(r1 - r0, -1)
        q0, k0 = q0 + lq, k0 + lk
    return {"out": out, "lse": lse}


def _plain_decode(s):
    c = s["case"]
    B, Hkv, G, d = c["batch"], c["Hkv"], c["H"] // c["Hkv"], c["d"]
    table = s["table"].long()
    L = table.shape[1] * c["page"]
    k = s["k_pages"][table].float().transpose(1, 2).reshape(B, Hkv, L, d)
    v = s["v_pages"][table].float().transpose(1, 2).reshape(B, Hkv, L, d)
    seen = (torch.arange(L, device="cuda") < s["seq_lens"][:, None])[:, None, None]
    x = (s["q"].float().view(B, Hkv, G, d) @ k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = (x - m).exp()
    n = p.sum(-1, keepdim=True)
    s["out"].copy_(((p @ v) / n).view(B, -1, d))
    s["lse"].copy_((m + n.log()).view(B, -1))
    if not c["weights"]:
        return {"out": s["out"], "lse": s["lse"]}
    w = (p / n).sum(2).view(B, Hkv, -1, c["page"]).transpose(1, 2)  # [B][pages][Hkv][page]
    s["weights"].index_put_((table.reshape(-1),), w.reshape(-1, Hkv, c["page"]), accumulate=True)
    return {"out": s["out"], "lse": s["lse"], "weights": s["weights"]}


def _plain_append(s, k, v, cu, idx, scores):
    """Writes tokens k, v of sequences cu (None: one each) behind what is held."""
    page, Hkv = s["case"]["page"], s["case"]["Hkv"]
    B, T = s["seq_lens"].numel(), k.shape[0]
    cu = torch.arange(B + 1, device="cuda") if cu is None else cu.long()
    n = cu[1:] - cu[:-1]
    if idx is None:
        b = torch.repeat_interleave(torch.arange(B, device="cuda"), n, output_size=T)
        r = torch.arange(T, device="cuda") - cu[b]
        t, head = torch.arange(T, device="cuda")[:, None], torch.arange(Hkv, device="cuda")[None]
        b, r, kept = b[:, None], r[:, None], n
    else:
        b, head, r = (idx >= 0).nonzero(as_tuple=True)
        t = cu[b] + idx[b, head, r].long()
        kept = n.clamp(max=idx.shape[2])
    slot = s["seq_lens"].long()[b] + r
    at = (s["table"][b, slot // page].long(), head, slot % page)
    s["k_pages"][at] = k[t, head]
    s["v_pages"][at] = v[t, head]
    s["pos"][at] = (s["next_pos"].long()[b] + t - cu[b]).to(torch.int32)
    s["weights"][at] = scores[head, t] if scores is not None else 0.0
    s["seq_lens"] += kept.to(torch.int32)
    s["next_pos"] += n.to(torch.int32)


def _plain_evict(s, budget, recent):
    page, Hkv = s["case"]["page"], s["case"]["Hkv"]
    table = s["table"].long()
    B, L = table.shape[0], table.shape[1] * page
    slot = torch.arange(L, device="cuda")
    held = (slot < s["seq_lens"][:, None])[:, None]  # [B][1][L]
    w = s["weights"][table].transpose(1, 2).reshape(B, Hkv, L)
    pos = s["pos"][table].transpose(1, 2).reshape(B, Hkv, L)
    w = w.masked_fill(pos >= (s["next_pos"] - recent)[:, None, None], math.inf).masked_fill(~held, -math.inf)
    order = w.sort(dim=2, descending=True, stable=True).indices
    kept = torch.zeros_like(w, dtype=torch.bool).scatter_(2, order[:, :, :budget], True) & held
    hole = (~kept & held & (slot < budget)).nonzero(as_tuple=True)
    move = (kept & (slot >= budget)).nonzero(as_tuple=True)
    to = (table[hole[0], hole[2] // page], hole[1], hole[2] % page)
    of = (table[move[0], move[2] // page], move[1], move[2] % page)
    for x in (s["k_pages"], s["v_pages"], s["weights"], s["pos"]):
        x[to] = x[of]
    s["seq_lens"].clamp_(max=budget)


def _restore(s):
    """The cache as the prompt left it: its lengths, weights and positions."""
    s["seq_lens"].copy_(s["lens0"])
    s["next_pos"].copy_(s["lens0"])
    if s["case"]["op"] != "append":
        s["weights"].copy_(s["weights0"])
        s["pos"].copy_(s["pos0"])


# --------------------------------------------------------------------------- #
# one pass
# --------------------------------------------------------------------------- #
def _cache(s):
    """The package's handle of the pages, made once, as a program keeps it."""
    if "cache" not in s:
        import long_context_kv_window_b200 as kvc

        s["kvc"] = kvc
        s["cache"] = kvc.PagedCache(s["k_pages"], s["v_pages"], s["table"], s["seq_lens"], weights=s["weights"],
                                    pos=s["pos"], next_pos=s["next_pos"])
    return s["kvc"], s["cache"]


def _pool(s):
    return {n: s[n] for n in ("k_pages", "v_pages", "weights", "pos", "seq_lens", "next_pos")}


def run(s):
    c = s["case"]
    if c["op"] == "prefill":
        if not own:
            return _plain_prefill(s)
        import long_context_kv_window_b200 as kvc

        out, lse = kvc.kvc_prefill_attention_varlen(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], max(s["q_lens"]),
                                                    max(s["lens"]), out=s["out"], lse=s["lse"])
        return {"out": out, "lse": lse}
    if c["op"] == "decode":
        if not own:
            return _plain_decode(s)
        kvc, cache = _cache(s)
        out, lse = kvc.kvc_paged_decode_attention(s["q"], cache, max_len=s["max_len"], accumulate=c["weights"],
                                                  out=s["out"], lse=s["lse"])
        return {"out": out, "lse": lse, "weights": s["weights"]} if c["weights"] else {"out": out, "lse": lse}
    if c["op"] == "append":
        _restore(s)  # the lengths go back first, so that every pass writes the same slots
        if not own:
            _plain_append(s, s["k"], s["v"], s["cu"], s["idx"], s["scores"])
        else:
            kvc, cache = _cache(s)
            kvc.kvc_paged_append(cache, s["k"], s["v"], s["cu"], s["max_seqlen"], idx=s["idx"], scores=s["scores"])
        return _pool(s)
    if not c["step"]:
        _restore(s)
    if not own:
        if c["step"]:
            _plain_append(s, s["k"], s["v"], None, None, None)
        _plain_evict(s, c["budget"], c["recent"])
    else:
        kvc, cache = _cache(s)
        if c["step"]:
            kvc.kvc_paged_append(cache, s["k"], s["v"])
        kvc.kvc_paged_evict(cache, c["budget"], c["recent"], max_len=s["max_len"])
    return _pool(s)


def work(case):
    lens = _lens(case)
    B, Hkv, d = case["batch"], case["Hkv"], case["d"]
    if case["op"] == "prefill":
        ql = _q_lens(case, lens)
        pairs = sum(q * (n - q) + q * (q + 1) // 2 for q, n in zip(ql, lens))
        return {"bytes": 2 * d * (2 * case["H"] * sum(ql) + 2 * Hkv * sum(lens)) + 4 * case["H"] * sum(ql),
                "flops": 4 * d * case["H"] * pairs}
    if case["op"] == "decode":
        entry = 4 * d + (8 if case["weights"] else 0)  # K and V, and the weight read and written
        return {"bytes": Hkv * sum(lens) * entry + B * case["H"] * (6 * d + 4),
                "flops": 4 * d * case["H"] * sum(lens)}
    if case["op"] == "append":
        kept = sum(min(n, case["keep"]) for n in lens) if case["keep"] else sum(lens)
        entry = 2 * 4 * d + 8 + (8 if case["keep"] else 0)  # K and V in and out, position and weight, index and score
        return {"bytes": Hkv * kept * entry + 16 * B, "flops": 0}
    held = [n + 1 if case["step"] else n for n in lens]
    over = [n for n in held if n > case["budget"]]
    # kept entries behind the budget, if any entry is as likely kept as another
    moved = sum(case["budget"] * (n - case["budget"]) / n for n in over)
    row = 2 * (4 * d + 8)
    return {"bytes": Hkv * (8 * sum(over) + row * moved + (row * B if case["step"] else 0)) + 16 * B, "flops": 0}


# --------------------------------------------------------------------------- #
# the definitions in 64 bits
# --------------------------------------------------------------------------- #
def exact(case, seed):
    if case["op"] not in ("prefill", "decode"):
        return None  # copies, and a selection among given numbers
    s = prepare(case, seed)
    H, G, d = case["H"], case["H"] // case["Hkv"], case["d"]
    scale = 1.0 / math.sqrt(d)
    if case["op"] == "prefill":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
        qs, ks = s["cu_q"].tolist(), s["cu_k"].tolist()
        for b in range(case["batch"]):
            nq, nk = qs[b + 1] - qs[b], ks[b + 1] - ks[b]
            for h in range(H):
                k = s["k"][ks[b]:ks[b + 1], h // G].double()
                v = s["v"][ks[b]:ks[b + 1], h // G].double()
                for i in range(0, nq, 8192):
                    j = min(nq, i + 8192)
                    end = j + nk - nq
                    x = (s["q"][qs[b] + i:qs[b] + j, h].double() * scale) @ k[:end].T
                    x += torch.full_like(x, -math.inf).triu_(i + nk - nq + 1)
                    z = torch.logsumexp(x, 1)
                    lse[qs[b] + i:qs[b] + j, h] = z
                    out[qs[b] + i:qs[b] + j, h] = x.sub_(z[:, None]).exp_() @ v[:end]
        return {"out": out, "lse": lse}
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    weights = s["weights"].double()
    for b, n in enumerate(s["lens"]):
        pages = s["table"][b, :-(-n // case["page"])].long()
        for g in range(case["Hkv"]):
            k = s["k_pages"][pages, g].reshape(-1, d)[:n].double()
            v = s["v_pages"][pages, g].reshape(-1, d)[:n].double()
            x = scale * s["q"][b, g * G:(g + 1) * G].double() @ k.T
            z = x.logsumexp(1)
            p = (x - z[:, None]).exp()
            out[b, g * G:(g + 1) * G], lse[b, g * G:(g + 1) * G] = p @ v, z
            w = weights[pages, g].reshape(-1)
            w[:n] += p.sum(0)
            weights[pages, g] = w.view(-1, case["page"])
    return {"out": out, "lse": lse, "weights": weights} if case["weights"] else {"out": out, "lse": lse}
