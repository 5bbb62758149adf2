"""The attention block's operators on measured cases: rotary positions, appending keys and values to a paged cache
(rotated on the way, the queries rotated in the same call), and attention of new tokens over the paged cache.

Shapes: head counts and widths of the layers that the workloads of this repository have linears for (hidden size 4096 as
32 heads of 128, 2048 as 16 of 128 or 8 of 256) and generic grouped-head ones. A batch is ragged: sequence b owns rows
cu_q[b] .. cu_q[b+1]-1 of the new tokens, and kv_lens[b] keys once these are in the cache; new token i of the sequence
sits at position kv_lens[b] - q_len[b] + i and sees the keys up to its own (the last `window` of them, where a window is
given). Pages are scattered over the cache at random.
"""

import math
import random

import numpy as np
import torch

own = False


# ------------------------------------------------------------------ cases
def _attn(name, batch, q, kv, hq, hkv, d, page, window=0, lse=False, mix=""):
    """mix: "" every sequence has q new tokens; "ragged" 1..q of them; "one" one sequence has q, the others one."""
    return {"name": name, "op": "attention", "batch": batch, "q": q, "kv": kv, "hq": hq, "hkv": hkv, "d": d, "page": page,
            "window": window, "lse": lse, "mix": mix}


def _append(name, batch, q, kv, hq, hkv, d, page, rotary, interleaved, mix=""):
    return {"name": name, "op": "append", "batch": batch, "q": q, "kv": kv, "hq": hq, "hkv": hkv, "d": d, "page": page,
            "rotary": rotary, "interleaved": interleaved, "mix": mix}


def _rope(name, tokens, heads, d, rotary, interleaved, scaled, far):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "d": d, "rotary": rotary, "interleaved": interleaved,
            "scaled": scaled, "far": far}


def listed():
    return [
        # one token of one request: latency
        _rope("rope_token", 1, 32, 128, 128, False, False, 4096),
        # a prompt's queries, half of each head rotated in interleaved pairs, scaled frequencies, far positions
        _rope("rope_prompt", 8191, 32, 128, 64, True, True, 131072),
        # one decode step of 64 requests
        _append("append_step", 64, 1, 8192, 32, 8, 128, 16, 128, False),
        # prompts of uneven length, together about 8K tokens, whole heads of 128
        _append("append_prompts", 5, 2600, 4096, 32, 8, 128, 64, 128, False, mix="ragged"),
        # one request's decode step on a short context: latency
        _attn("decode_one", 1, 1, 1000, 32, 8, 128, 16),
        # a serving batch's decode step, contexts up to 8K, ragged
        _attn("decode_batch", 64, 1, 8192, 32, 8, 128, 16),
        # one long context, no more: the split over the long axis; wide heads
        _attn("decode_long", 1, 1, 120001, 8, 4, 256, 64, lse=True),
        # a few draft tokens checked per request: 5 tokens x 8 heads a group
        _attn("draft_check", 24, 5, 4096, 32, 4, 128, 32, mix="ragged"),
        # a whole prompt of 8K tokens
        _attn("chunk_prompt", 1, 8192, 8192, 32, 8, 128, 64),
        # a chunk of a prompt beside decoding requests
        _attn("chunk_mixed", 17, 512, 8192, 32, 8, 128, 16, mix="one"),
        # a chunk in a sliding-window layer with wide heads
        _attn("chunk_window", 2, 2048, 8000, 8, 4, 256, 32, window=1024, lse=True, mix="ragged"),
        # one short odd prompt on small heads, no grouping
        _attn("chunk_small", 3, 333, 333, 16, 16, 64, 8, mix="ragged"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attention", "attention", "attention"])
    d = rng.choice([64, 128, 128, 256])
    page = rng.choice([8, 16, 16, 32, 64, 24])
    hkv, g = rng.choice([(8, 4), (4, 8), (8, 1), (2, 16), (5, 3), (4, 2), (1, 8), (2, 5)])
    if op == "rope":
        c = _rope("", _log(rng, 1, 8191), rng.choice([1, 8, 16, 32]), 128, rng.choice([32, 64, 128]), rng.random() < 0.5,
                  rng.random() < 0.5, _log(rng, 8192, 200000))
    elif op == "append":
        q = _log(rng, 1, 2048)
        kv = q + _log(rng, 1, 4000)
        most = max(1, min(4096 // q, 500000000 // (kv * hkv * d)))
        c = _append("", _log(rng, 1, most), q, kv, hkv * g, hkv, d, page, rng.choice([d, d // 2]), rng.random() < 0.5,
                    mix=rng.choice(["", "ragged", "one"]))
    else:
        kind = rng.choice(["decode", "draft", "chunk", "mixed"])
        window = rng.choice([0, 0, _log(rng, 16, 4096)])
        if kind == "decode":
            kv = _log(rng, 16, 65536)
            c = _attn("", max(1, min(128, _log(rng, 1, max(1, 7000000 // (kv * hkv * d // 64))))), 1, kv, hkv * g, hkv, d, page, window)
        elif kind == "draft":
            kv = _log(rng, 64, 8192)
            c = _attn("", _log(rng, 1, 24), rng.randint(2, 9), kv, hkv * g, hkv, d, page, window, mix="ragged")
        else:
            q = _log(rng, 10, 2000)
            kv = q + _log(rng, 1, 5000)
            most = max(1, min(16, int(1.3e11 / (q * kv * hkv * g * d))))
            c = _attn("", rng.randint(1, most), q, kv, hkv * g, hkv, d, page, window, mix="one" if kind == "mixed" else "ragged")
    del c["name"]
    return c


def _lens(case):
    """New tokens and keys of each sequence: by the case alone."""
    r = random.Random(case["batch"] * 1000003 + case["q"] * 1009 + case["kv"])
    q, kv = [], []
    for b in range(case["batch"]):
        n = case["q"]
        if case["mix"] == "one" and b != case["batch"] // 2:
            n = 1
        elif case["mix"] == "ragged" and case["batch"] > 1:
            n = r.randint(max(1, case["q"] // 4), case["q"])
        q.append(n)
        kv.append(case["kv"] if case["batch"] == 1 else r.randint(max(n, case["kv"] // 4), case["kv"]))
    return q, kv


# ------------------------------------------------------------------ inputs
def _inv_freq(rotary, scaled, device):
    """Frequencies of the rotated pairs, in radians a position; scaled: those of long wavelengths slowed 8 times, with a
    ramp between wavelengths 2048 and 8192."""
    f = 10000.0 ** (-np.arange(0, rotary, 2, dtype=np.float64) / rotary)
    if scaled:
        w = np.clip((2 * np.pi / f - 2048) / (8192 - 2048), 0.0, 1.0)
        f = f * (1 - w) + f / 8 * w
    return torch.from_numpy(f.astype(np.float32)).to(device)


def _paged(case, gen, device):
    """A cache with the pages of every sequence at random places, its table and the batch's offsets."""
    q, kv = _lens(case)
    page = case["page"]
    per = [-(-n // page) for n in kv]
    pages = sum(per) + 3
    perm = torch.randperm(pages, generator=gen, device=device).to(torch.int32)
    table = torch.full((len(kv), max(per)), -1, dtype=torch.int32, device=device)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = perm[at:at + n]
        at += n
    shape = (pages, page, case["hkv"], case["d"])
    cu = [0]
    for n in q:
        cu.append(cu[-1] + n)
    rows = [b for b, n in enumerate(q) for _ in range(n)]
    at = [i for n in q for i in range(n)]
    return {
        "k_cache": torch.randn(shape, generator=gen, device=device, dtype=torch.bfloat16),
        "v_cache": torch.randn(shape, generator=gen, device=device, dtype=torch.bfloat16),
        "page_table": table,
        "cu_q": torch.tensor(cu, dtype=torch.int32, device=device),
        "kv_lens": torch.tensor(kv, dtype=torch.int32, device=device),
        "max_q": max(q), "max_kv": max(kv),
        # for the plain form: the sequence of each row, its place in it, and its position
        "row_seq": torch.tensor(rows, device=device), "row_at": torch.tensor(at, device=device),
        "row_pos": torch.tensor([kv[b] - q[b] + i for b, i in zip(rows, at)], device=device),
        "tokens": len(rows),
    }


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    bf = {"generator": gen, "device": dev, "dtype": torch.bfloat16}
    s = {"case": case}
    if case["op"] == "rope":
        s["x"] = torch.randn((case["tokens"], case["heads"], case["d"]), **bf)
        s["positions"] = torch.randint(0, case["far"], (case["tokens"],), generator=gen, device=dev, dtype=torch.int32)
        s["inv_freq"] = _inv_freq(case["rotary"], case["scaled"], dev)
        return s
    s.update(_paged(case, gen, dev))
    s["q"] = torch.randn((s["tokens"], case["hq"], case["d"]), **bf)
    if case["op"] == "append":
        s["k"] = torch.randn((s["tokens"], case["hkv"], case["d"]), **bf)
        s["v"] = torch.randn((s["tokens"], case["hkv"], case["d"]), **bf)
        s["inv_freq"] = _inv_freq(case["rotary"], False, dev)
    else:
        s["q"] *= 1.5  # peaked enough that some keys matter more than others
    return s


# ------------------------------------------------------------------ plain forms
def _rotate(x, positions, inv_freq, interleaved):
    """x [T, H, D] with the first 2 * len(inv_freq) elements of each head rotated."""
    angle = positions.to(torch.float64)[:, None] * inv_freq.to(torch.float64)[None, :]
    c, s = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    n = inv_freq.numel()
    f = x.float()
    if interleaved:
        a, b = f[..., 0:2 * n:2], f[..., 1:2 * n:2]
        r = torch.stack((a * c - b * s, b * c + a * s), dim=-1).flatten(-2)
    else:
        a, b = f[..., :n], f[..., n:2 * n]
        r = torch.cat((a * c - b * s, b * c + a * s), dim=-1)
    return torch.cat((r, f[..., 2 * n:]), dim=-1).to(x.dtype)


def _plain_append(s):
    case = s["case"]
    q = _rotate(s["q"], s["row_pos"], s["inv_freq"], case["interleaved"])
    k = _rotate(s["k"], s["row_pos"], s["inv_freq"], case["interleaved"])
    page = s["page_table"][s["row_seq"], s["row_pos"] // case["page"]].long()
    at = s["row_pos"] % case["page"]
    s["k_cache"][page, at] = k
    s["v_cache"][page, at] = s["v"]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attention(s):
    """Padded to [batch, max_q] queries and [batch, max_kv] keys."""
    case = s["case"]
    b, hkv, d = case["batch"], case["hkv"], case["d"]
    g = case["hq"] // hkv
    q = torch.zeros((b, s["max_q"], hkv, g, d), dtype=torch.float32, device=s["q"].device)
    q[s["row_seq"], s["row_at"]] = s["q"].float().view(-1, hkv, g, d)
    table = s["page_table"].long().clamp(min=0)
    k = s["k_cache"][table].flatten(1, 2)[:, :s["max_kv"]].float()
    scores = torch.einsum("bqhgd,bkhd->bhgqk", q, k) * d ** -0.5
    del k
    position = torch.full((b, s["max_q"]), -1, dtype=torch.int64, device=q.device)
    position[s["row_seq"], s["row_at"]] = s["row_pos"]
    key = torch.arange(scores.shape[-1], device=q.device)
    seen = key[None, None, :] <= position[:, :, None]
    if case["window"]:
        seen &= key[None, None, :] > position[:, :, None] - case["window"]
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-3e38)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p /= total.clamp(min=1e-37)
    v = s["v_cache"][table].flatten(1, 2)[:, :s["max_kv"]].float()
    o = torch.einsum("bhgqk,bkhd->bqhgd", p, v)[s["row_seq"], s["row_at"]]
    out = {"out": o.reshape(-1, case["hq"], d).to(torch.bfloat16)}
    if case["lse"]:
        lse = (total.log() + top).squeeze(-1).permute(0, 3, 1, 2)
        out["lse"] = lse[s["row_seq"], s["row_at"]].reshape(-1, case["hq"])
    return out


# ------------------------------------------------------------------ one pass
def run(state):
    s, case = state, state["case"]
    if not own:
        if case["op"] == "rope":
            return {"y": _rotate(s["x"], s["positions"], s["inv_freq"], case["interleaved"])}
        return _plain_append(s) if case["op"] == "append" else _plain_attention(s)
    import fp8_w8a8_linear_b200 as f

    if case["op"] == "rope":
        return {"y": f.rope(s["x"], s["positions"], s["inv_freq"], interleaved=case["interleaved"])}
    if case["op"] == "append":
        q = f.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["cu_q"], s["kv_lens"],
                        inv_freq=s["inv_freq"], q=s["q"], interleaved=case["interleaved"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if "ws" not in s:  # a workspace, as a program keeps one for all of its layers
        s["ws"] = f.paged_attention_workspace(case["d"])
    lse = torch.empty((s["tokens"], case["hq"]), dtype=torch.float32, device=s["q"].device) if case["lse"] else None
    out = f.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["cu_q"], s["kv_lens"],
                            window=case["window"], max_q=s["max_q"], ws=s["ws"], lse=lse)
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    d = case["d"]
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 4 * n * d + 4 * case["tokens"] + 2 * case["rotary"], "flops": 3 * n * case["rotary"]}
    q, kv = _lens(case)
    tokens, batch = sum(q), case["batch"]
    if case["op"] == "append":
        heads = case["hq"] + 2 * case["hkv"]
        return {"bytes": 4 * tokens * heads * d + 8 * batch + 4 * tokens,
                "flops": 3 * tokens * (case["hq"] + case["hkv"]) * case["rotary"]}
    w = case["window"] or (1 << 40)
    keys = pairs = 0
    for n, m in zip(q, kv):
        first = m - n  # position of the first new token
        keys += m - max(0, first - w + 1)
        full = max(0, min(m, w) - first)  # rows that see all keys up to their own
        pairs += full * first + full * (full + 1) // 2 + (n - full) * w
    out = 4 * tokens * case["hq"] if case["lse"] else 0
    return {"bytes": 4 * tokens * case["hq"] * d + 4 * keys * case["hkv"] * d + out + 12 * batch,
            "flops": 4 * pairs * case["hq"] * d}


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _turned(x, positions, freq, interleaved):
    """Each pair as a complex number times exp(i p f)."""
    n = freq.numel()
    x = x.double()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), torch.outer(positions.double(), freq.double()))
    first, second = ((slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n)))
    z = torch.complex(x[..., first], x[..., second]) * turn[:, None]
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return {"y": _turned(s["x"], s["positions"], s["inv_freq"], case["interleaved"])}
    q_lens, kv_lens = _lens(case)
    page, g, at = case["page"], case["hq"] // case["hkv"], 0
    if case["op"] == "append":
        k_cache, v_cache, turned = s["k_cache"].double(), s["v_cache"].double(), []
        for b, (n, m) in enumerate(zip(q_lens, kv_lens)):
            rows, pos = slice(at, at + n), torch.arange(m - n, m, device=s["q"].device)
            slot = s["page_table"][b, pos // page].long() * page + pos % page
            turned.append(_turned(s["q"][rows], pos, s["inv_freq"], case["interleaved"]))
            k_cache.view(-1, case["hkv"], case["d"])[slot] = _turned(s["k"][rows], pos, s["inv_freq"], case["interleaved"])
            v_cache.view(-1, case["hkv"], case["d"])[slot] = s["v"][rows].double()
            at += n
        return {"q": torch.cat(turned), "k_cache": k_cache, "v_cache": v_cache}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=s["q"].device)
    for b, (n, m) in enumerate(zip(q_lens, kv_lens)):
        pages = s["page_table"][b, :-(-m // page)].long()
        k = s["k_cache"][pages].flatten(0, 1)[:m]
        v = s["v_cache"][pages].flatten(0, 1)[:m]
        behind = torch.arange(m - n, m, device=k.device)[:, None] - torch.arange(m, device=k.device)[None, :]
        hidden = behind < 0
        if case["window"]:
            hidden |= behind >= case["window"]
        for h in range(case["hkv"]):
            kh, vh = k[:, h].double(), v[:, h].double()
            for i in range(h * g, h * g + g):
                x = s["q"][at:at + n, i].double() @ kh.T / math.sqrt(case["d"])
                x[hidden] = -math.inf
                z = torch.logsumexp(x, -1)
                out[at:at + n, i] = torch.exp(x - z[:, None]) @ vh
                lse[at:at + n, i] = z
        at += n
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}
