"""The operators around a paged KV cache held in 4 bits: what is measured.

Four operators, in the order in which a decode step runs them:

* ``norm_rope``: RMS norm of every query and key head and the rotation by
  position, in one pass;
* ``cache``: quantising K/V rows to 4 bits as they are written into pages, and
  reading those tokens back in 16 bits;
* ``anchor``: dense decode attention over the 4-bit pages, with the
  probabilities pooled over each key head's query heads;
* ``reuse``: decode attention over selected tokens of the 4-bit pages.

A cache row (one token of one key head, K and V) has 160 bytes: 64 of K codes,
64 of V codes, and 16 bfloat16 numbers: K scales, K minima, V scales, V minima,
one per group of 32 channels.  A value is ``minimum + scale * code``.  The
codes are ordered as the attention's matrix fragments want them: see
``K_NIBBLE`` and ``V_NIBBLE``, the place of each channel's code in its row.
"""
from __future__ import annotations

import math

import torch

own = False

D = 128
GROUP = 32
ROW = 160
SCALE = 1.0 / math.sqrt(D)
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}

K_NIBBLE = [8 * (4 * ((c >> 3) & 3) + (c >> 5)) + (c & 7) for c in range(D)]
V_NIBBLE = [8 * (2 * ((c >> 2) & 7) + (c >> 6)) + 4 * ((c >> 5) & 1) + (c & 3) for c in range(D)]


def k_for_len(n):
    """Selected tokens of a context of n: a tenth, at least 128."""
    return min(max((n + 5) // 10, 128), n)


# ------------------------------------------------------------------ cases ----
def _list(text):
    """The whole numbers of a case's text: "4096 x 16" is 16 times 4096, "5, 17, 0" are three."""
    n, _, times = text.partition("x")
    return [int(n)] * int(times) if times else [int(x) for x in text.split(",")]


def _text(numbers):
    return ", ".join(str(n) for n in numbers)


def _ragged(rng, b, lo, hi):
    return [int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))) for _ in range(b)]


def listed():
    return [
        # one new token of each of 16 sequences (the 32K decode workload), norms as in Qwen3-8B
        {"name": "norm_rope_step_b16", "op": "norm_rope", "type": "bf16", "B": 16, "N": 1, "Hq": 32, "Hkv": 8,
         "norm": True, "interleaved": False, "pos": 32768},
        # a whole 16K prompt (the 16K prefill workload)
        {"name": "norm_rope_prompt_16k", "op": "norm_rope", "type": "bf16", "B": 1, "N": 16384, "Hq": 32, "Hkv": 8,
         "norm": True, "interleaved": False, "pos": 0},
        # odd prompts of a batch, far positions, neighbouring pairs, no norms (Llama-3.1-8B has none)
        {"name": "norm_rope_odd_f16", "op": "norm_rope", "type": "f16", "B": 3, "N": 2051, "Hq": 24, "Hkv": 6,
         "norm": False, "interleaved": True, "pos": 1000003},
        # the rows of one decode step appended to 16 sequences
        {"name": "cache_step_b16", "op": "cache", "type": "bf16", "Hkv": 8, "page": 64, "new": "1 x 16",
         "start": _text(32767 - 1000 * b for b in range(16))},
        # prompts of a batch written behind what is there, one of them short and one empty
        {"name": "cache_prompts_16k_f16", "op": "cache", "type": "f16", "Hkv": 8, "page": 48,
         "new": "16384, 9001, 0, 777", "start": "0, 130, 55, 16001"},
        # the smallest decode workload: one sequence of 4K
        {"name": "anchor_4k_b1", "op": "anchor", "type": "bf16", "Hq": 32, "Hkv": 8, "page": 64, "lens": "4096"},
        # the main decode workload: 16 sequences of 32K
        {"name": "anchor_32k_b16", "op": "anchor", "type": "bf16", "Hq": 32, "Hkv": 8, "page": 64,
         "lens": "32768 x 16"},
        # the long workload: 4 sequences of 128K
        {"name": "anchor_128k_b4", "op": "anchor", "type": "bf16", "Hq": 32, "Hkv": 8, "page": 128,
         "lens": "131072 x 4"},
        # lengths of every size at once, groups of 8 query heads, half precision
        {"name": "anchor_ragged_f16", "op": "anchor", "type": "f16", "Hq": 32, "Hkv": 4, "page": 16,
         "lens": "65536, 30001, 8191, 4097, 515, 17, 1, 0"},
        # one sequence of 4K, 410 tokens of it
        {"name": "reuse_4k_b1", "op": "reuse", "type": "bf16", "Hq": 32, "Hkv": 8, "page": 64, "lens": "4096"},
        # 16 sequences of 32K, a tenth of each
        {"name": "reuse_32k_b16", "op": "reuse", "type": "bf16", "Hq": 32, "Hkv": 8, "page": 64,
         "lens": "32768 x 16"},
        # a ragged batch of 8K to 64K, half precision
        {"name": "reuse_ragged_f16", "op": "reuse", "type": "f16", "Hq": 32, "Hkv": 8, "page": 16,
         "lens": _text(8192 + 2399 * b for b in range(24))},
    ]


def draw(rng):
    """One more case: sizes over their logarithm, bounded by the largest listed ones."""
    op = rng.choice(["norm_rope", "cache", "anchor", "reuse"])
    kind = rng.choice(["bf16", "f16"])
    hkv, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 4])
    if hkv <= 4 and rng.random() < 0.25:
        group = 8
    if op == "norm_rope":
        n = _ragged(rng, 1, 1, 16384)[0]
        return {"op": op, "type": kind, "B": rng.randint(1, max(1, min(16, 16384 // n))), "N": n, "Hq": hkv * group,
                "Hkv": hkv, "norm": rng.random() < 0.5, "interleaved": rng.random() < 0.5,
                "pos": rng.choice([0, rng.randint(1, 4000000)])}
    page = rng.choice([16, 32, 48, 64, 128])
    b = rng.randint(1, 16)
    if op == "cache":
        new = _ragged(rng, b, 1, 1 + 24000 // b)
        return {"op": op, "type": kind, "Hkv": hkv, "page": page, "new": _text(new),
                "start": _text(rng.randint(0, 2000) for _ in range(b))}
    lens = _ragged(rng, b, 1, rng.choice([4096, 32768]))
    if b > 1 and rng.random() < 0.3:
        lens[rng.randrange(b)] = 0
    return {"op": op, "type": kind, "Hq": hkv * group, "Hkv": hkv, "page": page, "lens": _text(lens)}


def work(case):
    op, hkv = case["op"], case["Hkv"]
    if op == "norm_rope":
        rows = case["B"] * case["N"] * (case["Hq"] + hkv)
        return {"bytes": rows * D * 4 + case["B"] * case["N"] * 4, "flops": rows * D * (7 if case["norm"] else 3)}
    if op == "cache":  # write: 16-bit rows in, cache rows out; read back: the other way
        rows = sum(_list(case["new"])) * hkv
        return {"bytes": 2 * rows * (ROW + 4 * D), "flops": rows * 2 * D * 6}
    hq, lens = case["Hq"], _list(case["lens"])
    heads = len(lens) * hq
    if op == "anchor":
        rows = sum(lens) * hkv
        return {"bytes": rows * (ROW + 4) + heads * (4 * D + 4), "flops": sum(lens) * hq * 4 * D}
    sel = sum(k_for_len(t) for t in lens)
    return {"bytes": sel * hkv * (ROW + 4) + heads * (4 * D + 4), "flops": sel * hq * 4 * D}


# ----------------------------------------------------------------- inputs ----
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _table(g, need, page):
    """Pages in random order for sequences of `need` tokens; unused entries are -1."""
    n = [(t + page - 1) // page for t in need]
    order = torch.randperm(sum(n) + 3, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(n), max(1, max(n))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(n):
        table[b, :c] = order[at:at + c]
        at += c
    return table, sum(n) + 3


def _fill(g, pages):
    """Pages of quantised rows: normal keys with a few strong channels, normal values."""
    strong = 1.0 + 3.0 * (torch.rand(pages.shape[1], 1, D, generator=g, device="cuda") < 0.06)
    for p in range(0, pages.shape[0], 4096):
        part = pages[p:p + 4096]
        k = _randn(g, *part.shape[:3], D) * strong
        part.copy_(_quantise(k, _randn(g, *part.shape[:3], D)))


def _queries(g, b, hq, dtype):
    return (1.5 * _randn(g, b, hq, D)).to(dtype)


def prepare(case, seed):
    g, dtype, op = _gen(seed), TYPES[case["type"]], case["op"]
    s = {"case": case, "op": op, "dtype": dtype, "Hkv": case["Hkv"]}
    if op == "norm_rope":
        b, n, hq, hkv = case["B"], case["N"], case["Hq"], case["Hkv"]
        qkv = _randn(g, b, n, (hq + 2 * hkv) * D).to(dtype)  # one row per token, as a projection leaves it
        s["q"] = qkv[..., :hq * D].view(b, n, hq, D)
        s["k"] = qkv[..., hq * D:(hq + hkv) * D].view(b, n, hkv, D)
        s["qw"] = (1 + 0.2 * _randn(g, D)).to(dtype) if case["norm"] else None
        s["kw"] = (1 + 0.2 * _randn(g, D)).to(dtype) if case["norm"] else None
        s["inv_freq"] = 500000.0 ** (-torch.arange(0, D, 2, dtype=torch.float32, device="cuda") / D)
        s["pos"] = (torch.arange(n, device="cuda") + case["pos"]).expand(b, n).to(torch.int32).contiguous()
        s["pos"] += torch.randint(0, 64, (b, 1), generator=g, device="cuda", dtype=torch.int32)
        s["q_out"] = torch.empty(b, hq, n, D, dtype=dtype, device="cuda")
        s["k_out"] = torch.empty(b, hkv, n, D, dtype=dtype, device="cuda")
        return s
    hkv, page = case["Hkv"], case["page"]
    s["page"] = page
    if op == "cache":
        new, start = _list(case["new"]), _list(case["start"])
        b, n = len(new), max(1, max(new))
        s["table"], pages = _table(g, [p + c for p, c in zip(start, new)], page)
        s["pages"] = torch.zeros(pages, hkv, page, ROW, dtype=torch.uint8, device="cuda")
        s["k"] = (_randn(g, b, hkv, n, D) * 2).to(dtype)
        s["v"] = _randn(g, b, n, hkv, D).to(dtype).transpose(1, 2)  # as a projection leaves it
        s["start"], s["new"] = _i32(start), _i32(new)
        s["k_out"] = torch.zeros(b, hkv, n, D, dtype=dtype, device="cuda")
        s["v_out"] = torch.zeros_like(s["k_out"])
        return s
    lens, hq = _list(case["lens"]), case["Hq"]
    b = len(lens)
    s["Hq"], s["len"], s["max_T"] = hq, _i32(lens), max(lens)
    s["table"], pages = _table(g, lens, page)
    s["pages"] = torch.empty(pages, hkv, page, ROW, dtype=torch.uint8, device="cuda")
    _fill(g, s["pages"])
    s["q"] = _queries(g, b, hq, dtype)
    s["out"] = torch.empty(b, hq, D, dtype=dtype, device="cuda")
    s["lse"] = torch.empty(b, hq, dtype=torch.float32, device="cuda")
    if op == "anchor":
        s["ld"] = (s["max_T"] + 3) // 4 * 4
        s["pooled"] = torch.zeros(b, hkv, s["ld"], dtype=torch.float32, device="cuda")
        return s
    ks = [k_for_len(t) for t in lens]
    s["idx"] = torch.full((b, hkv, max(1, max(ks))), -1, dtype=torch.int32, device="cuda")
    for i, (t, k) in enumerate(zip(lens, ks)):
        if k:
            pick = torch.rand(hkv, t, generator=g, device="cuda").argsort(dim=1)[:, :k]
            s["idx"][i, :, :k] = pick.sort(dim=1).values.to(torch.int32)
    s["idx_k"] = _i32(ks).repeat_interleave(hkv).contiguous()
    s["map"] = torch.randint(0, hkv, (hkv,), generator=g, device="cuda", dtype=torch.int32)
    return s


# ------------------------------------------------------------ plain forms ----
def _toward(x, up):
    """x (64 bits) as the nearest bfloat16 that is not below it (up) or not above it."""
    r = x.to(torch.float32).to(torch.bfloat16)
    wrong = r.double() < x if up else r.double() > x
    inf = torch.full_like(r, math.inf if up else -math.inf)
    return torch.where(wrong, torch.nextafter(r, inf), r)


def _codes(x):
    """Codes 0..15, scales and minima (bfloat16) of x [..., 128], by groups of 32; borders in 64 bits."""
    x = x.unflatten(-1, (D // GROUP, GROUP)).double()
    low = _toward(x.amin(-1), False)
    m = low.double()
    s = _toward((x.amax(-1) - m) / torch.full_like(m, 15.0), True)
    step = s.double().unsqueeze(-1)
    n = torch.where(step > 0, (x - m.unsqueeze(-1)) / step.clamp_min(1e-300), torch.zeros_like(x))
    return n.round().clamp(0, 15).to(torch.uint8).flatten(-2), s, low


def _pack(codes, place):
    """[..., 128] codes to 64 bytes, channel c at nibble place[c]."""
    at = torch.empty_like(codes)
    at[..., torch.tensor(place, device=codes.device)] = codes
    at = at.unflatten(-1, (D // 2, 2))
    return at[..., 0] | (at[..., 1] << 4)


def _quantise(k, v):
    """Cache rows uint8 [..., 160] of keys and values [..., 128]."""
    ck, sk, mk = _codes(k)
    cv, sv, mv = _codes(v)
    tail = torch.cat([sk, mk, sv, mv], dim=-1).contiguous().view(torch.uint8)
    return torch.cat([_pack(ck, K_NIBBLE), _pack(cv, V_NIBBLE), tail], dim=-1)


def _unpack(rows):
    """Keys and values fp32 [..., 128] of cache rows [..., 160]."""
    tail = rows[..., 128:].contiguous().view(torch.bfloat16).float().unflatten(-1, (4, D // GROUP))
    out = []
    for i, place in enumerate((K_NIBBLE, V_NIBBLE)):
        b = rows[..., 64 * i:64 * i + 64]
        n = torch.stack([b & 15, b >> 4], dim=-1).flatten(-2)[..., torch.tensor(place, device=b.device)]
        n = n.float().unflatten(-1, (D // GROUP, GROUP))
        out.append((tail[..., 2 * i + 1, :].unsqueeze(-1) + tail[..., 2 * i, :].unsqueeze(-1) * n).flatten(-2))
    return out


def _slots(table, page, t, there):
    """Page and slot of token t [B, n] of each sequence (page 0 where there is none)."""
    p = torch.gather(table.long(), 1, (t // page).clamp(0, table.shape[1] - 1))
    return torch.where(there, p, torch.zeros_like(p)), t % page


def _rows(pages, table, page, n):
    """Rows [B, Hkv, n, 160] of each sequence's first n tokens (page 0 where there is none)."""
    t = torch.arange(n, device=pages.device).expand(table.shape[0], n)
    p = torch.gather(table.long(), 1, t // page).clamp_min(0)
    return pages[p, :, t % page].transpose(1, 2)


def _plain_norm_rope(s):
    inter = s["case"]["interleaved"]
    a = s["pos"].double().unsqueeze(-1) * s["inv_freq"].double()
    cos, sin = a.cos().float().unsqueeze(2), a.sin().float().unsqueeze(2)

    def one(x, w):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
        if inter:
            a, b = y[..., 0::2], y[..., 1::2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        else:
            a, b = y[..., :D // 2], y[..., D // 2:]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
        return y.transpose(1, 2).to(x.dtype).contiguous()

    return {"q": one(s["q"], s["qw"]), "k": one(s["k"], s["kw"])}


def _plain_cache(s):
    n = s["k"].shape[2]
    i = torch.arange(n, device="cuda")
    there = i < s["new"].long().unsqueeze(1)
    page, slot = _slots(s["table"], s["page"], s["start"].long().unsqueeze(1) + i, there)
    rows = _quantise(s["k"].float(), s["v"].float()).transpose(1, 2)  # [B, n, Hkv, 160]
    s["pages"][page[there], :, slot[there]] = rows[there]
    k, v = _unpack(s["pages"][page, :, slot].transpose(1, 2))
    keep = there.unsqueeze(1).unsqueeze(-1)
    return {"k": torch.where(keep, k, torch.zeros_like(k)).to(s["dtype"]),
            "v": torch.where(keep, v, torch.zeros_like(v)).to(s["dtype"])}


def _attend(q, k, v, there):
    """q [B, Hkv, G, 128], k and v [B, Hkv, n, 128], there [B, 1 or Hkv, n]: outputs, log-sum-exp, probabilities."""
    x = torch.matmul(q, k.transpose(-1, -2)) * SCALE
    x = x.masked_fill(~there.unsqueeze(2), -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    some = total > 0
    p = torch.where(some, p / total.clamp_min(1e-30), torch.zeros_like(p))
    lse = torch.where(some, top + torch.log(total.clamp_min(1e-30)), torch.full_like(top, -math.inf))
    return torch.matmul(p, v), lse.squeeze(-1), p


def _plain_anchor(s):
    b, hkv, n = len(s["len"]), s["Hkv"], max(1, s["max_T"])
    k, v = _unpack(_rows(s["pages"], s["table"], s["page"], n))
    there = (torch.arange(n, device="cuda") < s["len"].unsqueeze(1)).unsqueeze(1)
    o, lse, p = _attend(s["q"].float().view(b, hkv, -1, D), k, v, there)
    pooled = torch.zeros(b, hkv, s["ld"], device="cuda")
    pooled[..., :n] = p.mean(2)
    return {"out": o.reshape(b, -1, D).to(s["dtype"]), "lse": lse.reshape(b, -1), "pooled": pooled}


def _plain_reuse(s):
    b, hkv = len(s["len"]), s["Hkv"]
    idx = s["idx"].long()[:, s["map"].long()]
    there = idx >= 0
    t = idx.clamp_min(0)
    seq = torch.arange(b, device="cuda").view(b, 1, 1)
    page = s["table"].long()[seq, t // s["page"]].clamp_min(0)
    head = torch.arange(hkv, device="cuda").view(1, hkv, 1)
    k, v = _unpack(s["pages"][page, head, t % s["page"]])
    o, lse, _ = _attend(s["q"].float().view(b, hkv, -1, D), k, v, there)
    return {"out": o.reshape(b, -1, D).to(s["dtype"]), "lse": lse.reshape(b, -1)}


# ------------------------------------------------------------- own kernels ----
def _own(s):
    from long_context_emitting_b200 import api

    if s["op"] == "norm_rope":
        q, k = api.qk_norm_rope(s["q"], s["k"], s["pos"], s["inv_freq"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS,
                                interleaved=s["case"]["interleaved"], q_out=s["q_out"], k_out=s["k_out"])
        return {"q": q, "k": k}
    if s["op"] == "cache":
        api.kv_write_paged_q4(s["k"], s["v"], s["pages"], s["table"], s["page"], s["start"], s["new"])
        k, v = api.kv_read_paged_q4(s["pages"], s["table"], s["page"], s["start"], s["new"], s["k"].shape[2],
                                    s["dtype"], k=s["k_out"], v=s["v_out"])
        return {"k": k, "v": v}
    if s["op"] == "anchor":
        out, lse, pooled = api.decode_anchor_paged_q4(s["q"], s["pages"], s["table"], s["page"], s["len"],
                                                      s["max_T"], SCALE, s["Hkv"], out=s["out"], lse=s["lse"],
                                                      pooled=s["pooled"], ld_pooled=s["ld"])
        return {"out": out, "lse": lse, "pooled": pooled}
    out, lse = api.decode_reuse_paged_q4(s["q"], s["pages"], s["table"], s["page"], s["len"], s["idx"], s["idx_k"],
                                         s["map"], SCALE, s["Hkv"], out=s["out"], lse=s["lse"])
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"norm_rope": _plain_norm_rope, "cache": _plain_cache, "anchor": _plain_anchor,
            "reuse": _plain_reuse}[state["op"]](state)


# ----------------------------------------------------------- in 64 bits ----
def _values(rows):
    """K and V in 64 bits of cache rows [..., 160], by shifts of the 32-bit words."""
    words = rows[..., :128].contiguous().view(torch.int32)
    shift = torch.arange(0, 32, 4, device=rows.device, dtype=torch.int32)
    n = ((words.unsqueeze(-1) >> shift) & 15).double()  # [..., 32 words, 8]
    lead = n.shape[:-2]
    k = n[..., :16, :].reshape(*lead, 4, 4, 8).transpose(-3, -2).reshape(*lead, 4, 32)
    v = n[..., 16:, :].reshape(*lead, 8, 2, 2, 4).movedim(-4, -2).reshape(*lead, 4, 32)
    par = rows[..., 128:].contiguous().view(torch.bfloat16).double().reshape(*lead, 4, 4, 1)
    return ((par[..., 1, :, :] + par[..., 0, :, :] * k).reshape(*lead, D),
            (par[..., 3, :, :] + par[..., 2, :, :] * v).reshape(*lead, D))


def _exact_norm_rope(s):
    out = {}
    ang = torch.einsum("bn,i->bni", s["pos"].double(), s["inv_freq"].double())
    turn = torch.polar(torch.ones_like(ang), ang)
    for name, x, w in (("q", s["q"], s["qw"]), ("k", s["k"], s["kw"])):
        y = x.double()
        if w is not None:
            y = w.double() * y / torch.sqrt(y.square().sum(-1, keepdim=True) / D + EPS)
        if s["case"]["interleaved"]:
            z = torch.view_as_complex(y.unflatten(-1, (D // 2, 2)).contiguous()) * turn[:, :, None]
            y = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(y[..., :64].contiguous(), y[..., 64:].contiguous()) * turn[:, :, None]
            y = torch.cat([z.real, z.imag], -1)
        out[name] = y.permute(0, 2, 1, 3).contiguous()
    return out


def _exact_cache(s):
    out = {}
    for name, x in (("k", s["k"]), ("v", s["v"])):
        y = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(_list(s["case"]["new"])):
            z = x[b, :, :n].double().reshape(x.shape[1], n, 4, 32)
            lo, hi = z.min(-1, keepdim=True).values, z.max(-1, keepdim=True).values
            m = _border(lo, -1)
            step = _border((hi - m) / 15.0, 1)
            code = torch.where(step > 0, torch.round((z - m) / step), torch.zeros_like(z)).clamp(0, 15)
            y[b, :, :n] = torch.where(step > 0, m + step * code, m).reshape(x.shape[1], n, D)
        out[name] = y
    return out


def _border(x, side):
    """x to 8 significant bits, away from it toward +inf (side 1) or -inf (side -1)."""
    f, e = torch.frexp(x)
    f = f * 256
    return torch.ldexp(torch.ceil(f) if side > 0 else torch.floor(f), e - 8)


def _exact_one(q, k, v):
    x = torch.einsum("hgd,hnd->hgn", q, k) * SCALE
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse.unsqueeze(-1))
    return torch.einsum("hgn,hnd->hgd", p, v), lse, p.mean(1)


def _exact_attention(s):
    b, hkv, page, anchor = len(s["len"]), s["Hkv"], s["page"], s["op"] == "anchor"
    o = torch.zeros(b, s["Hq"], D, dtype=torch.float64, device="cuda")
    lse = torch.full((b, s["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    pooled = torch.zeros(b, hkv, s["ld"], dtype=torch.float64, device="cuda") if anchor else None
    for i, t in enumerate(_list(s["case"]["lens"])):
        if not t:
            continue
        flat = s["pages"][s["table"][i, :(t + page - 1) // page].long()].transpose(0, 1).reshape(hkv, -1, ROW)[:, :t]
        if not anchor:
            sel = s["idx"][i, :, :k_for_len(t)][s["map"].long()].long()
            flat = flat.gather(1, sel.unsqueeze(-1).expand(-1, -1, ROW))
        k, v = _values(flat)
        x, l, p = _exact_one(s["q"][i].double().reshape(hkv, -1, D), k, v)
        o[i], lse[i] = x.reshape(-1, D), l.reshape(-1)
        if anchor:
            pooled[i, :, :t] = p
    return {"out": o, "lse": lse, "pooled": pooled} if anchor else {"out": o, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "norm_rope":
        return _exact_norm_rope(s)
    return _exact_cache(s) if s["op"] == "cache" else _exact_attention(s)
