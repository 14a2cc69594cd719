"""Cases, inputs, plain forms and 64-bit references of the 4-bit paged-cache operators.

Four kinds of pass, over one cache format (4-bit codes with two-level scales
beside the codes of each (token, kv head) row):

  tables     block tables and slot maps of a step, from the request lengths
  rows       a step's new K/V rows quantised into the cache, and rows of the
             cache read back as the values they stand for
  attention  causal attention over the cache (prompts, single tokens, both)
  step       a decode step: tables, then new rows written and attended

A cache row of D dims is D/2 code bytes and a 16-byte tail: an fp32 row scale
s, eight uint8 group multipliers m_g (group g = dims [g D/8, (g + 1) D/8)) and
four zero bytes.  s = amax / 889 (889 = 7 * 127), m_g = min(127, ceil((amax_g
/ s) / 7)), code = clamp(rint(x / (s m_g)), -7, 7), all in fp32 with rounded
divisions; the value is s * (m_g * code).  Nibble j of the little-endian word
w (8 dims) holds code + 8 of dim 8 w + 2 j (j < 4) or 8 w + 2 (j - 4) + 1.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPE = "int4_per_token_head"


def _case(op, name=None, **kw):
    c = {"op": op, "req": 1, "kind": "decode", "lo": 1, "hi": 1, "max_new": 1, "heads_q": 8, "heads_kv": 2,
         "dim": 128, "block": 16, "window": 0, "cap": 0.0, "alibi": False, "sinks": False, "tokens": 0,
         "pad": 0, "lens_seed": 1}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a decode step's slots for a serving batch, and the few blocks that begin in it
        _case("tables", "tables/step-64", req=64, lo=1024, hi=4096),
        # chunked prefill beside decodes, an odd batch, a padded token buffer
        _case("tables", "tables/mixed-509", req=509, kind="mixed", lo=1, hi=32768, max_new=512, block=32, pad=77),
        # admission of long prompts: about a million tokens placed at once
        _case("tables", "tables/prompts-1m", req=37, kind="prompt", lo=8192, hi=65536),
        # one decode step's rows
        _case("rows", "rows/step-64", tokens=64, heads_q=32, heads_kv=8),
        # the rows of a prompt batch, with the unused tail of a padded buffer
        _case("rows", "rows/prompt-20011", tokens=20011, pad=613, heads_q=32, heads_kv=8),
        # one short conversation: latency of a single call
        _case("attention", "attention/single-777", lo=777, hi=777, heads_q=8, heads_kv=2, dim=64, cap=30.0),
        # the framework's decode batch: 64 requests of 1024 to 4096 keys
        _case("attention", "attention/decode-64", req=64, lo=1024, hi=4096, heads_q=32, heads_kv=8),
        # long contexts at a wide head group
        _case("attention", "attention/long-32", req=32, lo=32768, hi=32768, heads_q=64, heads_kv=8),
        # a prompt batch at the framework's largest head size and block size
        _case("attention", "attention/prompts-4", req=4, kind="prompt", lo=1024, hi=1024, heads_q=16, heads_kv=2,
              dim=256, block=2176),
        # prompts' chunks beside decodes: ragged lengths, window, ALiBi and sinks
        _case("attention", "attention/mixed-13", req=13, kind="mixed", lo=300, hi=4099, max_new=511, heads_q=32,
              heads_kv=8, window=1024, alibi=True, sinks=True, lens_seed=4),
        # speculative tokens of a few requests, an odd head group
        _case("step", "step/verify-7", req=7, kind="verify", lo=5, hi=900, max_new=3, heads_q=10, heads_kv=2, dim=64),
        # the decode batch as one step
        _case("step", "step/decode-64", req=64, lo=1024, hi=4096, heads_q=32, heads_kv=8),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["tables", "rows", "attention", "attention", "attention", "step"])
    dim = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    c = {"dim": dim, "heads_kv": kv, "lens_seed": rng.randrange(1, 1 << 20), "block": rng.choice([16, 16, 32, 48, 64, 128])}
    if op == "tables":
        c["kind"] = rng.choice(["decode", "mixed", "prompt"])
        c["req"] = _log(rng, 1, 1024 if c["kind"] != "prompt" else 30)
        c["hi"] = _log(rng, 1, 65536 if c["kind"] != "decode" else 262144)
        c["lo"] = _log(rng, 1, c["hi"])
        c["max_new"] = _log(rng, 1, 2048) if c["kind"] == "mixed" else 1
        c["pad"] = rng.choice([0, 0, rng.randrange(1, 300)])
        return _case(op, **c)
    if op == "rows":
        c["tokens"] = _log(rng, 1, (20011 * 8 * 128) // (kv * dim))
        c["pad"] = rng.choice([0, rng.randrange(0, 1 + c["tokens"] // 8)])
        c["heads_q"] = kv * rng.choice([1, 2, 4, 8])
        return _case(op, **c)
    if op == "step":
        c["max_new"] = rng.choice([1, 1, 1, 2, 3])
        group = rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 16) if g * c["max_new"] <= 16])
        c["kind"] = "verify" if c["max_new"] > 1 else "decode"
        c["req"] = _log(rng, 1, 128)
    else:
        group = rng.choice([1, 2, 4, 5, 7, 8, 16])
        c["kind"] = rng.choice(["decode", "decode", "mixed", "prompt"])
        c["req"] = _log(rng, 1, {"decode": 128, "mixed": 16, "prompt": 8}[c["kind"]])
        c["max_new"] = _log(rng, 1, 300) if c["kind"] == "mixed" else 1
        c["window"] = rng.choice([0, 0, _log(rng, 1, 4096)])
        c["cap"] = rng.choice([0.0, 0.0, 30.0, 50.0])
        c["alibi"] = rng.random() < 0.25
        c["sinks"] = rng.random() < 0.25
    c["heads_q"] = kv * group
    # keys of all heads in memory at once in the plain form, and scores of all rows
    most = max(1, (1 << 28) // (c["req"] * kv * dim))
    if c["kind"] == "prompt":
        most = min(most, 2048, int(math.sqrt((1 << 28) / (c["req"] * c["heads_q"]))))
    elif c["kind"] == "mixed":
        most = min(most, (1 << 28) // (c["req"] * c["heads_q"] * c["max_new"]))
    c["hi"] = _log(rng, 1, max(1, min(most, 65536)))
    c["lo"] = _log(rng, 1, c["hi"])
    return _case(op, **c)


def _lens(case):
    """The batch's (length, new tokens) pairs: fixed by the case."""
    rng = random.Random(case["lens_seed"])
    out = []
    for _ in range(case["req"]):
        n = _log(rng, case["lo"], case["hi"])
        if case["kind"] == "decode":
            new = 1
        elif case["kind"] == "prompt":
            new = n
        elif case["kind"] == "verify":
            new = min(n, rng.randint(1, case["max_new"]))
        else:
            new = min(n, rng.randint(1, case["max_new"])) if rng.random() < 0.4 else 1
        out.append((n, new))
    return out


def _row_bytes(dim):
    return dim // 2 + 16


# ---- the cache format, plain -------------------------------------------------------


def _quantise(x):
    """bf16 [..., D] -> cache rows uint8 [..., D/2 + 16]."""
    x = x.float()
    d = x.shape[-1]
    g = x.unflatten(-1, (8, d // 8))
    amax_g = g.abs().amax(-1)
    # (a division by a tensor is a rounded division; by a number it may be a product)
    amax = amax_g.amax(-1, keepdim=True)
    s = amax / torch.full_like(amax, 889.0)
    live = s > 0
    m = torch.ceil(amax_g / torch.where(live, s, 1.0) / torch.full_like(amax_g, 7.0))
    m = torch.where(live, m.clamp(max=127.0), 0.0)
    step = (s * m).unsqueeze(-1)
    code = torch.where(step > 0, torch.round(g / torch.where(step > 0, step, 1.0)).clamp(-7, 7), 0.0)
    n = (code + 8).to(torch.uint8).flatten(-2).unflatten(-1, (d // 8, 4, 2)).transpose(-1, -2)  # [.., 2, 4]: nibbles
    n = n.flatten(-2).unflatten(-1, (4, 2))
    codes = (n[..., 0] | (n[..., 1] << 4)).flatten(-2)
    tail = s.contiguous().view(torch.uint8)
    return torch.cat((codes, tail, m.to(torch.uint8), torch.zeros_like(tail)), -1)


def _values(rows, d):
    """Cache rows uint8 [..., D/2 + 16] -> fp32 [..., D]."""
    b = rows[..., : d // 2].unflatten(-1, (d // 8, 4))
    n = torch.stack((b & 15, b >> 4), -1).flatten(-2).unflatten(-1, (2, 4)).transpose(-1, -2)
    code = n.flatten(-3).unflatten(-1, (8, d // 8)).float() - 8.0
    s = rows[..., d // 2 : d // 2 + 4].contiguous().view(torch.float32)
    m = rows[..., d // 2 + 4 : d // 2 + 12].float().unsqueeze(-1)
    return (code * m).flatten(-2) * s


def _tables(s):
    """Block tables and slot maps, plain: in place, as the operator does."""
    block, qsl, lens, table = s["block"], s["qsl"].long(), s["lens"].long(), s["table"]
    new = qsl[1:] - qsl[:-1]
    held = (lens - new + block - 1) // block
    need = (lens + block - 1) // block
    base = torch.cumsum(need - held, 0) - (need - held)
    t = s["token_ids"]
    r = torch.searchsorted(qsl, t, right=True) - 1
    live = r < new.numel()
    r = r.clamp(max=new.numel() - 1)
    pos = lens[r] - new[r] + t - qsl[r]
    lb = torch.where(live, pos // block, 0)
    at = base[r] + lb - held[r]
    count = s["free_count"].long()
    fresh = s["free"][(count - 1 - at).clamp(min=0, max=s["free"].numel() - 1)]
    ids = torch.where(lb >= held[r], fresh, table[r, lb])
    table[r, lb] = torch.where(live, ids, table[r, lb])
    s["slots"].copy_(torch.where(live, ids.long() * block + pos % block, -1))
    s["free_left"].copy_((count - (need - held).sum()).int())
    return s["slots"], table, s["free_left"]


def _put(s):
    """The new rows into the cache, plain; rows without a slot go to a spare one."""
    spare = s["slots_total"]
    at = torch.where(s["slots"] < 0, spare, s["slots"])
    for cache, x in ((s["k_pool"], s["key"]), (s["v_pool"], s["value"])):
        cache.flatten(0, 1)[at] = _quantise(x)


def _get(s):
    at = s["slots"].clamp(min=0)
    live = (s["slots"] >= 0)[:, None, None]
    return [torch.where(live, _values(c.flatten(0, 1)[at], s["dim"]), 0.0) for c in (s["k_pool"], s["v_pool"])]


def _attend(s):
    """Causal attention over the cache, plain: every request padded to the longest."""
    d, hkv = s["dim"], s["heads_kv"]
    group = s["q"].shape[1] // hkv
    lens, qsl = s["lens"].long(), s["qsl"].long()
    new = qsl[1:] - qsl[:-1]
    keys = torch.arange(s["max_len"], device="cuda")
    block = s["table"].long()[:, keys // s["block"]].clamp(0, s["k_pool"].shape[0] - 1)  # [R, L]
    at = block * s["block"] + keys % s["block"]
    k = _values(s["k_pool"].flatten(0, 1)[at], d)  # [R, L, Hkv, D]
    i = torch.arange(s["max_new"], device="cuda")
    rows = (qsl[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().unflatten(2, (hkv, group))  # [R, Q, Hkv, G, D]
    z = torch.matmul(q.permute(0, 2, 1, 3, 4).flatten(2, 3), k.permute(0, 2, 3, 1)) * s["sm_scale"]
    del k
    z = z.unflatten(2, (-1, group))  # [R, Hkv, Q, G, L]
    if s["cap"] > 0:
        z = s["cap"] * torch.tanh(z / s["cap"])
    pos = (lens - new)[:, None] + i  # [R, Q]
    far = keys - pos[..., None]  # [R, Q, L]
    if s["slopes"] is not None:
        z = z + s["slopes"].view(1, hkv, 1, group, 1) * far[:, None, :, None].float()
    seen = (far <= 0) & (keys < lens[:, None, None])
    if s["window"] > 0:
        seen = seen & (far > -s["window"])
    z = z.masked_fill(~seen[:, None, :, None], float("-inf"))
    top = z.amax(-1, keepdim=True)
    sinks = None
    if s["sinks"] is not None:
        sinks = s["sinks"].view(1, hkv, 1, group, 1)
        top = torch.maximum(top, sinks)
    top = torch.where(top == float("-inf"), 0.0, top)
    e = torch.exp(z - top)
    del z
    total = e.sum(-1, keepdim=True)
    if sinks is not None:
        total = total + torch.exp(sinks - top)
    v = _values(s["v_pool"].flatten(0, 1)[at], d)
    o = torch.matmul(e.flatten(2, 3), v.permute(0, 2, 1, 3)).unflatten(2, (-1, group)) / total
    o = o.permute(0, 2, 1, 3, 4).flatten(2, 3)  # [R, Q, Hq, D]
    t = torch.arange(s["q"].shape[0], device="cuda")
    r = torch.searchsorted(qsl, t, right=True) - 1
    return o[r, t - qsl[r]].to(torch.bfloat16)


# ---- inputs ------------------------------------------------------------------------


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    s = {"op": case["op"], "dim": case["dim"], "heads_kv": case["heads_kv"], "block": case["block"]}
    rnd = lambda *n: torch.randn(n, generator=gen, device="cuda")  # noqa: E731
    hq, hkv, d, block = case["heads_q"], case["heads_kv"], case["dim"], case["block"]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    batch = _lens(case)
    if case["op"] == "rows":
        tokens = case["tokens"]
        need = [-(-(tokens + 5) // block) + 3]
    else:
        tokens = sum(n for _, n in batch)
        need = [-(-n // block) for n, _ in batch]
    blocks = sum(need) + 2
    perm = torch.randperm(blocks, generator=gen, device="cuda").int()
    if case["op"] != "rows":
        s["lens"] = ints([n for n, _ in batch])
        s["qsl"] = ints([0] + list(np.cumsum([n for _, n in batch])))
        s["max_len"], s["max_new"] = max(n for n, _ in batch), max(n for _, n in batch)
        width = max(need)
        r = torch.repeat_interleave(torch.arange(len(need), device="cuda"), torch.tensor(need, device="cuda"))
        begin = torch.tensor([0] + list(np.cumsum(need)), device="cuda")
        col = torch.arange(r.numel(), device="cuda") - begin[r]
        s["table"] = torch.zeros((len(need), width), dtype=torch.int32, device="cuda")
        s["table"][r, col] = perm[: r.numel()]
        if case["op"] in ("tables", "step"):
            # the blocks that begin in this step are still on the free list, the next to be taken last
            held = torch.tensor([-(-(n - q) // block) for n, q in batch], device="cuda")
            begins = col >= held[r]
            taken = s["table"][r, col][begins]
            s["table"][r[begins], col[begins]] = -1
            s["free"] = torch.cat((perm[r.numel():], taken.flip(0))).contiguous()
            s["free_count"] = ints([s["free"].numel()])
            s["free_left"] = torch.zeros_like(s["free_count"])
            s["status"] = torch.zeros(4, dtype=torch.int32, device="cuda")
            s["slots"] = torch.zeros(tokens + case["pad"], dtype=torch.int64, device="cuda")
            s["token_ids"] = torch.arange(tokens + case["pad"], device="cuda")
    if case["op"] != "tables":
        # keys with a few large channels and tokens of unequal size, as projections give them
        s["k_pool"] = torch.empty((blocks + 1, block, hkv, _row_bytes(d)), dtype=torch.uint8, device="cuda")
        s["v_pool"] = torch.empty_like(s["k_pool"])
        s["slots_total"] = blocks * block
        gain = 1.0 + 7.0 * (torch.rand((hkv, d), generator=gen, device="cuda") < 0.03).float()
        a_time = max(1, (1 << 27) // (block * hkv * d))
        for b in range(0, blocks + 1, a_time) if case["op"] != "rows" else ():
            n = min(a_time, blocks + 1 - b)
            size = torch.exp(0.3 * rnd(n, block, 1, 1))
            s["k_pool"][b : b + n] = _quantise((rnd(n, block, hkv, d) * gain * size).to(torch.bfloat16))
            s["v_pool"][b : b + n] = _quantise((rnd(n, block, hkv, d) * size).to(torch.bfloat16))
        if case["op"] in ("rows", "step"):
            n = tokens
            qkv = rnd(n, hq + 2 * hkv, d)  # a fused projection's output: rows at its stride
            qkv[:, hq : hq + hkv] *= gain
            qkv = qkv.to(torch.bfloat16)
            s["key"], s["value"] = qkv[:, hq : hq + hkv], qkv[:, hq + hkv :]
        if case["op"] == "rows":
            s["k_pool"].zero_(), s["v_pool"].zero_()
            slots = perm.long()[:, None] * block + torch.arange(block, device="cuda")
            s["slots"] = slots.flatten()[:tokens].contiguous()
            if case["pad"]:
                s["slots"][tokens - min(case["pad"], tokens - 1):] = -1
            s["out"] = [torch.empty((tokens, hkv, d), dtype=torch.float32, device="cuda") for _ in range(2)]
    if case["op"] in ("attention", "step"):
        s["q"] = rnd(tokens, hq, d).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        s["sm_scale"], s["cap"], s["window"] = 1.0 / math.sqrt(d), case["cap"], case["window"]
        s["slopes"] = torch.exp2(-8.0 * (torch.arange(hq, device="cuda") + 1.0) / hq) if case["alibi"] else None
        s["sinks"] = 2.0 * rnd(hq) if case["sinks"] else None
    if own:
        from int8_kv_cache_reshape_gb300 import kvq

        if case["op"] != "tables":
            kc, vc = s["k_pool"][:blocks], s["v_pool"][:blocks]
        if case["op"] in ("tables", "step"):
            s["build"] = kvq.prepare_build_block_tables(
                s["qsl"], s["lens"], s["free"], s["free_count"], s["table"], s["slots"], block, blocks,
                s["free_left"], s["status"])
        if case["op"] == "rows":
            s["write"] = kvq.prepare_reshape_and_cache(s["key"], s["value"], kc, vc, s["slots"], DTYPE)
            s["read"] = kvq.prepare_gather_cache(kc, vc, s["slots"], s["out"][0], s["out"][1], DTYPE)
        if case["op"] == "attention":
            s["plan"] = kvq.get_scheduler_metadata(
                len(batch), hq, hkv, d, np.array([n for n, _ in batch], np.int32),
                np.cumsum([0] + [n for _, n in batch]).astype(np.int32), True, case["window"], DTYPE)
            s["scratch"] = torch.empty(max(256, s["plan"].workspace_bytes), dtype=torch.uint8, device="cuda")
            s["attend"] = kvq.prepare_attention_with_kv_cache(
                s["plan"], s["q"], kc, vc, s["qsl"], s["lens"], s["table"], s["sm_scale"], True, case["window"],
                case["cap"], 1.0, 1.0, s["out"], s["scratch"], DTYPE, hkv, alibi_slopes=s["slopes"], sinks=s["sinks"])
        if case["op"] == "step":
            size = kvq.decode_step_workspace_size(len(batch), hq, hkv, d, DTYPE, case["max_new"])
            s["scratch"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
            s["decode"] = kvq.prepare_decode_step(
                s["key"], s["value"], s["slots"], kc, vc, s["q"], s["qsl"], s["lens"], s["table"], case["max_new"],
                s["sm_scale"], 0, 0.0, 1.0, 1.0, s["out"], s["scratch"], DTYPE, hkv)
    return s


def run(s):
    op = s["op"]
    if own:
        if op == "tables":
            s["build"]()
            return {"slots": s["slots"], "table": s["table"], "free_left": s["free_left"]}
        if op == "rows":
            s["write"]()
            s["read"]()
            return {"key": s["out"][0], "value": s["out"][1]}
        if op == "attention":
            s["attend"]()
            return {"out": s["out"]}
        s["build"]()
        s["decode"]()
        return {"out": s["out"], "slots": s["slots"], "table": s["table"], "free_left": s["free_left"]}
    if op == "tables":
        slots, table, left = _tables(s)
        return {"slots": slots, "table": table, "free_left": left}
    if op == "rows":
        _put(s)
        key, value = _get(s)
        return {"key": key, "value": value}
    if op == "attention":
        return {"out": _attend(s)}
    slots, table, left = _tables(s)
    _put(s)
    return {"out": _attend(s), "slots": slots, "table": table, "free_left": left}


def work(case):
    batch = _lens(case)
    hq, hkv, d, block, row = case["heads_q"], case["heads_kv"], case["dim"], case["block"], _row_bytes(case["dim"])
    tables = 0
    for n, new in batch:
        begins = -(-n // block) - -(-(n - new) // block)
        tables += 8 + 8 * begins + 4 * ((n - new) % block != 0) + 8 * new
    if case["op"] == "tables":
        return {"bytes": tables + 8 * case["pad"], "flops": 0}
    if case["op"] == "rows":
        t = case["tokens"]
        live = t - min(case["pad"], t - 1)
        # bf16 rows in, codes out; codes in, fp32 values out
        return {"bytes": 8 * t + 2 * live * hkv * (2 * d + row) + 2 * hkv * (live * row + 4 * t * d), "flops": 0}
    pairs = keys = 0
    for n, new in batch:
        w = case["window"] or n
        keys += n - max(0, n - new - w + 1)
        first, last = n - new + 1, n  # keys at or before each query
        short = max(0, min(last, w) - first + 1)
        pairs += short * (first + min(last, w)) // 2 + (new - short) * w
    tokens = sum(new for _, new in batch)
    total = 2 * keys * hkv * row + 4 * tokens * hq * d + sum(4 * (-(-n // block)) for n, _ in batch)
    if case["op"] == "step":
        total += tables + 4 * tokens * hkv * d
    return {"bytes": total, "flops": 4 * d * hq * pairs}


# ---- from the definition, in 64 bits -------------------------------------------------


def _decode64(rows, d):
    """Values of cache rows, one nibble position at a time."""
    words = rows[..., : d // 2].contiguous().view(torch.int32).long() & 0xFFFFFFFF
    out = torch.zeros((*rows.shape[:-1], d), dtype=torch.float64, device=rows.device)
    for j in range(8):
        dim = 2 * j if j < 4 else 2 * (j - 4) + 1
        out[..., dim::8] = (((words >> (4 * j)) & 15) - 8).double()
    scale = rows[..., d // 2 : d // 2 + 4].contiguous().view(torch.float32).double()
    for g in range(8):
        out[..., g * d // 8 : (g + 1) * d // 8] *= rows[..., d // 2 + 4 + g : d // 2 + 5 + g].double()
    return out * scale


def _encode64(x):
    """Values that rows x [..., D] stand for after quantisation.  Each division and
    product is the exact one rounded to 32 bits, as the format defines them."""
    r32 = lambda v: v.float().double()  # noqa: E731
    x = x.double()
    d = x.shape[-1]
    s = r32(x.abs().max(-1, keepdim=True).values / 889.0)
    out = torch.zeros_like(x)
    for g in range(8):
        y = x[..., g * d // 8 : (g + 1) * d // 8]
        top = y.abs().max(-1, keepdim=True).values
        m = torch.ceil(r32(r32(top / s) / 7.0)).clamp(max=127.0)
        code = torch.round(r32(y / r32(s * m))).clamp(-7, 7)
        out[..., g * d // 8 : (g + 1) * d // 8] = torch.where((s > 0) & (m > 0), s * (m * code), 0.0)
    return out


def exact(case, seed):
    if case["op"] == "tables":
        return None
    s = prepare(case, seed)
    d, hkv, block = s["dim"], s["heads_kv"], s["block"]
    if case["op"] == "rows":
        live = (s["slots"] >= 0)[:, None, None]
        return {"key": torch.where(live, _encode64(s["key"]), 0.0), "value": torch.where(live, _encode64(s["value"]), 0.0)}
    batch = _lens(case)
    group = case["heads_q"] // hkv
    kc, vc = s["k_pool"].flatten(0, 1), s["v_pool"].flatten(0, 1)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    table = s["table"].tolist()
    free = s["free"].tolist() if case["op"] == "step" else []
    t = 0
    for r, (n, new) in enumerate(batch):
        need, held = -(-n // block), -(-(n - new) // block)
        ids = table[r][:need] if case["op"] == "attention" else table[r][:held] + [free.pop() for _ in range(need - held)]
        at = (torch.tensor(ids, device="cuda")[:, None] * block + torch.arange(block, device="cuda")).flatten()[:n]
        k, v = _decode64(kc[at], d), _decode64(vc[at], d)  # [L, Hkv, D]
        if case["op"] == "step":
            k[n - new :], v[n - new :] = _encode64(s["key"][t : t + new]), _encode64(s["value"][t : t + new])
        far = torch.arange(n, device="cuda") - torch.arange(n - new, n, device="cuda")[:, None]  # key - query
        hidden = far > 0
        if case["window"]:
            hidden |= far <= -case["window"]
        for h in range(hkv):
            q = s["q"][t : t + new, h * group : (h + 1) * group].double()
            z = torch.einsum("qgd,kd->qgk", q, k[:, h]) / math.sqrt(d)
            if case["cap"]:
                z = case["cap"] * torch.tanh(z / case["cap"])
            if s["slopes"] is not None:
                z = z + s["slopes"][h * group : (h + 1) * group].double()[None, :, None] * far[:, None].double()
            z[hidden[:, None].expand_as(z)] = float("-inf")
            if s["sinks"] is not None:
                z = torch.cat((z, s["sinks"][h * group : (h + 1) * group].double().view(1, group, 1).expand(new, group, 1)), -1)
            w = torch.exp(z - z.max(-1, keepdim=True).values)
            w = w / w.sum(-1, keepdim=True)
            out[t : t + new, h * group : (h + 1) * group] = torch.einsum("qgk,kd->qgd", w[..., :n], v[:, h])
        t += new
    got = {"out": out}
    return got if case["op"] == "attention" else {**got, "slots": None, "table": None, "free_left": None}
