"""Cases, inputs, plain forms and 64-bit references of the operators around a paged cache's life.

Four kinds of pass:

  append   a step's queries and keys rotated by their positions (cos / sin rows of a table), the keys and values
           stored in the paged cache in its format; the stored rows are read back as the values they stand for
  shared   causal attention of a batch whose requests begin with the same keys: the keys of a shared prefix are in
           the cache once, and each request goes on with keys of its own
  cross    attention of a batch's tokens to an encoder's states, cached once per request, of another length
  step     a decode step of a batch with a shared prefix: append, then shared

The rotation of a pair (a, b) by the angle of its position is (a c - b s, b c + a s), c and s from an fp32 table, each
product and sum rounded to 32 bits.  Pair j is the dims (j, j + R / 2) or, "interleaved", (2 j, 2 j + 1), of the first
R dims; the rest are not rotated.

Cache rows of D dims, by type (quotients and products rounded to 32 bits):
  auto                     D bf16 values
  fp8_e4m3, fp8_e5m2       D codes of x / scale (one scale for a tensor), nearest (ties to even), saturating
  int8_per_token_head,     D codes of x / s, then s (fp32) and 12 zero bytes; s = amax / 127, 448, 57344
  fp8_per_token_head, fp8_e5m2_per_token_head
  int4_per_token_head      D/2 code bytes, then s = amax / 889 (fp32), eight uint8 multipliers m_g = min(127,
                           ceil((amax_g / s) / 7)) of groups of D/8 dims, four zero bytes; code = clamp(rint(x / (s
                           m_g)), -7, 7), value s (m_g code).  Nibble j of the little-endian word w (8 dims) holds
                           code + 8 of dim 8 w + 2 j (j < 4) or 8 w + 2 (j - 4) + 1.
"""
import math
import random

import torch

own = False

DTYPES = ["auto", "fp8_e4m3", "fp8_e5m2", "int8_per_token_head", "fp8_per_token_head", "fp8_e5m2_per_token_head",
          "int4_per_token_head"]
QMAX = {"int8_per_token_head": 127.0, "fp8_per_token_head": 448.0, "fp8_e5m2_per_token_head": 57344.0,
        "fp8_e4m3": 448.0, "fp8_e5m2": 57344.0}
MAX_POSITION = 131072


def _case(op, name=None, **kw):
    c = {"op": op, "dtype": "int8_per_token_head", "heads_q": 8, "heads_kv": 2, "dim": 128, "block": 16, "req": 1,
         "lo": 1, "hi": 1, "max_new": 1, "prefixes": 1, "prefix": 0, "loose": False, "window": 0, "cap": 0.0,
         "alibi": False, "sinks": False, "tokens": 0, "pad": 0, "rotary": 128, "interleaved": False, "lens_seed": 1}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the next token of one conversation: latency of a single call
        _case("append", "append/token-1", tokens=1, dim=64, rotary=64),
        # a decode step's rows of the framework's decode batch
        _case("append", "append/step-64", tokens=64, heads_q=32, heads_kv=8, dtype="fp8_per_token_head"),
        # a chunk of prompts, the wide head size, half of its dims rotated pair by pair, bf16 rows
        _case("append", "append/chunk-4099", tokens=4099, heads_q=16, heads_kv=2, dim=256, rotary=128,
              interleaved=True, dtype="auto"),
        # a prompt batch into the 4-bit cache, with the unused tail of a padded buffer
        _case("append", "append/prompt-20011", tokens=20011, pad=613, heads_q=32, heads_kv=8,
              dtype="int4_per_token_head"),
        # a few users behind a short instruction
        _case("shared", "shared/small-5", req=5, prefix=304, lo=1, hi=90, dim=64, cap=30.0, dtype="int4_per_token_head"),
        # the decode batch behind a long instruction, each with a conversation of its own
        _case("shared", "shared/decode-64", req=64, prefix=8192, lo=64, hi=1024, heads_q=32, heads_kv=8),
        # many samples drawn from one long document
        _case("shared", "shared/samples-256", req=256, prefix=16384, lo=1, hi=512, heads_q=64, heads_kv=8,
              dtype="fp8_e4m3"),
        # three instructions and requests without one, tokens to verify, the wide head size, every option
        _case("shared", "shared/groups-37", req=37, prefixes=3, prefix=4000, loose=True, lo=2, hi=700, max_new=3,
              heads_q=8, heads_kv=2, dim=256, window=3500, alibi=True, sinks=True, dtype="fp8_e5m2_per_token_head"),
        # one decoder token for each of a batch of 30-second audio segments
        _case("cross", "cross/token-48", req=48, lo=1500, hi=1500, heads_q=20, heads_kv=20, dim=64, dtype="auto"),
        # decoder prompts against documents of very different lengths
        _case("cross", "cross/prompts-16", req=16, lo=100, hi=4096, max_new=448, heads_q=16, heads_kv=16, dim=64),
        # long outputs over long inputs
        _case("cross", "cross/long-4", req=4, lo=4096, hi=4096, max_new=1024, heads_q=32, heads_kv=8,
              dtype="fp8_e4m3"),
        # the decode batch behind the long instruction as one step
        _case("step", "step/decode-64", req=64, prefix=8192, lo=64, hi=1024, heads_q=32, heads_kv=8),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["append", "shared", "shared", "cross", "cross", "step"])
    dim = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    c = {"dim": dim, "heads_kv": kv, "dtype": rng.choice(DTYPES), "lens_seed": rng.randrange(1, 1 << 20),
         "block": rng.choice([16, 16, 32, 48, 64, 128]), "rotary": rng.choice([dim, dim, dim // 2, 16, 48]),
         "interleaved": rng.random() < 0.3}
    group = rng.choice([1, 2, 4, 5, 7, 8])
    c["heads_q"] = kv * group
    if op == "append":
        c["tokens"] = _log(rng, 1, 20011 * 48 * 128 // ((c["heads_q"] + 2 * kv) * dim))
        c["pad"] = rng.choice([0, rng.randrange(0, 1 + c["tokens"] // 8)])
        return _case(op, **c)
    c["cap"] = rng.choice([0.0, 0.0, 30.0, 50.0])
    c["sinks"] = rng.random() < 0.25
    pairs = (1 << 29) * 64 // dim  # (query head, key) pairs: no more products than the largest listed case's
    if op == "cross":
        c["req"] = _log(rng, 1, 64)
        c["max_new"] = rng.choice([1, _log(rng, 1, 2048)])
        most = min(pairs // (c["req"] * c["heads_q"] * c["max_new"]), (1 << 27) // (c["req"] * kv * dim))
        if most < 1:
            c["max_new"], most = 1, (1 << 27) // (c["req"] * kv * dim)
        c["hi"] = _log(rng, 1, min(most, 16384))
        c["lo"] = rng.choice([0, _log(rng, 1, c["hi"])])
        return _case(op, **c)
    c["req"] = _log(rng, 2, 256)
    c["max_new"] = rng.choice([n for n in (1, 1, 1, 2, 3) if n * group <= 16])
    c["prefixes"] = rng.choice([1, 1, 2, 3])
    c["loose"] = rng.random() < 0.3
    c["window"] = rng.choice([0, 0, 0, _log(rng, 64, 16384)])
    c["alibi"] = rng.random() < 0.25
    most = max(c["max_new"], (1 << 26) // (c["req"] * kv * dim))
    c["hi"] = _log(rng, c["max_new"], min(most, 4096))
    c["lo"] = _log(rng, 1, c["hi"])
    most = min(pairs // (c["req"] * c["heads_q"] * c["max_new"]), (1 << 27) // (kv * dim))
    c["prefix"] = _log(rng, 16, max(16, min(most, 65536)))
    return _case(op, **c)


def _lens(case):
    """The batch, fixed by the case: of each request (keys, new tokens, prefix or -1), and the prefixes' lengths."""
    if case["op"] == "append":
        return [], []
    rng = random.Random(case["lens_seed"])
    block, prefixes = case["block"], []
    if case["op"] != "cross":
        for n in range(case["prefixes"]):
            most = case["prefix"] if n == 0 else rng.randint(case["prefix"] // 2, case["prefix"])
            prefixes.append(most // block * block)  # (whole blocks are shared)
    batch = []
    for r in range(case["req"]):
        if case["op"] == "cross":
            n = 0 if case["lo"] == 0 and rng.random() < 0.2 else _log(rng, max(1, case["lo"]), max(1, case["hi"]))
            new = rng.randint(max(1, case["max_new"] // 2), case["max_new"])
            batch.append((n, new, -1))
            continue
        p = rng.randrange(len(prefixes))
        if case["loose"] and rng.random() < 0.2:
            p = -1
        mine = _log(rng, case["lo"], case["hi"])
        new = min(mine, rng.randint(1, case["max_new"]))
        batch.append((mine + (prefixes[p] if p >= 0 else 0), new, p))
    return batch, prefixes


def _row_bytes(dtype, dim):
    if dtype == "int4_per_token_head":
        return dim // 2 + 16
    return 2 * dim if dtype == "auto" else dim + (16 if "per_token" in dtype else 0)


# ---- the cache formats, plain ------------------------------------------------------


def _codes(dtype, y):
    """Codes uint8 [..., D] of the quotients y."""
    if dtype.startswith("int8"):
        return torch.round(y).clamp(-128, 127).to(torch.int8).view(torch.uint8)
    if "e5m2" in dtype:
        return y.clamp(-57344.0, 57344.0).to(torch.float8_e5m2).view(torch.uint8)
    return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _over(x, by):
    """x / by as rounded divisions (a division by a number may be a product)."""
    return x / torch.full_like(x, by)


def _quantise(dtype, x, scale):
    """fp32 [..., D] -> cache rows uint8."""
    if dtype == "auto":
        return x.to(torch.bfloat16).contiguous().view(torch.uint8)
    if "per_token" not in dtype:
        return _codes(dtype, _over(x, scale))
    d = x.shape[-1]
    amax = x.abs().amax(-1, keepdim=True)
    if dtype != "int4_per_token_head":
        s = _over(amax, QMAX[dtype])
        codes = _codes(dtype, torch.where(s > 0, x / torch.where(s > 0, s, 1.0), 0.0))
        tail = s.contiguous().view(torch.uint8)
        return torch.cat((codes, tail, torch.zeros_like(tail).repeat_interleave(3, -1)), -1)
    g = x.unflatten(-1, (8, d // 8))
    amax_g = g.abs().amax(-1)
    s = _over(amax, 889.0)
    live = s > 0
    m = torch.ceil(_over(amax_g / torch.where(live, s, 1.0), 7.0))
    m = torch.where(live, m.clamp(max=127.0), 0.0)
    step = (s * m).unsqueeze(-1)
    code = torch.where(step > 0, torch.round(g / torch.where(step > 0, step, 1.0)).clamp(-7, 7), 0.0)
    n = (code + 8).to(torch.uint8).flatten(-2).unflatten(-1, (d // 8, 4, 2)).transpose(-1, -2)  # [.., 2, 4]: nibbles
    n = n.flatten(-2).unflatten(-1, (4, 2))
    codes = (n[..., 0] | (n[..., 1] << 4)).flatten(-2)
    tail = s.contiguous().view(torch.uint8)
    return torch.cat((codes, tail, m.to(torch.uint8), torch.zeros_like(tail)), -1)


def _values(dtype, rows, d, scale):
    """Cache rows uint8 -> fp32 [..., D]."""
    if dtype == "auto":
        return rows.contiguous().view(torch.bfloat16).float()
    if dtype == "int4_per_token_head":
        b = rows[..., : d // 2].unflatten(-1, (d // 8, 4))
        n = torch.stack((b & 15, b >> 4), -1).flatten(-2).unflatten(-1, (2, 4)).transpose(-1, -2)
        code = n.flatten(-3).unflatten(-1, (8, d // 8)).float() - 8.0
        s = rows[..., d // 2 : d // 2 + 4].contiguous().view(torch.float32)
        m = rows[..., d // 2 + 4 : d // 2 + 12].float().unsqueeze(-1)
        return (code * m).flatten(-2) * s
    codes = rows[..., :d].contiguous()
    kind = torch.int8 if dtype.startswith("int8") else torch.float8_e5m2 if "e5m2" in dtype else torch.float8_e4m3fn
    v = codes.view(kind).float()
    return v * (rows[..., d : d + 4].contiguous().view(torch.float32) if "per_token" in dtype else scale)


# ---- the operators, plain ----------------------------------------------------------


def _rotate(s, x):
    """bf16 [T, H, D] -> fp32, rotated by the tokens' positions."""
    x = x.float()
    half = s["rotary"] // 2
    row = s["cos_sin"][s["positions"]]
    c, n = row[:, None, :half], row[:, None, half:]
    out = x.clone()
    if s["interleaved"]:
        a, b = slice(0, 2 * half, 2), slice(1, 2 * half, 2)
    else:
        a, b = slice(0, half), slice(half, 2 * half)
    out[..., a] = x[..., a] * c - x[..., b] * n
    out[..., b] = x[..., b] * c + x[..., a] * n
    return out


def _append(s):
    """Rotated queries, and the rows into the cache; rows without a slot go to a spare one."""
    at = torch.where(s["slots"] < 0, s["slots_total"], s["slots"])
    s["k_pool"].flatten(0, 1)[at] = _quantise(s["dtype"], _rotate(s, s["key"]), s["k_scale"])
    s["v_pool"].flatten(0, 1)[at] = _quantise(s["dtype"], s["value"].float(), s["v_scale"])
    return _rotate(s, s["query"]).to(torch.bfloat16)


def _rows(s, which, at):
    return _values(s["dtype"], s[which + "_pool"].flatten(0, 1)[at], s["dim"], s[which + "_scale"])


def _slots(s, table, keys):
    """Slots of the key positions of table rows [.., width]."""
    last = s["k_pool"].shape[0] - 1
    return table.long()[..., keys // s["block"]].clamp(0, last) * s["block"] + keys % s["block"]


def _soft(s, z, far, seen, group):
    """Scores [T, Hkv, G, K] with cap, bias and masks; far, seen [T, K]."""
    if s["cap"] > 0:
        z = s["cap"] * torch.tanh(z / s["cap"])
    if s["slopes"] is not None:
        z = z + s["slopes"].view(1, -1, group, 1) * far[:, None, None].float()
    return z.masked_fill(~seen[:, None, None], float("-inf"))


def _shared(s, q):
    """Causal attention, the keys of each prefix taken once; a request's own keys padded to the longest."""
    d, hkv = s["dim"], s["heads_kv"]
    t, hq = q.shape[0], q.shape[1]
    group = hq // hkv
    q = q.float().unflatten(1, (hkv, group))  # [T, Hkv, G, D]
    req, pos, begin = s["token_req"], s["token_pos"], s["begin"]
    longest = max(s["prefix_lens"], default=0)
    z_pre = torch.full((t, hkv, group, longest), float("-inf"), device="cuda")
    values = []
    for p, n in enumerate(s["prefix_lens"]):
        idx = s["members"][p]
        keys = torch.arange(n, device="cuda")
        if n == 0 or idx.numel() == 0:
            values.append(None)
            continue
        at = _slots(s, s["table"][req[idx[0]]], keys)
        z = torch.einsum("thgd,khd->thgk", q[idx], _rows(s, "k", at)) * s["sm_scale"]
        far = keys - pos[idx][:, None]
        seen = far > -s["window"] if s["window"] > 0 else far <= 0
        z_pre[idx, :, :, :n] = _soft(s, z, far, seen, group)
        values.append((idx, n, _rows(s, "v", at)))
    keys = begin[:, None] + torch.arange(s["own_len"], device="cuda")  # [R, K]
    lens = s["lens"].long()
    at = _slots_by_row(s, s["table"], keys)
    z = _by_request(s, q, _rows(s, "k", at))
    far = keys[req] - pos[:, None]
    seen = (far <= 0) & (keys < lens[:, None])[req]
    if s["window"] > 0:
        seen = seen & (far > -s["window"])
    z = _soft(s, z * s["sm_scale"], far, seen, group)
    top = torch.maximum(z.amax(-1, keepdim=True), z_pre.amax(-1, keepdim=True)) if longest else z.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        sinks = s["sinks"].view(1, hkv, group, 1)
        top = torch.maximum(top, sinks)
    e, e_pre = torch.exp(z - top), torch.exp(z_pre - top)
    total = e.sum(-1, keepdim=True) + e_pre.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        total = total + torch.exp(sinks - top)
    o = _weigh(s, e, _rows(s, "v", at))
    for v in values:
        if v is not None:
            idx, n, rows = v
            o[idx] += torch.einsum("thgk,khd->thgd", e_pre[idx, :, :, :n], rows)
    return (o / total).flatten(1, 2).to(torch.bfloat16)


def _slots_by_row(s, table, keys):
    """Slots of key positions [R, K] of each request's own table row."""
    last = table.shape[1] - 1
    block = torch.gather(table.long(), 1, (keys // s["block"]).clamp(max=last))
    return block.clamp(0, s["k_pool"].shape[0] - 1) * s["block"] + keys % s["block"]


def _padded(s, x):
    """[T, ...] -> [R, Q, ...], the last row again where a request has fewer tokens."""
    qsl = s["qsl"].long()
    rows = (qsl[:-1, None] + torch.arange(s["max_new"], device="cuda")).clamp(max=x.shape[0] - 1)
    return x[rows]


def _by_token(s, x):
    """[R, Q, ...] -> [T, ...]."""
    t = torch.arange(s["token_req"].numel(), device="cuda")
    return x[s["token_req"], t - s["qsl"].long()[s["token_req"]]]


def _by_request(s, q, k):
    return _by_token(s, torch.einsum("rqhgd,rkhd->rqhgk", _padded(s, q), k))


def _weigh(s, e, v):
    return _by_token(s, torch.einsum("rqhgk,rkhd->rqhgd", _padded(s, e), v))


def _cross(s, q):
    """Every token of a request against all keys of its encoder, padded to the longest."""
    d, hkv = s["dim"], s["heads_kv"]
    group = q.shape[1] // hkv
    keys = torch.arange(max(1, s["own_len"]), device="cuda").expand(s["lens"].numel(), -1)
    at = _slots_by_row(s, s["table"], keys)
    x = _padded(s, q.float().unflatten(1, (hkv, group)))  # [R, Q, Hkv, G, D]
    z = torch.matmul(x.permute(0, 2, 1, 3, 4).flatten(2, 3), _rows(s, "k", at).permute(0, 2, 3, 1)) * s["sm_scale"]
    if s["cap"] > 0:
        z = s["cap"] * torch.tanh(z / s["cap"])
    z = z.masked_fill((keys >= s["lens"].long()[:, None])[:, None, None], float("-inf"))  # [R, Hkv, Q G, K]
    top = z.amax(-1, keepdim=True)
    sinks = None
    if s["sinks"] is not None:
        sinks = s["sinks"].view(1, hkv, 1, group).expand(1, hkv, s["max_new"], group).reshape(1, hkv, -1, 1)
        top = torch.maximum(top, sinks)
    top = torch.where(top == float("-inf"), 0.0, top)
    e = torch.exp(z - top)
    del z
    total = e.sum(-1, keepdim=True)
    if sinks is not None:
        total = total + torch.exp(sinks - top)
    o = torch.matmul(e, _rows(s, "v", at).permute(0, 2, 1, 3)) / torch.where(total > 0, total, 1.0)
    o = o.unflatten(2, (-1, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [R, Q, Hq, D]
    return _by_token(s, o).to(torch.bfloat16)


# ---- inputs ------------------------------------------------------------------------


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    op, dtype, block = case["op"], case["dtype"], case["block"]
    hq, hkv, d = case["heads_q"], case["heads_kv"], case["dim"]
    s = {"op": op, "dtype": dtype, "dim": d, "heads_kv": hkv, "block": block, "rotary": case["rotary"],
         "interleaved": case["interleaved"], "k_scale": 1.0, "v_scale": 1.0}
    rnd = lambda *n: torch.randn(n, generator=gen, device="cuda")  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    batch, prefixes = _lens(case)
    if op == "append":
        tokens = case["tokens"]
        blocks = -(-(tokens + 5) // block) + 3
    else:
        tokens = sum(new for _, new, _ in batch)
        blocks = sum(n // block for n in prefixes) + 2
        blocks += sum(-(-n // block) - (prefixes[p] // block if p >= 0 else 0) for n, _, p in batch)
    perm = torch.randperm(blocks, generator=gen, device="cuda").int()
    if dtype in ("fp8_e4m3", "fp8_e5m2"):
        s["k_scale"], s["v_scale"] = 48.0 / QMAX[dtype], 6.0 / QMAX[dtype]
    if op != "append":
        # the blocks of the prefixes, then every request's own
        ids, at, first = perm.tolist(), 0, []
        for n in prefixes:
            first.append(ids[at : at + n // block])
            at += n // block
        width = max(1, max(-(-n // block) for n, _, _ in batch))
        table = []
        for n, _, p in batch:
            row = list(first[p]) if p >= 0 else []
            more = -(-n // block) - len(row)
            row += ids[at : at + more]
            at += more
            table.append(row + [-1] * (width - len(row)))
        s["table"] = ints(table)
        s["lens"] = ints([n for n, _, _ in batch])
        starts = [0]
        for _, new, _ in batch:
            starts.append(starts[-1] + new)
        s["qsl"] = ints(starts)
        s["max_new"] = max(new for _, new, _ in batch)
        held = [prefixes[p] if p >= 0 else 0 for _, _, p in batch]
        s["begin"] = torch.tensor(held, device="cuda")
        s["own_len"] = max(n - h for (n, _, _), h in zip(batch, held))
        s["prefix_lens"] = prefixes
        s["token_req"] = torch.repeat_interleave(torch.arange(len(batch), device="cuda"),
                                                 torch.tensor([new for _, new, _ in batch], device="cuda"))
        s["token_pos"] = torch.cat([torch.arange(n - new, n) for n, new, _ in batch]).to("cuda")
        of = torch.tensor([p for _, _, p in batch], device="cuda")[s["token_req"]]
        s["members"] = [torch.nonzero(of == p).flatten() for p in range(len(prefixes))]
    # keys with a few large channels and tokens of unequal size, as projections give them
    gain = 1.0 + 7.0 * (torch.rand((hkv, d), generator=gen, device="cuda") < 0.03).float()
    s["k_pool"] = torch.zeros((blocks + 1, block, hkv, _row_bytes(dtype, d)), dtype=torch.uint8, device="cuda")
    s["v_pool"] = torch.zeros_like(s["k_pool"])
    s["slots_total"] = blocks * block
    a_time = max(1, (1 << 27) // (block * hkv * d))
    for b in range(0, blocks, a_time) if op != "append" else ():
        n = min(a_time, blocks - b)
        size = torch.exp(0.3 * rnd(n, block, 1, 1))
        s["k_pool"][b : b + n] = _quantise(dtype, (rnd(n, block, hkv, d) * gain * size).bfloat16().float(), s["k_scale"])
        s["v_pool"][b : b + n] = _quantise(dtype, (rnd(n, block, hkv, d) * size).bfloat16().float(), s["v_scale"])
    if op in ("append", "step"):
        qkv = rnd(tokens, hq + 2 * hkv, d)  # a fused projection's output: rows at its stride
        qkv[:, hq : hq + hkv] *= gain
        qkv = qkv.to(torch.bfloat16)
        s["query"], s["key"], s["value"] = qkv[:, :hq], qkv[:, hq : hq + hkv], qkv[:, hq + hkv :]
        s["query_out"] = torch.empty((tokens, hq, d), dtype=torch.bfloat16, device="cuda")
        half = case["rotary"] // 2
        angle = torch.arange(MAX_POSITION, device="cuda").double()[:, None] * torch.pow(
            500000.0, -torch.arange(half, device="cuda").double() / half)
        s["cos_sin"] = torch.cat((torch.cos(angle), torch.sin(angle)), -1).float()
    if op == "append":
        # prompts of some hundred tokens, each from a position of its own
        each = torch.randint(0, MAX_POSITION - 1024, (tokens // 700 + 1,), generator=gen, device="cuda")
        i = torch.arange(tokens, device="cuda")
        s["positions"] = each[i // 700] + i % 700
        slots = perm.long()[:, None] * block + torch.arange(block, device="cuda")
        s["slots"] = slots.flatten()[:tokens].contiguous()
        if case["pad"]:
            s["slots"][tokens - min(case["pad"], tokens - 1):] = -1
        s["out"] = [torch.empty((tokens, hkv, d), dtype=torch.float32, device="cuda") for _ in range(2)]
    if op == "step":
        s["positions"] = s["token_pos"]
        row = s["table"].long()[s["token_req"], s["token_pos"] // block]
        s["slots"] = row * block + s["token_pos"] % block
    if op in ("shared", "cross"):
        s["query"] = rnd(tokens, hq, d).to(torch.bfloat16)
    if op != "append":
        s["result"] = torch.empty((tokens, hq, d), dtype=torch.bfloat16, device="cuda")
        s["sm_scale"], s["cap"], s["window"] = 1.0 / math.sqrt(d), case["cap"], case["window"]
        s["slopes"] = torch.exp2(-8.0 * (torch.arange(hq, device="cuda") + 1.0) / hq) if case["alibi"] else None
        s["sinks"] = 2.0 * rnd(hq) if case["sinks"] else None
    if own:
        from int8_kv_cache_reshape_gb300 import kvq

        kc, vc = s["k_pool"][:blocks], s["v_pool"][:blocks]
        if op in ("append", "step"):
            s["write"] = kvq.prepare_rotary_and_cache(
                s["query"], s["key"], s["value"], s["positions"], s["cos_sin"], s["query_out"], kc, vc, s["slots"],
                dtype, s["interleaved"], s["k_scale"], s["v_scale"])
        if op == "append":
            s["read"] = kvq.prepare_gather_cache(kc, vc, s["slots"], s["out"][0], s["out"][1], dtype, s["k_scale"],
                                                 s["v_scale"])
            return s
        lens, starts = s["lens"].cpu(), s["qsl"].cpu()
        if op == "cross":
            s["plan"] = kvq.get_cross_attention_metadata(len(batch), hq, hkv, d, lens, starts, dtype)
        else:
            s["plan"] = kvq.get_shared_prefix_metadata(len(batch), hq, hkv, d, lens, starts, prefixes,
                                                       [p for _, _, p in batch], case["window"], dtype)
        s["scratch"] = torch.empty(max(256, s["plan"].workspace_bytes), dtype=torch.uint8, device="cuda")
        s["attend"] = kvq.prepare_attention_with_kv_cache(
            s["plan"], s["query_out"] if op == "step" else s["query"], kc, vc, s["qsl"], s["lens"], s["table"],
            s["sm_scale"], op != "cross", case["window"], case["cap"], s["k_scale"], s["v_scale"], s["result"],
            s["scratch"], dtype, hkv, alibi_slopes=s["slopes"], sinks=s["sinks"])
    return s


def run(s):
    op = s["op"]
    if own:
        if op == "append":
            s["write"]()
            s["read"]()
            return {"query": s["query_out"], "key": s["out"][0], "value": s["out"][1]}
        if op == "step":
            s["write"]()
        s["attend"]()
        return {"out": s["result"], "query": s["query_out"]} if op == "step" else {"out": s["result"]}
    if op == "append":
        q = _append(s)
        live = (s["slots"] >= 0)[:, None, None]
        at = s["slots"].clamp(min=0)
        return {"query": q, "key": torch.where(live, _rows(s, "k", at), 0.0),
                "value": torch.where(live, _rows(s, "v", at), 0.0)}
    if op == "cross":
        return {"out": _cross(s, s["query"])}
    if op == "shared":
        return {"out": _shared(s, s["query"])}
    q = _append(s)
    return {"out": _shared(s, q), "query": q}


def work(case):
    batch, prefixes = _lens(case)
    hq, hkv, d, block, row = (case["heads_q"], case["heads_kv"], case["dim"], case["block"],
                              _row_bytes(case["dtype"], case["dim"]))

    def append(t, live):
        # queries, keys and values in, their positions, slots and cos / sin rows; queries and cache rows out
        return t * ((2 * hq + 2 * hkv) * d * 2 + 16 + 4 * case["rotary"]) + 2 * live * hkv * row

    if case["op"] == "append":
        t = case["tokens"]
        live = t - min(case["pad"], t - 1) if case["pad"] else t
        # and the rows read back: cache rows in, fp32 values out
        return {"bytes": append(t, live) + 8 * t + 2 * hkv * (live * row + 4 * t * d), "flops": 0}
    tokens = sum(new for _, new, _ in batch)
    pairs, keys, blocks = 0, 0, 0
    seen = [prefixes[p] for p in range(len(prefixes))]  # first key of each prefix that a row sees
    used = set()
    for n, new, p in batch:
        if case["op"] == "cross":
            pairs, keys, blocks = pairs + n * new, keys + n, blocks + -(-n // block)
            continue
        w = case["window"] or n
        held = prefixes[p] if p >= 0 else 0
        low = max(0, n - new - w + 1)
        keys += n - max(low, held)
        if p >= 0:
            seen[p] = min(seen[p], low)
            used.add(p)
        pairs += sum(min(n - new + 1 + i, w) for i in range(new))
        blocks += -(-n // block)
    keys += sum(prefixes[p] - seen[p] for p in used)
    total = 2 * keys * hkv * row + 4 * tokens * hq * d + 4 * blocks
    if case["op"] == "step":
        total += append(tokens, tokens) - 2 * tokens * hq * d  # (the rotated queries stay where they are needed)
    return {"bytes": total, "flops": 4 * d * hq * pairs}


# ---- from the definition, in 64 bits -------------------------------------------------


def _r32(v):
    return v.float().double()


def _decode64(dtype, rows, d, scale):
    """Values of cache rows: codes taken apart bit by bit."""
    rows = rows.contiguous()
    if dtype == "auto":
        return rows.view(torch.bfloat16).double()
    if dtype == "int4_per_token_head":
        words = rows[..., : d // 2].contiguous().view(torch.int32).long() & 0xFFFFFFFF
        out = torch.zeros((*rows.shape[:-1], d), dtype=torch.float64, device=rows.device)
        for j in range(8):
            dim = 2 * j if j < 4 else 2 * (j - 4) + 1
            out[..., dim::8] = (((words >> (4 * j)) & 15) - 8).double()
        for g in range(8):
            out[..., g * d // 8 : (g + 1) * d // 8] *= rows[..., d // 2 + 4 + g : d // 2 + 5 + g].double()
        return out * rows[..., d // 2 : d // 2 + 4].contiguous().view(torch.float32).double()
    c = rows[..., :d].long()
    if dtype.startswith("int8"):
        v = (c - 256 * (c > 127)).double()
    else:
        bits, bias = (2, 15) if "e5m2" in dtype else (3, 7)
        e, m = (c & 127) >> bits, (c & ((1 << bits) - 1)).double() / (1 << bits)
        v = torch.where(e > 0, torch.ldexp(1.0 + m, e - bias), torch.ldexp(m, torch.full_like(e, 1 - bias)))
        v = torch.where(c > 127, -v, v)
    by = rows[..., d : d + 4].contiguous().view(torch.float32).double() if "per_token" in dtype else float(scale)
    return v * by


def _nearest(dtype, y):
    """The code value nearest to y (64 bits), ties to even."""
    if dtype.startswith("int8"):
        return torch.round(y).clamp(-128, 127)
    bits, least, top = (2, -14, 57344.0) if "e5m2" in dtype else (3, -6, 448.0)
    y = y.clamp(-top, top)
    e = (torch.frexp(y)[1] - 1).clamp(min=least)  # |y| in [2^e, 2^(e + 1))
    step = torch.ldexp(torch.ones_like(y), e - bits)
    return (torch.round(y / step) * step).clamp(-top, top)


def _encode64(dtype, x, scale):
    """Values that rows x [..., D] stand for once stored.  Each division and product is
    the exact one rounded to 32 bits, as the formats define them."""
    if dtype == "auto":
        return x.bfloat16().double()
    if "per_token" not in dtype:
        by = torch.tensor(scale, dtype=torch.float32).double().item()
        return _nearest(dtype, _r32(x / by)) * by
    d = x.shape[-1]
    if dtype != "int4_per_token_head":
        s = _r32(x.abs().max(-1, keepdim=True).values / QMAX[dtype])
        return torch.where(s > 0, _nearest(dtype, _r32(x / torch.where(s > 0, s, 1.0))) * s, 0.0)
    s = _r32(x.abs().max(-1, keepdim=True).values / 889.0)
    out = torch.zeros_like(x)
    for g in range(8):
        y = x[..., g * d // 8 : (g + 1) * d // 8]
        top = y.abs().max(-1, keepdim=True).values
        m = torch.ceil(_r32(_r32(top / s) / 7.0)).clamp(max=127.0)
        code = torch.round(_r32(y / _r32(s * m))).clamp(-7, 7)
        out[..., g * d // 8 : (g + 1) * d // 8] = torch.where((s > 0) & (m > 0), s * (m * code), 0.0)
    return out


def _turn64(s, x):
    """Rows [T, H, D] rotated, dim by dim, products and sums rounded to 32 bits as the operator defines them."""
    x = x.double()
    half = s["rotary"] // 2
    dims = torch.arange(s["rotary"], device="cuda")
    pair, second = (dims // 2, dims % 2) if s["interleaved"] else (dims % half, dims // half)
    other = (dims ^ 1) if s["interleaved"] else (dims + half) % (2 * half)
    table = s["cos_sin"].double()[s["positions"]]
    c, n = table[:, pair][:, None], table[:, half + pair][:, None]
    sign = torch.where(second == 0, -1.0, 1.0).double()
    turned = _r32(_r32(x[..., : s["rotary"]] * c) + sign * _r32(x[..., other] * n))
    return torch.cat((turned, x[..., s["rotary"] :]), -1)


def exact(case, seed):
    s = prepare(case, seed)
    dtype, d, hkv, block = s["dtype"], s["dim"], s["heads_kv"], s["block"]
    if case["op"] in ("append", "step"):
        query = _turn64(s, s["query"])
        new_k = _encode64(dtype, _turn64(s, s["key"]), s["k_scale"])
        new_v = _encode64(dtype, s["value"].double(), s["v_scale"])
        if case["op"] == "append":
            live = (s["slots"] >= 0)[:, None, None]
            return {"query": query, "key": torch.where(live, new_k, 0.0), "value": torch.where(live, new_v, 0.0)}
        q = query.bfloat16().double()
    else:
        q = s["query"].double()
    batch, prefixes = _lens(case)
    group = case["heads_q"] // hkv
    kc, vc = s["k_pool"].flatten(0, 1), s["v_pool"].flatten(0, 1)
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    table = s["table"].tolist()

    def rows(r, lo, hi):
        ids = torch.tensor(table[r][lo // block : -(-hi // block)], dtype=torch.long, device="cuda")
        at = (ids[:, None] * block + torch.arange(block, device="cuda")).flatten()[: hi - lo]
        return _decode64(dtype, kc[at], d, s["k_scale"]), _decode64(dtype, vc[at], d, s["v_scale"])

    known = {}
    t = 0
    for r, (n, new, p) in enumerate(batch):
        begin = prefixes[p] if p >= 0 else 0
        if n == 0:
            t += new
            continue
        k, v = rows(r, begin, n)
        if case["op"] == "step":
            k[n - new - begin :], v[n - new - begin :] = new_k[t : t + new], new_v[t : t + new]
        if begin:
            if p not in known:
                known[p] = rows(r, 0, begin)
        far = torch.arange(n, device="cuda") - torch.arange(n - new, n, device="cuda")[:, None]  # key - query
        hidden = torch.zeros_like(far, dtype=torch.bool)
        if case["op"] != "cross":
            hidden = far > 0
            if case["window"]:
                hidden |= far <= -case["window"]
        for h in range(hkv):
            kh = torch.cat((known[p][0][:, h], k[:, h])) if begin else k[:, h]
            vh = torch.cat((known[p][1][:, h], v[:, h])) if begin else v[:, h]
            z = torch.einsum("qgd,kd->qgk", q[t : t + new, h * group : (h + 1) * group], kh) / math.sqrt(d)
            if case["cap"]:
                z = case["cap"] * torch.tanh(z / case["cap"])
            if s["slopes"] is not None:
                z = z + s["slopes"][h * group : (h + 1) * group].double()[None, :, None] * far[:, None].double()
            z[hidden[:, None].expand_as(z)] = float("-inf")
            if s["sinks"] is not None:
                z = torch.cat((z, s["sinks"][h * group : (h + 1) * group].double().view(1, group, 1).expand(new, group, 1)), -1)
            w = torch.exp(z - z.max(-1, keepdim=True).values)
            w = w / w.sum(-1, keepdim=True)
            out[t : t + new, h * group : (h + 1) * group] = torch.einsum("qgk,kd->qgd", w[..., :n], vh)
        t += new
    return {"out": out, "query": query} if case["op"] == "step" else {"out": out}
