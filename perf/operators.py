"""The attention operators' workloads: inputs, one pass of each, and what a pass has to move and compute.

    kv_write      rotary positions on fresh q and k, q handed on, k and v written into a paged cache
    kv_chunk      the same into an 8-bit (or 16-bit) cache, then the sequences read back from it packed, as a prompt
                  that arrives in chunks needs them
    attn_decode   one new token of every sequence over the paged cache
    attn_prompt   packed prompts of different lengths, grouped heads, causal or not

A cache is k_pages [pages][kv heads][slots][d] and v_pages [pages][kv heads][d][slots], in bf16, fp16, or int8 with one
fp32 step for every token and head ([pages][kv heads][slots]); slot = page * page_size + offset.  With own = False a pass
is plain torch arithmetic in 32 bits; with own = True it makes the package's calls.  exact() gives the same outputs from
the definitions in 64 bits."""
import math
import random

import torch

own = False

DEVICE = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "i8": torch.int8}
SIZES = {"f32": 4, "bf16": 2, "f16": 2, "i8": 1}


# ------------------------------------------------------------------- cases ----

def _write(name, *, tokens, hq, hkv, d, src, q, cache, page, rot, mix):
    return {"name": name, "op": "kv_write", "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "src": src, "q": q,
            "cache": cache, "page": page, "rot": rot, "mix": mix}


def _chunk(name, *, batch, new, context, hq, hkv, d, src, q, cache, page, rot, mix):
    return {"name": name, "op": "kv_chunk", "batch": batch, "new": new, "context": context, "hq": hq, "hkv": hkv,
            "d": d, "src": src, "q": q, "cache": cache, "page": page, "rot": rot, "mix": mix}


def _decode(name, *, batch, low, high, hq, hkv, d, q, cache, page, mix):
    return {"name": name, "op": "attn_decode", "batch": batch, "low": low, "high": high, "hq": hq, "hkv": hkv, "d": d,
            "q": q, "cache": cache, "page": page, "mix": mix}


def _prompt(name, *, batch, low, high, before, hq, hkv, d, dtype, causal, mix):
    return {"name": name, "op": "attn_prompt", "batch": batch, "low": low, "high": high, "before": before, "hq": hq,
            "hkv": hkv, "d": d, "dtype": dtype, "causal": causal, "mix": mix}


def listed():
    return [
        # the single-token step of one conversation: fp32 rows from the decode matvecs, nothing but latency
        _write("write_one_token", tokens=1, hq=40, hkv=8, d=128, src="f32", q="f32", cache="bf16", page=64, rot=128,
               mix=1),
        # packed prompts behind the prefill projections, 256-wide heads of which a quarter turns
        _write("write_prompts_d256", tokens=8191, hq=24, hkv=4, d=256, src="f32", q="bf16", cache="bf16", page=64,
               rot=64, mix=2),
        # a handful of short odd chunks into an 8-bit cache with small pages
        _chunk("chunk_small_i8", batch=3, new=45, context=201, hq=14, hkv=2, d=64, src="f32", q="bf16", cache="i8",
               page=16, rot=64, mix=3),
        # chunks of long prompts: a few hundred new tokens each behind contexts of many thousands, read back whole
        _chunk("chunk_long_i8", batch=8, new=512, context=12000, hq=40, hkv=8, d=128, src="f32", q="bf16", cache="i8",
               page=64, rot=128, mix=4),
        # the first tokens of one conversation, fp32 activations throughout: latency
        _decode("decode_one_short", batch=1, low=77, high=77, hq=40, hkv=8, d=128, q="f32", cache="bf16", page=64,
                mix=5),
        # a serving batch with lengths from a few tokens to the limit
        _decode("decode_batch_ragged", batch=64, low=3, high=8190, hq=32, hkv=8, d=128, q="bf16", cache="bf16",
                page=16, mix=6),
        # one very long conversation over an 8-bit cache
        _decode("decode_one_long_i8", batch=1, low=131071, high=131071, hq=40, hkv=8, d=128, q="f32", cache="i8",
                page=64, mix=7),
        # wide heads, few key heads, fp16
        _decode("decode_batch_d256_f16", batch=16, low=900, high=5000, hq=24, hkv=4, d=256, q="f16", cache="f16",
                page=32, mix=8),
        # one short question: latency
        _prompt("prompt_short", batch=1, low=33, high=33, before=0, hq=40, hkv=8, d=128, dtype="bf16", causal=True,
                mix=9),
        # a packed batch of prompts of very different lengths
        _prompt("prompts_packed", batch=9, low=5, high=2500, before=0, hq=32, hkv=8, d=128, dtype="bf16", causal=True,
                mix=10),
        # one long document
        _prompt("prompt_long", batch=1, low=16384, high=16384, before=0, hq=40, hkv=8, d=128, dtype="bf16",
                causal=True, mix=11),
        # chunks of wide-headed prompts behind what a cache holds already, fp16
        _prompt("prompt_chunks_d256_f16", batch=4, low=130, high=700, before=4000, hq=24, hkv=4, d=256, dtype="f16",
                causal=True, mix=12),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 5, 6, 7, 8])
    d = rng.choice([64, 128, 256])
    heads = {"hq": hkv * group, "hkv": hkv, "d": d}
    page = rng.choice([16, 32, 64, 128])
    mix = rng.randrange(1 << 30)
    op = rng.choice(["kv_write", "kv_chunk", "attn_decode", "attn_decode", "attn_prompt", "attn_prompt"])
    sixteen = rng.choice(["bf16", "f16"])
    cache = rng.choice([sixteen, sixteen, "i8"])
    q = rng.choice([sixteen, "f32"])
    src = rng.choice(["f32", "f32", sixteen])
    rot = rng.choice([0, d // 4, d // 2, d])
    if op == "kv_write":
        case = _write("", tokens=_log(rng, 1, 8000), src=src, q=q, cache=sixteen, page=page, rot=rot, mix=mix, **heads)
    elif op == "kv_chunk":
        case = _chunk("", batch=_log(rng, 1, 8), new=_log(rng, 1, 600), context=_log(rng, 1, 12000), src=src, q=q,
                      cache=cache, page=page, rot=rot, mix=mix, **heads)
    elif op == "attn_decode":
        batch = _log(rng, 1, 64)
        high = _log(rng, 1, min(131072, 400000 // batch))
        case = _decode("", batch=batch, low=_log(rng, 1, high), high=high, q=q, cache=cache, page=page, mix=mix,
                       **heads)
    else:
        batch = _log(rng, 1, 9)
        high = _log(rng, 1, 12000 // batch)
        case = _prompt("", batch=batch, low=_log(rng, 1, high), high=high, before=rng.choice([0, 0, _log(rng, 1, 4000)]),
                       dtype=sixteen, causal=rng.random() < 0.8, mix=mix, **heads)
    del case["name"]
    return case


def _lengths(case):
    """Tokens of every sequence: spread over [low, high] on a logarithmic scale, the first one the longest."""
    rng = random.Random(case["mix"])
    out = [_log(rng, case["low"], case["high"]) for _ in range(case["batch"])]
    out[0] = case["high"]
    return out


def _chunk_lengths(case):
    """(new tokens, tokens in the cache with them) of every sequence."""
    rng = random.Random(case["mix"])
    new = [rng.randint(max(1, case["new"] // 2), case["new"]) for _ in range(case["batch"])]
    old = [rng.randint(case["context"] // 2, case["context"]) for _ in range(case["batch"])]
    return new, [a + b for a, b in zip(new, old)]


def _pairs(lq, lk, causal):
    """Query-key pairs that see each other when the last query sees the last key."""
    if not causal:
        return lq * lk
    hidden = lq - 1 if lk >= lq else 0
    if lk >= lq:
        return lq * lk - hidden * (hidden + 1) // 2
    return lk * (lk + 1) // 2


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] in ("kv_write", "kv_chunk"):
        tokens = case["tokens"] if case["op"] == "kv_write" else sum(_chunk_lengths(case)[0])
        cell = d * SIZES[case["cache"]] + (4 if case["cache"] == "i8" else 0)
        moved = tokens * ((hq + 2 * hkv) * d * SIZES[case["src"]] + hq * d * SIZES[case["q"]] + 2 * hkv * cell + 8)
        moved += tokens * case["rot"] * 4 + (tokens * 4 if case["rot"] else 0)
        flops = 3 * tokens * (hq + hkv) * case["rot"]
        if case["op"] == "kv_chunk":
            total = sum(_chunk_lengths(case)[1])
            moved += 2 * total * hkv * (cell + d * 2)
            flops += 2 * total * hkv * d
        return {"bytes": moved, "flops": flops}
    if case["op"] == "attn_decode":
        total = sum(_lengths(case))
        cell = d * SIZES[case["cache"]] + (4 if case["cache"] == "i8" else 0)
        return {"bytes": 2 * total * hkv * cell + 2 * case["batch"] * hq * d * SIZES[case["q"]],
                "flops": 4 * total * hq * d}
    lens = _lengths(case)
    moved = 2 * sum(lens) * hq * d * 2 + 2 * sum(n + case["before"] for n in lens) * hkv * d * 2
    return {"bytes": moved, "flops": 4 * hq * d * sum(_pairs(n, n + case["before"], case["causal"]) for n in lens)}


# ------------------------------------------------------------------ inputs ----

def _channels(gen, d):
    """A gain for every dimension of a head: a few of them several times the others, as trained keys have."""
    gain = torch.ones(d, device=DEVICE)
    gain[torch.randperm(d, generator=gen, device=DEVICE)[: max(1, d // 32)]] = 4.0
    return gain


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32)


def _quantised(x, dim):
    """int8 codes and fp32 steps of x along dim (one step for every token and head)."""
    top = x.abs().amax(dim=dim, keepdim=True)
    return torch.round(x * (127.0 / top)).to(torch.int8), (top / 127.0).squeeze(dim)


def _filled_cache(gen, case, pages):
    hkv, d, page = case["hkv"], case["d"], case["page"]
    k = _normal(gen, pages, hkv, page, d) * _channels(gen, d)
    v = _normal(gen, pages, hkv, d, page)
    if case["cache"] == "i8":
        k, ks = _quantised(k, 3)
        v, vs = _quantised(v, 2)
        return {"k": k, "v": v, "ks": ks, "vs": vs}
    dtype = DTYPES[case["cache"]]
    return {"k": k.to(dtype), "v": v.to(dtype), "ks": None, "vs": None}


def _tables(gen, lens, page, spare):
    """Pages for every sequence in a random order, and the number of pages of the cache."""
    counts = [max(1, -(-n // page)) for n in lens]
    pages = sum(counts) + spare
    order = torch.randperm(pages, generator=gen, device=DEVICE).to(torch.int32)
    table = torch.zeros((len(lens), max(counts)), dtype=torch.int32, device=DEVICE)
    at = 0
    for row, n in enumerate(counts):
        table[row, :n] = order[at:at + n]
        at += n
    return table, pages


def _cumulated(lens):
    at, out = 0, [0]
    for n in lens:
        at += n
        out.append(at)
    return torch.tensor(out, dtype=torch.int32, device=DEVICE)


def _rope_table(positions, rot):
    """[positions][rot]: rot / 2 cosines, then rot / 2 sines."""
    half = rot // 2
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEVICE) / half)
    angle = torch.arange(positions, dtype=torch.float64, device=DEVICE)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], dim=1).to(torch.float32)


def _inputs(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed * 7919 + 13)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    s = {"case": case}
    if case["op"] in ("kv_write", "kv_chunk"):
        page = case["page"]
        if case["op"] == "kv_write":
            # whole prompts, each from its first position: about 1500 tokens apiece
            tokens = case["tokens"]
            new = [min(1500, tokens - at) for at in range(0, tokens, 1500)]
            lens = new if tokens > 1 else [777]
        else:
            new, lens = _chunk_lengths(case)
        table, pages = _tables(gen, lens, page, 3)
        positions = torch.cat([torch.arange(n - m, n, device=DEVICE) for m, n in zip(new, lens)])
        rows = torch.repeat_interleave(torch.arange(len(new), device=DEVICE), torch.tensor(new, device=DEVICE))
        s["slots"] = table[rows, positions // page].to(torch.int64) * page + positions % page
        s["positions"] = positions.to(torch.int32)
        s["rope"] = _rope_table(max(lens), case["rot"]) if case["rot"] else None
        # the stacked projection's rows: q, k and v are views of them
        x = _normal(gen, positions.numel(), (hq + 2 * hkv), d)
        x[:, hq:hq + hkv] *= _channels(gen, d)
        x = x.to(DTYPES[case["src"]])
        s["q"], s["k"], s["v"] = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        s["cache"] = _filled_cache(gen, case, pages)
        s["table"], s["lens"] = table, lens
        s["cu"] = _cumulated(lens)
    elif case["op"] == "attn_decode":
        lens = _lengths(case)
        s["table"], pages = _tables(gen, lens, case["page"], 3)
        s["cache"] = _filled_cache(gen, case, pages)
        s["q"] = _normal(gen, case["batch"], hq, d).to(DTYPES[case["q"]])
        s["lens"] = lens
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEVICE)
    else:
        lq = _lengths(case)
        lk = [n + case["before"] for n in lq]
        dtype = DTYPES[case["dtype"]]
        s["q"] = _normal(gen, sum(lq), hq, d).to(dtype)
        s["k"] = (_normal(gen, sum(lk), hkv, d) * _channels(gen, d)).to(dtype)
        s["v"] = _normal(gen, sum(lk), hkv, d).to(dtype)
        s["lq"], s["lk"] = lq, lk
        s["cu_q"], s["cu_k"] = _cumulated(lq), _cumulated(lk)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own and "cache" in s:
        import ternary_weight_ptq1_amd as P

        c = s["cache"]
        s["kv"] = P.KvCache(c["k"], c["v"], c["ks"], c["vs"])
    return s


# ----------------------------------------------------------- the plain form ----

def _turn(x, positions, table):
    """Rotary positions on the first rot dimensions of x [tokens][heads][d], in fp32."""
    x = x.float()
    if table is None:
        return x
    half = table.shape[1] // 2
    row = table[positions.long()][:, None]
    cos, sin = row[..., :half], row[..., half:]
    a, b = x[..., :half], x[..., half:2 * half]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., 2 * half:]], dim=-1)


def _plain_write(s):
    case, cache = s["case"], s["cache"]
    page = case["page"]
    q = _turn(s["q"], s["positions"], s["rope"]).to(DTYPES[case["q"]])
    k = _turn(s["k"], s["positions"], s["rope"])
    v = s["v"].float()
    at, off = s["slots"] // page, s["slots"] % page
    if case["cache"] == "i8":
        k, ks = _quantised(k, 2)
        v, vs = _quantised(v, 2)
        cache["ks"][at, :, off] = ks
        cache["vs"][at, :, off] = vs
    cache["k"][at, :, off] = k.to(cache["k"].dtype)
    cache["v"][at, :, :, off] = v.to(cache["v"].dtype)
    return q


def _pages_of(cache, rows):
    """K and V [pages][kv heads][slots][d] in fp32 of the pages named by rows."""
    k, v = cache["k"][rows].float(), cache["v"][rows].float().transpose(-1, -2)
    if cache["ks"] is not None:
        k, v = k * cache["ks"][rows][..., None], v * cache["vs"][rows][..., None]
    return k, v


def _plain_read(s, dtype):
    case, hkv, d = s["case"], s["case"]["hkv"], s["case"]["d"]
    ks, vs = [], []
    for row, n in enumerate(s["lens"]):
        k, v = _pages_of(s["cache"], s["table"][row, :-(-n // case["page"])])
        ks.append(k.transpose(1, 2).reshape(-1, hkv, d)[:n].to(dtype))
        vs.append(v.transpose(1, 2).reshape(-1, hkv, d)[:n].to(dtype))
    return torch.cat(ks), torch.cat(vs)


def _softmax(scores):
    e = torch.exp(scores - scores.amax(dim=-1, keepdim=True))
    return e / e.sum(dim=-1, keepdim=True)


def _plain_decode(s):
    case = s["case"]
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    pages = -(-max(s["lens"]) // page)
    at_once = max(1, (1 << 29) // (pages * page * hkv * d))
    out = []
    for b in range(0, case["batch"], at_once):
        table, lens = s["table"][b:b + at_once, :pages], s["seq_lens"][b:b + at_once]
        k, v = _pages_of(s["cache"], table)
        n = table.shape[0]
        k = k.transpose(1, 2).reshape(n, hkv, pages * page, d)
        v = v.transpose(1, 2).reshape(n, hkv, pages * page, d)
        q = s["q"][b:b + at_once].float().view(n, hkv, hq // hkv, d)
        scores = torch.matmul(q, k.transpose(-1, -2)) * d ** -0.5
        hidden = torch.arange(pages * page, device=q.device) >= lens[:, None]
        weights = _softmax(scores.masked_fill(hidden[:, None, None], float("-inf")))
        out.append(torch.matmul(weights, v).view(n, hq, d))
    return torch.cat(out).to(s["q"].dtype)


def _plain_prompt(s):
    case = s["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    group = hq // hkv
    out, at_q, at_k = [], 0, 0
    for lq, lk in zip(s["lq"], s["lk"]):
        q = s["q"][at_q:at_q + lq].float().view(lq, hkv, group, d).permute(1, 2, 0, 3)
        k = s["k"][at_k:at_k + lk].float().permute(1, 2, 0).contiguous()[:, None]
        v = s["v"][at_k:at_k + lk].float().transpose(0, 1).contiguous()[:, None]
        rows = max(1, (1 << 28) // (hq * lk))
        for first in range(0, lq, rows):
            last = min(lq, first + rows)
            seen = lk - lq + last if case["causal"] else lk
            scores = torch.matmul(q[:, :, first:last], k[..., :seen]) * d ** -0.5
            if case["causal"]:
                row = torch.arange(first, last, device=q.device)[:, None] + (lk - lq)
                scores = scores.masked_fill(torch.arange(seen, device=q.device) > row, float("-inf"))
            o = torch.matmul(_softmax(scores), v[:, :, :seen])
            out.append(o.permute(2, 0, 1, 3).reshape(last - first, hq, d).to(s["q"].dtype))
        at_q += lq
        at_k += lk
    return torch.cat(out)


# ---------------------------------------------------------------- one pass ----

def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        import ternary_weight_ptq1_amd as P

        if op == "attn_decode":
            return P.ptq1_attn_decode(s["q"], s["kv"], s["table"], s["seq_lens"], max_len=case["high"])
        if op == "attn_prompt":
            return P.ptq1_attn_prompt(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], max_q=case["high"],
                                      max_k=case["high"] + case["before"], causal=case["causal"])
        q = P.ptq1_kv_write(s["q"], s["k"], s["v"], s["slots"], s["kv"], positions=s["positions"], cos_sin=s["rope"],
                            q_dtype=DTYPES[case["q"]])
        if op == "kv_write":
            return q, s["cache"]["k"], s["cache"]["v"]
        k, v = P.ptq1_kv_read(s["kv"], s["table"], s["cu"], sum(s["lens"]), dtype=_read_type(case))
        return q, k, v
    if op == "attn_decode":
        return _plain_decode(s)
    if op == "attn_prompt":
        return _plain_prompt(s)
    q = _plain_write(s)
    if op == "kv_write":
        return q, s["cache"]["k"], s["cache"]["v"]
    k, v = _plain_read(s, _read_type(case))
    return q, k, v


def _read_type(case):
    """What the prompt attention behind the cache takes: the cache's own 16-bit type, bf16 for 8 bits."""
    return DTYPES["bf16" if case["cache"] == "i8" else case["cache"]]


# ------------------------------------------------------- the definitions ----

def _exact_heads(q, k, v, visible):
    """softmax(q k / sqrt(d)) v of one head in fp64; visible(first, last) masks rows first..last (None: all)."""
    n, d = q.shape
    out = torch.zeros((n, v.shape[1]), dtype=torch.float64, device=q.device)
    step = max(1, (1 << 26) // max(1, k.shape[0]))
    for first in range(0, n, step):
        last = min(n, first + step)
        logits = q[first:last] @ k.T.contiguous() / math.sqrt(d)
        mask = visible(first, last)
        if mask is not None:
            logits[~mask] = -math.inf
        weights = torch.softmax(logits, dim=1)
        out[first:last] = weights @ v
    return out


def _exact_turn(x, positions, table):
    x = x.double().clone()
    if table is not None:
        half = table.shape[1] // 2
        for at in range(half):
            c, sn = table[positions.long(), at].double()[:, None], table[positions.long(), half + at].double()[:, None]
            a, b = x[:, :, at].clone(), x[:, :, half + at].clone()
            x[:, :, at] = a * c - b * sn
            x[:, :, half + at] = a * sn + b * c
    return x


def exact(case, seed):
    s = _inputs(case, seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    group = hq // hkv
    if case["op"] == "attn_prompt":
        out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEVICE)
        at_q = at_k = 0
        for lq, lk in zip(s["lq"], s["lk"]):
            def visible(first, last):
                if not case["causal"]:
                    return None
                i = torch.arange(first, last, device=DEVICE)[:, None]
                return torch.arange(lk, device=DEVICE)[None] - (lk - lq) <= i

            for h in range(hq):
                out[at_q:at_q + lq, h] = _exact_heads(s["q"][at_q:at_q + lq, h].double(),
                                                      s["k"][at_k:at_k + lk, h // group].double(),
                                                      s["v"][at_k:at_k + lk, h // group].double(), visible)
            at_q += lq
            at_k += lk
        return out
    cache, page = s["cache"], case["page"]
    k, v = cache["k"].double(), cache["v"].double()
    if cache["ks"] is not None:
        k *= cache["ks"].double()[:, :, :, None]
        v *= cache["vs"].double()[:, :, None, :]
    if case["op"] == "attn_decode":
        out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEVICE)
        for b, n in enumerate(s["lens"]):
            rows = s["table"][b, :-(-n // page)].long()
            for h in range(hkv):
                kk = k[rows, h].reshape(-1, d)[:n]
                vv = v[rows, h].permute(0, 2, 1).reshape(-1, d)[:n]
                out[b, h * group:(h + 1) * group] = _exact_heads(s["q"][b, h * group:(h + 1) * group].double(), kk, vv,
                                                                 lambda first, last: None)
        return out
    q = _exact_turn(s["q"], s["positions"], s["rope"])
    kn, vn = _exact_turn(s["k"], s["positions"], s["rope"]), s["v"].double()
    if case["cache"] == "i8":
        for x in (kn, vn):
            step = x.abs().amax(dim=2, keepdim=True) / 127.0
            x.copy_(torch.round(x / step) * step)
    at, off = torch.div(s["slots"], page, rounding_mode="floor"), s["slots"] % page
    k[at, :, off] = kn
    v[at, :, :, off] = vn
    if case["op"] == "kv_write":
        return q, k, v
    ks, vs = [], []
    for b, n in enumerate(s["lens"]):
        place = torch.arange(n, device=DEVICE)
        rows = s["table"][b, torch.div(place, page, rounding_mode="floor")].long()
        ks.append(k[rows, :, place % page])
        vs.append(v[rows, :, :, place % page])
    return q, torch.cat(ks), torch.cat(vs)
