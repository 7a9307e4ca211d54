"""Cases for measuring the 4-bit KV cache: writing it, reading it back and attending over it.

A cache row (one token of one kv head, K or V) is a record of
16 * (1 + ceil(D / 32)) bytes: scale and minimum of each group of 32 values in
the first 16 bytes, then 16 bytes of codes per group.  ``own`` False computes
everything from elementary torch operations in fp32, ``own`` True through this
package's public calls.
"""
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # One generated token per sequence of a batch on a paged cache, stored and read back:
        # the smallest call, all latency.
        dict(name="store-token", kind="store", dtype="bf16", B=16, Hkv=8, D=128, cap=4608, n=1,
             ragged=False, page=64),
        # The prompts of a small batch on a contiguous cache.
        dict(name="store-prompt", kind="store", dtype="bf16", B=4, Hkv=8, D=128, cap=8192, n=4096,
             ragged=False, page=0),
        # A padded batch of prompts of different lengths, 64-wide heads, pages that end inside it.
        dict(name="store-padded", kind="store", dtype="fp16", B=8, Hkv=2, D=64, cap=2048, n=777,
             ragged=True, page=128),
        # Whole sequences taken back to 16 bits.
        dict(name="read-long", kind="read", dtype="bf16", B=8, Hkv=8, D=128, cap=8192, n=8192,
             ragged=False, page=0),
        # The same from a paged cache with ragged lengths and a head dim that is no multiple of 32.
        dict(name="read-odd", kind="read", dtype="fp16", B=3, Hkv=4, D=80, cap=1280, n=1001,
             ragged=True, page=64),
        # One short sequence: the smallest attention call.
        dict(name="attend-short", kind="attend", dtype="bf16", B=1, Hq=8, Hkv=2, D=128, cap=333,
             Sq=1, causal=False, window=0, mask=False, ragged=False, page=0),
        # Decoding one layer of Mistral 7B's shape.
        dict(name="attend-decode", kind="attend", dtype="bf16", B=16, Hq=32, Hkv=8, D=128,
             cap=4096, Sq=1, causal=False, window=0, mask=False, ragged=False, page=0),
        # Decoding one layer of Llama 2 70B's shape over a long context: the largest call.
        dict(name="attend-long", kind="attend", dtype="bf16", B=16, Hq=64, Hkv=8, D=128,
             cap=32768, Sq=1, causal=False, window=0, mask=False, ragged=False, page=0),
        # A serving batch: paged cache, every sequence at a length of its own, fp16.
        dict(name="attend-paged", kind="attend", dtype="fp16", B=32, Hq=32, Hkv=8, D=128,
             cap=8192, Sq=1, causal=False, window=0, mask=False, ragged=True, page=64),
        # Four drafted tokens per sequence scored at once, padding hidden by a mask.
        dict(name="attend-draft", kind="attend", dtype="bf16", B=8, Hq=32, Hkv=8, D=128, cap=6001,
             Sq=4, causal=True, window=0, mask=True, ragged=False, page=0),
        # A chunk of a prompt against all that came before it.
        dict(name="attend-chunk", kind="attend", dtype="bf16", B=2, Hq=32, Hkv=8, D=128,
             cap=16384, Sq=512, causal=True, window=0, mask=False, ragged=True, page=64),
        # A generation step of the 12-head, 2-group model with a sliding window: append, attend.
        dict(name="step-window", kind="step", dtype="bf16", B=16, Hq=12, Hkv=2, D=64, cap=2048,
             Sq=1, causal=True, window=1024, mask=False, ragged=True, page=0),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(["store", "read", "attend", "attend", "attend", "step"])
    c = dict(kind=kind, dtype=rng.choice(["bf16", "fp16"]), B=_spread(rng, 1, 32),
             Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([128, 128, 128, 64, 64, 96, 80, 40]),
             ragged=rng.random() < 0.5, page=rng.choice([0, 0, 64, 128, 256]))
    if kind in ("store", "read"):
        rows = max(1, (4 * 8 * 4096 if kind == "store" else 8 * 8 * 8192) // (c["B"] * c["Hkv"]))
        c["n"] = _spread(rng, 1, min(8192, rows))
        c["cap"] = c["n"] + _spread(rng, 1, 1024)
        return c
    c["Hq"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 6, 8, 8, 16])
    c["mask"] = rng.random() < 0.25
    c["Sq"] = 1
    if kind == "attend":
        c["Sq"] = rng.choice([1, 1, 1, _spread(rng, 2, 16), _spread(rng, 17, 1024)])
    most = 16 * 8 * 32768 // (c["B"] * c["Hkv"])
    if c["Sq"] > 1:  # no more products than the largest listed case has
        most = min(most, 16 * 64 * 32768 * 16 // (c["B"] * c["Hq"] * c["Sq"]))
    c["cap"] = max(c["Sq"] + 1, _spread(rng, 16, max(17, min(65536, most))))
    c["causal"] = c["Sq"] > 1 or rng.random() < 0.3
    c["window"] = _spread(rng, 16, 4096) if c["causal"] and rng.random() < 0.3 else 0
    return c


# ------------------------------------------------------------------ format

def _quantise(x, dtype):
    """fp32 rows [..., D] as (codes [..., G, 32], scale [..., G], minimum [..., G])."""
    D = x.shape[-1]
    G = -(-D // 32)
    # a last group of fewer than 32 values repeats its last one: same minimum and maximum
    x = torch.cat([x, x[..., -1:].expand(*x.shape[:-1], 32 * G - D)], -1).unflatten(-1, (G, 32))
    low, high = x.amin(-1), x.amax(-1)
    scale = ((high - low) / 15).to(dtype).float()
    step = torch.where(scale > 0, scale, torch.ones_like(scale))
    codes = ((x - low[..., None]) / step[..., None]).round().clamp(0, 15)
    return torch.where(scale[..., None] > 0, codes, torch.zeros_like(codes)), scale, low


def _pack(x, dtype):
    """fp32 rows [..., D] as records [..., 16 (1 + G)] of bytes."""
    D = x.shape[-1]
    codes, scale, low = _quantise(x, dtype)
    G = scale.shape[-1]
    keep = torch.arange(32 * G, device=x.device).view(G, 32) < D
    codes = (codes * keep).to(torch.uint8).flatten(-2)
    body = codes[..., 0::2] | (codes[..., 1::2] << 4)
    head = torch.zeros(*scale.shape[:-1], 16, dtype=torch.uint8, device=x.device)
    params = torch.stack([scale, low], -1).to(dtype).view(torch.uint8).flatten(-2)
    head[..., :4 * G] = params
    return torch.cat([head, body], -1)


def _unpack(records, D, dtype):
    """The fp32 values [..., D] that records stand for."""
    G = records.shape[-1] // 16 - 1
    params = records[..., :4 * G].contiguous().view(dtype).float().unflatten(-1, (G, 2))
    body = records[..., 16:]
    codes = torch.stack([body & 15, body >> 4], -1).float().flatten(-2).unflatten(-1, (G, 32))
    return (codes * params[..., :1] + params[..., 1:]).flatten(-2)[..., :D]


def _rows(cache, table):
    """The records of every sequence as [B, Hkv, capacity, R]."""
    if table is None:
        return cache
    return cache[table.long()].transpose(1, 2).flatten(2, 3)


def _write(s, cache, rows):
    """Records [B, Hkv, n, R] to rows lens[b] + t of the cache, t < count[b]."""
    B, _, n, _ = rows.shape
    t = torch.arange(n, device=rows.device)
    at = s["lens"].long()[:, None] + t
    count = s["after"].long() - s["lens"].long()
    b, t = (t < count[:, None]).nonzero(as_tuple=True)
    at = at[b, t]
    if s["table"] is None:
        cache[b, :, at] = rows[b, :, t]
    else:
        cache[s["table"].long()[b, at // s["page"]], :, at % s["page"]] = rows[b, :, t]


# ------------------------------------------------------------------ states

def _lengths(gen, case, least, most):
    if case["ragged"]:
        lens = torch.randint(least, most + 1, (case["B"],), generator=gen, device="cuda")
    else:
        lens = torch.full((case["B"],), most, device="cuda")
    return lens.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype, B, Hkv, D, cap = _DTYPES[case["dtype"]], case["B"], case["Hkv"], case["D"], case["cap"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    def rows(keys, n):
        # keys have channels that sit off zero, as projections with a bias and rotations leave them
        x = normal(B, Hkv, n, D)
        return (x + normal(1, Hkv, 1, D) if keys else x).to(dtype)

    s = dict(case, dtype=dtype, table=None)
    n = case["n"] if "n" in case else (1 if case["kind"] == "step" else 0)
    page = case["page"]
    pages = -(-cap // page) if page else 0
    if page:
        order = torch.randperm(B * pages + 3, generator=gen, device="cuda")[:B * pages]
        s["table"] = order.view(B, pages).to(torch.int32)
    caches = []
    for keys in (True, False):
        if case["kind"] == "store":
            shape = (B * pages + 3, Hkv, page) if page else (B, Hkv, cap)
            caches.append(torch.zeros(*shape, 16 * (1 + -(-D // 32)), dtype=torch.uint8,
                                      device="cuda"))
        elif page:
            pool = torch.zeros(B * pages + 3, Hkv, page, 16 * (1 + -(-D // 32)),
                               dtype=torch.uint8, device="cuda")
            rec = _pack(rows(keys, pages * page).float(), dtype)
            pool[s["table"].long()] = rec.unflatten(2, (pages, page)).transpose(1, 2)
            caches.append(pool)
        else:
            caches.append(_pack(rows(keys, cap).float(), dtype))
    s["cache_k"], s["cache_v"] = caches
    if case["kind"] in ("store", "step"):
        s["k_new"], s["v_new"] = rows(True, n), rows(False, n)
        s["lens"] = _lengths(gen, case, 0, cap - n)
        count = _lengths(gen, case, 1, n)
        s["count"] = count if case["kind"] == "store" and case["ragged"] else None
        s["after"] = s["lens"] + (count if s["count"] is not None else n)
    elif case["kind"] == "read":
        s["lens"] = _lengths(gen, case, 1, case["n"])
    else:
        s["after"] = _lengths(gen, case, min(cap, max(1, case["Sq"])), cap) \
            if case["ragged"] else None
    if case["kind"] in ("attend", "step"):
        s["q"] = normal(B, case["Hq"], case["Sq"], D).to(dtype)
        s["hide"] = None
        Sk = pages * page if page else cap
        if case["mask"]:
            # padding at the front of each sequence; the newest keys stay visible
            pad = torch.randint(0, max(1, cap // 4), (B, 1, 1), generator=gen, device="cuda")
            last = (s["after"] if s["after"] is not None
                    else torch.full((B,), Sk, device="cuda")).view(B, 1, 1) - case["Sq"]
            j = torch.arange(Sk, device="cuda")
            s["hide"] = ((j >= pad) | (j >= last)).expand(B, case["Sq"], Sk).contiguous()
    return s


# ------------------------------------------------------------------ one pass

def _attend(s):
    q = s["q"].float()
    B, Hq, Sq, D = q.shape
    k = _unpack(_rows(s["cache_k"], s["table"]), D, s["dtype"])
    v = _unpack(_rows(s["cache_v"], s["table"]), D, s["dtype"])
    Hkv, Sk = k.shape[1], k.shape[2]
    scores = q.reshape(B, Hkv, -1, D) @ k.transpose(-1, -2) * D ** -0.5
    scores = scores.view(B, Hkv, Hq // Hkv, Sq, Sk)
    j = torch.arange(Sk, device=q.device)
    lens = s["after"].long() if s["after"] is not None else torch.full((B,), Sk, device=q.device)
    last = lens[:, None] - Sq + torch.arange(Sq, device=q.device)  # each query's own position
    seen = (j < lens[:, None, None]).expand(B, Sq, Sk)
    if s["causal"]:
        seen = seen & (j <= last[..., None])
        if s["window"]:
            seen = seen & (j > last[..., None] - s["window"])
    if s["hide"] is not None:
        seen = seen & s["hide"]
    scores = scores.masked_fill(~seen[:, None, None], float("-inf"))
    w = torch.exp(scores - scores.amax(-1, keepdim=True))
    w = w / w.sum(-1, keepdim=True)
    return (w.view(B, Hkv, -1, Sk) @ v).view(B, Hq, Sq, D).to(s["dtype"])


def _read(s, start, lens, n):
    t = start.long()[:, None] + torch.arange(n, device="cuda")
    live = (t < lens.long()[:, None])[:, None, :, None]
    at = t.clamp(max=s["cap"] - 1)[:, None, :, None]

    def rows(cache):
        r = _rows(cache, s["table"])
        r = r.gather(2, at.expand(-1, s["Hkv"], -1, r.shape[-1]))
        return (_unpack(r, s["D"], s["dtype"]) * live).to(s["dtype"])

    return {"k": rows(s["cache_k"]), "v": rows(s["cache_v"])}


def run(state):
    s = state
    if own:
        import grouped_query_attention_fwd_b200 as gqa
        if s["kind"] in ("store", "step"):
            gqa.kv_append_q4(s["cache_k"], s["cache_v"], s["k_new"], s["v_new"], s["lens"],
                             new_lens=s["count"], advance=False, block_table=s["table"])
        if s["kind"] == "store":
            k, v = gqa.kv_read_q4(s["cache_k"], s["cache_v"], s["D"], s["dtype"],
                                  kv_lens=s["after"], start=s["lens"], n=s["n"],
                                  block_table=s["table"])
            return {"k": k, "v": v}
        if s["kind"] == "read":
            k, v = gqa.kv_read_q4(s["cache_k"], s["cache_v"], s["D"], s["dtype"],
                                  kv_lens=s["lens"], n=s["n"], block_table=s["table"])
            return {"k": k, "v": v}
        return {"out": gqa.forward_q4(
            s["q"], s["cache_k"], s["cache_v"], mask=s["hide"], causal=s["causal"],
            causal_offset="bottom_right", window=s["window"], kv_lens=s["after"],
            block_table=s["table"])}
    if s["kind"] in ("store", "step"):
        _write(s, s["cache_k"], _pack(s["k_new"].float(), s["dtype"]))
        _write(s, s["cache_v"], _pack(s["v_new"].float(), s["dtype"]))
    if s["kind"] == "store":
        return _read(s, s["lens"], s["after"], s["n"])
    if s["kind"] == "read":
        return _read(s, torch.zeros_like(s["lens"]), s["lens"], s["n"])
    return {"out": _attend(s)}


def work(case):
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    record = 16 * (1 + -(-D // 32))
    if case["kind"] in ("store", "read"):
        # the rows that a ragged batch has: half of the most, in the mean
        rows = 2 * B * Hkv * case["n"] * (0.5 if case["ragged"] else 1.0)
        written = 2 * B * Hkv * case["n"] * D * 2
        if case["kind"] == "read":
            return {"bytes": rows * record + written, "flops": 2 * rows * D}
        return {"bytes": rows * (2 * D + record) + written, "flops": 6 * rows * D}
    Sq, cap, window = case["Sq"], case["cap"], case["window"]
    mean = (cap + Sq) / 2 if case["ragged"] else cap
    keys = min(mean, window + Sq - 1) if window else mean
    # keys that a query sees, in the mean: under causal the last query's are all, the first's fewer
    pairs = min(mean, window) if window else (mean - (Sq - 1) / 2 if case["causal"] else mean)
    qo = 2 * B * case["Hq"] * Sq * D * 2
    mask = B * Sq * keys if case["mask"] else 0
    return {"bytes": 2 * B * Hkv * keys * record + qo + mask,
            "flops": 4 * B * case["Hq"] * Sq * max(1.0, pairs) * D}


# ------------------------------------------------------------------ the definition in 64 bits

def _values64(records, D, dtype):
    """fp64 values of records [..., R], group by group."""
    out = []
    for g in range(-(-D // 32)):
        p = records[..., 4 * g:4 * g + 4].contiguous().view(dtype).double()
        c = records[..., 16 + 16 * g:32 + 16 * g].long()
        x = torch.zeros(*c.shape[:-1], 32, dtype=torch.float64, device=c.device)
        x[..., 0::2] = (c % 16).double()
        x[..., 1::2] = (c // 16).double()
        out.append(x * p[..., 0:1] + p[..., 1:2])
    return torch.cat(out, -1)[..., :D]


def _rounded64(x, dtype):
    """What a cache of 4 bits keeps of 16-bit rows x [..., D], in fp64."""
    out = []
    for x in x.double().split(32, -1):
        low = x.min(-1, keepdim=True).values
        step = ((x.max(-1, keepdim=True).values - low) / 15).to(dtype).double()
        safe = torch.where(step > 0, step, 1.0)
        out.append(low + step * torch.round((x - low) / safe).clamp(0, 15))
    return torch.cat(out, -1)


def _sequence64(s, name, b):
    """Entry b's records [Hkv, capacity, R]."""
    if s["table"] is None:
        return s[name][b]
    return torch.cat([s[name][int(p)] for p in s["table"][b]], 1)


def exact(case, seed):
    s = prepare(case, seed)
    D, dtype, B, Hkv = case["D"], s["dtype"], case["B"], case["Hkv"]
    if case["kind"] in ("store", "read"):
        got = {}
        for name in ("k", "v"):
            full = torch.zeros(B, Hkv, case["n"], D, dtype=torch.float64, device="cuda")
            for b in range(B):
                if case["kind"] == "store":
                    n = int(s["after"][b] - s["lens"][b])
                    full[b, :, :n] = _rounded64(s[name + "_new"][b, :, :n], dtype)
                else:
                    n = int(s["lens"][b])
                    full[b, :, :n] = _values64(_sequence64(s, "cache_" + name, b)[:, :n], D, dtype)
            got[name] = full
        return got
    Hq, Sq, g = case["Hq"], case["Sq"], case["Hq"] // Hkv
    out = torch.empty(B, Hq, Sq, D, dtype=torch.float64, device="cuda")
    for b in range(B):
        kv = []
        for name in ("k", "v"):
            x = _values64(_sequence64(s, "cache_" + name, b), D, dtype)
            if case["kind"] == "step":
                x[:, int(s["lens"][b])] = _rounded64(s[name + "_new"][b, :, 0], dtype)
            kv.append(x)
        n = int(s["after"][b]) if s["after"] is not None else kv[0].shape[1]
        k, v = kv[0][:, :n], kv[1][:, :n]
        i = torch.arange(n - Sq, n, device="cuda")[:, None]
        j = torch.arange(n, device="cuda")[None, :]
        hidden = torch.zeros(Sq, n, dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden |= j > i
            if case["window"]:
                hidden |= i - j >= case["window"]
        if s["hide"] is not None:
            hidden |= ~s["hide"][b, :, :n]
        for h in range(Hq):
            a = s["q"][b, h].double() @ k[h // g].T / D ** 0.5
            a[hidden] = -torch.inf
            out[b, h] = torch.softmax(a, -1) @ v[h // g]
    return {"out": out}
