"""Measured cases of the 8-bit KV cache, the sliding-window decode and the chunk attention.

Each case is one call on data that a serving engine holds: block-paged caches in shuffled
block order, block tables, context lengths.  `run` computes the call either in plain torch
operations (own = False) or through this repository's package (own = True).

Shapes: 16 query / 8 KV heads of 128 dims with 256-token blocks, 32 / 8 heads with
16-token blocks, and 4 / 2 heads of 64 dims are the repository's own workloads; windows,
sinks and chunk lengths are generic.
"""

import math

import torch

own = False

E4M3_MAX = 448.0
MIN_EXP = -118
GOLDEN = 0.6180339887498949


# ------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------

def _case(name, op, **kw):
    c = dict(name=name, op=op, batch=1, lo=1, hi=1, hq=16, hkv=8, d=128, bs=256, fp8=True, window=0,
             sinks=0, new=1)
    c.update(kw)
    return c


def listed():
    return [
        # a decode step's new tokens, one per sequence, batch 512
        _case("store_b512", "store", batch=512),
        # the new tokens of 32 prompts (mean 768) written in one call
        _case("store_prompts", "store", batch=24594),
        # a few short sequences read back (small heads)
        _case("gather_b4", "gather", batch=4, lo=17, hi=700, hq=4, hkv=2, d=64),
        # 32 prompts' caches read back
        _case("gather_b32", "gather", batch=32, lo=64, hi=2048),
        # a single user's decode step over the 8-bit cache: latency
        _case("decode_fp8_b1", "decode", batch=1, lo=4096, hi=4096),
        # an ordinary decode batch over the 8-bit cache
        _case("decode_fp8_b64", "decode", batch=64, lo=512, hi=4096),
        # few long contexts in small blocks, group 4
        _case("decode_fp8_long", "decode", batch=8, lo=32768, hi=32768, hq=32, bs=16),
        # a large decode batch of a windowed model with 4 sinks, bf16 cache
        _case("decode_window_b256", "decode", batch=256, lo=512, hi=8192, hq=32, bs=16, fp8=False,
              window=1024, sinks=4),
        # draft tokens checked against long 8-bit caches: 5 tokens a sequence
        _case("chunk_verify", "chunk", batch=8, lo=8000, hi=8192, hq=32, bs=16, new=5),
        # chunks of 512 prompt tokens over long 8-bit caches
        _case("chunk_fp8_512", "chunk", batch=8, lo=4096, hi=8192, hq=32, bs=16, new=512),
        # chunks of 256 tokens of a windowed model, bf16 cache
        _case("chunk_window", "chunk", batch=16, lo=300, hi=8191, bs=256, fp8=False, window=1000,
              sinks=4, new=256),
        # whole prompts at once (every token new), bf16 cache, ragged lengths
        _case("chunk_prompts", "chunk", batch=32, lo=64, hi=2048, fp8=False, new=2048),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["store", "gather", "decode", "decode", "chunk", "chunk"])
    hq, hkv, d, bs = rng.choice([(16, 8, 128, 256), (32, 8, 128, 16), (4, 2, 64, 256), (16, 2, 128, 64),
                                 (8, 8, 64, 32), (12, 4, 128, 128), (7, 1, 128, 16)])
    c = dict(op=op, batch=1, lo=1, hi=1, hq=hq, hkv=hkv, d=d, bs=bs, fp8=True, window=0, sinks=0, new=1)
    if op == "store":
        c["batch"] = _log(rng, 1, 24594)
        return c
    # cache bytes at most those of 64 contexts of 2304 tokens (8 heads of 128 dims)
    c["hi"] = _log(rng, 1, 16384 if op == "decode" else 8192)
    c["lo"] = _log(rng, 1, c["hi"])
    c["batch"] = _log(rng, 1, max(1, min(256, 147456 // c["hi"])))
    if op != "gather":
        c["fp8"] = rng.random() < 0.6
        if rng.random() < 0.5:
            c["window"] = _log(rng, 1, 4096)
            c["sinks"] = rng.choice([0, 1, 4, 4, 16, 130])
    if op == "chunk":
        c["hi"] = max(2, c["hi"])
        c["new"] = _log(rng, 2, min(c["hi"], 2048))
        # the plain form's scores stay below those of 32 prompts of 2048 tokens
        c["batch"] = max(1, min(c["batch"], (1 << 31) // (c["hq"] * c["new"] * c["hi"])))
    return c


# ------------------------------------------------------------------------------------
# shapes of a case (the same for every seed)
# ------------------------------------------------------------------------------------

def _lens(c):
    """Context lengths spread over [lo, hi], the longest among them."""
    n = [c["lo"] + int((c["hi"] - c["lo"] + 1) * ((i * GOLDEN) % 1.0)) for i in range(c["batch"])]
    n[0] = c["hi"]
    return n


def _news(c):
    """New tokens of each sequence: `new`, or all of a shorter context."""
    return [min(c["new"], n) for n in _lens(c)]


def _visible(c, p):
    """Keys that a query at position p sees."""
    w, s = c["window"], c["sinks"]
    return p + 1 if w == 0 or p + 1 <= w else w + min(s, p + 1 - w)


def work(case):
    c = case
    row = c["hkv"] * (c["d"] + 1) if c["fp8"] else c["hkv"] * c["d"] * 2
    if c["op"] == "store":
        return {"bytes": c["batch"] * (2 * c["hkv"] * c["d"] * 2 + 2 * row + 4), "flops": 0}
    if c["op"] == "gather":
        return {"bytes": sum(_lens(c)) * (row + c["hkv"] * c["d"] * 2), "flops": 0}
    keys = pairs = 0
    rows = sum(_news(c))
    for n, m in zip(_lens(c), _news(c)):
        first = n - m
        # the union of the m queries' keys: those of the first one and the new tokens after it
        keys += _visible(c, first) + m - 1
        if c["window"] == 0 or n <= c["window"]:
            pairs += m * (first + 1) + m * (m - 1) // 2
        else:
            pairs += sum(_visible(c, p) for p in range(first, n))
    moved = keys * 2 * row + rows * c["hq"] * (4 * c["d"] + 4)
    return {"bytes": moved, "flops": 4 * c["d"] * c["hq"] * pairs}


# ------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------

def _quantise(x):
    """e4m3 codes and scale bytes of rows x [..., D] (finite values)."""
    x = x.float()
    frac, ex = torch.frexp(x.abs().amax(-1))              # amax = frac * 2^ex, frac in [0.5, 1)
    e = torch.clamp(ex - 9 + (frac > 0.875), min=MIN_EXP)  # amax <= 448 * 2^e = 0.875 * 2^(e + 9)
    e = torch.where(frac == 0, torch.full_like(e, MIN_EXP), e)
    code = torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn)
    return code, (e + 127).to(torch.uint8)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dev = torch.device("cuda")
    hq, hkv, d, bs = c["hq"], c["hkv"], c["d"], c["bs"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev).to(torch.bfloat16)

    # keys have a few channels that are larger than the others
    gain = 1.0 + 7.0 * (torch.rand((hkv, d), generator=g, device=dev) < 0.03)

    def keys(n):
        return (torch.randn((n, hkv, d), generator=g, device=dev) * gain).to(torch.bfloat16)

    s = {"c": c, "scale": 1.0 / math.sqrt(d)}
    lens = [1] * c["batch"] if c["op"] == "store" else _lens(c)
    need = [-(-n // bs) for n in lens] if c["op"] != "store" else [-(-c["batch"] // bs)]
    nb = sum(need) + 3
    order = torch.randperm(nb, generator=g, device=dev).to(torch.int32)
    if c["op"] == "store":
        n = c["batch"]
        s["k"], s["v"] = keys(n), normal(n, hkv, d)
        slots = torch.randperm(nb * bs, generator=g, device=dev)[:n].to(torch.int32)
        if n > 1:
            slots[n // 2] = -1          # a padding token
        s["slots"] = slots
        for x in ("k", "v"):
            s[x + "_cache"] = torch.zeros((nb, bs, hkv, d), dtype=torch.float8_e4m3fn, device=dev)
            s[x + "_scales"] = torch.zeros((nb, hkv, bs), dtype=torch.uint8, device=dev)
        return s
    width = max(need)
    tables = torch.full((c["batch"], width), -1, dtype=torch.int32)
    at = 0
    host_order = order.cpu()
    for b, k in enumerate(need):
        tables[b, :k] = host_order[at:at + k]
        at += k
    s["tables"] = tables.to(dev)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["max_len"] = max(lens)
    rows = nb * bs
    pools = [("k", keys(rows)), ("v", normal(rows, hkv, d))]
    for x, full in pools:
        s[x + "_scales"] = None
        if c["fp8"]:
            code, byte = _quantise(full)
            s[x + "_cache"] = code.view(nb, bs, hkv, d)
            s[x + "_scales"] = byte.view(nb, bs, hkv).transpose(1, 2).contiguous()
        else:
            s[x + "_cache"] = full.view(nb, bs, hkv, d)
    if c["op"] == "gather":
        cu = torch.zeros(c["batch"] + 1, dtype=torch.int32)
        cu[1:] = torch.cumsum(torch.tensor(lens), 0)
        s["cu"], s["total"] = cu.to(dev), sum(lens)
        return s
    news = _news(c)
    cu = torch.zeros(c["batch"] + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(news), 0)
    s["cu"], s["total"], s["max_new"] = cu.to(dev), sum(news), max(news)
    # where queries and keys of one model agree, some scores stand out
    s["q"] = (2.0 * torch.randn((s["total"], hq, d), generator=g, device=dev)).to(torch.bfloat16)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((s["total"], hq), dtype=torch.float32, device=dev)
    return s


# ------------------------------------------------------------------------------------
# plain forms
# ------------------------------------------------------------------------------------

def _scale_of(byte):
    return torch.ldexp(torch.ones_like(byte, dtype=torch.float32), byte.int() - 127)


def _rows(s, x, tables, pos):
    """Rows of cache x ("k" or "v") at positions pos of the sequences of `tables`, in float32."""
    cache, scales, bs = s[x + "_cache"], s[x + "_scales"], s["c"]["bs"]
    block = torch.gather(tables.long(), 1, torch.div(pos, bs, rounding_mode="floor")).clamp(min=0)
    row = pos % bs
    got = cache.view(torch.uint8)[block, row].view(cache.dtype).float() if cache.dtype != torch.bfloat16 \
        else cache[block, row].float()
    return got if scales is None else got * _scale_of(scales[block, :, row])[..., None]


def _plain_store(s):
    slots = s["slots"].long()
    keep = slots >= 0
    bs = s["c"]["bs"]
    block, row = slots[keep] // bs, slots[keep] % bs
    for x in ("k", "v"):
        code, byte = _quantise(s[x][keep])
        s[x + "_cache"].view(torch.uint8)[block, row] = code.view(torch.uint8)
        s[x + "_scales"][block, :, row] = byte
    return {x: s[x] for x in ("k_cache", "v_cache", "k_scales", "v_scales")}


def _plain_gather(s):
    lens = s["lens"].long()
    seq = torch.repeat_interleave(torch.arange(lens.numel(), device=lens.device), lens, output_size=s["total"])
    pos = torch.arange(s["total"], device=lens.device) - s["cu"].long()[seq]
    return _rows(s, "k", s["tables"][seq], pos[:, None])[:, 0].to(torch.bfloat16)


def _plain_attention(s):
    c, dev = s["c"], s["q"].device
    hq, hkv, d, w, sinks = c["hq"], c["hkv"], c["d"], c["window"], c["sinks"]
    lens, cu = s["lens"].long(), s["cu"].long()
    new = cu[1:] - cu[:-1]
    b, m = lens.numel(), s["max_new"]
    first = lens - new
    # positions of the keys that a sequence's queries see: sinks, then the window of the first query on
    width = s["max_len"] if w == 0 else min(s["max_len"], sinks + w + m)
    low = torch.zeros_like(lens) if w == 0 else (first - w + 1).clamp(min=0)
    skip = (low - sinks).clamp(min=0)
    v = torch.arange(width, device=dev)[None, :]
    pos = torch.where(v < sinks, v, v + skip[:, None]).expand(b, width)
    at = pos.clamp(max=s["max_len"] - 1)
    k, val = _rows(s, "k", s["tables"], at), _rows(s, "v", s["tables"], at)      # [b, width, hkv, d]
    t = torch.arange(m, device=dev)[None, :]
    real = t < new[:, None]
    src = (cu[:-1, None] + t).clamp(max=s["total"] - 1)
    q = s["q"].float()[src].view(b, m, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]                    # [b, hkv, g * m, width]
    p = (first[:, None] + t)[:, :, None]
    key = pos[:, None, :]
    seen = (key <= p) & (key < lens[:, None, None])
    if w:
        seen = seen & ((key > p - w) | (key < sinks))
    score = score.view(b, hkv, hq // hkv, m, width).masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    e = score.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e.view(b, hkv, -1, width), val.permute(0, 2, 1, 3)).view(b, hkv, hq // hkv, m, d) / total
    lse = (top + total.log())[..., 0]
    out = out.permute(0, 3, 1, 2, 4).reshape(b, m, hq, d)[real]
    lse = lse.permute(0, 3, 1, 2).reshape(b, m, hq)[real]
    return out.to(torch.bfloat16), lse


# ------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------

def run(state):
    s, c = state, state["c"]
    if own:
        import paged_kv_cache_422_b200 as nvpa
        if c["op"] == "store":
            nvpa.store_kvcache_fp8(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"],
                                   s["slots"])
            return {x: s[x] for x in ("k_cache", "v_cache", "k_scales", "v_scales")}
        if c["op"] == "gather":
            return nvpa.gather_kv_fp8(s["k_cache"], s["k_scales"], s["tables"], s["cu"], s["total"])
        if "workspace" not in s:
            if c["op"] == "decode":
                size = nvpa.paged_decode_window_workspace_size(c["batch"], c["hq"], c["hkv"], c["d"], s["max_len"],
                                                               c["bs"], c["window"], c["sinks"])
            else:
                size = nvpa.chunk_attention_workspace_size(c["batch"], s["total"], c["hq"], c["hkv"], c["d"],
                                                           s["max_new"], s["max_len"], c["bs"], c["window"],
                                                           c["sinks"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device=s["q"].device)
        if c["op"] == "decode":
            return nvpa.paged_decode_attention_window(
                s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["max_len"], s["scale"],
                window=c["window"], num_sinks=c["sinks"], k_scales=s["k_scales"], v_scales=s["v_scales"],
                out=s["out"], lse=s["lse"], workspace=s["workspace"], return_lse=True)
        return nvpa.chunk_attention(
            s["q"], s["k_cache"], s["v_cache"], s["tables"], s["cu"], s["lens"], s["max_new"], s["max_len"],
            s["scale"], window=c["window"], num_sinks=c["sinks"], k_scales=s["k_scales"],
            v_scales=s["v_scales"], out=s["out"], lse=s["lse"], workspace=s["workspace"], return_lse=True)
    if c["op"] == "store":
        return _plain_store(s)
    if c["op"] == "gather":
        return _plain_gather(s)
    return _plain_attention(s)


# ------------------------------------------------------------------------------------
# the definition in 64 bits, sequence by sequence
# ------------------------------------------------------------------------------------

def _e4m3_values(device):
    """The 128 non-negative e4m3 values in order of their codes (the last one is NaN)."""
    code = torch.arange(128, device=device)
    e, f = code // 8, (code % 8).double()
    v = torch.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * torch.exp2((e - 7).double()))
    v[127] = math.nan
    return v


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    table = _e4m3_values("cuda")

    def value(code):
        byte = code.contiguous().view(torch.uint8).long()
        return torch.where(byte >= 128, -1.0, 1.0).double() * table[byte & 127]

    if c["op"] == "store":
        got = {}
        for x in ("k", "v"):
            nb, bs, hkv, d = s[x + "_cache"].shape
            codes = torch.zeros((nb * bs, hkv, d), dtype=torch.float64, device="cuda")
            bytes_ = torch.zeros((nb * bs, hkv), dtype=torch.int64, device="cuda")
            slots = s["slots"].long()
            keep = slots >= 0
            rows = s[x][keep].double()
            top = rows.abs().amax(-1)
            # the smallest e from -118 on with top <= 448 * 2^e
            es = torch.arange(MIN_EXP, 121, device="cuda")
            e = es[(top[..., None] > E4M3_MAX * torch.exp2(es.double())).sum(-1)]
            y = rows * torch.exp2(-e.double())[..., None]
            # nearest value, ties to the even code
            mag = y.abs()
            above = torch.searchsorted(table[:127].contiguous(), mag.contiguous()).clamp(max=126)
            below = (above - 1).clamp(min=0)
            up, down = table[above] - mag, mag - table[below]
            pick = torch.where((up < down) | ((up == down) & (above % 2 == 0)), above, below)
            codes[slots[keep]] = torch.copysign(table[pick], y)
            bytes_[slots[keep]] = e + 127
            got[x + "_cache"] = codes.view(nb, bs, hkv, d)
            got[x + "_scales"] = bytes_.view(nb, bs, hkv).transpose(1, 2)
        return got

    def rows64(x, blocks, n):
        cache, scales = s[x + "_cache"][blocks], s[x + "_scales"]
        if scales is None:
            return cache.double().flatten(0, 1)[:n]
        power = torch.exp2(scales[blocks].double() - 127).transpose(1, 2)[..., None]
        return (value(cache) * power).flatten(0, 1)[:n]

    lens = _lens(c)
    outs, lses = [], []
    at = 0
    for b, n in enumerate(lens):
        blocks = s["tables"][b, :-(-n // c["bs"])].long()
        k = rows64("k", blocks, n)
        if c["op"] == "gather":
            outs.append(k)
            continue
        v = rows64("v", blocks, n)
        m = _news(c)[b]
        q = s["q"][at:at + m].double()
        at += m
        key = torch.arange(n, device="cuda")[None, :]
        p = torch.arange(n - m, n, device="cuda")[:, None]
        hide = key > p
        if c["window"]:
            hide |= (key <= p - c["window"]) & (key >= c["sinks"])
        out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
        lse = torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
        for h in range(c["hq"]):
            kh = h // (c["hq"] // c["hkv"])
            score = (q[:, h] @ k[:, kh].T) * s["scale"]
            score[hide] = -math.inf
            lse[:, h] = torch.logsumexp(score, -1)
            out[:, h] = torch.softmax(score, -1) @ v[:, kh]
        outs.append(out)
        lses.append(lse)
    if c["op"] == "gather":
        return torch.cat(outs)
    return torch.cat(outs), torch.cat(lses)
