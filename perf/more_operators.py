"""The paged cache of keys and values as measured work: appending the rows of a step to it with the rotation of
their positions (``append``), and attention of these rows over it (``attention``).

Where ``own`` is false every operator is computed in its plain form, by elementary torch operations. Where it is
true the calls are those of the package.

Definitions. A step has n requests; request i has K_i + 1 rows, row cu_num_draft[i] + i + j is its j-th (without
cu_num_draft one row a request), at place x = lengths[i] + j of its sequence. Place x is held in slot x mod P of page
page_table[i, x div P]. An element of an 8-bit cache stands for itself times its head's scale.
  append     key k, value v of the row: the slot takes rot(k) and v, divided by the scale of the head where there is one,
             rounded once. rot turns pair m of the first rotary_dim elements, (m, m + rotary_dim / 2) or (2 m, 2 m + 1), by the
             angle pos inv_freq[m]: (a cos - b sin, a sin + b cos); pos is x, or positions[axes[m], row]. The row's
             queries are turned the same way.
  attention  s_t = scale q . k_t over the keys t <= x, with a window w only t > x - w; out = sum_t exp(s_t) v_t / Z and
             lse = ln Z, Z = sum_t exp(s_t). Query head g reads key head g div (query heads / key heads).
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
MOST = 256 * 4096 * 8 * 128 * 4  # bytes of keys and values that the largest listed case reads


# ------------------------------------------------------------------------------------- cases

def append(name, **kw):
    return {"name": name, "op": "append", "dtype": "bf16", "cache": "bf16", "page": 16, "layout": "heads", "even": True,
            "rotary": kw["dim"], "interleaved": False, "axes": 1, "theta": 500000.0, **kw}


def attention(name, **kw):
    return {"name": name, "op": "attention", "dtype": "bf16", "cache": "bf16", "page": 16, "layout": "heads", "even": True,
            "window": 0, **kw}


def listed():
    return [
        # the next token of one request far into its sequence: latency counts
        append("append 1x1 bf16", n=1, new=1, ctx=131000, q_heads=32, kv_heads=8, dim=128),
        # a verification step: 256 requests of 5 drafts and the bonus position
        append("append 256x6 bf16", n=256, new=6, ctx=2048, q_heads=64, kv_heads=8, dim=128, even=False, page=64),
        # prompts with pictures (time, height and width positions) into an 8-bit cache
        append("append 4x2048 3 axes e4m3", n=4, new=2048, ctx=0, q_heads=28, kv_heads=4, dim=128, cache="e4m3", axes=3, theta=1e6),
        # one long odd chunk of a prompt: half precision, neighbouring pairs, half of every head turned
        append("append 1x16001 f16", n=1, new=16001, ctx=1000, q_heads=64, kv_heads=8, dim=64, dtype="f16", cache="f16", rotary=32,
               interleaved=True, theta=10000.0, page=40, layout="tokens"),
        # one short request's next token: latency counts
        attention("attention 1x1 over 600", n=1, new=1, ctx=600, q_heads=32, kv_heads=8, dim=128),
        # one long request's next token: all of the machine on one sequence
        attention("attention 1x1 over 131072", n=1, new=1, ctx=131072, q_heads=32, kv_heads=8, dim=128),
        # one request's verification at an ordinary length
        attention("attention 1x6 over 8192", n=1, new=6, ctx=8192, q_heads=64, kv_heads=8, dim=128, page=64),
        # a draft step of a full batch: the largest read
        attention("attention 256x1 over 4096", n=256, new=1, ctx=4096, q_heads=32, kv_heads=8, dim=128),
        # a verification of requests of all lengths, eight query heads to a key head
        attention("attention 64x6 ragged 16384", n=64, new=6, ctx=16384, q_heads=64, kv_heads=8, dim=128, even=False, page=64, layout="tokens"),
        # an 8-bit cache, seven query heads to a key head
        attention("attention 96x4 e4m3", n=96, new=4, ctx=8192, q_heads=28, kv_heads=4, dim=128, cache="e4m3", even=False),
        # a sliding window over long sequences, half precision, pages of odd length
        attention("attention 128x3 window", n=128, new=3, ctx=8000, q_heads=64, kv_heads=8, dim=64, dtype="f16", cache="f16", window=1024,
                  page=20, layout="tokens"),
        # wide heads, one key head for all
        attention("attention 200x2 dim 256", n=200, new=2, ctx=5000, q_heads=8, kv_heads=1, dim=256, even=False, page=32),
    ]


HEADS = {64: ((64, 8), (16, 2), (28, 4), (8, 1)), 128: ((32, 8), (64, 8), (28, 4), (16, 16), (8, 1)), 256: ((16, 4), (8, 1), (16, 16))}


def draw(rng):
    cache = rng.choice(("bf16", "bf16", "f16", "e4m3"))
    dim = rng.choice((64, 128, 128, 256))
    q_heads, kv_heads = rng.choice(HEADS[dim])
    case = {"op": rng.choice(("append", "attention", "attention")), "dtype": rng.choice(("bf16", "f16")) if cache == "e4m3" else cache,
            "cache": cache, "dim": dim, "q_heads": q_heads, "kv_heads": kv_heads, "page": rng.choice((16, 16, 20, 32, 40, 64, 128)),
            "layout": rng.choice(("heads", "tokens")), "even": rng.random() < 0.5}
    if case["op"] == "append":
        rows = round(2 ** rng.uniform(0, 14))
        case["n"] = min(rows, round(2 ** rng.uniform(0, 8)))
        case["new"] = max(1, rows // case["n"])
        case["ctx"] = round(2 ** rng.uniform(0, 13))
        case["rotary"] = rng.choice((dim, dim, dim // 2))
        case["interleaved"], case["axes"] = rng.random() < 0.3, rng.choice((1, 1, 3))
        case["theta"] = rng.choice((1e4, 5e5, 1e6))
        return case
    size = 1 if cache == "e4m3" else 2
    case["ctx"] = round(2 ** rng.uniform(0, 17))
    fit = MOST // ((case["ctx"] + 8) * kv_heads * dim * 2 * size)
    case["n"] = max(1, min(round(2 ** rng.uniform(0, 8)), fit))
    case["new"] = rng.choice((1, 1, 2, 3, 4, 6, 8))
    case["window"] = rng.choice((0, 0, 0, round(2 ** rng.uniform(4, 12))))
    return case


# ------------------------------------------------------------------------------------ inputs

def contexts(case):
    """Tokens of every request before the step: all alike, or from none to the most."""
    n, ctx = case["n"], case["ctx"]
    return [ctx if case["even"] or n == 1 else ctx * i // (n - 1) for i in range(n)]


def prepare(case, seed):
    host = torch.Generator()
    host.manual_seed(int(seed) * 2 + 1)
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2 + 1)
    n, new, P, dim, hq, hk = (case[x] for x in ("n", "new", "page", "dim", "q_heads", "kv_heads"))
    lengths = torch.tensor(contexts(case))[torch.randperm(n, generator=host)]
    # pages as a server hands them out: any page of the pool for any place, none used twice
    used = (lengths + new + P - 1) // P
    width, pool = int(used.max()) + 1, int(used.sum()) + 8
    at = torch.cumsum(used, 0)[:, None] - used[:, None] + torch.arange(width)
    order = torch.randperm(pool, generator=host)
    table = torch.where(torch.arange(width) < used[:, None], order[at.clamp(max=pool - 1)], 0)
    s = {"case": dict(case), "lengths": lengths.int().cuda(), "page_table": table.int().cuda(), "cu_num_draft": None}
    if new > 1:
        s["cu_num_draft"] = (torch.arange(n + 1, dtype=torch.int32) * (new - 1)).cuda()
    # the cache: some channels of the keys larger than the others, as trained models have them
    shape = (pool, hk, P, dim) if case["layout"] == "heads" else (pool, P, hk, dim)
    kind = TYPES[case["cache"]]
    s["k_scale"] = s["v_scale"] = None
    loud = torch.where(torch.rand(dim, generator=g, device="cuda") < 0.05, 4.0, 1.0)
    if case["cache"] == "e4m3":
        s["k_scale"] = 0.01 + 0.03 * torch.rand(hk, generator=g, device="cuda")
        s["v_scale"] = 0.01 + 0.03 * torch.rand(hk, generator=g, device="cuda")
    for name, factor in (("k_cache", loud), ("v_cache", torch.ones_like(loud))):
        c = torch.empty(shape, dtype=kind, device="cuda")
        for part in c.split(max(1, (1 << 27) // (hk * P * dim))):
            x = torch.randn(part.shape, generator=g, device="cuda", dtype=torch.bfloat16) * factor.bfloat16()
            part.copy_((x * 30).clamp_(-448, 448) if case["cache"] == "e4m3" else x)
        s[name] = c.transpose(1, 2) if case["layout"] == "heads" else c
    # queries, keys and values as one projection gives them
    rows = n * new
    if case["op"] == "append":
        qkv = torch.randn(rows, (hq + 2 * hk) * dim, generator=g, device="cuda").to(TYPES[case["dtype"]])
        s["q"], s["k"], s["v"] = (x.view(rows, -1, dim) for x in qkv.split((hq * dim, hk * dim, hk * dim), 1))
        half = case["rotary"] // 2
        s["inv_freq"] = (case["theta"] ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
        s["axes"] = s["positions"] = None
        if case["axes"] == 3:
            s["axes"] = [0] * (half - 2 * (half * 3 // 8)) + [1] * (half * 3 // 8) + [2] * (half * 3 // 8)
            x = lengths.repeat_interleave(new) + torch.arange(new).repeat(n)
            grid = torch.randint(0, 64, (2, rows), generator=host)
            s["positions"] = torch.stack((x, x + grid[0], x + grid[1])).int().cuda()
        s["out"] = torch.empty(rows, hq, dim, dtype=TYPES[case["dtype"]], device="cuda")
        return s
    # sharper than chance: a query prefers some keys, as in trained models
    share = 1 if case["cache"] == "e4m3" else 1.5
    s["q"] = (share * torch.randn(rows, hq, dim, generator=g, device="cuda")).to(TYPES[case["dtype"]])
    s["out"] = [torch.empty_like(s["q"]), torch.empty(rows, hq, device="cuda")]
    return s


def run(s):
    if own:
        return run_own(s)
    return plain_append(s) if s["case"]["op"] == "append" else plain_attention(s)


def run_own(s):
    import speculative_decoding_verification_rejection_gb300 as sv

    c = s["case"]
    if c["op"] == "append":
        q = sv.cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["lengths"], q=s["q"], inv_freq=s["inv_freq"],
                            cu_num_draft=s["cu_num_draft"], positions=s["positions"], axes=s["axes"], interleaved=c["interleaved"],
                            k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    out, lse = sv.cache_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["lengths"], cu_num_draft=s["cu_num_draft"],
                                  window=c["window"], k_scale=s["k_scale"], v_scale=s["v_scale"], lse=True, out=s["out"])
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------------------- plain forms

def places(s):
    """Of every row its request, its number there, and its place in the sequence."""
    rows, n = s["q"].shape[0], s["lengths"].shape[0]
    r = torch.arange(rows, device="cuda")
    if s["cu_num_draft"] is None:
        return r, torch.zeros_like(r), s["lengths"].long()
    first = s["cu_num_draft"][:-1].long() + torch.arange(n, device="cuda")
    i = torch.searchsorted(first, r, right=True) - 1
    return i, r - first[i], s["lengths"][i].long() + r - first[i]


def turned(x, cos, sin, half, interleaved):
    x = x.float()
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((y, x[..., 2 * half:]), -1)


def rounded(x, scale, kind):
    if scale is None:
        return x.to(kind)
    return (x / scale[:, None]).clamp(-448, 448).to(kind)


def plain_append(s):
    c = s["case"]
    i, _, x = places(s)
    half = s["inv_freq"].numel()
    pos = x[:, None].double() if s["positions"] is None else s["positions"].t()[:, s["axes"]].double()
    angle = pos * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    page = s["page_table"][i, x // c["page"]].long()
    kind = s["k_cache"].dtype
    s["k_cache"][page, x % c["page"]] = rounded(turned(s["k"], cos, sin, half, c["interleaved"]), s["k_scale"], kind)
    s["v_cache"][page, x % c["page"]] = rounded(s["v"].float(), s["v_scale"], kind)
    q = turned(s["q"], cos, sin, half, c["interleaved"]).to(s["q"].dtype)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def plain_attention(s):
    c = s["case"]
    n, new, P, dim, hq, hk = (c[x] for x in ("n", "new", "page", "dim", "q_heads", "kv_heads"))
    lengths, table, width = s["lengths"].long(), s["page_table"].long(), s["page_table"].shape[1]
    first, count = torch.zeros_like(lengths), width
    if c["window"]:  # the pages that a window can reach
        first, count = (lengths - c["window"] + 1).clamp(min=0) // P, min(width, (c["window"] + new) // P + 2)
    column = first[:, None] + torch.arange(count, device="cuda")
    page = table.gather(1, column.clamp(max=width - 1))
    at = (column[:, :, None] * P + torch.arange(P, device="cuda")).flatten(1)
    k = s["k_cache"][page].float().flatten(1, 2).permute(0, 2, 3, 1)
    q = s["q"].float().view(n, new, hk, hq // hk, dim).permute(0, 2, 1, 3, 4).reshape(n, hk, -1, dim)
    score = torch.matmul(q, k).view(n, hk, new, hq // hk, -1) * dim ** -0.5
    if s["k_scale"] is not None:
        score *= s["k_scale"][:, None, None, None]
    x = lengths[:, None] + torch.arange(new, device="cuda")
    seen = at[:, None] <= x[:, :, None]
    if c["window"]:
        seen &= at[:, None] > x[:, :, None] - c["window"]
    score.masked_fill_(~seen[:, None, :, None], -float("inf"))
    top = score.max(-1, keepdim=True).values
    weight = score.sub_(top).exp_()
    total = weight.sum(-1, keepdim=True)
    v = s["v_cache"][page].float().flatten(1, 2).permute(0, 2, 1, 3)
    out = torch.matmul(weight.view(n, hk, -1, count * P), v).view(n, hk, new, hq // hk, dim) / total
    if s["v_scale"] is not None:
        out *= s["v_scale"][:, None, None, None]
    lse = (top + torch.log(total))[..., 0]
    return {"out": out.permute(0, 2, 1, 3, 4).reshape(n * new, hq, dim).to(s["q"].dtype), "lse": lse.permute(0, 2, 1, 3).reshape(n * new, hq)}


# --------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return exact_append(s) if case["op"] == "append" else exact_attention(s)


def exact_append(s):
    """One complex number a pair, turned by multiplication; the slots written one request at a time."""
    c, m = s["case"], s["inv_freq"].numel()
    n, new, P, rows = c["n"], c["new"], c["page"], s["q"].shape[0]
    start = s["lengths"].double().cpu()
    pos = (start[:, None] + torch.arange(new)).view(rows, 1).expand(rows, m).clone()
    if s["positions"] is not None:
        for p, axis in enumerate(s["axes"]):
            pos[:, p] = s["positions"][axis].double().cpu()
    turn = torch.polar(torch.ones(rows, m, dtype=torch.float64), pos * s["inv_freq"].double().cpu()).cuda()[:, None]

    def rot(x):
        y = x.double().clone()
        one, two = (y[..., 0:2 * m:2], y[..., 1:2 * m:2]) if c["interleaved"] else (y[..., :m], y[..., m:2 * m])
        z = torch.complex(one.contiguous(), two.contiguous()) * turn
        one.copy_(z.real)
        two.copy_(z.imag)
        return y

    out = {"q": rot(s["q"])}
    for name, new_values, scale in (("k", rot(s["k"]), s["k_scale"]), ("v", s["v"].double(), s["v_scale"])):
        cache = s[name + "_cache"].double()
        if scale is not None:
            new_values = (new_values / scale.double()[:, None]).clamp(-448, 448)
        for i in range(n):
            x = int(start[i]) + torch.arange(new, device="cuda")
            cache[s["page_table"][i].long()[x // P], x % P] = new_values[i * new:(i + 1) * new]
        out[name + "_cache"] = cache
    return out


def exact_attention(s):
    """One request and one key head at a time, each row's keys alone."""
    c = s["case"]
    n, new, P, dim, hk, group = c["n"], c["new"], c["page"], c["dim"], c["kv_heads"], c["q_heads"] // c["kv_heads"]
    if n * hk * new > 4000:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for i, length in enumerate(s["lengths"].tolist()):
        pages = s["page_table"][i, :(length + new + P - 1) // P].long()
        keys, values = (s[x][pages].flatten(0, 1) for x in ("k_cache", "v_cache"))
        for h in range(hk):
            ks, vs = (1.0 if s[x] is None else s[x][h].double() for x in ("k_scale", "v_scale"))
            for j in range(new):
                hi = length + j + 1
                lo = max(0, hi - c["window"]) if c["window"] else 0
                q = s["q"][i * new + j, h * group:(h + 1) * group].double()
                score = q @ keys[lo:hi, h].double().t() * ks / math.sqrt(dim)
                z = torch.logsumexp(score, 1)
                lse[i * new + j, h * group:(h + 1) * group] = z
                out[i * new + j, h * group:(h + 1) * group] = (score - z[:, None]).exp() @ values[lo:hi, h].double() * vs
    return {"out": out, "lse": lse}


def work(case):
    """append: every element of the rows read once, the turned queries and the cache's slots written once; four
    products and two sums a turned pair. attention: every key and value that a row of the request sees read once, the
    queries and the outputs besides; two products and two sums an element of a key and value for every row that sees it."""
    n, new, dim, hq, hk = (case[x] for x in ("n", "new", "dim", "q_heads", "kv_heads"))
    rows, size = n * new, 1 if case["cache"] == "e4m3" else 2
    if case["op"] == "append":
        return {"bytes": rows * dim * ((hq + 2 * hk) * 2 + hq * 2 + 2 * hk * size) + 8 * n, "flops": rows * (hq + hk) * 3 * case["rotary"]}
    window = case["window"] or 1 << 40
    keys = sum(min(x + new, window + new - 1) for x in contexts(case))
    pairs = sum(min(x + j + 1, window) for x in contexts(case) for j in range(new))
    return {"bytes": keys * hk * dim * 2 * size + rows * hq * (dim * 4 + 4) + 8 * n, "flops": 4 * pairs * hq * dim}
