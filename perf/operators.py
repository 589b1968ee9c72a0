"""The row operators of the sampler as measured work: drawing a token of each row of logits from a
given uniform number under temperature, top-k, top-p and min-p (``sample``), the same with the
distribution it was drawn from (``draft``: what the verification takes as draft_probs), and the
log-probabilities, ranks and best tokens of rows (``logprobs``).

Where ``own`` is false every operator is computed in its plain form, by elementary torch
operations. Where it is true the calls are those of the package.

Definitions (V tokens, logits l_v; a NaN or -inf logit is never kept, L = max l_v):
  d_v = fl(fl(l_v - L) * fl(1 / T)) in binary32 (0 where l_v = L), t_v = exp(d_v) by the library's
  binary32 exp, W_v = rint(t_v 2^40) as a whole number, so that every sum of weights is exact.
  top-k keeps l_v >= the k-th largest logit (k < 1 or k >= V: all). top-p (P < 1, at least 1e-6)
  keeps, of those, the tokens whose strictly larger kept logits hold less than P of the W of
  top-k's set. min-p (0 < M, at most 1) keeps d_v >= fl(ln M). The token is the first kept v, in
  index order, whose running sum of kept W exceeds u Z, Z the kept sum (the last kept one where
  u >= 1), and its log-probability d_v - ln(Z / 2^40). T <= 0, or k = 1: the first largest logit,
  with probability 1. A row with nothing to keep: token -1, log-probability -inf, probabilities 0.
"""
import numpy as np
import torch

own = False

ONE = float(1 << 40)  # the weight of a row's largest logit


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one request's next token: a single row, where latency counts
        {"name": "sample 1x32000 bf16", "op": "sample", "rows": 1, "vocab": 32000, "dtype": "bf16", "kind": "top_k_top_p"},
        # a few requests of a large vocabulary, each with its own settings
        {"name": "sample 8x151936 bf16", "op": "sample", "rows": 8, "vocab": 151936, "dtype": "bf16", "kind": "mixed"},
        # a serving batch with mixed settings
        {"name": "sample 256x151936 bf16", "op": "sample", "rows": 256, "vocab": 151936, "dtype": "bf16", "kind": "mixed"},
        # plain temperature sampling of a serving batch: every token stays
        {"name": "sample 256x151936 open", "op": "sample", "rows": 256, "vocab": 151936, "dtype": "bf16", "kind": "open"},
        # top-p alone over float32 logits, the largest batch
        {"name": "sample 512x129280 f32", "op": "sample", "rows": 512, "vocab": 129280, "dtype": "f32", "kind": "top_p"},
        # an odd vocabulary (rows that start anywhere) with min-p
        {"name": "sample 48x40003 f32", "op": "sample", "rows": 48, "vocab": 40003, "dtype": "f32", "kind": "min_p"},
        # one draft step of one request, of 64 requests, and of a large batch: token and distribution
        {"name": "draft 1x32000 f32", "op": "draft", "rows": 1, "vocab": 32000, "dtype": "f32", "kind": "top_k_top_p"},
        {"name": "draft 64x32000 bf16", "op": "draft", "rows": 64, "vocab": 32000, "dtype": "bf16", "kind": "open"},
        {"name": "draft 256x151936 bf16", "op": "draft", "rows": 256, "vocab": 151936, "dtype": "bf16", "kind": "mixed"},
        # the answer of one request's step with its 20 best tokens
        {"name": "logprobs 1x151936 bf16", "op": "logprobs", "rows": 1, "vocab": 151936, "dtype": "bf16", "top": 20, "spec": 0},
        # a prompt's tokens (float32, an odd vocabulary), no best tokens
        {"name": "logprobs 640x40003 f32", "op": "logprobs", "rows": 640, "vocab": 40003, "dtype": "f32", "top": 0, "spec": 0},
        # what a verification of 256 requests with 5 drafts each emitted: rows after a rejection are left out
        {"name": "logprobs 1536x151936 bf16", "op": "logprobs", "rows": 1536, "vocab": 151936, "dtype": "bf16", "top": 5, "spec": 5},
    ]


KINDS = ("open", "top_k", "top_p", "min_p", "top_k_top_p", "mixed")


def draw(rng):
    op = rng.choice(("sample", "draft", "logprobs"))
    vocab = int(round(2 ** rng.uniform(10, 17.2)))
    most = 256 * 151936 if op != "logprobs" else 1536 * 151936
    rows = int(round(2 ** rng.uniform(0, 10)))
    case = {"op": op, "rows": rows, "vocab": vocab, "dtype": rng.choice(("bf16", "f32"))}
    if op == "logprobs":
        case["spec"] = rng.choice((0, 0, 1, 3, 5))
        case["top"] = rng.choice((0, 1, 5, 20))
        case["rows"] = rows * (case["spec"] + 1)
    else:
        case["kind"] = rng.choice(KINDS)
    size = 2 if case["dtype"] == "bf16" else 4
    step = case.get("spec", 0) + 1
    fit = max(1, most * 2 // (case["vocab"] * size) // step) * step
    case["rows"] = min(case["rows"], fit)
    return case


# ------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2 + 1)
    rows, vocab = case["rows"], case["vocab"]
    u = lambda *shape: torch.rand(*shape, generator=g, device="cuda")  # noqa: E731
    # a bell of unlikely tokens, and 32 tokens the model favours, more or less clearly from row to row
    logits = torch.randn(rows, vocab, generator=g, device="cuda").mul_(2.0)
    at = torch.randint(0, vocab, (rows, 32), generator=g, device="cuda")
    logits.scatter_(1, at, (8.0 + 14.0 * u(rows, 1)) * (0.5 + 0.5 * u(rows, 32)))
    if case["dtype"] == "bf16":
        logits = logits.to(torch.bfloat16)
    s = {"case": dict(case), "logits": logits}
    if case["op"] == "logprobs":
        prepare_tokens(s, u)
        n = case["top"]
        s["out"] = [torch.empty(rows, device="cuda"), torch.empty(rows, dtype=torch.int32, device="cuda")]
        if n:
            s["out"] += [torch.empty(rows, n, dtype=torch.int32, device="cuda"), torch.empty(rows, n, device="cuda")]
        return s
    kind = case["kind"]
    s["uniforms"] = u(rows)
    s["temperature"] = 0.5 + 0.8 * u(rows)
    k = torch.tensor([20, 50, 0, 1, 200, 50, 0, 40], dtype=torch.int32, device="cuda")
    p = torch.tensor([0.9, 1.0, 0.95, 0.8, 1.0, 0.9, 1.0], device="cuda")
    m = torch.tensor([0.0, 0.05, 0.0, 0.1, 0.0], device="cuda")
    i = torch.arange(rows, device="cuda")
    s["top_k"] = s["top_p"] = s["min_p"] = None
    if kind == "mixed":
        s["top_k"], s["top_p"], s["min_p"] = k[i % 8].contiguous(), p[i % 7].contiguous(), m[i % 5].contiguous()
        s["temperature"][i % 16 == 11] = 0.0
    if kind in ("top_k", "top_k_top_p"):
        s["top_k"] = torch.full((rows,), 50, dtype=torch.int32, device="cuda")
    if kind in ("top_p", "top_k_top_p"):
        s["top_p"] = torch.full((rows,), 0.9, device="cuda")
    if kind == "min_p":
        s["min_p"] = torch.full((rows,), 0.05, device="cuda")
    s["out"] = [torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(rows, device="cuda")]
    if case["op"] == "draft":
        s["out"].append(torch.empty(rows, vocab, device="cuda"))
    return s


def prepare_tokens(s, u):
    """Tokens whose log-probabilities are wanted: one a row, or with `spec` the output of a
    verification, [requests, spec + 1] with -1 behind each request's last token."""
    case = s["case"]
    rows, vocab, spec = case["rows"], case["vocab"], case["spec"]
    # a row's token is a likely one as a rule: the best of 64 places
    places = (u(rows, 64) * vocab).long().clamp_(max=vocab - 1)
    best = s["logits"].float().gather(1, places).argmax(1, keepdim=True)
    token = places.gather(1, best)[:, 0].to(torch.int32)
    s["cu_num_draft"] = None
    if spec:
        n = rows // (spec + 1)
        s["cu_num_draft"] = torch.arange(n + 1, dtype=torch.int32, device="cuda") * spec
        emitted = 1 + (u(n) * (spec + 1)).long().clamp_(max=spec)
        token = token.view(n, spec + 1)
        token[torch.arange(spec + 1, device="cuda") >= emitted[:, None]] = -1
    s["tokens"] = token.contiguous()


def run(s):
    if own:
        return run_own(s)
    return plain_logprobs(s) if s["case"]["op"] == "logprobs" else plain_sample(s)


def run_own(s):
    import speculative_decoding_verification_rejection_gb300 as sv

    if s["case"]["op"] == "logprobs":
        got = sv.logprobs(s["logits"], s["tokens"], num_top=s["case"]["top"], cu_num_draft=s["cu_num_draft"], out=s["out"])
        return dict(zip(("logprob", "rank", "top_ids", "top_logprob"), got))
    got = sv.sample(s["logits"], s["uniforms"], s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                    logprob=True, probs=s["case"]["op"] == "draft", out=s["out"])
    return dict(zip(("tokens", "logprob", "probs"), got))


# ------------------------------------------------------------------------------- plain forms

def fused(a, b, c):
    """fl(a b + c) in binary32, rounded once."""
    return (a.double() * b + c).float()


def plain_exp(d):
    """The library's binary32 exp for d <= 0: d = k ln 2 + r, the Taylor polynomial of degree 7
    of exp(r), times 2^k; 0 below -87."""
    ln2 = float(np.float32(np.log(2.0)))
    shift = 1.5 * 2.0 ** 23
    at = d.clamp(min=-87.0)
    k = fused(at, float(np.float32(1.0 / np.log(2.0))), shift) - shift
    r = fused(-k, ln2, at)
    r = fused(-k, float(np.float32(np.log(2.0) - ln2)), r)
    p = torch.full_like(r, float(np.float32(1 / 5040)))
    for c in (1 / 720, 1 / 120, 1 / 24, 1 / 6, 0.5, 1.0, 1.0):
        p = fused(p, r.double(), float(np.float32(c)))
    return torch.where(d >= -87.0, (p.double() * torch.exp2(k.double())).float(), torch.zeros_like(p))


def plain_rows(logits, temperature):
    """float32 logits (NaN as -inf), their maximum, 1 / T (1 for a greedy row), and d."""
    l = logits.float()
    l = torch.where(torch.isnan(l), torch.full_like(l, -float("inf")), l)
    top = l.max(1, keepdim=True).values
    inv = torch.ones_like(top) if temperature is None else torch.where(temperature > 0, 1.0 / temperature, torch.ones_like(temperature))[:, None]
    d = torch.where(l == top, torch.zeros_like(l), (l - top) * inv.clamp(max=torch.finfo(torch.float32).max))
    return l, top, torch.where(torch.isinf(l) & (l < 0), l, d)


def plain_sample(s):
    l, top, d = plain_rows(s["logits"], s["temperature"])
    rows, vocab = l.shape
    W = torch.round(plain_exp(d).double() * ONE).long()
    place = torch.arange(vocab, device=l.device)
    empty = torch.isinf(top[:, 0]) & (top[:, 0] < 0)
    tau = torch.full_like(top, -float("inf"))
    k, p, m = s["top_k"], s["top_p"], s["min_p"]
    if k is not None or p is not None:
        ls, order = torch.sort(l, 1, descending=True)
        run_sum = torch.cumsum(W.gather(1, order), 1)
        new = torch.ones_like(ls, dtype=torch.bool)
        new[:, 1:] = ls[:, 1:] < ls[:, :-1]
        first = torch.cummax(torch.where(new, place, torch.zeros_like(place)), 1).values  # of each run of equal logits
        above = torch.where(first > 0, run_sum.gather(1, (first - 1).clamp(min=0)), torch.zeros_like(run_sum))
        if k is not None:
            wide = (k < 1) | (k >= vocab)
            kth = ls.gather(1, torch.where(wide, vocab, k).long()[:, None] - 1)
            tau = torch.where(wide[:, None], tau, kth)
        within = ls >= tau
        total = torch.where(within, run_sum, torch.zeros_like(run_sum)).max(1, keepdim=True).values
        if p is not None:
            part = torch.where(p < 1, p.clamp(min=1e-6).double(), torch.full_like(p, 2.0).double())[:, None]
            within &= above.double() < part * total.double()
        tau = torch.where(within, ls, torch.full_like(ls, float("inf"))).min(1, keepdim=True).values
    keep = l >= tau
    if m is not None:
        keep &= (d >= torch.log(m.double().clamp(1e-300, 1.0)).float()[:, None]) | ~(m > 0)[:, None]
    W = torch.where(keep, W, torch.zeros_like(W))
    greedy = ~(s["temperature"] > 0)
    if k is not None:
        greedy |= k == 1
    best = torch.where(l == top, place, torch.full_like(place, vocab)).min(1, keepdim=True).values
    W = torch.where(greedy[:, None], torch.where(place == best, int(ONE), 0), W)
    W[empty] = 0
    run_sum = torch.cumsum(W, 1)
    Z = run_sum[:, -1:]
    token = (run_sum.double() <= s["uniforms"].double()[:, None] * Z.double()).sum(1)
    last = torch.where(W > 0, place, torch.zeros_like(place)).max(1).values
    token = torch.minimum(token, last)
    t = torch.where(greedy[:, None], W.double() / ONE, torch.where(keep, plain_exp(d).double(), torch.zeros((), dtype=torch.float64, device=l.device)))
    z = Z.double() / ONE
    at = torch.where(greedy, torch.zeros_like(top[:, 0]), d.gather(1, token[:, None])[:, 0]).double()
    out = {"tokens": torch.where(empty, -1, token).int(),
           "logprob": torch.where(empty, torch.full_like(at, -float("inf")), at - torch.log(z[:, 0])).float()}
    if s["case"]["op"] == "draft":
        out["probs"] = torch.where(empty[:, None], torch.zeros_like(t), t / z).float()
    return out


def flat_tokens(s):
    """The token of every row, -1 where none is wanted."""
    if s["cu_num_draft"] is None:
        return s["tokens"].long()
    cu, n = s["cu_num_draft"].long(), s["tokens"].shape[0]
    r = torch.arange(s["logits"].shape[0], device=cu.device)
    i = torch.searchsorted(cu[:-1] + torch.arange(n, device=cu.device), r, right=True) - 1
    return s["tokens"][i, r - cu[i] - i].long()


def plain_logprobs(s):
    l, top, d = plain_rows(s["logits"], None)
    vocab, n = l.shape[1], s["case"]["top"]
    token = flat_tokens(s)
    off = (token < 0) | (token >= vocab)
    at = token.clamp(0, vocab - 1)[:, None]
    norm = torch.log(torch.exp(d).double().sum(1, keepdim=True))
    none = torch.full_like(top, -float("inf"))
    out = {"logprob": torch.where(off[:, None], none, (d.gather(1, at).double() - norm).float())[:, 0],
           "rank": torch.where(off, 0, 1 + (l > l.gather(1, at)).sum(1)).int()}
    if n:
        ls, order = torch.sort(l, dim=1, descending=True, stable=True)
        ids = order[:, :n]
        out["top_ids"] = torch.where(off[:, None], -1, ids).int()
        out["top_logprob"] = torch.where(off[:, None], none, (d.gather(1, ids).double() - norm).float())
    return out


# --------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    if case["rows"] * case["vocab"] > 7e7:
        return None
    s = {k: v.cpu() if torch.is_tensor(v) else v for k, v in prepare(case, seed).items() if k != "out"}
    return exact_logprobs(s) if case["op"] == "logprobs" else exact_sample(s)


def exact_logprobs(s):
    logits, n = s["logits"], s["case"]["top"]
    spec = s["case"]["spec"]
    token = s["tokens"].numpy().reshape(-1)  # request after request, spec + 1 rows each
    rows, vocab = logits.shape
    lp, ids, best = np.full(rows, -np.inf), np.full((rows, n), -1, np.int32), np.full((rows, n), -np.inf)
    for r in range(rows):
        if token[r] < 0:
            continue
        l = logits[r].float().numpy().astype(np.float64)
        norm = l.max() + np.log(np.exp(l - l.max()).sum())
        lp[r] = l[token[r]] - norm
        if n:
            low = np.partition(l, vocab - n)[vocab - n]
            near = np.flatnonzero(l >= low)
            ids[r] = near[np.lexsort((near, -l[near]))][:n]
            best[r] = l[ids[r]] - norm
    assert spec == 0 or rows % (spec + 1) == 0
    out = {"logprob": lp, "rank": None}
    if n:
        out |= {"top_ids": ids, "top_logprob": best}
    return out


def exact_weights(d):
    """W by the definition: the binary32 exp with every operation rounded on its own."""
    f4 = np.float32
    one = lambda a, b, c: (a.astype(np.float64) * np.float64(f4(b)) + np.float64(c)).astype(f4)  # noqa: E731
    x = np.maximum(d, f4(-87))
    k = (one(x, 1 / np.log(2), 1.5 * 2**23) - f4(1.5 * 2**23)).astype(f4)
    r = one(-k, np.log(2), x.astype(np.float64))
    r = one(-k, np.log(2) - np.float64(f4(np.log(2))), r.astype(np.float64))
    p = np.full_like(r, 1 / 5040)
    for c in (1 / 720, 1 / 120, 1 / 24, 1 / 6, 0.5, 1.0, 1.0):
        p = (p.astype(np.float64) * r.astype(np.float64) + np.float64(f4(c))).astype(f4)
    t = np.where(d >= -87, np.ldexp(p, k.astype(np.int32)), f4(0))
    return np.rint(np.ldexp(t.astype(np.float64), 40)).astype(np.int64)


def exact_sample(s):
    logits = s["logits"]
    rows, vocab = logits.shape
    lp = np.empty(rows)
    probs = np.zeros((rows, vocab)) if s["case"]["op"] == "draft" else None
    val = lambda name, r: None if s[name] is None else s[name][r].item()  # noqa: E731
    for r in range(rows):
        l = logits[r].float().numpy()
        T, u, k, P, M = (val(x, r) for x in ("temperature", "uniforms", "top_k", "top_p", "min_p"))
        if not T > 0 or k == 1:
            lp[r] = 0.0
            if probs is not None:
                probs[r, int(np.argmax(l))] = 1.0
            continue
        with np.errstate(over="ignore"):
            d = ((l - l.max()) * (np.float32(1) / np.float32(T))).astype(np.float32)
        W = exact_weights(d)
        floor = -np.inf
        if k is not None and 1 <= k < vocab:
            floor = np.partition(l, vocab - k)[vocab - k]
        if P is not None and P < 1:
            inside = np.flatnonzero(l >= floor)
            value, back = np.unique(l[inside], return_inverse=True)
            mass = np.zeros(value.size, np.int64)
            np.add.at(mass, back, W[inside])
            above = mass.sum() - np.cumsum(mass)
            part = np.float64(np.float32(max(P, np.float32(1e-6))))
            floor = value[np.float64(above) < part * np.float64(mass.sum())].min()
        keep = l >= floor
        if M is not None and M > 0:
            keep &= d >= np.float32(np.log(np.float64(min(M, 1.0))))
        total = np.cumsum(np.where(keep, W, 0))
        token = int(np.searchsorted(total.astype(np.float64), np.float64(u) * np.float64(total[-1]), side="right"))
        x = (l.astype(np.float64) - np.float64(l.max())) / np.float64(T)
        z = np.exp(x[keep]).sum()
        lp[r] = x[min(token, int(np.flatnonzero(keep & (W > 0))[-1]))] - np.log(z)
        if probs is not None:
            probs[r, keep] = np.exp(x[keep]) / z
    out = {"tokens": None, "logprob": lp}
    if probs is not None:
        out["probs"] = probs
    return out


def work(case):
    """Every logit read once, every output written once; per logit a difference, a product, an
    exponential (one operation here) and a sum. Rows of a verification that emitted no token
    need not be read: on average spec / 2 of spec + 1."""
    rows, vocab, size = case["rows"], case["vocab"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "logprobs":
        spec = case["spec"]
        read = rows * (spec + 2) / (2 * (spec + 1))
        return {"bytes": int(read * vocab * size + rows * (12 + 8 * case["top"])), "flops": int(4 * read * vocab)}
    out = 4 * rows * vocab if case["op"] == "draft" else 0
    return {"bytes": rows * (vocab * size + 28) + out, "flops": 4 * rows * vocab}
