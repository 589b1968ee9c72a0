"""A plain implementation of the cache operators (spec_verify_cache_append, spec_verify_cache_attention) in 64
bits, one row at a time, with what each output may be off by, counted from the roundings the operators
make; and steps to run them on."""
from __future__ import annotations

import numpy as np
import torch

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
HALF = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.float32)}


def smallest(dtype) -> float:
    f = torch.finfo(dtype)
    return f.tiny * f.eps


class Step:
    """A step's requests, their places in a paged cache, and the cache, on the CPU. `lengths` before the step, `new`
    rows a request; every request that takes part gets the pages of its places, in any order."""

    def __init__(self, seed, lengths, new, *, hq=8, hk=2, dim=64, dtype="bf16", cache="bf16", page=16,
                 layout="tokens", share=1.0, spare=0, fill=None):
        g = torch.Generator().manual_seed(seed)
        self.n, self.hq, self.hk, self.dim, self.page = len(lengths), hq, hk, dim, page
        self.dtype, self.kind, self.layout = TYPES[dtype], TYPES[cache], layout
        self.lengths = torch.tensor(lengths, dtype=torch.int32)
        self.new = list(new)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(np.array(new) - 1)]), dtype=torch.int32)
        self.rows = int(sum(new))
        used = [-(-max(0, x + m) // page) if x >= 0 else 0 for x, m in zip(lengths, new)]
        self.width, self.pool = max(used) + spare, sum(used) + 3
        order = torch.randperm(self.pool, generator=g)
        self.table = torch.full((self.n, self.width), 2**30, dtype=torch.int32)  # (entries that are not read)
        at = 0
        for i, u in enumerate(used):
            self.table[i, :u] = order[at:at + u].int()
            at += u
        self.k_scale = self.v_scale = None
        shape = (self.pool, page, hk, dim)
        loud = 1.0
        if cache == "e4m3":
            self.k_scale, self.v_scale = 0.01 + 0.05 * torch.rand(hk, generator=g), 0.01 + 0.05 * torch.rand(hk, generator=g)
            loud = 30.0
        make = lambda s, f: (torch.randn(s, generator=g) * f).clamp(-440, 440)  # noqa: E731
        self.k_cache, self.v_cache = make(shape, loud).to(self.kind), make(shape, loud).to(self.kind)
        if fill is not None:
            self.k_cache.fill_(fill)
            self.v_cache.fill_(fill)
        self.q = make((self.rows, hq, dim), share).to(self.dtype)
        self.k, self.v = make((self.rows, hk, dim), 1.0).to(self.dtype), make((self.rows, hk, dim), 1.0).to(self.dtype)
        self.first = [int(self.cu[i]) + i for i in range(self.n)]

    def rows_of(self):
        """(row, request, place) of every row of the step."""
        for i in range(self.n):
            for j in range(self.new[i]):
                yield self.first[i] + j, i, int(self.lengths[i]) + j

    def slot(self, i, x):
        page = int(self.table[i, x // self.page]) if 0 <= x < self.width * self.page else -1
        return (page, x % self.page) if 0 <= page < self.pool else None

    def device_caches(self):
        """The caches on the GPU, in the step's layout: pages of tokens, pages of heads, or keys and values
        of a page side by side."""
        if self.layout == "tokens":
            return self.k_cache.cuda(), self.v_cache.cuda()
        if self.layout == "heads":
            return tuple(c.transpose(1, 2).contiguous().cuda().transpose(1, 2) for c in (self.k_cache, self.v_cache))
        both = torch.stack((self.k_cache, self.v_cache), 1).cuda()
        return both[:, 0], both[:, 1]


def ref_append(s: Step, inv_freq=None, positions=None, axes=None, interleaved=False):
    """(q, k cache, v cache) in 64 bits, and what each element may be off by."""
    inv = torch.zeros(0) if inv_freq is None else inv_freq
    m = inv.numel()
    q, qe = s.q.double(), torch.zeros(s.q.shape, dtype=torch.float64)
    out = {"k": s.k_cache.double(), "v": s.v_cache.double()}
    err = {x: torch.zeros(s.k_cache.shape, dtype=torch.float64) for x in out}
    lo, hi = (slice(0, 2 * m, 2), slice(1, 2 * m, 2)) if interleaved else (slice(0, m), slice(m, 2 * m))

    def turn(x, pos):
        """x [heads, dim] turned; the error before the last rounding."""
        y, e = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64)
        a = pos.double() * inv.double()
        cos, sin = torch.cos(a), torch.sin(a)
        one, two = y[:, lo].clone(), y[:, hi].clone()
        y[:, lo], y[:, hi] = one * cos - two * sin, one * sin + two * cos
        # the angle; sincospi's 2 units of 2^-24 (of values up to 1) and its argument's rounding (pi 2^-24);
        # two products and a sum
        size = (one.abs() + two.abs()) * (a.abs() * 2.0**-47 + 2.0**-29 + 8 * 2.0**-24)
        e[:, lo] = e[:, hi] = size
        return y, e

    for r, i, x in s.rows_of():
        if int(s.lengths[i]) < 0:
            q[r], qe[r] = float("nan"), 0      # (not written)
            continue
        pos = torch.full((m,), x) if positions is None else positions.view(-1, s.rows)[[0] * m if axes is None else list(axes), r]
        q[r], e = turn(s.q[r], pos)
        qe[r] = e + (q[r].abs() + e) * HALF[s.dtype] + smallest(s.dtype) / 2
        at = s.slot(i, x)
        if at is None:
            continue
        for name, (y, e), scale in (("k", turn(s.k[r], pos), s.k_scale), ("v", (s.v[r].double(), torch.zeros(s.v[r].shape, dtype=torch.float64)), s.v_scale)):
            if scale is not None:
                y, e = y / scale.double()[:, None], e / scale.double()[:, None]
                e = (e + y.abs() * 2.0**-23) * 1.01   # (the reciprocal's rounding and the product's)
            most = torch.finfo(s.kind).max
            e = e + (y.abs() + e) * HALF[s.kind] + smallest(s.kind) / 2
            out[name][at] = y.clamp(-most, most) if s.kind is TYPES["e4m3"] else y
            err[name][at] = e
    return (q, out["k"], out["v"]), (qe, err["k"], err["v"])


def ref_attention(s: Step, *, scale=None, window=0):
    """(out, lse) in 64 bits and what they may be off by. A weight is rounded to the 16-bit type of the products
    (binary16 for e4m3), relative to the largest of its row; sums and scores are binary32, added by units that
    may cut instead of round (a step of 2^-22 an addition)."""
    scale = s.dim ** -0.5 if scale is None else scale
    group = s.hq // s.hk
    out, lse = torch.full(s.q.shape, float("nan"), dtype=torch.float64), torch.full(s.q.shape[:2], float("nan"), dtype=torch.float64)
    oe, le = torch.zeros_like(out), torch.zeros_like(lse)
    keys, values = s.k_cache.double(), s.v_cache.double()
    weight = HALF[torch.bfloat16 if s.kind is torch.bfloat16 else torch.float16]
    for r, i, x in s.rows_of():
        last = x if int(s.lengths[i]) >= 0 else -1
        at = [p for t in range(max(0, x - window + 1) if window else 0, last + 1) if (p := s.slot(i, t)) is not None]
        if not at:
            out[r], lse[r] = 0, -float("inf")
            continue
        page, slot = (torch.tensor(a) for a in zip(*at))
        for h in range(s.hk):
            k, v = keys[page, slot, h], values[page, slot, h]
            ks, vs = (1.0 if c is None else float(c[h].double()) for c in (s.k_scale, s.v_scale))
            q = s.q[r, h * group:(h + 1) * group].double()
            score = q @ k.T * (ks * scale)
            z = torch.logsumexp(score, 1)
            p = (score - z[:, None]).exp()
            y = p @ v * vs
            big = abs(ks * scale)
            # a score: its products added one after another, the factor's rounding, the argument of 2^x
            off = (q.abs() @ k.abs().T * (s.dim * 2.0**-22) + q.abs().amax(1, keepdim=True) * k.abs().sum(1) * 2.0**-35) * big
            off = off.amax(1) + 3 * 2.0**-24 * torch.where(torch.isfinite(score), score.abs(), 0).amax() + 2.0**-22
            n = len(at)
            size = p @ v.abs() * abs(vs)
            o = slice(h * group, (h + 1) * group)
            out[r, o], lse[r, o] = y, z
            many = (n / 8 + 32) * 2.0**-22
            oe[r, o] = size * (weight + 2 * off[:, None] + 2 * many) * 1.01 + y.abs() * HALF[s.dtype] * 1.01 + smallest(s.dtype)
            # binary16 weights are held 11 doublings above the reference, itself at most the row's largest: half their
            # smallest step, 2^-24, is 2^-36 of that
            oe[r, o] += v.abs().sum(0) * abs(vs) * 2.0**-36 * p.amax(1, keepdim=True)
            le[r, o] = off + many + 2.0**-22 * z.abs()
    return (out, lse), (oe, le)


def off_by(got, want, err, what):
    """Assert that `got` is within `err` of `want`; NaN in `want`: not looked at."""
    got, want = got.detach().cpu().double(), want.double()
    looked = ~torch.isnan(want)
    same = (got == want) | ~looked
    far = ~same & ~((got - want).abs() <= err)
    if bool(far.any()):
        k = far.nonzero()[0].tolist()
        raise AssertionError(f"{what}: {int(far.sum())} of {int(looked.sum())} too far, first at {k}: {got[tuple(k)]} for {want[tuple(k)]}, "
                             f"allowed {err[tuple(k)]}; largest {float(((got - want).abs() / err.clamp(min=1e-300))[looked & ~same].max())} of the bound")


def cuda(t):
    return None if t is None else t.cuda()


def append(s: Step, caches=None, **kw):
    """The operator on a step: (q, k cache, v cache) on the GPU."""
    import speculative_decoding_verification_rejection_gb300 as sv

    k, v = caches or s.device_caches()
    q = sv.cache_append(cuda(s.k), cuda(s.v), k, v, cuda(s.table), cuda(s.lengths), q=cuda(s.q), cu_num_draft=cuda(s.cu), k_scale=cuda(s.k_scale),
                        v_scale=cuda(s.v_scale), **kw)
    return q, k, v


def attention(s: Step, caches=None, **kw):
    import speculative_decoding_verification_rejection_gb300 as sv

    k, v = caches or s.device_caches()
    return sv.cache_attention(cuda(s.q), k, v, cuda(s.table), cuda(s.lengths), cu_num_draft=cuda(s.cu), k_scale=cuda(s.k_scale),
                              v_scale=cuda(s.v_scale), lse=True, **kw)


def check_append(s: Step, label="", **kw):
    on = {a: cuda(b) if torch.is_tensor(b) else b for a, b in kw.items()}
    got = append(s, **on)
    want, err = ref_append(s, **kw)
    for name, g, w, e in zip(("q", "k_cache", "v_cache"), got, want, err):
        off_by(g, w, e, f"{label} {name}")


def check_attention(s: Step, label="", **kw):
    got = attention(s, **kw)
    want, err = ref_attention(s, **kw)
    for name, g, w, e in zip(("out", "lse"), got, want, err):
        off_by(g, w, e, f"{label} {name}")
