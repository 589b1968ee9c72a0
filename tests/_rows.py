"""A plain implementation of the row operators (spec_verify_sample, spec_verify_logprobs): weights
by the oracle's binary32 exp, sums in whole numbers or binary64, one row at a time, and the
comparison with the library's outputs."""
from __future__ import annotations

import numpy as np

import oracle

F4 = np.float32
ONE = 1 << 40


def clean(row) -> np.ndarray:
    """float32 logits, NaN as -inf."""
    l = np.asarray(row, F4)
    return np.where(np.isnan(l), F4(-np.inf), l)


def inverse(T) -> np.float32:
    with np.errstate(all="ignore"):
        return np.clip(F4(1) / F4(T), np.finfo(F4).tiny, np.finfo(F4).max)


def deltas(l: np.ndarray, inv) -> np.ndarray:
    with np.errstate(all="ignore"):
        d = ((l - l.max()).astype(F4) * F4(inv)).astype(F4)
    d[l == l.max()] = 0
    d[np.isneginf(l)] = -np.inf
    return d


def ref_sample_row(row, T=1.0, k=0, P=1.0, M=0.0, u=0.0):
    """(token, log-probability, probabilities, error of d as it enters the log-probability)."""
    l = clean(row)
    V = l.size
    probs = np.zeros(V)
    if np.isneginf(l.max()):
        return -1, -np.inf, probs
    if not T > 0 or k == 1:
        token = int(np.argmax(l))
        probs[token] = 1
        return token, 0.0, probs
    d = deltas(l, inverse(T))
    finite = ~np.isneginf(d)
    t = np.zeros(V, F4)
    t[finite] = oracle.exp32_n(d[finite])
    W = np.rint(t.astype(np.float64) * ONE).astype(np.int64)
    keep = finite.copy()
    if 1 <= k < V:
        keep &= l >= np.sort(l)[V - k]
    if P < 1:
        values, back = np.unique(l, return_inverse=True)       # (-0 and +0 are one value)
        mass = np.zeros(values.size, np.int64)
        np.add.at(mass, back, np.where(keep, W, 0))
        above = mass.sum() - np.cumsum(mass)
        part = np.float64(F4(max(F4(P), F4(1e-6))))
        keep &= (above.astype(np.float64) < part * np.float64(mass.sum()))[back]
    if M > 0:
        keep &= d >= F4(np.log(np.float64(min(F4(M), F4(1)))))
    run = np.cumsum(np.where(keep, W, 0))
    Z = run[-1]
    target = np.float64(u if u > 0 else 0) * np.float64(Z)
    hit = np.flatnonzero(run.astype(np.float64) > target)
    token = int(hit[0]) if hit.size else int(np.flatnonzero(keep & (W > 0))[-1])
    x = np.exp(d[keep].astype(np.float64))
    probs[keep] = x / x.sum()
    return token, float(d[token]) - float(np.log(x.sum())), probs


def check_sample(logits, got, T=None, k=None, P=None, M=None, u=None):
    """got: (tokens, logprob, probs) as numpy arrays, logprob and probs each or None.

    Tolerances. t is within one ulp of exp(d) (pinned by the oracle's tests), 2^-23 relative; Z, a
    sum of the W, the same plus half a unit of 2^-40 a token, over a sum of at least 1:
    2^-23 + V 2^-41. A log-probability is d - ln Z in binary64, rounded once: that bound, and 2^-24
    of its size. A probability is t / fl(Z) rounded once: 2^-23 + 2^-23 + V 2^-41 + 2 2^-24
    relative; and the binary32 exp is 0 below -87 by definition, where exp(d) / Z is below
    exp(-87) < 2^-125."""
    tokens, lp, probs = got
    V = logits.shape[1]
    z_tol = 2.0**-23 + V * 2.0**-41
    for r in range(logits.shape[0]):
        pick = lambda a, d: d if a is None else float(a[r])  # noqa: E731
        kk = 0 if k is None else int(k[r])
        token, l0, p0 = ref_sample_row(logits[r], pick(T, 1.0), kk, pick(P, 1.0), pick(M, 0.0), pick(u, 0.0))
        where = f"row {r}: T={pick(T, 1)} k={kk} P={pick(P, 1)} M={pick(M, 0)} u={pick(u, 0)}"
        assert tokens[r] == token, f"{where}: token {tokens[r]}, expected {token}"
        if lp is not None:
            if np.isinf(l0):
                assert lp[r] == l0, where
            else:
                assert abs(float(lp[r]) - l0) <= z_tol + 2.0**-24 * abs(l0), f"{where}: {lp[r]} {l0}"
        if probs is not None:
            tol = (2 * 2.0**-23 + 2 * 2.0**-24 + V * 2.0**-41) * p0 + 2.0**-125
            bad = np.flatnonzero(~(np.abs(probs[r].astype(np.float64) - p0) <= tol))
            assert bad.size == 0, f"{where}: {bad.size} probabilities off, first {bad[0]}: {probs[r, bad[0]]} {p0[bad[0]]}"


def ref_logprobs_row(row, token, n=0, T=1.0):
    """(log-probability, rank, best ids, their log-probabilities)."""
    l = clean(row)
    V = l.size
    ids, best = np.full(n, -1), np.full(n, -np.inf)
    if token is not None and not 0 <= token < V:
        return -np.inf, 0, ids, best
    if np.isneginf(l.max()):
        return -np.inf, 1, ids, best
    d = deltas(l, inverse(T) if T > 0 else 1.0).astype(np.float64)
    norm = np.log(np.exp(d).sum())
    order = np.lexsort((np.arange(V), -l))[:n]
    order = order[~np.isneginf(l[order])]
    ids[:order.size], best[:order.size] = order, d[order] - norm
    token = 0 if token is None else token
    return d[token] - norm, 1 + int((l > l[token]).sum()), ids, best


def check_logprobs(logits, got, tokens=None, n=0, T=None, exp_tol=2.0**-21):
    """got: (logprob, rank, top_ids, top_logprobs), those that were asked for.

    Tolerances: the sum's terms are taken within 2^-21 (a binary32 2^x of 2 ulp, 2^-22, and its
    argument's rounding: at most 2^-24 |x| ln 2 for an x whose term is 2^x, so below 2^-24 on
    average) and added in binary32, by threads that hold at most a few hundred terms each and then
    in pairs: below 2^-21 more for terms of one sign. Then one rounding of the result."""
    named = dict(zip((["logprob", "rank"] if tokens is not None else []) + ["ids", "best"], got))
    for r in range(logits.shape[0]):
        token = None if tokens is None else int(tokens[r])
        lp, rank, ids, best = ref_logprobs_row(logits[r], token, n, 1.0 if T is None else float(T[r]))
        close = lambda a, b: a == b or abs(a - b) <= 2 * exp_tol + 2.0**-23 * abs(b)  # noqa: E731
        where = f"row {r}, token {token}"
        if token is not None:
            assert named["rank"][r] == rank, f"{where}: rank {named['rank'][r]}, expected {rank}"
            assert close(float(named["logprob"][r]), lp), f"{where}: {named['logprob'][r]} {lp}"
        if n:
            np.testing.assert_array_equal(named["ids"][r], ids, err_msg=where)
            assert all(close(float(a), b) for a, b in zip(named["best"][r], best)), where


def rows_of(seed, R, V, dtype="bf16", sigma=2.0, peak=(8.0, 22.0), n_peak=32):
    """Rows of logits as float32 values of the type: a bell of unlikely tokens and some favoured ones."""
    rng = np.random.default_rng(seed)
    l = (rng.standard_normal((R, V)) * sigma).astype(F4)
    for r in range(R):
        n = min(n_peak, V)
        l[r, rng.integers(0, V, n)] = rng.uniform(*peak) * rng.uniform(0.5, 1.0, n)
    if dtype == "bf16":
        from _util import bf16_bits_to_f32, to_bf16_bits

        l = bf16_bits_to_f32(to_bf16_bits(l)).reshape(R, V)
    return l


def on_gpu(l, dtype, stride=None):
    """The rows on the GPU in `dtype`, `stride` elements apart (what lies between them is NaN)."""
    import torch

    t = torch.from_numpy(np.ascontiguousarray(l)).cuda()
    t = t.to(torch.bfloat16) if dtype == "bf16" else t
    if stride is None:
        return t
    wide = torch.full((t.shape[0], stride), float("nan"), dtype=t.dtype, device="cuda")
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]
