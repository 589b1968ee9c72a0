"""The row operators on the GPU against the plain implementation of tests/_rows.py."""
import os
import subprocess
import sys

import numpy as np
import pytest

from _parity import assert_parity, canary_buffer, check_canaries, to_device
from _rows import check_logprobs, check_sample, on_gpu, ref_sample_row, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch

    assert torch.cuda.is_available(), "these tests need a CUDA device"
    import speculative_decoding_verification_rejection_gb300 as sv

    sv.lib()


def dev(a, dtype):
    import torch

    return None if a is None else torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype))).cuda()


def run_sample(l, dtype, u, T=None, k=None, P=None, M=None, *, stride=None, probs=True, probs_stride=None):
    """The library on rows l, with canaries round every output and between the probs' rows."""
    import torch

    import speculative_decoding_verification_rejection_gb300 as sv

    R, V = l.shape
    bt, tok = canary_buffer((R,), torch.int32, "cuda")
    bl, lp = canary_buffer((R,), torch.float32, "cuda")
    out = [tok, lp]
    if probs:
        ps = probs_stride or V
        bp, pr = canary_buffer((R, ps), torch.float32, "cuda")
        pr.fill_(-7.0)
        out.append(pr[:, :V])
    got = sv.sample(on_gpu(l, dtype, stride), dev(u, np.float32), dev(T, np.float32), top_k=dev(k, np.int32),
                    top_p=dev(P, np.float32), min_p=dev(M, np.float32), logprob=True, probs=probs, out=out)
    torch.cuda.synchronize()
    check_canaries(bt, "tokens")
    check_canaries(bl, "logprob")
    if probs:
        check_canaries(bp, "probs")
        assert bool((pr[:, V:] == -7.0).all())
    return [g.cpu().numpy() for g in got] + ([] if probs else [None])


def same_tokens_without_probs(l, dtype, got, u, **kw):
    other = run_sample(l, dtype, u, probs=False, **kw)
    np.testing.assert_array_equal(other[0], got[0])
    np.testing.assert_array_equal(other[1], got[1])


SIZES = [1, 2, 3, 7, 8, 9, 31, 64, 129, 1000, 1001, 4099, 20011, 32000, 40003, 151936]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", SIZES)
def test_sample_sizes(V, dtype):
    """Every size with each constraint and their mixtures."""
    R = 24 if V < 30000 else 9
    rng = np.random.default_rng(V)
    l = rows_of(V, R, V, dtype)
    T = rng.uniform(0.3, 1.6, R)
    k = rng.choice([0, 1, 2, 5, 50, 300, 2000, V, V - 1], R)
    P = rng.choice([1.0, 0.99, 0.9, 0.5, 0.05], R)
    M = rng.choice([0.0, 0.0, 0.02, 0.3], R)
    u = rng.random(R)
    none = dict(T=T, u=u)
    for kw in (none, {**none, "k": k}, {**none, "P": P}, {**none, "M": M}, {**none, "k": k, "P": P, "M": M}):
        got = run_sample(l, dtype, **kw)
        check_sample(l, got, **kw)
    same_tokens_without_probs(l, dtype, got, **kw)


@pytest.mark.parametrize("sigma", [0.0, 0.01, 0.5, 2.0])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sample_flat_rows(dtype, sigma):
    """Rows without favoured tokens: kept sets of tens of thousands of tokens, and (sigma 0) of
    tokens that are all equal."""
    R, V = 8, 50021
    rng = np.random.default_rng(17)
    l = rows_of(18, R, V, dtype, sigma=sigma, n_peak=0)
    kw = dict(T=np.full(R, 1.0), k=np.array([0, 0, 0, 30000, 30000, 100, 0, 49000]),
              P=np.array([1.0, 0.9, 0.999, 1.0, 0.5, 0.5, 0.1, 0.97]),
              M=np.array([0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.1, 0.0]), u=rng.random(R))
    check_sample(l, run_sample(l, dtype, **kw), **kw)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sample_settings_at_their_ends(dtype):
    """Every value the arguments may take, those that mean no constraint among them."""
    V = 777
    ks = [-3, 0, 1, 2, V - 1, V, V + 9, 2**31 - 1, -2**31]
    Ps = [1.0, 2.0, NAN, INF, 0.0, -1.0, 1e-9, 0.5, np.nextafter(np.float32(1), np.float32(0))]
    Ms = [0.0, -1.0, NAN, 1.0, 5.0, 1e-38, 1e-45, 0.2, INF]
    Ts = [1.0, 0.0, -2.0, NAN, INF, 1e-45, 1e-30, 1e30, 0.01]
    us = [0.0, 0.5, 1 - 2.0**-24, 1.0, 7.0, -1.0, NAN, 2.0**-24, 1e-45]
    rows = []
    for vals, i in ((ks, 0), (Ps, 1), (Ms, 2), (Ts, 3), (us, 4)):
        for v in vals:
            row = [0, 1.0, 0.0, 1.0, 0.37]
            row[i] = v
            rows.append(row)
    rng = np.random.default_rng(3)
    for _ in range(60):
        rows.append([rng.choice(ks), rng.choice(Ps), rng.choice(Ms), rng.choice(Ts), rng.choice(us)])
    k, P, M, T, u = (np.array(c) for c in zip(*rows))
    l = rows_of(5, len(rows), V, dtype)
    kw = dict(T=T.astype(np.float32), k=k.astype(np.int64), P=P.astype(np.float32), M=M.astype(np.float32),
              u=u.astype(np.float32))
    got = run_sample(l, dtype, **kw)
    check_sample(l, got, **kw)
    same_tokens_without_probs(l, dtype, got, **kw)


def special_rows(V, seed, low):
    """Masked rows, infinities, NaN, ties, signed zeros, values at the type's ends."""
    rng = np.random.default_rng(seed)
    base = rows_of(seed, 14, V, "bf16")
    base[0] = -INF
    base[1] = NAN
    base[2] = -INF
    base[2, V // 2] = -3.0                                   # one token left
    base[3, rng.random(V) < 0.9] = -INF
    base[4, rng.random(V) < 0.5] = NAN
    base[5, [0, V // 3, V - 1]] = INF
    base[6, V // 3] = INF
    base[6, : V // 4] = -INF
    base[7] = 2.5                                            # all equal
    base[8] = np.where(rng.random(V) < 0.5, 0.0, -0.0)       # equal, though not bit for bit
    base[9] = low                                            # masked by the lowest value
    base[9, 5 % V] = 1.0
    base[10] = low                                           # all masked by it
    base[11] = -low
    base[11, V // 2:] = low
    base[12, : V - 1] = -INF
    base[13] = np.where(rng.random(V) < 0.3, -INF, np.round(base[13]))   # many ties
    return base


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [8, 61, 1000, 33333])
def test_sample_special_rows(V, dtype):
    low = -3.3895313892515355e38 if dtype == "bf16" else -3.4028234663852886e38
    l = special_rows(V, V, low)
    R = l.shape[0]
    rng = np.random.default_rng(V + 1)
    u = rng.random(R)
    for kw in (dict(u=u), dict(u=u, T=rng.uniform(0.3, 2, R), k=np.full(R, 40)), dict(u=u, P=np.full(R, 0.8)),
               dict(u=u, M=np.full(R, 0.1)), dict(u=0 * u, k=np.full(R, 3), P=np.full(R, 0.9)),
               dict(u=u, k=np.full(R, V - 1)), dict(u=u, T=np.zeros(R)), dict(u=0 * u + 1),
               dict(u=u, T=np.full(R, INF))):
        check_sample(l, run_sample(l, dtype, **kw), **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,stride,probs_stride", [(1000, 1024, 1000), (1001, 1003, 1002), (33, 40, 64), (20011, 20013, 20015)])
def test_sample_strides(V, stride, probs_stride, dtype):
    """Rows further apart than they are long, and starting at every offset from 16 bytes."""
    R = 19
    rng = np.random.default_rng(V)
    l = rows_of(V, R, V, dtype)
    for kw in (dict(u=rng.random(R)), dict(u=rng.random(R), k=np.full(R, 20), P=np.full(R, 0.9))):
        check_sample(l, run_sample(l, dtype, stride=stride, probs_stride=probs_stride, **kw), **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1500, 9001])
def test_sample_more_rows_than_the_device_holds(V, dtype):
    """Over 600 rows take the smaller blocks; every kind of row is among them."""
    R = 640
    rng = np.random.default_rng(V)
    l = rows_of(V, R, V, dtype)
    l[::7] = rows_of(V + 1, l[::7].shape[0], V, dtype, sigma=1.0, n_peak=0)
    special = special_rows(V, V + 2, -1e30)
    l[300:300 + special.shape[0]] = special
    if dtype == "bf16":
        from _util import bf16_bits_to_f32, to_bf16_bits

        l = bf16_bits_to_f32(to_bf16_bits(l)).reshape(R, V)
    kw = dict(T=rng.choice([0.0, 0.5, 1.0, 1.4], R), k=rng.choice([0, 0, 0, 1, 20, 200, 700, V - 2], R),
              P=rng.choice([1.0, 0.95, 0.5], R), M=rng.choice([0.0, 0.0, 0.05], R), u=rng.random(R))
    got = run_sample(l, dtype, **kw)
    check_sample(l, got, **kw)
    same_tokens_without_probs(l, dtype, got, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R", [4, 30, 160, 620])
def test_heavy_tailed_rows(R, dtype):
    """Probabilities that fall as a power of the rank: top-p sets of all sizes from one token to most
    of the row, with many equal bf16 logits at their borders; positive, mixed and negative logits."""
    V = 30011 if R < 100 else 5003
    rng = np.random.default_rng(V + R)
    l = np.empty((R, V))
    for r in range(R):
        l[r] = rng.permutation(-rng.uniform(0.9, 2.0) * np.log(np.arange(1, V + 1))) + rng.choice([0.0, 4.0, 30.0])
    l = (l + 0.3 * rng.standard_normal((R, V))).astype(np.float32)
    if dtype == "bf16":                                      # what the GPU gets
        from _util import bf16_bits_to_f32, to_bf16_bits

        l = bf16_bits_to_f32(to_bf16_bits(l)).reshape(R, V)
    kw = dict(P=rng.choice([0.5, 0.9, 0.99], R), u=rng.random(R))
    check_sample(l, run_sample(l, dtype, **kw), **kw)
    kw["T"] = rng.choice([0.6, 1.0, 1.5], R)
    got = run_sample(l, dtype, **kw)
    check_sample(l, got, **kw)
    same_tokens_without_probs(l, dtype, got, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R", [6, 24, 70, 160, 620])
def test_k_from_small_to_beyond_the_list(R, dtype):
    """Every k between what a CTA lists for sure and what no list holds, by rows split over many CTAs
    to rows of one small block."""
    V = 40003 if R < 100 else 6007
    rng = np.random.default_rng(R)
    l = rows_of(R, R, V, dtype, sigma=2.0, n_peak=0)
    for low, high in ((60, 200), (200, 520), (500, 1100)):
        kw = dict(k=rng.integers(low, high, R), P=rng.choice([1.0, 0.9], R), u=rng.random(R))
        check_sample(l, run_sample(l, dtype, **kw), **kw)


@pytest.mark.parametrize("R", [305, 512, 513, 608])
@pytest.mark.parametrize("kinds", ["both", "long", "short"])
def test_rows_of_both_kinds_in_any_number(R, kinds):
    """Where the device does not hold all rows at once those with large top-p sets or k may start
    first; each row is drawn once, by its own limits."""
    V = 1300
    rng = np.random.default_rng(R)
    l = rows_of(R, R, V, "f32", sigma=1.0, n_peak=4)
    k = {"both": [0, 0, 1, 30, 511, 512, 513, 900, V], "long": [0, 513, 1200], "short": [1, 20, 512]}[kinds]
    P = {"both": [1.0, 0.9, 0.3], "long": [0.99, 0.9], "short": [1.0, 0.8]}[kinds]
    kw = dict(k=rng.choice(k, R), P=rng.choice(P, R), u=rng.random(R))
    for more in ({}, {"T": rng.choice([0.0, 1.0, 0.7] if kinds == "both" else [0.9, 1.1], R)}):
        got = run_sample(l, "f32", **kw, **more)
        check_sample(l, got, **kw, **more)
    same_tokens_without_probs(l, "f32", got, **kw, **more)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R", [2, 40, 200])
def test_favoured_tokens_side_by_side(R, dtype):
    """The largest logits stand next to one another, so that one part of the row holds them all."""
    V, n = 70001, 400
    rng = np.random.default_rng(R)
    l = rows_of(R, R, V, dtype, n_peak=0)
    at = rng.integers(0, V - n, R)
    for r in range(R):
        l[r, at[r]:at[r] + n] = 12.0 + rng.permutation(n) / 64.0
    if dtype == "bf16":                                      # what the GPU gets
        from _util import bf16_bits_to_f32, to_bf16_bits

        l = bf16_bits_to_f32(to_bf16_bits(l)).reshape(R, V)
    k = rng.choice([0, 30, 90, 150, 399, 401, 900], R)
    kw = dict(k=k, P=rng.choice([1.0, 0.9], R), u=rng.random(R))
    check_sample(l, run_sample(l, dtype, **kw), **kw)
    tokens = at + rng.integers(0, n, R)
    check_logprobs(l, run_logprobs(l, dtype, tokens, 64), tokens, 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,V", [(3, 151936), (170, 20011), (2, 524288)])
def test_sample_wide_top_p(R, V, dtype):
    """Top-p sets of thousands of tokens: flat, steep and tied rows, with and without min-p and k."""
    rng = np.random.default_rng(V)
    l = rows_of(V, R, V, dtype, sigma=2.0, n_peak=8, peak=(6.0, 12.0))
    l[1] = np.round(l[1])
    kw = dict(T=rng.uniform(0.8, 2.0, R), P=rng.choice([0.9, 0.99, 0.6, 0.9999], R), u=rng.random(R))
    check_sample(l, run_sample(l, dtype, **kw), **kw)
    kw.update(M=rng.choice([0.0, 1e-3, 1e-2], R), k=rng.choice([0, V // 2, 5000], R))
    check_sample(l, run_sample(l, dtype, **kw), **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [{}, {"k": 7}, {"P": 0.8}, {"M": 0.03}, {"k": 40, "P": 0.95, "M": 0.01}])
def test_evenly_spaced_uniforms_draw_the_distribution(dtype, kw):
    """N uniforms (i + 1/2) / N on N copies of a row: token v is drawn N p_v times, to within one
    (its interval of the running sum holds that many of them)."""
    N, V = 4096, 300
    l = np.repeat(rows_of(11, 1, V, dtype, peak=(4.0, 8.0)), N, 0)
    u = ((np.arange(N) + 0.5) / N).astype(np.float32)
    args = {a: np.full(N, v) for a, v in kw.items()}
    tok, _, _ = run_sample(l, dtype, u, probs=False, **args)
    p = ref_sample_row(l[0], **kw, u=0.5)[2]
    assert np.abs(np.bincount(tok, minlength=V) - N * p).max() <= 1.0 + 1e-3
    assert (np.diff(tok) >= 0).all()                        # the inverse of a running sum


def test_many_rows_past_32_bit_offsets():
    """Rows whose elements lie beyond 2^31 (the last of 2^31 / V + 40 rows are compared)."""
    import torch

    import speculative_decoding_verification_rejection_gb300 as sv

    V = 151936
    R = 2**31 // V + 40
    logits = torch.full((R, V), -20.0, dtype=torch.bfloat16, device="cuda")
    l = rows_of(2, 6, V, "bf16")
    logits[-6:] = torch.from_numpy(l).cuda().bfloat16()
    u = torch.rand(R, device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    k = torch.full((R,), 50, dtype=torch.int32, device="cuda")
    tok, lp = sv.sample(logits, u, top_k=k, logprob=True)
    got = [tok[-6:].cpu().numpy(), lp[-6:].cpu().numpy(), None]
    check_sample(l, got, k=np.full(6, 50), u=u[-6:].cpu().numpy())
    want = (torch.clamp(u.double() * V, max=V - 1)).floor().int()    # equal logits: an even draw
    assert (tok[:-6] - want[:-6]).abs().max() <= 1
    t = torch.from_numpy(np.arange(R, dtype=np.int32) % V).cuda()
    got = sv.logprobs(logits, t, num_top=3)
    check_logprobs(l, [g[-6:].cpu().numpy() for g in got], t[-6:].cpu().numpy(), 3)


# ------------------------------------------------------------------------------- logprobs

def run_logprobs(l, dtype, tokens=None, n=0, T=None, *, stride=None, sampled=None, cu=None):
    import torch

    import speculative_decoding_verification_rejection_gb300 as sv

    R = l.shape[0]
    bufs, out = [], []
    want = [((R,), torch.float32), ((R,), torch.int32)] if tokens is not None or sampled is not None else []
    want += [((R, n), torch.int32), ((R, n), torch.float32)] if n else []
    for shape, dt in want:
        b, v = canary_buffer(shape, dt, "cuda")
        bufs.append(b)
        out.append(v)
    t = dev(tokens if sampled is None else sampled, np.int32) if tokens is not None or sampled is not None else None
    got = sv.logprobs(on_gpu(l, dtype, stride), t, num_top=n, temperature=dev(T, np.float32),
                      cu_num_draft=dev(cu, np.int32), out=out)
    torch.cuda.synchronize()
    for b in bufs:
        check_canaries(b, "logprobs output")
    return [g.cpu().numpy() for g in got]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", SIZES)
def test_logprobs_sizes(V, dtype):
    R = 14 if V < 30000 else 7
    rng = np.random.default_rng(V)
    l = rows_of(V + 1, R, V, dtype)
    tokens = rng.integers(0, V, R)
    tokens[0], tokens[1], tokens[2] = int(np.argmax(l[0])), -1, V
    T = rng.uniform(0.3, 1.7, R)
    T[3] = 0.0
    for n in (0, 1, 5, 20, 64):
        check_logprobs(l, run_logprobs(l, dtype, tokens, n), tokens, n)
    check_logprobs(l, run_logprobs(l, dtype, tokens, 4, T), tokens, 4, T)
    check_logprobs(l, run_logprobs(l, dtype, None, 3), None, 3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [8, 61, 1000, 33333])
def test_logprobs_special_rows(V, dtype):
    low = -3.3895313892515355e38 if dtype == "bf16" else -3.4028234663852886e38
    l = special_rows(V, V + 7, low)
    rng = np.random.default_rng(V)
    for n in (0, 3, 64):
        tokens = rng.integers(0, V, l.shape[0])
        check_logprobs(l, run_logprobs(l, dtype, tokens, n), tokens, n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,stride", [(1000, 1016), (1001, 1003), (20011, 20013)])
def test_logprobs_strides(V, stride, dtype):
    l = rows_of(V, 17, V, dtype)
    tokens = np.arange(17) * 50 % V
    check_logprobs(l, run_logprobs(l, dtype, tokens, 6, stride=stride), tokens, 6)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_start_off_a_16_byte_boundary(dtype):
    """A view whose first row starts one element into its storage and whose last row ends it."""
    import torch

    import speculative_decoding_verification_rejection_gb300 as sv

    R, V = 5, 3001
    l = rows_of(61, R, V, dtype)
    flat = torch.cat([torch.full((1,), float("inf"), device="cuda"), on_gpu(l, "f32").reshape(-1)])
    view = flat.to(torch.bfloat16 if dtype == "bf16" else torch.float32)[1:].view(R, V)
    u = np.random.default_rng(62).random(R)
    got = sv.sample(view, dev(u, np.float32), top_p=dev(np.full(R, 0.9), np.float32), logprob=True, probs=True)
    check_sample(l, [g.cpu().numpy() for g in got], P=np.full(R, 0.9), u=u.astype(np.float32))
    check_logprobs(l, [g.cpu().numpy() for g in sv.logprobs(view, got[0], num_top=4)], got[0].cpu().numpy(), 4)


def test_logprobs_of_a_verification_with_uneven_drafts():
    """Rows found through cu_num_draft, with tokens of -1 left out; and prefix sums that are not
    those of the rows, which may only leave rows out."""
    rng = np.random.default_rng(9)
    K = np.array([3, 0, 5, 1, 0, 0, 4, 2])
    cu = np.concatenate([[0], np.cumsum(K)])
    R, V, width = int(cu[-1]) + K.size, 5003, 6
    l = rows_of(10, R, V, "bf16")
    sampled = np.full((K.size, width), -1)
    flat = np.full(R, -1)
    for i, k in enumerate(K):
        m = rng.integers(0, k + 1) + 1
        sampled[i, :m] = rng.integers(0, V, m)
        flat[cu[i] + i: cu[i] + i + m] = sampled[i, :m]
    check_logprobs(l, run_logprobs(l, "bf16", sampled=sampled, cu=cu, n=4), flat, 4)
    for bad in ([0] * 9, [-2**31] * 9, [2**31 - 1] * 9, [0, 9, -5, 2**31 - 1, 3, -2**31, 7, 7, 8]):
        lp, rank = run_logprobs(l, "bf16", sampled=sampled, cu=np.array(bad))
        assert ((rank >= 0) & (rank <= V)).all() and not np.isnan(lp).any()


# -------------------------------------------------------------------- as they are used together

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_draft_verify_and_logprobs_in_a_row(dtype):
    """A step of speculative decoding: K draft tokens a request drawn from the draft's rows with
    their distributions, verified against the target's logits with those distributions as q,
    and the log-probabilities of what came out. Verification against the oracle, which gets the
    library's own draft."""
    import torch

    import oracle
    import speculative_decoding_verification_rejection_gb300 as sv
    import workloads

    n, K, V = 12, 3, 4001
    target, draft = rows_of(21, n * (K + 1), V, dtype), rows_of(22, n * K, V, dtype)
    tr = target.reshape(n, K + 1, V)
    draft = (0.7 * tr[:, :K] + 0.3 * draft.reshape(n, K, V)).reshape(n * K, V).astype(np.float32)
    if dtype == "bf16":
        from _util import bf16_bits_to_f32, to_bf16_bits

        draft = bf16_bits_to_f32(to_bf16_bits(draft)).reshape(n * K, V)
    rng = np.random.default_rng(23)
    T = np.repeat(rng.uniform(0.6, 1.2, n), K).astype(np.float32)
    u = rng.random(n * K).astype(np.float32)
    q = torch.full((n * K, V), -1.0, device="cuda")
    ids = torch.full((n * K,), -9, dtype=torch.int32, device="cuda")
    dl = on_gpu(draft, dtype).view(n, K, V)
    for j in range(K):                          # one draft step: row j of every request
        rows = torch.arange(n, device="cuda") * K + j
        tok, prob = sv.sample(dl[:, j], dev(u, np.float32)[rows], dev(T, np.float32)[rows].contiguous(), probs=True)
        ids[rows], q[rows] = tok, prob
    check_sample(draft, (ids.cpu().numpy(), None, q.cpu().numpy()), T=T, u=u)
    from _util import to_bf16_bits

    b = workloads.Batch(name="chain", logits=to_bf16_bits(target) if dtype == "bf16" else target, logits_dtype=dtype,
                        vocab_size=V, draft_ids=ids.cpu().numpy(), draft_probs=q.cpu().numpy(),
                        cu_num_draft=(np.arange(n + 1) * K).astype(np.int32), temperature=T[::K].copy(),
                        is_greedy=np.zeros(n, np.uint8), seed=77)
    ctx = sv.SpecVerify(n, K, V, dtype, True)
    d = to_device(b)
    outs = ctx.run(d["logits"], ids, q, d["cu_num_draft"], d["temperature"], d["is_greedy"], b.seed, row_stats=True)
    names = ("sampled", "num_sampled", "num_rejected", "row_max", "row_sumexp", "row_argmax")
    got = {name: o.cpu().numpy() for name, o in zip(names, outs)}
    got["error_word"] = ctx.last_error()
    ctx.close()
    assert_parity(b, got, oracle.run(b))
    assert (got["num_sampled"] > 1).any()
    res = sv.logprobs(on_gpu(target, dtype), outs[0], num_top=5, cu_num_draft=d["cu_num_draft"])
    check_logprobs(target, [r.cpu().numpy() for r in res], got["sampled"].reshape(-1), 5)


def test_captured_replayed_and_overlapping_calls():
    """Two graphs of the operators, replayed on two streams at once with changed inputs, beside
    calls on a third: there is no memory that calls share."""
    import torch

    import speculative_decoding_verification_rejection_gb300 as sv

    V, R = 30011, 40
    streams = [torch.cuda.Stream() for _ in range(3)]
    sets = []
    for i in range(2):
        l = on_gpu(rows_of(30 + i, R, V, "bf16"), "bf16")
        u = torch.rand(R, device="cuda")
        k = torch.full((R,), 40 + i, dtype=torch.int32, device="cuda")
        p = torch.full((R,), 0.9, device="cuda")
        out = [torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R, device="cuda"),
               torch.empty(R, V, device="cuda")]
        lo = [torch.empty(R, device="cuda"), torch.empty(R, dtype=torch.int32, device="cuda"),
              torch.empty(R, 5, dtype=torch.int32, device="cuda"), torch.empty(R, 5, device="cuda")]
        g = torch.cuda.CUDAGraph()
        sv.sample(l, u, top_k=k, top_p=p, logprob=True, probs=True, out=out)
        sv.logprobs(l, out[0], num_top=5, out=lo)
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            sv.sample(l, u, top_k=k, top_p=p, logprob=True, probs=True, out=out)
            sv.logprobs(l, out[0], num_top=5, out=lo)
        sets.append((l, u, k, p, out, lo, g))
    for i, s in enumerate(sets):
        s[0].copy_(on_gpu(rows_of(40 + i, R, V, "bf16"), "bf16"))
    l3, u3 = on_gpu(rows_of(50, R, V, "f32"), "f32"), torch.rand(R, device="cuda")
    torch.cuda.synchronize()
    for _ in range(5):
        for s, stream in zip(sets, streams):
            with torch.cuda.stream(stream):
                s[6].replay()
        third = sv.sample(l3, u3, logprob=True, probs=True, stream=streams[2])
    torch.cuda.synchronize()
    for i, (l, u, k, p, out, lo, _) in enumerate(sets):
        rows = rows_of(40 + i, R, V, "bf16")
        check_sample(rows, [o.cpu().numpy() for o in out], k=k.cpu().numpy(), P=p.cpu().numpy(), u=u.cpu().numpy())
        check_logprobs(rows, [o.cpu().numpy() for o in lo], out[0].cpu().numpy(), 5)
    check_sample(rows_of(50, R, V, "f32"), [o.cpu().numpy() for o in third], u=u3.cpu().numpy())


def test_wrong_arguments_on_the_device_are_refused():
    import torch

    import speculative_decoding_verification_rejection_gb300 as sv

    l, u = torch.zeros(4, 16, device="cuda"), torch.zeros(4, device="cuda")
    with pytest.raises(ValueError):
        sv.sample(l.t(), torch.zeros(16, device="cuda"))
    with pytest.raises(ValueError):
        sv.sample(l, u.cpu())
    with pytest.raises(ValueError):
        sv.sample(l.half(), u)
    with pytest.raises(ValueError):
        sv.logprobs(l, torch.zeros(4, dtype=torch.int64, device="cuda"))
    assert sv.sample(l[:0], u[:0])[0].shape == (0,)
    assert sv.logprobs(l[:0], torch.zeros(0, dtype=torch.int32, device="cuda"))[0].shape == (0,)


def test_new_outputs_belong_to_the_stream_that_writes_them():
    """Of a call on another stream than the current one the allocator knows the writer: their
    memory is reused in that stream's order."""
    import torch

    import speculative_decoding_verification_rejection_gb300 as sv

    gen = torch.Generator().manual_seed(5)
    logits = torch.randn(3, 5000, generator=gen).cuda()
    u = torch.rand(3, generator=gen).cuda()
    here = sv.sample(logits, u, logprob=True, probs=True)
    best = sv.logprobs(logits, here[0], num_top=3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        there = sv.sample(logits, u, logprob=True, probs=True, stream=stream)
        there += sv.logprobs(logits, there[0], num_top=3, stream=stream)
        owner = {}
        for seg in torch.cuda.memory_snapshot():
            for t in there:
                if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
                    owner[t.data_ptr()] = seg["stream"]
        assert [owner[t.data_ptr()] for t in there] == [side.cuda_stream] * len(there)
        torch.cuda.synchronize()
        for a, b in zip(here + best, there):
            assert torch.equal(a, b)


def test_a_process_may_capture_its_first_calls():
    code = """
import torch
import speculative_decoding_verification_rejection_gb300 as sv
torch.cuda.init()
gen = torch.Generator().manual_seed(6)
logits = torch.randn(5, 3001, generator=gen).cuda()
u = torch.rand(5, generator=gen).cuda()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = sv.sample(logits, u, logprob=True)
    got += sv.logprobs(logits, got[0], num_top=2)
graph.replay()
torch.cuda.synchronize()
want = sv.sample(logits, u, logprob=True)
want += sv.logprobs(logits, want[0], num_top=2)
assert all(torch.equal(a, b) for a, b in zip(got, want))
"""
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300,
                   cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
