"""The row operators at the ends of what they take: the largest vocabulary by one CTA a row, and the
smallest temperatures."""
import numpy as np
import pytest

from _rows import check_logprobs, check_sample, rows_of

pytestmark = pytest.mark.gpu


def dev(a, dtype):
    import torch

    return None if a is None else torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype))).cuda()


def sample(l, u, **kw):
    import speculative_decoding_verification_rejection_gb300 as sv

    got = sv.sample(dev(l, np.float32), dev(u, np.float32), dev(kw.get("T"), np.float32), top_k=dev(kw.get("k"), np.int32),
                    top_p=dev(kw.get("P"), np.float32), min_p=dev(kw.get("M"), np.float32), logprob=True, probs=True)
    return [g.cpu().numpy() for g in got]


@pytest.mark.parametrize("R", [3, 320, 640])
@pytest.mark.parametrize("kw", [{}, {"P": 0.2}, {"P": 0.6}, {"P": 0.95}, {"k": 300, "P": 0.5}, {"M": 0.3}])
def test_sample_at_subnormal_temperatures(R, kw):
    """1 / T near the largest float32, logits that differ by subnormal numbers: d is an ordinary number."""
    V = 1003
    rng = np.random.default_rng(R)
    T = rng.choice(np.array([2.95e-39, 3.0e-39, 3.6e-39, 4.2e-39, 4.3e-39, 1.2e-38], np.float32), R)
    l = np.stack([-rng.permutation(V) * np.float32(10.0 ** rng.uniform(-41.5, -40)) for _ in range(R)]).astype(np.float32)
    u = rng.random(R).astype(np.float32)
    kw = {"T": T, **{a: np.full(R, v) for a, v in kw.items()}}
    got = sample(l, u, **kw)
    some = np.arange(0, R, max(R // 32, 1))
    check_sample(l[some], [g[some] for g in got], u=u[some], **{a: v[some] for a, v in kw.items()})


@pytest.mark.parametrize("R", [3, 320])
def test_log_probabilities_at_subnormal_temperatures(R):
    """A subnormal temperature counts as the smallest normal number."""
    import speculative_decoding_verification_rejection_gb300 as sv

    V = 1003
    rng = np.random.default_rng(R)
    T = rng.choice(np.array([1e-45, 2.95e-39, 4.2e-39, 1.17e-38, 1.2e-38, 3e-38], np.float32), R)
    l = np.stack([-rng.permutation(V) * np.float32(10.0 ** rng.uniform(-41.5, -40)) for _ in range(R)]).astype(np.float32)
    tokens = rng.integers(0, V, R).astype(np.int32)
    for n in (0, 4):
        got = sv.logprobs(dev(l, np.float32), dev(tokens, np.int32), num_top=n, temperature=dev(T, np.float32))
        check_logprobs(l, [g.cpu().numpy() for g in got], tokens, n, np.maximum(T, np.finfo(np.float32).tiny))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_largest_vocabulary_by_one_cta_a_row(dtype):
    """More rows than four blocks on every SM: each lane adds up as many weights as it ever does, and on
    rows that rise along the way as many times goes from one largest logit to another."""
    import torch

    import speculative_decoding_verification_rejection_gb300 as sv

    V, R = sv.SV_ROWS_MAX_VOCAB, 612
    rng = np.random.default_rng(8)
    at = np.arange(V) / V
    kinds = np.stack([np.zeros(V), 30 * at, 0.4 * at, 0.5 * rng.standard_normal(V), np.where(at == 0, 9.0, 0.0),
                      np.round(2 * rng.standard_normal(V))]).astype(np.float32)
    kind = torch.from_numpy(kinds).cuda().to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    settings = [dict(), dict(P=0.9), dict(P=0.5), dict(P=0.9999), dict(k=5000, P=0.9), dict(M=0.5)]
    row = np.arange(R)
    P = np.array([s.get("P", 1.0) for s in settings], np.float32)[row // 6 % 6]
    k = np.array([s.get("k", 0) for s in settings], np.int32)[row // 6 % 6]
    M = np.array([s.get("M", 0.0) for s in settings], np.float32)[row // 6 % 6]
    u = rng.random(R).astype(np.float32)
    logits = kind[torch.arange(R, device="cuda") % 6]
    got = sv.sample(logits, dev(u, np.float32), top_k=dev(k, np.int32), top_p=dev(P, np.float32), min_p=dev(M, np.float32), logprob=True)
    tok, lp = (g.cpu().numpy() for g in got)
    some = np.r_[0:36, 576:582, 611]
    check_sample(kind.float().cpu().numpy()[some % 6], [tok[some], lp[some], None], u=u[some], k=k[some], P=P[some], M=M[some])
