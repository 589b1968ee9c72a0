"""Rows of logits between guards that any read past a row would show: what lies before the first row,
between rows and behind the last is +inf, or a large finite number, which would take over the row's
maximum, its sum, its ranks and its best tokens (a NaN would be left out like any other)."""
import numpy as np
import pytest

from _rows import check_logprobs, check_sample, rows_of

pytestmark = pytest.mark.gpu

# rows that get 8, 4, 2 and 1 CTAs of the kernels' blocks, and smaller blocks; sizes that end anywhere in a vector
SHAPES = [(3, 40003), (30, 9001), (70, 9010), (130, 5007), (320, 2502), (640, 1505), (5, 33), (2, 1)]


def between_guards(l, dtype, gap, start, guard):
    import torch

    R, V = l.shape
    stride = V + gap
    flat = torch.full((start + R * stride + 64,), guard, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")
    rows = torch.as_strided(flat, (R, V), (stride, 1), start)
    rows.copy_(torch.from_numpy(l).cuda())
    return rows


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,V", SHAPES)
def test_nothing_past_a_row_is_read(R, V, dtype):
    import torch

    import speculative_decoding_verification_rejection_gb300 as sv

    dev = lambda a, t: torch.from_numpy(np.asarray(a, t)).cuda()  # noqa: E731
    rng = np.random.default_rng(V)
    l, flat = rows_of(V, R, V, dtype), rows_of(V + 1, R, V, dtype, sigma=0.5, n_peak=0)
    u = rng.random(R).astype(np.float32)
    tokens = rng.integers(0, V, R).astype(np.int32)
    some = np.arange(0, R, max(R // 16, 1))                  # (the rows that are compared)
    for gap, start, guard in ((1, 1, np.inf), (2, 3, 3e38), (3, 8, np.inf), (5, 6, np.inf), (7, 7, 3e38), (8, 5, np.inf)):
        for rows, kw in ((l, {}), (l, {"k": np.full(R, 20)}), (l, {"P": np.full(R, 0.9)}), (flat, {"P": np.full(R, 0.95)}),
                         (flat, {"k": np.full(R, 700)}), (flat, {"M": np.full(R, 0.3)}), (l, {"T": np.zeros(R)})):
            T, k, P, M = (None if kw.get(a) is None else dev(kw[a], t) for a, t in zip("TkPM", (np.float32, np.int32, np.float32, np.float32)))
            got = sv.sample(between_guards(rows, dtype, gap, start, guard), dev(u, np.float32), T, top_k=k, top_p=P, min_p=M,
                            logprob=True, probs=True)
            check_sample(rows[some], [g.cpu().numpy()[some] for g in got], u=u[some], **{a: v[some] for a, v in kw.items()})
        for n in (0, 4):
            got = sv.logprobs(between_guards(l, dtype, gap, start, guard), dev(tokens, np.int32), num_top=n)
            check_logprobs(l[some], [g.cpu().numpy()[some] for g in got], tokens[some], n)
