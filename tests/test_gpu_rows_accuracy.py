"""Log-probabilities of rows on which a running sum of exponentials goes wrong most easily, one CTA
to a row, against binary64: logits that rise a little along the whole row, so that the sum's
reference would move again and again, and a likely token before a floor of unlikely ones, whose
small parts a large sum would take in with the same rounding each time."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0**-24
STEP = 4 * np.log(2.0)   # by how much a lane's logits pass its reference before that moves


def exact(l, tokens, T):
    """ln p of the tokens, ln sum exp(d), sum p |d|, |d| of the tokens, in binary64."""
    import torch

    out = [[] for _ in range(4)]
    for x, t, temp in zip(l.split(16), tokens.split(16), [None] * 1000 if T is None else T.split(16)):
        x = x.double()
        d = x - x.max(1, keepdim=True).values
        if temp is not None:
            d = d / temp.double()[:, None]
        e = d.exp()
        s = e.sum(1)
        at = d.gather(1, t.long()[:, None])[:, 0]
        for o, v in zip(out, (at - s.log(), s.log(), -(e * d).sum(1) / s, -at)):
            o.append(v)
    return [torch.cat(o).cpu().numpy() for o in out]


def half_ulp(x):
    return 0.5 * np.spacing(np.abs(x).astype(np.float32)).astype(np.float64)


def tolerance(lp, norm, mean, at, dtype, top, T, rise):
    """Bound of the error, u = 2^-24 a rounding to nearest.

    The sum's relative error. Arguments: a term 2^x of d = -|d| has x = (l - ref) * fl(log2 e / T):
    one rounding of the difference, one of the product, log2 e off by 0.25 u, and with a temperature
    one of 1 / T and one of its product with log2 e, each relative to the difference, so
    (2.25 or 4.25) u |d| of the term, and |d| weighed by the terms is `mean`; a logit may lie above its
    lane's reference, by at most `above` = min(rise, STEP) in d, and is then taken up and down again:
    2 `above` more. 2^x itself: 2^-22 = 4 u. A batch is added up in turn, two terms at a time: 4 (8 with
    best tokens) vectors of 2 pairs of float32 or 4 of bfloat16, and the two halves. The batches by
    compensated addition: 2 u. Where the reference moved (rises beyond STEP), each time by at least
    2^-4: what was there before is off by 5 u (2^x and a product) and has at least
    sixteenfold shrunk, beside the term of at least 1 that moved it; of a lane's at most 2064 terms of up
    to 16 the part that saw k moves is at most 1, 1, 1, 0.5, 0.04, ... of the sum for k = 1, 2, ...: below 4
    moves counted by weight, 20 u. To the warp's largest logit: 2^x and a
    product 5 u, 5 additions; to the row's: exp and product 3 u, at most 2 + 5 additions.
    Then the logarithm: half a unit of the result and 2 u for its series and parts; d of the token
    3 u |d|; the difference: half a unit of ln p."""
    above = min(rise, STEP)
    chain = (8 if top else 4) * (2 if dtype == "f32" else 4) + 1
    sum_err = (2.25 if T is None else 4.25) * (mean + 2 * above) + 4 + chain + 2 + (20 if rise > STEP else 0) + 10 + 10
    return U * (sum_err + 2 + 3 * at) * (1 + 2.0**-10) + half_ulp(norm) + half_ulp(lp)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [32000, 151936, 524288])
@pytest.mark.parametrize("kind", ["rise", "rise in eighths", "fall", "floor", "floor with a temperature"])
def test_log_probabilities_of_long_even_rows(V, dtype, kind):
    import torch

    import speculative_decoding_verification_rejection_gb300 as sv

    R = 320                                              # more than half of the CTAs the device holds: one a row
    place = torch.arange(V, device="cuda", dtype=torch.float32) / V
    T = None
    if kind.startswith("floor"):
        depth = torch.linspace(0.05, 14.0, R, device="cuda")
        l = (-depth)[:, None].expand(R, V).contiguous()
        l[:, 0] = 0.0
        rise = 0.0
        if kind != "floor":
            T = torch.rand(R, device="cuda", generator=torch.Generator("cuda").manual_seed(V)) + 0.5
    else:
        size = torch.logspace(-2, 2.5, R, device="cuda")
        l = size[:, None] * ({"rise": place, "fall": -place}.get(kind) if kind != "rise in eighths" else place * 8 % 1)
        rise = 0.0 if kind == "fall" else None
    l = l.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    tokens = l.float().argmax(1).int()
    tokens[::3] = torch.arange(R, device="cuda", dtype=torch.int32)[::3] * 97 % V
    lp, norm, mean, at = exact(l, tokens, T)
    for top in (0, 5):
        got = sv.logprobs(l, tokens, num_top=top, temperature=T)[0].cpu().numpy().astype(np.float64)
        for r in range(R):
            up = float(size[r]) if rise is None else rise
            tol = tolerance(lp[r], norm[r], mean[r], at[r], dtype, top, T, up)
            assert abs(got[r] - lp[r]) <= tol, f"row {r}: {got[r]} {lp[r]}, off by {got[r] - lp[r]:.3g}, tolerance {tol:.3g}"
