"""Draft steps that write their distributions where the verification reads them: row j of every request
of q [requests, K, vocab], and the tokens of step j; nothing else of either is touched."""
import numpy as np
import pytest

from _rows import check_sample, rows_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,K,V", [(1, 3, 4001), (12, 3, 1002), (330, 2, 515)])
def test_draft_steps_in_place(n, K, V, dtype):
    import torch

    import speculative_decoding_verification_rejection_gb300 as sv

    l = rows_of(n + V, n * K, V, dtype)
    draft = torch.from_numpy(l).cuda().to(torch.bfloat16 if dtype == "bf16" else torch.float32).view(n, K, V)
    rng = np.random.default_rng(V)
    u = rng.random((K, n)).astype(np.float32)
    P = torch.full((n,), 0.95, device="cuda")
    q = torch.full((n, K, V), -7.0, device="cuda")
    tokens = torch.full((K, n), -9, dtype=torch.int32, device="cuda")
    for j in range(K):
        sv.sample(draft[:, j], torch.from_numpy(u[j]).cuda(), top_p=P, probs=True, out=(tokens[j], q[:, j]))
        assert bool((q[:, j + 1:] == -7.0).all()) and bool((tokens[j + 1:] == -9).all())
        check_sample(l.reshape(n, K, V)[:, j], (tokens[j].cpu().numpy(), None, q[:, j].cpu().numpy()), P=np.full(n, 0.95), u=u[j])
    again = torch.empty(n * K, V, device="cuda")                 # all rows at once
    ids = torch.empty(n * K, dtype=torch.int32, device="cuda")
    sv.sample(draft.view(n * K, V), torch.from_numpy(np.ascontiguousarray(u.T).reshape(-1)).cuda(), top_p=P.repeat_interleave(K),
              probs=True, out=(ids, again))
    assert torch.equal(again, q.view(n * K, V)) and torch.equal(ids.view(n, K), tokens.T)
