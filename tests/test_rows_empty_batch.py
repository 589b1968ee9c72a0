"""A verification of no requests is a batch like any other: its (empty) output goes to the
log-probabilities, which have nothing to do."""
import pytest

import speculative_decoding_verification_rejection_gb300 as sv
from test_rows_refusals import FakeTensor as T


def test_log_probabilities_of_an_empty_verification(monkeypatch):
    import torch

    f32, i32 = torch.float32, torch.int32
    called = []
    monkeypatch.setattr(sv, "spec_verify_logprobs", lambda args, stream: called.append(sv.lib().spec_verify_logprobs(args, None)))
    monkeypatch.setattr(sv, "_current_stream", lambda index: 0)
    out = [T((0,), f32), T((0,), i32), T((0, 3), i32), T((0, 3), f32)]
    sv.logprobs(T((0, 10), f32), T((0, 4), i32), num_top=3, cu_num_draft=T((1,), i32), out=out)
    assert called == [sv.SV_OK]
    lp = [T((4,), f32), T((4,), i32)]
    for logits, tokens, cu in ((T((4, 10), f32), T((0, 4), i32), T((1,), i32)),      # rows, but no requests
                               (T((0, 10), f32), T((0, 4), i32), T((0,), i32)),      # no prefix sums
                               (T((0, 10), f32), T((1, 4), i32), T((1,), i32))):     # outputs of another batch
        with pytest.raises(ValueError):
            sv.logprobs(logits, tokens, cu_num_draft=cu, out=lp if logits.shape[0] else out[:2])
    assert len(called) == 1


@pytest.mark.gpu
def test_log_probabilities_of_an_empty_verification_on_the_device():
    import torch

    ctx = sv.SpecVerify(4, 3, 1000, "bf16", False)
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    logits, cu = z(0, 1000, t=torch.bfloat16), z(1)
    sampled, _, _ = ctx.run(logits, z(0), None, cu, z(0, t=torch.float32), z(0, t=torch.uint8), 5)
    got = sv.logprobs(logits, sampled, num_top=2, cu_num_draft=cu)
    assert [tuple(g.shape) for g in got] == [(0,), (0,), (0, 2), (0, 2)]
    ctx.close()
