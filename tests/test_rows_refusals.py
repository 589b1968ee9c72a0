"""Refusals of the row operators: host-visible mistakes give a status and need no device."""
import ctypes

import pytest

import speculative_decoding_verification_rejection_gb300 as sv

P = 0x10000  # an aligned address; nothing is read from it


def sample_args(**kw):
    base = dict(logits=P, logits_stride=1000, uniforms=P, tokens=P, num_rows=4, vocab_size=1000,
                logits_dtype=sv.SV_F32, device=0)
    return sv.SampleArgs(**{**base, **kw})


def logprob_args(**kw):
    base = dict(logits=P, logits_stride=1000, tokens=P, token_logprob=P, token_rank=P, num_rows=4,
                vocab_size=1000, logits_dtype=sv.SV_BF16, device=0)
    return sv.LogprobsArgs(**{**base, **kw})


ROWS = [
    (dict(logits=None), sv.SV_EINVAL), (dict(logits=P + 1), sv.SV_EINVAL),
    (dict(logits_stride=999), sv.SV_EINVAL), (dict(num_rows=-1), sv.SV_EINVAL),
    (dict(vocab_size=0), sv.SV_EINVAL), (dict(vocab_size=-5), sv.SV_EINVAL),
    (dict(vocab_size=sv.SV_ROWS_MAX_VOCAB + 1, logits_stride=1 << 21), sv.SV_ECAPACITY),
    (dict(logits_dtype=7), sv.SV_EDTYPE), (dict(temperature=P + 2), sv.SV_EINVAL),
    (dict(device=-1), sv.SV_EDEVICE), (dict(device=1000), sv.SV_EDEVICE),
]


@pytest.mark.parametrize("change,status", ROWS + [
    (dict(uniforms=None), sv.SV_EINVAL), (dict(tokens=None), sv.SV_EINVAL),
    (dict(probs=P, probs_stride=999), sv.SV_EINVAL), (dict(probs=P + 2, probs_stride=1000), sv.SV_EINVAL),
    (dict(top_p=P + 1), sv.SV_EINVAL), (dict(token_logprob=P + 3), sv.SV_EINVAL),
])
def test_sample_refuses(change, status):
    assert sv.lib().spec_verify_sample(ctypes.byref(sample_args(**change)), None) == status


# 4 rows of 1000 float32 logits 1000 apart: 16000 bytes; no device has this ordinal, so a call that
# is not refused for its memory ends there
@pytest.mark.parametrize("at,stride,status", [
    (P, 1000, sv.SV_EINVAL), (P + 16000 - 4, 1000, sv.SV_EINVAL), (P + 16000, 1000, sv.SV_EDEVICE),
    (P - 16000 + 4, 1000, sv.SV_EINVAL), (P - 16000, 1000, sv.SV_EDEVICE),
    (P - 16000, 1001, sv.SV_EINVAL), (4, (1 << 62) - 1, sv.SV_EINVAL), (P + 16000, (1 << 62) - 1, sv.SV_EDEVICE),
])
def test_distributions_over_the_logits_are_refused(at, stride, status):
    args = sample_args(probs=at, probs_stride=stride, device=1000)
    assert sv.lib().spec_verify_sample(ctypes.byref(args), None) == status


@pytest.mark.parametrize("change,status", ROWS + [
    (dict(num_top=-1), sv.SV_EINVAL), (dict(num_top=3), sv.SV_EINVAL),
    (dict(num_top=3, top_ids=P), sv.SV_EINVAL),
    (dict(num_top=sv.SV_MAX_TOP + 1, top_ids=P, top_logprobs=P), sv.SV_ECAPACITY),
    (dict(tokens=None), sv.SV_EINVAL),
    (dict(tokens=None, token_logprob=None, token_rank=None), sv.SV_EINVAL),
    (dict(cu_num_draft=P), sv.SV_EINVAL), (dict(cu_num_draft=P, num_reqs=2), sv.SV_EINVAL),
    (dict(cu_num_draft=P, token_stride=2), sv.SV_EINVAL), (dict(token_rank=P + 2), sv.SV_EINVAL),
])
def test_logprobs_refuses(change, status):
    assert sv.lib().spec_verify_logprobs(ctypes.byref(logprob_args(**change)), None) == status


def test_null_arguments_and_no_rows():
    assert sv.lib().spec_verify_sample(None, None) == sv.SV_EINVAL
    assert sv.lib().spec_verify_logprobs(None, None) == sv.SV_EINVAL
    assert sv.lib().spec_verify_sample(ctypes.byref(sample_args(num_rows=0, logits=None)), None) == sv.SV_OK
    assert sv.lib().spec_verify_logprobs(ctypes.byref(logprob_args(num_rows=0, logits=None)), None) == sv.SV_OK


def test_constants_match_the_header():
    import re

    with open(sv._HEADER, encoding="utf-8") as f:
        text = f.read()
    for name in ("SV_ROWS_MAX_VOCAB", "SV_MAX_TOP"):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == getattr(sv, name)


def test_python_refuses_tensors_that_are_not_on_a_device():
    import torch

    with pytest.raises(ValueError, match="CUDA device"):
        sv.sample(torch.zeros(2, 8), torch.zeros(2))
    with pytest.raises(ValueError, match="CUDA device"):
        sv.logprobs(torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="vocab_size"):
        sv.sample(torch.zeros(8), torch.zeros(1))


class FakeTensor:
    """What the argument checks look at, of a tensor said to be on a device."""

    def __init__(self, shape, dtype, strides=None, device="cuda:0"):
        import torch

        self.shape, self.dtype, self.device = shape, dtype, torch.device(device)
        self.strides = strides or tuple(int(__import__("math").prod(shape[i + 1:])) for i in range(len(shape)))
        self.is_cuda = self.device.type == "cuda"

    def dim(self):
        return len(self.shape)

    def numel(self):
        return int(__import__("math").prod(self.shape))

    def stride(self, i):
        return self.strides[i]

    def is_contiguous(self):
        return self.strides == tuple(int(__import__("math").prod(self.shape[i + 1:])) for i in range(len(self.shape)))

    def data_ptr(self):
        return P


def test_python_refuses_wrong_tensors(monkeypatch):
    import torch

    f32, i32 = torch.float32, torch.int32
    called = []
    monkeypatch.setattr(sv, "spec_verify_sample", lambda *a: called.append(a))
    monkeypatch.setattr(sv, "spec_verify_logprobs", lambda *a: called.append(a))
    monkeypatch.setattr(sv, "_current_stream", lambda index: 0)
    T = FakeTensor
    l, u, out = T((4, 10), f32), T((4,), f32), [T((4,), i32)]
    sv.sample(l, u, out=out)                                           # the good call
    sv.sample(T((4, 10), torch.bfloat16, (64, 1)), u, out=out)          # rows further apart
    assert len(called) == 2
    bad = [
        (T((4, 10), f32, (1, 4)), u, {}),                              # columns first
        (T((4, 10), f32, (9, 1)), u, {}),                              # rows that overlap
        (T((4, 10), torch.float16), u, {}), (T((4, 10), torch.float64), u, {}),
        (l, T((3,), f32), {}), (l, T((4,), torch.float64), {}), (l, T((4, 1), f32), {}),
        (l, T((4,), f32, (2,)), {}), (l, T((4,), f32, device="cpu"), {}),
        (l, T((4,), f32, device="cuda:1"), {}),
        (l, u, dict(temperature=T((5,), f32))), (l, u, dict(top_k=T((4,), f32))),
        (l, u, dict(top_p=T((4,), i32))), (l, u, dict(min_p=T((4,), f32, device="cpu"))),
        (l, u, dict(out=[T((4,), torch.int64)])), (l, u, dict(out=[T((4,), i32), T((4,), f32)])),
        (l, u, dict(probs=True, out=[T((4,), i32), T((4, 9), f32)])),
        (l, u, dict(probs=True, out=[T((4,), i32), T((4, 10), f32, (5, 1))])),
    ]
    for logits, uniforms, kw in bad:
        with pytest.raises(ValueError):
            sv.sample(logits, uniforms, **{"out": out, **kw})
    lp = [T((4,), f32), T((4,), i32)]
    sv.logprobs(l, T((4,), i32), out=lp)
    sv.logprobs(l, T((2, 2), i32), cu_num_draft=T((3,), i32), out=lp)
    assert len(called) == 4
    for tokens, kw in [
        (T((4,), torch.int64), {}), (T((2, 2), i32), {}), (None, {}),
        (T((4,), i32), dict(num_top=-1)), (T((4,), i32), dict(num_top=sv.SV_MAX_TOP + 1)),
        (T((4,), i32), dict(cu_num_draft=T((3,), i32))),
        (T((3, 2), i32), dict(cu_num_draft=T((3,), i32))),
        (T((2, 2), i32), dict(cu_num_draft=T((3,), torch.int64))),
        (T((4,), i32), dict(num_top=2)),                                # out lacks the best tokens
    ]:
        with pytest.raises(ValueError):
            sv.logprobs(l, tokens, **{"out": lp, **kw})
    assert len(called) == 4
