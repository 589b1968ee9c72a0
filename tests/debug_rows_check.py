"""Run by tests/test_gpu_debug_rows.py in a child process whose library is the bounds-checked build
(SPEC_VERIFY_DEBUG_BOUNDS=1): every global load of a row operator is checked against the rows of
its call's inputs and every store against those of its outputs, what lies between the rows of a
strided array being outside. Small cases over every form, launch shape and start of a row; each must
match the plain implementation and leave no mark. A positive control then leaves the last bytes of
every row of logits out of what is registered (the memory is there) and the mark must appear. Prints
OK at the end."""
import ctypes
import os
import sys

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, HERE)
sys.path.insert(0, os.path.dirname(HERE))

from _rows import check_logprobs, check_sample, rows_of  # noqa: E402


def outside() -> int:
    import torch

    torch.cuda.synchronize()
    word = ctypes.c_uint32()
    assert sv.lib().spec_verify_rows_outside(ctypes.byref(word)) == sv.SV_OK
    return word.value


def dev(a, dtype):
    import torch

    return None if a is None else torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype))).cuda()


def placed(l, dtype, stride, start):
    """The rows on the GPU, `stride` elements apart, the first `start` elements into its storage."""
    import torch

    R, V = l.shape
    flat = torch.zeros(start + (R - 1) * stride + V, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")
    rows = torch.as_strided(flat, (R, V), (stride, 1), start)
    rows.copy_(torch.from_numpy(l).cuda())
    return rows


def sample(l, dtype, stride, start, probs_stride, label, **kw):
    import torch

    R, V = l.shape
    out = [torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R, device="cuda")]
    if probs_stride:
        out.append(torch.empty(R, probs_stride, device="cuda")[:, :V])
    got = sv.sample(placed(l, dtype, stride, start), dev(kw["u"], np.float32), dev(kw.get("T"), np.float32),
                    top_k=dev(kw.get("k"), np.int32), top_p=dev(kw.get("P"), np.float32),
                    min_p=dev(kw.get("M"), np.float32), logprob=True, probs=bool(probs_stride), out=out)
    assert not outside(), f"{label}: an access outside the call's arrays"
    some = np.arange(0, R, max(R // 24, 1))                  # (the rows that are compared)
    pick = {a: np.asarray(v)[some] for a, v in kw.items()}
    check_sample(l[some], [g.cpu().numpy()[some] for g in got] + ([] if probs_stride else [None]), **pick)


def logprobs(l, dtype, stride, start, tokens, n, label, sampled=None, cu=None):
    got = sv.logprobs(placed(l, dtype, stride, start), dev(tokens if sampled is None else sampled, np.int32), num_top=n,
                      cu_num_draft=dev(cu, np.int32))
    assert not outside(), f"{label}: an access outside the call's arrays"
    some = np.arange(0, l.shape[0], max(l.shape[0] // 24, 1))
    check_logprobs(l[some], [g.cpu().numpy()[some] for g in got], None if tokens is None else np.asarray(tokens)[some], n)


def shapes():
    """Rows (clusters of 8, 4, 2 and 1 CTAs of 512 threads, and blocks of 256), sizes, strides, starts."""
    for dtype in ("bf16", "f32"):
        for R, V, stride, start in ((1, 30011, 30011, 0), (2, 7, 7, 1), (3, 40003, 40009, 3), (30, 20011, 20011, 5),
                                    (70, 9001, 9016, 0), (160, 5003, 5004, 1), (320, 2503, 2503, 2), (640, 1501, 1503, 7),
                                    (620, 1, 2, 1)):
            yield dtype, R, V, stride, start


if __name__ == "__main__":
    import torch

    import speculative_decoding_verification_rejection_gb300 as sv

    assert sv.DEBUG_BOUNDS and sv.LIB_PATH.endswith("libspecverify_debug.so")
    assert torch.cuda.is_available()
    sv.lib()
    for dtype, R, V, stride, start in shapes():
        rng = np.random.default_rng(V)
        l, u = rows_of(V, R, V, dtype), rng.random(R)
        flat = rows_of(V + 1, R, V, dtype, sigma=0.5, n_peak=0)
        T = rng.uniform(0.5, 1.5, R)
        label = f"{R} x {V} {dtype}"
        for rows, kw in ((l, {}), (l, {"T": 0 * T}), (l, {"k": rng.choice([1, 5, 50, 300, V], R), "T": T}),
                         (l, {"P": rng.choice([0.5, 0.9, 0.99], R)}), (l, {"M": rng.choice([0.01, 0.3], R)}),
                         (flat, {"P": rng.choice([0.9, 0.999], R)}), (flat, {"k": rng.choice([700, V - 1], R), "P": np.full(R, 0.9)}),
                         (flat, {"M": np.full(R, 0.2)}),
                         (l, {"k": rng.choice([0, 30, 600], R), "P": rng.choice([0.8, 1.0], R), "M": rng.choice([0, 0.05], R), "T": T})):
            sample(rows, dtype, stride, start, 0, label, u=u, **kw)
            sample(rows, dtype, stride, start, V + V % 3, label, u=u, **kw)
        tokens = rng.integers(0, V, R)
        tokens[::5] = -1
        for n in (0, 5, 64):
            logprobs(l, dtype, stride, start, tokens, n, label)
        logprobs(l, dtype, stride, start, None, 3, label)
        tied = np.round(flat)                                # more ties than a list holds
        logprobs(tied, dtype, stride, start, tokens, 3, label)
        print(f"{label}: clean", flush=True)
    K = np.array([3, 0, 5, 1, 0, 0, 4, 2])
    cu = np.concatenate([[0], np.cumsum(K)])
    R, V = int(cu[-1]) + K.size, 5003
    sampled, want = np.full((K.size, 6), -1), np.full(R, -1)
    for i, k in enumerate(K):
        sampled[i, : k + 1] = want[cu[i] + i: cu[i] + i + k + 1] = np.arange(k + 1) * 7 + i
    logprobs(rows_of(10, R, V, "bf16"), "bf16", V, 0, want, 4, "uneven drafts", sampled=sampled, cu=cu)
    for bad in ([0] * 9, [-2**31] * 9, [2**31 - 1] * 9, [0, 9, -5, 2**31 - 1, 3, -2**31, 7, 7, 8]):
        sv.logprobs(placed(rows_of(10, R, V, "bf16"), "bf16", V, 0), dev(sampled, np.int32), num_top=4, cu_num_draft=dev(bad, np.int32))
        assert not outside(), f"prefix sums {bad}: an access outside the call's arrays"
    print("uneven drafts: clean", flush=True)
    os.environ["SV_DEBUG_SHRINK"] = "2"
    rows, u = placed(rows_of(12, 3, 1001, "bf16"), "bf16", 1001, 0), dev([0.1, 0.5, 0.9], np.float32)
    sv.sample(rows, u)
    assert outside() & sv.SV_ERR_BOUNDS, "the check did not fire on sample"
    sv.logprobs(rows, None, num_top=2)
    assert outside() & sv.SV_ERR_BOUNDS, "the check did not fire on logprobs"
    del os.environ["SV_DEBUG_SHRINK"]
    sv.sample(rows, u)
    assert not outside()
    print("positive control: fired", flush=True)
    print("OK", flush=True)
