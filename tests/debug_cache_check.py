"""Run by tests/test_gpu_debug_cache.py in a child process whose library is the bounds-checked build
(SPEC_VERIFY_DEBUG_BOUNDS=1): every global load of a cache operator is checked against its call's inputs and
workspace, every store against its outputs and workspace. Small steps over every form; each must match the
plain implementation and leave no mark. A positive control then leaves the last bytes of the cached
keys out of what is registered (the memory is there) and the mark must appear. Prints OK at the end."""
import ctypes
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, HERE)
sys.path.insert(0, os.path.dirname(HERE))

from _cache import Step, append, attention, check_append, check_attention  # noqa: E402


def outside() -> int:
    import torch

    torch.cuda.synchronize()
    word = ctypes.c_uint32()
    assert sv.lib().spec_verify_cache_outside(ctypes.byref(word)) == sv.SV_OK
    return word.value


if __name__ == "__main__":
    import torch

    import speculative_decoding_verification_rejection_gb300 as sv

    assert sv.DEBUG_BOUNDS and sv.LIB_PATH.endswith("libspecverify_debug.so")
    assert torch.cuda.is_available()
    sv.lib()
    lengths, new = [0, 1, 63, 64, 300, -1, 2000, 17], [1, 3, 6, 1, 8, 2, 4, 50]
    for dtype, cache in (("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3")):
        for dim, hq, hk, page, layout in ((64, 8, 1, 16, "heads"), (128, 12, 3, 5, "tokens"), (256, 16, 2, 64, "both"), (128, 64, 2, 1, "heads")):
            s = Step(dim, lengths, new, hq=hq, hk=hk, dim=dim, dtype=dtype, cache=cache, page=page, layout=layout)
            inv = 10000.0 ** (-torch.arange(dim // 2) / (dim // 2))
            label = f"{dtype} {cache} {dim} {hq}/{hk} page {page}"
            check_append(s, label, inv_freq=inv)
            assert not outside(), f"{label}: append: an access outside the call's arrays"
            check_append(s, label, inv_freq=inv[:16], interleaved=True, positions=torch.ones(2, s.rows, dtype=torch.int32), axes=[0, 1] * 8)
            assert not outside(), f"{label}: append with positions: an access outside the call's arrays"
            for window in (0, 20):
                check_attention(s, label, window=window)
                assert not outside(), f"{label}: attention: an access outside the call's arrays"
            print(f"{label}: clean", flush=True)
    s = Step(1, [100, 5], [3, 2], dim=64)
    s.table[0, 1:3] = torch.tensor([s.pool, -1])
    append(s)
    attention(s)
    for cu in ([0, 1, 0], [0, -3, 2], [0, 2, 2**31 - 1], [-2**31, 0, 1], [0, 100, 100]):
        s.cu = torch.tensor(cu, dtype=torch.int32)
        append(s)
        attention(s)
    assert not outside(), "bad pages and prefix sums: an access outside the call's arrays"
    s = Step(2, [100, 200], [3, 2], dim=64)
    s.table[1, 200 // s.page] = s.pool - 1   # the last page holds places that are written and read
    os.environ["SV_DEBUG_SHRINK"] = str(16 * 64 * 2 * 2)
    append(s)
    assert outside() & sv.SV_ERR_BOUNDS, "the check did not fire on append"
    attention(s)
    assert outside() & sv.SV_ERR_BOUNDS, "the check did not fire on attention"
    del os.environ["SV_DEBUG_SHRINK"]
    attention(s)
    assert not outside()
    print("positive control: fired", flush=True)
    print("OK", flush=True)
