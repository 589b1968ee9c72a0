"""Run by tests/test_gpu_debug_cache.py in a child process whose library is the bounds-checked build
(SPEC_VERIFY_DEBUG_BOUNDS=1), in which SV_DEBUG_PATIENCE says how often a wait of the cache attention looks
before it is given up. From one look (nearly every CTA gives up at once) to many (none does) a call has to end, with each row
and head either as it is in a call of full patience, bit for bit, or all NaN, and an error word that says whether
waits were given up; the next call finds nothing changed.
Prints OK at the end."""
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, HERE)
sys.path.insert(0, os.path.dirname(HERE))

from _cache import Step, attention  # noqa: E402

LENGTHS, NEW = [0, 700, 63, -1, 2900, 17, 64, 300], [1, 3, 6, 2, 4, 50, 1, 8]
CASES = (
    dict(),                                                        # keys, values and queries by tensor map
    dict(hq=16, hk=1),                                             # 64 query rows, one buffer of queries
    dict(dim=256, hq=8, hk=1, dtype="f16", cache="f16", page=32),  # one slot of keys
    dict(dim=64, page=5),                                          # vector by vector
    dict(dim=256, hq=8, hk=1, page=5),
    dict(dim=128, cache="e4m3"),                                   # 8 bits by tensor map
    dict(dim=256, hq=8, hk=1, cache="e4m3"),
    dict(dim=64, hq=3, hk=1, cache="e4m3", page=5),                # 8 bits vector by vector
    dict(bad=True), dict(bad=True, cache="e4m3"),                  # values that are not finite where they are not seen
)


def with_patience(looks, s, caches):
    if looks:
        os.environ["SV_DEBUG_PATIENCE"] = str(looks)
    try:
        return attention(s, caches)
    finally:
        os.environ.pop("SV_DEBUG_PATIENCE", None)


if __name__ == "__main__":
    import torch

    import speculative_decoding_verification_rejection_gb300 as sv

    assert sv.DEBUG_BOUNDS and sv.LIB_PATH.endswith("libspecverify_debug.so")
    for case in CASES:
        kw = {**dict(hq=8, hk=2, dim=128, page=16, layout="heads"), **case}
        bad = kw.pop("bad", False)
        s = Step(len(str(case)), LENGTHS, NEW, **kw)
        if bad:   # the last new token's, seen by its own row alone, and a slot behind it
            for i in range(s.n):
                for x in (int(s.lengths[i]) + s.new[i] - 1, int(s.lengths[i]) + s.new[i]):
                    if s.slot(i, x) is not None:
                        s.v_cache[s.slot(i, x)] = float("nan")
        caches = s.device_caches()
        want = [t.view(torch.uint8) for t in with_patience(0, s, caches)]
        whole = [torch.isnan(t).all(-1) if t.dim() == 3 else torch.isnan(t) for t in with_patience(0, s, caches)]
        seen, looks = [], 1
        while looks < 1 << 20:
            got = with_patience(looks, s, caches)
            torch.cuda.synchronize()
            lost = torch.isnan(got[1])
            word = sv.spec_verify_cache_last_error()
            assert word in (0, sv.SV_ERR_WAIT)
            for t, w in zip(got, want):
                nan = torch.isnan(t).view(s.rows, s.hq, -1)
                same = (t.view(torch.uint8) == w).view(s.rows, s.hq, -1).all(-1)
                assert bool((same | nan.all(-1)).all()), f"{case}, {looks} looks: rows that are neither right nor NaN"
            again = with_patience(0, s, caches)
            assert all(torch.equal(t.view(torch.uint8), w) for t, w in zip(again, want)), f"{case}: the call after one of {looks} looks"
            assert sv.spec_verify_cache_last_error() == 0
            assert (word != 0) == bool((lost & ~whole[1]).any()), "every CTA that gives up has rows"
            seen.append(int((lost & ~whole[1]).sum()))
            looks = looks * 9 // 8 + 1
        print(f"{case}: {sorted(set(seen))} of {s.rows * s.hq} rows and heads given up", flush=True)
        assert seen[0] > 0 and seen[-1] == 0
    print("OK", flush=True)
