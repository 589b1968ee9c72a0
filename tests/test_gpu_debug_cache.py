"""The cache operators in the bounds-checked build of the library: small steps over every form match the plain
implementation with no access outside their arrays, and a planted shortfall of what is registered is
reported (the access is skipped; nothing traps). Runs in a child process, since a process loads one build
of the library."""
import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.gpu
def test_cache_operators_stay_inside_their_arrays():
    import speculative_decoding_verification_rejection_gb300 as sv

    sv.build(debug=True)
    env = dict(os.environ, SPEC_VERIFY_DEBUG_BOUNDS="1")
    env.pop("SV_DEBUG_SHRINK", None)
    r = subprocess.run([sys.executable, os.path.join(HERE, "debug_cache_check.py")], env=env,
                       capture_output=True, text=True, timeout=900)
    print(r.stdout[-3000:])
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-3000:]
    assert r.stdout.strip().splitlines()[-1] == "OK"


@pytest.mark.gpu
def test_waits_that_run_out_end_the_call():
    import speculative_decoding_verification_rejection_gb300 as sv

    sv.build(debug=True)
    env = dict(os.environ, SPEC_VERIFY_DEBUG_BOUNDS="1")
    env.pop("SV_DEBUG_PATIENCE", None)
    r = subprocess.run([sys.executable, os.path.join(HERE, "debug_cache_waits.py")], env=env,
                       capture_output=True, text=True, timeout=600)
    print(r.stdout[-3000:])
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-3000:]
    assert r.stdout.strip().splitlines()[-1] == "OK"
