"""The row operators in the bounds-checked build of the library: small cases over every form and launch
shape match the plain implementation with no access outside the rows of their arrays, and a planted
shortfall of what is registered is reported (the access is skipped; nothing traps). Runs in a
child process, since a process loads one build of the library."""
import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.gpu
def test_row_operators_stay_inside_their_arrays():
    import speculative_decoding_verification_rejection_gb300 as sv

    sv.build(debug=True)
    env = dict(os.environ, SPEC_VERIFY_DEBUG_BOUNDS="1")
    env.pop("SV_DEBUG_SHRINK", None)
    r = subprocess.run([sys.executable, os.path.join(HERE, "debug_rows_check.py")], env=env,
                       capture_output=True, text=True, timeout=900)
    print(r.stdout[-3000:])
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-3000:]
    assert r.stdout.strip().splitlines()[-1] == "OK"


def test_every_global_access_is_a_checked_one():
    """In the kernels' source: no load or store of a call's arrays but through the checked forms."""
    import re

    import speculative_decoding_verification_rejection_gb300 as sv

    with open(os.path.join(os.path.dirname(sv._UNITS[0]), "sv_rows_block.cuh"), encoding="utf-8") as f:
        code = re.sub(r"//.*", "", f.read())
    arrays = r"(?:row|vec|probs|logits|P\.[a-z_]+)\b"
    for plain in (r"__ldg|__stcs|[a-z]+\.global", rf"(?<![\w.&]){arrays}\s*\[", rf"(?:[=(,{{;]|return)\s*\*\s*\(?{arrays}",
                  r"(?:[=(,{;]|return)\s*\*\s*reinterpret_cast"):
        assert not (found := re.findall(plain, code)), found
