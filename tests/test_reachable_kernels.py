"""The library holds no variant of the channel norm's backward kernel that no
channel count reaches."""
import re
import shutil
import subprocess

import pytest

import convolution_video_vae_amd as cv


def reachable():
    """(lanes of a row, 16-byte vectors of a lane) of every channel count."""
    pairs = set()
    for c in range(8, 2049, 8):
        vectors, lanes = c // 8, 1
        while lanes < 64 and 3 * lanes < vectors:
            lanes *= 2
        pairs.add((lanes, -(-vectors // lanes)))
    return pairs


def test_channel_norm_backward_variants():
    if shutil.which("nm") is None:
        pytest.skip("nm not found")
    cv.lib()
    names = subprocess.run(["nm", "-C", cv.LIB_PATH], capture_output=True, text=True,
                           check=True).stdout
    built = {(int(g), int(k), dg, db) for g, k, dg, db in
             re.findall(r"ns_bwd_kernel<(\d+), (\d+), (\w+), (\w+)>", names)}
    sums = {("true", "true"), ("true", "false"), ("false", "false")}
    assert built == {(g, k, *s) for g, k in reachable() for s in sums}
