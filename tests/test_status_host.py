"""The device status words, without a GPU."""
import glob
import os
import re

from nvfp4_weight_only_gemv_gb300 import build


def test_two_words_hold_every_kernels_bits():
    # nvfp4_device_status waits for a copy of each
    text = "".join(open(f).read() for f in sorted(glob.glob(os.path.join(build.PKG_DIR, "csrc", "*.cu*"))))
    assert sorted(re.findall(r"__device__\s+\w+\s+(g_\w*status)", text)) == ["g_device_status", "g_plain_status"]
