"""Limits that the decode-step header states are the kernels' own. CPU only."""

import os
import re

import linear_attention_state_chunked_gb300 as L

PKG = os.path.dirname(L.__file__)


def test_the_longest_request():
    with open(os.path.join(PKG, "..", "include", "lin_step.h")) as f:
        stated = re.search(r"Longest request: 2\^31 - (\d+) tokens", f.read())
    with open(os.path.join(PKG, "csrc", "attn_common.cuh")) as f:
        made = re.search(r"kLongest = \(int64_t\(1\) << 31\) - (\d+);", f.read())
    assert made and stated.group(1) == made.group(1)
