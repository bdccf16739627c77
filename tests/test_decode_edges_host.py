"""What the plain-decoding and 8-bit-cache calls rest on, as far as it shows without a GPU."""

import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_tree_build_gb300", "csrc")


def test_no_launch_rule_holds_a_number_of_sms():
    """Launch rules ask the device (device_sm_count) and do not reckon with one GPU's 152 SMs."""
    for f in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, f), encoding="utf-8") as fh:
            code = re.sub(r"//[^\n]*|/\*.*?\*/", "", fh.read(), flags=re.S)
        assert not re.findall(r"\b152\s*\*|[*/]\s*\(?\s*152\b", code), f
