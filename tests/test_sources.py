"""The CUDA sources: the driver's tensor-map encoder is fetched in one place."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "delta_rule_sequence_b200", "csrc")
FILES = {f: re.sub(r"//[^\n]*|/\*.*?\*/", "", open(os.path.join(CSRC, f)).read(), flags=re.S) for f in sorted(os.listdir(CSRC))}


def test_the_tensor_map_encoder_is_fetched_once():
    assert [f for f, text in FILES.items() if '"cuTensorMapEncodeTiled"' in text] == ["tensor_map.cuh"]
