"""The CUDA sources: every shared device helper has a user, and the driver's tensor-map encoder is fetched in one place."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "delta_rule_sequence_b200", "csrc")
FILES = {f: re.sub(r"//[^\n]*|/\*.*?\*/", "", open(os.path.join(CSRC, f)).read(), flags=re.S) for f in sorted(os.listdir(CSRC))}


@pytest.mark.parametrize("header", [f for f in FILES if f.endswith(".cuh")])
def test_every_device_helper_has_a_user(header):
    names = set(re.findall(r"__device__ __forceinline__[^;{(]*?\b(\w+)\(", FILES[header]))
    text = "\n".join(FILES.values())
    names.discard("operator")
    unused = [n for n in sorted(names) if len(re.findall(rf"\b{n}\b", text)) <= len(re.findall(rf"__device__ __forceinline__[^;{{(]*?\b{n}\(", text))]
    assert not unused


def test_the_tensor_map_encoder_is_fetched_once():
    assert [f for f, text in FILES.items() if '"cuTensorMapEncodeTiled"' in text] == ["tensor_map.cuh"]
