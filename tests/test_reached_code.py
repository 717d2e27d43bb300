"""Template arguments of the attention's plan and operands: one form of each, that a kernel uses."""
import os
import re

from draft_sampling_verification_w1_amd import build


def read(name):
    with open(os.path.join(build.CSRC, name)) as f:
        return f.read()


def test_plan_has_one_form():
    """make_plan serves attend.hip alone, whose workgroups have a thread for each run of slots."""
    assert not re.search(r"template[^;{]*\n__device__ __forceinline__ void make_plan\(", read("attend_common.h"))
    assert "make_plan(a, kRows, plan)" in read("attend.hip")


def test_shared_helpers_are_defined_once():
    for name in ("scale_of", "max16"):
        at = [f for f in sorted(os.listdir(build.CSRC))
              if re.search(rf"__forceinline__ \w+ {name}\(", read(f))]
        assert at == ["device_common.h"], (name, at)
