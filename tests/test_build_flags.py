"""Compiler flags that a source's contract rules out."""
import os
import re

from draft_sampling_verification_w1_amd import build


def test_sources_that_promise_nan_honour_it():
    """include/dspark.h says which rows of dspark_attend4, and which rows of log probabilities, are NaN."""
    for src in ("attend4.hip", "cache_store.hip", "logprobs.hip"):
        flags = [*build.HIPCC_FLAGS, *build.EXTRA_FLAGS.get(src, [])]
        assert not [f for f in flags if re.search(r"no-honor-nans|finite-math|fast-math|Ofast", f)], src
    assert set(build.EXTRA_FLAGS) <= set(build.SOURCES)
    assert all(os.path.exists(os.path.join(build.CSRC, s)) for s in build.SOURCES)
