"""Counters in shared memory, by reading the source: between two block barriers a word is read or set, never both (a warp that
is late for its read would find what was set for later)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "speculative_decoding_verify_decode_gb300", "csrc")


def read_and_set(source):
    """(word, text) of every stretch between two barriers where a counter is set to 0 and its value is used as well.  A barrier
    inside a function that is called is none here: the call may stand under a condition."""
    source = re.sub(r"//[^\n]*|/\*.*?\*/", "", source, flags=re.S)
    counters = {word for chain in re.findall(r"((?:\bsh\.\w+ = )+)0;", source) for word in re.findall(r"sh\.(\w+)", chain)}
    found = []
    for part in re.split(r"__syncthreads\w*\(", source):
        for word in counters:
            sets = re.findall(rf"\bsh\.{word} = ", part)
            uses = [m for m in re.findall(rf"(.)\bsh\.{word}\b(?! =)", part) if m != "&"]       # &: an atomic's address
            if sets and uses:
                found.append((word, part))
    return counters, found


def test_counters_of_the_selection():
    with open(os.path.join(CSRC, "logprobs.cu")) as f:
        counters, found = read_and_set(f.read())
    assert counters >= {"n", "count"}
    assert not found, found


@pytest.mark.parametrize("text,bad", [
    ("__syncthreads(); int a = sh.n; if (t == 0) sh.n = 0; __syncthreads();", True),
    ("__syncthreads(); int a = sh.n; if (a > 3) { cut(sh); } if (t == 0) sh.n = 0; __syncthreads();", True),
    ("if (t == 0) sh.n = 0; if (sh.n > 3) f(); __syncthreads();", True),
    ("if (t == 0) sh.n = sh.m = 0; __syncthreads(); atomicAdd(&sh.n, 1); __syncthreads(); int a = sh.n; atomicAdd(&sh.m, a);", False),
    ("if (t == 0) sh.n = 0; __syncthreads(); atomicAdd(&sh.n, 1); __syncthreads_or(1); if (sh.n >= 4) f();", False),
])
def test_the_reading_itself(text, bad):
    assert bool(read_and_set(text)[1]) == bad
