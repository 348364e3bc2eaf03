"""The log probabilities' workspace over row counts, on the host: each call is checked against its own need."""
import pytest

from speculative_decoding_verify_decode_gb300 import build, native

FAKE = 0x10000   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return native.load()


@pytest.mark.parametrize("vocab,top", [(151936, 20), (32000, 0), (5001, 32)])
def test_fewer_rows_may_need_more(lib, vocab, top):
    def call(rows, ws_bytes):      # (of a refused call nothing is launched; FAKE has room for no alignment fault)
        return lib.sd_logprobs(rows, vocab, 0, FAKE, 0, 1.0, 0, None, None, top, FAKE << 4 if top else None, FAKE << 5 if top else None,
                               None, FAKE << 6, FAKE << 7, ws_bytes, None, None)
    need = {rows: native.sd_logprobs_workspace_size(rows, vocab, top) for rows in range(1, 400)}
    assert need[399] == 0 < need[100]                           # in one piece each; in pieces
    assert max(need.values()) > need[300]
    for rows in (1, 7, 100, 151):
        assert call(rows, need[399]) == native.SD_ERR_WORKSPACE and call(rows, need[rows] - 1) == native.SD_ERR_WORKSPACE
    largest = max(need, key=need.get)
    assert all(need[rows] <= need[largest] for rows in need) and need[largest] <= 608 * (16 + 8 * top) + 512


def test_the_header_says_so():
    import os
    with open(os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "include", "sd_logprobs.h")) as f:
        assert "fewer rows may need more" in f.read()
