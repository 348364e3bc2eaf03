"""What include/sd_kv4.h states in figures, against its own constants."""
import os
import re


def header():
    with open(os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "include", "sd_kv4.h")) as f:
        return f.read()


def test_where_magnitudes_saturate():
    text = header()
    largest = float.fromhex(re.search(r"#define SD_KV4_MAX_SCALE (\S+?)f\s", text).group(1))
    assert largest == 1.3125 * 2.0 ** 123
    stated = re.search(r"magnitudes beyond 8 SD_KV4_MAX_SCALE = ([\d.e]+) saturate", text).group(1)
    assert stated == f"{8 * largest:.2e}".replace("e+", "e")
