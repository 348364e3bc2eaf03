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


def test_what_is_said_of_infinities_without_a_range():
    """A block whose finite values are all below 2^-100 has scale 0, and holds everything as 0."""
    import math

    import oracle.kv4_oracle as kv4
    assert "as 0 where no finite value\n * of the block reaches 2^-100" in header()
    for others in (0.0, 2.0 ** -101, -math.inf, math.nan):
        codes, s = kv4.quantise([math.inf] + [others] * 31)
        assert s == 0.0 and (codes == 8).all()
    codes, s = kv4.quantise([math.inf, -math.inf] + [2.0 ** -100] * 30)
    assert s == -2.0 ** -103 and list(codes[:3]) == [0, 15, 0]
