"""The places of the fp32 product's rows in LDS: no two lanes that are served together use one bank twice, for the writes
(8 lanes of 16 bytes at a time over 32 banks) and the fragment reads (16 lanes over 64 banks)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "selective_state_space_17_amd", "csrc")
LINE = 128   # bytes of a row


def key_of_the_source():
    with open(os.path.join(CSRC, "fp8_product.hip")) as f:
        body = re.search(r"int fine_key\(int row\) \{ return ([^;]+); \}", f.read()).group(1)
    assert re.fullmatch(r"[row0-9/%^() ]+", body), body
    return eval("lambda row: " + body.replace("/", "//"))


def conflicts(key, together, banks, address):
    """Waves' accesses of 16 bytes: how often two of the lanes served together need the same bank."""
    n = 0
    for first in range(0, 64, together):
        used = [address(lane, key) // 16 % (banks // 4) for lane in range(first, first + together)]
        n += len(used) - len(set(used))
    return n


def write(second):
    """Lane's row lane / 4, its chunks 2 (lane % 4) and the next."""
    return lambda lane, key: lane // 4 * LINE + (((lane % 4 * 2 + second) ^ key(lane // 4)) << 4)


def read(q):
    """Fragment of 16 k: lane's row lane % 32, chunk 2 q + lane / 32."""
    return lambda lane, key: lane % 32 * LINE + (((2 * q + lane // 32) ^ key(lane % 32)) << 4)


def test_no_bank_twice():
    key = key_of_the_source()
    assert {key(r) for r in range(64)} == set(range(8)), "a chunk stays among its row's eight"
    assert all(key(r) == key(r + 32) for r in range(96)), "rows of 32 lanes, and a thread's second row, share their key"
    for second in (0, 1):
        assert conflicts(key, 8, 32, write(second)) == 0
    for q in range(4):
        assert conflicts(key, 16, 64, read(q)) == 0


def test_it_sees_conflicts():
    assert conflicts(lambda r: r // 2 % 8, 8, 32, write(0)) > 0     # rows 2 i and 2 i + 1 alike
    assert conflicts(lambda r: r % 2, 16, 64, read(0)) > 0
