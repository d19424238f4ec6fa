"""hla_timing_read's kernel kinds, host side."""
import ctypes
import os
import re

from gated_deltanet_hybrid_amd import hla

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "hla.h")


def test_every_kind_of_the_header_is_read_and_bound():
    with open(HEADER) as f:
        kinds = {n: int(v) for n, v in re.findall(r"\bHLA_KERNEL_(\w+) = (\d+)", f.read())}
    count = kinds.pop("COUNT")
    assert sorted(kinds.values()) == list(range(count))
    ms, n = ctypes.c_double(), ctypes.c_int64()
    for name, kind in kinds.items():
        assert getattr(hla, "KERNEL_" + name) == kind
        assert hla.library().hla_timing_read(kind, ctypes.byref(ms), ctypes.byref(n)) == 0 and n.value == 0
    assert hla.library().hla_timing_read(count, ctypes.byref(ms), ctypes.byref(n)) == 2

