"""The bits of the device error word: one list for all kernels, each bit once."""
import re
from pathlib import Path

CSRC = Path(__file__).resolve().parent.parent / "pagedattention_kvc_store_gb300" / "csrc"


def test_every_bit_is_in_the_shared_list_once():
    found = [(name, int(bit), path.name)
             for path in sorted(CSRC.glob("*.cu")) + sorted(CSRC.glob("*.cuh"))
             for name, bit in re.findall(r"\b(kErr\w+)\s*=\s*1u\s*<<\s*(\d+)", path.read_text())]
    assert len(found) >= 14
    assert {where for _, _, where in found} == {"kvc_device.cuh"}
    assert sorted(bit for _, bit, _ in found) == list(range(len(found)))
