"""Waits that may be as long as another warp's work, and what says that a wait ran out.

One expired wait has to end the others of its block: a limit many times as long as the usual one, run out by
every warp after another, would hold the GPU for minutes.  kvc_selftest_wait runs the shared wait on the GPU."""
import re
from pathlib import Path

from test_waits import CSRC, code_of

HEADER = Path(__file__).resolve().parent.parent / "include" / "kvc.h"


def test_long_waits_look_at_the_block_s_word():
    code = code_of(CSRC / "kvc_device.cuh")
    body = re.search(r"bool mbar_wait_work\([^)]*volatile uint32_t \*gave_up\)\s*\{(.*?)\n\}", code, flags=re.S)[1]
    assert re.search(r"if \(\*gave_up != 0\)\s*break;", body)      # after each second of its own
    assert re.search(r"\*gave_up = 1;\s*return false;", body)


def test_cross_attention_s_warps_wait_with_a_limit_and_say_when_it_ran_out():
    code = code_of(CSRC / "kvc_cross.cu")
    kernel = code[code.index("cross_kernel("):code.index("cross_merge_kernel(")]
    assert "named_barrier" not in kernel           # has no limit; one of its warps may have given up
    # the only unlimited meetings are those of all threads at the start and at the end
    assert kernel.count("__syncthreads()") == 5 and "bar.sync" not in kernel
    # every expired wait is told: of loads, products, items and softmax (waits for work tell it themselves)
    assert kernel.count("*gave_up = 1;") == 4
    # and the items' warp goes on asking for blocks without doing their work
    assert re.search(r"ok = ok && \*gave_up == 0;\s*if \(ok && make_item", kernel)


def test_every_bit_of_the_error_word_is_in_the_header():
    bits = [int(b) for b in re.findall(r"\bkErr\w+\s*=\s*1u\s*<<\s*(\d+)", (CSRC / "kvc_device.cuh").read_text())]
    text = HEADER.read_text()
    text = text[text.index("kvc_device_errors -- "):text.index("kvc_status kvc_device_errors")]
    told = {int(b) for b in re.findall(r"1 << (\d+)", text)}
    for lo, hi in re.findall(r"1 << (\d+) \.\. 1 << (\d+)", text):
        told |= set(range(int(lo), int(hi) + 1))
    assert told == set(bits)
