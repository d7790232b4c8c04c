"""Every wait in the kernels has a limit, and is one of the shared ones.

A warp that polls for itself takes the decision to give up by a vote (warp_wait_over): a lane that
left by its own clock would leave the others alone in the next vote.  kvc_selftest_wait runs both kinds
on the GPU."""
import re
from pathlib import Path

CSRC = Path(__file__).resolve().parent.parent / "pagedattention_kvc_store_gb300" / "csrc"


def code_of(path):
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", path.read_text(), flags=re.S)


def test_limits_are_looked_at_in_the_shared_waits_only():
    sources = sorted(CSRC.glob("*.cu")) + sorted(CSRC.glob("*.cuh"))
    assert len(sources) > 10
    for path in sources:
        code = code_of(path)
        if path.name == "kvc_device.cuh":
            bodies = {m[1]: m[2] for m in re.finditer(
                r"bool (\w+)\([^)]*\)\s*\{(.*?)\n\}", code, flags=re.S)}
            users = {name for name, body in bodies.items() if "kWaitLimitCycles" in body}
            assert users == {"mbar_wait", "warp_wait_over"}
            assert re.search(r"return __any_sync\(0xffffffffu, clock64\(\) - since > kWaitLimitCycles\);",
                             bodies["warp_wait_over"])
        elif "selftest_wait_kernel" not in code:
            assert "kWaitLimitCycles" not in code, path.name
