"""The repository's entry file: run as a script it builds, and with --smoke also runs smoke(), and
nothing else; smoke() takes in every call that it is said to."""
import runpy
import sys
from pathlib import Path

import pytest

ENTRY = Path(__file__).resolve().parent.parent / "__graft_entry__.py"


def test_as_a_script_it_builds_and_ends(monkeypatch):
    import pagedattention_kvc_store_gb300 as kvc
    from oracle import oracle
    from pagedattention_kvc_store_gb300 import build
    done = []
    monkeypatch.setattr(build, "build", lambda: done.append("library"))
    monkeypatch.setattr(oracle, "build", lambda: done.append("oracle"))
    monkeypatch.setattr(kvc, "lib", lambda: done.append("load"))
    monkeypatch.setattr(sys, "argv", [str(ENTRY)])
    runpy.run_path(str(ENTRY), run_name="__main__")
    assert done == ["library", "oracle", "load"]


@pytest.mark.gpu
def test_smoke_takes_in_4_bit_pages_weights_and_eviction(monkeypatch):
    import pagedattention_kvc_store_gb300 as kvc
    called = set()
    for name in ("kvc_decode", "kvc_decode_store", "kvc_append", "kvc_decode_int8_store",
                 "kvc_store_int4", "kvc_decode_int4", "kvc_decode_weights", "kvc_evict"):
        def wrapped(*args, _call=getattr(kvc, name), _name=name, **kwargs):
            called.add(_name)
            return _call(*args, **kwargs)
        monkeypatch.setattr(kvc, name, wrapped)
    runpy.run_path(str(ENTRY))["smoke"]()
    assert called == {"kvc_decode", "kvc_decode_store", "kvc_append", "kvc_decode_int8_store",
                      "kvc_store_int4", "kvc_decode_int4", "kvc_decode_weights", "kvc_evict"}
