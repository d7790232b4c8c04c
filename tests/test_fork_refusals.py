"""kvc_fork's new rows are written while its parents and lengths are read: memory that both have is refused."""
import ctypes

import pytest

from pagedattention_kvc_store_gb300.kvc import lib

TABLE, LENS, REFS, OUT, OUT_LENS, PARENTS, SHARE = (0x10000000 * (i + 1) for i in range(7))


def fork(**a):
    p = dict(out=OUT, out_lens=OUT_LENS, parents=PARENTS, share=SHARE)
    p.update(a)
    at = {k: ctypes.c_void_p(v) for k, v in p.items()}
    return lib().kvc_fork(at["out"], 8, at["out_lens"], at["parents"], at["share"], 4, ctypes.c_void_p(TABLE), 8,
                          ctypes.c_void_p(LENS), 4, ctypes.c_void_p(REFS), 32, 16, None)


@pytest.mark.parametrize("change", [
    dict(parents=OUT), dict(parents=OUT + 4 * 8 * 4 - 4), dict(parents=OUT - 12), dict(share=OUT + 16),
    dict(share=OUT - 4), dict(out_lens=OUT), dict(out_lens=OUT + 100), dict(out_lens=PARENTS),
    dict(out_lens=SHARE + 4), dict(out=TABLE + 64), dict(out=LENS - 4), dict(out_lens=LENS), dict(out_lens=TABLE),
])
def test_memory_that_is_read_and_written(change):
    assert fork(**change) == 1
    assert b"apart" in lib().kvc_last_error()
