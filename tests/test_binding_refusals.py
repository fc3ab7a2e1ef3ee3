"""What the bindings refuse before they compute with it, on the CPU.  Each call runs in a
process of its own: a division by zero in the C++ binding ends the process."""
import subprocess
import sys

import pytest

import conftest
import speculative_decoding_verify_03_gb300 as sv


@pytest.fixture(scope="module", autouse=True)
def built():
    sv.build()


CALL = """
import sys
import torch
import speculative_decoding_verify_03_gb300 as sv
i = lambda *s: torch.zeros(s, dtype=torch.int32)
z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
heads, slots, op = int(sys.argv[1]), int(sys.argv[2]), sys.argv[3]
c = sv.KVCache(z(3, heads, slots, 64), z(3, heads, slots, 64))
kw = dict(prefix_table=i(4), prefix_len=1)
try:
    if op == "attend_tree":
        sv.spec_attend_tree(z(2, 3, 4, 64), c, i(2, 4), i(2), i(2, 3, 1), **kw)
    elif op == "attend":
        sv.spec_attend(z(2, 3, 4, 64), c, i(2, 4), i(2), **kw)
    else:
        sv.spec_kv_read(c, i(2, 4), i(2), 1, **kw)
except ValueError as e:
    print("refused:", e)
"""


@pytest.mark.parametrize("heads,slots,op", [(0, 16, "attend_tree"), (2, 0, "attend_tree"), (0, 0, "attend_tree"),
                                            (0, 16, "attend"), (2, 0, "attend"), (2, 0, "read")])
def test_caches_without_heads_or_slots(heads, slots, op):
    run = subprocess.run([sys.executable, "-c", CALL, str(heads), str(slots), op], cwd=conftest.ROOT, capture_output=True,
                         text=True, timeout=600)
    assert run.returncode == 0 and "refused: the cache's pages must hold" in run.stdout, (run.returncode, run.stderr[-2000:])
