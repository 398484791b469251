"""nf_op_page_map at sizes where its shared memory passes the default limit, and calls of different sizes at once."""
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

# The sizes in ascending order and in a process of their own: a larger call before would raise the limit for them.
ASCENDING = """
import sys
sys.path[:0] = ['tests', '.']
import numpy as np
import intra_device_overlapped_b200 as nf
import kv4_reference as ref
from test_gpu_kv4 import _batch, _run_map, _same_map
for R in (4000, 4074, 4075, 4085, 4095, 4096, 4097):
    ctx, new, table, free, count, ids = _batch(np.random.default_rng(R), R, 40, 2, 3)
    pages, tokens = int((-(-(ctx + new) // 16)).sum()), int(new.sum())
    got = _run_map(nf, ctx, new, table, free, count, ids, pages, tokens)
    _same_map(got, ref.page_map(ctx, new, table, free, count, ids, pages, tokens), R)
print('all sizes')
"""


def test_sizes_around_the_default_limit_in_a_new_process():
    got = subprocess.run([sys.executable, "-c", ASCENDING], capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and "all sizes" in got.stdout, got.stderr[-2000:]
