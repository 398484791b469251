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


def _calls(nf, R, stream):
    """Arguments of a call of R requests on `stream` on arrays of its own, and a check of what it has to give."""
    import torch
    import kv4_reference as ref
    from test_gpu_kv4 import _batch, _i32
    ctx, new, table, free, count, ids = _batch(np.random.default_rng(R), R, 20, 1, 3)
    pages, tokens = int((-(-(ctx + new) // 16)).sum()), int(new.sum())
    want = ref.page_map(ctx, new, table, free, count, ids, pages, tokens)
    ins = [_i32(ctx), _i32(new), _i32(free), _i32([count])]
    out = {"table": _i32(table), "kv_len": _i32([-7] * R), "indptr": _i32([-7] * (R + 1)), "indices": _i32([-7] * pages),
           "slots": _i32([-7] * tokens), "positions": _i32([-7] * tokens), "left": _i32([-7]), "status": _i32([0])}
    torch.cuda.synchronize()

    args = (ins[0].data_ptr(), ins[1].data_ptr(), R, out["table"].data_ptr(), table.shape[1], ins[2].data_ptr(), len(free),
            ins[3].data_ptr(), ids, out["kv_len"].data_ptr(), out["indptr"].data_ptr(), out["indices"].data_ptr(), pages,
            out["slots"].data_ptr(), out["positions"].data_ptr(), tokens, out["left"].data_ptr(),
            out["status"].data_ptr(), stream.cuda_stream)

    def check():
        for name in ("kv_len", "indptr", "indices", "slots", "positions"):
            assert out[name].tolist() == want[name], (R, name)
        assert out["left"].item() == want["left"] and np.array_equal(out["table"].cpu().numpy(), want["table"])
        assert out["status"].item() == 0
        ins[0].data_ptr()   # (kept as long as this is)
    return args, check


# Two threads that call without a pause, which threads of the interpreter do not
HAMMER = """
#include <pthread.h>
#include <stdint.h>
struct args { void *ctx, *fresh; int32_t n; void* table; int32_t stride; void* free_pages; int32_t cap; void* count; int32_t pages;
              void *kv_len, *indptr, *indices; int32_t page_cap; void *slots, *positions; int32_t token_cap;
              void *left, *status, *stream; };
typedef int (*page_map)(void*, void*, int32_t, void*, int32_t, void*, int32_t, void*, int32_t, void*, void*, void*, int32_t,
                        void*, void*, int32_t, void*, void*, void*);
struct job { page_map f; struct args a; int32_t calls, failed; };
static void* work(void* p) {
    struct job* j = (struct job*)p;
    const struct args* a = &j->a;
    for (int32_t i = 0; i < j->calls; ++i)
        j->failed += j->f(a->ctx, a->fresh, a->n, a->table, a->stride, a->free_pages, a->cap, a->count, a->pages, a->kv_len,
                          a->indptr, a->indices, a->page_cap, a->slots, a->positions, a->token_cap, a->left,
                          a->status, a->stream) != 0;
    return 0;
}
void hammer(struct job* jobs, int32_t n) {
    pthread_t t[8];
    for (int32_t i = 0; i < n; ++i) pthread_create(&t[i], 0, work, &jobs[i]);
    for (int32_t i = 0; i < n; ++i) pthread_join(t[i], 0);
}
"""


def test_calls_of_different_sizes_from_two_threads(tmp_path):
    import ctypes
    import torch
    import intra_device_overlapped_b200 as nf
    (tmp_path / "hammer.c").write_text(HAMMER)
    subprocess.run(["gcc", "-O2", "-shared", "-fPIC", "-o", tmp_path / "hammer.so", tmp_path / "hammer.c", "-lpthread"],
                   check=True)
    lib = ctypes.CDLL(str(tmp_path / "hammer.so"))
    types = nf._lib.nf_op_page_map.argtypes

    class Args(ctypes.Structure):
        _fields_ = [("a%d" % i, t) for i, t in enumerate(types)]

    class Job(ctypes.Structure):
        _fields_ = [("f", ctypes.c_void_p), ("a", Args), ("calls", ctypes.c_int32), ("failed", ctypes.c_int32)]

    torch.cuda.init()
    streams = [torch.cuda.Stream() for _ in range(2)]
    made = [_calls(nf, R, st) for R, st in zip((16384, 5000), streams)]
    jobs = (Job * 2)(*[Job(ctypes.cast(nf._lib.nf_op_page_map, ctypes.c_void_p).value, Args(*args), 20000, 0)
                       for args, _ in made])
    lib.hammer(jobs, 2)
    torch.cuda.synchronize()
    assert [j.failed for j in jobs] == [0, 0]
    for _, check in made:
        check()


def test_a_smaller_call_behind_a_larger_one_in_a_graph():
    import torch
    import intra_device_overlapped_b200 as nf
    stream = torch.cuda.Stream()
    made = [_calls(nf, R, stream) for R in (16384, 5000, 9000)]
    between = _calls(nf, 4100, stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        codes = [nf.nf_op_page_map(*args) for args, _ in made]
    assert codes == [0, 0, 0]
    assert nf.nf_op_page_map(*between[0]) == 0     # between the capture and the replay
    graph.replay()
    torch.cuda.synchronize()
    for _, check in made + [between]:
        check()
