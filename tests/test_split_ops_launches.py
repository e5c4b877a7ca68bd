"""What embeddings, norms and 8-bit projections launch at the largest sizes that
include/rar.h allows: a grid holds less than 2^32 threads, and every workgroup
of a call is in one of its launches.  The addresses are made up; a stand-in
for HIP's launch, in a process of its own, writes down grids and blocks and
runs nothing.  No GPU needed."""
import ctypes
import json
import os
import shutil
import subprocess
import sys

import pytest

from ring_all_reduce_channelmask_amd import _lib

from .test_model_ops_args import A, BF16, F32, OK, _l, _p

G = 1 << 38  # between buffers; the largest here have 2^37 bytes

pytestmark = pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")

STUB = """
#include <stddef.h>
#include <string.h>
typedef struct { unsigned x, y, z; } dim3_t;
unsigned long long launches[64][4];  /* workgroups, threads of one, workgroups in the second dimension, LDS */
int count;
int hipLaunchKernel(const void* fn, dim3_t grid, dim3_t block, void** args, size_t lds, void* stream) {
  if (count < 64) {
    launches[count][0] = grid.x; launches[count][1] = block.x; launches[count][2] = (unsigned long long)grid.y * grid.z; launches[count][3] = lds;
  }
  ++count;
  return 0;
}
"""


def _embedding(tokens, width, dtype, vocab=10):
    return _lib.load().rar_embedding_allreduce(_p([A]), _l([vocab]), None, 1, width, dtype, A + G, tokens, 1.0, _p([A + 2 * G]), None, 1, None)


def _embedding_back(tokens, width, dtype, vocab, acc=0):
    return _lib.load().rar_embedding_allreduce_backward(_p([A]), None, 1, tokens, width, dtype, A + G, 1.0, _p([A + 2 * G]), _l([vocab]), None, 1, dtype, acc, A + 3 * G,
                                                        1 << 37, None)


def _norm(rows, width, dtype):
    n = _lib.Norm(rows=rows, width=width, dtype=dtype, eps=1e-6, residual_scale=1.0, pre_weight=A + G)
    return _lib.load().rar_norm_allreduce(ctypes.byref(n), _p([A]), None, 1, None, 0, _p([A]), None, 1, None, None, 0, None, 0, None)


def _norm_back(rows, width, dtype, groups):
    n = _lib.Norm(rows=rows, width=width, dtype=dtype, eps=1e-6, residual_scale=1.0, pre_weight=A + G, gate=A + 4 * G, gate_groups=groups)
    return _lib.load().rar_norm_allreduce_backward(ctypes.byref(n), _p([A]), None, 1, None, None, 0, A + 5 * G, 0, None, 0, _p([A]), None, 1, None, 0, None, A + 6 * G, 0,
                                                   None, A + 7 * G, 1 << 37, None)


def _quantize(rows, widths, dtype):
    xs, qs = [A + i * G for i in range(len(widths))], [A + (100 + i) * G for i in range(len(widths))]
    return _lib.load().rar_quantize_rows(_p(xs), _l(widths), None, len(widths), rows, dtype, _p(qs), None, A + 200 * G, None)


def _project(tokens, width, outer, dtype, skew=0):
    return _lib.load().rar_int8_projection_allreduce(_p([A + skew]), _l([width]), None, A + G, _p([A + 2 * G + skew]), None, A + 3 * G, 1, tokens, outer, dtype, None, 0,
                                                     _p([A + 4 * G]), None, 1, A + 10 * G, 1 << 38, None)


ALL = 1 << 24
# call, arguments, workgroups of each kind of launch (None: not looked at)
CASES = {
    "embedding, ordinary": (_embedding, (4096, 7168, BF16), [8192]),
    "embedding, 2^24 tokens of more than a wave": (_embedding, (ALL, 513, BF16), [ALL]),
    "embedding, 2^24 tokens of two workgroups": (_embedding, (ALL, 2500, F32), [2 * ALL]),
    "embedding, the last that one launch holds": (_embedding, (ALL - 1, 513, BF16), [ALL - 1]),
    "embedding gradient, ordinary": (_embedding_back, (100, 500, BF16, 1000), [100 + 250]),
    "embedding gradient, no tokens and 2^30 rows": (_embedding_back, (0, 1, BF16, 1 << 30), [1 << 24]),
    "embedding gradient, few tokens and 2^30 rows": (_embedding_back, (7, 1, F32, 1 << 30), [7 + (1 << 24)]),
    "embedding gradient, few tokens of 2^24": (_embedding_back, (1024, ALL, BF16, 2, 1), [1024 << 15]),
    "embedding gradient, by pairs and 2^30 rows": (_embedding_back, (2000, 5, BF16, 1 << 30), [32, None, 249]),
    "embedding gradient, by digits and 2^30 rows": (_embedding_back, (8193, 5, BF16, 1 << 30), [9] * 8 + [None, 1024]),
    "embedding gradient, 2^24 tokens": (_embedding_back, (ALL, 1000, BF16, 100, 1), [256] * 2 + [ALL // 64 * 2 // 4, (ALL // 64 - 1) * 2]),
    "norms, ordinary": (_norm, (4096, 7168, BF16), [4096]),
    "norms, 2^24 rows of 256 threads": (_norm, (ALL, 1544, BF16), [ALL]),
    "norms, 2^24 rows of 1024 threads": (_norm, (ALL, 4096, F32), [ALL]),
    "norms, 2^22 rows of 1024 threads": (_norm, (1 << 22, 7700, BF16), [1 << 22]),
    "norms gradient, a gate a row": (_norm_back, (ALL, 1544, BF16, ALL), [1024]),
    "quantisation, 2^24 rows of 64 ranks": (_quantize, (ALL, [1] * 64, BF16), [ALL]),
    "quantisation, ordinary": (_quantize, (4096, [1792] * 4, BF16), [4096]),
    "projection, 2^24 channels": (_project, (1, 100, ALL, BF16), [ALL // 16]),
    "projection, 2^24 tokens laid out first": (_project, (ALL, 5000, 1, F32, 1), [-(-ALL * 313 // 256), 2, None]),
    "projection, 2^24 channels laid out first": (_project, (17, 131071, ALL // 16, BF16, 1), [-(-17 * 8192 // 256), (ALL // 16) * 8192 // 256, None]),
    "projection, 256 and 192 channels a tile": (_project, (4000, 112, 7100, BF16), [16 * 16 + 16 * 16]),
    "projection, 256 and 192 channels a tile, whole": (_project, (4096, 64, 7168, BF16), [16 * 16 + 16 * 16]),
    "projection, 256 and 192 channels a tile, 32 rows": (_project, (8100, 96, 2900, F32), [32 * 8 + 32 * 5]),
    "projection, 2^38 results": (_project, (ALL, 112, 1 << 14, BF16), [1 << 22]),
    "projection, 2^38 results of another shape": (_project, (1 << 19, 112, 1 << 19, F32), [None]),
}


def child(stub):
    held = ctypes.CDLL(stub, mode=ctypes.RTLD_GLOBAL)  # found before HIP's own
    launches, count = (ctypes.c_uint64 * 4 * 64).in_dll(held, "launches"), ctypes.c_int.in_dll(held, "count")
    got = {}
    for name, (call, args, _) in CASES.items():
        count.value = 0
        code = call(*args)
        got[name] = [code, _lib.load().rar_get_last_error().decode(), [list(r) for r in launches[:count.value]]]
    print("GOT" + json.dumps(got))


@pytest.fixture(scope="module")
def got(tmp_path_factory):
    tmp = tmp_path_factory.mktemp("launches")
    src, stub = str(tmp / "stub.c"), str(tmp / "libstub.so")
    with open(src, "w") as f:
        f.write(STUB)
    subprocess.run(["gcc", "-shared", "-fPIC", src, "-o", stub], check=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", f"from tests import test_split_ops_launches as t; t.child({stub!r})"], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr
    return json.loads(run.stdout.split("GOT")[1])


@pytest.mark.parametrize("name", CASES)
def test_every_workgroup_is_launched_in_grids_that_hold_it(got, name):
    code, message, launches = got[name]
    assert code == OK, message
    for groups, threads, others, lds in launches:
        assert groups * threads < 1 << 32 and 0 < threads <= 1024 and 0 < others < 1 << 16 and lds <= 160 * 1024
    # several launches of a kernel follow each other, each but the last full
    for want in CASES[name][2]:
        assert launches, "a launch is missing"
        groups, threads = launches[0][:2]
        most = ((1 << 32) - 1) // threads
        n = 0
        while launches and launches[0][1] == threads and (want is None or n < want):
            g = launches.pop(0)[0]
            n += g
            if g < most:
                break
        assert want is None or n == want
    assert not launches


