"""What libnvfp4_ffn.so asks of the runtime, on the CPU: its launches, and the shared memory that it has its kernels
allowed, as a library loaded before it records them in the runtime's place. Nothing is computed: addresses are made up."""
import json
import os
import shutil
import subprocess
import sys
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# The runtime's entry points that the library calls, with one device of 256 compute units. A launch is recorded as
# thread, grid, block, dynamic shared memory, and the most that its kernel is allowed at that time.
RECORDER = r"""
#include <pthread.h>
#include <stddef.h>
typedef struct { unsigned x, y, z; } dim3;
static pthread_mutex_t lock = PTHREAD_MUTEX_INITIALIZER;
static const void* kernels[1024];
static long allowed[1024];
static int count;
static long launches[4096][8];
static int launched;
static __thread dim3 grid, block;
static __thread size_t shared;
static __thread void* stream;

static int slot(const void* f) {
  for (int i = 0; i < count; ++i)
    if (kernels[i] == f) return i;
  kernels[count] = f;
  allowed[count] = 65536;
  return count++;
}
int hipGetDevice(int* d) { *d = 0; return 0; }
int hipDeviceGetAttribute(int* v, int attribute, int device) { *v = 256; return 0; }
int hipGetLastError(void) { return 0; }
int hipFuncSetAttribute(const void* f, int attribute, int value) {
  pthread_mutex_lock(&lock);
  allowed[slot(f)] = value;
  pthread_mutex_unlock(&lock);
  return 0;
}
int __hipPushCallConfiguration(dim3 g, dim3 b, size_t s, void* st) { grid = g; block = b; shared = s; stream = st; return 0; }
int __hipPopCallConfiguration(dim3* g, dim3* b, size_t* s, void** st) { *g = grid; *b = block; *s = shared; *st = stream; return 0; }
int hipLaunchKernel(const void* f, dim3 g, dim3 b, void** args, size_t s, void* st) {
  pthread_mutex_lock(&lock);
  if (launched < 4096) {
    long* l = launches[launched++];
    l[0] = slot(f); l[1] = g.x; l[2] = g.y; l[3] = g.z; l[4] = b.x; l[5] = (long)s; l[6] = allowed[slot(f)];
  }
  pthread_mutex_unlock(&lock);
  return 0;
}
int recorded(long* out) {
  int n = launched;
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < 8; ++j) out[8 * i + j] = launches[i][j];
  launched = 0;
  return n;
}
"""

# `record()`: (kernel, grid x, y, z, threads, shared memory, the most allowed) of the launches since the last one.
PRELUDE = """
import ctypes, json, sys, threading
recorder = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
from moe_matmul_amd import _ffn_binding as c
def record():
    out = (ctypes.c_long * 32768)()
    return [tuple(out[8 * i:8 * i + 7]) for i in range(recorder.recorded(out))]
P = 0x10000000
"""


@pytest.fixture(scope="module")
def recorder(tmp_path_factory):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    room = tmp_path_factory.mktemp("recorder")
    source, lib = room / "recorder.c", room / "librecorder.so"
    source.write_text(RECORDER)
    subprocess.run([cc, "-shared", "-fPIC", "-O1", "-pthread", str(source), "-o", str(lib)], check=True)
    return str(lib)


def run(recorder, program, *args):
    """What the program's last line says."""
    done = subprocess.run([sys.executable, "-c", PRELUDE + textwrap.dedent(program), recorder, json.dumps(args)], cwd=ROOT,
                          capture_output=True, text=True, timeout=120)
    assert done.returncode == 0, done.stderr
    return json.loads(done.stdout.splitlines()[-1])


# kind, rows, n, k, experts: products that take tiles of 320 rows (few of rows that many, some in parts of k)
TALL = [("linear", 640, 16384, 520, 0), ("linear", 1280, 13120, 64, 0), ("linear", 320, 13120, 8192, 0), ("linear", 620, 4096, 14336, 0),
        ("linear", 1480, 8192, 64, 3), ("gated", 640, 16384, 520, 0), ("gated", 1280, 13120, 64, 0), ("again", 1280, 13120, 64, 0),
        ("dx", 620, 2048, 14336, 0), ("dx", 1280, 2048, 14336, 0), ("dx", 620, 12288, 4096, 0), ("dx", 1480, 2048, 4096, 3), ("dx", 1040, 8192, 2048, 2)]


@pytest.mark.parametrize("kind,rows,n,k,experts", TALL)
def test_rows_far_apart_are_within_reach_of_a_tiles_offsets(recorder, kind, rows, n, k, experts):
    """Offsets from a tile's first row are signed 32-bit ones: its last row's 128 bytes of a stage end below 2^31, at any
    stride that is taken. A tile that is too tall gives way to the one of 256 rows, in the same workspace."""
    got = run(recorder, """
        kind, rows, n, k, experts = json.loads(sys.argv[2])
        what = {"linear": c.NVFP4_FFN_FORWARD, "gated": c.NVFP4_FFN_FORWARD, "again": c.NVFP4_FFN_FORWARD, "dx": c.NVFP4_FFN_DX}[kind]
        parts = c.nvfp4_ffn_product_parts(what, rows, n, k, experts)
        cols, depth = (k, n) if kind == "dx" else (n, k)
        need = c.nvfp4_ffn_product_workspace_bytes(rows, cols, depth, experts)
        plan = ctypes.byref(c.nvfp4_ffn_plan(experts, 1, P, P)) if experts else None
        grids = []
        reach = (2 ** 31 - 128) // 2 // 319 // 8 * 8  # the last stride that 320 rows allow
        strides = [depth, reach - 8, reach, reach + 8, 2 ** 22 - 8]
        for stride in strides:
            if kind == "linear":
                c.nvfp4_ffn_linear(P, stride, P, 0, 0, 0, 0, 0, 0, P, 2, rows, n, k, plan, 0, P, need, 0)
            elif kind == "gated":
                c.nvfp4_ffn_gated(P, stride, P, 2, P, 0, 0, 0, 2, rows, n // 2, k, plan, 0, P, need, 0)
            elif kind == "again":
                c.nvfp4_ffn_gated_again(P, n // 2, P, stride, P, 2, P, 2, rows, n // 2, k, plan, P, need, 0)
            else:
                c.nvfp4_ffn_linear_dx(P, stride, P, P, 2, rows, n, k, plan, 0, P, need, 0)
            grids.append(record())
        print(json.dumps([parts, strides, grids]))
    """, kind, rows, n, k, experts)
    parts, strides, grids = got
    (_, tall, wide, splits), = parts
    assert tall == 320
    cols = k if kind == "dx" else n

    def tiles(high):
        if experts:
            most = rows // high + min(experts, rows) + 1
            return -(-most * -(-cols // wide) * splits // 64) * 64
        return -(-rows // high) * -(-cols // wide) * splits

    assert tiles(320) != tiles(256)
    for stride, launches in zip(strides, grids):
        high = 320 if 319 * stride * 2 + 128 < 2 ** 31 else 256
        assert (high - 1) * stride * 2 + 128 < 2 ** 31
        assert launches[0][1] == tiles(high), stride
        assert len(launches) == (1 if splits == 1 else 2)


def test_threads_do_not_lower_each_others_shared_memory(recorder):
    """What a kernel is allowed belongs to the process: a thread's product of few rows of a short k leaves another's of a
    long k the shared memory that it asks for."""
    launches = run(recorder, """
        def product(gated, k):
            if gated:
                c.nvfp4_ffn_gated(P, k, P, 2, P, 0, 0, 0, 2, 8, 64, k, None, 0, 0, 0, 0)
            else:
                c.nvfp4_ffn_linear(P, k, P, 0, 0, 0, 0, 0, 0, P, 2, 8, 64, k, None, 0, 0, 0, 0)
        def thread(*ks):
            t = threading.Thread(target=lambda: [product(g, k) for k in ks for g in (False, True)])
            t.start()
            t.join()
        product(False, 16384)
        product(True, 16384)
        thread(5120)
        thread(4104, 8192)
        thread(4104)
        product(False, 16384)
        product(True, 16384)
        print(json.dumps(record()))
    """)
    assert len(launches) == 12 and max(l[5] for l in launches) > 65536
    for _, _, _, _, _, shared, allowed in launches:
        assert shared <= allowed, launches
