"""Launches at extreme sizes: what the entry points ask the runtime for, recorded by a stand-in for its launch
calls (no GPU needed).  A launch dimension takes fewer than 2^32 threads, and a larger one wraps without an error."""
import os
import random
import shutil
import subprocess
import sys

import pytest

STAND_IN = r"""
#include <stddef.h>
typedef struct { unsigned x, y, z; } dim3;
static dim3 next_grid, next_block;
static unsigned last[6];
static int launches;
int __hipPushCallConfiguration(dim3 grid, dim3 block, size_t shared, void* stream) { next_grid = grid; next_block = block; return 0; }
int __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, void** stream) {
  *grid = next_grid; *block = next_block; *shared = 0; *stream = 0;
  return 0;
}
int hipLaunchKernel(const void* f, dim3 grid, dim3 block, void** args, size_t shared, void* stream) {
  last[0] = grid.x; last[1] = grid.y; last[2] = grid.z; last[3] = block.x; last[4] = block.y; last[5] = block.z;
  ++launches;
  return 0;
}
int hipGetLastError(void) { return 0; }
unsigned* recorded(int* count) { *count = launches; return last; }
"""

# argv: stand-in, then calls on stdin; a line "rc launches gx gy gz bx by bz" for each
RUN = r"""
import ctypes, sys
shim = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
shim.recorded.restype = ctypes.POINTER(ctypes.c_uint)
import scoring_exact_top_amd as st
L, at, ws = st.raw_library(), ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 30)
count = ctypes.c_int()
for line in sys.stdin:
    name, *n = line.split()
    n = [int(v) for v in n]
    shim.recorded(ctypes.byref(count))
    before = count.value
    if name == "matmul":
        M, N, K, kind = n
        rc = L.idx_topk_matmul_e4m3(at, K, at, 0, at, at, M, N, K, kind, at, N, None)
    elif name == "rotate":
        T, H, D = n
        rc = L.idx_topk_norm_rotate(at, 0, 0, 0, None, None, 0.0, at, at, 100, 0, 0, T, H, D, 0, None, 0, 0, at, at, None)
    elif name == "append":
        rc = L.idx_topk_cache_append_rotary(at, 576, 1, None, 0.0, 1, at, 128, 2, None, None, 0.0, 0, 0, at, at, at, 100, n[0], 0, at, at, at,
                                            1 << 40, None, None)
    last = shim.recorded(ctypes.byref(count))
    print(rc, count.value - before, *last[:6], flush=True)
"""


def _launches(tmp_path, calls):
    """(rc, launches, grid, block) of each call, the grid and block those of its last launch."""
    cc = shutil.which("gcc") or shutil.which("cc") or shutil.which("amdclang", path="/opt/rocm/bin:/opt/rocm/llvm/bin")
    if cc is None:
        pytest.skip("no C compiler")
    source, lib = tmp_path / "stand_in.c", tmp_path / "stand_in.so"
    source.write_text(STAND_IN)
    subprocess.run([cc, "-shared", "-fPIC", "-o", str(lib), str(source)], check=True)
    text = "".join(" ".join(map(str, c)) + "\n" for c in calls)
    env = dict(os.environ, HIP_VISIBLE_DEVICES="-1")  # no device: the addresses of these calls are made up
    r = subprocess.run([sys.executable, "-c", RUN, str(lib)], input=text, capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, r.stderr
    lines = [[int(v) for v in line.split()] for line in r.stdout.splitlines()]
    assert len(lines) == len(calls)
    return [(n[0], n[1], n[2:5], n[5:8]) for n in lines]


def _check(call, rc, launches, grid, block, least):
    """Refused, or launched with every dimension below 2^32 threads and `least` of them in all."""
    assert rc in (0, -2), (call, rc)
    if rc == 0:
        assert launches >= 1, call
        assert all(0 < g and g * b <= 0xFFFFFFFF for g, b in zip(grid, block)), (call, grid, block)
        assert grid[0] * grid[1] * grid[2] * block[0] >= least, (call, grid, block)


def test_matmul_launches(tmp_path):
    """Every route up to the largest calls that the header states; a thread holds 128 sums at most."""
    rng = random.Random(1)
    calls = [(m, n) for big in (1 << 29, (1 << 29) + 1, (1 << 30) - 128) for m, n in ((big, 1), (big, 64), (33, big), (64, big), (big, 65), (100, big))]
    calls += [(m, (1 << 27) - 16) for m in (1, 16)] + [(m, (1 << 26) - 16) for m in (17, 32)]
    served = len(calls)
    calls += [((1 << 31) - 1, 1), (1, (1 << 31) - 1), (32, (1 << 31) - 1), (33, (1 << 31) - 1), ((1 << 31) - 1, (1 << 31) - 1), (1 << 30, 1)]
    calls += [tuple(int(2 ** rng.uniform(0, 31)) for _ in range(2)) for _ in range(400)]
    got = _launches(tmp_path, [("matmul", m, n, 16, i % 2) for i, (m, n) in enumerate(calls)])
    for i, ((m, n), g) in enumerate(zip(calls, got)):
        _check((m, n), *g, least=m * n // 128)
        tiles = -(-m // 128) * -(-n // 128) if m > 32 else -(-m // 16) * -(-n // 16)
        assert (g[0] == 0) == (tiles < 1 << 23), (m, n, g)
    assert all(g[0] == 0 for g in got[:served])


def test_rotate_and_append_launches(tmp_path):
    """Heads and tokens up to 2^31 - 1 of them: a wave of 64 lanes takes 8 x 4 heads of 64 numbers at most, or a token's rows."""
    rng = random.Random(2)
    most = (1 << 31) - 1
    calls = [("rotate", 1, most - i, d) for i in range(5) for d in (64, 128, 192, 200, 1024)]
    calls += [("rotate", most, 1, 128), ("rotate", most // 4, 4, 64), ("rotate", most // 5, 5, 192), ("rotate", most // 7, 7, 1000)]
    for _ in range(200):
        t = int(2 ** rng.uniform(0, 31))
        calls.append(("rotate", t, max(1, int(2 ** rng.uniform(0, 31)) // t), 8 * rng.randint(8, 128)))
    calls += [("append", t) for t in (1, 1000, 1 << 24, 1 << 30, most)]
    for call, got in zip(calls, _launches(tmp_path, calls)):
        assert got[0] == 0, call
        _check(call, *got, least=call[1] * 64 if call[0] == "append" else call[1] * call[2] * 2)
