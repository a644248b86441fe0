"""How a product of linear_fp4's warp kernel is shared by blocks, warps and passes, over its sizes (no GPU needed): the
launch code's own arithmetic, compiled as plain C++."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

import moe_routed_expert_router_gb300 as moe

CSRC = os.path.join(os.path.dirname(os.path.abspath(moe.__file__)), "csrc")
FIELDS = ["blocks", "groups", "base", "extra", "passes", "pass_rows", "tile_rows", "wk", "wm", "tiles", "ring", "smem"]
SOURCE = r"""
#include "linear_split.cuh"
using namespace moe;
extern "C" {
void split(int T, int N, int K, LinearSplit *s) { *s = linear_split(linear_tokens(T), T, N, K); }
int smem_limit() { return (int)kSmemBlock; }
int sizes(int nt, int *out) { out[0] = linear_warps(nt), out[1] = linear_stage_bytes(nt), out[2] = linear_sum_bytes(nt); return linear_stage_k(nt); }
// Rows of tile `tile` of a block's pass, as the kernel takes them.
void tile(const LinearSplit *s, int block, int pass, int tile, int *out) {
    const RowRange b = linear_block_rows(*s, block), p = linear_pass_rows(*s, b, pass), t = linear_tile_rows(*s, p, tile);
    const int all[6] = {b.first, b.end, p.first, p.end, t.first, t.end};
    for (int i = 0; i < 6; ++i) out[i] = all[i];
}
// 0 where the tiles of a block's passes take its rows once and in order, up to `tile_rows` a tile; else where they stop.
long long not_covered(const LinearSplit *s, int block) {
    const RowRange b = linear_block_rows(*s, block);
    long long at = b.first;
    for (int pass = 0; pass < s->passes; ++pass) {
        const RowRange p = linear_pass_rows(*s, b, pass);
        if (p.first != at || p.end < p.first || p.end - p.first > s->pass_rows) return at + 1;
        for (int tile = 0; tile < s->wm * s->tiles; ++tile) {
            const RowRange t = linear_tile_rows(*s, p, tile);
            if (t.first != at || t.end < t.first || t.end - t.first > s->tile_rows || t.end > p.end) return at + 1;
            at = t.end;
        }
        if (at != p.end) return at + 1;
    }
    return at == b.end ? 0 : at + 1;
}
// The first of N = n0, n0 + step .. n1 whose block does not fit, or 0.
int first_too_large(int T, int n0, int n1, int step, int K) {
    const int nt = linear_tokens(T);
    for (int n = n0; n <= n1; n += step) {
        const LinearSplit s = linear_split(nt, T, n, K);
        const int warps = s.wk * s.wm;
        if (s.smem > (int)kSmemBlock || s.smem != warps * (s.ring * linear_stage_bytes(nt) + s.tiles * linear_sum_bytes(nt)) ||
            s.ring < kLeastLinearRing || s.ring > kMostLinearRing || warps < 1 || warps > linear_warps(nt) || s.tile_rows > kLinearRows || s.tiles < 1)
            return n;
    }
    return 0;
}
}
"""


class Split(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int) for f in FIELDS]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("split")
    (d / "split.cpp").write_text(SOURCE)
    so = d / "split.so"
    subprocess.run([cxx, "-O2", "-std=c++17", "-fwrapv", "-shared", "-fPIC", "-I", CSRC, "-o", str(so), str(d / "split.cpp")], check=True)
    c = ctypes.CDLL(str(so))
    c.not_covered.restype = ctypes.c_longlong
    return c


def split(lib, T, N, K):
    s = Split()
    lib.split(T, N, K, ctypes.byref(s))
    return s


def test_the_limit_is_what_a_kernel_may_ask_for():
    """One constant sets the kernels' limit and plans the rings."""
    with open(os.path.join(CSRC, "rows.cuh")) as f:
        assert "cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBlock)" in f.read()


@pytest.mark.parametrize("T,N,K", [(1, 25600, 2816), (8, 24321, 2688), (9, 30000, 2688), (16, 18000, 2688), (16, 19456, 2816), (32, 18000, 1408),
                                   (32, 17025, 1408), (64, 9000, 1408), (64, 28000, 1408)])
def test_splits_of_eleven_warps(lib, T, N, K):
    s = split(lib, T, N, K)
    assert s.wk * s.wm == 11 and s.smem <= lib.smem_limit()


@pytest.mark.parametrize("T", [1, 8, 9, 16, 17, 32, 33, 64, 65, 100, 152, 300, 1000, 2500, 4000, 4865, 10000, 1 << 20])
def test_every_split_fits_a_block(lib, T):
    """All K, and rows from 1 to the most: every count of tiles a block can have, many times over."""
    for K in range(128, 65537, 128):
        assert lib.first_too_large(T, 1, 300, 37, K) == 0
        assert lib.first_too_large(T, 301, 60000, 991, K) == 0
        assert lib.first_too_large(T, 60000, 3000000, 99991, K) == 0
        assert lib.first_too_large(T, 3000000, (1 << 31) - 100000000, 97000003, K) == 0


@pytest.mark.parametrize("seed", range(4))
def test_drawn_splits_fit_a_block(lib, seed):
    r = random.Random(seed)
    for _ in range(20000):
        T, N, K = int(2 ** r.uniform(0, 20)), int(2 ** r.uniform(0, 30.99)), 128 * int(2 ** r.uniform(0, 9))
        assert lib.first_too_large(T, N, N, 1, K) == 0, (T, N, K)


LARGEST = (1 << 31) - 1 - 1024                                    # rows that moe_linear_fp4 takes


def covered(lib, T, N, K):
    s = split(lib, T, N, K)
    assert linear_rows(lib, s, 0)[0] == 0 and linear_rows(lib, s, s.blocks - 1)[1] == N
    for block in {0, s.extra // 2, max(0, s.extra - 1), min(s.extra, s.blocks - 1), s.blocks // 2, s.blocks - 1}:
        assert lib.not_covered(ctypes.byref(s), block) == 0, (T, N, K, block)
        if block + 1 < s.blocks:
            assert linear_rows(lib, s, block)[1] == linear_rows(lib, s, block + 1)[0]
    return s


def linear_rows(lib, s, block):
    out = (ctypes.c_int * 6)()
    lib.tile(ctypes.byref(s), block, 0, 0, out)
    return out[0], out[1]


# the last block's passes times their rows pass 2^31: outputs of its last pass (up to 4607 rows) were left as they were
@pytest.mark.parametrize("T,N,K", [(1, 2147482151, 128), (8, 2147482623, 128), (9, 2147481962, 128), (16, LARGEST, 128), (20, 2147482349, 128),
                                   (64, LARGEST, 128), (1, LARGEST, 65536), (20000, LARGEST, 128), (1 << 20, LARGEST, 1280)])
def test_the_largest_weights_rows_are_all_taken(lib, T, N, K):
    s = covered(lib, T, N, K)
    assert s.passes > 1


@pytest.mark.parametrize("seed", range(4))
def test_every_row_is_taken_once(lib, seed):
    r = random.Random(100 + seed)
    for _ in range(3000):
        T, N, K = int(2 ** r.uniform(0, 20)), int(2 ** r.uniform(0, 24)), 128 * int(2 ** r.uniform(0, 9))
        covered(lib, T, N, K)
    for _ in range(20):
        covered(lib, r.choice([1, 12, 30, 100]), r.randint(LARGEST - (1 << 16), LARGEST), 128 * r.randint(1, 30))


@pytest.mark.parametrize("N,status", [(LARGEST, moe.ERR_INVALID_ARG), (LARGEST + 1, moe.ERR_UNSUPPORTED_SHAPE)])
def test_the_border_of_the_rows_taken(N, status):
    """The largest weight is refused for its missing pointers only."""
    w = moe.Nvfp4(None, None, None)
    assert moe.lib().moe_linear_fp4(256, 128, ctypes.byref(w), moe.WEIGHTS_MXFP4, 1, N, 128, moe.DTYPE_F16, moe.DTYPE_F16, 256, None, 0, None) == status
