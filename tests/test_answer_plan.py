"""How calls of the operators between a hidden state and text are cut into
launches, checked without a device: the arithmetic is host code of its own."""
import ctypes
import os
import subprocess

import pytest

import answers

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = """
#include "plan.hpp"
extern "C" {
uint64_t groups_in_x(uint64_t threads) { return bpek::groups_in_x(threads); }
uint64_t groups_in_y() { return bpek::GROUPS_IN_Y; }
// each part's first row, rows and workgroups; returns how many parts there are
int parts(uint64_t rows, uint64_t group_rows, uint64_t most_groups, uint64_t *out, int room) {
    int n = 0;
    bpek::in_parts(rows, group_rows, most_groups, [&](uint64_t at, uint32_t part, uint32_t groups) {
        if (n < room) out[3 * n] = at, out[3 * n + 1] = part, out[3 * n + 2] = groups;
        ++n;
    });
    return n;
}
int share_bytes(uint64_t a, uint64_t a_bytes, uint64_t b, uint64_t b_bytes) {
    return bpek::share_bytes((const void*)a, a_bytes, (const void*)b, b_bytes);
}
int share_rows(uint64_t a, uint64_t a_stride, uint64_t b, uint64_t b_stride, uint64_t rows, uint64_t width) {
    return bpek::share_rows((const void*)a, a_stride, (const void*)b, b_stride, rows, width);
}
int kernels() { return bpek::PK_COUNT; }
int first_tile() { return bpek::PK_TILE_128_64; }
// the kernel of a product and the kind of its pieces
int kernel(uint64_t m, uint64_t n, uint64_t k, int aligned_rows, int exact, int tiled, int *kind) {
    *kind = bpek::pieces_of(k, aligned_rows);
    return bpek::product_kernel(m, n, (k + 127) / 128, bpek::Pieces(*kind), exact, tiled);
}
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    where = tmp_path_factory.mktemp("plan")
    src, lib = where / "plan.cpp", where / "plan.so"
    src.write_text(SOURCE)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                           os.path.join(ROOT, "bpe_merge_amd", "csrc"), "-o", str(lib), str(src)])
    lib = ctypes.CDLL(str(lib))
    u64 = ctypes.c_uint64
    lib.groups_in_x.argtypes, lib.groups_in_x.restype, lib.groups_in_y.restype = [u64], u64, u64
    lib.kernel.argtypes = [u64, u64, u64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
    lib.share_bytes.argtypes, lib.share_rows.argtypes = [u64] * 4, [u64] * 6
    lib.parts.argtypes = [u64, u64, u64, ctypes.POINTER(u64), ctypes.c_int]
    return lib


def _parts(plan, rows, group_rows, most):
    room = 600
    out = (ctypes.c_uint64 * (3 * room))()
    n = plan.parts(rows, group_rows, most, out, room)
    assert n <= room
    return [tuple(out[3 * i:3 * i + 3]) for i in range(n)]


# threads of a workgroup and its rows, as norm and sampling launch them
@pytest.mark.parametrize("threads, group_rows", [(256, 4), (256, 1), (1024, 1)])
def test_rows_beyond_a_launch_go_in_parts(plan, threads, group_rows):
    most = plan.groups_in_x(threads)
    assert most * threads < 1 << 32 <= (most + 1) * threads
    limit = most * group_rows
    for rows in (1, 2, group_rows + 1, limit - 1, limit, limit + 1, 2 * limit + 3, 0x7FFFFFFF):
        parts = _parts(plan, rows, group_rows, most)
        assert len(parts) == -(-rows // limit)
        at = 0
        for first, part, groups in parts:
            assert first == at and 0 < part <= 0x7FFFFFFF
            assert (groups - 1) * group_rows < part <= groups * group_rows and groups * threads < 1 << 32
            at += part
        assert at == rows
    assert _parts(plan, 0, group_rows, most) == []


def test_rows_of_products_beyond_a_launch_go_in_parts(plan):
    """Workgroups of 16, 32 or 64 rows along y, up to the largest m."""
    most = plan.groups_in_y()
    assert most == 65535
    for group_rows in (16, 32, 64):
        limit = most * group_rows
        for rows in (1, limit, limit + 1, 0x7FFF80):
            parts = _parts(plan, rows, group_rows, most)
            assert [p[0] for p in parts] == list(range(0, rows, limit)) and sum(p[1] for p in parts) == rows
            assert all((g - 1) * group_rows < n <= g * group_rows and g <= most for _, n, g in parts)
    # along x the widest launch has a workgroup of 512 threads for each 16 rows of b
    assert -(-0x7FFF80 // 16) <= plan.groups_in_x(512)


def test_arrays_that_share_memory(plan):
    for a, n, b, m, want in [(0, 10, 10, 5, 0), (10, 5, 0, 10, 0), (0, 10, 9, 5, 1), (9, 5, 0, 10, 1), (0, 100, 40, 1, 1),
                             (40, 1, 0, 100, 1), (7, 3, 7, 3, 1), (7, 0, 7, 3, 0), (7, 3, 7, 0, 0), (5, 0, 0, 100, 0)]:
        assert plan.share_bytes(0x1000 + a, n, 0x1000 + b, m) == want


def test_rows_that_share_memory(plan):
    """Against the sets of their bytes."""
    def taken(at, stride, rows, width):
        return {at + r * stride + i for r in range(rows) for i in range(width)}
    for rows, stride, width in [(1, 9, 4), (2, 4, 4), (3, 9, 4), (4, 10, 5), (3, 7, 4), (2, 12, 3)]:
        for off in range(-40, 41):
            want = bool(taken(100, stride, rows, width) & taken(100 + off, stride, rows, width))
            assert plan.share_rows(100, stride, 100 + off, stride, rows, width) == want, (rows, stride, width, off)
    assert plan.share_rows(100, 4, 112, 8, 3, 4) == 0 and plan.share_rows(100, 4, 108, 8, 3, 4) == 1
    assert plan.share_rows(100, 4, 100, 4, 0, 4) == 0


def _kernel(plan, m, n, k, aligned_rows, exact, tiled=True):
    """What a product runs: (kernel, kind of its pieces where it is a tile)."""
    kind = ctypes.c_int()
    kernel = plan.kernel(m, n, k, aligned_rows, exact, tiled, ctypes.byref(kind))
    assert 0 <= kernel < plan.kernels()
    return kernel, kind.value if kernel >= plan.first_tile() else None


@pytest.mark.parametrize("exact", [False, True])
def test_the_products_tested_take_every_kernel(plan, exact):
    """Every kernel and kind of pieces that a sweep over sizes meets is taken
    by one of answers.PRODUCTS, whose rows the library is given aligned."""
    sizes = sorted({int(f * 2 ** e) + d for e in range(15) for f in (1, 1.25, 1.6) for d in (-1, 0, 1)} - {-1, 0})
    met = {}
    for m in sizes[::2]:
        for n in sizes[::2] + [33000, 65536]:
            for k in (64, 128, 130, 144, 1024, 1025, 1040, 2048, 2049, 2064, 8192):
                for aligned_rows in (0, 1):
                    met.setdefault(_kernel(plan, m, n, k, aligned_rows, exact), (m, n, k))
    tested = {_kernel(plan, m, n, k, 1, exact) for m, n, k in answers.PRODUCTS}
    assert {what: size for what, size in met.items() if what not in tested} == {}
    assert tested <= set(met)
    deep = [p for p in answers.PRODUCTS if _kernel(plan, *p, 1, False) == _kernel(plan, 520, 16640, 384, 1, False)]
    assert max(k for _, _, k in deep) >= 2048  # the widest tile over many blocks of K too
    names = {kernel for kernel, _ in met}
    # all kernels there are, but for those of the other form of sums: the widest
    # tile, and the tile of eight waves
    assert len(names) == plan.kernels() - 1


def test_rows_far_apart_take_streams(plan):
    for m, n, k in answers.PRODUCTS:
        assert _kernel(plan, m, n, k, 1, True, tiled=False)[0] < plan.first_tile()
