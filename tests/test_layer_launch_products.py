"""What the launcher of the integer products asks the runtime for, on the CPU, with
stand-ins for the runtime's launch calls: pieces that cover every output once, each
with the addresses of its first row and column; splits of K that the workspace and
the counters hold and that leave none empty; tiles only where K fills their ring."""
import ctypes
import os
import re
import subprocess

import pytest

from dense_linear_projection_amd import _build

STUBS = r"""
#include <map>
#include <string>
#include <vector>
#include "layer.hpp"
using namespace proj;
struct Launch {
    std::string name;
    dim3 grid, block;
    IntArgs a;
    uint32_t splits;
};
static std::vector<Launch> &launches() { static std::vector<Launch> v; return v; }
static std::map<const void *, std::string> &names() { static std::map<const void *, std::string> m; return m; }
static dim3 next_grid, next_block;
extern "C" {
void **__hipRegisterFatBinary(const void *) { static void *p; return &p; }
void __hipUnregisterFatBinary(void **) {}
void __hipRegisterFunction(void **, const void *f, char *, const char *name, unsigned, void *, void *, void *, void *, int *) {
    names()[f] = name;
}
hipError_t __hipPushCallConfiguration(dim3 g, dim3 b, size_t, hipStream_t) {
    next_grid = g, next_block = b;
    return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3 *g, dim3 *b, size_t *lds, hipStream_t *st) {
    *g = next_grid, *b = next_block, *lds = 0, *st = nullptr;
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void *f, dim3 g, dim3 b, void **args, size_t, hipStream_t) {
    if (g.x == 0 || static_cast<uint64_t>(g.x) * b.x > 0xffffffffull) return hipErrorInvalidConfiguration;
    const std::string name = names()[f];
    if (name.find("int_") != std::string::npos)
        launches().push_back({name, g, b, *static_cast<IntArgs *>(args[0]), name.find("stream") != std::string::npos ? *static_cast<uint32_t *>(args[1]) : 1u});
    return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }

int stub_count() { return static_cast<int>(launches().size()); }
void stub_clear() { launches().clear(); }
const char *stub_name(int i) { return launches()[i].name.c_str(); }
int64_t stub_field(int i, int what) {
    const Launch &l = launches()[i];
    const IntArgs &a = l.a;
    const int64_t at[] = {l.grid.x, l.block.x, l.splits, a.M, a.N, a.K, a.row, reinterpret_cast<int64_t>(a.X), reinterpret_cast<int64_t>(a.W),
                          reinterpret_cast<int64_t>(a.x_scales), reinterpret_cast<int64_t>(a.w_scales), reinterpret_cast<int64_t>(a.bias),
                          reinterpret_cast<int64_t>(a.Y), reinterpret_cast<int64_t>(a.rows)};
    return at[what];
}
int stub_int(int64_t M, int64_t N, int64_t K, int64_t ws, int f32, int fused, int ncounters) {
    IntArgs a{reinterpret_cast<int8_t *>(1ll << 52), reinterpret_cast<int8_t *>(2ll << 52), reinterpret_cast<float *>(3ll << 52),
              reinterpret_cast<float *>(4ll << 52), reinterpret_cast<uint16_t *>(5ll << 52), reinterpret_cast<void *>(6ll << 52), M, N, K, N, 3,
              f32 ? OUT_F32 : OUT_BF16, reinterpret_cast<int32_t *>(7ll << 52), static_cast<size_t>(ws), 256, nullptr, ncounters};
    if (!fused) return launch_int(a, nullptr);
    if (!int_fuses(M, N, K)) return -1;
    a.rows = reinterpret_cast<uint16_t *>(8ll << 52), a.rows_stride = a.rows_k = K;
    return launch_int_fused(a, nullptr);
}
}
"""
FIELDS = ["grid", "block", "splits", "M", "N", "K", "row", "X", "W", "xs", "ws", "bias", "Y", "rows"]
WS, COUNTERS = 64 << 20, 16384


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    at = tmp_path_factory.mktemp("layer_launch_products")
    (at / "stubs.cpp").write_text(STUBS)
    flags = ["--offload-arch=gfx950", "--cuda-host-only", "-O1", "-std=c++17", "-fPIC", "-I", _build.CSRC, "-x", "hip"]
    objs = []
    for src in (os.path.join(_build.CSRC, "int8.hip"), str(at / "stubs.cpp")):
        objs.append(str(at / (os.path.basename(src) + ".o")))
        subprocess.run([_build.hipcc()] + flags + ["-c", src, "-o", objs[-1]], check=True, capture_output=True)
    # the device code that a host half refers to by a name of its own, nowhere read
    names = set(re.findall(r"__hip_fatbin_\w+", subprocess.run(["nm", "-u"] + objs, check=True, capture_output=True, text=True).stdout))
    (at / "fatbin.c").write_text("".join("const char %s[16] = {0};\n" % n for n in sorted(names)))
    so = str(at / "layer_launch_products.so")
    subprocess.run(["gcc", "-fPIC", "-c", str(at / "fatbin.c"), "-o", str(at / "fatbin.o")], check=True)
    subprocess.run(["g++", "-shared", "-Wl,-Bsymbolic", "-o", so, str(at / "fatbin.o")] + objs, check=True)
    L = ctypes.CDLL(so)
    i64, ci = ctypes.c_int64, ctypes.c_int
    L.stub_name.restype = ctypes.c_char_p
    L.stub_field.argtypes, L.stub_field.restype = [ci, ci], i64
    L.stub_int.argtypes = [i64, i64, i64, i64, ci, ci, ci]
    return L


def product(host, M, N, K, ws, f32, fused=0, counters=COUNTERS):
    host.stub_clear()
    assert host.stub_int(M, N, K, ws, f32, fused, counters) == 0, (M, N, K, ws)
    return [(host.stub_name(i).decode(), {f: host.stub_field(i, j) for j, f in enumerate(FIELDS)}) for i in range(host.stub_count())]


def check(got, M, N, K, ws, f32, fused=0, counters=COUNTERS):
    size, area, pieces = 4 if f32 else 2, 0, []
    for name, a in got:
        m, n = (a["xs"] - (3 << 52)) // 4, (a["ws"] - (4 << 52)) // 4
        assert 0 <= m and m + a["M"] <= M and 0 <= n and n + a["N"] <= N and a["M"] > 0 and a["N"] > 0
        assert a["X"] == (1 << 52) + m * K and a["W"] == (2 << 52) + n * K and a["bias"] == (5 << 52) + 2 * n
        assert a["Y"] == (6 << 52) + (m * N + n) * size and a["row"] == N and a["K"] == K
        area += a["M"] * a["N"]
        pieces.append((m, m + a["M"], n, n + a["N"]))
        sizes = [int(x) for x in re.findall(r"Li(\d+)E", name)]
        if "int_stream_kernel" in name:
            mt, nt, waves, kc, _ = sizes
            tiles = -(-a["M"] // (16 * mt)) * -(-a["N"] // (16 * nt))
            assert K > 0 and a["block"] == 64 * waves and a["grid"] == tiles * a["splits"] and 1 <= a["splits"] <= -(-K // kc)
            if a["splits"] > 1:
                assert tiles * a["splits"] * mt * nt * 1024 <= ws and tiles <= counters
            assert ("Lb1E" in name) == bool(fused)
        elif "int_tile_kernel" in name:
            bm, bn = sizes[:2]
            assert K > 128 and a["block"] == 512 and 1 <= a["grid"] <= -(-a["M"] // bm) * -(-a["N"] // bn)
        else:
            assert K == 0 and "int_empty_kernel" in name
    assert area == M * N
    for i, p in enumerate(pieces):
        for q in pieces[:i]:
            assert p[0] >= q[1] or q[0] >= p[1] or p[2] >= q[3] or q[2] >= p[3]


@pytest.mark.parametrize("M", [1, 8, 16, 17, 32, 33, 64, 65, 128, 129, 256, 257, 512, 4096, (1 << 20) + 5, 1 << 33])
@pytest.mark.parametrize("N", [1, 64, 1000, 28672, (1 << 28) + 1, (1 << 33) + 77])
@pytest.mark.parametrize("ws", [0, 1 << 16, WS])
def test_pieces_cover_every_output_once(host, M, N, ws):
    for K in (0, 16, 128, 144, 8192, 131056):
        if M * N <= 1 << 40 and M * K <= 1 << 40 and N * K <= 1 << 40:
            for f32 in (0, 1):
                check(product(host, M, N, K, ws, f32), M, N, K, ws, f32)


@pytest.mark.parametrize("ws", [0, 3000, 1 << 14, 1 << 16, 1 << 18, 1 << 20, WS])
@pytest.mark.parametrize("counters", [0, 1, 7, COUNTERS])
def test_splits_fit(host, ws, counters):
    for M in (1, 16, 40, 64, 100, 128):
        for N in (16, 64, 512, 1000):
            for K in (4096, 8192, 12304, 65536, 131056):
                check(product(host, M, N, K, ws, 1, 0, counters), M, N, K, ws, 1, 0, counters)


@pytest.mark.parametrize("M", [1, 2, 4])
@pytest.mark.parametrize("N", [1, 16, 17, 1024, 8192, 28672, 1 << 26])
def test_fused_tokens(host, M, N):
    for K in (16, 512, 528, 4096, 8192):
        for ws in (0, 1 << 14, WS):
            got = product(host, M, N, K, ws, 0, 1)
            assert len(got) == 1 and got[0][1]["rows"] == 8 << 52
            check(got, M, N, K, ws, 0, 1)


def test_a_wrong_piece_is_seen(host):
    """The check itself: a piece whose weights are another's, one that is missing, a split that the workspace does not hold."""
    M, N, K = 1 << 20, 1 << 20, 16
    got = product(host, M, N, K, WS, 1)
    assert len(got) > 1
    check(got, M, N, K, WS, 1)
    for change in (lambda g: g.pop(), lambda g: g[1][1].update(W=g[0][1]["W"] + 16), lambda g: g[1][1].update(Y=g[0][1]["Y"]),
                   lambda g: g.append(g[0])):
        wrong = [(n, dict(a)) for n, a in got]
        change(wrong)
        with pytest.raises(AssertionError):
            check(wrong, M, N, K, WS, 1)
    split = product(host, 16, 64, 65536, WS, 1)
    assert split[0][1]["splits"] > 1
    with pytest.raises(AssertionError):
        check(split, 16, 64, 65536, 1024, 1)
