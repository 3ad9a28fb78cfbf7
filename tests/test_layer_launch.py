"""What the launchers of a decoding layer's operators ask the runtime for, on the
CPU: the host halves of their sources are linked with stand-ins for the runtime's
launch calls, which refuse what HIP refuses (2^32 threads or more, 2^31
workgroups or more) and keep the rest for inspection. Sizes that the entry points
accept have to be launched, whatever they are, within the workspace."""
import ctypes
import os
import re
import subprocess

import pytest

from dense_linear_projection_amd import _build

SOURCES = ["int8.hip", "prefix.hip", "attend.hip", "kvcache.hip"]
STUBS = r"""
#include <map>
#include <string>
#include <vector>
#include "layer.hpp"
using namespace proj;
struct Launch {
    std::string name;
    dim3 grid, block;
    PrefixArgs prefix;
    AttendArgs attend;
    IntArgs product;
};
static std::vector<Launch> &launches() { static std::vector<Launch> v; return v; }
static std::map<const void *, std::string> &names() { static std::map<const void *, std::string> m; return m; }
static dim3 next_grid, next_block;
static size_t next_lds;
extern "C" {
void **__hipRegisterFatBinary(const void *) { static void *p; return &p; }
void __hipUnregisterFatBinary(void **) {}
void __hipRegisterFunction(void **, const void *f, char *, const char *name, unsigned, void *, void *, void *, void *, int *) {
    names()[f] = name;
}
hipError_t __hipPushCallConfiguration(dim3 g, dim3 b, size_t lds, hipStream_t) {
    next_grid = g, next_block = b, next_lds = lds;
    return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3 *g, dim3 *b, size_t *lds, hipStream_t *st) {
    *g = next_grid, *b = next_block, *lds = next_lds, *st = nullptr;
    return hipSuccess;
}
static hipError_t last = hipSuccess;
hipError_t hipLaunchKernel(const void *f, dim3 g, dim3 b, void **args, size_t lds, hipStream_t) {
    if (g.x == 0 || g.x > 0x7fffffffu || g.y != 1 || g.z != 1 ||
        static_cast<uint64_t>(g.x) * b.x > 0xffffffffull || lds > 160 * 1024)
        return last = hipErrorInvalidConfiguration;
    Launch l{names()[f], g, b, {}, {}, {}};
    if (l.name.find("prefix") != std::string::npos) l.prefix = *static_cast<PrefixArgs *>(args[0]);
    else if (l.name.find("attend") != std::string::npos) l.attend = *static_cast<AttendArgs *>(args[0]);
    else if (l.name.find("int_") != std::string::npos) l.product = *static_cast<IntArgs *>(args[0]);
    launches().push_back(l);
    return hipSuccess;
}
hipError_t hipGetLastError() { hipError_t e = last; last = hipSuccess; return e; }
hipError_t hipFuncSetAttribute(const void *, hipFuncAttribute, int) { return hipSuccess; }

int stub_count() { return static_cast<int>(launches().size()); }
void stub_clear() { launches().clear(); }
const char *stub_name(int i) { return launches()[i].name.c_str(); }
int64_t stub_field(int i, const char *name) {
    const Launch &l = launches()[i];
    const std::string n = name;
    const AttendArgs &a = l.name.find("prefix") != std::string::npos ? l.prefix.a : l.attend;
    if (n == "grid") return l.grid.x;
    if (n == "block") return l.block.x;
    if (n == "q") return reinterpret_cast<int64_t>(a.q);
    if (n == "tables") return reinterpret_cast<int64_t>(a.tables);
    if (n == "lengths") return reinterpret_cast<int64_t>(a.lengths);
    if (n == "out") return reinterpret_cast<int64_t>(a.out);
    if (n == "lse") return reinterpret_cast<int64_t>(a.lse);
    if (n == "B") return a.B;
    if (n == "part") return a.part;
    if (n == "parts") return a.parts;
    if (n == "prefix_parts") return a.prefix_parts;
    if (n == "join") return a.join;
    if (n == "prefix_part") return l.prefix.part;
    if (n == "chunks") return l.prefix.chunks;
    return -1;
}
int stub_rows(int64_t M, int64_t K, int64_t stride) { return launch_quantize_rows(RowsArgs{nullptr, stride, M, K, nullptr, (K + 15) / 16 * 16, nullptr}, nullptr); }
int stub_int(int64_t M, int64_t N, int64_t K, int64_t ws, int f32) {
    return launch_int(IntArgs{nullptr, nullptr, nullptr, nullptr, nullptr, reinterpret_cast<void *>(1 << 20), M, N, K, N, 0, f32 ? OUT_F32 : OUT_BF16,
                              nullptr, static_cast<size_t>(ws), 256, nullptr, 16384}, nullptr);
}
int stub_append(int64_t T, int q_heads, int heads, int dim, int rot) {
    AppendArgs a{};
    a.c.heads = heads, a.c.dim = dim, a.c.pages = 1, a.T = T, a.q_heads = q_heads, a.rot = rot, a.rope_rows = 1;
    a.stride = (q_heads + 2 * heads) * dim, a.q_norm = a.k_norm = &a;
    return launch_append(a, nullptr);
}
int stub_shared(int64_t B, int q_heads, int heads, int dim, int fp8, int64_t prefix, int64_t max_len, int64_t window, int64_t ws, int f32) {
    PrefixArgs p{};
    AttendArgs &a = p.a;
    a.c.pages = 1 << 20, a.c.heads = heads, a.c.dim = dim, a.c.page_shift = 4, a.c.fp8 = fp8;
    a.c.kt = a.c.vt = dim, a.c.kh = a.c.vh = 16 * dim, a.c.kp = a.c.vp = 16 * dim * heads;
    a.q = reinterpret_cast<uint16_t *>(1ll << 40), a.q_stride = q_heads * dim + 64, a.B = B, a.q_heads = q_heads;
    a.tables = reinterpret_cast<int32_t *>(2ll << 40), a.table_stride = 77;
    a.lengths = reinterpret_cast<int32_t *>(3ll << 40);
    a.max_len = max_len, a.window = window, a.scale = 1.f, a.prefix = prefix;
    a.out = reinterpret_cast<void *>(4ll << 40), a.out_dtype = f32 ? OUT_F32 : OUT_BF16;
    a.lse = reinterpret_cast<float *>(5ll << 40);
    a.ws_bytes = ws, a.cus = 256, a.ncounters = 16384;
    return launch_attend_shared(p, nullptr);
}
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    at = tmp_path_factory.mktemp("layer_launch")
    (at / "stubs.cpp").write_text(STUBS)
    flags = ["--offload-arch=gfx950", "--cuda-host-only", "-O1", "-std=c++17", "-fPIC", "-I", _build.CSRC, "-x", "hip"]
    objs, procs = [], []
    for src in [os.path.join(_build.CSRC, s) for s in SOURCES] + [str(at / "stubs.cpp")]:
        objs.append(str(at / (os.path.basename(src) + ".o")))
        procs.append(subprocess.Popen([_build.hipcc()] + flags + ["-c", src, "-o", objs[-1]], stderr=subprocess.PIPE, text=True))
    for p in procs:
        err = p.communicate()[1]
        assert p.returncode == 0, err
    # the device code that a host half refers to by a name of its own, nowhere read
    names = set(re.findall(r"__hip_fatbin_\w+", subprocess.run(["nm", "-u"] + objs, check=True, capture_output=True, text=True).stdout))
    (at / "fatbin.c").write_text("".join("const char %s[16] = {0};\n" % n for n in sorted(names)))
    so = str(at / "layer_launch.so")
    subprocess.run(["gcc", "-fPIC", "-c", str(at / "fatbin.c"), "-o", str(at / "fatbin.o")], check=True)
    subprocess.run(["g++", "-shared", "-Wl,-Bsymbolic", "-o", so, str(at / "fatbin.o")] + objs, check=True)
    L = ctypes.CDLL(so)
    i64, ci = ctypes.c_int64, ctypes.c_int
    L.stub_name.restype = ctypes.c_char_p
    L.stub_field.argtypes, L.stub_field.restype = [ci, ctypes.c_char_p], i64
    L.stub_rows.argtypes = [i64, i64, i64]
    L.stub_int.argtypes = [i64, i64, i64, i64, ci]
    L.stub_append.argtypes = [i64, ci, ci, ci, ci]
    L.stub_shared.argtypes = [i64, ci, ci, ci, ci, i64, i64, i64, i64, ci]
    return L


def launched(host, status, name, *args):
    """The launches of one call: (kernel name, field reader) each."""
    host.stub_clear()
    assert getattr(host, name)(*args) == status, (name, args)
    return [(host.stub_name(i).decode(), lambda f, i=i: host.stub_field(i, f.encode())) for i in range(host.stub_count())]


WS = 64 << 20
OUT_OF_MEMORY = 2   # hipErrorOutOfMemory


@pytest.mark.parametrize("M,K", [(1, 1), (1, 1 << 26), (1 << 33, 16), (1 << 30, 1000), (16, 8192), (4096, 8192), (1, 0)])
def test_rows_of_any_number(host, M, K):
    for stride in (K, K + 1, (K + 7) // 8 * 8):
        assert len(launched(host, 0, "stub_rows", M, K, stride)) == 1


@pytest.mark.parametrize("M", [1, 8, 16, 17, 32, 33, 64, 65, 128, 129, 256, 257, 512, 4096, 1 << 20, 1 << 33])
@pytest.mark.parametrize("N", [1, 64, 1000, 28672, (1 << 28) + 1, 1 << 33])
@pytest.mark.parametrize("ws", [0, 1 << 16, WS])
def test_products_of_any_size(host, M, N, ws):
    for K in (0, 16, 128, 8192, 131056):
        if M * N <= 1 << 40 and M * K <= 1 << 40 and N * K <= 1 << 40:
            for f32 in (0, 1):
                assert len(launched(host, 0, "stub_int", M, N, K, ws, f32)) >= 1


@pytest.mark.parametrize("T,q_heads,heads,dim,rot", [(1, 4, 1, 64, 64), (8192, 64, 8, 128, 128), ((1 << 26) + 3, 0, 1, 80, 80),
                                                     ((1 << 27) + 5, 0, 1, 64, 34), (1 << 27, 1, 1, 192, 0)])
def test_append_of_any_length(host, T, q_heads, heads, dim, rot):
    assert len(launched(host, 0, "stub_append", T, q_heads, heads, dim, rot)) >= 1


@pytest.mark.parametrize("B,q_heads,heads,dim", [(1, 1, 1, 64), (1, 8, 1, 128), (4, 32, 8, 128), (64, 64, 8, 128), (256, 64, 8, 80),
                                                 (4096, 32, 32, 256), (32767, 32, 8, 128), (20000, 1024, 1024, 64), (300, 65536, 512, 64),
                                                 (1, 65536, 65536, 192), (1, 65536, 1, 64)])
@pytest.mark.parametrize("prefix,own", [(1, 0), (1, 1), (500, 100), (8192, 1000), (131072, 1), (2000000000, 100000000), (33, 131072)])
@pytest.mark.parametrize("ws", [WS, 1 << 42])
def test_attention_of_any_batch(host, B, q_heads, heads, dim, prefix, own, ws):
    """Launches together take every sequence once, each with the addresses of its first; the parts cover prefix and bound,
    and the workspace holds them."""
    row, at = q_heads * (dim + 4) * 4, 0
    if 2 * row > ws:
        assert launched(host, OUT_OF_MEMORY, "stub_shared", 1, q_heads, heads, dim, 0, prefix, prefix + own, 0, ws, 1) == []
        return
    got = launched(host, 0, "stub_shared", B, q_heads, heads, dim, B % 2, prefix, prefix + own, 0, ws, 1)
    seen = {}
    for name, f in got:
        if "prefix_kernel" in name:
            assert f("q") == (1 << 40) + 2 * at * (q_heads * dim + 64) and f("tables") == (2 << 40) + 4 * at * 77
            assert f("lengths") == (3 << 40) + 4 * at and f("out") == (4 << 40) + 4 * at * q_heads * dim
            assert f("lse") == (5 << 40) + 4 * at * q_heads
            rows = f("B") * (q_heads // heads)
            assert f("chunks") * 128 >= rows and f("block") == 256
            parts = f("prefix_parts")
            assert parts * f("prefix_part") >= prefix and (parts - 1) * f("prefix_part") < prefix
            assert f("grid") >= heads * parts * f("chunks")
            assert f("parts") * f("part") >= own and (own == 0) == (f("parts") == 0)
            assert f("B") * row * (f("parts") + f("prefix_parts")) <= ws
            seen = {x: f(x) for x in ("B", "parts", "prefix_parts", "part", "q")}
            at += f("B")
        else:
            assert all(f(x) == seen[x] for x in seen)       # the own tokens' parts, and the join
            assert f("join") == 0
            assert f("grid") >= (f("B") * q_heads if "join" in name else f("B") * f("parts") * heads)
    assert at == B
