"""What the decoding operators' launchers ask the runtime for, on the CPU: the
host halves of their sources are linked with stand-ins for the runtime's
launch calls, which refuse what HIP refuses (2^32 threads or more, 2^31
workgroups or more) and keep the rest for inspection.  Sizes that the entry
points accept have to be launched, whatever they are."""
import ctypes
import os
import re
import subprocess

import pytest

from dense_linear_projection_amd import _build

SOURCES = ["quant.hip", "kvcache.hip", "attend.hip"]
STUBS = r"""
#include <map>
#include <string>
#include <vector>
#include "decode.hpp"
#include "kernels.hpp"
using namespace proj;
struct Launch {
    std::string name;
    dim3 grid, block;
    size_t lds;
    QuantArgs quant;
    AppendArgs append;
    AttendArgs attend;
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
    Launch l{names()[f], g, b, lds, {}, {}, {}};
    if (l.name.find("append") != std::string::npos) l.append = *static_cast<AppendArgs *>(args[0]);
    else if (l.name.find("attend") != std::string::npos) l.attend = *static_cast<AttendArgs *>(args[0]);
    else if (l.name.find("quant_") != std::string::npos) l.quant = *static_cast<QuantArgs *>(args[0]);
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
    if (n == "grid") return l.grid.x;
    if (n == "block") return l.block.x;
    if (n == "qkv") return reinterpret_cast<int64_t>(l.append.qkv);
    if (n == "positions") return reinterpret_cast<int64_t>(l.append.positions);
    if (n == "slots") return reinterpret_cast<int64_t>(l.append.slots);
    if (n == "q_out") return reinterpret_cast<int64_t>(l.append.q_out);
    if (n == "T") return l.append.T;
    if (n == "q") return reinterpret_cast<int64_t>(l.attend.q);
    if (n == "tables") return reinterpret_cast<int64_t>(l.attend.tables);
    if (n == "lengths") return reinterpret_cast<int64_t>(l.attend.lengths);
    if (n == "out") return reinterpret_cast<int64_t>(l.attend.out);
    if (n == "lse") return reinterpret_cast<int64_t>(l.attend.lse);
    if (n == "B") return l.attend.B;
    if (n == "part") return l.attend.part;
    if (n == "parts") return l.attend.parts;
    if (n == "chunks") return l.attend.chunks;
    if (n == "by_die") return l.attend.by_die;
    if (n == "join") return l.attend.join;
    return -1;
}
int stub_quant(int64_t X, int64_t M, int64_t N, int64_t K, int group, int zeros, int f32, int64_t ws) {
    QuantArgs a{};
    a.X = reinterpret_cast<uint16_t *>(X);
    a.codes = reinterpret_cast<uint32_t *>(1 << 20);
    a.scales = reinterpret_cast<void *>(2 << 20);
    a.zeros = zeros ? reinterpret_cast<uint8_t *>(3 << 20) : nullptr;
    a.M = M, a.N = N, a.K = K, a.G = (K + group - 1) / group;
    a.group = group, a.scales_f32 = f32, a.cus = 256, a.ws_bytes = ws;
    return launch_quant(a, nullptr);
}
int stub_pack(int64_t N, int64_t K) { return launch_pack_codes(nullptr, N, K, nullptr, nullptr); }
int stub_quantize(int64_t N, int64_t K, int group) {
    return launch_quantize(nullptr, N, K, group, nullptr, nullptr, 0, nullptr, nullptr);
}
static CacheArgs cache(int heads, int dim, int page_shift, int64_t token_stride, int fp8) {
    CacheArgs c{};
    c.pages = 1 << 20, c.heads = heads, c.dim = dim, c.page_shift = page_shift, c.fp8 = fp8;
    c.kt = c.vt = token_stride, c.kh = c.vh = 1 << 16, c.kp = c.vp = 1 << 24;
    return c;
}
int stub_append(int64_t T, int64_t stride, int q_heads, int heads, int dim, int rot, int interleaved) {
    AppendArgs a{};
    a.c = cache(heads, dim, 4, dim, 0);
    a.qkv = reinterpret_cast<uint16_t *>(1ll << 40), a.stride = stride, a.T = T;
    a.q_heads = q_heads, a.rot = rot, a.interleaved = interleaved, a.rope_rows = 1;
    a.positions = reinterpret_cast<int32_t *>(2ll << 40), a.slots = reinterpret_cast<int64_t *>(3ll << 40);
    a.q_out = q_heads ? reinterpret_cast<uint16_t *>(4ll << 40) : nullptr;
    return launch_append(a, nullptr);
}
int stub_attend(int64_t B, int q_heads, int heads, int dim, int64_t token_stride, int fp8, int64_t max_len, int64_t window,
                int64_t ws, int f32, int lse) {
    AttendArgs a{};
    a.c = cache(heads, dim, 4, token_stride, fp8);
    a.q = reinterpret_cast<uint16_t *>(1ll << 40), a.q_stride = q_heads * dim + 64, a.B = B, a.q_heads = q_heads;
    a.tables = reinterpret_cast<int32_t *>(2ll << 40), a.table_stride = max_len / 16 + 5;
    a.lengths = reinterpret_cast<int32_t *>(3ll << 40);
    a.max_len = max_len, a.window = window, a.scale = 1.f;
    a.out = reinterpret_cast<void *>(4ll << 40), a.out_dtype = f32 ? OUT_F32 : OUT_BF16;
    a.lse = lse ? reinterpret_cast<float *>(5ll << 40) : nullptr;
    a.ws_bytes = ws, a.cus = 256, a.ncounters = 16384;
    return launch_attend(a, nullptr);
}
}
namespace proj {
hipError_t launch_splitk_reduce(const Args &, int, hipStream_t) { return hipSuccess; }
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    at = tmp_path_factory.mktemp("decode_launch")
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
    so = str(at / "decode_launch.so")
    subprocess.run(["gcc", "-fPIC", "-c", str(at / "fatbin.c"), "-o", str(at / "fatbin.o")], check=True)
    subprocess.run(["g++", "-shared", "-Wl,-Bsymbolic", "-o", so, str(at / "fatbin.o")] + objs, check=True)
    L = ctypes.CDLL(so)
    i64, ci = ctypes.c_int64, ctypes.c_int
    L.stub_name.restype = ctypes.c_char_p
    L.stub_field.argtypes, L.stub_field.restype = [ci, ctypes.c_char_p], i64
    L.stub_quant.argtypes = [i64, i64, i64, i64, ci, ci, ci, i64]
    L.stub_pack.argtypes = [i64, i64]
    L.stub_quantize.argtypes = [i64, i64, ci]
    L.stub_append.argtypes = [i64, i64, ci, ci, ci, ci, ci]
    L.stub_attend.argtypes = [i64, ci, ci, ci, i64, ci, i64, i64, i64, ci, ci]
    return L


def launched(host, name, *args):
    """The launches of one call that succeeds: (kernel name, field reader) each."""
    host.stub_clear()
    assert getattr(host, name)(*args) == 0, (name, args)
    return [(host.stub_name(i).decode(), lambda f, i=i: host.stub_field(i, f.encode())) for i in range(host.stub_count())]


ALIGNED, ODD = 4 << 20, (4 << 20) + 2
WS = 64 << 20


@pytest.mark.parametrize("M,N", [(1, 64), (4096, 16383), (4096, 16384), (8192, 8192), (8192, 262144), (1 << 20, 1 << 19)])
def test_projection_of_unaligned_rows(host, M, N):
    (kernel,) = launched(host, "stub_quant", ODD, M, N, 64, 32, 1, 0, WS)
    assert "quant_rows_kernel" in kernel[0]


@pytest.mark.parametrize("M", [1, 16, 17, 32, 33, 64, 200, 5000])
@pytest.mark.parametrize("N", [1, 64, 28672, (1 << 28) - 1, (1 << 28) + 1, (1 << 30) + 1, 1 << 33])
def test_projection_of_any_width(host, M, N):
    for K in (8, 128):
        if N * K <= 1 << 40 and M * N <= 1 << 40:
            assert len(launched(host, "stub_quant", ALIGNED, M, N, K, 128, 0, 0, WS)) >= 1


@pytest.mark.parametrize("N,K", [(1, 8), (1 << 26, 8), (262144, 8192), (1 << 33, 8), (1 << 22, 1 << 18)])
def test_registration_of_any_size(host, N, K):
    assert len(launched(host, "stub_quantize", N, K, 32)) == 1
    assert len(launched(host, "stub_pack", N, K)) == 1


@pytest.mark.parametrize("T,q_heads,heads,dim,rot", [(1, 4, 1, 64, 64), (8192, 64, 8, 128, 128), ((1 << 26) + 3, 0, 1, 64, 64),
                                                     ((1 << 27) + 5, 0, 1, 64, 34), (1 << 27, 1, 1, 64, 0)])
def test_append_of_any_length(host, T, q_heads, heads, dim, rot):
    """Launches together take every token once, each with the addresses of its first."""
    stride, at = (q_heads + 2 * heads) * dim + 8, 0
    for _, f in launched(host, "stub_append", T, stride, q_heads, heads, dim, rot, 0):
        assert f("qkv") == (1 << 40) + 2 * at * stride and f("positions") == (2 << 40) + 4 * at
        assert f("slots") == (3 << 40) + 8 * at
        assert f("q_out") == ((4 << 40) + 2 * at * q_heads * dim if q_heads else 0)
        at += f("T")
    assert at == T


@pytest.mark.parametrize("B,q_heads,heads,dim", [(1, 8, 1, 128), (32, 64, 8, 128), (4096, 32, 32, 128), (32767, 32, 8, 128),
                                                 (20000, 1024, 1024, 64), (32767, 65536, 512, 64), (1, 65536, 65536, 256)])
@pytest.mark.parametrize("max_len", [1, 500, 131072, (1 << 31) - 1])
@pytest.mark.parametrize("ws", [0, WS, 1 << 42])
@pytest.mark.parametrize("mixed", [0, 1])
def test_attention_of_any_batch(host, B, q_heads, heads, dim, max_len, ws, mixed):
    """Launches together take every sequence once, each with the addresses of its first; its parts cover the bound."""
    at = 0
    for name, f in launched(host, "stub_attend", B, q_heads, heads, dim, dim * (heads if mixed else 1), 0, max_len, 0, ws, 1, 1):
        if "join" in name:
            assert f("B") == before["B"] and f("grid") == f("B") * q_heads
            continue
        assert f("q") == (1 << 40) + 2 * at * (q_heads * dim + 64) and f("tables") == (2 << 40) + 4 * at * (max_len // 16 + 5)
        assert f("lengths") == (3 << 40) + 4 * at and f("out") == (4 << 40) + 4 * at * q_heads * dim
        assert f("lse") == (5 << 40) + 4 * at * q_heads
        groups = f("B") * f("parts")
        assert f("grid") >= groups * heads * f("chunks") and f("parts") * f("part") >= max_len
        assert f("parts") == 1 or groups * q_heads * (dim + 4) * 4 <= ws
        before = {"B": f("B")}
        at += f("B")
    assert at == B
