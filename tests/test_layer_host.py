"""The argument checks of csrc/layer.cpp's C entry points, on the CPU: built with
stand-ins for the context and the launchers (which keep their arguments), every
refusal is made before anything is launched, and the workspace is cut as the
sizes say."""
import ctypes
import os
import subprocess

import pytest

import dense_linear_projection_amd as dlp
from dense_linear_projection_amd import _build
from tests.test_decode_host import BAD, CTX, NO, OK, A, WRONG_CACHES, cache, call

STUBS = r"""
#include <cstdarg>
#include <cstdio>
#include "context.hpp"
#include "layer.hpp"
using namespace proj;
static int launches = 0;
static char message[512];
static size_t room = 64 << 20;
static RowsArgs rows[64];
static IntArgs products[64];
static int nrows, nproducts;
static AppendArgs appended;
static PrefixArgs shared;
static IntArgs fused;
extern "C" int stub_launches() { return launches; }
extern "C" const char *stub_message() { return message; }
extern "C" void stub_room(int64_t n) { room = n; nrows = nproducts = 0; }
extern "C" int stub_pieces() { return nrows == nproducts ? nrows : -1; }
extern "C" int64_t stub_piece(int i, int what) {
    const RowsArgs &r = rows[i];
    const IntArgs &p = products[i];
    switch (what) {
        case 0: return reinterpret_cast<int64_t>(r.X);
        case 1: return r.M;
        case 2: return reinterpret_cast<int64_t>(r.q);
        case 3: return reinterpret_cast<int64_t>(r.scales);
        case 4: return r.q == p.X && r.scales == p.x_scales && r.M == p.M && r.q_stride == p.K;
        case 5: return reinterpret_cast<int64_t>(p.Y);
        case 6: return reinterpret_cast<int64_t>(p.ws);
        case 7: return p.ws_bytes;
        case 8: return p.K;
    }
    return -1;
}
extern "C" int stub_fused(int64_t X) { return fused.rows == reinterpret_cast<uint16_t *>(X) && fused.rows_stride == 300 && fused.rows_k == 251 && fused.K == 256; }
extern "C" int64_t stub_prefix() { return shared.a.prefix; }
extern "C" int stub_norm() { return (appended.q_norm ? 1 : 0) | (appended.k_norm ? 2 : 0) | appended.norm_f32 * 4 | appended.norm_per_head * 8; }
namespace proj {
proj_status context_view(proj_ctx *c, ContextView *v) {
    if (!c) return PROJ_ERR_INVALID_ARG;
    *v = ContextView{0, 256, reinterpret_cast<float *>(1ll << 40), room};
    return PROJ_OK;
}
proj_status context_error(proj_ctx *, proj_status s, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(message, sizeof message, fmt, ap);
    va_end(ap);
    return s;
}
hipError_t launch_quantize_rows(const RowsArgs &a, hipStream_t) { ++launches; if (nrows < 64) rows[nrows++] = a; return hipSuccess; }
hipError_t launch_int(const IntArgs &a, hipStream_t) { ++launches; if (nproducts < 64) products[nproducts++] = a; return hipSuccess; }
bool int_fuses(int64_t M, int64_t, int64_t) { return M == 99; }
hipError_t launch_int_fused(const IntArgs &a, hipStream_t) { fused = a; ++launches; return hipSuccess; }
hipError_t launch_append(const AppendArgs &a, hipStream_t) { appended = a; ++launches; return hipSuccess; }
hipError_t launch_attend(const AttendArgs &a, hipStream_t) { shared = PrefixArgs{}; shared.a = a; ++launches; return hipSuccess; }
hipError_t launch_attend_shared(const PrefixArgs &p, hipStream_t) {
    if (p.a.ws_bytes < 1000) return hipErrorOutOfMemory;
    shared = p;
    ++launches;
    return hipSuccess;
}
bool attend_dim(int d) { return d == 64 || d == 128; }
}  // namespace proj
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    at = tmp_path_factory.mktemp("layer_host")
    (at / "stubs.cpp").write_text(STUBS)
    objs = []
    for src in (os.path.join(_build.CSRC, "layer.cpp"), str(at / "stubs.cpp")):
        objs.append(str(at / (os.path.basename(src) + ".o")))
        subprocess.run([_build.hipcc()] + _build.FLAGS + ["-I", _build.CSRC, "-x", "hip", "-c", src, "-o", objs[-1]],
                       check=True, capture_output=True)
    so = str(at / "layer_host.so")
    subprocess.run([_build.hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", "-o", so] + objs, check=True,
                   capture_output=True)
    L, real = ctypes.CDLL(so), dlp.lib()
    for name in ("proj_quantize_rows", "proj_run_int", "proj_run_int_dynamic", "proj_kv_append_norm", "proj_kv_attend_shared"):
        getattr(L, name).argtypes, getattr(L, name).restype = getattr(real, name).argtypes, ctypes.c_int
    L.stub_message.restype = ctypes.c_char_p
    L.stub_room.argtypes = [ctypes.c_int64]
    L.stub_piece.restype = L.stub_prefix.restype = ctypes.c_int64
    return L


def test_null_context(host):
    assert host.proj_quantize_rows(None, A, 16, 1, 16, A, 16, A, None) == BAD
    assert host.proj_run_int(None, A, A, A, A, None, 0, 1, 1, 16, A, 0, None) == BAD
    assert host.proj_run_int_dynamic(None, A, 16, A, A, None, 0, 1, 1, 16, A, 0, None) == BAD
    assert host.proj_kv_append_norm(None, None, A, 8, 1, 1, A, A, 0, 0, 0.1, A, 1, 0, 0, A, A, None, None) == BAD
    assert host.proj_kv_attend_shared(None, None, A, 8, 1, 1, A, 1, A, 1, 1, A, 1, 0, 1.0, A, 0, None, None) == BAD


def test_quantize_rows(host):
    ok = dict(ctx=CTX, X=A, xs=1000, M=10, K=1000, q=2 * A, qs=1008, scales=3 * A, stream=None)

    def case(status, launches=0, **kw):
        call(host, "proj_quantize_rows", list({**ok, **kw}.values()), status, launches)

    case(OK, 1)
    case(OK, 1, qs=1024)
    case(OK, 1, xs=1001, X=A + 2)
    case(OK, 1, K=0, qs=0, X=None, q=None)
    case(OK, M=0, X=None, q=None, scales=None)
    for kw in (dict(M=-1), dict(K=-1), dict(xs=999), dict(qs=1000), dict(qs=992), dict(X=None), dict(q=None), dict(scales=None),
               dict(X=A + 1), dict(q=2 * A + 8), dict(scales=3 * A + 2), dict(q=A), dict(scales=A + 2 * 9999 - 2),
               dict(scales=2 * A + 10076)):
        case(BAD, **kw)
    case(NO, M=1 << 40)
    case(NO, M=1 << 30, qs=1 << 14)


INT = dict(ctx=CTX, X=A, xs=2 * A, W=3 * A, ws=4 * A, bias=5 * A, epi=1, M=4, N=64, K=256, Y=6 * A, out=0, stream=None)


def test_run_int(host):
    def case(status, launches=0, **kw):
        call(host, "proj_run_int", list({**INT, **kw}.values()), status, launches)

    case(OK, 1)
    case(OK, 1, bias=None, epi=2)
    case(OK, 1, K=131056, M=1, N=1)
    case(OK, M=0, X=None)
    case(OK, N=0, Y=None)
    case(OK, 1, K=0, X=None, xs=None, W=None, ws=None)
    for kw in (dict(M=-1), dict(N=-1), dict(K=-16), dict(K=24), dict(epi=4), dict(epi=-1), dict(out=2), dict(X=None), dict(xs=None),
               dict(W=None), dict(ws=None), dict(Y=None), dict(bias=None), dict(X=A + 8), dict(xs=2 * A + 2), dict(W=3 * A + 4),
               dict(ws=4 * A + 1), dict(bias=5 * A + 1), dict(Y=6 * A + 2), dict(Y=A), dict(Y=2 * A), dict(Y=3 * A + 64), dict(Y=4 * A + 64),
               dict(Y=5 * A + 64)):
        case(BAD, **kw)
    case(OK, 1, out=1, Y=6 * A + 2)
    for kw in (dict(K=131072), dict(M=1 << 40), dict(N=1 << 40), dict(M=1 << 26, N=1 << 20), dict(M=1 << 30, N=1, K=1 << 16)):
        case(NO, **kw)


def test_run_int_dynamic(host):
    ok = dict(INT)
    ok["xs"] = 300   # the tokens' row stride takes the scales' place

    def case(status, launches=0, **kw):
        call(host, "proj_run_int_dynamic", list({**ok, **kw}.values()), status, launches)

    host.stub_room(64 << 20)
    case(OK, 2)
    case(OK, 2, K=251)
    case(OK, 1, M=99, K=251)
    assert host.stub_fused(ctypes.c_int64(A))
    case(OK, 2, X=A + 2)
    case(OK, 2, K=0, X=None, W=None, ws=None)
    case(OK, M=0, X=None)
    case(OK, N=0, Y=None)
    for kw in (dict(M=-1), dict(N=-1), dict(K=-1), dict(xs=255), dict(epi=4), dict(out=2), dict(X=None), dict(W=None), dict(ws=None),
               dict(Y=None), dict(bias=None), dict(X=A + 1), dict(W=3 * A + 8), dict(ws=4 * A + 2), dict(Y=6 * A + 2), dict(Y=A + 2 * 1000),
               dict(Y=3 * A), dict(Y=4 * A), dict(Y=5 * A)):
        case(BAD, **kw)
    for kw in (dict(K=131072, xs=1 << 20), dict(M=1 << 40), dict(N=1 << 40)):
        case(NO, **kw)
    host.stub_room(512 + 259)
    case(dlp.PROJ_ERR_NO_MEMORY)
    host.stub_room(0)
    case(dlp.PROJ_ERR_NO_MEMORY)


@pytest.mark.parametrize("room", [512 + 1012, 2048, 5000, 12345, 1 << 16, 1 << 20, 64 << 20])
@pytest.mark.parametrize("M,K", [(1, 1000), (7, 1000), (23, 996)])
def test_pieces_of_the_workspace(host, room, M, K):
    """Every row once, in order; integers, scales and what is left of the workspace apart and inside it."""
    host.stub_room(room)
    call(host, "proj_run_int_dynamic", [CTX, A, 1010, 3 * A, 4 * A, None, 0, M, 8, K, 6 * A, 0, None], OK, 2 * _count(host, room, M))
    at, base = 0, 1 << 40
    for i in range(host.stub_pieces()):
        X, rows, q, scales, same, Y, ws, wb, k = (host.stub_piece(i, j) for j in range(9))
        assert same == 1 and k == 1008 and X == A + 2 * at * 1010 and Y == 6 * A + at * 8 * 4
        spans = sorted(((scales, scales + 4 * rows), (q, q + rows * k), (ws, ws + wb)))
        assert spans[0][0] >= base and spans[-1][1] <= base + room
        assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:])) and q % 16 == 0 and ws % 16 == 0
        at += rows
    assert at == M


def _count(host, room, M):
    rows = min(M, (room - 512) // 1012)
    return -(-M // rows)


def test_append_norm(host):
    ok = dict(ctx=CTX, cache=None, qkv=A, stride=8 * 128, T=3, q_heads=4, qn=6 * A, kn=7 * A, ndt=0, per=0, eps=1e-6, rope=2 * A, rows=100,
              rot=128, inter=0, pos=3 * A, slots=4 * A, q=5 * A, stream=None)

    def case(status, launches=0, c=None, **kw):
        cc = cache() if c is None else c
        args = {**ok, "cache": ctypes.addressof(cc), **kw}
        call(host, "proj_kv_append_norm", list(args.values()), status, launches)

    case(OK, 1)
    assert host.stub_norm() == 7
    case(OK, 1, qn=None, ndt=1, per=1)
    assert host.stub_norm() == 2 + 8
    case(OK, 1, kn=None, eps=0.0)
    case(OK, 1, qn=None, kn=None)
    case(OK, 1, q=None)
    case(OK, 1, q_heads=0, stride=512)
    case(OK, 1, rot=0, rope=None)
    case(OK, T=0, qkv=None, pos=None)
    case(BAD, cache=None)
    for status, kw in WRONG_CACHES:
        case(status, c=cache(**kw))
    for kw in (dict(T=-1), dict(q_heads=-1), dict(rot=130), dict(rot=3), dict(rows=-1), dict(stride=7 * 128), dict(qkv=None), dict(pos=None),
               dict(slots=None), dict(rope=None), dict(qkv=A + 2), dict(q=5 * A + 8), dict(q=A + 1024), dict(q=64 * A), dict(rope=64 * A),
               dict(ndt=2), dict(ndt=-1), dict(eps=-1e-9), dict(eps=float("nan")), dict(eps=float("inf")), dict(qn=6 * A + 8), dict(kn=7 * A + 4),
               dict(qn=5 * A), dict(kn=5 * A + 1024), dict(qn=64 * A), dict(kn=128 * A + 4096), dict(qn=5 * A - 1024, per=1)):
        case(BAD, **kw)
    case(OK, 1, qn=5 * A - 512)
    case(NO, T=1 << 40)


def test_attend_shared(host):
    ok = dict(ctx=CTX, cache=None, q=A, stride=4 * 128, B=3, q_heads=4, prefix=6 * A, plen=50, tables=2 * A, tstride=8, twidth=5, lengths=3 * A,
              max_len=130, window=0, scale=0.1, out=4 * A, odt=0, lse=5 * A, stream=None)
    host.stub_room(64 << 20)

    def case(status, launches=0, c=None, **kw):
        cc = cache() if c is None else c
        args = {**ok, "cache": ctypes.addressof(cc), **kw}
        call(host, "proj_kv_attend_shared", list(args.values()), status, launches)

    case(OK, 1)
    assert host.stub_prefix() == 50
    case(OK, 1, plen=0, prefix=None, max_len=80)
    assert host.stub_prefix() == 0
    case(OK, 1, lse=None)
    case(OK, 1, max_len=50, tables=None, twidth=0)
    case(OK, 1, max_len=20, tables=None, twidth=0)
    case(OK, 1, max_len=0, tables=None)
    case(OK, 1, c=cache(pages=0))
    case(OK, B=0, q=None, lengths=None, out=None, prefix=None)
    case(BAD, cache=None)
    for status, kw in WRONG_CACHES:
        case(status, c=cache(**kw))
    for kw in (dict(B=-1), dict(B=1 << 20), dict(q_heads=0), dict(q_heads=3), dict(stride=511), dict(stride=516), dict(tstride=4),
               dict(twidth=-1), dict(max_len=131), dict(max_len=-1), dict(window=-1), dict(scale=float("nan")), dict(odt=2), dict(q=None),
               dict(tables=None), dict(lengths=None), dict(out=None), dict(q=A + 8), dict(tables=2 * A + 2), dict(out=4 * A + 4),
               dict(lse=5 * A + 2), dict(out=A), dict(out=2 * A), dict(out=3 * A - 16), dict(lse=2 * A), dict(out=64 * A), dict(lse=4 * A),
               dict(prefix=None), dict(prefix=6 * A + 2), dict(plen=-1), dict(plen=1 << 31), dict(prefix=4 * A + 64), dict(prefix=5 * A + 4)):
        case(BAD, **kw)
    case(NO, stride=1 << 40)
    host.stub_room(100)
    case(dlp.PROJ_ERR_NO_MEMORY)


def test_names_in_python_need_device_tensors():
    import torch
    t, i8 = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 64, dtype=torch.int8)
    for f in (lambda: dlp.proj_quantize_rows(1, t), lambda: dlp.proj_run_int(1, i8, t, i8, t, None, 0, t),
              lambda: dlp.proj_run_int_dynamic(1, t, i8, t, None, 0, t)):
        with pytest.raises(ValueError, match="must be on a GPU"):
            f()
