"""The argument checks of the decoding operators' C entry points, on the CPU:
csrc/decode.cpp is built with stand-ins for the context and the launchers (a
launcher counts its calls and keeps the arguments), and every refusal is made
before anything is launched."""
import ctypes
import os
import subprocess

import pytest

import dense_linear_projection_amd as dlp
from dense_linear_projection_amd import _build

STUBS = r"""
#include <cstdarg>
#include <cstdio>
#include "context.hpp"
#include "decode.hpp"
static int launches = 0;
static char message[512];
static proj::AttendArgs attended;
extern "C" int stub_launches() { return launches; }
extern "C" const char *stub_message() { return message; }
extern "C" int stub_page_shift() { return attended.c.page_shift; }
namespace proj {
proj_status context_view(proj_ctx *c, ContextView *v) {
    if (!c) return PROJ_ERR_INVALID_ARG;
    *v = ContextView{0, 256, nullptr, 0};
    return PROJ_OK;
}
proj_status context_error(proj_ctx *, proj_status s, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(message, sizeof message, fmt, ap);
    va_end(ap);
    return s;
}
hipError_t launch_quant(const QuantArgs &, hipStream_t) { ++launches; return hipSuccess; }
hipError_t launch_pack_codes(const uint8_t *, int64_t, int64_t, uint32_t *, hipStream_t) { ++launches; return hipSuccess; }
hipError_t launch_quantize(const uint16_t *, int64_t, int64_t, int, uint32_t *, void *, int, uint8_t *, hipStream_t) {
    ++launches;
    return hipSuccess;
}
hipError_t launch_append(const AppendArgs &, hipStream_t) { ++launches; return hipSuccess; }
hipError_t launch_attend(const AttendArgs &a, hipStream_t) { attended = a; ++launches; return hipSuccess; }
bool attend_dim(int d) { return d == 64 || d == 128; }
}  // namespace proj
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    at = tmp_path_factory.mktemp("decode_host")
    (at / "stubs.cpp").write_text(STUBS)
    objs = []
    for src in (os.path.join(_build.CSRC, "decode.cpp"), str(at / "stubs.cpp")):
        objs.append(str(at / (os.path.basename(src) + ".o")))
        subprocess.run([_build.hipcc()] + _build.FLAGS + ["-I", _build.CSRC, "-x", "hip", "-c", src, "-o", objs[-1]],
                       check=True, capture_output=True)
    so = str(at / "decode_host.so")
    subprocess.run([_build.hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", "-o", so] + objs, check=True,
                   capture_output=True)
    L, real = ctypes.CDLL(so), dlp.lib()
    for name in ("proj_pack_codes", "proj_quantize_weights", "proj_run_quant", "proj_kv_append", "proj_kv_attend"):
        getattr(L, name).argtypes, getattr(L, name).restype = getattr(real, name).argtypes, ctypes.c_int
    L.stub_message.restype = ctypes.c_char_p
    return L


CTX = 1      # any handle that is not NULL
OK, BAD, NO = dlp.PROJ_OK, dlp.PROJ_ERR_INVALID_ARG, dlp.PROJ_ERR_UNSUPPORTED
A = 1 << 20  # distinct, aligned addresses that nothing reads


def call(host, name, args, status, launches):
    before = host.stub_launches()
    assert getattr(host, name)(*args) == status, host.stub_message()
    assert host.stub_launches() - before == launches


def test_null_context(host):
    z = [None] * 3
    assert host.proj_pack_codes(None, A, 1, 8, A, None) == BAD
    assert host.proj_quantize_weights(None, A, 1, 8, 32, A, A, 0, None, None) == BAD
    assert host.proj_run_quant(None, A, A, A, 0, None, 32, None, 0, 1, 1, 8, A, 0, None) == BAD
    assert host.proj_kv_append(None, None, A, 8, 1, 1, A, 1, 0, 0, A, A, *z[:2]) == BAD
    assert host.proj_kv_attend(None, None, A, 8, 1, 1, A, 1, 1, A, 1, 0, 1.0, A, 0, None, None) == BAD


def test_quant(host):
    ok = dict(ctx=CTX, X=A, codes=2 * A, scales=3 * A, sdt=0, zeros=4 * A, group=128, bias=5 * A, epi=1, M=4, N=64, K=256,
              Y=6 * A, out=0, stream=None)

    def case(status, launches=0, **kw):
        call(host, "proj_run_quant", list({**ok, **kw}.values()), status, launches)

    case(OK, 1)
    case(OK, 1, zeros=None)
    case(OK, 1, bias=None, epi=2)
    case(OK, M=0, X=None)
    case(OK, N=0, Y=None)
    case(OK, 1, K=0, X=None, codes=None, scales=None)
    for kw in (dict(M=-1), dict(N=-1), dict(K=-8), dict(K=12), dict(group=0), dict(group=256), dict(epi=4), dict(epi=-1),
               dict(out=2), dict(sdt=2), dict(X=None), dict(codes=None), dict(scales=None), dict(Y=None), dict(bias=None),
               dict(X=A + 1), dict(codes=2 * A + 2), dict(scales=3 * A + 2), dict(Y=6 * A + 2), dict(Y=A), dict(Y=2 * A + 64),
               dict(Y=3 * A), dict(Y=4 * A + 64), dict(Y=5 * A + 64)):
        case(BAD, **kw)
    case(OK, 1, sdt=1, scales=3 * A + 2)
    case(NO, N=1 << 40, K=1 << 10)
    case(NO, M=1 << 40)


def test_registration(host):
    call(host, "proj_pack_codes", [CTX, A, 4, 64, 2 * A, None], OK, 1)
    call(host, "proj_pack_codes", [CTX, None, 0, 64, None, None], OK, 0)
    for args in ([CTX, A, 4, 60, 2 * A, None], [CTX, A, -4, 64, 2 * A, None], [CTX, None, 4, 64, 2 * A, None],
                 [CTX, A, 4, 64, 2 * A + 1, None], [CTX, A, 4, 64, A + 4, None]):
        call(host, "proj_pack_codes", args, BAD, 0)
    ok = [CTX, A, 4, 64, 32, 2 * A, 3 * A, 1, 4 * A, None]
    call(host, "proj_quantize_weights", ok, OK, 1)
    call(host, "proj_quantize_weights", ok[:8] + [None, None], OK, 1)
    for i, v in ((1, None), (2, -1), (3, 60), (4, 48), (5, None), (6, None), (7, 5), (8, 3 * A), (5, A), (6, 3 * A + 1)):
        call(host, "proj_quantize_weights", ok[:i] + [v] + ok[i + 1:], BAD, 0)


def cache(**kw):
    f = dict(k=64 * A, v=128 * A, dtype=dlp.KV_BF16, heads=2, head_dim=128, page_size=16, pages=10,
             k_strides=(2 * 16 * 128, 16 * 128, 128), v_strides=(2 * 16 * 128, 16 * 128, 128), k_scale=1.0, v_scale=1.0)
    f.update(kw)
    s3 = ctypes.c_int64 * 3
    f["k_strides"], f["v_strides"] = s3(*f["k_strides"]), s3(*f["v_strides"])
    return dlp._KvCache(*f.values())


WRONG_CACHES = [(BAD, dict(dtype=2)), (BAD, dict(heads=0)), (BAD, dict(pages=-1)), (BAD, dict(page_size=0)),
                (BAD, dict(page_size=12)), (BAD, dict(page_size=1 << 21)), (NO, dict(head_dim=72)), (NO, dict(head_dim=0)),
                (BAD, dict(k=None)), (BAD, dict(v=None)), (BAD, dict(k=64 * A + 8)), (BAD, dict(k_strides=(4096, 2048, 100))),
                (BAD, dict(v_strides=(4096, 0, 128))), (BAD, dict(v_strides=(-4096, 2048, 128))),
                (BAD, dict(dtype=dlp.KV_FP8, k_strides=(4096, 2048, 136))), (BAD, dict(k_scale=0.5)),
                (BAD, dict(dtype=dlp.KV_FP8, v_scale=0.0)), (BAD, dict(dtype=dlp.KV_FP8, k_scale=float("nan"))),
                (BAD, dict(dtype=dlp.KV_FP8, k_scale=float("inf"))), (NO, dict(k_strides=(1 << 40, 2048, 128))),
                (NO, dict(pages=1 << 31))]


def test_append(host):
    ok = dict(ctx=CTX, cache=None, qkv=A, stride=8 * 128, T=3, q_heads=4, rope=2 * A, rows=100, rot=128, inter=0, pos=3 * A,
              slots=4 * A, q=5 * A, stream=None)

    def case(status, launches=0, c=None, **kw):
        cc = cache() if c is None else c
        args = {**ok, "cache": ctypes.addressof(cc), **kw}
        call(host, "proj_kv_append", list(args.values()), status, launches)

    case(OK, 1)
    case(OK, 1, q=None)
    case(OK, 1, q_heads=0, stride=512)
    case(OK, 1, rot=0, rope=None)
    case(OK, 1, c=cache(pages=0))
    case(OK, T=0, qkv=None, pos=None)
    case(BAD, cache=None)
    for status, kw in WRONG_CACHES:
        case(status, c=cache(**kw))
    for kw in (dict(T=-1), dict(q_heads=-1), dict(rot=130), dict(rot=3), dict(rot=-2), dict(rows=-1), dict(stride=7 * 128),
               dict(stride=8 * 128 + 4), dict(qkv=None), dict(pos=None), dict(slots=None), dict(rope=None), dict(qkv=A + 2),
               dict(q=5 * A + 8), dict(slots=4 * A + 4), dict(q=A + 1024), dict(q=64 * A), dict(q=128 * A + 4096),
               dict(qkv=64 * A + 4096), dict(q=2 * A), dict(q=3 * A - 16), dict(q=4 * A - 16), dict(rope=64 * A)):
        case(BAD, **kw)
    case(NO, T=1 << 40)


def test_attend(host):
    ok = dict(ctx=CTX, cache=None, q=A, stride=4 * 128, B=3, q_heads=4, tables=2 * A, tstride=8, twidth=5, lengths=3 * A,
              max_len=80, window=0, scale=0.1, out=4 * A, odt=0, lse=5 * A, stream=None)

    def case(status, launches=0, c=None, **kw):
        cc = cache() if c is None else c
        args = {**ok, "cache": ctypes.addressof(cc), **kw}
        call(host, "proj_kv_attend", list(args.values()), status, launches)

    case(OK, 1)
    assert host.stub_page_shift() == 4
    case(OK, 1, lse=None)
    case(OK, 1, max_len=0, tables=None)
    case(OK, 1, c=cache(pages=0))
    case(OK, B=0, q=None, lengths=None, out=None)
    case(BAD, cache=None)
    for status, kw in WRONG_CACHES:
        case(status, c=cache(**kw))
    for kw in (dict(B=-1), dict(B=1 << 20), dict(q_heads=0), dict(q_heads=3), dict(stride=511), dict(stride=516), dict(tstride=4),
               dict(twidth=-1), dict(max_len=81), dict(max_len=-1), dict(window=-1), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(odt=2), dict(q=None), dict(tables=None), dict(lengths=None), dict(out=None),
               dict(q=A + 8), dict(tables=2 * A + 2), dict(out=4 * A + 4), dict(lse=5 * A + 2), dict(out=A), dict(out=2 * A),
               dict(out=3 * A - 16), dict(lse=2 * A), dict(out=64 * A), dict(lse=128 * A), dict(lse=4 * A)):
        case(BAD, **kw)
    case(NO, stride=1 << 40)


def test_names_in_python_need_device_tensors():
    import torch
    t = torch.zeros(4, 64, dtype=torch.bfloat16)
    for f in (lambda: dlp.proj_run_quant(1, t, t, t, None, 32, None, 0, t), lambda: dlp.proj_quantize_weights(1, t, 32),
              lambda: dlp.proj_pack_codes(1, t), lambda: dlp.kv_cache(t, t)):
        with pytest.raises(ValueError, match="must be on a GPU"):
            f()
