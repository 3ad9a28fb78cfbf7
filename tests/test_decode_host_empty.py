"""A paged cache without pages has no memory: its pointers may be null, on the
CPU with the stand-ins of the other argument checks."""
import ctypes

from tests.test_decode_host import A, BAD, CTX, OK, cache, call, host  # noqa: F401


def test_null_pointers_of_an_empty_cache(host):  # noqa: F811
    for pages, status, launches in ((0, OK, 1), (1, BAD, 0)):
        for kw in (dict(k=None), dict(v=None), dict(k=None, v=None)):
            c = ctypes.addressof(keep := cache(pages=pages, **kw))
            call(host, "proj_kv_append", [CTX, c, A, 8 * 128, 3, 4, 2 * A, 100, 128, 0, 3 * A, 4 * A, 5 * A, None], status, launches)
            call(host, "proj_kv_attend", [CTX, c, A, 4 * 128, 3, 4, 2 * A, 8, 5, 3 * A, 80, 0, 0.1, 4 * A, 0, 5 * A, None], status,
                 launches)
            del keep
    c = cache(pages=0, k=8, v=None)
    call(host, "proj_kv_append", [CTX, ctypes.addressof(c), A, 8 * 128, 3, 4, 2 * A, 100, 128, 0, 3 * A, 4 * A, 5 * A, None], BAD, 0)
