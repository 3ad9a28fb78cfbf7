"""The longest prefix that attention over a shared prefix takes, on the CPU, with
the stand-ins of test_layer_host.py: one part may be all of it, and the kernel
counts a part's tokens, rounded up to whole steps of 64, in 32 bits."""
import ctypes

import pytest

from tests.test_decode_host import BAD, CTX, OK, A, cache, call
from tests.test_layer_host import host  # noqa: F401

LONGEST = 2 ** 31 - 128


@pytest.mark.parametrize("length,status", [(1, OK), (LONGEST, OK), (LONGEST + 1, BAD), (2 ** 31 - 64, BAD), (2 ** 31 - 1, BAD)])
def test_the_longest_prefix(host, length, status):  # noqa: F811
    host.stub_room(64 << 20)
    cc = cache()
    args = dict(ctx=CTX, cache=ctypes.addressof(cc), q=A, stride=4 * 128, B=3, q_heads=4, prefix=1 << 50, plen=length, tables=2 * A, tstride=8,
                twidth=0, lengths=3 * A, max_len=length, window=0, scale=0.1, out=4 * A, odt=0, lse=5 * A, stream=None)
    call(host, "proj_kv_attend_shared", list(args.values()), status, 1 if status == OK else 0)
