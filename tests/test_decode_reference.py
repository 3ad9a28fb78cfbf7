"""The plain forms that the decoding operators are tested against, pinned by
hand-worked values and by a second, differently written form; and the test
that they would notice a wrong kernel (a mistake planted in a copy)."""
import math

import pytest
import torch

from tests import decode_reference as ref


def test_code_layout():
    q = torch.tensor([[1, 2, 3, 4, 5, 6, 7, 8]])
    # pairs (1,2) (3,4) (5,6) (7,8): first of each in the low half, second in the high half
    assert ref.pack(q).tolist() == [[0x86427531 - 2 ** 32]]
    q = torch.randint(0, 16, (5, 48))
    assert torch.equal(ref.unpack(ref.pack(q)), q)


def test_quant_by_hand():
    q = torch.tensor([[9, 8, 7, 0, 15, 8, 8, 8]])
    X = torch.tensor([[1., 2., 3., 4., 5., 6., 7., 8.]]).bfloat16()
    s = torch.tensor([[0.5]]).bfloat16()
    y, tol = ref.quant(X, ref.pack(q), s, None, 32, None, 0, torch.float32)
    assert y.tolist() == [[0.5 * (1 - 3 - 32 + 35)]]
    y, _ = ref.quant(X, ref.pack(q), s, torch.tensor([[0]], dtype=torch.uint8), 32, torch.ones(1).bfloat16(), 1, torch.float32)
    assert y.tolist() == [[0.5 * (9 + 16 + 21 + 75 + 48 + 56 + 64) + 1]]


def test_quant_notices_swapped_pairs():
    torch.manual_seed(0)
    q = torch.randint(0, 16, (8, 256))
    X, s = torch.randn(4, 256).bfloat16(), (torch.rand(8, 2) + 0.5).float()
    y, tol = ref.quant(X, ref.pack(q), s, None, 128, None, 0, torch.float32)
    swapped = q.reshape(8, -1, 2).flip(-1).reshape(8, -1)
    z, _ = ref.quant(X, ref.pack(swapped), s, None, 128, None, 0, torch.float32)
    ref.close(y, y, tol)
    with pytest.raises(AssertionError):
        ref.close(z, y, tol)
    with pytest.raises(AssertionError):
        ref.close(y * (1 + 1e-4), y, tol)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_length_and_composes(interleaved):
    torch.manual_seed(1)
    x = torch.randn(3, 2, 80).double()
    a, b = torch.rand(3, 1, 16).double(), torch.rand(3, 1, 16).double()
    one = ref.rotate(ref.rotate(x, a.cos(), a.sin(), 32, interleaved), b.cos(), b.sin(), 32, interleaved)
    two = ref.rotate(x, (a + b).cos(), (a + b).sin(), 32, interleaved)
    assert torch.allclose(one, two, atol=1e-12)
    assert torch.allclose(one.norm(dim=-1), x.norm(dim=-1))
    assert torch.equal(one[..., 32:], x[..., 32:])


def test_append_places_tokens():
    k, v = torch.zeros(2, 1, 4, 64).bfloat16(), torch.zeros(2, 1, 4, 64).bfloat16()
    qkv = torch.randn(3, 3 * 64).bfloat16()
    rope = torch.cat((torch.ones(5, 32), torch.zeros(5, 32)), 1)
    (q, kk, vv), _ = ref.append(k, v, qkv, rope, torch.tensor([0, 4, 5]), torch.tensor([5, -1, 0]), 1, (1., 1.), False)
    assert torch.equal(q[0, 0], qkv[0, :64].double()) and torch.equal(q[1, 0], qkv[1, :64].double())
    assert torch.isnan(q[2]).all()                       # position 5 is not in the table
    assert torch.equal(kk[1, 0, 1], qkv[0, 64:128].double()) and torch.equal(vv[1, 0, 1], qkv[0, 128:].double())
    assert kk.abs().sum() == kk[1, 0, 1].abs().sum()      # nothing else was stored


def test_attend_by_hand():
    k, v = torch.zeros(1, 1, 4, 64).bfloat16(), torch.zeros(1, 1, 4, 64).bfloat16()
    k[0, 0, 1, 0], v[0, 0, 0], v[0, 0, 1], v[0, 0, 2] = 1, 1, 2, float("nan")
    q = torch.zeros(1, 1, 64).bfloat16()
    q[0, 0, 0] = 2
    (o, lse), _ = ref.attend(k, v, q, torch.zeros(1, 1, dtype=torch.int32), torch.tensor([2]), 0.5, 0, (1., 1.), torch.float32)
    e = math.e
    assert torch.allclose(o, torch.full_like(o, (1 + 2 * e) / (1 + e))) and abs(float(lse) - math.log(1 + e)) < 1e-14
    (o, lse), _ = ref.attend(k, v, q, torch.zeros(1, 1, dtype=torch.int32), torch.tensor([2]), 0.5, 1, (1., 1.), torch.float32)
    assert torch.equal(o, torch.full_like(o, 2)) and abs(float(lse) - 1) < 1e-14
    (o, lse), _ = ref.attend(k, v, q, torch.zeros(1, 1, dtype=torch.int32), torch.tensor([0]), 0.5, 0, (1., 1.), torch.float32)
    assert torch.equal(o, torch.zeros_like(o)) and float(lse) == -math.inf


def test_attend_notices_a_token_too_many_or_few():
    torch.manual_seed(2)
    k, v = torch.randn(4, 2, 16, 64).bfloat16(), torch.randn(4, 2, 16, 64).bfloat16()
    q, tables = torch.randn(1, 4, 64).bfloat16(), torch.tensor([[2, 0, 3, 1]], dtype=torch.int32)
    (o, lse), (ot, lt) = ref.attend(k, v, q, tables, torch.tensor([50]), 0.125, 0, (1., 1.), torch.bfloat16)
    for n in (49, 51):
        (p, pl), _ = ref.attend(k, v, q, tables, torch.tensor([n]), 0.125, 0, (1., 1.), torch.bfloat16)
        for got, want, tol in ((p, o, ot), (pl, lse, lt)):
            with pytest.raises(AssertionError):
                ref.close(got, want, tol)
