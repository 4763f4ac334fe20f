"""The bound of the attention over selected pages rejects weights in one 16-bit piece and
weights that are lost at the range's lower end."""
import pytest
import torch

import selected_bound as sb

BF16, F16 = torch.bfloat16, torch.float16


def outputs(q, k, v, scale, weight):
    """The attention with its weights, relative to the largest, passed through `weight` for
    the products but not for their sum."""
    D = q.shape[-1]
    x = q.double()[0] @ k.double().reshape(-1, D).T * scale
    w = torch.exp(x - x.amax(-1, keepdim=True))
    return (weight(w) @ v.double().reshape(-1, D) / w.sum(-1, keepdim=True))[None]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("seed", range(5))
def test_one_piece_is_rejected(dtype, seed):
    q, k, v, table, lens, lists, scale = sb.cancelling(dtype, seed)
    want, bound = sb.attend(q, k, v, table, lens, lists, scale)
    one = outputs(q, k, v, scale, lambda w: w.to(dtype).double())
    wrong = (one.to(dtype).double() - want).abs() > bound
    assert wrong[0, 0].sum() >= 16  # a good part of the head that cancels
    good = outputs(q, k, v, scale, lambda w: w)
    assert not ((good.to(dtype).double() - want).abs() > bound).any()


@pytest.mark.parametrize("drop", [22, 25, 28, 32])
def test_lost_weights_are_rejected(drop):
    q, k, v, table, lens, lists, scale = sb.tail(F16, drop)
    want, bound = sb.attend(q, k, v, table, lens, lists, scale)

    def two(w, top):
        hi = (w * top).to(F16).double()
        return (hi + (w * top - hi).to(F16).double()) / top
    # the largest weight at 1: steps of 2^-24; at 2^15: of 2^-39
    lost = outputs(q, k, v, scale, lambda w: two(w, 1.0))
    assert ((lost.to(F16).double() - want).abs() > bound).any() == (drop >= 25)
    kept = outputs(q, k, v, scale, lambda w: two(w, 2.0 ** 15))
    assert not ((kept.to(F16).double() - want).abs() > bound).any()
