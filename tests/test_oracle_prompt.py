"""CPU pins of the prompt-side oracle: one axis is the plain rotation, an appended chunk attends as the
verify oracle's rows do, and chunks one after the other give what the whole prompt gives."""
import numpy as np
import pytest

from oracle import ops, prompt


def test_one_axis_is_the_plain_rotation():
    rng = np.random.default_rng(0)
    x, pos = rng.standard_normal((5, 3, 128)), np.array([0, 1, 17, 4000, 131071])
    for il in (False, True):
        got, _ = prompt.rotate(x, prompt.rope_table_axes(pos[None], [64], 128, 1e6, il))
        assert np.allclose(got, ops.rope(x, pos, 1e6), rtol=0, atol=1e-9)


def test_equal_axes_are_one_axis_and_sections_pick_their_axis():
    pos = np.array([3, 9, 200])
    one = prompt.rope_table_axes(pos[None], [64], 128, 1e4, False)
    for sections, il in (([16, 24, 24], False), ([24, 20, 20], True)):
        assert np.array_equal(prompt.rope_table_axes(np.stack([pos] * 3), sections, 128, 1e4, il), one)
    assert prompt.frequency_axes([2, 1, 3], 6, False).tolist() == [0, 0, 1, 2, 2, 2]
    assert prompt.frequency_axes([4, 2, 2], 8, True).tolist() == [0, 1, 2, 0, 1, 2, 0, 0]
    assert prompt.frequency_axes([6, 0, 2], 8, True).tolist() == [0, 0, 2, 0, 0, 2, 0, 0]
    assert prompt.frequency_axes([8, 0, 0], 8, True).tolist() == [0] * 8


@pytest.mark.parametrize("rows,ctx", [([3, 1, 4], [130, 0, 255]), ([5, 0, 2], [127, 3, 1])])
def test_chunk_attention_after_append_is_verify_attention(rows, ctx):
    rng = np.random.default_rng(1)
    Hq, Hkv, D, mp = 4, 2, 16, 3
    B = len(rows)
    cu = np.concatenate([[0], np.cumsum(rows)])
    table = rng.permutation(B * mp + 2)[:B * mp].reshape(B, mp)
    kp, vp = rng.standard_normal((2, Hkv, B * mp + 2, 128, D))
    gather = lambda p: np.stack([p[:, table[b]].reshape(Hkv, mp * 128, D) for b in range(B)])
    q, k, v = rng.standard_normal((cu[-1], Hq, D)), *rng.standard_normal((2, cu[-1], Hkv, D))
    ref, kc, vc = ops.verify_attention(q, k, v, cu, gather(kp), gather(vp), ctx, 0.25)
    kp2, vp2 = prompt.kv_append(k, v, cu, ctx, kp, vp, table)
    assert np.array_equal(gather(kp2), kc) and np.array_equal(gather(vp2), vc)
    got, mag = prompt.chunk_attention(q, cu, ctx, kp2, vp2, table, 0.25)
    assert np.allclose(got, ref, rtol=0, atol=1e-12) and np.all(mag >= abs(got) - 1e-12)


def test_chunks_in_turn_give_the_whole_prompt():
    rng = np.random.default_rng(2)
    D, n = 8, 300
    q, k, v = rng.standard_normal((n, 2, D)), *rng.standard_normal((2, n, 1, D))
    table = np.array([[2, 0, 1]])
    kp = vp = np.full((1, 3, 128, D), np.nan)
    outs, at = [], 0
    for m in (1, 130, 169):
        cu, ctx = np.array([0, m]), np.array([at])
        kp, vp = prompt.kv_append(k[at:at + m], v[at:at + m], cu, ctx, kp, vp, table)
        outs.append(prompt.chunk_attention(q[at:at + m], cu, ctx, kp, vp, table, 0.3)[0])
        at += m
    whole, _ = prompt.chunk_attention(q, np.array([0, n]), np.array([0]), kp, vp, table, 0.3)
    assert np.allclose(np.concatenate(outs), whole, rtol=0, atol=1e-12)
