"""The oracle of the ragged serving step pinned without a GPU: against the plain decode and
prefill oracles where a window covers everything, and against hand-made cases."""
import numpy as np

from compressed_paged_kv_tq4_b200 import inputs as I
from oracle import step_oracle as S
from oracle import tq4_oracle as O

SCALE = 1.0 / 16.0


def _pool(config, lens):
    signs, c = I.signs(config), O.codebook()[0]
    need = [-(-t // 256) for t in lens]
    ids = I.page_table_scattered(config, sum(need), sum(need) + 1)
    tab = np.full((len(lens), max(need)), -1, np.int32)
    pool, at = O.new_pool(sum(need) + 1), 0
    for r, t in enumerate(lens):
        tab[r, :need[r]] = ids[at:at + need[r]]
        at += need[r]
        k, v = I.kv_vectors(config, 0, t, request=r)
        O.encode_append(pool, tab[r], 0, k, v, signs, c)
    return pool, tab, signs, c


def test_a_window_of_everything_is_the_plain_decode_and_prefill():
    lens = [5, 300]
    pool, tab, signs, c = _pool(3, lens)
    q = I.bf16_bits_to_f32(I.queries(3, 0, (2, 3, 24, 256)))
    plain = O.decode_attention(pool, tab, lens, q, SCALE, signs, c)
    for window, sinks in ((300, 0), (1 << 30, 7), (1, 300)):
        got = S.decode_attention_window(pool, tab, lens, q, window, sinks, SCALE, signs, c)
        assert np.abs(got - plain).max() < 1e-12
    n = 9
    kb, vb = (I.bf16_bits_to_f32(x) for x in I.chunk_kv(3, 0, n))
    qc = I.bf16_bits_to_f32(I.queries(3, 1, (n, 24, 256)))
    plain = O.prefill_attention(pool, tab[1], 260, qc, kb, vb, SCALE, signs, c)
    got = S.prefill_attention_ragged(pool, tab[1:], [260 + n], [0, n], qc, kb, vb, 1 << 30, 0, SCALE, signs, c)
    assert np.abs(got - plain).max() < 1e-12


def test_a_window_of_one_without_sinks_is_the_own_value():
    pool, tab, signs, c = _pool(4, [40])
    q = I.bf16_bits_to_f32(I.queries(4, 0, (1, 2, 24, 256)))
    got = S.decode_attention_window(pool, tab, [40], q, 1, 0, SCALE, signs, c)
    _, v = O.reconstruct(pool, tab[0], 38, 2, signs, c)
    assert np.abs(got[0] - np.repeat(v, O.GROUP, axis=1)).max() < 1e-12


def test_masked_pages_are_not_read():
    pool, tab, signs, c = _pool(5, [900])
    q = I.bf16_bits_to_f32(I.queries(5, 0, (1, 1, 24, 256)))
    exp = S.decode_attention_window(pool, tab, [900], q, 100, 3, SCALE, signs, c)
    tab[0, 1:3] = 10 ** 6   # positions 256 .. 767: between the sinks and the window
    assert np.array_equal(S.decode_attention_window(pool, tab, [900], q, 100, 3, SCALE, signs, c), exp)


def test_rope_is_a_rotation_by_each_axis():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(4, 2, 256))
    ang = rng.normal(size=(4, 16))
    for adjacent in (False, True):
        y = S.rope_turn(x, np.cos(ang), np.sin(ang), adjacent)
        assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
        assert np.array_equal(y[..., 32:], x[..., 32:])
        back = S.rope_turn(y, np.cos(ang), -np.sin(ang), adjacent)
        assert np.abs(back - x).max() < 1e-14
    i, j = (3, 19), (6, 7)   # pair 3 of halves and of adjacent pairs
    for (a, b), adjacent in ((i, False), (j, True)):
        y = S.rope_turn(x, np.cos(ang), np.sin(ang), adjacent)
        assert np.allclose(y[..., a], x[..., a] * np.cos(ang)[:, None, 3] - x[..., b] * np.sin(ang)[:, None, 3])
    assert S.rope_axes(8, [4, 2, 2], False).tolist() == [0, 0, 0, 0, 1, 1, 2, 2]
    assert S.rope_axes(8, [4, 2, 2], True).tolist() == [0, 1, 2, 0, 1, 2, 0, 0]


def test_plan_by_hand():
    # 256 cached positions + 1 needs page 1; 10 + 5 needs none; the third finds one page of two
    tab = np.full((4, 3), -1)
    tab[0, 0], tab[1, 0] = 7, 2
    t, cu, lens, pos, slot, taken, codes = S.plan_step([256, 10, 0, 0], [1, 5, 300, 0], [9, 4], tab, 10, 310)
    assert t[0].tolist() == [7, 9, -1] and t[2].tolist() == [-1, -1, -1] and taken == 1 and codes == {"pages"}
    assert cu.tolist() == [0, 1, 6, 306, 306] and lens.tolist() == [257, 15, 0, 0]
    assert slot[0] == 9 * 256 and slot[1:6].tolist() == [2 * 256 + i for i in range(10, 15)] and (slot[6:] == -1).all()
    assert pos[0] == 256 and pos[6:10].tolist() == [0, 1, 2, 3] and (pos[306:] == 0).all()
