"""The 4-bit cache's oracle: rounding bounds, edge values, and its bytes against
a layout written out value by value."""
import numpy as np
import pytest

from oracle import int4


def _rows(seed, *shape):
    x = np.random.default_rng(seed).standard_normal(shape).astype(np.float32)
    return (x.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)  # bf16 values


@pytest.mark.parametrize("group_dims", [32, 64, 128])
def test_values_are_within_half_a_step(group_dims):
    x = _rows(0, 50, 128) * np.float32(3)
    c, s, m = int4.quantise(x, group_dims)
    back = int4.values(c, s, m)
    step = np.repeat(s.astype(np.float64), group_dims, axis=-1)
    # half a step, and what the rounding of s to 11 bits takes off the range's end
    assert (np.abs(back - x) <= step * (0.5 + 15 * 2.0 ** -11) + 1e-6).all()
    assert c.min() == 0 and c.max() == 15


def test_edge_values():
    x = np.zeros((6, 128), np.float32)
    x[1] = 2.5
    x[2, ::2] = np.inf
    x[3, :] = -np.inf
    x[4, 5] = np.nan
    x[5, 3] = 2.0 ** -30  # a range too small for an fp16 scale
    c, s, m = int4.quantise(x, 64)
    back = int4.values(c, s, m)
    assert (back[0] == 0).all() and (back[1] == 2.5).all()
    assert s[2, 0] == np.float16(65504 / 15) and (back[2, ::2] == float(s[2, 0]) * 15).all() and (back[2, 1::2] == 0).all()
    assert (back[3] == -65504).all() and (s[3] == 0).all()
    assert np.isnan(back[4, :64]).all() and (back[4, 64:] == 0).all()
    assert (back[5] == 0).all() and (c[5] == 0).all()


def test_halves_round_to_even():
    x = np.zeros((1, 128), np.float32)
    x[0, 0], x[0, 1] = -0.9375, 0.9375          # s = 1 / 8 exactly
    x[0, 2:6] = -0.9375 + np.array([0.5, 1.5, 2.5, 7.5]) / 8
    c, s, _ = int4.quantise(x, 128)
    assert s[0, 0] == np.float16(0.125) and c[0, :6].tolist() == [0, 15, 0, 2, 2, 8]


@pytest.mark.parametrize("group_dims", [32, 64, 128])
def test_bytes(group_dims):
    tokens, groups = 16, 128 // group_dims
    k, v = (int4.quantise(_rows(seed, tokens, 128), group_dims) for seed in (1, 2))
    one = [[x[None] for x in kv] for kv in (k, v)]  # one head
    got = int4.pack(*one)
    unit = 1024 + 64 * groups
    assert got.shape == (1, 1, 2 * unit)
    # slabs of 16 tokens (8 in a block of 8), in each the heads
    heads = [[np.stack([x, x[::-1]]) for x in kv] for kv in (k, v)]
    eight = int4.pack(*[[x[:, :8] for x in kv] for kv in heads])
    assert eight.shape == (1, 2, unit) and np.array_equal(eight[0, 0], got[0, 0, :unit])
    twice = int4.pack(*[[np.concatenate([x, x[:, ::-1]], axis=1) for x in kv] for kv in heads])
    assert twice.shape == (2, 2, 2 * unit)
    assert np.array_equal(twice[0, 0], got[0, 0]) and np.array_equal(twice[1, 1], got[0, 0])
    assert np.array_equal(twice[0, 1], twice[1, 0]) and not np.array_equal(twice[0, 0], twice[0, 1])
    got = got[0, 0]
    want = np.zeros(2 * unit, np.uint8)

    def nibble(byte, high, code):
        want[byte] |= code << (4 if high else 0)

    for t in range(tokens):
        u, i = unit * (t // 8), t % 8
        for d in range(128):
            w, c = d // 32, d % 32 // 8
            nibble(u + 64 * i + 4 * (4 * c + w) + d % 8 // 2, d % 2, k[0][t, d])
            r = d % 32 // 4
            nibble(u + 512 + 2 * (((r * 4 + i // 2) * 4 + w) * 2 + i % 2) + d % 4 // 2, d % 2, v[0][t, d])
        for g in range(groups):
            at = u + 1024 + 4 * (groups * i + g)
            want[at:at + 2], want[at + 2:at + 4] = (p[t, g:g + 1].view(np.uint8) for p in k[1:])
            for j, p in enumerate(v[1:]):
                at = u + 1024 + 32 * groups + 16 * groups * j + 2 * (8 * g + i)
                want[at:at + 2] = p[t, g:g + 1].view(np.uint8)
    assert got.shape == want.shape and np.array_equal(got, want)


def test_decode_is_attention_over_the_values():
    import torch
    k, v = (int4.quantise(_rows(seed, 5, 2, 8, 128), 64) for seed in (3, 4))
    q = _rows(5, 2, 4, 128).astype(np.float64)
    tables, ctx = np.array([[3, 0, 4], [1, -1, -1]]), np.array([19, 0])
    out, a, e = int4.decode(q, k, v, tables, ctx, 0.1)
    assert (out[1] == 0).all()
    rows = [int4.values(*x)[tables[0]].swapaxes(1, 2).reshape(24, 2, 128)[:19] for x in (k, v)]
    for h in range(4):
        key, val = (torch.from_numpy(np.ascontiguousarray(r[:, h // 2])) for r in rows)
        want = torch.softmax(0.1 * torch.from_numpy(q[0, h]) @ key.T, -1) @ val
        assert np.allclose(out[0, h], want.numpy(), atol=1e-12)
        assert (a[0, h] >= np.abs(out[0, h]) - 1e-12).all()
    assert (e[0] > 0).all()
