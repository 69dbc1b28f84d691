"""Norm, rotation and append in one pass against the oracle."""
import numpy as np
import pytest
import torch

from oracle import prompt_attention as po
from workloads import randn_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from tests.conftest import build_native
    build_native()
    import paged_kv_cache_49_gb300 as m
    return m


def _near(bits, want):
    """bf16 against float64: the rounding's half step, 2^-8 of the value; the
    pair's two fp32 products, their sum, the norm's sum of up to 256 squares and
    its root, some 2^-22 of the pair's size in all -- under 2^-19 of the row's
    largest value, which bounds either term of a pair up to a factor of 2."""
    g = (np.asarray(bits).astype(np.uint32) << np.uint32(16)).view(np.float32).astype(np.float64)
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * np.abs(want).max(axis=-1, keepdims=True)
    assert np.isfinite(g).all() and (np.abs(g - want) <= tol).all(), np.abs(g - want).max()


def _run(pkv, T, hq, hkv, d, rot, norm, interleaved, bt, padding=(), fused=True, seed=0, max_pos=5000, stream=None):
    rng = np.random.default_rng(seed)
    bits = {n: randn_bf16(rng, (T, h, d)) for n, h in (("q", hq), ("k", hkv), ("v", hkv))}
    wq, wk = (randn_bf16(rng, (d,)), randn_bf16(rng, (d,))) if norm else (None, None)
    dev = {n: pkv.bf16_from_bits(b).cuda() for n, b in bits.items()}
    if fused:  # views of one projection's output
        whole = torch.cat([dev[n].reshape(T, -1) for n in "qkv"], dim=1)
        at = np.cumsum([0, hq * d, hkv * d, hkv * d])
        dev = {n: whole[:, at[i] : at[i + 1]].view(T, h, d) for i, (n, h) in
               enumerate((("q", hq), ("k", hkv), ("v", hkv)))}
    table = pkv.rope_table(max_pos, rot, device="cuda") if rot else None
    positions = rng.integers(0, max_pos, size=T).astype(np.int32)
    nb = T // bt + 3
    slots = rng.permutation(nb * bt)[:T].astype(np.int64)
    slots[list(padding)] = -1
    positions[list(padding)] = -7  # whatever a padding row holds
    kc = torch.full((nb, hkv, bt, d), 3.0, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    err = pkv.new_error_word()
    w = [None if x is None else pkv.bf16_from_bits(x).cuda() for x in (wq, wk)]
    k_out = torch.full((T, hkv, d), 5.0, dtype=torch.bfloat16, device="cuda") if seed % 2 else None
    q = pkv.qk_norm_rope_append(dev["q"], dev["k"], dev["v"], table, torch.from_numpy(positions).cuda(),
                                torch.from_numpy(slots).cuda(), kc, vc, q_weight=w[0], k_weight=w[1], eps=1e-5,
                                interleaved=interleaved, k_out=k_out, device_error=err, stream=stream)
    torch.cuda.synchronize()
    assert pkv.read_device_error(err) == 0
    cs = table.cpu().numpy() if rot else None
    at = np.clip(positions, 0, None)
    _near(pkv.bits_from_bf16(q), po.norm_rope(bits["q"], wq, 1e-5, cs, at, interleaved))
    kept = slots >= 0
    blk, r = slots[kept] // bt, slots[kept] % bt
    kb, vb = pkv.bits_from_bf16(kc), pkv.bits_from_bf16(vc)
    _near(kb[blk, :, r], po.norm_rope(bits["k"], wk, 1e-5, cs, at, interleaved)[kept])
    assert np.array_equal(vb[blk, :, r], bits["v"][kept])
    if k_out is not None:  # every row's keys, padding included
        _near(pkv.bits_from_bf16(k_out), po.norm_rope(bits["k"], wk, 1e-5, cs, at, interleaved))
        assert np.array_equal(pkv.bits_from_bf16(k_out)[kept], kb[blk, :, r])
    untouched = np.ones((nb, bt), bool)
    untouched[blk, r] = False
    three = np.uint16(0x4040)
    for c in (kb, vb):
        assert (c.transpose(0, 2, 1, 3)[untouched] == three).all()
    return q


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (128, 0), (64, 64), (64, 32), (64, 16), (256, 256), (256, 64),
                                   (96, 96), (96, 48), (80, 32), (32, 32), (16, 16), (8, 0), (136, 112), (200, 176)])
def test_head_sizes(pkv, d, rot, norm, interleaved):
    _run(pkv, 37, 6, 2, d, rot, norm, interleaved, 16, padding=(3, 36), seed=d + rot)


@pytest.mark.parametrize("T", [1, 2, 64, 1000, 4099])
@pytest.mark.parametrize("hq,hkv", [(32, 8), (8, 1), (5, 5), (1, 1)])
def test_tokens_and_heads(pkv, T, hq, hkv):
    _run(pkv, T, hq, hkv, 128, 128, True, False, 16, padding=(0,) if T > 1 else (), seed=T + hq)


@pytest.mark.parametrize("bt", [8, 32, 64])
def test_block_sizes_and_separate_tensors(pkv, bt):
    _run(pkv, 100, 8, 2, 128, 128, True, False, bt, fused=False, seed=bt)


def test_far_positions(pkv):
    """Angles at 100,000 and more positions come from the table as they are."""
    _run(pkv, 300, 4, 2, 128, 128, True, False, 16, max_pos=1 << 17, seed=3)
    i = np.arange(64)
    want = np.cos(131071.0 * 10000.0 ** (-2.0 * i / 128))
    got = pkv.rope_table(1 << 17, 128, device="cuda")[131071, :64].cpu().numpy()
    assert np.abs(got - want).max() <= 2.0 ** -24  # the rounding to fp32 alone


def test_a_side_stream_and_a_graph(pkv):
    a = _run(pkv, 64, 8, 2, 128, 128, True, False, 16, seed=5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert torch.equal(a, _run(pkv, 64, 8, 2, 128, 128, True, False, 16, seed=5, stream=s))
    q = torch.randn(4, 8, 128, device="cuda").bfloat16()
    k = torch.randn(4, 2, 128, device="cuda").bfloat16()
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    slots = torch.arange(4, device="cuda")
    kc, vc = (torch.zeros(2, 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = pkv.rope_table(100, 128)
    out = torch.zeros_like(q)
    pkv.qk_norm_rope_append(q, k, k, table, pos, slots, kc, vc, q_out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.qk_norm_rope_append(q, k, k, table, pos, slots, kc, vc, q_out=out)
    pos += 50
    want_kc = torch.zeros_like(kc)
    want = pkv.qk_norm_rope_append(q, k, k, table, pos, slots, want_kc, vc).clone()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(kc, want_kc)


def test_bad_positions_and_slots_set_their_bits(pkv):
    q = torch.randn(4, 8, 128, device="cuda").bfloat16()
    k = torch.randn(4, 2, 128, device="cuda").bfloat16()
    kc, vc = (torch.zeros(2, 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = pkv.rope_table(100, 128)
    err = pkv.new_error_word()

    def run(pos, slots):
        pkv.qk_norm_rope_append(q, k, k, table, torch.tensor(pos, dtype=torch.int32, device="cuda"),
                                torch.tensor(slots, device="cuda"), kc, vc, device_error=err)
        return pkv.read_device_error(err)

    assert run([0, 1, 2, 99], [0, 1, 2, 31]) == 0
    assert run([0, 1, 2, 100], [0, 1, 2, 3]) == pkv.DEVERR_POSITION
    assert run([0, -1, 2, 3], [0, 1, 2, 3]) == pkv.DEVERR_POSITION
    assert run([0, -1, 2, 1 << 30], [0, -1, 2, -1]) == 0  # padding rows
    before = kc.clone(), vc.clone()
    assert run([5, 5, 5, 5], [-1, -1, -1, 32]) == pkv.DEVERR_SLOT
    assert torch.equal(kc, before[0]) and torch.equal(vc, before[1])
    slots = torch.arange(4, device="cuda")
    for bad in (dict(positions=None), dict(positions=torch.zeros(4, device="cuda")), dict(k=k[:, :1]), dict(k=k.cpu()),
                dict(slot_mapping=slots[:3]), dict(q_weight=torch.ones(64, dtype=torch.bfloat16, device="cuda")),
                dict(k_out=torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")), dict(v_cache=vc[:1])):
        a = dict(q=q, k=k, v=k, cos_sin=table, positions=torch.arange(4, dtype=torch.int32, device="cuda"),
                 slot_mapping=slots, k_cache=kc, v_cache=vc)
        a.update(bad)
        with pytest.raises(ValueError):
            pkv.qk_norm_rope_append(**a)
