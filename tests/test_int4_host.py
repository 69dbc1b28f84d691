"""What the calls of a 4-bit cache refuse before anything is launched (no GPU)."""
import pytest
import torch


@pytest.fixture(scope="module")
def pkv():
    from tests.conftest import build_native
    build_native()
    import paged_kv_cache_49_gb300 as m
    return m


def test_block_bytes(pkv):
    L = pkv._native.lib
    for groups, gd in ((4, 32), (2, 64), (1, 128)):
        for bt in (8, 16, 32, 64):
            assert L.pkv_int4_block_bytes(3, bt, gd) == 3 * bt // 8 * (1024 + 64 * groups)
    for hkv, bt, gd in ((0, 16, 64), (8, 12, 64), (8, 16, 16), (8, 16, 0), (8, 0, 64), (-1, 16, 64)):
        assert L.pkv_int4_block_bytes(hkv, bt, gd) == 0


def test_c_calls_refuse(pkv):
    from paged_kv_cache_49_gb300 import _native as nat
    L, P = nat.lib, 4096  # an aligned address that is never read: every call below is refused
    append = lambda k=P, ks=1024, v=P, vs=1024, slots=P, T=4, cache=P, nb=8, hkv=8, d=128, bt=16, gd=64: L.pkv_append_int4(
        k, ks, v, vs, slots, T, cache, nb, hkv, d, bt, gd, None, None)
    for bad in (dict(k=None), dict(v=None), dict(slots=None), dict(cache=None), dict(ks=1016), dict(vs=1028), dict(k=P + 2),
                dict(cache=P + 8), dict(T=-1), dict(nb=0), dict(hkv=0)):
        assert append(**bad) == nat.PKV_EINVAL, bad
    for bad in (dict(d=64), dict(bt=12), dict(gd=16)):
        assert append(**bad) == nat.PKV_EUNSUPPORTED, bad
    for bad in (dict(nb=1 << 27, bt=64), dict(ks=1 << 40), dict(T=(1 << 30) + 1)):
        assert append(**bad) == nat.PKV_ERANGE, bad
    assert append(T=0, k=None) == nat.PKV_OK

    load = lambda cache=P, pairs=P, n=2, k=P, v=P, nb=8, nd=8, hkv=8, d=128, bt=16, gd=64: L.pkv_load_int4(
        cache, pairs, n, k, v, nb, nd, hkv, d, bt, gd, None, None)
    for bad in (dict(cache=None), dict(pairs=None), dict(k=None), dict(v=None), dict(n=-1), dict(nd=0), dict(k=P + 4)):
        assert load(**bad) == nat.PKV_EINVAL, bad
    for bad in (dict(d=256), dict(bt=24), dict(gd=256)):
        assert load(**bad) == nat.PKV_EUNSUPPORTED, bad
    assert load(nd=1 << 28) == nat.PKV_ERANGE and load(n=0, pairs=None) == nat.PKV_OK

    copy = lambda cache=P, pairs=P, n=2, nb=8, hkv=8, d=128, bt=16, gd=64: L.pkv_block_copy_int4(
        cache, pairs, n, nb, hkv, d, bt, gd, None, None)
    for bad in (dict(cache=None), dict(pairs=None), dict(n=-1), dict(cache=P + 8)):
        assert copy(**bad) == nat.PKV_EINVAL, bad
    assert copy(n=65536) == nat.PKV_ERANGE and copy(gd=1) == nat.PKV_EUNSUPPORTED and copy(n=0, pairs=None) == nat.PKV_OK

    def decode(q=P, cache=P, tables=P, width=4, ctx=P, B=2, hq=32, hkv=8, d=128, nb=8, bt=16, gd=64, scale=0.1, ctas=0, ws=P,
               nbytes=1 << 20, out=P):
        return L.pkv_attn_decode_int4(q, cache, tables, width, ctx, B, hq, hkv, d, nb, bt, gd, scale, ctas, ws, nbytes, out,
                                      None)
    for bad in (dict(q=None), dict(cache=None), dict(tables=None), dict(ctx=None), dict(ws=None), dict(out=None), dict(B=0),
                dict(hq=0), dict(hkv=0), dict(nb=0), dict(width=0), dict(ctas=-1), dict(ctas=nat.MAX_CTAS + 1),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(q=P + 2), dict(ws=P + 16), dict(out=P + 8)):
        assert decode(**bad) == nat.PKV_EINVAL, bad
    for bad in (dict(B=4097), dict(d=64), dict(hq=33), dict(hq=72), dict(bt=48), dict(gd=96)):
        assert decode(**bad) == nat.PKV_EUNSUPPORTED, bad
    for bad in (dict(nb=1 << 25), dict(width=1 << 28), dict(B=4096, width=1 << 20)):
        assert decode(**bad) == nat.PKV_ERANGE, bad


def test_the_wait_test_refuses(pkv):
    from paged_kv_cache_49_gb300 import _native as nat
    call = lambda stop=0, gd=64, q=4096: nat.lib.pkv_attn_decode_int4_wait_test(
        q, 4096, 4096, 4, 4096, 2, 32, 8, 128, 8, 16, gd, 0.1, 0, 4096, 1 << 20, 4096, stop, None)
    assert call(stop=-1) == call(q=None) == nat.PKV_EINVAL and call(gd=32) == call(gd=128) == nat.PKV_EUNSUPPORTED


def _cache(pkv, blocks=4, hkv=2, bt=16, gd=64):
    return pkv.Int4Cache(blocks, hkv, bt, gd, device="cpu")


def test_the_cache_object(pkv):
    c = _cache(pkv)
    assert _cache(pkv, bt=64).data.shape == (4, 4, 2, 2 * 1152) and _cache(pkv, bt=8, gd=128).data.shape == (4, 1, 2, 1088)
    assert c.data.shape == (4, 1, 2, 2 * 1152) and c.data.dtype == torch.uint8 and not c.data.any()
    for bad in (dict(blocks=0), dict(hkv=0), dict(bt=24), dict(gd=48)):
        with pytest.raises(ValueError):
            _cache(pkv, **bad)


def test_python_calls_refuse(pkv):
    c = _cache(pkv)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    pairs = torch.zeros((1, 2), dtype=torch.int32)
    # host tensors are named, not read
    with pytest.raises(ValueError, match="cache"):
        pkv.append_int4(bf(3, 2, 128), bf(3, 2, 128), slots, c)
    with pytest.raises(ValueError, match="cache"):
        pkv.load_int4(c, pairs, bf(4, 2, 16, 128), bf(4, 2, 16, 128))
    with pytest.raises(ValueError, match="cache"):
        pkv.block_copy_int4(c, pairs)
    with pytest.raises(ValueError, match="q"):
        pkv.attn_decode_int4(bf(1, 4, 128), c, pairs, torch.zeros(1, dtype=torch.int32), 0.1)
