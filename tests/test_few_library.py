"""Host-side checks of the few-token layer's entry point: every call here is refused before
anything is launched."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def native():
    from routing_dispatch_expert_gemm_b200 import build, native
    build.build()
    native.lib()
    return native


FAKE = 1 << 20  # 16-byte aligned, never dereferenced
WS = 1 << 12


def few(native, cfg, x=FAKE, w_router=FAKE, w_gate=FAKE, w_up=FAKE, w_down=FAKE, s_gate=None,
        s_up=None, s_down=None, y=FAKE, ws=WS):
    return native.lib().moe_forward_few(ctypes.byref(cfg), x, w_router, None, w_gate, w_up,
                                        w_down, s_gate, s_up, s_down, y, None, None, None, None,
                                        None, ws, None)


@pytest.mark.parametrize("kw", [
    dict(T=33), dict(stats=True), dict(layout="padded", capacity=4),
    dict(layout="padded", capacity=4, overflow="reroute"), dict(fuse="gather"),
    dict(fuse="combine"), dict(d=96), dict(d_ff=130), dict(d=66, dtype="f32"), dict(E=257),
    dict(d=(1 << 24) + 128), dict(d_ff=(1 << 24) + 128), dict(E=255, d_ff=1 << 23)])
def test_unsupported(native, kw):
    shape = dict(T=8, d=128, E=4, k=2, d_ff=128)
    shape.update(kw)
    assert few(native, native.make_config(**shape)) == 2


def test_invalid(native):
    cfg = native.make_config(8, 128, 4, 2, 128)
    for name in ("x", "w_router", "w_gate", "w_up", "w_down", "y"):
        assert few(native, cfg, **{name: None}) == 1
    for name in ("x", "w_router", "w_gate", "w_up", "w_down"):
        assert few(native, cfg, **{name: FAKE + 8}) == 1     # rows are copied in 16 bytes
    for y in (FAKE + 2, FAKE + 8 * 128 * 2 - 2, FAKE - 8 * 128 * 2 + 2):  # inside x, not x
        assert few(native, cfg, y=y) == 1
    assert few(native, cfg, ws=None) == 3 and few(native, cfg, ws=WS + 16) == 3
    shared = native.make_config(8, 128, 4, 2, 128, has_shared=True)
    full = dict(s_gate=FAKE, s_up=FAKE, s_down=FAKE)
    for name in full:
        assert few(native, shared, **dict(full, **{name: None})) == 1
        assert few(native, shared, **dict(full, **{name: FAKE + 4})) == 1
    assert few(native, native.make_config(8, 128, 4, 5, 128)) == 1  # k > E


def test_workspace_covers_both_forwards(native):
    """One workspace serves moe_forward and moe_forward_few, also where moe_forward's own
    rows shrink (capacity) and the few-token layer's do not."""
    for kw in (dict(), dict(capacity=0), dict(capacity=1, has_shared=True)):
        for T in (1, 32):
            cfg = native.make_config(T, 256, 200, 8, 1024, **kw)
            rows = T * (8 + cfg.has_shared)
            assert native.moe_workspace_bytes(cfg) >= 256 + T * 200 * 4 + rows * 1024 * 2


@pytest.mark.parametrize("kw", [
    dict(), dict(capacity=0), dict(capacity=1, has_shared=True), dict(capacity=40),
    dict(dtype="f32", capacity=2), dict(stats=True, capacity=3), dict(fuse="gather+combine"),
    dict(layout="padded", capacity=8), dict(layout="padded", capacity=8, overflow="reroute")])
def test_workspace_serves_fewer_tokens(native, kw):
    """Bytes never fall as T grows, also from 32 tokens, the most of the few-token layer, to 33."""
    sizes = [native.moe_workspace_bytes(native.make_config(T, 256, 200, 8, 1024, **kw))
             for T in (*range(1, 300), 500, 1000, 4096, 4097)]
    assert sizes == sorted(sizes) and sizes[0] > 256


@pytest.mark.parametrize("T", [1, 7, 32, 33, 129])
@pytest.mark.parametrize("capacity", [0, 1, 17])
def test_an_option_only_adds_bytes(native, T, capacity):
    """Also where the few-token layer, which does not take the option, has the larger part."""
    shape = (T, 256, 200, 10, 1024)
    base = native.moe_workspace_bytes(native.make_config(*shape, capacity=capacity))
    for kw in (dict(stats=True), dict(layout="padded"), dict(layout="padded", overflow="reroute"),
               dict(fuse="gather"), dict(fuse="combine"), dict(has_shared=True)):
        cfg = native.make_config(*shape, capacity=capacity, **kw)
        assert native.moe_workspace_bytes(cfg) >= base, kw
