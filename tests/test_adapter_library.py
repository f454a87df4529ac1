"""Host-side checks of the adapter projections' entry points: every call here is refused
before anything is launched."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def native():
    from routing_dispatch_expert_gemm_b200 import build, native
    build.build()
    native.lib()
    return native


FAKE = 1 << 20  # 16-byte aligned, never dereferenced
OUT = 1 << 50   # behind the largest input
WS = 1 << 12
LINEAR = dict(x=FAKE, w=FAKE, a=FAKE, b=FAKE, scale=None, ids=FAKE, addend=None, y=OUT,
              n_tokens=None, ws=WS)
PAIR = dict(x=FAKE, w_gate=FAKE, w_up=FAKE, a_gate=FAKE, b_gate=FAKE, a_up=FAKE, b_up=FAKE,
            scale=None, ids=FAKE, h=OUT, n_tokens=None, ws=WS)


def linear(native, cfg, **kw):
    args = dict(LINEAR, **kw)
    return native.lib().moe_adapter_linear(ctypes.byref(cfg), *args.values(), None)


def gate_up(native, cfg, **kw):
    args = dict(PAIR, **kw)
    return native.lib().moe_adapter_gate_up(ctypes.byref(cfg), *args.values(), None)


SHAPE = dict(T=8, d_in=64, d_out=32, n_adapters=2, rank=8)


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), 1), (dict(d_in=0), 1), (dict(d_out=-8), 1), (dict(n_adapters=0), 1),
    (dict(rank=0), 1), (dict(d_in=60), 2), (dict(d_out=36), 2), (dict(rank=12), 2),
    (dict(rank=136), 2), (dict(d_in=62, dtype="f32"), 2), (dict(rank=6, dtype="f32"), 2),
    (dict(rank=132, dtype="f32"), 2), (dict(T=(1 << 24) + 1), 2),
    (dict(d_in=(1 << 24) + 8), 2), (dict(d_out=(1 << 20) + 8), 2),
    (dict(d_in=1 << 20, d_out=1 << 20), 2), (dict(T=1 << 20, d_in=1 << 20), 2)])
def test_shapes(native, kw, code):
    cfg = native.make_adapter_config(**dict(SHAPE, **kw))
    assert linear(native, cfg) == code and gate_up(native, cfg) == code
    assert native.moe_adapter_workspace_bytes(cfg) == 0
    with pytest.raises(native.MoeError):
        native.adapter_workspace(cfg, device="cpu")


def test_unknown_dtype(native):
    cfg = native.make_adapter_config(**SHAPE)
    cfg.dtype = 5
    assert linear(native, cfg) == 1


def test_pointers(native):
    cfg = native.make_adapter_config(**SHAPE)
    for name in ("x", "w", "a", "b", "ids", "y"):
        assert linear(native, cfg, **{name: None}) == 1, name
    for name in ("x", "w", "a", "b"):
        assert linear(native, cfg, **{name: FAKE + 8}) == 1, name
    for name in ("x", "w_gate", "w_up", "a_gate", "b_gate", "a_up", "b_up", "ids", "h"):
        assert gate_up(native, cfg, **{name: None}) == 1, name
    for name in ("x", "w_gate", "w_up", "a_gate", "b_gate", "a_up", "b_up"):
        assert gate_up(native, cfg, **{name: FAKE + 4}) == 1, name
    for call in (linear, gate_up):
        assert call(native, cfg, ws=None) == 3 and call(native, cfg, ws=WS + 64) == 3
    assert native.moe_status_string(7).startswith("adapter id")


def test_workspace_holds_the_shrunk_tokens(native):
    for T, rank in ((1, 8), (32, 128), (4099, 16)):
        cfg = native.make_adapter_config(T, 64, 32, 2, rank)
        assert native.moe_adapter_workspace_bytes(cfg) >= 256 + 2 * T * rank * 4
        assert native.moe_adapter_workspace_bytes(cfg) % 256 == 0


def test_overlapping_outputs(native):
    """y reaches into x, from either side; y and the addend overlap without being the same."""
    for dtype, esz in (("bf16", 2), ("f32", 4)):
        cfg = native.make_adapter_config(**SHAPE, dtype=dtype)
        x_bytes, y_bytes = 8 * 64 * esz, 8 * 32 * esz
        for y in (FAKE, FAKE + x_bytes - esz, FAKE - y_bytes + esz):
            assert linear(native, cfg, y=y) == 1 and gate_up(native, cfg, h=y) == 1
        for ad in (OUT + esz, OUT + y_bytes - esz, OUT - y_bytes + esz):
            assert linear(native, cfg, addend=ad) == 1


def test_types_of_ids_and_counts(native):
    """64-bit ids, torch's default, would be read as pairs of 32-bit ones."""
    torch = pytest.importorskip("torch")
    cfg = native.make_adapter_config(**SHAPE)
    ids, count = torch.zeros(8, dtype=torch.int64), torch.ones(1, dtype=torch.int64)
    with pytest.raises(ValueError):
        native.moe_adapter_linear(cfg, FAKE, FAKE, FAKE, FAKE, None, ids, None, OUT, None, WS, 0)
    with pytest.raises(ValueError):
        native.moe_adapter_linear(cfg, FAKE, FAKE, FAKE, FAKE, None, FAKE, None, OUT, count, WS,
                                  0)
    with pytest.raises(ValueError):
        native.moe_adapter_gate_up(cfg, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, ids, OUT,
                                   None, WS, 0)
    layer = native.make_config(8, 128, 4, 2, 128)
    with pytest.raises(ValueError):
        native.moe_forward_few(layer, FAKE, FAKE, None, FAKE, FAKE, FAKE, None, None, None, FAKE,
                               None, None, None, None, count, WS, 0)


def test_a_workspace_serves_smaller_calls(native):
    """Bytes never fall as T or the rank grows, and nothing else changes them: one workspace of
    the largest sizes serves all calls."""
    def size(T, rank, d_in=64, d_out=32, dtype="bf16", n=2):
        return native.moe_adapter_workspace_bytes(
            native.make_adapter_config(T, d_in, d_out, n, rank, dtype))

    Ts = sorted({*range(1, 5200), *(1 << i for i in range(13, 25)), 18944, 18945, (1 << 24) - 1})
    for rank in (8, 16, 128):
        sizes = [size(T, rank) for T in Ts]
        assert sizes == sorted(sizes) and sizes[0] > 256
    for T in (1, 40, 256, 257, 512, 513, 2304, 2305, 20000):
        ranks = [size(T, r) for r in range(8, 129, 8)]
        assert ranks == sorted(ranks)
        for d_in, d_out in ((4096, 4096), (4096, 8192), (4096, 1024), (64, 128), (16384, 8)):
            for dtype in ("bf16", "f32"):
                assert size(T, 16, d_in, d_out, dtype, 99) == size(T, 16)


def test_types_and_places_of_factors_and_counts(native):
    """32-bit values of another type, values on the host and plain numbers for a count would be
    read as what they are not, partly behind their end."""
    torch = pytest.importorskip("torch")
    cfg = native.make_adapter_config(**SHAPE)
    layer = native.make_config(8, 128, 4, 2, 128)

    def lin(scale=None, ids=FAKE, n_tokens=None):
        native.moe_adapter_linear(cfg, FAKE, FAKE, FAKE, FAKE, scale, ids, None, OUT, n_tokens,
                                  WS + 1, 0)

    def pair(scale=None, ids=FAKE, n_tokens=None):
        native.moe_adapter_gate_up(cfg, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, scale, ids, OUT,
                                   n_tokens, WS + 1, 0)

    def few(logit_bias=None, ids_out=None, gates_out=None, demand_out=None, offsets_out=None,
            n_tokens=None):
        native.moe_forward_few(layer, FAKE, FAKE, logit_bias, FAKE, FAKE, FAKE, None, None, None,
                               FAKE, ids_out, gates_out, demand_out, offsets_out, n_tokens, WS + 1,
                               0)

    i32, f32 = torch.zeros(64, dtype=torch.int32), torch.zeros(64)
    for call in (lin, pair, few):
        with pytest.raises(native.MoeError):  # of the workspace: the rest is well
            call()
        for bad in (f32, i32.long(), i32, 0, 5, True):  # i32: in pageable host memory
            with pytest.raises(ValueError):
                call(n_tokens=bad)
    for call in (lin, pair):
        for bad in (f32, i32):
            with pytest.raises(ValueError):
                call(ids=bad)
        for bad in (f32.bfloat16(), f32.double(), i32, f32):
            with pytest.raises(ValueError):
                call(scale=bad)
    for name, bad in (("logit_bias", f32.bfloat16()), ("gates_out", f32.bfloat16()),
                      ("ids_out", i32.long()), ("demand_out", i32.long()),
                      ("offsets_out", f32), ("ids_out", i32)):
        with pytest.raises(ValueError):
            few(**{name: bad})


def test_an_older_library_asks_for_a_rebuild(native, tmp_path, monkeypatch):
    """A library of the same ABI version from before an entry point was added, and one of another
    version: the message says what to do."""
    import subprocess
    older = [n for n in native.EXPORTS if n not in ("moe_forward_few", "moe_adapter_linear")]
    for version, names, text in ((native.ABI_VERSION, older, "lacks moe_forward_few, moe_adapter"),
                                 (native.ABI_VERSION - 1, native.EXPORTS, "ABI version")):
        src, so = tmp_path / f"v{version}.c", tmp_path / f"v{version}.so"
        src.write_text("".join(f"int {n}(void) {{ return {version}; }}\n" for n in names))
        subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", str(so)], check=True)
        monkeypatch.setattr(native, "_lib", None)
        monkeypatch.setattr(native, "LIB_PATH", str(so))
        with pytest.raises(ImportError, match=f"{text}.*rebuild"):
            native.lib()
