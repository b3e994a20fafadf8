"""The paged cache's entry points on the CPU: their workspaces, and the status codes with which
they reject invalid arguments before anything is launched."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "fp8_precision_amd", "libfp8_precision.so")

OK, INVALID, UNSUPPORTED = 0, 1, 2
# Well-aligned addresses far apart; validation rejects each call, so none is dereferenced.
K, V, KS, VS, TABLE, LENGTHS, BOUNDS, A, B, LSE, TOP, WS = (0x10000000 * i for i in range(1, 13))
i64, i32, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p


class Tensor(ctypes.Structure):
    _fields_ = [("data", vp), ("token_stride", i64), ("head_stride", i64)]


class Cache(ctypes.Structure):
    _fields_ = [("k", vp), ("v", vp), ("k_scale", vp), ("v_scale", vp), ("table", vp), ("lengths", vp), ("bounds", vp),
                ("pages", i64), ("heads", i64), ("page_tokens", i64), ("head_dim", i64), ("batch", i64), ("blocks", i64),
                ("tokens", i64)]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        pytest.fail(f"{LIB} not built: run `python fp8_precision_amd/build.py`")
    lib = ctypes.CDLL(LIB)
    pt, pc, pn = ctypes.POINTER(Tensor), ctypes.POINTER(Cache), ctypes.POINTER(i64)
    for name, args in {
        "fp8_kv_cache_write": [pc, pt, pt, vp],
        "fp8_kv_cache_read": [pc, pt, pt, vp],
        "fp8_attention_cached_workspace": [pc, i64, pn],
        "fp8_attention_cached": [pc, pt, pt, i64, i32, ctypes.c_float, vp, vp, vp, i64, vp],
    }.items():
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = i32
    lib.fp8_last_error.restype = ctypes.c_char_p
    return lib


def cache(**change):
    c = Cache(K, V, KS, VS, TABLE, LENGTHS, BOUNDS, 10, 2, 64, 64, 3, 4, 7)
    for k, v in change.items():
        setattr(c, k, v)
    return c


def tensor(data, **change):
    t = Tensor(data, 2 * 64, 64)
    for k, v in change.items():
        setattr(t, k, v)
    return t


SHAPES = [
    (INVALID, dict(pages=0)), (INVALID, dict(heads=0)), (INVALID, dict(head_dim=0)), (INVALID, dict(batch=-1)),
    (INVALID, dict(blocks=0)), (INVALID, dict(tokens=0)), (INVALID, dict(page_tokens=0)),
    (UNSUPPORTED, dict(page_tokens=48)), (UNSUPPORTED, dict(page_tokens=8)), (UNSUPPORTED, dict(page_tokens=256)),
    (UNSUPPORTED, dict(head_dim=60)), (UNSUPPORTED, dict(head_dim=136)), (UNSUPPORTED, dict(pages=1 << 31)),
    (UNSUPPORTED, dict(heads=1 << 17)), (UNSUPPORTED, dict(batch=(1 << 20) + 1)), (UNSUPPORTED, dict(tokens=1 << 31)),
    (UNSUPPORTED, dict(blocks=(1 << 24) + 1)),           # 2^30 tokens and a page of 64
    (INVALID, dict(bounds=None)),                        # 7 tokens of 3 sequences
]
POINTERS = [(INVALID, {n: None}) for n in ("k", "v", "k_scale", "v_scale", "table", "lengths")] + \
    [(UNSUPPORTED, {n: p + 2}) for n, p in (("k", K), ("v", V), ("table", TABLE), ("lengths", LENGTHS), ("bounds", BOUNDS))]


@pytest.mark.parametrize("call", ["write", "read"])
def test_move(lib, call):
    f = getattr(lib, f"fp8_kv_cache_{call}")
    no = lambda c=None, k=None, v=None: f(c or cache(), k or tensor(A), v or tensor(B), None)
    assert f(None, tensor(A), tensor(B), None) == INVALID
    for status, change in SHAPES + POINTERS:
        assert no(cache(**change)) == status, change
        assert call.encode() in lib.fp8_last_error()
    assert no(k=tensor(None)) == INVALID and no(v=tensor(None)) == INVALID
    assert no(k=tensor(A + 8)) == UNSUPPORTED and no(k=tensor(A, token_stride=100)) == UNSUPPORTED
    assert no(v=tensor(B, head_stride=4)) == UNSUPPORTED and no(v=tensor(B, token_stride=32)) == INVALID
    assert no(k=tensor(K)) == INVALID and b"overlap" in lib.fp8_last_error()
    assert no(v=tensor(KS)) == INVALID
    if call == "write":
        assert no(cache(v=K + 1024)) == INVALID and no(cache(k_scale=V)) == INVALID and no(cache(table=K)) == INVALID
    else:
        assert no(v=tensor(A)) == INVALID and no(v=tensor(A + 128)) == INVALID     # outputs that share elements
        assert no(k=tensor(A, head_stride=0)) == INVALID
        assert no(k=tensor(TABLE)) == INVALID and no(k=tensor(LENGTHS)) == INVALID and no(v=tensor(BOUNDS)) == INVALID


def test_attention(lib):
    n = i64()
    size = lambda c=None, hq=4: lib.fp8_attention_cached_workspace(c or cache(), hq, ctypes.byref(n))
    assert size() == OK and n.value == 0                 # 14 rows, 256 keys at most: no head of a sequence is shared out
    assert size(cache(blocks=100)) == OK and n.value > 0
    assert lib.fp8_attention_cached_workspace(None, 4, ctypes.byref(n)) == INVALID
    assert lib.fp8_attention_cached_workspace(cache(), 4, None) == INVALID
    for status, change in SHAPES:
        assert size(cache(**change)) == status, change
    assert size(hq=3) == INVALID and size(hq=0) == INVALID and size(hq=1 << 17) == UNSUPPORTED
    assert size(cache(tokens=(1 << 31) - 1)) == UNSUPPORTED          # 2^33 rows
    assert size(cache(batch=1 << 20, blocks=1 << 9)) == OK
    assert size(cache(batch=1 << 20, blocks=1 << 10)) == UNSUPPORTED and b"too many" in lib.fp8_last_error()
    assert size(cache(blocks=100)) == OK
    need = n.value
    assert need > 0
    base = dict(cache=cache(blocks=100), q=tensor(A, token_stride=256), out=tensor(B, token_stride=256), hq=4, causal=1, scale=0.125, lse=LSE,
                absmax=TOP, workspace=WS, bytes=need, stream=None)
    no = lambda **c: lib.fp8_attention_cached(*{**base, **c}.values())
    for status, change in SHAPES + POINTERS:
        assert no(cache=cache(**{"blocks": 100, **change})) == status, change
    assert no(lse=None) == INVALID and no(workspace=None) == INVALID and no(bytes=need - 1) == INVALID
    assert no(hq=5) == INVALID and no(causal=2) == INVALID
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert no(scale=bad) == INVALID
    assert no(lse=LSE + 2) == UNSUPPORTED and no(absmax=TOP + 1) == UNSUPPORTED and no(workspace=WS + 8) == UNSUPPORTED
    assert no(out=tensor(A, token_stride=256)) == INVALID and no(out=tensor(K, token_stride=256)) == INVALID
    assert no(lse=K) == INVALID and no(absmax=LSE) == INVALID and no(workspace=V) == INVALID and no(lse=A) == INVALID
    assert no(out=tensor(B, token_stride=256, head_stride=0)) == INVALID       # heads on top of one another
    assert no(q=tensor(A + 8, token_stride=256)) == UNSUPPORTED


def test_attention_scale(lib):
    """The kernel works with scale log2 e, which has to be finite (a score of 0 would be a NaN)."""
    n = i64()
    c = cache(blocks=100)
    assert lib.fp8_attention_cached_workspace(c, 4, ctypes.byref(n)) == OK
    call = lambda scale, out: lib.fp8_attention_cached(c, tensor(A, token_stride=256), out, 4, 1, scale, LSE, TOP, WS, n.value, None)
    bad_out = tensor(B + 8, token_stride=256)            # refused after the scale: nothing is launched
    for scale in (2.4e38, 2.5e38, 3.0e38, 3.4e38):
        assert call(scale, bad_out) == INVALID and b"scale" in lib.fp8_last_error(), scale
    for scale in (1e-45, 1.0, 2.3e38):
        assert call(scale, bad_out) == UNSUPPORTED and b"scale" not in lib.fp8_last_error(), scale
