"""The 4-bit layer calls of libbakron.so (include/bakron_q4.h) on the CPU:
exports, constants, sizes, every host-side refusal."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "bakron_q4.h")
FAKE = ctypes.c_void_p(4096)          # never dereferenced: every call below returns from its host checks


@pytest.fixture(scope="module")
def B():
    import two_sided_hessian_amd as B
    if not os.path.exists(B.LIB_PATH):
        from two_sided_hessian_amd import build
        build.build()
    return B


def _declared():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(bakron_\w+)\s*\(", src)))


def test_every_declared_call_is_exported_and_bound(B):
    from two_sided_hessian_amd._binding import SIGNATURES
    names = _declared()
    assert len(names) == 8
    for name in names:
        assert hasattr(B.lib(), name) and name in SIGNATURES, name


def test_constants_match(B):
    from two_sided_hessian_amd import q4
    for k, v in re.findall(r"#define\s+(BAKRON_Q4_[A-Z0-9_]+)\s+(\d+)", open(HEADER).read()):
        assert getattr(q4, k) == int(v), k


def test_sizes(B):
    L = B.lib()
    size = L.bakron_q4_packed_bytes
    assert size(1, 4096, 14336, 128) >= 4096 * 14336 // 2 + 8 * 4096 * 112
    assert size(1, 4096, 14336, 128) <= 4096 * 14336 // 2 + 8 * 4096 * 112 + 1024
    assert size(8, 100, 100, 0) == 8 * size(1, 100, 100, 0)
    assert size(1, 65536, 65536, 64) >= (65536 * 65536) // 2 + 8 * 65536 * 1024    # beyond 32 bits
    for bad in ((1, 65537, 64, 0), (1, 64, -1, 0), (257, 64, 64, 0), (-1, 64, 64, 0), (1, 64, 64, 32), (1, 64, 64, -64),
                (1, 0, 64, 0), (1, 64, 0, 0), (0, 64, 64, 0)):
        assert size(*bad) == 0, bad
    moe = L.bakron_q4_moe_workspace_bytes
    assert moe(1, 4096, 14336, 8, 2, 128) > 0
    assert moe(64, 4096, 14336, 8, 2, 128) > moe(1, 4096, 14336, 8, 2, 128)
    for bad in ((0, 64, 64, 8, 2, 0), (65, 64, 64, 8, 2, 0), (1, 64, 64, 1, 2, 0), (1, 64, 64, 300, 2, 0),
                (1, 64, 64, 64, 17, 0), (1, 64, 64, 8, 0, 0), (1, 64, 64, 8, 2, 65), (1, 64, 65537, 8, 2, 0)):
        assert moe(*bad) == 0, bad
    for call in (L.bakron_q4_linear_workspace_bytes, L.bakron_q4_linear_grad_workspace_bytes):
        assert call(16777216, 65536, 65536, 64) >= 0
        for bad in ((-1, 64, 64, 0), (16777217, 64, 64, 0), (5, 65537, 64, 0), (5, 64, 64, 7)):
            assert call(*bad) == 0, bad


def _with(args, **at):
    a = list(args)
    for k, v in at.items():
        a[int(k[1:])] = v
    return a


def test_pack_refusals(B):
    L = B.lib()
    # codes, scale, zero, count, m, n, group_size, packed, stream
    ok = [FAKE, FAKE, FAKE, 1, 64, 64, 0, FAKE, None]
    for k in (0, 1, 2, 7):
        assert L.bakron_q4_pack(*_with(ok, **{f"_{k}": None})) == -1, k
    assert L.bakron_q4_pack(*_with(ok, _4=65537)) == -2
    assert L.bakron_q4_pack(*_with(ok, _5=-1)) == -2
    assert L.bakron_q4_pack(*_with(ok, _3=257)) == -2
    assert L.bakron_q4_pack(*_with(ok, _3=-1)) == -2
    assert L.bakron_q4_pack(*_with(ok, _6=65)) == -4
    assert L.bakron_q4_pack(*_with(ok, _7=ctypes.c_void_p(4096 + 16))) == -4
    for k in (3, 4, 5):
        assert L.bakron_q4_pack(*_with(ok, **{f"_{k}": 0, "_0": None})) == 0, k


@pytest.mark.parametrize("name,cols_in,cols_out", [("bakron_q4_linear", 6, 5), ("bakron_q4_linear_grad", 5, 6)])
def test_linear_refusals(B, name, cols_in, cols_out):
    call = getattr(B.lib(), name)
    # in, ld, tokens, type, packed, m, n, group_size, out, ld, ws, ws_bytes, stream
    ok = [FAKE, 128, 3, 0, FAKE, 128, 128, 64, FAKE, 128, FAKE, 1 << 40, None]
    for k in (0, 4, 8):
        assert call(*_with(ok, **{f"_{k}": None})) == -1, k
    for at in ({"_2": -1}, {"_2": 16777217}, {"_5": -1}, {"_5": 65537}, {"_6": 65537}):
        assert call(*_with(ok, **at)) == -2, at
    for at in ({"_1": 127}, {"_9": 127}, {"_3": 2}, {"_3": -1}, {"_7": 32}, {"_7": -64}, {"_0": ctypes.c_void_p(4097)},
               {"_8": ctypes.c_void_p(4097)}, {"_4": ctypes.c_void_p(4096 + 128)}, {"_1": 1 << 32}, {"_9": 1 << 40}):
        assert call(*_with(ok, **at)) == -4, at
    assert call(*_with(ok, _2=0, _0=None, _8=None)) == 0
    assert call(*_with(ok, **{f"_{cols_out}": 0, "_8": None})) == 0
    size = getattr(B.lib(), name + "_workspace_bytes")
    for tokens in (1, 300, 4096):
        need = size(tokens, 1000, 1000, 64)
        if need:
            big = _with(ok, _1=1000, _2=tokens, _5=1000, _6=1000, _9=1000)
            assert call(*_with(big, _11=need - 1)) == -3
            assert call(*_with(big, _10=None)) == -3
            assert call(*_with(big, _10=ctypes.c_void_p(4096 + 16))) == -3


def test_moe_refusals(B):
    call = B.lib().bakron_q4_moe
    # x, ldx, tokens, type, router, gate, up, down, hidden, ffn, experts, top_k, group_size, y, ldy, ids, weights, ws, bytes, stream
    ok = [FAKE, 128, 3, 0, FAKE, FAKE, FAKE, FAKE, 128, 256, 8, 2, 64, FAKE, 128, FAKE, FAKE, FAKE, 1 << 40, None]
    for k in (0, 4, 5, 6, 7, 13, 15, 16):
        assert call(*_with(ok, **{f"_{k}": None})) == -1, k
    for at in ({"_2": 65}, {"_2": -1}, {"_8": 65537, "_1": 65537, "_14": 65537}, {"_9": -1}):
        assert call(*_with(ok, **at)) == -2, at
    for at in ({"_3": 3}, {"_10": 0}, {"_10": 257}, {"_11": 0}, {"_11": 9}, {"_10": 64, "_11": 17}, {"_12": 63}, {"_1": 127},
               {"_14": 100}, {"_0": ctypes.c_void_p(4097)}, {"_15": ctypes.c_void_p(4098)},
               {"_6": ctypes.c_void_p(4096 + 128)}):
        assert call(*_with(ok, **at)) == -4, at
    need = B.lib().bakron_q4_moe_workspace_bytes(3, 128, 256, 8, 2, 64)
    assert call(*_with(ok, _18=need - 1)) == -3
    assert call(*_with(ok, _17=None)) == -3
    assert call(*_with(ok, _2=0, _0=None)) == 0
