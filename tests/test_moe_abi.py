"""The calls of the expert layer for many tokens (include/bakron_moe.h) on the
CPU: exports, constants, sizes, every host-side refusal."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "bakron_moe.h")
FAKE = ctypes.c_void_p(4096)          # never dereferenced: every call below returns from its host checks
ODD, HALF = ctypes.c_void_p(4097), ctypes.c_void_p(4098)
BF16, FP16, F32 = 0, 1, 2


@pytest.fixture(scope="module")
def L():
    import two_sided_hessian_amd as B
    if not os.path.exists(B.LIB_PATH):
        from two_sided_hessian_amd import build
        build.build()
    return B.lib()


def test_every_declared_call_is_exported_and_bound(L):
    from two_sided_hessian_amd._binding import SIGNATURES
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(bakron_\w+)\s*\(", src))
    assert len(names) == 15
    for name in names:
        assert hasattr(L, name) and name in SIGNATURES, name
        # as many arguments as are declared
        args = re.search(name + r"\s*\((.*?)\)", src, re.S).group(1).split(",")
        assert len(SIGNATURES[name][1]) == len(args), name


def test_constants_match():
    from two_sided_hessian_amd import moe
    found = re.findall(r"#define\s+(BAKRON_MOE_[A-Z0-9_]+)\s+(\d+)", open(HEADER).read())
    assert len(found) == 7
    for k, v in found:
        assert getattr(moe, k) == int(v), k


def check(call, ok, null=(), size=(), arg=(), done=()):
    """Each change of the arguments `ok` is refused with its code; `done` ones
    are calls with nothing to do."""
    def with_(at):
        a = list(ok)
        for k, v in at.items():
            a[k] = v
        return call(*a)
    for k in null:
        assert with_({k: None}) == -1, k
    for code, cases in ((-2, size), (-4, arg), (0, done)):
        for at in cases:
            assert with_(at) == code, (code, at)


MOST = 16777216


def test_route_refusals(L):
    # logits, ld, tokens, type, experts, top_k, ids, weights, place, order, offsets, ws, bytes, stream
    ok = [FAKE, 64, 300, F32, 64, 6, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 40, None]
    check(L.bakron_moe_route, ok, null=(0, 6, 7, 8, 9, 10),
          size=[{2: -1}, {2: MOST + 1, 5: 1}, {2: MOST // 6 + 1}],
          arg=[{1: 63}, {1: 1 << 32}, {3: 3}, {3: -1}, {4: 0}, {4: 257, 1: 257}, {4: 5, 5: 6}, {5: 0}, {5: 17}, {5: -1}, {0: HALF},
               {3: BF16, 0: ODD}, {6: HALF}, {7: HALF}, {8: HALF}, {9: HALF}, {10: HALF}])
    need = L.bakron_moe_route_workspace_bytes(300, 64, 6)
    assert need > 0 and L.bakron_moe_route_workspace_bytes(1, 64, 6) == 0
    for at in ({12: need - 1}, {11: None}, {11: ctypes.c_void_p(4096 + 64)}):
        a = list(ok)
        for k, v in at.items():
            a[k] = v
        assert L.bakron_moe_route(*a) == -3, at
    for bad in ((0, 64, 6), (-1, 64, 6), (300, 0, 1), (300, 257, 6), (300, 4, 5), (300, 64, 0), (300, 64, 17), (MOST, 64, 2)):
        assert L.bakron_moe_route_workspace_bytes(*bad) == 0, bad
    assert 0 < L.bakron_moe_route_workspace_bytes(MOST, 256, 1) < 1 << 20
    # dweights, weights, ids, tokens, experts, top_k, dlogits, ld, type, stream
    ok = [FAKE, FAKE, FAKE, 300, 64, 6, FAKE, 64, BF16, None]
    check(L.bakron_moe_route_grad, ok, null=(0, 1, 2, 6), size=[{3: -1}, {3: MOST}],
          arg=[{7: 63}, {8: 3}, {4: 257, 7: 257}, {5: 65}, {5: 0}, {6: ODD}, {8: F32, 6: HALF}, {0: HALF}, {1: HALF}, {2: HALF}],
          done=[{3: 0, 0: None, 6: None}])


def test_rows_refusals(L):
    # x, ldx, tokens, type, cols, top_k, place, xs, ldxs, rows, stream
    ok = [FAKE, 100, 30, BF16, 100, 2, FAKE, FAKE, 100, 60, None]
    check(L.bakron_moe_gather, ok, null=(0, 6, 7),
          size=[{2: -1}, {2: MOST + 1}, {4: -1}, {4: 65537, 1: 65537, 8: 65537}, {9: -1}, {9: 2 * MOST + 1}],
          arg=[{1: 99}, {8: 99}, {1: 1 << 32}, {8: 1 << 32}, {3: F32}, {3: -1}, {5: 0}, {5: 33}, {0: ODD}, {7: ODD}, {6: HALF}],
          done=[{2: 0, 0: None}, {4: 0, 7: None}, {9: 0, 7: None}])
    # ys, ldys, rows, type, cols, top_k, place, weights, tokens, y, ldy, stream
    ok = [FAKE, 100, 60, FP16, 100, 2, FAKE, FAKE, 30, FAKE, 100, None]
    check(L.bakron_moe_combine, ok, null=(0, 6, 9),
          size=[{8: -1}, {8: MOST + 1}, {4: -1}, {2: -1}, {2: 2 * MOST + 1}],
          arg=[{1: 99}, {10: 99}, {3: F32}, {5: 0}, {5: 33}, {0: ODD}, {9: ODD}, {6: HALF}, {7: HALF}],
          done=[{8: 0, 9: None}, {4: 0, 0: None}])
    # dy, lddy, ys, ldys, rows, type, cols, top_k, place, weights, tokens, dys, lddys, dweights, stream
    ok = [FAKE, 100, FAKE, 100, 60, BF16, 100, 2, FAKE, FAKE, 30, FAKE, 100, FAKE, None]
    check(L.bakron_moe_combine_grad, ok, null=(0, 2, 8, 9, 11, 13), size=[{10: -1}, {4: -1}, {6: -1}],
          arg=[{1: 99}, {3: 99}, {12: 99}, {5: F32}, {7: 0}, {7: 33}, {0: ODD}, {2: ODD}, {11: ODD}, {9: HALF}, {13: HALF}],
          done=[{10: 0, 13: None}])


@pytest.mark.parametrize("name,cols_in,cols_out", [("bakron_q4_experts", 7, 6), ("bakron_q4_experts_grad", 6, 7)])
def test_experts_refusals(L, name, cols_in, cols_out):
    call, bytes_ = getattr(L, name), getattr(L, name + "_workspace_bytes")
    # in, ld, rows, type, packed, experts, m, n, group_size, offsets, out, ld, ws, bytes, stream
    ok = [FAKE, 1000, 3000, BF16, FAKE, 8, 1000, 1000, 64, FAKE, FAKE, 1000, FAKE, 1 << 40, None]
    check(call, ok, null=(0, 4, 9, 10),
          size=[{2: -1}, {2: MOST + 1}, {6: -1}, {7: 65537, 1: 65537, 11: 65537}, {6: 65537, 1: 65537, 11: 65537}],
          arg=[{1: 999}, {11: 999}, {1: 1 << 32}, {3: F32}, {3: 3}, {5: 0}, {5: 257}, {8: 63}, {8: -64}, {0: ODD}, {10: ODD}, {9: HALF},
               {4: ctypes.c_void_p(4096 + 128)}],
          done=[{2: 0, 0: None}, {cols_out: 0, 10: None}])
    need = bytes_(3000, 8, 1000, 1000, 64)
    assert need > 0
    for at in ({13: need - 1}, {12: None}, {12: ctypes.c_void_p(4096 + 16)}):
        a = list(ok)
        for k, v in at.items():
            a[k] = v
        assert call(*a) == -3, at
    for bad in ((0, 8, 64, 64, 0), (-1, 8, 64, 64, 0), (9, 0, 64, 64, 0), (9, 257, 64, 64, 0), (9, 8, 0, 64, 0), (9, 8, 64, 65537, 0),
                (9, 8, 64, 64, 7)):
        assert bytes_(*bad) == 0, bad
    # beyond 32 bits
    assert bytes_(MOST, 8, 14336, 4099, 64) >= 2 * MOST * 4099


def test_checkpoint_and_gated_refusals(L):
    size = L.bakron_ck8_bytes
    assert size(3, 33) == 256 + 256                      # 3 x 64 codes, 3 x 2 steps
    assert size(16384, 14336) == 16384 * 14336 // 32 * 33
    assert size(MOST, 65536) == MOST * 65536 // 32 * 33
    for bad in ((0, 5), (5, 0), (-1, 5), (MOST + 1, 5), (5, 65537)):
        assert size(*bad) == 0, bad
    off = ctypes.c_void_p(4096 + 128)
    # x, ldx, rows, type, cols, ck, stream
    check(L.bakron_ck8_pack, [FAKE, 100, 30, BF16, 100, FAKE, None], null=(0, 5), size=[{2: -1}, {4: 65537}],
          arg=[{1: 99}, {3: F32}, {0: ODD}, {5: off}], done=[{2: 0, 0: None}, {4: 0, 5: None}])
    # ck, rows, cols, type, x, ldx, stream
    check(L.bakron_ck8_unpack, [FAKE, 30, 100, F32, FAKE, 100, None], null=(0, 4), size=[{1: -1}, {2: 65537}],
          arg=[{5: 99}, {3: 3}, {4: HALF}, {3: FP16, 4: ODD}, {0: off}], done=[{1: 0, 0: None}])
    # a, lda, b, ldb, rows, type, cols, act, count, h, ldh, ck_a, ck_b, stream
    check(L.bakron_gated_act, [FAKE, 100, FAKE, 100, 30, BF16, 100, 0, None, FAKE, 100, FAKE, FAKE, None], null=(0, 2, 9),
          size=[{4: -1}, {4: MOST + 1}, {6: -1}, {6: 65537}],
          arg=[{1: 99}, {3: 99}, {10: 99}, {5: F32}, {7: 2}, {7: -1}, {0: ODD}, {2: ODD}, {9: ODD}, {8: HALF}, {11: None}, {12: None},
               {11: off}, {12: off}],
          done=[{4: 0, 0: None}, {6: 0, 9: None}])
    # dh, lddh, ck_a, ck_b, rows, type, cols, act, count, da, ldda, db, lddb, stream
    check(L.bakron_gated_act_grad, [FAKE, 100, FAKE, FAKE, 30, BF16, 100, 1, None, FAKE, 100, FAKE, 100, None],
          null=(0, 2, 3, 9, 11), size=[{4: -1}, {6: 65537}],
          arg=[{1: 99}, {10: 99}, {12: 99}, {5: F32}, {7: 2}, {0: ODD}, {9: ODD}, {11: ODD}, {8: HALF}, {2: off}, {3: off}],
          done=[{4: 0, 0: None}])
