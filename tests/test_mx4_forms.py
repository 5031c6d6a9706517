"""Which form of the product of CTA pairs serves a shape, asked of the library's
own rule (a test-hook build; host arithmetic, no GPU).  FORMS is what
tests/test_gpu_mx4_forms.py runs: every form the rule knows, with several rounds
of tiles on the 74 clusters where the rule lets the form have them, and a K that
ends inside a stage.  A change of the rule that leaves a form out of these
tests fails here."""
import ctypes

import pytest

CLUSTERS = 74
OUT = {"bf16": 0, "fp16": 1, "fp32": 2}

# form (0 rows, 1 columns, 8 sliced bf16 rows), rows of B a tile, least rounds; M, N, K, columns Y is wider than N
FORMS = [
    (0, 256, 4, 2165, 6248, 1056, 0),
    (0, 256, 4, 4096, 4096, 1216, 8),
    (0, 256, 5, 5131, 4160, 544, 0),
    (0, 192, 4, 3330, 3952, 1056, 0),
    (0, 192, 4, 1837, 6976, 1184, 16),
    (0, 128, 2, 800, 4688, 1056, 0),
    (0, 128, 1, 300, 1280, 2080, 0),
    (1, 192, 4, 4262, 2312, 1056, 1),
    (1, 192, 4, 5192, 2001, 1216, 0),
    (1, 128, 3, 4643, 1360, 1056, 1),
    (1, 128, 1, 333, 4999, 1056, 0),
    (1, 64, 1, 2325, 320, 1056, 1),
    (1, 64, 1, 385, 321, 1056, 0),
    (8, 192, 6, 600, 4100, 1056, 0),
    (8, 192, 4, 500, 3001, 1216, 0),
    (8, 192, 3, 1000, 1100, 1056, 3),
    (8, 208, 1, 100, 4096, 1056, 0),
    (8, 256, 1, 128, 4604, 1184, 1),
]


def hooks():
    from tests.test_gpu_timeout import _hooks_lib
    L = _hooks_lib()
    I64, I = ctypes.c_int64, ctypes.c_int
    L.mq_test_mx4_plan.argtypes = [I64, I64, I64, I, I64, I, ctypes.POINTER(I64)]
    return L


def plan(L, M, N, K, out, ldy, bf16_rows):
    """(form, rows of B a tile, tiles); form -1: the kernel for few rows."""
    t = (ctypes.c_int64 * 3)()
    form = L.mq_test_mx4_plan(M, N, K, OUT[out], ldy, bf16_rows, t)
    return form, t[0], t[1] * t[2]


@pytest.mark.parametrize("form,bn,rounds,M,N,K,wider", FORMS)
def test_the_shapes_take_the_forms_they_stand_for(form, bn, rounds, M, N, K, wider):
    L = hooks()
    for out in OUT:
        got, width, tiles = plan(L, M, N, K, out, N + wider, form == 8)
        assert (got, width) == (form, bn)
        assert -(-tiles // CLUSTERS) >= rounds and K % 256


def test_every_form_of_the_rule_is_in_the_list():
    L = hooks()
    have = {(f, bn if f != 8 else bn > 192) for f, bn, *_ in FORMS}
    for M in range(129, 5200, 173):
        for N in (8, 136, 1000, 3001, 4096, 6976):
            for K in (64, 1056, 14336):
                for ldy in (N, N + 1):
                    f, bn, _ = plan(L, M, N, K, "bf16", ldy, 0)
                    assert (f, bn) in have, (M, N, K, ldy)
                f, bn, _ = plan(L, M, N, K, "bf16", N, 1)
                assert (f, bn > 192) in have and bn <= 256
    assert plan(L, 128, 4096, 4096, "bf16", 4096, 0)[0] == plan(L, 16, 4096, 4096, "bf16", 4096, 1)[0] == -1
