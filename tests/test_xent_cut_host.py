"""How linear xent's products are cut into units (no GPU needed): every step of
every tile is taken once, and the parts' sums fit the workspace's room."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
FORMS = [(256, 256, 256), (128, 128, 512), (64, 128, 768), (32, 128, 1024)]
STATS, PROB, DX, DW = range(4)


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("cut") / "cut.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-shared", "-fPIC", "-o", so,
                    os.path.join(HERE, "xent_cut_check.cpp")], check=True)
    f = ctypes.CDLL(so).check
    f.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                  ctypes.c_uint32, ctypes.c_uint32, ctypes.c_void_p, ctypes.c_int64]

    def run(form, kind, m, most_m, n, steps, most_steps):
        tm, tn, _ = FORMS[form]
        size = -(-m // tm) * -(-n // tn) * steps
        seen = np.zeros(max(size, 1), np.uint8)
        return f(form, kind, m, most_m, n, steps, most_steps, seen.ctypes.data, size)
    return run


@pytest.mark.parametrize("form", range(4))
@pytest.mark.parametrize("kind", [STATS, PROB, DX, DW])
def test_units_take_everything_once_and_fit(check, form, kind):
    rng = random.Random(100 * form + kind)
    tm, tn, slots = FORMS[form]
    cases = [(1, 1, 1), (0, 5, 3), (tm, tn * slots, 8), (tm, tn * (slots + 1), 9),
             (tm * 3, tn * (slots // 2), 40), (tm * slots, tn, 64), (tm * 24, tn * 16, 33),
             (tm * 24 - 5, tn * 99 - 77, 64), (tm + 1, tn, 0)]
    for _ in range(60):
        cases.append((rng.randint(0, 24 * tm), rng.randint(1, 40 * tn), rng.randint(0, 130)))
    for m, n, steps in cases:
        assert check(form, kind, m, m, n, steps, steps) == 0, (m, n, steps)
        # rows that are left out: fewer rows, or fewer steps of them, than there is room for
        if kind == DW:
            assert check(form, kind, m, m, n, steps // 2, steps) == 0, (m, n, steps)
        else:
            assert check(form, kind, m // 2, m, n, steps, steps) == 0, (m, n, steps)
