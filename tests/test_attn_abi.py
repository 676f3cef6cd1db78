"""The attention entry points without a GPU: exported, declared to the binding, and
refusing bad arguments on the host; the rotary table against its formula."""
import ctypes
import math
import os
import re

import numpy as np
import pytest

from fp8_scaled_gemm_sm_gb300 import binding, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def test_exports(lib):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "scaled_attention.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(scaled_attn_\w+)\s*\(", src))
    assert {"scaled_attn_create", "scaled_attn_append", "scaled_attn_decode", "scaled_attn_prompt"} <= names
    raw = ctypes.CDLL(binding.LIB_PATH)
    for n in names:
        assert hasattr(raw, n) and n in binding.SIGNATURES, n


@pytest.mark.parametrize("hq,hk,d,page,status", [
    (0, 1, 64, 16, 1), (4, 0, 64, 16, 1), (4, 2, 0, 16, 1), (4, 2, 64, 0, 1),
    (4, 3, 64, 16, 2), (2048, 1, 64, 16, 2), (4, 2, 72, 16, 2), (4, 2, 256, 16, 2), (4, 2, 64, 24, 2), (4, 2, 64, 256, 2),
])
def test_create_refuses(lib, hq, hk, d, page, status):
    with pytest.raises(binding.ScaledGemmError) as e:
        binding.scaled_attn_create(hq, hk, d, page)
    assert e.value.status == status


def test_null_handles_are_refused(lib):
    assert lib.scaled_attn_create(None, 4, 2, 64, 16, -1) == 1
    assert lib.scaled_attn_destroy(None) == 0
    assert lib.scaled_attn_append(None, None, None, *[None, 0] * 3, None, 0, None, None, 0, 0, None, None, None) == 1
    assert lib.scaled_attn_decode(None, None, None, 0, 1, None, 0, None, 0, 1.0, None, None, None) == 1
    assert lib.scaled_attn_prompt(None, *[None, 0] * 3, None, None, 0, 0, 0, 1, 1.0, None, None, None) == 1
    assert lib.scaled_attn_debug_status(None, None, None, None) == 1


def test_rotary_table():
    from fp8_scaled_gemm_sm_gb300 import rotary_table

    t = rotary_table(50, 32, base=500.0, device="cpu").numpy()
    assert t.shape == (50, 2, 16)
    for p in (0, 1, 49):
        for i in range(16):
            a = p * 500.0 ** (-2 * i / 32)
            assert abs(t[p, 0, i] - math.cos(a)) < 1e-7 and abs(t[p, 1, i] - math.sin(a)) < 1e-7
    lin = rotary_table(50, 32, base=500.0, scaling=("linear", 4), device="cpu").numpy()
    assert np.allclose(lin[48], t[12], atol=1e-7)
    parts = rotary_table(50, 32, base=500.0, scaling=("parts", 4, 1.0, 8.0, 100), device="cpu").numpy()
    turns = 100 * 500.0 ** (-2 * np.arange(16) / 32) / (2 * math.pi)
    fast, slow = turns >= 8, turns <= 1
    assert fast.any() and slow.any()
    assert np.array_equal(parts[7][:, fast], t[7][:, fast])
    assert np.allclose(parts[48][:, slow], t[12][:, slow], atol=1e-7)
