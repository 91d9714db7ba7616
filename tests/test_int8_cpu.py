"""Refusals of the 8-bit cache that need no device."""
import ctypes
import os
import re

import pytest

from paged_kv_attention_25_gb300 import build as pkv_build
from paged_kv_attention_25_gb300 import pkv


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return pkv.load_library()


def test_int8_storage_and_exponents_go_together(lib):
    mem = ctypes.create_string_buffer(64)
    at = (ctypes.addressof(mem) + 15) // 16 * 16
    for k, v, ke, ve in [(at, at, None, None), (at, at, at, None), (None, None, at, at), (at, None, at, at)]:
        desc = pkv.pkv_pool_desc(1, 16, 1, 64, pkv.PKV_DTYPE_INT8, k, v, 1.0, 1.0, ke, ve)
        h = ctypes.c_void_p()
        assert lib.pkv_pool_create(ctypes.byref(desc), ctypes.byref(h)) == pkv.PKV_EINVAL
        assert not h.value


def test_calls_without_a_pool_are_refused(lib):
    assert lib.pkv_append_int8(None, None, 1, 1, None, None, None, None, None, 1, None) == pkv.PKV_EINVAL
    assert lib.pkv_read_rows(None, None, 1, 1, None, None, 1, None, None, None) == pkv.PKV_EINVAL
    assert lib.pkv_pool_exps(None, None, None) == pkv.PKV_EINVAL
    assert "pool" in pkv.pkv_last_error()


def test_binding_calls_let_go_of_the_interpreter():
    csrc = os.path.join(os.path.dirname(pkv.__file__), "csrc")
    with open(os.path.join(csrc, "binding_score.h")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    names = {"append_int8", "read_rows", "score_attn"}
    assert set(re.findall(r"run\(pkv_(\w+), p->handle", text)) == names
    assert not names & set(re.findall(r"pkv_(\w+)\(", text))


def test_only_metadata_is_read_through_the_non_coherent_path():
    """Rows, codes and exponents may be what the kernel ahead wrote."""
    csrc = os.path.join(os.path.dirname(pkv.__file__), "csrc")
    with open(os.path.join(csrc, "int8.cu")) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert {m.group(1) for m in re.finditer(r"__ldg\(\s*([A-Za-z_.]+|reinterpret_cast)", code)} <= {"pos", "cu", "bt", "held_lens"}
