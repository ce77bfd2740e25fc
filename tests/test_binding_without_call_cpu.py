"""The binding and the build where the binding's native part (_tq2call.so) is
not there: the library is what counts."""
import os
import subprocess
import sys

import pytest

from ternary_packed_weight_amd import build

ROOT = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..")

WITHOUT = r"""
import sys
sys.modules["ternary_packed_weight_amd._tq2call"] = None   # what an import of a module that is not there meets
import torch
from ternary_packed_weight_amd import tq2
assert tq2.tq2_abi_version() > 0 and tq2.tq2_kv4_page_bytes(64, 2, 128) == 2 * 64 * 136

def refused(match, fn, *a, **kw):
    try:
        fn(*a, **kw)
    except ValueError as e:
        assert match in str(e), e
    else:
        raise AssertionError(match)

codes, scales = torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((4, 1), dtype=torch.float16)
refused("device tensor", tq2.tq2_gemv, codes, scales, torch.zeros(256, dtype=torch.float16))
h, pos, inv = torch.zeros((3, 2, 64)), torch.zeros(3, dtype=torch.int32), torch.zeros(32)
cache, slots = torch.zeros((4, 2, 32 * 72), dtype=torch.uint8), torch.zeros(3, dtype=torch.int64)
table = torch.zeros((3, 4), dtype=torch.int32)
refused("device tensor", tq2.tq2_qk_norm_rope, h, h, pos, inv, q_out=torch.empty_like(h), k_out=torch.empty_like(h))
refused("device tensor", tq2.tq2_kv4_store, cache, h, h, slots)
refused("device tensor", tq2.tq2_kv4_load, cache, slots, 64, k_out=torch.empty_like(h), v_out=torch.empty_like(h))
refused("device tensor", tq2.tq2_kv4_attn, h.half(), cache, table, pos, out=torch.empty_like(h.half()))
refused("ctx_len must hold 3", tq2.tq2_kv4_attn, h.half(), cache, table, pos[:2])
print("all calls")
"""


def test_import_without_the_native_part():
    if not os.path.exists(build.LIB):
        build.build()
    r = subprocess.run([sys.executable, "-c", WITHOUT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "all calls" in r.stdout, r.stderr


def test_the_library_is_built_before_the_native_part(monkeypatch):
    made = []

    def fails(verbose):
        made.append("call")
        raise RuntimeError("no g++")

    monkeypatch.setattr(build, "_call", fails)
    monkeypatch.setattr(build, "_hipcc", lambda sources, out, verbose, extra=(): made.append(os.path.basename(out)) or out)
    with pytest.raises(RuntimeError, match="no g"):
        build.build()
    assert made == ["libtq2.so", "libtq2probe.so", "call"]


def test_a_native_part_that_does_not_build_does_not_stay(monkeypatch, tmp_path):
    """One of other sources must not be loaded beside the new library."""
    old = tmp_path / "_tq2call.so"
    old.write_bytes(b"")
    monkeypatch.setattr(build, "CALL_LIB", str(old))
    monkeypatch.setattr(build, "CSRC", str(tmp_path))   # no source there
    with pytest.raises(RuntimeError, match="g.. failed"):
        build._call(False)
    assert not old.exists()
