"""The bytes of an append into blocks, by which large calls choose their kernel, for calls past 2^31 of them.

Evaluated by the host compiler: an expression that overflows is no constant, and the file is not accepted."""

from __future__ import annotations

import os
import subprocess

import pytest

from tests.conftest import ROOT

CASES = [  # tokens, query heads, kv heads, width, queries given
    (4, 32, 8, 128, 1), (65536, 32, 8, 128, 1), (95326, 32, 8, 128, 1), (98304, 32, 8, 128, 1), (196608, 32, 8, 128, 1),
    (55189, 64, 8, 128, 1), (400000, 32, 8, 128, 0), (11184810, 32, 8, 128, 1), (1 << 30, 1, 1, 64, 0)]


@pytest.mark.parametrize("tokens,hq,hkv,width,queries", CASES)
def test_bytes_of_large_appends(tmp_path, tokens, hq, hkv, width, queries):
    want = tokens * width * (2 * hkv * 3 + queries * hq * 4)  # a bf16 number and its code, or two bf16 ones
    src = tmp_path / "bytes.cpp"
    src.write_text(f"""#include "kda_internal.h"
constexpr kda_kv_shape s{{1, {tokens}, {hq}, {hkv}, {width}, {width}, KDA_BF16, KDA_E4M3}};
static_assert(kda::append_blocks_bytes({tokens}, s, {queries}) == {want}LL, "");
""")
    r = subprocess.run(["g++", "-std=c++17", "-fsyntax-only", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
                        "-I", os.path.join(ROOT, "recurrent_state_amd", "csrc"), "-I", "/opt/rocm/include", str(src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
