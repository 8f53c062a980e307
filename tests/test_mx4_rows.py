"""The token rows that the projection on 4-bit weights loads, followed on the host: every load of every tile, stage and count of
rows fetches what its slot holds and nothing behind the last row."""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "gram_hash_embedding_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not installed")
def test_every_load_of_a_tile(tmp_path):
    exe = tmp_path / "mx4_rows_check"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Xlinker", "--no-undefined", f"-I{CSRC}", "-o", str(exe),
                    os.path.join(HERE, "mx4_rows_check.cc")], check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout == "", r.stdout


def test_loads_carry_no_scalar_offset():
    """What the check above follows is all of a load's offset: the scalar operand, which the range check may or may not cover, is
    zero in every load and store of the file, by a resource that ends with the rows."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "wkv_mx4.hip")).read())
    calls = {}
    for m in re.finditer(r"__builtin_amdgcn_raw_(?:ptr_)?buffer_(load_lds|load_b128|load_b32|store_b128)\(", text):
        depth, args, arg = 1, [], ""
        for ch in text[m.end():]:
            depth += {"(": 1, "[": 1, ")": -1, "]": -1}.get(ch, 0)
            if depth == 0:
                break
            if ch == "," and depth == 1:
                args.append(arg.strip())
                arg = ""
            else:
                arg += ch
        args.append(arg.strip())
        scalar = {"load_lds": 4, "load_b128": 2, "load_b32": 2, "store_b128": 3}[m.group(1)]
        calls.setdefault(m.group(1), []).append(args[scalar])
    assert calls == {"load_lds": ["0"] * 3, "load_b128": ["0"], "load_b32": ["0"], "store_b128": ["0"]}
