"""The launches that a call of libengram.so makes, without a GPU: the library in a process of its own, over
tests/launch_recorder.c instead of the HIP runtime's launches.

    with Library(tmp_path) as lib:
        status, launches = lib.call("engram_embed", [...], fail_at=None)

`launches` is a list of (grid x, y, z, block x, y, z).  Pointers are plain numbers, which nothing follows."""
import json
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
LIB = os.path.join(os.path.dirname(HERE), "gram_hash_embedding_amd", "libengram.so")

_CHILD = r"""
import ctypes, json, sys
rec = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)  # ahead of the runtime, whose launch calls it takes over
lib = ctypes.CDLL(sys.argv[2])
KINDS = {"p": ctypes.c_void_p, "i64": ctypes.c_int64, "i32": ctypes.c_int32, "f32": ctypes.c_float}
for line in sys.stdin:
    q = json.loads(line)
    args = []
    for kind, v in q["args"]:
        if kind.endswith("[]"):
            args.append((KINDS[kind[:-2]] * len(v))(*v))
        else:
            args.append(KINDS[kind](v))
    f = getattr(lib, q["name"])
    f.restype = ctypes.c_int64 if q["name"].endswith("_bytes") else ctypes.c_int
    rec.recorder_reset(-1 if q["fail_at"] is None else q["fail_at"])
    status = f(*args)
    out = (ctypes.c_uint32 * 6)()
    launches = []
    for i in range(rec.recorder_count()):
        rec.recorder_get(i, out)
        launches.append(list(out))
    print(json.dumps([status, launches]), flush=True)
"""


class Library:
    def __init__(self, tmp_path):
        self.rec = os.path.join(str(tmp_path), "launch_recorder.so")
        subprocess.run(["gcc", "-std=c11", "-O1", "-shared", "-fPIC", "-Wall", "-o", self.rec,
                        os.path.join(HERE, "launch_recorder.c")], check=True, capture_output=True, text=True)

    def __enter__(self):
        self.child = subprocess.Popen([sys.executable, "-c", _CHILD, self.rec, LIB], stdin=subprocess.PIPE,
                                      stdout=subprocess.PIPE, text=True)
        return self

    def __exit__(self, *_):
        self.child.stdin.close()
        self.child.wait(timeout=60)

    def call(self, name, args, fail_at=None):
        """args: (kind, value) with kind one of p, i64, i32, f32, or of those with [] for a host array."""
        self.child.stdin.write(json.dumps(dict(name=name, args=args, fail_at=fail_at)) + "\n")
        self.child.stdin.flush()
        status, launches = json.loads(self.child.stdout.readline())
        return status, [tuple(x) for x in launches]
