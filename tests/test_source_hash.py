"""The bench's source hash, which ties the measured traffic of the interpreter to its code, follows the interpreter's files
and no others."""
import os
import re
import shutil

import bench
from persistent_megakernel_decode_gb300 import build as b

ROOT = bench.ROOT


def included(name, seen):
    """name and the files of csrc it includes, at any depth."""
    if name not in seen:
        seen.add(name)
        with open(os.path.join(b.CSRC, name)) as f:
            for x in re.findall(r'#include "([\w.]+)"', f.read()):
                if os.path.exists(os.path.join(b.CSRC, x)):
                    included(x, seen)
    return seen


def test_interpreter_files_and_serving_files():
    own = set()
    for f in b.SOURCES:
        if f not in b.SERVING:
            included(f, own)
    assert own == set(b.SOURCES + b.HEADERS) - set(b.SERVING)
    assert "interp.cu" in own and set(b.SERVING) <= set(b.SOURCES + b.HEADERS)


def test_hash_follows_the_interpreter_only(tmp_path):
    root = str(tmp_path)
    csrc = os.path.join(root, "persistent_megakernel_decode_gb300", "csrc")
    shutil.copytree(b.CSRC, csrc)
    shutil.copytree(os.path.join(ROOT, "include"), os.path.join(root, "include"))
    h = bench.kernel_source_hash(root)
    assert h == bench.kernel_source_hash()

    def edited(path, old, new):
        with open(path) as f:
            s = f.read()
        assert old in s
        with open(path, "w") as f:
            f.write(s.replace(old, new, 1))
        now = bench.kernel_source_hash(root)
        with open(path, "w") as f:
            f.write(s)
        return now
    mk = os.path.join(root, "include", "mk.h")
    for f in b.SERVING:
        assert edited(os.path.join(csrc, f), "a", "b") == h
    assert edited(mk, "Attention of new tokens over one layer", "x") == h
    for f in set(b.SOURCES + b.HEADERS) - set(b.SERVING):
        assert edited(os.path.join(csrc, f), "a", "b") != h
    assert edited(mk, "mk_run(", "mk_runs(") != h and edited(mk, "mk_last_error", "mk_first_error") != h
