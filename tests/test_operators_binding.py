"""The operators' binding, as far as it goes without a GPU: what it raises, what it keeps, what it needs."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    from serving_layer_moe_gb300 import build as b
    if not (os.path.exists(b.LIB) and os.path.exists(b.HOST)):
        b.build()


def run(script, *args):
    """A script in a process of its own, so that an abort fails one test; its output's last line."""
    r = subprocess.run([sys.executable, "-c", script, *args], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr[-2000:])
    return r.stdout.strip().splitlines()[-1]


# Tensors that say they are on a GPU and have no memory: the constructors' own checks pass, reading an address throws.
WITHOUT_MEMORY = """
import sys, torch
from torch._subclasses.fake_tensor import FakeTensorMode
import serving_layer_moe_gb300 as moe
moe.operators._host()
with FakeTensorMode(allow_non_fake_inputs=True):
    i = lambda *s: torch.empty(3, *s, dtype=torch.int32, device="cuda")
    u = lambda *s: torch.empty(3, *s, dtype=torch.uint8, device="cuda")
    def groups(a, b, c, d):
        moe.ExpertGroups(a, b, c, d)
    def rows(a, b):
        moe.FP4Rows(a, b, "mxfp4")
    try:
        if sys.argv[1] == "groups":
            torch.vmap(groups)(i(5), i(5), i(6), i(3, 2))
        else:
            torch.vmap(rows)(u(4, 16), u(1, 1, 512))
    except RuntimeError as e:
        print("raised", type(e).__name__)
"""


@pytest.mark.parametrize("what", ["groups", "rows"])
def test_constructors_raise_on_tensors_without_memory(what):
    assert run(WITHOUT_MEMORY, what).startswith("raised")


# Nine integers look like the description that the binding keeps of groups; as an argument they are nobody's addresses.
NINE_INTEGERS = """
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
import serving_layer_moe_gb300 as moe
nine = (0, 8, 4, 2, 2, 4096, 8192, 12288, 16384)
with FakeTensorMode(allow_non_fake_inputs=True):
    u = lambda *s: torch.empty(*s, dtype=torch.uint8, device="cuda")
    try:
        moe.FP4Rows(u(4, 16), u(4, 1, 512), "mxfp4", groups=nine)
    except ValueError as e:
        print("refused", e)
"""


def test_integers_are_not_groups():
    assert run(NINE_INTEGERS).startswith("refused groups must be ExpertGroups")


def cpu_rows(groups=None):
    """FP4Rows as the binding makes them, of CPU memory that no kernel sees."""
    import torch

    import serving_layer_moe_gb300 as moe
    codes, scales, g = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 1, 512, dtype=torch.uint8), torch.ones(1)
    return moe.FP4Rows._of("nvfp4", groups, (0, 1, 4, 64, 3, codes, scales, g, 1))


def test_copies_of_rows_and_groups_have_their_own_memory():
    """No address is kept: all that a copy holds is its own tensors."""
    import copy
    import pickle

    import torch

    import serving_layer_moe_gb300 as moe
    gr = moe.ExpertGroups._of((0, 4, 4, 2, 2, torch.zeros(18, dtype=torch.int32), 0, None, None))
    q = cpu_rows(gr)
    for d in (copy.deepcopy(q), pickle.loads(pickle.dumps(q))):
        mine = [q.codes, q.scales, q.g, q.groups._c[5]]
        theirs = [d.codes, d.scales, d.g, d.groups._c[5]]
        assert {t.data_ptr() for t in mine}.isdisjoint(t.data_ptr() for t in theirs)
        addresses = {t.data_ptr() for t in mine}
        assert not addresses & {v for v in (*d._c, *d.groups._c) if isinstance(v, int)}
        assert all(any(v is t for v in (*d._c, *d.groups._c)) for t in theirs)
        assert (d.wdtype, d.shape, d.groups.E) == ("nvfp4", (4, 64), 4)


def test_rows_and_groups_do_not_change():
    import torch

    import serving_layer_moe_gb300 as moe
    q = cpu_rows()
    for name in ("codes", "scales", "wdtype", "g", "groups", "K", "shape"):
        with pytest.raises(AttributeError):
            setattr(q, name, None)
    gr = moe.ExpertGroups._of((0, 4, 4, 2, 2, torch.zeros(18, dtype=torch.int32), 0, None, None))
    for name in ("offsets", "tiles", "order", "place", "E", "P", "T", "k"):
        with pytest.raises(AttributeError):
            setattr(gr, name, None)


# Sizes past the library's limits, of tensors that take no memory.  Nothing may be cut to 32 bits on the way.
TOO_LARGE = """
import sys, torch
from torch._subclasses.fake_tensor import FakeTensorMode
import serving_layer_moe_gb300 as moe
moe.operators._host()
with FakeTensorMode(allow_non_fake_inputs=True):
    t = lambda dtype, *s: torch.empty(*s, dtype=dtype, device="cuda")
    i32, u8, bf16 = torch.int32, torch.uint8, torch.bfloat16
    big = 1 << 32
    groups = lambda: moe.ExpertGroups(t(i32, 2), t(i32, 2), t(i32, 4), t(i32, 4, 1))
    calls = {
        "route": lambda: moe.route(t(bf16, 950_000_000, 2), 2),
        "group_pairs": lambda: moe.group_pairs(t(i32, big + 1, 2), 4),
        "groups": lambda: moe.ExpertGroups(t(i32, 5), t(i32, 5), t(i32, 1 << 31), t(i32, 1 << 30, 2)),
        "scale": lambda: moe.fp4_scale(t(bf16, big + 1, 1, 1)),
        "quantize_K": lambda: moe.quantize_fp4(t(bf16, 1, big + 32), "mxfp4"),
        "quantize_N": lambda: moe.quantize_fp4(t(bf16, big + 1, 32), "mxfp4"),
        "quantize_G": lambda: moe.quantize_fp4(t(bf16, 70000, 1, 32), "mxfp4"),
        "rows_K": lambda: moe.FP4Rows(t(u8, 1, big // 2 + 16), t(u8, 1, big // 128 + 1, 512), "mxfp4"),
        "rows_N": lambda: moe.FP4Rows(t(u8, big + 1, 16), t(u8, big // 128 + 1, 1, 512), "mxfp4"),
        "rows_G": lambda: moe.FP4Rows(t(u8, 70000, 1, 16), t(u8, 70000, 1, 512), "mxfp4"),
        "matmul_K": lambda: moe.grouped_matmul(t(bf16, 4, big + 8), t(bf16, 1, 8, big + 8), groups()),
        "matmul_N": lambda: moe.grouped_matmul(t(bf16, 4, 8), t(bf16, 1, big + 8, 8), groups()),
    }
    try:
        calls[sys.argv[1]]()
    except ValueError as e:
        print("refused", e)
"""


@pytest.mark.parametrize("call", ["route", "group_pairs", "groups", "scale", "quantize_K", "quantize_N", "quantize_G", "rows_K", "rows_N", "rows_G",
                                  "matmul_K", "matmul_N"])
def test_sizes_past_the_limits_are_refused_as_values(call):
    line = run(TOO_LARGE, call)
    assert line.startswith("refused") and "most" in line or "more than" in line, line


# An argument whose truth value raises: that error, not the interpreter's own about a result with an error set.
NO_TRUTH = """
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
import serving_layer_moe_gb300 as moe
class No:
    def __bool__(self):
        raise KeyError("no truth")
with FakeTensorMode(allow_non_fake_inputs=True):
    t = lambda dtype, *s: torch.empty(*s, dtype=dtype, device="cuda")
    i32, bf16 = torch.int32, torch.bfloat16
    gr = moe.ExpertGroups(t(i32, 2), t(i32, 2), t(i32, 4), t(i32, 4, 1))
    try:
        moe.grouped_matmul(t(bf16, 3, 8), t(bf16, 1, 8, 8), gr, gather=No())
    except KeyError as e:
        print("raised", e)
"""


def test_an_argument_without_a_truth_value_raises_its_own_error():
    assert run(NO_TRUTH).startswith("raised")


WITHOUT_TORCH = """
import sys
sys.modules["torch"] = None                      # importing it raises, as where it is not installed
import serving_layer_moe_gb300 as moe
from serving_layer_moe_gb300 import *
assert MoECache is moe.MoECache and "moe_layer_decode" in moe.SYMBOLS
moe.load_library()
try:
    moe.route
except ImportError:
    print("needs torch")
"""

LATER = """
import sys
import serving_layer_moe_gb300 as moe
assert "torch" not in sys.modules and "route" in dir(moe) and not hasattr(moe, "nothing")
from serving_layer_moe_gb300 import *
assert route is moe.route is moe.operators.route and combine is moe.combine and "moe_route" in OPERATOR_SYMBOLS
print("later")
"""


@pytest.mark.parametrize("script,last", [(WITHOUT_TORCH, "needs torch"), (LATER, "later")])
def test_the_package_needs_torch_for_the_operators_only(script, last):
    assert run(script) == last


# The build with stand-ins for the compilers, in a folder of its own: what is asked of them, not what they make.
BUILD = """
import os, sys
here, torch = sys.argv[1:]
if torch == "no":
    sys.modules["torch"] = None
sys.path.insert(0, here)
import build as b
open(b.HOST, "w").close()                        # left from another build
try:
    print("built", b.build() == b.LIB, os.path.exists(b.LIB), os.path.exists(b.HOST))
except RuntimeError as e:
    print("raised", os.path.exists(b.LIB), str(e).split()[0])
"""


@pytest.mark.parametrize("torch,last", [("no", "built True True False"), ("yes", "raised True g++")])
def test_the_library_builds_without_the_operators_binding(tmp_path, monkeypatch, torch, last):
    """Without torch _operators.so is left out; where its compiler fails, libmoecache.so is there all the same."""
    import shutil
    shutil.copy(os.path.join(ROOT, "serving_layer_moe_gb300", "build.py"), tmp_path)
    (tmp_path / "csrc").mkdir()
    (tmp_path / "csrc" / "one.cu").touch()
    nvcc = tmp_path / "nvcc"
    nvcc.write_text('#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\ntouch "$2"\n')
    nvcc.chmod(0o755)
    monkeypatch.setenv("NVCC", str(nvcc))
    monkeypatch.setenv("CXX", "false")
    assert run(BUILD, str(tmp_path), torch) == last
