"""What the serving calls refuse on the host, beyond shapes and types, and how
their native module is built.  No kernel runs here."""
import os
import shutil
import stat
import subprocess
import sys

import pytest
import torch

from exact_attention_93_gb300 import attention, build, kvcache, rotary


def small():
    """A cache of one sequence of three keys, on the CPU: every call on it is refused."""
    kp, vp, _, _ = kvcache.alloc_kv_cache(2, 16, 2, 64, device="cpu")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    x, q = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    return x, q, kp, vp, (torch.zeros(1, 2, dtype=torch.int32), i32(0, 3), i32(3))


def test_tangents_are_refused():
    x, q, kp, vp, (table, cu, lens) = small()
    freq, _ = rotary.rotary_frequencies(64, device="cpu")
    with torch.autograd.forward_ad.dual_level():
        d = lambda t: torch.autograd.forward_ad.make_dual(t, torch.ones_like(t))  # noqa: E731
        for grad in (torch.enable_grad(), torch.no_grad()):
            with grad:
                for call in (lambda: rotary.rotary_func(d(x), None, freq),
                             lambda: rotary.rotary_func(x, d(x), freq, inplace=True),
                             lambda: rotary.rotary_func(x, None, d(freq)),
                             lambda: kvcache.kv_cache_append(x, d(x), kp, vp, table, cu, lens),
                             lambda: kvcache.kv_cache_read(kp, d(vp), table, cu, 3),
                             lambda: attention.flash_attn_paged_func(d(q), kp, vp, table, cu, lens)):
                    with pytest.raises(NotImplementedError):
                        call()


def test_reading_a_cache_that_needs_gradients_is_refused():
    _, _, kp, vp, (table, cu, _) = small()
    for pages in ((kp.clone().requires_grad_(), vp), (kp, vp.clone().requires_grad_())):
        with pytest.raises(ValueError, match="no gradients"):  # they would be lost
            kvcache.kv_cache_read(*pages, table, cu, 3)
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):  # allowed, but for the device
            kvcache.kv_cache_read(*pages, table, cu, 3)


# ---- building, with compilers that only write down what they are asked for

@pytest.fixture
def tree(tmp_path):
    """A copy of the sources beside an nvcc and a g++ that make empty files."""
    package = tmp_path / "exact_attention_93_gb300"
    package.mkdir()
    for f in ("__init__.py", "build.py"):
        shutil.copy(os.path.join(build.HERE, f), package)
    shutil.copytree(build.CSRC, package / "csrc")
    shutil.copytree(build.INCLUDE, tmp_path / "include")
    (tmp_path / "bin").mkdir()
    for name in ("nvcc", "g++"):
        tool = tmp_path / "bin" / name
        tool.write_text(f"""#!/bin/sh
echo {name} "$@" >> {tmp_path}/calls
[ -e {tmp_path}/no-{name} ] && exit 1
while [ $# -gt 0 ]; do [ "$1" = -o ] && : > "$2"; shift; done
exit 0
""")
        tool.chmod(tool.stat().st_mode | stat.S_IEXEC)
    return tmp_path


def run_in(tree, code):
    env = {**os.environ, "PATH": f"{tree}/bin:{os.environ['PATH']}", "PYTHONPATH": str(tree)}
    r = subprocess.run([sys.executable, "-c", code], cwd=tree, env=env, capture_output=True, text=True)
    calls = tree / "calls"
    lines = calls.read_text().splitlines() if calls.exists() else []
    calls.unlink(missing_ok=True)
    return r, [x.split()[0] for x in lines]


def test_the_library_is_built_without_torch(tree):
    code = "import sys; sys.modules['torch'] = None; from exact_attention_93_gb300 import build as b; b.build()"
    r, calls = run_in(tree, code)
    assert r.returncode == 0, r.stderr
    assert (tree / "exact_attention_93_gb300/libfattn.so").exists() and set(calls) == {"nvcc"}
    assert run_in(tree, code)[1] == []  # and is then up to date
    r, calls = run_in(tree, "from exact_attention_93_gb300 import build as b; b.build()")
    assert r.returncode == 0, r.stderr  # with torch the native module follows alone
    assert (tree / "exact_attention_93_gb300/_bind_torch.so").exists() and set(calls) == {"g++"}


def test_the_library_is_built_where_the_native_module_is_not(tree):
    (tree / "no-g++").touch()
    r, _ = run_in(tree, "from exact_attention_93_gb300 import build as b; b.build()")
    assert r.returncode != 0 and "g++ failed" in r.stderr
    assert (tree / "exact_attention_93_gb300/libfattn.so").exists()
    assert not (tree / "exact_attention_93_gb300/_bind_torch.so").exists()


def test_the_native_module_follows_torch_and_python(tree):
    get, code = "from exact_attention_93_gb300 import build as b; ", "b.build()"
    assert set(run_in(tree, get + code)[1]) == {"nvcc", "g++"}
    assert run_in(tree, get + code)[1] == []
    other = get + "b.torch_version = lambda: '0.0'; "
    assert set(run_in(tree, other + code)[1]) == {"g++"}
    assert run_in(tree, other + code)[1] == []
    assert set(run_in(tree, get + code)[1]) == {"g++"}  # and back
    shutil.rmtree(tree / "exact_attention_93_gb300/_build")  # the built files alone, as copied
    assert run_in(tree, get + code)[1] == []
    other = get + "import sysconfig as s; s.get_config_var = lambda n: 'cpython-399'; "
    assert set(run_in(tree, other + code)[1]) == {"g++"}
