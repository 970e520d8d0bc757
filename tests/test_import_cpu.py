"""What the package needs to be imported: prefill eviction takes libkvp.so alone, of any age; the paged
cache's calls say what they miss when they are called. And when its binding is built again."""
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "token_eviction_b200")

USE = """
import token_eviction_b200 as m
sh = m.make_cache_shape(1, 4, 2, 64, 16, 8, 4)
print("prefill", m.kvp_workspace_bytes((1, 32, 8, 128, 4096, 32, 256)))
for call in (lambda: m.kvp_cache_append(sh, *[None] * 7), lambda: m.kvp_cache_attend(sh, *[None] * 6, workspace=1),
             lambda: m.kvp_cache_evict(sh, m.make_evict(8), *[None] * 7, workspace=1),
             lambda: m.attend_workspace_for(sh), lambda: m.evict_workspace_for(sh, m.make_evict(8)),
             lambda: m.LayerCache(1, 4, 2, 64, 64, device="cpu")):
    try:
        call()
    except ImportError as e:
        print("refused", e)
    except Exception as e:
        print("other", type(e).__name__)
"""


def use(where, **env):
    got = subprocess.run([sys.executable, "-c", USE], cwd=where, env={**os.environ, "PYTHONPATH": str(where), **env},
                         capture_output=True, text=True)
    assert got.returncode == 0, got.stderr
    return got.stdout.splitlines()


def test_prefill_without_the_binding(tmp_path):
    os.mkdir(tmp_path / "token_eviction_b200")
    for name in ("__init__.py", "build.py", "libkvp.so"):
        shutil.copy(os.path.join(PKG, name), tmp_path / "token_eviction_b200" / name)
    lines = use(tmp_path)
    assert lines[0].startswith("prefill ") and int(lines[0].split()[1]) > 0
    refused = [x for x in lines[1:] if x.startswith("refused")]
    assert len(refused) == 3 and all("_kvp_binding.so" in x and "build.py" in x for x in refused)


def test_a_library_from_before_the_paged_cache(tmp_path):
    """KVP_LIBRARY may name another build: one without the paged cache's functions still evicts prefills."""
    import token_eviction_b200 as m
    names = [n for n in m.EXPORTED if "cache" not in n]
    src = "#include <stddef.h>\n" + "".join(f"size_t {n}(void) {{ return 4096; }}\n" for n in names)
    (tmp_path / "old.c").write_text(src)
    old = str(tmp_path / "libold.so")
    subprocess.check_call(["gcc", "-shared", "-fPIC", "-o", old, str(tmp_path / "old.c")])
    lines = use(ROOT, KVP_LIBRARY=old)
    assert lines[0] == "prefill 4096"
    assert len(lines) == 7 and all(x.startswith("refused") and "libold.so" in x for x in lines[1:])


def test_a_missing_library_is_still_refused_at_import(tmp_path):
    got = subprocess.run([sys.executable, "-c", "import token_eviction_b200"], cwd=ROOT, capture_output=True, text=True,
                         env={**os.environ, "KVP_LIBRARY": str(tmp_path / "none.so")})
    assert got.returncode != 0 and "no fallback" in got.stderr


@pytest.fixture
def builder(tmp_path, monkeypatch):
    spec = importlib.util.spec_from_file_location("kvp_build_for_test", os.path.join(PKG, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    monkeypatch.setattr(mod, "BINDING", str(tmp_path / "_kvp_binding.so"))
    monkeypatch.setattr(mod, "ROOT", str(tmp_path))
    made = []

    def compile(cmd):
        made.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(mod.subprocess, "check_call", compile)
    mod.made = made
    return mod


def test_the_binding_is_built_again_for_another_torch(builder, monkeypatch):
    import torch
    builder.build_binding()
    builder.build_binding()
    assert len(builder.made) == 1
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    builder.build_binding()
    builder.build_binding()
    assert len(builder.made) == 2
    builder.build_binding(force=True)
    assert len(builder.made) == 3
