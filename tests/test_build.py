"""What build() makes, from what, and when again (the compilers are stand-ins
that write a file)."""
import os
import stat

import pytest


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """_build with its outputs in tmp_path, nvcc and the host compiler replaced; returns (module, calls)."""
    from block_scaled_precision_03_gb300 import _build as b
    calls = tmp_path / "calls"
    fake = tmp_path / "compiler"
    fake.write_text(f"""#!/bin/sh
[ -e {tmp_path}/broken ] && [ "$(basename "$0")" = g++ ] && exit 1
echo "$(basename "$0") $*" >> {calls}
while [ $# -gt 1 ]; do [ "$1" = -o ] && : > "$2"; shift; done
exit 0
""")
    fake.chmod(fake.stat().st_mode | stat.S_IXUSR)
    for name in ("nvcc", "g++"):
        os.symlink(fake, tmp_path / name)
    monkeypatch.setenv("PATH", f"{tmp_path}{os.pathsep}{os.environ['PATH']}")
    monkeypatch.setattr(b, "nvcc", lambda: str(tmp_path / "nvcc"))
    for name, file in (("BUILD", "_build"), ("LIB", "libbsq.so"), ("BINDING", "_binding.so")):
        monkeypatch.setattr(b, name, str(tmp_path / file))

    def made():
        lines = calls.read_text().splitlines() if calls.exists() else []
        calls.write_text("")
        return sum(" -shared" in x and x.startswith("nvcc") for x in lines), sum(x.startswith("g++") for x in lines)
    return b, made, tmp_path


def test_each_is_built_when_it_is_out_of_date(tree):
    b, made, tmp = tree
    assert b.build() == b.LIB and made() == (1, 1)
    b.build()
    assert made() == (0, 0)
    os.remove(b.BINDING)
    b.build()
    assert made() == (0, 1)
    os.remove(b.LIB)
    b.build()
    assert made()[0] == 1 and os.path.exists(b.LIB)
    b.build(force=True)
    assert made() == (1, 1)


def test_the_library_does_not_need_the_binding(tree):
    # without a host compiler, Python's or PyTorch's headers: a user of the C ABI still gets libbsq.so
    b, made, tmp = tree
    (tmp / "broken").touch()
    with pytest.raises(RuntimeError, match="binding"):
        b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.BINDING)
    made()
    with pytest.raises(RuntimeError, match="binding"):
        b.build()
    assert made()[0] == 0                       # the library is up to date
    os.remove(tmp / "broken")
    b.build()
    assert made() == (0, 1) and os.path.exists(b.BINDING)


def test_the_binding_is_built_again_for_another_pytorch(tree, monkeypatch):
    # it is compiled against the installed one's headers
    b, made, tmp = tree
    b.build()
    made()
    import importlib.util
    other, find = tmp / "torch", importlib.util.find_spec
    other.mkdir()
    (other / "__init__.py").touch()
    (other / "version.py").write_text("__version__ = '1.0.0'")
    spec = importlib.util.spec_from_file_location("torch", other / "__init__.py")
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: spec if name == "torch" else find(name, *a))
    b.build()
    assert made() == (0, 1)
    b.build()
    assert made() == (0, 0)
