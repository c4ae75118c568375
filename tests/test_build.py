"""The build's parts fail apart: the library needs nvcc alone.  No GPU needed."""

import os

from ring_allreduce_gb300 import build


def _without_torch():
    raise RuntimeError("torch is not installed")


def test_library_is_linked_without_the_extension(monkeypatch, capsys, tmp_path):
    """Without torch the library is built all the same, the reason is reported, and no older extension is left."""
    ext = tmp_path / "_ra_torch.so"
    ext.write_bytes(b"of another header")
    lib = tmp_path / "libra_gb300.so"
    monkeypatch.setattr(build, "TORCH_EXT_PATH", str(ext))
    monkeypatch.setattr(build, "LIB_PATH", str(lib))
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "UNITS", [("ra_ops_host.cpp", "ra_ops_host", {})])   # one unit: seconds, not a minute
    monkeypatch.setattr(build, "_torch_dir", _without_torch)
    for _ in range(2):   # built, and found up to date
        assert build.build() == str(lib)
        assert lib.exists() and not ext.exists()
        assert "_ra_torch.so" in (err := capsys.readouterr().err) and "torch is not installed" in err


def test_extension_that_does_not_compile_is_reported(monkeypatch, capsys, tmp_path):
    build.build()
    capsys.readouterr()
    monkeypatch.setattr(build, "TORCH_EXT_PATH", str(tmp_path / "_ra_torch.so"))
    monkeypatch.setattr(build, "_torch_dir", lambda: str(tmp_path))   # no headers there
    assert build.build() == build.LIB_PATH and os.path.exists(build.LIB_PATH)
    assert "the compiler failed" in capsys.readouterr().err
