"""What the library's build watches."""
import os

from sparse_paged_decode_logical_gb300 import build


def test_every_file_that_is_compiled_in_is_watched():
    there = [os.path.join(d, f) for d in (build.CSRC, build.INCLUDE) for f in os.listdir(d)]
    assert any(f.endswith(".cuh") for f in there)
    assert sorted(build._deps()) == sorted(there)


def test_an_edit_of_a_kernel_header_asks_for_a_build(tmp_path, monkeypatch):
    lib = tmp_path / "lib.so"
    lib.write_text("")
    for f in build._deps() + [build.__file__]:
        assert os.path.getmtime(f) <= os.path.getmtime(lib)
    monkeypatch.setattr(build, "LIB", str(lib))
    assert build.up_to_date()
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    (csrc / "kernel.cuh").write_text("")
    later = os.path.getmtime(lib) + 10
    os.utime(csrc / "kernel.cuh", (later, later))
    monkeypatch.setattr(build, "CSRC", str(csrc))
    assert not build.up_to_date()
