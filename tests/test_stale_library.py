"""A library built before an entry point joined (CPU only)."""

import subprocess

import pytest


def test_library_that_lacks_an_entry_point(tmp_path, monkeypatch):
    """The version is the same (the calls it has are the same): loading names
    what is missing and how to build it, and takes nothing over."""
    from precision_moe_numerics_nvfp4_amd import binding
    src, so = tmp_path / "old.c", tmp_path / "old.so"
    names = [n for n in binding.SIGNATURES if n != "moe_route_bwd"]
    src.write_text("int nvfp4moe_abi_version(void) { return 3; }\n" +
                   "".join(f"int {n}(void) {{ return 0; }}\n" for n in names if n != "nvfp4moe_abi_version"))
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(so), str(src)], check=True)
    monkeypatch.setattr(binding, "_LIB", None)
    monkeypatch.setattr(binding, "LIB_PATH", str(so))
    with pytest.raises(RuntimeError, match="lacks moe_route_bwd.*build"):
        binding.abi_version()
    assert binding._LIB is None
