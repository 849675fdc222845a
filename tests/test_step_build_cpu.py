"""What a library or a compiled binding that does not fit is answered with, and what a failed compilation leaves."""
import subprocess

import pytest

from deterministic_split_lora_amd import _binding as B


def test_library_without_the_newer_entry_points_is_refused(tmp_path, monkeypatch):
    """A library of the same ABI version that lacks entry points of the binding: the error says to rebuild it."""
    src, so = tmp_path / "old.c", tmp_path / "old.so"
    src.write_text("int lora_abi_version(void) { return %d; }\n" % B.ABI_VERSION
                   + "".join("int %s(void) { return 0; }\n" % n for n in B.EXPORTED
                             if n != "lora_abi_version" and not n.startswith(("lora_mx4_", "lora_sample"))))
    subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", str(so)], check=True)
    monkeypatch.setattr(B, "_lib", None)
    monkeypatch.setattr(B, "LIBRARY_PATH", str(so))
    with pytest.raises(ImportError, match="lora_mx4_quantize.*lora_sample.*rebuild"):
        B.lib()
    assert B._lib is None


def test_the_library_is_built_where_the_binding_does_not_compile(tmp_path, monkeypatch):
    """The entry points that need no torch headers stay available, and the failure is still reported."""
    from deterministic_split_lora_amd import build as b
    lib, native = tmp_path / "liblora_det.so", tmp_path / "_native.so"
    monkeypatch.setattr(b, "LIB", str(lib))
    monkeypatch.setattr(b, "BINDING", str(native))
    monkeypatch.setattr(b, "SOURCES", ["sgmv_plan.hip"])       # one is enough here, and seconds
    monkeypatch.setattr(b, "_record_revision", lambda: None)
    native.write_text("an earlier build's")
    monkeypatch.setattr(b, "binding_command", lambda out: ["sh", "-c", "echo no such header >&2; exit 1"])
    with pytest.raises(RuntimeError, match="no such header"):
        b.build()
    assert lib.exists() and not native.exists()
    assert [p.name for p in tmp_path.iterdir()] == ["liblora_det.so"], "left temporary files"

    def no_torch(out):
        raise ImportError("no torch headers")
    lib.unlink()
    monkeypatch.setattr(b, "binding_command", no_torch)
    with pytest.raises(RuntimeError, match="no torch headers"):
        b.build()
    assert lib.exists()


def test_binding_of_another_torch_is_refused(monkeypatch):
    """The compiled marshalling reads torch's objects by the layout it was built for."""
    import torch
    B._native()
    monkeypatch.setattr(B, "_native_module", None)
    monkeypatch.setattr(torch, "__version__", "0.1+other")
    with pytest.raises(ImportError, match="0.1.other.*rebuild"):
        B._native()
    assert B._native_module is None


def test_binding_that_does_not_load_is_refused(tmp_path, monkeypatch):
    broken = tmp_path / "_native.so"
    broken.write_bytes(b"not a library")
    monkeypatch.setattr(B, "_native_module", None)
    monkeypatch.setattr(B, "NATIVE_PATH", str(broken))
    with pytest.raises(ImportError, match="rebuild"):
        B._native()
