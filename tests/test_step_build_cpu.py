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
