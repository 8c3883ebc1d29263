"""include/gemm_rs_ops.h and its binding agree (no GPU needed)."""
import os
import subprocess

from tensor_gemm_reduce_gb300 import build, ops_abi


def test_every_declared_function_is_exported_and_bound():
    names = ops_abi.header_symbols()
    assert set(names) == set(ops_abi.SIGS)
    for n in names:
        assert hasattr(ops_abi.lib(), n), n


def test_the_binding_is_of_these_sources_and_this_torch(tmp_path, monkeypatch):
    """An entry compiled from other sources or for another torch is not taken for the current one."""
    import torch
    at = ops_abi.ops().__file__
    assert at == build.binding_path() and os.path.exists(at)
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.1")
        assert build.binding_path() != at
    changed = tmp_path / "ops_binding.cpp"
    changed.write_text(open(build.BINDING_SOURCE).read() + "// another line\n")
    monkeypatch.setattr(build, "BINDING_SOURCE", str(changed))
    assert build.binding_path() != at
    wanted = []
    monkeypatch.setattr(ops_abi, "_OPS", None)
    monkeypatch.setattr(build, "build_binding", lambda: wanted.append(build.binding_path()) or at)
    assert ops_abi.ops() is not None and wanted == [build.binding_path()]


def test_header_is_c(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "gemm_rs_ops.h"\nint main(void) { return sizeof(gemm_rs_norm_desc) != %d; }\n'
                   % ops_abi.ctypes.sizeof(ops_abi.gemm_rs_norm_desc))
    exe = str(tmp_path / "h")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-I", os.path.join(build.ROOT, "include"),
                    "-o", exe, str(src)], check=True)
    assert subprocess.run([exe]).returncode == 0
