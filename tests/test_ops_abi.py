"""include/gemm_rs_ops.h and its binding agree (no GPU needed)."""
import os
import subprocess

from tensor_gemm_reduce_gb300 import build, ops_abi


def test_every_declared_function_is_exported_and_bound():
    names = ops_abi.header_symbols()
    assert set(names) == set(ops_abi.SIGS)
    for n in names:
        assert hasattr(ops_abi.lib(), n), n


def test_header_is_c(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "gemm_rs_ops.h"\nint main(void) { return sizeof(gemm_rs_norm_desc) != %d; }\n'
                   % ops_abi.ctypes.sizeof(ops_abi.gemm_rs_norm_desc))
    exe = str(tmp_path / "h")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-I", os.path.join(build.ROOT, "include"),
                    "-o", exe, str(src)], check=True)
    assert subprocess.run([exe]).returncode == 0
