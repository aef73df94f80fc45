"""The binding's gemm_adapters_t has the header's layout (no GPU needed)."""
import ctypes
import os
import subprocess

from tensor_core_dense_tma_gb300.adapters import Adapters

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_layout(tmp_path):
    names = [n for n, _ in Adapters._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "adapters.h"\nint main(void) {\n'
                   + "".join(f'    printf("{n} %zu\\n", offsetof(gemm_adapters_t, {n}));\n' for n in names)
                   + '    printf("size %zu\\n", sizeof(gemm_adapters_t));\n    return 0;\n}\n')
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    out = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    assert int(out.pop("size")) == ctypes.sizeof(Adapters)
    assert {n: int(v) for n, v in out.items()} == {n: getattr(Adapters, n).offset for n in names}
