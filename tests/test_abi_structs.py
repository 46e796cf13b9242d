"""The header is C, and the binding's structs lie as a C compiler lays out its own."""
import ctypes
import os
import shutil
import subprocess

import pytest

import combine_moe_gate_amd as M

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
STRUCTS = {"moe_layout_t": M.LayoutStruct, "moe_layout_options_t": M.LayoutOptions, "moe_expert_epilogue_t": M.Epilogue}


@pytest.mark.parametrize("language,compiler", [("c", "gcc"), ("c++", "g++")])
def test_fields_lie_where_the_compiler_puts_them(tmp_path, language, compiler):
    if shutil.which(compiler) is None:
        pytest.skip(f"no {compiler}")
    lines = [f'printf("%s {f[0]} %zu %zu\\n", "{s}", offsetof({s}, {f[0]}), sizeof((({s}*)0)->{f[0]}));'
             for s, c in STRUCTS.items() for f in c._fields_]
    lines += [f'printf("%s size %zu 0\\n", "{s}", sizeof({s}));' for s in STRUCTS]
    src = tmp_path / "offsets"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "moe_gate.h"\nint main(void) {\n' + "\n".join(lines)
                   + "\nreturn 0;\n}\n")
    exe = tmp_path / "run"
    subprocess.run([compiler, "-x", language, "-Wall", "-Werror", "-I", INCLUDE, str(src), "-o", str(exe)], check=True,
                   capture_output=True, text=True)
    got = set(subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")) - {""}
    want = {f"{s} {f[0]} {getattr(c, f[0]).offset} {getattr(c, f[0]).size}" for s, c in STRUCTS.items() for f in c._fields_}
    want |= {f"{s} size {ctypes.sizeof(c)} 0" for s, c in STRUCTS.items()}
    assert got == want
