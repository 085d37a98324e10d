"""The ctypes mirrors of the 8-bit layer's and optimizer's structs match the header (gcc's own offsets)."""

import ctypes
import os
import subprocess

from tests.conftest import ROOT


def test_scratch_size_matches_the_header(metis_lib):
    text = open(os.path.join(ROOT, "include", "metis.h")).read()
    copies = int(text.split("#define METIS_INT8_SCRATCH_COPIES ")[1].split()[0])
    assert metis_lib.INT8_SCRATCH == copies + 1


def test_new_struct_layouts(metis_lib, tmp_path):
    mirror = {"metis_int8": metis_lib.Int8Struct, "metis_adamw_tensor": metis_lib.AdamWTensor,
              "metis_adamw_params": metis_lib.AdamWParams, "metis_dense": metis_lib.Dense}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "%s"' % os.path.join(ROOT, "include", "metis.h"),
             "int main(void) {"]
    for name, cls in mirror.items():
        lines.append('printf("%s %%zu\\n", sizeof(%s));' % (name, name))
        for field, _ in cls._fields_:
            lines.append('printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (name, field, name, field))
    lines.append("return 0; }")
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines))
    subprocess.run(["gcc", "-std=c99", str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    got = dict(line.split() for line in out.splitlines())
    for name, cls in mirror.items():
        assert int(got[name]) == ctypes.sizeof(cls)
        for field, _ in cls._fields_:
            assert int(got[f"{name}.{field}"]) == getattr(cls, field).offset, (name, field)
