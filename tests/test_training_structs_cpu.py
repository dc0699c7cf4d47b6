"""The structures of the norms, the cross entropy and the AdamW step are laid
out in the binding as a C compiler lays them out."""
import ctypes
import os
import shutil
import subprocess

import pytest

import gated_deltanet_linear_03_amd as gdn


def test_struct_layouts(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    checks = {"gdn_norm_io": gdn.CNormIO, "gdn_norm_grad": gdn.CNormGrad, "gdn_loss_io": gdn.CLossIO, "gdn_loss_grad": gdn.CLossGrad,
              "gdn_adamw_tensor": gdn.CAdamWTensor, "gdn_adamw": gdn.CAdamW}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "gdn.h"', "int main(void) {"]
    for name, cls in checks.items():
        lines.append(f'  printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'  printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    for name in ("GDN_NORM_LAYER", "GDN_NORM_RMS", "GDN_ADAMW_BLOCK", "GDN_STATUS_BAD_INDEX"):
        lines.append(f'  printf("{name} %d\\n", {name});')
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["  return 0;\n}"]))
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run([cc, "-std=c11", "-I", inc, str(src), "-o", str(tmp_path / "layout")], check=True)
    got = dict(line.split() for line in subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True,
                                                       check=True).stdout.splitlines())
    for name, cls in checks.items():
        assert int(got[name]) == ctypes.sizeof(cls), name
        for f, _ in cls._fields_:
            assert int(got[f"{name}.{f}"]) == getattr(cls, f).offset, (name, f)
    for name in ("GDN_NORM_LAYER", "GDN_NORM_RMS", "GDN_ADAMW_BLOCK", "GDN_STATUS_BAD_INDEX"):
        assert int(got[name]) == getattr(gdn, name)
