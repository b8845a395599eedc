"""The ctypes structures of the gated block, layer norm and Muon have the C ones' sizes and offsets."""
import ctypes
import os
import shutil
import subprocess

import pytest

from tests import helpers as Hp

FIELDS = {"moe_gated_args": ("MoeGatedArgs", "moe_gated.h"), "moe_layernorm_args": ("MoeLayernormArgs", "moe_layernorm.h"),
          "moe_layernorm_grads": ("MoeLayernormGrads", "moe_layernorm.h"), "moe_newton_schulz": ("MoeNewtonSchulz", "moe_muon.h"),
          "moe_muon_args": ("MoeMuonArgs", "moe_muon.h"), "moe_orthogonalize_args": ("MoeOrthogonalizeArgs", "moe_muon.h")}


@pytest.mark.parametrize("name", sorted(FIELDS))
def test_layout(name, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    python, header = FIELDS[name]
    kind = getattr(Hp.lib(), python)
    names = [f for f, _ in kind._fields_]
    source = tmp_path / "layout.c"
    asked = ", ".join([f"sizeof({name})"] + [f"offsetof({name}, {f})" for f in names])
    source.write_text(f'#include <stdio.h>\n#include <stddef.h>\n#include "{header}"\nint main(void){{size_t v[] = {{{asked}}}; '
                      'for (size_t i = 0; i < sizeof v / sizeof *v; ++i) printf("%zu\\n", v[i]); return 0;}\n')
    program = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(Hp.ROOT, "include"), str(source), "-o", str(program)], check=True)
    got = [int(v) for v in subprocess.run([str(program)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(kind)] + [getattr(kind, f).offset for f in names]
