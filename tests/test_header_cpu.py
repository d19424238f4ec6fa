"""The public header as a reader and a C compiler meet it: every comment line is whole, every workspace function
is named where a buffer asks for its bytes, and the bindings declare what the header does."""
import os
import re
import subprocess

import pytest

from gated_deltanet_hybrid_amd import hla

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "hla.h")


def text():
    with open(HEADER) as f:
        return f.read()


def test_block_comments_are_whole():
    """A line inside a block comment that begins at the margin starts with ' *'."""
    inside = False
    for n, line in enumerate(text().splitlines(), 1):
        if inside:
            assert line.startswith(" *"), f"hla.h:{n}: {line}"
        if line.startswith("/*"):
            inside = "*/" not in line
        elif inside and "*/" in line:
            inside = False
    assert not inside


def test_every_workspace_function_is_named_beside_a_workspace():
    comments = " ".join(re.findall(r"/\*.*?\*/", text(), re.S))
    code = re.sub(r"/\*.*?\*/", "", text(), flags=re.S)
    names = re.findall(r"\b(hla_\w*workspace_bytes)\s*\(", code)
    assert len(names) >= 3
    for name in names:
        assert re.search(rf"\b{name}\(", comments), name


@pytest.mark.parametrize("language,standard", [("c", "c11"), ("c++", "c++17")])
def test_the_header_compiles_alone(language, standard):
    r = subprocess.run(["gcc" if language == "c" else "g++", "-x", language, f"-std={standard}", "-fsyntax-only", "-Wall", "-Werror",
                        "-D__HIP_PLATFORM_AMD__", "-isystem", "/opt/rocm/include", HEADER], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_the_bindings_declare_the_headers_functions():
    code = re.sub(r"/\*.*?\*/", "", text(), flags=re.S)
    declared = {m.group(1): m.group(2) for m in re.finditer(r"\b(hla_\w+)\s*\(([^)]*)\)\s*;", code)}
    assert set(declared) == set(hla._SIGS)
    for name, args in declared.items():
        count = 0 if args.strip() in ("", "void") else args.count(",") + 1
        assert count == len(hla._SIGS[name][1]), name
