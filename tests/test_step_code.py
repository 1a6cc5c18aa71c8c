"""The optimiser step's kernels as the compiler makes them (no GPU needed): what
a matrix product's test cannot see, an access past the end of a caller's buffer
or a stated alignment that its address need not have."""

import importlib.util
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def muon_ir(tmp_path_factory):
    """LLVM IR of every kernel of muon.hip, by its (mangled) name."""
    spec = importlib.util.spec_from_file_location(
        "_qlora_build", os.path.join(ROOT, "parameter_efficient_fine_nf4_amd", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    out = str(tmp_path_factory.mktemp("ir") / "muon.ll")
    subprocess.run([b.HIPCC, *b.FLAGS, "--offload-device-only", "-S", "-emit-llvm",
                    os.path.join(b.CSRC, "muon.hip"), "-o", out], check=True, capture_output=True)
    with open(out) as f:
        parts = re.split(r"\ndefine ", f.read())[1:]
    return {re.search(r"@(\w+)\(", p).group(1): p.split("\n}")[0] for p in parts}


def _accesses(body):
    """(load or store, number of elements, element type, alignment) of the accesses to global memory."""
    for op, kind, rest in re.findall(r"\b(load|store) (<[^>]+>|\w+) ?([^\n]*)", body):
        at = re.search(r"addrspace\((\d)\)[^\n]*align (\d+)", rest)
        if at and at.group(1) in "01":
            n, elem = re.match(r"<(\d+) x (\w+)>", kind).groups() if kind[0] == "<" else (1, kind)
            yield op, int(n), elem, int(at.group(2))


def test_three_values_are_read_as_three(muon_ir):
    # tall factors of 33 to 48 columns: a lane's three bf16 are 6 bytes, of which the last lane's end with the matrix;
    # and they stay in registers
    name = next(n for n in muon_ir if "k_muon_gramILi3ELb1E" in n)
    seen = list(_accesses(muon_ir[name]))
    for op in ("load", "store"):
        assert max(n for o, n, e, _ in seen if o == op and e == "float") == 3
    bits = {n * int(e[1:]) for o, n, e, _ in seen if o == "load" and e[0] == "i"}
    assert bits == {16, 32}, bits
    assert "alloca" not in muon_ir[name]


def test_no_access_claims_more_than_an_elements_alignment(muon_ir):
    # rows of an odd length start at any multiple of their element's size: 4 bytes for fp32, 2 for bf16 (which the IR
    # has as integers); the partial sums are fp64
    most = {"float": 4, "double": 8}
    wrong = {(name, *a) for name, body in muon_ir.items() for a in _accesses(body) if a[3] > most.get(a[2], 2)}
    assert not wrong, sorted(wrong)[:5]
