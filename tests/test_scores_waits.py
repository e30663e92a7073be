"""The machine code of the tiled 8-bit scores (no GPU): what the inline assembly leaves to the compiler holds."""
import os
import re
import subprocess

import pytest

from differentiable_gaussian_splat_amd import build

SRC = os.path.join(build.CSRC, "scores.hip")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """Each tiled kernel's instructions, in order."""
    try:
        build.hipcc()
    except RuntimeError:
        pytest.skip("no hipcc")
    out = str(tmp_path_factory.mktemp("scores") / "scores.s")
    subprocess.run([build.hipcc(), *build.CFLAGS, "--cuda-device-only", "-S", SRC, "-o", out], check=True,
                   capture_output=True)
    found, name = {}, None
    with open(out) as f:
        for line in f:
            m = re.match(r"(_Z\w*k_scores_tiles\w*):", line)
            if m:
                name = m.group(1)
                found[name] = []
            elif line.startswith(".Lfunc_end"):
                name = None
            elif name and re.match(r"\s+[a-z]+_\w+", line):
                found[name].append(line.split(";")[0].strip())
    return found


def scalars(operand):
    """The scalar registers that s7 or s[4:7] names."""
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m.group(1)), int(m.group(2)) + 1))
    m = re.fullmatch(r"s(\d+)", operand)
    return {int(m.group(1))} if m else set()


def test_descriptors_are_settled(kernels):
    """A vector instruction that writes a scalar register needs five wait states before a memory instruction that reads
    it: the compiler sees to that, but not inside inline assembly."""
    assert kernels
    for name, lines in kernels.items():
        loads = 0
        since = {}  # wait states since a vector instruction wrote the register
        for line in lines:
            op, _, rest = line.partition(" ")
            operands = [o.strip() for o in re.split(r",\s*(?![^\[]*\])", rest)]
            if op.startswith(("buffer_load", "global_load_lds")):
                loads += 1
                read = set().union(*(scalars(o.split()[0]) for o in operands[1:] if o.split()))
                assert all(since.get(r, 99) >= 5 for r in read), (name, line)
            states = int(rest) + 1 if op == "s_nop" else 1
            since = {r: k + states for r, k in since.items() if k < 16}
            if op.startswith(("v_readlane", "v_readfirstlane", "v_cmp")):
                for r in scalars(operands[0]):
                    since[r] = 0
        assert loads >= 8, name


def vectors(operand):
    """The vector registers that v7 or v[4:7] names."""
    m = re.fullmatch(r"v\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m.group(1)), int(m.group(2)) + 1))
    m = re.fullmatch(r"v(\d+)", operand)
    return {int(m.group(1))} if m else set()


def test_products_are_done_before_their_results_are_read(kernels):
    """Nineteen wait states between a product of sixteen passes and what reads its result, other than as the sum that
    another product adds to. Empty assembly stands between them, behind which the compiler need not see it."""
    for name, lines in kernels.items():
        since, products = {}, 0  # wait states since a product wrote the register
        for line in lines:
            op, _, rest = line.partition(" ")
            operands = [o.strip() for o in re.split(r",\s*(?![^\[]*\])", rest)]
            product = op.startswith("v_mfma")
            if op.startswith(("v_", "ds_", "global_", "buffer_")):
                first = 0 if "store" in op or "write" in op else 1
                read = [o for k, o in enumerate(operands) if k >= first and not (product and k == 3)]
                for o in read:
                    for r in vectors(o.split()[0] if o else ""):
                        assert since.get(r, 99) >= 19, (name, line)
            states = int(rest) + 1 if op == "s_nop" else 1
            since = {r: k + states for r, k in since.items() if k < 40}
            if product:
                products += 1
                since.update({r: 0 for r in vectors(operands[0])})
            elif op.startswith("v_"):
                for r in vectors(operands[0]):
                    since.pop(r, None)
        assert products >= 8, name


def test_steps_stay_in_registers(kernels):
    """Spilled operands would be memory accesses that every step waits for."""
    for name, lines in kernels.items():
        assert not [x for x in lines if x.startswith("scratch_")], name


def test_scores_are_stored_to_global_memory(kernels):
    """A step's wait counts the loads behind a tile's stores in order, and its LDS reads apart from them. A flat access
    is in neither's order; and of a tile's stores past the caches there are as many as the wait lets pass, 16 for each
    row of a wave's tiles."""
    for name, lines in kernels.items():
        assert not [x for x in lines if x.startswith("flat_")], name
        rows = int(re.search(r"k_scores_tilesI(?:f|DF16b)Li\d+ELi\d+ELi(\d+)E", name).group(1))
        assert len([x for x in lines if re.match(r"global_store_\w+ .* nt$", x)]) == 16 * rows, name
