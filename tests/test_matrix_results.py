"""CPU: the attention kernels' assembly, as built here, reads no matrix result early.

The hardware holds a product back that goes on with the same sum; any other instruction that reads (or overwrites) a
result has to come WAIT wait states after it: 12 for the eight passes of a 32x32x16 product.  The compiler counts them,
but was seen to miss a read beyond a branch; the kernels end such chains with waits of their own.  This follows every
path from every product until the wait is over, so that a chain without them is found."""
import concurrent.futures
import os
import re
import subprocess

import pytest

from schnet_cfconv_force_amd import build

WAIT = 12
REGISTERS = re.compile(r"\b([av])(?:(\d+)\b|\[(\d+):(\d+)\])")


def registers(text):
    out = set()
    for m in REGISTERS.finditer(text):
        first, last = (m.group(2), m.group(2)) if m.group(2) else (m.group(3), m.group(4))
        out.update((m.group(1), i) for i in range(int(first), int(last) + 1))
    return out


def kernels(assembly):
    """Name -> list of (operation, operands); a label is (None, label)."""
    found, body = {}, None
    for line in assembly.splitlines():
        line = line.split(";")[0].rstrip()
        start = re.match(r"^(_Z\w+):", line)
        if start:
            body = found.setdefault(start.group(1), [])
        elif line.startswith(".Lfunc_end"):
            body = None
        elif body is not None:
            label = re.match(r"^(\.LBB\w+):", line)
            words = line.split(None, 1)
            if label:
                body.append((None, label.group(1)))
            elif words and words[0][0] not in ".#":
                body.append((words[0], words[1] if len(words) > 1 else ""))
    return found


def operands(rest):
    """The two factors of a product."""
    parts = re.findall(r"[av]\[\d+:\d+\]|[^,\s]+", rest)
    return parts[1], parts[2]


def early_reads(body):
    """(product, reader, wait states between) for every read that comes too early on some path."""
    labels = {rest: i for i, (op, rest) in enumerate(body) if op is None}
    found = []
    for i, (op, rest) in enumerate(body):
        if op is None or not op.startswith("v_mfma"):
            continue
        result = registers(rest.split(",")[0])
        paths, seen = [(i + 1, 0, 0)], set()     # next instruction, wait states so far and when the last product went
        while paths:
            j, waited, last = paths.pop()
            while j < len(body) and waited < WAIT and (j, waited, last) not in seen:
                seen.add((j, waited, last))
                op, rest = body[j]
                if op is None:
                    j += 1
                    continue
                if op == "s_nop":
                    waited += int(rest, 0) + 1
                    j += 1
                    continue
                if op.startswith("v_mfma"):
                    target, left, right = rest.split(",")[0], *operands(rest)
                    if (registers(left) | registers(right)) & result:
                        found.append((i, j, waited))
                        break
                    if registers(target) & result:      # the same sum goes on: held back, and followed from there
                        break
                    waited = last = max(waited, last + 8)   # one goes when the eight passes of the one before are through
                    j += 1
                    continue
                if registers(rest) & result:
                    found.append((i, j, waited))
                    break
                if op.startswith("s_cbranch") and rest in labels:
                    paths.append((labels[rest], waited + 1, last))
                elif op == "s_branch":
                    if rest not in labels:
                        break
                    j, waited = labels[rest], waited + 1
                    continue
                elif op in ("s_endpgm", "s_setpc_b64"):
                    break
                waited += 1
                j += 1
    return found


def assembly_of(source, folder):
    out = os.path.join(folder, source.replace(".hip", ".s"))
    cmd = [build.HIPCC, *build.FLAGS, *build.PER_FILE.get(source, []), "--cuda-device-only", "-S", os.path.join(build.CSRC, source),
           "-o", out]
    subprocess.run(cmd, check=True, capture_output=True)
    with open(out) as f:
        return f.read()


def test_no_matrix_result_is_read_early(tmp_path):
    sources = ["attention_fwd.hip", "attention_bwd.hip"]
    with concurrent.futures.ThreadPoolExecutor() as pool:
        for source, text in zip(sources, pool.map(lambda s: assembly_of(s, str(tmp_path)), sources)):
            found = kernels(text)
            products = sum(op is not None and op.startswith("v_mfma") for body in found.values() for op, _ in body)
            assert products > 100, source
            for name, body in found.items():
                assert not early_reads(body), (source, name)


PRODUCT = "\tv_mfma_f32_32x32x16_bf16 v[0:15], v[16:19], v[20:23], v[0:15]\n"


@pytest.mark.parametrize("between,early", [
    ("", True), ("\ts_nop 7\n", True), ("\ts_nop 7\n\ts_nop 3\n", False), ("\tv_mov_b32_e32 v40, v41\n" * 11, True),
    ("\tv_mov_b32_e32 v40, v41\n" * 12, False), ("\ts_cbranch_vccz .LBB0_1\n" + "\ts_nop 7\n" * 2 + ".LBB0_1:\n", True),
    (PRODUCT.replace("v[0:15]", "v[60:75]") * 2, False), (PRODUCT.replace("v[0:15]", "v[60:75]"), True),
    (PRODUCT.replace("v[0:15]", "v[60:75]").replace("v[16:19]", "v[0:3]") + "\ts_nop 15\n", True),
    ("\ts_nop 7\n\ts_nop 3\n\ts_cbranch_vccz .LBB0_1\n\ts_nop 1\n.LBB0_1:\n", False)])
def test_early_reads_are_found(between, early):
    text = "_Zkernel:\n" + PRODUCT + between + "\tv_add_f32_e32 v50, v3, v50\n\ts_endpgm\n.Lfunc_end0:\n"
    assert bool(early_reads(kernels(text)["_Zkernel"])) == early
