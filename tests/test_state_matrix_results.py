"""CPU: the cache attention's assembly, as built here, reads no matrix result early.

As test_matrix_results.py follows the attention kernels, with this kernel's products: a 16x16x32 bf16 product runs four
passes and its result may be read 8 wait states after it, a 16x16x4 fp32 product eight passes and 12."""
import pytest

from test_matrix_results import assembly_of, kernels, operands, registers

PASSES = {"v_mfma_f32_16x16x32_bf16": 4, "v_mfma_f32_16x16x4_f32": 8}
WAIT = {4: 8, 8: 12}


def early_reads(body):
    """(product, reader, wait states between) for every read that comes too early on some path."""
    labels = {rest: i for i, (op, rest) in enumerate(body) if op is None}
    found = []
    for i, (op, rest) in enumerate(body):
        if op is None or not op.startswith("v_mfma"):
            continue
        need, own = WAIT[PASSES[op]], PASSES[op]
        result = registers(rest.split(",")[0])
        # next instruction, wait states so far, when the matrix unit is free
        paths, seen = [(i + 1, 0, own)], set()
        while paths:
            j, waited, free = paths.pop()
            while j < len(body) and waited < need and (j, waited, free) not in seen:
                seen.add((j, waited, free))
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
                    waited = max(waited, free)          # one goes when the one before is through
                    free = waited + PASSES[op]
                    waited += 1
                    j += 1
                    continue
                if registers(rest) & result:
                    found.append((i, j, waited))
                    break
                if op.startswith("s_cbranch") and rest in labels:
                    paths.append((labels[rest], waited + 1, free))
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


def test_no_matrix_result_is_read_early(tmp_path):
    found = kernels(assembly_of("cache_attend.hip", str(tmp_path)))
    products = sum(op is not None and op.startswith("v_mfma") for body in found.values() for op, _ in body)
    assert products > 500
    for name, body in found.items():
        assert not early_reads(body), name


BF16 = "\tv_mfma_f32_16x16x32_bf16 v[0:3], v[16:19], v[20:23], v[0:3]\n"
FP32 = "\tv_mfma_f32_16x16x4_f32 v[0:3], v16, v20, v[0:3]\n"


@pytest.mark.parametrize("product,between,early", [
    (BF16, "", True), (BF16, "\ts_nop 6\n", True), (BF16, "\ts_nop 7\n", False), (FP32, "\ts_nop 7\n", True),
    (FP32, "\ts_nop 7\n\ts_nop 3\n", False), (BF16, "\tv_mov_b32_e32 v40, v41\n" * 8, False),
    (BF16, "\ts_cbranch_vccz .LBB0_1\n" + "\ts_nop 7\n" + ".LBB0_1:\n", True),
    (BF16, BF16.replace("v[0:3]", "v[60:63]"), True), (BF16, BF16.replace("v[0:3]", "v[60:63]") * 2, False),
    (FP32, FP32.replace("v[0:3]", "v[60:63]"), True)])
def test_early_reads_are_found(product, between, early):
    text = "_Zkernel:\n" + product + between + "\tv_add_f32_e32 v50, v3, v50\n\ts_endpgm\n.Lfunc_end0:\n"
    assert bool(early_reads(kernels(text)["_Zkernel"])) == early
