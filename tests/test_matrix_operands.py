"""The gated block's matrix instructions are inline assembly, for which the compiler inserts no wait
states.  The assembly it makes of their kernels is held here to the distances that it keeps for
its own matrix instructions of this shape (v_mfma_f32_16x16x32_bf16, eight passes):

 - two wait states between a vector instruction and a matrix instruction that reads its result;
 - eight between a matrix instruction and anything else that touches its result;
 - none between matrix instructions that add to exactly the same registers (the hardware holds the
   second back); never to some of them.

CPU only: compiles for gfx950, runs nothing."""
import os
import re
import subprocess

import pytest

from activation_sparse_gemm_amd import build

pytestmark = pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="needs hipcc")

VALU_TO_MATRIX, MATRIX_TO_OTHER = 2, 8


def registers(text):
    """The vector ('v') and accumulation ('a') registers that operands name."""
    out = set()
    for kind, lo, hi, one in re.findall(r"\b([va])(?:\[(\d+):(\d+)\]|(\d+)\b)", text):
        out |= {(kind, i) for i in range(int(lo or one), int(hi or one) + 1)}
    return out


class Code:
    """One function: instructions (opcode, operands), and where each may go next."""

    def __init__(self, lines):
        self.ops, labels = [], {}
        for line in lines:
            line = line.split(";")[0].strip()
            label = re.match(r"^([.\w$]+):$", line)
            if label:
                labels[label[1]] = len(self.ops)
            elif line and not line.startswith("."):
                op, _, rest = line.replace("\t", " ").partition(" ")
                self.ops.append((op, [r.strip() for r in rest.split(",")]))
        self.next = []
        for i, (op, args) in enumerate(self.ops):
            on = [] if op in ("s_branch", "s_endpgm", "s_setpc_b64") else [i + 1]
            if op == "s_branch" or op.startswith("s_cbranch"):
                on.append(labels[args[0]])
            self.next.append(on)

    def after(self, i, states):
        """Instructions that can run fewer than `states` wait states after instruction i."""
        found, todo = set(), [(n, states) for n in self.next[i]]
        while todo:
            n, left = todo.pop()
            if n >= len(self.ops) or left <= 0 or (n, left) in found:
                continue
            found.add((n, left))
            op, args = self.ops[n]
            todo += [(k, left - (int(args[0], 0) + 1 if op == "s_nop" else 1)) for k in self.next[n]]
        return sorted({n for n, _ in found})


def faults(code):
    bad = []
    for i, (op, args) in enumerate(code.ops):
        if op.startswith("v_mfma"):
            dst = registers(args[0])
            for n in code.after(i, MATRIX_TO_OTHER):
                other, a = code.ops[n]
                if other.startswith("v_mfma"):
                    out, add = registers(a[0]), registers(a[3])
                    fine = not dst & registers(",".join(a[1:3])) and (add == dst or not dst & add) and \
                        (out == dst or not dst & out)
                else:
                    fine = not dst & registers(",".join(a))
                if not fine:
                    bad.append((op, args, other, a))
        elif op.startswith("v_"):
            wrote = registers(",".join(args[:2]) if "swap" in op else args[0])
            for n in code.after(i, VALU_TO_MATRIX):
                other, a = code.ops[n]
                if other.startswith("v_mfma") and wrote & registers(",".join(a[1:])):
                    bad.append((op, args, other, a))
    return bad


def functions(text):
    """name -> lines of every function of an assembly file."""
    out, name = {}, None
    for line in text.splitlines():
        start = re.match(r"^(_Z\w+):", line)
        if start:
            name = start[1]
            out[name] = []
        elif line.startswith("\t.section") or line.startswith(".Lfunc_end"):
            name = None
        elif name is not None:
            out[name].append(line)
    return out


def test_distances():
    """The distances, on code that keeps them and on code that does not."""
    def bad(*lines):
        return len(faults(Code(lines)))

    m = "v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]"
    assert bad("v_mov_b32 v0, v9", "s_nop 1", m, m) == 0
    assert bad("v_mov_b32 v0, v9", "s_nop 0", m) == 1
    assert bad("v_mov_b32 v0, v9", m, m) == 2
    assert bad("v_accvgpr_write_b32 a2, v9", "s_nop 0", m) == 1
    assert bad(m, "s_nop 6", "v_accvgpr_read_b32 v9, a3") == 1
    assert bad(m, "s_nop 7", "v_accvgpr_read_b32 v9, a3") == 0
    assert bad(m, "v_mfma_f32_16x16x32_bf16 a[2:5], v[0:3], v[4:7], a[2:5]") == 1
    assert bad(m, "v_mfma_f32_16x16x32_bf16 a[4:7], v[0:3], v[4:7], a[4:7]") == 0
    assert bad(".L1:", m, "s_nop 7", "v_mov_b32 v5, v9", "s_cbranch_scc1 .L1", "s_endpgm") == 1  # round the loop


def test_gated_block_kernels(tmp_path):
    out = tmp_path / "mlp_bf16.s"
    flags = [f for f in build.FLAGS if f != "-fPIC"]
    subprocess.run([build.HIPCC, *flags, "--cuda-device-only", "-S", os.path.join(build.CSRC, "mlp_bf16.hip"), "-o", str(out)],
                   check=True, capture_output=True)
    kernels = {n: lines for n, lines in functions(out.read_text()).items() if "glu_kernel" in n or "glu_grad_kernel" in n}
    assert len(kernels) >= 4
    for name, lines in kernels.items():
        code = Code(lines)
        assert any(op == "v_mfma_f32_16x16x32_bf16" for op, _ in code.ops), name
        assert faults(code) == [], name
