"""The direct loads into LDS are inline assembly, which the compiler's own
hazard handling does not look into: a vector memory instruction may read a
scalar register 5 wait states after a vector instruction (v_readlane, where the
compiler spilled scalars into vector lanes) wrote it, at the earliest.  Here the
machine code of the built library is read (CPU only): no load comes sooner,
on any path, and the grouped products' loads bring their own wait, so that no
other place for a spill can change that."""
import os
import re
import shutil
import subprocess

import pytest

import fp8_scaled_quantization_scale_amd as fm

BIN = "/opt/rocm/llvm/bin"
NEED = 5  # wait states

_LINE = re.compile(r"^\t(\S+)(?:\s+(.*?))?\s*// ([0-9A-F]+):.*?(?:<(\S+?)(?:\+0x([0-9a-f]+))?>)?$")
_HEAD = re.compile(r"^([0-9a-f]+) <(\S+)>:$")


def _registers(text):
    """scalar registers that an operand list names"""
    out = {"m0"} if re.search(r"\bm0\b", text) else set()
    if re.search(r"\bvcc\b", text):
        out.add("vcc")
    for a, b in re.findall(r"\bs\[(\d+):(\d+)\]", text):
        out |= set(range(int(a), int(b) + 1))
    return out | {int(n) for n in re.findall(r"\bs(\d+)\b", text)}


class _Function:
    def __init__(self, name, start):
        self.name, self.start = name, start
        self.ops, self.args, self.at, self.jumps = [], [], [], {}

    def add(self, op, args, at, symbol, offset):
        if op.startswith(("s_cbranch", "s_branch")):
            assert symbol == self.name
            self.jumps.setdefault(self.start + int(offset or "0", 16), []).append(len(self.ops))
        self.ops.append(op)
        self.args.append(args or "")
        self.at.append(at)

    def loads(self):
        return [i for i, (o, a) in enumerate(zip(self.ops, self.args)) if o.startswith("buffer_load") and a.endswith(" lds")]

    def _written_before(self, i, need, waits):
        """whether a vector instruction fewer than NEED wait states before instruction i writes one of `need`"""
        before = list(self.jumps.get(self.at[i], ()))
        if i > 0 and self.ops[i - 1] not in ("s_branch", "s_endpgm", "s_setpc_b64"):
            before.append(i - 1)
        for j in before:
            if self.ops[j].startswith("v_"):
                wrote = _registers(self.args[j].split(",")[0])
                if self.ops[j].startswith(("v_add_co", "v_sub_co", "v_addc_co", "v_subb_co", "v_div_scale", "v_mad_u64", "v_mad_i64")):
                    wrote |= _registers(self.args[j].split(",")[1])
                if wrote & need:
                    return True
            nop = int(self.args[j], 0) + 1 if self.ops[j] == "s_nop" else 1
            if waits + nop < NEED and self._written_before(j, need, waits + nop):
                return True
        return False

    def too_soon(self):
        return [i for i in self.loads() if self._written_before(i, _registers(self.args[i]) | {"m0"}, 0)]


def _functions(text):
    f = None
    for line in text.splitlines():
        head = _HEAD.match(line)
        if head:
            if f:
                yield f
            f = _Function(head.group(2), int(head.group(1), 16))
            continue
        m = _LINE.match(line)
        if m and f:
            f.add(m.group(1), m.group(2), int(m.group(3), 16), m.group(4), m.group(5))
    if f:
        yield f


def _text(lines, name="k"):
    """a function of these instructions, 4 bytes each, as the disassembler prints it"""
    out = ["0000000000001000 <%s>:" % name]
    for i, (line, target) in enumerate(lines):
        out.append("\t%s  // %012X: 00000000%s" % (line, 0x1000 + 4 * i, " <%s+0x%x>" % (name, 4 * target) if target is not None else ""))
    return "\n".join(out)


LOAD = ("buffer_load_dwordx4 v1, s[8:11], s20 offen lds", None)


@pytest.mark.parametrize("lines,soon", [
    ([("v_readlane_b32 s20, v9, 3", None), ("s_nop 0", None), LOAD], True),
    ([("v_readlane_b32 s20, v9, 3", None), ("s_nop 3", None), LOAD], True),
    ([("v_readlane_b32 s20, v9, 3", None), ("s_nop 4", None), LOAD], False),
    ([("v_readlane_b32 s10, v9, 3", None), ("s_mov_b32 m0, s4", None), ("s_nop 0", None), LOAD], True),
    ([("v_readfirstlane_b32 m0, v9", None), ("s_nop 0", None), LOAD], True),
    ([("v_readlane_b32 s21, v9, 3", None), ("s_nop 0", None), LOAD], False),  # not one of the load's
    ([("s_mov_b32 s20, s3", None), ("s_nop 0", None), LOAD], False),  # not a vector instruction
    ([("v_cmp_lt_i32_e64 s[10:11], v1, v2", None), ("s_nop 0", None), LOAD], True),
    # by a jump to the load's wait, past other instructions
    ([("v_readlane_b32 s20, v9, 3", None), ("s_branch 9", 8), *[("v_mov_b32_e32 v0, v1", None)] * 6, ("s_nop 0", None), LOAD], True),
    ([("v_readlane_b32 s20, v9, 3", None), ("s_branch 9", 8), *[("v_mov_b32_e32 v0, v1", None)] * 6, ("s_nop 4", None), LOAD], False),
    # what stands before an unconditional jump does not come before the load
    ([("v_mov_b32_e32 v0, v1", None), ("v_readlane_b32 s20, v9, 3", None), ("s_branch 0", 0), ("s_nop 0", None), LOAD], False),
])
def test_what_is_found(lines, soon):
    (f,) = _functions(_text(lines))
    assert len(f.loads()) == 1 and bool(f.too_soon()) == soon


@pytest.fixture(scope="module")
def functions(tmp_path_factory):
    if not os.path.exists(os.path.join(BIN, "llvm-objdump")):
        pytest.skip("needs llvm-objdump")
    fm.load()
    where = tmp_path_factory.mktemp("code")
    lib = shutil.copy(fm.LIB_PATH, where)
    subprocess.run([BIN + "/llvm-objdump", "--offloading", lib], cwd=where, check=True, capture_output=True)
    out = []
    for name in sorted(os.listdir(where)):
        if "amdgcn" not in name:
            continue
        r = subprocess.run([BIN + "/llvm-objdump", "-d", "--no-show-raw-insn", name], cwd=where, check=True, capture_output=True, text=True)
        if " lds" in r.stdout:
            out += [f for f in _functions(r.stdout) if f.loads()]
    return out


def test_no_load_comes_too_soon(functions):
    assert len(functions) > 50  # the products of every recipe, format and output
    bad = {f.name: len(f.too_soon()) for f in functions}
    assert not any(bad.values()), {k: v for k, v in bad.items() if v}


def test_grouped_loads_bring_their_wait(functions):
    """gemm_kernel<.., form> with form 1 (rows) and 2 (contraction), and the small tiles."""
    grouped = [f for f in functions if re.search(r"gemm_kernelILi\d+ELi\d+ELi\d+ELi\d+ELi[12]E|gemm_few_kernel", f.name)]
    assert len(grouped) >= 40
    for f in grouped:
        short = [i for i in f.loads() if f.ops[i - 1] != "s_nop" or int(f.args[i - 1], 0) < NEED - 1]
        assert not short, f"{f.name}: {len(short)} of {len(f.loads())} loads without their own wait"
