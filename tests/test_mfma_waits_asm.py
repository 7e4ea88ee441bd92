"""Static check of the waits between matrix instructions and what reads or
overwrites their results, in the generated gfx950 code (no GPU needed).

A result of a matrix instruction may be read by a vector or memory instruction,
or taken as A or B by another matrix instruction, passes + 4 wait states after
it at the earliest, and the sum that it started from overwritten after passes - 1
(an instruction counts one, s_nop N counts N + 1); nothing in the hardware waits.  The compiler adds the waits, but its search
misses a way: where a branch leads around a side block, it walks back through
the side block and does not pass the block before the branch again.  This test
compiles the library's device code and walks every way forward from every matrix
instruction, over branches and around loops.

Also: a transcendental's result is used one wait state later at the earliest, a
vector instruction's result two states later by a matrix instruction or an exchange
between lanes, and a buffer or global access uses scalar registers five states after a vector
instruction wrote them (the lane-less guard loads of the LDS DMA, which touch no
memory, aside)."""

import re

import pytest

from tests.test_dma_guard_asm import _device_asm

REGISTERS = re.compile(r"(?<![\w.])([vas])(?:(\d+)|\[(\d+):(\d+)\])(?!\w)|(?<![\w.])(vcc)(?!\w)")
TRANSCENDENTAL = ("v_exp_", "v_log_", "v_rcp_", "v_rsq_", "v_sqrt_", "v_sin_", "v_cos_")
GUARD = re.compile(r"buffer_load_dword (v\d+), \1, s\[\d+:\d+\], 0 offen$")


def registers(text):
    out = set()
    for kind, one, lo, hi, vcc in REGISTERS.findall(text):
        if vcc:
            out.add("vcc")
        elif one:
            out.add((kind, int(one)))
        else:
            out |= {(kind, i) for i in range(int(lo), int(hi) + 1)}
    return out


class Instruction:
    def __init__(self, text):
        self.text = text
        self.op, _, rest = text.partition(" ")
        ops = [x.strip() for x in re.split(r",(?![^\[]*\])", rest)] if rest else []
        self.mfma = self.op.startswith("v_mfma")
        self.valu = self.op.startswith("v_") and not self.mfma
        self.memory = self.op.startswith(("ds_", "global_", "buffer_", "flat_", "scratch_"))
        self.states = int(ops[0], 0) + 1 if self.op == "s_nop" else 1
        self.target = ops[-1] if self.op.startswith(("s_branch", "s_cbranch")) else None
        self.ends = self.op == "s_endpgm"
        self.falls = not self.ends and self.op not in ("s_branch", "s_setpc_b64")
        self.writes, self.reads, self.ab, self.c, self.passes = set(), set(), set(), set(), 0
        if self.mfma:
            self.writes, self.ab, self.c = registers(ops[0]), registers(ops[1]) | registers(ops[2]), registers(ops[3])
            for x in ops[4:]:
                self.ab |= registers(x)
            of = {k: int(n) for k, n in re.findall(r"(cbsz|blgp):(\d)", text)}
            # 16x16x128: 8 passes if A or B is in 8 bits
            self.passes = 8 if "16x16x128" in self.op and min(of.get("cbsz", 0), of.get("blgp", 0)) < 2 else 4
            self.reads = self.ab | self.c
        elif self.valu and ops:
            n = 2 if "_co_" in self.op or self.op.startswith(("v_div_scale", "v_mad_u64", "v_mad_i64")) else 1
            for x in ops[:n]:
                self.writes |= registers(x)
            for x in ops[n:]:
                self.reads |= registers(x)
            if self.op.startswith("v_swap"):
                self.reads, self.writes = self.reads | self.writes, self.reads | self.writes
        elif self.memory:
            loads = bool(re.search("load|read|permute|swizzle|_rtn", self.op)) and "lds" not in rest.split()
            self.writes = registers(ops[0]) if loads else set()
            for x in ops[loads:]:
                self.reads |= registers(x)


class Function:
    def __init__(self, lines):
        self.body, self.labels = [], {}
        for line in lines:
            label = re.match(r"^(\.LBB\w+):", line)
            if label:
                self.labels[label.group(1)] = len(self.body)
                continue
            text = re.sub(r"\s+", " ", line.split(";")[0]).strip()
            if text and not text.startswith(".") and not text.endswith(":"):
                self.body.append(Instruction(text))

    def after(self, at):
        i = self.body[at]
        return ([self.labels[i.target]] if i.target else []) + ([at + 1] if i.falls and at + 1 < len(self.body) else [])

    def walk(self, at, limit, stop):
        """Every instruction that is met fewer than `limit` states after `at`, until stop(instruction, states)."""
        least, todo = {}, [(n, 0) for n in self.after(at)]
        while todo:
            n, states = todo.pop()
            if states >= limit or least.get(n, limit) <= states:
                continue
            least[n] = states
            if not stop(self.body[n], states):
                todo += [(m, states + self.body[n].states) for m in self.after(n)]

    def early(self):
        """(what, first, second, states between, states needed) of everything that comes too early."""
        found = []
        for at, i in enumerate(self.body):
            scalars = {r for r in i.writes if r == "vcc" or r[0] == "s"} if i.valu else set()

            def matrix(j, states, i=i):
                if j.mfma:
                    if j.ab & i.writes:
                        found.append(("product of a product", i.text, j.text, states, i.passes + 4))
                    elif j.c & i.writes and j.c != i.writes and states < i.passes + 2:
                        found.append(("part of a sum", i.text, j.text, states, i.passes + 2))
                    return i.writes <= j.writes
                if j.valu and j.writes & (i.c - i.writes) and states < i.passes - 1:
                    found.append(("sum overwritten", i.text, j.text, states, i.passes - 1))
                if (j.valu or j.memory) and (j.reads | j.writes) & i.writes:
                    found.append(("product's result", i.text, j.text, states, i.passes + 4))
                    return True
                return False

            def transcendental(j, states, i=i):
                if (j.valu or j.mfma) and not j.op.startswith(TRANSCENDENTAL) and (j.reads | j.writes) & i.writes:
                    found.append(("transcendental", i.text, j.text, states, 1))
                return True

            def scalar(j, states, i=i, scalars=scalars):
                if j.memory and not j.op.startswith("ds_") and j.reads & scalars and not GUARD.match(j.text):
                    found.append(("scalar of a vector", i.text, j.text, states, 5))
                    return True
                return False

            def exchange(j, states, i=i):
                lanes = "permlane" in j.op or re.search("quad_perm|row_", j.text)
                if (j.mfma and j.reads & i.writes) or (lanes and (j.reads | (j.writes if "permlane" in j.op else set())) & i.writes):
                    found.append(("vector into a product or another lane", i.text, j.text, states, 2))
                return i.writes <= j.writes

            if i.valu:
                self.walk(at, 2, exchange)
            if i.mfma:
                self.walk(at, i.passes + 4, matrix)
            elif i.valu and i.op.startswith(TRANSCENDENTAL):
                self.walk(at, 1, transcendental)
            if scalars:
                self.walk(at, 5, scalar)
        return found


def functions(lines):
    """(name, lines) of every function of an assembly listing."""
    out, body = [], None
    for line in lines:
        name = re.match(r"^(_Z\w+):", line)
        if name:
            body = []
            out.append((name.group(1), body))
        elif line.startswith(".Lfunc_end"):
            body = None
        elif body is not None:
            body.append(line)
    return out


PRODUCT = "\tv_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], v[0:3]"


def found(*lines):
    return [(what, states) for what, _, _, states, _ in Function(lines).early()]


def test_straight_lines():
    use = "\tv_add_f32_e32 v20, v2, v21"
    assert found(PRODUCT, "\ts_nop 6", use) == [("product's result", 7)]
    assert found(PRODUCT, "\ts_nop 7", use) == []
    assert found(PRODUCT, "\ts_nop 6", "\tv_mov_b32_e32 v3, 0") == [("product's result", 7)]
    assert found(PRODUCT, "\tds_write_b128 v30, v[0:3]") == [("product's result", 0)]
    assert found(PRODUCT, PRODUCT, "\ts_nop 7", use) == []
    assert found(PRODUCT, PRODUCT.replace("v[8:11]", "v[0:3]")) == [("product of a product", 0)]
    assert found(PRODUCT, "\tv_mfma_f32_16x16x32_bf16 v[4:7], v[8:11], v[12:15], v[2:5]") == [("part of a sum", 0)]
    apart = "\tv_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], v[4:7]"
    assert found(apart, "\ts_nop 1", "\tv_mov_b32_e32 v7, 0") == [("sum overwritten", 2)]
    assert found(apart, "\ts_nop 2", "\tv_mov_b32_e32 v7, 0") == []
    wide = "\tv_mfma_f32_16x16x128_f8f6f4 v[0:3], v[8:15], v[16:23], 0"
    assert found(wide, "\ts_nop 10", use) == [("product's result", 11)] and found(wide, "\ts_nop 11", use) == []
    assert found(wide + " cbsz:4 blgp:4", "\ts_nop 7", use) == []


def test_the_way_around_a_side_block():
    side = ["\ts_nop 7", "\tv_mov_b32_e32 v0, v40"]
    use = "\tv_add_f32_e32 v20, v2, v21"
    around = [PRODUCT, "\ts_cbranch_vccnz .LBB0_2", "; %bb.1:", *side, ".LBB0_2:", use]
    assert found(*around) == [("product's result", 1)]
    assert found(PRODUCT, "\ts_nop 6", *around[1:]) == []
    loop = [".LBB0_1:", use, "\ts_nop 7", PRODUCT, "\ts_cbranch_scc1 .LBB0_1", "\ts_nop 7", "\ts_endpgm"]
    assert found(*loop) == [("product's result", 1)]


def test_other_waits():
    assert found("\tv_mov_b32_e32 v9, 0", "\ts_nop 0", PRODUCT) == [("vector into a product or another lane", 1)]
    assert found("\tv_mov_b32_e32 v9, 0", "\ts_nop 1", PRODUCT) == []
    assert found("\tv_mov_b32_e32 v9, 0", "\tv_permlane32_swap_b32_e32 v8, v9") == [("vector into a product or another lane", 0)]
    assert found("\tv_exp_f32_e32 v1, v2", "\tv_add_f32_e32 v3, v1, v1") == [("transcendental", 0)]
    assert found("\tv_exp_f32_e32 v1, v2", "\tv_exp_f32_e32 v4, v5", "\tv_add_f32_e32 v3, v1, v1") == []
    read = "\tv_readlane_b32 s7, v9, 3"
    load = "\tbuffer_load_dwordx4 v1, s[4:7], s11 offen lds"
    assert found(read, "\ts_nop 3", load) == [("scalar of a vector", 4)] and found(read, "\ts_nop 4", load) == []
    assert found(read, "\tbuffer_load_dword v1, v1, s[4:7], 0 offen", "\ts_nop 3", load) == []


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    out = [(name, Function(lines)) for name, lines in functions(_device_asm(tmp_path_factory.mktemp("asm")))]
    assert sum(any(i.mfma for i in f.body) for _, f in out) > 60
    return [(name, f.early()) for name, f in out]


def test_no_product_is_read_early(kernels):
    wrong = [(name, *x) for name, early in kernels for x in early
             if x[0] in ("product's result", "product of a product", "part of a sum", "sum overwritten")]
    assert not wrong, wrong[:10]


def test_no_transcendental_is_read_early(kernels):
    wrong = [(name, *x) for name, early in kernels for x in early if x[0] == "transcendental"]
    assert not wrong, wrong[:10]


def test_no_vector_is_used_early(kernels):
    wrong = [(name, *x) for name, early in kernels for x in early if x[0] == "vector into a product or another lane"]
    assert not wrong, wrong[:10]


def test_no_scalar_is_used_early(kernels):
    wrong = [(name, *x) for name, early in kernels for x in early if x[0] == "scalar of a vector"]
    assert not wrong, wrong[:10]
