"""Wait states in the built kernels. The hardware does not interlock some pairs of instructions; the compiler
keeps them apart by instructions or s_nop, but cannot see into inline assembly. This reads the gfx950 code of
libnhm.so and counts, over every path, the wait states between such pairs."""
import os
import re
import struct
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "fp8_w8a8_linear_amd", "libnhm.so")


def regs(text, kinds):
    """Registers named in text, of the kinds given (s, v, a), and m0 if kinds has m."""
    out = set()
    for kind, lo, hi in re.findall(r"\b([sva])\[(\d+):(\d+)\]", text):
        if kind in kinds:
            out |= {(kind, i) for i in range(int(lo), int(hi) + 1)}
    for kind, i in re.findall(r"\b([sva])(\d+)\b", text):
        if kind in kinds:
            out.add((kind, int(i)))
    if "m" in kinds and re.search(r"\bm0\b", text):
        out.add(("m", 0))
    return out


class Ins:
    __slots__ = ("op", "args", "target", "wait")

    def __init__(self, text, target=None):
        parts = text.split(None, 1)
        self.op, self.args = parts[0], [a.strip() for a in parts[1].split(",")] if len(parts) > 1 else []
        self.target = target          # index of a branch's target
        self.wait = int(self.args[0], 0) + 1 if self.op == "s_nop" else 1

    @property
    def vmem(self):
        return self.op.startswith(("buffer_", "global_", "flat_", "scratch_"))

    @property
    def store(self):
        return self.op.startswith(("buffer_store", "global_store", "flat_store", "scratch_store", "ds_write"))

    def text(self):
        return self.op + " " + ", ".join(self.args)


def writes_m0(i):
    return i.op.startswith("s_") and i.args and i.args[0] == "m0"


def valu_sgprs(i):
    """Scalar registers that a vector instruction writes."""
    if not i.op.startswith("v_") or not i.args:
        return set()
    out = regs(i.args[0], "s")
    if re.match(r"v_(add|sub|subrev|addc|subb|subbrev)_co|v_div_scale|v_mad_[ui]64", i.op) and len(i.args) > 1:
        out |= regs(i.args[1], "s")
    return out


def paths(code, start, limit, visit):
    """Instructions after start, each with the fewest wait states up to it, until visit says so or limit is reached."""
    stack, seen = [(start + 1, 0)], {}
    while stack:
        at, w = stack.pop()
        while at is not None and at < len(code) and w < limit and seen.get(at, limit) > w:
            seen[at] = w
            i = code[at]
            if i.op == "s_endpgm" or visit(i, w):
                break
            w += i.wait
            if i.op.startswith("s_cbranch") and i.target is not None:
                stack.append((i.target, w))
            at = i.target if i.op == "s_branch" else at + 1


def m0_before_lds(code):
    """A scalar write of M0, then a load to LDS, which takes its address there: one wait state."""
    out = []
    for n, i in enumerate(code):
        if not writes_m0(i):
            continue

        def visit(j, w):
            if j.vmem and j.args[-1].endswith(" lds"):
                out.append((w, 1, i.text(), j.text()))
                return True
            return writes_m0(j)
        paths(code, n, 1, visit)
    return out


def sgpr_before_vmem(code):
    """A scalar register that a vector instruction writes (v_readfirstlane, v_readlane, a spilled one's reload), then
    a memory instruction that reads it, in its descriptor or offset: five wait states."""
    out = []
    for n, i in enumerate(code):
        mine = valu_sgprs(i)
        if not mine:
            continue

        def visit(j, w, left=mine):
            if j.vmem and regs(",".join(j.args), "s") & left:
                out.append((w, 5, i.text(), j.text()))
                return True
            return False
        paths(code, n, 5, visit)
    return out


# Wait states until a matrix instruction's result may be read or overwritten by others: four per pass and four more
# stand between them wherever the compiler issues a result's use in a straight line.
MFMA_WAIT = {"v_mfma_f32_16x16x32_bf16": 8, "v_mfma_f32_16x16x128_f8f6f4": 12, "v_mfma_f32_32x32x16_bf16": 12,
             "v_mfma_f32_32x32x64_f8f6f4": 20}


def mfma_result(code):
    """A matrix instruction, then a read of its result that is not the sum of another one, or a write over it."""
    out = []
    for n, i in enumerate(code):
        if not i.op.startswith("v_mfma"):
            continue
        want, mine = MFMA_WAIT[i.op], regs(i.args[0], "va")

        def visit(j, w, i=i, want=want, mine=mine):
            if not j.args or j.op.startswith("s_"):
                return False
            load = (j.vmem or j.op.startswith("ds_")) and not j.store
            to_lds = j.vmem and j.args[-1].endswith(" lds")
            reads = regs(",".join(j.args if j.store or to_lds else j.args[1:3] if j.op.startswith("v_mfma") else j.args[1:]), "va")
            writes = set() if j.store or to_lds else regs(j.args[0], "va")
            if reads & mine or (writes & mine and not load and not j.op.startswith("v_mfma")):
                out.append((w, want, i.text(), j.text()))
                return True
            return bool(writes & mine)
        paths(code, n, want, visit)
    return out


RULES = {"m0_before_lds": m0_before_lds, "sgpr_before_vmem": sgpr_before_vmem, "mfma_result": mfma_result}


def parse(lines):
    """llvm-objdump's lines of one function."""
    ins, where, targets = [], {}, []
    for line in lines:
        m = re.match(r"^\s+([a-z]\S*[^/]*?)\s*//\s*([0-9A-F]+):(.*)$", line)
        if not m:
            continue
        where[int(m[2], 16)] = len(ins)
        ins.append(Ins(m[1]))
        t = re.search(r"<\S+?(?:\+0x([0-9a-f]+))?>", m[3]) if m[1].startswith(("s_cbranch", "s_branch")) else None
        targets.append(None if not t else int(t[1] or "0", 16))
    if ins:
        first = min(where)
        for i, t in zip(ins, targets):
            i.target = None if t is None else where.get(first + t)
    return ins


def device_code(path):
    """{kernel: instructions} of the gfx950 code objects bundled in a library."""
    blob, magic, objdump = open(path, "rb").read(), b"__CLANG_OFFLOAD_BUNDLE__", "/opt/rocm/llvm/bin/llvm-objdump"
    if not os.path.exists(objdump):
        pytest.skip("llvm-objdump not found")
    out, at = {}, blob.find(magic)
    while at >= 0:
        count, = struct.unpack_from("<Q", blob, at + len(magic))
        p = at + len(magic) + 8
        for _ in range(count if count < 16 else 0):
            off, size, n = struct.unpack_from("<QQQ", blob, p)
            triple = blob[p + 24:p + 24 + n]
            p += 24 + n
            if b"gfx950" in triple and size:
                r = subprocess.run([objdump, "-d", "-"], input=blob[at + off:at + off + size], capture_output=True)
                assert r.returncode == 0, r.stderr.decode()
                name, lines = None, []
                for line in r.stdout.decode().splitlines() + ["0 <>:"]:
                    m = re.match(r"^[0-9a-f]+ <(.*)>:$", line)
                    if m:
                        if name and lines:
                            out[name] = parse(lines)
                        name, lines = m[1], []
                    else:
                        lines.append(line)
        at = blob.find(magic, at + 1)
    return out


@pytest.fixture(scope="module")
def code():
    if not os.path.exists(LIB):
        pytest.skip("libnhm.so is not built")
    kernels = device_code(LIB)
    assert any("tile256_kernel" in k for k in kernels) and any("beam_strip_kernel" in k for k in kernels)
    return kernels


@pytest.mark.parametrize("rule", sorted(RULES))
def test_built_kernels(code, rule):
    bad = {}
    for name, ins in code.items():
        for got, want, a, b in RULES[rule](ins):
            if got < want:
                bad.setdefault(name, []).append(f"{got} of {want}: {a} | {b}")
    assert not bad, "\n".join(f"{k}: {len(v)}, the first {v[0]}" for k, v in bad.items())


def listing(text):
    """Instructions of a listing with `name:` labels, branches to them by name."""
    ins, labels = [], {}
    for line in text.strip().splitlines():
        line = line.strip()
        if line.endswith(":"):
            labels[line[:-1]] = len(ins)
        else:
            ins.append(Ins(line))
    for i in ins:
        if i.op.startswith(("s_cbranch", "s_branch")):
            i.target = labels[i.args[0]]
    return ins


@pytest.mark.parametrize("rule,text,worst", [
    ("m0_before_lds", "s_mov_b32 m0, s4\nbuffer_load_dwordx4 v1, s[0:3], 0 offen lds", 0),
    ("m0_before_lds", "s_mov_b32 m0, s4\ns_nop 0\nbuffer_load_dwordx4 v1, s[0:3], 0 offen lds", None),
    ("m0_before_lds", "s_mov_b32 m0, s4\nbuffer_load_dwordx4 v[4:7], v1, s[0:3], 0 offen", None),
    ("sgpr_before_vmem", "v_readfirstlane_b32 s6, v2\ns_nop 3\nbuffer_load_dwordx4 v0, s[4:7], 0 offen lds", 4),
    ("sgpr_before_vmem", "v_readfirstlane_b32 s6, v2\ns_nop 4\nbuffer_load_dwordx4 v0, s[4:7], 0 offen lds", None),
    ("sgpr_before_vmem", "v_cmp_lt_i32_e64 s[8:9], v0, v1\ns_nop 4\nglobal_load_dword v0, v1, s[8:9]", None),
    ("sgpr_before_vmem", "a:\nbuffer_load_dword v0, v1, s[4:7], 0 offen\nv_readlane_b32 s7, v2, 3\ns_cbranch_scc1 a", 1),
    ("mfma_result", "v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]\ns_nop 6\nv_accvgpr_read_b32 v8, a3", 7),
    ("mfma_result", "v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]\ns_nop 7\nv_accvgpr_read_b32 v8, a3", None),
    ("mfma_result", "v_mfma_f32_32x32x16_bf16 v[0:15], v[20:23], v[24:27], 0\nv_mfma_f32_32x32x16_bf16 v[0:15], v[20:23], "
     "v[24:27], v[0:15]", None),
    # a loop over the parts of an adapter's product, as the compiler left it: seven ahead of the read across the back edge
    ("mfma_result", "a:\nds_read_b128 v[158:161], v156\nv_accvgpr_read_b32 v174, a8\nv_accvgpr_read_b32 v170, a4\ns_nop 2\n"
     "v_accvgpr_read_b32 v165, a3\nv_accvgpr_write_b32 a3, v165\ns_nop 1\n"
     "v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[158:161], a[0:3]\ns_cbranch_scc1 a", 7),
])
def test_rules(rule, text, worst):
    """What each rule finds in a listing: the fewest wait states of a pair that is too close, None without one."""
    found = [got for got, want, _, _ in RULES[rule](listing(text)) if got < want]
    assert (min(found) if found else None) == worst
