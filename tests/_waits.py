"""Wait states in gfx950 assembly: how far apart dependent instructions stand, on
the shortest way through the control flow (loops' back edges included).

The hardware does not hold these back by itself, and the compiler, which puts
s_nop between them in its own code, does not look inside inline assembly.  An
instruction counts one wait state, s_nop n counts n + 1."""
import re

FAR = 64                        # distances are followed up to here

# What the compiler keeps between its own instructions on gfx950:
SGPR_TO_VMEM = 5        # a vector instruction writes a scalar register, a memory one reads it
M0_TO_LDS_LOAD = 1      # a scalar instruction writes m0, a load fills LDS from it
VALU_TO_MFMA = 2        # a vector instruction writes an operand of a matrix instruction
# a matrix instruction's result is read or overwritten by a vector or memory instruction
MFMA_TO_VALU = {"16x16x32": 8, "32x32x2": 18}
MFMA_TO_VALU_MOST = 19


def regs(tok):
    """The registers of one operand."""
    tok = tok.strip().lstrip("-|").rstrip("|")
    m = re.match(r"([avs])\[(\d+):(\d+)\]$", tok)
    if m:
        return [(m.group(1), i) for i in range(int(m.group(2)), int(m.group(3)) + 1)]
    m = re.match(r"([avs])(\d+)$", tok)
    if m:
        return [(m.group(1), int(m.group(2)))]
    if tok in ("vcc", "exec"):
        return [(tok, 0), (tok, 1)]
    if re.match(r"(vcc|exec)_(lo|hi)$", tok):
        return [(tok[:-3], int(tok.endswith("hi")))]
    return [("m0", 0)] if tok == "m0" else []


class Ins:
    def __init__(self, op, toks, inline, line):
        self.op, self.toks, self.inline, self.line = op, toks, inline, line
        self.states = int(toks[0], 0) + 1 if op == "s_nop" else 1
        self.mfma = op.startswith("v_mfma")
        self.valu = op.startswith("v_") and not self.mfma
        self.vmem = op.startswith(("buffer_", "global_", "scratch_", "flat_"))
        self.lds_load = self.vmem and "_load" in op and "lds" in toks
        outs = 1
        if self.valu and ("_co_" in op or op.startswith(("v_div_scale", "v_mad_u64", "v_mad_i64"))):
            outs = 2
        if "swap" in op:
            outs = 2
        if op.startswith(("s_cmp", "s_bitcmp", "s_waitcnt", "s_barrier", "s_nop", "s_cbranch",
                          "s_branch", "s_endpgm", "s_setprio", "s_trap", "ds_write")):
            outs = 0
        if self.vmem and "_store" in op or self.lds_load:
            outs = 0
        self.writes = [r for t in toks[:outs] for r in regs(t)]
        self.reads = [r for t in toks[0 if "swap" in op else outs:] for r in regs(t)]
        if op.startswith("v_cmp") and op.endswith("_e32"):
            self.writes = [("vcc", 0), ("vcc", 1)]
        self.wait = next((n for k, n in MFMA_TO_VALU.items() if k in op), MFMA_TO_VALU_MOST)


def functions(asm, match=r"\w+"):
    """-> name, [blocks]; a block is (instructions, the blocks that may follow)."""
    for m in re.finditer(r"^(%s):[^\n]*\n" % match, asm, re.M):
        end = asm.find("\n.Lfunc_end", m.end())
        if end > 0:
            yield m.group(1), blocks(asm[m.end():end])


def blocks(body):
    labels, ins, inline = {}, [[]], False
    for line in body.split("\n"):
        if ";;#ASMSTART" in line or ";;#ASMEND" in line:
            inline = "START" in line
            continue
        code = line.split(";")[0]
        lab = re.match(r"(\.?\w+):", code)
        if lab:
            ins.append([])
            labels[lab.group(1)] = len(ins) - 1
            continue
        if not code.startswith("\t") or not code.strip() or code.strip().startswith("."):
            continue
        p = code.strip().split(None, 1)
        toks = re.split(r"[,\s]+", p[1].strip()) if len(p) > 1 else []
        ins[-1].append(Ins(p[0], toks, inline, line.strip()))
        if p[0].startswith(("s_cbranch", "s_branch", "s_endpgm")):
            ins.append([])
    res = []
    for i, b in enumerate(ins):
        after = []
        if b and b[-1].op.startswith(("s_cbranch", "s_branch")):
            after.append(labels[b[-1].toks[0]])
        if not (b and b[-1].op in ("s_branch", "s_endpgm")) and i + 1 < len(ins):
            after.append(i + 1)
        res.append((b, after))
    return res


def walk(ins, entry, found=None):
    """Through a block's instructions from the distances at its entry to those at its
    end; those too short on the way go to `found`.  A distance: (kind of writer,
    register) -> (wait states since, inline, line, wait of a matrix instruction)."""
    now = 0
    state = {k: (-w[0],) + w[1:] for k, w in entry.items()}

    def near(kind, r, rule, least):
        w = state.get((kind, r))
        if w is None or not (w[1] or i.inline) or now - w[0] >= FAR:
            return
        d, least = now - w[0], w[3] if least is None else least
        found.least[rule] = min(found.least.get(rule, FAR), d)
        if d < least:
            found.append((rule, d, least, w[2], i.line))

    for i in ins:
        if found is not None:
            if i.vmem:
                for r in i.reads:
                    if r[0] in ("s", "vcc", "m0"):
                        near("valu", r, "sgpr", SGPR_TO_VMEM)
            if i.lds_load:
                near("salu", ("m0", 0), "m0", M0_TO_LDS_LOAD)
            if i.mfma:
                for r in i.reads:
                    near("valu", r, "mfma in", VALU_TO_MFMA)
            elif i.valu or i.vmem or i.op.startswith("ds_"):
                for r in i.reads + i.writes:
                    near("mfma", r, "mfma out", None)
        now += i.states
        kind = "valu" if i.valu else "mfma" if i.mfma else "salu" if i.op.startswith("s_") else None
        for r in i.writes:
            for other in ("valu", "salu", "mfma"):
                state.pop((other, r), None)
            if kind:
                state[(kind, r)] = (now, i.inline, i.line, i.wait)
    return {k: (now - w[0],) + w[1:] for k, w in state.items() if now - w[0] < FAR}


class Found(list):
    def __init__(self):
        self.least = {}


def scan(blks):
    """-> Found: (rule, distance, least, writer, reader) of every pair with inline
    assembly at one end that stands too close on some way through the blocks;
    .least: the shortest distance of each rule."""
    entry = [None] * len(blks)
    entry[0] = {}
    todo = [0]
    while todo:
        n = todo.pop()
        state = walk(blks[n][0], entry[n])
        for a in blks[n][1]:
            if entry[a] is None:
                entry[a] = dict(state)
                todo.append(a)
                continue
            nearer = {k: w for k, w in state.items() if k not in entry[a] or w[0] < entry[a][k][0]}
            if nearer:
                entry[a].update(nearer)
                todo.append(a)
    found = Found()
    for (ins, _), state in zip(blks, entry):
        if state is not None:
            walk(ins, state, found)
    return found
