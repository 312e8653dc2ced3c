"""Wait states before the gated delta rule's loads into LDS, from the assembly of its kernels (CPU only).

A vector instruction that writes a scalar register (v_readfirstlane, v_readlane, carries, comparisons) has
to be five wait states ahead of a vector memory instruction that reads the register as its descriptor or
offset; the hardware does not wait by itself.  The compiler sees to it for the accesses that it makes, but
does not look into inline assembly, so that each such access has to bring its own.  An instruction is one
wait state, s_nop N is N + 1.
"""
import concurrent.futures as cf
import os
import re
import subprocess

import pytest

from mamba2_ssd_chunked_amd import build as B

STATES = 5


def _registers(text):
    """Numbers of the scalar registers that an operand names; vcc's are 106 and 107, m0's 124."""
    out = set()
    for lo, hi in re.findall(r"\bs\[(\d+):(\d+)\]", text):
        out.update(range(int(lo), int(hi) + 1))
    out.update(int(n) for n in re.findall(r"\bs(\d+)\b", text))
    if re.search(r"\bvcc(_lo|_hi)?\b", text):
        out.update((106, 107))
    return out


def _written(op, args):
    """Scalar registers that a vector instruction writes: the first operand, or the second beside a vector
    register where there is a carry."""
    parts = [a.strip() for a in re.split(r",(?![^\[]*\])", args)]
    out = _registers(parts[0]) if parts else set()
    if len(parts) > 1 and re.match(r"v_(mad_[ui]64|add_co|sub_co|subrev_co|addc_co|subb_co|subbrev_co|div_scale)", op):
        out |= _registers(parts[1])
    if op.startswith("v_cmpx"):
        out = set()
    return out


def _blocks(lines):
    """Basic blocks of one function: [(label, instructions, labels it may go to, falls through)]."""
    blocks, label, code = [], "entry", []

    def end(to, through):
        nonlocal label, code
        blocks.append((label, code, to, through))
        label, code = None, []

    for line in lines:
        line = line.split(";")[0].split("//")[0].strip()
        m = re.match(r"(\.?[\w$]+):$", line)
        if m:
            end([], True)
            label = m.group(1)
        elif line and not line.startswith("."):
            op, _, args = line.partition(" ") if "\t" not in line else line.partition("\t")
            code.append((op, args.strip()))
            if op == "s_endpgm":
                end([], False)
            elif op == "s_branch":
                end([args.strip()], False)
            elif op.startswith("s_cbranch"):
                end([args.strip()], True)
            else:
                assert op not in ("s_setpc_b64", "s_swappc_b64"), line
    end([], False)
    return blocks


def _through(code, since, report=None):
    """The scalar registers written less than STATES ago, with the wait states since, behind a block."""
    since = dict(since)
    for op, args in code:
        if report is not None and re.match(r"(buffer|global|flat|scratch)_", op):
            for r in sorted(_registers(args) & set(since)):
                report.append((op + " " + args, r, since[r]))
        step = int(args) + 1 if op == "s_nop" else 1
        since = {r: n + step for r, n in since.items() if n + step < STATES}
        if op.startswith("v_"):
            since.update({r: 0 for r in _written(op, args)})
        else:  # whatever a scalar instruction writes is ready
            for r in _registers(args.split(",")[0]) if op.startswith("s_") and not op.startswith("s_cmp") else ():
                since.pop(r, None)
    return since


def hazards(text):
    """(function, access, register, wait states) of every access that comes too early."""
    found, count = [], 0
    for m in re.finditer(r"^(_Z\w+|\w+):[^\n]*\n(.*?)^\.Lfunc_end", text, re.S | re.M):
        blocks = _blocks(m.group(2).split("\n"))
        at = {b[0]: i for i, b in enumerate(blocks) if b[0]}
        enter = [{} for _ in blocks]
        todo = list(range(len(blocks)))
        while todo:
            i = todo.pop()
            _, code, to, through = blocks[i]
            out = _through(code, enter[i])
            for j in [at[t] for t in to] + ([i + 1] if through and i + 1 < len(blocks) else []):
                worse = {r: n for r, n in out.items() if n < enter[j].get(r, STATES)}
                if worse:
                    enter[j].update(worse)
                    todo.append(j)
        for i, (_, code, _, _) in enumerate(blocks):
            count += sum(1 for op, args in code if op.startswith("buffer_load") and args.endswith("lds"))
            report = []
            _through(code, enter[i], report)
            found += [(m.group(1),) + r for r in report]
    return found, count


def test_the_scan_sees_what_it_is_for():
    def kernel(*body):
        return "kernel:\n" + "\n".join(body) + "\n s_endpgm\n.Lfunc_end0:\n"

    load = " buffer_load_dword v1, s[4:7], 0 offen lds"
    near, count = hazards(kernel(" v_readfirstlane_b32 s6, v0", " s_mov_b32 m0, s9", " s_nop 0", load))
    assert count == 1 and [(f[2], f[3]) for f in near] == [(6, 2)]
    assert not hazards(kernel(" v_readfirstlane_b32 s6, v0", " s_mov_b32 m0, s9", " s_nop 3", load))[0]
    assert not hazards(kernel(" v_readfirstlane_b32 s8, v0", load))[0]
    assert hazards(kernel(" v_mad_u64_u32 v[2:3], s[4:5], v0, v1, v[2:3]", load))[0]
    assert not hazards(kernel(" v_readlane_b32 s4, v0, 1", " s_and_b32 s4, s4, s5", load))[0]
    # around a loop
    body = [" s_nop 4", ".LBB0_1:", load, " v_readfirstlane_b32 s4, v0", " s_cbranch_scc1 .LBB0_1"]
    assert [f[3] for f in hazards(kernel(*body))[0]] == [1]


@pytest.mark.skipif(not os.path.exists(B.HIPCC), reason="needs hipcc")
def test_loads_into_lds_wait_for_their_descriptors(tmp_path):
    def assembly(src):
        out = str(tmp_path / (src + ".s"))
        subprocess.run([B.HIPCC] + B.FLAGS + B.EXTRA_FLAGS.get(src, []) + ["-x", "hip", "-S", "--cuda-device-only",
                       os.path.join(B.CSRC, src), "-o", out], check=True, capture_output=True)
        with open(out) as f:
            return f.read()

    with cf.ThreadPoolExecutor(max_workers=2) as ex:
        for text in ex.map(assembly, ["gdelta_bwd.hip", "gdelta_fwd.hip"]):
            found, count = hazards(text)
            assert count > 100  # the loads are there
            assert not found, (len(found), found[:5])
