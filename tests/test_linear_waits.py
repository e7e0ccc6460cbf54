"""The waits of the product's 256 x 256 kernel, checked on its source (no GPU).

Its four waves fill LDS by copies that only a wave's own counter orders, and read it behind barriers.  The sequence of
copies, reads, waits and barriers is taken from the source and played through for several turns with the counters'
guarantees alone: behind a wait for (N, L) all that the wave issued is done but the last N copies and the last L reads.
Every wave runs the same sequence, so behind a barrier all waves have what the wait before it guarantees.
"""
import os
import re

import quantized_expert_gemv_sigmoid_amd as moe

SOURCE = os.path.join(os.path.dirname(moe.__file__), "csrc", "linear_dev.h")
WAIT = re.compile(r"wait_copies<(\d+)(?:, (\d+))?>\(\)|(\bbarrier\(\))|read([AB])\(\w+, (\w+), i\)")
UNIT = re.compile(r"unit\(D(\d)\{\}, r(\w+), (?:BUF \+ )?(\w+),")
STEP = re.compile(r"turn\(f([ab]), -?BUF\)|phase\(check, D(\d)\{\}, r(\w+), (?:BUF \+ )?(\w+),.*?read([AB])\(\w+, (\w+), i\)")


def waits(text):
    """The waits, barriers and reads of a piece of source in their order."""
    for n, lds, barrier, half, unit in WAIT.findall(text):
        yield ("read", unit, half) if half else ("barrier",) if barrier else ("wait", int(n), int(lds or 0))


def sequence(turns=5):
    """Operations in order: ("wait", N, L), ("barrier",), ("copy", unit, stage) of four copies, ("read", unit, stage) of one
    fragment, and ("phase", copied unit, its stage, read unit, its stage), four copies and eight reads in any order.  A
    unit: matrix half and number of the buffer."""
    text = open(SOURCE).read()
    text = re.sub(r"//[^\n]*", "", text[text.index("void k_linear_big("):])
    text = text[text.index("unit(D0{}, rA0"):text.index("two_stages(No{})")]
    first, rest = text.split("auto phase =")
    phase, stages = rest.split("auto two_stages =")

    filled = UNIT.findall(first)
    assert len(filled) == 8 and all(a == b for _, a, b in filled)
    seq = [("copy", (unit, int(d)), int(d)) for d, _, unit in filled]
    fragments = [op for op in waits(first) if op[0] == "read"]
    assert [op[1] for op in fragments] == ["A0", "B0"]
    for op in waits(first):
        if op == fragments[0]:   # one loop over both: any of them may be the last
            seq += [("read", (unit, 0), 0) for _ in range(8) for _, unit, _ in fragments]
        elif op[0] != "read":
            seq.append(op)

    head = list(waits(phase))
    assert [op[0] for op in head] == ["wait", "barrier"]
    steps = STEP.findall(stages)
    assert [bool(s[0]) for s in steps].count(False) == 8 and all(s[2] == s[3] for s in steps)
    stage = {"A": 0, "B": 0}     # which one's halves are read
    for turn in range(turns):
        for side, d, _, unit, half, read in steps:
            if side:
                stage[side.upper()] += 1
            else:
                seq += head + [("phase", (unit, int(d) % 2), 2 * turn + int(d), (read, stage[half] % 2), stage[half])]
    return seq


def play(seq):
    copies, reads = [], []             # (unit, stage) in the order of their issue
    done, all_done = (0, 0), (0, 0)    # how many of each this wave has waited for, and how many every wave has

    def check_read(unit, stage):
        last = max(i for i, c in enumerate(copies) if c[0] == unit)
        assert copies[last][1] == stage, f"{unit} holds stage {copies[last][1]} where {stage} is read"
        assert last < all_done[0], f"{unit}, stage {stage}: read before its copies are known to be there"

    def check_copy(unit, stage):
        held = [i for i, r in enumerate(reads) if r[0] == unit]
        assert not held or held[-1] < all_done[1], f"{unit} is filled with stage {stage} while reads of it may be under way"

    for op in seq:
        if op[0] == "wait":
            done = max(done[0], len(copies) - op[1]), max(done[1], len(reads) - op[2])
        elif op[0] == "barrier":
            all_done = done
        elif op[0] == "copy":
            check_copy(*op[1:])
            copies += [op[1:]] * 4
        elif op[0] == "read":
            check_read(*op[1:])
            reads.append(op[1:])
        else:
            check_read(*op[3:])
            check_copy(*op[1:3])
            assert op[1] != op[3]
            copies += [op[1:3]] * 4
            reads += [op[3:]] * 8


def test_copies_are_there_and_reads_are_done():
    seq = sequence()
    assert sum(op[0] == "phase" for op in seq) == 40
    play(seq)
