"""The waits of the two kernels of large products that test_linear_waits.py does not read, checked without a GPU.

k_mx_big: its copies, reads, waits and barriers are taken from the source and played through as there, with the scales'
copies and reads among them.  k_linear_pair: its schedule is played through by the index arithmetic of the source, whose
lines the test names.
"""
import os
import re

import pytest

import quantized_expert_gemv_sigmoid_amd as moe

SOURCE = open(os.path.join(os.path.dirname(moe.__file__), "csrc", "linear_dev.h")).read()
UNIT = re.compile(r"unit\(D(\d)\{\}, r(\w+), s(\w+), (?:BUF \+ )?(\w+), (\w+)\);")
STEP = re.compile(r"turn\(f([ab]), (-?)BUF\)|phase\(check, D(\d)\{\}, r(\w+), s(\w+), (?:BUF \+ )?(\w+), (\w+), .*?"
                  r"read([AB])\(\w+, (\w+), i\)")
COPIES, READS = 5, 12    # per unit and wave: four of codes, one of scales; of a half: eight fragments, four pairs of scales


class Wave:
    """Every wave runs the same sequence: behind a barrier all have what the wait before it guarantees."""

    def __init__(self):
        self.copies, self.reads, self.done, self.all = [], [], (0, 0), (0, 0)

    def wait(self, n, lds):
        self.done = max(self.done[0], len(self.copies) - n), max(self.done[1], len(self.reads) - lds)

    def barrier(self):
        self.all = self.done

    def copy(self, place, what, n=1):
        held = [i for i, r in enumerate(self.reads) if r[0] == place]
        assert not held or held[-1] < self.all[1], f"{place} is filled with {what} while reads of it may be under way"
        self.copies += [(place, what)] * n

    def read(self, place, what, n=1, whole=1):
        last = [i for i, c in enumerate(self.copies) if c[0] == place][-whole:]
        for i in last:
            assert self.copies[i][1] == what, f"{place} holds {self.copies[i][1]} where {what} is read"
            assert i < self.all[0], f"{place}, {what}: read before its copies are known to be there"
        self.reads += [(place, what)] * n


def test_mx_big():
    text = re.sub(r"//[^\n]*", "", SOURCE[SOURCE.index("void k_mx_big("):])
    text = text[text.index("unit(D0{}, rA0"):text.index("two_stages(No{})")]
    first, rest = text.split("auto phase =")
    head, stages = rest.split("auto two_stages =")
    wave = Wave()
    filled = UNIT.findall(first)
    assert len(filled) == 8 and all(r == s == at and (b == "true") == (r[0] == "B") for _, r, s, at, b in filled)
    for d, unit, _, _, _ in filled:
        wave.copy((unit, int(d)), int(d), COPIES)
    waits = re.findall(r"wait_copies<(\d+)>\(\);", first)
    assert len(waits) == 2 and first.index("barrier()") < first.index("readA(a0, A0, i)") < first.rindex("wait_copies")
    wave.wait(int(waits[0]), 0)
    wave.barrier()
    for unit in ("A0", "B0"):
        wave.read((unit, 0), 0, READS)
    wave.wait(int(waits[1]), 0)
    (n, lds), = re.findall(r"wait_copies<(\d+), (\d+)>\(\);\s*barrier\(\);", head)
    assert "if (i < 4) h.s[i] =" in SOURCE[SOURCE.index("void k_mx_big("):]
    assert "if (i % 4 == 0) read(i >> 2);" in head and "if (i % 6 == 2 && i < 30) copy(check, d, r, s, at, b, i / 6);" in head
    steps = STEP.findall(stages)
    assert sum(not s[0] for s in steps) == 8
    buffer = {"A": 0, "B": 0}
    for turn in range(5):
        for side, minus, d, r, s, at, b, half, unit in steps:
            if side:
                buffer[side.upper()] += -1 if minus else 1
                continue
            assert r == s == at and (b == "true") == (r[0] == "B") and half == unit[0]
            wave.wait(int(n), int(lds))
            wave.barrier()
            # copies and reads come in any order: each has to be sound beside the other
            place, stage = (r, int(d) % 2), 2 * turn + int(d)
            source = (unit, buffer[half])
            assert place != source
            now = max(w for p, w in wave.copies if p == source)
            wave.copy(place, stage, COPIES)
            wave.read(source, now, READS)
        assert buffer == {"A": 0, "B": 0}
    # what a phase reads is the stage that the next one multiplies
    read = [w for p, w in wave.reads if p[0] == "A1"][::READS]
    assert read == list(range(len(read)))


@pytest.mark.parametrize("mx", [False, True])
def test_pair(mx):
    text = SOURCE[SOURCE.index("void k_linear_pair("):SOURCE.index("served batches")]
    for line in ("wait_copies<4 * G::C - 1>();", "wait_copies<3 * G::C>();", "if (q == 0) read_b(s & 1);", "read_a((q + 1) & 1, next);",
                 "copy(i / 4, (q + 1) & 3, q == 3 ? s + 2 : s + 1, slot, true, q == 0 ? s + 1 : s + 2);",
                 "const int next = slot + 1 == G::NA ? 0 : slot + 1;", "const int j = (q + 2) & 3;", "static constexpr int C = MX ? 4 : 3;"):
        assert line in text or line in SOURCE, line
    assert re.search(r"first\(1\);\s*first\(2\);\s*first\(3\);\s*copies\(0, 0, 0, true, 0\);\s*copies\(1, 0, 1, false, 0\);\s*"
                     r"copies\(2, 0, 2, true, 1\);\s*copies\(3, 0, 3, true, 1\);\s*copies\(0, 1, 4, true, 1\);", text)
    na, c = int(re.search(r"NA = (\d+), NB = 2", SOURCE).group(1)), 4 if mx else 3
    wave = Wave()

    def copies(q, stage, slot, x, xstage):
        wave.copy(("A", slot), 4 * stage + q, 2)
        if x:
            wave.copy(("B", xstage & 1), (xstage, (q + 2) & 3))
        if mx:   # the scales' copy, to any of these places by the wave: the last of the phase
            wave.copies.append((("A", slot), 4 * stage + q))

    def read_b(slot, s):
        for j in range(4):
            last = max(i for i, e in enumerate(wave.copies) if e[0] == ("B", slot) and e[1][1] == j)
            assert wave.copies[last][1] == (s, j) and last < wave.all[0]
        wave.reads += [(("B", slot), s)] * 8

    for q in (1, 2, 3):
        wave.copy(("B", 0), (0, (q + 2) & 3))
        if mx:
            wave.copies.append((("pad", 0), 0))
    copies(0, 0, 0, True, 0)
    copies(1, 0, 1, False, 0)
    copies(2, 0, 2, True, 1)
    copies(3, 0, 3, True, 1)
    copies(0, 1, 4, True, 1)
    wave.wait(4 * c - 1, 0)
    wave.barrier()
    wave.read(("A", 0), 0, 4, 2)
    slot = 0
    for s in range(6):
        for q in range(4):
            nxt = (slot + 1) % na
            wave.wait(3 * c, 0)
            wave.barrier()
            if q == 0:
                read_b(s & 1, s)
            wave.read(("A", nxt), 4 * s + q + 1, 4, 2 + mx)
            copies((q + 1) & 3, s + 2 if q == 3 else s + 1, slot, True, s + 1 if q == 0 else s + 2)
            slot = nxt
