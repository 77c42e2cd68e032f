"""The order of the two softmax groups of the many-rows attention kernel, on a
model of them, under schedules in which some warps are late.

The model has the waits and arrivals of iq_kv_attention_rows.cu that concern a
segment's maximum (m_full, s_m, s_top) and what bounds how far the warps can
drift apart (scores, products, sums).  How many m_full there are, and whether a
barrier stands between reading s_top and storing the next one, is read from the
source.  A wait that returns too early or never, and a store over what some warp
has still to read, are seen as wrong data or as no progress."""

import random
import re
from pathlib import Path

import pytest

SOURCE = (Path(__file__).resolve().parents[1] / "fp4_fp8_quant_gb300" / "csrc" / "iq_kv_attention_rows.cu").read_text()
WARPS = 4                    # of a group; the model's unit of arrival


USES = re.findall(r"(?:mbar_arrive|mbar_wait)\((&?m_full[^,)]*)", SOURCE)
M_FULL = 2 if USES and all("[sb]" in u for u in USES) else 1      # one per parity of the segment, or one for all
TOP_READ = bool(re.search(r"mbar_wait\(&top_read\[group\].*?s_top\[.*?mbar_arrive\(&top_read\[group\]\)", SOURCE, re.S))


class Barrier:
    def __init__(self, count):
        self.count, self.here, self.phase = count, 0, 0

    def arrive(self):
        self.here += 1
        if self.here == self.count:
            self.here, self.phase = 0, self.phase + 1

    def passed(self, parity):
        """Whether the phase of that parity has completed, as the hardware sees it."""
        return (self.phase & 1) != parity


class Model:
    def __init__(self, lengths, m_full, top_read):
        self.lengths, self.n_mf = lengths, m_full
        self.top_read = [Barrier(WARPS) for _ in range(2)] if top_read else None
        self.s_top = {}
        self.tiles = sum(lengths)
        self.m_full = [Barrier(WARPS) for _ in range(m_full)]
        self.meet = [Barrier(WARPS) for _ in range(2)]
        self.sum_full = [Barrier(2 * WARPS) for _ in range(2)]
        self.sum_empty = [Barrier(1) for _ in range(2)]
        self.p_full = [0] * self.tiles                       # warps that have stored a tile's weights
        self.scored = self.multiplied = 0                    # tiles done by the tensor cores
        self.s_m = [None] * 2
        self.wrong = []

    def tensor_cores(self):
        """Scores up to three tiles ahead of the products, products in order."""
        while True:
            if self.multiplied < self.tiles and self.p_full[self.multiplied] == WARPS:
                self.multiplied += 1
            if self.scored < self.tiles and self.scored < self.multiplied + 3:
                self.scored += 1
            yield lambda: True
            if self.multiplied == self.tiles and self.scored == self.tiles:
                return

    def output(self):
        for seg in range(len(self.lengths)):
            b = seg & 1
            yield lambda: self.sum_full[b].passed(seg >> 1 & 1)
            last = sum(self.lengths[:seg + 1])
            yield lambda: self.multiplied >= last
            if self.s_m[b] != seg:
                self.wrong.append(("output", seg, self.s_m[b]))
            self.sum_empty[b].arrive()

    def softmax(self, group, warp):
        tile = meets = 0
        for seg, n in enumerate(self.lengths):
            b = seg & 1
            mine = (tile ^ group) & 1
            full = self.m_full[seg % self.n_mf]
            parity = (seg // self.n_mf) & 1
            for i in range(mine, n, 2):
                t = tile + i
                yield lambda: self.scored > t
                if i == 0:
                    if self.top_read:
                        yield lambda: self.top_read[group].passed((meets & 1) ^ 1)
                    self.s_top[group, warp] = seg
                    yield lambda: True
                    self.meet[group].arrive()
                    yield lambda: self.meet[group].passed(meets & 1)
                    meets += 1
                    for w in range(WARPS):                   # (the other half of a row is another warp's)
                        if self.s_top[group, w] != seg:
                            self.wrong.append(("s_top", seg, self.s_top[group, w]))
                    if self.top_read:
                        self.top_read[group].arrive()
                    yield lambda: self.sum_empty[b].passed((seg >> 1 & 1) ^ 1)
                    self.s_m[b] = seg
                    yield lambda: True
                    full.arrive()
                elif i == mine:
                    yield lambda: full.passed(parity)
                    if self.s_m[b] != seg:
                        self.wrong.append(("s_m", seg, self.s_m[b]))
                yield lambda: True
                self.p_full[t] += 1
            tile += n
            yield lambda: self.sum_empty[b].passed((seg >> 1 & 1) ^ 1)
            self.sum_full[b].arrive()


def _run(model, rng, late):
    """Steps the roles in random order, the late ones only when no other can
    move or once in a while; False when nothing can move."""
    roles = {"tensor": model.tensor_cores(), "output": model.output()}
    roles |= {(g, w): model.softmax(g, w) for g in range(2) for w in range(WARPS)}
    waits = {name: next(role) for name, role in roles.items()}
    while True:
        ready = [name for name in waits if name != "tensor" and waits[name]()]
        if "tensor" in waits:
            moved = (model.scored, model.multiplied)
            try:
                waits["tensor"] = next(roles["tensor"])
            except StopIteration:
                del waits["tensor"]
            if moved != (model.scored, model.multiplied):
                continue
        if not waits or not [n for n in waits if n != "tensor"]:
            return True
        if not ready:
            return False
        prompt = [name for name in ready if name not in late]
        name = rng.choice(prompt if prompt and rng.random() < 0.98 else ready)
        try:
            waits[name] = next(roles[name])
        except StopIteration:
            del waits[name]


SEGMENTS = [[2] * 8, [1] * 9, [1, 2] * 5, [1, 1, 2, 2, 1, 3] * 2, [2, 2, 1] * 4, [3, 2, 5, 1, 1, 4], [2, 1, 2, 1, 1, 7]]


def _faults(m_full, top_read):
    found = []
    for lengths in SEGMENTS:
        for seed in range(60):
            rng = random.Random(seed)
            late = set(rng.sample([(g, w) for g in range(2) for w in range(WARPS)], rng.randint(1, 4)))
            model = Model(lengths, m_full, top_read)
            if not _run(model, rng, late):
                found.append(("no progress", lengths, seed))
            found += model.wrong
    return found


def test_a_segment_s_maximum_is_ordered():
    assert _faults(M_FULL, True) == []


def test_the_halves_of_a_row_read_each_other_s_maximum():
    assert _faults(2, TOP_READ) == []


def test_the_model_sees_one_barrier_for_all_segments():
    seen = {f[0] for f in _faults(1, True)}
    assert "s_m" in seen and "no progress" in seen


def test_the_model_sees_a_maximum_stored_over_an_unread_one():
    assert {f[0] for f in _faults(2, False)} == {"s_top"}
