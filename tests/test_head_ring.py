"""The ring of shared-memory stages between the TMA warp and the groups of warps
of the 8-bit product of few tokens, followed step by step on the CPU: whichever
copy comes late, no group passes a wait for a stage that is not there."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Early(Exception):
    """A wait passed before what it waits for was there."""


def follow(slots, groups, total, late):
    """`total` stages through a ring of `slots`; the copy of stage `late` lands last of
    all that can.  Barriers are waited for by parity, as the hardware's are: a wait for a
    phase of parity p passes while the barrier's current phase has the other one."""
    full, empty = [0] * slots, [0] * slots      # completed phases
    issued, landed, at = 0, set(), [0] * groups
    passes = lambda done, phase: done % 2 != phase % 2  # noqa: E731

    def advance(hold):
        nonlocal issued
        moved = False
        slot, use = issued % slots, issued // slots
        if issued < total and (use == 0 or passes(empty[slot], use - 1)):
            if use and empty[slot] != use:
                raise Early
            issued += 1
            moved = True
        for i in range(issued):
            if i not in landed and i != hold:
                landed.add(i)
                full[i % slots] += 1
                moved = True
        for g in range(groups):
            if at[g] < total and at[g] % groups != g:      # another group's: passed over
                at[g] += 1
                moved = True
            elif at[g] < total and passes(full[at[g] % slots], at[g] // slots):
                if at[g] not in landed:
                    raise Early
                empty[at[g] % slots] += 1
                at[g] += 1
                moved = True
        return moved

    for hold in (late, None):
        while advance(hold):
            pass
    assert issued == total and len(landed) == total and min(at) == total   # nobody waits for ever


def every(slots, groups):
    for late in range(3 * slots):
        follow(slots, groups, 5 * slots, late)


def test_the_model_finds_a_slot_that_changes_its_group():
    for slots, groups in ((4, 1), (5, 1), (4, 2), (10, 2)):
        every(slots, groups)
    for slots in (9, 11):
        with pytest.raises(Early):
            every(slots, 2)


@pytest.mark.skipif(not shutil.which(os.environ.get("CXX") or "g++"), reason="no C++ compiler")
def test_the_ring_of_the_kernel(tmp_path):
    src = tmp_path / "ring.cpp"
    src.write_text('#include <cstdio>\n#include "i8_ring.h"\n'
                   "template <int NG> void say() { using F = os2i8::Few<NG>; "
                   'printf("%d %d %zu\\n", F::stages, F::groups, F::smem); }\n'
                   "int main() { say<1>(); say<2>(); say<4>(); say<8>(); }\n")
    exe = tmp_path / "ring"
    subprocess.run([os.environ.get("CXX") or "g++", "-std=c++17", "-I",
                    os.path.join(ROOT, "rns_emulated_fp64_gb300", "csrc"), str(src), "-o", str(exe)], check=True)
    rings = [[int(x) for x in line.split()] for line in subprocess.run([str(exe)], capture_output=True, text=True,
                                                                       check=True).stdout.splitlines()]
    assert len(rings) == 4
    for slots, groups, smem in rings:
        assert smem <= 227 * 1024
        every(slots, groups)


def follow_widening(raw, slots, groups, total, late_copy, late_mma):
    """The two rings of the product of more tokens: `raw` slots of 8-bit weights, which
    the groups in turn widen into `slots` others, which the MMAs read in order."""
    rfull, rempty, full, empty = [0] * raw, [0] * raw, [0] * slots, [0] * slots
    issued, landed, mma, done = 0, set(), 0, 0
    at, taken = [0] * groups, [False] * groups
    passes = lambda have, phase: have % 2 != phase % 2  # noqa: E731

    def advance(copy, held):
        nonlocal issued, mma, done
        moved = False
        if issued < total and (issued < raw or passes(rempty[issued % raw], issued // raw - 1)):
            issued += 1
            moved = True
        for i in range(issued):
            if i not in landed and i != copy:
                landed.add(i)
                rfull[i % raw] += 1
                moved = True
        for g in range(groups):
            j = at[g]
            if j >= total:
                continue
            if j % groups != g:
                at[g] += 1
                moved = True
            elif not taken[g] and passes(rfull[j % raw], j // raw):
                if j not in landed:
                    raise Early
                rempty[j % raw] += 1
                taken[g] = moved = True
            elif taken[g] and (j < slots or passes(empty[j % slots], j // slots - 1)):
                if j >= slots and done < j - slots + 1:
                    raise Early
                full[j % slots] += 1
                at[g], taken[g] = j + 1, False
                moved = True
        if mma < total and passes(full[mma % slots], mma // slots):
            mma += 1
            moved = True
        if done < mma and done != held:
            empty[done % slots] += 1
            done += 1
            moved = True
        return moved

    for hold in ((late_copy, late_mma), (None, late_mma), (None, None)):
        while advance(*hold):
            pass
    assert done == total and min(at) == total


def test_two_groups_that_widen_in_turn():
    def every(raw, slots, groups):
        for late in range(4 * raw):
            for held in [None] + list(range(0, 4 * raw, 3)):
                follow_widening(raw, slots, groups, 6 * raw, late, held)

    for raw in (5, 6, 7):                     # the kernel's: 6 for 64 tokens a tile, 5 for 128
        every(raw, 3, 2)
    every(4, 3, 1)
    with pytest.raises(Early):
        every(3, 3, 2)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 8, 9, 16])
@pytest.mark.parametrize("k", [2048, 5000])
def test_streams_longer_than_the_ring(m, k):
    """Tiles of many more stages than the ring has slots, with unit scales and sums that FP32
    holds: exact, every time."""
    import torch
    import rns_emulated_fp64_gb300 as os2
    g = torch.Generator(device="cuda")
    g.manual_seed(m + k)
    q = torch.randint(-15, 16, (m, k), generator=g, device="cuda").to(torch.int8)
    w = torch.randint(-128, 128, (32000, k), generator=g, device="cuda").to(torch.int8)
    one = torch.ones(32000, device="cuda")
    want = (q.double() @ w.double().t()).float()
    for _ in range(20):
        assert torch.equal(os2.i8gemm(q, one[:m], w, one, out_dtype=torch.float32), want)
    assert os2.get_status() == 0
