"""The barriers between the roles of a backward tile, on the CPU: every order in
which producer, MMA issuer, tensor core and softmax groups can take their steps.

An mbarrier wait names only the parity of its phase.  It is right when, whenever a
role tests it, the phase waited for is the current or the last completed one: one
phase earlier it would pass too soon, one later it would wait for good.

The model follows csrc/bwd_tc.cuh for one tile of several blocks:
  producer   block n into slot n % N1 once the slot's last use was released
  MMA        S_0 .. S_{ST-1}; then for n = 0, 1, ..: wait P_n, S_{n+ST}
             (S_n waits for Y1_n, and completes in issue order, later)
  softmax    group n % ST: wait Y1_n (its note), wait S_n, give P_n
and the release of a slot: with out1 (dK, dQ) when out1_n has completed, which
follows dS_n; without it (dV tiles) when S_n has, and the group of block n has
seen the slot full."""
import re
from pathlib import Path

import pytest

SOURCE = Path(__file__).resolve().parents[1] / "scaled_dot_product_13_b200" / "csrc" / "bwd_tc.cuh"


def explore(N1, ST, out1, seen_before_release, blocks):
    """Mistaken waits over all interleavings: a set of words, empty when sound."""
    wrong = set()
    # filled, started, completed S, out1 done; per softmax group its block and step
    start = (0, 0, 0, 0, tuple((k, 0) for k in range(ST)))
    seen, todo = {start}, [start]
    while todo:
        state = todo.pop()
        filled, started, done, outs, groups = state

        def gave_p(n):  # P_n (and then dS_n) of the group of block n
            at, step = groups[n % ST]
            return at > n

        def noted(n):  # the group of block n has seen its slot full
            at, step = groups[n % ST]
            return at > n or (at == n and step >= 1)

        def phases(slot):  # completed phases of y1_full[slot]
            return (filled - slot + N1 - 1) // N1 if filled > slot else 0

        nxt = []
        if filled < blocks:
            old = filled - N1
            free = old < 0 or (old < outs if out1 else old < done and (noted(old) or not seen_before_release))
            if free:
                nxt.append((filled + 1, started, done, outs, groups))
        if started < blocks and started < filled and (started < ST or gave_p(started - ST)):
            nxt.append((filled, started + 1, done, outs, groups))
        if done < started:
            nxt.append((filled, started, done + 1, outs, groups))
        if out1 and outs < done and gave_p(outs) and (outs + ST < started or outs + ST >= blocks):
            nxt.append((filled, started, done, outs + 1, groups))
        for k, (n, step) in enumerate(groups):
            if n >= blocks:
                continue
            go = None
            if step == 0:
                have, want = phases(n % N1), n // N1
                passes = have % 2 != want % 2  # what the parity says
                if passes and have <= want:
                    wrong.add("passed before its phase")
                if have > want + 1:
                    wrong.add("phase missed")
                if passes:
                    go = (n, 1)
            elif n < done:
                go = (n + ST, 0)
            if go:
                nxt.append((filled, started, done, outs, groups[:k] + (go,) + groups[k + 1:]))
        for s in nxt:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return wrong


def roles():
    """(N1, ST, OUT1) of every tile that the library has."""
    found = re.findall(r"BwdTcRole<\d+, \d+, \d+, (\d+), (\d+), \d+, (?:true|false), (true|false),", SOURCE.read_text())
    assert len(found) >= 17
    return sorted({(int(n1), int(st), out1 == "true") for st, n1, out1 in found})


@pytest.mark.parametrize("N1,ST,out1", roles())
def test_every_wait_names_its_phase(N1, ST, out1):
    assert explore(N1, ST, out1, True, 4 * N1 + 3) == set()


def test_a_slot_released_by_the_scores_alone_loses_a_phase():
    """What the model says of a release that does not wait for the softmax group."""
    assert explore(3, 2, False, False, 15) == {"phase missed"}


def test_the_release_counts_the_softmax_warps():
    text = SOURCE.read_text()
    assert "mbar_init(&y1_empty[s], 1 + (OUT1 ? 0 : kBwdTcSoftmaxWarps / ST));" in text
    assert re.search(r"if constexpr \(!OUT1\) \{\s+__syncwarp\(\);\s+if \(lane == 0\) mbar_arrive\(&y1_empty\[slot\]\);", text)


def test_no_read_only_loads_of_what_the_grid_before_writes():
    """bwd_tc_kernel starts while bwd_rows_kernel may still write the row terms and
    norms: a non-coherent load of them may be moved above the wait for it."""
    for name in ("bwd_tc.cuh", "bwd_params.cuh"):
        text = (SOURCE.parent / name).read_text()
        kernel = text.split("bwd_join_kernel")[0]  # the join is an ordinary launch
        assert "__ldg" not in kernel and ".nc" not in kernel, name
