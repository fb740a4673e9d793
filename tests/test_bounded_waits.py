"""Every wait in the kernels has a limit but the named barriers, which count
the warps that meet at them.  So a warp whose bounded wait gave up must not
leave a loop of named barriers alone: the other warps would wait for it for
good.  Read from the sources, without a GPU: the order of a loop's barriers
and bounded waits, and what a give-up does, run through a model of the
barriers' counts."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "lora_fine_tuning_qlora_b200", "csrc")


def _with_barriers():
    names = sorted(n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh")))
    return [n for n in names if n != "tile_epilogue.cuh" and "named_bar_sync(" in open(os.path.join(CSRC, n)).read()]


SOURCES = _with_barriers()


def plain_source(text):
    """Comments blanked out."""
    text = re.sub(r"//[^\n]*", "", text)
    return re.sub(r"/\*.*?\*/", "", text, flags=re.S)


def matching(text, at, pair):
    """Index behind the bracket that closes the one at `at`."""
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == pair[0]) - (text[i] == pair[1])
        if depth == 0:
            return i + 1
    raise AssertionError("unbalanced %s" % pair)


def loops(text):
    """(start, end) of the bodies of all braced for and while loops."""
    found = []
    for m in re.finditer(r"\b(for|while)\s*\(", text):
        end = matching(text, m.end() - 1, "()")
        body = re.match(r"\s*\{", text[end:])
        if body:
            start = end + body.end() - 1
            found.append((start, matching(text, start, "{}")))
    return found


def barrier_loops(text):
    """Bodies of the loops that hold named barriers, less their inner loops."""
    every = loops(text)
    for start, end in every:
        inner = [(a, b) for a, b in every if start < a and b < end]
        body = list(text[start:end])
        for a, b in inner:
            body[a - start:b - start] = " " * (b - a)
        body = "".join(body)
        if "named_bar_sync(" in body:
            yield body


def events(body):
    """The loop's steps in order: "bar", "wait" (a bounded wait, here or in an
    inner loop whose result is tested here), "leave" and "skip" (what a give-up
    does where it is tested), "together" (all warps leave by a shared flag)."""
    words = {r"named_bar_sync\(": "bar", r"mbar_wait(?:_cluster)?\(": "wait", r"if \(!ok\) break;": "leave",
             r"if \(!ok\) continue;": "skip", r"if \(abort_flag\[\w+\]\) break;": "together"}
    at = [(m.start(), what) for pattern, what in words.items() for m in re.finditer(pattern, body)]
    return [what for _, what in sorted(at)]


def stuck(steps, warps=4, rounds=3):
    """Whether some single warp's give-up leaves others at a barrier."""
    if "together" in steps:
        return False
    tests = [i for i, s in enumerate(steps) if s in ("leave", "skip")]
    for gives_up in [(r, i) for r in range(rounds) for i in tests]:
        arrived = [0] * warps
        for w in range(warps):
            dead = False
            for r in range(rounds):
                for i, step in enumerate(steps):
                    if step == "bar":
                        arrived[w] += 1
                    elif step in ("leave", "skip") and (dead or (w == 0 and (r, i) == gives_up)):
                        dead = True
                        break
                if dead and step == "leave":
                    break
        if len(set(arrived)) > 1:
            return True
    return False


def test_the_model():
    assert stuck(["bar", "bar", "wait", "leave"])
    assert not stuck(["bar", "bar", "wait", "skip"])
    assert not stuck(["bar", "bar", "wait", "skip", "skip"])
    assert stuck(["bar", "wait", "skip", "bar"])  # a barrier behind the skip
    assert not stuck(["wait", "bar", "together", "leave", "bar"])


@pytest.mark.parametrize("name", SOURCES)
def test_a_give_up_leaves_no_warp_at_a_named_barrier(name):
    with open(os.path.join(CSRC, name)) as f:
        bodies = list(barrier_loops(plain_source(f.read())))
    assert bodies or name == "k4_rank_q.cu"  # (its barriers stand in no loop)
    for body in bodies:
        steps = events(body)
        assert steps and not stuck(steps), (name, steps)
