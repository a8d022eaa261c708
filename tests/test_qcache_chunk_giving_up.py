"""The attention of chunks where a bounded wait gives up: the launch that joins its parts follows all the same, and must
find lines of this call or empty ones, whatever the workspace held. (No GPU is made to run into it: the source is read, and the
join's walk over the lines is played through on the CPU with workspaces of any contents.)"""
import random
import re

import pytest

from test_qcache_chunk_order import body_of, source


def test_lines_are_emptied_before_anything_can_give_up():
    text = source("qc_chunk_tc.cuh")
    kernel = text[text.index("chunk_tc(const Chunk p"):]
    at = kernel.index("= {};", kernel.index("parts.lines["))
    # after the wait for the launch before, whose join may still read them; before the roles, which all that waits is in
    assert kernel.index("griddep_wait()") < at < kernel.index("cluster_sync()") < kernel.index("setmaxnreg")
    assert not re.search(r"(mbar_wait|warp_wait|warp_poll|poll)\(", kernel[:at])
    # and the lines that say something come after the last wait of the warp that writes them
    body = body_of(text, "bool produce_tiles(")
    assert body.rindex("warp_wait") < body.index("lines[0] = line[0]")


def test_the_join_checks_a_line_before_it_follows_it():
    body = body_of(source("qc_chunk.cu"), "chunk_join(const Chunk p")
    for name, limit in (("b", "p.n_seq"), ("kv", "p.g.heads"), ("run", "runs_of(p, s, parts.rows)")):
        check = re.search(r"line\.%s < 0 \|\| line\.%s >= %s" % (name, name, re.escape(limit)), body)
        assert check and body.index("return", check.end()) < min(m.start() for m in re.finditer(r"line\.%s\b" % name, body)
                                                                 if m.start() > check.end())


def test_a_waits_outcome_is_kept():
    # a failed wait ends its loop at once, or is never assigned over
    text = source("qc_chunk_tc.cuh")
    for found in re.finditer(r"(?<!bool )\bok = ([^;]*(?:wait|poll)[^;]*);", text):
        kept = found.group(1).startswith("ok && ")
        after = text[found.end():found.end() + 80]
        before = text[text.rindex("for (", 0, found.start()):found.start()]
        assert kept or re.match(r"\s*if \(!ok\) break;", after) or "; ok &&" in before, found.group(0)


HOLDS, OPENS, CLOSES = 1, 2, 4


def join(lines, units, n_seq, heads, runs, empty, checked):
    """What the join of every unit goes by: the jobs, and the parts added. lines: two a unit, what the workspace held; those of
    `empty` are emptied by the call."""
    at = [None if x in empty else line for x, line in enumerate(lines)]
    at = [(0, 0, 0, 0) if line is None else line for line in at]
    done = []
    for unit in range(units - 1):
        first = 2 * unit + 1
        if not at[first][3]:
            first -= 1
        b, kv, run, what = at[first]
        if not what & OPENS or what & CLOSES:
            continue
        if checked and not (0 <= b < n_seq and 0 <= kv < heads and 0 <= run < runs[b]):
            continue
        last = unit + 1
        while last < units - 1 and not at[2 * last][3] & CLOSES:
            last += 1
        done.append((b, kv, run))
        assert 2 * last < len(at)
    return done


def outside(done, n_seq, heads, runs):
    return [j for j in done if not (0 <= j[0] < n_seq and 0 <= j[1] < heads and 0 <= j[2] < runs[j[0]])]


def workspaces(seed, emptied):
    """Lines as a call leaves them that gave up in some units, over those of an earlier call with more of everything."""
    r = random.Random(seed)
    units, n_seq, heads = r.randint(2, 20), r.randint(1, 5), r.randint(1, 4)
    runs = [r.randint(0, 3) for _ in range(n_seq)]
    word = lambda: r.choice([r.randint(0, 8), r.randint(-2 ** 31, 2 ** 31 - 1), -1])  # noqa: E731
    lines = [(word(), word(), word(), r.choice([0, 1, 3, 5, 7, word()])) for _ in range(2 * units)]
    gave_up = set(range(2 * units)) if emptied else set()
    return lines, units, n_seq, heads, runs, gave_up


def test_joins_stay_within_the_call():
    for seed in range(500):
        lines, units, n_seq, heads, runs, empty = workspaces(seed, True)
        assert not join(lines, units, n_seq, heads, runs, empty, True)
        lines, units, n_seq, heads, runs, empty = workspaces(seed, False)
        assert not outside(join(lines, units, n_seq, heads, runs, empty, True), n_seq, heads, runs)


def test_unchecked_lines_of_another_call_are_found():
    with pytest.raises(AssertionError):
        for seed in range(500):
            lines, units, n_seq, heads, runs, empty = workspaces(seed, False)
            assert not outside(join(lines, units, n_seq, heads, runs, empty, False), n_seq, heads, runs)
