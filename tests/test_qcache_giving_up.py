"""A bounded wait of the tensor-core attention kernel that gives up is told once the kernel ends, whatever waits come after
it: the outcome of a wait is never assigned over an earlier one, and the sums in TMEM are not touched after a
failed wait for them. (No GPU is made to run into it: the source is read.)"""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "random_access_kv_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_a_waits_outcome_is_kept():
    for name in ("qc_attend_tc.cu", "qc_tc.cuh"):
        found = re.findall(r"(?<!bool )\bok = ([^;]*wait[^;]*);", source(name))
        assert found
        for right in found:
            assert right.startswith("ok && "), (name, right)


def test_sums_are_left_alone_after_a_failed_wait():
    text = source("qc_attend_tc.cu")
    body = text[text.index("auto rescale"):]
    body = body[:body.index("};")]
    assert re.search(r"ok = ok && warp_wait\([^;]*\);\s*if \(!ok\) return;", body)
    assert body.index("return") < body.index("tmem_ld32") < body.index("tmem_st32")
    assert re.search(r"if \(sums\) rescale\(by\);\s*if \(!ok\) break;", text)
