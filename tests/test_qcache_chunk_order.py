"""Orders in the attention of chunks that no result shows for sure: stores to TMEM are asynchronous even towards later loads
of the same thread, and a wait for loads does not order them. (The source is read.)"""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "random_access_kv_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body_of(text, start):
    """From `start` on, what its first pair of braces encloses."""
    at = text.index("{", text.index(start))
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == "{") - (text[i] == "}")
        if depth == 0:
            return text[at:i + 1]
    raise AssertionError(start)


def test_rescaled_sums_are_there_before_they_are_rescaled_again():
    # once where a reference moves ahead of need, and again in the same tile where another row's has to
    body = body_of(source("qc_chunk_tc.cuh"), "auto rescale")
    assert body.index("tmem_ld32_nowait") < body.index("tmem_wait_ld") < body.index("tmem_st32") < body.index("tmem_wait_st")
    assert body.rstrip("} \n").endswith("tmem_wait_st();")


def test_weights_are_there_before_their_barrier():
    text = source("qc_chunk_tc.cuh")
    for found in re.finditer(r"arrive_first\(&bar\.p_ready\[rt\]\[half\]\)", text):
        before = text[:found.start()]
        assert before.rindex("tmem_wait_st") > before.rindex("put(s_col")
