"""What the AdamW lane's device code must hold to and no run can be trusted to
show (no GPU): read from the sources."""
import os
import re

import matrix_orthogonalizing_optimizer_step_b200 as mo

CSRC = os.path.join(os.path.dirname(mo.__file__), "csrc")


def source(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(text, signature):
    """The braces' contents of the function whose head matches `signature`."""
    start = re.search(signature, text).end()
    start = text.index("{", start)
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i + 1]
    raise AssertionError("unbalanced braces")


def test_sorting_cluster_waits_for_its_peers_before_it_writes_to_them():
    """A CTA may touch another's shared memory only once the whole cluster is
    known to run.  The sort's one remote write is in sort_bases; every thread
    of the cluster arrives before it sorts, and each call of sort_bases has the
    wait directly before it."""
    text = source("embedding.cu")
    assert text.count("st.shared::cluster") == body(text, r"void sort_bases\(").count("st.shared::cluster") == 1
    kernel = body(text, r"sort_and_fill_kernel\(const")
    assert 0 <= kernel.find("cluster_arrive()") < kernel.index("sort_cluster(")
    sort = body(text, r"void sort_cluster\(")
    calls = [m.start() for m in re.finditer(r"sort_bases\(", sort)]
    assert len(calls) == 2
    for at in calls:
        assert re.search(r"await_peers\(\);\s*$", sort[:at])
    assert "cluster_wait()" in body(sort, r"auto await_peers = ")
