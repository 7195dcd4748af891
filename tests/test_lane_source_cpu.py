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
    kernel = body(text, r"sort_kernel\(const")
    assert 0 <= kernel.find("cluster_arrive()") < kernel.index("sort_cluster(")
    sort = body(text, r"void sort_cluster\(")
    calls = [m.start() for m in re.finditer(r"sort_bases\(", sort)]
    assert len(calls) == 2
    for at in calls:
        assert re.search(r"await_peers\(\);\s*$", sort[:at])
    assert "cluster_wait()" in body(sort, r"auto await_peers = ")


def test_rows_near_the_most_tokens_stay_in_range():
    """The launch that finds the head's rows handles up to 2^31 - 1025 tokens in
    at most 256 stretches of a multiple of 32, and zeroes rows from behind the
    last that counts on: neither index may wrap.  (The sums of the signed form
    pass 2^31, which this shows; the kernel's own form is asserted where it
    stands.)"""
    tokens = 2 ** 31 - 1025
    per = -(-(-(-tokens // 256)) // 32) * 32
    last = -(-tokens // per) - 1
    assert last * per < tokens and last * per + per > 2 ** 31 - 1 >= tokens
    assert tokens - 1 + last * 32 + 31 > 2 ** 31 - 1
    kernel = body(source("head_loss.cu"), r"head_rows_kernel\(const")
    assert "t1 = rows_end(blockIdx.x, per, A.tokens)" in kernel
    assert re.search(r"for \(unsigned r = all \+ ", kernel)


def test_workspaces_for_more_tokens_do_for_fewer():
    """A program may size a workspace once, for its longest batch."""
    lib = mo.lib()
    counts = [*range(0, 70), 1000, 4095, 4096, 4097, 4100, 5000, 8191, 8192, 8193, 16383, 16384, 16385, 100_000]
    for dim in (1, 8, 256, 333, 4096):
        sizes = [lib.muon_embedding_backward_workspace(n, 1000, dim) for n in counts]
        assert sizes == sorted(sizes)
        sizes = [lib.muon_layer_norm_backward_workspace(n, dim) for n in counts]
        assert sizes == sorted(sizes)
