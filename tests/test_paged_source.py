"""Properties of the paged kernels that a run cannot show, read from their source."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "full_gqa_decode_gb300", "csrc")


def source(name):
    return re.sub(r"//.*", "", open(os.path.join(CSRC, name)).read())


def test_waits_for_a_peer_ctas_arrivals_acquire_at_cluster_scope():
    """The chunk kernel's CTAs arrive on each other's barriers with release.cluster; an acquire at the default scope, one
    CTA, does not synchronise with that."""
    text = source("paged_chunk.cu")
    assert "mbarrier.arrive.release.cluster.shared::cluster" in text
    waits = re.findall(r"mbarrier\.(?:try_wait|test_wait)[\w.:]*", text)
    assert waits and all(".acquire.cluster" in w for w in waits), waits
