"""What the library's sources may not hold (CPU only)."""
import glob
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_copy_or_commit_reaches_another_cta():
    """Every rank of a multi-process run loads this library, so its copies and tensor-core
    commits stay within one CTA: no multicast to a cluster."""
    sources = [p for d in ("paged_kv_cache_301_gb300/csrc", "include")
               for p in glob.glob(os.path.join(ROOT, d, "*"))]
    assert len(sources) > 15
    for path in sources:
        with open(path) as f:
            assert ".multicast" not in f.read(), path
