"""The recorded captures under profiles/ (not gpu): a summary names the sources that it was taken of and their hash, and its
figures are withheld once one of them changes. So what an operator declares for itself stays out of the sources of
the others, whose captures it would void."""
import glob
import os
import re
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402

PKG = "compressed_decode_attention_equal_b200"
RECORDED = [p for p in sorted(glob.glob(os.path.join(ROOT, "profiles", "*_summary.md"))) if "source_sha256_16:" in open(p).read()]


def covered(path):
    note = re.search(r"\(`source_sha256_16`.*?\)", open(path).read(), re.S).group(0)
    return [f"{PKG}/{f}" for f in re.findall(r"`(csrc/[\w.]+)`", note)]


@pytest.mark.parametrize("path", RECORDED, ids=[os.path.basename(p) for p in RECORDED])
def test_a_summary_names_its_sources_and_their_hash(path):
    files = covered(path)
    assert files and all(os.path.exists(os.path.join(ROOT, f)) for f in files)
    assert re.search(r"^source_sha256_16: [0-9a-f]{16}$", open(path).read(), re.M)
    if "token_cache" not in path:   # the decode's, the coarsener's and the streaming append's captures
        for f in files:
            assert not re.search(r"exact-token cache|PagedArgs|AppendArgs|ReadTable|token_cache\.cuh", open(os.path.join(ROOT, f)).read()), f


def test_the_bench_reads_the_captures_of_these_files():
    for name, sources in (("decode_gqa7_32k_summary.md", bench.DECODE_SOURCES), ("coarsen_131k_summary.md", bench.COARSEN_SOURCES)):
        assert covered(os.path.join(ROOT, "profiles", name)) == sources
