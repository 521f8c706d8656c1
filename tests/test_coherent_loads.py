"""Loads of what the kernel before on the stream may have written.  Kernels start while that one still runs and wait for it
(griddepcontrol.wait), so these loads must be ordinary ones: ld.global.nc, __ldg and const __restrict__ promise the
compiler and the hardware memory that is read-only for the kernel's whole life.  Read off the sources."""
import os
import re

import pytest

from fp4_compressed_sparse_02_gb300 import build

NC = re.compile(r"__ldg\s*\(|ld\.global\.nc|\bldg_(stream|gather)_v\d\(|const [\w ]+\*\s*__restrict__")


def lines(name):
    with open(os.path.join(build.CSRC, name)) as f:
        for n, line in enumerate(f, 1):
            yield n, line.split("//")[0]


@pytest.mark.parametrize("name", ["paged.cu", "kv8.cuh", "kv8_attn.cuh", "kv8_attn.cu", "kv8_tile.cu"])
def test_the_paged_8_bit_cache_is_read_coherently(name):
    """A step's plan, append, selection and attention follow one another: each reads the tables, summaries, scales and bytes
    that the ones before it write."""
    assert [(n, t.strip()) for n, t in lines(name) if NC.search(t)] == []


@pytest.mark.parametrize("name", ["common.cuh", "compress.cu", "proj_tc.cu", "index.cu", "score_tc.cu", "attn.cu"])
def test_what_a_plan_writes_is_read_coherently(name):
    """csa2_page_plan's table, sequences, positions and lengths go into the compressor, the indexer and the attention."""
    table = r"(?:\w+\.)*(?:page_table|seq|entry|pos|tok_pos|seq_of|n_vis)\b"
    bad = re.compile(rf"__ldg\(\s*{table}|const (?:int|int32_t)\*\s*__restrict__\s*(?:page_table|seq|entry|pos|tok_pos|seq_of|n_vis)\b")
    assert [(n, t.strip()) for n, t in lines(name) if bad.search(t)] == []
