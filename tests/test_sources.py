"""What the library's sources may not contain, whatever else they do."""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(sum((glob.glob(os.path.join(ROOT, "mla_latent_cache_decode_gb300", "csrc", "*" + e)) for e in (".cu", ".cuh", ".h")), []))


def asm_texts(source):
    """The string literals of every asm statement, joined."""
    return ["".join(re.findall(r'"((?:[^"\\]|\\.)*)"', body.split('"::')[0])) for body in re.findall(r"asm\s*(?:volatile)?\s*\((.*?)\);", source, re.S)]


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_load_writes_into_several_blocks(path):
    """One library serves every rank of a run on several GPUs, and its entry points take addresses
    without asking whose memory they are: a bulk copy goes into the block's own shared memory only."""
    with open(path) as f:
        source = f.read()
    several = "multi" + "cast"
    assert not [t for t in asm_texts(source) if "cp.async.bulk" in t and several in t], path


def test_the_search_sees_asm_statements():
    text = 'asm volatile(\n "cp.async.bulk.a"\n ".b [%0];" ::"r"(x) : "memory");'
    assert asm_texts(text)[0].startswith("cp.async.bulk.a.b [%0];")
    assert sum(len(asm_texts(open(p).read())) for p in SOURCES) > 40


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_32_byte_stores(path):
    """In a function that two kernels call, not inlined, nvcc 13.0 wrote only the first element of
    such a store in one of them."""
    with open(path) as f:
        source = f.read()
    assert not re.search(r"st\.global\.v8|_32a\b", re.sub(r"//[^\n]*", "", source)), path
