"""CPU checks of the kernels that start while the one before them on the stream ends (cudaLaunchAttributeProgrammaticStream-
Serialization). What the kernel before them may have written is no constant of theirs, and a stale value cannot be
provoked at will, so the source is checked: they read nothing by the loads for constants."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "split_kv_decode_bsr_gb300", "csrc")
CONSTANT = re.compile(r"__ldg\b|ld\.global\.(?:\w+\.)*nc\b|__restrict__")


def _source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name), encoding="utf-8").read())


def test_what_starts_early_reads_no_constants():
    for name in sorted(os.listdir(CSRC)):
        text = _source(name)
        if "ProgrammaticStreamSerialization" not in text:
            continue
        assert name in ("norm_rope.cu", "chunk.cu")
        for m in CONSTANT.finditer(text):
            # in a kernel that is launched in the common way, or in the branch of one that is
            before = text[:m.start()]
            kernel = re.findall(r"\b(\w+_kernel)\(|bool (\w+)\(|int32_t (list_word)\(", before)[-1]
            assert name == "chunk.cu" and "".join(kernel) in ("chunk_merge_kernel", "list_word"), (name, m.group(), kernel)
            assert "".join(kernel) != "list_word" or re.search(r"else return\s*$", before)
    merge = re.search(r"(\S+)\s*chunk_merge_kernel<D, CAP><<<", _source("chunk.cu"))
    assert merge, "launched in the common way"
