"""Launches that start while the launch before them still runs (launch_dependent) read nothing of it,
nor of anything before it, until they have waited, or until an acquire has shown that what was
written before the call is there; and what they read behind an acquire does not go through the
read-only cache.  Checked in the kernels' text: where a wait is missing the GPU mostly gives the
right answer."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_attention_52_gb300", "csrc")
FILES = ("attn_cache.cu", "attn_cache_prompt.cu", "attn_cache_rope.cu", "attn_rope.cu")
# what reads global memory through the parameters, or calls what does
READS = re.compile(r"__ld|ldcg|\bp\.(c|items|part|stat|border|q|positions|x|dy)\b\s*[.\[+]|find_share|prefix_share|prompt_share"
                   r"|cache_seq|query_count|group_(of|len|begin|end|start|tile)|load_weight|append_page|check_len")


def kernels():
    out = []
    for f in FILES:
        text = open(os.path.join(CSRC, f)).read()
        text = re.sub(r"//[^\n]*", "", text)
        for m in re.finditer(r"__global__[^;{]*?\b(\w+_kernel)\(", text):
            out.append((f, m.group(1), text[m.start():text.index("\n}\n", m.start())]))
    return out


KERNELS = kernels()


def test_the_kernels_are_found():
    assert {k for _, k, _ in KERNELS} == {
        "cache_append_kernel", "cache_decode_kernel", "cache_join_kernel", "cache_merge_kernel", "cache_prompt_kernel",
        "cache_append_rope_kernel", "rope_kernel", "rope_norm_bwd_kernel", "rope_dw_kernel"}


@pytest.mark.parametrize("file,name,body", KERNELS, ids=[k for _, k, _ in KERNELS])
def test_nothing_is_read_before_the_wait(file, name, body):
    lines = body.split("\n")
    at = next(i for i, x in enumerate(lines) if "pdl_wait();" in x)
    assert re.fullmatch(r"(if \((PART != kRest \|\| )?!opened\(p\)\) )?pdl_wait\(\);", lines[at].strip()), lines[at]
    before = "\n".join(lines[:at])
    assert not READS.search(before[before.index("{"):]), READS.search(before)


@pytest.mark.parametrize("file,name,body", [k for k in KERNELS if "opened(p)" in k[2]],
                         ids=[k for _, k, b in KERNELS if "opened(p)" in b])
def test_reads_behind_an_acquire_are_coherent(file, name, body):
    assert "__ldg(" not in body and "__ldcs(" not in body
    assert body.count("pdl_wait();") >= 2  # and the launch before it has ended before this one does
    ops = open(os.path.join(CSRC, "cache_ops.cuh")).read()
    assert re.search(r"PART == kRest \? __ldcg\(at\) : __ldg\(at\)", ops)
    assert ops.count("__ldg(") == 1


def test_the_launch_of_the_prefixes_opens_what_it_has_waited_for():
    body = next(b for _, k, b in KERNELS if k == "cache_prompt_kernel")
    assert 0 < body.index("pdl_wait();") < body.index("open_rest(p);") < body.index("pdl_launch_dependents();")
    ops = open(os.path.join(CSRC, "cache_ops.cuh")).read()
    assert "st.release.gpu.global.u64" in ops and "ld.acquire.gpu.global.u64" in ops
