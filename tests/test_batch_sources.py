"""Rules that the batched operators' kernels have to keep and that a run cannot
show, because a compiler may or may not make up for a breach: read from the
sources (CPU only)."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "moe_decode_layer_persistent_gb300", "csrc")

ONE_LANE = r"if \([^;{}]*(?:lane == 0|lane_id\(\) == 0|elect_one\(\))[^;{}]*\)"
MEETS = r"__syncwarp\(|__syncthreads\(|\bwait_warp\(|__(?:any|all|ballot|shfl|reduce)\w*_sync\("
ALIGNED = r"\b(?:tmem_ld|tmem_st|tmem_alloc|tmem_dealloc|tmem_relinquish|reg_alloc|reg_dealloc)\w*(?:<\d+>)?\("


def body(source, name):
    """The braces behind the definition of `name`, without comments."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, source)).read())
    at = re.search(r"\b%s\([^;{}]*\)\s*\{" % name, text).end()
    depth, end = 1, at
    while depth:
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        end += 1
    return text[at:end - 1]


def breaches(code):
    """Instructions for whole warps that follow a branch of one lane without
    anything in between that brings the warp together.  The code is gone
    through twice, as its loops do; what stands behind a short-circuit may not
    be reached and brings nothing together."""
    code += code
    found, apart = [], None
    for m in re.finditer("(?P<one>%s)|(?P<meets>%s)|(?P<aligned>%s)" % (ONE_LANE, MEETS, ALIGNED), code):
        if m.lastgroup == "one":
            apart = m.group()
        elif m.lastgroup == "meets":
            start = max(code.rfind(c, 0, m.start()) for c in ";{}")
            if not re.search(r"\|\||&&|\?", code[start + 1:m.start()]):
                apart = None
        elif apart:
            found.append((apart, m.group()))
    return found


@pytest.mark.parametrize("name", ["softmax", "produce", "issue_mmas"])
def test_warps_meet_before_instructions_for_whole_warps(name):
    assert breaches(body("prefix_attn.cu", name)) == []


def test_the_reading_sees_a_breach():
    bad = "if (lane == 0) arrive(); look = j == 0 || __any_sync(m, x); tmem_ld32(a, b);"
    assert len(breaches(bad)) == 2
    assert breaches(bad.replace("look", "__syncwarp(); look")) == []
    assert breaches("if (elect_one()) { commit(); } reg_alloc<168>();") != []
