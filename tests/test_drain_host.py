"""No TMA load may be on its way into a CTA's shared memory when the CTA ends: the next CTA on
that SM may own the memory by then.  Whether one still is after a wait ran out depends on when
the other warps give up, which no run shows for sure and none may try on the GPU, so the kernels'
source is read here (CPU): a loader that alone arms its barriers waits for its last loads whatever
became of the others, and one that shares them leaves it to the CTA's end, when every warp has
stopped and the abort flag is final."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dynamic_sparse_attention_build_b200", "csrc")


def source(name):
    """The file without comments."""
    text = open(os.path.join(CSRC, name), encoding="utf-8").read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def conditions_of(text, at):
    """The heads of the blocks that hold position `at`, innermost first, up to the function's own."""
    heads, depth = [], 0
    for i in range(at - 1, -1, -1):
        if text[i] == "}":
            depth += 1
        elif text[i] == "{":
            if depth:
                depth -= 1
                continue
            start = max(text.rfind(c, 0, i) for c in ";{}")
            heads.append(" ".join(text[start + 1:i].split()))
    return heads


def statement(text, at):
    return " ".join(text[max(text.rfind(c, 0, at) for c in "{};") + 1:at].split())


def test_packed_prefill_waits_for_its_last_loads():
    text = source("dsa_pack.cu")
    at = text.index("serve_drain(&bars[L::QFULL]")
    assert "serve_drain(&bars[L::FULL" in text[at:at + 400]
    assert not any("abort" in c for c in conditions_of(text, at)[:2] + [statement(text, at)])


def test_vs_estimate_waits_for_its_last_loads():
    text = source("dsa_index.cu")
    at = text.index("mbar_drain(&bars[VB_QFULL]")
    assert "mbar_drain(&bars[VB_KFULL" in text[at:at + 200]
    assert conditions_of(text, at)[:2] == ["if (lane == 0)", "if (warp == 0)"] and statement(text, at) == ""


def test_sparse_attention_waits_for_its_last_loads_when_every_warp_has_stopped():
    """The decoders arm the same barriers for column tiles, so a parity only tells when nobody goes on."""
    text = source("dsa_attn.cu")
    body = text[text.index("sparse_attn_kernel(const __grid_constant__"):text.index("\nconstexpr int kSchedSlots")]
    calls = [m.start() for m in re.finditer(r"drain_loads\(", body)]
    assert len(calls) == 1 and calls[0] > body.rindex("__syncthreads();")
    assert conditions_of(body, calls[0])[0].startswith("sparse_attn_kernel(") or "abort_flag" in conditions_of(body, calls[0])[0]
    for name in ("q_kc", "pk[0]", "pk[1]", "pv[0]", "pv[1]"):  # the loader leaves what it has issued, on every way out
        assert re.search(r"misc\[\d+\] = " + re.escape(name) + ";", body), name
