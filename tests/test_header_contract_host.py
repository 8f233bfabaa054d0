"""What include/wf.h promises about results that no GPU test can produce."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _text(*path):
    with open(os.path.join(ROOT, *path)) as f:
        return f.read()


def test_a_timeout_leaves_the_outputs_undefined():
    """A call whose wait ran out may have written some rows, and its join reads parts that were never
    written: the header says so."""
    entry = re.search(r"WF_ERR_TIMEOUT = 6,\s*/\*(.*?)\*/", _text("include", "wf.h"), re.S).group(1)
    assert "undefined" in entry and "outputs" in entry and "lse" in entry


def test_a_warp_that_lost_its_wait_stops_its_whole_cta():
    """Few rows: the warps' results are joined only if every warp of the CTA has all of its keys."""
    code = _text("block_causal_streaming_b200", "csrc", "attn_fp8_few_kernel.cuh")
    body = code[code.index("wf_attn_fp8_few_kernel(const"):]
    vote, join = body.index("if (!__syncthreads_and(ok)) return;"), body.index("// ---- join the warps")
    assert vote < join and not re.search(r"if \(!ok\) return", body[join:])


def test_attention_states_its_floor_against_the_largest_value():
    """Small values beside large ones: the bound in the header is the one the GPU tests hold the kernels
    to (test_gpu_fp8_value_range.py), and names the largest visible value, not only the weights."""
    head = _text("include", "wf.h")
    text = head[head.index("wf_attn_forward_fp8_block -- "):head.index("int wf_attn_forward_fp8_block(")]
    text = re.sub(r"\s*\n \*\s*", " ", text)
    assert "largest visible value" in text
    assert "2^-8 |exact| + (2^-10 + 2^-18 L) sum p_j |v_j| + n 2^-36 V" in text
