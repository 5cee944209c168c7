"""What the chunked attention kernel's mask becomes in the compiler's hands.

Scores lie in the matrix instruction's vectors. A hidden one set under a branch
(with a condition of several parts, `a && (b || c)`) went wrong behind the
optimizer: the block that sets element 0 came out empty, its store moved ahead
of a copy that undid it, and tokens 0 and 4 of a tile stayed visible. A select
has no such block. (No GPU is touched by this test.)"""
import os
import re
import subprocess

from quantized_decode_mat_amd import build


def test_hidden_scores_are_selected_not_branched_to(tmp_path):
    out = tmp_path / "prefill.ll"
    src = os.path.join(build.CSRC, "attn_prefill.hip")
    subprocess.run([build.HIPCC, "-x", "hip", *build.FLAGS, "--cuda-device-only", "-emit-llvm", "-S", src, "-o", str(out)],
                   check=True, capture_output=True)
    ir = out.read_text()
    minus_infinity = "0xFFF0000000000000"
    kernels = len(re.findall(r"^define .*attn_prefill_kernel", ir, re.M))
    assert kernels >= 40
    assert not re.findall(r"insertelement <16 x float> .*float " + minus_infinity, ir)
    # 32 scores of a lane in every kernel
    assert len(re.findall(r"select (?:contract )?i1 %\S+, float (?:%\S+, float )?" + minus_infinity, ir)) >= 32 * kernels
