"""The sizes of test_gpu_rope_forms.py against the rules that choose a form: a rule that moves shows here, before
those tests run the wrong form unnoticed. No GPU needed."""
import os
import re

from test_gpu_rope_forms import FEW_HEADS_ROWS, MANY_HEADS, MANY_ROWS, MANY_TOKENS, SMS

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_kv_cache_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"\s+", " ", f.read())


def test_the_sizes_follow_the_rules():
    assert f"constexpr int kTunedSms = {SMS};" in source("msa_host.h")
    rope = source("msa_rope.cu")
    at_once = int(re.search(r"constexpr int kThreads = (\d+); constexpr int kRowsAtOnce = kThreads / 16;", rope)[1]) // 16
    ctas = int(re.search(r"constexpr int kCtas = (\d+),", rope)[1])
    many = int(re.search(r"constexpr int kMany = (\d+) / sizeof\(In\);", rope)[1]) // 2 * at_once  # 16-bit rows a CTA
    assert "const int tokens = (kMany<In> * kRowsAtOnce + heads - 1) / heads; return tokens <= 16 && rows > " \
        "static_cast<int64_t>(kCtas * kRowsAtOnce) * msa_host::kTunedSms * (tokens <= 8 ? 1 : 8);" in rope
    assert many == 8 * MANY_HEADS
    assert "return 2 * n >= static_cast<int64_t>(3 * kRowsAtOnce) * msa_host::kTunedSms;" in rope
    assert MANY_ROWS == ctas * at_once * SMS + 1 and FEW_HEADS_ROWS == 8 * ctas * at_once * SMS + 1
    assert 2 * MANY_TOKENS == 3 * at_once * SMS
