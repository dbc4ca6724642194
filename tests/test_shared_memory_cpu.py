"""The kernels' hand-written shared-memory maps: the constants are read from the sources and no two things that are there
at the same time share a byte."""
import os
import re

import pytest

from kda_linear_attention_bounded_gb300 import build as kbuild


def constants(source, begin=None):
    """The integer constants of a source, in order; those of a part that begins with `begin` and ends with its namespace."""
    with open(os.path.join(kbuild.CSRC, source)) as f:
        text = f.read()
    text = re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))
    known = {"kD": 128}

    def take(part):
        for kind, body in re.findall(r"\b(constexpr (?:u?int(?:32_t)?)|enum) ?\{?([^;{}()]*=[^;{}]*?)\}?;", part):
            value = -1
            for item in body.split(","):
                name, _, expr = item.partition("=")
                try:
                    value = int(eval(expr.replace("/", "//"), {}, dict(known))) if expr else value + 1
                except (NameError, SyntaxError):   # (another source's, or none that is a number)
                    continue
                known[name.strip()] = value

    if begin is None:
        take(text)
        return known
    at = text.index(begin)
    end = re.compile(r"^}", re.M).search(text, at).start()
    take(text[:at])
    take(text[at:end])
    return known


F32 = 4
CASES = {
    # source, where the map stands, what it holds (name of the offset: bytes), and its end
    "gated delta rule, intra-chunk": ("kda_gdn_prefill.cu", "namespace in {", "SM_END", {
        "SM_NORM": 128 * F32, "SM_BETA": 64 * F32, "SM_BI": 64 * F32, "SM_BF": 64 * F32, "SM_UP": 64 * F32,
        "SM_POW": 64 * F32, "SM_BAR": 2 * 8, "SM_TMEM": 4, "SM_ABORT": 4, "SM_LONG": 16}),
    "gated delta rule, state pass": ("kda_gdn_prefill.cu", "namespace ch {", "SM_END", {
        "SM_BAR": "8 * kBarriers", "SM_TMEM": 4, "SM_ABORT": 4, "SM_SIG": 2 * 128 * F32, "SM_INV": 2 * 128 * F32}),
    "gated delta rule, state pass, tiles": ("kda_gdn_prefill.cu", "namespace ch {", "kSmemBytes", {
        "0": "2 * kStage", "OFF_ONE": 64 * 64 * 2, "OFF_K16": 64 * 128 * 2, "OFF_OUT": 64 * 128 * 2, "OFF_SMALL": "SM_END"}),
    "paged attention": ("kda_paged_attention.cu", None, "kSmemBytes", {
        "0": "kStages * kStageBytes", "OFF_INFO": "16 * kStages", "OFF_MASK": "8 * kStages", "OFF_ML": 4 * 16 * 2 * F32,
        "OFF_CML": 64 * 8, "OFF_SCAN": 8 * 8, "OFF_BAR": "8 * (2 * kStages + 1) + 4"}),
    "state pass": ("kda_chunk_chain.cu", None, "SM_END", {"SM_BAR": 6 * 8, "SM_TMEM": 4, "SM_ABORT": 4}),
    "state pass, values split": ("kda_chunk_chain.cu", "namespace vs {", "SM_END", {
        "SM_GAMMA": 3 * 128 * F32, "SM_BAR": 6 * 8, "SM_TMEM": 4, "SM_ABORT": 4}),
    "intra-chunk": ("kda_chunk_intra.cu", None, "SM_END", {
        "SM_NQ": 64 * F32, "SM_NK": 64 * F32, "SM_BETA": 64 * F32, "SM_H": 8 * 128 * F32, "SM_BAR": 3 * 8, "SM_TMEM": 4,
        "SM_ABORT": 4, "SM_BARU": 8, "SM_HALO": 3 * 3 * 64 * 4, "SM_VW": 128 * 4 * F32}),
    "one-kernel prefill": ("kda_prefill_fused.cu", None, "SM_END", {
        "SM_NQ": 3 * 64 * F32, "SM_NK": 64 * F32, "SM_BETA": 2 * 64 * F32, "SM_H": 8 * 128 * F32, "SM_GAMMA": 2 * 128 * F32,
        "SM_EM": 2 * 128 * F32, "SM_BAR": "8 * kNumBars", "SM_TMEM": 4, "SM_ABORT": 4}),
}


@pytest.mark.parametrize("name", CASES)
def test_nothing_overlaps(name):
    source, begin, end, things = CASES[name]
    known = constants(source, begin)
    value = lambda x: int(eval(str(x), {}, known))  # noqa: E731
    spans = sorted((value(at), value(at) + value(size), at) for at, size in things.items())
    for (_, stop, a), (start, _, b) in zip(spans, spans[1:]):
        assert stop <= start, (a, b)
    assert spans[-1][1] <= value(end)
