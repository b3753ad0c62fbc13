"""Sizes and numbers behind the prompt and 4-bit cache calls that need no GPU."""
import subprocess

import pytest


@pytest.fixture(scope="module")
def lib():
    from quantised_gemv_norm_gb300 import build, dq

    build.build()
    return dq.load()


def test_decode_scratch_goes_by_the_query_heads(lib):
    size = lib.dq_attention_decode_kv4_workspace_bytes
    one = size(5, 3, 3, 100000)
    assert one > 0
    for group in range(2, 9):
        assert size(5, 3 * group, 3, 100000) == group * one


@pytest.mark.parametrize("n_seq,n_q,n_kv,max_keys", [
    (2**31 - 1, 2**31 - 1, 2**31 - 1, 2**30), (2**31 - 1, 8, 1, 4096), (4, 9, 1, 4096), (4, 10, 4, 4096), (1, 8, 8, 2**30 + 1),
    (1, 1 << 17, 1 << 17, 4096),
])
def test_decode_scratch_is_zero_for_counts_that_the_call_refuses(lib, n_seq, n_q, n_kv, max_keys):
    assert lib.dq_attention_decode_kv4_workspace_bytes(n_seq, n_q, n_kv, max_keys) == 0


DIVISION = r"""
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>
int main(void) {
    unsigned long bad = 0, n = 0;
    for (uint32_t e = 126; e <= 130; ++e)      /* five binades: the quotient's exponent steps inside each */
        for (uint32_t m = 0; m < 1u << 23; ++m, ++n) {
            uint32_t bits = e << 23 | m;
            float x, part;
            memcpy(&x, &bits, 4);
            part = x * (1.f / 15.f);
            bad += fmaf(fmaf(-15.f, part, x), 1.f / 15.f, part) != x / 15.f;
        }
    printf("%lu %lu\n", bad, n);
    return 0;
}
"""


def test_the_stores_division_by_15_is_the_rounded_quotient(tmp_path):
    # the store's three steps against IEEE division, for every mantissa (an exponent only scales them while nothing
    # underflows, and ranges that small give d = 0 either way)
    src, exe = tmp_path / "division.c", tmp_path / "division"
    src.write_text(DIVISION)
    subprocess.run(["gcc", "-O2", "-std=c11", "-ffp-contract=off", str(src), "-o", str(exe), "-lm"], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    assert out.split() == ["0", str(5 << 23)]
